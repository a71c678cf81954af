"""Serve requests on a small hybrid model: gated-delta-rule layers with one full-attention
layer behind every three, random weights, prompts and one-token steps in the same pack.

    python examples/serve_hybrid.py [--requests 6] [--answer 24]

A step's pages, slots and positions are planned on the GPU once; every full-attention layer
then appends its keys and values to its paged 8-bit cache (rotating keys and queries on the
way) and attends over it; every linear layer reads and writes its states in its pool. The
projections are plain matrix products. Requests for whose rows there are no pages sit out the
step, in every layer, and are tried again in the next one.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import torch  # noqa: E402

from packed_linear_attention_gb300 import gdn  # noqa: E402

HIDDEN, DIM = 512, 128
LINEAR_K, LINEAR_V = 2, 4             # heads of a linear layer
QUERY, KV, ROTARY = 8, 2, 64          # heads of a full layer; rotated elements of a head
PAGE = 64


def _weight(rows, cols):
    return (torch.randn(rows, cols, device="cuda") * rows ** -0.5).bfloat16()


def _norm(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:])


def _pages_of(tokens):
    return -(-tokens // PAGE)


class Pages:
    """Page tables of `slots` requests and the stack of free pages: they serve every layer,
    since the layers' caches have the same pages. The host knows the lengths too, and so which
    requests a step has pages for."""

    def __init__(self, slots, num_pages, max_tokens):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.slots, self.num_pages, self.max_blocks = slots, num_pages, _pages_of(max_tokens)
        self.max_tokens = max_tokens
        self.table = torch.full((slots, self.max_blocks), -1, **i32)
        self.free = torch.arange(num_pages, **i32)
        self.count = torch.full((1,), num_pages, **i32)
        self.ctx = torch.zeros(slots, **i32)      # cached tokens of each slot's request
        self.kv_len = torch.zeros(slots, **i32)
        self.cu = torch.zeros(slots + 1, **i32)
        self.status = torch.zeros(1, **i32)
        self.length, self.left = [0] * slots, num_pages  # ctx and count, as the host has them

    def admit(self, new_len):
        """new_len without the requests that there are no pages for, in the plan's order."""
        taken, kept = 0, []
        for length, n in zip(self.length, new_len):
            if length + n > self.max_tokens:
                raise gdn.GdnError(gdn.GDN_ERR_INVALID_ARGUMENT, "serve: request too long")
            need = _pages_of(length + n) - _pages_of(length)
            fits = taken + need <= self.left
            taken += need if fits else 0
            kept.append(n if fits else 0)
        return kept

    def plan(self, handle, new_len):
        """Pages for new_len[slot] tokens of every slot (host list); the rows' positions/slots."""
        self.rows, self.longest, self.new = sum(new_len), max(new_len), new_len
        new = torch.tensor(new_len, dtype=torch.int32).cuda()
        self.positions = torch.empty(self.rows, dtype=torch.int32, device="cuda")
        self.places = torch.empty(self.rows, dtype=torch.int64, device="cuda")
        gdn.gdn_kv_plan(handle, PAGE, self.slots, self.rows, self.ctx, new, self.table,
                        self.max_blocks, self.num_pages, self.free, self.count, self.count,
                        self.cu, self.kv_len, self.positions, self.places, self.status)

    def advance(self):
        # kv_len is 0 for a request that the plan refused: it keeps its context
        self.ctx.copy_(torch.where(self.kv_len > 0, self.kv_len, self.ctx))
        for s, n in enumerate(self.new):
            self.left -= _pages_of(self.length[s] + n) - _pages_of(self.length[s])
            self.length[s] += n

    def release(self, handle, ended):
        flags = torch.zeros(self.slots, dtype=torch.int32)
        flags[ended] = 1
        flags = flags.cuda()
        gdn.gdn_kv_release(handle, PAGE, self.slots, self.ctx, flags, self.table,
                           self.max_blocks, self.num_pages, self.free, self.count, self.status)
        self.ctx *= 1 - flags
        for s in ended:
            self.left += _pages_of(self.length[s])
            self.length[s] = 0


class FullAttention:
    def __init__(self, pages):
        shape = (pages.num_pages, KV, PAGE, DIM)
        self.codes = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(shape[:2], device="cuda") for _ in range(2)]
        self.cache = gdn.make_kv_cache(*self.codes, *self.scales)
        self.rope = gdn.gdn_rope_init(DIM, ROTARY, [ROTARY // 2])
        self.cfg = gdn.make_attn_config(QUERY, scale=DIM ** -0.5)
        self.qkv, self.out = _weight(HIDDEN, (QUERY + 2 * KV) * DIM), _weight(QUERY * DIM, HIDDEN)

    def __call__(self, handle, pages, x):
        rows, width = pages.rows, (QUERY + 2 * KV) * DIM
        qkv = x @ self.qkv
        q, k, v = qkv.split([QUERY * DIM, KV * DIM, KV * DIM], dim=1)  # column ranges, not copies
        gdn.gdn_kv_append(handle, self.cache, gdn.GDN_BF16, rows, pages.places, k, width, v, width,
                          self.rope, pages.positions, rows, q, width, QUERY, q, width,
                          pages.status)
        o = torch.empty(rows, QUERY * DIM, dtype=torch.bfloat16, device="cuda")
        size = gdn.gdn_attn_workspace_size(self.cfg, self.cache, pages.slots, rows, pages.longest,
                                           pages.max_tokens)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        gdn.gdn_attn_paged(handle, self.cfg, self.cache, pages.slots, rows, pages.longest,
                           pages.max_tokens, pages.cu, pages.kv_len, pages.table,
                           pages.max_blocks, q, width, o, QUERY * DIM, None, work, size,
                           pages.status)
        return o @ self.out


class LinearAttention:
    def __init__(self, slots):
        self.slots = slots
        self.pool = torch.zeros(slots, LINEAR_V, DIM, DIM, device="cuda")
        self.cfg = gdn.make_config(LINEAR_K, LINEAR_V, DIM)
        self.q, self.k = _weight(HIDDEN, LINEAR_K * DIM), _weight(HIDDEN, LINEAR_K * DIM)
        self.v, self.out = _weight(HIDDEN, LINEAR_V * DIM), _weight(LINEAR_V * DIM, HIDDEN)
        self.gates = _weight(HIDDEN, 2 * LINEAR_V)

    def __call__(self, handle, cu, slots, fresh, x):
        a, beta = (x @ self.gates).float().chunk(2, dim=1)
        a = -torch.nn.functional.softplus(a).contiguous()
        o = torch.empty(x.shape[0], LINEAR_V * DIM, dtype=torch.bfloat16, device="cuda")
        size = gdn.gdn_prefill_workspace_size(self.cfg, cu)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        gdn.gdn_prefill_packed_pool(handle, self.cfg, cu, x @ self.q, x @ self.k, x @ self.v, a,
                                    beta.sigmoid().contiguous(), self.pool, self.slots, slots,
                                    fresh, None, None, o, None, work, size)
        return o @ self.out


class Server:
    """`slots` requests at a time. step() takes the new rows of some of them (a prompt or a
    single token each) and gives each one's last row back; a request without pages is left out
    of the step and of its results."""

    def __init__(self, slots=8, num_pages=128, max_tokens=2048, layers="LLLF"):
        self.handle = gdn.gdn_handle_create(torch.cuda.current_device())
        self.pages = Pages(slots, num_pages, max_tokens)
        self.layers = [FullAttention(self.pages) if c == "F" else LinearAttention(slots)
                       for c in layers]
        self.known = [False] * slots
        self.waiting = []  # requests that the last step had no pages for

    def step(self, rows):
        """rows: {slot: [n, HIDDEN] bf16}. A slot that was free takes a new request."""
        new = self.pages.admit([rows[s].shape[0] if s in rows else 0
                                for s in range(self.pages.slots)])
        used = [s for s in sorted(rows) if new[s]]
        self.waiting = [s for s in sorted(rows) if not new[s]]
        if not used:
            return {}
        cu = [0]
        for s in used:
            cu.append(cu[-1] + new[s])
        fresh = [0 if self.known[s] else 1 for s in used]
        self.pages.plan(self.handle, new)
        x = torch.cat([rows[s] for s in used])
        for layer in self.layers:
            if isinstance(layer, FullAttention):
                x = x + layer(self.handle, self.pages, _norm(x))
            else:
                x = x + layer(self.handle, cu, used, fresh, _norm(x))
        self.pages.advance()
        for s in used:
            self.known[s] = True
        return {s: x[cu[i + 1] - 1:cu[i + 1]] for i, s in enumerate(used)}

    def end(self, slots):
        self.pages.release(self.handle, slots)
        for s in slots:
            self.known[s] = False

    def check(self):
        """Raise what the kernels found (pages that ran out, values out of range)."""
        status = gdn.GDN_ERR_POOL_EXHAUSTED if self.waiting else int(self.pages.status.item())
        if status != gdn.GDN_OK:
            raise gdn.GdnError(status, "serve")

    def close(self):
        torch.cuda.synchronize()
        gdn.gdn_handle_destroy(self.handle)


def serve(server, prompts, answer):
    """Every prompt and `answer` steps behind it; a freed slot takes the next prompt, whose rows
    share the step with the others' single ones. What gets no pages waits for the others to end;
    where nothing can run, check() raises. Returns the prompts' last rows, in order."""
    waiting, running, last = list(range(len(prompts))), {}, [None] * len(prompts)
    left = [answer] * len(prompts)
    while waiting or running:
        rows = {s: last[r] if server.known[s] else prompts[r] for s, r in running.items()}
        for s in range(server.pages.slots):
            if s not in running and waiting:
                running[s] = waiting.pop(0)
                rows[s] = prompts[running[s]]
        out = server.step(rows)
        if not out:
            server.check()
        ended = []
        for s, r in [(s, r) for s, r in running.items() if s in out]:
            last[r] = out[s]
            left[r] -= 1
            if left[r] < 0:
                ended.append(s)
                del running[s]
        if ended:
            server.end(ended)
    server.check()
    return last


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=6)
    p.add_argument("--answer", type=int, default=24, help="tokens after each prompt")
    args = p.parse_args()
    torch.manual_seed(0)
    server = Server(slots=4)
    prompts = [torch.randn(37 + 211 * i, HIDDEN, device="cuda").bfloat16()
               for i in range(args.requests)]
    rows = serve(server, prompts, args.answer)
    free = int(server.pages.count.item())
    print(f"{args.requests} requests served, last rows' norms "
          + ", ".join(f"{float(r.float().norm()):.1f}" for r in rows)
          + f"; {free} of {server.pages.num_pages} pages free again")
    server.close()


if __name__ == "__main__":
    main()
