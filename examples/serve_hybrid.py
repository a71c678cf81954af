"""Serve requests on a small hybrid model: gated-delta-rule layers with one full-attention
layer behind every three, random weights, prompts and one-token steps in the same pack.

    python examples/serve_hybrid.py [--requests 6] [--answer 24] [--layers LLSF] [--vocab 1000]

A step's pages, slots and positions are planned on the GPU once; every full-attention layer
then appends its keys and values to its paged 8-bit cache (rotating keys and queries on the
way) and attends over it; every linear layer reads and writes its states in its pool. The
projections are plain matrix products. Requests for whose rows there are no pages sit out the
step, in every layer, and are tried again in the next one.

A layer S is a selective scan behind its short convolution, whose states and last inputs live in
pools beside the linear layers' states; the norm in front of it takes the residual's addition with
it. With --vocab the prompts are tokens: the last norm gives its rows in 8 bits to the projection
onto the vocabulary, and the next token is drawn from its logits.
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
INNER, STATE, RANK, TAPS = 1024, 16, 32, 4  # channels, states, rank of the steps and taps of a layer S


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


class StateSpace:
    def __init__(self, slots):
        self.states = torch.zeros(slots, INNER, STATE, device="cuda")
        self.inputs = torch.zeros(slots, TAPS - 1, INNER, dtype=torch.bfloat16, device="cuda")
        self.into, self.out = _weight(HIDDEN, 2 * INNER), _weight(INNER, HIDDEN)
        self.low, self.up = _weight(INNER, RANK + 2 * STATE), _weight(RANK, INNER)
        self.conv = gdn.make_conv_config(torch.randn(INNER, TAPS, device="cuda") * TAPS ** -0.5,
                                         0.1 * torch.randn(INNER, device="cuda"))
        rates = -torch.arange(1, STATE + 1, dtype=torch.float32, device="cuda")
        self.scan = gdn.make_ssm_config(rates.expand(INNER, STATE).contiguous(),
                                        torch.ones(INNER, device="cuda"),
                                        torch.empty(INNER, device="cuda").uniform_(-6, -2))

    def __call__(self, handle, pages, fresh, x):
        rows = pages.rows
        x, z = (x @ self.into).chunk(2, dim=1)  # column ranges, not copies
        # request n is slot n, as in the plan; a slot without rows in this step keeps its state
        req = gdn.make_requests(pages.cu, rows, pages.longest, pages.slots, start_zero=fresh)
        c = torch.empty(rows, INNER, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_conv_packed(handle, self.conv, req, x, x.stride(0), c, INNER, self.inputs, None,
                            pages.status)
        low = c @ self.low
        record = gdn.make_ssm_rows(c, low[:, :RANK] @ self.up, low[:, RANK:RANK + STATE],
                                   low[:, RANK + STATE:], c, z)  # the outputs over the inputs
        size = gdn.gdn_ssm_workspace_size(self.scan, req)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        gdn.gdn_ssm_packed(handle, self.scan, req, record, self.states, None, work, size,
                           pages.status)
        return c @ self.out


class AddNorm:
    """The norm of rows with what the layer in front adds to them."""

    def __init__(self):
        self.cfg = gdn.make_norm_config(HIDDEN, torch.ones(HIDDEN, device="cuda"))

    def __call__(self, handle, x, add=None):
        """(the sum, its norm); without `add` the rows and their norm."""
        y, s = torch.empty_like(x), x if add is None else torch.empty_like(x)
        gdn.gdn_rms_norm(handle, self.cfg, x.shape[0], x, HIDDEN, add, HIDDEN,
                         None if add is None else s, HIDDEN, y=y, y_stride=HIDDEN)
        return s, y


class Vocabulary:
    """Tokens to rows and rows to tokens."""

    def __init__(self, size):
        self.size, self.embed, self.head = size, _weight(size, HIDDEN), _weight(HIDDEN, size)
        self.embed *= size ** 0.5
        self.cfg = gdn.make_norm_config(HIDDEN, torch.ones(HIDDEN, device="cuda"))

    def draw(self, handle, x, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0):
        n = x.shape[0]
        codes = torch.empty(n, HIDDEN, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(n, 1, device="cuda")
        gdn.gdn_rms_norm(handle, self.cfg, n, x, HIDDEN, codes=codes, codes_stride=HIDDEN,
                         scales=scales)
        logits = (codes.bfloat16() @ self.head).float() * scales
        f = lambda v: torch.full((n,), v, device="cuda")  # noqa: E731
        token = torch.empty(n, dtype=torch.int32, device="cuda")
        gdn.gdn_sample(handle, gdn.GDN_F32, n, self.size, logits, self.size, f(temperature),
                       torch.full((n,), top_k, dtype=torch.int32, device="cuda"), f(top_p),
                       f(min_p), torch.rand(n, device="cuda"), token)
        return token


class Server:
    """`slots` requests at a time. step() takes the new rows of some of them (a prompt or a
    single token each) and gives each one's last row back; a request without pages is left out
    of the step and of its results. With a vocabulary, rows are token numbers, and what comes back
    is the next one."""

    def __init__(self, slots=8, num_pages=128, max_tokens=2048, layers="LLLF", vocab=0):
        self.handle = gdn.gdn_handle_create(torch.cuda.current_device())
        self.pages = Pages(slots, num_pages, max_tokens)
        kinds = dict(F=lambda: FullAttention(self.pages), L=lambda: LinearAttention(slots),
                     S=lambda: StateSpace(slots))
        self.layers = [kinds[c]() for c in layers]
        self.add_norm = AddNorm() if "S" in layers else None
        self.vocab = Vocabulary(vocab) if vocab else None
        self.known = [False] * slots
        self.waiting = []  # requests that the last step had no pages for

    def step(self, rows):
        """rows: {slot: [n, HIDDEN] bf16}, or {slot: [n] int32 tokens}. A slot that was free takes
        a new request."""
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
        if self.vocab:
            x = self.vocab.embed[x.long()]
        add = None  # what a layer S adds, until the next norm takes it
        for layer in self.layers:
            if isinstance(layer, StateSpace):
                x, normed = self.add_norm(self.handle, x, add)
                new_slots = torch.tensor([not k for k in self.known], dtype=torch.int32).cuda()
                add = layer(self.handle, self.pages, new_slots, normed)
                continue
            x, add = x if add is None else x + add, None
            if isinstance(layer, FullAttention):
                x = x + layer(self.handle, self.pages, _norm(x))
            else:
                x = x + layer(self.handle, cu, used, fresh, _norm(x))
        x = x if add is None else x + add
        self.pages.advance()
        for s in used:
            self.known[s] = True
        if self.vocab:
            x = x[torch.tensor(cu[1:]).cuda() - 1]
            token = self.vocab.draw(self.handle, x)
            return {s: token[i:i + 1] for i, s in enumerate(used)}
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
    where nothing can run, check() raises. Returns the prompts' last rows (or tokens), in order."""
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
    p.add_argument("--layers", default="LLLF", help="L linear, F full attention, S selective scan")
    p.add_argument("--vocab", type=int, default=0, help="serve tokens of a vocabulary of this size")
    args = p.parse_args()
    torch.manual_seed(0)
    server = Server(slots=4, layers=args.layers, vocab=args.vocab)
    if args.vocab:
        prompts = [torch.randint(0, args.vocab, (37 + 211 * i,), dtype=torch.int32, device="cuda")
                   for i in range(args.requests)]
    else:
        prompts = [torch.randn(37 + 211 * i, HIDDEN, device="cuda").bfloat16()
                   for i in range(args.requests)]
    rows = serve(server, prompts, args.answer)
    free = int(server.pages.count.item())
    last = "last tokens " + ", ".join(str(r.item()) for r in rows) if args.vocab else \
        "last rows' norms " + ", ".join(f"{float(r.float().norm()):.1f}" for r in rows)
    print(f"{args.requests} requests served, {last}; {free} of {server.pages.num_pages} pages "
          "free again")
    server.close()


if __name__ == "__main__":
    main()
