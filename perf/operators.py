"""Timed cases of the paged 8-bit attention operators: the step plan (block tables and slot
maps), the multi-axis rotary embedding, the quantising cache append and the attention that
reads the cache.

Every case can run in a plain form (elementary torch operations in 32 bits, 64 where angles
of far positions need them) or, with `own` set, through the library's entry points. `exact`
gives the same outputs from the operators' definitions in 64 bits.

Shapes: 16 query heads over 2 key/value heads of 256 with a rotary part of 64 in three axes
is the full-attention layer of the hybrid models whose linear layers this library serves;
heads of 64 and 128 and the lengths (1,024-token chat prompts, 8,192-token prompts, ragged
prefix-cache packs, decode batches, the tiny fp32 pack) are those of the library's own
workloads.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100  # exponent of the scale of a page that holds only zeros
THETA = 1.0e7
NEG = float("-inf")


# ---- cases -------------------------------------------------------------------------------

def listed():
    wide = dict(hq=16, hkv=2, d=256, dtype="bf16", page=64)
    return [
        # one scheduler step of a decode batch: every request grows by one token
        dict(name="plan_decode_256", op="plan", seqs=256, ctx_lo=1, ctx_hi=8192, new_lo=1,
             new_hi=1, page=64, lens=1),
        # a step that admits many prompts beside decoding requests
        dict(name="plan_admit_512", op="plan", seqs=512, ctx_lo=0, ctx_hi=2048, new_lo=1,
             new_hi=128, page=16, lens=2),
        # rotation of one decode step's queries and keys (positions of text after an image)
        dict(name="rope_decode_32", op="rope", tokens=32, hq=16, hkv=2, d=256, rot=64, axes=3,
             interleaved=True, dtype="bf16", far=262144),
        # rotation of a whole chat wave
        dict(name="rope_wave", op="rope", tokens=32768, hq=16, hkv=2, d=256, rot=64, axes=3,
             interleaved=True, dtype="bf16", far=8192),
        # a decode step's keys and values into half-filled pages, rotated on the way
        dict(name="append_decode_32", op="append", seqs=32, ctx_lo=1, ctx_hi=1024, new_lo=1,
             new_hi=1, rot=64, axes=3, interleaved=True, lens=3, **wide),
        # a chat wave's keys and values into fresh pages
        dict(name="append_wave", op="append", seqs=32, ctx_lo=0, ctx_hi=0, new_lo=1024,
             new_hi=1024, rot=64, axes=3, interleaved=True, lens=4, **wide),
        # the tiny fp32 pack's lengths
        dict(name="attn_tiny_f32", op="attn", seqs=4, ctx_lo=0, ctx_hi=0, new_lo=17, new_hi=255,
             hq=4, hkv=2, d=64, dtype="f32", page=16, lens=5),
        # one user's next token over a long context: few rows, a long axis
        dict(name="attn_decode_1x32k", op="attn", seqs=1, ctx_lo=32767, ctx_hi=32767, new_lo=1,
             new_hi=1, lens=6, **wide),
        # a large ragged decode batch
        dict(name="attn_decode_128", op="attn", seqs=128, ctx_lo=128, ctx_hi=16384, new_lo=1,
             new_hi=1, lens=7, **wide),
        # ragged prompts behind cached prefixes
        dict(name="attn_prefix_8", op="attn", seqs=8, ctx_lo=0, ctx_hi=2048, new_lo=128,
             new_hi=2048, hq=32, hkv=8, d=128, dtype="bf16", page=16, lens=8),
        # a chat wave of new prompts
        dict(name="attn_wave", op="attn", seqs=32, ctx_lo=0, ctx_hi=0, new_lo=1024, new_hi=1024,
             lens=9, **wide),
        # four long prompts
        dict(name="attn_long_4x8k", op="attn", seqs=4, ctx_lo=0, ctx_hi=0, new_lo=8192,
             new_hi=8192, lens=10, **wide),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attn", "attn", "attn"])
    lens = rng.randrange(1 << 20)
    hq, hkv, d = rng.choice([(16, 2, 256), (32, 8, 128), (32, 4, 128), (8, 1, 128), (12, 4, 64),
                             (16, 16, 64), (8, 2, 256), (7, 1, 64)])
    page = rng.choice([16, 32, 64, 128])
    dtype = "bf16"
    if op == "plan":
        new_hi = rng.choice([1, 4, 64, 256])
        return dict(op="plan", seqs=_log_int(rng, 1, 768), ctx_lo=0, ctx_hi=_log_int(rng, 64, 8192),
                    new_lo=rng.choice([0, 1]), new_hi=new_hi, page=page, lens=lens)
    rot = rng.choice([r for r in (32, 64, 128) if r <= d])
    axes = rng.choice([1, 3])
    if op == "rope":
        return dict(op="rope", tokens=_log_int(rng, 1, 32768), hq=hq, hkv=hkv, d=d, rot=rot,
                    axes=axes, interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), far=_log_int(rng, 64, 262144))
    shape = dict(hq=hq, hkv=hkv, d=d, dtype=dtype, page=page, lens=lens)
    if op == "append":
        new = _log_int(rng, 1, 1024)
        return dict(op="append", seqs=_log_int(rng, 1, 32), ctx_lo=0, ctx_hi=rng.choice([0, 500]),
                    new_lo=max(1, new // 2), new_hi=new, rot=rng.choice([0, rot]), axes=axes,
                    interleaved=rng.random() < 0.5, **shape)
    kind = rng.choice(["decode", "few", "prefill", "tiny"])
    if kind == "decode":
        seqs = _log_int(rng, 1, 128)
        hi = _log_int(rng, 64, min(32768, 1 << 20 if seqs == 1 else (1 << 20) // seqs))
        return dict(op="attn", seqs=seqs, ctx_lo=max(1, hi // 16), ctx_hi=hi, new_lo=1, new_hi=1,
                    **shape)
    if kind == "few":
        return dict(op="attn", seqs=_log_int(rng, 1, 32), ctx_lo=16, ctx_hi=_log_int(rng, 64, 8192),
                    new_lo=1, new_hi=rng.choice([2, 4, 8]), **shape)
    if kind == "prefill":
        new = _log_int(rng, 96, 4096)
        seqs = _log_int(rng, 1, max(1, min(16, 8192 // new)))
        return dict(op="attn", seqs=seqs, ctx_lo=0, ctx_hi=rng.choice([0, 1000, 4000]),
                    new_lo=max(1, new // 3), new_hi=new, **shape)
    shape["dtype"] = "f32"
    return dict(op="attn", seqs=_log_int(rng, 1, 8), ctx_lo=0, ctx_hi=_log_int(rng, 1, 300),
                new_lo=1, new_hi=_log_int(rng, 2, 100), **shape)


def _lengths(case):
    """(cached, new) tokens of every request: fixed by the case, not by the inputs' seed."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["seqs"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    return ctx, new


def _sections(case):
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [half]
    w = half // 3
    h = (half - w) // 2
    return [half - h - w, h, w]


# ---- inputs ------------------------------------------------------------------------------

def _ceil(a, b):
    return -(-a // b)


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _quantised(gen, pages, hkv, page, d):
    """A filled cache: normal values with a few strong channels, a power-of-two scale for
    each page and head."""
    x = _randn(gen, pages, hkv, page, d)
    x[..., :: max(1, d // 4)] *= 4.0
    amax = x.abs().amax(dim=(2, 3))
    scale = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    s = _PREPARE[case["op"]](case, gen)
    s["case"] = case
    _handle(s)
    return s


_library = {}


def _handle(s):
    """The library's handle and the argument records that a program keeps across calls."""
    if not own:
        return
    from packed_linear_attention_gb300 import gdn
    if "handle" not in _library:
        _library["handle"] = gdn.gdn_handle_create(torch.cuda.current_device(), 0)
    case = s["case"]
    s.update(gdn=gdn, handle=_library["handle"], stream=torch.cuda.current_stream())
    if case.get("rot"):
        s["rope"] = gdn.gdn_rope_init(
            case["d"], case["rot"], _sections(case),
            gdn.GDN_ROPE_INTERLEAVED if case["interleaved"] else gdn.GDN_ROPE_SECTIONS,
            gdn.GDN_ROPE_HALVES, THETA)
    if "k_cache" in s:
        s["cache"] = gdn.make_kv_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if case["op"] == "attn":
        io = gdn.GDN_BF16 if case["dtype"] == "bf16" else gdn.GDN_F32
        s["cfg"] = gdn.make_attn_config(case["hq"], scale=s["scale"], causal=True, io_dtype=io)
        n = gdn.gdn_attn_workspace_size(s["cfg"], s["cache"], case["seqs"], s["tokens"],
                                        s["max_q"], s["max_kv"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")


def _pages(gen, counts, spare):
    """Random distinct pages for requests of so many pages: table [B][max] (-1 past the end)."""
    total, width = sum(counts), max(1, max(counts))
    perm = torch.randperm(total + spare, device="cuda", generator=gen).to(torch.int32)
    n = torch.tensor(counts, device="cuda")
    at = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    table = perm[(at[:, None] + j).clamp(max=total + spare - 1)]
    return torch.where(j < n[:, None], table, -1).contiguous(), perm[total:].contiguous()


def _prepare_plan(case, gen):
    ctx, new = _lengths(case)
    page, b = case["page"], case["seqs"]
    width = _ceil(case["ctx_hi"] + case["new_hi"], page) + 1
    need = sum(_ceil(c + n, page) - _ceil(c, page) for c, n in zip(ctx, new))
    used, free = _pages(gen, [_ceil(c, page) for c in ctx], need + 64)
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    table[:, :used.shape[1]] = used
    tokens = _ceil(max(1, sum(new)), 64) * 64  # rows of the step, padded as a graph's are
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(
        tokens=tokens, num_pages=int(sum(_ceil(c, page) for c in ctx) + free.numel()),
        ctx=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), table=table, free=free,
        free_count=torch.tensor([free.numel()], **i32), free_out=torch.empty(1, **i32),
        cu=torch.empty(b + 1, **i32), kv_len=torch.empty(b, **i32),
        positions=torch.empty(tokens, **i32),
        slots=torch.empty(tokens, dtype=torch.int64, device="cuda"),
        status=torch.zeros(1, **i32))


def _fused(case, gen, tokens):
    """q, k and v as column ranges of one projection's output, as a layer has them."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = _randn(gen, tokens, (hq + 2 * hkv) * d).to(t)
    q = qkv[:, :hq * d].view(tokens, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(tokens, hkv, d)
    v = qkv[:, (hq + hkv) * d:].view(tokens, hkv, d)
    return qkv, q, k, v


def _positions(case, gen, tokens, far):
    """Positions on every axis: text moves all axes together, an image's patches differ."""
    base = torch.randint(0, far, (1, tokens), device="cuda", generator=gen)
    axes = base.expand(case["axes"], tokens).clone()
    if case["axes"] > 1:
        patch = torch.randint(0, 64, (case["axes"] - 1, tokens), device="cuda", generator=gen)
        image = (torch.arange(tokens, device="cuda") // 16) % 2 == 1
        axes[1:] += torch.where(image, patch, 0)
    return axes.to(torch.int32).contiguous()


def _prepare_rope(case, gen):
    n = case["tokens"]
    qkv, q, k, _ = _fused(case, gen, n)
    return dict(qkv=qkv, q=q, k=k, positions=_positions(case, gen, n, case["far"]),
                q_out=torch.empty(n, case["hq"], case["d"], dtype=q.dtype, device="cuda"),
                k_out=torch.empty(n, case["hkv"], case["d"], dtype=q.dtype, device="cuda"))


def _slots(ctx, new, table, page):
    n = torch.tensor(new, device="cuda")
    c = torch.tensor(ctx, device="cuda")
    cu = torch.cumsum(n, 0) - n
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), n)
    pos = c[seq] + torch.arange(seq.numel(), device="cuda") - cu[seq]
    return table[seq, pos // page].long() * page + pos % page


def _prepare_append(case, gen):
    ctx, new = _lengths(case)
    page, d, hkv = case["page"], case["d"], case["hkv"]
    counts = [_ceil(c + n, page) for c, n in zip(ctx, new)]
    table, _ = _pages(gen, counts, 0)
    k_cache, k_scale = _quantised(gen, sum(counts), hkv, page, d)
    v_cache, v_scale = _quantised(gen, sum(counts), hkv, page, d)
    tokens = sum(new)
    qkv, q, k, v = _fused(case, gen, tokens)
    s = dict(qkv=qkv, k=k, v=v, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale,
             v_scale=v_scale, slots=_slots(ctx, new, table, page),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["rot"]:
        s.update(q=q, positions=_positions(case, gen, tokens, 8192),
                 q_out=torch.empty(tokens, case["hq"], d, dtype=q.dtype, device="cuda"))
    return s


def _prepare_attn(case, gen):
    ctx, new = _lengths(case)
    page, d, hkv, hq = case["page"], case["d"], case["hkv"], case["hq"]
    kv = [c + n for c, n in zip(ctx, new)]
    counts = [_ceil(x, page) for x in kv]
    table, _ = _pages(gen, counts, 0)
    k_cache, k_scale = _quantised(gen, sum(counts), hkv, page, d)
    v_cache, v_scale = _quantised(gen, sum(counts), hkv, page, d)
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    tokens = sum(new)
    q = (1.5 * _randn(gen, tokens, hq, d)).to(t)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.zeros(len(new) + 1, **i32)
    cu[1:] = torch.cumsum(torch.tensor(new, **i32), 0)
    return dict(q=q, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                table=table, cu=cu, kv_len=torch.tensor(kv, **i32), scale=d ** -0.5,
                tokens=tokens, max_q=max(new), max_kv=max(kv), o=torch.empty_like(q),
                lse=torch.empty(tokens, hq, dtype=torch.float32, device="cuda"),
                status=torch.zeros(1, **i32))


_PREPARE = dict(plan=_prepare_plan, rope=_prepare_rope, append=_prepare_append,
                attn=_prepare_attn)


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_plan(s):
    gdn, c = s["gdn"], s["case"]
    gdn.gdn_kv_plan(s["handle"], c["page"], c["seqs"], s["tokens"], s["ctx"], s["new"],
                    s["table"], s["table"].shape[1], s["num_pages"], s["free"], s["free_count"],
                    s["free_out"], s["cu"], s["kv_len"], s["positions"], s["slots"], s["status"],
                    s["stream"])
    return dict(table=s["table"], cu=s["cu"], kv_len=s["kv_len"], positions=s["positions"],
                slots=s["slots"], free=s["free_out"])


def _own_rope(s):
    gdn, c = s["gdn"], s["case"]
    io = gdn.GDN_BF16 if c["dtype"] == "bf16" else gdn.GDN_F32
    width, n, d = s["qkv"].shape[1], c["tokens"], c["d"]
    gdn.gdn_rope_apply(s["handle"], s["rope"], io, n, s["positions"], n, s["q"], width, c["hq"],
                       s["q_out"], c["hq"] * d, s["k"], width, c["hkv"], s["k_out"],
                       c["hkv"] * d, s["stream"])
    return dict(q=s["q_out"], k=s["k_out"])


def _own_append(s):
    gdn, c = s["gdn"], s["case"]
    io = gdn.GDN_BF16 if c["dtype"] == "bf16" else gdn.GDN_F32
    width, n, d = s["qkv"].shape[1], s["k"].shape[0], c["d"]
    rot = (s["rope"], s["positions"], n, s["q"], width, c["hq"], s["q_out"], c["hq"] * d) \
        if c["rot"] else (None, None, 0, None, 0, 0, None, 0)
    gdn.gdn_kv_append(s["handle"], s["cache"], io, n, s["slots"], s["k"], width, s["v"], width,
                      *rot, s["status"], s["stream"])
    out = dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return dict(out, q=s["q_out"]) if c["rot"] else out


def _own_attn(s):
    gdn, c = s["gdn"], s["case"]
    row = c["hq"] * c["d"]
    gdn.gdn_attn_paged(s["handle"], s["cfg"], s["cache"], c["seqs"], s["tokens"], s["max_q"],
                       s["max_kv"], s["cu"], s["kv_len"], s["table"], s["table"].shape[1], s["q"],
                       row, s["o"], row, s["lse"], s["workspace"], s["workspace"].numel(),
                       s["status"], s["stream"])
    return dict(o=s["o"], lse=s["lse"])


_OWN = dict(plan=_own_plan, rope=_own_rope, append=_own_append, attn=_own_attn)


def _plain_plan(s):
    page, tokens, table = s["case"]["page"], s["tokens"], s["table"].clone()
    ctx, new = s["ctx"].long(), s["new"].long()
    end = ctx + new
    have, want = (ctx + page - 1) // page, (end + page - 1) // page
    need = want - have
    upto = torch.cumsum(need, 0)
    # pages leave the top of the free stack in request order
    j = torch.arange(table.shape[1], device=table.device)
    fresh = (j >= have[:, None]) & (j < want[:, None])
    k = s["free_count"].long() - 1 - ((upto - need)[:, None] + j - have[:, None])
    popped = s["free"][k.clamp(0, s["free"].numel() - 1)]
    table = torch.where(fresh, popped, table)
    cu = torch.zeros_like(s["cu"])
    cu[1:] = torch.cumsum(new, 0)
    row = torch.arange(tokens, device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), row.int(), right=True)
    live = seq < len(new)
    seq = seq.clamp(max=len(new) - 1)
    pos = torch.where(live, ctx[seq] + row - cu[seq], 0)
    slots = torch.where(live, table[seq, pos // page].long() * page + pos % page, -1)
    return dict(table=table, cu=cu, kv_len=end.int(), positions=pos.int(), slots=slots,
                free=(s["free_count"] - upto[-1]).int())


def _axis_of(case, half):
    """Axis of every rotated pair: whole sections, or the axes taking turns."""
    sec = _sections(case)
    i = torch.arange(half, device="cuda")
    if case["axes"] == 1:
        return torch.zeros_like(i)
    if not case["interleaved"]:
        return (i >= sec[0]).long() + (i >= sec[0] + sec[1]).long()
    a = i % 3
    limit = torch.tensor([half, 3 * sec[1], 3 * sec[2]], device="cuda")
    return torch.where(i < limit[a], a, 0)


def _rotate(case, positions, x):
    """Rotary embedding of x [T, H, D] (fp32), the pairs half a rotary part apart."""
    half = case["rot"] // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    freq = THETA ** (-i / half)
    angle = positions[_axis_of(case, half)].double().T * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    return dict(q=_rotate(c, s["positions"], s["q"].float()).to(s["q"].dtype),
                k=_rotate(c, s["positions"], s["k"].float()).to(s["k"].dtype))


def _page_scale(amax):
    """The least power of two 2^e with amax <= 448 * 2^e (e at least MIN_EXP)."""
    m, x = torch.frexp(amax)
    e = torch.where(amax > 0, x - 9 + (m > 0.875).int(), MIN_EXP).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_store(cache, scale, slots, x):
    """Store rows x [T, H, D] at their slots: pages' scales grow to what the new rows need,
    rows already there are rounded again where their scale grew."""
    pages, hkv, page, d = cache.shape
    at, off = slots // page, slots % page
    first = torch.full((pages,), page, device=x.device, dtype=off.dtype)
    first.scatter_reduce_(0, at, off, "amin")
    amax = torch.zeros(pages, hkv, device=x.device)
    amax.index_reduce_(0, at, x.abs().amax(-1), "amax")
    need = _page_scale(amax)
    old = torch.where((first > 0)[:, None], scale, 0.0)
    grown = torch.where((first < page)[:, None], torch.maximum(old, need), scale)
    touched = torch.unique(at)
    ratio = (scale[touched] / grown[touched])[:, :, None, None]
    keep = torch.arange(page, device=x.device) < first[touched][:, None]
    was = cache[touched].float()
    again = torch.where(keep[:, None, :, None], was * ratio, was).to(cache.dtype)
    cache.view(torch.uint8)[touched] = again.view(torch.uint8)
    code = (x / grown[at][:, :, None]).to(cache.dtype)
    cache.view(torch.uint8)[at, :, off] = code.view(torch.uint8)
    scale.copy_(grown)


def _plain_append(s):
    c = s["case"]
    k, v = s["k"].float(), s["v"].float()
    out = dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["rot"]:
        k = _rotate(c, s["positions"], k)
        out["q"] = _rotate(c, s["positions"], s["q"].float()).to(s["q"].dtype)
    _plain_store(s["k_cache"], s["k_scale"], s["slots"], k)
    _plain_store(s["v_cache"], s["v_scale"], s["slots"], v)
    return out


def _plain_attn(s):
    q, table, kv_len, cu = s["q"], s["table"], s["kv_len"].long(), s["cu"].long()
    tokens, hq, d = q.shape
    hkv, page = s["k_cache"].shape[1:3]
    group, b, mq = hq // hkv, table.shape[0], s["max_q"]
    nb = _ceil(s["max_kv"], page)
    ids = table[:, :nb].clamp(min=0).long()

    def dense(cache, scale):  # [B, Hkv, L, D]
        x = cache[ids].float() * scale[ids][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, hkv, nb * page, d)

    q_len = cu[1:] - cu[:-1]
    i = torch.arange(mq, device=q.device)
    rows = (cu[:-1, None] + i).clamp(max=tokens - 1)
    qp = q[rows].float().view(b, mq, hkv, group, d).permute(0, 2, 3, 1, 4)
    qp = qp.reshape(b, hkv, group * mq, d)
    score = torch.matmul(qp, dense(s["k_cache"], s["k_scale"]).transpose(2, 3))
    score = score.mul_(s["scale"]).view(b, hkv, group, mq, nb * page)
    last = kv_len[:, None] - q_len[:, None] + i
    j = torch.arange(nb * page, device=q.device)
    hidden = (j > last[..., None]) | (j >= kv_len[:, None, None])
    score = score.masked_fill_(hidden[:, None, None], NEG)
    top = score.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, group * mq, nb * page), dense(s["v_cache"], s["v_scale"]))
    o = o.view(b, hkv, group, mq, d) / total
    lse = (top + total.log())[..., 0]
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(tokens, device=q.device), right=True)
    at = torch.arange(tokens, device=q.device) - cu[seq]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, mq, hq, d)[seq, at]
    lse = lse.permute(0, 3, 1, 2).reshape(b, mq, hq)[seq, at]
    return dict(o=o.to(q.dtype), lse=lse)


_PLAIN = dict(plan=_plain_plan, rope=_plain_rope, append=_plain_append, attn=_plain_attn)


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    ctx, new = _lengths(case) if "lens" in case else ([], [])
    page, tokens = case.get("page", 1), sum(new)
    item = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "plan":
        grown = sum(_ceil(c + n, page) - _ceil(c, page) for c, n in zip(ctx, new))
        rows = _ceil(max(1, tokens), 64) * 64
        return dict(bytes=16 * case["seqs"] + 8 * grown + 12 * rows, flops=4 * rows)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        n = case["tokens"]
        return dict(bytes=n * (2 * item * (hq + hkv) * d + 4 * case["axes"]),
                    flops=n * (hq + hkv) * case["rot"] * 3)
    if case["op"] == "append":
        pages = sum((c + n - 1) // page - c // page + 1 for c, n in zip(ctx, new))
        b = tokens * (2 * (item + 1) * hkv * d + 8) + 16 * pages * hkv
        f = 4 * tokens * hkv * d
        if case["rot"]:
            b += tokens * (2 * item * hq * d + 4 * case["axes"])
            f += 3 * tokens * (hq + hkv) * case["rot"]
        return dict(bytes=b, flops=f)
    cached = sum(c + n for c, n in zip(ctx, new))
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    pages = sum(_ceil(c + n, page) for c, n in zip(ctx, new))
    return dict(bytes=cached * 2 * hkv * d + pages * (8 * hkv + 4)
                + tokens * hq * (2 * item * d + 4), flops=4 * d * hq * pairs)


# ---- the definitions in 64 bits ----------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _turn(case, positions, x):
    """Every pair (x_i, x_{i + R/2}) as a complex number times e^{i angle}."""
    half, sec = case["rot"] // 2, _sections(case)
    axis, count = [], [0, 0, 0]
    for i in range(half):
        if case["axes"] == 1:
            a = 0
        elif case["interleaved"]:
            a = i % 3 if i % 3 and count[i % 3] < sec[i % 3] else 0
        else:
            a = 0 if i < sec[0] else 1 if i < sec[0] + sec[1] else 2
        count[a] += 1
        axis.append(a)
    y = x.double().clone()
    for i in range(half):
        w = positions[axis[i]].double() * math.pow(THETA, -2.0 * i / case["rot"])
        z = torch.complex(x[:, :, i].double(), x[:, :, i + half].double())
        z = z * torch.polar(torch.ones_like(w), w)[:, None]
        y[:, :, i], y[:, :, i + half] = z.real, z.imag
    return y


def _exact_rope(case, s):
    return dict(q=_turn(case, s["positions"], s["q"]), k=_turn(case, s["positions"], s["k"]))


def _nearest_e4m3(x):
    """x (float64) rounded to the nearest e4m3 value, ties to even: three fraction bits above
    2^-6, steps of 2^-9 below."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step  # torch.round: ties to even


def _exact_append(case, s):
    page = case["page"]
    new = dict(k=s["k"].double(), v=s["v"].double())
    out = {}
    if case["rot"]:
        new["k"] = _turn(case, s["positions"], s["k"])
        out["q"] = _turn(case, s["positions"], s["q"])
    order = torch.argsort(s["slots"])
    slots = s["slots"][order].tolist()
    for name in ("k", "v"):
        codes, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        at = 0
        while at < len(slots):
            p, off = divmod(slots[at], page)
            n = 1
            while at + n < len(slots) and slots[at + n] // page == p:
                n += 1
            rows = new[name][order[at:at + n]].transpose(0, 1)  # [H, n, D]
            amax = rows.abs().amax(dim=(1, 2)) / E4M3_MAX
            e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** MIN_EXP)))
            e = torch.where(torch.exp2(e - 1) >= amax, e - 1, e).clamp(min=MIN_EXP)
            grown = torch.exp2(e)
            if off:
                grown = torch.maximum(grown, scale[p])
                codes[p, :, :off] = _nearest_e4m3(codes[p, :, :off]
                                                  * (scale[p] / grown)[:, None, None])
            codes[p, :, off:off + n] = _nearest_e4m3(rows / grown[:, None, None])
            scale[p] = grown
            at += n
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_attn(case, s):
    ctx, new = _lengths(case)
    hkv, group = case["hkv"], case["hq"] // case["hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        pages = s["table"][b, :_ceil(c + n, case["page"])].long()
        for h in range(hkv):
            k, v = ((s[x + "_cache"][pages, h].double() * s[x + "_scale"][pages, h].double()
                     [:, None, None]).flatten(0, 1)[:c + n] for x in ("k", "v"))
            heads = slice(h * group, (h + 1) * group)
            for r0 in range(0, n, 1024):
                r1 = min(n, r0 + 1024)
                see = c + r1
                q = s["q"][at + r0:at + r1, heads].double()
                x = torch.einsum("tgd,jd->gtj", q, k[:see]) * s["scale"]
                j = torch.arange(see, device="cuda")
                x[:, j[None] > c + torch.arange(r0, r1, device="cuda")[:, None]] = NEG
                total = torch.logsumexp(x, -1)
                o[at + r0:at + r1, heads] = torch.einsum("gtj,jd->tgd", (x - total[..., None]).exp(),
                                                         v[:see])
                lse[at + r0:at + r1, heads] = total.T
        at += n
    return dict(o=o, lse=lse)


_EXACT = dict(rope=_exact_rope, append=_exact_append, attn=_exact_attn)
