"""Timed cases of the operators around the recurrent layers of a hybrid model's serving step: the
short causal convolution and the selective scan (packed prompts and single tokens, states in
pools), the root-mean-square norm (residual, gate, 8-bit output) and the sampling of tokens.

Every case can run in a plain form (elementary torch operations in 32 bits, 64 where values lie
next to a border) or, with `own` set, through the library's entry points. `exact` gives the same
outputs from the operators' definitions in 64 bits.

Shapes: 8,192 convolved channels are the q, k and v columns of the library's chat-wave layer (16
key and 32 value heads of 128), 4,096 channels its value width, 32 heads of 128 its output; a
hidden size of 2,048, 1,024-token chat prompts, prompts behind cached prefixes, a 32,768-token
prompt, decode batches and the tiny fp32 pack are those of the library's own workloads.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100
GRID = 256  # checkpoints lie on multiples of it, out of a prompt's last 16 tokens


# ---- cases -------------------------------------------------------------------------------

def listed():
    return [
        # a decode batch's q, k and v columns
        dict(name="conv_step_32", op="conv_step", batch=32, ch=8192, width=4, bias=False,
             dtype="bf16"),
        # the same columns of a chat wave
        dict(name="conv_wave", op="conv", seqs=32, lo=1024, hi=1024, singles=0, ch=8192, width=4,
             bias=False, ckpt=True, dtype="bf16", lens=1),
        # one token of a large decode batch: the states go through memory once
        dict(name="ssm_step_128", op="ssm_step", batch=128, ch=4096, n=16, groups=1, gate=True,
             dtype="bf16"),
        # the tiny fp32 pack's lengths
        dict(name="ssm_tiny_f32", op="ssm", seqs=4, lo=17, hi=255, singles=0, ch=200, n=16,
             groups=1, gate=True, ckpt=False, dtype="f32", lens=2),
        # a chat wave of new prompts
        dict(name="ssm_wave", op="ssm", seqs=32, lo=1024, hi=1024, singles=0, ch=4096, n=16,
             groups=1, gate=True, ckpt=True, dtype="bf16", lens=3),
        # one user's long prompt: few rows, a long axis
        dict(name="ssm_long_32k", op="ssm", seqs=1, lo=32768, hi=32768, singles=0, ch=2048, n=16,
             groups=1, gate=True, ckpt=True, dtype="bf16", lens=4),
        # a mixed step: ragged prompt slices beside decoding requests, a wider state in groups
        dict(name="ssm_mixed", op="ssm", seqs=8, lo=60, hi=700, singles=32, ch=2000, n=64,
             groups=2, gate=False, ckpt=True, dtype="bf16", lens=5),
        # a decode step's block input: residual added, a scale a token for the 8-bit projection
        dict(name="norm_step_32", op="norm", tokens=32, heads=1, dim=2048, residual=True,
             gate=False, codes=True, group=0, pow2=False, dtype="bf16"),
        # the same for a chat wave, a scale for every 128 columns
        dict(name="norm_wave", op="norm", tokens=32768, heads=1, dim=2048, residual=True,
             gate=False, codes=True, group=128, pow2=True, dtype="bf16"),
        # the gated norm behind the wave's linear-attention heads
        dict(name="norm_heads_wave", op="norm", tokens=32768, heads=32, dim=128, residual=False,
             gate=True, codes=False, group=0, pow2=False, dtype="bf16"),
        # one user's next token under every filter
        dict(name="sample_1", op="sample", rows=1, vocab=151936, mix=False, dtype="f32"),
        # a large batch, every row with its own settings
        dict(name="sample_256", op="sample", rows=256, vocab=151936, mix=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "ssm_step", "ssm", "ssm", "norm", "norm", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 1 if dtype == "bf16" else 2
    if op == "conv_step":
        ch = _log_int(rng, 32, 8192)
        return dict(op=op, batch=_log_int(rng, 1, 512), ch=ch, width=rng.choice([2, 3, 4, 4]),
                    bias=rng.random() < 0.5, dtype=dtype)
    if op == "ssm_step":
        ch, n = _log_int(rng, 64, 4096), rng.choice([8, 16, 16, 32, 64])
        groups = rng.choice([1, 1, 2])
        return dict(op=op, batch=_log_int(rng, 1, max(1, 128 * 4096 * 16 // (ch * n))
                                          if ch * n > 16384 else 512),
                    ch=ch // groups * groups, n=n, groups=groups, gate=rng.random() < 0.7,
                    dtype=dtype)
    if op in ("conv", "ssm"):
        few = rng.random() < 0.4
        hi = _log_int(rng, 1024, 32768) if few else _log_int(rng, 8, 2048)
        seqs = rng.choice([1, 1, 2]) if few else _log_int(rng, 1, 32)
        singles = 0 if few else rng.choice([0, 0, 40])
        lo = max(1, hi // rng.choice([1, 2, 8]))
        tokens = seqs * hi + singles
        common = dict(op=op, seqs=seqs, lo=lo, hi=hi, singles=singles, ckpt=rng.random() < 0.5,
                      dtype=dtype, lens=rng.randrange(1 << 20))
        if op == "conv":
            most = min(8192, 32768 * 8192 // (tokens * size))
            return dict(common, ch=_log_int(rng, min(64, most), most),
                        width=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5)
        n, groups = rng.choice([8, 16, 16, 16, 32, 64]), rng.choice([1, 1, 2])
        most = min(4096, 32768 * 4096 * 16 // (tokens * n * size))
        ch = _log_int(rng, min(64, most), most)
        return dict(common, ch=ch // groups * groups, n=n, groups=groups,
                    gate=rng.random() < 0.7)
    if op == "norm":
        heads = rng.choice([1, 1, 4, 16, 32])
        dim = _log_int(rng, 64, 8192) if heads == 1 else rng.choice([64, 128, 256])
        group = rng.choice([0, 0, 64, 128]) if dim % 128 == 0 else 0
        codes = rng.random() < 0.6
        tokens = _log_int(rng, 1, min(32768, 32768 * 4096 // (heads * dim * size)))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, residual=heads == 1,
                    gate=heads > 1 or rng.random() < 0.2, codes=codes, group=group,
                    pow2=rng.random() < 0.5, dtype=dtype)
    vocab = rng.choice([32000, 50257, 128256, 151936, _log_int(rng, 1000, 200000)])
    most = 256 * 151936 // (vocab * size)
    return dict(op="sample", rows=_log_int(rng, 1, min(512, most)), vocab=vocab,
                mix=rng.random() < 0.7, dtype=dtype)


def _lengths(case):
    """Tokens of every request: fixed by the case, not by the inputs' seed."""
    r = random.Random(case["lens"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])] + [1] * case["singles"]
    r.shuffle(n)
    return n


def _checkpoints(case, lens):
    """Positions of every request's checkpoints: the last grid point that leaves 16 tokens."""
    at = [(n - 16) // GRID * GRID if case["ckpt"] else 0 for n in lens]
    return [[p] if p > 0 else [] for p in at]


# ---- inputs ------------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _rand(gen, *shape):
    return torch.rand(*shape, device="cuda", generator=gen)


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pad(n):
    return -(-n // 8) * 8  # rows start on 16-byte boundaries


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)
    s = _PREPARE[case["op"]](case, gen)
    s["case"] = case
    _handle(s)
    return s


_library = {}


def _handle(s):
    """The library's handle and the records that a program keeps across calls."""
    if not own:
        return
    from packed_linear_attention_gb300 import gdn
    if "handle" not in _library:
        _library["handle"] = gdn.gdn_handle_create(torch.cuda.current_device(), 0)
    case = s["case"]
    io = gdn.GDN_BF16 if case["dtype"] == "bf16" else gdn.GDN_F32
    s.update(gdn=gdn, handle=_library["handle"], stream=torch.cuda.current_stream(), io=io)
    op = case["op"]
    if op in ("conv", "ssm"):
        s["requests"] = gdn.make_requests(
            s["cu"], s["tokens"], s["max_len"], s["pool"].shape[0], slot_idx=s["slot"],
            start_zero=s["zero"], ckpt_cu=s["ckpt_cu"], ckpt_pos=s["ckpt_pos"],
            num_ckpt=s["num_ckpt"])
    if op in ("conv", "conv_step"):
        s["cfg"] = gdn.make_conv_config(s["weight"], s["bias"], activation=gdn.GDN_ACT_SILU,
                                        io_dtype=io)
    if op in ("ssm", "ssm_step"):
        s["cfg"] = gdn.make_ssm_config(s["a"], s["skip"], s["delta_bias"],
                                       num_groups=case["groups"], io_dtype=io)
        s["rows"] = gdn.make_ssm_rows(s["x"], s["delta"], s["b"], s["c"], s["y"], s["z"])
    if op == "ssm":
        n = gdn.gdn_ssm_workspace_size(s["cfg"], s["requests"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    if op == "norm":
        s["cfg"] = gdn.make_norm_config(case["dim"], s["weight"], num_heads=case["heads"],
                                        eps=1e-6, scale_group=case["group"],
                                        scale_pow2=case["pow2"], io_dtype=io)


def _prepare_requests(case, gen):
    lens = _lengths(case)
    b = len(lens)
    ckpt = _checkpoints(case, lens)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, ckpt_cu = [0], [0]
    for n, p in zip(lens, ckpt):
        cu.append(cu[-1] + n)
        ckpt_cu.append(ckpt_cu[-1] + len(p))
    return dict(tokens=sum(lens), max_len=max(lens), num_ckpt=ckpt_cu[-1],
                cu=torch.tensor(cu, **i32), ckpt_cu=torch.tensor(ckpt_cu, **i32),
                ckpt_pos=torch.tensor([p for q in ckpt for p in q] + [0], **i32),
                slot=torch.randperm(b + 2, device="cuda", generator=gen)[:b].int(),
                zero=(torch.arange(b, device="cuda") % 2).int())


def _conv_weights(case, gen):
    ch, w = case["ch"], case["width"]
    bias = 0.3 * _randn(gen, ch) if case["bias"] else None
    return dict(weight=(_randn(gen, ch, w) * w ** -0.5).contiguous(), bias=bias)


def _prepare_conv(case, gen):
    s, t, ch = _prepare_requests(case, gen), _type(case), case["ch"]
    # a column range of a wider projection, as a layer has it
    wide = _randn(gen, s["tokens"], _pad(ch) + 64).to(t)
    s.update(_conv_weights(case, gen), wide=wide, x=wide[:, 32:32 + ch],
             y=torch.empty(s["tokens"], _pad(ch), dtype=t, device="cuda")[:, :ch],
             pool=_randn(gen, len(s["slot"]) + 2, case["width"] - 1, ch).to(t),
             ckpt=torch.zeros(max(1, s["num_ckpt"]), case["width"] - 1, ch, dtype=t,
                              device="cuda"))
    return s


def _prepare_conv_step(case, gen):
    b, ch, t = case["batch"], case["ch"], _type(case)
    wide = _randn(gen, b, _pad(ch) + 64).to(t)
    return dict(_conv_weights(case, gen), wide=wide, x=wide[:, 32:32 + ch],
                y=torch.empty(b, _pad(ch), dtype=t, device="cuda")[:, :ch],
                pool=_randn(gen, b + 2, case["width"] - 1, ch).to(t),
                slot=torch.randperm(b + 2, device="cuda", generator=gen)[:b].int())


def _ssm_inputs(case, gen, rows, slots):
    ch, n, g, t = case["ch"], case["n"], case["groups"], _type(case)
    # time steps of 1e-3 .. 1e-1 around which the tokens' own move, decays of 1 .. n
    step = torch.exp(_rand(gen, ch) * math.log(100.0) + math.log(1e-3))
    a = -torch.arange(1, n + 1, device="cuda") * (0.5 + _rand(gen, ch, n))
    low = _randn(gen, rows, 32 + 2 * g * n).to(t)  # one projection's output: rank, B and C
    proj = _randn(gen, rows, 2 * _pad(ch)).to(t)
    return dict(low=low, proj=proj, x=_randn(gen, rows, _pad(ch)).to(t)[:, :ch],
                z=proj[:, _pad(ch):_pad(ch) + ch] if case["gate"] else None,
                delta=(0.5 * _randn(gen, rows, _pad(ch))).to(t)[:, :ch],
                b=low[:, 32:32 + g * n], c=low[:, 32 + g * n:],
                y=torch.empty(rows, _pad(ch), dtype=t, device="cuda")[:, :ch],
                a=a.contiguous(), skip=_randn(gen, ch),
                delta_bias=step + torch.log(-torch.expm1(-step)),
                pool=_randn(gen, slots, ch, n))


def _prepare_ssm(case, gen):
    s = _prepare_requests(case, gen)
    s.update(_ssm_inputs(case, gen, s["tokens"], len(s["slot"]) + 2),
             ckpt=torch.zeros(max(1, s["num_ckpt"]), case["ch"], case["n"], device="cuda"))
    return s


def _prepare_ssm_step(case, gen):
    b = case["batch"]
    return dict(_ssm_inputs(case, gen, b, b + 2),
                slot=torch.randperm(b + 2, device="cuda", generator=gen)[:b].int())


def _prepare_norm(case, gen):
    n, heads, dim, t = case["tokens"], case["heads"], case["dim"], _type(case)
    cols = _pad(heads * dim)
    s = dict(wide_x=_randn(gen, n, cols).to(t), weight=1.0 + 0.2 * _randn(gen, dim),
             residual=None, gate=None, sum=None, y=None, codes=None, scales=None)
    s["x"] = s["wide_x"][:, :heads * dim]
    if case["residual"]:
        # a residual stream: a few strong channels
        r = 3.0 * _randn(gen, n, cols)
        r[:, ::97] *= 8.0
        s["residual"] = r.to(t)[:, :heads * dim]
        s["sum"] = torch.empty(n, cols, dtype=t, device="cuda")[:, :heads * dim]
    if case["gate"]:
        s["gate"] = _randn(gen, n, 2 * cols).to(t)[:, cols:cols + heads * dim]
    if case["codes"]:
        groups = heads * dim // case["group"] if case["group"] else 1
        s["codes"] = torch.empty(n, -(-heads * dim // 16) * 16, dtype=torch.float8_e4m3fn,
                                 device="cuda")[:, :heads * dim]
        s["scales"] = torch.empty(n, groups, device="cuda")
    else:
        s["y"] = torch.empty(n, cols, dtype=t, device="cuda")[:, :heads * dim]
    return s


def _prepare_sample(case, gen):
    n, v = case["rows"], case["vocab"]
    logits = (2.5 * _randn(gen, n, v)).to(_type(case))
    f = dict(dtype=torch.float32, device="cuda")
    r = torch.arange(n, device="cuda")
    s = dict(logits=logits, u=_rand(gen, n), token=torch.empty(n, dtype=torch.int32, device="cuda"),
             logprob=torch.empty(n, **f),
             temperature=0.6 + 0.6 * _rand(gen, n), top_p=0.8 + 0.19 * _rand(gen, n),
             top_k=torch.randint(1, 200, (n,), device="cuda", generator=gen).int(),
             min_p=0.1 * _rand(gen, n))
    if case["mix"]:  # rows without a filter, greedy ones, each filter by itself
        s["temperature"] = torch.where(r % 8 == 7, torch.zeros(n, **f), s["temperature"])
        s["top_k"] = torch.where(r % 4 == 1, s["top_k"], 0).int()
        s["top_p"] = torch.where(r % 4 == 2, s["top_p"], torch.ones(n, **f))
        s["min_p"] = torch.where(r % 4 == 3, s["min_p"], torch.zeros(n, **f))
    return s


_PREPARE = dict(conv=_prepare_conv, conv_step=_prepare_conv_step, ssm=_prepare_ssm,
                ssm_step=_prepare_ssm_step, norm=_prepare_norm, sample=_prepare_sample)


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_conv(s):
    s["gdn"].gdn_conv_packed(s["handle"], s["cfg"], s["requests"], s["x"], s["x"].stride(0),
                             s["y"], s["y"].stride(0), s["pool"], s["ckpt"], None, s["stream"])
    return _outputs(s)


def _own_conv_step(s):
    s["gdn"].gdn_conv_step(s["handle"], s["cfg"], s["case"]["batch"], s["x"], s["x"].stride(0),
                           s["y"], s["y"].stride(0), s["pool"], s["pool"].shape[0], s["slot"],
                           None, s["stream"])
    return _outputs(s)


def _own_ssm(s):
    s["gdn"].gdn_ssm_packed(s["handle"], s["cfg"], s["requests"], s["rows"], s["pool"], s["ckpt"],
                            s["workspace"], s["workspace"].numel(), None, s["stream"])
    return _outputs(s)


def _own_ssm_step(s):
    s["gdn"].gdn_ssm_step(s["handle"], s["cfg"], s["case"]["batch"], s["rows"], s["pool"],
                          s["pool"].shape[0], s["slot"], None, s["stream"])
    return _outputs(s)


def _outputs(s):
    out = dict(y=s["y"], pool=s["pool"])
    return dict(out, ckpt=s["ckpt"]) if s.get("num_ckpt") else out


def _own_norm(s):
    width = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    s["gdn"].gdn_rms_norm(s["handle"], s["cfg"], s["case"]["tokens"], s["x"], width(s["x"]),
                          s["residual"], width(s["residual"]), s["sum"], width(s["sum"]),
                          s["gate"], width(s["gate"]), s["y"], width(s["y"]), s["codes"],
                          width(s["codes"]), s["scales"], s["stream"])
    return {k: s[k] for k in ("sum", "y", "codes", "scales") if s[k] is not None}


def _own_sample(s):
    c = s["case"]
    s["gdn"].gdn_sample(s["handle"], s["io"], c["rows"], c["vocab"], s["logits"], c["vocab"],
                        s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["token"],
                        s["logprob"], None, s["stream"])
    return dict(token=s["token"], logprob=s["logprob"])


_OWN = dict(conv=_own_conv, conv_step=_own_conv_step, ssm=_own_ssm, ssm_step=_own_ssm_step,
            norm=_own_norm, sample=_own_sample)


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(x.clamp(max=20.0))))


def _plain_conv(s):
    c, x, pool = s["case"], s["x"].float(), s["pool"]
    w, tokens, cu = c["width"], s["tokens"], s["cu"].long()
    slot, fresh = s["slot"].long(), s["zero"] != 0
    old = torch.where(fresh[:, None, None], 0.0, pool[slot].float())  # [B, W-1, C]
    row = torch.arange(tokens, device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    at = row - cu[seq]

    def input_at(seq, at):  # inputs of requests `seq` at positions `at`, the state's in front
        rows = x[(cu[seq] + at).clamp(0, tokens - 1)]
        held = old[seq, (w - 1 + at).clamp(0, w - 2)]
        return torch.where((at >= 0)[:, None], rows, held)

    y = torch.zeros_like(x) if s["bias"] is None else s["bias"].expand(tokens, -1).clone()
    for j in range(w):
        near = at - (w - 1 - j)
        taps = x[(row - (w - 1 - j)).clamp(min=0)]
        edge = torch.nonzero(near < 0)[:, 0]
        taps[edge] = old[seq[edge], w - 1 + near[edge]]
        y.addcmul_(taps, s["weight"][:, j])
    s["y"].copy_(_silu(y))
    every = torch.arange(len(slot), device=x.device)
    if s["num_ckpt"]:
        n = s["num_ckpt"]
        mine = torch.searchsorted(s["ckpt_cu"][1:].contiguous(),
                                  torch.arange(n, device=x.device).int(), right=True)
        for j in range(w - 1):
            s["ckpt"][:, j] = input_at(mine, s["ckpt_pos"][:n].long() - (w - 1) + j).to(pool.dtype)
    for j in range(w - 1):
        pool[slot, j] = input_at(every, cu[1:] - cu[:-1] - (w - 1) + j).to(pool.dtype)
    return _outputs(s)


def _plain_conv_step(s):
    slot, x = s["slot"].long(), s["x"].float()
    old = s["pool"][slot]
    taps = torch.cat([old.float(), x[:, None]], dim=1)
    y = (taps * s["weight"].T).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    s["y"].copy_(_silu(y))
    s["pool"][slot] = torch.cat([old[:, 1:], s["x"][:, None]], dim=1)
    return _outputs(s)


def _plain_ssm(s):
    """Requests side by side, padded to the longest (a step of 0 leaves a state as it is); the
    decays and inputs of some tokens at a time, then one product and sum a token."""
    c, cu = s["case"], s["cu"].long()
    ch, n, g = c["ch"], c["n"], c["groups"]
    slot, b, length = s["slot"].long(), len(s["slot"]), s["max_len"]
    lens = cu[1:] - cu[:-1]
    i = torch.arange(length, device="cuda")
    live = i[:, None] < lens  # [L, B]
    rows = torch.where(live, cu[:-1] + i[:, None], 0)
    h = torch.where((s["zero"] != 0)[:, None, None], 0.0, s["pool"][slot])
    chunk = max(1, min(length, (1 << 28) // (b * ch * n)))
    pos = s["ckpt_pos"][:s["num_ckpt"]].long()
    mine = torch.searchsorted(s["ckpt_cu"][1:].contiguous(),
                              torch.arange(s["num_ckpt"], device="cuda").int(), right=True)
    a, y = s["a"], torch.zeros(s["tokens"], ch, device="cuda")
    for t0 in range(0, length, chunk):
        r, on = rows[t0:t0 + chunk], live[t0:t0 + chunk]
        x = s["x"][r].float()
        dt = _softplus(s["delta"][r].float() + s["delta_bias"]) * on[..., None]
        bt, ct = (s[k][r].float().view(len(r), b, g, 1, n) for k in ("b", "c"))
        decay = torch.exp(dt[..., None] * a)
        wide = (len(r), b, g, ch // g, n)
        hist = ((dt * x).view(wide[:-1] + (1,)) * bt).reshape(len(r), b, ch, n)
        for j in range(len(r)):
            h = hist[j].addcmul_(decay[j], h)
        out = (hist.view(wide) * ct).sum(-1).view(len(r), b, ch) + s["skip"] * x
        if s["z"] is not None:
            out = out * _silu(s["z"][r].float())
        y[r[on]] = out[on]
        here = (pos > t0) & (pos <= t0 + len(r)) if s["num_ckpt"] else None
        if here is not None:
            k = torch.nonzero(here)[:, 0]
            s["ckpt"][k] = hist[pos[k] - 1 - t0, mine[k]]
        h = h.clone()
    s["y"].copy_(y)
    s["pool"][slot] = h
    return _outputs(s)


def _plain_ssm_step(s):
    c, slot = s["case"], s["slot"].long()
    b, ch, n, g = c["batch"], c["ch"], c["n"], c["groups"]
    x = s["x"].float()
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    bt, ct = (s[k].float().view(b, g, 1, n) for k in ("b", "c"))
    add = ((dt * x).view(b, g, ch // g, 1) * bt).reshape(b, ch, n)
    h = torch.exp(dt[..., None] * s["a"]) * s["pool"][slot] + add
    y = (h.view(b, g, ch // g, n) * ct).sum(-1).view(b, ch) + s["skip"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["y"].copy_(y)
    s["pool"][slot] = h
    return _outputs(s)


def _plain_norm(s):
    c = s["case"]
    n, heads, dim = c["tokens"], c["heads"], c["dim"]
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
        s["sum"].copy_(x)
    h = x.view(n, heads, dim)
    y = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["weight"]).view(n, -1)
    if s["gate"] is not None:
        y = y * _silu(s["gate"].float())
    if s["codes"] is None:
        s["y"].copy_(y)
    else:
        wide = y.view(n, s["scales"].shape[1], -1)
        top = wide.abs().amax(-1)
        scale = top / E4M3_MAX
        if c["pow2"]:  # the least power of two that holds the largest value
            m, e = torch.frexp(top)
            scale = torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875).int())
        scale = scale.clamp(min=MIN_SCALE)
        s["scales"].copy_(scale)
        code = (wide / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
        s["codes"].copy_(code.view(n, -1).to(torch.float8_e4m3fn))
    return {k: s[k] for k in ("sum", "y", "codes", "scales") if s[k] is not None}


def _plain_sample(s):
    """Rows sorted once; every filter is a prefix of the order. Sums in 64 bits: a row's number
    may lie next to a border."""
    logits = s["logits"].float()
    rows, v = logits.shape
    temp = s["temperature"].double()
    greedy = temp <= 0
    top = logits.amax(1, keepdim=True)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    scale = torch.where(greedy, 1.0, 1.0 / torch.where(greedy, 1.0, temp))
    w = torch.exp((order.values.double() - top) * scale[:, None])
    rank = torch.arange(v, device=w.device)
    k = torch.where(s["top_k"] > 0, s["top_k"].long(), v)
    w = torch.where(rank < k[:, None], w, 0.0)
    before = torch.cumsum(w, 1) - w  # weight in front of each
    total = w.sum(1)
    off = s["top_p"] >= 1
    keep = off[:, None] | (before < (s["top_p"].double() * total)[:, None]) | (rank == 0)
    keep &= (rank < k[:, None]) & (w >= s["min_p"].double()[:, None])
    kept = torch.zeros_like(w).scatter_(1, order.indices, torch.where(keep, w, 0.0))
    cum = torch.cumsum(kept, 1)
    token = torch.searchsorted(cum, s["u"].double()[:, None] * cum[:, -1:], right=True)[:, 0]
    token = torch.where(greedy, order.indices[:, 0], token)
    s["token"].copy_(token)
    share = kept.gather(1, token[:, None])[:, 0] / cum[:, -1]
    s["logprob"].copy_(torch.where(greedy, 0.0, torch.log(share)))
    return dict(token=s["token"], logprob=s["logprob"])


_PLAIN = dict(conv=_plain_conv, conv_step=_plain_conv_step, ssm=_plain_ssm,
              ssm_step=_plain_ssm_step, norm=_plain_norm, sample=_plain_sample)


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    item = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "norm":
        cells = case["tokens"] * case["heads"] * case["dim"]
        groups = case["heads"] * case["dim"] // case["group"] if case["group"] else 1
        b = cells * item * (1 + 2 * case["residual"] + case["gate"])
        b += cells + 4 * groups * case["tokens"] if case["codes"] else cells * item
        return dict(bytes=b + 4 * case["dim"], flops=cells * (4 + 4 * case["gate"]))
    if op == "sample":
        cells = case["rows"] * case["vocab"]
        return dict(bytes=cells * item + 28 * case["rows"], flops=4 * cells)
    ch = case["ch"]
    if op in ("conv", "ssm"):
        lens = _lengths(case)
        tokens, reqs = sum(lens), len(lens)
        ckpt = sum(len(p) for p in _checkpoints(case, lens))
        reads = reqs - reqs // 2  # every other request starts from zeros
    else:
        tokens, reqs, ckpt, reads = case["batch"], case["batch"], 0, case["batch"]
    if op in ("conv", "conv_step"):
        state = (case["width"] - 1) * ch * item
        return dict(bytes=2 * tokens * ch * item + (reads + reqs + ckpt) * state
                    + 4 * ch * (case["width"] + case["bias"]) + 12 * reqs,
                    flops=tokens * ch * (2 * case["width"] + 4))
    n = case["n"]
    row = (3 + case["gate"]) * ch + 2 * case["groups"] * n
    return dict(bytes=tokens * row * item + (reads + reqs + ckpt) * ch * n * 4
                + 4 * ch * (n + 2) + 12 * reqs,
                flops=tokens * ch * (7 * n + 8 + 4 * case["gate"]))


# ---- the definitions in 64 bits ----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _gated(x):
    return x * torch.sigmoid(x)


def _spans(s):
    cu, ck = s["cu"].tolist(), s["ckpt_cu"].tolist()
    pos = s["ckpt_pos"].tolist()
    return [(lo, hi, list(zip(range(a, b), pos[a:b])), s["slot"][i].item(), bool(s["zero"][i]))
            for i, (lo, hi, a, b) in enumerate(zip(cu[:-1], cu[1:], ck[:-1], ck[1:]))]


def _exact_conv(case, s):
    w, weight = case["width"], s["weight"].double()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    pool, ckpt = s["pool"].double(), s["ckpt"].double()
    for lo, hi, marks, slot, zero in _spans(s):
        front = torch.zeros_like(pool[slot]) if zero else pool[slot].clone()
        line = torch.cat([front, s["x"][lo:hi].double()])
        win = line.unfold(0, w, 1)  # [n, C, W]
        out = (win * weight).sum(-1)
        y[lo:hi] = _gated(out if s["bias"] is None else out + s["bias"].double())
        for j, p in marks:
            ckpt[j] = line[p:p + w - 1]
        pool[slot] = line[hi - lo:]
    out = dict(y=y, pool=pool)
    return dict(out, ckpt=ckpt) if s["num_ckpt"] else out


def _exact_conv_step(case, s):
    pool, slot = s["pool"].double(), s["slot"].long()
    line = torch.cat([pool[slot], s["x"].double()[:, None]], dim=1)
    y = torch.einsum("bwc,cw->bc", line, s["weight"].double())
    pool[slot] = line[:, 1:]
    return dict(y=_gated(y if s["bias"] is None else y + s["bias"].double()), pool=pool)


def _scan64(s, case, rows, h, marks):
    """The recurrence of one request's rows (a slice), token by token; outputs, states at marks."""
    ch, g = case["ch"], case["groups"]
    skip, a = s["skip"].double(), s["a"].double()
    x, d = s["x"][rows].double(), s["delta"][rows].double() + s["delta_bias"].double()
    dt = torch.logaddexp(d, torch.zeros_like(d))
    bt = s["b"][rows].double().view(len(x), g, -1).repeat_interleave(ch // g, 1)
    ct = s["c"][rows].double().view(len(x), g, -1)
    y, held = torch.empty_like(x), {}
    for t in range(len(x)):
        h = torch.exp(dt[t, :, None] * a) * h + (dt[t] * x[t])[:, None] * bt[t]
        y[t] = torch.einsum("gcn,gn->gc", h.view(g, ch // g, -1), ct[t]).reshape(ch)
        for j, p in marks:
            if p == t + 1:
                held[j] = h
    y += skip * x
    if s["z"] is not None:
        y *= _gated(s["z"][rows].double())
    return y, h, held


def _exact_ssm(case, s):
    if s["tokens"] > 40000 or s["tokens"] * case["ch"] * case["n"] > 1 << 32:
        return None
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    pool, ckpt = s["pool"].double(), s["ckpt"].double()
    for lo, hi, marks, slot, zero in _spans(s):
        h = torch.zeros_like(pool[slot]) if zero else pool[slot].clone()
        piece = max(1, (1 << 26) // (case["ch"] * case["n"]))
        for t0 in range(lo, hi, piece):
            t1, at = min(hi, t0 + piece), t0 - lo
            y[t0:t1], h, held = _scan64(s, case, slice(t0, t1), h,
                                        [(j, p - at) for j, p in marks])
            for j, x in held.items():
                ckpt[j] = x
        pool[slot] = h
    out = dict(y=y, pool=pool)
    return dict(out, ckpt=ckpt) if s["num_ckpt"] else out


def _exact_ssm_step(case, s):
    pool, ch, g = s["pool"].double(), case["ch"], case["groups"]
    slot = s["slot"].long()
    d = s["delta"].double() + s["delta_bias"].double()
    dt = torch.logaddexp(d, torch.zeros_like(d))
    each = [s[k].double().view(len(slot), g, -1).repeat_interleave(ch // g, 1) for k in ("b", "c")]
    h = torch.exp(torch.einsum("bc,cn->bcn", dt, s["a"].double())) * pool[slot]
    h += torch.einsum("bc,bcn->bcn", dt * s["x"].double(), each[0])
    y = torch.einsum("bcn,bcn->bc", h, each[1]) + s["skip"].double() * s["x"].double()
    pool[slot] = h
    return dict(y=y if s["z"] is None else y * _gated(s["z"].double()), pool=pool)


def _exact_norm(case, s):
    """Codes as the quotients that they round: within half a step of what they stand for."""
    out = {}
    x = s["x"].double()
    if s["residual"] is not None:
        x = x + s["residual"].double()
        out["sum"] = x
    n = len(x)
    h = x.reshape(n, case["heads"], case["dim"])
    y = h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / case["dim"] + 1e-6) * s["weight"].double()
    y = y.reshape(n, -1)
    if s["gate"] is not None:
        y = y * _gated(s["gate"].double())
    if s["codes"] is None:
        return dict(out, y=y)
    wide = y.view(n, s["scales"].shape[1], -1)
    scale = wide.abs().max(-1).values / E4M3_MAX
    if case["pow2"]:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    scale = scale.clamp(min=MIN_SCALE)
    return dict(out, codes=(wide / scale[..., None]).view(n, -1), scales=scale)


def _exact_sample(case, s):
    """Log-probabilities of the drawn tokens, row by row on the host (tokens are whole numbers)."""
    host = {k: s[k].double().cpu().numpy() for k in ("logits", "temperature", "top_p", "min_p", "u")}
    limit, out = s["top_k"].tolist(), []
    for i, l in enumerate(host["logits"]):
        t = host["temperature"][i]
        if t <= 0:
            out.append(0.0)
            continue
        order = np.lexsort((np.arange(len(l)), -l))
        if limit[i] > 0:
            order = order[:limit[i]]
        p = np.exp((l[order] - l.max()) / t)
        if host["top_p"][i] < 1:
            part = np.cumsum(p)
            last = np.searchsorted(part, host["top_p"][i] * part[-1], side="left")
            order, p = order[:last + 1], p[:last + 1]
        order, p = order[p >= host["min_p"][i]], p[p >= host["min_p"][i]]
        by_index = np.argsort(order)
        part = np.cumsum(p[by_index])
        drawn = np.searchsorted(part, host["u"][i] * part[-1], side="right")
        out.append(math.log(p[by_index][drawn] / part[-1]))
    return dict(token=None, logprob=torch.tensor(out, dtype=torch.float64, device="cuda"))


_EXACT = dict(sample=_exact_sample, conv=_exact_conv, conv_step=_exact_conv_step, ssm=_exact_ssm,
              ssm_step=_exact_ssm_step, norm=_exact_norm)
