"""Rotary embedding and the quantising append against the plain fp64 reference."""
import numpy as np
import pytest

from oracle import attn_ref as A
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda

pytestmark = pytest.mark.gpu


def _dtype(torch, io):
    return (torch.bfloat16, gdn.GDN_BF16, 2.0 ** -8) if io == "bf16" else \
        (torch.float32, gdn.GDN_F32, 2.0 ** -24)


def _rope_tol(x, half_step):
    """Sine and cosine are off by at most 2^-22 (their own rounding and an angle known to
    2^-31 of a half turn), the two products and the sum by 2^-24 each; then one rounding."""
    return np.abs(x) * half_step


ROPES = [  # head dim, rotary dim, sections, interleaved, adjacent
    (256, 64, [11, 11, 10], True, False), (128, 128, [64], False, False),
    (64, 64, [16, 8, 8], False, True), (128, 32, [6, 5, 5], True, True),
    (64, 16, [2, 2, 2, 2], True, False), (256, 256, [128], False, False),
    (64, 48, [24, 0], True, False)]


@pytest.mark.parametrize("head_dim,rot,sections,inter,adjacent", ROPES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,hq,hk,in_place", [(1, 1, 1, False), (37, 5, 2, False),
                                                   (130, 16, 0, True), (3, 0, 3, True)])
def test_rope_against_fp64(head_dim, rot, sections, inter, adjacent, io, tokens, hq, hk, in_place):
    torch = torch_cuda()
    t, code, half = _dtype(torch, io)
    rng = np.random.default_rng(tokens + rot)
    theta = 1.0e7
    pos = rng.integers(0, 1 << 18, (len(sections), tokens)).astype(np.int32)
    pos[:, 0] = [2**31 - 1, -2**31, -1, 0][:len(sections)]
    # q and k are column ranges of one array with a gap behind them
    width = (hq + hk) * head_dim + 24
    qkv = torch.from_numpy(rng.standard_normal((tokens, width)).astype(np.float32)).cuda().to(t)
    q, k = qkv[:, :hq * head_dim], qkv[:, hq * head_dim:(hq + hk) * head_dim]
    keep = qkv.clone()
    out = qkv if in_place else torch.full((tokens, width), 7.0, dtype=t, device="cuda")
    qo, ko = out[:, :hq * head_dim], out[:, hq * head_dim:(hq + hk) * head_dim]
    rope = gdn.gdn_rope_init(head_dim, rot, sections, int(inter), int(adjacent), theta)
    p = torch.from_numpy(np.concatenate([pos, pos[:, :1]], 1)).cuda()  # a stride of its own
    gdn.gdn_rope_apply(handle(), rope, code, tokens, p, tokens + 1, q if hq else None, width, hq,
                       qo if hq else None, width, k if hk else None, width, hk,
                       ko if hk else None, width)
    torch.cuda.synchronize()
    x = keep.float().cpu().numpy().astype(np.float64)[:, :(hq + hk) * head_dim]
    x = x.reshape(tokens, hq + hk, head_dim)
    want = A.rope(x, pos, rot, sections, inter, adjacent, theta)
    got = out.float().cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(got[:, (hq + hk) * head_dim:],
                                  (keep if in_place else torch.full_like(keep, 7.0)).float().cpu()
                                  .numpy()[:, (hq + hk) * head_dim:])
    got = got[:, :(hq + hk) * head_dim].reshape(x.shape)
    pair = np.zeros_like(x)  # |x| + |y| of the element's pair
    h = rot // 2
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, h), slice(h, rot))
    pair[..., a] = pair[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    bound = _rope_tol(want, half) + pair * (2.0 ** -22 + 3 * 2.0 ** -24)
    assert (np.abs(got - want) <= bound).all()
    np.testing.assert_array_equal(got[..., rot:], x[..., rot:])


def test_rope_with_given_frequencies_passes_other_values_through():
    """Frequencies of the caller's own; NaN and infinities outside the rotated part pass."""
    torch = torch_cuda()
    freq = np.linspace(0, 6.2, 16)
    rope = gdn.gdn_rope_init(64, 32, [16], inv_freq=freq)
    x = torch.randn(9, 2, 64, device="cuda")
    x[:, :, 40], x[:, :, 41], x[:, :, 42] = float("nan"), float("inf"), -0.0
    pos = torch.arange(100, 109, dtype=torch.int32, device="cuda")[None]
    out = torch.empty_like(x)
    gdn.gdn_rope_apply(handle(), rope, gdn.GDN_F32, 9, pos, 9, x, 128, 2, out, 128, None, 0, 0,
                       None, 0)
    torch.cuda.synchronize()
    assert torch.equal(out[..., 32:].view(torch.int32), x[..., 32:].view(torch.int32))
    x64 = x.cpu().numpy().astype(np.float64)
    want = A.rope(x64, pos.cpu().numpy(), 32, [16], False, False, inv_freq=freq)
    got = out.cpu().numpy()
    err = np.abs(got[..., :32] - want[..., :32])
    pair = np.abs(x64[..., :16]) + np.abs(x64[..., 16:32])
    bound = np.concatenate([pair, pair], -1) * (2.0 ** -22 + 4 * 2.0 ** -24)
    assert (err <= bound).all()


def _cache(rng, pages, heads, page, dim):
    codes = [rng.integers(0, 256, (pages, heads, page, dim)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 0
    scales = [(2.0 ** rng.integers(-12, -4, (pages, heads))).astype(np.float32) for _ in range(2)]
    return codes, scales


def _append(torch, codes, scales, slots, k, v, io, *, rope=None, pos=None, q=None, stream=None):
    """k, v: torch [T, H, D] (any strides over tokens). Returns codes and scales."""
    _, code, _ = _dtype(torch, io)
    c = [torch.from_numpy(x.copy()).cuda() for x in codes]
    s = [torch.from_numpy(x.copy()).cuda() for x in scales]
    cache = gdn.make_kv_cache(c[0], c[1], s[0], s[1])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(np.asarray(slots, np.int64)).cuda()
    qo = None
    rest = ()
    if rope is not None:
        rest = (rope, pos, pos.shape[1])
        if q is not None:
            qo = torch.empty(q.shape, dtype=q.dtype, device="cuda")
            rest += (q, q.stride(0), q.shape[1], qo, qo.stride(0))
    rest = rest + (None, None, 0, None, 0, 0, None, 0)[len(rest):]
    gdn.gdn_kv_append(handle(), cache, code, len(slots), sl, k, k.stride(0), v, v.stride(0),
                      *rest, status, stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in c], [x.cpu().numpy() for x in s], qo, int(status.item())


def _slots(rng, page, runs, pages):
    """Slots of requests' new tokens: runs of (offset in the first page, tokens)."""
    order, at, out = rng.permutation(pages), 0, []
    for off, n in runs:
        pos = off
        while n > 0:
            m = min(n, page - pos)
            out += [int(order[at]) * page + pos + i for i in range(m)]
            at, n, pos = at + 1, n - m, 0
    return out, at


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("head_dim,heads,page,runs", [
    (64, 1, 16, [(0, 1)]), (64, 3, 16, [(3, 1), (15, 1), (0, 40)]),
    (128, 2, 32, [(31, 70), (0, 32), (5, 2)]), (128, 8, 64, [(10, 1), (0, 200), (63, 1)]),
    (256, 2, 64, [(0, 64), (1, 63), (2, 300)]), (256, 1, 128, [(0, 128), (100, 300), (7, 1)]),
    (128, 1, 128, [(i, 1) for i in range(0, 128, 5)]), (256, 2, 16, [(i, 2) for i in range(16)])])
def test_append_matches_the_reference_bit_for_bit(io, head_dim, heads, page, runs):
    torch = torch_cuda()
    rng = np.random.default_rng(head_dim + page)
    pages = sum(-(-(o + n) // page) for o, n in runs) + 2
    slots, used = _slots(rng, page, runs, pages)
    T = len(slots)
    codes, scales = _cache(rng, pages, heads, page, head_dim)
    t, _, _ = _dtype(torch, io)
    # magnitudes from row to row so that scales grow in some pages and not in others
    x = rng.standard_normal((2, T, heads, head_dim)) * 2.0 ** rng.integers(-6, 6, (2, T, 1, 1))
    fused = torch.from_numpy(x.astype(np.float32)).cuda().to(t).permute(1, 0, 2, 3).contiguous()
    k, v = fused[:, 0], fused[:, 1]  # strides of a fused projection
    got_c, got_s, _, status = _append(torch, codes, scales, slots, k, v, io)
    assert status == 0
    kk, vv = (y.float().cpu().numpy().astype(np.float64) for y in (k, v))
    want = A.append(codes[0], codes[1], scales[0], scales[1], slots, kk, vv)
    for i in range(2):
        np.testing.assert_array_equal(got_s[i].astype(np.float64), want[2 + i])
        # +0 and -0 codes of values that rounded to zero count as equal
        np.testing.assert_array_equal(A.e4m3_values()[got_c[i]], A.e4m3_values()[want[i]])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_append_of_zeros_tiny_huge_infinite_and_nan_values(io):
    torch = torch_cuda()
    rng = np.random.default_rng(9)
    t, _, _ = _dtype(torch, io)
    page, heads, dim = 16, 2, 64
    rows = [np.zeros(dim), np.full(dim, 448.0), np.full(dim, 449.0), np.full(dim, 1e-38),
            np.full(dim, 3e38), rng.standard_normal(dim), rng.standard_normal(dim),
            rng.standard_normal(dim), rng.standard_normal(dim)]
    rows[5][3], rows[6][0], rows[7][7] = np.inf, -np.inf, np.nan
    rows[8][:] = np.nan
    n = len(rows)
    codes, scales = _cache(rng, 2 * n, heads, page, dim)
    x = np.stack(rows)[:, None].repeat(heads, 1)
    clean = rng.standard_normal((n, heads, dim))
    for a, b in ((x, clean), (clean, x), (x, x)):
        for slots in ([page * i for i in range(n)], [page * i + 5 for i in range(n)],
                      list(range(n))):
            k, v = (torch.from_numpy(y.astype(np.float32)).cuda().to(t) for y in (a, b))
            got_c, got_s, _, status = _append(torch, codes, scales, slots, k, v, io)
            assert status == 0
            want = A.append(codes[0], codes[1], scales[0], scales[1], slots,
                            k.double().cpu().numpy(), v.double().cpu().numpy())
            for i in range(2):
                np.testing.assert_array_equal(got_s[i].astype(np.float64), want[2 + i])
                np.testing.assert_array_equal(A.e4m3_values()[got_c[i]],
                                              A.e4m3_values()[want[i]])


def test_append_skips_negative_slots_and_flags_those_out_of_range():
    torch = torch_cuda()
    rng = np.random.default_rng(10)
    codes, scales = _cache(rng, 4, 2, 16, 64)
    slots = [-1, 5, 6, -1, 64, 2**40, 63, -2**40, 32, 33]
    k, v = (torch.randn(len(slots), 2, 64, device="cuda") for _ in range(2))
    got_c, got_s, _, status = _append(torch, codes, scales, slots, k, v, "f32")
    assert status == gdn.GDN_ERR_INVALID_ARGUMENT
    want = A.append(codes[0], codes[1], scales[0], scales[1], slots, k.double().cpu().numpy(),
                    v.double().cpu().numpy())
    for i in range(2):
        np.testing.assert_array_equal(got_s[i].astype(np.float64), want[2 + i])
        np.testing.assert_array_equal(A.e4m3_values()[got_c[i]], A.e4m3_values()[want[i]])


def test_append_token_by_token_grows_scales_like_the_reference():
    """The page's scale only grows, and the codes in front are rounded again when it does."""
    torch = torch_cuda()
    rng = np.random.default_rng(11)
    codes, scales = _cache(rng, 3, 2, 16, 128)
    want = codes[0], codes[1], scales[0], scales[1]
    got_c, got_s = codes, scales
    for i in range(20):
        x = (rng.standard_normal((2, 1, 2, 128)) * 2.0 ** rng.integers(-9, 9)).astype(np.float32)
        slot = [16 + i] if i < 16 else [2 * 16 + i - 16]
        k, v = (torch.from_numpy(y).cuda() for y in x)
        got_c, got_s, _, _ = _append(torch, got_c, got_s, slot, k, v, "f32")
        want = A.append(*want, slot, x[0].astype(np.float64), x[1].astype(np.float64))
        for j in range(2):
            np.testing.assert_array_equal(got_s[j].astype(np.float64), want[2 + j])
            np.testing.assert_array_equal(A.e4m3_values()[got_c[j]], A.e4m3_values()[want[j]])


@pytest.mark.parametrize("head_dim,rot,sections,inter,adjacent", ROPES)
@pytest.mark.parametrize("io,hq,runs", [("bf16", 4, [(0, 70), (9, 1), (3, 30)]),
                                        ("f32", 0, [(0, 16), (15, 2)]), ("bf16", 3, [(2, 1)])])
def test_append_with_rotation(head_dim, rot, sections, inter, adjacent, io, hq, runs):
    """The rotated key is quantised from fp32 without a rounding between: every stored value is
    within half an e4m3 step of the exact one, and q is rotated as gdn_rope_apply rotates it."""
    torch = torch_cuda()
    rng = np.random.default_rng(rot + hq)
    t, code, _ = _dtype(torch, io)
    page, heads, theta = 16, 2, 5.0e5
    slots, used = _slots(rng, page, runs, 20)
    T = len(slots)
    codes, scales = _cache(rng, 20, heads, page, head_dim)
    width = (hq + 2 * heads) * head_dim
    qkv = torch.from_numpy(rng.standard_normal((T, width)).astype(np.float32)).cuda().to(t)
    q = qkv[:, :hq * head_dim].view(T, hq, head_dim)
    k = qkv[:, hq * head_dim:(hq + heads) * head_dim].view(T, heads, head_dim)
    v = qkv[:, (hq + heads) * head_dim:].view(T, heads, head_dim)
    pos_np = rng.integers(0, 1 << 18, (len(sections), T)).astype(np.int32)
    pos = torch.from_numpy(pos_np).cuda()
    rope = gdn.gdn_rope_init(head_dim, rot, sections, int(inter), int(adjacent), theta)
    got_c, got_s, qo, status = _append(torch, codes, scales, slots, k, v, io, rope=rope, pos=pos,
                                       q=q if hq else None)
    assert status == 0
    k64 = k.double().cpu().numpy()
    turned = A.rope(k64, pos_np, rot, sections, inter, adjacent, theta)
    want = A.append(codes[0], codes[1], scales[0], scales[1], slots, turned,
                    v.double().cpu().numpy())
    np.testing.assert_array_equal(got_s[1].astype(np.float64), want[3])
    np.testing.assert_array_equal(A.e4m3_values()[got_c[1]], A.e4m3_values()[want[1]])
    # scales: equal, or a power of two apart where the largest value sits on the border
    ratio = got_s[0].astype(np.float64) / want[2]
    assert np.isin(ratio, [0.5, 1.0, 2.0]).all() and (ratio == 1).mean() > 0.9
    for tkn, s in enumerate(slots):
        p, off = divmod(s, page)
        for h in range(heads):
            sc = float(got_s[0][p, h])
            x = turned[tkn, h]
            got = A.e4m3_values()[got_c[0][p, h, off]] * sc
            # half a step is at most 2^-4 of the value, or half the smallest step 2^-9; the
            # rotation itself is off by 2^-22 + 3 * 2^-24 of its pair (at most sqrt(2) |pair|)
            slack = 8 * np.abs(k64[tkn, h]).max() * 2.0 ** -22
            assert (np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
                    + slack).all()
    if hq:
        alone = torch.empty_like(qo)
        gdn.gdn_rope_apply(handle(), rope, code, T, pos, T, q, width, hq, alone,
                           hq * head_dim, None, 0, 0, None, 0)
        torch.cuda.synchronize()
        assert torch.equal(alone, qo)
