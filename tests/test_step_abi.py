"""The calls around the recurrent layers on the host: sizes and every refusal (validation comes
before any CUDA call, and a NULL handle is the last thing checked)."""
import ctypes

import pytest

from packed_linear_attention_gb300 import build, gdn

INVALID, UNSUPPORTED = gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED
SMALL = gdn.GDN_ERR_WORKSPACE_TOO_SMALL
GB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return gdn.load()


def P(i):
    """Distinct fake device ranges, never touched."""
    return GB * (i + 1)


def requests(**kw):
    d = dict(num_seqs=4, num_tokens=100, max_len=50, num_slots=8, cu=P(20), slot_idx=P(21),
             start_zero=P(22), ckpt_cu=P(23), ckpt_pos=P(24), num_ckpt=3)
    d.update(kw)
    return gdn.gdn_requests(*(d[name] for name, _ in gdn.gdn_requests._fields_))


BAD_REQUESTS = (dict(num_seqs=0), dict(num_tokens=-1), dict(max_len=-1), dict(num_slots=0),
                dict(num_ckpt=-1), dict(cu=None), dict(cu=P(20) + 2), dict(slot_idx=P(21) + 1),
                dict(start_zero=P(22) + 2), dict(ckpt_cu=P(23) + 2), dict(ckpt_pos=None),
                dict(ckpt_pos=P(24) + 1), dict(slot_idx=None, num_slots=3))


# ---- convolution ----

def conv_config(**kw):
    d = dict(channels=96, width=4, activation=1, io_dtype=gdn.GDN_BF16, weight=P(10), bias=P(11))
    d.update(kw)
    return gdn.gdn_conv_config(*(d[name] for name, _ in gdn.gdn_conv_config._fields_))


BAD_CONV = (dict(channels=0), dict(width=0), dict(activation=2), dict(io_dtype=5),
            dict(weight=None), dict(weight=P(10) + 2), dict(bias=P(11) + 1))


def conv(cfg=None, req=None, **kw):
    d = dict(x=P(0), xs=96, y=P(1), ys=96, pool=P(2), ckpt=P(3), status=P(4))
    d.update(kw)
    return gdn.gdn_conv_packed(None, cfg or conv_config(), req or requests(), d["x"], d["xs"],
                               d["y"], d["ys"], d["pool"], d["ckpt"], d["status"],
                               raise_on_error=False)


# a call too large for a grid: refused after every other check
BIG = dict(num_seqs=4096, num_slots=5000, num_tokens=1 << 30)
WIDE = dict(channels=1 << 15)
FAR = dict(x=1 << 50, xs=1 << 15, y=1 << 54, ys=1 << 15, pool=P(2), ckpt=P(8000))


def test_conv_refusals():
    cfg, big = conv_config(**WIDE), requests(**BIG)
    assert conv() == INVALID  # the NULL handle
    assert conv(cfg, big, **FAR) == UNSUPPORTED
    assert conv(req=requests(num_seqs=4097, num_slots=5000)) == UNSUPPORTED
    assert conv(cfg=conv_config(width=5)) == UNSUPPORTED
    assert conv(cfg=conv_config(width=1)) == UNSUPPORTED
    assert gdn.load().gdn_conv_packed(None, None, ctypes.byref(big), P(0), 96, P(1), 96,
                                      P(2), P(3), None, None) == INVALID
    for kw in BAD_CONV:
        assert conv(conv_config(**dict(WIDE, **kw)), big, **FAR) == INVALID, kw
    for kw in BAD_REQUESTS:
        assert conv(cfg, requests(**dict(BIG, **kw)), **FAR) == INVALID, kw
    for kw in (dict(x=None), dict(x=(1 << 50) + 8), dict(xs=(1 << 15) - 8), dict(xs=(1 << 15) + 4),
               dict(y=None), dict(ys=88), dict(pool=None), dict(pool=P(2) + 4), dict(ckpt=None),
               dict(ckpt=P(8000) + 8), dict(status=P(4) + 2), dict(y=1 << 50),
               dict(y=(1 << 50) + 96), dict(pool=1 << 50), dict(pool=(1 << 54) + 1600),
               dict(ckpt=P(2)), dict(ckpt=1 << 54)):
        assert conv(cfg, big, **dict(FAR, **kw)) == INVALID, kw


def test_what_a_convolution_accepts():
    cfg, big = conv_config(**WIDE), requests(**BIG)
    plain = requests(**dict(BIG, ckpt_cu=None, ckpt_pos=None, start_zero=None))
    assert conv(cfg, plain, **dict(FAR, ckpt=None, status=None)) == UNSUPPORTED
    assert conv(conv_config(bias=None, **WIDE), big, **FAR) == UNSUPPORTED
    # column ranges of one array lie apart
    assert conv(cfg, big, **dict(FAR, xs=1 << 16, y=(1 << 50) + (1 << 16), ys=1 << 16)) == UNSUPPORTED
    assert conv(cfg, big, **dict(FAR, xs=1 << 16, y=(1 << 50) + (1 << 15), ys=1 << 16)) == INVALID


def test_conv_step_refusals():
    def call(cfg=None, batch=8, x=P(0), xs=96, y=P(1), ys=96, pool=P(2), slots=9, idx=P(3),
             status=P(4)):
        return gdn.gdn_conv_step(None, cfg or conv_config(), batch, x, xs, y, ys, pool, slots, idx,
                                 status, raise_on_error=False)
    assert call() == INVALID
    wide = conv_config(channels=1 << 24)
    far = dict(cfg=wide, batch=1 << 20, x=1 << 50, xs=1 << 24, y=1 << 54, ys=1 << 24, slots=1,
               pool=P(0))
    assert call(**far) == UNSUPPORTED and call(**dict(far, y=1 << 50)) == UNSUPPORTED  # in place
    for kw in (dict(batch=-1), dict(x=None), dict(xs=104), dict(y=P(0) + 16), dict(pool=None),
               dict(slots=0), dict(idx=None), dict(idx=P(3) + 2), dict(status=P(4) + 1),
               dict(pool=1 << 50)):
        if "xs" in kw:
            kw = dict(xs=(1 << 24) + 4)
        if "y" in kw:
            kw = dict(y=(1 << 50) + 16)
        assert call(**dict(far, **kw)) == INVALID, kw


# ---- selective scan ----

def ssm_config(**kw):
    d = dict(channels=64, num_groups=2, state_dim=16, io_dtype=gdn.GDN_BF16, delta_softplus=1,
             a=P(10), d=P(11), delta_bias=P(12))
    d.update(kw)
    return gdn.gdn_ssm_config(*(d[name] for name, _ in gdn.gdn_ssm_config._fields_))


def ssm_rows(**kw):
    d = dict(x=P(0), delta=P(1), b=P(2), c=P(3), z=P(4), y=P(5), x_stride=64, delta_stride=64,
             b_stride=32, c_stride=32, z_stride=64, y_stride=64)
    d.update(kw)
    return gdn.gdn_ssm_rows(*(d[name] for name, _ in gdn.gdn_ssm_rows._fields_))


BAD_SSM = (dict(channels=0), dict(num_groups=0), dict(num_groups=3), dict(state_dim=0),
           dict(io_dtype=-1))
BAD_SSM_ARRAYS = (dict(a=None), dict(a=P(10) + 4), dict(d=P(11) + 2), dict(delta_bias=P(12) + 1))
BAD_ROWS = (dict(x=None), dict(x=P(0) + 4), dict(x_stride=63), dict(x_stride=68), dict(delta=None),
            dict(delta_stride=32), dict(b=None), dict(b=P(2) + 1), dict(b_stride=31), dict(c=None),
            dict(c_stride=16), dict(z=P(4) + 8), dict(z_stride=60), dict(y=None), dict(y=P(0) + 16),
            dict(y=P(0), y_stride=72), dict(y=P(2)), dict(y=P(3) + 64), dict(y=P(4) + 128))


def test_ssm_refusals():
    def call(cfg=None, req=None, rows=None, pool=P(6), ckpt=P(7), work=P(8), size=1 << 20,
             status=P(9)):
        return gdn.gdn_ssm_packed(None, cfg or ssm_config(), req or requests(), rows or ssm_rows(),
                                  pool, ckpt, work, size, status, raise_on_error=False)
    assert call() == INVALID
    assert call(size=255) == SMALL  # the last check but the handle's
    assert call(req=requests(num_seqs=4097, num_slots=5000)) == UNSUPPORTED
    assert call(cfg=ssm_config(state_dim=129), rows=ssm_rows(b_stride=300, c_stride=300)) == UNSUPPORTED
    for kw in BAD_SSM + BAD_SSM_ARRAYS:
        assert call(cfg=ssm_config(**kw), size=0) == INVALID, kw
    for kw in BAD_REQUESTS:
        assert call(req=requests(**kw), size=0) == INVALID, kw
    for kw in BAD_ROWS:
        assert call(rows=ssm_rows(**kw), size=0) == INVALID, kw
    for kw in (dict(pool=None), dict(pool=P(6) + 4), dict(ckpt=None), dict(ckpt=P(7) + 8),
               dict(work=None), dict(work=P(8) + 16), dict(status=P(9) + 1), dict(pool=P(0)),
               dict(pool=P(5) + 16), dict(ckpt=P(6)), dict(ckpt=P(3)), dict(work=P(6)),
               dict(work=P(4))):
        assert call(size=0, **kw) == INVALID, kw
    # in place over x, delta or z; no gate, no checkpoints, no rows
    for kw in (dict(y=P(0)), dict(y=P(1)), dict(y=P(4)), dict(z=None), dict(b=P(2) + 2)):
        assert call(rows=ssm_rows(**kw), size=0) == SMALL, kw
    assert call(cfg=ssm_config(d=None, delta_bias=None), ckpt=None, size=0,
                req=requests(ckpt_cu=None, ckpt_pos=None, start_zero=None)) == SMALL
    assert call(req=requests(num_tokens=0), rows=ssm_rows(x=None, y=None, b=None), size=0) == SMALL


def test_ssm_workspace():
    def size(cfg=None, **kw):
        return gdn.gdn_ssm_workspace_size(cfg or ssm_config(), requests(**kw))
    assert size() == 256
    long = dict(num_seqs=1, num_tokens=32768, max_len=32768)
    n = size(**long)
    assert n % 256 == 0 and n > 64 * 16 * 4
    # many channels fill the GPU by themselves
    assert size(ssm_config(channels=1 << 17), **long) == 256
    for kw in BAD_SSM:
        with pytest.raises(gdn.GdnError):
            size(ssm_config(**kw))
    with pytest.raises(gdn.GdnError):
        size(num_seqs=0)
    assert gdn.load().gdn_ssm_workspace_size(ctypes.byref(ssm_config()),
                                             ctypes.byref(requests()), None) == INVALID


def test_ssm_step_refusals():
    def call(cfg=None, batch=8, rows=None, pool=P(6), slots=9, idx=P(7), status=P(9)):
        return gdn.gdn_ssm_step(None, cfg or ssm_config(), batch, rows or ssm_rows(), pool, slots,
                                idx, status, raise_on_error=False)
    assert call() == INVALID
    assert call(cfg=ssm_config(state_dim=130), rows=ssm_rows(b_stride=300, c_stride=300)) == UNSUPPORTED
    far = dict(cfg=ssm_config(channels=1 << 24, num_groups=1, state_dim=1), batch=1 << 20, slots=1,
               rows=ssm_rows(x=1 << 50, delta=1 << 51, z=1 << 52, y=1 << 53, b=1 << 54, c=1 << 55,
                             x_stride=1 << 24, delta_stride=1 << 24, z_stride=1 << 24,
                             y_stride=1 << 24))
    assert call(**far) == UNSUPPORTED
    for kw in (dict(batch=-1), dict(pool=None), dict(pool=P(6) + 8), dict(slots=0),
               dict(idx=None), dict(idx=P(7) + 1), dict(status=P(9) + 2), dict(pool=1 << 53)):
        assert call(**dict(far, **kw)) == INVALID, kw
    wide = {name: getattr(far["rows"], name) for name, _ in gdn.gdn_ssm_rows._fields_}
    for kw in (dict(x=None), dict(x=(1 << 50) + 4), dict(x_stride=(1 << 24) + 4), dict(delta=None),
               dict(b=None), dict(b=(1 << 54) + 1), dict(b_stride=0), dict(c_stride=0), dict(y=None),
               dict(z=(1 << 52) + 8), dict(y=(1 << 50) + 16), dict(y=1 << 54)):
        assert call(**dict(far, rows=ssm_rows(**dict(wide, **kw)))) == INVALID, kw
    for kw in (dict(y=1 << 50), dict(y=1 << 51), dict(y=1 << 52), dict(z=None)):  # in place
        assert call(**dict(far, rows=ssm_rows(**dict(wide, **kw)))) == UNSUPPORTED, kw


# ---- norm ----

def norm_config(**kw):
    d = dict(num_heads=1, dim=256, io_dtype=gdn.GDN_BF16, scale_group=0, scale_pow2=0, eps=1e-6,
             weight_offset=0.0, weight=P(10))
    d.update(kw)
    return gdn.gdn_norm_config(*(d[name] for name, _ in gdn.gdn_norm_config._fields_))


def test_norm_refusals():
    def call(cfg=None, tokens=10, x=P(0), xs=256, r=P(1), rs=256, s=P(2), ss=256, g=P(3), gs=256,
             y=P(4), ys=256, c=P(5), cs=256, k=P(6)):
        return gdn.gdn_rms_norm(None, cfg or norm_config(), tokens, x, xs, r, rs, s, ss, g, gs, y,
                                ys, c, cs, k, raise_on_error=False)
    odd = dict(num_heads=4, dim=96)  # refused after everything else
    wide = dict(xs=384, rs=384, ss=384, gs=384, ys=384, cs=384)
    assert call() == INVALID  # the NULL handle
    assert call(norm_config(**odd), **wide) == UNSUPPORTED
    for kw in (dict(dim=32769), dict(dim=256, num_heads=200), dict(dim=256, scale_group=16)):
        w = kw["dim"] * kw.get("num_heads", 1) // 16 * 16 + 16
        rows = dict(xs=w, rs=w, ss=w, gs=w, ys=w, cs=w)
        assert call(norm_config(**kw), **rows) == UNSUPPORTED, kw
    for kw in (dict(num_heads=0), dict(dim=0), dict(io_dtype=9), dict(scale_group=-1),
               dict(scale_group=64), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(weight_offset=float("nan")), dict(weight=P(10) + 4)):
        assert call(norm_config(**dict(odd, **kw)), **wide) == INVALID, kw
    for kw in (dict(tokens=-1), dict(k=None), dict(c=None), dict(y=None, c=None, k=None),
               dict(r=None), dict(x=None), dict(x=P(0) + 2), dict(xs=388), dict(r=P(1) + 8),
               dict(rs=383), dict(g=P(3) + 4), dict(ys=128), dict(c=P(5) + 8), dict(cs=392),
               dict(k=P(6) + 2), dict(s=P(0) + 512), dict(y=P(1), ys=392), dict(y=P(2)),
               dict(c=P(0)), dict(k=P(4)), dict(c=P(6)), dict(c=P(2))):
        assert call(norm_config(**odd), **dict(wide, **kw)) == INVALID, kw
    for kw in (dict(s=P(0)), dict(s=P(1)), dict(s=P(3)), dict(y=P(0)), dict(y=P(1), s=None),
               dict(r=None, s=None), dict(g=None), dict(y=None), dict(c=None, k=None),
               dict(tokens=0, x=None)):
        assert call(norm_config(**odd), **dict(wide, **kw)) == UNSUPPORTED, kw


# ---- sampling ----

def test_sample_refusals():
    def call(io=gdn.GDN_F32, rows=4, vocab=1000, logits=P(0), stride=1000, t=P(1), k=P(2), p=P(3),
             m=P(4), u=P(5), token=P(6), lp=P(7), status=P(8)):
        return gdn.gdn_sample(None, io, rows, vocab, logits, stride, t, k, p, m, u, token, lp,
                              status, raise_on_error=False)
    assert call() == INVALID
    big = dict(vocab=(1 << 18) + 1, stride=1 << 19)
    assert call(**big) == UNSUPPORTED
    assert call(t=None, k=None, p=None, m=None, lp=None, status=None, **big) == UNSUPPORTED
    assert call(rows=(1 << 24) + 1, vocab=1, stride=1, logits=1 << 50) == UNSUPPORTED
    assert call(rows=0, logits=None, u=None, token=None, **big) == UNSUPPORTED
    for kw in (dict(io=7), dict(rows=-1), dict(vocab=0), dict(logits=None), dict(logits=P(0) + 2),
               dict(stride=900), dict(t=P(1) + 2), dict(k=P(2) + 1), dict(p=P(3) + 2),
               dict(m=P(4) + 1), dict(u=None), dict(u=P(5) + 1), dict(token=None),
               dict(token=P(6) + 2), dict(lp=P(7) + 2), dict(status=P(8) + 1), dict(token=P(0)),
               dict(lp=P(6)), dict(token=P(5) + 4), dict(lp=P(2))):
        assert call(**dict(big, **kw)) == INVALID, kw
    assert call(io=gdn.GDN_BF16, logits=P(0) + 2, **big) == UNSUPPORTED


# ---- the Python records ----

def test_records_need_fp32_weights():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        gdn.make_conv_config(torch.zeros(4, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gdn.make_conv_config(torch.zeros(4, 8)[:, ::2])
    with pytest.raises(ValueError):
        gdn.make_ssm_config(torch.zeros(4))
    with pytest.raises(ValueError):
        gdn.make_norm_config(4, torch.zeros(4, dtype=torch.float64))
