"""The full-attention layers' calls on the host: sizes, the rotary table and every refusal
(validation comes before any CUDA call, and a NULL handle is the last thing checked)."""
import ctypes

import numpy as np
import pytest

from oracle import attn_ref as A
from packed_linear_attention_gb300 import build, gdn

INVALID, UNSUPPORTED = gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED
MB = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return gdn.load()


def P(i):
    """Distinct fake device ranges, never touched."""
    return MB * (i + 1)


# ---- rotary table ----

@pytest.mark.parametrize("rot,sections,inter", [
    (64, [11, 11, 10], True), (64, [32], False), (32, [6, 5, 5], True), (128, [16, 24, 24], False),
    (16, [2, 2, 2, 2], True), (48, [24, 0], True), (256, [100, 0, 28], False)])
def test_rope_table(rot, sections, inter):
    rope = gdn.gdn_rope_init(256, rot, sections, int(inter), gdn.GDN_ROPE_ADJACENT, 1e6)
    half = rot // 2
    assert list(rope.axis[:half]) == A.rope_axes(half, sections, inter)
    wide = np.longdouble
    f = wide(1e6) ** (wide(-2) * np.arange(half) / wide(rot)) / (8 * np.arctan(wide(1)))
    got = np.array([wide(int(x)) for x in rope.turns[:half]]) / wide(2) ** 64
    assert (np.abs(got - f) <= wide(2) ** -61).all()
    assert (rope.head_dim, rope.rotary_dim, rope.num_axes, rope.pair_layout) == \
        (256, rot, len(sections), 1)


def test_rope_refusals():
    lib = gdn.load()
    r = gdn.gdn_rope()
    sec = (ctypes.c_int32 * 5)(8, 8, 8, 8, 0)
    f = (ctypes.c_double * 32)(*([0.5] * 32))

    def call(rope=r, dim=128, rot=64, axes=4, sections=sec, layout=0, pairs=0, theta=1e4, freq=None):
        return lib.gdn_rope_init(None if rope is None else ctypes.byref(rope), dim, rot, axes,
                                 sections, layout, pairs, theta, freq)

    assert call() == 0 and call(freq=f, theta=0.0) == 0
    assert call(rope=None) == INVALID and call(sections=None) == INVALID
    for kw in (dict(rot=0), dict(rot=63), dict(rot=130), dict(axes=0), dict(axes=3),
               dict(layout=2), dict(pairs=-1), dict(theta=0.5), dict(theta=float("nan")),
               dict(rot=-16), dict(dim=0, rot=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dim=96), dict(axes=5), dict(rot=24, axes=1)):
        assert call(**kw) == UNSUPPORTED, kw
    sec[0] = -8
    assert call() == INVALID
    # an axis with more pairs than turns cannot be laid out in turns
    assert call(axes=2, sections=(ctypes.c_int32 * 2)(8, 24), layout=1) == INVALID
    f[3] = 7.0
    assert call(axes=1, sections=(ctypes.c_int32 * 1)(32), freq=f) == INVALID
    f[3] = -0.1
    assert call(axes=1, sections=(ctypes.c_int32 * 1)(32), freq=f) == INVALID


# ---- plan and release ----

def _plan(**kw):
    d = dict(page=16, seqs=4, tokens=100, ctx=P(0), new=P(1), table=P(2), blocks=8, pages=50,
             free=P(3), count=P(4), out=P(5), cu=P(6), kv=P(7), pos=P(8), slots=P(9), status=P(10))
    d.update(kw)
    return gdn.gdn_kv_plan(None, d["page"], d["seqs"], d["tokens"], d["ctx"], d["new"], d["table"],
                           d["blocks"], d["pages"], d["free"], d["count"], d["out"], d["cu"],
                           d["kv"], d["pos"], d["slots"], d["status"], raise_on_error=False)


def test_plan_refusals():
    assert _plan() == INVALID  # the NULL handle
    assert _plan(seqs=4097, ) == UNSUPPORTED and _plan(page=48) == UNSUPPORTED
    for kw in (dict(page=0), dict(seqs=0), dict(tokens=-1), dict(blocks=0), dict(pages=0),
               dict(ctx=None), dict(new=None), dict(table=None), dict(free=None), dict(count=None),
               dict(out=None), dict(cu=None), dict(kv=None), dict(slots=None), dict(ctx=P(0) + 2),
               dict(slots=P(9) + 4), dict(status=P(10) + 1)):
        assert _plan(seqs=kw.pop("seqs", 4097), **kw) == INVALID, kw  # before the size check
    # outputs over inputs or over one another
    for kw in (dict(kv=P(0)), dict(cu=P(1)), dict(table=P(3)), dict(slots=P(8)), dict(kv=P(6) + 4)):
        assert _plan(seqs=4097, **kw) == INVALID, kw
    # the count may be updated in place, positions and status may be missing
    assert _plan(seqs=4097, out=P(4), pos=None, status=None) == UNSUPPORTED


def test_release_refusals():
    def call(page=16, seqs=4, kv=P(0), flags=P(1), table=P(2), blocks=4, pages=9, free=P(3),
             count=P(4), status=P(5)):
        return gdn.gdn_kv_release(None, page, seqs, kv, flags, table, blocks, pages, free, count,
                                  status, raise_on_error=False)
    assert call() == INVALID and call(seqs=5000) == UNSUPPORTED and call(page=8) == UNSUPPORTED
    for kw in (dict(page=-1), dict(blocks=0), dict(pages=0), dict(kv=None), dict(flags=None),
               dict(table=None), dict(free=None), dict(count=None), dict(free=P(3) + 1)):
        assert call(seqs=5000, **kw) == INVALID, kw
    assert call(seqs=0) == INVALID


# ---- rotation ----

def _rope_call(rope=None, io=gdn.GDN_BF16, tokens=10, pos=P(0), ps=10, q=P(1), qs=512, hq=4,
               qo=P(2), qos=512, k=P(3), ks=256, hk=2, ko=P(4), kos=256, **bad):
    rope = rope or gdn.gdn_rope_init(128, 64, [32])
    for name, value in bad.items():
        setattr(rope, name, value)
    return gdn.gdn_rope_apply(None, rope, io, tokens, pos, ps, q, qs, hq, qo, qos, k, ks, hk, ko,
                              kos, raise_on_error=False)


BIG = 1 << 21  # heads: more than the call takes, refused after every other check


def test_rope_apply_refusals():
    assert _rope_call() == INVALID  # the NULL handle
    ok = dict(hq=BIG, qs=BIG * 128, qos=BIG * 128, qo=1 << 50, k=None, hk=0, ko=None)
    assert _rope_call(**ok) == UNSUPPORTED
    assert _rope_call(**{**ok, "qo": P(1)}) == UNSUPPORTED      # in place
    for kw in (dict(io=5), dict(tokens=-1), dict(hk=-1), dict(pos=None), dict(ps=9),
               dict(pos=P(0) + 2), dict(q=None), dict(qo=None), dict(q=P(1) + 8),
               dict(qs=BIG * 128 - 8), dict(qs=BIG * 128 + 4), dict(qo=P(1) + 16),
               dict(qo=P(1), qos=BIG * 128 + 8), dict(rotary_dim=24), dict(rotary_dim=256),
               dict(num_axes=0), dict(pair_layout=3)):
        assert _rope_call(**{**ok, **kw}) == INVALID, kw
    assert _rope_call(**ok, head_dim=80) == UNSUPPORTED
    rope = gdn.gdn_rope_init(128, 64, [32])
    rope.axis[5] = 1
    assert _rope_call(rope, **ok) == INVALID
    # q and k as column ranges of one array, in place: no overlap; one head too many: overlap
    fused = dict(q=P(1), qo=P(1), qs=768, qos=768, k=P(1) + 1024, ko=P(1) + 1024, ks=768, kos=768)
    lib = gdn.load()
    assert _rope_call(**fused) == INVALID  # only the NULL handle is left; see the GPU tests
    assert _rope_call(**{**fused, "hq": 5}) == INVALID
    assert lib.gdn_rope_apply(None, None, 1, 1, None, 1, None, 0, 0, None, 0, None, 0, 0, None, 0,
                              None) == INVALID


# ---- append ----

def _cache(pages=10, page=16, heads=2, dim=128, k=P(20), v=P(21), ks=P(22), vs=P(23)):
    return gdn.gdn_kv_cache(pages, page, heads, dim, k, v, ks, vs)


def _append(cache=None, io=gdn.GDN_BF16, tokens=5, slots=P(0), k=P(1), ks=256, v=P(2), vs=256,
            rope=None, pos=None, ps=0, q=None, qs=0, hq=0, qo=None, qos=0, status=P(3)):
    return gdn.gdn_kv_append(None, _cache() if cache is None else cache, io, tokens, slots, k, ks,
                             v, vs, rope, pos, ps, q, qs, hq, qo, qos, status,
                             raise_on_error=False)


def test_append_refusals():
    rope = gdn.gdn_rope_init(128, 64, [32])
    ok = dict(rope=rope, pos=P(4), ps=5, q=P(5), qs=BIG * 128, hq=BIG, qo=1 << 50, qos=BIG * 128)
    assert _append() == INVALID and _append(**ok) == UNSUPPORTED
    for kw in (dict(pages=0), dict(heads=0), dict(page=0), dict(dim=0), dict(k=None), dict(v=None),
               dict(ks=None), dict(vs=None), dict(k=P(20) + 8), dict(vs=P(23) + 2)):
        assert _append(_cache(**kw), **ok) == INVALID, kw
    for kw in (dict(page=24), dict(page=256), dict(dim=96), dict(dim=512),
               dict(pages=2**27, heads=2, page=16)):
        assert _append(_cache(**kw)) == UNSUPPORTED, kw
    for kw in (dict(io=9), dict(tokens=-1), dict(slots=None), dict(slots=P(0) + 4), dict(k=None),
               dict(v=None), dict(ks=248), dict(vs=260), dict(k=P(1) + 2), dict(pos=None),
               dict(ps=4), dict(q=None), dict(qo=None), dict(qo=P(1)), dict(qo=P(2)),
               dict(status=P(3) + 2), dict(rope=None), dict(hq=-1),
               dict(rope=gdn.gdn_rope_init(64, 64, [32]))):
        assert _append(**{**ok, **kw}) == INVALID, kw


# ---- attention ----

def _cfg(hq=8, scale=0.1, causal=1, io=gdn.GDN_BF16):
    return gdn.gdn_attn_config(hq, causal, io, scale)


def _attn(cfg=None, cache=None, seqs=3, tokens=20, max_q=10, max_kv=100, cu=P(0), kv=P(1),
          table=P(2), blocks=7, q=P(3), qs=1024, o=P(4), os=1024, lse=P(5), ws=P(6),
          ws_bytes=None, status=P(8)):
    cfg, cache = cfg or _cfg(), cache or _cache()
    if ws_bytes is None:
        ws_bytes = 1 << 30
    return gdn.gdn_attn_paged(None, cfg, cache, seqs, tokens, max_q, max_kv, cu, kv, table, blocks,
                              q, qs, o, os, lse, ws, ws_bytes, status, raise_on_error=False)


def test_attention_refusals():
    SMALL = gdn.GDN_ERR_WORKSPACE_TOO_SMALL
    assert _attn() == INVALID  # the NULL handle
    assert _attn(ws_bytes=255) == SMALL
    assert _attn(lse=None, status=None, ws_bytes=255) == SMALL
    for kw in (dict(seqs=0), dict(tokens=-1), dict(max_q=-1), dict(max_kv=-1), dict(cu=None),
               dict(kv=None), dict(table=None), dict(blocks=0), dict(q=None), dict(o=None),
               dict(qs=1016), dict(os=1028), dict(q=P(3) + 8), dict(o=P(3)), dict(o=P(3) + 1024),
               dict(lse=P(4)), dict(lse=P(5) + 1), dict(ws=None), dict(ws=P(6) + 128),
               dict(cu=P(0) + 2), dict(cfg=_cfg(hq=7)), dict(cfg=_cfg(hq=0)),
               dict(cfg=_cfg(scale=float("inf"))), dict(cfg=_cfg(io=4)),
               dict(cache=_cache(k=None)), dict(cache=_cache(pages=0))):
        assert _attn(ws_bytes=255, **kw) == INVALID, kw
    for kw in (dict(seqs=4097), dict(cache=_cache(dim=192)), dict(cache=_cache(page=8)),
               dict(tokens=2**30), dict(tokens=2**22, max_kv=2**30)):
        assert _attn(**kw) == UNSUPPORTED, kw


def test_attention_workspace_size():
    for dim in (64, 128, 256):
        n = gdn.gdn_attn_workspace_size(_cfg(), _cache(dim=dim), 3, 20, 10, 100)
        assert n % 256 == 0 and n >= 256
        assert _attn(cache=_cache(dim=dim), qs=8 * dim, os=8 * dim, ws_bytes=n - 1) == \
            gdn.GDN_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(gdn.GdnError):
        gdn.gdn_attn_workspace_size(_cfg(hq=3), _cache(), 3, 20, 10, 100)


def test_cache_record_of_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros(5, 2, 16, 64, dtype=torch.uint8)
    s = torch.ones(5, 2)
    c = gdn.make_kv_cache(k, k.clone(), s, s.clone())
    assert (c.num_pages, c.num_kv_heads, c.page_size, c.head_dim) == (5, 2, 16, 64)
    for bad in ((k, k[:4], s, s), (k, k, s[:, :1], s), (k.transpose(1, 2), k, s, s),
                (k.float(), k, s, s), (k, k, s.double(), s)):
        with pytest.raises(gdn.GdnError):
            gdn.make_kv_cache(*bad)
