"""Ranges of the attention calls' requests, as the kernels work them out from the caller's
device-side numbers: the kernels' own arithmetic, built for the host."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

from packed_linear_attention_gb300 import build, gdn

HERE = os.path.dirname(os.path.abspath(__file__))
LO, HI = -2**31, 2**31 - 1


@pytest.fixture(scope="module")
def ranges(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ranges") / "libattn_ranges.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-Xcompiler",
                    "-fPIC,-fwrapv", "-shared", "-I", build.INCLUDE, "-o", so,
                    os.path.join(HERE, "cuda", "attn_ranges.cu")], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(so)
    fn = lib.attn_ranges

    def call(cu, kv, tokens, max_q, max_kv, blocks=HI, page=16):
        n = len(kv)
        out = np.empty((4, n), np.int32)
        cu, kv = np.asarray(cu, np.int32), np.asarray(kv, np.int32)
        p = lambda x: x.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
        fn(n, tokens, max_q, max_kv, blocks, page, p(cu), p(kv), *(p(x) for x in out))
        return out.astype(np.int64)

    call.lib = lib
    return call


def test_rows_stay_inside_the_arrays(ranges):
    """Any two numbers as a request's first and last row: its rows are rows of the arrays, and
    the request is flagged unless the numbers were in order."""
    ends = [LO, LO + 1, LO + 5, -7, -1, 0, 1, 5, 6, 7, 100, HI - 1, HI]
    for tokens, max_q in ((6, 3), (6, HI), (0, 4), (1, 0), (HI, HI)):
        for r0, r1 in itertools.product(ends, ends):
            (row0,), (q,), _, (bad,) = ranges([r0, r1], [4], tokens, max_q, 100)
            assert 0 <= row0 <= tokens and 0 <= q <= max_q and row0 + q <= tokens, (r0, r1, tokens)
            lo, hi = max(r0, 0), min(r1, tokens)
            assert q == min(max(hi - min(lo, tokens), 0), max_q)
            assert bad == (not (0 <= r0 <= r1 <= tokens and r1 - r0 <= max_q))


def test_tokens_can_be_numbered_past_the_last_one(ranges):
    """The kernels number tokens by whole batches of 512, a batch ahead: no such number passes 32
    bits, whatever length the caller states, and a length that was cut is flagged."""
    for kv in (LO, -1, 0, 1, 1 << 30, HI - 4096, HI - 4095, HI - 1023, HI):
        for max_kv in (0, 100, HI - 2000, HI):
            for blocks in (1, HI):
                _, _, (length,), (bad,) = ranges([0, 1], [kv], 1, 1, max_kv, blocks)
                assert 0 <= length <= min(max(kv, 0), max_kv, 16 * blocks)
                assert -(-length // 512) * 512 + 2 * 512 <= HI
                assert length == min(max(kv, 0), max_kv, 16 * blocks, HI - 4096)
                assert bad == (length != kv)


def test_item_counts_stop_at_the_end_of_32_bits(ranges):
    """Overlapping requests may ask for any number of work items: the sum never wraps."""
    rng = np.random.default_rng(0)
    total = lambda x: ranges.lib.attn_items_sum(  # noqa: E731
        len(x), np.asarray(x, np.int32).ctypes.data_as(ctypes.c_void_p))
    assert total([HI - 5, 3]) == HI - 2 and total([HI - 5, 5]) == HI
    assert total([2304 * 1024] * 2048) == HI and total([HI] * 100) == HI
    for _ in range(200):
        x = rng.integers(0, rng.integers(1, HI), 40)
        assert total(x) == min(int(x.sum()), HI)


def _call(tokens, seqs=1, hq=16, hkv=2, dim=256, io=gdn.GDN_BF16, kv=None, max_q=None, page=64):
    """Status of a call's host checks (its NULL handle is refused after them)."""
    build.build()
    kv = tokens if kv is None else kv
    cache = gdn.gdn_kv_cache(min(HI // (hkv * page), 1 << 20), page, hkv, dim, 1 << 24, 1 << 25,
                             1 << 26, 1 << 27)
    cfg = gdn.gdn_attn_config(hq, 1, io, 0.1)
    at = lambda i: i << 44  # noqa: E731
    size = ctypes.c_size_t()
    sized = gdn.load().gdn_attn_workspace_size(ctypes.byref(cfg), ctypes.byref(cache), seqs,
                                               tokens, tokens if max_q is None else max_q, kv,
                                               ctypes.byref(size))
    st = gdn.gdn_attn_paged(None, cfg, cache, seqs, tokens, tokens if max_q is None else max_q, kv,
                            at(1), at(2), at(3), 1 << 20, at(4), hq * dim, at(5), hq * dim, at(6),
                            at(7), size.value - 1 if sized == 0 else 0, None,
                            raise_on_error=False)
    assert st == (gdn.GDN_ERR_WORKSPACE_TOO_SMALL if sized == 0 else sized)
    return sized


@pytest.mark.parametrize("tokens,seqs,hq,hkv,dim,kv", [
    (262144, 1, 16, 2, 256, None), (262144, 1, 64, 8, 128, None), (131072, 1, 64, 8, 128, None),
    (262144, 8, 32, 8, 128, 262144), (1 << 20, 4096, 16, 2, 256, 262144), (1000000, 1, 8, 1, 64, None)])
def test_long_prompts_are_taken(tokens, seqs, hq, hkv, dim, kv):
    """bf16 prompts of the longest contexts: only requests of few queries count work items over
    the cached tokens."""
    assert _call(tokens, seqs, hq, hkv, dim, kv=kv) == gdn.GDN_OK


def test_calls_of_more_work_items_than_32_bits_are_refused():
    f32 = dict(io=gdn.GDN_F32)
    # fp32: every row counts, 8 rows and 64 cached tokens an item
    assert _call(100000, kv=100000, **f32) == gdn.GDN_OK
    assert _call(262144, kv=262144, **f32) == gdn.GDN_ERR_UNSUPPORTED
    # bf16: many requests of few queries over the longest lengths
    assert _call(4096, 4096, 16, 2, 256, kv=1 << 20, max_q=1) == gdn.GDN_OK
    assert _call(65536, 4096, 16, 16, 256, kv=1 << 28, max_q=16) == gdn.GDN_ERR_UNSUPPORTED
    # rows
    assert _call(1 << 30, hq=64, hkv=8, kv=64) == gdn.GDN_ERR_UNSUPPORTED
