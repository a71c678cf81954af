"""Ranges of the attention calls' requests, as the kernels work them out from the caller's
device-side numbers: the kernels' own arithmetic, built for the host."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

from packed_linear_attention_gb300 import build

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
