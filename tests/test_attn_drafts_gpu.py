"""Drafts: a few queries a request, on either side of the rule that shares them out between the
kernel that splits the cached tokens and the one that takes 128 rows at a time."""
import pytest

from test_attn_gpu import Case

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 2, 128, 16), (16, 2, 256, 64), (6, 2, 64, 32)])
@pytest.mark.parametrize("requests", [2, 45, 180])
def test_drafts_of_many_lengths(hq, hkv, dim, page, requests):
    """1 to 9 queries a request, beside one without any and one without a cached token: with 2
    requests all are few, with 180 most go to the kernel for prompts, as partial units."""
    q_len = [i % 10 for i in range(1, requests + 1)]
    kv_len = [n + (37 * i) % 150 for i, n in enumerate(q_len)]
    kv_len[-1] = 0
    Case(requests + dim, q_len, kv_len, hq, hkv, dim, page).check(torch_cuda())


def test_drafts_beside_decode_and_a_prompt():
    q_len = [1, 5, 300, 2, 9, 1, 17, 33]
    kv_len = [900, 64, 300, 2, 700, 1, 400, 33]
    Case(3, q_len, kv_len, 16, 2, 256, 64).check(torch_cuda())
