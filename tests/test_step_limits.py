"""The calls around the recurrent layers at the ends of what they take, on the host: no call gets as
far as a kernel (validation comes before any CUDA call, and a NULL handle is the last thing checked)."""
import pytest

from packed_linear_attention_gb300 import build, gdn

from test_step_abi import (INVALID, P, UNSUPPORTED, conv_config, norm_config, requests, ssm_config,
                           ssm_rows)

TOP = (1 << 31) - 4096
FAR = [(1 << 50) * (i + 1) for i in range(8)]  # room for 2^31 rows each


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return gdn.load()


def conv(tokens):
    return gdn.gdn_conv_packed(None, conv_config(), requests(num_tokens=tokens), FAR[0], 96, FAR[1], 96,
                               P(2), P(3), P(4), raise_on_error=False)


def ssm(tokens):
    rows = ssm_rows(x=FAR[0], delta=FAR[1], b=FAR[2], c=FAR[3], z=FAR[4], y=FAR[5])
    return gdn.gdn_ssm_packed(None, ssm_config(), requests(num_tokens=tokens), rows, P(6), P(7), FAR[6],
                              1 << 40, P(9), raise_on_error=False)


@pytest.mark.parametrize("call", [conv, ssm])
def test_rows_of_a_packed_call(call):
    """The kernels count rows in 32 bits, a block past the last one too."""
    assert call(TOP - 1) == INVALID  # the NULL handle
    assert call(TOP) == UNSUPPORTED and call((1 << 31) - 1) == UNSUPPORTED


def test_norm_of_no_rows():
    """Empty tensors have no address."""
    odd = norm_config(num_heads=4, dim=96)  # refused after everything else
    call = lambda n, **kw: gdn.gdn_rms_norm(None, odd, n, None, 384, raise_on_error=False, **kw)  # noqa: E731
    assert call(0) == UNSUPPORTED and call(1) == INVALID and call(-1) == INVALID
    for kw in (dict(sum=P(0), sum_stride=384), dict(codes=P(1), codes_stride=384), dict(scales=P(2))):
        assert call(0, **kw) == UNSUPPORTED and call(1, **kw) == INVALID, kw


@pytest.mark.gpu
def test_norm_of_empty_tensors():
    from gpu_util import handle, torch_cuda
    torch = torch_cuda()
    empty = lambda dtype: torch.empty(0, 256, dtype=dtype, device="cuda")  # noqa: E731
    x = empty(torch.bfloat16)
    cfg = gdn.make_norm_config(256, torch.ones(256, device="cuda"))
    gdn.gdn_rms_norm(handle(), cfg, 0, x, 256, x, 256, x, 256, y=x, y_stride=256)
    gdn.gdn_rms_norm(handle(), cfg, 0, x, 256, codes=empty(torch.uint8), codes_stride=256,
                     scales=torch.empty(0, 1, device="cuda"))
    torch.cuda.synchronize()
