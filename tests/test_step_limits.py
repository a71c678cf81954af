"""The calls around the recurrent layers at the ends of what they take, on the host: no call gets as
far as a kernel (validation comes before any CUDA call, and a NULL handle is the last thing checked)."""
import pytest

from packed_linear_attention_gb300 import build, gdn

from test_step_abi import INVALID, P, UNSUPPORTED, conv_config, requests, ssm_config, ssm_rows

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
