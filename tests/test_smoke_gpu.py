"""The smoke step of the calls around the recurrent layers notices a call that did nothing."""
import pytest

import __graft_entry__ as entry
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda

pytestmark = pytest.mark.gpu


def test_all_calls_made():
    torch_cuda()
    entry._smoke_scan(handle())


@pytest.mark.parametrize("name", ["gdn_conv_packed", "gdn_ssm_packed", "gdn_conv_step", "gdn_ssm_step",
                                  "gdn_rms_norm", "gdn_sample"])
def test_a_call_left_out(monkeypatch, name):
    torch = torch_cuda()
    h = handle()
    empty = torch.empty
    # what a call leaves unwritten is zeros, not what an earlier one left in the same memory
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).zero_())
    monkeypatch.setattr(gdn, name, lambda *a, **k: gdn.GDN_OK)
    with pytest.raises(AssertionError):
        entry._smoke_scan(h)
