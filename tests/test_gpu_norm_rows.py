"""The gradient of ep_combine_norm by its number of rows: none at all, and more than there are workgroups."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


@pytest.mark.parametrize("f_type", [torch.float32, BF])
@pytest.mark.parametrize("what", ["no vectors asked for", "no vectors at all", "gate per token"])
def test_empty_batch(ep, what, f_type):
    rows, w = torch.empty(0, 64, dtype=BF, device=DEV), torch.ones(64, device=DEV)
    f = torch.empty(0, 64, dtype=f_type, device=DEV)
    if what == "no vectors asked for":
        got = ep.ep_combine_norm_backward(rows, rows, f, residual=rows, post_weight=w, pre_weight=w, gate=w, need_vectors=False)
        want = {"grad_f", "grad_residual"}
    elif what == "no vectors at all":
        got, want = ep.ep_combine_norm_backward(rows, None, f, residual=rows), {"grad_f", "grad_residual"}
    else:
        got, want = ep.ep_combine_norm_backward(rows, None, f, residual=rows, gate=rows), {"grad_f", "grad_residual", "grad_gate"}
    torch.cuda.synchronize()
    assert {k for k, v in got.items() if v is not None} == want
    assert all(got[k].shape == (0, 64) and got[k].dtype is BF for k in want)
