"""The gradient of ep_combine_norm by its number of rows: none at all, and more than there are workgroups."""
import pytest
import torch

import expert_reference as R
import harness as Hn
import norm_reference as N

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


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("f_type", [torch.float32, BF])
@pytest.mark.parametrize("T,H", [(515, 4104), (600, 7168), (259, 8192), (519, 8200), (257, 16392), (530, 32768)])
def test_more_rows_than_workgroups(ep, T, H, f_type, gate):
    """Wide rows, of which a workgroup takes two or three, some one more than others: the vectors' sums go on from row to row."""
    g = torch.Generator(device=DEV).manual_seed(T + H)
    n = lambda *s, std=1.0, mean=0.0, dtype=BF: (torch.randn(*s, generator=g, device=DEV) * std + mean).to(dtype)
    f, do, dn = n(T, H, dtype=f_type), n(T, H), n(T, H)
    a = dict(residual=n(T, H, std=2.0), post_weight=n(H, std=0.2, mean=1.0), gate=n(T, H, std=0.5) if gate == "token" else n(H, std=0.3, mean=0.4),
             residual_scale=0.7, pre_weight=n(H, std=0.2, mean=1.0), eps=1e-5)
    ws, gw = Hn.guarded_tensor((ep.ep_combine_norm_workspace_bytes(T, H),), torch.uint8, DEV, "ws")
    got = ep.ep_combine_norm_backward(do, dn, f, workspace=ws, **a)
    torch.cuda.synchronize()
    Hn.assert_guards(gw)
    want = N.gradients(f, a["residual"], a["post_weight"], a["gate"], a["residual_scale"], a["pre_weight"], a["eps"], do, dn)
    assert set(want) == {k for k, v in got.items() if v is not None}
    for k, (v, e) in want.items():
        R.assert_within(got[k], v, e, k)
