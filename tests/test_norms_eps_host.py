"""eps below the least normal float32 is refused: the kernels' reciprocal square root takes such
numbers for zero, and rows of zeros would turn NaN."""
import pytest

import selective_state_space_79_amd as ssm
from test_blocks_host import ADD, GATED, added, at, call, gated


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.1754942e-38])
def test_subnormal_eps(eps):
    assert call("ssm_gated_norm_fwd", gated(eps=eps), GATED, y=at(2)) == ssm.SSM_ERR_DIMS
    assert call("ssm_add_norm_fwd", added(eps=eps), ADD, y=at(5)) == ssm.SSM_ERR_DIMS
    assert ssm.ssm_gated_norm_bwd_workspace_bytes(gated(eps=eps)) == 0
    assert ssm.ssm_add_norm_bwd_workspace_bytes(added(eps=eps)) == 0


def test_least_normal_eps_is_taken():
    least = 2.0 ** -126
    assert call("ssm_gated_norm_fwd", gated(eps=least), GATED, y=at(2)) == ssm.SSM_ERR_ALIAS
    assert call("ssm_add_norm_fwd", added(eps=least), ADD, y=at(5)) == ssm.SSM_ERR_ALIAS


@pytest.mark.gpu
def test_rows_of_zeros_with_the_least_eps():
    import torch

    x, w = torch.zeros(3, 64, device="cuda"), torch.ones(64, device="cuda")
    x[1] = 1e-15
    for eps in (2.0 ** -126, 1e-30):
        y = ssm.gated_norm_fwd(x, None, w, eps=eps)
        r = ssm.gated_norm_bwd(x, None, w, dy=torch.ones_like(x), eps=eps)
        z, _ = ssm.add_norm_fwd(x, None, w, eps=eps)
        a = ssm.add_norm_bwd(x, x, w, dy=torch.ones_like(x), eps=eps, scale=w, post_weight=w)
        assert all(bool(t.isfinite().all()) for t in (y, z, *r.values(), *a.values())), eps
        assert not y[0].any() and not z[2].any()
