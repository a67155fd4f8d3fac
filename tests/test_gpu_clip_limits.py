"""Clipping by norms at the ends of their range."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
INF = float("inf")


@pytest.fixture(scope="module")
def cf():
    from cnn_conv3d_gb300 import build
    build.build()
    from cnn_conv3d_gb300 import cfconv
    return cfconv


@pytest.mark.parametrize("max_norm", [INF, 3e38, 1.0, 0.0])
@pytest.mark.parametrize("value,norm", [(INF, INF), (-INF, INF), (3e38, INF), (0.0, 0.0), (2.0, 60.0)])
def test_infinite_norms_give_a_factor_of_zero(cf, value, norm, max_norm):
    """Whatever the limit, an infinite one too; a finite norm below the limit leaves the gradients as they are."""
    g = torch.full((900,), value, device="cuda")
    lst = cf.cf_grads([g])
    size = cf.cf_grad_workspace_size(lst)
    ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    cf.cf_grad_norm(lst, max_norm, out, ws, size)
    factor = 0.0 if norm == INF else min(1.0, max_norm / (norm + 1e-6))
    assert out[0].item() == norm and abs(out[1].item() - factor) <= 1e-6 * factor
    cf.cf_clip_grads(lst, max_norm, out, ws, size)
    want = torch.full((900,), value, device="cuda") * out[1]
    assert torch.equal(torch.nan_to_num(g, nan=7.0), torch.nan_to_num(want, nan=7.0))
    # and the Adam step, in which a factor of 0 leaves the moments' decay
    if 0.0 < max_norm:
        w, m, v, g = (torch.full((900,), t, device="cuda") for t in (1.0, 0.5, 0.25, value))
        p = cf.cf_adam_params([(w, None, g, m, v)])
        size = cf.cf_clip_adam_workspace_size(p)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        cf.cf_clip_adam_step(p, cf.cf_adam_hyper(1e-3, 0.9, 0.999, 1e-8, 0.0, max_norm, 2), out, ws, size)
        assert out[0].item() == norm
        if norm == INF:
            assert bool(torch.isnan(m).all()) if value in (INF, -INF) else torch.allclose(m, torch.full_like(m, 0.45), rtol=1e-6)
