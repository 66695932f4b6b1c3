"""The attention's backward where it can go wrong: an empty batch, and the clipping of its gradients."""
import pytest
import torch

from lapl_workloads import WORKLOADS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def test_an_empty_batch_gives_a_zero_bias_gradient():
    """The sum over no batch, whatever its tensor held, clipped or not, given or not."""
    import laplacian_nystr_attention_gb300 as lna
    w = WORKLOADS["tiny_f32"].replace(heads=2, batch=0)
    att = lna.LaplacianNystromAttention(lna.make_config(**w.config()))
    none = torch.empty(0, 2, w.grid_h * w.grid_w, w.head_dim, device="cuda")
    att.forward(none, none, none, keep_for_backward=True)
    for max_norm in (None, 0.5):
        room = torch.full((2 * att.cfg.num_landmarks + 1,), 7.0, device="cuda")
        dbias = room[:-1].view(2, -1)
        got = att.backward(none, none, none, none, grads={"dbias": dbias}, max_norm=max_norm)
        assert got[3] is dbias and (dbias == 0).all() and room[-1] == 7.0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = att.backward(none, none, none, none, stream=side)
    side.synchronize()
    assert (got[3] == 0).all()
    att.close()


@pytest.mark.parametrize("bad", [-1.0, float("nan"), float("inf"), 1e39, -1e39])
def test_a_max_norm_that_is_none_is_refused_before_the_backward(bad):
    """What fp32 does not hold, too; no gradient is written."""
    import laplacian_nystr_attention_gb300 as lna
    w = WORKLOADS["tiny_f32"]
    att = lna.LaplacianNystromAttention(lna.make_config(**w.config()))
    q = torch.randn(w.batch, w.heads, w.n, w.head_dim, device="cuda")
    att.forward(q, q, q, keep_for_backward=True)
    grads = {name: torch.full_like(q, 7.0) for name in ("dq", "dk", "dv")}
    with pytest.raises(ValueError):
        att.backward(q, q, q, q, grads=grads, max_norm=bad)
    torch.cuda.synchronize()
    assert all((t == 7.0).all() for t in grads.values())
    att.backward(q, q, q, q, grads=grads, max_norm=3.4028234663852886e38)
    assert torch.isfinite(att.grad_norm)
    att.close()
