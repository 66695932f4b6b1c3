"""Edges of the AdamW step (lapl_adamw_*): an eps of any size, scalars in the tensors' memory, and what
clipping leaves in the states."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
from operators_reference import U, rounded
from test_gpu_adamw import check_coded, dev, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps,lr,scale", [(1e38, 1e22, 1e15), (3.4e38, 1e24, 1e14), (1e19, 1e4, 1e15), (4e18, 1e4, 1e15),
                                          (1e-37, 1e-3, 1.0)])
def test_an_eps_of_any_size(bits, eps, lr, scale, monkeypatch):
    """An update that eps makes small, and not nothing.

    The reference's bound of w counts roundings of w alone, which is enough where lr wd <= 1.  w (1 - lr wd)
    is formed by a product, a difference and a product, each rounded once: U lr wd |w|, and U (1 + lr wd) |w|
    twice; 4 U lr wd |w| more covers what grows with lr."""
    form = ref.adamw

    def adamw(w, g, m, v, step, lr, betas, eps, wd, clip=1.0):
        (w1, bound), *states = form(w, g, m, v, step, lr, betas, eps, wd, clip)
        return ((w1, bound + 4 * U * lr * wd * np.abs(w)), *states)

    monkeypatch.setattr(ref, "adamw", adamw)
    run([700, 256], ["f32", "f32"], bits=bits, eps=eps, lr=lr, scale=scale)


def test_scalars_in_what_the_step_writes_are_refused():
    """Every CTA reads them when it starts, and by then another may have written there."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.AdamW([8], ["f32"])
    p, g = [torch.ones(8, device="cuda")], [torch.ones(8, device="cuda")]
    s = plan.new_states(p)
    number = torch.ones((), dtype=torch.int64, device="cuda")
    one = torch.ones((), device="cuda")
    call = dict(params=p, grads=g, step=number, lr=one, **s)
    for bad in (dict(lr=p[0][3:4]), dict(norm=s["m"][0][7:], max_norm=1.0), dict(lr=s["v"][0][:1]),
                dict(step=p[0][2:4].view(torch.int64))):
        with pytest.raises(lna.LaplAttnError) as e:
            plan.step(**{**call, **bad})
        assert e.value.status == 1
    # What is only read may be one place, and a gradient.
    plan.step(**{**call, "lr": g[0][:1], "norm": g[0][:1], "max_norm": 1.0})
    assert (p[0] < 1).all()
