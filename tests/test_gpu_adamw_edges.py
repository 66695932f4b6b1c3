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
