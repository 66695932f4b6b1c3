"""The gradient norm and clipping where they can go wrong: the ends of fp32's range, and pieces of every
size with values in all of them."""
import numpy as np
import pytest
import torch

import operators_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# A thread adds at most 64 squares of a piece to each of two fp32 sums (fused: a rounding each; scaling
# by powers of two is exact), a few more at a piece's ends, and the two to one; pairs of floats then
# lose nothing that counts; the root halves that and is rounded once: 35 units, and 2^-24 that the
# largest range may lose.  Norms below the normal range are off by half of fp32's smallest step.
NORM, STEP = 36 * ref.U, 2.0 ** -150


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def true_norm(grads):
    scaled = [g.double() * 2.0 ** 200 if g.abs().max() < 1 else g.double() for g in grads]
    factor = 2.0 ** -200 if all(g.abs().max() < 1 for g in grads) else 1.0
    assert factor != 1.0 or all(g.abs().max() >= 1 for g in grads)
    return float(torch.stack([g.square().sum() for g in scaled]).sum().sqrt()) * factor


def check(grads):
    import laplacian_nystr_attention_gb300 as lna
    norm = true_norm(grads)
    plan = lna.GradClip.like(grads)
    assert abs(plan.norm(grads).item() - norm) <= NORM * norm + STEP
    top = float(np.float32(norm / 4))
    outs = [torch.full_like(g, 3.0) for g in grads]
    assert abs(plan.clip(grads, top, outs=outs).item() - norm) <= NORM * norm + STEP
    # The scale is off as the norm is (below the normal range by half a step of it as well), and
    # rounded once; the product is rounded to the type, in whose subnormals by half a step.
    scale = min(1.0, top / norm)
    off = NORM + 2 * ref.U + STEP / norm
    for g, out in zip(grads, outs):
        kind = "f32" if g.dtype == torch.float32 else "bf16"
        want = g.double() * scale
        tol = (off + ref.HALF[kind] * (1 + off)) * want.abs()
        tol += STEP if kind == "f32" else 2.0 ** -134
        assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("scale", [1e-29, 2.0 ** -98, 1e-31, 1e-33, 1e-34, 1e-36, 1e-38, 1e-40,
                                   2.0 ** -140])
@pytest.mark.parametrize("counts", [[1], [7, 3], [5000, 333], [1 << 20, 3]])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_small_norms(scale, counts, kind):
    """Down to fp32's smallest values (bf16: 2^-133): none vanishes, and all are clipped."""
    rng = np.random.default_rng(2)
    if kind == "bf16":
        scale = max(scale, 2.0 ** -130)
    grads = [torch.from_numpy(scale * (1 + rng.random(n)) * rng.choice([-1.0, 1.0], n))
             .to(TYPES[kind]).cuda() for n in counts]
    check(grads)


def test_the_smallest_value():
    import laplacian_nystr_attention_gb300 as lna
    g = [torch.tensor([0.0, 2.0 ** -149, 0.0], device="cuda")]
    plan = lna.GradClip.like(g)
    assert plan.norm(g).item() == 2.0 ** -149
    assert plan.clip(g, 0.0).item() == 2.0 ** -149 and (g[0] == 0).all()


@pytest.mark.parametrize("low,high", [(1e-44, 1e-32), (1e-36, 1e-24), (1e-32, 2e-7), (1e-30, 1e-6)])
def test_small_values_beside_larger_ones(low, high):
    """Both sides of where one range takes over from the next: many small values whose sum counts."""
    rng = np.random.default_rng(3)
    small = np.full(1 << 16, low)
    large = high * (1 + rng.random(5))
    check([torch.from_numpy(a.astype(np.float32)).cuda() for a in (small, large)])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[1 << 24, 5], [(1 << 26) + 4099], [1 << 25, 70001, 1 << 25, 3]])
def test_large_pieces(kind, counts):
    """Tensors that are cut into the larger pieces, with values in all of them."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    # Scaled by powers of two, within one of fp32's, so that 64-bit squares hold them.
    check([(4 + torch.randn(n, generator=gen, device="cuda")).to(TYPES[kind]) for n in counts])
