"""The residual + RMS norm where it can go wrong: 8-bit values at the middle of two, rows with a NaN, and
sums over many rows."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def randn(*shape, seed=0, dtype="f32"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(TYPES[dtype])


# ---- 8 bits -------------------------------------------------------------------------------

@pytest.mark.parametrize("H,d", [(1, 128), (2, 640), (32, 20), (1, 4096), (3, 150), (1, 16384), (1, 33)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [False, True])
def test_8_bit_values_are_the_rounded_quotients(H, d, group, x, shift):
    """q and the scales are, bit for bit, what the fp32 output of the same call gives: the largest
    magnitude / 448 and y / scale in fp32, and that rounded to nearest even."""
    import laplacian_nystr_attention_gb300 as lna
    W, N = H * d, 1 + 200000 // (H * d)
    if group and W % group:
        pytest.skip("no group of that size")
    place = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape) if shift else t
    xs, res = place(randn(1, H, N, d, dtype=x)), randn(1, N, W, seed=1, dtype=x)
    weight = 1 + 0.2 * randn(W, seed=2)
    outs = []
    for out, g in (("f32", 0), ("f8", group)):
        plan = lna.ResidualNorm(lna.make_norm_config(1, H, N, d, x_dtype=x, res_dtype=x, out_dtype=out,
                                                     scale_group=g))
        outs.append(plan.forward(xs, weight, residual=res))
    y = outs[0].cpu().numpy().reshape(1, N, -1, group or W)
    top = np.maximum(np.abs(y).max(-1), np.float32(2.0 ** -100))
    scales = top / np.float32(448)
    q = torch.from_numpy((y / scales[..., None]).reshape(1, N, W)).to(torch.float8_e4m3fn)
    assert torch.equal(outs[1][1].cpu(), torch.from_numpy(scales))
    assert torch.equal(outs[1][0].cpu().view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("d", [128, 2112])
def test_8_bit_rows_with_a_nan(group, d):
    """Such a row's values and scales are NaN, the others' as they are."""
    import laplacian_nystr_attention_gb300 as lna
    N = 50
    plan = lna.ResidualNorm(lna.make_norm_config(1, 1, N, d, out_dtype="f8", scale_group=group))
    x = randn(1, 1, N, d)
    good = [t.clone() for t in plan.forward(x)]
    x[0, 0, 7, 3], x[0, 0, 9, 0] = float("nan"), float("inf")
    q, scales = plan.forward(x)
    keep = torch.ones(N, dtype=torch.bool)
    keep[7] = keep[9] = False
    assert torch.equal(q[0, keep].view(torch.uint8), good[0][0, keep].view(torch.uint8))
    assert torch.equal(scales[0, keep], good[1][0, keep])
    assert torch.isnan(q[0, 7].float()).all() and torch.isnan(scales[0, 7]).all()
    assert torch.isnan(q[0, 9, 0].float()) and torch.isnan(scales[0, 9, 0])


# ---- sums over rows -----------------------------------------------------------------------

@pytest.mark.parametrize("rows,width", [(32, 64), (16, 100), (3, 256), (300, 1024), (60, 1024),
                                        (300, 2049), (300, 4096), (150, 16384), (150, 9999)])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_dweight_keeps_small_rows_beside_large_ones(rows, width, grad):
    """A row of 2^30, one of -2^30 and ones: what is left after the large ones cancel is the ones,
    exactly where each row has threads of its own (sums in fp32 lose tens of them).

    A thread adds its own rows in fp32.  152 CTAs or more share the rows, so that it has at most
    rows / 152 of them, rounded up, and beside a large one loses the others, 1 each: twice that less
    one in all."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.ResidualNorm(lna.make_norm_config(1, 1, rows, width, grad_dtype=grad))
    dy = torch.ones(1, rows, width, device="cuda", dtype=TYPES[grad])
    dy[0, 0], dy[0, rows // 2] = 2.0 ** 30, -(2.0 ** 30)
    total, rstd = torch.ones(1, rows, width, device="cuda"), torch.ones(1, rows, device="cuda")
    _, _, dweight = plan.backward(total, rstd, None, dy, grads={"dx": None})
    assert ((dweight - (rows - 2)).abs() <= 2 * (-(-rows // 152) - 1)).all()
