"""Edges of the heads' norm and rotary positions (lapl_rope_*): many heads in the weights' gradients,
frequencies of more than a turn."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
from operators_reference import U
from test_gpu_rope import EPS, dev, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def test_weights_gradients_of_thousands_of_equal_heads():
    """512 rows that a thread would add up in fp32, each of which loses 0.49 of a unit once the sum is over
    256: 125 U in all, where the bound of the terms' own errors is 54 U.  Fewer than 128 rows to an fp32
    sum lose at most 16 U of it."""
    import laplacian_nystr_attention_gb300 as lna
    H, d = 4096, 63
    u = 1 / np.sqrt(1 + EPS)
    c = np.float32((1 + 0.49 * 2.0 ** -15) / u)
    plan = lna.HeadRotary(lna.make_rope_config(1, 1, H, H, 0, d, (0,), [], eps=EPS))
    x = torch.ones(1, 1, H * d, device="cuda")
    dy = torch.full((1, H, 1, d), float(c), device="cuda")
    got = plan.backward(x, x, None, None, None, dy, dy)
    want = H * float(c) * u
    for dw in got[3:]:
        off = np.abs(dw.double().cpu().numpy() - want).max()
        assert off <= (d / 2 + 23) * U * want, off / want / U


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pairs,interleaved", [(24, (6, 6), False), (63, (20,), True), (256, (64, 64), False)])
def test_many_heads(dtype, d, pairs, interleaved):
    """Of queries and keys, not as many of one as of the other, over a few tokens."""
    run(B=1, N=2, heads=(1500, 700, 3), d=d, pairs=pairs, dtype=dtype, interleaved=interleaved)
    run(B=1, N=3, heads=(9, 1333, 0), d=d, pairs=pairs, dtype=dtype, interleaved=interleaved)


def turns(position, frequency):
    """position * frequency radians as a fraction of a turn, in integers: pi by Machin's formula."""
    bits = 400

    def arctan_of_one_over(x):
        term, total, k = (1 << bits + 32) // x, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term, k = term // (x * x), k + 2
        return total

    pi = 4 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)) >> 32
    n, d = float(frequency).as_integer_ratio()
    turn = 2 * pi * d                            # radians: position n 2^bits of these
    return float((int(position) * n << bits) % turn / turn)


@pytest.mark.parametrize("far", [0, 1 << 24, (1 << 31) - 60, -(1 << 31) + 60])
def test_frequencies_of_any_size(far, monkeypatch):
    """Of many turns a position and of next to none, of both signs, at positions of all 32 bits."""
    import test_gpu_rope
    freq = [1e5, -1e5, 50.0, 3.0e7 + 1 / 3, -1e-12, 7.0e30, 1e-310, -2.5]
    monkeypatch.setattr(test_gpu_rope, "frequencies", lambda pairs: freq)

    def angles(positions, pairs, frequencies):
        axis = [a for a, n in enumerate(pairs) for _ in range(n)]
        at = np.asarray(positions)[..., axis]
        t = [[[turns(x, f) for x, f in zip(row, frequencies)] for row in rows] for rows in at]
        return 2 * np.pi * np.asarray(t)[:, None]

    monkeypatch.setattr(ref, "angles", angles)
    run(far=far, pairs=(8,), d=16, N=12)
    run(far=far, pairs=(4, 4), d=17, N=12, interleaved=True)


@pytest.mark.parametrize("bad,status", [(2.0 ** 128, 2), (-1e300, 2), (float("inf"), 1)])
def test_frequencies_that_are_refused(bad, status):
    import laplacian_nystr_attention_gb300 as lna
    with pytest.raises(lna.LaplAttnError) as e:
        lna.HeadRotary(lna.make_rope_config(1, 4, 1, 1, 0, 8, (2,), [1.0, bad]))
    assert e.value.status == status
    lna.HeadRotary(lna.make_rope_config(1, 4, 1, 1, 0, 8, (2,), [1.0, -(2.0 ** 127)]))
