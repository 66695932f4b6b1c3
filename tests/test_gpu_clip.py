"""The global gradient norm and clipping (lapl_clip_*) against 64-bit sums."""
import numpy as np
import pytest
import torch

import operators_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# A thread sums at most 32 squares in fp32 (each two roundings, and two of the scaled value) before
# it goes on in double; the root halves that; the result is rounded once: under 64 units.
NORM = 64 * ref.U


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def make(counts, kinds, seed=0, scale=1.0):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy(scale * rng.standard_normal(n)).to(TYPES[k]).cuda()
            for n, k in zip(counts, kinds)]


def true_norm(grads):
    return float(np.sqrt(sum((g.double().cpu().numpy() ** 2).sum() for g in grads)))


def clip(grads, max_norm, in_place=False):
    """Clips, checks the norm and every value; returns the outputs."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.GradClip.like(grads)
    norm = true_norm(grads)
    src = [g.clone() for g in grads]
    outs = None if in_place else [torch.full_like(g, 3.0) for g in grads]
    got = plan.clip(grads, max_norm, outs=outs).item()
    assert plan.norm(src).item() == got
    if norm > np.finfo(np.float32).max:
        # fp32 does not hold it (1e37 sqrt(5333) = 7.3e38 against 3.4e38): infinity, no change.
        assert got == np.inf
        scale = 1.0
    else:
        assert abs(got - norm) <= NORM * norm
        scale = max_norm / norm if norm > max_norm else 1.0
    for s, o in zip(src, grads if in_place else outs):
        want = s.double().cpu().numpy() * scale
        kind = "f32" if s.dtype == torch.float32 else "bf16"
        ref.check("out", o, (want, (NORM + 2 * ref.U) * np.abs(want) * (scale != 1.0)), kind)
        if scale == 1.0:
            assert torch.equal(s, o)
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(src, grads))
    plan.close()
    return outs


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 511, 16383, 16384, 16385, 100001, 3000001])
@pytest.mark.parametrize("in_place", [False, True])
def test_one_tensor(kind, n, in_place):
    g = make([n], [kind])
    clip(g, 0.3 * true_norm(g), in_place)


def test_under_the_largest_norm_nothing_changes():
    g = make([1000, 5], ["f32", "bf16"])
    clip(g, 2 * true_norm(g))
    clip(g, 2 * true_norm(g), in_place=True)


@pytest.mark.parametrize("tensors", [2, 63, 64, 65, 999, 1000, 1001, 2300])
def test_many_tensors(tensors):
    counts = [(i * 37) % 200 for i in range(tensors)]       # some of them empty
    counts[0] = 40000
    g = make(counts, ["bf16" if i % 3 else "f32" for i in range(tensors)])
    clip(g, 0.5 * true_norm(g))
    clip(g, 0.5 * true_norm(g), in_place=True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_slices_of_one_buffer(kind):
    """Tensors that start anywhere, and outputs aligned otherwise; what lies between stays."""
    import laplacian_nystr_attention_gb300 as lna
    flat = make([50000], [kind])[0]
    cuts = [(0, 5), (5, 8), (9, 9), (10, 27), (27, 17000), (17003, 40000), (40001, 49999)]
    grads = [flat[a:b] for a, b in cuts]
    clip(grads, 0.4 * true_norm(grads))
    before, norm = flat.clone(), true_norm(grads)
    lna.GradClip.like(grads).clip(grads, 0.4 * norm)
    inside = torch.zeros(50000, dtype=torch.bool)
    for a, b in cuts:
        inside[a:b] = True
    assert torch.equal(flat[~inside], before[~inside])
    for shift in range(1, 9):                                # each relative alignment
        room = torch.zeros(40000 + shift, dtype=flat.dtype, device="cuda")
        outs = [room[shift:17000 + shift]]
        lna.GradClip([17000], [kind]).clip([before[:17000]], 1.0, outs=outs)
        want = before[:17000].double() / true_norm([before[:17000]])
        ref.check("out", outs[0], (want.cpu().numpy(), 70 * ref.U * want.abs().cpu().numpy()), kind)
        assert (room[:shift] == 0).all() and (room[17000 + shift:] == 0).all()


@pytest.mark.parametrize("scale", [1e-30, 2.0 ** -60, 1e-12, 1e8, 1e18, 1e30, 1e37])
def test_squares_neither_overflow_nor_vanish(scale):
    g = make([5000, 333], ["f32", "bf16"], scale=scale)
    clip(g, 0.25 * true_norm(g))


def test_one_large_value_among_many():
    for big in (2.0 ** 20, 2.0 ** 27, 2.0 ** 28, 2.0 ** 29, 2.0 ** 30, 1e12):
        g = make([1 << 18], ["f32"], scale=2.0 ** 10)
        g[0][12345] = big
        clip(g, 0.25 * true_norm(g))


def test_zeros_and_none():
    import laplacian_nystr_attention_gb300 as lna
    g = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    plan = lna.GradClip.like(g)
    assert plan.clip(g, 0.0).item() == 0.0 and (g[0] == 0).all()
    empty = lna.GradClip([], [])
    assert empty.norm([]).item() == 0.0 and empty.clip([], 1.0).item() == 0.0
    none = lna.GradClip([0, 0], ["f32", "bf16"])
    z = [torch.zeros(0, device="cuda"), torch.zeros(0, device="cuda", dtype=torch.bfloat16)]
    assert none.norm(z).item() == 0.0 and none.clip(z, 1.0).item() == 0.0
    g = make([100], ["f32"])
    assert lna.GradClip.like(g).clip(g, 0.0).item() > 0 and (g[0] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_not_finite_changes_nothing(bad, kind):
    import laplacian_nystr_attention_gb300 as lna
    g = make([20000, 50], [kind, "f32"])
    g[0][17777] = bad
    before = [t.clone() for t in g]
    norm = lna.GradClip.like(g).clip(g, 1e-3)
    assert not np.isfinite(norm.item()) and np.isnan(norm.item()) == np.isnan(bad)
    outs = [torch.zeros_like(t) for t in g]
    lna.GradClip.like(g).clip(g, 1e-3, outs=outs)
    for a, b, c in zip(before, g, outs):
        assert torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0))
        assert torch.equal(a.nan_to_num(5.0), c.nan_to_num(5.0))


def test_bit_for_bit_and_captured():
    """Two graphs of one plan, replayed one after the other on new values."""
    import laplacian_nystr_attention_gb300 as lna
    counts, kinds = [70000, 3, 40000], ["f32", "bf16", "bf16"]
    sets = [make(counts, kinds, seed=s) for s in (0, 1)]
    plan = lna.GradClip(counts, kinds)
    want = []
    for g in sets:
        outs = [torch.empty_like(t) for t in g]
        want.append(([plan.clip(g, 1.5, outs=outs)], outs))
    live = [[t.clone() for t in sets[0]] for _ in range(2)]
    graphs, got = [], []
    for g in live:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [torch.empty_like(t) for t in g]
            got.append(([plan.clip(g, 1.5, outs=outs)], outs))
        graphs.append(graph)
    for order in ((0, 1), (1, 0)):
        for k, s in enumerate(order):
            for t, new in zip(live[k], sets[s]):
                t.copy_(new)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for k, s in enumerate(order):
            for a, b in zip(want[s][0] + want[s][1], got[k][0] + got[k][1]):
                assert torch.equal(a, b)


def test_refusals():
    import ctypes

    import laplacian_nystr_attention_gb300 as lna
    from laplacian_nystr_attention_gb300 import _lib
    flat = torch.zeros(4096, device="cuda")
    a, b, c = flat[:100], flat[100:200], flat[50:150]
    plan = lna.GradClip([100, 100], ["f32", "f32"])
    for grads, outs in (([a, a], None), ([a, c], None), ([a, b], [c, flat[300:400]]),
                        ([a, b], [b, a]), ([a, b], [flat[300:400], flat[399:499]]),
                        ([a, b], [flat[300:400], a])):
        with pytest.raises(lna.LaplAttnError) as e:
            plan.clip(grads, 1.0, outs=outs)
        assert e.value.status == _lib.LAPL_ERR_INVALID_ARG
    plan.clip([a, a], 1.0, outs=[flat[300:400], flat[400:500]])     # read twice: allowed
    plan.clip([a, b], 1.0, outs=[a, flat[400:500]])                 # one of them in place
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(lna.LaplAttnError):
            plan.clip([a, b], bad)
    with pytest.raises(ValueError):
        plan.clip([a], 1.0)
    with pytest.raises(ValueError):
        plan.norm([a, b.cpu()])
    p, st = flat.data_ptr(), torch.cuda.current_stream().cuda_stream
    need, vp = plan.workspace_bytes, ctypes.c_void_p
    good, null, odd = (vp * 2)(p, p + 400), (vp * 2)(p, None), (vp * 2)(p, p + 402)
    f = _lib.LIB.lapl_clip_norm
    assert f(plan.handle, null, p, p, need, st) == _lib.LAPL_ERR_INVALID_ARG
    assert f(plan.handle, None, p, p, need, st) == _lib.LAPL_ERR_INVALID_ARG
    assert f(plan.handle, good, None, p, need, st) == _lib.LAPL_ERR_INVALID_ARG
    assert f(plan.handle, good, p, None, need, st) == _lib.LAPL_ERR_INVALID_ARG
    assert f(plan.handle, odd, p, p, need, st) == _lib.LAPL_ERR_ALIGNMENT
    assert f(plan.handle, good, p + 2, p, need, st) == _lib.LAPL_ERR_ALIGNMENT
    assert f(plan.handle, good, p, p + 8, need, st) == _lib.LAPL_ERR_ALIGNMENT
    assert f(plan.handle, good, p, p, need - 1, st) == _lib.LAPL_ERR_WORKSPACE


def test_offsets_past_32_bits():
    import laplacian_nystr_attention_gb300 as lna
    t = torch.zeros((1 << 31) + 4099, dtype=torch.bfloat16, device="cuda")
    t[-1], t[5] = 3.0, 4.0
    out = torch.empty_like(t)
    assert lna.GradClip.like([t]).clip([t], 1.0, outs=[out]).item() == 5.0
    # 3 and 4 by 1/5 in fp32, rounded to bf16.
    assert out[-1].item() == torch.tensor(0.6).bfloat16() and out[5].item() == torch.tensor(0.8).bfloat16()
    assert out.count_nonzero() == 2
