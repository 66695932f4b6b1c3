"""The operators as they are used together: a block of attention, residual + norm and recurrence,
forward and backward, and its gradients clipped, against the 64-bit oracle and references."""
import numpy as np
import pytest
import torch

import operators_reference as ref
from lapl_workloads import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import oracle
    oracle.build()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def rel(got, want):
    """Largest difference over the largest value, as the attention's own tests measure."""
    got = got.double().cpu().numpy()
    return np.abs(got - want).max() / np.abs(want).max()


def test_training_step():
    """attention -> + residual, norm -> recurrence over the tokens -> loss, and back to Q, K, V,
    the residual, the norm's weight, the gate and the state, clipped to a largest norm.

    Tolerance 2e-4: the attention's 1e-4 forward, whose error the norm (of about unit gain here)
    and the recurrence (a mean) hand on once in each direction."""
    import laplacian_nystr_attention_gb300 as lna
    import oracle
    w = WORKLOADS["tiny_f32"].replace(batch=2, heads=2)
    B, H, N, d = w.batch, w.heads, w.n, w.head_dim
    rng = np.random.default_rng(5)
    q, k, v = make_inputs(w)
    W = H * d
    res, gate, dh = (ref.rounded(rng.standard_normal((B, N, W)), "f32") for _ in range(3))
    weight = ref.rounded(1 + 0.1 * rng.standard_normal(W), "f32")
    h0 = ref.rounded(rng.standard_normal((B, W)), "f32")

    # 64 bits
    o, _ = oracle.forward(w.config(), q, k, v)
    n = ref.norm(o, res, weight, float(np.float32(1e-6)))
    s = ref.scan(n["y"][0], gate, "sigmoid", h0, dout=dh)
    nb = ref.norm_backward(n["sum"][0], n["rstd"][0], weight, s["dx"][0], None, H)
    dq, dk, dv, _, aq, ak = oracle.backward(w.config(), q, k, v, nb["dx"][0].astype(np.float32))

    # the library
    att = lna.LaplacianNystromAttention(lna.make_config(**w.config()))
    norm = lna.ResidualNorm(lna.make_norm_config(B, H, N, d))
    mix = lna.GatedScan(lna.make_scan_config(B, N, W))
    Q, K, V, R, G, Wt, H0 = (dev(a) for a in (q, k, v, res, gate, weight, h0))
    total, rstd = torch.empty(B, N, W, device="cuda"), torch.empty(B, N, device="cuda")
    states = torch.empty(mix.states_shape, device="cuda")
    out = att.forward(Q, K, V, keep_for_backward=True)
    y = norm.forward(out, Wt, residual=R, sum=total, rstd=rstd)
    h = mix.forward(y, G, h0=H0, states=states)
    dy, dgate, dh0 = mix.backward(y, G, states, dev(dh))
    dout, dres, dweight = norm.backward(total, rstd, Wt, dy)
    gq, gk, gv, gb = att.backward(Q, K, V, dout)

    assert rel(h, s["h"][0]) < 2e-4
    for name, got, want in (("dres", dres, nb["dres"][0]), ("dweight", dweight, nb["dweight"][0]),
                            ("dgate", dgate, s["dg"][0]), ("dh0", dh0, s["dh0"][0]),
                            ("dv", gv, dv)):
        assert rel(got, want) < 2e-4, name
    for got, want, tie in ((gq, dq, aq), (gk, dk, ak)):     # sign decisions at ties, as elsewhere
        off = np.abs(got.double().cpu().numpy() - want) - tie
        assert off.max() < 2e-4 * np.abs(want).max()

    grads = [gq, gk, gv, gb, dres, dweight, dgate, dh0]
    before = [g.clone() for g in grads]
    clip = lna.GradClip.like(grads)
    size = clip.clip(grads, 0.1).item()
    want = np.sqrt(sum((g.double().cpu().numpy() ** 2).sum() for g in before))
    assert abs(size - want) <= 64 * ref.U * want
    assert abs(clip.norm(grads).item() - 0.1) <= 0.1 * 2 * 64 * ref.U
    for a, b in zip(grads, before):
        assert torch.allclose(a, b * (0.1 / want), rtol=1e-5, atol=0)


def test_attention_backward_clips():
    """backward(max_norm=) is backward() and then GradClip on the four gradients."""
    import laplacian_nystr_attention_gb300 as lna
    w = WORKLOADS["tiny_f32"].replace(heads=2)
    q, k, v = (dev(a) for a in make_inputs(w))
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).cuda()
    att = lna.LaplacianNystromAttention(lna.make_config(**w.config()))
    att.forward(q, k, v, keep_for_backward=True)
    plain = [t.clone() for t in att.backward(q, k, v, dout)]
    att.forward(q, k, v, keep_for_backward=True)
    clipped = att.backward(q, k, v, dout, max_norm=0.5)
    size = lna.GradClip.like(plain).clip(plain, 0.5)
    assert torch.equal(att.grad_norm, size) and size.item() > 0.5
    for a, b in zip(plain, clipped):
        assert torch.equal(a, b)
    att.close()


def test_attention_backward_clips_an_empty_batch():
    """No gradient reaches the bias, whatever its tensor held."""
    import laplacian_nystr_attention_gb300 as lna
    w = WORKLOADS["tiny_f32"].replace(heads=2, batch=0)
    att = lna.LaplacianNystromAttention(lna.make_config(**w.config()))
    empty = torch.empty(0, 2, w.grid_h * w.grid_w, w.head_dim, device="cuda")
    dbias = torch.full((2, att.cfg.num_landmarks), 7.0, device="cuda")
    att.forward(empty, empty, empty, keep_for_backward=True)
    got = att.backward(empty, empty, empty, empty, grads={"dbias": dbias}, max_norm=0.5)
    assert att.grad_norm.item() == 0 and torch.equal(got[3], torch.zeros_like(dbias))
    with pytest.raises(ValueError):
        att.backward(empty, empty, empty, empty, grads={"dbias": dbias}, max_norm=-1.0)
    att.close()


def test_training_step_captured():
    """norm -> recurrence -> back -> clip in one graph, replayed."""
    import laplacian_nystr_attention_gb300 as lna
    B, H, N, d = 2, 2, 500, 32
    W = H * d
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(B, H, N, d, generator=gen, device="cuda")
    res, gate, dh = (torch.randn(B, N, W, generator=gen, device="cuda") for _ in range(3))
    weight = torch.ones(W, device="cuda")
    norm = lna.ResidualNorm(lna.make_norm_config(B, H, N, d))
    mix = lna.GatedScan(lna.make_scan_config(B, N, W))
    clip = lna.GradClip([x.numel(), W, gate.numel()], ["f32"] * 3)
    total, rstd = torch.empty(B, N, W, device="cuda"), torch.empty(B, N, device="cuda")
    states = torch.empty(mix.states_shape, device="cuda")

    def step():
        y = norm.forward(x, weight, residual=res, sum=total, rstd=rstd)
        mix.forward(y, gate, states=states)
        dy, dgate, _ = mix.backward(y, gate, states, dh)
        dx, _, dweight = norm.backward(total, rstd, weight, dy)
        return [clip.clip([dx, dweight, dgate], 1.0), dx, dweight, dgate]

    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
