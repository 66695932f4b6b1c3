"""The gated linear recurrence where its kernels can go wrong: waits that give up in the middle of a
sequence, gates at both ends of their range, states that are not finite."""
import numpy as np
import pytest
import torch

import operators_reference as ref

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


# ---- waits that give up -------------------------------------------------------------------

@pytest.mark.parametrize("S,N,C", [(1, 20000, 64), (40, 1500, 64), (1, 60000, 8), (200, 9000, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("wait_ns,skip_last", [(2_000_000, 1000000), (2_000_000, 7), (1, 0)])
def test_wait_that_gives_up_early(S, N, C, dtype, wait_ns, skip_last):
    """A wait gives up with many rounds to go, in clusters of one CTA up to eight: the first round's
    maps never come, or the seventh last's; or waits of 1 ns give up on maps that come a little later
    (which a quick cluster need not let happen).  The kernel ends, the report says so, and the next
    call is right."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.GatedScan(lna.make_scan_config(S, N, C, in_dtype=dtype, out_dtype=dtype,
                                              grad_dtype=dtype))
    assert lna.lapl_scan_plan_info_get(plan.handle)["teams"] > 0
    x, g, dout = (randn(S, N, C, seed=k, dtype=dtype) for k in range(3))
    h0, dfinal = randn(S, C, seed=3), randn(S, C, seed=4)
    states, other = (torch.empty(plan.states_shape, device="cuda") for _ in range(2))
    want = plan.forward(x, g, h0=h0, states=states)
    grads = plan.backward(x, g, states, dout, dfinal)
    st = torch.cuda.current_stream().cuda_stream
    assert lna.lapl_scan_device_errors(plan.handle, st) == 0
    lna.lapl_scan_set_fault_injection(plan.handle, wait_ns, skip_last)
    for call in (lambda: plan.forward(x, g, h0=h0, states=other),
                 lambda: plan.backward(x, g, states, dout, dfinal)):
        call()
        try:
            lna.lapl_scan_device_errors(plan.handle, st)
            assert not skip_last
        except lna.LaplAttnError as e:
            assert e.status == 6 and "recurrence" in str(e)
    lna.lapl_scan_set_fault_injection(plan.handle, 0, 0)
    assert torch.equal(plan.forward(x, g, h0=h0), want)
    assert all(torch.equal(a, b) for a, b in zip(grads, plan.backward(x, g, states, dout, dfinal)))
    assert lna.lapl_scan_device_errors(plan.handle, st) == 0


def test_a_wait_that_gave_up_is_told_in_python():
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.GatedScan(lna.make_scan_config(2, 5000, 64))
    x, g = randn(2, 5000, 64), randn(2, 5000, 64, seed=1)
    plan.forward(x, g)
    plan.check_device_errors()
    lna.lapl_scan_set_fault_injection(plan.handle, 2_000_000, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        plan.forward(x, g, stream=stream)
        with pytest.raises(lna.LaplAttnError) as e:
            plan.check_device_errors(stream=stream)
        assert e.value.status == 6
        plan.check_device_errors()
    lna.lapl_scan_set_fault_injection(plan.handle, 0, 0)
    plan.forward(x, g)
    plan.check_device_errors()


# ---- gates at both ends -------------------------------------------------------------------

def sigmoid_scan(x, g, h0, dout, dfinal):
    """{name: (value, bound)} in 64 bits; g in [-80, 80].

    U is half a step of fp32.  The kernels' a and z = 1 - a are each off by at most 12 U of themselves:
    exp(g) by 4 (the hardware's 2 ulp), 2 (what its argument lacks, a second-order term) and 1 (a
    product), and the sum by 1, the reciprocal by 2 (1 ulp), the last product by 1.  A step's two
    products and sum add 3, or as maps of runs of 16 tokens and their compositions at most the 4 that
    are left of 16 for every token: 16 U of |a h| + |z x|, each of them of itself.  Backward likewise,
    E = a D: 16 U of |a D|; dx = z D: 16; dg = a z (h - x) D: a and z 24, products and the difference 5,
    under 32."""
    U = ref.U
    S, N, C = x.shape
    a, z = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    b = z * x
    h, H, E = h0, np.abs(h0), np.zeros_like(h0)
    before, Hb, Eb, after, Ea = (np.empty((S, N, C)) for _ in range(5))
    for i in range(N):
        before[:, i], Hb[:, i], Eb[:, i] = h, H, E
        E = a[:, i] * E + 16 * U * (a[:, i] * H + np.abs(b[:, i]))
        H = a[:, i] * H + np.abs(b[:, i])
        h = a[:, i] * h + b[:, i]
        after[:, i], Ea[:, i] = h, E
    out = {"h": (after, Ea), "final": (h, E), "states": (before[:, ::16], Eb[:, ::16])}
    D, M, E = dfinal, np.abs(dfinal), np.zeros_like(h0)
    dx, ex, dg, eg = (np.empty((S, N, C)) for _ in range(4))
    for i in reversed(range(N)):
        here, mag = D + dout[:, i], M + np.abs(dout[:, i])
        eh = E + U * mag
        slope, ms = before[:, i] - x[:, i], Hb[:, i] + np.abs(x[:, i])
        k = a[:, i] * z[:, i]
        dx[:, i], ex[:, i] = z[:, i] * here, z[:, i] * (eh + 16 * U * mag)
        dg[:, i] = k * slope * here
        eg[:, i] = k * (np.abs(slope) * eh + Eb[:, i] * mag + 32 * U * ms * mag)
        D, M, E = a[:, i] * here, a[:, i] * mag, a[:, i] * (eh + 16 * U * mag)
    out.update(dx=(dx, ex), dg=(dg, eg), dh0=(D, E))
    return out


# The three kinds of kernels: few tokens (one at a time, up to eight, up to 32 with many channels),
# up to some hundred, and long ones; pairs of bf16 channels and not.
GATE_SHAPES = [(3, 1, 64), (3, 4, 64), (5, 7, 66), (120, 30, 2300), (3, 40, 65), (2, 300, 64),
               (600, 40, 64), (2, 1500, 64), (3, 900, 72)]


@pytest.mark.parametrize("S,N,C", GATE_SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("kind", [-8.0, -12.0, -17.0, -30.0, -80.0, 8.0, 17.0, "some"])
def test_gates_that_are_nearly_closed_or_open(S, N, C, dtype, reverse, kind):
    """States and gradients relative to a h, z x and a D, however small a or z is: gates all alike, or
    one token in six reset to one of them, with large first states before it."""
    import laplacian_nystr_attention_gb300 as lna
    rng = np.random.default_rng(11)
    x, dout = (ref.rounded(rng.standard_normal((S, N, C)), t) for t in (dtype, "f32"))
    h0, dfinal = (ref.rounded(rng.standard_normal((S, C)), "f32") for _ in range(2))
    if kind == "some":
        g = 1 + 2 * rng.standard_normal((S, N, C))
        pick = rng.choice([-8.0, -12.0, -17.0, -30.0, -60.0, 8.0, 12.0, 30.0], size=g.shape)
        g = ref.rounded(np.where(rng.random(g.shape) < 1 / 6, pick, g), dtype)
        h0 = ref.rounded(1e6 * h0, "f32")
    else:
        g = np.full((S, N, C), kind)
    turn = (lambda t: t[:, ::-1]) if reverse else (lambda t: t)
    want = sigmoid_scan(*(turn(t) for t in (x, g)), h0, turn(dout), dfinal)
    plan = lna.GatedScan(lna.make_scan_config(S, N, C, reverse=int(reverse), in_dtype=dtype))
    dev = lambda t, k="f32": torch.from_numpy(t).to(TYPES[k]).cuda()
    xs, gs = dev(x, dtype), dev(g, dtype)
    states, final = torch.empty(plan.states_shape, device="cuda"), torch.empty(S, C, device="cuda")
    h = plan.forward(xs, gs, h0=dev(h0), states=states, final=final)
    dx, dg, dh0 = plan.backward(xs, gs, states, dev(dout), dfinal=dev(dfinal))
    got = dict(h=h, final=final, states=states, dx=dx, dg=dg, dh0=dh0)
    for name, t in got.items():
        value, bound = want[name]
        if name in ("h", "dx", "dg"):
            value, bound = turn(value), turn(bound)
        ref.check(name, t, (value, bound))


def test_a_reset_gate_leaves_nothing_of_a_large_state():
    """h = 10^6 before a gate of -80: what is left is x, to its last bit (a h = 2e-29)."""
    import laplacian_nystr_attention_gb300 as lna
    for N, at in ((1, 0), (40, 7), (1500, 700)):
        x, g = torch.full((1, N, 8), 0.1, device="cuda"), torch.full((1, N, 8), 3.0, device="cuda")
        g[:, at] = -80.0
        h0 = torch.full((1, 8), 1e6, device="cuda")
        if at:
            x[:, at - 1] = 1e8
        h = lna.GatedScan(lna.make_scan_config(1, N, 8)).forward(x, g, h0=h0)
        assert (h[:, at] == x[:, at]).all()


# ---- states that are not finite -----------------------------------------------------------

@pytest.mark.parametrize("S,N,C,lens", [(2, 3, 8, [3, 2]), (2, 30, 9, [30, 20]),
                                        (2, 300, 64, [300, 150]), (2, 1500, 64, [1500, 700])])
@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_state_that_is_not_finite_stays_so(S, N, C, lens, gate, dtype, bad):
    """From the token on whose x (or, a NaN, whose g) is not finite its channel's states are not
    finite, to the last one, padding or not; everything else is as without it.  Backward likewise:
    dg from the next token on; dx and dh0 do not know of it."""
    import laplacian_nystr_attention_gb300 as lna
    x, g, dout = (randn(S, N, C, seed=k, dtype=dtype) for k in range(3))
    if gate == "decay":
        g = torch.sigmoid(g + 2)
    plan = lna.GatedScan(lna.make_scan_config(S, N, C, gate=gate, in_dtype=dtype, grad_dtype=dtype))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def both():
        states, final = torch.empty(plan.states_shape, device="cuda"), torch.empty(S, C, device="cuda")
        h = plan.forward(x, g, lengths=n, states=states, final=final)
        return [h, final, *plan.backward(x, g, states, dout, lengths=n)]

    want = [t.clone() for t in both()]
    at, c = lens[1] // 2, C - 1
    x[1, at, c] = bad
    h, final, dx, dg, dh0 = both()
    hit = torch.zeros(S, N, C, dtype=torch.bool, device="cuda")
    hit[1, at:lens[1], c] = True
    assert torch.equal(~torch.isfinite(h), hit)
    assert torch.equal(h[~hit], want[0][~hit])
    lost = torch.zeros_like(final, dtype=torch.bool)
    lost[1, c] = True
    assert torch.equal(~torch.isfinite(final), lost) and torch.equal(final[~lost], want[1][~lost])
    assert torch.equal(dx, want[2]) and torch.equal(dh0, want[4])
    if gate == "decay":     # dg is h_{i-1} D
        hit[1, at, c] = False
    assert torch.equal(~torch.isfinite(dg), hit)
    assert torch.equal(dg[~hit], want[3][~hit])
