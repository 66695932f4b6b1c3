"""GPU parity of the gated linear recurrence (lapl_scan_*) against its 64-bit reference, every value
within the bound of the roundings on its way (operators_reference.py)."""
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


def make(S, N, C, gate, dtype, seed=0, spread=1.5, shift=2.0):
    """(x, g, h0, dout, dfinal) as float64 arrays that dtype (fp32 for the states) holds."""
    rng = np.random.default_rng(seed)
    x, g = rng.standard_normal((S, N, C)), spread * rng.standard_normal((S, N, C)) + shift
    if gate == "decay":
        g = np.tanh(g)
    h0, dfinal = (ref.rounded(rng.standard_normal((S, C)), "f32") for _ in range(2))
    return ref.rounded(x, dtype), ref.rounded(g, dtype), h0, rng.standard_normal((S, N, C)), dfinal


def dev(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype]).cuda()


def run(S, N, C, gate="sigmoid", dtype="f32", out="f32", grad="f32", reverse=False, lens=None,
        h0=True, seed=0, packed=0, inputs=None):
    """Forward and backward, all results checked; the device results."""
    import laplacian_nystr_attention_gb300 as lna
    x, g, s0, dout, dfinal = inputs or make(S, N, C, gate, dtype, seed)
    s0 = s0 if h0 else None
    dfinal = dfinal if h0 else None
    dout = ref.rounded(dout, grad)
    want = ref.scan(x, g, gate, s0, lens, reverse, dout, dfinal)
    plan = lna.GatedScan(lna.make_scan_config(S, N, C, gate=gate, reverse=int(reverse),
                                              in_dtype=dtype, out_dtype=out, grad_dtype=grad,
                                              x_stride=packed, g_stride=packed))
    dx_, dg_ = dev(x, dtype), dev(g, dtype)
    if packed:
        both = torch.full((S, N, packed), 7.0, dtype=TYPES[dtype], device="cuda")
        both[..., :C], both[..., packed - C:] = dx_, dg_
        dx_, dg_ = both[..., :C], both[..., packed - C:]
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    states = torch.full(plan.states_shape, float("nan"), device="cuda")
    final = torch.full((S, C), float("nan"), device="cuda")
    y = torch.full((S, N, C), float("nan"), dtype=TYPES[out], device="cuda")
    plan.forward(dx_, dg_, h0=dev(s0), lengths=n, out=y, states=states, final=final)
    grads = None
    if packed:
        room = torch.full((S, N, packed), 5.0, dtype=TYPES[grad], device="cuda")
        grads = {"dx": room[..., :C], "dg": room[..., packed - C:]}
    bx, bg, b0 = plan.backward(dx_, dg_, states, dev(dout, grad), dfinal=dev(dfinal), lengths=n,
                               grads=grads)
    torch.cuda.synchronize()
    ref.check("h", y, want["h"], out)
    ref.check("final", final, want["final"])
    ref.check("states", states, want["states"])
    ref.check("dx", bx, want["dx"], grad)
    ref.check("dg", bg, want["dg"], grad)
    ref.check("dh0", b0, want["dh0"])
    if packed and packed > 2 * C:
        assert (room[..., C:packed - C] == 5.0).all()      # between the rows: left as it was
    info = _info(plan)
    plan.close()
    return (y, final, states, bx, bg, b0), info


def _info(plan):
    import laplacian_nystr_attention_gb300 as lna
    return lna.lapl_scan_plan_info_get(plan.handle)


@pytest.mark.parametrize("gate", ["decay", "sigmoid"])
@pytest.mark.parametrize("dtype,out,grad", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                            ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("N", [1, 16, 17, 300])
def test_types(gate, dtype, out, grad, N):
    run(3, N, 24, gate, dtype, out, grad)


@pytest.mark.parametrize("C", [1, 2, 3, 5, 8, 31, 33, 64, 65, 100, 130])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_channels(C, dtype):
    run(2, 83, C, "sigmoid", dtype, dtype, dtype)


@pytest.mark.parametrize("N", [2, 15, 31, 32, 127, 128, 129, 255, 257, 511, 1024, 2049, 5000])
def test_lengths_of_sequences(N):
    run(1, N, 40, "decay")


@pytest.mark.parametrize("gate", ["decay", "sigmoid"])
@pytest.mark.parametrize("S,N,C", [(1, 4100, 64), (1, 1040, 8), (700, 40, 64), (2, 6000, 320)])
def test_every_split_of_the_tokens(gate, S, N, C):
    """From one CTA a sequence to a cluster of CTAs."""
    _, info = run(S, N, C, gate, "bf16", "bf16", "bf16")
    assert (info["cluster"] > 1) == (S < 700)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padded_batch(reverse, dtype):
    lens = [0, 1, 15, 16, 17, 200, 213, 500, -3]           # 500: counts as N; -3: as 0
    run(9, 213, 48, "sigmoid", dtype, dtype, dtype, reverse=reverse, lens=lens)
    run(9, 213, 48, "decay", dtype, dtype, dtype, reverse=reverse, lens=lens, h0=False)


def test_padding_is_not_read():
    """Infinities and NaN behind a sequence's length change nothing."""
    import laplacian_nystr_attention_gb300 as lna
    S, N, C, lens = 3, 70, 16, [0, 33, 70]
    x, g, h0, dout, dfinal = (dev(a) for a in make(S, N, C, "sigmoid", "f32"))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    plan = lna.GatedScan(lna.make_scan_config(S, N, C))
    got = []
    for bad in (0.0, float("nan"), float("inf")):
        xs, gs, ds = x.clone(), g.clone(), dout.clone()
        for s, k in enumerate(lens):
            xs[s, k:], gs[s, k:], ds[s, k:] = bad, bad, bad
        states, final = torch.empty(plan.states_shape, device="cuda"), torch.empty_like(h0)
        y = plan.forward(xs, gs, h0=h0, lengths=n, states=states, final=final)
        got.append([y, states, final, *plan.backward(xs, gs, states, ds, dfinal, lengths=n)])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b) and torch.isfinite(a).all()
    assert torch.equal(got[0][2][0], h0[0])                # a length of zero hands h0 on


@pytest.mark.parametrize("gate", ["decay", "sigmoid"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("f32", "bf16")])
def test_few_tokens(gate, reverse, dtype, out):
    """One to eight tokens and just more; channels by four and not; several sequences a CTA and
    several CTAs a sequence; lengths of zero."""
    for N in (1, 2, 3, 4, 5, 8, 9):
        lens = [N, 0, 1, N - 1, N + 3, -2, N]
        for S, C, packed in ((7, 8, 0), (7, 65, 0), (7, 1100, 2200), (7, 12, 30)):
            run(S, N, C, gate, dtype, out, out, reverse=reverse, lens=lens, packed=packed)
    info = run(300, 1, 20, gate, dtype, out, h0=False)[1]
    assert info == {"cluster": 1, "lanes": 8, "threads": 256, "teams": 0}
    run(700, 32, 360, gate, dtype, out, reverse=reverse, lens=[32, 17, 16, 0, 31] * 140)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_tokens_misaligned(dtype):
    """Every pointer one element off 16 bytes, the states in place."""
    import laplacian_nystr_attention_gb300 as lna
    S, N, C = 3, 2, 64
    x, g, h0, dout, dfinal = make(S, N, C, "sigmoid", dtype, seed=4)
    dout = ref.rounded(dout, dtype)
    want = ref.scan(x, g, "sigmoid", h0, dout=dout, dfinal=dfinal)

    def off(a, kind):
        t = torch.empty(a.size + 1, dtype=TYPES[kind], device="cuda")[1:].view(a.shape)
        return t.copy_(dev(a, kind))

    state, out = off(h0, "f32"), off(x, dtype)
    plan = lna.GatedScan(lna.make_scan_config(S, N, C, in_dtype=dtype, out_dtype=dtype,
                                              grad_dtype=dtype))
    states = off(np.zeros(plan.states_shape), "f32")
    plan.forward(off(x, dtype), off(g, dtype), h0=state, states=states, final=state, out=out)
    ref.check("h", out, want["h"], dtype)
    ref.check("final", state, want["final"])
    last, dx, dg = off(dfinal, "f32"), off(x, dtype), off(g, dtype)
    plan.backward(off(x, dtype), off(g, dtype), states, off(dout, dtype), dfinal=last,
                  grads={"dx": dx, "dg": dg, "dh0": last})
    ref.check("dx", dx, want["dx"], dtype)
    ref.check("dg", dg, want["dg"], dtype)
    ref.check("dh0", last, want["dh0"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,packed", [(24, 48), (24, 64), (23, 47), (22, 46), (333, 700)])
def test_rows_apart(dtype, C, packed):
    run(2, 77, C, "sigmoid", dtype, dtype, dtype, packed=packed)


def test_reverse_is_the_recurrence_of_turned_tokens():
    import laplacian_nystr_attention_gb300 as lna
    S, N, C = 2, 401, 64
    x, g, h0, _, _ = (dev(a) for a in make(S, N, C, "sigmoid", "f32"))
    fwd = lna.GatedScan(lna.make_scan_config(S, N, C))
    rev = lna.GatedScan(lna.make_scan_config(S, N, C, reverse=1))
    a = fwd.forward(x, g, h0=h0)
    b = rev.forward(x.flip(1).contiguous(), g.flip(1).contiguous(), h0=h0)
    assert torch.equal(a, b.flip(1))


def test_four_dimensions_and_single_tokens():
    """[B, H, N, d] tensors; N tokens at once are N steps of one, the state handed on in place."""
    import laplacian_nystr_attention_gb300 as lna
    B, H, N, d = 2, 3, 37, 32
    x, g, h0, _, _ = make(B * H, N, d, "sigmoid", "bf16")
    want = ref.scan(x, g, "sigmoid", h0)
    xs, gs = (dev(a, "bf16").view(B, H, N, d) for a in (x, g))
    plan = lna.GatedScan(lna.make_scan_config(B * H, N, d, in_dtype="bf16"))
    y = plan.forward(xs, gs, h0=dev(h0))
    assert y.shape == (B, H, N, d)
    ref.check("h", y.view(B * H, N, d), want["h"])
    step = lna.GatedScan(lna.make_scan_config(B * H, 1, d, in_dtype="bf16"))
    state = dev(h0)
    for i in range(N):
        out = step.forward(xs[:, :, i:i + 1].contiguous(), gs[:, :, i:i + 1].contiguous(),
                           h0=state, final=state)
        ref.check("step", out.view(B * H, d), (want["h"][0][:, i], want["h"][1][:, i]))
    ref.check("final", state, want["final"])


@pytest.mark.parametrize("reverse", [False, True])
def test_state_in_place_with_clusters(reverse):
    """final may be h0, and dh0 dfinal, when several CTAs share a sequence."""
    import laplacian_nystr_attention_gb300 as lna
    S, N, C = 1, 5000, 64
    x, g, h0, dout, dfinal = (dev(a) for a in make(S, N, C, "sigmoid", "f32"))
    plan = lna.GatedScan(lna.make_scan_config(S, N, C, reverse=int(reverse)))
    assert _info(plan)["cluster"] > 1
    states, final = torch.empty(plan.states_shape, device="cuda"), torch.empty_like(h0)
    plan.forward(x, g, h0=h0, states=states, final=final)
    _, _, dh0 = plan.backward(x, g, states, dout, dfinal=dfinal)
    plan.forward(x, g, h0=h0, final=h0)
    plan.backward(x, g, states, dout, dfinal=dfinal, grads={"dh0": dfinal})
    assert torch.equal(h0, final) and torch.equal(dfinal, dh0)


@pytest.mark.parametrize("gate,value", [("decay", 0.0), ("decay", 1.0), ("decay", -1.0),
                                        ("sigmoid", 100.0), ("sigmoid", -100.0),
                                        ("sigmoid", float("inf")), ("sigmoid", float("-inf")),
                                        ("sigmoid", 12.0)])
def test_gates_at_their_ends(gate, value):
    """Closed, open and alternating gates over a length where sums grow; exp's ends."""
    S, N, C = 2, 1500, 32
    x, g, h0, dout, dfinal = make(S, N, C, gate, "f32")
    g[:] = value
    run(S, N, C, gate, inputs=(x, g, h0, dout, dfinal))


def test_bit_for_bit_and_captured():
    """Two calls agree bit for bit, and so does a replayed graph on changed inputs."""
    import laplacian_nystr_attention_gb300 as lna
    S, N, C = 2, 3000, 96
    plan = lna.GatedScan(lna.make_scan_config(S, N, C))
    ins = [[dev(a) for a in make(S, N, C, "sigmoid", "f32", seed=s)] for s in (0, 1)]
    states, final = torch.empty(plan.states_shape, device="cuda"), torch.empty(S, C, device="cuda")

    def both(x, g, h0, dout, dfinal):
        y = plan.forward(x, g, h0=h0, states=states, final=final)
        return (y, final, *plan.backward(x, g, states, dout, dfinal))

    want = [[t.clone() for t in both(*i)] for i in ins]
    again = [t.clone() for t in both(*ins[0])]
    assert all(torch.equal(a, b) for a, b in zip(want[0], again))
    live = [t.clone() for t in ins[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*live)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(*live)
    for k in (0, 1):
        for t, new in zip(live, ins[k]):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[k], got))


def test_given_stream():
    import laplacian_nystr_attention_gb300 as lna
    S, N, C = 4, 900, 64
    x, g, h0, dout, _ = (dev(a) for a in make(S, N, C, "sigmoid", "f32"))
    plan = lna.GatedScan(lna.make_scan_config(S, N, C))
    want = plan.forward(x, g, h0=h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.forward(x, g, h0=h0, stream=side)
    side.synchronize()
    assert torch.equal(want, got)


def test_refusals():
    import laplacian_nystr_attention_gb300 as lna
    from laplacian_nystr_attention_gb300 import _lib
    S, N, C = 2, 5, 8
    h = _lib.lapl_scan_create(lna.make_scan_config(S, N, C, in_dtype="bf16"))
    x = torch.zeros(S * N * C, device="cuda")
    p, st = x.data_ptr(), torch.cuda.current_stream().cuda_stream
    fwd, bwd = _lib.LIB.lapl_scan_forward, _lib.LIB.lapl_scan_backward
    for k in (1, 2, 5):                                     # x, g, out
        a = [h, p, p, None, None, p, None, None, st]
        a[k] = None
        assert fwd(*a) == _lib.LAPL_ERR_INVALID_ARG
    for k, off in ((1, 1), (2, 1), (3, 2), (4, 2), (5, 2), (6, 2), (7, 2)):
        a = [h, p, p, None, None, p, None, None, st]
        a[k] = p + off
        assert fwd(*a) == _lib.LAPL_ERR_ALIGNMENT
    for k in (1, 2, 3, 5, 7, 8):                            # x, g, states, dout, dx, dg
        a = [h, p, p, p, None, p, None, p, p, None, st]
        a[k] = None
        assert bwd(*a) == _lib.LAPL_ERR_INVALID_ARG
    for k, off in ((1, 1), (2, 1), (3, 2), (4, 2), (5, 2), (6, 2), (7, 2), (8, 2), (9, 2)):
        a = [h, p, p, p, None, p, None, p, p, None, st]
        a[k] = p + off
        assert bwd(*a) == _lib.LAPL_ERR_ALIGNMENT
    _lib.lapl_scan_destroy(h)
    empty = lna.GatedScan(lna.make_scan_config(0, N, C))
    y = empty.forward(x.view(-1, N, C)[:0], x.view(-1, N, C)[:0])
    assert y.shape == (0, N, C)
    plan = lna.GatedScan(lna.make_scan_config(S, N, C))
    good = x.view(S, N, C)
    for bad in (good.cpu(), good.bfloat16(), good[:1], good.transpose(0, 1)):
        with pytest.raises(ValueError):
            plan.forward(bad, good)
        with pytest.raises(ValueError):
            plan.forward(good, good, out=bad)
    with pytest.raises(lna.LaplAttnError):
        lna.GatedScan(lna.make_scan_config(S, 0, C))


# ---- long sequences: the pipelined kernels ------------------------------------------------

@pytest.mark.parametrize("gate", ["decay", "sigmoid"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype,out,grad", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                            ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")])
def test_long_types(gate, reverse, dtype, out, grad):
    run(3, 1111, 72, gate, dtype, out, grad, reverse=reverse, lens=[1111, 600, 1000])


@pytest.mark.parametrize("C", [1, 2, 8, 10, 15, 16, 31, 32, 33, 63, 64, 65, 100, 129, 334])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_channels(C, dtype):
    """Rows of 16 bytes, of 4, and of odd bf16 channels (the other kernels)."""
    run(2, 1025, C, "sigmoid", dtype, dtype, dtype)


@pytest.mark.parametrize("S,N,C", [(1, 512, 8), (50, 600, 64), (1, 768, 8), (1, 20000, 64),
                                   (3, 3000, 16), (40, 1500, 64), (160, 800, 32), (2, 9001, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_splits(S, N, C, dtype):
    """One CTA a sequence up to a cluster of eight; lanes over 8, 16 or 32 pieces of a row."""
    run(S, N, C, "sigmoid", dtype, dtype, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,packed", [(24, 48), (24, 64), (22, 46), (64, 128), (333, 672), (334, 670)])
def test_long_rows_apart(dtype, C, packed):
    run(2, 900, C, "sigmoid", dtype, dtype, dtype, packed=packed, lens=[900, 333])


def test_long_and_short_lengths():
    run(6, 2000, 48, "sigmoid", "bf16", "bf16", "bf16", lens=[0, 1, 17, 1999, 2000, 1024])
    run(6, 2000, 48, "decay", lens=[0, 1, 17, 1999, 2000, 1024], reverse=True, h0=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_misaligned(dtype):
    """Tensors off 16 bytes, and off the pairs that bf16 channels are read in."""
    import laplacian_nystr_attention_gb300 as lna
    S, N, C = 2, 1000, 32
    x, g, h0, dout, dfinal = make(S, N, C, "sigmoid", dtype)
    want = None
    for off in (0, 1, 2, 4, 8):
        def place(a, t, off=off):
            room = torch.zeros(a.size + 16, dtype=TYPES[t], device="cuda")
            got = room[off:off + a.size].view(a.shape)
            got.copy_(dev(a, t))
            return got
        plan = lna.GatedScan(lna.make_scan_config(S, N, C, in_dtype=dtype, out_dtype=dtype,
                                                  grad_dtype=dtype))
        xs, gs, ds = place(x, dtype), place(g, dtype), place(ref.rounded(dout, dtype), dtype)
        hs, dfs = place(h0, "f32"), place(dfinal, "f32")
        states = place(np.zeros(plan.states_shape), "f32")
        y = plan.forward(xs, gs, h0=hs, states=states, out=place(np.zeros((S, N, C)), dtype))
        grads = {"dx": place(np.zeros((S, N, C)), dtype), "dg": place(np.zeros((S, N, C)), dtype)}
        dx, dg, dh0 = plan.backward(xs, gs, states, ds, dfinal=dfs, grads=grads)
        if want is None:
            want = ref.scan(x, g, "sigmoid", h0, dout=ref.rounded(dout, dtype), dfinal=dfinal)
        ref.check("h", y, want["h"], dtype)
        ref.check("states", states, want["states"])
        ref.check("dx", dx, want["dx"], dtype)
        ref.check("dg", dg, want["dg"], dtype)
        ref.check("dh0", dh0, want["dh0"])


def test_long_bit_for_bit_on_two_streams():
    """Two plans at work at once, a few calls each, on streams of their own."""
    import laplacian_nystr_attention_gb300 as lna
    S, N, C = 4, 5000, 128
    plans = [lna.GatedScan(lna.make_scan_config(S, N, C)) for _ in range(2)]
    ins = [[dev(a) for a in make(S, N, C, "sigmoid", "f32", seed=s)] for s in (0, 1)]

    def both(plan, x, g, h0, dout, dfinal):
        states, final = torch.empty(plan.states_shape, device="cuda"), torch.empty_like(h0)
        y = plan.forward(x, g, h0=h0, states=states, final=final)
        return [y, final, states, *plan.backward(x, g, states, dout, dfinal)]

    want = [both(p, *i) for p, i in zip(plans, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in plans]
    for _ in range(3):
        got = []
        for p, i, s in zip(plans, ins, streams):
            with torch.cuda.stream(s):
                got.append(both(p, *i))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(t, u) for t, u in zip(a, b))


def test_long_plans_side_by_side():
    """A plan whose clusters need less shared memory, made after one that needs more."""
    import laplacian_nystr_attention_gb300 as lna
    made = []
    for S, N in ((1, 20000), (600, 800)):
        x, g, *_ = make(S, N, 64, "sigmoid", "bf16", seed=3)
        plan = lna.GatedScan(lna.make_scan_config(S, N, 64, in_dtype="bf16", grad_dtype="bf16"))
        made.append((plan, dev(x, "bf16"), dev(g, "bf16"), ref.scan(x, g, "sigmoid")))
    infos = [_info(m[0]) for m in made]
    assert infos[0]["cluster"] > infos[1]["cluster"] and infos[1]["teams"]
    for plan, x, g, want in made:
        states = torch.empty(plan.states_shape, device="cuda")
        ref.check("h", plan.forward(x, g, states=states), want["h"])
        plan.backward(x, g, states, x)
    torch.cuda.synchronize()


@pytest.mark.parametrize("S,N,C", [(1, 20000, 64), (40, 1500, 64)])
def test_wait_that_gives_up_is_reported(S, N, C):
    """The last round's maps are never sent: the waits for them run out after 2 ms, the kernel ends,
    and the report says so; the next call is right again."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.GatedScan(lna.make_scan_config(S, N, C))
    assert _info(plan)["teams"] > 0
    x, g, h0, dout, dfinal = (dev(a) for a in make(S, N, C, "sigmoid", "f32"))
    states, final = torch.empty(plan.states_shape, device="cuda"), torch.empty_like(h0)
    want = plan.forward(x, g, h0=h0, states=states)
    grads = plan.backward(x, g, states, dout, dfinal)
    st = torch.cuda.current_stream().cuda_stream
    lna.lapl_scan_set_fault_injection(plan.handle, 2_000_000, 1)
    for call in (lambda: plan.forward(x, g, h0=h0), lambda: plan.backward(x, g, states, dout)):
        call()
        with pytest.raises(lna.LaplAttnError) as e:
            lna.lapl_scan_device_errors(plan.handle, st)
        assert e.value.status == 6 and "recurrence" in str(e.value)
    lna.lapl_scan_set_fault_injection(plan.handle, 0, 0)
    assert torch.equal(plan.forward(x, g, h0=h0), want)
    assert all(torch.equal(a, b) for a, b in zip(grads, plan.backward(x, g, states, dout, dfinal)))
    assert lna.lapl_scan_device_errors(plan.handle, st) == 0


def test_no_wait_gave_up():
    """After all of the above the device error word is clear."""
    import laplacian_nystr_attention_gb300 as lna
    att = lna.LaplacianNystromAttention(lna.make_config(1, 1, 4, 4, 8, 4))
    assert lna.lapl_attn_device_errors(att.handle, torch.cuda.current_stream().cuda_stream) == 0
    att.close()


@pytest.mark.parametrize("S,N,C", [(36000, 512, 128), (2800, 3000, 258)])
def test_offsets_past_32_bits(S, N, C):
    """More than 2^31 values: the last sequence, by the kernels for short and for long ones."""
    import laplacian_nystr_attention_gb300 as lna
    assert S * N * C > 1 << 31
    x, g, _, dout, _ = make(1, N, C, "sigmoid", "bf16", seed=9)
    dout = ref.rounded(dout, "bf16")
    want = ref.scan(x, g, "sigmoid", dout=dout)
    # (S, N, C) tensors are 4.6 GB each: the others' values are those of zeros.
    big = [torch.zeros(S, N, C, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for t, a in zip(big, (x, g, dout)):
        t[-1:] = dev(a, "bf16")
    plan = lna.GatedScan(lna.make_scan_config(S, N, C, in_dtype="bf16", out_dtype="bf16",
                                              grad_dtype="bf16"))
    states = torch.empty(plan.states_shape, device="cuda")
    y = plan.forward(big[0], big[1], states=states)
    dx, dg, _ = plan.backward(big[0], big[1], states, big[2])
    ref.check("h", y[-1:], want["h"], "bf16")
    ref.check("dx", dx[-1:], want["dx"], "bf16")
    ref.check("dg", dg[-1:], want["dg"], "bf16")
    assert (y[:-1] == 0).all() and (dx[:-1] == 0).all()
