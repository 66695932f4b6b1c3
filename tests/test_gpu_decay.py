"""GPU parity of the linear attention with decays (lapl_decay_*) against its 64-bit reference, every
value within the bound of the roundings on its way (more_operators_reference.py)."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
from operators_reference import rounded

pytestmark = pytest.mark.gpu

TYPES = ref.TYPES


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def dev(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype]).cuda()


def off_by_one(t):
    """The same values one element off an allocation's start."""
    if t is None:
        return None
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    got = room[1:].view(t.shape)
    got.copy_(t)
    return got


LOGS = (-1e-3, -0.05, 0.0, -0.6, -3.0)


def make(B, H, N, a, b, dtype="bf16", grad=None, seed=0, state=True, logs=LOGS):
    rng = np.random.default_rng(seed)
    grad = grad or dtype
    draw = rng.standard_normal
    return dict(q=rounded(draw((B, H, N, a)), dtype), k=rounded(draw((B, H, N, a)), dtype),
                v=rounded(draw((B, H, N, b)), dtype), dout=rounded(draw((B, H, N, b)), grad),
                state=rounded(3 * draw((B, H, a, b)), "f32") if state else None,
                dfinal=rounded(draw((B, H, a, b)), "f32") if state else None,
                log_decay=rounded(np.resize(logs, H), "f32"))


def run(B, H, N, a, b, dtype="bf16", out=None, grad=None, reverse=False, lens=None, state=True,
        seed=0, shift=False, backward=True, tc=None, data=None, logs=LOGS):
    """Forward and backward of one shape, checked; the outputs."""
    import laplacian_nystr_attention_gb300 as lna
    out, grad = out or dtype, grad or dtype
    m = data or make(B, H, N, a, b, dtype, grad, seed, state, logs)
    scale = float(np.float32(a ** -0.5))
    plan = lna.DecayAttention(lna.make_decay_config(B, H, N, a, b, scale=scale, reverse=int(reverse),
                                                    in_dtype=dtype, out_dtype=out,
                                                    grad_dtype=grad))
    info = lna.lapl_decay_plan_info_get(plan.handle)
    if tc is not None:
        assert bool(info["tensor_cores"]) == tc, info
    place = off_by_one if shift else (lambda t: t)
    q, k, v = (place(dev(m[n], dtype)) for n in "qkv")
    log_decay, s0, df = dev(m["log_decay"]), place(dev(m["state"])), place(dev(m["dfinal"]))
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = ref.decay(*(m[n] for n in "qkv"), m["log_decay"], scale, m["state"], lens, reverse,
                     m["dout"] if backward else None, m["dfinal"],
                     tensor_cores=bool(info["tensor_cores"]))
    final = torch.full(plan.state_shape, float("nan"), device="cuda")
    o = place(torch.full((B, H, N, b), float("nan"), dtype=TYPES[out], device="cuda"))
    plan.forward(q, k, v, log_decay, state=s0, lengths=lengths, out=o, final=final)
    plan.check_device_errors()
    ref.check("out", o, want["out"], out)
    ref.check("final", final, want["final"])
    if not backward:
        return o, final
    dout = place(dev(m["dout"], grad))
    got = plan.backward(q, k, v, log_decay, dout, state=s0, dfinal=df, lengths=lengths)
    plan.check_device_errors()
    for name, t in zip(("dq", "dk", "dv", "dstate"), got):
        ref.check(name, t, want[name], "f32" if name == "dstate" else grad)
    return (o, final, *got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("other", ["f32", "bf16"])
def test_types(dtype, other):
    run(2, 3, 37, 16, 24, dtype, out=other, grad=other)
    run(2, 3, 150, 16, 24, dtype, out=other, grad=other)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 400])
@pytest.mark.parametrize("reverse", [False, True])
def test_lengths_of_sequences(N, reverse):
    run(1, 2, N, 64, 64, "bf16", reverse=reverse, seed=N, tc={1: False, 2: False}.get(
        N, True if N >= 63 else None))
    run(1, 2, N, 24, 40, "f32", reverse=reverse, seed=N, tc=False)


@pytest.mark.parametrize("a,b", [(1, 1), (3, 5), (8, 8), (16, 64), (64, 8), (32, 32), (33, 64),
                                 (64, 33), (48, 56), (65, 64), (64, 65), (128, 128), (100, 128),
                                 (128, 7), (127, 127)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dimensions(a, b, dtype):
    run(1, 2, 200, a, b, dtype, seed=a + b)


@pytest.mark.parametrize("a,b", [(16, 32), (16, 64), (32, 32), (32, 128), (48, 96), (64, 64), (80, 80),
                                 (80, 32), (76, 48), (96, 32), (96, 96), (128, 32)])
@pytest.mark.parametrize("N", [11, 13, 16, 33, 203])
def test_fp32_rows_at_a_stages_end(a, b, N):
    """Rows that are read as they were copied and rows that are padded, and last stages of one token,
    all and almost all."""
    run(1, 2, N, a, b, "f32", reverse=bool(N % 2), seed=a + N)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype,a,b", [("bf16", 64, 64), ("bf16", 32, 24), ("f32", 32, 40),
                                       ("bf16", 128, 128), ("bf16", 56, 88)])
def test_padding(dtype, a, b, reverse):
    """Lengths of 0, 1, whole chunks, past the end and below 0; what lies in the padding is not
    read, whatever it is, and outputs are zero there."""
    N, lens = 300, [300, 0, 1, 127, 128, 129, 256, 257, 299, 1000, -5]
    B = len(lens)
    m = make(B, 2, N, a, b, dtype)
    want = run(B, 2, N, a, b, dtype, reverse=reverse, lens=lens, data=m)
    bad = {n: (m[n].copy() if m[n] is not None else None) for n in m}
    rng = np.random.default_rng(7)
    for i, n in enumerate(lens):
        for name in ("q", "k", "v", "dout"):
            pad = bad[name][i, :, max(0, n):]
            pad[...] = rng.choice([np.nan, np.inf, -np.inf], pad.shape)
    got = run(B, 2, N, a, b, dtype, reverse=reverse, lens=lens, data=bad)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    for i, n in enumerate(lens):
        for t in (got[0], *got[2:5]):
            assert not t[i, :, max(0, min(n, N)):].any()
        if n <= 0:
            assert np.array_equal(got[1][i].cpu().numpy(), np.float32(m["state"][i]))
            assert np.array_equal(got[5][i].cpu().numpy(), np.float32(m["dfinal"][i]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("logs", [(0.0, 0.5, -1e-6), (-20.0, -100.0, -1e4), (-np.inf, -3e38, -0.17),
                                  (-0.25, -0.1733, -0.1732)])
def test_decays(dtype, logs):
    """None at all, above 0 (counts as none), forgetting everything, and around where the kernel
    that goes token by token changes how it holds the state."""
    run(1, 3, 300, 32, 32, dtype, logs=logs)


@pytest.mark.parametrize("dtype,a,b", [("bf16", 64, 64), ("bf16", 64, 48), ("f32", 32, 32),
                                       ("bf16", 128, 64), ("bf16", 64, 128), ("bf16", 128, 128),
                                       ("f32", 96, 128)])
@pytest.mark.parametrize("B,N", [(1, 3000), (5, 1111)])
def test_segments(dtype, a, b, B, N):
    """Long sequences in several segments, both ways, with lengths that end in each of them."""
    lens = None if B == 1 else [N, 5, 700, 0, 1024]
    for reverse in (False, True):
        run(B, 2, N, a, b, dtype, reverse=reverse, lens=lens, logs=(-1e-3, -0.01))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_states(dtype):
    run(2, 2, 130, 64, 64, dtype, state=False)


@pytest.mark.parametrize("dtype,N", [("f32", 40), ("bf16", 40), ("bf16", 200)])
def test_pointers_off_sixteen_bytes(dtype, N):
    run(1, 2, N, 40, 24, dtype, shift=True)
    run(1, 2, N, 33, 7, dtype, shift=True)


@pytest.mark.parametrize("dtype,a,N", [("f32", 64, 33), ("bf16", 64, 33), ("bf16", 64, 200),
                                       ("bf16", 64, 3000), ("f32", 16, 3000),
                                       ("bf16", 128, 1000)])
def test_states_in_place(dtype, a, N):
    """The final state over the first one, and the first's gradient over the final's."""
    import laplacian_nystr_attention_gb300 as lna
    m = make(1, 2, N, a, a, dtype)
    plan = lna.DecayAttention(lna.make_decay_config(1, 2, N, a, a, in_dtype=dtype, out_dtype=dtype,
                                                    grad_dtype=dtype))
    q, k, v, dout = (dev(m[n], dtype) for n in ("q", "k", "v", "dout"))
    log_decay, s0, df = (dev(m[n]) for n in ("log_decay", "state", "dfinal"))
    final = torch.empty_like(s0)
    out = plan.forward(q, k, v, log_decay, state=s0, final=final)
    want = plan.backward(q, k, v, log_decay, dout, state=s0, dfinal=df)
    held = s0.clone()
    again = plan.forward(q, k, v, log_decay, state=held, final=held)
    over = df.clone()
    got = plan.backward(q, k, v, log_decay, dout, state=s0, dfinal=over, grads={"dstate": over})
    assert torch.equal(out, again) and torch.equal(final, held)
    assert got[3].data_ptr() == over.data_ptr()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_after_token(dtype):
    """A prompt at once and then single tokens, each from the state of the one before, is one
    sequence."""
    import laplacian_nystr_attention_gb300 as lna
    B, H, N, P, d = 2, 3, 140, 130, 64
    m = make(B, H, N, d, d, dtype, state=False)
    q, k, v = (dev(m[n], dtype) for n in "qkv")
    log_decay = dev(m["log_decay"])
    kw = dict(in_dtype=dtype, out_dtype="f32", scale=0.125)
    prompt = lna.DecayAttention(lna.make_decay_config(B, H, P, d, d, **kw))
    step = lna.DecayAttention(lna.make_decay_config(B, H, 1, d, d, **kw))
    state = torch.empty(prompt.state_shape, device="cuda")
    cut = lambda t, i, j: t[:, :, i:j].contiguous()  # noqa: E731
    outs = [prompt.forward(*(cut(t, 0, P) for t in (q, k, v)), log_decay, final=state)]
    for i in range(P, N):
        outs.append(step.forward(*(cut(t, i, i + 1) for t in (q, k, v)), log_decay, state=state,
                                 final=state))
    want = ref.decay(m["q"], m["k"], m["v"], m["log_decay"], 0.125, tensor_cores=True)
    ref.check("out", torch.cat(outs, 2), want["out"])
    ref.check("final", state, want["final"])


@pytest.mark.parametrize("dtype,N", [("bf16", 1), ("bf16", 1500), ("f32", 1500)])
def test_streams_graphs_and_repeats(dtype, N):
    """The same bits from call to call, on another stream and from two replayed graphs at once."""
    import laplacian_nystr_attention_gb300 as lna
    m = make(2, 2, N, 64, 64, dtype)
    plan = lna.DecayAttention(lna.make_decay_config(2, 2, N, 64, 64, in_dtype=dtype,
                                                    out_dtype=dtype, grad_dtype=dtype))
    q, k, v, dout = (dev(m[n], dtype) for n in ("q", "k", "v", "dout"))
    log_decay, s0, df = (dev(m[n]) for n in ("log_decay", "state", "dfinal"))

    def both(stream=None):
        final = torch.empty(plan.state_shape, device="cuda")
        out = plan.forward(q, k, v, log_decay, state=s0, final=final, stream=stream)
        return (out, final, *plan.backward(q, k, v, log_decay, dout, state=s0, dfinal=df,
                                           stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both()
        graphs.append((g, outs))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """The last sequence of tensors of over 2^32 bytes and 2^31 values, on its own and among them."""
    import laplacian_nystr_attention_gb300 as lna
    H, N, d = 2, 1 << 18, 64
    B = 65                                    # B H N d = 2.18e9 values
    last = make(1, H, 512, d, d, "bf16", state=False)
    kw = dict(in_dtype="bf16", out_dtype="bf16", scale=0.125)
    big = lna.DecayAttention(lna.make_decay_config(B, H, N, d, d, **kw))
    log_decay = dev(last["log_decay"])
    rows = {}
    for n in "qkv":
        t = torch.zeros((B, H, N, d), dtype=torch.bfloat16, device="cuda")
        t[-1, :, -512:] = dev(last[n][0], "bf16")
        rows[n] = t
    out = big.forward(rows["q"], rows["k"], rows["v"], log_decay)
    want = ref.decay(last["q"], last["k"], last["v"], last["log_decay"], 0.125, tensor_cores=True)
    ref.check("out", out[-1:, :, -512:], want["out"], "bf16")
    assert not out[-1, :, :-512].any() and not out[:-1].any()


def test_empty_batch():
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.DecayAttention(lna.make_decay_config(0, 2, 5, 8, 8))
    t = torch.empty(0, 2, 5, 8, device="cuda")
    log_decay = torch.zeros(2, device="cuda")
    assert plan.forward(t, t, t, log_decay).shape == (0, 2, 5, 8)
    assert [x.shape[0] for x in plan.backward(t, t, t, log_decay, t)] == [0] * 4


def test_refusals():
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.DecayAttention(lna.make_decay_config(2, 2, 200, 64, 64, in_dtype="bf16",
                                                    out_dtype="bf16", grad_dtype="bf16"))
    t = torch.zeros(2, 2, 200, 64, dtype=torch.bfloat16, device="cuda")
    log_decay = torch.zeros(2, device="cuda")
    plan.forward(t, t, t, log_decay)
    wide = torch.zeros(2, 2, 200, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (t.float(), t[:, :, :199], t.cpu(), wide[..., :64], t.transpose(1, 2).contiguous()
                .transpose(1, 2)):
        with pytest.raises(ValueError):
            plan.forward(bad, t, t, log_decay)
        with pytest.raises(ValueError):
            plan.backward(t, t, t, log_decay, bad)
    for kw in (dict(state=t), dict(lengths=torch.zeros(2, device="cuda")), dict(final=log_decay),
               dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            plan.forward(t, t, t, log_decay, **kw)
    with pytest.raises(ValueError):
        plan.forward(t, t, t, torch.zeros(3, device="cuda"))
    long = lna.DecayAttention(lna.make_decay_config(1, 1, 4096, 64, 64, in_dtype="bf16"))
    assert long.workspace_bytes > 0 and long.workspace_bytes % 256 == 0
    x = torch.zeros(1, 1, 4096, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.empty(1, 1, 4096, 64, device="cuda")
    ws = torch.empty(long.workspace_bytes // 4 + 1, device="cuda")
    args = lambda w, n: (long.handle, x.data_ptr(), x.data_ptr(), x.data_ptr(),  # noqa: E731
                         log_decay.data_ptr(), None, None, o.data_ptr(), None, w, n, None)
    for w, n, status in ((None, long.workspace_bytes, 1), (ws.data_ptr(), long.workspace_bytes - 1, None),
                         (ws.data_ptr() + 4, long.workspace_bytes, None)):
        with pytest.raises(lna.LaplAttnError) as e:
            lna.lapl_decay_forward(*args(w, n))
        assert status is None or e.value.status == status


@pytest.mark.parametrize("backward", [False, True])
def test_wait_that_gives_up_is_told(backward):
    """A chunk that never arrives: the waits for it run out, the call ends, the error is told once,
    and the next call is right."""
    import laplacian_nystr_attention_gb300 as lna
    m = make(1, 2, 300, 64, 64, "bf16")
    plan = lna.DecayAttention(lna.make_decay_config(1, 2, 300, 64, 64, scale=0.125, in_dtype="bf16",
                                                    out_dtype="bf16", grad_dtype="bf16"))
    q, k, v, dout = (dev(m[n], "bf16") for n in ("q", "k", "v", "dout"))
    log_decay = dev(m["log_decay"])
    lna.lapl_decay_set_fault_injection(plan.handle, 20_000_000, 1)
    call = (lambda: plan.backward(q, k, v, log_decay, dout)) if backward else \
        (lambda: plan.forward(q, k, v, log_decay))
    call()
    with pytest.raises(lna.LaplAttnError) as e:
        plan.check_device_errors()
    assert e.value.status == lna._lib.LAPL_ERR_DEVICE_TIMEOUT and "linear attention" in str(e.value)
    plan.check_device_errors()
    lna.lapl_decay_set_fault_injection(plan.handle, 0, 0)
    out = plan.forward(q, k, v, log_decay)
    plan.check_device_errors()
    want = ref.decay(m["q"], m["k"], m["v"], m["log_decay"], 0.125, tensor_cores=True)
    ref.check("out", out, want["out"], "bf16")
