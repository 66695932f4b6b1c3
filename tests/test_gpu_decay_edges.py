"""Edges of the linear attention with decays (lapl_decay_*): what each type keeps, decays that are no
numbers, waits that give up in each launch, workspaces."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
from operators_reference import U
from test_gpu_decay import dev, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


@pytest.mark.parametrize("a,b", [(64, 64), (32, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("reverse", [False, True])
def test_fp32_outputs_of_bf16_rows_keep_fp32s_precision(a, b, reverse):
    """On the tensor cores too: root mean square, over every sequence's outputs.  A sum of up to 24
    products in tensor memory is cut off at each by up to 2 U of what it is by then, U on average: 24 U if
    it were as large from the start on.  (What is computed in two bf16 parts leaves out up to 2^-16 = 256 U
    of each term, some 40 U on average.)"""
    import laplacian_nystr_attention_gb300 as lna
    B, H, N = 2, 4, 700
    m = make(B, H, N, a, b, "bf16", seed=a + b, logs=(-1e-3, -0.01, -0.05, -0.3))
    plan = lna.DecayAttention(lna.make_decay_config(B, H, N, a, b, scale=0.125, reverse=int(reverse),
                                                    in_dtype="bf16", out_dtype="f32"))
    assert lna.lapl_decay_plan_info_get(plan.handle)["tensor_cores"]
    q, k, v = (dev(m[n], "bf16") for n in "qkv")
    final = torch.empty(plan.state_shape, device="cuda")
    out = plan.forward(q, k, v, dev(m["log_decay"]), state=dev(m["state"]), final=final)
    plan.check_device_errors()
    want = ref.decay(m["q"], m["k"], m["v"], m["log_decay"], 0.125, m["state"], None, reverse)
    for got, (value, _) in ((out, want["out"]), (final, want["final"])):
        off = got.double().cpu().numpy() - value
        rms = np.sqrt((off ** 2).sum((-1, -2)) / (value ** 2).sum((-1, -2)))
        assert rms.max() <= 24 * U, rms / U


@pytest.mark.parametrize("dtype,d,N", [("f32", 32, 1), ("f32", 32, 40), ("f32", 32, 3000), ("bf16", 64, 1),
                                       ("bf16", 64, 300), ("bf16", 64, 3000), ("bf16", 128, 300)])
@pytest.mark.parametrize("reverse", [False, True])
def test_a_decay_that_is_no_number(dtype, d, N, reverse):
    """It shows in all that it is part of, and in no other head and no sequence without tokens."""
    import laplacian_nystr_attention_gb300 as lna
    lens = [N, 0, max(1, N // 2)]
    m = make(3, 2, N, d, d, dtype, seed=N)
    plan = lna.DecayAttention(lna.make_decay_config(3, 2, N, d, d, scale=0.125, reverse=int(reverse),
                                                    in_dtype=dtype, out_dtype=dtype, grad_dtype=dtype))
    q, k, v, dout = (dev(m[n], dtype) for n in ("q", "k", "v", "dout"))
    s0, df = dev(m["state"]), dev(m["dfinal"])
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = []
    for bad in (-0.05, float("nan")):
        log_decay = torch.tensor([bad, -0.01], device="cuda")
        final = torch.empty(plan.state_shape, device="cuda")
        out = plan.forward(q, k, v, log_decay, state=s0, lengths=lengths, final=final)
        got.append((out, final, *plan.backward(q, k, v, log_decay, dout, state=s0, dfinal=df,
                                               lengths=lengths)))
        plan.check_device_errors()
    for x, y in zip(*got):
        assert torch.equal(x[:, 1], y[:, 1]) and not torch.isnan(x).any()
    out, final, dq, dk, dv, dstate = got[1]
    assert torch.equal(final[1], s0[1]) and torch.equal(dstate[1], df[1])
    for b, n in ((0, lens[0]), (2, lens[2])):
        assert torch.isnan(out[b, 0, :n]).all() and torch.isnan(dq[b, 0, :n]).all()
        assert torch.isnan(final[b, 0]).all() and torch.isnan(dstate[b, 0]).all()
        # The last token that is processed meets the final state's gradient undecayed.
        decayed = slice(1, n) if reverse else slice(0, n - 1)
        assert torch.isnan(dk[b, 0, decayed]).all() and torch.isnan(dv[b, 0, decayed]).all()
        for t in (out, dq, dk, dv):
            assert not t[b, :, n:].any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
def test_waits_that_give_up_in_a_call_of_three_launches(d, backward):
    """Segments whose last chunk never arrives, in the launch of their sums and in that of the outputs:
    each ends, the error is told once, and the next call is right."""
    import laplacian_nystr_attention_gb300 as lna
    H, N = 2, 3000
    m = make(1, H, N, d, d, "bf16", logs=(-1e-3, -0.05))
    plan = lna.DecayAttention(lna.make_decay_config(1, H, N, d, d, scale=0.125, in_dtype="bf16",
                                                    out_dtype="bf16", grad_dtype="bf16"))
    info = lna.lapl_decay_plan_info_get(plan.handle)
    kind = "backward_" if backward else ""
    assert info[kind + "tensor_cores"] and info[kind + "segments"] > 1, info
    q, k, v, dout = (dev(m[n], "bf16") for n in ("q", "k", "v", "dout"))
    log_decay = dev(m["log_decay"])
    call = (lambda: plan.backward(q, k, v, log_decay, dout)) if backward else \
        (lambda: (plan.forward(q, k, v, log_decay),))
    want = call()
    plan.check_device_errors()
    lna.lapl_decay_set_fault_injection(plan.handle, 5_000_000, 1)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    call()
    end.record()
    with pytest.raises(lna.LaplAttnError) as e:
        plan.check_device_errors()
    assert e.value.status == lna._lib.LAPL_ERR_DEVICE_TIMEOUT and "linear attention" in str(e.value)
    # Both launches waited.
    assert start.elapsed_time(end) >= 2 * 5.0
    plan.check_device_errors()
    lna.lapl_decay_set_fault_injection(plan.handle, 0, 0)
    got = call()
    plan.check_device_errors()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
@pytest.mark.parametrize("reverse", [False, True])
def test_long_sequences_off_sixteen_bytes(dtype, d, reverse):
    """By the rows' kernel in as many segments as the plan's workspace has room for."""
    run(1, 2, 3000, d, d, dtype, reverse=reverse, shift=True, logs=(-1e-3, -0.05))
    run(3, 2, 700, d, d, dtype, reverse=reverse, shift=True, lens=[700, 0, 333], logs=(-1e-3, -0.05))


def test_no_segment_is_empty():
    import laplacian_nystr_attention_gb300 as lna
    for B, N, d, dtype in ((16, 3136, 32, "f32"), (15, 2047, 48, "f32"), (8, 512, 128, "f32"), (3, 999, 64, "bf16"),
                           (32, 16384, 64, "bf16"), (2, 8192, 128, "bf16"), (1, 129, 64, "bf16"),
                           (1, 17, 8, "f32")):
        plan = lna.DecayAttention(lna.make_decay_config(B, 1, N, d, d, in_dtype=dtype, out_dtype=dtype,
                                                        grad_dtype=dtype))
        info = lna.lapl_decay_plan_info_get(plan.handle)
        for kind in ("", "backward_"):
            step, n = 128 if info[kind + "tensor_cores"] else 16, info[kind + "segments"]
            each = -(-(-(-N // n)) // step) * step
            assert -(-N // each) == n, info


@pytest.mark.parametrize("B,H,N,d,forward,backward", [(8, 32, 4096, 128, 0, 100e6), (2, 8, 8192, 128, 34e6, 34e6),
                                                      (512, 1, 128, 128, 0, 34e6)])
def test_workspaces_are_no_larger_than_a_tensor_of_the_call(B, H, N, d, forward, backward):
    """Nor than the states of all sequences, where those weigh more."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.DecayAttention(lna.make_decay_config(B, H, N, d, d, in_dtype="bf16", out_dtype="bf16",
                                                    grad_dtype="bf16"))
    assert plan.workspace_bytes <= forward and plan.backward_workspace_bytes <= backward


@pytest.mark.parametrize("dtype,d,N", [("f32", 48, 5), ("bf16", 64, 100), ("bf16", 64, 3000)])
def test_states_in_place_while_captured(dtype, d, N):
    """The first state's gradient over the final's, replayed: each time from what the place then holds."""
    import laplacian_nystr_attention_gb300 as lna
    m = make(2, 2, N, d, d, dtype)
    plan = lna.DecayAttention(lna.make_decay_config(2, 2, N, d, d, in_dtype=dtype, out_dtype=dtype,
                                                    grad_dtype=dtype))
    q, k, v, dout = (dev(m[n], dtype) for n in ("q", "k", "v", "dout"))
    log_decay, s0, df = (dev(m[n]) for n in ("log_decay", "state", "dfinal"))
    want = plan.backward(q, k, v, log_decay, dout, state=s0, dfinal=df)
    over = df.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = plan.backward(q, k, v, log_decay, dout, state=s0, dfinal=over, grads={"dstate": over})
    for _ in range(2):
        over.copy_(df)
        graph.replay()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("a,b", [(64, 64), (128, 128), (40, 104)])
@pytest.mark.parametrize("reverse", [False, True])
def test_fp32_outputs_of_bf16_rows_in_segments_and_padding(a, b, reverse):
    run(1, 2, 3000, a, b, "bf16", out="f32", reverse=reverse, backward=False, tc=True, logs=(-1e-3, -0.05))
    run(7, 2, 400, a, b, "bf16", out="f32", reverse=reverse, backward=False, tc=True,
        lens=[400, 0, 1, 127, 128, 129, 385], logs=(-0.2, -0.01))


@pytest.mark.parametrize("N", [300, 3000])
def test_waits_that_give_up_with_fp32_outputs(N):
    import laplacian_nystr_attention_gb300 as lna
    m = make(1, 2, N, 64, 64, "bf16", logs=(-1e-3, -0.05))
    plan = lna.DecayAttention(lna.make_decay_config(1, 2, N, 64, 64, in_dtype="bf16", out_dtype="f32"))
    assert lna.lapl_decay_plan_info_get(plan.handle)["tensor_cores"]
    q, k, v = (dev(m[n], "bf16") for n in "qkv")
    log_decay = dev(m["log_decay"])
    want = plan.forward(q, k, v, log_decay)
    lna.lapl_decay_set_fault_injection(plan.handle, 5_000_000, 1)
    plan.forward(q, k, v, log_decay)
    with pytest.raises(lna.LaplAttnError) as e:
        plan.check_device_errors()
    assert e.value.status == lna._lib.LAPL_ERR_DEVICE_TIMEOUT
    lna.lapl_decay_set_fault_injection(plan.handle, 0, 0)
    assert torch.equal(plan.forward(q, k, v, log_decay), want)
    plan.check_device_errors()
