"""The gated linear recurrence where its kernels can go wrong: waits that give up in the middle of a
sequence, gates at both ends of their range, states that are not finite."""
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
