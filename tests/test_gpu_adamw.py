"""GPU parity of the AdamW step (lapl_adamw_*) against its 64-bit reference, every value within the
bound of the roundings on its way (more_operators_reference.py)."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
from operators_reference import HALF, U, rounded

pytestmark = pytest.mark.gpu

TYPES = ref.TYPES


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype]).cuda()


def place(t, shift):
    room = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    got = room[shift:].view(t.shape)
    got.copy_(t)
    return got


def run(counts, kinds, grad_kinds=None, bits=32, masters=False, step=7, lr=1e-3, betas=(0.9, 0.99),
        eps=1e-8, wd=0.1, norm=None, max_norm=None, shift=0, seed=0, on_device=False, scale=1.0):
    """One step from states that steps have left, checked."""
    import laplacian_nystr_attention_gb300 as lna
    rng = np.random.default_rng(seed)
    grad_kinds = grad_kinds or kinds
    wds = wd if isinstance(wd, list) else [wd] * len(counts)
    plan = lna.AdamW(counts, kinds, grad_kinds, betas=betas, eps=eps, weight_decay=wd,
                     state_bits=bits, masters=masters)
    data = []
    for n, k, gk in zip(counts, kinds, grad_kinds):
        w = rounded(rng.standard_normal(n), "f32")
        data.append(dict(w=w if masters else rounded(w, k), g=scale * rounded(rng.standard_normal(n), gk),
                         m=rounded(0.1 * scale * rng.standard_normal(n), "f32"),
                         v=rounded((scale * rng.standard_normal(n)) ** 2, "f32")))
    params = [place(dev(d["w"], k), shift) for d, k in zip(data, kinds)]
    grads = [place(dev(d["g"], k), shift) for d, k in zip(data, grad_kinds)]
    kw = {}
    if masters:
        kw["masters"] = [place(dev(d["w"]), shift) if k == "bf16" else None
                         for d, k in zip(data, kinds)]
    if bits == 8:
        kw["m_scales"], kw["v_scales"], m, v = [], [], [], []
        for d in data:
            for name, codes, scales, root in (("m", m, kw["m_scales"], False),
                                              ("v", v, kw["v_scales"], True)):
                q, s = ref.coded(np.sqrt(d[name]) if root else d[name], root)
                q = torch.from_numpy(q).float().to(torch.float8_e4m3fn).cuda()
                s = dev(s)
                codes.append(place(q, shift))
                scales.append(s)
                # As it is held.
                back = q.double().cpu().numpy() * np.repeat(s.double().cpu().numpy(),
                                                            ref.BLOCK)[:q.numel()]
                d[name] = back ** 2 if root else back
    else:
        m, v = ([place(dev(d[x]), shift) for d in data] for x in "mv")
    if norm is not None:
        kw.update(norm=torch.tensor(norm, device="cuda", dtype=torch.float32), max_norm=max_norm)
    at = (torch.tensor(step, device="cuda"), torch.tensor(lr, device="cuda")) if on_device else \
        (step, lr)
    plan.step(params, grads, m, v, *at, **kw)
    clip = 1.0
    if norm is not None and norm > max_norm:
        clip = float(np.float32(max_norm)) / float(np.float32(norm))
    lr32 = float(np.float32(lr))
    for i, d in enumerate(data):
        want_w, want_m, want_v = ref.adamw(d["w"], d["g"], d["m"], d["v"], step, lr32, betas,
                                           float(np.float32(eps)), float(np.float32(wds[i])), clip)
        held = kw["masters"][i] if masters and kinds[i] == "bf16" else params[i]
        ref.check("w", held, want_w, "f32" if held.dtype == torch.float32 else "bf16")
        if masters and kinds[i] == "bf16":
            assert torch.equal(params[i], held.bfloat16())
        if bits == 32:
            ref.check("m", m[i], want_m)
            ref.check("v", v[i], want_v)
        else:
            check_coded("m", m[i], kw["m_scales"][i], *want_m, False)
            root = np.sqrt(want_v[0])
            check_coded("v", v[i], kw["v_scales"][i], root, 8 * U * root, True)
    return params, m, v, kw


def check_coded(name, codes, scales, value, bound, root):
    """A code is off by half of its step, 2^-4 of it or 2^-10 at least, and by what its value and
    scale are off; codes of roots below 2^-9 are 2^-9."""
    q, s = ref.coded(value, root)
    s_got = scales.double().cpu().numpy()
    top = np.pad(bound, (0, -value.size % ref.BLOCK)).reshape(-1, ref.BLOCK).max(-1) / ref.F8_MAX
    assert (np.abs(s_got - s) <= top + 4 * U * s).all(), name
    got = codes.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.repeat((top + 4 * U * s) / s, ref.BLOCK)[:q.size] * np.abs(q) \
        + bound / np.repeat(s, ref.BLOCK)[:q.size]
    tol = HALF["f8"] * np.abs(q) + 2.0 ** -10 + 2 * off
    assert (np.abs(got - q) <= tol).all(), name
    if root:
        assert ((got > 0) | (value == 0)).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind,grad,masters", [("f32", "f32", False), ("bf16", "bf16", False),
                                               ("bf16", "bf16", True), ("bf16", "f32", True),
                                               ("f32", "bf16", False)])
def test_types(bits, kind, grad, masters):
    run([1, 255, 256, 257, 5000, 0, 40000], [kind] * 7, [grad] * 7, bits, masters)


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_tensors(bits):
    kinds = ["f32", "bf16", "f32", "bf16", "bf16"]
    run([3, 1000, 4097, 1, 256 * 9], kinds, bits=bits, masters=True,
        wd=[0.0, 0.1, 0.3, 0.0, 0.01])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3, 4])
def test_pointers_off_sixteen_bytes(bits, shift):
    run([300, 1025, 7], ["f32", "bf16", "bf16"], bits=bits, shift=shift)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("T", [65, 401, 900])
def test_many_tensors(bits, T):
    rng = np.random.default_rng(T)
    run([int(n) for n in rng.integers(0, 700, T)], ["f32" if i % 2 else "bf16" for i in range(T)],
        bits=bits)


@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 7])
def test_steps(step, on_device):
    run([700], ["f32"], step=step, betas=(0.9, 0.999), on_device=on_device)


@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.0, 0.999), (0.95, 0.9999)])
@pytest.mark.parametrize("bits", [32, 8])
def test_betas(betas, bits):
    run([700], ["f32"], betas=betas, bits=bits, step=3)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("norm,max_norm", [(5.0, 1.0), (0.5, 1.0), (3.0, 0.0), (1e-3, 1e-4)])
def test_clipping(bits, norm, max_norm):
    run([700, 300], ["f32", "bf16"], bits=bits, norm=norm, max_norm=max_norm)


@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_small_and_large_gradients(scale):
    run([700], ["f32"], scale=scale, eps=1e-20)
    run([700], ["f32"], bits=8, scale=scale, eps=1e-20)


@pytest.mark.parametrize("bits", [32, 8])
def test_states_are_rounded_one_by_one(bits):
    """Every product and sum of the states rounded to fp32, bit for bit, and the codes of what that
    gives: nothing is contracted."""
    import laplacian_nystr_attention_gb300 as lna
    n, f = 256 * 400, np.float32
    rng = np.random.default_rng(9)
    g, m, v = (rng.standard_normal(n).astype(f) for _ in range(3))
    v = v * v
    norm, most = f(7.0), f(3.0)
    plan = lna.AdamW([n], ["f32"], betas=(0.9, 0.95), state_bits=bits)
    s = {k: [torch.from_numpy(a.copy()).cuda()] for k, a in (("m", m), ("v", v))}
    if bits == 8:
        s = {}
        for k, a in (("m", m), ("v", np.sqrt(v))):
            scale = np.abs(a).reshape(-1, 256).max(1) * f(1 / 448)
            q = torch.from_numpy(a / scale.repeat(256)).to(torch.float8_e4m3fn)
            held = q.float().numpy() * scale.repeat(256)
            s[k], s[k + "_scales"] = [q.cuda()], [torch.from_numpy(scale).cuda()]
            if k == "m":
                m = held
            else:
                v = held * held
    plan.step([torch.zeros(n, device="cuda")], [torch.from_numpy(g).cuda()], step=3, lr=0.1,
              norm=torch.tensor(norm, device="cuda"), max_norm=float(most), **s)
    g = g * (most * (f(1) / norm))
    m = f(0.9) * m + f(1 - 0.9) * g
    v = f(0.95) * v + f(1 - 0.95) * g * g
    if bits == 32:
        assert np.array_equal(s["m"][0].cpu().numpy(), m) and np.array_equal(s["v"][0].cpu().numpy(), v)
        return
    for k, a in (("m", m), ("v", np.sqrt(v))):
        scale = np.abs(a).reshape(-1, 256).max(1) * f(1 / 448)
        assert np.array_equal(s[k + "_scales"][0].cpu().numpy(), scale)
        q = a / scale.repeat(256)
        if k == "v":
            q = np.where(a > 0, np.maximum(q, f(2.0 ** -9)), q)
        want = torch.from_numpy(q).to(torch.float8_e4m3fn)
        assert torch.equal(s[k][0].cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("norm", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_changes_nothing(bits, norm):
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.AdamW([700], ["bf16"], state_bits=bits, masters=True)
    p, g = [torch.randn(700, device="cuda").bfloat16()], [torch.randn(700, device="cuda").bfloat16()]
    s = plan.new_states(p)
    plan.step(p, g, step=1, lr=0.1, **s)
    held = [t.clone() for t in (*p, *(t for x in s.values() for t in x))]
    plan.step(p, g, step=2, lr=0.1, norm=torch.tensor(norm, device="cuda"), max_norm=1.0, **s)
    for a, b in zip(held, (*p, *(t for x in s.values() for t in x))):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_from_the_start_over_steps(bits):
    """Ten steps from zeros, against 64 bits with the same states held in 32; in 8 bits each step's
    states are rounded as the library holds them."""
    import laplacian_nystr_attention_gb300 as lna
    n, lr, betas = 1500, 1e-2, (0.9, 0.99)
    rng = np.random.default_rng(2)
    w = rounded(rng.standard_normal(n), "f32")
    plan = lna.AdamW.like([dev(w)], betas=betas, state_bits=bits, weight_decay=0.1)
    p = [dev(w)]
    s = plan.new_states(p)
    for t in range(1, 11):
        g = rounded(rng.standard_normal(n), "f32")
        m, v = (x[0].double().cpu().numpy() for x in (s["m"], s["v"]))
        if bits == 8:
            m, v = (x * np.repeat(s[k][0].double().cpu().numpy(), 256)[:n]
                    for x, k in ((m, "m_scales"), (v, "v_scales")))
            v = v * v
        before = p[0].double().cpu().numpy()
        plan.step(p, [dev(g)], step=t, lr=lr, **s)
        want = ref.adamw(before, g, m, v, t, float(np.float32(lr)), betas, float(np.float32(1e-8)),
                         float(np.float32(0.1)))
        ref.check("w", p[0], want[0])


def test_nan_and_zeros():
    """A NaN stays in its value with 32-bit states, and in its block with 8-bit ones; zero gradients
    from zero states change nothing but the decay."""
    import laplacian_nystr_attention_gb300 as lna
    for bits, spoilt in ((32, slice(300, 301)), (8, slice(256, 512))):
        plan = lna.AdamW([1000], ["f32"], state_bits=bits, weight_decay=0.0)
        p, g = [torch.ones(1000, device="cuda")], [torch.zeros(1000, device="cuda")]
        s = plan.new_states(p)
        plan.step(p, g, step=1, lr=0.1, **s)
        assert (p[0] == 1).all() and not s["m"][0].float().any() and not s["v"][0].float().any()
        g[0][300] = float("nan")
        for t in (2, 3):
            plan.step(p, g, step=t, lr=0.1, **s)
            g[0][300] = 0.0
        bad = torch.zeros(1000, dtype=torch.bool, device="cuda")
        bad[spoilt] = True
        assert torch.isnan(p[0][bad]).all() and (p[0][~bad] == 1).all()


def test_streams_graphs_and_repeats():
    """A captured step whose number and rate are on the device, replayed, is the same as steps one by
    one on another stream."""
    import laplacian_nystr_attention_gb300 as lna
    counts, kinds = [5000, 33, 70000], ["bf16", "f32", "bf16"]
    plan = lna.AdamW(counts, kinds, state_bits=8, masters=True)
    gen = torch.Generator(device="cuda").manual_seed(0)
    new = lambda n, k: torch.randn(n, generator=gen, device="cuda").to(TYPES[k])  # noqa: E731
    p0, g = [new(n, k) for n, k in zip(counts, kinds)], [new(n, k) for n, k in zip(counts, kinds)]
    norm = torch.tensor(300.0, device="cuda")
    got = []
    for captured in (False, True):
        p = [t.clone() for t in p0]
        s = plan.new_states(p)
        number, lr = torch.zeros((), dtype=torch.int64, device="cuda"), torch.full((), 1e-2,
                                                                                   device="cuda")
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                number += 1
                plan.step(p, g, step=number, lr=lr, norm=norm, max_norm=1.0, **s)
            number.zero_()
            for t, x in zip(p, p0):
                t.copy_(x)
            fresh = plan.new_states(p)
            for name in s:
                for t, x in zip(s[name], fresh[name]):
                    if t is not None:
                        t.view(torch.uint8).copy_(x.view(torch.uint8))
            for _ in range(3):
                graph.replay()
        else:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            for _ in range(3):
                with torch.cuda.stream(side):
                    number += 1
                plan.step(p, g, step=number, lr=lr, norm=norm, max_norm=1.0, stream=side, **s)
            side.synchronize()
        torch.cuda.synchronize()
        got.append([*p, *(t for x in s.values() for t in x if t is not None)])
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_offsets_past_32_bits():
    """The last values of a tensor of over 2^32 values."""
    import laplacian_nystr_attention_gb300 as lna
    n = (1 << 32) + 777
    plan = lna.AdamW([n], ["bf16"], state_bits=8, weight_decay=0.0)
    p, g = [torch.zeros(n, dtype=torch.bfloat16, device="cuda")], \
        [torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
    s = plan.new_states(p)
    g[0][-600:] = 1.0
    plan.step(p, g, step=1, lr=0.5, **s)
    assert (p[0][-600:] == -0.5).all() and not p[0][-1400:-600].any() and not p[0][:1 << 20].any()
    assert not p[0][600:2000].any()


def test_refusals():
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.AdamW([8, 4], ["f32", "bf16"], masters=True)
    p = [torch.zeros(8, device="cuda"), torch.zeros(4, dtype=torch.bfloat16, device="cuda")]
    g = [torch.zeros_like(t) for t in p]
    s = plan.new_states(p)
    plan.step(p, g, step=1, lr=0.1, **s)
    one = torch.ones((), device="cuda")
    for bad in (dict(params=p[:1]), dict(grads=[g[0].bfloat16(), g[1]]), dict(m=[p[0]]),
                dict(masters=None), dict(masters=[p[0], p[0]]), dict(masters=[None, None]),
                dict(norm=one), dict(max_norm=1.0), dict(norm=one, max_norm=-1.0),
                dict(norm=one, max_norm=float("nan")), dict(m_scales=[one, one]),
                dict(params=[torch.zeros(8, 2, device="cuda")[:, 0], p[1]]),
                dict(step=torch.ones((), device="cuda")), dict(grads=[g[0].cpu(), g[1]])):
        with pytest.raises(ValueError):
            plan.step(**{**dict(params=p, grads=g, step=1, lr=0.1, **s), **bad})
    for bad in (dict(step=0), dict(lr=float("nan")), dict(grads=p), dict(v=s["m"])):
        with pytest.raises(lna.LaplAttnError) as e:
            plan.step(**{**dict(params=p, grads=g, step=1, lr=0.1, **s), **bad})
        assert e.value.status == 1
    # Gradients may share memory, and so may what only lies side by side.
    same = lna.AdamW([4, 4], ["f32", "f32"])
    room = torch.zeros(8, device="cuda")
    both = [room[:4], room[4:]]
    t = torch.ones(4, device="cuda")
    same.step(both, [t, t], step=1, lr=0.1, **same.new_states(both))
    eight = lna.AdamW([8], ["f32"], state_bits=8)
    with pytest.raises(ValueError):
        eight.step([p[0]], [g[0]], [s["m"][0]], [s["v"][0]], 1, 0.1)
