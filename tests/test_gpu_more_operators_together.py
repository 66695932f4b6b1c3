"""The operators as they are used together: a projection's rows to heads with a norm and rotary positions,
linear attention with decays, residual + norm, and back; the gradients' norm, and the AdamW step that
clips by it.  Then the same block token by token.  Against the 64-bit references."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
import operators_reference as first

pytestmark = pytest.mark.gpu

B, H, N, D, GRID = 2, 2, 144, 64, 12
W = H * D
EPS = float(np.float32(1e-6))
PAIRS, FREQ = (16, 16), [100.0 ** (-i / 16) for i in range(16)] * 2
LOGS = np.float32([-0.02, -0.002]).astype(np.float64)
SCALE = 0.125


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def rel(got, want):
    """Largest difference over the largest value."""
    got = got.double().cpu().numpy()
    return np.abs(got - want).max() / np.abs(want).max()


def inputs():
    rng = np.random.default_rng(8)
    new = lambda *s: first.rounded(rng.standard_normal(s), "f32")  # noqa: E731
    return dict(rows=new(B, N, 3 * W), res=new(B, N, W), dy=new(B, N, W), qw=1 + 0.1 * new(D),
                kw=1 + 0.1 * new(D), w=1 + 0.1 * new(W), state=new(B, H, D, D),
                pos=np.stack([np.arange(N) // GRID, np.arange(N) % GRID], -1)[None].repeat(B, 0))


def reference(m):
    """Values and gradients in 64 bits."""
    q, k, v = (m["rows"][..., i * W:(i + 1) * W] for i in range(3))
    turn = lambda x, w: ref.rope(x, H, m["pos"], PAIRS, FREQ, w, EPS)[0]  # noqa: E731
    qh, kh = turn(q, m["qw"]), turn(k, m["kw"])
    vh = v.reshape(B, N, H, D).transpose(0, 2, 1, 3)
    o = ref.decay(qh, kh, vh, LOGS, SCALE, m["state"])
    n = first.norm(o["out"][0], m["res"], m["w"], EPS)
    nb = first.norm_backward(n["sum"][0], n["rstd"][0], m["w"], m["dy"], None, H)
    a = ref.decay(qh, kh, vh, LOGS, SCALE, m["state"], dout=nb["dx"][0])
    back = lambda x, g, w: ref.rope_backward(x, H, m["pos"], PAIRS, FREQ, g, w, EPS)  # noqa: E731
    (dq, _), (dqw, _) = back(q, a["dq"][0], m["qw"])
    (dk, _), (dkw, _) = back(k, a["dk"][0], m["kw"])
    dv = a["dv"][0].transpose(0, 2, 1, 3).reshape(B, N, W)
    return n["y"][0], o["final"][0], dict(rows=np.concatenate([dq, dk, dv], -1), res=nb["dres"][0],
                                          qw=dqw, kw=dkw, w=nb["dweight"][0], state=a["dstate"][0])


def plans(lna, tokens, **kw):
    return (lna.HeadRotary(lna.make_rope_config(B, tokens, H, H, H, D, PAIRS, FREQ, eps=EPS, q_stride=3 * W,
                                                k_stride=3 * W, v_stride=3 * W, **kw)),
            lna.DecayAttention(lna.make_decay_config(B, H, tokens, D, D, scale=SCALE, **kw)),
            lna.ResidualNorm(lna.make_norm_config(B, H, tokens, D, eps=EPS)))


def parts(rows):
    return [rows[..., i * W:(i + 1) * W] for i in range(3)]


def test_training_step():
    """Tolerance 1e-5 of the largest value: each operator's own bound is within 2e-6 of its largest
    values here, and seven of them follow one another.  (Weights: the step moves each by lr times a
    number of size 1, whose sign a gradient next to zero decides: compared where it is not.)"""
    import laplacian_nystr_attention_gb300 as lna
    m = inputs()
    y, final, grads = reference(m)
    heads, mix, norm = plans(lna, N)
    t = {n: dev(m[n]) for n in ("rows", "res", "dy", "qw", "kw", "w", "state")}
    pos, logs = torch.from_numpy(m["pos"]).int().cuda(), dev(LOGS)
    q, k, v = heads.forward(*parts(t["rows"]), pos, t["qw"], t["kw"])
    end = torch.empty_like(t["state"])
    o = mix.forward(q, k, v, logs, state=t["state"], final=end)
    total, rstd = torch.empty_like(t["res"]), torch.empty(B, N, device="cuda")
    got = norm.forward(o, t["w"], residual=t["res"], sum=total, rstd=rstd)
    assert rel(got, y) < 1e-5 and rel(end, final) < 1e-5

    dout, dres, dw = norm.backward(total, rstd, t["w"], t["dy"])
    dq, dk, dv, dstate = mix.backward(q, k, v, logs, dout, state=t["state"])
    drows = torch.empty_like(t["rows"])
    _, _, _, dqw, dkw = heads.backward(*parts(t["rows"])[:2], pos, t["qw"], t["kw"], dq, dk, dv,
                                       grads=dict(zip(("dq", "dk", "dv"), parts(drows))))
    mix.check_device_errors()
    made = dict(rows=drows, res=dres, qw=dqw, kw=dkw, w=dw, state=dstate)
    for name, want in grads.items():
        assert rel(made[name], want) < 1e-5, name

    names = ("qw", "kw", "w")
    params, g = [t[n] for n in names], [made[n] for n in names]
    size = lna.GradClip.like(g).norm(g)
    length = np.sqrt(sum((grads[n] ** 2).sum() for n in names))
    assert abs(float(size) / length - 1) < 1e-5
    for bits in (32, 8):
        opt = lna.AdamW.like(params, g, state_bits=bits, weight_decay=0.1)
        moved = [p.clone() for p in params]
        s = opt.new_states(moved)
        opt.step(moved, g, step=1, lr=1e-2, norm=size, max_norm=0.5 * length, **s)
        for n, p in zip(names, moved):
            clear = np.abs(grads[n]) > 1e-3 * np.abs(grads[n]).max()
            want, _, _ = ref.adamw(m[n], grads[n], 0 * m[n], 0 * m[n], 1, 1e-2, (0.9, 0.999), 1e-8, 0.1,
                                   0.5)
            assert np.abs(p.double().cpu().numpy() - want[0])[clear].max() < 1e-5 * 1e-2 / 1e-3, n


def test_token_by_token():
    """Prompt and single tokens give what the whole sequence gives."""
    import laplacian_nystr_attention_gb300 as lna
    m = inputs()
    y, final, _ = reference(m)
    t = {n: dev(m[n]) for n in ("rows", "res", "qw", "kw", "w", "state")}
    pos, logs = torch.from_numpy(m["pos"]).int().cuda(), dev(LOGS)
    state, P, outs = t["state"].clone(), N - 5, []
    for at, count in [(0, P)] + [(i, 1) for i in range(P, N)]:
        if count in (P, 1) and (at == 0 or at == P):
            heads, mix, norm = plans(lna, count)
        rows = t["rows"][:, at:at + count].contiguous()
        q, k, v = heads.forward(*parts(rows), pos[:, at:at + count].contiguous(), t["qw"], t["kw"])
        o = mix.forward(q, k, v, logs, state=state, final=state)
        outs.append(norm.forward(o, t["w"], residual=t["res"][:, at:at + count].contiguous()))
    assert rel(torch.cat(outs, 1), y) < 1e-5 and rel(state, final) < 1e-5
