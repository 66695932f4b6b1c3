"""Edges of the AdamW step (lapl_adamw_*): an eps of any size, scalars in the tensors' memory, and what
clipping leaves in the states."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
from operators_reference import U, rounded
from test_gpu_adamw import check_coded, dev, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps,lr,scale", [(1e38, 1e22, 1e15), (3.4e38, 1e24, 1e14), (1e19, 1e4, 1e15), (4e18, 1e4, 1e15),
                                          (1e-37, 1e-3, 1.0)])
def test_an_eps_of_any_size(bits, eps, lr, scale, monkeypatch):
    """An update that eps makes small, and not nothing.

    The reference's bound of w counts roundings of w alone, which is enough where lr wd <= 1.  w (1 - lr wd)
    is formed by a product, a difference and a product, each rounded once: U lr wd |w|, and U (1 + lr wd) |w|
    twice; 4 U lr wd |w| more covers what grows with lr."""
    form = ref.adamw

    def adamw(w, g, m, v, step, lr, betas, eps, wd, clip=1.0):
        (w1, bound), *states = form(w, g, m, v, step, lr, betas, eps, wd, clip)
        return ((w1, bound + 4 * U * lr * wd * np.abs(w)), *states)

    monkeypatch.setattr(ref, "adamw", adamw)
    run([700, 256], ["f32", "f32"], bits=bits, eps=eps, lr=lr, scale=scale)


def test_scalars_in_what_the_step_writes_are_refused():
    """Every CTA reads them when it starts, and by then another may have written there."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.AdamW([8], ["f32"])
    p, g = [torch.ones(8, device="cuda")], [torch.ones(8, device="cuda")]
    s = plan.new_states(p)
    number = torch.ones((), dtype=torch.int64, device="cuda")
    one = torch.ones((), device="cuda")
    call = dict(params=p, grads=g, step=number, lr=one, **s)
    for bad in (dict(lr=p[0][3:4]), dict(norm=s["m"][0][7:], max_norm=1.0), dict(lr=s["v"][0][:1]),
                dict(step=p[0][2:4].view(torch.int64))):
        with pytest.raises(lna.LaplAttnError) as e:
            plan.step(**{**call, **bad})
        assert e.value.status == 1
    # What is only read may be one place, and a gradient.
    plan.step(**{**call, "lr": g[0][:1], "norm": g[0][:1], "max_norm": 1.0})
    assert (p[0] < 1).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kinds,masters", [(["f32", "f32", "f32"], False), (["bf16", "f32", "bf16"], True)])
def test_the_clipping_norm_reaches_states_and_weights(bits, kinds, masters):
    """Two steps with different gradients and norms, against 64 bits with the states that the first one
    left: the first step's weights, from zero states, do not depend on the gradients' scale."""
    import laplacian_nystr_attention_gb300 as lna
    counts, lr, betas, wd, most = [1000, 300, 77], 1e-2, (0.9, 0.95), 0.1, 2.0
    rng = np.random.default_rng(5)
    w = [rounded(rng.standard_normal(n), k) for n, k in zip(counts, kinds)]
    params = [dev(x, k) for x, k in zip(w, kinds)]
    opt = lna.AdamW.like(params, betas=betas, weight_decay=wd, state_bits=bits, masters=masters)
    clip = lna.GradClip.like(params)
    s = opt.new_states(params)
    for step, size in ((1, 3.0), (2, 0.5)):
        g = [rounded(size * rng.standard_normal(n), k) for n, k in zip(counts, kinds)]
        held = []
        for i, n in enumerate(counts):
            m, v = (s[x][i].double().cpu().numpy() for x in "mv")
            if bits == 8:
                m, v = (x * np.repeat(s[y][i].double().cpu().numpy(), ref.BLOCK)[:n]
                        for x, y in ((m, "m_scales"), (v, "v_scales")))
                v = v * v
            master = masters and kinds[i] == "bf16"
            held.append(((s["masters"] if master else params)[i].double().cpu().numpy(), m, v))
        grads = [dev(x, k) for x, k in zip(g, kinds)]
        norm = clip.norm(grads)
        opt.step(params, grads, step=step, lr=lr, norm=norm, max_norm=most, **s)
        size = np.sqrt(sum((x * x).sum() for x in g))
        assert abs(float(norm) - size) <= 4 * U * size and size > 2 * most
        for i, (w0, m0, v0) in enumerate(held):
            # (The norm and the factor are off by 8 U, as every g is then, and v by 16.)
            (w1, eb), (m1, mb), (v1, vb) = ref.adamw(w0, g[i], m0, v0, step, float(np.float32(lr)), betas,
                                                     float(np.float32(1e-8)), float(np.float32(wd)), most / size)
            late = np.abs(m1 - betas[0] * m0)
            mb, vb = mb + 8 * U * late, vb + 16 * U * v1
            down = np.sqrt(v1 / (1 - betas[1] ** step)) + 1e-8
            eb = eb + 16 * U * lr * (np.abs(betas[0] * m0) + late) / (1 - betas[0] ** step) / down
            if bits == 32:
                ref.check("m", s["m"][i], (m1, mb))
                ref.check("v", s["v"][i], (v1, vb))
            else:
                check_coded("m", s["m"][i], s["m_scales"][i], m1, mb, False)
                check_coded("v", s["v"][i], s["v_scales"][i], np.sqrt(v1), 16 * U * np.sqrt(v1), True)
            master = masters and kinds[i] == "bf16"
            ref.check("w", (s["masters"] if master else params)[i], (w1, eb),
                      "f32" if master or kinds[i] == "f32" else "bf16")
