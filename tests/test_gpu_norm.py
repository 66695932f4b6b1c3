"""GPU parity of the residual addition + RMS norm (lapl_norm_*) against its 64-bit reference, every
value within the bound of the roundings on its way (operators_reference.py)."""
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


def dev(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype]).cuda()


def make(B, H, N, d, x="f32", res="f32", grad="f32", seed=0):
    rng = np.random.default_rng(seed)
    W = H * d
    return dict(x=ref.rounded(rng.standard_normal((B, H, N, d)), x),
                res=ref.rounded(rng.standard_normal((B, N, W)), res),
                weight=ref.rounded(1 + 0.3 * rng.standard_normal(W), "f32"),
                dy=ref.rounded(rng.standard_normal((B, N, W)), grad),
                dsum=ref.rounded(rng.standard_normal((B, N, W)), grad))


def off_by_one(t):
    """The same values one element off an allocation's start."""
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    got = room[1:].view(t.shape)
    got.copy_(t)
    return got


def forward(B, H, N, d, x="f32", res="f32", out="f32", group=0, residual=True, weight=True,
            eps=1e-6, data=None, shift=False):
    import laplacian_nystr_attention_gb300 as lna
    m = data or make(B, H, N, d, x, res)
    r, w = (m["res"] if residual else None), (m["weight"] if weight else None)
    # eps is an fp32 argument
    want = ref.norm(m["x"], r, w, float(np.float32(eps)), group, out == "f8")
    plan = lna.ResidualNorm(lna.make_norm_config(B, H, N, d, eps=eps, x_dtype=x, res_dtype=res,
                                                 out_dtype=out, scale_group=group))
    place = off_by_one if shift else (lambda t: t)
    total = place(torch.full((B, N, H * d), float("nan"), dtype=TYPES[res], device="cuda"))
    rstd = torch.full((B, N), float("nan"), device="cuda")
    got = plan.forward(place(dev(m["x"], x)), dev(w), residual=dev(r, res), sum=total, rstd=rstd)
    torch.cuda.synchronize()
    ref.check("sum", total, want["sum"], res)
    ref.check("rstd", rstd, want["rstd"])
    if out != "f8":
        ref.check("y", got, want["y"], out)
        return got
    q, scales = got
    assert q.dtype == torch.float8_e4m3fn
    ref.check("scales", scales, want["scales"])
    # A stored value is off by half a step of e4m3: 2^-4 of it, or half of the smallest step,
    # 2^-10, of the scale; then by the roundings of y, of the scale and of their quotient.
    g = group or H * d
    s = scales.double().cpu().numpy().repeat(g, -1)
    back = q.float().double().cpu().numpy() * s
    value, bound = want["y"]
    tol = bound + ref.HALF["f8"] * (np.abs(value) + bound) + s * 2.0 ** -10 + 8 * ref.U * s * 448
    assert (np.abs(back - value) <= tol).all()
    return got


def backward(B, H, N, d, res="f32", grad="f32", dsum=True, weight=True, seed=0, shift=False):
    import laplacian_nystr_attention_gb300 as lna
    m = make(B, H, N, d, "f32", res, grad, seed)
    s = m["res"]
    rstd = ref.rounded(1 / np.sqrt((s * s).mean(-1) + 1e-6), "f32")
    w, ds = (m["weight"] if weight else None), (m["dsum"] if dsum else None)
    want = ref.norm_backward(s, rstd, w, m["dy"], ds, H)
    plan = lna.ResidualNorm(lna.make_norm_config(B, H, N, d, res_dtype=res, grad_dtype=grad))
    place = off_by_one if shift else (lambda t: t)
    dx, dres, dw = plan.backward(place(dev(s, res)), dev(rstd), dev(w), dev(m["dy"], grad),
                                 dsum=dev(ds, grad))
    torch.cuda.synchronize()
    assert dx.shape == (B, H, N, d) and dx.dtype == TYPES[grad]
    ref.check("dx", dx, want["dx"], grad)
    ref.check("dres", dres, want["dres"], grad)
    ref.check("dweight", dw, want["dweight"])
    return dx, dres, dw


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("res", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f8"])
def test_forward_types(x, res, out):
    forward(2, 3, 17, 24, x, res, out)
    forward(2, 3, 17, 23, x, res, out)


@pytest.mark.parametrize("res", ["f32", "bf16"])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_backward_types(res, grad):
    backward(2, 3, 17, 24, res, grad)
    backward(2, 3, 17, 23, res, grad)


WIDTHS = [(1, 1), (1, 2), (1, 7), (1, 8), (2, 8), (3, 8), (1, 33), (5, 13), (2, 64), (8, 64),
          (3, 100), (1, 1000), (1, 1025), (16, 128), (1, 2049), (1, 4096), (2, 2056), (1, 4099),
          (1, 8192), (1, 8200), (3, 4001), (1, 16384), (1, 16383), (128, 128)]


@pytest.mark.parametrize("H,d", WIDTHS)
def test_forward_widths(H, d):
    forward(2, H, 5, d)
    forward(1, H, 3, d, "bf16", "bf16", "bf16", residual=False, weight=False)


@pytest.mark.parametrize("H,d", WIDTHS)
def test_backward_widths(H, d):
    backward(2, H, 5, d)
    backward(1, H, 3, d, "bf16", "bf16", dsum=False, weight=False)


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 33, 257, 5000])
def test_rows(rows):
    forward(1, 2, rows, 32)
    backward(1, 2, rows, 32)
    backward(1, 1, rows, 37)


@pytest.mark.parametrize("H,d", [(3, 1), (4, 3), (8, 5), (5, 13), (2, 333), (8, 257), (3, 1001),
                                 (7, 2333), (9, 1819)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_heads_of_odd_lengths(H, d, kind):
    """Rows of several heads that start anywhere among the vectors, enough for every thread."""
    rows = 1 + 40000 // (H * d)
    forward(1, H, rows, d, kind, kind, kind)
    forward(3, H, 7, d, kind, "f32", "bf16")
    backward(1, H, rows, d, kind, kind)
    backward(3, H, 7, d, "f32", kind, dsum=False)


@pytest.mark.parametrize("rows", [150, 20000])
def test_many_partials_of_dweight(rows):
    backward(1, 1, rows, 64)
    backward(1, 2, min(rows, 2000), 4500)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("H,d", [(1, 128), (4, 32), (2, 640), (8, 16), (32, 20), (1, 4096),
                                 (1, 16384), (128, 51)])
def test_scales(group, H, d):
    if group and H * d % group:
        group = 32 if H * d % 32 == 0 else 0
    forward(2, H, 9, d, "bf16", "bf16", "f8", group=group)
    forward(2, H, 9, d, "f32", "f32", "f8", group=group, shift=True)


def test_rows_of_zeros_and_tiny_values():
    """Zeros give zeros (and a scale of the floor); groups of zeros beside others; subnormals."""
    m = make(1, 1, 4, 256)
    m["x"][:], m["res"][:] = 0.0, 0.0
    m["x"][0, 0, 1, :64] = ref.rounded(np.linspace(-1, 1, 64), "f32")
    m["x"][0, 0, 2] = 2.0 ** -60
    m["x"][0, 0, 3] = ref.rounded(1e15 * np.linspace(-1, 1, 256), "f32")
    for out, group in (("f32", 0), ("bf16", 0), ("f8", 0), ("f8", 64)):
        got = forward(1, 1, 4, 256, out=out, group=group, data=m)
        y = got[0] if out == "f8" else got
        assert (y[0, 0].float() == 0).all()
    assert got[1][0, 0, 0].item() == np.float32(2.0 ** -100 / 448)


def test_misaligned_pointers():
    forward(2, 2, 9, 64, shift=True)
    forward(2, 2, 9, 64, "bf16", "bf16", "bf16", shift=True)
    backward(2, 2, 9, 64, shift=True)
    backward(2, 2, 9, 64, "bf16", "bf16", shift=True)


@pytest.mark.parametrize("d", [64, 63])
def test_in_place(d):
    """sum may be residual, dres may be dsum."""
    import laplacian_nystr_attention_gb300 as lna
    B, H, N = 2, 2, 300
    m = {k: dev(v) for k, v in make(B, H, N, d).items()}
    plan = lna.ResidualNorm(lna.make_norm_config(B, H, N, d))
    total, rstd = torch.empty_like(m["res"]), torch.empty(B, N, device="cuda")
    y = plan.forward(m["x"], m["weight"], residual=m["res"], sum=total, rstd=rstd)
    dx, dres, dw = plan.backward(total, rstd, m["weight"], m["dy"], dsum=m["dsum"])
    y2 = plan.forward(m["x"], m["weight"], residual=m["res"], sum=m["res"])
    dx2, _, dw2 = plan.backward(total, rstd, m["weight"], m["dy"], dsum=m["dsum"],
                                grads={"dres": m["dsum"]})
    for a, b in ((y, y2), (total, m["res"]), (dx, dx2), (dres, m["dsum"]), (dw, dw2)):
        assert torch.equal(a, b)


def test_wanted_gradients_alone():
    import laplacian_nystr_attention_gb300 as lna
    B, H, N, d = 1, 2, 70, 32
    m = {k: dev(v) for k, v in make(B, H, N, d).items()}
    rstd = torch.full((B, N), 0.9, device="cuda")
    plan = lna.ResidualNorm(lna.make_norm_config(B, H, N, d))
    every = plan.backward(m["res"], rstd, m["weight"], m["dy"])
    for keep in range(3):
        names = ["dx", "dres", "dweight"]
        some = plan.backward(m["res"], rstd, m["weight"], m["dy"],
                             grads={n: None for i, n in enumerate(names) if i != keep})
        assert [t is None for t in some] == [i != keep for i in range(3)]
        assert torch.equal(some[keep], every[keep])


def test_empty_batch():
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.ResidualNorm(lna.make_norm_config(0, 2, 5, 8))
    none = torch.empty(0, 5, 16, device="cuda")
    assert plan.forward(torch.empty(0, 2, 5, 8, device="cuda"), residual=none).shape == (0, 5, 16)
    _, _, dw = plan.backward(none, torch.empty(0, 5, device="cuda"), None, none)
    assert (dw == 0).all()


def test_not_finite_rows_stay_alone():
    import laplacian_nystr_attention_gb300 as lna
    m = make(1, 1, 40, 64)
    plan = lna.ResidualNorm(lna.make_norm_config(1, 1, 40, 64))
    good = plan.forward(dev(m["x"]), dev(m["weight"]), residual=dev(m["res"]))
    m["x"][0, 0, 7, 3], m["x"][0, 0, 20, 0] = np.nan, np.inf
    got = plan.forward(dev(m["x"]), dev(m["weight"]), residual=dev(m["res"]))
    keep = [i for i in range(40) if i not in (7, 20)]
    assert torch.equal(good[:, keep], got[:, keep])
    assert torch.isnan(got[0, 7]).all() and torch.isnan(got[0, 20, 0])


def test_bit_for_bit_and_captured():
    import laplacian_nystr_attention_gb300 as lna
    B, H, N, d = 2, 4, 700, 64
    plan = lna.ResidualNorm(lna.make_norm_config(B, H, N, d))
    ins = [{k: dev(v) for k, v in make(B, H, N, d, seed=s).items()} for s in (0, 1)]
    total, rstd = torch.empty(B, N, H * d, device="cuda"), torch.empty(B, N, device="cuda")

    def both(m):
        y = plan.forward(m["x"], m["weight"], residual=m["res"], sum=total, rstd=rstd)
        return (y, *plan.backward(total, rstd, m["weight"], m["dy"], dsum=m["dsum"]))

    want = [[t.clone() for t in both(m)] for m in ins]
    live = {k: v.clone() for k, v in ins[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(live)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(live)
    for k in (1, 0):
        for n, t in live.items():
            t.copy_(ins[k][n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[k], got))


def test_refusals():
    import laplacian_nystr_attention_gb300 as lna
    from laplacian_nystr_attention_gb300 import _lib
    t = torch.zeros(4096, device="cuda")
    p, st = t.data_ptr(), torch.cuda.current_stream().cuda_stream
    h = _lib.lapl_norm_create(lna.make_norm_config(1, 1, 4, 16))
    h8 = _lib.lapl_norm_create(lna.make_norm_config(1, 1, 4, 16, out_dtype="f8"))
    fwd, bwd = _lib.LIB.lapl_norm_forward, _lib.LIB.lapl_norm_backward
    bad = _lib.LAPL_ERR_INVALID_ARG
    assert fwd(h, None, None, None, None, None, p, None, st) == bad
    assert fwd(h, p, None, None, None, None, None, None, st) == bad
    assert fwd(h, p, None, None, None, None, p, p, st) == bad          # scales without 8 bits
    assert fwd(h8, p, None, None, None, None, p, None, st) == bad      # 8 bits without scales
    for k in (1, 2, 3, 4, 5, 6):
        a = [h, p, None, None, None, None, p, None, st]
        a[k] = p + 2
        assert fwd(*a) == _lib.LAPL_ERR_ALIGNMENT
    need = _lib.lapl_norm_workspace_size(h)
    good = [h, p, p, None, p, None, p, None, p, p, need, st]
    for k in (1, 2, 4, 9):
        a = list(good)
        a[k] = None
        assert bwd(*a) == bad
    assert bwd(h, p, p, None, p, None, None, None, None, p, need, st) == bad
    assert bwd(*good[:10], need - 1, st) == _lib.LAPL_ERR_WORKSPACE
    for k in (1, 2, 3, 4, 5, 6, 7, 8, 9):
        a = list(good)
        a[k] = p + 2
        assert bwd(*a) == _lib.LAPL_ERR_ALIGNMENT
    _lib.lapl_norm_destroy(h)
    _lib.lapl_norm_destroy(h8)
    plan = lna.ResidualNorm(lna.make_norm_config(1, 2, 4, 8))
    with pytest.raises(ValueError):
        plan.forward(t[:64].view(1, 4, 16))
    with pytest.raises(ValueError):
        plan.forward(t[:64].view(1, 2, 4, 8), scales=t[:4])
    with pytest.raises(ValueError):
        plan.forward(t[:64].view(1, 2, 4, 8).cpu())


@pytest.mark.parametrize("H,d", [(2, 1024), (1, 2049), (3, 683)])
def test_offsets_past_32_bits(H, d):
    """More than 2^31 values: the last rows."""
    import laplacian_nystr_attention_gb300 as lna
    N, last, W = (1 << 20) + 8, 4, H * d
    assert N * W > 1 << 31
    m = make(1, H, last, d, "bf16", "bf16", "bf16")
    x = torch.zeros(1, H, N, d, dtype=torch.bfloat16, device="cuda")
    res, dy = (torch.zeros(1, N, W, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[:, :, N - last:], res[:, N - last:] = dev(m["x"], "bf16"), dev(m["res"], "bf16")
    dy[:, N - last:] = dev(m["dy"], "bf16")
    w = dev(m["weight"])
    plan = lna.ResidualNorm(lna.make_norm_config(1, H, N, d, x_dtype="bf16", res_dtype="bf16",
                                                 out_dtype="bf16", grad_dtype="bf16"))
    total, rstd = torch.empty_like(res), torch.empty(1, N, device="cuda")
    y = plan.forward(x, w, residual=res, sum=total, rstd=rstd)
    want = ref.norm(m["x"], m["res"], m["weight"], float(np.float32(1e-6)), 0, False)
    ref.check("y", y[:, N - last:], want["y"], "bf16")
    ref.check("sum", total[:, N - last:], want["sum"], "bf16")
    assert (y[:, :N - last] == 0).all()
    dx, dres, dw = plan.backward(total, rstd, w, dy)
    kept = [t[:, N - last:].double().cpu().numpy() for t in (total, rstd)]
    want = ref.norm_backward(kept[0], kept[1], m["weight"], m["dy"], None, H)
    ref.check("dx", dx[:, :, N - last:], want["dx"], "bf16")
    ref.check("dres", dres[:, N - last:], want["dres"], "bf16")
    ref.check("dweight", dw, want["dweight"])
    assert (dres[:, :N - last] == 0).all()
