"""Host-side checks of include/lapl_ops.h (no GPU needed): the library exports every entry point,
the binding wraps each and mirrors the structs, bad configurations are refused before the device is
touched, and the objects over tensors refuse bad tensors."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import operators_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "lapl_ops.h")).read()
BARE = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
ENTRY_POINTS = sorted(set(re.findall(r"\b(lapl_(?:scan|norm|clip)_\w+)\s*\(", BARE)))


@pytest.fixture(scope="module")
def lib():
    from conftest import build_library
    build_library()
    from laplacian_nystr_attention_gb300 import _lib
    return _lib


def test_every_entry_point_is_exported_and_wrapped(lib):
    assert len(ENTRY_POINTS) == 20
    raw = ctypes.CDLL(lib.LIB_PATH)
    for name in ENTRY_POINTS:
        assert hasattr(raw, name) and name in lib.EXPORTED and callable(getattr(lib, name)), name


def test_names_are_public():
    import laplacian_nystr_attention_gb300 as lna
    for name in ENTRY_POINTS + ["GatedScan", "ResidualNorm", "GradClip"]:
        assert name in lna.__all__ and hasattr(lna, name), name


@pytest.mark.parametrize("struct", ["lapl_scan_config", "lapl_scan_plan_info", "lapl_norm_config",
                                    "lapl_clip_config"])
def test_structs_match_header(lib, struct):
    body = BARE[:BARE.index("} %s;" % struct)]
    body = body[body.rindex("typedef struct {") + len("typedef struct {"):]
    names = [d.strip().split()[-1].lstrip("*") for d in body.split(";") if d.strip()]
    assert names == [n for n, _ in getattr(lib, struct)._fields_]


def test_chunk_matches_header(lib):
    assert int(re.search(r"#define LAPL_SCAN_CHUNK (\d+)", HEADER).group(1)) == lib.LAPL_SCAN_CHUNK


def _create(lib, kind, cfg):
    h = ctypes.c_void_p()
    st = getattr(lib.LIB, f"lapl_{kind}_create")(ctypes.byref(cfg), ctypes.byref(h))
    if st == 0:
        getattr(lib.LIB, f"lapl_{kind}_destroy")(h)
    else:
        assert not h.value
    return st


@pytest.mark.parametrize("bad,status", [
    (dict(sequences=-1), 1), (dict(tokens=0), 1), (dict(channels=0), 1), (dict(gate=2), 1),
    (dict(gate=-1), 1), (dict(reverse=2), 1), (dict(in_dtype=2), 1), (dict(out_dtype=2), 1),
    (dict(grad_dtype=-1), 1), (dict(x_stride=7), 1), (dict(g_stride=-8), 1),
    (dict(tokens=(1 << 30) + 1), 2), (dict(channels=(1 << 24) + 1), 2),
    (dict(sequences=1 << 28, channels=1), 2),
])
def test_scan_refuses_bad_configs(lib, bad, status):
    import laplacian_nystr_attention_gb300 as lna
    good = dict(sequences=2, tokens=5, channels=8)
    assert _create(lib, "scan", lna.make_scan_config(**{**good, **bad})) == status
    assert _create(lib, "scan", lna.make_scan_config(**good)) in (0, lib.LAPL_ERR_CUDA)


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), 1), (dict(heads=0), 1), (dict(tokens=0), 1), (dict(head_dim=0), 1),
    (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(x_dtype=2), 1), (dict(res_dtype=2), 1), (dict(out_dtype=3), 1), (dict(grad_dtype=2), 1),
    (dict(scale_group=32), 1), (dict(out_dtype="f8", scale_group=16), 1),
    (dict(out_dtype="f8", scale_group=64, head_dim=33), 1),
    (dict(heads=4, head_dim=4097), 2), (dict(batch=1 << 16, tokens=1 << 15), 2),
])
def test_norm_refuses_bad_configs(lib, bad, status):
    import laplacian_nystr_attention_gb300 as lna
    good = dict(batch=2, heads=2, tokens=5, head_dim=32)
    assert _create(lib, "norm", lna.make_norm_config(**{**good, **bad})) == status
    assert _create(lib, "norm", lna.make_norm_config(**good)) in (0, lib.LAPL_ERR_CUDA)


@pytest.mark.parametrize("counts,dtypes,status", [([3, -1], [0, 0], 1), ([3], [2], 1),
                                                  ([(1 << 40) + 1], [0], 2)])
def test_clip_refuses_bad_configs(lib, counts, dtypes, status):
    n = len(counts)
    cfg = lib.lapl_clip_config(n, (ctypes.c_longlong * n)(*counts), (ctypes.c_int * n)(*dtypes))
    assert _create(lib, "clip", cfg) == status
    assert _create(lib, "clip", lib.lapl_clip_config(-1, None, None)) == 1
    assert _create(lib, "clip", lib.lapl_clip_config(2, None, None)) == 1


def test_null_arguments(lib):
    for kind in ("scan", "norm", "clip"):
        assert getattr(lib.LIB, f"lapl_{kind}_create")(None, None) == 1
        assert getattr(lib.LIB, f"lapl_{kind}_destroy")(None) == 0
        assert getattr(lib.LIB, f"lapl_{kind}_last_error")(None) == b""
    assert lib.LIB.lapl_scan_forward(*[None] * 9) == 1
    assert lib.LIB.lapl_scan_backward(*[None] * 11) == 1
    assert lib.LIB.lapl_scan_plan_info_get(None, None) == 1
    assert lib.LIB.lapl_scan_device_errors(None, None, None) == 1
    assert lib.LIB.lapl_scan_set_fault_injection(None, 0, 0) == 1
    assert lib.LIB.lapl_norm_forward(*[None] * 9) == 1
    assert lib.LIB.lapl_norm_backward(*[None] * 10, 0, None) == 1
    assert lib.LIB.lapl_norm_workspace_size(None, None) == 1
    assert lib.LIB.lapl_clip_norm(None, None, None, None, 0, None) == 1
    assert lib.LIB.lapl_clip_apply(None, None, None, 1.0, None, None, 0, None) == 1
    assert lib.LIB.lapl_clip_workspace_size(None, None) == 1


def test_tensor_checks_refuse(lib):
    """An object without a handle, for tensors on the CPU (device index -1)."""
    import laplacian_nystr_attention_gb300 as lna
    p = lna.GatedScan.__new__(lna.GatedScan)
    p.device = torch.device("cpu")
    p._layouts(lna.make_scan_config(6, 5, 8, x_stride=16))
    wide = torch.zeros(6, 5, 16)
    for good in (wide[..., :8], wide[..., 8:], torch.zeros(2, 3, 5, 16)[..., :8]):
        assert p._check(good, p._x) == good.data_ptr()
    p._check(torch.zeros(6, 5, 8), p._g)
    for bad in (torch.zeros(6, 5, 8), wide, wide[:, :4, :8], wide[..., :8].bfloat16(),
                torch.zeros(5, 6, 16)[..., :8].transpose(0, 1), torch.zeros(30, 16)[:, :8],
                torch.zeros(6, 6, 16)[:, :5, :8], torch.zeros(2, 4, 5, 16)[..., :8]):
        with pytest.raises(ValueError):
            p._check(bad, p._x)
    with pytest.raises(ValueError):
        p._check(torch.zeros(6, 9), p._state["h0"])
    one = lna.GatedScan.__new__(lna.GatedScan)
    one.device = torch.device("cpu")
    one._layouts(lna.make_scan_config(3, 1, 8, x_stride=16))
    one._check(torch.zeros(3, 1, 16)[..., :8], one._x)       # a size-1 stride says nothing
    with pytest.raises(ValueError):
        one._check(torch.zeros(3, 1, 8), one._x)
    n = lna.ResidualNorm.__new__(lna.ResidualNorm)
    n.device = torch.device("cpu")
    n._layouts(lna.make_norm_config(2, 1, 5, 8))
    n._by_head(torch.zeros(2, 5, 8), n._x, n._x_row)
    n._by_head(torch.zeros(2, 1, 5, 8), n._x, n._x_row)
    with pytest.raises(ValueError):
        n._by_head(torch.zeros(2, 5, 1, 8), n._x, n._x_row)
    c = lna.GradClip.__new__(lna.GradClip)
    c.counts, c._torch_dtypes = [4, 0], [torch.float32, torch.bfloat16]
    c._devices = [-1, -1]
    c.device = torch.device("cpu")
    assert len(c._list([torch.zeros(2, 2), torch.zeros(0, dtype=torch.bfloat16)], "g")) == 2
    for bad in ([torch.zeros(4)], [torch.zeros(5), torch.zeros(0, dtype=torch.bfloat16)],
                [torch.zeros(4, 2)[:, 0], torch.zeros(0, dtype=torch.bfloat16)],
                [torch.zeros(4), torch.zeros(0)]):
        with pytest.raises(ValueError):
            c._list(bad, "g")
    with pytest.raises(ValueError):
        lna.GradClip([1, 2], ["f32"])


# ---- the references against differences --------------------------------------------------

@pytest.mark.parametrize("gate", ["decay", "sigmoid"])
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_reference_gradient_against_differences(gate, reverse):
    rng = np.random.default_rng(3)
    S, N, C, lens = 2, 7, 3, [7, 4]
    x, g, h0 = rng.standard_normal((S, N, C)), rng.standard_normal((S, N, C)), \
        rng.standard_normal((S, C))
    if gate == "decay":
        g = np.tanh(g)
    dout, dfinal = rng.standard_normal((S, N, C)), rng.standard_normal((S, C))

    def loss(x, g, h0):
        r = ref.scan(x, g, gate, h0, lens, reverse)
        return (r["h"][0] * dout).sum() + (r["final"][0] * dfinal).sum()

    got = ref.scan(x, g, gate, h0, lens, reverse, dout, dfinal)
    step = 1e-6                # differences are off by about step^2 and 1e-16 / step
    for name, k in (("dx", 0), ("dg", 1), ("dh0", 2)):
        args = [x, g, h0]
        want = np.zeros_like(args[k])
        for at in np.ndindex(want.shape):
            hi, lo = ([a.copy() for a in args] for _ in range(2))
            hi[k][at] += step
            lo[k][at] -= step
            want[at] = (loss(*hi) - loss(*lo)) / (2 * step)
        assert np.abs(got[name][0] - want).max() < 1e-7


def test_norm_reference_gradient_against_differences():
    rng = np.random.default_rng(4)
    B, H, N, d = 2, 2, 3, 4
    x, w = rng.standard_normal((B, H, N, d)), rng.standard_normal(H * d)
    res, dy, dsum = (rng.standard_normal((B, N, H * d)) for _ in range(3))

    def loss(x, w):
        r = ref.norm(x, res, w, 1e-3)
        return (r["y"][0] * dy).sum() + (r["sum"][0] * dsum).sum()

    fwd = ref.norm(x, res, w, 1e-3)
    got = ref.norm_backward(fwd["sum"][0], fwd["rstd"][0], w, dy, dsum, H)
    step = 1e-6
    for name, k in (("dx", 0), ("dweight", 1)):
        args = [x, w]
        want = np.zeros_like(args[k])
        for at in np.ndindex(want.shape):
            hi, lo = ([a.copy() for a in args] for _ in range(2))
            hi[k][at] += step
            lo[k][at] -= step
            want[at] = (loss(*hi) - loss(*lo)) / (2 * step)
        assert np.abs(got[name][0] - want).max() < 1e-7
