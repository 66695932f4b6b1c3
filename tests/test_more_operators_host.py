"""Host-side checks of lapl_rope_*, lapl_decay_* and lapl_adamw_* (no GPU needed): the library exports
every entry point, the binding wraps each and mirrors the structs, bad configurations are refused
before the device is touched, the objects refuse bad tensors, and the references' gradients are those
of differences."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import more_operators_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "lapl_ops.h")).read()
BARE = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
ENTRY_POINTS = sorted(set(re.findall(r"\b(lapl_(?:rope|decay|adamw)_\w+)\s*\(", BARE)))


@pytest.fixture(scope="module")
def lib():
    from conftest import build_library
    build_library()
    from laplacian_nystr_attention_gb300 import _lib
    return _lib


def test_every_entry_point_is_exported_and_wrapped(lib):
    import laplacian_nystr_attention_gb300 as lna
    assert len(ENTRY_POINTS) == 19
    raw = ctypes.CDLL(lib.LIB_PATH)
    for name in ENTRY_POINTS:
        assert hasattr(raw, name) and name in lib.EXPORTED and callable(getattr(lib, name)), name
    for name in ENTRY_POINTS + ["HeadRotary", "DecayAttention", "AdamW"]:
        assert name in lna.__all__ and hasattr(lna, name), name


@pytest.mark.parametrize("struct", ["lapl_rope_config", "lapl_decay_config", "lapl_decay_plan_info",
                                    "lapl_adamw_config"])
def test_structs_match_header(lib, struct):
    body = BARE[:BARE.index("} %s;" % struct)]
    body = body[body.rindex("typedef struct {") + len("typedef struct {"):]
    types = {"int": ctypes.c_int, "float": ctypes.c_float, "double": ctypes.c_double}
    want = []
    for d in (d.strip() for d in body.split(";") if d.strip()):
        name, star = d.split()[-1].lstrip("*"), "*" in d
        kind = types.get(d.replace("const ", "").split()[0].rstrip("*"), ctypes.c_longlong)
        want.append((name, ctypes.POINTER(kind) if star else kind))
    assert [(n, t) for n, t in getattr(lib, struct)._fields_] == want


def test_constants_match_header(lib):
    for name in ("LAPL_ADAMW_BLOCK", "LAPL_ROPE_MAX_DIM", "LAPL_DECAY_MAX_DIM"):
        assert int(re.search(rf"#define {name} (\d+)", HEADER).group(1)) == getattr(lib, name)


def _create(lib, kind, cfg):
    h = ctypes.c_void_p()
    st = getattr(lib.LIB, f"lapl_{kind}_create")(ctypes.byref(cfg), ctypes.byref(h))
    if st == 0:
        getattr(lib.LIB, f"lapl_{kind}_destroy")(h)
    else:
        assert not h.value
    return st


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), 1), (dict(tokens=0), 1), (dict(q_heads=0), 1), (dict(k_heads=-1), 1),
    (dict(v_heads=-1), 1), (dict(head_dim=0), 1), (dict(pairs=(), frequencies=()), 1),
    (dict(pairs=(1, 1, 1, 1)), 1), (dict(pairs=(5,), frequencies=[1.0] * 5), 1),
    (dict(pairs=(-1, 5)), 1), (dict(frequencies=[1.0, float("nan"), 1.0, 1.0]), 1),
    (dict(interleaved=2), 1), (dict(norm=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1),
    (dict(in_dtype=2), 1), (dict(out_dtype=-1), 1), (dict(grad_dtype=5), 1), (dict(q_stride=15), 1),
    (dict(k_stride=-8), 1), (dict(head_dim=257), 2), (dict(batch=1 << 16, tokens=1 << 15), 2),
    (dict(q_heads=5000), 2),
])
def test_rope_refuses_bad_configs(lib, bad, status):
    import laplacian_nystr_attention_gb300 as lna
    good = dict(batch=2, tokens=5, q_heads=2, k_heads=1, v_heads=1, head_dim=8, pairs=(4,),
                frequencies=[1.0] * 4)
    assert _create(lib, "rope", lna.make_rope_config(**{**good, **bad})) == status
    assert _create(lib, "rope", lna.make_rope_config(**good)) in (0, lib.LAPL_ERR_CUDA)
    with pytest.raises(ValueError):
        lna.make_rope_config(**{**good, "frequencies": [1.0] * 3})


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), 1), (dict(heads=0), 1), (dict(tokens=0), 1), (dict(key_dim=0), 1),
    (dict(value_dim=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(reverse=2), 1), (dict(in_dtype=2), 1), (dict(out_dtype=2), 1), (dict(grad_dtype=-1), 1),
    (dict(key_dim=129), 2), (dict(value_dim=129), 2), (dict(tokens=(1 << 30) + 1), 2),
    (dict(batch=1 << 12, heads=1 << 11), 2),
])
def test_decay_refuses_bad_configs(lib, bad, status):
    import laplacian_nystr_attention_gb300 as lna
    good = dict(batch=2, heads=2, tokens=5, key_dim=8, value_dim=8)
    assert _create(lib, "decay", lna.make_decay_config(**{**good, **bad})) == status
    assert _create(lib, "decay", lna.make_decay_config(**good)) in (0, lib.LAPL_ERR_CUDA)


def _adamw_config(lib, counts=(3, 4), dtypes=(0, 1), grads=(0, 1), decay=(0.0, 0.1), betas=(0.9, 0.99),
                  eps=1e-8, bits=32):
    n = len(counts)
    return lib.lapl_adamw_config(n, (ctypes.c_longlong * n)(*counts), (ctypes.c_int * n)(*dtypes),
                                 (ctypes.c_int * n)(*grads), (ctypes.c_float * n)(*decay), *betas,
                                 eps, bits)


@pytest.mark.parametrize("bad,status", [
    (dict(counts=(3, -1)), 1), (dict(dtypes=(0, 2)), 1), (dict(grads=(-1, 0)), 1),
    (dict(decay=(0.0, -0.1)), 1), (dict(decay=(float("nan"), 0.1)), 1), (dict(betas=(1.0, 0.9)), 1),
    (dict(betas=(0.9, -0.1)), 1), (dict(betas=(0.9, float("nan"))), 1), (dict(eps=0.0), 1),
    (dict(eps=1e-60), 1), (dict(eps=float("inf")), 1), (dict(bits=16), 1),
    (dict(counts=(3, (1 << 40) + 1)), 2),
])
def test_adamw_refuses_bad_configs(lib, bad, status):
    assert _create(lib, "adamw", _adamw_config(lib, **bad)) == status
    assert _create(lib, "adamw", _adamw_config(lib)) in (0, lib.LAPL_ERR_CUDA)
    assert _create(lib, "adamw", lib.lapl_adamw_config(-1)) == 1
    assert _create(lib, "adamw", lib.lapl_adamw_config(1, beta1=0.9, beta2=0.9, eps=1e-8,
                                                       state_bits=32)) == 1


def test_null_arguments(lib):
    for kind in ("rope", "decay", "adamw"):
        assert getattr(lib.LIB, f"lapl_{kind}_create")(None, None) == 1
        assert getattr(lib.LIB, f"lapl_{kind}_destroy")(None) == 0
        assert getattr(lib.LIB, f"lapl_{kind}_last_error")(None) == b""
    assert lib.LIB.lapl_rope_forward(*[None] * 11) == 1
    assert lib.LIB.lapl_rope_backward(*[None] * 15, 0, None) == 1
    assert lib.LIB.lapl_rope_workspace_size(None, None) == 1
    assert lib.LIB.lapl_decay_forward(*[None] * 10, 0, None) == 1
    assert lib.LIB.lapl_decay_backward(*[None] * 14, 0, None) == 1
    assert lib.LIB.lapl_decay_workspace_size(None, None, None) == 1
    assert lib.LIB.lapl_decay_plan_info_get(None, None) == 1
    assert lib.LIB.lapl_decay_device_errors(None, None, None) == 1
    assert lib.LIB.lapl_decay_set_fault_injection(None, 0, 0) == 1
    assert lib.LIB.lapl_adamw_step(*[None] * 8, 0.1, None, 1, None, None, 0.0, None) == 1


def test_tensor_checks_refuse(lib):
    """Objects without a handle, for tensors on the CPU (device index -1)."""
    import laplacian_nystr_attention_gb300 as lna
    r = lna.HeadRotary.__new__(lna.HeadRotary)
    r.device = torch.device("cpu")
    r._layouts(lna.make_rope_config(2, 5, 2, 1, 0, 8, (4,), [1.0] * 4, q_stride=24, k_stride=24))
    rows = torch.zeros(2, 5, 24)
    r._part("q", rows[..., :16], r._in)
    r._part("k", rows[..., 16:], r._in)
    assert r._part("v", None, r._in) is None
    for name, t in (("q", rows[..., :8]), ("k", torch.zeros(2, 5, 8)), ("q", None), ("v", rows)):
        with pytest.raises(ValueError):
            r._part(name, t, r._in)
    with pytest.raises(ValueError):
        r._common(None, None, None)
    with pytest.raises(ValueError):
        r._common(torch.zeros(2, 5, 1), None, None)
    d = lna.DecayAttention.__new__(lna.DecayAttention)
    d.device = torch.device("cpu")
    d._layouts(lna.make_decay_config(2, 3, 5, 8, 4))
    d._check(torch.zeros(2, 3, 5, 8), d._in["q"])
    d._check(torch.zeros(2, 3, 8, 4), d._state["state"])
    for t, want in ((torch.zeros(2, 3, 5, 4), d._in["k"]), (torch.zeros(2, 3, 4, 8), d._state["state"]),
                    (torch.zeros(2, 5, 3, 8).transpose(1, 2), d._in["q"]),
                    (torch.zeros(2), d._lengths), (torch.zeros(2), d._log_decay)):
        with pytest.raises(ValueError):
            d._check(t, want)
    a = lna.AdamW.__new__(lna.AdamW)
    a.device, a.counts, a.dtypes, a.grad_dtypes = torch.device("cpu"), [4, 300], [0, 1], [0, 1]
    a.state_bits, a.masters = 8, True
    a._layouts()
    p = [torch.zeros(2, 2), torch.zeros(300, dtype=torch.bfloat16)]
    s = a.new_states(p)
    assert [t.numel() for t in s["m_scales"]] == [1, 2] and s["m"][0].dtype is torch.float8_e4m3fn
    assert s["masters"][0] is None and a._masters(s["masters"])[0] is None
    for name, t in (("params", p[:1]), ("params", [p[1], p[0]]), ("m", p), ("v_scales", s["m"]),
                    ("grads", None), ("grads", [torch.zeros(4, 2)[:, 0], p[1]])):
        with pytest.raises(ValueError):
            a._list(t, name)
    for bad in (None, [None], [None, None], p):
        with pytest.raises(ValueError):
            a._masters(bad)
    with pytest.raises(ValueError):
        lna.AdamW([1, 2], ["f32"])
    with pytest.raises(ValueError):
        lna.AdamW([1, 2], ["f32", "f32"], weight_decay=[0.1])
    with pytest.raises(ValueError):
        lna.AdamW.like([torch.zeros(3, dtype=torch.float64)])


# ---- the references against differences --------------------------------------------------

def _differences(loss, args, got, names, step=1e-6):
    """Differences are off by about step^2 and 1e-16 / step, times the loss's size."""
    for name, k in names:
        want = np.zeros_like(args[k])
        for at in np.ndindex(want.shape):
            hi, lo = ([a.copy() for a in args] for _ in range(2))
            hi[k][at] += step
            lo[k][at] -= step
            want[at] = (loss(*hi) - loss(*lo)) / (2 * step)
        assert np.abs(got[name][0] - want).max() < 1e-6, name


@pytest.mark.parametrize("reverse", [False, True])
def test_decay_reference_gradient_against_differences(reverse):
    rng = np.random.default_rng(3)
    B, H, N, a, b, lens = 2, 2, 5, 3, 2, [5, 3]
    q, k = rng.standard_normal((2, B, H, N, a))
    v, dout = rng.standard_normal((2, B, H, N, b))
    state, dfinal = rng.standard_normal((2, B, H, a, b))
    logs = np.array([-0.3, 0.0])

    def loss(q, k, v, state):
        r = ref.decay(q, k, v, logs, 0.7, state, lens, reverse)
        return (r["out"][0] * dout).sum() + (r["final"][0] * dfinal).sum()

    got = ref.decay(q, k, v, logs, 0.7, state, lens, reverse, dout, dfinal)
    _differences(loss, [q, k, v, state], got, (("dq", 0), ("dk", 1), ("dv", 2), ("dstate", 3)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_reference_gradient_against_differences(interleaved):
    rng = np.random.default_rng(4)
    B, N, H, d, pairs, freq = 2, 3, 2, 7, (2, 1), [1.0, 0.3, 0.5]
    x, w = rng.standard_normal((B, N, H * d)), rng.standard_normal(d)
    dy, pos = rng.standard_normal((B, H, N, d)), rng.integers(0, 9, (B, N, 2))

    def loss(x, w):
        return (ref.rope(x, H, pos, pairs, freq, w, 1e-3, interleaved)[0] * dy).sum()

    dx, dw = ref.rope_backward(x, H, pos, pairs, freq, dy, w, 1e-3, interleaved)
    _differences(loss, [x, w], {"dx": dx, "dw": dw}, (("dx", 0), ("dw", 1)))


def test_angles_of_far_positions():
    """Reduced in long double: within 1e-9 of exact integer arithmetic on a frequency that is a whole
    fraction of a turn."""
    f = 2 * np.pi / 64
    pos = np.array([[[(1 << 31) - 5], [3]]])
    got = ref.angles(pos, (1,), [f])[0, 0, :, 0]
    want = np.array([(((1 << 31) - 5) % 64) * f, 3 * f])
    off = ((1 << 31) - 5) * abs(np.longdouble(f) * 64
                                - np.longdouble("6.283185307179586476925286766559005768")) / 64
    assert np.abs(got - want).max() < 1e-9 + float(off)
