"""GPU parity of the heads' norm and rotary positions (lapl_rope_*) against their 64-bit reference,
every value within the bound of the roundings on its way (more_operators_reference.py)."""
import numpy as np
import pytest
import torch

import more_operators_reference as ref
from operators_reference import rounded

pytestmark = pytest.mark.gpu

TYPES = ref.TYPES
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()


def dev(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype]).cuda()


def frequencies(pairs):
    return [10000.0 ** (-i / n) for n in pairs for i in range(n)]


def run(B=2, N=7, heads=(2, 1, 1), d=16, pairs=(4, 4), dtype="f32", out=None, grad=None, norm=True,
        weight=True, interleaved=False, pad=None, shift=0, far=0, seed=0):
    """Forward and backward, checked.  pad: elements between a token's rows and the next's, q, k and v
    in one buffer; shift: elements that everything starts off its allocation."""
    import laplacian_nystr_attention_gb300 as lna
    out, grad = out or dtype, grad or dtype
    rng = np.random.default_rng(seed)
    names = [n for n, h in zip("qkv", heads) if h]
    rows = {n: rounded(rng.standard_normal((B, N, h * d)), dtype) for n, h in zip("qkv", heads) if h}
    dy = {n: rounded(rng.standard_normal((B, h, N, d)), grad) for n, h in zip("qkv", heads) if h}
    w = {n: rounded(1 + 0.3 * rng.standard_normal(d), "f32") if norm and weight else None
         for n in "qk"}
    pos = rng.integers(-50, 50, (B, N, len(pairs))) + far
    freq = frequencies(pairs)
    stride = 0 if pad is None else sum(heads) * d + pad
    plan = lna.HeadRotary(lna.make_rope_config(
        B, N, *heads, d, pairs, freq, norm=int(norm), eps=EPS, interleaved=int(interleaved),
        in_dtype=dtype, out_dtype=out, grad_dtype=grad, q_stride=stride, k_stride=stride,
        v_stride=stride))

    def place(t, fill=float("nan")):
        room = torch.full((t.numel() + shift,), fill, dtype=t.dtype, device="cuda")
        got = room[shift:].view(t.shape)
        got.copy_(t)
        return got

    def packed(kind):
        """q, k and v as parts of one buffer's rows, or on their own."""
        both = place(torch.full((B, N, stride or 1), 7.0, dtype=TYPES[kind], device="cuda"))
        parts, at = {}, 0
        for n, h in zip("qkv", heads):
            if h:
                parts[n] = both[..., at:at + h * d] if stride else \
                    place(torch.full((B, N, h * d), 7.0, dtype=TYPES[kind], device="cuda"))
            at += h * d
        return both, parts

    _, ins = packed(dtype)
    for n in names:
        ins[n].copy_(dev(rows[n], dtype))
    positions = place(torch.from_numpy(pos).to(torch.int32).cuda(), 0)
    weights = [place(dev(w[n])) if w[n] is not None and n in names else None for n in "qk"]
    outs = {n: place(torch.full((B, h, N, d), float("nan"), dtype=TYPES[out], device="cuda"))
            for n, h in zip("qkv", heads) if h}
    got = plan.forward(ins.get("q"), ins.get("k"), ins.get("v"), positions, *weights, outs=outs)
    eps = EPS if norm else None
    for n, t, h in zip("qkv", got, heads):
        if not h:
            assert t is None
        elif n == "v":
            assert torch.equal(t, ins["v"].reshape(B, N, h, d).transpose(1, 2).to(TYPES[out]))
        else:
            ref.check(n, t, ref.rope(rows[n], h, pos, pairs, freq, w[n], eps, interleaved), out)
    room, grads = packed(grad)
    grads = {"d" + n: t for n, t in grads.items()}
    dys = [place(dev(dy[n], grad)) if n in names else None for n in "qkv"]
    back = plan.backward(ins.get("q") if norm else None, ins.get("k") if norm else None, positions,
                         *weights, *dys, grads=grads)
    for n, t, h in zip("qkv", back, heads):
        if not h:
            assert t is None
        elif n == "v":
            assert torch.equal(t, dys[2].transpose(1, 2).reshape(B, N, h * d))
        else:
            dx, dw = ref.rope_backward(rows[n], h, pos, pairs, freq, dy[n], w[n], eps, interleaved)
            ref.check("d" + n, t, dx, grad)
            if norm:
                ref.check(f"d{n}_weight", back[3 + "qk".index(n)], dw)
            else:
                assert back[3 + "qk".index(n)] is None
    if pad:
        assert (room[..., sum(heads) * d:] == 7).all()       # between rows: as it was
    return got, back


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("other", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types(dtype, other, interleaved):
    for pairs in ((8,), (3, 4), (2, 2, 2)):
        run(dtype=dtype, out=other, grad=other, interleaved=interleaved, pairs=pairs, d=16)


@pytest.mark.parametrize("d,pairs", [(1, (0,)), (2, (1,)), (3, (1,)), (4, (2,)), (8, (4,)), (16, (4,)),
                                     (16, (0,)), (17, (3, 2)), (31, (15,)), (32, (8, 8)), (64, (32,)),
                                     (65, (32,)), (66, (33,)), (90, (9, 13, 13)), (96, (16, 16, 16)),
                                     (128, (64,)), (129, (64,)), (130, (1,)), (200, (50, 50)),
                                     (254, (127,)), (256, (128,)), (256, (0, 5, 0))])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dimensions(d, pairs, interleaved):
    run(d=d, pairs=pairs, interleaved=interleaved, N=5)
    run(d=d, pairs=pairs, interleaved=interleaved, N=3, dtype="bf16", out="bf16")


@pytest.mark.parametrize("heads", [(1, 0, 0), (1, 1, 0), (3, 0, 2), (8, 2, 2), (1, 4, 1), (16, 16, 16)])
@pytest.mark.parametrize("pad", [None, 0, 4, 3])
def test_heads_and_strides(heads, pad):
    run(heads=heads, pad=pad, d=24, pairs=(4, 4))
    run(heads=heads, pad=pad, d=24, pairs=(4, 4), dtype="bf16")


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_pointers_off_sixteen_bytes(shift):
    run(shift=shift, d=32, pairs=(8, 8))
    run(shift=shift, d=32, pairs=(8, 8), dtype="bf16")


@pytest.mark.parametrize("norm,weight", [(True, False), (False, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_weights_and_without_a_norm(norm, weight, dtype):
    run(norm=norm, weight=weight, dtype=dtype, d=24, pairs=(6, 6))


@pytest.mark.parametrize("N", [1, 2, 8, 9, 64, 1000, 3001])
def test_tokens(N):
    run(B=3, N=N, heads=(2, 1, 1), d=32, pairs=(8, 8), seed=N)


@pytest.mark.parametrize("d,pairs", [(90, (9, 13, 13)), (250, (125,)), (256, (128,)), (256, (40,)),
                                     (4, (2,)), (1, (0,))])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_tokens_of_wide_and_narrow_heads(d, pairs, dtype):
    """Over 32 tokens for each of the GPU's SMs, with as many lanes to a head as there can be, or one."""
    for interleaved in (False, True):
        run(B=3, N=3400, heads=(1, 1, 1), d=d, pairs=pairs, dtype=dtype, interleaved=interleaved)


@pytest.mark.parametrize("far", [0, 1 << 24, (1 << 31) - 60, -(1 << 31) + 60])
@pytest.mark.parametrize("pairs", [(8,), (4, 4)])
def test_far_positions(far, pairs):
    """All 32 bits of a position: the angle is exact to 2^-32 of a turn."""
    run(far=far, pairs=pairs, N=40)


def test_many_rows_in_the_weights_gradient():
    """Few heads over many tokens; small rows beside large ones."""
    run(B=2, N=20000, heads=(2, 1, 0), d=64, pairs=(16, 16), dtype="bf16", grad="f32")


def test_weights_not_wanted():
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.HeadRotary(lna.make_rope_config(1, 4, 2, 1, 0, 8, (4,), frequencies((4,))))
    q, k = torch.randn(1, 4, 16, device="cuda"), torch.randn(1, 4, 8, device="cuda")
    pos = torch.zeros(1, 4, 1, dtype=torch.int32, device="cuda")
    dq, dk = torch.randn(1, 2, 4, 8, device="cuda"), torch.randn(1, 1, 4, 8, device="cuda")
    full = plan.backward(q, k, pos, None, None, dq, dk)
    none = plan.backward(q, k, pos, None, None, dq, dk, grads={"dq_weight": None, "dk_weight": None})
    assert none[3] is None and none[4] is None and torch.equal(none[0], full[0])
    one = plan.backward(q, k, pos, None, None, dq, dk, grads={"dq_weight": None})
    assert one[3] is None and torch.equal(one[4], full[4])


def test_streams_graphs_and_repeats():
    import laplacian_nystr_attention_gb300 as lna
    B, N, d = 2, 700, 64
    plan = lna.HeadRotary(lna.make_rope_config(B, N, 4, 2, 2, d, (16, 16), frequencies((16, 16)),
                                               in_dtype="bf16", out_dtype="bf16",
                                               grad_dtype="bf16"))
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = (new(B, N, h * d).bfloat16() for h in (4, 2, 2))
    pos = torch.randint(0, 99, (B, N, 2), generator=gen, device="cuda", dtype=torch.int32)
    w = new(d)
    dys = [new(B, h, N, d).bfloat16() for h in (4, 2, 2)]

    def both(stream=None):
        return (*plan.forward(q, k, v, pos, w, w, stream=stream),
                *plan.backward(q, k, pos, w, w, *dys, stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both()
        graphs.append((g, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for outs in (got, *(o for _, o, _ in graphs)):
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """The last rows of tensors of over 2^32 values."""
    import laplacian_nystr_attention_gb300 as lna
    N, H, d = 1 << 20, 34, 128                 # 4.56e9 values
    plan = lna.HeadRotary(lna.make_rope_config(1, N, H, 0, 0, d, (64,), frequencies((64,)),
                                               in_dtype="bf16", out_dtype="bf16",
                                               grad_dtype="bf16", eps=EPS))
    q = torch.zeros((1, N, H * d), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    rows = rounded(rng.standard_normal((1, 5, H * d)), "bf16")
    q[:, -5:] = dev(rows, "bf16")
    pos = torch.arange(N, dtype=torch.int32, device="cuda").view(1, N, 1)
    out, _, _ = plan.forward(q, positions=pos)
    at = np.arange(N - 5, N).reshape(1, 5, 1)
    ref.check("q", out[:, :, -5:], ref.rope(rows, H, at, (64,), frequencies((64,)), None, EPS), "bf16")
    dq = plan.backward(q, None, pos, None, None, out)[0]
    want, _ = ref.rope_backward(rows, H, at, (64,), frequencies((64,)),
                                out[:, :, -5:].double().cpu().numpy(), None, EPS)
    ref.check("dq", dq[:, -5:], want, "bf16")


def test_empty_batch():
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.HeadRotary(lna.make_rope_config(0, 4, 2, 1, 0, 8, (4,), frequencies((4,))))
    q, k = torch.empty(0, 4, 16, device="cuda"), torch.empty(0, 4, 8, device="cuda")
    pos = torch.empty(0, 4, 1, dtype=torch.int32, device="cuda")
    qo, ko, _ = plan.forward(q, k, positions=pos)
    assert qo.shape == (0, 2, 4, 8)
    got = plan.backward(q, k, pos, None, None, qo, ko)
    assert not got[3].any() and not got[4].any()


def test_not_finite_rows_stay_their_own():
    """A row with an infinity or NaN makes itself NaN, and no other row."""
    import laplacian_nystr_attention_gb300 as lna
    plan = lna.HeadRotary(lna.make_rope_config(1, 16, 2, 0, 0, 32, (16,), frequencies((16,))))
    q = torch.randn(1, 16, 64, device="cuda")
    pos = torch.arange(16, dtype=torch.int32, device="cuda").view(1, 16, 1)
    want, _, _ = plan.forward(q, positions=pos)
    q[0, 3, 5], q[0, 7, 40] = float("nan"), float("inf")
    got, _, _ = plan.forward(q, positions=pos)
    keep = torch.ones(1, 2, 16, dtype=torch.bool, device="cuda")
    keep[0, 0, 3] = keep[0, 1, 7] = False
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[0, 0, 3]).all() and torch.isnan(got[0, 1, 7]).any()


def test_refusals():
    import laplacian_nystr_attention_gb300 as lna
    make = lambda **kw: lna.HeadRotary(lna.make_rope_config(  # noqa: E731
        **{**dict(batch=1, tokens=4, q_heads=2, k_heads=1, v_heads=0, head_dim=8, pairs=(4,),
                  frequencies=frequencies((4,))), **kw}))
    plan = make()
    q, k = torch.zeros(1, 4, 16, device="cuda"), torch.zeros(1, 4, 8, device="cuda")
    pos = torch.zeros(1, 4, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(8, device="cuda")
    plan.forward(q, k, positions=pos, q_weight=w)
    for args, kw in (((q,), dict(positions=pos)), ((q, k, k), dict(positions=pos)), ((q, k), {}),
                     ((q, k), dict(positions=pos.long())), ((q, q), dict(positions=pos)),
                     ((q, k), dict(positions=pos[:, :3])), ((q.bfloat16(), k), dict(positions=pos)),
                     ((q, k), dict(positions=pos, q_weight=w[:4])),
                     ((q.cpu(), k), dict(positions=pos))):
        with pytest.raises(ValueError):
            plan.forward(*args, **kw)
    with pytest.raises(ValueError):
        make(norm=0).forward(q, k, positions=pos, q_weight=w)
    with pytest.raises(ValueError):
        plan.backward(None, None, pos, None, None, q.view(1, 2, 4, 8), k.view(1, 1, 4, 8))
