"""The operators beside the attention, as cases to measure: the gated linear recurrence over
tokens, the residual addition with the root-mean-square norm, and the global gradient norm with
clipping.

``run`` computes a case in plain torch operations in 32 bits where ``own`` is false, and by the
library's kernels where it is true; ``exact`` gives the same values in 64 bits.
"""
import math

import torch

own = False

#: Tokens between two states that the recurrence's forward keeps for its backward.
CHUNK = 16
#: Largest finite e4m3 value, and the smallest largest value a scale is made for.
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f8": 1}

# ---- cases -------------------------------------------------------------------------------


def _scan(op, sequences, tokens, channels, gate, dtype, out="", grad="", reverse=False,
          lengths=False, packed=False, h0=False, states=False, name=None):
    c = dict(op=op, sequences=sequences, tokens=tokens, channels=channels, gate=gate, dtype=dtype,
             out=out or dtype, grad=grad or dtype, reverse=reverse, lengths=lengths,
             packed=packed, h0=h0, states=states)
    return dict(c, name=name) if name else c


def _norm(op, batch, heads, tokens, head_dim, x, res, out="", grad="f32", group=0, residual=True,
          dsum=True, name=None):
    c = dict(op=op, batch=batch, heads=heads, tokens=tokens, head_dim=head_dim, x=x, res=res,
             out=out or res, grad=grad, group=group, residual=residual, dsum=dsum)
    return dict(c, name=name) if name else c


def _clip(op, tensors, elements, kinds, over, flat=False, name=None):
    c = dict(op=op, tensors=tensors, elements=elements, kinds=kinds, over=over, flat=flat)
    return dict(c, name=name) if name else c


def listed():
    return [
        # One token for each of 64 sequences from the state of the one before: generation.
        _scan("scan_forward", 64, 1, 512, "sigmoid", "bf16", h0=True, name="scan_step_bf16"),
        # The stage-1 vision shape: 8 images of 56 x 56 tokens, 2 heads of 32 channels.
        _scan("scan_forward", 16, 3136, 32, "decay", "f32", name="scan_fwd_stage1_f32"),
        # The longest sequence of the length sweep, its training forward: 8 heads, 256 x 256 tokens.
        _scan("scan_forward", 8, 65536, 64, "sigmoid", "bf16", states=True,
              name="scan_fwd_sweep_bf16"),
        # The high-resolution shape's backward: 4 images of 128 x 128 tokens, 8 heads.
        _scan("scan_backward", 32, 16384, 64, "sigmoid", "bf16", name="scan_bwd_hires_bf16"),
        # A padded batch of odd sizes, gate and input in one projection's output, last token first.
        _scan("scan_backward", 7, 2047, 333, "decay", "f32", reverse=True, lengths=True,
              packed=True, h0=True, name="scan_bwd_padded_f32"),
        # The tiny shape: 256 tokens of one head; latency.
        _norm("norm_forward", 1, 1, 256, 32, "f32", "f32", name="norm_fwd_tiny_f32"),
        # What follows the attention at the high-resolution shape: its fp32 output, heads merged.
        _norm("norm_forward", 4, 8, 16384, 64, "f32", "bf16", name="norm_fwd_hires"),
        # Wide rows for a product in 8 bits, a scale for each 128 values.
        _norm("norm_forward", 1, 1, 8192, 4096, "bf16", "bf16", out="f8", group=128,
              name="norm_fwd_f8"),
        # The stage-2/3 shape's backward: 32 images of 28 x 28 tokens, 4 heads of 64 channels.
        _norm("norm_backward", 32, 4, 784, 64, "f32", "f32", name="norm_bwd_stage23_f32"),
        # Wide rows of an odd length, gradients in bf16.
        _norm("norm_backward", 3, 1, 2731, 2049, "bf16", "bf16", grad="bf16",
              name="norm_bwd_odd_bf16"),
        # The gradients of one small block, clipped.
        _clip("clip", 24, 1 << 20, "f32", True, name="clip_block_f32"),
        # The gradients of a whole model, bf16 weights with fp32 vectors between them.
        _clip("clip", 60, 1 << 28, "mixed", True, name="clip_model_mixed"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["scan_forward", "scan_backward", "norm_forward", "norm_backward", "clip",
                       "norm"])
    if kind.startswith("scan"):
        tokens = 1 if kind == "scan_forward" and rng.random() < 0.2 else _spread(rng, 1, 65536)
        channels = _spread(rng, 1, 1024)
        if rng.random() < 0.6:
            channels = 8 * max(1, channels // 8)
        most = max(1, min(512, (1 << 24) // (tokens * channels)))
        sequences = _spread(rng, 1, most)
        dtype = rng.choice(["f32", "bf16"])
        return _scan(kind, sequences, tokens, channels, rng.choice(["decay", "sigmoid"]), dtype,
                     out=rng.choice(["f32", "bf16"]), grad=rng.choice(["f32", "bf16"]),
                     reverse=rng.random() < 0.3, lengths=rng.random() < 0.4,
                     packed=rng.random() < 0.3, h0=rng.random() < 0.5,
                     states=kind == "scan_forward" and rng.random() < 0.5)
    if kind.startswith("norm_"):
        heads = rng.choice([1, 1, 2, 3, 8])
        head_dim = _spread(rng, 1, 16384 // heads)
        if rng.random() < 0.6:
            head_dim = 8 * max(1, head_dim // 8)
        out = rng.choice(["f32", "bf16", "f8"]) if kind == "norm_forward" else "bf16"
        groups = [0] + [g for g in (32, 64, 128) if heads * head_dim % g == 0 and out == "f8"]
        most = max(1, min(1 << 17, (1 << 24) // (heads * head_dim)))
        batch = rng.choice([1, 2, 5])
        return _norm(kind, batch, heads, max(1, _spread(rng, 1, most) // batch), head_dim,
                     rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]), out=out,
                     grad=rng.choice(["f32", "bf16"]), group=rng.choice(groups),
                     residual=kind == "norm_backward" or rng.random() < 0.8,
                     dsum=rng.random() < 0.7)
    return _clip(kind, _spread(rng, 1, 60 if kind == "clip" else 400), _spread(rng, 64, 1 << 26),
                 rng.choice(["f32", "bf16", "mixed"]), rng.random() < 0.8,
                 flat=rng.random() < 0.4)


# ---- inputs ------------------------------------------------------------------------------


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, gen, dtype=torch.float32, scale=1.0, shift=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(scale).add_(shift).to(dtype)


def _scan_inputs(case, seed):
    gen = _rng(seed)
    S, N, C = case["sequences"], case["tokens"], case["channels"]
    t = TYPES[case["dtype"]]
    x = _normal((S, N, C), gen, t)
    # Gates around 0.9: memories of some tens of tokens, some of thousands.
    g = _normal((S, N, C), gen, scale=1.5, shift=2.2)
    g = (torch.sigmoid(g) if case["gate"] == "decay" else g).to(t)
    if case["packed"]:
        # One projection's output, x and g side by side; rows start at multiples of 16 bytes.
        per = 16 // BYTES[case["dtype"]]
        half = -(-C // per) * per
        both = torch.zeros((S, N, 2 * half), dtype=t, device="cuda")
        both[..., :C] = x
        both[..., half:half + C] = g
        x, g = both[..., :C], both[..., half:half + C]
    s = {"x": x, "g": g, "h0": None, "lengths": None}
    if case["h0"]:
        s["h0"] = _normal((S, C), gen)
    if case["lengths"]:
        n = torch.randint(0, N + 1, (S,), generator=gen, device="cuda", dtype=torch.int32)
        n[0] = N
        s["lengths"] = n
    if case["op"] == "scan_backward":
        s["dh"] = _normal((S, N, C), gen, TYPES[case["grad"]])
        s["dfinal"] = _normal((S, C), gen) if case["h0"] else None
    return s


def _norm_inputs(case, seed):
    gen = _rng(seed)
    B, H, N, d = case["batch"], case["heads"], case["tokens"], case["head_dim"]
    s = {"weight": _normal((H * d,), gen, scale=0.2, shift=1.0)}
    if case["op"] == "norm_forward":
        s["x"] = _normal((B, H, N, d), gen, TYPES[case["x"]], scale=0.5)
        s["residual"] = (_normal((B, N, H * d), gen, TYPES[case["res"]]) if case["residual"]
                         else None)
        return s
    s["sum"] = _normal((B, N, H * d), gen, TYPES[case["res"]])
    s["rstd"] = (s["sum"].float().square().mean(-1) + 1e-6).rsqrt()
    s["dy"] = _normal((B, N, H * d), gen, TYPES[case["grad"]])
    s["dsum"] = _normal((B, N, H * d), gen, TYPES[case["grad"]]) if case["dsum"] else None
    return s


def _sizes(case):
    """Sizes of a model's tensors: weights of a few sizes and many short vectors."""
    n, total = case["tensors"], case["elements"]
    weights = [1.0 / (1 + i % 7) ** 2 if i % 3 == 0 else 1e-4 * (1 + i % 11) for i in range(n)]
    unit = total / sum(weights)
    return [max(1, int(w * unit)) | 1 for w in weights]


def _kinds(case):
    if case["kinds"] != "mixed":
        return [case["kinds"]] * case["tensors"]
    return ["bf16" if i % 3 == 0 else "f32" for i in range(case["tensors"])]


def _clip_inputs(case, seed):
    gen = _rng(seed)
    grads = [_normal((n,), gen, TYPES[k], scale=1e-3 * (1 + i % 5))
             for i, (n, k) in enumerate(zip(_sizes(case), _kinds(case)))]
    if case["flat"]:
        # Slices of one buffer for each type, end to end, so that most start anywhere.
        for t in set(g.dtype for g in grads):
            mine = [i for i, g in enumerate(grads) if g.dtype == t]
            parts = torch.cat([grads[i] for i in mine]).split([grads[i].numel() for i in mine])
            for i, part in zip(mine, parts):
                grads[i] = part
    # Well over or well under the norm that they have.
    about = math.sqrt(sum(g.numel() * (1e-3 * (1 + i % 5)) ** 2 for i, g in enumerate(grads)))
    return {"grads": grads, "max_norm": about * (0.25 if case["over"] else 4.0)}


def _inputs(case, seed):
    if case["op"].startswith("scan"):
        return _scan_inputs(case, seed)
    if case["op"].startswith("norm_"):
        return _norm_inputs(case, seed)
    return _clip_inputs(case, seed)


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"] == "scan_backward":
        # The states that the forward kept, from the seed alone as everything here.
        s["states"] = _states(*_scan_coefficients(case, s), s["h0"])
    if own:
        s["plan"] = _plan(case)
    return s


def _plan(case):
    import laplacian_nystr_attention_gb300 as lna
    if case["op"].startswith("scan"):
        per = 16 // BYTES[case["dtype"]]
        stride = 2 * (-(-case["channels"] // per) * per) if case["packed"] else 0
        return lna.GatedScan(lna.make_scan_config(
            case["sequences"], case["tokens"], case["channels"], gate=case["gate"],
            reverse=int(case["reverse"]), in_dtype=case["dtype"], out_dtype=case["out"],
            grad_dtype=case["grad"], x_stride=stride, g_stride=stride))
    if case["op"].startswith("norm_"):
        return lna.ResidualNorm(lna.make_norm_config(
            case["batch"], case["heads"], case["tokens"], case["head_dim"], eps=1e-6,
            x_dtype=case["x"], res_dtype=case["res"], out_dtype=case["out"],
            grad_dtype=case["grad"], scale_group=case["group"]))
    return lna.GradClip(_sizes(case), _kinds(case))


# ---- plain forms -------------------------------------------------------------------------


def _order(case, lengths):
    """The token at each place of the processing order, [S, N, 1], and where that is a token."""
    S, N = case["sequences"], case["tokens"]
    i = torch.arange(N, device="cuda").expand(S, N)
    n = lengths.to(torch.int64)[:, None] if lengths is not None else torch.full_like(i[:, :1], N)
    valid = i < n
    at = torch.where(valid, n - 1 - i, i) if case["reverse"] else i
    return at[..., None], valid[..., None]


def _ordered(t, at):
    return t.gather(1, at.expand(t.shape))


def _recur(a, b):
    """h with h_i = a_i h_{i-1} + b_i along dim 1, from 0: pairs of steps first, then between."""
    if a.shape[1] == 1:
        return b
    if a.shape[1] % 2:
        h = _recur(a[:, :-1], b[:, :-1])
        return torch.cat([h, a[:, -1:] * h[:, -1:] + b[:, -1:]], 1)
    a0, a1, b0, b1 = a[:, 0::2], a[:, 1::2], b[:, 0::2], b[:, 1::2]
    late = _recur(a0 * a1, a1 * b0 + b1)
    early = torch.cat([b0[:, :1], a0[:, 1:] * late[:, :-1] + b0[:, 1:]], 1)
    return torch.stack([early, late], 2).reshape(a.shape)


def _scan_coefficients(case, s):
    """(a, 1 - a, x) in processing order, a step that leaves the state as it is where no token is."""
    at, valid = _order(case, s["lengths"])
    g, x = _ordered(s["g"].float(), at), _ordered(s["x"].float(), at)
    a = 1 / (1 + torch.exp(-g)) if case["gate"] == "sigmoid" else g
    z = 1 / (1 + torch.exp(g)) if case["gate"] == "sigmoid" else torch.ones_like(g)
    return torch.where(valid, a, 1.0), torch.where(valid, z, 0.0), torch.where(valid, x, 0.0)


def _from(a, b, h0):
    if h0 is not None:
        b = torch.cat([b[:, :1] + a[:, :1] * h0[:, None], b[:, 1:]], 1)
    return _recur(a, b)


def _before(h, h0):
    first = torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None]
    return torch.cat([first, h[:, :-1]], 1)


def _states(a, z, x, h0):
    return _before(_from(a, z * x, h0), h0)[:, ::CHUNK].contiguous()


def _plain_scan_forward(case, s):
    at, valid = _order(case, s["lengths"])
    a, z, x = _scan_coefficients(case, s)
    h = _from(a, z * x, s["h0"])
    out = {"h": _ordered(torch.where(valid, h, 0.0), at).to(TYPES[case["out"]]), "final": h[:, -1]}
    if case["states"]:
        out["states"] = _before(h, s["h0"])[:, ::CHUNK].contiguous()
    return out


def _plain_scan_backward(case, s):
    at, valid = _order(case, s["lengths"])
    a, z, x = _scan_coefficients(case, s)
    before = _before(_from(a, z * x, s["h0"]), s["h0"])
    dh = torch.where(valid, _ordered(s["dh"].float(), at), 0.0)
    # D_i = dh_i + a_{i+1} D_{i+1}, the last with the final state's gradient.
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    D = _from(later.flip(1), dh.flip(1), s["dfinal"]).flip(1)
    dx = z * D
    dg = (a * z * (before - x) if case["gate"] == "sigmoid" else before) * D
    t = TYPES[case["grad"]]
    return {"dx": _ordered(torch.where(valid, dx, 0.0), at).to(t),
            "dg": _ordered(torch.where(valid, dg, 0.0), at).to(t), "dh0": a[:, 0] * D[:, 0]}


def _rows(x):
    """[B, H, N, d] as rows [B, N, H d]."""
    B, H, N, d = x.shape
    return x.permute(0, 2, 1, 3).reshape(B, N, H * d)


def _heads(t, case):
    """Rows [B, N, H d] as [B, H, N, d]."""
    B, N, _ = t.shape
    return t.reshape(B, N, case["heads"], case["head_dim"]).permute(0, 2, 1, 3).contiguous()


def _plain_norm_forward(case, s):
    v = _rows(s["x"].float())
    if s["residual"] is not None:
        v = v + s["residual"].float()
    rstd = 1 / torch.sqrt(v.square().mean(-1) + 1e-6)
    y = v * rstd[..., None] * s["weight"]
    out = {"sum": v.to(TYPES[case["res"]]), "rstd": rstd}
    if case["out"] != "f8":
        return dict(out, y=y.to(TYPES[case["out"]]))
    parts = y.reshape(*y.shape[:2], -1, case["group"] or y.shape[-1])
    scale = parts.abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (parts / scale[..., None]).to(TYPES["f8"]).reshape(y.shape)
    return dict(out, y=q, scales=scale)


def _plain_norm_backward(case, s):
    xh = s["sum"].float() * s["rstd"][..., None]
    dy = s["dy"].float()
    t = dy * s["weight"]
    d = s["rstd"][..., None] * (t - xh * (t * xh).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        d = d + s["dsum"].float()
    d = d.to(TYPES[case["grad"]])
    # A sum over all rows: in 64 bits.
    dweight = (dy * xh).sum((0, 1), dtype=torch.float64).float()
    return {"dx": _heads(d, case), "dres": d, "dweight": dweight}


def _plain_clip(case, s):
    total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    if case["op"] == "norm":
        return {"norm": total.float()}
    scale = torch.where(total > s["max_norm"], s["max_norm"] / total, 1.0)
    return {"norm": total.float(),
            "grads": [(g.float() * scale.float()).to(g.dtype) for g in s["grads"]]}


# ---- the library's kernels ---------------------------------------------------------------


def _own_scan_forward(case, s):
    S, N, C = case["sequences"], case["tokens"], case["channels"]
    final = torch.empty((S, C), device="cuda")
    states = torch.empty((S, -(-N // CHUNK), C), device="cuda") if case["states"] else None
    h = s["plan"].forward(s["x"], s["g"], h0=s["h0"], lengths=s["lengths"], states=states,
                          final=final)
    return {"h": h, "final": final, **({"states": states} if case["states"] else {})}


def _own_scan_backward(case, s):
    C = case["channels"]
    grads = {}
    if case["packed"]:
        # The gradients side by side too, as the projection's backward takes them.
        per = 16 // BYTES[case["dtype"]]
        half = -(-C // per) * per
        both = torch.empty((case["sequences"], case["tokens"], 2 * half),
                           dtype=TYPES[case["grad"]], device="cuda")
        grads = {"dx": both[..., :C], "dg": both[..., half:half + C]}
    dx, dg, dh0 = s["plan"].backward(s["x"], s["g"], s["states"], s["dh"], dfinal=s["dfinal"],
                                     lengths=s["lengths"], grads=grads)
    return {"dx": dx, "dg": dg, "dh0": dh0}


def _own_norm_forward(case, s):
    rows = (case["batch"], case["tokens"])
    width = case["heads"] * case["head_dim"]
    total = torch.empty((*rows, width), dtype=TYPES[case["res"]], device="cuda")
    rstd = torch.empty(rows, device="cuda")
    y = s["plan"].forward(s["x"], s["weight"], residual=s["residual"], sum=total, rstd=rstd)
    if case["out"] == "f8":
        return {"sum": total, "rstd": rstd, "y": y[0], "scales": y[1]}
    return {"sum": total, "rstd": rstd, "y": y}


def _own_norm_backward(case, s):
    dx, dres, dweight = s["plan"].backward(s["sum"], s["rstd"], s["weight"], s["dy"],
                                           dsum=s["dsum"])
    return {"dx": dx, "dres": dres, "dweight": dweight}


def _own_clip(case, s):
    if case["op"] == "norm":
        return {"norm": s["plan"].norm(s["grads"])}
    outs = [torch.empty_like(g) for g in s["grads"]]
    norm = s["plan"].clip(s["grads"], s["max_norm"], outs=outs)
    return {"norm": norm, "grads": outs}


def run(state):
    case = state["case"]
    if own:
        form = {"scan_forward": _own_scan_forward, "scan_backward": _own_scan_backward,
                "norm_forward": _own_norm_forward, "norm_backward": _own_norm_backward}
        return form.get(case["op"], _own_clip)(case, state)
    form = {"scan_forward": _plain_scan_forward, "scan_backward": _plain_scan_backward,
            "norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward}
    return form.get(case["op"], _plain_clip)(case, state)


# ---- work --------------------------------------------------------------------------------


def work(case):
    if case["op"].startswith("scan"):
        rows = case["sequences"] * case["tokens"]
        n = rows * case["channels"]
        kept = case["sequences"] * -(-case["tokens"] // CHUNK) * case["channels"] * 4
        ends = 4 * case["sequences"] * case["channels"]
        i, o, g = BYTES[case["dtype"]], BYTES[case["out"]], BYTES[case["grad"]]
        if case["op"] == "scan_forward":
            return {"bytes": n * (2 * i + o) + kept * case["states"] + ends * (1 + case["h0"]),
                    "flops": 8 * n}
        return {"bytes": n * (2 * i + 3 * g) + kept + ends * (1 + case["h0"]), "flops": 16 * n}
    if case["op"].startswith("norm_"):
        rows = case["batch"] * case["tokens"]
        width = case["heads"] * case["head_dim"]
        n, r, g = rows * width, BYTES[case["res"]], BYTES[case["grad"]]
        if case["op"] == "norm_forward":
            scales = 0 if case["out"] != "f8" else 4 * (n // (case["group"] or width))
            return {"bytes": n * (BYTES[case["x"]] + r * (1 + case["residual"])
                                  + BYTES[case["out"]]) + 4 * (rows + width) + scales,
                    "flops": 6 * n}
        return {"bytes": n * (r + g * (3 + case["dsum"])) + 4 * (rows + 2 * width),
                "flops": 12 * n}
    n = sum(k * BYTES[t] for k, t in zip(_sizes(case), _kinds(case)))
    return {"bytes": n * (2 if case["op"] == "clip" else 1), "flops": 2 * sum(_sizes(case))}


# ---- in 64 bits --------------------------------------------------------------------------


def _exact_scan(case, s):
    """One token after another."""
    S, N, C = case["sequences"], case["tokens"], case["channels"]
    lens = [N] * S if s["lengths"] is None else s["lengths"].tolist()

    def turned(t):
        """Each sequence's tokens last to first, or as they are; the padding stays."""
        t = t.double()
        if case["reverse"]:
            t = torch.stack([torch.cat([t[k, :n].flip(0), t[k, n:]]) for k, n in enumerate(lens)])
        return t

    live = torch.tensor(lens, device="cuda")[:, None] > torch.arange(N, device="cuda")
    x, g, live = turned(s["x"]), turned(s["g"]), live[..., None]
    a = torch.sigmoid(g) if case["gate"] == "sigmoid" else g
    z = torch.sigmoid(-g) if case["gate"] == "sigmoid" else torch.ones_like(g)
    h = torch.zeros((S, C), dtype=torch.float64, device="cuda")
    h = h if s["h0"] is None else s["h0"].double()
    before = torch.empty((S, N, C), dtype=torch.float64, device="cuda")
    after = torch.empty_like(before)
    b = z * x
    for i in range(N):
        before[:, i] = h
        h = torch.where(live[:, i], torch.addcmul(b[:, i], a[:, i], h), h)
        after[:, i] = h
    if case["op"] == "scan_forward":
        got = {"h": turned(after * live), "final": h}
        if case["states"]:
            got["states"] = before[:, ::CHUNK].contiguous()
        return got
    dh = torch.where(live, turned(s["dh"]), 0.0)
    into = torch.zeros((S, C), dtype=torch.float64, device="cuda")
    into = into if s["dfinal"] is None else s["dfinal"].double()
    here = torch.empty_like(before)
    for i in reversed(range(N)):
        here[:, i] = into + dh[:, i]
        into = torch.where(live[:, i], a[:, i] * here[:, i], into)
    slope = a * z * (before - x) if case["gate"] == "sigmoid" else before
    return {"dx": turned(torch.where(live, z * here, 0.0)),
            "dg": turned(torch.where(live, slope * here, 0.0)), "dh0": into}


def _exact_norm(case, s):
    B, H, N, d = case["batch"], case["heads"], case["tokens"], case["head_dim"]
    w = s["weight"].double()
    if case["op"] == "norm_forward":
        v = torch.cat([s["x"][:, h].double() for h in range(H)], -1)
        if s["residual"] is not None:
            v += s["residual"].double()
        power = torch.linalg.vector_norm(v, dim=-1) ** 2 / (H * d) + 1e-6
        y = v * w / power.sqrt()[..., None]
        got = {"sum": v, "rstd": power ** -0.5}
        if case["out"] != "f8":
            return dict(got, y=y)
        group = case["group"] or H * d
        top = y.unflatten(-1, (-1, group)).abs().max(-1).values
        scale = torch.maximum(top, torch.full_like(top, AMAX_FLOOR)) / E4M3_MAX
        q = y / scale.repeat_interleave(group, -1)
        return dict(got, y=q.float().to(TYPES["f8"]).double(), scales=scale)
    v, r = s["sum"].double(), s["rstd"].double()[..., None]
    dy = s["dy"].double()
    inner = torch.linalg.vecdot(dy * w, v * r) / (H * d)
    out = r * (dy * w) - r * r * v * inner[..., None]
    if s["dsum"] is not None:
        out += s["dsum"].double()
    dx = torch.stack(out.split(d, -1), 1)
    return {"dx": dx, "dres": out, "dweight": torch.einsum("bnw,bnw->w", dy, v * r)}


def _exact_clip(case, s):
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2
                               for g in s["grads"]))
    got = {"norm": torch.tensor(norm, dtype=torch.float64)}
    if case["op"] == "clip":
        scale = min(1.0, s["max_norm"] / norm)
        got["grads"] = [g.double() * scale for g in s["grads"]]
    return got


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"].startswith("scan"):
        return _exact_scan(case, s)
    if case["op"].startswith("norm_"):
        return _exact_norm(case, s)
    return _exact_clip(case, s)
