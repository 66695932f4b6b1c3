"""What prepares a causal block's queries and keys, mixes its tokens and updates its weights, as cases
to measure: the norm of each head with the rotary positions, linear attention with a decay for each
head, and the AdamW step over many tensors.

``run`` computes a case in plain torch operations in 32 bits where ``own`` is false, and by the
library's kernels where it is true; ``exact`` gives the same values in 64 bits.
"""
import math

import torch

own = False

#: Tokens of a chunk in the plain form of the linear attention.
CHUNK = 64
#: Values that share a scale where the AdamW step's states are held in 8 bits.
BLOCK = 256
#: Largest and smallest finite e4m3 values, and the smallest largest value a scale is made for.
E4M3_MAX, E4M3_MIN = 448.0, 2.0 ** -9
AMAX_FLOOR = 2.0 ** -100
EPS = 1e-6

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}

# ---- cases -------------------------------------------------------------------------------


def _rope(op, batch, tokens, heads, head_dim, pairs, dtype, out="", grad="", norm=True,
          interleaved=False, packed=True, far=False, name=None):
    """heads: [q, k, v]; pairs: pairs of values that each axis turns."""
    c = dict(op=op, batch=batch, tokens=tokens, q_heads=heads[0], k_heads=heads[1],
             v_heads=heads[2], head_dim=head_dim, axes=len(pairs), pairs0=pairs[0],
             pairs1=pairs[1] if len(pairs) > 1 else 0, pairs2=pairs[2] if len(pairs) > 2 else 0,
             dtype=dtype, out=out or dtype, grad=grad or dtype, norm=norm, interleaved=interleaved,
             packed=packed, far=far)
    return dict(c, name=name) if name else c


def _decay(op, batch, heads, tokens, key_dim, value_dim, dtype, out="", grad="", reverse=False,
           lengths=False, state=False, name=None):
    c = dict(op=op, batch=batch, heads=heads, tokens=tokens, key_dim=key_dim, value_dim=value_dim,
             dtype=dtype, out=out or dtype, grad=grad or dtype, reverse=reverse, lengths=lengths,
             state=state)
    return dict(c, name=name) if name else c


def _adamw(tensors, elements, kinds, bits, master=False, clip=True, flat=False, name=None):
    c = dict(op="adamw", tensors=tensors, elements=elements, kinds=kinds, bits=bits, master=master,
             clip=clip, flat=flat)
    return dict(c, name=name) if name else c


def listed():
    return [
        # One token for each of 64 sequences, far into them: generation.
        _rope("rope_forward", 64, 1, (8, 8, 8), 64, (32,), "bf16", far=True, name="rope_step_bf16"),
        # The stage-1 vision shape: 8 images of 56 x 56 tokens, 2 heads of 32 channels, turned by
        # row and column.
        _rope("rope_forward", 8, 3136, (2, 2, 2), 32, (8, 8), "f32", name="rope_fwd_stage1_f32"),
        # The high-resolution shape: 4 images of 128 x 128 tokens, 8 heads, one projection's rows.
        _rope("rope_forward", 4, 16384, (8, 8, 8), 64, (16, 16), "bf16", name="rope_fwd_hires_bf16"),
        # Its backward.
        _rope("rope_backward", 4, 16384, (8, 8, 8), 64, (16, 16), "bf16",
              name="rope_bwd_hires_bf16"),
        # Clips of frames: time, row and column, keys and values shared by query heads, odd sizes,
        # a part of each head left unturned.
        _rope("rope_backward", 3, 2731, (6, 2, 2), 90, (9, 13, 13), "f32", interleaved=True,
              packed=False, name="rope_bwd_clips_f32"),
        # One token for each of 64 sequences from the state of the one before: generation.
        _decay("decay_forward", 64, 8, 1, 64, 64, "bf16", state=True, name="decay_step_bf16"),
        # The stage-1 shape in fp32.
        _decay("decay_forward", 8, 2, 3136, 32, 32, "f32", name="decay_fwd_stage1_f32"),
        # The high-resolution shape.
        _decay("decay_forward", 4, 8, 16384, 64, 64, "bf16", name="decay_fwd_hires_bf16"),
        # The stage-2/3 shape's backward as a padded batch: 32 sequences of up to 784 tokens.
        _decay("decay_backward", 32, 4, 784, 64, 64, "bf16", lengths=True,
               name="decay_bwd_stage23_bf16"),
        # Odd sizes in fp32, from the last token to the first, between two states.
        _decay("decay_backward", 3, 5, 2047, 48, 75, "f32", reverse=True, state=True,
               name="decay_bwd_odd_f32"),
        # The weights of one small block, states in 32 bits.
        _adamw(24, 1 << 20, "f32", 32, name="adamw_block_f32"),
        # A whole model: bf16 weights with fp32 masters and fp32 vectors between them, states in
        # 8 bits.
        _adamw(60, 1 << 27, "mixed", 8, master=True, name="adamw_model_8bit"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["rope_forward", "rope_backward", "decay_forward", "decay_forward",
                       "decay_backward", "adamw"])
    dtype = rng.choice(["f32", "bf16"])
    if kind.startswith("rope"):
        head_dim = _spread(rng, 2, 256)
        if rng.random() < 0.6:
            head_dim = max(16, 16 * (head_dim // 16))
        q = rng.choice([1, 2, 4, 5, 8, 16])
        k = rng.choice([n for n in (1, 2, 4, 5, 8, 16) if q % n == 0])
        v = rng.choice([0, k])
        turned = head_dim // 2 if rng.random() < 0.7 else rng.randint(0, head_dim // 2)
        axes = rng.choice([1, 2, 3])
        pairs = (turned - (axes - 1) * (turned // axes),) + (turned // axes,) * (axes - 1)
        most = max(1, min(1 << 16, (1 << 25) // ((q + k + v) * head_dim)))
        batch = rng.choice([1, 2, 5])
        return _rope(kind, batch, max(1, _spread(rng, 1, most) // batch), (q, k, v), head_dim, pairs,
                     dtype, out=rng.choice(["f32", "bf16"]), grad=rng.choice(["f32", "bf16"]),
                     norm=rng.random() < 0.8, interleaved=rng.random() < 0.3,
                     packed=rng.random() < 0.6, far=rng.random() < 0.3)
    if kind.startswith("decay"):
        if dtype == "bf16" and rng.random() < 0.6:
            key_dim, value_dim = rng.choice([(64, 64), (32, 32), (128, 128), (64, 128)])
        else:
            key_dim, value_dim = _spread(rng, 1, 128), _spread(rng, 1, 128)
        tokens = 1 if kind == "decay_forward" and rng.random() < 0.25 else _spread(rng, 1, 32768)
        most = max(1, (1 << 30) // (tokens * key_dim * value_dim))
        heads = min(rng.choice([1, 2, 3, 8, 16]), most)
        batch = _spread(rng, 1, max(1, min(64, most // heads)))
        other = rng.choice([dtype, dtype, "f32", "bf16"])
        return _decay(kind, batch, heads, tokens, key_dim, value_dim, dtype, out=other, grad=other,
                      reverse=rng.random() < 0.3, lengths=rng.random() < 0.4,
                      state=rng.random() < 0.5)
    kinds = rng.choice(["f32", "bf16", "mixed"])
    return _adamw(_spread(rng, 1, 400), _spread(rng, 64, 1 << 26), kinds, rng.choice([8, 32]),
                  master=kinds != "f32" and rng.random() < 0.5, clip=rng.random() < 0.7,
                  flat=rng.random() < 0.4)


# ---- inputs ------------------------------------------------------------------------------


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, gen, dtype=torch.float32, scale=1.0, shift=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(scale).add_(shift).to(dtype)


def _pairs(case):
    return [case["pairs0"], case["pairs1"], case["pairs2"]][:case["axes"]]


def _frequencies(case):
    """Radians a step of each pair, each axis from 1 down to about 1e-4."""
    return [10000.0 ** (-i / n) for n in _pairs(case) for i in range(n)]


def _split(rows, case):
    """The heads' parts of rows that hold q, k and v side by side."""
    widths = [case[n] * case["head_dim"] for n in ("q_heads", "k_heads", "v_heads")]
    return dict(zip("qkv", rows.split(widths, -1)))


def _rope_inputs(case, seed):
    gen = _rng(seed)
    B, N, d = case["batch"], case["tokens"], case["head_dim"]
    width = (case["q_heads"] + case["k_heads"] + case["v_heads"]) * d
    rows = _normal((B, N, width), gen, TYPES[case["dtype"]])
    s = _split(rows, case)
    if not case["packed"]:
        s = {n: t.contiguous() for n, t in s.items()}
    if case["v_heads"] == 0:
        s["v"] = None
    # A grid's positions, or places anywhere in long sequences.
    side = max(1, int(math.isqrt(N)))
    n = torch.arange(N, device="cuda")
    grid = torch.stack([n // (side * side), n // side, n % side], -1)[:, -case["axes"]:]
    if case["axes"] == 1:
        grid = n[:, None]
    pos = grid[None].expand(B, N, case["axes"])
    if case["far"]:
        pos = pos + torch.randint(0, 1 << 24, (B, 1, 1), generator=gen, device="cuda")
    s["positions"] = pos.to(torch.int32).contiguous()
    for n in ("q_weight", "k_weight"):
        s[n] = _normal((d,), gen, scale=0.2, shift=1.0) if case["norm"] else None
    if case["op"] == "rope_backward":
        for n, heads in (("dq", "q_heads"), ("dk", "k_heads"), ("dv", "v_heads")):
            s[n] = (_normal((B, case[heads], N, d), gen, TYPES[case["grad"]])
                    if case[heads] else None)
    return s


def _decay_inputs(case, seed):
    gen = _rng(seed)
    B, H, N, dk, dv = (case[n] for n in ("batch", "heads", "tokens", "key_dim", "value_dim"))
    t = TYPES[case["dtype"]]
    s = {"q": _normal((B, H, N, dk), gen, t), "k": _normal((B, H, N, dk), gen, t),
         "v": _normal((B, H, N, dv), gen, t)}
    # Memories of some tens of tokens in the first head to thousands in the last.
    away = torch.arange(H, device="cuda", dtype=torch.float64) * (7.0 / max(1, H - 1)) + 5.0
    s["log_decay"] = torch.log1p(-torch.exp2(-away)).float()
    s["state"] = _normal((B, H, dk, dv), gen, scale=4.0) if case["state"] else None
    s["lengths"] = None
    if case["lengths"]:
        n = torch.randint(0, N + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        n[0] = N
        s["lengths"] = n
    if case["op"] == "decay_backward":
        s["dout"] = _normal((B, H, N, dv), gen, TYPES[case["grad"]])
        s["dfinal"] = _normal((B, H, dk, dv), gen) if case["state"] else None
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


def _wd(case):
    """No decay for short vectors."""
    return [0.1 if i % 3 == 0 else 0.0 for i in range(case["tensors"])]


HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "step": 100}


def _quantised(x, at_least):
    """(codes, scales) of x in blocks of BLOCK values; at_least: of what is not zero."""
    n = x.numel()
    blocks = torch.nn.functional.pad(x, (0, -n % BLOCK)).reshape(-1, BLOCK)
    scale = blocks.abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = blocks / scale[:, None]
    if at_least:
        q = torch.where(blocks > 0, q.clamp_min(E4M3_MIN), q)
    return q.reshape(-1)[:n].to(torch.float8_e4m3fn), scale


def _joined(tensors, flat):
    """The tensors as slices of one buffer for each type, and those buffers; flat: end to end, so that
    most start anywhere."""
    parts, buffers, step = [None] * len(tensors), {}, 1 if flat else 128
    for name, t in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f8", torch.float8_e4m3fn),
                    ("f64", torch.float64)):
        mine = [i for i, x in enumerate(tensors) if x is not None and x.dtype == t]
        if not mine:
            continue
        starts = [0]
        for i in mine:
            starts.append(-(-(starts[-1] + tensors[i].numel()) // step) * step)
        buffers[name] = torch.zeros(starts[-1], dtype=t, device="cuda")
        for i, at in zip(mine, starts):
            parts[i] = buffers[name][at:at + tensors[i].numel()]
            parts[i].copy_(tensors[i])
    return parts, buffers


def _adamw_inputs(case, seed):
    gen = _rng(seed)
    sizes, kinds = _sizes(case), _kinds(case)
    weights = [_normal((n,), gen, scale=0.05) for n in sizes]
    grads = [_normal((n,), gen, TYPES[k], scale=1e-3 * (1 + i % 5))
             for i, (n, k) in enumerate(zip(sizes, kinds))]
    # What a hundred steps with such gradients leave.
    m = [_normal((n,), gen, scale=3e-4 * (1 + i % 5)) for i, n in enumerate(sizes)]
    v = [_normal((n,), gen, scale=1e-3 * (1 + i % 5)).square_() + 1e-8 for i, n in enumerate(sizes)]
    lists = {"params": [w.to(TYPES[k]) for w, k in zip(weights, kinds)], "grads": grads}
    if case["master"]:
        lists["masters"] = [w if k == "bf16" else None for w, k in zip(weights, kinds)]
    if case["bits"] == 8:
        m, v = [_quantised(x, False) for x in m], [_quantised(x.sqrt(), True) for x in v]
        lists["m_scales"], lists["v_scales"] = [x[1] for x in m], [x[1] for x in v]
        m, v = [x[0] for x in m], [x[0] for x in v]
    lists["m"], lists["v"] = m, v
    s = {"masters": None, "m_scales": None, "v_scales": None, "buffers": {}}
    for n, tensors in lists.items():
        s[n], s["buffers"][n] = _joined(tensors, case["flat"])
    about = math.sqrt(sum(n * (1e-3 * (1 + i % 5)) ** 2 for i, n in enumerate(sizes)))
    s["norm"], s["max_norm"] = None, None
    if case["clip"]:
        s["norm"] = torch.tensor(about, device="cuda", dtype=torch.float32)
        s["max_norm"] = 0.25 * about
    return s


def _inputs(case, seed):
    if case["op"].startswith("rope"):
        return _rope_inputs(case, seed)
    if case["op"].startswith("decay"):
        return _decay_inputs(case, seed)
    return _adamw_inputs(case, seed)


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if own:
        s["plan"] = _plan(case)
    return s


def _plan(case):
    import laplacian_nystr_attention_gb300 as lna
    if case["op"].startswith("rope"):
        heads = [case["q_heads"], case["k_heads"], case["v_heads"]]
        stride = sum(heads) * case["head_dim"] if case["packed"] else 0
        return lna.HeadRotary(lna.make_rope_config(
            case["batch"], case["tokens"], *heads, case["head_dim"], _pairs(case),
            _frequencies(case), norm=int(case["norm"]), eps=EPS,
            interleaved=int(case["interleaved"]), in_dtype=case["dtype"], out_dtype=case["out"],
            grad_dtype=case["grad"], q_stride=stride, k_stride=stride, v_stride=stride))
    if case["op"].startswith("decay"):
        return lna.DecayAttention(lna.make_decay_config(
            case["batch"], case["heads"], case["tokens"], case["key_dim"], case["value_dim"],
            scale=case["key_dim"] ** -0.5, reverse=int(case["reverse"]), in_dtype=case["dtype"],
            out_dtype=case["out"], grad_dtype=case["grad"]))
    return lna.AdamW(_sizes(case), _kinds(case), betas=(HYPER["beta1"], HYPER["beta2"]),
                     eps=HYPER["eps"], weight_decay=_wd(case), state_bits=case["bits"],
                     masters=case["master"])


# ---- plain forms -------------------------------------------------------------------------


def _turn(case, positions):
    """cos and sin of every token's pairs, [B, 1, N, P]; the angles in 64 bits."""
    f = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"),
                                   torch.tensor(_pairs(case), device="cuda"))
    angle = (positions.double()[..., axis] * f)[:, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotated(x, cos, sin, interleaved):
    """x [B, H, N, d] with its first 2 P values turned in pairs."""
    P = cos.shape[-1]
    rest = x[..., 2 * P:]
    if interleaved:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _heads(rows, n):
    """Rows [B, N, n d] as [B, n, N, d]."""
    return rows.reshape(*rows.shape[:2], n, -1).transpose(1, 2)


def _rows(x):
    """[B, H, N, d] as rows [B, N, H d]."""
    return x.transpose(1, 2).flatten(2)


def _plain_rope_forward(case, s):
    cos, sin = _turn(case, s["positions"])
    out = {}
    for n in "qk":
        x = _heads(s[n].float(), case[n + "_heads"])
        if case["norm"]:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * s[n + "_weight"]
        x = _rotated(x, cos, sin, case["interleaved"])
        out[n] = x.to(TYPES[case["out"]]).contiguous()
    if s["v"] is not None:
        out["v"] = _heads(s["v"], case["v_heads"]).to(TYPES[case["out"]]).contiguous()
    return out


def _plain_rope_backward(case, s):
    cos, sin = _turn(case, s["positions"])
    out, t = {}, TYPES[case["grad"]]
    for n in "qk":
        g = _rotated(s["d" + n].float(), cos, -sin, case["interleaved"])
        if case["norm"]:
            x = _heads(s[n].float(), case[n + "_heads"])
            rstd = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
            xh = x * rstd
            # A sum over all rows: in 64 bits.
            out[f"d{n}_weight"] = (g * xh).sum((0, 1, 2), dtype=torch.float64).float()
            g = g * s[n + "_weight"]
            g = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        out["d" + n] = _rows(g).to(t)
    if s["dv"] is not None:
        out["dv"] = _rows(s["dv"])
    return out


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
    return torch.stack([early, late], 2).reshape(b.shape)


def _order(case, lengths, reverse):
    """The token at each place of the processing order, [B, 1, N, 1], and where that is a token."""
    B, N = case["batch"], case["tokens"]
    i = torch.arange(N, device="cuda").expand(B, N)
    n = lengths.to(torch.int64)[:, None] if lengths is not None else torch.full_like(i[:, :1], N)
    valid = i < n
    at = torch.where(valid, n - 1 - i, i) if reverse else i
    return at[:, None, :, None], valid[:, None, :, None]


def _linear_attention(case, s, q, k, v, first, reverse):
    """(o, last): o_i = q_i S_i with S_i = g S_{i-1} + k_i v_i^T from S_{-1} = first, in chunks;
    last: the state after all tokens."""
    B, H, N = q.shape[:3]
    at, valid = _order(case, s["lengths"], reverse)
    q, k, v = (torch.where(valid, t.float().gather(2, at.expand(t.shape)), 0.0) for t in (q, k, v))
    pad = -N % CHUNK
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).reshape(B * H, -1, CHUNK, t.shape[-1])
               for t in (q, k, v))
    # Tokens of each chunk, and each token's place among them.
    count = torch.nn.functional.pad(valid[:, :, :, 0].float(), (0, pad)).reshape(B, 1, -1, CHUNK)
    count = count.expand(B, H, -1, CHUNK).reshape(B * H, -1, CHUNK).sum(-1)[..., None, None]
    rate = s["log_decay"].expand(B, H).reshape(B * H, 1, 1, 1)
    i = torch.arange(CHUNK, device="cuda", dtype=torch.float32)
    apart = i[:, None] - i
    within = torch.where(apart >= 0, torch.exp(rate * apart.clamp_min(0)), 0.0)
    local = ((q @ k.transpose(-1, -2)) * within) @ v
    late = torch.exp(rate * (count - 1 - i[:, None]).clamp_min(0))
    add = (k * late).transpose(-1, -2) @ v
    whole = torch.exp(rate * count)
    start = torch.zeros_like(add[:, :1]) if first is None else first.reshape(-1, 1, *add.shape[2:])
    add = torch.cat([whole[:, :1] * start + add[:, :1], add[:, 1:]], 1)
    after = _recur(whole, add)
    before = torch.cat([start, after[:, :-1]], 1)
    o = local + torch.exp(rate * (i[:, None] + 1)) * (q @ before)
    o = torch.where(valid, o.reshape(B, H, N + pad, -1)[:, :, :N], 0.0)
    return o.gather(2, at.expand(o.shape)), after[:, -1].reshape(B, H, *after.shape[2:])


def _plain_decay_forward(case, s):
    o, last = _linear_attention(case, s, s["q"], s["k"], s["v"], s["state"], case["reverse"])
    return {"out": (o * case["key_dim"] ** -0.5).to(TYPES[case["out"]]), "final": last}


def _plain_decay_backward(case, s):
    """The same operator with its parts exchanged: over the tokens as the forward for dq, the other
    way for dk and dv, where the final state's gradient meets its first token undecayed."""
    scale, t, r = case["key_dim"] ** -0.5, TYPES[case["grad"]], case["reverse"]
    state = None if s["state"] is None else s["state"].transpose(-1, -2)
    dq = _linear_attention(case, s, s["dout"], s["v"], s["k"], state, r)[0]
    rate = torch.exp(s["log_decay"])[:, None, None]
    first = None if s["dfinal"] is None else s["dfinal"] / (rate * scale)
    dv, last = _linear_attention(case, s, s["k"], s["q"], s["dout"], first, not r)
    first = None if first is None else first.transpose(-1, -2)
    dk = _linear_attention(case, s, s["v"], s["dout"], s["q"], first, not r)[0]
    return {**{n: (x * scale).to(t) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))},
            "dstate": last * (rate * scale)}


def _plain_adamw(case, s):
    h = HYPER
    late1, late2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    clip = 1.0
    if case["clip"]:
        clip = torch.where(s["norm"] > s["max_norm"], s["max_norm"] / s["norm"], 1.0)
    for i, wd in enumerate(_wd(case)):
        p, m, v = s["params"][i], s["m"][i], s["v"][i]
        master = s["masters"][i] if case["master"] else None
        w = p.float() if master is None else master
        g = s["grads"][i].float() * clip
        old_m, old_v = m.float(), v.float()
        if case["bits"] == 8:
            n = m.numel()
            old_m = old_m * s["m_scales"][i].repeat_interleave(BLOCK)[:n]
            old_v = (old_v * s["v_scales"][i].repeat_interleave(BLOCK)[:n]).square()
        new_m = h["beta1"] * old_m + (1 - h["beta1"]) * g
        new_v = h["beta2"] * old_v + (1 - h["beta2"]) * g * g
        step = new_m / late1 / (torch.sqrt(new_v / late2) + h["eps"])
        w = w * (1 - h["lr"] * wd) - h["lr"] * step
        p.copy_(w)
        if master is not None:
            master.copy_(w)
        if case["bits"] == 8:
            codes, scale = _quantised(new_m, False)
            m.copy_(codes)
            s["m_scales"][i].copy_(scale)
            codes, scale = _quantised(torch.sqrt(new_v), True)
            v.copy_(codes)
            s["v_scales"][i].copy_(scale)
        else:
            m.copy_(new_m)
            v.copy_(new_v)
    return _adamw_outputs(case, s)


def _adamw_outputs(case, s):
    """All buffers that the step updates."""
    return {f"{n}_{t}": b for n, of in s["buffers"].items() if n != "grads" for t, b in of.items()}


# ---- the library's kernels ---------------------------------------------------------------


def _own_rope_forward(case, s):
    q, k, v = s["plan"].forward(s["q"], s["k"], s["v"], s["positions"], s["q_weight"],
                                s["k_weight"])
    return {"q": q, "k": k, **({} if v is None else {"v": v})}


def _own_rope_backward(case, s):
    grads = {}
    if case["packed"]:
        # The gradients side by side too, as the projection's backward takes them.
        width = (case["q_heads"] + case["k_heads"] + case["v_heads"]) * case["head_dim"]
        rows = torch.empty((case["batch"], case["tokens"], width), dtype=TYPES[case["grad"]],
                           device="cuda")
        grads = {"d" + n: t for n, t in _split(rows, case).items() if case[n + "_heads"]}
    dq, dk, dv, dqw, dkw = s["plan"].backward(s["q"], s["k"], s["positions"], s["q_weight"],
                                              s["k_weight"], s["dq"], s["dk"], s["dv"], grads=grads)
    out = {}
    for n, d, w in (("q", dq, dqw), ("k", dk, dkw)):
        if case["norm"]:
            out[f"d{n}_weight"] = w
        out["d" + n] = d
    return {**out, **({} if dv is None else {"dv": dv})}


def _own_decay_forward(case, s):
    final = torch.empty((case["batch"], case["heads"], case["key_dim"], case["value_dim"]),
                        device="cuda")
    out = s["plan"].forward(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"],
                            lengths=s["lengths"], final=final)
    return {"out": out, "final": final}


def _own_decay_backward(case, s):
    dq, dk, dv, dstate = s["plan"].backward(s["q"], s["k"], s["v"], s["log_decay"], s["dout"],
                                            state=s["state"], dfinal=s["dfinal"],
                                            lengths=s["lengths"])
    return {"dq": dq, "dk": dk, "dv": dv, "dstate": dstate}


def _own_adamw(case, s):
    s["plan"].step(s["params"], s["grads"], s["m"], s["v"], HYPER["step"], HYPER["lr"],
                   m_scales=s["m_scales"], v_scales=s["v_scales"], masters=s["masters"],
                   norm=s["norm"], max_norm=s["max_norm"])
    return _adamw_outputs(case, s)


def run(state):
    case = state["case"]
    if own:
        form = {"rope_forward": _own_rope_forward, "rope_backward": _own_rope_backward,
                "decay_forward": _own_decay_forward, "decay_backward": _own_decay_backward}
        return form.get(case["op"], _own_adamw)(case, state)
    form = {"rope_forward": _plain_rope_forward, "rope_backward": _plain_rope_backward,
            "decay_forward": _plain_decay_forward, "decay_backward": _plain_decay_backward}
    return form.get(case["op"], _plain_adamw)(case, state)


# ---- work --------------------------------------------------------------------------------


def work(case):
    if case["op"].startswith("rope"):
        rows = case["batch"] * case["tokens"]
        heads = case["q_heads"] + case["k_heads"]
        n, v = rows * heads * case["head_dim"], rows * case["v_heads"] * case["head_dim"]
        i, o, g = BYTES[case["dtype"]], BYTES[case["out"]], BYTES[case["grad"]]
        pos = 4 * rows * case["axes"]
        if case["op"] == "rope_forward":
            return {"bytes": (n + v) * (i + o) + pos, "flops": 10 * n}
        return {"bytes": n * (i * case["norm"] + 2 * g) + 2 * v * g + pos, "flops": 20 * n}
    if case["op"].startswith("decay"):
        B, H, N, dk, dv = (case[n] for n in ("batch", "heads", "tokens", "key_dim", "value_dim"))
        rows, kept = B * H * N, 4 * B * H * dk * dv
        i, o, g = BYTES[case["dtype"]], BYTES[case["out"]], BYTES[case["grad"]]
        if case["op"] == "decay_forward":
            return {"bytes": rows * (i * (2 * dk + dv) + o * dv) + kept * (1 + case["state"]),
                    "flops": 4 * rows * dk * dv}
        return {"bytes": rows * (i * (2 * dk + dv) + g * (2 * dk + 2 * dv))
                + kept * (1 + 2 * case["state"]), "flops": 10 * rows * dk * dv}
    total = 0
    for n, k in zip(_sizes(case), _kinds(case)):
        weight = (2 + 8 if case["master"] else 4) if k == "bf16" else 8
        states = 16 if case["bits"] == 32 else 4
        total += n * (weight + BYTES[k] + states)
        if case["bits"] == 8:
            total += 16 * -(-n // BLOCK)
    return {"bytes": total, "flops": 15 * sum(_sizes(case))}


# ---- in 64 bits --------------------------------------------------------------------------


def _exact_rope(case, s):
    """Pairs as complex numbers; gradients by differentiating that."""
    d, pairs = case["head_dim"], sum(_pairs(case))
    axis = [a for a, n in enumerate(_pairs(case)) for _ in range(n)]
    turns = [s["positions"][..., a].double() * f for a, f in zip(axis, _frequencies(case))]
    angle = torch.stack(turns, -1) if turns else s["positions"].double()[..., :0]
    turn = torch.polar(torch.ones_like(angle), angle)[:, :, None]

    def form(rows, weight, heads):
        x = rows.unflatten(-1, (heads, d))
        if case["norm"]:
            power = torch.linalg.vecdot(x, x)[..., None] / d + EPS
            x = x * weight * power ** -0.5
        if pairs:
            step = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if case["interleaved"] else \
                (slice(0, pairs), slice(pairs, 2 * pairs))
            z = torch.complex(x[..., step[0]], x[..., step[1]]) * turn
            both = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2)
            x = torch.cat([both.flatten(-2), x[..., 2 * pairs:]], -1)
        return x.permute(0, 2, 1, 3)

    out = {}
    for n in "qk":
        rows, weight = s[n].double(), s[n + "_weight"]
        weight = None if weight is None else weight.double()
        if case["op"] == "rope_forward":
            out[n] = form(rows, weight, case[n + "_heads"])
            continue
        leaves = [t.detach().requires_grad_() for t in (rows, weight) if t is not None]
        with torch.enable_grad():
            y = form(leaves[0], leaves[-1], case[n + "_heads"])
        got = torch.autograd.grad(y, leaves, s["d" + n].double())
        if case["norm"]:
            out[f"d{n}_weight"] = got[1]
        out["d" + n] = got[0]
    if s["v"] is not None and case["op"] == "rope_forward":
        out["v"] = s["v"].double().unflatten(-1, (-1, d)).permute(0, 2, 1, 3)
    if case["op"] == "rope_backward" and s["dv"] is not None:
        out["dv"] = s["dv"].double().permute(0, 2, 1, 3).flatten(2)
    return out


def _exact_decay(case, s):
    """One token after another, and back."""
    B, H, N, dk, dv = (case[n] for n in ("batch", "heads", "tokens", "key_dim", "value_dim"))
    if N * (1 if case["op"] == "decay_forward" else 3) > 100000:
        return None
    lens = [N] * B if s["lengths"] is None else s["lengths"].tolist()

    def turned(t):
        """Each sequence's tokens last to first, or as they are; the padding stays."""
        t = t.double()
        if not case["reverse"]:
            return t
        return torch.stack([torch.cat([t[b, :, :n].flip(1), t[b, :, n:]], 1)
                            for b, n in enumerate(lens)])

    scale, g = dk ** -0.5, torch.exp(s["log_decay"].double())[:, None, None]
    live = torch.tensor(lens, device="cuda")[:, None] > torch.arange(N, device="cuda")
    q, k, v = (turned(s[n]) for n in "qkv")
    S = torch.zeros((B, H, dk, dv), dtype=torch.float64, device="cuda")
    S = S if s["state"] is None else s["state"].double()
    on = live[:, None, :, None].double()
    k, v = torch.where(on > 0, k, 0.0), torch.where(on > 0, v, 0.0)
    rate = torch.where(live[:, None, :, None, None], g[None, :, None], 1.0)
    if case["op"] == "decay_forward":
        o = torch.empty((B, H, N, dv), dtype=torch.float64, device="cuda")
        for i in range(N):
            S = torch.addcmul(rate[:, :, i] * S, k[:, :, i, :, None], v[:, :, i, None])
            o[:, :, i] = (q[:, :, i, None] @ S)[:, :, 0]
        return {"out": turned(o * on) * scale, "final": S}
    do = torch.where(on > 0, turned(s["dout"]), 0.0) * scale
    q = torch.where(on > 0, q, 0.0)
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for i in range(N):
        S = torch.addcmul(rate[:, :, i] * S, k[:, :, i, :, None], v[:, :, i, None])
        dq[:, :, i] = (S @ do[:, :, i, :, None])[..., 0]
    D = torch.zeros_like(S) if s["dfinal"] is None else s["dfinal"].double()
    for i in reversed(range(N)):
        D = torch.addcmul(D, q[:, :, i, :, None], do[:, :, i, None])
        dk_[:, :, i] = (D @ v[:, :, i, :, None])[..., 0]
        dv_[:, :, i] = (k[:, :, i, None] @ D)[:, :, 0]
        D = rate[:, :, i] * D
    return {"dq": turned(dq * on), "dk": turned(dk_ * on), "dv": turned(dv_ * on), "dstate": D}


def _exact_adamw(case, s):
    h, kinds = HYPER, _kinds(case)
    got = {n: [] for n in s["buffers"] if n != "grads"}
    clip = min(1.0, s["max_norm"] / float(s["norm"])) if case["clip"] else 1.0

    def held(x, scales):
        x = x.double()
        if scales is None:
            return x
        return x * scales.double()[torch.arange(x.numel(), device="cuda") // BLOCK]

    def coded(x, root):
        rows = x.new_zeros(-(-x.numel() // BLOCK), BLOCK)
        rows.view(-1)[:x.numel()] = x
        tops = torch.maximum(rows.max(1).values, -rows.min(1).values)
        tops = torch.where(tops > AMAX_FLOOR, tops, AMAX_FLOOR) / E4M3_MAX
        codes = x / tops.repeat_interleave(BLOCK)[:x.numel()]
        if root:
            codes[(x > 0) & (codes < E4M3_MIN)] = E4M3_MIN
        return codes.float().to(torch.float8_e4m3fn).double(), tops

    for i, wd in enumerate(_wd(case)):
        master = s["masters"][i] if case["master"] else None
        w = (s["params"][i] if master is None else master).double()
        m = held(s["m"][i], s["m_scales"][i] if case["bits"] == 8 else None)
        v = held(s["v"][i], s["v_scales"][i] if case["bits"] == 8 else None)
        v = v.square() if case["bits"] == 8 else v
        g = s["grads"][i].double() * clip
        m = torch.lerp(g, m, h["beta1"])
        v = torch.lerp(g.square(), v, h["beta2"])
        up = m / (1 - h["beta1"] ** h["step"])
        down = (v / (1 - h["beta2"] ** h["step"])).sqrt() + h["eps"]
        w = w - h["lr"] * (up / down + wd * w)
        got["params"].append(w)
        if case["master"]:
            got["masters"].append(None if master is None else w)
        if case["bits"] == 8:
            for n, x, root in (("m", m, False), ("v", v.sqrt(), True)):
                codes, tops = coded(x, root)
                got[n].append(codes)
                got[n + "_scales"].append(tops)
        else:
            got["m"].append(m)
            got["v"].append(v)
    out = {}
    for n, tensors in got.items():
        for t in s["buffers"][n]:
            # The parameters' two types apart, as their buffers are.
            own_type = [None if x is None or (n == "params" and k != t) else x
                        for x, k in zip(tensors, kinds)]
            out[f"{n}_{t}"] = _joined(own_type, case["flat"])[1]["f64"]
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"].startswith("rope"):
        return _exact_rope(case, s)
    if case["op"].startswith("decay"):
        return _exact_decay(case, s)
    return _exact_adamw(case, s)
