"""64-bit references of lapl_rope_*, lapl_decay_* and lapl_adamw_*, written from their formulas, each
value with a bound of the kernels' rounding.

U is fp32's unit of rounding.  Bounds are relative to sums of absolute values, so that cancellation
cannot hide a rounding, and count worst cases.
"""
from __future__ import annotations

import numpy as np
import torch

from operators_reference import HALF, U

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def check(name, got, want, dtype="f32"):
    """|got - value| within the bound and the rounding to dtype, everywhere; NaN is not."""
    value, bound = want
    got = got.detach().double().cpu().numpy()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    # Below the normal range a rounding is off by half of the smallest step, 2^-150 or 2^-134.
    least = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133}[dtype]
    tol = bound + HALF[dtype] * (np.abs(value) + bound) + least
    bad = ~(np.abs(got - value) <= tol)
    if bad.any():
        at = tuple(int(i) for i in np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} values off, first at {at}: "
                             f"{got[at]} for {value[at]}, tolerance {tol[at]}")


# ---- linear attention with decays ----------------------------------------------------------

def decay(q, k, v, log_decay, scale, state=None, lens=None, reverse=False, dout=None, dfinal=None,
          tensor_cores=False):
    """dict of (value, bound): out, final, and with dout dq, dk, dv, dstate.

    Sa is the state with absolute values throughout, in double like the state itself.
    Token by token: a step rounds once (a fused multiply-add), the decay's factors (powers of 2 with
    2 units of error and half a unit of an argument of up to 16 steps' decay) and the state's once for
    each 16 tokens: 16 U Sa a step, carried on as the state is.  An output sums key_dim products in
    fp32: key_dim + 16 roundings of |q| Sa.
    On the tensor cores also: P and S in two bf16 parts leave out 2^-18 = 64 U of each, Z' in three
    less than U; a sum of 24 products of 16 terms in tensor memory cuts each of them off at up to
    4 U of the sum so far, 96 U, and its decays' powers add 8 units and half a unit of an argument of at most
    149 before the product vanishes in fp32 (2 of them: 150 U, times ln 2); 512 U in all, of |q| Sa and of Sa."""
    B, H, N, a = q.shape
    lens = [N] * B if lens is None else [min(max(int(n), 0), N) for n in lens]
    flat = 512 * U if tensor_cores else 16 * U

    def turn(t, other=False):
        t = np.array(t, np.float64)
        if bool(reverse) != other:
            for b, n in enumerate(lens):
                t[b, :, :n] = t[b, :, :n][:, ::-1].copy()
        return t

    def one_way(x, y, z, first, by, z_by, other, late):
        """Outputs and the state of one pass; late: its first token does not decay the state."""
        x, y, z = turn(x, other), turn(y, other), turn(z, other)
        S = np.zeros((B, H, y.shape[-1], z.shape[-1])) if first is None else np.array(first)
        Sa, E = np.abs(S), np.zeros_like(S)
        g = np.exp(np.maximum(np.minimum(log_decay, 0), -1e30))[None, :, None, None]
        o = np.zeros((*x.shape[:3], z.shape[-1]))
        e = np.zeros_like(o)
        for i in range(N):
            live = (np.asarray(lens) > i)[:, None, None, None]
            f = np.where(live, 1.0 if late and i == 0 else g, 1.0)
            add = np.where(live, np.where(live, y[:, :, i, :, None], 0) *
                           np.where(live, z[:, :, i, None], 0) * z_by, 0.0)
            S, Sa = f * S + add, f * Sa + np.abs(add)
            E = f * E + np.where(live, 16 * U * Sa, 0.0)
            xi = np.where(live[..., 0], x[:, :, i], 0.0)
            o[:, :, i] = by * np.einsum("bha,bhac->bhc", xi, S)
            xa = np.abs(xi)
            e[:, :, i] = abs(by) * (np.einsum("bha,bhac->bhc", xa, E) + (flat + (x.shape[-1] + 16) * U)
                                    * np.einsum("bha,bhac->bhc", xa, Sa))
        return (turn(o, other), turn(e, other)), (S, E + flat * Sa)

    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        got = {}
        got["out"], got["final"] = one_way(q, k, v, state, scale, 1.0, False, False)
        if dout is None:
            return got
        across = lambda t: None if t is None else np.swapaxes(t, -1, -2)  # noqa: E731
        got["dq"], _ = one_way(dout, v, k, across(state), scale, 1.0, False, False)
        # From the last token that there is: what is read beyond it is zero either way.
        got["dk"], _ = one_way(v, dout, q, across(dfinal), 1.0, scale, True, True)
        got["dv"], (S, E) = one_way(k, q, dout, dfinal, 1.0, scale, True, True)
        g = np.exp(np.maximum(np.minimum(log_decay, 0), -1e30))[None, :, None, None]
        g = np.where(np.asarray(lens)[:, None, None, None] > 0, g, 1.0)
        got["dstate"] = (g * S, g * (E + 4 * U * np.abs(S)))
    return got


# ---- heads with a norm and rotary positions --------------------------------------------------

def _turned(x, cos, sin, interleaved, pairs):
    """x [B, H, N, d] with its pairs turned, and the sums of absolute values that each comes from."""
    y, m = x.copy(), np.abs(x)
    if pairs:
        one = np.s_[..., 0:2 * pairs:2] if interleaved else np.s_[..., :pairs]
        two = np.s_[..., 1:2 * pairs:2] if interleaved else np.s_[..., pairs:2 * pairs]
        a, b = x[one], x[two]
        y[one], y[two] = a * cos - b * sin, b * cos + a * sin
        m[one] = m[two] = np.abs(a) + np.abs(b)
    return y, m


def angles(positions, pairs, frequencies):
    """[B, 1, N, P] radians, exact in long double."""
    axis = [a for a, n in enumerate(pairs) for _ in range(n)]
    pos = np.asarray(positions).astype(np.longdouble)[..., axis]
    turn = np.longdouble("6.283185307179586476925286766559005768")
    t = pos * np.asarray(frequencies, np.longdouble)
    return np.remainder(t, turn).astype(np.float64)[:, None]


def rope(x, heads, positions, pairs, frequencies, weight=None, eps=None, interleaved=False):
    """(value, bound) of one part's outputs: rows x [B, N, heads d]; eps None: no norm.

    The mean square sums d values (d / 2 + 4 roundings of the root's reciprocal, at worst), the
    product with weights rounds three times, the turn twice, and cos and sin are off by 2 units and
    half of an angle's last bit, 2^-33 of a turn: 8 U."""
    B, N, W = x.shape
    d = W // heads
    v = np.asarray(x, np.float64).reshape(B, N, heads, d).transpose(0, 2, 1, 3)
    u = 0.0
    if eps is not None:
        v = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
        v = v * (1.0 if weight is None else weight)
        u = (d / 2 + 8) * U
    t = angles(positions, pairs, frequencies) if sum(pairs) else None
    y, m = _turned(v, None if t is None else np.cos(t), None if t is None else np.sin(t),
                   interleaved, sum(pairs))
    return y, (u + 10 * U) * m


def rope_backward(x, heads, positions, pairs, frequencies, dy, weight=None, eps=None,
                  interleaved=False):
    """(value, bound) of the rows' gradient and of the weight's (None without a norm).

    g = R^T dy: 10 U of |a| + |b| (m).  u = x rstd: (d / 2 + 8) U of itself.  The mean of t u sums d
    products: (d + d / 2 + 20) U of the mean of |t| |u|.  dweight sums rows of g u in pairs of floats: the
    terms' own errors, and one rounding."""
    B, H, N, d = dy.shape
    t = angles(positions, pairs, frequencies) if sum(pairs) else None
    cos, sin = (None, None) if t is None else (np.cos(t), -np.sin(t))
    g, m = _turned(np.asarray(dy, np.float64), cos, sin, interleaved, sum(pairs))
    rows = lambda a: a.transpose(0, 2, 1, 3).reshape(B, N, H * d)  # noqa: E731
    if eps is None:
        return (rows(g), rows(10 * U * m)), None
    v = np.asarray(x, np.float64).reshape(B, N, heads, d).transpose(0, 2, 1, 3)
    r = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    u, w = v * r, 1.0 if weight is None else weight
    eu = (d / 2 + 8) * U
    dw = (g * u).sum((0, 1, 2))
    dw_bound = ((eu + 14 * U) * (m * np.abs(u))).sum((0, 1, 2)) + U * np.abs(dw)
    gw, mw = g * w, m * np.abs(w)
    mean = (gw * u).mean(-1, keepdims=True)
    mean_bound = ((1.5 * d + 30) * U) * (mw * np.abs(u)).mean(-1, keepdims=True)
    dx = r * (gw - u * mean)
    bound = r * ((eu + 16 * U) * (mw + np.abs(u * mean)) + np.abs(u) * mean_bound)
    return (rows(dx), rows(bound)), (dw, dw_bound)


# ---- AdamW -----------------------------------------------------------------------------------

BLOCK, F8_MAX, F8_LEAST, FLOOR = 256, 448.0, 2.0 ** -9, 2.0 ** -100


def coded(x, root=False):
    """(codes before rounding, scales) of x in blocks."""
    n = x.size
    blocks = np.zeros(-(-n // BLOCK) * BLOCK)
    blocks[:n] = x
    scales = np.maximum(np.abs(blocks).reshape(-1, BLOCK).max(-1), FLOOR) / F8_MAX
    q = x / np.repeat(scales, BLOCK)[:n]
    if root:
        q = np.where(x > 0, np.maximum(q, F8_LEAST), q)
    return q, scales


def adamw(w, g, m, v, step, lr, betas, eps, wd, clip=1.0):
    """(value, bound) of w, m, v.  m and v: three roundings of each of two terms and g's own, twice in
    v: 8 U.  The update goes through m, v's root and two divisions: 24 U of itself; w rounds three
    times."""
    b1, b2 = betas
    g = g * clip
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    ma = np.abs(b1 * m) + np.abs((1 - b1) * g)
    down = np.sqrt(v1 / (1 - b2 ** step)) + eps
    up = lr * m1 / (1 - b1 ** step) / down
    upa = lr * ma / (1 - b1 ** step) / down
    w1 = w - lr * wd * w - up
    return (w1, 24 * U * upa + 4 * U * np.abs(w)), (m1, 8 * U * ma), (v1, 8 * U * v1)
