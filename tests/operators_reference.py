"""64-bit references of the operators of include/lapl_ops.h, written from their formulas, with a
bound of the fp32 kernels' rounding for every value.

U is fp32's unit of rounding.  The bounds count, for each output, the roundings that its value goes
through, each at most U relative to the magnitudes that it acts on (sums of absolute values, so that
cancellation cannot hide one); HALF[t] is the rounding to an output type.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f8": 2.0 ** -4}


def rounded(x, dtype):
    """x as float64, rounded to dtype."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64))
    return t.to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype]).double().numpy()


def _turned(t, lens, reverse):
    """Each sequence's tokens in processing order (its own inverse)."""
    t = np.array(t, dtype=np.float64)
    if reverse:
        for s, n in enumerate(lens):
            t[s, :n] = t[s, :n][::-1].copy()
    return t


def scan(x, g, gate, h0=None, lens=None, reverse=False, dout=None, dfinal=None):
    """dict of (value, bound): h, final, states, and with dout dx, dg, dh0.

    A step rounds its product and sum (2), the sigmoid gate rounds x - h (1) and its z is off by at
    most 4 (expf 2, the sum 1/2, the division 1, rounded up); the same step is taken a second time
    as a map, whose two parts round alike, and each composition of maps adds 2.  That is at most 16
    roundings for each step, relative to |h_{i-1}| + |b_i| with absolute values carried through the
    recurrence (H); errors decay as the state does.

    Backward the sigmoid gate's decay is 1 - z, too: with z (1 + t), |t| <= 4 U, in its place
    E = (1 - z) D is off by t z D, which is 4 U of z D and not of E: where a = 1 - z is small, more
    than any number of roundings of a D.  8 U z |D| is added to E's bound for that, and, as
    dg = z slope E, z |slope| times it to dg's."""
    S, N, C = x.shape
    lens = [N] * S if lens is None else [int(min(max(n, 0), N)) for n in lens]
    x, g = _turned(x, lens, reverse), _turned(g, lens, reverse)
    live = (np.asarray(lens)[:, None] > np.arange(N))[..., None]
    with np.errstate(over="ignore"):
        a = 1 / (1 + np.exp(-g)) if gate == "sigmoid" else g
        z = 1 / (1 + np.exp(g)) if gate == "sigmoid" else np.ones_like(g)
    a, z, x = np.where(live, a, 1.0), np.where(live, z, 0.0), np.where(live, x, 0.0)
    b = z * x
    h = np.zeros((S, C)) if h0 is None else np.array(h0, np.float64)
    H, E = np.abs(h), np.zeros((S, C))
    before, eb, after, ea, Hb = (np.empty((S, N, C)) for _ in range(5))
    for i in range(N):
        before[:, i], eb[:, i], Hb[:, i] = h, E, H
        E = np.abs(a[:, i]) * E + np.where(live[:, i], 16 * U * (H + np.abs(b[:, i])), 0.0)
        H = np.abs(a[:, i]) * H + np.abs(b[:, i])
        h = a[:, i] * h + b[:, i]
        after[:, i], ea[:, i] = h, E
    out = {"h": (_turned(after * live, lens, reverse), _turned(ea * live, lens, reverse)),
           "final": (h, E), "states": (before[:, ::16], eb[:, ::16])}
    if dout is None:
        return out
    dh = np.where(live, _turned(dout, lens, reverse), 0.0)
    D = np.zeros((S, C)) if dfinal is None else np.array(dfinal, np.float64)
    M, ED = np.abs(D), np.zeros((S, C))          # magnitude and error of what enters from later
    dx, dg, ex, eg = (np.zeros((S, N, C)) for _ in range(4))
    for i in reversed(range(N)):
        here, mag = D + dh[:, i], M + np.abs(dh[:, i])
        eh = ED + 16 * U * mag
        dx[:, i] = z[:, i] * here
        ex[:, i] = z[:, i] * (eh + 8 * U * mag)
        if gate == "sigmoid":
            k = a[:, i] * z[:, i]
            slope, es, ms = before[:, i] - x[:, i], eb[:, i], Hb[:, i] + np.abs(x[:, i])
        else:
            k = 1.0
            slope, es, ms = before[:, i], eb[:, i], Hb[:, i]
        dg[:, i] = k * slope * here
        eg[:, i] = k * ((es + 16 * U * ms) * mag + np.abs(slope) * eh + 16 * U * ms * mag)
        ez = 8 * U * z[:, i] * mag if gate == "sigmoid" else 0.0
        eg[:, i] += z[:, i] * np.abs(slope) * ez
        keep = live[:, i]
        ED = np.where(keep, np.abs(a[:, i]) * eh + ez, ED)
        M = np.where(keep, np.abs(a[:, i]) * mag, M)
        D = np.where(keep, a[:, i] * here, D)
    for name, v, e in (("dx", dx, ex), ("dg", dg, eg)):
        out[name] = (_turned(v * live, lens, reverse), _turned(e * live, lens, reverse))
    out["dh0"] = (D, ED)
    return out


# Roundings of a row's mean of squares and its root: at most 64 sums one after the other in a
# thread and 9 + 16 between threads, half of it after the root, and the root's own 2: under 64.
ROW = 64


def norm(x, res, weight, eps, group=0, f8=False):
    """dict of (value, bound): sum, rstd, y, and for f8 scales; x: [B,H,N,d], res: [B,N,W]."""
    B, H, N, d = x.shape
    v = np.transpose(x, (0, 2, 1, 3)).reshape(B, N, H * d)
    mag = np.abs(v)
    if res is not None:
        v, mag = v + res, mag + np.abs(res)
    rstd = 1 / np.sqrt((v * v).mean(-1) + eps)
    w = np.ones(H * d) if weight is None else weight
    y = v * rstd[..., None] * w
    ey = ROW * U * np.abs(y) + 2 * U * mag * rstd[..., None] * np.abs(w)
    out = {"sum": (v, U * mag), "rstd": (rstd, ROW * U * rstd), "y": (y, ey)}
    if f8:
        g = group or H * d
        top = np.abs(y).reshape(B, N, -1, g).max(-1)
        etop = ey.reshape(B, N, -1, g).max(-1)
        out["scales"] = (np.maximum(top, 2.0 ** -100) / 448, (etop + 2 * U * top) / 448)
    return out


def norm_backward(s, rstd, weight, dy, dsum, heads):
    """dict of (value, bound): dres, dx (by heads), dweight."""
    B, N, W = s.shape
    w = np.ones(W) if weight is None else weight
    r = rstd[..., None]
    n, t = s * r, dy * w
    mean = (t * n).mean(-1, keepdims=True)
    amean = np.abs(t * n).mean(-1, keepdims=True)
    v = r * (t - n * mean)
    e = ROW * U * r * (np.abs(t) + np.abs(n) * amean)
    if dsum is not None:
        v = v + dsum
        e = e + 2 * U * np.abs(dsum)
    by_head = [np.stack(np.split(a, heads, axis=-1), 1) for a in (v, e)]
    # Each column's sum: a thread's rows, the CTA's (256 at most), the CTAs' (some hundreds, 8
    # chains of them): under 512 roundings one after the other at the tests' sizes.
    return {"dres": (v, e), "dx": tuple(by_head),
            "dweight": ((dy * n).sum((0, 1)), 512 * U * np.abs(dy * n).sum((0, 1)))}


def check(name, got, want, dtype="f32"):
    """Every value of `got` within the bound, and the rounding to dtype."""
    value, bound = want
    got = got.detach().double().cpu().numpy() if hasattr(got, "detach") else np.asarray(got)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    if not value.size:
        return
    tiny = 2.0 ** -126          # results below the normal range may be flushed
    tol = bound + HALF[dtype] * (np.abs(value) + bound) + tiny
    off = np.abs(got - value)
    at = np.unravel_index(np.argmax(off - tol), off.shape)
    assert np.isfinite(got).all(), name
    assert (off <= tol).all(), (name, at, got[at], value[at], tol[at])
