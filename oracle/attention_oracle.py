"""CPU oracle of the attention calls, in 64 bits, from their definitions.

    rotation   (a, b) at position p turns by p * f: a cos - b sin, b cos + a sin
    attention  o = sum_j softmax(scale * q.k_j)_j v_j over the keys a query sees;
               lse = ln sum_j exp(scale * q.k_j); no key seen: 0 and -infinity

Every function also returns, element by element, how far a computation with f32
sums and weights and outputs rounded to 16 bits may be from it.
"""
import numpy as np

# half a step of each type, relative; and half of its smallest subnormal step
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150, "e4m3": 2.0 ** -10}
F32 = 2.0 ** -23  # an f32 operation whose rounding may be a truncation


def rotate(x, positions, inv_freq, interleaved):
    """x [T, heads, D]; positions [T]; (rotated, tolerance of the f32 computation)."""
    x = np.asarray(x, np.float64)
    y, tol = x.copy(), np.zeros_like(x)
    f = np.asarray(inv_freq, np.float64)
    r = 2 * f.size
    if r == 0:
        return y, tol
    ang = np.asarray(positions, np.float64)[:, None] * f[None]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    ia = np.arange(0, r, 2) if interleaved else np.arange(0, r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    # the angle to 2^-32 of a turn and its f32 rounding (pi 2^-24), sine and
    # cosine to 2 units (2^-22), two products and a sum: under 2^-20 in all.
    # The 64-bit angle itself is off by half a step of its size.
    t = (np.abs(a) + np.abs(b)) * (2.0 ** -20 + np.abs(ang)[:, None] * 2.0 ** -52)
    tol[..., ia] = t
    tol[..., ib] = t
    return y, tol


def rounded_tol(value, tol, kind):
    """Tolerance after one rounding to `kind` of a value known to `tol`."""
    return tol + (np.abs(value) + tol) * HALF[kind] + TINY[kind]


def attend(q, k, v, sees, scale, kind, weights=None):
    """q [R, D], k and v [L, D], sees [R] keys (the first ones) that each row sees.
    kind: the outputs' type; weights: the type of the rounded weights (kind).
    Returns (out, out_tol, lse, lse_tol)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    weights = weights or kind
    R, D = q.shape
    out, tol = np.zeros((R, v.shape[1])), np.zeros((R, v.shape[1]))
    lse, ltol = np.full(R, -np.inf), np.zeros(R)
    for r in range(R):
        n = int(min(max(sees[r], 0), k.shape[0]))
        if n == 0:
            continue
        s = k[:n] @ q[r] * scale
        top = s.max()
        w = np.exp(s - top)
        z = w.sum()
        out[r] = w @ v[:n] / z
        spread = w @ np.abs(v[:n]) / z
        lse[r] = top + np.log(z)
        # scores: D products summed in f32, one scaling, base 2 with its rounding
        es = (D + 4) * F32 * scale * (np.abs(k[:n]) @ np.abs(q[r])).max() + 4 * F32 * np.abs(s).max()
        # sums over n keys, exponentials, the joins' factors
        es_sum = (n + 64) * F32
        tol[r] = spread * (HALF[weights] + 2 * es + 2 * es_sum)
        if weights == "f16":  # subnormal weights: half a step of 2^-24, 2^8 below the largest
            tol[r] += n * 2.0 ** -33 * np.abs(v[:n]).max(0)
        tol[r] = rounded_tol(out[r], tol[r], kind)
        ltol[r] = es + es_sum + 4 * F32 * (1 + abs(lse[r]))
    return out, tol, lse, ltol
