"""References of the 8-bit rows, norms and 8-bit products, in numpy float64 and
apart from the kernels' order of work, with the error that each result may have.

A rounding is off by at most half a step: float32 U = 2^-24 relative, ``half`` of
the others (bf16 2^-8, fp16 2^-11)."""
import numpy as np
import torch
from scipy.special import erfc

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half(dtype):
    """Half a step of a type, relative to the value."""
    return float(torch.finfo(TYPES[dtype]).eps) / 2


def floor(dtype):
    """Half a step of its subnormal numbers."""
    f = torch.finfo(TYPES[dtype])
    return float(f.tiny) * float(f.eps) / 2


def rounded(y, err, dtype):
    """The error of y, known within err, after its rounding to dtype."""
    return err + half(dtype) * (np.abs(y) + err) + floor(dtype)


def rows8(x, s=None):
    """Codes and steps of float32 rows, every operation rounded to float32."""
    x = np.asarray(x, np.float32)
    if s is not None:
        x = x * np.asarray(s, np.float32)
    with np.errstate(all="ignore"):
        m = np.abs(x).max(1)
        bad = ~np.isfinite(x).all(1)
        m = np.maximum(np.where(bad, np.float32(1), m), np.float32(2.0 ** -100))
        codes = np.rint(x * (np.float32(127) / m)[:, None])
        codes = np.where(bad[:, None], 0, codes).astype(np.int8)
        steps = np.where(bad, np.float32(np.nan), m / np.float32(127)).astype(np.float32)
    return codes, steps


def norm(x, gamma, beta, eps, rms):
    """y, (mean, r) and the errors of y, mean and r (before an output's rounding).

    A lane adds at most 32 values, a row's lanes meet in 6 + 16 more sums: 64
    roundings bound any sum. The mean is off by at most 64·U·mean|x| = dm. The
    squares are taken around that mean, which adds dm² to their mean: r is off
    by (64 + 8)/2·U + dm²·r²/2 relative, taken as 80·U + dm²·r²."""
    x, gamma = np.asarray(x, np.float64), np.asarray(gamma, np.float64)
    n = x.shape[1]
    mean = np.zeros((len(x), 1)) if rms else x.mean(1, keepdims=True)
    r = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    y0 = (x - mean) * r * gamma
    y = y0 if beta is None else y0 + np.asarray(beta, np.float64)
    dm = 0.0 if rms else 66 * U * np.abs(x).mean(1, keepdims=True)
    dr = 80 * U + dm ** 2 * r ** 2
    err = np.abs(gamma) * r * dm + np.abs(y0) * (dr + 4 * U) + 2 * U * np.abs(y)
    return y, (mean[:, 0], r[:, 0]), err, (dm + np.zeros((len(x), 1)))[:, 0], (r * dr)[:, 0]


def norm_back(dy, x, stats, gamma, rms):
    """dx, dgamma, dbeta and their errors. Row sums as in norm(). A column's
    sum takes T / 256 rows in a group, 64 groups, 64 / 4 parts and the rest."""
    dy, x, gamma = (np.asarray(a, np.float64) for a in (dy, x, gamma))
    mean, r = (np.asarray(stats, np.float64)[:, i:i + 1] for i in (0, 1))
    if rms:
        mean = np.zeros_like(mean)
    xh = (x - mean) * r
    d = dy * gamma
    c1 = 0.0 if rms else d.mean(1, keepdims=True)
    c2 = (d * xh).mean(1, keepdims=True)
    dx = r * (d - c1 - xh * c2)
    e1 = 0.0 if rms else 70 * U * np.abs(d).mean(1, keepdims=True)
    e2 = 74 * U * np.abs(d * xh).mean(1, keepdims=True)
    edx = r * (e1 + np.abs(xh) * e2 + 6 * U * (np.abs(d) + np.abs(c1) + np.abs(xh * c2)))
    depth = (len(x) / 256 + 96) * U
    return (dx, (dy * xh).sum(0), dy.sum(0), edx, (depth + 4 * U) * np.abs(dy * xh).sum(0),
            depth * np.abs(dy).sum(0))


def matmul(a, b):
    """a·b in float64, on the GPU where it is large."""
    if a.shape[0] * a.shape[1] * b.shape[1] > 1 << 30 and torch.cuda.is_available():
        return (torch.from_numpy(a).cuda() @ torch.from_numpy(np.ascontiguousarray(b)).cuda()).cpu().numpy()
    return a @ b


def product(codes, steps, q, w, bias=None):
    """Y and its error: the sum's rounding, two products, the bias."""
    # int8 products in float64 are exact
    s = matmul(np.asarray(codes, np.float64), np.asarray(q, np.float64).T)
    y = s * np.asarray(steps, np.float64)[:, None] * np.asarray(w, np.float64)
    err = 3 * U * np.abs(y)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
        err = err + U * (np.abs(y) + err)
    return y, err


def act(g, kind):
    """act(g), act'(g) and the error of each with g exact.

    silu: the exponent's argument is off by 2·U·|g|, exp, sum and reciprocal add
    5·U: sigmoid within (2|g| + 5)·U of itself. gelu: Φ's tail is exp(-g²/2),
    whose argument is off by 3·U·g²/2, times a fit within 2^-22.5 whose nine steps
    add less than 2·U each, at most 40·U in all."""
    if kind == "silu":
        s = 1 / (1 + np.exp(-g))
        rel = (2 * np.abs(g) + 8) * U
        slope = s * (1 + g * (1 - s))
        return (g * s, slope, np.abs(g * s) * rel + 1e-35,
                s * (1 + np.abs(g)) * (2 * rel + 4 * U) + 1e-35)
    cdf = 0.5 * erfc(-g / np.sqrt(2))
    pdf = np.exp(-g * g / 2) / np.sqrt(2 * np.pi)
    rel = (3 * g * g + 40) * U
    return g * cdf, cdf + g * pdf, np.abs(g * cdf) * rel + 1e-35, (cdf + np.abs(g) * pdf) * rel + 1e-35


def gated(g, eg, u, eu, kind):
    """H and its error from G and U with theirs: act' is at most 1.13, and next
    to act's zeros the relative form holds as well, whichever is less."""
    a, slope, ea, es = act(g, kind)
    ea = ea + np.abs(eg) * (np.abs(slope) + es + eg)
    h = a * u
    return h, np.abs(u) * ea + np.abs(a) * eu + 3 * U * np.abs(h) + ea * eu


def back_product(pairs):
    """Σ over (d, ed, q, w) of (d·w)·q and its error: d known within ed, d·w
    rounded to float32 and, scaled by a power of two per row that takes the
    largest to 2^13 .. 2^14, to fp16 (half a step: 2^-11 relative; a subnormal's,
    2^-25, is 2^-38 of the largest), float32 sums of C terms whose tree is no
    deeper than C."""
    h = half("f16") + 2 * U
    total, err, mag = 0.0, 0.0, 0.0
    C = sum(p[0].shape[1] for p in pairs) + 256
    top = np.max([np.abs(d * w).max(1) for d, _, _, w in pairs], axis=0)[:, None]
    for d, ed, q, w in pairs:
        q, w = np.asarray(q, np.float64), np.asarray(w, np.float64)
        total = total + matmul(d * w, q)
        each = np.abs(d * w) * h + ed * np.abs(w) + 2.0 ** -38 * top
        err = err + matmul(each, np.abs(q))
        mag = mag + matmul(np.abs(d * w), np.abs(q))
    return total, err + C * U * (mag + err)
