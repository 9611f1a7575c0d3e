"""Float64 reference of the low-rank adapter calls and the 8-bit checkpoints,
with the magnitudes that their error bounds need. Plain NumPy."""
import numpy as np

import oracle as O

U32 = 2.0 ** -23      # a step of float32: the matrix cores need not round to nearest
UOUT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half a step of the 16-bit types
TINY = {"bf16": 2.0 ** -126, "f16": 2.0 ** -14}   # their smallest normal numbers
# H and G may meet the matrix cores as two 16-bit halves, hi = rnd(v) and
# lo = rnd(v - hi): at most u² of v is lost, 2^-16 for bf16 (f16: 2^-22, its
# rows scaled by a power of two so that neither half leaves fp16's normal
# range by more than the row's own largest value allows: 2^-23 of that value).
LOW = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}


def gamma(n):
    """Relative error of a float32 sum of n products, any order."""
    return n * U32 / (1 - n * U32)


def members(ids, L):
    return [np.flatnonzero(ids == a) for a in range(L)]


def forward(x, w, A, B, c, ids):
    """y, h and the magnitudes mh = |A||x|, ml = c |B| (|A||x|), mw = |w||x|."""
    T, r = x.shape[0], A.shape[1]
    y = x @ w.T
    h = np.zeros((T, r))
    mh = np.zeros((T, r))
    ml = np.zeros(y.shape)
    for a, t in enumerate(members(ids, len(A))):
        h[t] = x[t] @ A[a].T
        mh[t] = np.abs(x[t]) @ np.abs(A[a]).T
        y[t] += c[a] * (h[t] @ B[a].T)
        ml[t] = abs(c[a]) * (mh[t] @ np.abs(B[a]).T)
    return y, h, mh, ml, np.abs(x) @ np.abs(w).T


def backward(dy, x, h, w, A, B, c, ids):
    """(dx, dA, dB) and for each the magnitude of the terms in its sum."""
    dx = dy @ w
    mw = np.abs(dy) @ np.abs(w)
    mg_x = np.zeros(dx.shape)
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    mA, mB = np.zeros(A.shape), np.zeros(B.shape)
    for a, t in enumerate(members(ids, len(A))):
        g = c[a] * (dy[t] @ B[a])
        mg = abs(c[a]) * (np.abs(dy[t]) @ np.abs(B[a]))
        dx[t] += g @ A[a]
        mg_x[t] = mg @ np.abs(A[a])
        dA[a] = g.T @ x[t]
        mA[a] = mg.T @ np.abs(x[t])
        dB[a] = c[a] * (dy[t].T @ h[t])
        mB[a] = abs(c[a]) * (np.abs(dy[t]).T @ np.abs(h[t]))
    return dx, dA, dB, mw, mg_x, mA, mB


def decode_magnitude(x, qw, qz, sc, N, group):
    """Σ |x|·(32 + q + z)·scale: what float32 rounds in the matrix-core decode."""
    q = O.unpack_codes(qw, N, 4).astype(np.float64)
    z = np.repeat(O.unpack_codes(qz, N, 4), group, axis=0).astype(np.float64)
    s = np.repeat(sc.view(np.float16).astype(np.float64), group, axis=0)
    return np.abs(x) @ ((32.0 + q + z) * s)


def pack8(x32):
    """Codes and steps of float32 activations, every operation rounded once."""
    T, K = x32.shape
    x = x32.reshape(T, K // 128, 128)
    with np.errstate(invalid="ignore"):
        m = np.abs(x).max(axis=2)
    bad = ~np.isfinite(x).all(axis=2)
    m = np.where(bad, np.float32(1), np.maximum(m, np.float32(2.0 ** -100))).astype(np.float32)
    inv = (np.float32(127) / m).astype(np.float32)
    with np.errstate(invalid="ignore"):
        codes = np.rint((x * inv[:, :, None]).astype(np.float32))
    codes = np.where(bad[:, :, None], 0, codes).astype(np.int8)
    steps = np.where(bad, np.float32(np.nan), m / np.float32(127)).astype(np.float32)
    return codes.reshape(T, K), steps


def unpack8(codes, steps):
    T, K = codes.shape
    return (codes.reshape(T, K // 128, 128).astype(np.float32) *
            steps[:, :, None]).astype(np.float32).reshape(T, K)
