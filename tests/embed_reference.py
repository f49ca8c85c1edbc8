"""Plain float64 forms of the embedding head's operators, and the error bounds
that float32 arithmetic and one final rounding allow the kernels.

u = 2^-24 is half a float32 step, HALF[t] half a step of type t. A sum of n
terms added in any order, at most `chain` additions deep, is off by at most
chain * u times the sum of the terms' magnitudes (to first order; the bounds
below carry 1 % for the rest).
"""

import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half the smallest step (subnormals)
FLOOR = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TINY = 2.0 ** -110


def f64(t):
    return t.detach().double().cpu().numpy()


def depth(d):
    """Additions that a term of a row's sum passes through: at most 128 in a
    lane that holds its part of the row in registers (16 chunks of 8), or its
    64th of a long row; 6 across the lanes, 8 across waves, 1 of its own."""
    return max(128, -(-d // 64) + 8) + 15


def live_rows(x, mask):
    peak = np.abs(x).max(1)
    return (peak >= TINY) & (np.ones(len(x), bool) if mask is None else np.asarray(mask).astype(bool))


def quantize(x, mask=None, normalize=False):
    """(codes, scale, distance of 127 x / m from the nearest half)."""
    x = np.where(live_rows(np.nan_to_num(x), mask)[:, None], x, 0.0)
    live = np.abs(x).max(1) > 0
    peak = np.where(live, np.abs(x).max(1), 1.0)
    v = x * 127 / peak[:, None]
    scale = peak / 127 if not normalize else 1 / np.sqrt(np.where(live, (v * v).sum(1), 1.0))
    gap = np.abs(np.abs(v - np.floor(v)) - 0.5)
    return np.rint(v).astype(np.int8), np.where(live, scale, 1.0), gap


def normalize(x, mask=None):
    live = live_rows(np.nan_to_num(x), mask)
    x = np.where(live[:, None], x, 0.0)
    peak = np.where(live, np.abs(x).max(1), 1.0)
    v = x / peak[:, None]
    n = np.sqrt(np.where(live, (v * v).sum(1), 1.0))
    return v / n[:, None], np.where(live, 1 / n / peak, 0.0)


def normalize_bound(y, d, dtype):
    """Each square rounds (1), they are added (depth), the root and its
    reciprocal round (half of the sum's error, then 2), and the row may be
    scaled first (2) and is multiplied (2)."""
    return np.abs(y) * 1.01 * ((depth(d) + 1) / 2 + 6) * U + np.abs(y) * HALF[dtype] + FLOOR[dtype]


def normalize_grad(x, rnorm, g):
    u = x * rnorm[:, None]
    return rnorm[:, None] * (g - u * (u * g).sum(1, keepdims=True))


def normalize_grad_bound(x, rnorm, g, dtype):
    r = np.abs(rnorm)[:, None]
    u = np.abs(x * rnorm[:, None])
    dot = np.abs((x * rnorm[:, None] * g).sum(1, keepdims=True))
    slack = (u * np.abs(g)).sum(1, keepdims=True) * (depth(x.shape[1]) + 1) * U
    exact = np.abs(normalize_grad(x, rnorm, g))
    return (1.01 * r * (u * (slack + 3 * U * dot) + 2 * U * (np.abs(g) + u * dot))
            + exact * HALF[dtype] + FLOOR[dtype])


def linear(a, a_scale, w, w_scale, bias=None):
    """(y, the products without the bias): whole numbers below 2^53 are exact."""
    p = (a.astype(np.float64) @ w.astype(np.float64).T) * (a_scale[:, None] * w_scale[None, :])
    return (p if bias is None else p + bias), p


def linear_bound(y, p, dtype):
    """The scales' product, the sum's conversion and their product round on p,
    adding the bias and the output on y."""
    return 1.01 * (3 * U * np.abs(p) + U * np.abs(y)) + np.abs(y) * HALF[dtype] + FLOOR[dtype]


def embed_bound(y, p, dtype):
    """linear_bound's float32 error of y, over the norm, plus normalize_bound."""
    e = 1.01 * (3 * U * np.abs(p) + U * np.abs(y))
    size = np.sqrt((y * y).sum(1, keepdims=True))
    size = np.where(size > 0, size, 1.0)
    unit = y / size
    return (e + np.abs(unit) * np.sqrt((e * e).sum(1, keepdims=True))) / size * 1.01 + normalize_bound(
        unit, y.shape[1], dtype)


def philox(counter, key):
    """Philox4x32-10 of Salmon, Moraes, Dror and Shaw (SC 2011) in Python's own
    integers: counter of 4 and key of 2 32-bit words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        left, right = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [right >> 32 ^ c[1] ^ k[0], right & 0xFFFFFFFF, left >> 32 ^ c[3] ^ k[1], left & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropped(n, p, seed, step, first=0):
    """Which of elements first .. first + n - 1 are dropped (first: a multiple of 8)."""
    q = int(np.floor(p * 65536 + 0.5))
    out = []
    for i in range(first // 8, (first + n + 7) // 8):
        words = philox((i & 0xFFFFFFFF, i >> 32, step & 0xFFFFFFFF, step >> 32),
                       (seed & 0xFFFFFFFF, seed >> 32))
        for w in words:
            out += [(w & 0xFFFF) < q, (w >> 16) < q]
    return np.array(out[:n], dtype=bool)


def dropout(x, p, gone):
    q = int(np.floor(p * 65536 + 0.5))
    up = np.float64(np.float32(65536 / (65536 - q))) if q < 65536 else 0.0
    return np.where(gone, 0.0, np.where(gone, 0.0, x) * up)
