"""Plain float64 forms of the 4-bit operators, and the error bounds that float32
sums and one final rounding allow the kernels.

u = 2^-24 is half a float32 step. Products of two codes and their powers of two
are exact. One matrix instruction adds 64 or 128 of them to an accumulator with an
error of at most one unit in the last place of the sum of all magnitudes, 2^-23
of it; a sum that passes n instructions is off by at most n 2^-23 times the sum
of all its magnitudes (to first order; the bounds carry 1 % for the rest)."""

import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TINY = 2.0 ** -110
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def blocks(d):
    return -(-d // 32)


def quantize(x, mask=None, normalize=False):
    """(codes 0 .. 15 [T, 32 B], scale bytes [T, B]) of finite float64 rows."""
    x = np.array(x, dtype=np.float64)
    T, d = x.shape
    if mask is not None:
        x[np.asarray(mask) == 0] = 0.0
    if normalize:
        peak = np.abs(x).max(1)
        x[peak < TINY] = 0.0
        n = np.sqrt((x * x).sum(1))
        x = x / np.where(n > 0, n, 1.0)[:, None]
    v = np.zeros((T, blocks(d) * 32))
    v[:, :d] = x
    v = v.reshape(T, -1, 32)
    m = np.abs(v).max(2)
    e = np.clip(np.frexp(m)[1] - 3, -127, 127)
    e = np.where(m > 0, e, 0)
    a = np.abs(np.ldexp(v, -e[:, :, None]))
    # nearest level, the even code on a tie: levels are compared by their distance
    dist = np.abs(a[..., None] - LEVELS)
    best = dist.min(-1, keepdims=True)
    cand = dist == best
    first, last = cand.argmax(-1), 7 - cand[..., ::-1].argmax(-1)
    code = np.where(first % 2 == 0, first, last)
    return (code + 8 * np.signbit(v)).reshape(T, -1).astype(np.uint8), (e + 127).astype(np.uint8)


def pack(code):
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)


def values(codes, scale):
    """Float64 values [T, 32 B] of packed codes and scale bytes (numpy), NaN for 255."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    v = np.where(n >= 8, -1.0, 1.0) * LEVELS[n & 7]
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(int) - 127))
    return v * np.repeat(s, 32, 1)


def linear_bound(y, mag, K, bias, dtype):
    """mag: sums of the products' magnitudes. At most 4 instructions for each 8
    blocks begun, and 8 parts of k that are added."""
    n = 4 * -(-blocks(K) // 8) + 8
    return (1.01 * (n * 2 * U * mag + U * (np.abs(y) + np.abs(bias))) + np.abs(y) * HALF[dtype] + FLOOR[dtype])


def sim_error(mag, d):
    """Of one similarity: two instructions for each four blocks begun."""
    return 1.01 * (2 * -(-blocks(d) // 4)) * 2 * U * mag


def maxsim(q, d, q_mask=None, d_mask=None):
    """(scores, similarities with -inf at masked tokens, sums of magnitudes) of
    float64 tensors [Nq, Lq, k], [Nd, Ld, k] on any device."""
    Nq, Lq, k = q.shape
    Nd, Ld, _ = d.shape
    flat = d.reshape(Nd * Ld, k).T.contiguous()
    sim = (q.reshape(Nq * Lq, k) @ flat).view(Nq, Lq, Nd, Ld).permute(0, 2, 1, 3)
    mag = (q.abs().reshape(Nq * Lq, k) @ flat.abs()).view(Nq, Lq, Nd, Ld).permute(0, 2, 1, 3)
    if d_mask is not None:
        sim = sim.masked_fill(d_mask[None, :, None, :] == 0, -np.inf)
    best = sim.amax(3) if Ld else torch.full((Nq, Nd, Lq), -np.inf, dtype=torch.float64, device=q.device)
    best = torch.where(best == -np.inf, 0.0, best)
    if q_mask is not None:
        best = best * (q_mask[:, None, :] != 0)
    return best.sum(2), sim, mag
