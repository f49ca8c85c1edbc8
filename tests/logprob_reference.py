"""Plain float64 forms of the log probabilities and their gradient, and the error
bounds that the kernels' arithmetic allows.

u = 2^-24 is half a float32 step. z = scale (x - m) rounds twice and, where a row is
joined from chunks, is the sum of two such numbers: it is off by at most 4 u |z|.
exp adds at most 6 u (the hardware's 2^x one unit in the last place, its correction
and the product the rest). Sums are float64. So with A = sum p |z|, L is off by at
most 4 u A + 6 u, to first order; the bounds carry 1 % for the rest."""

import numpy as np

U = 2.0 ** -24


def candidates(x, mask):
    return (x != -np.inf) & (np.ones(x.shape, bool) if mask is None else mask != 0)


def forward(x, targets, mask, scale, k):
    """x float64 [Nq, Nd]. A dict of the outputs and of the bounds of the float ones."""
    Nq, Nd = x.shape
    P = targets.shape[1]
    live = candidates(x, mask)
    out = dict(logp=np.zeros((Nq, P)), rank=np.full((Nq, P), -1), norm=np.full((Nq, 2), -np.inf), entropy=np.zeros(Nq),
               top_idx=np.full((Nq, k), -1), top_logp=np.full((Nq, k), -np.inf))
    b = dict(logp=np.zeros((Nq, P)), norm=np.zeros((Nq, 2)), entropy=np.zeros(Nq), top_logp=np.zeros((Nq, k)))
    for i in range(Nq):
        cols = np.flatnonzero(live[i])
        lp, zs = np.full(Nd, -np.inf), np.zeros(Nd)
        place = np.full(Nd, -1)
        off_L = 0.0
        if len(cols):
            m = x[i, cols].max()
            z = scale * (x[i, cols] - m)
            e = np.exp(z)
            L = np.log(e.sum())
            p = e / e.sum()
            A = (p * np.abs(np.where(p > 0, z, 0))).sum()
            off_L = 1.01 * U * (4 * A + 6)
            off_H = off_L + 1.01 * U * (p * np.where(p > 0, np.abs(z), 0) * (4 * np.where(p > 0, np.abs(z), 0) + 12)).sum()
            out["norm"][i] = m, L
            b["norm"][i] = 0, off_L + U * abs(L)
            out["entropy"][i] = L - (p * np.where(p > 0, z, 0)).sum()
            b["entropy"][i] = off_H + U * abs(out["entropy"][i])
            lp[cols], zs[cols] = z - L, z
            order = cols[np.lexsort((cols, -x[i, cols]))]
            place[order] = np.arange(len(order))
            n = min(k, len(order))
            out["top_idx"][i, :n], out["top_logp"][i, :n] = order[:n], lp[order[:n]]
            with np.errstate(invalid="ignore"):
                b["top_logp"][i, :n] = off_L + 1.01 * U * (2 * np.abs(zs[order[:n]]) + np.abs(lp[order[:n]]))
        for q, t in enumerate(targets[i]):
            if 0 <= t < Nd:
                out["logp"][i, q], out["rank"][i, q] = lp[t], place[t]
                if np.isfinite(lp[t]):
                    b["logp"][i, q] = off_L + 1.01 * U * (2 * abs(zs[t]) + abs(lp[t]))
    return out, b


def backward(x, targets, mask, scale, g, norm, entropy=None, gh=None):
    """The formula at the given norm and entropy: (dX, bound of its float32 arithmetic)."""
    Nq, Nd = x.shape
    live = candidates(x, mask)
    dX, bound = np.zeros((Nq, Nd)), np.zeros((Nq, Nd))
    for i in range(Nq):
        if not live[i].any():
            continue
        z = scale * np.where(live[i], x[i] - norm[i, 0], 0.0)
        lp = z - norm[i, 1]
        p = np.where(live[i], np.exp(lp), 0.0)
        add, size, n = np.zeros(Nd), np.zeros(Nd), np.zeros(Nd)
        for t, v in zip(targets[i], g[i]):
            if 0 <= t < Nd and live[i, t]:
                add[t] += v
                size[t] += abs(v)
                n[t] += 1
        h, H = (0.0, 0.0) if gh is None else (gh[i], entropy[i])
        G, Gs = add.sum(), size.sum()
        w = h * (lp + H) + G
        d = add - p * w
        off_lp = U * (2 * np.abs(z) + np.abs(lp))          # the difference, the product, the sum
        off_p = p * (off_lp + 6 * U)
        off_w = np.abs(h) * (off_lp + U * np.abs(lp + H)) + U * np.abs(w) + U * (len(targets[i]) + 16) * Gs
        dX[i] = np.where(live[i], scale * d, 0.0)
        bound[i] = np.where(live[i], 1.01 * scale * (off_p * np.abs(w) + p * off_w + U * p * np.abs(w)
                                                     + U * n * size + 2 * U * np.abs(d)
                                                     # below 2^-126 a rounding is half of 2^-149: that of p,
                                                     # multiplied by w, and those of p w and the difference
                                                     + 2.0 ** -150 * (np.abs(w) + 2)), 0.0)
    return dX, bound
