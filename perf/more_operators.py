"""Scoring with 4-bit embeddings and the loss on scores, as they are timed and compared.

An index of token embeddings in 4-bit microscaled floats is a quarter of the 16-bit one, and the
cheapest thing to scan; what the scan finds is turned into log probabilities of judged documents,
which are the training loss, and into the best other documents, which are its hard negatives. The
operators, and what they stand for:

  quantize  rows of floats to E2M1 codes in blocks of 32 with one power of two each, and back
  linear    product of such rows with such weights: hidden states to embeddings
  score     MaxSim of 4-bit queries against 4-bit documents
  prob      log probabilities and ranks of given columns of a score matrix, each row's entropy, and
            its k best columns
  grad      the gradient of the log probabilities and the entropy with respect to the scores

``own`` is set by whoever runs the file: false runs the plain forms below, true the library.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
DOC = 180           # tokens of a padded document
TINY = 2.0 ** -110  # a row whose largest magnitude is below this has no direction
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # what the codes 0 .. 7 stand for; 8 .. 15 are their negatives


def listed():
    return [
        # the hidden states of one 32-token query, on the way into the 4-bit product: latency
        {"name": "quantize-query", "op": "quantize", "T": 32, "d": 768, "type": "bf16",
         "normalize": False, "mask": False},
        # the token embeddings of a corpus, normalised and stored in 4 bits, padding masked
        {"name": "quantize-corpus", "op": "quantize", "T": 360000, "d": 128, "type": "fp16",
         "normalize": True, "mask": True},
        # one token through a square layer: the weights' bytes
        {"name": "linear-token", "op": "linear", "T": 1, "N": 4096, "K": 4096, "to": "bf16",
         "bias": False},
        # a large batch through it: the matrix cores
        {"name": "linear-batch", "op": "linear", "T": 8192, "N": 4096, "K": 4096, "to": "bf16",
         "bias": False},
        # sizes that no tile divides, a last block that is not full
        {"name": "linear-odd", "op": "linear", "T": 1213, "N": 1001, "K": 1000, "to": "fp32",
         "bias": True},
        # one 32-token query over a padded corpus: the documents' bytes
        {"name": "score-scan", "op": "score", "Nq": 1, "Lq": 32, "Nd": 50000, "Ld": DOC, "d": 128,
         "q_mask": False, "d_mask": True},
        # a batch of queries over pages of 1024 patches: the matrix cores
        {"name": "score-pages", "op": "score", "Nq": 32, "Lq": 32, "Nd": 1000, "Ld": 1024, "d": 128,
         "q_mask": False, "d_mask": False},
        # short ragged queries and documents of a narrow model, three blocks to a token
        {"name": "score-odd", "op": "score", "Nq": 5, "Lq": 20, "Nd": 333, "Ld": 77, "d": 80,
         "q_mask": True, "d_mask": True},
        # the scores of a contrastive batch: one right document for each query
        {"name": "prob-batch", "op": "prob", "Nq": 128, "Nd": 128, "P": 1, "k": 8, "type": "fp32",
         "mask": False},
        # the scores of a scan: eight judged documents for each query, 100 hard negatives
        {"name": "prob-corpus", "op": "prob", "Nq": 32, "Nd": 100000, "P": 8, "k": 100, "type": "fp32",
         "mask": False},
        # the contrastive batch's gradient, false negatives masked
        {"name": "grad-batch", "op": "grad", "Nq": 128, "Nd": 128, "P": 1, "type": "fp32", "mask": True,
         "entropy": False},
        # distillation: 32 taught documents for each query over the scores of a scan, and an entropy term
        {"name": "grad-corpus", "op": "grad", "Nq": 512, "Nd": 100000, "P": 32, "type": "fp32", "mask": False,
         "entropy": True},
    ]


def _size(rng, lo, hi):
    """A size spread over its logarithm, odd as often as not a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = max(16, v // 16 * 16)
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "score", "score", "score", "prob", "prob", "grad", "grad"])
    kind = rng.choice(["bf16", "fp16", "fp32"])
    if op == "quantize":
        d = _size(rng, 16, 8192)
        return {"op": op, "T": _size(rng, 1, min(360000, 46000000 // d)), "d": d, "type": kind,
                "normalize": rng.random() < 0.5, "mask": rng.random() < 0.5}
    if op == "linear":
        return {"op": op, "T": _size(rng, 1, 8192), "N": _size(rng, 16, 4096),
                "K": _size(rng, 16, 4096), "to": kind, "bias": rng.random() < 0.5}
    if op == "score":
        d = rng.choice([32, 48, 64, 96, 100, 128, 128, 128, 128, 192, 256, 384, 768, 1024])
        Nq, Lq, Ld = _size(rng, 1, 64), rng.choice([1, 5, 16, 20, 32, 32, 32, 48, 64, 200, 1024]), _size(rng, 1, 1024)
        most = min(9000000 * 128 // d // Ld, 130000000000 // (d * Nq * -(-Lq // 32) * 32 * -(-Ld // 32) * 32))
        return {"op": op, "Nq": Nq, "Lq": Lq, "Nd": _size(rng, 1, max(2, min(50000, most))), "Ld": Ld, "d": d,
                "q_mask": rng.random() < 0.5, "d_mask": rng.random() < 0.5}
    Nd = _size(rng, 2, 100000)
    c = {"op": op, "Nq": _size(rng, 1, min(1024, (50000000 if op == "grad" else 3200000) // Nd)), "Nd": Nd,
         "P": rng.choice([1, 1, 2, 8, 32]), "type": kind, "mask": rng.random() < 0.5}
    if op == "prob":
        c["k"] = min(Nd, rng.choice([0, 1, 8, 20, 100, 256]))
    else:
        c["entropy"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(T, d, g):
    """Activations: unit normal, with channels of different gains (a few of them large)."""
    gain = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    gain[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] *= 8
    return torch.randn(T, d, generator=g, device="cuda").mul_(gain)


def _keep(T, g, doc=DOC):
    """The mask of documents padded to `doc` tokens, half to all of each kept."""
    length = torch.randint((doc + 1) // 2, doc + 1, ((T + doc - 1) // doc,), generator=g, device="cuda")
    at = torch.arange(T, device="cuda")
    return (at % doc < length[at // doc]).to(torch.uint8)


def _embeddings(n, length, d, g):
    """Unit rows of tokens that share a topic within their document, in 4 bits."""
    topic = torch.randn(n, 1, d, generator=g, device="cuda")
    codes, scale = [], []
    step = max(1, 40000000 // (length * d))
    for at in range(0, n, step):
        part = topic[at:at + step]
        x = torch.randn(part.shape[0], length, d, generator=g, device="cuda") + 0.7 * part
        q, s = _pack(x / x.norm(dim=2, keepdim=True))
        codes.append(q)
        scale.append(s)
    return torch.cat(codes), torch.cat(scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        s["x"] = _rows(case["T"], case["d"], g).to(TYPES[case["type"]])
        s["mask"] = _keep(case["T"], g) if case["mask"] else None
    elif op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["a"], s["a_scale"] = _pack(_rows(T, K, g))
        s["w"], s["w_scale"] = _pack(torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K))
        s["bias"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
    elif op == "score":
        Nq, Lq, Nd, Ld = case["Nq"], case["Lq"], case["Nd"], case["Ld"]
        s["q"], s["q_scale"] = _embeddings(Nq, Lq, case["d"], g)
        s["d"], s["d_scale"] = _embeddings(Nd, Ld, case["d"], g)
        s["q_mask"] = _keep(Nq * Lq, g, Lq).view(Nq, Lq) if case["q_mask"] else None
        s["d_mask"] = _keep(Nd * Ld, g, Ld).view(Nd, Ld) if case["d_mask"] else None
    else:
        Nq, Nd, P = case["Nq"], case["Nd"], case["P"]
        # scores of 32-token queries: sums of 32 maxima of cosines, the judged documents above the rest
        x = 14 + 1.5 * torch.randn(Nq, Nd, generator=g, device="cuda")
        s["targets"] = torch.randint(0, Nd, (Nq, P), generator=g, device="cuda", dtype=torch.int32)
        x.scatter_add_(1, s["targets"].long(), torch.full((Nq, P), 3.0, device="cuda"))
        s["x"] = x.to(TYPES[case["type"]])
        s["scale"] = 2.0
        s["mask"] = (torch.rand(Nq, Nd, generator=g, device="cuda") < 0.9).to(torch.uint8) if case["mask"] else None
        if s["mask"] is not None:
            s["mask"].scatter_(1, s["targets"].long(), 1)
        if op == "grad":
            # what the forward left, and the gradients that come back: a loss over the batch, weights of a teacher
            z = s["x"].double() if s["mask"] is None else s["x"].double().masked_fill(s["mask"] == 0, -math.inf)
            top = z.amax(1, keepdim=True)
            z = (z - top) * s["scale"]
            log_sum = torch.logsumexp(z, 1)
            s["norm"] = torch.stack([top[:, 0], log_sum], 1).float()
            p = torch.exp(z - log_sum[:, None])
            s["entropy"] = (log_sum - torch.where(p > 0, p * z, 0.0).sum(1)).float()
            s["g_logp"] = -torch.softmax(torch.randn(Nq, P, generator=g, device="cuda"), 1) / Nq
            s["g_entropy"] = (0.05 / Nq) * torch.randn(Nq, generator=g, device="cuda") if case["entropy"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _codes(v):
    """Codes (0 .. 15) and exponents of rows [..., blocks of 32]: the block's power of two puts its
    largest magnitude between 4 and 8; the nearest level, ties to the even code."""
    top = v.abs().amax(-1)
    e = torch.clamp(torch.frexp(top)[1] - 3, -127, 127)
    e = torch.where(top > 0, e, 0)
    a = v.abs() * torch.exp2(-e.to(v.dtype))[..., None]
    code = (a > 0.25).to(torch.uint8)
    for border, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border if up else a > border)
    return code + 8 * (v < 0).to(torch.uint8), e


def _blocks(x):
    """Rows [..., d] as [..., ceil(d / 32), 32], zeros behind the end."""
    d = x.shape[-1]
    n = (d + 31) // 32
    return torch.nn.functional.pad(x, (0, n * 32 - d)).view(*x.shape[:-1], n, 32)


def _pack(x):
    """Rows to packed codes, the first of two in the low half of a byte, and biased exponents."""
    code, e = _codes(_blocks(x))
    code = code.view(*x.shape[:-1], -1)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8)


def _values(codes, scale, bits=torch.float32):
    """What packed codes stand for, whole blocks."""
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=bits, device=codes.device)
    nibbles = torch.stack([codes & 15, codes >> 4], -1).view(*scale.shape, 32)
    return (levels[nibbles.int()] * torch.exp2(scale.to(bits) - 127)[..., None]).view(*scale.shape[:-1], -1)


def _plain_quantize(x, mask, normalize):
    """In 64 bits: a value next to the border between two codes must not change sides."""
    v = x.double()
    if mask is not None:
        v = torch.where(mask[:, None] == 0, 0.0, v)
    if normalize:
        top = v.abs().amax(1, keepdim=True)
        n = v.square().sum(1, keepdim=True).sqrt()
        v = torch.where(top < TINY, 0.0, v / torch.where(top < TINY, 1.0, n))
    code, e = _codes(_blocks(v))
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=x.device)
    y = levels[code.int()] * torch.exp2(e.float())[..., None]
    return y.view(x.shape[0], -1)[:, :x.shape[1]].contiguous()


def _plain_score(s):
    c = s["case"]
    q = _values(s["q"], s["q_scale"]).view(c["Nq"] * c["Lq"], -1)
    out = []
    step = max(1, min(c["Nd"], 400000000 // (c["Ld"] * max(c["Nq"] * c["Lq"], c["d"]))))
    for at in range(0, c["Nd"], step):
        d = _values(s["d"][at:at + step], s["d_scale"][at:at + step])
        n = d.shape[0]
        sim = (q @ d.view(n * c["Ld"], -1).T).view(c["Nq"], c["Lq"], n, c["Ld"])
        if s["d_mask"] is not None:
            sim = sim.masked_fill(s["d_mask"][at:at + step] == 0, -math.inf)
        best = sim.amax(3)
        best = torch.where(best == -math.inf, 0.0, best)
        if s["q_mask"] is not None:
            best = best * s["q_mask"][:, :, None]
        out.append(best.sum(1))
    return torch.cat(out, 1)


def _plain_prob(s):
    c = s["case"]
    x = s["x"].float()
    if s["mask"] is not None:
        x = x.masked_fill(s["mask"] == 0, -math.inf)
    top = x.amax(1, keepdim=True)
    z = (x - top) * s["scale"]
    e = torch.exp(z)
    total = e.double().sum(1)
    log_sum = torch.log(total)
    entropy = log_sum - torch.where(e > 0, e * z, 0.0).double().sum(1) / total
    t = s["targets"].long()
    at = torch.arange(c["Nd"], device=x.device)
    xt = x.gather(1, t)
    logp = (z.gather(1, t).double() - log_sum[:, None]).float()
    rank = torch.stack([((x > xt[:, p:p + 1]) | ((x == xt[:, p:p + 1]) & (at < t[:, p:p + 1]))).sum(1)
                        for p in range(c["P"])], 1).int()
    out = [logp, rank, torch.stack([top[:, 0], log_sum.float()], 1), entropy.float()]
    if c["k"]:
        val, idx = torch.sort(x, dim=1, descending=True, stable=True)
        val, idx = val[:, :c["k"]], idx[:, :c["k"]]
        none = val == -math.inf
        out += [torch.where(none, -1, idx).int(), (((val - top) * s["scale"]).double() - log_sum[:, None]).float()]
    return out


def _plain_grad(s):
    x = s["x"].float()
    if s["mask"] is not None:
        x = x.masked_fill(s["mask"] == 0, -math.inf)
    logp = (x - s["norm"][:, :1]) * s["scale"] - s["norm"][:, 1:]
    p = torch.exp(logp)
    dz = -p * s["g_logp"].sum(1, keepdim=True)
    if s["g_entropy"] is not None:
        dz -= s["g_entropy"][:, None] * torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0)
    dz.scatter_add_(1, s["targets"].long(), s["g_logp"])
    return dz * s["scale"]


def _plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        return _plain_quantize(s["x"], s["mask"], c["normalize"])
    if c["op"] == "linear":
        y = _values(s["a"], s["a_scale"]) @ _values(s["w"], s["w_scale"]).T
        return (y if s["bias"] is None else y + s["bias"]).to(TYPES[c["to"]])
    if c["op"] == "score":
        return _plain_score(s)
    return _plain_prob(s) if c["op"] == "prob" else _plain_grad(s)


def run(s):
    if not own:
        return _plain(s)
    import maxsim_scoring_amd as ms
    c = s["case"]
    if c["op"] == "quantize":
        codes, scale = ms.maxsim_quantize_mx4(s["x"], s["mask"], normalize=c["normalize"])
        return ms.maxsim_dequantize_mx4(codes, scale, c["d"], out_dtype=torch.float32)
    if c["op"] == "linear":
        return ms.maxsim_linear_mx4(s["a"], s["a_scale"], s["w"], s["w_scale"], s["bias"],
                                    out_dtype=TYPES[c["to"]])
    if c["op"] == "score":
        return ms.maxsim_fwd_mx4(s["q"], s["q_scale"], s["d"], s["d_scale"], s["q_mask"], s["d_mask"])[0]
    if c["op"] == "prob":
        logp, rank, norm, entropy, top_idx, top_logp = ms.maxsim_logprob_fwd(
            s["x"], s["targets"], s["mask"], scale=s["scale"], k=c["k"])
        return [logp, rank, norm, entropy] + ([top_idx, top_logp] if c["k"] else [])
    return ms.maxsim_logprob_bwd(s["x"], s["targets"], s["norm"], s["g_logp"], s["mask"], scale=s["scale"],
                                 entropy=s["entropy"] if c["entropy"] else None, grad_entropy=s["g_entropy"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_quantize(x, kept, normalize):
    """Each value to the nearest multiple of its binade's half step (a whole one from 4 on is 2)."""
    x = np.where(kept[:, None], x, 0.0)
    if normalize:
        live = np.abs(x).max(1) >= TINY
        size = np.sqrt(np.einsum("td,td->t", x, x))
        x = np.where(live[:, None], x / np.where(live, size, 1.0)[:, None], 0.0)
    T, d = x.shape
    n = -(-d // 32)
    b = np.zeros((T, n * 32))
    b[:, :d] = x
    b = b.reshape(T, n, 32)
    peak = np.abs(b).max(2, keepdims=True)
    unit = np.exp2(np.clip(np.floor(np.log2(np.where(peak > 0, peak, 1.0))) - 2, -127, 127))
    b /= unit
    step = np.exp2(np.maximum(np.frexp(b)[1] - 1, 0) - 1)
    q = np.clip(np.rint(b / step) * step, -6, 6) * unit
    return q.reshape(T, n * 32)[:, :d]


def _wide(codes, scale):
    """Packed codes as 64-bit values: sign, two exponent bits, one fraction bit."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    sign = torch.where(n >= 8, -1.0, 1.0).double()
    n = n % 8
    power = torch.floor(n / 2)
    size = torch.where(power == 0, n / 2, (1 + (n % 2) / 2) * 2 ** (power - 1))
    return sign * size * (2.0 ** (scale.double() - 127)).repeat_interleave(32, -1)


def _exact_score(s):
    """Product by product in 64-bit matrix products, a block of documents at a time."""
    c = s["case"]
    q = _wide(s["q"], s["q_scale"])
    total = np.zeros((c["Nq"], c["Nd"]))
    step = max(1, 100000000 // (c["Ld"] * max(c["Lq"], c["d"])))
    for at in range(0, c["Nd"], step):
        d = _wide(s["d"][at:at + step], s["d_scale"][at:at + step])
        hidden = None if s["d_mask"] is None else s["d_mask"][at:at + step] == 0
        flat = d.reshape(-1, d.shape[2]).T.contiguous()
        for i in range(c["Nq"]):
            sim = torch.mm(q[i], flat).view(c["Lq"], d.shape[0], c["Ld"])
            if hidden is not None:
                sim[:, hidden] = -math.inf
            best = sim.max(2).values
            best[best == -math.inf] = 0.0
            if s["q_mask"] is not None:
                best = best[s["q_mask"][i] != 0]
            total[i, at:at + step] = best.sum(0).cpu().numpy()
    return total


def _exact_prob(c, h, scale):
    x = h["x"]
    kept = np.ones(x.shape, bool) if h.get("mask") is None else h["mask"] != 0
    Nq, Nd = x.shape
    logp, rank = np.zeros((Nq, c["P"])), np.zeros((Nq, c["P"]), np.int32)
    norm, entropy = np.zeros((Nq, 2)), np.zeros(Nq)
    idx, best = np.full((Nq, c["k"]), -1, np.int32), np.full((Nq, c["k"]), -np.inf)
    for i in range(Nq):
        cols = np.flatnonzero(kept[i])
        v = x[i, cols]
        w = np.exp(scale * (v - v.max()))
        lp = scale * (v - v.max()) - math.log(w.sum())
        norm[i] = v.max(), math.log(w.sum())
        entropy[i] = -(np.exp(lp) * lp).sum()
        order = np.lexsort((cols, -v))
        place = np.empty(Nd, np.int64)
        place[cols[order]] = np.arange(len(cols))
        whole = np.full(Nd, -np.inf)
        whole[cols] = lp
        t = h["targets"][i].astype(np.int64)
        logp[i], rank[i] = whole[t], place[t]
        m = min(c["k"], len(cols))
        idx[i, :m], best[i, :m] = cols[order[:m]], lp[order[:m]]
    return [logp, rank, norm, entropy] + ([idx, best] if c["k"] else [])


def _exact_grad(c, s):
    """Row by row: the softmax's Jacobian on the given gradients."""
    out = torch.empty(s["x"].shape, dtype=torch.float64)
    for i in range(c["Nq"]):
        v = s["x"][i].double()
        kept = torch.ones_like(v, dtype=torch.bool) if s["mask"] is None else s["mask"][i] != 0
        z = s["scale"] * v
        p = torch.zeros_like(v)
        p[kept] = torch.softmax(z[kept], 0)
        up = torch.zeros_like(v)
        up.index_add_(0, s["targets"][i].long(), s["g_logp"][i].double())
        dz = up - p * up.sum()
        if s["g_entropy"] is not None:
            h = torch.zeros_like(v)
            h[kept] = torch.special.entr(p[kept])
            dz -= s["g_entropy"][i].double() * (p * h.sum() - h)
        out[i] = (s["scale"] * dz).cpu()
    return out.numpy()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        kept = np.ones(case["T"], bool) if s["mask"] is None else s["mask"].cpu().numpy() != 0
        return _exact_quantize(s["x"].double().cpu().numpy(), kept, case["normalize"])
    if op == "linear":
        w = _wide(s["w"], s["w_scale"]).T.contiguous()
        y = torch.cat([torch.mm(_wide(a, e), w) for a, e in zip(s["a"].split(2048), s["a_scale"].split(2048))])
        return (y if s["bias"] is None else y + s["bias"].double()).cpu().numpy()
    if op == "score":
        return _exact_score(s)
    if op == "grad":
        return _exact_grad(case, s)
    h = {k: v.double().cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor)}
    return _exact_prob(case, h, s["scale"])


def work(case):
    """Masked rows (a quarter of a padded batch) are not read; every output is written."""
    op = case["op"]
    if op == "quantize":
        T, d, n = case["T"], case["d"], -(-case["d"] // 32)
        live = 0.75 if case["mask"] else 1.0
        return {"bytes": T * (live * d * BYTES[case["type"]] + 2 * 17 * n + 4 * d + (1 if case["mask"] else 0)),
                "flops": 3 * live * T * d}
    if op == "linear":
        T, N, K, n = case["T"], case["N"], case["K"], -(-case["K"] // 32)
        return {"bytes": 17 * n * (T + N) + T * N * BYTES[case["to"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * T * N * K}
    if op == "score":
        Nq, Lq, Nd, Ld, d = (case[k] for k in ("Nq", "Lq", "Nd", "Ld", "d"))
        live, n = (0.75 if case["d_mask"] else 1.0), -(-d // 32)
        return {"bytes": 17 * n * (Nq * Lq + live * Nd * Ld) + 4 * Nq * Nd + (Nd * Ld if case["d_mask"] else 0)
                + (Nq * Lq if case["q_mask"] else 0), "flops": 2 * d * Nq * Lq * live * Nd * Ld}
    Nq, Nd, P = case["Nq"], case["Nd"], case["P"]
    read = Nq * Nd * (BYTES[case["type"]] + (1 if case["mask"] else 0)) + 4 * Nq * P
    if op == "prob":
        return {"bytes": read + Nq * (8 * P + 12 + 8 * case["k"]), "flops": (5 + 2 * P) * Nq * Nd}
    return {"bytes": read + 4 * Nq * Nd + Nq * (4 * P + 8 + (8 if case["entropy"] else 0)), "flops": 4 * Nq * Nd}
