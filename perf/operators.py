"""The operators of the embedding head, as they are timed and compared.

The head turns an encoder's hidden states into the token embeddings that MaxSim scores. Its
operators, and what they stand for:

  quantize   rows of 16- or 32-bit floats to 8-bit codes with one scale for each token
  linear     8-bit matrix product with a scale for each token and for each output channel
  embed      that product, each row of it divided by its Euclidean norm, as floats or as codes
  normalize  rows divided by their Euclidean norm, and the gradient of that
  dropout    dropout whose mask is recomputed from a counter and never stored, and its gradient

``own`` is set by whoever runs the file: false runs the plain forms below, true the library.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1}
DOC = 180          # tokens of a padded document
TINY = 2.0 ** -110  # a row whose largest magnitude is below this counts as zeros


def listed():
    return [
        # the hidden states of one 32-token query, on the way into the 8-bit product: latency
        {"name": "quantize-query", "op": "quantize", "T": 32, "d": 768, "type": "bf16",
         "normalize": False, "mask": False},
        # float token embeddings of a corpus, stored as 8-bit codes for the scan, padding masked
        {"name": "quantize-corpus", "op": "quantize", "T": 360000, "d": 128, "type": "fp16",
         "normalize": True, "mask": True},
        # the document side of a contrastive batch: 128 pages of 1024 patches
        {"name": "normalize-batch", "op": "normalize", "T": 131072, "d": 128, "type": "bf16",
         "to": "bf16", "mask": True},
        # its gradient, from the 32-bit gradients of the scoring backward
        {"name": "normalize-batch-grad", "op": "normalize_grad", "T": 131072, "d": 128,
         "type": "bf16", "to": "bf16"},
        # an odd width and a ragged packed batch, 32-bit rows to 16-bit embeddings
        {"name": "normalize-odd-width", "op": "normalize", "T": 12347, "d": 100, "type": "fp32",
         "to": "fp16", "mask": False},
        # the hidden states of that contrastive batch in front of the projection
        {"name": "dropout-batch", "op": "dropout", "n": 131072 * 768, "type": "bf16", "p": 0.1},
        # the gradient for the query side, 32-bit, a length that no vector width divides
        {"name": "dropout-queries-grad", "op": "dropout_grad", "n": 16383 * 129, "type": "fp32",
         "p": 0.25},
        # one token through a square layer: the weights' bytes
        {"name": "linear-token", "op": "linear", "T": 1, "N": 4096, "K": 4096, "to": "bf16",
         "bias": False},
        # a large batch through it: the matrix cores
        {"name": "linear-batch", "op": "linear", "T": 8192, "N": 4096, "K": 4096, "to": "bf16",
         "bias": False},
        # sizes that no tile divides, rows that are not 16-byte aligned
        {"name": "linear-odd", "op": "linear", "T": 1213, "N": 1001, "K": 1000, "to": "fp32",
         "bias": True},
        # one 32-token query from hidden states to embeddings: latency
        {"name": "embed-query", "op": "embed", "T": 32, "N": 128, "K": 768, "to": "fp16",
         "bias": False, "mask": False},
        # a block of documents from hidden states to 8-bit embeddings: the bytes of the states
        {"name": "embed-corpus", "op": "embed", "T": 360000, "N": 128, "K": 768, "to": "int8",
         "bias": True, "mask": True},
    ]


def _size(rng, lo, hi):
    """A size spread over its logarithm, odd as often as not a multiple of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = max(16, v // 16 * 16)
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["quantize", "normalize", "normalize_grad", "dropout", "dropout_grad",
                     "linear", "linear", "embed", "embed"])
    kind = rng.choice(["bf16", "fp16", "fp32"])
    if op == "quantize":
        d = _size(rng, 16, 8192)
        return {"op": op, "T": _size(rng, 1, min(360000, 46000000 // d)), "d": d, "type": kind,
                "normalize": rng.random() < 0.5, "mask": rng.random() < 0.5}
    if op in ("normalize", "normalize_grad"):
        d = _size(rng, 16, 1024)
        c = {"op": op, "T": _size(rng, 1, min(131072, 16000000 // d)), "d": d, "type": kind,
             "to": rng.choice(["bf16", "fp16", "fp32"])}
        if op == "normalize":
            c["mask"] = rng.random() < 0.5
        return c
    if op in ("dropout", "dropout_grad"):
        return {"op": op, "n": _size(rng, 128, 50000000), "type": kind,
                "p": rng.choice([0.0, 0.05, 0.1, 0.3, 0.5, 0.9])}
    if op == "linear":
        return {"op": op, "T": _size(rng, 1, 8192), "N": _size(rng, 16, 4096),
                "K": _size(rng, 16, 4096), "to": kind, "bias": rng.random() < 0.5}
    K = _size(rng, 64, 4096)
    N = _size(rng, 16, 1024)
    return {"op": op, "T": _size(rng, 1, min(200000, 30000000000 // (K * N))), "N": N, "K": K,
            "to": rng.choice(["int8", "bf16", "fp16", "fp32"]), "bias": rng.random() < 0.5,
            "mask": rng.random() < 0.5}


def _rows(T, d, g):
    """Activations: unit normal, with channels of different gains (a few of them large)."""
    gain = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    gain[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] *= 8
    return torch.randn(T, d, generator=g, device="cuda").mul_(gain)


def _keep(T, g):
    """The mask of documents padded to DOC tokens, half to all of each kept."""
    length = torch.randint(DOC // 2, DOC + 1, ((T + DOC - 1) // DOC,), generator=g, device="cuda")
    at = torch.arange(T, device="cuda")
    return (at % DOC < length[at // DOC]).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("quantize", "normalize", "normalize_grad"):
        s["x"] = _rows(case["T"], case["d"], g).to(TYPES[case["type"]])
        s["mask"] = _keep(case["T"], g) if case.get("mask") else None
        if op == "normalize_grad":
            s["g"] = torch.randn(case["T"], case["d"], generator=g, device="cuda")
            s["rnorm"] = (1 / s["x"].double().norm(dim=1)).float()
    elif op in ("dropout", "dropout_grad"):
        s["x"] = torch.randn(case["n"], generator=g, device="cuda").to(TYPES[case["type"]])
        s["seed"] = (0x9D2C5680A1B2C3D4 ^ (seed * 0x10001)) & 0xFFFFFFFFFFFFFFFF
        s["step"] = seed % 1000 + (1 << 33)
    else:
        T, N, K = case["T"], case["N"], case["K"]
        x = _rows(T, K, g)
        top = x.abs().amax(1, keepdim=True)
        s["a"] = (x * (127 / top)).round_().to(torch.int8)
        s["a_scale"] = (top[:, 0] / 127).contiguous()
        del x
        s["w"] = (torch.randn(N, K, generator=g, device="cuda") * 32).round_().clamp_(-127, 127).to(torch.int8)
        s["w_scale"] = torch.exp(0.3 * torch.randn(N, generator=g, device="cuda")) / (32 * math.sqrt(K))
        s["bias"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["mask"] = _keep(T, g) if case.get("mask") else None
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _philox(index, seed, step):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): four 32-bit words for each 64-bit index,
    counter (index, step), key seed. Products wrap in 64 bits, which keeps both their halves."""
    low = 0xFFFFFFFF
    c0, c1 = index & low, index >> 32
    c2, c3 = torch.full_like(index, step & low), torch.full_like(index, (step >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & low) ^ c1 ^ k0, p1 & low, (p0 >> 32 & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], 1)


def _dropped(n, p, seed, step):
    """Eight elements share a counter, 16 bits each; the probability is a multiple of 2^-16."""
    words = _philox(torch.arange((n + 7) // 8, device="cuda"), seed, step)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]
    return bits < math.floor(p * 65536 + 0.5)


def _dropout(x, p, seed, step):
    left = 65536 - math.floor(p * 65536 + 0.5)
    up = float(np.float32(65536 / left)) if left else 0.0
    return torch.where(_dropped(x.numel(), p, seed, step), 0.0, x.float() * up).to(x.dtype)


def _codes(y, mask, normalize):
    """Codes and scales of float rows, in 64 bits: a value next to the border between two codes
    must not change sides by an earlier rounding. The codes do not change with the row's norm."""
    y = y.double()
    top = y.abs().amax(1)
    empty = top < TINY if mask is None else (top < TINY) | (mask == 0)
    top = torch.where(empty, 1.0, top)
    v = torch.where(empty[:, None], 0.0, y * 127 / top[:, None])
    scale = 1 / (v * v).sum(1).sqrt() if normalize else top / 127
    return v.round().to(torch.int8), torch.where(empty, 1.0, scale).float()


def _unit(y, mask):
    """Rows over their norms, taken of the rows over their largest magnitude."""
    top = y.abs().amax(1)
    empty = top < TINY if mask is None else (top < TINY) | (mask == 0)
    top = torch.where(empty, torch.ones_like(top), top)
    v = torch.where(empty[:, None], 0.0, y / top[:, None])
    r = 1 / torch.where(empty, torch.ones_like(top), (v * v).sum(1)).sqrt()
    return v * r[:, None], torch.where(empty, 0.0, r / top)


def _linear(s, bits):
    """Products of whole numbers, whose sums pass 24 bits: in 64."""
    acc = (s["a"].double() @ s["w"].double().T).to(bits)
    y = acc * (s["a_scale"].to(bits)[:, None] * s["w_scale"].to(bits))
    return y if s["bias"] is None else y + s["bias"]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        codes, scale = _codes(s["x"], s["mask"], c["normalize"])
        return codes * scale[:, None], scale
    if op == "normalize":
        y, rnorm = _unit(s["x"].float(), s["mask"])
        return y.to(TYPES[c["to"]]), rnorm
    if op == "normalize_grad":
        u = s["x"].float() * s["rnorm"][:, None]
        return (s["rnorm"][:, None] * (s["g"] - u * (u * s["g"]).sum(1, keepdim=True))).to(TYPES[c["to"]])
    if op in ("dropout", "dropout_grad"):
        return _dropout(s["x"], c["p"], s["seed"], s["step"])
    y = _linear(s, torch.float64 if c["to"] == "int8" else torch.float32)
    if op == "linear":
        return y.to(TYPES[c["to"]])
    if c["to"] == "int8":
        codes, scale = _codes(y, s["mask"], True)
        return codes * scale[:, None], scale
    return _unit(y, s["mask"])[0].to(TYPES[c["to"]])


def run(s):
    if not own:
        return _plain(s)
    import maxsim_scoring_amd as ms
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        codes, scale = ms.maxsim_quantize_tok(s["x"], s["mask"], normalize=c["normalize"])
        return codes * scale[:, None], scale
    if op == "normalize":
        return ms.maxsim_normalize_fwd(s["x"], s["mask"], out_dtype=TYPES[c["to"]])
    if op == "normalize_grad":
        return ms.maxsim_normalize_bwd(s["x"], s["rnorm"], s["g"], out_dtype=TYPES[c["to"]])
    if op == "dropout":
        return ms.maxsim_dropout_fwd(s["x"], c["p"], s["seed"], s["step"])
    if op == "dropout_grad":
        return ms.maxsim_dropout_bwd(s["x"], c["p"], s["seed"], s["step"])
    if op == "linear":
        return ms.maxsim_linear_i8(s["a"], s["a_scale"], s["w"], s["w_scale"], s["bias"],
                                   out_dtype=TYPES[c["to"]])
    e, scale = ms.maxsim_embed_i8(s["a"], s["a_scale"], s["w"], s["w_scale"], s["bias"], s["mask"],
                                  out_dtype=TYPES[c["to"]])
    return (e * scale[:, None], scale) if c["to"] == "int8" else e


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_codes(y, kept, normalize):
    """Values that the codes stand for: the nearest of 255 steps of the row's largest magnitude."""
    peak = np.abs(y).max(1)
    live = kept & (peak >= TINY)
    peak = np.where(live, peak, 1.0)
    step = np.where(live, peak / 127, 1.0)
    q = np.rint(np.where(live[:, None], y, 0.0) * 127 / peak[:, None])
    if normalize:
        step = np.where(live, step / np.where(live, np.sqrt(np.einsum("td,td->t", y, y)), 1.0), 1.0)
    return q * step[:, None], step


def _exact_unit(y, kept):
    size = np.sqrt(np.einsum("td,td->t", y, y))
    live = kept & (np.abs(y).max(1) >= TINY)
    r = np.where(live, 1 / np.where(live, size, 1.0), 0.0)
    return np.where(live[:, None], y, 0.0) * r[:, None], r


def _exact_mask(n, p, seed, step):
    i = np.arange((n + 7) // 8, dtype=np.uint64)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    a, b = i & low, i >> half
    c, d = np.full_like(i, step & 0xFFFFFFFF), np.full_like(i, step >> 32)
    for r in range(10):
        key0 = np.uint64(((seed & 0xFFFFFFFF) + r * 0x9E3779B9) & 0xFFFFFFFF)
        key1 = np.uint64(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        left, right = np.uint64(0xD2511F53) * a, np.uint64(0xCD9E8D57) * c
        a, b, c, d = (right >> half) ^ b ^ key0, right & low, (left >> half) ^ d ^ key1, left & low
    w = np.empty((len(i), 4), dtype="<u4")
    w[:, 0], w[:, 1], w[:, 2], w[:, 3] = a, b, c, d
    return w.view("<u2").reshape(-1)[:n].astype(np.int64) >= math.floor(p * 65536 + 0.5)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    host = {k: v.double().cpu().numpy() for k, v in s.items()
            if isinstance(v, torch.Tensor) and k not in ("a", "w")}
    if op in ("dropout", "dropout_grad"):
        kept = _exact_mask(case["n"], case["p"], s["seed"], s["step"])
        left = 65536 - math.floor(case["p"] * 65536 + 0.5)
        return np.where(kept, host["x"] * (65536 / max(left, 1)), 0.0)
    T = case["T"]
    kept = host["mask"] != 0 if s.get("mask") is not None else np.ones(T, dtype=bool)
    if op == "quantize":
        return _exact_codes(host["x"], kept, case["normalize"])
    if op == "normalize":
        return _exact_unit(host["x"], kept)
    if op == "normalize_grad":
        x, up = host["x"], host["g"]
        size2 = np.einsum("td,td->t", x, x)
        along = np.einsum("td,td->t", x, up) / size2
        return (up - along[:, None] * x) / np.sqrt(size2)[:, None]
    # products of whole numbers, exact in 64-bit floats, by blocks of rows
    w = s["w"].double().T.contiguous()
    acc = torch.cat([torch.mm(part.double(), w) for part in s["a"].split(16384)]).cpu().numpy()
    y = acc * host["a_scale"][:, None] * host["w_scale"][None, :]
    if s["bias"] is not None:
        y = y + host["bias"]
    if op == "linear":
        return y
    return _exact_codes(y, kept, True) if case["to"] == "int8" else _exact_unit(y, kept)[0]


def work(case):
    """Masked rows (a quarter of a padded batch) are not read; every output is written."""
    op = case["op"]
    live = 0.75 if case.get("mask") else 1.0
    if op in ("dropout", "dropout_grad"):
        return {"bytes": 2 * case["n"] * BYTES[case["type"]], "flops": case["n"]}
    T = case["T"]
    flags = T if case.get("mask") else 0
    if op == "quantize":
        return {"bytes": T * case["d"] * (live * BYTES[case["type"]] + 1) + 4 * T + flags,
                "flops": 3 * live * T * case["d"]}
    if op == "normalize":
        return {"bytes": T * case["d"] * (live * BYTES[case["type"]] + BYTES[case["to"]]) + 4 * T + flags,
                "flops": 3 * live * T * case["d"]}
    if op == "normalize_grad":
        return {"bytes": T * case["d"] * (BYTES[case["type"]] + 4 + BYTES[case["to"]]) + 4 * T,
                "flops": 5 * T * case["d"]}
    N, K = case["N"], case["K"]
    out = T * N * BYTES[case["to"]] + (4 * T if case["to"] == "int8" else 0)
    return {"bytes": live * T * K + N * K + 4 * (live * T + N) + out + flags + (4 * N if case["bias"] else 0),
            "flops": 2 * live * T * N * K}
