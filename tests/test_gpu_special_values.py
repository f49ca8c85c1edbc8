"""Values at the ends of the float types on the GPU: NaN, infinities, the largest
and smallest magnitudes, exact ties."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import embed_reference as ref
from embed_reference import f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ms():
    import maxsim_scoring_amd as m
    m.binding.lib()
    assert torch.cuda.is_available()
    return m


# --------------------------------------------------------------------- top-k

def _ranked(v):
    """Columns in decreasing order of the values: positive NaN, +Inf ... -Inf,
    negative NaN (each by its bits), equal values by column."""
    b = v.view(np.uint32).astype(np.int64)
    b = np.where((b & 0x7FFFFFFF) == 0, 0, b)
    key = np.where(b & 0x80000000, 0xFFFFFFFF - b, b | 0x80000000)
    return np.lexsort((np.arange(len(v)), -key))


@pytest.mark.parametrize("Nd,k", [(5, 5), (64, 20), (8192, 100), (8193, 100), (30000, 1000), (100000, 100)])
def test_topk_with_nans(ms, Nd, k):
    """Rows with some NaN, with fewer than k other values, and with nothing else:
    every index is a column of the row, once, and in order."""
    rng = np.random.default_rng(Nd)
    v = rng.standard_normal((6, Nd)).astype(np.float32)
    v[0, ::3] = np.nan
    v[1, k - 1:] = np.nan                       # one value fewer than k
    v[2] = np.nan
    v[3] = np.array(0xFFC00000, np.uint32).view(np.float32)  # the sign bit set: below -Inf
    v[4, 1:] = np.array(0xFFFFFFFF, np.uint32).view(np.float32)
    v[4, -1] = -np.inf
    v[5, 1::2] = np.nan
    v[5, 3::4] = -np.inf
    s = torch.from_numpy(v).to(DEV)
    idx, val, rows = ms.maxsim_topk(s, k, want_rows=True)
    want = np.stack([_ranked(r)[:k] for r in v])
    assert np.array_equal(idx.cpu().numpy(), want)
    got = val.cpu().numpy().view(np.uint32)
    assert np.array_equal(got, np.take_along_axis(v, want, 1).view(np.uint32))
    assert np.array_equal(rows.cpu().numpy(), np.repeat(np.arange(6), k).reshape(6, k))


# -------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [96, 100, 768, 1030, 9001, 16640])
def test_quantize_rows_of_large_magnitude(ms, d, dtype):
    """Largest magnitudes on both sides of 2^120, from which on codes are always
    decided in float64, and of 2^126, from which on the reciprocal is subnormal.
    The scale's bound is that of ordinary rows: every value is rounded once more
    or once less before it is squared, well within the 3 of test_quantize."""
    g = torch.Generator(device=DEV).manual_seed(d)
    tops = [2.0 ** e for e in (100, 119, 119.99, 120, 120.5, 123, 125.9, 125.999, 126, 126.1, 127.9)]
    x = torch.rand(len(tops), d, generator=g, device=DEV, dtype=torch.float64) * 2 - 1
    x /= x.abs().amax(1, keepdim=True)
    x = (x * torch.tensor(tops, device=DEV, dtype=torch.float64)[:, None]).to(dtype)
    for normalize in (False, True):
        codes, scale = ms.maxsim_quantize_tok(x, normalize=normalize)
        want, ws, _ = ref.quantize(f64(x), None, normalize)
        assert np.array_equal(codes.cpu().numpy(), want)
        bound = np.abs(ws) * (((ref.depth(d) + 3) / 2 + 3 if normalize else 1) * 1.01 * ref.U)
        off = np.abs(f64(scale) - ws)
        assert (off <= bound).all(), (normalize, (f64(scale) / ws).tolist())


WRONG = [float("nan"), float("inf"), -float("inf")]


def _spoiled(T, d, dtype, seed):
    """Ordinary rows and the same rows with a NaN or an infinity in some of them
    (row 1 NaN throughout, row 4 masked): (clean, spoiled, mask, spoiled rows)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, d, generator=g, device=DEV).to(dtype)
    y = x.clone()
    y[1] = float("nan")
    for i, w in enumerate(WRONG):
        y[6 + i, (7 * i) % d] = w
    y[9, d - 1] = float("nan")
    y[9, 0] = float("inf")
    y[4] = float("nan")
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[4] = 0
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[[1, 6, 7, 8, 9]] = True
    return x, y, mask, bad


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [1, 7, 8, 100, 128, 768, 1030, 9001, 16640])
def test_quantize_shows_nan_and_inf(ms, d, dtype):
    """What a row with a NaN or an infinity stands for is NaN; masked rows and all
    others are as without them."""
    x, y, mask, bad = _spoiled(70, d, dtype, d)
    for normalize in (False, True):
        codes, scale = ms.maxsim_quantize_tok(y, mask, normalize=normalize)
        want, ws = ms.maxsim_quantize_tok(x, mask, normalize=normalize)
        assert torch.isnan(codes * scale[:, None])[bad].all(), normalize
        assert torch.equal(codes[~bad], want[~bad]) and torch.equal(scale[~bad], ws[~bad])
        assert scale[4] == 1 and not codes[4].any()


# ------------------------------------------------------------------ products

# T, d, K of every form of maxsim_embed_i8: streamed (4 and 8 waves), direct (8 and
# 16 waves), channels spread over workgroups, tiles of every width class, rows at
# any address
FORMS = [(40, 128, 768), (70, 100, 256), (40, 250, 384), (33, 100, 130), (40, 200, 96), (40, 512, 1024),
         (12, 272, 4096), (4120, 40, 48), (4120, 200, 272), (520, 300, 96), (600, 700, 64), (513, 1000, 77)]
forms = pytest.mark.parametrize("T,d,K", FORMS)


def _operands(T, d, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.randint(-128, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (d, K), generator=g, device=DEV, dtype=torch.int8)
    s = torch.exp(torch.randn(T, generator=g, device=DEV)) / 127
    ws = torch.exp(torch.randn(d, generator=g, device=DEV)) / (127 * K ** 0.5)
    return a, s, w, ws, torch.randn(d, generator=g, device=DEV)


@forms
def test_embed_shows_nan_and_inf(ms, T, d, K):
    """A row whose scale is NaN or infinite stands for NaN, in floats and in codes;
    all other rows are as without it."""
    a, s, w, ws, b = _operands(T, d, K, T + d + K)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[torch.tensor([1, 5, T - 1], device=DEV)] = True
    spoiled = s.clone()
    spoiled[bad] = torch.tensor(WRONG, device=DEV)
    for bias in (None, b):
        codes, scale = ms.maxsim_embed_i8(a, spoiled, w, ws, bias)
        want, wscale = ms.maxsim_embed_i8(a, s, w, ws, bias)
        assert torch.isnan(codes * scale[:, None])[bad].all()
        assert torch.equal(codes[~bad], want[~bad]) and torch.equal(scale[~bad], wscale[~bad])
        for out in (torch.float16, torch.bfloat16, torch.float32):
            e, _ = ms.maxsim_embed_i8(a, spoiled, w, ws, bias, out_dtype=out)
            want, _ = ms.maxsim_embed_i8(a, s, w, ws, bias, out_dtype=out)
            assert torch.isnan(e[bad]).all() and torch.equal(e[~bad], want[~bad])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K", [768, 100, 4096])
def test_hidden_states_with_nan_and_inf(ms, K, dtype):
    """From hidden states to embeddings: broken states give NaN, masked ones zeros."""
    x, y, mask, bad = _spoiled(70, K, dtype, K)
    _, _, w, ws, b = _operands(1, 128, K, K)
    codes, scale = ms.embed_tokens_i8(y, w, ws, b, mask)
    want, wscale = ms.embed_tokens_i8(x, w, ws, b, mask)
    assert torch.isnan(codes * scale[:, None])[bad].all()
    assert torch.equal(codes[~bad], want[~bad]) and torch.equal(scale[~bad], wscale[~bad])
    assert scale[4] == 1 and not codes[4].any()
    e, _ = ms.embed_tokens_i8(y, w, ws, b, mask, out_dtype=torch.bfloat16)
    assert torch.isnan(e[bad]).all() and torch.isfinite(e[~bad]).all() and not e[4].any()


@forms
def test_masked_rows_are_zeros_whatever_the_weights_hold(ms, T, d, K):
    """A scale or bias of one channel that is NaN or infinite spoils every row but
    the masked ones, which are written as zeros."""
    a, s, w, ws, b = _operands(T, d, K, 3 * T + d + K)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[torch.tensor([0, 3, T - 2], device=DEV)] = 0
    out_of = mask == 0
    for i, wrong in enumerate(WRONG):
        for spoil_bias in (False, True):
            ws2, b2 = ws.clone(), b.clone()
            (b2 if spoil_bias else ws2)[(5 * i) % d] = wrong
            for out in (torch.float16, torch.bfloat16, torch.float32):
                e, _ = ms.maxsim_embed_i8(a, s, w, ws2, b2, mask, out_dtype=out)
                assert (e[out_of] == 0).all() and torch.isnan(e[~out_of]).any(1).all()
            codes, scale = ms.maxsim_embed_i8(a, s, w, ws2, b2, mask)
            assert not codes[out_of].any() and (scale[out_of] == 1).all()
            assert torch.isnan(scale[~out_of]).all()


def _codes_of(y):
    """The nearest integers to 127 y / max|y| of a row of float64, ties to even, in
    rational arithmetic."""
    exact = {v: Fraction(v) for v in set(y.tolist())}
    top = max(abs(v) for v in exact.values())
    code = {v: round(127 * f / top) if top else 0 for v, f in exact.items()}  # round(): half to even
    return [code[v] for v in y.tolist()]


def _products(acc, s, ws, b):
    """float64 rows of sum * (a_scale * w_scale) + bias, rounded once (the scales'
    product is exact in float64)."""
    cache = {}

    def one(a, x, w, c):
        if (a, x, w, c) not in cache:
            cache[a, x, w, c] = float(a * Fraction(x) * Fraction(w) + Fraction(c))
        return cache[a, x, w, c]
    return np.array([[one(int(a), x, w, c) for a, w, c in zip(row, ws, b)] for row, x in zip(acc, s)])


@forms
def test_embed_codes_at_ties(ms, T, d, K):
    """Small sums under one weight scale put many channels on, and a tiny bias puts
    them next to, the middle between two codes; the nearest code is taken there
    too, and the even one on a tie."""
    rng = np.random.default_rng(T + d + K)
    a = np.zeros((T, K), np.int8)
    for i in range(6):  # a few entries a row: sums of at most 24
        a[np.arange(T), rng.integers(0, K, T)] = rng.integers(-2, 3, T)
    w = rng.integers(-2, 3, (d, K)).astype(np.int8)
    s = np.exp(rng.standard_normal(T)).astype(np.float32)
    at = np.unique(np.concatenate([rng.integers(0, T, 60), [0, T - 1]]))
    acc = a[at].astype(np.int64) @ w.T.astype(np.int64)
    tiny = np.where(rng.random(d) < 0.5, 0.0, rng.choice([-1, 1], d) * 2.0 ** -rng.integers(28, 46, d)).astype(np.float32)
    ties = 0
    for scale, bias in ((0.37, None), (1.0, tiny)):
        ws = np.full(d, scale, np.float32)
        sc = s if bias is None else np.exp2(np.round(np.log2(s))).astype(np.float32)
        dev = [torch.from_numpy(x).to(DEV) for x in (a, sc, w, ws)]
        codes, _ = ms.maxsim_embed_i8(*dev, None if bias is None else torch.from_numpy(bias).to(DEV))
        y = _products(acc, sc[at].tolist(), ws.tolist(), [0.0] * d if bias is None else bias.tolist())
        want = np.array([_codes_of(row) for row in y])
        top = np.abs(acc).max(1, keepdims=True)
        ties += ((254 * acc) % np.maximum(2 * top, 1) == top).sum() if bias is None else 0
        assert np.array_equal(codes.cpu().numpy()[at], want)
    assert ties > 20


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [1, 100, 128, 1030, 9001, 16640])
def test_normalize_shows_nan_and_inf(ms, d, dtype):
    """Rows with a NaN or an infinity are NaN, and so are their gradients; all
    others are as without them."""
    x, y, mask, bad = _spoiled(70, d, dtype, d + 1)
    g = torch.randn(70, d, generator=torch.Generator(device=DEV).manual_seed(d), device=DEV)
    u, rnorm = ms.maxsim_normalize_fwd(y, mask)
    want, wnorm = ms.maxsim_normalize_fwd(x, mask)
    # 1 / Inf is 0: only the row itself shows an infinity
    assert torch.isnan(u[bad]).any(1).all() and not u[4].any() and rnorm[4] == 0
    assert torch.equal(u[~bad], want[~bad]) and torch.equal(rnorm[~bad], wnorm[~bad])
    dx = ms.maxsim_normalize_bwd(y, rnorm, g, out_dtype=torch.float32)
    wx = ms.maxsim_normalize_bwd(x, wnorm, g, out_dtype=torch.float32)
    assert torch.equal(dx[~bad], wx[~bad]) and torch.isnan(dx[bad]).any(1).all()


def test_broken_states_reach_scores_and_top_k(ms):
    """A document with a NaN state: the others' scores are those without it, and
    the top-k's columns stay in range."""
    Nq, Nd, Lq, Ld, K, d = 3, 40, 32, 50, 256, 128
    g = torch.Generator(device=DEV).manual_seed(5)
    hq = torch.randn(Nq, Lq, K, generator=g, device=DEV).bfloat16()
    hd = torch.randn(Nd, Ld, K, generator=g, device=DEV).bfloat16()
    _, _, w, ws, _ = _operands(1, d, K, 6)
    eq, sq = ms.embed_tokens_i8(hq, w, ws)
    want, _ = ms.maxsim_fwd_i8_tok(eq, sq, *ms.embed_tokens_i8(hd, w, ws))
    hd[7, 3, 11] = float("nan")
    hd[30] = float("inf")
    ed, sd = ms.embed_tokens_i8(hd, w, ws)
    assert torch.isnan(sd[7, 3]) and torch.isnan(sd[30]).all() and int(torch.isnan(sd).sum()) == 1 + Ld
    scores, _ = ms.maxsim_fwd_i8_tok(eq, sq, ed, sd)
    fine = torch.ones(Nd, dtype=torch.bool, device=DEV)
    fine[[7, 30]] = False
    assert torch.equal(scores[:, fine], want[:, fine])
    idx, _, _ = ms.maxsim_topk(scores, Nd)
    assert torch.equal(idx.long().sort(1).values, torch.arange(Nd, device=DEV).expand(Nq, Nd))
    # a broken query token breaks that query alone
    hq[1, 0, 0] = float("nan")
    eq, sq = ms.embed_tokens_i8(hq, w, ws)
    scores, _ = ms.maxsim_fwd_i8_tok(eq, sq, *ms.embed_tokens_i8(hd.nan_to_num(0, 0, 0), w, ws))
    idx, _, _ = ms.maxsim_topk(scores, 10)
    assert torch.isfinite(scores[[0, 2]]).all() and ((idx >= 0) & (idx < Nd)).all()


@pytest.mark.parametrize("out", [torch.int8, torch.float16], ids=["i8", "fp16"])
def test_captured_embeddings_spread_over_workgroups(ms, out):
    """The form of three launches that keeps statistics in its output: two graphs of
    it, replayed at once on streams of their own, against the eager calls."""
    ops = [_operands(T, d, K, K) for T, d, K in ((32, 1024, 1024), (200, 272, 4096))]
    graphs, outs = [], []
    for o in ops:
        ms.maxsim_embed_i8(*o, out_dtype=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ms.maxsim_embed_i8(*o, out_dtype=out))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ops]
    for r in range(4):
        for a, s, *_ in ops:
            a.neg_()
            s.mul_(1.25)
        want = [ms.maxsim_embed_i8(*o, out_dtype=out) for o in ops]
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (e, s), (we, wsc) in zip(outs, want):
            assert torch.equal(e, we) and (s is None or torch.equal(s, wsc))
