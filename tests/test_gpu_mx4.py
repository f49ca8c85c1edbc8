"""4-bit rows on the GPU against plain float64 forms (mx4_reference.py, which
also derives the bounds). Codes and scales are compared exactly."""

import numpy as np
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
short = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
by_type = pytest.mark.parametrize("dtype", TYPES, ids=short.get)


@pytest.fixture(scope="module")
def ms():
    import maxsim_scoring_amd as m
    m.binding.lib()
    assert torch.cuda.is_available()
    return m


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(T, d, dtype, seed):
    g = _gen(seed)
    x = torch.randn(T, d, generator=g, device=DEV) * torch.exp(torch.randn(T, d, generator=g, device=DEV))
    return x.to(dtype)


def _mask(shape, seed, keep=0.7):
    return (torch.rand(shape, generator=_gen(seed), device=DEV) < keep).to(torch.uint8)


def _guarded(shape, dtype, fill):
    """A tensor with a guard behind it: (tensor, check of the guard)."""
    n = int(np.prod(shape))
    buf = torch.full((n + 256,), fill, dtype=dtype, device=DEV)
    return buf[:n].view(shape), lambda: bool((buf[n:] == fill).all())


def _off_by_one(t):
    """The same values at an odd address."""
    buf = torch.empty(t.numel() + 1, dtype=torch.uint8, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


def _random_mx4(lead, d, seed, spread=4):
    """Codes of every value and scales of a few neighbouring exponents; zeros behind d."""
    g = _gen(seed)
    B = ref.blocks(d)
    n = torch.randint(0, 16, (*lead, B * 32), generator=g, device=DEV, dtype=torch.int32)
    n[..., d:] = 0
    codes = (n[..., 0::2] | n[..., 1::2] << 4).to(torch.uint8)
    scale = torch.randint(120, 120 + spread, (*lead, B), generator=g, device=DEV).to(torch.uint8)
    return codes, scale


def _values(codes, scale):
    """Float64 on the GPU."""
    lead = scale.shape[:-1]
    v = ref.values(codes.reshape(-1, codes.shape[-1]).cpu().numpy(), scale.reshape(-1, scale.shape[-1]).cpu().numpy())
    return torch.from_numpy(v).to(DEV).view(*lead, -1)


# ------------------------------------------------------------- rows

ROWS = [(1, 1), (3, 7), (5, 31), (5, 32), (37, 33), (64, 64), (33, 100), (1000, 128), (17, 200), (9, 516), (32, 768),
        (7, 1000), (3, 1030), (5, 2050), (4, 4096), (3, 8192), (2, 9001), (2, 16640), (1, 131071)]


def _check_codes(got, want):
    codes, scale = got
    wcode, wscale = want
    assert np.array_equal(scale.cpu().numpy(), wscale)
    n = codes.cpu().numpy()
    n = np.stack([n & 15, n >> 4], -1).reshape(n.shape[0], -1)
    # a zero's sign is free where the value is not a negative zero itself
    differ = (n != wcode) & ~((n % 8 == 0) & (wcode % 8 == 0))
    assert not differ.any(), f"{differ.sum()} codes differ, first at {np.argwhere(differ)[0]}"


@by_type
@pytest.mark.parametrize("T,d", ROWS)
def test_quantize(ms, T, d, dtype):
    x = _rows(T, d, dtype, T + d)
    B = ref.blocks(d)
    for normalize in (False, True):
        for mask in (None, _mask((T,), d)):
            codes, ok1 = _guarded((T, 16 * B), torch.uint8, 0xA5)
            scale, ok2 = _guarded((T, B), torch.uint8, 0xA5)
            ms.maxsim_quantize_mx4(x, mask, normalize=normalize, codes=codes, scale=scale)
            torch.cuda.synchronize()
            assert ok1() and ok2()
            _check_codes((codes, scale), ref.quantize(x.double().cpu().numpy(), None if mask is None else mask.cpu().numpy(),
                                                      normalize))


@by_type
@pytest.mark.parametrize("T,d", [(9, 205), (9, 300), (9, 384), (5, 1600), (3, 8190)])
def test_quantize_more_widths(ms, T, d, dtype):
    """Widths of every number of lanes and units, whole eights of values and others."""
    test_quantize(ms, T, d, dtype)


def test_quantize_borders(ms):
    """Every border between levels, the values next to it, and the powers of two, at exponents over the whole range."""
    base = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.999999, 0.5, 1, 2, 3, 4, 0.0], dtype=np.float32)
    near = np.concatenate([base, np.nextafter(base, np.float32(9)), np.nextafter(base, np.float32(-9)), -base])
    rows = []
    for e in (0, 1, -1, 30, -30, 100, -100, 124, -120, -125, -126, -130, -140):
        for top in (4.0, 7.0, 6.0):
            for at in range(0, len(near), 31):
                row = np.zeros(32, dtype=np.float32)
                part = near[at:at + 31]
                row[:len(part)] = part
                row[31] = top
                rows.append(np.ldexp(row, e))
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(DEV)
    _check_codes(ms.maxsim_quantize_mx4(x), ref.quantize(x.double().cpu().numpy()))
    # a negative zero keeps its sign
    z = torch.full((1, 32), -0.0, device=DEV)
    codes, scale = ms.maxsim_quantize_mx4(z)
    assert (codes == 0x88).all() and (scale == 127).all()


@pytest.mark.parametrize("d", [100, 4096, 8192, 9001, 16640])
def test_quantize_normalized_zeros_keep_their_sign(ms, d):
    """Blocks of zeros beside a block that is not, a row of zeros, and a row too small to have a direction."""
    x = torch.zeros(4, d, device=DEV)
    x[0, 0], x[0, 1::2] = 3.0, -0.0
    x[1] = -0.0
    x[2, ::3] = -2.0 ** -120
    x[3, 1], x[3, 2:] = -2.0, -0.0
    codes, scale = ms.maxsim_quantize_mx4(x, normalize=True)
    n = torch.stack([codes & 15, codes >> 4], -1).view(4, -1)[:, :d]
    want = torch.signbit(x).to(torch.uint8) * 8
    assert torch.equal(n[1:3], want[1:3]) and (scale[1:3] == 127).all()
    assert torch.equal(n[0, 1:], want[0, 1:]) and torch.equal(n[3, 2:], want[3, 2:])
    assert int(n[0, 0]) == 6 and int(n[3, 1]) == 14 and (scale[:, 1:] == 127).all()


def test_quantize_normalized_ties(ms):
    """Rows whose norm is a whole number put values exactly on borders and powers of two."""
    rows = np.zeros((8, 64))
    rows[0, 5] = 3.0                                   # 1
    rows[1, [1, 2, 40, 41]] = [2, -2, 2, 2]            # 1/2 each
    rows[2, 0] = 5; rows[2, 1:40] = 1                  # norm 8: 5/8 and 1/8 in one block
    rows[3, 0] = 7; rows[3, 1:16] = 1                  # norm 8: 7/8
    rows[4, :16] = 1                                   # 1/4
    rows[5, 0] = 25; rows[5, 1] = -31; rows[5, 2] = 3; rows[5, 3:8] = 1  # norm 40: 25/40 = 5/8
    rows[5, 0:10] = [25, 31, 3, 1, 1, 1, 1, 1, 0, 0]
    rows[6, :64] = 1                                   # 1/8
    rows[7, 0] = 3; rows[7, 33] = -4                   # 3/5, 4/5
    for f in (1.0, 2.0 ** 90, 2.0 ** -100):
        x = torch.from_numpy(rows * f).float().to(DEV)
        _check_codes(ms.maxsim_quantize_mx4(x, normalize=True), ref.quantize(x.double().cpu().numpy(), normalize=True))
    x = torch.from_numpy(rows).to(torch.bfloat16).to(DEV)
    _check_codes(ms.maxsim_quantize_mx4(x, normalize=True), ref.quantize(x.double().cpu().numpy(), normalize=True))


def test_quantize_extremes(ms):
    """Zeros, subnormal rows, the largest values; with and without normalisation."""
    rows = np.zeros((9, 96), dtype=np.float32)
    rows[1, :] = 2.0 ** -149
    rows[2, ::3] = 2.0 ** -140
    rows[3, :] = 3.4028234e38
    rows[4, 0] = 3.4028234e38; rows[4, 50] = 2.0 ** -120
    rows[5, :] = 2.0 ** -110
    rows[6, :] = 2.0 ** -111
    rows[7, 0] = 1.0; rows[7, 32:64] = 2.0 ** -126; rows[7, 64:] = 1e-30
    rows[8, :] = np.linspace(1e37, 3e38, 96)
    x = torch.from_numpy(rows).to(DEV)
    for normalize in (False, True):
        _check_codes(ms.maxsim_quantize_mx4(x, normalize=normalize),
                     ref.quantize(x.double().cpu().numpy(), normalize=normalize))


@by_type
def test_quantize_marks_nan_and_infinity(ms, dtype):
    x = _rows(6, 100, dtype, 3)
    clean = x.clone()
    x[1, 40] = float("nan")
    x[2, 99] = float("inf")
    x[4, 3] = -float("inf")
    codes, scale = ms.maxsim_quantize_mx4(x)
    c0, s0 = ms.maxsim_quantize_mx4(clean)
    marked = torch.zeros_like(scale, dtype=torch.bool)
    marked[1, 1] = marked[2, 3] = marked[4, 0] = True
    assert torch.equal(scale == 255, marked)
    assert torch.equal(scale[~marked], s0[~marked])
    keep = (~marked).repeat_interleave(16, 1)
    assert torch.equal(codes[keep], c0[keep])
    codes, scale = ms.maxsim_quantize_mx4(x, normalize=True)
    rows = torch.tensor([False, True, True, False, True, False], device=DEV)
    assert (scale[rows] == 255).all()
    c0, s0 = ms.maxsim_quantize_mx4(clean, normalize=True)
    assert torch.equal(scale[~rows], s0[~rows]) and torch.equal(codes[~rows], c0[~rows])
    mask = (~rows).to(torch.uint8)
    for normalize in (False, True):  # masked rows are not looked at
        codes, scale = ms.maxsim_quantize_mx4(x, mask, normalize=normalize)
        assert (scale[rows] == 127).all() and (codes[rows] == 0).all() and not (scale == 255).any()


@by_type
def test_dequantize_every_code_and_scale(ms, dtype):
    codes = torch.arange(16, device=DEV).repeat(2).view(1, 32)
    codes = (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8).repeat(256, 1).contiguous()
    scale = torch.arange(256, device=DEV).to(torch.uint8).view(256, 1)
    want = torch.from_numpy(ref.values(codes.cpu().numpy(), scale.cpu().numpy())).to(dtype)
    got = ms.maxsim_dequantize_mx4(codes, scale, out_dtype=dtype).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine], want[fine])


@by_type
@pytest.mark.parametrize("T,d", ROWS)
def test_dequantize(ms, T, d, dtype):
    codes, scale = _random_mx4((T,), d, d)
    Y, ok = _guarded((T, d), dtype, -7.0)
    ms.maxsim_dequantize_mx4(codes, scale, d, Y=Y)
    torch.cuda.synchronize()
    assert ok()
    assert torch.equal(Y.double(), _values(codes, scale)[:, :d].to(dtype).double())


def test_rows_beyond_32_bit_offsets(ms):
    T, d = (1 << 32) // 256 + 9, 256
    x = torch.zeros(T, d, dtype=torch.float16, device=DEV)
    x[-9:] = _rows(9, d, torch.float16, 4)
    for normalize in (False, True):
        codes, scale = ms.maxsim_quantize_mx4(x, normalize=normalize)
        _check_codes((codes[-9:], scale[-9:]), ref.quantize(x[-9:].double().cpu().numpy(), normalize=normalize))
    y = ms.maxsim_dequantize_mx4(codes, scale, out_dtype=torch.float16)
    assert torch.equal(y[-9:].double(), _values(codes[-9:], scale[-9:]).half().double())


# ------------------------------------------------------------- product

LINEAR = [(1, 1, 1), (1, 16, 32), (2, 100, 33), (16, 3, 100), (17, 64, 768), (32, 257, 1000), (33, 128, 768), (1, 512, 4096),
          (40, 1, 64), (64, 64, 256), (65, 63, 257), (100, 200, 300), (130, 96, 1056), (300, 1001, 1000), (513, 128, 4096),
          (70, 70, 8192), (5, 33, 9000), (200, 40, 33)]


def _linear_want(A, As, W, Ws, bias):
    a, w = _values(A, As), _values(W, Ws)
    y = a @ w.T.contiguous()
    mag = a.abs() @ w.abs().T.contiguous()
    return (y if bias is None else y + bias.double()).cpu().numpy(), mag.cpu().numpy()


def _within(name, got, want, bound):
    off = np.abs(got.double().cpu().numpy() - want)
    bad = ~(off <= bound)
    assert not bad.any(), f"{name}: {bad.sum()} beyond the bound, first at {np.argwhere(bad)[0]}: " \
                          f"off {off[bad][0]:.3e}, bound {np.broadcast_to(bound, off.shape)[bad][0]:.3e}"


@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(ms, T, N, K):
    A, As = _random_mx4((T,), K, T + K, spread=6)
    W, Ws = _random_mx4((N,), K, N + K + 1, spread=6)
    for dtype, with_bias in ((torch.bfloat16, False), (torch.float16, True), (torch.float32, True)):
        bias = torch.randn(N, generator=_gen(N), device=DEV) if with_bias else None
        want, mag = _linear_want(A, As, W, Ws, bias)
        Y, ok = _guarded((T, N), dtype, -7.0)
        ms.maxsim_linear_mx4(A, As, W, Ws, bias, Y=Y)
        torch.cuda.synchronize()
        assert ok()
        b = 0.0 if bias is None else bias.double().cpu().numpy()
        fits = np.abs(want) < 60000 if dtype == torch.float16 else np.ones_like(want, bool)
        _within(str(dtype), torch.where(torch.from_numpy(fits).to(DEV), Y, 0), np.where(fits, want, 0),
                ref.linear_bound(want, mag, K, b, dtype))
    if As.numel() > 1:  # exponents at odd addresses
        assert torch.equal(ms.maxsim_linear_mx4(A, _off_by_one(As), W, _off_by_one(Ws), bias, out_dtype=torch.float32), Y)


@pytest.mark.parametrize("T,N,K", [(4096, 4096, 320), (2048, 4100, 512), (4100, 4099, 200)])
def test_linear_large_tiles(ms, T, N, K):
    A, As = _random_mx4((T,), K, 5, spread=3)
    W, Ws = _random_mx4((N,), K, 6, spread=3)
    want, mag = _linear_want(A, As, W, Ws, None)
    got = ms.maxsim_linear_mx4(A, As, W, Ws, out_dtype=torch.float32)
    _within("fp32", got, want, ref.linear_bound(want, mag, K, 0.0, torch.float32))


# Where 32 x 16 tiles are more than the CUs: 64 x 64 tiles with a ring of four steps, refilled
# from five steps on; 128 x 128 tiles, several a workgroup; 256 x 256 tiles. Steps of 8
# blocks and a rest, whole words of exponents (a multiple of 4 blocks) or not, outputs in rows
# that 16 bytes divide, that 8 divide, and that they don't.
TILES_64 = [(700, 600, K) for K in (100, 128, 256, 384, 1000, 1280, 1568, 2176, 2300)] + [(700, 601, 1280), (650, 604, 640)]
TILES_128 = [(2600, 4096, K) for K in (128, 256, 384, 512, 768, 1152, 1500)] + [(2600, 4099, 512), (2600, 4100, 640), (2560, 4096, 1024),
                                                                               (2050, 2100, 512)]
TILES_256 = [(4096, 4100, K) for K in (128, 512, 640, 1152)] + [(4000, 4096, 768), (4096, 4099, 512)]


@pytest.mark.parametrize("T,N,K", TILES_64 + TILES_128 + TILES_256)
def test_linear_of_every_tile(ms, T, N, K):
    test_linear(ms, T, N, K)


@pytest.mark.parametrize("T,N,K", [(700, 600, 1280), (2600, 4096, 512), (4096, 4100, 320)])
def test_linear_of_tiles_nan_and_overflow(ms, T, N, K):
    """NaN blocks give NaN rows and channels, products beyond the floats infinities of their
    sign, and neither reaches the others."""
    A, As = _random_mx4((T,), K, 1)
    W, Ws = _random_mx4((N,), K, 2)
    clean = ms.maxsim_linear_mx4(A, As, W, Ws, out_dtype=torch.float32)
    at, ch = [1, T // 2, T - 1], [0, N // 2, N - 1]
    for t, n in zip(at, ch):
        As[t, K // 32 - 1] = 255
        Ws[n, 1] = 255
    A[5], As[5] = 0x77, 254
    W[6], Ws[6] = 0x77, 254
    W[7], Ws[7] = 0xff, 254
    y = ms.maxsim_linear_mx4(A, As, W, Ws, out_dtype=torch.float32)
    assert torch.isnan(y[at]).all() and torch.isnan(y[:, ch]).all()
    assert y[5, 6] == float("inf") and y[5, 7] == -float("inf")
    rows, cols = torch.ones(T, dtype=torch.bool, device=DEV), torch.ones(N, dtype=torch.bool, device=DEV)
    rows[at + [5]] = False
    cols[ch + [6, 7]] = False
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    for _ in range(3):
        z = ms.maxsim_linear_mx4(A, As, W, Ws, out_dtype=torch.float32)
        assert torch.equal(torch.nan_to_num(z, nan=7.0), torch.nan_to_num(y, nan=7.0))


@pytest.mark.parametrize("T", [3, 40, 300])
def test_linear_nan_blocks_and_far_exponents(ms, T):
    K, N = 200, 70
    A, As = _random_mx4((T,), K, 1)
    W, Ws = _random_mx4((N,), K, 2)
    As[1, 3] = 255
    A[1, 48:64] = 0  # a block of zeros is NaN all the same
    Ws[5, 0] = 255
    Ws[6] = 0
    Ws[7] = 240
    y = ms.maxsim_linear_mx4(A, As, W, Ws, out_dtype=torch.float32)
    nan = torch.isnan(y)
    want = torch.zeros_like(nan)
    want[1] = True
    want[:, 5] = True
    assert torch.equal(nan, want)
    ref_y, mag = _linear_want(A, As, W, Ws, None)
    ok = ~want.cpu().numpy()
    bound = ref.linear_bound(ref_y, mag, K, 0.0, torch.float32)
    # products far below the others' range are subnormal sums: each addition rounds to 2^-149
    off = np.abs(y.double().cpu().numpy() - ref_y)
    assert (off[ok] <= bound[ok] + 64 * 2.0 ** -149).all()


def test_linear_rows_beyond_32_bit_offsets(ms):
    T, K, N = (1 << 33) // 16384 + 40, 16384 * 2, 40
    A = torch.zeros(T, K // 2, dtype=torch.uint8, device=DEV)
    As = torch.full((T, K // 32), 127, dtype=torch.uint8, device=DEV)
    A[-70:], As[-70:] = _random_mx4((70,), K, 1)
    W, Ws = _random_mx4((N,), K, 2)
    y = ms.maxsim_linear_mx4(A, As, W, Ws, out_dtype=torch.float32)
    want, mag = _linear_want(A[-70:], As[-70:], W, Ws, None)
    _within("last rows", y[-70:], want, ref.linear_bound(want, mag, K, 0.0, torch.float32))
    assert (y[:-70] == 0).all()


# ------------------------------------------------------------- scores

SCORE = [(1, 32, 3, 180, 128), (1, 1, 1, 1, 1), (2, 5, 7, 33, 31), (3, 20, 50, 77, 80), (1, 32, 300, 50, 128),
         (5, 33, 9, 64, 128), (9, 32, 40, 100, 128), (40, 7, 3, 31, 64), (2, 300, 5, 90, 128), (1, 1024, 4, 257, 128),
         (3, 70, 6, 45, 256), (2, 40, 10, 64, 384), (2, 32, 20, 70, 768), (2, 33, 5, 40, 1024), (1, 16, 4, 100, 1000),
         (3, 65, 4, 50, 200), (2, 260, 3, 40, 512), (1, 32, 2, 20000, 128), (2, 8, 70, 600, 96), (17, 16, 2, 2500, 128)]


def _check_scores(ms, Q, Qs, D, Ds, qm, dm, d, exact):
    Nq, Lq = Qs.shape[:2]
    Nd, Ld = Ds.shape[:2]
    want, sim, mag = ref.maxsim(_values(Q, Qs), _values(D, Ds), qm, dm)
    scores, ok1 = _guarded((Nq, Nd), torch.float32, -7.0)
    argmax, ok2 = _guarded((Nq, Nd, Lq), torch.int32, -7)
    ms.maxsim_fwd_mx4(Q, Qs, D, Ds, qm, dm, scores=scores, argmax=argmax)
    plain, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, qm, dm)
    torch.cuda.synchronize()
    assert ok1() and ok2()
    best = sim.amax(3)
    live = best > -np.inf
    err = torch.where(live, torch.from_numpy(ref.sim_error(mag.amax(3).cpu().numpy(), d)).to(DEV), 0.0)
    size = torch.where(live, best.abs(), 0.0)
    bound = err.sum(2) + 1.01 * (Lq + 8) * ref.U * size.sum(2) + ref.U * want.abs()
    for got in (scores, plain):
        if exact:
            assert torch.equal(got.double(), want)
        else:
            assert ((got.double() - want).abs() <= bound).all()
    a = argmax.long()
    assert ((a >= 0) & (a < Ld)).all()
    assert (a[~live] == 0).all()
    picked = sim.gather(3, a[..., None])[..., 0]
    first = (sim == best[..., None]).int().argmax(3)
    if exact:
        assert torch.equal(a[live], first[live])
    else:
        assert (picked >= best - 2 * err)[live].all()


@pytest.mark.parametrize("Nq,Lq,Nd,Ld,d", SCORE)
def test_scores(ms, Nq, Lq, Nd, Ld, d):
    for spread in (1, 5):  # one exponent: sums are exact, ties are many
        Q, Qs = _random_mx4((Nq, Lq), d, Lq + d, spread)
        D, Ds = _random_mx4((Nd, Ld), d, Ld + d, spread)
        _check_scores(ms, Q, Qs, D, Ds, None, None, d, spread == 1)
        qm, dm = _mask((Nq, Lq), 1), _mask((Nd, Ld), 2)
        dm[Nd // 2] = 0                                  # a document without a token
        if Nd > 2:
            dm[0, Ld // 2:] = 0                          # a padded one
            dm[1, :] = 0
            dm[1, Ld - 1] = 1                            # only the last token
        _check_scores(ms, Q, Qs, D, Ds, qm, dm, d, spread == 1)
    s, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, qm, dm)
    t, _ = ms.maxsim_fwd_mx4(Q, _off_by_one(Qs), D, _off_by_one(Ds), _off_by_one(qm), _off_by_one(dm))
    assert torch.equal(s, t)


@pytest.mark.parametrize("Nq,Lq,Nd,Ld", [(1, 32, 6, 70), (9, 40, 6, 70)])
def test_scores_nan(ms, Nq, Lq, Nd, Ld):
    """A NaN block shows in the scores that its token enters, and only there."""
    d = 128
    Q, Qs = _random_mx4((Nq, Lq), d, 1)
    D, Ds = _random_mx4((Nd, Ld), d, 2)
    clean, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds)
    Ds[2, 5, 1] = 255
    D[2, 5] = 0
    for want_argmax in (False, True):
        s, a = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, want_argmax=want_argmax)
        assert torch.isnan(s[:, 2]).all()
        keep = torch.arange(Nd, device=DEV) != 2
        assert torch.equal(s[:, keep], clean[:, keep])
        if a is not None:
            assert ((a >= 0) & (a < Ld)).all()
    dm = torch.ones(Nd, Ld, dtype=torch.uint8, device=DEV)
    dm[2, 5] = 0
    s, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm)
    assert not torch.isnan(s).any()
    Qs[0, 3, 0] = 255
    s, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm)
    assert torch.isnan(s[0]).all() and not torch.isnan(s[1:]).any()
    qm = torch.ones(Nq, Lq, dtype=torch.uint8, device=DEV)
    qm[0, 3] = 0
    s, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, qm, dm)
    assert not torch.isnan(s).any()


SHORT = [(1, 32, 9, 1, 128), (2, 40, 70, 2, 128), (5, 20, 333, 3, 80), (3, 5, 50, 4, 96), (9, 1, 100, 5, 64), (33, 2, 17, 7, 32),
         (20, 9, 31, 8, 100), (7, 16, 300, 9, 128), (2, 300, 40, 16, 128), (1, 130, 5, 13, 256), (6, 3, 64, 1, 200), (70, 16, 65, 2, 128),
         (3, 33, 40, 10, 384), (5, 8, 33, 16, 512), (4, 70, 21, 3, 768), (2, 17, 10, 6, 1024), (40, 4, 2000, 11, 128), (1, 1, 1, 1, 1)]


PACKED = [(2, 16, 9, 40, 128), (7, 9, 300, 50, 128), (33, 1, 40, 70, 64), (70, 2, 200, 33, 80), (9, 3, 20, 300, 200), (40, 5, 30, 65, 256),
          (5, 16, 700, 20, 96), (11, 8, 6, 100, 384), (6, 4, 9, 40, 512), (20, 12, 7, 35, 768), (3, 7, 5, 64, 1000), (200, 6, 60, 90, 128)]


@pytest.mark.parametrize("Nq,Lq,Nd,Ld,d", SHORT + PACKED)
def test_scores_of_short_documents_and_queries(ms, Nq, Lq, Nd, Ld, d):
    for spread in (1, 5):
        Q, Qs = _random_mx4((Nq, Lq), d, Lq + d, spread)
        D, Ds = _random_mx4((Nd, Ld), d, Ld + d, spread)
        _check_scores(ms, Q, Qs, D, Ds, None, None, d, spread == 1)
        qm, dm = _mask((Nq, Lq), 1), _mask((Nd, Ld), 2)
        dm[Nd // 2] = 0                                  # a document without a token
        qm[Nq // 2] = 0
        _check_scores(ms, Q, Qs, D, Ds, qm, dm, d, spread == 1)
    # a NaN block shows in the scores that its token enters, and only there
    clean, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds)
    Ds[Nd - 1, Ld - 1, 0] = 255
    got, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds)
    assert torch.isnan(got[:, -1]).all() and torch.equal(got[:, :-1], clean[:, :-1])
    dm = torch.ones(Nd, Ld, dtype=torch.uint8, device=DEV)
    dm[Nd - 1, Ld - 1] = 0
    got, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm)
    assert not torch.isnan(got).any() and torch.equal(got[:, :-1], clean[:, :-1])


@pytest.mark.parametrize("Nq,Lq,Nd,Ld,d", [(1, 32, 9, 70, 128), (9, 40, 6, 70, 100), (9, 3, 40, 40, 256), (2, 300, 5, 90, 128),
                                          (7, 16, 300, 9, 128), (40, 20, 300, 3, 200), (3, 20, 5, 17000, 64)])
def test_masked_tokens_beside_the_largest_exponents(ms, Nq, Lq, Nd, Ld, d):
    """Masked documents' tokens may hold anything: with the largest finite exponents, or
    NaN, beside queries of the largest ones, scores are those of harmless tokens."""
    Q, Qs = _random_mx4((Nq, Lq), d, 1, 1)
    Qs += 134  # 2^127
    D, Ds = _random_mx4((Nd, Ld), d, 2, 3)
    Ds -= 60   # 2^-67 and more, so that scores fit: 36 x 256 channels x 300 tokens x 2^60 x 2^3
    dm = _mask((Nd, Ld), 3, 0.6)
    dm[0] = 0
    _check_scores(ms, Q, Qs, D, Ds, None, dm, d, False)
    clean, arg = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm, want_argmax=True)
    for top in (254, 255):
        dirty = torch.where(dm[..., None] == 0, torch.tensor(top, dtype=torch.uint8, device=DEV), Ds)
        s, a = ms.maxsim_fwd_mx4(Q, Qs, D, dirty, None, dm, want_argmax=True)
        plain, _ = ms.maxsim_fwd_mx4(Q, Qs, D, dirty, None, dm)
        assert torch.equal(s, clean) and torch.equal(a, arg)
        assert torch.equal(plain, ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm)[0])


@pytest.mark.parametrize("Nq,Lq", [(1, 32), (3, 20), (9, 3), (2, 300)])
def test_argmax_of_similarities_that_overflow(ms, Nq, Lq):
    """Where every token that counts is at -Inf, the argmax is the first of them, not a masked one."""
    d, Nd, Ld = 128, 5, 70
    Q, Qs = torch.full((Nq, Lq, d // 2), 0x77, dtype=torch.uint8, device=DEV), torch.full((Nq, Lq, d // 32), 254, dtype=torch.uint8, device=DEV)
    D, Ds = torch.full((Nd, Ld, d // 2), 0xff, dtype=torch.uint8, device=DEV), torch.full((Nd, Ld, d // 32), 254, dtype=torch.uint8, device=DEV)
    dm = torch.ones(Nd, Ld, dtype=torch.uint8, device=DEV)
    first = [0, 5, 18, 45, 69]
    for j, t in enumerate(first):
        dm[j, :t] = 0
    dm[1, 6:40] = 0
    s, a = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm, want_argmax=True)
    assert (s == -float("inf")).all()
    assert torch.equal(a, torch.tensor(first, dtype=torch.int32, device=DEV)[None, :, None].expand(Nq, Nd, Lq))
    Ds[2, 60] = 100  # a finite one is larger
    Ds[4, 3] = 1     # but does not count
    s, a = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm, want_argmax=True)
    first[2] = 60
    assert torch.equal(a, torch.tensor(first, dtype=torch.int32, device=DEV)[None, :, None].expand(Nq, Nd, Lq))
    want = -36.0 * d * 2.0 ** (127 + 100 - 127) * Lq
    assert torch.allclose(s[:, 2].double(), torch.full((Nq,), want, dtype=torch.float64, device=DEV), rtol=1e-5, atol=0)
    assert (s[:, [0, 1, 3, 4]] == -float("inf")).all()


def _cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _up(n, b):
    return -(-n // b)


def _log2_up(n):
    return (n - 1).bit_length()


def _check_many_scores(ms, Nq, Lq, Nd, Ld, d, seed):
    """Without and with masks, aligned exponents and others; one exponent, where no sum
    rounds, if the largest possible score is below 2^24 quarters."""
    for spread in (1, 5):
        Q, Qs = _random_mx4((Nq, Lq), d, seed, spread)
        D, Ds = _random_mx4((Nd, Ld), d, seed + 1, spread)
        exact = spread == 1 and Lq * d * 144 < 1 << 24
        _check_scores(ms, Q, Qs, D, Ds, None, None, d, exact)
        qm, dm = _mask((Nq, Lq), 1), _mask((Nd, Ld), 2)
        dm[Nd // 2] = 0
        dm[-1] = 0
        dm[-1, -1] = 1
        qm[Nq // 2] = 0
        _check_scores(ms, Q, Qs, D, Ds, qm, dm, d, exact)
    s, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, qm, dm)
    t, _ = ms.maxsim_fwd_mx4(Q, _off_by_one(Qs), D, _off_by_one(Ds), _off_by_one(qm), _off_by_one(dm))
    assert torch.equal(s, t)
    want, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds)
    Ds[Nd - 1, Ld - 1, 0] = 255
    got, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds)
    assert torch.isnan(got[:, -1]).all() and torch.equal(got[:, :-1], want[:, :-1])
    dm = torch.ones(Nd, Ld, dtype=torch.uint8, device=DEV)
    dm[-1, -1] = 0
    got, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm)
    assert not torch.isnan(got).any() and torch.equal(got[:, :-1], want[:, :-1])


# Documents of up to 16 tokens share a tile where there are as many tiles as CUs, several
# query tiles a wave where there are 16 times as many. (Nq, Lq, whether many): queries that
# share tiles, of one tile, of two and three in one unit, of more than a unit holds; counts
# that units do not divide.
SHORT_QUERIES = [(1, 32, False), (3, 40, False), (20, 3, False), (1, 300, False), (70, 5, True), (9, 20, True), (7, 40, True),
                 (11, 70, True), (5, 300, True), (200, 1, True)]


@pytest.mark.parametrize("Nq,Lq,many", SHORT_QUERIES)
@pytest.mark.parametrize("d", [128, 96, 256, 200, 512, 1000])
@pytest.mark.parametrize("Ld", [1, 2, 3, 7, 16])
def test_scores_of_documents_that_share_tiles(ms, Ld, d, Nq, Lq, many):
    per = 32 >> _log2_up(Ld)
    tiles = Nq * _up(Lq, 32) if Lq > 32 else Nq if Lq > 16 else _up(Nq, 32 >> _log2_up(Lq))
    Nd = _up((16 if many else 1) * _cus(), tiles) * per + (1 if per > 1 else 0)
    _check_many_scores(ms, Nq, Lq, Nd, Ld, d, Ld + d)


# Queries of up to 16 tokens share tiles; four (two above 768 channels) tiles a wave where
# tiles times documents are 16 for each CU.
@pytest.mark.parametrize("Nq,Lq,many", [(200, 1, True), (70, 3, True), (39, 8, True), (13, 16, True), (5, 16, False), (40, 3, False)])
@pytest.mark.parametrize("d", [128, 80, 256, 200, 384, 300, 512, 768, 640, 1024, 1000])
def test_scores_of_queries_that_share_tiles(ms, d, Nq, Lq, many):
    tiles = _up(Nq, 32 >> _log2_up(Lq))
    Nd = _up(16 * _cus(), tiles) + 3 if many else 40
    _check_many_scores(ms, Nq, Lq, Nd, 33, d, d + Lq)


# Whole queries: as many tiles a wave, up to 8, as leave 8 documents' worth for each CU.
# (Nq, Lq, tiles a wave): one to three tiles a query, counts that units do not divide, and
# queries split over a workgroup's waves.
@pytest.mark.parametrize("Nq,Lq,n", [(11, 32, 8), (5, 40, 8), (5, 70, 8), (2, 300, 8), (11, 20, 4), (5, 40, 4), (3, 32, 2), (2, 130, 4)])
@pytest.mark.parametrize("d", [128, 100, 256, 200, 384, 512, 768, 1024])
def test_scores_of_several_queries_a_wave(ms, d, Nq, Lq, n):
    Nd = _up(n * 8 * _cus(), Nq * _up(Lq, 32)) + 1
    _check_many_scores(ms, Nq, Lq, Nd, 33 if Lq < 100 else 20, d, d + Lq)


# Little work: as few tiles a wave as the query's length leaves.
@pytest.mark.parametrize("Nq,Lq", [(1, 20), (2, 40), (1, 70), (1, 160), (2, 300), (2, 3), (3, 16)])
@pytest.mark.parametrize("d", [128, 100, 80, 256, 200, 384, 300, 512, 450, 768, 700, 1024, 1000, 900])
def test_scores_of_little_work(ms, d, Nq, Lq):
    _check_many_scores(ms, Nq, Lq, 5, 40, d, d + Lq)


def test_scores_without_tokens(ms):
    for Nq, Lq, Nd, Ld in ((2, 0, 3, 5), (2, 4, 3, 0), (0, 4, 3, 5), (2, 4, 0, 5), (2, 0, 3, 0)):
        Q, Qs = _random_mx4((Nq, Lq), 64, 1)
        D, Ds = _random_mx4((Nd, Ld), 64, 2)
        s, a = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, want_argmax=True)
        assert s.shape == (Nq, Nd) and (s == 0).all() and (a == 0).all()


def test_scores_of_many_queries(ms):
    """More queries than one launch takes, of one token and of several tiles."""
    for Nq, Lq, d in (((1 << 20) + 5, 1, 32), ((1 << 20) + 2, 40, 32)):
        Q, Qs = _random_mx4((7, Lq), d, 1, 1)  # sums are exact
        D, Ds = _random_mx4((2, 33), d, 2, 1)
        want, arg = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, want_argmax=True)
        of = torch.arange(Nq, device=DEV) % 7
        qm = torch.ones(Nq, Lq, dtype=torch.uint8, device=DEV)
        qm[-1] = 0
        s, a = ms.maxsim_fwd_mx4(Q[of].contiguous(), Qs[of].contiguous(), D, Ds, qm, want_argmax=True)
        assert torch.equal(s[:-1], want[of][:-1]) and torch.equal(a[:-1], arg[of][:-1])
        assert (s[-1] == 0).all()


def test_widest_rows(ms):
    """4096 blocks: quantised, multiplied and turned back without naming the width."""
    d = 131071
    x = _rows(3, d, torch.bfloat16, 1)
    codes, scale = ms.maxsim_quantize_mx4(x)
    assert scale.shape == (3, 4096)
    y = ms.maxsim_linear_mx4(codes, scale, codes, scale, out_dtype=torch.float32)
    want, mag = _linear_want(codes, scale, codes, scale, None)
    _within("product", y, want, ref.linear_bound(want, mag, d, 0.0, torch.float32))
    back = ms.maxsim_dequantize_mx4(codes, scale, out_dtype=torch.float32)
    assert torch.equal(back.double(), _values(codes, scale)[:, :d])


def test_scores_beyond_32_bit_offsets(ms):
    Nd, Ld, d = 70000, 1000, 128
    D = torch.zeros(Nd, Ld, d // 2, dtype=torch.uint8, device=DEV)
    Ds = torch.full((Nd, Ld, d // 32), 127, dtype=torch.uint8, device=DEV)
    D[-3:], Ds[-3:] = _random_mx4((3, Ld), d, 1)
    Q, Qs = _random_mx4((2, 32), d, 2)
    s, _ = ms.maxsim_fwd_mx4(Q, Qs, D, Ds)
    want, _, _ = ref.maxsim(_values(Q, Qs), _values(D[-3:], Ds[-3:]))
    assert torch.allclose(s[:, -3:].double(), want, rtol=1e-5, atol=0)
    assert (s[:, :-3] == 0).all()


# ------------------------------------------------------------- refusals, streams, graphs, runs

def test_refusals(ms):
    Q, Qs = _random_mx4((2, 4), 64, 1)
    x = torch.zeros(4, 64, device=DEV)
    for call in (lambda: ms.maxsim_quantize_mx4(x.t()),
                 lambda: ms.maxsim_quantize_mx4(x.cpu()),
                 lambda: ms.maxsim_quantize_mx4(x.int()),
                 lambda: ms.maxsim_quantize_mx4(x, torch.ones(3, dtype=torch.uint8, device=DEV)),
                 lambda: ms.maxsim_dequantize_mx4(Q, Qs, 100),
                 lambda: ms.maxsim_dequantize_mx4(Q, Qs[:, :, :1], 64),
                 lambda: ms.maxsim_dequantize_mx4(Q, Qs, out_dtype=torch.int8),
                 lambda: ms.maxsim_linear_mx4(Q, Qs, Q, Qs),
                 lambda: ms.maxsim_linear_mx4(Q, Qs, Q[0, :, :16].contiguous(), Qs[0, :, :1].contiguous()),
                 lambda: ms.maxsim_linear_mx4(Q, Qs, Q[0], Qs[0], torch.zeros(5, device=DEV)),
                 lambda: ms.maxsim_fwd_mx4(Q, Qs, Q[0], Qs[0]),
                 lambda: ms.maxsim_fwd_mx4(Q, Qs, Q, Qs, torch.ones(2, 5, dtype=torch.uint8, device=DEV)),
                 lambda: ms.maxsim_fwd_mx4(Q, Qs, Q.cpu(), Qs.cpu()),
                 lambda: ms.maxsim_fwd_mx4(Q.char(), Qs, Q, Qs)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ms.MaxSimError):  # 2048 channels
        B, Bs = _random_mx4((1, 2), 2048, 1)
        ms.maxsim_fwd_mx4(B, Bs, B, Bs)
    with pytest.raises(ms.MaxSimError):  # codes at an address that 16 does not divide
        ms.maxsim_dequantize_mx4(_off_by_one(Q), Qs)


def test_side_streams(ms):
    """Calls on streams of their own, outputs allocated there."""
    Q, Qs = _random_mx4((3, 32), 128, 1)
    Ds = [_random_mx4((200, 90), 128, 5 + i) for i in range(2)]
    want = [ms.maxsim_fwd_mx4(Q, Qs, *D)[0] for D in Ds]
    streams = [torch.cuda.Stream() for _ in Ds]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [ms.maxsim_fwd_mx4(Q, Qs, *D, stream=s)[0] for D, s in zip(Ds, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_serving_run(ms):
    """Hidden states to 4-bit embeddings, scan, top-k and exact rescoring: each
    step against float64 of the step's own inputs; then captured and replayed."""
    d, K, Nd, Ld, Nq, Lq = 128, 384, 60, 50, 4, 32
    Wf = torch.randn(d, K, generator=_gen(1), device=DEV) / K ** 0.5
    W, Ws = ms.maxsim_quantize_mx4(Wf)
    hd, hq = _rows(Nd * Ld, K, torch.bfloat16, 2).view(Nd, Ld, K), _rows(Nq * Lq, K, torch.bfloat16, 3).view(Nq, Lq, K)
    dm = _mask((Nd, Ld), 4)

    def run():
        D, Dsc = ms.embed_tokens_mx4(hd, W, Ws, mask=dm)
        Q, Qsc = ms.embed_tokens_mx4(hq, W, Ws)
        Df = ms.maxsim_dequantize_mx4(D, Dsc, d)
        Qf = ms.maxsim_dequantize_mx4(Q, Qsc, d)
        doc, val, scan = ms.two_stage_topk_mx4(Q, Qsc, D, Dsc, Qf, Df, 5, 20, None, dm)
        return D, Dsc, Q, Qsc, doc, val, scan

    D, Dsc, Q, Qsc, doc, val, scan = run()
    a, asc = ms.maxsim_quantize_mx4(hd, dm)
    y = ms.maxsim_linear_mx4(a, asc, W, Ws, out_dtype=torch.float32)
    _check_codes((D.view(-1, d // 2), Dsc.view(-1, d // 32)),
                 ref.quantize(y.view(-1, d).double().cpu().numpy(), dm.view(-1).cpu().numpy(), True))
    want, _, _ = ref.maxsim(_values(Q, Qsc), _values(D, Dsc), None, dm)
    assert torch.allclose(scan.double(), want, rtol=1e-5, atol=1e-5)
    # the embeddings are exact in 16 bits, so that rescoring gives the scan's scores again
    top = want.topk(5, 1)
    assert torch.allclose(val.double(), top.values, rtol=1e-5, atol=1e-5)
    assert torch.allclose(want.gather(1, doc.long()), top.values, rtol=1e-5, atol=1e-5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        hd.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        for x, z in zip(out, run()):
            assert torch.equal(x, z)


def test_bitwise_repeatable(ms):
    Q, Qs = _random_mx4((5, 70), 128, 1, 6)
    D, Ds = _random_mx4((300, 100), 128, 2, 6)
    A, As = _random_mx4((700,), 1000, 3, 6)
    first = None
    for _ in range(5):
        out = (*ms.maxsim_fwd_mx4(Q, Qs, D, Ds, want_argmax=True), ms.maxsim_linear_mx4(A, As, A[:90], As[:90]),
               ms.maxsim_linear_mx4(A[:9], As[:9], A[:90], As[:90]))
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))
