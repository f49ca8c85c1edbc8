"""The embedding head on the GPU against plain float64 forms (embed_reference.py,
which also derives the bounds). Codes, dropout masks and scales of masked rows
are compared exactly."""

import numpy as np
import pytest
import torch

import embed_reference as ref
from embed_reference import f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
short = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32", torch.int8: "i8"}
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
    x = torch.randn(T, d, generator=g, device=DEV) * torch.exp(torch.randn(T, 1, generator=g, device=DEV))
    return x.to(dtype)


def _mask(T, seed):
    """Some rows dropped; from three rows on at least one of them."""
    m = (torch.rand(T, generator=_gen(seed), device=DEV) < 0.7).to(torch.uint8)
    if T > 2:
        m[1] = 0
    return m


def _within(name, got, want, bound):
    off = np.abs(f64(got) - want)
    bad = ~(off <= bound)
    assert not bad.any(), f"{name}: {bad.sum()} beyond the bound, first at {np.argwhere(bad)[0]}: " \
                          f"off {off[bad][0]:.3e}, bound {np.broadcast_to(bound, off.shape)[bad][0]:.3e}"


def _guarded(shape, dtype, fill):
    """A tensor with a guard behind it: (tensor, check of the guard)."""
    n = int(np.prod(shape))
    buf = torch.full((n + 256,), fill, dtype=dtype, device=DEV)
    return buf[:n].view(shape), lambda: bool((buf[n:] == fill).all())


# ------------------------------------------------------------- quantisation

ROWS = [(1, 1), (1, 128), (3, 7), (5, 8), (37, 64), (33, 100), (1000, 128), (17, 200), (9, 516),
        (32, 768), (7, 1000), (3, 1030), (5, 2050), (4, 4096), (3, 8192), (2, 9001), (2, 16640),
        (1, 131071)]


@by_type
@pytest.mark.parametrize("T,d", ROWS)
def test_quantize(ms, T, d, dtype):
    x = _rows(T, d, dtype, T + d)
    m = _mask(T, d)
    dirty = x.clone()
    dirty[m == 0] = float("nan")
    for mask, normalize, given in ((None, False, x), (m, True, dirty)):
        codes, cg = _guarded((T, d), torch.int8, 77)
        scale, sg = _guarded((T,), torch.float32, -5.0)
        ms.maxsim_quantize_tok(given, mask, normalize=normalize, codes=codes, scale=scale)
        want, ws, _ = ref.quantize(f64(x), None if mask is None else f64(mask), normalize)
        assert np.array_equal(codes.cpu().numpy(), want)
        _within("scale", scale, ws, np.abs(ws) * (((ref.depth(d) + 3) / 2 + 3 if normalize else 1) * 1.01 * ref.U))
        assert cg() and sg()


def test_quantize_borders(ms):
    """Exact halves go to the even code; the float on either side of a half goes
    to its side, which float32 arithmetic alone would not decide."""
    k = torch.arange(-254, 255, device=DEV, dtype=torch.float32)
    x = torch.cat([k, k]).repeat(64, 1)
    # row r: magnitude 254 * s, so that 127 x / m = k / 2 exactly for x = k s
    s = torch.linspace(1.0, 1.9, 64, device=DEV).half().float()[:, None]
    x = x * s  # 9 x 11 bits: exact
    x[:, 509:] = torch.nextafter(x[:, 509:], torch.tensor(0.0, device=DEV))
    codes, _ = ms.maxsim_quantize_tok(x)
    want, _, gap = ref.quantize(f64(x))
    assert (gap == 0).sum() > 1000 and ((gap > 0) & (gap < 1e-4)).sum() > 1000
    assert np.array_equal(codes.cpu().numpy(), want)


@by_type
def test_empty_tiny_and_huge_rows(ms, dtype):
    top = float(torch.finfo(dtype).max)
    rows = [0.0, float(torch.finfo(dtype).smallest_normal), 1.0, top, top / 3]
    x = torch.tensor(rows, device=DEV)[:, None].to(dtype) * torch.ones(1, 96, device=DEV, dtype=dtype)
    x[:, ::5] *= -0.5
    if dtype == torch.float32:
        x = torch.cat([x, torch.full((1, 96), 2.0 ** -110, device=DEV), torch.full((1, 96), 1e-45, device=DEV),
                       torch.full((1, 96), 2.0 ** -100, device=DEV)])
    xd = f64(x)
    for normalize in (False, True):
        codes, scale = ms.maxsim_quantize_tok(x, normalize=normalize)
        want, ws, _ = ref.quantize(xd, None, normalize)
        assert np.array_equal(codes.cpu().numpy(), want)
        assert (scale > 0).all() and torch.isfinite(scale).all()
        _within("scale", scale, ws, np.abs(ws) * 100 * ref.U)
    y, rn = ms.maxsim_normalize_fwd(x, out_dtype=torch.float32)
    wy, wr = ref.normalize(xd)
    _within("unit rows", y, wy, ref.normalize_bound(wy, 96, torch.float32))
    # 1/norm of the largest rows is subnormal: half its last step
    _within("rnorm", rn, wr, np.abs(wr) * 100 * ref.U + 2.0 ** -149)


def test_rows_beyond_32_bit_offsets(ms):
    """4.4 GB of rows: element and byte offsets past 2^31 and 2^32."""
    T, d = 17_000_000, 128
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=_gen(3))
    at = torch.tensor([0, 1, T // 2, 8_388_608, 16_777_216, T - 2, T - 1], device=DEV)
    codes, scale = ms.maxsim_quantize_tok(x)
    want, ws, _ = ref.quantize(f64(x[at]))
    assert np.array_equal(codes[at].cpu().numpy(), want)
    _within("scale", scale[at], ws, ws * 2 * ref.U)
    del codes
    y, rn = ms.maxsim_normalize_fwd(x)
    wy, _ = ref.normalize(f64(x[at]))
    _within("unit rows", y[at], wy, ref.normalize_bound(wy, d, torch.bfloat16))
    del y
    p, seed = 0.5, 11
    z = ms.maxsim_dropout_fwd(x, p, seed)
    n = T * d
    for first in (0, 1 << 31, n - 64):
        gone = ref.dropped(64, p, seed, 0, first)
        got, src = f64(z.view(-1)[first:first + 64]), f64(x.view(-1)[first:first + 64])
        assert np.array_equal(got, np.where(gone, 0.0, 2 * src)), first  # twice a bf16 is exact


def test_more_rows_than_a_grid(ms):
    """Grids are capped and launches split; rows on both sides of every seam."""
    T = (1 << 28) + 77  # 2^22 workgroups of 64 rows
    x = torch.ones(T, 1, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, (1 << 28) - 1, 1 << 28, T - 1], device=DEV)
    x[at, 0] = torch.tensor([-2.0, 0.0, 4.0, -8.0], device=DEV).bfloat16()
    codes, scale = ms.maxsim_quantize_tok(x)
    assert codes[at, 0].tolist() == [-127, 0, 127, -127]
    assert torch.equal(scale[at], (torch.tensor([2.0, 127.0, 4.0, 8.0], device=DEV) / 127))
    assert bool((codes == 127).sum() == T - 3)
    del codes, scale
    y, rn = ms.maxsim_normalize_fwd(x)
    assert y[at, 0].tolist() == [-1, 0, 1, -1] and rn[at].tolist() == [0.5, 0, 0.25, 0.125]
    dx = ms.maxsim_normalize_bwd(x, rn, torch.ones(T, 1, device=DEV))
    assert not dx.any()  # a row of one value has no direction to change
    del x, y, rn, dx
    T, K, N = (1 << 26) + 333, 16, 5
    g = _gen(6)
    a = torch.empty(T, K, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    s = torch.rand(T, generator=g, device=DEV) + 0.5
    m = torch.ones(T, dtype=torch.uint8, device=DEV)
    _, _, w, ws, b = _operands(1, N, K, 8)
    at = torch.tensor([0, (1 << 24) - 1, 1 << 24, (1 << 26) - 1, 1 << 26, T - 1], device=DEV)
    m[at[2]] = 0
    y64, p64 = ref.linear(a[at].cpu().numpy(), f64(s[at]), w.cpu().numpy(), f64(ws), f64(b))
    y = ms.maxsim_linear_i8(a, s, w, ws, b)
    _within("product", y[at], y64, ref.linear_bound(y64, p64, torch.bfloat16))
    del y
    e, scale = ms.maxsim_embed_i8(a, s, w, ws, b, m)
    codes, want, gap = ref.quantize(y64, f64(m[at]), normalize=True)
    assert gap.min() > 1e-6 and np.array_equal(e[at].cpu().numpy(), codes)
    _within("scale", scale[at], want, want * 100 * ref.U)


def test_dropout_past_a_grid(ms):
    """2^22 workgroups of 2,048 elements and some more."""
    n = (1 << 33) + 1003
    x = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    windows = (0, (1 << 33) - 64, 1 << 33, n // 8 * 8 - 64)
    for i, first in enumerate(windows):
        x[first:first + 64] = torch.arange(1, 65, device=DEV) + i
    x[n - 3:] = 3
    y = ms.maxsim_dropout_fwd(x, 0.5, 21, 4)
    for i, first in enumerate(windows):
        gone = ref.dropped(64, 0.5, 21, 4, first)
        assert np.array_equal(f64(y[first:first + 64]), np.where(gone, 0.0, 2.0 * (np.arange(1, 65) + i))), first
    gone = ref.dropped(n % 8, 0.5, 21, 4, n // 8 * 8)
    assert np.array_equal(f64(y[n - 3:]), np.where(gone[-3:], 0.0, 6.0))


# ------------------------------------------------------------ normalisation

@by_type
@pytest.mark.parametrize("T,d", ROWS)
def test_normalize(ms, T, d, dtype):
    x = _rows(T, d, dtype, 3 * T + d)
    m = _mask(T, d + 1)
    dirty = x.clone()
    dirty[m == 0] = float("inf")
    for out in TYPES:
        y, yg = _guarded((T, d), out, 7.0)
        rn, rg = _guarded((T,), torch.float32, -5.0)
        ms.maxsim_normalize_fwd(dirty, m, Y=y, rnorm=rn)
        wy, wr = ref.normalize(f64(x), f64(m))
        _within("unit rows", y, wy, ref.normalize_bound(wy, d, out))
        _within("rnorm", rn, wr, np.abs(wr) * 1.01 * ((ref.depth(d) + 1) / 2 + 4) * ref.U)
        assert yg() and rg()
        # the gradient never looks at rows of rnorm 0
        g = torch.randn(T, d, generator=_gen(5), device=DEV)
        gd = g.clone()
        gd[rn == 0] = float("nan")
        dx, dg = _guarded((T, d), out, 7.0)
        ms.maxsim_normalize_bwd(dirty, rn, gd, dX=dx)
        want = ref.normalize_grad(f64(x), f64(rn), f64(g))
        _within("gradient", dx, want, ref.normalize_grad_bound(f64(x), f64(rn), f64(g), out))
        assert dg()


def test_normalize_gradient_by_differences(ms):
    """<dX, v> is the derivative of <dY, Y> along v. Central differences in
    float64 of step h are off by h^2 / 6 times the third derivative (below 20
    for unit v and rows of norm 1 .. 2), so by less than 4e-6; the kernel's
    gradient by its bound summed over the row."""
    x = _rows(6, 40, torch.float32, 1)
    x = x / x.norm(dim=1, keepdim=True) * torch.linspace(1, 2, 6, device=DEV)[:, None]
    g = torch.randn(6, 40, generator=_gen(2), device=DEV)
    g = g / g.norm(dim=1, keepdim=True)
    v = np.random.default_rng(0).standard_normal((6, 40))
    v /= np.linalg.norm(v, axis=1, keepdims=True)
    _, rn = ms.maxsim_normalize_fwd(x)
    dx = f64(ms.maxsim_normalize_bwd(x, rn, g))
    h = 1e-3
    up, down = ref.normalize(f64(x) + h * v)[0], ref.normalize(f64(x) - h * v)[0]
    slope = ((up - down) * f64(g)).sum(1) / (2 * h)
    assert np.abs((dx * v).sum(1) - slope).max() < 4e-6 + 40 * 20 * ref.U


def test_nan_in_one_row_stays_there_and_stays_visible(ms):
    x = _rows(70, 128, torch.bfloat16, 9)
    x[13, 5] = float("nan")
    y, rn = ms.maxsim_normalize_fwd(x)
    assert torch.isnan(y[13]).all() and not torch.isnan(y[torch.arange(70) != 13]).any()
    clean = _rows(70, 128, torch.bfloat16, 9)
    _, rn = ms.maxsim_normalize_fwd(clean)
    g = torch.ones(70, 128, device=DEV)
    g[20, 3] = float("inf")
    dx = ms.maxsim_normalize_bwd(clean, rn, g)
    assert not torch.isfinite(dx[20]).any() and torch.isfinite(dx[torch.arange(70) != 20]).all()


# ------------------------------------------------------------------ products

def _operands(T, N, K, seed, bias=True):
    g = _gen(seed)
    a = torch.randint(-128, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    s = torch.exp(torch.randn(T, generator=g, device=DEV)) / 127
    ws = torch.exp(torch.randn(N, generator=g, device=DEV)) / (127 * K ** 0.5)
    b = torch.randn(N, generator=g, device=DEV) if bias else None
    return a, s, w, ws, b


LINEAR = [
    # T, N, K: few tokens, every small tile, sizes around tile and chunk edges
    (1, 1, 1), (1, 16, 64), (1, 1000, 4096), (2, 130, 768), (16, 17, 100), (17, 128, 768),
    (31, 33, 15), (32, 512, 1024), (33, 64, 130), (64, 100, 2064), (65, 64, 128), (100, 300, 112),
    (128, 129, 1040), (300, 77, 999), (65, 65, 127), (1000, 1000, 1000), (500, 36, 16),
    (257, 4096, 256), (4000, 1030, 144), (2049, 2300, 400), (4097, 4112, 272), (5000, 4100, 77),
    (70, 128, 131071), (3, 20, 131071), (3, 20, 131056),
]


@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(ms, T, N, K):
    a, s, w, ws, b = _operands(T, N, K, T + N + K)
    y64, p64 = ref.linear(a.cpu().numpy(), f64(s), w.cpu().numpy(), f64(ws), f64(b))
    for out in TYPES:
        y, guard = _guarded((T, N), out, 7.0)
        ms.maxsim_linear_i8(a, s, w, ws, b, Y=y)
        _within("product", y, y64, ref.linear_bound(y64, p64, out))
        assert guard()
    y = ms.maxsim_linear_i8(a, s, w, ws, out_dtype=torch.float32)
    _within("without bias", y, p64, ref.linear_bound(p64, p64, torch.float32))


@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_extremes(ms, T):
    """-128 * -128 over the widest row: the largest sum int32 has to hold."""
    K = 131071
    a = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((20, K), -128, dtype=torch.int8, device=DEV)
    w[3] = 127
    one = torch.ones(T, device=DEV)
    y = ms.maxsim_linear_i8(a, one, w, torch.ones(20, device=DEV), out_dtype=torch.float32)
    want = torch.full((T, 20), 128.0 * 128 * K, device=DEV)
    want[:, 3] = -128.0 * 127 * K
    assert torch.equal(y, want)  # float32 of the whole numbers


@pytest.mark.parametrize("T", [2, 40])
def test_linear_most_channels(ms, T):
    """2^26 output channels: 1 GB of weights, 5 GB of outputs, launches in parts."""
    N, K = 1 << 26, 16
    g = _gen(T)
    a = torch.randint(-128, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.empty(N, K, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    s = torch.rand(T, generator=g, device=DEV) + 0.5
    ws = torch.rand(N, generator=g, device=DEV) + 0.5
    y = ms.maxsim_linear_i8(a, s, w, ws)
    at = torch.tensor([0, 1, (1 << 25) - 1, 1 << 25, N - 257, N - 1], device=DEV)
    y64, p64 = ref.linear(a.cpu().numpy(), f64(s), w[at].cpu().numpy(), f64(ws[at]))
    _within("product", y[:, at], y64, ref.linear_bound(y64, p64, torch.bfloat16))


def test_linear_rows_beyond_32_bit_offsets(ms):
    T, K, N = 4_300_000, 1024, 24
    g = _gen(4)
    a = torch.empty(T, K, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    s = torch.rand(T, generator=g, device=DEV) + 0.5
    _, _, w, ws, b = _operands(1, N, K, 8)
    at = torch.tensor([0, 2_097_152, 4_194_304, T - 300, T - 1], device=DEV)
    y64, p64 = ref.linear(a[at].cpu().numpy(), f64(s[at]), w.cpu().numpy(), f64(ws), f64(b))
    y = ms.maxsim_linear_i8(a, s, w, ws, b)
    _within("product", y[at], y64, ref.linear_bound(y64, p64, torch.bfloat16))
    e, _ = ms.maxsim_embed_i8(a, s, w, ws, b, out_dtype=torch.float16)
    _within("embedding", e[at], y64 / np.linalg.norm(y64, axis=1, keepdims=True),
            ref.embed_bound(y64, p64, torch.float16))


EMBED = [
    # T, d, K: few tokens and tiles at every width class
    (1, 1, 1), (1, 128, 768), (32, 128, 768), (33, 100, 130), (20, 129, 96), (17, 256, 768),
    (40, 300, 200), (50, 513, 1024), (10, 1024, 2048), (18, 1023, 77), (4097, 128, 768),
    (4500, 48, 300), (5000, 96, 77), (4200, 200, 256), (6000, 256, 400), (4300, 300, 96),
    (4100, 512, 1040), (4099, 513, 64), (5001, 1024, 320), (4098, 770, 130), (4200, 5, 33),
    (4120, 384, 72), (70, 600, 1000), (33, 768, 4096), (300, 128, 4096), (4200, 128, 8192), (4300, 250, 2049),
    # few tokens, wide rows: their channels spread over workgroups
    (32, 512, 1024), (100, 768, 300), (256, 1024, 77), (17, 272, 4096), (200, 1008, 33), (1, 1024, 64), (257, 784, 48),
    (32, 128, 2048), (512, 64, 4096), (513, 272, 600), (33, 256, 1001), (5, 16, 12000), (512, 1024, 200),
    # many tokens, a projection that stays in registers: every depth and width class
    (5000, 96, 128), (4999, 128, 384), (9000, 40, 640), (4111, 128, 1024), (40000, 128, 768),
    (4500, 130, 256), (4100, 256, 512), (9001, 250, 896), (5003, 200, 768), (20000, 256, 1024),
]


@pytest.mark.parametrize("T,d,K", EMBED)
def test_embed(ms, T, d, K):
    a, s, w, ws, b = _operands(T, d, K, T + 2 * d + K)
    m = torch.cat([torch.ones(T % 4, dtype=torch.uint8, device=DEV), _mask(T, d)])[T % 4:]  # any byte address
    s = torch.where(m != 0, s, float("nan"))  # what masked rows hold does not matter
    live = f64(m) != 0
    y64, p64 = ref.linear(a.cpu().numpy(), np.where(live, f64(s), 0.0), w.cpu().numpy(), f64(ws), f64(b))
    unit, _ = ref.normalize(y64, live)
    for out in TYPES:
        e, guard = _guarded((T, d), out, 7.0)
        got, none = ms.maxsim_embed_i8(a, s, w, ws, b, m, E=e)
        assert got is e and none is None
        _within("embedding", e, unit, np.where(live[:, None], ref.embed_bound(y64, p64, out), 0.0))
        assert guard()
    e, guard = _guarded((T, d), torch.int8, 77)
    scale, sg = _guarded((T,), torch.float32, -5.0)
    ms.maxsim_embed_i8(a, s, w, ws, b, m, E=e, e_scale=scale)
    codes, want, gap = ref.quantize(y64, live, normalize=True)
    # y rounds in float64 on both sides: nearer to a half than that is undecided.
    # Two roundings of 2^-53 of |p| + |b|, over the peak, times 127, twice over
    size = np.abs(p64).max(1) + float(b.abs().max())
    peak = np.where(live, np.abs(y64).max(1), 1.0)
    sure = gap > (size / peak * 127 * 16 * 2.0 ** -53)[:, None]
    assert np.array_equal(e.cpu().numpy()[sure], codes[sure])
    assert sure.mean() > 0.999
    _within("scale", scale, want, want * 1.01 * ((ref.depth(d) + 3) / 2 + 3) * ref.U)
    assert guard() and sg()


def test_embed_zero_rows(ms):
    a, s, w, ws, _ = _operands(40, 64, 96, 1)
    a[7] = 0
    e, scale = ms.maxsim_embed_i8(a, s, w, ws)
    assert (e[7] == 0).all() and scale[7] == 1 and (scale > 0).all()
    e, _ = ms.maxsim_embed_i8(a, s, w, ws, out_dtype=torch.bfloat16)
    assert (e[7] == 0).all() and torch.isfinite(e).all()


# ------------------------------------------------------------------- dropout

@by_type
@pytest.mark.parametrize("n", [1, 7, 8, 9, 127, 4095, 4096, 4097, 33333])
def test_dropout(ms, n, dtype):
    x = _rows(1, n, dtype, n).view(n)
    seed, step = 0x123456789ABCDEF0 + n, (1 << 40) + 5
    for p in (0.0, 1e-5, 0.1, 0.5, 0.999, 1.0):
        gone = ref.dropped(n, p, seed, step)
        dirty = x.clone()
        dirty[torch.from_numpy(gone).to(DEV)] = float("nan")  # dropped values do not matter
        y, guard = _guarded((n,), dtype, 7.0)
        ms.maxsim_dropout_fwd(dirty, p, seed, step, Y=y)
        want = ref.dropout(f64(x), p, gone)
        fits = np.abs(want) < float(torch.finfo(dtype).max)
        _within("kept", torch.where(torch.from_numpy(fits).to(DEV), y, 0), np.where(fits, want, 0.0),
                np.abs(want) * (1.01 * ref.U + ref.HALF[dtype]) + ref.FLOOR[dtype])
        assert (f64(y)[gone] == 0).all() and guard()
        assert torch.equal(ms.maxsim_dropout_bwd(x, p, seed, step), ms.maxsim_dropout_fwd(x, p, seed, step))


def test_dropout_shape_seed_and_rate(ms):
    x = torch.ones(1000, 1000, device=DEV)
    base = ms.maxsim_dropout_fwd(x, 0.3, 1)
    assert torch.equal(base.view(-1), ms.maxsim_dropout_fwd(x.view(-1), 0.3, 1))
    assert torch.equal(base, ms.maxsim_dropout_fwd(x, 0.3, 1))
    # a million independent draws: 6 standard deviations, other masks agree as often as chance has it
    q = round(0.3 * 65536) / 65536
    sd = (q * (1 - q) * 1e6) ** 0.5
    assert abs(int((base == 0).sum()) - q * 1e6) < 6 * sd
    for other in (ms.maxsim_dropout_fwd(x, 0.3, 2), ms.maxsim_dropout_fwd(x, 0.3, 1, step=1),
                  ms.maxsim_dropout_fwd(x, 0.3, 1 << 32), ms.maxsim_dropout_fwd(x, 0.3, 1, step=1 << 32)):
        both = int(((base == 0) & (other == 0)).sum())
        assert abs(both - q * q * 1e6) < 6 * (q * q * 1e6) ** 0.5


def test_dropout_step_in_device_memory(ms):
    x = torch.randn(5000, generator=_gen(1), device=DEV)
    dev = torch.tensor([1 << 35], dtype=torch.int64, device=DEV)
    assert torch.equal(ms.maxsim_dropout_fwd(x, 0.2, 9, step=3, step_dev=dev),
                       ms.maxsim_dropout_fwd(x, 0.2, 9, step=3 + (1 << 35)))
    dev.fill_(-1)  # modulo 2^64
    assert torch.equal(ms.maxsim_dropout_bwd(x, 0.2, 9, step=3, step_dev=dev),
                       ms.maxsim_dropout_bwd(x, 0.2, 9, step=2))


# ------------------------------------------------------ shapes, streams, graphs

def test_no_rows(ms):
    for lead in ((0,), (3, 0)):
        x = torch.empty(lead + (64,), dtype=torch.bfloat16, device=DEV)
        c, s = ms.maxsim_quantize_tok(x)
        assert c.shape == x.shape and s.shape == lead
        y, r = ms.maxsim_normalize_fwd(x)
        assert ms.maxsim_normalize_bwd(x, r, y.float()).shape == x.shape
        w, ws = torch.ones(8, 64, dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
        assert ms.maxsim_linear_i8(c, s, w, ws).shape == lead + (8,)
        assert ms.maxsim_embed_i8(c, s, w, ws)[1].shape == lead
        assert ms.maxsim_dropout_fwd(x, 0.5, 1).shape == x.shape


def test_one_row_without_leading_dimensions(ms):
    x = _rows(1, 200, torch.float32, 3).view(200)
    c, s = ms.maxsim_quantize_tok(x)
    assert c.shape == (200,) and s.shape == () and (c.abs() <= 127).all()
    y, r = ms.maxsim_normalize_fwd(x)
    assert y.shape == (200,) and abs(float(y.norm()) - 1) < 1e-5
    assert ms.maxsim_normalize_bwd(x, r, y).abs().max() < 1e-5  # along the row itself nothing changes


def test_leading_dimensions_and_refusals(ms):
    x = _rows(60, 64, torch.float16, 2).view(3, 4, 5, 64)
    m = _mask(60, 2).view(3, 4, 5)
    c, s = ms.maxsim_quantize_tok(x, m)
    c1, s1 = ms.maxsim_quantize_tok(x.view(60, 64), m.view(60))
    assert c.shape == x.shape and s.shape == m.shape and torch.equal(c.view(60, 64), c1) and torch.equal(s.view(60), s1)
    w, ws = torch.ones(8, 64, dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    assert ms.maxsim_embed_i8(c, s, w, ws, mask=m)[0].shape == (3, 4, 5, 8)
    cpu = torch.zeros(8)
    for call in (lambda: ms.maxsim_quantize_tok(x.transpose(0, 1)),            # not contiguous
                 lambda: ms.maxsim_quantize_tok(x, m.view(60)),                # mask shape
                 lambda: ms.maxsim_quantize_tok(x, m.bool()),                  # mask type
                 lambda: ms.maxsim_quantize_tok(x, codes=c.view(60, 64)),      # output shape
                 lambda: ms.maxsim_quantize_tok(x, scale=s.half()),            # output type
                 lambda: ms.maxsim_linear_i8(c, s.view(60), w, ws),
                 lambda: ms.maxsim_linear_i8(c, s, w, cpu),                    # another device
                 lambda: ms.maxsim_linear_i8(c, s, w, ws, bias=ws.half()),
                 lambda: ms.maxsim_embed_i8(c, s, w, ws, out_dtype=torch.float16, e_scale=s),
                 lambda: ms.maxsim_normalize_bwd(x, s, x),                     # dY is float32
                 lambda: ms.maxsim_dropout_fwd(x, 0.5, 1, step_dev=torch.zeros(1, device=DEV)),
                 lambda: ms.maxsim_dropout_fwd(x, 0.5, 1, step_dev=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ms.maxsim_dropout_fwd(x, 1.5, 1),
                 lambda: ms.maxsim_quantize_tok(x.view(-1)[1:3 * 64 + 1].view(3, 64)),  # not 16-byte aligned
                 lambda: ms.maxsim_embed_i8(c, s, torch.ones(1025, 64, dtype=torch.int8, device=DEV),
                                            torch.ones(1025, device=DEV))):
        with pytest.raises(ms.MaxSimError):
            call()


def test_side_streams(ms):
    """Two calls at once on streams of their own, outputs allocated there."""
    xs = [_rows(3000, 256, torch.bfloat16, 20 + i) for i in range(2)]
    w, ws = _operands(1, 128, 256, 5)[2:4]
    want = [ms.embed_tokens_i8(x, w, ws) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(5):
        got = [ms.embed_tokens_i8(x, w, ws, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for (e, s), (e0, s0) in zip(got, want):
        assert torch.equal(e, e0) and torch.equal(s, s0)


def test_captured_serving_run(ms):
    """Two captured graphs of the same operators, replayed in turn and at once
    on streams of their own, against the eager results."""
    w, ws = _operands(1, 128, 384, 5)[2:4]
    xs = [_rows(500 + 700 * i, 384, torch.bfloat16, 70 + i) for i in range(2)]
    graphs, outs = [], []
    for x in xs:
        ms.embed_tokens_i8(x, w, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ms.embed_tokens_i8(x, w, ws))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in xs]
    for i in range(4):
        for x in xs:
            x.mul_(-1.5)
        want = [ms.embed_tokens_i8(x, w, ws) for x in xs]
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (e, s), (e0, s0) in zip(outs, want):
            assert torch.equal(e, e0) and torch.equal(s, s0)


def test_captured_training_step(ms):
    """Dropout, normalisation, scoring and their gradients in a graph that is
    replayed with new inputs and steps; each replay against the eager calls."""
    Nq, Nd, Lq, Ld, d = 3, 4, 20, 50, 128
    hq = _rows(Nq * Lq, d, torch.float32, 31).view(Nq, Lq, d)
    hd = _rows(Nd * Ld, d, torch.float32, 32).view(Nd, Ld, d)
    gs = torch.randn(Nq, Nd, generator=_gen(33), device=DEV)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)

    def run():
        q, qn = ms.maxsim_normalize_fwd(ms.maxsim_dropout_fwd(hq, 0.1, 5, 0, step), out_dtype=torch.bfloat16)
        dd = ms.maxsim_dropout_fwd(hd, 0.1, 5, 1 << 32, step)
        k, kn = ms.maxsim_normalize_fwd(dd, out_dtype=torch.bfloat16)
        s, am = ms.maxsim_fwd(q, k, want_argmax=True)
        _, dk, _, _ = ms.maxsim_bwd(q, k, am, gs)
        return s, ms.maxsim_dropout_bwd(ms.maxsim_normalize_bwd(dd, kn, dk), 0.1, 5, 1 << 32, step)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    seen = []
    for i in range(4):
        step.fill_(i)
        hd.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
        seen.append(out[1].clone())
    assert all(not torch.equal(seen[0] == 0, x == 0) for x in seen[1:])


def test_serving_run(ms):
    """Hidden states to scores: quantise, project, normalise, scan, top-k,
    against float64 of the same codes."""
    Nq, Nd, Lq, Ld, K, d = 2, 30, 32, 40, 256, 128
    hq, hd = _rows(Nq * Lq, K, torch.bfloat16, 41).view(Nq, Lq, K), _rows(Nd * Ld, K, torch.bfloat16, 42).view(Nd, Ld, K)
    dm = _mask(Nd * Ld, 43).view(Nd, Ld)
    dm[:, 0] = 1
    w, ws = _operands(1, d, K, 44)[2:4]
    eq, sq = ms.embed_tokens_i8(hq, w, ws)
    ed, sd = ms.embed_tokens_i8(hd, w, ws, mask=dm)
    scores, _ = ms.maxsim_fwd_i8_tok(eq, sq, ed, sd, d_mask=dm)
    idx, val, _ = ms.maxsim_topk(scores, 5)

    def plain(h, mask):
        h = f64(h).reshape(-1, K)
        c, s, _ = ref.quantize(h, mask)
        y, _ = ref.linear(c, s, w.cpu().numpy(), f64(ws))
        return ref.normalize(y, mask)[0]

    q = plain(hq, None).reshape(Nq, Lq, d)
    k = plain(hd, f64(dm).reshape(-1)).reshape(Nd, Ld, d)
    sim = np.einsum("qsd,ntd->qnst", q, k)
    want = np.where(f64(dm)[None, :, None, :] != 0, sim, -np.inf).max(3).sum(2)
    # each embedding is off by at most half a step of its own scale per channel,
    # e = scale * sqrt(d) / 2 in norm, so a similarity by e_q + e_k + e_q e_k
    # (and float32 scoring by far less), a score by Lq of those
    eqn, ekn = float(sq.max()) * d ** 0.5 / 2, float(sd[dm != 0].max()) * d ** 0.5 / 2
    assert np.abs(f64(scores) - want).max() <= Lq * (eqn + ekn + eqn * ekn) * 1.01
    for i in range(Nq):
        assert torch.equal(idx[i].long(), torch.sort(scores[i], descending=True, stable=True).indices[:5])


def test_training_run_gradient(ms):
    """The gradient of the whole run (dropout, projection, normalisation, MaxSim)
    against float64 automatic differentiation with the same mask, argmax and
    16-bit embeddings' rounding left out of both."""
    Nq, Nd, Lq, Ld, K, d = 2, 3, 8, 24, 48, 64
    hq, hd = _rows(Nq * Lq, K, torch.float32, 51), _rows(Nd * Ld, K, torch.float32, 52)
    W = torch.randn(d, K, generator=_gen(53), device=DEV) / K ** 0.5
    gs = torch.randn(Nq, Nd, generator=_gen(54), device=DEV)
    p, seed = 0.25, 77
    dq, dk = ms.maxsim_dropout_fwd(hq, p, seed, 0), ms.maxsim_dropout_fwd(hd, p, seed, 1)
    pq, pk = dq @ W.T, dk @ W.T
    q, qn = ms.maxsim_normalize_fwd(pq, out_dtype=torch.float16)
    k, kn = ms.maxsim_normalize_fwd(pk, out_dtype=torch.float16)
    s, am = ms.maxsim_fwd(q.view(Nq, Lq, d), k.view(Nd, Ld, d), want_argmax=True)
    gq, gk, _, _ = ms.maxsim_bwd(q.view(Nq, Lq, d), k.view(Nd, Ld, d), am, gs)
    gpq = ms.maxsim_normalize_bwd(pq, qn, gq.view(-1, d))
    gpk = ms.maxsim_normalize_bwd(pk, kn, gk.view(-1, d))
    ghq, ghk = ms.maxsim_dropout_bwd(gpq @ W, p, seed, 0), ms.maxsim_dropout_bwd(gpk @ W, p, seed, 1)
    gW = gpq.T @ dq + gpk.T @ dk

    up = float(np.float32(65536 / (65536 - round(p * 65536))))
    leaf = [t.double().cpu().requires_grad_() for t in (hq, hd, W)]
    keep = [torch.from_numpy(~ref.dropped(t.numel(), p, seed, i)).view(t.shape) for i, t in enumerate((hq, hd))]
    eq, ek = ((leaf[i] * keep[i] * up) @ leaf[2].T for i in range(2))
    eq, ek = eq / eq.norm(dim=1, keepdim=True), ek / ek.norm(dim=1, keepdim=True)
    best = am.cpu().long()
    score = torch.stack([torch.stack([(eq.view(Nq, Lq, d)[i] * ek.view(Nd, Ld, d)[j][best[i, j]]).sum()
                                      for j in range(Nd)]) for i in range(Nq)])
    (score * gs.double().cpu()).sum().backward()
    # scoring's gradients are sums of at most Lq or Nd weighted fp16 rows, each
    # entry within 2^-11 of the row's own: relative to the gradients' largest
    # magnitude the fp16 rounding gives at most 2^-11 * sqrt(d) in each product,
    # float32 products of length 64 far less
    for got, want in ((ghq, leaf[0].grad), (ghk, leaf[1].grad), (gW, leaf[2].grad)):
        assert (got.double().cpu() - want).abs().max() <= want.abs().max() * 2.0 ** -11 * d ** 0.5
    assert (s.double().cpu() - score.detach()).abs().max() <= Lq * 2 * 2.0 ** -11 * 1.01


def test_bitwise_repeatable(ms):
    x = _rows(5000, 768, torch.bfloat16, 61)
    a, s, w, ws, b = _operands(5000, 384, 768, 62)
    few = _operands(40, 1024, 512, 63)
    for call in (lambda: ms.maxsim_quantize_tok(x, normalize=True), lambda: ms.maxsim_normalize_fwd(x),
                 lambda: ms.maxsim_embed_i8(*few),
                 lambda: ms.maxsim_embed_i8(a, s, w, ws, b), lambda: (ms.maxsim_linear_i8(a, s, w, ws, b),) * 2):
        first, again = call(), call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
