"""Log probabilities of columns of a score matrix on the GPU against plain float64
forms (logprob_reference.py, which also derives the bounds). Ranks and best columns
are compared exactly."""

import numpy as np
import pytest
import torch

import logprob_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
short = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
by_type = pytest.mark.parametrize("dtype", TYPES, ids=short.get)
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def ms():
    import maxsim_scoring_amd as m
    m.binding.lib()
    assert torch.cuda.is_available()
    return m


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _case(Nq, Nd, P, dtype, seed, masked):
    g = _gen(seed)
    x = (14 + 2 * torch.randn(Nq, Nd, generator=g, device=DEV)).to(dtype)
    t = torch.randint(0, max(1, Nd), (Nq, P), generator=g, device=DEV, dtype=torch.int32)
    mask = (torch.rand(Nq, Nd, generator=g, device=DEV) < 0.8).to(torch.uint8) if masked else None
    return x, t, mask


def _guarded(shape, dtype, fill):
    n = int(np.prod(shape))
    buf = torch.full((n + 64,), fill, dtype=dtype, device=DEV)
    return buf[:n].view(shape), lambda: bool((buf[n:] == fill).all())


def _close(name, got, want, bound):
    got = _np(got)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), name
    off = np.abs(got[fine] - want[fine])
    bad = ~(off <= np.broadcast_to(bound, want.shape)[fine])
    assert not bad.any(), f"{name}: {bad.sum()} beyond the bound: off {off[bad][0]:.3e}, " \
                          f"bound {np.broadcast_to(bound, want.shape)[fine][bad][0]:.3e}"


def _check_forward(ms, x, t, mask, scale, k):
    Nq, Nd = x.shape
    P = t.shape[1]
    outs, checks = {}, []
    for name, shape, dt in (("logp", (Nq, P), torch.float32), ("rank", (Nq, P), torch.int32), ("norm", (Nq, 2), torch.float32),
                            ("entropy", (Nq,), torch.float32), ("top_idx", (Nq, k), torch.int32), ("top_logp", (Nq, k), torch.float32)):
        outs[name], check = _guarded(shape, dt, -77)
        checks.append(check)
    need = ms.binding.lib().maxsim_logprob_workspace(Nq, Nd, P, k)
    ws, check = _guarded((need,), torch.uint8, 0x5A)
    ms.maxsim_logprob_fwd(x, t, mask, scale=scale, k=k, workspace=ws, **outs)
    torch.cuda.synchronize()
    assert all(c() for c in checks) and check()
    want, bound = ref.forward(_np(x), t.cpu().numpy(), _np(mask), np.float64(np.float32(scale)), k)
    for name in ("rank", "top_idx"):
        assert np.array_equal(outs[name].cpu().numpy(), want[name]), name
    for name in ("logp", "norm", "entropy", "top_logp"):
        _close(name, outs[name], want[name], bound[name])
    return outs


FORWARD = [(1, 1, 1, 1), (2, 2, 3, 2), (3, 63, 0, 5), (4, 64, 1, 0), (3, 65, 64, 65), (5, 128, 65, 20), (2, 1000, 200, 300),
           (3, 1024, 1, 1024), (2, 1025, 3, 7), (2, 4095, 5, 100), (3, 4096, 2, 1024), (3, 4097, 7, 33), (2, 10007, 130, 1024),
           (2, 100001, 8, 100), (1, 300000, 2, 50), (200, 17, 2, 4)]


@by_type
@pytest.mark.parametrize("Nq,Nd,P,k", FORWARD)
def test_forward(ms, Nq, Nd, P, k, dtype):
    for masked, scale in ((False, 1.0), (True, 3.7)):
        x, t, mask = _case(Nq, Nd, P, dtype, Nd + P, masked)
        _check_forward(ms, x, t, mask, scale, k)


@pytest.mark.parametrize("Nd", [40, 3000, 9000])
def test_forward_ties(ms, Nd):
    """Equal scores go by their column, also where they are far more than k."""
    g = _gen(1)
    t = torch.randint(0, Nd, (4, 9), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randint(0, 3, (4, Nd), generator=g, device=DEV).float()
    x[0] = 2.5
    x[1, ::2] = -0.0
    x[1, 1::2] = 0.0
    x[2] = -3.4028234663852886e38  # the type's lowest value is a score like others
    for k in (1, 30, min(Nd, 1000)):
        _check_forward(ms, x, t, None, 1.0, k)
    mask = torch.ones(4, Nd, dtype=torch.uint8, device=DEV)
    mask[:, :Nd // 2] = 0
    _check_forward(ms, x, t, mask, 1.0, 30)


@by_type
@pytest.mark.parametrize("Nd", [40, 3000, 9000])
def test_forward_empty_and_short_rows(ms, Nd, dtype):
    x, t, mask = _case(6, Nd, 12, dtype, 3, True)
    mask[0] = 0                         # nothing left
    mask[1] = 0
    mask[1, Nd - 3] = 1                 # one column
    x[2] = -float("inf")                # masked by its scores
    x[3, 5:] = -float("inf")
    x[4, 0] = torch.finfo(dtype).min
    x[5, mask[5] == 0] = float("nan")   # masked columns are not looked at
    t[:, 0] = Nd - 3
    t[:, 1] = -1
    t[:, 2] = Nd
    t[:, 3] = -2 ** 31
    t[:, 4] = 2 ** 31 - 1
    t[:, 5] = t[:, 6]
    out = _check_forward(ms, x, t, mask, 2.0, 20)
    assert (out["entropy"][:1] == 0).all() and (out["rank"][0] == -1).all()
    g = torch.randn(6, 12, generator=_gen(4), device=DEV)
    gh = torch.randn(6, generator=_gen(5), device=DEV)
    dX = ms.maxsim_logprob_bwd(x, t, out["norm"], g, mask, scale=2.0, entropy=out["entropy"], grad_entropy=gh)
    assert (dX[0] == 0).all() and (dX[2] == 0).all() and not torch.isnan(dX).any()
    assert (dX[mask == 0] == 0).all()


@pytest.mark.parametrize("Nd", [40, 3000, 9000])
def test_nan_and_infinity_stay_in_their_row(ms, Nd):
    x, t, _ = _case(5, Nd, 4, torch.float32, 6, False)
    clean = ms.maxsim_logprob_fwd(x, t, k=10)
    x[1, Nd - 1] = float("nan")
    x[3, 2] = float("inf")
    out = ms.maxsim_logprob_fwd(x, t, k=10)
    good = torch.tensor([True, False, True, False, True], device=DEV)
    for a, b in zip(out, clean):
        assert torch.equal(a[good], b[good])
        if a.dtype == torch.float32:
            assert torch.isnan(a[~good]).all()
        else:
            assert ((a >= -1) & (a < Nd)).all()
    dX = ms.maxsim_logprob_bwd(x, t, out[2], torch.ones(5, 4, device=DEV))
    assert torch.isnan(dX[~good]).all() and not torch.isnan(dX[good]).any()


def test_peaked_rows_keep_their_entropy(ms):
    """Probabilities next to 1: the entropy is the small rest, not lost in a rounded sum."""
    for Nd in (100, 6000):
        x = torch.zeros(3, Nd, device=DEV)
        x[0, 7], x[1, Nd - 1], x[2, 50] = 20.0, 30.0, 60.0
        t = torch.tensor([[7], [Nd - 1], [50]], dtype=torch.int32, device=DEV)
        _, _, norm, entropy, _, _ = ms.maxsim_logprob_fwd(x, t)
        z = -_np(x.amax(1))
        s = (Nd - 1) * np.exp(z)
        want = np.log1p(s) - s * z / (1 + s)
        # a float64 sum of 1 and s is off by up to 2^-53, and so are its logarithm and L
        for got, exact in ((entropy, want), (norm[:, 1], np.log1p(s))):
            assert np.allclose(_np(got), exact, rtol=1e-5, atol=2.0 ** -52)


@pytest.mark.parametrize("Nd", [100, 800, 6000])
def test_peaked_rows_keep_their_gradient(ms, Nd):
    """The gradient of a column whose probability is next to 1 is the small rest too:
    A (1 - p) - p (R + gH (log p + H)), A the gradients that name it, R the others'.
    With s = (Nd - 1) exp(z) the rest is s / (1 + s). s is off by 4 |z| + 6 units (u = 2^-24),
    and 34 are for L, H and the sums rounded to 32 bits, the exponential and the products.
    1 + s is a float64 sum whose partial sums pass 1: 15 additions in the thread that holds
    the 1, 6 over its wave, 3 over the waves, and 1 + 6 + 7 where chunks are joined, 38 in
    all, each off by 2^-53 of 1 at most: less than 2^-47."""
    u = 2.0 ** -24
    for scale, tops in ((1.0, (20.0, 30.0, 60.0)), (2.0, (8.0, 12.0, 17.0))):
        for case in range(3):
            x = torch.zeros(3, Nd, device=DEV)
            at = [7, Nd - 1, 50]
            for i in range(3):
                x[i, at[i]] = tops[i]
            # the sure column alone; named twice; beside another one, with the entropy
            names = [[[c] for c in at], [[c, c] for c in at], [[c, 3] for c in at]][case]
            t = torch.tensor(names, dtype=torch.int32, device=DEV)
            g = torch.tensor([[1.0], [0.7, 0.45], [1.5, -1e-7]][case], device=DEV).expand(3, -1).contiguous()
            gh = torch.full((3,), 0.3, device=DEV) if case == 2 else None
            out = ms.maxsim_logprob_fwd(x, t, scale=scale)
            dX = _np(ms.maxsim_logprob_bwd(x, t, out[2], g, scale=scale, entropy=out[3] if case == 2 else None, grad_entropy=gh))
            gs = _np(g)[0]
            A, R, h = (gs.sum(), 0.0, 0.0) if case < 2 else (gs[0], gs[1], float(gh[0]))
            for i in range(3):
                z = -scale * tops[i]
                s = (Nd - 1) * np.exp(z)
                L = np.log1p(s)
                parts = np.array([A * s / (1 + s), -R / (1 + s), -h * (-s * z / (1 + s)) / (1 + s)])  # log p + H = -s z / (1 + s)
                rtol = 1.01 * u * (4 * abs(z) + 40)
                assert abs(dX[i, at[i]] - scale * parts.sum()) <= scale * (rtol * np.abs(parts).sum() + 2.0 ** -47 * (A + 100 * h)), (case, i)
                # the columns' gradients cancel
                assert abs(dX[i].sum()) <= rtol * np.abs(dX[i]).sum() + scale * 2.0 ** -47 * (A + 100 * h), (case, i)


def _random_shape(seed):
    r = np.random.default_rng(seed)
    Nd = int(np.exp(r.uniform(0, np.log(60000))))
    return int(r.integers(1, 6)), Nd, int(r.integers(0, 80)), int(r.integers(0, min(Nd, 300) + 1))


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(ms, seed):
    Nq, Nd, P, k = _random_shape(seed)
    dtype = TYPES[seed % 3]
    x, t, mask = _case(Nq, Nd, P, dtype, seed, seed % 2 == 1)
    out = _check_forward(ms, x, t, mask, 0.5 + seed, k)
    _check_backward(ms, x, t, mask, 0.5 + seed, out, seed % 4 < 2, torch.float32)


def _check_backward(ms, x, t, mask, scale, out, with_entropy, to):
    Nq, Nd = x.shape
    g = torch.randn(*t.shape, generator=_gen(7), device=DEV)
    gh = torch.randn(Nq, generator=_gen(8), device=DEV) if with_entropy else None
    dX, check = _guarded((Nq, Nd), to, -77)
    ms.maxsim_logprob_bwd(x, t, out["norm"], g, mask, scale=scale, entropy=out["entropy"] if with_entropy else None,
                          grad_entropy=gh, dX=dX)
    torch.cuda.synchronize()
    assert check()
    want, bound = ref.backward(_np(x), t.cpu().numpy(), _np(mask), np.float64(np.float32(scale)), _np(g), _np(out["norm"]),
                               _np(out["entropy"]), _np(gh))
    _close("dX", dX, want, bound + np.abs(want) * HALF[to] + FLOOR[to])


BACKWARD = [(1, 1, 1), (2, 2, 3), (3, 63, 0), (5, 128, 65), (2, 1024, 1), (2, 1025, 3), (3, 4096, 300), (3, 4097, 1),
            (2, 10007, 1000), (2, 100001, 32), (2, 50, 5000)]


@by_type
@pytest.mark.parametrize("Nq,Nd,P", BACKWARD)
def test_backward(ms, Nq, Nd, P, dtype):
    for masked, with_entropy, to in ((False, False, torch.float32), (True, True, torch.float32), (True, True, dtype)):
        x, t, mask = _case(Nq, Nd, P, dtype, Nd + P, masked)
        if P > 2:
            t[:, 1] = t[:, 0]
            t[0, 2] = Nd + 5
        outs = ms.maxsim_logprob_fwd(x, t, mask, scale=1.5)
        _check_backward(ms, x, t, mask, 1.5, {"norm": outs[2], "entropy": outs[3]}, with_entropy, to)


def test_backward_by_differences(ms):
    """Central differences of the float64 forward: with steps of 2^-12 they are within
    2^-24 / 6 times the third derivative of the gradient, which is below 30 scale^3
    times the sum of the upstream gradients here (each p has derivatives of at most 6)."""
    Nq, Nd, P, scale = 3, 30, 4, 1.3
    x, t, mask = _case(Nq, Nd, P, torch.float32, 11, True)
    t[:, 1] = t[:, 0]
    mask.scatter_(1, t.long(), 1)
    g, gh = torch.randn(Nq, P, generator=_gen(1), device=DEV), torch.randn(Nq, generator=_gen(2), device=DEV)
    out = ms.maxsim_logprob_fwd(x, t, mask, scale=scale)
    got = _np(ms.maxsim_logprob_bwd(x, t, out[2], g, mask, scale=scale, entropy=out[3], grad_entropy=gh))
    xs, s64 = _np(x), np.float64(np.float32(scale))

    def loss(v):
        o, _ = ref.forward(v, t.cpu().numpy(), _np(mask), s64, 0)
        return ((_np(g) * o["logp"]).sum(1) + _np(gh) * o["entropy"])

    size = np.abs(_np(g)).sum(1) + np.abs(_np(gh)) * 30
    for c in range(Nd):
        up, dn = xs.copy(), xs.copy()
        up[:, c] += 2.0 ** -12
        dn[:, c] -= 2.0 ** -12
        diff = (loss(up) - loss(dn)) / 2.0 ** -11
        assert (np.abs(got[:, c] - diff) <= size * (2.0 ** -24 * 5 * s64 ** 3 + 1e-6)).all()


def test_rows_beyond_32_bit_offsets(ms):
    Nq, Nd = 33000, 70001
    x = torch.zeros(Nq, Nd, dtype=torch.float16, device=DEV)
    x[-2:] = torch.randn(2, Nd, generator=_gen(1), device=DEV).half()
    t = torch.randint(0, Nd, (Nq, 2), generator=_gen(2), device=DEV, dtype=torch.int32)
    out = ms.maxsim_logprob_fwd(x, t, k=3)
    want, bound = ref.forward(_np(x[-2:]), t[-2:].cpu().numpy(), None, 1.0, 3)
    for name, o in zip(("logp", "rank", "norm", "entropy", "top_idx", "top_logp"), out):
        if o.dtype == torch.int32:
            assert np.array_equal(o[-2:].cpu().numpy(), want[name])
        else:
            _close(name, o[-2:], want[name], bound[name])
    assert torch.equal(out[4][:-2], torch.arange(3, device=DEV, dtype=torch.int32).expand(Nq - 2, 3))
    g = torch.ones(Nq, 2, device=DEV)
    dX = ms.maxsim_logprob_bwd(x, t, out[2], g, out_dtype=torch.float16)
    want, bound = ref.backward(_np(x[-2:]), t[-2:].cpu().numpy(), None, 1.0, _np(g[-2:]), _np(out[2][-2:]))
    _close("dX", dX[-2:], want, bound + np.abs(want) * HALF[torch.float16] + FLOOR[torch.float16])


@pytest.mark.parametrize("Nd,P,k", [(2200001, 600, 1024), (2200001, 3, 1)])
def test_long_rows(ms, Nd, P, k):
    """More chunks, and more targets, than the join has threads."""
    x, t, mask = _case(1, Nd, P, torch.float32, 3, k > 1)
    out = _check_forward(ms, x, t, mask, 2.0, k)
    _check_backward(ms, x, t, mask, 2.0, out, True, torch.float32)


def test_many_rows(ms):
    """More rows than one launch takes."""
    Nq = (1 << 22) + 3
    x = torch.zeros(Nq, 3, device=DEV)
    x[-2:] = torch.tensor([[1.0, 5.0, 2.0], [7.0, -3.0, 7.5]], device=DEV)
    t = torch.ones(Nq, 1, dtype=torch.int32, device=DEV)
    out = ms.maxsim_logprob_fwd(x, t, k=2)
    g = torch.ones(Nq, 1, device=DEV)
    dX = ms.maxsim_logprob_bwd(x, t, out[2], g)
    assert all(torch.equal(o[:1].expand_as(o[:-2]), o[:-2]) for o in (*out, dX))
    want, bound = ref.forward(_np(x[-3:]), t[-3:].cpu().numpy(), None, 1.0, 2)
    for name, o in zip(("logp", "rank", "norm", "entropy", "top_idx", "top_logp"), out):
        if o.dtype == torch.int32:
            assert np.array_equal(o[-3:].cpu().numpy(), want[name])
        else:
            _close(name, o[-3:], want[name], bound[name])
    want, bound = ref.backward(_np(x[-3:]), t[-3:].cpu().numpy(), None, 1.0, _np(g[-3:]), _np(out[2][-3:]))
    _close("dX", dX[-3:], want, bound)


@pytest.mark.parametrize("Nd", [40, 6000])
def test_the_whole_range_of_scores(ms, Nd):
    """Differences of scores beyond the largest float: those columns' log probabilities
    are finite after the scale, their probabilities 0."""
    low, high, scale = -3.4028234663852886e38, 3.0e38, 2.0 ** -64
    x = torch.full((1, Nd), low, device=DEV)
    x[0, 5] = high
    t = torch.tensor([[5, 0, Nd - 1]], dtype=torch.int32, device=DEV)
    logp, rank, norm, entropy, top_idx, top_logp = ms.maxsim_logprob_fwd(x, t, scale=scale, k=3)
    far = torch.tensor(scale * (low - float(x[0, 5])), dtype=torch.float64).float().item()
    assert logp.tolist() == [[0.0, far, far]] and rank.tolist() == [[0, 1, Nd - 1]]
    assert entropy.tolist() == [0.0] and top_idx.tolist() == [[5, 0, 1]] and top_logp.tolist() == [[0.0, far, far]]
    dX = ms.maxsim_logprob_bwd(x, t, norm, torch.ones(1, 3, device=DEV), scale=scale, entropy=entropy,
                               grad_entropy=torch.ones(1, device=DEV))
    # the named ones 1, the sure one 1 - 3
    want = torch.zeros(Nd, device=DEV)
    want[0] = want[Nd - 1] = scale
    want[5] = -2 * scale
    assert torch.equal(dX[0], want)


def test_unaligned_rows(ms):
    """Scores and masks at any element, as views into larger buffers."""
    for dtype in TYPES:
        x, t, mask = _case(3, 5001, 4, dtype, 2, True)
        buf, mbuf = torch.empty(x.numel() + 1, dtype=dtype, device=DEV), torch.empty(x.numel() + 1, dtype=torch.uint8, device=DEV)
        buf[1:], mbuf[1:] = x.view(-1), mask.view(-1)
        a = ms.maxsim_logprob_fwd(x, t, mask, k=20)
        b = ms.maxsim_logprob_fwd(buf[1:].view(3, 5001), t, mbuf[1:].view(3, 5001), k=20)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals(ms):
    x, t, mask = _case(3, 50, 2, torch.float32, 1, True)
    out = ms.maxsim_logprob_fwd(x, t)
    g = torch.ones(3, 2, device=DEV)
    for call in (lambda: ms.maxsim_logprob_fwd(x.cpu(), t),
                 lambda: ms.maxsim_logprob_fwd(x.double(), t),
                 lambda: ms.maxsim_logprob_fwd(x[0], t),
                 lambda: ms.maxsim_logprob_fwd(x.t(), t[:1].expand(50, 2)),
                 lambda: ms.maxsim_logprob_fwd(x, t.long()),
                 lambda: ms.maxsim_logprob_fwd(x, t[:2]),
                 lambda: ms.maxsim_logprob_fwd(x, t, mask[:2]),
                 lambda: ms.maxsim_logprob_fwd(x, t, k=1025),
                 lambda: ms.maxsim_logprob_fwd(x, t, k=-1),
                 lambda: ms.maxsim_logprob_fwd(torch.zeros(1, 5000, device=DEV), t[:1], k=3,
                                               workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
                 lambda: ms.maxsim_logprob_bwd(x, t, out[2][:2], g),
                 lambda: ms.maxsim_logprob_bwd(x, t, out[2], g.double()),
                 lambda: ms.maxsim_logprob_bwd(x, t, out[2], g, entropy=out[3]),
                 lambda: ms.maxsim_logprob_bwd(x, t, out[2], g, out_dtype=torch.int8)):
        with pytest.raises(ValueError):
            call()
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ms.MaxSimError):
            ms.maxsim_logprob_fwd(x, t, scale=scale)
        with pytest.raises(ms.MaxSimError):
            ms.maxsim_logprob_bwd(x, t, out[2], g, scale=scale)


def test_no_rows_and_no_columns(ms):
    for Nq, Nd in ((0, 5), (3, 0)):
        x = torch.zeros(Nq, Nd, device=DEV)
        t = torch.zeros(Nq, 2, dtype=torch.int32, device=DEV)
        logp, rank, norm, entropy, idx, top = ms.maxsim_logprob_fwd(x, t, k=3)
        assert (logp == 0).all() and (rank == -1).all() and (norm == -float("inf")).all() and (entropy == 0).all()
        assert (idx == -1).all() and (top == -float("inf")).all()
        assert ms.maxsim_logprob_bwd(x, t, norm, torch.ones(Nq, 2, device=DEV)).shape == (Nq, Nd)


def test_side_streams_and_bitwise_repeatable(ms):
    xs = [_case(20, 30000, 5, torch.float32, i, False) for i in range(2)]
    want = [ms.maxsim_logprob_fwd(x, t, k=64) for x, t, _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [ms.maxsim_logprob_fwd(x, t, k=64, stream=s) for (x, t, _), s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    x, t, _ = xs[0]
    t[:, 1] = t[:, 0]
    g = torch.randn(20, 5, generator=_gen(1), device=DEV)
    first = ms.maxsim_logprob_bwd(x, t, want[0][2], g)
    for _ in range(5):
        assert torch.equal(first, ms.maxsim_logprob_bwd(x, t, want[0][2], g))


def test_captured_runs_replay_at_once(ms):
    """Two graphs of rows of several chunks, each with a workspace of its own."""
    cases = [_case(9, 20000 + 5000 * i, 6, torch.float32, i, True) for i in range(2)]
    g = torch.randn(9, 6, generator=_gen(1), device=DEV)

    def run(x, t, mask):
        o = ms.maxsim_logprob_fwd(x, t, mask, scale=1.5, k=50)
        return (*o, ms.maxsim_logprob_bwd(x, t, o[2], g, mask, scale=1.5, entropy=o[3], grad_entropy=o[3]))

    graphs, outs = [], []
    for c in cases:
        run(*c)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(*c))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in cases]
    for i in range(4):
        for x, _, _ in cases:
            x.copy_(14 + 2 * torch.randn(x.shape, generator=_gen(50 + i), device=DEV))
        want = [run(*c) for c in cases]
        for graph, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_training_run(ms):
    """A step of contrastive training on 4-bit scores: float embeddings are quantised,
    scored with their argmax, the loss is -log p of each query's document and an
    entropy term, and the gradient goes back through the argmax to the embeddings
    that the codes stand for. Against the gradient formula in float64; captured and
    replayed beside it."""
    Nq, Nd, Lq, Ld, d, scale = 4, 6, 10, 40, 128, 1.7
    qf = torch.nn.functional.normalize(torch.randn(Nq, Lq, d, generator=_gen(1), device=DEV), dim=2)
    df = torch.nn.functional.normalize(torch.randn(Nd, Ld, d, generator=_gen(2), device=DEV), dim=2)
    dm = (torch.rand(Nd, Ld, generator=_gen(3), device=DEV) < 0.8).to(torch.uint8)
    t = torch.arange(Nq, dtype=torch.int32, device=DEV)[:, None].contiguous()
    g = torch.full((Nq, 1), -1.0 / Nq, device=DEV)
    gh = torch.full((Nq,), 0.1 / Nq, device=DEV)

    def run():
        Q, Qs = ms.maxsim_quantize_mx4(qf, normalize=True)
        D, Ds = ms.maxsim_quantize_mx4(df, dm, normalize=True)
        s, am = ms.maxsim_fwd_mx4(Q, Qs, D, Ds, None, dm, want_argmax=True)
        logp, rank, norm, entropy, idx, _ = ms.maxsim_logprob_fwd(s, t, scale=scale, k=3)
        ds = ms.maxsim_logprob_bwd(s, t, norm, g, scale=scale, entropy=entropy, grad_entropy=gh)
        q, k = ms.maxsim_dequantize_mx4(Q, Qs, d), ms.maxsim_dequantize_mx4(D, Ds, d)
        dq, dd, _, _ = ms.maxsim_bwd(q, k, am, ds, None, dm)
        return q, k, s, logp, rank, entropy, idx, dq, dd

    q, k, s, logp, rank, entropy, idx, dq, dd = run()
    q64, k64 = q.double().cpu().requires_grad_(), k.double().cpu().requires_grad_()
    sim = (q64.view(-1, d) @ k64.view(-1, d).T).view(Nq, Lq, Nd, Ld).masked_fill(dm.cpu()[None, None] == 0, -float("inf"))
    # equal similarities are common among 4-bit tokens: the lowest index takes the gradient
    first = (sim == sim.amax(3, keepdim=True)).int().argmax(3, keepdim=True)
    sc = sim.gather(3, first)[..., 0].sum(1)
    lp = torch.log_softmax(np.float64(np.float32(scale)) * sc, 1)
    loss = (g.double().cpu()[:, 0] * lp.gather(1, t.long().cpu())[:, 0] - gh.double().cpu() * (lp.exp() * lp).sum(1)).sum()
    loss.backward()
    assert torch.allclose(s.double().cpu(), sc.detach(), rtol=1e-6, atol=1e-6)
    assert torch.allclose(logp.double().cpu()[:, 0], lp.gather(1, t.long().cpu())[:, 0].detach(), rtol=1e-5, atol=1e-5)
    for got, want in ((dq, q64.grad), (dd, k64.grad)):
        assert torch.allclose(got.double().cpu(), want, rtol=1e-4, atol=1e-6)
    order = sc.detach().argsort(1, descending=True)
    assert torch.equal(idx.long().cpu(), order[:, :3])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        qf.add_(0.05 * i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, run()):
            assert torch.equal(a, b)
