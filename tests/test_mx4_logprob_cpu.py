"""4-bit rows and log probabilities on a machine without a GPU: the declared entry
points are exported, the host refuses what the headers say it refuses, the binding
checks its tensors, and the test references agree with hand examples."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import logprob_reference as lref
import mx4_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_OVERFLOW, ERR_LAUNCH = range(6)
F16, BF16, F32, I8 = range(4)
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
MIS8 = ctypes.c_void_p(0x1008)
MIS2 = ctypes.c_void_p(0x1002)
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def L():
    from maxsim_scoring_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from maxsim_scoring_amd import build
        build.build()
    return binding.lib()


def test_exports_every_declared_symbol(L):
    import maxsim_scoring_amd as ms
    want = {"maxsim_mx4.h": ["maxsim_dequantize_mx4", "maxsim_fwd_mx4", "maxsim_linear_mx4", "maxsim_quantize_mx4"],
            "maxsim_loss.h": ["maxsim_logprob_bwd", "maxsim_logprob_fwd"]}
    for header, names in want.items():
        text = open(os.path.join(ROOT, "include", header)).read()
        assert sorted(re.findall(r"^maxsim_status_t\s+(maxsim_\w+)\s*\(", text, re.M)) == names
        for n in names:
            assert hasattr(L, n) and n in ms.__all__, n


def test_row_refusals(L):
    def quantize(dt=BF16, X=FAKE, T=4, d=128, c=FAKE, s=FAKE):
        return L.maxsim_quantize_mx4(dt, X, T, d, None, 0, c, s, None)

    def dequantize(dt=BF16, X=FAKE, T=4, d=128, c=FAKE, s=FAKE):
        return L.maxsim_dequantize_mx4(c, s, T, d, dt, X, None)

    for f in (quantize, dequantize):
        assert f(T=-1) == ERR_SHAPE
        assert f(d=-1) == ERR_SHAPE
        assert f(d=0) == ERR_UNSUPPORTED
        assert f(d=131072) == ERR_UNSUPPORTED
        assert f(dt=I8) == ERR_UNSUPPORTED
        assert f(dt=9) == ERR_UNSUPPORTED
        for k in ("X", "c", "s"):
            assert f(**{k: None}) == ERR_NULL, k
        for k in ("X", "c"):
            assert f(**{k: MIS8}) == ERR_UNSUPPORTED, k
        assert f(T=1 << 31) == ERR_OVERFLOW
        assert f(T=0, X=None, c=None, s=None) == OK


def test_product_refusals(L):
    def linear(dt=BF16, A=FAKE, s=FAKE, W=FAKE, ws=FAKE, b=None, T=4, N=8, K=64, Y=FAKE):
        return L.maxsim_linear_mx4(dt, A, s, W, ws, b, T, N, K, Y, None)

    for k in ("T", "N", "K"):
        assert linear(**{k: -1}) == ERR_SHAPE
    assert linear(K=0) == ERR_UNSUPPORTED
    assert linear(K=131072) == ERR_UNSUPPORTED
    assert linear(N=0) == ERR_UNSUPPORTED
    assert linear(dt=I8) == ERR_UNSUPPORTED
    for k in ("A", "s", "W", "ws", "Y"):
        assert linear(**{k: None}) == ERR_NULL, k
    for k in ("A", "W", "Y"):
        assert linear(**{k: MIS8}) == ERR_UNSUPPORTED, k
    assert linear(b=MIS2) == ERR_UNSUPPORTED
    assert linear(T=1 << 31) == ERR_OVERFLOW
    assert linear(N=(1 << 26) + 1) == ERR_OVERFLOW
    assert linear(T=0, A=None, Y=None) == OK


def test_score_refusals(L):
    def fwd(Q=FAKE, qs=FAKE, D=FAKE, ds=FAKE, Nq=2, Nd=3, Lq=4, Ld=5, d=128, s=FAKE, am=None):
        return L.maxsim_fwd_mx4(Q, qs, D, ds, Nq, Nd, Lq, Ld, d, None, None, s, am, None)

    for k in ("Nq", "Nd", "Lq", "Ld", "d"):
        assert fwd(**{k: -1}) == ERR_SHAPE, k
    assert fwd(d=0) == ERR_UNSUPPORTED
    assert fwd(d=1025) == ERR_UNSUPPORTED
    for k in ("Q", "qs", "D", "ds", "s"):
        assert fwd(**{k: None}) == ERR_NULL, k
    for k in ("Q", "D"):
        assert fwd(**{k: MIS8}) == ERR_UNSUPPORTED, k
    for k in ("s", "am"):
        assert fwd(**{k: MIS2}) == ERR_UNSUPPORTED, k
    for k in ("Nq", "Nd", "Lq", "Ld"):
        assert fwd(**{k: 1 << 31}) == ERR_OVERFLOW, k
    assert fwd(Nq=1 << 16, Nd=1 << 15) == ERR_OVERFLOW
    assert fwd(Nq=1 << 10, Nd=1 << 15, Lq=64, am=FAKE) == ERR_OVERFLOW
    assert fwd(Nq=0, Q=None, s=None) == OK
    assert fwd(Nd=0, D=None, s=None) == OK


def test_logprob_refusals(L):
    def fwd(dt=F32, X=FAKE, Nq=2, Nd=50, scale=1.0, t=FAKE, P=3, K=4, lp=FAKE, r=FAKE, n=FAKE, e=FAKE, ti=FAKE, tl=FAKE,
            ws=None, wb=0):
        return L.maxsim_logprob_fwd(dt, X, Nq, Nd, scale, None, t, P, K, lp, r, n, e, ti, tl, ws, wb, None)

    def bwd(dt=F32, X=FAKE, Nq=2, Nd=50, scale=1.0, t=FAKE, P=3, n=FAKE, e=None, g=FAKE, ge=None, xt=F32, dX=FAKE):
        return L.maxsim_logprob_bwd(dt, X, Nq, Nd, scale, None, t, P, n, e, g, ge, xt, dX, None)

    for f in (fwd, bwd):
        for k in ("Nq", "Nd", "P"):
            assert f(**{k: -1}) == ERR_SHAPE, k
        assert f(dt=I8) == ERR_UNSUPPORTED
        for s in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -65, 2.0 ** 65):
            assert f(scale=s) == ERR_UNSUPPORTED, s
        for k in ("X", "t", "n"):
            assert f(**{k: None}) == ERR_NULL, k
        assert f(X=MIS2) == ERR_UNSUPPORTED
        assert f(dt=BF16, X=ODD) == ERR_UNSUPPORTED
        assert f(t=MIS2) == ERR_UNSUPPORTED
        assert f(Nq=1 << 31) == ERR_OVERFLOW
        assert f(Nd=1 << 31, **({"ws": FAKE, "wb": 1 << 60} if f is fwd else {})) == ERR_OVERFLOW
        assert f(Nq=1 << 20, P=1 << 11) == ERR_OVERFLOW
        assert f(Nq=0, X=None, t=None) == OK
    assert fwd(K=-1) == ERR_SHAPE
    assert fwd(K=1025) == ERR_UNSUPPORTED
    for k in ("lp", "ti", "tl"):
        assert fwd(**{k: None}) == ERR_NULL, k
    for k in ("lp", "r", "n", "e", "ti", "tl"):
        assert fwd(**{k: MIS2}) == ERR_UNSUPPORTED, k
    assert fwd(Nd=5000) == ERR_NULL                              # rows of several chunks need a workspace
    assert fwd(Nd=5000, ws=FAKE, wb=16) == ERR_SHAPE
    assert fwd(Nd=5000, ws=MIS8, wb=1 << 30) == ERR_UNSUPPORTED
    assert bwd(e=FAKE) == ERR_NULL
    assert bwd(ge=FAKE) == ERR_NULL
    assert bwd(g=None) == ERR_NULL
    assert bwd(dX=None) == ERR_NULL
    assert bwd(xt=I8) == ERR_UNSUPPORTED
    assert bwd(dX=MIS2) == ERR_UNSUPPORTED
    assert bwd(Nd=0, X=None, dX=None) == OK


def test_logprob_workspace(L):
    f = L.maxsim_logprob_workspace
    assert f(0, 100, 1, 1) == 0
    assert f(7, 4096, 5, 1024) == 0
    assert f(7, 4097, 5, 1024) > f(7, 4097, 5, 8) > f(7, 4097, 0, 0) > 0
    for bad in ((-1, 5, 1, 1), (1, -5, 1, 1), (1, 5, -1, 1), (1, 5, 1, -1), (1, 5, 1, 1025), (1 << 31, 5, 1, 1),
                (1 << 20, 1 << 24, 1, 1)):
        assert f(*bad) == -1, bad


def test_binding_tells_the_workspace(L):
    """The size that maxsim_logprob_fwd's documentation names is to be had without the C library."""
    import maxsim_scoring_amd as ms
    assert "maxsim_logprob_workspace" in ms.__all__
    assert ms.maxsim_logprob_workspace(7, 4096, 5) == 0
    assert ms.maxsim_logprob_workspace(7, 4097, 5, 8) == L.maxsim_logprob_workspace(7, 4097, 5, 8) > 0
    for bad in ((7, -1, 5, 8), (7, 5000, 5, 1025), (1 << 31, 5, 1, 1)):
        with pytest.raises(ValueError):
            ms.maxsim_logprob_workspace(*bad)


def test_logprob_largest_sizes(L):
    """The header's limit itself: 2^31 - 4097 is the largest size, 2^31 - 4096 is refused."""
    f, most = L.maxsim_logprob_workspace, (1 << 31) - 4097
    for fine in ((1, most, 1, 1), (1, 5000, most, 1), (most, 5, 0, 0)):
        assert f(*fine) >= 0, fine
    for bad in ((1, most + 1, 1, 1), (1, 5000, most + 1, 1), (most + 1, 5, 0, 0)):
        assert f(*bad) == -1, bad


def test_binding_refuses_cpu_tensors():
    import maxsim_scoring_amd as ms
    x, u = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8)
    s, t = torch.zeros(4, 2, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: ms.maxsim_quantize_mx4(x),
                 lambda: ms.maxsim_dequantize_mx4(u, s),
                 lambda: ms.maxsim_linear_mx4(u, s, u, s),
                 lambda: ms.maxsim_fwd_mx4(u[None], s[None], u[None], s[None]),
                 lambda: ms.embed_tokens_mx4(x, u, s),
                 lambda: ms.maxsim_logprob_fwd(x, t),
                 lambda: ms.maxsim_logprob_bwd(x, t, torch.zeros(4, 2), torch.zeros(4, 1))):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_rows_of_more_blocks_than_the_widest():
    """Without a width the blocks say it: those of 4096 make 131071 values, more are no
    row that the library has. (They were taken as rows of 4096, read at the wrong places.)"""
    import maxsim_scoring_amd as ms
    for B, fine in ((4096, True), (4097, False), (5000, False)):
        u, s = torch.zeros(2, 16 * B, dtype=torch.uint8), torch.zeros(2, B, dtype=torch.uint8)
        for call in (lambda: ms.maxsim_dequantize_mx4(u, s),
                     lambda: ms.maxsim_linear_mx4(u, s, u, s),
                     lambda: ms.maxsim_fwd_mx4(u[None], s[None], u[None], s[None])):
            with pytest.raises(ValueError, match="GPU tensor" if fine else f"{B} blocks"):
                call()


def test_reference_codes_by_hand():
    row = [[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9, -0.3] + [0.0] * 21 + [4.0]]
    code, scale = ref.quantize(row)
    assert scale.tolist() == [[127]]
    assert code[0, :10].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 9] and code[0, 31] == 6
    v = ref.values(ref.pack(code), scale)
    assert v[0, :10].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6, -0.5]
    code, scale = ref.quantize([[3.0, 4.0]], normalize=True)    # 0.6 and 0.8 in steps of 2^-3: 4.8 and 6.4
    assert scale.tolist() == [[124]] and code[0, :2].tolist() == [6, 7]
    assert np.isnan(ref.values(np.zeros((1, 16), np.uint8), np.full((1, 1), 255, np.uint8))).all()


def test_reference_gradient_by_differences():
    r = np.random.default_rng(0)
    x, g, gh = r.normal(size=(2, 7)), r.normal(size=(2, 3)), r.normal(size=2)
    t = np.array([[0, 3, 3], [6, 9, 1]])
    mask = np.ones((2, 7))
    mask[0, 2] = mask[1, 1] = 0

    def loss(v):
        o, _ = lref.forward(v, t, mask, 1.7, 0)
        return (np.where(np.isfinite(o["logp"]), g * np.where(np.isfinite(o["logp"]), o["logp"], 0), 0)).sum() + (gh * o["entropy"]).sum()

    o, _ = lref.forward(x, t, mask, 1.7, 3)
    dX, _ = lref.backward(x, t, mask, 1.7, g, o["norm"], o["entropy"], gh)
    for i in range(2):
        for c in range(7):
            e = np.zeros_like(x)
            e[i, c] = 1e-5
            assert abs((loss(x + e) - loss(x - e)) / 2e-5 - dX[i, c]) < 1e-8
    assert o["top_idx"][0].tolist() == [c for c in np.argsort(-x[0]) if c != 2][:3]
