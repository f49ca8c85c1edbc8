"""The embedding head on a machine without a GPU: the declared entry points are
exported, the host refuses what the header says it refuses, the binding checks
its tensors, and the test reference's generator gives the published values."""

import ctypes
import os
import re

import pytest
import torch

import embed_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "maxsim_embed.h")

OK, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_OVERFLOW, ERR_LAUNCH = range(6)
F16, BF16, F32, I8 = range(4)
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
MIS8 = ctypes.c_void_p(0x1008)  # 8- but not 16-byte aligned
MIS4 = ctypes.c_void_p(0x1004)
MIS2 = ctypes.c_void_p(0x1002)


@pytest.fixture(scope="module")
def L():
    from maxsim_scoring_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from maxsim_scoring_amd import build
        build.build()
    return binding.lib()


def test_exports_every_declared_symbol(L):
    names = re.findall(r"^maxsim_status_t\s+(maxsim_\w+)\s*\(", open(HEADER).read(), re.M)
    assert sorted(names) == ["maxsim_dropout_bwd", "maxsim_dropout_fwd", "maxsim_embed_i8",
                             "maxsim_linear_i8", "maxsim_normalize_bwd", "maxsim_normalize_fwd",
                             "maxsim_quantize_tok"]
    import maxsim_scoring_amd as ms
    for n in names:
        assert hasattr(L, n) and n in ms.__all__, n


def quantize(L, dt=BF16, X=FAKE, T=4, d=128, m=None, c=FAKE, s=FAKE):
    return L.maxsim_quantize_tok(dt, X, T, d, m, 0, c, s, None)


def test_quantize_refusals(L):
    assert quantize(L, T=-1) == ERR_SHAPE
    assert quantize(L, d=-1) == ERR_SHAPE
    assert quantize(L, d=0) == ERR_UNSUPPORTED
    assert quantize(L, d=131072) == ERR_UNSUPPORTED
    assert quantize(L, dt=I8) == ERR_UNSUPPORTED
    assert quantize(L, dt=9) == ERR_UNSUPPORTED
    assert quantize(L, X=None) == ERR_NULL
    assert quantize(L, c=None) == ERR_NULL
    assert quantize(L, s=None) == ERR_NULL
    assert quantize(L, X=MIS8) == ERR_UNSUPPORTED
    assert quantize(L, c=MIS8) == ERR_UNSUPPORTED
    assert quantize(L, s=MIS2) == ERR_UNSUPPORTED
    assert quantize(L, T=1 << 31) == ERR_OVERFLOW
    assert quantize(L, T=0, X=None, c=None, s=None) == OK


def test_normalize_refusals(L):
    def fwd(xt=BF16, X=FAKE, T=4, d=128, yt=F16, Y=FAKE, r=FAKE):
        return L.maxsim_normalize_fwd(xt, X, T, d, None, yt, Y, r, None)

    def bwd(xt=BF16, X=FAKE, r=FAKE, g=FAKE, T=4, d=128, gt=F32, dX=FAKE):
        return L.maxsim_normalize_bwd(xt, X, r, g, T, d, gt, dX, None)

    for f in (fwd, bwd):
        assert f(T=-1) == ERR_SHAPE
        assert f(d=0) == ERR_UNSUPPORTED
        assert f(d=131072) == ERR_UNSUPPORTED
        assert f(xt=I8) == ERR_UNSUPPORTED
        assert f(X=None) == ERR_NULL
        assert f(r=None) == ERR_NULL
        assert f(X=MIS8) == ERR_UNSUPPORTED
        assert f(r=MIS2) == ERR_UNSUPPORTED
        assert f(T=1 << 31) == ERR_OVERFLOW
        assert f(T=0, X=None, r=None) == OK
    assert fwd(yt=I8) == ERR_UNSUPPORTED
    assert fwd(Y=None) == ERR_NULL
    assert fwd(Y=MIS8) == ERR_UNSUPPORTED
    assert bwd(gt=7) == ERR_UNSUPPORTED
    assert bwd(g=None) == ERR_NULL
    assert bwd(g=MIS8) == ERR_UNSUPPORTED
    assert bwd(dX=MIS4) == ERR_UNSUPPORTED


def test_linear_and_embed_refusals(L):
    def linear(dt=BF16, A=FAKE, s=FAKE, W=FAKE, ws=FAKE, b=None, T=4, N=8, K=64, Y=FAKE):
        return L.maxsim_linear_i8(dt, A, s, W, ws, b, T, N, K, Y, None)

    def embed(dt=BF16, A=FAKE, s=FAKE, W=FAKE, ws=FAKE, b=None, T=4, N=8, K=64, Y=FAKE, es=None):
        return L.maxsim_embed_i8(dt, A, s, W, ws, b, None, T, N, K, Y, es, None)

    for f in (linear, embed):
        assert f(T=-1) == ERR_SHAPE
        assert f(N=-1) == ERR_SHAPE
        assert f(K=-1) == ERR_SHAPE
        assert f(K=0) == ERR_UNSUPPORTED
        assert f(K=131072) == ERR_UNSUPPORTED  # 131072 * 128^2 = 2^31
        assert f(N=0) == ERR_UNSUPPORTED
        assert f(dt=5) == ERR_UNSUPPORTED
        for k in ("A", "s", "W", "ws", "Y"):
            assert f(**{k: None}) == ERR_NULL, k
        for k in ("A", "W", "Y"):
            assert f(**{k: MIS8}) == ERR_UNSUPPORTED, k
        for k in ("s", "ws", "b"):
            assert f(**{k: MIS2}) == ERR_UNSUPPORTED, k
        assert f(T=1 << 31) == ERR_OVERFLOW
        assert f(T=0, A=None, Y=None) == OK
    assert linear(dt=I8) == ERR_UNSUPPORTED
    assert linear(N=(1 << 26) + 1) == ERR_OVERFLOW
    assert embed(N=1025) == ERR_UNSUPPORTED
    assert embed(dt=I8) == ERR_NULL             # codes need a scale
    assert embed(dt=I8, es=MIS2) == ERR_UNSUPPORTED


def test_dropout_refusals(L):
    for f in (L.maxsim_dropout_fwd, L.maxsim_dropout_bwd):
        def call(dt=BF16, X=FAKE, n=64, p=0.1, sd=None, Y=FAKE):
            return f(dt, X, n, p, 1, 2, sd, Y, None)
        assert call(n=-1) == ERR_SHAPE
        assert call(dt=I8) == ERR_UNSUPPORTED
        for p in (-0.01, 1.01, float("nan"), float("inf")):
            assert call(p=p) == ERR_UNSUPPORTED, p
        assert call(X=None) == ERR_NULL
        assert call(Y=None) == ERR_NULL
        assert call(X=MIS8) == ERR_UNSUPPORTED
        assert call(Y=MIS8) == ERR_UNSUPPORTED
        assert call(sd=MIS4) == ERR_UNSUPPORTED
        assert call(n=1 << 43) == ERR_OVERFLOW
        assert call(n=0, X=None, Y=None) == OK


def test_scoring_entry_points_refuse_the_new_types(L):
    for dt in (F32, I8):
        assert L.maxsim_fwd(dt, FAKE, FAKE, 2, 3, 4, 5, 128, None, None, FAKE, None, None) == ERR_UNSUPPORTED


def test_binding_refusals():
    import maxsim_scoring_amd as ms
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    a, s = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    w, ws = torch.zeros(8, 32, dtype=torch.int8), torch.ones(8)
    for call in (lambda: ms.maxsim_quantize_tok(x),             # not on the GPU
                 lambda: ms.maxsim_quantize_tok(x.int()),       # not a float type
                 lambda: ms.maxsim_quantize_tok(x[0, 0]),       # no rows
                 lambda: ms.maxsim_normalize_fwd(x),
                 lambda: ms.maxsim_normalize_fwd(x, out_dtype=torch.int8),
                 lambda: ms.maxsim_normalize_bwd(x, s, x.float()),
                 lambda: ms.maxsim_linear_i8(a, s, w, ws),
                 lambda: ms.maxsim_linear_i8(a, s, w[:, :16], ws),
                 lambda: ms.maxsim_linear_i8(a, s, w, ws, out_dtype=torch.int8),
                 lambda: ms.maxsim_embed_i8(a, s, w, ws),
                 lambda: ms.embed_tokens_i8(x, w, ws),
                 lambda: ms.maxsim_dropout_fwd(x, 0.1, 1),
                 lambda: ms.maxsim_dropout_fwd(x, 0.1, -1),
                 lambda: ms.maxsim_dropout_fwd(x, 0.1, 1, step=1 << 64),
                 lambda: ms.maxsim_dropout_bwd(x.int(), 0.1, 1)):
        with pytest.raises(ValueError):
            call()


def test_reference_generator_gives_the_published_values():
    """Known answers of Philox4x32-10, published with the paper's library."""
    ones = 0xFFFFFFFF
    assert ref.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox((ones,) * 4, (ones,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_status_text_names_the_widths(L):
    text = L.maxsim_status_string(ERR_UNSUPPORTED).decode()
    assert "1..1024" in text and "1..131071" in text
