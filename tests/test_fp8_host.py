"""Host-side behaviour of the 8-bit operators (CPU only): the oracle's own pins,
the C ABI's refusals before any device work, and the binding's."""

import ctypes

import numpy as np
import pytest
import torch

from gemm_epilogue_fusion_tmem_b200 import binding as B
from oracle import fp8_oracle as O

P = ctypes.c_void_p
ONE = P(256)
BIG = 1 << 30


# ------------------------------------------------------------------ oracle pins

@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_round8_is_the_types_nearest_even(fmt, dtype):
    every = torch.arange(256, dtype=torch.uint8).view(dtype).float()
    every = torch.unique(every[torch.isfinite(every)]).double().numpy()
    assert np.array_equal(O.round8(every, fmt), every)
    mid = (every[1:] + every[:-1]) / 2   # ties go to the even neighbour
    x = np.concatenate([mid, np.random.default_rng(0).normal(0, 40, 4000)])
    want = torch.from_numpy(x).float().to(dtype).float().double().numpy()
    assert np.array_equal(O.round8(x, fmt), want)
    assert O.round8(np.array([1e9]), fmt)[0] == O.FMAX[fmt]


@pytest.mark.parametrize("form", ["rows", "cols", "blocks"])
def test_quant_covers_ragged_blocks(form):
    x = np.random.default_rng(1).normal(size=(130, 272))
    x[:128, :128] = 0
    q, s = O.quant(x, form, "e4m3")
    assert s.shape == {"rows": (3, 130), "cols": (2, 272), "blocks": (2, 3)}[form]
    assert np.all(s >= O.TINY / 448) and np.all(q[:128, :128] == 0)
    back = O.dequant(q, s, form)
    each = O.spread(s, form, *x.shape)
    assert np.all(np.abs(back - x) <= each * O.step8(x / each, "e4m3") / 2 * (1 + 1e-12))
    top = {"rows": np.abs(q).reshape(130, -1)[:, 128:256].max(1), "cols": np.abs(q)[:128].max(0)[128:],
           "blocks": np.array([np.abs(q)[:128, 128:256].max()])}[form]
    assert np.all(top == 448)


def test_gradients_against_differences():
    rng = np.random.default_rng(2)
    M, d, F, h = 3, 16, 8, 1e-6
    x, g, dn = rng.normal(size=(M, d)), rng.normal(size=d), rng.normal(size=(M, d))
    dhi = rng.normal(size=(M, d))
    loss = lambda x, g: np.sum(dn * O.rmsnorm(x, g, 1e-5)[1]) + np.sum(dhi * x)
    dh, dg = O.rmsnorm_bwd(dn, x, O.rmsnorm(x, g, 1e-5)[0], g, dhi)
    for i in np.ndindex(M, d):
        e = np.zeros((M, d))
        e[i] = h
        assert abs((loss(x + e, g) - loss(x - e, g)) / (2 * h) - dh[i]) < 1e-7
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        assert abs((loss(x, g + e) - loss(x, g - e)) / (2 * h) - dg[j]) < 1e-7
    a, b, dy = rng.normal(size=(M, F)) * 3, rng.normal(size=(M, F)), rng.normal(size=(M, F))
    da, db = O.swiglu_bwd(dy, a, b)
    assert np.allclose((O.swiglu(a + h, b) - O.swiglu(a - h, b)) / (2 * h) * dy, da, atol=1e-8)
    assert np.allclose((O.swiglu(a, b + h) - O.swiglu(a, b - h)) / (2 * h) * dy, db, atol=1e-8)


# ------------------------------------------------------------------ C ABI refusals

def _gemm(A=ONE, SA=ONE, Bm=ONE, SB=ONE, C=ONE, M=64, N=64, K=64, a_mn=0, b_mn=0, fa=0, fb=0, blocks=1, f32=0, acc=0,
          ws=ONE, wsb=256):
    return B.library().coda_gemm_fp8._fn(A, SA, Bm, SB, C, M, N, K, a_mn, b_mn, fa, fb, blocks, f32, acc, ws, wsb, None)


def test_gemm_refusals():
    for bad in (dict(A=None), dict(SA=None), dict(Bm=None), dict(SB=None), dict(C=None), dict(ws=None), dict(M=-1),
                dict(N=-16), dict(K=-16), dict(fa=2), dict(fb=-1), dict(acc=1)):
        assert _gemm(**bad) == 1, bad
    for bad in (dict(N=72), dict(K=72), dict(a_mn=1, b_mn=0, K=72), dict(a_mn=1, M=72), dict(N=8),
                dict(M=1 << 30, N=1 << 24)):
        assert _gemm(**bad) == 2, bad
    for bad in (dict(A=P(264)), dict(SB=P(260)), dict(C=P(258)), dict(ws=P(8))):
        assert _gemm(**bad) == 3, bad
    assert _gemm(wsb=255) == 4
    assert _gemm(M=0, A=None, C=None) == 0 and _gemm(N=0, C=None) == 0
    assert _gemm(K=0, C=None) == 1
    assert _gemm(K=0, f32=1, acc=1) == 0  # adds nothing


def test_gemm_swiglu_refusals():
    def call(A=ONE, SA=ONE, W=ONE, SW=ONE, Y=ONE, SY=ONE, AB=ONE, SAB=ONE, M=64, K=64, F=128, ws=ONE, wsb=256):
        return B.library().coda_gemm_swiglu_fp8._fn(A, SA, W, SW, Y, SY, AB, SAB, M, K, F, ws, wsb, None)

    for bad in (dict(A=None), dict(SA=None), dict(W=None), dict(SW=None), dict(Y=None), dict(SY=None), dict(AB=None),
                dict(SAB=None), dict(ws=None), dict(M=-1), dict(K=0), dict(F=0)):
        assert call(**bad) == 1, bad
    for bad in (dict(K=72), dict(F=64), dict(F=192)):
        assert call(**bad) == 2, bad
    assert call(Y=P(264)) == 3 and call(wsb=0) == 4
    assert call(M=0, A=None, Y=None, SY=None, AB=None, SAB=None, ws=None) == 0


def test_light_pass_refusals():
    lib = B.library()
    quant = lambda X=ONE, rv=None, cv=None, Qr=ONE, Sr=ONE, Qc=ONE, Sc=ONE, R=8, C=64, f=0: \
        lib.coda_quant_fp8._fn(X, rv, cv, Qr, Sr, Qc, Sc, R, C, f, None)
    for bad in (dict(X=None), dict(Qr=None), dict(Sr=None), dict(Qc=None), dict(Sc=None), dict(R=-1), dict(C=0),
                dict(f=2), dict(Qr=None, Sr=None, Qc=None, Sc=None)):
        assert quant(**bad) == 1, bad
    assert quant(C=72) == 2 and quant(C=(1 << 22) + 16) == 2 and quant(X=P(8)) == 3 and quant(cv=P(24)) == 3 and quant(R=0, X=None) == 0
    blocks = lambda W=ONE, Q=ONE, S=ONE, R=8, C=64, f=0: lib.coda_quant_fp8_blocks._fn(W, Q, S, R, C, f, None)
    assert blocks(W=None) == 1 and blocks(S=None) == 1 and blocks(f=7) == 1 and blocks(C=8) == 2
    assert blocks(Q=P(4)) == 3 and blocks(R=0) == 0
    swb = lambda dY=ONE, AB=ONE, SAB=ONE, dA=ONE, SdA=ONE, c=(ONE,) * 4, M=8, F=128, f=0: \
        lib.coda_swiglu_fp8_bwd._fn(dY, AB, SAB, dA, SdA, *c, M, F, f, None)
    for bad in (dict(dY=None), dict(AB=None), dict(SAB=None), dict(dA=None), dict(SdA=None),
                dict(c=(ONE, ONE, ONE, None)), dict(c=(None, None, ONE, ONE)), dict(M=-1), dict(f=3)):
        assert swb(**bad) == 1, bad
    assert swb(F=64) == 2 and swb(dY=P(8)) == 3 and swb(M=0, dY=None) == 0
    rf = lambda X=ONE, R=ONE, g=ONE, H=ONE, r=ONE, Q=ONE, S=ONE, M=8, d=64, eps=1e-6: \
        lib.coda_rmsnorm_fp8_fwd._fn(X, R, g, H, r, Q, S, M, d, eps, None)
    for bad in (dict(X=None), dict(R=None), dict(H=None), dict(g=None), dict(r=None), dict(Q=None), dict(S=None),
                dict(eps=0.0), dict(eps=float("nan")), dict(M=-2), dict(d=0)):
        assert rf(**bad) == 1, bad
    assert rf(d=72) == 2 and rf(d=32784) == 2 and rf(g=P(40)) == 3 and rf(M=0, X=None) == 0
    rb = lambda dN=ONE, H=ONE, r=ONE, g=ONE, hi=None, dH=ONE, dg=ONE, M=8, d=64, ws=ONE, wsb=BIG: \
        lib.coda_rmsnorm_fp8_bwd._fn(dN, H, r, g, hi, dH, dg, M, d, ws, wsb, None)
    for bad in (dict(dN=None), dict(H=None), dict(r=None), dict(g=None), dict(dH=None), dict(dg=None), dict(ws=None),
                dict(M=-1), dict(M=0, dg=None)):
        assert rb(**bad) == 1, bad
    need = lib.coda_rmsnorm_fp8_bwd_workspace_bytes(8, 64)
    assert need >= 256 + 4 * 64
    assert rb(d=8) == 2 and rb(hi=P(8)) == 3 and rb(wsb=need - 1) == 4


# ------------------------------------------------------------------ binding refusals

def test_binding_refusals_on_the_host():
    e4 = torch.float8_e4m3fn
    q, s = torch.zeros(64, 128, dtype=e4), torch.zeros(1, 64)
    bf = torch.zeros(64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.gemm_fp8(q, s, q, torch.zeros(1, 1), 64, 64, 128)
    with pytest.raises(TypeError, match="float8"):
        B.gemm_fp8(bf, s, q, s, 64, 64, 128)
    with pytest.raises(TypeError):
        B.gemm_fp8(None, s, q, s, 64, 64, 128)
    for call in (lambda: B.quant_fp8(bf), lambda: B.quant_fp8_blocks(bf), lambda: B.gemm_swiglu_fp8(q, s, q, s),
                 lambda: B.swiglu_fp8_bwd(bf, q, s), lambda: B.rmsnorm_fp8_fwd(bf, bf[0], 1e-6),
                 lambda: B.rmsnorm_fp8_bwd(bf, bf, s[0], bf[0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    for call in (lambda: B.quant_fp8("x"), lambda: B.rmsnorm_fp8_fwd(None, None, 1e-6)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="2 dimensions"):
        B.quant_fp8(bf[0])


def test_format_codes_match_the_header():
    src = open(B.__file__.replace("gemm_epilogue_fusion_tmem_b200/binding.py", "include/coda.h")).read()
    assert "#define CODA_FP8_E4M3 0" in src and "#define CODA_FP8_E5M2 1" in src
    assert B._FP8 == {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
    for name, code in (("GEMM_FP8", B.KERNEL_GEMM_FP8), ("GEMM_SWIGLU_FP8", B.KERNEL_GEMM_SWIGLU_FP8),
                       ("QUANT_FP8", B.KERNEL_QUANT_FP8), ("SWIGLU_FP8_BWD", B.KERNEL_SWIGLU_FP8_BWD),
                       ("RMSNORM_FP8_FWD", B.KERNEL_RMSNORM_FP8_FWD), ("RMSNORM_FP8_BWD", B.KERNEL_RMSNORM_FP8_BWD)):
        assert f"#define CODA_KERNEL_{name} {code} " in src


def test_row_limits():
    """Row numbers of a last tile, or one step of a grid further, stay below 2^31: more rows are refused."""
    lib, top, over = B.library(), 2 ** 31 - 4096, 2 ** 31 - 4095
    for bad in (dict(M=over, N=16), dict(M=16, N=2 ** 31 - 16), dict(M=16, N=16, K=2 ** 31 - 16),
                dict(a_mn=1, b_mn=1, blocks=0, M=2 ** 31 - 16, N=16)):
        assert _gemm(**bad) == 2, bad
    assert _gemm(M=top, N=16, wsb=0) == 4   # the limit itself passes the checks of shapes
    assert lib.coda_gemm_swiglu_fp8._fn(*[ONE] * 8, over, 16, 128, ONE, 256, None) == 2
    assert lib.coda_gemm_swiglu_fp8._fn(*[ONE] * 8, 16, 2 ** 31 - 16, 128, ONE, 256, None) == 2
    assert lib.coda_gemm_swiglu_fp8._fn(*[ONE] * 8, top, 16, 128, ONE, 0, None) == 4
    assert lib.coda_quant_fp8._fn(ONE, None, None, ONE, ONE, ONE, ONE, over, 16, 0, None) == 2
    assert lib.coda_quant_fp8._fn(P(8), None, None, ONE, ONE, ONE, ONE, top, 16, 0, None) == 3
    assert lib.coda_quant_fp8_blocks._fn(ONE, ONE, ONE, over, 16, 0, None) == 2
    assert lib.coda_swiglu_fp8_bwd._fn(*[ONE] * 9, over, 128, 0, None) == 2
    assert lib.coda_rmsnorm_fp8_fwd._fn(*[ONE] * 7, over, 16, 1e-6, None) == 2
    assert lib.coda_rmsnorm_fp8_bwd._fn(*[ONE] * 7, over, 16, ONE, BIG, None) == 2


def test_sizes_that_are_no_c_int_are_refused():
    """2^32 + 5 rows would be passed on as 5."""
    n, e4 = 2 ** 32 + 5, torch.float8_e4m3fn
    t = lambda *s, dtype=e4: torch.empty(*s, dtype=dtype, device="meta")
    bf = torch.bfloat16
    for call in (lambda: B.gemm_fp8(t(n, 16), t(1, n), t(16, 16), t(1, 1), n, 16, 16),
                 lambda: B.gemm_fp8(t(0, 16), t(1, 0), t(16, 16), t(1, 1), -1, 16, 16),
                 lambda: B.quant_fp8(t(n, 16, dtype=bf)), lambda: B.quant_fp8_blocks(t(n, 16, dtype=bf)),
                 lambda: B.gemm_swiglu_fp8(t(n, 16), t(1, n), t(256, 16), t(2, 1)),
                 lambda: B.swiglu_fp8_bwd(t(n, 128, dtype=bf), t(n, 256), t(2, n)),
                 lambda: B.rmsnorm_fp8_fwd(t(n, 16, dtype=bf), t(16, dtype=bf), 1e-6),
                 lambda: B.rmsnorm_fp8_bwd(t(n, 16, dtype=bf), t(n, 16, dtype=bf), t(n), t(16, dtype=bf))):
        with pytest.raises(ValueError, match="sizes must be from 0"):
            call()


def test_workspace_must_lie_where_the_tensors_do():
    """A kernel that is given host memory, or another device's, as its scratch would fault."""
    cpu, dev = B.Workspace(256, "cpu"), torch.device("cuda", 0)
    with pytest.raises(ValueError, match="ws is on cpu"):
        B._ws_on(cpu, dev)
    assert B._ws_on(cpu, torch.device("cpu")) is cpu


def test_parts_refusals():
    few, parts = ctypes.c_int(0), ctypes.c_int(0)
    fn = B.library().coda_gemm_fp8_parts
    for bad in ((0, 16, 16), (16, -1, 16), (16, 16, 0)):
        assert fn(*bad, 0, 0, 1, 0, ctypes.byref(few), ctypes.byref(parts)) == 1, bad
    assert fn(16, 16, 16, 0, 0, 1, 0, None, ctypes.byref(parts)) == 1
    with pytest.raises(ValueError, match="sizes must be"):
        B.gemm_fp8_parts(2 ** 31, 16, 16)
