"""The 8-bit operators on the GPU against their fp64 definitions.

Bounds are derived in tests/fp8_checks.py: half an 8-bit (or bf16) step at each
stored value, and the fp32 roundings before it.
"""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.fp8_checks import (BF16, FP32, check_close, check_quant, gemm_error, num, swiglu_bwd_error, swiglu_error)

pytestmark = pytest.mark.gpu

TYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * scale


def _bf(*shape, seed=0, scale=1.0):
    return _randn(*shape, seed=seed, scale=scale).bfloat16()


def _operand(B, x, form, fmt="e4m3"):
    """(q, s) tensors on the GPU of the fp32 matrix x and their dequantised fp64 values, made on the CPU."""
    q, s = O.quant(x.double().numpy(), form, fmt)
    s = s.astype(np.float32)
    q8 = torch.from_numpy(q).float().to(TYPES[fmt])
    assert np.array_equal(num(q8), q)
    return q8.cuda(), torch.from_numpy(np.ascontiguousarray(s)).cuda(), O.dequant(q, s, form)


# ------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("R,C", [(1, 16), (2, 128), (127, 144), (128, 128), (129, 272), (300, 1040), (257, 4096)])
def test_quant_rows_and_columns(cuda_lib, R, C, fmt):
    x = _bf(R, C, seed=R + C, scale=0.3)
    x[R // 2] = 0.0           # a row of zeros: the scale's floor
    x[:, C // 3] *= 50.0      # a wide channel
    o = cuda_lib.quant_fp8(x.cuda(), rows=True, cols=True, fmt=TYPES[fmt])
    check_quant(o["Qr"], o["Sr"], num(x), "rows", fmt, "rows")
    check_quant(o["Qc"], o["Sc"], num(x), "cols", fmt, "cols")
    alone = cuda_lib.quant_fp8(x.cuda(), rows=True, fmt=TYPES[fmt])
    cols = cuda_lib.quant_fp8(x.cuda(), rows=False, cols=True, fmt=TYPES[fmt])
    for k, v in {**alone, **cols}.items():
        assert torch.equal(v.view(torch.uint8), o[k].view(torch.uint8)), k


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("R,C", [(1, 16), (128, 128), (130, 400), (384, 1024)])
def test_quant_blocks(cuda_lib, R, C, fmt):
    x = _bf(R, C, seed=R, scale=0.02)
    x[:128, :128] = 0.0
    o = cuda_lib.quant_fp8_blocks(x.cuda(), fmt=TYPES[fmt])
    check_quant(o["Q"], o["S"], num(x), "blocks", fmt, "blocks")


def test_quant_scaled_by_vectors(cuda_lib):
    R, C = 200, 336
    x, r, g = _bf(R, C, seed=1), _randn(R, seed=2).abs() + 0.1, _bf(C, seed=3)
    ref = num(x) * num(r)[:, None] * num(g)
    for rv, cv, want in ((r, g, ref), (r, None, num(x) * num(r)[:, None]), (None, g, num(x) * num(g))):
        o = cuda_lib.quant_fp8(x.cuda(), cols=True, rowvec=None if rv is None else rv.cuda(),
                               colvec=None if cv is None else cv.cuda())
        err = np.abs(want) * 3 * FP32
        check_quant(o["Qr"], o["Sr"], want, "rows", "e4m3", "scaled rows", err)
        check_quant(o["Qc"], o["Sc"], want, "cols", "e4m3", "scaled cols", err)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quant_extremes(cuda_lib, fmt):
    """The largest and smallest magnitudes, values below the scale's floor, NaN and infinities."""
    big = float(torch.finfo(torch.bfloat16).max)
    x = _bf(256, 256, seed=5)
    x[0] *= 1e-30
    x[1, :128] = torch.tensor(2.0 ** -120).bfloat16()   # below the floor 2^-100
    x[2] = torch.where(x[2] > 0, big, -big).bfloat16()
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    q = cuda_lib.quant_fp8(x.cuda(), fmt=TYPES[fmt])
    keep = [i for i in range(256) if i not in (3, 4)]
    check_quant(q["Qr"][keep], q["Sr"][:, keep], num(x)[keep], "rows", fmt, "extremes")
    got = num(q["Qr"])
    assert np.isnan(got[3, 7]) and np.isfinite(np.delete(got[3], 7)).all()
    check_quant(q["Qr"][3:4, 128:], q["Sr"][1:, 3:4], num(x)[3:4, 128:], "rows", fmt, "the block beside a NaN")
    want3, _ = O.quant(num(x)[3:4], "rows", fmt)
    assert np.abs(np.delete(got[3], 7) - np.delete(want3[0], 7)).max() <= O.step8(O.FMAX[fmt], fmt)
    back = num(q["Qr"])[4] * np.repeat(num(q["Sr"])[:, 4], 128)
    assert np.isnan(back[:128]).all() and np.isfinite(back[128:]).all()
    # Under the floor a value keeps fmax / 2^-100 of itself: 448 * 2^-20 rounds to 0, 57344 * 2^-20 = 0.0546875 does not.
    assert (got[1, :128] == {"e4m3": 0.0, "e5m2": 0.0546875}[fmt]).all()


def _quotients(amax, fmt="e4m3"):
    """The fp32 scales of blocks whose largest magnitudes (fp32 values) are amax: correctly rounded quotients."""
    amax = np.maximum(np.asarray(amax, np.float32), np.float32(O.TINY))
    return amax / np.float32(O.FMAX[fmt])


def _same32(got, want):
    got = got.cpu().numpy()
    assert got.shape == want.shape and got.dtype == want.dtype == np.float32
    bad = got.view(np.uint32) != want.view(np.uint32)
    assert not bad.any(), f"{bad.sum()}/{bad.size} scales are not the nearest fp32 number"


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scales_are_correctly_rounded_quotients(cuda_lib, fmt):
    """S = c / fmax to the last bit, wherever c is known to the last bit."""
    B, f = cuda_lib, TYPES[fmt]
    x = _bf(300, 1040, seed=1, scale=0.3)
    x[7] *= 1e30
    x[8] *= 1e-30
    x[9] = 0.0
    amax = lambda form: O.block_max(num(x), form)
    o = B.quant_fp8(x.cuda(), cols=True, fmt=f)
    _same32(o["Sr"], _quotients(amax("rows"), fmt))
    _same32(o["Sc"], _quotients(amax("cols"), fmt))
    _same32(B.quant_fp8_blocks(x.cuda(), fmt=f)["S"], _quotients(amax("blocks"), fmt))
    two = torch.full((300,), 2.0)   # scaled by a power of two: c is exact
    o = B.quant_fp8(x.cuda(), cols=True, rowvec=two.cuda(), fmt=f)
    _same32(o["Sr"], _quotients(2 * amax("rows"), fmt))
    _same32(o["Sc"], _quotients(2 * amax("cols"), fmt))


def test_scales_of_the_norm_and_of_the_checkpoint_are_correctly_rounded(cuda_lib):
    B = cuda_lib
    x, g = _bf(40, 1040, seed=2).cuda(), (1 + 0.1 * _randn(1040, seed=3)).bfloat16().cuda()
    o = B.rmsnorm_fp8_fwd(x, g, 1e-6)
    n = x.float() * o["r"][:, None] * g.float()   # the kernel's own fp32 products
    _same32(o["S"], _quotients(O.block_max(num(n), "rows")))
    for M in (5, 100):  # few rows, and tiles: sums of small integers are exact
        rng = np.random.default_rng(M)
        a, w = rng.integers(-8, 9, (M, 128)), rng.integers(-8, 9, (512, 128))
        e4 = lambda v: torch.from_numpy(v).float().to(TYPES["e4m3"]).cuda()
        one = lambda *s: torch.ones(*s, device="cuda")
        o = B.gemm_swiglu_fp8(e4(a), one(1, M), e4(w), one(4, 1))
        _same32(o["SAB"], _quotients(O.block_max(a @ w.T, "rows")))


# ------------------------------------------------------------------ GEMM

def _gemm_case(B, M, N, K, a_mn, b_mn, blocks, fa, fb, f32, seed=0):
    a = _randn(K, M, seed=seed) if a_mn else _randn(M, K, seed=seed)
    b = _randn(K, N, seed=seed + 1, scale=0.1) if b_mn else _randn(N, K, seed=seed + 1, scale=0.1)
    qa, sa, da = _operand(B, a, "cols" if a_mn else "rows", fa)
    qb, sb, db = _operand(B, b, "blocks" if blocks else ("cols" if b_mn else "rows"), fb)
    da, db = (da.T if a_mn else da), (db.T if b_mn else db)
    ref, err = da @ db.T, gemm_error(da, db, K)
    kw = dict(a_mn_major=a_mn, b_mn_major=b_mn, b_blocks=blocks, out_dtype=torch.float32 if f32 else torch.bfloat16)
    return (qa, sa, qb, sb, M, N, K), kw, ref, err


MAJORS = [(False, False), (False, True), (True, True), (True, False)]


@pytest.mark.parametrize("blocks", [True, False])
@pytest.mark.parametrize("a_mn,b_mn", MAJORS)
@pytest.mark.parametrize("M,N,K", [(256, 256, 128), (16, 16, 16), (272, 528, 400), (144, 1040, 1296)])
def test_gemm_orientations(cuda_lib, M, N, K, a_mn, b_mn, blocks):
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, a_mn, b_mn, blocks, "e4m3", "e4m3", True, seed=M)
    ws = cuda_lib.Workspace(256)
    check_close(num(cuda_lib.gemm_fp8(*args, **kw, ws=ws)), ref, err, "fp32")
    kw["out_dtype"] = torch.bfloat16
    check_close(num(cuda_lib.gemm_fp8(*args, **kw, ws=ws)), ref, err + BF16 * (np.abs(ref) + err), "bf16")
    assert ws.query() == (0, 0)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("a_mn,b_mn", MAJORS)
def test_gemm_types(cuda_lib, fa, fb, a_mn, b_mn):
    args, kw, ref, err = _gemm_case(cuda_lib, 144, 272, 336, a_mn, b_mn, not a_mn, fa, fb, True, seed=9)
    check_close(num(cuda_lib.gemm_fp8(*args, **kw)), ref, err, f"{fa} x {fb}")


@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 600])
def test_gemm_any_number_of_rows(cuda_lib, M):
    N, K = 656, 1168
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, False, False, True, "e4m3", "e4m3", False, seed=M)
    # Rows behind the last one stay as they were.
    buf = torch.full((M + 40, N), 7.0, dtype=torch.bfloat16, device="cuda")
    cuda_lib.gemm_fp8(*args, **kw, out=buf[:M])
    check_close(num(buf[:M]), ref, err + BF16 * (np.abs(ref) + err), f"M={M}")
    assert (buf[M:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(2001, 2064, 400), (4000, 1296, 1040), (1500, 3344, 272)])
def test_gemm_ragged_tiles_of_many_rows(cuda_lib, M, N, K):
    """Weights in blocks with enough rows for 256 x 256 tiles, ragged in every direction."""
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, False, False, True, "e4m3", "e4m3", False, seed=M)
    buf = torch.full((M + 300, N), 7.0, dtype=torch.bfloat16, device="cuda")
    cuda_lib.gemm_fp8(*args, **kw, out=buf[:M])
    check_close(num(buf[:M]), ref, err + BF16 * (np.abs(ref) + err), f"M={M}")
    assert (buf[M:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (5, 4096, 4096), (16, 2048, 8192), (20, 1040, 11008), (48, 512, 65536),
                                   (200, 4096, 1024), (7, 128, 128), (64, 8192, 272), (100, 144, 2000)])
def test_gemm_few_rows(cuda_lib, M, N, K):
    """One to a few hundred rows: the reduction split over clusters of 1 to 8, with and without a remainder."""
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, False, False, True, "e4m3", "e5m2", True, seed=K)
    one = cuda_lib.gemm_fp8(*args, **kw)
    check_close(num(one), ref, err, "few rows")
    assert torch.equal(one, cuda_lib.gemm_fp8(*args, **kw))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,b_mn", [
    (65, 256, 2048, False),     # 4 pairs of 4 blocks each
    (129, 272, 2064, False),    # 17 blocks over 4 pairs, the last one short
    (700, 1040, 4112, True),    # a short last tile both ways, MN-major weight
    (257, 16, 4096, False),     # one row in the second tile, one tile of 16 columns
    (4700, 256, 2320, False),   # 19 tiles: 3 pairs each, shares of 42 and 43 rows
    (1001, 2048, 3344, True),   # 32 tiles: 2 pairs each
])
def test_gemm_reduction_shared_by_pairs(cuda_lib, M, N, K, b_mn, f32):
    """Fewer tiles than pairs of SMs: the partial tiles are added in a fixed order, rows behind the last one are left."""
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, False, b_mn, True, "e4m3", "e5m2", f32, seed=M)
    buf = torch.full((M + 300, N), 7.0, dtype=kw["out_dtype"], device="cuda")
    ws = cuda_lib.Workspace(256)
    cuda_lib.gemm_fp8(*args, **kw, out=buf[:M], ws=ws)
    first = buf[:M].clone()
    assert (buf[M:] == 7.0).all() and ws.query() == (0, 0)
    check_close(num(first), ref, err if f32 else err + BF16 * (np.abs(ref) + err), "shared")
    for _ in range(5):
        assert _same(cuda_lib.gemm_fp8(*args, **kw), first)
    if f32:
        start = _randn(M, N, seed=3)
        C = start.cuda()
        cuda_lib.gemm_fp8(*args, **kw, accumulate=True, out=C)
        want = num(start) + ref
        check_close(num(C), want, err + FP32 * (np.abs(want) + err), "added")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("parts,N,K,b_mn", [(4, 256, 2320, False), (3, 256, 2320, False), (3, 256, 2320, True), (2, 512, 4096, True),
                                            (2, 256, 3088, False), (1, 256, 2320, False)])
def test_gemm_reduction_shared_by_a_known_number_of_pairs(cuda_lib, parts, N, K, b_mn, f32):
    """The most tiles that this device shares between `parts` pairs (shares of 32, of 42 and 43, of 64 rows each),
    as the library says; one part: the fewest tiles that are not shared."""
    dtype = torch.float32 if f32 else torch.bfloat16
    how = lambda m: cuda_lib.gemm_fp8_parts(256 * m, N, K, b_mn_major=b_mn, out_dtype=dtype)
    tiles = [m for m in range(1, 80) if how(m) == (False, parts)]
    assert tiles, [how(m) for m in range(1, 80)]
    M = 256 * (tiles[0] if parts == 1 else tiles[-1]) - 39   # a short last tile
    assert cuda_lib.gemm_fp8_parts(M, N, K, b_mn_major=b_mn, out_dtype=dtype) == (False, parts)
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, False, b_mn, True, "e4m3", "e5m2", f32, seed=M)
    buf = torch.full((M + 300, N), 7.0, dtype=dtype, device="cuda")
    ws = cuda_lib.Workspace(256)
    cuda_lib.gemm_fp8(*args, **kw, out=buf[:M], ws=ws)
    assert (buf[M:] == 7.0).all() and ws.query() == (0, 0)
    check_close(num(buf[:M]), ref, err if f32 else err + BF16 * (np.abs(ref) + err), f"{parts} parts")
    first = buf[:M].clone()
    for _ in range(3):
        assert _same(cuda_lib.gemm_fp8(*args, **kw), first)


@pytest.mark.parametrize("M,N,K,kw,few,parts", [
    (65, 256, 2048, {}, False, (4,)), (129, 272, 2064, {}, False, (4,)), (257, 16, 4096, {}, False, (4,)),
    (8192, 4096, 11008, {}, False, (1,)), (256, 4096, 8192, dict(a_mn_major=True, b_mn_major=True, b_blocks=False), False, (1,)),
    (64, 4096, 4096, {}, True, (8,)), (1, 16, 16, {}, True, (1,)), (3, 8192, 4096, {}, True, (4,)),
    # 16 clusters of 8, or 32 of 4, fit into the number of SMs but not into the GPCs of every device.
    (64, 4096, 4096, dict(b_mn_major=True), False, (3, 4)), (1001, 2048, 3344, dict(b_mn_major=True), False, (1, 2))])
def test_gemm_parts(cuda_lib, M, N, K, kw, few, parts):
    got = cuda_lib.gemm_fp8_parts(M, N, K, **kw)
    assert got[0] == few and got[1] in parts


@pytest.mark.parametrize("K", [1, 2, 127, 128, 129, 1000])
def test_gemm_any_reduction_for_weight_gradients(cuda_lib, K):
    args, kw, ref, err = _gemm_case(cuda_lib, 272, 400, K, True, True, False, "e5m2", "e4m3", True, seed=K)
    check_close(num(cuda_lib.gemm_fp8(*args, **kw)), ref, err, f"K={K}")


@pytest.mark.parametrize("M,N,K,a_mn,b_mn,blocks", [(272, 400, 333, True, True, False), (3, 528, 640, False, False, True)])
def test_gemm_accumulates(cuda_lib, M, N, K, a_mn, b_mn, blocks):
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, a_mn, b_mn, blocks, "e4m3", "e4m3", True, seed=4)
    start = _randn(M + 8, N, seed=6)
    C = start.cuda()
    for n in (1, 2):
        cuda_lib.gemm_fp8(*args, **kw, accumulate=True, out=C[:M])
        want = num(start[:M]) + n * ref
        check_close(num(C[:M]), want, n * err + n * FP32 * (np.abs(want) + n * err + np.abs(num(start[:M]))), f"pass {n}")
    assert torch.equal(C[M:].cpu(), start[M:])


def test_gemm_many_tiles_and_long_reduction(cuda_lib):
    """More tiles than CTA pairs, every TMEM buffer and stage reused many times."""
    M, N, K = 2304, 2560, 2048
    args, kw, ref, err = _gemm_case(cuda_lib, M, N, K, False, False, True, "e4m3", "e4m3", True, seed=8)
    one = cuda_lib.gemm_fp8(*args, **kw)
    check_close(num(one), ref, err, "many tiles")
    assert torch.equal(one, cuda_lib.gemm_fp8(*args, **kw))  # bit-identical from run to run


def test_gemm_nan_and_zero_blocks(cuda_lib):
    """A NaN reaches its row only; all-zero blocks give exact zeros."""
    x = _bf(40, 512, seed=3)
    x[5, 100] = float("nan")
    x[6] = 0.0
    q = cuda_lib.quant_fp8(x.cuda())
    w = cuda_lib.quant_fp8_blocks(_bf(272, 512, seed=4).cuda())
    C = cuda_lib.gemm_fp8(q["Qr"], q["Sr"], w["Q"], w["S"], 40, 272, 512).float().cpu()
    assert torch.isnan(C[5]).all() and (C[6] == 0).all()
    keep = [i for i in range(40) if i != 5]
    assert torch.isfinite(C[keep]).all()


def test_gemm_empty(cuda_lib):
    e4 = torch.float8_e4m3fn
    z = lambda *s: torch.empty(*s, device="cuda", dtype=e4)
    f = lambda *s: torch.empty(*s, device="cuda")
    assert cuda_lib.gemm_fp8(z(0, 128), f(1, 0), z(256, 128), f(2, 1), 0, 256, 128).shape == (0, 256)
    C = torch.full((32, 64), 3.0, device="cuda")
    out = cuda_lib.gemm_fp8(z(0, 32), f(0, 32), z(0, 64), f(0, 64), 32, 64, 0, a_mn_major=True, b_mn_major=True,
                            b_blocks=False, out_dtype=torch.float32, out=C)
    assert (out == 0).all()
    C.fill_(3.0)
    cuda_lib.gemm_fp8(z(0, 32), f(0, 32), z(0, 64), f(0, 64), 32, 64, 0, a_mn_major=True, b_mn_major=True,
                      b_blocks=False, out_dtype=torch.float32, out=C, accumulate=True)
    assert (C == 3.0).all()


# ------------------------------------------------------------------ RMSNorm

RMS_SIZES = [(1, 16), (3, 128), (7, 272), (33, 1024), (20, 1040), (9, 2048), (5, 4096), (3, 4112), (2, 8192), (3, 16384),
             (2, 32768)]


@pytest.mark.parametrize("resid", [True, False])
@pytest.mark.parametrize("M,d", RMS_SIZES)
def test_rmsnorm_fwd(cuda_lib, M, d, resid):
    eps = 1e-5
    x, g = _bf(M, d, seed=d), (1 + 0.1 * _randn(d, seed=1)).bfloat16()
    res = _bf(M, d, seed=d + 1) if resid else None
    if M > 1:  # a row of zeros
        x[0] = 0.0
        if resid:
            res[0] = 0.0
    o = cuda_lib.rmsnorm_fp8_fwd(x.cuda(), g.cuda(), eps, R=res.cuda() if resid else None)
    h = (x.float() + res.float()).bfloat16() if resid else x
    if resid:
        assert torch.equal(o["H"].cpu(), h)
    else:
        assert "H" not in o
    r, n = O.rmsnorm(num(h), num(g), eps)
    # At most 32 + 10 fp32 additions of squares (halved by the root), 1/d and eps, and rsqrtf's 2 ulp.
    rel = (42 / 2 + 4 + 4) * FP32
    check_close(num(o["r"]), r, r * rel, "r")
    check_quant(o["Q"], o["S"], n, "rows", "e4m3", "n", np.abs(n) * (rel + 2 * FP32))


@pytest.mark.parametrize("M,d", RMS_SIZES + [(1500, 512), (700, 1040)])
def test_rmsnorm_bwd(cuda_lib, M, d):
    h, g = _bf(M, d, seed=d), (1 + 0.1 * _randn(d, seed=1)).bfloat16()
    dn, dhi = _bf(M, d, seed=2, scale=0.1), _bf(M, d, seed=3)
    r = torch.from_numpy(O.rmsnorm(num(h), num(g), 1e-6)[0]).float()
    u = num(dn) * num(g)
    for extra in (None, dhi):
        o = cuda_lib.rmsnorm_fp8_bwd(dn.cuda(), h.cuda(), r.cuda(), g.cuda(), dH_in=None if extra is None else extra.cuda())
        dh, dg = O.rmsnorm_bwd(num(dn), num(h), num(r), num(g), None if extra is None else num(extra))
        rr = num(r)[:, None]
        coef = np.abs(num(h)) * rr ** 3 * np.mean(np.abs(u * num(h)), axis=1, keepdims=True)
        # The row sum has at most 42 additions of products with two roundings; four more around it.
        err = 50 * FP32 * coef + 6 * FP32 * (np.abs(rr * u) + np.abs(dh))
        check_close(num(o["dH"]), dh, err + BF16 * (np.abs(dh) + err), "dH")
        each = np.abs(num(dn) * num(h) * rr)
        check_close(num(o["dg"]), dg, (M + 4) * FP32 * each.sum(0), "dg")
    # A gradient buffer longer than the batch keeps its tail.
    buf = torch.full((M + 3, d), 5.0, dtype=torch.bfloat16, device="cuda")
    cuda_lib.rmsnorm_fp8_bwd(dn.cuda(), h.cuda(), r.cuda(), g.cuda(), out={"dH": buf[:M]})
    assert (buf[M:] == 5.0).all()


def test_rmsnorm_empty(cuda_lib):
    z = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    o = cuda_lib.rmsnorm_fp8_fwd(z, g, 1e-6, R=z)
    assert o["Q"].shape == (0, 256) and o["S"].shape == (2, 0)
    b = cuda_lib.rmsnorm_fp8_bwd(z, z, torch.empty(0, device="cuda"), g)
    assert (b["dg"] == 0).all()


# ------------------------------------------------------------------ gate/up + SwiGLU and its backward

@pytest.mark.parametrize("M,K,F", [(1, 128, 128), (3, 272, 256), (16, 512, 384), (33, 400, 128), (64, 640, 1024), (2, 4096, 128), (17, 2048, 640), (40, 1296, 256),
                                   (65, 128, 256), (130, 1040, 384), (300, 512, 1280), (520, 256, 2560)])
def test_gemm_swiglu(cuda_lib, M, K, F):
    qa, sa, a64 = _operand(cuda_lib, _randn(M, K, seed=M), "rows")
    qw, sw, w64 = _operand(cuda_lib, _randn(2 * F, K, seed=K, scale=K ** -0.5), "blocks")
    ws = cuda_lib.Workspace(256)
    pad = 5  # rows behind the batch stay as they were
    buf = {"Y": torch.zeros(M + pad, F, device="cuda").fill_(9).to(TYPES["e4m3"]),
           "AB": torch.zeros(M + pad, 2 * F, device="cuda").fill_(9).to(TYPES["e4m3"])}
    o = cuda_lib.gemm_swiglu_fp8(qa, sa, qw, sw, out={k: v[:M] for k, v in buf.items()}, ws=ws)
    assert ws.query() == (0, 0)
    ab, err = a64 @ w64.T, gemm_error(a64, w64, K)
    a, b, ea, eb = ab[:, :F], ab[:, F:], err[:, :F], err[:, F:]
    check_quant(o["AB"], o["SAB"], ab, "rows", "e4m3", "[a | b]", err)
    check_quant(o["Y"], o["SY"], O.swiglu(a, b), "rows", "e4m3", "Y", swiglu_error(a, b, ea, eb))
    for v in buf.values():
        assert (v[M:].float() == 9).all()
    lean = cuda_lib.gemm_swiglu_fp8(qa, sa, qw, sw, save_ab=False)
    assert set(lean) == {"Y", "SY"}
    for k in lean:
        assert torch.equal(lean[k].view(torch.uint8), o[k].view(torch.uint8)), k


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,F", [(1, 128), (127, 256), (128, 128), (129, 384), (400, 1280)])
def test_swiglu_bwd(cuda_lib, M, F, fmt):
    pre = _randn(M, 2 * F, seed=M, scale=2.0)
    pre[:, 0] = 30.0   # saturated gates, both ways
    pre[:, 1] = -30.0
    q, s, ab = _operand(cuda_lib, pre, "rows")
    dy = _bf(M, F, seed=F, scale=0.05)
    dy[M // 2] = 0.0
    o = cuda_lib.swiglu_fp8_bwd(dy.cuda(), q, s, fmt=TYPES[fmt])
    a, b = ab[:, :F], ab[:, F:]
    da, db = O.swiglu_bwd(num(dy), a, b)
    ea, eb = swiglu_bwd_error(num(dy), a, b)
    dab, e = np.concatenate([da, db], 1), np.concatenate([ea, eb], 1)
    check_quant(o["dA"], o["SdA"], dab, "rows", fmt, "dA rows", e)
    check_quant(o["dAc"], o["SdAc"], dab, "cols", fmt, "dA cols", e)
    check_quant(o["Yc"], o["SYc"], O.swiglu(a, b), "cols", "e4m3", "Y cols",
                swiglu_error(a, b, np.abs(a) * FP32, np.abs(b) * FP32))
    lean = cuda_lib.swiglu_fp8_bwd(dy.cuda(), q, s, cols=False, fmt=TYPES[fmt])
    assert set(lean) == {"dA", "SdA"}
    for k in lean:
        assert torch.equal(lean[k].view(torch.uint8), o[k].view(torch.uint8)), k


# ------------------------------------------------------------------ the block with 8-bit operands

def _mlp(B, t, eps, M, d, F, o=None):
    """RMSNorm -> gate/up + SwiGLU -> down, forward and backward, every product on 8-bit operands."""
    o = o if o is not None else {}

    def keep(name, fn, *args, **kw):
        o[name] = fn(*args, **kw, out=o.get(name))
        return o[name]

    n = keep("n", B.rmsnorm_fp8_fwd, t["X"], t["g"], eps, R=t["R"])
    wgu, wd = keep("wgu", B.quant_fp8_blocks, t["Wgu"]), keep("wd", B.quant_fp8_blocks, t["Wd"])
    y = keep("y", B.gemm_swiglu_fp8, n["Q"], n["S"], wgu["Q"], wgu["S"])
    keep("Out", B.gemm_fp8, y["Y"], y["SY"], wd["Q"], wd["S"], M, d, F)
    e5 = torch.float8_e5m2
    go = keep("go", B.quant_fp8, t["dOut"], cols=True, fmt=e5)
    dy = keep("dY", B.gemm_fp8, go["Qr"], go["Sr"], wd["Q"], wd["S"], M, F, d, b_mn_major=True)
    da = keep("da", B.swiglu_fp8_bwd, dy, y["AB"], y["SAB"], fmt=e5)
    dn = keep("dN", B.gemm_fp8, da["dA"], da["SdA"], wgu["Q"], wgu["S"], M, d, 2 * F, b_mn_major=True)
    keep("nb", B.rmsnorm_fp8_bwd, dn, n["H"], n["r"], t["g"], dH_in=t["dOut"])
    nc = keep("nc", B.quant_fp8, n["H"], rows=False, cols=True, rowvec=n["r"], colvec=t["g"])
    w = dict(a_mn_major=True, b_mn_major=True, b_blocks=False, out_dtype=torch.float32)
    keep("dWd", B.gemm_fp8, go["Qc"], go["Sc"], da["Yc"], da["SYc"], d, F, M, **w)
    keep("dWgu", B.gemm_fp8, da["dAc"], da["SdAc"], nc["Qc"], nc["Sc"], 2 * F, d, M, **w)
    return o


def _mlp_inputs(M, d, F, seed=0):
    t = {"X": _bf(M, d, seed=seed), "R": _bf(M, d, seed=seed + 1), "g": (1 + 0.1 * _randn(d, seed=seed + 2)).bfloat16(),
         "Wgu": _bf(2 * F, d, seed=seed + 3, scale=d ** -0.5), "Wd": _bf(d, F, seed=seed + 4, scale=F ** -0.5),
         "dOut": _bf(M, d, seed=seed + 5, scale=0.05)}
    return {k: v.cuda() for k, v in t.items()}


def _flat(o):
    return {f"{k}.{j}": x for k, v in o.items() for j, x in (v.items() if isinstance(v, dict) else [("", v)])}


@pytest.mark.parametrize("M,d,F", [(300, 512, 640), (17, 256, 128)])
def test_mlp_on_8_bit_operands(cuda_lib, M, d, F):
    """The operators chained as a training step uses them; each is checked on what the one before gave it."""
    eps = 1e-6
    t = _mlp_inputs(M, d, F)
    o = _mlp(cuda_lib, t, eps, M, d, F)
    assert cuda_lib.fp8_status() == (0, 0)
    n, y, go, da, nb, nc = (o[k] for k in ("n", "y", "go", "da", "nb", "nc"))
    deq = lambda q, s, form: O.dequant(num(q), num(s), form)
    wgu, wd = deq(o["wgu"]["Q"], o["wgu"]["S"], "blocks"), deq(o["wd"]["Q"], o["wd"]["S"], "blocks")

    def product(got, a, b, k, name, f32=False):
        ref, err = a @ b.T, gemm_error(a, b, k)
        check_close(num(got), ref, err + (0 if f32 else BF16 * (np.abs(ref) + err)), name)

    r, nn = O.rmsnorm(num(n["H"]), num(t["g"]), eps)
    check_quant(n["Q"], n["S"], nn, "rows", "e4m3", "n", np.abs(nn) * 32 * FP32)
    a64 = deq(n["Q"], n["S"], "rows")
    ab, err = a64 @ wgu.T, gemm_error(a64, wgu, d)
    check_quant(y["AB"], y["SAB"], ab, "rows", "e4m3", "[a | b]", err)
    product(o["Out"], deq(y["Y"], y["SY"], "rows"), wd, F, "Out")
    product(o["dY"], deq(go["Qr"], go["Sr"], "rows"), wd.T, d, "dY")
    ab = deq(y["AB"], y["SAB"], "rows")
    a, b = ab[:, :F], ab[:, F:]
    dab = np.concatenate(O.swiglu_bwd(num(o["dY"]), a, b), 1)
    e = np.concatenate(swiglu_bwd_error(num(o["dY"]), a, b), 1)
    check_quant(da["dA"], da["SdA"], dab, "rows", "e5m2", "dA", e)
    product(o["dN"], deq(da["dA"], da["SdA"], "rows"), wgu.T, 2 * F, "dN")
    dh, dg = O.rmsnorm_bwd(num(o["dN"]), num(n["H"]), num(n["r"]), num(t["g"]), num(t["dOut"]))
    scale = np.abs(dh) + np.abs(num(o["dN"]) * num(n["r"])[:, None] * num(t["g"])) + np.abs(num(t["dOut"]))
    check_close(num(nb["dH"]), dh, (BF16 + 60 * FP32) * scale, "dH")
    product(o["dWd"], deq(go["Qc"], go["Sc"], "cols").T, deq(da["Yc"], da["SYc"], "cols").T, M, "dWd", True)
    want = num(n["H"]) * num(n["r"])[:, None] * num(t["g"])
    check_quant(nc["Qc"], nc["Sc"], want, "cols", "e4m3", "n cols", np.abs(want) * 3 * FP32)
    product(o["dWgu"], deq(da["dAc"], da["SdAc"], "cols").T, deq(nc["Qc"], nc["Sc"], "cols").T, M, "dWgu", True)


def test_mlp_graph_and_streams(cuda_lib):
    """A captured step replays bit for bit, on new inputs too; two captured graphs and a side stream share nothing."""
    M, d, F = 260, 256, 384
    t1, t2 = _mlp_inputs(M, d, F, seed=0), _mlp_inputs(M, d, F, seed=50)
    ref1, ref2 = (({k: v.clone() for k, v in _flat(_mlp(cuda_lib, t, 1e-6, M, d, F)).items()}) for t in (t1, t2))
    graphs, outs = [], []
    for t in (t1, t2):
        o = _mlp(cuda_lib, t, 1e-6, M, d, F)
        torch.cuda.synchronize()
        for v in _flat(o).values():
            v.view(torch.uint8).zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _mlp(cuda_lib, t, 1e-6, M, d, F, o)
        graphs.append(g), outs.append(o)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o, ref in zip(outs, (ref1, ref2)):
        for k, v in _flat(o).items():
            assert torch.equal(v.view(torch.uint8), ref[k].view(torch.uint8)), k
    for k in t1:  # the replay follows new values in the captured buffers
        t1[k].copy_(t2[k])
    graphs[0].replay()
    torch.cuda.synchronize()
    for k, v in _flat(outs[0]).items():
        assert torch.equal(v.view(torch.uint8), ref2[k].view(torch.uint8)), k
    assert cuda_lib.fp8_status() == (0, 0)


def test_first_call_inside_a_capture(cuda_lib):
    """A product whose status word does not exist yet can be captured: the graph gets one of its own."""
    q, s, a = _operand(cuda_lib, _randn(40, 256, seed=1), "rows")
    w, sw, b = _operand(cuda_lib, _randn(64, 256, seed=2), "blocks")
    out = torch.zeros(40, 64, dtype=torch.float32, device="cuda")
    kept = dict(cuda_lib._status_ws)
    cuda_lib._status_ws.clear()
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cuda_lib.gemm_fp8(q, s, w, sw, 40, 64, 256, out_dtype=torch.float32, out=out)
        assert not cuda_lib._status_ws
        g.replay()
        torch.cuda.synchronize()
    finally:
        cuda_lib._status_ws.update(kept)
    check_close(num(out), a @ b.T, gemm_error(a, b, 256), "captured")


def test_status_stays_until_cleared(cuda_lib):
    """The shared status word as a product that gave up would leave it (written here by the host)."""
    word = cuda_lib._status_workspace(torch.device("cuda", torch.cuda.current_device())).buf.view(torch.int32)
    word[0], word[1] = 7, 5
    assert cuda_lib.fp8_status() == (7, 5) and cuda_lib.fp8_status("cuda", clear=True) == (7, 5)
    assert cuda_lib.fp8_status("cuda:0") == (0, 0)


def test_profile_hook_names_the_8_bit_kernels(cuda_lib):
    B = cuda_lib
    t = _mlp_inputs(130, 256, 128)
    _mlp(B, t, 1e-6, 130, 256, 128)
    ids = (B.KERNEL_GEMM_FP8, B.KERNEL_GEMM_SWIGLU_FP8, B.KERNEL_QUANT_FP8, B.KERNEL_SWIGLU_FP8_BWD,
           B.KERNEL_RMSNORM_FP8_FWD, B.KERNEL_RMSNORM_FP8_BWD)
    ev = {k: (torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for k in ids}
    for k, (a, b) in ev.items():
        B.profile_arm(k, a, b)
    _mlp(B, t, 1e-6, 130, 256, 128)
    B.profile_arm(0)
    torch.cuda.synchronize()
    for k, (a, b) in ev.items():
        assert 0 < a.elapsed_time(b) < 50, k


# ------------------------------------------------------------------ addresses, streams, large tensors

def _shifted(t):
    """A copy of t whose storage starts 16 bytes behind a 32-byte boundary."""
    skip = 16 // t.element_size()
    buf = torch.zeros(t.numel() + 2 * skip, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
    v = buf[skip:skip + t.numel()].view(t.dtype).view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 32 == 16 and v.is_contiguous()
    return v


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("M", [20, 300])
def test_operands_and_outputs_at_16_byte_addresses(cuda_lib, M):
    B = cuda_lib
    N, K, F = 272, 400, 256
    args, kw, _, _ = _gemm_case(B, M, N, K, False, False, True, "e4m3", "e4m3", True, seed=1)
    moved = [_shifted(t) if isinstance(t, torch.Tensor) else t for t in args]
    for dtype in (torch.float32, torch.bfloat16):
        kw["out_dtype"] = dtype
        want = B.gemm_fp8(*args, **kw)
        out = _shifted(torch.zeros(M, N, dtype=dtype, device="cuda"))
        assert _same(B.gemm_fp8(*moved, **kw, out=out), want), dtype
    kw["out_dtype"] = torch.float32
    start = _randn(M, N, seed=2).cuda()
    sums = [B.gemm_fp8(*args, **kw, accumulate=True, out=c) for c in (start.clone(), _shifted(start))]
    assert _same(*sums)
    x = B.quant_fp8(_bf(M, K, seed=3).cuda())
    w = B.quant_fp8_blocks(_bf(2 * F, K, seed=4).cuda())
    o = B.gemm_swiglu_fp8(x["Qr"], x["Sr"], w["Q"], w["S"])
    at = {k: _shifted(torch.zeros_like(v, dtype=torch.float32).to(v.dtype)) for k, v in o.items()}
    B.gemm_swiglu_fp8(x["Qr"], x["Sr"], w["Q"], w["S"], out=at)
    for k in o:
        assert _same(at[k], o[k]), k
    dy = _bf(M, F, seed=5).cuda()
    g = B.swiglu_fp8_bwd(dy, o["AB"], o["SAB"])
    at = B.swiglu_fp8_bwd(_shifted(dy), _shifted(o["AB"]), _shifted(o["SAB"]),
                          out={k: _shifted(torch.zeros_like(v, dtype=torch.float32).to(v.dtype)) for k, v in g.items()})
    for k in g:
        assert _same(at[k], g[k]), k


def test_products_on_two_streams_at_once(cuda_lib):
    """Launches of the tile kernel, of the few-rows kernel and of the passes interleaved on two streams."""
    B = cuda_lib
    x, w = _bf(1030, 512, seed=1).cuda(), _bf(768, 512, seed=2).cuda()
    qx, qw = B.quant_fp8(x, cols=True), B.quant_fp8_blocks(w)
    few = {k: v[:7].contiguous() if k == "Qr" else v[:, :7].contiguous() for k, v in qx.items() if k in ("Qr", "Sr")}
    calls = [lambda: B.gemm_fp8(qx["Qr"], qx["Sr"], qw["Q"], qw["S"], 1030, 768, 512),
             lambda: B.gemm_fp8(few["Qr"], few["Sr"], qw["Q"], qw["S"], 7, 768, 512),
             lambda: B.gemm_fp8(qx["Qc"], qx["Sc"], qx["Qc"], qx["Sc"], 512, 512, 1030, a_mn_major=True, b_mn_major=True,
                                b_blocks=False, out_dtype=torch.float32),
             lambda: B.gemm_swiglu_fp8(qx["Qr"], qx["Sr"], qw["Q"], qw["S"])["Y"],
             lambda: B.quant_fp8(x, cols=True)["Qc"]]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for rep in range(10):
        for i, c in enumerate(calls):
            with torch.cuda.stream(streams[(rep + i) % 2]):
                got.append((i, c()))
    torch.cuda.synchronize()
    for i, t in got:
        assert _same(t, want[i]), i
    assert B.fp8_status() == (0, 0)


def test_shared_reductions_on_two_streams_and_in_a_graph(cuda_lib):
    """Products whose tiles are shared by clusters of pairs, at once on two streams and replayed."""
    B = cuda_lib
    cases = [(200, 512, 2304), (300, 1040, 4112)]
    calls, want = [], []
    for M, N, K in cases:
        x = B.quant_fp8(_bf(M, K, seed=M).cuda())
        w = B.quant_fp8_blocks(_bf(N, K, seed=N).cuda())
        calls.append(lambda x=x, w=w, M=M, N=N, K=K, **kw: B.gemm_fp8(x["Qr"], x["Sr"], w["Q"], w["S"], M, N, K, **kw))
        want.append(calls[-1]())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for rep in range(10):
        for i, c in enumerate(calls):
            with torch.cuda.stream(streams[(rep + i) % 2]):
                got.append((i, c()))
    torch.cuda.synchronize()
    for i, t in got:
        assert _same(t, want[i]), i
    outs = [torch.zeros_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c, o in zip(calls, outs):
            c(out=o)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(_same(o, t) for o, t in zip(outs, want)) and B.fp8_status() == (0, 0)


TAIL = 40  # rows checked at the end of a tensor of more than 2^32 elements


def test_quant_and_gemm_behind_32_bit_offsets(cuda_lib):
    B = cuda_lib
    R, C = 131200, 32768
    assert (R - TAIL) * C > 2 ** 32
    x = torch.randn(R, C, dtype=torch.bfloat16, device="cuda")
    o = B.quant_fp8(x, cols=True)
    tail = num(x[-128:])
    assert R % 128 == 0
    check_quant(o["Qr"][-TAIL:], o["Sr"][:, -TAIL:], tail[-TAIL:], "rows", "e4m3", "rows")
    check_quant(o["Qc"][-128:], o["Sc"][-1:], tail, "cols", "e4m3", "cols")
    del x, o["Qc"]
    # The long matrix as an operand, and (few columns in) as an output.
    qw, sw, w = _operand(B, _randn(16, C, seed=1), "blocks")
    c = B.gemm_fp8(o["Qr"], o["Sr"], qw, sw, R, 16, C, out_dtype=torch.float32)
    a = O.dequant(num(o["Qr"][-TAIL:]), num(o["Sr"][:, -TAIL:]), "rows")
    check_close(num(c[-TAIL:]), a @ w.T, gemm_error(a, w, C), "long operand")
    del o, c
    qx, sx, a = _operand(B, _randn(R, 16, seed=2), "rows")
    qw, sw, w = _operand(B, _randn(C, 16, seed=3), "blocks")
    c = B.gemm_fp8(qx, sx, qw, sw, R, C, 16)
    ref, err = a[-TAIL:] @ w.T, gemm_error(a[-TAIL:], w, 16)
    check_close(num(c[-TAIL:]), ref, err + BF16 * (np.abs(ref) + err), "long output")
    assert B.fp8_status() == (0, 0)


def test_rmsnorm_behind_32_bit_offsets(cuda_lib):
    M, d = 131200, 32768
    x = torch.randn(M, d, dtype=torch.bfloat16, device="cuda")
    g = (1 + 0.1 * _randn(d, seed=1)).bfloat16()
    o = cuda_lib.rmsnorm_fp8_fwd(x, g.cuda(), 1e-5)
    h = num(x[-TAIL:])
    r, n = O.rmsnorm(h, num(g), 1e-5)
    rel = (42 / 2 + 4 + 4) * FP32
    check_close(num(o["r"][-TAIL:]), r, r * rel, "r")
    check_quant(o["Q"][-TAIL:], o["S"][:, -TAIL:], n, "rows", "e4m3", "n", np.abs(n) * (rel + 2 * FP32))
    r32 = o["r"]
    del o
    b = cuda_lib.rmsnorm_fp8_bwd(x, x, r32, g.cuda())
    rr = num(r32[-TAIL:])
    dh, _ = O.rmsnorm_bwd(h, h, rr, num(g), None)
    u, rr = h * num(g), rr[:, None]
    coef = np.abs(h) * rr ** 3 * np.mean(np.abs(u * h), axis=1, keepdims=True)
    err = 50 * FP32 * coef + 6 * FP32 * (np.abs(rr * u) + np.abs(dh))
    check_close(num(b["dH"][-TAIL:]), dh, err + BF16 * (np.abs(dh) + err), "dH")


def test_swiglu_behind_32_bit_offsets(cuda_lib):
    B = cuda_lib
    M, F = 65664, 32768  # [a | b] has 2 F columns
    assert (M - TAIL) * 2 * F > 2 ** 32 and M % 128 == 0
    qx, sx, x = _operand(B, _randn(M, 16, seed=2), "rows")
    qw, sw, w = _operand(B, _randn(2 * F, 16, seed=3), "blocks")
    o = B.gemm_swiglu_fp8(qx, sx, qw, sw)
    ab, err = x[-128:] @ w.T, gemm_error(x[-128:], w, 16)
    a, b, ea, eb = ab[:, :F], ab[:, F:], err[:, :F], err[:, F:]
    check_quant(o["AB"][-128:], o["SAB"][:, -128:], ab, "rows", "e4m3", "[a | b]", err)
    check_quant(o["Y"][-128:], o["SY"][:, -128:], O.swiglu(a, b), "rows", "e4m3", "Y", swiglu_error(a, b, ea, eb))
    del o["Y"]
    dy = torch.randn(M, F, dtype=torch.bfloat16, device="cuda")
    g = B.swiglu_fp8_bwd(dy, o["AB"], o["SAB"])
    saved = O.dequant(num(o["AB"][-128:]), num(o["SAB"][:, -128:]), "rows")
    a, b, t = saved[:, :F], saved[:, F:], num(dy[-128:])
    dab, e = np.concatenate(O.swiglu_bwd(t, a, b), 1), np.concatenate(swiglu_bwd_error(t, a, b), 1)
    check_quant(g["dA"][-128:], g["SdA"][:, -128:], dab, "rows", "e4m3", "dA rows", e)
    check_quant(g["dAc"][-128:], g["SdAc"][-1:], dab, "cols", "e4m3", "dA cols", e)
    check_quant(g["Yc"][-128:], g["SYc"][-1:], O.swiglu(a, b), "cols", "e4m3", "Y cols",
                swiglu_error(a, b, np.abs(a) * FP32, np.abs(b) * FP32))
    assert B.fp8_status() == (0, 0)
