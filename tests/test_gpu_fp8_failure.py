"""The 8-bit products when an arrival is lost: every wait ends, the status word says so, nothing is
stored of the tile that was not completed, and the next call is as ever.

One role of one block is kept silent (coda_selftest_fp8_silence), so that the waits on it run out.  The
limit is far longer than any copy or product takes, so nothing is in flight when a role gives up.
"""

import contextlib
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

TIMEOUT = 7
LIMIT_NS = 50_000_000
LOADS, MMA, SCALES = 1, 2, 3


@contextlib.contextmanager
def silence(B, role, cta):
    B.set_wait_limit_ns(LIMIT_NS)
    B.selftest_fp8_silence(role, cta)
    try:
        yield
    finally:
        B.selftest_fp8_silence(0)
        B.set_wait_limit_ns(4_000_000_000)


def _bf(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def _raw(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def _call(B, name, M=600, N=512, K=1280):
    """(function of (out, ws) that runs the product on fixed operands, its outputs as they are before)."""
    if name == "wgrad":
        a, b = (B.quant_fp8(_bf(K, n, seed=n), rows=False, cols=True) for n in (M + 8, N))
        args = (a["Qc"], a["Sc"], b["Qc"], b["Sc"], M + 8, N, K)
        kw = dict(a_mn_major=True, b_mn_major=True, b_blocks=False, out_dtype=torch.float32, accumulate=True)
        return (lambda out, ws: B.gemm_fp8(*args, **kw, out=out["C"], ws=ws)), {"C": torch.full((M + 8, N), 7.0, device="cuda")}
    x = B.quant_fp8(_bf(M, K, seed=1))
    if name == "swiglu":
        w = B.quant_fp8_blocks(_bf(2 * N, K, seed=2))
        new = {k: torch.full(s, 1.5, device="cuda").to(torch.float8_e4m3fn) for k, s in (("Y", (M, N)), ("AB", (M, 2 * N)))}
        new |= {k: torch.full(s, 7.0, device="cuda") for k, s in (("SY", (N // 128, M)), ("SAB", (N // 64, M)))}
        return (lambda out, ws: B.gemm_swiglu_fp8(x["Qr"], x["Sr"], w["Q"], w["S"], out=out, ws=ws)), new
    w = B.quant_fp8_blocks(_bf(N, K, seed=2))
    f32 = name == "add"
    new = torch.full((M, N), 7.0, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    kw = dict(out_dtype=new.dtype, accumulate=f32)
    return (lambda out, ws: B.gemm_fp8(x["Qr"], x["Sr"], w["Q"], w["S"], M, N, K, **kw, out=out["C"], ws=ws)), {"C": new}


def _run(B, name, role, cta, tile, **sizes):
    """Run once as ever and once with a silent role; returns for each output (before, as ever, silent) and the
    part `tile` of it."""
    call, new = _call(B, name, **sizes)
    ws = B.Workspace(256)
    clone = lambda d: {k: v.clone() for k, v in d.items()}
    want = clone(new)
    call(want, ws)
    assert ws.query() == (0, 0)
    got = clone(new)
    t0 = time.perf_counter()
    with silence(B, role, cta):
        call(got, ws)
        status, detail = ws.query()
    assert time.perf_counter() - t0 < 3.0
    assert status == TIMEOUT and detail >> 16 != 0
    for k in new:
        here = tile(k, new[k])
        before, silent, ever = _raw(new[k]), _raw(got[k]), _raw(want[k])
        assert torch.equal(silent[here], before[here]), f"{k}: the tile was stored"
        rest = torch.ones(new[k].shape, dtype=torch.bool, device="cuda")
        rest[here] = False
        assert torch.equal(silent[rest], ever[rest]), f"{k}: other tiles"
    ws.clear()
    again = clone(new)
    call(again, ws)
    assert ws.query() == (0, 0)
    for k in new:
        assert torch.equal(_raw(again[k]), _raw(want[k])), k


def _first_tile(name):
    """What block 0's pair computes: 256 rows, and 256 columns or the 128 of a gate/up tile."""
    def part(key, t):
        if name != "swiglu":
            return (slice(0, 256), slice(0, 256))
        if key in ("SY", "SAB"):
            blocks = t.shape[0]
            rows = [0] if key == "SY" else [0, blocks // 2]
            return (torch.tensor(rows, device="cuda")[:, None], torch.arange(256, device="cuda")[None, :])
        cols = torch.arange(128, device="cuda")
        if key == "AB":
            cols = torch.cat([cols, cols + t.shape[1] // 2])
        return (torch.arange(256, device="cuda")[:, None], cols[None, :])
    return part


@pytest.mark.parametrize("name", ["bf16", "add", "wgrad", "swiglu"])
@pytest.mark.parametrize("role,cta", [(SCALES, 0), (SCALES, 1), (MMA, 0)])
def test_tile_of_a_pair_that_gave_up_is_not_stored(cuda_lib, name, role, cta):
    """The scales of either CTA, or the products: neither CTA of the pair stores its rows of the tile."""
    _run(cuda_lib, name, role, cta, _first_tile(name))


@pytest.mark.parametrize("name", ["bf16", "wgrad", "swiglu"])
@pytest.mark.parametrize("cta", [0, 1])
def test_copies_of_one_cta_of_a_pair_are_waited_for(cuda_lib, name, cta):
    """One CTA's operand copies never start: the other's stages, announced or not, are settled before the
    CTAs end, without waiting for bytes that will not come (six stages of at least two seconds each)."""
    _run(cuda_lib, name, LOADS, cta, _first_tile(name), K=1920)


def _few_rows_tile(name):
    """The 128 columns that cluster 0 computes of a product of few rows."""
    def part(key, t):
        if key in ("SY", "SAB"):
            rows = [0] if key == "SY" else [0, t.shape[0] // 2]
            return (torch.tensor(rows, device="cuda")[:, None], torch.arange(t.shape[1], device="cuda")[None, :])
        cols = torch.arange(128, device="cuda")
        if key == "AB":
            cols = torch.cat([cols, cols + t.shape[1] // 2])
        return (torch.arange(t.shape[0], device="cuda")[:, None], cols[None, :])
    return part


@pytest.mark.parametrize("name", ["bf16", "add"])
@pytest.mark.parametrize("role,cta", [(MMA, 2), (MMA, 0), (SCALES, 7), (SCALES, 2)])
def test_shared_tile_of_which_a_part_is_missing_is_not_stored(cuda_lib, name, role, cta):
    """Four pairs share the reduction of a tile and one of them gives up: none adds what is left in its place."""
    _run(cuda_lib, name, role, cta, _first_tile(name), M=300, K=4112)


@pytest.mark.parametrize("name", ["bf16", "add", "swiglu"])
@pytest.mark.parametrize("M,K,role,cta", [(5, 4096, MMA, 3), (5, 4096, LOADS, 0), (20, 2048, MMA, 7), (32, 2048, LOADS, 5),
                                          (3, 256, MMA, 0)])
def test_few_rows_of_which_a_part_is_missing_are_not_stored(cuda_lib, name, M, K, role, cta):
    """The same for the CTAs that share the reduction of a product of few rows."""
    _run(cuda_lib, name, role, cta, _few_rows_tile(name), M=M, N=256, K=K)


def _product(B, seed=1):
    x, w = B.quant_fp8(_bf(40, 256, seed=seed)), B.quant_fp8_blocks(_bf(64, 256, seed=seed + 1))
    return lambda **kw: B.gemm_fp8(x["Qr"], x["Sr"], w["Q"], w["S"], 40, 64, 256, **kw)


def test_status_of_products_captured_before_the_first_eager_one(cuda_lib):
    """All products without a workspace share one word, which fp8_status reads: captured ones too."""
    B = cuda_lib
    dev = torch.device("cuda", torch.cuda.current_device())
    word = B._status_workspace(dev).buf.data_ptr()
    call = _product(B)
    want = call()
    out = torch.zeros_like(want)
    kept = dict(B._status_ws)
    B._status_ws.clear()
    try:
        graphs = [torch.cuda.CUDAGraph() for _ in range(3)]
        for i, g in enumerate(graphs):
            with contextlib.ExitStack() as stack:
                if i == 1:
                    stack.enter_context(silence(B, MMA, 0))
                stack.enter_context(torch.cuda.graph(g))
                call(out=out)
        graphs[0].replay()
        assert B.fp8_status() == (0, 0) and torch.equal(out, want)
        graphs[1].replay()
        assert B.fp8_status()[0] == TIMEOUT
        graphs[2].replay()
        assert B.fp8_status(clear=True)[0] == TIMEOUT and torch.equal(out, want)   # it stays until cleared
        graphs[2].replay()
        assert B.fp8_status() == (0, 0)
        assert B._status_workspace(dev).buf.data_ptr() == word
    finally:
        B._status_ws.clear()
        B._status_ws.update(kept)


def test_status_word_of_first_calls_on_several_threads(cuda_lib):
    import threading
    B = cuda_lib
    dev = torch.device("cuda", torch.cuda.current_device())
    kept = dict(B._status_ws)
    B._status_ws.clear()
    try:
        start, seen = threading.Barrier(8), []

        def first():
            start.wait()
            seen.append(B._status_workspace(dev).buf.data_ptr())
        threads = [threading.Thread(target=first) for _ in range(8)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        B._status_ws.clear()
        assert len(seen) == 8 and set(seen) == {B._status_workspace(dev).buf.data_ptr()}
    finally:
        B._status_ws.clear()
        B._status_ws.update(kept)


FIRST = """
import torch
from gemm_epilogue_fusion_tmem_b200 import binding as B
e4 = torch.float8_e4m3fn
a, w = torch.ones(40, 256, device="cuda").to(e4), torch.ones(64, 256, device="cuda").to(e4)
sa, sw = torch.ones(2, 40, device="cuda"), torch.ones(1, 2, device="cuda")
out = torch.zeros(40, 64, device="cuda", dtype=torch.bfloat16)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.gemm_fp8(a, sa, w, sw, 40, 64, 256, out=out)
g.replay()
assert B.fp8_status() == (0, 0) and (out == 256).all()
print("captured first")
"""


def test_the_first_call_of_a_process_may_be_captured(cuda_lib):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured first" in run.stdout, run.stderr[-2000:]


def test_workspaces_of_another_device_are_refused(cuda_lib):
    B = cuda_lib
    ws = B.Workspace(1 << 20, "cpu")
    with pytest.raises(ValueError, match="ws is on cpu"):
        _product(B)(ws=ws)
    x, w = B.quant_fp8(_bf(40, 256, seed=1)), B.quant_fp8_blocks(_bf(256, 256, seed=2))
    with pytest.raises(ValueError, match="ws is on cpu"):
        B.gemm_swiglu_fp8(x["Qr"], x["Sr"], w["Q"], w["S"], ws=ws)
    h = _bf(4, 256, seed=3)
    with pytest.raises(ValueError, match="ws is on cpu"):
        B.rmsnorm_fp8_bwd(h, h, torch.ones(4, device="cuda"), h[0], ws=ws)
