"""Rules that the 8-bit GEMM's source keeps so that its waits end (CPU only).

What these guard against would hang a GPU, so it is checked by reading.
"""

import os
import re

from gemm_epilogue_fusion_tmem_b200 import build

SRC = open(os.path.join(build.CSRC, "coda_gemm_fp8.cuh")).read()


def _drain():
    """The drain warps' part of the tile kernel: from its heading to the set-down of the CTA."""
    return SRC[SRC.index("drain and epilogue (both CTAs)"):SRC.index("few rows\n")]


def test_a_drain_warp_leaves_its_loops_as_a_whole():
    """tcgen05.ld.sync.aligned and __syncwarp need every lane: a lane that saw the abort flag
    while another did not would leave that one waiting for good."""
    left = [line.strip() for line in _drain().splitlines() if "abort_flag" in line and re.search(r"\b(break|return)\b", line)]
    assert len(left) >= 3
    assert all("__any_sync(0xffffffffu, *abort_flag)" in line for line in left), left


def test_no_mma_is_issued_after_a_wait_that_gave_up():
    """The operands may not have landed then, and the commit would tell the other CTA of the pair that a
    product is complete: the issuer's waits have a result and it is looked at before anything else."""
    part = SRC[SRC.index("MMA issuers (pair's leader)"):SRC.index("// ---------------------------------------------------------------- scales")]
    waits, mma = part.index("mbar_wait_issue"), part.index("umma_f8_stage_pair<")
    assert "mbar_wait_drain" not in part and part.count("mbar_wait_issue") == 2
    assert "if (!ok) break;" in part[waits:mma]


def test_waits_for_own_copies_do_not_end_with_the_configurable_limit():
    """coda_set_wait_limit_ns may be as short as a microsecond, less than a copy takes: the waits before shared
    memory or TMEM is released have a bound of their own, and running out of it is recorded."""
    ptx = open(os.path.join(build.CSRC, "coda_ptx.cuh")).read()
    own = ptx[ptx.index("void mbar_wait_own("):]
    own = own[:own.index("\n}\n")]
    assert "c.limit_ns > kOwnWaitNs ? c.limit_ns : kOwnWaitNs" in own and "record_timeout(c, role, kWaitDrain)" in own
    assert int(re.search(r"kOwnWaitNs = (\d+)ull", ptx)[1]) >= 10**9
    waits = re.findall(r"mbar_wait_own\(.*?\);", SRC)
    assert len(waits) >= 3 and all(", ctl, " in w for w in waits)
    # Every commit that tells that all MMAs are complete is waited for before the roles meet.
    for m in re.finditer(r"umma_commit(_pair)?\([^;]*mma_done[^;]*;\s*(\w+)\(", SRC):
        assert m[2] == "mbar_wait_own"


def test_the_bf16_gemm_waits_for_its_own_copies_and_mmas_too():
    src = open(os.path.join(build.CSRC, "coda_gemm.cuh")).read()
    after = src[src.index("else umma_commit(mma_done);"):]
    assert after.splitlines()[1].strip().startswith("mbar_wait_own(mma_done, 0,")
    end = src[src.index("es.finish();"):]
    assert "pair_copies_landed<S>(" in end and "ctl.limit_ns" not in end
