// 8-bit GEMM with a scale for each block of 128 (sm_100a, tcgen05 kind::f8f6f4).
//
//   C[m, n] = sum_kb SA[kb, m] SB(kb, n) sum_{k in kb} A[m, k] B[n, k]
//
// The inner sum over 128 values runs in the tensor cores into fp32 TMEM; the
// outer sum cannot, because its scales change with kb, so every 128-deep
// partial tile is drained, scaled and added to fp32 registers.  The drain is
// what bounds the design: per 128 of k an SM's tensor core needs 512 clocks
// for 128 x 256 outputs, and in those the warps must read 128 KB of TMEM and
// issue 32768 fused multiply-adds (256 clocks each at full rate).
//
// Tile: a CTA pair (cta_group::2) computes 256 x 256, each CTA holding 128 rows
// of A and half of B.  The 256 columns are issued as two halves of 128, each
// with its own two TMEM buffers (4 x 128 columns) and its own four warps, so a
// half's drain has the time of three half-products (768 clocks) to hide the
// commit, the TMEM reads and the arrival that crosses to the pair's leader.
// Half h is columns [128 h, 128 h + 128): 64 rows of B from each CTA (the
// operand's pair order), which makes it one 128-wide scale block of a weight,
// and in the gate/up product 64 gate columns beside the same 64 up columns.
//
// Roles (384 threads, one CTA per SM): warp 0 TMA producer; warp 1 TMEM owner
// and MMA issuer (pair's leader); warp 2 copies the scales of the blocks ahead
// into a ring of their own (read by the drain directly, their latency was paid
// once per 128 of k: 743 us against NEWTIME for the 7B down projection); warps 4-7 drain half 0, warps 8-11 half 1,
// one output row and 128 columns (128 fp32 registers) per thread.  The first
// warpgroup hands registers to the other two: 128 x 40 + 256 x 232 is the
// launch's 384 x 168.  Waits are bounded (mbar_wait); a role that gives up
// records it and the CTA drains and exits.
#pragma once

#include "coda_fp8.cuh"
#include "coda_gemm.cuh"

namespace coda {

constexpr int F8_BK = 128;          // reduction depth of a stage and of a scale block
constexpr int F8_UMMA_K = 32;
constexpr int F8_THREADS = 384;
constexpr int F8_REGS_ISSUE = 40, F8_REGS_DRAIN = 232;
static_assert(128 * F8_REGS_ISSUE + 256 * F8_REGS_DRAIN <= 384 * 168, "registers of the launch");
constexpr int F8_STAGES = 5;
constexpr int F8_A_BYTES = 128 * F8_BK;
constexpr int F8_B_BYTES = 128 * F8_BK;
constexpr int F8_STAGE_BYTES = F8_A_BYTES + F8_B_BYTES;
constexpr int F8_EPI_WARPS = 8;
constexpr int F8_SLOTS = 3;                    // staging tiles per epilogue warp
constexpr int F8_SLOT_BYTES = 32 * 64;         // 32 rows x 64 bytes
constexpr int F8_WARP_STAGING = F8_SLOTS * F8_SLOT_BYTES;
constexpr int F8_SCALE_STAGES = 6;
constexpr int F8_SCALE_FLOATS = 128 + 256;     // row scales, column scales (or two block scales)
constexpr int F8_SCALE_BYTES = F8_SCALE_STAGES * F8_SCALE_FLOATS * 4;
constexpr int F8_XCH_BYTES = 2 * 2 * 3 * 128 * 4;         // row maxima of the two halves, double-buffered
constexpr int F8_SMEM_BYTES =
    F8_STAGES * F8_STAGE_BYTES + F8_EPI_WARPS * F8_WARP_STAGING + F8_SCALE_BYTES + F8_XCH_BYTES + 1024 + 256;
static_assert(F8_SMEM_BYTES <= 232448, "shared memory of one CTA");

enum F8Epi : int {
  F8_EPI_BF16 = 0,    // C bf16
  F8_EPI_F32 = 1,     // C fp32, stored or added to what is there
  F8_EPI_SWIGLU = 2,  // a | b -> Y = silu(a) b in 8 bits (+ [a | b] in 8 bits)
};

struct Gemm8Params {
  int M, N, K;      // F8_EPI_SWIGLU: N = F
  int num_m_tiles, num_n_tiles, k_blocks;
  int group_m;
  const float* sa;  // [k_blocks, M]
  const float* sb;  // blocks: sb[n_block * sb_n + kb * sb_k]; columns: [k_blocks, N]
  int sb_n, sb_k;
  int split;        // F8_EPI_SWIGLU: row offset of the up half in B (= F)
  int add;          // F8_EPI_F32: add to C
  int save_ab;      // F8_EPI_SWIGLU
  float* sy;        // [F / 128, M]
  float* sab;       // [2 F / 128, M]
  uint32_t idesc;
  uint32_t* status;
  unsigned long long wait_limit_ns;
  uint32_t kernel_id;
};

// Instruction descriptor for kind::f8f6f4, fp32 D (bit positions as make_idesc_bf16;
// operand formats 0 = e4m3, 1 = e5m2, which may differ between A and B).
inline uint32_t make_idesc_f8(int m, int n, int a_fmt, int b_fmt, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | ((uint32_t)b_fmt << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Shared-memory matrix descriptor with the 64-byte swizzle (layout 4).
__device__ __forceinline__ uint64_t make_sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (make_sdesc_sw128(saddr, lbo, sbo) & ~((uint64_t)7 << 61)) | ((uint64_t)4 << 61);
}

// True in one lane of a converged warp.  The MMA issuer is chosen this way:
// behind it the compiler knows that a single thread runs and keeps the
// descriptors in uniform registers.  Behind `lane == 0` an MMA took 120 clocks
// to issue whatever its size, which held the 8-bit product at half its rate.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// D = A B^T over one 128-deep stage: four MMAs of K = 32, A_STEP and B_STEP the
// descriptors' advance between them (bytes / 16).
template <int A_STEP, int B_STEP>
__device__ __forceinline__ void umma_f8_stage_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .b64 a, b;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, 0;\n\t"
      "add.u64 a, %1, %4;\n\tadd.u64 b, %2, %5;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
      "add.u64 a, %1, 2 * %4;\n\tadd.u64 b, %2, 2 * %5;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
      "add.u64 a, %1, 3 * %4;\n\tadd.u64 b, %2, 3 * %5;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(A_STEP), "n"(B_STEP)
      : "memory");
}

// 64 accumulator columns of this thread's TMEM lane; valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}
// Wait for every TMEM load of this thread; ties `r` to a point after the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

// Asynchronous 4- or 16-byte copy to shared memory; zeros when !valid.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES),
               "r"(valid ? BYTES : 0)
               : "memory");
}
// Arrive on `bar` (whose count includes this thread) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Hand a drained TMEM buffer to the pair's leader.  What is handed over are TMEM
// loads that tcgen05.wait::ld has completed, no ordinary memory, so the arrival
// needs no cluster-scope release: that one waits for a memory barrier, once per
// 128 of k.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), 0)) : "memory");
}

// Packed pairs of floats: one instruction for two multiply-adds.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pack_u32x2(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// acc[0..63] (128 columns in pairs) += TMEM columns times lo (columns 0-63) or
// hi (64-127); with VEC the columns have scales of their own in cs[128]
// (shared memory).  Two loads of 64 columns: each exposes its latency once, and
// the buffer is handed back (release) as soon as the second has arrived.
template <bool VEC, typename Release>
__device__ __forceinline__ void f8_promote(uint32_t taddr, float lo, float hi, const float* cs, uint64_t (&acc)[64],
                                           Release release) {
  uint32_t v[64];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    tmem_ld64(taddr + c * 64, v);
    tmem_wait_ld(v);
    if (c == 1) release();
    const float s = c ? hi : lo;
    const uint64_t s2 = pack_f32x2(s, s);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      uint64_t x = pack_u32x2(v[2 * i], v[2 * i + 1]);
      uint64_t y = pack_u32x2(v[2 * i + 2], v[2 * i + 3]);
      if constexpr (VEC) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(cs + c * 64 + 2 * i);
        x = mul_f32x2(x, q.x);
        y = mul_f32x2(y, q.y);
      }
      acc[c * 32 + i] = fma_f32x2(x, s2, acc[c * 32 + i]);
      acc[c * 32 + i + 1] = fma_f32x2(y, s2, acc[c * 32 + i + 1]);
    }
  }
}

// Per-warp tile store: 32 rows x 64 bytes per slot (any element type), 16-byte
// chunks swizzled as the tensor map's 64-byte swizzle, one TMA store (or
// fp32 add) per slot.  Slots rotate, so a step waits only for the store issued
// F8_SLOTS steps before it.
struct F8Store {
  uint8_t* stg;
  int lane, row0, rows, slot;

  __device__ __forceinline__ void put(const uint4 (&q)[4], const CUtensorMap* m, int x, bool add) {
    static_assert(F8_SLOTS == 3, "the wait below leaves F8_SLOTS - 1 = 2 groups in flight");
    if (lane == 0) bulk_wait_read_2();
    __syncwarp();
    uint8_t* t = stg + slot * F8_SLOT_BYTES;
    const int sw = (lane >> 1) & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = smem_u32(t + lane * 64 + ((j ^ sw) << 4));
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(q[j].x), "r"(q[j].y), "r"(q[j].z),
                   "r"(q[j].w)
                   : "memory");
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (row0 < rows) {
        if (add)
          asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                           reinterpret_cast<uint64_t>(m)),
                       "r"(smem_u32(t)), "r"(x), "r"(row0)
                       : "memory");
        else
          tma_store_2d_hint(m, t, x, row0, l2_policy_evict_first());
      }
      bulk_commit_group();  // an empty group keeps the count of groups in step with the slots
    }
    slot = slot + 1 == F8_SLOTS ? 0 : slot + 1;
  }
  __device__ __forceinline__ void finish() {
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

template <int EPI, bool A_MN, bool B_MN, bool VEC>
__global__ void __launch_bounds__(F8_THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmO1, const __grid_constant__ CUtensorMap tmO2,
                    const Gemm8Params p) {
  constexpr int S = F8_STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + S * F8_A_BYTES;
  uint8_t* sEpi = sB + S * F8_B_BYTES;
  float* sScale = reinterpret_cast<float*>(sEpi + F8_EPI_WARPS * F8_WARP_STAGING);
  float* sXch = sScale + F8_SCALE_BYTES / 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(sXch + F8_XCH_BYTES / 4);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;   // [2 * parity + half]
  uint64_t* tempty = tfull + 4;
  uint64_t* xch = tempty + 4;
  uint64_t* sfull = xch + 1;
  uint64_t* sempty = sfull + F8_SCALE_STAGES;
  uint64_t* mma_done = sempty + F8_SCALE_STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();  // 0 = the pair's leader
  const int first_tile = (int)cluster_id_x();
  const int tile_step = (int)num_clusters_x();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 4; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 8);  // four warps of each CTA
    }
    mbar_init(xch, F8_EPI_WARPS);
    for (int a = 0; a < F8_SCALE_STAGES; ++a) {
      mbar_init(&sfull[a], 32);
      mbar_init(&sempty[a], F8_EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns, p.kernel_id};
  const int num_tiles = p.num_m_tiles * p.num_n_tiles;
  int issued = 0;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F8_REGS_ISSUE));
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------------- producer (both CTAs)
      const uint64_t hint = l2_policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        int m_blk, n_blk;
        tile_coords(tile, p.num_m_tiles, p.num_n_tiles, p.group_m, m_blk, n_blk);
        const int a_row = m_blk * 256 + (int)rank * 128;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, ctl, 0, kWaitEmpty)) {
            ok = false;
            break;
          }
          uint8_t* a_dst = sA + stage * F8_A_BYTES;
          uint8_t* b_dst = sB + stage * F8_B_BYTES;
          const int k0 = kb * F8_BK;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * F8_STAGE_BYTES);
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          if constexpr (A_MN) tma_load_2d_pair(a_dst, &tmA, bar, a_row, k0, hint);
          else tma_load_2d_pair(a_dst, &tmA, bar, k0, a_row, hint);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // This CTA's 64 rows of half h.
            const int n0 = EPI == F8_EPI_SWIGLU ? (rank ? p.split : 0) + n_blk * 128 + h * 64
                                                : n_blk * 256 + h * 128 + (int)rank * 64;
            if constexpr (B_MN) tma_load_2d_pair(b_dst + h * 8192, &tmB, bar, n0, k0, hint);
            else tma_load_2d_pair(b_dst + h * 8192, &tmB, bar, k0, n0, hint);
          }
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 1 && rank == 0 && elect_one()) {
      // ---------------------------------------------------------------- MMA issuer (pair's leader)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t it = 0;  // 128-deep blocks issued: parity selects the TMEM buffers
      const uint64_t a_desc0 = make_sdesc_sw128(smem_u32(sA), 16, 1024);
      const uint64_t b_desc0 = B_MN ? make_sdesc_sw64(smem_u32(sB), 16, 512) : make_sdesc_sw128(smem_u32(sB), 16, 1024);
      bool ok = true;
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        for (int kb = 0; kb < p.k_blocks && ok; ++kb, ++it) {
          if (!mbar_wait(&full[stage], phase, ctl, 1, kWaitFull)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int buf = (int)(it & 1) * 2 + h;
            if (!mbar_wait(&tempty[buf], ((it >> 1) & 1u) ^ 1u, ctl, 1, kWaitAccEmpty)) {
              ok = false;
              break;
            }
            tc_fence_after();
            // K-major: 32 bytes inside the 128-byte swizzled row; MN-major: 32 k
            // rows of 128 bytes (A) or 64 bytes (B, one 64-row half per CTA).
            umma_f8_stage_pair<A_MN ? 256 : 2, B_MN ? 128 : 2>(
                tmem_base + (uint32_t)(buf * 128), a_desc0 + (uint64_t)(stage * (F8_A_BYTES >> 4)),
                b_desc0 + (uint64_t)(stage * (F8_B_BYTES >> 4) + h * (8192 >> 4)), p.idesc);
            umma_commit_pair_both(&tfull[buf]);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      umma_commit_pair(mapa_shared(smem_u32(mma_done), 0));
      mbar_wait(mma_done, 0, ctl, 1, kWaitDrain);
    } else if (warp == 2) {
      // ---------------------------------------------------------------- scales (both CTAs)
      int st = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        int m_blk, n_blk;
        tile_coords(tile, p.num_m_tiles, p.num_n_tiles, p.group_m, m_blk, n_blk);
        const int row = m_blk * 256 + (int)rank * 128 + lane;
        const float* sb = p.sb;
        bool sbv = true;
        if constexpr (VEC) {
          sb += n_blk * 256 + lane * 4;
        } else {
          // Lane h: the block of half h, or (gate/up) of the gate columns and of the up columns.
          const int nb = EPI == F8_EPI_SWIGLU ? n_blk + lane * (p.split / 128) : n_blk * 2 + lane;
          sbv = lane < 2 && (EPI == F8_EPI_SWIGLU || nb * 128 < p.N);
          sb += sbv ? (size_t)nb * p.sb_n : 0;
        }
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          ok = mbar_wait(&sempty[st], phase ^ 1u, ctl, 6, kWaitEmpty);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          float* dst = sScale + st * F8_SCALE_FLOATS;
          const float* sa = p.sa + (size_t)kb * p.M;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool v = row + 32 * i < p.M;
            cp_async<4>(dst + 32 * i + lane, sa + (v ? row + 32 * i : 0), v);
          }
          if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool v = n_blk * 256 + 128 * i + lane * 4 < p.N;
              cp_async<16>(dst + 128 + 128 * i + lane * 4, v ? sb + (size_t)kb * p.N + 128 * i : p.sb, v);
            }
          } else {
            if (lane < 2) cp_async<4>(dst + 128 + lane, sb + (sbv ? (size_t)kb * p.sb_k : 0), sbv);
          }
          cp_async_arrive(&sfull[st]);
          if (++st == F8_SCALE_STAGES) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---------------------------------------------------------------- drain and epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F8_REGS_DRAIN));
    const int q = warp & 3;           // TMEM lane quarter this warp may access
    const int h = (warp - 4) / 4;     // column half
    F8Store es;
    es.stg = sEpi + (warp - 4) * F8_WARP_STAGING;
    es.lane = lane;
    es.rows = p.M;
    es.slot = 0;
    uint32_t it = 0, tiles_done = 0, sphase = 0;
    int stage = 0, sst = 0;
    bool ok = true;
    for (int tile = first_tile; tile < num_tiles; tile += tile_step, ++tiles_done) {
      int m_blk, n_blk;
      tile_coords(tile, p.num_m_tiles, p.num_n_tiles, p.group_m, m_blk, n_blk);
      const int row0 = m_blk * 256 + (int)rank * 128 + q * 32;
      const int row = row0 + lane;
      const bool rv = row < p.M;
      const int col0 = EPI == F8_EPI_SWIGLU ? n_blk * 128 + h * 64 : n_blk * 256 + h * 128;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
        const float* sc = sScale + sst * F8_SCALE_FLOATS;
        ok = mbar_wait(&sfull[sst], sphase, ctl, 2 + q, kWaitFull);
        const float a_s = sc[q * 32 + lane];
        const float* cs = sc + 128 + (VEC ? h * 128 : 0);
        // Half h is one block of a weight; a gate/up half holds columns of a gate and of an up block.
        const float b_lo = VEC ? 1.f : (EPI == F8_EPI_SWIGLU ? cs[0] : cs[h]);
        const float b_hi = EPI == F8_EPI_SWIGLU ? cs[1] : b_lo;
        const int buf = (int)(it & 1) * 2 + h;
        ok = ok && mbar_wait(&tfull[buf], (it >> 1) & 1u, ctl, 2 + q, kWaitAccFull);
        ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld below needs all 32 lanes converged
        if (!ok) break;
        tc_fence_after();
        // Half 1 is the stage's last product: with it done, both CTAs' operand
        // tiles have been read and each CTA frees its own stage.
        if (warp == 8 && lane == 0) mbar_arrive(&empty[stage]);
        const uint32_t taddr = tmem_base + (uint32_t)(buf * 128) + ((uint32_t)(q * 32) << 16);
        f8_promote<VEC>(taddr, a_s * b_lo, a_s * b_hi, cs, acc, [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader(&tempty[buf]);
        });
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[sst]);
        if (++stage == S) stage = 0;
        if (++sst == F8_SCALE_STAGES) {
          sst = 0;
          sphase ^= 1u;
        }
      }
      if (!ok) break;
      es.row0 = row0;
      if constexpr (EPI == F8_EPI_BF16) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (col0 + c * 32 >= p.N) break;
          uint4 o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = unpack_f32x2(acc[c * 16 + j * 4 + i]);
              f[2 * i] = v.x;
              f[2 * i + 1] = v.y;
            }
            o[j] = pack8(f);
          }
          es.put(o, &tmO1, col0 + c * 32, false);
        }
      } else if constexpr (EPI == F8_EPI_F32) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (col0 + c * 16 >= p.N) break;
          uint4 o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = unpack_f32x2(acc[c * 8 + j * 2]), w = unpack_f32x2(acc[c * 8 + j * 2 + 1]);
            o[j] = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(w.x), __float_as_uint(w.y));
          }
          es.put(o, &tmO1, col0 + c * 16, p.add != 0);
        }
      } else {
        // Columns 0-63 are a, 64-127 the same columns of b.  One scale per row
        // and 128 columns: the two halves exchange their maxima.
        float my = 0.f, ma = 0.f, mb = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 a = unpack_f32x2(acc[i]), b = unpack_f32x2(acc[32 + i]);
          my = fmaxf(my, fmaxf(fabsf(a.x * sigmoid_f(a.x) * b.x), fabsf(a.y * sigmoid_f(a.y) * b.y)));
          ma = fmaxf(ma, fmaxf(fabsf(a.x), fabsf(a.y)));
          mb = fmaxf(mb, fmaxf(fabsf(b.x), fabsf(b.y)));
        }
        float* x = sXch + (tiles_done & 1) * 768 + q * 32 + lane;
        x[h * 384] = my;
        x[h * 384 + 128] = ma;
        x[h * 384 + 256] = mb;
        __syncwarp();
        if (lane == 0) mbar_arrive(xch);
        ok = mbar_wait(xch, tiles_done & 1u, ctl, 2 + q, kWaitAccFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        my = fmaxf(my, x[(h ^ 1) * 384]);
        ma = fmaxf(ma, x[(h ^ 1) * 384 + 128]);
        mb = fmaxf(mb, x[(h ^ 1) * 384 + 256]);
        if (rv && h == 0) {
          p.sy[(size_t)n_blk * p.M + row] = fp8_scale<FP8_E4M3>(my);
          if (p.save_ab) {
            p.sab[(size_t)n_blk * p.M + row] = fp8_scale<FP8_E4M3>(ma);
            p.sab[(size_t)(n_blk + p.split / 128) * p.M + row] = fp8_scale<FP8_E4M3>(mb);
          }
        }
        const float fy = fp8_factor<FP8_E4M3>(my);
        uint4 o[4];
        auto words = [&](auto value) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 u = value(j * 8 + i * 2), v = value(j * 8 + i * 2 + 1);
              w[i] = fp8_pack4<FP8_E4M3>(u.x, u.y, v.x, v.y);
            }
            o[j] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        };
        words([&](int i) {
          const float2 a = unpack_f32x2(acc[i]), b = unpack_f32x2(acc[32 + i]);
          return make_float2(a.x * sigmoid_f(a.x) * b.x * fy, a.y * sigmoid_f(a.y) * b.y * fy);
        });
        es.put(o, &tmO1, col0, false);
        if (p.save_ab) {
          const float fa = fp8_factor<FP8_E4M3>(ma), fb = fp8_factor<FP8_E4M3>(mb);
          words([&](int i) {
            const float2 a = unpack_f32x2(acc[i]);
            return make_float2(a.x * fa, a.y * fa);
          });
          es.put(o, &tmO2, col0, false);
          words([&](int i) {
            const float2 b = unpack_f32x2(acc[32 + i]);
            return make_float2(b.x * fb, b.y * fb);
          });
          es.put(o, &tmO2, p.split + col0, false);
        }
      }
    }
    es.finish();
  }

  tc_fence_before();
  cluster_sync();
  if (*abort_flag) {
    // A role gave up: let the last (up to STAGES) copies land before shared
    // memory is released.  Every wait here is bounded too.
    if (warp == 0 && lane == 0 && rank == 0) {
      const int first = issued > S ? issued - S : 0;
      for (int i = first; i < issued; ++i) {
        const uint32_t par = (uint32_t)((i / S) & 1);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&full[i % S], par) && global_timer_ns() - t0 < ctl.limit_ns) {
        }
      }
    }
    __syncthreads();
  }
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace coda
