// 8-bit GEMM with a scale for each block of 128 (sm_100a, tcgen05 kind::f8f6f4).
//
//   C[m, n] = sum_kb SA[kb, m] SB(kb, n) sum_{k in kb} A[m, k] B[n, k]
//
// The inner sum over 128 values runs in the tensor cores into fp32 TMEM; the
// outer sum cannot, because its scales change with kb, so every 128-deep
// partial tile is drained, scaled and added to fp32 registers.  The drain is
// what bounds the design: per 128 of k an SM's tensor core needs 512 clocks
// for 128 x 256 outputs, and in those the warps must read 128 KB of TMEM and
// issue 32768 fused multiply-adds (256 clocks each at full rate; with a scale
// per column as many products again).
//
// Tile: a CTA pair (cta_group::2) computes 256 x 256, each CTA holding 128 rows
// of A and half of B.  The 256 columns are issued as two halves of 128, each
// with its own two TMEM buffers (4 x 128 columns) and its own four warps, so a
// half's drain has the time of three half-products (768 clocks) to hide the
// commit, the TMEM reads and the arrival that crosses to the pair's leader.
// One 256-column product with two buffers was slower (7B down projection 315
// us against the 307 of the time).  Half h is columns [128 h, 128 h + 128): 64 rows of B from
// each CTA (the operand's pair order), which makes it one 128-wide scale block
// of a weight, and in the gate/up product 64 gate columns beside the same 64 up
// columns.
//
// Roles (384 threads, one CTA per SM): warp 0 TMA producer; warp 1 TMEM owner;
// warps 1 and 3 MMA issuers of the two halves (pair's leader); warp 2 copies the
// scales of 8 blocks ahead; warps 4-7 drain half 0, warps 8-11 half 1, 128 fp32
// sums in registers per thread: one output row and 128 columns, or (a scale per
// column) four rows and 32 columns.  The first warpgroup hands registers to the
// other two.  Waits are bounded; a role that gives up records it and the CTA
// drains and exits.
//
// Measured in steady use: M 8192, N 4096, K 11008 in 357-370 us (2000-2070 TFLOP/s),
// gate/up SwiGLU 8192 x 4096 x 11008 in 736-749 us (1970-2010), weight gradient 4096 x
// 4096 x 8191 in 189-192 us (1430-1450; 3.5 waves of tiles in 4).  The 1 kW power cap then holds the clock
// near 1400 MHz; in bursts from a cool GPU they take 287-310, 612-653 and 159-167
// us.  At 1965 MHz a block of 128 takes about 920 clocks, of which the tensor core
// works 512 (its pipe is busy 66-74 % of the time, 44 % with a scale per column):
// the rest is the round trip of a buffer (drain, arrival, product, commit).
#pragma once

#include "coda_fp8.cuh"
#include "coda_gemm.cuh"

namespace coda {

constexpr int F8_BK = 128;          // reduction depth of a stage and of a scale block
constexpr int F8_UMMA_K = 32;
constexpr int F8_THREADS = 384;
constexpr int F8_REGS_ISSUE = 40, F8_REGS_DRAIN = 232;
static_assert(128 * F8_REGS_ISSUE + 256 * F8_REGS_DRAIN <= 384 * 168, "registers of the launch");
constexpr int F8_STAGES = 6;
constexpr int F8_A_BYTES = 128 * F8_BK;
constexpr int F8_B_BYTES = 128 * F8_BK;
constexpr int F8_STAGE_BYTES = F8_A_BYTES + F8_B_BYTES;
constexpr int F8_EPI_WARPS = 8;
constexpr int F8_GROUP = 8;                     // 128-deep blocks whose scales are staged together
constexpr int F8_SCALE_BYTES = 2 * F8_GROUP * (128 + 256) * 4;  // two groups of row and column scales
constexpr int F8_SMEM_BYTES = F8_STAGES * F8_STAGE_BYTES + F8_SCALE_BYTES + 1024 + 256;
// The gate/up product has no column scales; its halves exchange row maxima (two
// buffers) in their place.
constexpr int F8_XCH_FLOATS = 2 * 2 * 3 * 128;
static_assert(2 * F8_GROUP * (128 + 2) + F8_XCH_FLOATS <= F8_SCALE_BYTES / 4, "scales and maxima share the room");
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
  float* sy;        // [F / 128, M]
  float* sab;       // [2 F / 128, M]
  void* out;        // C, or Y
  void* out2;       // AB, or null
  int wide;         // out (and out2) 32-byte aligned
  uint32_t idesc;
  uint32_t* status;
  unsigned long long wait_limit_ns;
  uint32_t kernel_id;
  uint32_t silent;  // self-test: a role that does nothing (f8_silent), 0 for none
};

// True in the CTA and role that a self-test keeps silent, so that the waits on it run out.
__device__ __forceinline__ bool f8_silent(uint32_t silent, uint32_t role) { return silent == (blockIdx.x << 2 | role); }

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

// 32 or 16 accumulator columns of this thread's TMEM lane as pairs of floats.
__device__ __forceinline__ void tmem_ld_pairs(uint32_t taddr, F2 (&v)[16]) {
  asm volatile(
      "{\n\t.reg .b32 t<32>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {t0,t1,t2,t3,t4,t5,t6,t7,t8,t9,t10,t11,t12,t13,t14,t15,"
      "t16,t17,t18,t19,t20,t21,t22,t23,t24,t25,t26,t27,t28,t29,t30,t31}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n\t"
      "mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n\t"
      "mov.b64 %8, {t16, t17}; mov.b64 %9, {t18, t19}; mov.b64 %10, {t20, t21}; mov.b64 %11, {t22, t23};\n\t"
      "mov.b64 %12, {t24, t25}; mov.b64 %13, {t26, t27}; mov.b64 %14, {t28, t29}; mov.b64 %15, {t30, t31};\n\t}\n"
      : "=l"(v[0].v), "=l"(v[1].v), "=l"(v[2].v), "=l"(v[3].v), "=l"(v[4].v), "=l"(v[5].v), "=l"(v[6].v), "=l"(v[7].v),
        "=l"(v[8].v), "=l"(v[9].v), "=l"(v[10].v), "=l"(v[11].v), "=l"(v[12].v), "=l"(v[13].v), "=l"(v[14].v), "=l"(v[15].v)
      : "r"(taddr)
      : "memory");
}
// 16 TMEM lanes x 32 columns: in groups of 8 columns, this thread's words are two
// neighbouring columns (2 (lane % 4)) of lane / 4 and the same of lane / 4 + 8.
// The words are there after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
        "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
      :
      : "memory");
}

// Asynchronous 4- or 16-byte copy to shared memory; zeros, and no read of src, when !valid.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
               "r"(valid ? BYTES : 0)
               : "memory");
}
// Arrive on `bar` (whose count includes this thread) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Control words of the drain's waits, in shared memory: the abort flag (nonzero:
// some role gave up; the detail word's role and reason, or 1 when mbar_wait has
// recorded it) and the limit; and, at the end, the stages this CTA's producer issued.
struct DrainCtl {
  uint32_t abort;
  uint32_t issued;
  uint64_t limit_ns;
};

// Bounded wait of a whole warp on a barrier that is about to complete.  The
// drain is latency-bound, so success costs a poll and a branch: there is no
// result.  A wait that runs out, or sees that another role has given up, sets or
// leaves the abort flag and returns; the caller looks at the flag every few
// blocks and what its CTA computed since then is not stored.  (The other CTA of
// the pair comes to the same end: no MMA is issued after a wait that gave up.)
__device__ __forceinline__ void mbar_wait_drain(uint32_t bar, uint32_t parity, uint32_t ctl, uint32_t detail) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u32 f;\n\t.reg .u64 t0, t1, lim;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t@p bra DONE;\n\t"
      "mov.u64 t0, %%globaltimer;\n\tld.shared.u64 lim, [%2 + 8];\n"
      "POLL:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t@p bra DONE;\n\t"
      "ld.volatile.shared.u32 f, [%2];\n\tsetp.ne.u32 p, f, 0;\n\t@p bra DONE;\n\t"
      "mov.u64 t1, %%globaltimer;\n\tsub.u64 t1, t1, t0;\n\tsetp.lt.u64 p, t1, lim;\n\t@p bra POLL;\n\t"
      "st.volatile.shared.u32 [%2], %3;\n"
      "DONE:\n\t}\n" ::"r"(bar),
      "r"(parity), "r"(ctl), "r"(detail)
      : "memory");
}
// The same for the thread that issues the MMAs.  It may not go on after a wait that
// gave up (false): the operands may not have landed, the buffer may not have been
// drained, and its commit would tell both CTAs that a product is complete.
__device__ __forceinline__ bool mbar_wait_issue(uint32_t bar, uint32_t parity, uint32_t ctl, uint32_t detail) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u32 f;\n\t.reg .u64 t0, t1, lim;\n\tmov.u32 %0, 1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
      "mov.u64 t0, %%globaltimer;\n\tld.shared.u64 lim, [%3 + 8];\n"
      "POLL:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
      "ld.volatile.shared.u32 f, [%3];\n\tsetp.ne.u32 p, f, 0;\n\t@p bra GAVE_UP;\n\t"
      "mov.u64 t1, %%globaltimer;\n\tsub.u64 t1, t1, t0;\n\tsetp.lt.u64 p, t1, lim;\n\t@p bra POLL;\n\t"
      "st.volatile.shared.u32 [%3], %4;\n"
      "GAVE_UP:\n\tmov.u32 %0, 0;\n"
      "DONE:\n\t}\n"
      : "=&r"(ok)
      : "r"(bar), "r"(parity), "r"(ctl), "r"(detail)
      : "memory");
  return ok != 0;
}
// Arrive where `pred` is set, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, uint32_t pred) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
               "r"(pred)
               : "memory");
}

// Hand a drained TMEM buffer to the pair's leader.  What is handed over are TMEM
// loads that tcgen05.wait::ld has completed, no ordinary memory, so the arrival
// needs no cluster-scope release: that one waits for a memory barrier, once per
// 128 of k.
__device__ __forceinline__ void mbar_arrive_leader_if(uint32_t leader_bar, uint32_t pred) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(
          leader_bar),
      "r"(pred)
      : "memory");
}

// A shared-memory read that stays where it is written.
__device__ __forceinline__ float lds_here(const float* p) {
  float v;
  asm volatile("ld.volatile.shared.f32 %0, [%1];" : "=f"(v) : "r"(smem_u32(p)) : "memory");
  return v;
}

__device__ __forceinline__ void lds_here(const float* p, F2& a) {
  asm volatile("ld.volatile.shared.u64 %0, [%1];" : "=l"(a.v) : "r"(smem_u32(p)) : "memory");
}

// Scales of one 128-deep block for a drain thread: its row's and those of its
// columns 0-63 and 64-127.
struct F8Scales {
  float a, b_lo, b_hi;
};

// acc += a * TMEM columns times b_lo (columns 0-63) or b_hi (64-127), two columns
// to an instruction.  release() hands the buffer back as soon as the last columns
// have arrived, and reads the next block's scales; the row scale is read again
// behind it, since the multiply-adds that depend on it are otherwise scheduled
// before the arrival.
template <typename Release>
__device__ __forceinline__ void f8_promote(uint32_t taddr, const F8Scales& sc, const float* a, F2 (&acc)[64],
                                           Release release) {
  const float lo = sc.a * sc.b_lo;
  float hi = sc.a * sc.b_hi;
#pragma unroll
  for (int c = 0; c < 64; c += 16) {
    F2 v[16];
    tmem_ld_pairs(taddr + 2 * c, v);
    if (c == 48) {
      const float b_hi = sc.b_hi;
      release();
      hi = lds_here(a) * b_hi;
    }
    const F2 s = c < 32 ? f2(lo, lo) : f2(hi, hi);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[c + i] = fma2(v[i], s, acc[c + i]);
  }
}

// The same where every column has a scale of its own, cs[128] in shared memory.
// A thread that holds one row would read all 128 of them: 512 bytes a thread, and
// with 256 threads the reads alone take 1024 clocks per 128 of k.  So a thread
// holds 4 rows (lane / 4 and 8, 16, 24 further, scales a[8 i]) and 32 columns
// (2 (lane % 4) and the next in each group of 8), and reads a quarter of that
// (4096 x 4096 x 8192: 193 -> 168 us).  The next columns' TMEM load and scales
// are in flight while these are added.
// acc[(half * 16 + group) * 2 + i]: rows 16 half + 8 i.
template <typename Release>
__device__ __forceinline__ void f8_promote_columns(uint32_t taddr, const float (&sc)[4], const float* a,
                                                   const float* cs, F2 (&acc)[64], Release release) {
  uint32_t t[2][16];
  float r[4] = {sc[0], sc[1], sc[2], sc[3]};
  F2 f[4], ahead[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) lds_here(cs + g * 8, ahead[g]);
  tmem_ld_16x32(taddr, t[0]);
#pragma unroll
  for (int c = 0; c < 8; ++c) {  // 32 columns c / 2, 16 rows c % 2
    const int h = c % 2;
    if (h == 0) {
#pragma unroll
      for (int g = 0; g < 4; ++g) f[g] = ahead[g];
    }
    tmem_ld_wait(t[h]);
    if (c < 7) tmem_ld_16x32(taddr + (uint32_t)((c + 1) / 2 * 32) + ((uint32_t)((c + 1) % 2 * 16) << 16), t[h ^ 1]);
    if (h == 0 && c < 6) {
#pragma unroll
      for (int g = 0; g < 4; ++g) lds_here(cs + (c + 2) * 16 + g * 8, ahead[g]);
    }
    if (c == 7) {
      release();
      r[2] = lds_here(a + 16);
      r[3] = lds_here(a + 24);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        F2& s = acc[(h * 16 + c / 2 * 4 + g) * 2 + i];
        const F2 x = f2(__uint_as_float(t[h][g * 4 + 2 * i]), __uint_as_float(t[h][g * 4 + 2 * i + 1])) * f[g];
        s = fma2(x, f2(r[h * 2 + i], r[h * 2 + i]), s);
      }
  }
}

// 32 bytes of a row: whole sectors, so a row per thread needs no staging.
__device__ __forceinline__ void f8_store32(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    stg_v4(dst, make_uint4(w[0], w[1], w[2], w[3]));
    stg_v4(static_cast<uint8_t*>(dst) + 16, make_uint4(w[4], w[5], w[6], w[7]));
  }
}
__device__ __forceinline__ void f8_add8(float* dst, F2 v) {
  float lo, hi;
  split(v, lo, hi);
  asm volatile("red.global.add.v2.f32 [%0], {%1,%2};" ::"l"(dst), "f"(lo), "f"(hi) : "memory");
}
__device__ __forceinline__ void f8_add16(float* dst, const float* f) {
  asm volatile("red.global.add.v4.f32 [%0], {%1,%2,%3,%4};" ::"l"(dst), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3])
               : "memory");
}
// 64 floats of a row, times factor, as 64 8-bit values.
template <typename Value>
__device__ __forceinline__ void f8_store_row64(uint8_t* dst, bool wide, Value value) {
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = fp8_pack4<FP8_E4M3>(value(c + 4 * i), value(c + 4 * i + 1), value(c + 4 * i + 2), value(c + 4 * i + 3));
    f8_store32(dst + c, w, wide);
  }
}

// Record a wait of a drain warp or an MMA issuer that ran out (mbar_wait records its own and sets 1).
__device__ __forceinline__ void f8_record(uint32_t flag, uint32_t* status, uint32_t kernel_id) {
  if (flag <= 1 || status == nullptr) return;
  atomicCAS(status, 0u, 7u /* CODA_ERR_DEVICE_TIMEOUT */);
  atomicCAS(status + 1, 0u, (kernel_id << 16) | flag);
}
// Where the CTAs of a cluster add each other's partial tiles: if a role of this CTA
// gave up, its partial tile is not one, and every CTA of the cluster has to know
// before the barrier behind which it reads it.  By one thread, when all the CTA's
// roles have come to their end; costs a look at the flag when none gave up.
__device__ __forceinline__ void f8_tell_cluster(uint32_t* abort_flag, int ctas, uint32_t* status, uint32_t kernel_id) {
  const uint32_t flag = *const_cast<volatile uint32_t*>(abort_flag);
  if (flag == 0) return;
  f8_record(flag, status, kernel_id);
  for (int r = 0; r < ctas; ++r)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(abort_flag), (uint32_t)r)), "r"(1u) : "memory");
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Arrive on the barrier at this offset in the CTAs of `mask` when this thread's pair MMAs so far are complete.
__device__ __forceinline__ void umma_commit_pair_mask(const uint64_t* bar, uint32_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"((uint16_t)mask)
               : "memory");
}

// With SPLIT the reduction of a tile is shared by the pairs of a cluster (2 to 4;
// few tiles, long reductions): each pair takes a range of the blocks, leaves its
// fp32 partial tile in its own shared memory, where the operands were, and then
// finishes a share of the rows, adding the partials in the pairs' order and
// reading the others' through distributed shared memory, whole rows at a time
// (sent to the finisher from the drain, a row per thread: 45 us for 36 at 1001 x
// 2048 x 16384).  One tile per cluster.
constexpr int F8_PART_PITCH = (256 + 4) * 4;  // bytes per row of a partial tile: rows 16 bytes apart in the banks
static_assert(128 * F8_PART_PITCH <= F8_STAGES * F8_STAGE_BYTES, "the partial tile takes the ring's place");

// The second half of a SPLIT tile, by the drain warps: this pair's share of the
// rows, 64 threads to a row.
template <int EPI>
__device__ __forceinline__ void f8_finish_share(const Gemm8Params& p, const uint8_t* smem) {
  // Read again rather than kept: the drain has no registers to spare.
  const int crank = (int)cluster_ctarank(), part = crank / 2, parts = (int)cluster_nctarank() / 2;
  int m_blk, n_blk;
  tile_coords((int)cluster_id_x(), p.num_m_tiles, p.num_n_tiles, p.group_m, m_blk, n_blk);
  const int t = (int)threadIdx.x - 128;
  const int col = n_blk * 256 + t % 64 * 4, m0 = m_blk * 256 + crank % 2 * 128;
  const int end = min((part + 1) * 128 / parts, p.M - m0);
  const uint8_t* own = smem + t % 64 * 16;
  uint32_t from[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) from[j] = mapa_shared(smem_u32(own), (uint32_t)(min(j, parts - 1) * 2 + crank % 2));
  if (col < p.N) {
#pragma unroll 2
    for (int r = part * 128 / parts + t / 64; r < end; r += 4) {
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j == part) v[j] = *reinterpret_cast<const float4*>(own + r * F8_PART_PITCH);
        else if (j < parts) v[j] = ld_cluster_f32x4(from[j] + r * F8_PART_PITCH);
      }
      float f[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int j = 1; j < 4; ++j) {
        f[0] += v[j].x;
        f[1] += v[j].y;
        f[2] += v[j].z;
        f[3] += v[j].w;
      }
      const size_t o = (size_t)(m0 + r) * p.N + col;
      if constexpr (EPI == F8_EPI_BF16) {
        stg_v2(static_cast<__nv_bfloat16*>(p.out) + o, make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])));
      } else if (p.add) {
        f8_add16(static_cast<float*>(p.out) + o, f);
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
  }
}

template <int EPI, bool A_MN, bool B_MN, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(F8_THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const Gemm8Params p) {
  constexpr int S = F8_STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + S * F8_A_BYTES;
  float* sScale = reinterpret_cast<float*>(sB + S * F8_B_BYTES);
  constexpr int GROUP_FLOATS = F8_GROUP * (128 + (VEC ? 256 : 2));
  float* sXch = sScale + 2 * GROUP_FLOATS;
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sScale) + F8_SCALE_BYTES);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;   // [2 * parity + half]
  uint64_t* tempty = tfull + 4;
  uint64_t* xch = tempty + 4;
  uint64_t* sfull = xch + 1;
  uint64_t* sempty = sfull + 2;
  uint64_t* mma_done = sempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  DrainCtl* drain_ctl = reinterpret_cast<DrainCtl*>(
      (reinterpret_cast<uintptr_t>(tmem_slot + 1) + 15) & ~static_cast<uintptr_t>(15));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&drain_ctl->abort);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0);  // known uniform
  const int lane = threadIdx.x % 32;
  static_assert(!SPLIT || (EPI != F8_EPI_SWIGLU && !VEC), "split products");
  const uint32_t rank = SPLIT ? cluster_ctarank() & 1 : cluster_ctarank();  // 0 = the pair's leader
  const uint32_t leader = SPLIT ? cluster_ctarank() & ~1u : 0u;             // its rank in the cluster
  // This pair's 128-deep blocks.
  int kb0 = 0, num_kb = p.k_blocks;
  if constexpr (SPLIT) {
    const int parts = (int)cluster_nctarank() / 2, part = (int)leader / 2;
    kb0 = (int)((long long)part * p.k_blocks / parts);
    num_kb = (int)((long long)(part + 1) * p.k_blocks / parts) - kb0;
  }
  const int first_tile = (int)cluster_id_x();
  const int tile_step = (int)num_clusters_x();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);  // the two MMA issuers
    }
    for (int a = 0; a < 4; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 8);  // four warps of each CTA
    }
    mbar_init(xch, F8_EPI_WARPS);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sfull[a], 32);
      mbar_init(&sempty[a], F8_EPI_WARPS);
    }
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    drain_ctl->limit_ns = p.wait_limit_ns;
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
      bool ok = !f8_silent(p.silent, CODA_FP8_ROLE_LOADS);
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        int m_blk, n_blk;
        tile_coords(tile, p.num_m_tiles, p.num_n_tiles, p.group_m, m_blk, n_blk);
        const int a_row = m_blk * 256 + (int)rank * 128;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, ctl, 0, kWaitEmpty)) {
            ok = false;
            break;
          }
          uint8_t* a_dst = sA + stage * F8_A_BYTES;
          uint8_t* b_dst = sB + stage * F8_B_BYTES;
          const int k0 = (kb0 + kb) * F8_BK;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * F8_STAGE_BYTES);
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), leader);
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
    } else if ((warp == 1 || warp == 3) && rank == 0 && elect_one()) {
      // ---------------------------------------------------------------- MMA issuers (pair's leader)
      // One thread per half: per 128 of k a thread has two waits, four MMAs and
      // two commits to get through, each some tens of clocks on an SM whose
      // issue slots the drain fills; one thread for both halves needed 810
      // clocks for what the tensor core does in 512.
      const uint32_t half = (uint32_t)warp / 2;
      const uint32_t wctl = smem_u32(drain_ctl);
      uint32_t full_s = smem_u32(full), phase = 0, stage = 0;
      uint32_t it = 0;  // 128-deep blocks issued: parity selects the TMEM buffer
      const uint64_t a_desc0 = make_sdesc_sw128(smem_u32(sA), 16, 1024);
      const uint64_t b_desc0 = (B_MN ? make_sdesc_sw64(smem_u32(sB), 16, 512) : make_sdesc_sw128(smem_u32(sB), 16, 1024)) +
                               half * (8192 >> 4);
      bool ok = !f8_silent(p.silent, CODA_FP8_ROLE_MMA);
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
#pragma unroll 1
        for (int kb = num_kb; kb > 0; --kb, ++it) {
          const uint32_t buf = (it & 1) * 2 + half;
          ok = mbar_wait_issue(full_s + stage * 8, phase, wctl, 1 << 8 | kWaitFull) &&
               mbar_wait_issue(smem_u32(tempty) + buf * 8, ((it >> 1) & 1u) ^ 1u, wctl, 1 << 8 | kWaitAccEmpty);
          if (!ok) break;
          tc_fence_after();
          // K-major: 32 bytes inside the 128-byte swizzled row; MN-major: 32 k
          // rows of 128 bytes (A) or 64 bytes (B, one 64-row half per CTA).
          umma_f8_stage_pair<A_MN ? 256 : 2, B_MN ? 128 : 2>(
              tmem_base + buf * 128, a_desc0 + (uint64_t)(stage * (F8_A_BYTES >> 4)),
              b_desc0 + (uint64_t)(stage * (F8_B_BYTES >> 4)), p.idesc);
          if constexpr (SPLIT) umma_commit_pair_mask(&tfull[buf], 3u << leader);
          else umma_commit_pair_both(&tfull[buf]);
          if constexpr (SPLIT) umma_commit_pair_mask(&empty[stage], 3u << leader);
          else umma_commit_pair_both(&empty[stage]);  // with the other half's: both CTAs' operand tiles have been read
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      umma_commit_pair(mapa_shared(smem_u32(mma_done), leader));
      mbar_wait_own(mma_done, 0, ctl, 1);
    } else if (warp == 2) {
      // ---------------------------------------------------------------- scales (both CTAs)
      int st = 0;
      uint32_t phase = 0;
      bool ok = !f8_silent(p.silent, CODA_FP8_ROLE_SCALES);
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        int m_blk, n_blk;
        tile_coords(tile, p.num_m_tiles, p.num_n_tiles, p.group_m, m_blk, n_blk);
        // This lane's rows (32 apart) and columns, and which of them exist.
        const int row = m_blk * 256 + (int)rank * 128 + lane;
        const float* sa = p.sa + (size_t)kb0 * p.M + row;
        const float* sb = p.sb + (size_t)kb0 * p.sb_k;
        int b_ok = 0;
        if constexpr (VEC) {
          sb += n_blk * 256 + lane * 4;
        } else {
          // Lane h: the block of half h, or (gate/up) of the gate columns and of the up columns.
          const int nb = EPI == F8_EPI_SWIGLU ? n_blk + lane * (p.split / 128) : n_blk * 2 + lane;
          b_ok = EPI == F8_EPI_SWIGLU || nb * 128 < p.N;
          sb += (size_t)nb * p.sb_n;
        }
        for (int left = num_kb; left > 0; left -= F8_GROUP) {
          ok = __all_sync(0xffffffffu, mbar_wait(&sempty[st], phase ^ 1u, ctl, 6, kWaitEmpty));
          if (!ok) break;
          uint32_t dst = smem_u32(sScale + st * GROUP_FLOATS) + lane * 4;
          uint32_t dst_b = smem_u32(sScale + st * GROUP_FLOATS + F8_GROUP * 128) + lane * (VEC ? 16 : 4);
#pragma unroll 2
          for (int n = min(left, F8_GROUP); n > 0; --n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async<4>(dst + 128 * i, sa + 32 * i, row + 32 * i < p.M);
            sa += p.M;
            dst += 512;
            if constexpr (VEC) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                cp_async<16>(dst_b + 512 * i, sb + 128 * i, n_blk * 256 + lane * 4 + 128 * i < p.N);
              sb += p.N;
              dst_b += 1024;
            } else {
              if (lane < 2) cp_async<4>(dst_b, sb, b_ok);
              sb += p.sb_k;
              dst_b += 8;
            }
          }
          cp_async_arrive(&sfull[st]);
          st ^= 1;
          phase ^= st == 0;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_sync();
      // Every role of the cluster has come to its end.  By a warp that is known uniform:
      // behind threadIdx.x == 0 the whole kernel took longer (1001 x 2048 x 16384 45 us for 36).
      if (warp == 2 && lane == 0) f8_tell_cluster(&drain_ctl->abort, (int)cluster_nctarank(), p.status, p.kernel_id);
      cluster_sync();
    }
  } else {
    // ---------------------------------------------------------------- drain and epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F8_REGS_DRAIN));
    const int q = warp & 3;           // TMEM lane quarter this warp may access
    const int h = (warp - 4) / 4;     // column half
    const uint32_t one = lane == 0;  // this warp's arrivals
    const uint32_t wctl = smem_u32(drain_ctl);
    // Buffers of parity 0; parity 1 is 16 bytes and 256 columns on (bits that are 0 here).
    uint32_t tfull_h = smem_u32(&tfull[h]);
    uint32_t tempty_h = mapa_shared(smem_u32(&tempty[h]), leader);
    uint32_t taddr_h = tmem_base + (uint32_t)(h * 128) + ((uint32_t)(q * 32) << 16);
    uint32_t it = 0, groups = 0, tiles_done = 0;
    bool given = false;  // SPLIT: the partial tile is in shared memory
    for (int tile = first_tile; tile < num_tiles; tile += tile_step, ++tiles_done) {
      int m_blk, n_blk;
      tile_coords(tile, p.num_m_tiles, p.num_n_tiles, p.group_m, m_blk, n_blk);
      const int row0 = m_blk * 256 + (int)rank * 128 + q * 32;
      const int row = row0 + lane;
      const bool rv = row < p.M;
      const int col0 = EPI == F8_EPI_SWIGLU ? n_blk * 128 + h * 64 : n_blk * 256 + h * 128;
      F2 sums[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sums[i] = F2{0};
#pragma unroll 1
      for (int left = num_kb; left > 0; left -= F8_GROUP, ++groups) {
        mbar_wait_drain(smem_u32(&sfull[groups & 1]), (groups >> 1) & 1u, wctl, (2 + q) << 8 | kWaitFull);
        // A vote: the lanes come out of the wait one by one while another warp may
        // be setting the flag, and what follows needs the whole warp.  Behind it the
        // compiler knows the warp converged: the whole kernel takes 4-7 % less time
        // than with a look at the flag by each lane (gate/up 626 us for 667).
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        const float* sc = sScale + (groups & 1) * GROUP_FLOATS;
        const float* cs = sc + F8_GROUP * 128 + (VEC ? h * 128 + lane % 4 * 2 : EPI == F8_EPI_SWIGLU ? 0 : h);
        sc += q * 32 + (VEC ? lane / 4 : lane);
        // Half h is one block of a weight; a gate/up half holds columns of a gate and of an up block.
        F8Scales cur, next;
        float rows[4], next_rows[4];
        auto scales = [&](int ahead, F8Scales& f, float (&r)[4]) {
          if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = lds_here(sc + ahead * 128 + 8 * i);
          } else {
            f.a = lds_here(sc + ahead * 128);
            f.b_lo = lds_here(cs + ahead * 2);
            f.b_hi = EPI == F8_EPI_SWIGLU ? lds_here(cs + ahead * 2 + 1) : f.b_lo;
          }
        };
        scales(0, cur, rows);
#pragma unroll 1
        for (int n = min(left, F8_GROUP); n > 0; --n, ++it) {
          mbar_wait_drain(tfull_h, (it >> 1) & 1u, wctl, (2 + q) << 8 | kWaitAccFull);
          tc_fence_after();
          auto release = [&] {
            tc_fence_before();
            __syncwarp();
            mbar_arrive_leader_if(tempty_h, one);
            scales(1, next, next_rows);  // behind the group's last block: not used
          };
          if constexpr (VEC) {
            f8_promote_columns(taddr_h, rows, sc, cs, sums, release);
#pragma unroll
            for (int i = 0; i < 4; ++i) rows[i] = next_rows[i];
          } else {
            f8_promote(taddr_h, cur, sc, sums, release);
            cur = next;
          }
          tfull_h ^= 16;
          tempty_h ^= 16;
          taddr_h ^= 256;
          sc += 128;
          cs += VEC ? 256 : 2;
        }
        __syncwarp();
        mbar_arrive_if(smem_u32(&sempty[groups & 1]), one);
      }
      if (__any_sync(0xffffffffu, *abort_flag)) break;  // some block above may not have been complete
      if constexpr (SPLIT) {
        cluster_sync();  // both halves' MMAs have read the operands
        given = true;
        uint8_t* dst = smem + (q * 32 + lane) * F8_PART_PITCH + h * 512;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float4 v;
          split(sums[i], v.x, v.y);
          split(sums[i + 1], v.z, v.w);
          *reinterpret_cast<float4*>(dst + 8 * i) = v;
        }
      } else if constexpr (VEC) {
        // Four lanes hold 8 neighbouring columns of a row.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = row0 + lane / 4 + 8 * i, c0 = col0 + lane % 4 * 2;
          if (m >= p.M) break;
          const size_t o = (size_t)m * p.N + c0;
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            if (col0 + 8 * g >= p.N) break;
            const F2 v = sums[(i / 2 * 16 + g) * 2 + i % 2];
            float lo, hi;
            split(v, lo, hi);
            if constexpr (EPI == F8_EPI_BF16) {
              stg_u32(static_cast<__nv_bfloat16*>(p.out) + o + 8 * g, pack_bf16x2(lo, hi));
            } else if (p.add) {
              f8_add8(static_cast<float*>(p.out) + o + 8 * g, v);
            } else {
              stg_v2(static_cast<float*>(p.out) + o + 8 * g, make_uint2(__float_as_uint(lo), __float_as_uint(hi)));
            }
          }
        }
      } else {
        float acc[128];
#pragma unroll
        for (int i = 0; i < 64; ++i) split(sums[i], acc[2 * i], acc[2 * i + 1]);
        if constexpr (EPI == F8_EPI_BF16) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (size_t)row * p.N + col0;
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            if (!rv || col0 + c >= p.N) break;
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(acc[c + 2 * i], acc[c + 2 * i + 1]);
            f8_store32(o + c, w, p.wide);
          }
        } else if constexpr (EPI == F8_EPI_F32) {
          float* o = static_cast<float*>(p.out) + (size_t)row * p.N + col0;
          if (p.add) {
#pragma unroll
            for (int c = 0; c < 128; c += 4) {
              if (!rv || col0 + c >= p.N) break;
              f8_add16(o + c, acc + c);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 128; c += 8) {
              if (!rv || col0 + c >= p.N) break;
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(acc[c + i]);
              f8_store32(o + c, w, p.wide);
            }
          }
        } else {
          // Columns 0-63 are a, 64-127 the same columns of b.  One scale per row
          // and 128 columns: the two halves exchange their maxima.
          float my = 0.f, ma = 0.f, mb = 0.f;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            my = fmaxf(my, fabsf(acc[i] * sigmoid_f(acc[i]) * acc[64 + i]));
            ma = fmaxf(ma, fabsf(acc[i]));
            mb = fmaxf(mb, fabsf(acc[64 + i]));
          }
          float* x = sXch + (tiles_done & 1) * 768 + q * 32 + lane;
          x[h * 384] = my;
          x[h * 384 + 128] = ma;
          x[h * 384 + 256] = mb;
          __syncwarp();
          if (lane == 0) mbar_arrive(xch);
          mbar_wait_drain(smem_u32(xch), tiles_done & 1u, wctl, (2 + q) << 8 | kWaitAccFull);
          if (__any_sync(0xffffffffu, *abort_flag)) break;
          my = fmaxf(my, x[(h ^ 1) * 384]);
          ma = fmaxf(ma, x[(h ^ 1) * 384 + 128]);
          mb = fmaxf(mb, x[(h ^ 1) * 384 + 256]);
          if (rv) {
            if (h == 0) {
              p.sy[(size_t)n_blk * p.M + row] = fp8_scale<FP8_E4M3>(my);
              if (p.out2 != nullptr) {
                p.sab[(size_t)n_blk * p.M + row] = fp8_scale<FP8_E4M3>(ma);
                p.sab[(size_t)(n_blk + p.split / 128) * p.M + row] = fp8_scale<FP8_E4M3>(mb);
              }
            }
            const float fy = fp8_factor<FP8_E4M3>(my);
            f8_store_row64(static_cast<uint8_t*>(p.out) + (size_t)row * p.N + col0, p.wide,
                           [&](int i) { return acc[i] * sigmoid_f(acc[i]) * acc[64 + i] * fy; });
            if (p.out2 != nullptr) {
              const float fa = fp8_factor<FP8_E4M3>(ma), fb = fp8_factor<FP8_E4M3>(mb);
              uint8_t* ab = static_cast<uint8_t*>(p.out2) + (size_t)row * 2 * p.N + col0;
              f8_store_row64(ab, p.wide, [&](int i) { return acc[i] * fa; });
              f8_store_row64(ab + p.split, p.wide, [&](int i) { return acc[64 + i] * fb; });
            }
          }
        }
      }
    }
    if constexpr (SPLIT) {
      if (!given) cluster_sync();
      cluster_sync();  // all partial tiles are there, or the abort flag is set in every CTA
      if (!*abort_flag) f8_finish_share<EPI>(p, smem);
    }
  }

  if (warp == 0 && lane == 0) drain_ctl->issued = (uint32_t)issued;
  tc_fence_before();
  cluster_sync();
  if (*abort_flag) {
    if (threadIdx.x == 0) f8_record((uint32_t)*abort_flag, p.status, p.kernel_id);
    // A role gave up: the last (up to STAGES) copies of both CTAs land before
    // shared memory is released.  Copies are only left over where the leader's
    // issuers stopped, so the leader's flag is set.
    if (warp == 0 && lane == 0 && rank == 0)
      pair_copies_landed<S>(full, issued, (int)ld_cluster_u32(mapa_shared(smem_u32(&drain_ctl->issued), leader + 1)),
                            F8_STAGE_BYTES, ctl);
    __syncthreads();
  }
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ------------------------------------------------------------------ few rows
//
// C[m, n] for few rows m (decoding steps, short prompts): the weight is the
// MMA's 128-row operand and the rows of A, TN of them, are its columns, so no
// MMA row is padding.  The product is then a stream of the weight, and the k
// axis is split over a cluster of up to 8 CTAs so that about two CTAs per SM
// have loads in flight; their fp32 partial tiles are added through distributed
// shared memory, in rank order, each CTA finishing its share of the rows.
// Measured (replayed graph): N = K = 4096, 1 to 16 rows 6.5-7.0 us, 64 rows 9.5
// us; N 4096, K 11008, 3 rows 10.3 us (4.4 TB/s of weight).  The 16.8 MB of the
// first take 2.6 us at the copy rate: what is left is the launch, the pipeline's
// filling and the cluster's exchange, once each.
// Roles (192 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA issuer,
// warps 2-5 one weight row per thread.
constexpr int F8S_THREADS = 192;

template <int TN, bool SWIGLU>
struct F8SkinnyCfg {
  static constexpr int W = SWIGLU ? 2 : 1;  // products per tile: gate and up
  static constexpr int STAGE_BYTES = W * F8_A_BYTES + TN * F8_BK;
  static constexpr int STAGES = SWIGLU ? (TN == 16 ? 3 : 2) : TN <= 32 ? 5 : 4;
  static constexpr int CHUNK = 1024 / W;  // scales staged at a time, per product
  static constexpr int BUFS = 4;  // TMEM buffers
  static constexpr uint32_t TMEM = BUFS * TN * W;
  static constexpr int SCALE_BYTES = 2 * W * CHUNK * 4;
  // Row maxima of the 8-bit outputs: [TN][3][4 warps].
  static constexpr int MAX_BYTES = SWIGLU ? TN * 12 * 4 : 0;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SCALE_BYTES + MAX_BYTES + 1024 + 256;
  static_assert(TN * W * 128 * 4 <= STAGES * STAGE_BYTES, "the partial tile takes the ring's place");
  static_assert(TMEM <= 256 && 2 * (SMEM_BYTES + 1024) <= 233472, "two CTAs per SM");
};

struct Skinny8Params {
  int M, N, K;      // M <= TN; SWIGLU: N = F
  int k_blocks;
  const float* sa;  // [k_blocks, M]
  const float* sb;  // [blocks of rows, k_blocks]
  int split;        // SWIGLU: row offset of the up half
  int c_fp32, add;
  void* out;        // C, or Y
  uint8_t* out2;    // AB, or null
  float *sy, *sab;
  uint32_t idesc;
  uint32_t* status;
  unsigned long long wait_limit_ns;
  uint32_t kernel_id;
  uint32_t silent;  // self-test, as Gemm8Params
};

__device__ __forceinline__ void umma_f8_stage(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .b64 a, b;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, 0;\n\t"
      "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
      "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
      "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc)
      : "memory");
}

// 16 accumulator columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}

// Sum of the cluster's copies of one partial, in rank order; the loads are in flight together.
__device__ __forceinline__ float f8_cluster_sum(uint32_t addr, int splits) {
  float v[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) v[r] = r < splits ? ld_cluster_f32(mapa_shared(addr, (uint32_t)r)) : 0.f;
  float s = v[0];
#pragma unroll
  for (int r = 1; r < 8; ++r) s += v[r];
  return s;
}

// SELFTEST: the instance that coda_selftest_fp8_silence launches.  The look for a
// silent role took 0.1 us of 6.4 for one row, 4096 x 4096.
template <int TN, bool SWIGLU, bool SELFTEST>
__global__ void __launch_bounds__(F8S_THREADS, 2)
    gemm_fp8_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                           const Skinny8Params p) {
  using C = F8SkinnyCfg<TN, SWIGLU>;
  constexpr int S = C::STAGES, W = C::W;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sScale = reinterpret_cast<float*>(smem + S * C::STAGE_BYTES);
  float* sMax = sScale + C::SCALE_BYTES / 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(sMax + C::MAX_BYTES / 4);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + C::BUFS;
  uint64_t* mma_done = tempty + C::BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  DrainCtl* drain_ctl =
      reinterpret_cast<DrainCtl*>((reinterpret_cast<uintptr_t>(tmem_slot + 1) + 15) & ~static_cast<uintptr_t>(15));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&drain_ctl->abort);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0);
  const int lane = threadIdx.x % 32;
  const int rank = (int)cluster_ctarank();
  const int splits = (int)cluster_nctarank();
  const int n_blk = (int)blockIdx.x / splits;
  const int kb0 = (int)((long long)rank * p.k_blocks / splits);
  const int nkb = (int)((long long)(rank + 1) * p.k_blocks / splits) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < C::BUFS; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    drain_ctl->limit_ns = p.wait_limit_ns;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns, p.kernel_id};

  float acc[W][TN];
  if (warp == 0) {
    if (lane == 0) {
      // The weight is read once (evict-first); the rows of A by every tile.
      const uint64_t hint_w = l2_policy_evict_first(), hint_x = l2_policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (; issued < nkb; ++issued) {
        if (SELFTEST && f8_silent(p.silent, CODA_FP8_ROLE_LOADS)) break;
        if (!mbar_wait(&empty[stage], phase ^ 1u, ctl, 0, kWaitEmpty)) break;
        uint8_t* dst = smem + stage * C::STAGE_BYTES;
        const int k0 = (kb0 + issued) * F8_BK;
        mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
        tma_load_2d(dst, &tmW, &full[stage], k0, n_blk * 128, hint_w);
        if constexpr (SWIGLU) tma_load_2d(dst + F8_A_BYTES, &tmW, &full[stage], k0, p.split + n_blk * 128, hint_w);
        tma_load_2d(dst + W * F8_A_BYTES, &tmX, &full[stage], k0, 0, hint_x);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // Every copy has landed before this CTA's shared memory is used for anything else or released.
      for (int i = issued > S ? issued - S : 0; i < issued; ++i)
        mbar_wait_own(&full[i % S], (uint32_t)((i / S) & 1), ctl, 0);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      const uint64_t desc0 = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      for (int kb = 0; kb < nkb; ++kb) {
        if (SELFTEST && f8_silent(p.silent, CODA_FP8_ROLE_MMA)) break;
        if (!mbar_wait(&full[stage], phase, ctl, 1, kWaitFull)) break;
        const int buf = kb % C::BUFS;
        if (!mbar_wait(&tempty[buf], ((uint32_t)(kb / C::BUFS) & 1u) ^ 1u, ctl, 1, kWaitAccEmpty)) break;
        tc_fence_after();
        const uint64_t wd = desc0 + (uint64_t)((stage * C::STAGE_BYTES) >> 4);
        const uint64_t xd = wd + ((W * F8_A_BYTES) >> 4);
        const uint32_t d = tmem_base + (uint32_t)(buf * W * TN);
        umma_f8_stage(d, wd, xd, p.idesc);
        if constexpr (SWIGLU) umma_f8_stage(d + TN, wd + (F8_A_BYTES >> 4), xd, p.idesc);
        umma_commit(&tfull[buf]);
        umma_commit(&empty[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      umma_commit(mma_done);
      mbar_wait_own(mma_done, 0, ctl, 1);
    }
  } else {
    const int q = warp & 3;
    const int t128 = q * 32 + lane;  // this thread's weight row
    const uint32_t wctl = smem_u32(drain_ctl);
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int t = 0; t < TN; ++t) acc[w][t] = 0.f;
    // Scales of CHUNK / TN blocks at a time, A's times the weight's, fetched one chunk ahead.
    constexpr int PER = C::CHUNK / 128;
    constexpr int CH = C::CHUNK / TN;  // blocks per chunk
    const float* sb = p.sb + (size_t)n_blk * p.k_blocks + kb0;
    const float* sb2 = sb + (SWIGLU ? (size_t)(p.split / 128) * p.k_blocks : 0);
    float pre[W][PER];
    auto fetch = [&](int c0) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int idx = i * 128 + t128, kb = c0 + idx / TN, m = idx % TN;
        const bool v = kb < nkb && m < p.M;
        const float a = v ? __ldg(p.sa + (size_t)(kb0 + kb) * p.M + m) : 0.f;
        pre[0][i] = v ? a * __ldg(sb + kb) : 0.f;
        if constexpr (SWIGLU) pre[1][i] = v ? a * __ldg(sb2 + kb) : 0.f;
      }
    };
    fetch(0);
    int buf = 0;
    uint32_t phase = 0;
    for (int c0 = 0, par = 0; c0 < nkb; c0 += CH, par ^= 1) {
      float* sc = sScale + par * W * C::CHUNK;
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int i = 0; i < PER; ++i) sc[w * C::CHUNK + i * 128 + t128] = pre[w][i];
      asm volatile("bar.sync 1, 128;" ::: "memory");  // no drain warp leaves this loop early
      if (c0 + CH < nkb) fetch(c0 + CH);
      const int n = min(CH, nkb - c0);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        mbar_wait_drain(smem_u32(&tfull[buf]), phase, wctl, (2 + q) << 8 | kWaitAccFull);
        tc_fence_after();
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* s = sc + w * C::CHUNK + j * TN;
#pragma unroll
          for (int c = 0; c < TN; c += 16) {
            float v[16];
            tmem_ld16(taddr + (uint32_t)((buf * W + w) * TN + c), v);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 f = *reinterpret_cast<const float4*>(s + c + i);
              acc[w][c + i] = fmaf(v[i], f.x, acc[w][c + i]);
              acc[w][c + i + 1] = fmaf(v[i + 1], f.y, acc[w][c + i + 1]);
              acc[w][c + i + 2] = fmaf(v[i + 2], f.z, acc[w][c + i + 2]);
              acc[w][c + i + 3] = fmaf(v[i + 3], f.w, acc[w][c + i + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(smem_u32(&tempty[buf]), lane == 0);
        if (++buf == C::BUFS) {
          buf = 0;
          phase ^= 1u;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();  // the ring is free: every copy has landed and every MMA has read it
  tc_fence_after();

  // The partial tiles, [W][TN][128], in the ring's place.  Everything from here
  // on is rolled loops over shared memory: it runs once per CTA, where unrolled
  // code costs more to fetch than to run (some 100 us over a launch of several
  // waves).
  const int row = (warp & 3) * 32 + lane;
  const bool drains = warp >= 2;
  float* part = reinterpret_cast<float*>(smem);
  if (drains) {
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int t = 0; t < TN; ++t) part[(w * TN + t) * 128 + row] = acc[w][t];
  }
  if (splits > 1) {
    if (threadIdx.x == 0) f8_tell_cluster(&drain_ctl->abort, splits, p.status, p.kernel_id);
    cluster_sync();
  }
  // This CTA's share of the tile's rows of A: [t0, t0 + share).
  const int share = TN / splits, t0 = rank * share;
  const int used = min(share, p.M - t0);  // rows that exist
  const bool bad = *abort_flag != 0;
  const int col = n_blk * 128 + row;
  if (drains && !bad) {
#pragma unroll 1
    for (int t = 0; t < used; ++t) {
      const int m = t0 + t;
      float sum[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float* own = part + (w * TN + t0 + t) * 128 + row;
        sum[w] = splits == 1 ? *own : f8_cluster_sum(smem_u32(own), splits);
      }
      if constexpr (!SWIGLU) {
        if (col < p.N) {
          const size_t o = (size_t)m * p.N + col;
          if (!p.c_fp32) {
            static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(sum[0]);
          } else {
            float* c = static_cast<float*>(p.out) + o;
            *c = p.add ? *c + sum[0] : sum[0];
          }
        }
      } else {
        // Only this CTA reads its own share of its own partial tile.
        const float a = sum[0], b = sum[1], y = a * sigmoid_f(a) * b;
        part[(t0 + t) * 128 + row] = a;
        part[(TN + t0 + t) * 128 + row] = b;
        // fmaxf leaves NaNs out of the maxima.
        const float my = warp_max(fmaxf(fabsf(y), 0.f)), ma = warp_max(fmaxf(fabsf(a), 0.f)),
                    mb = warp_max(fmaxf(fabsf(b), 0.f));
        if (lane == 0) {
          sMax[(t * 3 + 0) * 4 + (warp & 3)] = my;
          sMax[(t * 3 + 1) * 4 + (warp & 3)] = ma;
          sMax[(t * 3 + 2) * 4 + (warp & 3)] = mb;
        }
      }
    }
  }
  if constexpr (SWIGLU) {
    __syncthreads();
    if (drains && !bad) {
#pragma unroll 1
      for (int t = 0; t < used; ++t) {
        const int m = t0 + t;
        float mx[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(sMax + (t * 3 + i) * 4);
          mx[i] = fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w));
        }
        const float a = part[(t0 + t) * 128 + row], b = part[(TN + t0 + t) * 128 + row];
        static_cast<uint8_t*>(p.out)[(size_t)m * p.N + col] =
            (uint8_t)fp8_pack2<FP8_E4M3>(a * sigmoid_f(a) * b * fp8_factor<FP8_E4M3>(mx[0]), 0.f);
        if (p.out2 != nullptr) {
          uint8_t* ab = p.out2 + (size_t)m * 2 * p.N + col;
          ab[0] = (uint8_t)fp8_pack2<FP8_E4M3>(a * fp8_factor<FP8_E4M3>(mx[1]), 0.f);
          ab[p.N] = (uint8_t)fp8_pack2<FP8_E4M3>(b * fp8_factor<FP8_E4M3>(mx[2]), 0.f);
        }
        if (row == 0) {
          p.sy[(size_t)n_blk * p.M + m] = fp8_scale<FP8_E4M3>(mx[0]);
          if (p.out2 != nullptr) {
            p.sab[(size_t)n_blk * p.M + m] = fp8_scale<FP8_E4M3>(mx[1]);
            p.sab[(size_t)(n_blk + p.split / 128) * p.M + m] = fp8_scale<FP8_E4M3>(mx[2]);
          }
        }
      }
    }
  }
  if (splits > 1) cluster_sync();  // peers are done with this CTA's partial tile
  if (threadIdx.x == 0) f8_record((uint32_t)*abort_flag, p.status, p.kernel_id);
  if (warp == 1) tmem_dealloc(tmem_base, C::TMEM);
}

}  // namespace coda
