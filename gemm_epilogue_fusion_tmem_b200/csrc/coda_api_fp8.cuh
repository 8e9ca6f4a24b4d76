// C-ABI entry points of the 8-bit operators (include/coda.h): argument
// validation, tensor maps and launches.  Included at the end of coda_api.cu,
// whose launch, device and timing-hook helpers it uses.
#pragma once

#include "coda_fp8.cuh"
#include "coda_gemm_fp8.cuh"

namespace coda {
namespace {

// Armed by coda_selftest_fp8_silence for this thread's next 8-bit product.
thread_local uint32_t g_fp8_silent = 0;

constexpr int kScaleBlock = 128;  // values per scale along a blocked axis
// Rows of every matrix (and K of the products): row numbers of a partial last tile, and
// those one step of a grid further, are still ints.
constexpr int kMax8Rows = 0x7FFFFFFF - 4095;
constexpr int kMax8Cols = 1 << 22;  // columns of the light passes' matrices: 32-bit offsets in a 128-row tile

// 8-bit matrix [rows][cols], boxes of box_cols x box_rows; out-of-range elements load as zero.
bool make_tmap8(CUtensorMap* m, const void* base, long long rows, long long cols, int box_cols, int box_rows,
                CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Operand with logical shape [mn, k], stored [mn][k] or (mn_major) [k][mn]: boxes
// of 128 k x box_mn, box_mn 64 or 128 when mn_major (its swizzle is the box's width).
bool operand8_map(CUtensorMap* m, const void* p, long long mn, long long k, bool mn_major, int box_mn) {
  if (!mn_major) return make_tmap8(m, p, mn, k, F8_BK, box_mn, CU_TENSOR_MAP_SWIZZLE_128B);
  return make_tmap8(m, p, k, mn, box_mn, F8_BK, box_mn == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Few rows of A: the weight becomes the MMA's 128-row operand, the rows its
// columns (gemm_fp8_skinny_kernel).  Measured at N = K = 4096, few-rows form and
// 256 x 256 tiles (whose reduction four pairs share): 33 rows 9.4 and 13.3 us, 64
// rows 9.7 and 13.9; with 128 columns the few-rows form took 30 us where the tiles
// take 14.  At 64 rows it is ahead or even (2048 x 8192 10.2 and 14.8, 22016 x
// 4096 26.4 and 32.7, 1024 x 1024 7.2 and 7.4) but for 11008 x 4096 (20.2 and
// 17.8).  The gate/up product holds two accumulators and changes over at half the
// rows: K 4096, F 11008, 32 rows 30.8 us in the few-rows form and 34.9 in tiles, 64
// rows 69 and 34.5; K 2048, F 8192, 32 rows 15.0 and 31.4.
inline int skinny8_rows(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

// Rasterisation as pick_group, in bytes of 8-bit operands.
int pick_group8(long long a_rows, long long b_rows, int num_m, int num_n, int k_blocks, int clusters) {
  int side = 1;
  while (side * side < clusters) ++side;
  const long long budget = (long long)raster_budget_mb() << 20;
  const long long g = std::max<long long>(side, budget / (256LL * k_blocks * F8_BK));
  if (a_rows <= b_rows) return (int)std::min<long long>(num_m, g);
  return -(int)std::min<long long>(num_n, g);
}

// Clusters of 2 * parts CTAs of a kernel that the device holds at once.
template <int EPI, bool A_MN, bool B_MN, bool VEC, bool SPLIT>
coda_status gemm8_clusters(int parts, int& clusters) {
  static std::atomic<int> of[kMaxDevices][5];  // 0: not set up on this device yet
  int dev = 0;
  CODA_TRY(current_device(dev));
  auto kern = gemm_fp8_kernel<EPI, A_MN, B_MN, VEC, SPLIT>;
  clusters = of[dev][parts].load();
  if (clusters == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F8_SMEM_BYTES) != cudaSuccess)
      return CODA_ERR_CUDA;
    clusters = g_dev[dev].num_sms / (2 * parts);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * parts * clusters, 1, 1);
    cfg.blockDim = dim3(F8_THREADS, 1, 1);
    cfg.dynamicSmemBytes = F8_SMEM_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0) clusters = std::min(clusters, n);
    of[dev][parts].store(clusters);
  }
  return CODA_OK;
}

template <int EPI, bool A_MN, bool B_MN, bool VEC, bool SPLIT = false>
coda_status launch_gemm8(const CUtensorMap& ta, const CUtensorMap& tb, Gemm8Params p, cudaStream_t s, int parts = 1) {
  auto kern = gemm_fp8_kernel<EPI, A_MN, B_MN, VEC, SPLIT>;
  int clusters = 0;
  CODA_TRY((gemm8_clusters<EPI, A_MN, B_MN, VEC, SPLIT>(parts, clusters)));
  p.wait_limit_ns = g_wait_limit_ns.load();
  p.silent = std::exchange(g_fp8_silent, 0u);
  p.kernel_id = 0x40 + (uint32_t)(EPI * 8 + (A_MN ? 4 : 0) + (B_MN ? 2 : 0) + (VEC ? 1 : 0)) + (SPLIT ? 0x40 : 0);
  const long long tiles = (long long)p.num_m_tiles * p.num_n_tiles;
  const int units = SPLIT ? (int)tiles : (int)std::min<long long>(tiles, clusters);
  g_launch_tag = EPI == F8_EPI_SWIGLU ? CODA_KERNEL_GEMM_SWIGLU_FP8 : CODA_KERNEL_GEMM_FP8;
  const cudaError_t e = launch_ex(kern, dim3(2 * parts * units), dim3(F8_THREADS), F8_SMEM_BYTES, s, 2 * parts, ta, tb, p);
  g_launch_tag = -1;
  return e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess ? CODA_OK : CODA_ERR_CUDA;
}

// An activation's product with a weight: when its tiles leave pairs idle, the
// reduction of each is shared by 2 to 4 of them, as many as the device holds at
// once.  The exchange costs 4 to 5 us, a block of k 0.4: it is done where a pair
// is spared 12 blocks.  Measured without and with it, N = 2048: 256 rows (4
// pairs), K 2048 11.4 and 11.2 us, K 8192 27.5 and 15.9; 1001 rows (32 tiles, 2
// pairs), K 4096 16.9 and 16.1, K 16384 50.2 and 34.7; below the limit, K 2688
// 13.5 and 14.3.
// Weight gradients are not shared: a scale per column needs another layout of the
// partial tiles.  A weight of fewer than 74 tiles leaves pairs idle (K 8192: 2048 x
// 2048, 64 tiles, 43 us; 512 x 2048, 16 tiles, 40 us).
template <int EPI, bool B_MN>
coda_status activation_parts(long long tiles, int k_blocks, int& parts) {
  for (parts = 4; parts > 1; --parts) {
    if (tiles * 2 * parts > num_sms() || k_blocks - cdiv(k_blocks, parts) < 12) continue;
    int clusters = 0;
    CODA_TRY((gemm8_clusters<EPI, false, B_MN, false, true>(parts, clusters)));
    if (tiles <= clusters) return CODA_OK;
  }
  return CODA_OK;  // 1: not shared
}
template <int EPI, bool B_MN>
coda_status launch_gemm8_activation(const CUtensorMap& ta, const CUtensorMap& tb, const Gemm8Params& p, cudaStream_t s) {
  int parts = 1;
  CODA_TRY((activation_parts<EPI, B_MN>((long long)p.num_m_tiles * p.num_n_tiles, p.k_blocks, parts)));
  if (parts > 1) return launch_gemm8<EPI, false, B_MN, false, true>(ta, tb, p, s, parts);
  return launch_gemm8<EPI, false, B_MN, false>(ta, tb, p, s);
}

template <int EPI, bool VEC>
coda_status launch_gemm8_majors(const CUtensorMap& ta, const CUtensorMap& tb, bool a_mn, bool b_mn,
                                const Gemm8Params& p, cudaStream_t s) {
  if constexpr (!VEC) {
    if (!a_mn) return b_mn ? launch_gemm8_activation<EPI, true>(ta, tb, p, s) : launch_gemm8_activation<EPI, false>(ta, tb, p, s);
  } else {
    if (!a_mn && !b_mn) return launch_gemm8<EPI, false, false, VEC>(ta, tb, p, s);
    if (!a_mn && b_mn) return launch_gemm8<EPI, false, true, VEC>(ta, tb, p, s);
  }
  if (a_mn && b_mn) return launch_gemm8<EPI, true, true, VEC>(ta, tb, p, s);
  return launch_gemm8<EPI, true, false, VEC>(ta, tb, p, s);
}

// CTAs that share the reduction of a tile of the few-rows kernel: doubled while there
// are two CTAs per SM to be had and two blocks of k for each.
inline int skinny8_splits(int tiles, int k_blocks) {
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= 2 * num_sms() && splits * 4 <= k_blocks) splits *= 2;
  return splits;
}

// Tiles of the few-rows kernel: 128 weight rows (and their partners in the up
// half) x up to TN rows of A, split over k by a cluster.
template <int TN, bool SWIGLU, bool SELFTEST>
coda_status launch_skinny8_as(const CUtensorMap& tw, const CUtensorMap& tx, Skinny8Params p, cudaStream_t s) {
  using C = F8SkinnyCfg<TN, SWIGLU>;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  coda_status st = current_device(dev);
  if (st != CODA_OK) return st;
  auto kern = gemm_fp8_skinny_kernel<TN, SWIGLU, SELFTEST>;
  if (!ready[dev].load()) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
      return CODA_ERR_CUDA;
    ready[dev].store(true);
  }
  const int tiles = cdiv(p.N, 128);
  const int splits = skinny8_splits(tiles, p.k_blocks);
  p.idesc = (p.idesc & ~(0x3Fu << 17)) | ((uint32_t)(TN >> 3) << 17);
  p.wait_limit_ns = g_wait_limit_ns.load();
  p.silent = std::exchange(g_fp8_silent, 0u);
  p.kernel_id = 0x60 + (uint32_t)(TN / 16 * 2 + (SWIGLU ? 1 : 0));
  g_launch_tag = SWIGLU ? CODA_KERNEL_GEMM_SWIGLU_FP8 : CODA_KERNEL_GEMM_FP8;
  const cudaError_t e =
      launch_ex(kern, dim3(tiles * splits), dim3(F8S_THREADS), C::SMEM_BYTES, s, splits, tw, tx, p);
  g_launch_tag = -1;
  return e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess ? CODA_OK : CODA_ERR_CUDA;
}

template <int TN, bool SWIGLU>
coda_status launch_skinny8(const CUtensorMap& tw, const CUtensorMap& tx, const Skinny8Params& p, cudaStream_t s) {
  return g_fp8_silent ? launch_skinny8_as<TN, SWIGLU, true>(tw, tx, p, s)
                      : launch_skinny8_as<TN, SWIGLU, false>(tw, tx, p, s);
}

// Few rows of an activation by a weight as it is stored.
inline bool gemm8_few_rows(int M, bool a_mn, bool b_mn, bool b_blocks) { return M <= 64 && !a_mn && !b_mn && b_blocks; }

inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
inline bool known_format(int f) { return f == CODA_FP8_E4M3 || f == CODA_FP8_E5M2; }
inline bool tiles_fit(long long a, long long b) { return a * b <= 0x7FFFFFFFLL; }

// One launch of a light pass under its timing-hook id.
template <typename... KArgs, typename P>
coda_status launch_pass(int tag, void (*kern)(KArgs...), int grid, int block, void* stream, const P& p) {
  g_launch_tag = tag;
  const cudaError_t e = launch_ex(kern, dim3(grid), dim3(block), 0, static_cast<cudaStream_t>(stream), 1, p);
  g_launch_tag = -1;
  return launch_status(e);
}

template <int FMT>
coda_status quant8(const QuantParams& p, bool rows, bool cols, bool vec, int grid, void* stream) {
  const int tag = CODA_KERNEL_QUANT_FP8;
  if (vec) {
    if (rows && cols) return launch_pass(tag, quant_fp8_kernel<FMT, true, true, false, true>, grid, kQuantThreads, stream, p);
    if (rows) return launch_pass(tag, quant_fp8_kernel<FMT, true, false, false, true>, grid, kQuantThreads, stream, p);
    return launch_pass(tag, quant_fp8_kernel<FMT, false, true, false, true>, grid, kQuantThreads, stream, p);
  }
  if (rows && cols) return launch_pass(tag, quant_fp8_kernel<FMT, true, true, false, false>, grid, kQuantThreads, stream, p);
  if (rows) return launch_pass(tag, quant_fp8_kernel<FMT, true, false, false, false>, grid, kQuantThreads, stream, p);
  return launch_pass(tag, quant_fp8_kernel<FMT, false, true, false, false>, grid, kQuantThreads, stream, p);
}

// A row over 256 threads from d = 1025 to 8192: fewer threads of more columns leave
// too few loads in flight per SM, more of them wait for one another (8192 rows;
// 128, 256 and 512 threads: d = 2048 23.6, 22.1 us, -; d = 4096 42.6, 40.0, 42.1
// us; d = 8192 -, 76.5, 80.6 us).  Wider rows need the registers of more threads.
template <int T, int CH>
coda_status rms8_fwd(const RmsParams& p, void* stream) {
  return launch_pass(CODA_KERNEL_RMSNORM_FP8_FWD, rmsnorm_fp8_fwd_kernel<T, CH>, p.M, T, stream, p);
}

// Widest row the norms hold in registers.
constexpr int kRms8MaxD = 1024 * 4 * 8;

// Threads per row of the norm's backward (8 columns each up to d = 8192: with 16
// columns the next row's loads no longer fit in registers, 67 us against 45 for
// 8192 x 4096 in L2-warm runs; wider rows, of 16 and 32 columns a thread, spill 56
// and 416 bytes: 4096 x 16384 110 us, 2048 x 32768 199 us), and its CTAs: a thousand threads per SM, each
// CTA keeping its share of dg in registers and writing one partial row.
int rms8_bwd_threads(int d) { return d <= 1024 ? 128 : d <= 2048 ? 256 : d <= 4096 ? 512 : 1024; }
int rms8_bwd_ctas(int M, int d) { return std::min(M, 148 * (1024 / rms8_bwd_threads(d))); }

template <int T, int CH>
coda_status rms8_bwd(const RmsBwdParams& p, void* stream) {
  return launch_pass(CODA_KERNEL_RMSNORM_FP8_BWD, rmsnorm_fp8_bwd_kernel<T, CH>, rms8_bwd_ctas(p.M, p.d), T, stream, p);
}

// The status word of calls that bring no workspace, one per device.
__device__ __align__(256) unsigned char g_shared_status[kStatusBytes];
std::atomic<void*> g_shared_status_addr[kMaxDevices];

}  // namespace
}  // namespace coda

extern "C" {

coda_status coda_shared_status(void** ws) {
  if (ws == nullptr) return CODA_ERR_INVALID_ARG;
  int dev;
  CODA_TRY(current_device(dev));
  void* p = g_shared_status_addr[dev].load();
  if (p == nullptr) {
    if (cudaGetSymbolAddress(&p, g_shared_status) != cudaSuccess || p == nullptr) return CODA_ERR_CUDA;
    g_shared_status_addr[dev].store(p);
  }
  *ws = p;
  return CODA_OK;
}

coda_status coda_selftest_fp8_silence(int role, int cta) {
  if (role < 0 || role > CODA_FP8_ROLE_SCALES || cta < 0 || cta >= 1 << 20) return CODA_ERR_INVALID_ARG;
  g_fp8_silent = role == 0 ? 0u : (uint32_t)cta << 2 | (uint32_t)role;
  return CODA_OK;
}

// ------------------------------------------------------------------ quantiser

coda_status coda_quant_fp8(const void* X, const float* rowvec_or_null, const void* colvec_or_null, void* Qr_or_null,
                           float* Sr_or_null, void* Qc_or_null, float* Sc_or_null, int R, int C, int format,
                           void* stream) {
  const bool rows = Qr_or_null != nullptr || Sr_or_null != nullptr;
  const bool cols = Qc_or_null != nullptr || Sc_or_null != nullptr;
  if (R < 0 || C < 1 || !known_format(format)) return CODA_ERR_INVALID_ARG;
  if (C % 16 != 0 || C > kMax8Cols || R > kMax8Rows || !tiles_fit(cdiv(R, kScaleBlock), cdiv(C, kScaleBlock)))
    return CODA_ERR_UNSUPPORTED_SHAPE;
  if (R == 0) return CODA_OK;
  if (!X || (!rows && !cols)) return CODA_ERR_INVALID_ARG;
  if (rows && (!Qr_or_null || !Sr_or_null)) return CODA_ERR_INVALID_ARG;
  if (cols && (!Qc_or_null || !Sc_or_null)) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {X, rowvec_or_null, colvec_or_null, Qr_or_null, Sr_or_null, Qc_or_null, Sc_or_null};
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return CODA_ERR_MISALIGNED;
  int dev;
  CODA_TRY(current_device(dev));
  QuantParams p;
  p.x = cbf(X);
  p.rowvec = rowvec_or_null;
  p.colvec = cbf(colvec_or_null);
  p.qr = static_cast<uint8_t*>(Qr_or_null);
  p.sr = Sr_or_null;
  p.qc = static_cast<uint8_t*>(Qc_or_null);
  p.sc = Sc_or_null;
  p.R = R;
  p.C = C;
  p.tiles_c = cdiv(C, kScaleBlock);
  const int grid = cdiv(R, kScaleBlock) * p.tiles_c;
  const bool vec = rowvec_or_null != nullptr || colvec_or_null != nullptr;
  return format == CODA_FP8_E4M3 ? quant8<FP8_E4M3>(p, rows, cols, vec, grid, stream)
                                 : quant8<FP8_E5M2>(p, rows, cols, vec, grid, stream);
}

coda_status coda_quant_fp8_blocks(const void* W, void* Q, float* S, int R, int C, int format, void* stream) {
  if (R < 0 || C < 1 || !known_format(format)) return CODA_ERR_INVALID_ARG;
  if (C % 16 != 0 || C > kMax8Cols || R > kMax8Rows || !tiles_fit(cdiv(R, kScaleBlock), cdiv(C, kScaleBlock)))
    return CODA_ERR_UNSUPPORTED_SHAPE;
  if (R == 0) return CODA_OK;
  if (!W || !Q || !S) return CODA_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(Q) || !aligned16(S)) return CODA_ERR_MISALIGNED;
  int dev;
  CODA_TRY(current_device(dev));
  QuantParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = cbf(W);
  p.qc = static_cast<uint8_t*>(Q);
  p.sc = S;
  p.R = R;
  p.C = C;
  p.tiles_c = cdiv(C, kScaleBlock);
  const int grid = cdiv(R, kScaleBlock) * p.tiles_c;
  if (format == CODA_FP8_E4M3)
    return launch_pass(CODA_KERNEL_QUANT_FP8, quant_fp8_kernel<FP8_E4M3, false, false, true, false>, grid,
                       kQuantThreads, stream, p);
  return launch_pass(CODA_KERNEL_QUANT_FP8, quant_fp8_kernel<FP8_E5M2, false, false, true, false>, grid,
                     kQuantThreads, stream, p);
}

// ------------------------------------------------------------------ GEMM

coda_status coda_gemm_fp8(const void* A, const float* SA, const void* B, const float* SB, void* C, int M, int N, int K,
                          int a_mn_major, int b_mn_major, int a_format, int b_format, int b_blocks, int c_fp32,
                          int accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !known_format(a_format) || !known_format(b_format)) return CODA_ERR_INVALID_ARG;
  if (accumulate && !c_fp32) return CODA_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return CODA_OK;  // empty output
  if (N % 16 != 0 || (a_mn_major ? M : K) % 16 != 0 || (!b_mn_major && K % 16 != 0)) return CODA_ERR_UNSUPPORTED_SHAPE;
  if (M > kMax8Rows || N > kMax8Rows || K > kMax8Rows || !tiles_fit(cdiv(M, 256), cdiv(N, 256)))
    return CODA_ERR_UNSUPPORTED_SHAPE;
  if (K == 0) {  // empty sums
    if (!C) return CODA_ERR_INVALID_ARG;
    return accumulate ? CODA_OK : zero_fill({{C, (size_t)M * N * (c_fp32 ? 4 : 2)}}, stream);
  }
  if (!A || !SA || !B || !SB || !C || !ws) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {A, SA, B, SB, C, ws};
  for (const void* q : ptrs)
    if (!aligned16(q)) return CODA_ERR_MISALIGNED;
  if (ws_bytes < coda_gemm_workspace_bytes()) return CODA_ERR_WORKSPACE_TOO_SMALL;
  int dev;
  CODA_TRY(current_device(dev));
  const bool a_mn = a_mn_major != 0, b_mn = b_mn_major != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap ta, tb;
  if (gemm8_few_rows(M, a_mn, b_mn, b_blocks != 0)) {
    const int tn = skinny8_rows(M);
    if (!operand8_map(&tb, B, N, K, false, 128) || !operand8_map(&ta, A, M, K, false, tn)) return CODA_ERR_CUDA;
    Skinny8Params p;
    std::memset(&p, 0, sizeof(p));
    p.M = M;
    p.N = N;
    p.K = K;
    p.k_blocks = cdiv(K, F8_BK);
    p.sa = SA;
    p.sb = SB;
    p.c_fp32 = c_fp32;
    p.add = accumulate;
    p.out = C;
    p.idesc = make_idesc_f8(128, 0, b_format, a_format, false, false);  // the weight is the MMA's first operand
    p.status = static_cast<uint32_t*>(ws);
    if (tn == 16) return launch_skinny8<16, false>(tb, ta, p, s);
    if (tn == 32) return launch_skinny8<32, false>(tb, ta, p, s);
    return launch_skinny8<64, false>(tb, ta, p, s);
  }
  if (!operand8_map(&ta, A, M, K, a_mn, 128) || !operand8_map(&tb, B, N, K, b_mn, 64)) return CODA_ERR_CUDA;
  Gemm8Params p;
  std::memset(&p, 0, sizeof(p));
  p.M = M;
  p.N = N;
  p.K = K;
  p.num_m_tiles = cdiv(M, 256);
  p.num_n_tiles = cdiv(N, 256);
  p.k_blocks = cdiv(K, F8_BK);
  p.group_m = pick_group8(M, N, p.num_m_tiles, p.num_n_tiles, p.k_blocks, num_sms() / 2);
  p.sa = SA;
  p.sb = SB;
  // Block scales of the stored matrix: [N / 128, K / 128], or [K / 128, N / 128] when k is the row.
  p.sb_n = b_mn ? 1 : p.k_blocks;
  p.sb_k = b_mn ? cdiv(N, kScaleBlock) : 1;
  p.add = accumulate;
  p.out = C;
  p.wide = aligned32(C);
  p.idesc = make_idesc_f8(256, 128, a_format, b_format, a_mn, b_mn);
  p.status = static_cast<uint32_t*>(ws);
  if (c_fp32)
    return b_blocks ? launch_gemm8_majors<F8_EPI_F32, false>(ta, tb, a_mn, b_mn, p, s)
                    : launch_gemm8_majors<F8_EPI_F32, true>(ta, tb, a_mn, b_mn, p, s);
  return b_blocks ? launch_gemm8_majors<F8_EPI_BF16, false>(ta, tb, a_mn, b_mn, p, s)
                  : launch_gemm8_majors<F8_EPI_BF16, true>(ta, tb, a_mn, b_mn, p, s);
}

coda_status coda_gemm_fp8_parts(int M, int N, int K, int a_mn_major, int b_mn_major, int b_blocks, int c_fp32,
                                int* few_rows, int* parts) {
  if (M < 1 || N < 1 || K < 1 || few_rows == nullptr || parts == nullptr) return CODA_ERR_INVALID_ARG;
  int dev;
  CODA_TRY(current_device(dev));
  *few_rows = gemm8_few_rows(M, a_mn_major != 0, b_mn_major != 0, b_blocks != 0);
  *parts = 1;
  const int k_blocks = cdiv(K, F8_BK);
  const long long tiles = (long long)cdiv(M, 256) * cdiv(N, 256);
  if (*few_rows) {
    *parts = skinny8_splits(cdiv(N, 128), k_blocks);
    return CODA_OK;
  }
  if (a_mn_major || !b_blocks) return CODA_OK;
  if (c_fp32) return b_mn_major ? activation_parts<F8_EPI_F32, true>(tiles, k_blocks, *parts)
                                : activation_parts<F8_EPI_F32, false>(tiles, k_blocks, *parts);
  return b_mn_major ? activation_parts<F8_EPI_BF16, true>(tiles, k_blocks, *parts)
                    : activation_parts<F8_EPI_BF16, false>(tiles, k_blocks, *parts);
}

coda_status coda_gemm_swiglu_fp8(const void* A, const float* SA, const void* Wgu, const float* SW, void* Y, float* SY,
                                 void* AB_or_null, float* SAB_or_null, int M, int K, int F, void* ws, size_t ws_bytes,
                                 void* stream) {
  if (M < 0 || K < 1 || F < 1) return CODA_ERR_INVALID_ARG;
  if (K % 16 != 0 || F % kScaleBlock != 0 || F > kMax8Cols || M > kMax8Rows || K > kMax8Rows ||
      !tiles_fit(cdiv(M, 256), F / kScaleBlock))
    return CODA_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return CODA_OK;
  if (!A || !SA || !Wgu || !SW || !Y || !SY || !ws) return CODA_ERR_INVALID_ARG;
  if ((AB_or_null == nullptr) != (SAB_or_null == nullptr)) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {A, SA, Wgu, SW, Y, SY, AB_or_null, SAB_or_null, ws};
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return CODA_ERR_MISALIGNED;
  if (ws_bytes < coda_gemm_workspace_bytes()) return CODA_ERR_WORKSPACE_TOO_SMALL;
  int dev;
  CODA_TRY(current_device(dev));
  CUtensorMap ta, tb;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M <= 32) {
    const int tn = skinny8_rows(M);
    if (!operand8_map(&tb, Wgu, 2LL * F, K, false, 128) || !operand8_map(&ta, A, M, K, false, tn)) return CODA_ERR_CUDA;
    Skinny8Params p;
    std::memset(&p, 0, sizeof(p));
    p.M = M;
    p.N = F;
    p.K = K;
    p.k_blocks = cdiv(K, F8_BK);
    p.sa = SA;
    p.sb = SW;
    p.split = F;
    p.out = Y;
    p.out2 = static_cast<uint8_t*>(AB_or_null);
    p.sy = SY;
    p.sab = SAB_or_null;
    p.idesc = make_idesc_f8(128, 0, FP8_E4M3, FP8_E4M3, false, false);
    p.status = static_cast<uint32_t*>(ws);
    if (tn == 16) return launch_skinny8<16, true>(tb, ta, p, s);
    return launch_skinny8<32, true>(tb, ta, p, s);
  }
  if (!operand8_map(&ta, A, M, K, false, 128) || !operand8_map(&tb, Wgu, 2LL * F, K, false, 64)) return CODA_ERR_CUDA;
  Gemm8Params p;
  std::memset(&p, 0, sizeof(p));
  p.M = M;
  p.N = F;
  p.K = K;
  p.num_m_tiles = cdiv(M, 256);
  p.num_n_tiles = F / kScaleBlock;
  p.k_blocks = cdiv(K, F8_BK);
  p.group_m = pick_group8(M, 2LL * F, p.num_m_tiles, p.num_n_tiles, p.k_blocks, num_sms() / 2);
  p.sa = SA;
  p.sb = SW;
  p.sb_n = p.k_blocks;
  p.sb_k = 1;
  p.split = F;
  p.out = Y;
  p.out2 = AB_or_null;
  p.wide = aligned32(Y) && aligned32(AB_or_null);
  p.sy = SY;
  p.sab = SAB_or_null;
  p.idesc = make_idesc_f8(256, 128, FP8_E4M3, FP8_E4M3, false, false);
  p.status = static_cast<uint32_t*>(ws);
  return launch_gemm8<F8_EPI_SWIGLU, false, false, false>(ta, tb, p, s);
}

// ------------------------------------------------------------------ SwiGLU backward

coda_status coda_swiglu_fp8_bwd(const void* dY, const void* AB, const float* SAB, void* dA, float* SdA,
                                void* dAc_or_null, float* SdAc_or_null, void* Yc_or_null, float* SYc_or_null, int M,
                                int F, int format, void* stream) {
  if (M < 0 || F < 1 || !known_format(format)) return CODA_ERR_INVALID_ARG;
  if (F % kScaleBlock != 0 || F > kMax8Cols || M > kMax8Rows || !tiles_fit(cdiv(M, kScaleBlock), F / kScaleBlock))
    return CODA_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return CODA_OK;
  if (!dY || !AB || !SAB || !dA || !SdA) return CODA_ERR_INVALID_ARG;
  const void* cols[] = {dAc_or_null, SdAc_or_null, Yc_or_null, SYc_or_null};
  int given = 0;
  for (const void* q : cols) given += q != nullptr;
  if (given != 0 && given != 4) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {dY, AB, SAB, dA, SdA, dAc_or_null, SdAc_or_null, Yc_or_null, SYc_or_null};
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return CODA_ERR_MISALIGNED;
  int dev;
  CODA_TRY(current_device(dev));
  SwigluBwd8Params p;
  p.dy = cbf(dY);
  p.ab = static_cast<const uint8_t*>(AB);
  p.sab = SAB;
  p.da = static_cast<uint8_t*>(dA);
  p.sda = SdA;
  p.dac = static_cast<uint8_t*>(dAc_or_null);
  p.sdac = SdAc_or_null;
  p.yc = static_cast<uint8_t*>(Yc_or_null);
  p.syc = SYc_or_null;
  p.M = M;
  p.F = F;
  const int grid = cdiv(M, kScaleBlock) * (F / kScaleBlock);
  const int tag = CODA_KERNEL_SWIGLU_FP8_BWD;
  if (format == CODA_FP8_E4M3)
    return given ? launch_pass(tag, swiglu_fp8_bwd_kernel<FP8_E4M3, true>, grid, kSwBwdThreads, stream, p)
                 : launch_pass(tag, swiglu_fp8_bwd_kernel<FP8_E4M3, false>, grid, kSwBwdThreads, stream, p);
  return given ? launch_pass(tag, swiglu_fp8_bwd_kernel<FP8_E5M2, true>, grid, kSwBwdThreads, stream, p)
               : launch_pass(tag, swiglu_fp8_bwd_kernel<FP8_E5M2, false>, grid, kSwBwdThreads, stream, p);
}

// ------------------------------------------------------------------ RMSNorm

coda_status coda_rmsnorm_fp8_fwd(const void* X, const void* R_or_null, const void* g, void* H_or_null, float* r,
                                 void* Q, float* S, int M, int d, float eps, void* stream) {
  if (M < 0 || d < 1 || !(eps > 0.f)) return CODA_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > kRms8MaxD || M > kMax8Rows) return CODA_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return CODA_OK;
  if (!X || !g || !r || !Q || !S || (R_or_null == nullptr) != (H_or_null == nullptr)) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {X, R_or_null, g, H_or_null, r, Q, S};
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return CODA_ERR_MISALIGNED;
  int dev;
  CODA_TRY(current_device(dev));
  RmsParams p;
  p.x = cbf(X);
  p.res = cbf(R_or_null);
  p.g = cbf(g);
  p.h = bf(H_or_null);
  p.r = r;
  p.q = static_cast<uint8_t*>(Q);
  p.s = S;
  p.M = M;
  p.d = d;
  p.inv_d = 1.0f / (float)d;
  p.eps = eps;
  const int chunks = d / 8;
  if (chunks <= 128) return rms8_fwd<128, 1>(p, stream);
  if (chunks <= 256) return rms8_fwd<256, 1>(p, stream);
  if (chunks <= 512) return rms8_fwd<256, 2>(p, stream);
  if (chunks <= 1024) return rms8_fwd<256, 4>(p, stream);
  if (chunks <= 2048) return rms8_fwd<512, 4>(p, stream);
  return rms8_fwd<1024, 4>(p, stream);
}

size_t coda_rmsnorm_fp8_bwd_workspace_bytes(int M, int d) {
  if (M < 1 || d < 1) return kStatusBytes;
  return kStatusBytes + (size_t)rms8_bwd_ctas(M, d) * d * 4;
}

coda_status coda_rmsnorm_fp8_bwd(const void* dN, const void* H, const float* r, const void* g,
                                 const void* dH_in_or_null, void* dH, float* dg, int M, int d, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (M < 0 || d < 1) return CODA_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > kRms8MaxD || M > kMax8Rows) return CODA_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return zero_fill({{dg, (size_t)d * 4}}, stream);
  if (!dN || !H || !r || !g || !dH || !dg || !ws) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {dN, H, r, g, dH_in_or_null, dH, dg, ws};
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return CODA_ERR_MISALIGNED;
  if (ws_bytes < coda_rmsnorm_fp8_bwd_workspace_bytes(M, d)) return CODA_ERR_WORKSPACE_TOO_SMALL;
  int dev;
  CODA_TRY(current_device(dev));
  RmsBwdParams p;
  p.dn = cbf(dN);
  p.h = cbf(H);
  p.r = r;
  p.g = cbf(g);
  p.dh_in = cbf(dH_in_or_null);
  p.dh = bf(dH);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes);
  p.M = M;
  p.d = d;
  p.inv_d = 1.0f / (float)d;
  coda_status st;
  if (d <= 1024) st = rms8_bwd<128, 1>(p, stream);
  else if (d <= 2048) st = rms8_bwd<256, 1>(p, stream);
  else if (d <= 4096) st = rms8_bwd<512, 1>(p, stream);
  else if (d <= 8192) st = rms8_bwd<1024, 1>(p, stream);
  else if (d <= 16384) st = rms8_bwd<1024, 2>(p, stream);
  else st = rms8_bwd<1024, 4>(p, stream);
  if (st != CODA_OK) return st;
  return launch_status(launch_ex(rmsnorm_fp8_dg_kernel, dim3(cdiv(d, 32)), dim3(kRmsDgThreads), 0,
                                 static_cast<cudaStream_t>(stream), 1, (const float*)p.part, rms8_bwd_ctas(M, d), d,
                                 dg));
}

}  // extern "C"
