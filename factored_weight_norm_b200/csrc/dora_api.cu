// dora_api.cu - the C ABI declared in include/dora.h: argument validation,
// launch planning, TMA descriptor encoding and kernel launches.
//
// The library never allocates device memory: every buffer, including the
// workspace, comes from the caller.  All work is enqueued on the caller's
// stream.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>
#include <atomic>
#include <chrono>
#include <mutex>

#include "../../include/dora.h"
#include "ckpt8.cuh"
#include "compose.cuh"
#include "linear_ckpt8.cuh"
#include "linear_i8.cuh"
#include "linear_slice.cuh"
#include "linear_tc.cuh"
#include "norm_bwd.cuh"
#include "norm_simt.cuh"
#include "norm_tc.cuh"
#include "gram_cluster.cuh"
#include "norm_batched.cuh"

namespace dora {

// Device-side status word: kernels write DORA_ERR_TIMEOUT here when a bounded
// wait gives up.  One per device (a __device__ variable lives in every
// context that loads the library).
__device__ int g_status = 0;

namespace {

constexpr long long kWaitLimitCycles = 2000000000LL;  // ~1 s at B200 clocks

// linear_pair_kernel: as many 32 KB stages as fit, at most kLinStagesMax
int linear_pair_stages(int smem_optin) {
  return static_cast<int>(std::min<size_t>(kLinStagesMax, (smem_optin - 1024 - kLinBarrierBytes) / kPairStageBytes));
}
size_t linear_pair_smem(int smem_optin) {
  return static_cast<size_t>(linear_pair_stages(smem_optin)) * kPairStageBytes + 1024 + kLinBarrierBytes;
}
// Pair tile width along N for an output of N columns: the one of 256, 192,
// 128 that pads N least (the wider on a tie), e.g. r = 384 -> 2 x 192.
int pick_bn(long long N) {
  int best = 256;
  long long waste = (N + 255) / 256 * 256 - N;
  for (int bn : {192, 128}) {
    const long long w = (N + bn - 1) / bn * bn - N;
    if (w < waste) {
      waste = w;
      best = bn;
    }
  }
  return best;
}

// linear_i8_pair_kernel: the same stages beside its column factors
int linear_i8_stages(int smem_optin) {
  return static_cast<int>(
      std::min<size_t>(kLinStagesMax, (smem_optin - 1024 - kI8ColBytes - kI8BarrierBytes) / kPairStageBytes));
}
size_t linear_i8_smem(int smem_optin) {
  return static_cast<size_t>(linear_i8_stages(smem_optin)) * kPairStageBytes + 1024 + kI8ColBytes + kI8BarrierBytes;
}

typedef void (*SliceKernel)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, SliceArgs);
template <bool I8>
SliceKernel slice_kernel(int bn) {
  return bn == 16   ? linear_slice_kernel<I8, 16>
         : bn == 32 ? linear_slice_kernel<I8, 32>
         : bn == 64 ? linear_slice_kernel<I8, 64>
                    : linear_slice_kernel<I8, 128>;
}
SliceKernel slice_kernel(bool i8, int bn) { return i8 ? slice_kernel<true>(bn) : slice_kernel<false>(bn); }

template <typename K>
int pair_attrs(K kernel, int smem_optin) {
  return (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_optin) != cudaSuccess ||
          cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 0) != cudaSuccess)
             ? DORA_ERR_CUDA
             : DORA_OK;
}
constexpr int kMaxGrid = 1024;                         // bound on the persistent grid
constexpr int kMaxGramSplits = 32;
constexpr int kGramMinBlocks = 4;                      // fewest K blocks a Gram CTA of the norm takes
constexpr int kMaxBwdChunks = 64;
constexpr int kMaxDevices = 64;
constexpr int64_t kMaxRank = 4096;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

template <typename K>
int ctas_per_sm(K kernel, int threads);

struct DeviceInfo {
  bool ready = false;
  int num_sms = 0;
  int smem_optin = 0;
  int* status = nullptr;
  int pair_clusters = 0;  // co-resident 2-CTA clusters of linear_pair_kernel
  int ckpt_bwd_ctas[3] = {1, 1, 1};  // resident CTAs per SM of compose_bwd_ckpt8_kernel, by L::kIndex
};

std::mutex g_mu;

// Kernels this library has launched in this process (every launch site
// counts itself once, before it launches).
std::atomic<unsigned long long> g_launches{0};
inline void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }
DeviceInfo g_dev[kMaxDevices];

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

// Per-device set-up, done once with that device current.
template <typename K>
int gram_cluster_attrs(K kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kGcSmem)) !=
                 cudaSuccess ||
             cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                  cudaSharedmemCarveoutMaxShared) != cudaSuccess
             ? DORA_ERR_CUDA
             : DORA_OK;
}

int device_info(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DORA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    if (cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DORA_ERR_CUDA;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) return DORA_ERR_CUDA;
    d.status = static_cast<int*>(p);
    if (cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
      return DORA_ERR_CUDA;
    if (cudaFuncSetAttribute(norm_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem_optin) != cudaSuccess)
      return DORA_ERR_CUDA;
    if (cudaFuncSetAttribute(gram_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem_optin) != cudaSuccess)
      return DORA_ERR_CUDA;
    // Kernels that run beside the first CTAs of a GEMM launched behind them
    // ask for the largest shared-memory carveout: an SM configured for a
    // small one (the default for a kernel with little shared memory) takes no
    // GEMM CTA until it drains.
    if (cudaFuncSetAttribute(gram_reduce_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
        cudaFuncSetAttribute(gram_tc_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
        cudaFuncSetAttribute(norm_tc_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return DORA_ERR_CUDA;
    if (gram_cluster_attrs(gram_cluster_kernel<1>) || gram_cluster_attrs(gram_cluster_kernel<2>) ||
        gram_cluster_attrs(gram_cluster_kernel<4>) || gram_cluster_attrs(gram_cluster_kernel<8>))
      return DORA_ERR_CUDA;
    if (cudaFuncSetAttribute(norm_batched_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem_optin) !=
            cudaSuccess ||
        cudaFuncSetAttribute(gram_batched_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem_optin) !=
            cudaSuccess)
      return DORA_ERR_CUDA;
    if (pair_attrs(linear_pair_kernel<false, false>, d.smem_optin) ||
        pair_attrs(linear_pair_kernel<false, true>, d.smem_optin) ||
        pair_attrs(linear_pair_kernel<true, true>, d.smem_optin) ||
        pair_attrs(linear_i8_pair_kernel, d.smem_optin) || pair_attrs(linear_ckpt8_pair_kernel, d.smem_optin))
      return DORA_ERR_CUDA;
    d.ckpt_bwd_ctas[LanesBf16::kIndex] = ctas_per_sm(compose_bwd_ckpt8_kernel<LanesBf16>, kCkptBwdThreads);
    d.ckpt_bwd_ctas[LanesF32::kIndex] = ctas_per_sm(compose_bwd_ckpt8_kernel<LanesF32>, kCkptBwdThreads);
    d.ckpt_bwd_ctas[LanesF32Any::kIndex] = ctas_per_sm(compose_bwd_ckpt8_kernel<LanesF32Any>, kCkptBwdThreads);
    for (int i8 = 0; i8 < 2; ++i8)
      for (int bn : {16, 32, 64, 128})
        if (cudaFuncSetAttribute(slice_kernel(i8 != 0, bn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSlSmemOne)) != cudaSuccess ||
            cudaFuncSetAttribute(slice_kernel(i8 != 0, bn), cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared) != cudaSuccess)
          return DORA_ERR_CUDA;
    {
      cudaLaunchConfig_t occ{};
      cudaLaunchAttribute cl[1];
      cl[0].id = cudaLaunchAttributeClusterDimension;
      cl[0].val.clusterDim.x = 2;
      cl[0].val.clusterDim.y = 1;
      cl[0].val.clusterDim.z = 1;
      occ.gridDim = dim3(2 * (d.num_sms / 2));
      occ.blockDim = dim3(kLinThreads);
      occ.dynamicSmemBytes = linear_pair_smem(d.smem_optin);
      occ.attrs = cl;
      occ.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&d.pair_clusters, linear_pair_kernel<false, false>, &occ) != cudaSuccess ||
          d.pair_clusters < 1)
        return DORA_ERR_CUDA;
    }
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || fn == nullptr)
        return DORA_ERR_CUDA;
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    d.ready = true;
  }
  *out = &d;
  return DORA_OK;
}

// 2-D bf16 tensor map over a row-major [rows, cols] matrix, 64 x 128 boxes,
// 128-byte swizzle, zero fill outside the matrix.
int make_map(CUtensorMap* map, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows = kBoxRows) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DORA_OK : DORA_ERR_CUDA;
}

// 2-D int8 tensor map over a row-major [rows, cols] matrix, 128 x box_rows
// boxes, 128-byte swizzle, zero fill outside the matrix.
int make_map_i8(CUtensorMap* map, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kI8BK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DORA_OK : DORA_ERR_CUDA;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// One compose backward launch; the bias picks the instantiation.
// Tag of one compose-backward launch for its arrival counters (56 bits, new
// for every call in this process; the start mixes in the clock so that a
// buffer left by another process is unlikely to carry a live tag).
unsigned long long next_bwd_epoch() {
  static std::atomic<unsigned long long> counter{
      static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count()) * 0x9E3779B97F4A7C15ull};
  return counter.fetch_add(1) & ((1ull << 56) - 1);
}

template <typename T, int VEC>
void launch_compose_bwd(dim3 grid, cudaStream_t st, const void* dy, const void* base_out, const void* lora_out,
                        const void* bias, const float* m, const float* n, float s, long long tokens, long long nvec,
                        long long d_out, void* d_base, void* d_lora, float* part, unsigned long long* cnt, float* d_m,
                        long long rows) {
  auto kernel = bias ? compose_bwd_kernel<T, VEC, true> : compose_bwd_kernel<T, VEC, false>;
  note_launch();
  kernel<<<grid, kBwdThreads, 0, st>>>(static_cast<const T*>(dy), static_cast<const T*>(base_out),
                                       static_cast<const T*>(lora_out), static_cast<const T*>(bias), m, n, s, tokens,
                                       nvec, d_out, static_cast<T*>(d_base), static_cast<T*>(d_lora), part, cnt, d_m,
                                       rows, next_bwd_epoch());
}

// ------------------------------------------------------------ norm planning
struct TcPlan {
  int m_tiles, n_chunks, chunk_n, kb_main, kb_ext, kb_total;
  long long units;
  size_t off_gs, off_part, off_cnt, total;
};

TcPlan plan_tc(int64_t d_out, int64_t d_in, int64_t r) {
  TcPlan p{};
  p.m_tiles = static_cast<int>(cdiv(d_out, kBM));
  p.n_chunks = static_cast<int>(cdiv(r, kMaxChunkN));
  p.chunk_n = static_cast<int>(align_up(static_cast<size_t>(cdiv(r, p.n_chunks)), 16));
  p.kb_main = static_cast<int>(cdiv(d_in, kBK));
  p.kb_ext = static_cast<int>(cdiv(r, kBK));
  p.kb_total = p.kb_main + p.kb_ext;
  p.units = static_cast<long long>(p.m_tiles) * p.n_chunks * p.kb_total;
  size_t off = 0;
  p.off_gs = off;
  off = align_up(off + static_cast<size_t>(r) * r * 2, 1024);
  // (the Gram clusters keep their K-split partials in shared memory)
  p.off_part = off;
  off = align_up(off + static_cast<size_t>(kMaxGrid + p.m_tiles * p.n_chunks) * kBM * 4, 256);
  p.off_cnt = off;
  off = align_up(off + static_cast<size_t>(p.m_tiles) * 4, 256);
  p.total = off;
  return p;
}

size_t f32_norm_ws(int64_t r) { return align_up(static_cast<size_t>(r) * r * 4, 256) + 256; }

int launch_error() { return cudaGetLastError() == cudaSuccess ? DORA_OK : DORA_ERR_CUDA; }

// Launches a kernel that starts under the launch before it and waits itself for
// that launch's end (programmatic dependent launch).
template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? DORA_OK : DORA_ERR_CUDA;
}

// Resident CTAs per SM of a kernel at the given block size (at least 1).
template <typename K>
int ctas_per_sm(K kernel, int threads) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 1;
  }
  return n;
}

// Row chunks of the compose backward for `strips` column strips (at most
// k_max, at least one): as many as one wave of `slots` resident CTAs holds
// while that leaves each CTA at most kBwdWaveRows rows, else about two waves.
// Measured at d_out = 8192: one wave of longer CTAs beats two waves of
// shorter ones up to 8192 tokens (110.6 against 112.6 us; 57.3 against
// 59.4 us at 4096), since each CTA pays a ramp-up of its loads and a
// partial-sum write at its end; two waves win from 16384 tokens on (215.0
// against 218.9 us; 848.8 against 869.4 us at 65536).
constexpr long long kBwdWaveRows = 2048;
long long bwd_chunks(long long strips, long long slots, long long tokens, long long k_max) {
  long long k = std::max<long long>(1, slots / strips);
  if (cdiv(tokens, k) > kBwdWaveRows) k = std::max<long long>(1, 2 * slots / strips);
  return std::max<long long>(1, std::min<long long>(k, k_max));
}

int norm_bf16(const void* W, const void* A, const void* B, int64_t d_out, int64_t d_in, int64_t r, float s,
              float* n_out, void* ws, cudaStream_t st, DeviceInfo* dev, bool squared) {
  const TcPlan p = plan_tc(d_out, d_in, r);
  if (p.units > (1ll << 30)) return DORA_ERR_UNSUPPORTED;  // unit indices are 32-bit in the kernel
  uint8_t* w = static_cast<uint8_t*>(ws);
  __nv_bfloat16* Gs = reinterpret_cast<__nv_bfloat16*>(w + p.off_gs);
  float* part = reinterpret_cast<float*>(w + p.off_part);
  int* cnt = reinterpret_cast<int*>(w + p.off_cnt);

  CUtensorMap tmW, tmA, tmB, tmG;
  if (make_map(&tmW, W, d_out, d_in) || make_map(&tmA, A, r, d_in) || make_map(&tmB, B, d_out, r) ||
      make_map(&tmG, Gs, r, r))
    return DORA_ERR_CUDA;

  // 1) G' = (s/2) A A^T: one cluster of `splits` CTAs per tile on or above
  // the diagonal, each CTA a K split, summed inside the cluster; the launch
  // also zeroes the GEMM's tile counters.  2) The persistent GEMM behind it
  // with programmatic dependent launch: its CTAs start on the SMs the Gram
  // clusters leave free, meet G' only at the ends of their ranges and wait
  // for the Gram launch only there.
  const int nt = static_cast<int>(cdiv(r, kBoxRows));
  const int up_tiles = nt * (nt + 1) / 2;
  // as many K splits as a cluster holds (8), while each keeps at least
  // kGramMinBlocks K blocks and the clusters take at most a third of the
  // SMs: the Gram latency then stays well inside the GEMM's, small
  // problems included
  int splits = 1;
  while (splits < 8 && 2 * splits * kGramMinBlocks <= p.kb_main && up_tiles * 2 * splits <= std::max(1, dev->num_sms / 3))
    splits *= 2;
  {
    GramClusterArgs gca{};
    gca.r = static_cast<int>(r);
    gca.kb_main = p.kb_main;
    gca.nt = nt;
    gca.half_s = 0.5f * s;
    gca.Gs = Gs;
    gca.wait_limit = kWaitLimitCycles;
    gca.status = dev->status;
    gca.zero_cnt = cnt;
    gca.n_zero = p.m_tiles;
    cudaLaunchAttribute gat[1];
    gat[0].id = cudaLaunchAttributeClusterDimension;
    gat[0].val.clusterDim.x = static_cast<unsigned>(splits);
    gat[0].val.clusterDim.y = 1;
    gat[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t gcfg{};
    gcfg.stream = st;
    gcfg.attrs = gat;
    gcfg.numAttrs = 1;
    gcfg.gridDim = dim3(static_cast<unsigned>(up_tiles * splits));
    gcfg.blockDim = dim3(kGcThreads);
    gcfg.dynamicSmemBytes = kGcSmem;
    cudaError_t e = cudaSuccess;
    note_launch();
    switch (splits) {
      case 1: e = cudaLaunchKernelEx(&gcfg, gram_cluster_kernel<1>, tmA, gca); break;
      case 2: e = cudaLaunchKernelEx(&gcfg, gram_cluster_kernel<2>, tmA, gca); break;
      case 4: e = cudaLaunchKernelEx(&gcfg, gram_cluster_kernel<4>, tmA, gca); break;
      default: e = cudaLaunchKernelEx(&gcfg, gram_cluster_kernel<8>, tmA, gca); break;
    }
    if (e != cudaSuccess) return DORA_ERR_CUDA;
  }

  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;

  NormArgs na{};
  na.d_out = static_cast<int>(d_out);
  na.d_in = static_cast<int>(d_in);
  na.r = static_cast<int>(r);
  na.m_tiles = p.m_tiles;
  na.n_chunks = p.n_chunks;
  na.chunk_n = p.chunk_n;
  na.kb_main = p.kb_main;
  na.kb_total = p.kb_total;
  na.units = p.units;
  const int grid = static_cast<int>(std::min<long long>({static_cast<long long>(dev->num_sms), p.units, kMaxGrid}));
  const size_t smem_fixed = kNormTcSmemFixed + static_cast<size_t>(grid + 1) * 4;  // + the range-start table
  na.stage_bytes = static_cast<uint32_t>(kBoxBytes * (1 + cdiv(p.chunk_n, kBoxRows)));
  na.stages = static_cast<int>(std::min<size_t>(kMaxStages, (dev->smem_optin - smem_fixed) / (na.stage_bytes + 16)));
  if (na.stages < 2) return DORA_ERR_UNSUPPORTED;
  // a power of two of at least 64 columns: the epilogue reads V 64 columns at a time
  uint32_t cols = 64;
  while (cols < static_cast<uint32_t>(p.chunk_n)) cols <<= 1;
  na.tmem_cols = cols;
  na.two_s = 2.0f * s;
  na.wait_limit = kWaitLimitCycles;
  na.partials = part;
  na.counters = cnt;
  na.n_out = n_out;
  na.status = dev->status;
  na.squared = squared ? 1 : 0;
  {
    // The Gram CTAs hold one SM each (their shared memory): that many CTAs of
    // the GEMM start late and get that much less, so that all end together.
    // Start delay and GEMM unit time from traces of these kernels on B200
    // (8192 x 8192, r = 64 and 384): a Gram CTA takes about 3 us plus
    // 0.43 us per K block of its split, plus about 5 us to sum and mirror
    // off-diagonal tiles; a GEMM unit about 0.18 us plus 0.01 us per KB of its
    // ring stage.  A late CTA that ends early costs the grid a little; one
    // that ends late costs the whole gap, so the delay is taken 10% long,
    // 25% for Gram phases past 20 us, which the linear model underestimates
    // (r = 768 at 8192 x 8192: 111.7 against 115.7 us with 10%).
    const int gram_sms = std::min(dev->num_sms, up_tiles * splits);
    const int late = grid > gram_sms ? gram_sms : 0;
    const double gram_us = 3.0 + 0.43 * static_cast<double>(cdiv(p.kb_main, splits)) + (nt > 1 ? 5.0 : 1.0);
    const double unit_us = 0.18 + 0.01 * (static_cast<double>(na.stage_bytes) / 1024.0);
    const double delay = (gram_us > 20.0 ? 1.25 : 1.1) * gram_us / unit_us;
    const double f = (static_cast<double>(p.units) + late * delay) / grid;
    na.early = grid - late;
    na.w_early = std::max<long long>(1, std::llround(16.0 * f));
    na.w_late = late > 0 ? std::max<long long>(0, std::llround(16.0 * (f - delay))) : na.w_early;
  }
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kNormTcThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(na.stages) * (na.stage_bytes + 16) + smem_fixed;
  note_launch();
  if (cudaLaunchKernelEx(&cfg, norm_tc_kernel, tmW, tmA, tmB, tmG, na) != cudaSuccess) return DORA_ERR_CUDA;
  return launch_error();
}

// Argument checks of one factored norm, workspace aside.
int norm_arg_status(const void* W, const void* A, const void* B, int64_t d_out, int64_t d_in, int64_t r, dora_dtype dt,
                    const float* n_out) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (d_out < 0 || d_in < 0 || r < 0) return DORA_ERR_INVALID_ARG;
  if (d_out > INT32_MAX / 2 || d_in > INT32_MAX / 2 || r > kMaxRank) return DORA_ERR_UNSUPPORTED;
  if (d_out == 0) return DORA_OK;
  if (!n_out || (d_in > 0 && !W) || (r > 0 && d_in > 0 && (!A || !B))) return DORA_ERR_INVALID_ARG;
  if (!aligned(n_out, 4)) return DORA_ERR_UNSUPPORTED;
  if (dt == DORA_BF16) {
    if (d_in > 0 && (d_in % 8 != 0 || r % 16 != 0)) return DORA_ERR_UNSUPPORTED;
    if (!aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16)) return DORA_ERR_UNSUPPORTED;
  } else {
    if (!aligned(W, 4) || !aligned(A, 4) || !aligned(B, 4)) return DORA_ERR_UNSUPPORTED;
  }
  return DORA_OK;
}

// ------------------------------------------------------- batched norms
// Modules that share the two batched launches: bf16, 16 <= r <= 512 (one
// TMEM chunk), something to compute.
bool batchable(const dora_norm_problem& q, dora_dtype dt) {
  return dt == DORA_BF16 && q.d_out > 0 && q.d_in > 0 && q.r >= 16 && q.r <= 512 && q.r % 16 == 0;
}

struct BatchLayout {
  std::vector<int> batched, single;  // problem indices on each path
  std::vector<size_t> off_gs;        // per batched problem: its G' in the workspace
  size_t off_items = 0, off_gitems = 0, off_single = 0, single_bytes = 0, total = 0;
  int n_items = 0, n_gitems = 0;
  uint32_t stage_bytes = 0;
};

int batch_layout(const dora_norm_problem* q, int count, dora_dtype dt, BatchLayout* L) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (count < 0 || (count > 0 && !q)) return DORA_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (q[i].d_out < 0 || q[i].d_in < 0 || q[i].r < 0) return DORA_ERR_INVALID_ARG;
    if (batchable(q[i], dt)) {
      L->batched.push_back(i);
      L->n_items += static_cast<int>(cdiv(q[i].d_out, kBM));
      const int nt = static_cast<int>(cdiv(q[i].r, kBoxRows));
      L->n_gitems += nt * nt;
      L->stage_bytes = std::max<uint32_t>(L->stage_bytes, kBoxBytes * (1 + nt));
    } else {
      L->single.push_back(i);
      L->single_bytes = std::max(L->single_bytes, dora_factored_norm_workspace_size(q[i].d_out, q[i].d_in, q[i].r, dt));
    }
  }
  size_t off = align_up(L->batched.size() * sizeof(BatchDesc), 256);
  L->off_items = off;
  off = align_up(off + static_cast<size_t>(L->n_items) * sizeof(BatchItem), 256);
  L->off_gitems = off;
  off = align_up(off + static_cast<size_t>(L->n_gitems) * sizeof(BatchItem), 256);
  for (int i : L->batched) {
    L->off_gs.push_back(off);
    off = align_up(off + static_cast<size_t>(q[i].r) * q[i].r * 2, 256);
  }
  L->off_single = off;
  L->total = off + L->single_bytes;
  return DORA_OK;
}

int norm_batched(const dora_norm_problem* q, const BatchLayout& L, uint8_t* ws, cudaStream_t st, DeviceInfo* dev) {
  const size_t nb = L.batched.size();
  // the descriptor table and both work lists, built here and copied in one go
  std::vector<uint8_t> host(L.off_gs.empty() ? L.off_gitems : L.off_gs[0]);
  BatchDesc* descs = reinterpret_cast<BatchDesc*>(host.data());
  BatchItem* items = reinterpret_cast<BatchItem*>(host.data() + L.off_items);
  BatchItem* gitems = reinterpret_cast<BatchItem*>(host.data() + L.off_gitems);
  int ni = 0, ng = 0;
  for (size_t j = 0; j < nb; ++j) {
    const dora_norm_problem& p = q[L.batched[j]];
    BatchDesc& d = descs[j];
    std::memset(&d, 0, sizeof(d));
    __nv_bfloat16* gs = reinterpret_cast<__nv_bfloat16*>(ws + L.off_gs[j]);
    if (make_map(&d.tmW, p.W, p.d_out, p.d_in) || make_map(&d.tmA, p.A, p.r, p.d_in) ||
        make_map(&d.tmB, p.B, p.d_out, p.r) || make_map(&d.tmG, gs, p.r, p.r))
      return DORA_ERR_CUDA;
    d.n_out = p.n_out;
    d.gs = gs;
    d.d_out = static_cast<int>(p.d_out);
    d.d_in = static_cast<int>(p.d_in);
    d.r = static_cast<int>(p.r);
    d.kb_main = static_cast<int>(cdiv(p.d_in, kBK));
    d.kb_total = d.kb_main + static_cast<int>(cdiv(p.r, kBK));
    d.two_s = 2.0f * p.s;
    d.half_s = 0.5f * p.s;
    for (int t = 0; t < cdiv(p.d_out, kBM); ++t) items[ni++] = BatchItem{static_cast<int>(j), t};
    const int nt = static_cast<int>(cdiv(p.r, kBoxRows));
    for (int t = 0; t < nt * nt; ++t) gitems[ng++] = BatchItem{static_cast<int>(j), t};
  }
  // longest items first, dealt round-robin over the persistent grid
  auto cost = [&](const BatchItem& it) {
    const BatchDesc& d = descs[it.prob];
    return static_cast<long long>(d.kb_total) * (1 + cdiv(d.r, kBoxRows));
  };
  std::stable_sort(items, items + ni, [&](const BatchItem& x, const BatchItem& y) { return cost(x) > cost(y); });
  if (cudaMemcpyAsync(ws, host.data(), host.size(), cudaMemcpyHostToDevice, st) != cudaSuccess) return DORA_ERR_CUDA;

  const BatchDesc* d_descs = reinterpret_cast<const BatchDesc*>(ws);
  const size_t gram_smem = kGramStages * kGramStageBytes + (2 * kGramStages + 1) * 8 + 16 + 1024;
  note_launch();
  gram_batched_kernel<<<ng, kNormThreads, gram_smem, st>>>(d_descs, reinterpret_cast<const BatchItem*>(ws + L.off_gitems),
                                                          kWaitLimitCycles, dev->status);
  if (launch_error()) return DORA_ERR_CUDA;

  BatchNormArgs a{};
  a.n_items = ni;
  a.stage_bytes = L.stage_bytes;
  const size_t fixed = 1024 + 64 + 16;
  a.stages = static_cast<int>(std::min<size_t>(kMaxStages, (dev->smem_optin - fixed) / (a.stage_bytes + 16)));
  if (a.stages < 2) return DORA_ERR_UNSUPPORTED;
  a.wait_limit = kWaitLimitCycles;
  a.status = dev->status;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>({static_cast<long long>(dev->num_sms), ni, kMaxGrid})));
  cfg.blockDim = dim3(kNormThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.stages) * a.stage_bytes + (2 * a.stages + 3) * 8 + 16 + 1024;
  note_launch();
  if (cudaLaunchKernelEx(&cfg, norm_batched_kernel, d_descs, reinterpret_cast<const BatchItem*>(ws + L.off_items), a) !=
      cudaSuccess)
    return DORA_ERR_CUDA;
  return launch_error();
}

}  // namespace
}  // namespace dora

using namespace dora;

namespace dora {
namespace {
// The factored norm, n = sqrt(max(n^2, 0)) or, with `squared`, n^2 as summed.
int factored_norm(const void* W, const void* A, const void* B, int64_t d_out, int64_t d_in, int64_t r, float s,
                  dora_dtype dt, float* n_out, void* workspace, size_t workspace_bytes, void* stream, bool squared);
}  // namespace
}  // namespace dora

extern "C" {

const char* dora_status_string(int status) {
  switch (status) {
    case DORA_OK: return "DORA_OK";
    case DORA_ERR_INVALID_ARG: return "DORA_ERR_INVALID_ARG: invalid argument";
    case DORA_ERR_UNSUPPORTED: return "DORA_ERR_UNSUPPORTED: shape, alignment or dtype not supported";
    case DORA_ERR_WORKSPACE: return "DORA_ERR_WORKSPACE: workspace missing or too small";
    case DORA_ERR_CUDA: return "DORA_ERR_CUDA: a CUDA runtime call failed";
    case DORA_ERR_TIMEOUT: return "DORA_ERR_TIMEOUT: a bounded device-side wait gave up";
    default: return "unknown dora status";
  }
}

size_t dora_factored_norm_workspace_size(int64_t d_out, int64_t d_in, int64_t r, dora_dtype dt) {
  if (d_out < 0 || d_in < 0 || r < 0) return 0;
  if (dt == DORA_F32) return f32_norm_ws(r);
  if (dt != DORA_BF16) return 0;
  if (d_out == 0 || d_in == 0 || r == 0) return 256;
  return plan_tc(d_out, d_in, r).total;
}

int dora_factored_norm(const void* W, const void* A, const void* B, int64_t d_out, int64_t d_in, int64_t r, float s,
                       dora_dtype dt, float* n_out, void* workspace, size_t workspace_bytes, void* stream) {
  return factored_norm(W, A, B, d_out, d_in, r, s, dt, n_out, workspace, workspace_bytes, stream, false);
}

int dora_factored_norm_sq(const void* W, const void* A, const void* B, int64_t d_out, int64_t d_in, int64_t r,
                          float s, dora_dtype dt, float* n2_out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  return factored_norm(W, A, B, d_out, d_in, r, s, dt, n2_out, workspace, workspace_bytes, stream, true);
}

int dora_norm_finish(float* n, int64_t d_out, void* stream) {
  if (d_out < 0) return DORA_ERR_INVALID_ARG;
  if (d_out == 0) return DORA_OK;
  if (!n) return DORA_ERR_INVALID_ARG;
  if (!aligned(n, 4)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  note_launch();
  norm_finish_kernel<<<static_cast<unsigned>(cdiv(d_out, 256)), 256, 0, static_cast<cudaStream_t>(stream)>>>(n, d_out);
  return launch_error();
}

}  // extern "C"

namespace dora {
namespace {
int factored_norm(const void* W, const void* A, const void* B, int64_t d_out, int64_t d_in, int64_t r, float s,
                  dora_dtype dt, float* n_out, void* workspace, size_t workspace_bytes, void* stream, bool squared) {
  const int arg = norm_arg_status(W, A, B, d_out, d_in, r, dt, n_out);
  if (arg != DORA_OK || d_out == 0) return arg;
  const size_t need = dora_factored_norm_workspace_size(d_out, d_in, r, dt);
  const bool trivial = (d_in == 0);
  if (!trivial && (!workspace || workspace_bytes < need)) return DORA_ERR_WORKSPACE;
  if (!trivial && !aligned(workspace, 256)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (trivial) {
    return cudaMemsetAsync(n_out, 0, static_cast<size_t>(d_out) * 4, st) == cudaSuccess ? DORA_OK : DORA_ERR_CUDA;
  }
  if (r == 0) {
    const int blocks = static_cast<int>(cdiv(d_out, 8));
    note_launch();
    if (dt == DORA_BF16)
      rownorm_kernel<__nv_bfloat16><<<blocks, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(W), static_cast<int>(d_out),
                                                            static_cast<int>(d_in), n_out, squared ? 1 : 0);
    else
      rownorm_kernel<float><<<blocks, 256, 0, st>>>(static_cast<const float*>(W), static_cast<int>(d_out),
                                                    static_cast<int>(d_in), n_out, squared ? 1 : 0);
    return launch_error();
  }
  if (dt == DORA_BF16) return norm_bf16(W, A, B, d_out, d_in, r, s, n_out, workspace, st, dev, squared);
  float* G = static_cast<float*>(workspace);
  const long long pairs = r * (r + 1) / 2;
  const int gblocks = static_cast<int>(std::min<long long>(cdiv(pairs, 8), 8LL * dev->num_sms));
  note_launch();
  gram_f32_kernel<<<gblocks, 256, 0, st>>>(static_cast<const float*>(A), static_cast<int>(r), static_cast<int>(d_in), G);
  if (launch_error()) return DORA_ERR_CUDA;
  note_launch();
  norm_f32_kernel<<<static_cast<unsigned>(d_out), 256, 0, st>>>(
      static_cast<const float*>(W), static_cast<const float*>(A), static_cast<const float*>(B), G,
      static_cast<int>(d_out), static_cast<int>(d_in), static_cast<int>(r), s, n_out, squared ? 1 : 0);
  return launch_error();
}
}  // namespace
}  // namespace dora

extern "C" {

int dora_compose_fwd(const void* base_out, const void* lora_out, const float* m, const float* n, float s,
                     int64_t tokens, int64_t d_out, dora_dtype dt, void* y, void* stream) {
  return dora_compose_fwd_bias(base_out, lora_out, nullptr, m, n, s, tokens, d_out, dt, y, stream);
}

int dora_compose_fwd_bias(const void* base_out, const void* lora_out, const void* bias, const float* m,
                          const float* n, float s, int64_t tokens, int64_t d_out, dora_dtype dt, void* y,
                          void* stream) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (tokens < 0 || d_out < 0) return DORA_ERR_INVALID_ARG;
  if (tokens == 0 || d_out == 0) return DORA_OK;
  if (!base_out || !lora_out || !m || !n || !y) return DORA_ERR_INVALID_ARG;
  const int vec_bf16 = 8;
  int vec = 1;
  if (dt == DORA_BF16) {
    if (d_out % vec_bf16 != 0) return DORA_ERR_UNSUPPORTED;
    if (!aligned(base_out, 16) || !aligned(lora_out, 16) || !aligned(y, 16)) return DORA_ERR_UNSUPPORTED;
    vec = vec_bf16;
  } else {
    if (!aligned(base_out, 4) || !aligned(lora_out, 4) || !aligned(y, 4)) return DORA_ERR_UNSUPPORTED;
    vec = (d_out % 4 == 0 && aligned(base_out, 16) && aligned(lora_out, 16) && aligned(y, 16)) ? 4 : 1;
  }
  if (!aligned(m, 4) || !aligned(n, 4) || !aligned(bias, dt == DORA_BF16 ? 16 : 4)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long nvec = d_out / vec;
  const int threads = static_cast<int>(std::min<long long>(256, align_up(static_cast<size_t>(nvec), 32)));
  const long long gx = cdiv(nvec, threads);
  if (gx > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  // Several short waves of small CTAs stream better than one wave of long
  // ones here: about 8 CTAs per SM in total, whatever the residency.
  const long long gy = std::max<long long>(1, std::min<long long>({8LL * dev->num_sms / gx, tokens, 65535}));
  const long long rows = cdiv(tokens, gy);
  const long long gy2 = cdiv(tokens, rows);
  dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy2));
  note_launch();
  if (dt == DORA_BF16)
    compose_fwd_kernel<__nv_bfloat16, 8><<<grid, threads, 0, st>>>(
        static_cast<const __nv_bfloat16*>(base_out), static_cast<const __nv_bfloat16*>(lora_out),
        static_cast<const __nv_bfloat16*>(bias), m, n, s, tokens, nvec, d_out, static_cast<__nv_bfloat16*>(y), rows);
  else if (vec == 4)
    compose_fwd_kernel<float, 4><<<grid, threads, 0, st>>>(static_cast<const float*>(base_out),
                                                           static_cast<const float*>(lora_out),
                                                           static_cast<const float*>(bias), m, n, s, tokens, nvec,
                                                           d_out, static_cast<float*>(y), rows);
  else
    compose_fwd_kernel<float, 1><<<grid, threads, 0, st>>>(static_cast<const float*>(base_out),
                                                           static_cast<const float*>(lora_out),
                                                           static_cast<const float*>(bias), m, n, s, tokens, nvec,
                                                           d_out, static_cast<float*>(y), rows);
  return launch_error();
}

size_t dora_compose_bwd_workspace_size(int64_t tokens, int64_t d_out) {
  if (tokens < 0 || d_out < 0) return 0;
  const size_t strips = static_cast<size_t>(cdiv(std::max<int64_t>(d_out, 1), dora::kBwdVecs));
  return align_up(strips * 8, 256) + align_up(static_cast<size_t>(kMaxBwdChunks) * std::max<int64_t>(d_out, 1) * 4, 256);
}

int dora_compose_bwd(const void* dy, const void* base_out, const void* lora_out, const float* m, const float* n,
                     float s, int64_t tokens, int64_t d_out, dora_dtype dt, void* d_base, void* d_lora, float* d_m,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return dora_compose_bwd_bias(dy, base_out, lora_out, nullptr, m, n, s, tokens, d_out, dt, d_base, d_lora, d_m,
                               workspace, workspace_bytes, stream);
}

int dora_compose_bwd_bias(const void* dy, const void* base_out, const void* lora_out, const void* bias,
                          const float* m, const float* n, float s, int64_t tokens, int64_t d_out, dora_dtype dt,
                          void* d_base, void* d_lora, float* d_m, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (tokens < 0 || d_out < 0) return DORA_ERR_INVALID_ARG;
  if (d_out == 0) return DORA_OK;
  if (!m || !n || !d_m) return DORA_ERR_INVALID_ARG;
  if (tokens > 0 && (!dy || !base_out || !lora_out || !d_base || !d_lora)) return DORA_ERR_INVALID_ARG;
  int vec = 1;
  if (dt == DORA_BF16) {
    if (d_out % 8 != 0) return DORA_ERR_UNSUPPORTED;
    if (tokens > 0 && (!aligned(dy, 16) || !aligned(base_out, 16) || !aligned(lora_out, 16) ||
                       !aligned(d_base, 16) || !aligned(d_lora, 16)))
      return DORA_ERR_UNSUPPORTED;
    vec = 8;
  } else {
    const bool a16 = aligned(dy, 16) && aligned(base_out, 16) && aligned(lora_out, 16) && aligned(d_base, 16) &&
                     aligned(d_lora, 16) && aligned(bias, 16);
    if (!aligned(dy, 4) || !aligned(base_out, 4) || !aligned(lora_out, 4) || !aligned(d_base, 4) ||
        !aligned(d_lora, 4))
      return DORA_ERR_UNSUPPORTED;
    vec = (d_out % 4 == 0 && a16) ? 4 : 1;
  }
  if (!aligned(m, 4) || !aligned(n, 4) || !aligned(d_m, 4) || !aligned(bias, dt == DORA_BF16 ? 16 : 4))
    return DORA_ERR_UNSUPPORTED;
  const size_t need = dora_compose_bwd_workspace_size(tokens, d_out);
  if (!workspace || workspace_bytes < need) return DORA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens == 0) return cudaMemsetAsync(d_m, 0, static_cast<size_t>(d_out) * 4, st) == cudaSuccess ? DORA_OK : DORA_ERR_CUDA;

  const long long nvec = d_out / vec;
  const long long strips = cdiv(nvec, kBwdVecs);
  if (strips > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  int occ = 1;
  if (dt == DORA_BF16)
    occ = ctas_per_sm(compose_bwd_kernel<__nv_bfloat16, 8, false>, kBwdThreads);
  else if (vec == 4)
    occ = ctas_per_sm(compose_bwd_kernel<float, 4, false>, kBwdThreads);
  else
    occ = ctas_per_sm(compose_bwd_kernel<float, 1, false>, kBwdThreads);
  const long long chunks = bwd_chunks(strips, static_cast<long long>(dev->num_sms) * occ, tokens,
                                      std::min<long long>(kMaxBwdChunks, cdiv(tokens, kBwdSlots)));
  const long long rows = cdiv(tokens, chunks);
  const long long chunks2 = cdiv(tokens, rows);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  unsigned long long* cnt = reinterpret_cast<unsigned long long*>(w);  // tagged: no clearing needed
  const size_t strips_all = static_cast<size_t>(cdiv(d_out, kBwdVecs));
  float* part = reinterpret_cast<float*>(w + align_up(strips_all * 8, 256));
  dim3 grid(static_cast<unsigned>(strips), static_cast<unsigned>(chunks2));
  if (dt == DORA_BF16)
    launch_compose_bwd<__nv_bfloat16, 8>(grid, st, dy, base_out, lora_out, bias, m, n, s, tokens, nvec, d_out, d_base,
                                         d_lora, part, cnt, d_m, rows);
  else if (vec == 4)
    launch_compose_bwd<float, 4>(grid, st, dy, base_out, lora_out, bias, m, n, s, tokens, nvec, d_out, d_base, d_lora,
                                part, cnt, d_m, rows);
  else
    launch_compose_bwd<float, 1>(grid, st, dy, base_out, lora_out, bias, m, n, s, tokens, nvec, d_out, d_base, d_lora,
                                part, cnt, d_m, rows);
  return launch_error();
}

size_t dora_factored_norm_batched_workspace_size(const dora_norm_problem* problems, int count, dora_dtype dt) {
  BatchLayout L;
  if (batch_layout(problems, count, dt, &L) != DORA_OK) return 0;
  return std::max<size_t>(L.total, 256);
}

int dora_factored_norm_batched(const dora_norm_problem* problems, int count, dora_dtype dt, void* workspace,
                               size_t workspace_bytes, void* stream) {
  BatchLayout L;
  const int lay = batch_layout(problems, count, dt, &L);
  if (lay != DORA_OK) return lay;
  // every module's arguments are checked before anything is launched
  for (int i = 0; i < count; ++i) {
    const dora_norm_problem& q = problems[i];
    const int arg = norm_arg_status(q.W, q.A, q.B, q.d_out, q.d_in, q.r, dt, q.n_out);
    if (arg != DORA_OK) return arg;
  }
  if (count == 0) return DORA_OK;
  if (!workspace || workspace_bytes < L.total) return DORA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (!L.batched.empty()) {
    const int rc = norm_batched(problems, L, ws, static_cast<cudaStream_t>(stream), dev);
    if (rc != DORA_OK) return rc;
  }
  for (int i : L.single) {
    const dora_norm_problem& q = problems[i];
    const int rc = dora_factored_norm(q.W, q.A, q.B, q.d_out, q.d_in, q.r, q.s, dt, q.n_out, ws + L.off_single,
                                      L.single_bytes, stream);
    if (rc != DORA_OK) return rc;
  }
  return DORA_OK;
}

int dora_device_status(void* stream) {
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return DORA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return DORA_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  }
  return v;
}

int dora_selftest_timeout(int64_t limit_cycles, void* stream) {
  if (limit_cycles <= 0 || limit_cycles > kWaitLimitCycles) return DORA_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  note_launch();
  timeout_probe_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(limit_cycles, dev->status);
  return launch_error();
}

uint64_t dora_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int dora_num_sms(void) {
  int n = 0;
  if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
    cudaGetLastError();
    return 0;
  }
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return 0;
  return dev->num_sms;
}


size_t dora_fused_linear_fwd_workspace_size(int64_t tokens, int64_t r) {
  if (tokens < 0 || r < 0) return 0;
  return std::max<size_t>(256, align_up(static_cast<size_t>(tokens) * static_cast<size_t>(r) * 2, 256));
}

}  // extern "C"

namespace dora {
namespace {

// Launch configuration of a CTA-pair kernel over `tiles` output tiles: as many
// pairs as are resident at once.  `after`: it starts under the launch before it
// (programmatic dependent launch) and waits itself for what it reads of that.
cudaLaunchConfig_t pair_config(cudaLaunchAttribute (&attrs)[2], int threads, size_t smem, long long tiles, bool after,
                               const DeviceInfo* dev, cudaStream_t st) {
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = 2;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = after ? 2 : 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<long long>(dev->pair_clusters, tiles)));
  return cfg;
}

// P = bf16(s * x A^T) into `P` [tokens, r]; ordered after everything before it
// on the stream.  tmA has boxes of pick_bn(r) / 2 rows.
int launch_p(const CUtensorMap& tmX, const CUtensorMap& tmA, __nv_bfloat16* P, float s, int64_t tokens, int64_t d_in,
             int64_t r, const DeviceInfo* dev, cudaStream_t st) {
  LinearArgs pa{};
  pa.M = static_cast<int>(tokens);
  pa.N = static_cast<int>(r);
  pa.kb_main = pa.kb_total = static_cast<int>(cdiv(d_in, kLinBK));
  pa.tiles_m = static_cast<int>(cdiv(tokens, kPairBM));
  pa.bn = pick_bn(r);
  pa.tiles_n = static_cast<int>(cdiv(r, pa.bn));
  pa.stages = linear_pair_stages(dev->smem_optin);
  pa.alpha = s;
  pa.out = P;
  pa.ldo = r;
  pa.wait_limit = kWaitLimitCycles;
  pa.status = dev->status;
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = pair_config(attrs, kLinThreads, linear_pair_smem(dev->smem_optin),
                                       static_cast<long long>(pa.tiles_m) * pa.tiles_n, false, dev, st);
  note_launch();
  return cudaLaunchKernelEx(&cfg, linear_pair_kernel<false, false>, tmX, tmA, tmX, tmA, pa) == cudaSuccess
             ? DORA_OK
             : DORA_ERR_CUDA;
}

// Up to this many tokens the int8 linear runs on slices of the weight (8192 x
// 8192 without an adapter: 65 tokens 19.5 us, 23.9 on pairs; 128 tokens 21.1 and
// 24.2; 129 tokens 32.0 on two token tiles of slices, 24.4 on pairs; 4096 x 4096:
// 9.5 and 12.9, 11.4 and 13.1, 12.9 and 13.3).  The rule looks at the tokens
// alone: beside an adapter of rank 384 the pairs are ahead from 65 tokens on
// (8192 x 8192: 35.6 us on slices, 31.1 on pairs; 128 tokens 39.9 and 31.9).
constexpr int64_t kSliceTokens = 128;

// Up to this many tokens the down projection runs on down_tokens_kernel (the
// whole call; 8192 x 8192 at rank 384: one token 19.7 us, 21.9 on slices; four
// 21.2 and 22.1; five 23.8 and 22.3; 4096 x 4096 at rank 64: 8.7 and 11.7, 10.2
// and 11.8).  Beside a wide product it loses from two tokens on (5120 -> 27648 at
// rank 384: one token 32.0 and 32.7, two 33.3 and 32.8, four 36.2 and 33.2).
constexpr int64_t kDownTokens = 4;

// Token tile of the slice kernels.
int slice_bn(int64_t tokens) { return tokens <= 16 ? 16 : (tokens <= 32 ? 32 : (tokens <= 64 ? 64 : 128)); }

// One slice launch over `a`: K split over as many CTAs of a cluster as keep
// the grid within `room` CTAs (0: what is resident at once), with eight K blocks
// each at least: 64 tokens through 4096 x 2048 took 18.0 us in eighths of four
// blocks, 14.2 in quarters.  A product of 64 tokens and more takes at most four:
// its join reads every split's tile (8192 x 4096: 21.6 us, 24.6 in eighths).
int launch_slice(bool i8, const CUtensorMap& tmW, const CUtensorMap& tmX, const CUtensorMap& tmB,
                 const CUtensorMap& tmP, SliceArgs a, bool after, long long room, const DeviceInfo* dev,
                 cudaStream_t st) {
  const int bn = slice_bn(a.tokens);
  const long long row_tiles = cdiv(a.rows, kLinBM), tok_tiles = cdiv(a.tokens, bn);
  if (row_tiles * tok_tiles > INT32_MAX / 8) return DORA_ERR_UNSUPPORTED;
  const bool one = (i8 && bn > 64) || room > 0;  // a CTA an SM
  if (room == 0) room = (one ? 1LL : 2LL) * dev->num_sms;
  int splits = 1;
  while (splits < (i8 && bn >= 64 ? 4 : 8) && 16 * splits <= a.kb_main && 2 * row_tiles * tok_tiles * splits <= room) splits *= 2;
  const size_t smem = one ? kSlSmemOne : kSlSmemTwo;
  a.stages = static_cast<int>(std::min<size_t>(kSlMaxStages, (smem - kSlFixed) / slice_stage_bytes(bn)));
  a.wait_limit = kWaitLimitCycles;
  a.status = dev->status;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = after ? 2 : 1;
  cfg.blockDim = dim3(kSlThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(static_cast<unsigned>(row_tiles * tok_tiles * splits));
  note_launch();
  return cudaLaunchKernelEx(&cfg, slice_kernel(i8, bn), tmW, tmX, tmB, tmP, a) == cudaSuccess ? DORA_OK
                                                                                               : DORA_ERR_CUDA;
}

// P = bf16(s * x A^T), and what the rounding leaves unless P_lo is null, on
// slices: few rank rows make few large tiles, so K is split instead.  The
// product behind it starts at once and takes the SMs that this grid leaves, but
// its pairs share none with a CTA of this one: where that product's `pairs`
// leave SMs idle (one wave), P keeps to those if its tiles fit there.  Measured
// with P beside the product and with P on more SMs: 1000 tokens through 4096 x
// 4096 at rank 64, int8 25.6 and 28.9 us, with a checkpoint 39.6 and 46.5; 512
// through 8192 x 8192 at rank 64 36.2 and 45.3; 257 at rank 384 38.1 and 48.4.
// The rule asks whether the tiles fit, not how long they take there: where they
// leave no room to split K the product waits for P (rank 384, 8192 x 8192: 400
// tokens 74.6 us beside, 49.0 otherwise; 512 with a checkpoint 112 and 81).
int launch_p_slice(const void* x, const void* A, __nv_bfloat16* P, __nv_bfloat16* P_lo, float s, int64_t tokens,
                   int64_t d_in, int64_t r, long long pairs, const DeviceInfo* dev, cudaStream_t st) {
  const long long spare = dev->num_sms - 2 * std::min<long long>(pairs, dev->pair_clusters);
  const bool beside = pairs > 0 && cdiv(r, kLinBM) * cdiv(tokens, slice_bn(tokens)) <= spare;
  if (tokens <= kDownTokens && !P_lo) {
    const auto* xb = static_cast<const __nv_bfloat16*>(x);
    const auto* ab = static_cast<const __nv_bfloat16*>(A);
    const auto kernel = tokens == 1 ? down_tokens_kernel<1> : (tokens == 2 ? down_tokens_kernel<2> : down_tokens_kernel<4>);
    note_launch();
    kernel<<<static_cast<unsigned>(r), kDownThreads, 0, st>>>(xb, ab, s, static_cast<int>(tokens),
                                                              static_cast<int>(d_in), static_cast<int>(r), P);
    return launch_error();
  }
  CUtensorMap tmX, tmA;
  if (make_map(&tmA, A, r, d_in) || make_map(&tmX, x, tokens, d_in, slice_bn(tokens))) return DORA_ERR_CUDA;
  SliceArgs sa{};
  sa.rows = static_cast<int>(r);
  sa.tokens = static_cast<int>(tokens);
  sa.kb_main = sa.kb_total = static_cast<int>(cdiv(d_in, kLinBK));
  // P in two halves is wanted as exact as fp32: summed as z is.  One bf16 value
  // (2^-8) does not show what a single sum drops (1e-5 of it at K = 8192).
  sa.chunk = P_lo ? kCkChunk * kPairKps : INT32_MAX;
  sa.alpha = s;
  sa.out = P;
  sa.out_lo = P_lo;
  return launch_slice(false, tmA, tmX, tmA, tmX, sa, false, beside ? spare : 0, dev, st);
}

// Tile width of the products with whole accumulators in registers: 128-wide
// tiles take about 0.58 of a 256-wide one's time, so the width whose waves over
// the pairs end first.  In 8 bits: 256 tokens through 8192 x 8192 24.6 us, 29.0 on
// 256-wide tiles that fill 32 of 74 pairs; 2000 tokens through 4096 x 4096 (four
// waves or two) 42.6 and 28.6, 4096 tokens (seven or four) 74 to 76 and 54 to 62;
// with a checkpoint 88 and 60, 149 and 116 to 131.
int pick_bn_waves(long long tiles_m, long long N, const DeviceInfo* dev) {
  const auto waves = [&](int width) { return cdiv(tiles_m * cdiv(N, width), dev->pair_clusters); };
  return 58 * waves(128) < 100 * waves(256) ? 128 : 256;
}

int fused_linear(const void* x, const void* W, const void* A, const void* B, const void* bias, const float* m,
                 const float* n, float s, int64_t tokens, int64_t d_in, int64_t d_out, int64_t r, dora_dtype dt,
                 void* y, bool ckpt, int8_t* z8, float* z_scale, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (dt != DORA_BF16) return DORA_ERR_UNSUPPORTED;
  if (tokens < 0 || d_in < 0 || d_out < 0 || r < 0) return DORA_ERR_INVALID_ARG;
  if (tokens == 0 || d_out == 0) return DORA_OK;
  if (d_in == 0) return DORA_ERR_UNSUPPORTED;
  if (tokens > INT32_MAX / 2 || d_in > INT32_MAX / 2 || d_out > INT32_MAX / 2 || r > INT32_MAX / 2)
    return DORA_ERR_UNSUPPORTED;
  if (!x || !W || !m || !n || !y || (r > 0 && (!A || !B))) return DORA_ERR_INVALID_ARG;
  if (ckpt && (!z8 || !z_scale)) return DORA_ERR_INVALID_ARG;
  if (d_in % 8 != 0 || d_out % 8 != 0 || r % 8 != 0) return DORA_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(y, 16) ||
      !aligned(bias, 2) || !aligned(m, 4) || !aligned(n, 4) || !aligned(z8, 16) || !aligned(z_scale, 4))
    return DORA_ERR_UNSUPPORTED;
  if (cdiv(tokens, kPairBM) * cdiv(d_out, 128) > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  const size_t p_bytes = dora_fused_linear_fwd_workspace_size(tokens, r);
  if (r > 0 && (!workspace || workspace_bytes < (ckpt ? 2 : 1) * p_bytes)) return DORA_ERR_WORKSPACE;
  if (r > 0 && !aligned(workspace, 256)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  __nv_bfloat16* P = static_cast<__nv_bfloat16*>(workspace);

  // B-side boxes hold the bn / 2 rows one CTA of a pair owns
  const int bn_y = ckpt ? pick_bn_waves(cdiv(tokens, kPairBM), d_out, dev) : pick_bn(d_out);
  CUtensorMap tmX, tmW, tmP, tmB;
  if (make_map(&tmX, x, tokens, d_in) || make_map(&tmW, W, d_out, d_in, bn_y / 2)) return DORA_ERR_CUDA;
  if (r > 0 && (make_map(&tmP, P, tokens, r) || make_map(&tmB, B, d_out, r, bn_y / 2))) return DORA_ERR_CUDA;
  const int kb_main = static_cast<int>(cdiv(d_in, kLinBK));
  const int stages = linear_pair_stages(dev->smem_optin);
  if (stages < 2) return DORA_ERR_UNSUPPORTED;
  const long long tiles_m2 = cdiv(tokens, kPairBM);
  cudaLaunchAttribute attrs[2];
  if (ckpt) {
    __nv_bfloat16* P_lo = r > 0 ? P + p_bytes / 2 : nullptr;
    if (r > 0 && launch_p_slice(x, A, P, P_lo, s, tokens, d_in, r, tiles_m2 * cdiv(d_out, bn_y), dev, st))
      return DORA_ERR_CUDA;
    CUtensorMap tmLo;
    if (r > 0 && make_map(&tmLo, P_lo, tokens, r)) return DORA_ERR_CUDA;
    LinearCkptArgs ca{};
    ca.M = static_cast<int>(tokens);
    ca.N = static_cast<int>(d_out);
    ca.kb_main = kb_main;
    ca.kb_r = static_cast<int>(cdiv(r, kLinBK));
    ca.tiles_m = static_cast<int>(tiles_m2);
    ca.tiles_n = static_cast<int>(cdiv(d_out, bn_y));
    ca.bn = bn_y;
    ca.stages = linear_i8_stages(dev->smem_optin);
    ca.m = m;
    ca.n = n;
    ca.bias = static_cast<const __nv_bfloat16*>(bias);
    ca.y = static_cast<__nv_bfloat16*>(y);
    ca.z8 = z8;
    ca.z_scale = z_scale;
    ca.wait_limit = kWaitLimitCycles;
    ca.status = dev->status;
    cudaLaunchConfig_t cfg = pair_config(attrs, kI8Threads, linear_i8_smem(dev->smem_optin),
                                         static_cast<long long>(ca.tiles_m) * ca.tiles_n, true, dev, st);
    note_launch();
    if (cudaLaunchKernelEx(&cfg, linear_ckpt8_pair_kernel, tmX, tmW, r > 0 ? tmP : tmX, r > 0 ? tmLo : tmX,
                           r > 0 ? tmB : tmW, ca) != cudaSuccess)
      return DORA_ERR_CUDA;
    return launch_error();
  }

  CUtensorMap tmA;
  if (r > 0 && (make_map(&tmA, A, r, d_in, pick_bn(r) / 2) || launch_p(tmX, tmA, P, s, tokens, d_in, r, dev, st)))
    return DORA_ERR_CUDA;
  // 2) y = bf16(g * [x | P] [W | B]^T + b), dependent on 1) only for the extension blocks
  LinearArgs la{};
  la.M = static_cast<int>(tokens);
  la.N = static_cast<int>(d_out);
  la.kb_main = kb_main;
  la.kb_total = kb_main + static_cast<int>(cdiv(r, kLinBK));
  la.tiles_m = static_cast<int>(tiles_m2);
  la.bn = bn_y;
  la.tiles_n = static_cast<int>(cdiv(d_out, bn_y));
  la.stages = stages;
  la.alpha = 1.f;
  la.m = m;
  la.n = n;
  la.bias = static_cast<const __nv_bfloat16*>(bias);
  la.out = static_cast<__nv_bfloat16*>(y);
  la.ldo = d_out;
  la.ext_waits = r > 0 ? 1 : 0;
  la.wait_limit = kWaitLimitCycles;
  la.status = dev->status;
  cudaLaunchConfig_t cfg = pair_config(attrs, kLinThreads, linear_pair_smem(dev->smem_optin),
                                       static_cast<long long>(la.tiles_m) * la.tiles_n, r > 0, dev, st);
  const CUtensorMap& tmA2 = r > 0 ? tmP : tmX;
  const CUtensorMap& tmB2 = r > 0 ? tmB : tmW;
  note_launch();
  if (cudaLaunchKernelEx(&cfg, linear_pair_kernel<false, false>, tmX, tmW, tmA2, tmB2, la) != cudaSuccess)
    return DORA_ERR_CUDA;
  return launch_error();
}

}  // namespace
}  // namespace dora

extern "C" {

int dora_fused_linear_fwd(const void* x, const void* W, const void* A, const void* B, const void* bias, const float* m,
                          const float* n, float s, int64_t tokens, int64_t d_in, int64_t d_out, int64_t r,
                          dora_dtype dt, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  return fused_linear(x, W, A, B, bias, m, n, s, tokens, d_in, d_out, r, dt, y, false, nullptr, nullptr, workspace,
                      workspace_bytes, stream);
}

size_t dora_fused_linear_fwd_ckpt8_workspace_size(int64_t tokens, int64_t r) {
  return 2 * dora_fused_linear_fwd_workspace_size(tokens, r);
}

int dora_fused_linear_fwd_ckpt8(const void* x, const void* W, const void* A, const void* B, const void* bias,
                                const float* m, const float* n, float s, int64_t tokens, int64_t d_in, int64_t d_out,
                                int64_t r, dora_dtype dt, void* y, int8_t* z8, float* z_scale, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return fused_linear(x, W, A, B, bias, m, n, s, tokens, d_in, d_out, r, dt, y, true, z8, z_scale, workspace,
                      workspace_bytes, stream);
}

// ------------------------------------------------------------ 8-bit operators
}  // extern "C"

namespace dora {
namespace {

// Rows to codes.  Many rows take 32 columns a thread (down to 64 threads), so
// that an SM holds many rows and one's reduction overlaps another's loads: 8192
// rows of 4096 bf16 with a residual took 39.4 us, 47.4 with 16 columns.  Few
// rows, and rows of single fp32 values (whose 32 loads a thread are too many),
// take up to 1024 threads, 8 columns each where that is enough.  Rows past 8192
// columns take 1024 threads of 64 registers, which spill in some types, and past
// 32768 they are read twice; with the reader (dequant_i8_kernel) after them:
// 8192 x 16384 bf16 with norm, residual and y 242.6 us (its bytes: 246), 8192 x
// 27648 bf16 268.2 (208), 4096 x 53248 bf16 440.8 (200), 2000 x 16384 fp32 with
// norm, residual and y 141 (110), 2000 x 16385 fp32 without y 418 (90).
template <typename T, int VEC, bool HAS_W>
int launch_rows_i8(const RowsI8Args& a, const DeviceInfo* dev, cudaStream_t st) {
  const long long most = VEC == 1 || a.rows < 2LL * dev->num_sms ? 1024 : 64;
  const dim3 grid(static_cast<unsigned>(a.rows));
  const auto threads = [&](long long nv) { return static_cast<unsigned>(align_up(cdiv(cdiv(a.d, VEC), nv), 32)); };
  if (cdiv(a.d, 8) <= most) return launch_after(rows_i8_kernel<T, VEC, 8 / VEC, 1024, HAS_W>, grid, threads(8 / VEC), st, a);
  if (cdiv(a.d, 16) <= most)
    return launch_after(rows_i8_kernel<T, VEC, 16 / VEC, 1024, HAS_W>, grid, threads(16 / VEC), st, a);
  if constexpr (VEC > 1) {  // single values take 16 columns a thread up to 16384
    if (cdiv(a.d, 32) <= 256)
      return launch_after(rows_i8_kernel<T, VEC, 32 / VEC, 256, HAS_W>, grid, threads(32 / VEC), st, a);
  }
  if (cdiv(a.d, 32) <= 1024)
    return launch_after(rows_i8_kernel<T, VEC, 32 / VEC, 1024, HAS_W>, grid, threads(32 / VEC), st, a);
  return launch_after(rows_i8_long_kernel<T, VEC>, grid, 1024, st, a);
}

template <typename T, int VEC>
int launch_rows_i8(const RowsI8Args& a, const DeviceInfo* dev, cudaStream_t st) {
  return a.weight ? launch_rows_i8<T, VEC, true>(a, dev, st) : launch_rows_i8<T, VEC, false>(a, dev, st);
}

int rows_i8(const void* x, const void* residual, const void* weight, bool norm, float eps, int64_t rows, int64_t d,
            dora_dtype dt, void* h, void* y, int8_t* q, float* scale, void* stream) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (rows < 0 || d < 0) return DORA_ERR_INVALID_ARG;
  if (rows == 0) return DORA_OK;
  if (d == 0) return DORA_ERR_UNSUPPORTED;
  if (!x || !q || !scale || (norm && !weight) || (residual && !h)) return DORA_ERR_INVALID_ARG;
  if (norm && !(eps >= 0.f)) return DORA_ERR_INVALID_ARG;
  if (rows > INT32_MAX || d > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  const auto all_aligned = [&](size_t e) {
    return aligned(x, e) && aligned(residual, e) && aligned(weight, e) && (!residual || aligned(h, e)) && aligned(y, e);
  };
  if (dt == DORA_BF16 && (d % 8 != 0 || !all_aligned(16) || !aligned(q, 8))) return DORA_ERR_UNSUPPORTED;
  if (!all_aligned(4) || !aligned(scale, 4)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  RowsI8Args a{};
  a.x = x;
  a.residual = residual;
  a.weight = norm ? weight : nullptr;
  a.h = h;
  a.y = y;
  a.q = q;
  a.scale = scale;
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dt == DORA_BF16) return launch_rows_i8<__nv_bfloat16, 8>(a, dev, st);
  if (d % 4 == 0 && all_aligned(16) && aligned(q, 4)) return launch_rows_i8<float, 4>(a, dev, st);
  return launch_rows_i8<float, 1>(a, dev, st);
}

template <typename L>
int launch_compose_fwd_ckpt8(const void* base_out, const void* lora_out, const void* bias, const float* m,
                              const float* n, float s, int64_t tokens, int64_t d_out, void* y, int8_t* z8,
                              float* z_scale, const DeviceInfo* dev, cudaStream_t st) {
  using T = typename L::T;
  const long long blocks = cdiv(d_out, kCkptBlock);
  const int threads = static_cast<int>(std::min<long long>(256, align_up(blocks * L::kLanes, 32)));
  const long long gx = cdiv(blocks, threads / L::kLanes);
  // one wave of resident CTAs (two an SM): a CTA starts its loads once and then
  // keeps the next group's in flight (8192 x 8192 bf16, while each CTA took a
  // stretch of rows: 87.6 us, 90.7 with 8 CTAs an SM, 103.6 with 16; with rows in
  // turn over the grid one wave takes 78)
  const long long gy = std::max<long long>(1, std::min<long long>({2LL * dev->num_sms / gx, cdiv(tokens, kCkptRows), 65535}));
  return launch_after(bias ? compose_fwd_ckpt8_kernel<L, true> : compose_fwd_ckpt8_kernel<L, false>,
                      dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), threads, st,
                      static_cast<const T*>(base_out), static_cast<const T*>(lora_out), static_cast<const T*>(bias), m, n,
                      s, tokens, d_out, blocks, static_cast<T*>(y), z8, z_scale);
}

template <typename L>
int launch_compose_bwd_ckpt8(const void* dy, const int8_t* z8, const float* z_scale, const float* m, const float* n,
                              float s, int64_t tokens, int64_t d_out, void* d_base, void* d_lora, float* d_m,
                              uint8_t* ws, const DeviceInfo* dev, cudaStream_t st) {
  using T = typename L::T;
  const long long blocks = cdiv(d_out, kCkptBlock);
  const long long slots = static_cast<long long>(dev->num_sms) * dev->ckpt_bwd_ctas[L::kIndex];
  // at least one row for each row of lanes
  const long long most = cdiv(tokens, kCkptBwdThreads / L::kLanes);
  // one wave of resident CTAs (32768 x 8192 bf16: 309.7 us, 320.6 in two)
  const long long chunks =
      std::max<long long>(1, std::min<long long>({slots / blocks, static_cast<long long>(kCkptMaxChunks), most}));
  unsigned long long* marks = reinterpret_cast<unsigned long long*>(ws);  // tagged: no clearing needed
  float* part = reinterpret_cast<float*>(ws + blocks * kCkptMaxChunks * 8);
  return launch_after(compose_bwd_ckpt8_kernel<L>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(chunks)),
                      kCkptBwdThreads, st, static_cast<const T*>(dy), z8, z_scale, m, n, s, tokens, d_out, blocks,
                      static_cast<T*>(d_base), static_cast<T*>(d_lora), part, marks, d_m, next_bwd_epoch() + 1);
}

}  // namespace
}  // namespace dora

extern "C" {

int dora_rms_norm_i8(const void* x, const void* residual, const void* weight, float eps, int64_t tokens, int64_t d,
                     dora_dtype dt, void* h, void* y, int8_t* q, float* scale, void* stream) {
  return rows_i8(x, residual, weight, true, eps, tokens, d, dt, h, y, q, scale, stream);
}

int dora_quantize_rows_i8(const void* x, const void* residual, int64_t rows, int64_t cols, dora_dtype dt, void* h,
                          int8_t* q, float* scale, void* stream) {
  return rows_i8(x, residual, nullptr, false, 0.f, rows, cols, dt, h, nullptr, q, scale, stream);
}

int dora_dequantize_i8(const int8_t* q, const float* scale, int64_t rows, int64_t cols, int64_t block, dora_dtype dt,
                       void* out, void* stream) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (rows < 0 || cols < 0) return DORA_ERR_INVALID_ARG;
  if (block != 0 && block != kCkptBlock) return DORA_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return DORA_OK;
  if (!q || !scale || !out) return DORA_ERR_INVALID_ARG;
  if (rows > INT32_MAX || cols > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  if (!aligned(out, dt == DORA_BF16 ? 2 : 4) || !aligned(scale, 4)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long width = block ? block : cols;
  const long long blocks = cdiv(cols, width);
  const auto launch = [&](auto kernel, int vec, int u, auto* o) {
    const long long vecs = cdiv(cols, vec);
    const int threads = static_cast<int>(std::min<long long>(256, align_up(vecs, 32)));
    const long long gx = cdiv(vecs, threads);
    // short CTAs, 32 an SM in all; of the wider single-column ones 8 (2000 x
    // 4099 fp32: 13.5 us, 17.6 with 32; 8192 x 8192 bf16: 31.7, 34.1 with 8).  The
    // former's 41 MB would take 6.3: it moves one byte in and four out an access
    const long long ctas = (vec > 1 ? 32LL : 8LL) * dev->num_sms;
    const long long gy = std::max<long long>(1, std::min<long long>({cdiv(rows, u), 65535, ctas / gx}));
    return launch_after(kernel, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), threads, st, q, scale, rows,
                        cols, width, blocks, o);
  };
  if (dt == DORA_BF16) {
    auto* o = static_cast<__nv_bfloat16*>(out);
    if (cols % 8 == 0 && aligned(q, 8) && aligned(out, 16)) return launch(dequant_i8_kernel<__nv_bfloat16, 8, 4>, 8, 4, o);
    return launch(dequant_i8_kernel<__nv_bfloat16, 1, 8>, 1, 8, o);
  }
  auto* o = static_cast<float*>(out);
  if (cols % 4 == 0 && aligned(q, 4) && aligned(out, 16)) return launch(dequant_i8_kernel<float, 4, 4>, 4, 4, o);
  return launch(dequant_i8_kernel<float, 1, 8>, 1, 8, o);
}

size_t dora_linear_i8_fwd_workspace_size(int64_t tokens, int64_t r) {
  return dora_fused_linear_fwd_workspace_size(tokens, r);
}

int dora_linear_i8_fwd(const int8_t* x_q, const float* x_scale, const int8_t* W_q, const float* w_scale, const void* x,
                       const void* A, const void* B, const void* bias, const float* m, const float* n, float s,
                       int64_t tokens, int64_t d_in, int64_t d_out, int64_t r, dora_dtype dt, void* y, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (dt != DORA_BF16) return DORA_ERR_UNSUPPORTED;
  if (tokens < 0 || d_in < 0 || d_out < 0 || r < 0) return DORA_ERR_INVALID_ARG;
  if (tokens == 0 || d_out == 0) return DORA_OK;
  if (!x_q || !x_scale || !W_q || !w_scale || !y || (r > 0 && (!x || !A || !B)) || ((m == nullptr) != (n == nullptr)))
    return DORA_ERR_INVALID_ARG;
  if (d_in == 0 || d_in % 16 != 0 || d_out % 8 != 0 || r % 8 != 0) return DORA_ERR_UNSUPPORTED;
  // int32 holds d_in products of two codes, -128 among them: 2^14 * d_in < 2^31
  if (d_in > kI8MaxDIn || tokens > INT32_MAX / 2 || d_out > INT32_MAX / 2 || r > INT32_MAX / 2)
    return DORA_ERR_UNSUPPORTED;
  if (cdiv(tokens, kPairBM) * cdiv(d_out, 128) > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  if (!aligned(x_q, 16) || !aligned(W_q, 16) || !aligned(y, 16) || !aligned(bias, 2) || !aligned(x_scale, 4) ||
      !aligned(w_scale, 4) || !aligned(m, 4) || !aligned(n, 4))
    return DORA_ERR_UNSUPPORTED;
  if (r > 0 && (!aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16))) return DORA_ERR_UNSUPPORTED;
  if (r > 0 && (!workspace || workspace_bytes < dora_linear_i8_fwd_workspace_size(tokens, r)))
    return DORA_ERR_WORKSPACE;
  if (r > 0 && !aligned(workspace, 256)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  __nv_bfloat16* P = static_cast<__nv_bfloat16*>(workspace);
  CUtensorMap tmXq, tmWq, tmP, tmB;
  if (tokens <= kSliceTokens) {
    const uint32_t bn = slice_bn(tokens);
    if (make_map_i8(&tmWq, W_q, d_out, d_in, kLinBM) || make_map_i8(&tmXq, x_q, tokens, d_in, bn)) return DORA_ERR_CUDA;
    SliceArgs sa{};
    sa.tokens = static_cast<int>(tokens);
    if (r > 0 && (make_map(&tmB, B, d_out, r) || make_map(&tmP, P, tokens, r, bn) ||
                  launch_p_slice(x, A, P, nullptr, s, tokens, d_in, r, 0, dev, st)))
      return DORA_ERR_CUDA;
    sa.rows = static_cast<int>(d_out);
    sa.kb_main = static_cast<int>(cdiv(d_in, kI8BK));
    sa.kb_total = sa.kb_main + static_cast<int>(cdiv(r, kLinBK));
    sa.x_scale = x_scale;
    sa.w_scale = w_scale;
    sa.m = m;
    sa.n = n;
    sa.bias = static_cast<const __nv_bfloat16*>(bias);
    sa.out = static_cast<__nv_bfloat16*>(y);
    return launch_slice(true, tmWq, tmXq, r > 0 ? tmB : tmWq, r > 0 ? tmP : tmXq, sa, true, 0, dev, st);
  }
  const long long tiles_m = cdiv(tokens, kPairBM);
  const int bn = pick_bn_waves(tiles_m, d_out, dev);
  if (make_map_i8(&tmXq, x_q, tokens, d_in, kLinBM) || make_map_i8(&tmWq, W_q, d_out, d_in, bn / 2)) return DORA_ERR_CUDA;
  if (r > 0 && (make_map(&tmP, P, tokens, r) || make_map(&tmB, B, d_out, r, bn / 2) ||
                launch_p_slice(x, A, P, nullptr, s, tokens, d_in, r, tiles_m * cdiv(d_out, bn), dev, st)))
    return DORA_ERR_CUDA;
  LinearI8Args la{};
  la.M = static_cast<int>(tokens);
  la.N = static_cast<int>(d_out);
  la.kb_main = static_cast<int>(cdiv(d_in, kI8BK));
  la.kb_total = la.kb_main + static_cast<int>(cdiv(r, kLinBK));
  la.tiles_m = static_cast<int>(tiles_m);
  la.tiles_n = static_cast<int>(cdiv(d_out, bn));
  la.bn = bn;
  la.stages = linear_i8_stages(dev->smem_optin);
  la.x_scale = x_scale;
  la.w_scale = w_scale;
  la.m = m;
  la.n = n;
  la.bias = static_cast<const __nv_bfloat16*>(bias);
  la.y = static_cast<__nv_bfloat16*>(y);
  la.wait_limit = kWaitLimitCycles;
  la.status = dev->status;
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = pair_config(attrs, kI8Threads, linear_i8_smem(dev->smem_optin),
                                       static_cast<long long>(la.tiles_m) * la.tiles_n, true, dev, st);
  note_launch();
  if (cudaLaunchKernelEx(&cfg, linear_i8_pair_kernel, tmXq, tmWq, r > 0 ? tmP : tmXq, r > 0 ? tmB : tmWq, la) !=
      cudaSuccess)
    return DORA_ERR_CUDA;
  return launch_error();
}

int dora_compose_fwd_ckpt8(const void* base_out, const void* lora_out, const void* bias, const float* m,
                           const float* n, float s, int64_t tokens, int64_t d_out, dora_dtype dt, void* y, int8_t* z8,
                           float* z_scale, void* stream) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (tokens < 0 || d_out < 0) return DORA_ERR_INVALID_ARG;
  if (tokens == 0 || d_out == 0) return DORA_OK;
  if (!base_out || !lora_out || !m || !n || !y || !z8 || !z_scale) return DORA_ERR_INVALID_ARG;
  if (tokens > INT32_MAX || d_out > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  const auto all_aligned = [&](size_t e) {
    return aligned(base_out, e) && aligned(lora_out, e) && aligned(bias, e) && aligned(y, e);
  };
  if (dt == DORA_BF16 && (d_out % 8 != 0 || !all_aligned(16) || !aligned(z8, 8))) return DORA_ERR_UNSUPPORTED;
  if (!all_aligned(4) || !aligned(m, 4) || !aligned(n, 4) || !aligned(z_scale, 4)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dt == DORA_BF16)
    return launch_compose_fwd_ckpt8<LanesBf16>(base_out, lora_out, bias, m, n, s, tokens, d_out, y, z8, z_scale, dev, st);
  if (d_out % 4 == 0 && all_aligned(16) && aligned(z8, 4))
    return launch_compose_fwd_ckpt8<LanesF32>(base_out, lora_out, bias, m, n, s, tokens, d_out, y, z8, z_scale, dev, st);
  return launch_compose_fwd_ckpt8<LanesF32Any>(base_out, lora_out, bias, m, n, s, tokens, d_out, y, z8, z_scale, dev, st);
}

size_t dora_compose_bwd_ckpt8_workspace_size(int64_t tokens, int64_t d_out) {
  if (tokens < 0 || d_out < 0) return 0;
  const int64_t d = std::max<int64_t>(d_out, 1);
  return static_cast<size_t>(cdiv(d, kCkptBlock)) * kCkptMaxChunks * 8 +
         align_up(static_cast<size_t>(kCkptMaxChunks) * d * 4, 256);
}

int dora_compose_bwd_ckpt8(const void* dy, const int8_t* z8, const float* z_scale, const float* m, const float* n,
                           float s, int64_t tokens, int64_t d_out, dora_dtype dt, void* d_base, void* d_lora,
                           float* d_m, void* workspace, size_t workspace_bytes, void* stream) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (tokens < 0 || d_out < 0) return DORA_ERR_INVALID_ARG;
  if (d_out == 0) return DORA_OK;
  if (!m || !n || !d_m) return DORA_ERR_INVALID_ARG;
  if (tokens > 0 && (!dy || !z8 || !z_scale || !d_base || !d_lora)) return DORA_ERR_INVALID_ARG;
  if (tokens > INT32_MAX || d_out > INT32_MAX) return DORA_ERR_UNSUPPORTED;
  const auto all_aligned = [&](size_t e) { return aligned(dy, e) && aligned(d_base, e) && aligned(d_lora, e); };
  if (dt == DORA_BF16 && (d_out % 8 != 0 || (tokens > 0 && (!all_aligned(16) || !aligned(z8, 8)))))
    return DORA_ERR_UNSUPPORTED;
  if (tokens > 0 && (!all_aligned(4) || !aligned(z_scale, 4))) return DORA_ERR_UNSUPPORTED;
  if (!aligned(m, 4) || !aligned(n, 4) || !aligned(d_m, 4)) return DORA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < dora_compose_bwd_ckpt8_workspace_size(tokens, d_out)) return DORA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens == 0)
    return cudaMemsetAsync(d_m, 0, static_cast<size_t>(d_out) * 4, st) == cudaSuccess ? DORA_OK : DORA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (dt == DORA_BF16)
    return launch_compose_bwd_ckpt8<LanesBf16>(dy, z8, z_scale, m, n, s, tokens, d_out, d_base, d_lora, d_m, ws, dev, st);
  if (d_out % 4 == 0 && all_aligned(16) && aligned(z8, 4))
    return launch_compose_bwd_ckpt8<LanesF32>(dy, z8, z_scale, m, n, s, tokens, d_out, d_base, d_lora, d_m, ws, dev, st);
  return launch_compose_bwd_ckpt8<LanesF32Any>(dy, z8, z_scale, m, n, s, tokens, d_out, d_base, d_lora, d_m, ws, dev, st);
}

// ---------------------------------------------------- attached-norm backward
namespace {
struct BwdLayout {
  int nt, splits_max;  // K splits of each of the two Gram products (G and H) in one launch
  size_t off_part, off_part2, off_sg, off_h, off_bt, off_bct, total;
};
BwdLayout bwd_layout(int64_t d_out, int64_t r) {
  BwdLayout L{};
  L.nt = static_cast<int>(cdiv(r, kBoxRows));
  L.splits_max = std::max(1, std::min(kMaxGramSplits, 80 / (L.nt * L.nt)));
  const size_t part_bytes = static_cast<size_t>(L.splits_max) * L.nt * L.nt * kBoxRows * kBoxRows * 4;
  size_t off = 0;
  L.off_part = off;
  off = align_up(off + part_bytes, 256);
  L.off_part2 = off;
  off = align_up(off + part_bytes, 256);
  L.off_sg = off;
  off = align_up(off + static_cast<size_t>(r) * r * 2, 256);
  L.off_h = off;
  off = align_up(off + static_cast<size_t>(r) * r * 2, 256);
  L.off_bt = off;
  off = align_up(off + static_cast<size_t>(r) * d_out * 2, 256);
  L.off_bct = off;
  off = align_up(off + static_cast<size_t>(r) * d_out * 2, 256);
  L.total = std::max<size_t>(off, 256);
  return L;
}
}  // namespace

size_t dora_factored_norm_bwd_workspace_size(int64_t d_out, int64_t d_in, int64_t r) {
  if (d_out < 0 || d_in < 0 || r < 0) return 0;
  return bwd_layout(d_out, r).total;
}

int dora_factored_norm_bwd(const void* W, const void* A, const void* B, float s, const float* n, const float* d_n,
                           int64_t d_out, int64_t d_in, int64_t r, dora_dtype dt, float* dA, float* dB,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (dt != DORA_BF16) return DORA_ERR_UNSUPPORTED;
  if (d_out < 0 || d_in < 0 || r < 0) return DORA_ERR_INVALID_ARG;
  if (d_out > INT32_MAX / 2 || d_in > INT32_MAX / 2 || r > INT32_MAX / 2) return DORA_ERR_UNSUPPORTED;
  if (r == 0) return DORA_OK;  // dA and dB are empty
  if ((d_in > 0 && !dA) || (d_out > 0 && !dB)) return DORA_ERR_INVALID_ARG;
  if (!aligned(dA, 16) || !aligned(dB, 16)) return DORA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d_out == 0 || d_in == 0) {
    // no rows: dA = 0; no columns: V = 0 + s B A with A empty, so dB = 0
    float* z = d_out == 0 ? dA : dB;
    const size_t bytes = static_cast<size_t>(r) * (d_out == 0 ? d_in : d_out) * 4;
    if (bytes == 0) return DORA_OK;
    return cudaMemsetAsync(z, 0, bytes, st) == cudaSuccess ? DORA_OK : DORA_ERR_CUDA;
  }
  if (!W || !A || !B || !n || !d_n) return DORA_ERR_INVALID_ARG;
  if (d_in % 8 != 0 || d_out % 8 != 0 || r % 8 != 0) return DORA_ERR_UNSUPPORTED;
  if (!aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(n, 4) || !aligned(d_n, 4))
    return DORA_ERR_UNSUPPORTED;
  const BwdLayout L = bwd_layout(d_out, r);
  if (!workspace || workspace_bytes < L.total) return DORA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part = reinterpret_cast<float*>(ws + L.off_part);
  float* part2 = reinterpret_cast<float*>(ws + L.off_part2);
  __nv_bfloat16* sG = reinterpret_cast<__nv_bfloat16*>(ws + L.off_sg);
  __nv_bfloat16* s2H = reinterpret_cast<__nv_bfloat16*>(ws + L.off_h);
  __nv_bfloat16* Bt = reinterpret_cast<__nv_bfloat16*>(ws + L.off_bt);
  __nv_bfloat16* Bct = reinterpret_cast<__nv_bfloat16*>(ws + L.off_bct);

  const int bn_b = pick_bn(r), bn_a = pick_bn(d_in);
  CUtensorMap tmW, tmA, tmAb, tmB, tmSG, tmBt, tmBct, tmH, tmWmn, tmAmn;
  if (make_map(&tmW, W, d_out, d_in) || make_map(&tmA, A, r, d_in) || make_map(&tmAb, A, r, d_in, bn_b / 2) ||
      make_map(&tmB, B, d_out, r) || make_map(&tmSG, sG, r, r, bn_b / 2) || make_map(&tmBt, Bt, r, d_out) ||
      make_map(&tmBct, Bct, r, d_out) || make_map(&tmH, s2H, r, r) || make_map(&tmWmn, W, d_out, d_in, 64) ||
      make_map(&tmAmn, A, r, d_in, 64))
    return DORA_ERR_CUDA;

  // 1) B^T and (s c B)^T
  note_launch();
  norm_bwd_prep_kernel<<<dim3(static_cast<unsigned>(cdiv(d_out, kPrepTile)), static_cast<unsigned>(cdiv(r, kPrepTile))),
                         256, 0, st>>>(static_cast<const __nv_bfloat16*>(B), d_n, n, s, static_cast<int>(d_out),
                               static_cast<int>(r), Bt, Bct);
  if (launch_error()) return DORA_ERR_CUDA;

  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;

  // 2) one Gram launch for both products: G = A A^T over d_in and
  //    s H = (s c B)^T B over d_out (split-K partial tiles), then one fixed-order
  //    reduction writing bf16 s G and s^2 H
  const int kb_g = static_cast<int>(cdiv(d_in, kBK)), kb_h = static_cast<int>(cdiv(d_out, kBK));
  GramArgs ga{};
  ga.r = static_cast<int>(r);
  ga.n_tiles = L.nt;
  ga.kb_main = kb_g;
  ga.splits = std::max(1, std::min({L.splits_max, (dev->num_sms / 2) / (L.nt * L.nt), kb_g}));
  ga.kb_main2 = kb_h;
  ga.splits2 = std::max(1, std::min({L.splits_max, (dev->num_sms / 2) / (L.nt * L.nt), kb_h}));
  ga.upper = 1;  // G = A A^T is symmetric: its tiles on or above the diagonal only
  ga.n_ctas1 = L.nt * (L.nt + 1) / 2 * ga.splits;
  ga.partial = part;
  ga.partial2 = part2;
  ga.wait_limit = kWaitLimitCycles;
  ga.status = dev->status;
  const size_t gram_smem = kGramStages * kGramStageBytes + (2 * kGramStages + 1) * 8 + 16 + 1024;
  note_launch();
  gram_tc_kernel<<<ga.n_ctas1 + L.nt * L.nt * ga.splits2, kNormThreads, gram_smem, st>>>(tmA, tmA, tmBct, tmBt, ga);
  if (launch_error()) return DORA_ERR_CUDA;
  {
    cudaLaunchConfig_t cfg{};
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    const long long rr = static_cast<long long>(r) * r;
    const int g1 = static_cast<int>(std::max<long long>(1, std::min<long long>(cdiv(rr, 1024), 2 * dev->num_sms)));
    cfg.gridDim = dim3(static_cast<unsigned>(2 * g1));
    cfg.blockDim = dim3(256);
    note_launch();
    if (cudaLaunchKernelEx(&cfg, gram_reduce_kernel, static_cast<const float*>(part), ga.splits, static_cast<int>(r), s,
                           sG, static_cast<int*>(nullptr), 0, g1, static_cast<const float*>(part2), ga.splits2, s,
                           s2H, 1) != cudaSuccess)
      return DORA_ERR_CUDA;
  }

  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = 2;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  attrs[1] = pdl[0];
  cudaLaunchConfig_t pcfg{};
  pcfg.stream = st;
  pcfg.attrs = attrs;
  pcfg.numAttrs = 2;
  pcfg.blockDim = dim3(kLinThreads);
  pcfg.dynamicSmemBytes = linear_pair_smem(dev->smem_optin);
  const int stages = linear_pair_stages(dev->smem_optin);
  if (stages < 2) return DORA_ERR_UNSUPPORTED;
  auto pair_grid = [&](const LinearArgs& la) {
    return dim3(static_cast<unsigned>(2 * std::min<long long>(dev->pair_clusters,
                                                              static_cast<long long>(la.tiles_m) * la.tiles_n)));
  };

  // 3) dB = s c * ([W | B] [A | s G]^T), waiting for the reduction only
  //    before its K-extension blocks
  LinearArgs lb{};
  lb.M = static_cast<int>(d_out);
  lb.N = static_cast<int>(r);
  lb.kb_main = static_cast<int>(cdiv(d_in, kLinBK));
  lb.kb_total = lb.kb_main + static_cast<int>(cdiv(r, kLinBK));
  lb.tiles_m = static_cast<int>(cdiv(d_out, kPairBM));
  lb.bn = bn_b;
  lb.tiles_n = static_cast<int>(cdiv(r, bn_b));
  lb.stages = stages;
  lb.alpha = s;
  lb.rs_num = d_n;
  lb.rs_den = n;
  lb.out = dB;
  lb.ldo = r;
  lb.ext_waits = 1;
  lb.wait_limit = kWaitLimitCycles;
  lb.status = dev->status;
  pcfg.gridDim = pair_grid(lb);
  note_launch();
  if (cudaLaunchKernelEx(&pcfg, linear_pair_kernel<false, true>, tmW, tmAb, tmB, tmSG, lb) != cudaSuccess)
    return DORA_ERR_CUDA;

  // 4) dA = [(s c B)^T | s^2 H] [W ; A], dependent on dB through programmatic
  //    dependent launch: its CTAs take the SMs dB leaves free or finishes
  //    with; before its extension blocks it waits for dB's completion, which
  //    follows the reduction's
  LinearArgs la{};
  la.M = static_cast<int>(r);
  la.N = static_cast<int>(d_in);
  la.kb_main = static_cast<int>(cdiv(d_out, kLinBK));
  la.kb_total = la.kb_main + static_cast<int>(cdiv(r, kLinBK));
  la.tiles_m = static_cast<int>(cdiv(r, kPairBM));
  la.bn = bn_a;
  la.tiles_n = static_cast<int>(cdiv(d_in, bn_a));
  la.stages = stages;
  la.alpha = 1.f;
  la.out = dA;
  la.ldo = d_in;
  la.ext_waits = 1;
  la.wait_limit = kWaitLimitCycles;
  la.status = dev->status;
  pcfg.gridDim = pair_grid(la);
  note_launch();
  if (cudaLaunchKernelEx(&pcfg, linear_pair_kernel<true, true>, tmBct, tmWmn, tmH, tmAmn, la) != cudaSuccess)
    return DORA_ERR_CUDA;
  return launch_error();
}

}  // extern "C"

// ------------------------------------------------------------------------
// dora_compose_bwd_noalloc: the compose backward with library-owned scratch.
// The scratch is one file-scope device array; host code must not pass the
// array's name to a kernel (on the host it is only a stand-in symbol), so its
// device address is looked up once per device with that device current.
namespace dora {
namespace {

constexpr int kNoallocChunks = 16;     // row chunks of column partials
constexpr size_t kNoallocCounterBytes = 16384;
// 64-bit tagged arrival counters, one per 16-vector column strip; the most
// strips come with 1-element vectors at the largest d_out
static_assert((DORA_NOALLOC_MAX_D_OUT + kBwdVecs - 1) / kBwdVecs * 8 <= kNoallocCounterBytes,
              "counter area too small for the largest d_out");
static_assert(DORA_NOALLOC_SCRATCH_BYTES == kNoallocCounterBytes + kNoallocChunks * 4ull * DORA_NOALLOC_MAX_D_OUT,
              "scratch layout and the header's size disagree");

static __device__ __align__(256) unsigned char g_noalloc_scratch[DORA_NOALLOC_SCRATCH_BYTES];

std::mutex g_noalloc_mu;
unsigned char* g_noalloc_ptr[kMaxDevices] = {};
CUcontext g_noalloc_ctx[kMaxDevices] = {};

typedef CUresult (*CtxGetCurrentFn)(CUcontext*);
CtxGetCurrentFn g_ctx_current = nullptr;

// The array's device address for the current device, looked up (with that
// device current) the first time this device's current context is seen.  A
// context torn down and created again (cudaDeviceReset) may load the module
// at another address, so the cached address is tied to the context it was
// looked up in.
int noalloc_scratch(unsigned char** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DORA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (!g_ctx_current) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return DORA_ERR_CUDA;
    g_ctx_current = reinterpret_cast<CtxGetCurrentFn>(fn);
  }
  CUcontext ctx = nullptr;
  if (g_ctx_current(&ctx) != CUDA_SUCCESS) return DORA_ERR_CUDA;
  if (!g_noalloc_ptr[dev] || ctx == nullptr || ctx != g_noalloc_ctx[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) {
      cudaGetLastError();
      return DORA_ERR_CUDA;
    }
    // the lookup makes the device's primary context current if none was
    if (g_ctx_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return DORA_ERR_CUDA;
    g_noalloc_ptr[dev] = static_cast<unsigned char*>(p);
    g_noalloc_ctx[dev] = ctx;
  }
  *out = g_noalloc_ptr[dev];
  return DORA_OK;
}

}  // namespace
}  // namespace dora

extern "C" int dora_compose_bwd_noalloc(const void* dy, const void* base_out, const void* lora_out, const float* m,
                                        const float* n, float s, int64_t tokens, int64_t d_out, dora_dtype dt,
                                        void* d_base, void* d_lora, float* d_m, void* stream) {
  return dora_compose_bwd_noalloc_bias(dy, base_out, lora_out, nullptr, m, n, s, tokens, d_out, dt, d_base, d_lora,
                                       d_m, stream);
}

extern "C" int dora_compose_bwd_noalloc_bias(const void* dy, const void* base_out, const void* lora_out,
                                             const void* bias, const float* m, const float* n, float s,
                                             int64_t tokens, int64_t d_out, dora_dtype dt, void* d_base,
                                             void* d_lora, float* d_m, void* stream) {
  if (dt != DORA_BF16 && dt != DORA_F32) return DORA_ERR_UNSUPPORTED;
  if (tokens < 0 || d_out < 0) return DORA_ERR_INVALID_ARG;
  if (d_out > DORA_NOALLOC_MAX_D_OUT) return DORA_ERR_UNSUPPORTED;
  if (d_out == 0) return DORA_OK;
  if (!m || !n || !d_m) return DORA_ERR_INVALID_ARG;
  if (tokens > 0 && (!dy || !base_out || !lora_out || !d_base || !d_lora)) return DORA_ERR_INVALID_ARG;
  int vec = 1;
  if (dt == DORA_BF16) {
    if (d_out % 8 != 0) return DORA_ERR_UNSUPPORTED;
    if (tokens > 0 && (!aligned(dy, 16) || !aligned(base_out, 16) || !aligned(lora_out, 16) ||
                       !aligned(d_base, 16) || !aligned(d_lora, 16)))
      return DORA_ERR_UNSUPPORTED;
    vec = 8;
  } else {
    const bool a16 = aligned(dy, 16) && aligned(base_out, 16) && aligned(lora_out, 16) && aligned(d_base, 16) &&
                     aligned(d_lora, 16) && aligned(bias, 16);
    if (!aligned(dy, 4) || !aligned(base_out, 4) || !aligned(lora_out, 4) || !aligned(d_base, 4) ||
        !aligned(d_lora, 4))
      return DORA_ERR_UNSUPPORTED;
    vec = (d_out % 4 == 0 && a16) ? 4 : 1;
  }
  if (!aligned(m, 4) || !aligned(n, 4) || !aligned(d_m, 4) || !aligned(bias, dt == DORA_BF16 ? 16 : 4))
    return DORA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev)) return DORA_ERR_CUDA;
  unsigned char* scratch = nullptr;
  if (noalloc_scratch(&scratch)) return DORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens == 0) return cudaMemsetAsync(d_m, 0, static_cast<size_t>(d_out) * 4, st) == cudaSuccess ? DORA_OK : DORA_ERR_CUDA;

  const long long nvec = d_out / vec;
  const long long strips = cdiv(nvec, kBwdVecs);
  int occ = 1;
  if (dt == DORA_BF16)
    occ = ctas_per_sm(compose_bwd_kernel<__nv_bfloat16, 8, false>, kBwdThreads);
  else if (vec == 4)
    occ = ctas_per_sm(compose_bwd_kernel<float, 4, false>, kBwdThreads);
  else
    occ = ctas_per_sm(compose_bwd_kernel<float, 1, false>, kBwdThreads);
  const long long chunks = bwd_chunks(strips, static_cast<long long>(dev->num_sms) * occ, tokens,
                                      std::min<long long>(kNoallocChunks, cdiv(tokens, kBwdSlots)));
  const long long rows = cdiv(tokens, chunks);
  const long long chunks2 = cdiv(tokens, rows);
  // tagged strip counters (no clearing needed); the partials are written before read
  if (static_cast<size_t>(strips) * 8 > kNoallocCounterBytes) return DORA_ERR_UNSUPPORTED;
  unsigned long long* cnt = reinterpret_cast<unsigned long long*>(scratch);
  float* part = reinterpret_cast<float*>(scratch + kNoallocCounterBytes);
  dim3 grid(static_cast<unsigned>(strips), static_cast<unsigned>(chunks2));
  if (dt == DORA_BF16)
    launch_compose_bwd<__nv_bfloat16, 8>(grid, st, dy, base_out, lora_out, bias, m, n, s, tokens, nvec, d_out, d_base,
                                         d_lora, part, cnt, d_m, rows);
  else if (vec == 4)
    launch_compose_bwd<float, 4>(grid, st, dy, base_out, lora_out, bias, m, n, s, tokens, nvec, d_out, d_base, d_lora,
                                part, cnt, d_m, rows);
  else
    launch_compose_bwd<float, 1>(grid, st, dy, base_out, lora_out, bias, m, n, s, tokens, nvec, d_out, d_base, d_lora,
                                part, cnt, d_m, rows);
  return launch_error();
}
