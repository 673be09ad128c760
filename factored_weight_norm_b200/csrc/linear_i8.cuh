// linear_i8.cuh - the DoRA linear forward with the base weight and its input
// in 8-bit integers, on tcgen05 tensor cores (sm_100a).
//
//   y = b + g * (sx_t * sw_o * sum_k xq[t,k] Wq[o,k] + sum_j P[t,j] B[o,j]),
//   g = m / n,  P = bf16(s * x A^T)
//
// The base product runs in kind::i8 with int32 accumulation: exact, so its
// order never shows.  The adapter's product runs in kind::f16 (bf16, fp32
// accumulation) into an accumulator of its own, since the two differ in their
// scales.  The epilogue joins them in fp32 with one rounding to bf16.
#pragma once

#include "linear_tc.cuh"

namespace dora {

// Three warpgroups: producer and MMA issuer (two warps idle), two of epilogue
// warps.  The epilogue holds 128 accumulators a thread beside its factors and
// outputs, so the first warpgroup gives it registers: 384 threads are launched
// with 168 each, and 128 * 40 + 256 * 232 = 384 * 168.
constexpr int kI8Threads = 384;
constexpr int kI8RegsFew = 40, kI8RegsMany = 232;
static_assert(128 * kI8RegsFew + 256 * kI8RegsMany <= kI8Threads * 168, "register shares");
constexpr int kI8BK = 128;       // int8 K block: 128 bytes, as 64 bf16 are
constexpr int64_t kI8MaxDIn = 131056;  // the largest multiple of 16 with 2^14 * d_in < 2^31
constexpr int kI8EpiThreads = 256;
// barriers: full / empty per stage, base and adapter accumulators full (one)
// and empty (one each), drain; the TMEM slot and the abort flag
constexpr size_t kI8BarrierBytes = 256;
// per-column epilogue factors of two tiles: sw * g, g, b
constexpr size_t kI8ColBytes = 2 * 3 * kPairBN * sizeof(float);

// A sum over K in chunks: first of `steps` K steps that chunk c of `chunks` sums.  The product passes 32
// bits from 14.7 million input columns on.
__host__ __device__ __forceinline__ int chunk_start(int steps, int c, int chunks) {
  return static_cast<int>(static_cast<long long>(steps) * c / chunks);
}

struct LinearI8Args {
  int M, N;              // tokens and output channels
  int kb_main, kb_total; // K blocks of the int8 operands; total with the adapter's
  int tiles_m, tiles_n;
  int bn;                // pair tile width along N: 256 or 128
  int stages;
  const float* x_scale;  // [M]
  const float* w_scale;  // [N]
  const float* m;        // [N], or null: g = 1
  const float* n;
  const __nv_bfloat16* bias;
  __nv_bfloat16* y;      // [M, N]
  long long wait_limit;
  int* status;
};

// Eight neighbouring floats of shared memory (16-byte aligned).
__device__ __forceinline__ void ld_shared8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Synchronises the eight epilogue warps.
__device__ __forceinline__ void epi_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kI8EpiThreads) : "memory");
}

// Transposes the 16-byte pieces of four neighbouring lanes: lane i of a quad
// ends with every lane's piece i, c[j] being lane j's.  A thread of the epilogue
// has a row of its tile; stored as it is, each store touches 32 rows, 16 bytes
// of each, and takes the memory pipeline 32 passes.  Transposed, a store
// touches 64 bytes of 8 rows.
__device__ __forceinline__ void quad_transpose(uint4 (&c)[4], int lane) {
  const auto swap = [&](uint4& lo, uint4& hi, bool upper, int o) {
    // the upper lane of the two gives its lo for the lower one's hi
    const uint4 give = upper ? lo : hi;
    uint4 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, o);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, o);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, o);
    got.w = __shfl_xor_sync(0xffffffffu, give.w, o);
    if (upper)
      lo = got;
    else
      hi = got;
  };
  swap(c[0], c[1], lane & 1, 1);
  swap(c[2], c[3], lane & 1, 1);
  swap(c[0], c[2], lane & 2, 2);
  swap(c[1], c[3], lane & 2, 2);
}

// Stores the transposed pieces of a quad: lane i has piece i (16 bytes, 64 of
// them a row) of rows row4 .. row4 + 3; `at` is the address of its piece in
// row4, rows are `pitch` bytes apart.
__device__ __forceinline__ void quad_store(uint8_t* at, long long pitch, const uint4 (&c)[4], long long row4,
                                           int rows, bool col_ok) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col_ok && row4 + j < rows) *reinterpret_cast<uint4*>(at + j * pitch) = c[j];
}

// The pair GEMM of linear_tc.cuh (256 x 256 tiles, two K blocks per stage, the
// same barriers and ring) with the int8 base in TMEM columns 0..255 and the
// adapter in 256..511.  One tile's two accumulators fill the TMEM, so the next
// tile's base product waits for the epilogue; to keep that wait short the
// eight epilogue warps (two per lane quarter, 128 columns each) first pull
// their whole base part into registers and release it, then finish the tile
// beside the next main loop.  The next adapter product comes last in its tile,
// long after its accumulator has been read.  Tiles of 128 channels (each warp
// then has 64 of them) serve products whose 256-wide tiles leave half of the
// pairs without one.  Measured: 8192 x 8192 x 8192 at rank 384 in 439 us, 2.74
// P operations a second with P's launch, 516 us (2.33) at the clocks that the
// power limit leaves in a loop; 1000 x 4096 x 4096 in 16.9 us, of which the main
// loop is 10.3 (0.64 us a stage of 128 KB a pair) and the epilogue 3.3.
__global__ void __launch_bounds__(kI8Threads, 1)
    linear_i8_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmB,
                          const LinearI8Args a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_s - raw_s);
  float* cols = reinterpret_cast<float*>(smem + a.stages * kPairStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(cols) + kI8ColBytes);
  uint64_t* empty = full + a.stages;
  uint64_t* acc_full = empty + a.stages;
  uint64_t* base_empty = acc_full + 1;  // the even CTA's are used
  uint64_t* ext_empty = base_empty + 1;
  uint64_t* drain = ext_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1;
  const int n_pairs = gridDim.x >> 1;
  const long long limit = a.wait_limit;
  const int n_tiles = a.tiles_m * a.tiles_n;
  const bool has_ext = a.kb_total > a.kb_main;
  // bytes that both CTAs' copies bring per stage
  const uint32_t stage_tx = 2 * kPairKps * (kLinABytes + a.bn / 2 * 128u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(base_empty, 16);  // eight epilogue warps in each CTA of the pair
    mbar_init(ext_empty, 16);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * kPairBN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
  // without an adapter the launch before may be anything; with one it is P's,
  // which itself came after all others, and only P has to be waited for
  if (!has_ext) {
    grid_dep_wait();
    fence_proxy_async_all();
  }
  grid_dep_launch();

  if (warp < 4) {
    regs_give<kI8RegsFew>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      int stage = 0;
      uint32_t phase = 0;
      uint32_t parity_bits = 0;
      uint32_t filled_mask = 0;
      bool ext_ready = !has_ext;
      bool ok = true;
      for (int t = cid; t < n_tiles && ok; t += n_pairs) {
        int tm, tn;
        lin_tile_of(t, a.tiles_m, a.tiles_n, tm, tn);
        const int yx = tm * kPairBM + static_cast<int>(rank) * kLinBM;
        const int yw = tn * a.bn + static_cast<int>(rank) * (a.bn / 2);
        for (int kb0 = 0; kb0 < a.kb_total; kb0 += kPairKps) {
          if (kb0 + kPairKps > a.kb_main && !ext_ready) {
            grid_dep_wait();  // P comes from the launch before
            fence_proxy_async_all();
            ext_ready = true;
          }
          bool got = true;
          if (lane == 0) {
            got = mbar_wait(&empty[stage], phase ^ 1u, limit);
            if (got && leader) mbar_arrive_expect_tx(&full[stage], stage_tx);
            if (!got) lin_timeout(a.status, abort_flag);
          }
          got = __shfl_sync(0xffffffffu, got, 0);
          __syncwarp();
          if (!got) {
            ok = false;
            break;
          }
          const uint32_t dst = base_s + stage * kPairStageBytes;
          const uint32_t bar = full_leader + static_cast<uint32_t>(stage) * 8u;
          if (lane < 2 * kPairKps) {
            const bool w_side = lane >= kPairKps;
            const int kb = kb0 + (w_side ? lane - kPairKps : lane);
            // K blocks past kb_total lie wholly outside the tensor: zero-filled
            const bool ext = has_ext && kb >= a.kb_main;
            const int xk = ext ? (kb - a.kb_main) * kLinBK : kb * kI8BK;
            const CUtensorMap* map = w_side ? (ext ? &tmB : &tmW) : (ext ? &tmP : &tmX);
            tma_load_2d_pair(dst + lane * kLinABytes, map, bar, xk, w_side ? yw : yx);
          }
          parity_bits = (parity_bits & ~(1u << stage)) | (phase << stage);
          filled_mask |= 1u << stage;
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // never leave a TMA copy in flight: the even CTA's full barriers count both CTAs' bytes
      if (lane == 0 && leader)
        for (int s2 = 0; s2 < a.stages; ++s2)
          if ((filled_mask >> s2) & 1u) mbar_wait(&full[s2], (parity_bits >> s2) & 1u, limit);
    } else if (warp == 1) {
      // ------------------------------------------- MMA issuer (even CTA only)
      if (leader && lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t idesc_b = idesc_i8_s32(kPairBM, a.bn);
        const uint32_t idesc_e = idesc_bf16_f32(kPairBM, a.bn);
        const uint64_t desc0 = sw128_kmajor_desc(base_s);
        const uint64_t desc_step = kPairStageBytes >> 4;
        uint32_t it = 0;
        for (int t = cid; t < n_tiles && ok; t += n_pairs, ++it) {
          if (!mbar_wait(base_empty, (it & 1u) ^ 1u, limit)) {
            lin_timeout(a.status, abort_flag);
            break;
          }
          tc_fence_after();
          bool ext_free = false;
          for (int kb0 = 0; kb0 < a.kb_total; kb0 += kPairKps) {
            if (!mbar_wait(&full[stage], phase, limit)) {
              lin_timeout(a.status, abort_flag);
              ok = false;
              break;
            }
            if (has_ext && !ext_free && kb0 + kPairKps > a.kb_main) {
              if (!mbar_wait(ext_empty, (it & 1u) ^ 1u, limit)) {
                lin_timeout(a.status, abort_flag);
                ok = false;
                break;
              }
              ext_free = true;
            }
            tc_fence_after();
            const uint64_t adesc = desc0 + static_cast<uint64_t>(stage) * desc_step;
            const uint64_t bdesc = adesc + ((kPairKps * kLinABytes) >> 4);
#pragma unroll
            for (int i = 0; i < kPairKps; ++i) {
              const int kb = kb0 + i;
              const uint64_t ad = adesc + i * (kLinABytes >> 4), bd = bdesc + i * (kLinABytes >> 4);
              if (has_ext && kb >= a.kb_main) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_bf16_pair(tmem + kPairBN, ad + 2 * k, bd + 2 * k, idesc_e, (kb > a.kb_main || k > 0) ? 1u : 0u);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_i8_pair(tmem, ad + 2 * k, bd + 2 * k, idesc_b, (kb > 0 || k > 0) ? 1u : 0u);
              }
            }
            mma_commit_pair(&empty[stage], 0x3);
            if (++stage == a.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) mma_commit_pair(acc_full, 0x3);
        }
        mma_commit_pair(drain, 0x1);
        mbar_wait(drain, 0, limit);
      }
    }
  } else {
    regs_take<kI8RegsMany>();
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int width = a.bn / 2;
    const int first = ((warp - 4) >> 2) * width;  // columns first .. first + width - 1 of the tile
    const int et = threadIdx.x - 128;
    const uint32_t tmem_lane = tmem + (static_cast<uint32_t>(q * 32) << 16) + first;
    const uint32_t base_empty_leader = mapa_shared(smem_u32(base_empty), 0);
    const uint32_t ext_empty_leader = mapa_shared(smem_u32(ext_empty), 0);
    uint32_t it = 0;
    bool alive = true;  // a warp whose wait gave up still meets the others at epi_sync
    for (int t = cid; t < n_tiles; t += n_pairs, ++it) {
      int tm, tn;
      lin_tile_of(t, a.tiles_m, a.tiles_n, tm, tn);
      // this tile's column factors; the other half of the buffer may still be
      // read by warps finishing the tile before
      float* cf = cols + (it & 1u) * 3 * kPairBN;
      {
        const int c = tn * a.bn + et;
        float g = 0.f, sw = 0.f, b = 0.f;
        if (et < a.bn && c < a.N) {
          g = a.m ? __ldg(a.m + c) / __ldg(a.n + c) : 1.f;
          sw = __ldg(a.w_scale + c);
          if (a.bias) b = __bfloat162float(a.bias[c]);
        }
        cf[et] = sw * g;
        cf[kPairBN + et] = g;
        cf[2 * kPairBN + et] = b;
      }
      const long long row = static_cast<long long>(tm) * kPairBM + rank * kLinBM + q * 32 + lane;
      const bool row_ok = row < a.M;
      const float sx = row_ok ? __ldg(a.x_scale + row) : 0.f;
      epi_sync();
      if (alive && !mbar_wait_warp(acc_full, it & 1u, limit)) {
        if (lane == 0) lin_timeout(a.status, abort_flag);
        __syncwarp();
        alive = false;
      }
      if (!alive) continue;
      tc_fence_after();
      uint32_t acc[128];
      tmem_ld128(tmem_lane, acc);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(base_empty_leader);
      __syncwarp();
      const int col0 = tn * a.bn + first;
      const float* swg = cf + first;
      const int piece = lane & 3;
      const long long row4 = row - piece;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c * 32 >= width) break;
        float u[32];
        if (has_ext) {
          tmem_ld32(tmem_lane + kPairBN + c * 32, u);
          if (c == 3 || (c + 1) * 32 == width) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(ext_empty_leader);
          }
        }
        if (col0 + c * 32 >= a.N) continue;  // warp-uniform
        uint4 pk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float sw[8], g[8], o[8];
          const int k = c * 32 + j * 8;
          ld_shared8(swg + k, sw);
          ld_shared8(swg + 2 * kPairBN + k, o);
          if (has_ext) {
            ld_shared8(swg + kPairBN + k, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(g[e], u[j * 8 + e], o[e]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(static_cast<float>(static_cast<int>(acc[k + e])) * sx, sw[e], o[e]);
          pk[j].x = pack_bf16x2(o[0], o[1]);
          pk[j].y = pack_bf16x2(o[2], o[3]);
          pk[j].z = pack_bf16x2(o[4], o[5]);
          pk[j].w = pack_bf16x2(o[6], o[7]);
        }
        quad_transpose(pk, lane);
        const int col = col0 + c * 32 + piece * 8;
        quad_store(reinterpret_cast<uint8_t*>(a.y + row4 * a.N + col), a.N * 2ll, pk, row4, a.M, col < a.N);
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * kPairBN);
}

}  // namespace dora
