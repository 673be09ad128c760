// linear_slice.cuh - the int8 DoRA linear and its adapter's down projection
// for few tokens, on tcgen05 tensor cores (sm_100a).
//
// With few tokens the product reads the whole weight for little arithmetic:
// it is bound by memory, and what matters is that every SM streams.  So the
// weight's rows are the MMA's M side (128 of them a tile) and the tokens its N
// side (BN = 16 to 128 of them), and K is split over a cluster of up to 8 CTAs
// until the grid fills two CTAs an SM; each CTA streams its slice of 128
// weight rows through a ring of TMA boxes (about 100 KB in flight).  The
// splits meet in distributed shared memory: each CTA puts its partial tile
// into its own (the ring is free by then), and each finishes its share of the
// tokens from all of them.  int32 partial sums are exact in any order; the
// adapter's product lies wholly in the last split, so its fp32 sum is one
// CTA's; the fp32 sums of the down projection are added in split order, so P's
// last bits depend on the number of splits, and with it on the batch.
// The meeting is what costs beyond the stream: it is done once for the whole
// tile, by all warps, with the loads from all splits in flight together (in
// two rounds of 64 tokens by four warps, split after split, 128 tokens took 10
// of 25 us).  Measured at 8192 x 8192 without an adapter: one token 15.2 us (67
// MB streamed in 10, 6 TB/s or more; 2.5 to the first bytes, 2.5 to join; 0.4 for
// the proxy fence before them), 128 tokens 21.1.
#pragma once

#include "linear_i8.cuh"
#include "quant8.cuh"

namespace dora {

constexpr int kSlThreads = 192;  // producer, MMA issuer, four epilogue warps
constexpr int kSlMaxStages = 8;
// alignment; row factors (sw * g, g, b) and token scales; barriers
constexpr size_t kSlFixed = 1024 + (3 * kLinBM + 128) * 4 + 256;

// Shared memory of a CTA: two fit on an SM, or one with a ring of twice the
// depth (200 KB): for the product of 128 tokens, whose exchange (int32 sums and
// the adapter's fp32 beside them) takes 128 KB, and for a grid so small that
// its CTAs have an SM each anyway.
constexpr size_t kSlSmemTwo = 112 * 1024, kSlSmemOne = 200 * 1024;
__host__ __device__ constexpr uint32_t slice_stage_bytes(int bn) { return kLinABytes + bn * 128u; }

struct SliceArgs {
  int rows;               // weight rows (d_out; r for the down projection)
  int tokens;
  int kb_main, kb_total;  // K blocks; total with the adapter's
  int stages;             // of the ring
  const float* x_scale;   // I8: as in LinearI8Args
  const float* w_scale;
  const float* m;
  const float* n;
  const __nv_bfloat16* bias;
  int chunk;              // !I8: K blocks that one TMEM sum takes at most
  float alpha;            // !I8: scale of the product
  __nv_bfloat16* out;     // [tokens, rows]
  __nv_bfloat16* out_lo;  // !I8: what the output's rounding leaves, or null
  long long wait_limit;
  int* status;
};

// First K block of split i of `splits`: even shares of all blocks, but every
// split keeps a main block and the adapter's blocks all go to the last.
__device__ __forceinline__ int slice_start(const SliceArgs& a, int i, int splits) {
  if (i == splits) return a.kb_total;
  return min(static_cast<int>(static_cast<long long>(a.kb_total) * i / splits), a.kb_main - (splits - i));
}

__device__ __forceinline__ uint4 ld_cluster_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// D[tmem] (+)= A[smem] * B[smem]^T, signed 8-bit operands, int32 accumulation.
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                      uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// v = hi + lo: returns hi, a bf16 value, and what that leaves.  A finite v past
// bf16's largest number keeps that one (v may round to infinity, and the rest
// would be minus infinity); of an infinity nothing is left (and not NaN).
__device__ __forceinline__ float split_bf16(float v, float& lo) {
  constexpr float kBf16Max = 255.f * 0x1p120f, kInf = __builtin_huge_valf();
  const float hi = __bfloat162float(__float2bfloat16_rn(fabsf(v) < kInf ? fminf(fmaxf(v, -kBf16Max), kBf16Max) : v));
  lo = fabsf(v) == kInf ? 0.f : v - hi;
  return hi;
}

// One thread's share of the joined tile: eight rows (from `group`) of every
// token j with j % S == rank that falls to it, from the S splits' exchange
// areas ([token][128 rows] words; the adapter's behind them in the last one).
template <bool I8, int BN, int S>
__device__ __forceinline__ void slice_join(const SliceArgs& a, uint32_t area, const float* rowf, const float* sxs,
                                           uint32_t rank, int row0, int tok0, bool ext_any) {
  const int group = (threadIdx.x & 15) * 8;
  if (row0 + group >= a.rows) return;
  float swg[8], g[8], b[8];
  if (I8) {
    ld_shared8(rowf + group, swg);
    ld_shared8(rowf + kLinBM + group, g);
    ld_shared8(rowf + 2 * kLinBM + group, b);
  }
#pragma unroll (S == 1 ? 4 : 1)
  for (int j = (threadIdx.x >> 4) * S + static_cast<int>(rank); j < BN; j += (kSlThreads / 16) * S) {
    const int t = tok0 + j;
    if (t >= a.tokens) break;
    const uint32_t at = area + static_cast<uint32_t>(j) * 512u + static_cast<uint32_t>(group) * 4u;
    uint4 x[S][2], low[2];
#pragma unroll
    for (int p = 0; p < S; ++p) {
      const uint32_t from = mapa_shared(at, p);
      x[p][0] = ld_cluster_u4(from);
      x[p][1] = ld_cluster_u4(from + 16);
    }
    if (ext_any) {
      const uint32_t from = mapa_shared(at + BN * 512u, S - 1);
      low[0] = ld_cluster_u4(from);
      low[1] = ld_cluster_u4(from + 16);
    }
    float o[8];
    if (I8) {
      int sum[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0;
#pragma unroll
      for (int p = 0; p < S; ++p) {
        const uint32_t w[8] = {x[p][0].x, x[p][0].y, x[p][0].z, x[p][0].w, x[p][1].x, x[p][1].y, x[p][1].z, x[p][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += static_cast<int>(w[e]);
      }
      const float sx = sxs[j];
      const uint32_t w[8] = {low[0].x, low[0].y, low[0].z, low[0].w, low[1].x, low[1].y, low[1].z, low[1].w};
      // as linear_i8_pair_kernel's epilogue, operation by operation
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = ext_any ? fmaf(g[e], __uint_as_float(w[e]), b[e]) : b[e];
        o[e] = fmaf(static_cast<float>(sum[e]) * sx, swg[e], c);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
      for (int p = 0; p < S; ++p) {
        const uint32_t w[8] = {x[p][0].x, x[p][0].y, x[p][0].z, x[p][0].w, x[p][1].x, x[p][1].y, x[p][1].z, x[p][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += __uint_as_float(w[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= a.alpha;
    }
    const long long off = static_cast<long long>(t) * a.rows + row0 + group;
    if (!I8 && a.out_lo) {
      float rest[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = split_bf16(o[e], rest[e]);
      *reinterpret_cast<uint4*>(a.out_lo + off) = pack_bf16x8(rest);
    }
    *reinterpret_cast<uint4*>(a.out + off) = pack_bf16x8(o);
  }
}

// P = bf16(alpha * x A^T) for up to TOK tokens: one CTA per rank row, each
// thread eight columns at a time, fp32 sums joined in a fixed order.  The
// product behind it streams the base weight at the same time, and a slice
// kernel's 24 CTAs get little of the memory's attention beside its 256 (6 MB
// of A took 13 us, and the product then waited); these CTAs are many and small,
// and fit beside the product's.
constexpr int kDownThreads = 256;
template <int TOK>
__global__ void __launch_bounds__(kDownThreads) down_tokens_kernel(const __nv_bfloat16* __restrict__ x,
                                                                   const __nv_bfloat16* __restrict__ A, float alpha,
                                                                   int tokens, int d_in, int r,
                                                                   __nv_bfloat16* __restrict__ P) {
  __shared__ float part[kDownThreads / 32][TOK];
  grid_dep_launch();
  const __nv_bfloat16* row = A + static_cast<long long>(blockIdx.x) * d_in;
  float acc[TOK];
#pragma unroll
  for (int t = 0; t < TOK; ++t) acc[t] = 0.f;
#pragma unroll 4
  for (int k = threadIdx.x * 8; k < d_in; k += kDownThreads * 8) {
    float w[8];
    VecIO<__nv_bfloat16, 8>::unpack(ld_stream_u4(row + k), w);
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      if (t < tokens) {
        float v[8];
        VecIO<__nv_bfloat16, 8>::unpack(
            __ldg(reinterpret_cast<const uint4*>(x + static_cast<long long>(t) * d_in + k)), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[t] = fmaf(w[e], v[e], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TOK; ++t)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int t = 0; t < TOK; ++t) part[threadIdx.x >> 5][t] = acc[t];
  }
  __syncthreads();
  if (threadIdx.x < TOK && threadIdx.x < tokens) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kDownThreads / 32; ++w) sum += part[w][threadIdx.x];
    P[static_cast<long long>(threadIdx.x) * r + blockIdx.x] = __float2bfloat16_rn(alpha * sum);
  }
}

// I8: out = bf16(b + g * (sx sw * (W_q x_q^T) + B P^T)), tmW/tmX int8 and
// tmB/tmP the adapter's; else out = bf16(alpha * W x^T), all bf16, whose sum over
// K runs in chunks of a.chunk blocks: each in one of two TMEM accumulators, added
// by the epilogue warps in fp32 registers while the next one is summed.  (The
// tensor core drops bits toward zero as it adds; one chunk is the plain sum.)
template <bool I8, int BN>
__global__ void __launch_bounds__(kSlThreads, 2)
    linear_slice_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmP,
                        const SliceArgs a) {
  constexpr uint32_t kStageBytes = slice_stage_bytes(BN);
  constexpr uint32_t kColsTmem = 2 * BN;  // I8: the base and the adapter; else two chunks
  const int stages = a.stages;  // the host's: the exchange fits in the ring
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_s - raw_s);
  float* rowf = reinterpret_cast<float*>(smem + stages * kStageBytes);  // sw * g, g, b of the tile's rows
  float* sxs = rowf + 3 * kLinBM;                                        // the tokens' scales
  uint64_t* full = reinterpret_cast<uint64_t*>(sxs + 128);
  uint64_t* empty = full + stages;
  uint64_t* acc_full = empty + stages;  // [2], I8 uses one
  uint64_t* acc_empty = acc_full + 2;   // [2], for chunks
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t splits;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
  const uint32_t rank = cluster_ctarank();
  // clusters along x: all row tiles of a token tile, then the next token tile
  const unsigned tile = blockIdx.x / splits, row_tiles = (a.rows + kLinBM - 1) / kLinBM;
  const int row0 = static_cast<int>(tile % row_tiles) * kLinBM;
  const int tok0 = static_cast<int>(tile / row_tiles) * BN;
  const int kb0 = slice_start(a, static_cast<int>(rank), static_cast<int>(splits));
  const int kb1 = slice_start(a, static_cast<int>(rank) + 1, static_cast<int>(splits));
  const bool has_ext = I8 && kb1 > a.kb_main;
  const int n_chunks = I8 ? 1 : (kb1 - kb0 - 1) / a.chunk + 1;
  const long long limit = a.wait_limit;

  // K block kb into a stage of the ring
  const auto fill = [&](int stage, int kb) {
    const bool ext = I8 && kb >= a.kb_main;
    mbar_arrive_expect_tx(&full[stage], kStageBytes);
    const int xk = I8 && !ext ? kb * kI8BK : (ext ? kb - a.kb_main : kb) * kLinBK;
    const uint32_t dst = base_s + stage * kStageBytes;
    tma_load_2d(dst, ext ? &tmB : &tmW, &full[stage], xk, row0);
    tma_load_2d(dst + kLinABytes, ext ? &tmP : &tmX, &full[stage], xk, tok0);
  };
  // without an adapter the launch before may be anything; with one it is P's,
  // which itself came after all others, and only P has to be waited for
  const bool wait_all = I8 && a.kb_total == a.kb_main;
  // the first fills wait for nothing else, so they go out before the rest is set up
  const int early = min(stages, min(kb1, a.kb_main) - kb0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);  // the epilogue warps
    }
    fence_mbar_init();
    if (wait_all) {
      grid_dep_wait();
      fence_proxy_async_all();
    }
    for (int s = 0; s < early; ++s) fill(s, kb0 + s);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kColsTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (wait_all) grid_dep_wait();
  grid_dep_launch();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int filled = early, stage = early == stages ? 0 : early;
      uint32_t phase = early == stages ? 1u : 0u;
      for (int kb = kb0 + early; kb < kb1; ++kb, ++filled) {
        if (I8 && kb == a.kb_main) {
          grid_dep_wait();  // P comes from the launch before
          fence_proxy_async_all();
        }
        if (!mbar_wait(&empty[stage], phase ^ 1u, limit)) {
          atomicExch(a.status, 5);  // DORA_ERR_TIMEOUT
          break;
        }
        fill(stage, kb);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // never leave a TMA copy in flight: the last fill of every stage
      for (int f = max(0, filled - stages); f < filled; ++f)
        mbar_wait(&full[f % stages], static_cast<uint32_t>(f / stages & 1), limit);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc_m = I8 ? idesc_i8_s32(kLinBM, BN) : idesc_bf16_f32(kLinBM, BN);
      const uint32_t idesc_e = idesc_bf16_f32(kLinBM, BN);
      const uint64_t desc0 = sw128_kmajor_desc(base_s);
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      for (int c = 0; c < n_chunks && ok; ++c) {
        const int c0 = kb0 + chunk_start(kb1 - kb0, c, n_chunks), c1 = kb0 + chunk_start(kb1 - kb0, c + 1, n_chunks);
        const uint32_t d = tmem + (c & 1) * BN;
        if (!I8 && !mbar_wait(&acc_empty[c & 1], ((c >> 1) & 1u) ^ 1u, limit)) {
          atomicExch(a.status, 5);
          ok = false;
        }
        if (!I8) tc_fence_after();
        for (int kb = c0; kb < c1 && ok; ++kb) {
          if (!mbar_wait(&full[stage], phase, limit)) {
            atomicExch(a.status, 5);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc0 + static_cast<uint64_t>(stage) * (kStageBytes >> 4);
          const uint64_t bd = ad + (kLinABytes >> 4);
          const bool ext = I8 && kb >= a.kb_main;
          const int first = ext ? a.kb_main : c0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t acc = (kb > first || k > 0) ? 1u : 0u;
            if (ext)
              mma_bf16(tmem + BN, ad + 2 * k, bd + 2 * k, idesc_e, acc);
            else if (I8)
              mma_i8(tmem, ad + 2 * k, bd + 2 * k, idesc_m, acc);
            else
              mma_bf16(d, ad + 2 * k, bd + 2 * k, idesc_m, acc);
          }
          mma_commit(&empty[stage]);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        // after a wait that gave up the MMAs already issued must still end before TMEM is freed
        mma_commit(&acc_full[c & 1]);
        if (!ok) mbar_wait(&acc_full[c & 1], (c >> 1) & 1u, limit);
      }
    }
  }
  __syncwarp();

  // ---------------------------------------------------------------- exchange
  const bool ext_any = I8 && a.kb_total > a.kb_main;
  if (warp >= 2) {
    const int q = warp & 3;  // TMEM lane quarter
    if (I8) {
      const int et = static_cast<int>(threadIdx.x) - 64, c = row0 + et;
      float g = 0.f, sw = 0.f, b = 0.f;
      if (c < a.rows) {
        g = a.m ? __ldg(a.m + c) / __ldg(a.n + c) : 1.f;
        sw = __ldg(a.w_scale + c) * g;
        if (a.bias) b = __bfloat162float(a.bias[c]);
      }
      rowf[et] = sw;
      rowf[kLinBM + et] = g;
      rowf[2 * kLinBM + et] = b;
      if (et < BN) sxs[et] = tok0 + et < a.tokens ? __ldg(a.x_scale + tok0 + et) : 0.f;
      __syncwarp();
    }
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t* dst = reinterpret_cast<uint32_t*>(smem) + q * 32 + lane;
    bool alive = true;
    float v[I8 ? 1 : BN];  // !I8: the chunks' sum
    if (!I8) {
#pragma unroll
      for (int e = 0; e < BN; ++e) v[I8 ? 0 : e] = 0.f;
    }
#pragma unroll 1
    for (int c = 0; c < n_chunks && alive; ++c) {
      if (!mbar_wait_warp(&acc_full[c & 1], (c >> 1) & 1u, limit)) {
        if (lane == 0) atomicExch(a.status, 5);
        __syncwarp();
        alive = false;
        break;
      }
      tc_fence_after();
      if (!I8) {
#pragma unroll
        for (int j = 0; j < BN; j += 16) {
          if (tok0 + j < a.tokens) {  // warp-uniform
            uint32_t u[16];
            tmem_ld16(lane_addr + (c & 1) * BN + j, u);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[I8 ? 0 : j + e] += __uint_as_float(u[e]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[c & 1]);
        __syncwarp();
      }
    }
    // every MMA has ended: the ring is free
    if (alive && I8) {
#pragma unroll 4
      for (int j = 0; j < BN; j += 16) {
        if (tok0 + j >= a.tokens) break;  // warp-uniform
        uint32_t u[16];
        tmem_ld16(lane_addr + j, u);
#pragma unroll
        for (int e = 0; e < 16; ++e) dst[(j + e) * 128] = u[e];
        if (has_ext) {
          tmem_ld16(lane_addr + BN + j, u);
#pragma unroll
          for (int e = 0; e < 16; ++e) dst[(BN + j + e) * 128] = u[e];
        }
      }
    } else if (alive) {
#pragma unroll
      for (int e = 0; e < BN; ++e)
        if (tok0 + e < a.tokens) dst[e * 128] = __float_as_uint(v[I8 ? 0 : e]);
    }
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync_all();
  switch (splits) {
    case 1: slice_join<I8, BN, 1>(a, base_s, rowf, sxs, rank, row0, tok0, ext_any); break;
    case 2: slice_join<I8, BN, 2>(a, base_s, rowf, sxs, rank, row0, tok0, ext_any); break;
    case 4: slice_join<I8, BN, 4>(a, base_s, rowf, sxs, rank, row0, tok0, ext_any); break;
    default: slice_join<I8, BN, 8>(a, base_s, rowf, sxs, rank, row0, tok0, ext_any); break;
  }
  __syncwarp();  // the join's loops end at different tokens, and rows, for the lanes of a warp
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kColsTmem);
  cluster_sync_all();  // no CTA leaves while another reads its exchange area
}

}  // namespace dora
