// linear_ckpt8.cuh - the fused DoRA linear forward that keeps its product in 8
// bits for the backward, on tcgen05 tensor cores (sm_100a).
//
//   z = x W^T + P B^T,  P = s * x A^T       (the product, before g and b)
//   y = bf16(g * z + b),  z8, z_scale = 8-bit stretches of 128 columns of z
//
// The GEMM is linear_tc.cuh's pair GEMM with two changes that keep z near fp32's
// exactness, since its scales are returned in fp32:
//  * P = P_hi + P_lo, two bf16 matrices (the extension runs over both): off by
//    at most 2^-16 of P, to either side; one alone would move z by 2^-8 of the
//    adapter's share.
//  * The tensor core drops the bits below its accumulator as it adds, always
//    toward zero: over K = 8192 that took 8.5e-6 of the largest values of
//    signed operands (4.0e-6 at 4096) and 3.0e-5 of a sum of positive ones.  So
//    K is cut into chunks of at most kCkChunk stages (768 of K), each summed in
//    TMEM from zero, and the epilogue warps add the chunks in fp32 registers,
//    which round to nearest.  P's own sum over K runs in the same chunks
//    (linear_slice.cuh).
// Eight epilogue warps hold a 128 x 256 tile in 128 registers a thread; a
// thread's 128 columns of its row are one stretch, so the maximum and the
// codes come from registers without any exchange.  Two TMEM accumulators: the
// tensor core sums one chunk while the warps fetch the other, and a tile's
// last step overlaps the next tile's first two chunks.  Tiles of 128 columns
// (four of the warps then only keep step) serve products whose 256-wide tiles
// leave half of the pairs without one.  Measured: 8192 x 8192 x 8192 at rank
// 384 in 930 to 1030 us with P's launch and the reader's 31 (1.25 TFLOP with P's
// second half), bound by the tensor cores under the power limit; 1000 x 4096 x
// 4096 at rank 64 in 35 us, of which the main loop is 20 to 25 and the epilogue
// 4.2.
#pragma once

#include "linear_i8.cuh"
#include "quant8.cuh"

namespace dora {

constexpr int kCkChunk = 6;  // ring stages (of two 64-deep K blocks) summed in TMEM at a time

struct LinearCkptArgs {
  int M, N;
  int kb_main, kb_r;      // K blocks of x W^T and of each half of P B^T
  int tiles_m, tiles_n;
  int bn;                 // pair tile width along N: 256 or 128
  int stages;
  const float* m;
  const float* n;
  const __nv_bfloat16* bias;  // or null
  __nv_bfloat16* y;       // [M, N]
  int8_t* z8;             // [M, N]
  float* z_scale;         // [M, ceil(N / 128)]
  long long wait_limit;
  int* status;
};

__global__ void __launch_bounds__(kI8Threads, 1)
    linear_ckpt8_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                             const __grid_constant__ CUtensorMap tmHi, const __grid_constant__ CUtensorMap tmLo,
                             const __grid_constant__ CUtensorMap tmB, const LinearCkptArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_s - raw_s);
  float* cols = reinterpret_cast<float*>(smem + a.stages * kPairStageBytes);  // g, b of two tiles
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(cols) + kI8ColBytes);
  uint64_t* empty = full + a.stages;
  uint64_t* acc_full = empty + a.stages;  // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2], the even CTA's are used
  uint64_t* drain = acc_empty + 2;
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
  const int kb_total = a.kb_main + 2 * a.kb_r;
  const int n_stages = (kb_total + kPairKps - 1) / kPairKps;  // per tile
  const int n_chunks = (n_stages + kCkChunk - 1) / kCkChunk;

  // bytes that both CTAs' copies bring per stage
  const uint32_t stage_tx = 2 * kPairKps * (kLinABytes + a.bn / 2 * 128u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 16);  // eight epilogue warps in each CTA of the pair
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmHi);
    tma_prefetch_desc(&tmLo);
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
  if (a.kb_r == 0) {
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
      bool ext_ready = a.kb_r == 0;
      bool ok = true;
      for (int t = cid; t < n_tiles && ok; t += n_pairs) {
        int tm, tn;
        lin_tile_of(t, a.tiles_m, a.tiles_n, tm, tn);
        const int yx = tm * kPairBM + static_cast<int>(rank) * kLinBM;
        const int yw = tn * a.bn + static_cast<int>(rank) * (a.bn / 2);
        for (int kb0 = 0; kb0 < kb_total; kb0 += kPairKps) {
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
            const bool ext = a.kb_r > 0 && kb >= a.kb_main;
            const bool lo = ext && kb >= a.kb_main + a.kb_r;
            const int xk = (kb - (ext ? a.kb_main : 0) - (lo ? a.kb_r : 0)) * kLinBK;
            const CUtensorMap* map = w_side ? (ext ? &tmB : &tmW) : (lo ? &tmLo : (ext ? &tmHi : &tmX));
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
        const uint32_t idesc = idesc_bf16_f32(kPairBM, a.bn);
        const uint64_t desc0 = sw128_kmajor_desc(base_s);
        const uint64_t desc_step = kPairStageBytes >> 4;
        uint32_t it = 0;  // chunks so far
        for (int t = cid; t < n_tiles && ok; t += n_pairs) {
          for (int c = 0; c < n_chunks && ok; ++c, ++it) {
            const uint32_t ab = it & 1u;
            if (!mbar_wait(&acc_empty[ab], ((it >> 1) & 1u) ^ 1u, limit)) {
              lin_timeout(a.status, abort_flag);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem + ab * kPairBN;
            const int s0 = chunk_start(n_stages, c, n_chunks), s1 = chunk_start(n_stages, c + 1, n_chunks);
            for (int s = s0; s < s1; ++s) {
              if (!mbar_wait(&full[stage], phase, limit)) {
                lin_timeout(a.status, abort_flag);
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t adesc = desc0 + static_cast<uint64_t>(stage) * desc_step;
              const uint64_t bdesc = adesc + ((kPairKps * kLinABytes) >> 4);
#pragma unroll
              for (int i = 0; i < kPairKps; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_bf16_pair(d, adesc + i * (kLinABytes >> 4) + 2 * k, bdesc + i * (kLinABytes >> 4) + 2 * k, idesc,
                                (s > s0 || i > 0 || k > 0) ? 1u : 0u);
              mma_commit_pair(&empty[stage], 0x3);
              if (++stage == a.stages) {
                stage = 0;
                phase ^= 1u;
              }
            }
            if (ok) mma_commit_pair(&acc_full[ab], 0x3);
          }
        }
        mma_commit_pair(drain, 0x1);
        mbar_wait(drain, 0, limit);
      }
    }
  } else {
    regs_take<kI8RegsMany>();
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int half = (warp - 4) >> 2;  // columns half * 128 .. of the tile
    const bool mine = half * 128 < a.bn;
    const int et = threadIdx.x - 128;
    const uint32_t tmem_lane = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
    const uint32_t acc_empty_leader = mapa_shared(smem_u32(acc_empty), 0);
    const int blocks = (a.N + kCkptBlock - 1) / kCkptBlock;
    uint32_t it = 0, tile = 0;
    bool alive = true;  // a warp whose wait gave up still meets the others at epi_sync
    for (int t = cid; t < n_tiles; t += n_pairs, ++tile) {
      int tm, tn;
      lin_tile_of(t, a.tiles_m, a.tiles_n, tm, tn);
      // this tile's column factors; the other half of the buffer may still be
      // read by warps finishing the tile before
      float* cf = cols + (tile & 1u) * 3 * kPairBN;
      {
        const int c = tn * a.bn + et;
        float g = 0.f, b = 0.f;
        if (et < a.bn && c < a.N) {
          g = __ldg(a.m + c) / __ldg(a.n + c);
          if (a.bias) b = __bfloat162float(a.bias[c]);
        }
        cf[et] = g;
        cf[kPairBN + et] = b;
      }
      epi_sync();
      float v[128];
#pragma unroll
      for (int e = 0; e < 128; ++e) v[e] = 0.f;
#pragma unroll 1
      for (int c = 0; c < n_chunks; ++c, ++it) {
        const uint32_t ab = it & 1u;
        if (alive && !mbar_wait_warp(&acc_full[ab], (it >> 1) & 1u, limit)) {
          if (lane == 0) lin_timeout(a.status, abort_flag);
          __syncwarp();
          alive = false;
        }
        if (!alive) continue;
        tc_fence_after();
        if (mine) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t u[16];
            tmem_ld16(tmem_lane + ab * kPairBN + j * 16, u);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[j * 16 + e] += __uint_as_float(u[e]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_leader + ab * 8u);
      }
      const long long row = static_cast<long long>(tm) * kPairBM + rank * kLinBM + q * 32 + lane;
      const int col0 = tn * a.bn + half * 128;
      uint32_t open = 0;  // groups of eight codes that fp32 leaves open
      if (alive && mine && col0 < a.N) {  // warp-uniform
        // columns past N are sums of zero-filled operands: they do not count
        const uint32_t top = __float_as_uint(max_abs<128>(0.f, v));
        const float inv = top_inverse(top);
        if (row < a.M) a.z_scale[row * blocks + col0 / kCkptBlock] = top_scale(top);
        const float* gv = cf + half * 128;
        const int piece = lane & 3;
        const long long row4 = row - piece;
        uint4 zk[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (col0 + c * 32 >= a.N) {
            // pieces past N are transposed with the others and not stored
            zk[(c & 1) * 2] = zk[(c & 1) * 2 + 1] = make_uint4(0u, 0u, 0u, 0u);
          } else {
            uint4 pk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = c * 32 + j * 8;
              float z[8];
              uint32_t qc[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) z[e] = v[k + e];
              if (!codes_fast<8>(z, inv, qc)) open |= 1u << (k / 8);
              const uint32_t lo = pack_codes(qc[0], qc[1], qc[2], qc[3]), hi = pack_codes(qc[4], qc[5], qc[6], qc[7]);
              uint4& zp = zk[(c & 1) * 2 + j / 2];
              if (j & 1) {
                zp.z = lo;
                zp.w = hi;
              } else {
                zp.x = lo;
                zp.y = hi;
              }
              float g[8], b[8];
              ld_shared8(gv + k, g);
              ld_shared8(gv + kPairBN + k, b);
#pragma unroll
              for (int e = 0; e < 8; ++e) z[e] = fmaf(g[e], z[e], b[e]);
              pk[j].x = pack_bf16x2(z[0], z[1]);
              pk[j].y = pack_bf16x2(z[2], z[3]);
              pk[j].z = pack_bf16x2(z[4], z[5]);
              pk[j].w = pack_bf16x2(z[6], z[7]);
            }
            __syncwarp();
            quad_transpose(pk, lane);
            const int col = col0 + c * 32 + piece * 8;
            quad_store(reinterpret_cast<uint8_t*>(a.y + row4 * a.N + col), a.N * 2ll, pk, row4, a.M, col < a.N);
          }
          if (c & 1) {  // 64 codes a row are whole
            __syncwarp();
            quad_transpose(zk, lane);
            const int col = col0 + (c - 1) * 32 + piece * 16;
            int8_t* at = a.z8 + row4 * a.N + col;
            if (a.N % 16 == 0) {
              quad_store(reinterpret_cast<uint8_t*>(at), a.N, zk, row4, a.M, col < a.N);
            } else {  // rows start on 8 bytes, and the last piece may be half a one
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (row4 + j < a.M) {
                  if (col < a.N) *reinterpret_cast<uint2*>(at + static_cast<long long>(j) * a.N) = make_uint2(zk[j].x, zk[j].y);
                  if (col + 8 < a.N)
                    *reinterpret_cast<uint2*>(at + static_cast<long long>(j) * a.N + 8) = make_uint2(zk[j].z, zk[j].w);
                }
            }
          }
        }
      }
      // settled here, by one piece of code behind the stores, and stored again:
      // inlined sixteen times it made the epilogue's code too long for the
      // instruction cache
      __syncwarp();  // the quad's stores come first
      if (open != 0 && row < a.M) {
        const uint32_t top = __float_as_uint(max_abs<128>(0.f, v));
        const float inv = top_inverse(top);
#pragma unroll 1
        for (; open != 0; open &= open - 1) {
          const int k = (__ffs(open) - 1) * 8;
          float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          uint32_t qc[8];
#pragma unroll
          for (int g = 0; g < 16; ++g)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = k == g * 8 ? v[g * 8 + e] : z[e];
          codes_fast<8>(z, inv, qc);
          codes_settle<8>(z, top, inv, qc);
          if (col0 + k < a.N)
            *reinterpret_cast<uint2*>(a.z8 + row * a.N + col0 + k) = make_uint2(
                pack_codes(qc[0], qc[1], qc[2], qc[3]), pack_codes(qc[4], qc[5], qc[6], qc[7]));
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * kPairBN);
}

}  // namespace dora
