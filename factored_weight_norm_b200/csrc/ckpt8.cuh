// ckpt8.cuh - the compose forward that keeps its backward's input in 8 bits,
// and the backward that reads it.
//
// The compose backward needs the two activations only through
//   z = (base - b) + s * lora,   d_m = (sum_t dy * z) / n,
// so the forward keeps z alone, as int8 codes with one fp32 scale per token
// and 128 columns (quant8.cuh): 1.03 bytes an element instead of the 4 (bf16)
// or 8 (fp32) of base and lora.  A code is off by at most half its scale,
// top / 254; d_m sums many of them, d_base and d_lora do not depend on z.
//
// z is formed as fp32 (base - b) + (s * lora) with each operation rounded, so
// that the codes are those of the same expression anywhere else; y is
// compose_fwd_kernel's expression, bit for bit.
//
// Both kernels are bound by memory (bf16: 7.03 bytes an element each).  A
// group of lanes owns the 128 columns of a scale, so that their maximum is one
// warp reduction: 16 lanes of 8 bf16 (two groups a warp), or 32 lanes of 4
// fp32, neighbours where rows are whole 16-byte vectors, else 32 columns
// apart (4-byte accesses, still coalesced).
#pragma once

#include "quant8.cuh"

namespace dora {

// How the lanes of a warp cover a row's 128-column blocks.
struct LanesBf16 {
  using T = __nv_bfloat16;
  using Raw = uint4;
  static constexpr int kIndex = 0;
  static constexpr int kE = 8, kLanes = 16;
  static __device__ __forceinline__ int col(int gl, int e) { return gl * 8 + e; }
  static __device__ __forceinline__ bool any(int gl, long long left) { return gl * 8 < left; }
  static __device__ __forceinline__ Raw load(const T* p, int gl, long long) { return ld_stream_u4(p + gl * 8); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[8]) { VecIO<T, 8>::unpack(r, v); }
  static __device__ __forceinline__ void store(T* p, int gl, long long, const float (&v)[8]) {
    VecIO<T, 8>::store(p + gl * 8, v);
  }
  using Codes = uint2;
  static __device__ __forceinline__ Codes load_codes(const int8_t* p, int gl, long long) {
    return ld_stream_u2(p + gl * 8);
  }
  static __device__ __forceinline__ void unpack_code(const Codes& c, float (&v)[8]) {
    float lo[4], hi[4];
    unpack_codes(c.x, lo);
    unpack_codes(c.y, hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = lo[e];
      v[4 + e] = hi[e];
    }
  }
  static __device__ __forceinline__ void store_codes(int8_t* p, int gl, long long, const uint32_t (&q)[8]) {
    CodeIO<8>::store(p + gl * 8, q);
  }
};

struct LanesF32 {
  using T = float;
  using Raw = uint4;
  static constexpr int kIndex = 1;
  static constexpr int kE = 4, kLanes = 32;
  static __device__ __forceinline__ int col(int gl, int e) { return gl * 4 + e; }
  static __device__ __forceinline__ bool any(int gl, long long left) { return gl * 4 < left; }
  static __device__ __forceinline__ Raw load(const T* p, int gl, long long) { return ld_stream_u4(p + gl * 4); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[4]) { VecIO<T, 4>::unpack(r, v); }
  static __device__ __forceinline__ void store(T* p, int gl, long long, const float (&v)[4]) {
    VecIO<T, 4>::store(p + gl * 4, v);
  }
  using Codes = uint32_t;
  static __device__ __forceinline__ Codes load_codes(const int8_t* p, int gl, long long) {
    return ld_stream_u1(p + gl * 4);
  }
  static __device__ __forceinline__ void unpack_code(const Codes& c, float (&v)[4]) { unpack_codes(c, v); }
  static __device__ __forceinline__ void store_codes(int8_t* p, int gl, long long, const uint32_t (&q)[4]) {
    CodeIO<4>::store(p + gl * 4, q);
  }
};

// Any width and 4-byte alignment: columns gl, gl + 32, gl + 64, gl + 96.
struct LanesF32Any {
  using T = float;
  struct Raw {
    float v[4];
  };
  static constexpr int kIndex = 2;
  static constexpr int kE = 4, kLanes = 32;
  static __device__ __forceinline__ int col(int gl, int e) { return gl + 32 * e; }
  static __device__ __forceinline__ bool any(int gl, long long left) { return gl < left; }
  static __device__ __forceinline__ Raw load(const T* p, int gl, long long left) {
    Raw r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[e] = gl + 32 * e < left ? __ldg(p + gl + 32 * e) : 0.f;
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r.v[e];
  }
  static __device__ __forceinline__ void store(T* p, int gl, long long left, const float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (gl + 32 * e < left) p[gl + 32 * e] = v[e];
  }
  struct Codes {
    int8_t q[4];
  };
  static __device__ __forceinline__ Codes load_codes(const int8_t* p, int gl, long long left) {
    Codes c;
#pragma unroll
    for (int e = 0; e < 4; ++e) c.q[e] = gl + 32 * e < left ? __ldg(p + gl + 32 * e) : static_cast<int8_t>(0);
    return c;
  }
  static __device__ __forceinline__ void unpack_code(const Codes& c, float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(c.q[e]);
  }
  static __device__ __forceinline__ void store_codes(int8_t* p, int gl, long long left, const uint32_t (&q)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (gl + 32 * e < left) p[gl + 32 * e] = static_cast<int8_t>(q[e]);
  }
};

// ------------------------------------------------------------------ forward
// Four rows go through a group of lanes at a time.  Their maxima are reduced
// together: each of the first two exchange steps halves the rows that a lane
// still carries, so that the four reductions take 5 (16 lanes) or 6 (32)
// shuffles instead of 16 or 20, each lane ends with one row's maximum, and one
// division gives four rows' factors.  Measured at 8192 x 8192 bf16 (472 MB): 78
// us, 6.0 TB/s, with 0.62 of the issue slots used; per-row reductions and
// divisions took 36 instructions an element and 120 us.
constexpr int kCkptRows = 4;

// The row that a lane carries after the reduction, and a lane that carries row k.
template <int LANES>
__device__ __forceinline__ int row_of_lane(int gl) {
  return ((gl & (LANES / 2)) ? 2 : 0) | ((gl & (LANES / 4)) ? 1 : 0);
}
template <int LANES>
__device__ __forceinline__ int lane_of_row(int k) {
  return ((k & 2) ? LANES / 2 : 0) + ((k & 1) ? LANES / 4 : 0);
}

// Maximum over a group's lanes of row_of_lane(gl)'s value (bits ordered as integers).
template <int LANES>
__device__ __forceinline__ uint32_t reduce_rows(uint32_t mask, int gl, const uint32_t (&t)[4]) {
  const bool hi = gl & (LANES / 2), odd = gl & (LANES / 4);
  const uint32_t a0 = max(hi ? t[2] : t[0], __shfl_xor_sync(mask, hi ? t[0] : t[2], LANES / 2));
  const uint32_t a1 = max(hi ? t[3] : t[1], __shfl_xor_sync(mask, hi ? t[1] : t[3], LANES / 2));
  uint32_t b = max(odd ? a1 : a0, __shfl_xor_sync(mask, odd ? a0 : a1, LANES / 4));
#pragma unroll
  for (int o = LANES / 8; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(mask, b, o));
  return b;
}

template <typename L, bool HAS_BIAS>
__global__ void __launch_bounds__(256, 2) compose_fwd_ckpt8_kernel(
    const typename L::T* __restrict__ base, const typename L::T* __restrict__ lora,
    const typename L::T* __restrict__ bias, const float* __restrict__ m, const float* __restrict__ n, float s,
    long long tokens, long long d_out, long long blocks, typename L::T* __restrict__ y, int8_t* __restrict__ z8,
    float* __restrict__ z_scale) {
  constexpr int E = L::kE;
  const int gl = threadIdx.x % L::kLanes;
  const long long block = blockIdx.x * static_cast<long long>(blockDim.x / L::kLanes) + threadIdx.x / L::kLanes;
  const uint32_t group = L::kLanes == 32 ? 0xFFFFFFFFu : 0xFFFFu << (threadIdx.x & 16);
  after_previous();
  if (block >= blocks) return;  // a whole group of lanes
  const long long col0 = block * kCkptBlock;
  const long long left = d_out - col0;
  const bool any = L::any(gl, left);
  float delta[E], gs[E], bb[HAS_BIAS ? E : 1];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = L::col(gl, e);
    const bool ok = c < left;
    const float mm = ok ? __ldg(m + col0 + c) : 1.f, nn = ok ? __ldg(n + col0 + c) : 1.f;
    delta[e] = (mm - nn) / nn;
    gs[e] = (mm / nn) * s;
    if (HAS_BIAS) bb[e] = ok ? ld_param(bias + col0 + c) : 0.f;
  }
  const int my_row = row_of_lane<L::kLanes>(gl);
  typename L::Raw rb[kCkptRows], rl[kCkptRows];
  const auto fetch = [&](long long row) {
#pragma unroll
    for (int k = 0; k < kCkptRows; ++k) {
      rb[k] = typename L::Raw{};
      rl[k] = typename L::Raw{};
      if (any && row + k < tokens) {
        rb[k] = L::load(base + (row + k) * d_out + col0, gl, left);
        rl[k] = L::load(lora + (row + k) * d_out + col0, gl, left);
      }
    }
  };
  // the CTAs of a strip take groups of rows in turn, so that at any time the
  // whole grid is on neighbouring rows
  const long long step = static_cast<long long>(gridDim.y) * kCkptRows;
  fetch(blockIdx.y * static_cast<long long>(kCkptRows));
  for (long long row = blockIdx.y * static_cast<long long>(kCkptRows); row < tokens; row += step) {
    const long long at = row * d_out + col0;
    const int rows = static_cast<int>(min(static_cast<long long>(kCkptRows), tokens - row));
    float z[kCkptRows][E];
    uint32_t tops[kCkptRows];
#pragma unroll
    for (int k = 0; k < kCkptRows; ++k) {
      float b[E], l[E], o[E];
      L::unpack(rb[k], b);
      L::unpack(rl[k], l);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float inner = HAS_BIAS ? b[e] - bb[e] : b[e];
        o[e] = b[e] + fmaf(delta[e], inner, gs[e] * l[e]);
        z[k][e] = __fadd_rn(inner, __fmul_rn(s, l[e]));
      }
      // a lane wholly past the end has zeros for base and lora, but a bias must not count there either
      tops[k] = any ? __float_as_uint(max_abs<E>(0.f, z[k])) : 0u;
      if (any && k < rows) L::store(y + at + k * d_out, gl, left, o);
    }
    fetch(row + step);  // in flight under the reduction and the codes
    const uint32_t my_top = reduce_rows<L::kLanes>(group, gl, tops);
    const float my_inv = top_inverse(my_top);
    if ((gl & (L::kLanes / 4 - 1)) == 0 && my_row < rows) z_scale[(row + my_row) * blocks + block] = top_scale(my_top);
    bool settled = true;
#pragma unroll
    for (int k = 0; k < kCkptRows; ++k) {
      const float inv = __shfl_sync(group, my_inv, lane_of_row<L::kLanes>(k), L::kLanes);
      uint32_t q[E];
      settled = codes_fast<E>(z[k], inv, q) && settled;
      if (any && k < rows) L::store_codes(z8 + at + k * d_out, gl, left, q);
    }
    if (!__all_sync(group, settled)) {
#pragma unroll 1
      for (int k = 0; k < rows; ++k) {
        const uint32_t top = __shfl_sync(group, my_top, lane_of_row<L::kLanes>(k), L::kLanes);
        float zk[E];
        uint32_t q[E];
#pragma unroll
        for (int e = 0; e < E; ++e) zk[e] = k == 0 ? z[0][e] : (k == 1 ? z[1][e] : (k == 2 ? z[2][e] : z[3][e]));
        const float inv = top_inverse(top);
        if (!codes_fast<E>(zk, inv, q)) {
          codes_settle<E>(zk, top, inv, q);
          if (any) L::store_codes(z8 + at + k * d_out, gl, left, q);
        }
        __syncwarp(group);
      }
    }
  }
}

// ----------------------------------------------------------------- backward
// compose_bwd_kernel's schedule (compose.cuh) with z read from the codes: a
// CTA takes one 128-column strip of a share of the rows (a chunk: every n-th
// group of them), each thread carries its columns' sums in fp32, and the last
// CTA of a strip adds the chunks' sums in order.  Measured at 8192 x 8192 bf16
// (472 MB, 57 % of it written): 80 us, 5.9 TB/s; strips of four blocks took 82
// to 86, of eight 85 to 97, asynchronous copies through shared memory 79 to 90,
// three CTAs an SM 85 and more.  The next rows are in flight while these are
// multiplied and stored.
constexpr int kCkptBwdThreads = 256;
constexpr int kCkptBwdRows = 4;  // rows in flight per thread
constexpr int kCkptMaxChunks = 64;

template <typename L>
__global__ void __launch_bounds__(kCkptBwdThreads) compose_bwd_ckpt8_kernel(
    const typename L::T* __restrict__ dy, const int8_t* __restrict__ z8, const float* __restrict__ z_scale,
    const float* __restrict__ m, const float* __restrict__ n, float s, long long tokens, long long d_out,
    long long blocks, typename L::T* __restrict__ d_base, typename L::T* __restrict__ d_lora,
    float* __restrict__ partial, unsigned long long* __restrict__ marks, float* __restrict__ d_m,
    unsigned long long tag) {
  constexpr int E = L::kE;
  constexpr int kSlots = kCkptBwdThreads / L::kLanes;  // rows visited at once
  __shared__ float red[kSlots][kCkptBlock];
  const int gl = threadIdx.x % L::kLanes, slot = threadIdx.x / L::kLanes;
  const long long block = blockIdx.x;
  const long long col0 = block * kCkptBlock;
  const long long left = d_out - col0;
  after_previous();
  float g[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = L::col(gl, e);
    g[e] = c < left ? __ldg(m + col0 + c) / __ldg(n + col0 + c) : 0.f;
    acc[e] = 0.f;
  }
  if (L::any(gl, left)) {
    // the CTAs of a strip take groups of rows in turn, so that at any time the
    // whole grid is on neighbouring rows
    const long long step = gridDim.y * static_cast<long long>(kCkptBwdRows * kSlots);
    const long long first = blockIdx.y * static_cast<long long>(kCkptBwdRows * kSlots) + slot;
    typename L::Raw ra[kCkptBwdRows];
    typename L::Codes rz[kCkptBwdRows];
    float sc[kCkptBwdRows];
    const auto fetch = [&](long long row) {
#pragma unroll
      for (int u = 0; u < kCkptBwdRows; ++u) {
        const long long rr = row + u * kSlots;
        if (rr < tokens) {
          ra[u] = L::load(dy + rr * d_out + col0, gl, left);
          rz[u] = L::load_codes(z8 + rr * d_out + col0, gl, left);
          sc[u] = __ldg(z_scale + rr * blocks + block);
        }
      }
    };
    fetch(first);
    for (long long row = first; row < tokens; row += step) {
      typename L::Raw ca[kCkptBwdRows];
      typename L::Codes cz[kCkptBwdRows];
      float cs[kCkptBwdRows];
#pragma unroll
      for (int u = 0; u < kCkptBwdRows; ++u) {
        ca[u] = ra[u];
        cz[u] = rz[u];
        cs[u] = sc[u];
      }
      fetch(row + step);
#pragma unroll
      for (int u = 0; u < kCkptBwdRows; ++u) {
        const long long rr = row + u * kSlots;
        if (rr < tokens) {
          float a[E], z[E], db[E], dl[E];
          L::unpack(ca[u], a);
          L::unpack_code(cz[u], z);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            db[e] = g[e] * a[e];
            dl[e] = s * db[e];
            acc[e] = fmaf(a[e], z[e] * cs[u], acc[e]);
          }
          L::store(d_base + rr * d_out + col0, gl, left, db);
          L::store(d_lora + rr * d_out + col0, gl, left, dl);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) red[slot][L::col(gl, e)] = acc[e];
  __syncthreads();
  const int t = threadIdx.x;
  const bool t_ok = t < kCkptBlock && t < left;
  if (t_ok) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kSlots; ++w) sum += red[w][t];
    partial[blockIdx.y * d_out + col0 + t] = sum;
  }
  // Each CTA marks its chunk with this call's tag and then looks whether every
  // chunk of the strip carries it; the one whose mark comes last does (between
  // a CTA's mark and its look stands a sequentially consistent fence), and any
  // other that sees all marks writes the same values.  The marks need no
  // clearing before the launch, whatever the workspace held; they are wiped at
  // the end, so that a replay of the same launch starts clean.  (A tagged
  // counter per strip, raised by compare-and-swap, took 12 us of 17 at 512 x
  // 1024: 32 CTAs arrive at once and retry one after another.)
  __threadfence();
  __syncthreads();
  unsigned long long* strip_marks = marks + blockIdx.x * static_cast<long long>(kCkptMaxChunks);
  if (t == 0) *reinterpret_cast<volatile unsigned long long*>(strip_marks + blockIdx.y) = tag;
  asm volatile("fence.sc.gpu;" ::: "memory");
  __syncthreads();
  asm volatile("fence.sc.gpu;" ::: "memory");
  const bool seen = t >= static_cast<int>(gridDim.y) ||
                    *reinterpret_cast<volatile unsigned long long*>(strip_marks + t) == tag;
  if (__syncthreads_and(seen)) {
    __threadfence();
    if (t_ok) {
      float total = 0.f;  // in chunk order, the loads of 16 chunks at a time
      for (unsigned k = 0; k < gridDim.y; k += 16) {
        float p[16];
#pragma unroll
        for (unsigned j = 0; j < 16; ++j) p[j] = k + j < gridDim.y ? __ldcg(&partial[(k + j) * d_out + col0 + t]) : 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) total += p[j];
      }
      d_m[col0 + t] = total / __ldg(n + col0 + t);
    }
    if (t < static_cast<int>(gridDim.y)) strip_marks[t] = 0;
  }
}

}  // namespace dora
