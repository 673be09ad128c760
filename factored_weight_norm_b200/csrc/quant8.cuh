// quant8.cuh - the 8-bit format of the activations and weights, and the
// kernels that write and read it.
//
// A stretch of values v (a whole row, or 128 columns of one) is kept as int8
// codes q with one fp32 scale:
//   top = max |v|,  scale = top / 127,  q = 127 v / top rounded to the nearest
//   integer, ties to even;  the value that is kept is q * scale.
// q is the rounding of the exact quotient, whatever the arithmetic: the fp32
// product v * (127 / top) is off by at most 127 * 2^-23, and a product that
// lands within kTieBand of a half is rounded again in fp64 (127 v is exact
// there, and an fp64 quotient cannot cross a half that an fp32 ratio missed).
// A stretch below 2^-100 everywhere keeps zeros and the scale 0 (127 / top
// would leave fp32's range); one that holds an infinity or a NaN keeps the
// scale NaN, so that its values come back as NaN and not as numbers.
#pragma once

#include "compose.cuh"

namespace dora {

constexpr int kCkptBlock = 128;              // columns of a token that share a scale in a checkpoint
constexpr uint32_t kTopTiny = 0x0D800000u;   // 2^-100
constexpr uint32_t kTopInf = 0x7F800000u;
constexpr float kTieBand = 3e-5f;            // above 127 * 2^-23
constexpr float kRoundMagic = 12582912.f;    // 1.5 * 2^23: x + magic rounds x to an integer in the low bits

// |v| as bits: ordered as unsigned integers, NaN above infinity, so that an
// integer maximum never loses one.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ bool top_kept(uint32_t top) { return top >= kTopTiny && top < kTopInf; }

__device__ __forceinline__ float top_inverse(uint32_t top) {
  return top_kept(top) ? 127.f / __uint_as_float(top) : 0.f;
}

__device__ __forceinline__ float top_scale(uint32_t top) {
  return top_kept(top) ? __uint_as_float(top) / 127.f : (top >= kTopInf ? __uint_as_float(0x7FC00000u) : 0.f);
}

// Codes of E values that share (top, inv), one in the low byte of each word.
// Values of a stretch that keeps no codes (inv == 0) give zeros.
template <int E>
__device__ __forceinline__ void codes_of(const float (&v)[E], uint32_t top, float inv, uint32_t (&q)[E]) {
  bool near = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float r = fmaf(v[e], inv, kRoundMagic);
    q[e] = __float_as_uint(r);
    near = near || fabsf(fmaf(v[e], inv, -(r - kRoundMagic))) > 0.5f - kTieBand;
  }
  if (inv == 0.f) {
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = 0;
  } else if (near) {  // about one value in 10^4
    const double d = static_cast<double>(__uint_as_float(top));
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
      float ve = 0.f;
#pragma unroll
      for (int k = 0; k < E; ++k) ve = k == e ? v[k] : ve;
      const uint32_t qe = static_cast<uint32_t>(__double2int_rn(127.0 * static_cast<double>(ve) / d));
#pragma unroll
      for (int k = 0; k < E; ++k) q[k] = k == e ? qe : q[k];
    }
  }
}

// Low bytes of four words, the first lowest.
__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four codes as floats: the byte with its sign bit flipped, under the exponent
// of 2^23, is 2^23 + 128 + q.
__device__ __forceinline__ void unpack_codes(uint32_t w, float (&v)[4]) {
  const uint32_t u = w ^ 0x80808080u;
  v[0] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - 8388736.f;
  v[1] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - 8388736.f;
  v[2] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - 8388736.f;
  v[3] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - 8388736.f;
}

__device__ __forceinline__ uint2 ld_stream_u2(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t ld_stream_u1(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void st_stream_u2(void* p, uint2 v) {
  asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

// Codes of VEC neighbouring columns to and from memory.
template <int VEC>
struct CodeIO;
template <>
struct CodeIO<8> {
  static __device__ __forceinline__ void store(int8_t* p, const uint32_t (&q)[8]) {
    st_stream_u2(p, make_uint2(pack_codes(q[0], q[1], q[2], q[3]), pack_codes(q[4], q[5], q[6], q[7])));
  }
};
template <>
struct CodeIO<4> {
  static __device__ __forceinline__ void store(int8_t* p, const uint32_t (&q)[4]) {
    *reinterpret_cast<uint32_t*>(p) = pack_codes(q[0], q[1], q[2], q[3]);
  }
};
template <>
struct CodeIO<1> {
  static __device__ __forceinline__ void store(int8_t* p, const uint32_t (&q)[1]) {
    *p = static_cast<int8_t>(q[0]);
  }
};

// A sum rounded to the activation type, widened again.
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}
__device__ __forceinline__ float round_to(float v, const float*) { return v; }

// -------------------------------------------------- rows to codes, with a norm
// One CTA per row of d columns: h = x + residual in the activation type (the
// residual stream, written back), then
//   with a weight w: v = h * w, rstd = 1 / sqrt(mean(h^2) + eps);
//   without: v = h, rstd = 1;
//   top = max |v|, codes of v by top, scale = top / 127 * rstd, y = v * rstd.
// The row's norm is one factor of all its values, so it never enters the
// codes: they are exact in v, which for bf16 is an exact product in fp32.
struct RowsI8Args {
  const void* x;
  const void* residual;  // or null
  const void* weight;    // [d], or null: no norm
  void* h;               // written when there is a residual
  void* y;               // or null
  int8_t* q;
  float* scale;
  long long rows, d;
  float eps;
};

// (sum, maximum) over the CTA, the same bits in every thread.
__device__ __forceinline__ void rows_i8_reduce(float& sum, uint32_t& top, float* s_sum, uint32_t* s_top) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    s_sum[warp] = sum;
    s_top[warp] = top;
  }
  __syncthreads();
  sum = lane < warps ? s_sum[lane] : 0.f;
  top = lane < warps ? s_top[lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  top = __reduce_max_sync(0xffffffffu, top);
}

// The row's factor 1 / sqrt(mean + eps); NaN where the squares left fp32's
// range, so that the row does not come back as zeros.
__device__ __forceinline__ float rows_i8_rstd(float sum, long long d, float eps) {
  const float ms = sum / static_cast<float>(d);
  return ms < __uint_as_float(kTopInf) ? 1.f / sqrtf(ms + eps) : __uint_as_float(0x7FC00000u);
}

// NV vectors of VEC columns per thread, the row kept in registers.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024) rows_i8_kernel(const RowsI8Args a) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.d;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.d : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  float v[NV][VEC];
  float sum = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const long long col = (static_cast<long long>(i) * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
    if (col < a.d) {
      VecIO<T, VEC>::unpack(VecIO<T, VEC>::raw(x + col), v[i]);
      if (res) {
        float r[VEC];
        VecIO<T, VEC>::unpack(VecIO<T, VEC>::raw(res + col), r);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = round_to(v[i][e] + r[e], x);
        VecIO<T, VEC>::store(static_cast<T*>(a.h) + row * a.d + col, v[i]);
      }
      if (w) {
        float ww[VEC];
        VecIO<T, VEC>::unpack(VecIO<T, VEC>::raw_param(w + col), ww);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          sum = fmaf(v[i][e], v[i][e], sum);
          v[i][e] *= ww[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) top = max(top, abs_bits(v[i][e]));
  }
  rows_i8_reduce(sum, top, s_sum, s_top);
  const float rstd = w ? rows_i8_rstd(sum, a.d, a.eps) : 1.f;
  const float inv = top_inverse(top);
  if (threadIdx.x == 0) a.scale[row] = top_scale(top) * rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const long long col = (static_cast<long long>(i) * blockDim.x + threadIdx.x) * VEC;
    if (col < a.d) {
      uint32_t q[VEC];
      codes_of<VEC>(v[i], top, inv, q);
      CodeIO<VEC>::store(a.q + row * a.d + col, q);
      if (a.y) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= rstd;
        VecIO<T, VEC>::store(static_cast<T*>(a.y) + row * a.d + col, v[i]);
      }
    }
  }
}

// Rows longer than a CTA's registers hold: the row is read twice, the second
// time as written (h) where there is a residual.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) rows_i8_long_kernel(const RowsI8Args a) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.d;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.d : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  T* h = static_cast<T*>(a.h) + row * a.d;
  float sum = 0.f;
  uint32_t top = 0;
  for (long long col = static_cast<long long>(threadIdx.x) * VEC; col < a.d;
       col += static_cast<long long>(blockDim.x) * VEC) {
    float v[VEC];
    VecIO<T, VEC>::load(x + col, v);
    if (res) {
      float r[VEC];
      VecIO<T, VEC>::load(res + col, r);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = round_to(v[e] + r[e], x);
      VecIO<T, VEC>::store(h + col, v);
    }
    if (w) {
      float ww[VEC];
      VecIO<T, VEC>::unpack(VecIO<T, VEC>::raw_param(w + col), ww);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sum = fmaf(v[e], v[e], sum);
        v[e] *= ww[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) top = max(top, abs_bits(v[e]));
  }
  rows_i8_reduce(sum, top, s_sum, s_top);
  const float rstd = w ? rows_i8_rstd(sum, a.d, a.eps) : 1.f;
  const float inv = top_inverse(top);
  if (threadIdx.x == 0) a.scale[row] = top_scale(top) * rstd;
  for (long long col = static_cast<long long>(threadIdx.x) * VEC; col < a.d;
       col += static_cast<long long>(blockDim.x) * VEC) {
    float v[VEC];
    uint32_t q[VEC];
    // each thread reads back only what it wrote itself (plain loads)
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(res ? h[col + e] : x[col + e]);
    if (w) {
      float ww[VEC];
      VecIO<T, VEC>::unpack(VecIO<T, VEC>::raw_param(w + col), ww);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] *= ww[e];
    }
    codes_of<VEC>(v, top, inv, q);
    CodeIO<VEC>::store(a.q + row * a.d + col, q);
    if (a.y) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] *= rstd;
      VecIO<T, VEC>::store(static_cast<T*>(a.y) + row * a.d + col, v);
    }
  }
}

// --------------------------------------------------------------- codes to rows
// out = q * scale, one rounding to T; `block` columns share a scale.
template <typename T>
__device__ __forceinline__ void st_value(T* p, float v);
template <>
__device__ __forceinline__ void st_value<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void st_value<__nv_bfloat16>(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T, int VEC>
__global__ void __launch_bounds__(256) dequant_i8_kernel(const int8_t* __restrict__ q, const float* __restrict__ scale,
                                                         long long rows, long long cols, long long block,
                                                         long long blocks, T* __restrict__ out) {
  const long long col = (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x) * VEC;
  if (col >= cols) return;
  const long long b = col / block;
  for (long long row = blockIdx.y; row < rows; row += gridDim.y) {
    const float sc = __ldg(scale + row * blocks + b);
    const int8_t* src = q + row * cols + col;
    T* dst = out + row * cols + col;
    if constexpr (VEC == 8) {
      const uint2 w = ld_stream_u2(src);
      float v[8], u[4];
      unpack_codes(w.x, u);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = u[e] * sc;
      unpack_codes(w.y, u);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 + e] = u[e] * sc;
      if constexpr (sizeof(T) == 2) {
        VecIO<T, 8>::store(dst, v);
      } else {
        float lo[4], hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = v[e];
          hi[e] = v[4 + e];
        }
        VecIO<T, 4>::store(dst, lo);
        VecIO<T, 4>::store(dst + 4, hi);
      }
    } else {
      st_value<T>(dst, static_cast<float>(src[0]) * sc);
    }
  }
}

}  // namespace dora
