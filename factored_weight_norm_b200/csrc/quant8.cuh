// quant8.cuh - the 8-bit format of the activations and weights, and the
// kernels that write and read it.
//
// A stretch of values v (a whole row, or 128 columns of one) is kept as int8
// codes q with one fp32 scale:
//   top = max |v|,  scale = top / 127,  q = 127 v / top rounded to the nearest
//   integer, ties to even;  the value that is kept is q * scale.
// q is the rounding of the exact quotient, whatever the arithmetic: v * (127 /
// top) in one fused rounding is off by at most 127 * 2^-24 (the factor's own
// rounding), and a product that lands within kTieBand of a half is decided by
// exact arithmetic (codes_settle).
// A stretch below 2^-100 everywhere keeps zeros and the scale 0 (127 / top
// would leave fp32's range); one that holds an infinity or a NaN keeps the
// scale NaN, so that its values come back as NaN and not as numbers.
#pragma once

#include "compose.cuh"

namespace dora {

constexpr int kCkptBlock = 128;              // columns of a token that share a scale in a checkpoint
constexpr uint32_t kTopTiny = 0x0D800000u;   // 2^-100
constexpr uint32_t kTopInf = 0x7F800000u;
constexpr float kTieBand = 1e-5f;            // above 127 * 2^-24
constexpr float kRoundMagic = 12582912.f;    // 1.5 * 2^23: x + magic rounds x to an integer in the low bits

// For kernels that start under the launch before them (programmatic dependent
// launch): everything that reads or writes global memory comes after the whole
// of that launch, and the next launch may then be made ready in turn.  A launch
// that waits for its predecessor's end costs 3 to 4 us of an idle GPU here.
__device__ __forceinline__ void after_previous() {
  grid_dep_wait();
  grid_dep_launch();
}

// A maximum is kept as |v|'s bits: ordered as unsigned integers, NaN above infinity.
__device__ __forceinline__ bool top_kept(uint32_t top) { return top >= kTopTiny && top < kTopInf; }

__device__ __forceinline__ float top_inverse(uint32_t top) {
  return top_kept(top) ? 127.f / __uint_as_float(top) : 0.f;
}

__device__ __forceinline__ float top_scale(uint32_t top) {
  return top_kept(top) ? __uint_as_float(top) / 127.f : (top >= kTopInf ? __uint_as_float(0x7FC00000u) : 0.f);
}

// max(a, |b|, |c|) that keeps a NaN: its bits are then above infinity's.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int E>
__device__ __forceinline__ float max_abs(float a, const float (&v)[E]) {
  if constexpr (E == 1) {
    return max_abs(a, v[0], v[0]);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) a = max_abs(a, v[e], v[e + 1]);
    return a;
  }
}

// Codes of E values by inv = 127 / top, one in the low byte of each word;
// returns whether they are settled: not so if one of them lies too near a half
// for fp32 (inv is off by 2^-24 of itself, and each product meets one
// rounding) or is no number.
template <int E>
__device__ __forceinline__ bool codes_fast(const float (&v)[E], float inv, uint32_t (&q)[E]) {
  float rest[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float r = fmaf(v[e], inv, kRoundMagic);
    q[e] = __float_as_uint(r);
    rest[e] = fmaf(v[e], inv, kRoundMagic - r);
  }
  return max_abs<E>(0.f, rest) <= 0.5f - kTieBand;
}

// Settles the codes that codes_fast left open.  A product near the half
// h = k +- 1/2 is decided by the sign of 127 v - h top, which two-term products
// give exactly: a product's rounding error is a float (an fma finds it), the
// two leading terms are within a factor of two, so that their difference is
// exact, and the errors' difference has few enough bits to be exact as well.
// bf16 rows meet this often: their values are few, and v = top / 2 is a tie
// (one value in a thousand of a normal row), so it has to be cheap.
template <int E>
__device__ __forceinline__ void codes_settle(const float (&v)[E], uint32_t top, float inv, uint32_t (&q)[E]) {
  if (!top_kept(top)) {
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = 0;
    return;
  }
  float t = __uint_as_float(top);
  const float scale = t > 0x1p64f ? 0x1p-64f : 1.f;  // keeps 127 v in range; exact
  t *= scale;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float k = __uint_as_float(q[e]) - kRoundMagic;
    const float d = fmaf(v[e], inv, -k);
    if (fabsf(d) > 0.5f - kTieBand) {
      const float x = v[e] * scale, h = k + copysignf(0.5f, d);
      const float hi = 127.f * x, hh = h * t;
      const float past = copysignf(1.f, d) * ((hi - hh) + (fmaf(127.f, x, -hi) - fmaf(h, t, -hh)));
      if (past > 0.f || (past == 0.f && (q[e] & 1u))) q[e] += d > 0.f ? 1u : ~0u;
    }
  }
}

// Codes of E values that share (top, inv).
template <int E>
__device__ __forceinline__ void codes_of(const float (&v)[E], uint32_t top, float inv, uint32_t (&q)[E]) {
  if (!codes_fast<E>(v, inv, q)) codes_settle<E>(v, top, inv, q);
}

// Codes of bf16 values that share (top, inv): with 8 bits of v, 127 v / 256 is
// exact, so that one step of Markstein's correction (the quotient plus its
// exact remainder times the reciprocal; IBM J. Res. Dev. 34(1), 1990) gives the
// rounded quotient itself: a tie stays a tie and no other quotient of two bf16
// numbers is near one.  Without branches: ties are common here (v = top / 2 is
// one; one value in a thousand of a normal row), and settling them one by one
// took 91 us instead of 80.5 for 27648 rows of 5120.
template <int E>
__device__ __forceinline__ void codes_of_bf16(const float (&v)[E], uint32_t top, float inv, uint32_t (&q)[E]) {
  const bool kept = top_kept(top);
  const float t = __uint_as_float(top) * 0x1p-8f, back = kept ? 1.f / t : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float q0 = v[e] * inv;
    q[e] = __float_as_uint(fmaf(fmaf(-q0, t, v[e] * (127.f * 0x1p-8f)), back, q0) + kRoundMagic);
  }
  if (!kept) {
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = 0;
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

// VEC neighbouring values of a row that this kernel may write back in place (h
// over x or residual): coherent loads, since the non-coherent path holds only
// for memory that nothing writes while the kernel runs.
template <typename T, int VEC>
__device__ __forceinline__ typename VecIO<T, VEC>::Raw ld_row(const T* p) {
  if constexpr (VEC == 1) {
    return *p;
  } else {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
  }
}

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

// (sum, maximum) over the CTA's `warps` warps, the same bits in every thread:
// each warp leaves its own in shared memory and every thread adds them in order
// (a second round of shuffles would take longer).
struct RowsI8Shared {
  float sum[32];
  uint32_t top[32];
};
__device__ __forceinline__ void rows_i8_reduce(float& sum, uint32_t& top, RowsI8Shared& sh, int warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    sh.sum[warp] = sum;
    sh.top[warp] = top;
  }
  __syncthreads();  // every warp of the CTA; the compiler joins the lanes that the branch above parted
  top = __reduce_max_sync(0xffffffffu, lane < warps ? sh.top[lane] : 0u);
  float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int w = 0; w < warps; w += 4) {
    const float4 p = *reinterpret_cast<const float4*>(&sh.sum[w]);
    s4[0] += p.x;
    if (w + 1 < warps) s4[1] += p.y;
    if (w + 2 < warps) s4[2] += p.z;
    if (w + 3 < warps) s4[3] += p.w;
  }
  sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
}

// The row's factor 1 / sqrt(mean + eps); NaN where the squares left fp32's range,
// so that the row comes back neither as zeros nor as infinities: their sum past
// it, or mean + eps below its normal numbers (an eps of zero, or nearly, and
// values below 2^-63 or so).  A row of zeros (top, its largest |h * w|, is zero)
// stays zeros whatever eps.
__device__ __forceinline__ float rows_i8_rstd(float sum, uint32_t top, long long d, float eps) {
  const float ms = sum / static_cast<float>(d), t = ms + eps;
  if (ms < __uint_as_float(kTopInf)) {
    if (t >= 0x1p-126f) return 1.f / sqrtf(t);
    if (top == 0u) return 1.f;
  }
  return __uint_as_float(0x7FC00000u);
}

// One row in a thread's registers: NV vectors of VEC columns, `stride` columns
// apart.  All of a row's steps are written without branches (columns past the
// end are zeros that are not stored), so that the vectors overlap.
template <typename T, int VEC, int NV, bool HAS_W>
struct RowI8 {
  using IO = VecIO<T, VEC>;
  using Raw = typename IO::Raw;
  float v[NV][VEC];
  float sum, top;

  // h = x + residual (stored), v = h * w, and this thread's share of the sums
  __device__ __forceinline__ void take(const Raw (&x)[NV], const Raw (&r)[NV], const Raw (&w)[NV], bool has_res, T* h, int col, int stride, int d) {
    sum = top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      IO::unpack(x[i], v[i]);
      if (has_res) {
        float f[VEC];
        IO::unpack(r[i], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = round_to(v[i][e] + f[e], h);
        if (col + i * stride < d) IO::store(h + col + i * stride, v[i]);
      }
      if (HAS_W) {
        float f[VEC];
        IO::unpack(w[i], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          sum = fmaf(v[i][e], v[i][e], sum);
          v[i][e] *= f[e];
        }
      }
      top = max_abs<VEC>(top, v[i]);
    }
  }

  // codes by the row's maximum, and y
  __device__ __forceinline__ void give(uint32_t row_top, float inv, float rstd, int8_t* q, T* y, int col, int stride,
                                       int d) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t c[VEC];
      if constexpr (!HAS_W && sizeof(T) == 2)
        codes_of_bf16<VEC>(v[i], row_top, inv, c);
      else
        codes_of<VEC>(v[i], row_top, inv, c);
      if (col + i * stride < d) CodeIO<VEC>::store(q + col + i * stride, c);
    }
    if (y) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = v[i][e] * rstd;
        if (col + i * stride < d) IO::store(y + col + i * stride, o);
      }
    }
  }
};

// One CTA of at most MAXT threads per row, the row in registers.  Bound by
// memory: 8192 x 8192 bf16 with a residual and y (604 MB) takes 91.3 us, 6.6
// TB/s, the copy rate, since several rows of an SM cover one another's
// reductions; a ring of bulk copies that kept the next rows in flight took 110.
// One row of 8192 takes 3.5 us, most of it the launch and two trips to memory.
template <typename T, int VEC, int NV, int MAXT, bool HAS_W>
__global__ void __launch_bounds__(MAXT) rows_i8_kernel(const RowsI8Args a) {
  __shared__ __align__(16) RowsI8Shared sh;
  using IO = VecIO<T, VEC>;
  const long long off = static_cast<long long>(blockIdx.x) * a.d;
  const int d = static_cast<int>(a.d), col = threadIdx.x * VEC, stride = blockDim.x * VEC;
  const bool has_res = a.residual != nullptr;
  after_previous();
  typename IO::Raw x[NV], r[NV], w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = r[i] = w[i] = typename IO::Raw{};
    if (col + i * stride < d) {
      x[i] = ld_row<T, VEC>(static_cast<const T*>(a.x) + off + col + i * stride);
      if (has_res) r[i] = ld_row<T, VEC>(static_cast<const T*>(a.residual) + off + col + i * stride);
      if (HAS_W) w[i] = IO::raw_param(static_cast<const T*>(a.weight) + col + i * stride);
    }
  }
  RowI8<T, VEC, NV, HAS_W> row;
  row.take(x, r, w, has_res, static_cast<T*>(a.h) + off, col, stride, d);
  float sum = row.sum;
  uint32_t top = __float_as_uint(row.top);
  rows_i8_reduce(sum, top, sh, blockDim.x >> 5);
  const float rstd = HAS_W ? rows_i8_rstd(sum, top, a.d, a.eps) : 1.f;
  if (threadIdx.x == 0) a.scale[blockIdx.x] = top_scale(top) * rstd;
  row.give(top, top_inverse(top), rstd, a.q + off, a.y ? static_cast<T*>(a.y) + off : nullptr, col, stride, d);
}

// Rows longer than a CTA's registers hold: the row is read twice, the second
// time as written (h) where there is a residual.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) rows_i8_long_kernel(const RowsI8Args a) {
  __shared__ __align__(16) RowsI8Shared sh;
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.d;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.d : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  T* h = static_cast<T*>(a.h) + row * a.d;
  after_previous();
  float sum = 0.f, top_f = 0.f;
  for (long long col = static_cast<long long>(threadIdx.x) * VEC; col < a.d;
       col += static_cast<long long>(blockDim.x) * VEC) {
    float v[VEC];
    VecIO<T, VEC>::unpack(ld_row<T, VEC>(x + col), v);
    if (res) {
      float r[VEC];
      VecIO<T, VEC>::unpack(ld_row<T, VEC>(res + col), r);
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
    top_f = max_abs<VEC>(top_f, v);
  }
  uint32_t top = __float_as_uint(top_f);
  rows_i8_reduce(sum, top, sh, blockDim.x >> 5);
  const float rstd = w ? rows_i8_rstd(sum, top, a.d, a.eps) : 1.f;
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

// U rows of VEC neighbouring columns per thread and step, their loads issued
// together; VEC fills one 16-byte store (8 bf16, 4 fp32), so that a warp's
// stores are whole lines.  Measured at 8192 x 8192 to bf16 (201 MB): 31.7 us;
// one row a step 36.2, and 16 codes a thread (two half-line stores) 41.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) dequant_i8_kernel(const int8_t* __restrict__ q, const float* __restrict__ scale,
                                                         long long rows, long long cols, long long block,
                                                         long long blocks, T* __restrict__ out) {
  const long long col = (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x) * VEC;
  after_previous();
  if (col >= cols) return;
  const float* sc0 = scale + col / block;
  for (long long row = blockIdx.y * static_cast<long long>(U); row < rows; row += gridDim.y * static_cast<long long>(U)) {
    float sc[U];
    uint2 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row + u < rows) {
        const int8_t* src = q + (row + u) * cols + col;
        sc[u] = __ldg(sc0 + (row + u) * blocks);
        if constexpr (VEC == 8)
          w[u] = ld_stream_u2(src);
        else if constexpr (VEC == 4)
          w[u].x = ld_stream_u1(src);
        else
          w[u].x = static_cast<uint32_t>(static_cast<int32_t>(__ldg(src)));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row + u < rows) {
        T* dst = out + (row + u) * cols + col;
        if constexpr (VEC == 1) {
          st_value<T>(dst, static_cast<float>(static_cast<int32_t>(w[u].x)) * sc[u]);
        } else {
          float v[VEC], a[4];
          unpack_codes(w[u].x, a);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = a[e] * sc[u];
          if constexpr (VEC == 8) {
            unpack_codes(w[u].y, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 + e] = a[e] * sc[u];
          }
          VecIO<T, VEC>::store(dst, v);
        }
      }
    }
  }
}

}  // namespace dora
