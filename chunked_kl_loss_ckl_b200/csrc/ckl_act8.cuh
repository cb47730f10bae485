// Activations kept in 8 bits between the forward and the backward pass.
//
// A row's elements are taken in groups of 32.  A group keeps one exponent byte
// b and per element an integer q of -127..127; the element's value is
// q 2^(b - 133).  b is the smallest one that holds the group's largest
// magnitude a: b = floor(log2 a) + 127 puts a / 2^(b - 133) in [64, 128), one
// more where that would round to 128.  Both scalings are powers of two, so the
// only rounding is the one to the integer (nearest, ties to even): an element
// is off by at most half a step, 2^(b - 134) <= a / 127.  Groups of 32 follow
// the outlier channels of a residual stream, which a scale per row would not;
// they cost 1/32 byte an element.  A power of two instead of a / 127 gives up
// half a bit on average, and makes the stored values the same whatever order
// or precision they were computed in; |q| <= 127 is exact in bf16.
// Subnormal groups use b = 0; b = 255 is never written (its values would pass
// the largest float), so the largest floats clamp to 127.  An element that is
// not finite is stored as q = -128 and read back as NaN, and does not count
// towards its group's scale.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace ckl {

constexpr int ACT8_GROUP = 32;
constexpr int ACT8_THREADS = 256;

// 2^k for k of normal floats.
__device__ __forceinline__ float pow2f(int k) {
  return __int_as_float((k + 127) << 23);
}

// Magnitude bits of x where it counts towards the group's scale (finite).
__device__ __forceinline__ uint32_t act8_mag(float x) {
  const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

// The exponent byte of a group whose largest magnitude has bits `a`: from
// 1.9921875 x 2^E on, a / 2^(E - 6) >= 127.5 rounds to 128.
__device__ __forceinline__ uint32_t act8_byte(uint32_t a) {
  const uint32_t b = (a >> 23) + ((a & 0x7FFFFFu) >= 0x7F0000u ? 1u : 0u);
  return b > 254u ? 254u : b;
}

// The two factors whose product is 2^(133 - b) (either alone may leave the
// range of normal floats).
struct Act8Scale {
  float f1, f2;
};
__device__ __forceinline__ Act8Scale act8_inv_scale(uint32_t b) {
  const int k = 133 - static_cast<int>(b), k1 = k >> 1;
  return {pow2f(k1), pow2f(k - k1)};
}
__device__ __forceinline__ Act8Scale act8_scale(uint32_t b) {
  const int k = static_cast<int>(b) - 133, k1 = k >> 1;
  return {pow2f(k1), pow2f(k - k1)};
}

// q in the low byte.  1.5 2^23 + v rounds v to the nearest integer, ties to
// even, and leaves its two's complement in the low bits (one FADD in place of
// a conversion, which the SM issues at an eighth of the rate).
__device__ __forceinline__ uint32_t act8_q(float x, Act8Scale s) {
  float v = x * s.f1 * s.f2;
  v = fminf(fmaxf(v, -127.f), 127.f);  // the largest floats only
  const uint32_t q = __float_as_uint(v + 12582912.f) & 0xFFu;
  return (__float_as_uint(x) & 0x7FFFFFFFu) < 0x7F800000u ? q : 0x80u;
}

// Byte j of the packed word as its value.  2^23 + (q + 128) is the float whose
// low byte is q ^ 0x80.
template <int J>
__device__ __forceinline__ float act8_value(uint32_t word, Act8Scale s) {
  const uint32_t w = word ^ 0x80808080u;
  const float f = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | J)) - 8388736.f;
  const float v = f * s.f1 * s.f2;
  return f == -128.f ? __int_as_float(0x7FC00000) : v;
}

__device__ __forceinline__ float act8_value1(int8_t q, Act8Scale s) {
  const float v = static_cast<float>(q) * s.f1 * s.f2;
  return q == -128 ? __int_as_float(0x7FC00000) : v;
}

// ------------------------------------------------------------ element access
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Eight consecutive elements as loaded: one 16-byte vector of bf16 or two of
// float.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = a;
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

// Eight elements of one lane to 8 bits; the four lanes of an aligned quad hold
// one group of 32 (all lanes of the warp take part).  Returns the exponent
// byte; q is the eight bytes.
__device__ __forceinline__ uint32_t act8_pack8(const float (&v)[8], uint2& q) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, act8_mag(v[j]));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  const uint32_t b = act8_byte(a);
  const Act8Scale s = act8_inv_scale(b);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = act8_q(v[4 * h], s) | (act8_q(v[4 * h + 1], s) << 8) | (act8_q(v[4 * h + 2], s) << 16) |
           (act8_q(v[4 * h + 3], s) << 24);
  q = make_uint2(w[0], w[1]);
  return b;
}

__device__ __forceinline__ void act8_unpack8(uint2 q, uint32_t b, float (&v)[8]) {
  const Act8Scale s = act8_scale(b);
  v[0] = act8_value<0>(q.x, s);
  v[1] = act8_value<1>(q.x, s);
  v[2] = act8_value<2>(q.x, s);
  v[3] = act8_value<3>(q.x, s);
  v[4] = act8_value<0>(q.y, s);
  v[5] = act8_value<1>(q.y, s);
  v[6] = act8_value<2>(q.y, s);
  v[7] = act8_value<3>(q.y, s);
}

// ------------------------------------------------------------------- kernels
// Rows of T x d elements, `units` units of a group (VEC: four lanes with eight
// elements each, d % 8 == 0 and 16-byte rows; otherwise a warp, an element a
// lane) taken in a grid-stride loop.  A thread's next unit is found from its
// last one by adding the stride's rows and groups, so that only the first
// costs a division.
struct Act8Pos {
  int64_t row;
  int32_t g;
  int64_t step_row;
  int32_t step_g;
  __device__ __forceinline__ Act8Pos(int64_t first, int64_t stride, int32_t groups)
      : row(first / groups), g(static_cast<int32_t>(first % groups)), step_row(stride / groups),
        step_g(static_cast<int32_t>(stride % groups)) {}
  __device__ __forceinline__ void next(int32_t groups) {
    row += step_row;
    g += step_g;
    if (g >= groups) {
      g -= groups;
      ++row;
    }
  }
};

template <typename TX, bool VEC>
__global__ void __launch_bounds__(ACT8_THREADS)
act8_pack_kernel(const TX* __restrict__ x, int64_t T, int32_t d, int32_t groups,
                 int8_t* __restrict__ q, uint8_t* __restrict__ e) {
  constexpr int LANES = VEC ? 4 : 32;  // lanes of a unit
  const int sub = threadIdx.x % LANES;
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * ACT8_THREADS + threadIdx.x;
  const int64_t nthr = static_cast<int64_t>(gridDim.x) * ACT8_THREADS;
  const int64_t units = T * groups;
  Act8Pos p(tid / LANES, nthr / LANES, groups);
  // whole warps take part in the group maxima: the loop runs while the
  // warp's first lane has a unit
  for (int64_t u = (tid & ~int64_t(31)) / LANES; u < units; u += nthr / LANES, p.next(groups)) {
    if constexpr (VEC) {
      const int32_t c = p.g * 32 + sub * 8;
      const bool on = p.row < T && c < d;
      Raw8<TX> r;
      r.clear();
      if (on) r.load(x + p.row * d + c);
      float v[8];
      r.get(v);
      uint2 qq;
      const uint32_t b = act8_pack8(v, qq);
      if (on) {
        *reinterpret_cast<uint2*>(q + p.row * d + c) = qq;
        if (sub == 0) e[p.row * groups + p.g] = static_cast<uint8_t>(b);
      }
    } else {
      const int32_t c = p.g * 32 + sub;
      const bool on = c < d;
      const float v = on ? to_f32(x[p.row * d + c]) : 0.f;
      const uint32_t b = act8_byte(__reduce_max_sync(0xffffffffu, act8_mag(v)));
      if (on) q[p.row * d + c] = static_cast<int8_t>(act8_q(v, act8_inv_scale(b)));
      if (sub == 0) e[p.row * groups + p.g] = static_cast<uint8_t>(b);
    }
  }
}

template <typename TX, bool VEC>
__global__ void __launch_bounds__(ACT8_THREADS)
act8_unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e, int64_t T,
                   int32_t d, int32_t groups, TX* __restrict__ x) {
  constexpr int LANES = VEC ? 4 : 32;
  const int sub = threadIdx.x % LANES;
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * ACT8_THREADS + threadIdx.x;
  const int64_t nthr = static_cast<int64_t>(gridDim.x) * ACT8_THREADS;
  const int64_t units = T * groups;
  Act8Pos p(tid / LANES, nthr / LANES, groups);
  for (int64_t u = tid / LANES; u < units; u += nthr / LANES, p.next(groups)) {
    if constexpr (VEC) {
      const int32_t c = p.g * 32 + sub * 8;
      if (c >= d) continue;
      float v[8];
      act8_unpack8(*reinterpret_cast<const uint2*>(q + p.row * d + c),
                   e[p.row * groups + p.g], v);
      Raw8<TX> r;
      r.set(v);
      r.store(x + p.row * d + c);
    } else {
      const int32_t c = p.g * 32 + sub;
      if (c < d)
        x[p.row * d + c] =
            from_f32<TX>(act8_value1(q[p.row * d + c], act8_scale(e[p.row * groups + p.g])));
    }
  }
}

}  // namespace ckl
