// Activations kept in 8 bits between the forward and the backward pass.
//
// A row's elements are taken in groups of 32.  A group keeps one exponent byte
// b and per element an integer q of -127..127; the element's value is
// q 2^(b - 133).  b is the smallest one that holds the group's largest
// magnitude a: b = floor(log2 a) + 127 puts a / 2^(b - 133) in [64, 128), one
// more where that would round to 128.  Both scalings are powers of two, so the
// only rounding is the one to the integer (nearest, ties to even): an element
// is off by at most half a step, 2^(b - 134) <= max(a / 127, 2^-134).  Groups of
// 32 follow the outlier channels of a residual stream, which a scale per row would
// not; they cost 1/32 byte an element.  A power of two instead of a / 127 gives up
// half a bit on average, and makes the stored values the same whatever order
// or precision they were computed in; |q| <= 127 is exact in bf16.
// Subnormal groups use b = 0 (exact in bf16, whose values are multiples of 2^-133;
// fp32 magnitudes up to 2^-134 read back as 0); b = 255 is never written (its
// values would pass the largest float), so the largest floats clamp to 127.  An
// element that is not finite is stored as q = -128 and read back as NaN, and does
// not count towards its group's scale.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "ckl_bf16.cuh"

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
// 1.9921875 x 2^E on, a / 2^(E - 6) >= 127.5 rounds to 128, and the sum carries
// into the exponent.  Below 2^-126 a has no leading 1: a / 2^-133 is its bits /
// 2^16, which passes 127.5 half a step later.
__device__ __forceinline__ uint32_t act8_byte(uint32_t a) {
  const uint32_t b = (a + (a < 0x800000u ? 0x8000u : 0x10000u)) >> 23;
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
// even, and leaves its two's complement in the low bits (no conversion
// instruction, which the SM issues at an eighth of the rate).
__device__ __forceinline__ uint32_t act8_q(float x, Act8Scale s) {
  float v = x * s.f1 * s.f2;
  v = fminf(fmaxf(v, -127.f), 127.f);  // the largest floats only
  const uint32_t q = __float_as_uint(v + 12582912.f) & 0xFFu;
  return (__float_as_uint(x) & 0x7FFFFFFFu) < 0x7F800000u ? q : 0x80u;
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

// VEC elements of a row in registers: packed pairs of fp32 (for the two-lane
// instructions, which halve what a row costs to issue), or one float.
template <int VEC>
struct Lane {
  static constexpr int N = VEC / 2;
  using E = uint64_t;
  E e[N];
  __device__ __forceinline__ float get(int j) const {
    return (j & 1) ? f32x2_hi(e[j / 2]) : f32x2_lo(e[j / 2]);
  }
};
template <>
struct Lane<1> {
  static constexpr int N = 1;
  using E = float;
  E e[N];
  __device__ __forceinline__ float get(int) const { return e[0]; }
};
template <typename E>
__device__ __forceinline__ E both(float x);
template <>
__device__ __forceinline__ float both<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint64_t both<uint64_t>(float x) { return f32x2_pack(x, x); }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ uint64_t vadd(uint64_t a, uint64_t b) { return f32x2_add(a, b); }
__device__ __forceinline__ float vsub(float a, float b) { return a - b; }
__device__ __forceinline__ uint64_t vsub(uint64_t a, uint64_t b) { return f32x2_sub(a, b); }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ uint64_t vmul(uint64_t a, uint64_t b) { return f32x2_mul(a, b); }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ uint64_t vfma(uint64_t a, uint64_t b, uint64_t c) {
  return f32x2_fma(a, b, c);
}
__device__ __forceinline__ float vsum(float a) { return a; }
__device__ __forceinline__ float vsum(uint64_t a) { return f32x2_lo(a) + f32x2_hi(a); }

// 16 bytes of consecutive elements as they are in memory: eight bf16 or four
// floats.  (A float thread with eight would touch every 32-byte sector twice.)
template <typename T>
constexpr int VEC16 = 16 / static_cast<int>(sizeof(T));
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p) { a = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(void* p) const { *static_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
  // largest magnitude bits (as a float's), non-finite ones included
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t k = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
    return max(m & 0xFFFF0000u, m << 16);
  }
  __device__ __forceinline__ void get(Lane<8>& v) const {
    v.e[0] = bf16x2_widen(a.x);
    v.e[1] = bf16x2_widen(a.y);
    v.e[2] = bf16x2_widen(a.z);
    v.e[3] = bf16x2_widen(a.w);
  }
  __device__ __forceinline__ void set(const Lane<8>& v) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f32x2_lo(v.e[j]), f32x2_hi(v.e[j]));
      w[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Raw<float> {
  ulonglong2 a;
  __device__ __forceinline__ void load(const void* p) { a = *static_cast<const ulonglong2*>(p); }
  __device__ __forceinline__ void store(void* p) const { *static_cast<ulonglong2*>(p) = a; }
  __device__ __forceinline__ void clear() { a = make_ulonglong2(0ull, 0ull); }
  __device__ __forceinline__ uint32_t top() const {
    const uint64_t x = a.x & 0x7FFFFFFF7FFFFFFFull, y = a.y & 0x7FFFFFFF7FFFFFFFull;
    return max(max(static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32)),
               max(static_cast<uint32_t>(y), static_cast<uint32_t>(y >> 32)));
  }
  __device__ __forceinline__ void get(Lane<4>& v) const {
    v.e[0] = a.x;
    v.e[1] = a.y;
  }
  __device__ __forceinline__ void set(const Lane<4>& v) { a = make_ulonglong2(v.e[0], v.e[1]); }
};

// The 8-bit form of VEC elements: VEC bytes.
template <int VEC>
struct Bytes {
  uint32_t w[VEC / 4];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (VEC == 8) {
      const uint2 v = *static_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = *static_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (VEC == 8) *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *static_cast<uint32_t*>(p) = w[0];
  }
};

// VEC elements of one lane to 8 bits; 32 / VEC neighbouring lanes hold one
// group of 32 (all of them call it).  `top` is the lane's Raw::top().  Returns
// the exponent byte.  Where the group is finite and both 2^(133 - b) and the
// sums below are normal floats, one FMA scales and rounds an element:
// v 2^(133 - b) + 1.5 2^23 has the integer in its low byte.
template <int VEC>
__device__ __forceinline__ uint32_t act8_pack(const Lane<VEC>& v, uint32_t top, Bytes<VEC>& q) {
#pragma unroll
  for (int o = 1; o < 32 / VEC; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  uint32_t b = act8_byte(top);
  if (b >= 7u && b <= 253u && top < 0x7F800000u) {
    const uint64_t f = both<uint64_t>(pow2f(133 - static_cast<int>(b)));
    const uint64_t c = both<uint64_t>(12582912.f);
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h) {
      const uint64_t s = f32x2_fma(v.e[2 * h], f, c), t = f32x2_fma(v.e[2 * h + 1], f, c);
      q.w[h] = __byte_perm(
          __byte_perm(static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32), 0x0040),
          __byte_perm(static_cast<uint32_t>(t), static_cast<uint32_t>(t >> 32), 0x0040), 0x5410);
    }
  } else {  // the same in all of the group's lanes
    constexpr uint32_t LANES = 32 / VEC;
    const uint32_t mask = ((1u << LANES) - 1u) << (threadIdx.x & (32u - LANES));
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < VEC; ++j) a = max(a, act8_mag(v.get(j)));
#pragma unroll
    for (int o = 1; o < static_cast<int>(LANES); o <<= 1) a = max(a, __shfl_xor_sync(mask, a, o));
    b = act8_byte(a);
    const Act8Scale s = act8_inv_scale(b);
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h)
      q.w[h] = act8_q(v.get(4 * h), s) | (act8_q(v.get(4 * h + 1), s) << 8) |
               (act8_q(v.get(4 * h + 2), s) << 16) | (act8_q(v.get(4 * h + 3), s) << 24);
  }
  return b;
}

// The values of VEC bytes.  Where 2^(b - 133) and 2^23 times it are normal
// floats and no byte is -128, one FMA an element: (2^23 + 128 + q) s - (2^23 +
// 128) s, both products exact.
template <int VEC>
__device__ __forceinline__ void act8_unpack(const Bytes<VEC>& q, uint32_t b, Lane<VEC>& v) {
  uint32_t x[VEC / 4], nan = 0;
#pragma unroll
  for (int h = 0; h < VEC / 4; ++h) {
    x[h] = q.w[h] ^ 0x80808080u;  // q + 128: 0 marks a NaN
    nan |= (x[h] - 0x01010101u) & ~x[h];
  }
  if (b >= 7u && b <= 228u && (nan & 0x80808080u) == 0u) {
    const float s = pow2f(static_cast<int>(b) - 133);
    const uint64_t s2 = both<uint64_t>(s), c2 = both<uint64_t>(-8388736.f * s);
    const uint32_t k = 0x4B000000u;
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h) {
      v.e[2 * h] = f32x2_fma(f32x2_pack(__uint_as_float(__byte_perm(x[h], k, 0x7440)),
                                        __uint_as_float(__byte_perm(x[h], k, 0x7441))), s2, c2);
      v.e[2 * h + 1] = f32x2_fma(f32x2_pack(__uint_as_float(__byte_perm(x[h], k, 0x7442)),
                                            __uint_as_float(__byte_perm(x[h], k, 0x7443))), s2, c2);
    }
  } else {
    const Act8Scale s = act8_scale(b);
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const uint32_t w = q.w[j / 2] >> (16 * (j & 1));
      v.e[j] = f32x2_pack(act8_value1(static_cast<int8_t>(w & 0xFFu), s),
                          act8_value1(static_cast<int8_t>((w >> 8) & 0xFFu), s));
    }
  }
}

// ------------------------------------------------------------------- kernels
// Rows of T x d elements, `units` units of a group (32 / VEC lanes with VEC
// elements each: 16 bytes where rows allow it, or an element a lane) taken in a
// grid-stride loop.  A thread's next unit is found from its
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

// Bound by HBM: 32768 x 2880 bf16 there and back 103 us, 5.6 TB/s (0.85 of the
// copy bandwidth).  With one load under way a thread instead of four: 145 us.
constexpr int ACT8_UNROLL = 4;  // vectors a thread loads before it works on them

template <typename TX, int VEC>
__global__ void __launch_bounds__(ACT8_THREADS)
act8_pack_kernel(const TX* __restrict__ x, int64_t T, int32_t d, int32_t groups,
                 int8_t* __restrict__ q, uint8_t* __restrict__ e) {
  constexpr int LANES = 32 / VEC;  // lanes of a unit
  using R = typename std::conditional<VEC == 1, float, Raw<TX>>::type;
  const int sub = threadIdx.x % LANES;
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * ACT8_THREADS + threadIdx.x;
  const int64_t nthr = static_cast<int64_t>(gridDim.x) * ACT8_THREADS;
  const int64_t units = T * groups, step = nthr / LANES;
  Act8Pos p(tid / LANES, step, groups);
  // whole warps take part in the group maxima: the loop runs while the
  // warp's first lane has a unit
  for (int64_t u = (tid & ~int64_t(31)) / LANES; u < units; u += ACT8_UNROLL * step) {
    R r[ACT8_UNROLL];
    int64_t at[ACT8_UNROLL], at_e[ACT8_UNROLL];  // first element (-1: none), exponent
#pragma unroll
    for (int k = 0; k < ACT8_UNROLL; ++k) {
      const int32_t c = p.g * 32 + sub * VEC;
      at[k] = p.row < T && c < d ? p.row * d + c : -1;
      at_e[k] = p.row * groups + p.g;
      if constexpr (VEC == 1) {
        r[k] = at[k] >= 0 ? to_f32(x[at[k]]) : 0.f;
      } else {
        r[k].clear();
        if (at[k] >= 0) r[k].load(x + at[k]);
      }
      p.next(groups);
    }
#pragma unroll
    for (int k = 0; k < ACT8_UNROLL; ++k) {
      if constexpr (VEC == 1) {
        const uint32_t b = act8_byte(__reduce_max_sync(0xffffffffu, act8_mag(r[k])));
        if (at[k] < 0) continue;
        q[at[k]] = static_cast<int8_t>(act8_q(r[k], act8_inv_scale(b)));
        if (sub == 0) e[at_e[k]] = static_cast<uint8_t>(b);
      } else {
        Lane<VEC> v;
        r[k].get(v);
        Bytes<VEC> bytes;
        const uint32_t b = act8_pack<VEC>(v, r[k].top(), bytes);
        if (at[k] < 0) continue;
        bytes.store(q + at[k]);
        if (sub == 0) e[at_e[k]] = static_cast<uint8_t>(b);
      }
    }
  }
}

template <typename TX, int VEC>
__global__ void __launch_bounds__(ACT8_THREADS)
act8_unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e, int64_t T,
                   int32_t d, int32_t groups, TX* __restrict__ x) {
  constexpr int LANES = 32 / VEC;
  using Q = typename std::conditional<VEC == 1, int8_t, Bytes<VEC == 1 ? 4 : VEC>>::type;
  const int sub = threadIdx.x % LANES;
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * ACT8_THREADS + threadIdx.x;
  const int64_t nthr = static_cast<int64_t>(gridDim.x) * ACT8_THREADS;
  const int64_t units = T * groups, step = nthr / LANES;
  Act8Pos p(tid / LANES, step, groups);
  for (int64_t u = tid / LANES; u < units; u += ACT8_UNROLL * step) {
    Q bytes[ACT8_UNROLL];
    uint32_t b[ACT8_UNROLL];
    int64_t at[ACT8_UNROLL];  // first element, -1: none
#pragma unroll
    for (int k = 0; k < ACT8_UNROLL; ++k) {
      const int32_t c = p.g * 32 + sub * VEC;
      at[k] = p.row < T && c < d ? p.row * d + c : -1;
      if (at[k] >= 0) {
        if constexpr (VEC == 1) bytes[k] = q[at[k]];
        else bytes[k].load(q + at[k]);
        b[k] = e[p.row * groups + p.g];
      }
      p.next(groups);
    }
#pragma unroll
    for (int k = 0; k < ACT8_UNROLL; ++k) {
      if (at[k] < 0) continue;
      if constexpr (VEC == 1) {
        x[at[k]] = from_f32<TX>(act8_value1(bytes[k], act8_scale(b[k])));
      } else {
        Lane<VEC> v;
        act8_unpack<VEC>(bytes[k], b[k], v);
        Raw<TX> r;
        r.set(v);
        r.store(x + at[k]);
      }
    }
  }
}

}  // namespace ckl
