// Layer norm and RMS norm of rows [T, d], forward and backward: what makes the
// loss's hidden states, and what takes their gradient back.
//
//   mu = mean(x) (0 without centring), r = (mean((x - mu)^2) + eps)^-1/2
//   xh = (x - mu) r,  y = xh gamma + beta
//   a = dy gamma,  dx = r (a - mean(a) [centred] - xh mean(a xh))
//   dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Bound by HBM: a row is read once into registers and every sum over it is
// taken there.  A row belongs to `tpr` threads (whole warps); a thread holds
// NV vectors of VEC elements, vector i at column (i tpr + t) VEC, so loads are
// coalesced and the columns of a thread are the same in every row.  VEC = 8
// (16-byte loads) needs d % 8 == 0 and 16-byte pointers; VEC = 1 takes the
// rest.  The variance is summed about the mean (a second sum over registers,
// not E[x^2] - mu^2, which cancels when the mean is large).
//
// The backward reads x, or the 8 bits the forward kept of it (ckl_act8.cuh).
// A thread adds its columns' dgamma and dbeta over the rows it sees in fp32
// registers; the row groups' sums go to the workspace and a second kernel adds
// them in a fixed order, so that results do not change from run to run.
#pragma once

#include "ckl_act8.cuh"

namespace ckl {

constexpr int NORM_MAX_D = 32768;
constexpr int NORM_MAX_PARTS = 592;  // row groups whose gradient sums the workspace holds

struct NormFwd {
  const void* x;
  const void* gamma;  // may be null: 1
  const void* beta;   // may be null: 0
  void* y;
  float* mean;  // null: not centred
  float* rstd;
  int8_t* q;  // null: no 8-bit copy of x
  uint8_t* e;
  int64_t T;
  int32_t d, groups, tpr, param_f32;
  float eps;
};

struct NormBwd {
  const void* dy;
  const void* x;     // null: q and e
  const int8_t* q;
  const uint8_t* e;
  const float* mean;  // null: not centred
  const float* rstd;
  const void* gamma;  // may be null: 1
  void* dx;
  float* parts;  // [parts, 2, d]: dgamma's and dbeta's sums (a null gradient's row is not written)
  int64_t T;
  int32_t d, groups, tpr, param_f32, want_gamma, want_beta;
};

// Sums over the threads of a row, the same in all of them: shuffles within a
// warp, then the warps' sums through shared memory in warp order.  Two buffers
// take turns, so that one barrier a sum is enough.
struct RowSum {
  float2 (*red)[32];
  int buf, warp0, warps, bar, tpr;
  __device__ __forceinline__ RowSum(float2 (*r)[32], int tpr_)
      : red(r), buf(0), warp0((threadIdx.x / tpr_) * (tpr_ / 32)), warps(tpr_ / 32),
        bar(1 + threadIdx.x / tpr_), tpr(tpr_) {}
  __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (warps == 1) return make_float2(a, b);
    if ((threadIdx.x & 31) == 0) red[buf][threadIdx.x >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
    a = b = 0.f;
    for (int w = 0; w < warps; ++w) {
      const float2 s = red[buf][warp0 + w];
      a += s.x;
      b += s.y;
    }
    buf ^= 1;
    return make_float2(a, b);
  }
};

template <int VEC>
__device__ __forceinline__ void norm_param(const void* p, int f32, int col, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    if (f32) {
      Raw8<float> r;
      r.load(static_cast<const float*>(p) + col);
      r.get(v);
    } else {
      Raw8<__nv_bfloat16> r;
      r.load(static_cast<const __nv_bfloat16*>(p) + col);
      r.get(v);
    }
  } else {
    v[0] = f32 ? static_cast<const float*>(p)[col]
               : to_f32(static_cast<const __nv_bfloat16*>(p)[col]);
  }
}

template <typename TX, int VEC>
__device__ __forceinline__ void norm_load(const TX* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    Raw8<TX> r;
    r.load(p);
    r.get(v);
  } else {
    v[0] = to_f32(*p);
  }
}

template <typename TX, int VEC>
__device__ __forceinline__ void norm_store(TX* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    Raw8<TX> r;
    r.set(v);
    r.store(p);
  } else {
    *p = from_f32<TX>(v[0]);
  }
}

template <typename TX, int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormFwd p) {
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, rpb = blockDim.x / p.tpr;
  RowSum sum(red, p.tpr);
  const float inv_d = 1.f / static_cast<float>(p.d);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rpb + group; row < p.T;
       row += static_cast<int64_t>(gridDim.x) * rpb) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    float v[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
      if (col < p.d) norm_load<TX, VEC>(x + col, v[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += v[i][j];
    }
    const float mu = p.mean ? sum(s, 0.f).x * inv_d : 0.f;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * p.tpr + t) * VEC < p.d)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s += (v[i][j] - mu) * (v[i][j] - mu);
    const float rstd = 1.f / sqrtf(sum(s, 0.f).x * inv_d + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
      if (p.q) {  // all lanes take part in the groups' maxima
        if constexpr (VEC == 8) {
          uint2 qq;
          const uint32_t b = act8_pack8(v[i], qq);
          if (col < p.d) {
            *reinterpret_cast<uint2*>(p.q + row * p.d + col) = qq;
            if ((t & 3) == 0) p.e[row * p.groups + col / 32] = static_cast<uint8_t>(b);
          }
        } else {
          const uint32_t b = act8_byte(__reduce_max_sync(0xffffffffu, act8_mag(v[i][0])));
          if (col < p.d) {
            p.q[row * p.d + col] = static_cast<int8_t>(act8_q(v[i][0], act8_inv_scale(b)));
            if ((t & 31) == 0) p.e[row * p.groups + col / 32] = static_cast<uint8_t>(b);
          }
        }
      }
      if (col < p.d) {
        float g[VEC], b[VEC], y[VEC];
        if (p.gamma) norm_param<VEC>(p.gamma, p.param_f32, col, g);
        if (p.beta) norm_param<VEC>(p.beta, p.param_f32, col, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          y[j] = (v[i][j] - mu) * rstd;
          if (p.gamma) y[j] *= g[j];
          if (p.beta) y[j] += b[j];
        }
        norm_store<TX, VEC>(static_cast<TX*>(p.y) + row * p.d + col, y);
      }
    }
  }
}

template <typename TX, int VEC, int NV, bool Q8>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const NormBwd p) {
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, rpb = blockDim.x / p.tpr;
  RowSum sum(red, p.tpr);
  const float inv_d = 1.f / static_cast<float>(p.d);
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;

  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rpb + group; row < p.T;
       row += static_cast<int64_t>(gridDim.x) * rpb) {
    const float mu = p.mean ? p.mean[row] : 0.f, rstd = p.rstd[row];
    float a[NV][VEC], xh[NV][VEC];
    float s1 = 0.f, s2 = 0.f;  // of a xh, of a
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[i][j] = xh[i][j] = 0.f;
      if (col >= p.d) continue;
      norm_load<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.d + col, a[i]);
      if constexpr (Q8) {
        const uint32_t b = p.e[row * p.groups + col / 32];
        if constexpr (VEC == 8)
          act8_unpack8(*reinterpret_cast<const uint2*>(p.q + row * p.d + col), b, xh[i]);
        else
          xh[i][0] = act8_value1(p.q[row * p.d + col], act8_scale(b));
      } else {
        norm_load<TX, VEC>(static_cast<const TX*>(p.x) + row * p.d + col, xh[i]);
      }
      float g[VEC];
      if (p.gamma) norm_param<VEC>(p.gamma, p.param_f32, col, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        xh[i][j] = (xh[i][j] - mu) * rstd;
        dg[i][j] += a[i][j] * xh[i][j];
        db[i][j] += a[i][j];
        if (p.gamma) a[i][j] *= g[j];
        s1 += a[i][j] * xh[i][j];
        s2 += a[i][j];
      }
    }
    const float2 c = sum(s1, s2);
    const float c1 = c.x * inv_d, c2 = p.mean ? c.y * inv_d : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
      if (col >= p.d) continue;
      float dx[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) dx[j] = rstd * (a[i][j] - c2 - xh[i][j] * c1);
      norm_store<TX, VEC>(static_cast<TX*>(p.dx) + row * p.d + col, dx);
    }
  }

  // part k is the row group's whose first row is k; one without rows has none
  const int64_t k = static_cast<int64_t>(blockIdx.x) * rpb + group;
  if (k >= p.T) return;
  float* part = p.parts + k * 2 * p.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * p.tpr + t) * VEC;
    if (col >= p.d) continue;
    if (p.want_gamma) norm_store<float, VEC>(part + col, dg[i]);
    if (p.want_beta) norm_store<float, VEC>(part + p.d + col, db[i]);
  }
}

constexpr int NORM_RED_COLS = 32, NORM_RED_ROWS = 16;

// dgamma (blockIdx.y = 0) and dbeta (1): the sum of the row groups' parts, 32
// columns a block, the parts shared by 16 threads a column.
__global__ void __launch_bounds__(NORM_RED_COLS* NORM_RED_ROWS)
norm_reduce_kernel(const float* __restrict__ parts, int n, int32_t d, float* __restrict__ dgamma,
                   float* __restrict__ dbeta, int accumulate) {
  __shared__ float s[NORM_RED_ROWS][NORM_RED_COLS + 1];
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  const int c = threadIdx.x % NORM_RED_COLS, r = threadIdx.x / NORM_RED_COLS;
  const int col = blockIdx.x * NORM_RED_COLS + c;
  if (out == nullptr) return;
  float v = 0.f;
  if (col < d)
    for (int k = r; k < n; k += NORM_RED_ROWS)
      v += parts[(static_cast<int64_t>(k) * 2 + blockIdx.y) * d + col];
  s[r][c] = v;
  __syncthreads();
  if (r == 0 && col < d) {
    v = 0.f;
    for (int k = 0; k < NORM_RED_ROWS; ++k) v += s[k][c];
    out[col] = accumulate ? out[col] + v : v;
  }
}

}  // namespace ckl
