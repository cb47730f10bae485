// Layer norm and RMS norm of rows [T, d], forward and backward: what makes the
// loss's hidden states, and what takes their gradient back.
//
//   mu = mean(x) (0 without centring), r = (mean((x - mu)^2) + eps)^-1/2
//   xh = (x - mu) r,  y = xh gamma + beta
//   a = dy gamma,  dx = r (a - mean(a) [centred] - xh mean(a xh))
//   dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Bound by HBM: a row is read once and every sum over it is taken in
// registers.  A row belongs to a group of `tpr` threads (whole warps); a
// thread holds NV vectors of VEC elements, vector i at column (i tpr + t) VEC,
// so loads are coalesced and a thread's columns are the same in every row.
// VEC = 8 (16-byte loads) needs d % 8 == 0 and 16-byte pointers; VEC = 1 takes
// the rest.  Groups take rows in a grid-stride loop.
//
// An SM needs about 35 KB of loads under way to keep HBM busy, and a row's
// sums are a dependent chain during which a thread would load nothing.  So
// with VEC = 8 a thread copies its own vectors of the next rows to shared
// memory (cp.async, NORM stages of them) and only ever reads what it copied
// itself: no barrier and no wait on another thread.
//
// The backward reads x, or the 8 bits the forward kept of it (ckl_act8.cuh).
// A thread adds its columns' dgamma and dbeta over its rows in fp32 registers;
// the block's groups are added in shared memory, and a second kernel adds the
// blocks' sums ("parts", in the workspace) in a fixed order, so that results
// do not change from run to run.
//
// Rows too long for registers (d > 16384, or 8192 element-wise) are read again
// from L1 / L2 for each of their sums, and their gradients' sums over T get a
// kernel of their own.
#pragma once

#include "ckl_act8.cuh"
#include "ckl_ptx.cuh"

namespace ckl {

constexpr int NORM_THREADS = 512;
constexpr int NORM_MAX_PARTS = 592;  // blocks whose gradient sums the workspace holds

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
  float* parts;  // [parts, 2, d]: sums of dgamma and dbeta
  int64_t T;
  int32_t d, groups, tpr, param_f32, want_gamma, want_beta;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Stages of a ring whose stage takes `bytes` a thread: four where 512 threads'
// fit in 200 KB, otherwise as many as do.
__host__ __device__ constexpr int norm_stages(int bytes) {
  return 200 * 1024 / (NORM_THREADS * bytes) >= 4 ? 4 : 200 * 1024 / (NORM_THREADS * bytes);
}
template <typename TX, int NV>
constexpr int NORM_FWD_BYTES = NV * 8 * static_cast<int>(sizeof(TX));
template <typename TX, int NV, bool Q8>
constexpr int NORM_BWD_BYTES = NV * 8 * (static_cast<int>(sizeof(TX)) * (Q8 ? 1 : 2) + (Q8 ? 1 : 0));

__device__ __forceinline__ float2 warp_sum2(float a, float b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_float2(a, b);
}

// What the warps of a row's group tell each other through shared memory.  Two
// buffers take turns, so that one barrier an exchange is enough.
struct RowGroup {
  float2 (*red)[32];
  int buf, warp0, warps, bar, tpr;
  __device__ __forceinline__ RowGroup(float2 (*r)[32], int tpr_)
      : red(r), buf(0), warp0((threadIdx.x / tpr_) * (tpr_ / 32)), warps(tpr_ / 32),
        bar(1 + threadIdx.x / tpr_), tpr(tpr_) {}
  __device__ __forceinline__ const float2* exchange(float2 mine) {
    if ((threadIdx.x & 31) == 0) red[buf][threadIdx.x >> 5] = mine;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
    const float2* all = &red[buf][warp0];
    buf ^= 1;
    return all;
  }
  // sums over the row, the same in all of its threads (warp order)
  __device__ __forceinline__ float2 sum(float a, float b) {
    float2 s = warp_sum2(a, b);
    if (warps == 1) return s;
    const float2* all = exchange(s);
    s = make_float2(0.f, 0.f);
    for (int w = 0; w < warps; ++w) {
      s.x += all[w].x;
      s.y += all[w].y;
    }
    return s;
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

// x's elements at `col` of a row, from x or from its 8 bits.
template <typename TX, int VEC, bool Q8>
__device__ __forceinline__ void norm_load_x(const NormBwd& p, int64_t row, int col,
                                            float (&v)[VEC]) {
  if constexpr (!Q8) {
    norm_load<TX, VEC>(static_cast<const TX*>(p.x) + row * p.d + col, v);
  } else {
    const uint32_t b = p.e[row * p.groups + col / 32];
    if constexpr (VEC == 8)
      act8_unpack8(*reinterpret_cast<const uint2*>(p.q + row * p.d + col), b, v);
    else
      v[0] = act8_value1(p.q[row * p.d + col], act8_scale(b));
  }
}

// The 8-bit copy of one vector (VEC = 8) or element: all lanes of the warp take
// part in the groups' maxima, `on` says whether the columns exist.
template <int VEC>
__device__ __forceinline__ void norm_keep8(const NormFwd& p, int64_t row, int col, bool on,
                                           const float (&v)[VEC], uint32_t top) {
  if constexpr (VEC == 8) {
    uint2 qq;
    const uint32_t b = act8_pack8(v, top, qq);
    if (on) {
      *reinterpret_cast<uint2*>(p.q + row * p.d + col) = qq;
      if ((threadIdx.x & 3) == 0) p.e[row * p.groups + col / 32] = static_cast<uint8_t>(b);
    }
  } else {
    const uint32_t b = act8_byte(__reduce_max_sync(0xffffffffu, act8_mag(v[0])));
    if (on) {
      p.q[row * p.d + col] = static_cast<int8_t>(act8_q(v[0], act8_inv_scale(b)));
      if ((threadIdx.x & 31) == 0) p.e[row * p.groups + col / 32] = static_cast<uint8_t>(b);
    }
  }
}

// ------------------------------------------------------------------- forward
// The mean and the sum of squares about it come from one exchange: a warp
// takes both of its own columns (the squares about the warp's mean, so that a
// large mean cancels nothing), and the warps' are joined by
//   mu = sum n_w mu_w / d,  M = sum M_w + n_w (mu_w - mu)^2.
template <typename TX, int VEC, int NV>
__global__ void __launch_bounds__(NORM_THREADS, NV <= 2 ? 2 : 1)
norm_fwd_kernel(const NormFwd p) {
  constexpr int BYTES = NORM_FWD_BYTES<TX, NV>;
  constexpr int S = norm_stages(BYTES);
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float2 red[2][32];
  __shared__ float cols[32];  // columns of each warp
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, G = blockDim.x / p.tpr;
  RowGroup rg(red, p.tpr);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const bool center = p.mean != nullptr;
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * p.tpr + t) * VEC < p.d) n += VEC;
  const float nw = static_cast<float>(__reduce_add_sync(0xffffffffu, n));
  const float inv_nw = nw > 0.f ? 1.f / nw : 0.f;
  if ((threadIdx.x & 31) == 0) cols[threadIdx.x >> 5] = nw;
  __syncthreads();

  // vectors of a row in shared memory: 16-byte pieces, a thread's own
  const uint32_t ring = smem_u32(norm_smem) + threadIdx.x * 16;
  const uint32_t piece = blockDim.x * 16;
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (VEC == 8) {
      if (row < p.T) {
        const TX* x = static_cast<const TX*>(p.x) + row * p.d;
        const uint32_t at = ring + stage * (BYTES / 16) * piece;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int col = (i * p.tpr + t) * VEC;
          if (col < p.d)
#pragma unroll
            for (int h = 0; h < static_cast<int>(sizeof(TX)) / 2; ++h)
              cp_async16(at + (i * (sizeof(TX) / 2) + h) * piece,
                         reinterpret_cast<const uint8_t*>(x + col) + 16 * h);
        }
      }
      cp_async_commit();
    }
  };

  const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(gridDim.x) * group + blockIdx.x;
  for (int s = 0; s < S - 1; ++s) fetch(row + s * stride, s);
  int stage = 0;
  for (; row < p.T; row += stride) {
    Raw8<TX> raw[NV];
    float v1[NV];
    if constexpr (VEC == 8) {
      fetch(row + (S - 1) * stride, (stage + S - 1) % S);
      cp_async_wait<S - 1>();
      const uint8_t* at = norm_smem + threadIdx.x * 16 + stage * (BYTES / 16) * piece;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        raw[i].clear();
        if ((i * p.tpr + t) * VEC < p.d) raw[i].load_pieces(at + i * (sizeof(TX) / 2) * piece, piece);
      }
      stage = (stage + 1) % S;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = i * p.tpr + t;
        v1[i] = col < p.d ? to_f32(static_cast<const TX*>(p.x)[row * p.d + col]) : 0.f;
      }
    }
    auto get = [&](int i, float (&v)[VEC]) {
      if constexpr (VEC == 8) raw[i].get(v);
      else v[0] = v1[i];
    };

    float mu = 0.f, m2 = 0.f;
    if (center) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[VEC];
        get(i, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s += v[j];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      mu = s * inv_nw;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * p.tpr + t) * VEC >= p.d) continue;
      float v[VEC];
      get(i, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) m2 = fmaf(v[j] - mu, v[j] - mu, m2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
    if (rg.warps > 1) {
      const float2* all = rg.exchange(make_float2(mu, m2));
      const float* nws = cols + rg.warp0;
      m2 = 0.f;
      if (center) {
        mu = 0.f;
        for (int w = 0; w < rg.warps; ++w) mu = fmaf(all[w].x, nws[w], mu);
        mu *= inv_d;
        for (int w = 0; w < rg.warps; ++w) {
          const float c = all[w].x - mu;
          m2 += fmaf(c * c, nws[w], all[w].y);
        }
      } else {
        for (int w = 0; w < rg.warps; ++w) m2 += all[w].y;
      }
    }
    const float rstd = 1.f / sqrtf(fmaf(m2, inv_d, p.eps));
    if (t == 0) {
      if (center) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }

#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
      float v[VEC];
      get(i, v);
      if (p.q) {
        uint32_t top = 0;
        if constexpr (VEC == 8) top = raw[i].top();
        norm_keep8<VEC>(p, row, col, col < p.d, v, top);
      }
      if (col >= p.d) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = (v[j] - mu) * rstd;
      if (p.gamma) {
        float g[VEC];
        norm_param<VEC>(p.gamma, p.param_f32, col, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] *= g[j];
      }
      if (p.beta) {
        float b[VEC];
        norm_param<VEC>(p.beta, p.param_f32, col, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += b[j];
      }
      norm_store<TX, VEC>(static_cast<TX*>(p.y) + row * p.d + col, v);
    }
  }
}

// Rows of any length: a block a row, read three times.
template <typename TX, int VEC>
__global__ void __launch_bounds__(NORM_THREADS) norm_fwd_long_kernel(const NormFwd p) {
  __shared__ float2 red[2][32];
  RowGroup rg(red, NORM_THREADS);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int64_t span = static_cast<int64_t>(NORM_THREADS) * VEC;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    float mu = 0.f, s = 0.f;
    if (p.mean) {
      for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
        float v[VEC];
        norm_load<TX, VEC>(x + c, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s += v[j];
      }
      mu = rg.sum(s, 0.f).x * inv_d;
      s = 0.f;
    }
    for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
      float v[VEC];
      norm_load<TX, VEC>(x + c, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s = fmaf(v[j] - mu, v[j] - mu, s);
    }
    const float rstd = 1.f / sqrtf(fmaf(rg.sum(s, 0.f).x, inv_d, p.eps));
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
    for (int64_t c0 = 0; c0 < p.d; c0 += span) {
      const int64_t c = c0 + threadIdx.x * VEC;
      const bool on = c < p.d;
      float v[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = 0.f;
      if (on) norm_load<TX, VEC>(x + c, v);
      if (p.q) {
        uint32_t top = 0;
        if constexpr (VEC == 8) top = act8_top8(v);
        norm_keep8<VEC>(p, row, static_cast<int>(c), on, v, top);
      }
      if (!on) continue;
      float g[VEC], b[VEC];
      if (p.gamma) norm_param<VEC>(p.gamma, p.param_f32, static_cast<int>(c), g);
      if (p.beta) norm_param<VEC>(p.beta, p.param_f32, static_cast<int>(c), b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[j] = (v[j] - mu) * rstd;
        if (p.gamma) v[j] *= g[j];
        if (p.beta) v[j] += b[j];
      }
      norm_store<TX, VEC>(static_cast<TX*>(p.y) + row * p.d + c, v);
    }
  }
}

// ------------------------------------------------------------------ backward
template <typename TX, int VEC, int NV, bool Q8>
__global__ void __launch_bounds__(NORM_THREADS) norm_bwd_kernel(const NormBwd p) {
  constexpr int BYTES = NORM_BWD_BYTES<TX, NV, Q8>;
  constexpr int S = norm_stages(BYTES);
  constexpr int H = sizeof(TX) / 2;  // 16-byte pieces of a vector
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, G = blockDim.x / p.tpr;
  RowGroup rg(red, p.tpr);
  const float inv_d = 1.f / static_cast<float>(p.d);
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;

  // a stage: dy's pieces, then x's, or the 8-byte pieces of q
  const uint32_t piece = blockDim.x * 16;
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (VEC == 8) {
      if (row < p.T) {
        const uint32_t base = smem_u32(norm_smem) + stage * BYTES * blockDim.x;
        const uint32_t at = base + threadIdx.x * 16;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int col = (i * p.tpr + t) * VEC;
          if (col >= p.d) continue;
          const int64_t o = row * p.d + col;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            cp_async16(at + (i * H + h) * piece,
                       reinterpret_cast<const uint8_t*>(static_cast<const TX*>(p.dy) + o) + 16 * h);
            if constexpr (!Q8)
              cp_async16(at + (NV * H + i * H + h) * piece,
                         reinterpret_cast<const uint8_t*>(static_cast<const TX*>(p.x) + o) + 16 * h);
          }
          if constexpr (Q8)
            cp_async8(base + NV * H * piece + (i * blockDim.x + threadIdx.x) * 8, p.q + o);
        }
      }
      cp_async_commit();
    }
  };
  // what a row has besides: loaded a row ahead
  float mu_next = 0.f, rstd_next = 0.f;
  uint32_t e_next[NV];
  auto ahead = [&](int64_t row) {
    if (row >= p.T) return;
    if (p.mean) mu_next = p.mean[row];
    rstd_next = p.rstd[row];
    if constexpr (Q8 && VEC == 8) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * p.tpr + t) * VEC;
        if (col < p.d) e_next[i] = p.e[row * p.groups + col / 32];
      }
    }
  };

  const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(gridDim.x) * group + blockIdx.x;
  for (int s = 0; s < S - 1; ++s) fetch(row + s * stride, s);
  ahead(row);
  int stage = 0;
  for (; row < p.T; row += stride) {
    const float mu = mu_next, rstd = rstd_next;
    uint32_t e_row[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) e_row[i] = e_next[i];
    ahead(row + stride);
    const uint8_t* base = norm_smem + stage * BYTES * blockDim.x;
    if constexpr (VEC == 8) {
      fetch(row + (S - 1) * stride, (stage + S - 1) % S);
      cp_async_wait<S - 1>();
      stage = (stage + 1) % S;
    }
    float a[NV][VEC], xh[NV][VEC];
    float s1 = 0.f, s2 = 0.f;  // of a xh, of a
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[i][j] = xh[i][j] = 0.f;
      if (col >= p.d) continue;
      if constexpr (VEC == 8) {
        Raw8<TX> r;
        r.load_pieces(base + i * H * piece + threadIdx.x * 16, piece);
        r.get(a[i]);
        if constexpr (Q8) {
          act8_unpack8(*reinterpret_cast<const uint2*>(base + NV * H * piece +
                                                       (i * blockDim.x + threadIdx.x) * 8),
                       e_row[i], xh[i]);
        } else {
          r.load_pieces(base + (NV + i) * H * piece + threadIdx.x * 16, piece);
          r.get(xh[i]);
        }
      } else {
        norm_load<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.d + col, a[i]);
        norm_load_x<TX, VEC, Q8>(p, row, col, xh[i]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        xh[i][j] = (xh[i][j] - mu) * rstd;
        dg[i][j] = fmaf(a[i][j], xh[i][j], dg[i][j]);
        db[i][j] += a[i][j];
      }
      if (p.gamma) {
        float g[VEC];
        norm_param<VEC>(p.gamma, p.param_f32, col, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s1 = fmaf(a[i][j], xh[i][j], s1);
        s2 += a[i][j];
      }
    }
    const float2 c = rg.sum(s1, s2);
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
  if (!p.want_gamma && !p.want_beta) return;
  griddep_launch();  // norm_reduce_kernel may start; it waits for this kernel's end

  // the block's groups, one after another, into the first
  float* sums = reinterpret_cast<float*>(norm_smem);
  __syncthreads();  // the ring is read
  for (int k = 1; k < G; ++k) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
      if (group != k || col >= p.d) continue;
      norm_store<float, VEC>(sums + col, dg[i]);
      norm_store<float, VEC>(sums + p.d + col, db[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
      if (group != 0 || col >= p.d) continue;
      float v[VEC];
      norm_load<float, VEC>(sums + col, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) dg[i][j] += v[j];
      norm_load<float, VEC>(sums + p.d + col, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) db[i][j] += v[j];
    }
    __syncthreads();
  }
  if (group != 0) return;
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * p.tpr + t) * VEC;
    if (col >= p.d) continue;
    if (p.want_gamma) norm_store<float, VEC>(part + col, dg[i]);
    if (p.want_beta) norm_store<float, VEC>(part + p.d + col, db[i]);
  }
}

// Rows of any length: dx, a block a row, read twice.
template <typename TX, int VEC, bool Q8>
__global__ void __launch_bounds__(NORM_THREADS) norm_bwd_long_kernel(const NormBwd p) {
  __shared__ float2 red[2][32];
  RowGroup rg(red, NORM_THREADS);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int64_t span = static_cast<int64_t>(NORM_THREADS) * VEC;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const float mu = p.mean ? p.mean[row] : 0.f, rstd = p.rstd[row];
    auto load = [&](int64_t c, float (&a)[VEC], float (&xh)[VEC]) {
      norm_load<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.d + c, a);
      norm_load_x<TX, VEC, Q8>(p, row, static_cast<int>(c), xh);
      if (p.gamma) {
        float g[VEC];
        norm_param<VEC>(p.gamma, p.param_f32, static_cast<int>(c), g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) xh[j] = (xh[j] - mu) * rstd;
    };
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
      float a[VEC], xh[VEC];
      load(c, a, xh);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s1 = fmaf(a[j], xh[j], s1);
        s2 += a[j];
      }
    }
    const float2 s = rg.sum(s1, s2);
    const float c1 = s.x * inv_d, c2 = p.mean ? s.y * inv_d : 0.f;
    for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
      float a[VEC], xh[VEC];
      load(c, a, xh);
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[j] = rstd * (a[j] - c2 - xh[j] * c1);
      norm_store<TX, VEC>(static_cast<TX*>(p.dx) + row * p.d + c, a);
    }
  }
}

constexpr int NORM_COL_WARPS = 8;

// Rows of any length: the sums over T, a block 32 VEC columns of the rows
// blockIdx.y, blockIdx.y + gridDim.y, ... of eight.
template <typename TX, int VEC, bool Q8>
__global__ void __launch_bounds__(32 * NORM_COL_WARPS) norm_cols_kernel(const NormBwd p) {
  __shared__ float s[NORM_COL_WARPS][2 * VEC][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * VEC;
  float dg[VEC], db[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) dg[j] = db[j] = 0.f;
  if (col < p.d) {
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * NORM_COL_WARPS + warp; row < p.T;
         row += static_cast<int64_t>(gridDim.y) * NORM_COL_WARPS) {
      const float mu = p.mean ? p.mean[row] : 0.f, rstd = p.rstd[row];
      float a[VEC], x[VEC];
      norm_load<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.d + col, a);
      norm_load_x<TX, VEC, Q8>(p, row, static_cast<int>(col), x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dg[j] = fmaf(a[j], (x[j] - mu) * rstd, dg[j]);
        db[j] += a[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    s[warp][j][lane] = dg[j];
    s[warp][VEC + j][lane] = db[j];
  }
  __syncthreads();
  // thread -> (sum, column of the block)
  for (int k = threadIdx.x; k < 2 * 32 * VEC; k += 32 * NORM_COL_WARPS) {
    const int which = k / (32 * VEC), c = k % (32 * VEC);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 32 * VEC + c;
    if (at >= p.d || !(which ? p.want_beta : p.want_gamma)) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NORM_COL_WARPS; ++w) v += s[w][which * VEC + c % VEC][c / VEC];
    p.parts[(static_cast<int64_t>(blockIdx.y) * 2 + which) * p.d + at] = v;
  }
}

constexpr int NORM_RED_COLS = 32, NORM_RED_ROWS = 16;

// dgamma (blockIdx.y = 0) and dbeta (1): the sum of the blocks' parts, 32
// columns a block, the parts shared by 16 threads a column.  Launched so that
// it may start before the kernel that writes the parts has ended.
__global__ void __launch_bounds__(NORM_RED_COLS* NORM_RED_ROWS)
norm_reduce_kernel(const float* parts, int n, int32_t d, float* __restrict__ dgamma,
                   float* __restrict__ dbeta, int accumulate) {
  __shared__ float s[NORM_RED_ROWS][NORM_RED_COLS + 1];
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  const int c = threadIdx.x % NORM_RED_COLS, r = threadIdx.x / NORM_RED_COLS;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * NORM_RED_COLS + c;
  griddep_wait();
  if (out == nullptr) return;
  float v = 0.f;
  if (col < d) {
#pragma unroll 4
    for (int k = r; k < n; k += NORM_RED_ROWS)
      v += parts[(static_cast<int64_t>(k) * 2 + blockIdx.y) * d + col];
  }
  s[r][c] = v;
  __syncthreads();
  if (r == 0 && col < d) {
    v = 0.f;
    for (int k = 0; k < NORM_RED_ROWS; ++k) v += s[k][c];
    out[col] = accumulate ? out[col] + v : v;
  }
}

}  // namespace ckl
