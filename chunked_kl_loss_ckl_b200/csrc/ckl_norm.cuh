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
  int32_t d, groups, tpr, param_f32, staged;  // staged: the parameters go to shared memory
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
  int32_t d, groups, tpr, param_f32, staged, want_gamma, want_beta;
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

// What the warps of a row's group tell each other through shared memory.  Two
// buffers take turns, so that one barrier an exchange is enough.  Warp w's two
// numbers are at [0][w] and [1][w]; lanes 0-15 and 16-31 read one of the two
// each and add them up in a butterfly, so that the sums cost the same few
// instructions however many warps a row has.
struct RowGroup {
  float (*red)[2][16];
  int buf, warp0, warps, half, bar, tpr;
  __device__ __forceinline__ RowGroup(float (*r)[2][16], int tpr_)
      : red(r), buf(0), warp0((threadIdx.x / tpr_) * (tpr_ / 32)), warps(tpr_ / 32), half(1),
        bar(1 + threadIdx.x / tpr_), tpr(tpr_) {
    while (half < warps) half <<= 1;
    half >>= 1;
  }
  // the two sums over the warp, a in lanes 0-15 and b in lanes 16-31: the
  // first step swaps halves, so that five shuffles do
  static __device__ __forceinline__ float warp_halves(float a, float b) {
    const bool hi = threadIdx.x & 16;
    float v = hi ? b : a;
    v += __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ void put(float v) {  // of lanes 0 and 16
    if ((threadIdx.x & 15) == 0) red[buf][(threadIdx.x >> 4) & 1][threadIdx.x >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
  }
  __device__ __forceinline__ float get(int which) const {  // 0 past the row's warps
    const int w = threadIdx.x & 15;
    return w < warps ? red[buf][which][warp0 + w] : 0.f;
  }
  // sum over the row's warps of what the 16 lanes of a half hold
  __device__ __forceinline__ float over_warps(float v) const {
    for (int o = half; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  // sums over the row, the same in all of its threads
  __device__ __forceinline__ float2 sum(float a, float b) {
    float v = warp_halves(a, b);
    if (warps > 1) {
      put(v);
      v = over_warps(get((threadIdx.x >> 4) & 1));
      buf ^= 1;
    }
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  }
};

template <typename TX, int VEC>
__device__ __forceinline__ void norm_load(const TX* p, Lane<VEC>& v) {
  if constexpr (VEC == 8) {
    Raw8<TX> r;
    r.load(p);
    r.get(v);
  } else {
    v.e[0] = to_f32(*p);
  }
}

template <int VEC>
__device__ __forceinline__ void norm_param(const void* p, int f32, int64_t col, Lane<VEC>& v) {
  if (f32) norm_load<float, VEC>(static_cast<const float*>(p) + col, v);
  else norm_load<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(p) + col, v);
}

template <typename TX, int VEC>
__device__ __forceinline__ void norm_store(TX* p, const Lane<VEC>& v) {
  if constexpr (VEC == 8) {
    Raw8<TX> r;
    r.set(v);
    r.store(p);
  } else {
    *p = from_f32<TX>(v.e[0]);
  }
}

// gamma or beta in fp32 in shared memory, for kernels that pass over many rows
// (VEC = 8): two planes of four floats a vector, so that reads do not conflict.
__device__ __forceinline__ void norm_stage_param(const void* p, int f32, int32_t d, uint8_t* to) {
  for (int c = threadIdx.x; c < d / 8; c += blockDim.x) {
    Lane<8> v;
    norm_param<8>(p, f32, 8 * c, v);
    reinterpret_cast<ulonglong2*>(to)[c] = make_ulonglong2(v.e[0], v.e[1]);
    reinterpret_cast<ulonglong2*>(to)[d / 8 + c] = make_ulonglong2(v.e[2], v.e[3]);
  }
}
__device__ __forceinline__ void norm_staged(const uint8_t* from, int32_t d, int col, Lane<8>& v) {
  Raw8<float> r;
  r.load_pieces(from + 2 * col, 2 * d);
  r.get(v);
}

// x's elements at `col` of a row, from x or from its 8 bits.
template <typename TX, int VEC, bool Q8>
__device__ __forceinline__ void norm_load_x(const NormBwd& p, int64_t row, int64_t col,
                                            Lane<VEC>& v) {
  if constexpr (!Q8) {
    norm_load<TX, VEC>(static_cast<const TX*>(p.x) + row * p.d + col, v);
  } else {
    const uint32_t b = p.e[row * p.groups + col / 32];
    if constexpr (VEC == 8)
      act8_unpack8(*reinterpret_cast<const uint2*>(p.q + row * p.d + col), b, v);
    else
      v.e[0] = act8_value1(p.q[row * p.d + col], act8_scale(b));
  }
}

// The 8-bit copy of one vector (VEC = 8) or element: all lanes of the warp take
// part in the groups' maxima, `on` says whether the columns exist.
template <int VEC>
__device__ __forceinline__ void norm_keep8(const NormFwd& p, int64_t row, int64_t col, bool on,
                                           const Lane<VEC>& v, uint32_t top) {
  if constexpr (VEC == 8) {
    uint2 qq;
    const uint32_t b = act8_pack8(v, top, qq);
    if (on) {
      *reinterpret_cast<uint2*>(p.q + row * p.d + col) = qq;
      if ((threadIdx.x & 3) == 0) p.e[row * p.groups + col / 32] = static_cast<uint8_t>(b);
    }
  } else {
    const uint32_t b = act8_byte(__reduce_max_sync(0xffffffffu, act8_mag(v.e[0])));
    if (on) {
      p.q[row * p.d + col] = static_cast<int8_t>(act8_q(v.e[0], act8_inv_scale(b)));
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
__global__ void __launch_bounds__(NORM_THREADS) norm_fwd_kernel(const NormFwd p) {
  constexpr int BYTES = NORM_FWD_BYTES<TX, NV>;
  constexpr int S = norm_stages(BYTES);
  constexpr int H = sizeof(TX) / 2;  // 16-byte pieces of a vector
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float red[2][2][16];
  __shared__ float cols[16];  // columns of each warp
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
  // vectors of a row in shared memory: 16-byte pieces, a thread's own
  const uint32_t piece = blockDim.x * 16;
  const uint32_t ring = smem_u32(norm_smem) + threadIdx.x * 16;
  uint8_t* const gs = norm_smem + (VEC == 8 ? BYTES * S * blockDim.x : 0);
  uint8_t* const bs = gs + (p.gamma ? 4 * p.d : 0);
  if (VEC == 8 && p.staged) {
    if (p.gamma) norm_stage_param(p.gamma, p.param_f32, p.d, gs);
    if (p.beta) norm_stage_param(p.beta, p.param_f32, p.d, bs);
  }
  __syncthreads();
  const float n_lane = (threadIdx.x & 15) < rg.warps ? cols[rg.warp0 + (threadIdx.x & 15)] : 0.f;

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
            for (int h = 0; h < H; ++h)
              cp_async16(at + (i * H + h) * piece,
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
    Lane<VEC> v[NV];
    if constexpr (VEC == 8) {
      fetch(row + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
      cp_async_wait<S - 1>();
      const uint8_t* at = norm_smem + threadIdx.x * 16 + stage * (BYTES / 16) * piece;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        raw[i].clear();
        if ((i * p.tpr + t) * VEC < p.d) raw[i].load_pieces(at + i * H * piece, piece);
        raw[i].get(v[i]);
      }
      stage = stage + 1 == S ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = i * p.tpr + t;
        v[i].e[0] = col < p.d ? to_f32(static_cast<const TX*>(p.x)[row * p.d + col]) : 0.f;
      }
    }

    float mu = 0.f;
    if (center) {
      E s = both<E>(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) s = vadd(s, v[i].e[j]);
      mu = vsum(s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mu += __shfl_xor_sync(0xffffffffu, mu, o);
      mu *= inv_nw;
    }
    E ss = both<E>(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * p.tpr + t) * VEC >= p.d) continue;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const E c = vsub(v[i].e[j], both<E>(mu));
        ss = vfma(c, c, ss);
      }
    }
    float m2 = vsum(ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
    if (rg.warps > 1) {
      rg.put((threadIdx.x & 16) ? m2 : mu);
      m2 = rg.get(1);
      if (center) {
        const float muw = rg.get(0);
        mu = rg.over_warps(muw * n_lane) * inv_d;
        m2 = fmaf((muw - mu) * (muw - mu), n_lane, m2);
        mu = __shfl_sync(0xffffffffu, mu, 0);
      }
      m2 = __shfl_sync(0xffffffffu, rg.over_warps(m2), 0);
      rg.buf ^= 1;
    }
    const float rstd = rsqrtf(fmaf(m2, inv_d, p.eps));
    if (t == 0) {
      if (center) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }

#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
      if (p.q) {
        uint32_t top = 0;
        if constexpr (VEC == 8) top = raw[i].top();
        norm_keep8<VEC>(p, row, col, col < p.d, v[i], top);
      }
      if (col >= p.d) continue;
      Lane<VEC> g, b;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        g.e[j] = both<E>(1.f);
        b.e[j] = both<E>(0.f);
      }
      if (VEC == 8 && p.staged) {
        if constexpr (VEC == 8) {
          if (p.gamma) norm_staged(gs, p.d, col, g);
          if (p.beta) norm_staged(bs, p.d, col, b);
        }
      } else {
        if (p.gamma) norm_param<VEC>(p.gamma, p.param_f32, col, g);
        if (p.beta) norm_param<VEC>(p.beta, p.param_f32, col, b);
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        b.e[j] = vfma(vmul(vsub(v[i].e[j], both<E>(mu)), both<E>(rstd)), g.e[j], b.e[j]);
      norm_store<TX, VEC>(static_cast<TX*>(p.y) + row * p.d + col, b);
    }
  }
}

// Rows of any length: a block a row, read three times.
template <typename TX, int VEC>
__global__ void __launch_bounds__(NORM_THREADS) norm_fwd_long_kernel(const NormFwd p) {
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  __shared__ float red[2][2][16];
  RowGroup rg(red, NORM_THREADS);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int64_t span = static_cast<int64_t>(NORM_THREADS) * VEC;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    float mu = 0.f;
    E s = both<E>(0.f);
    if (p.mean) {
      for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
        Lane<VEC> v;
        norm_load<TX, VEC>(x + c, v);
#pragma unroll
        for (int j = 0; j < N; ++j) s = vadd(s, v.e[j]);
      }
      mu = rg.sum(vsum(s), 0.f).x * inv_d;
      s = both<E>(0.f);
    }
    for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
      Lane<VEC> v;
      norm_load<TX, VEC>(x + c, v);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const E e = vsub(v.e[j], both<E>(mu));
        s = vfma(e, e, s);
      }
    }
    const float rstd = rsqrtf(fmaf(rg.sum(vsum(s), 0.f).x, inv_d, p.eps));
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
    for (int64_t c0 = 0; c0 < p.d; c0 += span) {
      const int64_t c = c0 + threadIdx.x * VEC;
      const bool on = c < p.d;
      Lane<VEC> v;
#pragma unroll
      for (int j = 0; j < N; ++j) v.e[j] = both<E>(0.f);
      uint32_t top = 0;
      if constexpr (VEC == 8) {
        Raw8<TX> r;
        r.clear();
        if (on) r.load(x + c);
        r.get(v);
        top = r.top();
      } else if (on) {
        norm_load<TX, VEC>(x + c, v);
      }
      if (p.q) norm_keep8<VEC>(p, row, c, on, v, top);
      if (!on) continue;
      Lane<VEC> g, b;
      if (p.gamma) norm_param<VEC>(p.gamma, p.param_f32, c, g);
      if (p.beta) norm_param<VEC>(p.beta, p.param_f32, c, b);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v.e[j] = vmul(vsub(v.e[j], both<E>(mu)), both<E>(rstd));
        if (p.gamma) v.e[j] = vmul(v.e[j], g.e[j]);
        if (p.beta) v.e[j] = vadd(v.e[j], b.e[j]);
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
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float red[2][2][16];
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, G = blockDim.x / p.tpr;
  RowGroup rg(red, p.tpr);
  const float inv_d = 1.f / static_cast<float>(p.d);
  Lane<VEC> dg[NV], db[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) dg[i].e[j] = db[i].e[j] = both<E>(0.f);
  uint8_t* const gs = norm_smem + (VEC == 8 ? BYTES * S * blockDim.x : 0);
  if (VEC == 8 && p.staged && p.gamma) norm_stage_param(p.gamma, p.param_f32, p.d, gs);
  __syncthreads();

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
      fetch(row + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
      cp_async_wait<S - 1>();
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    Lane<VEC> a[NV], xh[NV];
    E s1 = both<E>(0.f), s2 = both<E>(0.f);  // of a xh, of a
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < N; ++j) a[i].e[j] = xh[i].e[j] = both<E>(0.f);
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
      Lane<VEC> g;
#pragma unroll
      for (int j = 0; j < N; ++j) g.e[j] = both<E>(1.f);
      if (p.gamma) {
        if (VEC == 8 && p.staged) {
          if constexpr (VEC == 8) norm_staged(gs, p.d, col, g);
        } else {
          norm_param<VEC>(p.gamma, p.param_f32, col, g);
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const E x = vmul(vsub(xh[i].e[j], both<E>(mu)), both<E>(rstd));
        dg[i].e[j] = vfma(a[i].e[j], x, dg[i].e[j]);
        db[i].e[j] = vadd(db[i].e[j], a[i].e[j]);
        a[i].e[j] = vmul(a[i].e[j], g.e[j]);
        s1 = vfma(a[i].e[j], x, s1);
        s2 = vadd(s2, a[i].e[j]);
        xh[i].e[j] = x;
      }
    }
    const float2 c = rg.sum(vsum(s1), vsum(s2));
    const E c1 = both<E>(-c.x * inv_d), c2 = both<E>(p.mean ? c.y * inv_d : 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * p.tpr + t) * VEC;
      if (col >= p.d) continue;
#pragma unroll
      for (int j = 0; j < N; ++j)
        a[i].e[j] = vmul(vfma(xh[i].e[j], c1, vsub(a[i].e[j], c2)), both<E>(rstd));
      norm_store<TX, VEC>(static_cast<TX*>(p.dx) + row * p.d + col, a[i]);
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
      Lane<VEC> v;
      norm_load<float, VEC>(sums + col, v);
#pragma unroll
      for (int j = 0; j < N; ++j) dg[i].e[j] = vadd(dg[i].e[j], v.e[j]);
      norm_load<float, VEC>(sums + p.d + col, v);
#pragma unroll
      for (int j = 0; j < N; ++j) db[i].e[j] = vadd(db[i].e[j], v.e[j]);
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
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  __shared__ float red[2][2][16];
  RowGroup rg(red, NORM_THREADS);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int64_t span = static_cast<int64_t>(NORM_THREADS) * VEC;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const E mu = both<E>(p.mean ? p.mean[row] : 0.f), rstd = both<E>(p.rstd[row]);
    auto load = [&](int64_t c, Lane<VEC>& a, Lane<VEC>& xh) {
      norm_load<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.d + c, a);
      norm_load_x<TX, VEC, Q8>(p, row, c, xh);
      if (p.gamma) {
        Lane<VEC> g;
        norm_param<VEC>(p.gamma, p.param_f32, c, g);
#pragma unroll
        for (int j = 0; j < N; ++j) a.e[j] = vmul(a.e[j], g.e[j]);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) xh.e[j] = vmul(vsub(xh.e[j], mu), rstd);
    };
    E s1 = both<E>(0.f), s2 = both<E>(0.f);
    for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
      Lane<VEC> a, xh;
      load(c, a, xh);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s1 = vfma(a.e[j], xh.e[j], s1);
        s2 = vadd(s2, a.e[j]);
      }
    }
    const float2 s = rg.sum(vsum(s1), vsum(s2));
    const E c1 = both<E>(-s.x * inv_d), c2 = both<E>(p.mean ? s.y * inv_d : 0.f);
    for (int64_t c = threadIdx.x * VEC; c < p.d; c += span) {
      Lane<VEC> a, xh;
      load(c, a, xh);
#pragma unroll
      for (int j = 0; j < N; ++j) a.e[j] = vmul(vfma(xh.e[j], c1, vsub(a.e[j], c2)), rstd);
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
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  Lane<VEC> dg, db;
#pragma unroll
  for (int j = 0; j < N; ++j) dg.e[j] = db.e[j] = both<E>(0.f);
  if (col < p.d) {
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * NORM_COL_WARPS + warp; row < p.T;
         row += static_cast<int64_t>(gridDim.y) * NORM_COL_WARPS) {
      const E mu = both<E>(p.mean ? p.mean[row] : 0.f), rstd = both<E>(p.rstd[row]);
      Lane<VEC> a, x;
      norm_load<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.d + col, a);
      norm_load_x<TX, VEC, Q8>(p, row, col, x);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        dg.e[j] = vfma(a.e[j], vmul(vsub(x.e[j], mu), rstd), dg.e[j]);
        db.e[j] = vadd(db.e[j], a.e[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    s[warp][j][lane] = dg.get(j);
    s[warp][VEC + j][lane] = db.get(j);
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
