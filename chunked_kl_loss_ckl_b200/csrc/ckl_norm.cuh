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
// 16-byte loads (VEC = 8 bf16, 4 fp32) need d % VEC == 0 and 16-byte pointers;
// VEC = 1 takes the rest.  Groups take rows in a grid-stride loop.
//
// An SM needs about 35 KB of loads under way to keep HBM busy, and a row's
// sums are a dependent chain during which a thread would load nothing.  So
// with 16-byte loads a thread copies its own vectors of the next rows to shared
// memory (cp.async, NORM stages of them) and only ever reads what it copied
// itself: no barrier and no wait on another thread.
//
// The backward reads x, or the 8 bits the forward kept of it (ckl_act8.cuh).
// A thread adds its columns' dgamma and dbeta over its rows in fp32 registers;
// the block's groups are added in shared memory, and a second kernel adds the
// blocks' sums ("parts", in the workspace) in a fixed order, so that results
// do not change from run to run.
//
// Rows too long for registers (d > 16384, fp32 gradients and element-wise rows
// > 8192) are read again from L1 / L2 for each of their sums, and their
// gradients' sums over T get a kernel of their own.
//
// On a B200 (share of the copy bandwidth, 6.54 TB/s): forward 16384 x 4096 bf16
// 48 us (0.86), 4096 x 8192 fp32 43 to 45 us (0.91 to 0.96); backward 68 us
// (0.91); forward with the 8-bit copy 63 us (0.82); backward from it 74 us (0.70);
// backward 4096 x 16384 83 us (0.75), from 8 bits 127 us (0.41; 72 bytes of spills
// a thread).  The backward from 8 bits is bound by latency: no unit is above 62 %
// (issue slots), with a quarter of the SM's warps.  A row's fixed cost is what
// short rows pay: backward 131072 x 256 50 us (0.62).  Element-wise rows are bound
// by the instructions that two bytes at a time take: 16384 x 1001 bf16 43 us
// forward (0.23), 42 us backward (0.36); their backward from 8 bits spills (472
// bytes a thread above 4096 columns).  Long rows, launch included: 4096 x 20000
// bf16 100 us forward (0.50), 188 us backward (0.40); 1024 x 100003 801 and 805 us
// (0.08 and 0.12: element-wise).
#pragma once

#include "ckl_act8.cuh"
#include "ckl_ptx.cuh"

namespace ckl {

constexpr int NORM_THREADS = 512;
constexpr int NORM_WARPS = 16;  // of a block, at most
// Blocks whose gradient sums the workspace holds: one an SM (148 on a B200; a
// launch takes no more than this, whatever the device has), and where the sums
// have a kernel of their own (every d above NORM_REGS_D) one for 64 rows, 64 at
// most.
constexpr int NORM_MAX_PARTS = 160;
constexpr int NORM_REGS_D = 16384;
__host__ __device__ constexpr int64_t norm_cols_parts(int64_t T) {
  return (T + 63) / 64 < 64 ? (T + 63) / 64 : 64;
}

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

// n = 16 (4, 8) bytes, or 0: zeros are written and nothing is read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_bytes(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
               "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Stages of a ring whose stage takes `bytes` a thread: as many as fit in 200 KB
// for 512 threads, four at most.
__host__ __device__ constexpr int norm_stages(int bytes) {
  return 200 * 1024 / (512 * bytes) >= 4 ? 4 : 200 * 1024 / (512 * bytes);
}
// Of the forward where two blocks share an SM.
__host__ __device__ constexpr int norm_fwd_stages(int bytes) { return bytes <= 32 ? 3 : 2; }
template <int NV>
constexpr int NORM_FWD_BYTES = NV * 16;
template <typename TX, int NV, bool Q8>
constexpr int NORM_BWD_BYTES = NV * (16 + (Q8 ? VEC16<TX> : 16));

// What the warps of a row's group tell each other through shared memory: two
// numbers a warp.  Two buffers take turns, so that one barrier an exchange is
// enough.  Lane l reads those of warp l mod `span` (4, 8 or 16, at least the
// row's warps, 16 at most), so that log2(span) butterfly steps leave a sum over
// the warps in every lane of a half.
struct RowGroup {
  float2* red;  // [2][NORM_WARPS]
  int buf, warps, span, at, bar, tpr;
  bool on;  // the lane's warp exists
  __device__ __forceinline__ RowGroup(float2* r, int tpr_)
      : red(r), buf(0), warps(tpr_ / 32), bar(1 + threadIdx.x / tpr_), tpr(tpr_) {
    span = warps <= 4 ? 4 : warps <= 8 ? 8 : 16;
    const int w = threadIdx.x & (span - 1);
    on = w < warps;
    at = (threadIdx.x / tpr_) * warps + (on ? w : 0);
  }
  __device__ __forceinline__ void barrier() const {
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
  }
  __device__ __forceinline__ float2 exchange(float a, float b) {
    if ((threadIdx.x & 31) == 0) red[buf + (threadIdx.x >> 5)] = make_float2(a, b);
    barrier();
    const float2 v = red[buf + at];
    buf ^= NORM_WARPS;
    return v;
  }
  __device__ __forceinline__ float over_warps(float v) const {
    if (span > 8) v += __shfl_xor_sync(0xffffffffu, v, 8);
    if (span > 4) v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    return v + __shfl_xor_sync(0xffffffffu, v, 1);
  }
  // Sums over the row, the same in all of its threads.  The first step swaps
  // halves: lanes 0-15 go on with a, 16-31 with b, so that two sums take the
  // shuffles of one.
  __device__ __forceinline__ float2 sum(float a, float b) {
    const bool hi = threadIdx.x & 16;
    float v = hi ? b : a;
    v += __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps > 1) {
      float* f = reinterpret_cast<float*>(red + buf);
      if ((threadIdx.x & 15) == 0) f[2 * (threadIdx.x >> 5) + hi] = v;
      barrier();
      v = on ? f[2 * at + hi] : 0.f;
      v = over_warps(v);
      buf ^= NORM_WARPS;
    }
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  }
};

template <typename TX, int VEC>
__device__ __forceinline__ void norm_load(const TX* p, Lane<VEC>& v) {
  if constexpr (VEC == 1) {
    v.e[0] = to_f32(*p);
  } else if constexpr (VEC == VEC16<TX>) {
    Raw<TX> r;
    r.load(p);
    r.get(v);
  } else if constexpr (sizeof(TX) == 4) {  // eight floats
    Raw<float> r;
    Lane<4> lo, hi;
    r.load(p);
    r.get(lo);
    r.load(p + 4);
    r.get(hi);
    v.e[0] = lo.e[0];
    v.e[1] = lo.e[1];
    v.e[2] = hi.e[0];
    v.e[3] = hi.e[1];
  } else {  // four bf16
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v.e[0] = bf16x2_widen(w.x);
    v.e[1] = bf16x2_widen(w.y);
  }
}

// gamma's or beta's elements, `none` each without one.
template <int VEC>
__device__ __forceinline__ void norm_param(const void* p, int f32, float none, int64_t col,
                                           Lane<VEC>& v) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < Lane<VEC>::N; ++j) v.e[j] = both<typename Lane<VEC>::E>(none);
  } else if (f32) {
    norm_load<float, VEC>(static_cast<const float*>(p) + col, v);
  } else {
    norm_load<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(p) + col, v);
  }
}

template <typename TX, int VEC>
__device__ __forceinline__ void norm_store(TX* p, const Lane<VEC>& v) {
  if constexpr (VEC == 1) {
    *p = from_f32<TX>(v.e[0]);
  } else if constexpr (VEC == VEC16<TX>) {
    Raw<TX> r;
    r.set(v);
    r.store(p);
  } else {  // eight floats (sums of the gradients)
    static_assert(sizeof(TX) == 4 && VEC == 8, "sums are floats");
    reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(v.e[0], v.e[1]);
    reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(v.e[2], v.e[3]);
  }
}

// gamma or beta in fp32 in shared memory, for kernels that pass over many rows:
// planes of four floats a vector, so that reads do not conflict, filled up to
// the threads' columns (span >= d).
template <int VEC>
__device__ __forceinline__ void norm_stage_param(const void* p, int f32, float none, int32_t d,
                                                 int32_t span, uint8_t* to) {
  for (int c = threadIdx.x; c < span / VEC; c += blockDim.x) {
    Lane<VEC> v;
    norm_param<VEC>(VEC * c < d ? p : nullptr, f32, none, VEC * c, v);
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h)
      reinterpret_cast<ulonglong2*>(to)[h * (span / VEC) + c] =
          make_ulonglong2(v.e[2 * h], v.e[2 * h + 1]);
  }
}
template <int VEC>
__device__ __forceinline__ void norm_staged(const uint8_t* from, int32_t span, int col,
                                            Lane<VEC>& v) {
#pragma unroll
  for (int h = 0; h < VEC / 4; ++h) {
    const ulonglong2 w =
        reinterpret_cast<const ulonglong2*>(from)[h * (span / VEC) + col / VEC];
    v.e[2 * h] = w.x;
    v.e[2 * h + 1] = w.y;
  }
}

// x's elements at `col` of a row, from x or from its 8 bits.
template <typename TX, int VEC, bool Q8>
__device__ __forceinline__ void norm_load_x(const NormBwd& p, int64_t row, int64_t col,
                                            Lane<VEC>& v) {
  if constexpr (!Q8) {
    norm_load<TX, VEC>(static_cast<const TX*>(p.x) + row * p.d + col, v);
  } else {
    const uint32_t b = p.e[row * p.groups + col / 32];
    if constexpr (VEC == 1) {
      v.e[0] = act8_value1(p.q[row * p.d + col], act8_scale(b));
    } else {
      Bytes<VEC> q;
      q.load(p.q + row * p.d + col);
      act8_unpack<VEC>(q, b, v);
    }
  }
}

// The 8-bit copy of one vector or element: all lanes of the warp take
// part in the groups' maxima, `on` says whether the columns exist.
template <int VEC>
__device__ __forceinline__ void norm_keep8(const NormFwd& p, int64_t row, int64_t col, bool on,
                                           const Lane<VEC>& v, uint32_t top) {
  if constexpr (VEC > 1) {
    Bytes<VEC> q;
    const uint32_t b = act8_pack<VEC>(v, top, q);
    if (on) {
      q.store(p.q + row * p.d + col);
      if (threadIdx.x % (32 / VEC) == 0) p.e[row * p.groups + col / 32] = static_cast<uint8_t>(b);
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
//
// STAGED: gamma and beta in shared memory and 64 registers, so that two blocks
// run on an SM (the sums are a chain of shuffles that only other warps hide);
// otherwise they are in registers.  With 32 elements a thread then (RELOAD) the
// row is read from shared memory for each of its three uses: more rows are
// under way, and a chain's shuffles are shared by twice the elements.  KEEP:
// x's 8 bits are written too.
template <typename TX, int VEC, int NV, bool STAGED, bool KEEP>
__global__ void __launch_bounds__(NORM_THREADS, STAGED ? 2 : 1) norm_fwd_kernel(const NormFwd p) {
  constexpr int BYTES = NORM_FWD_BYTES<NV>;
  constexpr int S =
      VEC == 1 ? 1 : STAGED ? norm_fwd_stages(BYTES) : norm_stages(BYTES);
  constexpr bool RELOAD = STAGED && VEC * NV > 16;
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float2 red[2 * NORM_WARPS];
  __shared__ float cols[NORM_WARPS];  // columns of each warp
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, G = blockDim.x / p.tpr;
  RowGroup rg(red, p.tpr);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const bool center = p.mean != nullptr;
  const int step = p.tpr * VEC;  // columns from a thread's vector to its next
  const int col0 = t * VEC;
  // only a thread's last vector may be past the row's end: it is zeros then,
  // worked on like the others and not stored
  auto on = [&](int i) { return (VEC > 1 && i < NV - 1) || col0 + i * step < p.d; };
  const float last = on(NV - 1) ? 1.f : 0.f;
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (on(i)) n += VEC;
  const float nw = static_cast<float>(__reduce_add_sync(0xffffffffu, n));
  const float inv_nw = nw > 0.f ? 1.f / nw : 0.f;
  if ((threadIdx.x & 31) == 0) cols[threadIdx.x >> 5] = nw;
  // vectors of a row in shared memory: 16-byte pieces, a thread's own
  const uint32_t piece = blockDim.x * 16, stage_bytes = BYTES * blockDim.x;
  uint8_t* const mine = norm_smem + threadIdx.x * 16;

  const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(gridDim.x) * group + blockIdx.x;
  int64_t row_in = row;  // the next row to fetch
  const TX* in = static_cast<const TX*>(p.x) + row * p.d + col0;
  auto fetch = [&](uint32_t at) {
    if constexpr (VEC > 1) {
      if (row_in < p.T) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          cp_async16(at + i * piece, in + (on(i) ? i * step : 0), on(i) ? 16u : 0u);
        row_in += stride;
        in += stride * p.d;
      }
      cp_async_commit();
    }
  };
  if constexpr (VEC > 1)
    for (int s = 0; s < S - 1; ++s) fetch(smem_u32(mine) + s * stage_bytes);
  // VEC = 1: the next row's elements, in registers
  float next[NV];
  auto ahead = [&](int64_t r) {
    if constexpr (VEC == 1) {
      if (r >= p.T) return;
      const TX* x = static_cast<const TX*>(p.x) + r * p.d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float v = to_f32(x[on(i) ? col0 + i * step : 0]);
        next[i] = on(i) ? v : 0.f;
      }
    }
  };
  ahead(row);
  // gamma and beta: the thread's columns in registers, or all in shared memory
  uint8_t* const gs = norm_smem + S * stage_bytes;
  uint8_t* const bs = gs + 4 * NV * step;
  Lane<VEC> g[NV], b[NV];
  if constexpr (STAGED) {
    norm_stage_param<VEC>(p.gamma, p.param_f32, 1.f, p.d, NV * step, gs);
    norm_stage_param<VEC>(p.beta, p.param_f32, 0.f, p.d, NV * step, bs);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      norm_param<VEC>(on(i) ? p.gamma : nullptr, p.param_f32, 1.f, col0 + i * step, g[i]);
      norm_param<VEC>(on(i) ? p.beta : nullptr, p.param_f32, 0.f, col0 + i * step, b[i]);
    }
  }
  __syncthreads();
  const float n_lane = rg.on ? cols[rg.at] : 0.f;
  uint32_t off = 0;  // of the current row's stage
  TX* out = static_cast<TX*>(p.y) + row * p.d + col0;
  for (; row < p.T; row += stride) {
    Lane<VEC> v[NV];
    uint32_t top[NV];
    auto get = [&](int i) {
      if constexpr (VEC > 1) {
        Raw<TX> raw;
        raw.load(mine + off + i * piece);
        raw.get(v[i]);
        if constexpr (KEEP) top[i] = raw.top();
      }
    };
    if constexpr (VEC > 1) {
      fetch(smem_u32(mine) + (off == 0 ? (S - 1) * stage_bytes : off - stage_bytes));
      cp_async_wait<S - 1>();
      if constexpr (!RELOAD)
#pragma unroll
        for (int i = 0; i < NV; ++i) get(i);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i].e[0] = next[i];
      ahead(row + stride);
    }

    float mu = 0.f;
    if (center) {
      E s = both<E>(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if constexpr (RELOAD) get(i);
#pragma unroll
        for (int j = 0; j < N; ++j) s = vadd(s, v[i].e[j]);
      }
      mu = vsum(s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mu += __shfl_xor_sync(0xffffffffu, mu, o);
      mu *= inv_nw;
    }
    E ss = both<E>(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (RELOAD) get(i);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        E c = vsub(v[i].e[j], both<E>(mu));
        if (VEC == 1) c = on(i) ? c : both<E>(0.f);
        else if (i == NV - 1) c = vmul(c, both<E>(last));
        ss = vfma(c, c, ss);
      }
    }
    float m2 = vsum(ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
    if (rg.warps > 1) {
      const float2 w = rg.exchange(mu, m2);
      m2 = rg.on ? w.y : 0.f;
      if (center) {
        mu = rg.over_warps(w.x * n_lane) * inv_d;
        // (a lane without a warp adds nothing, where the square is infinite too)
        if (rg.on) m2 = fmaf((w.x - mu) * (w.x - mu), n_lane, m2);
      }
      m2 = rg.over_warps(m2);
    }
    const float rstd = rsqrtf(fmaf(m2, inv_d, p.eps));
    if (t == 0) {
      if (center) p.mean[row] = mu;
      p.rstd[row] = rstd;
    }

#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col0 + i * step;
      if constexpr (RELOAD) get(i);
      if constexpr (KEEP) norm_keep8<VEC>(p, row, col, on(i), v[i], VEC > 1 ? top[i] : 0u);
      if constexpr (STAGED) {
        norm_staged<VEC>(gs, NV * step, col, g[i]);
        norm_staged<VEC>(bs, NV * step, col, b[i]);
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        v[i].e[j] = vfma(vmul(vsub(v[i].e[j], both<E>(mu)), both<E>(rstd)), g[i].e[j], b[i].e[j]);
      if (on(i)) norm_store<TX, VEC>(out + i * step, v[i]);
    }
    if constexpr (VEC > 1) off = off == (S - 1) * stage_bytes ? 0 : off + stage_bytes;
    out += stride * p.d;
  }
}

// Rows of any length: a block a row, read three times.
template <typename TX, int VEC>
__global__ void __launch_bounds__(NORM_THREADS) norm_fwd_long_kernel(const NormFwd p) {
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  __shared__ float2 red[2 * NORM_WARPS];
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
      if constexpr (VEC > 1) {
        Raw<TX> r;
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
      norm_param<VEC>(p.gamma, p.param_f32, 1.f, c, g);
      norm_param<VEC>(p.beta, p.param_f32, 0.f, c, b);
#pragma unroll
      for (int j = 0; j < N; ++j)
        v.e[j] = vfma(vmul(vsub(v.e[j], both<E>(mu)), both<E>(rstd)), g.e[j], b.e[j]);
      norm_store<TX, VEC>(static_cast<TX*>(p.y) + row * p.d + c, v);
    }
  }
}

// ------------------------------------------------------------------ backward
// With 32 elements a thread (RELOAD) the gradients' sums take 64 registers, and
// the row is read from shared memory a second time instead of being held in
// another 64.
template <int VEC, int NV>
constexpr bool NORM_RELOAD = VEC * NV > 16 && VEC > 1;
template <typename TX, int VEC, int NV, bool Q8>
__host__ __device__ constexpr int norm_bwd_stages() {
  return NORM_RELOAD<VEC, NV> ? 2 : norm_stages(NORM_BWD_BYTES<TX, NV, Q8>);
}

template <typename TX, int VEC, int NV, bool Q8, bool STAGED>
__global__ void __launch_bounds__(NORM_THREADS) norm_bwd_kernel(const NormBwd p) {
  constexpr bool RELOAD = NORM_RELOAD<VEC, NV>;
  constexpr int BYTES = NORM_BWD_BYTES<TX, NV, Q8>;
  constexpr int S = VEC == 1 ? 1 : norm_bwd_stages<TX, VEC, NV, Q8>();
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float2 red[2 * NORM_WARPS];
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, G = blockDim.x / p.tpr;
  RowGroup rg(red, p.tpr);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int step = p.tpr * VEC;  // columns from a thread's vector to its next
  const int col0 = t * VEC;
  // only a thread's last vector may be past the row's end: dy is zeros there, which
  // adds nothing to a sum as long as xh is finite where the row's is.  So x is one
  // of the row's own vectors then (`elsewhere`: the thread's first, or the row's;
  // VEC = 1: the row's last) and not zeros, whose mean r may pass the largest float.
  auto on = [&](int i) { return (VEC > 1 && i < NV - 1) || col0 + i * step < p.d; };
  const int elsewhere = NV > 1 ? 0 : -col0;
  Lane<VEC> dg[NV], db[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) dg[i].e[j] = db[i].e[j] = both<E>(0.f);
  // a stage: dy's 16-byte pieces, then x's, or q's pieces of VEC bytes
  const uint32_t piece = blockDim.x * 16, stage_bytes = BYTES * blockDim.x;
  uint8_t* const mine = norm_smem + threadIdx.x * 16;
  uint8_t* const mine8 = norm_smem + NV * piece + threadIdx.x * VEC;
  uint8_t* const gs = norm_smem + S * stage_bytes;

  const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(gridDim.x) * group + blockIdx.x;
  int64_t row_in = row, at_in = row * p.d + col0;  // the next row to fetch, its first element
  auto fetch = [&](uint32_t off) {
    if constexpr (VEC > 1) {
      if (row_in < p.T) {
        const TX* dy = static_cast<const TX*>(p.dy) + at_in;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int o = on(i) ? i * step : elsewhere;
          cp_async16(smem_u32(mine) + off + i * piece, dy + o, on(i) ? 16u : 0u);
          if constexpr (Q8)
            cp_async_bytes<VEC>(smem_u32(mine8) + off + i * blockDim.x * VEC, p.q + at_in + o, VEC);
          else
            cp_async16(smem_u32(mine) + off + (NV + i) * piece,
                       static_cast<const TX*>(p.x) + at_in + o, 16u);
        }
        row_in += stride;
        at_in += stride * p.d;
      }
      cp_async_commit();
    }
  };
  // what a row has besides (VEC = 1: all of it): loaded a row ahead
  float mu_next = 0.f, rstd_next = 0.f;
  float dy_next[NV], x_next[NV];
  uint32_t e_next[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) e_next[i] = 133;
  auto ahead = [&](int64_t r) {
    if (r >= p.T) return;
    if (p.mean) mu_next = p.mean[r];
    rstd_next = p.rstd[r];
    if constexpr (Q8 && VEC > 1) {
      const uint8_t* e = p.e + r * p.groups + col0 / 32;
#pragma unroll
      for (int i = 0; i < NV; ++i)  // step is a multiple of 128
        e_next[i] = e[on(i) ? i * (step / 32) : NV > 1 ? 0 : -(col0 / 32)];
    }
    if constexpr (VEC == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = on(i) ? col0 + i * step : p.d - 1;
        Lane<1> x;
        norm_load_x<TX, 1, Q8>(p, r, c, x);
        const float dy = to_f32(static_cast<const TX*>(p.dy)[r * p.d + c]);
        x_next[i] = x.e[0];
        dy_next[i] = on(i) ? dy : 0.f;
      }
    }
  };
  if constexpr (VEC > 1)
    for (int s = 0; s < S - 1; ++s) fetch(s * stage_bytes);
  ahead(row);
  Lane<VEC> g1[NV];  // VEC = 1: the thread's columns of gamma
  if constexpr (VEC == 1)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      norm_param<VEC>(on(i) ? p.gamma : nullptr, p.param_f32, 1.f, col0 + i * step, g1[i]);
  if constexpr (STAGED) {
    norm_stage_param<VEC>(p.gamma, p.param_f32, 1.f, p.d, NV * step, gs);
    __syncthreads();
  }

  uint32_t off = 0;  // of the current row's stage
  TX* out = static_cast<TX*>(p.dx) + row * p.d + col0;
  for (; row < p.T; row += stride) {
    const float mu = mu_next, rstd = rstd_next;
    uint32_t e_row[NV];
    Lane<VEC> a[NV], xh[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      e_row[i] = e_next[i];
      if constexpr (VEC == 1) {
        a[i].e[0] = dy_next[i];
        xh[i].e[0] = x_next[i];
      }
    }
    ahead(row + stride);
    if constexpr (VEC > 1) {
      fetch(off == 0 ? (S - 1) * stage_bytes : off - stage_bytes);
      cp_async_wait<S - 1>();
    }
    // dy, xh and gamma of vector i
    auto get = [&](int i, Lane<VEC>& dy, Lane<VEC>& x, Lane<VEC>& g) {
      if constexpr (VEC == 1) {
        dy = a[i];
        x = xh[i];
        g = g1[i];
      } else {
        Raw<TX> r;
        r.load(mine + off + i * piece);
        r.get(dy);
        if constexpr (Q8) {
          Bytes<VEC> q;
          q.load(mine8 + off + i * blockDim.x * VEC);
          act8_unpack<VEC>(q, e_row[i], x);
        } else {
          r.load(mine + off + (NV + i) * piece);
          r.get(x);
        }
        const int col = col0 + i * step;
        if constexpr (STAGED) norm_staged<VEC>(gs, NV * step, col, g);
        else norm_param<VEC>(on(i) ? p.gamma : nullptr, p.param_f32, 1.f, col, g);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) x.e[j] = vmul(vsub(x.e[j], both<E>(mu)), both<E>(rstd));
    };
    E s1 = both<E>(0.f), s2 = both<E>(0.f);  // of a xh, of a
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Lane<VEC> dy, x, g;
      get(i, dy, x, g);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        dg[i].e[j] = vfma(dy.e[j], x.e[j], dg[i].e[j]);
        db[i].e[j] = vadd(db[i].e[j], dy.e[j]);
        const E ag = vmul(dy.e[j], g.e[j]);
        s1 = vfma(ag, x.e[j], s1);
        s2 = vadd(s2, ag);
        if constexpr (!RELOAD) {
          a[i].e[j] = ag;
          xh[i].e[j] = x.e[j];
        }
      }
    }
    const float2 c = rg.sum(vsum(s1), vsum(s2));
    const E c1 = both<E>(-c.x * inv_d), c2 = both<E>(p.mean ? c.y * inv_d : 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (RELOAD) {
        Lane<VEC> g;
        get(i, a[i], xh[i], g);
#pragma unroll
        for (int j = 0; j < N; ++j) a[i].e[j] = vmul(a[i].e[j], g.e[j]);
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        a[i].e[j] = vmul(vfma(xh[i].e[j], c1, vsub(a[i].e[j], c2)), both<E>(rstd));
      if (on(i)) norm_store<TX, VEC>(out + i * step, a[i]);
    }
    out += stride * p.d;
    off = off == (S - 1) * stage_bytes ? 0 : off + stage_bytes;
  }
  if (!p.want_gamma && !p.want_beta) return;
  griddep_launch();  // norm_reduce_kernel may start; it waits for this kernel's end

  // the block's groups, one after another, into the first
  float* sums = reinterpret_cast<float*>(norm_smem);
  __syncthreads();  // the ring is read
  for (int k = 1; k < G; ++k) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col0 + i * step;
      if (group != k || !on(i)) continue;
      norm_store<float, VEC>(sums + col, dg[i]);
      norm_store<float, VEC>(sums + p.d + col, db[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col0 + i * step;
      if (group != 0 || !on(i)) continue;
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
    const int col = col0 + i * step;
    if (!on(i)) continue;
    if (p.want_gamma) norm_store<float, VEC>(part + col, dg[i]);
    if (p.want_beta) norm_store<float, VEC>(part + p.d + col, db[i]);
  }
}

// Rows of any length: dx, a block a row, read twice.
template <typename TX, int VEC, bool Q8>
__global__ void __launch_bounds__(NORM_THREADS) norm_bwd_long_kernel(const NormBwd p) {
  using E = typename Lane<VEC>::E;
  constexpr int N = Lane<VEC>::N;
  __shared__ float2 red[2 * NORM_WARPS];
  RowGroup rg(red, NORM_THREADS);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int64_t span = static_cast<int64_t>(NORM_THREADS) * VEC;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const E mu = both<E>(p.mean ? p.mean[row] : 0.f), rstd = both<E>(p.rstd[row]);
    auto load = [&](int64_t c, Lane<VEC>& a, Lane<VEC>& xh) {
      norm_load<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.d + c, a);
      norm_load_x<TX, VEC, Q8>(p, row, c, xh);
      Lane<VEC> g;
      norm_param<VEC>(p.gamma, p.param_f32, 1.f, c, g);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        a.e[j] = vmul(a.e[j], g.e[j]);
        xh.e[j] = vmul(vsub(xh.e[j], mu), rstd);
      }
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

constexpr int NORM_RED_COLS = 32, NORM_RED_ROWS = 32;

// dgamma (blockIdx.y = 0) and dbeta (1): the sum of the blocks' parts, 32
// columns a block, the parts shared by 32 threads a column.  Launched so that
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
#pragma unroll 8
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
