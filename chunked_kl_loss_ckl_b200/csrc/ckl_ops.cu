// Host side of the operators around the loss: argument checks and launches.
// See include/ckl_ops.h for the contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/ckl_ops.h"
#include "ckl_act8.cuh"
#include "ckl_norm.cuh"
#include "ckl_sample.cuh"

static_assert(CKL_ACT8_GROUP == ckl::ACT8_GROUP && CKL_SAMPLE_BAD_INPUT == CKL_DEV_BAD_SAMPLE,
              "the header's constants");

namespace {

using bf16 = __nv_bfloat16;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

struct OpsDev {
  int sms = 0, major = 0;
};

// CKL_OK, or why the current device cannot be used.
int ops_device(OpsDev& out) {
  static std::mutex mu;
  static OpsDev cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CKL_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  OpsDev& d = cache[dev];
  if (d.sms == 0 &&
      (cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
       cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)) {
    d = OpsDev();
    return CKL_ERR_CUDA;
  }
  out = d;
  return d.major == 10 ? CKL_OK : CKL_ERR_UNSUPPORTED;
}

int launched() { return cudaGetLastError() == cudaSuccess ? CKL_OK : CKL_ERR_CUDA; }

size_t elem_bytes(int32_t dtype) { return dtype == CKL_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == CKL_DTYPE_BF16 || dtype == CKL_DTYPE_F32; }

constexpr int64_t kLim = (int64_t(1) << 31) - 1;

bool act8_sizes_ok(int64_t T, int64_t d) {
  return T >= 0 && d >= 1 && d < kLim - 64 && T < (int64_t(1) << 62) / (d + 32);
}

template <typename TX>
void act8_pack_launch(const void* x, int64_t T, int64_t d, int8_t* q, uint8_t* e, bool vec,
                      int sms, cudaStream_t st) {
  const int64_t groups = cdiv(d, 32);
  const int64_t thr = T * groups * (vec ? 4 : 32);
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(cdiv(thr, ckl::ACT8_THREADS), static_cast<int64_t>(sms) * 8));
  auto* k = vec ? ckl::act8_pack_kernel<TX, true> : ckl::act8_pack_kernel<TX, false>;
  k<<<grid, ckl::ACT8_THREADS, 0, st>>>(static_cast<const TX*>(x), T, static_cast<int32_t>(d),
                                        static_cast<int32_t>(groups), q, e);
}

template <typename TX>
void act8_unpack_launch(const int8_t* q, const uint8_t* e, int64_t T, int64_t d, void* x,
                        bool vec, int sms, cudaStream_t st) {
  const int64_t groups = cdiv(d, 32);
  const int64_t thr = T * groups * (vec ? 4 : 32);
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(cdiv(thr, ckl::ACT8_THREADS), static_cast<int64_t>(sms) * 8));
  auto* k = vec ? ckl::act8_unpack_kernel<TX, true> : ckl::act8_unpack_kernel<TX, false>;
  k<<<grid, ckl::ACT8_THREADS, 0, st>>>(q, e, T, static_cast<int32_t>(d),
                                        static_cast<int32_t>(groups), static_cast<TX*>(x));
}

// How a norm's rows are taken: `vec` elements a load, `nv` vectors a thread,
// `tpr` threads a row, `threads` a block; nv 0 = the kernels for long rows.
struct NormShape {
  int vec, nv, tpr, threads;
};

// `want_nv` vectors a thread where a row has that many for two warps: what a
// row costs a warp beside its elements (sums over lanes and warps, a barrier)
// is then shared by more of them.  Four vectors where 512 threads need them, if
// the kernel has that form (max_nv).
NormShape norm_shape(int64_t d, bool vec, int want_nv, int max_nv) {
  NormShape s{vec ? 8 : 1, 0, 0, 0};
  const int64_t n = cdiv(d, s.vec);  // vectors of a row
  if (n > static_cast<int64_t>(ckl::NORM_THREADS) * max_nv) return s;
  if (!vec) s.nv = n <= ckl::NORM_THREADS * 8 ? 8 : 16;
  else if (n > ckl::NORM_THREADS * want_nv) s.nv = 4;
  else s.nv = n <= 32 ? 1 : n <= 64 ? 2 : want_nv;
  s.tpr = static_cast<int>(cdiv(cdiv(n, s.nv), 32) * 32);
  s.threads = ckl::NORM_THREADS / s.tpr * s.tpr;
  return s;
}

constexpr size_t kNormSmem = 220 * 1024;  // of a block, its ring and parameters

template <typename P>
int norm_launch(void (*k)(P), const P& p, dim3 grid, int threads, size_t smem, cudaStream_t st) {
  // 48 KB, the kernel's static part included, need no opting in
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return CKL_ERR_CUDA;
  k<<<grid, threads, smem, st>>>(p);
  return launched();
}

template <typename TX>
int norm_fwd_launch(const ckl::NormFwd& p, const NormShape& s, int sms, cudaStream_t st) {
  using ckl::NORM_FWD_BYTES;
  using ckl::norm_stages;
  const int64_t rows = std::min<int64_t>(p.T, static_cast<int64_t>(sms) * 4);
  if (s.nv == 0)
    return norm_launch(s.vec == 8 ? ckl::norm_fwd_long_kernel<TX, 8>
                                  : ckl::norm_fwd_long_kernel<TX, 1>,
                       p, dim3(static_cast<unsigned>(rows)), ckl::NORM_THREADS, 0, st);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(p.T, sms)));
  auto go = [&](void (*k)(ckl::NormFwd), int bytes) {
    const size_t ring = static_cast<size_t>(s.threads) * bytes * norm_stages(bytes);
    const size_t params = static_cast<size_t>(p.d) * 4 * ((p.gamma != nullptr) + (p.beta != nullptr));
    ckl::NormFwd f = p;
    f.staged = p.T > sms && ring + params <= kNormSmem;
    return norm_launch(k, f, grid, s.threads, f.staged ? ring + params : ring, st);
  };
  if (s.vec == 8)
    return s.nv == 1   ? go(ckl::norm_fwd_kernel<TX, 8, 1>, NORM_FWD_BYTES<TX, 1>)
           : s.nv == 2 ? go(ckl::norm_fwd_kernel<TX, 8, 2>, NORM_FWD_BYTES<TX, 2>)
                       : go(ckl::norm_fwd_kernel<TX, 8, 4>, NORM_FWD_BYTES<TX, 4>);
  return norm_launch(s.nv == 8 ? ckl::norm_fwd_kernel<TX, 1, 8> : ckl::norm_fwd_kernel<TX, 1, 16>,
                     p, grid, s.threads, 0, st);
}

// Returns the status; `parts` is how many sums the workspace then holds.
template <typename TX, bool Q8>
int norm_bwd_launch(const ckl::NormBwd& p, const NormShape& s, int sms, cudaStream_t st,
                    int& parts) {
  using ckl::NORM_BWD_BYTES;
  using ckl::norm_stages;
  if (s.nv == 0) {
    parts = static_cast<int>(std::min<int64_t>(cdiv(p.T, 8 * ckl::NORM_COL_WARPS), 64));
    if (p.want_gamma || p.want_beta) {  // first: dx may take dy's place
      const dim3 grid(static_cast<unsigned>(cdiv(p.d, 32 * s.vec)), static_cast<unsigned>(parts));
      const int rc = norm_launch(s.vec == 8 ? ckl::norm_cols_kernel<TX, 8, Q8>
                                            : ckl::norm_cols_kernel<TX, 1, Q8>,
                                 p, grid, 32 * ckl::NORM_COL_WARPS, 0, st);
      if (rc != CKL_OK) return rc;
    }
    return norm_launch(s.vec == 8 ? ckl::norm_bwd_long_kernel<TX, 8, Q8>
                                  : ckl::norm_bwd_long_kernel<TX, 1, Q8>,
                       p, dim3(static_cast<unsigned>(std::min<int64_t>(p.T, sms * 4))),
                       ckl::NORM_THREADS, 0, st);
  }
  parts = static_cast<int>(std::min<int64_t>(p.T, std::min(sms, ckl::NORM_MAX_PARTS)));
  const dim3 grid(static_cast<unsigned>(parts));
  const size_t sums = static_cast<size_t>(p.d) * 8;  // a row group's, on the way to the first's
  auto go = [&](void (*k)(ckl::NormBwd), int bytes) {
    const size_t ring = static_cast<size_t>(s.threads) * bytes * norm_stages(bytes);
    const size_t params = p.gamma ? static_cast<size_t>(p.d) * 4 : 0;
    ckl::NormBwd f = p;
    f.staged = p.T > sms && ring + params <= kNormSmem;
    return norm_launch(k, f, grid, s.threads, std::max(f.staged ? ring + params : ring, sums), st);
  };
  if (s.vec == 8) {
    if constexpr (sizeof(TX) == 2)
      if (s.nv == 4) return go(ckl::norm_bwd_kernel<TX, 8, 4, Q8>, NORM_BWD_BYTES<TX, 4, Q8>);
    return s.nv == 1 ? go(ckl::norm_bwd_kernel<TX, 8, 1, Q8>, NORM_BWD_BYTES<TX, 1, Q8>)
                     : go(ckl::norm_bwd_kernel<TX, 8, 2, Q8>, NORM_BWD_BYTES<TX, 2, Q8>);
  }
  return norm_launch(s.nv == 8 ? ckl::norm_bwd_kernel<TX, 1, 8, Q8>
                               : ckl::norm_bwd_kernel<TX, 1, 16, Q8>,
                     p, grid, s.threads, sums, st);
}

bool norm_sizes_ok(int64_t T, int64_t d) {
  return T >= 0 && d >= 1 && d < kLim - 65536 && T < (int64_t(1) << 60) / d;
}

}  // namespace

extern "C" {

int ckl_act8_pack(const void* x, int32_t dtype, int64_t T, int64_t d, int8_t* q,
                  uint8_t* exponents, void* stream) {
  if (!act8_sizes_ok(T, d) || !dtype_ok(dtype)) return CKL_ERR_INVALID_ARG;
  if (T > 0 && (!x || !q || !exponents)) return CKL_ERR_INVALID_ARG;
  if (!aligned(x, elem_bytes(dtype))) return CKL_ERR_INVALID_ARG;
  OpsDev dev;
  if (const int rc = ops_device(dev)) return rc;
  if (T == 0) return CKL_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = d % 8 == 0 && aligned(x, 16) && aligned(q, 8);
  if (dtype == CKL_DTYPE_F32)
    act8_pack_launch<float>(x, T, d, q, exponents, vec, dev.sms, st);
  else
    act8_pack_launch<bf16>(x, T, d, q, exponents, vec, dev.sms, st);
  return launched();
}

int ckl_act8_unpack(const int8_t* q, const uint8_t* exponents, int64_t T, int64_t d, int32_t dtype,
                    void* x, void* stream) {
  if (!act8_sizes_ok(T, d) || !dtype_ok(dtype)) return CKL_ERR_INVALID_ARG;
  if (T > 0 && (!x || !q || !exponents)) return CKL_ERR_INVALID_ARG;
  if (!aligned(x, elem_bytes(dtype))) return CKL_ERR_INVALID_ARG;
  OpsDev dev;
  if (const int rc = ops_device(dev)) return rc;
  if (T == 0) return CKL_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = d % 8 == 0 && aligned(x, 16) && aligned(q, 8);
  if (dtype == CKL_DTYPE_F32)
    act8_unpack_launch<float>(q, exponents, T, d, x, vec, dev.sms, st);
  else
    act8_unpack_launch<bf16>(q, exponents, T, d, x, vec, dev.sms, st);
  return launched();
}

int ckl_norm_forward(const void* x, int32_t dtype, const void* gamma, const void* beta,
                     int32_t param_dtype, int64_t T, int64_t d, float eps, void* y, float* mean,
                     float* rstd, int8_t* q, uint8_t* exponents, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !(eps >= 0.f) || std::isinf(eps))
    return CKL_ERR_INVALID_ARG;
  if (!norm_sizes_ok(T, d)) return CKL_ERR_INVALID_ARG;
  if (T > 0 && (!x || !y || !rstd)) return CKL_ERR_INVALID_ARG;
  if ((q == nullptr) != (exponents == nullptr)) return CKL_ERR_INVALID_ARG;
  const size_t eb = elem_bytes(dtype), pb = elem_bytes(param_dtype);
  if (!aligned(x, eb) || !aligned(y, eb) || !aligned(gamma, pb) || !aligned(beta, pb) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return CKL_ERR_INVALID_ARG;
  OpsDev dev;
  if (const int rc = ops_device(dev)) return rc;
  if (T == 0) return CKL_OK;
  const bool vec = d % 8 == 0 && aligned(x, 16) && aligned(y, 16) && aligned(gamma, 16) &&
                   aligned(beta, 16) && aligned(q, 8);
  const NormShape s = norm_shape(d, vec, 4, vec ? 4 : 16);
  ckl::NormFwd p{};
  p.x = x;
  p.gamma = gamma;
  p.beta = beta;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.q = q;
  p.e = exponents;
  p.T = T;
  p.d = static_cast<int32_t>(d);
  p.groups = static_cast<int32_t>(cdiv(d, 32));
  p.tpr = s.tpr;
  p.param_f32 = param_dtype == CKL_DTYPE_F32;
  p.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == CKL_DTYPE_F32 ? norm_fwd_launch<float>(p, s, dev.sms, st)
                                : norm_fwd_launch<bf16>(p, s, dev.sms, st);
}

size_t ckl_norm_workspace_bytes(int64_t T, int64_t d) {
  if (!norm_sizes_ok(T, d)) return 0;
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(T, ckl::NORM_MAX_PARTS));
  return static_cast<size_t>(parts) * 2 * d * 4;
}

int ckl_norm_backward(const void* dy, int32_t dtype, const void* x, const int8_t* q,
                      const uint8_t* exponents, const float* mean, const float* rstd,
                      const void* gamma, int32_t param_dtype, int64_t T, int64_t d, void* dx,
                      float* dgamma, float* dbeta, int32_t accumulate, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return CKL_ERR_INVALID_ARG;
  if (!norm_sizes_ok(T, d)) return CKL_ERR_INVALID_ARG;
  if (T > 0 && (!dy || !dx || !rstd)) return CKL_ERR_INVALID_ARG;
  if (T > 0 && !x && (!q || !exponents)) return CKL_ERR_INVALID_ARG;
  const bool grads = dgamma || dbeta;
  if (grads && !workspace) return CKL_ERR_INVALID_ARG;
  const size_t eb = elem_bytes(dtype), pb = elem_bytes(param_dtype);
  if (!aligned(dy, eb) || !aligned(x, eb) || !aligned(dx, eb) || !aligned(gamma, pb) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4) ||
      !aligned(workspace, 16))
    return CKL_ERR_INVALID_ARG;
  if (grads && workspace_bytes < ckl_norm_workspace_bytes(T, d)) return CKL_ERR_WORKSPACE;
  OpsDev dev;
  if (const int rc = ops_device(dev)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool q8 = x == nullptr;
  const bool vec = d % 8 == 0 && aligned(dy, 16) && aligned(x, 16) && aligned(dx, 16) &&
                   aligned(gamma, 16) && (!q8 || aligned(q, 8));
  const NormShape s = norm_shape(d, vec, 2, !vec ? 16 : dtype == CKL_DTYPE_F32 ? 2 : 4);
  int parts = 0;
  if (T > 0) {
    ckl::NormBwd p{};
    p.dy = dy;
    p.x = x;
    p.q = q;
    p.e = exponents;
    p.mean = mean;
    p.rstd = rstd;
    p.gamma = gamma;
    p.dx = dx;
    p.parts = static_cast<float*>(workspace);
    p.T = T;
    p.d = static_cast<int32_t>(d);
    p.groups = static_cast<int32_t>(cdiv(d, 32));
    p.tpr = s.tpr;
    p.param_f32 = param_dtype == CKL_DTYPE_F32;
    p.want_gamma = dgamma != nullptr;
    p.want_beta = dbeta != nullptr;
    const int rc =
        dtype == CKL_DTYPE_F32
            ? (q8 ? norm_bwd_launch<float, true>(p, s, dev.sms, st, parts)
                  : norm_bwd_launch<float, false>(p, s, dev.sms, st, parts))
            : (q8 ? norm_bwd_launch<bf16, true>(p, s, dev.sms, st, parts)
                  : norm_bwd_launch<bf16, false>(p, s, dev.sms, st, parts));
    if (rc != CKL_OK) return rc;
  }
  if (!grads) return CKL_OK;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(d, ckl::NORM_RED_COLS)), 2);
  cfg.blockDim = dim3(ckl::NORM_RED_COLS * ckl::NORM_RED_ROWS);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ckl::norm_reduce_kernel, static_cast<const float*>(workspace),
                            parts, static_cast<int32_t>(d), dgamma, dbeta, accumulate) ==
                 cudaSuccess
             ? CKL_OK
             : CKL_ERR_CUDA;
}

int ckl_sample(const uint16_t* logits, int64_t ld, int64_t T, int64_t V, const float* u, int32_t N,
               double temperature, int32_t top_k, double top_p, double min_p,
               const float* temperature_rows, const int32_t* top_k_rows, const float* top_p_rows,
               const float* min_p_rows, int32_t* ids, float* logp, int32_t* device_status,
               void* stream) {
  if (T < 0 || V < 1 || ld < V || N < 1 || T >= kLim / N) return CKL_ERR_INVALID_ARG;
  if (T > 0 && ld > (int64_t(1) << 61) / T) return CKL_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !u || !ids)) return CKL_ERR_INVALID_ARG;
  if (!aligned(logits, 2) || !aligned(u, 4) || !aligned(ids, 4) || !aligned(logp, 4) ||
      !aligned(device_status, 4) || !aligned(temperature_rows, 4) || !aligned(top_k_rows, 4) ||
      !aligned(top_p_rows, 4) || !aligned(min_p_rows, 4))
    return CKL_ERR_INVALID_ARG;
  if (!temperature_rows && !(temperature >= 0.0 && std::isfinite(temperature)))
    return CKL_ERR_INVALID_ARG;
  if (!top_p_rows && !(top_p > 0.0)) return CKL_ERR_INVALID_ARG;
  if (!min_p_rows && !(min_p >= 0.0 && min_p <= 1.0)) return CKL_ERR_INVALID_ARG;
  if (V > CKL_SAMPLE_MAX_V) return CKL_ERR_UNSUPPORTED;
  OpsDev dev;
  if (const int rc = ops_device(dev)) return rc;
  if (T == 0) return CKL_OK;
  ckl::SampleParams p{};
  p.logits = logits;
  p.ld = ld;
  p.T = T;
  p.V = static_cast<int32_t>(V);
  p.N = N;
  p.u = u;
  p.temperature = temperature;
  p.top_p = top_p;
  p.min_p = min_p;
  p.top_k = top_k;
  p.temperature_rows = temperature_rows;
  p.top_k_rows = top_k_rows;
  p.top_p_rows = top_p_rows;
  p.min_p_rows = min_p_rows;
  p.ids = ids;
  p.logp = logp;
  p.status = device_status;
  const size_t smem = sizeof(ckl::SampleShared);
  if (cudaFuncSetAttribute(ckl::sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return CKL_ERR_CUDA;
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(T, static_cast<int64_t>(dev.sms) * 3));
  ckl::sample_kernel<<<grid, ckl::SM_THREADS, smem, static_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

}  // extern "C"
