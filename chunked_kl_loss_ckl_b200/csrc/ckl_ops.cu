// Host side of the operators around the loss: argument checks and launches.
// See include/ckl_ops.h for the contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "../../include/ckl_ops.h"
#include "ckl_act8.cuh"
#include "ckl_norm.cuh"
#include "ckl_sample.cuh"

static_assert(CKL_ACT8_GROUP == ckl::ACT8_GROUP && CKL_SAMPLE_BAD_INPUT == CKL_DEV_BAD_SAMPLE,
              "the header's constants");

namespace {

using bf16 = __nv_bfloat16;

constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

struct OpsDev {
  int sms = 0, major = 0;
};

// A runtime call failed: its error is this call's status, and is taken back, as
// it would be read as a later call's otherwise.
int failed() {
  cudaGetLastError();
  return CKL_ERR_CUDA;
}

// Status of one launch, whatever errors earlier calls of the process left.
template <typename... P, typename... A>
int launch(void (*k)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
           cudaLaunchAttribute* attr, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = attr ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...) == cudaSuccess ? CKL_OK : failed();
}

template <typename... P>
bool allow_smem(void (*k)(P...), size_t bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bytes)) == cudaSuccess;
}

// CKL_OK, or why the current device cannot be used.
int ops_device(OpsDev& out) {
  static std::mutex mu;
  static OpsDev cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return failed();
  std::lock_guard<std::mutex> lock(mu);
  OpsDev& d = cache[dev];
  if (d.sms == 0 &&
      (cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
       cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)) {
    d = OpsDev();
    return failed();
  }
  out = d;
  return d.major == 10 ? CKL_OK : CKL_ERR_UNSUPPORTED;
}

size_t elem_bytes(int32_t dtype) { return dtype == CKL_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == CKL_DTYPE_BF16 || dtype == CKL_DTYPE_F32; }

constexpr int64_t kLim = (int64_t(1) << 31) - 1;

bool act8_sizes_ok(int64_t T, int64_t d) {
  return T >= 0 && d >= 1 && d < kLim - 64 && T < (int64_t(1) << 62) / (d + 32);
}

template <typename TX>
int act8_pack_launch(const void* x, int64_t T, int64_t d, int8_t* q, uint8_t* e, int sms,
                     cudaStream_t st) {
  constexpr int V = ckl::VEC16<TX>;
  const bool vec = d % V == 0 && aligned(x, 16) && aligned(q, V);
  const int64_t groups = cdiv(d, 32), thr = T * groups * (vec ? 32 / V : 32);
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(cdiv(thr, ckl::ACT8_THREADS), static_cast<int64_t>(sms) * 8));
  auto* k = vec ? ckl::act8_pack_kernel<TX, V> : ckl::act8_pack_kernel<TX, 1>;
  return launch(k, dim3(grid), ckl::ACT8_THREADS, 0, st, nullptr, static_cast<const TX*>(x), T,
                static_cast<int32_t>(d), static_cast<int32_t>(groups), q, e);
}

template <typename TX>
int act8_unpack_launch(const int8_t* q, const uint8_t* e, int64_t T, int64_t d, void* x, int sms,
                       cudaStream_t st) {
  constexpr int V = ckl::VEC16<TX>;
  const bool vec = d % V == 0 && aligned(x, 16) && aligned(q, V);
  const int64_t groups = cdiv(d, 32), thr = T * groups * (vec ? 32 / V : 32);
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(cdiv(thr, ckl::ACT8_THREADS), static_cast<int64_t>(sms) * 8));
  auto* k = vec ? ckl::act8_unpack_kernel<TX, V> : ckl::act8_unpack_kernel<TX, 1>;
  return launch(k, dim3(grid), ckl::ACT8_THREADS, 0, st, nullptr, q, e, T,
                static_cast<int32_t>(d), static_cast<int32_t>(groups), static_cast<TX*>(x));
}

// How a norm's rows are taken: `vec` elements a load, `nv` vectors a thread,
// `tpr` threads a row, `threads` a block; nv 0 = the kernels for long rows.
struct NormShape {
  int vec, nv, tpr, threads;
};

// Rows of up to 512 threads with `want` vectors a thread; longer ones `more`
// vectors (0: the kernels for long rows).  With the threads chosen first, only
// a thread's last vector may be past the row's end.
constexpr NormShape norm_shape(int64_t d, int vec, int want, int more) {
  NormShape s{vec, 0, 0, 0};
  const int64_t n = cdiv(d, vec);  // vectors of a row
  const int nv = n <= static_cast<int64_t>(ckl::NORM_THREADS) * want ? want : more;
  if (n > static_cast<int64_t>(ckl::NORM_THREADS) * nv) return s;
  s.tpr = static_cast<int>(cdiv(n, 32 * nv) * 32);
  s.nv = vec > 1 ? static_cast<int>(cdiv(n, s.tpr)) : nv;
  s.threads = ckl::NORM_THREADS / s.tpr * s.tpr;
  return s;
}

// Forward (V: elements of 16 bytes; many: more rows than 8 an SM): 16 elements a
// thread, 32 in long rows; in many bf16 rows from 2560 to what fits beside gamma
// and beta, 32 as well.  us with 16 / 32 a thread: 16384 x 4096 52 / 48 (with the
// 8-bit copy 70 / 63), 8192 x 6144 45 / 41, 32768 x 2880 76 / 68 (RMS norm 64 /
// 68), 32768 x 2560 62 / 63, keeping 8 bits 86 / 98.
constexpr NormShape norm_fwd_shape(int64_t d, int V, bool vec, bool many) {
  if (!vec) return norm_shape(d, 1, 8, 16);
  if (V == 8 && many && d > 2560 && d <= 7168) return norm_shape(d, V, 4, 0);
  return norm_shape(d, V, 16 / V, 32 / V);
}

// Backward: bf16 rows of 32 elements a thread are all that 16 do not hold, and
// from 2560 on where there are rows enough, as more rows are then under way.  us
// with 16 / 32 a thread: 32768 x 2880 103 / 93, 8192 x 5120 59 / 49, 16384 x 4096
// 68.5 / 67.6, 32768 x 2560 83 / 90, 500 x 4096 9.6 / 11.0.  From 8 bits, which
// are converted twice then, 16384 x 4096 75 / 97.
constexpr NormShape norm_bwd_shape(int64_t d, int V, bool vec, bool q8, bool many) {
  if (!vec) return norm_shape(d, 1, 8, 16);
  const NormShape s = norm_shape(d, V, 16 / V, 0);
  if (V == 8 && d <= ckl::NORM_REGS_D && (s.nv == 0 || (!q8 && many && d > 2560)))
    return norm_shape(d, V, 4, 0);
  return s;
}

// Vectors a thread of the kernels that are compiled, and one launch of them.
template <int... NV>
struct NormCounts {
  static constexpr bool has(int nv) { return ((nv == NV) || ...); }
  template <typename F>
  static int launch(int nv, F&& go) {
    int rc = CKL_ERR_UNSUPPORTED;
    ((nv == NV && (rc = go(std::integral_constant<int, NV>()), true)) || ...);
    return rc;
  }
};
template <int V>
using NormFwdCounts = std::conditional_t<V == 8, NormCounts<1, 2, 4>, NormCounts<1, 2, 3, 4, 8>>;
template <int V>
using NormBwdCounts = std::conditional_t<V == 8, NormCounts<1, 2, 4>, NormCounts<1, 2, 3, 4>>;

// A kernel takes all of a thread's vectors but the last for granted, so a rule
// above that gave a width another count, or more than one vector past the row,
// would read and write behind rows.  Checked for every width that has a shape:
// moving a threshold to where it would (d = 1280 with four vectors wanted: three)
// does not compile.
template <typename Counts>
constexpr bool norm_shape_ok(const NormShape& s, int64_t n) {
  return s.nv == 0 || (Counts::has(s.nv) && s.tpr % 32 == 0 && s.tpr <= s.threads &&
                       s.threads <= ckl::NORM_THREADS && (s.nv - 1) * s.tpr <= n &&
                       s.nv * s.tpr >= n);
}
template <int V>
constexpr bool norm_fwd_shapes_ok(bool many) {
  for (int64_t n = 1; n <= ckl::NORM_REGS_D / V + 1; ++n)
    if (!norm_shape_ok<NormFwdCounts<V>>(norm_fwd_shape(n * V, V, true, many), n)) return false;
  return true;
}
template <int V>
constexpr bool norm_bwd_shapes_ok(bool q8, bool many) {
  for (int64_t n = 1; n <= ckl::NORM_REGS_D / V + 1; ++n)
    if (!norm_shape_ok<NormBwdCounts<V>>(norm_bwd_shape(n * V, V, true, q8, many), n)) return false;
  return true;
}
static_assert(norm_fwd_shapes_ok<8>(false) && norm_fwd_shapes_ok<8>(true), "bf16 forward");
static_assert(norm_fwd_shapes_ok<4>(false) && norm_fwd_shapes_ok<4>(true), "fp32 forward");
static_assert(norm_bwd_shapes_ok<8>(false, false) && norm_bwd_shapes_ok<8>(false, true) &&
                  norm_bwd_shapes_ok<8>(true, false) && norm_bwd_shapes_ok<8>(true, true),
              "bf16 backward");
static_assert(norm_bwd_shapes_ok<4>(false, false) && norm_bwd_shapes_ok<4>(false, true) &&
                  norm_bwd_shapes_ok<4>(true, false) && norm_bwd_shapes_ok<4>(true, true),
              "fp32 backward");
constexpr int64_t kPast = ckl::NORM_REGS_D + 8;
static_assert(norm_fwd_shape(kPast, 8, true, false).nv == 0 &&
                  norm_fwd_shape(kPast, 4, true, false).nv == 0 &&
                  norm_bwd_shape(kPast, 8, true, false, true).nv == 0 &&
                  norm_bwd_shape(kPast, 8, true, true, true).nv == 0 &&
                  norm_bwd_shape(kPast, 4, true, false, true).nv == 0 &&
                  norm_bwd_shape(ckl::NORM_REGS_D + 1, 1, false, false, true).nv == 0,
              "no width behind the checked ones has a shape");

// Of an SM, for the blocks' dynamic shared memory; also the most a block takes
// (with the kernels' static part, under 0.5 KB, within the 227 KB that it may).
constexpr size_t kNormSmem = 224 * 1024;

template <typename P>
int norm_launch(void (*k)(P), const P& p, dim3 grid, int threads, size_t smem, cudaStream_t st) {
  // 48 KB, the kernel's static part included, need no opting in.  The limit is
  // the kernel's, not this call's: every call sets the same one, so that none
  // lowers what another thread is about to launch with.
  if (smem > 40 * 1024 && !allow_smem(k, kNormSmem)) return failed();
  return launch(k, grid, threads, smem, st, nullptr, p);
}

template <typename TX, bool KEEP>
int norm_fwd_launch(const ckl::NormFwd& p0, bool vec, int sms, cudaStream_t st) {
  constexpr int V = ckl::VEC16<TX>;
  ckl::NormFwd p = p0;
  const NormShape s = norm_fwd_shape(p.d, V, vec, p.T > 8 * sms);
  p.tpr = s.tpr;
  if (s.nv == 0) {
    const unsigned rows = static_cast<unsigned>(std::min<int64_t>(p.T, sms * 4));
    return norm_launch(vec ? ckl::norm_fwd_long_kernel<TX, V> : ckl::norm_fwd_long_kernel<TX, 1>, p,
                       dim3(rows), ckl::NORM_THREADS, 0, st);
  }
  const dim3 one(static_cast<unsigned>(std::min<int64_t>(p.T, sms)));
  if (!vec)
    return norm_launch(s.nv == 8 ? ckl::norm_fwd_kernel<TX, 1, 8, false, KEEP>
                                 : ckl::norm_fwd_kernel<TX, 1, 16, false, KEEP>,
                       p, one, s.threads, 0, st);
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value, BYTES = ckl::NORM_FWD_BYTES<NV>;
    if constexpr (NV * V <= (V == 8 ? 32 : 16)) {
      // the parameters in shared memory where two blocks' fit and groups have
      // more than a row or two: bf16 16 elements a thread 16384 x 4096 51 us,
      // 8192 x 5120 37 us (55 and 46 with them in registers, one block an SM);
      // fp32 is within 5 % either way but for 8192 x 4096 (51 and 42)
      const size_t smem = static_cast<size_t>(s.threads) * BYTES * ckl::norm_fwd_stages(BYTES) +
                          static_cast<size_t>(s.tpr) * NV * V * 8;
      if (p.T > 2 * sms && smem <= kNormSmem / 2) {
        // 64 registers a thread, 1 KB of shared memory beside a block's own
        const int64_t fit = std::min<int64_t>(1024 / s.threads, kNormSmem / (smem + 1024));
        const dim3 all(static_cast<unsigned>(std::min<int64_t>(p.T, sms * std::max<int64_t>(fit, 2))));
        return norm_launch(ckl::norm_fwd_kernel<TX, V, NV, true, KEEP>, p, all, s.threads, smem,
                           st);
      }
    }
    return norm_launch(
        ckl::norm_fwd_kernel<TX, V, NV, false, KEEP>, p, one, s.threads,
        static_cast<size_t>(s.threads) * BYTES * ckl::norm_stages(BYTES), st);
  };
  return NormFwdCounts<V>::launch(s.nv, go);
}

// Returns the status; `parts` is how many sums the workspace then holds.
template <typename TX, bool Q8>
int norm_bwd_launch(const ckl::NormBwd& p0, bool vec, int sms, cudaStream_t st, int& parts) {
  constexpr int V = ckl::VEC16<TX>;
  ckl::NormBwd p = p0;
  const NormShape s = norm_bwd_shape(p.d, V, vec, Q8, p.T > 8 * sms);
  p.tpr = s.tpr;
  parts = static_cast<int>(std::min<int64_t>(p.T, std::min(sms, ckl::NORM_MAX_PARTS)));
  const dim3 grid(static_cast<unsigned>(parts));
  const size_t sums = static_cast<size_t>(p.d) * 8;  // a row group's, on the way to the first's
  if (s.nv != 0 && !vec)
    return norm_launch(s.nv == 8 ? ckl::norm_bwd_kernel<TX, 1, 8, Q8, false>
                                 : ckl::norm_bwd_kernel<TX, 1, 16, Q8, false>,
                       p, grid, s.threads, sums, st);
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    const size_t ring = static_cast<size_t>(s.threads) * ckl::NORM_BWD_BYTES<TX, NV, Q8> *
                        ckl::norm_bwd_stages<TX, V, NV, Q8>();
    const size_t params = static_cast<size_t>(s.tpr) * NV * V * 4;
    if (p.T > 2 * sms && ring + params <= kNormSmem)
      return norm_launch(ckl::norm_bwd_kernel<TX, V, NV, Q8, true>, p, grid, s.threads,
                         std::max(ring + params, sums), st);
    return norm_launch(ckl::norm_bwd_kernel<TX, V, NV, Q8, false>, p, grid, s.threads,
                       std::max(ring, sums), st);
  };
  if (s.nv != 0) return NormBwdCounts<V>::launch(s.nv, go);
  parts = static_cast<int>(ckl::norm_cols_parts(p.T));
  if (p.want_gamma || p.want_beta) {  // first: dx may take dy's place
    const dim3 cols(static_cast<unsigned>(cdiv(p.d, 32 * (vec ? V : 1))),
                    static_cast<unsigned>(parts));
    const int rc = norm_launch(
        vec ? ckl::norm_cols_kernel<TX, V, Q8> : ckl::norm_cols_kernel<TX, 1, Q8>, p, cols,
        32 * ckl::NORM_COL_WARPS, 0, st);
    if (rc != CKL_OK) return rc;
  }
  const unsigned rows = static_cast<unsigned>(std::min<int64_t>(p.T, sms * 4));
  return norm_launch(
      vec ? ckl::norm_bwd_long_kernel<TX, V, Q8> : ckl::norm_bwd_long_kernel<TX, 1, Q8>, p,
      dim3(rows), ckl::NORM_THREADS, 0, st);
}

template <int C, bool MANY>
int sample_launch(const ckl::SampleParams& p, int sms, cudaStream_t st) {
  auto* k = ckl::sample_kernel<C, MANY>;
  const size_t smem = MANY ? sizeof(ckl::SampleShared) : ckl::SM_ONE_BYTES;
  if (!allow_smem(k, smem)) return failed();
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = C;
  cluster.val.clusterDim.y = 1;
  cluster.val.clusterDim.z = 1;
  const int64_t rows = std::max(1, sms * ckl::sample_blocks(MANY) / C);  // at a time
  return launch(k, dim3(static_cast<unsigned>(std::min(p.T, rows) * C)), ckl::sample_threads(MANY),
                smem, st, C > 1 ? &cluster : nullptr, p);
}

template <int E>
int sample_short(const ckl::SampleParams& p, int sms, cudaStream_t st) {
  auto* k = ckl::sample_short_kernel<E>;
  const size_t smem = static_cast<size_t>(ckl::SM_SHORT_THREADS) * E * 12;
  if (!allow_smem(k, smem)) return failed();
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.T, static_cast<int64_t>(sms) * 8));
  return launch(k, dim3(grid), ckl::SM_SHORT_THREADS, smem, st, nullptr, p);
}

// Blocks a row: as many as leave every SM one; of long rows with one draw, as
// many as run at once (three an SM).  Clusters of 4 have to fit into groups of
// SMs and do so to about 7/8, those of 8 to about 2/3.  us with 1 / 2 / 4 / 8
// blocks, one draw: 128256 logits 8 rows 33 / 24 / 18 / 16, 16 rows 33 / 24 / 18 /
// 20, 64 rows 33 / 24 / 23 / 44, 74 rows 33 / 24 / 27 / 45, 148 rows 33 / 29 / 47 /
// 83, 222 rows 42 / 37 / 82 / 152, 296 rows 43 / 53; 201088 logits 96 rows 46 / 38 /
// 33 / 55; 32000 logits 32 rows 16 / 16 / 15 / 20, 96 rows 17 / 18 / 24 / 46.  64
// draws of 128256: 8 rows 49 / 38 / 32 / 30, 32 rows 49 / 39 / 33 / 43, 74 rows 50 /
// 39 / 69 / 138, 96 rows 50 / 52 / 77 / 145.
template <bool MANY>
int sample_rows(const ckl::SampleParams& p, int sms, cudaStream_t st) {
  const int64_t at_once = static_cast<int64_t>(sms) * (!MANY && p.V >= 65536 ? 3 : 1);
  if (p.T * 8 <= sms * 2 / 3) return sample_launch<8, MANY>(p, sms, st);
  if (p.T * 4 <= at_once * 7 / 8) return sample_launch<4, MANY>(p, sms, st);
  if (p.T * 2 <= at_once) return sample_launch<2, MANY>(p, sms, st);
  return sample_launch<1, MANY>(p, sms, st);
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
  return dtype == CKL_DTYPE_F32
             ? act8_pack_launch<float>(x, T, d, q, exponents, dev.sms, st)
             : act8_pack_launch<bf16>(x, T, d, q, exponents, dev.sms, st);
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
  return dtype == CKL_DTYPE_F32
             ? act8_unpack_launch<float>(q, exponents, T, d, x, dev.sms, st)
             : act8_unpack_launch<bf16>(q, exponents, T, d, x, dev.sms, st);
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
  const bool vec = d % static_cast<int64_t>(16 / eb) == 0 && aligned(x, 16) && aligned(y, 16) &&
                   aligned(gamma, 16) && aligned(beta, 16) && aligned(q, 8);
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
  p.param_f32 = param_dtype == CKL_DTYPE_F32;
  p.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == CKL_DTYPE_F32)
    return q ? norm_fwd_launch<float, true>(p, vec, dev.sms, st)
             : norm_fwd_launch<float, false>(p, vec, dev.sms, st);
  return q ? norm_fwd_launch<bf16, true>(p, vec, dev.sms, st)
           : norm_fwd_launch<bf16, false>(p, vec, dev.sms, st);
}

size_t ckl_norm_workspace_bytes(int64_t T, int64_t d) {
  if (!norm_sizes_ok(T, d)) return 0;
  const int64_t parts = d > ckl::NORM_REGS_D ? ckl::norm_cols_parts(T)
                                             : std::min<int64_t>(T, ckl::NORM_MAX_PARTS);
  return static_cast<size_t>(std::max<int64_t>(1, parts)) * 2 * d * 4;
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
  const bool vec = d % static_cast<int64_t>(16 / eb) == 0 && aligned(dy, 16) && aligned(x, 16) &&
                   aligned(dx, 16) && aligned(gamma, 16) && (!q8 || aligned(q, 8));
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
    p.param_f32 = param_dtype == CKL_DTYPE_F32;
    p.want_gamma = dgamma != nullptr;
    p.want_beta = dbeta != nullptr;
    const int rc =
        dtype == CKL_DTYPE_F32
            ? (q8 ? norm_bwd_launch<float, true>(p, vec, dev.sms, st, parts)
                  : norm_bwd_launch<float, false>(p, vec, dev.sms, st, parts))
            : (q8 ? norm_bwd_launch<bf16, true>(p, vec, dev.sms, st, parts)
                  : norm_bwd_launch<bf16, false>(p, vec, dev.sms, st, parts));
    if (rc != CKL_OK) return rc;
  }
  if (!grads) return CKL_OK;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  return launch(ckl::norm_reduce_kernel, dim3(static_cast<unsigned>(cdiv(d, ckl::NORM_RED_COLS)), 2),
                ckl::NORM_RED_COLS * ckl::NORM_RED_ROWS, 0, st, &early,
                static_cast<const float*>(workspace), parts, static_cast<int32_t>(d), dgamma, dbeta,
                accumulate);
}

int ckl_sample(const uint16_t* logits, int64_t ld, int64_t T, int64_t V, const float* u, int32_t N,
               double temperature, int32_t top_k, double top_p, double min_p,
               const float* temperature_rows, const int32_t* top_k_rows, const float* top_p_rows,
               const float* min_p_rows, int32_t* ids, float* logp, int32_t* device_status,
               void* stream) {
  if (T < 0 || V < 1 || ld < V || N < 1 || T > kLim / N) return CKL_ERR_INVALID_ARG;
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (V <= (N == 1 ? ckl::SM_SHORT_V : ckl::SM_SHORT_V_MANY)) {
    const int64_t per = cdiv(V, ckl::SM_SHORT_THREADS);
    return per == 1   ? sample_short<1>(p, dev.sms, st)
           : per == 2 ? sample_short<2>(p, dev.sms, st)
           : per <= 4 ? sample_short<4>(p, dev.sms, st)
           : per <= 8 ? sample_short<8>(p, dev.sms, st)
                      : sample_short<16>(p, dev.sms, st);
  }
  return N == 1 ? sample_rows<false>(p, dev.sms, st) : sample_rows<true>(p, dev.sms, st);
}

}  // extern "C"
