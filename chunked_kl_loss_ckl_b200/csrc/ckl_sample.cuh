// Sampling token ids from rows of bf16 logits, with temperature, top-k, top-p
// and min-p, from given uniform numbers.
//
// The tokens of a row are ordered by descending logit, equal logits by lowest
// id.  With w = exp((z - max) / temperature), each filter keeps a prefix of
// that order: top-k the first k; top-p the smallest prefix with at least p of
// the mass that top-k left; min-p the tokens with w >= min_p.  The kept tokens
// are the shortest of the three, S is their mass, and a number u draws the
// first token whose running mass passes u S.  Its log-prob is log(w / S).
//
// What makes this cheap and exact is that a bf16 logit has few values.  One
// pass over the row counts how often each value occurs (integer adds to
// shared memory: no order of the adds changes a result); everything else - the
// largest logit, the masses, the three prefixes, the draw - follows from the
// counts with one fp64 exponential per value that occurs, a few thousand
// instead of one per token, so all sums are in 64 bits and a draw next to the
// border of two tokens falls on the right one.  A draw gives a value and which
// of its occurrences; a second pass over the row (from L2) finds its id.
//
// The counters cover |z| in [2^-40, 256) and zero: 2 x 6144 + 1 bins in order.
// A row with other finite values takes them in eight windows of 8192 keys
// instead (sample_row_any: one block, eight passes over the row and one more for
// every chunk looked into; 128256 logits 1.2 ms with one draw, 9 ms with 64, 296
// such rows 1.3 and 11 ms), unless all of them are so far below the largest
// logit (2^-64 of its weight) that their mass, under 2^-40 of the row's, is
// never reached by a u of 24 bits.
//
// Bound by the adds to shared memory: 32 lanes' random bins meet 3.5 to a bank,
// and 32 logits cost an SM 5 cycles where HBM brings them in 2.7; a row of
// 128256 takes 20 thousand cycles of them, 15 to 20 thousand of fp64 steps that
// wait on each other (other blocks run meanwhile), and 10 thousand to find the
// drawn occurrence.  Few rows: a row is shared by a cluster of up to 8 blocks,
// which count their parts and add each other's counters over distributed shared
// memory; the one whose part has the drawn occurrence looks for it.  On a B200:
// 1 x 128256 16 us (fp64 steps and barriers), 96 x 201088 33 us, 4096 x 128256
// 533 us with one draw a row (2.0 TB/s), 1020 us with 64 (1.0 TB/s: the marks'
// pass and the searches take as long as the counting).
#pragma once

#include <cstddef>
#include <cstdint>

#include "ckl_bf16.cuh"
#include "ckl_ptx.cuh"

#define CKL_DEV_BAD_SAMPLE 16  // NaN or +inf logit, or a parameter or number out of range

namespace ckl {

// Threads of a block and blocks of an SM: by shared memory three blocks fit
// that draw once a row, two that draw many times.
__host__ __device__ constexpr int sample_threads(bool many) { return many ? 512 : 256; }
__host__ __device__ constexpr int sample_blocks(bool many) { return many ? 2 : 3; }
constexpr int SM_MAX_WARPS = 16;
constexpr int SM_UNROLL = 4;                    // 16-byte loads a thread has under way
constexpr int SM_TILE_UNROLL = 8;               // the same, where little is done to them
constexpr int SM_MAX_CLUSTER = 8;
constexpr uint32_t SM_LO = 0x2B80;              // bf16 bits of 2^-40
constexpr uint32_t SM_HI = 0x4380;              // bf16 bits of 256
constexpr int SM_HALF = SM_HI - SM_LO;          // bins of one sign
constexpr int SM_CB = 16;                       // bins of a chunk
constexpr int SM_NEG = SM_HALF + SM_CB;         // first negative bin (zero has a chunk of its own)
constexpr int SM_BINS = SM_NEG + SM_HALF;
constexpr int SM_CHUNKS = SM_BINS / SM_CB;
static_assert(SM_HALF % 128 == 0 && SM_LO % 128 == 0 && 128 % SM_CB == 0,
              "a chunk's bins are of one binade");
constexpr int SM_WIN = 8192;                    // keys of a window (rows of any values)
constexpr int SM_ANY_CB = 32;
constexpr int SM_ANY_CHUNKS = 65536 / SM_ANY_CB;
constexpr int SM_SEGS = 128;                    // parts of the row counted per draw
constexpr int SM_BATCH = 64;                    // draws found in one pass
static_assert(SM_BATCH <= sample_threads(true), "a thread a draw, for the marks");

struct SampleParams {
  const uint16_t* logits;
  int64_t ld;  // elements from a row to the next
  int64_t T;
  int32_t V, N;
  const float* u;  // [T, N]
  double temperature, top_p, min_p;
  int32_t top_k;
  const float* temperature_rows;  // null: the number above for every row
  const int32_t* top_k_rows;
  const float* top_p_rows;
  const float* min_p_rows;
  int32_t* ids;  // [T, N]
  float* logp;   // [T, N], may be null
  int32_t* status;
};

// A row's own parameters.
struct SampleRow {
  double inv_temp, top_p, min_p;
  int32_t top_k;
  bool greedy, ok;
};

struct alignas(16) SampleShared {
  // counters of the bins (slot order below), or of a window's keys; behind a
  // window's 8192 counters, the prefix masses of all 2048 chunks
  uint32_t hist[SM_BINS];
  double pw[SM_CHUNKS + 1];    // mass before each chunk
  double scan_w[SM_MAX_WARPS];
  double mass;                 // what the filters keep
  double draw_w;               // of the one draw
  SampleRow par;
  uint32_t pc[SM_CHUNKS + 1];  // tokens before each chunk
  uint32_t scan_c[SM_MAX_WARPS];
  uint32_t kept;
  uint32_t cb[SM_ANY_CB];  // one chunk's counters (rows of any values)
  uint32_t flags[SM_MAX_WARPS];
  uint32_t seen[SM_MAX_CLUSTER * SM_MAX_WARPS];  // each warp's largest key and flags
  uint32_t draw_bin[SM_BATCH], draw_rank[SM_BATCH];
  uint32_t found[SM_MAX_CLUSTER][SM_BATCH];  // how often each block has each drawn value
  union {
    uint32_t any_pc[SM_ANY_CHUNKS + 1];
    struct {                   // many draws; not there in launches for one
      uint32_t segs[SM_SEGS][SM_BATCH / 2];  // matches of 64 values in each part, 16 bits each
      uint32_t drawn[65536 / 32];            // a bit for each bf16 pattern that was drawn
    };
  };
};
// Bytes of a launch for one draw a row.
constexpr size_t SM_ONE_BYTES =
    offsetof(SampleShared, any_pc) + sizeof(uint32_t) * (SM_ANY_CHUNKS + 1);
static_assert(SM_WIN * 4 + (SM_ANY_CHUNKS + 1) * 8 <= SM_BINS * 4, "prefix masses behind a window");

__device__ __forceinline__ int sample_nt() { return static_cast<int>(blockDim.x); }
__device__ __forceinline__ int sample_nw() { return static_cast<int>(blockDim.x) / 32; }

enum : uint32_t { SF_BAD = 1, SF_LOW = 2, SF_ANY = 4 };

// A row's elements: up to 7 before the first 16-byte boundary (the first
// block's), whole vectors of eight, up to 7 behind the last (the last block's).
// A block has vectors [0, nvec) of `v`.
struct SampleSpan {
  const uint16_t* z;
  const uint4* v;
  int head, first, nvec, tail, tail_at;
  __device__ __forceinline__ SampleSpan(const uint16_t* row, int V, int blocks, int rank) : z(row) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
    head = min(V, static_cast<int>(((16u - off) & 15u) / 2u));
    const int all = (V - head) / 8;
    const int per = ((all + blocks - 1) / blocks + 31) / 32 * 32;
    const int v0 = min(all, rank * per);
    nvec = min(all, v0 + per) - v0;
    first = head + 8 * v0;  // id of the first vector's first element
    v = reinterpret_cast<const uint4*>(row + head) + v0;
    tail_at = head + 8 * all;
    tail = rank == blocks - 1 ? V - tail_at : 0;
    if (rank != 0) head = 0;
  }
};

// The counter of a value of the covered range: the positive values ascending,
// zero, the negative ones descending (bits apart from the sign, plus SM_NEG
// when it is set).
__device__ __forceinline__ uint32_t sample_slot(uint32_t x) {
  return (x & 0x7FFFu) + (x >> 15) * SM_NEG - SM_LO;
}
// Bin b (descending values) -> its counter, and its value.
__device__ __forceinline__ int sample_bin_slot(int b) {
  return b < SM_HALF ? SM_HALF - 1 - b : b;
}
__device__ __forceinline__ uint32_t sample_bin_bits(int b) {
  if (b < SM_HALF) return SM_LO + (SM_HALF - 1 - b);
  return b < SM_NEG ? 0u : 0x8000u + SM_LO + (b - SM_NEG);
}
// The bin whose counter a covered value or zero has.
__device__ __forceinline__ int sample_slot_of(uint32_t x) {
  return (x & 0x7FFFu) == 0u ? SM_HALF : static_cast<int>(sample_slot(x));
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Non-zero where one of the word's two values is outside the covered range
// (zero is outside too): |x| + (0x8000 - bound) carries into bit 15 from the
// bound on.
__device__ __forceinline__ uint32_t sample_outside(uint32_t w) {
  const uint32_t a = w & 0x7FFF7FFFu;
  return ((a + (0x8000u - SM_HI) * 0x10001u) | ~(a + (0x8000u - SM_LO) * 0x10001u)) & 0x80008000u;
}

// Counts one value that may lie anywhere.
__device__ __forceinline__ void sample_count1(uint32_t* hist, uint32_t x, uint32_t& flags) {
  const uint32_t a = x & 0x7FFFu;
  if (a >= SM_LO && a < SM_HI) {
    atomicAdd(&hist[sample_slot(x)], 1u);
  } else if (a == 0u) {
    atomicAdd(&hist[SM_HALF], 1u);
  } else if (a >= 0x7F80u) {
    if (x != 0xFF80u) flags |= SF_BAD;  // NaN or +inf; -inf is never drawn
  } else {
    flags |= (x & 0x8000u) && a >= SM_HI ? SF_LOW : SF_ANY;
  }
}

// Counts eight values, and keeps the largest of those seen.  Values outside
// the covered range are skipped; unless they are -inf (a mask's), they are
// looked at one by one.
__device__ __forceinline__ void sample_count8(uint32_t* hist, const uint4& v, uint32_t& m2,
                                              uint32_t& flags) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint32_t out[4] = {sample_outside(v.x), sample_outside(v.y), sample_outside(v.z),
                           sample_outside(v.w)};
  m2 = bf16x2_max(m2, bf16x2_max(bf16x2_max(v.x, v.y), bf16x2_max(v.z, v.w)));
  if ((out[0] | out[1] | out[2] | out[3]) == 0u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      atomicAdd(&hist[sample_slot(w[j] & 0xFFFFu)], 1u);
      atomicAdd(&hist[sample_slot(w[j] >> 16)], 1u);
    }
    return;
  }
  uint32_t others = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!(out[j] & 0x8000u)) atomicAdd(&hist[sample_slot(w[j] & 0xFFFFu)], 1u);
    if (!(out[j] & 0x80000000u)) atomicAdd(&hist[sample_slot(w[j] >> 16)], 1u);
    // the halves that are outside and not -inf
    const uint32_t d = w[j] ^ 0xFF80FF80u;
    others |= out[j] & (((d & 0x7FFF7FFFu) + 0x7FFF7FFFu) | d);
  }
  if (others) {
    for (int j = 0; j < 4; ++j) {
      if (out[j] & 0x8000u) sample_count1(hist, w[j] & 0xFFFFu, flags);
      if (out[j] & 0x80000000u) sample_count1(hist, w[j] >> 16, flags);
    }
  }
}

// The passes over a row are functions of their own, with few arguments, so
// that what the rest of the kernel holds does not push their loads in flight
// out of registers.
//
// Counts the vectors' values; returns the thread's packed maximum and, in the
// high half, its flags.
// AHEAD: the next vectors are loaded before these are counted (in the blocks of
// 256 threads, which have the registers; 4096 x 128256: 567 us without, 552 us
// so).
template <bool AHEAD>
__device__ __noinline__ uint64_t sample_count_pass(uint32_t* hist, const uint4* __restrict__ z,
                                                   int nvec) {
  uint32_t flags = 0, m2 = 0xFF80FF80u;
  const int step = SM_UNROLL * sample_nt();
  int i = threadIdx.x;
  if constexpr (AHEAD) {
    uint4 v[SM_UNROLL], next[SM_UNROLL];
    auto load = [&](uint4 (&to)[SM_UNROLL], int at) {
#pragma unroll
      for (int k = 0; k < SM_UNROLL; ++k)  // -inf is not counted
        to[k] = at + k * sample_nt() < nvec
                    ? z[at + k * sample_nt()]
                    : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
    };
    load(v, i);
    for (; i < nvec; i += step) {
      load(next, i + step);
#pragma unroll
      for (int k = 0; k < SM_UNROLL; ++k) sample_count8(hist, v[k], m2, flags);
#pragma unroll
      for (int k = 0; k < SM_UNROLL; ++k) v[k] = next[k];
    }
  } else {
    for (; i + (SM_UNROLL - 1) * sample_nt() < nvec; i += step) {
      uint4 v[SM_UNROLL];
#pragma unroll
      for (int k = 0; k < SM_UNROLL; ++k) v[k] = z[i + k * sample_nt()];
#pragma unroll
      for (int k = 0; k < SM_UNROLL; ++k) sample_count8(hist, v[k], m2, flags);
    }
    for (; i < nvec; i += sample_nt()) sample_count8(hist, z[i], m2, flags);
  }
  return m2 | (static_cast<uint64_t>(flags) << 32);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the lanes up to and with this one.
template <int W = 32, typename T>
__device__ __forceinline__ T warp_scan(T v) {
  const int lane = threadIdx.x % W;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o, W);
    if (lane >= o) v += u;
  }
  return v;
}

__device__ __forceinline__ double sample_weight(float v, float m, const SampleRow& r) {
  return exp((static_cast<double>(v) - static_cast<double>(m)) * r.inv_temp);
}

// Distributed shared memory of a cluster of C blocks: the address of a variable
// of this block in another one, and a barrier of all threads of the cluster
// (of the block where there is one).
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  return mapa_shared(smem_u32(p), rank);
}
__device__ __forceinline__ uint32_t peer_load(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 peer_load4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void peer_store(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t a, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}
template <int C>
__device__ __forceinline__ void arrive_all() {
  if constexpr (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
template <int C>
__device__ __forceinline__ void wait_all() {
  if constexpr (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int C>
__device__ __forceinline__ void sync_all() {
  if constexpr (C == 1) __syncthreads();
  arrive_all<C>();
  wait_all<C>();
}

// The counts of a row, read chunk by chunk: the bins of a row of covered
// values, in the shared memory of its C blocks.
template <int C>
struct SampleBins {
  SampleShared& sm;
  static constexpr int CHUNKS = SM_CHUNKS, BINS = SM_BINS, CB = SM_CB;
  __device__ __forceinline__ const double* pw() const { return sm.pw; }
  __device__ __forceinline__ const uint32_t* pc() const { return sm.pc; }
  // of bin lane % CB of the chunk
  __device__ __forceinline__ uint32_t count(int chunk) const {
    return count_of(chunk * CB + threadIdx.x % CB);
  }
  __device__ __forceinline__ uint32_t count_of(int b) const {
    const uint32_t* at = &sm.hist[sample_bin_slot(b)];
    if constexpr (C == 1) return *at;
    uint32_t n = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) n += peer_load(peer(at, r));
    return n;
  }
  __device__ __forceinline__ float value(int b) const { return bf16_value(sample_bin_bits(b)); }
};

// The same of a row of any values: 65536 keys, a chunk's counts taken by a
// pass of the whole block over the row.
struct SampleKeys {
  SampleShared& sm;
  const uint16_t* z;
  int V;
  // bins up to that of -inf; behind it come the keys of NaNs
  static constexpr int CHUNKS = SM_ANY_CHUNKS, BINS = 0xFF81, CB = SM_ANY_CB;
  __device__ __forceinline__ double* pw() const {
    return reinterpret_cast<double*>(sm.hist + SM_WIN);
  }
  __device__ __forceinline__ uint32_t* pc() const { return sm.any_pc; }
  __device__ __noinline__ uint32_t count(int chunk) const {
    __syncthreads();
    if (threadIdx.x < CB) sm.cb[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < V; i += sample_nt()) {
      const uint32_t b = 0xFFFFu - bf16_key(z[i]);
      if (static_cast<int>(b / CB) == chunk && z[i] != 0xFF80u) atomicAdd(&sm.cb[b % CB], 1u);
    }
    __syncthreads();
    return sm.cb[threadIdx.x % CB];
  }
  __device__ __forceinline__ float value(int b) const {
    return key_value(0xFFFFu - static_cast<uint32_t>(b));
  }
};

// A place in the order of the row's tokens: a bin, which of its occurrences,
// how many tokens and how much mass come before that occurrence.
struct SamplePlace {
  int bin;
  uint32_t in_bin;
  uint32_t rank;
  double mass;  // of the tokens before the bin, plus in_bin of the bin's
  double w;     // of one token of the bin
};

// The last of entries 0 .. n - 1 with pred; pred holds for the first one and
// changes once.  32 entries are tried at a time.
template <typename F>
__device__ __forceinline__ int sample_chunk(int n, F&& pred) {
  int lo = 0, size = n;  // the answer is in [lo, lo + size)
  while (size > 1) {
    const int step = (size + 31) / 32;
    const int i = lo + static_cast<int>(threadIdx.x & 31) * step;
    const bool yes = i < lo + size && pred(i);
    const int k = __popc(__ballot_sync(0xffffffffu, yes)) - 1;  // lane 0's holds
    size = min(step, lo + size - (lo + k * step));
    lo += k * step;
  }
  return lo;
}

// The token at a rank.
template <typename S>
__device__ __forceinline__ SamplePlace sample_at_rank(const S& s, float m, const SampleRow& r,
                                                      uint32_t rank) {
  constexpr int CB = S::CB;
  const int c = sample_chunk(S::CHUNKS, [&](int i) { return s.pc()[i] <= rank; });
  const uint32_t n = s.count(c);
  const double w = n ? sample_weight(s.value(c * CB + threadIdx.x % CB), m, r) : 0.0;
  const uint32_t upto = warp_scan<CB>(n) + s.pc()[c];
  const double mass = warp_scan<CB>(n * w) - n * w + s.pw()[c];
  const uint32_t hit = __ballot_sync(0xffffffffu, upto > rank);
  const int l = hit ? __ffs(hit) - 1 : CB - 1;
  SamplePlace p;
  p.bin = c * CB + l;
  const uint32_t before = __shfl_sync(0xffffffffu, upto - n, l);
  p.in_bin = rank - before;
  p.rank = rank;
  p.w = __shfl_sync(0xffffffffu, w, l);
  p.mass = __shfl_sync(0xffffffffu, mass, l) + p.in_bin * p.w;
  return p;
}

// The first token whose running mass is > target (STRICT) or >= target.
template <bool STRICT, typename S>
__device__ __forceinline__ SamplePlace sample_at_mass(const S& s, float m, const SampleRow& r,
                                                      double target) {
  constexpr int CB = S::CB;
  auto past = [&](double x) { return STRICT ? x > target : x >= target; };
  const int c = sample_chunk(S::CHUNKS, [&](int i) { return i == 0 || !past(s.pw()[i]); });
  const uint32_t n = s.count(c);
  const double w = n ? sample_weight(s.value(c * CB + threadIdx.x % CB), m, r) : 0.0;
  const uint32_t rank0 = warp_scan<CB>(n) - n + s.pc()[c];
  const double upto = warp_scan<CB>(n * w) + s.pw()[c];
  constexpr uint32_t LANES = CB == 32 ? 0xffffffffu : (1u << CB) - 1u;  // lanes of one copy
  const uint32_t some = __ballot_sync(0xffffffffu, n > 0) & LANES;
  const uint32_t hit = __ballot_sync(0xffffffffu, n > 0 && past(upto)) & LANES;
  // sums taken in another order may differ in the last bit: then the chunk's last
  const int l = hit ? __ffs(hit) - 1 : (some ? 31 - __clz(some) : 0);
  const uint32_t nl = __shfl_sync(0xffffffffu, n, l);
  SamplePlace p;
  p.bin = c * CB + l;
  p.w = __shfl_sync(0xffffffffu, w, l);
  const double before = __shfl_sync(0xffffffffu, upto - n * w, l);
  const double x = (target - before) / p.w;  // tokens of the bin before the target
  double j = STRICT ? floor(x) : ceil(x) - 1.0;
  j = fmin(fmax(j, 0.0), nl ? nl - 1.0 : 0.0);
  p.in_bin = static_cast<uint32_t>(j);
  p.rank = __shfl_sync(0xffffffffu, rank0, l) + p.in_bin;
  p.mass = before + j * p.w;
  return p;
}

// How many tokens have w >= min_p: the bins whose value does, by bisection
// (their order is the weights'), then the tokens in them.
template <typename S>
__device__ __forceinline__ uint32_t sample_min_p(const S& s, float m, const SampleRow& r) {
  int lo = 0, hi = S::BINS;  // bins below lo have it, from hi on do not
  const int lane = threadIdx.x & 31;
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + lane * step;
    // not (w < min_p): the keys before +inf's are NaNs'
    const bool has = b < hi && !(sample_weight(s.value(b), m, r) < r.min_p);
    const uint32_t bits = __ballot_sync(0xffffffffu, has);
    const int k = __popc(bits);  // lanes 0 .. k - 1 have it
    if (k == 0) break;
    const int last = lo + (k - 1) * step;
    hi = min(hi, last + step);
    lo = last + 1;
  }
  if (lo >= S::CHUNKS * S::CB) return s.pc()[S::CHUNKS];
  const uint32_t n = s.count(lo / S::CB);
  const uint32_t in = __reduce_add_sync(0xffffffffu, lane < lo % S::CB ? n : 0u);
  return s.pc()[lo / S::CB] + in;
}

// How many tokens the filters keep and their mass.
template <typename S>
__device__ __noinline__ uint32_t sample_kept(const S& s, float m, const SampleRow& r,
                                                double& mass) {
  uint32_t L = s.pc()[S::CHUNKS];
  mass = s.pw()[S::CHUNKS];
  uint32_t cut = r.greedy ? 1u : r.top_k > 0 ? static_cast<uint32_t>(r.top_k) : L;
  if (cut < L) {
    L = cut;
    const SamplePlace p = sample_at_rank(s, m, r, L - 1);
    mass = p.mass + p.w;
  }
  if (r.greedy) return L;
  cut = L;
  if (r.min_p > 0.0) cut = max(1u, sample_min_p(s, m, r));
  if (r.top_p < 1.0) {
    const SamplePlace p = sample_at_mass<false>(s, m, r, r.top_p * mass);
    if (p.rank < L && p.rank < cut) {
      mass = p.mass + p.w;
      return p.rank + 1;
    }
  }
  if (cut < L) {
    L = cut;
    const SamplePlace p = sample_at_rank(s, m, r, L - 1);
    mass = p.mass + p.w;
  }
  return L;
}

// One draw among the first L tokens.
template <typename S>
__device__ __forceinline__ SamplePlace sample_draw(const S& s, float m, const SampleRow& r,
                                                   uint32_t L, double mass, float u) {
  const SamplePlace p = sample_at_mass<true>(s, m, r, static_cast<double>(u) * mass);
  // rounding may leave the kept tokens, or a chunk's
  return p.rank < L && p.w > 0.0 ? p : sample_at_rank(s, m, r, min(p.rank, L - 1));
}

// A draw by eight lanes, among the first L tokens: the chunk by bisection, then
// two bins a lane (SampleBins only; the same result in all eight).
template <typename S>
__device__ __forceinline__ SamplePlace sample_draw8(const S& s, float m, const SampleRow& r,
                                                    uint32_t L, double mass, float u) {
  static_assert(S::CB == 16, "two bins a lane");
  const double target = static_cast<double>(u) * mass;
  int c = 0, hi = S::CHUNKS;  // pw[c] <= target
  while (hi - c > 1) {
    const int mid = (c + hi) / 2;
    if (s.pw()[mid] <= target) c = mid;
    else hi = mid;
  }
  const int lane = threadIdx.x & 31, b = c * S::CB + 2 * (lane & 7);
  const uint32_t n0 = s.count_of(b), n1 = s.count_of(b + 1);
  const double w0 = n0 ? sample_weight(s.value(b), m, r) : 0.0;
  const double w1 = n1 ? sample_weight(s.value(b + 1), m, r) : 0.0;
  const double x0 = n0 * w0, x = x0 + n1 * w1;
  const double before = warp_scan<8>(x) - x + s.pw()[c];
  const uint32_t rank0 = warp_scan<8>(n0 + n1) - (n0 + n1) + s.pc()[c];
  const uint32_t mine = 0xFFu << (lane & 24);  // the draw's lanes
  const uint32_t some = __ballot_sync(0xffffffffu, n0 + n1 > 0) & mine;
  const uint32_t hit = __ballot_sync(0xffffffffu, n0 + n1 > 0 && before + x > target) & mine;
  // rounding may leave the target behind the chunk's last token
  const int l = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : lane & 24;
  const bool second = n1 && (n0 == 0 || !(before + x0 > target));
  SamplePlace p;
  p.bin = __shfl_sync(0xffffffffu, second ? b + 1 : b, l);
  p.w = __shfl_sync(0xffffffffu, second ? w1 : w0, l);
  p.mass = __shfl_sync(0xffffffffu, second ? before + x0 : before, l);
  p.rank = __shfl_sync(0xffffffffu, second ? rank0 + n0 : rank0, l);
  const uint32_t n = __shfl_sync(0xffffffffu, second ? n1 : n0, l);
  double j = floor((target - p.mass) / p.w);
  j = fmin(fmax(j, 0.0), n ? n - 1.0 : 0.0);
  if (p.rank + j >= L) j = fmax(0.0, static_cast<double>(L) - 1.0 - p.rank);  // rounding
  p.in_bin = static_cast<uint32_t>(j);
  return p;
}

__device__ __forceinline__ bool sample_u_ok(float u) { return u >= 0.f && u < 1.f; }

// Turns the chunks' counts and masses into those before each chunk (the block).
__device__ __forceinline__ void sample_prefix(SampleShared& sm, uint32_t* pc, double* pw, int n) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (n + sample_nt() - 1) / sample_nt();
  const int b = min(n, static_cast<int>(threadIdx.x) * per), e = min(n, b + per);
  uint32_t c = 0;
  double w = 0.0;
  for (int i = b; i < e; ++i) {
    c += pc[i];
    w += pw[i];
  }
  uint32_t c0 = warp_scan(c);
  double w0 = warp_scan(w);
  if (lane == 31) {
    sm.scan_c[warp] = c0;
    sm.scan_w[warp] = w0;
  }
  __syncthreads();
  // every warp scans the warps' sums for itself
  const uint32_t ca = lane < sample_nw() ? sm.scan_c[lane] : 0u;
  const double wa = lane < sample_nw() ? sm.scan_w[lane] : 0.0;
  const uint32_t cu = warp_scan(ca);
  const double wu = warp_scan(wa);
  c0 += __shfl_sync(0xffffffffu, cu - ca, warp) - c;
  w0 = __shfl_sync(0xffffffffu, wu - wa, warp) + (w0 - w);
  for (int i = b; i < e; ++i) {
    const uint32_t ci = pc[i];
    const double wi = pw[i];
    pc[i] = c0;
    pw[i] = w0;
    c0 += ci;
    w0 += wi;
  }
  if (threadIdx.x == sample_nt() - 1) {  // lane 31: the sum over all warps
    pc[n] = cu;
    pw[n] = wu;
  }
  __syncthreads();
}

// A value to look for among packed bf16 pairs (zero: of either sign).
struct SampleMatch {
  uint32_t pat, msk;
  __device__ __forceinline__ explicit SampleMatch(uint32_t bits)
      : pat(bits * 0x10001u), msk((bits & 0x7FFFu) ? 0xFFFFFFFFu : 0x7FFF7FFFu) {
    pat &= msk;
  }
  // bit 15 and bit 31 set where the half is not the value
  __device__ __forceinline__ uint32_t differs(uint32_t w) const {
    const uint32_t x = (w & msk) ^ pat;
    return (((x & 0x7FFF7FFFu) + 0x7FFF7FFFu) | x) & 0x80008000u;
  }
  // a bit for each of the eight values that is it not: value 2 j in bit
  // 15 - j, value 2 j + 1 in bit 31 - j
  __device__ __forceinline__ uint32_t differs8(const uint4& v) const {
    return differs(v.x) | (differs(v.y) >> 1) | (differs(v.z) >> 2) | (differs(v.w) >> 3);
  }
  __device__ __forceinline__ bool is(uint32_t x) const { return ((x ^ pat) & msk & 0xFFFFu) == 0; }
};
constexpr uint32_t SM_EIGHT = 0xF000F000u;

// Id of occurrence `rank` (from 0) of a value among vectors [v0, v1) of the
// row, by one warp, four loads under way.  Returns -1 if it is not there.
__device__ __forceinline__ int sample_scan(const SampleSpan& sp, const SampleMatch& mt, int v0,
                                           int v1, uint32_t rank) {
  const int lane = threadIdx.x & 31;
  for (int b = v0; b < v1; b += 32 * SM_UNROLL) {
    uint4 v[SM_UNROLL];
    uint32_t no[SM_UNROLL];
#pragma unroll
    for (int k = 0; k < SM_UNROLL; ++k)
      if (b + k * 32 + lane < v1) v[k] = sp.v[b + k * 32 + lane];
#pragma unroll
    for (int k = 0; k < SM_UNROLL; ++k)
      no[k] = b + k * 32 + lane < v1 ? mt.differs8(v[k]) : SM_EIGHT;
#pragma unroll
    for (int k = 0; k < SM_UNROLL; ++k) {
      const uint32_t n = 8u - __popc(no[k]);
      const uint32_t all = __reduce_add_sync(0xffffffffu, n);
      if (rank >= all) {
        rank -= all;
        continue;
      }
      const uint32_t upto = warp_scan(n);
      const int l = __ffs(__ballot_sync(0xffffffffu, upto > rank)) - 1;
      int id = 0;
      if (lane == l) {
        uint32_t left = rank - (upto - n);
        for (int j = 0; j < 8; ++j) {
          const bool is = !((no[k] >> ((j & 1) ? 31 - j / 2 : 15 - j / 2)) & 1u);
          if (is && left-- == 0) {
            id = sp.first + 8 * (b + k * 32 + lane) + j;
            break;
          }
        }
      }
      return __shfl_sync(0xffffffffu, id, l);
    }
  }
  return -1;
}

// The same among up to 7 elements before or behind the vectors; rank is
// lowered by the ones found.
__device__ __forceinline__ int sample_scan_few(const SampleSpan& sp, const SampleMatch& mt, int at,
                                               int n, uint32_t& rank) {
  const int lane = threadIdx.x & 31;
  const bool is = lane < n && mt.is(sp.z[at + lane]);
  const uint32_t bits = __ballot_sync(0xffffffffu, is);
  const uint32_t all = __popc(bits);
  if (rank >= all) {
    rank -= all;
    return -1;
  }
  const bool me = is && __popc(bits & ((1u << lane) - 1u)) == static_cast<int>(rank);
  return at + __ffs(__ballot_sync(0xffffffffu, me)) - 1;
}

// Writes the id of occurrence `rank` of a value among the vectors, the first of
// which starts at id `first`; the block goes through them in order, a round of
// eight tiles of 32 vectors a warp at a time, and stops where it is found.
// Returns 0xFFFFFFFF, or what is left of the rank if the occurrence is not there.
__device__ __noinline__ uint32_t sample_find_pass(SampleShared& sm, const uint4* __restrict__ z,
                                                  int nvec, int first, uint32_t bits,
                                                  uint32_t rank, int32_t* id_out) {
  const SampleMatch mt(bits);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int U = SM_TILE_UNROLL;
  int turn = 0;  // two buffers, so that one barrier a round is enough
  for (int base = 0; base < nvec; base += 32 * U * sample_nw(), turn ^= 1) {
    const int i0 = base + warp * 32 * U + lane;
    uint32_t no[U], n = 0;
    {
      uint4 v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = i0 + 32 * k < nvec ? z[i0 + 32 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        no[k] = i0 + 32 * k < nvec ? mt.differs8(v[k]) : SM_EIGHT;
        n += 8u - __popc(no[k]);
      }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    uint32_t* sums = turn ? sm.flags : sm.scan_c;
    if (lane == 0) sums[warp] = n;
    __syncthreads();
    const uint32_t mine = lane < sample_nw() ? sums[lane] : 0u;
    const uint32_t upto = warp_scan(mine);
    const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
    if (rank >= all) {
      rank -= all;
      continue;
    }
    const int w = __ffs(__ballot_sync(0xffffffffu, upto > rank)) - 1;
    rank -= __shfl_sync(0xffffffffu, upto - mine, w);
    if (warp != w) return 0xFFFFFFFFu;
    bool done = false;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (done) continue;
      const uint32_t here = 8u - __popc(no[k]);
      const uint32_t tile = __reduce_add_sync(0xffffffffu, here);
      if (rank >= tile) {
        rank -= tile;
        continue;
      }
      done = true;
      const uint32_t before = warp_scan(here) - here;
      if (rank >= before && rank < before + here) {  // one lane
        uint32_t left = rank - before;
        for (int j = 0; j < 8; ++j) {
          const bool is = !((no[k] >> ((j & 1) ? 31 - j / 2 : 15 - j / 2)) & 1u);
          if (is && left-- == 0) {
            *id_out = first + 8 * (i0 + 32 * k) + j;
            break;
          }
        }
      }
    }
    return 0xFFFFFFFFu;
  }
  return rank;
}

// Writes the id of one occurrence of a bin's value.  In a cluster the blocks'
// counters say which of them has it, and that one looks for it.
template <int C>
__device__ __forceinline__ void sample_find(SampleShared& sm, const SampleSpan& sp, uint32_t rank0,
                                            int bin, uint32_t rank, int32_t* id_out) {
  const uint32_t bits = sample_bin_bits(bin);
  const SampleMatch mt(bits);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (C > 1) {
    const uint32_t n = lane < C ? peer_load(peer(&sm.hist[sample_bin_slot(bin)], lane)) : 0u;
    const uint32_t upto = warp_scan(n);
    const uint32_t before = __shfl_sync(0xffffffffu, upto - n, rank0);
    if (rank < before || rank - before >= __shfl_sync(0xffffffffu, n, rank0)) return;
    rank -= before;
  }
  const int few = sample_scan_few(sp, mt, 0, sp.head, rank);
  if (few >= 0) {
    if (threadIdx.x == 0) *id_out = few;
    return;
  }
  rank = sample_find_pass(sm, sp.v, sp.nvec, sp.first, bits, rank, id_out);
  if (rank == 0xFFFFFFFFu || warp != 0) return;
  const int id = sample_scan_few(sp, mt, sp.tail_at, sp.tail, rank);
  if (lane == 0) *id_out = id;
}

// Draws of a row, for loops over them in steps: N may be 2^31 - 1, and an int
// would pass its end with the last step.
__device__ __forceinline__ uint32_t sample_draws(const SampleParams& p) {
  return static_cast<uint32_t>(p.N);
}

__device__ __forceinline__ void sample_put(const SampleParams& p, int64_t row, int n, int id,
                                           float logp) {
  p.ids[row * p.N + n] = id;
  if (p.logp) p.logp[row * p.N + n] = logp;
}

__device__ __forceinline__ void sample_bad(const SampleParams& p) {
  if (p.status) atomicOr(p.status, CKL_DEV_BAD_SAMPLE);
}

// Bits of those of eight values that were drawn (value j: bit j).  Most were
// not: a bit for each bf16 pattern says so, which 32 lanes read with few bank
// conflicts (32 neighbouring values share a word).
__device__ __forceinline__ uint32_t sample_marked8(const uint32_t* drawn, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t hits = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = drawn[(w[j] >> 5) & 0x7FFu], hi = drawn[w[j] >> 21];
    hits |= ((lo >> (w[j] & 31u)) & 1u) << (2 * j);
    hits |= ((hi >> ((w[j] >> 16) & 31u)) & 1u) << (2 * j + 1);
  }
  return hits;
}

// Counts the drawn values in each part (2^shift vectors) of the row.  The lanes
// go through their hits of SM_UNROLL vectors together: the more elements that
// is, the nearer the busiest lane is to the mean.
__device__ __noinline__ void sample_marked_pass(SampleShared& sm, const uint4* __restrict__ z,
                                                int nvec, int shift) {
  static_assert(SM_UNROLL == 4, "32 values, a bit each");
  for (int i = threadIdx.x; i < nvec; i += SM_UNROLL * sample_nt()) {
    uint32_t hits = 0;
    {
      uint4 v[SM_UNROLL];
#pragma unroll
      for (int k = 0; k < SM_UNROLL; ++k)
        v[k] = z[i + k * sample_nt() < nvec ? i + k * sample_nt() : i];
#pragma unroll
      for (int k = 0; k < SM_UNROLL; ++k)
        if (i + k * sample_nt() < nvec) hits |= sample_marked8(sm.drawn, v[k]) << (8 * k);
    }
    while (hits) {
      const int j = __ffs(hits) - 1;
      hits &= hits - 1u;
      const int at = i + (j >> 3) * sample_nt();
      const uint32_t x = reinterpret_cast<const uint16_t*>(z)[8 * at + (j & 7)];
      const uint32_t col = sm.hist[sample_slot_of(x)] & (SM_BATCH - 1u);
      atomicAdd(&sm.segs[at >> shift][col >> 1], (col & 1u) ? 0x10000u : 1u);
    }
  }
}

// A row whose finite values are not all covered: the key space in eight
// windows, one pass over the row each, and a pass for every chunk looked into.
__device__ __noinline__ void sample_row_any(SampleShared& sm, const SampleParams& p, int64_t row) {
  const SampleRow& r = sm.par;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint16_t* z = p.logits + row * p.ld;
  SampleKeys s{sm, z, p.V};
  float m = 0.f;
  bool have = false;
  for (int win = 0; win < 65536 / SM_WIN; ++win) {
    __syncthreads();
    for (int i = tid; i < SM_WIN; i += sample_nt()) sm.hist[i] = 0;
    if (tid < sample_nw()) sm.flags[tid] = 0xFFFFFFFFu;
    __syncthreads();
    uint32_t top = 0xFFFFFFFFu;  // the first bin of the window that occurs
    for (int i = tid; i < p.V; i += sample_nt()) {
      const uint32_t x = z[i], b = 0xFFFFu - bf16_key(x);
      if (static_cast<int>(b / SM_WIN) == win && x != 0xFF80u) {
        atomicAdd(&sm.hist[b % SM_WIN], 1u);
        top = min(top, b);
      }
    }
    top = __reduce_min_sync(0xffffffffu, top);
    if (lane == 0) sm.flags[warp] = top;
    __syncthreads();
    for (int w = 0; w < sample_nw(); ++w) top = min(top, sm.flags[w]);
    if (!have && top != 0xFFFFFFFFu) {
      m = s.value(static_cast<int>(top));
      have = true;
    }
    for (int c = warp; c < SM_WIN / 32; c += sample_nw()) {
      const uint32_t n = sm.hist[c * 32 + lane];
      const int b = win * SM_WIN + c * 32 + lane;
      const double w = warp_sum(n ? n * sample_weight(s.value(b), m, r) : 0.0);
      const uint32_t cnt = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) {
        s.pc()[win * (SM_WIN / 32) + c] = cnt;
        s.pw()[win * (SM_WIN / 32) + c] = w;
      }
    }
  }
  __syncthreads();
  sample_prefix(sm, s.pc(), s.pw(), SM_ANY_CHUNKS);
  double mass;
  const uint32_t L = sample_kept(s, m, r, mass);
  const SampleSpan sp(z, p.V, 1, 0);
  for (int n = 0; n < p.N; ++n) {
    const float u = p.u[row * p.N + n];
    if (!sample_u_ok(u)) {  // the same in all threads
      if (tid == 0) {
        sample_put(p, row, n, -1, __int_as_float(0x7FC00000));
        sample_bad(p);
      }
      continue;
    }
    const SamplePlace d = sample_draw(s, m, r, L, mass, u);
    // one warp looks for it, on its own: the prefix tables stay as they are
    if (warp == 0) {
      const SampleMatch mt(__float_as_uint(s.value(d.bin)) >> 16);
      uint32_t rank = d.in_bin;
      int id = sample_scan_few(sp, mt, 0, sp.head, rank);
      if (id < 0) {
        for (int v0 = 0; v0 < sp.nvec && id < 0; v0 += 32) {
          const uint32_t no =
              v0 + lane < sp.nvec ? mt.differs8(sp.v[v0 + lane]) : SM_EIGHT;
          const uint32_t all = __reduce_add_sync(0xffffffffu, 8u - __popc(no));
          if (rank >= all) rank -= all;
          else id = sample_scan(sp, mt, v0, min(sp.nvec, v0 + 32), rank);
        }
        if (id < 0) id = sample_scan_few(sp, mt, sp.tail_at, sp.tail, rank);
      }
      if (lane == 0) sample_put(p, row, n, id, static_cast<float>(log(d.w / mass)));
    }
  }
  __syncthreads();
}

__device__ __forceinline__ SampleRow sample_row_params(const SampleParams& p, int64_t row) {
  SampleRow r;
  const double temp =
      p.temperature_rows ? static_cast<double>(p.temperature_rows[row]) : p.temperature;
  r.top_k = p.top_k_rows ? p.top_k_rows[row] : p.top_k;
  r.top_p = p.top_p_rows ? static_cast<double>(p.top_p_rows[row]) : p.top_p;
  r.min_p = p.min_p_rows ? static_cast<double>(p.min_p_rows[row]) : p.min_p;
  r.ok = temp >= 0.0 && temp < INFINITY && r.top_p > 0.0 && r.min_p >= 0.0 && r.min_p <= 1.0;
  r.greedy = temp == 0.0;
  // finite, so that the largest logit's weight stays exp(0)
  r.inv_temp = r.greedy ? 1.0 : fmin(1.0 / temp, 1e300);
  return r;
}

// Tokens and mass of the chunks a block of the row's C has (every C-th), to
// all of them; four lanes a chunk.  The bins of a chunk are neighbours of one
// binade, so their weights are a geometric series: two exponentials and a
// product a bin.
template <int C>
__device__ __noinline__ void sample_chunks(SampleShared& sm, uint32_t rank, float m) {
  const SampleRow r = sm.par;
  static_assert(SM_CB == 16, "four lanes a chunk, four bins each");
  const int PER = sample_nt() / 4;  // chunks of a pass
  const int sub = threadIdx.x & 3;
  for (int k0 = 0; k0 * C < SM_CHUNKS; k0 += PER) {  // whole warps: lanes add up below
    const int c = rank + C * (k0 + static_cast<int>(threadIdx.x) / 4);
    uint32_t n[4] = {0, 0, 0, 0};
    // the lane's bins in slot order: ascending magnitudes
    const int slot0 = c * SM_CB < SM_HALF ? SM_HALF - SM_CB - c * SM_CB : c * SM_CB;
    const int slot = slot0 + 4 * sub;
    if (c < SM_CHUNKS) {
      uint4 v[C];
#pragma unroll
      for (int b = 0; b < C; ++b)
        v[b] = C == 1 ? *reinterpret_cast<const uint4*>(&sm.hist[slot])
                      : peer_load4(peer(&sm.hist[slot], b));
#pragma unroll
      for (int b = 0; b < C; ++b) {
        n[0] += v[b].x;
        n[1] += v[b].y;
        n[2] += v[b].z;
        n[3] += v[b].w;
      }
    }
    uint32_t cnt = n[0] + n[1] + n[2] + n[3];
    double w = 0.0;
    if (cnt) {
      const uint32_t b0 = slot < SM_HALF ? SM_LO + slot
                                         : slot < SM_NEG ? 0u : 0x8000u + SM_LO + (slot - SM_NEG);
      const float step = fabsf(bf16_value(b0 + 1) - bf16_value(b0));
      float top = bf16_value(b0);
      if (slot < SM_HALF) {  // the largest of positive values is the last
        top = bf16_value(b0 + 3);
        uint32_t t = n[0];
        n[0] = n[3];
        n[3] = t;
        t = n[1];
        n[1] = n[2];
        n[2] = t;
      }
      // the bins above the row's largest value are empty; from that value on,
      // its own weight is 1 exactly
      for (int k = 0; k < 3 && top > m; ++k, top -= step) {
        n[0] = n[1];
        n[1] = n[2];
        n[2] = n[3];
        n[3] = 0;
      }
      const double e = sample_weight(top, m, r);
      const double ratio = exp(-static_cast<double>(step) * r.inv_temp);
      w = e * (n[0] + ratio * (n[1] + ratio * (n[2] + ratio * n[3])));
    }
    cnt += __shfl_xor_sync(0xffffffffu, cnt, 1);
    cnt += __shfl_xor_sync(0xffffffffu, cnt, 2);
    w += __shfl_xor_sync(0xffffffffu, w, 1);
    w += __shfl_xor_sync(0xffffffffu, w, 2);
    if (c >= SM_CHUNKS) continue;
    if constexpr (C == 1) {
      if (sub == 0) {
        sm.pc[c] = cnt;
        sm.pw[c] = w;
      }
    } else {
      for (int b = sub; b < C; b += 4) {
        peer_store(peer(&sm.pc[c], b), cnt);
        peer_store(peer(&sm.pw[c], b), w);
      }
    }
  }
}

__device__ __forceinline__ void sample_no_draw(const SampleParams& p, int64_t row, int n) {
  sample_put(p, row, n, -1, __int_as_float(0x7FC00000));
}

// Up to 64 draws of a row: the counters of the drawn values become marks, one
// pass counts each marked value in every part of the row, and each draw reads
// the one part that holds its occurrence.
template <int C>
__device__ __noinline__ void sample_batch(SampleShared& sm, const SampleParams& p, int64_t row,
                                          const SampleSpan sp, uint32_t rank, float m, int n0) {
  const SampleRow& r = sm.par;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const SampleBins<C> s{sm};
  const uint32_t L = sm.kept;
  const double mass = sm.mass;
  const int nb = min(SM_BATCH, p.N - n0);
  int shift = 5;  // a part: the fewest times 32 vectors, a power of two
  while ((SM_SEGS << shift) < sp.nvec) ++shift;
  for (int k = 0; k < nb; k += sample_nt() / 8) {  // eight threads a draw
    const int n = k + tid / 8;
    const float u = n < nb ? p.u[row * p.N + n0 + n] : 0.f;
    const bool ok = sample_u_ok(u);
    const SamplePlace d = sample_draw8(s, m, r, L, mass, ok ? u : 0.f);
    if ((tid & 7) != 0 || n >= nb) continue;
    sm.draw_bin[n] = ok ? d.bin : 0xFFFFFFFFu;
    sm.draw_rank[n] = d.in_bin;
    if (rank == 0) {
      if (!ok) {
        sample_no_draw(p, row, n0 + n);
        sample_bad(p);
      } else if (p.logp) {
        p.logp[row * p.N + n0 + n] = static_cast<float>(log(d.w / mass));
      }
    }
  }
  for (int i = tid; i < SM_SEGS * SM_BATCH / 2; i += sample_nt()) (&sm.segs[0][0])[i] = 0;
  for (int i = tid; i < 65536 / 32; i += sample_nt()) sm.drawn[i] = 0;
  sync_all<C>();  // no block reads another's counters any more
  // mark: 0x80000000 | the draw whose column counts the value; the count
  // itself is kept by the draw's thread and put back behind the pass
  uint32_t* at = nullptr;
  uint32_t kept = 0;
  if (tid < nb && sm.draw_bin[tid] != 0xFFFFFFFFu) {
    const int bin = static_cast<int>(sm.draw_bin[tid]);
    at = &sm.hist[sample_bin_slot(bin)];
    kept = *at;
    if constexpr (C > 1)
      for (int b = 0; b < C; ++b) peer_store(peer(&sm.found[rank][tid], b), kept);
    const uint32_t x = sample_bin_bits(bin);
    atomicOr(&sm.drawn[x / 32], 1u << (x % 32));
    if (x == 0u) atomicOr(&sm.drawn[0x8000 / 32], 1u);  // -0
  }
  __syncthreads();
  if (at) atomicMax(at, 0x80000000u | static_cast<uint32_t>(tid));
  __syncthreads();
  sample_marked_pass(sm, sp.v, sp.nvec, shift);
  sync_all<C>();  // and every block's counts of the drawn values are there
  auto in_part = [&](uint32_t seg, uint32_t col) {
    return (sm.segs[seg][col >> 1] >> ((col & 1u) * 16u)) & 0xFFFFu;
  };
  for (int n = warp; n < nb; n += sample_nw()) {
    const uint32_t bin = sm.draw_bin[n];
    if (bin == 0xFFFFFFFFu) continue;
    const uint32_t col = sm.hist[sample_bin_slot(static_cast<int>(bin))] & (SM_BATCH - 1u);
    const SampleMatch mt(sample_bin_bits(static_cast<int>(bin)));
    uint32_t left = sm.draw_rank[n];
    if constexpr (C > 1) {
      bool here = true;
      for (uint32_t k = 0; k < rank && here; ++k) {
        if (left < sm.found[k][n]) here = false;  // in a block before this one
        else left -= sm.found[k][n];
      }
      if (!here || left >= sm.found[rank][n]) continue;
    }
    int id = sp.head ? sample_scan_few(sp, mt, 0, sp.head, left) : -1;
    if (id < 0) {
      // lane l: parts 4 l .. 4 l + 3
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k] = in_part(4 * lane + k, col);
        sum += c[k];
      }
      const uint32_t upto = warp_scan(sum);
      const uint32_t hit = __ballot_sync(0xffffffffu, upto > left);
      if (hit == 0) {
        left -= __shfl_sync(0xffffffffu, upto, 31);
        id = sample_scan_few(sp, mt, sp.tail_at, sp.tail, left);
      } else {
        const int l = __ffs(hit) - 1;
        uint32_t in = left - (upto - sum);
        int seg = 4 * lane;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (seg == 4 * lane + k && in >= c[k]) {
            in -= c[k];
            ++seg;
          }
        in = __shfl_sync(0xffffffffu, in, l);
        seg = __shfl_sync(0xffffffffu, seg, l);
        id = sample_scan(sp, mt, seg << shift, min(sp.nvec, (seg + 1) << shift), in);
      }
    }
    if (lane == 0) p.ids[row * p.N + n0 + n] = id;
  }
  __syncthreads();
  if (at) *at = kept;
  sync_all<C>();  // the counters are as they were, for the next draws
}

template <int C, bool MANY>
__global__ void __launch_bounds__(sample_threads(MANY), sample_blocks(MANY))
sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t sample_smem[];
  SampleShared& sm = *reinterpret_cast<SampleShared*>(sample_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = C == 1 ? 0u : cluster_ctarank();
  for (int64_t row = blockIdx.x / C; row < p.T; row += gridDim.x / C) {
    const SampleSpan sp(p.logits + row * p.ld, p.V, C, rank);
    const bool first = row == blockIdx.x / C;
    arrive_all<C>();
    if (!first) {  // the last row's reads of shared memory
      wait_all<C>();
      if constexpr (C == 1) __syncthreads();
    }
    for (int i = tid; i < SM_BINS / 4; i += sample_nt())
      reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (tid == sample_nt() - 1) sm.par = sample_row_params(p, row);

    // ---- how often each value occurs, and the largest
    const uint64_t seen = sample_count_pass<!MANY>(sm.hist, sp.v, sp.nvec);
    const uint32_t m2 = static_cast<uint32_t>(seen);
    uint32_t flags = static_cast<uint32_t>(seen >> 32);
    float m = fmaxf(bf16_lo(m2), bf16_hi(m2));
    if (tid < sp.head + sp.tail) {
      const uint32_t x = sp.z[tid < sp.head ? tid : sp.tail_at + tid - sp.head];
      sample_count1(sm.hist, x, flags);
      m = fmaxf(m, bf16_value(x));
    }
    // every warp's, to all blocks
    const uint32_t key =
        (__reduce_max_sync(0xffffffffu, bf16_key(__float_as_uint(m) >> 16)) << 16) |
        __reduce_or_sync(0xffffffffu, flags);
    if (first) wait_all<C>();  // the other blocks run by now
    if constexpr (C == 1) {
      if (lane == 0) sm.seen[warp] = key;
    } else {
      if (lane < C) peer_store(peer(&sm.seen[rank * sample_nw() + warp], lane), key);
    }
    sync_all<C>();
    uint32_t top = 0;
    flags = 0;
    for (int i = lane; i < C * sample_nw(); i += 32) {
      top = max(top, sm.seen[i] >> 16);
      flags |= sm.seen[i] & 0xFFFFu;
    }
    m = key_value(__reduce_max_sync(0xffffffffu, top));  // -0 is +0
    flags = __reduce_or_sync(0xffffffffu, flags);

    // the rest is decided alike in all blocks of the row
    const SampleRow& r = sm.par;
    const bool bad = !r.ok || (flags & SF_BAD);
    if (bad || m == -INFINITY) {  // no answer: bad numbers, or nothing left to draw
      if (rank == 0)
        for (uint32_t n = tid; n < sample_draws(p); n += sample_nt()) sample_no_draw(p, row, n);
      if (bad && rank == 0 && tid == 0) sample_bad(p);
      continue;
    }
    // values of -256 and less weigh at most 2^((-256 - m) log2(e) / temp)
    const bool low_counts =
        (flags & SF_LOW) &&
        (m <= -256.f || (!r.greedy && (m + 256.0) * 1.4426950408889634 * r.inv_temp < 64.0));
    if ((flags & SF_ANY) || low_counts) {
      if (rank == 0) sample_row_any(sm, p, row);
      continue;
    }

    // ---- tokens and mass before every chunk of values
    sample_chunks<C>(sm, rank, m);
    sync_all<C>();
    sample_prefix(sm, sm.pc, sm.pw, SM_CHUNKS);

    // ---- what the filters keep, the draws
    if (warp == 0) {
      const SampleBins<C> s{sm};
      double mass;
      const uint32_t L = sample_kept(s, m, r, mass);
      if constexpr (!MANY) {
        const float u = p.u[row];
        const bool ok = sample_u_ok(u);
        const SamplePlace d = sample_draw(s, m, r, L, mass, ok ? u : 0.f);
        if (lane == 0) {
          sm.draw_bin[0] = ok ? d.bin : 0xFFFFFFFFu;
          sm.draw_rank[0] = d.in_bin;
          sm.draw_w = d.w;
        }
      }
      if (lane == 0) {
        sm.kept = L;
        sm.mass = mass;
      }
    }
    __syncthreads();
    if constexpr (MANY) {
      for (uint32_t n0 = 0; n0 < sample_draws(p); n0 += SM_BATCH)
        sample_batch<C>(sm, p, row, sp, rank, m, n0);
    } else {
      const uint32_t bin = sm.draw_bin[0];
      if (bin == 0xFFFFFFFFu) {
        if (rank == 0 && tid == 0) {
          sample_no_draw(p, row, 0);
          sample_bad(p);
        }
        continue;
      }
      if (rank == 0 && tid == 32 && p.logp)
        p.logp[row] = static_cast<float>(log(sm.draw_w / sm.mass));
      sample_find<C>(sm, sp, rank, static_cast<int>(bin), sm.draw_rank[0], p.ids + row);
    }
  }
  if constexpr (C > 1) sync_all<C>();  // no block leaves while another reads its counters
}

// ------------------------------------------------------------- short rows
// Rows of up to 4096 logits: sorted whole (value descending, id ascending, one
// 32-bit word each), with the running masses beside them, so that a draw is a
// bisection.  The counters' fixed cost a row (12304 of them to clear and to turn
// into masses, and the search for an occurrence) would be several times the
// row's own work: 4000 x 1499, 32 draws each, 341 us with them, 128 us so; one
// draw 136 and 128.  4000 x 4096: 32 draws 345 and 263, one draw 141 and 263, so
// that form is for rows of up to 2048, and up to 4096 with several draws.
// A thread holds E neighbours, so that only the last of the sort's steps, over
// more than a warp's 32 E, go through shared memory (six of 66 at 2048).
constexpr int SM_SHORT_V = 2048, SM_SHORT_V_MANY = 4096;
constexpr int SM_SHORT_THREADS = 256;
constexpr int SM_SHORT_WARPS = SM_SHORT_THREADS / 32;

__device__ __forceinline__ void sample_order(uint32_t& a, uint32_t& b, bool up) {
  const uint32_t lo = min(a, b), hi = max(a, b);
  a = up ? lo : hi;
  b = up ? hi : lo;
}

// Bitonic sort, ascending, of the block's SM_SHORT_THREADS E words, E a thread.
template <int E>
__device__ __forceinline__ void sample_sort(uint32_t (&x)[E], uint32_t* buf0, uint32_t* buf1) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int k = 2; k <= E; k <<= 1) {  // runs of a thread's own
#pragma unroll
    for (int j = k / 2; j > 0; j >>= 1)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((e & j) == 0) sample_order(x[e], x[e + j], ((tid * E + e) & k) == 0);
  }
#pragma unroll 1
  for (int t = 2; t <= SM_SHORT_THREADS; t <<= 1) {  // runs of t threads
    const bool up = (tid & t) == 0;
#pragma unroll 1
    for (int d = t / 2; d >= 32; d >>= 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) buf0[e * SM_SHORT_THREADS + tid] = x[e];
      __syncthreads();
      const bool low = (tid & d) == 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t y = buf0[e * SM_SHORT_THREADS + (tid ^ d)];
        x[e] = low == up ? min(x[e], y) : max(x[e], y);
      }
      uint32_t* turn = buf0;  // the next step writes the other one: one barrier a step
      buf0 = buf1;
      buf1 = turn;
    }
#pragma unroll 1
    for (int d = min(t / 2, 16); d > 0; d >>= 1) {
      const bool low = (tid & d) == 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t y = __shfl_xor_sync(0xffffffffu, x[e], d);
        x[e] = low == up ? min(x[e], y) : max(x[e], y);
      }
    }
#pragma unroll
    for (int j = E / 2; j > 0; j >>= 1)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((e & j) == 0) sample_order(x[e], x[e + j], up);
  }
}

template <int E>
__global__ void __launch_bounds__(SM_SHORT_THREADS)
sample_short_kernel(const __grid_constant__ SampleParams p) {
  constexpr int P = SM_SHORT_THREADS * E;
  extern __shared__ __align__(16) uint8_t sample_smem[];
  double* cum = reinterpret_cast<double*>(sample_smem);  // [P] running masses
  uint32_t* tok = reinterpret_cast<uint32_t*>(cum + P);  // [P] order << 16 | id
  __shared__ double scan_w[SM_SHORT_WARPS];
  __shared__ uint32_t scan_n[SM_SHORT_WARPS], scan_k[SM_SHORT_WARPS], scan_f[SM_SHORT_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const uint16_t* z = p.logits + row * p.ld;
    const SampleRow r = sample_row_params(p, row);
    uint32_t x[E], n = 0, flags = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int i = k * SM_SHORT_THREADS + tid;
      x[k] = 0xFFFFFFFFu;  // -inf and what is behind the row: last
      if (i < p.V) {
        const uint32_t v = z[i];
        if ((v & 0x7FFFu) >= 0x7F80u) {
          if (v != 0xFF80u) flags = SF_BAD;
        } else {
          x[k] = (0xFFFFu - bf16_key(v)) << 16 | static_cast<uint32_t>(i);
          ++n;
        }
      }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    flags = __reduce_or_sync(0xffffffffu, flags);
    __syncthreads();  // the last row's reads of shared memory
    if (lane == 0) {
      scan_n[warp] = n;
      scan_f[warp] = flags;
    }
    sample_sort<E>(x, tok, reinterpret_cast<uint32_t*>(cum));
    __syncthreads();
#pragma unroll
    for (int k = 0; k < E; ++k) tok[tid * E + k] = x[k];
    __syncthreads();
    n = 0;
    for (int w = 0; w < SM_SHORT_WARPS; ++w) {
      n += scan_n[w];
      flags |= scan_f[w];
    }
    const bool bad = !r.ok || flags;
    if (bad || n == 0) {
      for (uint32_t k = tid; k < sample_draws(p); k += SM_SHORT_THREADS) sample_no_draw(p, row, k);
      if (bad && tid == 0) sample_bad(p);
      continue;
    }
    auto value = [](uint32_t t) { return key_value(0xFFFFu - (t >> 16)); };
    const float m = value(tok[0]);

    // running masses: over a thread's tokens, then over the threads
    double sums[E];
    uint32_t above = 0;  // tokens with w >= min_p
#pragma unroll
    for (int k = 0; k < E; ++k) {
      double w = 0.0;
      if (tid * E + k < static_cast<int>(n)) {
        w = sample_weight(value(x[k]), m, r);
        above += w >= r.min_p;
      }
      sums[k] = k ? sums[k - 1] + w : w;
    }
    const double upto = warp_scan(sums[E - 1]);
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 31) {
      scan_w[warp] = upto;
      scan_k[warp] = above;
    }
    __syncthreads();
    double before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0) before = 0.0;
    above = 0;
    double warps = 0.0;
    for (int w = 0; w < SM_SHORT_WARPS; ++w) {
      if (w < warp) warps += scan_w[w];
      above += scan_k[w];
    }
    before += warps;
#pragma unroll
    for (int k = 0; k < E; ++k) cum[tid * E + k] = before + sums[k];
    __syncthreads();

    // the first of [0, count) with past, or count
    auto first = [&](uint32_t count, auto past) {
      uint32_t lo = 0, hi = count;
      while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (past(cum[mid])) hi = mid;
        else lo = mid + 1;
      }
      return lo;
    };
    uint32_t L = n;
    if (r.greedy) {
      L = 1;
    } else {
      if (r.top_k > 0) L = min(L, static_cast<uint32_t>(r.top_k));
      uint32_t keep = L;
      if (r.top_p < 1.0) {
        const double mass = r.top_p * cum[L - 1];
        keep = min(keep, first(L, [&](double x) { return x >= mass; }) + 1);
      }
      if (r.min_p > 0.0) keep = min(keep, max(1u, above));
      L = keep;
    }
    const double mass = cum[L - 1];
    for (uint32_t k = tid; k < sample_draws(p); k += SM_SHORT_THREADS) {
      const float u = p.u[row * p.N + k];
      if (!sample_u_ok(u)) {
        sample_no_draw(p, row, k);
        sample_bad(p);
        continue;
      }
      const double target = static_cast<double>(u) * mass;
      const uint32_t at = min(first(L, [&](double x) { return x > target; }), L - 1);
      sample_put(p, row, k, static_cast<int>(tok[at] & 0xFFFFu),
                 p.logp ? static_cast<float>(log(sample_weight(value(tok[at]), m, r) / mass)) : 0.f);
    }
  }
}

}  // namespace ckl
