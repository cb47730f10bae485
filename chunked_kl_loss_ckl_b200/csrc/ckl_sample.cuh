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
// instead (sample_row_any), unless all of them are so far below the largest
// logit (2^-64 of its weight) that their mass, under 2^-40 of the row's, is
// never reached by a u of 24 bits.
#pragma once

#include <cstdint>

#include "ckl_bf16.cuh"

#define CKL_DEV_BAD_SAMPLE 16  // NaN or +inf logit, or a parameter or number out of range

namespace ckl {

constexpr int SM_THREADS = 512;
constexpr int SM_WARPS = SM_THREADS / 32;
constexpr uint32_t SM_LO = 0x2B80;              // bf16 bits of 2^-40
constexpr uint32_t SM_HI = 0x4380;              // bf16 bits of 256
constexpr int SM_HALF = SM_HI - SM_LO;          // bins of one sign
constexpr int SM_BINS = 2 * SM_HALF + 1;
constexpr int SM_CHUNKS = (SM_BINS + 31) / 32;  // 32 bins, one a lane
constexpr int SM_SLOTS = SM_CHUNKS * 32;
constexpr int SM_WIN = 8192;                    // keys of a window (rows of any values)
constexpr int SM_ANY_CHUNKS = 65536 / 32;
constexpr int SM_TILES = 1024;                  // tiles whose matches are counted, at most
constexpr int SM_SEGS = 128;                    // parts of the row counted per draw
constexpr int SM_BATCH = 64;                    // draws found in one pass

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
  double temp, top_p, min_p;
  int32_t top_k;
  bool greedy, ok;
};

struct alignas(16) SampleShared {
  // counters of the bins (slot order below), or of a window's keys; behind a
  // window's 8192 counters, the prefix masses of all 2048 chunks
  uint32_t hist[SM_SLOTS];
  double pw[SM_CHUNKS + 1];    // mass before each chunk
  uint32_t pc[SM_CHUNKS + 1];  // tokens before each chunk
  union {
    uint16_t tiles[SM_TILES + 2];           // matches of one value in each tile
    uint32_t segs[SM_SEGS][SM_BATCH / 2];   // matches of up to 64 values in each part, 16 bits each
    uint32_t any_pc[SM_ANY_CHUNKS + 1];
  };
  uint32_t draw_bin[SM_BATCH], draw_rank[SM_BATCH];
  uint32_t cb[32];  // one chunk's counters (rows of any values)
  float red[SM_WARPS];
  uint32_t flags[SM_WARPS];
};
static_assert(SM_WIN * 4 + (SM_ANY_CHUNKS + 1) * 8 <= SM_SLOTS * 4, "prefix masses behind a window");

enum : uint32_t { SF_BAD = 1, SF_LOW = 2, SF_ANY = 4 };

// A row's elements: up to 7 before the first 16-byte boundary, whole vectors
// of eight, up to 7 behind the last.
struct SampleSpan {
  const uint16_t* z;
  const uint4* v;
  int head, nvec, tail;
  __device__ __forceinline__ SampleSpan(const uint16_t* row, int V) : z(row) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
    head = min(V, static_cast<int>(((16u - off) & 15u) / 2u));
    v = reinterpret_cast<const uint4*>(row + head);
    nvec = (V - head) / 8;
    tail = V - head - 8 * nvec;
  }
  __device__ __forceinline__ int tail_at() const { return head + 8 * nvec; }
};

// The counter of a value of the covered range: the positive values ascending,
// zero, the negative ones descending (bits apart from the sign, plus SM_HALF
// + 1 when it is set).
__device__ __forceinline__ uint32_t sample_slot(uint32_t x) {
  return (x & 0x7FFFu) + (x >> 15) * (SM_HALF + 1) - SM_LO;
}
// Bin b (descending values) -> its counter, and its value.
__device__ __forceinline__ int sample_bin_slot(int b) {
  return b < SM_HALF ? SM_HALF - 1 - b : b;
}
__device__ __forceinline__ uint32_t sample_bin_bits(int b) {
  if (b < SM_HALF) return SM_LO + (SM_HALF - 1 - b);
  return b == SM_HALF ? 0u : 0x8000u + SM_LO + (b - SM_HALF - 1);
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

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the lanes up to and with this one.
__device__ __forceinline__ double warp_scan(double v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__device__ __forceinline__ double sample_weight(float v, float m, const SampleRow& r) {
  return exp((static_cast<double>(v) - static_cast<double>(m)) / r.temp);
}

// The counts of a row, read chunk by chunk: the bins of a row of covered
// values, in shared memory.
struct SampleBins {
  SampleShared& sm;
  static constexpr int CHUNKS = SM_CHUNKS, BINS = SM_BINS;
  static constexpr bool BLOCK = false;  // a warp can read a chunk on its own
  __device__ __forceinline__ const double* pw() const { return sm.pw; }
  __device__ __forceinline__ const uint32_t* pc() const { return sm.pc; }
  __device__ __forceinline__ uint32_t count(int chunk) const {
    const int b = chunk * 32 + (threadIdx.x & 31);
    return b < SM_BINS ? sm.hist[sample_bin_slot(b)] : 0u;
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
  static constexpr int CHUNKS = SM_ANY_CHUNKS, BINS = 0xFF81;
  static constexpr bool BLOCK = true;
  __device__ __forceinline__ double* pw() const {
    return reinterpret_cast<double*>(sm.hist + SM_WIN);
  }
  __device__ __forceinline__ uint32_t* pc() const { return sm.any_pc; }
  __device__ __noinline__ uint32_t count(int chunk) const {
    __syncthreads();
    if (threadIdx.x < 32) sm.cb[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < V; i += SM_THREADS) {
      const uint32_t b = 0xFFFFu - bf16_key(z[i]);
      if (static_cast<int>(b >> 5) == chunk && z[i] != 0xFF80u) atomicAdd(&sm.cb[b & 31u], 1u);
    }
    __syncthreads();
    return sm.cb[threadIdx.x & 31];
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

// The last chunk c with pred(prefix c); pred holds for the first one and
// changes once.
template <typename F>
__device__ __forceinline__ int sample_chunk(int n, F&& pred) {
  int lo = 0, hi = n;  // pred(lo), not pred(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pred(mid)) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The token at a rank.
template <typename S>
__device__ __forceinline__ SamplePlace sample_at_rank(const S& s, float m, const SampleRow& r,
                                                      uint32_t rank) {
  const int c = sample_chunk(S::CHUNKS, [&](int i) { return s.pc()[i] <= rank; });
  const int lane = threadIdx.x & 31;
  const uint32_t n = s.count(c);
  const double w = n ? sample_weight(s.value(c * 32 + lane), m, r) : 0.0;
  const uint32_t upto = warp_scan(n) + s.pc()[c];
  const double mass = warp_scan(n * w) - n * w + s.pw()[c];
  const uint32_t hit = __ballot_sync(0xffffffffu, upto > rank);
  const int l = hit ? __ffs(hit) - 1 : 31;
  SamplePlace p;
  p.bin = c * 32 + l;
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
  auto past = [&](double x) { return STRICT ? x > target : x >= target; };
  const int c = sample_chunk(S::CHUNKS, [&](int i) { return i == 0 || !past(s.pw()[i]); });
  const int lane = threadIdx.x & 31;
  const uint32_t n = s.count(c);
  const double w = n ? sample_weight(s.value(c * 32 + lane), m, r) : 0.0;
  const uint32_t rank0 = warp_scan(n) - n + s.pc()[c];
  const double upto = warp_scan(n * w) + s.pw()[c];
  const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
  const uint32_t hit = __ballot_sync(0xffffffffu, n > 0 && past(upto));
  // sums taken in another order may differ in the last bit: then the chunk's last
  const int l = hit ? __ffs(hit) - 1 : (some ? 31 - __clz(some) : 0);
  const uint32_t nl = __shfl_sync(0xffffffffu, n, l);
  SamplePlace p;
  p.bin = c * 32 + l;
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
  if (lo >= S::BINS) return s.pc()[S::CHUNKS];
  const uint32_t n = s.count(lo / 32);
  const uint32_t in = __reduce_add_sync(0xffffffffu, lane < (lo & 31) ? n : 0u);
  return s.pc()[lo / 32] + in;
}

// How many tokens the filters keep and their mass.
template <typename S>
__device__ __forceinline__ uint32_t sample_kept(const S& s, float m, const SampleRow& r,
                                                double& mass) {
  const uint32_t n = s.pc()[S::CHUNKS];
  uint32_t L = n;
  mass = s.pw()[S::CHUNKS];
  if (r.greedy) {
    L = 1;
  } else {
    if (r.top_k > 0 && static_cast<uint32_t>(r.top_k) < n) {
      L = static_cast<uint32_t>(r.top_k);
      const SamplePlace p = sample_at_rank(s, m, r, L - 1);
      mass = p.mass + p.w;
    }
    uint32_t keep = L;
    if (r.top_p < 1.0) keep = min(keep, sample_at_mass<false>(s, m, r, r.top_p * mass).rank + 1);
    if (r.min_p > 0.0) keep = min(keep, max(1u, sample_min_p(s, m, r)));
    if (keep == L) return L;
    L = keep;
  }
  const SamplePlace p = sample_at_rank(s, m, r, L - 1);
  mass = p.mass + p.w;
  return L;
}

// One draw among the first L tokens.
template <typename S>
__device__ __forceinline__ SamplePlace sample_draw(const S& s, float m, const SampleRow& r,
                                                   uint32_t L, double mass, float u) {
  const SamplePlace p = sample_at_mass<true>(s, m, r, static_cast<double>(u) * mass);
  return p.rank < L ? p : sample_at_rank(s, m, r, L - 1);  // u mass rounded up to the mass
}

__device__ __forceinline__ bool sample_u_ok(float u) { return u >= 0.f && u < 1.f; }

// Turns the chunks' counts and masses into those before each chunk (one warp).
__device__ __forceinline__ void sample_prefix(uint32_t* pc, double* pw, int n) {
  const int lane = threadIdx.x & 31;
  const int per = (n + 31) / 32, b = min(n, lane * per), e = min(n, b + per);
  uint32_t c = 0;
  double w = 0.0;
  for (int i = b; i < e; ++i) {
    c += pc[i];
    w += pw[i];
  }
  uint32_t c0 = warp_scan(c) - c;
  double w0 = warp_scan(w) - w;
  if (lane == 31) {
    pc[n] = c0 + c;
    pw[n] = w0 + w;
  }
  for (int i = b; i < e; ++i) {
    const uint32_t ci = pc[i];
    const double wi = pw[i];
    pc[i] = c0;
    pw[i] = w0;
    c0 += ci;
    w0 += wi;
  }
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

// Id of occurrence `rank` (from 0) of a value, by one warp over vectors
// [v0, v1) of the row; before them come `rank` of its occurrences fewer.
// Returns -1 if they are not there.
__device__ __forceinline__ int sample_scan(const SampleSpan& sp, const SampleMatch& mt, int v0,
                                           int v1, uint32_t rank) {
  const int lane = threadIdx.x & 31;
  for (int b = v0; b < v1; b += 32) {
    uint32_t no = SM_EIGHT;
    if (b + lane < v1) no = mt.differs8(sp.v[b + lane]);
    const uint32_t n = 8u - __popc(no);
    const uint32_t upto = warp_scan(n);
    const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
    if (rank >= all) {
      rank -= all;
      continue;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, upto > rank);
    const int l = __ffs(hit) - 1;
    int id = 0;
    if (lane == l) {
      uint32_t left = rank - (upto - n);
      for (int j = 0; j < 8; ++j) {
        const bool is = !((no >> ((j & 1) ? 31 - j / 2 : 15 - j / 2)) & 1u);
        if (is && left-- == 0) {
          id = sp.head + 8 * (b + lane) + j;
          break;
        }
      }
    }
    return __shfl_sync(0xffffffffu, id, l);
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

// Id of one (value, occurrence), by the block: the matches of every tile of
// the row are counted, and the tile that holds the occurrence is read again.
// The result is valid in warp 0.
__device__ int sample_find(SampleShared& sm, const SampleSpan& sp, uint32_t bits, uint32_t rank) {
  const SampleMatch mt(bits);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int steps = max(1, (sp.nvec + 32 * SM_TILES - 1) / (32 * SM_TILES));  // 32 vectors each
  const int tv = 32 * steps, nt = (sp.nvec + tv - 1) / tv;
  __syncthreads();  // the counters of tiles share memory with what was read before
  for (int t = warp; t < nt; t += SM_WARPS) {
    uint32_t n = 0;
    for (int k = 0; k < steps; ++k) {
      const int i = t * tv + k * 32 + lane;
      if (i < sp.nvec) n += 8u - __popc(mt.differs8(sp.v[i]));
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sm.tiles[t] = static_cast<uint16_t>(n);
  }
  __syncthreads();
  if (warp != 0) return -1;
  const int few = sample_scan_few(sp, mt, 0, sp.head, rank);
  if (few >= 0) return few;
  const int per = (nt + 31) / 32;
  uint32_t mine = 0;
  for (int i = lane * per; i < min(nt, (lane + 1) * per); ++i) mine += sm.tiles[i];
  const uint32_t upto = warp_scan(mine);
  const uint32_t hit = __ballot_sync(0xffffffffu, upto > rank);
  if (hit == 0) {
    rank -= __shfl_sync(0xffffffffu, upto, 31);
    return sample_scan_few(sp, mt, sp.tail_at(), sp.tail, rank);
  }
  const int l = __ffs(hit) - 1;
  rank -= __shfl_sync(0xffffffffu, upto - mine, l);
  int t = l * per;
  while (rank >= sm.tiles[t]) rank -= sm.tiles[t++];
  return sample_scan(sp, mt, t * tv, min(sp.nvec, (t + 1) * tv), rank);
}

__device__ __forceinline__ void sample_put(const SampleParams& p, int64_t row, int n, int id,
                                           float logp) {
  p.ids[row * p.N + n] = id;
  if (p.logp) p.logp[row * p.N + n] = logp;
}

__device__ __forceinline__ void sample_bad(const SampleParams& p) {
  if (p.status) atomicOr(p.status, CKL_DEV_BAD_SAMPLE);
}

// A row whose finite values are not all covered: the key space in eight
// windows, one pass over the row each, and a pass for every chunk looked into.
__device__ __noinline__ void sample_row_any(SampleShared& sm, const SampleParams& p, int64_t row,
                                            const SampleRow& r) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint16_t* z = p.logits + row * p.ld;
  SampleKeys s{sm, z, p.V};
  float m = 0.f;
  bool have = false;
  for (int win = 0; win < 65536 / SM_WIN; ++win) {
    __syncthreads();
    for (int i = tid; i < SM_WIN; i += SM_THREADS) sm.hist[i] = 0;
    if (tid < SM_WARPS) sm.flags[tid] = 0xFFFFFFFFu;
    __syncthreads();
    uint32_t top = 0xFFFFFFFFu;  // the first bin of the window that occurs
    for (int i = tid; i < p.V; i += SM_THREADS) {
      const uint32_t x = z[i], b = 0xFFFFu - bf16_key(x);
      if (static_cast<int>(b / SM_WIN) == win && x != 0xFF80u) {
        atomicAdd(&sm.hist[b % SM_WIN], 1u);
        top = min(top, b);
      }
    }
    top = __reduce_min_sync(0xffffffffu, top);
    if (lane == 0) sm.flags[warp] = top;
    __syncthreads();
    for (int w = 0; w < SM_WARPS; ++w) top = min(top, sm.flags[w]);
    if (!have && top != 0xFFFFFFFFu) {
      m = s.value(static_cast<int>(top));
      have = true;
    }
    for (int c = warp; c < SM_WIN / 32; c += SM_WARPS) {
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
  if (warp == 0) sample_prefix(s.pc(), s.pw(), SM_ANY_CHUNKS);
  __syncthreads();
  double mass;
  const uint32_t L = sample_kept(s, m, r, mass);
  const SampleSpan sp(z, p.V);
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
        if (id < 0) id = sample_scan_few(sp, mt, sp.tail_at(), sp.tail, rank);
      }
      if (lane == 0) sample_put(p, row, n, id, static_cast<float>(log(d.w / mass)));
    }
  }
  __syncthreads();
}

__device__ __forceinline__ SampleRow sample_row_params(const SampleParams& p, int64_t row) {
  SampleRow r;
  r.temp = p.temperature_rows ? static_cast<double>(p.temperature_rows[row]) : p.temperature;
  r.top_k = p.top_k_rows ? p.top_k_rows[row] : p.top_k;
  r.top_p = p.top_p_rows ? static_cast<double>(p.top_p_rows[row]) : p.top_p;
  r.min_p = p.min_p_rows ? static_cast<double>(p.min_p_rows[row]) : p.min_p;
  r.ok = r.temp >= 0.0 && r.temp < INFINITY && r.top_p > 0.0 && r.min_p >= 0.0 && r.min_p <= 1.0;
  r.greedy = r.temp == 0.0;
  if (r.greedy) r.temp = 1.0;
  return r;
}

__global__ void __launch_bounds__(SM_THREADS, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t sample_smem[];
  SampleShared& sm = *reinterpret_cast<SampleShared*>(sample_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const SampleSpan sp(p.logits + row * p.ld, p.V);
    const SampleRow r = sample_row_params(p, row);
    __syncthreads();  // the last row's reads of shared memory
    for (int i = tid; i < SM_SLOTS / 4; i += SM_THREADS)
      reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();

    // ---- how often each value occurs, and the largest
    uint32_t flags = 0;
    uint32_t m2 = 0xFF80FF80u;
    for (int i = tid; i < sp.nvec; i += SM_THREADS) {
      const uint4 v = sp.v[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      m2 = bf16x2_max(m2, bf16x2_max(bf16x2_max(v.x, v.y), bf16x2_max(v.z, v.w)));
      if ((sample_outside(v.x) | sample_outside(v.y) | sample_outside(v.z) |
           sample_outside(v.w)) == 0u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          atomicAdd(&sm.hist[sample_slot(w[j] & 0xFFFFu)], 1u);
          atomicAdd(&sm.hist[sample_slot(w[j] >> 16)], 1u);
        }
      } else {
        for (int j = 0; j < 4; ++j) {
          sample_count1(sm.hist, w[j] & 0xFFFFu, flags);
          sample_count1(sm.hist, w[j] >> 16, flags);
        }
      }
    }
    float m = fmaxf(bf16_lo(m2), bf16_hi(m2));
    if (tid < sp.head + sp.tail) {
      const uint32_t x = sp.z[tid < sp.head ? tid : sp.tail_at() + tid - sp.head];
      sample_count1(sm.hist, x, flags);
      m = fmaxf(m, bf16_value(x));
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) {
      sm.red[warp] = m;
      sm.flags[warp] = flags;
    }
    __syncthreads();
    for (int w = 0; w < SM_WARPS; ++w) {
      m = fmaxf(m, sm.red[w]);
      flags |= sm.flags[w];
    }
    if (m == 0.f) m = 0.f;  // -0 counts as +0

    const bool bad = !r.ok || (flags & SF_BAD);
    if (bad || m == -INFINITY) {  // no answer: bad numbers, or nothing left to draw
      for (int n = tid; n < p.N; n += SM_THREADS)
        sample_put(p, row, n, -1, __int_as_float(0x7FC00000));
      if (bad && tid == 0) sample_bad(p);
      continue;
    }
    // values of -256 and less weigh at most 2^((-256 - m) log2(e) / temp)
    const bool low_counts =
        (flags & SF_LOW) &&
        (m <= -256.f || (!r.greedy && (m + 256.0) * 1.4426950408889634 < 64.0 * r.temp));
    if ((flags & SF_ANY) || low_counts) {
      sample_row_any(sm, p, row, r);
      continue;
    }

    // ---- tokens and mass of every chunk of 32 values, then before each
    const SampleBins s{sm};
    for (int c = warp; c < SM_CHUNKS; c += SM_WARPS) {
      const uint32_t n = s.count(c);
      uint32_t cnt = 0;
      double w = 0.0;
      if (__any_sync(0xffffffffu, n != 0)) {
        if (n) w = n * sample_weight(s.value(c * 32 + lane), m, r);
        w = warp_sum(w);
        cnt = __reduce_add_sync(0xffffffffu, n);
      }
      if (lane == 0) {
        sm.pc[c] = cnt;
        sm.pw[c] = w;
      }
    }
    __syncthreads();
    if (warp == 0) sample_prefix(sm.pc, sm.pw, SM_CHUNKS);
    __syncthreads();

    // ---- what the filters keep (every warp for itself), the draws
    double mass;
    const uint32_t L = sample_kept(s, m, r, mass);
    if (p.N == 1) {
      const float u = p.u[row];
      if (!sample_u_ok(u)) {
        if (tid == 0) {
          sample_put(p, row, 0, -1, __int_as_float(0x7FC00000));
          sample_bad(p);
        }
        continue;
      }
      const SamplePlace d = sample_draw(s, m, r, L, mass, u);
      const int id = sample_find(sm, sp, sample_bin_bits(d.bin), d.in_bin);
      if (tid == 0) sample_put(p, row, 0, id, static_cast<float>(log(d.w / mass)));
      continue;
    }

    // ---- many draws: the counters of the drawn values become marks, and one
    // pass counts each marked value in every part of the row
    const int seg_vecs = max(32, ((sp.nvec + SM_SEGS - 1) / SM_SEGS + 31) / 32 * 32);
    for (int n0 = 0; n0 < p.N; n0 += SM_BATCH) {
      const int nb = min(SM_BATCH, p.N - n0);
      __syncthreads();
      for (int n = warp; n < nb; n += SM_WARPS) {
        const float u = p.u[row * p.N + n0 + n];
        const bool ok = sample_u_ok(u);
        const SamplePlace d = sample_draw(s, m, r, L, mass, ok ? u : 0.f);
        if (lane == 0) {
          sm.draw_bin[n] = ok ? d.bin : 0xFFFFFFFFu;
          sm.draw_rank[n] = d.in_bin;
          if (!ok) {
            sample_put(p, row, n0 + n, -1, __int_as_float(0x7FC00000));
            sample_bad(p);
          } else if (p.logp) {
            p.logp[row * p.N + n0 + n] = static_cast<float>(log(d.w / mass));
          }
        }
      }
      for (int i = tid; i < SM_SEGS * SM_BATCH / 2; i += SM_THREADS) (&sm.segs[0][0])[i] = 0;
      __syncthreads();
      // mark: 0x80000000 | the draw whose column counts the value; the count
      // itself is kept by the draw's thread and put back behind the pass
      uint32_t* at = nullptr;
      uint32_t kept = 0;
      if (tid < nb && sm.draw_bin[tid] != 0xFFFFFFFFu) {
        at = &sm.hist[sample_bin_slot(static_cast<int>(sm.draw_bin[tid]))];
        kept = *at;
      }
      __syncthreads();
      if (at) atomicMax(at, 0x80000000u | static_cast<uint32_t>(tid));
      __syncthreads();
      auto count = [&](uint32_t x, int seg) {
        const uint32_t a = x & 0x7FFFu;
        if (a != 0u && (a < SM_LO || a >= SM_HI)) return;
        const uint32_t h = sm.hist[sample_slot_of(x)];
        if (h & 0x80000000u)
          atomicAdd(&sm.segs[seg][(h & 63u) >> 1], (h & 1u) ? 0x10000u : 1u);
      };
      for (int i = tid; i < sp.nvec; i += SM_THREADS) {
        const uint4 v = sp.v[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const int seg = i / seg_vecs;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          count(w[j] & 0xFFFFu, seg);
          count(w[j] >> 16, seg);
        }
      }
      __syncthreads();
      for (int n = warp; n < nb; n += SM_WARPS) {
        const uint32_t bin = sm.draw_bin[n];
        if (bin == 0xFFFFFFFFu) continue;
        const uint32_t col = sm.hist[sample_bin_slot(static_cast<int>(bin))] & 63u;
        const SampleMatch mt(sample_bin_bits(static_cast<int>(bin)));
        uint32_t rank = sm.draw_rank[n];
        int id = sample_scan_few(sp, mt, 0, sp.head, rank);
        if (id < 0) {
          // lane l: parts 4 l .. 4 l + 3
          uint32_t c[4], sum = 0;
          for (int k = 0; k < 4; ++k) {
            c[k] = (sm.segs[4 * lane + k][col >> 1] >> ((col & 1u) * 16u)) & 0xFFFFu;
            sum += c[k];
          }
          const uint32_t upto = warp_scan(sum);
          const uint32_t hit = __ballot_sync(0xffffffffu, upto > rank);
          if (hit == 0) {
            rank -= __shfl_sync(0xffffffffu, upto, 31);
            id = sample_scan_few(sp, mt, sp.tail_at(), sp.tail, rank);
          } else {
            const int l = __ffs(hit) - 1;
            uint32_t left = rank - (upto - sum);
            int seg = 4 * lane;
            for (int k = 0; k < 3 && left >= c[k]; ++k) {
              left -= c[k];
              ++seg;
            }
            left = __shfl_sync(0xffffffffu, left, l);
            seg = __shfl_sync(0xffffffffu, seg, l);
            id = sample_scan(sp, mt, seg * seg_vecs, min(sp.nvec, (seg + 1) * seg_vecs), left);
          }
        }
        if (lane == 0) p.ids[row * p.N + n0 + n] = id;
      }
      __syncthreads();
      if (at) *at = kept;
    }
  }
}

}  // namespace ckl
