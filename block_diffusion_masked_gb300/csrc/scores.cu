// Scores of tokens from logits: log probability of a given token, entropy of the
// distribution, the likeliest alternatives, and the gradient of the first two.
//
// Mathematics.  For a row x of V logits, m = max x, S = sum_j exp(x_j - m):
//   log p_j  = x_j - m - ln S
//   entropy  = -sum_j p_j log p_j = ln S - (sum_j exp(x_j - m) (x_j - m)) / S
//   d(log p_t) / dx_j    = [j = t] - p_j
//   d(entropy) / dx_j    = -p_j (log p_j + entropy).
// Everything is taken relative to m, so that nothing cancels where the logits are
// large against their spread; sums are float32 (a thread's own, then a tree).  A
// logit of -inf is a token that cannot be: it counts for nothing.
//
// The alternatives are those of the largest keys: a logit's bits, ordered as
// unsigned integers (-0 as 0), above the complement of its index, so that equal
// logits come lowest index first and no two keys are equal.
//
// Bound by memory: one pass over the logits, 16 bytes a thread and access, two or three of
// them on their way while as many are summed (some 8 operations a logit with the entropy,
// which all rows have).  Measured: 8192 rows of 50001 bf16 logits (819 MB) 140 us, 5.9 TB/s,
// their gradient 194 us where half of the rows have a token (the others' logits are not read:
// 1.23 GB), 256 us where all have (1.64 GB, 6.4 TB/s), 274 us for 50257 logits cut out of rows
// of 50304, which do not lie in their vectors as the gradient does (contiguous ones 257); 511
// rows of 131001 float32 logits (268 MB) with 32 alternatives 55.7 us, 4.8 TB/s; 20 rows of
// 32768 with 8 9.6 us, two launches' latency.  Tried and slower, in place of the registers that
// hold the next vectors: a ring in shared memory filled by asynchronous copies (148 us against
// 140); sums two to an operation (237: the pairs have to be put together).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "device.cuh"
#include "dfa.h"
#include "params.cuh"
#include "sm100.cuh"

namespace dfa {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;  // of the kernel that reads the logits, 64 registers a thread
constexpr int kMaxTop = 32;
constexpr int kMaxSplits = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A logit this far below the maximum, in powers of two, has probability 0 in float32;
// what is further, -inf too, is taken as this far, for 0 * inf is not a number.
constexpr float kFar = -220.f;
// Up to this magnitude of the maximum, m log2 e is rounded by 1/4 at most (extreme(), below).
constexpr float kFirst = 0x1p22f;

// ------------------------------------------------------------------ rows of logits

template <typename T>
struct Logit;
template <>
struct Logit<__nv_bfloat16> {
  static constexpr int kPer = 8;  // values of a 16-byte vector
  static constexpr uint32_t kNone = 0xff80ff80u;
  __device__ static void unpack(const uint4& w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  // Values no lower than one whose product with log2 e is finite (a NaN stays), two to an
  // operation.
  __device__ static uint4 finite(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w}, low = 0xff00ff00u;  // -2^127
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 x = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&u[i]),
                                           *reinterpret_cast<const __nv_bfloat162*>(&low));
      y[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
  }
  // Whether what finite() replaces, and whatever else is far, is out of m's reach, and m
  // itself not extreme.
  __device__ static bool plain(float m) { return fabsf(m) <= kFirst; }
  // The largest of m and N vectors' values.
  template <int N>
  __device__ static float most(float m, const uint4* w) {
    __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[0].x);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const uint32_t v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x = __hmax2(x, *reinterpret_cast<const __nv_bfloat162*>(&v[i]));
    }
    return fmax3(m, __low2float(x), __high2float(x));
  }
  __device__ static float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  __device__ static __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Logit<__half> {
  static constexpr int kPer = 8;
  static constexpr uint32_t kNone = 0xfc00fc00u;
  __device__ static void unpack(const uint4& w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = y.x, f[2 * i + 1] = y.y;
    }
  }
  __device__ static uint4 pack(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 y = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ static uint4 finite(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w}, low = 0xfbfffbffu;
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 x = __hmax2_nan(*reinterpret_cast<const __half2*>(&u[i]),
                                    *reinterpret_cast<const __half2*>(&low));
      y[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
  }
  __device__ static bool plain(float m) { return m > -60000.f && m < INFINITY; }
  template <int N>
  __device__ static float most(float m, const uint4* w) {
    __half2 x = *reinterpret_cast<const __half2*>(&w[0].x);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const uint32_t v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x = __hmax2(x, *reinterpret_cast<const __half2*>(&v[i]));
    }
    return fmax3(m, __low2float(x), __high2float(x));
  }
  __device__ static float get(__half x) { return __half2float(x); }
  __device__ static __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Logit<float> {
  static constexpr int kPer = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  __device__ static void unpack(const uint4& w, float* f) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  __device__ static uint4 finite(const uint4& w) { return w; }
  __device__ static bool plain(float m) { return fabsf(m) <= kFirst; }
  template <int N>
  __device__ static float most(float m, const uint4* w) {
#pragma unroll
    for (int u = 0; u < N; ++u)
      m = fmax3(fmax3(m, __uint_as_float(w[u].x), __uint_as_float(w[u].y)),
                __uint_as_float(w[u].z), __uint_as_float(w[u].w));
    return m;
  }
  __device__ static float get(float x) { return x; }
  __device__ static float put(float x) { return x; }
};

// A row as 16-byte vectors of the memory it lies in: vector v holds the row's
// values v * kPer - lead ..., of which the first and the last vector may hold some
// only.  Those are read value by value, so that nothing outside the row is read.
// Ordinary loads, not those of the read-only path: a block may be there while the kernel
// before it still writes the logits.
template <typename T>
struct Row {
  static constexpr int kPer = Logit<T>::kPer;
  const T* x;
  int vocab, lead, vectors;
  __device__ Row(const T* at, int v) : x(at), vocab(v) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(at) & 15) / sizeof(T));
    vectors = (lead + vocab + kPer - 1) / kPer;
  }
  __device__ __forceinline__ uint4 load(int v, int end) const {
    constexpr uint32_t none = Logit<T>::kNone;
    uint4 w = make_uint4(none, none, none, none);
    if (v >= end) return w;
    const int e0 = v * kPer - lead;
    if (e0 >= 0 && e0 + kPer <= vocab) return *reinterpret_cast<const uint4*>(x + e0);
    alignas(16) T part[kPer];
    *reinterpret_cast<uint4*>(part) = w;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e0 + i >= 0 && e0 + i < vocab) part[i] = x[e0 + i];
    return *reinterpret_cast<const uint4*>(part);
  }
};

// Vectors that are read once, past the first-level cache: 140 us for 8192 rows of 50001 bf16
// logits, 143 without the hint; 511 rows of 131001 float32 with alternatives 55.7 and 57.4.
// (The gradient loses with it: 205 and 195.)
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// max(x, kFar), NaN kept.
__device__ __forceinline__ float not_far(float x) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(kFar));
  return x;
}

// Running statistics of a softmax: the maximum m, and against its reference r = m log2 e,
// rounded, with z = x log2 e - r, the sum s of 2^z and the sum t of 2^z z.  A z is one
// operation, rounded once, relative to itself; what the rounding of r adds to all of them
// is taken off at the end (finish).  Nothing yet: m -inf, s and t 0.
struct Stats {
  float m, s, t;
};
// Past kFirst z is (x - m) log2 e in its place: what the rounding of r adds to all of them
// grows with m, and past 2^32 it alone would take a 2^z to infinity or to 0.
__device__ __forceinline__ bool extreme(float m) { return fabsf(m) > kFirst && m != -INFINITY; }
// (__fmul_rn: the rounding is to be the same wherever r appears, so the product is not to be
// drawn into a sum.)
__device__ __forceinline__ float reference(float m) {
  return m == -INFINITY ? 0.f : __fmul_rn(m, kLog2e);
}
// What every z against m is too large by, for r is too small by it; at most 1/4.
__device__ __forceinline__ float excess(float m) {
  return extreme(m) || m == -INFINITY ? 0.f : fmaf(m, kLog2e, -reference(m));
}
// a against the maximum m >= a.m.
__device__ __forceinline__ Stats rebase(const Stats& a, float m) {
  if (a.m == -INFINITY) return {m, a.s, a.t};  // nothing yet, or not a number
  const float d = not_far(extreme(a.m) || extreme(m)
                              ? (a.m - m) * kLog2e + (excess(m) - excess(a.m))
                              : reference(a.m) - reference(m));
  const float f = ex2_approx(d);
  return {m, a.s * f, f * fmaf(a.s, d, a.t)};
}
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b) {
  const float m = fmaxf(a.m, b.m);
  const Stats x = rebase(a, m), y = rebase(b, m);
  return {m, x.s + y.s, x.t + y.t};
}
__device__ __forceinline__ Stats warp_join(Stats a) {
  float m = a.m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  a = rebase(a, m);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, off);
    a.t += __shfl_xor_sync(0xffffffffu, a.t, off);
  }
  return a;
}

// ------------------------------------------------------------------ keys

using Key = unsigned long long;

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kOrderedNone = 0x007fffffu;  // of -inf: no alternative
__device__ __forceinline__ Key make_key(float x, int index) {
  return static_cast<Key>(ordered(x)) << 32 | static_cast<uint32_t>(~index);
}
// The largest of the warp's keys (0: none).
__device__ __forceinline__ Key warp_max(Key k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
  const uint32_t lo = __reduce_max_sync(
      0xffffffffu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return static_cast<Key>(hi) << 32 | lo;
}

struct ScoresParams {
  const void* x;       // (rows, vocab), rows `stride` values apart
  const void* tokens;  // (rows) or null
  long long stride;
  float* logprobs;      // (rows) or null
  float* entropy;       // (rows)
  float* stats;         // (rows, 2): m, ln S
  float* top_logprobs;  // (rows, top)
  int* top_tokens;
  Stats* part;    // (rows, splits): of a split row's pieces
  Key* part_top;  // (rows, splits, top)
  unsigned* status;
  int rows, vocab, top, splits;
  bool wide_tokens;  // 64 bits
};

// What every thread needs of a finished row.
struct Finished {
  float m, log_s, entropy;
  bool none, nan;  // no token can be (every logit -inf); a logit is not a number
};
__device__ __forceinline__ Finished finish(const Stats& a) {
  Finished f;
  f.none = a.m == -INFINITY && a.s == 0.f;
  f.nan = !f.none && !(a.s < INFINITY);
  f.m = f.nan ? NAN : a.m;
  const float off = f.none || f.nan ? 0.f : excess(a.m);
  const float log2_s = lg2_approx(a.s) - off;
  f.log_s = f.none ? 0.f : f.nan ? NAN : log2_s * kLn2;
  f.entropy = f.none ? 0.f : f.nan ? NAN : fmaxf((log2_s - (a.t / a.s - off)) * kLn2, 0.f);
  return f;
}
// The row's token and its logit.
struct Token {
  int index;  // -1: none
  float logit;
};
template <typename T>
__device__ __forceinline__ Token load_token(const ScoresParams& p, int row) {
  Token t = {-1, 0.f};
  if (p.tokens == nullptr) return t;
  const long long i = p.wide_tokens ? static_cast<const long long*>(p.tokens)[row]
                                    : static_cast<const int*>(p.tokens)[row];
  if (i >= p.vocab) atomicOr(p.status, kStatusIndex);
  if (i >= 0 && i < p.vocab) {
    t.index = static_cast<int>(i);
    t.logit = Logit<T>::get((static_cast<const T*>(p.x) + row * p.stride)[t.index]);
  }
  return t;
}
// One thread writes the row's numbers.
__device__ __forceinline__ void write_row(const ScoresParams& p, int row, const Finished& f,
                                          const Token& t) {
  p.entropy[row] = f.entropy;
  *reinterpret_cast<float2*>(p.stats + 2LL * row) = make_float2(f.m, f.log_s);
  if (p.logprobs == nullptr) return;
  p.logprobs[row] = t.index < 0 ? 0.f : f.none ? -INFINITY : (t.logit - f.m) - f.log_s;
}
// Alternative i of a row, of its key (0: there is none).
__device__ __forceinline__ void write_top(const ScoresParams& p, int row, int i, Key key,
                                          const Finished& f) {
  const uint32_t order = static_cast<uint32_t>(key >> 32);
  const bool is = order > kOrderedNone && !f.nan;
  const long long at = static_cast<long long>(row) * p.top + i;
  p.top_logprobs[at] = f.nan ? NAN : is ? (unordered(order) - f.m) - f.log_s : -INFINITY;
  p.top_tokens[at] = is ? static_cast<int>(~static_cast<uint32_t>(key)) : -1;
}

// ------------------------------------------------------------------ forward

// Alternatives are gathered in shared memory, in a list.  Where there may be more than it
// has room for, some threads add a vector each and it is cut down between such rounds.
constexpr int kListThreads = 64;          // that add to it in a round
constexpr int kListMost = kListThreads * 8;
constexpr int kListKeep = 512;            // a longer list is cut down between rounds
constexpr int kListMore = 16;             // the two vectors that are not whole
constexpr int kList = kListKeep + kListMost + kListMore;
constexpr int kSlots = 32;
struct TopSpace {
  Key list[kList];
  Key best[kMaxTop];
  float slot[kSlots][kThreads];  // the largest logit of every run of a thread's batches
  uint32_t top[kThreads];  // the threads' largest logits, ordered; each warp's sorted
  int hot[kThreads];       // threads that may have one of the alternatives
  int count, hots;
  uint32_t least;          // no alternative is below this (ordered)
};

// The larger of x and lane ^ mask's in the lanes that `up` says, the smaller in the others.
__device__ __forceinline__ uint32_t exchange(uint32_t x, int mask, bool up) {
  const uint32_t y = __shfl_xor_sync(0xffffffffu, x, mask);
  return up ? max(x, y) : min(x, y);
}
// The warp's values, the largest in lane 0: a bitonic sort.
__device__ __forceinline__ uint32_t warp_sorted(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int mask = size >> 1; mask > 0; mask >>= 1)
      x = exchange(x, mask, ((lane & mask) == 0) == ((lane & size) == 0));
  return x;
}
// The 32 largest of the warp's and of another sorted 32, sorted.
__device__ __forceinline__ uint32_t warp_merged(uint32_t x, const uint32_t* other) {
  const int lane = threadIdx.x & 31;
  x = max(x, other[31 - lane]);  // rises, then falls
#pragma unroll
  for (int mask = 16; mask > 0; mask >>= 1) x = exchange(x, mask, (lane & mask) == 0);
  return x;
}

// The `top` largest keys of the list, in order, into `best` (0 behind the last).
__device__ __forceinline__ void best_of_list(TopSpace& s, int top) {
  const int n = s.count;
  for (int i = threadIdx.x; i < top; i += kThreads)
    if (i >= n) s.best[i] = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key key = s.list[i];
    int above = 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 8) {
      Key other[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = j + e < n ? s.list[j + e] : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) above += other[e] > key;
    }
    if (above < top) s.best[above] = key;
  }
}

// A block takes rows, or pieces of rows, one after another: a thread walks vectors of a
// piece, the block's width apart, with statistics of its own against its own maximum, the
// next vectors on their way; one join at the piece's end, while the next piece's first
// vectors are.
//
// Alternatives: the block's `top` largest logits are not below the top-th largest of the
// threads' largest.  The threads have noted the largest logit of each of up to 32 runs of
// their vectors; those of the few runs that reach that bound are read again, and what is
// not below it goes to a list.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    dfa_scores_kernel(const ScoresParams p) {
  using L = Logit<T>;
  constexpr int kPer = L::kPer, kAhead = TOP ? 2 : 3;
  __shared__ Stats s_warp[kThreads / 32];
  extern __shared__ uint4 smem[];
  TopSpace& space = *reinterpret_cast<TopSpace*>(smem);  // with TOP
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = p.rows * p.splits;
  // A thread's vectors of a piece: whole ones, `step` apart, batches of kAhead and the rest;
  // the piece's first or last vector, where the row holds some of its values only, is one
  // more, of the block's first or last thread.
  struct Piece {
    int row, lo, hi;   // vectors [lo, hi)
    int at, end;       // the thread's first whole one, one past the piece's last
    bool ragged;       // the thread has a vector that is not whole: v
    int v;
  };
  auto row_of = [&](int row) {
    return Row<T>(static_cast<const T*>(p.x) + row * p.stride, p.vocab);
  };
  auto enter = [&](int item) {
    Piece c;
    c.row = item / p.splits;
    const Row<T> r = row_of(c.row);
    const int per = (r.vectors + p.splits - 1) / p.splits;
    c.lo = min((item - c.row * p.splits) * per, r.vectors), c.hi = min(c.lo + per, r.vectors);
    const bool head = c.lo == 0 && (r.lead > 0 || r.vocab < kPer);
    const bool tail = c.hi == r.vectors && (r.lead + r.vocab) % kPer != 0 && c.hi - c.lo > head;
    c.at = c.lo + head + tid, c.end = c.hi - tail;
    c.ragged = (head && tid == 0) || (tail && tid == kThreads - 1);
    c.v = tid == 0 ? c.lo : c.hi - 1;
    return c;
  };
  // The first batch of a piece (a batch is whole or not loaded).
  auto load = [&](const uint4* x, int v, int end, uint4 (&w)[kAhead]) {
    if (v + (kAhead - 1) * kThreads < end) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) w[u] = load_stream(x + v + u * kThreads);
    }
  };
  auto vectors_of = [&](const Row<T>& r) {
    return reinterpret_cast<const uint4*>(r.x - r.lead);
  };
  uint4 w[kAhead];
  Piece c = {};
  if (static_cast<int>(blockIdx.x) < items) {
    c = enter(blockIdx.x);
    load(vectors_of(row_of(c.row)), c.at, c.end, w);
  }
#pragma unroll 1
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    Stats a = {-INFINITY, 0.f, 0.f};
    float run = -INFINITY;  // the largest logit of the run of batches
    // N vectors against the maximum so far.
    auto take = [&](auto count, const uint4* x) {
      constexpr int N = decltype(count)::value;
      const float m = fmaxf(a.m, run = L::template most<N>(run, x));
      if (m > a.m) a = rebase(a, m);
      if (L::plain(m)) {
        const float ref = -reference(m);
        float s1 = 0.f, t1 = 0.f;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          float f[kPer];
          L::unpack(L::finite(x[u]), f);
#pragma unroll
          for (int i = 0; i < kPer; i += 2) {
            float z0 = fmaf(f[i], kLog2e, ref), z1 = fmaf(f[i + 1], kLog2e, ref);
            if constexpr (sizeof(T) == 4) z0 = not_far(z0), z1 = not_far(z1);
            const float e0 = ex2_approx(z0), e1 = ex2_approx(z1);
            a.s += e0, s1 += e1;
            a.t = fmaf(e0, z0, a.t), t1 = fmaf(e1, z1, t1);
          }
        }
        a.s += s1, a.t += t1;
      } else {  // one by one, differences first unless there is nothing but -inf
#pragma unroll 1
        for (int u = 0; u < N; ++u) {
          float f[kPer];
          uint4 y = x[0];
#pragma unroll
          for (int i = 1; i < N; ++i)
            if (u == i) y = x[i];
          L::unpack(y, f);
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const float z = extreme(m) ? not_far((f[i] - m) * kLog2e)
                                       : not_far(fmaf(f[i], kLog2e, -reference(m)));
            const float e = ex2_approx(z);
            a.s += e;
            a.t = fmaf(e, z, a.t);
          }
        }
      }
    };
    const Row<T> r = row_of(c.row);
    const uint4* x = vectors_of(r);
    constexpr int kBatch = kAhead * kThreads;
    const int batches = (c.end - (c.at - tid) + kBatch - 1) / kBatch;  // of whole vectors
    const int per_slot = TOP ? (batches + kSlots - 1) / kSlots : 1;
    int slot = 0, in_slot = 0;
    auto note = [&](bool last) {  // a batch has been taken
      if constexpr (TOP) {
        if (++in_slot == per_slot || last) {
          space.slot[slot][tid] = run;
          ++slot, in_slot = 0;
          run = -INFINITY;
        }
      }
    };
    int v = c.at;
#pragma unroll 1
    for (; v + kBatch - kThreads < c.end; v += 2 * kBatch) {
      uint4 w2[kAhead];
      load(x, v + kBatch, c.end, w2);
      take(std::integral_constant<int, kAhead>{}, w);
      note(false);
      if (v + 2 * kBatch - kThreads >= c.end) {
        v += kBatch;
        break;
      }
      load(x, v + 2 * kBatch, c.end, w);
      take(std::integral_constant<int, kAhead>{}, w2);
      note(false);
    }
    {  // the rest: fewer than kAhead, and the one that is not whole
      uint4 rest[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead - 1; ++u)
        if (v + u * kThreads < c.end) rest[u] = x[v + u * kThreads];
      if (c.ragged) rest[kAhead - 1] = r.load(c.v, c.hi);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (u == kAhead - 1 && slot < kSlots) note(true);  // the rest is the last run's
        if (u < kAhead - 1 ? v + u * kThreads < c.end : c.ragged)
          take(std::integral_constant<int, 1>{}, rest + u);
      }
    }
    const float mine = a.m;
    const Piece c0 = c;  // the piece that is done
    if (item + static_cast<int>(gridDim.x) < items) {
      c = enter(item + gridDim.x);
      load(vectors_of(row_of(c.row)), c.at, c.end, w);
    }
    a = warp_join(a);
    if (lane == 0) s_warp[warp] = a;

    if constexpr (TOP) {
      TopSpace& s = space;
      if (tid == 0) s.count = s.hots = 0;
      // The bound: the top-th largest of the threads' largest.
      uint32_t most = warp_sorted(ordered(mine));
      s.top[tid] = most;
#pragma unroll
      for (int n = kThreads / 64; n > 0; n >>= 1) {  // warps below n take those n behind in
        __syncthreads();
        if (warp < n) {
          most = warp_merged(most, s.top + 32 * (warp + n));
          s.top[tid] = most;
        }
      }
      if (tid == p.top - 1) s.least = max(most, kOrderedNone + 1);
      __syncthreads();
      if (ordered(mine) >= s.least) s.hot[atomicAdd(&s.hots, 1)] = tid;
      __syncthreads();
      const int first = c0.at - tid;  // whole vectors of the piece: [first, c0.end)
      const int hots = s.hots, steps = (c0.end - first + kThreads - 1) / kThreads;
      const float least = unordered(s.least);
      Key bound = static_cast<Key>(s.least) << 32;  // below every key of that logit
      auto offer = [&](const uint4& x, int v) {
        float f[kPer];
        L::unpack(x, f);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (f[i] >= least) {
            const Key key = make_key(f[i], v * kPer - r.lead + i);
            if (key >= bound) {
              const int at = atomicAdd(&s.count, 1);
              if (at < kList) s.list[at] = key;
            }
          }
      };
      auto vector_of = [&](int q) {  // of the hot threads' whole vectors, in order
        const int step = q / hots;
        return first + step * kThreads + s.hot[q - step * hots];
      };
      const bool offers = c0.ragged && ordered(mine) >= s.least;
      if (offers) offer(r.load(c0.v, c0.hi), c0.v);
      // Of the hot threads the runs that reach the bound; then, where the list was too short,
      // all of their vectors in rounds.
      if (ordered(mine) >= s.least) {
        unsigned reach = 0;
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
          if (i < slot && space.slot[i][tid] >= least) reach |= 1u << i;
        for (; reach != 0; reach &= reach - 1) {
          const int i = __ffs(reach) - 1;
          for (int j = 0; j < per_slot; ++j) {
            const int v = first + tid + (i * per_slot + j) * kBatch;
            uint4 y[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
              if (v + u * kThreads < c0.end) y[u] = x[v + u * kThreads];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
              if (v + u * kThreads < c0.end) offer(y[u], v + u * kThreads);
          }
        }
      }
      __syncthreads();
      const bool again = s.count > kList;
      __syncthreads();  // the count has been read
      if (again) {
        if (tid == 0) s.count = 0;
        __syncthreads();
        if (offers) offer(r.load(c0.v, c0.hi), c0.v);
#pragma unroll 1
        for (int q0 = 0; q0 < hots * steps; q0 += kListThreads) {
          const int q = q0 + tid;
          const int v = tid < kListThreads && q < hots * steps ? vector_of(q) : c0.end;
          if (v < c0.end) offer(x[v], v);
          __syncthreads();
          const bool full = s.count > kListKeep;
          __syncthreads();  // the count has been read
          if (full) {
            best_of_list(s, p.top);
            __syncthreads();
            bound = s.best[p.top - 1];  // the list holds more than `top` keys
            if (tid < p.top) s.list[tid] = s.best[tid];
            if (tid == 0) s.count = p.top;
            __syncthreads();
          }
        }
      }
      best_of_list(s, p.top);
      __syncthreads();
      if (p.splits > 1) {
        if (tid < p.top)
          p.part_top[static_cast<long long>(item) * p.top + tid] = s.best[tid];
      }
    } else {
      __syncthreads();
    }
    if (warp == 0) {
      Stats b = lane < kThreads / 32 ? s_warp[lane] : Stats{-INFINITY, 0.f, 0.f};
      b = warp_join(b);
      if (p.splits > 1) {
        if (lane == 0) p.part[item] = b;
      } else {
        const Finished f = finish(b);
        if (lane == 0) write_row(p, c0.row, f, load_token<T>(p, c0.row));
        if constexpr (TOP) {
          if (lane < p.top) write_top(p, c0.row, lane, space.best[lane], f);
        }
      }
    }
    __syncthreads();  // the statistics and the list have been read
  }
}

// The pieces of split rows, a warp a row: statistics joined, then the alternatives
// one at a time, each lane at the head of its pieces' lists.
constexpr int kJoinRows = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinRows) dfa_scores_join_kernel(const ScoresParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, row = blockIdx.x * kJoinRows + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  constexpr int kLists = kMaxSplits / 32;
  Token token;
  if (lane == 0) token = load_token<T>(p, row);
  const long long first = static_cast<long long>(row) * p.splits;
  Stats a = {-INFINITY, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kLists; ++i)
    if (lane + 32 * i < p.splits) a = join(a, p.part[first + lane + 32 * i]);
  a = warp_join(a);
  const Finished f = finish(a);
  if (lane == 0) write_row(p, row, f, token);
  if (p.top == 0) return;
  const Key* lists = p.part_top + first * p.top;
  Key head[kLists];
  int at[kLists];
#pragma unroll
  for (int i = 0; i < kLists; ++i) {
    at[i] = 0;
    head[i] = lane + 32 * i < p.splits ? lists[(lane + 32 * i) * p.top] : 0;
  }
  Key mine = 0;
  for (int n = 0; n < p.top; ++n) {
    Key k = 0;
#pragma unroll
    for (int i = 0; i < kLists; ++i) k = max(k, head[i]);
    const Key best = warp_max(k);
    if (lane == n) mine = best;
#pragma unroll
    for (int i = 0; i < kLists; ++i)
      if (best != 0 && head[i] == best)
        head[i] = ++at[i] < p.top ? lists[(lane + 32 * i) * p.top + at[i]] : 0;
  }
  if (lane < p.top) write_top(p, row, lane, mine, f);
}

// ------------------------------------------------------------------ backward

struct ScoresGradParams {
  const void* x;
  const void* tokens;
  long long stride;
  const float* stats;
  const float* entropy;
  const float* dlogprobs;  // (rows) or null
  const float* dentropy;   // (rows) or null
  void* dx;                // (rows, vocab) contiguous
  int rows, vocab, splits;
  bool wide_tokens;
};

// dx_j = g ([j = t] - p_j) - h p_j (log p_j + entropy), for the gradients g of the
// row's log probability and h of its entropy: one pass, logits in, gradient out,
// vectors of the gradient's memory.  A row of zero gradients, or where no token can
// be, is set to zero and not read.
template <typename T>
__global__ void __launch_bounds__(kThreads) dfa_scores_grad_kernel(const ScoresGradParams p) {
  using L = Logit<T>;
  constexpr int kPer = L::kPer;
  grid_launch_dependents();
  grid_dependency_wait();
  const int row = blockIdx.x / p.splits, piece = blockIdx.x - row * p.splits;
  const T* x = static_cast<const T*>(p.x) + row * p.stride;
  T* dx = static_cast<T*>(p.dx) + static_cast<long long>(row) * p.vocab;
  const Row<T> r(dx, p.vocab);
  const int per = (r.vectors + p.splits - 1) / p.splits;
  const int lo = min(piece * per, r.vectors), hi = min(lo + per, r.vectors);
  const float2 st = *reinterpret_cast<const float2*>(p.stats + 2LL * row);
  const float ent = p.dentropy ? p.entropy[row] : 0.f;
  const float h = p.dentropy ? p.dentropy[row] : 0.f;
  int token = -1;
  if (p.tokens != nullptr) {
    const long long t = p.wide_tokens ? static_cast<const long long*>(p.tokens)[row]
                                      : static_cast<const int*>(p.tokens)[row];
    token = t >= 0 && t < p.vocab ? static_cast<int>(t) : -1;
  }
  const float g = p.dlogprobs && token >= 0 ? p.dlogprobs[row] : 0.f;
  const bool zero = (g == 0.f && h == 0.f) || st.x == -INFINITY;
  // whether the logits lie in their vectors as the gradient does in its own
  const bool aligned =
      (reinterpret_cast<uintptr_t>(x) & 15) == (reinterpret_cast<uintptr_t>(dx) & 15);
  const float base = fmaf(h, ent, g);  // dx_j = -p_j (g + h (log p_j + ent))
  for (int v = lo + threadIdx.x; v < hi; v += kThreads) {
    const int e0 = v * kPer - r.lead;
    const bool whole = e0 >= 0 && e0 + kPer <= p.vocab;
    float f[kPer];
    if (zero) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) f[i] = 0.f;
    } else {
      if (whole && aligned) {
        L::unpack(*reinterpret_cast<const uint4*>(x + e0), f);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          f[i] = e0 + i >= 0 && e0 + i < p.vocab ? L::get(x[e0 + i]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float lp = not_far((f[i] - st.x) - st.y);
        f[i] = -ex2_approx(lp * kLog2e) * fmaf(h, lp, base);
      }
      if (token >= e0 && token < e0 + kPer) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (e0 + i == token) f[i] += g;
      }
    }
    if (whole) {
      *reinterpret_cast<uint4*>(dx + e0) = L::pack(f);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (e0 + i >= 0 && e0 + i < p.vocab) dx[e0 + i] = L::put(f[i]);
    }
  }
}

// ------------------------------------------------------------------ host

// Pieces of a row: enough that the blocks fill the device once, at least two
// vectors a thread, and such that the last wave is not mostly empty.
int splits_for(int rows, int vocab, int size, int top, int sms) {
  const long long vectors = (static_cast<long long>(vocab) * size + 15) / 16;
  const long long most = vectors / (2 * kThreads);
  const long long slots = static_cast<long long>(sms) * kBlocksPerSm;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= kMaxSplits && (s == 1 || s <= most); ++s) {
    const long long waves = (static_cast<long long>(rows) * s + slots - 1) / slots;
    // a piece's end costs as much as about two vectors a thread, alternatives some more
    const double cost =
        static_cast<double>(waves) * (static_cast<double>(vectors) / s + (top ? 4 : 2) * kThreads);
    if (s == 1 || cost < 0.97 * least) best = s, least = cost;
  }
  return best;
}

int type_size(int dtype) {
  return dtype == DFA_BF16 || dtype == DFA_F16 ? 2 : dtype == DFA_F32 ? 4 : 0;
}

int check_scores(const void* logits, const void* tokens, int token_bytes, int rows, int vocab,
                 long long stride, int dtype) {
  if (rows < 0 || rows > (1 << 24) || vocab < 1 || vocab > (1 << 30) || !type_size(dtype))
    return DFA_EINVAL;
  if (tokens && token_bytes != 4 && token_bytes != 8) return DFA_EINVAL;
  if (rows == 0) return DFA_OK;
  auto aligned = [](const void* x, unsigned n) {
    return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0;
  };
  if (!logits || !aligned(logits, type_size(dtype)) ||
      (tokens && !aligned(tokens, static_cast<unsigned>(token_bytes))) || stride < 0 ||
      stride > (1LL << 40))
    return DFA_EINVAL;
  return DFA_OK;
}

long long scores_workspace(int rows, int top, int splits) {
  if (splits == 1) return 0;
  const long long pieces = static_cast<long long>(rows) * splits;
  return pieces * top * static_cast<long long>(sizeof(Key)) +
         pieces * static_cast<long long>(sizeof(Stats));
}

template <typename T>
cudaError_t launch_scores(const ScoresParams& p, int sms, cudaStream_t stream) {
  auto kern = p.top > 0 ? dfa_scores_kernel<T, true> : dfa_scores_kernel<T, false>;
  const long long items = static_cast<long long>(p.rows) * p.splits;
  const long long most = static_cast<long long>(sms) * kBlocksPerSm;
  const unsigned blocks = static_cast<unsigned>(items < most ? items : most);
  const size_t smem = p.top > 0 ? sizeof(TopSpace) : 0;
  cudaError_t e = smem ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(smem))
                       : cudaSuccess;
  if (e == cudaSuccess) e = launch_chained(kern, dim3(blocks), dim3(kThreads), smem, stream, p);
  if (e == cudaSuccess && p.splits > 1)
    e = launch_chained(dfa_scores_join_kernel<T>,
                       dim3((static_cast<unsigned>(p.rows) + kJoinRows - 1) / kJoinRows),
                       dim3(32 * kJoinRows), 0, stream, p);
  return e;
}

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" {

long long dfa_token_logprobs_workspace_bytes(int rows, int vocab, int top, int dtype) {
  if (rows < 0 || rows > (1 << 24) || vocab < 1 || vocab > (1 << 30) || !type_size(dtype) ||
      top < 0 || top > kMaxTop)
    return DFA_EINVAL;
  if (rows == 0) return 0;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  return scores_workspace(rows, top, splits_for(rows, vocab, type_size(dtype), top, di.sms));
}

int dfa_token_logprobs(const void* logits, const void* tokens, int token_bytes, float* logprobs,
                       float* entropy, float* stats, float* top_logprobs, int* top_tokens,
                       void* workspace, long long workspace_bytes, int rows, int vocab, int top,
                       long long stride, int dtype, dfa_stream_t stream) {
  if (top < 0 || top > kMaxTop) return DFA_EINVAL;
  if (const int rc = check_scores(logits, tokens, token_bytes, rows, vocab, stride, dtype))
    return rc;
  if (rows == 0) return DFA_OK;
  auto aligned = [](const void* x, unsigned n) {
    return x && (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0;
  };
  if (!aligned(entropy, 4) || !aligned(stats, 8) || (tokens && !logprobs) ||
      (logprobs && !aligned(logprobs, 4)) ||
      (top && (!aligned(top_logprobs, 4) || !aligned(top_tokens, 4))) ||
      (workspace && !aligned(workspace, 8)))
    return DFA_EINVAL;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  const int splits = splits_for(rows, vocab, type_size(dtype), top, di.sms);
  const long long need = scores_workspace(rows, top, splits);
  if (need && (!workspace || workspace_bytes < need)) return DFA_EINVAL;
  ScoresParams p{};
  p.x = logits;
  p.tokens = tokens;
  p.stride = stride;
  p.logprobs = logprobs;
  p.entropy = entropy;
  p.stats = stats;
  p.top_logprobs = top_logprobs;
  p.top_tokens = top_tokens;
  p.part_top = static_cast<Key*>(workspace);
  p.part = reinterpret_cast<Stats*>(p.part_top + static_cast<long long>(rows) * splits * top);
  p.status = di.status;
  p.rows = rows;
  p.vocab = vocab;
  p.top = top;
  p.splits = splits;
  p.wide_tokens = token_bytes == 8;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DFA_BF16  ? launch_scores<__nv_bfloat16>(p, di.sms, s)
                        : dtype == DFA_F16 ? launch_scores<__half>(p, di.sms, s)
                                           : launch_scores<float>(p, di.sms, s);
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

int dfa_token_logprobs_backward(const void* logits, const void* tokens, int token_bytes,
                                const float* stats, const float* entropy, const float* dlogprobs,
                                const float* dentropy, void* dlogits, int rows, int vocab,
                                long long stride, int dtype, dfa_stream_t stream) {
  if (const int rc = check_scores(logits, tokens, token_bytes, rows, vocab, stride, dtype))
    return rc;
  if (rows == 0) return DFA_OK;
  auto aligned = [](const void* x, unsigned n) {
    return x && (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0;
  };
  if (!aligned(stats, 8) || !aligned(dlogits, 16) || (dentropy && !aligned(dentropy, 4)) ||
      (dentropy && !aligned(entropy, 4)) || (dlogprobs && !aligned(dlogprobs, 4)))
    return DFA_EINVAL;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  ScoresGradParams p{};
  p.x = logits;
  p.tokens = tokens;
  p.stride = stride;
  p.stats = stats;
  p.entropy = entropy;
  p.dlogprobs = dlogprobs;
  p.dentropy = dentropy;
  p.dx = dlogits;
  p.rows = rows;
  p.vocab = vocab;
  p.splits = splits_for(rows, vocab, type_size(dtype), 0, di.sms);
  p.wide_tokens = token_bytes == 8;
  const unsigned blocks = static_cast<unsigned>(rows) * static_cast<unsigned>(p.splits);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto kern = dtype == DFA_BF16  ? dfa_scores_grad_kernel<__nv_bfloat16>
              : dtype == DFA_F16 ? dfa_scores_grad_kernel<__half>
                                 : dfa_scores_grad_kernel<float>;
  const cudaError_t e = launch_chained(kern, dim3(blocks), dim3(kThreads), 0, s, p);
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

}  // extern "C"
