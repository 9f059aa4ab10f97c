// Attention of new rows over a paged 4-bit key/value cache (cache4.cuh) and, optionally,
// over the new rows' own keys and values in bf16, for few rows to a key and for headdim 256
// (many: cache_wide.cuh): one block of a block diffusion sampler against the clean tokens
// before it ("Fast Diffusion Attention", "Block diffusion in one picture").
//
// Mathematics.  Row i of request b (position len_b + i) and query head h see the len_b
// cached tokens and the own rows of its block or earlier blocks:
//   s_j = scale * q . k_j,  out = sum_j softmax(s)_j v_j,  lse = ln sum_j exp(s_j),
// cached k_j = (n_j - 8) s(j, group of 32 dims), v_j alike.
//
// Everything is transposed, for a tensor-core product has 16 rows on its one side and 8
// on the other, and the 8 are enough for many a step's queries: scores are K Q^T, 16
// keys by 8 query rows, the output V^T P^T, 16 head dims by 8 rows; the probabilities
// are turned from the one's result to the other's operand by a transposing move.
//
// Keys.  Four bits of a word, masked out where they stand, are a subnormal f16: n 2^-24
// or n 2^-20, so that two of a half word's codes cost an AND each and the next two a
// shift more; the queries make up for the powers of two.  The scores of a group of 32
// dims are two products, begun at -8 times the sum of the group's queries (a product of
// its own, once per piece) and added up in float32 times the keys' scales: 5 operations
// for eight codes and one per group and score instead of the 9 that decoding takes.
// q is bf16: a row is brought to f16 by a power of two of its own (its largest magnitude
// lands in [2^15, 2^16), below f16's largest as bf16 has 8 bits), which keeps every value
// down to 2^-28 of the row's largest exact.  The codes' 2^24 is undone in two parts, 2^6 by
// the keys' scales, the rest by the row's factor, for the whole does not fit the factor of
// a row near bf16's largest.
//
// Values.  cache4_decode, with the scales of the two keys of a pair; the probabilities
// are rounded to f16 (2^-11) while the sums use them unrounded.  Own keys and values are
// bf16 products, their probabilities bf16 (2^-8).  The reference of a row's exponentials
// moves only where a unit's probabilities outgrow f16 (cache_fwd.cuh).
//
// Work.  Segments (request, key/value head, tile of rows) are dealt to the blocks in
// equal runs of 128-key units (cache.cuh).  A block's four warps take the 32-key units of
// a piece in turn, each with a ring of stages of its own, filled by asynchronous copies
// that run ahead over the pieces' ends, and with softmax statistics of its own: no warp
// waits for another but at a piece's end, where they join through shared memory.  The
// pieces of a cut segment are joined by a second launch.
//
// Measured (headdim 128, 8 heads for keys): 64 ragged requests of up to 16000 tokens, 4 rows
// to a key, 689 MB: 180 us, 3.8 TB/s, against 102 us for the bytes; 24 of up to 8000, 16
// rows, 126 MB: 57 us against 18.5; one request of 500 tokens, 4 heads: 10.1 us, launches
// and latency.  Bound by the decoding: a unit is some 770 instructions of a warp, and the
// schedulers issue in 70% of the cycles while all warps have work (a copy of the kernel that
// only loads moves 6.5 TB/s).  Ends of pieces cost a block some 10000 cycles (requests'
// sizes, queries, own keys, join: one latency after another), which is what the shorter
// requests pay for.
#include <type_traits>

#include "cache4.cuh"
#include "cache_fwd.cuh"

namespace dfa {
namespace {

constexpr int kUnit = 32;  // keys a warp takes at a time

// D (16 x 8, float32) = A (16 x 16) B (16 x 8) + C.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, const uint32_t* b,
                                        const float* c) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, const uint32_t* b) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// Four 8 x 8 matrices of 16-bit elements, the addresses of their rows (16 bytes each) in
// the lanes 8 i ..: lane 4 g + t receives elements 2t, 2t + 1 of row g of each.
__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t* w) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
// An 8 x 8 matrix of 16-bit elements, a row's pair in each lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ T lds(uint32_t addr) {
  T v;
  if constexpr (sizeof(T) == 8) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  } else if constexpr (sizeof(T) == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  } else {
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  }
  return v;
}

// The reference of a row's exponentials is rounded, and a score less it (one operation) is
// not: past 2^27 that alone could put a probability out of f16's range, past 2^32 out of
// float32's, or all of a row's at 0.  So the reference is rounded down, which leaves the
// largest score's exponent at kShift or above, and exponents are cut here, above what
// kMostSum notices and below f16's limit.  Scores that are cut are the largest to within
// their own rounding.  A NaN stays one.  (1 us of 180 for 64 requests of 4 rows.)
constexpr float kMostExponent = 15.5f;
__device__ __forceinline__ float cut_exponent(float x) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(kMostExponent));
  return x;
}

__device__ __forceinline__ void sts(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

// 16 bytes of global memory into shared memory; zeros instead where !there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_end_group() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // until all but the last N groups are there
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// NT tiles of 8 query rows; WK warps, RESIDENT blocks per SM; STAGES units on their way to
// a warp; KEPT outputs kept at the join, to which the other warps add theirs.
template <int D, int NT, int WK, int STAGES, int RESIDENT, int KEPT>
struct Cache4Tile {
  static constexpr int kThreads = 32 * WK;
  static constexpr int kResident = RESIDENT;
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = kUnit * D / 2;  // bytes of a unit's k, and of its v
  static constexpr int kScales = D;            // and of either's scales, a group after another
  static constexpr int kPitch = D + 4;         // floats per row of a warp's output at the join
  static constexpr int kJoin = KEPT * kRows * kPitch * 4;
  static constexpr int kBeginAt = NT * (D / 16) * 32 * 8;  // behind the query fragments
  static constexpr int kQ = kBeginAt + NT * (D / 32) * 32 * 8;
  // rings (1024-byte aligned): k, v of each stage | scales | join, before it the query
  // fragments | statistics | valid keys
  static constexpr int kOffScale = WK * STAGES * 2 * kTile;
  static constexpr int kOffJoin = kOffScale + WK * STAGES * 2 * kScales;
  static constexpr int kOffStat = kOffJoin + (kJoin > kQ ? kJoin : kQ);
  static constexpr int kOffC = kOffStat + WK * kRows * 8;
  static constexpr int kOffKeys = kOffC + WK * 4;
  static constexpr int kSmem = kOffKeys + WK * STAGES * 4 + 1024;
  static_assert(kSmem <= 232448 && (kSmem + 1024) * RESIDENT <= 233472, "shared memory budget");
};

// Key of a 16-key tile's row: such that the rows of a matrix, and the keys of a value
// access, lie on different banks under the tile's swizzle, and the scales of a thread's
// keys beside one another.
template <int D>
__device__ __forceinline__ int key_of_row(int r) {
  return D == 256 ? r : 2 * (r & 7) + (r >> 3);
}
// Byte `at` of token `key` inside a unit's tile: rows of 128 bytes (headdim 64: of 64),
// two tokens each (headdim 256: one), under the row's own swizzle.
template <int D>
__device__ __forceinline__ uint32_t tile4_at(uint32_t base, int key, int at) {
  const uint32_t x = key * (D / 2) + at;
  return base + (x ^ (((x >> 7) & (D == 64 ? 3 : 7)) << 4));
}

template <int D, int NT, int WK, int STAGES, int RESIDENT, int KEPT>
__global__ void __launch_bounds__(Cache4Tile<D, NT, WK, STAGES, RESIDENT, KEPT>::kThreads, RESIDENT)
    dfa_cache4_rows_kernel(const __grid_constant__ Cache4FwdParams p) {
  using T = Cache4Tile<D, NT, WK, STAGES, RESIDENT, KEPT>;
  constexpr int kGroups = D / kCache4Group;
  constexpr int kHalf = D == 256 ? 2 : 1;  // value accesses per key
  constexpr int kM = D == 64 ? 4 : 8;      // tiles of 16 head dims per access
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem0 - smem_u32(smem_raw));
  float* s_m = reinterpret_cast<float*>(smem + T::kOffStat);
  float* s_l = s_m + WK * T::kRows;
  float* s_c = reinterpret_cast<float*>(smem + T::kOffC);
  const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5;
  const int g = lane >> 2, t = lane & 3;

  grid_dependency_wait();
  grid_launch_dependents();
  bool bad = false;
  Piece w = first_piece(p, blockIdx.x, &bad);
  if (bad) atomicOr(p.status, kStatusIndex);
  if (w.b < 0) return;  // the whole block

  // A piece's units go to the warps in turn: warp wk takes units wk, wk + WK, ...  A unit of
  // 16-token pages spans two.
  const bool two = p.page_size < kUnit;
  auto warp_units = [&](const Piece& x) {
    const int n = piece_end(p, x) - piece_begin(p, x);
    const int units = n > 0 ? (n + kUnit - 1) / kUnit : 0;
    return units > wk ? (units - wk + WK - 1) / WK : 0;
  };
  const uint32_t ring = smem0 + wk * STAGES * 2 * T::kTile;
  const uint32_t scales = smem0 + T::kOffScale + wk * STAGES * 2 * T::kScales;
  uint32_t* valid = reinterpret_cast<uint32_t*>(smem + T::kOffKeys) + wk * STAGES;
  // Copies run ahead of the products, over the ends of pieces: each warp walks the run on
  // its own (`la`) and fills a stage of its ring as it comes free.  Lane l keeps the pages
  // of the warp's units 32 i + l.
  Piece la = w;
  int la_units, la_u, la_h, la_key, la_end, to_fill = 0;
  int la_page[2] = {-1, -1};
  auto enter = [&] {
    la_units = warp_units(la);
    la_u = 0;
    la_h = la.seg / row_tiles(p, la.rq);
    la_key = piece_begin(p, la) + wk * kUnit;
    la_end = piece_end(p, la);
  };
  enter();
  auto ahead = [&] {
    while (la.b >= 0 && la_u >= la_units) {
      next_piece(p, la);
      if (la.b >= 0) enter();
    }
    if (la.b >= 0) {
      if ((la_u & 31) == 0) {
        la_page[0] = la_page[1] = -1;
        if (la_u + lane < la_units) {
          const int key = la_key + lane * (WK * kUnit);
          const int* table = p.block_table + static_cast<long long>(la.b) * p.max_pages;
          la_page[0] = table[key >> p.page_shift];
          const bool second = two && key + 16 < la_end;
          if (second) la_page[1] = table[(key + 16) >> p.page_shift];
          if (!cache_page_ok(la_page[0], p.num_pages) ||
              (second && !cache_page_ok(la_page[1], p.num_pages)))
            atomicOr(p.status, kStatusIndex);
        }
      }
      constexpr int kCopies = T::kTile / 512;
      const uint32_t dst = ring + to_fill * 2 * T::kTile;
      const uint32_t dst_scale = scales + to_fill * 2 * T::kScales + 16 * lane;
      // the i-th 512 bytes of the unit's k or v: 16 bytes a lane
      auto to = [&](int i) {
        return dst + 512 * i + (16 * lane ^ ((((lane >> 3) + 4 * i) & (D == 64 ? 3 : 7)) << 4));
      };
      // a lane's scales, 16 tokens of a group: of k, then of v
      const int half = lane & 1, grp = (lane >> 1) % kGroups;
      const uint8_t* scale = lane >= 2 * kGroups ? p.v4_scale : p.k4_scale;
      const int page = __shfl_sync(0xffffffffu, la_page[0], la_u & 31);
      const bool ok = cache_page_ok(page, p.num_pages);
      int count = ok ? min(16, la_end - la_key) : 0;  // valid keys of either half
      if (!two) {
        const int in_page = la_key & (p.page_size - 1);
        const long long head = static_cast<long long>(ok ? page : 0) * p.Hk + la_h;
        const long long from = (head * p.page_size + in_page) * (D / 2) + 16 * lane;
        const uint8_t *k = p.k4 + from, *v = p.v4 + from;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          copy16(to(i), k + 512 * i, ok);
          copy16(to(i) + T::kTile, v + 512 * i, ok);
        }
        if (lane < 4 * kGroups)
          copy16(dst_scale, scale + (head * kGroups + grp) * p.page_size + in_page + 16 * half, ok);
        if (ok) count |= max(0, min(16, la_end - la_key - 16)) << 8;
      } else {
        const int page1 = __shfl_sync(0xffffffffu, la_page[1], la_u & 31);
        const bool ok1 = cache_page_ok(page1, p.num_pages);
        const long long heads[2] = {static_cast<long long>(ok ? page : 0) * p.Hk + la_h,
                                    static_cast<long long>(ok1 ? page1 : 0) * p.Hk + la_h};
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int x = i / (kCopies / 2);
          const long long from = heads[x] * (16 * D / 2) + 512 * (i % (kCopies / 2)) + 16 * lane;
          copy16(to(i), p.k4 + from, x ? ok1 : ok);
          copy16(to(i) + T::kTile, p.v4 + from, x ? ok1 : ok);
        }
        if (lane < 4 * kGroups)
          copy16(dst_scale, scale + ((half ? heads[1] : heads[0]) * kGroups + grp) * 16,
                 half ? ok1 : ok);
        if (ok1) count |= max(0, min(16, la_end - la_key - 16)) << 8;
      }
      if (lane == 0) valid[to_fill] = count;
      ++la_u;
      la_key += WK * kUnit;
    }
    copies_end_group();
    if (++to_fill == STAGES) to_fill = 0;
  };

  // rows of the matrices that this lane addresses: matrix i = lane / 8 holds rows 8 (i %
  // 2) ... of the 16-key tile i / 2
  const int mat_key = 16 * (lane >> 4) + key_of_row<D>((lane & 7) + (lane & 8));
  const uint32_t mat_at = tile4_at<D>(0, mat_key, 0);
  // where the values of this lane's four keys of a 16-key tile begin (headdim 256: the
  // first half's), and the scales of its keys of either product's first group
  uint32_t val_at[4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    val_at[x] = tile4_at<D>(T::kTile, key_of_row<D>(2 * t + (x & 1) + 8 * (x >> 1)), kM * g);
  const uint32_t ks_at = D == 256 ? g : 2 * g;
  const uint32_t vs_at =
      T::kScales + (D == 256 ? 2 * t : 4 * t) + (D == 64 ? g >> 2 : g >> 1) * kUnit;
  int stage = 0;
  bool primed = false;

#pragma unroll 1
  for (; w.b >= 0; next_piece(p, w)) {
    const int rtiles = row_tiles(p, w.rq);
    const int h = w.seg / rtiles, tile = w.seg - h * rtiles;
    const int R = w.rq.n * p.G;  // rows of the request and key/value head
    const int row_base = tile * T::kRows, units = warp_units(w);
    // 8 head dims of a query row: those of word t of a group of 32
    auto load_q = [&](int nt, int grp) {
      const int r = row_base + 8 * nt + g;
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (r < R) {
        const int tok = r / p.G, hq = h * p.G + (r - tok * p.G);
        q = *reinterpret_cast<const uint4*>(p.q + (w.rq.row0 + tok) * p.q_sr + hq * p.q_sh +
                                            kCache4Group * grp + 8 * t);
      }
      return q;
    };
    // The queries' fragments for the cached keys, the powers of two, and what the groups'
    // scores begin at.  Fragments and beginnings are read from shared memory by every unit:
    // registers are better spent on the sums (held in registers: 181 us against 177 for 64
    // requests of 4 rows, 68 against 52 for 32 requests of 16 rows of headdim 256).
    float factor[NT][2];
    const uint32_t q_at = smem0 + T::kOffJoin + lane * 16;
    const uint32_t begin_at = smem0 + T::kOffJoin + T::kBeginAt + lane * 8;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint4 q[kGroups];
      unsigned top = 0;
#pragma unroll
      for (int grp = 0; grp < kGroups; ++grp) q[grp] = load_q(nt, grp);
#pragma unroll
      for (int grp = 0; grp < kGroups; ++grp) {
        const uint32_t v[4] = {q[grp].x, q[grp].y, q[grp].z, q[grp].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const unsigned lo = v[x] & 0x7fffu, hi = (v[x] >> 16) & 0x7fffu;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^-e brings the row's largest magnitude into [2^15, 2^16)
      int e = static_cast<int>(top >> 7) - 127 - 15;
      if (e < -100) e = -100;
      const float inv = pow2_bits(-e);
      // undoes that, and 2^-18 of the codes' 2^-24, with the softmax scale: within 2^-86 and
      // 2^127.6, so never 0, for a score may be -inf
      const float f = pow2_bits(e) * (p.scale_log2 * 0x1p18f);
#pragma unroll
      for (int x = 0; x < 2; ++x) factor[nt][x] = __shfl_sync(0xffffffffu, f, 8 * t + 4 * x);
#pragma unroll
      for (int grp = 0; grp < kGroups; ++grp) {
        const uint32_t v[4] = {q[grp].x, q[grp].y, q[grp].z, q[grp].w};
        uint32_t b[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // codes 2x, 2x + 1 stand at 2^-24, those after at 2^-20
          const float s = x & 1 ? inv * 0.0625f : inv;
          b[x] = pack_f16x2(__uint_as_float(v[x] << 16) * s,
                            __uint_as_float(v[x] & 0xffff0000u) * s);
        }
        constexpr uint32_t minus8[4] = {0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u};
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        float c[4];
        mma_f16(c, minus8, b, zero);
        mma_f16(c, minus8, b + 2, c);
        if (wk == 0) {
          st_shared_v4(q_at + (nt * kGroups + grp) * 512, b[0], b[1], b[2], b[3]);
          sts(begin_at + (nt * kGroups + grp) * 256, __float_as_uint(c[0]), __float_as_uint(c[1]));
        }
      }
    }
    if (!primed) {  // the run's first copies, behind the queries' loads
      primed = true;
#pragma unroll 1
      for (int i = 0; i < STAGES; ++i) ahead();
    }
    int own = 0;
    if (p.k != nullptr && w.last())
      own = cache_own_end(w.rq.len, min(R - 1, row_base + T::kRows - 1) / p.G, w.rq.n, p.bs);

    // o[nt][i]: of the dims 2i, 2i + 1 of the thread's run, rows 2t, 2t + 1 of the tile:
    // (2i, 2t), (2i, 2t + 1), (2i + 1, 2t), (2i + 1, 2t + 1)
    float o[NT][kHalf * kM][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kHalf * kM; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[nt][i][x] = 0.f;
    }
    // The output's unit, a power of two: the cached values' own, or larger for own ones.
    float unit = kCache4Unit;

    // Probabilities of raw scores sc (KT tiles of 16 keys; -inf: not seen) times the rows'
    // factors f, over the output's unit, in the products' other operand's order.  They are
    // taken against the reference as it stands; only where their sum says that one may have
    // outgrown f16, or with `look`, is the maximum found and the unit done again.
    // (The weight is 1 but behind own keys.  A copy of the code without it costs more in
    // instructions to be fetched than the products do: 3 us of 184 for 64 requests.)
    auto soften = [&](auto kt, auto f16, auto& sc, const float (&f)[NT][2], bool look, auto& pf) {
      constexpr int KT = decltype(kt)::value;
      float shrink[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) shrink[nt][0] = shrink[nt][1] = 1.f;
      const float weight = (decltype(f16)::value ? kCache4Unit : 1.f) / unit;
#pragma unroll 1
      for (;;) {
        if (look) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float top = fmaxf(sc[nt][0][x], sc[nt][0][2 + x]);
#pragma unroll
              for (int i = 1; i < KT; ++i) top = fmax3(top, sc[nt][i][x], sc[nt][i][2 + x]);
              top = __fmul_rd(top, f[nt][x]);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
              if (top > m[nt][x]) {
                const float a = ex2_approx(m[nt][x] - top);
                m[nt][x] = top;
                l[nt][x] *= a;
                shrink[nt][x] *= a;
              }
            }
        }
        float sum[NT][2];
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // a row that has met no finite score keeps probabilities of 0
          float ref[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            ref[x] = m[nt][x] == -INFINITY ? 0.f : kShift - m[nt][x];
            sum[nt][x] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float e0 = ex2_approx(cut_exponent(fmaf(sc[nt][i][2 * y], f[nt][0], ref[0])));
              float e1 = ex2_approx(cut_exponent(fmaf(sc[nt][i][2 * y + 1], f[nt][1], ref[1])));
              sum[nt][0] += e0;
              sum[nt][1] += e1;
              e0 *= weight, e1 *= weight;
              pf[nt][i][y] = transposed(decltype(f16)::value ? pack_f16x2(e0, e1)
                                                             : pack_bf16x2(e0, e1));
            }
#pragma unroll
          for (int x = 0; x < 2; ++x)
            over = over || sum[nt][x] > kMostSum || m[nt][x] == -INFINITY;
        }
        if (look || !__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) l[nt][0] += sum[nt][0], l[nt][1] += sum[nt][1];
          break;
        }
        look = true;
      }
      if (look) {
        bool any = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          any = any || shrink[nt][0] != 1.f || shrink[nt][1] != 1.f;
        if (__any_sync(0xffffffffu, any)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < kHalf * kM; ++i) {
              o[nt][i][0] *= shrink[nt][0];
              o[nt][i][1] *= shrink[nt][1];
              o[nt][i][2] *= shrink[nt][0];
              o[nt][i][3] *= shrink[nt][1];
            }
        }
      }
    };

    // Own keys and values first, bf16, with the segment's end, while the cached keys are on
    // their way: units of 16 keys, the warps in turn, operands straight from global memory.
    if (16 * wk < own) {
      unit = kOwnUnit;
      float own_factor[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) own_factor[nt][0] = own_factor[nt][1] = p.scale_log2;
#pragma unroll 1
      for (int k0 = 16 * wk; k0 < own; k0 += 16 * WK) {
        float sc[NT][1][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[nt][0][x] = 0.f;
#pragma unroll
        for (int grp = 0; grp < kGroups; ++grp) {
          uint4 kx[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int key = k0 + 8 * y + g;
            kx[y] = make_uint4(0u, 0u, 0u, 0u);
            if (key < w.rq.n)
              kx[y] = *reinterpret_cast<const uint4*>(p.k + (w.rq.row0 + key) * p.k_sr +
                                                      h * p.k_sh + kCache4Group * grp + 8 * t);
          }
          const uint32_t a[2][4] = {{kx[0].x, kx[1].x, kx[0].y, kx[1].y},
                                    {kx[0].z, kx[1].z, kx[0].w, kx[1].w}};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 q = load_q(nt, grp);
            const uint32_t b[2][2] = {{q.x, q.y}, {q.z, q.w}};
            mma_bf16(sc[nt][0], a[0], b[0]);
            mma_bf16(sc[nt][0], a[1], b[1]);
          }
        }
        int end[NT][2];  // one past the last own key of the thread's rows
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = row_base + 8 * nt + 2 * t + x;
            end[nt][x] = r < R ? cache_own_end(w.rq.len, r / p.G, w.rq.n, p.bs) : 0;
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (k0 + 8 * y + g >= end[nt][x]) sc[nt][0][2 * y + x] = -INFINITY;
          }
        uint32_t pf[NT][1][2];
        soften(std::integral_constant<int, 1>{}, std::false_type{}, sc, own_factor, true, pf);
        // A row's probability of an own key it does not see is 0, but 0 times a value that is
        // not finite is not: such values leave the product and are added to the rows that
        // see them.
        bool odd = false;
        const __nv_bfloat16* vsrc = p.v + static_cast<long long>(w.rq.row0) * p.v_sr + h * p.v_sh;
#pragma unroll
        for (int half = 0; half < kHalf; ++half)
#pragma unroll
          for (int part = 0; part < kM / 4; ++part) {  // 8 dims at a time
            uint32_t vw[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = k0 + 8 * (x >> 1) + 2 * t + (x & 1);
              uint4 v4 = make_uint4(0u, 0u, 0u, 0u);
              if (key < w.rq.n)
                v4 = *reinterpret_cast<const uint4*>(vsrc + key * p.v_sr + 128 * half + 2 * kM * g +
                                                     8 * part);
              vw[x][0] = v4.x, vw[x][1] = v4.y, vw[x][2] = v4.z, vw[x][3] = v4.w;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                if ((vw[x][y] & 0x7f80u) == 0x7f80u) vw[x][y] &= 0xffff0000u, odd = true;
                if ((vw[x][y] & 0x7f800000u) == 0x7f800000u) vw[x][y] &= 0xffffu, odd = true;
              }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t a[4] = {__byte_perm(vw[0][y], vw[1][y], 0x5410),
                                     __byte_perm(vw[0][y], vw[1][y], 0x7632),
                                     __byte_perm(vw[2][y], vw[3][y], 0x5410),
                                     __byte_perm(vw[2][y], vw[3][y], 0x7632)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_bf16(o[nt][half * kM + 4 * part + y], a, pf[nt][0]);
            }
          }
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
          for (int key = k0; key < min(k0 + 16, w.rq.n); ++key) {
            const __nv_bfloat16* src = vsrc + key * p.v_sr + 2 * kM * g;
#pragma unroll
            for (int i = 0; i < kHalf * kM; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float v = __bfloat162float(src[128 * (i / kM) + 2 * (i % kM) + y]);
                if (isfinite(v)) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int x = 0; x < 2; ++x)
                    if (key < end[nt][x]) o[nt][i][2 * y + x] += v;
              }
          }
        }
      }
      // Cached probabilities are f16 and relative to the output's unit, which is to be theirs:
      // it comes down, but not so far that the own keys' output, in the new unit, would pass
      // 2^100 (what cached keys lose to that is below 2^-100 of it).
      if (units > 0) {
        unsigned top = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < kHalf * kM; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const unsigned y = __float_as_uint(o[nt][i][x]) & 0x7fffffffu;
              top = max(top, y < 0x7f800000u ? y : 0u);
            }
        top = __reduce_max_sync(0xffffffffu, top);
        const int down = max(min(127 + 99 - static_cast<int>(top >> 23), kOwnExp - 4), 0);
        const float grow = pow2_bits(down);
        unit *= pow2_bits(-down);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < kHalf * kM; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[nt][i][x] *= grow;
      }
    }
    __syncthreads();  // the queries' fragments

#pragma unroll 1
    for (int u = 0; u < units; ++u) {
      copies_wait<STAGES - 1>();
      __syncwarp();  // every lane's copies
      const uint32_t kt = ring + stage * 2 * T::kTile;
      const uint32_t sct = scales + stage * 2 * T::kScales;
      const unsigned both = valid[stage];
      if (++stage == STAGES) stage = 0;
      const int nv[2] = {static_cast<int>(both & 255u), static_cast<int>(both >> 8)};
      if (both != 0) {  // else nothing is to be followed
        const bool whole = both == 0x1010u;
        // Scores: sums over the groups of 32 dims.
        float sc[NT][2][4];
        const uint32_t k_at = kt + mat_at;
#pragma unroll
        for (int grp = 0; grp < kGroups; ++grp) {
          uint32_t word[4];
          load_matrices(k_at ^ (16 * grp), word);
          uint4 b[NT];
          float c0[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            b[nt] = lds128(q_at + (nt * kGroups + grp) * 512);
            const uint2 x = lds<uint2>(begin_at + (nt * kGroups + grp) * 256);
            c0[nt][0] = c0[nt][2] = __uint_as_float(x.x);
            c0[nt][1] = c0[nt][3] = __uint_as_float(x.y);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // the scales of the thread's two keys, times 2^6
            float ks[2];
            {
              uint32_t s2;
              if constexpr (D == 256) {
                const uint32_t at = sct + ks_at + 16 * i + kUnit * grp;
                uint32_t s0, s1;
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s0) : "r"(at) : "memory");
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s1) : "r"(at + 8) : "memory");
                s2 = s0 << 8 | s1 << 24;
              } else {
                s2 = __byte_perm(lds<unsigned short>(sct + ks_at + 16 * i + kUnit * grp), 0,
                                 0x1404);
              }
#pragma unroll
              for (int y = 0; y < 2; ++y)  // with the conversion (apart: 58 us for blocks of 4)
                asm("fma.rn.f32.f16 %0, %1, %2, %3;"
                    : "=f"(ks[y])
                    : "h"(static_cast<unsigned short>(s2 >> (16 * y))),
                      "h"(static_cast<unsigned short>(0x5400)), "f"(0.f));
            }
            const uint32_t lo = word[2 * i], hi = word[2 * i + 1];
            const uint32_t a[2][4] = {
                {lo & 0x000f000fu, hi & 0x000f000fu, lo & 0x00f000f0u, hi & 0x00f000f0u},
                {(lo >> 8) & 0x000f000fu, (hi >> 8) & 0x000f000fu, (lo >> 8) & 0x00f000f0u,
                 (hi >> 8) & 0x00f000f0u}};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t b0[2] = {b[nt].x, b[nt].y}, b1[2] = {b[nt].z, b[nt].w};
              float c[4];
              mma_f16(c, a[0], b0, c0[nt]);
              mma_f16(c, a[1], b1, c);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                sc[nt][i][x] = grp == 0 ? c[x] * ks[x >> 1] : fmaf(c[x], ks[x >> 1], sc[nt][i][x]);
            }
          }
        }
        if (!whole) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (key_of_row<D>(g + 8 * (x >> 1)) >= nv[i]) sc[nt][i][x] = -INFINITY;
        }
        uint32_t pf[NT][2][2];
        soften(std::integral_constant<int, 2>{}, std::true_type{}, sc, factor, false, pf);
        // Values: keys 2t, 2t + 1 and 2t + 8, 2t + 9 of a tile's rows, the thread's run of
        // dims of each.  What lies behind the last key may be anything: its scale becomes
        // zero, and with it the value.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int half = 0; half < kHalf; ++half) {
            const uint32_t s_at = sct + vs_at + 16 * i + 4 * kUnit * half;
            uint32_t s2[2];
            if constexpr (D == 256) {
#pragma unroll
              for (int y = 0; y < 2; ++y)
                s2[y] = __byte_perm(lds<unsigned short>(s_at + 8 * y), 0, 0x1404);
            } else {  // keys 4t, 4t + 2, then 4t + 1, 4t + 3
              const uint32_t s4 = lds<uint32_t>(s_at);
              s2[0] = __byte_perm(s4, 0, 0x2404), s2[1] = __byte_perm(s4, 0, 0x3414);
            }
            uint32_t vw[4][kM / 4];
            Cache4Scale sv[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t at = kt + (val_at[2 * y + x] ^ (64 * half)) + i * (16 * D / 2);
                if constexpr (D == 64) {
                  vw[2 * y + x][0] = lds<uint32_t>(at);
                } else {
                  const uint2 w2 = lds<uint2>(at);
                  vw[2 * y + x][0] = w2.x, vw[2 * y + x][1] = w2.y;
                }
                if (!whole && key_of_row<D>(2 * t + x + 8 * y) >= nv[i])
                  s2[y] &= x ? 0x0000ffffu : 0xffff0000u;
              }
              sv[y] = cache4_prepare(s2[y]);
            }
#pragma unroll
            for (int y = 0; y < kM / 4; ++y) {
              uint32_t a[2][2][4];  // even and odd dims, first and second pair of keys
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                cache4_decode(__byte_perm(vw[0][y], vw[1][y], q ? 0x7632 : 0x5410), sv[0], a[q][0]);
                cache4_decode(__byte_perm(vw[2][y], vw[3][y], q ? 0x7632 : 0x5410), sv[1], a[q][1]);
              }
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const uint32_t av[4] = {a[0][0][z], a[1][0][z], a[0][1][z], a[1][1][z]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(o[nt][half * kM + 4 * y + z], av, pf[nt][i],
                          o[nt][half * kM + 4 * y + z]);
              }
            }
          }
        }
      }
      __syncwarp();  // the unit has been read
      ahead();
    }

    // Join the warps: statistics first, then each warp's output in a common unit, summed.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], off);
        if (g == 0) s_m[wk * T::kRows + 8 * nt + 2 * t + x] = m[nt][x];
      }
    if (lane == 0) s_c[wk] = unit;
    __syncthreads();  // statistics written, the last piece's join read
    float unit_all = s_c[0];
#pragma unroll
    for (int i = 1; i < WK; ++i) unit_all = fmaxf(unit_all, s_c[i]);
    // kKept warps of a row leave their outputs, the others, as many at a time, add theirs.
    float* join = reinterpret_cast<float*>(smem + T::kOffJoin);
#pragma unroll 1
    for (int turn = 0; turn < (WK + KEPT - 1) / KEPT; ++turn) {
      const bool add = turn > 0;
      if (wk / KEPT == turn) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = 8 * nt + 2 * t + x;
            float top = s_m[r];
#pragma unroll
            for (int i = 1; i < WK; ++i) top = fmaxf(top, s_m[i * T::kRows + r]);
            const float f = m[nt][x] == -INFINITY ? 0.f : ex2_approx(m[nt][x] - top);
            const float fo = f * (unit / unit_all);
            if (g == 0) s_l[wk * T::kRows + r] = l[nt][x] * f;
            float* dst = join + ((wk % KEPT) * T::kRows + r) * T::kPitch;
#pragma unroll
            for (int i = 0; i < kHalf * kM; i += 2) {
              float4* at = reinterpret_cast<float4*>(dst + 128 * (i / kM) + 2 * kM * g +
                                                     2 * (i % kM));
              float4 y = make_float4(o[nt][i][x] * fo, o[nt][i][2 + x] * fo,
                                     o[nt][i + 1][x] * fo, o[nt][i + 1][2 + x] * fo);
              if (add) {
                const float4 z = *at;
                y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
              }
              *at = y;
            }
          }
      }
      __syncthreads();
    }
    const bool single = w.whole();
    for (int i = tid; i < T::kRows * (D / 4); i += T::kThreads) {
      const int r = i / (D / 4), d4 = i - r * (D / 4);
      if (row_base + r >= R) break;
      float sum = 0.f, top = -INFINITY;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < WK; ++x) {
        sum += s_l[x * T::kRows + r];
        top = fmaxf(top, s_m[x * T::kRows + r]);
      }
#pragma unroll
      for (int x = 0; x < KEPT; ++x) {
        const float4 y =
            *reinterpret_cast<const float4*>(join + (x * T::kRows + r) * T::kPitch + 4 * d4);
        a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
      }
      // no key (sum 0): output 0 and -inf; scores that are not numbers: NaN
      const bool none = top == -INFINITY && sum == 0.f;
      const float inv = none ? 0.f : unit_all / sum;
      const float lse2 = none ? -INFINITY : top - kShift + lg2_approx(sum);
      a.x *= inv, a.y *= inv, a.z *= inv, a.w *= inv;
      if (single) {
        const int tok = (row_base + r) / p.G, hq = h * p.G + (row_base + r - tok * p.G);
        const long long row = w.rq.row0 + tok;
        *reinterpret_cast<uint2*>(p.out + (row * p.H + hq) * D + 4 * d4) =
            make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        if (d4 == 0) p.lse[static_cast<long long>(hq) * p.rows + row] = lse2 * 0.6931471805599453f;
      } else {
        const long long at = (2LL * blockIdx.x + (w.first ? 0 : 1)) * T::kRows + r;
        *reinterpret_cast<float4*>(p.part_o + at * D + 4 * d4) = a;
        if (d4 == 0) p.part_lse[at] = lse2;
      }
    }
    __syncthreads();  // the join has been read
  }  // pieces
}

// Row tiles, warps, stages, blocks per SM and outputs kept, for a head dimension and a
// segment's rows.
//
// Blocks per SM: what the registers allow without spilling much (headdim 128: 3 blocks of
// 161 registers for 8 rows, 2 of 244 for 16).  More lose to spills, fewer to idle schedulers
// (us, 32 ragged requests of up to 8192 tokens, 512 / headdim heads for keys): headdim 128,
// 16 rows 41 with 2 and 44 with 3; headdim 64, 8 rows 38 with 4 and 41 with 3, 16 rows 46
// with 3 and 49 with 4.  Stages: two keep enough in flight with 8 or 12 warps (headdim 128,
// 64 requests of up to 16000 tokens: two, three and four within 1 us of 186), and what they
// leave is L1 for what the registers spill.
template <int D, int ROWS>
struct Variant;
template <> struct Variant<64, 8> { using T = Cache4Tile<64, 1, 4, 4, 4, 4>; };
template <> struct Variant<64, 16> { using T = Cache4Tile<64, 2, 4, 5, 3, 4>; };
template <> struct Variant<64, 32> { using T = Cache4Tile<64, 4, 4, 3, 2, 4>; };
template <> struct Variant<128, 8> { using T = Cache4Tile<128, 1, 4, 2, 3, 4>; };
template <> struct Variant<128, 16> { using T = Cache4Tile<128, 2, 4, 2, 2, 4>; };
template <> struct Variant<256, 8> { using T = Cache4Tile<256, 1, 4, 2, 2, 4>; };
template <> struct Variant<256, 16> { using T = Cache4Tile<256, 2, 4, 2, 2, 2>; };

template <int D, int NT, int WK, int STAGES, int RESIDENT, int KEPT>
cudaError_t launch_tile(Cache4Tile<D, NT, WK, STAGES, RESIDENT, KEPT>, const Cache4FwdParams& p,
                        cudaStream_t stream) {
  using T = Cache4Tile<D, NT, WK, STAGES, RESIDENT, KEPT>;
  auto kern = dfa_cache4_rows_kernel<D, NT, WK, STAGES, RESIDENT, KEPT>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(p.blocks), dim3(T::kThreads), T::kSmem, stream, p);
}

// What f gives for the variant of a head dimension and rows.
template <typename R, typename F>
R for_variant(int d, int rows, R none, F f) {
  if (d == 64) {
    if (rows == 8) return f(Variant<64, 8>::T{});
    if (rows == 16) return f(Variant<64, 16>::T{});
    if (rows == 32) return f(Variant<64, 32>::T{});
  } else if (d == 128) {
    if (rows == 8) return f(Variant<128, 8>::T{});
    if (rows == 16) return f(Variant<128, 16>::T{});
  } else if (d == 256) {
    if (rows == 8) return f(Variant<256, 8>::T{});
    if (rows == 16) return f(Variant<256, 16>::T{});
  }
  return none;
}

}  // namespace

cudaError_t launch_cache4_rows(const Cache4FwdParams& p, int headdim, int tile_rows,
                               cudaStream_t stream) {
  return for_variant(headdim, tile_rows, cudaErrorInvalidValue,
                     [&](auto tile) { return launch_tile(tile, p, stream); });
}

int cache4_blocks_per_sm(int headdim, int tile_rows) {
  return for_variant(headdim, tile_rows, 1, [](auto tile) { return decltype(tile)::kResident; });
}

}  // namespace dfa
