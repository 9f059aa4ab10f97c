// Attention of new rows over a paged 8-bit key/value cache and, optionally,
// over the new rows' own keys and values in bf16: one block of a block
// diffusion sampler against the clean tokens before it ("Fast Diffusion
// Attention", "Block diffusion in one picture": a block sees itself and the
// clean blocks before it).
//
// Mathematics.  Row i of request b (position len_b + i) and query head h see
// the len_b cached tokens and the own rows of its block or earlier blocks:
//   s_j = scale * q . (k8_j * ks(page of j, head))   cached
//   s_j = scale * q . k_j                            own
//   out = sum_j softmax(s)_j v_j,  lse = ln sum_j exp(s_j).
// k8 is e4m3 and ks a power of two, so k8 converts to f16 exactly and the
// page's scale multiplies the score.  q is bf16: a row is brought to f16 by a
// power of two of its own (its largest magnitude lands in [2^14, 2^15)),
// which keeps every value down to 2^-31 of the row's largest exact.  The
// probabilities are rounded to f16 (2^-11) for P V while the sums use them
// unrounded; a value page's scale, relative to the largest one met so far (the
// output's unit), multiplies its probabilities.  Own keys and values are bf16
// products, exact in any unit but for the probabilities' 2^-8.
//
// The reference of a row's exponentials moves only where a unit's
// probabilities outgrow f16 (cache_fwd.cuh), so that most units need neither a
// maximum nor a rescaling of the output.
//
// Work.  All query heads of a key/value head share its keys: row r of a
// segment's tile is query row r / G and head r % G.  Segments (request,
// key/value head, tile of rows) are dealt to the blocks in equal runs of
// 128-key units (cache.cuh); a block walks its run piece by piece.  Its WK warp
// groups take 32-key units of a piece in turn, each with a ring of stages of
// its own, filled by TMA boxes (32 tokens of one page and head) that run ahead
// over the pieces' ends, and with softmax statistics of its own; the groups
// join through shared memory at a piece's end, the pieces of a cut segment
// through a float32 workspace and a second launch.  mma.sync fragments are
// read straight out of the swizzled e4m3 tiles: the head dims (and the keys)
// may be numbered in any order inside a product, so each thread takes 16
// contiguous bytes of a token, which are the operands of four k steps of
// Q K^T or 16 column tiles of P V.
//
// For up to 32 rows to a key (headdim 256: any number), where the tcgen05
// kernel's 128 rows would be mostly empty: 32 rows 111 us here, 121 there
// (headdim 128), 132 and 188 (headdim 64); 64 rows as two tiles here 197, 124
// there.  (32 ragged requests of up to 8192 tokens, 330 MB.)
//
// Measured, 16 rows, headdim 128: 74 us for those 330 MB (4.5 TB/s, 66% of
// what a copy reaches), 58 us for 24 requests of up to 8000 tokens (4.1 TB/s).
// Bound by latency: 255 registers a thread leave 8 warps to an SM, which issue
// in 36% of the cycles (DRAM 50%, tensor pipe 20%), and some 7 us pass before
// the first products (lengths, queries, first tiles: each a trip to memory),
// 4 at a piece's end.  Two blocks of four groups against others, when the 24
// requests took 60.1 us: four of two 62.5; one of eight 73.7; loops over the
// products rolled 63 to 66.
#pragma once

#include <type_traits>

#include "cache4.cuh"
#include "cache_fwd.cuh"

namespace dfa {
namespace {

constexpr int kUnit = 32;  // keys per unit

// D (16 x 8, float32) += A (16 x 16) B (16 x 8).
__device__ __forceinline__ void mma_f16(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}


template <int BITS, int D, int MT, int WR, int WK, int STAGES>
struct CacheTile {
  static constexpr int kThreads = 32 * WR * WK;
  static constexpr int kResident = D == 256 ? 1 : D == 64 && MT == 1 ? 3 : 2;  // blocks per SM
  static constexpr int kRows = 16 * MT * WR;
  static constexpr int kUnitBytes = kUnit * D * BITS / 8;  // of k, and of v
  static constexpr int kRing = WK * STAGES * 2 * kUnitBytes;
  // 4 bits: the units' scales, a slot for the groups of 16 tokens of k, and of v (32
  // tokens of a page lie in both of theirs)
  static constexpr int kSlot = 128;
  static constexpr int kScales = BITS == 4 ? WK * STAGES * 4 * kSlot : 0;
  static constexpr int kFrags = (D / 64) * 4;  // k steps of Q K^T
  static constexpr int kQ = WR * MT * kFrags * 512;
  static constexpr int kPitch = D + 4;   // floats per row of a group's output at the join
  // Outputs that are kept at the join: every group's where there is room (one
  // token over 500: 11.7 us, 12.0 with half as many), else half as many, to
  // which the other half of the groups adds.
  static constexpr int kKept = kRows == 16 && D <= 128 ? WK : WK / 2;
  static constexpr int kJoin = kKept * kRows * kPitch * 4;
  // ring (1024-byte aligned) | scales | join | q fragments | row factors | statistics | barriers
  static constexpr int kOffScale = kRing;
  static constexpr int kOffJoin = kOffScale + kScales;
  static constexpr int kOffQ = kOffJoin + kJoin;
  static constexpr int kOffFactor = kOffQ + kQ;
  static constexpr int kOffStat = kOffFactor + kRows * 4;  // m, l per group and row
  static constexpr int kOffC = kOffStat + WK * kRows * 8;
  static constexpr int kOffBar = (kOffC + WK * WR * 4 + 7) / 8 * 8;
  static constexpr int kOffFlag = kOffBar + WK * STAGES * 16;
  static constexpr int kSmem = kOffFlag + 16 + 1024;
  static_assert(WK % 2 == 0 && kSmem <= 232448, "shared memory budget");
};

// Plain loads: the compiler may move them among the products, but not over a
// barrier wait (which clobbers memory).
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// 16-byte chunk c of token row r inside a TMA tile of 8-bit values: the tile's
// swizzle.
template <int D>
__device__ __forceinline__ const uint8_t* tile_at(const uint8_t* base, int r, int c) {
  if constexpr (D == 64) return base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return base + (c >> 3) * (kUnit * 128) + r * 128 + (((c ^ r) & 7) << 4);
}

// Keys of a fragment column pair.  headdim 64 numbers the eight keys of a
// column tile in order; wider heads put keys t and t + 4 into columns 2t and
// 2t + 1, so that the eight lanes of a shared-memory phase (two keys, four
// chunks) fall on different banks under the 128-byte swizzle.
template <int D>
__device__ __forceinline__ int key_of(int n) {
  return D == 64 ? n : (n >> 1) + 4 * (n & 1);
}

// Byte `at` of token r inside a tile of 4-bit values: rows of 128 bytes (headdim 64:
// of 64), two tokens each (headdim 256: one), under the row's own swizzle.
template <int D>
__device__ __forceinline__ const uint8_t* tile4_at(const uint8_t* base, int r, int at) {
  const int x = r * (D / 2) + at;
  return base + (x ^ (((x >> 7) & (D == 64 ? 3 : 7)) << 4));
}

// The key of a unit in column c of column tile n.  8 bits: tiles of eight keys in
// order of key_of.  4 bits: such that the two keys of a thread's column pair are
// neighbours (one access for their scales), that its pairs of 16 keys lie close, and
// that the threads of a shared-memory phase, which read four keys' halves or the
// same half of eight, fall on different banks under tile4_at's swizzle.
template <int BITS, int D>
__device__ __forceinline__ int unit_key(int n, int c) {
  if constexpr (BITS == 8) return 8 * n + key_of<D>(c);
  const int t = c >> 1, x = c & 1;
  if constexpr (D == 64) return 16 * (n >> 1) + 8 * (t >> 1) + 4 * (n & 1) + 2 * (t & 1) + x;
  if constexpr (D == 128) return 16 * (n >> 1) + 4 * t + 2 * (n & 1) + x;
  return 8 * n + c;
}
// The run of head dims that column c of the output's column tiles stands for.
template <int BITS, int D>
__device__ __forceinline__ int run_of(int c) {
  return BITS == 4 ? c : key_of<D>(c);
}

template <int BITS, int D, int MT, int WR, int WK, int STAGES>
__global__ void __launch_bounds__(CacheTile<BITS, D, MT, WR, WK, STAGES>::kThreads,
                                  CacheTile<BITS, D, MT, WR, WK, STAGES>::kResident)
    dfa_cache_fwd_kernel(const __grid_constant__ CacheParams<BITS> p) {
  using T = CacheTile<BITS, D, MT, WR, WK, STAGES>;
  constexpr int kSeg = D / 64;       // 64-dim segments of Q K^T
  constexpr int kCols = D == 64 ? 8 : 16;  // column tiles of P V per value load
  constexpr int kHalf = D == 256 ? 2 : 1;  // value loads per key
  constexpr int kOut = kCols * kHalf;      // column tiles of the output, D / 8
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem0 - smem_u32(smem_raw));
  float* s_factor = reinterpret_cast<float*>(smem + T::kOffFactor);
  float* s_m = reinterpret_cast<float*>(smem + T::kOffStat);
  float* s_l = s_m + WK * T::kRows;
  float* s_c = reinterpret_cast<float*>(smem + T::kOffC);
  volatile int* s_flag = reinterpret_cast<volatile int*>(smem + T::kOffFlag);
  const uint32_t bars = smem0 + T::kOffBar;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp % WR, wk = warp / WR;

  if (tid == 0) {
    for (int i = 0; i < WK * STAGES; ++i) {
      mbar_init(bars + 16 * i, 1);       // full
      mbar_init(bars + 16 * i + 8, WR);  // empty
    }
    fence_mbar_init();
    *s_flag = 0;
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
    if constexpr (BITS == 4) {
      tma_prefetch_desc(&p.tm_ks);
      tma_prefetch_desc(&p.tm_vs);
    }
  }
  grid_dependency_wait();
  grid_launch_dependents();
  bool bad = false;
  Piece w = first_piece(p, blockIdx.x, &bad);
  if (bad) atomicOr(p.status, kStatusIndex);
  if (w.b < 0) return;  // the whole block
  __syncthreads();      // barriers initialised
  const AbortFlag ab{const_cast<int*>(s_flag), p.status};

  // A piece's 32-key units go to the groups in turn: group wk takes units wk,
  // wk + WK, ...  Lane l keeps the pages (and scales) of the group's units 32 i
  // + l; a unit of 16-token pages spans two.
  const bool two = p.page_size < kUnit;
  auto key_first = [&](const Piece& x) { return piece_begin(p, x); };
  auto key_end = [&](const Piece& x) { return piece_end(p, x); };
  auto group_units = [&](const Piece& x) {
    const int n = key_end(x) - key_first(x);
    const int units = n > 0 ? (n + kUnit - 1) / kUnit : 0;
    return units > wk ? (units - wk + WK - 1) / WK : 0;
  };
  auto load_pages = [&](const Piece& x, int units, int u, int* page) {  // of the group's unit u
    page[0] = page[1] = -1;
    if (u >= units) return;
    const int key = key_first(x) + (wk + u * WK) * kUnit;
    const int* table = p.block_table + static_cast<long long>(x.b) * p.max_pages;
    page[0] = table[key >> p.page_shift];
    const bool second = two && key + 16 < key_end(x);
    if (second) page[1] = table[(key + 16) >> p.page_shift];
    if (!cache_page_ok(page[0], p.num_pages) || (second && !cache_page_ok(page[1], p.num_pages)))
      atomicOr(p.status, kStatusIndex);
    if (!two) page[1] = page[0];
  };
  // 4 bits: the scales come with the unit, and a page's own is 1.
  auto load_scales = [&](int h, const int* page, float* ks, float* vs) {
    if constexpr (BITS == 4) {
      ks[0] = ks[1] = vs[0] = vs[1] = 1.f;
      return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool ok = cache_page_ok(page[i], p.num_pages);
      const long long at = static_cast<long long>(page[i]) * p.Hk + h;
      ks[i] = ok ? p.k_scale[at] : 0.f;
      vs[i] = ok ? p.v_scale[at] : 0.f;
    }
  };
  const uint32_t ring = smem0 + wk * STAGES * 2 * T::kUnitBytes;
  const uint32_t gbar = bars + 16 * wk * STAGES;
  // Loads run ahead of the products, over the ends of pieces: the first warp
  // of a group walks the run on its own (`la`) and fills each stage of the
  // group's ring as it comes free.
  Piece la = w;
  int la_units = group_units(la), la_u = 0, issued = 0;
  int la_page[2];
  auto ahead = [&]() -> bool {
    while (la.b >= 0 && la_u >= la_units) {
      next_piece(p, la);
      if (la.b < 0) return true;
      la_units = group_units(la);
      la_u = 0;
    }
    if (la.b < 0) return true;
    const int h = la.seg / row_tiles(p, la.rq);
    if ((la_u & 31) == 0) {
      load_pages(la, la_units, la_u + lane, la_page);
#pragma unroll
      for (int i = 0; i < (BITS == 8 ? 2 : 0); ++i)
        if (cache_page_ok(la_page[i], p.num_pages)) {  // the products read them next
          const long long at = static_cast<long long>(la_page[i]) * p.Hk + h;
          asm volatile("prefetch.global.L1 [%0];" ::"l"(p.k_scale + at));
          asm volatile("prefetch.global.L1 [%0];" ::"l"(p.v_scale + at));
        }
    }
    const int page0 = __shfl_sync(0xffffffffu, la_page[0], la_u & 31);
    const int page1 = __shfl_sync(0xffffffffu, la_page[1], la_u & 31);
    const int s = issued % STAGES;
    const uint32_t dst = ring + s * 2 * T::kUnitBytes, bar = gbar + 16 * s;
    if (issued >= STAGES && !mbar_wait_warp(bar + 8, (issued / STAGES - 1) & 1, ab)) return false;
    if (lane == 0) {
      const int key = key_first(la) + (wk + la_u * WK) * kUnit;
      const bool ok0 = cache_page_ok(page0, p.num_pages);
      const bool ok1 = two && cache_page_ok(page1, p.num_pages);
      const int rows = two ? 16 : kUnit;
      const int bytes = rows * (BITS == 8 ? D * 2 : D + D / 16);  // of k and v
      mbar_arrive_expect_tx(bar, (ok0 ? bytes : 0) + (ok1 ? bytes : 0));
      const int off = h * p.page_size + (key & (p.page_size - 1));
      if constexpr (BITS == 4) {
        constexpr int kPair = D == 256 ? 1 : 2;  // tokens of a tile's row
        const uint32_t ds = smem0 + T::kOffScale + (wk * STAGES + s) * 4 * T::kSlot;
        auto load = [&](int page, int key, int half) {
          const int at = key & (p.page_size - 1), row = (h * p.page_size + at) / kPair;
          const uint32_t d = dst + half * (16 * D / 2), sc = ds + half * T::kSlot;
          tma_load_3d(d, &p.tm_k, bar, 0, row, page);
          tma_load_3d(d + T::kUnitBytes, &p.tm_v, bar, 0, row, page);
          tma_load_3d(sc, &p.tm_ks, bar, at, h * (D / 32), page);
          tma_load_3d(sc + 2 * T::kSlot, &p.tm_vs, bar, at, h * (D / 32), page);
        };
        if (ok0) load(page0, key, 0);
        if (ok1) load(page1, key + 16, 1);
      }
#pragma unroll
      for (int half = 0; half < (BITS == 8 ? kHalf : 0); ++half) {
        const uint32_t d = dst + half * kUnit * 128;
        if (ok0) {
          tma_load_3d(d, &p.tm_k, bar, half * 128, off, page0);
          tma_load_3d(d + T::kUnitBytes, &p.tm_v, bar, half * 128, off, page0);
        }
        if (ok1) {
          constexpr int kRow = D == 64 ? 64 : 128;
          const int off1 = h * p.page_size + ((key + 16) & (p.page_size - 1));
          tma_load_3d(d + 16 * kRow, &p.tm_k, bar, half * 128, off1, page1);
          tma_load_3d(d + T::kUnitBytes + 16 * kRow, &p.tm_v, bar, half * 128, off1, page1);
        }
      }
    }
    __syncwarp();
    ++issued;
    ++la_u;
    return true;
  };
  int consumed = 0;
  bool primed = false;
  bool ok = true;

#pragma unroll 1
  for (; w.b >= 0 && ok; next_piece(p, w)) {
    const int rtiles = row_tiles(p, w.rq);
    const int h = w.seg / rtiles, tile = w.seg - h * rtiles;
    const int R = w.rq.n * p.G;  // rows of the request and key/value head
    const int row_base = tile * T::kRows;
    const int key_lo = key_first(w), key_hi = key_end(w), my_units = group_units(w);
    // The piece's queries: the f16 fragments of the cached keys' products (built
    // by the first group for all) and the bf16 ones of the own keys', which stay
    // in registers where there is room (kHoldQ) and are read again where not.
    constexpr bool kHoldQ = MT * D <= 128;
    // the first of the 16 head dims that the thread has of the products' segment sg
    auto dim_of = [&](int sg) { return BITS == 8 ? 64 * sg + 16 * t : 16 * sg + (D / 4) * t; };
    auto load_q = [&](int mt, int i, int sg, uint4* q2) {
      const int r = row_base + 16 * (wr * MT + mt) + g + 8 * i;
      q2[0] = q2[1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < R) {
        const int tok = r / p.G, hq = h * p.G + (r - tok * p.G);
        const __nv_bfloat16* src =
            p.q + (w.rq.row0 + tok) * p.q_sr + hq * p.q_sh + dim_of(sg);
        q2[0] = *reinterpret_cast<const uint4*>(src);
        q2[1] = *reinterpret_cast<const uint4*>(src + 8);
      }
    };
    uint4 qv[kHoldQ ? MT : 1][2][kSeg][2];
    if constexpr (kHoldQ) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int sg = 0; sg < kSeg; ++sg) load_q(mt, i, sg, qv[mt][i][sg]);
    }
    if (!primed && wr == 0) {  // the run's first loads, behind the queries'
#pragma unroll 1
      for (int s = 0; s < STAGES; ++s) ahead();
    }
    primed = true;
    int own = 0;
    if (p.k != nullptr && w.last())
      own = cache_own_end(w.rq.len, min(R - 1, row_base + T::kRows - 1) / p.G, w.rq.n, p.bs);
    auto load_own_k = [&](int k0, int sg, int n, uint4* k2) {
      const int key = k0 + 8 * n + g;
      k2[0] = k2[1] = make_uint4(0u, 0u, 0u, 0u);
      if (key < w.rq.n) {
        const __nv_bfloat16* src =
            p.k + (w.rq.row0 + key) * p.k_sr + h * p.k_sh + dim_of(sg);
        k2[0] = *reinterpret_cast<const uint4*>(src);
        k2[1] = *reinterpret_cast<const uint4*>(src + 8);
      }
    };
    // the first own unit's keys of this group, on their way early
    uint4 kw0[kHoldQ ? kSeg : 1][2][2];
    if constexpr (kHoldQ) {
      if (16 * wk < own) {
#pragma unroll
        for (int sg = 0; sg < kSeg; ++sg)
#pragma unroll
          for (int n = 0; n < 2; ++n) load_own_k(16 * wk, sg, n, kw0[sg][n]);
      }
    }
    int page[2];
    float ks[2], vs[2];
    load_pages(w, my_units, lane, page);
    load_scales(h, page, ks, vs);
    if (wk == 0) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float inv[2];
        uint4 qt[2][kSeg][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int sg = 0; sg < kSeg; ++sg) {
            if constexpr (kHoldQ) qt[i][sg][0] = qv[mt][i][sg][0], qt[i][sg][1] = qv[mt][i][sg][1];
            else load_q(mt, i, sg, qt[i][sg]);
          }
          unsigned top = 0;
#pragma unroll
          for (int sg = 0; sg < kSeg; ++sg)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint4& q4 = qt[i][sg][c];
              const uint32_t v[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const unsigned lo = v[x] & 0x7fffu, hi = (v[x] >> 16) & 0x7fffu;
                top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
              }
            }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // 2^-e brings the row's largest magnitude into [2^14, 2^15)
          int e = static_cast<int>(top >> 7) - 127 - 14;
          if (e < -100) e = -100;
          if (t == 0) s_factor[16 * (wr * MT + mt) + g + 8 * i] = pow2_bits(e) * p.scale_log2;
          inv[i] = pow2_bits(-e);
        }
#pragma unroll
        for (int sg = 0; sg < kSeg; ++sg)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t a[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4& q4 = qt[i][sg][s >> 1];
              const uint32_t x0 = s & 1 ? q4.z : q4.x, x1 = s & 1 ? q4.w : q4.y;
              a[i][0] = pack_f16x2(__uint_as_float(x0 << 16) * inv[i],
                                   __uint_as_float(x0 & 0xffff0000u) * inv[i]);
              a[i][1] = pack_f16x2(__uint_as_float(x1 << 16) * inv[i],
                                   __uint_as_float(x1 & 0xffff0000u) * inv[i]);
            }
            const uint32_t at =
                smem0 + T::kOffQ + (((wr * MT + mt) * T::kFrags + sg * 4 + s) * 32 + lane) * 16;
            st_shared_v4(at, a[0][0], a[1][0], a[0][1], a[1][1]);
          }
      }
    }

    float o[MT][kOut][4];
    float m[MT][2], l[MT][2], factor[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[mt][i] = -INFINITY;
        l[mt][i] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kOut; ++e)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[mt][e][x] = 0.f;
    }
    float c = pow2_bits(kCacheMinExp);  // the output's unit: the largest value scale so far
    float inv_c = pow2_bits(-kCacheMinExp);
    const uint8_t* qbase = smem + T::kOffQ + (wr * MT * T::kFrags * 32 + lane) * 16;

    // A score's factor (the row's power of two times the page's scale) is never 0,
    // be the row zero, the page zero or not there: 0 * -inf is not a number.  A
    // raw score is below 2^33, so what is raised to kTiny adds less than 2^-93.
    constexpr float kTiny = 1.1754944e-38f;  // 2^-126

    // Probabilities of a unit's raw scores sc (NT column tiles of 8 keys; -inf:
    // not seen), packed as the products' A operand: score factors row[.][.] times
    // f0 (first half of the column tiles) or f1, value weights w0 or w1 (times
    // the new unit c_new's inverse).  They are taken against the reference as it
    // stands; only where their sum says that one may have outgrown f16, or with
    // `look`, is the maximum found and the unit done again.
    auto soften = [&](auto nt, auto f16, auto& sc, const float (&row)[MT][2], float f0, float f1,
                      float w0, float w1, float c_new, bool look, auto& pf) {
      constexpr int NT = decltype(nt)::value;
      float shrink[MT][2];
      const float cr = c_new != c ? c / c_new : 1.f;
      if (c_new != c) c = c_new, inv_c = 1.f / c;
      w0 *= inv_c, w1 *= inv_c;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) shrink[mt][0] = shrink[mt][1] = cr;
#pragma unroll 1
      for (;;) {
        if (look) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = -INFINITY, y = -INFINITY;
#pragma unroll
              for (int n = 0; n < NT / 2; ++n) {
                x = fmax3(x, sc[mt][n][2 * i], sc[mt][n][2 * i + 1]);
                y = fmax3(y, sc[mt][n + NT / 2][2 * i], sc[mt][n + NT / 2][2 * i + 1]);
              }
              x = fmaxf(x * fmaxf(row[mt][i] * f0, kTiny), y * fmaxf(row[mt][i] * f1, kTiny));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              if (x > m[mt][i]) {
                const float a = ex2_approx(m[mt][i] - x);
                m[mt][i] = x;
                l[mt][i] *= a;
                shrink[mt][i] *= a;
              }
            }
        }
        float sum[MT][2];
        bool over = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // a row that has met no finite score keeps probabilities of 0
            const float ref = m[mt][i] == -INFINITY ? 0.f : kShift - m[mt][i];
            const float g0 = fmaxf(row[mt][i] * f0, kTiny), g1 = fmaxf(row[mt][i] * f1, kTiny);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float e0 = ex2_approx(fmaf(sc[mt][n][2 * i], n < NT / 2 ? g0 : g1, ref));
              const float e1 = ex2_approx(fmaf(sc[mt][n][2 * i + 1], n < NT / 2 ? g0 : g1, ref));
              s0 += e0;
              s1 += e1;
              const float wn = n < NT / 2 ? w0 : w1;
              (&pf[mt][n / 2].x)[2 * (n & 1) + i] =
                  decltype(f16)::value ? pack_f16x2(e0 * wn, e1 * wn)
                                       : pack_bf16x2(e0 * wn, e1 * wn);
            }
            sum[mt][i] = s0 + s1;
            over = over || sum[mt][i] > kMostSum || m[mt][i] == -INFINITY;
          }
        }
        if (look || !__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) l[mt][0] += sum[mt][0], l[mt][1] += sum[mt][1];
          break;
        }
        look = true;
      }
      bool any = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) any = any || shrink[mt][0] != 1.f || shrink[mt][1] != 1.f;
      if (__any_sync(0xffffffffu, any)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < kOut; ++e) {
            o[mt][e][0] *= shrink[mt][0];
            o[mt][e][1] *= shrink[mt][0];
            o[mt][e][2] *= shrink[mt][1];
            o[mt][e][3] *= shrink[mt][1];
          }
      }
    };
    // Own keys and values first, bf16, with the segment's end, while the cached
    // keys are on their way: units of 16 keys, the groups in turn, operands
    // straight from global memory.
    {
#pragma unroll 1
      for (int k0 = 16 * wk; k0 < own; k0 += 16 * WK) {
        float sc[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[mt][n][x] = 0.f;
#pragma unroll
        for (int sg = 0; sg < kSeg; ++sg) {
          uint4 kx[2][2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (kHoldQ && k0 == 16 * wk) {
              kx[n][0] = kw0[kHoldQ ? sg : 0][n][0];
              kx[n][1] = kw0[kHoldQ ? sg : 0][n][1];
            } else {
              load_own_k(k0, sg, n, kx[n]);
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint4 qx[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if constexpr (kHoldQ) qx[i][0] = qv[mt][i][sg][0], qx[i][1] = qv[mt][i][sg][1];
              else load_q(mt, i, sg, qx[i]);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint4& q0 = qx[0][s >> 1];
              const uint4& q1 = qx[1][s >> 1];
              const uint4 a = s & 1 ? make_uint4(q0.z, q1.z, q0.w, q1.w)
                                    : make_uint4(q0.x, q1.x, q0.y, q1.y);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const uint4& k4 = kx[n][s >> 1];
                mma_bf16(sc[mt][n], a, s & 1 ? k4.z : k4.x, s & 1 ? k4.w : k4.y);
              }
            }
          }
        }
        int end[MT][2];  // one past the last own key of the thread's rows
        float row[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = row_base + 16 * (wr * MT + mt) + g + 8 * i;
            end[mt][i] = r < R ? cache_own_end(w.rq.len, r / p.G, w.rq.n, p.bs) : 0;
            row[mt][i] = p.scale_log2;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (k0 + 8 * n + 2 * t + x >= end[mt][i]) sc[mt][n][2 * i + x] = -INFINITY;
          }
        uint4 pf[MT][1];
        soften(std::integral_constant<int, 2>{}, std::false_type{}, sc, row, 1.f, 1.f, 1.f, 1.f,
               fmaxf(c, kOwnUnit), true, pf);
        // A row's probability of an own key it does not see is 0, but 0 times a
        // value that is not finite is not: such values leave the product and
        // are added to the rows that see them.
        bool odd = false;
#pragma unroll
        for (int half = 0; half < kHalf; ++half)
#pragma unroll
          for (int part = 0; part < kCols / 8; ++part) {  // 8 dims at a time
            uint32_t vw[4][4];
            const int dim = 128 * half + kCols * run_of<BITS, D>(g) + 8 * part;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = k0 + 8 * (x >> 1) + 2 * t + (x & 1);
              uint4 v4 = make_uint4(0u, 0u, 0u, 0u);
              if (key < w.rq.n)
                v4 = *reinterpret_cast<const uint4*>(p.v + (w.rq.row0 + key) * p.v_sr + h * p.v_sh +
                                                     dim);
              vw[x][0] = v4.x, vw[x][1] = v4.y, vw[x][2] = v4.z, vw[x][3] = v4.w;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                if ((vw[x][y] & 0x7f80u) == 0x7f80u) vw[x][y] &= 0xffff0000u, odd = true;
                if ((vw[x][y] & 0x7f800000u) == 0x7f800000u) vw[x][y] &= 0xffffu, odd = true;
              }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const uint32_t b0 = __byte_perm(vw[0][y], vw[1][y], z ? 0x7632 : 0x5410);
                const uint32_t b1 = __byte_perm(vw[2][y], vw[3][y], z ? 0x7632 : 0x5410);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  mma_bf16(o[mt][half * kCols + 8 * part + 2 * y + z], pf[mt][0], b0, b1);
              }
            }
          }
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
          for (int key = k0; key < min(k0 + 16, w.rq.n); ++key) {
            const __nv_bfloat16* src = p.v + (w.rq.row0 + key) * p.v_sr + h * p.v_sh;
#pragma unroll
            for (int e = 0; e < kOut; ++e)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float y = __bfloat162float(
                    src[128 * (e / kCols) + kCols * run_of<BITS, D>(2 * t + x) + e % kCols]);
                if (isfinite(y)) continue;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (key < end[mt][i]) o[mt][e][2 * i + x] += y;
              }
          }
        }
      }
      // Cached probabilities are f16 and relative to the output's unit, which the
      // pages' scales alone are to set: it comes down to the largest of the group's
      // first units, but not so far that the own keys' output, in the new unit,
      // would pass 2^100 (what cached keys lose to that is below 2^-100 of it).
      if (16 * wk < own && my_units > 0) {
        unsigned top = 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < kOut; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const unsigned y = __float_as_uint(o[mt][e][x]) & 0x7fffffffu;
              top = max(top, y < 0x7f800000u ? y : 0u);
            }
        top = __reduce_max_sync(0xffffffffu, top);
        const unsigned most = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vs[0], vs[1])));
        const int want = kOwnExp - max(static_cast<int>(most >> 23) - 127, kCacheMinExp);
        const int down = max(min(127 + 99 - static_cast<int>(top >> 23), want), 0);
        const float grow = pow2_bits(down);
        c *= pow2_bits(-down);
        inv_c *= grow;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < kOut; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[mt][e][x] *= grow;
      }
    }

    __syncthreads();  // the queries' fragments
    // Held in registers where there is room; headdim 64, three blocks to an SM,
    // reads them for every unit (89.6 us against 93.9, 16 rows).
    constexpr bool kHoldF = kHoldQ && D != 64;
    uint4 qf[kHoldF ? MT : 1][T::kFrags];
    if constexpr (kHoldF) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int f = 0; f < T::kFrags; ++f) qf[mt][f] = load16(qbase + (mt * T::kFrags + f) * 512);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) factor[mt][i] = s_factor[16 * (wr * MT + mt) + g + 8 * i];

#pragma unroll 1
    for (int u = 0; u < my_units; ++u) {
      const int stage = consumed % STAGES;
      if ((u & 31) == 0 && u > 0) {
        load_pages(w, my_units, u + lane, page);
        load_scales(h, page, ks, vs);
      }
      float ks0 = __shfl_sync(0xffffffffu, ks[0], u & 31);
      float ks1 = __shfl_sync(0xffffffffu, ks[1], u & 31);
      const float vs0 = __shfl_sync(0xffffffffu, vs[0], u & 31);
      const float vs1 = __shfl_sync(0xffffffffu, vs[1], u & 31);
      const int p0 = __shfl_sync(0xffffffffu, page[0], u & 31);
      const int p1 = __shfl_sync(0xffffffffu, page[1], u & 31);
      const int key = key_lo + (wk + u * WK) * kUnit;
      // valid keys of the unit's 16-key halves
      const int nv0 = cache_page_ok(p0, p.num_pages) ? min(16, key_hi - key) : 0;
      const int nv1 = cache_page_ok(p1, p.num_pages) ? max(0, min(16, key_hi - key - 16)) : 0;
      const uint8_t* kt = smem + wk * STAGES * 2 * T::kUnitBytes + stage * 2 * T::kUnitBytes;
      const uint8_t* vt = kt + T::kUnitBytes;
      if (!(ok = mbar_wait_warp(gbar + 16 * stage, (consumed / STAGES) & 1, ab))) break;

      float sc[MT][4][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[mt][n][x] = 0.f;
      // 4 bits: where the unit's scales lie
      const uint8_t* sct = smem + T::kOffScale + (wk * STAGES + stage) * 4 * T::kSlot;
      const int pitch = two ? 16 : kUnit, half_off = two ? T::kSlot : 16;
      // the four scales of a group around the unit's key
      auto scales4 = [&](const uint8_t* of, int group, int key) {
        return *reinterpret_cast<const uint32_t*>(of + group * pitch + (key >> 4) * half_off +
                                                  (key & 12));
      };
      if constexpr (BITS == 4) {
        constexpr int kPart = D == 256 ? 2 : 1, kWords = D == 64 ? 2 : 4;
#pragma unroll
        for (int part = 0; part < kPart; ++part) {
          uint32_t kw[4][kWords];
          Cache4Scale sk[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int key = unit_key<BITS, D>(n, g);
            const uint8_t* src = tile4_at<D>(kt, key, (D / 8) * t + 16 * part);
            if constexpr (D == 64) {
              const uint2 x = *reinterpret_cast<const uint2*>(src);
              kw[n][0] = x.x, kw[n][1] = x.y;
            } else {
              const uint4 x = load16(src);
              kw[n][0] = x.x, kw[n][1] = x.y, kw[n][2] = x.z, kw[n][3] = x.w;
            }
            const uint32_t sc4 =
                scales4(sct, D == 64 ? t >> 1 : D == 128 ? t : 2 * t + part, key);
            sk[n] = cache4_prepare(__byte_perm(sc4, 0u, 0x0404 + 0x1010 * (key & 3)));
          }
#pragma unroll
          for (int x = 0; x < kWords; ++x) {
            uint32_t b[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) cache4_decode(kw[n][x], sk[n], b[n]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int f = 2 * (kWords * part + x) + s;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const uint4 a = kHoldF ? qf[kHoldF ? mt : 0][f]
                                       : load16(qbase + (mt * T::kFrags + f) * 512);
#pragma unroll
                for (int n = 0; n < 4; ++n) mma_f16(sc[mt][n], a, b[n][2 * s], b[n][2 * s + 1]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int sg = 0; sg < (BITS == 8 ? kSeg : 0); ++sg) {
        uint4 kw[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          kw[n] = load16(tile_at<D>(kt, 8 * n + key_of<D>(g), 4 * sg + t));
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t b[4][2];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t w = s == 0 ? kw[n].x : s == 1 ? kw[n].y : s == 2 ? kw[n].z : kw[n].w;
            b[n][0] = e4m3_lo(w);
            b[n][1] = e4m3_hi(w);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 a = kHoldF ? qf[kHoldF ? mt : 0][sg * 4 + s]
                                   : load16(qbase + (mt * T::kFrags + sg * 4 + s) * 512);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma_f16(sc[mt][n], a, b[n][0], b[n][1]);
          }
        }
      }
      const bool whole = nv0 == 16 && nv1 == 16;
      if (!whole) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if ((unit_key<BITS, D>(n, 2 * t + (x & 1)) & 15) >= (n < 2 ? nv0 : nv1))
                sc[mt][n][x] = -INFINITY;
      }
      uint4 pf[MT][2];
      soften(std::integral_constant<int, 4>{}, std::true_type{}, sc, factor, ks0, ks1, vs0, vs1,
             fmaxf(c, fmaxf(vs0, vs1)), false, pf);
      // P V: the four keys of a thread's fragment rows, 16 dims each (headdim
      // 64: 8).  What lies behind the last key may be anything, NaN included,
      // and is replaced by zero.
      // 4 bits: their scale is, which makes them zero.
      if constexpr (BITS == 4) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const int nv = kk == 0 ? nv0 : nv1;
#pragma unroll
          for (int half = 0; half < kHalf; ++half) {
            uint32_t vw[4][kCols / 8];
            Cache4Scale sv[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int key = unit_key<BITS, D>(2 * kk + y, 2 * t);  // and the one behind it
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint8_t* src = tile4_at<D>(vt, key + x, (kCols / 2) * g + 64 * half);
                if constexpr (D == 64) {
                  vw[2 * y + x][0] = *reinterpret_cast<const uint32_t*>(src);
                } else {
                  const uint2 w2 = *reinterpret_cast<const uint2*>(src);
                  vw[2 * y + x][0] = w2.x, vw[2 * y + x][1] = w2.y;
                }
              }
              const uint32_t sc4 =
                  scales4(sct + 2 * T::kSlot, (D == 64 ? g >> 2 : g >> 1) + 4 * half, key);
              uint32_t s2 = __byte_perm(sc4, 0u, 0x1404 + 0x1010 * (key & 3));
              if (!whole) {
                if ((key & 15) >= nv) s2 &= 0xffff0000u;
                if ((key & 15) + 1 >= nv) s2 &= 0x0000ffffu;
              }
              sv[y] = cache4_prepare(s2);
            }
#pragma unroll
            for (int y = 0; y < kCols / 8; ++y)
#pragma unroll
              for (int q = 0; q < 2; ++q) {  // the even dims, the odd ones
                uint32_t b0[4], b1[4];
                cache4_decode(__byte_perm(vw[0][y], vw[1][y], q ? 0x7632 : 0x5410), sv[0], b0);
                cache4_decode(__byte_perm(vw[2][y], vw[3][y], q ? 0x7632 : 0x5410), sv[1], b1);
#pragma unroll
                for (int z = 0; z < 4; ++z)
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt)
                    mma_f16(o[mt][half * kCols + 8 * y + 2 * z + q], pf[mt][kk], b0[z], b1[z]);
              }
          }
        }
      }
#pragma unroll
      for (int kk = 0; kk < (BITS == 8 ? 2 : 0); ++kk) {
        const int nv = kk == 0 ? nv0 : nv1;
#pragma unroll
        for (int half = 0; half < kHalf; ++half) {
          uint32_t vw[4][kCols / 4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = 8 * (x >> 1) + key_of<D>(2 * t + (x & 1));
            if constexpr (D == 64) {
              const uint2 w2 = *reinterpret_cast<const uint2*>(
                  tile_at<D>(vt, 16 * kk + r, g >> 1) + 8 * (g & 1));
              vw[x][0] = w2.x, vw[x][1] = w2.y;
            } else {
              const uint4 w4 = load16(tile_at<D>(vt, 16 * kk + r, 8 * half + key_of<D>(g)));
              vw[x][0] = w4.x, vw[x][1] = w4.y, vw[x][2] = w4.z, vw[x][3] = w4.w;
            }
            if (!whole && r >= nv) {
#pragma unroll
              for (int y = 0; y < kCols / 4; ++y) vw[x][y] = 0u;
            }
          }
#pragma unroll
          for (int y = 0; y < kCols / 4; ++y) {
            const uint32_t lo0 = __byte_perm(vw[0][y], vw[1][y], 0x5140);
            const uint32_t hi0 = __byte_perm(vw[0][y], vw[1][y], 0x7362);
            const uint32_t lo1 = __byte_perm(vw[2][y], vw[3][y], 0x5140);
            const uint32_t hi1 = __byte_perm(vw[2][y], vw[3][y], 0x7362);
            const uint32_t b[4][2] = {{e4m3_lo(lo0), e4m3_lo(lo1)},
                                      {e4m3_hi(lo0), e4m3_hi(lo1)},
                                      {e4m3_lo(hi0), e4m3_lo(hi1)},
                                      {e4m3_hi(hi0), e4m3_hi(hi1)}};
#pragma unroll
            for (int z = 0; z < 4; ++z)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma_f16(o[mt][half * kCols + 4 * y + z], pf[mt][kk], b[z][0], b[z][1]);
          }
        }
      }
      mbar_arrive_warp(gbar + 16 * stage + 8);
      ++consumed;
      if (wr == 0 && !(ok = ahead())) break;
    }

    // Join the groups: statistics first, then each group's output in a common
    // unit, summed.
    if (t == 0) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) s_m[wk * T::kRows + 16 * (wr * MT + mt) + g + 8 * i] = m[mt][i];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 1);
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 2);
      }
    if (lane == 0) s_c[warp] = c;
    __syncthreads();  // statistics written
    float c_all = s_c[0];
#pragma unroll
    for (int i = 1; i < WK * WR; ++i) c_all = fmaxf(c_all, s_c[i]);
    // The last kKept groups leave their outputs, the others add theirs to them.
    float* join = reinterpret_cast<float*>(smem + T::kOffJoin);
#pragma unroll 1
    for (int turn = 0; turn < WK / T::kKept; ++turn) {
      const bool add = turn == 1;
      if ((wk >= WK - T::kKept) != add) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 16 * (wr * MT + mt) + g + 8 * i;
            float top = s_m[r];
#pragma unroll
            for (int x = 1; x < WK; ++x) top = fmaxf(top, s_m[x * T::kRows + r]);
            const float f = m[mt][i] == -INFINITY ? 0.f : ex2_approx(m[mt][i] - top);
            const float fo = f * (c / c_all);
            if (t == 0) s_l[wk * T::kRows + r] = l[mt][i] * f;
            float* dst = join + ((wk % T::kKept) * T::kRows + r) * T::kPitch;
            // columns 2t and 2t + 1 of the column tiles are runs of kCols dims
#pragma unroll
            for (int half = 0; half < kHalf; ++half)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int dim = 128 * half + kCols * run_of<BITS, D>(2 * t + x);
#pragma unroll
                for (int e = 0; e < kCols; e += 4) {
                  float4 y = make_float4(o[mt][half * kCols + e][2 * i + x] * fo,
                                         o[mt][half * kCols + e + 1][2 * i + x] * fo,
                                         o[mt][half * kCols + e + 2][2 * i + x] * fo,
                                         o[mt][half * kCols + e + 3][2 * i + x] * fo);
                  float4* at = reinterpret_cast<float4*>(dst + dim + e);
                  if (add) {
                    const float4 z = *at;
                    y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
                  }
                  *at = y;
                }
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
      for (int x = 0; x < T::kKept; ++x) {
        const float4 y =
            *reinterpret_cast<const float4*>(join + (x * T::kRows + r) * T::kPitch + 4 * d4);
        a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
      }
      // no key (sum 0): output 0 and -inf; scores that are not numbers: NaN
      const bool none = top == -INFINITY && sum == 0.f;
      const float inv = none ? 0.f : c_all / sum;
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
  }  // pieces
  if (!ok && wr == 0 && lane == 0) {
    // Giving up: nothing may land in shared memory after the block is gone.
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
      mbar_wait_limited(gbar + 16 * (i % STAGES), (i / STAGES) & 1, kWaitLimitNs / 8);
  }
}

template <int BITS, int D, int MT, int WR, int WK, int STAGES>
cudaError_t launch_cache_tile(const CacheParams<BITS>& p, cudaStream_t stream) {
  using T = CacheTile<BITS, D, MT, WR, WK, STAGES>;
  auto kern = dfa_cache_fwd_kernel<BITS, D, MT, WR, WK, STAGES>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(p.blocks), dim3(T::kThreads), T::kSmem, stream, p);
}

template <int BITS, int D>
cudaError_t launch_cache_rows(const CacheParams<BITS>& p, int tile_rows, cudaStream_t stream) {
  if constexpr (D == 256) {
    if (tile_rows == 16) return launch_cache_tile<BITS, D, 1, 1, 4, 2>(p, stream);
    if (tile_rows == 32) return launch_cache_tile<BITS, D, 1, 2, 4, 2>(p, stream);
    return launch_cache_tile<BITS, D, 1, 4, 2, 3>(p, stream);
  } else {
    if (tile_rows == 16) return launch_cache_tile<BITS, D, 1, 1, 4, D == 64 ? 3 : 2>(p, stream);
    if (tile_rows == 32) return launch_cache_tile<BITS, D, 2, 1, 4, D == 64 ? 5 : 2>(p, stream);
    return launch_cache_wide(p, D, stream);
  }
}

}  // namespace
}  // namespace dfa
