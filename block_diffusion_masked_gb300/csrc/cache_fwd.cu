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
#include <cmath>
#include <type_traits>

#include "cache_fwd.cuh"
#include "device.cuh"
#include "dfa.h"

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


template <int D, int MT, int WR, int WK, int STAGES>
struct CacheTile {
  static constexpr int kThreads = 32 * WR * WK;
  static constexpr int kResident = D == 256 ? 1 : D == 64 && MT == 1 ? 3 : 2;  // blocks per SM
  static constexpr int kRows = 16 * MT * WR;
  static constexpr int kUnitBytes = kUnit * D;  // of k, and of v
  static constexpr int kRing = WK * STAGES * 2 * kUnitBytes;
  static constexpr int kFrags = (D / 64) * 4;  // k steps of Q K^T
  static constexpr int kQ = WR * MT * kFrags * 512;
  static constexpr int kPitch = D + 4;   // floats per row of a group's output at the join
  // Outputs that are kept at the join: every group's where there is room (one
  // token over 500: 11.7 us, 12.0 with half as many), else half as many, to
  // which the other half of the groups adds.
  static constexpr int kKept = kRows == 16 && D <= 128 ? WK : WK / 2;
  static constexpr int kJoin = kKept * kRows * kPitch * 4;
  // ring (1024-byte aligned) | join | q fragments | row factors | statistics | barriers
  static constexpr int kOffJoin = kRing;
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

// 16-byte chunk c of token row r inside a TMA tile: the tile's swizzle.
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

template <int D, int MT, int WR, int WK, int STAGES>
__global__ void __launch_bounds__(CacheTile<D, MT, WR, WK, STAGES>::kThreads,
                                  CacheTile<D, MT, WR, WK, STAGES>::kResident)
    dfa_cache_fwd_kernel(const __grid_constant__ CacheFwdParams p) {
  using T = CacheTile<D, MT, WR, WK, STAGES>;
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
  auto load_scales = [&](int h, const int* page, float* ks, float* vs) {
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
      for (int i = 0; i < 2; ++i)
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
      mbar_arrive_expect_tx(bar, (ok0 ? rows * D * 2 : 0) + (ok1 ? rows * D * 2 : 0));
      const int off = h * p.page_size + (key & (p.page_size - 1));
#pragma unroll
      for (int half = 0; half < kHalf; ++half) {
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
    auto load_q = [&](int mt, int i, int sg, uint4* q2) {
      const int r = row_base + 16 * (wr * MT + mt) + g + 8 * i;
      q2[0] = q2[1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < R) {
        const int tok = r / p.G, hq = h * p.G + (r - tok * p.G);
        const __nv_bfloat16* src =
            p.q + (w.rq.row0 + tok) * p.q_sr + hq * p.q_sh + 64 * sg + 16 * t;
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
            p.k + (w.rq.row0 + key) * p.k_sr + h * p.k_sh + 64 * sg + 16 * t;
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
            const int dim = D == 64 ? 8 * g : 128 * half + 16 * key_of<D>(g) + 8 * part;
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
                    src[128 * (e / kCols) + kCols * key_of<D>(2 * t + x) + e % kCols]);
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
#pragma unroll
      for (int sg = 0; sg < kSeg; ++sg) {
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
              if (8 * (n & 1) + key_of<D>(2 * t + (x & 1)) >= (n < 2 ? nv0 : nv1))
                sc[mt][n][x] = -INFINITY;
      }
      uint4 pf[MT][2];
      soften(std::integral_constant<int, 4>{}, std::true_type{}, sc, factor, ks0, ks1, vs0, vs1,
             fmaxf(c, fmaxf(vs0, vs1)), false, pf);
      // P V: the four keys of a thread's fragment rows, 16 dims each (headdim
      // 64: 8).  What lies behind the last key may be anything, NaN included,
      // and is replaced by zero.
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
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
                const int dim = 128 * half + kCols * key_of<D>(2 * t + x);
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

// The pieces of the segments that runs' ends have cut, joined: weights
// 2^(lse_s - max), a warp a row and query head, the pieces' outputs read once,
// a batch of them in flight together.  4 us for 16 rows, 9 us for 128 (304 and
// 152 blocks before it).
// Blocks (x, y): the cut that block x of the launch before answers for, rows y,
// y + gridDim.y, ... of kJoinWarps.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
    dfa_cache_join_kernel(const __grid_constant__ CacheFwdParams p) {
  constexpr int kVec = D / 32;  // floats per lane
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Cut cut = p.cuts[blockIdx.x];
  const int n = cut.pieces;
  if (n == 0) return;
  for (int r = warp + kJoinWarps * blockIdx.y; r < cut.rows; r += kJoinWarps * gridDim.y) {
    auto at = [&](int s) {
      return static_cast<long long>(s == 0 ? cut.slot0 : 2 * (cut.x0 + s)) * p.tile_rows + r;
    };
    // kBatch pieces at a time: their outputs and, a lane each, their lse are
    // read together, then weighed against the maximum so far
    constexpr int kBatch = 8;
    float top = -INFINITY, sum = 0.f, acc[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
    for (int s0 = 0; s0 < n; s0 += kBatch) {
      float y[kBatch][kVec];
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[s][i] = 0.f;
        if (s0 + s < n) {
          const float* src = p.part_o + at(s0 + s) * D + lane * kVec;
          if constexpr (kVec == 2) {
            *reinterpret_cast<float2*>(y[s]) = *reinterpret_cast<const float2*>(src);
          } else {
#pragma unroll
            for (int i = 0; i < kVec; i += 4)
              *reinterpret_cast<float4*>(y[s] + i) = *reinterpret_cast<const float4*>(src + i);
          }
        }
      }
      const float lse = lane < kBatch && s0 + lane < n ? p.part_lse[at(s0 + lane)] : -INFINITY;
      float m = lse;
#pragma unroll
      for (int off = kBatch / 2; off > 0; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      m = fmaxf(top, __shfl_sync(0xffffffffu, m, 0));
      const float ref = m == -INFINITY ? 0.f : m;
      const float shrink = ex2_approx(top - ref), wgt = ex2_approx(lse - ref);
      top = m;
      sum *= shrink;
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] *= shrink;
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const float ws = __shfl_sync(0xffffffffu, wgt, s);
        sum += ws;
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[i] = fmaf(ws, y[s][i], acc[i]);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tok = (cut.row_base + r) / p.G;
    const int hq = cut.h * p.G + (cut.row_base + r - tok * p.G);
    const long long row = cut.row0 + tok;
    __nv_bfloat16* dst = p.out + (row * p.H + hq) * D + lane * kVec;
#pragma unroll
    for (int i = 0; i < kVec; i += 2)
      *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0)
      p.lse[static_cast<long long>(hq) * p.rows + row] =
          sum == 0.f ? -INFINITY : (top + lg2_approx(sum)) * 0.6931471805599453f;
  }
}

// ------------------------------------------------------------------ host

// Tables of up to this many keys are not cut, see CachePlan.
constexpr int kWholeKeys = 512;

// The launch's shape for given sizes.
//
// tile_rows: query rows of a segment, the fewest that hold a request's rows, for
// every tile reads the keys anew (headdim 256: 32 rows 128 us in a tile of 32,
// 211 in one of 64; 64 rows 214 in one of 64, 225 in two of 32; headdim 64 and
// 128: above).  blocks: as many as are resident at once (CacheTile::kResident).
//
// whole: segments are not cut.  Short tables are not worth it, for one unit a
// segment needs no join (a launch) and no workspace: up to kWholeKeys keys, and
// up to twice that where the segments are half the blocks or more.  Measured,
// not cut against cut: 64 requests of 500 keys and 4 heads 14.7 and 18.5 us, of
// 1000 keys 22.3 and 26.2; one request of 250 keys 8.8 and 9.8, of 500 11.7 and
// 9.8 but for the second launch, of 1000 17.9 and 10.5.
//
// finish: units of 128 keys that a segment's end is taken to cost.  Too few, and
// blocks with many ends finish last; too many, and blocks with few do.  Measured
// (us; 32 ragged requests of up to 8192 tokens, a quarter of the heads for keys):
//                      finish 3     4     5     6     8    10
//   headdim 128,  16 rows    76    74    74    75    77    79
//   headdim 128,  32 rows   139   132   125   118   111   112
//   headdim 128, 128 rows   143   136   135   133   132   131
//   headdim  64, 128 rows   205   200   197   196   197   197
//   headdim 256,  16 rows   113   110   106   104   101   102
//   headdim 256,  64 rows   214   214   219   224   233   240
struct CachePlan {
  int tile_rows, blocks, finish;
  bool whole;
  // bytes of the pieces' outputs and lse and of the cuts
  long long workspace(int d) const {
    return whole ? 0
                 : 2LL * blocks * tile_rows * (d + 1) * 4 +
                       blocks * static_cast<long long>(sizeof(Cut));
  }
};
CachePlan cache_plan_for(int batch, int max_new, int G, int kv_heads, int d, long long keys,
                         int sms) {
  CachePlan c;
  const long long rows = static_cast<long long>(max_new) * G;
  c.tile_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : d == 256 ? 64 : 128;
  c.finish = d == 256 && c.tile_rows == 64 ? 4 : d < 256 && c.tile_rows == 16 ? 5 : 8;
  c.blocks = sms * (d == 256 || c.tile_rows == 128 ? 1 : d == 64 && c.tile_rows == 16 ? 3 : 2);
  const long long segments =
      static_cast<long long>(batch) * kv_heads * ((rows - 1) / c.tile_rows + 1);
  c.whole = keys <= kWholeKeys || (keys <= 2 * kWholeKeys && 2 * segments >= c.blocks);
  return c;
}

template <int D, int MT, int WR, int WK, int STAGES>
cudaError_t launch_cache_tile(const CacheFwdParams& p, cudaStream_t stream) {
  using T = CacheTile<D, MT, WR, WK, STAGES>;
  auto kern = dfa_cache_fwd_kernel<D, MT, WR, WK, STAGES>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(p.blocks), dim3(T::kThreads), T::kSmem, stream, p);
}

template <int D>
cudaError_t launch_cache_rows(const CacheFwdParams& p, int tile_rows, cudaStream_t stream) {
  if constexpr (D == 256) {
    if (tile_rows == 16) return launch_cache_tile<D, 1, 1, 4, 2>(p, stream);
    if (tile_rows == 32) return launch_cache_tile<D, 1, 2, 4, 2>(p, stream);
    return launch_cache_tile<D, 1, 4, 2, 3>(p, stream);
  } else {
    if (tile_rows == 16) return launch_cache_tile<D, 1, 1, 4, D == 64 ? 3 : 2>(p, stream);
    if (tile_rows == 32) return launch_cache_tile<D, 2, 1, 4, D == 64 ? 5 : 2>(p, stream);
    return launch_cache_wide(p, D, stream);
  }
}

int check_cache_sizes(int batch, int rows, int max_new, int heads, int kv_heads, int headdim,
                      int page_size, int max_pages) {
  const int most = max_new < rows ? max_new : rows;  // rows of one request
  if (batch < 0 || batch > 32768 || rows < 0 || rows > (1 << 30) || max_new < 0 ||
      most > (1 << 24) || heads < 1 || heads > (1 << 16) || kv_heads < 1 || kv_heads > heads ||
      heads % kv_heads || static_cast<long long>(most) * (heads / kv_heads) > (1 << 30) ||
      max_pages < 1 ||
      (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) ||
      static_cast<long long>(max_pages) * page_size > (1 << 30))
    return DFA_EINVAL;
  if (headdim != 64 && headdim != 128 && headdim != 256) return DFA_EUNSUPPORTED;
  return DFA_OK;
}

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" {

long long dfa_cache_workspace_bytes(int batch, int rows, int max_new, int heads, int kv_heads,
                                    int headdim, int page_size, int max_pages) {
  if (const int rc = check_cache_sizes(batch, rows, max_new, heads, kv_heads, headdim, page_size,
                                       max_pages))
    return rc;
  if (batch == 0 || rows == 0 || max_new == 0) return 0;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  if (max_new > rows) max_new = rows;
  return cache_plan_for(batch, max_new, heads / kv_heads, kv_heads, headdim,
                        static_cast<long long>(max_pages) * page_size, di.sms)
      .workspace(headdim);
}

int dfa_cache_forward(const void* q, const void* k, const void* v, const void* k_cache,
                      const void* v_cache, const float* k_scale, const float* v_scale,
                      const int* block_table, const int* cache_lens, const int* cu_new, void* out,
                      float* lse, void* workspace, long long workspace_bytes, int batch, int rows,
                      int max_new, int heads, int kv_heads, int headdim, int block_size,
                      int page_size, int num_pages, int max_pages, const long long* q_strides,
                      const long long* k_strides, const long long* v_strides,
                      dfa_stream_t stream) {
  if (const int rc = check_cache_sizes(batch, rows, max_new, heads, kv_heads, headdim, page_size,
                                       max_pages))
    return rc;
  if (block_size < 1 || num_pages < 1) return DFA_EINVAL;
  if (batch == 0 || rows == 0 || max_new == 0) return DFA_OK;
  auto aligned = [](const void* x, unsigned n) {
    return x && (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0;
  };
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(block_table, 4) || !aligned(cache_lens, 4) || !aligned(cu_new, 4) ||
      (workspace && !aligned(workspace, 16)) || (k == nullptr) != (v == nullptr) ||
      (k && (!aligned(k, 16) || !aligned(v, 16))))
    return DFA_EINVAL;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  if (max_new > rows) max_new = rows;
  const int G = heads / kv_heads, d = headdim;
  const CachePlan c = cache_plan_for(batch, max_new, G, kv_heads, d,
                                     static_cast<long long>(max_pages) * page_size, di.sms);
  if (!c.whole && (!workspace || workspace_bytes < c.workspace(d))) return DFA_EINVAL;
  CacheFwdParams p{};
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d),
                              static_cast<cuuint64_t>(kv_heads) * page_size,
                              static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), dims[1] * d};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(d < 128 ? d : 128),
                             static_cast<cuuint32_t>(c.tile_rows < 128 && page_size > kUnit ? kUnit
                                                                                      : page_size),
                             1};
  const CUtensorMapSwizzle swizzle =
      d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (const int rc = encode_map_u8(&p.tm_k, k_cache, 3, dims, strides, box, swizzle)) return rc;
  if (const int rc = encode_map_u8(&p.tm_v, v_cache, 3, dims, strides, box, swizzle)) return rc;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  auto set = [d](const long long* s, int n, long long* row, long long* head) {
    *row = s ? s[0] : static_cast<long long>(n) * d;
    *head = s ? s[1] : d;
    return (*row & 7) == 0 && (*head & 7) == 0;
  };
  if (!set(q_strides, heads, &p.q_sr, &p.q_sh) || !set(k_strides, kv_heads, &p.k_sr, &p.k_sh) ||
      !set(v_strides, kv_heads, &p.v_sr, &p.v_sh))
    return DFA_EINVAL;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.cache_lens = cache_lens;
  p.cu_new = cu_new;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  if (!c.whole) {
    const long long parts = 2LL * c.blocks * c.tile_rows;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = p.part_o + parts * d;
    p.cuts = reinterpret_cast<Cut*>(p.part_lse + parts);
  }
  p.status = di.status;
  p.batch = batch;
  p.rows = rows;
  p.max_new = max_new;
  p.H = heads;
  p.Hk = kv_heads;
  p.G = G;
  p.bs = block_size;
  p.page_size = page_size;
  p.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.tile_rows = c.tile_rows;
  p.blocks = c.blocks;
  p.unit = c.whole ? 0 : 128;
  p.finish = c.whole ? 1 : c.finish;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = d == 64    ? launch_cache_rows<64>(p, c.tile_rows, s)
                  : d == 128 ? launch_cache_rows<128>(p, c.tile_rows, s)
                             : launch_cache_rows<256>(p, c.tile_rows, s);
  if (e == cudaSuccess && !c.whole) {
    auto join = d == 64 ? dfa_cache_join_kernel<64>
                        : d == 128 ? dfa_cache_join_kernel<128> : dfa_cache_join_kernel<256>;
    const int rows = (c.tile_rows + kJoinWarps - 1) / kJoinWarps;
    const dim3 grid(c.blocks, rows < 16 ? rows : 16);
    e = launch_chained(join, grid, dim3(32 * kJoinWarps), 0, s, p);
  }
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

}  // extern "C"
