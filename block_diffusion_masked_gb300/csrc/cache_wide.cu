// Attention over the paged 8-bit cache for many query rows per key (more than
// 32: blocks of tokens times grouped heads), headdim 64 and 128, on the
// tensor cores' tcgen05 path.  The mathematics is that of cache_fwd.cu.
//
// One CTA per SM takes a run of units (cache.cuh) and walks its pieces: a piece
// is part of the keys of one request, key/value head and 128 query rows, in
// 128-key tiles, the own keys last.
//   TMA        raw e4m3 tiles of k and v, a box per page, into a ring;
//   convert    e4m3 -> f16 (exact) into the 128-byte-swizzled operand tiles
//              (own keys: bf16, copied from global memory), two of k and two
//              of v;
//   S = Q K^T  A = Q (f16 after the row's power of two, or bf16 for own keys;
//              put into shared memory by the warps that convert k, as soon as
//              the products with the Q before are complete), B = the key tile,
//              into one of two score buffers in TMEM;
//   softmax    against a reference that stands still but where probabilities
//              outgrow f16, times the value page's scale, into one of two
//              buffers of probabilities;
//   O += P V   A = P from TMEM, B = the value tile (keys outermost).
// Rings, buffers and barrier phases run on across pieces.
//
// Warps: 0-7 softmax (16 rows each, thread t on row t % 16, key columns
// [64 (t / 16), ...)), 8-11 convert k, 12-15 convert v, 16 and 17 load k and
// v, 18 issues S, 19 issues P V; the softmax warps take registers from the
// others (setmaxnreg).
//
// Measured, 128 rows, headdim 128, 32 ragged requests of up to 8192 tokens
// (342 MB, 81 GFLOP): 132 us, 2.6 TB/s, 610 TFLOP/s; 64 rows 124, headdim 64
// 197 (twice the heads: twice the scores).  Bound by the softmax warps: a tile
// takes them some 2400 cycles, of which its 128 x 128 exponentials need 512 of
// the special function units'; what is left is latency (waits that find their
// barrier complete, TMEM round trips) and the fetching of instructions, five
// roles on each scheduler: code that only got longer (the second half's scores
// loaded ahead, loops unrolled) made the kernel 30% slower, and rolled
// converters made it 5% faster.  Ends of pieces take 10 us each, of which the
// last tiles' chain is most, and the first products come after 11.
#include <type_traits>

#include "cache_fwd.cuh"
#include "dfa.h"

namespace dfa {
namespace {

// Instruction descriptor of tcgen05.mma kind::f16 with f16 A and B (format
// 0), f32 accumulator; fields as idesc_bf16.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 16 bytes of global memory into shared memory, zeros instead where !there.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// What the softmax needs to know of a cached tile: scales and keys of its
// eight 16-key groups, the largest value scale, whether every key is there.
struct TileInfo {
  float ks[8], vs[8];
  unsigned char keys[8];
  float vmax;
  int whole;
};

template <int D, int RS>
struct WideCfg {
  static constexpr int BM = 128, BN = 128;
  static constexpr int kSoftWarps = 8;
  static constexpr int kWarpConvV = 12, kWarpLoadK = 16, kWarpLoadV = 17, kWarpS = 18, kWarpPV = 19;
  static constexpr int kThreads = 32 * 20;
  // setmaxnreg split of the launch's 96 registers a thread:
  // 256 * 136 + 256 * 72 + 128 * 64 == 640 * 96
  static constexpr int kRegSoft = 136, kRegConv = 72, kRegRest = 64;
  static constexpr int kRaw = BN * D;       // a raw tile of k or of v, RS of each
  static constexpr int kTile = BN * D * 2;  // an operand tile, two of each
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + BM * D * 2;
  static constexpr int kOffV = kOffK + 2 * kTile;
  static constexpr int kOffRaw = kOffV + 2 * kTile;  // k, then v
  // Infos of the last kInfo cached tiles.  The load of tile i has seen tile
  // i - RS converted, so the product before the last before that one complete
  // and the scores two further back read: those up to i - RS - 4 are done with.
  static constexpr int kInfo = RS + 4 <= 8 ? 8 : 16;
  static_assert(RS + 4 <= kInfo, "infos still in use");
  // Row exponents of the last four versions of Q in f16.  A version is put
  // when the products with the one before are complete: three versions on, the
  // softmax is past the first tile of this one, where it reads them.
  static constexpr int kExps = 4;
  static constexpr int kOffInfo = kOffRaw + RS * 2 * kRaw;
  static constexpr int kOffExp = kOffInfo + kInfo * static_cast<int>(sizeof(TileInfo));
  static constexpr int kOffBar = kOffExp + kExps * BM;
  enum {
    BAR_Q = 0,
    BAR_RAWFULL = 1,                    // [RS] of k, [RS] of v
    BAR_RAWEMPTY = BAR_RAWFULL + 2 * RS,
    BAR_KFULL = BAR_RAWEMPTY + 2 * RS,  // [2] each, of the operand tiles
    BAR_KEMPTY = BAR_KFULL + 2,
    BAR_VFULL = BAR_KEMPTY + 2,
    BAR_VEMPTY = BAR_VFULL + 2,
    BAR_SFULL = BAR_VEMPTY + 2,    // [2] scores complete
    BAR_SREAD = BAR_SFULL + 2,     // [2] scores read
    BAR_PFULL = BAR_SREAD + 2,     // [2] probabilities written
    BAR_PVDONE = BAR_PFULL + 2,    // [2] P V complete: P free, the tile in O
    BAR_DRAIN = BAR_PVDONE + 2,    // every product complete
    NUM_BARS = BAR_DRAIN + 1
  };
  static constexpr int kOffTmem = kOffBar + NUM_BARS * 8;
  static constexpr int kOffAbort = kOffTmem + 4;
  static constexpr int kOffOdd = kOffAbort + 4;  // [4][4 warps]: own values that are not finite
  static_assert(kOffOdd % 4 == 0, "a piece's notes are read as a word");
  static constexpr int kSmem = kOffOdd + 16 + 1024;
  // TMEM: two buffers of scores, two of probabilities, O
  static constexpr int kTmemP = 2 * BN, kTmemO = kTmemP + BN, kTmemCols = 512;
  static_assert(kSmem <= 232448, "shared memory budget");
};

// Position in a ring of N: slot and round, counted up one at a time.
template <int N>
struct Ring {
  int slot = 0, round = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, ++round;
  }
};

template <int D, int RS>
__global__ void __launch_bounds__(WideCfg<D, RS>::kThreads, 1)
    dfa_cache_wide_kernel(const __grid_constant__ CacheFwdParams p) {
  using C = WideCfg<D, RS>;
  constexpr int BN = C::BN;
  constexpr int DH = D / 2;  // head dims of a softmax thread's half row
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - smem_u32(smem_raw));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  volatile unsigned char* s_odd = smem + C::kOffOdd;
  TileInfo* s_info = reinterpret_cast<TileInfo*>(smem + C::kOffInfo);
  signed char* s_exp = reinterpret_cast<signed char*>(smem + C::kOffExp);
  const AbortFlag ab{const_cast<int*>(abort_flag), p.status};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#define BAR(i) (sbase + C::kOffBar + 8 * (i))

  if (tid == 0) {
    mbar_init(BAR(C::BAR_Q), 4);
    for (int s = 0; s < 2 * RS; ++s) {
      mbar_init(BAR(C::BAR_RAWFULL + s), s < RS ? 2 : 1);  // k: the tile, its info
      mbar_init(BAR(C::BAR_RAWEMPTY + s), 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(C::BAR_KFULL + s), 4);
      mbar_init(BAR(C::BAR_KEMPTY + s), 1);
      mbar_init(BAR(C::BAR_VFULL + s), 4);
      mbar_init(BAR(C::BAR_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(C::BAR_SFULL + s), 1);
      mbar_init(BAR(C::BAR_SREAD + s), C::kSoftWarps);
      mbar_init(BAR(C::BAR_PFULL + s), C::kSoftWarps);
      mbar_init(BAR(C::BAR_PVDONE + s), 1);
    }
    mbar_init(BAR(C::BAR_DRAIN), 2);
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  bool bad = false;
  Piece w = first_piece(p, blockIdx.x, &bad);
  if (bad) atomicOr(p.status, kStatusIndex);
  if (w.b < 0) return;  // the whole block
  if (warp == C::kWarpPV) {
    tmem_alloc(sbase + C::kOffTmem, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::kOffTmem);

  // A piece's tiles: its cached keys, then the own keys its rows can see.
  struct Tiles {
    int h, row_base, R, key_lo, key_hi, nc, own, all;
  };
  auto tiles_of = [&](const Piece& x) {
    Tiles k;
    const int rt = row_tiles(p, x.rq);
    k.h = x.seg / rt;
    k.row_base = (x.seg - k.h * rt) * C::BM;
    k.R = x.rq.n * p.G;
    k.key_lo = piece_begin(p, x);
    k.key_hi = piece_end(p, x);
    k.nc = k.key_hi > k.key_lo ? (k.key_hi - k.key_lo + BN - 1) / BN : 0;
    k.own = 0;
    if (p.k != nullptr && x.last())
      k.own = cache_own_end(x.rq.len, min(k.R - 1, k.row_base + C::BM - 1) / p.G, x.rq.n, p.bs);
    k.all = k.nc + (k.own + BN - 1) / BN;
    return k;
  };
  // Pages of four tiles at a time, eight 16-key groups each: lane 8 t + g
  // holds group g of tile `first` + t.  The load (-1: nothing there) and the
  // look at what it brought are apart, a few tiles, so that nothing waits;
  // group_keys is 0 for a page that may not be followed.
  auto load_page = [&](const Piece& x, const Tiles& k, int first) {
    const int j = first + (lane >> 3);
    const int key = k.key_lo + BN * j + 16 * (lane & 7);
    return j < k.nc && key < k.key_hi
               ? p.block_table[static_cast<long long>(x.b) * p.max_pages + (key >> p.page_shift)]
               : -1;
  };
  auto keys_of = [&](const Tiles& k, int first, int page) {
    const int key = k.key_lo + BN * (first + (lane >> 3)) + 16 * (lane & 7);
    return cache_page_ok(page, p.num_pages) ? max(0, min(16, k.key_hi - key)) : 0;
  };

  if (warp >= C::kWarpLoadK) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegRest));
   if (warp == C::kWarpLoadK || warp == C::kWarpLoadV) {
    // ------------------------------------------------------------ loads
    // k and v each through a ring of its own: a tile of k is wanted, and its
    // place free again, well before the same tile of v.
    const bool isv = warp == C::kWarpLoadV;
    const CUtensorMap* map = isv ? &p.tm_v : &p.tm_k;
    const int full = C::BAR_RAWFULL + (isv ? RS : 0), empty = C::BAR_RAWEMPTY + (isv ? RS : 0);
    const uint32_t raw0 = sbase + C::kOffRaw + (isv ? RS * C::kRaw : 0);
    // The loads of k also write the tiles' infos; pages are asked for four tiles
    // ahead, scales three: they may come from memory under full load.
    auto load_scales = [&](int h, int page, float* ks, float* vs) {
      const bool has = !isv && cache_page_ok(page, p.num_pages);
      const long long at = static_cast<long long>(page) * p.Hk + h;
      *ks = has ? p.k_scale[at] : 0.f;
      *vs = has ? p.v_scale[at] : 0.f;
    };
    bool ok = true;
    int n = 0;  // cached tiles
    Ring<RS> at;
    for (; w.b >= 0 && ok; next_piece(p, w)) {
      const Tiles k = tiles_of(w);
      int page = load_page(w, k, 0), next_page = load_page(w, k, 4);
      int keys = keys_of(k, 0, page);
      float ks, vs, next_ks = 0.f, next_vs = 0.f;
      load_scales(k.h, page, &ks, &vs);
      for (int j = 0; j < k.nc; ++j, ++n) {
        if ((j & 3) == 0) {
          if (j > 0) {
            page = next_page, keys = keys_of(k, j, page);
            ks = next_ks, vs = next_vs;
            next_page = load_page(w, k, j + 4);
          }
        }
        // the first group of each page of this tile issues the page's box
        const int per = p.page_size >> 4;
        const bool mine = (lane >> 3) == (j & 3);
        const bool first = mine && (lane & 7) % per == 0;
        if (first && keys == 0 && k.key_lo + BN * j + 16 * (lane & 7) < k.key_hi)
          atomicOr(p.status, kStatusIndex);
        const bool load = first && keys > 0;
        const unsigned count = __popc(__ballot_sync(0xffffffffu, load));
        if (at.round > 0 &&
            !(ok = mbar_wait_warp(BAR(empty + at.slot), (at.round - 1) & 1, ab)))
          break;
        if (lane == 0) mbar_arrive_expect_tx(BAR(full + at.slot), count * p.page_size * D);
        __syncwarp();
        if (load)
          tma_load_3d(raw0 + at.slot * C::kRaw + (lane & 7) * 16 * D, map, BAR(full + at.slot), 0,
                      k.h * p.page_size, page);
        if (!isv) {
          if ((j & 3) == 1) load_scales(k.h, next_page, &next_ks, &next_vs);
          float vmax = vs;
#pragma unroll
          for (int off = 1; off < 8; off <<= 1)
            vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
          const unsigned there = __ballot_sync(0xffffffffu, keys == 16) >> (8 * (j & 3));
          if (mine) {
            TileInfo& info = s_info[n & (C::kInfo - 1)];
            info.ks[lane & 7] = ks;
            info.vs[lane & 7] = vs;
            info.keys[lane & 7] = static_cast<unsigned char>(keys);
            if ((lane & 7) == 0) {
              info.vmax = vmax;
              info.whole = (there & 0xffu) == 0xffu;
            }
          }
          mbar_arrive_warp(BAR(full + at.slot));
        }
        __syncwarp();
        at.next();
      }
    }
    if (!ok && lane == 0)  // giving up: what is in flight lands first
      for (int i = 1; i <= RS && i <= at.round * RS + at.slot; ++i) {
        const int n = at.round * RS + at.slot - i;
        mbar_wait_limited(BAR(full + n % RS), (n / RS) & 1, 100000000ull);
      }
    __syncwarp();
   } else if (warp == C::kWarpS || warp == C::kWarpPV) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      bool ok = true;
      int n = 0, q = 0;  // tiles, versions of Q
      for (; w.b >= 0 && ok; next_piece(p, w)) {
        const Tiles k = tiles_of(w);
#pragma unroll 1
        for (int j = 0; j < k.all; ++j, ++n) {
          const int b = n & 1;
          const uint32_t done = ((n >> 1) - 1) & 1, now = (n >> 1) & 1;
          if (warp == C::kWarpS) {
            // Q as f16 at the first cached tile, as bf16 at the first own one
            if ((j == 0 || j == k.nc) && !(ok = mbar_wait(BAR(C::BAR_Q), q++ & 1, ab))) break;
            if (!(ok = mbar_wait(BAR(C::BAR_KFULL + b), now, ab))) break;
            if (n >= 2 && !(ok = mbar_wait(BAR(C::BAR_SREAD + b), done, ab))) break;
            tc_fence_after();
            const uint32_t id = j < k.nc ? idesc_f16(C::BM, BN, false, false)
                                         : idesc_bf16(C::BM, BN, false, false);
            uint64_t qd = sdesc_sw128(sbase + C::kOffQ, 16, 1024);
            uint64_t kd = sdesc_sw128(sbase + C::kOffK + b * C::kTile, 16, 1024);
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {  // descriptors count 16 bytes
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss(tmem + b * BN, qd + 2 * kk, kd + 2 * kk, id, c > 0 || kk > 0 ? 1u : 0u);
              qd += BN * 128 / 16;
              kd += BN * 128 / 16;
            }
            mma_commit(BAR(C::BAR_SFULL + b));
            mma_commit(BAR(C::BAR_KEMPTY + b));
          } else {
            if (!(ok = mbar_wait(BAR(C::BAR_VFULL + b), now, ab))) break;
            if (!(ok = mbar_wait(BAR(C::BAR_PFULL + b), now, ab))) break;
            tc_fence_after();
            const uint32_t id =
                j < k.nc ? idesc_f16(C::BM, D, false, true) : idesc_bf16(C::BM, D, false, true);
            uint64_t vd = sdesc_sw128(sbase + C::kOffV + b * C::kTile, BN * 128, 1024);
            uint32_t pa = tmem + C::kTmemP + b * (BN / 2);
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts(tmem + C::kTmemO, pa + 8 * kk, vd + kk * (16 * 128 / 16), id,
                       j > 0 || c > 0 || kk > 0 ? 1u : 0u);
              pa += 32;
              vd += 64 * 128 / 16;
            }
            mma_commit(BAR(C::BAR_VEMPTY + b));
            mma_commit(BAR(C::BAR_PVDONE + b));
          }
        }
      }
      mma_commit(BAR(C::BAR_DRAIN));
      mbar_wait_limited(BAR(C::BAR_DRAIN), 0, 1000000000ull);
    }
    __syncwarp();
   }
  } else if (warp >= C::kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegConv));
    // ------------------------------------------------------------ conversion
    const bool isv = warp >= C::kWarpConvV;
    const int cw = warp & 3;             // warp of its four
    const int c = cw * 32 + lane;        // 0 .. 127
    const int full = isv ? C::BAR_VFULL : C::BAR_KFULL, empty = full + 2;
    const uint32_t tiles0 = sbase + (isv ? C::kOffV : C::kOffK);
    const uint32_t raw0 = sbase + C::kOffRaw + (isv ? RS * C::kRaw : 0);
    const int rawfull = C::BAR_RAWFULL + (isv ? RS : 0);
    const int rawempty = C::BAR_RAWEMPTY + (isv ? RS : 0);
    // e4m3 -> f16: a thread turns 16 values (a 16-byte piece) into two pieces
    // of its row.  Eight lanes, one phase of a shared-memory access, take four
    // neighbouring pieces of rows r and r ^ 5: under either tile's swizzle
    // their reads and their writes fall on different banks.  From 32 rows to
    // the next the addresses differ by a constant.
    // `mask`: rows past their group's keys (lane g: those of group g) become
    // zero, whatever the raw bytes are there, NaN included.
    const int pc = lane & 3;
    const int r0 = 8 * cw + ((lane >> 3) ^ (5 * ((lane >> 2) & 1)));  // row of 32
    const uint32_t put_at = r0 * 128 + (((2 * pc) ^ (r0 & 7)) << 4);
    const uint32_t get_at = D == 64 ? r0 * 64 + ((pc ^ ((r0 >> 1) & 3)) << 4)
                                    : r0 * 128 + ((pc ^ (r0 & 7)) << 4);
    auto convert = [&](uint32_t raw, uint32_t dst, bool mask, int group_keys) {
      uint32_t from = raw + get_at, to = dst + put_at;
#pragma unroll 1
      for (int i = 0; i < 4; ++i, from += 32 * D, to += 32 * 128) {
        uint4 x[D / 64];
#pragma unroll
        for (int f = 0; f < D / 64; ++f) x[f] = lds128(from ^ (64 * f));
        if (mask && (r0 & 15) >= __shfl_sync(0xffffffffu, group_keys, 2 * i + (r0 >> 4))) {
#pragma unroll
          for (int f = 0; f < D / 64; ++f) x[f] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int f = 0; f < D / 64; ++f) {
          st_shared_v4(to + f * (BN * 128), e4m3_lo(x[f].x), e4m3_hi(x[f].x), e4m3_lo(x[f].y),
                       e4m3_hi(x[f].y));
          st_shared_v4((to ^ 16) + f * (BN * 128), e4m3_lo(x[f].z), e4m3_hi(x[f].z),
                       e4m3_lo(x[f].w), e4m3_hi(x[f].w));
        }
      }
    };
    // Own rows as they are, and Q: all copies of a tile are in flight at once,
    // straight into place; a thread looks again only at what it copied itself.
    auto copy_own = [&](const Piece& x, const Tiles& k, int first, uint32_t dst) {
      const __nv_bfloat16* src = isv ? p.v + x.rq.row0 * p.v_sr + k.h * p.v_sh
                                     : p.k + x.rq.row0 * p.k_sr + k.h * p.k_sh;
      const long long sr = isv ? p.v_sr : p.k_sr;
#pragma unroll 1
      for (int i = 0; i < D / 8; ++i) {
        const int at = i * 128 + c, r = at / (D / 8), u = at % (D / 8);
        const bool there = first + r < x.rq.n;
        copy16_async(dst + (u >> 3) * (BN * 128) + r * 128 + (((u ^ r) & 7) << 4),
                     src + (there ? first + r : 0) * sr + 8 * u, there);
      }
    };
    auto copy_q = [&](const Piece& x, const Tiles& k) {
#pragma unroll 1
      for (int i = 0; i < D / 8; ++i) {
        const int at = i * 128 + c, row = at / (D / 8), u = at % (D / 8);
        const int r = min(k.row_base + row, k.R - 1);
        const int tok = r / p.G, hq = k.h * p.G + (r - tok * p.G);
        const uint32_t to = (u >> 3) * (C::BM * 128) + row * 128 + (((u ^ row) & 7) << 4);
        copy16_async(sbase + C::kOffQ + to,
                     p.q + (x.rq.row0 + tok) * p.q_sr + hq * p.q_sh + 8 * u,
                     k.row_base + row < k.R);
      }
    };
    // Values that are not finite are kept out of the product (their weight is 0
    // in rows that do not see them) and noted.
    auto drop_odd = [&](uint32_t dst) {
      bool odd = false;
#pragma unroll 1
      for (int i = 0; i < D / 8; ++i) {
        const int at = i * 128 + c, r = at / (D / 8), u = at % (D / 8);
        const uint32_t to = dst + (u >> 3) * (BN * 128) + r * 128 + (((u ^ r) & 7) << 4);
        const uint4 y = lds128(to);
        uint32_t v[4] = {y.x, y.y, y.z, y.w};
        bool drop = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u, drop = true;
          if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0xffffu, drop = true;
        }
        if (drop) st_shared_v4(to, v[0], v[1], v[2], v[3]);
        odd = odd || drop;
      }
      return odd;
    };
    // Q from bf16 to f16 after a power of two of each row's, whose exponents go
    // to `exps`.
    auto scale_q = [&](signed char* exps) {
#pragma unroll 1
      for (int i = 0; i < D / 8; ++i) {
        const int at = i * 128 + c, row = at / (D / 8), u = at % (D / 8);
        // 16-byte unit u of a row: 64-dim chunk u / 8, swizzled by the row
        const uint32_t to =
            sbase + C::kOffQ + (u >> 3) * (C::BM * 128) + row * 128 + (((u ^ row) & 7) << 4);
        const uint4 y = lds128(to);
        uint32_t v[4] = {y.x, y.y, y.z, y.w};
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const unsigned lo = v[e] & 0x7fffu, hi = (v[e] >> 16) & 0x7fffu;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
#pragma unroll
        for (int off = 1; off < D / 8; off <<= 1)
          top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        int e = static_cast<int>(top >> 7) - 127 - 14;
        if (e < -100) e = -100;
        const float inv = pow2_bits(-e);
        if (u == 0) exps[row] = static_cast<signed char>(e);
#pragma unroll
        for (int z = 0; z < 4; ++z)
          v[z] = pack_f16x2(__uint_as_float(v[z] << 16) * inv,
                            __uint_as_float(v[z] & 0xffff0000u) * inv);
        st_shared_v4(to, v[0], v[1], v[2], v[3]);
      }
    };
    bool ok = true;
    int n = 0, owns = 0;  // operand tiles, pieces with own keys
    int q = 0;            // versions of Q in f16
    bool odd = false;     // the piece has own values that are not finite
    Ring<RS> at;
    for (; w.b >= 0 && ok; next_piece(p, w)) {
      const Tiles k = tiles_of(w);
      int keys = 0, next_page = -1;
      if (isv) keys = keys_of(k, 0, load_page(w, k, 0));
      for (int j = 0; j < k.all; ++j, ++n) {
        const int b = n & 1;
        if (isv && (j & 3) == 0) {
          if (j > 0) keys = keys_of(k, j, next_page);
          next_page = load_page(w, k, j + 4);
        }
        // A tile of k that comes with a new Q: the first cached one, the first
        // own one.  Q may be replaced when the products with it are complete,
        // which is when this tile is ready already.
        const bool with_q = !isv && (j == 0 || j == k.nc);
        if (with_q && n == 0) copy_q(w, k);
        if (n >= 2 && !(ok = mbar_wait_warp(BAR(empty + b), ((n >> 1) - 1) & 1, ab))) break;
        const uint32_t dst = tiles0 + b * C::kTile;
        if (j < k.nc) {
          if (!(ok = mbar_wait_warp(BAR(rawfull + at.slot), at.round & 1, ab))) break;
          const uint32_t src = raw0 + at.slot * C::kRaw;
          const int group_keys = __shfl_sync(0xffffffffu, keys, 8 * (j & 3) + (lane & 7));
          convert(src, dst, isv && __any_sync(0xffffffffu, group_keys < 16), group_keys);
          mbar_arrive_warp(BAR(rawempty + at.slot));
          at.next();
        } else {
          if (j == k.nc) {
            ++owns;
            odd = false;
          }
          copy_own(w, k, BN * (j - k.nc), dst);
        }
        if (with_q) {
          if (n > 0) {
            if (!(ok = mbar_wait_warp(BAR(empty + (b ^ 1)), ((n - 1) >> 1) & 1, ab))) break;
            copy_q(w, k);
          }
          copy16_wait();
          if (j < k.nc) scale_q(s_exp + (q++ & (C::kExps - 1)) * C::BM);
          fence_proxy_async_smem();
          mbar_arrive_warp(BAR(C::BAR_Q));
        }
        if (j >= k.nc) {
          copy16_wait();
          if (isv) {
            // Each warp writes a note of its own, four to a piece with own keys,
            // a word for each of the last four such pieces.  This tile's place
            // was free when the products two tiles back were complete: the
            // softmax has read out all such pieces but this and two before it.
            odd = __any_sync(0xffffffffu, drop_odd(dst)) || odd;
            if (lane == 0) s_odd[4 * (owns & 3) + cw] = odd;
          }
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(BAR(full + b));
      }
    }
    copy16_wait();  // giving up: nothing lands after the block is gone
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegSoft));
    // ------------------------------------------------------------ softmax
    const int half = lane >> 4;
    const int lb = (warp & 3) * 32 + (warp >> 2) * 16;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lb) << 16);
    bool ok = true;
    // tiles, cached ones, pieces with own keys, versions of Q
    int n = 0, cached = 0, owns = 0, q = 0;
    for (; w.b >= 0 && ok; next_piece(p, w)) {
      const Tiles k = tiles_of(w);
      const int r = k.row_base + lb + (lane & 15);  // row of the request and head
      const int tok = min(r, k.R - 1) / p.G;
      const int hq = k.h * p.G + (min(r, k.R - 1) - tok * p.G);
      const int end = r < k.R ? cache_own_end(w.rq.len, tok, w.rq.n, p.bs) : 0;
      float factor = 0.f;  // undoes the row's power of two, with the softmax scale
      float m = -INFINITY, l = 0.f;
      float c = pow2_bits(kCacheMinExp), inv_c = pow2_bits(-kCacheMinExp);  // unit of O
      // One tile, in three copies so that the common one is short: cached with
      // all its keys, cached with some, own keys (bf16, row by row).
      constexpr int kWhole = 0, kPart = 1, kOwn = 2;
      auto tile = [&](auto kind, int j, const TileInfo& info) -> bool {
        constexpr int kKind = decltype(kind)::value;
        const int b = n & 1;
        const uint32_t s_col = t_lane + b * BN, p_col = t_lane + C::kTmemP + b * (BN / 2);
        // Of 32 keys of the half row: score factors and value weights of their two
        // groups (never 0, where a group has no keys: 0 * -inf is not a
        // number), and which of them count.
        auto groups = [&](int x, float* f, float* wt) {
          if constexpr (kKind == kOwn) {
            f[0] = f[1] = p.scale_log2;
            wt[0] = wt[1] = inv_c;
          } else {
            const float2 ks = *reinterpret_cast<const float2*>(info.ks + 4 * half + 2 * x);
            const float2 vs = *reinterpret_cast<const float2*>(info.vs + 4 * half + 2 * x);
            f[0] = fmaxf(factor * ks.x, 1.1754944e-38f);
            f[1] = fmaxf(factor * ks.y, 1.1754944e-38f);
            wt[0] = vs.x * inv_c, wt[1] = vs.y * inv_c;
          }
        };
        auto scores = [&](int x, uint32_t* sr) {
          tmem_ld_half<32, 64>(s_col + 32 * x, sr);
          tmem_wait_ld();
          tmem_pin<32>(sr);
          if constexpr (kKind != kWhole) {
            uint32_t keep;
            if constexpr (kKind == kPart) {
              const int k0 = info.keys[4 * half + 2 * x], k1 = info.keys[4 * half + 2 * x + 1];
              keep = ((1u << k0) - 1u) | (((1u << k1) - 1u) << 16);
            } else {
              const int left = end - BN * (j - k.nc) - 64 * half - 32 * x;
              keep = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t mk = bit_spread(keep, e);
              sr[e] = (sr[e] & mk) | (0xff800000u & ~mk);
            }
          }
        };
        const float c_new = fmaxf(c, kKind == kOwn ? kOwnUnit : info.vmax);
        float shrink = 1.f;
        if (c_new != c) {
          shrink = c / c_new;
          c = c_new;
          inv_c = 1.f / c;
        }
        if (n >= 2 && !mbar_wait_warp(BAR(C::BAR_PVDONE + b), ((n >> 1) - 1) & 1, ab)) return false;
        tc_fence_after();
        // The probabilities are taken against the reference as it stands; only
        // where their sum says that one may have outgrown f16, or where the
        // piece begins, is the maximum looked for and the tile done (again).
        // All loops are rolled: with five roles on a scheduler the fetching of
        // instructions costs more than their issue.
        bool look = j == 0;
#pragma unroll 1
        for (;;) {
          if (look) {
            float top = m;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              uint32_t sr[32];
              float f[2], wt[2];
              groups(x, f, wt);
              scores(x, sr);
              top = fmaxf(top, fmaxf(max_tree<16>(sr) * f[0], max_tree<16>(sr + 16) * f[1]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            if (top > m) {
              const float a = ex2_approx(m - top);
              m = top;
              l *= a;
              shrink *= a;
            }
          }
          const float ref = m == -INFINITY ? 0.f : kShift - m;
          const uint64_t ref2 = f2_pack(ref, ref);
          uint64_t acc[2] = {0ull, 0ull};
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            uint32_t sr[32], pk[16];
            float f[2], wt[2];
            groups(x, f, wt);
            scores(x, sr);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint64_t f2 = f2_pack(f[i], f[i]), w2 = f2_pack(wt[i], wt[i]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int at = 16 * i + 2 * e;
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[at]), __uint_as_float(sr[at + 1])), f2,
                                 ref2),
                          x0, x1);
                const uint64_t pr = f2_pack(ex2_approx(x0), ex2_approx(x1));
                acc[e & 1] = f2_add(acc[e & 1], pr);
                f2_unpack(f2_mul(pr, w2), x0, x1);
                pk[8 * i + e] = kKind == kOwn ? pack_bf16x2(x0, x1) : pack_f16x2(x0, x1);
              }
            }
            tmem_st_half<16, 32>(p_col + 16 * x, pk);
          }
          float a0, a1;
          f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
          a0 += a1;
          if (look || !__any_sync(0xffffffffu, a0 > kMostSum || m == -INFINITY)) {
            l += a0;
            break;
          }
          look = true;
        }
        tc_fence_before();
        mbar_arrive_warp(BAR(C::BAR_SREAD + b));
        // a moved reference or unit: O of the tiles before, once they are in it
        if (j > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {
          if (!mbar_wait_warp(BAR(C::BAR_PVDONE + (b ^ 1)), ((n - 1) >> 1) & 1, ab)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < DH / 16; ++x) {
            uint32_t o[16];
            tmem_ld_half<16, DH>(t_lane + C::kTmemO + 16 * x, o);
            tmem_wait_ld();
            tmem_pin<16>(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * shrink);
            tmem_st_half<16, DH>(t_lane + C::kTmemO + 16 * x, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(BAR(C::BAR_PFULL + b));
        return true;
      };
#pragma unroll 1
      for (int j = 0; j < k.all && ok; ++j) {
        if (!(ok = mbar_wait_warp(BAR(C::BAR_SFULL + (n & 1)), (n >> 1) & 1, ab))) break;
        const TileInfo& info = s_info[cached & (C::kInfo - 1)];
        if (j >= k.nc) {
          ok = tile(std::integral_constant<int, kOwn>{}, j, info);
        } else {
          if (j == 0) {
            const int e = s_exp[(q++ & (C::kExps - 1)) * C::BM + lb + (lane & 15)];
            factor = pow2_bits(e) * p.scale_log2;
          }
          if (info.whole) ok = tile(std::integral_constant<int, kWhole>{}, j, info);
          else ok = tile(std::integral_constant<int, kPart>{}, j, info);
          ++cached;
        }
        if (ok) ++n;
      }

      // -------------------------------------------------------- read-out
      if (!ok) break;
      if (k.all > 0 &&
          !(ok = mbar_wait_warp(BAR(C::BAR_PVDONE + ((n - 1) & 1)), ((n - 1) >> 1) & 1, ab)))
        break;
      tc_fence_after();
      if (k.own > 0) ++owns;
      const bool odd = k.own > 0 && *reinterpret_cast<volatile int*>(s_odd + 4 * (owns & 3)) != 0;
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const bool none = m == -INFINITY && l == 0.f;
      const float inv = none ? 0.f : c / l;
      const float lse2 = none ? -INFINITY : m - kShift + lg2_approx(l);
      const bool single = w.whole();
      const long long at =
          (2LL * blockIdx.x + (w.first ? 0 : 1)) * C::BM + lb + (lane & 15);
      __nv_bfloat16* dst =
          p.out + ((w.rq.row0 + static_cast<long long>(tok)) * p.H + hq) * D + half * DH;
      float* part = p.part_o + at * D + half * DH;
#pragma unroll
      for (int x = 0; x < DH / 32; ++x) {
        uint32_t o[32];
        if (k.all > 0) {
          tmem_ld_half<32, DH>(t_lane + C::kTmemO + 32 * x, o);
          tmem_wait_ld();
          tmem_pin<32>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (odd) {  // own values that are not finite, for the rows that see them
#pragma unroll 1
          for (int key = 0; key < end; ++key) {
            const __nv_bfloat16* v =
                p.v + (w.rq.row0 + key) * p.v_sr + k.h * p.v_sh + half * DH + 32 * x;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float y = __bfloat162float(v[e]);
              if (!isfinite(y)) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
            }
          }
        }
        if (r < k.R) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
          if (single) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t v[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                v[y] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * y]),
                                   __uint_as_float(o[8 * e + 2 * y + 1]));
              st_global_v4(dst + 32 * x + 8 * e, v[0], v[1], v[2], v[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st_global_v4(part + 32 * x + 4 * e, o[4 * e], o[4 * e + 1], o[4 * e + 2],
                           o[4 * e + 3]);
          }
        }
      }
      if (r < k.R && half == 0) {
        if (single)
          p.lse[static_cast<long long>(hq) * p.rows + w.rq.row0 + tok] =
              lse2 * 0.6931471805599453f;
        else
          p.part_lse[at] = lse2;
      }
    }
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpPV) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int RS>
cudaError_t launch_wide(const CacheFwdParams& p, cudaStream_t stream) {
  using C = WideCfg<D, RS>;
  auto kern = dfa_cache_wide_kernel<D, RS>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(p.blocks), dim3(C::kThreads), C::kSmem, stream, p);
}

}  // namespace

cudaError_t launch_cache_wide(const CacheFwdParams& p, int headdim, cudaStream_t stream) {
  if (headdim == 64) return launch_wide<64, 6>(p, stream);
  if (headdim == 128) return launch_wide<128, 2>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace dfa
