// What the kernels of attention over the paged cache share: parameters, the
// walk over a block's run of units, conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache.cuh"
#include "params.cuh"
#include "sm100.cuh"

namespace dfa {

// A segment that runs' ends have cut, for the launch that joins its pieces:
// `pieces` of them (0: nothing to join), the first in slot `slot0`, the s-th in
// slot 2 (x0 + s); the segment's head, first row and rows, and its request's
// first row.
struct Cut {
  int pieces, slot0, x0, h, row_base, rows, row0, unused;
};

struct CacheFwdParams {
  CUtensorMap tm_k, tm_v;  // (headdim, kv_heads * page_size, pages) bytes
  const __nv_bfloat16* q;  // (rows, heads, headdim), strided
  const __nv_bfloat16* k;  // own keys (rows, kv_heads, headdim) or null
  const __nv_bfloat16* v;
  long long q_sr, q_sh, k_sr, k_sh, v_sr, v_sh;
  const float* k_scale;  // (pages, kv_heads)
  const float* v_scale;
  const int* block_table;
  const int* cache_lens;
  const int* cu_new;
  __nv_bfloat16* out;  // (rows, heads, headdim)
  float* lse;          // (heads, rows)
  float* part_o;       // (2 * blocks, tile rows, headdim): pieces of split segments
  float* part_lse;     // (2 * blocks, tile rows), log2
  Cut* cuts;           // (blocks), each written by the block it is numbered after
  unsigned* status;
  int batch, rows, max_new, H, Hk, G, bs;
  int page_size, page_shift, num_pages, max_pages;
  int tile_rows;  // query rows of a segment
  int unit;       // keys per unit of the split, 0: segments are not cut
  int finish;     // units a segment's end counts for
  int blocks;     // blocks of the launch
  float scale_log2;
};

// One request's sizes, checked: a length past its table or rows past the
// packed ones are errors, and the request is then taken as empty.
struct Request {
  int len, row0, n;
};
__device__ __forceinline__ Request load_request(const CacheFwdParams& p, int b, bool* bad) {
  const int len = p.cache_lens[b], r0 = p.cu_new[b], r1 = p.cu_new[b + 1];
  const bool ok = len >= 0 && len <= p.max_pages * p.page_size && r0 >= 0 && r1 >= r0 &&
                  r1 <= p.rows && r1 - r0 <= p.max_new;
  if (!ok) {
    *bad = true;
    return {0, 0, 0};
  }
  return {len, r0, r1 - r0};
}

// A block's run of units, piece by piece: the part of it that lies in one
// segment.  Every warp walks for itself; all lanes hold the same values.
struct Piece {
  int b;         // request; -1: the run is done
  int seg;       // head * row tiles + row tile
  int u0, u1;    // units of the segment the piece covers
  int keys;      // key units of the segment
  int first;     // the run begins with this piece
  long long left;  // units of the run after this piece
  Request rq;
  // The piece has the segment's end (own keys, read-out of a whole segment).
  __device__ __forceinline__ bool last() const { return u1 > keys; }
  __device__ __forceinline__ bool whole() const { return u0 == 0 && last(); }
};
// The cached keys of a piece.
__device__ __forceinline__ int piece_begin(const CacheFwdParams& p, const Piece& w) {
  return w.u0 * p.unit;
}
__device__ __forceinline__ int piece_end(const CacheFwdParams& p, const Piece& w) {
  const long long e = static_cast<long long>(w.u1) * p.unit;
  return p.unit == 0 || e > w.rq.len ? w.rq.len : static_cast<int>(e);
}

__device__ __forceinline__ int row_tiles(const CacheFwdParams& p, const Request& r) {
  return (r.n * p.G + p.tile_rows - 1) / p.tile_rows;
}

// Units of all segments, and this lane's share of the requests [b0, b1) with
// the units before it and in it.
struct Census {
  long long total, before, mine;
  int b0, b1, blocks;
};
__device__ __forceinline__ Census take_census(const CacheFwdParams& p, bool* bad) {
  const int lane = threadIdx.x & 31;
  const int per = (p.batch + 31) / 32;
  Census c;
  c.b0 = min(lane * per, p.batch);
  c.b1 = min(c.b0 + per, p.batch);
  c.mine = 0;
  for (int b = c.b0; b < c.b1; ++b) {
    const Request r = load_request(p, b, bad);
    c.mine += static_cast<long long>(cache_units(r.len, r.n, p.unit, p.finish)) * p.Hk *
              row_tiles(p, r);
  }
  long long upto = c.mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += o;
  }
  c.before = upto - c.mine;
  c.total = __shfl_sync(0xffffffffu, upto, 31);
  c.blocks = cache_blocks(c.total, p.blocks);
  return c;
}

// The segment that holds unit `at` of all: its request, number, key units, and
// the unit's place in it (b, seg, keys, u0 and rq of w).
__device__ __forceinline__ void find_unit(const CacheFwdParams& p, const Census& c, long long at,
                                          bool* bad, Piece* w) {
  int fb = -1, fseg = 0, fu = 0, fkeys = 0;
  Request frq = {0, 0, 0};
  if (at >= c.before && at < c.before + c.mine) {
    long long before = c.before;
    for (int b = c.b0; b < c.b1; ++b) {
      const Request r = load_request(p, b, bad);
      const int u = cache_units(r.len, r.n, p.unit, p.finish);
      const long long n = static_cast<long long>(u) * p.Hk * row_tiles(p, r);
      if (at < before + n) {
        const long long in = at - before;
        if (in < (1LL << 31)) {
          fseg = static_cast<int>(in) / u;
          fu = static_cast<int>(in) - fseg * u;
        } else {
          fseg = static_cast<int>(in / u);
          fu = static_cast<int>(in % u);
        }
        fb = b;
        fkeys = u - p.finish, frq = r;
        break;
      }
      before += n;
    }
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, fb >= 0)) - 1;
  w->b = __shfl_sync(0xffffffffu, fb, src);
  w->seg = __shfl_sync(0xffffffffu, fseg, src);
  w->u0 = __shfl_sync(0xffffffffu, fu, src);
  w->keys = __shfl_sync(0xffffffffu, fkeys, src);
  w->rq.len = __shfl_sync(0xffffffffu, frq.len, src);
  w->rq.row0 = __shfl_sync(0xffffffffu, frq.row0, src);
  w->rq.n = __shfl_sync(0xffffffffu, frq.n, src);
}

__device__ __forceinline__ void enter_segment(const CacheFwdParams& p, Piece& w, long long run) {
  const int units = w.keys + p.finish;
  const long long n = units - w.u0 < run ? units - w.u0 : run;
  w.u1 = w.u0 + static_cast<int>(n);
  w.left = run - n;
}
__device__ __forceinline__ void next_piece(const CacheFwdParams& p, Piece& w) {
  if (w.left == 0) {
    w.b = -1;
    return;
  }
  w.first = 0;
  w.u0 = 0;
  const long long run = w.left;
  if (++w.seg == p.Hk * row_tiles(p, w.rq)) {
    w.seg = 0;
    bool bad = false;
    do {  // the units left are those of a request behind this one
      w.rq = load_request(p, ++w.b, &bad);
    } while (w.rq.n == 0 && w.b + 1 < p.batch);
    w.keys = cache_key_units(w.rq.len, p.unit);
  }
  enter_segment(p, w, run);
}
// The first piece of block x's run.  The block's thread 0 also writes down the
// segment that this block answers for at the join: one that is cut and begins
// with the block's run, or began in the block before and goes on in this one.
__device__ __forceinline__ Piece first_piece(const CacheFwdParams& p, int x, bool* bad) {
  const Census c = take_census(p, bad);
  Piece w;
  w.b = -1;
  w.first = 1;
  Cut cut = {};
  if (x < c.blocks) {
    const long long lo = cache_run(x, c.total, c.blocks), hi = cache_run(x + 1, c.total, c.blocks);
    find_unit(p, c, lo, bad, &w);
    enter_segment(p, w, hi - lo);
    if (threadIdx.x == 0 && p.unit > 0 && w.u0 <= w.keys) {
      const long long start = lo - w.u0;
      const int x0 = cache_owner(start, c.total, c.blocks);
      const int x1 = cache_owner(start + w.keys, c.total, c.blocks);
      const bool at_start = cache_run(x0, c.total, c.blocks) == start;
      if (x1 > x0 && x == (at_start ? x0 : x0 + 1)) {
        const int rtiles = row_tiles(p, w.rq);
        cut.pieces = x1 - x0 + 1;
        // the first piece is its block's last unless the block begins with it
        cut.slot0 = 2 * x0 + (at_start ? 0 : 1);
        cut.x0 = x0;
        cut.h = w.seg / rtiles;
        cut.row_base = (w.seg - cut.h * rtiles) * p.tile_rows;
        cut.rows = min(p.tile_rows, w.rq.n * p.G - cut.row_base);
        cut.row0 = w.rq.row0;
      }
    }
    if (w.u0 > w.keys) next_piece(p, w);  // the segment's end is another block's
  }
  if (threadIdx.x == 0 && p.unit > 0) p.cuts[x] = cut;
  return w;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Two e4m3 values (low / high half of w) as f16, exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(h)
      : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}"
      : "=r"(h)
      : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  ld_shared_v4(addr, v.x, v.y, v.z, v.w);
  return v;
}

__device__ __forceinline__ float pow2_bits(int e) { return __int_as_float((e + 127) << 23); }

// Probabilities are 2^(s - m + kShift) against a reference m that is a row's
// largest score at some point: it moves only where the probabilities of a
// tile's row sum to more than kMostSum, so that most tiles need no maximum and
// rescale nothing.  No probability exceeds kMostSum then, which f16 holds; and
// kShift moves f16's smallest subnormal to 2^-30 of the reference.
constexpr float kShift = 6.f;
constexpr float kMostSum = 32768.f;
// The output's unit for own keys.  Their probabilities are bf16 and lose nothing
// to any unit; this one keeps float32 sums of 2^10 own values of 2^127, the
// probabilities' 2^kShift included, from overflowing, and the bits of 2^-126.
constexpr int kOwnExp = 16;
constexpr float kOwnUnit = 1 << kOwnExp;

// More than 32 query rows per key/value head, headdim 64 or 128 (tiles of 128
// rows; the tensor maps' boxes are whole pages).
cudaError_t launch_cache_wide(const CacheFwdParams& p, int headdim, cudaStream_t stream);

}  // namespace dfa
