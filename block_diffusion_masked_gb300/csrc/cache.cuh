// Paged 8-bit key/value cache: index arithmetic shared by the host (argument
// checks, workspace sizes, tests) and the kernels.
//
// Layout.  k_cache, v_cache: (pages, kv_heads, page_size, headdim) e4m3, one
// page of one head contiguous.  k_scale, v_scale: (pages, kv_heads) float32,
// powers of two: a cached value is its e4m3 value times the scale of its page
// and head.  block_table: (batch, max_pages) page numbers of each request.
// A request's new rows are packed behind one another: request b has rows
// [cu_new[b], cu_new[b + 1]), at positions cache_lens[b], cache_lens[b] + 1 ...
#pragma once

#include "geometry.cuh"

namespace dfa {

// Smallest exponent of a page scale, and the e4m3 range it maps to.
constexpr int kCacheMinExp = -100;

// Exponent e of the scale 2^e of a page whose largest finite magnitude has
// the bf16 bits `bits` (sign cleared): the smallest e >= kCacheMinExp with
// amax <= 448 * 2^e.  448 = 1.75 * 2^8, so a magnitude (1 + m / 128) * 2^E
// needs e = E - 8 while m <= 96, else one more.  Subnormal bf16 magnitudes
// are below 2^-126 and take kCacheMinExp like every magnitude below it.
DFA_HD int cache_scale_exp(unsigned bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 96u ? 1 : 0);
  return e < kCacheMinExp ? kCacheMinExp : e;
}

// Pages a request can touch when it appends up to max_new tokens.
DFA_HD int cache_append_pages(int max_new, int page_size) {
  return (max_new + page_size - 2) / page_size + 1;
}

// Tokens [lo, hi) that an append of n tokens behind `len` cached ones puts
// into the j-th page it touches.
DFA_HD Interval cache_append_range(int len, int n, int j, int page_size) {
  const long long first = (static_cast<long long>(len / page_size) + j) * page_size;
  const long long end = static_cast<long long>(len) + n;
  const long long lo = first > len ? first : len;
  const long long hi = first + page_size < end ? first + page_size : end;
  if (lo >= hi) return {0, 0};
  return {static_cast<int>(lo), static_cast<int>(hi)};
}

// A page number a kernel may follow.
DFA_HD bool cache_page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }

// Split of a launch over its blocks.  A segment is one request, key/value head
// and tile of query rows; it counts a unit for every `unit` cached keys
// (unit 0: none, the segment is not to be cut) and `finish` units more for
// what every segment costs: its queries, own keys and read-out.  The units of
// all segments, in order, are dealt to the blocks in equal runs: block x takes
// [cache_run(x), cache_run(x + 1)).  A run may end among a segment's key
// units, and the pieces are joined afterwards; the block that reaches the
// finish units has the segment's end, a run that begins inside them skips the
// rest.
DFA_HD int cache_key_units(int len, int unit) {
  return unit > 0 && len > 0 ? (len - 1) / unit + 1 : 0;
}
DFA_HD int cache_units(int len, int n, int unit, int finish) {
  return n > 0 ? cache_key_units(len, unit) + finish : 0;
}
// Blocks that get work.  One unit is enough for a block: the join of a few
// pieces more costs less than a longer chain of keys (one request of 2000
// tokens, 4 heads: 11 us; with at least 4 units a block 14, with 8 19).
DFA_HD int cache_blocks(long long total, int limit) {
  return static_cast<int>(total < limit ? total : limit);
}
DFA_HD long long cache_run(int x, long long total, int blocks) {
  // 32-bit division where the product fits (blocks < 2^10): the usual case
  if (total < (1 << 22) && blocks < (1 << 10))
    return static_cast<unsigned>(x) * static_cast<unsigned>(total) / static_cast<unsigned>(blocks);
  return x * total / blocks;
}
// The block whose run holds unit w.
DFA_HD int cache_owner(long long w, long long total, int blocks) {
  if (total < (1 << 22) && blocks < (1 << 10))
    return static_cast<int>((static_cast<unsigned>(w + 1) * static_cast<unsigned>(blocks) - 1u) /
                            static_cast<unsigned>(total));
  return static_cast<int>(((w + 1) * blocks - 1) / total);
}

// One past the last own key that own row i of n sees: the rows of its block
// or earlier ones, for positions len + i and blocks of bs tokens from 0.  In
// unsigned 32 bits: len <= 2^30, i < n <= 2^24 and bs < 2^31 leave room.
DFA_HD int cache_own_end(int len, int i, int n, int bs) {
  const unsigned b = static_cast<unsigned>(bs);
  const unsigned e = ((static_cast<unsigned>(len) + i) / b + 1u) * b - len;
  return e < static_cast<unsigned>(n) ? static_cast<int>(e) : n;
}

}  // namespace dfa
