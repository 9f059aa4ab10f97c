// Paged 4-bit key/value cache: the append of finished tokens; and the reading back
// of tokens from either cache.  Format: cache4.cuh (4 bits), cache.cuh (8 bits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache.cuh"
#include "cache4.cuh"
#include "device.cuh"
#include "dfa.h"
#include "params.cuh"
#include "sm100.cuh"

namespace dfa {
namespace {

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }
bool aligned_to(const void* p, unsigned n) {
  return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// ------------------------------------------------------------------ append

struct Append4Params {
  const __nv_bfloat16* x[2];  // k, v: (rows, kv_heads, headdim), strided
  long long sr[2], sh[2];     // row and head strides in elements
  uint8_t* cache[2];
  uint8_t* scale[2];
  const int* cu_new;
  const int* cache_lens;
  const int* block_table;
  unsigned* status;
  int rows, max_new, Hk, page_size, num_pages, max_pages, touch;
};

// The key (cache4_scale_byte) of a group of 32 values: the largest value and the largest
// negated one, two to an operation, NaN where there is one.
__device__ __forceinline__ unsigned group_key(const uint4 (&w)[4]) {
  auto as2 = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
  auto bits = [](__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); };
  __nv_bfloat162 most[4], least[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    most[i] = __hmax2_nan(__hmax2_nan(as2(w[i].x), as2(w[i].y)),
                          __hmax2_nan(as2(w[i].z), as2(w[i].w)));
    least[i] = __hmin2_nan(__hmin2_nan(as2(w[i].x), as2(w[i].y)),
                           __hmin2_nan(as2(w[i].z), as2(w[i].w)));
  }
  const uint32_t hi = bits(__hmax2_nan(__hmax2_nan(most[0], most[1]),
                                       __hmax2_nan(most[2], most[3])));
  const uint32_t lo = bits(__hmin2_nan(__hmin2_nan(least[0], least[1]),
                                       __hmin2_nan(least[2], least[3]))) ^
                      0x80008000u;
  // the largest value in the low half, the largest negated one in the high half
  const uint32_t top = bits(__hmax2_nan(as2(__byte_perm(hi, lo, 0x5410)),
                                        as2(__byte_perm(hi, lo, 0x7632))));
  // Of the two the larger is the group's largest magnitude (both are negative zeros at
  // least): as signed integers, of which a NaN's is the largest.
  const int pos = static_cast<short>(top & 0xffffu), neg = static_cast<short>(top >> 16);
  return 2u * static_cast<unsigned>(max(max(pos, neg), 0)) + (neg >= pos ? 1u : 0u);
}

// Codes of eight values whose group has the scale s, packed.
//
// x / s to the nearest, ties away from 0, without a division: x times r, the reciprocal of s
// made larger by 2^-14.  x / s is half of an odd number exactly or off by at least 2^-8 of
// itself (x has 8 significant bits, s has 3, |x / s| <= 8.5 below), so the excess moves ties
// away from 0, by 2^-15 at least, and nothing else over a border; what the roundings below
// may be off by (the reciprocal by 2^-23 of itself, the products by 2^-22 of 8.5 codes) is
// less than 2^-18 of a code.  The first product, with 8 more, is kept within
// 0 and 15.4375 by taking it as a fraction of that, within 0 and 1; the second is rounded by
// 1.5 * 2^23, which leaves the code in the sum's lowest bits.
constexpr float kMost = 15.4375f;  // rounds to 15
__device__ __forceinline__ uint32_t encode8(const uint4& w, float r) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t out = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const int at = i < 4 ? 2 * i : 2 * i - 7;  // dims 0, 2, 4, 6, 1, 3, 5, 7 from the lowest bits
    const float x =
        __uint_as_float(at & 1 ? u[at >> 1] & 0xffff0000u : u[at >> 1] << 16);
    const float y = __saturatef(fmaf(x, r, 8.f / kMost));
    out = (out << 4) + __float_as_uint(fmaf(y, kMost, 12582912.f));
  }
  // the sum's own bits, 0x4b400000, have come in eight times, moved by 0, 4, 8, ... bits
  return out - (0x4b400000u + 0xb4000000u + 0x40000000u);
}

// Single tokens are bound by latency (lengths, page and tokens one after another), prompts
// by memory: 8 requests of 8190 tokens, 8 heads of 128, 340 MB, in 53 us, 6.4 TB/s; with
// their reading back 94 us, 145 before extremes were packed, codes made without a division,
// scales written by words and a group given to one thread.
//
// One CTA per (request, touched page; key/value head; k or v), as for the 8-bit
// append; but the tokens do not depend on one another.  A thread takes groups of 32
// values, so that what a scale costs is paid once (four threads to a group: 61 us).
template <int D, int NT, int GPT>
__global__ void __launch_bounds__(NT) dfa_cache4_append_kernel(const Append4Params p) {
  constexpr int kGroups = D / kCache4Group;  // per token and head
  constexpr int kTokens = NT * GPT / kGroups < 128 ? NT * GPT / kGroups : 128;
  __shared__ uint8_t s_scale[kGroups][kTokens + 4];  // of tokens from a multiple of four on
  grid_launch_dependents();
  grid_dependency_wait();
  // heads fastest: neighbouring blocks read neighbouring pieces of the rows
  const unsigned head = blockIdx.x % (2u * p.Hk), at = blockIdx.x / (2u * p.Hk);
  const int which = head >= static_cast<unsigned>(p.Hk), h = head - which * p.Hk;
  const int b = at / p.touch, j = at - b * p.touch, tid = threadIdx.x;
  const int r0 = p.cu_new[b], r1 = p.cu_new[b + 1], len = p.cache_lens[b];
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= p.rows && r1 - r0 <= p.max_new && len >= 0 &&
                  len <= (1 << 30);
  const int n = ok ? r1 - r0 : 0;
  const Interval span = ok ? cache_append_range(len, n, j, p.page_size) : Interval{0, 0};
  const int slot = len / p.page_size + j;
  if (span.lo >= span.hi) {  // nothing for this page
    if (tid == 0 && !ok) atomicOr(p.status, kStatusIndex);
    return;
  }
  int page = -1;
  if (slot < p.max_pages)
    page = p.block_table[static_cast<long long>(b) * p.max_pages + slot];
  const int first = span.lo & (p.page_size - 1);  // older tokens of the page
  const int tokens = span.hi - span.lo, groups = tokens * kGroups;
  const long long sr = p.sr[which];
  const __nv_bfloat16* x = p.x[which] + (r0 + (span.lo - len)) * sr + h * p.sh[which];
  uint4 w[GPT][4];
#pragma unroll
  for (int u = 0; u < GPT; ++u) {
    const int i = u * NT + tid;
    const uint4* src =
        reinterpret_cast<const uint4*>(x + (i / kGroups) * sr + (i % kGroups) * kCache4Group);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[u][e] = i < groups ? src[e] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (!cache_page_ok(page, p.num_pages)) {  // nowhere to put it
    if (tid == 0) atomicOr(p.status, kStatusIndex);
    return;
  }
  const long long base = static_cast<long long>(page) * p.Hk + h;
  uint4* codes =
      reinterpret_cast<uint4*>(p.cache[which] + (base * p.page_size + first) * (D / 2));
  uint8_t* scale = p.scale[which] + base * p.page_size * (D / kCache4Group);
#pragma unroll
  for (int u = 0; u < GPT; ++u) {
    const int i = u * NT + tid;
    if (i >= groups) break;
    const int byte = cache4_scale_byte(group_key(w[u]));
    float r;  // off by 2^-23 of itself at most
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(cache4_scale(byte)));
    r *= (1.f + 0x1p-14f) / kMost;
    codes[i] = make_uint4(encode8(w[u][0], r), encode8(w[u][1], r), encode8(w[u][2], r),
                          encode8(w[u][3], r));
    s_scale[i % kGroups][(first & 3) + i / kGroups] = static_cast<uint8_t>(byte);
  }
  // The scales, tokens of a group next to one another: four at a time where all are new.
  if constexpr (NT > 32) __syncthreads();
  else __syncwarp();
  const int from = first & ~3, words = (tokens + (first & 3) + 3) >> 2;
  const int end = first + tokens;
  for (int i = tid; i < kGroups * words; i += NT) {
    const int grp = i / words, word = i - grp * words, token = from + 4 * word;
    uint8_t* dst = scale + grp * p.page_size + token;
    const uint8_t* src = &s_scale[grp][4 * word];
    if (token >= first && token + 4 <= end) {
      *reinterpret_cast<uchar4*>(dst) = make_uchar4(src[0], src[1], src[2], src[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (token + e >= first && token + e < end) dst[e] = src[e];
    }
  }
}

template <int D, int NT, int GPT>
cudaError_t launch_append_block(const Append4Params& p, unsigned blocks, cudaStream_t stream) {
  return launch_chained(dfa_cache4_append_kernel<D, NT, GPT>, dim3(blocks), dim3(NT), 0, stream,
                        p);
}

template <int D>
cudaError_t launch_append(const Append4Params& p, int batch, cudaStream_t stream) {
  const unsigned n = 2u * p.Hk * batch * p.touch;
  const int groups = (p.max_new < p.page_size ? p.max_new : p.page_size) * (D / kCache4Group);
  if (groups <= 32) return launch_append_block<D, 32, 1>(p, n, stream);
  if (groups <= 128) return launch_append_block<D, 128, 1>(p, n, stream);
  // a page of 128 tokens is 256, 512 or 1024 groups
  if constexpr (D == 128) {
    if (groups > 256) return launch_append_block<D, 256, 2>(p, n, stream);
  } else if constexpr (D == 256) {
    if (groups > 512) return launch_append_block<D, 512, 2>(p, n, stream);
    if (groups > 256) return launch_append_block<D, 256, 2>(p, n, stream);
  }
  return launch_append_block<D, 128, 2>(p, n, stream);
}

// ------------------------------------------------------------------ read

struct ReadParams {
  const uint8_t* cache[2];
  const void* scale[2];
  __nv_bfloat16* y[2];
  const int* block_table;
  const int* cache_lens;
  const int* first;  // or null
  const int* cu_rows;
  unsigned* status;
  int batch, rows, Hk, page_size, page_shift, num_pages, max_pages;
  int vec_shift;  // headdim 8 << vec_shift
  int per_block;  // rows
};

// The last request b with cu[b] <= row, among [0, batch), by 32 looks at a time; all
// lanes of the warp agree.  -1 where there is none.
__device__ __forceinline__ int find_request(const int* cu, int batch, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;  // the answer is in [lo - 1, lo + n)
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < n && cu[lo + at] <= row);
    const int hits = __popc(below);  // a prefix, if cu is in order
    if (hits == 0) break;
    lo += (hits - 1) * step + 1;
    n = min(step - 1, n - (hits - 1) * step - 1);
  }
  return lo - 1;
}

constexpr int kReadWarps = 8, kReadRows = 32;  // a row for each lane of a warp
static_assert(kReadRows == 32, "each lane of the first warp writes a row's page and place");

// Bound by memory: 80 k tokens of 8 heads of 128 read back from 4 bits in 55 us (318 MB
// written and read at 5.8 TB/s; 91 us while each warp looked up its own rows' places).
//
// A block takes up to 32 rows.  The lanes of its first warp find a row's request, page and
// place each, so that the chain of their loads is paid once; then every warp moves rows,
// their heads' keys and values, 16 bytes of output a lane and access, several on their way.
template <int BITS>
__global__ void __launch_bounds__(32 * kReadWarps) dfa_cache_read_kernel(const ReadParams p) {
  __shared__ int s_page[kReadRows], s_at[kReadRows];  // page -1: zeros; place -1: leave alone
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * p.per_block, rows = min(p.per_block, p.rows - row0);
  if (warp == 0) {
    // requests whose rows there are not: what fits is read
    if (blockIdx.x == 0 && lane == 0 && p.cu_rows[p.batch] > p.rows)
      atomicOr(p.status, kStatusIndex);
    int b = find_request(p.cu_rows, p.batch, row0);
    const int row = row0 + lane;
    int page = -1, place = -1;
    if (lane < rows) {
      while (b + 1 < p.batch && p.cu_rows[b + 1] <= row) ++b;
      const int r0 = b >= 0 ? p.cu_rows[b] : -1, r1 = b >= 0 ? p.cu_rows[b + 1] : 0;
      if (r0 < 0 || row < r0 || row >= r1) {
        // behind the last request's rows, or rows out of order
        if (row < p.cu_rows[p.batch]) atomicOr(p.status, kStatusIndex);
      } else {
        const int len = p.cache_lens[b];
        const long long pos = static_cast<long long>(p.first ? p.first[b] : 0) + (row - r0);
        if (len >= 0 && len <= p.max_pages << p.page_shift && pos >= 0 && pos < len)
          page = p.block_table[static_cast<long long>(b) * p.max_pages + (pos >> p.page_shift)];
        place = static_cast<int>(pos) & (p.page_size - 1);
        if (!cache_page_ok(page, p.num_pages)) {
          page = -1;
          atomicOr(p.status, kStatusIndex);
        }
      }
    }
    s_page[lane] = page;
    s_at[lane] = place;
  }
  __syncthreads();
  const int per = p.Hk << p.vec_shift;  // vectors of a row
#pragma unroll 1
  for (int r = warp; r < 2 * rows; r += kReadWarps) {
    const int which = r >= rows, row = r - which * rows, page = s_page[row], at = s_at[row];
    if (at < 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(which ? p.y[1] : p.y[0]) +
                 static_cast<long long>(row0 + row) * per;
    if (page < 0) {
      for (int i = lane; i < per; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const uint8_t* cache = which ? p.cache[1] : p.cache[0];
    const void* scales = which ? p.scale[1] : p.scale[0];
    const long long heads = static_cast<long long>(page) * p.Hk;
    // (Ordinary loads: the cache may have been written by the kernel before, during which this
    // block may have been here already, so its lines are not read-only for a kernel's time.)
    // Vectors a lane has on their way.  80 k tokens of 1024 values, or as many values (but 2^20
    // tokens at most) in rows of other sizes, us with 2, 4 and 8, 4 bits: rows of 64 values 283,
    // 278, 312 (8 of a warp's lanes have a vector: such rows are bound by their number), of 256
    // 97, 96, 113, of 512 75, 76, 82, of 1024 77, 71, 70, of 2048 86, 79, 73; 8 bits: 303, 284,
    // 381, 117, 113, 150, 85, 86, 101, 83, 78, 84, 89, 82, 81.
    constexpr int kAtOnce = 4;
#pragma unroll 1
    for (int i0 = lane; i0 < per; i0 += 32 * kAtOnce) {
      uint2 w[kAtOnce];
      float s[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int i = i0 + 32 * e;
        if (i >= per) break;
        const int h = i >> p.vec_shift, vec = i & ((1 << p.vec_shift) - 1);
        const long long token = ((heads + h) << p.page_shift) + at;
        const uint8_t* src = cache + ((token << p.vec_shift) + vec) * BITS;
        if constexpr (BITS == 4) {
          w[e].x = *reinterpret_cast<const uint32_t*>(src);
          const long long group = ((heads + h) << p.vec_shift >> 2) + (vec >> 2);
          s[e] = __uint_as_float(
              static_cast<const uint8_t*>(scales)[(group << p.page_shift) + at]);
        } else {
          w[e] = *reinterpret_cast<const uint2*>(src);
          s[e] = static_cast<const float*>(scales)[heads + h];
        }
      }
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int i = i0 + 32 * e;
        if (i >= per) break;
        uint32_t o[4];
        if constexpr (BITS == 4) {
          uint32_t f[4];
          const uint32_t byte = __float_as_uint(s[e]);
          cache4_decode(w[e].x, cache4_prepare(byte << 8 | byte << 24), f);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[x]));
            o[x] = pack_bf16x2(y.x * kCache4Unit, y.y * kCache4Unit);
          }
        } else {
          const uint32_t u[2] = {w[e].x, w[e].y};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t f16;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                : "=r"(f16)
                : "h"(static_cast<uint16_t>(u[x >> 1] >> (16 * (x & 1)))));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f16));
            o[x] = pack_bf16x2(y.x * s[e], y.y * s[e]);
          }
        }
        dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

int cache_read(int bits, const void* k_cache, const void* v_cache, const void* k_scale,
               const void* v_scale, const int* block_table, const int* cache_lens,
               const int* first, const int* cu_rows, void* k, void* v, int batch, int rows,
               int kv_heads, int headdim, int page_size, int num_pages, int max_pages,
               dfa_stream_t stream) {
  if (batch < 0 || batch > 32768 || rows < 0 || rows > (1 << 30) || kv_heads < 1 ||
      kv_heads > 65535 || num_pages < 1 || max_pages < 1 || !page_size_ok(page_size) ||
      static_cast<long long>(max_pages) * page_size > (1 << 30))
    return DFA_EINVAL;
  if (headdim != 64 && headdim != 128 && headdim != 256) return DFA_EUNSUPPORTED;
  if (batch == 0 || rows == 0) return DFA_OK;
  for (const void* q : {k_cache, v_cache, static_cast<const void*>(k), static_cast<const void*>(v)})
    if (!aligned_to(q, 16)) return DFA_EINVAL;
  for (const void* q : {static_cast<const void*>(block_table), static_cast<const void*>(cache_lens),
                        static_cast<const void*>(cu_rows)})
    if (!aligned_to(q, 4)) return DFA_EINVAL;
  if (!aligned_to(k_scale, bits == 4 ? 16 : 4) || !aligned_to(v_scale, bits == 4 ? 16 : 4) ||
      (first && !aligned_to(first, 4)))
    return DFA_EINVAL;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  ReadParams p{};
  p.cache[0] = static_cast<const uint8_t*>(k_cache);
  p.cache[1] = static_cast<const uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.y[0] = static_cast<__nv_bfloat16*>(k);
  p.y[1] = static_cast<__nv_bfloat16*>(v);
  p.block_table = block_table;
  p.cache_lens = cache_lens;
  p.first = first;
  p.cu_rows = cu_rows;
  p.status = di.status;
  p.batch = batch;
  p.rows = rows;
  p.Hk = kv_heads;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.vec_shift = headdim == 64 ? 3 : headdim == 128 ? 4 : 5;
  p.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  // A few rows are spread over the device.
  p.per_block = rows <= 4 * kReadWarps * di.sms ? kReadWarps / 2 : kReadRows;
  const cudaError_t e = launch_chained(
      bits == 4 ? dfa_cache_read_kernel<4> : dfa_cache_read_kernel<8>,
      dim3((static_cast<unsigned>(rows) + p.per_block - 1) / p.per_block), dim3(32 * kReadWarps), 0,
      static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" {

int dfa_cache4_scale_byte(unsigned top) { return cache4_scale_byte(top & 0xffffu); }

int dfa_cache4_append(const void* k, const void* v, const int* cu_new, const int* cache_lens,
                      const int* block_table, void* k_cache, void* v_cache, void* k_scale,
                      void* v_scale, int batch, int rows, int max_new, int kv_heads, int headdim,
                      int page_size, int num_pages, int max_pages, const long long* k_strides,
                      const long long* v_strides, dfa_stream_t stream) {
  if (batch < 0 || rows < 0 || rows > (1 << 30) || max_new < 0 || max_new > (1 << 30) ||
      kv_heads < 1 || kv_heads > 65535 || num_pages < 1 || max_pages < 1 ||
      !page_size_ok(page_size) || static_cast<long long>(max_pages) * page_size > (1 << 30))
    return DFA_EINVAL;
  if (headdim != 64 && headdim != 128 && headdim != 256) return DFA_EUNSUPPORTED;
  if (batch == 0 || rows == 0 || max_new == 0) return DFA_OK;
  const int touch = cache_append_pages(max_new < rows ? max_new : rows, page_size);
  if (static_cast<long long>(batch) * touch > 0x7fffffffLL / (2 * kv_heads)) return DFA_EINVAL;
  for (const void* q : {k, v, static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
    if (!aligned_to(q, 16)) return DFA_EINVAL;
  for (const void* q : {static_cast<const void*>(cu_new), static_cast<const void*>(cache_lens),
                        static_cast<const void*>(block_table)})
    if (!aligned_to(q, 4)) return DFA_EINVAL;
  if (!aligned_to(k_scale, 16) || !aligned_to(v_scale, 16)) return DFA_EINVAL;
  Append4Params p{};
  const long long* strides[2] = {k_strides, v_strides};
  for (int i = 0; i < 2; ++i) {
    p.x[i] = static_cast<const __nv_bfloat16*>(i ? v : k);
    p.sr[i] = strides[i] ? strides[i][0] : static_cast<long long>(kv_heads) * headdim;
    p.sh[i] = strides[i] ? strides[i][1] : headdim;
    if ((p.sr[i] & 7) || (p.sh[i] & 7)) return DFA_EINVAL;
    p.cache[i] = static_cast<uint8_t*>(i ? v_cache : k_cache);
    p.scale[i] = static_cast<uint8_t*>(i ? v_scale : k_scale);
  }
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  p.cu_new = cu_new;
  p.cache_lens = cache_lens;
  p.block_table = block_table;
  p.status = di.status;
  p.rows = rows;
  p.max_new = max_new < rows ? max_new : rows;
  p.Hk = kv_heads;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.touch = touch;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = headdim == 64    ? launch_append<64>(p, batch, s)
                        : headdim == 128 ? launch_append<128>(p, batch, s)
                                         : launch_append<256>(p, batch, s);
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

int dfa_cache_read(const void* k_cache, const void* v_cache, const float* k_scale,
                   const float* v_scale, const int* block_table, const int* cache_lens,
                   const int* first, const int* cu_rows, void* k, void* v, int batch, int rows,
                   int kv_heads, int headdim, int page_size, int num_pages, int max_pages,
                   dfa_stream_t stream) {
  return cache_read(8, k_cache, v_cache, k_scale, v_scale, block_table, cache_lens, first, cu_rows,
                    k, v, batch, rows, kv_heads, headdim, page_size, num_pages, max_pages, stream);
}

int dfa_cache4_read(const void* k_cache, const void* v_cache, const void* k_scale,
                    const void* v_scale, const int* block_table, const int* cache_lens,
                    const int* first, const int* cu_rows, void* k, void* v, int batch, int rows,
                    int kv_heads, int headdim, int page_size, int num_pages, int max_pages,
                    dfa_stream_t stream) {
  return cache_read(4, k_cache, v_cache, k_scale, v_scale, block_table, cache_lens, first, cu_rows,
                    k, v, batch, rows, kv_heads, headdim, page_size, num_pages, max_pages, stream);
}

}  // extern "C"
