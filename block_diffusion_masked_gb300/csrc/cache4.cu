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

// The keys (cache4_scale_byte) of the two bf16 values of a word: each turned left by
// one bit.
__device__ __forceinline__ uint32_t keys2(uint32_t w) {
  return ((w << 1) & 0xfffefffeu) | ((w >> 15) & 0x00010001u);
}

// Codes of eight values whose group has the scale s, packed.
//
// x / s to the nearest, ties away from 0, without a division: x times r, the
// reciprocal of s made larger by 2^-20.  x / s is half of an odd number exactly or
// off by at least 2^-8 of itself (x has 8 significant bits, s has 3, |x / s| <= 8.5
// below), so the excess moves ties away from 0 and nothing else over a border.  The
// product is exact in the fma that adds 1.5 * 2^23 + 8, which leaves the code in the
// lowest bits of its sum.
__device__ __forceinline__ uint32_t encode8(const uint4& w, float r) {
  constexpr float kBase = 12582912.f;  // 1.5 * 2^23, whose bits are 0x4b400000
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
    const float y = fminf(fmaxf(fmaf(x, r, kBase + 8.f), kBase), kBase + 15.f);
    out += (__float_as_uint(y) - 0x4b400000u) << (16 * (i & 1) + 4 * (i >> 1));
  }
  return out;
}

// One CTA per (request, touched page; key/value head; k or v), as for the 8-bit
// append; but the tokens do not depend on one another.  Four neighbouring threads
// hold a group of 32 values, eight each: they settle its scale by two exchanges and
// write four bytes of codes each, one of them the scale's byte.
template <int D, int NT, int VPT>
__global__ void __launch_bounds__(NT) dfa_cache4_append_kernel(const Append4Params p) {
  constexpr int kVec = D / 8;  // vectors per token and head
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
  const int nvec = (span.hi - span.lo) * kVec;
  const long long sr = p.sr[which];
  const __nv_bfloat16* x = p.x[which] + (r0 + (span.lo - len)) * sr + h * p.sh[which];
  uint4 w[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = u * NT + tid;
    w[u] = make_uint4(0u, 0u, 0u, 0u);
    if (i < nvec) w[u] = *reinterpret_cast<const uint4*>(x + (i / kVec) * sr + (i % kVec) * 8);
  }
  if (!cache_page_ok(page, p.num_pages)) {  // nowhere to put it
    if (tid == 0) atomicOr(p.status, kStatusIndex);
    return;
  }
  const long long base = static_cast<long long>(page) * p.Hk + h;
  uint32_t* codes =
      reinterpret_cast<uint32_t*>(p.cache[which] + (base * p.page_size + first) * (D / 2));
  uint8_t* scale = p.scale[which] + base * p.page_size * (D / kCache4Group);
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = u * NT + tid;
    uint32_t top = __vmaxu2(__vmaxu2(keys2(w[u].x), keys2(w[u].y)),
                            __vmaxu2(keys2(w[u].z), keys2(w[u].w)));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int byte = cache4_scale_byte(max(top & 0xffffu, top >> 16));
    const float r = __frcp_rn(cache4_scale(byte)) * (1.f + 0x1p-20f);
    if (i < nvec) {
      codes[i] = encode8(w[u], r);
      const int token = i / kVec, vec = i % kVec;
      if ((vec & 3) == 0)
        scale[(vec >> 2) * p.page_size + first + token] = static_cast<uint8_t>(byte);
    }
  }
}

template <int D, int NT, int VPT>
cudaError_t launch_append_block(const Append4Params& p, unsigned blocks, cudaStream_t stream) {
  return launch_chained(dfa_cache4_append_kernel<D, NT, VPT>, dim3(blocks), dim3(NT), 0, stream,
                        p);
}

template <int D>
cudaError_t launch_append(const Append4Params& p, int batch, cudaStream_t stream) {
  const unsigned n = 2u * p.Hk * batch * p.touch;
  const int vectors = (p.max_new < p.page_size ? p.max_new : p.page_size) * (D / 8);
  if (vectors <= 128) return launch_append_block<D, 32, 4>(p, n, stream);
  if (vectors <= 512) return launch_append_block<D, 128, 4>(p, n, stream);
  // a page of 128 tokens is 1024, 2048 or 4096 vectors
  if constexpr (D == 128) {
    if (vectors > 1024) return launch_append_block<D, 256, 8>(p, n, stream);
  } else if constexpr (D == 256) {
    if (vectors > 2048) return launch_append_block<D, 512, 8>(p, n, stream);
    if (vectors > 1024) return launch_append_block<D, 256, 8>(p, n, stream);
  }
  return launch_append_block<D, 128, 8>(p, n, stream);
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
  int batch, rows, Hk, page_size, num_pages, max_pages, vec_shift;  // headdim 8 << vec_shift
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

constexpr int kReadWarps = 8;

// A warp takes a row: it finds the row's request and page, then moves the row's heads,
// keys and values, 16 bytes of output a lane at a time.
template <int BITS>
__global__ void __launch_bounds__(32 * kReadWarps) dfa_cache_read_kernel(const ReadParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  if (row >= p.rows || p.batch == 0) return;
  const int b = find_request(p.cu_rows, p.batch, row);
  const int r0 = b >= 0 ? p.cu_rows[b] : -1, r1 = b >= 0 ? p.cu_rows[b + 1] : 0;
  if (r0 < 0 || row < r0 || row >= r1) {
    // behind the last request's rows, or rows out of order
    if (lane == 0 && row < p.cu_rows[p.batch]) atomicOr(p.status, kStatusIndex);
    return;
  }
  const int len = p.cache_lens[b];
  const long long pos = static_cast<long long>(p.first ? p.first[b] : 0) + (row - r0);
  int page = -1;
  if (len >= 0 && len <= p.max_pages * p.page_size && pos >= 0 && pos < len)
    page = p.block_table[static_cast<long long>(b) * p.max_pages + pos / p.page_size];
  const bool ok = cache_page_ok(page, p.num_pages);
  if (!ok && lane == 0) atomicOr(p.status, kStatusIndex);
  const int at = static_cast<int>(pos) & (p.page_size - 1);
  const int per = p.Hk << p.vec_shift;  // vectors of a row
  const long long heads = static_cast<long long>(page) * p.Hk;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    uint4* dst = reinterpret_cast<uint4*>(p.y[which]) + static_cast<long long>(row) * per;
    const uint8_t* cache = p.cache[which];
#pragma unroll 4
    for (int i = lane; i < per; i += 32) {
      uint4 out = make_uint4(0u, 0u, 0u, 0u);
      if (ok) {
        const int h = i >> p.vec_shift, vec = i & ((1 << p.vec_shift) - 1);
        const long long token = (heads + h) * p.page_size + at;
        if constexpr (BITS == 4) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(
              cache + ((token << p.vec_shift) + vec) * 4);
          const uint8_t* scale = static_cast<const uint8_t*>(p.scale[which]);
          const long long group = ((heads + h) << p.vec_shift >> 2) + (vec >> 2);
          const float s = cache4_scale(scale[group * p.page_size + at]);
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            f[e] = static_cast<float>(
                       static_cast<int>((w >> (16 * (e & 1) + 4 * (e >> 1))) & 15u) - 8) * s;
          out = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                           pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(
              cache + ((token << p.vec_shift) + vec) * 8);
          const float s = static_cast<const float*>(p.scale[which])[heads + h];
          const uint32_t u[2] = {w.x, w.y};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t f16;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                : "=r"(f16)
                : "h"(static_cast<uint16_t>(u[e >> 1] >> (16 * (e & 1)))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16));
            o[e] = pack_bf16x2(f.x * s, f.y * s);
          }
          out = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      dst[i] = out;
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
  const cudaError_t e = launch_chained(
      bits == 4 ? dfa_cache_read_kernel<4> : dfa_cache_read_kernel<8>,
      dim3((static_cast<unsigned>(rows) + kReadWarps - 1) / kReadWarps), dim3(32 * kReadWarps), 0,
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
