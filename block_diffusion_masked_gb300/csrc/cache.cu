// Paged 8-bit key/value cache: the pages of a sampling step (plan, release)
// and the append of finished tokens.  Layout and arithmetic: cache.cuh.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache.cuh"
#include "device.cuh"
#include "dfa.h"
#include "params.cuh"
#include "sm100.cuh"

namespace dfa {
namespace {

namespace cg = cooperative_groups;

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }
bool aligned_to(const void* p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// ------------------------------------------------------------------ plan

// Two running sums of one request: its new pages and its new rows.
struct Sums {
  long long pages, rows;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return {a.pages + b.pages, a.rows + b.rows};
}

constexpr int kPlanThreads = 512;

// Inclusive scan over the block; `total` receives the block's sum.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sums o = {__shfl_up_sync(0xffffffffu, v.pages, off),
                    __shfl_up_sync(0xffffffffu, v.rows, off)};
    if (lane >= off) v = v + o;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Sums before = {0, 0}, all = {0, 0};
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w == warp) before = all;
    all = all + warp_sums[w];
  }
  *total = all;
  return before + v;
}

struct PlanParams {
  const int* cache_lens;
  const int* new_lens;
  int* block_table;
  const int* free_pages;
  const int* free_count;
  int* cu_new;
  int* positions;
  int* next_lens;
  int* next_free;
  int* missing;
  unsigned* status;
  int batch, max_pages, num_free, page_size, rows;
};

// The pages, rows and positions of one sampling step.  Request b holds
// len_b tokens in ceil(len_b / page_size) pages and gets n_b more: its new
// pages come off the top of the free stack, requests in order, pages in
// order; its rows are numbered behind those of the requests before it.
//
// Two exclusive sums over the requests, then independent stores: bound by
// latency (a launch, two dependent loads, two scans).  One cluster of CTAs
// runs the scans redundantly, 512 requests at a time, and shares the stores:
// the owner of a row or of a new page is found by binary search in the sums
// of the 512.  A cluster barrier stands between the loads and the stores, so
// that next_lens and next_free may be cache_lens and free_count.
// Measured: 5 requests, 80 rows 3.6 us; 1024 requests of 32 rows 10.5 us.
__global__ void __launch_bounds__(kPlanThreads) dfa_cache_plan_kernel(const PlanParams p) {
  __shared__ Sums warp_sums[kPlanThreads / 32];
  __shared__ long long s_pages[kPlanThreads + 1], s_rows[kPlanThreads + 1];
  __shared__ int s_len[kPlanThreads], s_has[kPlanThreads];
  cg::cluster_group cluster = cg::this_cluster();
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const int part = static_cast<int>(cluster.block_rank());
  const int parts = static_cast<int>(cluster.num_blocks());
  const long long capacity = static_cast<long long>(p.max_pages) * p.page_size;
  int top = p.free_count[0];
  bool bad = top < 0 || top > p.num_free;
  top = top < 0 ? 0 : top > p.num_free ? p.num_free : top;
  Sums carry = {0, 0};
  long long lost = 0;  // pages a request wants past its table's end
  for (int base = 0; base < p.batch; base += kPlanThreads) {
    const int b = base + tid;
    int len = 0, n = 0, has = 0;
    Sums mine = {0, 0};
    long long past = 0;
    auto wants = [&](int rows) {  // pages and rows of a request that adds `rows`
      const long long want =
          (static_cast<long long>(len) + rows + p.page_size - 1) / p.page_size - has;
      const long long room = p.max_pages - has;
      past = want > room ? want - room : 0;
      mine = {want - past, rows};
    };
    if (b < p.batch) {
      len = p.cache_lens[b];
      n = p.new_lens[b];
      if (len < 0 || len > capacity || n < 0) {
        bad = true;
        len = len < 0 ? 0 : len > capacity ? static_cast<int>(capacity) : len;
        n = n < 0 ? 0 : n;
      }
      has = (len + p.page_size - 1) / p.page_size;
      wants(n);
    }
    Sums all;
    Sums upto = block_scan(mine, warp_sums, &all);
    if (carry.rows + all.rows > p.rows) {  // rows are cut, and with them their pages
      bad = true;
      const long long room = p.rows - (carry.rows + upto.rows - mine.rows);
      if (b < p.batch) wants(room < 0 ? 0 : room < n ? static_cast<int>(room) : n);
      upto = block_scan(mine, warp_sums, &all);
    }
    // the requests' own exclusive sums, and the end of the last
    s_pages[tid + 1] = upto.pages;
    s_rows[tid + 1] = upto.rows;
    if (tid == 0) s_pages[0] = s_rows[0] = 0;
    s_len[tid] = len;
    s_has[tid] = has;
    for (int off = 16; off > 0; off >>= 1) past += __shfl_xor_sync(0xffffffffu, past, off);
    if ((tid & 31) == 0) lost += past;
    __syncthreads();
    cluster.sync();  // every CTA has read this part's lengths (and the free count)
    const int count = p.batch - base < kPlanThreads ? p.batch - base : kPlanThreads;
    if (part == 0 && b < p.batch) {
      const long long r0 = carry.rows + upto.rows - mine.rows;
      const long long r1 = carry.rows + upto.rows;
      p.cu_new[b] = static_cast<int>(r0);
      if (b == p.batch - 1) p.cu_new[p.batch] = static_cast<int>(r1);
      const long long before = carry.pages + upto.pages - mine.pages;
      const long long left = before >= top ? 0 : top - before;
      const long long got = mine.pages > left ? left : mine.pages;
      const long long cap = (has + got) * p.page_size;
      const long long next = len + mine.rows;
      p.next_lens[b] = static_cast<int>(next < cap ? next : cap);
    }
    const int step = parts * kPlanThreads, me = part * kPlanThreads + tid;
    for (long long i = me; i < all.pages; i += step) {
      int lo = 0, hi = count - 1;  // the last request whose first new page is at most i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pages[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      const long long at = top - 1 - (carry.pages + i);
      p.block_table[static_cast<long long>(base + lo) * p.max_pages + s_has[lo] +
                    (i - s_pages[lo])] = at >= 0 ? p.free_pages[at] : -1;
    }
    for (long long i = me; i < all.rows; i += step) {
      int lo = 0, hi = count - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_rows[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      p.positions[carry.rows + i] = s_len[lo] + static_cast<int>(i - s_rows[lo]);
    }
    carry = carry + all;
    __syncthreads();  // the sums of this part have been read
  }
  for (long long i = carry.rows + part * kPlanThreads + tid; i < p.rows; i += parts * kPlanThreads)
    p.positions[i] = -1;
  if (p.batch == 0) cluster.sync();  // the free count has been read
  // pages past the tables' ends, summed over the block's warps
  __syncthreads();
  if ((tid & 31) == 0) warp_sums[tid >> 5].pages = lost;
  __syncthreads();
  if (part == 0 && tid == 0) {
    for (int w = 1; w < kPlanThreads / 32; ++w) lost += warp_sums[w].pages;
    const long long left = top - carry.pages;
    p.next_free[0] = static_cast<int>(left > 0 ? left : 0);
    const long long miss = lost + (left < 0 ? -left : 0);
    p.missing[0] = static_cast<int>(miss < 0x7fffffffLL ? miss : 0x7fffffffLL);
    if (p.batch == 0) p.cu_new[0] = 0;
  }
  if (bad) atomicOr(p.status, kStatusIndex);
}

struct ReleaseParams {
  const int* finished;
  int* cache_lens;
  int* block_table;
  int* free_pages;
  int* free_count;
  unsigned* status;
  int batch, max_pages, num_free, page_size;
};

// Finished requests give their pages back: pushed on the free stack in the
// order of the requests and of their pages, table entries set to -1, lengths
// to 0.  One CTA; a warp takes one request of a group of 16 at a time: bound by
// the chain of trips to memory of a group, 64 groups one after another for 1024
// requests.  Measured: half of 8 requests of up to 2000 tokens (81 pages of 64)
// 5 us, half of 64 of up to 8000 (2020 pages) 11, half of 1024 of up to 16000
// (62.7 k pages) 190.
__global__ void __launch_bounds__(kPlanThreads) dfa_cache_release_kernel(const ReleaseParams p) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int s_count[kWarps];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long capacity = static_cast<long long>(p.max_pages) * p.page_size;
  int top = p.free_count[0];
  bool bad = top < 0 || top > p.num_free;
  top = top < 0 ? 0 : top > p.num_free ? p.num_free : top;
  __syncthreads();
  for (int base = 0; base < p.batch; base += kWarps) {
    const int b = base + warp;
    int pages = 0;
    if (b < p.batch && p.finished[b] != 0) {
      const int len = p.cache_lens[b];
      bad = bad || len < 0 || len > capacity;
      pages = len <= 0 ? 0
              : len > capacity ? p.max_pages
                               : (len + p.page_size - 1) / p.page_size;
    }
    int* row = p.block_table + static_cast<long long>(b) * p.max_pages;
    int valid = 0;  // pages of the request that name one
    for (int j0 = 0; j0 < pages; j0 += 32) {
      const bool ok = j0 + lane < pages && row[j0 + lane] >= 0;
      valid += __popc(__ballot_sync(0xffffffffu, ok));
    }
    if (lane == 0) s_count[warp] = valid;
    __syncthreads();
    int at = top;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += s_count[w];
      top += s_count[w];
    }
    for (int j0 = 0; j0 < pages; j0 += 32) {
      const int page = j0 + lane < pages ? row[j0 + lane] : -1;
      const unsigned ok = __ballot_sync(0xffffffffu, page >= 0);
      const int to = at + __popc(ok & ((1u << lane) - 1));
      if (page >= 0) {
        if (to < p.num_free) p.free_pages[to] = page;
        else bad = true;
      }
      if (j0 + lane < pages) row[j0 + lane] = -1;
      at += __popc(ok);
    }
    if (b < p.batch && lane == 0 && p.finished[b] != 0) p.cache_lens[b] = 0;
    __syncthreads();  // the counts have been read
  }
  if (threadIdx.x == 0) p.free_count[0] = top < p.num_free ? top : p.num_free;
  if (bad) atomicOr(p.status, kStatusIndex);
}

// ------------------------------------------------------------------ append

struct AppendParams {
  const __nv_bfloat16* x[2];  // k, v: (rows, kv_heads, headdim), strided
  long long sr[2], sh[2];     // row and head strides in elements
  uint8_t* cache[2];
  float* scale[2];
  const int* cu_new;
  const int* cache_lens;
  const int* block_table;
  unsigned* status;
  int rows, max_new, Hk, page_size, num_pages, max_pages, touch;
};

// Eight bf16 values times `inv`, as e4m3; with `odd`, values that are not
// finite become NaN (e4m3 holds no infinity).
__device__ __forceinline__ uint2 quantise8(const uint4& w, float inv, bool odd) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = pack_e4m3x2(__uint_as_float(u[i] << 16) * inv,
                       __uint_as_float(u[i] & 0xffff0000u) * inv);
  }
  if (odd) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((u[i] & 0x7f80u) == 0x7f80u) o[i] |= 0x007fu;
      if ((u[i] & 0x7f800000u) == 0x7f800000u) o[i] |= 0x7f00u;
    }
  }
  return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

// Two e4m3 values (the low 16 bits) as floats.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// One CTA per (request, touched page; key/value head; k or v): it reads the
// page's new tokens once into registers, takes their largest magnitude,
// settles the scale and writes the tokens.  The scale is the smallest power
// of two that holds the page's values within e4m3's range: a power of two
// costs e4m3 nothing (its spacing is relative), multiplies exactly, and makes
// the requantisation of older tokens, when a later token raises the scale,
// exact but for subnormals.  A page whose tokens all arrive in this call
// takes a fresh scale, whatever it held before.
//
// Bound by memory: 2 bytes read and 1 written per value; for short appends by
// the chain lengths -> page number -> scale -> tokens rounded anew, so the
// rows are read while the page number is on its way.  NT threads hold VPT
// vectors of 8 values each, the smallest block that holds a page's share:
// registers limit how many blocks, and so how many bytes, are in flight.
// Measured (8 heads of 128): 8 prompts of 8190 tokens 54 us (327 MB, 6.1 TB/s,
// 90% of what a copy reaches); 127 blocks of 32 tokens behind ragged lengths
// 8.7 us (10.7 with registers for 1024 vectors instead of 512); 64 single
// tokens 2.6 us (3.8 with four warps to a page instead of one).
template <int D, int NT, int VPT>
__global__ void __launch_bounds__(NT) dfa_cache_append_kernel(const AppendParams p) {
  constexpr int kVec = D / 8;  // vectors per token and head
  __shared__ unsigned s_top[NT / 32];
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
  unsigned top = 0;
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
  float* scale = p.scale[which] + static_cast<long long>(page) * p.Hk + h;
  const float was = *scale;
  // The page's largest magnitude, of every value first, two to an operation;
  // only a page with values that are not finite is looked at value by value.
  auto block_max = [&](unsigned x) {
    x = __reduce_max_sync(0xffffffffu, x);
    if constexpr (NT > 32) {
      if ((tid & 31) == 0) s_top[tid >> 5] = x;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) x = max(x, s_top[i]);
    }
    return x;
  };
#pragma unroll
  for (int u = 0; u < VPT; ++u)
    top = __vmaxu2(__vmaxu2(top, __vmaxu2(w[u].x & 0x7fff7fffu, w[u].y & 0x7fff7fffu)),
                   __vmaxu2(w[u].z & 0x7fff7fffu, w[u].w & 0x7fff7fffu));
  top = block_max(max(top & 0xffffu, top >> 16));
  const bool odd = top >= 0x7f80u;
  if (odd) {
    top = 0;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const uint32_t v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned lo = v[e] & 0x7fffu, hi = (v[e] >> 16) & 0x7fffu;
        top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
      }
    }
    if constexpr (NT > 32) __syncthreads();  // the first maxima have been read
    top = block_max(top);
  }
  int e = cache_scale_exp(top);
  float now = __int_as_float((e + 127) << 23);
  uint8_t* c = p.cache[which] + (static_cast<long long>(page) * p.Hk + h) * p.page_size * D;
  if (first > 0) {
    if (was >= now) {
      now = was;
    } else {
      const float ratio = was / now;
      uint2* old = reinterpret_cast<uint2*>(c);
      for (int i = tid; i < first * kVec; i += NT) {
        const uint2 v = old[i];
        const float2 f0 = unpack_e4m3x2(v.x), f1 = unpack_e4m3x2(v.x >> 16);
        const float2 f2 = unpack_e4m3x2(v.y), f3 = unpack_e4m3x2(v.y >> 16);
        old[i] = make_uint2(pack_e4m3x2(f0.x * ratio, f0.y * ratio) |
                                pack_e4m3x2(f1.x * ratio, f1.y * ratio) << 16,
                            pack_e4m3x2(f2.x * ratio, f2.y * ratio) |
                                pack_e4m3x2(f3.x * ratio, f3.y * ratio) << 16);
      }
    }
  }
  const float inv = 1.f / now;
  uint2* dst = reinterpret_cast<uint2*>(c + first * D);
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = u * NT + tid;
    if (i < nvec) dst[i] = quantise8(w[u], inv, odd);
  }
  if constexpr (NT > 32) __syncthreads();  // every thread has read the old scale
  else __syncwarp();
  if (tid == 0) *scale = now;
}

template <int D, int NT, int VPT>
cudaError_t launch_append_block(const AppendParams& p, unsigned blocks, cudaStream_t stream) {
  return launch_chained(dfa_cache_append_kernel<D, NT, VPT>, dim3(blocks), dim3(NT), 0, stream, p);
}

template <int D>
cudaError_t launch_append(const AppendParams& p, int batch, cudaStream_t stream) {
  const unsigned n = 2u * p.Hk * batch * p.touch;
  const int vectors = (p.max_new < p.page_size ? p.max_new : p.page_size) * (D / 8);
  if (vectors <= 128) return launch_append_block<D, 32, 4>(p, n, stream);
  if (vectors <= 512) return launch_append_block<D, 128, 4>(p, n, stream);
  // a page of 128 tokens is 1024, 2048 or 4096 vectors
  if constexpr (D == 128) {
    if (vectors > 1024) return launch_append_block<D, 256, 8>(p, n, stream);
  } else if constexpr (D == 256) {
    if (vectors > 1024) return launch_append_block<D, 256, 16>(p, n, stream);
  }
  return launch_append_block<D, 128, 8>(p, n, stream);
}

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" {

int dfa_cache_plan(const int* cache_lens, const int* new_lens, int* block_table,
                   const int* free_pages, const int* free_count, int* cu_new, int* positions,
                   int* next_lens, int* next_free, int* missing, int batch, int max_pages,
                   int num_free, int page_size, int rows, dfa_stream_t stream) {
  if (batch < 0 || max_pages < 1 || num_free < 0 || rows < 0 || rows > (1 << 30) ||
      !page_size_ok(page_size) || static_cast<long long>(max_pages) * page_size > (1 << 30))
    return DFA_EINVAL;
  if (!free_count || !cu_new || !next_free || !missing || (num_free && !free_pages) ||
      (rows && !positions) ||
      (batch && (!cache_lens || !new_lens || !block_table || !next_lens)))
    return DFA_EINVAL;
  for (const void* q : {static_cast<const void*>(cache_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_table),
                        static_cast<const void*>(free_pages), static_cast<const void*>(free_count),
                        static_cast<const void*>(cu_new), static_cast<const void*>(positions),
                        static_cast<const void*>(next_lens), static_cast<const void*>(next_free),
                        static_cast<const void*>(missing)})
    if (!aligned_to(q, 4)) return DFA_EINVAL;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  const PlanParams p{cache_lens, new_lens,  block_table, free_pages, free_count,
                     cu_new,     positions, next_lens,   next_free,  missing,
                     di.status,  batch,     max_pages,   num_free,   page_size,
                     rows};
  // A cluster of eight CTAs where the stores take more than one CTA a few
  // passes, one CTA for a handful of requests: 1024 requests of 32 rows 10.5 us
  // with eight, 36.5 with one; 5 requests of 16 rows 3.6 us with one, 3.7 with
  // eight.
  const unsigned parts = rows > 4 * kPlanThreads ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, dfa_cache_plan_kernel, p);
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

int dfa_cache_scale_exp(unsigned bits) { return cache_scale_exp(bits); }
int dfa_cache_page_ok(int page, int num_pages) { return cache_page_ok(page, num_pages) ? 1 : 0; }
int dfa_cache_append_pages(int max_new, int page_size) {
  if (max_new < 0 || !page_size_ok(page_size)) return DFA_EINVAL;
  return cache_append_pages(max_new, page_size);
}
int dfa_cache_append_span(int len, int n, int j, int page_size, int* span) {
  if (len < 0 || n < 0 || j < 0 || !page_size_ok(page_size) || !span) return DFA_EINVAL;
  const Interval s = cache_append_range(len, n, j, page_size);
  span[0] = s.lo;
  span[1] = s.hi;
  return DFA_OK;
}
int dfa_cache_units(int len, int n, int unit, int finish) {
  if (len < 0 || unit < 0 || finish < 1) return DFA_EINVAL;
  return cache_units(len, n, unit, finish);
}
int dfa_cache_blocks(long long total, int limit) {
  if (total < 0 || limit < 1) return DFA_EINVAL;
  return cache_blocks(total, limit);
}
long long dfa_cache_run(int x, long long total, int blocks) {
  if (total < 0 || blocks < 1 || x < 0 || x > blocks) return DFA_EINVAL;
  return cache_run(x, total, blocks);
}
int dfa_cache_owner(long long w, long long total, int blocks) {
  if (blocks < 1 || w < 0 || w >= total) return DFA_EINVAL;
  return cache_owner(w, total, blocks);
}
int dfa_cache_own_end(int len, int i, int n, int block_size) {
  if (len < 0 || i < 0 || i >= n || block_size < 1) return DFA_EINVAL;
  return cache_own_end(len, i, n, block_size);
}

int dfa_cache_release(const int* finished, int* cache_lens, int* block_table, int* free_pages,
                      int* free_count, int batch, int max_pages, int num_free, int page_size,
                      dfa_stream_t stream) {
  if (batch < 0 || max_pages < 1 || num_free < 0 || !page_size_ok(page_size) ||
      static_cast<long long>(max_pages) * page_size > (1 << 30))
    return DFA_EINVAL;
  if (batch == 0) return DFA_OK;
  if (!finished || !cache_lens || !block_table || !free_pages || !free_count) return DFA_EINVAL;
  for (const void* q : {static_cast<const void*>(finished), static_cast<const void*>(cache_lens),
                        static_cast<const void*>(block_table),
                        static_cast<const void*>(free_pages),
                        static_cast<const void*>(free_count)})
    if (!aligned_to(q, 4)) return DFA_EINVAL;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  const ReleaseParams p{finished,  cache_lens, block_table, free_pages, free_count,
                        di.status, batch,      max_pages,   num_free,   page_size};
  const cudaError_t e = launch_chained(dfa_cache_release_kernel, dim3(1), dim3(kPlanThreads), 0,
                                       static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

int dfa_cache_append(const void* k, const void* v, const int* cu_new, const int* cache_lens,
                     const int* block_table, void* k_cache, void* v_cache, float* k_scale,
                     float* v_scale, int batch, int rows, int max_new, int kv_heads, int headdim,
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
    if (!q || !aligned_to(q, 16)) return DFA_EINVAL;
  for (const void* q : {static_cast<const void*>(cu_new), static_cast<const void*>(cache_lens),
                        static_cast<const void*>(block_table), static_cast<const void*>(k_scale),
                        static_cast<const void*>(v_scale)})
    if (!q || !aligned_to(q, 4)) return DFA_EINVAL;
  AppendParams p{};
  const long long* strides[2] = {k_strides, v_strides};
  for (int i = 0; i < 2; ++i) {
    p.x[i] = static_cast<const __nv_bfloat16*>(i ? v : k);
    p.sr[i] = strides[i] ? strides[i][0] : static_cast<long long>(kv_heads) * headdim;
    p.sh[i] = strides[i] ? strides[i][1] : headdim;
    if ((p.sr[i] & 7) || (p.sh[i] & 7)) return DFA_EINVAL;
    p.cache[i] = static_cast<uint8_t*>(i ? v_cache : k_cache);
    p.scale[i] = i ? v_scale : k_scale;
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

}  // extern "C"
