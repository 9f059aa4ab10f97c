// Attention of new rows over a paged key/value cache: the join of what a launch has
// cut, the launch's shape, the entry points.  The kernels: cache_rows.cuh (up to 32
// rows to a key), cache_wide.cuh (more).
#include <cmath>

#include "cache_rows.cuh"
#include "device.cuh"
#include "dfa.h"

namespace dfa {
namespace {

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

long long cache_workspace_bytes(int batch, int rows, int max_new, int heads, int kv_heads,
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

template <int BITS>
int cache_forward(const void* q, const void* k, const void* v, const void* k_cache,
                  const void* v_cache, const void* k_scale, const void* v_scale,
                  const int* block_table, const int* cache_lens, const int* cu_new, void* out,
                  float* lse, void* workspace, long long workspace_bytes, int batch, int rows,
                  int max_new, int heads, int kv_heads, int headdim, int block_size,
                  int page_size, int num_pages, int max_pages, const long long* q_strides,
                  const long long* k_strides, const long long* v_strides, dfa_stream_t stream) {
  if (const int rc = check_cache_sizes(batch, rows, max_new, heads, kv_heads, headdim, page_size,
                                       max_pages))
    return rc;
  if (block_size < 1 || num_pages < 1) return DFA_EINVAL;
  if (batch == 0 || rows == 0 || max_new == 0) return DFA_OK;
  auto aligned = [](const void* x, unsigned n) {
    return x && (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0;
  };
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(k_scale, BITS == 8 ? 4 : 16) ||
      !aligned(v_scale, BITS == 8 ? 4 : 16) ||
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
  CacheParams<BITS> p{};
  const bool wide = c.tile_rows == 128;  // its boxes are whole pages
  const int box_keys = !wide && page_size > kUnit ? kUnit : page_size;
  const cuuint64_t head_keys = static_cast<cuuint64_t>(kv_heads) * page_size;
  // A row of a map: a token's values, or 4 bits: of two tokens up to headdim 128.
  const int pair = BITS == 4 && d < 256 ? 2 : 1, width = d * pair * BITS / 8;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), head_keys / pair,
                              static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width), dims[1] * width};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(width < 128 ? width : 128),
                             static_cast<cuuint32_t>(box_keys / pair), 1};
  const CUtensorMapSwizzle swizzle =
      d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (const int rc = encode_map_u8(&p.tm_k, k_cache, 3, dims, strides, box, swizzle)) return rc;
  if (const int rc = encode_map_u8(&p.tm_v, v_cache, 3, dims, strides, box, swizzle)) return rc;
  if constexpr (BITS == 4) {
    const cuuint64_t groups = static_cast<cuuint64_t>(kv_heads) * (d / kCache4Group);
    const cuuint64_t sdims[3] = {static_cast<cuuint64_t>(page_size), groups, dims[2]};
    const cuuint64_t sstrides[2] = {sdims[0], sdims[0] * groups};
    const cuuint32_t sbox[3] = {static_cast<cuuint32_t>(box_keys),
                                static_cast<cuuint32_t>(d / kCache4Group), 1};
    for (int i = 0; i < 2; ++i)
      if (const int rc = encode_map_u8(i ? &p.tm_vs : &p.tm_ks, i ? v_scale : k_scale, 3, sdims,
                                       sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE))
        return rc;
  } else {
    p.k_scale = static_cast<const float*>(k_scale);
    p.v_scale = static_cast<const float*>(v_scale);
  }
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
  cudaError_t e;
  if constexpr (BITS == 4)
    e = launch_cache4_rows(p, d, c.tile_rows, s);
  else
    e = d == 64    ? launch_cache_rows<8, 64>(p, c.tile_rows, s)
        : d == 128 ? launch_cache_rows<8, 128>(p, c.tile_rows, s)
                   : launch_cache_rows<8, 256>(p, c.tile_rows, s);
  if (e == cudaSuccess && !c.whole) {
    auto join = d == 64 ? dfa_cache_join_kernel<64>
                        : d == 128 ? dfa_cache_join_kernel<128> : dfa_cache_join_kernel<256>;
    const int rows = (c.tile_rows + kJoinWarps - 1) / kJoinWarps;
    const dim3 grid(c.blocks, rows < 16 ? rows : 16);
    e = launch_chained(join, grid, dim3(32 * kJoinWarps), 0, s, static_cast<CacheFwdParams>(p));
  }
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" {

long long dfa_cache_workspace_bytes(int batch, int rows, int max_new, int heads, int kv_heads,
                                    int headdim, int page_size, int max_pages) {
  return cache_workspace_bytes(batch, rows, max_new, heads, kv_heads, headdim, page_size,
                               max_pages);
}
long long dfa_cache4_workspace_bytes(int batch, int rows, int max_new, int heads, int kv_heads,
                                     int headdim, int page_size, int max_pages) {
  return cache_workspace_bytes(batch, rows, max_new, heads, kv_heads, headdim, page_size,
                               max_pages);
}

int dfa_cache_forward(const void* q, const void* k, const void* v, const void* k_cache,
                      const void* v_cache, const float* k_scale, const float* v_scale,
                      const int* block_table, const int* cache_lens, const int* cu_new, void* out,
                      float* lse, void* workspace, long long workspace_bytes, int batch, int rows,
                      int max_new, int heads, int kv_heads, int headdim, int block_size,
                      int page_size, int num_pages, int max_pages, const long long* q_strides,
                      const long long* k_strides, const long long* v_strides,
                      dfa_stream_t stream) {
  return cache_forward<8>(q, k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_lens,
                          cu_new, out, lse, workspace, workspace_bytes, batch, rows, max_new,
                          heads, kv_heads, headdim, block_size, page_size, num_pages, max_pages,
                          q_strides, k_strides, v_strides, stream);
}
int dfa_cache4_forward(const void* q, const void* k, const void* v, const void* k_cache,
                      const void* v_cache, const void* k_scale, const void* v_scale,
                      const int* block_table, const int* cache_lens, const int* cu_new, void* out,
                      float* lse, void* workspace, long long workspace_bytes, int batch, int rows,
                      int max_new, int heads, int kv_heads, int headdim, int block_size,
                      int page_size, int num_pages, int max_pages, const long long* q_strides,
                      const long long* k_strides, const long long* v_strides,
                      dfa_stream_t stream) {
  return cache_forward<4>(q, k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_lens,
                          cu_new, out, lse, workspace, workspace_bytes, batch, rows, max_new,
                          heads, kv_heads, headdim, block_size, page_size, num_pages, max_pages,
                          q_strides, k_strides, v_strides, stream);
}

}  // extern "C"
