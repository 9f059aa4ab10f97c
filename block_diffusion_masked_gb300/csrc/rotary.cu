// Rotary positions of queries and keys, forward and backward.
//
// A head's first rot_dim values are rot_dim / 2 pairs; pair i at position p
// turns by the angle whose cosine and sine the table holds at (p, i) and
// (p, rot_dim / 2 + i):
//   y1 = c x1 - s x2,  y2 = s x1 + c x2.
// The pair is (i, i + rot_dim / 2) in the half layout and (2i, 2i + 1) in the
// interleaved one; the remaining headdim - rot_dim values pass through.  The
// map is linear, its transpose (the backward pass) has s replaced by -s.
//
// In the [noisy | clean] layout ("Fast Diffusion Attention", "Block diffusion
// in one picture") both halves hold positions 0 .. n - 1: row r of a sample
// has position r mod n, so no position array is read.
//
// Bound by memory: 2 bytes read and 2 written per value, 3 flops a value.
// One thread takes a unit of 16 values (8 pairs: two 16-byte loads and two
// stores) of kHeads heads of one row, so the row's cosines and sines (64
// bytes a thread) are loaded once per kHeads heads and stay in registers.
// Arithmetic in float32, one rounding to bf16.
//
// Measured: a pass (forward or backward) over 538 MB of headdim 128 takes 74
// us, one over 340 MB of headdim 256, interleaved, 48 us: 7.2 and 7.0 TB/s, a
// little above what a copy from memory to memory reaches (the last output
// stays in L2).  40 heads of 64 packed rows take 2.8 us, a launch's latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device.cuh"
#include "dfa.h"
#include "params.cuh"
#include "sm100.cuh"

namespace dfa {
namespace {

struct RotaryTensor {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;  // contiguous (batch, rows, heads, headdim)
  long long sb, sr, sh;  // strides of x in elements: batch, row, head
  int heads;
};

struct RotaryParams {
  RotaryTensor q, k;
  const float* table;    // (max_pos, rot): cosines, then sines
  const int* positions;  // (batch * rows) or null: row mod period
  unsigned* status;
  long long items;  // batch * rows * head groups
  int rows, period, max_pos, rot, groups;
  float sign;  // -1: the transposed map
  bool clear;  // rows that are not in use are set to zero, not left
};

constexpr int kHeads = 4;

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <int D, bool INTER>
__global__ void __launch_bounds__(256) dfa_rotary_kernel(const RotaryParams p) {
  constexpr int kUnits = D / 16;  // threads per head
  const long long thread = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long item = thread / kUnits;
  const int unit = static_cast<int>(thread % kUnits);
  grid_launch_dependents();
  grid_dependency_wait();  // q and k come from the kernels before this one
  if (item >= p.items) return;
  const long long row = item / p.groups;  // over batch and rows
  const int h0 = static_cast<int>(item - row * p.groups) * kHeads;
  const long long b = row / p.rows;
  const int r = static_cast<int>(row - b * p.rows);
  int pos = r;
  if (p.positions != nullptr) {
    pos = p.positions[row];
    if (pos >= p.max_pos) {
      if (unit == 0) atomicOr(p.status, kStatusIndex);
      pos = -1;
    }
    if (pos < 0) {  // a row that is not in use
      if (!p.clear) return;
      for (int h = h0; h < min(h0 + kHeads, p.q.heads + p.k.heads); ++h) {
        const bool isq = h < p.q.heads;
        const RotaryTensor& t = isq ? p.q : p.k;
        uint4* y = reinterpret_cast<uint4*>(
            t.y + (row * t.heads + (isq ? h : h - p.q.heads)) * D + 16 * unit);
        y[0] = y[1] = make_uint4(0u, 0u, 0u, 0u);
      }
      return;
    }
  } else if (pos >= p.period) {
    pos %= p.period;
  }
  const bool turned = 16 * unit < p.rot;
  // the two 8-value pieces of the unit inside a head
  const int o0 = turned && !INTER ? 8 * unit : 16 * unit;
  const int o1 = turned && !INTER ? p.rot / 2 + 8 * unit : 16 * unit + 8;
  uint4 a[kHeads], c[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = h0 + j;
    if (h >= p.q.heads + p.k.heads) break;
    const bool isq = h < p.q.heads;
    const RotaryTensor& t = isq ? p.q : p.k;
    const __nv_bfloat16* x = t.x + b * t.sb + r * t.sr + (isq ? h : h - p.q.heads) * t.sh;
    a[j] = *reinterpret_cast<const uint4*>(x + o0);
    c[j] = *reinterpret_cast<const uint4*>(x + o1);
  }
  float co[8], si[8];
  if (turned) {
    const float4* t = reinterpret_cast<const float4*>(
        p.table + static_cast<long long>(pos) * p.rot + 8 * unit);
    const float4* u = reinterpret_cast<const float4*>(
        p.table + static_cast<long long>(pos) * p.rot + p.rot / 2 + 8 * unit);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = t[i], y = u[i];
      co[4 * i] = x.x, co[4 * i + 1] = x.y, co[4 * i + 2] = x.z, co[4 * i + 3] = x.w;
      si[4 * i] = y.x, si[4 * i + 1] = y.y, si[4 * i + 2] = y.z, si[4 * i + 3] = y.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) si[i] *= p.sign;
  }
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = h0 + j;
    if (h >= p.q.heads + p.k.heads) break;
    if (turned) {
      float x[16], y[16];
      unpack8(a[j], x);
      unpack8(c[j], x + 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int i1 = INTER ? 2 * i : i, i2 = INTER ? 2 * i + 1 : i + 8;
        y[i1] = co[i] * x[i1] - si[i] * x[i2];
        y[i2] = si[i] * x[i1] + co[i] * x[i2];
      }
      a[j] = pack8(y);
      c[j] = pack8(y + 8);
    }
    const bool isq = h < p.q.heads;
    const RotaryTensor& t = isq ? p.q : p.k;
    __nv_bfloat16* y = t.y + (row * t.heads + (isq ? h : h - p.q.heads)) * D;
    *reinterpret_cast<uint4*>(y + o0) = a[j];
    *reinterpret_cast<uint4*>(y + o1) = c[j];
  }
}

bool rotary_tensor(RotaryTensor* t, const void* x, void* y, const long long* strides, int rows,
                   int heads, int d) {
  t->x = static_cast<const __nv_bfloat16*>(x);
  t->y = static_cast<__nv_bfloat16*>(y);
  t->heads = heads;
  t->sh = strides ? strides[2] : d;
  t->sr = strides ? strides[1] : static_cast<long long>(heads) * d;
  t->sb = strides ? strides[0] : static_cast<long long>(rows) * heads * d;
  if (heads == 0) return true;
  if (!x || !y || (reinterpret_cast<uintptr_t>(x) & 15u) || (reinterpret_cast<uintptr_t>(y) & 15u))
    return false;
  return (t->sh & 7) == 0 && (t->sr & 7) == 0 && (t->sb & 7) == 0;
}

template <int D>
cudaError_t launch_rotary(const RotaryParams& p, bool interleaved, cudaStream_t stream) {
  const long long threads = p.items * (D / 16);
  const long long blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (interleaved) return launch_chained(dfa_rotary_kernel<D, true>, grid, dim3(256), 0, stream, p);
  return launch_chained(dfa_rotary_kernel<D, false>, grid, dim3(256), 0, stream, p);
}

}  // namespace
}  // namespace dfa

extern "C" int dfa_rotary(const void* q, const void* k, void* q_out, void* k_out,
                          const float* table, const int* positions, int batch, int rows,
                          int period, int heads, int kv_heads, int headdim, int rot_dim,
                          int max_pos, const long long* q_strides, const long long* k_strides,
                          int flags, dfa_stream_t stream) {
  using namespace dfa;
  if (batch < 0 || rows < 0 || heads < 0 || kv_heads < 0 || max_pos < 1 || rows > (1 << 30) ||
      heads > (1 << 20) || kv_heads > (1 << 20) || heads + kv_heads < 1)
    return DFA_EINVAL;
  if (flags & ~(DFA_ROTARY_INTERLEAVED | DFA_ROTARY_INVERSE | DFA_ROTARY_CLEAR)) return DFA_EINVAL;
  if (headdim != 64 && headdim != 128 && headdim != 256) return DFA_EUNSUPPORTED;
  if (rot_dim < 16 || rot_dim > headdim || rot_dim % 16) return DFA_EINVAL;
  if (!positions && (period < 1 || (rows < period ? rows : period) > max_pos)) return DFA_EINVAL;
  if (batch == 0 || rows == 0) return DFA_OK;
  if (!table || (reinterpret_cast<uintptr_t>(table) & 15u) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return DFA_EINVAL;
  RotaryParams p{};
  if (!rotary_tensor(&p.q, q, q_out, q_strides, rows, heads, headdim) ||
      !rotary_tensor(&p.k, k, k_out, k_strides, rows, kv_heads, headdim))
    return DFA_EINVAL;
  DeviceInfo di;
  if (const int rc = device_info(&di)) return rc;
  p.table = table;
  p.positions = positions;
  p.status = di.status;
  p.rows = rows;
  p.period = period;
  p.max_pos = max_pos;
  p.rot = rot_dim;
  p.groups = (heads + kv_heads + kHeads - 1) / kHeads;
  p.items = static_cast<long long>(batch) * rows * p.groups;
  p.sign = flags & DFA_ROTARY_INVERSE ? -1.f : 1.f;
  p.clear = flags & DFA_ROTARY_CLEAR;
  const bool inter = flags & DFA_ROTARY_INTERLEAVED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = headdim == 64    ? launch_rotary<64>(p, inter, s)
                        : headdim == 128 ? launch_rotary<128>(p, inter, s)
                                         : launch_rotary<256>(p, inter, s);
  return e == cudaSuccess ? DFA_OK : record_cuda_failure(e);
}
