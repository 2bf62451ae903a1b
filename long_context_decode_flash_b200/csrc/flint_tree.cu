// flint_tree.cu -- attention of drafted tokens over a committed cache and
// their own tree: node i of request b, at depth d_i (its ancestors), attends
// the cached positions [max(0, L + d_i - window + 1), L) (or all of [0, L)),
// its ancestors and itself,
//     out = sum_j e^(s_j - M) V_j / (sum_j e^(s_j - M) + e^(sink - M)),
//     s_j = q . K_j / sqrt(128),  M = max(max_j s_j, sink).
//
// One warp per (request, node, query head), a lane per 4 dims: one pass over
// the keys with the running maximum and sum.
#include <math.h>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

__device__ __forceinline__ float4 load4(const uint8_t* rows, long long row, int g, int lane, bool fp8, float scale) {
  if (fp8) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(rows + row * (kKvHeads * kDim) + g * kDim + 4 * lane);
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(c, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
  }
  const uint2 c = *reinterpret_cast<const uint2*>(rows + (row * (kKvHeads * kDim) + g * kDim + 4 * lane) * 2);
  return make_float4(bf16_lo(c.x), bf16_hi(c.x), bf16_lo(c.y), bf16_hi(c.y));
}

__device__ __forceinline__ float quantised(float x, float scale) {
  const uint32_t c = f32x2_to_e4m3x2(__fdiv_rn(x, scale), 0.f);
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(c, lo, hi);
  return __half22float2(*reinterpret_cast<__half2*>(&lo)).x * scale;
}

__global__ void __launch_bounds__(256) tree_kernel(const __grid_constant__ TreeParams p) {
  const int b = blockIdx.y / kKvHeads, g = blockIdx.y % kKvHeads, i = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = g * kGroup + warp;
  if (i >= p.n_draft[b]) return;
  const int L = p.len[b];
  const int32_t* parent = p.parent + static_cast<long long>(b) * p.N;
  unsigned long long line = 0;
  for (int j = i; j >= 0;) {
    line |= 1ull << j;
    const int up = parent[j];
    if (up < -1 || up >= j) {
      report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
      break;
    }
    j = up;
  }
  const int depth = __popcll(line) - 1;
  const float scale = 0.08838834764831845f;
  const long long node = static_cast<long long>(b) * p.N + i;
  const uint2 qr = reinterpret_cast<const uint2*>(p.q + (node * kHeads + h) * kDim)[lane];
  const float4 q = make_float4(bf16_lo(qr.x) * scale, bf16_hi(qr.x) * scale, bf16_lo(qr.y) * scale, bf16_hi(qr.y) * scale);
  const float ks = p.fp8 ? p.k_scale[g] : 1.f, vs = p.fp8 ? p.v_scale[g] : 1.f;
  float m = p.sinks[h], l = m == -INFINITY ? 0.f : 1.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto take = [&](const float4& k, const float4& v) {
    float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : expf(m - mn), e = mn == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * a + e;
    o = make_float4(o.x * a + e * v.x, o.y * a + e * v.y, o.z * a + e * v.z, o.w * a + e * v.w);
  };
  for (int t = p.window > 0 ? max(0, L + depth - p.window + 1) : 0; t < L; ++t) {
    long long row;
    if (p.layout == FLINT_KV_PAGED) {
      const int blk = p.table[static_cast<long long>(b) * p.max_blocks + t / kBlock];
      if (blk < 0 || blk >= p.num_blocks) {
        report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
        continue;
      }
      row = static_cast<long long>(blk) * kBlock + t % kBlock;
    } else {
      row = b * (p.req_stride / (kKvHeads * kDim)) + (p.layout == FLINT_KV_RING ? t % p.capacity : t);
    }
    // a request stride that is no whole number of rows
    const long long off = p.layout == FLINT_KV_PAGED ? 0 : b * (p.req_stride % (kKvHeads * kDim)) * (p.fp8 ? 1 : 2);
    take(load4(p.k_rows + off, row, g, lane, p.fp8, ks), load4(p.v_rows + off, row, g, lane, p.fp8, vs));
  }
  for (int j = 0; j <= i; ++j)
    if (line >> j & 1) {
      const long long row = static_cast<long long>(b) * p.N + j;
      float4 k = load4(reinterpret_cast<const uint8_t*>(p.k_draft), row, g, lane, false, 1.f);
      float4 v = load4(reinterpret_cast<const uint8_t*>(p.v_draft), row, g, lane, false, 1.f);
      if (p.fp8) {
        k = make_float4(quantised(k.x, ks), quantised(k.y, ks), quantised(k.z, ks), quantised(k.w, ks));
        v = make_float4(quantised(v.x, vs), quantised(v.y, vs), quantised(v.z, vs), quantised(v.w, vs));
      }
      take(k, v);
    }
  const float r = 1.f / l;
  reinterpret_cast<uint2*>(p.out + (node * kHeads + h) * kDim)[lane] =
      make_uint2(pack_bf16x2(o.x * r, o.y * r), pack_bf16x2(o.z * r, o.w * r));
}

}  // namespace

cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  tree_kernel<<<dim3(p.N, p.B * kKvHeads), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flint
