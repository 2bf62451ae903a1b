// flint_path.cu -- append of the accepted path of a drafted tree to every
// layer's cache: the k and v of node path[b][j] go to position L_b + j of
// request b, in any layout, quantised for an E4M3 cache (code = e4m3(float32
// value / scale), nearest even, saturating).  Bound by latency and, for a
// full batch over all layers, by HBM: each accepted token's 2 KiB is read and
// written once per layer.
//
// One CTA per (token of a path, request, up to 8 layers): two layers at a time, 32
// threads for k and 32 for v, 16 values each, with the loads of all its layers in
// flight together.  64 requests of up to 8 tokens, 49 E4M3 layers: 9 to 11 us for 38 MB
// (the two dependent loads, then the arithmetic of the codes); 14 bf16 layers of one
// request: 2.0 us.
#include <algorithm>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

constexpr int kApThreads = 128;
constexpr int kApLayers = 8;               // layers a CTA has in flight, at most

// The codes of 8 values over s, each quotient a float32 rounded to nearest.  q = x
// r with r = 1 / s rounded is within 2^-23 of the quotient, two units in the last
// place; codes change only at numbers of 5 significant bits (midpoints of codes),
// so unless q is within 3 units of such a number the quotient itself has q's code.
// Where one of the 8 is, or 1 / s may not be a normal number (r = 0), division
// decides.
__device__ __forceinline__ uint2 codes_of(uint4 x, float s, float r) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t code[4], far = 0x7FFFFu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = bf16_lo(w[i]) * r, b = bf16_hi(w[i]) * r;
    far = min(far, min((__float_as_uint(a) + 3u) & 0x7FFFFu, (__float_as_uint(b) + 3u) & 0x7FFFFu));
    code[i] = f32x2_to_e4m3x2(a, b);
  }
  if (far <= 6u) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
      const uint32_t z = f32x2_to_e4m3x2(__fdiv_rn(bf16_lo(y), s), __fdiv_rn(bf16_hi(y), s));
      if (i == 0) code[0] = z;
      else if (i == 1) code[1] = z;
      else if (i == 2) code[2] = z;
      else code[3] = z;
    }
  }
  return make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
}

__global__ void __launch_bounds__(kApThreads) append_path_kernel(const __grid_constant__ AppendPathParams p, int layers) {
  const int b = blockIdx.y, j = blockIdx.x, l0 = blockIdx.z * layers, nl = min(layers, p.n_layers - l0);
  const int n = p.n_accepted[b], node = p.path[static_cast<long long>(b) * p.N + j], pos = p.len[b] + j;
  if (n < 0 || n > p.N) {
    if (threadIdx.x == 0) report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
    return;
  }
  if (j >= n) return;
  const int c = threadIdx.x & 31;  // 16-dim chunk of the token's 512 values
  const bool is_v = threadIdx.x & 32;
  const int k0 = threadIdx.x >> 6;  // layers k0, k0 + 2, ..
  const bool exists = node >= 0 && node < p.N;
  const long long from = (static_cast<long long>(b) * p.N + node) * kKvHeads * kDim;
  uint4 x[kApLayers / 2][2];
  int blk[kApLayers / 2];
#pragma unroll
  for (int i = 0; i < kApLayers / 2; ++i) {
    if (k0 + 2 * i >= nl) continue;
    const PathLayer& ly = p.layer[l0 + k0 + 2 * i];
    if (exists) {
      const uint4* src = reinterpret_cast<const uint4*>((is_v ? ly.v : ly.k) + from) + 2 * c;
      x[i][0] = src[0];
      x[i][1] = src[1];
    }
    blk[i] = -1;
    if (ly.layout == FLINT_KV_PAGED && pos / kBlock < ly.max_blocks) blk[i] = ly.table[static_cast<long long>(b) * ly.max_blocks + pos / kBlock];
  }
#pragma unroll
  for (int i = 0; i < kApLayers / 2; ++i) {
    if (k0 + 2 * i >= nl) continue;
    const PathLayer& ly = p.layer[l0 + k0 + 2 * i];
    long long row = -1;  // element offset of the slot
    if (exists) {
      if (ly.layout == FLINT_KV_PAGED) {
        if (blk[i] >= 0 && blk[i] < ly.num_blocks) row = (static_cast<long long>(blk[i]) * kBlock + pos % kBlock) * kKvHeads * kDim;
      } else if (ly.layout == FLINT_KV_RING || pos < ly.capacity) {
        row = b * ly.req_stride + static_cast<long long>(pos % ly.capacity) * kKvHeads * kDim;
      }
    }
    if (row < 0) {
      if (c == 0) report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
      continue;
    }
    uint8_t* dst = is_v ? ly.v_rows : ly.k_rows;
    if (!ly.fp8) {
      uint4* to = reinterpret_cast<uint4*>(dst + 2 * row) + 2 * c;
      to[0] = x[i][0];
      to[1] = x[i][1];
    } else {
      const float s = is_v ? ly.v_scale[c / 8] : ly.k_scale[c / 8], r = is_v ? ly.v_inv[c / 8] : ly.k_inv[c / 8];
      const uint2 a = codes_of(x[i][0], s, r), d = codes_of(x[i][1], s, r);
      reinterpret_cast<uint4*>(dst + row)[c] = make_uint4(a.x, a.y, d.x, d.y);
    }
  }
}

}  // namespace

cudaError_t launch_append_path(const AppendPathParams& p, int num_sms, cudaStream_t stream) {
  // as many layers a CTA as leave a full set of CTAs (16 a SM)
  const long long jobs = static_cast<long long>(p.B) * p.N * p.n_layers;
  const int layers = static_cast<int>(std::min<long long>(kApLayers, std::max<long long>(1, jobs / (16ll * num_sms))));
  append_path_kernel<<<dim3(p.N, p.B, (p.n_layers + layers - 1) / layers), kApThreads, 0, stream>>>(p, layers);
  return cudaGetLastError();
}

}  // namespace flint
