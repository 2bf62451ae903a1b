// flint_path.cu -- append of the accepted path of a drafted tree to every
// layer's cache: the k and v of node path[b][j] go to position L_b + j of
// request b, in any layout, quantised for an E4M3 cache (code = e4m3(float32
// value / scale), nearest even, saturating).  Bound by latency and, for a
// full batch over all layers, by HBM: each accepted token's 2 KiB is read and
// written once per layer.
//
// One CTA per (request, layer); warps take the path's tokens in turn, four warps
// to a token (k and v of 512 values, 8 a lane), so that the tokens of a path are
// in flight together.
#include <algorithm>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

constexpr int kApTokens = 2;               // tokens a CTA has in flight
constexpr int kApThreads = 128 * kApTokens;

// The code of x / s, the quotient a float32 rounded to nearest.  q0 = x r with r
// = 1 / s rounded is within 2^-23 of the quotient, two units in the last place;
// codes change only at numbers of 5 significant bits (midpoints of codes), so
// unless q0 is within 3 units of such a number the quotient itself has q0's code.
// There, and where 1 / s may not be a normal number (r = 0), the division decides.
__device__ __forceinline__ float quotient_for_code(float x, float s, float r) {
  const float q0 = x * r;
  if (((__float_as_uint(q0) + 3u) & 0x7FFFFu) > 6u) return q0;
  return __fdiv_rn(x, s);
}

__global__ void __launch_bounds__(kApThreads) append_path_kernel(const __grid_constant__ AppendPathParams p) {
  const int b = blockIdx.x;
  const PathLayer& ly = p.layer[blockIdx.y];
  const int c = threadIdx.x & 63;  // 8-dim chunk of the token's 512 values
  const bool is_v = threadIdx.x & 64;
  const int n = p.n_accepted[b];
  if (n < 0 || n > p.N) {
    if (threadIdx.x == 0) report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
    return;
  }
  const float s = is_v ? ly.v_scale[c / 16] : ly.k_scale[c / 16];
  const float r = s > 1e-30f && s < 1e30f ? 1.0f / s : 0.f;
  for (int j = threadIdx.x / 128; j < n; j += kApTokens) {
    const int node = p.path[static_cast<long long>(b) * p.N + j], pos = p.len[b] + j;
    long long row = -1;  // element offset of the slot
    if (node >= 0 && node < p.N) {
      if (ly.layout == FLINT_KV_PAGED) {
        if (pos / kBlock < ly.max_blocks) {
          const int blk = ly.table[static_cast<long long>(b) * ly.max_blocks + pos / kBlock];
          if (blk >= 0 && blk < ly.num_blocks) row = (static_cast<long long>(blk) * kBlock + pos % kBlock) * kKvHeads * kDim;
        }
      } else if (ly.layout == FLINT_KV_RING || pos < ly.capacity) {
        row = b * ly.req_stride + static_cast<long long>(pos % ly.capacity) * kKvHeads * kDim;
      }
    }
    if (row < 0) {
      if (c == 0) report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
      continue;
    }
    const uint4 x = reinterpret_cast<const uint4*>((is_v ? ly.v : ly.k) + (static_cast<long long>(b) * p.N + node) * kKvHeads * kDim)[c];
    uint8_t* dst = is_v ? ly.v_rows : ly.k_rows;
    if (!ly.fp8) {
      *reinterpret_cast<uint4*>(dst + 2 * (row + 8 * c)) = x;
    } else {
      auto two = [&](uint32_t w) { return f32x2_to_e4m3x2(quotient_for_code(bf16_lo(w), s, r), quotient_for_code(bf16_hi(w), s, r)); };
      *reinterpret_cast<uint2*>(dst + row + 8 * c) = make_uint2(two(x.x) | two(x.y) << 16, two(x.z) | two(x.w) << 16);
    }
  }
}

}  // namespace

cudaError_t launch_append_path(const AppendPathParams& p, cudaStream_t stream) {
  append_path_kernel<<<dim3(p.B, p.n_layers), kApThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flint
