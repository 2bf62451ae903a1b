// flint_path.cu -- append of the accepted path of a drafted tree to every
// layer's cache: the k and v of node path[b][j] go to position L_b + j of
// request b, in any layout, quantised for an E4M3 cache (code = e4m3(float32
// value / scale), nearest even, saturating).  Bound by latency and, for a
// full batch over all layers, by HBM: each accepted token's 2 KiB is read and
// written once per layer.
//
// One CTA per (request, layer); 128 threads, 64 for k and 64 for v, 8 dims each.
#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

__global__ void __launch_bounds__(128) append_path_kernel(const __grid_constant__ AppendPathParams p) {
  const int b = blockIdx.x;
  const PathLayer& ly = p.layer[blockIdx.y];
  const bool is_v = threadIdx.x >= 64;
  const int c = threadIdx.x & 63;  // 8-dim chunk of the token's 512 values
  int n = p.n_accepted[b];
  if (n < 0 || n > p.N) {
    if (threadIdx.x == 0) report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
    return;
  }
  for (int j = 0; j < n; ++j) {
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
      if (threadIdx.x == 0) report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
      continue;
    }
    const uint4 x = reinterpret_cast<const uint4*>((is_v ? ly.v : ly.k) + (static_cast<long long>(b) * p.N + node) * kKvHeads * kDim)[c];
    uint8_t* dst = is_v ? ly.v_rows : ly.k_rows;
    if (!ly.fp8) {
      *reinterpret_cast<uint4*>(dst + 2 * (row + 8 * c)) = x;
    } else {
      const float s = is_v ? ly.v_scale[c / 16] : ly.k_scale[c / 16];
      auto two = [&](uint32_t w) { return f32x2_to_e4m3x2(__fdiv_rn(bf16_lo(w), s), __fdiv_rn(bf16_hi(w), s)); };
      *reinterpret_cast<uint2*>(dst + row + 8 * c) = make_uint2(two(x.x) | two(x.y) << 16, two(x.z) | two(x.w) << 16);
    }
  }
}

}  // namespace

cudaError_t launch_append_path(const AppendPathParams& p, cudaStream_t stream) {
  append_path_kernel<<<dim3(p.B, p.n_layers), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flint
