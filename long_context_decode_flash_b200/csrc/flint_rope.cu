// flint_rope.cu -- per-head Q/K RMSNorm and rotary positions of T tokens at
// given positions, in either pair layout, on the first rotary_dim dims, with
// per-pair frequencies from the host:
//     y = x w / sqrt(mean(x^2) + eps),
//     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin),  angle pos f_i.
// The angle is formed in double as pos * (f_i / 2 pi) turns and reduced to
// [-1/2, 1/2] turns before its cos and sin are taken in float32.
//
// One CTA per token; a warp per row, partners of a pair through shared memory.
#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

constexpr int kRaThreads = 256;

__global__ void __launch_bounds__(kRaThreads) rope_at_kernel(const __grid_constant__ RopeAtParams p) {
  __shared__ float2 cs[kDim / 2];
  __shared__ float rows[kRaThreads / 32][kDim];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < p.rotary_dim / 2) {
    const double turns = p.pos[t] * p.turns[threadIdx.x];
    float s, c;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
    cs[threadIdx.x] = make_float2(c * p.attn_factor, s * p.attn_factor);
  }
  __syncthreads();
  for (int r = warp; r < kHeads + kKvHeads; r += kRaThreads / 32) {
    const bool is_q = r < kHeads;
    if (!(is_q ? p.q_out : p.k_out)) continue;
    const uint16_t* x = is_q ? p.q_raw + t * p.q_stride + r * kDim : p.k_raw + t * p.k_stride + (r - kHeads) * kDim;
    uint16_t* o = is_q ? p.q_out + (static_cast<long long>(t) * kHeads + r) * kDim
                       : p.k_out + (static_cast<long long>(t) * kKvHeads + r - kHeads) * kDim;
    const uint16_t* w = is_q ? p.w_q : p.w_k;
    const uint2 raw = reinterpret_cast<const uint2*>(x)[lane];
    float y[4] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y)};
    if (w) {
      float ss = y[0] * y[0] + y[1] * y[1] + y[2] * y[2] + y[3] * y[3];
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
      const float inv = 1.0f / sqrtf(ss * (1.0f / kDim) + p.eps);
      const uint2 wr = reinterpret_cast<const uint2*>(w)[lane];
      y[0] = y[0] * inv * bf16_lo(wr.x);
      y[1] = y[1] * inv * bf16_hi(wr.x);
      y[2] = y[2] * inv * bf16_lo(wr.y);
      y[3] = y[3] * inv * bf16_hi(wr.y);
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) rows[warp][4 * lane + e] = y[e];
    __syncwarp();
    const int half = p.rotary_dim / 2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 4 * lane + e;
      if (d >= p.rotary_dim) continue;
      const bool second = p.layout == FLINT_ROPE_INTERLEAVED ? (d & 1) : d >= half;
      const int i = p.layout == FLINT_ROPE_INTERLEAVED ? d >> 1 : (second ? d - half : d);
      const int other = p.layout == FLINT_ROPE_INTERLEAVED ? d ^ 1 : (second ? d - half : d + half);
      const float2 a = cs[i];
      const float z = rows[warp][other];
      y[e] = second ? y[e] * a.x + z * a.y : y[e] * a.x - z * a.y;
    }
    reinterpret_cast<uint2*>(o)[lane] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  }
}

}  // namespace

cudaError_t launch_rope_at(const RopeAtParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  rope_at_kernel<<<p.T, kRaThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flint
