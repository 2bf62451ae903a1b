// flint_rope.cu -- per-head Q/K RMSNorm and rotary positions of T tokens at
// given positions, in either pair layout, on the first rotary_dim dims, with
// per-pair frequencies from the host:
//     y = x w / sqrt(mean(x^2) + eps),
//     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin),  angle pos f_i.
// The angle is formed in double as pos * (f_i / 2 pi) turns and reduced to
// [-1/2, 1/2] turns before its cos and sin are taken in float32.
//
// Bound by HBM (each row read and written once) for many tokens, by latency for
// few.  A warp takes rows of one token, two at a time, 16 lanes of 8 dims each
// (16-byte loads, four pairs of rows in flight), so that cos, sin and the weights
// are formed once for all of them; few tokens are spread over up to 6 warps each.
// The partner of a value is in its own lane (interleaved), in another lane of its
// row at the same place (half layout, rotary_dim a multiple of 16), or else found
// through shared memory.  8,191 tokens: 28.4 us, 5.3 TB/s, 81 % of a plain copy's
// rate; 40 tokens: 3.9 us, most of it the launch.
#include <algorithm>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

constexpr int kRaWarps = 4, kRaThreads = kRaWarps * 32;

enum { kInLane, kByLanes, kByShared };

// Warp job: token job / parts, the row pairs of part job % parts.
template <int kAt>
__global__ void __launch_bounds__(kRaThreads) rope_at_kernel(const __grid_constant__ RopeAtParams p, int parts) {
  __shared__ double turns[kDim / 2];
  __shared__ float2 cs[kRaWarps][kDim / 2];
  __shared__ float rows[kAt == kByShared ? kRaWarps : 1][2 * kDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 15;
  const int half = p.rotary_dim / 2, d0 = 8 * c;  // this lane's dims d0 .. d0 + 7
  for (int i = threadIdx.x; i < half; i += kRaThreads) turns[i] = p.turns[i];
  __syncthreads();
  const int job = blockIdx.x * kRaWarps + warp, part = job % parts;
  const long long t = job / parts;
  if (t >= p.T) return;
  const int pos = p.pos[t];
  for (int i = lane; i < half; i += 32) {
    const double a = pos * turns[i];
    float s, co;
    sincospif(static_cast<float>(2.0 * (a - rint(a))), &s, &co);
    cs[warp][i] = make_float2(co * p.attn_factor, s * p.attn_factor);
  }
  __syncwarp();
  // a value's own: y cos + (its partner) sin, sin negative for the first of a pair
  constexpr int kCs = kAt == kInLane ? 4 : 8;
  float2 mine[kCs];
#pragma unroll
  for (int e = 0; e < kCs; ++e) {
    if (kAt == kInLane) {
      mine[e] = d0 / 2 + e < half ? cs[warp][d0 / 2 + e] : make_float2(1.f, 0.f);
    } else {
      const int d = d0 + e;
      const bool second = d >= half;
      mine[e] = d < 2 * half ? cs[warp][second ? d - half : d] : make_float2(1.f, 0.f);
      if (!second) mine[e].y = -mine[e].y;
    }
  }
  // `pairs` pairs of rows from `x` on to `o`
  auto turn = [&](const uint16_t* x, const uint16_t* w, uint16_t* o, int pairs) {
    float2 wf[4];
    if (w) {
      const uint4 wr = reinterpret_cast<const uint4*>(w)[c];
      const uint32_t wx[4] = {wr.x, wr.y, wr.z, wr.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) wf[e] = make_float2(bf16_lo(wx[e]), bf16_hi(wx[e]));
    }
    const uint4* from = reinterpret_cast<const uint4*>(x) + lane;  // (a pair of rows is 32 chunks)
    uint4* to = reinterpret_cast<uint4*>(o) + lane;
#pragma unroll 1
    for (int i0 = part; i0 < pairs; i0 += 4 * parts) {
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i * parts < pairs) raw[i] = from[(i0 + i * parts) * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i * parts >= pairs) break;
        const uint32_t r[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = make_float2(bf16_lo(r[e]), bf16_hi(r[e]));
        if (w) {
          float2 sq = mul2(y[0], y[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) sq = fma2(y[e], y[e], sq);
          float ss = sq.x + sq.y;
#pragma unroll
          for (int k = 8; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
          const float inv = rsqrtf(fmaf(ss, 1.0f / kDim, p.eps));
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = mul2(mul2(y[e], make_float2(inv, inv)), wf[e]);
        }
        if (kAt == kInLane) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (d0 / 2 + e < half)
              y[e] = make_float2(y[e].x * mine[e].x - y[e].y * mine[e].y, y[e].y * mine[e].x + y[e].x * mine[e].y);
        } else if (kAt == kByLanes) {  // half is a multiple of 8: whole lanes pair up
          const bool turned = d0 < 2 * half;
          const int other = turned ? (d0 >= half ? lane - half / 8 : lane + half / 8) : lane;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = __shfl_sync(0xffffffffu, y[e].x, other), v = __shfl_sync(0xffffffffu, y[e].y, other);
            if (turned)
              y[e] = make_float2(y[e].x * mine[2 * e].x + u * mine[2 * e].y, y[e].y * mine[2 * e + 1].x + v * mine[2 * e + 1].y);
          }
        } else {
          float* row = rows[warp] + (lane >> 4) * kDim;
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            row[d0 + 2 * e] = y[e].x;
            row[d0 + 2 * e + 1] = y[e].y;
          }
          __syncwarp();
          auto one = [&](float z, int e) {
            const int d = d0 + e;
            return d < 2 * half ? z * mine[e].x + row[d >= half ? d - half : d + half] * mine[e].y : z;
          };
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = make_float2(one(y[e].x, 2 * e), one(y[e].y, 2 * e + 1));
        }
        to[(i0 + i * parts) * 32] = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y), pack_bf16x2(y[2].x, y[2].y),
                                               pack_bf16x2(y[3].x, y[3].y));
      }
    }
  };
  if (p.q_out) turn(p.q_raw + t * p.q_stride, p.w_q, p.q_out + t * kHeads * kDim, kHeads / 2);
  if (p.k_out) turn(p.k_raw + t * p.k_stride, p.w_k, p.k_out + t * kKvHeads * kDim, kKvHeads / 2);
}

template <int kAt>
cudaError_t launch_at(const RopeAtParams& p, int num_sms, cudaStream_t stream) {
  // up to 6 warps a token while they fit 16 warps a SM
  const int parts = p.T * 6 <= num_sms * 16 ? 6 : p.T * 3 <= num_sms * 16 ? 3 : 1;
  const int ctas = (p.T * parts + kRaWarps - 1) / kRaWarps;  // (T <= FLINT_MAX_CONTEXT)
  rope_at_kernel<kAt><<<ctas, kRaThreads, 0, stream>>>(p, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_at(const RopeAtParams& p, int num_sms, cudaStream_t stream) {
  if (p.layout == FLINT_ROPE_INTERLEAVED) return launch_at<kInLane>(p, num_sms, stream);
  return p.rotary_dim % 16 == 0 ? launch_at<kByLanes>(p, num_sms, stream) : launch_at<kByShared>(p, num_sms, stream);
}

}  // namespace flint
