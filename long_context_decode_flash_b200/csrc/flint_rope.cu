// flint_rope.cu -- per-head Q/K RMSNorm and rotary positions of T tokens at
// given positions, in either pair layout, on the first rotary_dim dims, with
// per-pair frequencies from the host:
//     y = x w / sqrt(mean(x^2) + eps),
//     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin),  angle pos f_i.
// The angle is formed in double as pos * (f_i / 2 pi) turns and reduced to
// [-1/2, 1/2] turns before its cos and sin are taken in float32.
//
// Bound by HBM (each row read and written once) for many tokens, by latency for
// few.  A warp takes whole rows of one token, two at a time, 16 lanes of 8 dims
// each (16-byte loads), so that cos and sin are formed once for all of them; few
// tokens are spread over up to 6 warps each.  The partner of a value is in its
// own lane (interleaved), in another lane of its row at the same place (half
// layout, rotary_dim a multiple of 16), or else found through shared memory.
#include <algorithm>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

constexpr int kRaWarps = 8, kRaThreads = kRaWarps * 32;
constexpr int kAhead = 3;
constexpr int kPairsOfRows = (kHeads + kKvHeads) / 2;  // 18: 16 of q, 2 of k

enum { kInLane, kByLanes, kByShared };

// One CTA per step of kRaWarps * tokens / parts; warp: token t, row pairs part,
// part + parts, ...  kAt: where the partner of a value is.
template <int kAt>
__global__ void __launch_bounds__(kRaThreads) rope_at_kernel(const __grid_constant__ RopeAtParams p, int parts) {
  __shared__ double turns[kDim / 2];
  __shared__ float2 cs[kRaWarps][kDim / 2];
  __shared__ float rows[kAt == kByShared ? kRaWarps : 1][2 * kDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 15;
  const int half = p.rotary_dim / 2, d0 = 8 * c;  // this lane's dims d0 .. d0 + 7
  if (threadIdx.x < half) turns[threadIdx.x] = p.turns[threadIdx.x];
  __syncthreads();
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (p.w_q) {
    wq = reinterpret_cast<const uint4*>(p.w_q)[c];
    wk = reinterpret_cast<const uint4*>(p.w_k)[c];
  }
  const long long jobs = static_cast<long long>(p.T) * parts;
#pragma unroll 1
  for (long long job = static_cast<long long>(blockIdx.x) * kRaWarps + warp; job < jobs; job += static_cast<long long>(gridDim.x) * kRaWarps) {
    const long long t = job / parts;
    const int part = static_cast<int>(job % parts);
    // rows 2 * pair + (lane >> 4), q's first; the next kAhead pairs are in flight
    auto load = [&](int pair) {
      uint4 x = make_uint4(0, 0, 0, 0);
      const int r = 2 * pair + (lane >> 4);
      if (pair < kHeads / 2) {
        if (p.q_out) x = reinterpret_cast<const uint4*>(p.q_raw + t * p.q_stride + r * kDim)[c];
      } else if (pair < kPairsOfRows && p.k_out) {
        x = reinterpret_cast<const uint4*>(p.k_raw + t * p.k_stride + (r - kHeads) * kDim)[c];
      }
      return x;
    };
    uint4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = load(part + i * parts);
    // cos and sin of the token's pairs
    const int pos = p.pos[t];
    __syncwarp();
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
#pragma unroll 1
    for (int pair = part; pair < kPairsOfRows; pair += parts) {
      const uint4 raw = ahead[0];
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) ahead[i] = ahead[i + 1];
      ahead[kAhead - 1] = load(pair + kAhead * parts);
      const bool is_q = pair < kHeads / 2;
      uint16_t* o = is_q ? p.q_out : p.k_out;
      if (!o) continue;
      const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = bf16_lo(x[e]);
        y[2 * e + 1] = bf16_hi(x[e]);
      }
      if (p.w_q) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int k = 8; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
        const float inv = rsqrtf(fmaf(ss, 1.0f / kDim, p.eps));
        const uint4 wr = is_q ? wq : wk;
        const uint32_t wx[4] = {wr.x, wr.y, wr.z, wr.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = y[2 * e] * inv * bf16_lo(wx[e]);
          y[2 * e + 1] = y[2 * e + 1] * inv * bf16_hi(wx[e]);
        }
      }
      if (kAt == kInLane) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (d0 / 2 + e < half) {
            const float u = y[2 * e], v = y[2 * e + 1];
            y[2 * e] = u * mine[e].x - v * mine[e].y;
            y[2 * e + 1] = v * mine[e].x + u * mine[e].y;
          }
      } else if (kAt == kByLanes) {  // half is a multiple of 8: whole lanes pair up
        const bool turned = d0 < 2 * half;
        const int other = turned ? (d0 >= half ? lane - half / 8 : lane + half / 8) : lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = __shfl_sync(0xffffffffu, y[e], other);
          if (turned) y[e] = y[e] * mine[e].x + z * mine[e].y;
        }
      } else {
        float* row = rows[warp] + (lane >> 4) * kDim;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) row[d0 + e] = y[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          if (d < 2 * half) y[e] = y[e] * mine[e].x + row[d >= half ? d - half : d + half] * mine[e].y;
        }
      }
      const int r = 2 * pair + (lane >> 4);
      o += is_q ? (t * kHeads + r) * kDim : (t * kKvHeads + r - kHeads) * kDim;
      reinterpret_cast<uint4*>(o)[c] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                                  pack_bf16x2(y[6], y[7]));
    }
  }
}

template <int kAt>
cudaError_t launch_at(const RopeAtParams& p, int num_sms, cudaStream_t stream) {
  // up to 6 warps a token while they fit the SMs' warps eight times over
  const int parts = p.T * 6 <= num_sms * kRaWarps ? 6 : p.T * 3 <= num_sms * kRaWarps ? 3 : 1;
  const long long ctas = (static_cast<long long>(p.T) * parts + kRaWarps - 1) / kRaWarps;
  rope_at_kernel<kAt><<<static_cast<int>(std::min<long long>(ctas, 8ll * num_sms)), kRaThreads, 0, stream>>>(p, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_at(const RopeAtParams& p, int num_sms, cudaStream_t stream) {
  if (p.layout == FLINT_ROPE_INTERLEAVED) return launch_at<kInLane>(p, num_sms, stream);
  return p.rotary_dim % 16 == 0 ? launch_at<kByLanes>(p, num_sms, stream) : launch_at<kByShared>(p, num_sms, stream);
}

}  // namespace flint
