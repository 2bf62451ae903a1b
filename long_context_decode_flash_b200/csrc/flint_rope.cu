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
  const long long jobs = static_cast<long long>(p.T) * parts;
#pragma unroll 1
  for (long long job = static_cast<long long>(blockIdx.x) * kRaWarps + warp; job < jobs; job += static_cast<long long>(gridDim.x) * kRaWarps) {
    const long long t = job / parts;
    const int part = static_cast<int>(job % parts);
    // rows part * 2 + (lane >> 4), ...: q rows first
    constexpr int kAhead = 3;
    auto want = [&](int pair) { return pair < kPairsOfRows && (pair < kHeads / 2 ? p.q_out : p.k_out) != nullptr; };
    auto load = [&](int pair) {
      const int r = 2 * pair + (lane >> 4);
      const uint16_t* x = r < kHeads ? p.q_raw + t * p.q_stride + r * kDim : p.k_raw + t * p.k_stride + (r - kHeads) * kDim;
      return reinterpret_cast<const uint4*>(x)[c];
    };
    uint4 next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (want(part + i * parts)) next[i] = load(part + i * parts);
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
#pragma unroll 1
    for (int pair0 = part; pair0 < kPairsOfRows; pair0 += kAhead * parts) {
      uint4 now[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) now[i] = next[i];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (want(pair0 + (kAhead + i) * parts)) next[i] = load(pair0 + (kAhead + i) * parts);
#pragma unroll 1
      for (int i = 0; i < kAhead; ++i) {
        const int pair = pair0 + i * parts;
        if (!want(pair)) continue;
        const int r = 2 * pair + (lane >> 4);
        const uint4 raw = i == 0 ? now[0] : i == 1 ? now[1] : now[2];
        const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = bf16_lo(x[e]);
          y[2 * e + 1] = bf16_hi(x[e]);
        }
        const uint16_t* w = r < kHeads ? p.w_q : p.w_k;
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += y[e] * y[e];
#pragma unroll
          for (int k = 8; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
          const float inv = 1.0f / sqrtf(ss * (1.0f / kDim) + p.eps);
          const uint4 wr = reinterpret_cast<const uint4*>(w)[c];
          const uint32_t wx[4] = {wr.x, wr.y, wr.z, wr.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[2 * e] = y[2 * e] * inv * bf16_lo(wx[e]);
            y[2 * e + 1] = y[2 * e + 1] * inv * bf16_hi(wx[e]);
          }
        }
        if (kAt == kInLane) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int j = (d0 + e) >> 1;
            if (j < half) {
              const float2 a = cs[warp][j];
              const float u = y[e], v = y[e + 1];
              y[e] = u * a.x - v * a.y;
              y[e + 1] = v * a.x + u * a.y;
            }
          }
        } else if (kAt == kByLanes) {  // half is a multiple of 8: whole lanes pair up
          const bool turned = d0 < 2 * half, second = d0 >= half;
          const int other = turned ? (second ? lane - half / 8 : lane + half / 8) : lane;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = __shfl_sync(0xffffffffu, y[e], other);
            if (turned) {
              const float2 a = cs[warp][(second ? d0 - half : d0) + e];
              y[e] = second ? y[e] * a.x + z * a.y : y[e] * a.x - z * a.y;
            }
          }
        } else {
          float* mine = rows[warp] + (lane >> 4) * kDim;
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) mine[d0 + e] = y[e];
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            if (d < 2 * half) {
              const bool second = d >= half;
              const float2 a = cs[warp][second ? d - half : d];
              const float z = mine[second ? d - half : d + half];
              y[e] = second ? y[e] * a.x + z * a.y : y[e] * a.x - z * a.y;
            }
          }
        }
        uint16_t* o = r < kHeads ? p.q_out + (t * kHeads + r) * kDim : p.k_out + (t * kKvHeads + r - kHeads) * kDim;
        reinterpret_cast<uint4*>(o)[c] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                                    pack_bf16x2(y[6], y[7]));
      }
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
