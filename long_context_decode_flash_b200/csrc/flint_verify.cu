// flint_verify.cu -- verification of a tree of drafted tokens against the
// target's probabilities from given random numbers (speculative sampling with
// several candidates per position).  At the node cur with the residual w (the
// target's row at first) and its total Z, the children i of cur are tried in
// order: x = tokens[i] is accepted if u_i q(x) Z < w(x); a rejection leaves
// w = max(w - Z q, 0), Z = sum w.  All children of a node share q, so after
// rejections w = max(p - c q, 0) with c the sum of the Z before them: w is
// never stored.  Then the next token is the first whose running sum of w
// exceeds u sum(w).
//
// One CTA per request; sums in double, over the warps' contiguous shares of
// the row, so that the sums also tell which share holds the drawn token.
#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

constexpr int kVfWarps = 16;

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__global__ void __launch_bounds__(kVfWarps * 32) verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ double pt[kMaxTree], pd[kMaxTree];  // target and draft probability of node i's token at its parent
  __shared__ double sums[kVfWarps];
  __shared__ int held[kVfWarps];
  __shared__ int tok[kMaxTree], par[kMaxTree];
  __shared__ double u[kMaxTree];
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = p.n_draft[b];
  const float* target = p.target + static_cast<long long>(b) * (p.N + 1) * p.target_stride;
  const float* draft = p.draft ? p.draft + static_cast<long long>(b) * p.N * p.draft_stride : nullptr;
  if (threadIdx.x < n) {
    const int i = threadIdx.x;
    const long long at = static_cast<long long>(b) * p.N + i;
    int up = p.parent[at], x = p.tokens[at];
    if (up < -1 || up >= i) {
      report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
      up = -1;
    }
    if (x < 0 || x >= p.V) {
      report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
      x = -1;
    }
    tok[i] = x;
    par[i] = up;
    u[i] = p.u_accept[at];
    pt[i] = x < 0 ? 0.0 : target[(up + 1) * p.target_stride + x];
    pd[i] = x < 0 || !draft ? 1.0 : draft[(up + 1) * p.draft_stride + x];
  }
  __syncthreads();
  const int share = (p.V + kVfWarps - 1) / kVfWarps, v0 = min(p.V, warp * share), v1 = min(p.V, v0 + share);
  int cur = -1, taken = 0;
  double c = 0.0, Z = 1.0;
  unsigned long long out_of_w = 0;  // fixed candidates rejected at cur
  // w at the token y: fixed candidates by their list
  auto w_at = [&](int y, double pv) {
    for (unsigned long long r = out_of_w; r; r &= r - 1)
      if (tok[__ffsll(r) - 1] == y) return 0.0;
    return pv;
  };
  auto row_sum = [&](double cc, double* own) {  // sum of w over the row; *own: this warp's share
    const float* tr = target + (cur + 1) * p.target_stride;
    const float* dr = draft && cc != 0.0 ? draft + (cur + 1) * p.draft_stride : nullptr;
    double s = 0.0;
    for (int y = v0 + lane; y < v1; y += 32) {
      const double t = tr[y];
      s += dr ? fmax(__dsub_rn(t, __dmul_rn(cc, dr[y])), 0.0) : w_at(y, t);
    }
    s = warp_sum(s);
    *own = s;
    __syncthreads();
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    double all = 0.0;
    for (int k = 0; k < kVfWarps; ++k) all += sums[k];
    return all;
  };
  for (int i = 0; i < n; ++i) {
    if (par[i] != cur || tok[i] < 0) continue;
    const double w = draft ? fmax(__dsub_rn(pt[i], __dmul_rn(c, pd[i])), 0.0) : w_at(tok[i], pt[i]);
    if (u[i] * pd[i] * Z < w) {
      if (threadIdx.x == 0) p.path[static_cast<long long>(b) * p.N + taken] = i;
      ++taken;
      cur = i;
      c = 0.0;
      Z = 1.0;
      out_of_w = 0;
    } else if (draft) {
      double own;
      const double left = row_sum(c + Z, &own);
      if (left > 0.0) {
        c += Z;
        Z = left;
      }
    } else if (Z - w > 0.0) {
      out_of_w |= 1ull << i;
      Z -= w;
    }
  }
  double own;
  const double total = row_sum(c, &own);
  const double goal = static_cast<double>(p.u_sample[b]) * total;
  // the warp whose share holds the drawn token scans it
  double base = 0.0;
  for (int k = 0; k < warp; ++k) base += sums[k];
  const float* tr = target + (cur + 1) * p.target_stride;
  const float* dr = draft && c != 0.0 ? draft + (cur + 1) * p.draft_stride : nullptr;
  int found = -1, last = -1;
  // (w > 0: where base and the running sums differ by a rounding, no token of
  // probability 0 is drawn)
  for (int y0 = v0; y0 < v1 && found < 0; y0 += 32) {
    const int y = y0 + lane;
    double w = 0.0;
    if (y < v1) {
      const double t = tr[y];
      w = dr ? fmax(__dsub_rn(t, __dmul_rn(c, dr[y])), 0.0) : w_at(y, t);
    }
    double s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && base + s > goal);
    const unsigned pos = __ballot_sync(0xffffffffu, w > 0.0);
    if (hit) found = y0 + __ffs(hit) - 1;
    if (pos) last = y0 + 31 - __clz(pos);
    base += __shfl_sync(0xffffffffu, s, 31);
  }
  __syncthreads();
  if (lane == 0) {
    sums[warp] = found;
    held[warp] = last;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int y = -1, z = 0;
    for (int k = 0; k < kVfWarps; ++k) {
      if (y < 0) y = static_cast<int>(sums[k]);
      if (held[k] >= 0) z = held[k];
    }
    p.next_token[b] = y >= 0 ? y : z;
    p.n_accepted[b] = taken;
  }
  for (int j = taken + threadIdx.x; j < p.N; j += blockDim.x) p.path[static_cast<long long>(b) * p.N + j] = -1;
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  verify_kernel<<<p.B, kVfWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flint
