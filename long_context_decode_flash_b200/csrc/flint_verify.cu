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
// A cluster of CTAs per request, up to 16 so that a batch fills the SMs.  The
// walk needs two numbers a node, fetched at once; only a rejection, and the
// draw at the end, reads a row, each CTA its part.  The warps' sums over
// contiguous shares (in double: the draw decides at borders) meet through the
// cluster's shared memory, and every thread walks on with the same totals.  The
// shares' sums also tell which share holds the drawn token: its CTA alone reads
// it again.  Bound by the rows' loads for large batches (64 chains of
// 6 over 150,001 tokens: 69 MB at 4.9 TB/s for 14 us of the 22 to 25; three times as many
// loads in flight measured no faster), and else by the steps in turn: launch 2 us,
// the gathers 1 to 2 us, a pass over a row 1.5 to 3 us, the draw 1 to 4 us (one
// chain of 4: 6.2 to 6.9 us; 16 trees of 31: 12 to 14 us).
#include <cooperative_groups.h>

#include <algorithm>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace cg = cooperative_groups;

namespace flint {

namespace {

constexpr int kVfWarps = 8, kVfThreads = kVfWarps * 32;
constexpr int kVfCluster = 16;             // CTAs per request, at most
constexpr int kVfShares = kVfCluster * kVfWarps;
static_assert(kVfShares == 128, "four shares a lane");

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// w over a row: the target's probabilities less c times the draft's (draft ==
// nullptr: none), or with tokens taken out (fixed candidates).
struct Residual {
  const float* target;
  const float* draft;
  double c;
  const int* tok;
  unsigned long long out;   // candidates taken out
  __device__ __forceinline__ double of(int y, float t, float d) const {
    if (draft) return fmax(__dsub_rn(t, __dmul_rn(c, d)), 0.0);
    for (unsigned long long r = out; r; r &= r - 1)
      if (tok[__ffsll(r) - 1] == y) return 0.0;
    return t;
  }
  // A warp's sum over [v0, v1): 8 loads a lane (16 with a draft) in flight while
  // the 8 before them are summed.
  template <bool kDraft>
  __device__ __forceinline__ double sum_of(int v0, int v1, int lane) const {
    double s0 = 0.0, s1 = 0.0;
    constexpr int kStep = 8 * 32;
    const int full = v0 + (v1 - v0) / kStep * kStep;
    auto add = [&](int k, float a, float e) {
      const double x = kDraft ? fmax(__dsub_rn(a, __dmul_rn(c, e)), 0.0) : static_cast<double>(a);
      if (k & 1) s1 += x;
      else s0 += x;
    };
    float t[8], d[8];
    if (full > v0) {
      auto load = [&](int y) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          t[k] = target[y + 32 * k];
          if (kDraft) d[k] = draft[y + 32 * k];
        }
      };
      load(v0 + lane);
      for (int y = v0; y < full; y += kStep) {
        float a[8], e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] = t[k];
          e[k] = kDraft ? d[k] : 0.f;
        }
        load((y + kStep < full ? y + kStep : v0) + lane);
#pragma unroll
        for (int k = 0; k < 8; ++k) add(k, a[k], e[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int z = full + lane + 32 * k;
      t[k] = z < v1 ? target[z] : 0.f;
      d[k] = kDraft && z < v1 ? draft[z] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) add(k, t[k], d[k]);
    return warp_sum(s0 + s1);
  }
  __device__ __forceinline__ double sum(int v0, int v1, int lane) const {
    if (draft) return sum_of<true>(v0, v1, lane);
    // the ranges between the candidates that were taken out, in order
    double s = 0.0;
    for (int from = v0; from < v1;) {
      int to = v1;
      for (unsigned long long r = out; r; r &= r - 1) {
        const int x = tok[__ffsll(r) - 1];
        if (x >= from && x < to) to = x;
      }
      s += sum_of<false>(from, to, lane);
      from = to + 1;
    }
    return s;
  }
};

__global__ void __launch_bounds__(kVfThreads, 4) verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ double pt[kMaxTree], pd[kMaxTree];  // target and draft probability of node i's token at its parent
  __shared__ double mine[2][kVfWarps];           // this CTA's shares' sums (by pass parity: others read them)
  __shared__ double all[kVfShares], below[kVfShares];  // every share's sum, and the sum of those before it
  __shared__ double total;
  __shared__ double part[kVfWarps];
  __shared__ int tok[kMaxTree], par[kMaxTree], last_held[kVfWarps], hit[kVfWarps];
  __shared__ double u[kMaxTree];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = p.n_draft[b];
  const float* target = p.target + static_cast<long long>(b) * (p.N + 1) * p.target_stride;
  const float* draft = p.draft ? p.draft + static_cast<long long>(b) * p.N * p.draft_stride : nullptr;
  if (threadIdx.x < n) {
    const int i = threadIdx.x;
    const long long at = static_cast<long long>(b) * p.N + i;
    int up = p.parent[at], x = p.tokens[at];
    const float ui = p.u_accept[at];
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
    u[i] = ui;
    pt[i] = x < 0 ? 0.0 : target[(up + 1) * p.target_stride + x];
    pd[i] = x < 0 || !draft ? 1.0 : draft[(up + 1) * p.draft_stride + x];
  }
  const double u_sample = p.u_sample[b];
  __syncthreads();
  const int shares = C * kVfWarps;
  const int share = (p.V + shares - 1) / shares;
  auto begin_of = [&](int k) { return static_cast<int>(min(static_cast<long long>(p.V), static_cast<long long>(k) * share)); };

  int cur = -1, taken = 0, pass = 0;
  Residual w{target, nullptr, 0.0, tok, 0};
  double Z = 1.0;
  // the sums of `r` over the row: all[], below[], total
  auto row_sums = [&](const Residual& r) {
    const int k = rank * kVfWarps + warp;
    const double s = r.sum(begin_of(k), begin_of(k + 1), lane);
    if (lane == 0) mine[pass & 1][warp] = s;
    cluster.sync();
    if (threadIdx.x < shares)
      all[threadIdx.x] = *cluster.map_shared_rank(&mine[pass & 1][threadIdx.x % kVfWarps], threadIdx.x / kVfWarps);
    __syncthreads();
    if (warp == 0) {  // prefix sums, 4 shares a lane
      double x[4], run = 0.0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * lane + j;
        x[j] = run;
        run += i < shares ? all[i] : 0.0;
      }
      double before = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      if (lane == 31) total = before;
      before = __shfl_up_sync(0xffffffffu, before, 1);
      if (lane == 0) before = 0.0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * lane + j < shares) below[4 * lane + j] = before + x[j];
    }
    __syncthreads();
    ++pass;
  };
  bool summed = false;  // all[], below[] and total are w's
  // the nodes behind node i whose parent is `node`, as bits
  auto children = [&](int node, int i) {
    const int a = lane, e = lane + 32;
    const unsigned lo = __ballot_sync(0xffffffffu, a < n && par[a] == node && tok[a] >= 0);
    const unsigned hi = __ballot_sync(0xffffffffu, e < n && par[e] == node && tok[e] >= 0);
    const unsigned long long all_of = static_cast<unsigned long long>(hi) << 32 | lo;
    return i < 0 ? all_of : i >= 63 ? 0ull : all_of & (~0ull << (i + 1));
  };
  for (unsigned long long left = children(-1, -1); left;) {
    const int i = __ffsll(left) - 1;
    left &= left - 1;
    const double wx = draft ? fmax(__dsub_rn(pt[i], __dmul_rn(w.c, pd[i])), 0.0) : w.of(tok[i], static_cast<float>(pt[i]), 0.f);
    if (u[i] * pd[i] * Z < wx) {
      if (rank == 0 && threadIdx.x == 0) p.path[static_cast<long long>(b) * p.N + taken] = i;
      ++taken;
      cur = i;
      w = Residual{target + (cur + 1) * p.target_stride, nullptr, 0.0, tok, 0};
      Z = 1.0;
      summed = false;
      left = children(cur, i);
    } else if (draft) {
      Residual r = w;
      r.draft = draft + (cur + 1) * p.draft_stride;
      r.c = w.c + Z;
      row_sums(r);
      summed = total > 0.0;
      if (summed) {
        w = r;
        Z = total;
      }
    } else if (Z - wx > 0.0) {
      w.out |= 1ull << i;
      Z -= wx;
    }
  }
  if (rank == 0) {
    if (threadIdx.x == 0) p.n_accepted[b] = taken;
    for (int j = taken + threadIdx.x; j < p.N; j += kVfThreads) p.path[static_cast<long long>(b) * p.N + j] = -1;
  }
  if (!summed) row_sums(w);
  // nobody's sums are read from here on
  auto token = cluster.barrier_arrive();
  const double goal = u_sample * total;
  // The share with the drawn token: the first whose end exceeds the goal, or
  // where rounding leaves none the last that holds anything.
  __shared__ int chosen[2];
  if (warp == 0) {
    int first = kVfShares, held = -1;
    for (int k = lane; k < shares; k += 32) {
      if (all[k] > 0.0) {
        held = k;
        if (below[k] + all[k] > goal) first = min(first, k);
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    held = __reduce_max_sync(0xffffffffu, held);
    if (lane == 0) {
      chosen[0] = first < kVfShares ? first : held;
      chosen[1] = held;
    }
  }
  __syncthreads();
  const int at = chosen[0];
  if (at < 0) {
    if (rank == 0 && threadIdx.x == 0) p.next_token[b] = 0;  // w is 0 everywhere
  } else if (at / kVfWarps == rank) {
    // its CTA's warps take a part of it each, then the warp whose part holds the
    // token scans it
    const int s0 = begin_of(at), s1 = begin_of(at + 1), len = (s1 - s0 + kVfWarps - 1) / kVfWarps;
    const int v0 = min(s1, s0 + warp * len), v1 = min(s1, v0 + len);
    const double s = w.sum(v0, v1, lane);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    double base = below[at];
    for (int k = 0; k < warp; ++k) base += part[k];
    int found = -1, last = -1;
    // (w > 0: where base and the running sums differ by a rounding, no token of
    // probability 0 is drawn)
    if (s > 0.0)
      for (int y0 = v0; y0 < v1 && found < 0; y0 += 32) {
        const int y = y0 + lane;
        const double x = y < v1 ? w.of(y, w.target[y], w.draft ? w.draft[y] : 0.f) : 0.0;
        double run = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double z = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += z;
        }
        const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && base + run > goal);
        const unsigned pos = __ballot_sync(0xffffffffu, x > 0.0);
        if (over) found = y0 + __ffs(over) - 1;
        if (pos) last = y0 + 31 - __clz(pos);
        base += __shfl_sync(0xffffffffu, run, 31);
      }
    if (lane == 0) {
      hit[warp] = found;
      last_held[warp] = last;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int y = -1, z = 0;
      for (int k = 0; k < kVfWarps; ++k) {
        if (y < 0) y = hit[k];
        if (last_held[k] >= 0) z = last_held[k];
      }
      p.next_token[b] = y >= 0 ? y : z;
    }
  }
  cluster.barrier_wait(std::move(token));
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int num_sms, cudaStream_t stream) {
  // CTAs per request: up to four a SM over the batch, at least 512 values each
  int C = 1;
  while (C < kVfCluster && 2 * C * p.B <= 4 * num_sms && p.V / (2 * C) >= 2 * kVfThreads) C *= 2;
  if (C > 8) {  // a cluster beyond the portable size
    static ContextSet configured;
    void* ctx = current_context();
    std::lock_guard<std::mutex> lock(configured.mu);
    if (!ctx || std::find(configured.ctxs.begin(), configured.ctxs.end(), ctx) == configured.ctxs.end()) {
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(verify_kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (ctx) configured.ctxs.push_back(ctx);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C * p.B);
  cfg.blockDim = dim3(kVfThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace flint
