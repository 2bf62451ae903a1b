// flint_tree.cu -- attention of drafted tokens over a committed cache and
// their own tree: node i of request b, at depth d_i (its ancestors), attends
// the cached positions [max(0, L + d_i - window + 1), L) (or all of [0, L)),
// its ancestors and itself,
//     out = sum_j e^(s_j - M) V_j / (sum_j e^(s_j - M) + e^(sink - M)),
//     s_j = q . K_j / sqrt(128),  M = max(max_j s_j, sink).
//
// How (tcgen05).  The 8 query heads of a KV head share its keys, so 16 nodes
// of a request are the 128 rows of one MMA tile (row r = 8 * node + head), and
// a unit is a request's block of up to 32 nodes (one or two row tiles).  Its
// keys come in tiles of 128, two 64-key halves each: half 0 is the drafted
// tokens themselves, the halves behind it 64-token boxes of the cache (whole
// pages of a paged cache, slots of a ring).  Groups of four CTAs, one per KV
// head, take contiguous shares of all (unit, tile) pairs, so that the four
// read the same token rows at the same time; a unit cut between groups leaves
// one partial per share (O, m, l), and a second launch folds them in order.
//
// A CTA is 14 warps over two streams of steps, a step being one row tile
// against one key tile.  Two row tiles: stream w is row tile w.  One row tile:
// stream w is the key tiles of parity w, the two streams' states joined at the
// item's end.  So either way one stream's softmax runs beside the other's MMAs:
//   warp 12     TMA producer: 64-row boxes of K and V through one ring of
//               32 KiB stages (128-byte swizzle).
//   warps 8-11  make the stages MMA operands: V from bf16 to fp16 in place, or
//               E4M3 codes (landed in the stage's upper half) of K and V to
//               fp16; the drafted tokens' rows; Q; V rows that hold no token
//               become 0 (whatever lies there must not meet a probability 0).
//   warp 13     issues S_w = Q K^T (M 128, N 128) and O_w += P_w V.
//   warps 0-7   softmax, warpgroup w on stream w, a thread per row: fp32 online
//               softmax in log2 units with a running maximum that moves only
//               by more than 2^8; P goes back to TMEM over S's upper columns.
// P is held in fp16 as 2^(x - m + 7): at most 2^15 under the lazy maximum, so
// that probabilities keep 11 bits down to 2^-21 of the largest and lose at
// most 2^-32 of it below (a bf16 P would round each by 2^-9).  V is fp16 (exact
// for E4M3 and for bf16 in fp16's normal range, saturating at 65504).
// TMEM columns: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512); P_w
// (fp16 pairs) is S_w's [64,128).  Every wait is bounded; a timeout raises
// FLINT_ERR_TIMEOUT.
#include <math.h>

#include <algorithm>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

namespace {

constexpr int kTrRows = 128;               // rows of a row tile: 16 nodes x 8 heads
constexpr int kTrNodes = kTrRows / kGroup;
constexpr int kHalf = 64;                  // keys of a half tile
constexpr int kTrKeys = 2 * kHalf;         // keys of a tile
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kConvThreads = kConvWarps * 32;
constexpr int kTmaWarp = kSoftWarps + kConvWarps, kMmaWarp = kTmaWarp + 1;
constexpr int kTrThreads = (kMmaWarp + 1) * 32;
constexpr uint32_t kBox16 = kHalf * 128;            // 64 keys x 64 dims x 16 bit (or 128 dims x 8 bit): 8 KiB
constexpr uint32_t kDimHalf = kTrKeys * 128;        // 64 dims of a 16-bit tile: 16 KiB
constexpr uint32_t kStage = 2 * kDimHalf;           // a K or V tile: 32 KiB
constexpr uint32_t kQTile = 2 * kTrRows * 128;      // a Q row tile: 32 KiB
constexpr float kTrLog2e = 1.4426950408889634f;
constexpr float kTrScale = static_cast<float>(1.4426950408889634 * 0.08838834764831845);
constexpr float kTau = 8.0f;               // the running maximum lags by at most this (log2 units)
constexpr float kBias = 7.0f;              // P = 2^(x - m + kBias)
constexpr uint32_t kColS = 0, kColP = 64, kColO = 256;  // + 128 * stream
constexpr int kInfo = 8;                   // tiles whose NaN record is kept

// MT row tiles a unit (1 or 2): the ring gets what Q leaves.
template <int MT>
struct Lay {
  static constexpr int kStages = MT == 1 ? 6 : 5;
  static constexpr uint32_t kRing = MT * kQTile;
  static constexpr uint32_t kEx = kRing + kStages * kStage;        // m, l of the two streams: [2 streams][128] float2
  static constexpr uint32_t kNan = kEx + 2 * kTrRows * 8;          // [kInfo][4] words
  static constexpr uint32_t kBar = kNan + kInfo * 16;
  static constexpr size_t kBytes = kBar + 256;
};
static_assert(Lay<1>::kBytes <= 232448 && Lay<2>::kBytes <= 232448, "shared memory of a CTA");

struct Bars {
  uint64_t full[6], ready[6], empty[6];  // stage landed / is an operand / was consumed
  uint64_t s_full[2];                    // S_w complete (and every MMA issued before it)
  uint64_t p_ready[2];                   // P_w written, S_w read
  uint64_t q_ready, q_empty;             // per item: Q filled; every S of the item complete
  uint64_t o_full, o_free;               // per item: O complete; O read
  uint64_t ex_full;                      // per item with one row tile: m, l of both streams written
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// Instruction descriptors (kind::f16), fp32 D, M 128, N 128, A K-major.  S: B
// (K) K-major, both bf16 or both fp16; PV: fp16, B (V) dims-major.
constexpr uint32_t kIdescBase = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescSBf16 = kIdescBase | (1u << 7) | (1u << 10);
constexpr uint32_t kIdescSF16 = kIdescBase;
constexpr uint32_t kIdescPV = kIdescBase | (1u << 16);

// Shared-memory matrix descriptor, 128-byte swizzle.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define FLINT_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                    "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define FLINT_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                    "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 consecutive columns of this warp's 32 lanes: lane i gets row i.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : FLINT_R8(0), FLINT_R8(8), FLINT_R8(16), FLINT_R8(24)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      FLINT_W8(0), FLINT_W8(8), FLINT_W8(16), FLINT_W8(24)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max(a, b, c), NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two floats -> packed f16x2 (first in the low half), nearest even, saturating
// at +-65504; NaN stays NaN.
__device__ __forceinline__ uint32_t f16x2_sat(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// acc + 0 * x per half: a half of acc turns NaN where x is.
__device__ __forceinline__ uint32_t nan_acc(uint32_t acc, uint32_t x) {
  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  return acc;
}
__device__ __forceinline__ uint32_t nan_to_zero(uint32_t x) {
  if ((x & 0x7FFFu) > 0x7C00u) x &= 0xFFFF0000u;
  if ((x & 0x7FFF0000u) > 0x7C000000u) x &= 0xFFFFu;
  return x;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// True on every converter thread if `ok` is true on all of them.
__device__ __forceinline__ bool conv_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok)), "n"(kConvThreads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, Bars* B) {
  const bool ok = mbar_wait(bar, parity, &B->abort);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool aborted(const Bars* B) {
  return *reinterpret_cast<const volatile int*>(&B->abort) != 0;
}
__device__ __forceinline__ void raise_abort(const TreeParams& p, Bars* B) {
  if (!aborted(B)) report_error(p.dev_err, FLINT_ERR_TIMEOUT);
  *reinterpret_cast<volatile int*>(&B->abort) = 1;
}

// The items of a CTA's group: (unit, tiles [t0, t1)) in order.
struct Item {
  int u, t0, t1, i;      // i: number of the item in the group's list
  int T, n[2];           // tiles and steps per stream of the items before this one
  int steps, mt;
  int x;                 // items with one row tile before this one
  __device__ bool whole(const TreeParams& p) const { return t0 == 0 && t1 == p.unit[u].tiles; }
  __device__ int stream_steps(int w) const { return mt == 2 ? t1 - t0 : (t1 - t0 - w + 1) / 2; }
};
__device__ __forceinline__ bool clip(const TreeParams& p, int q, Item& it) {
  const TreeCut e = p.cut[q + 1];
  if (it.u > e.unit || (it.u == e.unit && it.t0 >= e.tile)) return false;
  it.t1 = it.u < e.unit ? p.unit[it.u].tiles : e.tile;
  it.mt = p.unit[it.u].mt;
  it.steps = (it.t1 - it.t0) * it.mt;
  return true;
}
__device__ __forceinline__ bool first_item(const TreeParams& p, int q, Item& it) {
  it.u = p.cut[q].unit;
  it.t0 = p.cut[q].tile;
  it.i = it.x = 0;
  it.T = it.n[0] = it.n[1] = 0;
  return clip(p, q, it);
}
__device__ __forceinline__ bool next_item(const TreeParams& p, int q, Item& it) {
  it.n[0] += it.stream_steps(0);
  it.n[1] += it.stream_steps(1);
  it.T += it.t1 - it.t0;
  it.x += it.mt == 1;
  ++it.i;
  ++it.u;
  it.t0 = 0;
  return clip(p, q, it);
}

// The producer warp (lane 0 issues; 32 page numbers are fetched at a time, a
// batch ahead).  c counts stages: tile T's K is 2T, its V 2T + 1.  Returns the
// stages armed.
template <int MT, bool FP8>
__device__ int run_tma(const TreeParams& p, int q, int g, uint32_t base, Bars* B, int lane) {
  constexpr int NS = Lay<MT>::kStages;
  int c = 0;
  Item it;
  for (bool more = first_item(p, q, it); more; more = next_item(p, q, it)) {
    const TreeUnit& un = p.unit[it.u];
    const int b = un.b;
    const bool paged = p.layout == FLINT_KV_PAGED;
    const int h0 = 2 * it.t0, h1 = min(2 * it.t1, un.halves);  // halves of the item; half h >= 1: box at base + 64 (h - 1)
    auto page_of = [&](int h) {
      int blk = 0;
      if (h >= 1 && h < h1) {
        blk = p.table[static_cast<long long>(b) * p.max_blocks + un.base / kBlock + h - 1];
        if (blk < 0 || blk >= p.num_blocks) {  // never handed to a load
          report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
          blk = 0;
        }
      }
      return blk;
    };
    int now = 0, ahead = paged ? page_of(h0 + lane) : 0;
    for (int t = it.t0; t < it.t1; ++t) {
      const int k = 2 * (t - it.t0);
      if (paged && (k & 31) == 0) {
        now = ahead;
        ahead = page_of(h0 + k + 32 + lane);
      }
      int row[2], req[2];
      bool box[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * t + e;
        box[e] = h >= 1 && h < h1;
        row[e] = paged ? 0 : un.base + (h - 1) * kHalf;
        req[e] = paged ? __shfl_sync(0xffffffffu, now, (k & 31) + e) : b;
      }
      const uint32_t bytes = (box[0] ? 1u : 0u) + (box[1] ? 1u : 0u);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++c) {
        const int st = c % NS;
        if (c >= NS && !warp_wait(smem_u32(&B->empty[st]), static_cast<uint32_t>(c / NS - 1) & 1u, B)) {
          if (lane == 0) raise_abort(p, B);
          return c;
        }
        if (__any_sync(0xffffffffu, aborted(B))) return c;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&B->full[st]), dst = base + Lay<MT>::kRing + st * kStage;
          const CUtensorMap* map = kv ? &p.v_map : &p.k_map;
          mbar_expect_tx(bar, bytes * (FP8 ? kBox16 : 2 * kBox16));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!box[e]) continue;
            if (FP8) {
              tma_load_4d(dst + kDimHalf + e * kBox16, map, bar, 0, g, row[e], req[e]);
            } else {
              tma_load_4d(dst + e * kBox16, map, bar, 0, g, row[e], req[e]);
              tma_load_4d(dst + kDimHalf + e * kBox16, map, bar, 64, g, row[e], req[e]);
            }
          }
        }
        __syncwarp();
      }
    }
  }
  return c;
}

// Chunk `c` (8 values of 16 bit, c in [0, 16)) of row r in a 128-byte-swizzled
// operand tile of two 64-dim halves.
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int r, int c) {
  return tile + (c >> 3) * kDimHalf + r * 128 + ((c ^ r) & 7) * 16;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 bf16x8_to_f16(uint4 v) {
  return make_uint4(f16x2_sat(bf16_lo(v.x), bf16_hi(v.x)), f16x2_sat(bf16_lo(v.y), bf16_hi(v.y)),
                    f16x2_sat(bf16_lo(v.z), bf16_hi(v.z)), f16x2_sat(bf16_lo(v.w), bf16_hi(v.w)));
}
// bf16 values as an E4M3 cache of this scale holds them, in units of the scale.
__device__ __forceinline__ uint32_t bf16x2_through_e4m3(uint32_t w, float scale) {
  const uint32_t code = f32x2_to_e4m3x2(__fdiv_rn(bf16_lo(w), scale), __fdiv_rn(bf16_hi(w), scale));
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(code, lo, hi);
  return lo;
}

// The converter warps (thread ct of 128).  Every barrier of theirs is reached
// by all four warps, whatever their waits returned.
template <int MT, bool FP8>
__device__ void run_conv(const TreeParams& p, int q, int g, uint32_t base, uint8_t* smem, Bars* B, int ct) {
  constexpr int NS = Lay<MT>::kStages;
  const int lane = ct & 31, warp = ct >> 5;
  uint32_t* nans = reinterpret_cast<uint32_t*>(smem + Lay<MT>::kNan);
  Item it;
  for (bool more = first_item(p, q, it); more; more = next_item(p, q, it)) {
    const TreeUnit& un = p.unit[it.u];
    const int b = un.b, n = p.n_draft[b];
    const long long node0 = static_cast<long long>(b) * p.N;
    // Q: row r of tile m is head g * 8 + (r & 7) of node 32 rb + 16 m + (r >> 3)
    bool ok = it.i == 0 || warp_wait(smem_u32(&B->q_empty), static_cast<uint32_t>(it.i - 1) & 1u, B);
    if (!conv_all(ok)) {
      if (ct == 0) raise_abort(p, B);
      return;
    }
#pragma unroll 4
    for (int i = 0; i < it.mt * (kTrRows * 16 / kConvThreads); ++i) {
      const int x = i * kConvThreads + ct, c = x & 15, r = x >> 4;
      const int node = un.rb * 2 * kTrNodes + (r >> 3);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (node < n) v = reinterpret_cast<const uint4*>(p.q + ((node0 + node) * kHeads + g * kGroup + (r & 7)) * kDim)[c];
      if (FP8) v = bf16x8_to_f16(v);
      sts128(chunk_at(base + (r >> 7) * kQTile, r & 127, c), v);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&B->q_ready));

    for (int t = it.t0; t < it.t1; ++t) {
      const int T = it.T + t - it.t0;
      // row ct of the tile: does a token stand there?  (V; half 0 is the drafts')
      const int h = 2 * t + (ct >> 6), j = ct & 63;
      bool token;
      if (h == 0) {
        token = j < n;
      } else {
        const int s = un.base + (h - 1) * kHalf + j;
        token = h < un.halves && s >= un.lo && s < un.hi;
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int c = 2 * T + kv, st = c % NS;
        const uint32_t tile = base + Lay<MT>::kRing + st * kStage;
        ok = warp_wait(smem_u32(&B->full[st]), static_cast<uint32_t>(c / NS) & 1u, B);
        uint4 code[8];
        if (FP8) {
          // (rows of an absent box hold old bytes; they are zeroed or masked)
          if (ok) {
#pragma unroll
            for (int k = 0; k < 8; ++k) code[k] = lds128(tile + kDimHalf + ct * 128 + ((k ^ ct) & 7) * 16);
          }
        }
        if (!conv_all(ok)) {
          if (ct == 0) raise_abort(p, B);
          return;
        }
        uint32_t bad = 0;  // NaN in this row?
        if (FP8 && h > 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint4 a = make_uint4(0, 0, 0, 0), d = a;
            if (kv == 0 || token) {
              e4m3x4_to_f16x2x2(code[k].x, a.x, a.y);
              e4m3x4_to_f16x2x2(code[k].y, a.z, a.w);
              e4m3x4_to_f16x2x2(code[k].z, d.x, d.y);
              e4m3x4_to_f16x2x2(code[k].w, d.z, d.w);
            }
            if (kv) {
              bad = nan_acc(nan_acc(nan_acc(nan_acc(bad, a.x), a.y), a.z), a.w);
              bad = nan_acc(nan_acc(nan_acc(nan_acc(bad, d.x), d.y), d.z), d.w);
            }
            sts128(chunk_at(tile, ct, 2 * k), a);
            sts128(chunk_at(tile, ct, 2 * k + 1), d);
          }
        }
        if (!FP8 && kv == 1 && h > 0) {
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {
            const uint32_t at = chunk_at(tile, ct, k);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (token) v = bf16x8_to_f16(lds128(at));
            bad = nan_acc(nan_acc(nan_acc(nan_acc(bad, v.x), v.y), v.z), v.w);
            sts128(at, v);
          }
        }
        if (t == 0) {  // the drafts: rows 0..63, 16 lanes a row
          const uint16_t* src = kv ? p.v_draft : p.k_draft;
          const float scale = FP8 ? (kv ? p.v_scale[g] : p.k_scale[g]) : 1.f;
#pragma unroll 2
          for (int i = 0; i < kHalf * 16 / kConvThreads; ++i) {
            const int x = i * kConvThreads + ct, cc = x & 15, r = x >> 4;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < n) v = reinterpret_cast<const uint4*>(src + ((node0 + r) * kKvHeads + g) * kDim)[cc];
            if (FP8) {
              v = make_uint4(bf16x2_through_e4m3(v.x, scale), bf16x2_through_e4m3(v.y, scale),
                             bf16x2_through_e4m3(v.z, scale), bf16x2_through_e4m3(v.w, scale));
            } else if (kv) {
              v = bf16x8_to_f16(v);
            }
            sts128(chunk_at(tile, r, cc), v);
          }
          if (kv) {  // their NaN record wants whole rows
            if (!conv_all(true)) return;
            if (h == 0) {
#pragma unroll 4
              for (int k = 0; k < 16; ++k) {
                const uint4 v = lds128(chunk_at(tile, ct, k));
                bad = nan_acc(nan_acc(nan_acc(nan_acc(bad, v.x), v.y), v.z), v.w);
              }
            }
          }
        }
        if (kv) {
          const bool has = nan_to_zero(bad) != bad;
          if (has) {  // 0 in its place, for rows that do not attend the key; the others learn of it by the record
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              const uint32_t at = chunk_at(tile, ct, k);
              const uint4 v = lds128(at);
              sts128(at, make_uint4(nan_to_zero(v.x), nan_to_zero(v.y), nan_to_zero(v.z), nan_to_zero(v.w)));
            }
          }
          const uint32_t word = __ballot_sync(0xffffffffu, has);
          if (lane == 0) nans[(T % kInfo) * 4 + warp] = word;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B->ready[st]));
      }
    }
  }
}

// S of the item's step s (row tile and key tile by the mode): 8 MMAs of 16 dims.
template <int MT, bool FP8>
__device__ __forceinline__ bool issue_s(const Item& it, int s, uint32_t base, uint32_t tmem, Bars* B) {
  constexpr int NS = Lay<MT>::kStages;
  const int w = s & 1, two = it.mt == 2;
  const int T = it.T + (two ? s >> 1 : s), c = 2 * T, st = c % NS;
  const uint32_t parity = static_cast<uint32_t>(c / NS) & 1u;
  if (!mbar_wait(smem_u32(&B->ready[st]), parity, &B->abort) || !mbar_wait(smem_u32(&B->full[st]), parity, &B->abort))
    return false;
  tc_fence_after();
  const uint32_t qa = base + (two ? w * kQTile : 0), kb = base + Lay<MT>::kRing + st * kStage;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = (kk >> 2) * kDimHalf + (kk & 3) * 32;
    umma_ss(tmem + kColS + 128 * w, sw128_desc(qa + off, 16, 1024), sw128_desc(kb + off, 16, 1024),
            FP8 ? kIdescSF16 : kIdescSBf16, kk > 0 ? 1u : 0u);
  }
  if (!two || w) umma_commit(smem_u32(&B->empty[st]));
  umma_commit(smem_u32(&B->s_full[w]));
  if (s == it.steps - 1) umma_commit(smem_u32(&B->q_empty));
  return true;
}

// The MMA thread: per item S of the first two steps, then per step PV and the
// S two steps ahead (same stream: it overwrites P, whose PV is issued before).
template <int MT, bool FP8>
__device__ void run_mma(const TreeParams& p, int q, uint32_t base, uint32_t tmem, Bars* B) {
  constexpr int NS = Lay<MT>::kStages;
  bool ok = true;
  Item it;
  for (bool more = first_item(p, q, it); ok && more; more = next_item(p, q, it)) {
    ok = mbar_wait(smem_u32(&B->q_ready), static_cast<uint32_t>(it.i) & 1u, &B->abort);
    if (ok) ok = issue_s<MT, FP8>(it, 0, base, tmem, B);
    if (ok && it.steps > 1) ok = issue_s<MT, FP8>(it, 1, base, tmem, B);
    // O of the item before must have been read
    if (ok && it.i > 0) ok = mbar_wait(smem_u32(&B->o_free), static_cast<uint32_t>(it.i - 1) & 1u, &B->abort);
    for (int s = 0; ok && s < it.steps; ++s) {
      const int w = s & 1, two = it.mt == 2;
      const int T = it.T + (two ? s >> 1 : s), c = 2 * T + 1, st = c % NS;
      const uint32_t parity = static_cast<uint32_t>(c / NS) & 1u;
      ok = mbar_wait(smem_u32(&B->p_ready[w]), static_cast<uint32_t>(it.n[w] + (s >> 1)) & 1u, &B->abort) &&
           mbar_wait(smem_u32(&B->ready[st]), parity, &B->abort) && mbar_wait(smem_u32(&B->full[st]), parity, &B->abort);
      if (!ok) break;
      tc_fence_after();
      const uint32_t vb = base + Lay<MT>::kRing + st * kStage;
      // O += P V: 16 keys per MMA (their fp16 pairs are 8 columns of P)
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_ts(tmem + kColO + 128 * w, tmem + kColP + 128 * w + kk * 8, sw128_desc(vb + kk * 16 * 128, kDimHalf, 1024),
                kIdescPV, (s > 1 || kk > 0) ? 1u : 0u);
      if (!two || w) umma_commit(smem_u32(&B->empty[st]));
      if (s == it.steps - 1) umma_commit(smem_u32(&B->o_full));
      if (s + 2 < it.steps) ok = issue_s<MT, FP8>(it, s + 2, base, tmem, B);
    }
  }
  if (!ok) raise_abort(p, B);
  // let every issued MMA finish before the CTA ends (its TMEM is freed)
  umma_commit(smem_u32(&B->mma_done));
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(smem_u32(&B->mma_done), 0))
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
}

// Bits j of 32 with lo <= k0 + j < hi.
__device__ __forceinline__ uint32_t range_bits(int k0, int lo, int hi) {
  const int a = min(max(lo - k0, 0), 32), e = min(max(hi - k0, 0), 32);
  const uint32_t upto = e >= 32 ? 0xffffffffu : (1u << e) - 1u, from = a >= 32 ? 0xffffffffu : (1u << a) - 1u;
  return upto & ~from;
}

// What a softmax thread knows of its row.
struct Row {
  unsigned long long line;  // the node and its ancestors
  int lo, hi;               // attended storage positions (contiguous, paged)
  int r0, r1;               // ring: attended slots [r0, r1), and [0, r1 - 513)
};

// Ancestor lines of a request's nodes by pointer doubling, nodes lane and
// lane + 32 in each lane; returns this thread's node's.
__device__ __forceinline__ unsigned long long tree_line(const TreeParams& p, int b, int n, int node, int lane) {
  int up[2];
  unsigned long long line[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = lane + 32 * e;
    int a = -1;
    if (i < n) {
      a = p.parent[static_cast<long long>(b) * p.N + i];
      if (a < -1 || a >= i) {
        report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
        a = -1;
      }
    }
    up[e] = a;
    line[e] = 1ull << i;
  }
  auto from = [&](unsigned long long x0, unsigned long long x1, int i) {
    const unsigned long long a = __shfl_sync(0xffffffffu, x0, i & 31), c = __shfl_sync(0xffffffffu, x1, i & 31);
    return i & 32 ? c : a;
  };
#pragma unroll 1
  for (int round = 0; round < 6; ++round) {
    unsigned long long add[2];
    int next[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int a = up[e];
      const unsigned long long l = from(line[0], line[1], a);
      const int x0 = __shfl_sync(0xffffffffu, up[0], a & 31), x1 = __shfl_sync(0xffffffffu, up[1], a & 31);
      add[e] = a < 0 ? 0ull : l;
      next[e] = a < 0 ? -1 : (a & 32 ? x1 : x0);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      line[e] |= add[e];
      up[e] = next[e];
    }
  }
  return from(line[0], line[1], node);
}

// The mask word of keys 32 k .. 32 k + 31 of tile t for a row.
__device__ __forceinline__ uint32_t mask_word(const TreeParams& p, const TreeUnit& un, const Row& row, int t, int k) {
  const int h = 2 * t + (k >> 1);
  if (h == 0) return static_cast<uint32_t>(row.line >> (32 * (k & 1)));
  if (h >= un.halves) return 0u;
  const int s0 = un.base + (h - 1) * kHalf + 32 * (k & 1);
  if (p.layout == FLINT_KV_RING) return range_bits(s0, row.r0, min(row.r1, kWindow)) | range_bits(s0, 0, row.r1 - kWindow);
  return range_bits(s0, row.lo, row.hi);
}

// Softmax of one item by warpgroup w.  False if a wait ran out.
template <int MT>
__device__ bool softmax_item(const TreeParams& p, const Item& it, int q, int g, float scale, uint32_t tmem, uint8_t* smem,
                             Bars* B, int warp, int lane) {
  constexpr int NS = Lay<MT>::kStages;
  const TreeUnit& un = p.unit[it.u];
  const int w = warp >> 2, b = un.b, n = p.n_draft[b], L = p.len[b], two = it.mt == 2;
  const int r = (warp & 3) * 32 + lane;
  const int tile0 = un.rb * 2 * kTrNodes + (two ? w * kTrNodes : 0);  // first node of this row tile
  const int node = tile0 + (r >> 3), h = g * kGroup + (r & 7);
  const bool work = tile0 + (warp & 3) * 4 < n;  // some row of this warp is a node's
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t* nans = reinterpret_cast<const uint32_t*>(smem + Lay<MT>::kNan);
  const int steps = it.stream_steps(w);

  Row row;
  row.line = tree_line(p, b, n, min(node, n - 1), lane);
  const int depth = __popcll(row.line) - 1;
  row.lo = p.window > 0 ? max(0, L + depth - (p.window - 1)) : 0;
  row.hi = L;
  row.r0 = row.lo % kWindow;
  row.r1 = row.r0 + max(0, L - row.lo);
  // positions that every row of the warp attends
  const int lo_all = __reduce_max_sync(0xffffffffu, row.lo);

  float m = -INFINITY, l = 0.f;  // m in log2 units, less kBias
  for (int s = 0; s < steps; ++s) {
    const int ph = it.n[w] + s;
    const int ti = two ? s : 2 * s + w;  // tile of the item
    if (!warp_wait(smem_u32(&B->s_full[w]), static_cast<uint32_t>(ph) & 1u, B)) return false;
    tc_fence_after();
    if (work) {
      const int t = it.t0 + ti, T = it.T + ti;
      const uint32_t sp = lane_base + kColS + 128 * w, pp = lane_base + kColP + 128 * w;
      // NaN in v: recorded when V is an operand
      const int cv = 2 * T + 1;
      if (!warp_wait(smem_u32(&B->ready[cv % NS]), static_cast<uint32_t>(cv / NS) & 1u, B)) return false;
      const uint4 nan4 = *reinterpret_cast<const uint4*>(nans + (T % kInfo) * 4);
      const int s_lo = un.base + (2 * t - 1) * kHalf;
      const bool plain = p.layout != FLINT_KV_RING && t > 0 && s_lo >= lo_all && s_lo + kTrKeys <= L &&
                         (nan4.x | nan4.y | nan4.z | nan4.w) == 0;
      uint32_t mask[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      uint32_t nan[4] = {nan4.x, nan4.y, nan4.z, nan4.w};
      if (!plain) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mask[k] = mask_word(p, un, row, t, k);
          nan[k] &= mask[k];
        }
      }
      auto load = [&](int k, uint32_t (&v)[32]) { tmem_ld32(sp + 32 * k, v); };
      auto masked = [&](int k, uint32_t (&v)[32]) {
        if (!plain) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = mask[k] >> i & 1u ? v[i] : 0xff800000u;
            if (nan[k] >> i & 1u) v[i] = 0x7fc00000u;
          }
        }
      };
      uint32_t va[32], vb[32];
      float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto maxima = [&](const uint32_t (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          mq[(i >> 1) & 3] = max3_nan(mq[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
      };
      load(0, va);
      load(1, vb);
      tmem_wait_ld();
      masked(0, va);
      masked(1, vb);
      maxima(va);
      maxima(vb);
      load(2, va);
      load(3, vb);
      tmem_wait_ld();
      masked(2, va);
      masked(3, vb);
      maxima(va);
      maxima(vb);
      const float mx = max3_nan(max3_nan(mq[0], mq[1], mq[2]), mq[3], mq[3]) * scale - kBias;
      float factor = 1.f;
      const bool need = !(mx <= m + kTau) && mx != -INFINITY;  // (NaN needs)
      if (need) {
        factor = m == -INFINITY ? 0.f : ex2(m - mx);
        m = mx;
        l *= factor;
      }
      const float2 scale2 = make_float2(scale, scale), nmu = m == -INFINITY ? make_float2(0.f, 0.f) : make_float2(-m, -m);
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t pk[32];
      auto probs = [&](const uint32_t (&v)[32], int at) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 x = fma2(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), scale2, nmu);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          ls[c & 1] = add2(ls[c & 1], e);
          const __half2 hp = __floats2half2_rn(e.x, e.y);
          pk[at + c] = *reinterpret_cast<const uint32_t*>(&hp);
        }
      };
      probs(va, 0);
      probs(vb, 16);
      tmem_st32(pp + 32, pk);  // keys 64..127 over S's last columns, which are read
      load(0, va);
      load(1, vb);
      tmem_wait_ld();
      masked(0, va);
      masked(1, vb);
      probs(va, 0);
      probs(vb, 16);
      const float2 lsum = add2(ls[0], ls[1]);
      l += lsum.x + lsum.y;
      tmem_st32(pp, pk);
      if (s > 0 && __any_sync(0xffffffffu, need)) {
        // O_w holds the stream's earlier steps: their PV completed before this S
        const uint32_t op = lane_base + kColO + 128 * w;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tmem_ld32(op + 32 * c, va);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) va[i] = __float_as_uint(__uint_as_float(va[i]) * factor);
          tmem_st32(op + 32 * c, va);
        }
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&B->p_ready[w]));
  }

  // The item's end.  One row tile: both warpgroups' threads of a row join the
  // streams' states, warpgroup w for dims 64 w .. 64 w + 63.
  float a0 = 1.f, a1 = 0.f;
  int first = 0, chunks = 4;
  if (!two) {
    float2* ex = reinterpret_cast<float2*>(smem + Lay<MT>::kEx);
    ex[w * kTrRows + r] = make_float2(m, l);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&B->ex_full));
    if (!warp_wait(smem_u32(&B->ex_full), static_cast<uint32_t>(it.x) & 1u, B)) return false;
    const float2 x0 = ex[r], x1 = ex[kTrRows + r];
    m = x0.x == x0.x && x1.x == x1.x ? fmaxf(x0.x, x1.x) : NAN;
    a0 = x0.x == -INFINITY ? 0.f : ex2(x0.x - m);
    a1 = x1.x == -INFINITY ? 0.f : ex2(x1.x - m);
    l = x0.y * a0 + x1.y * a1;
    first = 2 * w;
    chunks = 2;
  }
  if (!warp_wait(smem_u32(&B->o_full), static_cast<uint32_t>(it.i) & 1u, B)) return false;
  tc_fence_after();
  const bool whole = it.whole(p);
  if (work) {
    const float s2 = p.sinks[h] * kTrLog2e;
    const float vs = p.fp8 ? p.v_scale[g] : 1.f;
    const float sc = whole ? vs / (l + ex2(s2 - m)) : 1.f;
    const int slot = it.i == 0 ? 0 : 1;
    float* part = p.partials + ((static_cast<long long>(q) * kKvHeads + g) * 4 + slot * 2 + (two ? w : 0)) * kTreePartialFloats;
    const bool both = !two && it.steps > 1;
#pragma unroll 1
    for (int c = first; c < first + chunks; ++c) {
      uint32_t v0[32];
      float o[32];
      tmem_ld32(lane_base + kColO + (two ? 128 * w : 0) + 32 * c, v0);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v0[i]);
      if (!two) {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= a0;
        if (both) {
          tmem_ld32(lane_base + kColO + 128 + 32 * c, v0);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = fmaf(__uint_as_float(v0[i]), a1, o[i]);
        }
      }
      if (node < n) {
        if (whole) {
          uint4* out = reinterpret_cast<uint4*>(p.out + ((static_cast<long long>(b) * p.N + node) * kHeads + h) * kDim + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            out[i] = make_uint4(pack_bf16x2(o[8 * i] * sc, o[8 * i + 1] * sc), pack_bf16x2(o[8 * i + 2] * sc, o[8 * i + 3] * sc),
                                pack_bf16x2(o[8 * i + 4] * sc, o[8 * i + 5] * sc), pack_bf16x2(o[8 * i + 6] * sc, o[8 * i + 7] * sc));
        } else {  // [chunk of 4 dims][row]: a warp's stores are whole lines
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<float4*>(part)[(8 * c + i) * kTrRows + r] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
    }
    if (!whole && node < n && (two || w == 0)) {
      part[kTrRows * kDim + r] = m;
      part[kTrRows * kDim + kTrRows + r] = l;
    }
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&B->o_free));
  return true;
}

template <int MT, bool FP8>
__global__ void __launch_bounds__(kTrThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* B = reinterpret_cast<Bars*>(smem + Lay<MT>::kBar);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = blockIdx.x / kKvHeads, g = blockIdx.x % kKvHeads;
  if (base & 1023u) {  // the swizzled tiles need it; the same for every thread
    if (threadIdx.x == 0) report_error(p.dev_err, FLINT_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 6; ++s) {
      mbar_init(smem_u32(&B->full[s]), 1);
      mbar_init(smem_u32(&B->ready[s]), kConvWarps);
      mbar_init(smem_u32(&B->empty[s]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&B->s_full[w]), 1);
      mbar_init(smem_u32(&B->p_ready[w]), 4);
    }
    mbar_init(smem_u32(&B->q_ready), kConvWarps);
    mbar_init(smem_u32(&B->q_empty), 1);
    mbar_init(smem_u32(&B->o_full), 1);
    mbar_init(smem_u32(&B->o_free), kSoftWarps);
    mbar_init(smem_u32(&B->ex_full), kSoftWarps);
    mbar_init(smem_u32(&B->mma_done), 1);
    B->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tensormap(&p.k_map);
    prefetch_tensormap(&p.v_map);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&B->tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base;

  int armed = 0;
  if (warp < kSoftWarps) {
    const float scale = FP8 ? kTrScale * p.k_scale[g] : kTrScale;
    Item it;
    for (bool more = first_item(p, q, it); more; more = next_item(p, q, it))
      if (!softmax_item<MT>(p, it, q, g, scale, tmem, smem, B, warp, lane)) {
        if (lane == 0) raise_abort(p, B);
        break;
      }
  } else if (warp < kTmaWarp) {
    run_conv<MT, FP8>(p, q, g, base, smem, B, threadIdx.x - kSoftWarps * 32);
  } else if (warp == kTmaWarp) {
    armed = run_tma<MT, FP8>(p, q, g, base, B, lane);
  } else if (lane == 0) {
    run_mma<MT, FP8>(p, q, base, tmem, B);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTmaWarp && lane == 0 && aborted(B)) {
    // copies in flight land before the CTA's shared memory goes away: the last
    // kStages stages armed (an earlier one was consumed, so it landed)
    constexpr int NS = Lay<MT>::kStages;
    const unsigned long long t0 = globaltimer_ns();
    for (int c = max(0, armed - NS); c < armed; ++c)
      while (!mbar_try_wait(smem_u32(&B->full[c % NS]), static_cast<uint32_t>(c / NS) & 1u))
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Joins the partials of the units that were cut: a CTA per (unit, node, KV
// head), thread (row of 8, chunk of 4 dims); with M = max m_p,
//     out = sum_p 2^(m_p - M) O_p / (sum_p 2^(m_p - M) l_p + 2^(sink - M)).
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = blockIdx.x % kKvHeads, u = blockIdx.z;
  const TreeUnit& un = p.unit[u];
  const int nd = blockIdx.x / kKvHeads, b = un.b, node = un.rb * 2 * kTrNodes + nd;
  if (un.q0 == un.q1 || node >= p.n_draft[b]) return;
  const int row = threadIdx.x & 7, c = threadIdx.x >> 3, r = (nd & (kTrNodes - 1)) * kGroup + row;
  auto part = [&](int q) {
    const int slot = p.cut[q].unit == u ? 0 : 1;
    return p.partials + ((static_cast<long long>(q) * kKvHeads + g) * 4 + slot * 2 + (nd >> 4)) * kTreePartialFloats;
  };
  float M = -INFINITY;
  bool nan = false;
  for (int q = un.q0; q <= un.q1; ++q) {
    const float m = part(q)[kTrRows * kDim + r];
    nan |= m != m;
    M = fmaxf(M, m);
  }
  if (nan) M = NAN;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int q = un.q0; q <= un.q1; ++q) {
    const float* x = part(q);
    const float m = x[kTrRows * kDim + r], wt = m == -INFINITY ? 0.f : ex2(m - M);
    l = fmaf(x[kTrRows * kDim + kTrRows + r], wt, l);
    const float4 y = reinterpret_cast<const float4*>(x)[c * kTrRows + r];
    o = make_float4(fmaf(y.x, wt, o.x), fmaf(y.y, wt, o.y), fmaf(y.z, wt, o.z), fmaf(y.w, wt, o.w));
  }
  const int h = g * kGroup + row;
  const float sc = (p.fp8 ? p.v_scale[g] : 1.f) / (l + ex2(p.sinks[h] * kTrLog2e - M));
  reinterpret_cast<uint2*>(p.out + ((static_cast<long long>(b) * p.N + node) * kHeads + h) * kDim)[c] =
      make_uint2(pack_bf16x2(o.x * sc, o.y * sc), pack_bf16x2(o.z * sc, o.w * sc));
}

template <int MT, bool FP8>
cudaError_t launch_one(const TreeParams& p, cudaStream_t stream) {
  static ContextSet configured;
  const cudaError_t e = configure_once(configured, reinterpret_cast<const void*>(tree_kernel<MT, FP8>), static_cast<int>(Lay<MT>::kBytes));
  if (e != cudaSuccess) return e;
  tree_kernel<MT, FP8><<<p.n_groups * kKvHeads, kTrThreads, Lay<MT>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

void plan_tree(TreeParams& p, int num_groups) {
  // Units, and what a tile of each costs: with E4M3 a tile is bound by the
  // arithmetic of its row tiles, with bf16 by its bytes.
  int n_units = 0;
  int64_t total = 0;
  int64_t cost[kMaxTreeUnits], begin[kMaxTreeUnits + 1];
  for (int b = 0; b < p.B; ++b) {
    const int L = p.len[b], lo = p.window > 0 ? std::max(0, L - (p.window - 1)) : 0;
    for (int rb = 0; rb * 2 * kTrNodes < p.n_draft[b]; ++rb) {
      TreeUnit& u = p.unit[n_units];
      u.b = static_cast<int16_t>(b);
      u.rb = static_cast<int8_t>(rb);
      u.mt = p.n_draft[b] - rb * 2 * kTrNodes > kTrNodes ? 2 : 1;
      u.base = p.layout == FLINT_KV_RING ? 0 : p.layout == FLINT_KV_PAGED ? lo / kBlock * kBlock : lo;
      u.lo = p.layout == FLINT_KV_RING ? 0 : lo;
      u.hi = p.layout == FLINT_KV_RING ? std::min(L, kWindow) : L;
      u.halves = 1 + (u.hi - u.base + kHalf - 1) / kHalf;
      u.tiles = (u.halves + 1) / 2;
      cost[n_units] = p.fp8 ? u.mt : 1;
      begin[n_units] = total;
      total += cost[n_units] * u.tiles;
      ++n_units;
    }
  }
  begin[n_units] = total;
  p.n_units = n_units;
  // Equal shares, cut at whole tiles; a share without a tile falls away.
  int u = 0, groups = 0;
  for (int k = 0; k <= num_groups; ++k) {
    const int64_t at = total * k / num_groups;
    while (u < n_units && begin[u + 1] <= at) ++u;
    const TreeCut c{static_cast<int16_t>(u), static_cast<int16_t>(u < n_units ? (at - begin[u]) / cost[u] : 0)};
    if (groups > 0 && p.cut[groups - 1].unit == c.unit && p.cut[groups - 1].tile == c.tile) continue;
    p.cut[groups++] = c;
  }
  p.n_groups = groups - 1;
  p.split = 0;
  for (int x = 0; x < n_units; ++x) {
    // the groups with a share of unit x
    int q0 = p.n_groups, q1 = -1;
    for (int q = 0; q < p.n_groups; ++q) {
      const TreeCut a = p.cut[q], e = p.cut[q + 1];
      const int t0 = a.unit < x ? 0 : a.unit == x ? a.tile : p.unit[x].tiles;
      const int t1 = e.unit > x ? p.unit[x].tiles : e.unit == x ? e.tile : 0;
      if (t0 < t1) {
        q0 = std::min(q0, q);
        q1 = std::max(q1, q);
      }
    }
    p.unit[x].q0 = static_cast<int16_t>(q0);
    p.unit[x].q1 = static_cast<int16_t>(q1);
    if (q1 > q0) p.split = 1;
  }
}

cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  if (p.n_units == 0) return cudaSuccess;
  bool two = false;
  int nodes = 0;
  for (int b = 0; b < p.B; ++b) {
    two |= p.n_draft[b] > kTrNodes;
    nodes = std::max(nodes, static_cast<int>(p.n_draft[b]));
  }
  const cudaError_t e = two ? (p.fp8 ? launch_one<2, true>(p, stream) : launch_one<2, false>(p, stream))
                            : (p.fp8 ? launch_one<1, true>(p, stream) : launch_one<1, false>(p, stream));
  if (e != cudaSuccess || !p.split) return e;
  // The second launch's set-up overlaps the first kernel; it waits for that
  // kernel's end before it reads.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(nodes, 2 * kTrNodes) * kKvHeads, 1, p.n_units);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel, p);
}

}  // namespace flint
