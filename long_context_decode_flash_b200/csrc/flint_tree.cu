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
// head, so that the four read the same token rows at the same time, take either
// whole units, dealt by size, or contiguous shares of all (unit, tile) pairs,
// whichever the plan finds shorter; a unit cut between groups leaves one partial
// per share (O, m, l), and a second launch folds them in order.
//
// A CTA is 15 working warps over two streams of steps, a step being one row tile
// against one key tile.  Two row tiles: stream w is row tile w.  One row tile:
// stream w is the key tiles of parity w, the two streams' states joined at the
// item's end.  So either way one stream's softmax runs beside the other's MMAs:
//   warps 12, 14  TMA producers of K and V: 64-row boxes, the drafts' among them
//               (128-byte swizzle).
//   warps 8-11  make MMA operands of what is none: V to fp16 (bf16 in place, or
//               E4M3 codes), the drafts through the cache's quantisation, Q against
//               E4M3 to its two terms; V rows that hold no token become 0 (whatever
//               lies there must not meet a probability 0).
//   warp 13     issues S_w = Q K^T (M 128, N 128) and O_w += P_w V.
//   warps 0-7   softmax, warpgroup w on stream w, a thread per row: fp32 online
//               softmax in log2 units with a running maximum that moves only
//               by more than 2^8; P goes back to TMEM over S.
// A unit of at most 8 nodes that is cut has its rows twice in the row tile, copy c
// taking the c-th half of each key tile's keys with the other probabilities 0:
// the MMAs cost the same, the softmax half.  The copies are partials of their
// own, joined by the second launch.
// P is one fp16 term, 2^(x - m + 7): at most 2^15 under the lazy maximum, so that
// probabilities keep 11 bits down to 2^-21 of the largest and lose at most 2^-32
// of it below (a bf16 P would round each by 2^-9; two bf16 terms made the softmax
// and the PV product half as long again).  V is fp16 for it: exact for E4M3 and
// for bf16 values from 2^-14 to 65504, to 2^-25 below.  An item (a share of a unit)
// that holds a bf16 v beyond, or where a converter warp met none of 2^-12 (so that
// 2^-25 could be more than 2^-13 of the largest), is done again in fp32 after the
// CTA's last one (exact_items).  Against E4M3, K is the codes themselves and q two
// E4M3 terms a value (split_q_rows), at twice the MMA rate of 16-bit operands.
// TMEM columns: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512).  P_w's fp16
// pairs lie over S_w: those of keys 32 k .. 32 k + 31 at columns 32 k ..  32 k + 15.
// Every wait is bounded; a timeout raises FLINT_ERR_TIMEOUT.
//
// What bounds it, and what it measured (one B200, launches back to back; a tile is
// 128 keys): up to 16 nodes on a bf16 cache the bytes (8 nodes at 100,000 tokens
// 50 to 51 us, of which 31 us are the cache's 205 MB; 32 requests of up to 16 nodes
// 510 us in a burst for 2.65 GB, 5.2 TB/s, and 600 us sustained, when the power limit
// takes the clock from 1,965 to 1,537 MHz); else a row tile's chain softmax ->
// PV -> S -> softmax, 4,400 cycles over two streams, ~2,200 a step where the MMAs
// alone take 1,024 and the exponentials (16 a clock) 1,024 (30 nodes, E4M3, 100,000
// tokens: 72 to 75 us; 64 nodes, batch of 4: 122 to 127 us).  A launch's first and last 4 to 5 us
// are set-up, the first tile, the end of the item and the join.
#include <math.h>

#include <algorithm>

#include "flint_device.cuh"
#include "flint_spec.h"

namespace flint {

#ifdef FLINT_TEST_HOOKS
// {block, K tile}: that CTA's producer leaves that K tile unarmed; {-1, -1} = off.
__device__ int g_stall_tree[2] = {-1, -1};
#endif

namespace {

constexpr int kTrRows = 128;               // rows of a row tile: 16 nodes x 8 heads
constexpr int kTrNodes = kTrRows / kGroup;
constexpr int kHalf = 64;                  // keys of a half tile
constexpr int kTrKeys = 2 * kHalf;         // keys of a tile
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kTmaWarp = kSoftWarps + kConvWarps, kMmaWarp = kTmaWarp + 1, kTmaWarpV = kTmaWarp + 2;
constexpr int kTrThreads = 16 * 32;        // (one warp idle: registers are dealt out by warpgroups)
// Registers a thread: launched with 128, then 256 softmax threads at 192 (a
// row's 128 scores stay in registers), 128 converters and 128 others at 64.
constexpr int kRegSoft = 192, kRegConv = 64, kRegRest = 64;
static_assert(kTrThreads * 128 == 256 * kRegSoft + 128 * kRegConv + 128 * kRegRest, "the launch's registers");
constexpr uint32_t kBox16 = kHalf * 128;            // 64 keys x 64 dims x 16 bit (or 128 dims x 8 bit): 8 KiB
constexpr uint32_t kDimHalf = kTrKeys * 128;        // 64 dims of a 16-bit tile: 16 KiB
constexpr uint32_t kStage = 2 * kDimHalf;           // a K or V tile: 32 KiB
constexpr uint32_t kCodes = 2 * kBox16;             // 128 keys of codes, or 64 drafted rows in bf16: 16 KiB
constexpr uint32_t kQTile = 2 * kTrRows * 128;      // a Q row tile: 32 KiB
constexpr float kTrLog2e = 1.4426950408889634f;
constexpr float kTrScale = static_cast<float>(1.4426950408889634 * 0.08838834764831845);
constexpr float kBias = 7.0f;              // P = 2^(x - m + kBias)
constexpr float kTau = 8.0f;               // the running maximum lags by at most this (log2 units)
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 * stream
constexpr int kInfo = 4;                   // tiles whose record of non-finite v is kept

// Shared memory for MT row tiles a unit (1 or 2): Q; a ring of K and V tiles in
// bf16, or with an E4M3 cache rings of K codes (operands as they land), of V's
// codes and of V's fp16 tiles.
template <int MT, bool FP8>
struct Lay {
  static constexpr int kTiles = FP8 ? 3 : MT == 1 ? 6 : 5;  // bf16 K and V, or K codes
  static constexpr uint32_t kTileBytes = FP8 ? kCodes : kStage;
  static constexpr int kRaws = 3;                             // E4M3: V's codes, the drafts
  // E4M3: V in fp16.  (One row tile: two streams' tiles are in use at once, and a
  // third lets the converters work ahead: 16 requests x 12 nodes 182 -> 180 us.)
  static constexpr int kVs = MT == 1 ? 3 : 2;
  static constexpr uint32_t kTile = MT * kQTile;
  static constexpr uint32_t kRaw = kTile + kTiles * kTileBytes;
  static constexpr uint32_t kV = kRaw + (FP8 ? kRaws * kCodes : 0);
  static constexpr uint32_t kEx = kV + (FP8 ? kVs * kStage : 0);   // m, l of the two streams: [2 streams][128] float2
  static constexpr uint32_t kNan = kEx + 2 * kTrRows * 8;          // [kInfo][8] words
  static constexpr uint32_t kQExp = kNan + kInfo * 32;             // E4M3: exponents of Q's rows, int8 [2][128]
  static constexpr uint32_t kBar = kQExp + 2 * kTrRows;
  static constexpr size_t kBytes = kBar + 512;
};
static_assert(Lay<1, false>::kBytes <= 232448 && Lay<2, false>::kBytes <= 232448 && Lay<1, true>::kBytes <= 232448 &&
              Lay<2, true>::kBytes <= 232448, "shared memory of a CTA");

struct Bars {
  uint64_t full[6], empty[6];            // a K tile landed; a tile (E4M3: K tile) was consumed
  // bf16: a V tile landed.  (Apart from K's: a parity tells a phase from its
  // neighbours only, and who waits for V tiles does not wait for the K tiles between.)
  uint64_t full_v[6];
  uint64_t raw_full[4], raw_free[4];     // E4M3: V's codes, or drafts, landed; were read
  uint64_t v_empty[3];                   // E4M3: an fp16 V tile was consumed
  uint64_t v_ready[4];                   // V of tile T (mod 4) is an operand
  uint64_t kd_ready;                     // E4M3, per item that begins its unit: the drafts' K codes written
  uint64_t s_full[2];                    // S_w complete (and every MMA issued before it)
  uint64_t p_ready[2];                   // P_w written, S_w read
  uint64_t q_full, q_empty;              // per item: Q landed; every S of the item complete
  uint64_t q_ready, q_known;             // E4M3, per item: Q in two terms; its exponents read
  uint64_t o_full, o_free;               // per item: O complete; O read
  uint64_t ex_full;                      // per item with one row tile: m, l of both streams written
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int q_armed;                           // items whose Q loads were issued
  int armed[6], armed_v[6], raw_armed[4];  // per barrier: phases armed
  int odd;                               // bf16: some item is to be done again:
  unsigned v_odd[kMaxTreeUnits / 32];    // ... these
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// Instruction descriptors, fp32 D, M 128, N 128, A K-major; both operands bf16 or
// both fp16 (kind::f16), or both E4M3 (kind::f8f6f4).  S: B (K) K-major; PV: B (V) dims-major.
constexpr uint32_t kIdescBase = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescSBf16 = kIdescBase | (1u << 7) | (1u << 10);
constexpr uint32_t kIdescSE4m3 = kIdescBase;  // (kind::f8f6f4)
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
__device__ __forceinline__ void umma_ss8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : FLINT_R8(0), FLINT_R8(8)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      FLINT_W8(0), FLINT_W8(8), FLINT_W8(16), FLINT_W8(24)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      FLINT_W8(0), FLINT_W8(8)
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
// An fp16 pair, where `clear` with NaN made 0; any NaN sets `nan`, any infinity
// `inf`.
__device__ __forceinline__ uint32_t mend_pair(uint32_t x, bool clear, bool& nan, bool& inf) {
#pragma unroll
  for (int e = 0; e < 32; e += 16) {
    const uint32_t mag = x >> e & 0x7FFFu;
    inf |= mag == 0x7C00u;
    if (mag > 0x7C00u) {
      nan = true;
      if (clear) x &= ~(0xFFFFu << e);
    }
  }
  return x;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A bounded wait of a whole warp: true only if every lane saw the phase
// complete.  The limit is counted in SM cycles (two to a nanosecond at the
// highest clock).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, Bars* B) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    do ok = mbar_try_wait(bar, parity);
    while (!ok && *reinterpret_cast<const volatile int*>(&B->abort) == 0 && clock64() - t0 <= static_cast<long long>(2 * kWaitLimitNs));
  }
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
  int T, n0, n1;         // tiles and steps of stream 0, 1 of the items before this one
  int steps, mt;
  int x, d;              // items with one row tile, items that begin their unit, before this one
  __device__ bool whole(const TreeParams& p) const { return t0 == 0 && t1 == p.unit[u].tiles; }
  __device__ int done(int w) const { return w ? n1 : n0; }
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
  it.i = it.x = it.d = 0;
  it.T = it.n0 = it.n1 = 0;
  return clip(p, q, it);
}
__device__ __forceinline__ bool next_item(const TreeParams& p, int q, Item& it) {
  it.n0 += it.stream_steps(0);
  it.n1 += it.stream_steps(1);
  it.T += it.t1 - it.t0;
  it.x += it.mt == 1;
  it.d += it.t0 == 0;
  ++it.i;
  ++it.u;
  it.t0 = 0;
  return clip(p, q, it);
}

// Some node may not attend storage row s (TreeUnit::part).
__device__ __forceinline__ bool row_in_part(const TreeParams& p, const TreeUnit& un, int s) {
  int t = s - un.part;
  if (p.layout == FLINT_KV_RING && t < 0) t += kWindow;
  return t >= 0 && t < un.part_n;
}
// Every node attends every key of the unit's tile t.
__device__ __forceinline__ bool tile_whole(const TreeParams& p, const TreeUnit& un, int t) {
  const int s0 = un.base + (2 * t - 1) * kHalf, s1 = s0 + kTrKeys, end = un.part + un.part_n;
  return t > 0 && s0 >= un.lo && s1 <= un.hi && (un.part_n == 0 || ((un.part >= s1 || end <= s0) && (p.layout != FLINT_KV_RING || end - kWindow <= s0)));
}

// The order of an item's 2 n operand tiles is that of their first use.  Two row
// tiles: K0 V0 K1 V1 ..; one (S runs two key tiles ahead): K0 K1 V0 K2 V1 .. V.
__device__ __forceinline__ int seq_of(bool v, int j, int n, int mt) {
  if (mt == 2) return 2 * j + v;
  return v ? (j == n - 1 ? 2 * n - 1 : 2 * j + 2) : (j == 0 ? 0 : 2 * j - 1);
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\t.reg .b32 r;\n\telect.sync r|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// Waits for stage `c` of a ring of `size` and arms it with `bytes` (the elected
// lane of a converged warp).
__device__ __forceinline__ bool arm(int c, int size, uint64_t* gone, uint64_t* full, int* armed, uint32_t bytes, Bars* B) {
  if (c >= size && !warp_wait(smem_u32(&gone[c % size]), static_cast<uint32_t>(c / size - 1) & 1u, B)) return false;
  if (elect()) {
    ++armed[c % size];
    mbar_expect_tx(smem_u32(&full[c % size]), bytes);
  }
  return true;
}

// A producer warp: K's (kV false) or V's tiles of the items, in order.  As the
// MMA warp, it runs converged and elects the issuing lane (one warp for both
// kinds took ~1,300 cycles a tile: the kernel's pace).  Page numbers are fetched 32
// at a time, a batch ahead.  False if a wait ran out.
template <int MT, bool FP8, bool kV>
__device__ __forceinline__ bool run_tma(const TreeParams& p, int q, int g, uint32_t base, Bars* B, int lane, bool any, const Item& it0) {
  using Y = Lay<MT, FP8>;
  const CUtensorMap* map = kV ? &p.v_map : &p.k_map;
  const CUtensorMap* draft = kV ? &p.vd_map : &p.kd_map;
  int raws = 0;  // raw stages armed
  Item it = it0;
  for (bool more = any; more; more = next_item(p, q, it)) {
    const TreeUnit& un = p.unit[it.u];
    const int b = un.b, n = it.t1 - it.t0;
    const bool paged = p.layout == FLINT_KV_PAGED;
    const int h0 = 2 * it.t0, h1 = min(2 * it.t1, un.halves);  // halves of the item; half h >= 1: box at base + 64 (h - 1)
    auto pages = [&](int batch) {
      const int h = h0 + 32 * batch + lane;
      int blk = 0;
      if (paged && h >= 1 && h < h1) {
        blk = p.table[static_cast<long long>(b) * p.max_blocks + un.base / kBlock + h - 1];
        if (blk < 0 || blk >= p.num_blocks) {  // never handed to a load
          report_error(p.dev_err, FLINT_ERR_INVALID_ARG);
          blk = 0;
        }
      }
      return blk;
    };
    int now = 0, ahead = pages(0);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      if ((j & 15) == 0) {
        now = ahead;
        ahead = pages((j >> 4) + 1);
      }
#ifdef FLINT_TEST_HOOKS
      if (!kV && static_cast<int>(blockIdx.x) == g_stall_tree[0] && it.T + j == g_stall_tree[1]) continue;
#endif
      const int h = h0 + 2 * j;
      const bool box0 = h >= 1, box1 = h + 1 < h1;  // (box 0 exists behind half 0: h < h1)
      const int row0 = paged ? 0 : un.base + (h - 1) * kHalf, row1 = paged ? 0 : row0 + kHalf;
      const int req0 = paged ? __shfl_sync(0xffffffffu, now, 2 * j & 31) : b;
      const int req1 = paged ? __shfl_sync(0xffffffffu, now, (2 * j & 31) + 1) : b;
      const uint32_t boxes = (box0 ? 1u : 0u) + (box1 ? 1u : 0u);
      if (FP8) {
        // K's codes to their ring, V's to theirs; the drafts (64 rows from the
        // request's first node on) in bf16 to V's, K's by V's producer too
        if (kV && h == 0) {
#pragma unroll 1
          for (int d = 0; d < 2; ++d) {
            if (!arm(raws, Y::kRaws, B->raw_free, B->raw_full, B->raw_armed, 2 * kBox16, B)) return false;
            const uint32_t bar = smem_u32(&B->raw_full[raws % Y::kRaws]), dst = base + Y::kRaw + (raws % Y::kRaws) * kCodes;
            if (elect()) {
              tma_load_4d(dst, d ? &p.vd_map : &p.kd_map, bar, 0, g, b * p.N, 0);
              tma_load_4d(dst + kBox16, d ? &p.vd_map : &p.kd_map, bar, 64, g, b * p.N, 0);
            }
            ++raws;
          }
        }
        const int c = kV ? raws : it.T + j, size = kV ? Y::kRaws : Y::kTiles;
        uint64_t* full = kV ? B->raw_full : B->full;
        if (!arm(c, size, kV ? B->raw_free : B->empty, full, kV ? B->raw_armed : B->armed, boxes * kBox16, B)) return false;
        const uint32_t bar = smem_u32(&full[c % size]), dst = base + (kV ? Y::kRaw : Y::kTile) + (c % size) * kCodes;
        if (elect()) {
          if (box0) tma_load_4d(dst, map, bar, 0, g, row0, req0);
          if (box1) tma_load_4d(dst + kBox16, map, bar, 0, g, row1, req1);
        }
        if (kV) ++raws;
      } else {
        const int c = 2 * it.T + seq_of(kV, j, n, it.mt);
        if (!arm(c, Y::kTiles, B->empty, kV ? B->full_v : B->full, kV ? B->armed_v : B->armed, (boxes + (h == 0 ? 1u : 0u)) * 2 * kBox16, B)) return false;
        const uint32_t bar = smem_u32(&(kV ? B->full_v : B->full)[c % Y::kTiles]), dst = base + Y::kTile + (c % Y::kTiles) * kStage;
        if (elect()) {
          if (box0) {
            tma_load_4d(dst, map, bar, 0, g, row0, req0);
            tma_load_4d(dst + kDimHalf, map, bar, 64, g, row0, req0);
          }
          if (box1) {
            tma_load_4d(dst + kBox16, map, bar, 0, g, row1, req1);
            tma_load_4d(dst + kDimHalf + kBox16, map, bar, 64, g, row1, req1);
          }
          if (h == 0) {
            tma_load_4d(dst, draft, bar, 0, g, b * p.N, 0);
            tma_load_4d(dst + kDimHalf, draft, bar, 64, g, b * p.N, 0);
          }
        }
      }
    }
  }
  return true;
}

// Byte offset of chunk `c` (8 values of 16 bit, c in [0, 16)) of row r in a
// 128-byte-swizzled operand tile of two 64-dim halves.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (c >> 3) * kDimHalf + r * 128 + ((c ^ r) & 7) * 16;
}
__device__ __forceinline__ uint4& smem4(uint8_t* p) { return *reinterpret_cast<uint4*>(p); }
__device__ __forceinline__ uint32_t bf16x2_to_f16(uint32_t w) {
  const __half2 h = __floats2half2_rn(bf16_lo(w), bf16_hi(w));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 bf16x8_to_f16(uint4 v) {
  return make_uint4(bf16x2_to_f16(v.x), bf16x2_to_f16(v.y), bf16x2_to_f16(v.z), bf16x2_to_f16(v.w));
}
// The codes that an E4M3 cache holds for two bf16 values, from the reciprocal of
// its scale in double: x / scale rounded to float, then to E4M3.  The product in
// double is within 2^-52 of the quotient, and a quotient of 8 by 24 bits that is
// not a midpoint of floats (25 bits) is at least 2^-49 away from one: the float is
// the rounded quotient.  (A float division measured several times as long.)
__device__ __forceinline__ uint32_t bf16x2_to_e4m3(uint32_t w, double inv) {
  return f32x2_to_e4m3x2(static_cast<float>(bf16_lo(w) * inv), static_cast<float>(bf16_hi(w) * inv));
}
// acc + 0 * x per half: a half of acc turns NaN where x is not finite (fp16).
__device__ __forceinline__ uint32_t nan_acc(uint32_t acc, uint4 x) {
  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.x), "r"(0u));
  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.y), "r"(0u));
  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.z), "r"(0u));
  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x.w), "r"(0u));
  return acc;
}

__device__ __forceinline__ uint4 mend(uint4 v, bool clear, bool& nan, bool& inf) {
  return make_uint4(mend_pair(v.x, clear, nan, inf), mend_pair(v.y, clear, nan, inf), mend_pair(v.z, clear, nan, inf),
                    mend_pair(v.w, clear, nan, inf));
}
// Per half of acc: the larger of it and the magnitudes of x (fp16), NaN if one is.
constexpr uint32_t kSmallV = 0x0C00u;      // fp16 2^-12
__device__ __forceinline__ void once_more(Bars* B, int item) {
  atomicOr(&B->v_odd[item >> 5], 1u << (item & 31));
  *reinterpret_cast<volatile int*>(&B->odd) = 1;
}
__device__ __forceinline__ uint32_t max_acc(uint32_t acc, uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t a;
    asm("abs.f16x2 %0, %1;" : "=r"(a) : "r"(w[k]));
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(acc) : "r"(a));
  }
  return acc;
}

// A warp's 32 rows of a Q tile, bf16, into two E4M3 terms in place: with 2^e the
// power of two that brings a row's largest magnitude into [128, 256), q 2^e = t1
// + t2 up to 2^-10 (exact for magnitudes down to 2^-9 of the largest: bf16 has 8
// bits, each term 4).  t1's 128 codes take the first 64-dim half's row, t2's the
// second's.  Two rows at a time, 16 lanes each, four times over.  exps gets e; a row with
// something not finite becomes NaN.
__device__ __forceinline__ void split_q_rows(uint8_t* tile, int row0, int8_t* exps, int lane) {
  const int c = lane & 15;
#pragma unroll 1
  for (int i0 = 0; i0 < 16; i0 += 4) {
    uint2 t1[4], t2[4];
    int exp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 y = smem4(tile + chunk_at(row0 + 2 * (i0 + i) + (lane >> 4), c));
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
      // magnitudes of bf16 order as integers, NaN above all
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
      top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int field = static_cast<int>(top >> 7);           // biased exponent
      exp[i] = field == 0 ? 0 : min(126, 134 - field);        // (a row of 0 or subnormal: any)
      const float up = field == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(127 + exp[i]) << 23);
      uint32_t a1[2], a2[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float a = bf16_lo(w[2 * k]) * up, b = bf16_hi(w[2 * k]) * up;
        const float u = bf16_lo(w[2 * k + 1]) * up, v = bf16_hi(w[2 * k + 1]) * up;
        a1[k] = f32x2_to_e4m3x2(a, b) | f32x2_to_e4m3x2(u, v) << 16;
        uint32_t lo, hi;
        e4m3x4_to_f16x2x2(a1[k], lo, hi);
        const float2 ab = __half22float2(*reinterpret_cast<__half2*>(&lo)), uv = __half22float2(*reinterpret_cast<__half2*>(&hi));
        a2[k] = f32x2_to_e4m3x2(a - ab.x, b - ab.y) | f32x2_to_e4m3x2(u - uv.x, v - uv.y) << 16;
      }
      t1[i] = make_uint2(a1[0], a1[1]);
      t2[i] = make_uint2(a2[0], a2[1]);
    }
    __syncwarp();  // these rows are read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 2 * (i0 + i) + (lane >> 4);
      uint8_t* at = tile + chunk_at(r, c >> 1) + (c & 1) * 8;
      *reinterpret_cast<uint2*>(at) = t1[i];
      *reinterpret_cast<uint2*>(at + kDimHalf) = t2[i];
      if (c == 0) exps[r] = static_cast<int8_t>(exp[i]);
    }
  }
}

// The converter warps (thread ct of 128, which owns row ct of a tile).  False
// if a wait ran out.
template <int MT, bool FP8>
__device__ __forceinline__ bool run_conv(const TreeParams& p, int q, int g, uint8_t* smem, Bars* B, int ct, bool any, const Item& it0) {
  using Y = Lay<MT, FP8>;
  const int lane = ct & 31, warp = ct >> 5;
  int raw = 0;  // E4M3: stages of codes and drafts read so far
  uint32_t phases = 0;  // bf16: the parity of each stage's next V tile
  auto raw_stage = [&] { return smem + Y::kRaw + (raw % Y::kRaws) * kCodes; };
  auto raw_wait = [&] { return warp_wait(smem_u32(&B->raw_full[raw % Y::kRaws]), static_cast<uint32_t>(raw / Y::kRaws) & 1u, B); };
  // (Behind the stores of what was made of the stage: a store needs its loads
  // answered, an arrival does not.  Given back right behind the loads, stages were
  // filled again before the last loads of a warp were answered.)
  auto raw_done = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&B->raw_free[raw % Y::kRaws]));
    ++raw;
  };
  Item it = it0;
  for (bool more = any; more; more = next_item(p, q, it)) {
    const TreeUnit& un = p.unit[it.u];
    const int b = un.b, nd = un.nodes, n = it.t1 - it.t0;
    uint32_t largest = 0;  // bf16: this thread's v of the item, fp16 magnitudes
    bool met = false;      // bf16: there was one
    const uint32_t before = static_cast<uint32_t>(it.i - 1) & 1u;
    if (warp == 0) {
      if (it.i > 0 && !warp_wait(smem_u32(&B->q_empty), before, B)) return false;
      if (lane == 0) {
        // Q: row r of tile m is head g * 8 + (r & 7) of node 32 rb + 16 m + (r >> 3);
        // boxes of 8 nodes, the first one again for a second copy of the rows
        // (rows behind the request's nodes are anything: no row meets another)
        const uint32_t bar = smem_u32(&B->q_full), dst = smem_u32(smem);
        B->q_armed = it.i + 1;
        mbar_expect_tx(bar, it.mt * kQTile);
#pragma unroll 1
        for (int x = 0; x < 4 * it.mt; ++x) {
          const int m = x >> 2, half = x >> 1 & 1, dims = x & 1;
          const int node = b * p.N + un.rb * 2 * kTrNodes + m * kTrNodes + (un.dup == 1 ? half * 8 : 0);
          tma_load_4d(dst + m * kQTile + dims * kDimHalf + half * kBox16, &p.q_map, bar, 64 * dims, g * kGroup, node, 0);
        }
      }
      __syncwarp();
    }
    if (FP8) {
      const int j = ct & 63;
      if (it.t0 == 0) {  // the drafts' K as the cache would hold it: codes, half a row a thread
        const int c = it.T;  // (the item's first K tile)
        // (the stage's K tile before has landed: PV has passed the tile behind it)
        if (!raw_wait() || !warp_wait(smem_u32(&B->full[c % Y::kTiles]), static_cast<uint32_t>(c / Y::kTiles) & 1u, B)) return false;
        const uint8_t* from = raw_stage() + (ct >> 6) * kBox16 + j * 128;
        uint8_t* to = smem + Y::kTile + (c % Y::kTiles) * kCodes + j * 128;
        const double inv = p.k_inv[g];
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {  // 16 values, one chunk of codes
          uint32_t code[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 y = *reinterpret_cast<const uint4*>(from + (((2 * i + k) ^ j) & 7) * 16);
            code[2 * k] = bf16x2_to_e4m3(y.x, inv) | bf16x2_to_e4m3(y.y, inv) << 16;
            code[2 * k + 1] = bf16x2_to_e4m3(y.z, inv) | bf16x2_to_e4m3(y.w, inv) << 16;
          }
          smem4(to + (((4 * (ct >> 6) + i) ^ j) & 7) * 16) = make_uint4(code[0], code[1], code[2], code[3]);
        }
        fence_async_smem();
        raw_done();
        if (lane == 0) mbar_arrive(smem_u32(&B->kd_ready));
      }
      if (it.i > 0 && !warp_wait(smem_u32(&B->q_known), before, B)) return false;
      if (!warp_wait(smem_u32(&B->q_full), static_cast<uint32_t>(it.i) & 1u, B)) return false;
#pragma unroll 1
      for (int m = 0; m < it.mt; ++m)
        split_q_rows(smem + m * kQTile, 32 * warp, reinterpret_cast<int8_t*>(smem + Y::kQExp) + m * kTrRows, lane);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B->q_ready));
    }
#pragma unroll 1
    for (int tj = 0; tj < n; ++tj) {  // V
      const int t = it.t0 + tj, T = it.T + tj;
      uint32_t* lost = reinterpret_cast<uint32_t*>(smem + Y::kNan) + (T % kInfo) * 8;
      // does a token stand in row ct of the tile (half 0 is the drafts'), and may
      // some node not attend it?
      const int h = 2 * t + (ct >> 6), j = ct & 63;
      bool token, scan;
      if (h == 0) {
        token = scan = j < nd;
      } else {
        const int s = un.base + (h - 1) * kHalf + j;
        token = h < un.halves && s >= un.lo && s < un.hi;
        scan = token && row_in_part(p, un, s);
      }
      uint8_t* tile;
      uint32_t half_rows = 0;  // record of the drafts' rows' second halves
      bool has = false;   // the row held NaN, and it is for the record
      uint32_t bad = 0;   // an fp16 pair, NaN if so
      if (FP8) {
        tile = smem + Y::kV + (T % Y::kVs) * kStage;
        if (T >= Y::kVs && !warp_wait(smem_u32(&B->v_empty[T % Y::kVs]), static_cast<uint32_t>(T / Y::kVs - 1) & 1u, B)) return false;
        if (t == 0) {  // the drafts, half a row a thread
          if (!raw_wait()) return false;
          const uint8_t* from = raw_stage() + (ct >> 6) * kBox16 + j * 128;
          const double inv = p.v_inv[g];
          bool lost_half = false;
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const uint4 y = *reinterpret_cast<const uint4*>(from + ((i ^ j) & 7) * 16);
            uint4 z = make_uint4(0, 0, 0, 0);
            if (j < nd) {
              const uint32_t a = bf16x2_to_e4m3(y.x, inv) | bf16x2_to_e4m3(y.y, inv) << 16;
              const uint32_t d = bf16x2_to_e4m3(y.z, inv) | bf16x2_to_e4m3(y.w, inv) << 16;
              e4m3x4_to_f16x2x2(a, z.x, z.y);
              e4m3x4_to_f16x2x2(d, z.z, z.w);
            }
            bool none;
            z = mend(z, true, lost_half, none);
            smem4(tile + chunk_at(j, 8 * (ct >> 6) + i)) = z;
          }
          half_rows = __ballot_sync(0xffffffffu, lost_half);
          raw_done();
        }
        if (!raw_wait()) return false;
        uint4 code[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) code[k] = smem4(raw_stage() + ct * 128 + ((k ^ ct) & 7) * 16);
        if (h > 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (!token) code[k] = make_uint4(0, 0, 0, 0);
            uint4 a, d;
            e4m3x4_to_f16x2x2(code[k].x, a.x, a.y);
            e4m3x4_to_f16x2x2(code[k].y, a.z, a.w);
            e4m3x4_to_f16x2x2(code[k].z, d.x, d.y);
            e4m3x4_to_f16x2x2(code[k].w, d.z, d.w);
            bad = nan_acc(nan_acc(bad, a), d);
            smem4(tile + chunk_at(ct, 2 * k)) = a;
            smem4(tile + chunk_at(ct, 2 * k + 1)) = d;
          }
        }
        raw_done();
      } else {
        const int c = 2 * it.T + seq_of(true, tj, n, it.mt);
        tile = smem + Y::kTile + (c % Y::kTiles) * kStage;
        if (!warp_wait(smem_u32(&B->full_v[c % Y::kTiles]), phases >> (c % Y::kTiles) & 1u, B)) return false;
        phases ^= 1u << (c % Y::kTiles);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint4 y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = smem4(tile + chunk_at(ct, 8 * x + k));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[k] = token ? bf16x8_to_f16(y[k]) : make_uint4(0, 0, 0, 0);
            bad = max_acc(bad, y[k]);
            smem4(tile + chunk_at(ct, 8 * x + k)) = y[k];
          }
        }
        bad = max(bad & 0xFFFFu, bad >> 16);
        if (bad < 0x7C00u) largest = max(largest, bad);
        met |= token;
      }
      if (FP8 ? (bad & 0x7FFF7FFFu) != 0u : bad >= 0x7C00u) {
        // NaN becomes 0 where some rows do not attend the key; the rows that do
        // learn of it by the record.  (Where all do, it stays.)  Infinities: the
        // item is done again.
        bool over = false;
#pragma unroll 1
        for (int k = 0; k < 16; ++k) {
          bool nan = false;
          smem4(tile + chunk_at(ct, k)) = mend(smem4(tile + chunk_at(ct, k)), scan, nan, over);
          has |= nan && scan;
        }
        if (over) once_more(B, it.u - p.cut[q].unit);
      }
      if (!FP8 && tj == n - 1 && __any_sync(0xffffffffu, met) && !__any_sync(0xffffffffu, largest >= kSmallV))
        once_more(B, it.u - p.cut[q].unit);
      const uint32_t word = __ballot_sync(0xffffffffu, has);
      if (lane == 0) {
        // words 0..3: the rows; 4, 5: the drafts' rows, their second halves
        lost[warp] = FP8 && t == 0 && warp < 2 ? half_rows : word;
        if (warp >= 2) lost[2 + warp] = half_rows;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B->v_ready[T & 3]));
    }
  }
  return true;
}

// The MMA warp, over its items' steps: S of the first two, then per step PV and
// the S two steps ahead (of the same stream: it overwrites P, whose PV is issued
// before).  The warp runs converged and elects the issuing lane around the MMAs,
// on operands that are the same for the whole warp: then the compiler keeps them
// in uniform registers and an M128 N128 K16 MMA issues every 64 cycles, the
// tensor core's own rate.  (Issued by `if (lane == 0)` code, it measured 143.)
// A barrier's test takes ~130 cycles, so a step's are issued together.
template <int MT, bool FP8>
__device__ __forceinline__ void run_mma(const TreeParams& p, int q, uint32_t base, uint32_t tmem, Bars* B, int lane, bool any, const Item& it0) {
  using Y = Lay<MT, FP8>;
  bool ok = true;
  uint32_t phases = 0;  // bf16: the parity of each stage's next K tile
  Item it = it0;
  for (bool more = any; ok && more; more = next_item(p, q, it)) {
    const int n = it.t1 - it.t0, two = it.mt == 2;
    ok = warp_wait(smem_u32(FP8 ? &B->q_ready : &B->q_full), static_cast<uint32_t>(it.i) & 1u, B);
    if (FP8 && ok && it.t0 == 0) ok = warp_wait(smem_u32(&B->kd_ready), static_cast<uint32_t>(it.d) & 1u, B);
#pragma unroll 1
    for (int s = -2; ok && s < it.steps; ++s) {
      const int w = s & 1, s2 = s + 2;
      // step s2's K tile
      const bool more_s = s2 < it.steps;
      const int tk = two ? s2 >> 1 : s2, ck = FP8 ? it.T + tk : 2 * it.T + seq_of(false, tk, n, it.mt), sk = ck % Y::kTiles;
      const uint32_t k_bar = smem_u32(&B->full[sk]), k_par = FP8 ? static_cast<uint32_t>(ck / Y::kTiles) & 1u : phases >> sk & 1u;
      bool k_ok = !more_s || mbar_try_wait(k_bar, k_par);
      if (s >= 0) {
        const int tv = two ? s >> 1 : s, T = it.T + tv, cv = 2 * it.T + seq_of(true, tv, n, it.mt), sv = cv % Y::kTiles;
        const uint32_t p_bar = smem_u32(&B->p_ready[w]), p_par = static_cast<uint32_t>(it.done(w) + (s >> 1)) & 1u;
        const uint32_t v_bar = smem_u32(&B->v_ready[T & 3]), v_par = static_cast<uint32_t>(T >> 2) & 1u;
        const bool p_ok = mbar_try_wait(p_bar, p_par), v_ok = mbar_try_wait(v_bar, v_par);
        if (!__all_sync(0xffffffffu, p_ok && v_ok)) {
          ok = warp_wait(p_bar, p_par, B) && warp_wait(v_bar, v_par, B);
          if (!ok) break;
        }
        // O of the item before must have been read
        if (s == 0 && it.i > 0 && !(ok = warp_wait(smem_u32(&B->o_free), static_cast<uint32_t>(it.i - 1) & 1u, B))) break;
        tc_fence_after();
        const uint64_t vd = sw128_desc(base + (FP8 ? Y::kV + (T % Y::kVs) * kStage : Y::kTile + sv * kStage), kDimHalf, 1024);
        const uint32_t d = tmem + kColO + 128 * w, at = tmem + kColS + 128 * w, acc = s > 1 ? 1u : 0u;
        if (elect()) {
          // O += P V: 16 keys per MMA (their pairs are 8 columns of P)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t v = vd + ((kk * 16 * 128) >> 4);
            umma_ts(d, at + 32 * (kk >> 1) + 8 * (kk & 1), v, kIdescPV, kk > 0 ? 1u : acc);
          }
          if (!two || w) umma_commit(smem_u32(FP8 ? &B->v_empty[T % Y::kVs] : &B->empty[sv]));
          if (s == it.steps - 1) umma_commit(smem_u32(&B->o_full));
        }
        __syncwarp();
      }
      if (more_s) {
        if (!__all_sync(0xffffffffu, k_ok)) {
          ok = warp_wait(k_bar, k_par, B);
          if (!ok) break;
        }
        if (!FP8 && (!two || w)) phases ^= 1u << sk;
        tc_fence_after();
        // S = Q K^T: 16 dims per MMA, or 32 in each of Q's two E4M3 terms
        const uint64_t qd = sw128_desc(base + (two ? w * kQTile : 0), 16, 1024);
        const uint64_t kd = sw128_desc(base + Y::kTile + sk * Y::kTileBytes, 16, 1024);
        const uint32_t d = tmem + kColS + 128 * w;
        if (elect()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * kDimHalf + (kk & 3) * 32) >> 4;
            if (FP8) umma_ss8(d, qd + off, kd + (((kk & 3) * 32) >> 4), kIdescSE4m3, kk > 0 ? 1u : 0u);
            else umma_ss(d, qd + off, kd + off, kIdescSBf16, kk > 0 ? 1u : 0u);
          }
          umma_commit(smem_u32(&B->s_full[w]));
          if (!two || w) umma_commit(smem_u32(&B->empty[sk]));
          if (s2 == it.steps - 1) umma_commit(smem_u32(&B->q_empty));
        }
        __syncwarp();
      }
    }
  }
  if (!ok && lane == 0) raise_abort(p, B);
  // let every issued MMA finish before the CTA ends (its TMEM is freed)
  if (elect()) umma_commit(smem_u32(&B->mma_done));
  __syncwarp();
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(smem_u32(&B->mma_done), 0))
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
}

// Bits j of 64 with lo <= k0 + j < hi.
__device__ __forceinline__ unsigned long long range_bits(int k0, int lo, int hi) {
  const int a = min(max(lo - k0, 0), 64), e = min(max(hi - k0, 0), 64);
  if (a >= e) return 0ull;
  return ~0ull >> (64 - e) & ~0ull << a;
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

// (All lanes of a warp; rows behind the request's nodes are as its last one's.)
__device__ __forceinline__ Row row_of_node(const TreeParams& p, int b, int n, int L, int node, int lane) {
  Row row;
  row.line = tree_line(p, b, n, min(node, n - 1), lane);
  const int depth = __popcll(row.line) - 1;
  row.lo = p.window > 0 ? max(0, L + depth - (p.window - 1)) : 0;
  row.hi = L;
  row.r0 = row.lo % kWindow;
  row.r1 = row.r0 + max(0, L - row.lo);
  return row;
}

// The mask of half h (of the unit) for a row.
__device__ __forceinline__ unsigned long long half_mask(const TreeParams& p, const TreeUnit& un, const Row& row, int h) {
  if (h == 0) return row.line;
  if (h >= un.halves) return 0ull;
  const int s0 = un.base + (h - 1) * kHalf;
  if (p.layout == FLINT_KV_RING) return range_bits(s0, row.r0, min(row.r1, kWindow)) | range_bits(s0, 0, row.r1 - kWindow);
  return range_bits(s0, row.lo, row.hi);
}

// One step of a row: S to P (P's pairs lie over their own 32-key chunk of S),
// and O brought to the new maximum where it moved.  The row's scores stay in
// registers (one TMEM wait).  masked: keys outside `mask` are not attended; lost:
// one that is has NaN in v, and the row becomes NaN.  The row's chunks are the nk
// from kb on (all four, or its copy's two; the same for a warp); the others get
// probability 0.  (A bit mask of chunks tested at each use instead, and all four
// always loaded: 16 requests x 12 nodes 180 us for 173, 4 x 64 nodes 130 for 124.)
__device__ __forceinline__ void softmax_step(uint32_t sp, uint32_t op, float scale, int kb, int nk, bool first, bool masked,
                                             const uint4& mask, bool lost, float& m, float& l) {
  uint32_t v[4][32];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < nk) tmem_ld32(sp + 32 * (kb + k), v[k]);
  tmem_wait_ld();
  if (masked) {
    const uint32_t words[4] = {kb ? mask.z : mask.x, kb ? mask.w : mask.y, mask.z, mask.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < nk) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[k][i] = words[k] & 1u << i ? v[k][i] : 0xff800000u;
      }
  }
  float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 4; k += 2)
    if (k < nk) {
#pragma unroll
      for (int i = 0; i < 64; i += 2)
        mq[(i >> 1) & 3] = max3_nan(mq[(i >> 1) & 3], __uint_as_float(v[k + (i >> 5)][i & 31]), __uint_as_float(v[k + (i >> 5)][(i & 31) + 1]));
    }
  const float mx = lost ? NAN : max3_nan(max3_nan(mq[0], mq[1], mq[2]), mq[3], mq[3]) * scale - kBias;
  float factor = 1.f;
  const bool need = !(mx <= m + kTau) && mx != -INFINITY;  // (NaN needs)
  if (need) {
    factor = m == -INFINITY ? 0.f : ex2(m - mx);
    m = mx;
    l *= factor;
  }
  const float2 scale2 = make_float2(scale, scale), nmu = m == -INFINITY ? make_float2(0.f, 0.f) : make_float2(-m, -m);
  float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < nk) {
      uint32_t pk[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float2 x = fma2(make_float2(__uint_as_float(v[k][2 * c]), __uint_as_float(v[k][2 * c + 1])), scale2, nmu);
        const float2 e = make_float2(ex2(x.x), ex2(x.y));
        ls[c & 1] = add2(ls[c & 1], e);
        const __half2 hp = __floats2half2_rn(e.x, e.y);
        pk[c] = *reinterpret_cast<const uint32_t*>(&hp);
      }
      tmem_st16(sp + 32 * (kb + k), pk);
    }
  }
  if (nk == 2) {
    const uint32_t zero[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    tmem_st16(sp + 32 * (kb ^ 2), zero);
    tmem_st16(sp + 32 * (kb ^ 2) + 32, zero);
  }
  const float2 lsum = add2(ls[0], ls[1]);
  l += lsum.x + lsum.y;
  if (!first && __any_sync(0xffffffffu, need)) {
    // O_w holds the stream's earlier steps: their PV completed before this S
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      tmem_ld32(op + 32 * c, v[0]);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) v[0][i] = __float_as_uint(__uint_as_float(v[0][i]) * factor);
      tmem_st32(op + 32 * c, v[0]);
    }
  }
  tmem_wait_st();
}

// Softmax of one item by warpgroup w.  False if a wait ran out.
template <int MT, bool FP8>
__device__ __forceinline__ bool softmax_item(const TreeParams& p, const Item& it, int q, int g, float scale, uint32_t tmem,
                                             uint8_t* smem, Bars* B, int warp, int lane) {
  using Y = Lay<MT, FP8>;
  const TreeUnit& un = p.unit[it.u];
  const int w = warp >> 2, b = un.b, n = un.nodes, L = un.len, two = it.mt == 2, dup = un.dup;
  const int r = (warp & 3) * 32 + lane, copy_rows = kTrRows / dup, copy = (warp & 3) * 32 / copy_rows;
  const int tile0 = un.rb * 2 * kTrNodes + (two ? w * kTrNodes : 0);  // first node of this row tile
  const int node = tile0 + ((r & (copy_rows - 1)) >> 3), h = g * kGroup + (r & 7);
  const bool work = __any_sync(0xffffffffu, node < n);  // some row of this warp is a node's
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t* losts = reinterpret_cast<const uint32_t*>(smem + Y::kNan);
  const int steps = it.stream_steps(w);

  const Row row = row_of_node(p, b, n, L, node, lane);
  if (FP8) {
    if (!warp_wait(smem_u32(&B->q_ready), static_cast<uint32_t>(it.i) & 1u, B)) return false;
    const int e = reinterpret_cast<const int8_t*>(smem + Y::kQExp)[(two ? w * kTrRows : 0) + r];
    scale *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    // (an exponent is above -127: lane 0 arrives, once every lane's load is answered)
    const bool none = __any_sync(0xffffffffu, e < -126);
    if (lane == (none ? 1 : 0)) mbar_arrive(smem_u32(&B->q_known));
  }
  float m = -INFINITY, l = 0.f;  // m in log2 units, less P's bias
  for (int s = 0; s < steps; ++s) {
    const int ti = two ? s : 2 * s + w;  // tile of the item
    if (!warp_wait(smem_u32(&B->s_full[w]), static_cast<uint32_t>(it.done(w) + s) & 1u, B)) return false;
    tc_fence_after();
    if (work) {
      const int t = it.t0 + ti, T = it.T + ti;
      const uint32_t sp = lane_base + kColS + 128 * w, op = lane_base + kColO + 128 * w;
      const bool masked = !tile_whole(p, un, t);
      uint4 mask = make_uint4(0, 0, 0, 0);
      bool lost = false;  // an attended key's v is NaN (recorded when V is an operand)
      if (masked) {
        const unsigned long long lo = half_mask(p, un, row, 2 * t), hi = half_mask(p, un, row, 2 * t + 1);
        mask = make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32));
        if (!warp_wait(smem_u32(&B->v_ready[T & 3]), static_cast<uint32_t>(T >> 2) & 1u, B)) return false;
        const uint32_t* rec = losts + (T % kInfo) * 8;
        lost = (((rec[0] | rec[4]) & mask.x) | ((rec[1] | rec[5]) & mask.y) | (rec[2] & mask.z) | (rec[3] & mask.w)) != 0u;
      }
      softmax_step(sp, op, scale, 2 * copy, dup == 1 ? 4 : 2, s == 0, masked, mask, lost, m, l);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&B->p_ready[w]));
  }

  // The item's end.  One row tile: both warpgroups' threads of a row join the
  // streams' states, warpgroup w for dims 64 w .. 64 w + 63.
  float a0 = 1.f, a1 = 0.f;
  int first = 0, chunks = 8;  // of 16 dims
  if (!two) {
    // The exchange is the item's before until all eight warps have read it there,
    // which their arrivals at that item's end tell.  (Nothing else orders the two:
    // this item's first S does not wait for that end, and a stream may have no step.)
    if (it.i > 0 && !warp_wait(smem_u32(&B->o_free), static_cast<uint32_t>(it.i - 1) & 1u, B)) return false;
    float2* ex = reinterpret_cast<float2*>(smem + Y::kEx);
    ex[w * kTrRows + r] = make_float2(m, l);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&B->ex_full));
    if (!warp_wait(smem_u32(&B->ex_full), static_cast<uint32_t>(it.x) & 1u, B)) return false;
    const float2 x0 = ex[r], x1 = ex[kTrRows + r];
    m = x0.x == x0.x && x1.x == x1.x ? fmaxf(x0.x, x1.x) : NAN;
    a0 = x0.x == -INFINITY ? 0.f : ex2(x0.x - m);
    a1 = x1.x == -INFINITY ? 0.f : ex2(x1.x - m);
    l = x0.y * a0 + x1.y * a1;
    first = 4 * w;
    chunks = 4;
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
      uint32_t v0[16], v1[16];
      float o[16];
      tmem_ld16(lane_base + kColO + (two ? 128 * w : 0) + 16 * c, v0);
      if (both) tmem_ld16(lane_base + kColO + 128 + 16 * c, v1);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        o[i] = __uint_as_float(v0[i]) * a0;
        if (both) o[i] = fmaf(__uint_as_float(v1[i]), a1, o[i]);
      }
      if (node < n) {
        if (whole) {
          uint4* out = reinterpret_cast<uint4*>(p.out + ((static_cast<long long>(b) * p.N + node) * kHeads + h) * kDim + 16 * c);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            out[i] = make_uint4(pack_bf16x2(o[8 * i] * sc, o[8 * i + 1] * sc), pack_bf16x2(o[8 * i + 2] * sc, o[8 * i + 3] * sc),
                                pack_bf16x2(o[8 * i + 4] * sc, o[8 * i + 5] * sc), pack_bf16x2(o[8 * i + 6] * sc, o[8 * i + 7] * sc));
        } else {  // [chunk of 4 dims][row]: a warp's stores are whole lines
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(part)[(4 * c + i) * kTrRows + r] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
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

// A node's share of an item once more, bf16, in fp32 throughout, by one warp: v of
// any size counts as the formula has it, infinite and NaN as well.  First the
// maximum and the sum of the keys' scores, then the product with probabilities that
// are divided by the sum already (so that nothing passes the largest v).  A lane
// holds 4 dims of the 8 heads' q and O; a key's 8 scores are summed over the lanes
// so that a lane is left with one head's (head_of).  Bound by the latency of its
// loads: 8 nodes at 100,000 tokens 7.2 ms where the product in fp16 takes 52 us, and
// 92 us where all v are 0 (which is seen first).  It is for values that the caches
// of trained models do not hold; calls without them take what they took without it
// (52 us; 32 paged requests of 16 nodes 531 us).
__device__ __forceinline__ int head_of(int lane) { return lane >> 2; }
// The element offset of a half's first row of KV head g, in the drafts (half 0) or
// in the cache, for a half that holds a token.
__device__ __forceinline__ long long first_row(const TreeParams& p, const TreeUnit& un, int half, int g) {
  if (half == 0) return (static_cast<long long>(un.b) * p.N * kKvHeads + g) * kDim;
  const int s0 = un.base + (half - 1) * kHalf;
  if (p.layout != FLINT_KV_PAGED) return un.b * p.req_stride + (static_cast<long long>(s0) * kKvHeads + g) * kDim;
  const int blk = p.table[static_cast<long long>(un.b) * p.max_blocks + s0 / kBlock];
  return (static_cast<long long>(blk >= 0 && blk < p.num_blocks ? blk : 0) * kBlock * kKvHeads + g) * kDim;
}
// Whether an item has a v that is not 0 (by the softmax warps together).
__device__ __forceinline__ bool some_v(const TreeParams& p, const Item& it, int g, int warp, int lane) {
  const TreeUnit& un = p.unit[it.u];
  uint32_t bits = 0;
#pragma unroll 1
  for (int half = 2 * it.t0 + warp; half < min(2 * it.t1, un.halves); half += kSoftWarps) {
    const int s0 = un.base + (half - 1) * kHalf;
    const int j0 = half > 0 ? max(0, un.lo - s0) : 0, j1 = half > 0 ? min(kHalf, un.hi - s0) : un.nodes;
    const uint16_t* v = (half > 0 ? p.v : p.v_draft) + first_row(p, un, half, g) + 4 * lane;
#pragma unroll 8
    for (int j = j0; j < j1; ++j) {
      const uint2 x = *reinterpret_cast<const uint2*>(v + j * (kKvHeads * kDim));
      bits |= (x.x | x.y) & 0x7FFF7FFFu;
    }
  }
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(bits), "n"(kSoftWarps * 32)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void exact_node(const TreeParams& p, const Item& it, int q, int g, int node, int lane) {
  const TreeUnit& un = p.unit[it.u];
  const int b = un.b, h0 = 2 * it.t0, h1 = min(2 * it.t1, un.halves);
  const Row row = row_of_node(p, b, un.nodes, un.len, node, lane);
  // visit(k, v, i): the lane's dims of each attended key, in order
  auto keys = [&](auto&& visit) {
#pragma unroll 1
    for (int half = h0; half < h1; ++half) {
      const unsigned long long mask = half_mask(p, un, row, half);
      if (!mask) continue;
      const long long at = first_row(p, un, half, g) + 4 * lane;
      const uint16_t *k = (half > 0 ? p.k : p.k_draft) + at, *v = (half > 0 ? p.v : p.v_draft) + at;
#pragma unroll 1
      for (int j = 0; j < kHalf; j += 2) {
        uint2 kr[2], vr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (mask >> (j + i) & 1) {
            kr[i] = *reinterpret_cast<const uint2*>(k + (j + i) * (kKvHeads * kDim));
            vr[i] = *reinterpret_cast<const uint2*>(v + (j + i) * (kKvHeads * kDim));
          }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (mask >> (j + i) & 1) visit(kr[i], vr[i]);
      }
    }
  };
  uint2 qr[kGroup];
#pragma unroll
  for (int h = 0; h < kGroup; ++h)
    qr[h] = *reinterpret_cast<const uint2*>(p.q + ((static_cast<long long>(b) * p.N + node) * kHeads + g * kGroup + h) * kDim + 4 * lane);
  // the score of the lane's head, in log2 units
  auto score = [&](uint2 k) {
    float s[kGroup];
#pragma unroll
    for (int h = 0; h < kGroup; ++h)
      s[h] = fmaf(bf16_lo(qr[h].x), bf16_lo(k.x), bf16_hi(qr[h].x) * bf16_hi(k.x)) + fmaf(bf16_lo(qr[h].y), bf16_lo(k.y), bf16_hi(qr[h].y) * bf16_hi(k.y));
#pragma unroll
    for (int o = 16, n = kGroup / 2; n > 0; o >>= 1, n >>= 1)
#pragma unroll
      for (int h = 0; h < n; ++h) {
        const bool upper = (lane & o) != 0;
        const float give = upper ? s[h] : s[h + n], keep = upper ? s[h + n] : s[h];
        s[h] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 2);
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
    return s[0] * kTrScale;
  };
  float m = -INFINITY, l = 0.f;
  keys([&](uint2 k, uint2) {
    const float x = score(k), top = fmaxf(m, x);
    if (x != x) l = x;
    if (top != -INFINITY) {
      l = l * ex2(m - top) + ex2(x - top);
      m = top;
    }
  });
  const float inv = 1.f / l;
  float o[kGroup][4];
#pragma unroll
  for (int h = 0; h < kGroup; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[h][i] = 0.f;
  keys([&](uint2 k, uint2 v) {
    const float mine = ex2(score(k) - m) * inv;
#pragma unroll
    for (int h = 0; h < kGroup; ++h) {
      const float pr = __shfl_sync(0xffffffffu, mine, 4 * h);
      o[h][0] = fmaf(pr, bf16_lo(v.x), o[h][0]);
      o[h][1] = fmaf(pr, bf16_hi(v.x), o[h][1]);
      o[h][2] = fmaf(pr, bf16_lo(v.y), o[h][2]);
      o[h][3] = fmaf(pr, bf16_hi(v.y), o[h][3]);
    }
  });
  // whole: the sink's share off; else a partial with l in [1/2, 1)
  const bool whole = it.whole(p);
  int e = 0;
  const float f = whole ? l / (l + ex2(p.sinks[g * kGroup + head_of(lane)] * kTrLog2e - m)) : frexpf(l, &e);
  const int in_unit = node - un.rb * 2 * kTrNodes, r0 = (in_unit & (kTrNodes - 1)) * kGroup, slot = it.u == p.cut[q].unit ? 0 : 1;
  float* part = p.partials + ((static_cast<long long>(q) * kKvHeads + g) * 4 + slot * 2 + (in_unit >> 4)) * kTreePartialFloats;
#pragma unroll
  for (int h = 0; h < kGroup; ++h) {
    const float x = __shfl_sync(0xffffffffu, f, 4 * h);
    const float4 y = make_float4(o[h][0] * x, o[h][1] * x, o[h][2] * x, o[h][3] * x);
    if (whole)
      reinterpret_cast<uint2*>(p.out + ((static_cast<long long>(b) * p.N + node) * kHeads + g * kGroup + h) * kDim)[lane] =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    else
      reinterpret_cast<float4*>(part)[lane * kTrRows + r0 + h] = y;
  }
  if (!whole && (lane & 3) == 0) {
    float* ml = part + kTrRows * kDim + r0 + head_of(lane);
    ml[0] = m + static_cast<float>(e);
    ml[kTrRows] = f;
    if (un.dup == 2) {  // the second copy of the row: nothing (O is 0 times it)
      ml[kTrRows / 2] = -INFINITY;
      ml[kTrRows + kTrRows / 2] = 0.f;
    }
  }
  if (!whole && un.dup == 2)
#pragma unroll
    for (int h = 0; h < kGroup; ++h) reinterpret_cast<float4*>(part)[lane * kTrRows + kTrRows / 2 + r0 + h] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// After a CTA's last item (bf16): those whose v left fp16's range, a node a warp.
// (Not inlined: the code that every call runs stays short.)
__device__ __noinline__ void exact_items(const TreeParams& p, int q, int g, const Bars* B, int warp, int lane) {
  const int u0 = p.cut[q].unit;
  const volatile unsigned* odd = B->v_odd;
  Item it;
  it.u = u0;
  it.t0 = p.cut[q].tile;
#pragma unroll 1
  for (; clip(p, q, it); ++it.u, it.t0 = 0) {
    if (!(odd[(it.u - u0) >> 5] >> ((it.u - u0) & 31) & 1u) || !some_v(p, it, g, warp, lane)) continue;  // (of 0 alone O is 0 already)
    const int first = p.unit[it.u].rb * 2 * kTrNodes, end = min(first + 2 * kTrNodes, static_cast<int>(p.unit[it.u].nodes));
#pragma unroll 1
    for (int node = first + warp; node < end; node += kSoftWarps) exact_node(p, it, q, g, node, lane);
  }
}

template <int MT, bool FP8>
__global__ void __launch_bounds__(kTrThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using Y = Lay<MT, FP8>;
  Bars* B = reinterpret_cast<Bars*>(smem + Y::kBar);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = blockIdx.x / kKvHeads, g = blockIdx.x % kKvHeads;
  // (read while the set-up runs: the first touch of parameters takes microseconds)
  Item it0;
  const bool any = first_item(p, q, it0);
  if (base & 1023u) {  // the swizzled tiles need it; the same for every thread
    if (threadIdx.x == 0) report_error(p.dev_err, FLINT_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 6; ++s) {
      B->armed[s] = B->armed_v[s] = 0;
      mbar_init(smem_u32(&B->full[s]), 1);
      mbar_init(smem_u32(&B->full_v[s]), 1);
      mbar_init(smem_u32(&B->empty[s]), 1);
    }
    for (int s = 0; s < 4; ++s) {
      B->raw_armed[s] = 0;
      mbar_init(smem_u32(&B->raw_full[s]), 1);
      mbar_init(smem_u32(&B->raw_free[s]), kConvWarps);
      mbar_init(smem_u32(&B->v_ready[s]), kConvWarps);
    }
    for (int s = 0; s < 3; ++s) mbar_init(smem_u32(&B->v_empty[s]), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&B->s_full[w]), 1);
      mbar_init(smem_u32(&B->p_ready[w]), 4);
    }
    mbar_init(smem_u32(&B->kd_ready), kConvWarps);
    mbar_init(smem_u32(&B->q_full), 1);
    mbar_init(smem_u32(&B->q_empty), 1);
    mbar_init(smem_u32(&B->q_ready), kConvWarps);
    mbar_init(smem_u32(&B->q_known), kSoftWarps);
    mbar_init(smem_u32(&B->o_full), 1);
    mbar_init(smem_u32(&B->o_free), kSoftWarps);
    mbar_init(smem_u32(&B->ex_full), kSoftWarps);
    for (int k = 0; k < kMaxTreeUnits / 32; ++k) B->v_odd[k] = 0;
    B->odd = 0;
    mbar_init(smem_u32(&B->mma_done), 1);
    B->abort = 0;
    B->q_armed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == kTmaWarp && lane == 0) {
    const CUtensorMap* maps[] = {&p.k_map, &p.v_map, &p.q_map, &p.kd_map, &p.vd_map};
#pragma unroll
    for (const CUtensorMap* m : maps) prefetch_tensormap(m);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&B->tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The set-up above overlaps the end of the launch before; what that one wrote
  // is there from here on.  The join may be set up as CTAs end.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, B->tmem_base, 0);

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoft));
    const float scale = FP8 ? kTrScale * p.k_scale[g] : kTrScale;
    Item it = it0;
    for (bool more = any; more; more = next_item(p, q, it))
      if (!softmax_item<MT, FP8>(p, it, q, g, scale, tmem, smem, B, warp, lane)) {
        if (lane == 0) raise_abort(p, B);
        break;
      }
  } else if (warp < kTmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegConv));
    if (!run_conv<MT, FP8>(p, q, g, smem, B, threadIdx.x - kSoftWarps * 32, any, it0) && lane == 0) raise_abort(p, B);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegRest));
    if (warp == kTmaWarp && !run_tma<MT, FP8, false>(p, q, g, base, B, lane, any, it0) && lane == 0) raise_abort(p, B);
    if (warp == kTmaWarpV && !run_tma<MT, FP8, true>(p, q, g, base, B, lane, any, it0) && lane == 0) raise_abort(p, B);
    if (warp == kMmaWarp) run_mma<MT, FP8>(p, q, base, tmem, B, lane, any, it0);
  }
  tc_fence_before();
  __syncthreads();
  if (!FP8 && *reinterpret_cast<const volatile int*>(&B->odd) && warp < kSoftWarps && !aborted(B)) exact_items(p, q, g, B, warp, lane);
  if (warp == kTmaWarp && lane == 0 && aborted(B)) {
    // copies in flight land before the CTA's shared memory goes away: Q and the
    // last of each stage (an earlier one was consumed, so it landed)
    const unsigned long long t0 = globaltimer_ns();
    auto land = [&](uint64_t* bar, int c) {
      while (!mbar_try_wait(smem_u32(bar), static_cast<uint32_t>(c) & 1u))
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
    };
    if (B->q_armed > 0) land(&B->q_full, B->q_armed - 1);
    for (int st = 0; st < Y::kTiles; ++st) {
      if (B->armed[st] > 0) land(&B->full[st], B->armed[st] - 1);
      if (B->armed_v[st] > 0) land(&B->full_v[st], B->armed_v[st] - 1);
    }
    for (int st = 0; st < Y::kRaws; ++st)
      if (B->raw_armed[st] > 0) land(&B->raw_full[st], B->raw_armed[st] - 1);
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Joins the partials of the units that left some: a CTA per (unit, node, KV
// head, 32 dims); thread (row of 8, chunk of 4 dims, share of the partials); with
// M = max m_k,
//     out = sum_k 2^(m_k - M) O_k / (sum_k 2^(m_k - M) l_k + 2^(sink - M)).
// Partial k is copy k % dup of the unit's k / dup-th group.  Bound by the
// latency of its loads: the weights once, then O's of as many
// partials at once as kJoinShares thread groups hold.
constexpr int kJoinShares = 8, kJoinThreads = kGroup * 8 * kJoinShares;
constexpr int kJoinMax = kMaxTreeGroups * 2;
static_assert(kJoinThreads >= kGroup * 32, "a warp per row");
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float2 wt[kJoinMax][kGroup];  // m (then 2^(m - M)), l
  __shared__ float ltot[kGroup], mtop[kGroup];
  __shared__ float4 sum[kJoinShares - 1][kGroup * 8];
  const int g = blockIdx.x % kKvHeads, u = p.cut_unit[blockIdx.z];
  const TreeUnit& un = p.unit[u];
  const int nd = blockIdx.x / kKvHeads, b = un.b, node = un.rb * 2 * kTrNodes + nd;
  const int q0 = un.q0, shift = un.dup >> 1;  // dup 1, 2: 0, 1
  if (node >= un.nodes || nd >= 2 * kTrNodes) return;
  const int parts = (un.q1 - q0 + 1) << shift;
  const int r0 = (nd & (kTrNodes - 1)) * kGroup;
  // only the unit's first group may hold it as a later item than its first
  const int slot0 = p.cut[q0].unit == u ? 0 : 2 * kTreePartialFloats;
  constexpr int kGroupFloats = kKvHeads * 4 * kTreePartialFloats;
  const float* base = p.partials + static_cast<long long>(q0) * kGroupFloats + (g * 4 + (nd >> 4)) * kTreePartialFloats;
  // partial k: its offset, and its row of the node's first head
  auto part = [&](int k) {
    const int q = k >> shift;
    return q * kGroupFloats + (q == 0 ? slot0 : 0);
  };
  auto row_of = [&](int k) { return r0 + (k & shift) * (kTrRows / 2); };
  static_assert(static_cast<long long>(kMaxTreeGroups) * kKvHeads * 4 * kTreePartialFloats < (1ll << 31), "offsets in 32 bits");
  const int row = threadIdx.x & 7, c = blockIdx.y * 8 + (threadIdx.x >> 3 & 7), share = threadIdx.x >> 6;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the first loads of O and those of m and l are in flight together
  constexpr int kAhead = 5;
  float4 y[kAhead];
  auto load = [&](int k) { return *reinterpret_cast<const float4*>(base + part(k) + 4 * (c * kTrRows + row_of(k) + row)); };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (share + i * kJoinShares < parts) y[i] = load(share + i * kJoinShares);
  for (int x = threadIdx.x; x < parts * kGroup; x += kJoinThreads) {
    const float* ml = base + part(x >> 3) + kTrRows * kDim + row_of(x >> 3) + (x & 7);
    wt[x >> 3][x & 7] = make_float2(ml[0], ml[kTrRows]);
  }
  __syncthreads();
  if (threadIdx.x < kGroup * 32) {  // a warp per row
    const int wr = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float M = -INFINITY;
    for (int k = lane; k < parts; k += 32) M = max3_nan(M, wt[k][wr].x, wt[k][wr].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = max3_nan(M, __shfl_xor_sync(0xffffffffu, M, o), M);
    M += 8.0f;  // (so that up to 2^8 partials of the largest bf16 sum to something finite)
    float l = 0.f;
    for (int k = lane; k < parts; k += 32) {
      const float2 ml = wt[k][wr];
      const float e = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
      wt[k][wr].x = e;
      l = fmaf(ml.y, e, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      ltot[wr] = l;
      mtop[wr] = M;
    }
  }
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int k, const float4& v) {
    const float e = wt[k][row].x;
    o = make_float4(fmaf(v.x, e, o.x), fmaf(v.y, e, o.y), fmaf(v.z, e, o.z), fmaf(v.w, e, o.w));
  };
  for (int k0 = share; k0 < parts; k0 += kAhead * kJoinShares) {
    if (k0 != share) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (k0 + i * kJoinShares < parts) y[i] = load(k0 + i * kJoinShares);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (k0 + i * kJoinShares < parts) add(k0 + i * kJoinShares, y[i]);
  }
  if (share > 0) sum[share - 1][threadIdx.x & 63] = o;
  __syncthreads();
  if (share > 0) return;
#pragma unroll
  for (int k = 0; k < kJoinShares - 1; ++k) {
    const float4 v = sum[k][threadIdx.x];
    o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
  }
  const int h = g * kGroup + row;
  const float sc = (p.fp8 ? p.v_scale[g] : 1.f) / (ltot[row] + ex2(p.sinks[h] * kTrLog2e - mtop[row]));
  reinterpret_cast<uint2*>(p.out + ((static_cast<long long>(b) * p.N + node) * kHeads + h) * kDim)[c] =
      make_uint2(pack_bf16x2(o.x * sc, o.y * sc), pack_bf16x2(o.z * sc, o.w * sc));
}

// Launches that overlap their set-up with the end of the launch before
// (griddepcontrol.wait comes before anything is read or written).
cudaError_t launch_overlapped(dim3 grid, int threads, size_t smem, cudaStream_t stream, void (*kernel)(TreeParams), const TreeParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int MT, bool FP8>
cudaError_t launch_one(const TreeParams& p, cudaStream_t stream) {
  static ContextSet configured;
  constexpr size_t bytes = Lay<MT, FP8>::kBytes;
  const cudaError_t e = configure_once(configured, reinterpret_cast<const void*>(tree_kernel<MT, FP8>), static_cast<int>(bytes));
  if (e != cudaSuccess) return e;
  return launch_overlapped(dim3(p.n_groups * kKvHeads), kTrThreads, bytes, stream, tree_kernel<MT, FP8>, p);
}

}  // namespace

// What the beginning of a unit costs a CTA beside its tiles, in tiles of one row
// tile: its Q, its drafts, and the end of the unit before.  (Against E4M3, Q and
// the drafts are converted.  64 nodes, batch of 4: 137 us with 2, 132 with 8, 129
// with 12; bf16 measures the same from 2 to 12.)
constexpr int kUnitCost = 4, kUnitCostE4m3 = 12;
// What the second launch and the partials cost, in the same measure, for one unit;
// half as much more for each unit beside it, up to 17.  (Windows of 513 of 32
// requests with 8 nodes: 16.0 us whole, 28.5 cut; of one request: 13.2 whole, 9.9
// cut; 64 requests of 100 to 4,000 tokens: 56 whole, 69 cut.)
constexpr int kJoinCost = 3;

void plan_tree(TreeParams& p, int num_groups) {
  // Units, and what a tile of each costs: with E4M3 a tile is bound by the
  // arithmetic of its row tiles, with bf16 by its bytes.
  int n_units = 0;
  const int unit_cost = p.fp8 ? kUnitCostE4m3 : kUnitCost;
  int64_t total = 0;
  int64_t cost[kMaxTreeUnits], begin[kMaxTreeUnits + 1];
  for (int b = 0; b < p.B; ++b) {
    const int L = p.len[b], lo = p.window > 0 ? std::max(0, L - (p.window - 1)) : 0;
    for (int rb = 0; rb * 2 * kTrNodes < p.n_draft[b]; ++rb) {
      TreeUnit& u = p.unit[n_units];
      u.b = static_cast<int16_t>(b);
      u.nodes = p.n_draft[b];
      u.len = L;
      u.rb = static_cast<int8_t>(rb);
      u.mt = p.n_draft[b] - rb * 2 * kTrNodes > kTrNodes ? 2 : 1;
      u.base = p.layout == FLINT_KV_RING ? 0 : p.layout == FLINT_KV_PAGED ? lo / kBlock * kBlock : lo;
      u.lo = p.layout == FLINT_KV_RING ? 0 : lo;
      u.hi = p.layout == FLINT_KV_RING ? std::min(L, kWindow) : L;
      const int left = std::max(0, L - kWindow), deep = std::max(0, L - (p.window - 1) + p.n_draft[b] - 1);  // positions
      const bool ring = p.layout == FLINT_KV_RING;
      u.part = ring ? left % kWindow : lo;
      u.part_n = p.window == 0 ? 0 : std::min(L, deep) - (ring ? left : lo);
      u.halves = 1 + (u.hi - u.base + kHalf - 1) / kHalf;
      u.tiles = (u.halves + 1) / 2;
      cost[n_units] = p.fp8 ? u.mt : 1;
      begin[n_units] = total;
      total += cost[n_units] * u.tiles + unit_cost;
      ++n_units;
    }
  }
  begin[n_units] = total;
  p.n_units = n_units;
  int groups = 0;
  // Whole units, the longest first, each to the group with the least ...
  int order[kMaxTreeUnits], of[kMaxTreeUnits];
  for (int u = 0; u < n_units; ++u) order[u] = u;
  auto cost_of = [&](int u) { return begin[u + 1] - begin[u]; };
  std::stable_sort(order, order + n_units, [&](int a, int b) { return cost_of(a) > cost_of(b); });
  int64_t load[kMaxTreeGroups] = {}, fullest = 0;
  const int usable = std::min(num_groups, n_units);
  for (int i = 0; i < n_units; ++i) {
    const int g = static_cast<int>(std::min_element(load, load + usable) - load);
    of[order[i]] = g;
    load[g] += cost_of(order[i]);
    fullest = std::max(fullest, load[g]);
  }
  // ... where that takes no longer than even shares and their join
  const int64_t join = kJoinCost + std::min(17, n_units / 2);
  if (n_units > 0 && fullest <= std::max<int64_t>(total / num_groups, unit_cost + 1) + join) {
    TreeUnit unit[kMaxTreeUnits];
    std::copy(p.unit, p.unit + n_units, unit);
    int n = 0;
    for (int g = 0; g < usable; ++g) {
      p.cut[groups++] = TreeCut{static_cast<int16_t>(n), 0};
      for (int u = 0; u < n_units; ++u)
        if (of[u] == g) p.unit[n++] = unit[u];
    }
    p.cut[groups++] = TreeCut{static_cast<int16_t>(n), 0};
  } else {
    // Equal shares, cut at whole tiles; a share without a tile falls away.
    int u = 0;
    for (int k = 0; k <= num_groups; ++k) {
      const int64_t at = total * k / num_groups;
      while (u < n_units && begin[u + 1] <= at) ++u;
      const TreeCut c{static_cast<int16_t>(u), static_cast<int16_t>(u < n_units ? std::max<int64_t>(0, at - begin[u] - unit_cost) / cost[u] : 0)};
      if (groups > 0 && p.cut[groups - 1].unit == c.unit && p.cut[groups - 1].tile == c.tile) continue;
      p.cut[groups++] = c;
    }
  }
  p.n_groups = groups - 1;
  // the groups with a share of each unit (no group is empty: they are a range)
  p.n_cut = p.cut_nodes = 0;
  int q = 0;
  for (int x = 0; x < n_units; ++x) {
    while (p.cut[q + 1].unit < x || (p.cut[q + 1].unit == x && p.cut[q + 1].tile == 0)) ++q;
    p.unit[x].q0 = static_cast<int16_t>(q);
    while (p.cut[q + 1].unit == x) ++q;  // (group q ends within x, so q + 1 goes on with it)
    p.unit[x].q1 = static_cast<int16_t>(q);
    const bool cut = p.unit[x].q1 > p.unit[x].q0;
    const int nodes = p.n_draft[p.unit[x].b] - p.unit[x].rb * 2 * kTrNodes;
    p.unit[x].dup = cut && nodes <= kTrNodes / 2 ? 2 : 1;
    if (cut) {
      p.cut_unit[p.n_cut++] = static_cast<int16_t>(x);
      p.cut_nodes = std::max(p.cut_nodes, std::min(nodes, 2 * kTrNodes));
    }
  }
}

#ifdef FLINT_TEST_HOOKS
// Test builds only: CTA `block` leaves its K tile `tile` unarmed; block = -1
// turns the hook off.
extern "C" int flint_test_stall_tree(int block, int tile) {
  const int v[2] = {block, tile};
  return static_cast<int>(cudaMemcpyToSymbol(g_stall_tree, v, sizeof v));
}
#endif

cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  if (p.n_units == 0) return cudaSuccess;
  bool two = false;
  for (int b = 0; b < p.B; ++b) two |= p.n_draft[b] > kTrNodes;
  const cudaError_t e = two ? (p.fp8 ? launch_one<2, true>(p, stream) : launch_one<2, false>(p, stream))
                            : (p.fp8 ? launch_one<1, true>(p, stream) : launch_one<1, false>(p, stream));
  if (e != cudaSuccess || p.n_cut == 0) return e;
  return launch_overlapped(dim3(p.cut_nodes * kKvHeads, 4, p.n_cut), kJoinThreads, 0, stream, tree_join_kernel, p);
}

}  // namespace flint
