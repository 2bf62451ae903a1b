// flint_spec_abi.cu -- the extern "C" entry points of the speculative-decode
// calls: argument checks and launches.  No entry point allocates, frees or
// synchronises; everything is queued on the caller's stream.
#include <string.h>

#include <algorithm>
#include <cmath>

#include "flint_spec.h"

using namespace flint;

namespace {

template <typename... A>
flint_status invalid(const char* fmt, A... a) {
  return record_error(FLINT_ERR_INVALID_ARG, fmt, a...);
}

flint_status launched(cudaError_t e, const char* who) {
  if (e != cudaSuccess) return record_error(FLINT_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return record_ok();
}

flint_status check_batch(int32_t B, int32_t N, const char* who) {
  if (B < 1 || B > FLINT_MAX_BATCH) return invalid("%s: B=%d outside [1, %d]", who, B, FLINT_MAX_BATCH);
  if (N < 1 || N > FLINT_MAX_TREE) return invalid("%s: N=%d outside [1, %d]", who, N, FLINT_MAX_TREE);
  return FLINT_OK;
}

flint_status check_counts(const int32_t* n_draft, int32_t B, int32_t N, int8_t* to, const char* who) {
  for (int b = 0; b < B; ++b) {
    if (n_draft[b] < 0 || n_draft[b] > N) return invalid("%s: n_draft[%d]=%d outside [0, %d]", who, b, n_draft[b], N);
    to[b] = static_cast<int8_t>(n_draft[b]);
  }
  return FLINT_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int64_t request_stride(const flint_kv_cache& c) {
  return c.req_stride ? c.req_stride : static_cast<int64_t>(c.capacity) * kKvHeads * kDim;
}

// The frequencies of the pairs as turns per position; false if the
// description is not a valid one.
flint_status rope_turns(const flint_rope* r, RopeAtParams* p, const char* who) {
  if (!r) return FLINT_OK;
  if (r->rotary_dim < 0 || r->rotary_dim > kDim || r->rotary_dim % 2)
    return invalid("%s: rotary_dim %d must be even and in [0, %d]", who, r->rotary_dim, kDim);
  if (r->layout != FLINT_ROPE_HALF && r->layout != FLINT_ROPE_INTERLEAVED)
    return invalid("%s: unknown rotary layout %d", who, r->layout);
  if (r->scaling != FLINT_ROPE_UNSCALED && r->scaling != FLINT_ROPE_LINEAR && r->scaling != FLINT_ROPE_BY_PARTS)
    return invalid("%s: unknown rotary scaling %d", who, r->scaling);
  if (!(r->theta > 0.0) || !std::isfinite(r->theta) || !(r->factor >= 1.0) || !std::isfinite(r->factor) ||
      !(r->attn_factor > 0.0) || !std::isfinite(r->attn_factor))
    return invalid("%s: theta and attn_factor must be finite and > 0, factor finite and >= 1", who);
  if (r->scaling == FLINT_ROPE_BY_PARTS &&
      (!(r->original_context > 0.0) || !std::isfinite(r->original_context) || !(r->beta_slow >= 0.0) ||
       !(r->beta_fast > r->beta_slow) || !std::isfinite(r->beta_fast)))
    return invalid("%s: scaling by parts needs original_context > 0 and beta_fast > beta_slow >= 0", who);
  if (r->reserved != 0) return invalid("%s: the reserved field of the rope must be 0", who);
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int i = 0; i < r->rotary_dim / 2; ++i) {
    double f = std::pow(r->theta, -2.0 * i / r->rotary_dim);
    if (r->scaling == FLINT_ROPE_LINEAR) f /= r->factor;
    if (r->scaling == FLINT_ROPE_BY_PARTS) {
      const double turns = r->original_context * f / kTwoPi;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - r->beta_slow) / (r->beta_fast - r->beta_slow)));
      f = keep * f + (1.0 - keep) * f / r->factor;
    }
    p->turns[i] = f / kTwoPi;
  }
  p->rotary_dim = r->rotary_dim;
  p->layout = r->layout;
  p->attn_factor = static_cast<float>(r->attn_factor);
  return FLINT_OK;
}

// A 4-D tensor map (128-byte swizzle) of rows of 128 dims: 64 bf16 or 128 E4M3
// values wide boxes of box1 x box2 rows.
flint_status encode_map(CUtensorMap* map, const void* base, bool fp8, const cuuint64_t (&dims)[4], const cuuint64_t (&apart)[3],
                        cuuint32_t box1, cuuint32_t box2, const char* who) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return record_error(FLINT_ERR_CUDA, "%s: cuTensorMapEncodeTiled is not available from the driver", who);
  const cuuint64_t eb = fp8 ? 1 : 2, strides[3] = {apart[0] * eb, apart[1] * eb, apart[2] * eb};
  const cuuint32_t box[4] = {fp8 ? 128u : 64u, box1, box2, 1}, each[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
                        dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        static_cast<CUtensorMapL2promotion>(FLINT_L2_PROMOTION), CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return record_error(FLINT_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (CUresult %d)", who, static_cast<int>(r));
  return FLINT_OK;
}

// A cache buffer, and q or a draft, as the tree attention reads them
// (TreeParams).
flint_status tree_map(CUtensorMap* map, const void* base, const flint_kv_cache& c, int B, const char* who) {
  const bool paged = c.layout == FLINT_KV_PAGED;
  const cuuint64_t request = paged ? static_cast<cuuint64_t>(kBlock) * kKvHeads * kDim : static_cast<cuuint64_t>(request_stride(c));
  return encode_map(map, base, c.dtype == FLINT_KV_FP8_E4M3,
                    {kDim, kKvHeads, static_cast<cuuint64_t>(paged ? kBlock : c.capacity), static_cast<cuuint64_t>(paged ? c.num_blocks : B)},
                    {kDim, kKvHeads * kDim, request}, 1, 64, who);
}
flint_status rows_map(CUtensorMap* map, const void* base, int heads, int rows, cuuint32_t box1, cuuint32_t box2, const char* who) {
  const cuuint64_t row = static_cast<cuuint64_t>(heads) * kDim;
  return encode_map(map, base, false, {kDim, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows), 1},
                    {kDim, row, row * rows}, box1, box2, who);
}

}  // namespace

extern "C" {

flint_status flint_qk_norm_rope_at(const uint16_t* q_raw, int64_t q_stride, const uint16_t* k_raw, int64_t k_stride,
                                   const uint16_t* w_q, const uint16_t* w_k, const int32_t* pos, int32_t T, float eps,
                                   const flint_rope* rope, uint16_t* q_out, uint16_t* k_out, void* stream) {
  FLINT_NVTX_RANGE("flint_qk_norm_rope_at");
  const char* who = "flint_qk_norm_rope_at";
  if (T < 0 || T > FLINT_MAX_CONTEXT) return invalid("%s: T=%d outside [0, %d]", who, T, FLINT_MAX_CONTEXT);
  RopeAtParams p;
  memset(&p, 0, sizeof p);
  const flint_status s = rope_turns(rope, &p, who);
  if (s != FLINT_OK) return s;
  if (T == 0) return record_ok();  // (tensors without elements have no address)
  if (!q_out && !k_out) return invalid("%s: no output requested", who);
  if ((q_out && !q_raw) || (k_out && !k_raw)) return invalid("%s: an output without its input", who);
  if (!pos) return invalid("%s: pos is NULL", who);
  if (!w_q != !w_k) return invalid("%s: w_q and w_k must both be given, or neither", who);
  if (!(eps >= 0.f)) return invalid("%s: eps must be >= 0", who);
  const void* ptrs[] = {q_raw, k_raw, w_q, w_k, q_out, k_out};
  for (const void* x : ptrs)
    if (x && !aligned16(x)) return invalid("%s: pointers must be 16-byte aligned", who);
  if (!aligned4(pos)) return invalid("%s: pos must be 4-byte aligned", who);
  if (q_stride == 0) q_stride = kHeads * kDim;
  if (k_stride == 0) k_stride = kKvHeads * kDim;
  if (q_stride % 8 || k_stride % 8 || q_stride < kHeads * kDim || k_stride < kKvHeads * kDim)
    return invalid("%s: strides must be multiples of 8 and no shorter than a token's row", who);
  if (q_out && q_out == q_raw && q_stride != kHeads * kDim) return invalid("%s: q_out may be q_raw only where that is dense", who);
  if (k_out && k_out == k_raw && k_stride != kKvHeads * kDim) return invalid("%s: k_out may be k_raw only where that is dense", who);
  p.q_raw = q_raw;
  p.k_raw = k_raw;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.w_q = w_q;
  p.w_k = w_k;
  p.pos = pos;
  p.q_out = q_out;
  p.k_out = k_out;
  p.T = T;
  p.eps = eps;
  int sms = 0;
  if (device_num_sms(&sms) != 0) return record_error(FLINT_ERR_CUDA, "%s: cannot read the device's SM count", who);
  return launched(launch_rope_at(p, sms, static_cast<cudaStream_t>(stream)), who);
}

size_t flint_tree_workspace_bytes(int32_t num_ctas) {
  if (num_ctas < 0 || num_ctas > kMaxCtas) return 0;
  int sms = kMaxCtas;
  if (num_ctas == 0 && device_num_sms(&sms) != 0) sms = kMaxCtas;
  return static_cast<size_t>(std::max(1, (num_ctas ? num_ctas : sms) / 4)) * kTreeGroupBytes;
}

flint_status flint_attn_tree(const uint16_t* q, const uint16_t* k_draft, const uint16_t* v_draft, const int32_t* parent,
                             int32_t N, const flint_kv_cache* cache, const int32_t* seq_lens, const int32_t* n_draft,
                             int32_t B, const float* sinks, int32_t window, uint16_t* out, void* workspace,
                             size_t ws_bytes, int32_t num_ctas, int32_t* dev_err, void* stream) {
  FLINT_NVTX_RANGE("flint_attn_tree");
  const char* who = "flint_attn_tree";
  if (!q || !k_draft || !v_draft || !parent || !seq_lens || !n_draft || !sinks || !out || !workspace)
    return invalid("%s: NULL pointer argument", who);
  flint_status s = check_batch(B, N, who);
  if (s != FLINT_OK) return s;
  if (window != 0 && window != kWindow) return record_error(FLINT_ERR_UNSUPPORTED, "%s: window must be 0 or %d", who, kWindow);
  if (num_ctas < 0 || num_ctas > kMaxCtas) return invalid("%s: num_ctas %d outside [0, %d]", who, num_ctas, kMaxCtas);
  const void* ptrs[] = {q, k_draft, v_draft, out, workspace};
  for (const void* x : ptrs)
    if (!aligned16(x)) return invalid("%s: q, drafts, out and workspace must be 16-byte aligned", who);
  if (!aligned4(parent) || !aligned4(sinks)) return invalid("%s: parent and sinks must be 4-byte aligned", who);
  s = check_cache(cache, B, who);
  if (s != FLINT_OK) return s;
  const flint_kv_cache& c = *cache;
  if (c.layout == FLINT_KV_RING && window != kWindow)
    return record_error(FLINT_ERR_UNSUPPORTED, "%s: a ring cache needs window %d", who, kWindow);
  static thread_local TreeParams p;
  memset(&p, 0, sizeof p);
  s = check_counts(n_draft, B, N, p.n_draft, who);
  if (s != FLINT_OK) return s;
  for (int b = 0; b < B; ++b) {
    const int L = seq_lens[b];
    if (L < 0 || L > FLINT_MAX_CONTEXT)
      return invalid("%s: length %d of item %d outside [0, %d]", who, L, b, FLINT_MAX_CONTEXT);
    if (c.layout == FLINT_KV_CONTIGUOUS && L > c.capacity)
      return invalid("%s: length %d of item %d exceeds capacity %d", who, L, b, c.capacity);
    if (c.layout == FLINT_KV_PAGED && static_cast<int64_t>(L) > static_cast<int64_t>(c.max_blocks_per_req) * kBlock)
      return invalid("%s: length %d of item %d exceeds the block table (%d blocks)", who, L, b, c.max_blocks_per_req);
    p.len[b] = L;
  }
  const size_t need = flint_tree_workspace_bytes(num_ctas);
  if (ws_bytes < need)
    return record_error(FLINT_ERR_WORKSPACE, "%s: workspace of %zu bytes is below the %zu needed", who, ws_bytes, need);
  p.q = q;
  p.k_draft = k_draft;
  p.v_draft = v_draft;
  p.k = static_cast<const uint16_t*>(c.k);
  p.v = static_cast<const uint16_t*>(c.v);
  p.req_stride = request_stride(c);
  p.parent = parent;
  p.sinks = sinks;
  p.out = out;
  p.partials = static_cast<float*>(workspace);
  p.table = c.block_table;
  p.layout = c.layout;
  p.max_blocks = c.max_blocks_per_req;
  p.num_blocks = c.num_blocks;
  p.fp8 = c.dtype == FLINT_KV_FP8_E4M3;
  for (int g = 0; g < kKvHeads; ++g) {
    p.k_scale[g] = c.k_scale[g];
    p.v_scale[g] = c.v_scale[g];
    p.k_inv[g] = p.fp8 ? 1.0 / c.k_scale[g] : 0.0;
    p.v_inv[g] = p.fp8 ? 1.0 / c.v_scale[g] : 0.0;
  }
  p.N = N;
  p.B = B;
  p.window = window;
  p.dev_err = dev_err;
  int sms = kMaxCtas;
  if (num_ctas == 0 && device_num_sms(&sms) != 0) return record_error(FLINT_ERR_CUDA, "%s: cannot read the device's SM count", who);
  plan_tree(p, std::max(1, (num_ctas ? num_ctas : sms) / kKvHeads));
  if (p.n_units == 0) return record_ok();
  s = tree_map(&p.k_map, c.k, c, B, who);
  if (s == FLINT_OK) s = tree_map(&p.v_map, c.v, c, B, who);
  if (s == FLINT_OK) s = rows_map(&p.q_map, q, kHeads, B * N, kGroup, 8, who);
  if (s == FLINT_OK) s = rows_map(&p.kd_map, k_draft, kKvHeads, B * N, 1, 64, who);
  if (s == FLINT_OK) s = rows_map(&p.vd_map, v_draft, kKvHeads, B * N, 1, 64, who);
  if (s != FLINT_OK) return s;
  return launched(launch_tree(p, static_cast<cudaStream_t>(stream)), who);
}

int32_t flint_plan_tree(const int32_t* seq_lens, const int32_t* n_draft, int32_t B, int32_t window, int32_t layout, int32_t fp8,
                        int32_t num_ctas, int32_t* units, int32_t max_units, int32_t* n_units, int32_t* cuts, int32_t max_groups) {
  if (!seq_lens || !n_draft || !units || !n_units || !cuts || B < 1 || B > FLINT_MAX_BATCH || num_ctas < 1 || num_ctas > kMaxCtas ||
      (window != 0 && window != kWindow) || layout < FLINT_KV_CONTIGUOUS || layout > FLINT_KV_PAGED)
    return -1;
  static thread_local TreeParams p;
  memset(&p, 0, sizeof p);
  for (int b = 0; b < B; ++b) {
    if (seq_lens[b] < 0 || seq_lens[b] > FLINT_MAX_CONTEXT || n_draft[b] < 0 || n_draft[b] > FLINT_MAX_TREE) return -1;
    p.len[b] = seq_lens[b];
    p.n_draft[b] = static_cast<int8_t>(n_draft[b]);
  }
  p.B = B;
  p.N = FLINT_MAX_TREE;
  p.window = window;
  p.layout = layout;
  p.fp8 = fp8 != 0;
  plan_tree(p, std::max(1, num_ctas / kKvHeads));
  if (p.n_units > max_units || p.n_groups > max_groups) return -1;
  *n_units = p.n_units;
  for (int u = 0; u < p.n_units; ++u) {
    units[4 * u] = p.unit[u].b;
    units[4 * u + 1] = p.unit[u].rb;
    units[4 * u + 2] = p.unit[u].tiles;
    units[4 * u + 3] = p.unit[u].mt;
  }
  for (int q = 0; q <= p.n_groups; ++q) {
    cuts[2 * q] = p.cut[q].unit;
    cuts[2 * q + 1] = p.cut[q].tile;
  }
  return p.n_groups;
}

flint_status flint_verify_tree(const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                               const int32_t* tokens, const int32_t* parent, const int32_t* n_draft, int32_t B, int32_t N,
                               int32_t V, const float* u_accept, const float* u_sample, int32_t* path,
                               int32_t* n_accepted, int32_t* next_token, int32_t* dev_err, void* stream) {
  FLINT_NVTX_RANGE("flint_verify_tree");
  const char* who = "flint_verify_tree";
  if (!target || !tokens || !parent || !n_draft || !u_accept || !u_sample || !path || !n_accepted || !next_token)
    return invalid("%s: NULL pointer argument", who);
  flint_status s = check_batch(B, N, who);
  if (s != FLINT_OK) return s;
  if (V < 1 || V > FLINT_MAX_VOCAB) return invalid("%s: V=%d outside [1, %d]", who, V, FLINT_MAX_VOCAB);
  if (target_stride == 0) target_stride = V;
  if (draft_stride == 0) draft_stride = V;
  if (target_stride < V || draft_stride < V) return invalid("%s: row strides must be 0 or >= V=%d", who, V);
  const void* ptrs[] = {target, draft, tokens, parent, u_accept, u_sample, path, n_accepted, next_token};
  for (const void* x : ptrs)
    if (!aligned4(x)) return invalid("%s: pointers must be 4-byte aligned", who);
  VerifyParams p;
  memset(&p, 0, sizeof p);
  s = check_counts(n_draft, B, N, p.n_draft, who);
  if (s != FLINT_OK) return s;
  p.target = target;
  p.draft = draft;
  p.target_stride = target_stride;
  p.draft_stride = draft_stride;
  p.tokens = tokens;
  p.parent = parent;
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.path = path;
  p.n_accepted = n_accepted;
  p.next_token = next_token;
  p.dev_err = dev_err;
  p.B = B;
  p.N = N;
  p.V = V;
  int sms = 0;
  if (device_num_sms(&sms) != 0) return record_error(FLINT_ERR_CUDA, "%s: cannot read the device's SM count", who);
  return launched(launch_verify(p, sms, static_cast<cudaStream_t>(stream)), who);
}

flint_status flint_kv_append_path(const flint_path_layer* layers, int32_t n_layers, const int32_t* path,
                                  const int32_t* n_accepted, int32_t N, const int32_t* seq_lens, int32_t B,
                                  int32_t* dev_err, void* stream) {
  FLINT_NVTX_RANGE("flint_kv_append_path");
  const char* who = "flint_kv_append_path";
  if (!layers || !path || !n_accepted || !seq_lens) return invalid("%s: NULL pointer argument", who);
  flint_status s = check_batch(B, N, who);
  if (s != FLINT_OK) return s;
  if (n_layers < 1 || n_layers > FLINT_MAX_LAYERS)
    return invalid("%s: n_layers=%d outside [1, %d]", who, n_layers, FLINT_MAX_LAYERS);
  if (!aligned4(path) || !aligned4(n_accepted)) return invalid("%s: path and n_accepted must be 4-byte aligned", who);
  static thread_local AppendPathParams p;
  memset(&p, 0, sizeof p);
  for (int b = 0; b < B; ++b) {
    if (seq_lens[b] < 0 || seq_lens[b] > FLINT_MAX_CONTEXT)
      return invalid("%s: length %d of item %d outside [0, %d]", who, seq_lens[b], b, FLINT_MAX_CONTEXT);
    p.len[b] = seq_lens[b];
  }
  for (int i = 0; i < n_layers; ++i) {
    const flint_path_layer& ly = layers[i];
    if (!ly.k || !ly.v) return invalid("%s: layer %d has a NULL pointer", who, i);
    if (!aligned16(ly.k) || !aligned16(ly.v)) return invalid("%s: layer %d pointers must be 16-byte aligned", who, i);
    s = check_cache(&ly.cache, B, who);
    if (s != FLINT_OK) return s;
    const flint_kv_cache& c = ly.cache;
    PathLayer& to = p.layer[i];
    to.k = ly.k;
    to.v = ly.v;
    to.k_rows = static_cast<uint8_t*>(c.k);
    to.v_rows = static_cast<uint8_t*>(c.v);
    to.table = c.block_table;
    to.req_stride = request_stride(c);
    to.layout = c.layout;
    to.capacity = c.capacity;
    to.max_blocks = c.max_blocks_per_req;
    to.num_blocks = c.num_blocks;
    to.fp8 = c.dtype == FLINT_KV_FP8_E4M3;
    for (int g = 0; g < kKvHeads; ++g) {
      to.k_scale[g] = c.k_scale[g];
      to.v_scale[g] = c.v_scale[g];
      to.k_inv[g] = to.k_scale[g] > 1e-30f && to.k_scale[g] < 1e30f ? 1.0f / to.k_scale[g] : 0.f;
      to.v_inv[g] = to.v_scale[g] > 1e-30f && to.v_scale[g] < 1e30f ? 1.0f / to.v_scale[g] : 0.f;
    }
  }
  p.path = path;
  p.n_accepted = n_accepted;
  p.dev_err = dev_err;
  p.n_layers = n_layers;
  p.N = N;
  p.B = B;
  int sms = 0;
  if (device_num_sms(&sms) != 0) return record_error(FLINT_ERR_CUDA, "%s: cannot read the device's SM count", who);
  return launched(launch_append_path(p, sms, static_cast<cudaStream_t>(stream)), who);
}

}  // extern "C"
