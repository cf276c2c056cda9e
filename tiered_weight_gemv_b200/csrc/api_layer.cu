// api_layer.cu — the extern "C" entry points of the decode layer between its projections: argument
// checks and launches. As in api.cu, everything is checked on the host and nothing is launched on
// an error; include/spax.h has the contract of each call.
#include <climits>
#include <cmath>

#include "internal.h"

namespace spax {

// A cache descriptor the kernels may use; strides of dimensions of length 1 are cleared (they are
// never multiplied by more than 0, whatever the caller holds there).
static spax_status check_cache(const spax_kv_cache* h, spax_kv_cache* c) {
  if (!h || !h->d_k || !h->d_v) return SPAX_ERR_ARG;
  *c = *h;
  if (c->dtype != SPAX_KV_BF16 && c->dtype != SPAX_KV_E4M3) return SPAX_ERR_ARG;
  if (c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1) return SPAX_ERR_SHAPE;
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0) return SPAX_ERR_SHAPE;
  const bool bf16 = c->dtype == SPAX_KV_BF16;
  for (const float s : {c->k_scale, c->v_scale})
    if (!std::isfinite(s) || !(s > 0.0f) || (bf16 && s != 1.0f)) return SPAX_ERR_ARG;
  if (!aligned16(c->d_k) || !aligned16(c->d_v)) return SPAX_ERR_ARG;
  const int dims[3] = {c->n_pages, c->page_size, c->n_kv_heads};
  int64_t* const strides[3] = {&c->page_stride, &c->token_stride, &c->head_stride};
  for (int i = 0; i < 3; ++i) {
    if (dims[i] == 1) {
      *strides[i] = 0;
      continue;
    }
    if (*strides[i] < c->head_dim || *strides[i] % (bf16 ? 8 : 16) != 0) return SPAX_ERR_ARG;
    if (*strides[i] > INT64_MAX / 4 / dims[i]) return SPAX_ERR_SHAPE;  // the offsets fit 64 bits
  }
  return SPAX_OK;
}

// A table of max_pages pages for each sequence; sums of a position and a tile's stride fit 32 bits.
static bool pages_ok(const spax_kv_cache& c, int max_pages) {
  return max_pages >= 1 && (long long)max_pages * c.page_size <= 1 << 30;
}

constexpr int64_t kMaxStride = 1ll << 32;  // of rows: the last row's offset fits 64 bits

// Pointers to 4-byte elements (NULL too).
template <class... T>
static bool aligned4(const T*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ... | 0) & 3u) == 0;
}

// Rows of `width` floats: aligned for 16-byte accesses, and apart from one another.
static bool rows_ok(const float* p, int64_t stride, int64_t width, int n) {
  return p && aligned16(p) && (n <= 1 || (stride >= width && stride <= kMaxStride && stride % 4 == 0));
}

// Rows of a residual norm: 8 CTAs (the most that a row takes) for each stay below 2^31, a grid's limit.
constexpr int kMaxRows = 1 << 28;

static bool overlap(const float* a, long long na, const float* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * nb && y < x + 4 * na;
}

}  // namespace spax

using namespace spax;

extern "C" {

spax_status spax_kv_append(const spax_kv_cache* h_cache, const float* q, int64_t q_stride,
                           const float* k, int64_t k_stride, const float* v, int64_t v_stride,
                           int n_tok, int n_heads, const int32_t* seq, const int32_t* pos,
                           const int32_t* page_table, int n_seq, int max_pages,
                           const spax_rope* h_rope, float* q_out, int64_t q_out_stride,
                           int32_t* status, void* stream) {
  AppendLaunch a = {};
  const spax_status st = check_cache(h_cache, &a.cache);
  if (st != SPAX_OK) return st;
  if (n_tok < 0 || n_seq < 0 || n_heads < 0 || n_heads > 65536) return SPAX_ERR_SHAPE;
  if (a.cache.n_kv_heads > 65536) return SPAX_ERR_SHAPE;
  if (n_tok == 0) return SPAX_OK;  // no pointer counts: those of empty tensors are null
  if ((n_heads == 0) != (q == nullptr)) return SPAX_ERR_ARG;
  if (!pos || !page_table || n_seq < 1) return SPAX_ERR_ARG;
  if (!seq && n_tok > n_seq) return SPAX_ERR_ARG;
  if (!aligned4(seq, pos, page_table, status)) return SPAX_ERR_ARG;
  if (!pages_ok(a.cache, max_pages)) return SPAX_ERR_SHAPE;
  const int64_t D = a.cache.head_dim, kv = a.cache.n_kv_heads * D;
  if (q && (!rows_ok(q, q_stride, n_heads * D, n_tok) ||
            !rows_ok(q_out, q_out_stride, n_heads * D, n_tok)))
    return SPAX_ERR_ARG;
  if (!rows_ok(k, k_stride, kv, n_tok) || !rows_ok(v, v_stride, kv, n_tok)) return SPAX_ERR_ARG;
  if (q && q == q_out && n_tok > 1 && q_stride != q_out_stride) return SPAX_ERR_ARG;
  if (h_rope) {
    a.rope = *h_rope;
    if (a.rope.rot_dim < 0 || a.rope.rot_dim > D || a.rope.rot_dim % 8 != 0) return SPAX_ERR_SHAPE;
    if (a.rope.interleaved != 0 && a.rope.interleaved != 1) return SPAX_ERR_ARG;
    if (a.rope.rot_dim > 0 && !a.rope.d_inv_freq) return SPAX_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(a.rope.d_inv_freq) & 7u) return SPAX_ERR_ARG;
  }
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.seq = seq;
  a.pos = pos;
  a.table = page_table;
  a.status = status;
  a.n_tok = n_tok;
  a.n_heads = n_heads;
  a.n_seq = n_seq;
  a.max_pages = max_pages;
  const int sms = sm_count_current_device();
  if (sms < 1) return SPAX_ERR_CUDA;
  return launch_status(launch_kv_append(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t spax_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim) {
  if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads != 0) return 0;
  if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0) return 0;
  const int sms = sm_count_current_device();
  return sms < 1 ? 0 : attention_ws_bytes(n_heads, n_kv_heads, head_dim, sms);
}

spax_status spax_attention_plan_sms(int n_seq, int n_heads, int n_kv_heads, int head_dim, int kv_dtype,
                                    int64_t max_positions, int window, int sm_count, int32_t* ctas,
                                    size_t* ws_bytes) {
  if (kv_dtype != SPAX_KV_BF16 && kv_dtype != SPAX_KV_E4M3) return SPAX_ERR_ARG;
  if (window < 0 || sm_count < 1 || sm_count > 65536) return SPAX_ERR_ARG;  // 4 sm_count CTAs fit an int
  if (n_seq < 1 || n_seq > 65535 || n_heads < 1 || n_heads > 65535) return SPAX_ERR_SHAPE;
  if (n_kv_heads < 1 || n_heads % n_kv_heads != 0) return SPAX_ERR_SHAPE;
  if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0) return SPAX_ERR_SHAPE;
  if (max_positions < 1 || max_positions > 1 << 30) return SPAX_ERR_SHAPE;
  if (ctas)
    *ctas = attention_ctas(n_seq, n_heads, n_kv_heads, head_dim, kv_dtype == SPAX_KV_E4M3, max_positions, window,
                           sm_count);
  if (ws_bytes) *ws_bytes = attention_ws_bytes(n_heads, n_kv_heads, head_dim, sm_count);
  return SPAX_OK;
}

spax_status spax_paged_attention(const spax_kv_cache* h_cache, const float* q, int64_t q_stride,
                                 int n_seq, int n_heads, const int32_t* page_table, int max_pages,
                                 const int32_t* seq_lens, const spax_attn_params* h_params,
                                 float* out, float* lse, int32_t* status, void* ws,
                                 size_t ws_bytes, void* stream) {
  AttnLaunch a = {};
  const spax_status st = check_cache(h_cache, &a.cache);
  if (st != SPAX_OK) return st;
  if (!h_params) return SPAX_ERR_ARG;
  a.prm = *h_params;
  const float cap = a.prm.softcap;  // its reciprocal is formed too
  if (!std::isfinite(a.prm.scale) || !(cap == 0.0f || (cap >= 0x1p-60f && cap <= 0x1p60f)) ||
      a.prm.window < 0)
    return SPAX_ERR_ARG;
  if (n_seq < 0 || n_seq > 65535 || n_heads < 1 || n_heads > 65535) return SPAX_ERR_SHAPE;
  if (n_heads % a.cache.n_kv_heads != 0) return SPAX_ERR_SHAPE;
  if (n_seq == 0) return SPAX_OK;
  if (!page_table || !seq_lens || !out || !aligned16(out)) return SPAX_ERR_ARG;
  if (!aligned4(page_table, seq_lens, lse, status)) return SPAX_ERR_ARG;
  if (!pages_ok(a.cache, max_pages)) return SPAX_ERR_SHAPE;
  const int64_t width = (int64_t)n_heads * a.cache.head_dim;
  if (!rows_ok(q, q_stride, width, n_seq)) return SPAX_ERR_ARG;
  if (overlap(q, (n_seq - 1) * (n_seq > 1 ? q_stride : 0) + width, out, n_seq * width))
    return SPAX_ERR_ARG;
  // the kernel counts units of 64 positions of all rows, and up to 8 more for each row, in 32 bits
  const long long row_units = ((long long)max_pages * a.cache.page_size + 63) / 64 + 1 + 8;
  const long long rows = (long long)a.cache.n_kv_heads * ((n_heads / a.cache.n_kv_heads + 7) / 8);
  if (row_units * rows * n_seq >= INT_MAX) return SPAX_ERR_SHAPE;
  const int sms = sm_count_current_device();
  if (sms < 1) return SPAX_ERR_CUDA;
  if (!ws || ws_bytes < attention_ws_bytes(n_heads, a.cache.n_kv_heads, a.cache.head_dim, sms))
    return SPAX_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return SPAX_ERR_ARG;
  a.q = q;
  a.q_stride = q_stride;
  a.table = page_table;
  a.lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.ws = ws;
  a.n_seq = n_seq;
  a.n_heads = n_heads;
  a.max_pages = max_pages;
  return launch_status(launch_paged_attention(a, sms, static_cast<cudaStream_t>(stream)));
}

static spax_status check_norm(const spax_norm* n) {
  if (!n) return SPAX_OK;
  if (n->kind != SPAX_NORM_RMS && n->kind != SPAX_NORM_LAYER) return SPAX_ERR_ARG;
  if (n->w_dtype != SPAX_W_FP32 && n->w_dtype != SPAX_W_BF16) return SPAX_ERR_ARG;
  if (!(n->eps >= 0.0f) || !std::isfinite(n->eps)) return SPAX_ERR_ARG;
  const uintptr_t align = n->w_dtype == SPAX_W_FP32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(n->d_weight) | reinterpret_cast<uintptr_t>(n->d_bias)) & align)
    return SPAX_ERR_ARG;
  return SPAX_OK;
}

spax_status spax_residual_norm(const float* h, const float* y, int n_tok, int d,
                               const spax_norm* h_post, const float* gate, int64_t gate_stride,
                               float res_scale, float out_scale, const spax_norm* h_pre, float* r,
                               float* x, void* stream) {
  spax_status st = check_norm(h_post);
  if (st == SPAX_OK) st = check_norm(h_pre);
  if (st != SPAX_OK) return st;
  if (n_tok < 0 || n_tok >= kMaxRows || d < 1 || d > 32768) return SPAX_ERR_SHAPE;
  if (!std::isfinite(res_scale) || !std::isfinite(out_scale)) return SPAX_ERR_ARG;
  if (n_tok == 0) return SPAX_OK;
  if (!h || (!r && !x) || (!y && (h_post || gate)) || !aligned4(h, y, gate, r, x)) return SPAX_ERR_ARG;
  if (gate && gate_stride != 0 && (gate_stride < d || gate_stride > kMaxStride)) return SPAX_ERR_ARG;
  // outputs may be an input as a whole, and nothing else
  const long long n = (long long)n_tok * d;
  for (const float* o : {static_cast<const float*>(r), static_cast<const float*>(x)}) {
    if (!o) continue;
    if ((o != h && overlap(o, n, h, n)) || (y && o != y && overlap(o, n, y, n))) return SPAX_ERR_ARG;
    if (gate && overlap(o, n, gate, (n_tok - 1) * gate_stride + d)) return SPAX_ERR_ARG;
  }
  if (r && x && overlap(r, n, x, n)) return SPAX_ERR_ARG;
  NormLaunch a = {};
  a.has_post = h_post != nullptr;
  a.has_pre = h_pre != nullptr;
  if (h_post) a.post = *h_post;
  if (h_pre) a.pre = *h_pre;
  a.h = h;
  a.y = y;
  a.gate = gate;
  a.gate_stride = gate_stride;
  a.r = r;
  a.x = x;
  a.res_scale = res_scale;
  a.out_scale = out_scale;
  a.n_tok = n_tok;
  a.d = d;
  const int sms = sm_count_current_device();
  if (sms < 1) return SPAX_ERR_CUDA;
  return launch_status(launch_residual_norm(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
