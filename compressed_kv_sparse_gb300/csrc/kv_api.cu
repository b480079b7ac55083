// C ABI of the operators around a paged cache of keys and values: argument checks and
// dispatch. Every check happens on the host before the launch; a failed check launches
// nothing.
#include <cmath>
#include <vector>

#include "internal.h"

using namespace ds4a;

namespace {

ds4a_status cuda_status(cudaError_t e) { return note_error(e) == cudaSuccess ? DS4A_OK : DS4A_ERR_CUDA; }

bool is_row_type(int dtype) { return dtype == DS4A_F32 || dtype == DS4A_BF16; }
uint32_t bytes_of(int dtype) { return dtype == DS4A_F32 ? 4u : dtype == DS4A_BF16 ? 2u : 1u; }

// Whether n rows of `row` elements at x and at y, their strides apart, share memory without being the same rows: threads
// would read what others have written.
bool rows_clash(const void *x, uint64_t xs, const void *y, uint64_t ys, uint32_t n, uint64_t row, uint32_t es) {
  typedef unsigned __int128 wide;
  const wide a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y), last = n - 1u;
  if (a + (last * xs + row) * es <= b || b + (last * ys + row) * es <= a) return false;
  if (n == 1) return x != y;
  if (xs != ys) return true;
  if (x == y) return false;
  const wide step = (wide)xs * es, d = (a < b ? b - a : a - b) % step, len = (wide)row * es;
  return d < len || step - d < len;   // (else: other columns of the same rows)
}

// Whether any of n rows of `row` elements at x, xs apart, shares memory with the `len` contiguous elements at y.
bool rows_meet(const void *x, uint64_t xs, uint64_t row, uint32_t n, const void *y, uint64_t len, uint32_t es) {
  typedef unsigned __int128 wide;
  const wide a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y), end = b + (wide)len * es;
  const wide step = (wide)xs * es, width = (wide)row * es;
  const wide i = b < a + width ? 0 : (b - a - width) / step + 1;   // the first row that ends behind y's start
  return i < n && a + i * step < end;
}

// `inverse`: the flag is allowed.
ds4a_status check_rope(const ds4a_rope_spec &r, uint32_t D, bool inverse) {
  if (r.flags & ~(DS4A_ROPE_HALF | (inverse ? DS4A_ROPE_INVERSE : 0u))) return DS4A_ERR_ARG;
  if (r.n_rot == 0) return DS4A_OK;
  if (r.n_rot % 2 || r.rot_at % 2 || r.n_rot > D || r.rot_at > D - r.n_rot) return DS4A_ERR_SHAPE;
  if (!r.cos || !r.sin || r.max_pos == 0 || !aligned(4, {r.cos, r.sin})) return DS4A_ERR_ARG;
  return DS4A_OK;
}

// The sizes of a cache of keys and values alone.
ds4a_status check_kv_sizes(const ds4a_kv_cache *c) {
  if (!c) return DS4A_ERR_ARG;
  if (!is_row_type(c->dtype) || (c->kv_dtype != c->dtype && c->kv_dtype != DS4A_E4M3)) return DS4A_ERR_DTYPE;
  if (c->head_dim == 0 || c->head_dim > 256 || c->head_dim % 2) return DS4A_ERR_SHAPE;
  if (c->n_kv_heads == 0 || c->n_kv_heads > 128) return DS4A_ERR_SHAPE;
  if (c->batch == 0 || c->batch > DS4A_MAX_TABLE_ROWS) return DS4A_ERR_SHAPE;
  if (c->max_blocks == 0 || c->max_blocks > (1u << 23) || c->n_blocks == 0) return DS4A_ERR_SHAPE;
  if ((uint64_t)c->n_blocks * c->n_kv_heads * 256u > 0x7fffffffu) return DS4A_ERR_SHAPE;
  return DS4A_OK;
}

ds4a_status check_kv(const ds4a_kv_cache *c) {
  ds4a_status st = check_kv_sizes(c);
  if (st) return st;
  if (!c->k || !c->v || !c->block_table) return DS4A_ERR_ARG;
  if (!aligned(16, {c->k, c->v}) || !aligned(4, {c->block_table, c->seq_pos, c->k_scale, c->v_scale}))
    return DS4A_ERR_ARG;
  const bool f8 = c->kv_dtype == DS4A_E4M3;
  if (f8 != (c->k_scale != nullptr) || f8 != (c->v_scale != nullptr)) return DS4A_ERR_ARG;
  return check_rope(c->rope, c->head_dim, false);
}

// The sizes of an attention call.
ds4a_status check_attn_sizes(const ds4a_kv_cache *c, uint32_t max_new, uint32_t n_heads) {
  if (max_new == 0 || max_new > 256 || n_heads == 0 || n_heads > 1024) return DS4A_ERR_SHAPE;
  return n_heads % c->n_kv_heads ? DS4A_ERR_SHAPE : DS4A_OK;
}

PagedArgs paged_args(const ds4a_kv_cache *c, uint32_t max_new, uint32_t n_heads) {
  PagedArgs a = {};
  a.dtype = c->dtype;
  a.kv_dtype = c->kv_dtype;
  a.head_dim = c->head_dim;
  a.n_kv = c->n_kv_heads;
  a.batch = c->batch;
  a.max_blocks = c->max_blocks;
  a.n_blocks = c->n_blocks;
  a.max_new = max_new;
  a.n_heads = n_heads;
  a.k = c->k;
  a.v = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.table = c->block_table;
  a.seq_pos = c->seq_pos;
  return a;
}

}  // namespace

extern "C" {

ds4a_status ds4a_rope_table_scaled(int kind, double base, double factor, double orig_len, double beta_fast,
                                   double beta_slow, double magnitude, uint32_t n_rot, uint32_t n_pos,
                                   float *cos_out, float *sin_out) {
  if (!cos_out || !sin_out || n_rot == 0 || n_rot % 2) return DS4A_ERR_ARG;
  if (kind < DS4A_SCALE_NONE || kind > DS4A_SCALE_YARN) return DS4A_ERR_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return DS4A_ERR_ARG;
  if (kind != DS4A_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return DS4A_ERR_ARG;
  if (kind == DS4A_SCALE_NTK && n_rot <= 2) return DS4A_ERR_ARG;
  const uint32_t half = n_rot / 2;
  double mag = 1.0, low = 0.0, high = 0.0;
  if (kind == DS4A_SCALE_NTK) base *= std::pow(factor, (double)n_rot / (double)(n_rot - 2));
  if (kind == DS4A_SCALE_YARN) {
    if (!(orig_len > 0.0) || !(beta_fast > 0.0) || !(beta_slow > 0.0) || !std::isfinite(orig_len) ||
        !std::isfinite(beta_fast) || !std::isfinite(beta_slow) || !std::isfinite(magnitude) || magnitude < 0.0)
      return DS4A_ERR_ARG;
    const double two_pi = 6.283185307179586;
    auto at = [&](double turns) { return n_rot * std::log(orig_len / (two_pi * turns)) / (2.0 * std::log(base)); };
    low = std::fmax(std::floor(at(beta_fast)), 0.0);
    high = std::fmin(std::ceil(at(beta_slow)), (double)n_rot - 1.0);   // (may lie behind the last pair)
    mag = magnitude > 0.0 ? magnitude : 0.1 * std::log(factor) + 1.0;
  }
  std::vector<double> theta;
  try {
    theta.resize(half);
  } catch (...) {
    return DS4A_ERR_ARG;
  }
  for (uint32_t i = 0; i < half; ++i) {
    double th = std::pow(base, -2.0 * (double)i / (double)n_rot);
    if (kind == DS4A_SCALE_LINEAR) th /= factor;
    if (kind == DS4A_SCALE_YARN) {
      const double g = 1.0 - std::fmin(std::fmax(((double)i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      th *= g + (1.0 - g) / factor;
    }
    theta[i] = th;
  }
  for (uint32_t p = 0; p < n_pos; ++p)
    for (uint32_t i = 0; i < half; ++i) {
      const double ang = (double)p * theta[i];
      cos_out[(size_t)p * half + i] = (float)(std::cos(ang) * mag);
      sin_out[(size_t)p * half + i] = (float)(std::sin(ang) * mag);
    }
  return DS4A_OK;
}

ds4a_status ds4a_rope(const ds4a_rope_spec *rope, int dtype, uint32_t n, const int32_t *pos, const void *x,
                      uint64_t x_stride, uint32_t n_heads, uint32_t head_dim, void *y, uint64_t y_stride,
                      ds4a_stream_t stream) {
  if (!rope) return DS4A_ERR_ARG;
  if (!is_row_type(dtype)) return DS4A_ERR_DTYPE;
  if (head_dim == 0 || head_dim > 512 || head_dim % 2 || n_heads == 0 || n_heads > 1024) return DS4A_ERR_SHAPE;
  const ds4a_status st = check_rope(*rope, head_dim, true);
  if (st) return st;
  const uint64_t row = (uint64_t)n_heads * head_dim;
  if (x_stride < row || y_stride < row || n > 0x7fffffffu) return DS4A_ERR_SHAPE;
  if (n == 0) return DS4A_OK;
  if (!pos || !x || !y || !aligned(4, {pos}) || !aligned(bytes_of(dtype), {x, y})) return DS4A_ERR_ARG;
  if ((x == y && x_stride != y_stride) || rows_clash(x, x_stride, y, y_stride, n, row, bytes_of(dtype))) return DS4A_ERR_ARG;
  RopeArgs a = {};
  a.dtype = a.kv_dtype = dtype;
  a.n = n;
  a.n_heads = n_heads;
  a.head_dim = head_dim;
  a.rot_at = rope->rot_at;
  a.n_rot = rope->n_rot;
  a.max_pos = rope->max_pos;
  a.half = (rope->flags & DS4A_ROPE_HALF) != 0;
  a.inverse = (rope->flags & DS4A_ROPE_INVERSE) != 0;
  a.x = x;
  a.x_stride = x_stride;
  a.y = y;
  a.y_stride = y_stride;
  a.pos = pos;
  a.cos = rope->cos;
  a.sin = rope->sin;
  return cuda_status(launch_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

ds4a_status ds4a_kv_append(const ds4a_kv_cache *c, uint32_t n, const int32_t *tok_seq, const int32_t *tok_pos,
                           const void *k, uint64_t k_stride, const void *v, uint64_t v_stride, const void *q,
                           uint64_t q_stride, uint32_t n_heads, void *q_out, ds4a_stream_t stream) {
  const ds4a_status st = check_kv(c);
  if (st) return st;
  const uint32_t es = bytes_of(c->dtype);
  const uint64_t kv_row = (uint64_t)c->n_kv_heads * c->head_dim, q_row = (uint64_t)n_heads * c->head_dim;
  if (n > 0x7fffffffu || k_stride < kv_row || v_stride < kv_row) return DS4A_ERR_SHAPE;
  if ((q == nullptr) != (q_out == nullptr) || (q == nullptr && n && n_heads)) return DS4A_ERR_ARG;
  if (q && (n_heads == 0 || n_heads > 1024 || q_stride < q_row)) return DS4A_ERR_SHAPE;
  if (q && q == q_out && q_stride != q_row) return DS4A_ERR_ARG;
  if (n == 0) return DS4A_OK;
  if (!tok_seq || !tok_pos || !k || !v || !aligned(4, {tok_seq, tok_pos}) || !aligned(es, {k, v, q, q_out}))
    return DS4A_ERR_ARG;
  if (q && (rows_clash(q, q_stride, q_out, q_row, n, q_row, es) || rows_meet(k, k_stride, kv_row, n, q_out, n * q_row, es) ||
            rows_meet(v, v_stride, kv_row, n, q_out, n * q_row, es)))
    return DS4A_ERR_ARG;
  RopeArgs a = {};
  a.dtype = c->dtype;
  a.kv_dtype = c->kv_dtype;
  a.n = n;
  a.n_heads = n_heads;
  a.n_kv = c->n_kv_heads;
  a.head_dim = c->head_dim;
  a.rot_at = c->rope.rot_at;
  a.n_rot = c->rope.n_rot;
  a.max_pos = c->rope.max_pos;
  a.half = (c->rope.flags & DS4A_ROPE_HALF) != 0;
  a.x = q;
  a.k = k;
  a.v = v;
  a.x_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.y = q_out;
  a.y_stride = q_row;
  a.k_pool = c->k;
  a.v_pool = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.cos = c->rope.cos;
  a.sin = c->rope.sin;
  a.pos = tok_pos;
  a.seq = tok_seq;
  a.table = c->block_table;
  a.batch = c->batch;
  a.max_blocks = c->max_blocks;
  a.n_blocks = c->n_blocks;
  return cuda_status(launch_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t ds4a_paged_attn_ws_bytes(const ds4a_kv_cache *c, uint32_t max_new, uint32_t n_heads) {
  if (check_kv_sizes(c) != DS4A_OK || check_attn_sizes(c, max_new, n_heads) != DS4A_OK) return 0;
  return paged_attn_ws_bytes(paged_args(c, max_new, n_heads));
}

ds4a_status ds4a_paged_attn_decode(const ds4a_kv_cache *c, const uint32_t *cu_len, uint32_t max_new,
                                   const void *q, uint64_t q_stride, uint32_t n_heads, uint32_t window,
                                   float scale, void *out, float *lse, void *ws, size_t ws_bytes,
                                   ds4a_stream_t stream) {
  ds4a_status st = check_kv(c);
  if (st) return st;
  st = check_attn_sizes(c, max_new, n_heads);
  if (st) return st;
  if (q_stride < (uint64_t)n_heads * c->head_dim) return DS4A_ERR_SHAPE;
  if (!c->seq_pos || !q || !out || !std::isfinite(scale)) return DS4A_ERR_ARG;
  if (!aligned(bytes_of(c->dtype), {q, out}) || !aligned(4, {cu_len, lse})) return DS4A_ERR_ARG;
  PagedArgs a = paged_args(c, max_new, n_heads);
  if (!ws || ws_bytes < paged_attn_ws_bytes(a)) return DS4A_ERR_WORKSPACE;
  if (!aligned(16, {ws})) return DS4A_ERR_ARG;
  a.window = window;
  a.scale = scale;
  a.q = q;
  a.q_stride = q_stride;
  a.cu_len = cu_len;
  a.out = out;
  a.lse = lse;
  a.ws = ws;
  return cuda_status(launch_paged_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

ds4a_status ds4a_verify_drafts(int dtype, uint32_t batch, uint32_t max_drafts, uint32_t vocab,
                               const uint32_t *cu_len, const uint32_t *seq_pos, const int32_t *drafts,
                               const void *target, uint64_t target_stride, const void *draft_probs,
                               const float *u_accept, const float *u_sample, int32_t *tokens,
                               uint32_t *n_out, uint32_t *ctx_out, ds4a_stream_t stream) {
  if (!is_row_type(dtype)) return DS4A_ERR_DTYPE;
  if (batch == 0 || batch > DS4A_MAX_TABLE_ROWS || max_drafts == 0 || max_drafts > 255) return DS4A_ERR_SHAPE;
  if (vocab == 0 || vocab > (1u << 20) || target_stride < vocab) return DS4A_ERR_SHAPE;
  if (!drafts || !target || !u_accept || !u_sample || !tokens || !n_out || (ctx_out && !seq_pos))
    return DS4A_ERR_ARG;
  if (!aligned(4, {cu_len, seq_pos, drafts, u_accept, u_sample, tokens, n_out, ctx_out}) ||
      !aligned(bytes_of(dtype), {target, draft_probs}))
    return DS4A_ERR_ARG;
  VerifyArgs a = {};
  a.dtype = dtype;
  a.batch = batch;
  a.max_drafts = max_drafts;
  a.vocab = vocab;
  a.cu_len = cu_len;
  a.seq_pos = seq_pos;
  a.drafts = drafts;
  a.target = target;
  a.target_stride = target_stride;
  a.draft_probs = draft_probs;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.tokens = tokens;
  a.n_out = n_out;
  a.ctx_out = ctx_out;
  return cuda_status(launch_verify(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
