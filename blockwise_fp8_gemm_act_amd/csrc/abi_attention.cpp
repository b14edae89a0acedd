// C ABI of the attention block's operators: argument validation on the host,
// device check, dispatch to the gfx950 kernels.  See include/puro_attention.h for
// the contract of every call; checks run in the order of abi.cpp, the values of
// scalars after the shapes.
#include "puro_attention.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "abi_check.h"
#include "launch_attention.h"

using namespace puro_abi;

namespace {

constexpr int64_t kMaxPositions = int64_t(1) << 24;
constexpr int64_t kMaxRows = int64_t(1) << 30;      // of q and of k: positions plus a window stay in 32 bits
constexpr int64_t kMaxStride = int64_t(1) << 23;    // 64 rows of it stay in 32 bits of bytes

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A tensor of `rows` rows of `width` elements, `stride` elements apart.
struct Rows {
  const void *p;
  int64_t rows, width, stride;
  int64_t elem = 2;
};

Range rng(const Rows &t) {
  return puro_abi::rng(t.p, t.p && t.rows > 0 && t.width > 0 ? ((t.rows - 1) * t.stride + t.width) * t.elem : 0);
}

// Two slices of the same rows are apart when their columns are.
bool overlap(const Rows &a, const Rows &b) {
  const Range ra = rng(a), rb = rng(b);
  if (!puro_abi::overlap(ra, rb)) return false;
  if (a.elem != b.elem || a.stride != b.stride) return true;
  const int64_t s = a.stride * a.elem;
  const int64_t diff = rb.lo >= ra.lo ? (int64_t)((rb.lo - ra.lo) % (uintptr_t)s)
                                      : (s - (int64_t)((ra.lo - rb.lo) % (uintptr_t)s)) % s;
  return !(diff >= a.width * a.elem && diff + b.width * b.elem <= s);
}

bool any_alias(const Rows *in, int nin, const Rows *out, int nout) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = i + 1; j < nout; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

bool strided_ok(int64_t rows, int64_t width, int64_t stride) {
  return stride >= width && stride < kMaxStride && stride % 8 == 0 && shape_ok(rows, width) && shape_ok(rows, stride);
}

bool head_dim_ok(int64_t d) { return d == 64 || d == 128; }

// The rotation's scalars and pointers.
puro_status rotation_mode(const puro_rotation *r) {
  if (!r) return PURO_ERR_NULL;
  return r->layout == PURO_ROPE_HALF || r->layout == PURO_ROPE_INTERLEAVED ? PURO_OK : PURO_ERR_MODE;
}
bool rotation_shape(const puro_rotation *r, int64_t head_dim) {
  return r->rot > 0 && r->rot % 16 == 0 && r->rot <= head_dim && r->positions > 0 && r->positions < kMaxPositions;
}
Rows table_rows(const puro_rotation *r) { return Rows{r->table, r->positions, r->rot, r->rot, 4}; }
Rows pos_rows(const puro_rotation *r, int64_t tokens) { return Rows{r->pos, 1, tokens, tokens, 4}; }

// The checks the two forward forms and the backward form of the norms share.
bool heads_ok(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim) {
  return head_dim_ok(head_dim) && tokens >= 0 && q_heads >= 0 && k_heads >= 0 && q_heads <= 65536 && k_heads <= 65536 &&
         tokens <= kMaxDim;
}

puro::RopeArgs rope_args(const puro_rotation *r, const uint16_t *x, int64_t xs, int64_t tokens) {
  puro::RopeArgs a{};
  a.x = x;
  a.xs = xs;
  a.tokens = tokens;
  a.table = r->table;
  a.positions = r->positions;
  a.rot = (int)r->rot;
  a.pos = r->pos;
  a.sign = 1.0f;
  return a;
}

puro_status norm_rope(const puro_rotation *r, const uint16_t *x, int64_t x_stride, int64_t tokens, int64_t q_heads,
                      int64_t k_heads, int64_t head_dim, const uint16_t *wq, const uint16_t *wk, float eps, uint16_t *q,
                      int64_t q_stride, uint16_t *k, int64_t k_stride, bool append, uint16_t *v, int64_t v_stride,
                      const int32_t *rows, int64_t cache_rows, puro_stream_t stream) {
  if (puro_status s = rotation_mode(r)) return s;
  if (!heads_ok(tokens, q_heads, k_heads, head_dim) || !rotation_shape(r, head_dim)) return PURO_ERR_SHAPE;
  const int64_t v_heads = append ? k_heads : 0, heads = q_heads + k_heads + v_heads;
  const int64_t k_rows = append ? cache_rows : tokens;
  if (!strided_ok(tokens, heads * head_dim, x_stride) || !strided_ok(tokens, q_heads * head_dim, q_stride))
    return PURO_ERR_SHAPE;
  if (k_rows < 0 || k_rows > kMaxDim || !strided_ok(k_rows, k_heads * head_dim, k_stride)) return PURO_ERR_SHAPE;
  if (append && !strided_ok(k_rows, k_heads * head_dim, v_stride)) return PURO_ERR_SHAPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return PURO_ERR_VALUE;
  if (tokens == 0 || heads == 0) return PURO_OK;
  const bool keys = k_heads > 0 && k_rows > 0;
  if (!r->table || !x || (q_heads > 0 && (!q || !wq)) || (k_heads > 0 && !wk)) return PURO_ERR_NULL;
  if ((keys && (!k || (append && !v))) || (append && !rows)) return PURO_ERR_NULL;
  if (!aligned16(r->table) || !aligned16(x) || !aligned16(q) || !aligned16(wq) || !aligned16(wk) || !aligned16(k) ||
      !aligned16(v) || !aligned4(r->pos) || !aligned4(rows))
    return PURO_ERR_ALIGN;
  const Rows in[] = {table_rows(r), pos_rows(r, tokens), {x, tokens, heads * head_dim, x_stride},
                     {wq, 1, head_dim, head_dim}, {wk, 1, head_dim, head_dim}, {rows, 1, append ? tokens : 0, tokens, 4}};
  const Rows out[] = {{q, tokens, q_heads * head_dim, q_stride}, {k, k_rows, k_heads * head_dim, k_stride},
                      {v, append ? k_rows : 0, k_heads * head_dim, v_stride}};
  if (any_alias(in, 6, out, 3)) return PURO_ERR_ALIAS;
  if (puro_status d = check_device()) return d;
  puro::RopeArgs a = rope_args(r, x, x_stride, tokens);
  a.heads_q = (int)q_heads;
  a.heads_k = (int)k_heads;
  a.heads_v = (int)v_heads;
  a.wq = wq ? wq : wk;          // the kernel reads both, whichever heads there are
  a.wk = wk ? wk : wq;
  a.eps = eps;
  a.q = q;
  a.qs = q_stride;
  a.k = k;
  a.ks = k_stride;
  a.v = v;
  a.vs = v_stride;
  a.rows = append ? rows : nullptr;
  a.cache_rows = cache_rows;
  return launched(puro::run_rope(a, (int)head_dim, r->layout == PURO_ROPE_INTERLEAVED, (hipStream_t)stream));
}

// Shapes of an attention call; backward adds its strides.
bool attention_shape_ok(const puro_attention_shape *a, bool backward) {
  if (!head_dim_ok(a->head_dim)) return false;
  if (a->q_tokens < 0 || a->q_tokens > kMaxRows || a->k_tokens < 0 || a->k_tokens > kMaxRows) return false;
  if (a->sequences < 1 || a->sequences > (1 << 24) || a->q_heads < 1 || a->k_heads < 1 || a->q_heads > 65536 ||
      a->q_heads % a->k_heads != 0)
    return false;
  // What the runtime takes, fewer than 2^32 threads: forward at most 2 (tokens + 512 sequences) heads, backward a third
  // of the query heads' more for the far queries of first keys; the join of its partials takes any number in strides.
  const int64_t most = backward ? kMaxDim / 4 * 3 : kMaxDim;
  if ((a->q_tokens + 512 * a->sequences) * a->q_heads > most) return false;
  if (backward && (a->k_tokens + 512 * a->sequences) * a->k_heads > most) return false;
  if (a->max_k < 0 || a->window < 0 || a->sinks < 0) return false;
  const int64_t qw = a->q_heads * a->head_dim, kw = a->k_heads * a->head_dim;
  if (!strided_ok(a->q_tokens, qw, a->q_stride) || !strided_ok(a->k_tokens, kw, a->k_stride) ||
      !strided_ok(a->k_tokens, kw, a->v_stride) || !strided_ok(a->q_tokens, qw, a->o_stride))
    return false;
  return !backward || (strided_ok(a->q_tokens, qw, a->dq_stride) && strided_ok(a->k_tokens, kw, a->dk_stride) &&
                       strided_ok(a->k_tokens, kw, a->dv_stride));
}

// A window that reaches every key is none.
puro_attention_shape without_idle_window(puro_attention_shape a) {
  if (a.window >= a.k_tokens) a.window = 0;
  if (a.window == 0) a.sinks = 0;
  if (a.sinks > a.k_tokens) a.sinks = a.k_tokens;
  return a;
}

puro::AttnArgs attention_args(const puro_attention_shape &s, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              const int32_t *q_start, const int32_t *k_start, const int32_t *k_len, void *ws) {
  puro::AttnArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = s.q_stride;
  a.ks = s.k_stride;
  a.vs = s.v_stride;
  a.os = s.o_stride;
  a.q_tokens = (int)s.q_tokens;
  a.k_tokens = (int)s.k_tokens;
  a.sequences = (int)s.sequences;
  a.q_heads = (int)s.q_heads;
  a.k_heads = (int)s.k_heads;
  a.group = (int)(s.q_heads / s.k_heads);
  a.q_start = q_start;
  a.k_start = k_start;
  a.k_len = k_len;
  a.window = (int)s.window;
  a.sinks = (int)s.sinks;
  a.scale = s.scale;
  a.ws = static_cast<float *>(ws);
  return a;
}

bool scale_ok(float s) { return s >= 1e-30f && std::isfinite(s); }      // so that lse / scale stays finite

}  // namespace

extern "C" {

puro_status puro_rope_table(int64_t positions, int64_t rot, double base, puro_rope_scaling scaling, double factor,
                            int64_t trained, float *table, puro_stream_t stream) {
  if (scaling != PURO_ROPE_PLAIN && scaling != PURO_ROPE_LINEAR && scaling != PURO_ROPE_NTK && scaling != PURO_ROPE_YARN)
    return PURO_ERR_MODE;
  if (positions < 0 || positions >= kMaxPositions || rot <= 0 || rot % 16 != 0 || rot > 128) return PURO_ERR_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base)) return PURO_ERR_VALUE;
  if (scaling != PURO_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return PURO_ERR_VALUE;
  if (scaling == PURO_ROPE_YARN && trained <= 0) return PURO_ERR_VALUE;
  if (positions == 0) return PURO_OK;
  if (!table) return PURO_ERR_NULL;
  if (!aligned16(table)) return PURO_ERR_ALIGN;
  if (puro_status d = check_device()) return d;
  return launched(puro::run_rope_table(positions, rot, base, (int)scaling, factor, trained, table, (hipStream_t)stream));
}

puro_status puro_rope(const puro_rotation *r, int inverse, const uint16_t *x, int64_t x_stride, int64_t tokens,
                      int64_t heads, int64_t head_dim, uint16_t *y, int64_t y_stride, puro_stream_t stream) {
  if (puro_status s = rotation_mode(r)) return s;
  if (!heads_ok(tokens, heads, 0, head_dim) || !rotation_shape(r, head_dim)) return PURO_ERR_SHAPE;
  if (!strided_ok(tokens, heads * head_dim, x_stride) || !strided_ok(tokens, heads * head_dim, y_stride))
    return PURO_ERR_SHAPE;
  if (tokens == 0 || heads == 0) return PURO_OK;
  if (!r->table || !x || !y) return PURO_ERR_NULL;
  if (!aligned16(r->table) || !aligned16(x) || !aligned16(y) || !aligned4(r->pos)) return PURO_ERR_ALIGN;
  const Rows in[] = {table_rows(r), pos_rows(r, tokens), {x, tokens, heads * head_dim, x_stride}};
  const Rows out[] = {{y, tokens, heads * head_dim, y_stride}};
  if (any_alias(in, 3, out, 1)) return PURO_ERR_ALIAS;
  if (puro_status d = check_device()) return d;
  puro::RopeArgs a = rope_args(r, x, x_stride, tokens);
  a.heads_q = (int)heads;
  a.sign = inverse ? -1.0f : 1.0f;
  a.q = y;
  a.qs = y_stride;
  return launched(puro::run_rope(a, (int)head_dim, r->layout == PURO_ROPE_INTERLEAVED, (hipStream_t)stream));
}

puro_status puro_qk_norm_rope(const puro_rotation *r, const uint16_t *x, int64_t x_stride, int64_t tokens,
                              int64_t q_heads, int64_t k_heads, int64_t head_dim, const uint16_t *wq,
                              const uint16_t *wk, float eps, uint16_t *q, int64_t q_stride, uint16_t *k,
                              int64_t k_stride, puro_stream_t stream) {
  return norm_rope(r, x, x_stride, tokens, q_heads, k_heads, head_dim, wq, wk, eps, q, q_stride, k, k_stride, false,
                   nullptr, 0, nullptr, 0, stream);
}

puro_status puro_qk_norm_rope_append(const puro_rotation *r, const uint16_t *x, int64_t x_stride, int64_t tokens,
                                     int64_t q_heads, int64_t k_heads, int64_t head_dim, const uint16_t *wq,
                                     const uint16_t *wk, float eps, uint16_t *q, int64_t q_stride, uint16_t *cache_k,
                                     int64_t k_stride, uint16_t *cache_v, int64_t v_stride, const int32_t *rows,
                                     int64_t cache_rows, puro_stream_t stream) {
  return norm_rope(r, x, x_stride, tokens, q_heads, k_heads, head_dim, wq, wk, eps, q, q_stride, cache_k, k_stride, true,
                   cache_v, v_stride, rows, cache_rows, stream);
}

size_t puro_qk_norm_rope_backward_workspace_bytes(int64_t tokens, int64_t head_dim) {
  if (tokens < 0 || tokens > kMaxDim || !head_dim_ok(head_dim)) return 0;
  return (size_t)puro::rope_back_blocks(tokens) * 2 * (size_t)head_dim * 4;
}

puro_status puro_qk_norm_rope_backward(const puro_rotation *r, const uint16_t *dq, int64_t dq_stride,
                                       const uint16_t *dk, int64_t dk_stride, const uint16_t *x, int64_t x_stride,
                                       int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                                       const uint16_t *wq, const uint16_t *wk, float eps, uint16_t *dx,
                                       int64_t dx_stride, float *dwq, float *dwk, void *workspace,
                                       size_t workspace_bytes, puro_stream_t stream) {
  if (puro_status s = rotation_mode(r)) return s;
  if (!heads_ok(tokens, q_heads, k_heads, head_dim) || !rotation_shape(r, head_dim)) return PURO_ERR_SHAPE;
  const int64_t heads = q_heads + k_heads;
  if (!strided_ok(tokens, q_heads * head_dim, dq_stride) || !strided_ok(tokens, k_heads * head_dim, dk_stride) ||
      !strided_ok(tokens, heads * head_dim, x_stride) || !strided_ok(tokens, heads * head_dim, dx_stride))
    return PURO_ERR_SHAPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return PURO_ERR_VALUE;
  const bool some = tokens > 0 && heads > 0;
  if (!dwq || !dwk) return PURO_ERR_NULL;
  if (some && (!r->table || !x || !dx || (q_heads > 0 && (!dq || !wq)) || (k_heads > 0 && (!dk || !wk))))
    return PURO_ERR_NULL;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(x) || !aligned16(wq) || !aligned16(wk) || !aligned16(dx) ||
      !aligned16(dwq) || !aligned16(dwk) || !aligned16(r->table) || !aligned16(workspace) || !aligned4(r->pos))
    return PURO_ERR_ALIGN;
  const size_t need = some ? puro_qk_norm_rope_backward_workspace_bytes(tokens, head_dim) : 0;
  const Rows in[] = {table_rows(r), pos_rows(r, tokens), {x, tokens, heads * head_dim, x_stride},
                     {wq, 1, head_dim, head_dim}, {wk, 1, head_dim, head_dim},
                     {dq, tokens, q_heads * head_dim, dq_stride}, {dk, tokens, k_heads * head_dim, dk_stride}};
  const Rows out[] = {{dx, tokens, heads * head_dim, dx_stride}, {dwq, 1, head_dim, head_dim, 4},
                      {dwk, 1, head_dim, head_dim, 4}, {workspace, 1, (int64_t)need, (int64_t)need, 1}};
  if (any_alias(in, 7, out, 4)) return PURO_ERR_ALIAS;
  if (need > 0 && (!workspace || workspace_bytes < need)) return PURO_ERR_WORKSPACE;
  if (puro_status d = check_device()) return d;
  puro::RopeBackArgs a{};
  a.dq = dq;
  a.dk = dk;
  a.x = x;
  a.dqs = dq_stride;
  a.dks = dk_stride;
  a.xs = x_stride;
  a.tokens = some ? tokens : 0;
  a.heads_q = (int)q_heads;
  a.heads_k = (int)k_heads;
  a.wq = wq ? wq : wk;
  a.wk = wk ? wk : wq;
  a.eps = eps;
  a.table = r->table;
  a.positions = r->positions;
  a.rot = (int)r->rot;
  a.pos = r->pos;
  a.dx = dx;
  a.dxs = dx_stride;
  a.dwq = dwq;
  a.dwk = dwk;
  a.partial = static_cast<float *>(workspace);
  return launched(puro::run_rope_back(a, (int)head_dim, r->layout == PURO_ROPE_INTERLEAVED, (hipStream_t)stream));
}

size_t puro_attention_workspace_bytes(const puro_attention_shape *a) {
  if (!a || !attention_shape_ok(a, false) || a->q_tokens == 0) return 0;
  return puro::plan_attention(without_idle_window(*a)).ws_bytes;
}

size_t puro_attention_backward_workspace_bytes(const puro_attention_shape *a) {
  if (!a || !attention_shape_ok(a, true) || (a->q_tokens == 0 && a->k_tokens == 0)) return 0;
  return puro::attention_backward_ws_bytes(without_idle_window(*a));
}

puro_status puro_attention(const puro_attention_shape *a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                           const int32_t *q_start, const int32_t *k_start, const int32_t *k_len, uint16_t *o,
                           float *lse, void *workspace, size_t workspace_bytes, puro_stream_t stream) {
  if (!a) return PURO_ERR_NULL;
  if (!attention_shape_ok(a, false)) return PURO_ERR_SHAPE;
  if (!scale_ok(a->scale)) return PURO_ERR_VALUE;
  if (a->q_tokens == 0) return PURO_OK;
  if ((q_start == nullptr) != (k_start == nullptr) || (!q_start && a->sequences > 1)) return PURO_ERR_NULL;
  if (!q || !o || (a->k_tokens > 0 && (!k || !v))) return PURO_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(workspace) || !aligned16(lse) ||
      !aligned4(q_start) || !aligned4(k_start) || !aligned4(k_len))
    return PURO_ERR_ALIGN;
  const int64_t qw = a->q_heads * a->head_dim, kw = a->k_heads * a->head_dim, n = a->sequences;
  const puro_attention_shape s = without_idle_window(*a);
  const puro::AttnPlan plan = puro::plan_attention(s);
  const Rows in[] = {{q, a->q_tokens, qw, a->q_stride}, {k, a->k_tokens, kw, a->k_stride},
                     {v, a->k_tokens, kw, a->v_stride}, {q_start, 1, n + 1, n + 1, 4}, {k_start, 1, n + 1, n + 1, 4},
                     {k_len, 1, n, n, 4}};
  const Rows out[] = {{o, a->q_tokens, qw, a->o_stride}, {lse, a->q_heads, a->q_tokens, a->q_tokens, 4},
                      {workspace, 1, (int64_t)plan.ws_bytes, (int64_t)plan.ws_bytes, 1}};
  if (any_alias(in, 6, out, 3)) return PURO_ERR_ALIAS;
  if (plan.ws_bytes > 0 && (!workspace || workspace_bytes < plan.ws_bytes)) return PURO_ERR_WORKSPACE;
  if (puro_status d = check_device()) return d;
  puro::AttnArgs args = attention_args(s, q, k, v, q_start, k_start, k_len, workspace);
  args.o = o;
  args.lse = lse;
  return launched(puro::run_attention(args, (int)a->head_dim, plan, (hipStream_t)stream));
}

puro_status puro_attention_backward(const puro_attention_shape *a, const uint16_t *d_o, const uint16_t *q,
                                    const uint16_t *k, const uint16_t *v, const uint16_t *o, const float *lse,
                                    const int32_t *q_start, const int32_t *k_start, uint16_t *dq, uint16_t *dk,
                                    uint16_t *dv, void *workspace, size_t workspace_bytes, puro_stream_t stream) {
  if (!a) return PURO_ERR_NULL;
  if (!attention_shape_ok(a, true)) return PURO_ERR_SHAPE;
  if (!scale_ok(a->scale)) return PURO_ERR_VALUE;
  if (a->q_tokens == 0 && a->k_tokens == 0) return PURO_OK;
  if ((q_start == nullptr) != (k_start == nullptr) || (!q_start && a->sequences > 1)) return PURO_ERR_NULL;
  if (a->q_tokens > 0 && (!d_o || !q || !o || !lse || !dq)) return PURO_ERR_NULL;
  if (a->k_tokens > 0 && (!k || !v || !dk || !dv)) return PURO_ERR_NULL;
  if (!aligned16(d_o) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned16(workspace) || !aligned16(lse) || !aligned4(q_start) || !aligned4(k_start))
    return PURO_ERR_ALIGN;
  const int64_t qw = a->q_heads * a->head_dim, kw = a->k_heads * a->head_dim, n = a->sequences;
  const puro_attention_shape s = without_idle_window(*a);
  const size_t need = puro::attention_backward_ws_bytes(s);
  const Rows in[] = {{q, a->q_tokens, qw, a->q_stride}, {k, a->k_tokens, kw, a->k_stride},
                     {v, a->k_tokens, kw, a->v_stride}, {q_start, 1, n + 1, n + 1, 4}, {k_start, 1, n + 1, n + 1, 4},
                     {o, a->q_tokens, qw, a->o_stride}, {d_o, a->q_tokens, qw, a->o_stride},
                     {lse, a->q_heads, a->q_tokens, a->q_tokens, 4}};
  const Rows out[] = {{dq, a->q_tokens, qw, a->dq_stride}, {dk, a->k_tokens, kw, a->dk_stride},
                      {dv, a->k_tokens, kw, a->dv_stride}, {workspace, 1, (int64_t)need, (int64_t)need, 1}};
  if (any_alias(in, 8, out, 4)) return PURO_ERR_ALIAS;
  if (need > 0 && (!workspace || workspace_bytes < need)) return PURO_ERR_WORKSPACE;
  if (puro_status d = check_device()) return d;
  puro::AttnArgs args = attention_args(s, q, k, v, q_start, k_start, nullptr, workspace);
  args.o = const_cast<uint16_t *>(o);
  args.lse = const_cast<float *>(lse);
  args.d_o = d_o;
  args.dq = dq;
  args.dk = dk;
  args.dv = dv;
  args.dqs = a->dq_stride;
  args.dks = a->dk_stride;
  args.dvs = a->dv_stride;
  return launched(puro::run_attention_backward(args, (int)a->head_dim, (hipStream_t)stream));
}

}  // extern "C"
