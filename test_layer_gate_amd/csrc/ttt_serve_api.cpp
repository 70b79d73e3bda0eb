// C ABI of the attention half of a decoder block: rotary positions, the paged
// 4-bit cache and attention over it. Argument checking and launches; the
// contract of every entry point is in include/ttt.h.
#include <cmath>

#include "ttt_check.h"

namespace {

ttt_status check_rope(const ttt_rope* rope, int64_t dim, tttk::RopeArgs* a) {
  if (rope == nullptr) return fail(TTT_ERR_INVALID_ARG, "rope is NULL");
  if (rope->reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved fields must be 0");
  if (rope->flags & ~(uint32_t)TTT_ROPE_INTERLEAVED)
    return fail(TTT_ERR_INVALID_ARG, "unknown flag bits");
  if (rope->rot_dim < 2 || rope->rot_dim > dim)
    return fail(TTT_ERR_INVALID_ARG, "rot_dim must lie in [2, head_dim]");
  if (rope->rot_dim % 16 != 0)
    return fail(TTT_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16");
  if (rope->max_pos < 1) return fail(TTT_ERR_INVALID_ARG, "max_pos must be >= 1");
  TTT_TRY(check_ptr(rope->table, "rope table", 16));
  *a = {rope->table, rope->rot_dim, rope->max_pos, (rope->flags & TTT_ROPE_INTERLEAVED) != 0, 1.f};
  return TTT_OK;
}

size_t rope_bytes(const tttk::RopeArgs& r) { return (size_t)r.max_pos * r.rot * 4; }

ttt_status check_cache(const ttt_cache* c, int64_t tokens, tttk::Pool* p) {
  if (c == nullptr) return fail(TTT_ERR_INVALID_ARG, "cache is NULL");
  if (c->reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved fields must be 0");
  if (c->batch < 1) return fail(TTT_ERR_INVALID_ARG, "batch must be >= 1");
  if (c->batch > 65535) return fail(TTT_ERR_UNSUPPORTED, "batch above 65535");
  if (c->n_pages < 1 || c->max_pages < 1)
    return fail(TTT_ERR_INVALID_ARG, "n_pages and max_pages must be >= 1");
  size_t bytes = 0;
  TTT_TRY(ttt_kv_page_bytes(c->page_size, c->kv_heads, c->head_dim, &bytes));
  if ((int64_t)c->max_pages * c->page_size > tttk::kMaxKeys)
    return fail(TTT_ERR_UNSUPPORTED, "max_pages * page_size above 2^30");
  if (c->page_stride < (int64_t)bytes || c->page_stride % 16 != 0)
    return fail(TTT_ERR_INVALID_ARG,
                "page_stride must be a multiple of 16, at least ttt_kv_page_bytes()");
  if (c->page_stride > (int64_t)1 << 40)
    return fail(TTT_ERR_UNSUPPORTED, "page_stride above 2^40");
  TTT_TRY(check_ptr(c->pages, "pages", 16));
  TTT_TRY(check_ptr(c->page_table, "page_table", 4));
  TTT_TRY(check_ptr(c->kv_lens, "kv_lens", 4));
  if (c->q_starts != nullptr)
    TTT_TRY(check_ptr(c->q_starts, "q_starts", 4));
  else if (tokens % c->batch != 0)
    return fail(TTT_ERR_INVALID_ARG, "without q_starts, tokens must be a multiple of batch");
  *p = {static_cast<uint8_t*>(c->pages), c->page_stride, c->page_table, c->kv_lens, c->q_starts,
        c->batch, c->max_pages, c->n_pages, c->page_size, c->kv_heads, c->head_dim, (int)tokens};
  return TTT_OK;
}

Reach pool_reach(const tttk::Pool& p) {
  return reach_of("pages", p.pages,
                  (size_t)(p.n_pages - 1) * p.page_stride +
                      (size_t)p.heads * p.page * (p.dim + p.dim / 16));
}

// What the kernels read of the tables that stand beside the pool.
ttt_status check_tables_apart(const Reach& out, const tttk::Pool& p, const int32_t* positions) {
  TTT_TRY(check_apart(out, reach_of("page_table", p.table, (size_t)p.batch * p.max_pages * 4), false));
  TTT_TRY(check_apart(out, reach_of("kv_lens", p.lens, (size_t)p.batch * 4), false));
  if (p.starts != nullptr)
    TTT_TRY(check_apart(out, reach_of("q_starts", p.starts, (size_t)(p.batch + 1) * 4), false));
  if (positions != nullptr)
    TTT_TRY(check_apart(out, reach_of("positions", positions, (size_t)p.tokens * 4), false));
  return TTT_OK;
}

ttt_status rope_impl(int32_t tokens, int32_t seq_len, int32_t head_dim, int32_t act_dtype,
                     const ttt_rope* rope, const int32_t* positions, const ttt_rows* q,
                     const ttt_rows* k, const ttt_rows* q_out, const ttt_rows* k_out, float sign,
                     const char* name, void* stream) {
  TTT_TRY(check_tokens(tokens, act_dtype));
  const bool f32 = act_dtype == TTT_F32;
  if (head_dim < 16) return fail(TTT_ERR_INVALID_ARG, "head_dim must be >= 16");
  if (head_dim % 16 != 0 || head_dim > kMaxRopeDim)
    return fail(TTT_ERR_UNSUPPORTED, "head_dim must be a multiple of 16, at most 1024");
  if (positions != nullptr)
    TTT_TRY(check_ptr(positions, "positions", 4));
  else if (seq_len < 1)
    return fail(TTT_ERR_INVALID_ARG, "seq_len must be >= 1 where positions is NULL");
  tttk::RopeLaunch a = {};
  TTT_TRY(check_rope(rope, head_dim, &a.rope));
  TTT_TRY(check_rows(q, "q", tokens, head_dim, f32, false));
  TTT_TRY(check_rows(q_out, "q_out", tokens, head_dim, f32, true));
  if ((k == nullptr) != (k_out == nullptr))
    return fail(TTT_ERR_INVALID_ARG, "k and k_out go together");
  if (k != nullptr) {
    TTT_TRY(check_rows(k, "k", tokens, head_dim, f32, false));
    TTT_TRY(check_rows(k_out, "k_out", tokens, head_dim, f32, true));
  }
  if (q->heads != q_out->heads || (k != nullptr && k->heads != k_out->heads))
    return fail(TTT_ERR_INVALID_ARG, "an output needs its input's heads");
  if (tokens == 0) return TTT_OK;
  const int64_t size = f32 ? 4 : 2;
  const Reach qi = reach_of("q", *q, tokens, head_dim, size);
  const Reach qo = reach_of("q_out", *q_out, tokens, head_dim, size);
  const Reach tab = reach_of("rope table", a.rope.table, rope_bytes(a.rope));
  TTT_TRY(check_apart(qo, qi, true));
  TTT_TRY(check_apart(qo, tab, false));
  if (positions != nullptr)
    TTT_TRY(check_apart(qo, reach_of("positions", positions, (size_t)tokens * 4), false));
  if (k != nullptr) {
    const Reach ki = reach_of("k", *k, tokens, head_dim, size);
    const Reach ko = reach_of("k_out", *k_out, tokens, head_dim, size);
    TTT_TRY(check_apart(ko, ki, true));
    TTT_TRY(check_apart(ko, qi, false));
    TTT_TRY(check_apart(qo, ki, false));
    TTT_TRY(check_apart(ko, qo, false));
    TTT_TRY(check_apart(ko, tab, false));
    if (positions != nullptr)
      TTT_TRY(check_apart(ko, reach_of("positions", positions, (size_t)tokens * 4), false));
  }
  a.x[0] = to_rows(q), a.y[0] = to_rows(q_out);
  a.x[1] = to_rows(k), a.y[1] = to_rows(k_out);
  a.tokens = tokens, a.dim = head_dim, a.seq_len = seq_len > 0 ? seq_len : 1;
  a.positions = positions;
  a.rope.sign = sign;
  a.f32 = f32;
  return launch<tttk::RopeLaunch, tttk::launch_rope>(name, a, stream);
}

struct TableArgs {
  float* table;
  int max_pos, rot, kind;
  double base, factor, orig, lo, hi, mul;
};
hipError_t launch_table(const TableArgs& t, hipStream_t s) {
  return tttk::launch_rope_table(t.table, t.max_pos, t.rot, t.base, t.kind, t.factor, t.orig, t.lo,
                                 t.hi, t.mul, s);
}

ttt_status check_attn(const ttt_attn* at, int32_t batch, int32_t kv_heads, int32_t q_heads) {
  if (at == nullptr) return fail(TTT_ERR_INVALID_ARG, "attn is NULL");
  if (at->reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved fields must be 0");
  if (at->flags & ~(uint32_t)TTT_ATTN_ALL_KEYS)
    return fail(TTT_ERR_INVALID_ARG, "unknown flag bits");
  if (!std::isfinite(at->scale)) return fail(TTT_ERR_INVALID_ARG, "scale must be finite");
  if (at->window < 0) return fail(TTT_ERR_INVALID_ARG, "window must be >= 0");
  if (at->window > 0 && (at->flags & TTT_ATTN_ALL_KEYS))
    return fail(TTT_ERR_INVALID_ARG, "a window needs causal rows");
  if (at->max_new < 1 || at->max_kv < 1)
    return fail(TTT_ERR_INVALID_ARG, "max_new and max_kv must be >= 1");
  if (at->max_new > kMaxTokens) return fail(TTT_ERR_UNSUPPORTED, "max_new above 2^24");
  if (batch < 1 || kv_heads < 1 || q_heads < 1)
    return fail(TTT_ERR_INVALID_ARG, "batch and heads must be >= 1");
  if (kv_heads > kMaxHeads || q_heads > kMaxHeads)
    return fail(TTT_ERR_UNSUPPORTED, "heads above 1024");
  if (q_heads % kv_heads != 0)
    return fail(TTT_ERR_INVALID_ARG, "q heads must be a multiple of kv heads");
  return TTT_OK;
}

// Bytes of the parts' weighted sums, of their maxima and sums, and of where
// the parts of each row are.
struct PartBytes {
  size_t part, ml, of;
  size_t all() const { return part + ml + of; }
};
PartBytes part_bytes(const tttk::AttnPlan& p, int64_t batch, int64_t tokens, int64_t kv_heads, int64_t q_heads,
                     int64_t dim) {
  const size_t rows = p.slices > 0   ? (size_t)(p.slices + batch - 1) * kv_heads * p.tile
                      : p.splits > 1 ? (size_t)p.splits * tokens * q_heads
                                     : 0;
  return {align256(rows * dim * 4), align256(rows * 8), p.slices > 0 ? align256((size_t)tokens * q_heads * 8) : 0};
}

}  // namespace

extern "C" {

ttt_status ttt_rope_table(float* table, int32_t max_pos, int32_t rot_dim, double base,
                          const ttt_rope_scaling* scaling, void* stream) {
  TTT_ENTRY_BEGIN
  TTT_TRY(check_ptr(table, "table", 16));
  if (max_pos < 1) return fail(TTT_ERR_INVALID_ARG, "max_pos must be >= 1");
  if (rot_dim < 2) return fail(TTT_ERR_INVALID_ARG, "rot_dim must be >= 2");
  if (rot_dim % 16 != 0 || rot_dim > kMaxRopeDim)
    return fail(TTT_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16, at most 1024");
  if ((int64_t)max_pos * rot_dim > (int64_t)1 << 32)
    return fail(TTT_ERR_UNSUPPORTED, "max_pos * rot_dim above 2^32");
  if (!std::isfinite(base) || !(base > 1.0))
    return fail(TTT_ERR_INVALID_ARG, "base must be finite and > 1");
  TableArgs t = {table, max_pos, rot_dim, TTT_ROPE_PLAIN, base, 1.0, 1.0, 1.0, 1.0, 1.0};
  if (scaling != nullptr) {
    const ttt_rope_scaling& s = *scaling;
    if (s.reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved fields must be 0");
    if (s.kind < TTT_ROPE_PLAIN || s.kind > TTT_ROPE_BANDS)
      return fail(TTT_ERR_INVALID_ARG, "unknown kind of scaling");
    if (!std::isfinite(s.amplitude) || !(s.amplitude > 0.0))
      return fail(TTT_ERR_INVALID_ARG, "amplitude must be finite and > 0");
    if (s.kind != TTT_ROPE_PLAIN && (!std::isfinite(s.factor) || !(s.factor >= 1.0)))
      return fail(TTT_ERR_INVALID_ARG, "factor must be finite and >= 1");
    if (s.kind == TTT_ROPE_YARN || s.kind == TTT_ROPE_BANDS) {
      if (!std::isfinite(s.original) || !(s.original >= 1.0))
        return fail(TTT_ERR_INVALID_ARG, "original must be finite and >= 1");
      if (!std::isfinite(s.low) || !std::isfinite(s.high) || !(s.low > 0.0) || !(s.high > s.low))
        return fail(TTT_ERR_INVALID_ARG, "0 < low < high is needed");
    }
    t.kind = s.kind, t.factor = s.factor, t.orig = s.original, t.lo = s.low, t.hi = s.high;
    t.mul = s.amplitude;
  }
  return launch<TableArgs, launch_table>("rope_table", t, stream);
  TTT_ENTRY_END
}

ttt_status ttt_rope_forward(int32_t tokens, int32_t seq_len, int32_t head_dim, int32_t act_dtype,
                            const ttt_rope* rope, const int32_t* positions, const ttt_rows* q,
                            const ttt_rows* k, const ttt_rows* q_out, const ttt_rows* k_out,
                            void* stream) {
  TTT_ENTRY_BEGIN
  return rope_impl(tokens, seq_len, head_dim, act_dtype, rope, positions, q, k, q_out, k_out, 1.f,
                   "rope", stream);
  TTT_ENTRY_END
}

ttt_status ttt_rope_backward(int32_t tokens, int32_t seq_len, int32_t head_dim, int32_t act_dtype,
                             const ttt_rope* rope, const int32_t* positions, const ttt_rows* dq_out,
                             const ttt_rows* dk_out, const ttt_rows* dq, const ttt_rows* dk,
                             void* stream) {
  TTT_ENTRY_BEGIN
  return rope_impl(tokens, seq_len, head_dim, act_dtype, rope, positions, dq_out, dk_out, dq, dk,
                   -1.f, "rope_backward", stream);
  TTT_ENTRY_END
}

ttt_status ttt_kv_page_bytes(int32_t page_size, int32_t kv_heads, int32_t head_dim, size_t* bytes) {
  TTT_ENTRY_BEGIN
  if (bytes == nullptr) return fail(TTT_ERR_INVALID_ARG, "bytes is NULL");
  if (page_size < 1 || kv_heads < 1 || head_dim < 1)
    return fail(TTT_ERR_INVALID_ARG, "page_size, kv_heads and head_dim must be >= 1");
  if (page_size % 16 != 0 || page_size > 4096)
    return fail(TTT_ERR_UNSUPPORTED, "page_size must be a multiple of 16, at most 4096");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(TTT_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (kv_heads > kMaxHeads) return fail(TTT_ERR_UNSUPPORTED, "heads above 1024");
  *bytes = (size_t)kv_heads * page_size * (head_dim + head_dim / 16);
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_kv_append(const ttt_cache* cache, int32_t tokens, int32_t act_dtype,
                         const ttt_rows* k, const ttt_rows* v, const ttt_rows* q,
                         const ttt_rows* q_out, const ttt_rope* rope, const int32_t* positions,
                         void* stream) {
  TTT_ENTRY_BEGIN
  TTT_TRY(check_tokens(tokens, act_dtype));
  tttk::AppendLaunch a = {};
  TTT_TRY(check_cache(cache, tokens, &a.pool));
  const int dim = a.pool.dim;
  const bool f32 = act_dtype == TTT_F32;
  TTT_TRY(check_rows(k, "k", tokens, dim, f32, false));
  TTT_TRY(check_rows(v, "v", tokens, dim, f32, false));
  if (k->heads != a.pool.heads || v->heads != a.pool.heads)
    return fail(TTT_ERR_INVALID_ARG, "k and v need the cache's heads");
  if ((q == nullptr) != (q_out == nullptr))
    return fail(TTT_ERR_INVALID_ARG, "q and q_out go together");
  if (q != nullptr) {
    if (rope == nullptr) return fail(TTT_ERR_INVALID_ARG, "q is only taken to be rotated");
    TTT_TRY(check_rows(q, "q", tokens, dim, f32, false));
    TTT_TRY(check_rows(q_out, "q_out", tokens, dim, f32, true));
    if (q->heads != q_out->heads)
      return fail(TTT_ERR_INVALID_ARG, "an output needs its input's heads");
  }
  if (rope != nullptr) TTT_TRY(check_rope(rope, dim, &a.rope));
  if (positions != nullptr) TTT_TRY(check_ptr(positions, "positions", 4));
  if (tokens == 0) return TTT_OK;
  const int64_t size = f32 ? 4 : 2;
  const Reach pool = pool_reach(a.pool);
  const Reach ki = reach_of("k", *k, tokens, dim, size), vi = reach_of("v", *v, tokens, dim, size);
  TTT_TRY(check_apart(pool, ki, false));
  TTT_TRY(check_apart(pool, vi, false));
  TTT_TRY(check_tables_apart(pool, a.pool, positions));
  if (rope != nullptr)
    TTT_TRY(check_apart(pool, reach_of("rope table", a.rope.table, rope_bytes(a.rope)), false));
  if (q != nullptr) {
    const Reach qi = reach_of("q", *q, tokens, dim, size);
    const Reach qo = reach_of("q_out", *q_out, tokens, dim, size);
    TTT_TRY(check_apart(qo, qi, true));
    TTT_TRY(check_apart(qo, ki, false));
    TTT_TRY(check_apart(qo, vi, false));
    TTT_TRY(check_apart(qo, pool, false));
    TTT_TRY(check_apart(pool, qi, false));
    TTT_TRY(check_apart(qo, reach_of("rope table", a.rope.table, rope_bytes(a.rope)), false));
    TTT_TRY(check_tables_apart(qo, a.pool, positions));
  }
  a.q = to_rows(q), a.qo = to_rows(q_out), a.k = to_rows(k), a.v = to_rows(v);
  a.positions = positions;
  a.f32 = f32;
  return launch<tttk::AppendLaunch, tttk::launch_append>("kv_append", a, stream);
  TTT_ENTRY_END
}

ttt_status ttt_kv_read(const ttt_cache* cache, int32_t tokens, int32_t act_dtype,
                       const ttt_rows* k_out, const ttt_rows* v_out, void* stream) {
  TTT_ENTRY_BEGIN
  TTT_TRY(check_tokens(tokens, act_dtype));
  tttk::ReadLaunch a = {};
  TTT_TRY(check_cache(cache, tokens, &a.pool));
  const int dim = a.pool.dim;
  a.f32 = act_dtype == TTT_F32;
  TTT_TRY(check_rows(k_out, "k_out", tokens, dim, a.f32, true));
  TTT_TRY(check_rows(v_out, "v_out", tokens, dim, a.f32, true));
  if (k_out->heads != a.pool.heads || v_out->heads != a.pool.heads)
    return fail(TTT_ERR_INVALID_ARG, "k_out and v_out need the cache's heads");
  if (tokens == 0) return TTT_OK;
  const int64_t size = a.f32 ? 4 : 2;
  const Reach pool = pool_reach(a.pool);
  const Reach ko = reach_of("k_out", *k_out, tokens, dim, size);
  const Reach vo = reach_of("v_out", *v_out, tokens, dim, size);
  TTT_TRY(check_apart(ko, pool, false));
  TTT_TRY(check_apart(vo, pool, false));
  TTT_TRY(check_apart(ko, vo, false));
  TTT_TRY(check_tables_apart(ko, a.pool, nullptr));
  TTT_TRY(check_tables_apart(vo, a.pool, nullptr));
  a.k = to_rows(k_out), a.v = to_rows(v_out);
  return launch<tttk::ReadLaunch, tttk::launch_read>("kv_read", a, stream);
  TTT_ENTRY_END
}

ttt_status ttt_kv_attention_workspace_size(const ttt_attn* attn, int32_t batch, int32_t tokens,
                                           int32_t act_dtype, int32_t kv_heads, int32_t q_heads,
                                           int32_t head_dim, size_t* bytes) {
  TTT_ENTRY_BEGIN
  if (bytes == nullptr) return fail(TTT_ERR_INVALID_ARG, "bytes is NULL");
  TTT_TRY(check_attn(attn, batch, kv_heads, q_heads));
  TTT_TRY(check_tokens(tokens, act_dtype));
  size_t page = 0;
  TTT_TRY(ttt_kv_page_bytes(16, kv_heads, head_dim, &page));
  const tttk::AttnPlan plan = tttk::attn_plan(batch, kv_heads, q_heads, attn->max_new, attn->max_kv,
                                              attn->window, act_dtype == TTT_F32, head_dim);
  *bytes = part_bytes(plan, batch, tokens, kv_heads, q_heads, head_dim).all();
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_kv_attention_plan(const ttt_attn* attn, int32_t batch, int32_t tokens,
                                 int32_t act_dtype, int32_t kv_heads, int32_t q_heads,
                                 int32_t head_dim, ttt_attn_plan* plan) {
  TTT_ENTRY_BEGIN
  if (plan == nullptr) return fail(TTT_ERR_INVALID_ARG, "plan is NULL");
  size_t bytes = 0;
  TTT_TRY(ttt_kv_attention_workspace_size(attn, batch, tokens, act_dtype, kv_heads, q_heads, head_dim,
                                          &bytes));
  const tttk::AttnPlan p = tttk::attn_plan(batch, kv_heads, q_heads, attn->max_new, attn->max_kv,
                                           attn->window, act_dtype == TTT_F32, head_dim);
  tttk::AttnLaunch a = {};
  a.pool.batch = batch, a.pool.heads = kv_heads, a.pool.tokens = tokens, a.q.heads = q_heads;
  a.max_new = attn->max_new;
  a.many = p.many, a.splits = p.splits, a.each = p.each, a.slices = p.slices, a.tile = p.tile;
  a.pool.dim = head_dim, a.f32 = act_dtype == TTT_F32;
  const tttk::AttnGrid g = tttk::attn_grid(a);
  *plan = {p.many, p.many ? tttk::kManyTile : p.tile, p.splits, p.slices, g.waves, 0, g.groups};
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_kv_attention(const ttt_cache* cache, const ttt_attn* attn, int32_t tokens,
                            int32_t act_dtype, const ttt_rows* q, const ttt_rows* o, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  TTT_ENTRY_BEGIN
  TTT_TRY(check_tokens(tokens, act_dtype));
  tttk::AttnLaunch a = {};
  TTT_TRY(check_cache(cache, tokens, &a.pool));
  const int dim = a.pool.dim;
  a.f32 = act_dtype == TTT_F32;
  TTT_TRY(check_rows(q, "q", tokens, dim, a.f32, false));
  TTT_TRY(check_rows(o, "o", tokens, dim, a.f32, true));
  if (q->heads != o->heads)
    return fail(TTT_ERR_INVALID_ARG, "an output needs its input's heads");
  TTT_TRY(check_attn(attn, a.pool.batch, a.pool.heads, q->heads));
  if ((int64_t)tokens * q->heads > (int64_t)1 << 30)
    return fail(TTT_ERR_UNSUPPORTED, "tokens * q heads above 2^30");
  if (lse != nullptr) TTT_TRY(check_ptr(lse, "lse", 4));
  if (tokens == 0) return TTT_OK;
  const tttk::AttnPlan plan = tttk::attn_plan(a.pool.batch, a.pool.heads, q->heads, attn->max_new,
                                              attn->max_kv, attn->window, a.f32, dim);
  a.many = plan.many, a.splits = plan.splits, a.each = plan.each, a.slices = plan.slices, a.tile = plan.tile;
  const PartBytes parts = part_bytes(plan, a.pool.batch, tokens, a.pool.heads, q->heads, dim);
  const size_t need = parts.all();
  const int64_t size = a.f32 ? 4 : 2;
  const Reach pool = pool_reach(a.pool);
  const Reach qi = reach_of("q", *q, tokens, dim, size), oo = reach_of("o", *o, tokens, dim, size);
  if (need > 0) {
    TTT_TRY(check_ptr(workspace, "workspace", 256));
    if (workspace_bytes < need)
      return fail(TTT_ERR_WORKSPACE, "workspace has " + std::to_string(workspace_bytes) +
                                         " bytes, " + std::to_string(need) + " are needed");
    const Reach ws = reach_of("workspace", workspace, need);
    TTT_TRY(check_apart(ws, qi, false));
    TTT_TRY(check_apart(ws, oo, false));
    TTT_TRY(check_apart(ws, pool, false));
    TTT_TRY(check_tables_apart(ws, a.pool, nullptr));
  }
  TTT_TRY(check_apart(oo, qi, false));
  TTT_TRY(check_apart(oo, pool, false));
  TTT_TRY(check_tables_apart(oo, a.pool, nullptr));
  if (lse != nullptr) {
    const Reach le = reach_of("lse", lse, (size_t)tokens * q->heads * 4);
    TTT_TRY(check_apart(le, qi, false));
    TTT_TRY(check_apart(le, oo, false));
    TTT_TRY(check_apart(le, pool, false));
    TTT_TRY(check_tables_apart(le, a.pool, nullptr));
    if (need > 0) TTT_TRY(check_apart(le, reach_of("workspace", workspace, need), false));
  }
  a.q = to_rows(q), a.o = to_rows(o);
  a.lse = lse;
  a.scale = attn->scale;
  a.causal = (attn->flags & TTT_ATTN_ALL_KEYS) == 0;
  a.window = attn->window, a.max_new = attn->max_new, a.max_kv = attn->max_kv;
  a.part = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + parts.part);
  a.part_of = reinterpret_cast<int*>(static_cast<char*>(workspace) + parts.part + parts.ml);
  TTT_TRY((launch<tttk::AttnLaunch, tttk::launch_attention>("kv_attention", a, stream)));
  if (need > 0)
    TTT_TRY((launch<tttk::AttnLaunch, tttk::launch_attention_join>("kv_attention_join", a, stream)));
  return TTT_OK;
  TTT_ENTRY_END
}

}  // extern "C"
