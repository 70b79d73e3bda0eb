// C ABI of the operators around and beside a decoder block: norms, linear
// attention, the AdamW step. Argument checking and launches; the contract of
// every entry point is in include/ttt.h.
#include <algorithm>
#include <cmath>
#include <utility>
#include <vector>

#include "ttt_block.h"
#include "ttt_check.h"

namespace {

ttt_status check_dtype(int32_t d, const char* name) {
  if (d != TTT_BF16 && d != TTT_F32)
    return fail(TTT_ERR_INVALID_ARG, std::string(name) + " must be TTT_BF16 or TTT_F32");
  return TTT_OK;
}

int64_t size_of(int32_t dtype) { return dtype == TTT_F32 ? 4 : 2; }

// Inputs and outputs of a call, checked against each other.
struct Reaches {
  std::vector<Reach> in, out;
  ttt_status check() const {
    for (size_t i = 0; i < out.size(); ++i) {
      for (const Reach& x : in) TTT_TRY(check_apart(out[i], x, false));
      for (size_t j = 0; j < i; ++j) TTT_TRY(check_apart(out[i], out[j], false));
    }
    return TTT_OK;
  }
};

ttt_status check_workspace(void* workspace, size_t bytes, size_t need) {
  if (need == 0) return TTT_OK;
  TTT_TRY(check_ptr(workspace, "workspace", 256));
  if (bytes < need)
    return fail(TTT_ERR_WORKSPACE, "workspace has " + std::to_string(bytes) + " bytes, " +
                                       std::to_string(need) + " are needed");
  return TTT_OK;
}

// ------------------------------------------------------------------ norms

ttt_status check_norm(const ttt_norm* n, tttk::NormLaunch* a) {
  if (n == nullptr) return fail(TTT_ERR_INVALID_ARG, "norm is NULL");
  if (n->reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved fields must be 0");
  if (n->flags & ~(uint32_t)(TTT_NORM_POST | TTT_NORM_PRE))
    return fail(TTT_ERR_INVALID_ARG, "unknown flag bits");
  TTT_TRY(check_tokens(n->rows, n->act_dtype));
  TTT_TRY(check_dtype(n->res_dtype, "res_dtype"));
  TTT_TRY(check_dtype(n->weight_dtype, "weight_dtype"));
  if (n->act_dtype == TTT_F32 && n->res_dtype != TTT_F32)
    return fail(TTT_ERR_UNSUPPORTED, "fp32 rows need an fp32 residual");
  if (n->d < 1) return fail(TTT_ERR_INVALID_ARG, "d must be >= 1");
  if (n->d % 8 != 0 || n->d > 16384)
    return fail(TTT_ERR_UNSUPPORTED, "d must be a multiple of 8, at most 16384");
  if (n->gates < 0) return fail(TTT_ERR_INVALID_ARG, "gates must be >= 0");
  if (n->gates > 0 && n->rows % n->gates != 0)
    return fail(TTT_ERR_INVALID_ARG, "rows must be a multiple of gates");
  if (!std::isfinite(n->scale)) return fail(TTT_ERR_INVALID_ARG, "scale must be finite");
  if (!std::isfinite(n->eps) || n->eps < 0.f)
    return fail(TTT_ERR_INVALID_ARG, "eps must be finite and >= 0");
  a->rows = n->rows, a->d = n->d, a->per_gate = n->gates > 0 ? n->rows / n->gates : 0;
  a->scale = n->scale, a->eps = n->eps;
  a->norm_post = (n->flags & TTT_NORM_POST) != 0, a->norm_pre = (n->flags & TTT_NORM_PRE) != 0;
  a->act_f32 = n->act_dtype == TTT_F32, a->res_f32 = n->res_dtype == TTT_F32;
  a->w_f32 = n->weight_dtype == TTT_F32;
  return TTT_OK;
}

ttt_status check_row(const ttt_rows* r, const char* name, int64_t rows, int64_t d, int32_t dtype, bool out) {
  TTT_TRY(check_rows(r, name, rows, d, dtype == TTT_F32, out));
  if (r->heads != 1) return fail(TTT_ERR_INVALID_ARG, std::string(name) + " must have one head");
  return TTT_OK;
}

// What forward and backward take alike: f with its weight and gate, and pre.
ttt_status check_block(const ttt_norm* n, const ttt_rows* f, const void* post, const void* pre,
                       const ttt_rows* gate, tttk::NormLaunch* a, Reaches* all) {
  const int64_t size = size_of(n->act_dtype), w = n->d * size_of(n->weight_dtype);
  if (f == nullptr && (gate != nullptr || a->norm_post))
    return fail(TTT_ERR_INVALID_ARG, "a gate and a norm behind the block need f");
  if ((gate != nullptr) != (n->gates > 0)) return fail(TTT_ERR_INVALID_ARG, "gate and gates go together");
  if ((post != nullptr && !a->norm_post) || (pre != nullptr && !a->norm_pre))
    return fail(TTT_ERR_INVALID_ARG, "a weight without its norm");
  if (f == nullptr && !a->norm_pre) return fail(TTT_ERR_INVALID_ARG, "nothing to compute");
  if (f != nullptr) {
    TTT_TRY(check_row(f, "f", n->rows, n->d, n->act_dtype, false));
    a->f = to_rows(f);
    if (n->rows > 0) all->in.push_back(reach_of("f", *f, n->rows, n->d, size));
  }
  if (gate != nullptr) {
    TTT_TRY(check_row(gate, "gate", n->gates, n->d, n->act_dtype, false));
    a->gate = to_rows(gate);
    all->in.push_back(reach_of("gate", *gate, n->gates, n->d, size));
  }
  if (post != nullptr) {
    TTT_TRY(check_ptr(post, "post", 16));
    all->in.push_back(reach_of("post", post, w));
  }
  if (pre != nullptr) {
    TTT_TRY(check_ptr(pre, "pre", 16));
    all->in.push_back(reach_of("pre", pre, w));
  }
  a->post = post, a->pre = pre;
  return TTT_OK;
}

// The backward's workspace: the workgroups' sums.
struct NormParts {
  size_t post, pre, gate;
  size_t all() const { return post + pre + gate; }
};
NormParts norm_parts(const ttt_norm* n) {
  const tttk::NormPlan p = tttk::norm_plan(n->rows, n->d, n->gates > 0 ? n->rows / n->gates : 0);
  const size_t one = align256((size_t)p.groups * n->d * 4);
  return {(n->flags & TTT_NORM_POST) ? one : 0, (n->flags & TTT_NORM_PRE) ? one : 0,
          n->gates > 0 && p.slices > 1 ? one : 0};
}

// -------------------------------------------------------- linear attention

ttt_status check_linear(const ttt_linear* l, tttk::LinearLaunch* a) {
  if (l == nullptr) return fail(TTT_ERR_INVALID_ARG, "linear is NULL");
  if (l->reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved fields must be 0");
  TTT_TRY(check_tokens(l->tokens, l->act_dtype));
  if (l->batch < 1) return fail(TTT_ERR_INVALID_ARG, "batch must be >= 1");
  if (l->batch > 65535) return fail(TTT_ERR_UNSUPPORTED, "batch above 65535");
  if (l->kv_heads < 1 || l->q_heads < 1) return fail(TTT_ERR_INVALID_ARG, "heads must be >= 1");
  if (l->kv_heads > kMaxHeads || l->q_heads > kMaxHeads)
    return fail(TTT_ERR_UNSUPPORTED, "heads above 1024");
  if (l->q_heads % l->kv_heads != 0)
    return fail(TTT_ERR_INVALID_ARG, "q heads must be a multiple of kv heads");
  for (const int32_t d : {l->dim_k, l->dim_v}) {
    if (d < 1) return fail(TTT_ERR_INVALID_ARG, "dim_k and dim_v must be >= 1");
    if (d != 64 && d != 128 && d != 256)
      return fail(TTT_ERR_UNSUPPORTED, "dim_k and dim_v must be 64, 128 or 256");
  }
  if ((int64_t)l->batch * l->kv_heads > (int64_t)1 << 22)
    return fail(TTT_ERR_UNSUPPORTED, "batch * kv heads above 2^22");
  if (l->max_new < 1) return fail(TTT_ERR_INVALID_ARG, "max_new must be >= 1");
  if (l->max_new > kMaxTokens) return fail(TTT_ERR_UNSUPPORTED, "max_new above 2^24");
  if (!std::isfinite(l->scale)) return fail(TTT_ERR_INVALID_ARG, "scale must be finite");
  if (l->q_starts == nullptr && l->tokens % l->batch != 0)
    return fail(TTT_ERR_INVALID_ARG, "without q_starts, tokens must be a multiple of batch");
  a->log_decay = l->log_decay, a->starts = l->q_starts;
  a->batch = l->batch, a->tokens = l->tokens, a->max_new = l->max_new, a->kv_heads = l->kv_heads;
  a->dk = l->dim_k, a->dv = l->dim_v, a->scale = l->scale, a->f32 = l->act_dtype == TTT_F32;
  return TTT_OK;
}

size_t state_bytes(const tttk::LinearLaunch& a) {
  return (size_t)a.batch * a.kv_heads * a.dk * a.dv * 4;
}

// Bytes of the states before every part; 0 where there is one.
size_t part_bytes(const tttk::LinearLaunch& a) { return a.parts > 1 ? align256(state_bytes(a) * a.parts) : 0; }

ttt_status check_linear_tables(const ttt_linear* l, Reaches* all) {
  TTT_TRY(check_ptr(l->log_decay, "log_decay", 4));
  all->in.push_back(reach_of("log_decay", l->log_decay, (size_t)l->kv_heads * 4));
  if (l->q_starts != nullptr) {
    TTT_TRY(check_ptr(l->q_starts, "q_starts", 4));
    all->in.push_back(reach_of("q_starts", l->q_starts, (size_t)(l->batch + 1) * 4));
  }
  return TTT_OK;
}

ttt_status check_heads(const ttt_rows* r, const char* name, const ttt_linear* l, int32_t heads, int32_t dim,
                       bool out, Reaches* all) {
  TTT_TRY(check_rows(r, name, l->tokens, dim, l->act_dtype == TTT_F32, out));
  if (r->heads != heads)
    return fail(TTT_ERR_INVALID_ARG, std::string(name) + " must have " + std::to_string(heads) + " heads");
  if (l->tokens > 0)
    (out ? all->out : all->in).push_back(reach_of(name, *r, l->tokens, dim, size_of(l->act_dtype)));
  return TTT_OK;
}

// ------------------------------------------------------------------- AdamW

constexpr int64_t kMaxValues = (int64_t)1 << 40;
int64_t padded(int64_t n) { return (n + tttk::kStateBlock - 1) / tttk::kStateBlock * tttk::kStateBlock; }

ttt_status check_sizes(int64_t n) {
  if (n < 0) return fail(TTT_ERR_INVALID_ARG, "a tensor's size must be >= 0");
  if (n > kMaxValues) return fail(TTT_ERR_UNSUPPORTED, "a tensor above 2^40 values");
  return TTT_OK;
}

ttt_status check_bits(int32_t bits) {
  if (bits != 8 && bits != 32) return fail(TTT_ERR_INVALID_ARG, "bits must be 8 or 32");
  return TTT_OK;
}

size_t adamw_bytes(int64_t total, int32_t bits) {
  return bits == 32 ? (size_t)total * 8 : (size_t)total * 2 + (size_t)(total / tttk::kStateBlock) * 8;
}

}  // namespace

extern "C" {

ttt_status ttt_block_norm(const ttt_norm* norm, const ttt_rows* x, const ttt_rows* f, const void* post,
                          const void* pre, const ttt_rows* gate, const ttt_rows* r, const ttt_rows* h,
                          void* stream) {
  TTT_ENTRY_BEGIN
  tttk::NormLaunch a = {};
  Reaches all;
  TTT_TRY(check_norm(norm, &a));
  TTT_TRY(check_row(x, "x", norm->rows, norm->d, norm->res_dtype, false));
  TTT_TRY(check_block(norm, f, post, pre, gate, &a, &all));
  if ((f != nullptr) != (r != nullptr)) return fail(TTT_ERR_INVALID_ARG, "f and r go together");
  if ((h != nullptr) != a.norm_pre) return fail(TTT_ERR_INVALID_ARG, "h and TTT_NORM_PRE go together");
  const int64_t res = size_of(norm->res_dtype), act = size_of(norm->act_dtype);
  if (r != nullptr) TTT_TRY(check_row(r, "r", norm->rows, norm->d, norm->res_dtype, true));
  if (h != nullptr) TTT_TRY(check_row(h, "h", norm->rows, norm->d, norm->act_dtype, true));
  if (norm->rows == 0) return TTT_OK;
  const Reach xi = reach_of("x", *x, norm->rows, norm->d, res);
  if (r != nullptr) {
    all.out.push_back(reach_of("r", *r, norm->rows, norm->d, res));
    TTT_TRY(check_apart(all.out.back(), xi, true));
  }
  if (h != nullptr) {
    all.out.push_back(reach_of("h", *h, norm->rows, norm->d, act));
    TTT_TRY(check_apart(all.out.back(), xi, false));
  }
  TTT_TRY(all.check());
  a.x = to_rows(x), a.r = to_rows(r), a.h = to_rows(h);
  return launch<tttk::NormLaunch, tttk::launch_norm>("block_norm", a, stream);
  TTT_ENTRY_END
}

ttt_status ttt_block_norm_backward_workspace_size(const ttt_norm* norm, size_t* bytes) {
  TTT_ENTRY_BEGIN
  if (bytes == nullptr) return fail(TTT_ERR_INVALID_ARG, "bytes is NULL");
  tttk::NormLaunch a = {};
  TTT_TRY(check_norm(norm, &a));
  *bytes = norm_parts(norm).all();
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_block_norm_backward(const ttt_norm* norm, const ttt_rows* dr, const ttt_rows* dh,
                                   const ttt_rows* r, const ttt_rows* f, const void* post, const void* pre,
                                   const ttt_rows* gate, const ttt_rows* dx, const ttt_rows* df,
                                   const ttt_rows* dgate, float* dpost, float* dpre, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  TTT_ENTRY_BEGIN
  tttk::NormBackLaunch b = {};
  Reaches all;
  TTT_TRY(check_norm(norm, &b.n));
  TTT_TRY(check_block(norm, f, post, pre, gate, &b.n, &all));
  const int64_t rows = norm->rows, d = norm->d;
  const int64_t res = size_of(norm->res_dtype), act = size_of(norm->act_dtype);
  if ((dh != nullptr) != b.n.norm_pre || (r != nullptr) != b.n.norm_pre)
    return fail(TTT_ERR_INVALID_ARG, "dh, r and TTT_NORM_PRE go together");
  if ((df != nullptr) != (f != nullptr)) return fail(TTT_ERR_INVALID_ARG, "df and f go together");
  if ((dgate != nullptr) != (gate != nullptr)) return fail(TTT_ERR_INVALID_ARG, "dgate and gate go together");
  if ((dpost != nullptr) != (post != nullptr) || (dpre != nullptr) != (pre != nullptr))
    return fail(TTT_ERR_INVALID_ARG, "a weight and its gradient go together");
  if (dr != nullptr) TTT_TRY(check_row(dr, "dr", rows, d, norm->res_dtype, false));
  if (dh != nullptr) TTT_TRY(check_row(dh, "dh", rows, d, norm->act_dtype, false));
  if (r != nullptr) TTT_TRY(check_row(r, "r", rows, d, norm->res_dtype, false));
  TTT_TRY(check_row(dx, "dx", rows, d, norm->res_dtype, true));
  if (df != nullptr) TTT_TRY(check_row(df, "df", rows, d, norm->act_dtype, true));
  const bool each = norm->gates > 0 && norm->gates == rows;  // a gate a row: no sums
  if (dgate != nullptr) {
    TTT_TRY(check_row(dgate, "dgate", norm->gates, d, each ? norm->act_dtype : TTT_F32, true));
    all.out.push_back(reach_of("dgate", *dgate, norm->gates, d, each ? act : 4));
  }
  if (dpost != nullptr) {
    TTT_TRY(check_ptr(dpost, "dpost", 16));
    all.out.push_back(reach_of("dpost", dpost, d * 4));
  }
  if (dpre != nullptr) {
    TTT_TRY(check_ptr(dpre, "dpre", 16));
    all.out.push_back(reach_of("dpre", dpre, d * 4));
  }
  if (rows > 0) {
    if (dh != nullptr) all.in.push_back(reach_of("dh", *dh, rows, d, act));
    if (r != nullptr) all.in.push_back(reach_of("r", *r, rows, d, res));
    if (df != nullptr) all.out.push_back(reach_of("df", *df, rows, d, act));
    all.out.push_back(reach_of("dx", *dx, rows, d, res));
    if (dr != nullptr) {
      const Reach dri = reach_of("dr", *dr, rows, d, res);
      for (const Reach& o : all.out) TTT_TRY(check_apart(o, dri, &o == &all.out.back()));
    }
  }
  const NormParts parts = norm_parts(norm);
  TTT_TRY(check_workspace(workspace, workspace_bytes, parts.all()));
  if (parts.all() > 0) {
    all.out.push_back(reach_of("workspace", workspace, parts.all()));
    if (dr != nullptr && rows > 0) TTT_TRY(check_apart(all.out.back(), reach_of("dr", *dr, rows, d, res), false));
  }
  TTT_TRY(all.check());
  b.n.x = to_rows(r);
  b.dr = to_rows(dr), b.dh = to_rows(dh), b.dx = to_rows(dx), b.df = to_rows(df), b.dgate = to_rows(dgate);
  b.dgate.heads = norm->gates;
  b.dpost = dpost, b.dpre = dpre;
  char* w = static_cast<char*>(workspace);
  b.part_post = reinterpret_cast<float*>(w);
  b.part_pre = reinterpret_cast<float*>(w + parts.post);
  b.part_gate = reinterpret_cast<float*>(w + parts.post + parts.pre);
  if (rows > 0)
    TTT_TRY((launch<tttk::NormBackLaunch, tttk::launch_norm_backward>("block_norm_backward", b, stream)));
  const bool sums = dpost != nullptr || dpre != nullptr || parts.gate > 0 || (dgate != nullptr && rows == 0);
  if (sums) TTT_TRY((launch<tttk::NormBackLaunch, tttk::launch_norm_sums>("block_norm_sums", b, stream)));
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_linear_attention_workspace_size(const ttt_linear* linear, size_t* bytes) {
  TTT_ENTRY_BEGIN
  if (bytes == nullptr) return fail(TTT_ERR_INVALID_ARG, "bytes is NULL");
  tttk::LinearLaunch a = {};
  TTT_TRY(check_linear(linear, &a));
  tttk::linear_parts(&a, false);
  *bytes = tttk::linear_by_token(a) ? 0 : part_bytes(a);
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_linear_attention(const ttt_linear* linear, const ttt_rows* q, const ttt_rows* k,
                                const ttt_rows* v, const ttt_rows* o, float* state, void* workspace,
                                size_t workspace_bytes, void* stream) {
  TTT_ENTRY_BEGIN
  tttk::LinearLaunch a = {};
  Reaches all;
  TTT_TRY(check_linear(linear, &a));
  TTT_TRY(check_linear_tables(linear, &all));
  TTT_TRY(check_heads(q, "q", linear, linear->q_heads, a.dk, false, &all));
  TTT_TRY(check_heads(k, "k", linear, linear->kv_heads, a.dk, false, &all));
  TTT_TRY(check_heads(v, "v", linear, linear->kv_heads, a.dv, false, &all));
  TTT_TRY(check_heads(o, "o", linear, linear->q_heads, a.dv, true, &all));
  if (state != nullptr) {
    TTT_TRY(check_ptr(state, "state", 16));
    all.out.push_back(reach_of("state", state, state_bytes(a)));
  }
  if (a.tokens == 0) return TTT_OK;
  tttk::linear_parts(&a, false);
  const size_t need = tttk::linear_by_token(a) ? 0 : part_bytes(a);
  TTT_TRY(check_workspace(workspace, workspace_bytes, need));
  if (need > 0) all.out.push_back(reach_of("workspace", workspace, need));
  TTT_TRY(all.check());
  a.q = to_rows(q), a.k = to_rows(k), a.v = to_rows(v), a.o = to_rows(o);
  a.first = state, a.last = state, a.sums = static_cast<float*>(workspace);
  return launch<tttk::LinearLaunch, tttk::launch_linear>("linear_attention", a, stream);
  TTT_ENTRY_END
}

ttt_status ttt_linear_attention_backward_workspace_size(const ttt_linear* linear, size_t* bytes) {
  TTT_ENTRY_BEGIN
  if (bytes == nullptr) return fail(TTT_ERR_INVALID_ARG, "bytes is NULL");
  tttk::LinearLaunch a = {};
  TTT_TRY(check_linear(linear, &a));
  tttk::linear_parts(&a, true);
  *bytes = 2 * part_bytes(a);
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_linear_attention_backward(const ttt_linear* linear, const ttt_rows* d_o, const ttt_rows* q,
                                         const ttt_rows* k, const ttt_rows* v, const float* state,
                                         const float* d_state, const ttt_rows* dq, const ttt_rows* dk,
                                         const ttt_rows* dv, float* d_state0, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  TTT_ENTRY_BEGIN
  tttk::LinearBackLaunch b = {};
  tttk::LinearLaunch& a = b.f;
  Reaches all;
  TTT_TRY(check_linear(linear, &a));
  TTT_TRY(check_linear_tables(linear, &all));
  TTT_TRY(check_heads(d_o, "d_o", linear, linear->q_heads, a.dv, false, &all));
  TTT_TRY(check_heads(q, "q", linear, linear->q_heads, a.dk, false, &all));
  TTT_TRY(check_heads(k, "k", linear, linear->kv_heads, a.dk, false, &all));
  TTT_TRY(check_heads(v, "v", linear, linear->kv_heads, a.dv, false, &all));
  TTT_TRY(check_heads(dq, "dq", linear, linear->q_heads, a.dk, true, &all));
  TTT_TRY(check_heads(dk, "dk", linear, linear->kv_heads, a.dk, true, &all));
  TTT_TRY(check_heads(dv, "dv", linear, linear->kv_heads, a.dv, true, &all));
  if (state != nullptr) {
    TTT_TRY(check_ptr(state, "state", 16));
    all.in.push_back(reach_of("state", state, state_bytes(a)));
  }
  if (d_state != nullptr) {
    TTT_TRY(check_ptr(d_state, "d_state", 16));
    if (d_state != d_state0) all.in.push_back(reach_of("d_state", d_state, state_bytes(a)));
  }
  if (d_state0 != nullptr) {
    TTT_TRY(check_ptr(d_state0, "d_state0", 16));
    all.out.push_back(reach_of("d_state0", d_state0, state_bytes(a)));
  }
  tttk::linear_parts(&a, true);
  const size_t need = a.tokens > 0 ? part_bytes(a) : 0;
  TTT_TRY(check_workspace(workspace, workspace_bytes, 2 * need));
  if (need > 0) all.out.push_back(reach_of("workspace", workspace, 2 * need));
  TTT_TRY(all.check());
  a.q = to_rows(q), a.k = to_rows(k), a.v = to_rows(v);
  b.d_o = to_rows(d_o), b.dq = to_rows(dq), b.dk = to_rows(dk), b.dv = to_rows(dv);
  a.first = state, b.d_last = d_state, b.d_first = d_state0;
  a.sums = static_cast<float*>(workspace);
  b.back_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + need);
  if (a.tokens == 0) {  // no row: the state's gradient goes through
    if (d_state0 == nullptr) return TTT_OK;
    return launch<tttk::LinearBackLaunch, tttk::launch_linear_through>("linear_attention_backward", b, stream);
  }
  return launch<tttk::LinearBackLaunch, tttk::launch_linear_backward>("linear_attention_backward", b, stream);
  TTT_ENTRY_END
}

ttt_status ttt_adamw_state_size(const int64_t* sizes, int32_t n, int32_t bits, size_t* bytes) {
  TTT_ENTRY_BEGIN
  if (bytes == nullptr) return fail(TTT_ERR_INVALID_ARG, "bytes is NULL");
  if (n < 0 || (n > 0 && sizes == nullptr)) return fail(TTT_ERR_INVALID_ARG, "n sizes are needed, n >= 0");
  TTT_TRY(check_bits(bits));
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    TTT_TRY(check_sizes(sizes[i]));
    total += padded(sizes[i]);
    if (total > kMaxValues) return fail(TTT_ERR_UNSUPPORTED, "tensors above 2^40 values together");
  }
  *bytes = adamw_bytes(total, bits);
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_adamw_step(const ttt_adamw* adamw, const ttt_param* params, int32_t n, void* state,
                          size_t state_bytes, void* stream) {
  TTT_ENTRY_BEGIN
  if (adamw == nullptr) return fail(TTT_ERR_INVALID_ARG, "adamw is NULL");
  const ttt_adamw& h = *adamw;
  TTT_TRY(check_dtype(h.param_dtype, "param_dtype"));
  TTT_TRY(check_dtype(h.grad_dtype, "grad_dtype"));
  TTT_TRY(check_bits(h.bits));
  if (n < 0 || (n > 0 && params == nullptr)) return fail(TTT_ERR_INVALID_ARG, "n params are needed, n >= 0");
  if (h.step_device == nullptr && h.step < 1) return fail(TTT_ERR_INVALID_ARG, "step must be >= 1");
  for (const double x : {h.lr, h.eps, h.weight_decay, h.max_norm})
    if (!std::isfinite(x) || x < 0.0)
      return fail(TTT_ERR_INVALID_ARG, "lr, eps, weight_decay and max_norm must be finite and >= 0");
  for (const double x : {h.beta1, h.beta2})
    if (!(x >= 0.0 && x < 1.0)) return fail(TTT_ERR_INVALID_ARG, "betas must lie in [0, 1)");
  if (h.norm != nullptr) {
    TTT_TRY(check_ptr(h.norm, "norm", 4));
    if (!(h.max_norm > 0.0)) return fail(TTT_ERR_INVALID_ARG, "max_norm must be > 0 with norm");
  }
  if (h.lr_device != nullptr) TTT_TRY(check_ptr(h.lr_device, "lr_device", 4));
  if (h.step_device != nullptr) TTT_TRY(check_ptr(h.step_device, "step_device", 4));

  const int64_t ps = size_of(h.param_dtype), gs = size_of(h.grad_dtype);
  int64_t total = 0;
  // what is written, and everything: sorted, what is written may meet nothing
  struct Span {
    uintptr_t lo, hi;
    const char* name;
    bool out;
  };
  std::vector<Span> spans;
  spans.reserve((size_t)n * 3 + 4);
  auto span = [&](const char* name, const void* p, int64_t bytes, bool out) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    spans.push_back({lo, lo + (uintptr_t)bytes, name, out});
  };
  bool master = false, plain = false;
  for (int32_t i = 0; i < n; ++i) {
    const ttt_param& t = params[i];
    TTT_TRY(check_sizes(t.n));
    total += padded(t.n);
    if (total > kMaxValues) return fail(TTT_ERR_UNSUPPORTED, "tensors above 2^40 values together");
    if (t.n == 0) continue;
    TTT_TRY(check_ptr(t.p, "p", 16));
    TTT_TRY(check_ptr(t.g, "g", 16));
    span("p", t.p, t.n * ps, true);
    span("g", t.g, t.n * gs, false);
    if (t.master != nullptr) {
      if (h.param_dtype != TTT_BF16) return fail(TTT_ERR_INVALID_ARG, "only bf16 tensors have masters");
      TTT_TRY(check_ptr(t.master, "master", 16));
      span("master", t.master, t.n * 4, true);
      master = true;
    } else {
      plain = true;
    }
  }
  if (master && plain) return fail(TTT_ERR_INVALID_ARG, "masters are given for all tensors or for none");
  if (total == 0) return TTT_OK;
  const size_t need = adamw_bytes(total, h.bits);
  TTT_TRY(check_ptr(state, "state", 256));
  if (state_bytes < need)
    return fail(TTT_ERR_WORKSPACE, "state has " + std::to_string(state_bytes) + " bytes, " +
                                       std::to_string(need) + " are needed");
  span("state", state, (int64_t)need, true);
  if (h.norm != nullptr) span("norm", h.norm, 4, false);
  if (h.lr_device != nullptr) span("lr_device", h.lr_device, 4, false);
  if (h.step_device != nullptr) span("step_device", h.step_device, 4, false);
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  const Span *far = nullptr, *far_out = nullptr;  // of those before, the one that reaches furthest
  for (const Span& s : spans) {
    const Span* met = s.out ? far : far_out;
    if (met != nullptr && met->hi > s.lo)
      return fail(TTT_ERR_ALIAS, std::string(met->name) + " overlaps " + s.name);
    if (far == nullptr || s.hi > far->hi) far = &s;
    if (s.out && (far_out == nullptr || s.hi > far_out->hi)) far_out = &s;
  }

  tttk::StepLaunch a = {};
  char* w = static_cast<char*>(state);
  a.m = w;
  if (h.bits == 32) {
    a.v = w + total * 4;
  } else {
    a.v = w + total;
    a.m_scale = reinterpret_cast<float*>(w + total * 2);
    a.v_scale = a.m_scale + total / tttk::kStateBlock;
  }
  a.b1 = (float)h.beta1, a.b2 = (float)h.beta2, a.c1 = (float)(1.0 - h.beta1), a.c2 = (float)(1.0 - h.beta2);
  a.eps = (float)h.eps, a.lr = (float)h.lr, a.wd = (float)h.weight_decay;
  const bool dev = h.lr_device != nullptr || h.step_device != nullptr;
  const int step = std::max(h.step, 1);
  const double f1 = 1.0 / (1.0 - std::pow(h.beta1, step)), f2 = 1.0 / std::sqrt(1.0 - std::pow(h.beta2, step));
  a.a = (float)(dev ? f1 : h.lr * f1);
  a.k = (float)(1.0 - h.lr * h.weight_decay);
  a.rs = (float)f2;
  a.ln1 = (float)std::log(h.beta1), a.ln2 = (float)std::log(h.beta2);
  a.max_norm = (float)h.max_norm;
  a.norm = h.norm, a.lr_dev = h.lr_device, a.step_dev = h.step_device;
  int64_t off = 0;
  int32_t i = 0;
  while (i < n) {
    // as many tensors as one launch takes
    a.count = 0;
    int64_t chunks = 0;
    for (; i < n && a.count < tttk::kStepTensors; ++i) {
      const ttt_param& t = params[i];
      if (t.n == 0) continue;
      const int64_t c = (t.n + tttk::kStepChunk - 1) / tttk::kStepChunk;  // (2^29 of them at most)
      a.t[a.count] = {t.p, t.master, t.g, t.n, off};
      a.first[a.count++] = (int)chunks;
      chunks += c;
      off += padded(t.n);
    }
    if (a.count == 0) break;
    a.first[a.count] = (int)chunks;
    const tttk::StepCall c = {&a, h.param_dtype == TTT_F32, h.grad_dtype == TTT_F32, master, h.bits == 8};
    TTT_TRY((launch<tttk::StepCall, tttk::launch_adamw>("adamw_step", c, stream)));
  }
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_adamw_read(const void* state, int64_t N, int32_t out_dtype, void* m, void* v, void* stream) {
  TTT_ENTRY_BEGIN
  TTT_TRY(check_dtype(out_dtype, "out_dtype"));
  TTT_TRY(check_sizes(N));
  if (N % tttk::kStateBlock != 0) return fail(TTT_ERR_INVALID_ARG, "N must be a multiple of 256");
  if (N == 0) return TTT_OK;
  TTT_TRY(check_ptr(state, "state", 256));
  TTT_TRY(check_ptr(m, "m", 16));
  TTT_TRY(check_ptr(v, "v", 16));
  const int64_t out = N * size_of(out_dtype);
  Reaches all;
  all.in = {reach_of("state", state, adamw_bytes(N, 8))};
  all.out = {reach_of("m", m, out), reach_of("v", v, out)};
  TTT_TRY(all.check());
  const char* w = static_cast<const char*>(state);
  const float* scales = reinterpret_cast<const float*>(w + 2 * N);
  const tttk::StateRead a = {w, w + N, scales, scales + N / tttk::kStateBlock, m, v, N, out_dtype == TTT_F32};
  return launch<tttk::StateRead, tttk::launch_state_read>("adamw_read", a, stream);
  TTT_ENTRY_END
}

ttt_status ttt_grad_norm_workspace_size(int32_t n, size_t* bytes) {
  TTT_ENTRY_BEGIN
  if (bytes == nullptr) return fail(TTT_ERR_INVALID_ARG, "bytes is NULL");
  if (n < 0) return fail(TTT_ERR_INVALID_ARG, "n must be >= 0");
  const int64_t launches = std::max(1, (n + tttk::kNormTensors - 1) / tttk::kNormTensors);
  *bytes = align256((size_t)launches * tttk::kNormGroups * sizeof(double));
  return TTT_OK;
  TTT_ENTRY_END
}

ttt_status ttt_grad_norm(const void* const* grads, const int64_t* sizes, int32_t n, int32_t grad_dtype,
                         float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  TTT_ENTRY_BEGIN
  TTT_TRY(check_dtype(grad_dtype, "grad_dtype"));
  if (n < 0 || (n > 0 && (grads == nullptr || sizes == nullptr)))
    return fail(TTT_ERR_INVALID_ARG, "n grads and sizes are needed, n >= 0");
  TTT_TRY(check_ptr(norm, "norm", 4));
  size_t need = 0;
  TTT_TRY(ttt_grad_norm_workspace_size(n, &need));
  TTT_TRY(check_workspace(workspace, workspace_bytes, need));
  const Reach ws = reach_of("workspace", workspace, need), no = reach_of("norm", norm, 4);
  TTT_TRY(check_apart(ws, no, false));
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    TTT_TRY(check_sizes(sizes[i]));
    total += sizes[i];
    if (total > kMaxValues) return fail(TTT_ERR_UNSUPPORTED, "tensors above 2^40 values together");
    if (sizes[i] == 0) continue;
    TTT_TRY(check_ptr(grads[i], "grad", 16));
    const Reach g = reach_of("grad", grads[i], sizes[i] * size_of(grad_dtype));
    TTT_TRY(check_apart(ws, g, false));
    TTT_TRY(check_apart(no, g, false));
  }
  tttk::GradNormLaunch a = {};
  const tttk::GradNormCall call = {&a, grad_dtype == TTT_F32};
  double* part = static_cast<double*>(workspace);
  int64_t parts = 0;
  for (int32_t i = 0; i < n;) {
    a.count = 0;
    int64_t chunks = 0;
    for (; i < n && a.count < tttk::kNormTensors; ++i) {
      if (sizes[i] == 0) continue;
      const int64_t c = (sizes[i] + tttk::kNormChunk - 1) / tttk::kNormChunk;
      a.g[a.count] = grads[i], a.n[a.count] = sizes[i];
      a.first[a.count++] = (int)chunks;
      chunks += c;
    }
    if (a.count == 0) break;
    a.first[a.count] = (int)chunks;
    a.part = part + parts;
    TTT_TRY((launch<tttk::GradNormCall, tttk::launch_grad_norm>("grad_norm", call, stream)));
    parts += tttk::kNormGroups;
  }
  const tttk::GradNormJoin join = {part, parts, norm};
  return launch<tttk::GradNormJoin, tttk::launch_grad_norm_join>("grad_norm_join", join, stream);
  TTT_ENTRY_END
}

}  // extern "C"
