// Argument checks that the C ABI's files for the operators of a decoder block
// share, and the launch that the optional per-launch timing sees. Each file
// includes it once; everything here is internal to that file.
#pragma once
#include "ttt.h"

#include <hip/hip_runtime.h>

#include <string>

#include "ttt_serve.h"

// Defined in ttt_api.cpp: the thread-local error record, and a launch that
// the optional per-launch timing sees.
namespace tttk_api {
ttt_status set_error(ttt_status s, const std::string& msg);
hipError_t timed_launch(const char* name, hipStream_t s,
                        hipError_t (*launch)(const void*, hipStream_t), const void* args);
}  // namespace tttk_api

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 24;   // rows of one call
constexpr int kMaxHeads = 1024, kMaxRopeDim = 1024;

ttt_status fail(ttt_status s, const std::string& msg) { return tttk_api::set_error(s, msg); }

#define TTT_TRY(expr)                 \
  do {                                \
    ttt_status _s = (expr);           \
    if (_s != TTT_OK) return _s;      \
  } while (0)

// No exception leaves an entry point (the messages allocate).
#define TTT_ENTRY_BEGIN try {
#define TTT_ENTRY_END                      \
  }                                        \
  catch (...) {                            \
    return TTT_ERR_HIP;                    \
  }

template <class A, hipError_t (*F)(const A&, hipStream_t)>
ttt_status launch(const char* name, const A& a, void* stream) {
  const hipError_t e = tttk_api::timed_launch(
      name, static_cast<hipStream_t>(stream),
      [](const void* p, hipStream_t s) { return F(*static_cast<const A*>(p), s); }, &a);
  return e == hipSuccess ? TTT_OK : fail(TTT_ERR_HIP, std::string(name) + ": " + hipGetErrorString(e));
}

ttt_status check_ptr(const void* p, const char* name, size_t align) {
  if (p == nullptr) return fail(TTT_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return fail(TTT_ERR_INVALID_ARG,
                std::string(name) + " is not " + std::to_string(align) + "-byte aligned");
  return TTT_OK;
}

ttt_status check_tokens(int64_t tokens, int32_t act_dtype) {
  if (act_dtype != TTT_BF16 && act_dtype != TTT_F32)
    return fail(TTT_ERR_INVALID_ARG, "act_dtype must be TTT_BF16 or TTT_F32");
  if (tokens < 0) return fail(TTT_ERR_INVALID_ARG, "tokens must be >= 0");
  if (tokens > kMaxTokens) return fail(TTT_ERR_UNSUPPORTED, "tokens above 2^24");
  return TTT_OK;
}

// The bytes a view reaches, first to one past the last.
struct Reach {
  const char* name;
  uintptr_t lo, hi;
  bool rows;                    // a view of rows (else a plain buffer)
  int64_t ts, hs, row;          // bytes: strides, and one head's values
  int64_t heads, tokens;
};

Reach reach_of(const char* name, const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {name, lo, lo + bytes, false, 0, 0, 0, 0, 0};
}

Reach reach_of(const char* name, const ttt_rows& r, int64_t tokens, int64_t dim, int64_t size) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(r.data);
  const int64_t last = ((tokens - 1) * r.token_stride + (r.heads - 1) * r.head_stride + dim) * size;
  return {name, lo, lo + (uintptr_t)last, true, r.token_stride * size, r.head_stride * size,
          dim * size, r.heads, tokens};
}

bool same_view(const Reach& a, const Reach& b) {
  return a.rows && b.rows && a.lo == b.lo && a.ts == b.ts && a.hs == b.hs && a.heads == b.heads;
}

// Whether two views can share a byte. Views of one buffer that repeat with
// the same period (the parts of a fused projection: same token stride; or
// head-major parts: same head stride) are compared within the period.
bool meet(const Reach& a, const Reach& b) {
  if (a.hi <= b.lo || b.hi <= a.lo) return false;
  if (!a.rows || !b.rows) return true;
  auto apart = [](uintptr_t alo, uintptr_t blo, int64_t period, int64_t aspan, int64_t bspan) {
    if (period <= 0 || aspan > period || bspan > period) return false;
    int64_t off = (int64_t)(blo - alo) % period;
    if (off < 0) off += period;
    return off >= aspan && off + bspan <= period;
  };
  const int64_t ah = (a.heads - 1) * a.hs + a.row, bh = (b.heads - 1) * b.hs + b.row;
  if (a.ts == b.ts && apart(a.lo, b.lo, a.ts, ah, bh)) return false;
  const int64_t at = (a.tokens - 1) * a.ts + a.row, bt = (b.tokens - 1) * b.ts + b.row;
  if (a.hs == b.hs && apart(a.lo, b.lo, a.hs, at, bt)) return false;
  return true;
}

ttt_status check_apart(const Reach& out, const Reach& other, bool may_be_same) {
  if (may_be_same && same_view(out, other)) return TTT_OK;
  if (meet(out, other))
    return fail(TTT_ERR_ALIAS, std::string(out.name) + " overlaps " + other.name);
  return TTT_OK;
}

ttt_status check_rows(const ttt_rows* r, const char* name, int64_t tokens, int64_t dim, bool f32,
                      bool out) {
  if (r == nullptr) return fail(TTT_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (r->reserved != 0) return fail(TTT_ERR_INVALID_ARG, "reserved fields must be 0");
  if (r->heads < 1) return fail(TTT_ERR_INVALID_ARG, std::string(name) + ": heads must be >= 1");
  if (r->heads > kMaxHeads)
    return fail(TTT_ERR_UNSUPPORTED, std::string(name) + ": heads above 1024");
  if (tokens > 0) TTT_TRY(check_ptr(r->data, name, 16));
  const int64_t granule = f32 ? 4 : 8;
  const int64_t most = (int64_t)1 << 40;
  if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride > most || r->head_stride > most)
    return fail(TTT_ERR_INVALID_ARG, std::string(name) + ": strides must lie in [0, 2^40]");
  if (r->token_stride % granule != 0 || r->head_stride % granule != 0)
    return fail(TTT_ERR_INVALID_ARG,
                std::string(name) + ": strides must keep every head 16-byte aligned");
  if (out) {
    const int64_t heads = (r->heads - 1) * r->head_stride + dim;
    const int64_t rows = (tokens - 1) * r->token_stride + dim;
    const bool inner_h = (r->heads == 1 || r->head_stride >= dim) &&
                         (tokens <= 1 || r->token_stride >= heads);
    const bool inner_t = (tokens <= 1 || r->token_stride >= dim) &&
                         (r->heads == 1 || r->head_stride >= rows);
    if (!inner_h && !inner_t)
      return fail(TTT_ERR_ALIAS, std::string(name) + " overlaps itself: its strides are too small");
  }
  return TTT_OK;
}

tttk::Rows to_rows(const ttt_rows* r) {
  if (r == nullptr) return {nullptr, 0, 0, 0};
  return {r->data, r->token_stride, r->head_stride, r->heads};
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace
