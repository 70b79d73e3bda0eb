// Device helpers shared by the rotary, cache and attention kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_device.h"
#include "ttt_serve.h"

namespace tttk {

// Eight consecutive values as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const u16*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<u16*>(p) + i) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                   pack_bf16(v[6], v[7]));
  }
}

// 16 bytes (W = 8 bf16 or 4 fp32 values) that are read or written once, past
// the caches' replacement: 64k tokens of 40 rotated heads took 220 us so and
// 237 with plain accesses. Only where a wave's accesses fill whole lines: half
// lines written this way cost a read and a write each.
template <bool F32>
constexpr int kWide = F32 ? 4 : 8;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <bool F32>
__device__ __forceinline__ void stream_load(const void* p, int64_t i, float (&v)[kWide<F32>]) {
  const u32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(
      static_cast<const char*>(p) + i * (F32 ? 4 : 2)));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (F32) {
      v[e] = __uint_as_float(w[e]);
    } else {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void stream_store(void* p, int64_t i, const float (&v)[kWide<F32>]) {
  u32x4_t w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (F32)
      w[e] = __float_as_uint(v[e]);
    else
      w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
  }
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(static_cast<char*>(p) + i * (F32 ? 4 : 2)));
}

// cos and sin of the N pairs i .. i + N - 1 (N even) of position `pos`; NaN
// for a position that the table does not hold (selected after a read of its
// first row: branches here kept the arrays from registers).
template <int N>
__device__ __forceinline__ void load_cs(const RopeArgs& r, int pos, int i, float (&c)[N],
                                        float (&s)[N]) {
  const bool in = (uint32_t)pos < (uint32_t)r.max_pos;
  const float4* t = reinterpret_cast<const float4*>(r.table + ((int64_t)(in ? pos : 0) * (r.rot >> 1) + i) * 2);
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    const float4 a = t[e];
    c[2 * e] = in ? a.x : __builtin_nanf(""), s[2 * e] = in ? r.sign * a.y : __builtin_nanf("");
    c[2 * e + 1] = in ? a.z : __builtin_nanf(""), s[2 * e + 1] = in ? r.sign * a.w : __builtin_nanf("");
  }
}

// (a, b) turned by the angle of (c, s): both products are rounded before the
// sum (no contraction), so that what is quantised afterwards does not depend
// on which product a fused operation would have kept exact.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float* ya, float* yb) {
#pragma clang fp contract(off)
  const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
  *ya = ac - bs;
  *yb = bc + as;
}

// One half of it, s with its sign: a c - b s is a c + b (-s) to the bit.
__device__ __forceinline__ float turn_half(float x, float mate, float c, float s) {
#pragma clang fp contract(off)
  const float xc = x * c, ms = mate * s;
  return xc + ms;
}

// Where new token n belongs: its sequence, and its index among the
// sequence's tokens. Lanes may ask for different tokens. One that no sequence
// claims gets index -1.
struct Token {
  int seq, idx;
};
__device__ __forceinline__ Token find_token(const Pool& p, int n) {
  if (p.starts == nullptr) {
    const int each = p.tokens / p.batch;
    const int b = n / each;
    return {b, p.lens[b] - each + (n - b * each)};
  }
  // the last b with starts[b] <= n: found by halves
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.starts[mid] <= n) lo = mid; else hi = mid;
  }
  const int end = p.starts[lo + 1];
  return {lo, n >= p.starts[lo] && n < end ? p.lens[lo] - end + n : -1};
}

__device__ __forceinline__ int64_t head_block_bytes(int page, int dim) {
  return (int64_t)page * (dim + dim / 16);
}

// The page that holds token idx of sequence seq, and the token's place in it;
// null where the sequence has no such page.
struct InPage {
  uint8_t* page;
  int off;
};
__device__ __forceinline__ InPage page_of(const Pool& p, Token t) {
  if (t.idx < 0) return {nullptr, 0};
  const int pg = t.idx / p.page;
  if (pg >= p.max_pages) return {nullptr, 0};
  const int id = p.table[(int64_t)t.seq * p.max_pages + pg];
  if ((uint32_t)id >= (uint32_t)p.n_pages) return {nullptr, 0};
  return {p.pages + id * p.page_stride, t.idx - pg * p.page};
}

}  // namespace tttk
