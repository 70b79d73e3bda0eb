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

// cos and sin of the 8 pairs i .. i + 7 of position `pos`; NaN for a position
// that the table does not hold.
__device__ __forceinline__ void load_cs8(const RopeArgs& r, int pos, int i, float (&c)[8],
                                         float (&s)[8]) {
  if ((uint32_t)pos < (uint32_t)r.max_pos) {
    const float4* t = reinterpret_cast<const float4*>(r.table + ((int64_t)pos * (r.rot >> 1) + i) * 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 a = t[e];
      c[2 * e] = a.x, s[2 * e] = r.sign * a.y, c[2 * e + 1] = a.z, s[2 * e + 1] = r.sign * a.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = s[e] = __builtin_nanf("");
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

// Where new token n belongs: its sequence, and its index among the
// sequence's tokens. n is the same for the lanes that ask for it; every lane
// of the wave must call it. A token that no sequence claims gets index -1.
__device__ __forceinline__ void find_token(const Pool& p, int n, int* seq, int* idx) {
  int b;
  if (p.starts == nullptr) {
    const int each = p.tokens / p.batch;
    b = n / each;
    *seq = b;
    *idx = p.lens[b] - each + (n - b * each);
    return;
  }
  // the last b with starts[b] <= n: found by halves
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.starts[mid] <= n) lo = mid; else hi = mid;
  }
  *seq = lo;
  const int end = p.starts[lo + 1];
  *idx = n >= p.starts[lo] && n < end ? p.lens[lo] - end + n : -1;
}

__device__ __forceinline__ int64_t head_block_bytes(int page, int dim) {
  return (int64_t)page * (dim + dim / 16);
}

// The head's block of the page that holds token idx of sequence seq, and the
// token's place in it; null where the sequence has no such page.
__device__ __forceinline__ uint8_t* token_block(const Pool& p, int seq, int idx, int head, int* off) {
  if (idx < 0) return nullptr;
  const int pg = idx / p.page;
  if (pg >= p.max_pages) return nullptr;
  *off = idx - pg * p.page;
  const int id = p.table[(int64_t)seq * p.max_pages + pg];
  if ((uint32_t)id >= (uint32_t)p.n_pages) return nullptr;
  return p.pages + id * p.page_stride + head * head_block_bytes(p.page, p.dim);
}

}  // namespace tttk
