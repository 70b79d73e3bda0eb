// Device helpers of the attention kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_fp4.h"
#include "ttt_serve_device.h"

namespace tttk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -__builtin_huge_valf();

typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// c + a0 b0 + a1 b1 of pairs of bf16.
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a), __builtin_bit_cast(bf16x2_t, b), c, false);
}

struct U4 {
  uint32_t v[4];
};
__device__ __forceinline__ bf16x8_t frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, U4{{a, b, c, d}});
}

// x as T bf16 terms (T = 1: rounded to nearest; T = 3: 24 bits, exact but for
// the last term's rounding), pairs packed.
template <int T>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&w)[T]) {
  w[0] = pack_bf16(x, y);
#pragma unroll
  for (int t = 1; t < T; ++t) {
    x -= __uint_as_float(w[t - 1] << 16);
    y -= __uint_as_float(w[t - 1] & 0xffff0000u);
    w[t] = pack_bf16(x, y);
  }
}

// The value of lane i + 8 of the same 16 (a rotation, row_ror:8).
__device__ __forceinline__ float eight_lanes_on(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xf, 0xf, true));
}

// Bits [a, b) of a word.
__device__ __forceinline__ uint32_t bits_between(int a, int b) {
  a = min(max(a, 0), 32), b = min(max(b, 0), 32);
  const uint32_t below_b = b == 32 ? ~0u : (1u << b) - 1u;
  const uint32_t below_a = a == 32 ? ~0u : (1u << a) - 1u;
  return below_b & ~below_a;
}

// All ones where bit k of w is set.
__device__ __forceinline__ uint32_t spread(uint32_t w, int k) {
  return (uint32_t)__builtin_amdgcn_sbfe((int)w, k, 1);
}
constexpr uint32_t kNanBits = 0x7fc00000u, kNoneBits = 0xff800000u;

// In a block that few waves take: keeps the compiler from running its plain
// arithmetic always and selecting the result, which it does to save a branch
// (the masks of 64 keys were a third of the many-row kernel's vector work).
__device__ __forceinline__ void rare_path() { asm volatile(""); }

// The bytes of four scales that stand for NaN, each as its top bit.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  static_assert(kScaleMax == 252, "bytes from 253 on");
  return ((w & 0x7f7f7f7fu) + 0x03030303u) & w & 0x80808080u;
}

// A word at an address that is the same for the whole wave, of memory that
// the kernel does not write: through the scalar cache, so that a page number
// needed later is not waited for with the vector loads that are under way.
__device__ __forceinline__ int uniform_load(const int32_t* p, int64_t i) {
  typedef const __attribute__((address_space(4))) int32_t* Constant;
  return reinterpret_cast<Constant>(reinterpret_cast<uint64_t>(p))[i];
}

// Loads of an address put together from integers, which has to be marked as
// global memory's.
typedef const __attribute__((address_space(1))) uint8_t* Global;
// ONCE: past the caches' replacement, for what no other wave will read.
template <bool ONCE = false>
__device__ __forceinline__ uint4 load16(Global p) {
  const auto* q = reinterpret_cast<const __attribute__((address_space(1))) u32x4_t*>(p);
  u32x4_t w;
  if constexpr (ONCE)
    w = __builtin_nontemporal_load(q);
  else
    w = *q;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t load4(Global p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) uint32_t*>(p);
}

// n workgroups, numbered along x and then y: a dimension of a launch holds
// less than 2^32 threads. The last of y may have workgroups too many.
inline dim3 grid_of(int64_t n) {
  constexpr int64_t kWidth = (int64_t)1 << 22;
  if (n <= kWidth) return dim3((uint32_t)n);
  return dim3((uint32_t)kWidth, (uint32_t)((n + kWidth - 1) / kWidth));
}
__device__ __forceinline__ int64_t block_of_grid() {
  return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

// Sequence b's rows, its length, and how many of its keys the page table has
// entries for. UNIFORM: b is the same for the whole wave.
struct Seq {
  int row0, news, len, held;
};
template <bool UNIFORM>
__device__ __forceinline__ Seq seq_at(const Pool& p, int b) {
  auto word = [](const int32_t* w, int i) { return UNIFORM ? uniform_load(w, i) : w[i]; };
  const int each = p.tokens / p.batch;
  const int r0 = p.starts ? word(p.starts, b) : b * each;
  const int r1 = p.starts ? word(p.starts, b + 1) : r0 + each;
  Seq s;
  s.row0 = r0;
  s.news = r0 < 0 ? 0 : min(r1, p.tokens) - r0;
  s.len = max(word(p.lens, b), 0);
  s.held = min(s.len, p.max_pages * p.page);
  return s;
}
__device__ __forceinline__ Seq seq_of(const Pool& p, int b) { return seq_at<true>(p, b); }

// The keys that a sequence's new token t sees and that the table has entries
// for: [lo, hi). The token stands where the length puts it, whatever the table
// holds.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span span_of(const AttnLaunch& a, const Seq& q, int t) {
  const int p = q.len - q.news + t;
  Span s;
  s.hi = a.causal ? min(p + 1, q.held) : q.held;
  s.lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
  return s;
}

// Units of keys that a sequence's first `tile` rows see; at least one, so that
// rows that see nothing are written, and none without rows.
__device__ __forceinline__ uint32_t units_of(const AttnLaunch& a, const Seq& s, int tile, int group, int unit) {
  if (s.news <= 0) return 0;
  const Span first = span_of(a, s, 0);
  const Span last = span_of(a, s, (min(tile, s.news * group) - 1) / group);
  return (uint32_t)(max(last.hi - (first.lo & ~31), 1) + unit - 1) / unit;
}

// A slice of the units of all sequences, one after the other: [at, end), which
// begins in sequence b, whose n units begin at `off`; slices are of `per`.
struct Line {
  uint32_t at, end, off, n, per;
  int b;
};
constexpr int kSliceBatch = 256;  // sequences at most: four a lane
__device__ __forceinline__ Line line_of(const AttnLaunch& a, int slice, int tile, int group, int unit,
                                     int lane) {
  uint32_t n[kSliceBatch / 64], sum[kSliceBatch / 64], total = 0;
#pragma unroll
  for (int c = 0; c < kSliceBatch / 64; ++c) {
    n[c] = sum[c] = 0;
    if (c * 64 >= a.pool.batch) continue;
    const int b = c * 64 + lane;
    if (b < a.pool.batch) n[c] = units_of(a, seq_at<false>(a.pool, b), tile, group, unit);
    uint32_t x = n[c];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    sum[c] = total + x;
    total += __builtin_amdgcn_readlane(x, 63);
  }
  Line l = {};
  l.per = (total + a.slices - 1) / a.slices;
  l.at = slice * l.per;
  l.end = min(total, l.at + l.per);
  if (l.at >= total) {
    l.end = l.at;
    return l;
  }
  bool found = false;
#pragma unroll
  for (int c = 0; c < kSliceBatch / 64; ++c) {
    const uint64_t past = __ballot(sum[c] > l.at);
    if (found || past == 0) continue;
    found = true;
    const int i = __builtin_ctzll(past);
    l.b = c * 64 + i;
    l.n = __builtin_amdgcn_readlane(n[c], i);
    l.off = __builtin_amdgcn_readlane(sum[c], i) - l.n;
  }
  return l;
}

}  // namespace tttk
