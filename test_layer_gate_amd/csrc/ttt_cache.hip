// gfx950 kernels of the paged 4-bit cache: new tokens' keys and values go in
// (the keys, and the queries beside them, rotated on the way), and tokens are
// read back.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_fp4.h"
#include "ttt_serve_device.h"

namespace tttk {
namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheWaves = kCacheThreads / 64;

// A wave holds TOK = 512 / D tokens of one head, 8 values a lane: lane t +
// TOK * u has values 8u .. 8u + 7 of token t, so that the four lanes of a
// block sit TOK apart and the lanes of neighbouring tokens next to each
// other, as the V codes lie in the page.
template <int D>
struct WaveTile {
  static constexpr int kTok = 512 / D;
};

// Writes one token-lane's 8 values x (a non-finite one anywhere in the head
// makes the whole head vector NaN). Every lane of the wave must call it;
// block == null: nothing is written.
template <int D, bool V>
__device__ __forceinline__ void put8(const float (&x)[8], int u, int page, uint8_t* block, int off) {
  constexpr int kTok = WaveTile<D>::kTok;
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
  // fmax drops a NaN: find non-finite values by their sum's
  float z = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) z += x[e] * 0.f;
  m = fmaxf(m, __shfl_xor(m, kTok));
  m = fmaxf(m, __shfl_xor(m, 2 * kTok));
#pragma unroll
  for (int o = kTok; o < 64; o <<= 1) z += __shfl_xor(z, o);
  const bool bad = !(z == 0.f);
  const uint32_t sb = bad ? kScaleNan : scale_byte(m);
  const uint32_t w = bad ? 0u : encode8(x, scale_value(sb));
  if (block == nullptr) return;
  const int codes = page * (D / 2);
  if constexpr (!V) {
    *reinterpret_cast<uint32_t*>(block + off * (D / 2) + u * 4) = w;
    if ((u & 3) == 0) block[2 * codes + off * (D / 32) + (u >> 2)] = (uint8_t)sb;
  } else {
    *reinterpret_cast<uint32_t*>(block + codes + (off >> 2) * (2 * D) + u * 16 + (off & 3) * 4) = w;
    if ((u & 3) == 0)
      block[2 * codes + page * (D / 32) + (u >> 2) * page + off] = (uint8_t)sb;
  }
}

// Each wave walks over the heads of its tokens: queries (rotated, written in
// their own type), keys (rotated, quantised) and values (quantised). Bound by
// HBM for prompts, by latency for single tokens (there every wave has one
// head). A lane of a rotated tensor reads its partner's 8 values too, which
// the first level of cache holds from the partner's own read.
template <int D, bool F32>
__global__ __launch_bounds__(kCacheThreads) void append_kernel(AppendLaunch a, int lanes) {
  constexpr int kTok = WaveTile<D>::kTok;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kCacheWaves + (threadIdx.x >> 6);
  const int h0 = (int)(wave % lanes);
  const int64_t n64 = wave / lanes * kTok + (lane % kTok);
  const int u = lane / kTok;
  const bool live = n64 < a.pool.tokens;
  const int n = live ? (int)n64 : a.pool.tokens - 1;
  int seq, idx;
  find_token(a.pool, n, &seq, &idx);
  const RopeArgs& rope = a.rope;
  const int half = rope.rot >> 1;
  const int i = u * 8;
  const bool turned = i < rope.rot;
  const bool upper = !rope.interleaved && i >= half;
  const int mate = !turned || rope.interleaved ? i : upper ? i - half : i + half;
  float c[8], s[8];
  if (turned) {
    const int pos = a.positions ? a.positions[n] : idx;
    if (rope.interleaved) {
      // 4 pairs: 8 floats of the table
      if ((uint32_t)pos < (uint32_t)rope.max_pos) {
        const float4* t = reinterpret_cast<const float4*>(rope.table + (int64_t)pos * rope.rot + i);
        const float4 x = t[0], y = t[1];
        c[0] = x.x, s[0] = x.y, c[1] = x.z, s[1] = x.w;
        c[2] = y.x, s[2] = y.y, c[3] = y.z, s[3] = y.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = s[e] = __builtin_nanf("");
      }
    } else {
      load_cs8(rope, pos, upper ? i - half : i, c, s);
    }
  }
  const int nq = a.q.heads, nk = a.k.heads;
  for (int h = h0; h < nq + 2 * nk; h += lanes) {
    const int kind = h < nq ? 0 : h < nq + nk ? 1 : 2;
    const Rows& x = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int hh = h - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk);
    const int64_t at = n * x.ts + hh * x.hs;
    float v[8];
    load8<F32>(x.p, at + i, v);
    if (kind < 2 && turned) {
      if (rope.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(v[2 * e], v[2 * e + 1], c[e], s[e], &v[2 * e], &v[2 * e + 1]);
      } else {
        float w[8], other;
        load8<F32>(x.p, at + mate, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (upper)
            turn(w[e], v[e], c[e], s[e], &other, &v[e]);
          else
            turn(v[e], w[e], c[e], s[e], &v[e], &other);
        }
      }
    }
    if (kind == 0) {
      if (live) store8<F32>(a.qo.p, n * a.qo.ts + hh * a.qo.hs + i, v);
    } else {
      int off = 0;
      uint8_t* block = live ? token_block(a.pool, seq, idx, hh, &off) : nullptr;
      if (kind == 1)
        put8<D, false>(v, u, a.pool.page, block, off);
      else
        put8<D, true>(v, u, a.pool.page, block, off);
    }
  }
}

// The stored values of the same tokens, in the layout of their rows. A token
// without a page reads as zero.
template <int D, bool F32>
__global__ __launch_bounds__(kCacheThreads) void read_kernel(ReadLaunch a, int lanes) {
  constexpr int kTok = WaveTile<D>::kTok;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kCacheWaves + (threadIdx.x >> 6);
  const int h0 = (int)(wave % lanes);
  const int64_t n64 = wave / lanes * kTok + (lane % kTok);
  const int u = lane / kTok;
  if (n64 >= a.pool.tokens) return;
  const int n = (int)n64;
  int seq, idx;
  find_token(a.pool, n, &seq, &idx);
  const int nk = a.k.heads, page = a.pool.page, codes = page * (D / 2);
  for (int h = h0; h < 2 * nk; h += lanes) {
    const bool is_v = h >= nk;
    const int hh = is_v ? h - nk : h;
    int off = 0;
    const uint8_t* block = token_block(a.pool, seq, idx, hh, &off);
    float v[8] = {};
    if (block != nullptr) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(
          block + (is_v ? codes + (off >> 2) * (2 * D) + u * 16 + (off & 3) * 4
                        : off * (D / 2) + u * 4));
      const uint32_t sb = block[2 * codes + (is_v ? page * (D / 32) + (u >> 2) * page + off
                                                  : off * (D / 32) + (u >> 2))];
      uint32_t d[4];
      decode8(w, scale_value(sb), d);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(d[e] << 16);
        v[2 * e + 1] = __uint_as_float(d[e] & 0xffff0000u);
      }
      if (sb > kScaleMax) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_nanf("");
      }
    }
    const Rows& y = is_v ? a.v : a.k;
    store8<F32>(y.p, n * y.ts + hh * y.hs + u * 8, v);
  }
}

// Waves of a launch over `heads` heads of every token group: each wave walks
// over heads / lanes of them, as many as still leave the chip full of waves
// (the table's row and the token's place are then looked up once for them).
int head_lanes(int64_t groups, int heads) {
  int lanes = heads;
  while (lanes > 1 && groups * ((lanes + 1) / 2) >= 256 * 32) lanes = (lanes + 1) / 2;
  return lanes;
}

}  // namespace

#define TTT_BY_DIM(dim, f32, CALL)              \
  switch (dim) {                                \
    case 64: if (f32) { CALL(64, true); } else { CALL(64, false); } break;    \
    case 128: if (f32) { CALL(128, true); } else { CALL(128, false); } break; \
    default: if (f32) { CALL(256, true); } else { CALL(256, false); } break;  \
  }

hipError_t launch_append(const AppendLaunch& a, hipStream_t s) {
  const int64_t groups = (a.pool.tokens + 512 / a.pool.dim - 1) / (512 / a.pool.dim);
  const int lanes = head_lanes(groups, a.q.heads + 2 * a.k.heads);
  const uint32_t grid = (uint32_t)((groups * lanes + kCacheWaves - 1) / kCacheWaves);
#define TTT_CALL(D, F) append_kernel<D, F><<<grid, kCacheThreads, 0, s>>>(a, lanes)
  TTT_BY_DIM(a.pool.dim, a.f32, TTT_CALL)
#undef TTT_CALL
  return hipGetLastError();
}

hipError_t launch_read(const ReadLaunch& a, hipStream_t s) {
  const int64_t groups = (a.pool.tokens + 512 / a.pool.dim - 1) / (512 / a.pool.dim);
  const int lanes = head_lanes(groups, 2 * a.k.heads);
  const uint32_t grid = (uint32_t)((groups * lanes + kCacheWaves - 1) / kCacheWaves);
#define TTT_CALL(D, F) read_kernel<D, F><<<grid, kCacheThreads, 0, s>>>(a, lanes)
  TTT_BY_DIM(a.pool.dim, a.f32, TTT_CALL)
#undef TTT_CALL
  return hipGetLastError();
}

}  // namespace tttk
