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

// A wave holds 512 / D tokens of one head, 8 values a lane: lane t * D / 8 + u
// has values 8u .. 8u + 7 of token t, so that neighbouring lanes read and
// write neighbouring pieces of 16 bytes. (In the order of V's codes in the
// page, neighbouring lanes at neighbouring tokens: 323 us for 296.)
template <int D>
struct WaveTile {
  static constexpr int kTok = 512 / D, kPieces = D / 8;
};

// A lane's place in its token's page: the page's address (null: the token has
// none), and offsets into a head's block of its code word and scale byte.
template <int D>
struct Place {
  uint8_t* page;
  uint32_t k_code, v_code, k_scale, v_scale;
};

template <int D>
__device__ __forceinline__ Place<D> place_of(const Pool& p, Token tok, int u) {
  const InPage in = page_of(p, tok);
  const uint32_t off = in.off;
  Place<D> at;
  at.page = in.page;
  const uint32_t codes = p.page * (D / 2);
  at.k_code = off * (D / 2) + u * 4;
  at.v_code = codes + (off >> 2) * (2 * D) + u * 16 + (off & 3) * 4;
  at.k_scale = 2 * codes + off * (D / 32) + (u >> 2);
  at.v_scale = 2 * codes + p.page * (D / 32) + (u >> 2) * p.page + off;
  return at;
}

// Writes a lane's 8 values of one head; a non-finite one anywhere in the head
// makes the whole head vector NaN. Every lane of the wave must call it; block
// == null: nothing is written.
template <int D>
__device__ __forceinline__ void put8(const float (&x)[8], int t, int u, uint8_t* block, uint32_t code,
                                     uint32_t scale) {
  float m = 0.f, z = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
  for (int e = 0; e < 8; ++e) z += x[e] * 0.f;  // NaN where any is not finite (fmax drops a NaN)
  m = fmaxf(m, __shfl_xor(m, 1));
  m = fmaxf(m, __shfl_xor(m, 2));
  uint32_t sb = scale_byte(m);
  uint32_t w = encode8(x, scale_value(sb));
  const uint64_t odd = __ballot(!(z == 0.f));
  if (odd != 0) {
    constexpr uint64_t kLanes = (1ull << WaveTile<D>::kPieces) - 1;  // of a token
    if (odd >> (t * WaveTile<D>::kPieces) & kLanes) sb = kScaleNan, w = 0;
  }
  if (block == nullptr) return;
  *reinterpret_cast<uint32_t*>(block + code) = w;
  if ((u & 3) == 0) block[scale] = (uint8_t)sb;
}

// A lane's 8 values as they lie in memory. bf16 rows are read past the
// caches' replacement (a lane's two halves of fp32 are half lines each).
template <bool F32>
struct Words {
  uint32_t w[F32 ? 8 : 4];
};

template <bool F32>
__device__ __forceinline__ Words<F32> load_words(const void* p, int64_t i) {
  Words<F32> x;
  if constexpr (F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    const uint4 a = q[0], b = q[1];
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w, x.w[4] = b.x, x.w[5] = b.y, x.w[6] = b.z, x.w[7] = b.w;
  } else {
    const u32x4_t a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(static_cast<const u16*>(p) + i));
#pragma unroll
    for (int e = 0; e < 4; ++e) x.w[e] = a[e];
  }
  return x;
}

template <bool F32>
__device__ __forceinline__ void values_of(const Words<F32>& x, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if constexpr (F32)
      v[e] = __uint_as_float(x.w[e]);
    else
      v[e] = __uint_as_float(e & 1 ? x.w[e >> 1] & 0xffff0000u : x.w[e >> 1] << 16);
}

// Each wave walks over the heads of its tokens: queries (rotated, written in
// their own type), keys (rotated, quantised) and values (quantised), the next
// head on its way meanwhile. Bound by HBM for prompts (64k tokens of 32 + 8 + 8
// heads of 128 in bf16: 253 us, 5.6 TB/s), by latency for single tokens (there
// every wave has one head). Of the half layout a lane gets its partners from
// the lane that holds them.
template <int D, bool F32>
__global__ __launch_bounds__(kCacheThreads) void append_kernel(AppendLaunch a, int lanes) {
  constexpr int kTok = WaveTile<D>::kTok;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kCacheWaves + (threadIdx.x >> 6);
  int h = (int)(wave % lanes);
  const int t = lane / WaveTile<D>::kPieces, u = lane % WaveTile<D>::kPieces;
  const int64_t n64 = wave / lanes * kTok + t;
  const bool live = n64 < a.pool.tokens;
  const int n = live ? (int)n64 : a.pool.tokens - 1;
  const int nq = a.q.heads, nk = a.k.heads, all = nq + 2 * nk;
  const int i = u * 8;
  auto load = [&](int h) {
    if (h < nq) return load_words<F32>(a.q.p, n * a.q.ts + h * a.q.hs + i);
    if (h < nq + nk) return load_words<F32>(a.k.p, n * a.k.ts + (h - nq) * a.k.hs + i);
    return load_words<F32>(a.v.p, n * a.v.ts + (h - nq - nk) * a.v.hs + i);
  };
  if (h >= all) return;
  Words<F32> next = load(h);
  const Token tok = find_token(a.pool, n);
  const RopeArgs& rope = a.rope;
  const int half = rope.rot >> 1;
  const bool turned = i < rope.rot;
  const bool upper = !rope.interleaved && i >= half;
  // The lane of the 8 values that the lane's are paired with: itself where
  // neighbours are.
  const int mate = lane + (!turned || rope.interleaved ? 0 : upper ? -(half / 8) : half / 8);
  float c[8], s[8];
  if (turned) {
    const int pos = a.positions ? a.positions[n] : tok.idx;
    if (rope.interleaved) {
      float cc[4], ss[4];
      load_cs<4>(rope, pos, i / 2, cc, ss);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = cc[e], s[e] = ss[e];
    } else {
      load_cs<8>(rope, pos, upper ? i - half : i, c, s);
      // y = x c -+ x' s of the halves: the sign goes to s
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = upper ? s[e] : -s[e];
    }
  }
  const Place<D> pl = place_of<D>(a.pool, live ? tok : Token{0, -1}, u);
  const int64_t block = head_block_bytes(a.pool.page, D);
  for (; h < all; h += lanes) {
    const Words<F32> now = next;
    if (h + lanes < all) next = load(h + lanes);
    float v[8];
    values_of<F32>(now, v);
    if (h < nq + nk && rope.rot > 0) {
      if (rope.interleaved) {
        if (turned) {
#pragma unroll
          for (int e = 0; e < 4; ++e) turn(v[2 * e], v[2 * e + 1], c[e], s[e], &v[2 * e], &v[2 * e + 1]);
        }
      } else {
        Words<F32> other;
#pragma unroll
        for (int e = 0; e < (F32 ? 8 : 4); ++e) other.w[e] = __shfl(now.w[e], mate);
        if (turned) {
          float w[8];
          values_of<F32>(other, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = turn_half(v[e], w[e], c[e], s[e]);
        }
      }
    }
    if (h < nq) {
      if (live) {
        const int64_t to = n * a.qo.ts + h * a.qo.hs + i;
        if constexpr (F32)
          store8<true>(a.qo.p, to, v);
        else
          stream_store<false>(a.qo.p, to, v);
      }
    } else {
      const bool is_v = h >= nq + nk;
      put8<D>(v, t, u, pl.page ? pl.page + (h - nq - (is_v ? nk : 0)) * block : nullptr,
              is_v ? pl.v_code : pl.k_code, is_v ? pl.v_scale : pl.k_scale);
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
  const int64_t n64 = wave / lanes * kTok + lane / WaveTile<D>::kPieces;
  const int u = lane % WaveTile<D>::kPieces;
  if (n64 >= a.pool.tokens) return;
  const int n = (int)n64;
  const Token tok = find_token(a.pool, n);
  const Place<D> pl = place_of<D>(a.pool, tok, u);
  const int64_t block = head_block_bytes(a.pool.page, D);
  const int nk = a.k.heads;
  for (int h = h0; h < 2 * nk; h += lanes) {
    const bool is_v = h >= nk;
    const int hh = is_v ? h - nk : h;
    float v[8] = {};
    if (pl.page != nullptr) {
      const uint8_t* from = pl.page + hh * block;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(from + (is_v ? pl.v_code : pl.k_code));
      const uint32_t sb = from[is_v ? pl.v_scale : pl.k_scale];
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
    void* p = is_v ? a.v.p : a.k.p;
    const int64_t to = is_v ? n * a.v.ts + hh * a.v.hs + u * 8 : n * a.k.ts + hh * a.k.hs + u * 8;
    if constexpr (F32)
      store8<true>(p, to, v);
    else
      stream_store<false>(p, to, v);
  }
}

// Waves side by side over the heads of a token group; each walks over the
// heads a stride apart with the table's row and the token's place it has
// loaded. Four (a workgroup) where there are tokens enough to fill the chip:
// 64k tokens of 32 + 8 + 8 heads of 128 in bf16 are appended and read back in
// 325 us with 2, 306 with 4, 311 with 8 and 355 with 16.
int head_lanes(int64_t groups, int heads) {
  int lanes = heads;
  while (lanes > 4 && groups * ((lanes + 1) / 2) >= 256 * 32) lanes = (lanes + 1) / 2;
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
