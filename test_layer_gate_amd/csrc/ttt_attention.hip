// gfx950 kernels of attention over the paged 4-bit cache.
//
// Row (t, h) of a sequence stands at position p = len - new + t and sees the
// keys j with max(0, p - window + 1) <= j <= p (causal; else j < len):
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j,
// in one pass over the keys with the running maximum m, sum and weighted sum
// (rescaled whenever m grows).
//
// Codes times their power-of-two scale are exact in bf16, so keys and values
// enter the matrix instructions without a rounding; what is rounded is the
// weights p (to bf16), and, for fp32 rows, nothing: q and p are then three
// bf16 terms each, whose products are all accumulated in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_attention.h"

namespace tttk {
namespace {

// ---------------------------------------------------------------------------
// Few rows. A wave takes 16 rows (query heads of one key head, times tokens)
// and a stretch of the keys, 32 at a time. S^T = K Q^T with 16x16x32: lane
// (i, g) = (lane % 16, lane / 16) brings D / 4 neighbouring values of key i;
// of the result it holds, for row i, keys 4g .. 4g + 3 of either 16. Those
// eight are what the second product O^T = V^T P^T asks of it (the order of
// the contraction is free as long as V agrees), so P goes over without a
// move between lanes. Of V it brings the same eight keys' values
// i D / 16 .. + D / 16 - 1.
constexpr int kFewWaves = 4;

template <int D, int T, bool F32>
__global__ __launch_bounds__(64 * kFewWaves) void attend_few_kernel(AttnLaunch a, int row_tiles) {
  constexpr int NB = D / 64;        // 16-byte pieces (D = 64: half a piece) of K per lane
  constexpr int KS = D / 32;        // steps of the first product
  constexpr int F = D / 16;         // V fragments = values per lane
  __shared__ float red_o[kFewWaves - 1][16][D + 4];
  __shared__ float red_ml[kFewWaves][16][2];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, g = lane >> 4;
  const int b = blockIdx.z, split = blockIdx.x;
  const int hk = blockIdx.y % a.pool.heads;
  const int group = a.q.heads / a.pool.heads;
  const int page = a.pool.page, gpp = page >> 4;  // 16-key pieces a page

  const Seq seq = seq_of(a.pool, b);
  if (seq.news <= 0) return;
  const int row0 = seq.row0, news = seq.news, len = seq.len;
  const int rows = news * group;

  for (int tile = blockIdx.y / a.pool.heads; tile * 16 < rows; tile += row_tiles) {
    const int r = tile * 16 + i16;
    const bool live = r < rows;
    const int t = min(r, rows - 1) / group;
    const int head = hk * group + min(r, rows - 1) % group;
    const Span sp = span_of(a, len, news, t);
    // the tile's keys, and this split's part of them
    const Span first = span_of(a, len, news, tile * 16 / group);
    const Span last = span_of(a, len, news, min(tile * 16 + 15, rows - 1) / group);
    const int lo = first.lo & ~31, hi = last.hi;
    const int all_lo = last.lo, all_hi = first.hi;  // keys that every row sees
    int each = max(128 * kFewWaves / 4, (hi - lo + a.splits - 1) / a.splits);
    each = (each + 127) & ~127;
    const int s0 = lo + split * each, s1 = min(hi, s0 + each);
    const int per = ((s1 - s0 + kFewWaves - 1) / kFewWaves + 31) & ~31;
    const int k0 = s0 + wave * per, k1 = min(s1, k0 + per);

    // Q as the first product's B operand: step s, values (D / 4) g + 8 s ..
    uint32_t qf[T][KS][4];
    {
      const int64_t at = (int64_t)(row0 + t) * a.q.ts + head * a.q.hs + g * (D / 4);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float v[8];
        load8<F32>(a.q.p, at + 8 * s, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[T];
          split2<T>(live ? v[2 * e] : 0.f, live ? v[2 * e + 1] : 0.f, w);
#pragma unroll
          for (int x = 0; x < T; ++x) qf[x][s][e] = w[x];
        }
      }
    }
    f32x4_t o[F];
#pragma unroll
    for (int f = 0; f < F; ++f) o[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m = kNone, l = 0.f;
    const float sc = a.scale * kLog2e;

    for (int base = k0; base < k1; base += 1024) {
      // Where the next 64 pieces of 16 keys lie: one a lane.
      int64_t my_block = -1;
      int my_off = 0;
      {
        const int piece = (base >> 4) + lane;
        const int pg = piece / gpp;
        if (pg < a.pool.max_pages && piece * 16 < k1) {
          const int id = a.pool.table[(int64_t)b * a.pool.max_pages + pg];
          if ((uint32_t)id < (uint32_t)a.pool.n_pages) {
            my_block = id * a.pool.page_stride + hk * head_block_bytes(page, D);
            my_off = (piece - pg * gpp) * 16;
          }
        }
      }
      const int stop = min(k1, base + 1024);
      for (int j = base; j < stop; j += 32) {
        uint32_t kw[2][KS], ks[2][NB], vw[2][4][D == 256 ? 2 : 1], vs[2];
        bool have[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int src = ((j - base) >> 4) + x;
          const int64_t blk = __shfl(my_block, src);
          have[x] = blk >= 0;
          const uint8_t* bp = a.pool.pages + (have[x] ? blk : 0);
          const int off = have[x] ? __shfl(my_off, src) : 0;
          const uint8_t* kc = bp + (off + i16) * (D / 2) + g * (D / 8);
          const uint8_t* vc = bp + page * (D / 2) + ((off >> 2) + g) * (2 * D) +
                              (D == 64 ? (i16 >> 1) * 16 : i16 * (D / 8));
          const uint8_t* kp = bp + page * D + (off + i16) * (D / 32);
          const uint8_t* vp = bp + page * D + page * (D / 32) + (i16 * (D / 16) / 32) * page + off + 4 * g;
          if constexpr (D == 64) {
            const uint2 w = *reinterpret_cast<const uint2*>(kc);
            kw[x][0] = w.x, kw[x][1] = w.y;
            ks[x][0] = kp[g >> 1];
          } else {
#pragma unroll
            for (int p = 0; p < D / 128; ++p) {
              const uint4 w = reinterpret_cast<const uint4*>(kc)[p];
              kw[x][4 * p] = w.x, kw[x][4 * p + 1] = w.y, kw[x][4 * p + 2] = w.z, kw[x][4 * p + 3] = w.w;
              ks[x][p] = kp[g * (D / 128) + p];
            }
          }
#pragma unroll
          for (int p = 0; p < (D == 256 ? 2 : 1); ++p) {
            const uint4 w = reinterpret_cast<const uint4*>(vc)[p];
            vw[x][0][p] = w.x, vw[x][1][p] = w.y, vw[x][2][p] = w.z, vw[x][3][p] = w.w;
          }
          vs[x] = *reinterpret_cast<const uint32_t*>(vp);
        }
        // S^T
        f32x4_t s[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          s[x] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < KS; ++q) {
            uint32_t d[4];
            decode8(kw[x][q], scale_value(ks[x][D == 256 ? q >> 2 : 0]), d);
            const bf16x8_t kf = frag(d[0], d[1], d[2], d[3]);
#pragma unroll
            for (int y = T - 1; y >= 0; --y)
              s[x] = mfma16(kf, frag(qf[y][q][0], qf[y][q][1], qf[y][q][2], qf[y][q][3]), s[x]);
          }
        }
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = s[e >> 2][e & 3] * sc;
        // Keys that some row does not see, that have no page, or that hold NaN
        bool odd = j < all_lo || j + 32 > all_hi || !have[0] || !have[1];
        {
          uint32_t nan = 0;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int q = 0; q < (D == 256 ? 2 : 1); ++q) nan |= ks[x][q] > kScaleMax;
            static_assert(kScaleMax == 252, "bytes from 253 on");
            nan |= ((vs[x] & 0x7f7f7f7fu) + 0x03030303u) & vs[x] & 0x80808080u;
          }
          odd = odd || __any(nan != 0);
        }
        uint32_t poison = 0;  // this row's keys whose value is NaN
        if (odd) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint64_t kn = __ballot(ks[x][0] > kScaleMax);
            kn |= kn >> 32;
            kn |= kn >> 16;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = j + 16 * x + 4 * g + e;
              const bool seen = have[x] && key >= sp.lo && key < sp.hi;
              const uint32_t vb = (vs[x] >> (8 * e)) & 255u;
              float& pe = p[4 * x + e];
              pe = !seen ? kNone : (kn >> (4 * g + e)) & 1 ? __builtin_nanf("") : pe;
              // A NaN value must not reach the rows that do not see it (0 * NaN):
              // it goes out of V, and into the weight of those that do.
              if (seen && vb > kScaleMax) poison |= 1u << (4 * x + e);
              if (!have[x] || vb > kScaleMax) {
                vs[x] = (vs[x] & ~(255u << (8 * e))) | (127u << (8 * e));
#pragma unroll
                for (int q = 0; q < (D == 256 ? 2 : 1); ++q) vw[x][e][q] = 0;
              }
            }
          }
        }
        // running maximum over the tile's keys of this row
        float mx = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])),
                         fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, mx);
        const float m0 = mn == kNone ? 0.f : mn;
        const float al = __builtin_amdgcn_exp2f(m - m0);
        m = mn;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = __builtin_amdgcn_exp2f(p[e] - m0);
          sum += p[e];
        }
        l = l * al + sum;
        if (odd) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (poison >> e & 1) p[e] = __builtin_nanf("");
        }
        if (__any(al != 1.f)) {
#pragma unroll
          for (int f = 0; f < F; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[f][e] *= al;
        }
        uint32_t pw[T][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[T];
          split2<T>(p[2 * e], p[2 * e + 1], w);
#pragma unroll
          for (int x = 0; x < T; ++x) pw[x][e] = w[x];
        }
        // O^T
        float vsc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) vsc[e] = scale_value((vs[e >> 2] >> (8 * (e & 3))) & 255u);
#pragma unroll
        for (int c = 0; c < (F + 7) / 8; ++c) {
          uint32_t d[8][4];  // [key][value pair]
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t w = vw[e >> 2][e & 3][c];
            if constexpr (D == 64) w >>= 16 * (i16 & 1);
            decode8(w, vsc[e], d[e]);
          }
#pragma unroll
          for (int f = 0; f < (F < 8 ? F : 8); ++f) {
            const uint32_t sel = f & 1 ? 0x07060302u : 0x05040100u;
            const bf16x8_t vf = frag(__builtin_amdgcn_perm(d[1][f >> 1], d[0][f >> 1], sel),
                                     __builtin_amdgcn_perm(d[3][f >> 1], d[2][f >> 1], sel),
                                     __builtin_amdgcn_perm(d[5][f >> 1], d[4][f >> 1], sel),
                                     __builtin_amdgcn_perm(d[7][f >> 1], d[6][f >> 1], sel));
#pragma unroll
            for (int y = T - 1; y >= 0; --y)
              o[8 * c + f] = mfma16(vf, frag(pw[y][0], pw[y][1], pw[y][2], pw[y][3]), o[8 * c + f]);
          }
        }
      }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // Join the waves: all to the common maximum, then added in their order.
    __syncthreads();  // the last tile's readers are done
    if (g == 0) red_ml[wave][i16][0] = m, red_ml[wave][i16][1] = l;
    __syncthreads();
    float mj = kNone;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) mj = fmaxf(mj, red_ml[w][i16][0]);
    const float mj0 = mj == kNone ? 0.f : mj;
    float lj = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w)
      lj += red_ml[w][i16][1] * __builtin_amdgcn_exp2f(red_ml[w][i16][0] - mj0);
    const float al = __builtin_amdgcn_exp2f(m - mj0);
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[f][e] *= al;
    // lane (i, g), o[f][e]: row i, value F (4g + e) + f
    if (wave > 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int f = 0; f < F; f += 4)
          *reinterpret_cast<float4*>(&red_o[wave - 1][i16][F * (4 * g + e) + f]) =
              make_float4(o[f][e], o[f + 1][e], o[f + 2][e], o[f + 3][e]);
    }
    __syncthreads();
    if (wave == 0 && live) {
#pragma unroll
      for (int w = 0; w < kFewWaves - 1; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int f = 0; f < F; ++f) o[f][e] += red_o[w][i16][F * (4 * g + e) + f];
      const int64_t row = (int64_t)(row0 + t) * a.q.heads + head;
      if (a.splits > 1) {
        const int64_t at = (int64_t)split * a.pool.tokens * a.q.heads + row;
        if (g == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(mj, lj);
        float* dst = a.part + at * D;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int f = 0; f < F; f += 4)
            *reinterpret_cast<float4*>(dst + F * (4 * g + e) + f) =
                make_float4(o[f][e], o[f + 1][e], o[f + 2][e], o[f + 3][e]);
      } else {
        const float inv = lj == 0.f ? 0.f : 1.f / lj;
        if (a.lse != nullptr && g == 0)
          a.lse[row] = lj == 0.f ? kNone : (mj + __builtin_amdgcn_logf(lj)) * kLn2;
        const int64_t at = (int64_t)(row0 + t) * a.o.ts + head * a.o.hs;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (F >= 8) {
#pragma unroll
            for (int f = 0; f < F; f += 8) {
              float v[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) v[x] = o[f + x][e] * inv;
              store8<F32>(a.o.p, at + F * (4 * g + e) + f, v);
            }
          } else {
            const int64_t x = at + F * (4 * g + e);
            if constexpr (F32)
              *reinterpret_cast<float4*>(static_cast<float*>(a.o.p) + x) =
                  make_float4(o[0][e] * inv, o[1][e] * inv, o[2][e] * inv, o[3][e] * inv);
            else
              *reinterpret_cast<uint2*>(static_cast<u16*>(a.o.p) + x) =
                  make_uint2(pack_bf16(o[0][e] * inv, o[1][e] * inv),
                             pack_bf16(o[2][e] * inv, o[3][e] * inv));
          }
        }
      }
    }
  }
}

// Joins the splits of every row, in their order: a wave takes one row.
template <int D, bool F32>
__global__ __launch_bounds__(256) void attend_join_kernel(AttnLaunch a) {
  constexpr int V = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)a.pool.tokens * a.q.heads;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  float m = kNone;
  for (int s = lane; s < a.splits; s += 64) m = fmaxf(m, a.part_ml[2 * (s * rows + row)]);
  m = wave_max(m);
  const float m0 = m == kNone ? 0.f : m;
  float l = 0.f, acc[V] = {};
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * (s * rows + row));
    if (ml.y == 0.f) continue;
    const float w = __builtin_amdgcn_exp2f(ml.x - m0);
    l += ml.y * w;
    const float* p = a.part + (s * rows + row) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += p[v] * w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int n = (int)(row / a.q.heads), h = (int)(row % a.q.heads);
  if (a.lse != nullptr && lane == 0)
    a.lse[row] = l == 0.f ? kNone : (m + __builtin_amdgcn_logf(l)) * kLn2;
  const int64_t at = (int64_t)n * a.o.ts + h * a.o.hs + lane * V;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (F32)
      static_cast<float*>(a.o.p)[at + v] = acc[v] * inv;
    else
      static_cast<u16*>(a.o.p)[at + v] = bf16_rne(acc[v] * inv);
  }
}

}  // namespace

namespace {

// Rows of one sequence and key head from which the many-row kernel is taken.
constexpr int kManyFrom = 64;

}  // namespace

int attn_splits(int batch, int kv_heads, int q_heads, int max_new, int max_kv, int window, bool f32,
                int dim) {
  const int64_t rows = (int64_t)max_new * (q_heads / kv_heads);
  int64_t keys = max_kv;
  if (window > 0) keys = keys < (int64_t)window + max_new ? keys : (int64_t)window + max_new;
  if (attn_many(rows, f32, dim)) {
    const int per = 32 * many_waves(dim, f32);
    const int64_t groups = (rows + per - 1) / per * kv_heads * batch;
    const int64_t most = (keys + 511) / 512;
    int64_t want = 256 / groups;
    if (want > most) want = most;
    return (int)(want < 1 ? 1 : want);
  }
  const int64_t tiles = (rows + 15) / 16 * kv_heads * batch;
  const int64_t most = (keys + 255) / 256;   // no fewer than 64 keys a wave
  int64_t want = (1024 + tiles - 1) / tiles;  // four workgroups a CU
  if (want > most) want = most;
  return (int)(want < 1 ? 1 : want);
}

bool attn_many(int64_t rows, bool f32, int dim) { return rows >= kManyFrom && !(f32 && dim == 256); }

hipError_t launch_attention(const AttnLaunch& a, hipStream_t s) {
  const int group = a.q.heads / a.pool.heads;
  if (attn_many((int64_t)a.max_new * group, a.f32, a.pool.dim)) return launch_attend_many(a, s);
  int64_t tiles = ((int64_t)a.max_new * group + 15) / 16;
  if (tiles * a.pool.heads > 65535) tiles = 65535 / a.pool.heads;
  const dim3 grid(a.splits, (uint32_t)(tiles * a.pool.heads), a.pool.batch);
#define TTT_CALL(D, T, F) attend_few_kernel<D, T, F><<<grid, 64 * kFewWaves, 0, s>>>(a, (int)tiles)
  switch (a.pool.dim) {
    case 64: if (a.f32) { TTT_CALL(64, 3, true); } else { TTT_CALL(64, 1, false); } break;
    case 128: if (a.f32) { TTT_CALL(128, 3, true); } else { TTT_CALL(128, 1, false); } break;
    default: if (a.f32) { TTT_CALL(256, 3, true); } else { TTT_CALL(256, 1, false); } break;
  }
#undef TTT_CALL
  return hipGetLastError();
}

hipError_t launch_attention_join(const AttnLaunch& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.pool.tokens * a.q.heads;
  const uint32_t grid = (uint32_t)((rows + 3) / 4);
#define TTT_CALL(D, F) attend_join_kernel<D, F><<<grid, 256, 0, s>>>(a)
  switch (a.pool.dim) {
    case 64: if (a.f32) { TTT_CALL(64, true); } else { TTT_CALL(64, false); } break;
    case 128: if (a.f32) { TTT_CALL(128, true); } else { TTT_CALL(128, false); } break;
    default: if (a.f32) { TTT_CALL(256, true); } else { TTT_CALL(256, false); } break;
  }
#undef TTT_CALL
  return hipGetLastError();
}

}  // namespace tttk
