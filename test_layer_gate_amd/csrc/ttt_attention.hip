// gfx950 kernels of attention over the paged 4-bit cache.
//
// Row (t, h) of a sequence stands at position p = len - new + t and sees the
// keys j with max(0, p - window + 1) <= j <= p (causal; else j < len):
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j,
// in one pass over the keys with the running maximum m, sum and weighted sum
// (rescaled whenever m has grown by more than a factor 2^8 of the weights).
//
// Codes times their power-of-two scale are exact in bf16, so keys and values
// enter the matrix instructions without a rounding; what is rounded is the
// weights p (to two bf16 terms where a sequence has up to 16 rows a key head,
// to one where it has more), and, for fp32 rows, nothing: q and p are then
// three bf16 terms each. Everything accumulates in fp32. (The scaled matrix
// instructions would take keys as codes against 8-bit terms of q, in the same
// time and without decoding; they keep about 17 bits of a sum of 8 products,
// which left scores and lse off by 1e-4, and were not taken.)
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ttt_attention.h"

namespace tttk {
namespace {

// ---------------------------------------------------------------------------
// Few rows. A wave takes 16 rows (query heads of one key head, times tokens),
// or 8, each twice, or 32 that share the decoded keys, and a stretch of the keys, 32 at a time,
// the next 32 on their way meanwhile. S^T = K Q^T with 16x16x32: lane (i, g) =
// (lane % 16, lane / 16) brings D / 4 neighbouring values of key i; of the
// result it holds, for row i, keys 4g .. 4g + 3 of either 16. Those eight are
// what the second product O^T = V^T P^T (16x16x32) asks of it: the order of the
// contraction is free as long as V agrees, so P goes over without a move
// between lanes. Of V it brings the same eight keys' values i D / 16 .. + D /
// 16 - 1. Four waves share a workgroup's stretch of keys and join in LDS, or,
// where there are tiles enough for all, each has its own.
//
// Long caches are bound by HBM: three waves a SIMD (bf16, 128) have 32 keys each
// under way, 4.3 KB. One token of 40/8 heads of 128 over 128k keys (143 MB) takes
// 27 us, 5.3 TB/s, and its join 4; 32 sequences of 4k to 32k keys, 32/8 heads
// (0.56 GB), 91 to 94 us, 6.0 to 6.2 TB/s, and 5. A stream that only reads reaches
// 6.6 TB/s. (Keys that came through LDS, two tiles ahead, took 5% longer: it is
// not the bytes on their way that are few.) From 17 rows on decoding is what
// bounds it, which 32 rows share where registers allow (bf16, heads of 64 and
// 128): 4 tokens of 40/8 heads of 128 after 93k keys in 10 sequences 315 us for
// 16 and 228 for 32 when that was chosen, 205 now.

// Who else reads a workgroup's keys: those of the sequence's other rows; no
// one, where one tile of rows is all; no one, and the keys are a slice of all
// sequences'; no one, and the sequences are short (of 9 to 16 bf16 rows; else as
// where they are shared). Codes that are read once are read past the caches'
// replacement:
// one token over 128k keys 33.8 / 31.0 us a call, 32 ragged sequences 109 / 97.
// Rows that share them are slower so (windowed fp32 rows 66 / 69), and so are
// short sequences in one workgroup (12.1 / 12.6) and heads of 256, of which a
// read takes half of a lane's 32 bytes (32 sequences 138 / 141).
enum Keys { kShared, kAlone, kSliced, kShort };

// One lane's share of 32 keys (two pieces of 16): raw codes and scales.
template <int D>
struct FewTile {
  static constexpr int kN = D == 256 ? 2 : 1;
  uint4 kw[2][kN], vw[2][kN];
  uint32_t ks[2], vs[2];  // of K the word that holds the lane's scale bytes
  bool have[2];
};

template <int D, int T, bool F32, int ROWS, Keys KEYS, int NW = 4>
__global__ __launch_bounds__(64 * NW, D == 64 && ROWS <= 16 ? 4 : 2) void attend_few_kernel(
    AttnLaunch a, int row_tiles) {
  constexpr bool SLICED = KEYS == kSliced, kOnce = D < 256 && (KEYS == kAlone || KEYS == kSliced);
  constexpr int NP = D == 256 ? 2 : 1;  // 16-byte pieces a lane takes of a key
  constexpr int KS = D / 32;            // steps of the first product
  constexpr int F = D / 16;             // V fragments = values per lane
  constexpr int kRows = ROWS;           // of a tile
  constexpr int RT = ROWS == 32 ? 2 : 1;
  constexpr bool kPairs = ROWS == 8;
  // Terms of the weights of bf16 rows. One term is off by about what rounding
  // the output costs (0.0013 rms beside 0.0016), and by more where one key has
  // nearly all of the weight, which few rows do not average out (one token over
  // 777 keys 0.0021 to 0.0027 against 64 bits). Up to 8 rows fill half of the
  // matrix instructions' columns: row i's second terms are column i + 8, at the
  // cost of the split alone (0.0016 in all; 32 sequences of 4k to 32k keys, 32/8
  // heads of 128, 97.9 us for 95.9 with one term, of 64 72.7 for 69.9). Up to 16
  // rows get them by a second product (32/2 heads 39.2 us for 38.0). More rows
  // have one term: there the matrix unit is what the call waits for. The choice
  // is by max_new alone, so that a bound of the lengths changes no result.
  constexpr int TP = F32 ? 3 : kPairs || ROWS == 32 || KEYS == kShared ? 1 : 2;
  // Three terms of the rows' queries would be the registers of a second wave:
  // the waves, whose rows are the same, read them from LDS.
  constexpr bool kShareQ = T > 1;
  static_assert(RT == 1 || !kShareQ, "shared queries are of one tile");
  constexpr size_t kRed = NW == 1 ? 16 : sizeof(float) * (NW - 1) * kRows * (D + 4), kQ = kShareQ ? T * KS * 1024 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t pool[kRed > kQ ? kRed : kQ];
  float(*red_o)[kRows][D + 4] = reinterpret_cast<float(*)[kRows][D + 4]>(pool);
  uint4(*shared_q)[KS][64] = reinterpret_cast<uint4(*)[KS][64]>(pool);
  __shared__ float red_ml[NW][kRows][2];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int i_row = kPairs ? i16 & 7 : i16;
  const bool first_term = !kPairs || i16 < 8;
  const uint32_t less = first_term ? 0u : 0xbf80u;  // -1 in bf16: a second term lacks the first
  // Key heads vary fastest, then slices, or rows, sequences and at last splits:
  // workgroups go round the XCDs in this order, and a split that short
  // sequences do not have must not be one XCD's.
  int id = (int)block_of_grid();  // kMostGroups keeps it in 32 bits
  const int hk = id % a.pool.heads;
  id /= a.pool.heads;
  const int group = a.q.heads / a.pool.heads;
  const int page = a.pool.page, gpp = page >> 4;  // 16-key pieces a page
  int b, tile, split = 0;
  Line line = {};
  if constexpr (SLICED) {
    if (id >= a.slices) return;
    line = line_of(a, id, kRows, group, 32 * NW, lane);
    if (line.at >= line.end) return;
    b = line.b, tile = 0;
  } else {
    tile = row_tiles - 1 - id % row_tiles;  // the last, which see most, first
    id /= row_tiles;
    b = id % a.pool.batch, split = id / a.pool.batch;
    if (split >= a.splits) return;
  }

  for (;;) {
    const Seq seq = seq_of(a.pool, b);
    const int row0 = seq.row0, news = seq.news;
    const int rows = max(news, 0) * group;
    if (tile * kRows >= rows) break;  // (of a slice's sequences, the first tile has rows)
    bool live[RT];
    int t[RT], head[RT];
    Span sp[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int r = tile * kRows + 16 * x + i_row;
      live[x] = first_term && r < rows;
      t[x] = min(r, rows - 1) / group;
      head[x] = hk * group + min(r, rows - 1) % group;
      sp[x] = span_of(a, seq, t[x]);
    }
    // the tile's keys
    const Span first = span_of(a, seq, tile * kRows / group);
    const Span last = span_of(a, seq, min(tile * kRows + kRows - 1, rows - 1) / group);
    const int lo = first.lo & ~31, hi = last.hi;
    const int all_lo = last.lo, all_hi = first.hi;  // keys that every row sees

    // Q as the first product's B operand: step s, values (D / 4) g + 8 s ..
    uint4 qf[RT][kShareQ ? 1 : KS];
    {
      if constexpr (kShareQ) __syncthreads();  // the last tile's readers are done
      const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        const int64_t at = (int64_t)(row0 + t[x]) * a.q.ts + head[x] * a.q.hs + g * (D / 4);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if (kShareQ && s % NW != wave) continue;
          float v[8];
          load8<F32>(a.q.p, at + 8 * s, v);
          uint32_t w[4][T];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2<T>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
          for (int y = 0; y < T; ++y) {
            const uint4 z = make_uint4(w[0][y] ^ flip, w[1][y] ^ flip, w[2][y] ^ flip, w[3][y] ^ flip);
            if constexpr (kShareQ)
              shared_q[y][s][lane] = z;
            else
              qf[x][s] = z;
          }
        }
      }
      if constexpr (kShareQ) __syncthreads();
    }
    const float sc = fmaxf(fabsf(a.scale) * kLog2e, 1.2e-38f), grown = fminf(8.f / sc, 1e38f);
    f32x4_t o[RT][F];
    float m[RT], ms[RT], l[RT];  // maximum (unscaled), its scaled value (0 for none), sum
#pragma unroll
    for (int x = 0; x < RT; ++x) {
#pragma unroll
      for (int f = 0; f < F; ++f) o[x][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      m[x] = kNone, ms[x] = 0.f, l[x] = 0.f;
    }

    const uint32_t k_lane = i16 * (D / 2) + (D == 64 ? g >> 1 : g * NP) * 16;
    const uint32_t v_lane = page * (D / 2) + g * (2 * D) + (D == 64 ? (i16 >> 1) * 16 : i16 * (D / 8));
    // K's scales are read as words (a byte load's widening would be waited for
    // at once) and cut to the lane's byte where they are used.
    const uint32_t ks_lane = page * D + (D == 64 ? (i16 >> 1) * 4 : D == 128 ? i16 * 4 : i16 * 8 + (g >> 1) * 4);
    const int ks_shift = D == 64 ? 16 * (i16 & 1) + 8 * (g >> 1) : D == 128 ? 8 * g : 16 * (g & 1);
    const uint32_t vs_lane = page * D + page * (D / 32) + (i16 * (D / 16) / 32) * page + 4 * g;

    // This part's stretches of keys, a wave's share of each: of a slice what it
    // has of the sequence; of a split every splits-th; of one part all of the
    // tile's keys, whatever the launch expected. What a slice has no part for,
    // rows past the first tile (more than max_new allowed for), are done whole
    // by the workgroup that has the sequence's first keys.
    const bool sliced = SLICED && tile == 0;
    const uint32_t u0 = line.at - line.off, u1 = min(line.n, line.end - line.off);  // of a slice
    const int per = sliced ? (int)(u1 - u0) * 32
                    : SLICED || a.splits == 1 ? (max(hi - lo, 1) + 32 * NW - 1) / (32 * NW) * 32
                                                    : a.each / NW;
    const int64_t begin = lo + (sliced ? (int64_t)u0 * 32 * NW : (int64_t)split * per * NW);
    const int64_t end = sliced ? min((int64_t)hi, lo + (int64_t)u1 * 32 * NW) : hi;
    for (int64_t s0 = begin; s0 < end; s0 += (int64_t)(SLICED ? 1 : a.splits) * per * NW) {
      const int k0 = (int)s0 + wave * per, k1 = min((int)end, k0 + per);
      // Where 64 pieces of 16 keys lie, one a lane: the address of the head's
      // block and the first key's place in it. Loads take the address from
      // scalar registers and a 32-bit offset of the lane's.
      uint64_t my_block = (uint64_t)a.pool.pages;
      uint32_t my_off = 0;
      uint64_t gone = 0;  // pieces that have no page, or are past the end
      auto find = [&](int base) {
        const int piece = (base >> 4) + lane;
        const int pg = piece / gpp;
        my_block = (uint64_t)a.pool.pages, my_off = 0;
        bool ok = pg < a.pool.max_pages && piece * 16 < k1;
        if (ok) {
          const int id = a.pool.table[(int64_t)b * a.pool.max_pages + pg];
          ok = (uint32_t)id < (uint32_t)a.pool.n_pages;
          if (ok) {
            my_block += id * a.pool.page_stride + hk * head_block_bytes(page, D);
            my_off = (piece - pg * gpp) * 16;
          }
        }
        gone = __ballot(!ok);
      };
      auto fetch = [&](FewTile<D>& x, int src) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t lo32 = __builtin_amdgcn_readlane((int)(uint32_t)my_block, src + u);
          const uint32_t hi32 = __builtin_amdgcn_readlane((int)(my_block >> 32), src + u);
          const uint32_t off = __builtin_amdgcn_readlane((int)my_off, src + u);
          x.have[u] = (gone >> (src + u) & 1) == 0;
          const Global bp = reinterpret_cast<Global>((uint64_t)hi32 << 32 | lo32);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            x.kw[u][p] = load16<kOnce>(bp + (k_lane + off * (D / 2)) + 16 * p);
            x.vw[u][p] = load16<kOnce>(bp + (v_lane + off * (D / 2)) + 16 * p);
          }
          x.ks[u] = load4(bp + (ks_lane + off * (D / 32)));
          x.vs[u] = load4(bp + (vs_lane + off));
        }
      };
      FewTile<D> cur, nxt;
      if (k0 < k1) {
        find(k0);
        fetch(nxt, 0);
      }
      for (int j = k0; j < k1; j += 32) {
        cur = nxt;
        if (j + 32 < k1) {
          const int ahead = (j + 32 - k0) & 1023;
          if (ahead == 0) find(j + 32);
          fetch(nxt, ahead >> 4);
        }
        uint32_t ks[2][NP];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int q = 0; q < NP; ++q) ks[u][q] = (cur.ks[u] >> (ks_shift + 8 * q)) & 255u;
        // S^T
        if constexpr (kShareQ) asm volatile("" ::: "memory");  // not all at once, ahead of the loop
        f32x4_t s[RT][2];
#pragma unroll
        for (int x = 0; x < RT; ++x) s[x][0] = s[x][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < KS; ++q) {
          bf16x8_t kf[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint4 w = cur.kw[u][q >> 2];
            uint32_t c = (q & 3) == 0 ? w.x : (q & 3) == 1 ? w.y : (q & 3) == 2 ? w.z : w.w;
            // D = 64: a lane's 16 values are half of a block
            if constexpr (D == 64) c = g & 1 ? (q == 0 ? w.z : w.w) : c;
            uint32_t d[4];
            decode8(c, scale_value(ks[u][q >> 2]), d);
            kf[u] = frag(d[0], d[1], d[2], d[3]);
          }
#pragma unroll
          for (int y = T - 1; y >= 0; --y)
#pragma unroll
            for (int x = 0; x < RT; ++x) {
              const uint4 z = kShareQ ? shared_q[y][q][lane] : qf[x][kShareQ ? 0 : q];
#pragma unroll
              for (int u = 0; u < 2; ++u) s[x][u] = mfma16(kf[u], frag(z.x, z.y, z.z, z.w), s[x][u]);
            }
        }
        float p[RT][8];
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int e = 0; e < 8; ++e) p[x][e] = s[x][e >> 2][e & 3];
        // Keys that some row does not see, that have no page, or that hold NaN
        const uint32_t nan = nan_bytes(cur.ks[0]) | nan_bytes(cur.vs[0]) | nan_bytes(cur.ks[1]) | nan_bytes(cur.vs[1]);
        const bool odd = j < all_lo || j + 32 > all_hi || !cur.have[0] || !cur.have[1] || __any(nan != 0);
        if (odd) {
          rare_path();
          const uint32_t there = (cur.have[0] ? 0xffffu : 0u) | (cur.have[1] ? 0xffff0000u : 0u);
          uint32_t seen[RT];
#pragma unroll
          for (int x = 0; x < RT; ++x) seen[x] = bits_between(sp[x].lo - j, sp[x].hi - j) & there;
          uint32_t nan_v[NP] = {};  // keys that are NaN in the blocks of V whose sums the lane holds
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint64_t kn = __ballot(ks[u][0] > kScaleMax || ks[u][NP - 1] > kScaleMax);
            kn |= kn >> 32;
            const uint32_t kn32 = (uint32_t)kn | (uint32_t)kn >> 16;
#pragma unroll
            for (int x = 0; x < RT; ++x) {
              const uint32_t mine = seen[x] >> (16 * u + 4 * g);  // of this lane's four keys
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t keep = spread(mine, e);
                float& w = p[x][4 * u + e];
                w = __uint_as_float((__float_as_uint(w) & keep) | (kNoneBits & ~keep) |
                                    (spread(kn32 >> (4 * g), e) & keep & kNanBits));
              }
            }
            // A NaN value must not reach the rows that do not see it (0 * NaN):
            // it goes out of V, and into the sums of those that do. Lane (i, g)
            // has the scales of block i D / 512 of V, and sums of block g D /
            // 128 (of 256: and the next).
            const uint32_t bad = cur.have[u] ? nan_bytes(cur.vs[u]) : 0u;
            if (__any(bad != 0)) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint64_t all = __ballot(bad >> (8 * e + 7) & 1);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                  const uint64_t at = all >> ((g * D / 128 + q) * (512 / D));
                  const uint32_t a0 = (uint32_t)at, a1 = (uint32_t)(at >> 32);
                  nan_v[q] |= ((a0 & 1) | (a0 >> 16 & 1) << 4 | (a1 & 1) << 8 | (a1 >> 16 & 1) << 12) << (16 * u + e);
                }
              }
            }
            const uint32_t out = cur.have[u] ? bad : 0x80808080u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t gone_v = spread(out, 8 * e + 7);
              cur.vs[u] = (cur.vs[u] & ~(gone_v & 255u << (8 * e))) | (gone_v & 127u << (8 * e));
#pragma unroll
              for (int q = 0; q < NP; ++q) {
                uint4& y = cur.vw[u][q];
                uint32_t& w = e == 0 ? y.x : e == 1 ? y.y : e == 2 ? y.z : y.w;
                w &= ~gone_v;
              }
            }
          }
#pragma unroll
          for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (nan_v[NP * e / 4] & seen[x]) {
#pragma unroll
                for (int f = 0; f < F; ++f) o[x][f][e] = __builtin_nanf("");
              }
        }
        // The maximum is only followed when a weight would pass 2^8: until
        // then the lanes need not agree on a new one, and nothing is rescaled.
        float mx[RT];
        bool up = false;
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          mx[x] = fmaxf(fmaxf(fmaxf(p[x][0], p[x][1]), fmaxf(p[x][2], p[x][3])),
                        fmaxf(fmaxf(p[x][4], p[x][5]), fmaxf(p[x][6], p[x][7])));
          up |= mx[x] > m[x] + grown;
        }
        if (__any(up)) {
#pragma unroll
          for (int x = 0; x < RT; ++x) {
            float mn = fmaxf(mx[x], __shfl_xor(mx[x], 16));
            mn = fmaxf(fmaxf(mn, __shfl_xor(mn, 32)), m[x]);
            const float n0 = mn == kNone ? 0.f : mn * sc;
            const float al = m[x] == kNone ? 0.f : __builtin_amdgcn_exp2f(ms[x] - n0);
            m[x] = mn, ms[x] = n0;
            l[x] *= al;
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[x][f][e] *= al;
          }
        }
        uint32_t pw[RT][TP][4];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          float(&w)[8] = p[x];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = __builtin_amdgcn_exp2f(fmaf(w[e], sc, -ms[x]));
          l[x] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kPairs) {
              const uint32_t z = pack_bf16(w[2 * e], w[2 * e + 1]);
              pw[x][0][e] = pack_bf16(dot2(z, less, w[2 * e]), dot2(z, less << 16, w[2 * e + 1]));
              continue;
            }
            uint32_t z[TP];
            split2<TP>(w[2 * e], w[2 * e + 1], z);
#pragma unroll
            for (int y = 0; y < TP; ++y) pw[x][y][e] = z[y];
          }
        }
        // O^T
        float vsc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) vsc[e] = scale_at(cur.vs[e >> 2], e & 3);
#pragma unroll
        for (int c = 0; c < NP; ++c) {
#pragma unroll
          for (int f = 0; f < (F < 8 ? F : 8); f += 2) {
            uint32_t d[8];  // values f and f + 1 of each key
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint4 y = cur.vw[e >> 2][c];
              uint32_t w = (e & 3) == 0 ? y.x : (e & 3) == 1 ? y.y : (e & 3) == 2 ? y.z : y.w;
              if constexpr (D == 64) w >>= 16 * (i16 & 1);
              d[e] = decode2(w, vsc[e], f >> 1);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t sel = h ? 0x07060302u : 0x05040100u;
              const bf16x8_t vf = frag(__builtin_amdgcn_perm(d[1], d[0], sel), __builtin_amdgcn_perm(d[3], d[2], sel),
                                       __builtin_amdgcn_perm(d[5], d[4], sel), __builtin_amdgcn_perm(d[7], d[6], sel));
#pragma unroll
              for (int y = TP - 1; y >= 0; --y)
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                  const auto& w = pw[x][y];
                  o[x][8 * c + f + h] = mfma16(vf, frag(w[0], w[1], w[2], w[3]), o[x][8 * c + f + h]);
                }
            }
          }
        }
      }
    }
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      l[x] += __shfl_xor(l[x], 16);
      l[x] += __shfl_xor(l[x], 32);
      m[x] = m[x] == kNone ? kNone : ms[x];
      if constexpr (kPairs) {  // both terms' sums
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[x][f][e] += eight_lanes_on(o[x][f][e]);
      }
    }

    // Join the waves: all to the common maximum, then added in their order.
    __syncthreads();  // the last tile's readers are done
#pragma unroll
    for (int x = 0; x < RT; ++x)
      if (g == 0 && first_term) red_ml[wave][16 * x + i_row][0] = m[x], red_ml[wave][16 * x + i_row][1] = l[x];
    __syncthreads();
    float mj[RT], lj[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      mj[x] = kNone, lj[x] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) mj[x] = fmaxf(mj[x], red_ml[w][16 * x + i_row][0]);
      const float mj0 = mj[x] == kNone ? 0.f : mj[x];
#pragma unroll
      for (int w = 0; w < NW; ++w)
        lj[x] += red_ml[w][16 * x + i_row][1] * __builtin_amdgcn_exp2f(red_ml[w][16 * x + i_row][0] - mj0);
      const float al = __builtin_amdgcn_exp2f(m[x] - mj0);
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][f][e] *= al;
      // lane (i, g), o[f][e]: row i, value F (4g + e) + f
      if (wave > 0 && first_term) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int f = 0; f < F; f += 4)
            *reinterpret_cast<float4*>(&red_o[wave - 1][16 * x + i_row][F * (4 * g + e) + f]) =
                make_float4(o[x][f][e], o[x][f + 1][e], o[x][f + 2][e], o[x][f + 3][e]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      if (wave > 0 || !live[x]) continue;
#pragma unroll 1  // all at once would need the most registers of the kernel
      for (int w = 0; w < NW - 1; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int f = 0; f < F; ++f) o[x][f][e] += red_o[w][16 * x + i_row][F * (4 * g + e) + f];
      const int64_t row = (int64_t)(row0 + t[x]) * a.q.heads + head[x];
      if (sliced ? u0 > 0 || u1 < line.n : a.splits > 1) {
        // slice + sequence: no two pairs that meet have the same sum
        const int part = (((int)(line.at / line.per) + b) * a.pool.heads + hk) * kRows + 16 * x + i_row;
        const int64_t at = sliced ? (int64_t)part : (int64_t)split * a.pool.tokens * a.q.heads + row;
        if (sliced && u0 == 0 && g == 0)
          *reinterpret_cast<int2*>(a.part_of + 2 * row) =
              make_int2(part, (int)((line.off + line.n - 1) / line.per - line.at / line.per) + 1);
        if (g == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(mj[x], lj[x]);
        float* dst = a.part + at * D;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int f = 0; f < F; f += 4)
            *reinterpret_cast<float4*>(dst + F * (4 * g + e) + f) =
                make_float4(o[x][f][e], o[x][f + 1][e], o[x][f + 2][e], o[x][f + 3][e]);
      } else {
        const float inv = lj[x] == 0.f ? 0.f : 1.f / lj[x];
        if (a.lse != nullptr && g == 0)
          a.lse[row] = lj[x] == 0.f ? kNone : (mj[x] + __builtin_amdgcn_logf(lj[x])) * kLn2;
        if (SLICED && g == 0) *reinterpret_cast<int2*>(a.part_of + 2 * row) = make_int2(0, 0);
        const int64_t at = (int64_t)(row0 + t[x]) * a.o.ts + head[x] * a.o.hs;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (F >= 8) {
#pragma unroll
            for (int f = 0; f < F; f += 8) {
              float v[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) v[y] = o[x][f + y][e] * inv;
              store8<F32>(a.o.p, at + F * (4 * g + e) + f, v);
            }
          } else {
            const int64_t y = at + F * (4 * g + e);
            if constexpr (F32)
              *reinterpret_cast<float4*>(static_cast<float*>(a.o.p) + y) =
                  make_float4(o[x][0][e] * inv, o[x][1][e] * inv, o[x][2][e] * inv, o[x][3][e] * inv);
            else
              *reinterpret_cast<uint2*>(static_cast<u16*>(a.o.p) + y) =
                  make_uint2(pack_bf16(o[x][0][e] * inv, o[x][1][e] * inv),
                             pack_bf16(o[x][2][e] * inv, o[x][3][e] * inv));
          }
        }
      }
    }
    if constexpr (!SLICED) {
      tile += row_tiles;
      continue;
    }
    if (u0 == 0 && (tile + 1) * kRows < rows) {
      ++tile;
      continue;
    }
    // the slice's next sequence that has rows
    tile = 0;
    line.at = line.off += line.n;
    line.n = 0;
    while (line.at < line.end && line.n == 0 && ++b < a.pool.batch)
      line.n = units_of(a, seq_of(a.pool, b), kRows, group, 32 * NW);
    if (line.n == 0) break;
  }
}

// Joins the parts of every row, in their order. ROWS rows a workgroup: each
// has 256 / ROWS threads, D / 4 of which hold 4 values each of one split; the
// others take every LANES-th split beside them and are added at the end. With
// many splits there are few rows: one a workgroup.
template <int D, bool F32, int ROWS>
__global__ __launch_bounds__(256) void attend_join_kernel(AttnLaunch a) {
  constexpr int TPR = 256 / ROWS, LANES = TPR / (D / 4);
  static_assert(LANES == 1 || ROWS == 1, "threads of a row");
  __shared__ float4 red[ROWS][LANES][D / 4];
  __shared__ float red_l[ROWS][LANES];
  const int rr = threadIdx.x / TPR, c = threadIdx.x % TPR % (D / 4), y = threadIdx.x % TPR / (D / 4);
  const int64_t rows = (int64_t)a.pool.tokens * a.q.heads;
  const int64_t row0 = block_of_grid() * ROWS;
  if (row0 >= rows) return;
  const int64_t row = min(row0 + rr, rows - 1);
  // The row's parts: `count` from `base`, `stride` apart. Rows that no sequence
  // claims have nothing in part_of: whatever is there is kept in bounds.
  int64_t base = row, stride = rows;
  int count = a.splits;
  if (a.slices > 0) {
    stride = a.pool.heads * a.tile;
    const int all = (a.slices + a.pool.batch - 1) * (int)stride;
    const int2 d = *reinterpret_cast<const int2*>(a.part_of + 2 * row);
    if (d.y <= 0 || (uint32_t)d.x >= (uint32_t)all) return;
    base = d.x;
    count = min(d.y, (all - 1 - d.x) / (int)stride + 1);
  }
  float m = kNone;
  if constexpr (LANES > 1) {
    // the maximum, one part a thread
    for (int s = threadIdx.x; s < count; s += 256) m = fmaxf(m, a.part_ml[2 * (base + s * stride)]);
    m = wave_max(m);
    __shared__ float red_m[4];
    if ((threadIdx.x & 63) == 0) red_m[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red_m[0], red_m[1]), fmaxf(red_m[2], red_m[3]));
  } else {
    for (int s = 0; s < count; ++s) m = fmaxf(m, a.part_ml[2 * (base + s * stride)]);
  }
  const float m0 = m == kNone ? 0.f : m;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = y; s < count; s += LANES) {
    const int64_t at = base + s * stride;
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
    const float4 v = *reinterpret_cast<const float4*>(a.part + at * D + 4 * c);
    const float w = __builtin_amdgcn_exp2f(ml.x - m0);
    l += ml.y * w;
    acc.x += v.x * w, acc.y += v.y * w, acc.z += v.z * w, acc.w += v.w * w;
  }
  if constexpr (LANES > 1) {
    red[rr][y][c] = acc;
    if (c == 0) red_l[rr][y] = l;
    __syncthreads();
    if (y > 0) return;
#pragma unroll
    for (int z = 1; z < LANES; ++z) {
      const float4 v = red[rr][z][c];
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      l += red_l[rr][z];
    }
  }
  if (row0 + rr >= rows) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int n = (int)(row / a.q.heads), h = (int)(row % a.q.heads);
  if (a.lse != nullptr && c == 0)
    a.lse[row] = l == 0.f ? kNone : (m + __builtin_amdgcn_logf(l)) * kLn2;
  const int64_t at = (int64_t)n * a.o.ts + h * a.o.hs + 4 * c;
  if constexpr (F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.o.p) + at) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2*>(static_cast<u16*>(a.o.p) + at) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

}  // namespace

namespace {

// Keys up to which one workgroup of the few-row kernel takes a whole sequence,
// without the join's launch and its workspace. On the GPU alone (one token,
// 32/8 heads of 128) one sequence of 512 keys takes 7.4 us so and 8.2 in parts,
// of 777 9.6 and 8.2, of 1024 10.5 and 8.3; 16 sequences of 1024 11.1 and 12.6.
// A launch and an allocation saved are 4 us of the caller's time, which is what
// a call as short as this waits for. (Eight waves a workgroup instead of four:
// 10.1 us for 777 keys, 10.4 for 1024, 12.6 for 32 sequences of 1024 either way.)
constexpr int kOneGroup = 1024;

// Tiles of rows from which on every wave takes one of its own, all of its keys,
// and none are joined, instead of sharing its keys with three others: fp32 rows,
// and bf16 rows with heads of 256 (the others' many tiles are the many-row
// kernel's). us, four waves a tile / one, causal prompts, sequences x tokens:
//   fp32, 64/8 heads of 128, 4 x 1738 650 / 573; 32/8, 4 x 512 53 / 49, 1 x 8k 1447 / 1403
//   fp32, 64/8 heads of 64, 6 x 603 124 / 98; 32/8, 4 x 1k 94 / 88, 2 x 2k 151 / 170
//   bf16, 128/8 heads of 256, 2 x 1976 1091 / 887; 32/8, 4 x 512 77 / 51, 1 x 8k 1832 / 1737
//   fp32, 32/8 heads of 256, 4 x 512 106 / 91, 4 x 1k 288 / 263, 2 x 2k 436 / 445,
//   1 x 8k 2830 / 3145; 128/8, 1k tokens after 15k 5273 / 6612; 64/8, 2k tokens under
//   a window of 64 160 / 109
// With 2048 tiles it is even (fp32, 2048 tokens, 16/4 heads of 64: 46 / 45). fp32
// queries of 256 take 24 KB of LDS, which leaves such waves 1.5 a SIMD: theirs
// is for up to kOneGroup keys alone. (Of 64, 4 waves a SIMD, of 128, 3; bf16 of
// 256, 2.)
constexpr int kOwnTile = 4096;

// Whether the many-row kernel is taken, for bf16 rows with heads of 64 or 128:
// by what either kernel takes, in us, of heads of 128 (of 64 both take about 4/5).
// A workgroup of the many-row kernel takes 2 us for 64 keys of its 256 rows,
// one CU each, after 12 us of start; the rounds after the first start in 20.
// The few-row kernel takes 0.8 us for 2^20 pairs of a row and a key, and 9 us
// to start each round of 512 workgroups. Parts cost a join and their way
// through memory. keys: of a tile of rows; seen: of them, on average.
//   many / few, measured (32/8 heads of 128 and, in brackets, 64; sequences x
//   tokens): 1 x 256 after 16k 93 / 99 (80 / 82), 1 x 128 after 64k 153 / 182 (115 /
//   145), 4 x 512 over 4k 135 / 171 (104 / 136); prompts of 1 x 1k tokens 43 / 26
//   (32 / 21), 4 x 1k 69 / 88 (55 / 70), 1 x 2k 69 / 65 (55 / 51); of 64 also 1 x 256
//   12.8 / 12.2, 4 x 256 13.4 / 15.6, 1 x 8k 415 / 544.
// fp32 rows keep the matrix unit three times as long, beside which decoding
// for 16 rows alone costs little, and with wide heads a workgroup's sums leave
// no registers for a second wave: built for them, it took 879 us for the
// few-row kernel's 783 (fp32, 64), 1146 for 1162 (fp32, 128), 2148 for 1351
// (fp32, 256) and 612 for 689 (bf16, 256) over 16384 rows and 8k keys, and
// lost wherever there were fewer.
struct Costs {
  double rows, heads;  // rows a key head; key heads of all sequences
  static double parts(double rows, double n) { return n > 1 ? 5 + rows * n * 2.6e-4 : 0; }
  double many(double keys, double seen, double splits) const {
    const double groups = ceil(rows / kManyTile) * heads;
    const double longest = ceil(keys / 64 / splits), mean = groups * seen / 64 / 256;
    return 12 + 20 * fmax(groups * splits / 256 - 1, 0) + 2 * fmax(longest, mean) + parts(rows * heads, splits);
  }
  double few(double tile, double seen, double splits) const {
    const double groups = ceil(rows / tile) * heads * splits;
    return 9 * fmax(groups / 512, 1) + 0.8 * rows * heads * seen / (1 << 20) + parts(rows * heads, splits);
  }
};

// Workgroups that parts and tiles of rows may make of a launch (of a sequence's
// tiles, in the many-row kernel). Beyond them there is one a sequence and key
// head, so that their number fits the kernels' 32 bits (2^26 at most).
constexpr int64_t kMostGroups = (int64_t)1 << 20;

AttnPlan few_plan(int batch, int kv_heads, int64_t rows, int64_t keys, int tile, bool f32, int dim) {
  // A short sequence is one workgroup.
  if (keys <= kOneGroup) return {false, 1, kOneGroup, 0, tile};
  // Several sequences with one tile of rows each: a slice for every workgroup
  // that the card holds at once, whatever the lengths are, which only the GPU
  // knows. Against parts of 8192 keys each (us, with the join, 32/8 heads of
  // 128): 24 sequences of 16k keys 101 / 89, 32 of 4k to 32k 155 / 134, one of
  // 128k and 31 of 1k 380 / 51, 128 of 1 to 8k 133 / 124; 2 of 1500 14.4 / 15.2,
  // 200 of 1 to 4k (one part each then) 92 / 99. 512 slices 134 us for the 32,
  // 1024 152, 1536 139.
  if (rows <= tile && batch > 1 && batch <= kSliceBatch) {
    const int64_t units = (keys + 127) / 128 * batch;
    const int64_t fit = dim == 256 || tile == 32 ? 512 : dim == 64 && !f32 ? 1024 : 768;
    int64_t slices = fit / kv_heads < 1 ? 1 : fit / kv_heads;
    if (slices > units) slices = units;
    return {false, 1, 0, (int)slices, tile};
  }
  // Stretches that give 512 workgroups of four waves, or 1024 where some
  // sequences may be shorter than max_kv; of 512 keys or more where there is
  // much to do (each workgroup loads its rows and hands in its sums), and of
  // 128 at least. 1 token over 128k keys: 512 take 35.4 us, 768 36.8, 1024
  // 40.6, 2304 44.0.
  const double work = (double)keys * ((rows + tile - 1) / tile) * kv_heads * batch;
  const double fair = work / (batch > 1 ? 1024 : 512), least = work < 512 * 256 ? 128 : 512;
  const double most = 1 << 20, e = fair < least ? least : fair > most ? most : fair;
  const int each = ((int)e + 127) / 128 * 128;
  // max_kv is a bound: with many sequences and heads, parts of what it allows
  // for would be more workgroups than 32 bits count (and the chip is full
  // without them). A part walks over all keys, whatever their number.
  const int64_t parts = (keys + each - 1) / each, most_parts = kMostGroups / ((int64_t)kv_heads * batch);
  if (most_parts <= 1) return {false, 1, (int)keys, 0, tile};
  return {false, (int)(parts < most_parts ? parts : most_parts), each, 0, tile};
}

}  // namespace

AttnPlan attn_plan(int batch, int kv_heads, int q_heads, int max_new, int max_kv, int window, bool f32,
                   int dim) {
  const int group = q_heads / kv_heads;
  const int64_t rows = (int64_t)max_new * group, all = max_kv < kMaxKeys ? max_kv : kMaxKeys;
  // The keys of so many rows in a row.
  auto span = [&](int tile) {
    const int64_t near = (int64_t)window + (tile + group - 1) / group;
    return window > 0 && near < all ? near : all;
  };
  const int tile = f32 ? 16 : rows <= 8 ? 8 : dim <= 128 && rows > 16 ? 32 : 16;
  const AttnPlan few = few_plan(batch, kv_heads, rows, span(tile), tile, f32, dim);
  if (f32 || dim > 128 || rows <= 32) return few;
  // Parts until there is a workgroup for every CU, of 512 keys at least: 1024
  // tokens of 32/8 heads after 64k keys take 1050 us in 256 workgroups, 1390 in
  // 128, 1058 in 512; 64 tokens 94, 113 and 108. Parts of 2k or more where there
  // are 512 keys: 4 x 128 tokens over 4k keys 67 us for 60.
  const double heads = (double)kv_heads * batch, groups = ceil((double)rows / kManyTile) * heads;
  const int64_t keys = span(kManyTile), most = (keys + 511) / 512;
  int64_t want = (int64_t)(256 / groups);
  if (want > most) want = most;
  if (want < 1) want = 1;
  const double before = 0.5 * (max_new < all ? max_new : all);  // keys that causal rows miss
  const Costs c = {(double)rows, heads};
  const double many = c.many((double)keys, fmin((double)keys, all - before), (double)want);
  return many < c.few(tile, fmin((double)span(tile), all - before), few.splits)
             ? AttnPlan{true, (int)want, 0, 0, 0} : few;
}

// Tiles of rows as max_new and the rows there are at all allow, within
// kMostGroups: a workgroup then takes several.
AttnGrid attn_grid(const AttnLaunch& a) {
  if (a.slices > 0) return {(int64_t)a.slices * a.pool.heads, 1, 4};
  const int64_t each = a.many ? kManyTile : a.tile, batch = a.pool.batch;
  const int64_t news = a.max_new < a.pool.tokens ? a.max_new : a.pool.tokens;
  const int64_t others = (int64_t)a.splits * a.pool.heads * (a.many ? 1 : batch);
  int64_t tiles = (news * (a.q.heads / a.pool.heads) + each - 1) / each;
  const int64_t most = kMostGroups / others;
  if (tiles > most) tiles = most;
  if (tiles < 1) tiles = 1;
  const int64_t groups = tiles * others * (a.many ? batch : 1);
  if (a.many) return {groups, tiles, kManyTile / 32};
  const bool alone = (int64_t)a.max_new * (a.q.heads / a.pool.heads) <= a.tile;
  const bool may = a.tile == 16 && !alone && a.splits == 1 && (a.f32 || a.pool.dim == 256) &&
                   !(a.f32 && a.pool.dim == 256 && a.each > kOneGroup);
  return {groups, tiles, may && groups >= kOwnTile ? 1 : 4};
}

namespace {

template <int D, bool F32, int ROWS>
void launch_few(const AttnLaunch& a, hipStream_t s) {
  constexpr int T = F32 ? 3 : 1;
  const AttnGrid g = attn_grid(a);
  const dim3 grid = grid_of(g.groups);
  const int tiles = (int)g.tiles;
  const bool alone = (int64_t)a.max_new * (a.q.heads / a.pool.heads) <= ROWS;
  if (a.slices > 0) {
    attend_few_kernel<D, T, F32, ROWS, kSliced><<<grid, 256, 0, s>>>(a, 1);
    return;
  }
  // bf16 rows in tiles that more rows would not fit are alone.
  if constexpr (F32 || (D == 256 && ROWS == 16) || ROWS == 32) {
    if (!alone) {
      if constexpr (ROWS == 16) {
        if (g.waves == 1) {
          attend_few_kernel<D, T, F32, ROWS, kShared, 1><<<grid, 64, 0, s>>>(a, tiles);
          return;
        }
      }
      attend_few_kernel<D, T, F32, ROWS, kShared><<<grid, 256, 0, s>>>(a, tiles);
      return;
    }
  }
  // (of the others' a short launch is no different)
  constexpr Keys kBrief = !F32 && ROWS == 16 ? kShort : kShared;
  if (a.splits == 1 && a.each <= kOneGroup)
    attend_few_kernel<D, T, F32, ROWS, kBrief><<<grid, 256, 0, s>>>(a, tiles);
  else
    attend_few_kernel<D, T, F32, ROWS, kAlone><<<grid, 256, 0, s>>>(a, tiles);
}

template <int D>
void launch_few(const AttnLaunch& a, hipStream_t s) {
  if (a.f32)
    launch_few<D, true, 16>(a, s);
  else if (a.tile == 8)
    launch_few<D, false, 8>(a, s);
  else if (a.tile == 16)
    launch_few<D, false, 16>(a, s);
  else if constexpr (D < 256)
    launch_few<D, false, 32>(a, s);
}

}  // namespace

hipError_t launch_attention(const AttnLaunch& a, hipStream_t s) {
  if (a.many) return launch_attend_many(a, s);
  switch (a.pool.dim) {
    case 64: launch_few<64>(a, s); break;
    case 128: launch_few<128>(a, s); break;
    default: launch_few<256>(a, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_attention_join(const AttnLaunch& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.pool.tokens * a.q.heads;
  // One row a workgroup has up to 16 parts in flight at once; with few of them
  // to join, as many rows as have threads for one each (1024 rows of 32
  // sequences in 96 slices: one 4.8 us, eight 6.9).
  const bool one = (a.slices > 0 ? a.slices > a.pool.batch : a.splits > 4) || rows < 512;
#define TTT_CALL(D, F)                                                                        \
  if (one)                                                                                    \
    attend_join_kernel<D, F, 1><<<grid_of(rows), 256, 0, s>>>(a);                             \
  else                                                                                        \
    attend_join_kernel<D, F, 1024 / D>                                                        \
        <<<grid_of((rows + 1024 / D - 1) / (1024 / D)), 256, 0, s>>>(a)
  switch (a.pool.dim) {
    case 64: if (a.f32) { TTT_CALL(64, true); } else { TTT_CALL(64, false); } break;
    case 128: if (a.f32) { TTT_CALL(128, true); } else { TTT_CALL(128, false); } break;
    default: if (a.f32) { TTT_CALL(256, true); } else { TTT_CALL(256, false); } break;
  }
#undef TTT_CALL
  return hipGetLastError();
}

}  // namespace tttk
