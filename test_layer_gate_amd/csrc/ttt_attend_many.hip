// gfx950 kernel of attention over the paged 4-bit cache for many bf16 rows
// with heads of 64 and 128 (prompts and segments); the method, the few-row
// kernel and the choice between them are in ttt_attention.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_attention.h"

namespace tttk {
namespace {

// A workgroup of 8 waves takes 256 rows of one key head, 32 a wave, and walks
// over its keys 64 at a time. Codes are turned into bf16 once for all of the
// rows: waves 0-3 decode the tile's keys, waves 4-7 its values (each 16
// tokens), and leave them in LDS in the order in which the matrix
// instructions read them, 1 KB a fragment, so that a fragment is one
// contiguous read. Three tiles of keys and two of values are held: the keys of
// the next tile are read by this one's work, those after it written meanwhile.
// Raw codes are on their way one tile longer, and where a wave's pieces of 64
// tiles lie is looked up at once, a tile a lane.
//
// Bound by the matrix unit and by what has to run beside it: of a matrix
// instruction's 32 clocks a wave's exponentials, packing and fragment reads
// take most, and decoding the rest. 1024 tokens of 32/8 heads of 128 at the end
// of 64k keys take 1.0 ms, 1085 TFLOP/s (large library products reach 1211 to
// 1361). Of 1.11 ms, an earlier step's, copies without decoding took 0.91,
// without exponentials 0.95, with neither 0.79.
//
// S^T = K Q^T with 32x32x16: a lane holds, of one row, the keys 8 (i / 4) + 4
// (lane / 32) + i % 4 of a 32-key tile. Taken eight at a time these are what
// the second product O^T = V^T P^T wants from that lane if V's fragments
// list the keys of 16 in the order 0-3, 8-11 | 4-7, 12-15, which is how they
// are written. The rows of V^T are numbered so that a lane of O^T holds
// neighbouring values: fragment t, row i is value i D / 32 + t.
constexpr int kManyWaves = 8, kManyRows = 32 * kManyWaves, kManyKeys = 64;
static_assert(kManyRows == kManyTile, "rows a workgroup");

// Which of a tile's keys have no page or are NaN, and which have a NaN value in
// any block of 32, and in which: one bit a key, 32 keys a word.
struct KeyMarks {
  uint32_t absent[2], nan[2];
};
struct ValueMarks {
  uint32_t nan[2], of[4][2];
};

template <int D>
struct Raw {  // a lane's share of 16 tokens' codes, and their scales
  uint4 w;
  uint32_t s;
  bool have;
};

// D = 64: half the lanes have no unit.
template <int D>
__device__ __forceinline__ bool unit_live(int lane) { return D == 128 || lane < 32; }

// Keys: unit (block of 32 values c, token t), lane = 16 c + t. Values: unit
// (four tokens q, 8 values c), lane = (D / 8) q + c. p: the head's block of
// the page, off: the first token's place there.
template <int D>
__device__ __forceinline__ void fetch(Raw<D>& r, bool is_v, Global p, uint32_t off, bool have, int page,
                                      int lane) {
  r.have = have;
  if (!unit_live<D>(lane)) return;
  if (is_v) {
    const int q = lane / (D / 8), c = lane % (D / 8);
    r.w = load16(p + (uint32_t)(page * (D / 2) + lane * 16 + off * (D / 2)));
    r.s = load4(p + (uint32_t)(page * D + page * (D / 32) + (c >> 2) * page + 4 * q + off));
  } else {
    const int c = lane >> 4, t = lane & 15;
    // the token's scales are read as a word (a byte's widening would be
    // waited for at once): D = 64's two bytes with a neighbour's
    r.w = load16(p + (uint32_t)(t * (D / 2) + c * 16 + off * (D / 2)));
    r.s = load4(p + (uint32_t)(page * D + (D == 64 ? (t >> 1) * 4 : t * 4) + off * (D / 32)));
  }
}

// 16 tokens' keys or values into LDS, as the fragments want them.
template <int D>
__device__ __forceinline__ void unpack(Raw<D>& r, bool is_v, int piece, uint8_t* kbuf, uint8_t* vbuf,
                                       KeyMarks* kmarks, ValueMarks* vmarks, int lane) {
  const bool live = unit_live<D>(lane);
  const int shift = 16 * (piece & 1);  // of the piece in its word of marks
  if (!r.have) {  // no such page, or past the end: zeros, which no row counts
    r.w = make_uint4(0, 0, 0, 0);
    r.s = 0x7f7f7f7fu;
    if (lane == 0 && !is_v) atomicOr(&kmarks->absent[piece >> 1], 0xffffu << shift);
  }
  uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
  if (is_v) {
    const uint32_t bad = live ? nan_bytes(r.s) : 0u;
    const int q = lane / (D / 8), c = lane % (D / 8);
    if (__any(bad != 0)) {
      rare_path();
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (bad >> (8 * e + 7) & 1) {
          const uint32_t bit = 1u << (shift + 4 * q + e);
          atomicOr(&vmarks->nan[piece >> 1], bit);
          atomicOr(&vmarks->of[c >> 2][piece >> 1], bit);
          w[e] = 0;
          r.s = (r.s & ~(255u << (8 * e))) | (127u << (8 * e));
        }
    }
    if (!live) return;
    uint32_t d[4][4];  // [token][value pair]
#pragma unroll
    for (int e = 0; e < 4; ++e) decode8(w[e], scale_at(r.s, e), d[e]);
    constexpr int NT = D / 32;  // fragments; value 8c + j is row (8c + j) / NT of fragment j % NT
    uint8_t* at = vbuf + piece * (NT * 1024) + (q & 1) * 512 + (q >> 1) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
      const uint2 x = make_uint2(__builtin_amdgcn_perm(d[1][j >> 1], d[0][j >> 1], sel),
                                 __builtin_amdgcn_perm(d[3][j >> 1], d[2][j >> 1], sel));
      *reinterpret_cast<uint2*>(at + (j % NT) * 1024 + (8 * c / NT + j / NT) * 16) = x;
    }
  } else {
    const int c = lane >> 4, t = lane & 15;
    const uint32_t byte = r.s >> (D == 64 ? 16 * (t & 1) + 8 * c : 8 * c) & 255u;
    const bool bad = live && byte > kScaleMax;
    if (__any(bad)) {
      rare_path();
      if (bad) atomicOr(&kmarks->nan[piece >> 1], 1u << (shift + t));
    }
    if (!live) return;
    constexpr int KS = D / 16;  // steps; values 32c + 8j .. are half j % 2 of step 2c + j / 2
    uint8_t* at = kbuf + ((piece >> 1) * KS + 2 * c) * 1024 + ((piece & 1) * 16 + t) * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t d[4];
      decode8(w[j], scale_value(byte), d);
      *reinterpret_cast<uint4*>(at + (j >> 1) * 1024 + (j & 1) * 512) = make_uint4(d[0], d[1], d[2], d[3]);
    }
  }
}

template <int D>
__global__ __launch_bounds__(64 * kManyWaves) void attend_many_kernel(AttnLaunch a, int row_tiles) {
  constexpr int KS = D / 16;           // steps of the first product
  constexpr int NT = D / 32;           // fragments of V^T
  constexpr int kFence = 0x406;        // lets vector, scalar and exponential instructions pass
  constexpr int RD = D == 64 ? 4 : 8;  // fragments read ahead
  __shared__ __attribute__((aligned(16))) uint8_t kbuf[3][kManyKeys * D * 2];
  __shared__ __attribute__((aligned(16))) uint8_t vbuf[2][kManyKeys * D * 2];
  __shared__ KeyMarks kmarks[4];
  __shared__ ValueMarks vmarks[3];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i32 = lane & 31, half = lane >> 5;
  const int b = blockIdx.y;
  int id = blockIdx.x;
  const int hk = id % a.pool.heads;
  id /= a.pool.heads;
  const int split = id % a.splits;
  id /= a.splits;
  const int group = a.q.heads / a.pool.heads, page = a.pool.page;
  const Seq seq = seq_of(a.pool, b);
  if (seq.news <= 0) return;
  const int rows = seq.news * group;
  const int piece = wave & 3;
  const float sc = fmaxf(fabsf(a.scale) * kLog2e, 1.2e-38f), grown = fminf(8.f / sc, 1e38f);

  // Tiles of rows from the last, which sees most, to the first.
  for (int tile = row_tiles - 1 - id; tile * kManyRows < rows; tile += row_tiles) {
    const int r = tile * kManyRows + wave * 32 + i32;
    const bool live = r < rows;
    const int t = min(r, rows - 1) / group;
    const int head = hk * group + min(r, rows - 1) % group;
    const Span sp = span_of(a, seq, t);
    const Span tile_first = span_of(a, seq, tile * kManyRows / group);
    const Span tile_last = span_of(a, seq, min(tile * kManyRows + kManyRows - 1, rows - 1) / group);
    const int w0 = min(tile * kManyRows + wave * 32, rows - 1), w1 = min(w0 + 31, rows - 1);
    const Span first = span_of(a, seq, w0 / group);
    const Span last = span_of(a, seq, w1 / group);
    const int lo = tile_first.lo & ~(kManyKeys - 1), hi = tile_last.hi;
    int each = (max(hi - lo, 0) + a.splits - 1) / a.splits;
    each = (each + kManyKeys - 1) & ~(kManyKeys - 1);
    const int s0 = lo + split * each, s1 = min(hi, s0 + each);

    // Q as the first product's B operand; a negative scale turns its sign.
    bf16x8_t qf[KS];
    {
      const u16* at = static_cast<const u16*>(a.q.p) + (int64_t)(seq.row0 + t) * a.q.ts + head * a.q.hs + half * 8;
      const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint4 w = *reinterpret_cast<const uint4*>(at + 16 * s);
        qf[s] = frag(w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip);
      }
    }
    f32x16_t o[NT];
#pragma unroll
    for (int f = 0; f < NT; ++f)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[f][e] = 0.f;
    float m = kNone, ms = 0.f, l = 0.f;  // maximum (unscaled), its scaled value (0 for none), sum

    // Tile t holds the keys from s0 + 64 t. Where this wave's 16 tokens of the
    // tiles t0 .. t0 + 63 lie: one tile a lane.
    const int tiles = (max(s1 - s0, 0) + kManyKeys - 1) / kManyKeys;
    uint64_t my_block = (uint64_t)a.pool.pages;
    uint32_t my_off = 0;
    uint64_t gone = 0;  // tiles whose page is none, or that are past the end
    int t0 = 0;
    auto find = [&](int t) {
      t0 = t;
      const int key = s0 + (t + lane) * kManyKeys + 16 * piece, pg = key / page;
      my_block = (uint64_t)a.pool.pages, my_off = 0;
      bool ok = key < s1 && pg < a.pool.max_pages;
      if (ok) {
        const int id = a.pool.table[(int64_t)b * a.pool.max_pages + pg];
        ok = (uint32_t)id < (uint32_t)a.pool.n_pages;
        if (ok) {
          my_block += id * a.pool.page_stride + hk * head_block_bytes(page, D);
          my_off = key - pg * page;
        }
      }
      gone = __ballot(!ok);
    };
    auto fetch_tile = [&](Raw<D>& r, bool is_v, int t) {
      if (t - t0 >= 64) find(t);
      const int i = t - t0;
      const uint32_t lo32 = __builtin_amdgcn_readlane((int)(uint32_t)my_block, i);
      const uint32_t hi32 = __builtin_amdgcn_readlane((int)(my_block >> 32), i);
      fetch<D>(r, is_v, reinterpret_cast<Global>((uint64_t)hi32 << 32 | lo32),
               __builtin_amdgcn_readlane((int)my_off, i), (gone >> i & 1) == 0, page, lane);
    };
    auto unpack_tile = [&](Raw<D>& r, bool is_v, int t) {
      unpack<D>(r, is_v, piece, kbuf[t % 3], vbuf[t & 1], &kmarks[t & 3], &vmarks[t % 3], lane);
    };

    auto fragment = [&](const uint8_t* at, int i) { return *reinterpret_cast<const bf16x8_t*>(at + i * 1024); };
    // S^T of half u of a tile: 32 keys.
    auto scores = [&](f32x16_t& s, int t, int u) {
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = 0.f;
      const uint8_t* at = kbuf[t % 3] + u * (KS * 1024) + lane * 16;
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        const bf16x8_t kf = fragment(at, q);
        s = mfma32(kf, qf[q], s);
      }
    };

    auto largest = [&](const f32x16_t& s) {
      float x = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) x = fmaxf(x, s[e]);
      return x;
    };

    // Half u of tile t: its scores `s` are there and mx is their largest of
    // this lane's; `n` gets those of the half after it meanwhile, and mx theirs.
    float mx = kNone;
    auto step = [&](f32x16_t& s, f32x16_t& n, int t, int u, bool odd) {
      const uint8_t* kat = kbuf[(u ? t + 1 : t) % 3] + (u ^ 1) * (KS * 1024) + lane * 16;
      bf16x8_t ring[RD];
#pragma unroll
      for (int q = 0; q < RD; ++q) ring[q] = fragment(kat, q);
      if (odd) {
        rare_path();
        const int j = s0 + t * kManyKeys + 32 * u;
        const uint32_t all = bits_between(sp.lo - j, sp.hi - j) & ~kmarks[t & 3].absent[u];
        const uint32_t seen = all >> (4 * half);
        const uint32_t nan = (kmarks[t & 3].nan[u] >> (4 * half)) & seen;
        // A NaN value is out of V, where it would reach every row: it enters
        // the sums of the rows that see it. Register e is of block e D / 512.
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          if (vmarks[t % 3].of[c][u] & all) {
#pragma unroll
            for (int f = 0; f < NT; ++f)
#pragma unroll
              for (int e = c * 512 / D; e < (c + 1) * 512 / D; ++e) o[f][e] = __builtin_nanf("");
          }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = 8 * (e >> 2) + (e & 3);
          const uint32_t keep = spread(seen, k);
          s[e] = __uint_as_float((__float_as_uint(s[e]) & keep) | (kNoneBits & ~keep) |
                                 (spread(nan, k) & kNanBits));
        }
        mx = largest(s);
      }
      // The maximum is only followed when a weight would pass 2^8: fp32 and
      // bf16 hold weights up to there as well as up to 1, and until then the
      // lanes need not agree on a new one and nothing is rescaled.
      if (__any(mx > m + grown)) {
        rare_path();
        const float mn = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32)));
        const float n0 = mn == kNone ? 0.f : mn * sc;
        const float al = m == kNone ? 0.f : __builtin_amdgcn_exp2f(ms - n0);
        m = mn, ms = n0;
        l *= al;
#pragma unroll
        for (int f = 0; f < NT; ++f)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[f][e] *= al;
      }
      // The next half's first product runs on the matrix unit while the vector
      // unit takes this one's exponentials: a matrix instruction holds its
      // unit for 32 clocks, in which a wave can issue up to seven others. They
      // are laid out in turns, and the fences keep matrix instructions and LDS
      // reads in this order, the latter RD fragments ahead of their use (at
      // last those of the second product); vector instructions may move.
      // (Past the last tile the first product is of old keys, and unused.)
      const uint8_t* vat = vbuf[t & 1] + 2 * u * (NT * 1024) + lane * 16;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pw[8];  // the weights, two keys a word
#pragma unroll
      for (int e = 0; e < 16; ++e) n[e] = 0.f;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        n = mfma32(ring[q % RD], qf[q], n);
        ring[q % RD] = q + RD < KS ? fragment(kat, q + RD) : fragment(vat, q + RD - KS);
#pragma unroll
        for (int e = q * 16 / KS; e < (q + 1) * 16 / KS; ++e) {
          s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], sc, -ms));
          sum[e & 3] += s[e];
          if (e & 1) pw[e >> 1] = pack_bf16(s[e - 1], s[e]);
        }
        __builtin_amdgcn_sched_barrier(kFence);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        const int g = i / NT, f = i % NT;
        o[f] = mfma32(ring[i % RD], frag(pw[4 * g], pw[4 * g + 1], pw[4 * g + 2], pw[4 * g + 3]), o[f]);
        if (i + RD < 2 * NT) ring[i % RD] = fragment(vat, i + RD);
        // the next half's maximum, beside the second product
#pragma unroll
        for (int e = i * 8 / NT; e < (i + 1) * 8 / NT; ++e) mx = e == 0 ? n[0] : fmaxf(mx, n[e]);
        __builtin_amdgcn_sched_barrier(kFence);
      }
    };
    auto wanted = [&](int t) {
      const int j = s0 + t * kManyKeys;
      return t < tiles && j < last.hi && j + kManyKeys > first.lo;
    };

    // Tile t is computed from keys t and t + 1 and values t; keys t + 2 and
    // values t + 1 are decoded meanwhile into the buffers that t - 1 has left,
    // and keys t + 3 and values t + 2 are on their way. Waves 0-3 decode keys,
    // first of all, and waves 4-7 values, last of all, so that the two of a
    // SIMD are not at the same work.
    const bool is_v = wave >= 4;
    __syncthreads();  // the last tile of rows is done with LDS
    if (threadIdx.x < 4) kmarks[threadIdx.x] = KeyMarks{};
    if (threadIdx.x < 3) vmarks[threadIdx.x] = ValueMarks{};
    __syncthreads();
    Raw<D> raw;
    f32x16_t sa, sb;
    if (tiles > 0) {
      find(0);
      fetch_tile(raw, is_v, 0);
      unpack_tile(raw, is_v, 0);
      fetch_tile(raw, is_v, 1);
      if (!is_v) {
        unpack_tile(raw, false, 1);
        fetch_tile(raw, false, 2);
      }
      __syncthreads();
      scores(sa, 0, 0);
      mx = largest(sa);
    }
    for (int t = 0; t < tiles; ++t) {
      __syncthreads();
      if (threadIdx.x == 0) {  // of tiles t + 3 and t + 2: read before this barrier, written after the next
        kmarks[(t + 3) & 3] = KeyMarks{};
        vmarks[(t + 2) % 3] = ValueMarks{};
      }
      if (!is_v && t + 2 < tiles) {
        unpack_tile(raw, false, t + 2);
        fetch_tile(raw, false, t + 3);
      }
      if (wanted(t)) {
        const KeyMarks km = kmarks[t & 3];
        const ValueMarks vm = vmarks[t % 3];
        const int j = s0 + t * kManyKeys;
        const bool odd = __builtin_amdgcn_readfirstlane(
            (km.absent[0] | km.absent[1] | km.nan[0] | km.nan[1] | vm.nan[0] | vm.nan[1]) != 0 ||
            j < last.lo || j + kManyKeys > first.hi);
        step(sa, sb, t, 0, odd);
        step(sb, sa, t, 1, odd);
      } else if (wanted(t + 1)) {
        scores(sa, t + 1, 0);
        mx = largest(sa);
      }
      if (is_v && t + 1 < tiles) {
        unpack_tile(raw, true, t + 1);
        fetch_tile(raw, true, t + 2);
      }
    }
    l += __shfl_xor(l, 32);
    if (!live) continue;
    const int64_t row = (int64_t)(seq.row0 + t) * a.q.heads + head;
    const float m2 = m == kNone ? kNone : ms;
    // lane (row, half): fragment f, register e is value NT (8 (e / 4) + 4 half + e % 4) + f
    if (a.splits > 1) {
      const int64_t at = (int64_t)split * a.pool.tokens * a.q.heads + row;
      if (half == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(m2, l);
      float* dst = a.part + at * D;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float* x = dst + NT * (8 * (e >> 2) + 4 * half + (e & 3));
        if constexpr (NT == 2) {
          *reinterpret_cast<float2*>(x) = make_float2(o[0][e], o[1][e]);
        } else {
#pragma unroll
          for (int f = 0; f < NT; f += 4)
            *reinterpret_cast<float4*>(x + f) = make_float4(o[f][e], o[f + 1][e], o[f + 2][e], o[f + 3][e]);
        }
      }
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (a.lse != nullptr && half == 0)
        a.lse[row] = l == 0.f ? kNone : (m2 + __builtin_amdgcn_logf(l)) * kLn2;
      const int64_t at = (int64_t)(seq.row0 + t) * a.o.ts + head * a.o.hs;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t x = at + NT * (8 * (e >> 2) + 4 * half + (e & 3));
#pragma unroll
        for (int f = 0; f < NT; f += 2)
          *reinterpret_cast<uint32_t*>(static_cast<u16*>(a.o.p) + x + f) =
              pack_bf16(o[f][e] * inv, o[f + 1][e] * inv);
      }
    }
  }
}

}  // namespace

hipError_t launch_attend_many(const AttnLaunch& a, hipStream_t s) {
  const AttnGrid g = attn_grid(a);
  const dim3 grid((uint32_t)(g.groups / a.pool.batch), a.pool.batch);
  if (a.pool.dim == 64)
    attend_many_kernel<64><<<grid, 64 * kManyWaves, 0, s>>>(a, (int)g.tiles);
  else
    attend_many_kernel<128><<<grid, 64 * kManyWaves, 0, s>>>(a, (int)g.tiles);
  return hipGetLastError();
}

}  // namespace tttk
