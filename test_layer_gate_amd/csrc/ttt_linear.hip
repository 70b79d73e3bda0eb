// gfx950 kernels of linear attention with a decay for each head:
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// in chunks on the matrix cores, and token by token.
//
// One chunked kernel serves the forward and, with the arguments in other
// roles, all three gradients. For rows of q, k (A values a head) and v (B):
//   o_i = s_in sum_{j <= i} g^(i - j) (q_i k_j) v_j + s_out g^(i + lead) E^T q_i
//   E'  = g^C E + s_up sum_j g^(C - lead - j) k_j v_j^T         (C rows on)
//   forward  (q, k, v),  lead 1, s = (scale, scale, 1),  E = S
//   dq       (do, v, k), the same with E = S^T
//   dk       (v, do, q), rows backwards, lead 0, s = (scale, 1, scale)
//   dv       (k, q, do), likewise; E: the gradient of the state behind a row,
//            times the rows' decays, from d_last on; its end is d_first
// Where query heads share a state (q for the forward and dq; k and v for dk
// and dv), the kernel goes over them within a chunk.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "ttt_attention.h"
#include "ttt_block.h"

namespace tttk {
namespace {

// What one launch of the chunked kernel takes.
struct Chunks {
  Rows q, k, v, o;
  const float* log_decay;
  const int32_t* starts;
  const float* state;           // E before a part's first row, or null: zeros
  float* out;                   // E after the last (or, for sums alone, the part's own)
  int64_t state_part, state_head, state_seq;  // strides of `state`, values; a part of 0: parts share one
  int64_t out_part, out_head, out_seq;
  int state_turned;             // state is [B][A]
  int batch, tokens, heads, parts, part_rows, slices;
  int lead, back;
  float s_in, s_out, s_up;
};

// Up to three of them in one launch, where they are of one kind: what one leaves
// idle while its first tiles are on their way, and when its last parts end,
// another uses. The parts of all follow each other by eights, one a die, so that
// what reads the same rows does so at about the same time.
struct Roles {
  Chunks c[3];
  int n;
};

// Tiles of rows in LDS, swizzled by 16-byte pieces. LDS takes a wave's 16-byte
// reads 16 lanes at a time, lanes 0-3, 12-15 and 20-27 first, then the other
// half of 32: in each of these groups one piece of every lane's row has to fall
// on another 16 bytes of the 256 of all banks. So do, for a transposing read,
// four neighbouring pieces of each of four neighbouring rows.
template <bool F32>
struct Elem {
  static constexpr int size = F32 ? 4 : 2;
  static constexpr int per16 = 16 / size;
  static constexpr int kb = F32 ? 8 : 16;       // contraction of one mma()
};

template <bool F32, int W>  // W values a row
struct Tile {
  static constexpr int pieces = W * Elem<F32>::size / 16;
  static constexpr __device__ __forceinline__ int swz(int row) {
    if constexpr (pieces >= 16)
      return ((row & 3) << 2) | ((row >> 2) & 3);
    else
      return ((row >> 1) & 3) | (((row >> 1) ^ (row >> 3)) & 1) << 2;
  }
  static __device__ __forceinline__ uint32_t at(int row, int piece) {
    return (uint32_t)(row * pieces + (piece ^ swz(row))) * 16;
  }
};

// c + a b over kb values of the contraction: one 32x32x16 product of bf16, or
// four 32x32x2 of fp32. A lane holds row (column) l % 32 and half of the
// contraction's values; which ones does not matter as long as both operands
// agree. They are chosen so that a product's result, whose lanes hold rows 8a +
// 4 (l / 32) + e, can be an operand of the next one from its registers: states
// and weights never leave them.
template <bool F32>
__device__ __forceinline__ f32x16_t mma(const uint4& a, const uint4& b, f32x16_t c) {
  if constexpr (F32) {
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  } else {
    return mfma32(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c);
  }
}

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// Where a lane reads a tile: byte offsets that further rows add to and further
// pieces are xored into (a row's pieces are a power of two, so a swizzled piece
// is the row's start xor the swizzle xor the piece). They are kept from being
// known across chunks: the compiler would hold an address for every read.
//
// For bf16, columns come turned: lane l has column l with bits 2 and 3
// exchanged. A product's rows, in such an order, are held with a lane's eight of
// every 16 as neighbours: what it meets next is one piece of 16 bytes, and so is
// what it stores.
template <bool F32>
__device__ __forceinline__ int column_of(int l) {
  return F32 ? l : (l & ~12) | (l & 4) << 1 | (l & 8) >> 1;
}
template <bool F32, int W>
struct Reader {
  static constexpr int row_bytes = W * Elem<F32>::size;
  static constexpr uint32_t eight = 16 * Tile<F32, W>::swz(8);  // what eight rows change in a piece's place
  uint32_t r, c[F32 ? 4 : 1];
  __device__ __forceinline__ Reader() {
    const int lane = threadIdx.x & 63, hf = lane >> 5;
    if constexpr (F32) {
      r = Tile<true, W>::at(lane & 31, hf);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = Tile<true, W>::at(4 * hf + e, (lane & 31) >> 2) + (lane & 3) * 4;
    } else {
      r = Tile<false, W>::at(lane & 31, hf);
      // a transposing read: lane 4e + j of 16 addresses four values of row e,
      // and lane i gets value i % 4 of lane i / 4's of the four rows
      const int e = (lane >> 2) & 3, j = lane & 3, k = (j >> 1) | (j & 1) << 1;
      c[0] = Tile<false, W>::at(4 * hf + e, 2 * ((lane >> 4) & 1) + (k >> 1)) + (k & 1) * 8;
    }
  }
  __device__ __forceinline__ void forget() {
    asm volatile("" : "+v"(r));
#pragma unroll
    for (int e = 0; e < (F32 ? 4 : 1); ++e) asm volatile("" : "+v"(c[e]));
  }
  // The lane's row 32 rt + l % 32 and of its values those of piece 2 kb + l / 32.
  __device__ __forceinline__ uint4 row(const char* tile, int rt, int kb) const {
    return *reinterpret_cast<const uint4*>(tile + 32 * rt * row_bytes + (r ^ (uint32_t)(kb * 32)));
  }
  // The lane's column of 32 from 32 cb (column_of(l % 32) of them) of the rows of
  // block kb.
  __device__ __forceinline__ uint4 col(const char* tile, int kb, int cb) const {
    const char* p = tile + Elem<F32>::kb * kb * row_bytes;
    if constexpr (F32) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = *reinterpret_cast<const uint32_t*>(p + (c[e] ^ (uint32_t)(cb * 128 ^ (kb & 1) * eight)));
      return make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const uint32_t at = c[0] ^ (uint32_t)(cb * 64);
      const s16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + at));
      const s16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + (at ^ eight) + 8 * row_bytes));
      const uint2 u = __builtin_bit_cast(uint2, x), w = __builtin_bit_cast(uint2, y);
      return make_uint4(u.x, u.y, w.x, w.y);
    }
  }
};

// x and y as T bf16 terms (each the rounding of what those before it leave), in
// pairs. What a rounding leaves is exact, and dot2 with (-1, 0) or (0, -1) gives
// it without unpacking the pair. (A NaN or an infinity of one of the two makes
// the other NaN: both go into the same sums.) The pairs are registers: the bits
// of (0, -1) are those of fp32's -1, which the compiler would put into the
// instruction as a constant that means another pair there.
template <int T>
__device__ __forceinline__ void terms(float x, float y, uint32_t (&w)[T]) {
  uint32_t low = 0x0000bf80u, high = 0xbf800000u;
  asm("" : "+s"(low), "+s"(high));
  w[0] = pack_bf16(x, y);
#pragma unroll
  for (int t = 1; t < T; ++t) {
    x = dot2(w[t - 1], low, x);
    y = dot2(w[t - 1], high, y);
    w[t] = pack_bf16(x, y);
  }
}

// Values of a product's result (kb of its rows) as an operand: fp32 as they
// are, bf16 as T terms.
template <bool F32, int T>
__device__ __forceinline__ void as_operand(const f32x16_t& x, int u, uint4 (&f)[T]) {
  if constexpr (F32) {
    f[0] = make_uint4(__float_as_uint(x[4 * u]), __float_as_uint(x[4 * u + 1]), __float_as_uint(x[4 * u + 2]),
                      __float_as_uint(x[4 * u + 3]));
  } else {
    uint32_t w[4][T];
#pragma unroll
    for (int e = 0; e < 4; ++e) terms<T>(x[8 * u + 2 * e], x[8 * u + 2 * e + 1], w[e]);
#pragma unroll
    for (int t = 0; t < T; ++t) f[t] = make_uint4(w[0][t], w[1][t], w[2][t], w[3][t]);
  }
}

// g^n for a whole n >= 0; 1 for n = 0 whatever g is.
__device__ __forceinline__ float power(float lg, int n) { return n == 0 ? 1.f : exp2f(lg * (float)n); }

// A tile on its way: its rows are loaded to registers (get) while the kernel
// works on others, and written to LDS (put) when their place is free. Rows
// from `count` on are zero; dir -1 goes backwards; heads count from the first
// one's.
template <bool F32, int W, int NT, int C>
struct Fetch {
  static constexpr int P = W * Elem<F32>::size / 16, R = NT / P;  // R rows at a time
  static constexpr int N = C / R;
  static_assert(NT % P == 0 && C % R == 0, "whole passes");
  uint4 v[N];
  const char* at;  // the lane's place in the next chunk, of the first head
  __device__ __forceinline__ Fetch(const Rows& x, int head, int col, int64_t row0, int dir)
      : at(static_cast<const char*>(x.p) +
           (head * x.hs + col + (row0 + (int)(threadIdx.x / P) * dir) * x.ts) * Elem<F32>::size + threadIdx.x % P * 16) {}
  __device__ __forceinline__ void on(const Rows& x, int rows) { at += rows * x.ts * Elem<F32>::size; }
  __device__ __forceinline__ void get(const Rows& x, int head, int dir, int count) {
    const int64_t step = x.ts * Elem<F32>::size * (dir * R);
    const char* p = at + head * x.hs * Elem<F32>::size;
    if (count >= C) {
#pragma unroll
      for (int i = 0; i < N; ++i, p += step) v[i] = *reinterpret_cast<const uint4*>(p);
    } else {
      const int r = threadIdx.x / P;
#pragma unroll
      for (int i = 0; i < N; ++i, p += step) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (r + i * R < count) v[i] = *reinterpret_cast<const uint4*>(p);
      }
    }
  }
  __device__ __forceinline__ void put(char* tile) const {
    const int r = threadIdx.x / P, c = threadIdx.x % P;
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<uint4*>(tile + Tile<F32, W>::at(r + i * R, c)) = v[i];
  }
};

// A barrier for what the waves share through LDS alone. __syncthreads() also
// waits for every load and store on its way to memory: those of the tiles that
// are fetched ahead, and of the rows that leave, would stand in the way of each.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Bound by the chain of a chunk's products, one after the other in a wave, with two
// waves a SIMD. 64k rows of 8/32 heads of 128 take 433 us, 87 of them the parts' sums:
// the outputs' launch keeps the matrix unit busy for 37% of its time and the vector
// unit for 36%, and its waves wait for their turn at either for 45% of theirs, for
// memory and barriers for 24%. Memory: 1.74 GB with the second pass over k and v and
// the parts' states, which a parallel form reads beyond the operator's own rows, 4.0
// TB/s; the sums 3.4 TB/s. The gradients of 2 x 8k rows of 16 heads take 278 us (matrix
// unit 34%, vector unit 35%), with the rows that several roles read in the caches.
//
// One part of a sequence's rows for one state head and a slice of NW * 32 of
// the B columns; wave w has columns 32 w .. of the slice, with its part of the
// state in registers (fp32, 16 values a lane for each 32 of A).
//
// MANY: heads of k and v share the state (else heads of q do). SUMS: the
// part's own sum alone, from zero.
//
// bf16: weights (q k) and states enter their products with v and q as two bf16
// terms (16 bits), so that what is left of a result's error is its own rounding:
// 2-norm error against 64 bits 0.0017, as of fp32 sums. (One term each: 0.0023, and
// 374 us for the prompt's 433; the state alone as two: 0.0018 and 415; three each:
// 501.) In the update, whose sums stay in fp32 from chunk to chunk, v times its
// decay is three terms (24 bits). fp32: the matrix cores' fp32 products throughout.
// FEW: a chunk is 32 rows of bf16, and weights and states are three terms (24 bits).
template <bool F32, int A, int NW, bool MANY, bool SUMS, bool FEW>
__global__ __launch_bounds__(NW * 64, A == 256 ? 1 : 2) void chunk_kernel(Roles roles, int first) {
  constexpr int C = F32 || FEW ? 32 : 64, KB = Elem<F32>::kb, NT = NW * 64, B = NW * 32;
  constexpr int RT = C / 32, AT = A / 32, PER = 32 / KB;
  constexpr int T = F32 ? 1 : FEW ? 3 : 2;  // terms of weights, and of a state that meets q
  constexpr int kBytesA = C * A * Elem<F32>::size, kBytesB = C * B * Elem<F32>::size;
  __shared__ __attribute__((aligned(16))) char kt[kBytesA];
  __shared__ __attribute__((aligned(16))) char vt[kBytesB];
  __shared__ __attribute__((aligned(16))) char qt[SUMS ? 16 : kBytesA];
  __shared__ __attribute__((aligned(16))) float up_f[C];
  __shared__ __attribute__((aligned(16))) int odd_from[SUMS ? 1 : NW][32];  // see take_odd
  constexpr int NB = RT * (RT + 1) / 2 * PER;  // pieces of a chunk's weights
  __shared__ uint4 shared[SUMS ? 1 : F32 ? 4 * NW : T * NB][64];
  Reader<F32, A> ra;
  Reader<F32, B> rb;

  const int group = first + blockIdx.x;
  const int eights = group / 8, turn = __builtin_amdgcn_readfirstlane(eights / roles.n);
  const Chunks& a = roles.c[eights - turn * roles.n];
  int id = turn * 8 + group % 8;
  const int slice = id % a.slices;
  id /= a.slices;
  const int part = id % a.parts;
  id /= a.parts;
  const int head = id % a.heads, seq = id / a.heads;
  if (seq >= a.batch) return;
  int64_t base, len;
  if (a.starts) {
    const int lo = min(max(a.starts[seq], 0), a.tokens), hi = min(max(a.starts[seq + 1], 0), a.tokens);
    base = lo, len = max(hi - lo, 0);
  } else {
    len = a.tokens / a.batch, base = seq * len;
  }
  // the last part takes what the others leave
  const int64_t mine = (int64_t)part * a.part_rows;
  const bool last = part == a.parts - 1 || mine + a.part_rows >= len;
  if (part > 0 && mine >= len) return;
  if (SUMS && last) return;  // (nobody reads it)
  const int64_t end = last ? len : mine + a.part_rows;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hf = lane >> 5, col = lane & 31;
  const int b0 = slice * B + wave * 32 + column_of<F32>(col);  // the lane's column of the state
  const int b_all = a.slices * B;
  // (the first loads before what is computed from the decay: it takes as long)
  const int q_heads = MANY ? 1 : a.q.heads / a.heads, k_heads = MANY ? a.k.heads / a.heads : 1;
  const int dir = a.back ? -1 : 1;
  int64_t t0 = mine;
  const int64_t row0 = a.back ? base + len - 1 - t0 : base + t0;
  int take = (int)min((int64_t)C, end - t0);
  Fetch<F32, A, NT, C> fk(a.k, head * k_heads, 0, row0, dir), fq(a.q, head * q_heads, 0, row0, dir);
  Fetch<F32, B, NT, C> fv(a.v, head * k_heads, slice * B, row0, dir);
  fk.get(a.k, 0, dir, take);
  fv.get(a.v, 0, dir, take);
  if constexpr (!SUMS) fq.get(a.q, 0, dir, take);
  char* o_at = static_cast<char*>(a.o.p) +
               (head * q_heads * a.o.hs + slice * B + wave * 32 + (row0 + col * dir) * a.o.ts) * Elem<F32>::size + 16 * hf;
  // value r of a lane's 16 of a state is row state_row(r) + state_hf of the 32
  auto state_row = [](int r) { return F32 ? 8 * (r >> 2) + (r & 3) : 16 * (r >> 3) + (r & 7); };
  const int state_hf = (F32 ? 4 : 8) * hf;
  f32x16_t st[AT];
  if (!SUMS && a.state != nullptr) {
    const float* e = a.state + seq * a.state_seq + head * a.state_head + part * a.state_part;
    if (a.state_turned) {
      e += (int64_t)b0 * A + state_hf;
#pragma unroll
      for (int t = 0; t < AT; ++t)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const float4 w = *reinterpret_cast<const float4*>(e + 32 * t + state_row(r));
          st[t][r] = w.x, st[t][r + 1] = w.y, st[t][r + 2] = w.z, st[t][r + 3] = w.w;
        }
    } else {
      e += (int64_t)state_hf * b_all + b0;
#pragma unroll
      for (int t = 0; t < AT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) st[t][r] = e[(32 * t + state_row(r)) * b_all];
    }
  } else {
#pragma unroll
    for (int t = 0; t < AT; ++t) st[t] = f32x16_t{};
  }

  __builtin_amdgcn_sched_barrier(0);

  const float lg = a.log_decay[head] * kLog2e;

  float row_f[RT];  // of the lane's row of x
#pragma unroll
  for (int it = 0; it < RT; ++it) row_f[it] = a.s_out * power(lg, 32 * it + col + a.lead);
  auto set_up = [&](int count) {
    for (int i = threadIdx.x; i < C; i += NT) up_f[i] = a.s_up * power(lg, max(count - a.lead - i, 0));
  };
  set_up(C);
  int up_for = C;
  // s_in g^(i - j) of 32 x 32 blocks on the diagonal (0 for j > i) and beside it,
  // as the lanes hold the weights
  __shared__ float4 decay[SUMS ? 1 : RT][4][64];
  if (!SUMS && wave < RT) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int n = 32 * wave + col - 8 * u - 4 * hf;
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = n < e ? 0.f : a.s_in * power(lg, max(n - e, 0));
      decay[SUMS ? 0 : wave][u][lane] = make_float4(f[0], f[1], f[2], f[3]);
    }
  }
  while (t0 < end) {
    ra.forget();
    rb.forget();

    // x of every row tile (column i: its row) = its product with the state before
    // the chunk
    auto with_state = [&](f32x16_t(&x)[RT]) {
      uint4 qf[2][RT];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int it = 0; it < RT; ++it) qf[kb][it] = ra.row(qt, it, kb);
#pragma unroll
      for (int it = 0; it < RT; ++it) x[it] = f32x16_t{};
#pragma unroll
      for (int kb = 0; kb < A / KB; ++kb) {
        uint4 sf[T];
        as_operand<F32, T>(st[kb / PER], kb % PER, sf);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int it = 0; it < RT; ++it) {
            x[it] = mma<F32>(sf[t], qf[kb & 1][it], x[it]);
            if (t == T - 1 && kb + 2 < A / KB) qf[kb & 1][it] = ra.row(qt, it, kb + 2);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto decay_rows = [&](f32x16_t(&x)[RT]) {
#pragma unroll
      for (int it = 0; it < RT; ++it)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[it][r] *= row_f[it];
    };
    // The weights of a chunk's rows (rows j of tile jt <= it, column i of tile it),
    // shared by the waves through LDS as the lanes will hold them: bf16 tiles a
    // wave each, decayed and in terms; of fp32's one tile, each wave a part of the
    // contraction over A.
    // (x, the product with the state, while the first ones are under way)
    auto weights_and_state = [&](bool state, f32x16_t(&x)[RT]) {
      if constexpr (F32) {
        constexpr int N = A / KB / NW;
        f32x16_t p = {};
#pragma unroll
        for (int n = 0; n < N; ++n) p = mma<true>(ra.row(kt, 0, wave * N + n), ra.row(qt, 0, wave * N + n), p);
        if (state) with_state(x);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          shared[wave * 4 + u][lane] = make_uint4(__float_as_uint(p[4 * u]), __float_as_uint(p[4 * u + 1]),
                                                  __float_as_uint(p[4 * u + 2]), __float_as_uint(p[4 * u + 3]));
      } else {
        constexpr int blocks = RT * (RT + 1) / 2;
        f32x16_t p = {};
        auto begin = [&](int b) {
          const char *kp = kt + 32 * (b > 1) * ra.row_bytes, *qp = qt + 32 * (b > 0) * ra.row_bytes;
          p = f32x16_t{};
          constexpr int D = 4;  // so many reads ahead: their latency is that of as many products
          uint4 kf[D], qf[D];
#pragma unroll
          for (int kb = 0; kb < D; ++kb) kf[kb] = ra.row(kp, 0, kb), qf[kb] = ra.row(qp, 0, kb);
#pragma unroll
          for (int kb = 0; kb < A / KB; ++kb) {
            p = mma<false>(kf[kb % D], qf[kb % D], p);
            if (kb + D < A / KB) kf[kb % D] = ra.row(kp, 0, kb + D), qf[kb % D] = ra.row(qp, 0, kb + D);
            __builtin_amdgcn_sched_barrier(0);
          }
        };
        auto finish = [&](int b) {
          const int d = b == 1;  // the block below the diagonal's
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float4 f = decay[SUMS ? 0 : d][u][lane];
            float w[4] = {f.x, f.y, f.z, f.w};
            asm("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));  // (no branches around their reads)
            // (a weight that is not taken may be a NaN)
            const int n = 32 * d + col - 8 * u - 4 * hf;
#pragma unroll
            for (int e = 0; e < 4; ++e) p[4 * u + e] = e > n ? 0.f : p[4 * u + e] * w[e];
          }
#pragma unroll
          for (int u = 0; u < PER; ++u) {
            uint4 w[T];
            as_operand<false, T>(p, u, w);
#pragma unroll
            for (int t = 0; t < T; ++t) shared[t * NB + b * PER + u][lane] = w[t];
          }
        };
        if (wave < blocks) begin(wave);
        if (state) with_state(x);
        if (wave < blocks) finish(wave);
        for (int b = wave + NW; b < blocks; b += NW) begin(b), finish(b);
      }
    };
    // x += those weights times v
    auto take_weights = [&](const uint4(&vf)[C / KB], f32x16_t(&x)[RT]) {
      if constexpr (F32) {
        if constexpr (!MANY) decay_rows(x);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 f = decay[0][u][lane];
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const uint4 p = shared[w * 4 + u][lane];
            s[0] += __uint_as_float(p.x), s[1] += __uint_as_float(p.y), s[2] += __uint_as_float(p.z), s[3] += __uint_as_float(p.w);
          }
          const float g[4] = {f.x, f.y, f.z, f.w};
          const int n = col - 8 * u - 4 * hf;  // (a weight that is not taken may be a NaN)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = e > n ? 0.f : s[e] * g[e];
          x[0] = mma<true>(vf[u], make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]), __float_as_uint(s[3])), x[0]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          uint4 w[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n) w[n] = shared[t * NB + n][lane];
          __builtin_amdgcn_sched_barrier(0);
          if (!MANY && t == 0) decay_rows(x);
#pragma unroll
          for (int kb = 0; kb < RT * PER; ++kb)
#pragma unroll
            for (int it = kb / PER; it < RT; ++it) x[it] = mma<false>(vf[kb], w[it * PER + kb], x[it]);
        }
      }
    };
    auto load_v = [&](uint4(&vf)[C / KB]) {
#pragma unroll
      for (int kb = 0; kb < C / KB; ++kb) vf[kb] = rb.col(vt, kb, wave);
    };
    // An infinity or a NaN in v times an earlier row's weight of 0 would be NaN.
    // Such values become 0 in the wave's columns, whose first rows that held one (C:
    // none) are kept in LDS. Whether there are any.
    auto take_odd = [&](uint4(&vf)[C / KB]) {
      uint32_t bits = 0;
#pragma unroll
      for (int kb = 0; kb < C / KB; ++kb) {
        const uint32_t w[4] = {vf[kb].x, vf[kb].y, vf[kb].z, vf[kb].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)  // (an exponent of all ones carries into the sign's place)
          bits |= F32 ? (w[e] & 0x7f800000u) + 0x00800000u : (w[e] & 0x7f807f80u) + 0x00800080u;
      }
      const bool odd = __any((bits & (F32 ? 0x80000000u : 0x80008000u)) != 0);
      if (odd) {
        int first = C;
#pragma unroll
        for (int kb = 0; kb < C / KB; ++kb) {
          uint32_t w[4] = {vf[kb].x, vf[kb].y, vf[kb].z, vf[kb].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int h = 0; h < (F32 ? 1 : 2); ++h) {
              const uint32_t all = F32 ? 0x7f800000u : h ? 0x7f800000u : 0x7f80u;
              const int row = KB * kb + (F32 ? e : 8 * (e >> 1) + 2 * (e & 1) + h);
              if ((w[e] & all) == all) first = min(first, row), w[e] &= F32 ? 0u : h ? 0xffffu : 0xffff0000u;
            }
          }
          vf[kb] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (first < C) first += 4 * hf;  // (rows of the lane's half)
        first = min(first, __shfl_xor(first, 32));
        odd_from[SUMS ? 0 : wave][col] = first;
      }
      return odd;
    };
    // NaN in the columns of x that take_odd found such a value in, from its row on.
    auto spoil = [&](f32x16_t(&x)[RT]) {
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int4 n = *reinterpret_cast<const int4*>(&odd_from[SUMS ? 0 : wave][2 * r + 4 * hf]);
        const int from[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int it = 0; it < RT; ++it)
            if (32 * it + col >= from[e]) x[it][r + e] = __builtin_nanf("");
      }
    };
    // Row tile `it` of a head's outputs.
    auto store = [&](int it, int q_head, const f32x16_t& x, int take) {
      if (32 * it + col >= take) return;
      char* to = o_at + (32 * it * dir * a.o.ts + q_head * a.o.hs) * Elem<F32>::size;
      if constexpr (F32) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<float4*>(to + 32 * u) = make_float4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 w[1];
          as_operand<false, 1>(x, u, w);
          *reinterpret_cast<uint4*>(to + 32 * u) = w[0];
        }
      }
    };
    // st += (k decayed)^T v of the chunk in LDS; what a block's products take is
    // read and computed beside those before it.
    auto update = [&](const uint4(&vf)[C / KB]) {
      constexpr int TU = F32 ? 1 : 3;  // terms
      uint4 u[2][TU], kf[2][AT];
      float4 f, g;
      auto read = [&](int kb, uint4(&kf)[AT]) {
        f = *reinterpret_cast<const float4*>(&up_f[KB * kb + 4 * hf]);
        if constexpr (!F32) g = *reinterpret_cast<const float4*>(&up_f[KB * kb + 8 + 4 * hf]);
#pragma unroll
        for (int t = 0; t < AT; ++t) kf[t] = ra.col(kt, kb, t);
        __builtin_amdgcn_sched_barrier(0);
      };
      auto ready = [&](int kb, uint4(&u)[TU]) {
        if constexpr (F32) {
          u[0] = make_uint4(__float_as_uint(__uint_as_float(vf[kb].x) * f.x), __float_as_uint(__uint_as_float(vf[kb].y) * f.y),
                            __float_as_uint(__uint_as_float(vf[kb].z) * f.z), __float_as_uint(__uint_as_float(vf[kb].w) * f.w));
        } else {
          const uint32_t w[4] = {vf[kb].x, vf[kb].y, vf[kb].z, vf[kb].w};
          const float m[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
          uint32_t z[4][TU];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            terms<TU>(__uint_as_float(w[e] << 16) * m[2 * e], __uint_as_float(w[e] & 0xffff0000u) * m[2 * e + 1], z[e]);
#pragma unroll
          for (int t = 0; t < TU; ++t) u[t] = make_uint4(z[0][t], z[1][t], z[2][t], z[3][t]);
        }
      };
      read(0, kf[0]);
      ready(0, u[0]);
#pragma unroll
      for (int kb = 0; kb < C / KB; ++kb) {
        if (kb + 1 < C / KB) {
          read(kb + 1, kf[(kb + 1) & 1]);
          ready(kb + 1, u[(kb + 1) & 1]);
        }
#pragma unroll
        for (int x = 0; x < TU; ++x)
#pragma unroll
          for (int t = 0; t < AT; ++t) st[t] = mma<F32>(kf[kb & 1][t], u[kb & 1][x], st[t]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // the next chunk's tiles, behind this one's `now` rows
    auto next = [&](int now) {
      t0 += now;
      // (a count of 0 behind the end: without a value of their own here, the
      // registers would be taken through the whole loop)
      take = (int)min((int64_t)C, end - t0);
      fk.on(a.k, now * dir);
      fv.on(a.v, now * dir);
      if constexpr (!SUMS) fq.on(a.q, now * dir);
      fk.get(a.k, 0, dir, take);
      fv.get(a.v, 0, dir, take);
      if constexpr (!SUMS) fq.get(a.q, 0, dir, take);
      __builtin_amdgcn_sched_barrier(0);
    };
    const int now = take;
    uint4 vf[C / KB];
    lds_barrier();  // (the tiles' last readers are done)
    fk.put(kt);
    fv.put(vt);
    if constexpr (!SUMS) fq.put(qt);
    lds_barrier();
    if (now != up_for) {
      set_up(now);
      up_for = now;
      lds_barrier();
    }
    const float g = power(lg, now);
    if constexpr (!MANY) {
      // k and v once, heads of q in turn
      load_v(vf);
      if constexpr (!SUMS) {
        f32x16_t x[RT];
        const bool odd = take_odd(vf);
        int h = 0;
        for (; h + 1 < q_heads; ++h) {
          fq.get(a.q, h + 1, dir, now);
          __builtin_amdgcn_sched_barrier(0);
          // (so that the state's conversion stays inside the loop: kept over the
          // heads it would take as many registers again)
#pragma unroll
          for (int t = 0; t < AT; ++t) asm volatile("" : "+v"(st[t]));
          weights_and_state(true, x);
          lds_barrier();
          fq.put(qt);
          take_weights(vf, x);
          if (odd) spoil(x);
#pragma unroll
          for (int it = 0; it < RT; ++it) store(it, h, x[it], now);
          lds_barrier();
        }
        next(now);
        weights_and_state(true, x);
        lds_barrier();
        take_weights(vf, x);
        if (odd) spoil(x), load_v(vf);
#pragma unroll
        for (int it = 0; it < RT; ++it) store(it, h, x[it], now);
      } else {
        next(now);
      }
#pragma unroll
      for (int t = 0; t < AT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) st[t][r] *= g;
      update(vf);
    } else {
      // q once, heads of k and v in turn
      f32x16_t x[RT];
      if constexpr (!SUMS) {
        with_state(x);
        decay_rows(x);
      }
#pragma unroll
      for (int t = 0; t < AT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) st[t][r] *= g;
      for (int h = 0; h < k_heads; ++h) {
        if (h > 0) {
          lds_barrier();
          fk.put(kt);
          fv.put(vt);
          lds_barrier();
        }
        load_v(vf);
        if constexpr (!SUMS) {
          const bool odd = take_odd(vf);
          weights_and_state(false, x);
          lds_barrier();
          take_weights(vf, x);
          if (odd) spoil(x), load_v(vf);
        }
        const int more = h + 1 < k_heads ? now : 0;
        fk.get(a.k, h + 1, dir, more);
        fv.get(a.v, h + 1, dir, more);
        __builtin_amdgcn_sched_barrier(0);
        update(vf);
      }
      next(now);
      if constexpr (!SUMS) {
#pragma unroll
        for (int it = 0; it < RT; ++it) store(it, 0, x[it], now);
      }
    }
    o_at += now * dir * a.o.ts * Elem<F32>::size;
  }

  if (a.out != nullptr && (SUMS || last)) {
    float* e = a.out + seq * a.out_seq + head * a.out_head + part * a.out_part + (int64_t)state_hf * b_all + b0;
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) e[(32 * t + state_row(r)) * b_all] = st[t][r];
  }
}

// The states before every part from the parts' own sums, in their place: E_0
// is the state before the sequence (or zero), E_{p+1} = g^rows E_p + U_p.
constexpr int kScanThreads = 256, kScanAhead = 8;
struct Scan {
  float* sums;
  const float* first;
};
__global__ __launch_bounds__(kScanThreads) void scan_kernel(Scan one, Scan two, const float* log_decay,
                                                            const int32_t* starts, int batch, int tokens, int heads,
                                                            int parts, int part_rows, int size) {
  const int blocks = size / (4 * kScanThreads);
  float* const sums = blockIdx.y == 0 ? one.sums : two.sums;
  const float* const first = blockIdx.y == 0 ? one.first : two.first;
  const int64_t sh = blockIdx.x / blocks;
  const int i = ((blockIdx.x % blocks) * kScanThreads + threadIdx.x) * 4;
  const int seq = (int)(sh / heads), head = (int)(sh % heads);
  int64_t len = tokens / batch;
  if (starts) {
    const int lo = min(max(starts[seq], 0), tokens), hi = min(max(starts[seq + 1], 0), tokens);
    len = max(hi - lo, 0);
  }
  const float g = power(log_decay[head] * kLog2e, part_rows);
  float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
  if (first) e = *reinterpret_cast<const float4*>(first + sh * size + i);
  float* p = sums + sh * parts * size + i;
  // of these parts the sums are read, several at once; the one behind them only
  // gets its state
  const int whole = (int)min((int64_t)(parts - 1), max((len - 1) / part_rows, (int64_t)0));
  for (int n = 0; n < whole; n += kScanAhead) {
    float4 u[kScanAhead];
#pragma unroll
    for (int j = 0; j < kScanAhead; ++j)
      if (n + j < whole) u[j] = *reinterpret_cast<const float4*>(p + (int64_t)j * size);
#pragma unroll
    for (int j = 0; j < kScanAhead; ++j)
      if (n + j < whole) {
        *reinterpret_cast<float4*>(p) = e;
        e = make_float4(g * e.x + u[j].x, g * e.y + u[j].y, g * e.z + u[j].z, g * e.w + u[j].w);
        p += size;
      }
  }
  *reinterpret_cast<float4*>(p) = e;
}

// A few tokens a sequence: the state's slice of SB columns is read once, kept
// in registers over the tokens, and written once: bound by HBM. Eight lanes
// hold 32 neighbouring columns of a row of the state; 32 rows at a time. A token
// of 48 sequences, 8/32 heads of 128: 12.3 us for 51 MB, 4.2 TB/s.
constexpr int kTokenColumns = 32;
template <bool F32, int A, int G>
__global__ __launch_bounds__(256) void token_kernel(LinearLaunch a, int first) {
  constexpr int SB = kTokenColumns, R = A / 32;
  __shared__ float kq[(1 + G) * A], vv[SB];
  __shared__ float4 red[4][G][8];
  const int slices = a.dv / SB;
  int id = first + blockIdx.x;
  const int slice = id % slices;
  id /= slices;
  const int head = id % a.kv_heads, seq = id / a.kv_heads;
  int64_t base, len;
  if (a.starts) {
    const int lo = min(max(a.starts[seq], 0), a.tokens), hi = min(max(a.starts[seq + 1], 0), a.tokens);
    base = lo, len = max(hi - lo, 0);
  } else {
    len = a.tokens / a.batch, base = seq * len;
  }
  const int group = a.q.heads / a.kv_heads;
  const int c4 = threadIdx.x & 7, row = threadIdx.x >> 3;
  const int64_t at = ((int64_t)(seq * a.kv_heads + head) * A + row) * a.dv + slice * SB + c4 * 4;
  float4 st[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    st[r] = a.first ? *reinterpret_cast<const float4*>(a.first + at + (int64_t)r * 32 * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float g = power(a.log_decay[head] * kLog2e, 1);
  auto value = [](const Rows& x, int64_t i) {
    return F32 ? static_cast<const float*>(x.p)[i] : bf16_f32(static_cast<const u16*>(x.p)[i]);
  };
  for (int64_t t = 0; t < len; ++t) {
    const int64_t n = base + t;
    for (int h0 = 0; h0 < group; h0 += G) {
      __syncthreads();
      for (int i = threadIdx.x; i < A; i += 256) {
        if (h0 == 0) kq[i] = value(a.k, n * a.k.ts + head * a.k.hs + i);
#pragma unroll
        for (int x = 0; x < G; ++x)
          if (h0 + x < group) kq[(1 + x) * A + i] = value(a.q, n * a.q.ts + (head * group + h0 + x) * a.q.hs + i);
      }
      if (h0 == 0 && threadIdx.x < SB) vv[threadIdx.x] = value(a.v, n * a.v.ts + head * a.v.hs + slice * SB + threadIdx.x);
      __syncthreads();
      if (h0 == 0) {
        const float4 v = *reinterpret_cast<const float4*>(&vv[c4 * 4]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float k = kq[row + 32 * r];
          st[r] = make_float4(g * st[r].x + k * v.x, g * st[r].y + k * v.y, g * st[r].z + k * v.z, g * st[r].w + k * v.w);
        }
      }
#pragma unroll
      for (int x = 0; x < G; ++x) {
        if (h0 + x >= group) break;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float q = kq[(1 + x) * A + row + 32 * r];
          o.x += q * st[r].x, o.y += q * st[r].y, o.z += q * st[r].z, o.w += q * st[r].w;
        }
#pragma unroll
        for (int m = 8; m < 64; m <<= 1)
          o.x += __shfl_xor(o.x, m), o.y += __shfl_xor(o.y, m), o.z += __shfl_xor(o.z, m), o.w += __shfl_xor(o.w, m);
        if ((threadIdx.x & 63) < 8) red[threadIdx.x >> 6][x][c4] = o;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < G * SB; i += 256) {
        const int x = i / SB, c = i % SB;
        if (h0 + x < group) {
          float o = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) o += reinterpret_cast<const float*>(&red[w][x][0])[c];
          o *= a.scale;
          const int64_t to = n * a.o.ts + (head * group + h0 + x) * a.o.hs + slice * SB + c;
          if constexpr (F32)
            static_cast<float*>(a.o.p)[to] = o;
          else
            static_cast<u16*>(a.o.p)[to] = bf16_rne(o);
        }
      }
    }
  }
  if (a.last) {
#pragma unroll
    for (int r = 0; r < R; ++r) *reinterpret_cast<float4*>(a.last + at + (int64_t)r * 32 * a.dv) = st[r];
  }
}

__global__ __launch_bounds__(256) void through_kernel(const float* from, float* to, int64_t n4) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256)
    reinterpret_cast<float4*>(to)[i] = from ? reinterpret_cast<const float4*>(from)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
}

// Zeros for the gradients of rows that no sequence claims: those before the first
// start and from the last one on (what lies between is within a sequence, whatever
// the starts between them are). Ahead of the gradients' own launches: of starts out
// of order it may write more. A few us where there are none.
struct Outside {
  Rows x[3];
  int dim[3];
  const int32_t* starts;
  int batch, tokens, size;      // size: bytes of a value
};
__global__ __launch_bounds__(256) void outside_kernel(Outside a) {
  const int lo = min(max(a.starts[0], 0), a.tokens), hi = min(max(a.starts[a.batch], 0), a.tokens);
  const int rows = lo + a.tokens - hi;
  for (int n = blockIdx.x; n < rows; n += gridDim.x) {
    const int64_t row = n < lo ? n : n - lo + hi;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const Rows& x = a.x[i];
      const int per = a.dim[i] * a.size / 16;
      for (int e = threadIdx.x; e < x.heads * per; e += 256)
        *reinterpret_cast<uint4*>(static_cast<char*>(x.p) + (row * x.ts + e / per * x.hs) * a.size + e % per * 16) =
            make_uint4(0, 0, 0, 0);
    }
  }
}

template <bool F32, bool MANY, bool SUMS, bool FEW>
hipError_t chunks_of(const Roles& r, int A, int B, hipStream_t s) {
  const Chunks& a = r.c[0];
  int64_t n = (int64_t)a.batch * a.heads * a.parts * a.slices;
  if (r.n > 1) n = (n + 7) / 8 * 8 * r.n;
  in_pieces(n, [&](uint32_t g, int64_t at) {
    const int first = (int)at;  // (n is below 2^25)
    if (B == 64) {
      if (A == 64) chunk_kernel<F32, 64, 2, MANY, SUMS, FEW><<<g, 128, 0, s>>>(r, first);
      else if (A == 128) chunk_kernel<F32, 128, 2, MANY, SUMS, FEW><<<g, 128, 0, s>>>(r, first);
      else chunk_kernel<F32, 256, 2, MANY, SUMS, FEW><<<g, 128, 0, s>>>(r, first);
    } else {
      if (A == 64) chunk_kernel<F32, 64, 4, MANY, SUMS, FEW><<<g, 256, 0, s>>>(r, first);
      else if (A == 128) chunk_kernel<F32, 128, 4, MANY, SUMS, FEW><<<g, 256, 0, s>>>(r, first);
      else chunk_kernel<F32, 256, 4, MANY, SUMS, FEW><<<g, 256, 0, s>>>(r, first);
    }
  });
  return hipGetLastError();
}

// (all of the same parts and slices)
template <bool MANY, bool SUMS>
hipError_t chunks(std::initializer_list<Chunks> c, int A, int B, bool f32, hipStream_t s) {
  Roles r = {};
  for (const Chunks& x : c) r.c[r.n++] = x;
  return f32 ? chunks_of<true, MANY, SUMS, false>(r, A, B, s) : chunks_of<false, MANY, SUMS, false>(r, A, B, s);
}

int slices_of(int B) { return B == 256 ? 2 : 1; }

Chunks base_of(const LinearLaunch& a, int B) {
  Chunks c = {};
  c.log_decay = a.log_decay, c.starts = a.starts;
  c.batch = a.batch, c.tokens = a.tokens, c.heads = a.kv_heads, c.parts = a.parts, c.part_rows = a.part_rows;
  c.slices = slices_of(B);
  const int64_t size = (int64_t)a.dk * a.dv;
  c.state_head = c.out_head = size, c.state_seq = c.out_seq = size * a.kv_heads;
  return c;
}

// The same rows' launch for the parts' own sums, in `sums`.
Chunks sums_of(Chunks c, const LinearLaunch& a, float* sums) {
  const int64_t size = (int64_t)a.dk * a.dv;
  c.out = sums, c.out_part = size, c.out_head = size * a.parts, c.out_seq = c.out_head * a.kv_heads;
  return c;
}
hipError_t scan(const LinearLaunch& a, int n, Scan one, Scan two, hipStream_t s) {
  const int size = a.dk * a.dv;
  const dim3 g((uint32_t)((int64_t)a.batch * a.kv_heads * (size / (4 * kScanThreads))), (uint32_t)n);
  scan_kernel<<<g, kScanThreads, 0, s>>>(one, two, a.log_decay, a.starts, a.batch, a.tokens, a.kv_heads, a.parts,
                                         a.part_rows, size);
  return hipGetLastError();
}

// Where the states before a part are: in `sums`, or with one part the first.
void states_from(Chunks* c, const LinearLaunch& a, const float* first, const float* sums) {
  if (a.parts == 1) {
    c->state = first;
    return;
  }
  const int64_t size = (int64_t)a.dk * a.dv;
  c->state = sums, c->state_part = size, c->state_head = size * a.parts, c->state_seq = c->state_head * a.kv_heads;
}

template <bool F32, int G>
hipError_t tokens_of(const LinearLaunch& a, hipStream_t s) {
  in_pieces((int64_t)a.batch * a.kv_heads * (a.dv / kTokenColumns), [&](uint32_t g, int64_t at) {
    const int first = (int)at;  // (at most 2^25 of them)
    if (a.dk == 64) token_kernel<F32, 64, G><<<g, 256, 0, s>>>(a, first);
    else if (a.dk == 128) token_kernel<F32, 128, G><<<g, 256, 0, s>>>(a, first);
    else token_kernel<F32, 256, G><<<g, 256, 0, s>>>(a, first);
  });
  return hipGetLastError();
}

}  // namespace

// Token by token for a few rows a sequence, whose state is read and written by any
// kernel: its time grows by the row, a chunk's does not. Measured, us (token by
// token for 2, 3, 4, 6 and 8 rows a sequence; a chunk of 32 rows):
//   8/32 heads of 128, one sequence   6.8,  8.6, 10.4, 14.0, 17.7; 14.7
//   8/32 heads of 128, 48            15.6, 22.3, 28.9, 38.9, 48.8; 23.0
//   16/16 heads of 128, one           4.6,  5.2,  6.0,  7.4,  9.0;  9.2
//   16/16 heads of 128, 48           20.8, 22.6, 25.0, 30.3, 35.6; 26.5
//   8/16 heads of 256, 48            38.1, 42.9, 45.2, 54.0, 64.0; 66.5
//   8/32 heads of 128, fp32, one      6.7,  8.5, 10.2, 13.7, 17.6; 23.5
//   8/32 heads of 128, fp32, 48      17.5, 24.4, 31.0, 39.6, 49.4; 40.7
// so up to 6 rows, but where there are more than two workgroups a compute unit, and
// a chunk is faster (bf16, and two of its workgroups to a unit), up to 3.
bool linear_by_token(const LinearLaunch& a) {
  const int64_t groups = (int64_t)a.batch * a.kv_heads * (a.dv / kTokenColumns);
  return a.max_new <= (a.f32 || a.dk == 256 || groups <= 512 ? 6 : 3);
}

// Rows a sequence up to which bf16 takes a chunk of 32 rows and three terms: fp32's
// precision, and for one sequence of 8/32 heads of 128 14.7 us for the 16.8 of a
// chunk of 64 and two terms, for 48 22.8 for 25.2.
constexpr int kFewRows = 32;

// Parts of the sequences: as many workgroups as have a place at once, two a
// compute unit (of two waves for dim_v 64, else of four; one where dim_k is 256 and
// the state takes the registers of two), of a chunk at least. The parts' states
// cost a read or write of their own each, so that the gradients, whose launches
// have two or three roles, take half as many, whatever the heads. Measured, us:
//   64k rows, 8/32 heads of 128:          1024 parts 477, 512 457, 256 510
//   4 x 8k rows, 16 heads of 64:          2048 parts 120, 1024 118, 512 123
//   8k rows, 4 heads of 256:              512 parts 112, 256 90, 128 116
//   gradients of 2 x 8k rows, 16 of 128:  512 parts 305, 256 285, 128 317
//   gradients of 8k rows, 4/16 of 256:    256 parts 394, 128 494
//   2048 rows, 8/32 heads of 128: parts of one chunk 37, of two 43, of four 66
void linear_parts(LinearLaunch* a, bool back) {
  const int rows = a->f32 ? 32 : 64;
  const int64_t states = (int64_t)a->batch * a->kv_heads * slices_of(a->dv);
  const int64_t places = (a->dv == 64 ? 1024 : 512) / (back || a->dk == 256 ? 2 : 1);
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(places / states, a->max_new / rows));
  a->part_rows = (int)((((int64_t)a->max_new + parts - 1) / parts + rows - 1) / rows * rows);
  a->parts = (int)(((int64_t)a->max_new + a->part_rows - 1) / a->part_rows);
}

hipError_t launch_linear(const LinearLaunch& a, hipStream_t s) {
  if (linear_by_token(a)) {
    const int group = a.q.heads / a.kv_heads;
    if (group == 1) return a.f32 ? tokens_of<true, 1>(a, s) : tokens_of<false, 1>(a, s);
    return a.f32 ? tokens_of<true, 4>(a, s) : tokens_of<false, 4>(a, s);
  }
  Chunks c = base_of(a, a.dv);
  c.q = a.q, c.k = a.k, c.v = a.v, c.o = a.o;
  c.lead = 1, c.s_in = c.s_out = a.scale, c.s_up = 1.f;
  hipError_t e;
  if (a.parts > 1 && ((e = chunks<false, true>({sums_of(c, a, a.sums)}, a.dk, a.dv, a.f32, s)) != hipSuccess ||
                      (e = scan(a, 1, {a.sums, a.first}, {}, s)) != hipSuccess))
    return e;
  states_from(&c, a, a.first, a.sums);
  c.out = a.last;
  if (!a.f32 && a.max_new <= kFewRows) return chunks_of<false, false, false, true>({{c}, 1}, a.dk, a.dv, s);
  return chunks<false, false>({c}, a.dk, a.dv, a.f32, s);
}

hipError_t launch_linear_backward(const LinearBackLaunch& b, hipStream_t s) {
  const LinearLaunch& a = b.f;
  const bool many = a.q.heads > a.kv_heads;
  hipError_t e;
  if (a.starts) {
    const Outside o = {{b.dq, b.dk, b.dv}, {a.dk, a.dk, a.dv}, a.starts, a.batch, a.tokens, a.f32 ? 4 : 2};
    outside_kernel<<<std::min(a.tokens, 512), 256, 0, s>>>(o);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  // the states before each part, and the gradients of those behind each part
  Chunks f = base_of(a, a.dv), r = f;
  f.k = a.k, f.v = a.v;
  f.lead = 1, f.s_in = f.s_out = a.scale, f.s_up = 1.f;
  r.k = a.q, r.v = b.d_o;
  r.lead = 0, r.back = 1, r.s_in = a.scale, r.s_out = 1.f, r.s_up = a.scale;
  if (a.parts > 1) {
    const Chunks u = sums_of(f, a, a.sums), w = sums_of(r, a, b.back_sums);
    if (many) {
      if ((e = chunks<false, true>({u}, a.dk, a.dv, a.f32, s)) != hipSuccess) return e;
      e = chunks<true, true>({w}, a.dk, a.dv, a.f32, s);
    } else {
      e = chunks<false, true>({u, w}, a.dk, a.dv, a.f32, s);
    }
    if (e != hipSuccess || (e = scan(a, 2, {a.sums, a.first}, {b.back_sums, b.d_last}, s)) != hipSuccess) return e;
  }
  states_from(&f, a, a.first, a.sums);
  states_from(&r, a, b.d_last, b.back_sums);
  Chunks q = f, k = r, v = r;
  q.slices = k.slices = slices_of(a.dk);
  q.q = b.d_o, q.k = a.v, q.v = a.k, q.o = b.dq, q.state_turned = 1;
  k.q = a.v, k.k = b.d_o, k.v = a.q, k.o = b.dk, k.state_turned = 1;
  v.q = a.k, v.o = b.dv, v.out = b.d_first;
  // (dv's writes d_first, which may be d_last: with one part the others read that
  // at the same time)
  const bool with_v = a.dk == a.dv && (a.parts > 1 || b.d_first == nullptr || b.d_first != b.d_last);
  if (many) {
    if ((e = chunks<false, false>({q}, a.dv, a.dk, a.f32, s)) != hipSuccess) return e;
    if (with_v) return chunks<true, false>({k, v}, a.dv, a.dk, a.f32, s);
    if ((e = chunks<true, false>({k}, a.dv, a.dk, a.f32, s)) != hipSuccess) return e;
    return chunks<true, false>({v}, a.dk, a.dv, a.f32, s);
  }
  if (with_v) return chunks<false, false>({q, k, v}, a.dv, a.dk, a.f32, s);
  if ((e = chunks<false, false>({q, k}, a.dv, a.dk, a.f32, s)) != hipSuccess) return e;
  return chunks<false, false>({v}, a.dk, a.dv, a.f32, s);
}

hipError_t launch_linear_through(const LinearBackLaunch& b, hipStream_t s) {
  const int64_t n4 = (int64_t)b.f.batch * b.f.kv_heads * b.f.dk * b.f.dv / 4;
  if (b.d_first == b.d_last) return hipSuccess;
  through_kernel<<<(uint32_t)std::min<int64_t>((n4 + 255) / 256, 4096), 256, 0, s>>>(b.d_last, b.d_first, n4);
  return hipGetLastError();
}

}  // namespace tttk
