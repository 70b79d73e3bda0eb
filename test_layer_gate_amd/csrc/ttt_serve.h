// Host-side launchers of the attention half of a decoder block (rotary
// positions, the paged 4-bit cache and attention over it) and the argument
// structs their kernels take; internal to libttt_layer. Every launcher
// enqueues on `s` and returns hipGetLastError().
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tttk {

// Rows of heads: element (token n, head h, i) at p[n * ts + h * hs + i].
struct Rows {
  void* p;
  int64_t ts, hs;
  int heads;
};

struct RopeArgs {
  const float* table;    // [max_pos][rot / 2][2]: cos, sin
  int rot, max_pos, interleaved;
  float sign;            // 1: rotate; -1: its transpose
};

struct RopeLaunch {
  Rows x[2], y[2];       // two tensors of heads (the second may have none)
  int tokens, dim, seq_len;
  const int32_t* positions;  // [tokens], or null: token % seq_len
  RopeArgs rope;
  bool f32;
};

// The page pool and who owns which page. Inside a page each head has its own
// block of page * (D + D / 16) bytes:
//   K codes   [page][D / 2]            byte j: value 2j (low), 2j + 1 (high)
//   V codes   [page / 4][D / 8][4][4]  of four tokens, 8 values of each
//   K scales  [page][D / 32]
//   V scales  [D / 32][page]
// Keys keep a token's values together: one lane's 16 bytes are one block of
// 32 values, the MFMA's contraction runs along them. Values keep four
// tokens' 8 values together: the second product contracts over tokens, and
// 16 bytes then hold what one lane contributes.
struct Pool {
  uint8_t* pages;
  int64_t page_stride;
  const int32_t* table;  // [batch][max_pages]
  const int32_t* lens;   // [batch] tokens, the new ones included
  const int32_t* starts; // [batch + 1] first new row of each, or null: tokens / batch each
  int batch, max_pages, n_pages, page, heads, dim, tokens;
};

struct AppendLaunch {
  Pool pool;
  Rows q, qo, k, v;      // q.heads may be 0
  RopeArgs rope;         // rot 0: no rotation
  const int32_t* positions;  // [tokens], or null: the index in the sequence
  bool f32;
};

struct ReadLaunch {
  Pool pool;
  Rows k, v;
  bool f32;
};

struct AttnLaunch {
  Pool pool;
  Rows q, o;
  float* lse;            // [tokens][q heads], or null
  float scale;
  int causal, window, max_new, max_kv;
  bool f32;
  bool many;             // attn_plan()
  int splits, each, slices, tile;
  float* part;           // [splits][tokens * q heads][D] (splits > 1), or
                         // [slices + batch - 1][kv heads][tile][D] (slices > 0)
  float* part_ml;        // likewise, [2] for [D]
  int* part_of;          // [tokens * q heads][2]: a row's first part, and how many (slices > 0)
};

hipError_t launch_rope(const RopeLaunch& a, hipStream_t s);
hipError_t launch_rope_table(float* table, int max_pos, int rot, double base, int kind,
                             double factor, double orig, double lo, double hi, double mul,
                             hipStream_t s);
hipError_t launch_append(const AppendLaunch& a, hipStream_t s);
hipError_t launch_read(const ReadLaunch& a, hipStream_t s);
// Tokens that a sequence may have: sums of two places among them stay in 32 bits.
constexpr int64_t kMaxKeys = (int64_t)1 << 30;
// How attention is launched: by which kernel, in how many parts of each
// sequence's keys, and for the few-row kernel in stretches of how many keys
// (part s takes every splits-th stretch from the s-th). slices > 0: the keys of
// all sequences, one after the other, are cut into that many even slices.
struct AttnPlan {
  bool many;
  int splits, each, slices;
  int tile;  // rows a wave of the few-row kernel takes
};
AttnPlan attn_plan(int batch, int kv_heads, int q_heads, int max_new, int max_kv, int window, bool f32,
                   int dim);
constexpr int kManyTile = 256;  // rows of a workgroup of the many-row kernel
// The workgroups of the launch (from its pool's sizes, the query heads, max_new
// and the plan), how many tiles of rows a sequence gets, and the waves of a
// workgroup.
struct AttnGrid {
  int64_t groups, tiles;
  int waves;
};
AttnGrid attn_grid(const AttnLaunch& a);
hipError_t launch_attention(const AttnLaunch& a, hipStream_t s);
hipError_t launch_attend_many(const AttnLaunch& a, hipStream_t s);
hipError_t launch_attention_join(const AttnLaunch& a, hipStream_t s);

}  // namespace tttk
