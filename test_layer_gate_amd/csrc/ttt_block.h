// Host-side launchers of the operators around and beside a decoder block (the
// norms of its residual stream, linear attention, the AdamW step) and the
// argument structs their kernels take; internal to libttt_layer. Every
// launcher enqueues on `s` and returns hipGetLastError().
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_serve.h"

namespace tttk {

// Workgroups of one launch, of up to 1024 threads: a launch holds fewer than 2^32
// threads. More of them are launched one after the other: f(workgroups, first).
constexpr int64_t kMostGroups = (int64_t)1 << 21;
template <class F>
void in_pieces(int64_t groups, const F& f) {
  for (int64_t at = 0; at < groups; at += kMostGroups)
    f((uint32_t)(groups - at < kMostGroups ? groups - at : kMostGroups), at);
}

// ------------------------------------------------------------------ norms

// Rows of one head: row n of a view at p + n * ts elements.
struct NormLaunch {
  Rows x, f, gate, r, h;        // a part that is not taken has no p
  const void *post, *pre;       // weights [d], or null: ones
  int rows, d, per_gate;        // rows that share a gate
  float scale, eps;
  bool norm_post, norm_pre;
  bool act_f32, res_f32, w_f32;
};

struct NormBackLaunch {
  NormLaunch n;                 // x: the stored sums; r, h unused
  Rows dr, dh, dx, df, dgate;   // dgate: [gates][d] fp32 where rows share one
  float *dpost, *dpre;          // [d], or null
  float *part_post, *part_pre, *part_gate;  // workspace, see NormPlan
};
// How the backward's rows are dealt out. Workgroup w takes rows [w * each,
// ..) of its own, or, where rows share a gate and slices > 1, slice w % slices
// of gate w / slices, `each` rows of it. Its sums of dpost and dpre are row w
// of part_post and part_pre [groups][d]; with slices > 1 its sum of dgate is
// row w of part_gate.
struct NormPlan {
  int groups, each, slices;
};
NormPlan norm_plan(int rows, int d, int per_gate);
hipError_t launch_norm(const NormLaunch& a, hipStream_t s);
hipError_t launch_norm_backward(const NormBackLaunch& a, hipStream_t s);
hipError_t launch_norm_sums(const NormBackLaunch& a, hipStream_t s);

// -------------------------------------------------------- linear attention

struct LinearLaunch {
  Rows q, k, v, o;
  const float* log_decay;       // [kv heads]
  const int32_t* starts;        // [batch + 1], or null: tokens / batch each
  const float* first;           // [batch][kv heads][dk][dv], or null: zeros
  float* last;                  // likewise, or null
  float* sums;                  // [batch][kv heads][parts][dk][dv] (parts > 1)
  int batch, tokens, max_new, kv_heads, dk, dv;
  int parts, part_rows;         // a sequence's rows are cut into `parts`
  float scale;
  bool f32;
};
struct LinearBackLaunch {
  LinearLaunch f;               // o unused; first: the states before
  Rows d_o, dq, dk, dv;
  const float* d_last;          // or null
  float* d_first;               // or null
  float* back_sums;             // like f.sums
};
// Whether a call goes token by token (and needs no parts).
bool linear_by_token(const LinearLaunch& a);
void linear_parts(LinearLaunch* a, bool back);
hipError_t launch_linear(const LinearLaunch& a, hipStream_t s);
hipError_t launch_linear_backward(const LinearBackLaunch& a, hipStream_t s);
// d_last (or zeros) to d_first: the backward of a call without rows.
hipError_t launch_linear_through(const LinearBackLaunch& a, hipStream_t s);

// ------------------------------------------------------------------- AdamW

constexpr int kStateBlock = 256;    // values that share a scale; tensors are padded to it
constexpr int kStepTensors = 64;    // of one launch

struct StepTensor {
  void* p;
  float* master;                // or null
  const void* g;
  int64_t n, off;               // values, and where its states start
};
struct StepLaunch {
  StepTensor t[kStepTensors];
  int first[kStepTensors + 1];  // chunk of kStepChunk values that each starts with
  int count;
  void *m, *v;
  float *m_scale, *v_scale;     // 8-bit states
  float b1, b2, c1, c2;         // c: 1 - b
  float eps, lr, wd, a, k, rs;  // a = lr / (1 - b1^t), k = 1 - lr wd, rs = 1 / sqrt(1 - b2^t)
  float ln1, ln2;               // logarithms of b1, b2 (a step kept on the device)
  float max_norm;
  const float* norm;            // or null
  const float* lr_dev;          // or null
  const int32_t* step_dev;      // or null
};
struct StepCall {
  const StepLaunch* a;
  bool p_f32, g_f32, master, bits8;
};
struct StateRead {
  const void *m, *v;
  const float *m_scale, *v_scale;
  void *m_out, *v_out;
  int64_t n;                    // a multiple of kStateBlock
  bool out_f32;
};
constexpr int kNormTensors = 128, kNormGroups = 512;  // of one launch of the norm's sums
struct GradNormLaunch {
  const void* g[kNormTensors];
  int64_t n[kNormTensors];
  int first[kNormTensors + 1];  // chunk of kNormChunk values that each starts with
  int count;
  double* part;                 // [kNormGroups] of this launch
};
struct GradNormCall {
  const GradNormLaunch* a;
  bool f32;
};
struct GradNormJoin {
  const double* part;
  int64_t count;
  float* norm;
};
constexpr int kStepChunk = 2048, kNormChunk = 8192;
hipError_t launch_adamw(const StepCall& c, hipStream_t s);
hipError_t launch_state_read(const StateRead& a, hipStream_t s);
hipError_t launch_grad_norm(const GradNormCall& c, hipStream_t s);
hipError_t launch_grad_norm_join(const GradNormJoin& a, hipStream_t s);

}  // namespace tttk
