// gfx950 kernels of the norms before and after a block, fused with the
// block's gate and residual scale:
//   n = f, or f rsqrt(mean f^2 + eps) post
//   r = x + scale gate n                       (stored in x's type)
//   h = r rsqrt(mean r^2 + eps) pre            (of r as it is stored)
// and their gradients.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ttt_block.h"
#include "ttt_serve_device.h"

namespace tttk {
namespace {

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

// The wave's sum, in every lane: within 16 lanes by DPP (neighbour, pair,
// half row mirrored, row mirrored), then across them.
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp<0xb1>(x);
  x += dpp<0x4e>(x);
  x += dpp<0x141>(x);
  x += dpp<0x140>(x);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

constexpr int kMaxWaves = 16;

// The workgroup's sums of N values, in every lane. `red` alternates between
// two buffers from call to call, so that one barrier is enough: nobody writes
// a buffer again before everybody has passed the other one's barrier.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[kMaxWaves], int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = red[i][0];
    for (int w = 1; w < waves; ++w) s += red[i][w];
    v[i] = s;
  }
}

__device__ __forceinline__ void load_weight(const void* p, bool f32, int64_t i, float (&v)[8]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
  } else if (f32) {
    load8<true>(p, i, v);
  } else {
    load8<false>(p, i, v);
  }
}

__device__ __forceinline__ float rounded(float x, bool f32) { return f32 ? x : bf16_f32(bf16_rne(x)); }

// A workgroup of `waves` waves takes a row at a time, a lane K vectors of 8
// neighbouring values of it, so that a row is read once and stays in registers
// through both norms.
template <bool AF32, bool RF32, int K>
__global__ void norm_kernel(NormLaunch a, int waves) {
  __shared__ float red[2][1][kMaxWaves];
  const int vecs = a.d >> 3, step = waves << 6;
  const float inv_d = 1.f / (float)a.d;
  for (int64_t n = blockIdx.x; n < a.rows; n += gridDim.x) {
    float x[K][8], f[K][8];
    const bool has_f = a.f.p != nullptr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * step + threadIdx.x;
      if (v < vecs) {
        load8<RF32>(a.x.p, n * a.x.ts + v * 8, x[k]);
        if (has_f) load8<AF32>(a.f.p, n * a.f.ts + v * 8, f[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = f[k][e] = 0.f;
      }
    }
    if (has_f) {
      if (a.norm_post) {
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] += f[k][e] * f[k][e];
        block_sum(s, red[0], waves);
        const float phi = 1.f / sqrtf(s[0] * inv_d + a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int v = k * step + threadIdx.x;
          if (v < vecs) {
            float w[8];
            load_weight(a.post, a.w_f32, v * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[k][e] = f[k][e] * phi * w[e];
          }
        }
      }
      const int64_t gate = a.gate.p ? n / a.per_gate * a.gate.ts : 0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int v = k * step + threadIdx.x;
        if (v < vecs) {
          if (a.gate.p) {
            float g[8];
            load8<AF32>(a.gate.p, gate + v * 8, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[k][e] *= g[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = rounded(x[k][e] + a.scale * f[k][e], RF32);
          store8<RF32>(a.r.p, n * a.r.ts + v * 8, x[k]);
        }
      }
    }
    if (!a.norm_pre) {
      if (waves > 1 && has_f && a.norm_post) __syncthreads();  // (see below)
      continue;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += x[k][e] * x[k][e];
    block_sum(s, red[1], waves);
    const float rho = 1.f / sqrtf(s[0] * inv_d + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * step + threadIdx.x;
      if (v < vecs) {
        float w[8];
        load_weight(a.pre, a.w_f32, v * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= x[k][e] * rho;
        store8<AF32>(a.h.p, n * a.h.ts + v * 8, w);
      }
    }
    // with one of the two sums alone, the next row writes its buffer again with
    // no barrier of the other's between
    if (waves > 1 && !(has_f && a.norm_post)) __syncthreads();
  }
}

// The gradients of a row, with rho and phi the two norms' factors:
//   t = pre dh;  D = dr + rho (t - r rho^2 mean(r t))            dx
//   a = f post scale gate;  df = phi (post dn - f phi^2 mean(a D)),  dn = scale gate D
// mean(a D) is taken apart into sums of a dr, a t and a r, so that all sums of
// a row are joined at once. The sums over rows are kept in registers over a
// workgroup's rows.
template <bool AF32, bool RF32, int K>
__global__ void norm_backward_kernel(NormBackLaunch b, NormPlan plan, int waves) {
  __shared__ float red[2][6][kMaxWaves];
  const NormLaunch& a = b.n;
  const int vecs = a.d >> 3, step = waves << 6, w = blockIdx.x;
  const float inv_d = 1.f / (float)a.d;
  const bool has_f = a.f.p != nullptr, gated = a.gate.p != nullptr;
  int64_t lo, hi;
  if (plan.slices > 1) {
    const int64_t g = w / plan.slices, first = g * a.per_gate;
    lo = first + (int64_t)(w % plan.slices) * plan.each;
    hi = min(lo + plan.each, first + a.per_gate);
  } else {
    lo = (int64_t)w * plan.each;
    hi = min(lo + plan.each, (int64_t)a.rows);
  }
  float d_post[K][8], d_pre[K][8], d_gate[K][8], g[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) d_post[k][e] = d_pre[k][e] = d_gate[k][e] = 0.f, g[k][e] = 1.f;
  int turn = 0;
  for (int64_t n = lo; n < hi; ++n, turn ^= 1) {
    const int64_t gi = gated ? n / a.per_gate : 0;
    if (gated && (n == lo || n % a.per_gate == 0)) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int v = k * step + threadIdx.x;
        if (v < vecs) load8<AF32>(a.gate.p, gi * a.gate.ts + v * 8, g[k]);
      }
    }
    float r[K][8], f[K][8], dr[K][8], dh[K][8], post[K][8];
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * step + threadIdx.x;
#pragma unroll
      for (int e = 0; e < 8; ++e) r[k][e] = f[k][e] = dr[k][e] = dh[k][e] = post[k][e] = 0.f;
      if (v < vecs) {
        if (a.norm_pre) {
          load8<RF32>(a.x.p, n * a.x.ts + v * 8, r[k]);
          load8<AF32>(b.dh.p, n * b.dh.ts + v * 8, dh[k]);
        }
        if (b.dr.p) load8<RF32>(b.dr.p, n * b.dr.ts + v * 8, dr[k]);
        if (has_f) {
          load8<AF32>(a.f.p, n * a.f.ts + v * 8, f[k]);
          load_weight(a.norm_post ? a.post : nullptr, a.w_f32, v * 8, post[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * step + threadIdx.x;
      float pre[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) pre[e] = 0.f;
      if (v < vecs && a.norm_pre) load_weight(a.pre, a.w_f32, v * 8, pre);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = pre[e] * dh[k][e];
        const float c = f[k][e] * post[k][e] * g[k][e];
        s[0] += r[k][e] * r[k][e];
        s[1] += r[k][e] * t;
        s[2] += f[k][e] * f[k][e];
        s[3] += c * dr[k][e];
        s[4] += c * t;
        s[5] += c * r[k][e];
      }
    }
    block_sum(s, red[turn], waves);
    float rho = 0.f, back = 0.f, phi = 1.f, fall = 0.f;
    if (a.norm_pre) {
      rho = 1.f / sqrtf(s[0] * inv_d + a.eps);
      back = rho * rho * rho * (s[1] * inv_d);
    }
    if (has_f && a.norm_post) {
      phi = 1.f / sqrtf(s[2] * inv_d + a.eps);
      fall = phi * phi * phi * a.scale * ((s[3] + rho * s[4] - back * s[5]) * inv_d);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * step + threadIdx.x;
      if (v < vecs) {
        float pre[8], df[8], dg[8];
        if (a.norm_pre) load_weight(a.pre, a.w_f32, v * 8, pre);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float D = dr[k][e];
          if (a.norm_pre) {
            D += rho * (pre[e] * dh[k][e]) - back * r[k][e];
            d_pre[k][e] += dh[k][e] * (r[k][e] * rho);
          }
          dr[k][e] = D;
          const float fn = f[k][e] * phi, sD = a.scale * D;
          dg[e] = fn * post[k][e] * sD;
          d_gate[k][e] += dg[e];
          const float dn = g[k][e] * sD;
          d_post[k][e] += dn * fn;
          df[e] = phi * (post[k][e] * dn) - fall * f[k][e];
        }
        store8<RF32>(b.dx.p, n * b.dx.ts + v * 8, dr[k]);
        if (has_f) store8<AF32>(b.df.p, n * b.df.ts + v * 8, df);
        if (gated && a.per_gate == 1) store8<AF32>(b.dgate.p, n * b.dgate.ts + v * 8, dg);
      }
    }
    if (gated && a.per_gate > 1 && plan.slices == 1 && (n + 1) % a.per_gate == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int v = k * step + threadIdx.x;
        if (v < vecs) store8<true>(b.dgate.p, gi * b.dgate.ts + v * 8, d_gate[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) d_gate[k][e] = 0.f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = k * step + threadIdx.x;
    if (v < vecs) {
      const int64_t at = (int64_t)w * a.d + v * 8;
      if (b.dpost) store8<true>(b.part_post, at, d_post[k]);
      if (b.dpre) store8<true>(b.part_pre, at, d_pre[k]);
      if (gated && plan.slices > 1) store8<true>(b.part_gate, at, d_gate[k]);
    }
  }
}

// Sums of the workgroups' parts, 64 columns a workgroup, in a fixed order: 16
// rows of threads each take every 16th part.
constexpr int kSumRows = 16;
__global__ __launch_bounds__(64 * kSumRows) void norm_sums_kernel(NormBackLaunch b, NormPlan plan, int blocks,
                                                                  int jobs_w) {
  __shared__ float red[kSumRows][64];
  const int d = b.n.d, job = blockIdx.x / blocks;
  const int col = (blockIdx.x % blocks) * 64 + (threadIdx.x & 63), row = threadIdx.x >> 6;
  const float* part;
  float* out;
  int count = plan.groups;
  if (job < jobs_w) {
    const bool post = b.dpost != nullptr && job == 0;
    part = post ? b.part_post : b.part_pre;
    out = post ? b.dpost : b.dpre;
  } else {
    const int64_t g = job - jobs_w;
    count = plan.slices;
    part = b.part_gate + g * count * d;
    out = static_cast<float*>(b.dgate.p) + g * b.dgate.ts;
  }
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int i = row; i < count; i += kSumRows) s += part[(int64_t)i * d + col];
  }
  red[row][threadIdx.x & 63] = s;
  __syncthreads();
  if (row == 0 && col < d) {
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) s += red[i][threadIdx.x];
    out[col] = s;
  }
}

int waves_of(int d, int k) { return (d / 8 + 64 * k - 1) / (64 * k); }

template <bool AF32, bool RF32>
hipError_t norm_of(const NormLaunch& a, hipStream_t s) {
  const int vecs = a.d / 8;
  const int K = vecs <= 64 ? 1 : vecs <= 128 ? 2 : vecs <= 192 ? 3 : vecs <= 320 ? 5 : 8;
  const int waves = waves_of(a.d, K);
  const int grid = (int)std::min<int64_t>(a.rows, 256 * 32 / waves);
  const dim3 g(grid), t(64 * waves);
  switch (K) {
    case 1: norm_kernel<AF32, RF32, 1><<<g, t, 0, s>>>(a, waves); break;
    case 2: norm_kernel<AF32, RF32, 2><<<g, t, 0, s>>>(a, waves); break;
    case 3: norm_kernel<AF32, RF32, 3><<<g, t, 0, s>>>(a, waves); break;
    case 5: norm_kernel<AF32, RF32, 5><<<g, t, 0, s>>>(a, waves); break;
    default: norm_kernel<AF32, RF32, 8><<<g, t, 0, s>>>(a, waves); break;
  }
  return hipGetLastError();
}

// Vectors of a lane in the backward: its sums over rows take 24 registers for
// each.
int back_vecs(int d) { return d <= 4096 ? 1 : 2; }

template <bool AF32, bool RF32>
hipError_t back_of(const NormBackLaunch& b, hipStream_t s) {
  const NormPlan plan = norm_plan(b.n.rows, b.n.d, b.n.gate.p ? b.n.per_gate : 0);
  const int K = back_vecs(b.n.d), waves = waves_of(b.n.d, K);
  const dim3 g(plan.groups), t(64 * waves);
  if (K == 1)
    norm_backward_kernel<AF32, RF32, 1><<<g, t, 0, s>>>(b, plan, waves);
  else
    norm_backward_kernel<AF32, RF32, 2><<<g, t, 0, s>>>(b, plan, waves);
  return hipGetLastError();
}

}  // namespace

NormPlan norm_plan(int rows, int d, int per_gate) {
  if (rows == 0) return {0, 1, 0};
  const int waves = waves_of(d, back_vecs(d));
  const int groups = std::max(1, 4096 / waves);
  const int each = std::max(4, (rows + groups - 1) / groups);
  if (per_gate <= 1) return {(rows + each - 1) / each, each, 1};
  if (per_gate >= 2 * each) {
    const int slices = (per_gate + each - 1) / each, part = (per_gate + slices - 1) / slices;
    return {rows / per_gate * ((per_gate + part - 1) / part), part, (per_gate + part - 1) / part};
  }
  const int whole = std::max(1, each / per_gate) * per_gate;
  return {(rows + whole - 1) / whole, whole, 1};
}

hipError_t launch_norm(const NormLaunch& a, hipStream_t s) {
  if (a.act_f32) return norm_of<true, true>(a, s);
  return a.res_f32 ? norm_of<false, true>(a, s) : norm_of<false, false>(a, s);
}

hipError_t launch_norm_backward(const NormBackLaunch& b, hipStream_t s) {
  if (b.n.act_f32) return back_of<true, true>(b, s);
  return b.n.res_f32 ? back_of<false, true>(b, s) : back_of<false, false>(b, s);
}

hipError_t launch_norm_sums(const NormBackLaunch& b, hipStream_t s) {
  const NormPlan plan = norm_plan(b.n.rows, b.n.d, b.n.gate.p ? b.n.per_gate : 0);
  const int jobs_w = (b.dpost != nullptr) + (b.dpre != nullptr);
  const int64_t jobs = jobs_w + (b.n.gate.p && plan.slices != 1 ? b.dgate.heads : 0);
  if (jobs == 0) return hipSuccess;
  const int blocks = (b.n.d + 63) / 64;
  norm_sums_kernel<<<(uint32_t)(jobs * blocks), 64 * kSumRows, 0, s>>>(b, plan, blocks, jobs_w);
  return hipGetLastError();
}

}  // namespace tttk
