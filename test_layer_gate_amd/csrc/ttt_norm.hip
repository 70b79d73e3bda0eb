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
// a buffer again before everybody has passed the other one's barrier. Of the
// backward's six, those that its norms need.
template <int N, bool PRE = true, bool POST = true>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[kMaxWaves], int waves) {
  constexpr auto on = [](int i) { return N != 6 || (i < 2 ? PRE : i < 4 ? POST : PRE && POST); };
  if constexpr (N == 6 && !PRE && !POST) return;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (on(i)) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on(i)) red[i][threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!on(i)) continue;
    float s = red[i][0];
    for (int w = 1; w < waves; ++w) s += red[i][w];
    v[i] = s;
  }
}

// Eight values of a row that leaves: whole lines of bf16 pass the caches by
// (64k rows of 2560 took 258 us so and 294 with plain stores); of fp32 a lane's
// two pieces are half lines, which would each cost a read.
template <bool F32>
__device__ __forceinline__ void store_row(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (F32)
    store8<true>(p, i, v);
  else
    stream_store<false>(p, i, v);
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

// A workgroup of `waves` waves takes a row, a lane K vectors of 8 neighbouring
// values of it, so that the row is read once and stays in registers through both
// norms. Bound by HBM: 64k rows of 2560 in bf16, with a gate vector and the norm
// before the next block, take 250 us, 5.4 TB/s. (Workgroups that stay for more
// rows and load the next one ahead took 256 us, and more of them 271: there are
// enough rows on their way.)
template <bool AF32, bool RF32, int K>
__global__ __launch_bounds__(512) void norm_kernel(NormLaunch a, int waves, int64_t first) {
  __shared__ float red[2][1][kMaxWaves];
  const int vecs = a.d >> 3, step = waves << 6;
  const float inv_d = 1.f / (float)a.d;
  const int64_t n = first + blockIdx.x;
  const bool has_f = a.f.p != nullptr;
  float x[K][8], f[K][8];
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
    float by = a.scale;
    if (a.norm_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += f[k][e] * f[k][e];
      block_sum(s, red[0], waves);
      by *= 1.f / sqrtf(s[0] * inv_d + a.eps);
    }
    const int64_t gate = a.gate.p ? (int64_t)((int)n / a.per_gate) * a.gate.ts : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * step + threadIdx.x;
      if (v < vecs) {
        float w[8], g[8];
        load_weight(a.norm_post ? a.post : nullptr, a.w_f32, v * 8, w);
        if (a.gate.p) {
          load8<AF32>(a.gate.p, gate + v * 8, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = rounded(x[k][e] + by * (f[k][e] * w[e]), RF32);
        store_row<RF32>(a.r.p, n * a.r.ts + v * 8, x[k]);
      }
    }
  }
  if (!a.norm_pre) return;
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
      store_row<AF32>(a.h.p, n * a.h.ts + v * 8, w);
    }
  }
}

// Eight values on their way: loaded as they are, unpacked where they are used.
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (F32 ? 4 : 2));
    v[0] = q[0];
    if constexpr (F32) v[1] = q[1];
  }
  // Keeps the compiler from knowing the values from before.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) asm volatile("" : "+v"(v[i].x), "+v"(v[i].y), "+v"(v[i].z), "+v"(v[i].w));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint4& u = v[F32 ? e >> 1 : 0];
      if constexpr (F32) {
        x[2 * e] = __uint_as_float(e & 1 ? u.z : u.x), x[2 * e + 1] = __uint_as_float(e & 1 ? u.w : u.y);
      } else {
        const uint32_t w = e == 0 ? u.x : e == 1 ? u.y : e == 2 ? u.z : u.w;
        x[2 * e] = __uint_as_float(w << 16), x[2 * e + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
};

// The gradients of a row, with rho and phi the two norms' factors:
//   t = pre dh;  D = dr + rho (t - r rho^2 mean(r t))            dx
//   c = f post scale gate;  df = phi (post dn - f phi^2 mean(c D)),  dn = scale gate D
// mean(c D) is taken apart into sums of c dr, c t and c r, so that all sums of
// a row are joined at once. The sums over rows are kept in registers over a
// workgroup's rows; the next row is loaded meanwhile.
// Bound by HBM: 8 x 2k rows of 4096 with both norms and a gate a sequence take
// 186 us for 0.81 GB, 4.3 TB/s (255 with the rows unpacked once and kept so: the
// registers left too few waves).
//
// PRE, POST, GATED: whether the norms and the gate can be there (registers are
// kept for what can).
template <bool AF32, bool RF32, int K, bool PRE, bool POST, bool GATED>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormBackLaunch b, NormPlan plan, int waves) {
  __shared__ float red[2][6][kMaxWaves];
  const NormLaunch& a = b.n;
  const int vecs = a.d >> 3, step = waves << 6, w = blockIdx.x;
  const float inv_d = 1.f / (float)a.d;
  const bool has_f = a.f.p != nullptr, gated = GATED && a.gate.p != nullptr;
  const bool has_pre = PRE && a.norm_pre, has_post = POST && has_f && a.norm_post;
  int lo, hi, gate = 0;  // its rows, and the first one's gate
  if (plan.slices > 1) {
    gate = w / plan.slices;
    lo = gate * a.per_gate + w % plan.slices * plan.each;
    hi = min(lo + plan.each, (gate + 1) * a.per_gate);
  } else {
    lo = w * plan.each;
    hi = min(lo + plan.each, a.rows);
    if (gated) gate = lo / a.per_gate;
  }
  int left = gated ? (gate + 1) * a.per_gate - lo : 0;  // rows of that gate
  Raw<RF32> rn[K], drn[K];
  Raw<AF32> fn[K], dhn[K], gn[K];
  auto fetch = [&](int row, int gate) {
    const int64_t n = row;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = min(k * step + (int)threadIdx.x, vecs - 1);
      if (has_pre) {
        rn[k].load(a.x.p, n * a.x.ts + v * 8);
        dhn[k].load(b.dh.p, n * b.dh.ts + v * 8);
      }
      if (b.dr.p) drn[k].load(b.dr.p, n * b.dr.ts + v * 8);
      if (has_f) fn[k].load(a.f.p, n * a.f.ts + v * 8);
      if (gated) gn[k].load(a.gate.p, gate * a.gate.ts + v * 8);
    }
  };
  float d_post[K][8], d_pre[K][8], d_gate[K][8], post[K][8], pre[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) d_post[k][e] = d_pre[k][e] = d_gate[k][e] = 0.f;
    const int v = min(k * step + (int)threadIdx.x, vecs - 1);
    load_weight(has_post ? a.post : nullptr, a.w_f32, v * 8, post[k]);
    load_weight(has_pre ? a.pre : nullptr, a.w_f32, v * 8, pre[k]);
  }
  int turn = 0;
  if (lo < hi) fetch(lo, gate);
  for (int64_t n = lo; n < hi; ++n, turn ^= 1) {
    // the row stays as it was loaded, and is unpacked again behind the sums
    Raw<RF32> rc[K], drc[K];
    Raw<AF32> fc[K], dhc[K], gc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) rc[k] = rn[k], drc[k] = drn[k], fc[k] = fn[k], dhc[k] = dhn[k], gc[k] = gn[k];
    auto unpack = [&](int k, float (&r)[8], float (&f)[8], float (&dr)[8], float (&dh)[8], float (&g)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = f[e] = dr[e] = dh[e] = 0.f, g[e] = 1.f;
      if (has_pre) rc[k].get(r), dhc[k].get(dh);
      if (b.dr.p) drc[k].get(dr);
      if (has_f) fc[k].get(f);
      if (gated) gc[k].get(g);
    };
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * step + (int)threadIdx.x >= vecs) continue;
      float r[8], f[8], dr[8], dh[8], g[8];
      unpack(k, r, f, dr, dh, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = pre[k][e] * dh[e];
        const float c = f[e] * post[k][e] * g[e];
        if constexpr (PRE) s[0] += r[e] * r[e], s[1] += r[e] * t;
        if constexpr (POST) s[2] += f[e] * f[e], s[3] += c * dr[e];
        if constexpr (PRE && POST) s[4] += c * t, s[5] += c * r[e];
      }
    }
    const int64_t this_gate = gate;
    const bool gate_done = gated && --left == 0;
    if (gate_done && n + 1 < hi) ++gate, left = a.per_gate;
    fetch(min((int)n + 1, hi - 1), gate);
    // (unpacked at once, the values would take twice the registers)
#pragma unroll
    for (int k = 0; k < K; ++k) rc[k].forget(), drc[k].forget(), fc[k].forget(), dhc[k].forget(), gc[k].forget();
    block_sum<6, PRE, POST>(s, red[turn], waves);
    float rho = 0.f, back = 0.f, phi = 1.f, fall = 0.f;
    if (has_pre) {
      rho = 1.f / sqrtf(s[0] * inv_d + a.eps);
      back = rho * rho * rho * (s[1] * inv_d);
    }
    if (has_post) {
      phi = 1.f / sqrtf(s[2] * inv_d + a.eps);
      fall = phi * phi * phi * a.scale * ((s[3] + rho * s[4] - back * s[5]) * inv_d);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * step + threadIdx.x;
      if (v < vecs) {
        float r[8], f[8], dr[8], dh[8], g[8], df[8], dg[8];
        unpack(k, r, f, dr, dh, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float D = dr[e];
          if (has_pre) {
            D += rho * (pre[k][e] * dh[e]) - back * r[e];
            d_pre[k][e] += dh[e] * (r[e] * rho);
          }
          dr[e] = D;
          const float fn = f[e] * phi, sD = a.scale * D;
          dg[e] = fn * post[k][e] * sD;
          if constexpr (GATED) d_gate[k][e] += dg[e];
          const float dn = g[e] * sD;
          if constexpr (POST) d_post[k][e] += dn * fn;
          df[e] = phi * (post[k][e] * dn) - fall * f[e];
        }
        store_row<RF32>(b.dx.p, n * b.dx.ts + v * 8, dr);
        if (has_f) store_row<AF32>(b.df.p, n * b.df.ts + v * 8, df);
        if (gated && a.per_gate == 1) store_row<AF32>(b.dgate.p, n * b.dgate.ts + v * 8, dg);
      }
    }
    if (gate_done && a.per_gate > 1 && plan.slices == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int v = k * step + threadIdx.x;
        if (v < vecs) store8<true>(b.dgate.p, this_gate * b.dgate.ts + v * 8, d_gate[k]);
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
      if (POST && b.dpost) store8<true>(b.part_post, at, d_post[k]);
      if (PRE && b.dpre) store8<true>(b.part_pre, at, d_pre[k]);
      if (gated && plan.slices > 1) store8<true>(b.part_gate, at, d_gate[k]);
    }
  }
}

// Sums of the workgroups' parts, 64 columns a workgroup, in a fixed order: 16
// rows of threads each take every 16th part.
constexpr int kSumRows = 16;
__global__ __launch_bounds__(64 * kSumRows) void norm_sums_kernel(NormBackLaunch b, NormPlan plan, int blocks,
                                                                  int jobs_w, int64_t first) {
  __shared__ float red[kSumRows][64];
  const int d = b.n.d, job = (int)((first + blockIdx.x) / blocks);
  const int col = (int)((first + blockIdx.x) % blocks) * 64 + (threadIdx.x & 63), row = threadIdx.x >> 6;
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
  const int K = a.d <= 4096 ? 1 : a.d <= 8192 ? 2 : 4, waves = waves_of(a.d, K);
  const dim3 t(64 * waves);
  in_pieces(a.rows, [&](uint32_t g, int64_t first) {
    if (K == 1)
      norm_kernel<AF32, RF32, 1><<<g, t, 0, s>>>(a, waves, first);
    else if (K == 2)
      norm_kernel<AF32, RF32, 2><<<g, t, 0, s>>>(a, waves, first);
    else
      norm_kernel<AF32, RF32, 4><<<g, t, 0, s>>>(a, waves, first);
  });
  return hipGetLastError();
}

// Vectors of a lane in the backward: its sums over rows take 24 registers for
// each.
int back_vecs(int d) { return d <= 8192 ? 1 : 2; }

template <bool AF32, bool RF32, bool PRE, bool POST>
void back_of(const NormBackLaunch& b, const NormPlan& plan, int waves, hipStream_t s) {
  const dim3 g(plan.groups), t(64 * waves);
  if (b.n.gate.p)
    norm_backward_kernel<AF32, RF32, 1, PRE, POST, true><<<g, t, 0, s>>>(b, plan, waves);
  else
    norm_backward_kernel<AF32, RF32, 1, PRE, POST, false><<<g, t, 0, s>>>(b, plan, waves);
}

template <bool AF32, bool RF32>
hipError_t back_of(const NormBackLaunch& b, hipStream_t s) {
  const NormPlan plan = norm_plan(b.n.rows, b.n.d, b.n.gate.p ? b.n.per_gate : 0);
  const int K = back_vecs(b.n.d), waves = waves_of(b.n.d, K);
  if (K == 1) {
    if (b.n.norm_pre && b.n.norm_post)
      back_of<AF32, RF32, true, true>(b, plan, waves, s);
    else if (b.n.norm_pre)
      back_of<AF32, RF32, true, false>(b, plan, waves, s);
    else if (b.n.norm_post)
      back_of<AF32, RF32, false, true>(b, plan, waves, s);
    else
      back_of<AF32, RF32, false, false>(b, plan, waves, s);
  } else {
    norm_backward_kernel<AF32, RF32, 2, true, true, true><<<plan.groups, 64 * waves, 0, s>>>(b, plan, waves);
  }
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
  in_pieces(jobs * blocks, [&](uint32_t g, int64_t first) {
    norm_sums_kernel<<<g, 64 * kSumRows, 0, s>>>(b, plan, blocks, jobs_w, first);
  });
  return hipGetLastError();
}

}  // namespace tttk
