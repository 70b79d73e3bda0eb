// gfx950 kernels of the AdamW step over many tensors, of the 2-norm of their
// gradients that may limit it, and of reading 8-bit states back.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_block.h"
#include "ttt_serve_device.h"

namespace tttk {
namespace {

constexpr int kStepThreads = kStepChunk / 8;

// Which tensor chunk `c` belongs to: the last t with first[t] <= c.
__device__ __forceinline__ int tensor_of(const int* first, int count, int c) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= c) lo = mid; else hi = mid;
  }
  return lo;
}

// Eight values from i of a tensor of n (i < n); 0 behind its end.
template <bool F32>
__device__ __forceinline__ void load_tail(const void* p, int64_t i, int64_t n, float (&v)[8]) {
  if (i + 8 <= n) {
    load8<F32>(p, i, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = 0.f;
    if (i + e < n) v[e] = F32 ? static_cast<const float*>(p)[i + e] : bf16_f32(static_cast<const u16*>(p)[i + e]);
  }
}
template <bool F32>
__device__ __forceinline__ void store_tail(void* p, int64_t i, int64_t n, const float (&v)[8]) {
  if (i + 8 <= n) {
    store8<F32>(p, i, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (i + e < n) {
      if constexpr (F32)
        static_cast<float*>(p)[i + e] = v[e];
      else
        static_cast<u16*>(p)[i + e] = bf16_rne(v[e]);
    }
  }
}

// 8-bit states: a block of 256 values shares an fp32 scale. m's codes are e4m3
// (the hardware's conversion: nearest, ties to even), 448 the largest. The root
// of v, in whose half range of exponents 8 bits go further, has codes of 4
// exponent and 4 fraction bits and no sign: value (16 + c % 16) 2^(c / 16 - 11),
// below 16 c 2^-10, 496 the largest. The scales are the blocks' maxima over
// those, not powers of two: a block whose values only decay keeps its codes and
// lets the scale decay, where rounding to a fixed grid would hold them for good.
// A NaN or an infinity makes its block's scale, so the whole block, NaN.
constexpr float kCodeM = 448.f, kCodeR = 496.f, kScaleLeast = 0x1p-126f;

// max over the half wave (32 lanes: a block of 256 values); NaN if any is NaN.
__device__ __forceinline__ float nan_max(float a, float b) { return a != a ? a : (b > a || b != b) ? b : a; }
__device__ __forceinline__ float half_max(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x = nan_max(x, __shfl_xor(x, o));
  return x;
}
__device__ __forceinline__ float scale_of(float top, float most) {
  const float s = top / most;
  return s < kScaleLeast ? kScaleLeast : s + (s - s);  // (an infinity becomes a NaN)
}

__device__ __forceinline__ uint32_t code_of(float r, float scale) {
  // four fraction bits: half of what is dropped, and one more above a tie with
  // an odd code, is added to the bits; values below the least normal 2^-6 have
  // steps of 2^-10
  const float y = r / scale;
  const uint32_t u = __float_as_uint(y);
  const uint32_t normal = ((u + 0x3ffffu + ((u >> 19) & 1u)) >> 19) - (120u << 4);
  const uint32_t small = (uint32_t)__builtin_rintf(y * 0x1p10f);
  const uint32_t c = y < 0x1p-6f ? small : min(normal, 255u);
  return r > 0.f ? max(c, 1u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t c) {
  return c < 16u ? (float)c * 0x1p-10f : __uint_as_float((c << 19) + (120u << 23));
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ void load_states(const StepLaunch& a, int64_t i, float (&m)[8], float (&v)[8]) {
  const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.m) + i);
  const uint2 cr = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v) + i);
  const float sm = a.m_scale[i >> 8], sr = a.v_scale[i >> 8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int wm = (int)(e < 4 ? cm.x : cm.y);
    const uint32_t wr = e < 4 ? cr.x : cr.y;
    const float x = e % 4 == 0   ? __builtin_amdgcn_cvt_f32_fp8(wm, 0)
                    : e % 4 == 1 ? __builtin_amdgcn_cvt_f32_fp8(wm, 1)
                    : e % 4 == 2 ? __builtin_amdgcn_cvt_f32_fp8(wm, 2)
                                 : __builtin_amdgcn_cvt_f32_fp8(wm, 3);
    m[e] = x * sm;
    const float r = value_of((wr >> (8 * (e % 4))) & 255u) * sr;
    v[e] = r * r;
  }
}

// A workgroup takes 2048 values of one tensor, a lane 8. Bound by HBM: every
// array is read and written once: 2.4 GB of bf16 weights, fp32 masters and states in
// 452 us, 5.4 TB/s.
template <bool PF32, bool GF32, bool MASTER, bool BITS8>
__global__ __launch_bounds__(kStepThreads) void adamw_kernel(StepLaunch a, int first) {
#pragma clang fp contract(off)
  // (products are rounded before they are added: what is quantised afterwards
  // does not depend on which of them a fused operation would have kept exact)
  const int chunk = first + (int)blockIdx.x, t = tensor_of(a.first, a.count, chunk);
  const StepTensor x = a.t[t];
  const int64_t i = (int64_t)(chunk - a.first[t]) * kStepChunk + threadIdx.x * 8;
  float coef = 1.f;
  if (a.norm != nullptr) {
    const float norm = *a.norm;
    if (!(norm < __builtin_huge_valf())) return;  // infinite or NaN: no step
    if (a.max_norm < norm) coef = a.max_norm / norm;
  }
  float k = a.k, step = a.a, rs = a.rs;
  if (a.lr_dev != nullptr || a.step_dev != nullptr) {
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    k = 1.f - lr * a.wd;
    float c1 = a.a, c2 = a.rs;  // (a is 1 / (1 - b1^t) then)
    if (a.step_dev != nullptr) {
      if (*a.step_dev < 1) return;  // (its 1 - b^0 would divide by 0)
      const float n = (float)*a.step_dev;
      c1 = 1.f / -expm1f(n * a.ln1);
      c2 = 1.f / sqrtf(-expm1f(n * a.ln2));
    }
    step = lr * c1;
    rs = c2;
  }
  const int64_t padded = (x.n + kStateBlock - 1) / kStateBlock * kStateBlock;
  if (i >= padded) return;  // (whole half waves: a block's lanes stay together)
  float g[8], p[8], m[8], v[8];
  const bool some = i < x.n;
#pragma unroll
  for (int e = 0; e < 8; ++e) g[e] = p[e] = 0.f;
  if (some) {
    load_tail<GF32>(x.g, i, x.n, g);
    if constexpr (MASTER)
      load_tail<true>(x.master, i, x.n, p);
    else
      load_tail<PF32>(x.p, i, x.n, p);
  }
  const int64_t at = x.off + i;
  if constexpr (BITS8) {
    load_states(a, at, m, v);
  } else {
    load8<true>(a.m, at, m);
    load8<true>(a.v, at, v);
  }
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    g[e] *= coef;
    const float m0 = m[e] * a.b1, m1 = g[e] * a.c1;
    m[e] = m0 + m1;
    const float v0 = v[e] * a.b2, v1 = g[e] * g[e] * a.c2;
    v[e] = v0 + v1;
    r[e] = sqrtf(v[e]);
    const float rb = r[e] * rs;
    const float u = m[e] / (rb + a.eps) * step, pk = p[e] * k;
    p[e] = pk - u;
  }
  if (some) {
    if constexpr (MASTER) store_tail<true>(x.master, i, x.n, p);
    store_tail<PF32>(x.p, i, x.n, p);
  }
  if constexpr (BITS8) {
    float top_m = 0.f, top_r = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top_m = nan_max(top_m, fabsf(m[e])), top_r = nan_max(top_r, r[e]);
    const float sm = scale_of(half_max(top_m), kCodeM), sr = scale_of(half_max(top_r), kCodeR);
    uint2 cm, cr;
    cm.x = pack_e4m3(m[0] / sm, m[1] / sm, m[2] / sm, m[3] / sm);
    cm.y = pack_e4m3(m[4] / sm, m[5] / sm, m[6] / sm, m[7] / sm);
    cr.x = code_of(r[0], sr) | code_of(r[1], sr) << 8 | code_of(r[2], sr) << 16 | code_of(r[3], sr) << 24;
    cr.y = code_of(r[4], sr) | code_of(r[5], sr) << 8 | code_of(r[6], sr) << 16 | code_of(r[7], sr) << 24;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + at) = cm;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + at) = cr;
    if ((threadIdx.x & 31) == 0) a.m_scale[at >> 8] = sm, a.v_scale[at >> 8] = sr;
  } else {
    store8<true>(a.m, at, m);
    store8<true>(a.v, at, v);
  }
}

// What 8-bit states stand for: m and v, rounded to the outputs' type.
template <bool F32>
__global__ __launch_bounds__(256) void state_read_kernel(StateRead a, int64_t first) {
#pragma clang fp contract(off)
  const int64_t i = ((first + blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= a.n) return;
  StepLaunch s;
  s.m = const_cast<void*>(a.m), s.v = const_cast<void*>(a.v);
  s.m_scale = const_cast<float*>(a.m_scale), s.v_scale = const_cast<float*>(a.v_scale);
  float m[8], v[8];
  load_states(s, i, m, v);
  store8<F32>(a.m_out, i, m);
  store8<F32>(a.v_out, i, v);
}

// The sums of squares of the gradients, in 64 bits (no square overflows), a
// part a workgroup; a workgroup walks over every kNormGroups-th chunk.
template <bool F32>
__global__ __launch_bounds__(256) void grad_norm_kernel(GradNormLaunch a) {
  double s = 0.0;
  const int chunks = a.first[a.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(a.first, a.count, c);
    const int64_t n = a.n[t], lo = (int64_t)(c - a.first[t]) * kNormChunk;
#pragma unroll
    for (int j = 0; j < kNormChunk / 2048; ++j) {
      const int64_t i = lo + j * 2048 + threadIdx.x * 8;
      if (i < n) {
        float g[8];
        load_tail<F32>(a.g[t], i, n, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fma((double)g[e], (double)g[e], s);
      }
    }
  }
  __shared__ double red[256];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o >= 1; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.part[blockIdx.x] = red[0];
}

__global__ __launch_bounds__(256) void grad_norm_join_kernel(GradNormJoin a) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.count; i += 256) s += a.part[i];
  __shared__ double red[256];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o >= 1; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.norm = (float)sqrt(red[0]);
}

template <bool PF32, bool MASTER>
void adamw_of(const StepCall& c, hipStream_t s) {
  const dim3 t(kStepThreads);
  in_pieces(c.a->first[c.a->count], [&](uint32_t g, int64_t at) {
    const int first = (int)at;
    if (c.bits8) {
      if (c.g_f32)
        adamw_kernel<PF32, true, MASTER, true><<<g, t, 0, s>>>(*c.a, first);
      else
        adamw_kernel<PF32, false, MASTER, true><<<g, t, 0, s>>>(*c.a, first);
    } else if (c.g_f32) {
      adamw_kernel<PF32, true, MASTER, false><<<g, t, 0, s>>>(*c.a, first);
    } else {
      adamw_kernel<PF32, false, MASTER, false><<<g, t, 0, s>>>(*c.a, first);
    }
  });
}

}  // namespace

hipError_t launch_adamw(const StepCall& c, hipStream_t s) {
  if (c.p_f32)
    adamw_of<true, false>(c, s);
  else if (c.master)
    adamw_of<false, true>(c, s);
  else
    adamw_of<false, false>(c, s);
  return hipGetLastError();
}

hipError_t launch_state_read(const StateRead& a, hipStream_t s) {
  in_pieces((a.n / 8 + 255) / 256, [&](uint32_t grid, int64_t first) {
    if (a.out_f32)
      state_read_kernel<true><<<grid, 256, 0, s>>>(a, first);
    else
      state_read_kernel<false><<<grid, 256, 0, s>>>(a, first);
  });
  return hipGetLastError();
}

hipError_t launch_grad_norm(const GradNormCall& c, hipStream_t s) {
  if (c.f32)
    grad_norm_kernel<true><<<kNormGroups, 256, 0, s>>>(*c.a);
  else
    grad_norm_kernel<false><<<kNormGroups, 256, 0, s>>>(*c.a);
  return hipGetLastError();
}

hipError_t launch_grad_norm_join(const GradNormJoin& a, hipStream_t s) {
  grad_norm_join_kernel<<<1, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace tttk
