// gfx950 kernels of the rotary positions: y = R(pos) x on the first `rot`
// values of every head, its transpose for the gradient, and the table of
// cosines and sines they read.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_serve_device.h"

namespace tttk {
namespace {

constexpr int kRopeThreads = 256;

// A unit is two pieces of 16 bytes (W values) of one head: W values from i
// and W from i + rot / 2, W pairs of the half layout and of the interleaved
// one W / 2 pairs each; of the part that is copied, likewise. Neighbouring
// lanes take neighbouring pieces, then neighbouring heads of the token, so
// that a wave reads and writes whole lines; a lane then walks over the
// remaining heads with the cosines and sines it has loaded. Bound by HBM:
// 64k tokens of 32 + 8 heads of 128 in bf16 take 216 us, 6.4 TB/s.
template <bool F32>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeLaunch a, int units, int lanes,
                                                            int64_t total) {
  constexpr int W = kWide<F32>;
  const int64_t id = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  if (id >= total) return;
  const int u = (int)(id % units);
  const int64_t r = id / units;
  const int h0 = (int)(r % lanes);
  const int n = (int)(r / lanes);
  const RopeArgs& rope = a.rope;
  const int rot_units = rope.rot / (2 * W);
  const bool turned = u < rot_units;
  const int i0 = turned ? u * W : rope.rot + (u - rot_units) * W;
  const int i1 = i0 + (turned ? rope.rot / 2 : (a.dim - rope.rot) / 2);
  // the pieces' pairs: of the half layout the first W, of the other W / 2 each
  float c[W], s[W];
  if (turned) {
    const int pos = a.positions ? a.positions[n] : n % a.seq_len;
    if (rope.interleaved) {
      float cc[W / 2], ss[W / 2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        load_cs<W / 2>(rope, pos, (x ? i1 : i0) / 2, cc, ss);
#pragma unroll
        for (int e = 0; e < W / 2; ++e) c[x * W / 2 + e] = cc[e], s[x * W / 2 + e] = ss[e];
      }
    } else {
      load_cs<W>(rope, pos, i0, c, s);
    }
  }
  const int heads = a.x[0].heads + a.x[1].heads;
  for (int h = h0; h < heads; h += lanes) {
    const int t = h >= a.x[0].heads;
    const int hh = t ? h - a.x[0].heads : h;
    const int64_t xi = n * a.x[t].ts + hh * a.x[t].hs, yi = n * a.y[t].ts + hh * a.y[t].hs;
    float p[W], q[W];
    stream_load<F32>(a.x[t].p, xi + i0, p);
    stream_load<F32>(a.x[t].p, xi + i1, q);
    if (turned) {
      if (rope.interleaved) {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
          turn(p[2 * e], p[2 * e + 1], c[e], s[e], &p[2 * e], &p[2 * e + 1]);
          turn(q[2 * e], q[2 * e + 1], c[W / 2 + e], s[W / 2 + e], &q[2 * e], &q[2 * e + 1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) turn(p[e], q[e], c[e], s[e], &p[e], &q[e]);
      }
    }
    stream_store<F32>(a.y[t].p, yi + i0, p);
    stream_store<F32>(a.y[t].p, yi + i1, q);
  }
}

// The angle step of pair i: w = base^(-2i / rot), changed for long contexts by
// published methods: position interpolation (1; Chen et al., 2023), the changed
// base known as NTK-aware (2), YaRN (3; Peng et al., 2023), and the banded scaling
// published with LLaMA 3.1 (4).
//   1 linear: w / factor
//   2 by base: base * factor^(rot / (rot - 2)), which leaves the fastest pair
//     alone and divides the slowest one's step by factor
//   3 by parts (YaRN): pairs that turn more than `hi` times over the original
//     context keep w, those below `lo` turns take w / factor, a linear ramp
//     in the pair's index lies between
//   4 bands: the same two ends by wavelength (orig / hi and orig / lo), a
//     linear ramp in orig / wavelength between
__device__ double angle_step(int i, int rot, double base, int kind, double factor, double orig,
                             double lo, double hi) {
  const double two_pi = 6.283185307179586476925286766559;
  if (kind == 2) base *= pow(factor, (double)rot / (rot - 2));
  const double w = pow(base, -2.0 * i / rot);
  if (kind == 1) return w / factor;
  if (kind == 3) {
    // the (real) index of the pair that turns r times: w orig = 2 pi r
    const double lg = log(base);
    double first = floor(rot * log(orig / (hi * two_pi)) / (2 * lg));
    double last = ceil(rot * log(orig / (lo * two_pi)) / (2 * lg));
    first = fmax(first, 0.0);
    last = fmin(last, rot - 1.0);
    if (first == last) last += 0.001;  // a step: no ramp, and no 0 / 0
    const double ramp = fmin(fmax((i - first) / (last - first), 0.0), 1.0);
    return w * (1.0 - ramp) + w / factor * ramp;
  }
  if (kind == 4) {
    const double turns = orig * w / two_pi;
    if (turns > hi) return w;
    if (turns < lo) return w / factor;
    const double keep = (turns - lo) / (hi - lo);
    return (1.0 - keep) * w / factor + keep * w;
  }
  return w;
}

// Angles and their functions in 64 bits: pos * w reaches 10^6 rad, where a
// 32-bit product is off by several hundredths. Run once for a model.
__global__ __launch_bounds__(kRopeThreads) void rope_table_kernel(
    float* __restrict__ table, int64_t total, int half, int rot, double base, int kind,
    double factor, double orig, double lo, double hi, double mul) {
  const int64_t id = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  if (id >= total) return;
  const int i = (int)(id % half);
  const double w = angle_step(i, rot, base, kind, factor, orig, lo, hi);
  double s, c;
  sincos((double)(id / half) * w, &s, &c);
  table[2 * id] = (float)(c * mul);
  table[2 * id + 1] = (float)(s * mul);
}

}  // namespace

hipError_t launch_rope(const RopeLaunch& a, hipStream_t s) {
  const int units = a.dim / (2 * (a.f32 ? kWide<true> : kWide<false>)), heads = a.x[0].heads + a.x[1].heads;
  // Heads that are not walked over: enough for a wave or two to stay within
  // a token (with plain accesses, of 1: 304 us for the 64k tokens above, 8: 249,
  // 16: 237, all: 267), and for the chip to be full.
  int lanes = heads;
  const int64_t one = (int64_t)a.tokens * units;
  while (lanes > 1 && units * ((lanes + 1) / 2) >= 128 && one * ((lanes + 1) / 2) >= (int64_t)256 * 2048)
    lanes = (lanes + 1) / 2;
  const int64_t total = one * lanes;
  const int64_t grid = (total + kRopeThreads - 1) / kRopeThreads;
  if (a.f32)
    rope_kernel<true><<<(uint32_t)grid, kRopeThreads, 0, s>>>(a, units, lanes, total);
  else
    rope_kernel<false><<<(uint32_t)grid, kRopeThreads, 0, s>>>(a, units, lanes, total);
  return hipGetLastError();
}

hipError_t launch_rope_table(float* table, int max_pos, int rot, double base, int kind,
                             double factor, double orig, double lo, double hi, double mul,
                             hipStream_t s) {
  const int64_t total = (int64_t)max_pos * (rot / 2);
  rope_table_kernel<<<(uint32_t)((total + kRopeThreads - 1) / kRopeThreads), kRopeThreads, 0, s>>>(
      table, total, rot / 2, rot, base, kind, factor, orig, lo, hi, mul);
  return hipGetLastError();
}

}  // namespace tttk
