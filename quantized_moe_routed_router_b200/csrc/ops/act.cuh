// The activation between an expert's two products, as 8-bit rows with one scale
// per 128 columns.  Elementwise: HBM bounds it (gate and up read once, codes and
// scales written once).
#pragma once
#include "elem.cuh"

namespace tsm {

constexpr int ACT_THREADS = 256;

TSM_DEV float sigmoid_f(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

// Sixteen lanes per (row, group) unit, eight columns each; units row-major.
template <bool VEC>
__global__ void __launch_bounds__(ACT_THREADS) act_quant_kernel(const ts_moe_act_quant_args a) {
  grid_dep_wait();
  grid_dep_launch();
  const int groups = cdiv(a.inter, SCALE_BLOCK);
  const int64_t units = (int64_t)a.rows * groups;
  const int lane = threadIdx.x & 15;
  // both halves of a warp take every step together: the shuffles name all lanes
  for (int64_t u0 = ((int64_t)blockIdx.x * ACT_THREADS + threadIdx.x) / 32 * 2; u0 < units; u0 += (int64_t)gridDim.x * (ACT_THREADS / 16)) {
    const int64_t u = u0 + ((threadIdx.x >> 4) & 1);
    const int64_t row = u / groups;
    const int group = (int)(u - row * groups), col = group * SCALE_BLOCK + lane * 8;
    const int n = u < units ? min(8, a.inter - col) : 0;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
      const Raw8 rg = load_raw8<VEC>(a.gate, a.in_type, row * a.ld_gate + col, n);
      const Raw8 ru = load_raw8<VEC>(a.up, a.in_type, row * a.ld_up + col, n);
      float g[8], up[8];
      cvt8(rg, a.in_type, g);
      cvt8(ru, a.in_type, up);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (a.act == TS_ACT_SWIGLU) {
          v[j] = g[j] * sigmoid_f(g[j]) * up[j];
        } else {
          // comparisons that keep a NaN, as a clamp does
          const float gc = g[j] > a.act_limit ? a.act_limit : g[j];
          const float uc = up[j] > a.act_limit ? a.act_limit : up[j] < -a.act_limit ? -a.act_limit : up[j];
          v[j] = gc * sigmoid_f(a.act_alpha * gc) * (uc + 1.f);
        }
        if (!VEC && j >= n) v[j] = 0.f;
      }
    }
    quant_group16<VEC>(v, a.q, row * a.ld_q + col, n, a.q_scale + row * a.qs_row + (int64_t)group * a.qs_group);
  }
}

}  // namespace tsm
