// The activation between an expert's two products, as 8-bit rows with one scale
// per 128 columns.  Elementwise: HBM bounds it (gate and up read once, codes and
// scales written once).
#pragma once
#include "elem.cuh"

namespace tsm {

constexpr int ACT_THREADS = 256;

// 1 / (1 + 2^(-x log2 e)).  The exponent's rounding is off by |x| 2^-24 relative, which shows only where the
// sigmoid itself is small; four instructions, two of them on the special-function unit, whose rate would
// otherwise come to bound the kernel before HBM does.
TSM_DEV float sigmoid_f(float x) { return rcp(1.f + ex2(-LOG2E * x)); }

// A warp takes two neighbouring groups of a row (its halves, eight columns a lane) at a time; pairs row-major.
// step_rows, step_pairs: the grid's warps as whole rows of pairs and the rest, so that the loop divides nothing.
template <bool VEC>
__global__ void __launch_bounds__(ACT_THREADS) act_quant_kernel(const ts_moe_act_quant_args a, int pairs, int step_rows, int step_pairs) {
  grid_dep_wait();
  grid_dep_launch();
  const unsigned w = blockIdx.x * (ACT_THREADS / 32) + (threadIdx.x >> 5);
  int64_t row = w / (unsigned)pairs;
  int pair = (int)(w - (unsigned)row * (unsigned)pairs);
  while (row < a.rows) {
    const int group = pair * 2 + ((threadIdx.x >> 4) & 1), col = group * SCALE_BLOCK + (threadIdx.x & 15) * 8;
    const int n = min(8, a.inter - col);
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
    row += step_rows;
    pair += step_pairs;
    if (pair >= pairs) {
      pair -= pairs;
      ++row;
    }
  }
}

}  // namespace tsm
