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

// v from gate and up, eight values.
TSM_DEV void act8(const ts_moe_act_quant_args& a, const float (&g)[8], const float (&u)[8], int n, float (&v)[8]) {
  if (a.act == TS_ACT_SWIGLU) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = g[j] * sigmoid_f(g[j]) * u[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // written with comparisons so that a NaN stays one
      const float gg = g[j] > a.act_limit ? a.act_limit : g[j];
      const float uu = u[j] > a.act_limit ? a.act_limit : u[j] < -a.act_limit ? -a.act_limit : u[j];
      v[j] = j < n ? gg * sigmoid_f(a.act_alpha * gg) * (uu + 1.f) : 0.f;
    }
  }
}

// A warp takes four neighbouring groups of a row, eight lanes and two chunks of eight columns a lane each; quads
// row-major.  step_rows, step_quads: the grid's warps as whole rows of quads and the rest, so that the loop divides
// nothing.  With VEC the next quad's loads are issued before this one is worked on: 8192 x 14336 bf16 in 96 us
// (6.1 TB/s, HBM bounds it); without, and with 16 lanes a group and IEEE divisions, 162 us.
template <bool VEC, bool WIDE>
__global__ void __launch_bounds__(ACT_THREADS, VEC && WIDE ? 2 : 4)
    act_quant_kernel(const ts_moe_act_quant_args a, int quads, int step_rows, int step_quads) {
  grid_dep_wait();
  grid_dep_launch();
  const unsigned w = blockIdx.x * (ACT_THREADS / 32) + (threadIdx.x >> 5);
  int64_t row = w / (unsigned)quads;
  int quad = (int)(w - (unsigned)row * (unsigned)quads);
  const int sub = (threadIdx.x >> 3) & 3, lane_col = (threadIdx.x & 7) * 8;
  Raw<WIDE> ng[2], nu[2];
  auto fetch = [&]() {
    const int col = (quad * 4 + sub) * SCALE_BLOCK + lane_col;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (row < a.rows && col + c * 64 < a.inter) {
        ng[c] = load_vec<WIDE>(a.gate, row * a.ld_gate + col + c * 64);
        nu[c] = load_vec<WIDE>(a.up, row * a.ld_up + col + c * 64);
      }
    }
  };
  if (VEC) fetch();
  while (row < a.rows) {
    const int64_t at = row;
    const int group = quad * 4 + sub, col = group * SCALE_BLOCK + lane_col;
    float v[2][8];
    Raw<WIDE> g2[2], u2[2];
    if (VEC) {
#pragma unroll
      for (int c = 0; c < 2; ++c) g2[c] = ng[c], u2[c] = nu[c];
    }
    row += step_rows;
    quad += step_quads;
    if (quad >= quads) {
      quad -= quads;
      ++row;
    }
    if (VEC) fetch();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = min(8, a.inter - col - c * 64);
      if (n > 0) {
        float g[8], u[8];
        if (VEC) {
          cvt_vec<WIDE>(g2[c], a.in_type, g);
          cvt_vec<WIDE>(u2[c], a.in_type, u);
        } else {
          cvt8(load_raw8<false>(a.gate, a.in_type, at * a.ld_gate + col + c * 64, n), a.in_type, g);
          cvt8(load_raw8<false>(a.up, a.in_type, at * a.ld_up + col + c * 64, n), a.in_type, u);
        }
        act8(a, g, u, VEC ? 8 : n, v[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = 0.f;
      }
    }
    quant_group<8, VEC>(v, a.q, at * a.ld_q + col, a.inter - col, a.q_scale + at * a.qs_row + (int64_t)group * a.qs_group);
  }
}

}  // namespace tsm
