// The activation between an expert's two products, as 8-bit rows with one scale
// per 128 columns.  Elementwise: HBM bounds it (gate and up read once, codes and
// scales written once).
#pragma once
#include <type_traits>

#include "elem.cuh"

namespace tsm {

constexpr int ACT_THREADS = 256;

// sigmoid(x) = 1 / (1 + 2^(-x log2 e)): the exponent's rounding is off by |x| 2^-24 relative, which shows only where
// the sigmoid itself is small; two instructions of the special-function unit, whose rate would otherwise come to bound
// the kernel before HBM does.  Below -87 that is 0, though e^x times a large factor may be an ordinary value: below FAR,
// where sigmoid(x) is e^x, the product is formed with e^(x / 2) on either side.
constexpr float FAR = -64.f;
TSM_DEV float times_far_sigmoid(float a, float x, float b) {
  const float h = ex2(0.5f * LOG2E * x);
  return (a * h) * (b * h);
}

// v from gate and up, eight values, two to an instruction; ANY: with the far gates' way.  The clamps keep a NaN.
template <bool CLAMPED, bool ANY>
TSM_DEV void act8(const ts_moe_act_quant_args& a, const float (&g)[8], const float (&u)[8], int n, float (&v)[8]) {
  const uint64_t one = pair(1.f, 1.f);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    uint64_t p, b;
    if (CLAMPED) {
      p = pair(min_nan(g[j], a.act_limit), min_nan(g[j + 1], a.act_limit));
      b = add2(pair(max_nan(min_nan(u[j], a.act_limit), -a.act_limit), max_nan(min_nan(u[j + 1], a.act_limit), -a.act_limit)), one);
    } else {
      p = pair(g[j], g[j + 1]);
      b = pair(u[j], u[j + 1]);
    }
    const uint64_t x = CLAMPED ? mul2(p, pair(a.act_alpha, a.act_alpha)) : p;
    const float2 e = unpair(mul2(x, pair(-LOG2E, -LOG2E)));
    const float2 d = unpair(add2(pair(ex2(e.x), ex2(e.y)), one));
    const float2 r = unpair(mul2(mul2(p, pair(rcp(d.x), rcp(d.y))), b));
    v[j] = r.x, v[j + 1] = r.y;
    if (ANY) {
      const float2 xs = unpair(x), ps = unpair(p), bs = unpair(b);
      if (xs.x < FAR) v[j] = times_far_sigmoid(ps.x, xs.x, bs.x);
      if (xs.y < FAR) v[j + 1] = times_far_sigmoid(ps.y, xs.y, bs.y);
    }
    if (CLAMPED && j >= n) v[j] = 0.f;  // past the row's end, where u + 1 is not 0
    if (CLAMPED && j + 1 >= n) v[j + 1] = 0.f;
  }
}

// Whether some of sixteen gates as they lie in memory have bits above `far` (act_far_bits): one whole-number maximum for two
// or more of them, before any is converted.
template <bool WIDE>
TSM_DEV bool any_far(const Raw<WIDE> (&g)[2], uint32_t far) {
  if constexpr (WIDE) {
    uint32_t m[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
      m[c] = __vimax3_u32(__vimax3_u32(g[c].a.x, g[c].a.y, g[c].a.z), __vimax3_u32(g[c].a.w, g[c].b.x, g[c].b.y), max(g[c].b.z, g[c].b.w));
    return max(m[0], m[1]) > far;
  } else {
    const uint32_t m = __vimax3_u16x2(__vimax3_u16x2(g[0].a.x, g[0].a.y, g[0].a.z), __vimax3_u16x2(g[0].a.w, g[1].a.x, g[1].a.y),
                                      __vmaxu2(g[1].a.z, g[1].a.w));
    return max(m >> 16, m & 0xFFFF) > far;
  }
}

// A warp takes four neighbouring groups of a row, eight lanes and two chunks of eight columns a lane each; quads
// row-major.  step_rows, step_quads: the grid's warps as whole rows of quads and the rest, so that the loop divides
// nothing.  With VEC the next quad's loads are issued before this one is worked on: 8192 x 14336 bf16 in 95 us
// (6.2 TB/s, HBM bounds it), clamped in 104 us; without, and with 16 lanes a group and IEEE divisions, 162 us.  The far
// gates' way as a branch beside the other cost 6 us; chosen before the conversions, and with values in pairs, none.
template <bool VEC, bool WIDE, bool CLAMPED>
__global__ void __launch_bounds__(ACT_THREADS, VEC && WIDE ? 2 : 4)
    act_quant_kernel(const ts_moe_act_quant_args a, int quads, int step_rows, int step_quads, uint32_t far) {
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
    auto values = [&](auto any) {
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
          act8<CLAMPED, decltype(any)::value>(a, g, u, VEC ? 8 : n, v[c]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] = 0.f;
        }
      }
    };
    if (!VEC || any_far<WIDE>(g2, far))
      values(std::true_type());
    else
      values(std::false_type());
    quant_group<8, VEC>(v, a.q, at * a.ld_q + col, a.inter - col, a.q_scale + at * a.qs_row + (int64_t)group * a.qs_group);
  }
}

}  // namespace tsm
