// Root-mean-square norm with the residual's addition before it and 16-, 32- and
// 8-bit outputs.
//
//   r = rnd(resid + delta),  v = r * rsqrt(mean(r^2) + eps) * gamma
//
// One pass: a CTA holds its row in registers between the sum of squares and the
// outputs, so every byte is read and written once and HBM bounds the kernel:
// 16384 x 4096 bf16, with the sum, y and q, 99.9 us (6.1 TB/s); walking the rows
// with the next one's loads in flight took it there from 180 us at a CTA a row.
#pragma once
#include "elem.cuh"

namespace tsm {

constexpr int NORM_MAX_THREADS = 1024;

// Sum over the CTA; `slots` holds one value a warp and must not be written again before the next barrier but one.
TSM_DEV float norm_cta_sum(float x, float* slots) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  if (blockDim.x > 32) {
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) x += slots[w];
  }
  return x;
}

// One CTA per row; thread t holds the eight-column chunks t, t + blockDim.x, ...
// (IT of them), so sixteen neighbouring lanes hold one 128-column scale group.
template <int IT, bool VEC>
__global__ void __launch_bounds__(NORM_MAX_THREADS) rmsnorm_kernel(const ts_moe_rmsnorm_args a) {
  __shared__ float warp_sum[NORM_MAX_THREADS / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = blockIdx.x;
  const int H = a.hidden;
  Raw8 rr[IT], dd[IT], gg[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int col = (i * (int)blockDim.x + (int)threadIdx.x) * 8, n = min(8, H - col);
    if (n > 0) {
      rr[i] = load_raw8<VEC>(a.resid, a.resid_type, row * a.ld_resid + col, n);
      if (a.delta) dd[i] = load_raw8<VEC>(a.delta, a.delta_type, row * a.ld_delta + col, n);
      if (a.gamma) gg[i] = load_raw8<VEC>(a.gamma, a.gamma_type, col, n);
    }
  }
  float v[IT][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int col = (i * (int)blockDim.x + (int)threadIdx.x) * 8, n = min(8, H - col);
    if (n > 0) {
      cvt8(rr[i], a.resid_type, v[i]);
      if (a.delta) {
        float d[8];
        cvt8(dd[i], a.delta_type, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += d[j];
        const Raw8 r = round8(v[i], a.resid_type);  // the stream's own type: the norm reads what the stream holds
        cvt8(r, a.resid_type, v[i]);
        if (a.resid_out) store_raw8<VEC>(a.resid_out, a.resid_type, row * a.ld_resid_out + col, n, r);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += VEC || j < n ? v[i][j] * v[i][j] : 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  ss = norm_cta_sum(ss, warp_sum);
  const float rstd = rsqrtf(ss / (float)H + a.eps);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int chunk = i * (int)blockDim.x + (int)threadIdx.x, col = chunk * 8, n = min(8, H - col);
    if (n > 0) {
      float g[8];
      if (a.gamma) cvt8(gg[i], a.gamma_type, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] *= rstd;
        if (a.gamma) v[i][j] *= g[j];
        if (!VEC && j >= n) v[i][j] = 0.f;  // past the row's end: nothing for the group's amax, whatever rstd is
      }
      if (a.y) store_raw8<VEC>(a.y, a.y_type, row * a.ld_y + col, n, round8(v[i], a.y_type));
    }
    if (a.q)
      quant_group<16, VEC>(*reinterpret_cast<const float(*)[1][8]>(&v[i]), a.q, row * a.ld_q + col, n,
                           a.q_scale + row * a.qs_row + (int64_t)(chunk >> 4) * a.qs_group);
  }
}

// Many rows: resident CTAs walk over the rows, and the next row's loads are in
// flight while this row is summed and written.  Eight lanes hold a 128-column
// group, two chunks of eight columns each: thread t's stand in group t / 8.
// RW, DW: resid, delta in 32 bits.
template <int MAX_THREADS, bool RW, bool DW>
__global__ void __launch_bounds__(MAX_THREADS, MAX_THREADS > 256 ? 1024 / MAX_THREADS : RW || DW ? 2 : 3) rmsnorm_rows_kernel(const ts_moe_rmsnorm_args a) {
  __shared__ float warp_sum[2][MAX_THREADS / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int H = a.hidden, group = (int)threadIdx.x / 8, col0 = group * SCALE_BLOCK + ((int)threadIdx.x & 7) * 8;
  Raw<RW> nr[2];
  Raw<DW> nd[2];
  constexpr bool HOLD = MAX_THREADS <= 256;  // else the registers go to the loads in flight, and gamma comes from L1
  Raw8 gg[2];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = col0 + c * 64;
      if (row < a.rows && col < H) {
        nr[c] = load_vec<RW>(a.resid, row * a.ld_resid + col);
        if (a.delta) nd[c] = load_vec<DW>(a.delta, row * a.ld_delta + col);
      }
    }
  };
  int64_t row = blockIdx.x;
  fetch(row);
  if (HOLD && a.gamma) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = col0 + c * 64;
      if (col < H) gg[c] = load_raw8<true>(a.gamma, a.gamma_type, col, 8);
    }
  }
  for (int buf = 0; row < a.rows; buf ^= 1) {
    float v[2][8], ss = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = col0 + c * 64;
      if (col < H) {
        cvt_vec<RW>(nr[c], a.resid_type, v[c]);
        if (a.delta) {
          float d[8];
          cvt_vec<DW>(nd[c], a.delta_type, d);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] += d[j];
          const Raw8 r = round8(v[c], RW ? TS_DT_FP32 : a.resid_type);
          cvt8(r, RW ? TS_DT_FP32 : a.resid_type, v[c]);
          if (a.resid_out) store_raw8<true>(a.resid_out, RW ? TS_DT_FP32 : a.resid_type, row * a.ld_resid_out + col, 8, r);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += v[c][j] * v[c][j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = 0.f;
      }
    }
    const int64_t at = row;
    row += gridDim.x;
    fetch(row);
    const float rstd = rsqrtf(norm_cta_sum(ss, warp_sum[buf]) / (float)H + a.eps);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = col0 + c * 64;
      if (col < H) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] *= rstd;
        if (a.gamma) {
          float g[8];
          cvt8(HOLD ? gg[c] : load_raw8<true>(a.gamma, a.gamma_type, col, 8), a.gamma_type, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] *= g[j];
        }
        if (a.y) store_raw8<true>(a.y, a.y_type, at * a.ld_y + col, 8, round8(v[c], a.y_type));
      }
    }
    if (a.q) quant_group<8, true>(v, a.q, at * a.ld_q + col0, H - col0, a.q_scale + at * a.qs_row + (int64_t)group * a.qs_group);
  }
}

}  // namespace tsm
