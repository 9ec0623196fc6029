// Root-mean-square norm with the residual's addition before it and 16-, 32- and
// 8-bit outputs.
//
//   r = rnd(resid + delta),  v = r * rsqrt(mean(r^2) + eps) * gamma
//
// One pass: a CTA holds its row in registers between the sum of squares and the
// outputs, so every byte is read and written once and HBM bounds the kernel.
#pragma once
#include "elem.cuh"

namespace tsm {

// Threads of the largest row's CTA: one or two chunks per thread for few rows, four for many.
template <int IT>
constexpr int NORM_MAX_THREADS = IT == 4 ? 512 : 1024;

// One CTA per row; thread t holds the eight-column chunks t, t + blockDim.x, ...
// (IT of them), so sixteen neighbouring lanes hold one 128-column scale group.
template <int IT, bool VEC>
__global__ void __launch_bounds__(NORM_MAX_THREADS<IT>) rmsnorm_kernel(const ts_moe_rmsnorm_args a) {
  __shared__ float warp_sum[NORM_MAX_THREADS<IT> / 32];
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
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
  if (blockDim.x > 32) {
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) ss += warp_sum[w];
  }
  const float rstd = 1.f / sqrtf(ss / (float)H + a.eps);
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
      quant_group16<VEC>(v[i], a.q, row * a.ld_q + col, n, a.q_scale + row * a.qs_row + (int64_t)(chunk >> 4) * a.qs_group);
  }
}

}  // namespace tsm
