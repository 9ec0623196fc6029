// E4M3 product with block scales, dense and grouped: the plain form on the FP32 pipe.
#pragma once
#include "elem.cuh"

namespace tsm {

// Row range of group g; see ts_moe_fp8_matmul_args.offsets.
TSM_DEV void group_rows(const ts_moe_fp8_matmul_args& a, int g, int& lo, int& hi) {
  lo = 0;
  hi = a.rows;
  if (!a.offsets) return;
  hi = 0;
  for (int i = 0; i <= g + 1; ++i) {
    lo = hi;
    hi = max(hi, min(a.offsets[i], a.rows));
  }
}

TSM_DEV float e4m3_to_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

TSM_DEV float load1(const void* p, int type, int64_t i) {
  return type == TS_DT_FP32 ? ((const float*)p)[i]
         : type == TS_DT_BF16 ? __bfloat162float(((const __nv_bfloat16*)p)[i])
                              : __half2float(((const __half*)p)[i]);
}
TSM_DEV void store1(void* p, int type, int64_t i, float v) {
  if (type == TS_DT_FP32)
    ((float*)p)[i] = v;
  else if (type == TS_DT_BF16)
    ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
  else
    ((__half*)p)[i] = __float2half_rn(v);
}

constexpr int SM_T = 32;

// 32 x 32 outputs per CTA of 256 threads; blockIdx = (n tile, group, 0), row tiles of the group in a loop.
__global__ void __launch_bounds__(256) fp8_matmul_simple_kernel(const ts_moe_fp8_matmul_args a) {
  __shared__ float sa[SM_T][SCALE_BLOCK + 1], sb[SM_T][SCALE_BLOCK + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int g = blockIdx.y, n0 = blockIdx.x * SM_T, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  int lo, hi;
  group_rows(a, g, lo, hi);
  for (int m0 = lo + blockIdx.z * SM_T; m0 < hi; m0 += gridDim.z * SM_T) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < a.k; k0 += SCALE_BLOCK) {
      __syncthreads();
      for (int i = threadIdx.x; i < SM_T * SCALE_BLOCK; i += 256) {
        const int r = i / SCALE_BLOCK, c = i % SCALE_BLOCK;
        const bool kin = k0 + c < a.k;
        sa[r][c] = kin && m0 + r < hi ? e4m3_to_f32(a.a[(int64_t)(m0 + r) * a.ld_a + k0 + c]) : 0.f;
        sb[r][c] = kin && n0 + r < a.n ? e4m3_to_f32(a.b[g * a.b_group + (int64_t)(n0 + r) * a.ld_b + k0 + c]) : 0.f;
      }
      __syncthreads();
      const int kb = k0 / SCALE_BLOCK;
      const float bs = a.b_scale[g * a.bs_group + (int64_t)(n0 / SCALE_BLOCK) * a.bs_row + kb * a.bs_block];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty + 8 * i;
        float p = 0.f;
        for (int c = 0; c < SCALE_BLOCK; ++c) p += sa[r][c] * sb[tx][c];
        if (m0 + r < hi) acc[i] += p * (a.a_scale[(int64_t)(m0 + r) * a.as_row + kb * a.as_block] * bs);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + ty + 8 * i;
      if (m < hi && n0 + tx < a.n) {
        float v = acc[i];
        if (a.add) v += load1(a.add, a.out_type, m * a.ld_add + n0 + tx);
        store1(a.out, a.out_type, m * a.ld_out + n0 + tx, v);
      }
    }
  }
}

}  // namespace tsm
