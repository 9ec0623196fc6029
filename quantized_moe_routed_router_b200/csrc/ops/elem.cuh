// Element access shared by the operators: eight consecutive elements of a
// 16- or 32-bit row as float32, and groups of 128 columns as E4M3.
#pragma once
#include <cfloat>
#include <cuda_fp8.h>

#include "../../../include/ts_moe_ops.h"
#include "../common.cuh"

namespace tsm {

constexpr int GPU_SMS = 148;  // a B200's; kernels that walk over rows size their grids by it, so another number costs time only
constexpr int SCALE_BLOCK = TS_MOE_SCALE_BLOCK;
constexpr float E4M3_MAX = 448.f;
constexpr float AMAX_FLOOR = 0x1p-100f;  // the smallest amax a scale is formed from: scale and 1 / scale stay normal

__host__ __device__ inline int cdiv(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline int dt_size(int type) { return type == TS_DT_FP32 ? 4 : 2; }

// Eight elements as they lie in memory: 16-bit types fill `a` only.
struct Raw8 {
  uint4 a, b;
};

// Loads elements [off, off + n) of a row, n <= 8.  VEC: n = 8 and the address
// is 16-byte aligned; otherwise at whatever place an element can have, the rest zero.
template <bool VEC>
TSM_DEV Raw8 load_raw8(const void* base, int type, int64_t off, int n) {
  Raw8 r;
  if (VEC) {
    if (type == TS_DT_FP32) {
      const uint4* p = (const uint4*)((const float*)base + off);
      r.a = p[0];
      r.b = p[1];
    } else {
      r.a = *(const uint4*)((const uint16_t*)base + off);
    }
    return r;
  }
  uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (type == TS_DT_FP32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j] = ((const uint32_t*)base)[off + j];
  } else if (n == 8) {
    // four words, or three between two halves where the row starts at an odd element
    const uint16_t* p = (const uint16_t*)base + off;
    if ((uintptr_t)p % 4 == 0) {
      const uint32_t* q = (const uint32_t*)p;
      w[0] = q[0], w[1] = q[1], w[2] = q[2], w[3] = q[3];
    } else {
      const uint32_t* q = (const uint32_t*)(p + 1);
      const uint32_t a = q[0], b = q[1], c = q[2], first = p[0], last = p[7];
      w[0] = first | a << 16, w[1] = a >> 16 | b << 16, w[2] = b >> 16 | c << 16, w[3] = c >> 16 | last << 16;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j / 2] |= (uint32_t)((const uint16_t*)base)[off + j] << (16 * (j % 2));
  }
  r.a = make_uint4(w[0], w[1], w[2], w[3]);
  r.b = make_uint4(w[4], w[5], w[6], w[7]);
  return r;
}

TSM_DEV void cvt8(const Raw8& r, int type, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if (type == TS_DT_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else if (type == TS_DT_FP16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  } else {
    const uint32_t u[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(w[j]);
      v[4 + j] = __uint_as_float(u[j]);
    }
  }
}

// The same where the kernel's instance knows the width: eight 16-bit elements take one uint4.
template <bool WIDE>
struct Raw;
template <>
struct Raw<false> {
  uint4 a;
};
template <>
struct Raw<true> {
  uint4 a, b;
};
// Eight elements at a 16-byte boundary; streamed: each is read once.
template <bool WIDE>
TSM_DEV Raw<WIDE> load_vec(const void* base, int64_t off) {
  Raw<WIDE> r;
  if constexpr (WIDE) {
    const uint4* p = (const uint4*)((const float*)base + off);
    r.a = __ldcs(p);
    r.b = __ldcs(p + 1);
  } else {
    r.a = __ldcs((const uint4*)((const uint16_t*)base + off));
  }
  return r;
}
template <bool WIDE>
TSM_DEV void cvt_vec(const Raw<WIDE>& r, int type, float (&v)[8]) {
  Raw8 w;
  w.a = r.a;
  if constexpr (WIDE) {
    w.b = r.b;
    cvt8(w, TS_DT_FP32, v);
  } else {
    cvt8(w, type == TS_DT_BF16 ? TS_DT_BF16 : TS_DT_FP16, v);
  }
}

TSM_DEV uint32_t pack2(float x, float y, int type) {
  if (type == TS_DT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight float32 values rounded once to the type.
TSM_DEV Raw8 round8(const float (&v)[8], int type) {
  Raw8 r;
  if (type == TS_DT_FP32) {
    r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    r.a = make_uint4(pack2(v[0], v[1], type), pack2(v[2], v[3], type), pack2(v[4], v[5], type), pack2(v[6], v[7], type));
    r.b = make_uint4(0, 0, 0, 0);
  }
  return r;
}

template <bool VEC>
TSM_DEV void store_raw8(void* base, int type, int64_t off, int n, const Raw8& r) {
  if (VEC) {
    if (type == TS_DT_FP32) {
      uint4* p = (uint4*)((float*)base + off);
      p[0] = r.a;
      p[1] = r.b;
    } else {
      *(uint4*)((uint16_t*)base + off) = r.a;
    }
    return;
  }
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (type == TS_DT_FP32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) ((uint32_t*)base)[off + j] = w[j];
  } else if (n == 8) {
    uint16_t* p = (uint16_t*)base + off;
    if ((uintptr_t)p % 4 == 0) {
      uint32_t* q = (uint32_t*)p;
      q[0] = w[0], q[1] = w[1], q[2] = w[2], q[3] = w[3];
    } else {
      uint32_t* q = (uint32_t*)(p + 1);
      p[0] = (uint16_t)w[0], p[7] = (uint16_t)(w[3] >> 16);
      q[0] = w[0] >> 16 | w[1] << 16, q[1] = w[1] >> 16 | w[2] << 16, q[2] = w[2] >> 16 | w[3] << 16;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) ((uint16_t*)base)[off + j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
  }
}

constexpr float LOG2E = 1.4426950408889634f;

// 2^x and 1 / x by the special-function unit (each within 2 ulp); 2^x is 0 below the normal range.
TSM_DEV float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
TSM_DEV float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Maximum and minimum that keep a NaN (fmaxf and fminf drop it).
TSM_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

TSM_DEV float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two values to an instruction.
TSM_DEV uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
TSM_DEV float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
TSM_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
TSM_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
TSM_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// LANES neighbouring lanes hold the 128 columns of one group in chunks of eight
// columns: chunk c of lane l stands at column (c LANES + l) 8 of the group (lanes
// past the row's end hold zeros).  Writes the group's E4M3 codes and, from its
// first lane, its scale, amax times the rounded 1 / 448.  The codes are of the
// rounded quotients by that scale: with 16-bit inputs some values in ten thousand
// stand exactly between two codes, and a product with an approximate reciprocal put
// a tenth of those on the other one.  One FMA forms what a first quotient q0 = v r
// (r the rounded 1 / scale) leaves of v, exactly while nothing in it is subnormal,
// and another adds its share (Markstein, IBM Journal of Research and Development 34,
// 1990).  A group's values share r, so a quotient costs two FMAs more than a
// product, and two values share an instruction: 16384 x 4096 norm 98.7 -> 99.9 us.
// The conversion saturates, so the group's largest value lands on 448 whichever way
// it rounds.
template <int LANES, bool VEC>
TSM_DEV void quant_group(const float (&v)[16 / LANES][8], uint8_t* q, int64_t off, int n, float* scale) {
  constexpr int C = 16 / LANES;
  float m = AMAX_FLOOR;
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[c][j]));
  }
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d, LANES));
  const float s = m * (1.f / E4M3_MAX);
  // A tiny group is taken times 2^64, which keeps the remainders out of the subnormal range; for an infinite scale they are
  // left out (0 and NaN stay what they are).  The reciprocal is rounded by the same step from the approximate one.
  const bool tiny = s < 0x1p-60f;
  const float b = tiny ? s * 0x1p64f : s, rest = b <= FLT_MAX ? -b : 0.f, r0 = rcp(b), inv = fmaf(fmaf(rest, r0, 1.f), r0, r0);
  uint64_t t[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) t[c][j] = pair(v[c][2 * j], v[c][2 * j + 1]);
  }
  if (tiny) {
    const uint64_t up = pair(0x1p64f, 0x1p64f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int j = 0; j < 4; ++j) t[c][j] = mul2(t[c][j], up);
    }
  }
  const uint64_t inv2 = pair(inv, inv), rest2 = pair(rest, rest);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t q0 = mul2(t[c][j], inv2);
      h[j] = __nv_cvt_float2_to_fp8x2(unpair(fma2(fma2(q0, rest2, t[c][j]), inv2, q0)), __NV_SATFINITE, __NV_E4M3);
    }
    const uint32_t w[2] = {h[0] | h[1] << 16, h[2] | h[3] << 16};
    const int64_t at = off + c * LANES * 8;
    const int nc = n - c * LANES * 8;
    if (VEC) {
      if (nc > 0) *(uint2*)(q + at) = make_uint2(w[0], w[1]);
    } else if (nc >= 8 && (uintptr_t)(q + at) % 8 == 0) {
      *(uint2*)(q + at) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < nc) q[at + j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    }
  }
  if (n > 0 && (threadIdx.x & (LANES - 1)) == 0) *scale = s;
}

}  // namespace tsm
