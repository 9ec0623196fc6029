// C ABI of the operators next to the routed half: argument checks, launch
// shapes and launches.  No call allocates or synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "../../../include/ts_moe_ops.h"
#include "../errors.h"
#include "act.cuh"
#include "balance.cuh"
#include "matmul_simple.cuh"
#include "norm.cuh"

using namespace tsm;

namespace {

ts_moe_status bad(const char* msg) noexcept { return set_last_error(TS_MOE_EINVAL, msg); }

ts_moe_status cuda_bad(cudaError_t e, const char* what) noexcept {
  char buf[256];
  std::snprintf(buf, sizeof(buf), "%s: %s", what, cudaGetErrorString(e));
  return set_last_error(TS_MOE_ECUDA, buf);
}

bool known_type(int t) { return t == TS_DT_BF16 || t == TS_DT_FP16 || t == TS_DT_FP32; }

bool aligned(const void* p, int64_t ld_bytes, int to) { return (uintptr_t)p % to == 0 && ld_bytes % to == 0; }
bool aligned_rows(const void* p, int64_t ld, int type) { return !p || aligned(p, ld * dt_size(type), 16); }

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int block, size_t smem, void* stream, Args... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(block);
  lc.dynamicSmemBytes = smem;
  lc.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

ts_moe_status done(cudaError_t e, const char* what) { return e == cudaSuccess ? TS_MOE_OK : cuda_bad(e, what); }

template <bool VEC>
cudaError_t launch_norm(const ts_moe_rmsnorm_args& a, void* stream) {
  const int chunks = cdiv(a.hidden, 8);
  const int it = a.rows <= 1024 ? (chunks <= 1024 ? 1 : 2) : 4;
  const int threads = std::max(32, cdiv(cdiv(chunks, it), 32) * 32);
  auto k = it == 1 ? rmsnorm_kernel<1, VEC> : it == 2 ? rmsnorm_kernel<2, VEC> : rmsnorm_kernel<4, VEC>;
  return launch(k, dim3(a.rows), threads, 0, stream, a);
}

}  // namespace

extern "C" {

ts_moe_status ts_moe_rmsnorm(const ts_moe_rmsnorm_args* args, void* stream) {
  if (!args) return bad("rmsnorm: args is NULL");
  const ts_moe_rmsnorm_args& a = *args;
  if (a.rows < 0 || a.rows > TS_MOE_MAX_ROWS) return bad("rmsnorm: rows must be in [0, 2^24]");
  if (a.hidden < 1 || a.hidden > 16384) return bad("rmsnorm: hidden must be in [1, 16384]");
  if (!known_type(a.resid_type) || (a.delta && !known_type(a.delta_type)) || (a.gamma && !known_type(a.gamma_type)) ||
      (a.y && !known_type(a.y_type)))
    return bad("rmsnorm: unknown element type");
  if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return bad("rmsnorm: eps must be finite and not negative");
  if (!a.y && !a.q) return bad("rmsnorm: y and q are both NULL");
  if ((a.q != nullptr) != (a.q_scale != nullptr)) return bad("rmsnorm: q and q_scale must be given together");
  if (a.resid_out && !a.delta) return bad("rmsnorm: resid_out without delta");
  if (a.rows == 0) return TS_MOE_OK;
  if (!a.resid) return bad("rmsnorm: resid is NULL");
  if (a.ld_resid < a.hidden || (a.delta && a.ld_delta < a.hidden) || (a.resid_out && a.ld_resid_out < a.hidden) ||
      (a.y && a.ld_y < a.hidden) || (a.q && a.ld_q < a.hidden))
    return bad("rmsnorm: a row stride is smaller than hidden");
  if (a.resid_out == a.resid && a.ld_resid_out != a.ld_resid && a.resid_out) return bad("rmsnorm: resid_out in place needs resid's stride");
  const bool vec = a.hidden % 8 == 0 && aligned_rows(a.resid, a.ld_resid, a.resid_type) &&
                   aligned_rows(a.delta, a.ld_delta, a.delta_type) && aligned_rows(a.gamma, 0, a.gamma_type) &&
                   aligned_rows(a.resid_out, a.ld_resid_out, a.resid_type) && aligned_rows(a.y, a.ld_y, a.y_type) &&
                   (!a.q || aligned(a.q, a.ld_q, 8));
  return done(vec ? launch_norm<true>(a, stream) : launch_norm<false>(a, stream), "rmsnorm launch");
}

ts_moe_status ts_moe_act_quant(const ts_moe_act_quant_args* args, void* stream) {
  if (!args) return bad("act_quant: args is NULL");
  const ts_moe_act_quant_args& a = *args;
  if (a.rows < 0 || a.rows > TS_MOE_MAX_ROWS) return bad("act_quant: rows must be in [0, 2^24]");
  if (a.inter < 1 || a.inter > 65536) return bad("act_quant: inter must be in [1, 65536]");
  if (a.act != TS_ACT_SWIGLU && a.act != TS_ACT_SWIGLU_CLAMPED) return bad("act_quant: unknown act");
  if (!known_type(a.in_type)) return bad("act_quant: unknown element type");
  if (a.act == TS_ACT_SWIGLU_CLAMPED && (!std::isfinite(a.act_alpha) || !(a.act_limit > 0.f)))
    return bad("act_quant: clamped SwiGLU needs a finite alpha and a positive limit");
  if (a.rows == 0) return TS_MOE_OK;
  if (!a.gate || !a.up || !a.q || !a.q_scale) return bad("act_quant: gate, up, q and q_scale must be non-NULL");
  if (a.ld_gate < a.inter || a.ld_up < a.inter || a.ld_q < a.inter) return bad("act_quant: a row stride is smaller than inter");
  const bool vec = a.inter % 8 == 0 && aligned_rows(a.gate, a.ld_gate, a.in_type) && aligned_rows(a.up, a.ld_up, a.in_type) &&
                   aligned(a.q, a.ld_q, 8);
  const int64_t units = (int64_t)a.rows * cdiv(a.inter, SCALE_BLOCK);
  const int grid = (int)std::min<int64_t>((units + ACT_THREADS / 16 - 1) / (ACT_THREADS / 16), 148 * 8);
  return done(launch(vec ? act_quant_kernel<true> : act_quant_kernel<false>, dim3(grid), ACT_THREADS, 0, stream, a), "act_quant launch");
}

ts_moe_status ts_moe_fp8_matmul(const ts_moe_fp8_matmul_args* args, void* stream) {
  if (!args) return bad("fp8_matmul: args is NULL");
  const ts_moe_fp8_matmul_args& a = *args;
  if (a.rows < 0 || a.rows > TS_MOE_MAX_ROWS) return bad("fp8_matmul: rows must be in [0, 2^24]");
  if (a.n < 1 || a.n > 1 << 20 || a.k < 1 || a.k > 1 << 20) return bad("fp8_matmul: n and k must be in [1, 2^20]");
  if (a.num_groups < 1 || a.num_groups > TS_MOE_MAX_EXPERTS) return bad("fp8_matmul: num_groups must be in [1, 256]");
  if (!a.offsets && a.num_groups != 1) return bad("fp8_matmul: more than one group needs offsets");
  if (!known_type(a.out_type)) return bad("fp8_matmul: unknown out_type");
  if (a.reserved) return bad("fp8_matmul: reserved must be 0");
  if (a.rows == 0) return TS_MOE_OK;
  if (!a.a || !a.a_scale || !a.b || !a.b_scale || !a.out) return bad("fp8_matmul: a, a_scale, b, b_scale and out must be non-NULL");
  if (a.ld_a < a.k || a.ld_b < a.k || a.ld_out < a.n || (a.add && a.ld_add < a.n)) return bad("fp8_matmul: a row stride is smaller than the row");
  if (!aligned(a.a, a.ld_a, 16) || !aligned(a.b, a.ld_b, 16) || a.b_group % 16)
    return bad("fp8_matmul: the rows of a and b must start at 16-byte boundaries");
  if (a.num_groups > 1 && a.b_group < (int64_t)(a.n - 1) * a.ld_b + a.k) return bad("fp8_matmul: b_group is smaller than a matrix");
  if (a.add == a.out && a.ld_add != a.ld_out) return bad("fp8_matmul: add in place needs out's stride");
  const int row_tiles = std::min(cdiv(a.rows, SM_T), 64);
  return done(launch(fp8_matmul_simple_kernel, dim3(cdiv(a.n, SM_T), a.num_groups, row_tiles), 256, 0, stream, a), "fp8_matmul launch");
}

static int balance_ctas(int rows, int experts) {
  const int rows_per_pass = BAL_WARPS * (32 / balance_lanes(experts));
  return std::min(cdiv(std::max(rows, 1), rows_per_pass * 4), BAL_MAX_CTAS);
}

uint64_t ts_moe_balance_workspace(int32_t rows, int32_t experts) {
  if (rows < 0 || rows > TS_MOE_MAX_ROWS || experts < 1 || experts > BAL_MAX_E) return 0;
  return sizeof(BalanceHead) + (uint64_t)balance_ctas(rows, experts) * experts * sizeof(float);
}

ts_moe_status ts_moe_balance(const ts_moe_balance_args* args, void* stream) {
  if (!args) return bad("balance: args is NULL");
  const ts_moe_balance_args& a = *args;
  if (a.rows < 0 || a.rows > TS_MOE_MAX_ROWS) return bad("balance: rows must be in [0, 2^24]");
  if (a.experts < 1 || a.experts > BAL_MAX_E) return bad("balance: experts must be in [1, 256]");
  if (a.top_k < 1 || a.top_k > TS_MOE_MAX_TOPK || a.top_k > a.experts) return bad("balance: top_k must be in [1, min(8, experts)]");
  if (a.score != TS_SCORE_SOFTMAX_SELECTED && a.score != TS_SCORE_SOFTMAX_ALL_NORENORM && a.score != TS_SCORE_SIGMOID_RENORM)
    return bad("balance: unknown score");
  if (!known_type(a.dtype)) return bad("balance: unknown element type");
  if (!std::isfinite(a.coef)) return bad("balance: coef must be finite");
  if (!a.loss || !a.counts) return bad("balance: loss and counts must be non-NULL");
  if (a.rows > 0) {
    if (!a.logits || !a.idx) return bad("balance: logits and idx must be non-NULL");
    if (a.ld_logits < a.experts || a.ld_idx < a.top_k || (a.dlogits && a.ld_dlogits < a.experts))
      return bad("balance: a row stride is smaller than the row");
  }
  if (!a.workspace || (uintptr_t)a.workspace % 16) return bad("balance: workspace must be non-NULL and 16-byte aligned");
  if (a.workspace_bytes < ts_moe_balance_workspace(a.rows, a.experts)) return bad("balance: workspace is too small");

  BalanceParams p;
  p.a = a;
  p.head = (BalanceHead*)a.workspace;
  p.part = (float*)((char*)a.workspace + sizeof(BalanceHead));
  const int lanes = balance_lanes(a.experts);
  int ctas = balance_ctas(a.rows, a.experts);
  if ((int64_t)a.rows * a.experts <= 16384) ctas = 1;
  p.counted = ctas > 1 && a.dlogits ? 1 : 0;
  if (ctas > 1) {
    const cudaError_t e = cudaMemsetAsync(p.head, 0, sizeof(BalanceHead), (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_bad(e, "balance workspace");
  }
  if (p.counted) {
    const int n = std::min(cdiv(a.rows * a.top_k, BAL_THREADS * 8), 148);
    const cudaError_t e = launch(balance_count_kernel, dim3(n), BAL_THREADS, 0, stream, p);
    if (e != cudaSuccess) return cuda_bad(e, "balance count launch");
  }
  auto k = lanes == 2   ? balance_kernel<2, 1>
           : lanes == 4  ? balance_kernel<4, 1>
           : lanes == 8  ? balance_kernel<8, 1>
           : lanes == 16 ? balance_kernel<16, 1>
           : a.experts <= 128 ? balance_kernel<32, 1>
                              : balance_kernel<32, 2>;
  return done(launch(k, dim3(ctas), BAL_THREADS, 0, stream, p), "balance launch");
}

}  // extern "C"
