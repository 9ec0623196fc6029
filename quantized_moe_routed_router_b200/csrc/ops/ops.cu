// C ABI of the operators next to the routed half: argument checks, launch
// shapes and launches.  No call allocates or synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <numeric>

#include "../../../include/ts_moe_debug.h"
#include "../../../include/ts_moe_ops.h"
#include "../errors.h"
#include "act.cuh"
#include "balance.cuh"
#include "matmul.cuh"
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

// An element's place: loads and stores of elements need it.  NULL passes.
bool at_elements(const void* p, int type) { return (uintptr_t)p % dt_size(type) == 0; }
bool at_words(const void* p) { return (uintptr_t)p % 4 == 0; }

// Whether two of an output's [rows][cols] elements, at row * r + col * c, are one: dr rows and dc columns apart, dr r = dc c.
bool overlap(int64_t rows, int64_t cols, int64_t r, int64_t c) {
  const int64_t g = std::gcd(r, c);
  if (g == 0) return rows > 1 || cols > 1;
  return std::abs(c / g) < rows && std::abs(r / g) < cols;
}

// With programmatic dependent launch: the kernel's set-up overlaps the previous kernel's tail, and
// griddepcontrol.wait orders the data.  cluster: CTAs of a cluster along x.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), dim3 grid, int block, size_t smem, void* stream, int cluster, const Args&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(block);
  lc.dynamicSmemBytes = smem;
  lc.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int block, size_t smem, void* stream, const Args&... args) {
  return launch_clusters(kernel, grid, block, smem, stream, 1, args...);
}

// ----------------------------------------------------------------------------- product
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
constexpr int MAX_DEVICES = 64;

struct MatmulDevice {
  bool ready = false;
  int sms = 0;
};
std::mutex g_matmul_mu;
MatmulDevice g_matmul[MAX_DEVICES];
EncodeTiled g_encode = nullptr;

template <int BT>
constexpr size_t stream_smem() {
  return sizeof(StreamSmem<BT>) + 1024;  // the struct starts at a 1024-byte boundary inside
}
constexpr size_t tile_smem() { return sizeof(TileSmem); }
static_assert(tile_smem() <= 227 * 1024, "a CTA's shared memory");

template <int BT>
cudaError_t allow_stream() {
  return cudaFuncSetAttribute(fp8_stream_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)stream_smem<BT>());
}

// Once per device, with that device current: the SM count, the kernels' shared-memory attributes, and the driver's
// tensor-map encoder.
ts_moe_status matmul_setup(const MatmulDevice** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_bad(e, "cudaGetDevice");
  if (dev < 0 || dev >= MAX_DEVICES) return set_last_error(TS_MOE_EUNSUPPORTED, "device ordinal >= 64");
  std::unique_lock<std::mutex> lk(g_matmul_mu, std::defer_lock);
  try {
    lk.lock();
  } catch (...) {  // no exception leaves a C entry
    return set_last_error(TS_MOE_ECUDA, "fp8_matmul: the set-up's lock failed");
  }
  MatmulDevice& d = g_matmul[dev];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tile_smem());
    if (e == cudaSuccess) e = allow_stream<16>();
    if (e == cudaSuccess) e = allow_stream<32>();
    if (e != cudaSuccess) return cuda_bad(e, "fp8_matmul set-up");
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult r;
      e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r);
      if (e != cudaSuccess || r != cudaDriverEntryPointSuccess || !fn)
        return set_last_error(TS_MOE_ECUDA, "the driver has no cuTensorMapEncodeTiled");
      g_encode = (EncodeTiled)fn;
    }
    d.ready = true;
  }
  *out = &d;
  return TS_MOE_OK;
}

// Map of 8-bit rows, boxes of box_rows x 128 codes in the 128-byte swizzle; what lies past an extent reads as zero.
// groups < 0: two dimensions.
bool encode_rows(CUtensorMap* m, const uint8_t* p, int k, int rows, int64_t ld, int groups, int64_t group, int box_rows) {
  cuuint64_t dims[3] = {(cuuint64_t)k, (cuuint64_t)rows, (cuuint64_t)std::max(groups, 1)};
  cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)group};
  cuuint32_t box[3] = {SCALE_BLOCK, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, groups < 0 ? 2 : 3, (void*)p, dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of out for stores of 32 rows x 128 bytes; rows start and end at 16-byte boundaries.
bool encode_out(CUtensorMap* m, const ts_moe_fp8_matmul_args& a) {
  const int es = dt_size(a.out_type);
  cuuint64_t dims[2] = {(cuuint64_t)a.n, (cuuint64_t)a.rows}, strides[1] = {(cuuint64_t)a.ld_out * es};
  cuuint32_t box[2] = {(cuuint32_t)(128 / es), 32}, one[2] = {1, 1};
  const CUtensorMapDataType type = a.out_type == TS_DT_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : a.out_type == TS_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return g_encode(m, type, 2, a.out, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BT>
cudaError_t launch_stream(const MatmulParams& p, const CUtensorMap& ma, const CUtensorMap& mb, int clusters, void* stream) {
  return launch_clusters(fp8_stream_kernel<BT>, dim3(clusters * p.splits), ST_THREADS, stream_smem<BT>(), stream, p.splits, p, ma, mb);
}

// Which kernel, and how its work is cut.
struct MatmulPlan {
  enum Kind { ROWS, STREAM, TILE } kind;
  int bt;      // rows of an fp8_stream_kernel tile
  int splits;  // CTAs that share K
  int grid;    // CTAs, or clusters
};

// The times below are microseconds, of calls one after another.
MatmulPlan matmul_plan(const ts_moe_fp8_matmul_args& a, int sms) {
  const int kb = cdiv(a.k, SCALE_BLOCK), G = a.num_groups;
  const int64_t reached = std::min(G, a.rows);  // groups that can hold a row
  const int64_t mean = cdiv(a.rows, (int)reached);
  const int64_t tiles = (cdiv(a.rows, TL_M) + reached - 1) * cdiv(a.n, TL_N);
  const MatmulPlan tile = {MatmulPlan::TILE, 0, 1, (int)std::min<int64_t>(tiles, sms)};
  // A decode step: without set-up, while the CTAs run at once and a warp's share of K is a few blocks (against
  // fp8_stream_kernel: 1 x 1024 x 2048 3.4 : 5.3, 4 x 2880 x 2880 4.9 : 6.1, 1 x 4096 x 4096 6.2 : 6.4, 16 x 1024 x 2048
  // 4.6 : 5.6; but 8 x 5760 x 2880 8.0 : 6.7, 1 x 2048 x 8192 8.7 : 8.2, 16 x 2048 x 4096 7.0 : 6.6)
  const int row_ctas = cdiv(a.n, RW_N);
  if (!a.offsets && a.rows <= RW_MAX_ROWS && row_ctas <= 2 * sms && kb <= (a.rows <= 8 ? 32 : 16))
    return {MatmulPlan::ROWS, 0, 1, row_ctas};
  const int bt = mean <= 16 ? 16 : 32;
  const int64_t items = (cdiv(a.rows, bt) + reached - 1) * cdiv(a.n, ST_N);
  // K is split while that leaves one CTA an SM, or two where one would leave K whole, never into a second wave: a cluster
  // joins its shares in about a microsecond (64 x 4096 x 4096, with an earlier, slower join: whole 14.8,
  // 2 ways 11.5, 4 ways 11.4, 8 ways 25.0).
  const int splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(MAX_SPLITS, kb), (items * 2 <= sms ? sms : 2 * sms) / items));
  // A split makes at most sms or 2 sms CTAs of all items: every cluster has one item, as the kernel's join needs it.
  const MatmulPlan stream = {MatmulPlan::STREAM, bt, splits, (int)std::min<int64_t>(items, 2 * sms / splits)};
  // Groups: the sizes are not known here.  Up to 32 rows a group on average the narrow tiles read the matrices faster
  // (tile : stream; 32 groups of 5760 x 2880: 64 rows 79.4 : 72.6, 640 rows 105 : 90, 1024 rows 109 : 100, 1536 rows 116 : 116,
  // 2048 rows 120 : 137; 64 groups of 2816 x 2048: 1280 rows 75 : 67, 4096 rows 85 : 94).
  if (G > 1 && mean <= 32) return stream;
  // One matrix, or larger groups with the most tiles that they can make: what each would take, by 0.5 a block of K and tile
  // against a fixed 5 and the larger of 0.13 a block in sequence and the traffic from L2 at 8 TB/s (tile : stream:
  // 128 x 2880 x 2880 16.1 : 9.8, 333 x 2048 x 1408 10.7 : 7.6, 600 x 1024 x 1024 9.2 : 6.4, 256 x 4096 x 1024 9.2 : 9.2,
  // 128 x 14336 x 4096 22.7 : 36.7; groups, rows of all: 2 of 512 x 4096, 100 rows 21.0 : 7.2, 4 of 1024 x 2048, 256 rows
  // 13.8 : 8.4, 8 of 1408 x 2048, 1024 rows 15.3 : 17.0).  Tiles wait for what they add, and shift rows at odd places.
  const double rest = (a.add ? 5.0 : 0.0) + (aligned(a.out, a.ld_out * dt_size(a.out_type), 16) ? 0.0 : 3.0);
  const double t_tile = 4.0 + (double)((tiles + sms - 1) / sms) * (1.5 + 0.5 * kb + rest);
  const double t_stream = 5.0 + std::max(0.13 * (double)((items * splits + 2 * sms - 1) / (2 * sms)) * cdiv(kb, splits),
                                         (double)items * kb * (SCALE_BLOCK * (ST_N + bt)) / 8e6);
  return t_tile <= t_stream ? tile : stream;
}

ts_moe_status done(cudaError_t e, const char* what) { return e == cudaSuccess ? TS_MOE_OK : cuda_bad(e, what); }

template <int MAX_THREADS>
cudaError_t launch_norm_rows(const ts_moe_rmsnorm_args& a, void* stream) {
  const int threads = cdiv(cdiv(a.hidden, SCALE_BLOCK) * 8, 32) * 32;
  const bool rw = a.resid_type == TS_DT_FP32, dw = a.delta && a.delta_type == TS_DT_FP32;
  auto k = rw ? (dw ? rmsnorm_rows_kernel<MAX_THREADS, true, true> : rmsnorm_rows_kernel<MAX_THREADS, true, false>)
              : (dw ? rmsnorm_rows_kernel<MAX_THREADS, false, true> : rmsnorm_rows_kernel<MAX_THREADS, false, false>);
  int per_sm = 1;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, 0);
  if (e != cudaSuccess) return e;
  return launch(k, dim3(std::min(a.rows, GPU_SMS * std::max(per_sm, 1))), threads, 0, stream, a);
}

cudaError_t launch_norm(const ts_moe_rmsnorm_args& a, bool vec, void* stream) {
  const int chunks = cdiv(a.hidden, 8);
  // Many rows (us, a CTA a row : CTAs that walk, bf16: 512 x 512 2.5 : 2.9, 512 x 5120 6.8 : 7.1, 1024 x 2048 5.1 : 5.6,
  // 1024 x 4096 12.5 : 9.7, 2048 x 2880 16.1 : 13.7, 2048 x 4096 21.9 : 16.4, 4096 x 8192 89 : 63; fp32: 1024 x 5120 15.5 : 17.0)
  if (vec && a.rows > 1024)
    return a.hidden <= 4096   ? launch_norm_rows<256>(a, stream)
           : a.hidden <= 8192 ? launch_norm_rows<512>(a, stream)
                              : launch_norm_rows<1024>(a, stream);
  const int it = chunks <= 1024 ? 1 : 2;
  const int threads = std::max(32, cdiv(cdiv(chunks, it), 32) * 32);
  auto k = it == 1 ? (vec ? rmsnorm_kernel<1, true> : rmsnorm_kernel<1, false>) : (vec ? rmsnorm_kernel<2, true> : rmsnorm_kernel<2, false>);
  return launch(k, dim3(a.rows), threads, 0, stream, a);
}

// The largest bits of a gate in memory whose sigmoid is not a far one: those of -64, or of -64 / alpha rounded towards 0.
// Above them are larger negative gates and negative NaN.  With a negative alpha any gate may be far.
uint32_t act_far_bits(const ts_moe_act_quant_args& a) {
  const float alpha = a.act == TS_ACT_SWIGLU ? 1.f : a.act_alpha;
  if (alpha < 0.f) return 0;
  const float t = std::min(-FAR / alpha, FLT_MAX);  // alpha = 0: no finite gate is far
  uint32_t bits;
  std::memcpy(&bits, &t, sizeof(bits));
  if (a.in_type == TS_DT_FP32) return bits | 0x80000000u;
  if (a.in_type == TS_DT_BF16) return bits >> 16 | 0x8000u;
  if (t >= 65504.f) return 0xFBFFu;          // fp16's largest
  if (t < 0x1p-14f) return 0x8000u;          // below its normal range: every negative gate
  return 0x8000u | ((bits >> 13) - (112u << 10));
}

template <bool CLAMPED>
auto act_instance(bool vec, bool wide) {
  return vec ? (wide ? act_quant_kernel<true, true, CLAMPED> : act_quant_kernel<true, false, CLAMPED>) : act_quant_kernel<false, false, CLAMPED>;
}

template <bool SIGMOID, bool WIDE>
void (*balance_instance(int experts))(const BalanceParams) {
  const int lanes = balance_lanes(experts);
  return lanes == 2     ? balance_kernel<2, 1, SIGMOID, WIDE>
         : lanes == 4   ? balance_kernel<4, 1, SIGMOID, WIDE>
         : lanes == 8   ? balance_kernel<8, 1, SIGMOID, WIDE>
         : lanes == 16  ? balance_kernel<16, 1, SIGMOID, WIDE>
         : experts <= 128 ? balance_kernel<32, 1, SIGMOID, WIDE>
                        : balance_kernel<32, 2, SIGMOID, WIDE>;
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
  if (!at_elements(a.resid, a.resid_type) || !at_elements(a.delta, a.delta_type) || !at_elements(a.gamma, a.gamma_type) ||
      !at_elements(a.resid_out, a.resid_type) || !at_elements(a.y, a.y_type) || !at_words(a.q_scale))
    return bad("rmsnorm: a pointer is not aligned to its elements");
  if (a.q && overlap(a.rows, cdiv(a.hidden, SCALE_BLOCK), a.qs_row, a.qs_group)) return bad("rmsnorm: elements of q_scale overlap");
  if (a.resid_out == a.resid && a.ld_resid_out != a.ld_resid && a.resid_out) return bad("rmsnorm: resid_out in place needs resid's stride");
  const bool vec = a.hidden % 8 == 0 && aligned_rows(a.resid, a.ld_resid, a.resid_type) &&
                   aligned_rows(a.delta, a.ld_delta, a.delta_type) && aligned_rows(a.gamma, 0, a.gamma_type) &&
                   aligned_rows(a.resid_out, a.ld_resid_out, a.resid_type) && aligned_rows(a.y, a.ld_y, a.y_type) &&
                   (!a.q || aligned(a.q, a.ld_q, 8));
  return done(launch_norm(a, vec, stream), "rmsnorm launch");
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
  if (!at_elements(a.gate, a.in_type) || !at_elements(a.up, a.in_type) || !at_words(a.q_scale))
    return bad("act_quant: a pointer is not aligned to its elements");
  if (overlap(a.rows, cdiv(a.inter, SCALE_BLOCK), a.qs_row, a.qs_group)) return bad("act_quant: elements of q_scale overlap");
  const bool vec = a.inter % 8 == 0 && aligned_rows(a.gate, a.ld_gate, a.in_type) && aligned_rows(a.up, a.ld_up, a.in_type) &&
                   aligned(a.q, a.ld_q, 8);
  const bool wide = a.in_type == TS_DT_FP32;
  const int quads = cdiv(a.inter, 4 * SCALE_BLOCK);
  const int64_t units = (int64_t)a.rows * quads;
  const int resident = vec && wide ? 2 : 4;  // CTAs per SM by the kernel's launch bounds
  const int grid = (int)std::min<int64_t>((units + ACT_THREADS / 32 - 1) / (ACT_THREADS / 32), GPU_SMS * resident);
  const int warps = grid * (ACT_THREADS / 32);
  auto k = a.act == TS_ACT_SWIGLU ? act_instance<false>(vec, wide) : act_instance<true>(vec, wide);
  return done(launch(k, dim3(grid), ACT_THREADS, 0, stream, a, quads, warps / quads, warps % quads, act_far_bits(a)), "act_quant launch");
}

static ts_moe_status fp8_matmul(const ts_moe_fp8_matmul_args* args, int held, unsigned held_us, void* stream) {
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
  if (!aligned(a.a, a.rows > 1 ? a.ld_a : 0, 16) || !aligned(a.b, a.n > 1 ? a.ld_b : 0, 16) || (a.num_groups > 1 && a.b_group % 16))
    return bad("fp8_matmul: the rows of a and b must start at 16-byte boundaries");
  if (!at_elements(a.out, a.out_type) || !at_elements(a.add, a.out_type) || !at_words(a.a_scale) || !at_words(a.b_scale) || !at_words(a.offsets))
    return bad("fp8_matmul: a pointer is not aligned to its elements");
  if (a.num_groups > 1 && a.b_group < (int64_t)(a.n - 1) * a.ld_b + a.k) return bad("fp8_matmul: b_group is smaller than a matrix");
  if (a.add == a.out && a.ld_add != a.ld_out) return bad("fp8_matmul: add in place needs out's stride");
  if (a.ld_a >= (int64_t)1 << 40 || a.ld_b >= (int64_t)1 << 40 || a.b_group >= (int64_t)1 << 40)
    return set_last_error(TS_MOE_EUNSUPPORTED, "fp8_matmul: a stride of 2^40 or more");

  const MatmulDevice* d = nullptr;
  const ts_moe_status st = matmul_setup(&d);
  if (st != TS_MOE_OK) return st;
  const MatmulPlan plan = matmul_plan(a, d->sms);
  MatmulParams p;
  p.a = a;
  p.kb = cdiv(a.k, SCALE_BLOCK);
  p.splits = plan.splits;
  p.held = held;
  p.held_us = held_us;
  // strides no row or matrix follows may be anything: give the map valid ones
  const int64_t row = (a.k + 15) / 16 * 16, ld_a = a.rows > 1 ? a.ld_a : row, ld_b = a.n > 1 ? a.ld_b : row;
  const int64_t group = a.num_groups > 1 ? a.b_group : (int64_t)a.n * ld_b;
  cudaError_t e;
  if (plan.kind == MatmulPlan::ROWS) {
    if (held >= 0) return bad("fp8_matmul: this call has no waits");
    p.out_map = 0;
    auto k = a.rows <= 8 ? fp8_row_kernel<1> : fp8_row_kernel<2>;
    e = launch(k, dim3(plan.grid), RW_THREADS, 0, stream, p);
    return done(e, "fp8_matmul launch");
  }
  const bool tile = plan.kind == MatmulPlan::TILE;
  CUtensorMap ma, mb, mo = {};
  // a map's stores end at 16-byte places, not at elements: rows of another length would write past their end
  const int es = dt_size(a.out_type);
  p.out_map = tile && aligned(a.out, a.ld_out * es, 16) && (int64_t)a.n * es % 16 == 0 && a.ld_out < (int64_t)1 << 37;
  if (!encode_rows(&ma, a.a, a.k, a.rows, ld_a, -1, 0, tile ? TL_M : plan.bt) ||
      !encode_rows(&mb, a.b, a.k, a.n, ld_b, a.num_groups, group, tile ? TL_N : ST_N) || (p.out_map && !encode_out(&mo, a)))
    return set_last_error(TS_MOE_ECUDA, "fp8_matmul: the driver refused a tensor map");
  if (tile)
    e = launch(fp8_tile_kernel, dim3(plan.grid), TL_THREADS, tile_smem(), stream, p, ma, mb, mo);
  else
    e = plan.bt == 16 ? launch_stream<16>(p, ma, mb, plan.grid, stream) : launch_stream<32>(p, ma, mb, plan.grid, stream);
  return done(e, "fp8_matmul launch");
}

ts_moe_status ts_moe_fp8_matmul(const ts_moe_fp8_matmul_args* args, void* stream) { return fp8_matmul(args, -1, 0, stream); }

void ts_moe_debug_fp8_matmul_plan(const ts_moe_fp8_matmul_args* args, int sms, int32_t plan[4]) {
  const MatmulPlan p = args->rows > 0 ? matmul_plan(*args, sms) : MatmulPlan{MatmulPlan::ROWS, 0, 1, 0};  // no rows: no launch
  plan[0] = p.kind;
  plan[1] = p.bt;
  plan[2] = p.splits;
  plan[3] = p.grid;
}

ts_moe_status ts_moe_debug_fp8_matmul_held(const ts_moe_fp8_matmul_args* args, int cta, uint32_t wait_us, void* stream) {
  if (cta < 0) return bad("fp8_matmul: cta must not be negative");
  if (wait_us > WAIT_LIMIT_US) return bad("fp8_matmul: wait_us is above the limit of the kernels' waits");
  return fp8_matmul(args, cta, wait_us, stream);
}

// Up to 16384 logits one CTA does everything: the counting launch and the joins take longer than it (us, one CTA : many, with
// the gradient: 512 x 32 6.8 : 7.9, 64 x 256 6.5 : 8.5, 1024 x 32 9.9 : 8.2, 256 x 256 13.4 : 9.7).
static int balance_ctas(int rows, int experts) {
  if ((int64_t)rows * experts <= 16384) return 1;
  return std::min(cdiv(rows, BAL_WARPS * (32 / balance_lanes(experts))), BAL_MAX_CTAS);
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
  if ((a.rows > 0 && (!at_elements(a.logits, a.dtype) || !at_elements(a.dlogits, a.dtype) || !at_words(a.idx))) || !at_words(a.dloss) ||
      !at_words(a.loss) || !at_words(a.prob) || !at_words(a.counts) || !at_words(a.offsets))
    return bad("balance: a pointer is not aligned to its elements");
  if (!a.workspace || (uintptr_t)a.workspace % 16) return bad("balance: workspace must be non-NULL and 16-byte aligned");
  if (a.workspace_bytes < ts_moe_balance_workspace(a.rows, a.experts)) return bad("balance: workspace is too small");

  BalanceParams p;
  p.a = a;
  p.head = (BalanceHead*)a.workspace;
  p.part = (float*)((char*)a.workspace + sizeof(BalanceHead));
  const int ctas = balance_ctas(a.rows, a.experts);
  p.count_ctas = ctas > 1 ? std::min(cdiv(a.rows * a.top_k, 4 * BAL_COUNT_THREADS), BAL_COUNT_CTAS) : 0;
  if (p.count_ctas) {
    const cudaError_t e = launch(balance_count_kernel, dim3(p.count_ctas), BAL_COUNT_THREADS, 0, stream, p);
    if (e != cudaSuccess) return cuda_bad(e, "balance count launch");
  }
  const bool sigmoid = a.score == TS_SCORE_SIGMOID_RENORM, wide = a.dtype == TS_DT_FP32;
  auto k = sigmoid ? (wide ? balance_instance<true, true>(a.experts) : balance_instance<true, false>(a.experts))
                   : (wide ? balance_instance<false, true>(a.experts) : balance_instance<false, false>(a.experts));
  // fewer warps meet at fewer barriers (us, 256 threads : 1024: 64 x 32 3.7 : 4.1, 16 x 256 4.1 : 4.9, 128 x 32 4.6 : 4.4,
  // 256 x 32 6.3 : 5.4, 64 x 256 7.5 : 6.5)
  const int threads = (int64_t)a.rows * a.experts <= 4096 ? BAL_ALONE : BAL_THREADS;
  return done(launch(k, dim3(ctas), threads, 0, stream, p), "balance launch");
}

}  // extern "C"
