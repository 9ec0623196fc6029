// Per-expert counts, the router's balance loss and its gradient.
//
//   f[e] = counts[e] E / (K T),  prob[e] = mean_t p[t][e],  loss = coef sum_e f[e] prob[e]
//   dlogits[t][e] = dloss coef / T  p[t][e] s[t][e] (f[e] - sum_j f[j] p[t][j])
//
// with s = 1 for p = softmax(l), and s = 1 - sigmoid(l) for p = sigmoid(l) / sum
// sigmoid(l).  There every sigmoid of a row is taken times e^-m, m = min(max l, 0),
// which the quotient cancels: no sum underflows for a row of very negative logits.
//
// The gradient needs all counts, and the counts need idx only: the counts come
// first (idx is a small share of the bytes), then one pass over the logits forms
// the probabilities' sums and the gradient together, so the logits are read once.
// The last CTA to finish adds the CTAs' sums in CTA order: equal bits on every
// call.  Few rows run in one CTA and one launch.
#pragma once
#include "elem.cuh"

namespace tsm {

constexpr int BAL_ALONE = 256, BAL_THREADS = 1024;  // threads of the only CTA, and of many: 32 warps a SM to hide the loads
constexpr int BAL_WARPS = BAL_THREADS / 32;
constexpr int BAL_MAX_E = TS_MOE_MAX_EXPERTS;
constexpr int BAL_MAX_CTAS = 148;  // one per SM: part of the workspace's size, so fixed
static_assert(BAL_MAX_E <= BAL_ALONE, "one thread per expert in the finish");

// Head of the workspace; the CTAs' probability sums [CTAs][E] follow it.
struct BalanceHead {
  int counts[BAL_MAX_E];
  int tokens;
  unsigned ticket;
  int pad[62];
};
static_assert(sizeof(BalanceHead) % 256 == 0, "the sums behind it stay aligned");

struct BalanceParams {
  ts_moe_balance_args a;
  BalanceHead* head;
  float* part;
  int counted;  // 1: the head already holds the counts (balance_count_kernel ran)
};

__host__ __device__ inline int balance_lanes(int E) {  // lanes that share a row, four or eight logits each
  int l = 2;
  while (l < 32 && l * 4 < E) l *= 2;
  return l;
}

// Adds rows [r0, r1) to the CTA's histogram; hist[BAL_MAX_E] counts rows.
TSM_DEV void balance_count(const ts_moe_balance_args& a, int r0, int r1, int* hist) {
  const int K = a.top_k;
  for (int i = threadIdx.x; i < (r1 - r0) * K; i += blockDim.x) {
    const int t = i / K, k = i - t * K;
    const int64_t row = r0 + t;
    if (a.mask && !a.mask[row]) continue;
    if (k == 0) atomicAdd(&hist[BAL_MAX_E], 1);
    const int e = a.idx[row * a.ld_idx + k];
    if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
  }
}

// Integer adds: their order does not change the counts.
TSM_DEV void balance_publish_counts(const BalanceParams& p, const int* hist) {
  for (int e = threadIdx.x; e <= BAL_MAX_E; e += blockDim.x)
    if (hist[e]) atomicAdd(e < BAL_MAX_E ? &p.head->counts[e] : &p.head->tokens, hist[e]);
}

__global__ void __launch_bounds__(BAL_THREADS) balance_count_kernel(const BalanceParams p) {
  __shared__ int hist[BAL_MAX_E + 1];
  grid_dep_wait();
  grid_dep_launch();
  for (int e = threadIdx.x; e <= BAL_MAX_E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int per = cdiv(p.a.rows, gridDim.x), r0 = min(p.a.rows, (int)blockIdx.x * per);
  balance_count(p.a, r0, min(p.a.rows, r0 + per), hist);
  __syncthreads();
  balance_publish_counts(p, hist);
}

// Quads of one row as they lie in memory.
template <int NV>
struct RawRow {
  uint4 q[NV];
};

// LPR lanes share a row, NV quads of logits each: quad v of lane l holds experts
// (v LPR + l) 4 .. + 3.
template <int LPR, int NV>
TSM_DEV RawRow<NV> balance_load(const ts_moe_balance_args& a, int64_t row, int lane, bool live, bool vec) {
  RawRow<NV> r;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e0 = (v * LPR + lane) * 4;
    r.q[v] = make_uint4(0, 0, 0, 0);
    if (!live || e0 >= a.experts) continue;
    const int64_t off = row * a.ld_logits + e0;
    if (!vec)
      r.q[v] = load_raw8<false>(a.logits, a.dtype, off, min(4, a.experts - e0)).a;
    else if (a.dtype == TS_DT_FP32)
      r.q[v] = *(const uint4*)((const float*)a.logits + off);
    else {
      const uint2 w = *(const uint2*)((const uint16_t*)a.logits + off);
      r.q[v].x = w.x, r.q[v].y = w.y;
    }
  }
  return r;
}

template <int LPR, int NV>
__global__ void __launch_bounds__(BAL_THREADS) balance_kernel(const BalanceParams p) {
  constexpr int N = 4 * NV;
  __shared__ int hist[BAL_MAX_E + 1];
  __shared__ float sums[BAL_WARPS][BAL_MAX_E];
  __shared__ float red[BAL_MAX_E / 32];
  __shared__ int last;
  const ts_moe_balance_args& a = p.a;
  const int E = a.experts, tid = threadIdx.x, warp = tid >> 5, lane = tid & (LPR - 1), sub = (tid & 31) / LPR;
  const int warps = blockDim.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const bool alone = gridDim.x == 1;
  const int per = cdiv(a.rows, (int)gridDim.x);
  const int r0 = min(a.rows, (int)blockIdx.x * per), r1 = min(a.rows, r0 + per);
  if (p.counted) {
    for (int e = tid; e <= BAL_MAX_E; e += blockDim.x) hist[e] = e < BAL_MAX_E ? p.head->counts[e] : p.head->tokens;
    __syncthreads();
  } else {
    for (int e = tid; e <= BAL_MAX_E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    balance_count(a, r0, r1, hist);
    __syncthreads();
    if (!alone) balance_publish_counts(p, hist);
  }

  // the gradient's constants (all counts are known whenever dlogits is wanted)
  float f[N], psum[N];
  const int T = hist[BAL_MAX_E];
  const float gscale = a.dlogits && T > 0 ? a.coef * (a.dloss ? *a.dloss : 1.f) / (float)T : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (i / 4 * LPR + lane) * 4 + i % 4;
    f[i] = e < E && T > 0 ? (float)hist[e] * ((float)E / ((float)a.top_k * (float)T)) : 0.f;
    psum[i] = 0.f;
  }
  const int align = a.dtype == TS_DT_FP32 ? 16 : 8, es = dt_size(a.dtype);
  const bool vec = ((uintptr_t)a.logits | (uintptr_t)(a.ld_logits * es)) % align == 0 && E % 4 == 0;
  const bool vec_out = ((uintptr_t)a.dlogits | (uintptr_t)(a.ld_dlogits * es)) % align == 0 && E % 4 == 0;
  const int step = warps * (32 / LPR);
  // every lane of a warp takes every step: the shuffles name all of them
  int64_t row = r0 + warp * (32 / LPR) + sub;
  bool live = row < r1 && (!a.mask || a.mask[row]);
  RawRow<NV> raw = balance_load<LPR, NV>(a, row, lane, live, vec);
  for (int rb = r0 + warp * (32 / LPR); rb < r1; rb += step) {
    const RawRow<NV> now = raw;
    const int64_t at = row;
    const bool in = at < r1, on = live;
    row += step;  // the next row's loads run while this one is worked on
    live = row < r1 && (!a.mask || a.mask[row]);
    raw = balance_load<LPR, NV>(a, row, lane, live, vec);
    float t[N], m = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Raw8 r;
      r.a = now.q[v];
      r.b = make_uint4(0, 0, 0, 0);
      float w[8];
      cvt8(r, a.dtype, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = (v * LPR + lane) * 4 + j;
        t[4 * v + j] = on && e < E ? w[j] : -INFINITY;
        m = fmaxf(m, t[4 * v + j]);
      }
    }
#pragma unroll
    for (int d = LPR / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (m == -INFINITY) m = 0.f;  // nothing left in the row: p = 0
    float slope[N], s = 0.f, fp = 0.f;
    if (a.score == TS_SCORE_SIGMOID_RENORM) {
      const float low = fminf(m, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // u = e^-|l|: sigmoid(l) = (l >= 0 ? 1 : u) / (1 + u), 1 - sigmoid(l) = (l >= 0 ? u : 1) / (1 + u)
        const float l = t[i], u = ex2(-LOG2E * fabsf(l)), d = rcp(1.f + u);
        const float e = low < 0.f ? ex2(LOG2E * (l - low)) : u;  // e^(l - low), for l < 0
        slope[i] = l >= 0.f ? u * d : d;
        t[i] = l >= 0.f ? d : e * d;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        t[i] = ex2(LOG2E * (t[i] - m));
        slope[i] = 1.f;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s += t[i];
      fp += f[i] * t[i];
    }
#pragma unroll
    for (int d = LPR / 2; d >= 1; d >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      fp += __shfl_xor_sync(0xFFFFFFFFu, fp, d);
    }
    const float inv = s == 0.f ? 0.f : 1.f / s;  // a NaN stays
    fp *= inv;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      t[i] *= inv;
      if (on) psum[i] += t[i];
    }
    if (a.dlogits && in) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e0 = (v * LPR + lane) * 4;
        float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (on) g[j] = gscale * t[4 * v + j] * (f[4 * v + j] - fp) * slope[4 * v + j];
        if (e0 < E) {
          const int64_t off = at * a.ld_dlogits + e0;
          const Raw8 r = round8(g, a.dtype);
          if (!vec_out)
            store_raw8<false>(a.dlogits, a.dtype, off, min(4, E - e0), r);
          else if (a.dtype == TS_DT_FP32)
            *(uint4*)((float*)a.dlogits + off) = r.a;
          else
            *(uint2*)((uint16_t*)a.dlogits + off) = make_uint2(r.a.x, r.a.y);
        }
      }
    }
  }

  // the CTA's sum of probabilities: lanes of a warp, then warps in order
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int d = LPR; d < 32; d <<= 1) psum[i] += __shfl_xor_sync(0xFFFFFFFFu, psum[i], d);
    const int e = (i / 4 * LPR + lane) * 4 + i % 4;
    if (sub == 0 && e < E) sums[warp][e] = psum[i];
  }
  __syncthreads();
  float P = 0.f;
  if (tid < E)
    for (int w = 0; w < warps; ++w) P += sums[w][tid];
  if (!alone) {
    if (tid < E) p.part[(int64_t)blockIdx.x * E + tid] = P;
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(&p.head->ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    // the CTAs' sums: four threads an expert where there are four, CTAs a stride apart, many loads in flight
    const int segs = (int)blockDim.x / BAL_MAX_E, seg = tid / BAL_MAX_E, e = tid % BAL_MAX_E;
    float part = 0.f;
    if (e < E) {
#pragma unroll 8
      for (int b = seg; b < (int)gridDim.x; b += segs) part += __ldcg(&p.part[(int64_t)b * E + e]);
    }
    sums[seg][e] = part;
    __syncthreads();
    P = 0.f;
    if (tid < E)
      for (int w = 0; w < segs; ++w) P += sums[w][tid];
    for (int e = tid; e <= BAL_MAX_E; e += blockDim.x)
      hist[e] = (int)__ldcg((const unsigned*)(e < BAL_MAX_E ? &p.head->counts[e] : &p.head->tokens));
    __syncthreads();
  }
  // finish: prob, loss, counts and their running sum, one thread per expert
  const int tokens = hist[BAL_MAX_E];
  const int count = tid < E ? hist[tid] : 0;
  float term = 0.f;
  if (tid < E) {
    const float prob = tokens > 0 ? P / (float)tokens : 0.f;
    const float load = tokens > 0 ? (float)count * ((float)E / ((float)a.top_k * (float)tokens)) : 0.f;
    term = load * prob;
    if (a.prob) a.prob[tid] = prob;
    a.counts[tid] = count;
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, d);
  if ((tid & 31) == 0 && tid < BAL_MAX_E) red[warp] = term;
  int run = count;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, run, d);
    if ((tid & 31) >= d) run += o;
  }
  __syncthreads();
  if ((tid & 31) == 31 && tid < BAL_MAX_E) hist[warp] = run;  // the counts are in registers by now
  __syncthreads();
  if (a.offsets && tid < BAL_MAX_E) {
    int base = 0;
    for (int w = 0; w < warp; ++w) base += hist[w];
    if (tid < E) a.offsets[tid + 1] = base + run;
    if (tid == 0) a.offsets[0] = 0;
  }
  if (tid == 0) {
    float loss = 0.f;
    for (int w = 0; w < BAL_MAX_E / 32; ++w) loss += red[w];
    *a.loss = a.coef * loss;
  }
}

}  // namespace tsm
