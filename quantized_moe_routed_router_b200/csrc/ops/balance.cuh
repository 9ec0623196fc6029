// Per-expert counts, the router's balance loss and its gradient.
//
//   f[e] = counts[e] E / (K T),  prob[e] = mean_t p[t][e],  loss = coef sum_e f[e] prob[e]
//   dlogits[t][e] = dloss coef / T  p[t][e] s[t][e] (f[e] - sum_j f[j] p[t][j])
//
// with s = 1 for p = softmax(l), and s = 1 - sigmoid(l) for p = sigmoid(l) / sum
// sigmoid(l).  For a row whose sigmoids sum to little they are taken times e^-m,
// m = min(max l, 0), which the quotient cancels: no share is lost to underflow.
//
// The gradient needs all counts, and the counts need idx only: the counts come
// first (idx is a small share of the bytes), then one pass over the logits forms
// the probabilities' sums and the gradient together, so the logits are read once.
// The last CTA to finish adds the CTAs' sums in CTA order: equal bits on every
// call.  Few rows run in one CTA and one launch.
#pragma once
#include "elem.cuh"

namespace tsm {

constexpr int BAL_ALONE = 256;  // threads of the only CTA of a small call
constexpr int BAL_THREADS = 1024;  // otherwise: 32 warps a SM to hide the loads
constexpr int BAL_WARPS = BAL_THREADS / 32;
constexpr int BAL_MAX_E = TS_MOE_MAX_EXPERTS;
constexpr int BAL_MAX_CTAS = GPU_SMS;  // part of the workspace's size, so fixed
constexpr int BAL_COUNT_CTAS = 128, BAL_COUNT_THREADS = 512, BAL_COUNT_LD = BAL_MAX_E + 4;
static_assert(BAL_COUNT_CTAS <= BAL_ALONE, "one thread per counting CTA");
static_assert(BAL_MAX_E <= BAL_ALONE, "one thread per expert in the finish");

// The workspace: this, and the CTAs' probability sums [CTAs][E] behind it.
struct BalanceHead {
  unsigned ticket;
  int pad[63];
  int counts[BAL_COUNT_CTAS][BAL_COUNT_LD];  // of each counting CTA; its tokens at BAL_MAX_E
};
static_assert(sizeof(BalanceHead) % 256 == 0, "the sums behind it stay aligned");

struct BalanceParams {
  ts_moe_balance_args a;
  BalanceHead* head;
  float* part;
  int count_ctas;  // CTAs of balance_count_kernel, which ran before; 0: the only CTA counts by itself
};

__host__ __device__ inline int balance_lanes(int E) {  // lanes that share a row, four or eight logits each
  int l = 2;
  while (l < 32 && l * 4 < E) l *= 2;
  return l;
}

// Adds rows [r0, r1) to the CTA's histogram; hist[BAL_MAX_E] counts rows.
TSM_DEV void balance_count(const ts_moe_balance_args& a, int r0, int r1, int* hist) {
  const int K = a.top_k, n = (r1 - r0) * K;
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * blockDim.x) {
    int e[4];
    bool first[4], on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // four entries' loads side by side
      const int i = i0 + u * (int)blockDim.x, t = i / K, k = i - t * K;
      const int64_t row = r0 + t;
      const bool in = i < n;
      e[u] = in ? a.idx[row * a.ld_idx + k] : -1;
      on[u] = in && (!a.mask || a.mask[row]);
      first[u] = k == 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (!on[u]) continue;
      if (first[u]) atomicAdd(&hist[BAL_MAX_E], 1);
      if (e[u] >= 0 && e[u] < a.experts) atomicAdd(&hist[e[u]], 1);
    }
  }
}

__global__ void __launch_bounds__(BAL_COUNT_THREADS) balance_count_kernel(const BalanceParams p) {
  __shared__ int hist[BAL_MAX_E + 1];
  grid_dep_wait();
  grid_dep_launch();
  for (int e = threadIdx.x; e <= BAL_MAX_E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int per = cdiv(p.a.rows, gridDim.x), r0 = min(p.a.rows, (int)blockIdx.x * per);
  balance_count(p.a, r0, min(p.a.rows, r0 + per), hist);
  __syncthreads();
  for (int e = threadIdx.x; e <= BAL_MAX_E; e += blockDim.x) p.head->counts[blockIdx.x][e] = hist[e];
  if (blockIdx.x == 0 && threadIdx.x == 0) p.head->ticket = 0;
}

// Quads of one row as they lie in memory: four words of 32 bits, or two of two 16-bit values.
template <int NV, bool WIDE>
struct RawRow {
  uint32_t q[NV][WIDE ? 4 : 2];
};

// LPR lanes share a row, NV quads of logits each: quad v of lane l holds experts
// (v LPR + l) 4 .. + 3.
template <int LPR, int NV, bool WIDE>
TSM_DEV RawRow<NV, WIDE> balance_load(const ts_moe_balance_args& a, int64_t row, int lane, bool live, bool vec) {
  RawRow<NV, WIDE> r;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e0 = (v * LPR + lane) * 4;
#pragma unroll
    for (int j = 0; j < (WIDE ? 4 : 2); ++j) r.q[v][j] = 0;
    if (!live || e0 >= a.experts) continue;
    const int64_t off = row * a.ld_logits + e0;
    if constexpr (WIDE) {
      const uint32_t* p = (const uint32_t*)a.logits + off;
      if (vec) {
        const uint4 w = __ldcs((const uint4*)p);
        r.q[v][0] = w.x, r.q[v][1] = w.y, r.q[v][2] = w.z, r.q[v][3] = w.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e0 + j < a.experts) r.q[v][j] = p[j];
      }
    } else {
      const uint16_t* p = (const uint16_t*)a.logits + off;
      if (vec) {
        const uint2 w = __ldcs((const uint2*)p);
        r.q[v][0] = w.x, r.q[v][1] = w.y;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e0 + j < a.experts) r.q[v][j / 2] |= (uint32_t)p[j] << (16 * (j % 2));
      }
    }
  }
  return r;
}

template <bool WIDE>
TSM_DEV void balance_quad(const uint32_t (&q)[WIDE ? 4 : 2], int type, float (&v)[4]) {
  if constexpr (WIDE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(q[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (type == TS_DT_BF16) {
        v[2 * j] = __uint_as_float(q[j] << 16);
        v[2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  }
}

// SIGMOID: the score.  WIDE: logits and their gradient in 32 bits.
// 65536 x 256 sigmoid with the gradient: 45 us with the counting launch (134 MB, floor 20.8); issue slots bound the pass
// over the logits (71 % busy, 38 instructions a logit counted); that instance spills 32 bytes at 64 registers.
template <int LPR, int NV, bool SIGMOID, bool WIDE>
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
  for (int e = tid; e <= BAL_MAX_E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  if (p.count_ctas == 0) {
    balance_count(a, r0, r1, hist);
  } else {
    // whole numbers: the order of the additions does not change the counts
    const int segs = (int)blockDim.x / BAL_MAX_E, e = tid % BAL_MAX_E;
    int sum = 0;
#pragma unroll 16
    for (int b = tid / BAL_MAX_E; b < p.count_ctas; b += segs) sum += p.head->counts[b][e];
    if (sum) atomicAdd(&hist[e], sum);
    if (tid < p.count_ctas) atomicAdd(&hist[BAL_MAX_E], p.head->counts[tid][BAL_MAX_E]);
  }
  __syncthreads();

  float f[N], psum[N];
  const int T = hist[BAL_MAX_E];
  const float gscale = a.dlogits && T > 0 ? a.coef * (a.dloss ? *a.dloss : 1.f) / (float)T : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (i / 4 * LPR + lane) * 4 + i % 4;
    f[i] = e < E && T > 0 ? (float)hist[e] * ((float)E / ((float)a.top_k * (float)T)) : 0.f;
    psum[i] = 0.f;
  }
  constexpr int ES = WIDE ? 4 : 2;
  const bool vec = ((uintptr_t)a.logits | (uintptr_t)(a.ld_logits * ES)) % (4 * ES) == 0 && E % 4 == 0;
  const bool vec_out = ((uintptr_t)a.dlogits | (uintptr_t)(a.ld_dlogits * ES)) % (4 * ES) == 0 && E % 4 == 0;
  const bool full = E == N * LPR;  // every place holds an expert
  const int step = warps * (32 / LPR);
  // -inf stands at the places past E: their p is 0
  auto logits_of = [&](const RawRow<NV, WIDE>& r, float (&l)[N]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[4];
      balance_quad<WIDE>(r.q[v], a.dtype, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) l[4 * v + j] = w[j];
    }
    if (!full) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i / 4 * LPR + lane) * 4 + i % 4 >= E) l[i] = -INFINITY;
    }
  };
  auto row_max = [&](const float (&l)[N]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int d = LPR / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    return m;
  };
  // every lane of a warp takes every step: the shuffles name all of them
  int64_t row = r0 + warp * (32 / LPR) + sub;
  bool live = row < r1 && (!a.mask || a.mask[row]);
  RawRow<NV, WIDE> raw = balance_load<LPR, NV, WIDE>(a, row, lane, live, vec);
  for (int rb = r0 + warp * (32 / LPR); rb < r1; rb += step) {
    const RawRow<NV, WIDE> now = raw;
    const int64_t at = row;
    const bool in = at < r1, on = live;
    row += step;  // the next row's loads run while this one is worked on
    live = row < r1 && (!a.mask || a.mask[row]);
    raw = balance_load<LPR, NV, WIDE>(a, row, lane, live, vec);
    float t[N], slope[N], s = 0.f, fp = 0.f;
    logits_of(now, t);
    auto reduce = [&]() {
      s = fp = 0.f;
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
    };
    if (SIGMOID) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // u = e^-l, at most 2^127, whose 1 / (1 + u) is 0: sigmoid(l) = 1 / (1 + u), 1 - sigmoid(l) = u / (1 + u)
        const float u = ex2(min_nan(-LOG2E * t[i], 127.f));
        t[i] = rcp(1.f + u);
        slope[i] = u * t[i];
      }
      reduce();
      const bool small = s < 0.25f;  // the same in all lanes of the row
      if (__any_sync(0xFFFFFFFFu, small)) {
        // a row of very negative logits, whose sigmoids would lose their smallest: all of them times e^-m, m = min(max l, 0).
        // The warp's other rows keep what they have: a row's bits do not depend on the rows beside it.
        float l[N];
        logits_of(now, l);
        const float top = row_max(l), m = top == -INFINITY ? 0.f : fminf(top, 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float u = ex2(min_nan(-LOG2E * l[i], 127.f));
          const float far = l[i] < -60.f ? 1.f : u * rcp(1.f + u);  // from e^87 on the reciprocal is below the normal range
          if (small) slope[i] = far;
          if (small && m < 0.f) t[i] = ex2(LOG2E * (l[i] - m)) * far;
        }
        reduce();
      }
    } else {
      float m = row_max(t);
      if (m == -INFINITY) m = 0.f;  // nothing left in the row: p = 0
#pragma unroll
      for (int i = 0; i < N; ++i) {
        t[i] = ex2(LOG2E * (t[i] - m));
        slope[i] = 1.f;
      }
      reduce();
    }
    const float inv = !on || s == 0.f ? 0.f : rcp(s);  // s is 0 or in the normal range: at least 0.25 or one term near 1
    fp *= inv;
    const float c = on ? gscale * inv : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) psum[i] += inv * t[i];
    if (a.dlogits && in) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e0 = (v * LPR + lane) * 4;
        float g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * v + j;
          g[j] = (SIGMOID ? c * t[i] * slope[i] : c * t[i]) * (f[i] - fp);  // a row left out: zeros were loaded, c is 0
        }
        if (e0 < E) {
          const int64_t off = at * a.ld_dlogits + e0;
          if constexpr (WIDE) {
            float* q = (float*)a.dlogits + off;
            if (vec_out) {
              __stcs((float4*)q, make_float4(g[0], g[1], g[2], g[3]));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (e0 + j < E) q[j] = g[j];
            }
          } else {
            uint16_t* q = (uint16_t*)a.dlogits + off;
            const uint32_t lo = pack2(g[0], g[1], a.dtype), hi = pack2(g[2], g[3], a.dtype);
            if (vec_out) {
              __stcs((uint2*)q, make_uint2(lo, hi));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (e0 + j < E) q[j] = (uint16_t)((j < 2 ? lo : hi) >> (16 * (j % 2)));
            }
          }
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
#pragma unroll 16
      for (int b = seg; b < (int)gridDim.x; b += segs) part += __ldcg(&p.part[(int64_t)b * E + e]);
    }
    sums[seg][e] = part;
    __syncthreads();
    P = 0.f;
    if (tid < E)
      for (int w = 0; w < segs; ++w) P += sums[w][tid];
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
