// Product of E4M3 rows with E4M3 matrices whose scales cover 128 x 128 blocks,
// dense and grouped, on the tensor cores.
//
//   out[m][n] = sum_c sa[m][c] sb[n / 128][c] P_c[m][n],   P_c = A_c B_c^T over the 128 codes of block c
//
// A tcgen05.mma pass over one block c leaves P_c in tensor memory in float32;
// the scales differ from block to block, so each P_c is read back, scaled and
// added in registers while the next block's MMAs write another part of tensor
// memory.  Two kernels share this scheme:
//
//   fp8_tile_kernel    128 rows x 256 columns per CTA, persistent: the tensor pipe bounds it.
//   fp8_stream_kernel  128 columns x BT rows per CTA with the matrix as the MMA's first operand, K split
//                      over a cluster: few rows, where reading the matrix bounds it.
#pragma once
#include "umma.cuh"

namespace tsm {

constexpr int MAX_GROUPS = TS_MOE_MAX_EXPERTS;

struct MatmulParams {
  ts_moe_fp8_matmul_args a;
  int kb;      // scale blocks of K
  int splits;  // fp8_stream_kernel: CTAs of a cluster, which share K
};

// ----------------------------------------------------------------------------- groups
// Row tiles of all groups in order: group g has tiles [first[g], first[g + 1]) over rows [lo[g], lo[g + 1]).
struct GroupTable {
  int first[MAX_GROUPS + 1];
  int lo[MAX_GROUPS + 1];
};

// One warp fills the table: offsets clamped to [0, rows] and made non-decreasing.
TSM_DEV void fill_groups(const ts_moe_fp8_matmul_args& a, int tile_rows, GroupTable& t) {
  const int lane = threadIdx.x & 31, G = a.num_groups;
  if (!a.offsets) {
    if (lane == 0) {
      t.lo[0] = t.first[0] = 0;
      t.lo[1] = a.rows;
      t.first[1] = cdiv(a.rows, tile_rows);
    }
    __syncwarp();
    return;
  }
  int base_lo = 0, base_first = 0;
  for (int g0 = 0; g0 <= G; g0 += 32) {
    const int g = g0 + lane;
    int o = g <= G ? max(0, min(a.offsets[g], a.rows)) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, o, d);
      if (lane >= d) o = max(o, v);
    }
    o = max(o, base_lo);
    int prev = __shfl_up_sync(0xFFFFFFFFu, o, 1);
    if (lane == 0) prev = g0 == 0 ? o : base_lo;
    int n = cdiv(o - prev, tile_rows);  // tiles of group g - 1
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, n, d);
      if (lane >= d) n += v;
    }
    n += base_first;
    if (g <= G) {
      t.lo[g] = o;
      t.first[g] = n;
    }
    base_lo = __shfl_sync(0xFFFFFFFFu, o, 31);
    base_first = __shfl_sync(0xFFFFFFFFu, n, 31);
  }
  __syncwarp();
}

// The group whose tiles hold tile `t` (t < first[G]).
TSM_DEV int group_of(const GroupTable& tab, int G, int t) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// ----------------------------------------------------------------------------- outputs
TSM_DEV float load1(const void* p, int type, int64_t i) {
  return type == TS_DT_FP32   ? ((const float*)p)[i]
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

// ----------------------------------------------------------------------------- many rows
constexpr int TL_M = 128, TL_N = 256, TL_STAGES = 4, TL_ACC = 2;  // TL_ACC x TL_N = all 512 columns of tensor memory
constexpr int TL_BAND = 16;     // row tiles that run side by side over the columns: their rows of A stay in L2
constexpr int TL_THREADS = 320; // producer warp, MMA warp, 8 warps that scale and add

struct TileSmem {
  uint8_t a[TL_STAGES][TL_M * SCALE_BLOCK];
  uint8_t b[TL_STAGES][TL_N * SCALE_BLOCK];
  uint64_t full[TL_STAGES], empty[TL_STAGES], acc_full[TL_ACC], acc_empty[TL_ACC], drain;
  uint32_t tmem;
  int dead;
  GroupTable groups;
};

struct Tile {
  int g, m0, hi, n0;
};

TSM_DEV Tile locate_tile(const MatmulParams& p, const GroupTable& tab, int t) {
  const int nt = cdiv(p.a.n, TL_N);
  Tile r;
  int u;
  if (p.a.offsets) {
    // tiles of a group are contiguous: first[g] * nt ..
    r.g = group_of(tab, p.a.num_groups, t / nt);
    u = t - tab.first[r.g] * nt;
  } else {
    r.g = 0;
    u = t;
  }
  const int mt = tab.first[r.g + 1] - tab.first[r.g];
  const int band = u / (TL_BAND * nt), in_band = u - band * TL_BAND * nt;
  const int bm = min(TL_BAND, mt - band * TL_BAND);
  r.m0 = tab.lo[r.g] + (band * TL_BAND + in_band % bm) * TL_M;
  r.hi = tab.lo[r.g + 1];
  r.n0 = in_band / bm * TL_N;
  return r;
}

__global__ void __launch_bounds__(TL_THREADS, 1)
    fp8_tile_kernel(const MatmulParams p, const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb) {
  extern __shared__ uint8_t raw[];
  TileSmem& s = *reinterpret_cast<TileSmem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* dead = &s.dead;
  if (threadIdx.x == 0) {
    for (int i = 0; i < TL_STAGES; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < TL_ACC; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], 8);
    mbar_init(&s.drain, 1);
    s.dead = 0;
    fence_barrier_init();
    prefetch_map(&ma);
    prefetch_map(&mb);
  }
  if (warp == 1) tmem_alloc<512>(&s.tmem);
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 0) fill_groups(p.a, TL_M, s.groups);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int tiles = s.groups.first[p.a.num_groups] * cdiv(p.a.n, TL_N);

  if (warp == 0) {
    if (lane == 0) {
      unsigned it = 0;
      for (int t = blockIdx.x; t < tiles && !*dead; t += gridDim.x) {
        const Tile tl = locate_tile(p, s.groups, t);
        for (int c = 0; c < p.kb; ++c, ++it) {
          const int st = it % TL_STAGES;
          if (!wait_or_die(&s.empty[st], (it / TL_STAGES & 1) ^ 1, dead)) break;
          mbar_arrive_expect_tx(&s.full[st], (TL_M + TL_N) * SCALE_BLOCK);
          tma_load_2d(s.a[st], &ma, c * SCALE_BLOCK, tl.m0, &s.full[st]);
          tma_load_3d(s.b[st], &mb, c * SCALE_BLOCK, tl.n0, tl.g, &s.full[st]);
        }
      }
      // no copy may be in flight when the CTA ends
      if (*dead) {
        for (unsigned i = it > TL_STAGES ? it - TL_STAGES : 0; i < it; ++i) {
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(&s.full[i % TL_STAGES], i / TL_STAGES & 1) && globaltimer() - t0 < WAIT_LIMIT_NS) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = umma_idesc(TL_M, TL_N);
      unsigned it = 0;
      for (int t = blockIdx.x; t < tiles && !*dead; t += gridDim.x) {
        for (int c = 0; c < p.kb; ++c, ++it) {
          const int st = it % TL_STAGES, ac = it % TL_ACC;
          if (!wait_or_die(&s.acc_empty[ac], (it / TL_ACC & 1) ^ 1, dead)) break;
          if (!wait_or_die(&s.full[st], it / TL_STAGES & 1, dead)) break;
          tc_fence_after();
          const uint64_t da = umma_desc(smem_addr(s.a[st])), db = umma_desc(smem_addr(s.b[st]));
#pragma unroll
          for (int k = 0; k < SCALE_BLOCK / 32; ++k) umma_e4m3(tmem + ac * TL_N, da + 2 * k, db + 2 * k, idesc, k > 0);
          umma_commit(&s.empty[st]);
          umma_commit(&s.acc_full[ac]);
        }
      }
      // no MMA may be in flight when tensor memory is freed
      umma_commit(&s.drain);
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(&s.drain, 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
      }
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
    const int nblocks = cdiv(p.a.n, SCALE_BLOCK);
    unsigned it = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile tl = locate_tile(p, s.groups, t);
      const int row = tl.m0 + quarter * 32 + lane, col0 = tl.n0 + half * 128;
      const float* sa = p.a.a_scale + (int64_t)min(row, tl.hi - 1) * p.a.as_row;
      const float* sb = p.a.b_scale + tl.g * p.a.bs_group + (int64_t)min(col0 / SCALE_BLOCK, nblocks - 1) * p.a.bs_row;
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.f;
      float na = *sa, nb = *sb;
      for (int c = 0; c < p.kb; ++c, ++it) {
        const int ac = it % TL_ACC;
        const float sc = na * nb;
        if (c + 1 < p.kb) {
          na = sa[(int64_t)(c + 1) * p.a.as_block];
          nb = sb[(int64_t)(c + 1) * p.a.bs_block];
        }
        wait_or_die(&s.acc_full[ac], it / TL_ACC & 1, dead);  // a dead CTA runs on without waiting
        __syncwarp();
        tc_fence_after();
        float v[2][16];
        tmem_ld16(mine + ac * TL_N, v[0]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          tc_wait_ld(v[q & 1]);
          if (q < 7) tmem_ld16(mine + ac * TL_N + (q + 1) * 16, v[(q + 1) & 1]);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[q * 16 + j] += sc * v[q & 1][j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.acc_empty[ac]);
      }
      if (row < tl.hi) {
        const bool lost = *dead;
        const int type = p.a.out_type, n = min(128, p.a.n - col0);
        const bool vec = ((uintptr_t)p.a.out | (uintptr_t)(p.a.ld_out * dt_size(type))) % 16 == 0;
        const bool vadd = ((uintptr_t)p.a.add | (uintptr_t)(p.a.ld_add * dt_size(type))) % 16 == 0;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int w = min(8, n - q * 8);
          if (w > 0) {
            const int64_t col = col0 + q * 8;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = lost ? NAN : acc[q * 8 + j];
            if (p.a.add) {
              const int64_t off = (int64_t)row * p.a.ld_add + col;
              const Raw8 r = vadd && w == 8 ? load_raw8<true>(p.a.add, type, off, 8) : load_raw8<false>(p.a.add, type, off, w);
              float d[8];
              cvt8(r, type, d);
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] += d[j];
            }
            const int64_t off = (int64_t)row * p.a.ld_out + col;
            if (vec && w == 8)
              store_raw8<true>(p.a.out, type, off, 8, round8(v, type));
            else
              store_raw8<false>(p.a.out, type, off, w, round8(v, type));
          }
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) tmem_free<512>(tmem);
}

// ----------------------------------------------------------------------------- few rows
constexpr int ST_N = 128, ST_THREADS = 192;  // producer warp, MMA warp, 4 warps that scale and add
constexpr int ST_CHUNK = 8;                  // scale blocks whose row scales are staged at a time

template <int BT>
struct StreamShape {
  static constexpr int STAGES = BT == 16 ? 5 : BT == 32 ? 4 : BT == 64 ? 3 : 4;
  static constexpr int ACC = BT == 16 ? 8 : 4;  // parts of tensor memory
  static constexpr int COLS = ACC * BT;
  static constexpr int CTAS = BT == 128 ? 1 : 2;  // per SM
};

template <int BT>
struct StreamSmem {
  using S = StreamShape<BT>;
  uint8_t b[S::STAGES][ST_N * SCALE_BLOCK];
  uint8_t a[S::STAGES][BT * SCALE_BLOCK];
  float red[BT][ST_N];              // this CTA's share of K, for the cluster's CTAs to add
  float scale[2][ST_CHUNK][BT];     // sa * sb of the blocks at hand
  uint64_t full[S::STAGES], empty[S::STAGES], acc_full[S::ACC], acc_empty[S::ACC], red_full, red_free, drain;
  uint32_t tmem;
  int dead;
  GroupTable groups;
};

template <int BT>
__global__ void __launch_bounds__(ST_THREADS, StreamShape<BT>::CTAS)
    fp8_stream_kernel(const MatmulParams p, const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb) {
  using S = StreamShape<BT>;
  extern __shared__ uint8_t raw[];
  StreamSmem<BT>& s = *reinterpret_cast<StreamSmem<BT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* dead = &s.dead;
  const int splits = p.splits, rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::STAGES; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < S::ACC; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], 4);
    mbar_init(&s.red_full, 4 * splits);
    mbar_init(&s.red_free, 4 * splits);
    mbar_init(&s.drain, 1);
    s.dead = 0;
    fence_barrier_init();
    prefetch_map(&ma);
    prefetch_map(&mb);
  }
  if (warp == 1) tmem_alloc<S::COLS>(&s.tmem);
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 0) fill_groups(p.a, BT, s.groups);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the peers' barriers are ready
  const uint32_t tmem = s.tmem;
  const int nt = cdiv(p.a.n, ST_N);
  const int items = s.groups.first[p.a.num_groups] * nt;
  const int c0 = (int)((int64_t)p.kb * rank / splits), c1 = (int)((int64_t)p.kb * (rank + 1) / splits);
  const int first = blockIdx.x / splits, step = gridDim.x / splits;

  if (warp == 0) {
    if (lane == 0) {
      unsigned it = 0;
      for (int t = first; t < items && !*dead; t += step) {
        const int tt = t / nt, g = group_of(s.groups, p.a.num_groups, tt);
        const int m0 = s.groups.lo[g] + (tt - s.groups.first[g]) * BT, n0 = (t - tt * nt) * ST_N;
        for (int c = c0; c < c1; ++c, ++it) {
          const int st = it % S::STAGES;
          if (!wait_or_die(&s.empty[st], (it / S::STAGES & 1) ^ 1, dead)) break;
          mbar_arrive_expect_tx(&s.full[st], (ST_N + BT) * SCALE_BLOCK);
          tma_load_3d(s.b[st], &mb, c * SCALE_BLOCK, n0, g, &s.full[st]);
          tma_load_2d(s.a[st], &ma, c * SCALE_BLOCK, m0, &s.full[st]);
        }
      }
      if (*dead) {
        for (unsigned i = it > S::STAGES ? it - S::STAGES : 0; i < it; ++i) {
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(&s.full[i % S::STAGES], i / S::STAGES & 1) && globaltimer() - t0 < WAIT_LIMIT_NS) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = umma_idesc(ST_N, BT);
      unsigned it = 0;
      for (int t = first; t < items && !*dead; t += step) {
        for (int c = c0; c < c1; ++c, ++it) {
          const int st = it % S::STAGES, ac = it % S::ACC;
          if (!wait_or_die(&s.acc_empty[ac], (it / S::ACC & 1) ^ 1, dead)) break;
          if (!wait_or_die(&s.full[st], it / S::STAGES & 1, dead)) break;
          tc_fence_after();
          const uint64_t db = umma_desc(smem_addr(s.b[st])), da = umma_desc(smem_addr(s.a[st]));
#pragma unroll
          for (int k = 0; k < SCALE_BLOCK / 32; ++k) umma_e4m3(tmem + ac * BT, db + 2 * k, da + 2 * k, idesc, k > 0);
          umma_commit(&s.empty[st]);
          umma_commit(&s.acc_full[ac]);
        }
      }
      umma_commit(&s.drain);
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(&s.drain, 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
      }
    }
  } else {
    // thread r of these 128: column n0 + r of the tile, all BT rows
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int PER = ST_CHUNK * BT / 128;  // scales a thread stages per chunk
    const int type = p.a.out_type;
    unsigned it = 0, round = 0;
    for (int t = first; t < items; t += step, ++round) {
      const int tt = t / nt, g = group_of(s.groups, p.a.num_groups, tt);
      const int m0 = s.groups.lo[g] + (tt - s.groups.first[g]) * BT, rows = min(BT, s.groups.lo[g + 1] - m0);
      const int n0 = (t - tt * nt) * ST_N;
      const float* sb = p.a.b_scale + g * p.a.bs_group + (int64_t)(n0 / SCALE_BLOCK) * p.a.bs_row;
      float acc[BT], next[PER];
#pragma unroll
      for (int j = 0; j < BT; ++j) acc[j] = 0.f;
      auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = i * 128 + r, cc = c + e / BT, m = e % BT;
          next[i] = cc < c1 && m < rows
                        ? p.a.a_scale[(int64_t)(m0 + m) * p.a.as_row + (int64_t)cc * p.a.as_block] * sb[(int64_t)cc * p.a.bs_block]
                        : 0.f;
        }
      };
      fetch(c0);
      int buf = 0;
      for (int c = c0; c < c1; c += ST_CHUNK, buf ^= 1) {
#pragma unroll
        for (int i = 0; i < PER; ++i) (&s.scale[buf][0][0])[i * 128 + r] = next[i];
        bar_sync(1, 128);  // also: everybody is done with the buffer of two chunks ago
        if (c + ST_CHUNK < c1) fetch(c + ST_CHUNK);
        const int ce = min(c1 - c, ST_CHUNK);
        for (int i = 0; i < ce; ++i, ++it) {
          const int ac = it % S::ACC;
          wait_or_die(&s.acc_full[ac], it / S::ACC & 1, dead);  // a dead CTA runs on without waiting: equal barrier counts
          __syncwarp();
          tc_fence_after();
          float v[2][16];
          tmem_ld16(mine + ac * BT, v[0]);
#pragma unroll
          for (int q = 0; q < BT / 16; ++q) {
            tc_wait_ld(v[q & 1]);
            if (q + 1 < BT / 16) tmem_ld16(mine + ac * BT + (q + 1) * 16, v[(q + 1) & 1]);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 f = *(const float4*)&s.scale[buf][i][q * 16 + j];
              acc[q * 16 + j] += f.x * v[q & 1][j];
              acc[q * 16 + j + 1] += f.y * v[q & 1][j + 1];
              acc[q * 16 + j + 2] += f.z * v[q & 1][j + 2];
              acc[q * 16 + j + 3] += f.w * v[q & 1][j + 3];
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.acc_empty[ac]);
        }
      }
      bar_sync(1, 128);  // the scale buffers are free for the next item
      const int64_t n = n0 + r;
      if (splits == 1) {
        const bool lost = *dead;
#pragma unroll
        for (int j = 0; j < BT; ++j) {
          if (j < rows && n < p.a.n) {
            const int64_t m = m0 + j;
            float v = lost ? NAN : acc[j];
            if (p.a.add) v += load1(p.a.add, type, m * p.a.ld_add + n);
            store1(p.a.out, type, m * p.a.ld_out + n, v);
          }
        }
        continue;
      }
      // every CTA of the cluster adds a share of the rows, over the CTAs in order
      if (round > 0) wait_cluster_or_die(&s.red_free, (round - 1) & 1, dead);
#pragma unroll
      for (int j = 0; j < BT; ++j) s.red[j][r] = acc[j];
      __syncwarp();
      if (lane < splits) peer_arrive(peer_addr(smem_addr(&s.red_full), lane));
      wait_cluster_or_die(&s.red_full, round & 1, dead);
      __syncwarp();
      const bool lost = *dead;
      const int j0 = rows * rank / splits, j1 = rows * (rank + 1) / splits;
      for (int j = j0; j < j1; ++j) {
        float v = 0.f;
        for (int q = 0; q < splits; ++q) v += peer_load(peer_addr(smem_addr(&s.red[j][r]), q));
        if (n < p.a.n) {
          const int64_t m = m0 + j;
          if (lost) v = NAN;
          if (p.a.add) v += load1(p.a.add, type, m * p.a.ld_add + n);
          store1(p.a.out, type, m * p.a.ld_out + n, v);
        }
      }
      __syncwarp();
      if (lane < splits) peer_arrive(peer_addr(smem_addr(&s.red_free), lane));
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) tmem_free<S::COLS>(tmem);
  cluster_sync();  // no peer reads this CTA's memory any more
}

}  // namespace tsm
