// Product of E4M3 rows with E4M3 matrices whose scales cover 128 x 128 blocks,
// dense and grouped, on the tensor cores.
//
//   out[m][n] = sum_c sa[m][c] sb[n / 128][c] P_c[m][n],   P_c = A_c B_c^T over the 128 codes of block c
//
// A tcgen05.mma pass over one block c leaves P_c in tensor memory in float32;
// the scales differ from block to block, so each P_c is read back, scaled and
// added in registers while the next block's MMAs write another part of tensor
// memory.  Three kernels share the sum:
//
//   fp8_tile_kernel    128 rows x 256 columns per CTA, persistent.
//   fp8_stream_kernel  128 columns x 16 or 32 rows per CTA with the matrix as the MMA's first operand, K split
//                      over a cluster: few rows, where reading the matrix bounds it.
//   fp8_row_kernel     16 columns x up to 16 rows per CTA, K split over its warps, the matrix from global memory
//                      straight into registers: the shortest way for a decode step's rows.
#pragma once
#include "umma.cuh"

namespace tsm {

constexpr int MAX_GROUPS = TS_MOE_MAX_EXPERTS;

struct MatmulParams {
  ts_moe_fp8_matmul_args a;
  int kb;      // scale blocks of K
  int splits;  // fp8_stream_kernel: CTAs of a cluster, which share K
  int out_map; // fp8_tile_kernel: out has a tensor map (rows from 16-byte boundary to 16-byte boundary)
  int held;    // a CTA that issues no copies and waits held_us at most: the failure path, for tests; -1: none
  unsigned held_us;
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

// Column n of rows m0 .. m0 + count - 1 (count <= R; past it the last row again): the loads go out one after another, with
// no branch between them.
template <int R>
TSM_DEV void load_column(const void* base, int type, int64_t ld, int64_t m0, int count, int64_t n, float (&v)[R]) {
  const int64_t at = m0 * ld + n;
  if (type == TS_DT_FP32) {
#pragma unroll
    for (int j = 0; j < R; ++j) v[j] = ((const float*)base)[at + min(j, count - 1) * ld];
  } else {
    uint16_t w[R];
#pragma unroll
    for (int j = 0; j < R; ++j) w[j] = ((const uint16_t*)base)[at + min(j, count - 1) * ld];
#pragma unroll
    for (int j = 0; j < R; ++j) v[j] = type == TS_DT_BF16 ? __uint_as_float((uint32_t)w[j] << 16) : __half2float(__ushort_as_half(w[j]));
  }
}
template <int R>
TSM_DEV void store_column(void* base, int type, int64_t ld, int64_t m0, int count, int64_t n, const float (&v)[R]) {
  const int64_t at = m0 * ld + n;
  if (type == TS_DT_FP32) {
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (j < count) ((float*)base)[at + j * ld] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (j < count) ((uint16_t*)base)[at + j * ld] = (uint16_t)pack2(v[j], 0.f, type);
  }
}

// ----------------------------------------------------------------------------- many rows
constexpr int TL_M = 128, TL_N = 256, TL_STAGES = 3, TL_ACC = 2;  // TL_ACC x TL_N = all 512 columns of tensor memory
constexpr int TL_BAND = 16;     // row tiles that run side by side over the columns: their rows of A stay in L2
constexpr int TL_CHUNK = 4;     // scale blocks whose scales are staged at a time
constexpr int TL_PARTS = 2, TL_COLS = TL_N / TL_PARTS;  // column parts of a tile: four warps scale and add one each
constexpr int TL_ADDERS = 4 * TL_PARTS, TL_THREADS = 128 + 32 * TL_ADDERS;  // after the producer, the MMA and two scale warps
// Registers a thread: at launch (what fits 384 threads), and as the two roles split them afterwards.
constexpr int TL_REGS = 168, TL_REGS_ISSUE = 56, TL_REGS_ADD = 224;
static_assert(128 * TL_REGS_ISSUE + 32 * TL_ADDERS * TL_REGS_ADD <= TL_THREADS * TL_REGS, "the split fits the launch's registers");

struct TileSmem {
  uint8_t a[TL_STAGES][TL_M * SCALE_BLOCK];
  uint8_t b[TL_STAGES][TL_N * SCALE_BLOCK];
  uint4 out[TL_ADDERS][2][32 * 8];  // a warp's 32 rows on their way out: two boxes of 128 bytes of each
  float scale[2][TL_CHUNK][TL_N / SCALE_BLOCK][TL_M];  // products of the scales, TL_CHUNK blocks at a time
  uint64_t full[TL_STAGES], empty[TL_STAGES], acc_full[TL_ACC], acc_empty[TL_ACC], sc_full[2], sc_empty[2], drain;
  uint32_t tmem;
  DeadMark dead;
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

// A warp's 32 rows of a tile go out through `stage`: two boxes of 128 bytes of each row at a time, 16-byte place c of
// row r at c ^ (r & 7) (the 128-byte swizzle, which also spreads rows over the banks).  Outputs from one 16-byte place to
// another leave by tensor-map stores, which run beside the next tile: all SMs reach their stores at about the same
// time, and stores by the threads kept them from the next tile's sums until HBM had taken them.  Odd places and a
// group's last rows are stored by the threads; `add` comes in the same way, a row's columns side by side.
TSM_DEV int stage_at(int r, int c) { return c / 8 * 256 + r * 8 + (c % 8 ^ (r & 7)); }

// Rows of `bytes` bytes (at most 256) from the stage to dst, ld bytes apart, at any places that elements of 2 or 4 bytes
// can have: each lane shifts two 16-byte places into the 16 bytes that stand at a boundary in memory.  Stores of single
// elements are kept to the rows' ends: sectors written in parts are several times as dear.
TSM_DEV void flush_rows(const uint4* stage, char* dst, int64_t ld, int bytes, int rows) {
  const int lane = threadIdx.x & 31, half = lane / 16, j = lane % 16;
#pragma unroll 2
  for (int r = half; r < rows; r += 2) {
    char* row = dst + r * ld;
    const int shift = (int)((uintptr_t)row & 15), at = 16 * j - shift;
    const uint4 hi = stage[stage_at(r, j)], lo = j > 0 ? stage[stage_at(r, j - 1)] : make_uint4(0, 0, 0, 0);
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int skip = 16 - shift;  // bytes of lo and hi before the ones wanted
    if (skip & 16) w[0] = w[4], w[1] = w[5], w[2] = w[6], w[3] = w[7];
    if (skip & 8) w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = w[6], w[5] = w[7];
    if (skip & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5];
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = skip & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    if (at >= 0 && at + 16 <= bytes) {
      *(uint4*)(row + at) = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + 2 * e >= 0 && at + 2 * e < bytes) *(uint16_t*)(row + at + 2 * e) = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
    }
  }
  // what shifts past the sixteenth place
  if (lane < rows) {
    char* row = dst + lane * ld;
    const int shift = (int)((uintptr_t)row & 15);
    if (256 - shift < bytes) {
      const uint4 last = stage[stage_at(lane, 15)];
      const uint32_t v[4] = {last.x, last.y, last.z, last.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (2 * e >= 16 - shift && 240 + 2 * e < bytes) *(uint16_t*)(row + 240 + 2 * e) = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
    }
  }
}

// Rows of `bytes` bytes (at most 256, even) to the stage, ld bytes apart.  The copies go on side by side and take no
// registers from the sums; only 16-bit rows at odd places come by registers, sixteen elements a lane at a time.
TSM_DEV void fetch_rows(uint4* stage, const char* src, int64_t ld, int bytes, int rows) {
  const int lane = threadIdx.x & 31;
  const uintptr_t place = (uintptr_t)src | (uintptr_t)ld;
  if (place % 16 == 0) {
    const int half = lane / 16, j = lane % 16, n = min(16, bytes - 16 * j);
    if (n > 0) {
#pragma unroll 2
      for (int r = half; r < rows; r += 2) copy16_async(&stage[stage_at(r, j)], src + r * ld + 16 * j, n);
    }
    copy_wait();
  } else if (place % 4 == 0 && bytes % 4 == 0) {
#pragma unroll 2
    for (int i = 0; i < 2 * rows; ++i) {
      const int r = i / 2, at = i % 2 * 128 + lane * 4;
      if (at < bytes) copy4_async((char*)&stage[stage_at(r, at / 16)] + at % 16, src + r * ld + at);
    }
    copy_wait();
  } else {
    for (int r0 = 0; r0 < rows; r0 += 4) {
      uint16_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = r0 + i / 4, at = i % 4 * 64 + lane * 2;
        v[i] = r < rows && at < bytes ? *(const uint16_t*)(src + r * ld + at) : (uint16_t)0;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = r0 + i / 4, at = i % 4 * 64 + lane * 2;
        *(uint16_t*)((char*)&stage[stage_at(r, at / 16)] + at % 16) = v[i];
      }
    }
  }
}

// Rows row0 .. row0 + 31 (below hi), columns col0 .. of one warp: lane l holds row row0 + l.
TSM_DEV void store_tile(const MatmulParams& p, const CUtensorMap* mo, float (&acc)[TL_COLS], uint4* stage, int row0, int hi, int col0) {
  const ts_moe_fp8_matmul_args& a = p.a;
  const int lane = threadIdx.x & 31, type = a.out_type, es = dt_size(type), rows = min(32, hi - row0);
  if (rows <= 0 || col0 >= a.n) return;  // uniform in the warp
  const bool mapped = p.out_map && (rows == 32 || hi == a.rows);  // the map ends at row a.rows
  char* const out = (char*)a.out + ((int64_t)row0 * a.ld_out + col0) * es;
  const char* const add = (const char*)a.add + ((int64_t)row0 * a.ld_add + col0) * es;
  if (lane == 0) bulk_wait_read();
  __syncwarp();
  if (type != TS_DT_FP32) {
    const int n = min(TL_COLS, a.n - col0);
    if (a.add) {
      fetch_rows(stage, add, a.ld_add * 2, n * 2, rows);
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        Raw8 raw;
        raw.a = stage[stage_at(lane, c)];
        float d[8];
        cvt8(raw, type, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[c * 8 + j] += d[j];
      }
    }
    // each lane writes the places that it alone has read
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float* v = &acc[c * 8];
      stage[stage_at(lane, c)] = make_uint4(pack2(v[0], v[1], type), pack2(v[2], v[3], type), pack2(v[4], v[5], type), pack2(v[6], v[7], type));
    }
    if (mapped) fence_proxy_async_smem();
    __syncwarp();
    if (!mapped) {
      flush_rows(stage, out, a.ld_out * 2, n * 2, rows);
      __syncwarp();
    } else if (lane == 0) {
      tma_store_2d(mo, col0, row0, stage);
      if (n > 64) tma_store_2d(mo, col0 + 64, row0, stage + 256);
      bulk_commit();
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < TL_COLS / 64; ++h) {
    const int n = min(64, a.n - col0 - h * 64);
    if (n <= 0) return;
    if (h > 0) {
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    }
    if (a.add) {
      fetch_rows(stage, add + h * 256, a.ld_add * 4, n * 4, rows);
      __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float* v = &acc[h * 64 + c * 4];
      float4 s = make_float4(v[0], v[1], v[2], v[3]);
      uint4& at = stage[stage_at(lane, c)];
      if (a.add) {
        const uint4 d = at;
        s.x += __uint_as_float(d.x), s.y += __uint_as_float(d.y), s.z += __uint_as_float(d.z), s.w += __uint_as_float(d.w);
      }
      at = make_uint4(__float_as_uint(s.x), __float_as_uint(s.y), __float_as_uint(s.z), __float_as_uint(s.w));
    }
    if (mapped) fence_proxy_async_smem();
    __syncwarp();
    if (!mapped) {
      flush_rows(stage, out + h * 256, a.ld_out * 4, n * 4, rows);
      __syncwarp();
    } else if (lane == 0) {
      tma_store_2d(mo, col0 + h * 64, row0, stage);
      if (n > 32) tma_store_2d(mo, col0 + h * 64 + 32, row0, stage + 256);
      bulk_commit();
    }
  }
}

// Persistent, a tile at a time; the MMAs of a tile's first blocks run while the last one is stored.  Per block of K the
// MMAs of 128 x 256 take 512 cycles at the tensor pipe's peak, and so does nothing else alone; what bounds the kernel is
// the chain from the MMAs' end over the read-back to the next MMAs in the same half of tensor memory, and the chip's
// power: 8192 x 14336 x 4096 in 480 us at first (2.0 PFLOP/s, tensor pipe 53 %), 550 us over a second, when the clock has come
// down to 1.5 GHz (1.75 PFLOP/s); 312 us with the sums taken out.  The adders' 128 sums each spill 160 bytes.  128 rows, not
// 256: groups waste half a tile on average.
__global__ void __launch_bounds__(TL_THREADS, 1)
    fp8_tile_kernel(const __grid_constant__ MatmulParams p, const __grid_constant__ CUtensorMap ma,
                    const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mo) {
  // Without static shared memory the dynamic part starts at a 1024-byte boundary, as the swizzled tiles need it; were it
  // otherwise, the CTA would be dead from the start and its outputs NaN.
  extern __shared__ uint8_t raw[];
  TileSmem& s = *reinterpret_cast<TileSmem*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Dead dead = {&s.dead};
  if (threadIdx.x == 0) {
    for (int i = 0; i < TL_STAGES; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < TL_ACC; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], TL_ADDERS);
    for (int i = 0; i < 2; ++i) mbar_init(&s.sc_full[i], 64), mbar_init(&s.sc_empty[i], TL_ADDERS);
    mbar_init(&s.drain, 1);
    s.dead.set = (smem_addr(raw) & 1023) != 0;
    s.dead.limit_us = (int)blockIdx.x == p.held ? p.held_us : WAIT_LIMIT_US;
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

  if (warp < 4) set_regs_down<TL_REGS_ISSUE>();
  if (warp == 0) {
    if (lane == 0) {
      unsigned it = 0;
      for (int t = blockIdx.x; t < tiles && !dead; t += gridDim.x) {
        const Tile tl = locate_tile(p, s.groups, t);
        for (int c = 0; c < p.kb; ++c, ++it) {
          const int st = it % TL_STAGES;
          if (!wait_or_die(&s.empty[st], (it / TL_STAGES & 1) ^ 1, dead)) break;
          if ((int)blockIdx.x == p.held) continue;
          mbar_arrive_expect_tx(&s.full[st], (TL_M + TL_N) * SCALE_BLOCK);
          tma_load_2d(s.a[st], &ma, c * SCALE_BLOCK, tl.m0, &s.full[st]);
          tma_load_3d(s.b[st], &mb, c * SCALE_BLOCK, tl.n0, tl.g, &s.full[st]);
        }
      }
      // no copy may be in flight when the CTA ends
      if (dead) {
        for (unsigned i = it > TL_STAGES ? it - TL_STAGES : 0; i < it; ++i) {
          wait_at_end(&s.full[i % TL_STAGES], i / TL_STAGES & 1, dead);
        }
      }
    }
  } else if (warp == 1) {
    // The whole warp runs the loop and one lane issues: descriptors computed where the warp is converged stay in uniform
    // registers.  With the loop inside a branch of one lane a block's four MMAs and two commits took 550 cycles to issue
    // and each wait 250, more than the 512 that the MMAs run.
    constexpr uint32_t idesc = umma_idesc(TL_M, TL_N);
    const uint64_t da0 = umma_desc(smem_addr(s.a[0])), db0 = umma_desc(smem_addr(s.b[0]));
    unsigned it = 0;
    for (int t = blockIdx.x; t < tiles && !dead; t += gridDim.x) {
      for (int c = 0; c < p.kb; ++c, ++it) {
        const int st = it % TL_STAGES, ac = it % TL_ACC;
        const bool ok = wait_both_or_die(&s.acc_empty[ac], (it / TL_ACC & 1) ^ 1, &s.full[st], it / TL_STAGES & 1, dead);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        const uint64_t da = da0 + st * (TL_M * SCALE_BLOCK / 16), db = db0 + st * (TL_N * SCALE_BLOCK / 16);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < SCALE_BLOCK / 32; ++k) umma_e4m3(tmem + ac * TL_N, da + 2 * k, db + 2 * k, idesc, k > 0);
          umma_commit(&s.empty[st]);
          umma_commit(&s.acc_full[ac]);
        }
        __syncwarp();
      }
    }
    // no MMA may be in flight when tensor memory is freed
    if (elect_one()) umma_commit(&s.drain);
    wait_at_end(&s.drain, 0, dead);
  } else if (warp < 4) {
    // the scales: thread i those of the tile's rows i and i + 64, times the column blocks'
    const int r = threadIdx.x - 64, nblocks = cdiv(p.a.n, SCALE_BLOCK);
    const bool vec = p.a.as_block == 1 && ((uintptr_t)p.a.a_scale | (uintptr_t)(p.a.as_row * 4)) % 16 == 0;
    unsigned it = 0;
    for (int t = blockIdx.x; t < tiles && !dead; t += gridDim.x) {
      const Tile tl = locate_tile(p, s.groups, t);
      const float* sb = p.a.b_scale + tl.g * p.a.bs_group;
      const int64_t b0 = (int64_t)(tl.n0 / SCALE_BLOCK) * p.a.bs_row, b1 = (int64_t)min(tl.n0 / SCALE_BLOCK + 1, nblocks - 1) * p.a.bs_row;
      for (int c0 = 0; c0 < p.kb; c0 += TL_CHUNK, ++it) {
        if (!wait_or_die(&s.sc_empty[it & 1], (it / 2 & 1) ^ 1, dead)) break;
        float(*out)[TL_N / SCALE_BLOCK][TL_M] = s.scale[it & 1];
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int row = r + h * 64;
          const float* sa = p.a.a_scale + (int64_t)min(tl.m0 + row, tl.hi - 1) * p.a.as_row;
          float v[TL_CHUNK];
          if (vec && c0 + TL_CHUNK <= p.kb) {
            const float4 w = *(const float4*)(sa + c0);
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
          } else {
#pragma unroll
            for (int i = 0; i < TL_CHUNK; ++i) v[i] = c0 + i < p.kb ? sa[(int64_t)(c0 + i) * p.a.as_block] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < TL_CHUNK; ++i) {
            const int64_t c = (int64_t)min(c0 + i, p.kb - 1) * p.a.bs_block;
            out[i][0][row] = v[i] * sb[b0 + c];
            out[i][1][row] = v[i] * sb[b1 + c];
          }
        }
        mbar_arrive(&s.sc_full[it & 1]);
      }
    }
  } else {
    set_regs_up<TL_REGS_ADD>();
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + part * TL_COLS;
    const float* scale = &s.scale[0][0][part * TL_COLS / SCALE_BLOCK][quarter * 32 + lane];
    unsigned it = 0, chunk = 0;
    bool ready = false;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      float acc[TL_COLS];
#pragma unroll
      for (int j = 0; j < TL_COLS; ++j) acc[j] = 0.f;
      for (int c0 = 0; c0 < p.kb; c0 += TL_CHUNK, ++chunk) {
        wait_or_die(&s.sc_full[chunk & 1], chunk / 2 & 1, dead);  // a dead CTA runs on without waiting
        const float* from = scale + (chunk & 1) * (TL_CHUNK * (TL_N / SCALE_BLOCK) * TL_M);
        const int ce = min(TL_CHUNK, p.kb - c0);
        float next = *from;
        for (int i = 0; i < ce; ++i, ++it) {
          const int ac = it % TL_ACC;
          const float sc = next;
          if (!ready) wait_or_die(&s.acc_full[ac], it / TL_ACC & 1, dead);
          __syncwarp();
          tc_fence_after();
          float v[2][32];
          tmem_ld(mine + ac * TL_N, v[0]);
          // Shared memory answers after some 200 cycles beside the MMAs' and the copies' traffic: what the next block needs
          // is asked for here.
          if (i + 1 < ce) next = from[(i + 1) * (TL_N / SCALE_BLOCK * TL_M)];
#pragma unroll
          for (int q = 0; q < TL_COLS / 32; ++q) {
            tc_wait_ld(v[q & 1]);
            if (q + 1 < TL_COLS / 32) {
              tmem_ld(mine + ac * TL_N + (q + 1) * 32, v[(q + 1) & 1]);
            } else {  // all read: the MMAs may write here again
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&s.acc_empty[ac]);
                if (i == ce - 1) mbar_arrive(&s.sc_empty[chunk & 1]);
              }
            }
            if (q == 3) ready = mbar_test(&s.acc_full[(it + 1) % TL_ACC], (it + 1) / TL_ACC & 1);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[q * 32 + j] += sc * v[q & 1][j];
          }
        }
      }
      if (dead) {
#pragma unroll
        for (int j = 0; j < TL_COLS; ++j) acc[j] = NAN;
      }
      const Tile tl = locate_tile(p, s.groups, t);
      store_tile(p, &mo, acc, s.out[warp - 4][0], tl.m0 + quarter * 32, tl.hi, tl.n0 + part * TL_COLS);
    }
    if (lane == 0) bulk_wait();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) tmem_free<512>(tmem);
}

// ----------------------------------------------------------------------------- few rows
constexpr int ST_N = 128, ST_THREADS = 192;  // producer warp, MMA warp, 4 warps that scale and add
constexpr int MAX_SPLITS = 4;                // CTAs of a cluster
constexpr int ST_CHUNK = 8;                  // scale blocks whose row scales are staged at a time

template <int BT>
struct StreamShape {
  static constexpr int STAGES = BT == 16 ? 5 : 4;
  static constexpr int ACC = BT == 16 ? 8 : 4;  // parts of tensor memory
  static constexpr int COLS = ACC * BT;
  static constexpr int CTAS = 2;  // per SM
};

template <int BT>
struct StreamSmem {
  using S = StreamShape<BT>;
  uint8_t b[S::STAGES][ST_N * SCALE_BLOCK];
  uint8_t a[S::STAGES][BT * SCALE_BLOCK];
  float red[BT][ST_N];              // this CTA's share of K, for the cluster's CTAs to add
  float scale[2][ST_CHUNK][BT];     // sa * sb of the blocks at hand
  uint64_t full[S::STAGES], empty[S::STAGES], acc_full[S::ACC], acc_empty[S::ACC], red_full, drain;
  uint32_t tmem;
  DeadMark dead;
  GroupTable groups;
};

// The matrix as the MMA's first operand: 128 of its rows are one instruction's, whatever few tokens there are.  64 routes
// that reach 28 of 32 experts of 5760 x 2880 in 76.2 us (6.1 TB/s: HBM bounds it); 16 x 5760 x 2880 in 6.3 us, of which 2.6 us are
// traffic and the rest a chain of latencies (launch, TMA, MMA, read-back, the cluster's sum).
template <int BT>
__global__ void __launch_bounds__(ST_THREADS, StreamShape<BT>::CTAS)
    fp8_stream_kernel(const MatmulParams p, const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb) {
  using S = StreamShape<BT>;
  extern __shared__ uint8_t raw[];
  StreamSmem<BT>& s = *reinterpret_cast<StreamSmem<BT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Dead dead = {&s.dead};
  const int splits = p.splits, rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::STAGES; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < S::ACC; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], 4);
    mbar_init(&s.red_full, 4 * splits);
    mbar_init(&s.drain, 1);
    s.dead.set = 0;
    s.dead.limit_us = (int)blockIdx.x == p.held ? p.held_us : WAIT_LIMIT_US;
    fence_barrier_init();
    prefetch_map(&ma);
    prefetch_map(&mb);
  }
  cluster_sync();  // the peers' barriers are ready
  // Tensor memory is taken after the cluster has met: from here on a CTA that holds some waits for its peers for a limited
  // time only.  Before, a peer that waits for tensor memory (which has no limit) could have kept it from others for good.
  if (warp == 1) tmem_alloc<S::COLS>(&s.tmem);
  if (warp == 0 && !p.a.offsets) fill_groups(p.a, BT, s.groups);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // what needs no other kernel's results comes before the wait for them: divisions here took most of a microsecond
  const uint32_t tmem = s.tmem;
  const int nt = cdiv(p.a.n, ST_N);
  const int c0 = p.kb * rank / splits, c1 = p.kb * (rank + 1) / splits;
  const int first = blockIdx.x / splits, step = gridDim.x / splits;
  const int t0 = first / nt, n00 = (first - t0 * nt) * ST_N;  // row tile and column of the first item
  grid_dep_wait();
  grid_dep_launch();
  if (p.a.offsets) {
    if (warp == 0) fill_groups(p.a, BT, s.groups);
    __syncthreads();
  }
  const int items = s.groups.first[p.a.num_groups] * nt;

  if (warp == 0) {
    if (lane == 0) {
      unsigned it = 0;
      for (int t = first; t < items && !dead; t += step) {
        const int tt = t == first ? t0 : t / nt, g = group_of(s.groups, p.a.num_groups, tt);
        const int m0 = s.groups.lo[g] + (tt - s.groups.first[g]) * BT, n0 = t == first ? n00 : (t - tt * nt) * ST_N;
        for (int c = c0; c < c1; ++c, ++it) {
          const int st = it % S::STAGES;
          if (!wait_or_die(&s.empty[st], (it / S::STAGES & 1) ^ 1, dead)) break;
          if ((int)blockIdx.x == p.held) continue;
          mbar_arrive_expect_tx(&s.full[st], (ST_N + BT) * SCALE_BLOCK);
          tma_load_3d(s.b[st], &mb, c * SCALE_BLOCK, n0, g, &s.full[st]);
          tma_load_2d(s.a[st], &ma, c * SCALE_BLOCK, m0, &s.full[st]);
        }
      }
      if (dead) {
        for (unsigned i = it > S::STAGES ? it - S::STAGES : 0; i < it; ++i) {
          wait_at_end(&s.full[i % S::STAGES], i / S::STAGES & 1, dead);
        }
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = umma_idesc(ST_N, BT);
    const uint64_t db0 = umma_desc(smem_addr(s.b[0])), da0 = umma_desc(smem_addr(s.a[0]));
    unsigned it = 0;
    for (int t = first; t < items && !dead; t += step) {
      for (int c = c0; c < c1; ++c, ++it) {
        const int st = it % S::STAGES, ac = it % S::ACC;
        const bool ok = wait_both_or_die(&s.acc_empty[ac], (it / S::ACC & 1) ^ 1, &s.full[st], it / S::STAGES & 1, dead);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        const uint64_t db = db0 + st * (ST_N * SCALE_BLOCK / 16), da = da0 + st * (BT * SCALE_BLOCK / 16);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < SCALE_BLOCK / 32; ++k) umma_e4m3(tmem + ac * BT, db + 2 * k, da + 2 * k, idesc, k > 0);
          umma_commit(&s.empty[st]);
          umma_commit(&s.acc_full[ac]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(&s.drain);
    wait_at_end(&s.drain, 0, dead);
  } else {
    // thread r of these 128: column n0 + r of the tile, all BT rows
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int PER = ST_CHUNK * BT / 128;  // scales a thread stages per chunk
    const int type = p.a.out_type;
    unsigned it = 0;
    for (int t = first; t < items; t += step) {
      const int tt = t == first ? t0 : t / nt, g = group_of(s.groups, p.a.num_groups, tt);
      const int m0 = s.groups.lo[g] + (tt - s.groups.first[g]) * BT, rows = min(BT, s.groups.lo[g + 1] - m0);
      const int n0 = t == first ? n00 : (t - tt * nt) * ST_N;
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
          float v[BT];
          tmem_ld(mine + ac * BT, v);
          tc_wait_ld(v);
#pragma unroll
          for (int j = 0; j < BT; j += 4) {
            const float4 f = *(const float4*)&s.scale[buf][i][j];
            acc[j] += f.x * v[j];
            acc[j + 1] += f.y * v[j + 1];
            acc[j + 2] += f.z * v[j + 2];
            acc[j + 3] += f.w * v[j + 3];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.acc_empty[ac]);
        }
      }
      bar_sync(1, 128);  // the scale buffers are free for the next item
      const int64_t n = n0 + r;
      if (splits == 1) {
        const bool lost = (bool)dead;
#pragma unroll
        for (int j0 = 0; j0 < BT; j0 += 8) {
          if (j0 < rows && n < p.a.n) {
            float v[8], d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (p.a.add) load_column<8>(p.a.add, type, p.a.ld_add, m0 + j0, min(rows - j0, 8), n, d);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (lost ? NAN : acc[j0 + j]) + d[j];
            store_column<8>(p.a.out, type, p.a.ld_out, m0 + j0, min(rows - j0, 8), n, v);
          }
        }
        continue;
      }
      // Every CTA of the cluster adds a share of the rows, over the CTAs in order.  K is split only where the grid has a
      // cluster for every item (matmul_plan), so this is the cluster's one item and s.red is written once.  A CTA that gave up
      // has no sum to give: NaN, which every CTA's share of the rows takes over.
      const bool none = (bool)dead;
#pragma unroll
      for (int j = 0; j < BT; ++j) s.red[j][r] = none ? NAN : acc[j];
      __syncwarp();
      if (lane < splits) peer_arrive(peer_addr(smem_addr(&s.red_full), lane));
      wait_cluster_or_die(&s.red_full, 0, dead);
      __syncwarp();
      const bool lost = (bool)dead;
      const int j0 = rows * rank / splits, j1 = rows * (rank + 1) / splits;
      // eight rows at a time of all CTAs: no load waits for another, nor for a branch (rows past the share are read and
      // dropped; loads behind a condition each took 5500 cycles for six rows of three CTAs)
      constexpr int R = 8;
      const uint32_t mine_at = smem_addr(&s.red[0][r]);
      uint32_t at[MAX_SPLITS];
#pragma unroll
      for (int q = 0; q < MAX_SPLITS; ++q) at[q] = peer_addr(mine_at, min(q, splits - 1));
      for (int jb = j0; jb < j1; jb += R) {
        float w[MAX_SPLITS][R], d[R] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < MAX_SPLITS; ++q) {
          if (q < splits) {
#pragma unroll
            for (int j = 0; j < R; ++j) w[q][j] = peer_load(at[q] + min(jb + j, BT - 1) * (uint32_t)(ST_N * sizeof(float)));
          } else {
#pragma unroll
            for (int j = 0; j < R; ++j) w[q][j] = 0.f;
          }
        }
        if (n < p.a.n) {
          if (p.a.add) load_column<R>(p.a.add, type, p.a.ld_add, m0 + jb, min(j1 - jb, R), n, d);
#pragma unroll
          for (int j = 0; j < R; ++j) {
            float v = w[0][j];
#pragma unroll
            for (int q = 1; q < MAX_SPLITS; ++q) v += w[q][j];
            d[j] += lost ? NAN : v;
          }
          store_column<R>(p.a.out, type, p.a.ld_out, m0 + jb, min(j1 - jb, R), n, d);
        }
      }
      break;
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) tmem_free<S::COLS>(tmem);
  cluster_sync();  // no peer reads this CTA's memory any more
}

// ----------------------------------------------------------------------------- a decode step's rows
// mma.sync m16n8k16 in FP16 (every E4M3 code is an FP16 value, products and sums in float32): the matrix's rows are the
// MMA's, tokens its columns.  Which k stands at which place of a fragment is free as long as both operands agree, so a
// lane takes sixteen neighbouring codes of a row and they serve four MMAs.  Registers, one barrier and no other
// set-up: 1 x 1024 x 2048 in 3.4 us against 5.3 by fp8_stream_kernel, 1 x 4096 x 4096 in 6.2 us (2.7 TB/s); the launch and
// the trips to HBM of a warp's few blocks one after another bound it.
constexpr int RW_N = 16, RW_MAX_ROWS = 16, RW_WARPS = 8, RW_THREADS = 32 * RW_WARPS;

// Sixteen codes from `at` of a row of k; past k they are zeros.
TSM_DEV uint4 load_codes(const uint8_t* row, int at, int k, bool in) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (!in || at >= k) return v;
  if (at + 16 <= k) return *(const uint4*)(row + at);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (at + i < k) w[i / 4] |= (uint32_t)row[at + i] << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four E4M3 codes as two pairs of FP16.
TSM_DEV uint2 e4m3x4_to_f16(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}

// NT: groups of eight tokens.  The CTA's warps share K.
template <int NT>
__global__ void __launch_bounds__(RW_THREADS, 2) fp8_row_kernel(const MatmulParams p) {
  constexpr int AHEAD = NT == 1 ? 3 : 2;  // scale blocks of the matrix on their way to a warp
  __shared__ float red[RW_WARPS][8 * NT][RW_N + 1];
  const ts_moe_fp8_matmul_args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.x * RW_N;
  const int b0 = p.kb * warp / RW_WARPS, b1 = p.kb * (warp + 1) / RW_WARPS;
  grid_dep_wait();
  grid_dep_launch();
  const uint8_t* w0 = a.b + (int64_t)(n0 + g) * a.ld_b;
  const uint8_t* w1 = w0 + 8 * a.ld_b;
  const bool in0 = n0 + g < a.n, in1 = n0 + g + 8 < a.n;
  // lane (g, c) holds codes 64 h + 16 c .. + 15 of a block, h = 0, 1, of its two rows and of tokens g, g + 8
  uint4 A[AHEAD][2][2], X[2][NT][2];
  float sa[2][NT][2], sb[2];
  auto fetch_a = [&](int b, uint4 (&f)[2][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = b < b1 ? b * SCALE_BLOCK + h * 64 + c * 16 : a.k;
      f[h][0] = load_codes(w0, at, a.k, in0);
      f[h][1] = load_codes(w1, at, a.k, in1);
    }
  };
  auto fetch_x = [&](int b, int buf) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int m = t * 8 + g;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        X[buf][t][h] = load_codes(a.a + (int64_t)m * a.ld_a, b < b1 ? b * SCALE_BLOCK + h * 64 + c * 16 : a.k, a.k, m < a.rows);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = t * 8 + c * 2 + j;  // the tokens of this lane's sums
        sa[buf][t][j] = b < b1 && q < a.rows ? a.a_scale[(int64_t)q * a.as_row + (int64_t)b * a.as_block] : 0.f;
      }
    }
    sb[buf] = b < b1 ? a.b_scale[(int64_t)(n0 / SCALE_BLOCK) * a.bs_row + (int64_t)b * a.bs_block] : 0.f;
  };
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch_a(b0 + i, A[i]);
  fetch_x(b0, 0);
  for (int b = b0; b < b1; b += 2 * AHEAD) {
#pragma unroll
    for (int i = 0; i < 2 * AHEAD; ++i) {  // an even number of steps: buffers of X and slots of A by constants
      if (b + i >= b1) break;
      const int buf = i & 1, slot = i % AHEAD;
      fetch_x(b + i + 1, buf ^ 1);
      float P[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) P[t][0] = P[t][1] = P[t][2] = P[t][3] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t r0[4] = {A[slot][h][0].x, A[slot][h][0].y, A[slot][h][0].z, A[slot][h][0].w};
        const uint32_t r1[4] = {A[slot][h][1].x, A[slot][h][1].y, A[slot][h][1].z, A[slot][h][1].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint2 lo = e4m3x4_to_f16(r0[s]), hi = e4m3x4_to_f16(r1[s]);
          const uint32_t fa[4] = {lo.x, hi.x, lo.y, hi.y};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 x = X[buf][t][h];
            const uint2 fx = e4m3x4_to_f16(s == 0 ? x.x : s == 1 ? x.y : s == 2 ? x.z : x.w);
            mma_f16_acc(P[t], fa, fx.x, fx.y);
          }
        }
      }
      fetch_a(b + i + AHEAD, A[slot]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] += sa[buf][t][j & 1] * sb[buf] * P[t][j];
      }
    }
  }
  // D: rows g and g + 8 of the matrix, tokens 2c and 2c + 1
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int j = 0; j < 4; ++j) red[warp][t * 8 + c * 2 + (j & 1)][g + 8 * (j >> 1)] = acc[t][j];
  }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < 8 * NT * RW_N; i += RW_THREADS) {
    const int m = i / RW_N, n = i % RW_N;
    if (m < a.rows && n0 + n < a.n) {
      float v = a.add ? load1(a.add, a.out_type, (int64_t)m * a.ld_add + n0 + n) : 0.f, s = 0.f;
#pragma unroll
      for (int q = 0; q < RW_WARPS; ++q) s += red[q][m][n];
      store1(a.out, a.out_type, (int64_t)m * a.ld_out + n0 + n, s + v);
    }
  }
}

}  // namespace tsm
