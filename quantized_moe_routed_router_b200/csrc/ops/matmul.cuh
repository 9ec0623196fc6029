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
  int out_map; // fp8_tile_kernel: out has a tensor map (rows at 16-byte boundaries)
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

// Rows row0 .. row0 + 31 (below hi), columns col0 .. of one warp: lane l holds row row0 + l.  They go out through
// `stage`: two boxes of 128 bytes of each row at a time, 16-byte place c of row r at c ^ (r & 7) (the 128-byte swizzle,
// which also spreads rows over the banks).  Plain outputs leave by tensor-map stores, which run beside the next tile:
// all SMs reach their stores at about the same time, and stores by the threads kept them from the next tile's sums
// until HBM had taken them.  Odd places and a group's last rows are stored by the threads, and so are sums with `add`.
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

TSM_DEV void store_tile(const MatmulParams& p, const CUtensorMap* mo, const float (&acc)[TL_COLS], uint4* stage, int row0, int hi, int col0) {
  const ts_moe_fp8_matmul_args& a = p.a;
  const int lane = threadIdx.x & 31, type = a.out_type, es = dt_size(type), rows = min(32, hi - row0);
  if (rows <= 0 || col0 >= a.n) return;  // uniform in the warp
  const bool vec = ((uintptr_t)a.out | (uintptr_t)(a.ld_out * es)) % 16 == 0;
  const bool mapped = p.out_map && !a.add && (rows == 32 || hi == a.rows);  // the map ends at row a.rows
  char* const out0 = (char*)a.out + ((int64_t)row0 * a.ld_out + col0) * es;
  if (type != TS_DT_FP32 && !a.add) {
    if (lane == 0) bulk_wait_read();
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float* v = &acc[c * 8];
      stage[stage_at(lane, c)] = make_uint4(pack2(v[0], v[1], type), pack2(v[2], v[3], type), pack2(v[4], v[5], type), pack2(v[6], v[7], type));
    }
    if (mapped) fence_proxy_async_smem();
    __syncwarp();
    if (!mapped) {
      flush_rows(stage, out0, a.ld_out * 2, min(TL_COLS, a.n - col0) * 2, rows);
    } else if (lane == 0) {
      tma_store_2d(mo, col0, row0, stage);
      if (col0 + 64 < a.n) tma_store_2d(mo, col0 + 64, row0, stage + 256);
      bulk_commit();
    }
    return;
  }
  const bool vec4 = vec && a.n % 4 == 0 && ((uintptr_t)a.add | (uintptr_t)(a.ld_add * es)) % 16 == 0;
#pragma unroll
  for (int h = 0; h < TL_COLS / 64; ++h) {
    const int c0 = col0 + h * 64, n = min(64, a.n - c0);
    if (n <= 0) return;
    if (lane == 0) bulk_wait_read();
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float* v = &acc[h * 64 + c * 4];
      stage[stage_at(lane, c)] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    if (type == TS_DT_FP32 && mapped) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(mo, c0, row0, stage);
        if (n > 32) tma_store_2d(mo, c0 + 32, row0, stage + 256);
        bulk_commit();
      }
      continue;
    }
    __syncwarp();
    if (!a.add) {
      flush_rows(stage, out0 + h * 256, a.ld_out * 4, n * 4, rows);
    } else if (vec4) {
      const int half = lane / 16, place = lane % 16;
      const int64_t col = c0 + place * 4;
      if (place * 4 < n) {
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 16) {
          float d[8][4];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = r0 + i * 2 + half;
            d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
            if (r < rows) {
              const int64_t at = (int64_t)(row0 + r) * a.ld_add + col;
              if (type == TS_DT_FP32) {
                const float4 w = *(const float4*)((const float*)a.add + at);
                d[i][0] = w.x, d[i][1] = w.y, d[i][2] = w.z, d[i][3] = w.w;
              } else {
                const uint2 w = *(const uint2*)((const uint16_t*)a.add + at);
                Raw8 raw;
                raw.a = make_uint4(w.x, w.y, 0, 0);
                float f[8];
                cvt8(raw, type, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = f[j];
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = r0 + i * 2 + half;
            if (r < rows) {
              const uint4 w = stage[stage_at(r, place)];
              const float v[4] = {__uint_as_float(w.x) + d[i][0], __uint_as_float(w.y) + d[i][1], __uint_as_float(w.z) + d[i][2],
                                  __uint_as_float(w.w) + d[i][3]};
              const int64_t at = (int64_t)(row0 + r) * a.ld_out + col;
              if (type == TS_DT_FP32)
                *(float4*)((float*)a.out + at) = make_float4(v[0], v[1], v[2], v[3]);
              else
                *(uint2*)((uint16_t*)a.out + at) = make_uint2(pack2(v[0], v[1], type), pack2(v[2], v[3], type));
            }
          }
        }
      }
    } else {
      // odd places: 32 columns of a row at a time, element by element
      const float* f = (const float*)stage;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 8) {
        float d[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = r0 + i / 2, c = i % 2 * 32 + lane;
          d[i] = r < rows && c < n ? load1(a.add, type, (int64_t)(row0 + r) * a.ld_add + c0 + c) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = r0 + i / 2, c = i % 2 * 32 + lane;
          if (r < rows && c < n) store1(a.out, type, (int64_t)(row0 + r) * a.ld_out + c0 + c, f[stage_at(r, c / 4) * 4 + c % 4] + d[i]);
        }
      }
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(TL_THREADS, 1)
    fp8_tile_kernel(const __grid_constant__ MatmulParams p, const __grid_constant__ CUtensorMap ma,
                    const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mo) {
  // Without static shared memory the dynamic part starts at a 1024-byte boundary, as the swizzled tiles need it; were it
  // otherwise, the CTA would be dead from the start and its outputs NaN.
  extern __shared__ uint8_t raw[];
  TileSmem& s = *reinterpret_cast<TileSmem*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* dead = &s.dead;
  if (threadIdx.x == 0) {
    for (int i = 0; i < TL_STAGES; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < TL_ACC; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], TL_ADDERS);
    for (int i = 0; i < 2; ++i) mbar_init(&s.sc_full[i], 64), mbar_init(&s.sc_empty[i], TL_ADDERS);
    mbar_init(&s.drain, 1);
    s.dead = (smem_addr(raw) & 1023) != 0;
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
    // The whole warp runs the loop and one lane issues: descriptors computed where the warp is converged stay in uniform
    // registers.  With the loop inside a branch of one lane a block's four MMAs and two commits took 550 cycles to issue
    // and each wait 250, more than the 512 that the MMAs run.
    constexpr uint32_t idesc = umma_idesc(TL_M, TL_N);
    const uint64_t da0 = umma_desc(smem_addr(s.a[0])), db0 = umma_desc(smem_addr(s.b[0]));
    unsigned it = 0;
    for (int t = blockIdx.x; t < tiles && !*dead; t += gridDim.x) {
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
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(&s.drain, 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
    }
  } else if (warp < 4) {
    // the scales: thread i those of the tile's rows i and i + 64, times the column blocks'
    const int r = threadIdx.x - 64, nblocks = cdiv(p.a.n, SCALE_BLOCK);
    const bool vec = p.a.as_block == 1 && ((uintptr_t)p.a.a_scale | (uintptr_t)(p.a.as_row * 4)) % 16 == 0;
    unsigned it = 0;
    for (int t = blockIdx.x; t < tiles && !*dead; t += gridDim.x) {
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
          tmem_ld32(mine + ac * TL_N, v[0]);
          // Shared memory answers after some 200 cycles beside the MMAs' and the copies' traffic: what the next block needs
          // is asked for here.
          if (i + 1 < ce) next = from[(i + 1) * (TL_N / SCALE_BLOCK * TL_M)];
#pragma unroll
          for (int q = 0; q < TL_COLS / 32; ++q) {
            tc_wait_ld(v[q & 1]);
            if (q + 1 < TL_COLS / 32) {
              tmem_ld32(mine + ac * TL_N + (q + 1) * 32, v[(q + 1) & 1]);
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
      if (*dead) {
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
  if (warp == 0 && !p.a.offsets) fill_groups(p.a, BT, s.groups);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the peers' barriers are ready
  grid_dep_wait();
  grid_dep_launch();
  if (p.a.offsets) {
    if (warp == 0) fill_groups(p.a, BT, s.groups);
    __syncthreads();
  }
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
        for (int j0 = 0; j0 < BT; j0 += 8) {
          float d[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            d[j] = p.a.add && j0 + j < rows && n < p.a.n ? load1(p.a.add, type, (int64_t)(m0 + j0 + j) * p.a.ld_add + n) : 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < rows && n < p.a.n)
              store1(p.a.out, type, (int64_t)(m0 + j0 + j) * p.a.ld_out + n, (lost ? NAN : acc[j0 + j]) + d[j]);
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
      // eight rows at a time: their loads run side by side
      for (int jb = j0; jb < j1; jb += 8) {
        float v[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = jb + j < j1 && n < p.a.n;
          d[j] = p.a.add && in ? load1(p.a.add, type, (int64_t)(m0 + jb + j) * p.a.ld_add + n) : 0.f;
          v[j] = 0.f;
        }
        for (int q = 0; q < splits; ++q) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (jb + j < j1) v[j] += peer_load(peer_addr(smem_addr(&s.red[jb + j][r]), q));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (jb + j < j1 && n < p.a.n) store1(p.a.out, type, (int64_t)(m0 + jb + j) * p.a.ld_out + n, (lost ? NAN : v[j]) + d[j]);
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
