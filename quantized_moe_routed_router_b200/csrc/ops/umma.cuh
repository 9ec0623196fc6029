// Tensor-core (tcgen05) and tensor-map (TMA) helpers of the 8-bit product, and
// its bounded waits.  Hand-written inline PTX.
#pragma once
#include <cuda.h>

#include "elem.cuh"

namespace tsm {

// ----------------------------------------------------------------------------- waits
// Waits for the phase with `parity` of `bar`; gives up after dead.limit() nanoseconds, or when another thread of the CTA
// has, and marks the CTA dead.  The clock and the mark are looked at once in WAIT_TRIES tries: both reads take longer than
// a try, and a wait that ends meanwhile would be noticed late.  wait_cluster_or_die sees
// what the cluster's other CTAs wrote before their arrivals.
constexpr unsigned WAIT_TRIES = 64;

TSM_DEV bool try_wait_cluster(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Whether the phase has completed, without waiting.
TSM_DEV bool mbar_test(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

constexpr unsigned WAIT_LIMIT_US = WAIT_LIMIT_NS / 1000;

// The CTA's mark, and how long its waits last: WAIT_LIMIT_NS, but for a CTA that a test holds back.
struct DeadMark {
  int set;
  unsigned limit_us;
};
struct Dead {
  volatile DeadMark* mark;
  TSM_DEV explicit operator bool() const { return mark->set != 0; }
  TSM_DEV void set() const { mark->set = 1; }
  TSM_DEV unsigned long long limit() const { return mark->limit_us * 1000ull; }
};

// `ready` tries once.
template <typename Try>
TSM_DEV bool bounded_wait(const Try& ready, const Dead& dead) {
  unsigned long long t0 = 0;
  while (true) {
    for (unsigned i = 0; i < WAIT_TRIES; ++i)
      if (ready()) return true;
    if (dead) return false;
    const unsigned long long now = globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 > dead.limit()) {
      dead.set();
      return false;
    }
  }
}
TSM_DEV bool wait_or_die(uint64_t* bar, unsigned parity, const Dead& dead) {
  return bounded_wait([&] { return mbar_try_wait(bar, parity); }, dead);
}
TSM_DEV bool wait_cluster_or_die(uint64_t* bar, unsigned parity, const Dead& dead) {
  return bounded_wait([&] { return try_wait_cluster(bar, parity); }, dead);
}
// The same where the mark says nothing (the CTA's copies and MMAs in flight, at its end).
TSM_DEV void wait_at_end(uint64_t* bar, unsigned parity, const Dead& dead) {
  const unsigned long long t0 = globaltimer(), limit = dead.limit();
  while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < limit) {
  }
}
// Two barriers at once: the tries run side by side.
TSM_DEV bool wait_both_or_die(uint64_t* a, unsigned pa, uint64_t* b, unsigned pb, const Dead& dead) {
  return bounded_wait(
      [&] {
        const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
        return x && y;
      },
      dead);
}

// One lane of a converged warp, the same each time.
TSM_DEV bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// ----------------------------------------------------------------------------- registers of a warpgroup (all four warps call)
template <int N>
TSM_DEV void set_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
TSM_DEV void set_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// ----------------------------------------------------------------------------- cluster
TSM_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
TSM_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The shared-memory address `addr` names in CTA `rank` of the cluster.
TSM_DEV uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
TSM_DEV void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
TSM_DEV float peer_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ----------------------------------------------------------------------------- tensor-map loads (no multicast)
TSM_DEV void prefetch_map(const CUtensorMap* m) { asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory"); }

TSM_DEV void tma_load_2d(void* dst, const CUtensorMap* m, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(m), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
TSM_DEV void tma_load_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// ----------------------------------------------------------------------------- tensor-map stores
// Stores a tile of shared memory that this thread fenced; what lies past the map's extents is left out.
TSM_DEV void tma_store_2d(const CUtensorMap* m, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m), "r"(x), "r"(y),
               "r"(smem_addr(src))
               : "memory");
}
TSM_DEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
TSM_DEV void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }  // the sources may be written again
TSM_DEV void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ----------------------------------------------------------------------------- element copies
// global -> shared without registers: 16 bytes at 16-byte places, of which `bytes` are read and the rest zeros; 4 bytes.
TSM_DEV void copy16_async(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
TSM_DEV void copy4_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
TSM_DEV void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ----------------------------------------------------------------------------- tcgen05
template <int COLS>
TSM_DEV void tmem_alloc(uint32_t* slot) {  // one whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "n"(COLS)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS>
TSM_DEV void tmem_free(uint32_t addr) {  // the warp that allocated
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS) : "memory");
}
TSM_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
TSM_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor: K-major rows of 128 bytes, 128-byte swizzle,
// eight-row groups 1024 bytes apart.  `addr`: a 1024-byte aligned tile, plus 32
// bytes per K step of 32 codes.
TSM_DEV uint64_t umma_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Instruction descriptor: E4M3 x E4M3 -> float32, both operands K-major.
__host__ __device__ constexpr uint32_t umma_idesc(int m, int n) {
  return 1u << 4 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// D (tensor memory) = A B^T (+ D): 32 codes of K, one thread issues.
TSM_DEV void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// One arrival at `bar` when all of this thread's earlier MMAs are done.
TSM_DEV void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// Sixteen columns of this warp's 32 lanes (lane quarter warp % 4); tc_wait_ld(v) before use.
TSM_DEV void tmem_ld(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Thirty-two columns.
TSM_DEV void tmem_ld(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr));
}

// Waits for this thread's loads from tensor memory.  Naming the registers keeps their uses behind it.
TSM_DEV void tc_wait_ld(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
TSM_DEV void tc_wait_ld(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                 "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
               :
               : "memory");
  asm volatile("" : "+f"(v[30]), "+f"(v[31]));
}

}  // namespace tsm
