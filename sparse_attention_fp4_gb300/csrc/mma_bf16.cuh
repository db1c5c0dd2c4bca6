// tcgen05 helpers of the bf16 attention kernels: descriptors of 128-byte-swizzled operands,
// the bf16 MMA, tensor-memory loads and stores, cp.async and stmatrix.
#pragma once

#include "pipeline.cuh"
#include "ptx.cuh"

namespace fp4idx {
namespace mma {

// Bounded wait of the warp for an mbarrier phase, as pipe::wait_warp, but timed by the SM's
// clock (ctl.timeout_ns holds cycles): reading the global timer takes longer than most
// waits here last.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const pipe::Ctl& c, bool honor_abort = true) {
  bool ok = ptx::mbar_try_wait(bar, parity);
  if (!ok) {
    const int64_t t0 = clock64();
    for (uint32_t it = 1;; ++it) {
      ok = ptx::mbar_try_wait(bar, parity);
      if (ok) break;
      if ((it & 15u) == 0) {
        if (honor_abort && *c.abort) break;
        if (clock64() - t0 > (int64_t)c.timeout_ns) {
          pipe::give_up(c);
          break;
        }
      }
    }
  }
  return __all_sync(pipe::kFull, ok);
}

// Before a barrier is set up anew; nothing may be waiting on it.
__device__ __forceinline__ void mbar_inval(uint32_t bar) {
  asm volatile("mbarrier.inval.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// Operands lie in shared memory as rows of 128 bytes (64 bf16), eight rows an atom of 1,024
// bytes whose 16-byte pieces are stored at piece ^ (row & 7).  K-major: rows are M or N,
// 1,024 bytes (sbo) between groups of eight rows; the 16 elements of K of one MMA start 32
// bytes after the last one's.  M-major (the transposed use of the same bytes): rows are K,
// `lbo` bytes between runs of 64 M, 1,024 (sbo) between groups of eight K.
//
// A descriptor is kept as its low word (address and lbo) and its constant high word, so that
// the step from one MMA to the next is one 32-bit addition of a constant: descriptors built
// from addresses each time cost the issuing thread some 15 cycles an MMA.  The issuing warp
// runs as one, with warp-uniform descriptors, and elects a thread for each burst: issued
// from a branch of one lane, an MMA takes 46 cycles whatever its size, since the operands
// then go through per-thread registers.  Measured for K = 16 and M x N on one SM: 64x16 24
// cycles, 64x64 33, 128x64 48, 64x128 and 128x128 63, 128x256 123.
// (In a cluster the addresses of shared memory have the CTA's rank in their upper bits.)
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // sbo 1,024, version, 128-byte swizzle
// kind::f16: D f32, A and B bf16; a_m_major: A is stored with M contiguous.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool a_m_major, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_m_major ? 1u : 0u) << 15) | ((b_n_major ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// D[tmem] (+)= A[smem] x B[smem]^T, issued by one thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHi)
      : "memory");
}

// The same with A (K-major, two bf16 a column) in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHi)
      : "memory");
}

// Shared-memory offset of 16-byte piece `piece` of row `row` of a swizzled block.
__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t piece) {
  return row * 128 + ((piece ^ (row & 7)) << 4);
}

// One box of a 2-D tensor map, its bytes counted on `bar`.
__device__ __forceinline__ void tma_2d(uint32_t dst, const void* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// 16 bytes from global to shared memory, or 16 zero bytes (`bytes` = 0: nothing is read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Distributed shared memory: the address of `addr` in CTA `cta` of the cluster, a store to such
// an address, and a barrier of all the cluster's threads that orders those stores.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Four 8x8 b16 matrices, each stored transposed: lane l gives the address of row l % 8 of
// matrix l / 8; register i of lane l holds elements (row l / 4, cols 2 (l % 4) + {0, 1}) of
// matrix i before the transposition.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Packed pairs: a * b + c and a + b, each element rounded once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
      "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\tmov.b64 pc, {%6, %7};\n\t"
      "fma.rn.f32x2 pc, pa, pb, pc;\n\tmov.b64 {%0, %1}, pc;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 pa, pb;\n\t"
      "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
      "add.rn.f32x2 pa, pa, pb;\n\tmov.b64 {%0, %1}, pa;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Whether any of the `threads` threads at named barrier `id` has pred.
__device__ __forceinline__ bool bar_any(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

#define FP4IDX_R8(o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
                     "=r"(r[o + 6]), "=r"(r[o + 7])
// 16 lanes x 8 * kBlocks columns: v[4 j + {0, 1}] = (lane l / 4, columns 8 j + 2 (l % 4) +
// {0, 1}), v[4 j + {2, 3}] the same columns of lane l / 4 + 8.  The load and its wait are one
// statement.
template <int kBlocks>
__device__ __forceinline__ void ld_16x256b(uint32_t taddr, float* v) {
  uint32_t r[4 * kBlocks];
  if constexpr (kBlocks == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : FP4IDX_R8(0), FP4IDX_R8(8), FP4IDX_R8(16), FP4IDX_R8(24)
        : "r"(taddr)
        : "memory");
  } else if constexpr (kBlocks == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : FP4IDX_R8(0), FP4IDX_R8(8)
        : "r"(taddr)
        : "memory");
  } else {
    static_assert(kBlocks == 2, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
        : FP4IDX_R8(0)
        : "r"(taddr)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < 4 * kBlocks; i++) v[i] = __uint_as_float(r[i]);
}
// 32 lanes x 16 columns, one lane a thread; the load and its wait are one statement.
__device__ __forceinline__ void ld_32x16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : FP4IDX_R8(0), FP4IDX_R8(8)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
// 32 lanes x 32 columns.
__device__ __forceinline__ void ld_32x32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : FP4IDX_R8(0), FP4IDX_R8(8), FP4IDX_R8(16), FP4IDX_R8(24)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}
// 32 lanes x 56 columns: three loads in flight together, one wait.  (The first load's results
// must not share registers with the others' addresses.)
#define FP4IDX_R8E(o) "=&r"(r[o]), "=&r"(r[o + 1]), "=&r"(r[o + 2]), "=&r"(r[o + 3]), "=&r"(r[o + 4]), "=&r"(r[o + 5]), \
                      "=&r"(r[o + 6]), "=&r"(r[o + 7])
__device__ __forceinline__ void ld_32x56(uint32_t taddr, float* v) {
  uint32_t r[56];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%56];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%57];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%48,%49,%50,%51,%52,%53,%54,%55}, [%58];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : FP4IDX_R8E(0), FP4IDX_R8E(8), FP4IDX_R8E(16), FP4IDX_R8E(24), FP4IDX_R8E(32), FP4IDX_R8E(40), FP4IDX_R8E(48)
      : "r"(taddr), "r"(taddr + 32), "r"(taddr + 48)
      : "memory");
#pragma unroll
  for (int i = 0; i < 56; i++) v[i] = __uint_as_float(r[i]);
}
// 32 lanes x 8 columns.
__device__ __forceinline__ void ld_32x8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : FP4IDX_R8(0)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = __uint_as_float(r[i]);
}
#undef FP4IDX_R8
#undef FP4IDX_R8E
__device__ __forceinline__ void st_32x16(uint32_t taddr, const float* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; i++) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 32 lanes x 28 columns.
__device__ __forceinline__ void st_32x28(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
  ptx::tmem_st8(taddr + 16, v + 16);
  ptx::tmem_st4(taddr + 24, v[24], v[25], v[26], v[27]);
}

}  // namespace mma
}  // namespace fp4idx
