// tc_warp.cuh -- what the warp-specialised tcgen05 attention kernels share: barriers,
// copies and MMAs issued by one elected lane of a converged warp, bounded waits, TMEM
// rows, packed fp32 arithmetic and the rescaling of softmax sums.
#pragma once

#include "common.cuh"

// rounds (of up to kSleepNs) before a wait gives up
#ifndef BSP_WAIT_ROUNDS
#define BSP_WAIT_ROUNDS kSleepWaitLimit
#endif

namespace bsp {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoMax = -3.402823466e38f;  // the maximum of no keys (finite: -inf - kNoMax stays -inf)

// The producer warp runs converged and one lane of it, always the same, issues:
// with a branch around each issue the descriptors would be vector registers,
// moved to uniform ones one by one (765 clocks for the eight MMAs of a block).
#define BSP_ELECT "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
// C fp32 columns of the warp's 32 TMEM lanes, and back
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[C]) {
  static_assert(C == 8 || C == 16);
  uint32_t r[C];
  if constexpr (C == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = __uint_as_float(r[i]);
}
template <int C>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[C]) {
#pragma unroll
  for (int i = 0; i < C; i += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr + i),
                 "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]), "f"(v[i + 6]),
                 "f"(v[i + 7])
                 : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 words a lane (no wait)
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// D (+)= A B: A [128][16] in TMEM (two 16-bit values a column), B in shared memory
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      BSP_ELECT " .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 lds128f(uint32_t addr) {
  const uint4 v = lds128(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void stsf(uint32_t addr, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ float ldsf(uint32_t addr) { return __uint_as_float(lds32(addr)); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// barrier of the compute warps that returns whether every / any thread says so
template <int THREADS>
__device__ __forceinline__ bool all_of(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "n"(THREADS)
      : "memory");
  return r != 0;
}
template <int THREADS>
__device__ __forceinline__ bool any_of(bool x) {
  return !all_of<THREADS>(!x);
}
// mbarriers and copies by shared address
__device__ __forceinline__ void arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile(BSP_ELECT " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(BSP_ELECT
               " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kSleepNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, int32_t* err, uint32_t rounds) {
#pragma unroll 1
  for (uint32_t i = 0; i < rounds; ++i)
    if (try_wait(bar, parity)) return true;
  set_err(err, BSP_DEVERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// A converged warp waits, with one answer for all of its lanes, and comes out
// converged (what follows are .aligned loads, stores and barriers).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int32_t* err,
                                          uint32_t rounds = BSP_WAIT_ROUNDS) {
  if (__builtin_expect(__all_sync(0xffffffffu, test_wait(bar, parity)), 1)) return true;
  return __all_sync(0xffffffffu, wait_slow(bar, parity, err, rounds));
}
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t x, y, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
// what a sum with the reference `from` is multiplied by to have the reference `to` >= from
__device__ __forceinline__ float rescale(float from, float to, float qk) {
  return ex2_approx(fminf((from - to) * qk, 0.f));  // (NaN, of a scale of 0: 0)
}
// x times that, in two steps where the factor itself is below fp32's range
__device__ __forceinline__ float rescaled(float x, float from, float to, float qk) {
  const float f = rescale(from, to, qk);
  if (f != 0.f) return x * f;
  const float half = ex2_approx(fminf((from - to) * qk, 0.f) * 0.5f);
  return x * half * half;
}
// R values of each lane reduced over the warp, all of them at once: each step hands
// half of the values to the lane that differs in one bit.  Lane i ends with value
// i * R / 32 (of R = 16, lanes 2j and 2j + 1 both with value j).
template <int R, typename OP>
__device__ __forceinline__ float warp_reduce(float (&x)[R], int lane, OP op) {
  static_assert(R == 16 || R == 32);
#pragma unroll
  for (int h = R / 2, d = 16; h >= 1; h >>= 1, d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float mine = up ? x[i + h] : x[i], theirs = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + h], d);
      x[i] = op(mine, theirs);
    }
  }
  return R == 32 ? x[0] : op(x[0], __shfl_xor_sync(0xffffffffu, x[0], 1));
}

}  // namespace bsp
