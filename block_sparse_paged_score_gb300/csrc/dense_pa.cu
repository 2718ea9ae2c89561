// dense_pa.cu -- dense grouped-query attention over an MXFP4 paged cache
// (bsp_dense_pa_decode).
//
//   z[r, t] = scale * sum_c 2^(ek[t, c] - 127) sum_{d in c} q[r, d] k4[t, d]
//   o[r, d] = sum_t p[r, t] 2^(ev[t, c(d)] - 127) v4[t, d] / sum_t p[r, t],   p = exp(z)
//
// with k4, v4 the e2m1 values, e the e8m0 bytes of the four 32-dim groups c.
//
// Work.  A unit = (query group, KV head): its rows, q_group tokens times G
// heads, share every byte of the cache; more than 64 rows are cut into units
// that neighbouring CTAs take at the same time (the second finds the bytes in
// L2).  The units' 128-token blocks laid end to end are cut into equal
// shares, one per resident CTA, so ragged batches load every SM alike; a CTA
// finds its share by a prefix sum over the groups' lengths.  A unit that lies
// in one share is written at once; of a unit cut by share borders each CTA
// leaves (m, l, O) in the workspace, and a second kernel joins them (it reads
// a list of cut units, no counters: the workspace carries nothing from call to
// call and the sums' order is fixed).
//
// Both products are tcgen05 MMAs with the block's tokens or V's dims as their 128
// rows and the unit's N = 16, 32 or 64 rows as their columns:
//   z^T = K Q^T      A = K from shared memory, e2m1, block-scaled by the cache's own
//                    e8m0 bytes (K = 32 = one scale group an MMA), B = q; a bf16
//                    query is the sum of two e4m3 parts (see stage_q)
//   O^T += V^T P     A = V^T, f16, from TMEM, B = P, f16, from shared memory
// so that O, N columns of 128 dims, stays in TMEM, and what the warps do per
// block is the exponentials of N rows and the conversion of V, once for all rows.
// V goes to TMEM: through shared memory its f16 tile would be 32 KB written and
// 32 KB read a block, more than a block's time at the memory's rate.
//
// A CTA is a producer warp, which loads blocks by TMA (K unpacked to one byte
// slot a value, the layout the tensor core reads; V packed; scales as they lie)
// and issues all MMAs, and four or eight compute warps.  Thread = token of the
// logits: it takes its exponentials 2^((z - m) qk + kBias) against the row's reference
// m and adds them up (one reduction at the end of the unit); z and m are the MMA's
// sums, the scale qk comes after the difference, so that equal logits of any size have
// equal weights.  References move only when a row's maximum passes its reference by
// kMaxGrow; a vote of the CTA finds
// those blocks, and the ones that some row does not see whole, and takes them
// through an uncommon way that rescales O and l.  Then the warp turns a quarter of
// V's dims into f16: ldmatrix.trans hands a thread four nibbles of two tokens in a
// register, bit moves make f16 pairs of them, times 2^-14 exactly, and a product
// with 2^(byte - kVRef + 14) puts the scale on, exact for bytes kVLow .. kVHigh.
// Blocks with other scales are multiplied in bf16, which holds any v * 2^e, with the
// weights in two bf16 parts (2^-17 off), in two rounds.  Outputs of 2^90 and more
// may overflow on the way.
//
// Roundings: a weight is f16, at most half a step, 2^-11, off, and with a reference
// of 2^kBias f16's range, down to 2^-25, reaches 2^-32 of the row's largest.  z, m,
// l and O are fp32.  The sums l are those of the unrounded weights.
//
// Measured (64 requests x 131072 tokens, 16 rows: 1.14 GB): 226 us, 5.1 TB/s; 128 x
// 32768 with 64 rows: 0.57 GB in 224 to 233 us.  What bounds it is the chain of a block
// through a CTA (wait, logits, vote, exponentials, V's conversion, fences), which four
// CTAs an SM (two of 64 rows) overlap, beside instruction issue: 2 560 warp
// instructions a block of 16 rows, 1 000 of them V's conversion, at 67 % of the
// issue slots; 4 670 of 64 rows, at 61 %.  The tensor cores are 10 and 20 % busy.
// With three CTAs an SM 16 rows took 249 us.  PV on mma.sync, weights and V as
// register fragments, took 289 us and 536 us: V's conversion and the loads of P
// were repeated for every 16 rows.
//
// Every wait for a copy or an MMA is bounded.  After a timed-out wait (the error word
// is set, the results are void) the producer issues nothing more and waits, with a
// limit again, for what it has under way; a compute warp walks through its blocks
// without waits and arrives nowhere, so that the producer stops too.  Then the CTA
// frees its TMEM and returns.
#include <algorithm>
#include <cmath>
#include <type_traits>

// rounds (of up to kSleepNs) before a wait gives up; a build may set fewer, to see what
// a kernel whose waits run out leaves behind
#ifdef BSP_DENSE_PA_WAIT_ROUNDS
#define BSP_WAIT_ROUNDS (BSP_DENSE_PA_WAIT_ROUNDS)
#endif
#include "common.cuh"
#include "dense_work.cuh"
#include "kernels.h"
#include "tc_warp.cuh"
#include "tcgen05.cuh"

namespace bsp {

namespace {

// A field (128 tokens x 64 bytes, then 128 x 4 bytes of scales) comes as one box.
// K: 136 rows of 64 bytes, unpacked to 128; V: 68 rows of 128 bytes.
constexpr int kKRows = 136, kVRows = 68;
constexpr int kKTile = kKRows * 128, kVTile = (kVRows + 7) / 8 * 8 * 128;
static_assert(kKRows * 64 == kMxField && kVRows * 128 == kMxField && kKTile % 1024 == 0);
// V enters the MMA as v * 2^(scale byte - kVRef).  f16 holds that exactly for
// bytes from kVLow to kVHigh (2^-17 to 2^7); see scale_words.

constexpr int kVRef = 133, kVLow = kVRef - 23, kVHigh = kVRef + 1;

// ---- shared memory -----------------------------------------------------------
// Units of 16 rows: four compute warps a CTA, four CTAs an SM; of more: eight, two.
// Then the producer.
template <int N>
struct Shape {
  static constexpr int kCompute = N == 16 ? 4 : 8, kThreads = 32 * (kCompute + 1), kCtasPerSm = N == 16 ? 4 : 2;
  static constexpr int kHalves = kCompute / 4;          // warps that share 32 TMEM lanes
  static constexpr int kRows = N / kHalves;             // a compute warp's
  static constexpr int kTokens = kBlock / kHalves;      // of V
};
template <int N, bool Q16>
struct Smem {
  // (as much as the CTAs of an SM leave room for)
  static constexpr int kCompute = Shape<N>::kCompute;
  static constexpr int kKStages = N == 16 ? 1 : N == 32 ? 3 : 2, kVStages = N == 16 ? 2 : 3;
  static constexpr int kPBytes = kBlock * N * 2;  // P [128 tokens][N rows] f16, two of them
  static constexpr int v = kKStages * kKTile;
  static constexpr int p = v + kVStages * kVTile;
  static constexpr int q = p + 2 * kPBytes;
  static constexpr int scales = q + N * 128 * (Q16 ? 2 : 1);  // per compute warp: a word for two tokens
  static constexpr int refs = scales + kCompute * Shape<N>::kTokens * 2;        // [2][N] -m
  static constexpr int fac = refs + 2 * N * 4;                // [N] rescale factors
  static constexpr int tops = fac + N * 4;                    // [4][N] maxima, later sums
  static constexpr int len = tops + 4 * N * 4;                // [N] lengths
  static constexpr int nan = len + N * 4;                     // [N] 32-dim groups that hold a NaN scale
  static constexpr int sfq = nan + N * 4;                     // [2][N] scale cells of q
  static constexpr int bars = sfq + 2 * N * 4;
  static constexpr int misc = bars + 24 * 8;  // bad[4], TMEM address, commands[2], what is uncommon[2]
  static constexpr int total = misc + 48;
  static_assert(p % 1024 == 0 && q % 1024 == 0 && refs % 16 == 0);
};

// ---- device helpers ------------------------------------------------------------
__device__ __forceinline__ void tile_g2s(uint32_t dst, const CUtensorMap* m, int head, int block, uint32_t bar) {
  asm volatile(
      BSP_ELECT " @e cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
                "[%1, {%2, %3, %4, %5}], [%6];\n}\n" ::"r"(dst),
      "l"(m), "r"(0), "r"(0), "r"(head), "r"(block), "r"(bar)
      : "memory");
}
// 512 bytes (32 rows of 16) to four TMEM columns of every 32-lane sub-partition
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint32_t saddr) {
  uint64_t d = (saddr & 0x3FFFF) >> 4;            // start address
  d |= static_cast<uint64_t>(128 >> 4) << 16;     // leading byte offset (one core matrix wide: unused)
  d |= static_cast<uint64_t>(128 >> 4) << 32;     // 8-row core matrices 128 bytes apart
  d |= static_cast<uint64_t>(1) << 46;            // descriptor version; no swizzle
  asm volatile(BSP_ELECT " @e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(taddr), "l"(d) : "memory");
}
// 16 lanes x 16 columns: register 2j + h of thread t is lane t / 4 + 8h, column 4j + t % 4
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// D (+)= (A * 2^(sa - 127)) (B * 2^(sb - 127)), both in shared memory (see umma_mx)
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
  asm volatile(
      BSP_ELECT " .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                " @e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], "
                "p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// four nibbles of token a (low half) and of token b (high half) -> f16x2
// (a_i, b_i) times 2^-14: sign to bit 15, the three magnitude bits under the exponent
__device__ __forceinline__ void e2m1x4x2_to_f16x2(uint32_t z, uint32_t (&v)[4]) {
  const uint32_t even = ((z << 4) & 0x80808080u) | ((z << 1) & 0x0E0E0E0Eu);
  const uint32_t odd = (z & 0x80808080u) | ((z >> 3) & 0x0E0E0E0Eu);
  v[0] = __byte_perm(even, 0, 0x2404);
  v[1] = __byte_perm(odd, 0, 0x2404);
  v[2] = even & 0xFF00FF00u;
  v[3] = odd & 0xFF00FF00u;
}
// the same as bf16x2, exactly
__device__ __forceinline__ void e2m1x4x2_to_bf16x2(uint32_t z, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = z >> (4 * i);  // the magnitude bits under the exponent: times 2^-126
    v[i] = bmul2(((t & 0x00080008u) << 12) | ((t & 0x00070007u) << 6), 0x7E807E80u);  // times 2^126
  }
}
// x * 2^e for any e (two factors, each a normal float, where one would overflow)
__device__ __forceinline__ float scale_pow2(float x, int e) {
  const int a = max(-126, min(127, e)), b = max(-126, min(127, e - a));
  return x * __uint_as_float(static_cast<uint32_t>(a + 127) << 23) * __uint_as_float(static_cast<uint32_t>(b + 127) << 23);
}

// q of a unit in shared memory as the MMA reads it (rows of 128 e4m3 bytes,
// 128-byte swizzle), with its scale cells: thread = 16-byte chunk j of row n.
// e4m3 queries are copied, scales 1.  Of a bf16 row each 32-dim group is scaled
// by 2^-a, its largest magnitude then in [128, 256), and split: hi = e4m3(x), lo
// = e4m3((x - hi) * 2^4), multiplied by 2^a and 2^(a-4) in the MMAs.  bf16 has 8
// significant bits and each part 4, so the sum is exact for elements down to
// 2^-13 of the group's largest, and off by at most 2^-21 of it below.  A group with an
// infinite element is NaN: the conversions saturate, and every logit of the row is
// infinite or NaN, so the row is NaN either way.
template <bool Q16>
__device__ __noinline__ void stage_q(const DensePaParams& a, int tok0, int tokens, int h, uint8_t* q, int rows,
                                        uint8_t* cells, int tid) {
  const int n = tid >> 3, j = tid & 7;
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  const bool live = n / a.group < tokens;
  const int64_t e = ((tok0 + n / a.group) * hq + static_cast<int64_t>(h) * a.group + n % a.group) * kDim + 16 * j;
  uint8_t* dst = q + n * 128 + ((j ^ (n & 7)) << 4);
  if (!Q16) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + e);
    const uint32_t sign = a.sm_scale < 0.f ? 0x80808080u : 0u;
    *reinterpret_cast<uint4*>(dst) = make_uint4(w.x ^ sign, w.y ^ sign, w.z ^ sign, w.w ^ sign);
    if (!(j & 1)) cells[n * 4 + (j >> 1)] = 127;
    return;
  }
  uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (live) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + e);
    w[0] = src[0], w[1] = src[1];
  }
  const uint32_t ws[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  float x[16], top = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    x[k] = bf16_bits_to_float(k & 1 ? ws[k >> 1] >> 16 : ws[k >> 1] & 0xFFFF);
    if (a.sm_scale < 0.f) x[k] = -x[k];
    top = fmaxf(top, fabsf(x[k]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));  // the group's other chunk
  if (top == INFINITY) {
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(0x7FC00000u);
  }
  const int ex = max(-110, static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127) - 7;
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    uint32_t hb[2], lb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float u = scale_pow2(x[k + 2 * i], -ex), v = scale_pow2(x[k + 2 * i + 1], -ex);
      hb[i] = float2_to_e4m3x2(u, v);
      lb[i] = float2_to_e4m3x2((u - e4m3_to_float(hb[i])) * 16.f, (v - e4m3_to_float(hb[i] >> 8)) * 16.f);
    }
    hi[k >> 2] = hb[0] | (hb[1] << 16);
    lo[k >> 2] = lb[0] | (lb[1] << 16);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(dst + rows * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  if (!(j & 1)) {
    cells[n * 4 + (j >> 1)] = static_cast<uint8_t>(ex + 127);
    cells[(rows + n) * 4 + (j >> 1)] = static_cast<uint8_t>(ex + 123);
  }
}

// ---- pieces of a compute warp's block -------------------------------------------
// The cells of V's scales of a lane's two tokens, at `cell`, and of the two 64 tokens
// on (i = 64): two rows of 128 bytes on, where a chunk's place in its row turns by two
__device__ __forceinline__ uint2 scale_cells(uint32_t cell, int i) { return lds64(i ? (cell + 256) ^ 32 : cell); }
// The pair of factors that put_v multiplies the lane's two tokens by, f16
// 2^(byte - kVRef + 14), to the warp's words.  Returns whether f16 holds
// v * 2^(byte - kVRef) exactly for both (and then the words are right).
__device__ __forceinline__ bool scale_words(uint32_t cell, uint32_t word_at, uint32_t pick, int i) {
  constexpr uint32_t k2 = 0x00010001u;
  const uint2 c = scale_cells(cell, i);
  const uint32_t b = __byte_perm(c.x, c.y, pick) & 0x00FF00FFu;
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(word_at + 2 * i), "r"((b - (kVLow - 6) * k2) << 10) : "memory");
  const uint32_t low = b + (512 - kVLow) * k2, high = b + (512 - kVHigh - 1) * k2;  // bit 9: not below, above
  return (low & ~high & (512 * k2)) == 512 * k2;
}
// The same with care: factors 0 for tokens at or behind max_len, and for groups of
// zeros, which may have any scale below the range.
__device__ __noinline__ bool scale_words_exact(uint32_t cell, int n, int max_len, uint32_t word_at, uint32_t vt,
                                               int tok, int quad, int i) {
  const uint2 c = scale_cells(cell, i);
  uint32_t word = 0;
  bool in = true;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (n + i + k >= max_len) continue;
    const uint32_t b = (k ? c.y : c.x) >> (8 * quad) & 0xFF;
    if (b >= kVLow && b <= kVHigh) {
      word |= (b - (kVLow - 6)) << (10 + 16 * k);
    } else {
      const int r = (tok + i) >> 1;
      const uint4 v = lds128(vt + r * 128 + (((k * 4 + quad) ^ (r & 7)) << 4));
      in &= b < kVLow && ((v.x | v.y | v.z | v.w) & 0x77777777u) == 0;
    }
  }
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(word_at + 2 * i), "r"(word) : "memory");
  return in;
}
// The factors for bf16, 2^(byte - kVRef), over f16's (for any byte but the NaN's,
// whose tokens count as 0 here); which rows see a NaN in the group.
__device__ __noinline__ void wide_words(uint32_t cell, int n, int max_len, uint32_t word_at, int quad, int i,
                                        const int* lens, uint32_t* nan_of, int rows) {
  const uint2 c = scale_cells(cell, i);
  uint32_t word = 0;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const uint32_t b = (k ? c.y : c.x) >> (8 * quad) & 0xFF;
    if (n + i + k >= max_len) continue;
    if (b == 255) {
      for (int r = 0; r < rows; ++r)
        if (n + i + k < lens[r]) atomicOr(nan_of + r, 1u << quad);
    } else {
      word |= (b > kVRef - 127 ? (b - (kVRef - 127)) << 7 : 1u << b) << (16 * k);
    }
  }
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(word_at + 2 * i), "r"(word) : "memory");
}

// z - m of CH rows
template <int CH>
__device__ __forceinline__ void load_logits(float2 (&x)[CH / 2], uint32_t zt, uint32_t refs) {
  float z[CH];
  tmem_ld<CH>(zt, z);
#pragma unroll
  for (int i = 0; i < CH / 4; ++i) {
    const float4 m = lds128f(refs + 16 * i);
    x[2 * i] = fadd2({z[4 * i], z[4 * i + 1]}, {m.x, m.y});
    x[2 * i + 1] = fadd2({z[4 * i + 2], z[4 * i + 3]}, {m.z, m.w});
  }
}
template <int CH>
__device__ __forceinline__ void mask_logits(float2 (&x)[CH / 2], int n, uint32_t lens) {
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {
    if (n >= static_cast<int>(lds32(lens + 8 * i))) x[i].x = -INFINITY;
    if (n >= static_cast<int>(lds32(lens + 8 * i + 4))) x[i].y = -INFINITY;
  }
}

// V of TOKENS tokens and the warp's 32 dims to TMEM: lane = dim, column = two tokens.
// ldmatrix.trans hands thread t four nibbles (dims 4 (t / 4) + i) of tokens 2 (t % 4)
// and + 1 of each 8: dim 4 r + i goes to lane 8 i + r, which the 16x128b stores want.
template <bool BF16, int TOKENS>
__device__ __forceinline__ void put_v(uint32_t vt, uint32_t ld_at, uint32_t words) {
#pragma unroll
  for (int k = 0; k < TOKENS / 32; ++k) {
    uint32_t z[4], lo[8], hi[8];
    ldsm_x4_trans(z, ld_at + k * 2048);
    const uint4 s4 = lds128(words + (k >> 1) * 128 + (k & 1) * 16);
    const uint32_t s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[4];
      if (BF16) {
        e2m1x4x2_to_bf16x2(z[j], v);
        lo[2 * j] = bmul2(v[0], s[j]), lo[2 * j + 1] = bmul2(v[1], s[j]);
        hi[2 * j] = bmul2(v[2], s[j]), hi[2 * j + 1] = bmul2(v[3], s[j]);
      } else {
        e2m1x4x2_to_f16x2(z[j], v);
        lo[2 * j] = hmul2(v[0], s[j]), lo[2 * j + 1] = hmul2(v[1], s[j]);
        hi[2 * j] = hmul2(v[2], s[j]), hi[2 * j + 1] = hmul2(v[3], s[j]);
      }
    }
    tmem_st_16x128(vt + 16 * k, lo);
    tmem_st_16x128(vt + 16 * k + (16u << 16), hi);
  }
}

// ---- the main kernel -----------------------------------------------------------
// barriers, by their byte offset in shared memory
template <int N, bool Q16>
struct Bars {
  static constexpr int NK = Smem<N, Q16>::kKStages, NV = Smem<N, Q16>::kVStages;
  static constexpr int k_full = Smem<N, Q16>::bars, k_empty = k_full + 8 * NK, v_full = k_empty + 8 * NK,
                       v_empty = v_full + 8 * NV,  // v_full: V is loaded, and the block's logits are there
                       z_empty = v_empty + 8 * NV,
                       pv_full = z_empty + 16,  // P and V's tile are written
      pv_done = pv_full + 16,                   // and multiplied
      q_full = pv_done + 16;
  static_assert(q_full + 8 <= Smem<N, Q16>::misc);
};

// TMEM columns: V's tiles (64 columns of token pairs), O, the logits, the scale
// cells of K and q
template <int N, bool Q16>
struct Tmem {
  static constexpr int kV = N == 32 ? 2 : 1, kZ = N == 64 ? 1 : 2;  // buffers
  static constexpr int v = 0, o = v + kV * 64, z = o + N, k = z + kZ * N, q = k + 4 * Smem<N, Q16>::kKStages;
  static constexpr int kColumns = N == 16 ? 128 : 256;
  static_assert(q + 8 <= kColumns && kColumns * Shape<N>::kCtasPerSm <= 512);
};
// what a PV round is
constexpr uint32_t kAccumulate = 1, kBf16 = 2, kMore = 4, kNothing = 8;
constexpr uint32_t kWide = 1, kSkip = 2;

template <int N, bool Q16>
__global__ void __launch_bounds__(Shape<N>::kThreads, Shape<N>::kCtasPerSm)
    dense_pa_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const __grid_constant__ Params p) {
  using S = Smem<N, Q16>;
  using T = Tmem<N, Q16>;
  constexpr int kCompute = Shape<N>::kCompute, kThreads = Shape<N>::kThreads;
  extern __shared__ __align__(1024) uint8_t smem[];  // (all of it: no static shared memory moves its start)
  // before the first block P's place serves the scan
  int64_t* s_sum = reinterpret_cast<int64_t*>(smem + S::p);  // [warps]
  int64_t* s_start = s_sum + kThreads / 32;  // the share's first group, the blocks before it, its blocks
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + S::misc);
  const DensePaParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform, and known to be)
  using B = Bars<N, Q16>;
  const uint32_t base = smem_u32(smem);
  if (tid == 0) {
    auto init = [&](int at, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + at) + i, count);
    };
    init(B::k_full, S::kKStages, 1), init(B::k_empty, S::kKStages, 1);
    init(B::v_full, S::kVStages, 2), init(B::v_empty, S::kVStages, kCompute);
    init(B::z_empty, 2, kCompute);
    init(B::pv_full, 2, kCompute), init(B::pv_done, 2, 1);
    init(B::q_full, 1, 4);
    misc[7] = misc[8] = 0;
    mbar_fence_init();
  }
  pdl_wait();
  // TMEM only after the wait: a CTA that held columns while it waited could
  // keep the kernel before it from getting its own.  And the next kernel's CTAs
  // come (at the trigger below) only once this one has got its columns.
  if (warp == kCompute) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     base + S::misc + 16),
                 "n"(T::kColumns));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  const int sub = blockIdx.x % p.subs, turn = blockIdx.x / p.subs;
  const Share sh = find_share<kThreads>(p, turn, s_sum, s_start);
  const int64_t share = sh.share;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  pdl_trigger();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[4], 0);
  Walk w = walk_of(p, sh, s_start);
  __syncthreads();  // the scan's place is P's again
  // cut units: (first CTA, pieces) per unit, or (unit, pieces) per first CTA
  int2* cut = reinterpret_cast<int2*>(a.ws);
  if (!p.by_unit && tid == 0) cut[blockIdx.x] = make_int2(0, 0);
  bool alive = true;

  if (warp == kCompute) {
    // ---- producer ----
    // It walks the share, reads the block table, 32 entries at a time, loads, and
    // issues all MMAs.  K is loaded kAhead blocks ahead of the MMAs, V kAheadV: a
    // block less than its stages would hold, so that waiting for a stage does not
    // hold up the next MMAs.
    // (One warp does all of it, and its code is out of the instruction cache
    // most of the time: what counts here is few instructions.)
    constexpr int kAheadV = S::kVStages - 2, kAhead = S::kKStages;
    static_assert(kAheadV <= kAhead);
    const uint32_t k_full = base + B::k_full, k_empty = base + B::k_empty, v_full = base + B::v_full;
    const uint32_t v_empty = base + B::v_empty, z_empty = base + B::z_empty;
    const uint32_t q_full = base + B::q_full, bad_at = base + S::misc;
    const uint64_t k_desc = smem_desc_sw128(base), q_desc = smem_desc_sw128(base + S::q);
    const int limit = static_cast<int>(min(a.num_blocks, int64_t{0x7FFFFFFF}));
    const int bad_id = max(limit, 1);  // outside the map, which has a block at least: its copies write zeros
    // scales of tokens 32j + lane in K's unpacked rows 128..: 16 tokens a row, two an
    // 8-byte piece, each piece in a 16-byte chunk at j ^ (row % 8)
    uint32_t from[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tok = 32 * j + lane, row = tok >> 4;
      from[j] = base + (128 + row) * 128 + ((((tok & 15) >> 1) ^ (row & 7)) << 4) + (tok & 1) * 4;
    }
    const int32_t* table = nullptr;
    int left = 0, at_id = 32, head = 0;  // blocks left of the piece, the next one's lane in ids
    int32_t ids = 0;
    bool done = false;
    // the next blocks to be multiplied: id (kNone: none) and head (~head: the first of its piece)
    constexpr int kNone = -1;
    int q_id[kAhead + 1], q_head[kAhead + 1];
    uint32_t vst = 0, v_phase = 1;  // of the next V load (an empty stage's wait passes at once)
    uint32_t kst = 0, k_phase = 1;  // of the next K load
    uint32_t mst = 0, m_phase = 0, z_phase = 1, q_phase = 0, buf = 0, sst = 0;  // of the next MMAs
    auto learn = [&](int& id, int& hd) {  // the next block of the share
      hd = head;
      if (__builtin_expect(left == 0, 0)) {
        while (left == 0 && !done) {
          done = !w.next(p, sub, lane);
          if (!done) {
            table = a.block_table + static_cast<int64_t>(w.seq) * a.bt_stride + w.b0;
            left = w.nblk, at_id = 32, head = w.h;
          }
        }
        id = kNone, hd = ~head;
        if (done) return;
      }
      if (__builtin_expect(at_id == 32, 0)) {
        ids = lane < left ? table[lane] : 0;
        if (static_cast<uint32_t>(ids) >= static_cast<uint32_t>(limit)) {
          set_err(a.err, BSP_DEVERR_BLOCK_ID);
          ids = bad_id;
        }
        table += 32, at_id = 0;
      }
      id = __shfl_sync(0xffffffffu, ids, at_id);
      ++at_id, --left;
    };
    // (a wait that gives up ends the loop: nothing is issued after it)
    auto ready = [&](uint32_t bar, uint32_t parity) { return alive = wait_warp(bar, parity, a.err); };
    auto load_v = [&](int id, int hd) {
      if (!ready(v_empty + 8 * vst, v_phase)) return;
      const uint32_t bar = v_full + 8 * vst;
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(bad_at + 4 * vst), "r"(static_cast<uint32_t>(id == bad_id)) : "memory");
      __syncwarp();
      arrive_expect(bar, kMxField);
      tile_g2s(base + S::v + vst * kVTile, &map_v, hd ^ (hd >> 31), id, bar);
      if (++vst == S::kVStages) vst = 0, v_phase ^= 1;
    };
    auto load_k = [&](int id, int hd) {
      if (!ready(k_empty + 8 * kst, k_phase)) return;
      const uint32_t bar = k_full + 8 * kst;
      arrive_expect(bar, kMxField);
      tile_g2s(base + kst * kKTile, &map_k, hd ^ (hd >> 31), id, bar);
      if (++kst == S::kKStages) kst = 0, k_phase ^= 1;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      learn(q_id[i], q_head[i]);
      if (q_id[i] != kNone) {  // (these stages are empty: no wait gives up)
        load_k(q_id[i], q_head[i]);
        if (i < kAheadV) load_v(q_id[i], q_head[i]);
      }
    }
    // O += V^T P of the next block, in a round, or in two (kMore)
    uint64_t p_desc = ((base + S::p) & 0x3FFFF) >> 4;
    // P: rows of 2N bytes, one atom of the 2N-byte swizzle wide, 8 tokens an atom
    p_desc |= static_cast<uint64_t>(1) << 16;                                // leading offset: unused
    p_desc |= static_cast<uint64_t>(8 * 2 * N >> 4) << 32;                   // 8 tokens
    p_desc |= static_cast<uint64_t>(1) << 46;                                // descriptor version
    p_desc |= static_cast<uint64_t>(N == 16 ? 6 : N == 32 ? 4 : 2) << 61;    // 32-, 64-, 128-byte swizzle
    uint32_t round = 0;
    auto multiply = [&]() {
      uint32_t cmd = kMore;
      while (cmd & kMore) {
        const uint32_t b = round & 1;
        if (!ready(base + B::pv_full + 8 * b, (round >> 1) & 1)) return;
        cmd = misc[5 + b];
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        // f32 += A (f16 or bf16, TMEM) B (the same, rows contiguous), M = 128
        const uint32_t id = (1u << 4) | (1u << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24) |
                            (cmd & kBf16 ? (1u << 7) | (1u << 10) : 0);
        const uint32_t v = tmem + T::v + (T::kV == 2 ? b * 64 : 0);
        if (!(cmd & kNothing)) {
#pragma unroll
          for (int k = 0; k < kBlock / 16; ++k)
            umma_ts(tmem + T::o, v + 8 * k, p_desc + (b * S::kPBytes + k * 16 * 2 * N) / 16, id,
                    k > 0 || (cmd & kAccumulate));
        }
        commit(base + B::pv_done + 8 * b);
        ++round;
      }
    };
    int behind = 0;  // blocks whose logits are under way and whose PV is not
#pragma unroll 1
    while (q_id[0] != kNone) {
      learn(q_id[kAhead], q_head[kAhead]);
      // PV of the block before the last; of all of them before another piece's q,
      // which comes once the piece's O has been read
      while (alive && behind > (q_head[0] < 0 ? 0 : 1)) {
        multiply();
        --behind;
      }
      if (!alive) break;
      ++behind;
      // K is there: its scales from token order to the cells tcgen05.cp reads,
      // lane i of column j = token 32j + i
      if (!ready(k_full + 8 * mst, m_phase)) break;
      const uint32_t off = mst * kKTile, cells = base + off + kBlock * 128;  // (in their own rows)
      const uint32_t cell[4] = {lds32(from[0] + off), lds32(from[1] + off), lds32(from[2] + off), lds32(from[3] + off)};
      __syncwarp();
      sts128(cells + lane * 16, cell[0], cell[1], cell[2], cell[3]);
      fence_proxy_async();
      __syncwarp();
      if (__builtin_expect(q_head[0] < 0, 0)) {
        if (!ready(q_full, q_phase)) break;
        q_phase ^= 1;
      }
      if (!ready(z_empty + 8 * buf, z_phase)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t sk = tmem + T::k + 4 * mst, z = tmem + T::z + buf * N;
      const uint64_t kd = k_desc + mst * (kKTile / 16);
      scales_to_tmem(sk, cells);
#pragma unroll
      for (int part = 0; part < (Q16 ? 2 : 1); ++part)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          umma_ss(z, kd + 2 * c, q_desc + (part * N * 128 + 32 * c) / 16,
                  idesc_mxf8f6f4(kFmtE2m1, kFmtE4m3, N, 128, c, c), sk, tmem + T::q + 4 * part,
                  part > 0 || c > 0);
      commit(k_empty + 8 * mst);
      commit(v_full + 8 * sst);
      if (++sst == S::kVStages) sst = 0;
      if (++mst == S::kKStages) mst = 0, m_phase ^= 1;
      if (++buf == T::kZ) buf = 0, z_phase ^= 1;
      if (q_id[kAheadV] != kNone) load_v(q_id[kAheadV], q_head[kAheadV]);  // once the compute warps have left its stage
      if (!alive) break;
      if (q_id[kAhead] != kNone) load_k(q_id[kAhead], q_head[kAhead]);  // once the MMAs that used it are done
      if (!alive) break;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) q_id[j] = q_id[j + 1], q_head[j] = q_head[j + 1];
      __syncwarp();
    }
    while (alive && behind-- > 0) multiply();
    // Nothing may still write shared memory or TMEM when the CTA leaves.
    auto settle = [&](uint32_t bar, uint32_t parity) { wait_warp(bar, parity, a.err, kSleepWaitLimit); };
    if (round) settle(base + B::pv_done + 8 * ((round - 1) & 1), ((round - 1) >> 1) & 1);
    if (__builtin_expect(!alive, 0)) {
      // What a healthy end has waited for by now: the round before, the copies (a stage's
      // last load is of this turn of the ring below the next load's, of the last turn
      // from there on) and the commits of the logits.
      if (round > 1) settle(base + B::pv_done + 8 * (round & 1), ((round - 2) >> 1) & 1);
      // V's barriers take a copy and a commit a block; one of the two may have come alone
      if (vst != sst) {
        if (kAheadV > 0) {  // a block's V that no logits follow
          commit(v_full + 8 * sst);
        } else {  // logits that no V follows
          if (lane == 0) arrive(v_full + 8 * vst);
          if (++vst == S::kVStages) vst = 0, v_phase ^= 1;
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < S::kVStages; ++i) settle(v_full + 8 * i, i < vst ? v_phase ^ 1 : v_phase);
#pragma unroll
      for (uint32_t i = 0; i < S::kKStages; ++i) {
        settle(k_full + 8 * i, i < kst ? k_phase ^ 1 : k_phase);
        settle(k_empty + 8 * i, i < mst ? m_phase : m_phase ^ 1);
      }
    }
    __syncwarp();
  } else {
    // ---- compute ----
    // Warp: TMEM lanes 32 * quad .., that is the logits of the block's tokens
    // 32 * quad .. and O's dims of 32-dim group quad; R rows of both.  Of V it takes
    // that group of VT tokens.
    constexpr int R = Shape<N>::kRows, CH = 16, VT = Shape<N>::kTokens;  // rows of a warp, and of them at a time
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t tops = base + S::tops, lens_at = base + S::len, fac = base + S::fac;
    int* lens = reinterpret_cast<int*>(smem + S::len);
    uint32_t* nan_of = reinterpret_cast<uint32_t*>(smem + S::nan);
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t z_at = tmem + lane_base + T::z + half * R, o_at = tmem + lane_base + T::o + half * R;
    const uint32_t vt_at = tmem + lane_base + T::v + half * (VT / 2);
    const uint32_t z_empty = base + B::z_empty, v_full = base + B::v_full;
    const uint32_t v_empty = base + B::v_empty, pv_full = base + B::pv_full, pv_done = base + B::pv_done;
    const uint32_t bad_at = base + S::misc, flags = base + S::misc + 28;  // V beyond f16; a bad block
    // scales of V: the lane's tokens vtok, vtok + 1 (and 64 further on); their cells,
    // in row 64 + token / 32
    const int vtok = VT * half + 2 * lane;
    const uint32_t cell_at = base + S::v + (64 + (vtok >> 5)) * 128 + ((((vtok & 31) >> 2) ^ (vtok >> 5)) << 4) +
                             (vtok & 3) * 4;
    const uint32_t pick = quad | (4 + quad) << 8;  // byte quad of two cells, to bytes 0 and 2
    const uint32_t words = base + S::scales + warp * VT * 2;
    const uint32_t word_at = words + ((lane & 3) * 8 + (lane >> 2)) * 4, my_words = words + (lane & 3) * 32;
    // the lane's row for ldmatrix: token VT * half + lane (+ 32 k), two tokens a row of 128 bytes
    const int vrow = VT / 2 * half + (lane >> 1);
    const uint32_t ld_at = base + S::v + vrow * 128 + ((((lane & 1) * 4 + quad) ^ (vrow & 7)) << 4);
    // the lane's token in P
    const int tok = 32 * quad + lane;
    const uint32_t swz = (tok & 7) >> (N == 16 ? 2 : N == 32 ? 1 : 0);
    const uint32_t p_at = base + S::p + tok * 2 * N;
    uint32_t zb = 0, vst = 0, v_phase = 0;  // of the next block
    uint32_t round = 0;                                  // of PV
    uint32_t cur = 0;                                    // which reference maxima
    auto done = [&](uint32_t r) {  // round r - 1 has ended
      if (r && alive) alive = wait_warp(pv_done + 8 * ((r - 1) & 1), ((r - 1) >> 1) & 1, a.err);
    };
    while (w.next(p, sub, lane)) {
      bar_sync(1, 32 * kCompute);  // the last unit's q, lengths and sums are no longer read
      if (w.nblk)
        for (int i = tid; i < N * 8; i += 32 * kCompute)
          stage_q<Q16>(a, w.tok0, w.tokens, w.h, smem + S::q, N, smem + S::sfq, i);
      if (tid < N) {
        const int j = tid / a.group;
        // (rows that no token has see what the longest sees: they must not look uncommon)
        lens[tid] = j < w.tokens ? min(max(a.row_len[static_cast<int64_t>(w.tok0 + j) * a.hkv + w.h], 0), w.max_len)
                                 : w.max_len;
        nan_of[tid] = 0;
        stsf(base + S::refs + (cur * N + tid) * 4, -kNoMax);
      }
      if (tid < w.tokens && a.row_seq[static_cast<int64_t>(w.tok0 + tid) * a.hkv + w.h] != w.seq)
        set_err(a.err, BSP_DEVERR_GROUP_SEQ);
      float2 l[R / 2];  // of the lane's token in every block
#pragma unroll
      for (int i = 0; i < R / 2; ++i) l[i] = make_float2(0.f, 0.f);
      fence_proxy_async();  // the tensor core reads q through the async proxy
      bar_sync(1, 32 * kCompute);
      if (w.nblk && half == 0) {
#pragma unroll
        for (int k = 0; k < (Q16 ? 2 : 1); ++k) {  // q's scale cells, in this sub-partition's copy
          const uint32_t* c = reinterpret_cast<const uint32_t*>(smem + S::sfq) + k * N;
          tmem_st4(tmem + lane_base + T::q + 4 * k, lane < N ? c[lane] : 0x7F7F7F7Fu,
                   32 + lane < N ? c[32 + lane] : 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0 && alive) arrive(base + B::q_full);
      }
      bool first = true;  // no PV round of the unit yet
      const int max_len = w.max_len, min_len = w.min_len;
      int n0 = w.b0 * kBlock;  // at most 2^31 - 128 in the loop
#pragma unroll 1
      for (int k = w.nblk; k > 0; --k, n0 = static_cast<int>(n0 + static_cast<uint32_t>(kBlock))) {
        // after a timed-out wait the warp goes on without waits and arrivals (the
        // barriers of the compute warps need every one); its results are void
        if (alive) alive = wait_warp(v_full + 8 * vst, v_phase, a.err);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const bool bad = lds32(bad_at + 4 * vst) != 0, whole = n0 <= min_len - kBlock;
        const uint32_t z = z_at + zb * N, voff = vst * kVTile;
        auto exact = [&]() {
          bool in = true;
#pragma unroll 1
          for (int i = 0; i < VT; i += 64)
            in &= scale_words_exact(cell_at + voff, n0 + vtok, max_len, word_at, base + S::v + voff, vtok, quad, i);
          return in;
        };
        // one PV round: the weights (of bf16 ones part 0 or 1) and V's tile
        auto send = [&](auto wide, int part) {
          const uint32_t b = round & 1;
          // P and V's tile are free: of two the round before the last, which used
          // them, has ended; with one tile the wait below for the last round was that
          // for P's sake too
          if (T::kV == 2) done(round < 2 ? 0 : round - 1);
#pragma unroll
          for (int c = 0; c < R; c += CH) {
            float2 x[CH / 2];  // (read again rather than held: registers)
            load_logits<CH>(x, z + c, base + S::refs + (cur * N + half * R + c) * 4);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) x[i] = ffma2(x[i], {p.qk_scale, p.qk_scale}, {kBias, kBias});
            if (!whole) mask_logits<CH>(x, n0 + tok, lens_at + (half * R + c) * 4);
            uint32_t pk[CH / 2];
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              const float2 e = make_float2(ex2_approx(x[i].x), ex2_approx(x[i].y));
              if (!wide) {
                l[c / 2 + i] = fadd2(l[c / 2 + i], e);
                pk[i] = pack_f16x2(e.x, e.y);
              } else {
                pk[i] = pack_bf16x2(e.x, e.y);
                if (part == 0)
                  l[c / 2 + i] = fadd2(l[c / 2 + i], e);
                else
                  pk[i] = pack_bf16x2(e.x - bf16_bits_to_float(pk[i] & 0xFFFF), e.y - bf16_bits_to_float(pk[i] >> 16));
              }
            }
#pragma unroll
            for (int i = 0; i < CH / 8; ++i)
              sts128(p_at + b * S::kPBytes + (((half * R + c) / 8 + i) ^ swz) * 16, pk[4 * i], pk[4 * i + 1],
                     pk[4 * i + 2], pk[4 * i + 3]);
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();  // the logits are read, V's factors written
          if ((!wide || part) && lane == 0 && alive) arrive(z_empty + 8 * zb);
          if (T::kV == 1) done(round);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          put_v<wide, VT>(vt_at + (T::kV == 2 ? b * 64 : 0), ld_at + voff, my_words);
          if (tid == 0) misc[5 + b] = (first ? 0 : kAccumulate) | (wide ? kBf16 | (part ? 0 : kMore) : 0);
          first = false;
          fence_proxy_async();  // the tensor core reads P through the async proxy
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0 && alive) arrive(pv_full + 8 * b);
          ++round;
        };
        // V's factors
        bool in = true;
#pragma unroll
        for (int i = 0; i < VT; i += 64) in &= scale_words(cell_at + voff, word_at, pick, i);
        if (__builtin_expect(!in || !whole, 0)) in = exact();
        if (__builtin_expect(bad || !in, 0))
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(flags + (bad ? 4 : 0)), "r"(1u) : "memory");
        __syncwarp();  // (lanes differ in `in`; the loads and the vote below are the whole warp's)
        // first pass: does a row's maximum grow?
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < R; c += CH) {
          float2 x[CH / 2];
          load_logits<CH>(x, z + c, base + S::refs + (cur * N + half * R + c) * 4);
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) top = fmax3(top, x[i].x, x[i].y);
        }
        uint32_t mode = 0;  // kWide: V in bf16; kSkip: a block whose id is out of range
        if (__builtin_expect(!all_of<32 * kCompute>(!bad && whole && in && top * p.qk_scale <= kMaxGrow), 0)) {
          // The uncommon way: the rows' maxima, where a row may not see the
          // token, new references, and O and l in their terms; are V's scales
          // outside f16's range?
          const bool skip = lds32(flags + 4) != 0, wide = !skip && lds32(flags) != 0;
          mode = skip ? kSkip : wide ? kWide : 0;
          if (!skip) {
#pragma unroll 1
            for (int c = 0; c < R; c += CH) {
              float y[CH];
              tmem_ld<CH>(z + c, y);
              if (!whole) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                  if (n0 + tok >= static_cast<int>(lds32(lens_at + (half * R + c + i) * 4))) y[i] = -INFINITY;
              }
              const float mx = warp_reduce<CH>(y, lane, [](float u, float v) { return fmaxf(u, v); });
              if (!(lane & 1)) stsf(tops + (quad * N + half * R + c + (lane >> 1)) * 4, mx);
              __syncwarp();
            }
          }
          bar_sync(1, 32 * kCompute);
          float f = 1.f;
          if (tid == 0 && mode) misc[7] = misc[8] = 0;  // (every warp has read them, and sets none before the next vote)
          if (tid < N && !skip) {
            float mx = ldsf(tops + tid * 4);
#pragma unroll
            for (int i = 1; i < 4; ++i) mx = fmaxf(mx, ldsf(tops + (i * N + tid) * 4));
            const float old = -ldsf(base + S::refs + (cur * N + tid) * 4);
            const float ref = mx > old ? mx : old;  // (every row: fewer such blocks to come)
            f = rescale(old, ref, p.qk_scale);
            stsf(base + S::refs + ((cur ^ 1) * N + tid) * 4, -ref);
            stsf(fac + tid * 4, f);
          }
          if (!skip) cur ^= 1;
          if (any_of<32 * kCompute>(f != 1.f) && !first) {
            done(round);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
            for (int c = 0; c < R; c += CH) {
              float y[CH];
              tmem_ld<CH>(o_at + c, y);
#pragma unroll
              for (int i = 0; i < CH; ++i) {
                const float g = ldsf(fac + (half * R + c + i) * 4);
                y[i] *= g;
                (i & 1 ? l[(c + i) >> 1].y : l[(c + i) >> 1].x) *= g;
              }
              tmem_st<CH>(o_at + c, y);
            }
          }
          if (wide)
#pragma unroll 1
            for (int i = 0; i < VT; i += 64)
              wide_words(cell_at + voff, n0 + vtok, max_len, word_at, quad, i, lens, nan_of, N);
          __syncwarp();  // (its lanes' ways differ)
        }
        // second pass: the weights, and V as the MMA reads it.  Where V's scales
        // are beyond f16, both are bf16 and the weights go in two parts.
        if (__builtin_expect(mode == 0, 1)) {
          send(std::false_type{}, 0);
        } else if (mode == kWide) {
#pragma unroll 1
          for (int part = 0; part < 2; ++part) send(std::true_type{}, part);
        } else {
          done(round);
          if (tid == 0) misc[5 + (round & 1)] = kNothing;
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0 && alive) arrive(z_empty + 8 * zb), arrive(pv_full + 8 * (round & 1));
          ++round;
        }
        __syncwarp();
        if (lane == 0 && alive) arrive(v_empty + 8 * vst);
        if (++zb == T::kZ) zb = 0;
        if (++vst == S::kVStages) vst = 0, v_phase ^= 1;
      }

      // -- the unit's sums, and O to where it goes
#pragma unroll
      for (int c = 0; c < R; c += CH) {
        float y[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) y[i] = i & 1 ? l[(c + i) >> 1].y : l[(c + i) >> 1].x;
        const float sum = warp_reduce<CH>(y, lane, [](float u, float v) { return u + v; });
        if (!(lane & 1)) stsf(tops + (quad * N + half * R + c + (lane >> 1)) * 4, sum);
      }
      bar_sync(1, 32 * kCompute);
      const bool all = w.starts && w.ends;
      // a CTA's slots: 2 * CTA for a unit that began before its share, + 1 for one
      // that goes on after it
      float* po = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + list_bytes(p.ctas)) +
                  (2LL * blockIdx.x + (w.starts ? 1 : 0)) * N * (kDim + 2);
      const int rows = w.tokens * a.group;
      if (tid < N) {  // what O is multiplied by: V's 2^(kVRef - 127), over the sum
        const float sum = (ldsf(tops + tid * 4) + ldsf(tops + (N + tid) * 4)) +
                          (ldsf(tops + (2 * N + tid) * 4) + ldsf(tops + (3 * N + tid) * 4));
        stsf(fac + tid * 4, static_cast<float>(1 << (kVRef - 127)) * (!all ? 1.f : sum == 0.f ? 0.f : 1.f / sum));
        if (!all && tid < rows)
          *reinterpret_cast<float2*>(po + N * kDim + 2 * tid) =
              make_float2(-ldsf(base + S::refs + (cur * N + tid) * 4), sum);
      }
      bar_sync(1, 32 * kCompute);
      if (!first) done(round);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int d = 32 * quad + 4 * (lane & 7) + (lane >> 3);  // the lane's dim (see put_v)
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                           (static_cast<int64_t>(w.tok0) * a.hkv + w.h) * a.group * kDim + d;
      const int64_t hop = static_cast<int64_t>(a.hkv - 1) * a.group * kDim;  // from a token's rows to the next's
      int in_token = (half * R) % a.group;
      out += (half * R) / a.group * hop + half * R * kDim;
#pragma unroll 1
      for (int c = 0; c < R; c += 8) {
        float y[8];
        if (!first) {
          tmem_ld<8>(o_at + c, y);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = half * R + c + i;
          if (r < rows) {
            const float o = lds32(base + S::nan + r * 4) >> quad & 1 ? __uint_as_float(0x7FC00000u) : y[i] * ldsf(fac + r * 4);
            if (all) {
              *out = __float2bfloat16_rn(o);
              out += kDim;
              if (++in_token == a.group) in_token = 0, out += hop;
            } else {
              po[r * kDim + d] = o;
            }
          }
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      if (w.starts && tid == 0) {
        // the pieces of the unit: shares from this one to that of its last block
        const int64_t last = w.c0 * a.hkv + static_cast<int64_t>(w.h + 1) * w.nb - 1;
        const int pieces = w.ends ? 0 : static_cast<int>(last / share) - turn + 1;
        if (p.by_unit)
          cut[w.unit] = make_int2(blockIdx.x, pieces);
        else if (pieces)
          cut[blockIdx.x] = make_int2(w.unit, pieces);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kCompute) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(T::kColumns));
  }
}

// ---- host ------------------------------------------------------------------------
// One side of the cache as [blocks][heads][rows][row].  K: a row is a token's 128
// 4-bit values, unpacked to 16-byte slots of 16; V: 128 bytes, two tokens (half
// the rows for the copy engine to fetch).  128-byte swizzle.
bool make_map_side(CUtensorMap* m, bool unpack, const void* base, uint64_t heads, uint64_t blocks, uint64_t stride) {
  auto fn = encode_fn();
  if (!fn) return false;
  const uint32_t rows = unpack ? kKRows : kVRows;
  const cuuint64_t dims[4] = {128, rows, heads, blocks};
  const cuuint64_t strides[3] = {unpack ? 64u : 128u, kMxField, stride};
  const cuuint32_t box[4] = {128, rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, unpack ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// How a group's rows are cut into units of at most 64, and the rows the kernel is
// built for.  128 requests of 32768 tokens, us, units of at most 16, 32 and 64 rows:
// 32 rows a group 220, 187, 186; 64 rows 413, 348, 231; 128 rows 803, 673, 418; a
// group of 32 rows in the kernel for 64: 223.
Plan plan_of(int group, int q_group) {
  const int sub = std::min(q_group, 64 / group), subs = (q_group + sub - 1) / sub;
  const int tokens = (q_group + subs - 1) / subs, rows = tokens * group;  // units of about the same size
  if (rows <= 16) return {tokens, subs, 16, Shape<16>::kCtasPerSm};
  if (rows <= 32) return {tokens, subs, 32, Shape<32>::kCtasPerSm};
  return {tokens, subs, 64, Shape<64>::kCtasPerSm};
}

template <int N, bool Q16>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, cudaStream_t s) {
  using S = Smem<N, Q16>;
  static_assert((S::total + 1024) * Shape<N>::kCtasPerSm <= 228 * 1024);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {  // the shared-memory opt-in
    return cudaFuncSetAttribute(dense_pa_kernel<N, Q16>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::total);
  });
  if (e != cudaSuccess) return e;
  return launch_kernel(dense_pa_kernel<N, Q16>, dim3(static_cast<unsigned>(p.ctas)), dim3(Shape<N>::kThreads), S::total, s, 0, mk,
                       mv, p);
}

}  // namespace

size_t dense_pa_ws_bytes(int32_t num_rows, int32_t hkv, int32_t group, int32_t q_group, int num_sms) {
  (void)num_rows, (void)hkv;
  const Plan pl = plan_of(group, q_group);
  const int64_t ctas = static_cast<int64_t>(pl.ctas_per_sm) * num_sms;
  return list_bytes(ctas) + 2 * ctas * pl.rows * (kDim + 2) * sizeof(float);
}

cudaError_t launch_dense_pa(const DensePaParams& a, int num_sms, cudaStream_t s, int* launches) {
  if (a.num_rows == 0) return cudaSuccess;
  const Plan pl = plan_of(a.group, a.q_group);
  const bool q16 = a.q_dtype == BSP_BF16;
  Params p{};
  p.a = a;
  p.qk_scale = std::fabs(a.sm_scale) * kLog2e;
  set_work(p, pl, num_sms);
  CUtensorMap mk, mv;
  const uint64_t blocks = std::max<int64_t>(a.num_blocks, 1);
  if (!make_map_side(&mk, true, a.k_base, a.hkv, blocks, a.id_stride) ||
      !make_map_side(&mv, false, a.v_base, a.hkv, blocks, a.id_stride))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (pl.rows == 16)
    e = q16 ? launch_main<16, true>(mk, mv, p, s) : launch_main<16, false>(mk, mv, p, s);
  else if (pl.rows == 32)
    e = q16 ? launch_main<32, true>(mk, mv, p, s) : launch_main<32, false>(mk, mv, p, s);
  else
    e = q16 ? launch_main<64, true>(mk, mv, p, s) : launch_main<64, false>(mk, mv, p, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if ((e = launch_join(p, s, launches)) != cudaSuccess) return e;
  return cudaPeekAtLastError();
}

}  // namespace bsp
