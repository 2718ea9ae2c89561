// dense_pa.cu -- dense grouped-query attention over an MXFP4 paged cache
// (bsp_dense_pa_decode).
//
//   z[r, t] = scale * sum_c 2^(ek[t, c] - 127) sum_{d in c} q[r, d] k4[t, d]
//   o[r, d] = sum_t p[r, t] 2^(ev[t, c(d)] - 127) v4[t, d] / sum_t p[r, t],   p = exp(z)
//
// with k4, v4 the e2m1 values, e the e8m0 bytes of the four 32-dim groups c.
//
// Work.  A unit = (query group, KV head, at most 64 rows): its rows, tokens
// times G heads, share every byte of the cache.  The units' 128-token blocks
// laid end to end are cut into equal shares, one per resident CTA, so ragged
// batches load every SM alike; a CTA finds its share by a prefix sum over the
// groups' lengths.  A unit that lies in one share is written at once; of a
// unit cut by share borders each CTA leaves (m, l, O) in the workspace, and a
// second kernel joins them (it reads a list of cut units, no counters: the
// workspace carries nothing from call to call and the sums' order is fixed).
//
// A CTA is one producer warp and 4 * sets compute warps; each set has 16 rows.
//   - The producer loads blocks by TMA (K unpacked to one byte slot a value,
//     the layout the tensor core reads; V packed, 64-byte swizzle; the scales
//     as they lie) and issues, per block, four tcgen05.mma block-scaled by the
//     cache's own e8m0 bytes: z^T = K Q^T, M = 128 tokens, N = 16 * sets rows,
//     K = 32 = one scale group each, in TMEM, double-buffered.  Row 32j + i of
//     the tile is token 4i + j (a tensor-map order): then the 512 scale bytes
//     are, as they lie in the cache, the cells tcgen05.cp wants.  A bf16 query is
//     the sum of two e4m3 parts (see stage_q), eight MMAs.
//   - A compute warp reads 32 tokens x 16 rows of z^T (thread = token), takes
//     the exponentials, turns the f16 weights around through shared memory
//     into mma A fragments and multiplies by V: mma.sync m16n8k16 f16.  V
//     comes through ldmatrix.trans as four nibbles of two tokens a register;
//     bit moves turn them into f16 pairs, times 2^-14 exactly.  V's scales go
//     onto P: 2^(ev - R_c), a power of two at most 1, multiplies the weights of
//     each group.  R_c is the largest scale byte so far (O is rescaled when it
//     grows).  Tokens whose scale is 15 or more binades below R_c, which f16
//     could not hold, make the warp take its tokens again in bands of 15.
//   - p is f16, at most half a step, 2^-11, off; weights are kept times 2^7 so
//     that f16's range, down to 2^-25, reaches 2^-32 of the largest.
// tcgen05 takes the scores because it reads e2m1 and the scales itself: on
// mma.sync the conversions of K cost more issue slots than all else.  PV stays
// on mma.sync: with V^T as A its dequantised tile would have to go through
// shared memory, 32 KB written and read a block, more than a block's time at
// the memory's rate.
//
// Every wait is bounded; after a timed-out wait a role waits no more (the
// error word is set) and the CTA frees its TMEM and returns.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace bsp {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxRows = 64;       // rows of a unit
constexpr int kKStages = 2, kVStages = 3;
constexpr int kKTile = kBlock * 128;  // unpacked keys of a block
constexpr int kVTile = kBlock * 64;   // packed values of a block
constexpr int kRowPad = kDim + 4;  // floats of a row in the merge buffer
constexpr float kMaxGrow = 8.f;    // the reference maximum moves when a row's maximum grows by more (log2)
constexpr float kBias = 7.f;       // weights are 2^(z - m + kBias)
constexpr float kNoMax = -1e30f;   // the maximum of no tokens (finite: -inf - kNoMax stays -inf)
constexpr int kBand = 15;          // binades a band of V scales spans
constexpr int kQueue = 8;          // blocks the producer knows ahead

// bytes of the list of cut units at the start of the workspace
__host__ __device__ constexpr int64_t list_bytes(int64_t ctas) { return (ctas * 8 + 255) / 256 * 256; }

struct Params {
  DensePaParams a;
  float qk_scale;  // sm_scale * log2(e)
  int32_t groups, subs, sub_tokens;  // query groups; units a group and head is cut into, of sub_tokens tokens
  int32_t units, ctas;
  int32_t by_unit;  // the list of cut units has an entry per unit (else per CTA)
};

// ---- shared memory -----------------------------------------------------------
// per compute warp: P [32 tokens][16 rows] f16, V's scales [4][16 pairs] f16x2,
// reference maxima and rescale factors of 16 rows; the sets' merge buffers
// take the same place once a unit's blocks are done
constexpr int kScratch = 1024 + 256 + 64 + 64;
template <int SETS>
struct Smem {
  static constexpr int kCompute = 4 * SETS;
  static constexpr int kThreads = 32 * (kCompute + 1);
  static constexpr int kRows = 16 * SETS;
  static constexpr int kMerge = 16 * kRowPad * 4 + 128;  // a set's O, m, l
  static constexpr int v = kKStages * kKTile;
  static constexpr int ks = v + kVStages * kVTile;  // K scales, with K's stages
  static constexpr int vs = ks + kKStages * 512;
  static constexpr int scratch = vs + kVStages * 512;
  static constexpr int scratch_bytes = std::max(kCompute * kScratch, SETS * kMerge);
  static constexpr int len = scratch + scratch_bytes;  // [rows] lengths
  static constexpr int sfq = len + kRows * 4;          // [2][rows] scale cells of q
  static constexpr int bars = sfq + 2 * kRows * 4;
  static constexpr int queue = bars + 20 * 8;
  static constexpr int q = (queue + kQueue * 8 + 16 + 1023) / 1024 * 1024;
  static constexpr int total(bool q16) { return q + kRows * 128 * (q16 ? 2 : 1) + 1024; }
};

// ---- device helpers ------------------------------------------------------------
__device__ __forceinline__ void tile_g2s(void* dst, const CUtensorMap* m, int head, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(0), "r"(head), "r"(block), "r"(smem_u32(bar))
      : "memory");
}
// 512 bytes (32 rows of 16) to four TMEM columns of every 32-lane sub-partition
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint32_t saddr) {
  uint64_t d = (saddr & 0x3FFFF) >> 4;            // start address
  d |= static_cast<uint64_t>(128 >> 4) << 16;     // leading byte offset (one core matrix wide: unused)
  d |= static_cast<uint64_t>(128 >> 4) << 32;     // 8-row core matrices 128 bytes apart
  d |= static_cast<uint64_t>(1) << 46;            // descriptor version; no swizzle
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float4 lds128f(uint32_t addr) {
  const uint4 v = lds128(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void stsf(uint32_t addr, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ float ldsf(uint32_t addr) { return __uint_as_float(lds32(addr)); }
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(x)) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// mbarriers by shared address
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
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, int32_t* err) {
  for (uint32_t i = 0; i < kSleepWaitLimit; ++i)
    if (try_wait(bar, parity)) return true;
  set_err(err, BSP_DEVERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, int32_t* err) {
  if (__builtin_expect(try_wait(bar, parity), 1)) return true;
  return wait_slow(bar, parity, err);
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
// x * 2^e for any e (two factors, each a normal float, where one would overflow)
__device__ __forceinline__ float scale_pow2(float x, int e) {
  const int a = max(-126, min(127, e)), b = max(-126, min(127, e - a));
  return x * __uint_as_float(static_cast<uint32_t>(a + 127) << 23) * __uint_as_float(static_cast<uint32_t>(b + 127) << 23);
}
// largest of the warp's values
__device__ __forceinline__ float warp_max(float x) {
  const int b = __float_as_int(x), k = b ^ ((b >> 31) & 0x7FFFFFFF);  // ordered as integers
  const int m = __reduce_max_sync(0xffffffffu, k);
  return __int_as_float(m ^ ((m >> 31) & 0x7FFFFFFF));
}

// ---- units ---------------------------------------------------------------------
// blocks of group g: the longest of its rows, at least one (an empty unit
// still writes its zeros)
__device__ __forceinline__ int blocks_of(const DensePaParams& a, int len) {
  return static_cast<int>(max(1u, min((static_cast<uint32_t>(len) + 127u) / 128u, static_cast<uint32_t>(a.bt_stride))));
}
__device__ __forceinline__ int group_len(const DensePaParams& a, int g, int first, int step) {
  const int64_t tok0 = static_cast<int64_t>(g) * a.q_group;
  const int n = static_cast<int>(min(static_cast<int64_t>(a.q_group), a.num_rows / a.hkv - tok0)) * a.hkv;
  int len = 0;
  for (int i = first; i < n; i += step) len = max(len, a.row_len[tok0 * a.hkv + i]);
  return len;
}

// A warp's walk over the pieces of a share [at, end) of the units' blocks.
// Every lane holds the same values.
struct Walk {
  int64_t at, end, c0;  // c0: blocks of the groups before g
  int g, nb;
  // the piece at `at`
  int unit, h, tok0, tokens, seq, b0, b1, max_len, min_len, len;  // len: of the lane's token
  bool starts, ends;  // the unit's first and last blocks are in the piece

  __device__ __forceinline__ bool next(const Params& p, int lane) {
    if (at >= end) return false;
    const DensePaParams& a = p.a;
    const int64_t per = static_cast<int64_t>(a.hkv) * p.subs;
    while ((c0 + nb) * per <= at) {
      c0 += nb;
      ++g;
      nb = blocks_of(a, __reduce_max_sync(0xffffffffu, group_len(a, g, lane, 32)));
    }
    const int x = static_cast<int>((at - c0 * per) / nb);
    const int64_t ustart = c0 * per + static_cast<int64_t>(x) * nb, uend = ustart + nb;
    unit = static_cast<int>(g * per + x);
    h = x / p.subs;
    const int sub = x % p.subs;
    const int gtok = g * a.q_group;
    tok0 = gtok + sub * p.sub_tokens;
    tokens = min(min(p.sub_tokens, a.q_group - sub * p.sub_tokens), a.num_rows / a.hkv - tok0);
    seq = a.row_seq[static_cast<int64_t>(gtok) * a.hkv];
    const int cap = static_cast<int>(min(static_cast<int64_t>(a.bt_stride) * kBlock, int64_t{0x7FFFFFFF}));
    len = 0;
    if (lane < tokens) len = min(max(a.row_len[static_cast<int64_t>(tok0 + lane) * a.hkv + h], 0), cap);
    max_len = __reduce_max_sync(0xffffffffu, len);
    min_len = __reduce_min_sync(0xffffffffu, lane < tokens ? len : 0x7FFFFFFF);
    if (tokens <= 0) max_len = 0;  // the last group may lack this unit's tokens
    b0 = static_cast<int>(at - ustart);
    b1 = min(static_cast<int>(min(end, uend) - ustart), (max_len + 127) >> 7);
    starts = at == ustart, ends = end >= uend;
    at = min(end, uend);
    return true;
  }
};

// q of a unit in shared memory as the MMA reads it (rows of 128 e4m3 bytes,
// 128-byte swizzle), with its scale cells: thread = 16-byte chunk j of row n.
// e4m3 queries are copied, scales 1.  Of a bf16 row each 32-dim group is scaled
// by 2^-a, its largest magnitude then in [128, 256), and split: hi = e4m3(x), lo
// = e4m3((x - hi) * 2^4), multiplied by 2^a and 2^(a-4) in the MMAs.  bf16 has 8
// significant bits and each part 4, so the sum is exact for elements down to
// 2^-13 of the group's largest, and off by at most 2^-21 of it below.
template <bool Q16>
__device__ __forceinline__ void stage_q(const DensePaParams& a, int tok0, int tokens, int h, uint8_t* q, int rows,
                                        uint8_t* cells, int tid) {
  const int n = tid >> 3, j = tid & 7;
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  const bool live = n / a.group < tokens;
  const int64_t e = ((tok0 + n / a.group) * hq + static_cast<int64_t>(h) * a.group + n % a.group) * kDim + 16 * j;
  uint8_t* dst = q + n * 128 + ((j ^ (n & 7)) << 4);
  if (!Q16) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + e);
    *reinterpret_cast<uint4*>(dst) = w;
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
    top = fmaxf(top, fabsf(x[k]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));  // the group's other chunk
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

// one compute warp's running softmax: O of 16 rows in mma accumulators (tile
// 4c + i: dims 32c + 8t + i and 32c + 8t + 4 + i of rows g and g + 8), the sums l
// as a tile of their own (P times ones), and 271 - R_c of groups (0, 2) and (1, 3)
// in the halves of two words
struct State {
  float o[16][4];
  float l[4];
  uint32_t r02, r13;
};
constexpr uint32_t kHalves = 0x00010001u;
constexpr uint32_t kNoScale = 271 * kHalves;  // R_c = 0

// V's scales where some byte is above R_c, zero or 15 binades and more below it:
// raises R_c (O moves to the new unit), writes band `band`'s f16 scales, and says
// whether lower ones are left
__device__ __forceinline__ bool odd_vscales(State& st, uint32_t vw, uint32_t vcell, int band) {
  const uint32_t rr[4] = {271 - (st.r02 & 0xFFFF), 271 - (st.r13 & 0xFFFF), 271 - (st.r02 >> 16), 271 - (st.r13 >> 16)};
  uint32_t now[4];
  bool low = false;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t b = vw >> (8 * c) & 0xFF;
    now[c] = band ? rr[c] : max(rr[c], __reduce_max_sync(0xffffffffu, b));
    if (now[c] != rr[c]) {
      const float f = scale_pow2(1.f, static_cast<int>(rr[c]) - static_cast<int>(now[c]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[4 * c + i][e] *= f;
    }
    const int x = static_cast<int>(b) - static_cast<int>(now[c]) + kBand * band + 15;  // f16 exponent field
    low |= b && x <= 0;
    sts16(vcell + c * 64, b && x > 0 && x <= 15 ? x << 10 : 0);
  }
  st.r02 = kNoScale - (now[0] | (now[2] << 16));
  st.r13 = kNoScale - (now[1] | (now[3] << 16));
  return __any_sync(0xffffffffu, low);
}

// The uncommon half of attend(): a block that some row does not see whole, V
// scales outside R_c's band, or a row whose maximum grew (x then starts afresh
// from the logits, as it does not hold them where the reference was that of no
// tokens).  Returns whether lower bands of V scales are left.
__device__ __forceinline__ bool adjust(State& st, float2 (&x)[8], uint32_t zt, float qk, int n, uint32_t lens,
                                       uint32_t vw, uint32_t vcell, uint32_t scratch, int lane) {
  const uint32_t mp = scratch + 1280, ap = scratch + 1344;
  const bool more = odd_vscales(st, vw, vcell, 0);
  float z[16];
  tmem_ld16(zt, z);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float y = n < static_cast<int>(lds32(lens + 4 * i)) ? z[i] * qk : -INFINITY, mx = warp_max(y);
    const float old = ldsf(mp + 4 * i);  // kBias - m
    const float now = mx > kBias - old + kMaxGrow ? kBias - mx : old;
    (i & 1 ? x[i >> 1].y : x[i >> 1].x) = y + now;
    __syncwarp();  // every lane has the old reference
    if (lane == 0) stsf(ap + 4 * i, ex2_approx(now - old)), stsf(mp + 4 * i, now);
  }
  __syncwarp();
  const float a0 = ldsf(ap + 4 * (lane >> 2)), a1 = ldsf(ap + 4 * (lane >> 2) + 32);
  st.l[0] *= a0, st.l[2] *= a1;
#pragma unroll
  for (int i = 0; i < 16; ++i) st.o[i][0] *= a0, st.o[i][1] *= a0, st.o[i][2] *= a1, st.o[i][3] *= a1;
  return more;
}

// 32 tokens of the warp: their logits are at TMEM address zt (thread = the lane's
// token n, column = row h, which sees the token if n < lens[h]; whole: every row
// sees every token); vw the token's V scale bytes (0 where no row sees it), vt the
// V rows.  Arrives at z_empty once the logits are read.
__device__ __forceinline__ void attend(State& st, uint32_t zt, uint32_t z_empty, float qk, bool whole, int n,
                                       uint32_t lens, uint32_t vw, uint32_t vt, uint32_t scratch, int lane) {
  const uint32_t vp = scratch + 1024, mp = scratch + 1280;
  const int t = lane & 3;
  const uint32_t vcell = vp + ((lane >> 1) & 3) * 16 + (lane >> 3) * 4 + (lane & 1) * 2;  // [c][pair][octet][2]
  // V's scales as f16 2^(byte - R_c): exponent fields 1..15, two groups a word.
  // y = byte + 271 - R_c; in 257..271 where f16 holds the scale.
  const uint32_t y02 = (vw & 0x00FF00FFu) + st.r02, y13 = (vw >> 8 & 0x00FF00FFu) + st.r13;
  const uint32_t over = (y02 + 240 * kHalves) | (y13 + 240 * kHalves);  // bit 9: y >= 272
  const uint32_t in = (y02 + 255 * kHalves) & (y13 + 255 * kHalves);    // bit 9: y >= 257
  // weights: 2^(z - m + kBias), m the rows' reference maxima
  float2 x[8];
  {
    float z[16];
    tmem_ld16(zt, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 m = lds128f(mp + 16 * i);  // kBias - m
      x[2 * i] = ffma2({z[4 * i], z[4 * i + 1]}, {qk, qk}, {m.x, m.y});
      x[2 * i + 1] = ffma2({z[4 * i + 2], z[4 * i + 3]}, {qk, qk}, {m.z, m.w});
    }
  }
  float top = fmaxf(x[0].x, x[0].y);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = fmax3(top, x[i].x, x[i].y);
  const bool plain = whole && top <= kBias + kMaxGrow && (over & (512 * kHalves)) == 0 &&
                     (in & (512 * kHalves)) == 512 * kHalves;
  bool more = false;
  if (__builtin_expect(__all_sync(0xffffffffu, plain), 1)) {
    const uint32_t h02 = (y02 - 256 * kHalves) << 10, h13 = (y13 - 256 * kHalves) << 10;
    sts16(vcell, h02), sts16(vcell + 64, h13);
    sts16(vcell + 128, h02 >> 16), sts16(vcell + 192, h13 >> 16);
  } else {
    more = adjust(st, x, zt, qk, n, lens, vw, vcell, scratch, lane);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  uint32_t pk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) pk[i] = pack_f16x2(ex2_approx(x[i].x), ex2_approx(x[i].y));
  // [token][16 rows]; the halves of rows 4..7 of each 8 swap places (banks)
  const uint32_t prow = scratch + lane * 32, flip = (lane & 4) << 2;
  sts128(prow + flip, pk[0], pk[1], pk[2], pk[3]);
  sts128(prow + (16 ^ flip), pk[4], pk[5], pk[6], pk[7]);
  __syncwarp();
  if (lane == 0) arrive(z_empty);
  uint32_t pa[4], pb[4];  // rows g / g + 8, tokens 8o + 2t, + 1
  const int row8 = lane & 7, mat = lane >> 3;
  {
    // matrices: octet 2k, 2k + 1 x row halves
    const uint32_t at = scratch + ((mat >> 1) * 8 + row8) * 32 + (((mat & 1) << 4) ^ ((row8 & 4) << 2));
    uint32_t r[4];
    ldsm_x4_trans(r, at);
    pa[0] = r[0], pb[0] = r[1], pa[1] = r[2], pb[1] = r[3];
    ldsm_x4_trans(r, at + 512);
    pa[2] = r[0], pb[2] = r[1], pa[3] = r[2], pb[3] = r[3];
  }
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
    mma_f16(st.l, pa[2 * ks], pb[2 * ks], pa[2 * ks + 1], pb[2 * ks + 1], 0x3C003C00u, 0x3C003C00u);

  // -- O += P V
  const int swz = (row8 >> 1) & 3;
  const uint32_t vrow = vt + (mat * 8 + row8) * 64;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t zr[4];
    ldsm_x4_trans(zr, vrow + ((c ^ swz) << 4));
    const uint4 s4 = lds128(vp + c * 64 + t * 16);
    const uint32_t vs[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint32_t v0[4], v1[4];
      e2m1x4x2_to_f16x2(zr[2 * ks], v0);
      e2m1x4x2_to_f16x2(zr[2 * ks + 1], v1);
      const uint32_t a0 = hmul2(pa[2 * ks], vs[2 * ks]), a1 = hmul2(pb[2 * ks], vs[2 * ks]);
      const uint32_t a2 = hmul2(pa[2 * ks + 1], vs[2 * ks + 1]), a3 = hmul2(pb[2 * ks + 1], vs[2 * ks + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mma_f16(st.o[4 * c + i], a0, a1, a2, a3, v0[i], v1[i]);
    }
  }
  for (int band = 1; __builtin_expect(more, 0); ++band) {  // the lower bands of V's scales
    __syncwarp();
    more = odd_vscales(st, vw, vcell, band);
    __syncwarp();
    const float f = scale_pow2(1.f, -kBand * band);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t zr[4];
      ldsm_x4_trans(zr, vrow + ((c ^ swz) << 4));
      const uint4 s4 = lds128(vp + c * 64 + t * 16);
      const uint32_t vs[4] = {s4.x, s4.y, s4.z, s4.w};
      float y[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t v0[4], v1[4];
        e2m1x4x2_to_f16x2(zr[2 * ks], v0);
        e2m1x4x2_to_f16x2(zr[2 * ks + 1], v1);
        const uint32_t a0 = hmul2(pa[2 * ks], vs[2 * ks]), a1 = hmul2(pb[2 * ks], vs[2 * ks]);
        const uint32_t a2 = hmul2(pa[2 * ks + 1], vs[2 * ks + 1]), a3 = hmul2(pb[2 * ks + 1], vs[2 * ks + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_f16(y[i], a0, a1, a2, a3, v0[i], v1[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[4 * c + i][e] += y[i][e] * f;
    }
  }
}

// ---- the main kernel -----------------------------------------------------------
template <int SETS>
struct Bars {
  uint64_t* b;
  __device__ uint64_t* k_full(int i) const { return b + i; }
  __device__ uint64_t* k_empty(int i) const { return b + kKStages + i; }
  __device__ uint64_t* v_full(int i) const { return b + 2 * kKStages + i; }
  __device__ uint64_t* v_empty(int i) const { return b + 2 * kKStages + kVStages + i; }
  __device__ uint64_t* z_full(int i) const { return b + 2 * kKStages + 2 * kVStages + i; }
  __device__ uint64_t* z_empty(int i) const { return b + 2 * kKStages + 2 * kVStages + 2 + i; }
  __device__ uint64_t* q_full() const { return b + 2 * kKStages + 2 * kVStages + 4; }
};

template <int SETS>
constexpr int min_ctas() {
  return SETS == 1 ? 3 : 1;
}
// TMEM columns: two z buffers, the scale cells of K (per stage) and q
template <int SETS>
struct Tmem {
  static constexpr int z = 0, sk = 32 * SETS, sq = sk + 4 * kKStages, used = sq + 8;
  static constexpr int columns = used <= 64 ? 64 : (used <= 128 ? 128 : 256);
};

template <int SETS, bool Q16>
__global__ void __launch_bounds__(Smem<SETS>::kThreads, min_ctas<SETS>())
    dense_pa_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const __grid_constant__ Params p) {
  using S = Smem<SETS>;
  using T = Tmem<SETS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_sum[17];
  __shared__ int64_t s_start[2];  // the share's first group and the blocks before it
  __shared__ int s_nb;
  __shared__ uint32_t s_tmem;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  const DensePaParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Bars<SETS> bars{reinterpret_cast<uint64_t*>(smem + S::bars)};
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) mbar_init(bars.k_full(i), 1), mbar_init(bars.k_empty(i), 1);
    for (int i = 0; i < kVStages; ++i) mbar_init(bars.v_full(i), 1), mbar_init(bars.v_empty(i), S::kCompute);
    for (int i = 0; i < 2; ++i) mbar_init(bars.z_full(i), 1), mbar_init(bars.z_empty(i), S::kCompute);
    mbar_init(bars.q_full(), S::kCompute);
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();
  // TMEM only after the wait: a CTA that held columns while it waited could
  // keep the kernel before it from getting its own
  if (warp == S::kCompute) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "n"(T::columns));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  // the groups' blocks, kThreads groups at a time: first their sum, then the
  // group the share starts in
  const int64_t per = static_cast<int64_t>(a.hkv) * p.subs;
  int64_t total = 0, at = 0, share = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t base = 0;
    for (int g0 = 0; g0 < p.groups; g0 += S::kThreads) {
      const int g = g0 + tid;
      const int nb = g < p.groups ? blocks_of(a, group_len(a, g, 0, 1)) : 0;
      int64_t x = nb;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = x;
      __syncthreads();
      int64_t before = base;
      for (int w = 0; w <= S::kCompute; ++w) {
        if (w < warp) before += s_sum[w];
        base += s_sum[w];
      }
      const int64_t c1 = before + x, c0 = c1 - nb;  // blocks before and up to group g
      if (pass == 0 && p.groups <= S::kThreads) {  // one tile: the sum and the start at once
        total = base;
        share = (total * per + p.ctas - 1) / p.ctas;
        at = blockIdx.x * share;
      }
      if ((pass == 1 || p.groups <= S::kThreads) && nb && c0 * per <= at && at < c1 * per)
        s_start[0] = g, s_start[1] = c0, s_nb = nb;
      if (pass == 1 && base * per > at) break;
    }
    if (pass == 0) {
      total = base;
      share = (total * per + p.ctas - 1) / p.ctas;
      at = blockIdx.x * share;
      if (p.groups <= S::kThreads) break;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  Walk w;
  w.at = at, w.end = min(at + share, total * per);
  w.g = static_cast<int>(s_start[0]), w.c0 = s_start[1], w.nb = s_nb;  // unset, and unused, past the last share
  // cut units: (first CTA, pieces) per unit, or (unit, pieces) per first CTA
  int2* cut = reinterpret_cast<int2*>(a.ws);
  if (!p.by_unit && tid == 0) cut[blockIdx.x] = make_int2(0, 0);
  volatile uint32_t* bad = reinterpret_cast<volatile uint32_t*>(smem + S::queue + kQueue * 8);  // per V stage
  bool alive = true;

  if (warp == S::kCompute) {
    // ---- producer ----
    struct Block {
      int32_t id, head;  // head < 0: ~head, the first block of a piece
    };
    volatile Block* queue = reinterpret_cast<volatile Block*>(smem + S::queue);
    const int32_t* table = nullptr;
    int nblk = 0, blk = 0, chunk = 0, head = 0;
    int32_t ids = 0;
    bool done = false, first = false;
    int known = 0;  // blocks in the queue so far
    auto learn = [&]() {  // the next block of the share; false at its end
      while (!done && blk == nblk) {
        if (!w.next(p, lane)) {
          done = true;
          break;
        }
        table = a.block_table + static_cast<int64_t>(w.seq) * a.bt_stride + w.b0;
        nblk = max(0, w.b1 - w.b0), blk = 0, chunk = -1, head = w.h, first = true;
      }
      if (done) return false;
      if ((blk >> 5) != chunk) {
        chunk = blk >> 5;
        ids = 32 * chunk + lane < nblk ? table[32 * chunk + lane] : 0;
      }
      int32_t id = __shfl_sync(0xffffffffu, ids, blk & 31);
      if (id < 0 || id >= a.num_blocks) {
        if (lane == 0) set_err(a.err, BSP_DEVERR_BLOCK_ID);
        id = -1;
      }
      if (lane == 0) queue[known % kQueue].id = id, queue[known % kQueue].head = first ? ~head : head;
      first = false;
      ++blk, ++known;
      return true;
    };
    // a bad block's stages complete without data; the compute warps leave it out
    auto load_k = [&](int i) {
      const int st = i % kKStages;
      const int32_t id = queue[i % kQueue].id, hh = queue[i % kQueue].head, h = hh < 0 ? ~hh : hh;
      if (id < 0) return mbar_arrive(bars.k_full(st));
      mbar_arrive_expect_tx(bars.k_full(st), kBlock * 64 + 512);
      tile_g2s(smem + st * kKTile, &map_k, h, id, bars.k_full(st));
      bulk_g2s(smem + S::ks + st * 512,
               a.k_base + static_cast<int64_t>(id) * a.id_stride + static_cast<int64_t>(h) * kMxField + kMxScaleOff, 512,
               bars.k_full(st));
    };
    auto load_v = [&](int i) {
      const int st = i % kVStages;
      const int32_t id = queue[i % kQueue].id, hh = queue[i % kQueue].head, h = hh < 0 ? ~hh : hh;
      bad[st] = id < 0;
      if (id < 0) return mbar_arrive(bars.v_full(st));
      mbar_arrive_expect_tx(bars.v_full(st), kVTile + 512);
      tile_g2s(smem + S::v + st * kVTile, &map_v, h, id, bars.v_full(st));
      bulk_g2s(smem + S::vs + st * 512,
               a.v_base + static_cast<int64_t>(id) * a.id_stride + static_cast<int64_t>(h) * kMxField + kMxScaleOff, 512,
               bars.v_full(st));
    };
    // ahead of block 0: V of two blocks, K of one
    for (int i = 0; i < 2; ++i)
      if (learn() && lane == 0) load_v(i);
    if (known > 0 && lane == 0) load_k(0);
    const uint32_t q_addr = smem_u32(smem + S::q);
    int pieces = 0;
    for (int i = 0; i < known; ++i) {
      const bool more = learn();  // block i + 2
      if (lane == 0) {
        const int st = i % kKStages, buf = i & 1;
        const int32_t id = queue[i % kQueue].id;
        if (queue[i % kQueue].head < 0) {
          if (alive) alive = mbar_wait_sleep(bars.q_full(), pieces & 1, a.err);
          ++pieces;
        }
        if (alive && i + 1 < known) {  // K of the next block, once block i - 1's MMAs have left its stage
          if (i > 0) alive = mbar_wait_sleep(bars.k_empty((i + 1) % kKStages), ((i - 1) / kKStages) & 1, a.err);
          if (alive) load_k(i + 1);
        }
        if (alive) alive = mbar_wait_sleep(bars.k_full(st), (i / kKStages) & 1, a.err);
        if (alive && i > 1) alive = mbar_wait_sleep(bars.z_empty(buf), ((i >> 1) - 1) & 1, a.err);
        if (alive) {
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (id >= 0) {
            const uint32_t k_addr = smem_u32(smem + st * kKTile), sk = tmem + T::sk + 4 * st;
            scales_to_tmem(sk, smem_u32(smem + S::ks + st * 512));
#pragma unroll
            for (int part = 0; part < (Q16 ? 2 : 1); ++part)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                umma_mx(tmem + T::z + buf * S::kRows, smem_desc_sw128(k_addr + 32 * c),
                        smem_desc_sw128(q_addr + part * S::kRows * 128 + 32 * c),
                        idesc_mxf8f6f4(kFmtE2m1, kFmtE4m3, S::kRows, 128, c, c), sk, tmem + T::sq + 4 * part,
                        part > 0 || c > 0);
          }
          umma_commit(bars.k_empty(st));
          umma_commit(bars.z_full(buf));
          if (more) {  // V of block i + 2, once the compute warps have left its stage
            if (i + 2 >= kVStages)
              alive = mbar_wait_sleep(bars.v_empty((i + 2) % kVStages), ((i + 2) / kVStages - 1) & 1, a.err);
            if (alive) {
              fence_proxy_async();
              load_v(i + 2);
            }
          }
        }
      }
      __syncwarp();
    }
    // nothing may still be writing shared memory or TMEM when the CTA leaves
    if (lane == 0 && alive && known > 0)
      mbar_wait_sleep(bars.k_empty((known - 1) % kKStages), ((known - 1) / kKStages) & 1, a.err);
    __syncwarp();
  } else {
    // ---- compute ----
    const int set = warp >> 2, part = warp & 3;
    const uint32_t scratch = smem_u32(smem + S::scratch) + warp * kScratch;
    const uint32_t merge = smem_u32(smem + S::scratch) + set * S::kMerge;
    int* lens = reinterpret_cast<int*>(smem + S::len);
    uint8_t* cells = smem + S::sfq;
    const uint32_t lane_base = static_cast<uint32_t>(32 * part) << 16;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t z_full = smem_u32(bars.z_full(0)), z_empty = smem_u32(bars.z_empty(0));
    const uint32_t v_full = smem_u32(bars.v_full(0)), v_empty = smem_u32(bars.v_empty(0));
    const uint32_t bad_at = smem_u32(const_cast<const uint32_t*>(bad)), z_at = tmem + lane_base + T::z + 16 * set;
    const uint32_t vs_at = smem_u32(smem + S::vs) + lane * 16 + part * 4, v_at = smem_u32(smem + S::v) + part * 2048;
    uint32_t buf = 0, z_phase = 0, vst = 0, v_phase = 0;  // of the next block
    while (w.next(p, lane)) {
      const int nblk = max(0, w.b1 - w.b0);
      bar_sync(1, 32 * S::kCompute);  // the last unit's q, lengths and merge buffers are no longer read
      if (nblk) stage_q<Q16>(a, w.tok0, w.tokens, w.h, smem + S::q, S::kRows, cells, tid);
      if (tid < S::kRows) {
        const int j = tid / a.group;
        lens[tid] = j < w.tokens ? min(max(a.row_len[static_cast<int64_t>(w.tok0 + j) * a.hkv + w.h], 0), w.max_len) : 0;
      }
      if (tid == 0)
        for (int j = 0; j < w.tokens; ++j)
          if (a.row_seq[static_cast<int64_t>(w.tok0 + j) * a.hkv + w.h] != w.seq) set_err(a.err, BSP_DEVERR_GROUP_SEQ);
      State st;
#pragma unroll
      for (int k = 0; k < 16; ++k) st.o[k][0] = st.o[k][1] = st.o[k][2] = st.o[k][3] = 0.f;
      st.l[0] = st.l[1] = st.l[2] = st.l[3] = 0.f;
      st.r02 = st.r13 = kNoScale;
      if (lane < 16) stsf(scratch + 1280 + 4 * lane, kBias - kNoMax);
      fence_proxy_async();  // the tensor core reads q through the async proxy
      bar_sync(1, 32 * S::kCompute);
      if (nblk) {
        if (set == 0) {  // q's scale cells, in this sub-partition's copy
#pragma unroll
          for (int k = 0; k < (Q16 ? 2 : 1); ++k) {
            uint32_t cell[2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
              cell[c] = 32 * c + lane < S::kRows
                            ? *reinterpret_cast<const uint32_t*>(cells + (k * S::kRows + 32 * c + lane) * 4)
                            : 0x7F7F7F7Fu;
            tmem_st4(tmem + lane_base + T::sq + 4 * k, cell[0], cell[1], 0x7F7F7F7Fu, 0x7F7F7F7Fu);
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.q_full());
      }
      const uint32_t lens_at = smem_u32(lens + 16 * set);
      int n = w.b0 * kBlock + 4 * lane + part;  // the lane's token
      const int n_whole = w.min_len - (kBlock - 1) + (4 * lane + part);  // blocks up to here are whole for every row
      for (int k = 0; k < nblk; ++k, n += kBlock) {
        // one test of both barriers: V is there before z is
        if (alive) alive = wait_for(z_full + 8 * buf, z_phase, a.err) && wait_for(v_full + 8 * vst, v_phase, a.err);
        alive = __all_sync(0xffffffffu, alive);  // the rest is warp-wide
        if (!alive) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (lds32(bad_at + 4 * vst) == 0) {
          uint32_t vw = lds32(vs_at + vst * 512);
          if (n >= w.max_len) vw = 0;
          attend(st, z_at + buf * S::kRows, z_empty + 8 * buf, p.qk_scale, n < n_whole, n, lens_at, vw,
                 v_at + vst * kVTile, scratch, lane);
        } else if (lane == 0) {
          arrive(z_empty + 8 * buf);
        }
        __syncwarp();
        if (lane == 0) arrive(v_empty + 8 * vst);
        buf ^= 1, z_phase ^= buf ^ 1;
        if (++vst == kVStages) vst = 0, v_phase ^= 1;
      }

      // -- the four warps of a set joined: 1, 2, 3 hand theirs to 0 in turn
      float m0 = kBias - ldsf(scratch + 1280 + 4 * g), m1 = kBias - ldsf(scratch + 1280 + 4 * (g + 8));
      float l0 = st.l[0], l1 = st.l[2];  // every column of the tile is the sum
      const uint32_t rr[4] = {271 - (st.r02 & 0xFFFF), 271 - (st.r13 & 0xFFFF), 271 - (st.r02 >> 16),
                              271 - (st.r13 >> 16)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = static_cast<int>(rr[c]) - 127 + 14;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) st.o[4 * c + k][j] = scale_pow2(st.o[4 * c + k][j], e);
      }
      bar_sync(1, 32 * S::kCompute);  // the scratch becomes the merge buffers
      const uint32_t mrow = merge + (g * kRowPad + 8 * t) * 4, mml = merge + 16 * kRowPad * 4;
      for (int k = 1; k < 4; ++k) {
        if (part == k) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                sts128(mrow + (8 * e * kRowPad + 32 * c + 4 * j) * 4, __float_as_uint(st.o[4 * c][2 * e + j]),
                       __float_as_uint(st.o[4 * c + 1][2 * e + j]), __float_as_uint(st.o[4 * c + 2][2 * e + j]),
                       __float_as_uint(st.o[4 * c + 3][2 * e + j]));
          if (t == 0) {
            stsf(mml + 8 * g, m0), stsf(mml + 8 * g + 4, l0);
            stsf(mml + 8 * (g + 8), m1), stsf(mml + 8 * (g + 8) + 4, l1);
          }
        }
        bar_sync(2 + set, 128);
        if (part == 0) {
          const float n0 = ldsf(mml + 8 * g), n1 = ldsf(mml + 8 * (g + 8));
          const float M0 = fmaxf(m0, n0), M1 = fmaxf(m1, n1);
          const float f0 = ex2_approx(m0 - M0), f1 = ex2_approx(m1 - M1), h0 = ex2_approx(n0 - M0), h1 = ex2_approx(n1 - M1);
          l0 = l0 * f0 + h0 * ldsf(mml + 8 * g + 4);
          l1 = l1 * f1 + h1 * ldsf(mml + 8 * (g + 8) + 4);
          m0 = M0, m1 = M1;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float4 y = lds128f(mrow + (8 * e * kRowPad + 32 * c + 4 * j) * 4);
                const float f = e ? f1 : f0, hh = e ? h1 : h0;
                st.o[4 * c][2 * e + j] = st.o[4 * c][2 * e + j] * f + y.x * hh;
                st.o[4 * c + 1][2 * e + j] = st.o[4 * c + 1][2 * e + j] * f + y.y * hh;
                st.o[4 * c + 2][2 * e + j] = st.o[4 * c + 2][2 * e + j] * f + y.z * hh;
                st.o[4 * c + 3][2 * e + j] = st.o[4 * c + 3][2 * e + j] * f + y.w * hh;
              }
        }
        bar_sync(2 + set, 128);
      }
      if (part == 0) {
        // a CTA's slots: 2 * CTA for a unit that began before its share, + 1
        // for one that goes on after it
        float* po = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + list_bytes(p.ctas)) +
                    (2LL * blockIdx.x + (w.starts ? 1 : 0)) * S::kRows * (kDim + 2);
        const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * set + g + 8 * e;
          if (r >= w.tokens * a.group) continue;
          const float l = e ? l1 : l0;
          if (w.starts && w.ends) {
            const float f = l > 0.f ? 1.f / l : 0.f;
            uint16_t* dst = static_cast<uint16_t*>(a.out) +
                            ((w.tok0 + r / a.group) * hq + static_cast<int64_t>(w.h) * a.group + r % a.group) * kDim + 8 * t;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(dst + 32 * c) =
                  make_uint4(pack_bf16x2(st.o[4 * c][2 * e] * f, st.o[4 * c + 1][2 * e] * f),
                             pack_bf16x2(st.o[4 * c + 2][2 * e] * f, st.o[4 * c + 3][2 * e] * f),
                             pack_bf16x2(st.o[4 * c][2 * e + 1] * f, st.o[4 * c + 1][2 * e + 1] * f),
                             pack_bf16x2(st.o[4 * c + 2][2 * e + 1] * f, st.o[4 * c + 3][2 * e + 1] * f));
          } else {
            float* dst = po + r * kDim + 8 * t;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                *reinterpret_cast<float4*>(dst + 32 * c + 4 * j) =
                    make_float4(st.o[4 * c][2 * e + j], st.o[4 * c + 1][2 * e + j], st.o[4 * c + 2][2 * e + j],
                                st.o[4 * c + 3][2 * e + j]);
            if (t == 0) *reinterpret_cast<float2*>(po + S::kRows * kDim + 2 * r) = make_float2(e ? m1 : m0, l);
          }
        }
      }
      if (w.starts && tid == 0) {
        // the pieces of the unit: shares from this one to that of its last block
        const int pieces =
            w.ends ? 0 : static_cast<int>((static_cast<int64_t>(w.c0) * per + (w.unit - w.g * per + 1) * w.nb - 1) / share -
                                          blockIdx.x + 1);
        if (p.by_unit)
          cut[w.unit] = make_int2(blockIdx.x, pieces);
        else if (pieces)
          cut[blockIdx.x] = make_int2(w.unit, pieces);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == S::kCompute) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(T::columns));
  }
}

// ---- cut units -----------------------------------------------------------------
// Joins the pieces of the units that share borders cut.  A warp takes one row
// and every `parts`-th of its pieces; the `parts` warps of a row are joined in
// shared memory.
__global__ void __launch_bounds__(256) dense_pa_join_kernel(const __grid_constant__ Params p, int rows_pad, int parts) {
  __shared__ float4 s_o[8][32];
  __shared__ float2 s_ml[8];
  pdl_wait();
  pdl_trigger();
  const DensePaParams& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_cta = 8 / parts;  // rows of a CTA
  const int chunks = (p.sub_tokens * a.group + per_cta - 1) / per_cta;
  const int item = blockIdx.x / chunks, row = (blockIdx.x % chunks) * per_cta + warp / parts, part = warp % parts;
  const int2 info = reinterpret_cast<const int2*>(a.ws)[item];
  const int pieces = info.y, c0 = p.by_unit ? info.x : item, unit = p.by_unit ? item : info.x;
  if (pieces == 0) return;
  const int per = a.hkv * p.subs, g = unit / per, h = unit % per / p.subs, sub = unit % p.subs;
  const int64_t tok0 = static_cast<int64_t>(g) * a.q_group + sub * p.sub_tokens;
  const int tokens = static_cast<int>(
      min(static_cast<int64_t>(min(p.sub_tokens, a.q_group - sub * p.sub_tokens)), a.num_rows / a.hkv - tok0));
  const bool live = row < tokens * a.group;
  const float* base = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + list_bytes(p.ctas));
  const int64_t slot_floats = static_cast<int64_t>(rows_pad) * (kDim + 2);

  float M = kNoMax, L = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    for (int k0 = part; k0 < pieces; k0 += 32 * parts) {
      // lane j: piece k0 + j * parts
      const int k = k0 + lane * parts;
      const int64_t slot = k == 0 ? 2LL * c0 + 1 : 2LL * (c0 + k);
      float2 ml = make_float2(kNoMax, 0.f);
      if (k < pieces) ml = *reinterpret_cast<const float2*>(base + slot * slot_floats + rows_pad * kDim + 2 * row);
      float mx = ml.x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(M, mx), f = ex2_approx(M - mn), w = ex2_approx(ml.x - mn);
      float ls = w * ml.y;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
      L = L * f + ls;
      M = mn;
      x.x *= f, x.y *= f, x.z *= f, x.w *= f;
      const int here = min(32, (pieces - k0 + parts - 1) / parts);
#pragma unroll 8
      for (int j = 0; j < here; ++j) {
        const int kj = k0 + j * parts;
        const int64_t sj = kj == 0 ? 2LL * c0 + 1 : 2LL * (c0 + kj);
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const float4 y = *reinterpret_cast<const float4*>(base + sj * slot_floats + row * kDim + 4 * lane);
        x.x += wj * y.x, x.y += wj * y.y, x.z += wj * y.z, x.w += wj * y.w;
      }
    }
  }
  if (parts > 1) {
    s_o[warp][lane] = x;
    if (lane == 0) s_ml[warp] = make_float2(M, L);
    __syncthreads();
    if (part) return;
    float mn = kNoMax;
    for (int k = 0; k < parts; ++k) mn = fmaxf(mn, s_ml[warp + k].x);
    x = make_float4(0.f, 0.f, 0.f, 0.f), L = 0.f;
    for (int k = 0; k < parts; ++k) {
      const float w = ex2_approx(s_ml[warp + k].x - mn);
      const float4 y = s_o[warp + k][lane];
      L += w * s_ml[warp + k].y;
      x.x += w * y.x, x.y += w * y.y, x.z += w * y.z, x.w += w * y.w;
    }
  }
  if (!live) return;
  const float f = L > 0.f ? 1.f / L : 0.f;
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  const int64_t e = ((tok0 + row / a.group) * hq + static_cast<int64_t>(h) * a.group + row % a.group) * kDim + 4 * lane;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e) =
      make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
}

// ---- host ------------------------------------------------------------------------
// One side of the cache as [blocks][heads][4][32][row]: row 32j + i of a box
// is token 4i + j.  K's rows are 128 4-bit values, unpacked to 16-byte slots of
// 16 with 128-byte swizzle; V's are 64 bytes, 64-byte swizzle.
bool make_map_side(CUtensorMap* m, bool unpack, const void* base, uint64_t heads, uint64_t blocks, uint64_t stride) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[5] = {unpack ? 128u : 64u, 32, 4, heads, blocks};
  const cuuint64_t strides[4] = {256, 64, kMxField, stride};
  const cuuint32_t box[5] = {unpack ? 128u : 64u, 32, 4, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, unpack ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 5,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            unpack ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// how a group's rows are cut into units
struct Plan {
  int sub_tokens, subs, sets;
};
Plan plan_of(int group, int q_group) {
  const int sub = std::min(q_group, kMaxRows / group), subs = (q_group + sub - 1) / sub;
  const int even = (q_group + subs - 1) / subs;  // units of about the same size
  return {even, subs, (even * group + 15) / 16};
}

// CTAs per SM: what the register bound allows, as far as shared memory holds
// them (TMEM: 512 columns).  The occupancy query answers 1 for a kernel that
// allocates TMEM.
template <int SETS, bool Q16>
constexpr int ctas_per_sm() {
  return std::min(min_ctas<SETS>(), 228 * 1024 / (Smem<SETS>::total(Q16) + 1024 + 256));
}
int ctas_of(int sets, bool q16) {
  switch (sets) {
    case 1:
      return q16 ? ctas_per_sm<1, true>() : ctas_per_sm<1, false>();
    case 2:
      return q16 ? ctas_per_sm<2, true>() : ctas_per_sm<2, false>();
    case 3:
      return q16 ? ctas_per_sm<3, true>() : ctas_per_sm<3, false>();
    default:
      return q16 ? ctas_per_sm<4, true>() : ctas_per_sm<4, false>();
  }
}

template <int SETS, bool Q16>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, cudaStream_t s) {
  static_assert(Smem<SETS>::total(Q16) <= 227 * 1024 && Tmem<SETS>::used <= Tmem<SETS>::columns);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {  // the shared-memory opt-in
    return cudaFuncSetAttribute(dense_pa_kernel<SETS, Q16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<SETS>::total(Q16));
  });
  if (e != cudaSuccess) return e;
  return launch_kernel(dense_pa_kernel<SETS, Q16>, dim3(static_cast<unsigned>(p.ctas)), dim3(Smem<SETS>::kThreads),
                       Smem<SETS>::total(Q16), s, 0, mk, mv, p);
}
template <bool Q16>
cudaError_t launch_sets(int sets, const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, cudaStream_t s) {
  return sets == 1   ? launch_main<1, Q16>(mk, mv, p, s)
         : sets == 2 ? launch_main<2, Q16>(mk, mv, p, s)
         : sets == 3 ? launch_main<3, Q16>(mk, mv, p, s)
                     : launch_main<4, Q16>(mk, mv, p, s);
}

}  // namespace

size_t dense_pa_ws_bytes(int32_t num_rows, int32_t hkv, int32_t group, int32_t q_group, int num_sms) {
  (void)num_rows, (void)hkv;
  const Plan pl = plan_of(group, q_group);
  const int64_t ctas = static_cast<int64_t>(std::max(ctas_of(pl.sets, false), ctas_of(pl.sets, true))) * num_sms;
  return list_bytes(ctas) + 2 * ctas * 16 * pl.sets * (kDim + 2) * sizeof(float);
}

cudaError_t launch_dense_pa(const DensePaParams& a, int num_sms, cudaStream_t s, int* launches) {
  if (a.num_rows == 0) return cudaSuccess;
  const Plan pl = plan_of(a.group, a.q_group);
  const bool q16 = a.q_dtype == BSP_BF16;
  Params p{};
  p.a = a;
  p.qk_scale = a.sm_scale * kLog2e;
  const int tokens = a.num_rows / a.hkv;
  p.groups = (tokens + a.q_group - 1) / a.q_group;
  p.subs = pl.subs;
  p.sub_tokens = pl.sub_tokens;
  const int64_t units = static_cast<int64_t>(p.groups) * a.hkv * pl.subs;
  if (units > INT32_MAX) return cudaErrorNotSupported;
  p.units = static_cast<int32_t>(units);
  const int per_sm = ctas_of(pl.sets, q16);
  p.ctas = static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(per_sm) * num_sms, units * a.bt_stride));
  p.by_unit = units <= p.ctas;
  CUtensorMap mk, mv;
  const uint64_t blocks = std::max<int64_t>(a.num_blocks, 1);
  if (!make_map_side(&mk, true, a.k_base, a.hkv, blocks, a.id_stride) ||
      !make_map_side(&mv, false, a.v_base, a.hkv, blocks, a.id_stride))
    return cudaErrorInvalidValue;
  cudaError_t e = q16 ? launch_sets<true>(pl.sets, mk, mv, p, s) : launch_sets<false>(pl.sets, mk, mv, p, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.ctas > 1) {
    // pieces of a unit are about ctas / units: more warps a row where they are many
    const int64_t pieces = std::min<int64_t>(p.ctas / units + 1, a.bt_stride);
    const int parts = pieces >= 64 ? 8 : (pieces >= 32 ? 4 : (pieces >= 16 ? 2 : 1));
    const int64_t chunks = (pl.sub_tokens * a.group + 8 / parts - 1) / (8 / parts);
    const int64_t items = p.by_unit ? units : p.ctas;
    e = launch_kernel(dense_pa_join_kernel, dim3(static_cast<unsigned>(items * chunks)), dim3(256), 0, s, 0, p,
                      16 * pl.sets, parts);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaPeekAtLastError();
}

}  // namespace bsp
