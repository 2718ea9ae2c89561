// dense_pa_fp8.cu -- dense grouped-query attention over an fp8 paged cache, with scales
// per block and head or per tensor (bsp_dense_pa_decode_fp8).
//
//   t[r, s] = (scale log2(e) ks[b(s)]) q_r . k8_s + log2 vs[b(s)],   w[r, s] = 2^(t[r, s] - R_r)
//   o_r = sum_s w[r, s] v8_s / sum_s w[r, s] / vs[b(s)]
//
// with k8, v8 the e4m3 values: a block's V scale is part of its tokens' weights, so that
// V enters the product as it lies, and a row's reference R counts it; the sums l get the
// weights without it, a multiplication by 1 / vs that the addition takes along.  Where V's
// scales lie far apart a token may have a weight below fp32's range whose share of l counts: a
// block 2^64 below an earlier one's scale has its l from exponentials of its own, and where a
// reference moves by more than 2^126, l moves in two steps.  l itself stays in range: it is at
// least the row's largest exp(z) 2^(kBias - R), and that is 2^(kBias - 128) or more.
//
// Work: units, equal shares and the join of cut units as in the MXFP4 kernel
// (dense_work.cuh).  Both products are tcgen05 MMAs with the block's tokens or V's dims as
// their 128 rows and the unit's N = 16, 32 or 64 rows as their columns:
//   z^T = K Q^T      A = K from shared memory, e4m3, B = q; a bf16 query row is the sum of
//                    two e4m3 parts with one scale (see stage_q)
//   O^T += V^T P     A = V^T, f16, from TMEM, B = P, f16, from shared memory
// The interleaved pages are what the tensor core reads: a K page holds 8-token x 16-byte
// cells, so a TMA box with its 256-byte pieces (16 tokens of 16 dims) turned to dims-major
// order is the unswizzled K-major operand; a V page holds the 16 tokens of a dim side by
// side, and thread = dim reads them as one vector.  P V in e4m3, V straight from shared
// memory, would need no conversion, but weights of four bits do not do, and several
// parts of them reach down 2^-26 of the largest at best: the many small weights of a long
// context would be lost.  f16 has 11 bits and, with a reference of 2^kBias, reaches 2^-32.
//
// A CTA is a loader warp, an issuer warp and four or eight compute warps.  Thread = token
// of the logits: its exponentials against the rows' references, which move only when a
// row's maximum passes its own by kMaxGrow; a vote of the four warps that share rows
// finds those blocks, and the ones that some row does not see whole, and takes them
// through an uncommon way (of eight warps: 214.5 us for 207 of 64 rows a request).  Then thread = dim turns V to f16, 16 tokens a load.  0 times a NaN byte of
// V is NaN: in blocks that some row does not see whole such bytes are read as 0, and
// the rows that see the first of them get their NaN at the end.
//
// Measured (a call of a row of twenty in a graph): 64 requests of 131072 tokens, 16 rows each, 318 to
// 323 us, 6.6 to 6.7 TB/s, 98 to 100 % of the copy rate: memory; 128 of 32768 with 64 rows 200 us, 5.4
// TB/s, and with bf16 queries, whose logits take twice the MMAs and a factor each, 227: a
// block's chain of logits, exponentials, P and V, with the two CTAs that TMEM has room for;
// 32 of 4k to 8k 22.8 us (24.9 with other inputs each time): 6 us to a CTA's first block, 1.8 for
// each of four, 2.5 for sums and O, 4.5 for the join; one of 1000 tokens 10.9 us.
//
// Every wait is bounded: after one that gave up (the error word is set, the results are
// void) loader and issuer issue nothing more and wait for what they have under way; a
// compute warp walks through its blocks without waits and arrivals.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "dense_work.cuh"
#include "kernels.h"
#include "tc_warp.cuh"
#include "tcgen05.cuh"

namespace bsp {

namespace {

constexpr int kTileBytes = kBlock * kDim;  // of K or V
constexpr int kMetas = 8;                  // blocks that may be loaded ahead of the compute warps, at least
constexpr float kLeastScale = 0x1p-60f;
constexpr float kFarScales = 64.f;  // log2 between V scales from which l does not go by the weights with the scale
// A share's blocks at least, where there are 512 in all (2 from 256 on): few long pieces are
// joined faster than many short ones are attended.  Requests of 128k tokens, us, shares of at
// least 1 and 4 blocks: one 36.4, 28.7, four of 32k 25.5, 24.4; one of 1000 tokens 15.8, 19.8.
constexpr int kLeastBlocks = 4;
// Blocks that a share may grow by so as to hold one unit's only: a second unit costs a CTA some 5 us
// (its queries, the first one's output), a block of a CTA 1.8 to 2.8.  us, shares as they come and of
// one unit: 32 requests of 4k to 8k 32.6, 28.6, 100 of 2k 32.3, 27.3, 32 of 16k 43.6, 39.1, 64 of
// 8k with 64 rows 57.5, 50.4; they grow by 2, 1, 1 and 3 blocks.  Long shares (64 x 128k: by 13) stay.
constexpr int kMoreBlocks = 6;

struct Fp8Params {
  Params w;  // qk_scale 1: references are log2 of weights
  const float* k_scales;
  const float* v_scales;
  float k_scale, v_scale;
  float qk;  // sm_scale * log2(e)
};

// ---- shared memory -----------------------------------------------------------
template <int N>
struct Shape {
  static constexpr int kCompute = N == 16 ? 4 : 8, kThreads = 32 * (kCompute + 2), kCtasPerSm = N == 16 ? 4 : 2;
  static constexpr int kHalves = kCompute / 4;  // warps that share 32 TMEM lanes
  static constexpr int kRows = N / kHalves;     // a compute warp's
  static constexpr int kPages = 8 / kHalves;    // of V
};
template <int N, bool Q16>
struct Smem {
  // stages (as much as the CTAs of an SM leave room for)
  static constexpr int kK = N == 32 ? 3 : N == 16 ? 1 : 2, kV = N == 16 ? 1 : 2;
  static constexpr int v = kK * kTileBytes;
  static constexpr int p = v + kV * kTileBytes;        // P [128 tokens][N rows] f16
  static constexpr int q = p + kBlock * N * 2;
  // [kMetas] of a block: k factor, log2 vs, 1 / vs (negative where vs is far below an earlier one of the
  // piece), whether it is not and every row sees the block whole
  static constexpr int meta = q + N * 128 * (Q16 ? 2 : 1);
  static constexpr int refs = meta + kMetas * 16;      // [2][N] kBias - R
  static constexpr int rowfac = refs + 2 * N * 4;      // [N] scales of the query rows
  static constexpr int fac = rowfac + N * 4;           // [N] rescale factors
  static constexpr int tops = fac + N * 4;             // [4][N] maxima, later sums
  static constexpr int len = tops + 4 * N * 4;         // [N] lengths
  static constexpr int nan = len + N * 4;              // [128] the first token whose byte of a dim is a NaN
  static constexpr int bars = nan + 128 * 4;
  static constexpr int k_full = bars, k_empty = k_full + 8 * kK, v_full = k_empty + 8 * kK, v_empty = v_full + 8 * kV,
                       z_full = v_empty + 8 * kV, z_empty = z_full + 16, pv_full = z_empty + 16, pv_done = pv_full + 16,
                       q_full = pv_done + 16, fin = q_full + 8;
  static constexpr int misc = fin + 8;  // TMEM address
  static constexpr int total = misc + 16;
  static_assert(kK + 3 <= kMetas);
  static_assert(p % 1024 == 0 && q % 1024 == 0 && meta % 16 == 0 && refs % 16 == 0);
};
// TMEM columns: V's tile (64 columns of token pairs), O, two buffers of logits
template <int N>
struct Tmem {
  static constexpr int v = 0, o = 64, z = o + N, kColumns = N == 16 ? 128 : 256;
  static_assert(z + 2 * N <= kColumns && kColumns * Shape<N>::kCtasPerSm <= 512);
};

// ---- device helpers ------------------------------------------------------------
// a K or V tile of a block and head; the 5-d map's innermost dims are in the tile's order
__device__ __forceinline__ void tile_g2s_5d(uint32_t dst, const CUtensorMap* m, int head, int block, uint32_t bar) {
  asm volatile(
      BSP_ELECT " @e cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
                "[%1, {%2, %3, %4, %5, %6}], [%7];\n}\n" ::"r"(dst),
      "l"(m), "r"(0), "r"(0), "r"(0), "r"(head), "r"(block), "r"(bar)
      : "memory");
}
// D (+)= A B, both e4m3 in shared memory
__device__ __forceinline__ void umma_ss_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      BSP_ELECT " .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// K: 8-token x 16-byte cells of 128 bytes, 128 bytes apart along the tokens and 2048 along the dims; no swizzle
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  uint64_t d = (saddr & 0x3FFFF) >> 4;
  d |= static_cast<uint64_t>(2048 >> 4) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}
// bytes 0xFF where a byte of w is an e4m3 NaN
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// q of a unit in shared memory as the MMA reads it (rows of 128 e4m3 bytes, 128-byte
// swizzle): thread = 16-byte chunk j of row n.  e4m3 queries are copied.  A bf16 row is
// scaled by 2^-a, its largest magnitude then in [128, 256), and split: hi = e4m3(x), lo =
// e4m3(x - hi), whose products add up in one accumulator; 2^a goes to the row's factor.
// bf16 has 8 significant bits and each part 4, so the sum is exact for elements down to
// 2^-9 of the row's largest, and off by at most 2^-17 of it below.  A row with an infinity
// or a NaN gets the factor NaN.
template <bool Q16>
__device__ __noinline__ void stage_q(const DensePaParams& a, int tok0, int tokens, int h, uint8_t* q, int rows,
                                     float* rowfac, int tid) {
  const int n = tid >> 3, j = tid & 7;
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  const bool live = n / a.group < tokens;
  const int64_t e = ((tok0 + n / a.group) * hq + static_cast<int64_t>(h) * a.group + n % a.group) * kDim + 16 * j;
  uint8_t* dst = q + n * 128 + ((j ^ (n & 7)) << 4);
  if (!Q16) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + e);
    *reinterpret_cast<uint4*>(dst) = w;
    if (j == 0) rowfac[n] = 1.f;
    return;
  }
  uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (live) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + e);
    w[0] = src[0], w[1] = src[1];
  }
  const uint32_t ws[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  uint32_t top = 0;  // bits of the largest magnitude: not finite from 0x7F80 on
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, max(ws[k] & 0x7FFFu, (ws[k] >> 16) & 0x7FFFu));
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  const int ex = max(-100, static_cast<int>(top >> 7) - 127) - 7;
  const float down = __uint_as_float(static_cast<uint32_t>(127 - ex / 2) << 23),
              down2 = __uint_as_float(static_cast<uint32_t>(127 - (ex - ex / 2)) << 23);  // (2^-ex may be no float)
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t hb[2], lb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = ws[2 * k + i];
      const float u = __uint_as_float(x << 16) * down * down2, v = __uint_as_float(x & 0xFFFF0000u) * down * down2;
      hb[i] = float2_to_e4m3x2(u, v);
      lb[i] = float2_to_e4m3x2(u - e4m3_to_float(hb[i]), v - e4m3_to_float(hb[i] >> 8));
    }
    hi[k] = hb[0] | (hb[1] << 16);
    lo[k] = lb[0] | (lb[1] << 16);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(dst + rows * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  if (j == 0)
    rowfac[n] = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
}

// CH logits of a lane's token as t, in the rows' and the block's terms
template <int CH, bool Q16>
__device__ __forceinline__ void load_t(float2 (&t)[CH / 2], uint32_t z_at, uint32_t rowfac, float kc, float lv) {
  float z[CH];
  tmem_ld<CH>(z_at, z);
#pragma unroll
  for (int i = 0; i < CH / 4; ++i) {
    float2 c0 = {kc, kc}, c1 = {kc, kc};
    if (Q16) {
      const float4 f = lds128f(rowfac + 16 * i);
      c0 = fmul2(c0, {f.x, f.y}), c1 = fmul2(c1, {f.z, f.w});
    }
    t[2 * i] = ffma2({z[4 * i], z[4 * i + 1]}, c0, {lv, lv});
    t[2 * i + 1] = ffma2({z[4 * i + 2], z[4 * i + 3]}, c1, {lv, lv});
  }
}

// barrier of four warps that returns whether every thread says so
__device__ __forceinline__ bool four_agree(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id)
      : "memory");
  return r != 0;
}

// ---- the main kernel -----------------------------------------------------------
template <int N, bool Q16>
__global__ void __launch_bounds__(Shape<N>::kThreads, Shape<N>::kCtasPerSm)
    dense_pa_fp8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ Fp8Params fp) {
  using S = Smem<N, Q16>;
  using T = Tmem<N>;
  constexpr int kCompute = Shape<N>::kCompute, kThreads = Shape<N>::kThreads;
  extern __shared__ __align__(1024) uint8_t smem[];
  // before the first block P's place serves the scan
  int64_t* s_sum = reinterpret_cast<int64_t*>(smem + S::p);
  int64_t* s_start = s_sum + kThreads / 32;
  const Params& p = fp.w;
  const DensePaParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t base = smem_u32(smem);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + S::misc);
  if (tid == 0) {
    auto init = [&](int at, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + at) + i, count);
    };
    init(S::k_full, S::kK, 1), init(S::k_empty, S::kK, 1);
    init(S::v_full, S::kV, 1), init(S::v_empty, S::kV, kCompute);
    init(S::z_full, 2, 1), init(S::z_empty, 2, kCompute);
    init(S::pv_full, 2, kCompute), init(S::pv_done, 2, 1);
    init(S::q_full, 1, kCompute), init(S::fin, 1, 1);
    mbar_fence_init();
  }
  pdl_wait();
  // (TMEM only after the wait, and the next kernel's CTAs only once this one has got its
  // columns: one that waits while it holds some could keep the other from its own)
  if (warp == kCompute) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + S::misc), "n"(T::kColumns));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  const int sub = blockIdx.x % p.subs, turn = blockIdx.x / p.subs;
  const Share sh = find_share<kThreads>(p, turn, s_sum, s_start);
  const int64_t share = sh.share;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  pdl_trigger();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
  Walk w = walk_of(p, sh, s_start);
  __syncthreads();  // the scan's place is P's again
  // cut units: (first CTA, pieces) per unit, or (unit, pieces) per first CTA
  int2* cut = reinterpret_cast<int2*>(a.ws);
  if (!p.by_unit && tid == 0) cut[blockIdx.x] = make_int2(0, 0);
  bool alive = true;
  auto wait = [&](uint32_t bar, uint32_t parity) { return alive = alive && wait_warp(bar, parity, a.err); };

  if (warp == kCompute + 1) {
    // ---- loader: walks the share, reads the block table and the scales, 32 blocks at a time ----
    const int limit = static_cast<int>(min(a.num_blocks, int64_t{0x7FFFFFFF}));
    const int bad_id = max(limit, 1);  // outside the map, which has a block at least: its copies write zeros
    uint32_t ks = 0, k_phase = 1, vs = 0, v_phase = 1, number = 0;  // (an empty stage's wait passes at once)
    while (alive && w.next(p, sub, lane)) {
      const int32_t* table = a.block_table + static_cast<int64_t>(w.seq) * a.bt_stride + w.b0;
      int32_t ids = 0;
      float k_raw = 0.f, v_raw = 0.f, kc = 0.f, lv = 0.f, inv = 0.f, most = -INFINITY;
#pragma unroll 1
      for (int i = 0; i < w.nblk; ++i) {
        if ((i & 31) == 0) {
          ids = i + lane < w.nblk ? table[i + lane] : 0;
          k_raw = fp.k_scale, v_raw = fp.v_scale;
          if (static_cast<uint32_t>(ids) >= static_cast<uint32_t>(limit)) {
            set_err(a.err, BSP_DEVERR_BLOCK_ID);
            ids = bad_id;
          } else if (fp.k_scales) {
            k_raw = fp.k_scales[static_cast<int64_t>(ids) * a.hkv + w.h];
            v_raw = fp.v_scales[static_cast<int64_t>(ids) * a.hkv + w.h];
          }
          __syncwarp();
        }
        const int id = __shfl_sync(0xffffffffu, ids, i & 31);
        if (!wait(base + S::k_empty + 8 * ks, k_phase)) break;
        tile_g2s_5d(base + ks * kTileBytes, &map_k, w.h, id, base + S::k_full + 8 * ks);
        if ((i & 31) == 0) {  // (the scales' loads are on their way while K's copy is)
          kc = k_raw * fp.qk;
          const float v = v_raw >= 0.f ? fmaxf(v_raw, kLeastScale) : __uint_as_float(0x7FC00000u);
          lv = __log2f(v);
          inv = v == v ? 1.f / v : 1.f;  // (a NaN comes with the weights, to the rows that have any)
          if (ids == bad_id) kc = 0.f, lv = -INFINITY, inv = 0.f;  // no weights (K and V are zeros)
        }
        const float k = __shfl_sync(0xffffffffu, kc, i & 31), l = __shfl_sync(0xffffffffu, lv, i & 31),
                    v = __shfl_sync(0xffffffffu, inv, i & 31);
        const bool far = l < most - kFarScales && l > -INFINITY;
        most = fmaxf(most, l);
        sts128(base + S::meta + 16 * (number++ % kMetas), __float_as_uint(k), __float_as_uint(l), __float_as_uint(far ? -v : v),
               __float_as_uint(!far && (w.b0 + i) * kBlock <= w.min_len - kBlock ? 1.f : 0.f));
        __syncwarp();
        arrive_expect(base + S::k_full + 8 * ks, kTileBytes);  // (with the block's word there)
        if (++ks == S::kK) ks = 0, k_phase ^= 1;
        if (!wait(base + S::v_empty + 8 * vs, v_phase)) break;
        arrive_expect(base + S::v_full + 8 * vs, kTileBytes);
        tile_g2s_5d(base + S::v + vs * kTileBytes, &map_v, w.h, id, base + S::v_full + 8 * vs);
        if (++vs == S::kV) vs = 0, v_phase ^= 1;
      }
    }
    // nothing may still write shared memory when the CTA leaves
    for (uint32_t i = 0; i < S::kK; ++i)
      wait_warp(base + S::k_full + 8 * i, i < ks ? k_phase ^ 1 : k_phase, a.err, kSleepWaitLimit);
    for (uint32_t i = 0; i < S::kV; ++i)
      wait_warp(base + S::v_full + 8 * i, i < vs ? v_phase ^ 1 : v_phase, a.err, kSleepWaitLimit);
    __syncwarp();
  } else if (warp == kCompute) {
    // ---- issuer: the logits of a block, then P V of the one before ----
    const uint64_t k_desc = desc_k(base), q_desc = smem_desc_sw128(base + S::q);
    // P: rows of 2N bytes, one atom of the 2N-byte swizzle wide, 8 tokens an atom
    uint64_t p_desc = ((base + S::p) & 0x3FFFF) >> 4;
    p_desc |= static_cast<uint64_t>(1) << 16;                              // leading offset: unused
    p_desc |= static_cast<uint64_t>(8 * 2 * N >> 4) << 32;                 // 8 tokens
    p_desc |= static_cast<uint64_t>(1) << 46;                              // descriptor version
    p_desc |= static_cast<uint64_t>(N == 16 ? 6 : N == 32 ? 4 : 2) << 61;  // 32-, 64-, 128-byte swizzle
    // f32 += A (f16, TMEM) B (f16, rows contiguous), M = 128
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
    uint32_t ks = 0, k_phase = 0, q_phase = 0, buf = 0, z_phase = 1, round = 0;
    auto multiply = [&](bool accumulate) {
      const uint32_t b = round & 1;
      if (!wait(base + S::pv_full + 8 * b, (round >> 1) & 1)) return;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
      for (int k = 0; k < kBlock / 16; ++k)
        umma_ts(tmem + T::o, tmem + T::v + 8 * k, p_desc + (k * 16 * 2 * N) / 16, kIdescO, k > 0 || accumulate);
      commit(base + S::pv_done + 8 * b);
      ++round;
    };
    while (alive && w.next(p, sub, lane)) {
      if (!w.nblk) continue;
      if (!wait(base + S::q_full, q_phase)) break;
      q_phase ^= 1;
#pragma unroll 1
      for (int i = 0; i < w.nblk; ++i) {
        if (!wait(base + S::k_full + 8 * ks, k_phase)) break;
        if (!wait(base + S::z_empty + 8 * buf, z_phase)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t kd = k_desc + ks * (kTileBytes / 16);
#pragma unroll
        for (int part = 0; part < (Q16 ? 2 : 1); ++part)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            umma_ss_f8(tmem + T::z + buf * N, kd + c * (4096 / 16), q_desc + (part * N * 128 + 32 * c) / 16,
                       idesc_f8f6f4(kFmtE4m3, kFmtE4m3, N, 128), part > 0 || c > 0);
        commit(base + S::k_empty + 8 * ks);
        commit(base + S::z_full + 8 * buf);
        if (++ks == S::kK) ks = 0, k_phase ^= 1;
        if (++buf == 2) buf = 0, z_phase ^= 1;
        if (i) multiply(i > 1);
        if (!alive) break;
      }
      if (alive) multiply(w.nblk > 1);
    }
    // every MMA and commit has ended
    commit(base + S::fin);
    wait_warp(base + S::fin, 0, a.err, kSleepWaitLimit);
    __syncwarp();
  } else {
    // ---- compute ----
    // Warp: TMEM lanes 32 * quad .., that is the logits of the block's tokens 32 * quad ..
    // and O's and V's dims 32 * quad ..; R rows of the former, VP pages of V.
    constexpr int R = Shape<N>::kRows, CH = 16, VP = Shape<N>::kPages;
    // The four warps of a half look after its rows by themselves.
    const int quad = warp & 3, half = warp >> 2, group = 2 + half;           // group: their barrier
    const int mine = (tid & 127) < R ? half * R + (tid & 127) : 0x7FFFFFFF;  // a row of theirs
    const uint32_t tops = base + S::tops, lens_at = base + S::len, fac = base + S::fac;
    int* lens = reinterpret_cast<int*>(smem + S::len);
    int* nans = reinterpret_cast<int*>(smem + S::nan);
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t z_at = tmem + lane_base + T::z + half * R, o_at = tmem + lane_base + T::o + half * R;
    const uint32_t vt_at = tmem + lane_base + T::v + half * VP * 8;
    const uint32_t rowfac = base + S::rowfac + half * R * 4;
    const int dim = 32 * quad + lane, tok = dim;  // the lane's dim of V and O, and its token
    const uint32_t v_at = base + S::v + half * VP * 2048 + dim * 16;
    const uint32_t swz = (tok & 7) >> (N == 16 ? 2 : N == 32 ? 1 : 0);
    const uint32_t p_at = base + S::p + tok * 2 * N;
    uint32_t zb = 0, z_phase = 0, vst = 0, v_phase = 0, number = 0;  // of the next block
    uint32_t round = 0;                                  // of PV
    uint32_t cur = 0;                                    // which references
    auto done = [&](uint32_t r) {  // round r - 1 has ended
      if (r) wait(base + S::pv_done + 8 * ((r - 1) & 1), ((r - 1) >> 1) & 1);
    };
    while (w.next(p, sub, lane)) {
      bar_sync(1, 32 * kCompute);  // the last unit's q, lengths and sums are no longer read
      if (w.nblk)
        for (int i = tid; i < N * 8; i += 32 * kCompute)
          stage_q<Q16>(a, w.tok0, w.tokens, w.h, smem + S::q, N, reinterpret_cast<float*>(smem + S::rowfac), i);
      if (tid < N) {
        const int j = tid / a.group;
        // (rows that no token has see what the longest sees: they must not look uncommon)
        lens[tid] = j < w.tokens ? min(max(a.row_len[static_cast<int64_t>(w.tok0 + j) * a.hkv + w.h], 0), w.max_len)
                                 : w.max_len;
      }
      if (mine < N) stsf(base + S::refs + (cur * N + mine) * 4, -kNoMax);
      if (tid < kDim) nans[tid] = 0x7FFFFFFF;
      if (tid < w.tokens && a.row_seq[static_cast<int64_t>(w.tok0 + tid) * a.hkv + w.h] != w.seq)
        set_err(a.err, BSP_DEVERR_GROUP_SEQ);
      float2 l[R / 2];  // of the lane's token in every block
#pragma unroll
      for (int i = 0; i < R / 2; ++i) l[i] = make_float2(0.f, 0.f);
      fence_proxy_async();  // the tensor core reads q through the async proxy
      bar_sync(1, 32 * kCompute);
      if (w.nblk && lane == 0 && alive) arrive(base + S::q_full);
      __syncwarp();
      bool first = true;  // no PV round of the unit yet
      int n0 = w.b0 * kBlock;  // at most 2^31 - 128 in the loop
#pragma unroll 1
      for (int k = w.nblk; k > 0; --k, n0 = static_cast<int>(n0 + static_cast<uint32_t>(kBlock))) {
        // after a timed-out wait the warp goes on without waits and arrivals (the
        // barriers of the compute warps need every one); its results are void
        wait(base + S::z_full + 8 * zb, z_phase);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const float4 m4 = lds128f(base + S::meta + 16 * (number++ % kMetas));
        const float kc = m4.x, lv = m4.y;
        float inv = m4.z;
        const bool plain = m4.w != 0.f;
        const uint32_t z = z_at + zb * N;
        float2 x[R / 2];
        float top = -INFINITY;
        auto load = [&] {
#pragma unroll
          for (int c = 0; c < R; c += CH) {
            float2 t[CH / 2];
            load_t<CH, Q16>(t, z + c, rowfac + 4 * c, kc, lv);
            const uint32_t refs = base + S::refs + (cur * N + half * R + c) * 4;
#pragma unroll
            for (int i = 0; i < CH / 4; ++i) {
              const float4 m = lds128f(refs + 16 * i);
              x[c / 2 + 2 * i] = fadd2(t[2 * i], {m.x, m.y});
              x[c / 2 + 2 * i + 1] = fadd2(t[2 * i + 1], {m.z, m.w});
            }
          }
        };
        load();
#pragma unroll
        for (int i = 0; i < R / 2; ++i) top = fmax3(top, x[i].x, x[i].y);
        if (__builtin_expect(!four_agree(group, plain && top <= kMaxGrow + kBias), 0)) {
          // The uncommon way: the rows' maxima over what they see, new references, and
          // O and l in their terms; and the blocks whose scale is far below.
#pragma unroll 1
          for (int c = 0; c < R; c += CH) {
            float2 t[CH / 2];
            load_t<CH, Q16>(t, z + c, rowfac + 4 * c, kc, lv);
            float y[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              y[i] = i & 1 ? t[i >> 1].y : t[i >> 1].x;
              if (n0 + tok >= static_cast<int>(lds32(lens_at + (half * R + c + i) * 4))) y[i] = -INFINITY;
            }
            const float mx = warp_reduce<CH>(y, lane, [](float u, float v) { return fmaxf(u, v); });
            if (!(lane & 1)) stsf(tops + (quad * N + half * R + c + (lane >> 1)) * 4, mx);
            __syncwarp();
          }
          bar_sync(group, 128);
          float f = 1.f;
          if (mine < N) {
            float mx = ldsf(tops + mine * 4);
#pragma unroll
            for (int i = 1; i < 4; ++i) mx = fmaxf(mx, ldsf(tops + (i * N + mine) * 4));
            const float old = ldsf(base + S::refs + (cur * N + mine) * 4), ref = fminf(old, kBias - mx);
            f = rescale(-old, -ref, 1.f);
            stsf(base + S::refs + ((cur ^ 1) * N + mine) * 4, ref);
            // (below fp32's range as a factor to apply twice, which the sign says)
            stsf(fac + mine * 4, f != 0.f ? f : -ex2_approx((ref - old) * 0.5f));
          }
          cur ^= 1;
          if (!four_agree(group, f == 1.f) && !first) {
            done(round);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
            for (int c = 0; c < R; c += CH) {
              float y[CH];
              tmem_ld<CH>(o_at + c, y);
#pragma unroll
              for (int i = 0; i < CH; ++i) {
                const float g = ldsf(fac + (half * R + c + i) * 4), again = g < 0.f ? g : 1.f;
                y[i] = y[i] * g * again;
                float& sum = i & 1 ? l[(c + i) >> 1].y : l[(c + i) >> 1].x;
                sum = sum * g * again;
              }
              tmem_st<CH>(o_at + c, y);
            }
          }
          if (inv < 0.f) {  // l by itself (here, not of x below: 56 bytes of spills, not 108)
#pragma unroll
            for (int c = 0; c < R; c += CH) {
              float2 t[CH / 2];
              load_t<CH, Q16>(t, z + c, rowfac + 4 * c, kc, 0.f);
#pragma unroll
              for (int i = 0; i < CH; ++i) {
                const int r = half * R + c + i;
                const float e = ex2_approx((i & 1 ? t[i >> 1].y : t[i >> 1].x) + ldsf(base + S::refs + (cur * N + r) * 4));
                (i & 1 ? l[(c + i) >> 1].y : l[(c + i) >> 1].x) += n0 + tok < static_cast<int>(lds32(lens_at + r * 4)) ? e : 0.f;
              }
              __syncwarp();
            }
            inv = 0.f;
          }
          load();
          if (!plain) {
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
              if (n0 + tok >= static_cast<int>(lds32(lens_at + (half * R + 2 * i) * 4))) x[i].x = -INFINITY;
              if (n0 + tok >= static_cast<int>(lds32(lens_at + (half * R + 2 * i + 1) * 4))) x[i].y = -INFINITY;
            }
          }
          __syncwarp();
        }
        // the logits are read
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0 && alive) arrive(base + S::z_empty + 8 * zb);
        uint32_t pk[R / 2];
#pragma unroll
        for (int i = 0; i < R / 2; ++i) {
          const float2 e = make_float2(ex2_approx(x[i].x), ex2_approx(x[i].y));
          l[i] = ffma2(e, {inv, inv}, l[i]);
          pk[i] = pack_f16x2(e.x, e.y);
        }
        __syncwarp();
        done(round);  // P and V's tile are free
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int i = 0; i < R / 8; ++i)
          sts128(p_at + ((half * R / 8 + i) ^ swz) * 16, pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        wait(base + S::v_full + 8 * vst, v_phase);
#pragma unroll
        for (int g = 0; g < VP; g += 4) {
          uint32_t r[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 b = lds128(v_at + vst * kTileBytes + (g + j) * 2048);
            uint32_t b4[4] = {b.x, b.y, b.z, b.w};
            if (__builtin_expect(!plain, 0)) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t m = nan_bytes(b4[i]);
                if (m) atomicMin(nans + dim, n0 + (half * VP + g + j) * kPage + 4 * i + ((__ffs(m) - 1) >> 3));
                b4[i] &= ~m;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) e4m3x4_to_f16x2_cvt(b4[i], r[8 * j + 2 * i], r[8 * j + 2 * i + 1]);
          }
          __syncwarp();
          tmem_st32(vt_at + 8 * g, r);
        }
        first = false;
        fence_proxy_async();  // the tensor core reads P through the async proxy
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0 && alive) arrive(base + S::pv_full + 8 * (round & 1)), arrive(base + S::v_empty + 8 * vst);
        ++round;
        if (++zb == 2) zb = 0, z_phase ^= 1;
        if (++vst == S::kV) vst = 0, v_phase ^= 1;
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
      if (mine < N) {  // what O is multiplied by
        const float sum = (ldsf(tops + mine * 4) + ldsf(tops + (N + mine) * 4)) +
                          (ldsf(tops + (2 * N + mine) * 4) + ldsf(tops + (3 * N + mine) * 4));
        stsf(fac + mine * 4, !all ? 1.f : sum == 0.f ? 0.f : 1.f / sum);
        if (!all && mine < rows)
          *reinterpret_cast<float2*>(po + N * kDim + 2 * mine) =
              make_float2(-ldsf(base + S::refs + (cur * N + mine) * 4), sum);
      }
      bar_sync(1, 32 * kCompute);
      if (!first) done(round);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int nan_from = nans[dim];
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                           (static_cast<int64_t>(w.tok0) * a.hkv + w.h) * a.group * kDim + dim;
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
            const float o = nan_from < static_cast<int>(lds32(lens_at + r * 4)) ? __uint_as_float(0x7FC00000u)
                                                                                : y[i] * ldsf(fac + r * 4);
            if (all) {
              *out = __float2bfloat16_rn(o);
              out += kDim;
              if (++in_token == a.group) in_token = 0, out += hop;
            } else {
              po[r * kDim + dim] = o;
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
// One side of the cache in boxes of a block and head, 256-byte pieces.  K: [blocks][heads]
// [dims / 16][pages][16 tokens x 16], so that a box is dims-major; V: pages as they lie.
bool make_map_side(CUtensorMap* m, bool k, const void* base, uint64_t heads, uint64_t blocks, uint64_t stride) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[5] = {256, 8, 8, heads, blocks};
  const cuuint64_t strides[4] = {k ? stride : 256, k ? 256 : stride, 2048, 16 * stride};
  const cuuint32_t box[5] = {256, 8, 8, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Plan plan_of(int group, int q_group) {
  const int sub = std::min(q_group, 64 / group), subs = (q_group + sub - 1) / sub;
  const int tokens = (q_group + subs - 1) / subs, rows = tokens * group;  // units of about the same size
  if (rows <= 16) return {tokens, subs, 16, Shape<16>::kCtasPerSm};
  if (rows <= 32) return {tokens, subs, 32, Shape<32>::kCtasPerSm};
  return {tokens, subs, 64, Shape<64>::kCtasPerSm};
}

template <int N, bool Q16>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, const Fp8Params& p, cudaStream_t s) {
  using S = Smem<N, Q16>;
  static_assert((S::total + 1024) * Shape<N>::kCtasPerSm <= 228 * 1024);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {  // the shared-memory opt-in
    return cudaFuncSetAttribute(dense_pa_fp8_kernel<N, Q16>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::total);
  });
  if (e != cudaSuccess) return e;
  return launch_kernel(dense_pa_fp8_kernel<N, Q16>, dim3(static_cast<unsigned>(p.w.ctas)), dim3(Shape<N>::kThreads),
                       S::total, s, 0, mk, mv, p);
}

}  // namespace

size_t dense_pa_fp8_ws_bytes(int32_t num_rows, int32_t hkv, int32_t group, int32_t q_group, int num_sms) {
  (void)num_rows, (void)hkv;
  const Plan pl = plan_of(group, q_group);
  const int64_t ctas = static_cast<int64_t>(pl.ctas_per_sm) * num_sms;
  return list_bytes(ctas) + 2 * ctas * pl.rows * (kDim + 2) * sizeof(float);
}

cudaError_t launch_dense_pa_fp8(const DensePaFp8Params& a, int num_sms, cudaStream_t s, int* launches) {
  if (a.a.num_rows == 0) return cudaSuccess;
  const Plan pl = plan_of(a.a.group, a.a.q_group);
  const bool q16 = a.a.q_dtype == BSP_BF16;
  Fp8Params p{};
  p.w.a = a.a;
  p.w.qk_scale = 1.f;
  p.qk = a.a.sm_scale * kLog2e;
  p.k_scales = a.k_scales, p.v_scales = a.v_scales, p.k_scale = a.k_scale, p.v_scale = a.v_scale;
  set_work(p.w, pl, num_sms);
  p.w.least = kLeastBlocks;
  p.w.more = kMoreBlocks;
  CUtensorMap mk, mv;
  const uint64_t blocks = std::max<int64_t>(a.a.num_blocks, 1);
  if (!make_map_side(&mk, true, a.a.k_base, a.a.hkv, blocks, a.a.id_stride) ||
      !make_map_side(&mv, false, a.a.v_base, a.a.hkv, blocks, a.a.id_stride))
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
  if ((e = launch_join(p.w, s, launches)) != cudaSuccess) return e;
  return cudaPeekAtLastError();
}

}  // namespace bsp
