// dense_pa.cu -- dense grouped-query attention over an MXFP4 paged cache
// (bsp_dense_pa_decode).
//
//   z[r, t] = scale * sum_c 2^(ek[t, c] - 127) sum_{d in c} q[r, d] k4[t, d]
//   o[r, d] = sum_t p[r, t] 2^(ev[t, c(d)] - 127) v4[t, d] / sum_t p[r, t],   p = exp(z)
//
// with k4, v4 the e2m1 values, e the e8m0 bytes of the four 32-dim groups c.
//
// Unit = (query group, KV head): its rows, q_group tokens times G heads, share
// every byte of the cache.  The units' 128-token blocks laid end to end are
// cut into equal shares, one per resident CTA, so ragged batches load every SM
// alike; a CTA finds its share by a prefix sum over the groups' lengths.  A
// unit that lies in one share is written at once; of a unit cut by share
// borders each CTA leaves (m, l, O) in the workspace, and a second kernel joins
// them (it reads a list of cut units, no counters, so the workspace carries
// nothing from call to call and the sums' order is fixed).
//
// A warp takes 32 tokens (a slice) at a time.  Slices arrive by TMA in a ring
// of each team's own: 2 KB of K and of V by tensor copies with the 64-byte
// swizzle (ldmatrix rows are 64 bytes apart; without it four would share a
// bank), 128 B of each side's scales by plain bulk copies.  The warps of a team
// hold different rows (MT tiles of 16) and read the same slice.
//
//   z: mma.sync m16n8k32 e4m3, one k-step per scale group into accumulators of
//      its own, multiplied by the token's scale as it is added to z.  e2m1
//      bits moved under the e4m3 exponent are the value times 2^-6, exactly,
//      so four ALU operations convert four values.  A bf16 query is the sum of
//      two e4m3 parts, each with its own power of two (see stage_q).
//   o: mma.sync m16n8k16 f16.  V's bytes come through ldmatrix.trans as four
//      nibbles of two neighbouring tokens a register, which bit moves turn into
//      f16 pairs, times 2^-14 exactly.  V's scales go onto P: 2^(ev - R_c), a
//      power of two at most 1, multiplies the f16 weights of each group.  R_c
//      is the largest scale byte so far (O is rescaled when it grows).  Tokens
//      whose scale is 15 or more binades below R_c, which f16 could not hold,
//      make the warp take the slice again in bands of 15 binades.
//   p is f16: at most half a step, 2^-11, off; weights are kept times 2^7 so that
//      the f16 range, down to 2^-25, reaches 2^-32 of the largest.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace bsp {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSlice = 32;
constexpr int kStages = 2;             // slices in flight per team
constexpr int kTileBytes = kSlice * 64;  // one side of a slice
constexpr int kRowPad = kDim + 4;      // floats of a row in the teams' merge area
constexpr float kMaxGrow = 8.f;        // the reference maximum moves when a row's maximum grows by more (log2)
constexpr float kBias = 7.f;           // weights are 2^(z - m + kBias)
constexpr float kNoMax = -1e30f;       // the maximum of no tokens (finite: -inf - kNoMax stays -inf)
constexpr int kBand = 15;              // binades a band of V scales spans

// rows of a unit split over the CTA's warps: `sets` warps of MT tiles make a
// team, `teams` teams share the slices
struct Shape {
  int mt, sets, teams;
  __host__ __device__ int warps() const { return sets * teams; }
  __host__ __device__ int rows() const { return sets * mt * 16; }
};
__host__ __device__ inline Shape shape_of(int rows) {
  if (rows <= 16) return {1, 1, 4};
  const int sets = (rows + 31) / 32;
  return {2, sets, sets <= 2 ? 4 : 2};
}

// bytes of the list of cut units at the start of the workspace
__host__ __device__ constexpr int64_t list_bytes(int64_t ctas) { return (ctas * 8 + 255) / 256 * 256; }

struct Params {
  DensePaParams a;
  float qk_scale;  // sm_scale * log2(e) * 2^6 (K's exponent shift)
  int32_t groups, units, ctas, sets, teams;
  int32_t by_unit;  // the list of cut units has an entry per unit (else per CTA)
};

// ---- shared memory -----------------------------------------------------------
struct Layout {
  int scales, merge_ml, q, scratch, bars, bad, total;
};
__host__ __device__ inline Layout layout(const Shape& s, bool q16) {
  Layout l;
  const int ring = s.teams * kStages;
  l.scales = ring * 2 * kTileBytes;
  const int ring_bytes = l.scales + ring * 256;
  l.merge_ml = s.warps() * s.mt * 16 * kRowPad * 4;
  const int merge_bytes = l.merge_ml + s.warps() * s.mt * 16 * 8;
  l.q = (std::max(ring_bytes, merge_bytes) + 127) / 128 * 128;
  l.scratch = l.q + s.rows() / 16 * 4 * 512 * (q16 ? 2 : 1) + s.rows() * 4;
  l.bars = l.scratch + s.warps() * 768;
  l.bad = l.bars + 2 * ring * 8;
  l.total = l.bad + ring * 4 + 1024;  // slack: the tiles start on 1024 bytes
  return l;
}

// ---- device helpers ------------------------------------------------------------
__device__ __forceinline__ void tile_g2s(void* dst, const CUtensorMap* m, int row, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(m), "r"(0), "r"(row), "r"(block), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_e4m3_zero(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// eight e2m1 nibbles -> e4m3 bytes of the even (b0) and odd (b1) nibbles, times 2^-6
__device__ __forceinline__ void e2m1x8_to_e4m3(uint32_t w, uint32_t& b0, uint32_t& b1) {
  b0 = ((w << 4) & 0x80808080u) | ((w << 2) & 0x1C1C1C1Cu);
  b1 = (w & 0x80808080u) | ((w >> 2) & 0x1C1C1C1Cu);
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
// 2^e for any e (two factors, each a normal float, where one would overflow)
__device__ __forceinline__ float scale_pow2(float x, int e) {
  const int a = max(-126, min(127, e)), b = max(-126, min(127, e - a));
  return x * __uint_as_float(static_cast<uint32_t>(a + 127) << 23) * __uint_as_float(static_cast<uint32_t>(b + 127) << 23);
}

// one warp's running softmax over MT tiles of 16 rows (rows g and g + 8 of a
// tile in a thread)
template <int MT>
struct State {
  float o[MT][16][4];  // tile 4c + i: dims 32c + 8t + i and 32c + 8t + 4 + i
  float m[MT][2], l[MT][2];
  uint32_t r;  // R_c: the largest V scale byte so far, group c in byte c
};

// blocks of group g: the longest of its rows, at least one (an empty unit
// still writes its zeros)
__device__ __forceinline__ int group_blocks(const DensePaParams& a, int g) {
  const int tokens = a.num_rows / a.hkv;
  const int64_t r0 = static_cast<int64_t>(g) * a.q_group * a.hkv;
  const int n = min(a.q_group, tokens - g * a.q_group) * a.hkv;
  int len = 0;
  for (int i = 0; i < n; ++i) len = max(len, a.row_len[r0 + i]);
  return max(1, min((len + 127u) / 128u, static_cast<uint32_t>(a.bt_stride)));
}

// q of a unit as mma A fragments: [tile][group c][lane] of 16 bytes, thread
// (g, t) rows g, g + 8 and dims 32c + 8t + (0,2,4,6 | 1,3,5,7), the order in
// which the K conversion hands out its nibbles.  A bf16 row is scaled by 2^-a,
// its largest magnitude then in [128, 256), and split: hi = e4m3(x), lo =
// e4m3((x - hi) * 2^4).  bf16 has 8 significant bits and each part 4, so the sum is exact
// for elements down to 2^-13 of the row's largest and off by at most 2^-21 of it below.  The row's 2^a goes to row_scale.
template <bool Q16>
__device__ __forceinline__ void stage_q(const DensePaParams& a, int tok0, int tokens, int h, uint8_t* qs, int rows,
                                        int tid, int threads) {
  float* row_scale = reinterpret_cast<float*>(qs + rows / 16 * 4 * 512 * (Q16 ? 2 : 1));
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  // a quad of lanes per (row, group c): lane t of it owns dims 32c + 8t..+7
  for (int i = tid; i < rows * 16; i += threads) {
    const int row = i >> 4, c = (i >> 2) & 3, t = i & 3;
    const int j = row / a.group, hh = row % a.group;
    const bool live = j < tokens;
    const int64_t e = ((tok0 + j) * hq + static_cast<int64_t>(h) * a.group + hh) * kDim + 32 * c + 8 * t;
    const int g = row & 7, half = (row >> 3) & 1;
    uint8_t* dst = qs + (((row >> 4) * 4 + c) * 32 + g * 4 + t) * 16 + half * 4;
    if (Q16) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (live) w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + e);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      float x[8], top = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = bf16_bits_to_float(k & 1 ? ws[k >> 1] >> 16 : ws[k >> 1] & 0xFFFF);
        top = fmaxf(top, fabsf(x[k]));
      }
      // the row's 16 lanes are one half-warp
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      const int ex = max(-110, static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127) - 7;  // 2^ex * [128, 256)
      uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
#pragma unroll
        for (int par = 0; par < 2; ++par) {  // par 0: even dims, 1: odd
          const float u = scale_pow2(x[k + par], -ex), v = scale_pow2(x[k + 2 + par], -ex);
          const uint32_t hb = float2_to_e4m3x2(u, v);
          const uint32_t lb = float2_to_e4m3x2((u - e4m3_to_float(hb)) * 16.f, (v - e4m3_to_float(hb >> 8)) * 16.f);
          hi[par] |= hb << (8 * (k >> 1));
          lo[par] |= lb << (8 * (k >> 1));
        }
      }
      *reinterpret_cast<uint32_t*>(dst) = hi[0];
      *reinterpret_cast<uint32_t*>(dst + 8) = hi[1];
      uint8_t* dl = dst + rows / 16 * 4 * 512;
      *reinterpret_cast<uint32_t*>(dl) = lo[0];
      *reinterpret_cast<uint32_t*>(dl + 8) = lo[1];
      if (c == 0 && t == 0) row_scale[row] = scale_pow2(1.f, ex);
    } else {
      uint2 w = make_uint2(0, 0);
      if (live) w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.q) + e);
      *reinterpret_cast<uint32_t*>(dst) = __byte_perm(w.x, w.y, 0x6420);
      *reinterpret_cast<uint32_t*>(dst + 8) = __byte_perm(w.x, w.y, 0x7531);
      if (c == 0 && t == 0) row_scale[row] = 1.f;
    }
  }
}

// One slice: K, V tiles and scales in shared memory, tokens n0 .. n0 + 31 of
// the sequence; rows see tokens below len[tile][half] (all zero for a bad block).
template <int MT, bool Q16>
__device__ __forceinline__ void slice(State<MT>& st, uint32_t kt, uint32_t vt, const uint8_t* sc, uint32_t qs,
                                      uint32_t qlo, uint8_t* scratch, int n0, const int (&len)[MT][2], int max_len,
                                      bool whole, const float (&zs)[MT][2], int lane) {
  const int t = lane & 3;
  const uint32_t kp = smem_u32(scratch), vp = kp + 512;
  // -- scales: lane = token.  Neighbours trade words, so that the even lane
  // writes groups 0, 1 and the odd one groups 2, 3 of their pair of tokens:
  // K's as float pairs [c][t][octet], V's as f16 pairs in the same order.
  const int odd = lane & 1, sh = odd * 16;
  const uint32_t kw = *reinterpret_cast<const uint32_t*>(sc + 4 * lane);
  const uint32_t vw = n0 + lane < max_len ? *reinterpret_cast<const uint32_t*>(sc + 128 + 4 * lane) : 0;
  const uint32_t kx = __shfl_xor_sync(0xffffffffu, kw, 1), vx = __shfl_xor_sync(0xffffffffu, vw, 1);
  const int cell = ((lane >> 1) & 3) * 4 + (lane >> 3);  // [t][octet]
  {
    const uint32_t a = (odd ? kx : kw) >> sh, b = (odd ? kw : kx) >> sh;
    const uint32_t at = kp + (2 * odd * 16 + cell) * 8;
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"((a << 23) & 0x7F800000u), "r"((b << 23) & 0x7F800000u)
                 : "memory");
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + 128), "r"((a << 15) & 0x7F800000u),
                 "r"((b << 15) & 0x7F800000u)
                 : "memory");
  }
  const uint32_t va = (odd ? vx : vw) >> sh, vb = (odd ? vw : vx) >> sh;  // bytes 0, 1: this lane's groups
  {
    const uint32_t rr = st.r >> sh;
    const bool up = (va & 0xFF) > (rr & 0xFF) || (vb & 0xFF) > (rr & 0xFF) || (va >> 8 & 0xFF) > (rr >> 8 & 0xFF) ||
                    (vb >> 8 & 0xFF) > (rr >> 8 & 0xFF);
    if (__any_sync(0xffffffffu, up)) {  // R_c grows: O moves to the new unit
      uint32_t nr = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t old = st.r >> (8 * c) & 0xFF;
        const uint32_t now = max(old, __reduce_max_sync(0xffffffffu, vw >> (8 * c) & 0xFF));
        nr |= now << (8 * c);
        const float f = scale_pow2(1.f, static_cast<int>(old) - static_cast<int>(now));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[mt][4 * c + i][e] *= f;
      }
      st.r = nr;
    }
  }
  // f16 2^(byte - R_c + kBand*band) of this lane's groups and pair, 0 outside the band
  auto put_vscales = [&](int band) {
    const uint32_t rr = st.r >> sh;
    bool low = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = rr >> (8 * k) & 0xFF;
      uint32_t h[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int b = (e ? vb : va) >> (8 * k) & 0xFF;
        const int x = b - r + kBand * band + 15;  // f16 exponent field: 1..15 within the band
        h[e] = x > 0 && x <= 15 && b ? x << 10 : 0;
        low |= b != 0 && x <= 0;
      }
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(vp + ((2 * odd + k) * 16 + cell) * 4), "r"(h[0] | (h[1] << 16))
                   : "memory");
    }
    return __any_sync(0xffffffffu, low);
  };
  bool more = put_vscales(0);
  __syncwarp();

  // -- z
  float z[MT][4][4];
  const int row8 = lane & 7, mat = lane >> 3;
  const uint32_t row_off = (mat * 8 + row8) * 64;
  const int swz = (row8 >> 1) & 3;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t kr[4];
    ldsm_x4(kr[0], kr[1], kr[2], kr[3], kt + row_off + ((c ^ swz) << 4));
    const uint4 s01 = lds128(kp + (c * 16 + t * 4) * 8), s23 = lds128(kp + (c * 16 + t * 4) * 8 + 16);
    const float2 ks[4] = {{__uint_as_float(s01.x), __uint_as_float(s01.y)},
                          {__uint_as_float(s01.z), __uint_as_float(s01.w)},
                          {__uint_as_float(s23.x), __uint_as_float(s23.y)},
                          {__uint_as_float(s23.z), __uint_as_float(s23.w)}};
    uint4 qa[MT], ql[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      qa[mt] = lds128(qs + (mt * 4 + c) * 512 + lane * 16);
      if (Q16) ql[mt] = lds128(qlo + (mt * 4 + c) * 512 + lane * 16);
    }
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      uint32_t b0, b1;
      e2m1x8_to_e4m3(kr[o], b0, b1);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float acc[4];
        if (Q16) {
          mma_e4m3_zero(acc, ql[mt], b0, b1);
          const float2 lo = fmul2({acc[0], acc[1]}, {0.0625f, 0.0625f}), hi = fmul2({acc[2], acc[3]}, {0.0625f, 0.0625f});
          acc[0] = lo.x, acc[1] = lo.y, acc[2] = hi.x, acc[3] = hi.y;
          mma_e4m3(acc, qa[mt].x, qa[mt].y, qa[mt].z, qa[mt].w, b0, b1);
        } else {
          mma_e4m3_zero(acc, qa[mt], b0, b1);
        }
        float2 x, y;
        if (c == 0) {
          x = fmul2({acc[0], acc[1]}, ks[o]), y = fmul2({acc[2], acc[3]}, ks[o]);
        } else {
          x = ffma2({acc[0], acc[1]}, ks[o], {z[mt][o][0], z[mt][o][1]});
          y = ffma2({acc[2], acc[3]}, ks[o], {z[mt][o][2], z[mt][o][3]});
        }
        z[mt][o][0] = x.x, z[mt][o][1] = x.y, z[mt][o][2] = y.x, z[mt][o][3] = y.y;
      }
    }
  }

  // -- weights
  uint32_t pa[MT][4], pb[MT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      const float2 x = fmul2({z[mt][o][0], z[mt][o][1]}, {zs[mt][0], zs[mt][0]});
      const float2 y = fmul2({z[mt][o][2], z[mt][o][3]}, {zs[mt][1], zs[mt][1]});
      z[mt][o][0] = x.x, z[mt][o][1] = x.y, z[mt][o][2] = y.x, z[mt][o][3] = y.y;
      if (!whole) {
        const int n = n0 + 8 * o + 2 * t;
        if (n >= len[mt][0]) z[mt][o][0] = -INFINITY;
        if (n + 1 >= len[mt][0]) z[mt][o][1] = -INFINITY;
        if (n >= len[mt][1]) z[mt][o][2] = -INFINITY;
        if (n + 1 >= len[mt][1]) z[mt][o][3] = -INFINITY;
      }
      mx0 = fmax3(mx0, z[mt][o][0], z[mt][o][1]);
      mx1 = fmax3(mx1, z[mt][o][2], z[mt][o][3]);
    }
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    const bool mv0 = mx0 > st.m[mt][0] + kMaxGrow, mv1 = mx1 > st.m[mt][1] + kMaxGrow;
    if (__any_sync(0xffffffffu, mv0 || mv1)) {
      const float n0m = mv0 ? mx0 : st.m[mt][0], n1m = mv1 ? mx1 : st.m[mt][1];
      const float a0 = ex2_approx(st.m[mt][0] - n0m), a1 = ex2_approx(st.m[mt][1] - n1m);
      st.m[mt][0] = n0m, st.m[mt][1] = n1m;
      st.l[mt][0] *= a0, st.l[mt][1] *= a1;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        st.o[mt][i][0] *= a0, st.o[mt][i][1] *= a0, st.o[mt][i][2] *= a1, st.o[mt][i][3] *= a1;
    }
    const float r0 = st.m[mt][0] - kBias, r1 = st.m[mt][1] - kBias;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      const float p0 = ex2_approx(z[mt][o][0] - r0), p1 = ex2_approx(z[mt][o][1] - r0);
      const float p2 = ex2_approx(z[mt][o][2] - r1), p3 = ex2_approx(z[mt][o][3] - r1);
      s0 += p0 + p1;
      s1 += p2 + p3;
      pa[mt][o] = pack_f16x2(p0, p1);
      pb[mt][o] = pack_f16x2(p2, p3);
    }
    st.l[mt][0] += s0, st.l[mt][1] += s1;
  }

  // -- o
  const uint32_t vrow = vt + row_off;
  for (int band = 0;; ++band) {
    const bool direct = band == 0 && !more;
    const float f = band == 0 ? 1.f : scale_pow2(1.f, -kBand * band);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t zr[4];
      ldsm_x4_trans(zr, vrow + ((c ^ swz) << 4));
      const uint4 vs4 = lds128(vp + (c * 16 + t * 4) * 4);
      const uint32_t vs[4] = {vs4.x, vs4.y, vs4.z, vs4.w};
      uint32_t v[4][4];
#pragma unroll
      for (int o = 0; o < 4; ++o) e2m1x4x2_to_f16x2(zr[o], v[o]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t a[4], b[4];
#pragma unroll
        for (int o = 0; o < 4; ++o) a[o] = hmul2(pa[mt][o], vs[o]), b[o] = hmul2(pb[mt][o], vs[o]);
        if (direct) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16(st.o[mt][4 * c + i], a[2 * ks], b[2 * ks], a[2 * ks + 1], b[2 * ks + 1], v[2 * ks][i],
                      v[2 * ks + 1][i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
              mma_f16(x, a[2 * ks], b[2 * ks], a[2 * ks + 1], b[2 * ks + 1], v[2 * ks][i], v[2 * ks + 1][i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[mt][4 * c + i][e] += x[e] * f;
          }
        }
      }
    }
    if (!more) break;
    __syncwarp();  // the band's scales are read
    more = put_vscales(band + 1);
    __syncwarp();
  }
}

// ---- the main kernel -----------------------------------------------------------
template <int MT, bool Q16>
__global__ void __launch_bounds__(MT == 1 ? 128 : 256, MT == 1 ? 4 : 1)
    dense_pa_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_cum[257];  // blocks before group tile_g0 + i
  __shared__ int64_t s_part[8];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  const Shape sh{MT, p.sets, p.teams};
  const Layout lay = layout(sh, Q16);
  const DensePaParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int set = warp % p.sets, team = warp / p.sets;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars) + team * kStages;
  uint64_t* empty = full + p.teams * kStages;
  volatile uint32_t* bad = reinterpret_cast<uint32_t*>(smem + lay.bad) + team * kStages;
  uint8_t* ring = smem + team * kStages * 2 * kTileBytes;
  uint8_t* ring_sc = smem + lay.scales + team * kStages * 256;
  if (tid == 0) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + lay.bars);
    for (int i = 0; i < p.teams * kStages; ++i) {
      mbar_init(&bars[i], 1);
      mbar_init(&bars[p.teams * kStages + i], p.sets);
    }
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();

  // the groups' blocks, scanned a tile of `threads` groups at a time
  auto scan_tile = [&](int g0, int64_t base) -> int64_t {  // returns the blocks up to the tile's end
    const int g = g0 + tid;
    const int64_t nb = g < p.groups ? group_blocks(a, g) : 0;
    int64_t x = nb;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) s_part[warp] = x;
    __syncthreads();
    int64_t before = base, all = base;
    for (int w = 0; w < threads / 32; ++w) {
      if (w < warp) before += s_part[w];
      all += s_part[w];
    }
    s_cum[tid] = before + x - nb;
    if (tid == 0) s_cum[threads] = all;
    __syncthreads();
    return all;
  };
  int64_t total = 0;
  int tile_g0 = 0;
  for (int g0 = 0; g0 < p.groups; g0 += threads) {
    total = scan_tile(g0, total);
    tile_g0 = g0;
  }
  const int64_t work = total * a.hkv;
  const int64_t share = (work + p.ctas - 1) / p.ctas;
  int64_t at = blockIdx.x * share;  // this CTA's blocks: [at, end)
  const int64_t end = min(at + share, work);
  // cut units: (first CTA, pieces) per unit, or (unit, pieces) per first CTA
  int2* cut = reinterpret_cast<int2*>(a.ws);
  if (!p.by_unit && tid == 0) cut[blockIdx.x] = make_int2(0, 0);
  if (at >= end) return;
  // back to the tile the share starts in
  if (s_cum[0] * a.hkv > at) {
    int64_t base = 0;
    for (tile_g0 = 0;; tile_g0 += threads) {
      base = scan_tile(tile_g0, base);
      if (base * a.hkv > at) break;
    }
  }

  const int rows_pad = sh.rows();
  uint8_t* qs = smem + lay.q;
  const uint32_t qs_set = smem_u32(qs) + set * MT * 4 * 512, qlo_set = qs_set + rows_pad / 16 * 4 * 512;
  const float* row_scale = reinterpret_cast<const float*>(qs + rows_pad / 16 * 4 * 512 * (Q16 ? 2 : 1));
  uint8_t* scratch = smem + lay.scratch + warp * 768;
  uint32_t fill = 0, used = 0;  // slices issued and consumed by this team
  bool alive = true;
  int gi = 0;

  while (at < end) {
    // the unit at `at`
    while (s_cum[gi + 1] * a.hkv <= at) {
      if (++gi == threads) {
        const int64_t base = s_cum[threads];
        __syncthreads();
        tile_g0 += threads, gi = 0;
        scan_tile(tile_g0, base);
      }
    }
    const int g = tile_g0 + gi;
    const int64_t c0 = s_cum[gi], nb = s_cum[gi + 1] - c0;
    const int h = static_cast<int>((at - c0 * a.hkv) / nb);
    const int64_t ustart = c0 * a.hkv + h * nb, uend = ustart + nb;
    const int b0 = static_cast<int>(at - ustart), b1 = static_cast<int>(min(end, uend) - ustart);
    const int tok0 = g * a.q_group, tokens = min(a.q_group, a.num_rows / a.hkv - tok0);
    const int64_t row0 = static_cast<int64_t>(tok0) * a.hkv + h;
    const int seq = a.row_seq[static_cast<int64_t>(tok0) * a.hkv];
    const int32_t* table = a.block_table + static_cast<int64_t>(seq) * a.bt_stride;
    const int cap = min(static_cast<int64_t>(a.bt_stride) * kBlock, int64_t{0x7FFFFFFF});
    int max_len = 0, min_len = 0x7FFFFFFF;
    for (int j = 0; j < tokens; ++j) {
      const int n = min(max(a.row_len[row0 + static_cast<int64_t>(j) * a.hkv], 0), cap);
      max_len = max(max_len, n), min_len = min(min_len, n);
      if (tid == 0 && a.row_seq[row0 + static_cast<int64_t>(j) * a.hkv] != seq) set_err(a.err, BSP_DEVERR_GROUP_SEQ);
    }
    // this team's slices of blocks [b0, b1), none past the rows' tokens
    const int s0 = b0 * 4, s1 = min(b1 * 4, (max_len + kSlice - 1) / kSlice);
    const int n = s1 > s0 + team ? (s1 - s0 - team + p.teams - 1) / p.teams : 0;

    int32_t ids = 0;  // lane i: the block id of the team's slice 32 * chunk + i
    int chunk = -1;
    auto issue = [&](int i) {  // slice i of the team into its ring (warp `set` 0)
      if ((i >> 5) != chunk) {
        chunk = i >> 5;
        const int k = 32 * chunk + lane;
        ids = k < n ? table[(s0 + team + k * p.teams) >> 2] : 0;
      }
      const int32_t id = __shfl_sync(0xffffffffu, ids, i & 31);
      if (lane == 0) {
        const int stg = fill % kStages;
        if (p.sets > 1 && fill >= kStages && alive)
          alive = mbar_wait(&empty[stg], ((fill / kStages) - 1) & 1, a.err);
        if (id < 0 || id >= a.num_blocks) {
          set_err(a.err, BSP_DEVERR_BLOCK_ID);
          bad[stg] = 1;
          mbar_arrive(&full[stg]);
        } else {
          bad[stg] = 0;
          const int o0 = ((s0 + team + i * p.teams) & 3) * kSlice;
          const int64_t off = static_cast<int64_t>(id) * a.id_stride + static_cast<int64_t>(h) * kMxField + kMxScaleOff + o0 * 4;
          uint8_t* dst = ring + stg * 2 * kTileBytes;
          fence_proxy_async();
          mbar_arrive_expect_tx(&full[stg], 2 * kTileBytes + 256);
          tile_g2s(dst, &map_k, h * (kMxField / 64) + o0, id, &full[stg]);
          tile_g2s(dst + kTileBytes, &map_v, h * (kMxField / 64) + o0, id, &full[stg]);
          bulk_g2s(ring_sc + stg * 256, a.k_base + off, 128, &full[stg]);
          bulk_g2s(ring_sc + stg * 256 + 128, a.v_base + off, 128, &full[stg]);
        }
      }
      ++fill;
    };
    if (set == 0)
      for (int i = 0; i < min(n, kStages); ++i) issue(i);

    stage_q<Q16>(a, tok0, tokens, h, qs, rows_pad, tid, threads);
    State<MT> st;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[mt][i][0] = st.o[mt][i][1] = st.o[mt][i][2] = st.o[mt][i][3] = 0.f;
      st.m[mt][0] = st.m[mt][1] = kNoMax, st.l[mt][0] = st.l[mt][1] = 0.f;
    }
    st.r = 0;
    int len[MT][2];
    float zs[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (set * MT + mt) * 16 + (lane >> 2) + 8 * k, j = row / a.group;
        len[mt][k] = j < tokens ? min(max(a.row_len[row0 + static_cast<int64_t>(j) * a.hkv], 0), cap) : 0;
      }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) zs[mt][k] = p.qk_scale * row_scale[(set * MT + mt) * 16 + (lane >> 2) + 8 * k];

    for (int i = 0; i < n; ++i) {
      const int stg = used % kStages;
      if (alive) alive = mbar_wait_sleep(&full[stg], (used / kStages) & 1, a.err);
      alive = __all_sync(0xffffffffu, alive);  // after a timed-out wait the warp waits no more
      ++used;
      const int n0 = (s0 + team + i * p.teams) * kSlice;
      const bool skip = !alive || bad[stg];  // nothing of the slice is used
      const uint32_t kt = smem_u32(ring + stg * 2 * kTileBytes);
      if (!skip)
        slice<MT, Q16>(st, kt, kt + kTileBytes, ring_sc + stg * 256, qs_set, qlo_set, scratch, n0, len, max_len,
                       n0 + kSlice <= min_len, zs, lane);
      __syncwarp();
      if (p.sets > 1 && lane == 0) mbar_arrive(&empty[stg]);
      if (set == 0 && i + kStages < n) issue(i + kStages);
    }

    // -- the teams' states joined in shared memory (the ring is drained)
    __syncthreads();
    float* mo = reinterpret_cast<float*>(smem);
    float2* ml = reinterpret_cast<float2*>(smem + lay.merge_ml);
    const int gq = lane >> 2, t = lane & 3;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float l = st.l[mt][k];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int r = (warp * MT + mt) * 16 + gq + 8 * k;
        if (t == 0) ml[r] = make_float2(st.m[mt][k], l);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int e = static_cast<int>(st.r >> (8 * c) & 0xFF) - 127 + 14;
          float x[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            x[q] = scale_pow2(st.o[mt][4 * c + q][2 * k], e);
            x[4 + q] = scale_pow2(st.o[mt][4 * c + q][2 * k + 1], e);
          }
          float* dst = mo + r * kRowPad + 32 * c + 8 * t;
          *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
    __syncthreads();
    const bool whole_unit = at == ustart && end >= uend;
    // a CTA's slots: 2 * CTA for a unit that began before its share, + 1 for
    // one that goes on after it
    const int64_t piece = 2LL * blockIdx.x + (at == ustart ? 1 : 0);
    float* po = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + list_bytes(p.ctas)) + piece * rows_pad * (kDim + 2);
    float2* pml = reinterpret_cast<float2*>(po + rows_pad * kDim);
    const int live_rows = tokens * a.group;
    const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
    for (int r = warp; r < live_rows; r += threads / 32) {
      const int rs = r / (MT * 16), ri = r % (MT * 16);
      float M = kNoMax;
      for (int k = 0; k < p.teams; ++k) M = fmaxf(M, ml[(k * p.sets + rs) * MT * 16 + ri].x);
      float L = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < p.teams; ++k) {
        const int s = (k * p.sets + rs) * MT * 16 + ri;
        const float2 v = ml[s];
        const float w = ex2_approx(v.x - M);
        const float4 y = *reinterpret_cast<const float4*>(mo + s * kRowPad + 4 * lane);
        L += w * v.y;
        x.x += w * y.x, x.y += w * y.y, x.z += w * y.z, x.w += w * y.w;
      }
      if (whole_unit) {
        const float f = L > 0.f ? 1.f / L : 0.f;
        const int64_t e = ((tok0 + r / a.group) * hq + static_cast<int64_t>(h) * a.group + r % a.group) * kDim + 4 * lane;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e) =
            make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
      } else {
        *reinterpret_cast<float4*>(po + r * kDim + 4 * lane) = x;
        if (lane == 0) pml[r] = make_float2(M, L);
      }
    }
    if (at == ustart && tid == 0) {
      const int pieces = whole_unit ? 0 : static_cast<int>((uend - 1) / share - blockIdx.x + 1);
      const int unit = g * a.hkv + h;
      if (p.by_unit)
        cut[unit] = make_int2(blockIdx.x, pieces);
      else if (pieces)
        cut[blockIdx.x] = make_int2(unit, pieces);
    }
    __syncthreads();  // the merge area becomes the ring again
    at = min(end, uend);
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
  const int chunks = (a.q_group * a.group + per_cta - 1) / per_cta;
  const int item = blockIdx.x / chunks, row = (blockIdx.x % chunks) * per_cta + warp / parts, part = warp % parts;
  const int2 info = reinterpret_cast<const int2*>(a.ws)[item];
  const int pieces = info.y, c0 = p.by_unit ? info.x : item, unit = p.by_unit ? item : info.x;
  if (pieces == 0) return;
  const int g = unit / a.hkv, h = unit % a.hkv;
  const int64_t tok0 = static_cast<int64_t>(g) * a.q_group;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.q_group), a.num_rows / a.hkv - tok0));
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
// [rows of 64 B][blocks] of one side, boxes of one slice
bool make_map_side(CUtensorMap* m, const void* base, uint64_t rows, uint64_t blocks, uint64_t stride) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {64, rows, blocks};
  const cuuint64_t strides[2] = {64, stride};
  const cuuint32_t box[3] = {64, kSlice, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// resident CTAs per SM, with the shared-memory opt-in (once per device and shape)
template <int MT, bool Q16>
int occupancy(const Shape& sh) {
  static std::atomic<int> table[5][kMaxDevices];
  return cached_per_device(table[sh.sets], [&] {
    int n = 0;
    const int bytes = layout(sh, Q16).total;
    int most = 0;  // of the shapes this kernel runs in
    for (int rows = MT == 1 ? 16 : 32; rows <= (MT == 1 ? 16 : 128); rows += 32)
      most = std::max(most, layout(shape_of(rows), Q16).total);
    const cudaError_t e =
        cudaFuncSetAttribute(dense_pa_kernel<MT, Q16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess || cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, dense_pa_kernel<MT, Q16>,
                                                                           sh.warps() * 32, bytes) != cudaSuccess)
      n = 0;
    return n > 0 ? n : 1;
  });
}
int occupancy_of(const Shape& sh, bool q16) {
  if (sh.mt == 1) return q16 ? occupancy<1, true>(sh) : occupancy<1, false>(sh);
  return q16 ? occupancy<2, true>(sh) : occupancy<2, false>(sh);
}

template <int MT, bool Q16>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, const Shape& sh, cudaStream_t s) {
  return launch_kernel(dense_pa_kernel<MT, Q16>, dim3(static_cast<unsigned>(p.ctas)), dim3(sh.warps() * 32),
                       layout(sh, Q16).total, s, 0, mk, mv, p);
}

}  // namespace

size_t dense_pa_ws_bytes(int32_t num_rows, int32_t hkv, int32_t group, int32_t q_group, int num_sms) {
  (void)num_rows, (void)hkv;
  const Shape sh = shape_of(group * q_group);
  const int64_t ctas = static_cast<int64_t>(std::max(occupancy_of(sh, false), occupancy_of(sh, true))) * num_sms;
  return list_bytes(ctas) + 2 * ctas * sh.rows() * (kDim + 2) * sizeof(float);
}

cudaError_t launch_dense_pa(const DensePaParams& a, int num_sms, cudaStream_t s, int* launches) {
  if (a.num_rows == 0) return cudaSuccess;
  const Shape sh = shape_of(a.group * a.q_group);
  const bool q16 = a.q_dtype == BSP_BF16;
  Params p{};
  p.a = a;
  p.qk_scale = a.sm_scale * kLog2e * 64.f;
  const int tokens = a.num_rows / a.hkv;
  p.groups = (tokens + a.q_group - 1) / a.q_group;
  const int64_t units = static_cast<int64_t>(p.groups) * a.hkv;
  p.units = static_cast<int32_t>(units);
  p.ctas = static_cast<int32_t>(
      std::min<int64_t>(static_cast<int64_t>(occupancy_of(sh, q16)) * num_sms, units * a.bt_stride));
  p.sets = sh.sets;
  p.teams = sh.teams;
  p.by_unit = units <= p.ctas;
  CUtensorMap mk, mv;
  const uint64_t rows = static_cast<uint64_t>(a.hkv) * (kMxField / 64), blocks = std::max<int64_t>(a.num_blocks, 1);
  if (!make_map_side(&mk, a.k_base, rows, blocks, a.id_stride) || !make_map_side(&mv, a.v_base, rows, blocks, a.id_stride))
    return cudaErrorInvalidValue;
  cudaError_t e = sh.mt == 1 ? (q16 ? launch_main<1, true>(mk, mv, p, sh, s) : launch_main<1, false>(mk, mv, p, sh, s))
                             : (q16 ? launch_main<2, true>(mk, mv, p, sh, s) : launch_main<2, false>(mk, mv, p, sh, s));
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.ctas > 1) {
    // pieces of a unit are about ctas / units: more warps a row where they are many
    const int64_t pieces = std::min<int64_t>(p.ctas / units + 1, a.bt_stride);
    const int parts = pieces >= 64 ? 8 : (pieces >= 32 ? 4 : (pieces >= 16 ? 2 : 1));
    const int64_t chunks = (a.q_group * a.group + 8 / parts - 1) / (8 / parts);
    const int64_t items = p.by_unit ? units : p.ctas;
    e = launch_kernel(dense_pa_join_kernel, dim3(static_cast<unsigned>(items * chunks)), dim3(256), 0, s, 0, p,
                      sh.rows(), parts);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaPeekAtLastError();
}

}  // namespace bsp
