// dense_work.cuh -- how the dense attention kernels divide their work: units, equal shares
// of the units' blocks, a CTA's walk over its share, and the join of the units that
// share borders cut.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "tc_warp.cuh"

namespace bsp {

namespace {

constexpr float kMaxGrow = 8.f;   // the reference maximum moves when a row's maximum grows by more (log2)
constexpr float kBias = 7.f;      // weights are 2^((z - m) qk + kBias): at most 2^15

// bytes of the list of cut units at the start of the workspace
__host__ __device__ constexpr int64_t list_bytes(int64_t ctas) { return (ctas * 8 + 255) / 256 * 256; }

struct Params {
  DensePaParams a;
  float qk_scale;  // |sm_scale| * log2(e): a negative scale's sign goes to q
  int32_t groups, subs, sub_tokens;  // query groups; units each is cut into, of sub_tokens tokens
  int32_t units, ctas, shares;       // shares = ctas / subs
  int32_t rows;                      // of a unit's slot in the workspace
  int32_t by_unit;                   // the list of cut units has an entry per unit (else per CTA)
  int32_t least;                     // shares of enough blocks in all (128 of them for each) have so many at least
  int32_t more;                      // blocks that a share may grow by so as to hold one unit's only; < 0: none
};

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
#pragma unroll 1
  for (int i = first; i < n; i += step) len = max(len, a.row_len[tok0 * a.hkv + i]);
  return len;
}

// ... as shares are measured: a multiple of `pad`, the share's length where no share is to
// hold parts of two units, else 1
__device__ __forceinline__ int length_of(const DensePaParams& a, int len, int pad) {
  const int nb = blocks_of(a, len);
  return pad == 1 ? nb : (nb + pad - 1) / pad * pad;
}

// A warp's walk over the pieces of a share [at, end) of the units' blocks.
// Every lane holds the same values.
struct Walk {
  int64_t at, end, c0;  // c0: length of the groups before g
  int g, nb, pad;       // nb: length of g
  // the piece at `at`
  int unit, h, tok0, tokens, seq, b0, nblk, max_len, min_len;
  bool starts, ends;  // the unit's first and last blocks are in the piece

  __device__ __noinline__ bool next(const Params& p, int sub, int lane) {
    if (at >= end) return false;
    const DensePaParams& a = p.a;
    while ((c0 + nb) * a.hkv <= at) {
      c0 += nb;
      ++g;
      nb = length_of(a, __reduce_max_sync(0xffffffffu, group_len(a, g, lane, 32)), pad);
    }
    h = a.hkv == 1 ? 0 : static_cast<int>((at - c0 * a.hkv) / nb);
    const int64_t ustart = c0 * a.hkv + static_cast<int64_t>(h) * nb, uend = ustart + nb;
    unit = (g * a.hkv + h) * p.subs + sub;
    const int gtok = g * a.q_group;
    tok0 = gtok + sub * p.sub_tokens;
    tokens = min(min(p.sub_tokens, a.q_group - sub * p.sub_tokens), a.num_rows / a.hkv - tok0);
    seq = a.row_seq[static_cast<int64_t>(gtok) * a.hkv];
    const int cap = static_cast<int>(min(static_cast<int64_t>(a.bt_stride) * kBlock, int64_t{0x7FFFFFFF}));
    int len = 0;
    if (lane < tokens) len = min(max(a.row_len[static_cast<int64_t>(tok0 + lane) * a.hkv + h], 0), cap);
    max_len = __reduce_max_sync(0xffffffffu, len);  // 0 where the last group lacks this unit's tokens
    min_len = __reduce_min_sync(0xffffffffu, lane < tokens ? len : 0x7FFFFFFF);
    b0 = static_cast<int>(at - ustart);
    nblk = max(0, min(static_cast<int>(min(end, uend) - ustart), (max_len >> 7) + ((max_len & 127) != 0)) - b0);
    starts = at == ustart, ends = end >= uend;
    at = min(end, uend);
    return true;
  }
};

// The `turn`-th of the equal shares.  A thread sums the blocks of some neighbouring groups, and
// the one whose groups hold the share's start looks through them again: the share's first
// group, the blocks before it, its blocks to `start`, which the next barrier publishes.
struct Share {
  int64_t at, share, total;
  int pad;
};
template <int THREADS>
__device__ __forceinline__ Share find_share(const Params& p, int turn, int64_t* s_sum, int64_t* s_start) {
  const DensePaParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.groups + THREADS - 1) / THREADS;
  const int g_lo = static_cast<int>(min(static_cast<int64_t>(tid) * per, static_cast<int64_t>(p.groups)));
  const int g_hi = min(g_lo + per, p.groups);
  int64_t mine, upto, total, share = 0;
  int pad = 1;
#pragma unroll 1
  for (bool again = false;; again = true) {
    mine = 0;
#pragma unroll 4
    for (int g = g_lo; g < g_hi; ++g) mine += length_of(a, group_len(a, g, 0, 1), pad);
    upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) upto += s_sum[w];
      total += s_sum[w];
    }
    if (again) break;
    const int64_t blocks = total * a.hkv, least = min(static_cast<int64_t>(p.least), max(blocks >> 7, int64_t{1}));
    share = max((blocks + p.shares - 1) / p.shares, least);
    // Shares of one unit's blocks only: as many as there are do for this length (a unit's last may be short).
    const int64_t pairs = static_cast<int64_t>(p.groups) * a.hkv, spare = p.shares - pairs;
    if (p.more < 0 || pairs == 1 || spare <= 0) break;
    const int64_t whole = max((blocks + spare - 1) / spare, least);
    if (whole == 1 || whole > share + p.more) break;
    share = whole, pad = static_cast<int>(whole);
    __syncthreads();  // the sums are read
  }
  const int64_t at = turn * share;
  if ((upto - mine) * a.hkv <= at && at < upto * a.hkv) {
    int64_t c = upto - mine;
    int g = g_lo, nb = length_of(a, group_len(a, g, 0, 1), pad);
    while (at >= (c + nb) * a.hkv) c += nb, nb = length_of(a, group_len(a, ++g, 0, 1), pad);
    s_start[0] = g, s_start[1] = c, s_start[2] = nb;
  }
  return {at, share, total, pad};
}
__device__ __forceinline__ Walk walk_of(const Params& p, const Share& sh, const int64_t* s_start) {
  Walk w;
  w.at = sh.at, w.end = min(sh.at + sh.share, sh.total * p.a.hkv);
  w.g = 0, w.c0 = 0, w.nb = 1, w.pad = sh.pad;
  if (w.at < w.end) w.g = static_cast<int>(s_start[0]), w.c0 = s_start[1], w.nb = static_cast<int>(s_start[2]);
  return w;
}

// ---- cut units -----------------------------------------------------------------
// Joins the pieces of the units that share borders cut.  A warp takes one row
// and every `parts`-th of its pieces; the `parts` warps of a row are joined in
// shared memory.  A piece's O that lies 2^126 below the row's is gone; its sum of weights
// need not be (over fp8 references count V's scales, the sums do not): see rescaled.
__global__ void __launch_bounds__(256) dense_pa_join_kernel(const __grid_constant__ Params p, int parts) {
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
  const int sub = unit % p.subs, h = unit / p.subs % a.hkv, g = unit / p.subs / a.hkv;
  const int64_t tok0 = static_cast<int64_t>(g) * a.q_group + sub * p.sub_tokens;
  const int tokens = static_cast<int>(
      min(static_cast<int64_t>(min(p.sub_tokens, a.q_group - sub * p.sub_tokens)), a.num_rows / a.hkv - tok0));
  const bool live = row < tokens * a.group;
  const float* base = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + list_bytes(p.ctas));
  const int64_t slot_floats = static_cast<int64_t>(p.rows) * (kDim + 2);

  float M = kNoMax, L = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    for (int k0 = part; k0 < pieces; k0 += 32 * parts) {
      // lane j: piece k0 + j * parts
      const int k = k0 + lane * parts;
      const int64_t slot = k == 0 ? 2LL * c0 + 1 : 2LL * (c0 + static_cast<int64_t>(k) * p.subs);
      float2 ml = make_float2(kNoMax, 0.f);
      if (k < pieces) ml = *reinterpret_cast<const float2*>(base + slot * slot_floats + p.rows * kDim + 2 * row);
      const int here = min(32, (pieces - k0 + parts - 1) / parts);
      // the first pieces' rows, on their way while the weights are worked out (16 of them took
      // longer where there are few)
      constexpr int kFirst = 8;
      float4 first[kFirst];
#pragma unroll
      for (int j = 0; j < kFirst; ++j) {
        const int kj = k0 + j * parts;
        const int64_t sj = kj == 0 ? 2LL * c0 + 1 : 2LL * (c0 + static_cast<int64_t>(kj) * p.subs);
        first[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < here) first[j] = *reinterpret_cast<const float4*>(base + sj * slot_floats + row * kDim + 4 * lane);
      }
      float mx = ml.x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(M, mx), f = rescale(M, mn, p.qk_scale), w = rescale(ml.x, mn, p.qk_scale);
      float ls = rescaled(ml.y, ml.x, mn, p.qk_scale);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
      L = rescaled(L, M, mn, p.qk_scale) + ls;
      M = mn;
      x.x *= f, x.y *= f, x.z *= f, x.w *= f;
#pragma unroll
      for (int j = 0; j < kFirst; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const float4 y = first[j];
        if (j < here) x.x += wj * y.x, x.y += wj * y.y, x.z += wj * y.z, x.w += wj * y.w;
      }
#pragma unroll 8
      for (int j = kFirst; j < here; ++j) {
        const int kj = k0 + j * parts;
        const int64_t sj = kj == 0 ? 2LL * c0 + 1 : 2LL * (c0 + static_cast<int64_t>(kj) * p.subs);
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
      const float w = rescale(s_ml[warp + k].x, mn, p.qk_scale);
      const float4 y = s_o[warp + k][lane];
      L += rescaled(s_ml[warp + k].y, s_ml[warp + k].x, mn, p.qk_scale);
      x.x += w * y.x, x.y += w * y.y, x.z += w * y.z, x.w += w * y.w;
    }
  }
  if (!live) return;
  const float f = L == 0.f ? 0.f : 1.f / L;
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  const int64_t e = ((tok0 + row / a.group) * hq + static_cast<int64_t>(h) * a.group + row % a.group) * kDim + 4 * lane;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e) =
      make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
}

// ---- host ------------------------------------------------------------------------
// units of sub_tokens query tokens, subs of them a group, in the kernel for `rows` rows
struct Plan {
  int sub_tokens, subs, rows, ctas_per_sm;
};
// the counts of p.a's work
inline void set_work(Params& p, const Plan& pl, int num_sms) {
  const DensePaParams& a = p.a;
  const int tokens = a.num_rows / a.hkv;
  p.groups = (tokens + a.q_group - 1) / a.q_group;
  p.subs = pl.subs;
  p.sub_tokens = pl.sub_tokens;
  p.rows = pl.rows;
  const int64_t pairs = static_cast<int64_t>(p.groups) * a.hkv, units = pairs * pl.subs;
  p.units = static_cast<int32_t>(units);
  p.shares = static_cast<int32_t>(
      std::min<int64_t>(static_cast<int64_t>(pl.ctas_per_sm) * num_sms / pl.subs, pairs * a.bt_stride));
  p.ctas = p.shares * pl.subs;
  p.by_unit = units <= p.ctas;
  p.least = 1;
  p.more = -1;
}

// the second launch, where shares may cut units
inline cudaError_t launch_join(const Params& p, cudaStream_t s, int* launches) {
  if (p.shares <= 1) return cudaSuccess;
  const int64_t pairs = static_cast<int64_t>(p.groups) * p.a.hkv;
  // pieces of a unit are about shares / (groups x heads): more warps a row where they are many
  const int64_t pieces = std::min<int64_t>(p.shares / pairs + 1, p.a.bt_stride);
  const int parts = pieces >= 64 ? 8 : (pieces >= 32 ? 4 : (pieces >= 16 ? 2 : 1));
  const int64_t chunks = (p.sub_tokens * p.a.group + 8 / parts - 1) / (8 / parts);
  const int64_t items = p.by_unit ? p.units : p.ctas;
  const cudaError_t e = launch_kernel(dense_pa_join_kernel, dim3(static_cast<unsigned>(items * chunks)), dim3(256), 0, s, 0, p,
                    parts);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaSuccess;
}

}  // namespace

}  // namespace bsp
