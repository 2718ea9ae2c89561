// norm_rope.cu -- RMS norm of each query and key head, the position rotation
// in the same pass, and the result stored where the step reads it: queries as
// bf16 or e4m3 rows, keys and values quantised straight into the caches
// (bsp_norm_rope_write; ROCm/ATOM PR 2962, commit "... index key": one writer
// norms, rotates and stores K, V and the index key onto the pool pages and
// emits the e4m3 queries).
//
//   y_d = x_d / sqrt(mean(x^2) + eps) * (w_d + offset)        (q, k, index q, index k)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)      for the pairs of the first rot_dim dims
//
// V takes neither.  Everything is fp32 until the one rounding of each output;
// in particular the caches are quantised from the fp32 rows, not from a bf16
// copy of them.
//
// 16 lanes hold a head, 8 dims each (16-byte loads; mean and MXFP4 group
// maxima are shuffles within 16 and 4 lanes).  A half-warp takes one token; the
// head's type and number are the same for a whole warp.
//
// Measured: 1 token 2.0 us (a launch); 16456 tokens of 16 + 1 + 1 + 1 + 1 heads, bf16
// queries and fp8 caches, 42 us for 167 MB: 4.0 TB/s, 60 % of the copy rate.  There
// the latency of loads and of shuffles (the mean's, and of rotation by halves the
// partners', which this lane layout puts into another lane) bounds it, beside 177 warp
// instructions for a head of two tokens at 60 % of the issue slots; loads further
// ahead did not shorten it.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "encode.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_bits_to_float(w[i] & 0xFFFF);
    x[2 * i + 1] = bf16_bits_to_float(w[i] >> 16);
  }
}
// packed fp32 pairs: a * b + c
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
__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8]) {
  return make_uint2(float2_to_e4m3x2(x[0], x[1]) | (float2_to_e4m3x2(x[2], x[3]) << 16),
                    float2_to_e4m3x2(x[4], x[5]) | (float2_to_e4m3x2(x[6], x[7]) << 16));
}
__device__ __forceinline__ float absmax8(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}
// dims 8*l.. of token o of an MXFP4 field; a: the 32-group's largest magnitude
__device__ __forceinline__ void store_mx(uint8_t* field, int o, int l, const float (&x)[8], float a) {
  const int e = mx_shared_exp(a);
  const float sc = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, normal for e in [-127, 125]
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= float2_to_e2m1x2(x[2 * i] * sc, x[2 * i + 1] * sc) << (8 * i);
  *reinterpret_cast<uint32_t*>(field + o * 64 + 4 * l) = w;
  if ((l & 3) == 0) field[kMxScaleOff + o * 4 + (l >> 2)] = static_cast<uint8_t>(e + 127);
}

// Stores a row (dims 8l.. of the lane) of K, V or the index key into its cache.
// Every lane of the warp calls it; `store`: the lane's token has a place.
__device__ __forceinline__ void store_cached(const NormRopeParams& p, int ty, int h, int64_t slot, bool store, int l,
                                             float (&x)[8]) {
  const KvWriteParams& c = p.cache;
  const bool is_idx = ty == kHeadIdxK;
  const int dtype = is_idx ? c.idx_dtype : c.kv_dtype;
  // group maxima of the quantised forms: 32 dims (4 lanes), 128 dims (16)
  float amax = 0.f;
  if (dtype == BSP_MXFP4 || (is_idx && dtype == BSP_FP8_E4M3)) {
    amax = absmax8(x);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if (dtype == BSP_FP8_E4M3) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
    }
  }
  const int64_t block = slot / kBlock;
  const int o = static_cast<int>(slot % kBlock);
  if (store && block >= (is_idx ? c.idx_num_blocks : c.num_blocks)) {
    if (l == 0) set_err(p.err, BSP_DEVERR_SLOT);
    store = false;
  }
  if (!store) return;
  if (is_idx) {
    uint8_t* f = c.idx_base + block * c.idx_block_stride;
    if (dtype == BSP_BF16) {
      *reinterpret_cast<uint4*>(f + static_cast<int64_t>(h) * kBf16IndexField + o * 256 + 16 * l) = pack8_bf16(x);
    } else if (dtype == BSP_FP8_E4M3) {
      f += static_cast<int64_t>(h) * kFp8IndexField;
      const float s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], s);
      *reinterpret_cast<uint2*>(f + o * 128 + 8 * l) = pack8_e4m3(x);
      if (l == 0) *reinterpret_cast<float*>(f + kFp8IndexScaleOff + o * 4) = s;
    } else {
      store_mx(f + static_cast<int64_t>(h) * kMxField, o, l, x, amax);
    }
    return;
  }
  uint8_t* base = ty == kHeadK ? c.k_base : c.v_base;
  if (dtype == BSP_MXFP4) {
    store_mx(base + block * c.id_stride + static_cast<int64_t>(h) * kMxField, o, l, x, amax);
    return;
  }
  uint8_t* page = base + (block * 16 + o / kPage) * c.id_stride;
  const int t = o % kPage;
  if (dtype == BSP_FP8_E4M3) {
    page += static_cast<int64_t>(h) * 2048;
    const float sc = ty == kHeadK ? c.k_scale : c.v_scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], sc);
    const uint2 v = pack8_e4m3(x);
    if (ty == kHeadK) {  // [d/16][t][16]
      *reinterpret_cast<uint2*>(page + (l >> 1) * 256 + t * 16 + (l & 1) * 8) = v;
    } else {  // [d][16 t]
#pragma unroll
      for (int j = 0; j < 8; ++j) page[(8 * l + j) * 16 + t] = static_cast<uint8_t>((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
    }
  } else {
    uint16_t* pg = reinterpret_cast<uint16_t*>(page + static_cast<int64_t>(h) * 4096);
    const uint4 v = pack8_bf16(x);
    if (ty == kHeadK) {  // [d/8][t][8]
      *reinterpret_cast<uint4*>(pg + l * 128 + t * 8) = v;
    } else {  // [t/8][d][8]
      const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        pg[(t >> 3) * 1024 + (8 * l + j) * 8 + (t & 7)] = static_cast<uint16_t>(vv[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// what the heads of a half-warp's token share
struct Token {
  int64_t token, slot;
  bool live, pad;    // pad: zeros out, nothing stored
  bool turns;        // the lane's dims are rotated
  int l, partner;    // lane of the half-warp; the lane that holds the pairs' other dims
  float cs[8], sn[8];
};

__device__ __forceinline__ Token load_token(const NormRopeParams& p, int64_t mine) {
  Token t;
  t.l = threadIdx.x & 15;
  t.live = mine < p.num_tokens;
  t.token = t.live ? mine : 0;  // the shuffles need every lane
  const int32_t pos = p.positions ? p.positions[t.token] : 0;
  t.slot = p.slot ? p.slot[t.token] : -1;
  t.pad = pos < 0;
  if (p.rot_dim && pos >= p.rope_rows) {
    if (t.l == 0 && t.live) set_err(p.err, BSP_DEVERR_POSITION);
    t.pad = true;
  }
  // cosines and sines of this lane's dims: halves, dims d and d + rot/2 share
  // entry d % (rot/2), the first of a pair takes the sine negated; adjacent pairs,
  // dims 2i and 2i+1 share entry i
  const int hl = p.rot_dim >> 4;  // lanes of half the rotated dims
  t.turns = t.l < 2 * hl;
  t.partner = threadIdx.x & 31;
  if (t.turns && !t.pad) {
    const float* row = p.rope + static_cast<int64_t>(pos) * p.rot_dim;
    if (p.rope_pairs) {
      const float4 c = *reinterpret_cast<const float4*>(row + 4 * t.l);
      const float4 s = *reinterpret_cast<const float4*>(row + (p.rot_dim >> 1) + 4 * t.l);
      t.cs[0] = t.cs[1] = c.x, t.cs[2] = t.cs[3] = c.y, t.cs[4] = t.cs[5] = c.z, t.cs[6] = t.cs[7] = c.w;
      t.sn[1] = s.x, t.sn[3] = s.y, t.sn[5] = s.z, t.sn[7] = s.w;
      t.sn[0] = -s.x, t.sn[2] = -s.y, t.sn[4] = -s.z, t.sn[6] = -s.w;
    } else {
      const float* c = row + 8 * (t.l < hl ? t.l : t.l - hl);
      const float* s = c + (p.rot_dim >> 1);
      *reinterpret_cast<float4*>(t.cs) = *reinterpret_cast<const float4*>(c);
      *reinterpret_cast<float4*>(t.cs + 4) = *reinterpret_cast<const float4*>(c + 4);
      *reinterpret_cast<float4*>(t.sn) = *reinterpret_cast<const float4*>(s);
      *reinterpret_cast<float4*>(t.sn + 4) = *reinterpret_cast<const float4*>(s + 4);
      if (t.l < hl) {
#pragma unroll
        for (int j = 0; j < 8; ++j) t.sn[j] = -t.sn[j];
      }
    }
  }
  if (t.turns && !p.rope_pairs) t.partner += t.l < hl ? hl : -hl;
  return t;
}

__device__ __forceinline__ void load_weights(const NormRopeParams& p, int ty, int l, float (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.f;
  if (p.weight[ty]) {
    unpack8(*reinterpret_cast<const uint4*>(p.weight[ty] + 8 * l), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] += p.weight_offset;
  }
}

template <int kHeads>
__device__ __forceinline__ void load_heads(const NormRopeParams& p, int ty, int h0, const Token& t, uint4 (&raw)[kHeads]) {
  const uint16_t* src = p.src[ty] + t.token * p.stride[ty] + h0 * kDim + 8 * t.l;
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    raw[i] = h0 + i < p.heads[ty] ? *reinterpret_cast<const uint4*>(src + i * kDim) : make_uint4(0, 0, 0, 0);
}

// What the heads of one type share.
struct Type {
  int ty, heads;
  bool normed, bf16, cached;
  uint8_t* out;  // the lane's place in head 0, NULL: none
};
__device__ __forceinline__ Type type_of(const NormRopeParams& p, int ty, const Token& t) {
  Type a;
  a.ty = ty, a.heads = p.heads[ty];
  a.normed = ty != kHeadV, a.bf16 = p.out_dtype[ty] == BSP_BF16;
  a.cached = ty == kHeadIdxK ? p.cache.idx_base != nullptr : (ty == kHeadK || ty == kHeadV) && p.cache.k_base;
  a.out = static_cast<uint8_t*>(p.out[ty]);
  if (!t.live) a.out = nullptr;
  if (a.out) a.out += (t.token * a.heads * kDim + 8 * t.l) * (a.bf16 ? 2 : 1);
  return a;
}

// sum of x^2 over the head, in every lane
__device__ __forceinline__ float sum_squares(const float (&x)[8]) {
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 8; j += 2) s2 = ffma2({x[j], x[j + 1]}, {x[j], x[j + 1]}, s2);
  float ss = s2.x + s2.y;
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  return ss;
}

// norm, weight and rotation of a head.  The weight (of bf16 values, exact or nearly)
// and the rotation come first: neither waits for the mean, and the one factor at the
// end rounds once.
template <bool PAIRS>
__device__ __forceinline__ void norm_rotate(const NormRopeParams& p, const Token& t, const float (&w)[8], float (&x)[8]) {
  float m = fmaf(sum_squares(x), 1.f / kDim, p.eps);
  // Rows of such a size that squares, or products with the weight, would leave fp32's
  // range are brought to an ordinary one first, by a power of two, exactly.
  constexpr uint32_t kLow = (127u - 80) << 23, kHigh = (127u + 80) << 23;
  const bool odd = __float_as_uint(m) - kLow >= kHigh - kLow;
  if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
    const float k = !odd ? 1.f : m < 1.f ? 0x1p96f : 0x1p-96f;  // (odd and NaN: any)
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= k;
    m = fmaf(sum_squares(x), 1.f / kDim, p.eps * k * k);
  }
  const float inv = __frsqrt_rn(m);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 y = fmul2({x[j], x[j + 1]}, {w[j], w[j + 1]});
    x[j] = y.x, x[j + 1] = y.y;
  }
  if (p.rot_dim) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = PAIRS ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], t.partner);
    if (t.turns) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 z = ffma2({x[j], x[j + 1]}, {t.cs[j], t.cs[j + 1]}, fmul2({y[j], y[j + 1]}, {t.sn[j], t.sn[j + 1]}));
        x[j] = z.x, x[j + 1] = z.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 y = fmul2({x[j], x[j + 1]}, {inv, inv});
    x[j] = y.x, x[j + 1] = y.y;
  }
}

// heads h0 .. of a type: norm, rotation, stores.  The type and head are the
// same for the whole warp.  QUERY: neither V nor cached.
template <bool PAIRS, bool QUERY, int kHeads>
__device__ __forceinline__ void put_heads(const NormRopeParams& p, const Type& a, int h0, const Token& t,
                                          const float (&w)[8], const uint4 (&raw)[kHeads]) {
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (h0 + i >= a.heads) break;
    float x[8];
    unpack8(raw[i], x);
    if (QUERY || a.normed) norm_rotate<PAIRS>(p, t, w, x);
    if (t.pad) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
    if (a.out) {
      if (a.bf16)
        *reinterpret_cast<uint4*>(a.out + (h0 + i) * (kDim * 2)) = pack8_bf16(x);
      else
        *reinterpret_cast<uint2*>(a.out + (h0 + i) * kDim) = pack8_e4m3(x);
    }
    if (!QUERY && a.cached) store_cached(p, a.ty, h0 + i, t.slot, t.live && !t.pad && t.slot >= 0, t.l, x);
  }
}

// Few tokens: a CTA takes one head of eight tokens (latency: everything is in
// flight at once).
template <bool PAIRS>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p, unsigned total) {
  pdl_wait();
  pdl_trigger();
  const unsigned group = blockIdx.x / total;  // of eight tokens
  int ty = 0, h = static_cast<int>(blockIdx.x - group * total);
#pragma unroll
  for (int k = 0; k < kHeadTypes - 1; ++k)
    if (ty == k && h >= p.heads[k]) h -= p.heads[k], ty = k + 1;
  const Token t = load_token(p, static_cast<int64_t>(group) * (kThreads / 16) + (threadIdx.x >> 4));
  uint4 raw[1];
  load_heads(p, ty, h, t, raw);
  float w[8];
  load_weights(p, ty, t.l, w);
  put_heads<PAIRS, false>(p, type_of(p, ty, t), h, t, w, raw);
}

// Many tokens: a half-warp takes all heads of its token, kStep at a time, the next
// in flight: positions, angles and addresses are worked out once a token, and query
// heads go through a loop of their own.  (16456 tokens, us: a head a CTA 60; kStep 2
// at 5, 6, 7 and 8 CTAs an SM 47, 47, 42, 45; kStep 1 and 4 47; the heads shared by
// two or four half-warps 49, 55.  40000 tokens: 92, with loads two steps ahead 97.)
constexpr int kStep = 2;
template <bool PAIRS>
__global__ void __launch_bounds__(kThreads, 7) norm_rope_token_kernel(const __grid_constant__ NormRopeParams p) {
  pdl_wait();
  pdl_trigger();
  const Token t = load_token(p, static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4));
  // the loads, a step before their use: type lty, `left` of its heads from src on
  int lty = -1, left = 0;
  const uint16_t* src = nullptr;
  auto fetch = [&](uint4 (&to)[kStep]) {
    if (left <= 0) {
      do ++lty;
      while (lty < kHeadTypes && p.heads[lty] == 0);
      if (lty >= kHeadTypes) {
        lty = kHeadTypes - 1;  // (nothing more)
        return;
      }
      left = p.heads[lty];
      src = p.src[lty] + t.token * p.stride[lty] + 8 * t.l;
    }
#pragma unroll
    for (int i = 0; i < kStep; ++i)
      if (i < left) to[i] = *reinterpret_cast<const uint4*>(src + i * kDim);
    left -= kStep, src += kStep * kDim;
  };
  uint4 next[kStep];
  fetch(next);
  float w[8];
#pragma unroll 1
  for (int ty = 0; ty < kHeadTypes; ++ty) {
    if (p.heads[ty] == 0) continue;
    const Type a = type_of(p, ty, t);
    load_weights(p, ty, t.l, w);
    auto step = [&](int h, auto query) {
      uint4 raw[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) raw[i] = next[i];
      fetch(next);
      put_heads<PAIRS, query>(p, a, h, t, w, raw);
    };
    if (a.normed && !a.cached) {
#pragma unroll 1
      for (int h = 0; h < a.heads; h += kStep) step(h, std::true_type{});
    } else {
#pragma unroll 1
      for (int h = 0; h < a.heads; h += kStep) step(h, std::false_type{});
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int num_sms, cudaStream_t s) {
  int64_t total = 0;
  for (int k = 0; k < kHeadTypes; ++k) total += p.heads[k];
  if (total == 0 || p.num_tokens == 0) return cudaSuccess;
  const int64_t groups = (static_cast<int64_t>(p.num_tokens) + kThreads / 16 - 1) / (kThreads / 16);
  // All heads of a token in one half-warp, from 2 + 15 / (heads - 4) CTAs an SM on: what
  // a token costs once is spared only with some heads more, and the chain of a token's
  // heads has to fit the batch.  Measured, us, a head a CTA and a token a half-warp:
  //   5 heads    4096 tokens  8.4, 10.1   8192 13.5, 14.2   16456  23.6, 24.6
  //   8 heads    4096        10.1, 11.2   6000 13.2, 14.9    8192  17.1, 15.5
  //   20 heads   2048        10.0, 13.3   3648 15.9, 15.0    8192  33.3, 21.5
  //   40 heads   2560        21.2, 23.8   4096 33.2, 27.1   16456 149.7, 76.9
  //   80 heads   2048        33.1, 42.8   2560 45.2, 45.1    4096  75.2, 54.8
  const int64_t more = total - 4;
  const bool many = more > 0 && groups * more >= num_sms * (2 * more + 15);
  auto launch = [&](auto pairs) {
    return many ? launch_kernel(norm_rope_token_kernel<pairs>, dim3(static_cast<unsigned>(groups)), dim3(kThreads), 0, s,
                                0, p)
                : launch_kernel(norm_rope_kernel<pairs>, dim3(static_cast<unsigned>(groups * total)), dim3(kThreads), 0,
                                s, 0, p, static_cast<unsigned>(total));
  };
  const cudaError_t e = p.rope_pairs ? launch(std::true_type{}) : launch(std::false_type{});
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace bsp
