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
// maxima are shuffles within 16 and 4 lanes).  A CTA takes eight tokens, one a
// half-warp, and the same kHeads heads of one type of each: their loads are in
// flight together, the token's cosines and sines and the weights are loaded once,
// and what depends on the type is the same for the whole CTA.
#include <algorithm>

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

template <int kHeads>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p, unsigned chunks) {
  pdl_wait();
  pdl_trigger();
  const int l = threadIdx.x & 15;
  const unsigned group = blockIdx.x / chunks;  // of eight tokens
  const int64_t mine = static_cast<int64_t>(group) * (kThreads / 16) + (threadIdx.x >> 4);
  const bool live = mine < p.num_tokens;
  const int64_t token = live ? mine : 0;  // the shuffles below need every lane
  // the CTA's type and first head
  int ty = 0, h0 = static_cast<int>(blockIdx.x - group * chunks) * kHeads;
#pragma unroll
  for (int k = 0; k < kHeadTypes - 1; ++k) {
    const int n = (p.heads[k] + kHeads - 1) / kHeads * kHeads;
    if (ty == k && h0 >= n) h0 -= n, ty = k + 1;
  }
  const int heads = p.heads[ty];
  const bool normed = ty != kHeadV;
  const uint16_t* src = p.src[ty] + token * p.stride[ty] + static_cast<int64_t>(h0) * kDim + 8 * l;
  uint4 raw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    raw[i] = h0 + i < heads ? *reinterpret_cast<const uint4*>(src + i * kDim) : make_uint4(0, 0, 0, 0);
  const int32_t pos = p.positions ? p.positions[token] : 0;
  const bool cached = ty == kHeadIdxK ? p.cache.idx_base != nullptr : (ty == kHeadK || ty == kHeadV) && p.cache.k_base;
  const int64_t slot = cached ? p.slot[token] : -1;
  float w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.f;
  if (normed && p.weight[ty]) {
    unpack8(*reinterpret_cast<const uint4*>(p.weight[ty] + 8 * l), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] += p.weight_offset;
  }
  bool pad = pos < 0;  // a pad row: zeros out, nothing stored
  if (p.rot_dim && pos >= p.rope_rows) {
    if (l == 0 && live) set_err(p.err, BSP_DEVERR_POSITION);
    pad = true;
  }
  // cosines and sines of this lane's dims: halves, dims d and d + rot/2 share
  // entry d % (rot/2), the first of a pair takes the sine negated; adjacent pairs,
  // dims 2i and 2i+1 share entry i
  const int hl = p.rot_dim >> 4;  // lanes of half the rotated dims
  const bool turns = normed && l < 2 * hl;
  float cs[8], sn[8];
  int partner = threadIdx.x & 31;
  if (turns && !pad) {
    const float* row = p.rope + static_cast<int64_t>(pos) * p.rot_dim;
    if (p.rope_pairs) {
      const float4 c = *reinterpret_cast<const float4*>(row + 4 * l);
      const float4 s = *reinterpret_cast<const float4*>(row + (p.rot_dim >> 1) + 4 * l);
      cs[0] = cs[1] = c.x, cs[2] = cs[3] = c.y, cs[4] = cs[5] = c.z, cs[6] = cs[7] = c.w;
      sn[1] = s.x, sn[3] = s.y, sn[5] = s.z, sn[7] = s.w;
      sn[0] = -s.x, sn[2] = -s.y, sn[4] = -s.z, sn[6] = -s.w;
    } else {
      const float* c = row + 8 * (l < hl ? l : l - hl);
      const float* s = c + (p.rot_dim >> 1);
      *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(c);
      *reinterpret_cast<float4*>(cs + 4) = *reinterpret_cast<const float4*>(c + 4);
      *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(s);
      *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(s + 4);
      if (l < hl) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sn[j] = -sn[j];
      }
    }
  }
  if (turns && !p.rope_pairs) partner += l < hl ? hl : -hl;
  uint8_t* out = static_cast<uint8_t*>(p.out[ty]);
  const bool bf16 = p.out_dtype[ty] == BSP_BF16;
  int64_t e = (token * heads + h0) * kDim + 8 * l;

#pragma unroll
  for (int i = 0; i < kHeads; ++i, e += kDim) {
    if (h0 + i >= heads) break;
    float x[8];
    unpack8(raw[i], x);
    if (normed) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float inv = rsqrtf(fmaf(ss, 1.f / kDim, p.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * w[j];
      if (p.rot_dim) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = p.rope_pairs ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], partner);
        if (turns) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], cs[j], y[j] * sn[j]);
        }
      }
    }
    if (pad) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
    if (out && live) {
      if (bf16)
        *reinterpret_cast<uint4*>(out + 2 * e) = pack8_bf16(x);
      else
        *reinterpret_cast<uint2*>(out + e) = pack8_e4m3(x);
    }
    if (cached) store_cached(p, ty, h0 + i, slot, live && !pad && slot >= 0, l, x);
  }
}

template <int kHeads>
cudaError_t launch_heads(const NormRopeParams& p, cudaStream_t s) {
  int64_t chunks = 0;  // of heads of one type
  for (int k = 0; k < kHeadTypes; ++k) chunks += (p.heads[k] + kHeads - 1) / kHeads;
  const int64_t ctas = (static_cast<int64_t>(p.num_tokens) + kThreads / 16 - 1) / (kThreads / 16) * chunks;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = launch_kernel(norm_rope_kernel<kHeads>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s,
                                      0, p, static_cast<unsigned>(chunks));
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int num_sms, cudaStream_t s) {
  int64_t total = 0;
  for (int k = 0; k < kHeadTypes; ++k) total += p.heads[k];
  if (total == 0 || p.num_tokens == 0) return cudaSuccess;
  // one head a half-warp while that fills less than two waves of half-warps
  // (128 an SM), else four
  const bool few = total * p.num_tokens <= static_cast<int64_t>(num_sms) * 256;
  return few ? launch_heads<1>(p, s) : launch_heads<4>(p, s);
}

}  // namespace bsp
