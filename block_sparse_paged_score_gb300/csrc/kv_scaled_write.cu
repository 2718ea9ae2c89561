// kv_scaled_write.cu -- new tokens into an fp8 cache whose scales are per block and
// head (bsp_kv_scaled_write).
//
//   a = max |x| over the run's rows,  s_run = 2^e, the least with a <= 448 * 2^e
//   s = s_run (the run holds offset 0) or max(s_run, the block's scale)
//   byte = e4m3(x / s);  where s grew, the block's other bytes = e4m3(byte * old / s)
//
// Scales are powers of two: e4m3 is a floating format, so a finer scale would hold no
// value better, and a growing one moves the bytes by whole exponents, exactly until
// they become subnormal.  What is written token by token is what a whole block at
// once gives, but for those.
//
// A CTA owns a run, a head and a side: no two CTAs touch the same bytes or scale.  It
// is found by its first token (the one before lies in another block); which token of
// the run is at which offset goes to a table in shared memory, so that the bytes are
// made page by page however the tokens are ordered, and V's pages, 16 tokens of a dim
// side by side, leave as 16-byte stores.
#include "common.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr int kThreads = 256;

// the block of token i, -1 for a skipped one
__device__ __forceinline__ int64_t block_of(const KvScaledWriteParams& p, int64_t i) {
  const int64_t slot = p.slot[i];
  return slot >= 0 && slot < p.num_blocks * kBlock ? slot / kBlock : -1;
}

// The least power of two s with a <= 448 s (448 = 1.75 * 2^8), within 2^-60 .. 2^119.
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t b = __float_as_uint(a);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u);
  return __uint_as_float(static_cast<uint32_t>(max(-60, min(119, e)) + 127) << 23);
}

__global__ void __launch_bounds__(kThreads) kv_scaled_write_kernel(KvScaledWriteParams p, int per) {
  __shared__ int s_at[kBlock];  // token of an offset, + 1
  __shared__ int s_end;
  __shared__ float s_top[kThreads / 32];
  __shared__ __align__(16) uint8_t s_v[kDim][16];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, l = tid & 15, t16 = tid >> 4;
  const int h = blockIdx.y, side = blockIdx.z;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per;
#pragma unroll 1
  for (int64_t i = first; i < min(first + per, static_cast<int64_t>(p.num_tokens)); ++i) {
    const int64_t b = block_of(p, i);
    if (b < 0) {
      if (tid == 0 && p.slot[i] >= 0) set_err(p.err, BSP_DEVERR_SLOT);
      continue;
    }
    if (i > 0 && block_of(p, i - 1) == b) continue;
    // the run's tokens by offset (the last of a slot)
    __syncthreads();
    if (tid < kBlock) s_at[tid] = 0;
    int64_t at = i;
    do {
      if (tid == 0) s_end = kThreads;
      __syncthreads();
      const int64_t j = at + tid;
      if (j >= p.num_tokens || block_of(p, j) != b) atomicMin(&s_end, tid);
      __syncthreads();
      if (tid < s_end) atomicMax(&s_at[p.slot[j] % kBlock], static_cast<int>(j) + 1);
      at += s_end;
      __syncthreads();
    } while (s_end == kThreads);
    // the rows, 16 lanes a token, and their largest magnitude
    uint4 x[kPagesPerSide];
    uint32_t top = 0;
#pragma unroll
    for (int g = 0; g < kPagesPerSide; ++g) {
      const int tok = s_at[kPage * g + t16] - 1;
      x[g] = make_uint4(0, 0, 0, 0);
      if (tok >= 0)
        x[g] = *reinterpret_cast<const uint4*>(p.src[side] + tok * p.stride[side] + h * kDim + 8 * l);
    }
#pragma unroll
    for (int g = 0; g < kPagesPerSide; ++g) {
      const uint32_t w[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t m = (k & 1 ? w[k >> 1] >> 16 : w[k >> 1]) & 0x7FFFu;
        if (m < 0x7F80u) top = max(top, m);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) s_top[tid >> 5] = __uint_as_float(top << 16);
    float* const scale_at = p.scales[side] + b * p.hkv + h;
    const float old = *scale_at;
    __syncthreads();
    float a = s_top[0];
#pragma unroll
    for (int k = 1; k < kThreads / 32; ++k) a = fmaxf(a, s_top[k]);
    const bool anew = s_at[0] > 0;
    const float run = scale_for(a), s = anew ? run : fmaxf(old, run);
    if (tid == 0) *scale_at = s;
    uint8_t* const block = p.base[side] + b * 16 * p.id_stride + static_cast<int64_t>(h) * 2048;
    if (!anew && !(s <= old)) {  // what the block holds, in the new scale's terms
      const float f = old / s;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = tid + kThreads * k;
        uint4* at16 = reinterpret_cast<uint4*>(block + (c >> 7) * p.id_stride) + (c & 127);
        uint4 w = *at16;
        uint32_t* ws = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int n = 0; n < 4; ++n)
          ws[n] = float2_to_e4m3x2(e4m3_to_float(ws[n]) * f, e4m3_to_float(ws[n] >> 8) * f) |
                  float2_to_e4m3x2(e4m3_to_float(ws[n] >> 16) * f, e4m3_to_float(ws[n] >> 24) * f) << 16;
        *at16 = w;
      }
      __syncthreads();
    }
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
    const float inv = 1.f / s;
#pragma unroll
    for (int g = 0; g < kPagesPerSide; ++g) {
      const bool here = s_at[kPage * g + t16] > 0;
      const int n = __syncthreads_count(here);
      if (n == 0) continue;
      const uint32_t w[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float u = __uint_as_float(w[k] << 16), v = __uint_as_float(w[k] & 0xFFFF0000u);
        r[k] = pow2 ? float2_to_e4m3x2(u * inv, v * inv) : float2_to_e4m3x2(u / s, v / s);
      }
      uint8_t* const page = block + g * p.id_stride;
      if (side == 0) {  // K page [128 / 16][16 tokens][16]
        if (here)
          *reinterpret_cast<uint2*>(page + (l >> 1) * 256 + t16 * 16 + (l & 1) * 8) =
              make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
        continue;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s_v[8 * l + k][t16] = static_cast<uint8_t>(r[k >> 1] >> (8 * (k & 1)));
      __syncthreads();
      if (n == kThreads) {  // V page [128][16 tokens], all of them new
        if (tid < kDim) reinterpret_cast<uint4*>(page)[tid] = *reinterpret_cast<const uint4*>(s_v[tid]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int d = 16 * k + (tid >> 4), t = tid & 15;
          if (s_at[kPage * g + t] > 0) page[d * 16 + t] = s_v[d][t];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_scaled_write(const KvScaledWriteParams& p, int num_sms, cudaStream_t s) {
  // a token a CTA while that is at most some waves of CTAs; else 16 (most of which begin no run)
  const int per = static_cast<int64_t>(p.num_tokens) * p.hkv * 2 <= 32LL * num_sms ? 1 : 16;
  const dim3 grid(static_cast<unsigned>((p.num_tokens + per - 1) / per), static_cast<unsigned>(p.hkv), 2);
  const cudaError_t e = launch_kernel(kv_scaled_write_kernel, grid, dim3(kThreads), 0, s, 0, p, per);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace bsp
