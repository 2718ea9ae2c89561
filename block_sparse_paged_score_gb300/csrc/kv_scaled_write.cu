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
// A run, a head and a side have one owner, so that no two touch the same bytes or
// scale: a CTA, or of short runs that lie close together a warp.  It is found by the
// run's first token (the one before lies in another block).  In a CTA, which token of
// the run is at which offset goes to a table in shared memory, so that the bytes are
// made page by page however the tokens are ordered.  The run's rows stay in registers
// between the maximum and the bytes: of K a thread has 8 dims of a token of each page,
// of V two dims of the 32 tokens of two pages, which its pages hold side by side, so
// that both leave as vectors.
//
// Measured (a call of a row of twenty in a graph, warm, no scale growing): 64 decode tokens of
// a head 3.8 us, a launch; 8 prompts of 300 to 2400 tokens, two heads, 10.8 us for 17 MB.  There a
// run's chain of dependent steps is what it takes (slots, table, rows, maximum, bytes), not
// bandwidth: loading a run's slots at once, and more tokens a CTA, did not shorten it.  What
// growing scales add is beside the launch.
#include "common.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kShort = 8;  // tokens of a run that a warp takes
constexpr int kCtasPerSm = 4;

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

// what a CTA works on: a head of K or of V
struct Side {
  const uint16_t* src;  // rows, `stride` apart
  int64_t stride;
  uint8_t* base;        // of the head's pages
  float* scales;        // of the head, hkv apart
  bool v;
};

// four e4m3 bytes times f, rounded again
__device__ __forceinline__ uint32_t times(uint32_t w, float f) {
  uint32_t l, h;
  e4m3x4_to_f16x2_cvt(w, l, h);
  const float2 x = fmul2(f16x2_to_float2(l), {f, f}), y = fmul2(f16x2_to_float2(h), {f, f});
  return float2_to_e4m3x2(x.x, x.y) | float2_to_e4m3x2(y.x, y.y) << 16;
}
// A block's bytes in a new scale's terms: 16-byte chunks first, first + step .. of 1024.
__device__ __forceinline__ void rescale_block(uint8_t* block, int64_t id_stride, float f, int first, int step) {
#pragma unroll 4
  for (int c = first; c < 1024; c += step) {
    uint4* at = reinterpret_cast<uint4*>(block + (c >> 7) * id_stride) + (c & 127);
    const uint4 w = *at;
    *at = make_uint4(times(w.x, f), times(w.y, f), times(w.z, f), times(w.w, f));
  }
}
// (out of the way: a division's code at each use would be most of the kernel's 100 KB)
__device__ __noinline__ uint32_t divided(float u, float v, float s) { return float2_to_e4m3x2(u / s, v / s); }
// two of a run's bytes, of the scale s
struct Encode {
  float s, inv;
  bool pow2;
  __device__ __forceinline__ uint32_t operator()(float u, float v) const {
    return pow2 ? float2_to_e4m3x2(u * inv, v * inv) : divided(u, v, s);
  }
};
__device__ __forceinline__ Encode encode_by(float s) { return {s, 1.f / s, (__float_as_uint(s) & 0x7FFFFFu) == 0}; }
__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// the larger of top and the finite magnitudes (as bits) of two bf16
__device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) {
  const uint32_t u = w & 0x7FFFu, v = w >> 16 & 0x7FFFu;
  if (u < 0x7F80u) top = max(top, u);
  if (v < 0x7F80u) top = max(top, v);
  return top;
}

// A run of at most kShort tokens, from token i on, by a warp: a lane has four dims.
__device__ __forceinline__ void write_short(const KvScaledWriteParams& p, const Side& d, int64_t i, int n, int lane) {
  const int64_t slot = lane < n ? p.slot[i + lane] : -1 - lane, b = __shfl_sync(0xffffffffu, slot, 0) / kBlock;
  float* const scale_at = d.scales + b * p.hkv;
  const float old = *scale_at;
  // of tokens with the same slot the last one counts
  const uint32_t same = __match_any_sync(0xffffffffu, slot);
  const uint32_t live = __ballot_sync(0xffffffffu, lane < n && 31 - __clz(same) == lane);
  uint2 x[kShort];
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kShort; ++k) {
    x[k] = make_uint2(0, 0);
    if (live >> k & 1) x[k] = *reinterpret_cast<const uint2*>(d.src + (i + k) * d.stride + 4 * lane);
  }
#pragma unroll
  for (int k = 0; k < kShort; ++k) top = larger(larger(top, x[k].x), x[k].y);
  top = __reduce_max_sync(0xffffffffu, top);
  const bool anew = __any_sync(0xffffffffu, lane < n && slot % kBlock == 0);
  const float run = scale_for(__uint_as_float(top << 16)), s = anew ? run : fmaxf(old, run);
  __syncwarp();  // (every lane has the old one)
  if (lane == 0) *scale_at = s;
  uint8_t* const block = d.base + b * 16 * p.id_stride;
  if (!anew && !(s <= old)) {
    rescale_block(block, p.id_stride, old / s, lane, 32);
    __syncwarp();
  }
  const Encode bytes = encode_by(s);
#pragma unroll
  for (int k = 0; k < kShort; ++k) {
    if (!(live >> k & 1)) continue;
    const int o = static_cast<int>(__shfl_sync(0xffffffffu, slot, k) % kBlock), t = o % kPage;
    uint8_t* const page = block + o / kPage * p.id_stride;
    const uint32_t w = bytes(lo(x[k].x), hi(x[k].x)) | bytes(lo(x[k].y), hi(x[k].y)) << 16;
    if (!d.v) {  // K page [128 / 16][16 tokens][16]
      *reinterpret_cast<uint32_t*>(page + (lane >> 2) * 256 + t * 16 + (lane & 3) * 4) = w;
    } else {  // V page [128][16 tokens]
#pragma unroll
      for (int j = 0; j < 4; ++j) page[(4 * lane + j) * 16 + t] = static_cast<uint8_t>(w >> (8 * j));
    }
  }
}

// (four CTAs an SM: most begin no run, and leave; with three, of 80 registers, 8 prompts of 300 to
// 2400 tokens take 15.4 us of a graph's replay for 14.2, with five 15.7; four spill 32 bytes, five more)
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_scaled_write_kernel(KvScaledWriteParams p, int per) {
  __shared__ int s_at[kBlock];  // token of an offset, + 1
  __shared__ int s_end;
  __shared__ uint32_t s_long, s_short;  // the CTA's tokens that begin a run
  __shared__ int s_len[32];
  __shared__ uint32_t s_top[kWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const Side d{(is_v ? p.src[1] : p.src[0]) + h * kDim, is_v ? p.stride[1] : p.stride[0],
               (is_v ? p.base[1] : p.base[0]) + static_cast<int64_t>(h) * 2048, (is_v ? p.scales[1] : p.scales[0]) + h, is_v};
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per;
  if (tid < 32) {
    const int64_t i = first + lane;
    int len = 0;
    if (lane < per && i < p.num_tokens) {
      const int64_t b = block_of(p, i);
      if (b < 0 && p.slot[i] >= 0) set_err(p.err, BSP_DEVERR_SLOT);
      if (b >= 0 && (i == 0 || block_of(p, i - 1) != b))
        for (len = 1; len <= kShort && i + len < p.num_tokens && block_of(p, i + len) == b;) ++len;
    }
    // (a single run takes all warps: most of its time may be its block's new scale)
    const uint32_t runs = __ballot_sync(0xffffffffu, len > 0);
    const uint32_t brief = __popc(runs) > 1 ? __ballot_sync(0xffffffffu, len > 0 && len <= kShort) : 0;
    s_len[lane] = len;
    if (lane == 0) s_long = runs & ~brief, s_short = brief;
  }
  __syncthreads();
#pragma unroll 1
  for (uint32_t left = s_short, k = 0; left; left &= left - 1, ++k) {
    const int at = __ffs(left) - 1;
    if (k % kWarps == static_cast<uint32_t>(warp)) write_short(p, d, first + at, s_len[at], lane);
  }
#pragma unroll 1
  for (uint32_t left = s_long; left; left &= left - 1) {
    const int64_t i = first + __ffs(left) - 1, b = p.slot[i] / kBlock;
    // the run's tokens by offset (the last of a slot)
    if (tid < kBlock) s_at[tid] = 0;
    int64_t at = i;
    int end;
    do {
      if (tid == 0) s_end = kThreads;
      __syncthreads();
      const int64_t j = at + tid;
      const bool in = j < p.num_tokens && block_of(p, j) == b;
      if (!in) atomicMin(&s_end, tid);
      __syncthreads();
      end = s_end;
      if (tid < end) atomicMax(&s_at[p.slot[j] % kBlock], static_cast<int>(j) + 1);
      at += end;
      __syncthreads();
    } while (end == kThreads);
    float* const scale_at = d.scales + b * p.hkv;
    const float old = *scale_at;
    // the rows and their largest magnitude
    uint32_t x[32], top = 0;
    const int l = tid & 15, t16 = tid >> 4, dims = 2 * (tid & 63), page0 = tid >> 6 << 1;
    if (!d.v) {
#pragma unroll
      for (int g = 0; g < kPagesPerSide; ++g) {  // 16 lanes a token
        const int64_t tok = s_at[kPage * g + t16] - 1;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (tok >= 0) w = *reinterpret_cast<const uint4*>(d.src + tok * d.stride + 8 * l);
        x[4 * g] = w.x, x[4 * g + 1] = w.y, x[4 * g + 2] = w.z, x[4 * g + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2 * kPage; ++k) {  // 64 threads a token
        const int64_t tok = s_at[kPage * page0 + k] - 1;
        x[k] = 0;
        if (tok >= 0) x[k] = *reinterpret_cast<const uint32_t*>(d.src + tok * d.stride + dims);
      }
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) top = larger(top, x[k]);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) top = max(top, s_top[k]);
    const bool anew = s_at[0] > 0;
    const float run = scale_for(__uint_as_float(top << 16)), s = anew ? run : fmaxf(old, run);
    if (tid == 0) *scale_at = s;
    uint8_t* const block = d.base + b * 16 * p.id_stride;
    if (!anew && !(s <= old)) {  // what the block holds, in the new scale's terms
      rescale_block(block, p.id_stride, old / s, tid, kThreads);
      __syncthreads();
    }
    const Encode bytes = encode_by(s);
    if (!d.v) {
#pragma unroll
      for (int g = 0; g < kPagesPerSide; ++g) {  // K page [128 / 16][16 tokens][16]
        if (s_at[kPage * g + t16] == 0) continue;
        const uint32_t* w = x + 4 * g;
        *reinterpret_cast<uint2*>(block + g * p.id_stride + (l >> 1) * 256 + t16 * 16 + (l & 1) * 8) =
            make_uint2(bytes(lo(w[0]), hi(w[0])) | bytes(lo(w[1]), hi(w[1])) << 16,
                       bytes(lo(w[2]), hi(w[2])) | bytes(lo(w[3]), hi(w[3])) << 16);
      }
    } else {
#pragma unroll
      for (int g = 0; g < 2; ++g) {  // V page [128][16 tokens]
        uint8_t* const to = block + (page0 + g) * p.id_stride + dims * 16;
        uint32_t d0[4], d1[4];
        bool all = true, any = false;
#pragma unroll
        for (int t = 0; t < kPage; ++t) {
          const bool here = s_at[kPage * (page0 + g) + t] > 0;
          all &= here, any |= here;
        }
        if (!any) continue;
#pragma unroll
        for (int t = 0; t < kPage; t += 4) {
          const uint32_t* w = x + kPage * g + t;
          d0[t / 4] = bytes(lo(w[0]), lo(w[1])) | bytes(lo(w[2]), lo(w[3])) << 16;
          d1[t / 4] = bytes(hi(w[0]), hi(w[1])) | bytes(hi(w[2]), hi(w[3])) << 16;
        }
        if (all) {
          reinterpret_cast<uint4*>(to)[0] = make_uint4(d0[0], d0[1], d0[2], d0[3]);
          reinterpret_cast<uint4*>(to)[1] = make_uint4(d1[0], d1[1], d1[2], d1[3]);
        } else {
#pragma unroll
          for (int t = 0; t < kPage; ++t)
            if (s_at[kPage * (page0 + g) + t] > 0) {
              to[t] = static_cast<uint8_t>(d0[t / 4] >> (8 * (t & 3)));
              to[16 + t] = static_cast<uint8_t>(d1[t / 4] >> (8 * (t & 3)));
            }
        }
      }
    }
    __syncthreads();  // the table may be made anew
  }
}

}  // namespace

cudaError_t launch_kv_scaled_write(const KvScaledWriteParams& p, int num_sms, cudaStream_t s) {
  // A token a CTA while the CTAs are resident together, so that a decode token's block has
  // eight warps for its new scale; else 32, whose runs share the warps.  us of a graph's replay
  // of one call (cold L2, from event to event), a token a CTA and 32, where no block's scale grows, one in
  // eight, all: 64 tokens of a head 12, 17 / 14, 48 / 14, 49; 256 15, 17 / 17, 49 / 17, 51; 304 15, 17 /
  // 17, 49 / 18, 50; 320 16, 17 / 18.5, 49 / 20.5, 51; 512 18, 17 / 21, 49 / 25, 51; 1024 26, 17 / 29, 49 /
  // 36, 53; heads count as tokens do (64 of four as 256).  A prompt of 16000 tokens 56, 17.
  const int per = static_cast<int64_t>(p.num_tokens) * p.hkv * 2 <= int64_t{kCtasPerSm} * num_sms ? 1 : 32;
  const dim3 grid(static_cast<unsigned>((p.num_tokens + per - 1) / per), static_cast<unsigned>(p.hkv), 2);
  const cudaError_t e = launch_kernel(kv_scaled_write_kernel, grid, dim3(kThreads), 0, s, 0, p, per);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace bsp
