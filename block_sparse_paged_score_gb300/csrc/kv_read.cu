// kv_read.cu -- the writer's inverse: cached K, V and index keys gathered by
// slot and dequantised to bf16 rows (bsp_kv_page_read, bsp_kv_scaled_read).
//
//   bf16   as stored;  fp8  e4m3 * scale (the cache's, or the block's and head's), rounded to bf16
//   MXFP4  e2m1 * 2^(e8m0 - 127), exact in bf16 (until it leaves its range); NaN for
//          a scale byte 255
//
// One CTA reads 16 consecutive tokens of one head, so that slots which follow
// each other (the usual case: a sequence's page) share sectors.  Rows that
// are contiguous per token (K pages' 16-byte chunks, MXFP4 fields, index
// fields) are read 8 dims a lane, 16 lanes a token.  An interleaved cache's V
// page holds 16 (fp8) or 8 (bf16) tokens of one dim together; there a lane
// is a token, a warp reads two dims at a time, and the tile is turned around
// in shared memory before it is stored in rows.
//
// Sixteen tokens of an fp8 block one behind the other are read with all loads in flight
// at once, V's page rows as 8-byte pieces of a dim's tokens.
//
// Measured (a call of a row of twenty in a graph): 333 fp8 tokens 2.5 us, a launch; 131072 MXFP4
// tokens of a shuffled cache 16.2 us for 86 MB, 5.3 TB/s, 78 % of the copy rate: memory.  131072
// fp8 tokens from offset 5 of a block on, block-scaled: 17.8 us for 102 MB, 5.7 TB/s, 85 % (byte by
// byte 20.7; 19.0 with other inputs each time), 500000 62.9 us, 6.2 TB/s.  Tokens in no order pay
// for the look at their slots: 20000 13.1 us for 12.5, 131072 44.6 for 44.5.
#include "common.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr int kTok = 16;  // tokens of a CTA

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// 8 e4m3 bytes times sc
__device__ __forceinline__ uint4 from_e4m3(uint2 w, float sc) {
  uint32_t h[4], o[4];
  e4m3x4_to_f16x2_cvt(w.x, h[0], h[1]), e4m3x4_to_f16x2_cvt(w.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = fmul2(f16x2_to_float2(h[i]), {sc, sc});
    o[i] = pack_bf16x2(x.x, x.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// dims 8*l.. of token o of an MXFP4 field
__device__ __forceinline__ uint4 from_mx(const uint8_t* field, int o, int l) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(field + o * 64 + 4 * l);
  const uint32_t e = field[kMxScaleOff + o * 4 + (l >> 2)];
  const float sc = e == 255 ? __uint_as_float(0x7FC00000u) : e8m0_to_float(e);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = f16x2_to_float2(e2m1x2_to_f16x2((w >> (8 * i)) & 0xFF));
    x[2 * i] = f.x * sc, x[2 * i + 1] = f.y * sc;
  }
  return pack8(x);
}

__global__ void __launch_bounds__(128) kv_page_read_kernel(KvReadParams p) {
  __shared__ int64_t s_slot[kTok];
  __shared__ __align__(16) uint16_t s_v[kTok][kDim + 8];
  pdl_wait();
  pdl_trigger();
  const KvWriteParams& c = p.cache;
  const int units = (p.k ? c.hkv : 0) + (p.idx_k ? c.hidx : 0);
  const int u = static_cast<int>(blockIdx.x % units);
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x / units) * kTok;
  const bool is_idx = !(p.k && u < c.hkv);
  const int h = is_idx ? u - (p.k ? c.hkv : 0) : u;
  const int tid = threadIdx.x;
  if (tid < kTok) {  // slots outside the cache read as -1
    int64_t slot = tok0 + tid < c.num_tokens ? c.slot[tok0 + tid] : -1;
    if (slot >= (is_idx ? c.idx_num_blocks : c.num_blocks) * kBlock) {
      set_err(c.err, BSP_DEVERR_SLOT);
      slot = -1;
    }
    s_slot[tid] = slot;
  }
  __syncthreads();
  const int l = tid & 15;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  if (!is_idx && c.kv_dtype == BSP_FP8_E4M3) {
    // sixteen tokens of a block, one behind the other?
    const int64_t s0 = s_slot[0];
    if (__all_sync(0xffffffffu, s0 >= 0 && s_slot[l] == s0 + l) && s0 / kBlock == (s0 + kTok - 1) / kBlock) {
      // K and V are on their way together: of K a thread has 8 dims of two tokens, of V two
      // dims of 8 tokens, which begin anywhere in the dims' 8-byte pieces (of one page or two)
      const int64_t block = s0 / kBlock;
      const int o = static_cast<int>(s0 % kBlock), r = o % kPage, j = tid & 63, t0 = tid >> 6 << 3;
      const float ks = p.k_scales ? p.k_scales[block * c.hkv + h] : c.k_scale;
      const float vs = p.v_scales ? p.v_scales[block * c.hkv + h] : c.v_scale;
      const uint8_t* const kp = c.k_base + block * 16 * c.id_stride + static_cast<int64_t>(h) * 2048;
      const uint8_t* const vp = c.v_base + (block * 16 + o / kPage) * c.id_stride + static_cast<int64_t>(h) * 2048 + j * 32;
      uint2 kw[2], va[2], vb[2] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = o + (tid >> 4) + 8 * i;
        kw[i] = *reinterpret_cast<const uint2*>(kp + (t / kPage) * c.id_stride + (l >> 1) * 256 + t % kPage * 16 + (l & 1) * 8);
      }
      const int piece = (r + t0) >> 3;
      const uint8_t* const at = vp + (piece >> 1) * c.id_stride + (piece & 1) * 8;
      const uint8_t* const next = vp + ((piece + 1) >> 1) * c.id_stride + ((piece + 1) & 1) * 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) va[i] = *reinterpret_cast<const uint2*>(at + i * 16);
      if (r & 7) {
#pragma unroll
        for (int i = 0; i < 2; ++i) vb[i] = *reinterpret_cast<const uint2*>(next + i * 16);
      }
      const int64_t row = ((tok0 + (tid >> 4)) * c.hkv + h) * kDim + 8 * l, hop = 8LL * c.hkv * kDim;
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(p.k + row + i * hop) = from_e4m3(kw[i], ks);
      float2 x[2][4];  // of a dim, pairs of tokens
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t y0 = r & 4 ? va[i].y : va[i].x, y1 = r & 4 ? vb[i].x : va[i].y, y2 = r & 4 ? vb[i].y : vb[i].x;
        uint32_t f[4];
        e4m3x4_to_f16x2_cvt(__funnelshift_r(y0, y1, 8 * (r & 3)), f[0], f[1]);
        e4m3x4_to_f16x2_cvt(__funnelshift_r(y1, y2, 8 * (r & 3)), f[2], f[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k] = fmul2(f16x2_to_float2(f[k]), {vs, vs});
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        *reinterpret_cast<uint32_t*>(&s_v[t0 + 2 * k][2 * j]) = pack_bf16x2(x[0][k].x, x[1][k].x);
        *reinterpret_cast<uint32_t*>(&s_v[t0 + 2 * k + 1][2 * j]) = pack_bf16x2(x[0][k].y, x[1][k].y);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4*>(p.v + row + i * hop) = *reinterpret_cast<const uint4*>(&s_v[(tid >> 4) + 8 * i][8 * l]);
      return;
    }
  }

#pragma unroll
  for (int side = 0; side < 2; ++side) {  // K (or the index key), then V
    if (side == 1 && is_idx) break;
    const int dtype = is_idx ? c.idx_dtype : c.kv_dtype;
    uint16_t* out = is_idx ? p.idx_k : (side == 0 ? p.k : p.v);
    const int heads = is_idx ? c.hidx : c.hkv;
    if (side == 1 && dtype != BSP_MXFP4) {
      // V page of an interleaved cache: lane = token, 2 dims a warp at a time
      const int t = tid & 15, dd = tid >> 4;  // dims dd, dd + 8, ...
      const int64_t slot = s_slot[t];
      const int64_t page = slot / kBlock * 16 + slot % kBlock / kPage;
      const int pt = static_cast<int>(slot % kPage);
      if (slot < 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s_v[t][dd + 8 * i] = 0;
      } else if (dtype == BSP_FP8_E4M3) {
        const uint8_t* src = c.v_base + page * c.id_stride + static_cast<int64_t>(h) * 2048 + pt;
        uint8_t b[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = src[(dd + 8 * i) * 16];
        const float sc = p.v_scales ? p.v_scales[slot / kBlock * heads + h] : c.v_scale;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s_v[t][dd + 8 * i] = static_cast<uint16_t>(pack_bf16x2(e4m3_to_float(b[i]) * sc, 0.f));
      } else {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(c.v_base + page * c.id_stride +
                                                                static_cast<int64_t>(h) * 4096) +
                              (pt >> 3) * 1024 + (pt & 7);
        uint16_t b[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = src[(dd + 8 * i) * 8];
#pragma unroll
        for (int i = 0; i < 16; ++i) s_v[t][dd + 8 * i] = b[i];
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tk = (tid >> 4) + 8 * r;
        if (tok0 + tk < c.num_tokens)
          *reinterpret_cast<uint4*>(out + ((tok0 + tk) * heads + h) * kDim + 8 * l) =
              *reinterpret_cast<const uint4*>(&s_v[tk][8 * l]);
      }
      continue;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int tk = (tid >> 4) + 8 * r;
      if (tok0 + tk >= c.num_tokens) continue;
      const int64_t slot = s_slot[tk];
      uint4 w = zero;
      if (slot >= 0) {
        const int64_t block = slot / kBlock;
        const int o = static_cast<int>(slot % kBlock);
        if (is_idx) {
          const uint8_t* f = c.idx_base + block * c.idx_block_stride;
          if (dtype == BSP_BF16) {
            w = *reinterpret_cast<const uint4*>(f + static_cast<int64_t>(h) * kBf16IndexField + o * 256 + 16 * l);
          } else if (dtype == BSP_FP8_E4M3) {
            f += static_cast<int64_t>(h) * kFp8IndexField;
            w = from_e4m3(*reinterpret_cast<const uint2*>(f + o * 128 + 8 * l),
                          *reinterpret_cast<const float*>(f + kFp8IndexScaleOff + o * 4));
          } else {
            w = from_mx(f + static_cast<int64_t>(h) * kMxField, o, l);
          }
        } else if (dtype == BSP_MXFP4) {
          w = from_mx((side == 0 ? c.k_base : c.v_base) + block * c.id_stride + static_cast<int64_t>(h) * kMxField, o,
                      l);
        } else {  // K page [d/x][16 tokens][x]
          const uint8_t* page = c.k_base + (block * 16 + o / kPage) * c.id_stride;
          const int t = o % kPage;
          if (dtype == BSP_FP8_E4M3)
            w = from_e4m3(*reinterpret_cast<const uint2*>(page + static_cast<int64_t>(h) * 2048 + (l >> 1) * 256 +
                                                          t * 16 + (l & 1) * 8),
                          p.k_scales ? p.k_scales[block * heads + h] : c.k_scale);
          else
            w = *reinterpret_cast<const uint4*>(page + static_cast<int64_t>(h) * 4096 + l * 256 + t * 16);
        }
      }
      *reinterpret_cast<uint4*>(out + ((tok0 + tk) * heads + h) * kDim + 8 * l) = w;
    }
  }
}

}  // namespace

cudaError_t launch_kv_page_read(const KvReadParams& p, cudaStream_t s) {
  const int64_t units = (p.k ? p.cache.hkv : 0) + (p.idx_k ? p.cache.hidx : 0);
  const int64_t ctas = (static_cast<int64_t>(p.cache.num_tokens) + kTok - 1) / kTok * units;
  if (ctas == 0) return cudaSuccess;
  const cudaError_t e = launch_kernel(kv_page_read_kernel, dim3(static_cast<unsigned>(ctas)), dim3(128), 0, s, 0, p);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace bsp
