// dense_pa.cu -- dense grouped-query attention over an MXFP4 paged cache
// (bsp_dense_pa_decode): o = softmax(scale q K^T) V over the first L_r tokens
// of row r's sequence.  One CTA per row, tiles of 32 tokens dequantised into
// shared memory, running maximum and sum per head.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr int kTile = 32;

__device__ __forceinline__ void load_tile(const uint8_t* field, int o0, float (*dst)[kDim + 1]) {
  // 128 threads: thread = (token, quarter of the dims)
  const int t = threadIdx.x >> 2, g = threadIdx.x & 3;
  const uint4 w = *reinterpret_cast<const uint4*>(field + (o0 + t) * 64 + g * 16);
  const float sc = e8m0_to_float(field[kMxScaleOff + (o0 + t) * 4 + g]);
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 f = f16x2_to_float2(e2m1x2_to_f16x2((ws[i >> 2] >> (8 * (i & 3))) & 0xFF));
    dst[t][g * 32 + 2 * i] = f.x * sc;
    dst[t][g * 32 + 2 * i + 1] = f.y * sc;
  }
}

__global__ void __launch_bounds__(128) dense_pa_kernel(DensePaParams p) {
  __shared__ float sq[16][kDim], sk[kTile][kDim + 1], sv[kTile][kDim + 1], ss[16][kTile], sm[16], sl[16], sa[16];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, row = blockIdx.x, h = row % p.hkv;
  const int64_t token = row / p.hkv, hq = static_cast<int64_t>(p.hkv) * p.group;
  const int64_t q0 = (token * hq + static_cast<int64_t>(h) * p.group) * kDim;
  const int first = static_cast<int>(token / p.q_group * p.q_group) * p.hkv;  // the group's first row
  const int seq = p.row_seq[first];
  if (tid == 0 && p.row_seq[row] != seq) set_err(p.err, BSP_DEVERR_GROUP_SEQ);
  const int64_t L = min(static_cast<int64_t>(max(p.row_len[row], 0)), static_cast<int64_t>(p.bt_stride) * kBlock);
  for (int i = tid; i < 16 * kDim; i += 128) {
    const int hh = i / kDim;
    float x = 0.f;
    if (hh < p.group)
      x = p.q_dtype == BSP_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p.q)[q0 + i])
                                : e4m3_to_float(static_cast<const uint8_t*>(p.q)[q0 + i]);
    sq[hh][i % kDim] = x * p.sm_scale;
  }
  if (tid < 16) sm[tid] = -INFINITY, sl[tid] = 0.f;
  float o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  for (int64_t t0 = 0; t0 < L; t0 += kTile) {
    const int64_t b = p.block_table[static_cast<int64_t>(seq) * p.bt_stride + t0 / kBlock];
    if (b < 0 || b >= p.num_blocks) {  // the block's tokens are left out
      if (tid == 0) set_err(p.err, BSP_DEVERR_BLOCK_ID);
      continue;
    }
    __syncthreads();
    const int64_t f = b * p.id_stride + static_cast<int64_t>(h) * kMxField;
    load_tile(p.k_base + f, static_cast<int>(t0 % kBlock), sk);
    load_tile(p.v_base + f, static_cast<int>(t0 % kBlock), sv);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int hh = (tid >> 5) + 4 * r, t = tid & 31;
      float z = 0.f;
      for (int d = 0; d < kDim; ++d) z += sq[hh][d] * sk[t][d];
      if (t0 + t >= L) z = -INFINITY;
      float mx = z;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
      const float mo = sm[hh], mn = fmaxf(mo, mx);  // every tile has a token below L: mn is finite
      const float pr = expf(z - mn);
      float sum = pr;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      ss[hh][t] = pr;
      __syncwarp();
      if (t == 0) {
        sa[hh] = expf(mo - mn);
        sl[hh] = sl[hh] * sa[hh] + sum;
        sm[hh] = mn;
      }
    }
    __syncthreads();
#pragma unroll
    for (int hh = 0; hh < 16; ++hh) o[hh] *= sa[hh];
    for (int t = 0; t < kTile && t0 + t < L; ++t) {
      const float v = sv[t][tid];
#pragma unroll
      for (int hh = 0; hh < 16; ++hh) o[hh] += ss[hh][t] * v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int hh = 0; hh < 16; ++hh)
    if (hh < p.group)
      static_cast<__nv_bfloat16*>(p.out)[q0 + hh * kDim + tid] =
          __float2bfloat16_rn(sl[hh] > 0.f ? o[hh] / sl[hh] : 0.f);
}

}  // namespace

size_t dense_pa_ws_bytes(int32_t num_rows, int32_t hkv, int32_t group, int32_t q_group, int num_sms) {
  (void)num_rows, (void)hkv, (void)group, (void)q_group, (void)num_sms;
  return 0;
}

cudaError_t launch_dense_pa(const DensePaParams& p, int num_sms, cudaStream_t s, int* launches) {
  (void)num_sms;
  if (p.num_rows == 0) return cudaSuccess;
  const cudaError_t e =
      launch_kernel(dense_pa_kernel, dim3(static_cast<unsigned>(p.num_rows)), dim3(128), 0, s, 0, p);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaPeekAtLastError();
}

}  // namespace bsp
