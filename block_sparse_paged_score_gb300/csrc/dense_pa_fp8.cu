// dense_pa_fp8.cu -- dense grouped-query attention over an fp8 paged cache
// (bsp_dense_pa_decode_fp8): a warp per query head and row, a key at a time.
#include "common.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(128) dense_pa_fp8_kernel(DensePaFp8Params p) {
  pdl_wait();
  pdl_trigger();
  const DensePaParams& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);  // token * heads + head
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  if (w >= a.num_rows / a.hkv * hq) return;
  const int64_t tok = w / hq, row = tok * a.hkv + w % hq / a.group;
  const int h = static_cast<int>(w % hq) / a.group;
  const int64_t first = tok / a.q_group * a.q_group * a.hkv;
  const int seq = a.row_seq[first];
  if (a.row_seq[row] != seq) set_err(a.err, BSP_DEVERR_GROUP_SEQ);
  const int64_t len = min(static_cast<int64_t>(max(a.row_len[row], 0)), static_cast<int64_t>(a.bt_stride) * kBlock);
  float q[4], o[4] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t e = w * kDim + 4 * lane + i;
    q[i] = a.q_dtype == BSP_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.q)[e])
                                 : e4m3_to_float(static_cast<const uint8_t*>(a.q)[e]);
  }
  int64_t id = 0;
  float ks = 0.f, vs = 0.f;
  for (int64_t t = 0; t < len; ++t) {
    if (t % kBlock == 0) {
      id = a.block_table[static_cast<int64_t>(seq) * a.bt_stride + t / kBlock];
      if (id < 0 || id >= a.num_blocks) {
        set_err(a.err, BSP_DEVERR_BLOCK_ID);
        t += kBlock - 1;
        continue;
      }
      ks = p.k_scales ? p.k_scales[id * a.hkv + h] : p.k_scale;
      vs = p.v_scales ? p.v_scales[id * a.hkv + h] : p.v_scale;
      vs = vs >= 0.f ? fmaxf(vs, 0x1p-60f) : NAN;
    }
    const int64_t page = (id * 16 + t % kBlock / kPage) * a.id_stride + static_cast<int64_t>(h) * 2048;
    const int pt = static_cast<int>(t % kPage);
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(a.k_base + page + lane / 4 * 256 + pt * 16 + lane % 4 * 4);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) z = fmaf(q[i], e4m3_to_float(kw >> (8 * i)), z);
#pragma unroll
    for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    z *= ks * a.sm_scale;
    const float mn = fmaxf(m, z), f = m == mn ? 1.f : exp2f((m - mn) * kLog2e), e = exp2f((z - mn) * kLog2e);
    m = mn;
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = o[i] * f + e * (vs * e4m3_to_float(a.v_base[page + (4 * lane + i) * 16 + pt]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    static_cast<__nv_bfloat16*>(a.out)[w * kDim + 4 * lane + i] = __float2bfloat16_rn(m == -INFINITY && l == 0.f ? 0.f : o[i] / l);
}

}  // namespace

size_t dense_pa_fp8_ws_bytes(int32_t, int32_t, int32_t, int32_t, int) { return 0; }

cudaError_t launch_dense_pa_fp8(const DensePaFp8Params& p, int, cudaStream_t s, int* launches) {
  const int64_t warps = static_cast<int64_t>(p.a.num_rows) * p.a.group;
  const cudaError_t e = launch_kernel(dense_pa_fp8_kernel, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, s, 0, p);
  if (e == cudaSuccess) ++*launches;
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace bsp
