// prompt.cu -- causal grouped-query attention of packed prompts
// (bsp_prompt_attention): a warp per query head and row, a key at a time.
#include "common.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(128) prompt_kernel(PromptParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);  // token * heads + head
  const int64_t hq = static_cast<int64_t>(p.hkv) * p.group;
  if (w >= p.num_tokens * hq) return;
  const int tok = static_cast<int>(w / hq), head = static_cast<int>(w % hq), h = head / p.group;
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < p.num_seqs; s += 128)
      if (p.cu_q[s] < 0 || p.cu_q[s + 1] < p.cu_q[s] || p.cu_q[s + 1] > p.num_tokens || p.cu_k[s] < 0 ||
          p.cu_k[s + 1] < p.cu_k[s] || p.cu_k[s + 1] > p.num_keys)
        set_err(p.err, BSP_DEVERR_CAPACITY);
  // the first sequence that has the token
  int seq = p.num_seqs;
  for (int s0 = 0; s0 < p.num_seqs && seq == p.num_seqs; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < p.num_seqs && p.cu_q[s] <= tok && tok < p.cu_q[s + 1];
    const uint32_t any = __ballot_sync(0xffffffffu, in);
    if (any) seq = s0 + __ffs(any) - 1;
  }
  if (seq == p.num_seqs) return;
  const int q0 = max(p.cu_q[seq], 0), q1 = min(p.cu_q[seq + 1], p.num_tokens);
  const int k0 = min(max(p.cu_k[seq], 0), p.num_keys), k1 = max(min(p.cu_k[seq + 1], p.num_keys), k0);
  const int len = max(0, k1 - k0 - (q1 - q0) + (tok - q0) + 1);
  float q[4], o[4] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = bf16_bits_to_float(p.q[tok * p.q_stride + head * kDim + 4 * lane + i]);
  for (int t = k0; t < k0 + len; ++t) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) z = fmaf(q[i], bf16_bits_to_float(p.k[t * p.k_stride + h * kDim + 4 * lane + i]), z);
#pragma unroll
    for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    z *= p.sm_scale;
    const float mn = fmaxf(m, z), f = m == mn ? 1.f : exp2f((m - mn) * kLog2e), e = exp2f((z - mn) * kLog2e);
    m = mn;
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = o[i] * f + e * bf16_bits_to_float(p.v[t * p.v_stride + h * kDim + 4 * lane + i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p.out[w * kDim + 4 * lane + i] = static_cast<uint16_t>(pack_bf16x2(len ? o[i] / l : 0.f, 0.f));
}

}  // namespace

size_t prompt_ws_bytes(int32_t, int32_t, int32_t, int32_t, int) { return 0; }

cudaError_t launch_prompt(const PromptParams& p, int, cudaStream_t s, int* launches) {
  const int64_t warps = static_cast<int64_t>(p.num_tokens) * p.hkv * p.group;
  const cudaError_t e = launch_kernel(prompt_kernel, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, s, 0, p);
  if (e == cudaSuccess) ++*launches;
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace bsp
