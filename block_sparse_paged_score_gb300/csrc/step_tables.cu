// step_tables.cu -- the paged bookkeeping of one step, built on the GPU from
// the requests' lengths (bsp_step_tables):
//
//   have_s = ceil(context_s / 128), want_s = ceil((context_s + new_s) / 128)
//   table[s][have_s + i] = free[head + sum_{r<s} (want_r - have_r) + i]
//   token t of request s at position p = context_s + t - cu_s:
//     slot = table[s][p / 128] * 128 + p % 128
//
// All of it follows from two exclusive prefix sums over the requests (new
// tokens and fresh blocks).  One launch: every CTA scans all requests in
// tiles of 1024 (4 a thread, warp shuffles, the tile's sums in shared memory)
// and, while a tile is at hand, writes its own share of the tokens and fresh
// blocks by a binary search in the tile's sums.  The scan is repeated by
// every CTA, which costs less than a second launch as long as the requests
// fit a few tiles; the loads of up to 1024 requests are one round trip.
// Measured: 1 request 2.5 us and 64 with four 4096-token chunks 3.3 us, a launch and
// two round trips; 4112 requests with 135 184 tokens 10.6 us, most of it the five
// tiles' chain of loads, shuffles and barriers (the bytes are worth 0.34 us).  Tiles
// twice as wide, in CTAs of 512 or 1024 threads: 10.5 and 11.7 us there, 2.7 and 4.1
// for 1 request.
// Sums saturate at 2^31 - 1 (saturating addition of non-negative numbers is
// associative, so the scan's order does not matter).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace bsp {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                 // requests a thread scans
constexpr int kTile = kThreads * kPer;  // requests a tile holds
constexpr uint32_t kMax = 0x7FFFFFFFu;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kMax); }

// largest i in [0, n) with cu[i] <= t, given cu[0] <= t < cu[n]
__device__ __forceinline__ int find(const uint32_t* cu, int n, uint32_t t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) step_tables_kernel(StepTablesParams p, int tokens_per_cta) {
  __shared__ uint32_t s_tok[kTile + 1], s_blk[kTile + 1];
  __shared__ int32_t s_ctx[kTile];
  __shared__ uint32_t s_warp[2][kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens_per_cta;
  const uint32_t t0 = static_cast<uint32_t>(min(first, static_cast<int64_t>(p.token_capacity)));
  const uint32_t t1 = static_cast<uint32_t>(min(first + tokens_per_cta, static_cast<int64_t>(p.token_capacity)));
  const int64_t head = p.free_head ? *p.free_head : 0;
  uint32_t tok_base = 0, blk_base = 0;  // of the tile's first request

  // the id of fresh block j, -1 (and a flag) where the free list has none
  auto fresh_id = [&](uint32_t j) -> int32_t {
    const int64_t at = head + j;
    if (at < 0 || at >= p.num_free || j >= kMax) {
      set_err(p.err, BSP_DEVERR_CAPACITY);
      return -1;
    }
    const int32_t id = p.free_blocks[at];
    if (id < 0 || id >= p.num_blocks) {
      set_err(p.err, BSP_DEVERR_BLOCK_ID);
      return -1;
    }
    return id;
  };

  int32_t next_ctx[kPer], next_new[kPer];  // of the tile to come
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t s = static_cast<int64_t>(tile) * kTile + tid * kPer + i;
      next_ctx[i] = s < p.num_seqs ? p.context_lens[s] : 0;
      next_new[i] = s < p.num_seqs ? p.new_lens[s] : 0;
    }
  };
  fetch(0);
  for (int tile = 0; tile * kTile < p.num_seqs; ++tile) {
    const int s0 = tile * kTile, n = min(kTile, p.num_seqs - s0);
    uint32_t tok[kPer], blk[kPer], tsum = 0, bsum = 0;
    int32_t ctx[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      ctx[i] = max(next_ctx[i], 0);
      tok[i] = static_cast<uint32_t>(max(next_new[i], 0));
    }
    fetch(tile + 1);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t len = sat_add(ctx[i], tok[i]);
      const uint32_t have = min((ctx[i] + 127u) / 128u, static_cast<uint32_t>(p.bt_stride));
      const uint32_t want = min((len + 127u) / 128u, static_cast<uint32_t>(p.bt_stride));
      blk[i] = want - have;
      tsum = sat_add(tsum, tok[i]);
      bsum = sat_add(bsum, blk[i]);
    }
    uint32_t ti = tsum, bi = bsum;  // inclusive over the threads
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, ti, d), b = __shfl_up_sync(0xffffffffu, bi, d);
      if (lane >= d) ti = sat_add(ti, a), bi = sat_add(bi, b);
    }
    __syncthreads();  // the previous tile's sums are no longer read
    if (lane == 31) s_warp[0][warp] = ti, s_warp[1][warp] = bi;
    __syncthreads();
    // exclusive start of this thread: the tile's base, the warps before, the lanes before
    uint32_t ts = __shfl_up_sync(0xffffffffu, ti, 1), bs = __shfl_up_sync(0xffffffffu, bi, 1);
    if (lane == 0) ts = 0, bs = 0;
    ts = sat_add(ts, tok_base), bs = sat_add(bs, blk_base);
    uint32_t tok_end = tok_base, blk_end = blk_base;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) ts = sat_add(ts, s_warp[0][w]), bs = sat_add(bs, s_warp[1][w]);
      tok_end = sat_add(tok_end, s_warp[0][w]), blk_end = sat_add(blk_end, s_warp[1][w]);
    }
    const bool mine = tile % gridDim.x == blockIdx.x;  // this CTA writes the tile's per-request outputs
    // fresh blocks: chunks of kThreads dealt to the CTAs in turn, c the first of this CTA
    const uint32_t chunks = blk_end / kThreads;
    uint32_t c = blk_base / kThreads;
    c += (blockIdx.x + gridDim.x - c % gridDim.x) % gridDim.x;
    if (!mine && (c > chunks || blk_end == blk_base) && (t1 <= tok_base || t0 >= tok_end)) {
      tok_base = tok_end, blk_base = blk_end;
      continue;         // nothing of the tile is this CTA's
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = tid * kPer + i;
      s_tok[s] = ts, s_blk[s] = bs, s_ctx[s] = ctx[i];
      if (mine && s < n) {
        p.cu_tokens[s0 + s] = static_cast<int32_t>(min(ts, static_cast<uint32_t>(p.token_capacity)));
        p.seq_lens[s0 + s] = static_cast<int32_t>(sat_add(ctx[i], tok[i]));
      }
      ts = sat_add(ts, tok[i]), bs = sat_add(bs, blk[i]);
    }
    if (tid == 0) s_tok[kTile] = tok_end, s_blk[kTile] = blk_end;
    __syncthreads();

    for (; c <= chunks; c += gridDim.x) {
      const uint32_t j = c * kThreads + tid;
      if (j < blk_base || j >= blk_end) continue;
      const int s = find(s_blk, kTile, j);
      const uint32_t have = min((s_ctx[s] + 127u) / 128u, static_cast<uint32_t>(p.bt_stride));
      p.block_table[static_cast<int64_t>(s0 + s) * p.bt_stride + have + (j - s_blk[s])] = fresh_id(j);
    }
    // this CTA's tokens in the tile
    for (uint32_t t = max(t0, tok_base) + tid; t < min(t1, tok_end); t += kThreads) {
      const int s = find(s_tok, kTile, t);
      const uint32_t pos = sat_add(s_ctx[s], t - s_tok[s]);
      const uint32_t have = min((s_ctx[s] + 127u) / 128u, static_cast<uint32_t>(p.bt_stride)), pb = pos / 128u;
      int32_t id = -1;
      if (pb >= static_cast<uint32_t>(p.bt_stride)) {
        set_err(p.err, BSP_DEVERR_CAPACITY);
      } else if (pb >= have) {
        id = fresh_id(s_blk[s] + (pb - have));
      } else {
        id = p.block_table[static_cast<int64_t>(s0 + s) * p.bt_stride + pb];
        if (id < 0 || id >= p.num_blocks) {
          set_err(p.err, BSP_DEVERR_BLOCK_ID);
          id = -1;
        }
      }
      p.slot[t] = id < 0 ? -1 : static_cast<int64_t>(id) * kBlock + pos % 128u;
      p.query_req_id[t] = s0 + s;
      p.query_abs_pos[t] = static_cast<int32_t>(pos);
    }
    tok_base = tok_end, blk_base = blk_end;
  }
  for (uint32_t t = max(t0, tok_base) + tid; t < t1; t += kThreads) {  // pad rows
    p.slot[t] = -1;
    p.query_req_id[t] = 0;
    p.query_abs_pos[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.cu_tokens[p.num_seqs] = static_cast<int32_t>(min(tok_base, static_cast<uint32_t>(p.token_capacity)));
    p.blocks_taken[0] = static_cast<int32_t>(blk_base);
    if (tok_base > static_cast<uint32_t>(p.token_capacity)) set_err(p.err, BSP_DEVERR_CAPACITY);
  }
}

}  // namespace

cudaError_t launch_step_tables(const StepTablesParams& p, int num_sms, cudaStream_t s) {
  // one token a thread up to two CTAs an SM, then more of them (135 184 tokens of 4112
  // requests: 11.4 us with one CTA an SM, 10.7 with two, 14.2 with four, each scanning)
  const int64_t wide = (static_cast<int64_t>(p.token_capacity) + kThreads - 1) / kThreads;
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(wide, 2 * num_sms));
  const int64_t per = (static_cast<int64_t>(p.token_capacity) + ctas - 1) / ctas;
  const cudaError_t e = launch_kernel(step_tables_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, 0,
                                      p, static_cast<int>(per));
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace bsp
