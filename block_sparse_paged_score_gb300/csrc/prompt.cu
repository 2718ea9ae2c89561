// prompt.cu -- causal grouped-query attention of packed prompts, or of chunks over
// their contexts (bsp_prompt_attention).
//
//   z[r, t] = scale * q_r . k_t,  t < L_r;   o_r = sum_t p[r, t] v_t / sum_t p[r, t],  p = exp(z)
//
// Work.  A unit = (sequence, KV head, 256 rows): 256 / G neighbouring tokens with the G
// query heads of the KV head, so that short prompts fill the tensor cores' rows too and
// a unit's keys end together.  It is two tiles of 128 rows.  Units' 128-key blocks laid
// end to end, causal ones only, are cut into equal shares, one per CTA: the blocks of
// a sequence's units are a closed sum, and a CTA finds its share by a prefix sum over the
// sequences.  Of a unit that share borders cut each CTA leaves (m, l, O) in the
// workspace, and a second kernel joins them; the order of all sums is fixed.
//
// Both products are tcgen05 MMAs, 128 x 128 x 16:
//   S = Q K^T     A = Q, B = K, both from shared memory (TMA, 128-byte swizzle)
//   O += P V      A = P, bf16, from TMEM, where it takes the place of S; B = V from
//                 shared memory, its dims contiguous
// TMEM holds S and O of both tiles, 512 columns.  While the tensor core works on one
// tile, four warps take the exponentials of the other: a thread has a whole row, so
// maxima and sums need no exchange.  Weights are 2^((z - m) c) against the row's
// reference m, which moves (and O and l with it) only when the row's maximum passes it by
// kMaxGrow.  That S of a block is there says that P V of the one before has ended: the
// MMAs run in order, so the thread may then rescale its row of O.
//
// Keys that a row does not see have p = 0, and V's rows of such keys may hold
// infinities and NaN, which 0 does not silence: two warps look through V's tile of
// those blocks that some row does not see whole, put zeros in place of what is not
// finite, and the rows that do see it get it added at the end.
//
// Roundings: a weight is bf16, half a step 2^-8 off; z, m, l and O are fp32, and l sums
// the unrounded weights.
//
// Every wait is bounded: after one that gave up (the error word is set, the results are
// void) its warp issues nothing more and waits for what it has under way, with a limit
// again; the others' waits run out in turn.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "tc_warp.cuh"
#include "tcgen05.cuh"

namespace bsp {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxGrow = 8.f;             // log2
constexpr float kNoMax = -3.402823466e38f;  // the maximum of no keys (finite: -inf - kNoMax stays -inf)
constexpr float kBigRef = 1048576.f;        // references above it: (z - m) c instead of z c - (m c), whose rounding then counts
constexpr int kRows = 256, kTile = 128;     // rows of a unit, of a tile
constexpr int kThreads = 384;               // four warps for each tile, a producer, an issuer, two that check V
constexpr int kWarpTma = 8, kWarpMma = 9;
constexpr int kHalf = 16384, kTileBytes = 2 * kHalf;  // 128 rows of 64 dims; of 128
constexpr int kStages = 5;                  // of K and V tiles, in the order K V K V
constexpr int kRegsRow = 208, kRegsRest = 88;
static_assert((8 * kRegsRow + 4 * kRegsRest) * 32 <= kThreads * 168);

struct Params {
  PromptParams a;
  float c;  // |sm_scale| * log2(e)
  int32_t tokens, log_tokens;  // of a unit: 256 / G
  int32_t ctas, least;         // shares have `least` blocks at least
};

struct Smem {
  static constexpr int q = 0, kv = 2 * kTileBytes, bars = kv + kStages * kTileBytes;
  static constexpr int q_full = bars, q_empty = bars + 8, kv_full = bars + 16, kv_empty = kv_full + 8 * kStages,
                       s_full = kv_empty + 8 * kStages, p_full = s_full + 16, o_full = p_full + 16, v_ok = o_full + 16,
                       fin = v_ok + 8 * kStages, misc = fin + 8;
  static constexpr int tmem = misc, bad = misc + 8;  // bad[8]: pieces with values of V that are not finite
  static constexpr int walks = (bad + 32 + 7) / 8 * 8;
};

// a unit that share borders cut, by its first CTA
struct Cut {
  int32_t pieces, tok0, tokens, h, see, pad[3];  // see: keys that its first token sees (may be <= 0)
};
__host__ __device__ constexpr int64_t list_bytes(int64_t ctas) { return (ctas * sizeof(Cut) + 255) / 256 * 256; }
constexpr int64_t kSlotFloats = kRows * (kDim + 2);

// ---- units -----------------------------------------------------------------------
struct Seq {
  int q0, nq, k0, nk;
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const PromptParams& a, int s) {
  const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
  Seq r;
  r.q0 = min(max(q0, 0), a.num_tokens);
  r.nq = max(min(q1, a.num_tokens), r.q0) - r.q0;
  r.k0 = min(max(k0, 0), a.num_keys);
  r.nk = max(min(k1, a.num_keys), r.k0) - r.k0;
  r.bad = q0 < 0 || q1 < q0 || q1 > a.num_tokens || k0 < 0 || k1 < k0 || k1 > a.num_keys;
  return r;
}
__device__ __forceinline__ int units_of(const Seq& s, const Params& p) { return (s.nq + p.tokens - 1) >> p.log_tokens; }
// blocks of unit u: at least one (rows without keys still get their zeros)
__device__ __forceinline__ int blocks_of(const Seq& s, const Params& p, int u) {
  const int64_t see = static_cast<int64_t>(s.nk) - s.nq + min((static_cast<int64_t>(u) + 1) << p.log_tokens, static_cast<int64_t>(s.nq));
  return max(1, static_cast<int>((max(see, int64_t{0}) + 127) >> 7));
}
// blocks of the units before u.  Unit i but the last sees off + (i + 1) T keys: the first
// units have one block, the others ceil((off + (i + 1) T) / 128), T a power of two.
__device__ __forceinline__ int64_t blocks_before(const Seq& s, const Params& p, int u) {
  const int n = units_of(s, p);
  const int64_t off = static_cast<int64_t>(s.nk) - s.nq, m = min(u, n - 1);
  const int lg = p.log_tokens;
  const int64_t one = max(int64_t{0}, min(m, (128 - off) >> lg));
  int64_t sum = one;
  if (lg <= 7) {  // ceil((A + i + 1) / R), A = ceil(off / T), R = 128 / T
    const int64_t A = -((-off) >> lg);
    const int lr = 7 - lg;
    auto upto = [&](int64_t x) {  // sum of ceil(y / R), 1 <= y <= x
      const int64_t q = x >> lr, r = x & ((1 << lr) - 1);
      return ((q * (q + 1) / 2) << lr) + r * (q + 1);
    };
    if (m > one) sum += upto(A + m) - upto(A + one);
  } else {  // T = 256
    const int64_t A = -((-off) >> 7);
    if (m > one) sum += (m - one) * A + (m * (m + 1) - one * (one + 1));
  }
  return u == n && n > 0 ? sum + blocks_of(s, p, n - 1) : sum;
}
__device__ __forceinline__ int64_t blocks_of_seq(const Seq& s, const Params& p) { return blocks_before(s, p, units_of(s, p)); }

// A warp's walk over the pieces of a share [at, end) of the units' blocks, in shared
// memory (a thread of a row has no registers for it); every lane writes the same values.
struct Walk {
  int64_t at, end, c0;  // c0: blocks of the sequences before s
  int64_t per;          // blocks of a KV head of sequence s
  int s, piece;
  Seq q;
  // the piece at `at`
  int64_t uend;
  int h, tok0, tokens, see, b0, nblk;  // see: keys that the unit's first token sees
  bool starts, ends;

  __device__ __forceinline__ bool next(const Params& p) {
    __syncwarp();  // (the lanes have read the piece before)
    if (at >= end) return false;
    const int64_t at = this->at;
    const int number = piece + 1;
    int s = this->s;
    int64_t c0 = this->c0, per = this->per;
    Seq q = this->q;
    while (c0 + per * p.a.hkv <= at) {
      c0 += per * p.a.hkv;
      q = load_seq(p.a, ++s);
      per = blocks_of_seq(q, p);
    }
    const int h = static_cast<int>((at - c0) / per);
    const int64_t x = at - c0 - h * per;
    int lo = 0, hi = units_of(q, p) - 1;  // the last unit with blocks_before <= x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (blocks_before(q, p, mid) <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int64_t ustart = c0 + h * per + blocks_before(q, p, lo), uend = ustart + blocks_of(q, p, lo);
    const int t = lo << p.log_tokens;
    __syncwarp();
    this->s = s, this->c0 = c0, this->per = per, this->q = q, this->h = h;
    this->uend = uend;
    piece = number;
    tok0 = q.q0 + t;
    tokens = min(p.tokens, q.nq - t);
    see = q.nk - q.nq + t + 1;
    b0 = static_cast<int>(at - ustart);
    nblk = static_cast<int>(min(end, uend) - at);
    starts = at == ustart, ends = end >= uend;
    this->at = min(end, uend);
    __syncwarp();
    return true;
  }
};

constexpr int kSmem = Smem::walks + kThreads / 32 * static_cast<int>(sizeof(Walk));
static_assert(kSmem <= 227 * 1024);

// ---- device helpers ------------------------------------------------------------------
__device__ __forceinline__ void tile_g2s_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      BSP_ELECT " @e cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
                "[%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// D (+)= A B, both bf16 in shared memory
__device__ __forceinline__ void umma_ss_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      BSP_ELECT " .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// After the wait for loads: what reads the registers comes behind it.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// K-major rows of 128 bytes, 128-byte swizzle (see smem_desc_sw128); V as the B operand
// with its dims contiguous: atoms of 64 dims x 8 keys, dims 64.. kHalf on
__device__ __forceinline__ uint64_t desc_v(uint32_t saddr) {
  uint64_t d = (saddr & 0x3FFFF) >> 4;
  d |= static_cast<uint64_t>(kHalf >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// fp32 += bf16 x bf16, M = 128, N = 128; V's rows are its contiguous ones
constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescO = kIdescS | (1u << 16);

// one 32-bit word of two bf16: bits 15 and 31 where a half is infinite or NaN
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// What rows see of V's values that are not finite, in keys [from, to) (the tiles that
// the MMAs read hold zeros in their place), added to dims d0 .. d0 + 31 of a row.
__device__ __forceinline__ void add_not_finite(const PromptParams& a, float (&o)[32], int k0, int h, int from, int to, int d0) {
  for (int t = from; t < to; ++t) {
    const uint16_t* v = a.v + (k0 + static_cast<int64_t>(t)) * a.v_stride + h * kDim + d0;
    for (int i = 0; i < 32; ++i)
      if ((v[i] & 0x7F80) == 0x7F80) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (k == i) o[k] += bf16_bits_to_float(v[i]);
      }
  }
}

// ---- the main kernel -------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  // before the first tile Q's place serves the scan
  int64_t* s_sum = reinterpret_cast<int64_t*>(smem);  // [warps]
  int64_t* s_start = s_sum + kThreads / 32;           // the share's first sequence, the blocks before it
  const PromptParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t base = smem_u32(smem);
  if (tid == 0) {
    auto init = [&](int at, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + at) + i, count);
    };
    init(Smem::q_full, 1, 1), init(Smem::q_empty, 1, 1);
    init(Smem::kv_full, kStages, 1), init(Smem::kv_empty, kStages, 1);
    init(Smem::s_full, 2, 1), init(Smem::p_full, 2, 4), init(Smem::o_full, 2, 1);
    init(Smem::v_ok, kStages, 2), init(Smem::fin, 1, 1);
    mbar_fence_init();
  }
  if (tid < 8) reinterpret_cast<volatile int*>(smem + Smem::bad)[tid] = 0;
  pdl_wait();
  // (TMEM only after the wait, and the next kernel's CTAs only once this one has got its
  // columns: one that waits while it holds some could keep the other from its own)
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + Smem::tmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // The sequences' blocks: a thread sums those of some neighbouring sequences, and the
  // one whose sequences hold the share's start looks through them again.
  const int n = a.num_seqs;
  const int chunk = (n + kThreads - 1) / kThreads;
  const int s_lo = min(tid * chunk, n), s_hi = min(s_lo + chunk, n);
  int64_t mine = 0;
  bool bad = false;
#pragma unroll 1
  for (int s = s_lo; s < s_hi; ++s) {
    const Seq q = load_seq(a, s);
    bad |= q.bad;
    mine += blocks_of_seq(q, p) * a.hkv;
  }
  if (bad && blockIdx.x == 0) set_err(a.err, BSP_DEVERR_CAPACITY);
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) upto += s_sum[w];
    total += s_sum[w];
  }
  const int64_t share = max((total + p.ctas - 1) / p.ctas, static_cast<int64_t>(p.least)), at = blockIdx.x * share;
  if (upto - mine <= at && at < upto) {
    int64_t c = upto - mine;
    int s = s_lo;
    for (; s < s_hi; ++s) {
      const int64_t b = blocks_of_seq(load_seq(a, s), p) * a.hkv;
      if (at < c + b) break;
      c += b;
    }
    s_start[0] = s, s_start[1] = c;
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  pdl_trigger();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + Smem::tmem), 0);
  Walk& w = reinterpret_cast<Walk*>(smem + Smem::walks)[warp];
  if (lane == 0) {
    w.at = at, w.end = min(at + share, total);
    w.piece = -1, w.s = 0, w.c0 = 0, w.per = 0;
    if (at < w.end) {
      w.s = static_cast<int>(s_start[0]), w.c0 = s_start[1];
      w.q = load_seq(a, w.s);
      w.per = blocks_of_seq(w.q, p);
    }
  }
  __syncthreads();  // the scan's place is Q's again
  Cut* cut = static_cast<Cut*>(a.ws);
  if (tid == 0) cut[blockIdx.x].pieces = 0;
  bool alive = true;
  auto wait = [&](uint32_t bar, uint32_t parity) { return alive = alive && wait_warp(bar, parity, a.err); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kWarpTma) {
      // ---- producer: Q of each piece, then K and V of its blocks ----
      uint32_t st = 0, phase = 1, q_phase = 1;  // (an empty stage's wait passes at once)
      auto load = [&](const CUtensorMap* m, int h, int row) {
        if (!wait(base + Smem::kv_empty + 8 * st, phase)) return;
        const uint32_t bar = base + Smem::kv_full + 8 * st, dst = base + Smem::kv + st * kTileBytes;
        arrive_expect(bar, kTileBytes);
        tile_g2s_3d(dst, m, 0, h, row, bar);
        tile_g2s_3d(dst + kHalf, m, 64, h, row, bar);
        if (++st == kStages) st = 0, phase ^= 1;
      };
      while (alive && w.next(p)) {
        if (!wait(base + Smem::q_empty, q_phase)) break;
        const bool two = w.tokens > p.tokens / 2;
        arrive_expect(base + Smem::q_full, two ? 2 * kTileBytes : kTileBytes);
        for (int i = 0; i < (two ? 2 : 1); ++i)
          for (int d = 0; d < 2; ++d)
            tile_g2s_3d(base + Smem::q + i * kTileBytes + d * kHalf, &map_q, 64 * d, w.h * a.group,
                        w.tok0 + i * (p.tokens / 2), base + Smem::q_full);
        q_phase ^= 1;
#pragma unroll 1
        for (int b = w.b0; alive && b < w.b0 + w.nblk; ++b) {
          load(&map_k, w.h, w.q.k0 + b * kBlock);
          if (alive) load(&map_v, w.h, w.q.k0 + b * kBlock);
        }
      }
      // nothing may still write shared memory when the CTA leaves
      if (q_phase == 0 || w.piece > 0) wait_warp(base + Smem::q_full, q_phase, a.err, kSleepWaitLimit);
      for (uint32_t i = 0; i < kStages; ++i)
        wait_warp(base + Smem::kv_full + 8 * i, i < st ? phase ^ 1 : phase, a.err, kSleepWaitLimit);
    } else if (warp == kWarpMma) {
      // ---- issuer ----
      uint32_t st = 0, phase = 0, q_phase = 0, p_phase = 0, ok_phase = 0;
      const uint64_t q_desc = smem_desc_sw128(base + Smem::q), k_desc = smem_desc_sw128(base + Smem::kv);
      const uint64_t v_desc = desc_v(base + Smem::kv);
      auto scores = [&](int i, uint32_t stage) {  // S = Q K^T of a tile
        const uint64_t qd = q_desc + i * (kTileBytes / 16), kd = k_desc + stage * (kTileBytes / 16);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t o = (k >> 2) * (kHalf / 16) + (k & 3) * 2;
          umma_ss_f16(tmem + i * 128, qd + o, kd + o, kIdescS, k > 0);
        }
        commit(base + Smem::s_full + 8 * i);
      };
      auto values = [&](int i, uint32_t stage, bool accumulate) {  // O (+)= P V of a tile
        const uint64_t vd = v_desc + stage * (kTileBytes / 16);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ts(tmem + 256 + i * 128, tmem + i * 128 + 8 * k, vd + k * (2048 / 16), kIdescO, accumulate || k > 0);
      };
      auto fence = [] { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); };
      auto step = [&] {
        const uint32_t was = st;
        if (++st == kStages) st = 0, phase ^= 1;
        return was;
      };
      while (alive && w.next(p)) {
        const bool two = w.tokens > p.tokens / 2;
        const int masked = w.see >> 7;  // blocks from here on some row does not see whole (see < 0: all)
        if (!wait(base + Smem::q_full, q_phase)) break;
        q_phase ^= 1;
        if (!wait(base + Smem::kv_full + 8 * st, phase)) break;
        uint32_t ks = step();
        fence();
        scores(0, ks);
        if (two) scores(1, ks);
        commit(base + Smem::kv_empty + 8 * ks);
        if (w.nblk == 1) commit(base + Smem::q_empty);
#pragma unroll 1
        for (int j = 0; j < w.nblk; ++j) {
          const bool more = j + 1 < w.nblk;
          if (!wait(base + Smem::kv_full + 8 * st, phase)) break;
          const uint32_t vs = step();
          if (w.b0 + j >= masked) {
            if (!wait(base + Smem::v_ok + 8 * vs, ok_phase >> vs & 1)) break;
            ok_phase ^= 1u << vs;
          }
          if (more && !wait(base + Smem::kv_full + 8 * st, phase)) break;
          if (more) ks = step();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i && !two) break;
            if (!wait(base + Smem::p_full + 8 * i, p_phase >> i & 1)) break;
            p_phase ^= 1u << i;
            fence();
            values(i, vs, j > 0);
            if (more)
              scores(i, ks);
            else
              commit(base + Smem::o_full + 8 * i);
          }
          if (!alive) break;
          commit(base + Smem::kv_empty + 8 * vs);
          if (more) commit(base + Smem::kv_empty + 8 * ks);
          if (j + 2 == w.nblk) commit(base + Smem::q_empty);
        }
      }
      // every MMA and commit has ended
      commit(base + Smem::fin);
      wait_warp(base + Smem::fin, 0, a.err, kSleepWaitLimit);
    } else {
      // ---- V of the blocks that some row does not see whole: each warp takes 64 dims ----
      uint32_t st = 0, phase = 0;
      const uint32_t half = base + Smem::kv + (warp - 10) * kHalf;
      while (alive && w.next(p)) {
        const int masked = w.see >> 7;
#pragma unroll 1
        for (int b = w.b0; b < w.b0 + w.nblk; ++b) {
          if (++st == kStages) st = 0, phase ^= 1;  // (K's stage)
          if (!wait(base + Smem::kv_full + 8 * st, phase)) break;  // (every one: a parity tells two turns of the ring apart)
          if (b >= masked) {
            const uint32_t at = half + st * kTileBytes + lane * 16;
            uint32_t any = 0;
#pragma unroll 4
            for (int i = 0; i < 32; ++i) {
              const uint4 v = lds128(at + i * 512);
              any |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
            }
            if (__any_sync(0xffffffffu, any != 0)) {
#pragma unroll 1
              for (int i = 0; i < 32; ++i) {
                const uint4 v = lds128(at + i * 512);
                auto clean = [](uint32_t x) {
                  const uint32_t m = not_finite(x);
                  return x & ~((m >> 15) * 0xFFFFu);
                };
                sts128(at + i * 512, clean(v.x), clean(v.y), clean(v.z), clean(v.w));
              }
              if (lane == 0) reinterpret_cast<volatile int*>(smem + Smem::bad)[w.piece & 7] = w.piece + 1;
              fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) arrive(base + Smem::v_ok + 8 * st);
          }
          if (++st == kStages) st = 0, phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: thread = row ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRow));
    const int tile = warp >> 2, row = tid;  // of the unit
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + tile * 128, o_at = tmem + lanes + 256 + tile * 128;
    const uint32_t s_full = base + Smem::s_full + 8 * tile, p_full = base + Smem::p_full + 8 * tile;
    uint32_t s_phase = 0, o_phase = 0;
    const float c = p.c;
    const bool neg = a.sm_scale < 0.f;
    const int log_group = 8 - p.log_tokens;
    while (alive && w.next(p)) {
      const int tok = row >> log_group;  // of the unit
      if (tile && w.tokens <= p.tokens / 2) continue;
      const int see = tok < w.tokens ? max(w.see + tok, 0) : 0;                  // keys that the row sees
      const int whole = (w.see + (tile ? p.tokens / 2 : 0)) >> 7;               // blocks that all rows of the tile see whole
      float ref = kNoMax;
      float2 l[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
      for (int j = 0; j < w.nblk; ++j) {
        if (!wait(s_full, s_phase)) break;
        s_phase ^= 1;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        uint32_t r[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32_issue(s_at + 32 * k, r[k]);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int k = 0; k < 4; ++k) loaded(r[k]);
        const int b = w.b0 + j;
        auto z = [&](int i) { return __uint_as_float(r[i >> 5][i & 31]); };
        bool slow = b >= whole || neg;
        if (slow) {
          const int lim = b >= whole ? see - b * kBlock : kBlock;
#pragma unroll
          for (int i = 0; i < 128; ++i) {
            const float x = neg ? -z(i) : z(i);
            r[i >> 5][i & 31] = __float_as_uint(i < lim ? x : -INFINITY);
          }
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mx[k] = fmax3(z(32 * k), z(32 * k + 1), z(32 * k + 2));
#pragma unroll
          for (int i = 3; i < 31; i += 2) mx[k] = fmax3(mx[k], z(32 * k + i), z(32 * k + i + 1));
          mx[k] = fmaxf(mx[k], z(32 * k + 31));
        }
        const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        const bool moves = !((top - ref) * c <= kMaxGrow);
        if (__any_sync(0xffffffffu, moves)) {
          // the rows' references, and O and l in their terms
          const float to = moves && top > ref ? top : ref, f = rescale(ref, to, c);
          ref = to;
          l[0].x *= f, l[0].y *= f, l[1].x *= f, l[1].y *= f;
          if (j) {
#pragma unroll 1
            for (int k = 0; k < 128; k += 16) {
              float y[16];
              tmem_ld<16>(o_at + k, y);
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] *= f;
              tmem_st<16>(o_at + k, y);
            }
          }
        }
        const float rc = ref * c;
        slow |= __any_sync(0xffffffffu, !(fabsf(rc) < kBigRef));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t pk[16];
          if (__builtin_expect(!slow, 1)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = ffma2({z(32 * k + 2 * i), z(32 * k + 2 * i + 1)}, {c, c}, {-rc, -rc});
              const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
              l[i & 1] = fadd2(l[i & 1], e);
              pk[i] = pack_bf16x2(e.x, e.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = fmul2(fadd2({z(32 * k + 2 * i), z(32 * k + 2 * i + 1)}, {-ref, -ref}), {c, c});
              const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
              l[i & 1] = fadd2(l[i & 1], e);
              pk[i] = pack_bf16x2(e.x, e.y);
            }
          }
          tmem_st16(s_at + 16 * k, pk);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive(p_full);
      }
      if (!wait(base + Smem::o_full + 8 * tile, o_phase)) break;
      o_phase ^= 1;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      // -- O to where it goes
      const float sum = (l[0].x + l[0].y) + (l[1].x + l[1].y);
      const bool all = w.starts && w.ends;
      const float f = !all ? 1.f : see == 0 ? 0.f : 1.f / sum;
      const bool fix = reinterpret_cast<volatile int*>(smem + Smem::bad)[w.piece & 7] == w.piece + 1;
      // a CTA's slots: 2 * CTA for a unit that began before its share, + 1 for one that
      // goes on after it
      float* po = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + list_bytes(p.ctas)) +
                  (2LL * blockIdx.x + (w.starts ? 1 : 0)) * kSlotFloats;
      const bool live = tok < w.tokens;
      uint16_t* out = a.out + (static_cast<int64_t>(w.tok0 + tok) * a.hkv * a.group + w.h * a.group + (row & (a.group - 1))) * kDim;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t r[32];
        tmem_ld32_issue(o_at + 32 * k, r);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        loaded(r);
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(r[i]);
        if (__builtin_expect(fix, 0))
          add_not_finite(a, o, w.q.k0, w.h, max(w.b0, max(w.see >> 7, 0)) * kBlock,
                         live ? min(see, (w.b0 + w.nblk) * kBlock) : 0, 32 * k);
        if (live) {
          if (all) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(out + 32 * k + i) =
                  make_uint4(pack_bf16x2(o[i] * f, o[i + 1] * f), pack_bf16x2(o[i + 2] * f, o[i + 3] * f),
                             pack_bf16x2(o[i + 4] * f, o[i + 5] * f), pack_bf16x2(o[i + 6] * f, o[i + 7] * f));
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(po + row * kDim + 32 * k + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        __syncwarp();
      }
      if (!all) *reinterpret_cast<float2*>(po + kRows * kDim + 2 * row) = make_float2(ref, sum);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      if (w.starts && !w.ends && tid == 0) {
        // the pieces of the unit: shares from this one to that of its last block
        cut[blockIdx.x] = {static_cast<int>((w.uend - 1) / share) - static_cast<int>(blockIdx.x) + 1, w.tok0, w.tokens, w.h,
                           w.see, {0, 0, 0}};
      }
    }
    __syncwarp();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kWarpMma) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ---- cut units -----------------------------------------------------------------------------
// Joins the pieces of the units that share borders cut: a warp takes a row.
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  pdl_trigger();
  const PromptParams& a = p.a;
  const int lane = threadIdx.x & 31;
  const int c0 = blockIdx.x / (kRows / 8), row = (blockIdx.x % (kRows / 8)) * 8 + (threadIdx.x >> 5);
  const Cut u = static_cast<const Cut*>(a.ws)[c0];
  const int log_group = 8 - p.log_tokens, tok = row >> log_group;
  if (u.pieces == 0 || tok >= u.tokens) return;
  const float* base = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + list_bytes(p.ctas));
  float M = kNoMax, L = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < u.pieces; k0 += 32) {
    const int k = k0 + lane;  // lane j: piece k0 + j
    float2 ml = make_float2(kNoMax, 0.f);
    if (k < u.pieces)
      ml = *reinterpret_cast<const float2*>(base + (k ? 2LL * (c0 + k) : 2LL * c0 + 1) * kSlotFloats + kRows * kDim + 2 * row);
    float mx = ml.x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float mn = fmaxf(M, mx), f = rescale(M, mn, p.c), wt = rescale(ml.x, mn, p.c);
    float ls = wt * ml.y;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
    L = L * f + ls;
    M = mn;
    x.x *= f, x.y *= f, x.z *= f, x.w *= f;
    const int here = min(32, u.pieces - k0);
#pragma unroll 8
    for (int j = 0; j < here; ++j) {
      const int kj = k0 + j;
      const float wj = __shfl_sync(0xffffffffu, wt, j);
      const float4 y = *reinterpret_cast<const float4*>(base + (kj ? 2LL * (c0 + kj) : 2LL * c0 + 1) * kSlotFloats +
                                                        row * kDim + 4 * lane);
      x.x += wj * y.x, x.y += wj * y.y, x.z += wj * y.z, x.w += wj * y.w;
    }
  }
  const float f = u.see + tok <= 0 ? 0.f : 1.f / L;
  const int64_t e = (static_cast<int64_t>(u.tok0 + tok) * a.hkv * a.group + u.h * a.group + (row & (a.group - 1))) * kDim + 4 * lane;
  *reinterpret_cast<uint2*>(a.out + e) = make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
}

// ---- host ------------------------------------------------------------------------------------
// rows as [tokens][heads][128], boxes of 64 dims x `heads` x `rows`, 128-byte swizzle
bool make_map_rows(CUtensorMap* m, const void* base, uint64_t heads, uint64_t tokens, int64_t stride, uint32_t box_heads,
                   uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {kDim, heads, tokens};
  const cuuint64_t strides[2] = {kDim * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, box_heads, box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t prompt_ws_bytes(int32_t, int32_t, int32_t, int32_t, int num_sms) {
  return list_bytes(num_sms) + 2 * static_cast<int64_t>(num_sms) * kSlotFloats * sizeof(float);
}

cudaError_t launch_prompt(const PromptParams& a, int num_sms, cudaStream_t s, int* launches) {
  Params p{};
  p.a = a;
  // (a scale of 0 as the least float: masked logits stay -inf, all others become 0 as near as counts)
  p.c = std::max(std::fabs(a.sm_scale) * kLog2e, 1.401298464e-45f);
  p.tokens = kRows / a.group;
  while ((1 << p.log_tokens) < p.tokens) ++p.log_tokens;
  p.ctas = num_sms;
  p.least = 2;
  CUtensorMap mq, mk, mv;
  // (no keys at all: the maps of K and V have one row, Q's first, which no row sees)
  const bool keys = a.num_keys > 0;
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  if (!make_map_rows(&mq, a.q, hq, a.num_tokens, a.q_stride, a.group, kTile / a.group) ||
      !make_map_rows(&mk, keys ? a.k : a.q, a.hkv, keys ? a.num_keys : 1, keys ? a.k_stride : a.q_stride, 1, kBlock) ||
      !make_map_rows(&mv, keys ? a.v : a.q, a.hkv, keys ? a.num_keys : 1, keys ? a.v_stride : a.q_stride, 1, kBlock))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [] {  // the shared-memory opt-in
    return cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  e = launch_kernel(prompt_kernel, dim3(static_cast<unsigned>(p.ctas)), dim3(kThreads), kSmem, s, 0, mq, mk, mv, p);
  if (e != cudaSuccess) return e;
  ++*launches;
  e = launch_kernel(prompt_join_kernel, dim3(static_cast<unsigned>(p.ctas * (kRows / 8))), dim3(256), 0, s, 0, p);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaPeekAtLastError();
}

}  // namespace bsp
