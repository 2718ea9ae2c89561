// prompt.cu -- causal grouped-query attention of packed prompts, or of chunks over
// their contexts (bsp_prompt_attention).
//
//   z[r, t] = scale * q_r . k_t,  t < L_r;   o_r = sum_t p[r, t] v_t / sum_t p[r, t],  p = exp(z)
//
// Work.  A unit = (sequence, KV head, 256 rows): 256 / G neighbouring tokens with the G
// query heads of the KV head, so that short prompts fill the tensor cores' rows too and
// a unit's keys end together.  It is two tiles of 128 rows.  Units' 128-key blocks laid
// end to end, causal ones only, and kUnitCost for each unit's beginning and end, are cut into
// equal shares, one per CTA: the length of a sequence's units is a closed sum, and a CTA
// finds its share by a prefix sum over the sequences.  Units of at most kWhole blocks stay
// whole.  Of a unit that share borders
// cut each CTA leaves (m, l, O) in the workspace, and a second kernel joins them; the
// order of all sums is fixed.
//
// Both products are tcgen05 MMAs, 128 x 128 x 16:
//   S = Q K^T     A = Q, B = K, both from shared memory (TMA, 128-byte swizzle)
//   O += P V      A = P, bf16, from TMEM, where it takes the place of S; B = V from
//                 shared memory, its dims contiguous
// TMEM holds S and O of both tiles, 512 columns.  While the tensor core works on one
// tile, four warps take the exponentials of the other: a thread has a whole row, so sums
// need no exchange.  Weights are 2^((z - m) c) against the row's reference m, the maximum of
// its first block; there is no maximum in the loop.  A half block whose weights sum to
// more than kMaxSum (each is at most that) takes a new reference from its own maximum, and O
// and l with it.  P leaves in halves, and P V of the first runs while the second's
// exponentials are taken.
//
// Keys that a row does not see have p = 0, and V's rows of such keys may hold
// infinities and NaN, which 0 does not silence: four warps look through those keys of
// V's tiles that some row does not see, put zeros in place of what is not
// finite, and the rows that do see it get it added at the end.
//
// A producer warp finds the pieces, announces them to the others in a ring, and loads Q, K
// and V; an issuer warp issues the MMAs; a fourth kind stores O: bf16 rows are staged in a
// stage of the K / V ring that the producer grants after a piece's last block, and leave by
// TMA (a row's 256 bytes from one thread touch 16 lines, 4096 clocks of a tile).
//
// Roundings: a weight is bf16, half a step 2^-8 off; z, m, l and O are fp32, and l sums
// the unrounded weights.  The MMA wants P and V of one type, and V is bf16 with its range; the
// rest of a weight as a second bf16 (as the sparse attention over bf16 keeps it, which memory
// bounds) would be half as many MMAs again where MMAs are what bounds it.  Against 64 bits the
// outputs are off by 0.0018 to 0.0023 of their norm, where their own rounding to bf16 alone
// makes 0.0016 to 0.0017.
//
// Measured (a call of a row of twenty in a graph): a prompt of 32768 tokens of 16 heads 2.22 to
// 2.54 ms, 1.73 to 1.98 PFLOP/s by the clock that the power limit leaves (cuBLAS 1.87); 32 prompts of
// 250 to 2000 tokens 165 us, 1.22 PFLOP/s: there a unit's beginning and end, a chain of some 6000
// clocks, bound it; 3 x 77 tokens over 100000 keys 144 us; one prompt of 100 tokens 8.4 us.  With other
// inputs each time 179, 153 and 11.3.  The kernels' code counts: at 117 KB instead of 81 instruction
// fetches were the first stall.
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

constexpr float kMaxSum = 1073741824.f;     // of a half block's weights (bf16 and fp32 hold any)
// references above it: (z - m) c instead of z c - (m c), whose rounding then counts
constexpr float kBigRef = 1048576.f;
constexpr int kRows = 256, kTile = 128;     // rows of a unit, of a tile
// Blocks of a unit that is not cut.  2, 4, 8: 165.6, 165.2, 165.6 us on 32 prompts of 250 to 2000
// tokens of 16 heads, 27.6, 29.0, 29.3 on 6 of 2500 of one.  (Up to as many there is no second launch.)
constexpr int kWhole = 4;
// What a unit costs beside its blocks, in blocks: 0, 1, 2, 3 take 214.7, 174.3, 165.2, 173.8 us on 32
// prompts of 250 to 2000 tokens, 2.65, 2.53, 2.48, 2.48 ms on one of 32768.
constexpr int kUnitCost = 2;
// Shares of so many blocks, over so many keys and heads (60 MB), may be lengthened, see aligned_share.
// (The keys are the rows given: where only some are any sequence's, shares may be lengthened earlier,
// which changes the time alone.)
constexpr int kLongShare = 64, kManyKeys = 60 * 1024 * 1024 / (4 * kDim);
// four warps for each tile, then a producer, an issuer, one that stores, one that idles, four that check V
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpStore = 10, kWarpCheck = 12, kThreads = 512;
constexpr int kReaders = 8 + 2 + 4;         // warps that read the announced pieces
constexpr int kHalf = 16384, kTileBytes = 2 * kHalf;  // 128 rows of 64 dims; of 128
constexpr int kStages = 5, kPieces = 4;     // of K, V and O tiles; of announced pieces
constexpr int kRegsRow = 184, kRegsRest = 64;
static_assert((kRegsRow + kRegsRest) * 256 <= kThreads * 128);

struct Params {
  PromptParams a;
  float c;  // |sm_scale| * log2(e)
  int32_t tokens, log_tokens;  // of a unit: 256 / G
  int32_t ctas;
};

// A part of a unit, as its CTA's producer announces it.
struct Piece {
  int32_t tok0, tokens, see;  // first token, tokens, keys that the first one sees (may be <= 0)
  int32_t b0, nblk;           // blocks; nblk 0: no more pieces
  int32_t h, k0;              // KV head, the sequence's first key
  uint32_t item;              // number of its first K tile in the ring's order
  int32_t starts, ends;       // whether the unit's first and last blocks are in it
  int32_t pieces, pad;        // of the unit, where it starts here and goes on
};
struct Smem {
  static constexpr int q = 0, kv = 2 * kTileBytes, bars = kv + kStages * kTileBytes;
  static constexpr int q_full = bars, q_empty = bars + 8, kv_full = bars + 16, kv_empty = kv_full + 8 * kStages,
                       v_look = kv_empty + 8 * kStages, v_ok = v_look + 8 * kStages, s_full = v_ok + 8 * kStages,
                       p_full = s_full + 16, half = p_full + 32, o_full = half + 16, staged = o_full + 16,
                       piece_full = staged + 16, piece_empty = piece_full + 8 * kPieces, fin = piece_empty + 8 * kPieces;
  static constexpr int pieces = fin + 8;
  static constexpr int tmem = pieces + kPieces * sizeof(Piece);
  static constexpr int bad = tmem + 8;  // [8]: pieces with values of V that are not finite
  static constexpr int total = bad + 32;
  static_assert(pieces % 8 == 0 && total <= 227 * 1024);
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
// blocks of unit u < units_of: at least one (rows without keys still get their zeros)
__device__ __forceinline__ int blocks_of(const Seq& s, const Params& p, int u) {
  const int after = max(s.nq - static_cast<int>(min((static_cast<int64_t>(u) + 1) << p.log_tokens, int64_t{0x7FFFFFFF})), 0);
  return static_cast<int>((static_cast<uint32_t>(max(s.nk - after, 1)) + 127u) >> 7);
}
// blocks of the units before u.  Unit i but the last sees off + (i + 1) T keys: the first
// units have one block, the others ceil((off + (i + 1) T) / 128), T a power of two.
__device__ __forceinline__ int64_t blocks_before(const Seq& s, const Params& p, int u) {
  const int n = units_of(s, p), m = min(u, n - 1), lg = p.log_tokens, off = s.nk - s.nq;  // (of both signs)
  const int one = max(0, min(m, off > 128 ? 0 : static_cast<int>((128 - static_cast<int64_t>(off)) >> lg)));
  int64_t sum = one;
  if (m > one) {
    if (lg <= 7) {  // ceil((A + i + 1) / R), A = ceil(off / T), R = 128 / T
      const int A = -((-off) >> lg), lr = 7 - lg;
      auto upto = [&](int x) {  // sum of ceil(y / R), 1 <= y <= x
        const int64_t q = x >> lr;
        return ((q * (q + 1) >> 1) << lr) + (x & ((1 << lr) - 1)) * (q + 1);
      };
      sum += upto(A + m) - upto(A + one);
    } else {  // T = 256
      sum += static_cast<int64_t>(m - one) * -((-off) >> 7) +
             (static_cast<int64_t>(m) * (m + 1) - static_cast<int64_t>(one) * (one + 1));
    }
  }
  return u == n && n > 0 ? sum + blocks_of(s, p, n - 1) : sum;
}
// the length of a sequence's units, and of those before u, as shares are measured
__device__ __forceinline__ int64_t length_before(const Seq& s, const Params& p, int u) {
  return blocks_before(s, p, u) + static_cast<int64_t>(u) * kUnitCost;
}
__device__ __forceinline__ int64_t length_of_seq(const Seq& s, const Params& p) { return length_before(s, p, units_of(s, p)); }

// The producer's walk over the pieces of its share [at, end).  A unit is nb + kUnitCost
// long; a border behind its blocks, or inside a unit of at most kWhole blocks, stands for
// its end.
struct Walk {
  int64_t at, end, share;
  int64_t ustart;  // of unit (s, h, u)
  int s, h, u, nb;
  Seq q;

  // the unit that holds `at`, of sequence s0 with a length of c0 before it
  __device__ __forceinline__ void find(const Params& p, int s0, int64_t c0) {
    s = s0, q = load_seq(p.a, s);
    const int64_t per = length_of_seq(q, p);
    h = p.a.hkv == 1 ? 0 : static_cast<int>((at - c0) / per);
    const int64_t x = at - c0 - h * per;
    int lo = 0, hi = units_of(q, p) - 1;  // the last unit with length_before <= x
#pragma unroll 1
    while (lo < hi) {
      const int mid = lo + ((hi - lo + 1) >> 1);
      if (length_before(q, p, mid) <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    u = lo, nb = blocks_of(q, p, u), ustart = c0 + h * per + length_before(q, p, u);
    if (at > ustart && (nb <= kWhole || at >= ustart + nb)) at = ustart + nb + kUnitCost;
  }
  __device__ __forceinline__ bool next(const Params& p, Piece& e) {
    if (at >= end) return false;
    if (at == ustart + nb + kUnitCost) {  // the next unit
      ustart = at, ++u;
#pragma unroll 1
      while (u >= units_of(q, p)) {
        u = 0;
        if (++h == p.a.hkv || units_of(q, p) == 0) h = 0, q = load_seq(p.a, ++s);
      }
      nb = blocks_of(q, p, u);
    }
    const int64_t uend = ustart + nb, to = nb <= kWhole ? uend : min(end, uend);
    const int t = u << p.log_tokens;
    e.tok0 = q.q0 + t, e.tokens = min(p.tokens, q.nq - t), e.see = q.nk - q.nq + t + 1;
    e.b0 = static_cast<int>(at - ustart), e.nblk = static_cast<int>(to - at);
    e.h = h, e.k0 = q.k0;
    e.starts = at == ustart, e.ends = to == uend;
    // pieces of the unit: shares from this one to that of its last block
    e.pieces = e.starts && !e.ends ? static_cast<int>((uend - 1) / share) - static_cast<int>(blockIdx.x) + 1 : 0;
    at = to == uend ? uend + kUnitCost : to;
    return true;
  }
};

// ---- device helpers ------------------------------------------------------------------
__device__ __forceinline__ void tile_g2s_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      BSP_ELECT " @e cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
                "[%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// by the calling thread
__device__ __forceinline__ void tile_s2g_3d(const CUtensorMap* m, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(m), "r"(x), "r"(y),
               "r"(z), "r"(src)
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
// Waits for the warp's loads; what reads the registers comes behind it.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]));
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
// acc + 0 * w, both halves: NaN once a half of a w was infinite or NaN
__device__ __forceinline__ uint32_t add_zero_times(uint32_t acc, uint32_t w) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
  return r;
}

// Few long units, such as some tokens of each request over long contexts: a head's units
// read the same keys, and each key comes from DRAM once if the shares of those units begin at
// nearly the same blocks, as they do when a unit is about a whole number of shares
// long.  Of 16 lengths, the given one and up to 15 / 128 more, the first with the least part
// of a share left over in all, counted in 64ths of the units.  us, without and with: 3 x 77
// queries of 16 heads over 100000 keys of two (307 MB) 166, 144; 2 x 200 of 16 over 40000 of two (82 MB)
// 105 to 112, 104 to 106; within 2 % on eleven others of 61 to 123 MB, of 1, 2 and 4 KV heads; but 2 x
// 500 of 8 over 50000 of one (52 MB, which L2 holds) 127, 129, and 2000 of 8 over 100000 (52 MB) 465, 474.
__device__ __noinline__ int64_t aligned_share(const Params& p, int64_t total, int64_t share, Seq q, int64_t* smem) {
  int* const s_count = reinterpret_cast<int*>(smem + kThreads / 32 + 2);
  int* const s_left = s_count + 1;
  int* const s_list = s_left + kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, most = p.ctas / p.a.hkv;
  if (tid == 0) s_count[0] = 0;
  __syncthreads();
  const int mine = min(units_of(q, p), most + 1);
  const int slot = mine ? atomicAdd(s_count, mine) : 0;
  __syncthreads();
  const int units = s_count[0];
  if (units > most || units * p.a.hkv < 2) return share;
#pragma unroll 1
  for (int u = 0; u < mine; ++u) s_list[slot + u] = blocks_of(q, p, u) + kUnitCost;
  __syncthreads();
  const int64_t trial = share + (share * warp >> 7);
  int left = 0;
#pragma unroll 1
  for (int i = lane; i < units; i += 32) {
    const int over = static_cast<int>(s_list[i] % trial);
    left += static_cast<int>(64 * (over ? trial - over : 0) / trial);
  }
  left = __reduce_add_sync(0xffffffffu, left);
  if (lane == 0) s_left[warp] = left;
  __syncthreads();
  int best = 0;
#pragma unroll 1
  for (int w = 1; w < kThreads / 32; ++w)
    if (s_left[w] < s_left[best]) best = w;
  return share + (share * best >> 7);
}

// ---- the main kernel -------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                  const __grid_constant__ CUtensorMap map_o1, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  // before the first tile Q's place serves the scan
  int64_t* s_sum = reinterpret_cast<int64_t*>(smem);  // [warps]
  int64_t* s_start = s_sum + kThreads / 32;           // the share's first sequence, the length before it
  const PromptParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t base = smem_u32(smem);
  if (tid == 0) {
    auto init = [&](int at, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + at) + i, count);
    };
    init(Smem::q_full, 1, 1), init(Smem::q_empty, 1, 1);
    init(Smem::kv_full, kStages, 1), init(Smem::kv_empty, kStages, 1), init(Smem::v_look, kStages, 1), init(Smem::v_ok, kStages, 4);
    init(Smem::s_full, 2, 1), init(Smem::p_full, 4, 4), init(Smem::half, 2, 1), init(Smem::o_full, 2, 1);
    init(Smem::staged, 2, 4), init(Smem::piece_full, kPieces, 1), init(Smem::piece_empty, kPieces, kReaders);
    init(Smem::fin, 1, 1);
    mbar_fence_init();
    for (const CUtensorMap* m : {&map_k, &map_q, &map_v, &map_o, &map_o1})
      asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
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
    mine += length_of_seq(q, p) * a.hkv;
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
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t x = s_sum[w];
    if (w < warp) upto += x;
    total += x;
  }
  int64_t share = max((total + p.ctas - 1) / p.ctas, int64_t{1});
  if (chunk <= 1 && share >= kLongShare && a.num_keys * static_cast<int64_t>(a.hkv) >= kManyKeys)
    share = aligned_share(p, total, share, tid < n ? load_seq(a, tid) : Seq{}, s_sum);
  const int64_t at = blockIdx.x * share;
  if (upto - mine <= at && at < upto) {
    int64_t c = upto - mine;
    int s = s_lo;
#pragma unroll 1
    for (; s + 1 < s_hi; ++s) {
      const int64_t b = length_of_seq(load_seq(a, s), p) * a.hkv;
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
  const int start_s = at < total ? static_cast<int>(s_start[0]) : 0;
  const int64_t start_c = at < total ? s_start[1] : 0;
  __syncthreads();  // the scan's place is Q's again
  // (short: the code of all kinds of warps shares the instruction cache; who gave up says so at the end)
  bool alive = true;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    bool there = false;
#pragma unroll 1
    for (uint32_t i = 0; alive && !there && i < BSP_WAIT_ROUNDS; ++i) there = __all_sync(0xffffffffu, try_wait(bar, parity));
    return alive = there;
  };
  // the next announced piece (nblk 0: no more)
  uint32_t number = 0;
  auto next = [&](Piece& e) {
    const uint32_t i = number % kPieces;
    if (!wait(base + Smem::piece_full + 8 * i, number / kPieces & 1)) return false;
    e = reinterpret_cast<const Piece*>(smem + Smem::pieces)[i];
    __syncwarp();
    if (lane == 0) arrive(base + Smem::piece_empty + 8 * i);
    ++number;
    return e.nblk > 0;
  };
  auto stage_of = [](uint32_t item) { return item % kStages; };
  auto phase_of = [](uint32_t item) { return item / kStages & 1; };
  Piece e;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kWarpTma) {
      // ---- producer: announces each piece, loads Q, and K and V of its blocks ----
      Walk w;
      w.at = at, w.end = min(at + share, total), w.share = share;
      const bool any = at < w.end;
      if (any) w.find(p, start_s, start_c);
      Cut* cut = static_cast<Cut*>(a.ws);
      if (lane == 0) cut[blockIdx.x].pieces = 0;
      uint32_t item = 0, q_loads = 0;
      auto load = [&](const CUtensorMap* m, int h, int row) {
        const uint32_t st = stage_of(item);
        if (!wait(base + Smem::kv_empty + 8 * st, phase_of(item) ^ 1)) return;
        const uint32_t bar = base + Smem::kv_full + 8 * st, dst = base + Smem::kv + st * kTileBytes;
        arrive_expect(bar, kTileBytes);
        tile_g2s_3d(dst, m, 0, h, row, bar);
        tile_g2s_3d(dst + kHalf, m, 64, h, row, bar);
        ++item;
      };
      bool more = true;
#pragma unroll 1
      for (uint32_t k = 0; alive && more; ++k) {
        more = any && w.next(p, e);
        if (!more) e.nblk = 0;
        e.item = item;
        const uint32_t i = k % kPieces;
        if (!wait(base + Smem::piece_empty + 8 * i, (k / kPieces & 1) ^ 1)) break;
        if (lane == 0) {
          reinterpret_cast<Piece*>(smem + Smem::pieces)[i] = e;
          if (more && e.pieces) cut[blockIdx.x] = {e.pieces, e.tok0, e.tokens, e.h, e.see, {0, 0, 0}};
          arrive(base + Smem::piece_full + 8 * i);
        }
        __syncwarp();
        if (!more) break;
        const bool two = e.tokens > p.tokens / 2;
        load(&map_k, e.h, e.k0 + e.b0 * kBlock);
        if (!wait(base + Smem::q_empty, (q_loads & 1) ^ 1)) break;
        arrive_expect(base + Smem::q_full, two ? 2 * kTileBytes : kTileBytes);
        for (int t = 0; t < (two ? 2 : 1); ++t)
          for (int d = 0; d < 2; ++d)
            tile_g2s_3d(base + Smem::q + t * kTileBytes + d * kHalf, &map_q, 64 * d, e.h * a.group,
                        e.tok0 + t * (p.tokens / 2), base + Smem::q_full);
        ++q_loads;
        load(&map_v, e.h, e.k0 + e.b0 * kBlock);
#pragma unroll 1
        for (int b = e.b0 + 1; alive && b < e.b0 + e.nblk; ++b) {
          load(&map_k, e.h, e.k0 + b * kBlock);
          if (alive) load(&map_v, e.h, e.k0 + b * kBlock);
        }
        if (e.starts && e.ends) {  // a stage each for O of the tiles
          for (int t = 0; alive && t < (two ? 2 : 1); ++t) {
            const uint32_t st = stage_of(item);
            if (!wait(base + Smem::kv_empty + 8 * st, phase_of(item) ^ 1)) break;
            if (lane == 0) arrive(base + Smem::kv_full + 8 * st);
            ++item;
          }
        }
      }
      // nothing may still write shared memory when the CTA leaves
      if (q_loads) wait_warp(base + Smem::q_full, (q_loads - 1) & 1, a.err, kSleepWaitLimit);
      for (uint32_t i = item > kStages ? item - kStages : 0; i < item; ++i)
        wait_warp(base + Smem::kv_full + 8 * stage_of(i), phase_of(i), a.err, kSleepWaitLimit);
    } else if (warp == kWarpMma) {
      // ---- issuer ----
      uint32_t q_phase = 0, p_phase = 0, ok_phase = 0;
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
      auto fence = [] { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); };
      while (alive && next(e)) {
        const bool two = e.tokens > p.tokens / 2;
        const int masked = e.see >> 7;  // blocks from here on some row does not see whole (see < 0: all)
        uint32_t st = stage_of(e.item), ph = phase_of(e.item);
        auto step = [&] {
          if (++st == kStages) st = 0, ph ^= 1;
        };
        uint32_t vs = 0, ks = st;
        // V of block j and K of the one behind it
        auto ready = [&](int j) {
          vs = st;
          if (!wait(base + Smem::kv_full + 8 * st, ph)) return;
          step();
          // (the ones that check wait for this one's word, not for the copy: of a stage whose
          // turns they do not follow one by one its parity says nothing)
          if (e.b0 + j >= masked && lane == 0) arrive(base + Smem::v_look + 8 * vs);
          __syncwarp();
          if (j + 1 < e.nblk) {
            ks = st;
            if (!wait(base + Smem::kv_full + 8 * st, ph)) return;
            step();
          }
        };
        if (!wait(base + Smem::q_full, q_phase)) break;
        q_phase ^= 1;
        if (!wait(base + Smem::kv_full + 8 * st, ph)) break;
        step();
        fence();
        scores(0, ks);
        if (two) scores(1, ks);
        commit(base + Smem::kv_empty + 8 * ks);
        if (e.nblk == 1) commit(base + Smem::q_empty);
        ready(0);
#pragma unroll 1
        for (int j = 0; alive && j < e.nblk; ++j) {
          const bool more = j + 1 < e.nblk;
          const uint32_t v = vs, k = ks;
          const uint64_t vd = v_desc + v * (kTileBytes / 16);
          if (e.b0 + j >= masked) {
            if (!wait(base + Smem::v_ok + 8 * v, ok_phase >> v & 1)) break;
            ok_phase ^= 1u << v;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i && !two) break;
            if (!wait(base + Smem::p_full + 16 * i, p_phase >> i & 1)) break;
            fence();
#pragma unroll
            for (int c = 0; c < 4; ++c)  // O (+)= P V of 64 keys
              umma_ts(tmem + 256 + i * 128, tmem + i * 128 + 8 * c, vd + c * (2048 / 16), kIdescO, j > 0 || c > 0);
            commit(base + Smem::half + 8 * i);
            if (!wait(base + Smem::p_full + 16 * i + 8, p_phase >> i & 1)) break;
            p_phase ^= 1u << i;
            fence();
#pragma unroll
            for (int c = 4; c < 8; ++c)
              umma_ts(tmem + 256 + i * 128, tmem + i * 128 + 8 * c, vd + c * (2048 / 16), kIdescO, 1);
            if (i == (two ? 1 : 0)) {
              commit(base + Smem::kv_empty + 8 * v);
              // (the next block's V and K are waited for while the tensor core has work queued)
              if (more) ready(j + 1);
              if (!alive) break;
            }
            if (more)
              scores(i, k);
            else
              commit(base + Smem::o_full + 8 * i);
          }
          if (more) commit(base + Smem::kv_empty + 8 * k);
          if (j + 2 == e.nblk) commit(base + Smem::q_empty);
        }
      }
      // every MMA and commit has ended
      commit(base + Smem::fin);
      wait_warp(base + Smem::fin, 0, a.err, kSleepWaitLimit);
    } else if (warp == kWarpStore) {
      // ---- the staged rows of O to global memory ----
      uint32_t phase = 0;
      while (alive && next(e)) {
        if (!(e.starts && e.ends)) continue;
        const bool two = e.tokens > p.tokens / 2;
        for (int t = 0; t < (two ? 2 : 1); ++t) {
          const uint32_t st = stage_of(e.item + 2 * e.nblk + t), src = base + Smem::kv + st * kTileBytes;
          if (!wait(base + Smem::staged + 8 * t, phase >> t & 1)) break;
          phase ^= 1u << t;
          const int tok0 = e.tok0 + t * (p.tokens / 2), tokens = min(e.tokens - t * (p.tokens / 2), p.tokens / 2);
          if (tokens == p.tokens / 2) {
            if (lane < 2) tile_s2g_3d(&map_o, 64 * lane, e.h * a.group, tok0, src + lane * kHalf);
          } else {  // a token at a time: the rows behind are another sequence's
            for (int i = lane; i < 2 * tokens; i += 32)
              tile_s2g_3d(&map_o1, 64 * (i & 1), e.h * a.group, tok0 + (i >> 1), src + (i & 1) * kHalf + (i >> 1) * a.group * 128);
          }
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
          if (lane == 0) arrive(base + Smem::kv_empty + 8 * st);
        }
      }
    } else if (warp >= kWarpCheck) {
      // ---- V of the blocks that some row does not see whole: a warp takes 64 dims of half the keys ----
      uint32_t look_phase = 0;
      const uint32_t part = base + Smem::kv + ((warp - kWarpCheck) & 1) * kHalf + lane * 16;
      while (alive && next(e)) {
        const int masked = max(e.see >> 7, e.b0);
#pragma unroll 1
        for (int b = masked; b < e.b0 + e.nblk; ++b) {
          const uint32_t item = e.item + 2 * (b - e.b0) + 1, st = stage_of(item);
          if (!wait(base + Smem::v_look + 8 * st, look_phase >> st & 1)) break;
          look_phase ^= 1u << st;
          if (!wait(base + Smem::kv_full + 8 * st, phase_of(item))) break;
          const uint32_t at = part + st * kTileBytes;
          // keys from the first that some row does not see on, four at a time
          const int from = (max(e.see - b * kBlock, 0) & ~3) + 4 * ((warp - kWarpCheck) >> 1);
          uint32_t acc[4] = {0, 0, 0, 0};
#pragma unroll 4
          for (int i = from; i < kBlock; i += 8) {
            const uint4 v = lds128(at + i * 128);
            acc[0] = add_zero_times(acc[0], v.x), acc[1] = add_zero_times(acc[1], v.y);
            acc[2] = add_zero_times(acc[2], v.z), acc[3] = add_zero_times(acc[3], v.w);
          }
          const uint32_t any = not_finite(acc[0]) | not_finite(acc[1]) | not_finite(acc[2]) | not_finite(acc[3]);
          if (__any_sync(0xffffffffu, any != 0)) {
#pragma unroll 1
            for (int i = from; i < kBlock; i += 8) {
              const uint4 v = lds128(at + i * 128);
              auto clean = [](uint32_t x) { return x & ~((not_finite(x) >> 15) * 0xFFFFu); };
              sts128(at + i * 128, clean(v.x), clean(v.y), clean(v.z), clean(v.w));
            }
            if (lane == 0) reinterpret_cast<volatile int*>(smem + Smem::bad)[number & 7] = number;
            fence_proxy_async();
          }
          __syncwarp();
          if (lane == 0) arrive(base + Smem::v_ok + 8 * st);
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
    const uint32_t s_full = base + Smem::s_full + 8 * tile, p_full = base + Smem::p_full + 16 * tile;
    uint32_t s_phase = 0, o_phase = 0;
    const float c = p.c, cs = a.sm_scale < 0.f ? -c : c;
    const int log_group = 8 - p.log_tokens, tok = row >> log_group;
    const int tok_lo = (row & ~31) >> log_group, tok_hi = (row | 31) >> log_group;  // the warp's
    while (alive && next(e)) {
      if (tile && e.tokens <= p.tokens / 2) continue;
      float ref = kNoMax, l = 0.f;
      bool huge = false;
#pragma unroll 1
      for (int j = 0; j < e.nblk; ++j) {
        if (!wait(s_full, s_phase)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        // keys of the block that the row, and the first and last rows of the warp, see
        const int from = (e.b0 + j) * kBlock, lim = e.see + tok - from, lim_lo = e.see + tok_lo - from,
                  lim_hi = e.see + tok_hi - from;
        // the weights of 64 logits against the rows' references, as P's words, and their sum
        auto weights = [&](const uint32_t(&r)[2][32], uint32_t(&pk)[32]) {
          const float rc = -ref * c;
          float2 t[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 x = ffma2({__uint_as_float(r[i >> 4][2 * (i & 15)]), __uint_as_float(r[i >> 4][2 * (i & 15) + 1])},
                                   {cs, cs}, {rc, rc});
            const float2 w = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            t[i & 1] = fadd2(t[i & 1], w);
            pk[i] = pack_bf16x2(w.x, w.y);
          }
          return (t[0].x + t[0].y) + (t[1].x + t[1].y);
        };
        auto send = [&](int half, const uint32_t(&pk)[32], float sum) {
          l += sum;
          tmem_st32(s_at + 32 * half, pk);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0 && alive) arrive(p_full + 8 * half);
        };
        int half = 0;
        if (__builtin_expect(j > 0 && lim_lo >= kBlock && !huge, 1)) {  // the common way
          uint32_t r[2][32], r2[2][32], pk[32];
          tmem_ld32_issue(s_at, r[0]), tmem_ld32_issue(s_at + 32, r[1]);
          loaded(r[0]), loaded(r[1]);
          tmem_ld32_issue(s_at + 64, r2[0]), tmem_ld32_issue(s_at + 96, r2[1]);
          float sum = weights(r, pk);
          const bool fits = !__any_sync(0xffffffffu, sum > kMaxSum);
          loaded(r2[0]), loaded(r2[1]);
          if (__builtin_expect(fits, 1)) {
            send(0, pk, sum);
            half = 1;
            sum = weights(r2, pk);
            if (__builtin_expect(!__any_sync(0xffffffffu, sum > kMaxSum), 1)) {
              send(1, pk, sum);
              half = 2;
            }
          }
        }
#pragma unroll 1
        for (; half < 2; ++half) {
          uint32_t r[2][32], pk[32];
          float sum = 0.f;
          if (lim_hi <= 64 * half) {  // no row of the warp sees any
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = 0;
          } else {
            tmem_ld32_issue(s_at + 64 * half, r[0]), tmem_ld32_issue(s_at + 64 * half + 32, r[1]);
            loaded(r[0]), loaded(r[1]);
            if (cs < 0.f) {  // (c is positive from here on)
#pragma unroll
              for (int i = 0; i < 64; ++i) r[i >> 5][i & 31] ^= 0x80000000u;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
              if (lim_lo < 64 * half + 32 * q + 32) {
                const int m = lim - 64 * half - 32 * q;
#pragma unroll
                for (int i = 0; i < 32; ++i) r[q][i] = i < m ? r[q][i] : 0xFF800000u;
              }
            bool again = half == 0 && j == 0;  // the first reference is the half's maximum
#pragma unroll 1
            for (int turn = 0; turn < 2; ++turn) {
              if (again) {
                // the rows' references pass this half's maxima; O and l in their terms
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  auto z = [&](int i) { return __uint_as_float(r[k >> 1][16 * (k & 1) + i]); };
                  mx[k] = fmax3(z(0), z(1), z(2));
#pragma unroll
                  for (int i = 3; i < 15; i += 2) mx[k] = fmax3(mx[k], z(i), z(i + 1));
                  mx[k] = fmaxf(mx[k], z(15));
                }
                const float to = fmaxf(fmax3(ref, mx[0], mx[1]), fmaxf(mx[2], mx[3])), f = rescale(ref, to, c);
                ref = to;
                huge = __any_sync(0xffffffffu, !(fabsf(ref * c) < kBigRef));
                l *= f;
                if (j > 0 || half) {  // (S says that the block before is in O)
                  if (half) {
                    wait(base + Smem::half + 8 * tile, s_phase);
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                  }
#pragma unroll 1
                  for (int k = 0; k < 128; k += 8) {
                    float y[8];
                    tmem_ld<8>(o_at + k, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] *= f;
                    tmem_st<8>(o_at + k, y);
                  }
                }
              }
              float2 t[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float2 x = fmul2(fadd2({__uint_as_float(r[i >> 4][2 * (i & 15)]), __uint_as_float(r[i >> 4][2 * (i & 15) + 1])},
                                             {-ref, -ref}), {c, c});
                const float2 w = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                t[i & 1] = fadd2(t[i & 1], w);
                pk[i] = pack_bf16x2(w.x, w.y);
              }
              sum = (t[0].x + t[0].y) + (t[1].x + t[1].y);
              if (again || !__any_sync(0xffffffffu, sum > kMaxSum)) break;
              again = true;
            }
          }
          send(half, pk, sum);
        }
        s_phase ^= 1;
      }
      if (!wait(base + Smem::o_full + 8 * tile, o_phase)) break;
      o_phase ^= 1;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      // -- O to where it goes
      const bool all = e.starts && e.ends;
      const int see = max(e.see + tok, 0);
      const float f = !all ? 1.f : see == 0 ? 0.f : 1.f / l;
      const bool fix = reinterpret_cast<volatile int*>(smem + Smem::bad)[number & 7] == static_cast<int>(number);
      const uint32_t item = e.item + 2 * e.nblk + tile, stage = base + Smem::kv + stage_of(item) * kTileBytes + (row & 127) * 128;
      if (all && !wait(base + Smem::kv_full + 8 * stage_of(item), phase_of(item))) break;
      // a CTA's slots: 2 * CTA for a unit that began before its share, + 1 for one that
      // goes on after it; [dims / 4][rows][4], then (m, l) of the rows
      float* po = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + list_bytes(p.ctas)) +
                  (2LL * blockIdx.x + (e.starts ? 1 : 0)) * kSlotFloats;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t r[32];
        tmem_ld32_issue(o_at + 32 * k, r);
        loaded(r);
        auto o = [&](int i) { return __uint_as_float(r[i]); };
        if (all) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // 16-byte chunks of the swizzled row
            uint32_t w[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const float2 x = fmul2({o(8 * i + 2 * n), o(8 * i + 2 * n + 1)}, {f, f});
              w[n] = pack_bf16x2(x.x, x.y);
            }
            sts128(stage + (k >> 1) * kHalf + (((4 * (k & 1) + i) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<float4*>(po)[(8 * k + i) * kRows + row] =
                make_float4(o(4 * i), o(4 * i + 1), o(4 * i + 2), o(4 * i + 3));
        }
      }
      if (__builtin_expect(fix, 0) && tok < e.tokens) {
        // what the row sees of V's values that are not finite (the MMAs read zeros in their place)
        const int to = min(see, (e.b0 + e.nblk) * kBlock);
#pragma unroll 1
        for (int t = max(e.b0, max(e.see >> 7, 0)) * kBlock; t < to; ++t) {
          const uint16_t* v = a.v + (e.k0 + static_cast<int64_t>(t)) * a.v_stride + e.h * kDim;
#pragma unroll 1
          for (int d = 0; d < kDim; ++d) {
            if ((v[d] & 0x7F80) != 0x7F80) continue;
            uint16_t* x = reinterpret_cast<uint16_t*>(smem + (stage - base) + (d >> 6) * kHalf +
                                                      ((((d & 63) >> 3) ^ (row & 7)) << 4)) + (d & 7);
            float* y = po + (d >> 2) * (kRows * 4) + row * 4 + (d & 3);
            const float sum = (all ? bf16_bits_to_float(*x) : *y) + bf16_bits_to_float(v[d]);
            if (all)
              *x = static_cast<uint16_t>(pack_bf16x2(sum, 0.f));
            else
              *y = sum;
          }
        }
      }
      __syncwarp();
      if (!all) *reinterpret_cast<float2*>(po + kRows * kDim + 2 * row) = make_float2(ref, l);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      if (all) {
        fence_proxy_async();  // the copies read the stage through the async proxy
        __syncwarp();
        if (lane == 0) arrive(base + Smem::staged + 8 * tile);
      }
    }
    __syncwarp();
  }
  if (!alive && lane == 0) set_err(a.err, BSP_DEVERR_TIMEOUT);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kWarpMma) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ---- cut units -----------------------------------------------------------------------------
// Joins the pieces of the units that share borders cut.  A warp takes eight rows, a lane 32
// dims of one of them, a fourth of each 16.
constexpr int kJoinParts = 4;  // CTAs of a unit
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  pdl_trigger();
  const PromptParams& a = p.a;
  const int lane = threadIdx.x & 31, log_group = 8 - p.log_tokens;
  const int c0 = blockIdx.x / kJoinParts;
  const Cut u = static_cast<const Cut*>(a.ws)[c0];
  if (u.pieces == 0) return;
  const int row = blockIdx.x % kJoinParts * (kRows / kJoinParts) + (threadIdx.x >> 5) * 8 + (lane & 7), part = lane >> 3;
  static_assert(kRows / kJoinParts == 64);
  const int tok = row >> log_group;
  if (tok >= u.tokens) return;
  const float* base = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + list_bytes(p.ctas));
  auto slot = [&](int k) { return base + (k ? 2LL * (c0 + k) : 2LL * c0 + 1) * kSlotFloats; };
  float M = kNoMax;
#pragma unroll 8
  for (int k = 0; k < u.pieces; ++k) M = fmaxf(M, slot(k)[kRows * kDim + 2 * row]);
  float L = 0.f;
  float4 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < u.pieces; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(slot(k) + kRows * kDim + 2 * row);
    const float w = rescale(ml.x, M, p.c);
    L += w * ml.y;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 y = reinterpret_cast<const float4*>(slot(k))[(4 * i + part) * kRows + row];
      x[i].x += w * y.x, x[i].y += w * y.y, x[i].z += w * y.z, x[i].w += w * y.w;
    }
  }
  const float f = u.see + tok <= 0 ? 0.f : 1.f / L;
  uint16_t* out = a.out + (static_cast<int64_t>(u.tok0 + tok) * a.hkv * a.group + u.h * a.group + (row & (a.group - 1))) * kDim;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint2*>(out + 16 * i + 4 * part) =
        make_uint2(pack_bf16x2(x[i].x * f, x[i].y * f), pack_bf16x2(x[i].z * f, x[i].w * f));
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
  CUtensorMap mq, mk, mv, mo, mo1;
  // (no keys at all: the maps of K and V have one row, Q's first, which no row sees)
  const bool keys = a.num_keys > 0;
  const int64_t hq = static_cast<int64_t>(a.hkv) * a.group;
  if (!make_map_rows(&mq, a.q, hq, a.num_tokens, a.q_stride, a.group, kTile / a.group) ||
      !make_map_rows(&mk, keys ? a.k : a.q, a.hkv, keys ? a.num_keys : 1, keys ? a.k_stride : a.q_stride, 1, kBlock) ||
      !make_map_rows(&mv, keys ? a.v : a.q, a.hkv, keys ? a.num_keys : 1, keys ? a.v_stride : a.q_stride, 1, kBlock) ||
      !make_map_rows(&mo, a.out, hq, a.num_tokens, hq * kDim, a.group, kTile / a.group) ||
      !make_map_rows(&mo1, a.out, hq, a.num_tokens, hq * kDim, a.group, 1))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [] {  // the shared-memory opt-in
    return cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::total);
  });
  if (e != cudaSuccess) return e;
  e = launch_kernel(prompt_kernel, dim3(static_cast<unsigned>(p.ctas)), dim3(kThreads), Smem::total, s, 0, mq, mk, mv, mo, mo1, p);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (a.num_keys > kWhole * kBlock) {  // units may be cut
    e = launch_kernel(prompt_join_kernel, dim3(static_cast<unsigned>(p.ctas * kJoinParts)), dim3(256), 0, s, 0, p);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaPeekAtLastError();
}

}  // namespace bsp
