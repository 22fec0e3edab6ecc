// Attention over the paged cache (hyq_paged_attention and its block-sparse
// form hyq_paged_attention_blocks).
//
// For each query token i of a sequence and query head h of a KV head,
//   out = sum_j 2^(x_j - M) v_j / sum_j 2^(x_j - M),  x_j = log2(e) q.k_j / sqrt(128),
// over the positions j that the token sees, k_j and v_j = c s + z from the
// pages: one pass with the running maximum and sum of a softmax (q_tiles in
// hyq_qtile.cuh: codes as fp16 subnormals on mma.sync, scales and zeros
// applied outside).
//
// What bounds it: the cache is read once, 160 bytes per (position, KV head)
// for 4-bit codes, against 4 * 128 * g flops: HBM, then instruction issue.
//
// Work split: a group is one (sequence, KV head, tile of up to 8 query rows)
// and has ceil(len / rows of a unit) units, a unit being what a warp copies
// and multiplies in one go.  The units of all groups, laid end to end, are cut
// into equal runs, one per block (two blocks an SM), so that unlike lengths
// and single long sequences use the GPU alike and the launch does not depend
// on the lengths (they live on the device; a captured call stays valid as
// they grow).  In the line each group begins with kCost units that are not
// there, about what preparing its queries and joining its warps takes: with too
// few of them a block that meets many short groups finishes last (two tokens of
// 16 sequences over chosen blocks: 142 us with 8 tiles' worth, 118 with 16, 102
// with 48).
// A group inside one run is finished by its block; one that several runs share
// is joined from their partials (maximum, sum, accumulator) in run order by
// the last block to finish, an atomic ticket that nobody waits for.
#include "hyq_paged.cuh"
#include "hyq_qtile.cuh"

namespace {

constexpr int kWarps = 8;              // warps that share out a group's units, each with a ring of its own
constexpr int kThreads = kWarps * 32;
constexpr int kRowsQ = HYQ_MAX_GQA;    // query rows per tile (MMA N)
constexpr int kPart = kPartFloats;
constexpr int kMinUnits = 8;           // units per block before a group is split further
constexpr int kMaxNQ = 4;             // query tiles that one block takes together

// The kernel's shape for NQ query tiles a group.  One tile: two blocks an SM
// (one's group change hides behind the other) and, for 4-bit codes, units of
// two adjacent 16-row tiles.  kMaxNQ: one block an SM, and two warps to a ring,
// each with half of the query tiles, whose accumulators leave 16 warps' worth of
// registers (one warp with all four at 8 warps an SM waited more than the codes
// unpacked twice cost: 74 against 66 us for 32 query rows a KV head, 8-bit codes,
// 8 sequences of up to 16 thousand positions).
template <int BK, int BV, int NQ>
struct Ring : QFmt<BK, BV> {
  static constexpr int kHalves = NQ == 1 ? 1 : 2;  // warps that work on one ring
  static constexpr int kNW = NQ / kHalves;         // query tiles of a warp
  static constexpr int kQuery = NQ == 1 ? 2048 : kPairQuery;  // bytes of a query tile's operands
  static_assert(kNW <= 2, "one query tile, or a pair");
  static constexpr int kPerSm = NQ == 1 ? 2 : 1;
  static constexpr int kBlockThreads = kThreads * kHalves;
  static constexpr int kTiles = BK + BV == 8 && NQ == 1 ? 2 : 1;  // tiles per unit
  static constexpr int kUnit = kTiles * QFmt<BK, BV>::kTile;
  static constexpr int kSlots = NQ > 1 ? (4096 * NQ + kUnit - 1) / kUnit : BK + BV == 12 ? 3 : 2;
  static constexpr int kCost = (NQ == 1 ? 48 : 16 * NQ) / kTiles;  // units that a group's fixed work is worth
  static constexpr int kRows = 16 * kTiles;
  static constexpr int kPerPage = HYQ_PAGE_ROWS / kRows;
  static constexpr int kWarpBytes = kSlots * kUnit;
  static constexpr int kSmemBytes = kWarps * kWarpBytes;
  static_assert(NQ * 4096 <= kWarpBytes && kSlots <= 32, "the query tiles' partials fit a ring");
  static_assert(kWarps % kPerPage == 0, "a warp's units take the same part of their pages");
};

// What a call leaves behind for a query row: its output; that and the logarithm of
// its softmax sum (hyq_paged_attention_lse); or, over the positions behind what
// its group shares, its accumulator, maximum and sum, which are joined with the
// shared positions' later (hyq_paged_attention_shared).
enum { kOut, kOutLse, kRest };

struct Params {
  PageView pv;
  const int32_t* seqs;
  const __nv_bfloat16* q;
  int64_t ldq;
  const int32_t* sel;  // [batch][n_q][HKV][k_sel] or nullptr
  __nv_bfloat16* out;
  float* part;         // [grid][2][NQ][8][kPart]
  int32_t* tickets;    // [groups]
  int32_t batch, n_q, HQ, HKV, gq, k_sel;
  int32_t QT;          // groups per (sequence, KV head)
  float* lse;          // kOutLse: [batch][n_q][HQ]
  SharedRows shared;   // kRest
  float* rest;         // kRest: [batch][n_q][HQ][kPart]
};

// Length of call row b, 0 for a sequence out of range.
__device__ __forceinline__ int row_len(const Params& p, int b, int* seq) {
  const int s = page_seq(p.seqs, b, p.pv.n_seqs);
  *seq = s;
  if (s < 0) return 0;
  const int64_t cap = (int64_t)p.pv.max_blocks * HYQ_PAGE_ROWS;
  const int n = p.pv.lens[s];
  return n < 0 ? 0 : (int64_t)n > cap ? (int)cap : n;
}

// a / b for 0 <= a, 0 < b: 32-bit arithmetic whenever both fit.
__device__ __forceinline__ int64_t div_fast(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// T units over nb blocks: the first `more` blocks take `each` + 1 tiles, the others `each`.
struct Shares {
  int64_t each, more;
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int owner(int64_t x) const {  // of unit x
    const int64_t wide = more * (each + 1);
    return (int)(x < wide ? div_fast(x, each + 1) : more + div_fast(x - wide, each));
  }
};

// A block's run of units and what it is doing: kept in shared memory, where
// thread 0 keeps it up, so that the main loop's registers are its own.
struct Run {
  Shares sh;
  int64_t pos, end;
};
struct Segment {
  int b, h, qt, len;        // row of the call, KV head, group of its query rows; positions
  int w0, w1, n_units;      // units [w0, w1) of the group's n_units (w0 < 0: none are left)
  int n_rows, flat0;        // query rows of the group, the first one's (token, head) pair
  const int32_t* table;     // of the sequence
  const int32_t* sel;       // the group's list of blocks, or nullptr
  __nv_bfloat16* out;       // of (row b, KV head h)
  int64_t base;             // of the group's first unit in the line
};

// A ring's state beside its bytes: of one warp, or of two.
template <int kHalves, int kSlots>
struct Ctl {
  uint64_t full[kSlots];  // the slot's copy is there
};
template <int kSlots>
struct Ctl<2, kSlots> {
  uint64_t full[kSlots];
  uint64_t free[kSlots];  // the second half's warp is done with it
  int at[kSlots];         // position of the slot's first row, or -1 (nothing was copied)
};
// Barriers by their shared memory addresses.
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_at(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done;
}
// A warp's wait, bounded like mbar_wait; false for every lane if one gave up.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_at(bar, parity))) return true;  // as a rule
  bool done = false;
  for (int it = 0; !done && it < (1 << 22); ++it) done = mbar_try_at(bar, parity);
  return __all_sync(0xffffffffu, done);
}
__device__ __forceinline__ void mbar_expect_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_g2s_at(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Output row of (token, head) pair `flat` of a KV head whose first row is `out`.
__device__ __forceinline__ __nv_bfloat16* out_row(__nv_bfloat16* out, int HQ, int gq, int flat) {
  const int tok = flat / gq;
  return out + ((size_t)tok * HQ + (flat - tok * gq)) * HYQ_D;
}

// The same row of an array with n floats a row.
__device__ __forceinline__ float* extra_row(float* extra, int HQ, int gq, int flat, int n) {
  const int tok = flat / gq;
  return extra + ((size_t)tok * HQ + (flat - tok * gq)) * n;
}
// ln(2^M L): of nothing minus infinity.
__device__ __forceinline__ float log_sum(float M, float L) { return (M + log2f(L)) * 0.6931471805599453f; }

// One block: joins the n partials of a group's n_rows rows, eight rows per 256 threads.  Part i lies at
// parts + i stride, the first one `first` further.  A thread takes four elements
// of a row over every S-th part, kHold parts at a time, with an online softmax
// of its own (each part's maximum and sum come with its elements, so there is
// one round of loads and nothing to wait for between them).  Out of line and
// short: the code runs once a launch, cold, and its instructions are fetched
// while the call waits (unrolled further it was slower).
template <int kHalves, int kLeave>
__device__ __noinline__ void join_parts(const float* parts, int first, int stride, int n, int n_rows, uint8_t* smem,
                                        __nv_bfloat16* out, int HQ, int gq, int flat0, float* extra) {
  const int half = kHalves > 1 ? threadIdx.x / kThreads : 0, tid = threadIdx.x - kThreads * half;
  smem += half * kThreads * (sizeof(float4) + sizeof(float2));
  float4* sums = reinterpret_cast<float4*>(smem);                                // [kThreads]
  float2* stats = reinterpret_cast<float2*>(smem + kThreads * sizeof(float4));  // [kThreads]
  constexpr int kHold = 10;
  for (int r0 = half * kRowsQ; r0 < n_rows; r0 += kHalves * kRowsQ) {
    const int items = min(kRowsQ, n_rows - r0) * (HYQ_D / 4), S = kThreads / items, share = tid / items;
    const int item = tid - share * items, r = r0 + (item >> 5), d = 4 * (item & 31);
    const int mine = share < S ? (n - share + S - 1) / S : 0;  // parts share, share + S, ...
    const size_t step = (size_t)S * stride;
    const float* at = parts + (size_t)share * stride + r * kPart;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < mine; k0 += kHold) {
      float2 ml[kHold];
      float4 v[kHold];
#pragma unroll
      for (int k = 0; k < kHold; ++k, at += step) {
        const bool in = k0 + k < mine;
        const float* e = at + (share + k0 + k == 0 ? first : 0);
        ml[k] = in ? __ldcg(reinterpret_cast<const float2*>(e + HYQ_D)) : make_float2(-INFINITY, 0.f);
        v[k] = in ? __ldcg(reinterpret_cast<const float4*>(e + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < kHold; ++k) top = fmaxf(top, ml[k].x);
      const float ref = top == -INFINITY ? 0.f : top, corr = ex2(M - ref);
      M = top;
      L *= corr, a.x *= corr, a.y *= corr, a.z *= corr, a.w *= corr;
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const float w = ex2(ml[k].x - ref);
        L = fmaf(ml[k].y, w, L);
        a.x = fmaf(w, v[k].x, a.x), a.y = fmaf(w, v[k].y, a.y), a.z = fmaf(w, v[k].z, a.z), a.w = fmaf(w, v[k].w, a.w);
      }
    }
    if (S > 1) {  // fewer than eight rows, or the last ones of a group
      sums[tid] = a;
      stats[tid] = make_float2(M, L);
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + half), "n"(kThreads) : "memory");  // this half's threads
    }
    if (share == 0) {
      float top = M;
      for (int k = 1; k < S; ++k) top = fmaxf(top, stats[k * items + item].x);
      const float ref = top == -INFINITY ? 0.f : top, own = ex2(M - ref);
      L *= own, a.x *= own, a.y *= own, a.z *= own, a.w *= own;
      for (int k = 1; k < S; ++k) {
        const float4 x = sums[k * items + item];
        const float2 ml = stats[k * items + item];
        const float w = ex2(ml.x - ref);
        L = fmaf(ml.y, w, L);
        a.x = fmaf(w, x.x, a.x), a.y = fmaf(w, x.y, a.y), a.z = fmaf(w, x.z, a.z), a.w = fmaf(w, x.w, a.w);
      }
      if (kLeave == kRest) {
        float* e = extra_row(extra, HQ, gq, flat0 + r, kPart);
        *reinterpret_cast<float4*>(e + d) = a;
        if (d == 0) *reinterpret_cast<float2*>(e + HYQ_D) = make_float2(top, L);
        continue;
      }
      if (kLeave == kOutLse && d == 0) *extra_row(extra, HQ, gq, flat0 + r, 1) = log_sum(top, L);
      const float inv = L > 0.f ? 1.f / L : 0.f;
      *reinterpret_cast<uint2*>(out_row(out, HQ, gq, flat0 + r) + d) =
          make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    }
  }
  __syncthreads();
}

template <int BK, int BV, int NQ, int kLeave>
__global__ void __launch_bounds__(Ring<BK, BV, NQ>::kBlockThreads, Ring<BK, BV, NQ>::kPerSm)
    paged_kernel(const Params p) {
  using R = Ring<BK, BV, NQ>;
  constexpr int kSlots = R::kSlots, kRowsG = NQ * kRowsQ;  // query rows per group
  constexpr int kHalves = R::kHalves, kNW = R::kNW;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_cum[HYQ_PAGED_MAX_BATCH + 1];  // units per (KV head, query tile) of the rows before b
  __shared__ int s_len[HYQ_PAGED_MAX_BATCH], s_seq[HYQ_PAGED_MAX_BATCH];
  __shared__ int s_skip[kLeave == kRest ? HYQ_PAGED_MAX_BATCH : 1];  // pages that are left to the group
  __shared__ float s_top[kLeave == kOut ? 1 : kRowsG];
  __shared__ int64_t s_warp[kWarps * kHalves];
  using Fragments = uint32_t[4][kRowsQ][4][4];
  __shared__ __align__(16) uint8_t query_s[NQ][R::kQuery];  // each begins with Fragments
  auto bq_s = [&](int k) -> Fragments& { return *reinterpret_cast<Fragments*>(query_s[k]); };
  __shared__ __align__(16) float rowc_s[NQ][kRowsQ][4];
  __shared__ uint32_t bz_s[NQ][kRowsQ][4];
  __shared__ int lim_s[NQ][kRowsQ];
  using RingCtl = Ctl<kHalves, kSlots>;
  __shared__ __align__(8) RingCtl s_ctl[kWarps];
  __shared__ float red_m[kWarps][NQ][kRowsQ], red_l[kWarps][NQ][kRowsQ];
  __shared__ __align__(16) uint32_t steps_s[kHalves == 1 ? 1 : kWarps * kHalves][32];  // each warp's scaled steps
  __shared__ float s_wt[kRowsG][kWarps];                // weights of the warps' partials
  __shared__ float s_sum[kRowsG];
  __shared__ int s_last;
  __shared__ Run run;
  __shared__ Segment seg;

  const int tid = threadIdx.x;
  int lane = tid & 31, half = kHalves > 1 ? tid / kThreads : 0, warp = (tid >> 5) - kWarps * half;
  // What a shuffle returns is kept: it cannot be formed anew, from the thread's
  // number or a variable's address, in each pass of the loop.
  auto kept = [&](uint32_t x) { return kHalves > 1 ? __shfl_sync(0xffffffffu, x, tid & 31) : x; };
  lane = (int)kept(lane), warp = (int)kept(warp), half = (int)kept(half);
  const int g = lane >> 2, t = lane & 3;
  // The warps w and w + 8 of two halves work on the same ring, w filling it.
  const int kq = kNW * half;
  uint8_t* ring = smem + warp * R::kWarpBytes;
  uint64_t* wb = s_ctl[warp].full;
  if (half == 0 && lane < kSlots) {
    mbar_init(&wb[lane], 1);
    if constexpr (kHalves > 1) mbar_init(&s_ctl[warp].free[lane], 1);
  }
  mbar_fence_init();
  chain_kernel();

  // Units of a group of row b: its own and those of the fixed work; 0 when
  // there is nothing to read.
  auto units_of = [&](int len) {
    int n = (len + R::kRows - 1) / R::kRows;
    if (p.sel) n = R::kPerPage * min(p.k_sel, (len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS);
    return n == 0 ? 0 : n + R::kCost;
  };
  // ---- the rows' units, summed up: a row a thread (the loads of several rows in
  // one thread would follow one another) --------------------------------------
  const int unit = p.HKV * p.QT;
  {
    int64_t before = 0;
    for (int row0 = 0; row0 < p.batch; row0 += R::kBlockThreads) {
      const int b = row0 + tid;
      int64_t w = 0;
      if (b < p.batch) {
        int seq;
        int len = row_len(p, b, &seq);
        if (kLeave == kRest) {
          const int skip = shared_len(p.shared, p.pv, p.seqs, b, p.batch, p.n_q);
          s_skip[b] = skip / HYQ_PAGE_ROWS;
          if (skip == 0 && seq >= 0 && blockIdx.x == 0 && p.shared.n) {  // a row that cannot share what it should
            const int i = group_of(p.shared, b);
            if (p.shared.cu[i] <= b && b < p.shared.cu[i + 1] && p.shared.len[i] != 0)
              hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
          }
          len -= skip;
        }
        s_len[b] = len;
        s_seq[b] = seq;
        if (seq < 0 && blockIdx.x == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        w = units_of(len);
      }
      int64_t pre = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
      }
      if (row0 > 0) __syncthreads();  // the sums of the rows before have been read
      if (lane == 31) s_warp[tid >> 5] = pre;
      __syncthreads();
      int64_t at = before + pre - w;
      for (int i = 0; i < kWarps * kHalves; ++i) {
        const int64_t x = s_warp[i];
        if (i < tid >> 5) at += x;
        before += x;
      }
      if (b < p.batch) s_cum[b] = at;
    }
    if (tid == 0) s_cum[p.batch] = before;
  }
  __syncthreads();
  // rows without positions: their outputs are zero
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x)
    if (s_cum[b] == s_cum[b + 1]) {
      uint4* o = reinterpret_cast<uint4*>(p.out + (size_t)b * p.n_q * p.HQ * HYQ_D);
      if (kLeave != kRest)
        for (int k = tid; k < p.n_q * p.HQ * (HYQ_D / 8); k += R::kBlockThreads) o[k] = make_uint4(0, 0, 0, 0);
      if (kLeave == kOutLse)
        for (int k = tid; k < p.n_q * p.HQ; k += R::kBlockThreads) p.lse[(size_t)b * p.n_q * p.HQ + k] = -INFINITY;
      if (kLeave == kRest)
        for (int k = tid; k < p.n_q * p.HQ; k += R::kBlockThreads) {
          float* e = p.rest + ((size_t)b * p.n_q * p.HQ + k) * kPart;
          for (int d = 0; d < HYQ_D; ++d) e[d] = 0.f;
          e[HYQ_D] = -INFINITY, e[HYQ_D + 1] = 0.f;
        }
    }
  // ---- this block's run -------------------------------------------------------
  // No more blocks than give each kMinUnits.  With few groups every group gets
  // the same number of blocks, unless that would leave more than a sixteenth of
  // the blocks out: equal lengths are then cut at the groups' borders.
  if (tid == 0) {
    const int64_t T = s_cum[p.batch] * unit, groups = (int64_t)p.batch * unit;
    const int64_t want = max((int64_t)1, div_fast(T, kMinUnits));
    int64_t nb = gridDim.x;
    if (groups <= nb) {
      const int64_t most = div_fast(nb, groups), by_size = max((int64_t)1, div_fast(want, groups));
      if (by_size < most || 16 * groups * most >= 15 * nb) nb = groups * min(most, by_size);
    }
    nb = max((int64_t)1, min(nb, T));
    run.sh.each = div_fast(T, nb);
    run.sh.more = T - run.sh.each * nb;
    run.pos = run.sh.begin(min((int64_t)blockIdx.x, nb));  // blocks past nb: an empty run
    run.end = run.sh.begin(min((int64_t)blockIdx.x + 1, nb));
  }

  uint32_t done = 0;  // units that this warp's ring has seen: slot done % kSlots, parity (done / kSlots) & 1
  bool dead = false;

  while (true) {
    // ---- the next group that the run meets (not only its fixed work) ----------
    if (tid == 0) {
      seg.w0 = -1;
      while (run.pos < run.end) {
        int lo = 0, hi = p.batch;  // the last b with unit * s_cum[b] <= pos
        while (hi - lo > 1) {
          const int m = (lo + hi) >> 1;
          if (s_cum[m] * unit <= run.pos) lo = m;
          else hi = m;
        }
        const int W = (int)(s_cum[lo + 1] - s_cum[lo]);  // with the fixed work's units
        const int64_t off = run.pos - s_cum[lo] * unit;
        const int grp = (int)div_fast(off, W), x0 = (int)(off - (int64_t)grp * W);
        const int x1 = (int)min((int64_t)W, x0 + (run.end - run.pos));
        run.pos += x1 - x0;
        if (x1 <= R::kCost) continue;  // the group is the next blocks'
        const int h = grp / p.QT, qt = grp - h * p.QT;
        seg.b = lo;
        seg.h = h;
        seg.qt = qt;
        seg.len = s_len[lo];
        seg.w0 = max(0, x0 - R::kCost);
        seg.w1 = x1 - R::kCost;
        seg.n_units = W - R::kCost;
        seg.n_rows = p.sel ? p.gq : min(kRowsG, p.n_q * p.gq - kRowsG * qt);
        seg.flat0 = p.sel ? qt * p.gq : qt * kRowsG;  // with block lists a group is one token's heads
        seg.table = p.pv.table + (size_t)s_seq[lo] * p.pv.max_blocks + (kLeave == kRest ? s_skip[lo] : 0);
        seg.sel = p.sel ? p.sel + (((size_t)lo * p.n_q + qt) * p.HKV + h) * p.k_sel : nullptr;
        seg.out = p.out + ((size_t)lo * p.n_q * p.HQ + (size_t)h * p.gq) * HYQ_D;
        seg.base = s_cum[lo] * unit + (int64_t)grp * W + R::kCost;
        break;
      }
    }
    __syncthreads();
    const int w0 = seg.w0, w1 = seg.w1;
    if (w0 < 0) break;
    // Row r of the group is (token, head) pair flat0 + r of the KV head's.
    auto token_of = [&](int r) { return (seg.flat0 + r) / p.gq; };
    // the query rows, row `warp` of each query tile: loaded ahead of the page
    // numbers, prepared while the first copies are under way
    uint2 qv[kNW];
#pragma unroll
    for (int k = 0; k < kNW; ++k) {
      const int r = kRowsQ * (kq + k) + warp, tok = token_of(r);
      qv[k] = make_uint2(0, 0);
      if (r < seg.n_rows)
        qv[k] = *reinterpret_cast<const uint2*>(
            p.q + ((size_t)seg.b * p.n_q + tok) * p.ldq +
            (size_t)(seg.h * p.gq + seg.flat0 + r - tok * p.gq) * HYQ_D + 4 * lane);
    }

    // ---- this warp's units: w0 + warp, + 8, ... ---------------------------
    // kPerPage divides 8, so all of them take the same part of their pages.
    const int nj = w1 - w0 > warp ? (w1 - w0 - warp + kWarps - 1) / kWarps : 0;
    const int part = (w0 + warp) % R::kPerPage, x_first = (w0 + warp) / R::kPerPage;
    const uint8_t* heads = p.pv.pool + (size_t)seg.h * R::kBlock + part * R::kUnit;
    // Block of the sequence that unit j lies in, or -1 for one that must not
    // be read.
    auto entry = [&](int j) -> int {
      if (j >= nj) return -1;
      const int x = x_first + j * (kWarps / R::kPerPage);
      if (NQ > 1 || !seg.sel) return x;  // several query tiles: never with lists
      const int e = seg.sel[x], pe = x > 0 ? seg.sel[x - 1] : -1;
      if (e < 0) return -1;
      if ((x > 0 && pe < 0) || pe >= e || (int64_t)e * HYQ_PAGE_ROWS >= seg.len) {
        hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        return -1;
      }
      return e;
    };
    auto page_of = [&](int e) -> int { return e < 0 ? -1 : seg.table[e]; };
    // Lane l holds block and page of unit 32 r + l of the present round r of 32
    // units, and of the next one; the pages arrive while the round is worked off.
    int e_cur = half == 0 ? entry(lane) : -1, pg_cur = page_of(e_cur);
    int e_nxt = half == 0 ? entry(32 + lane) : -1, pg_nxt = page_of(e_nxt);
    auto next_pages = [&](int j) {  // after unit j
      if ((j & 31) != 31) return;
      e_cur = e_nxt;
      pg_cur = pg_nxt;
      e_nxt = entry(j + 33 + lane);
      pg_nxt = page_of(e_nxt);
    };
    // Position of unit j's first row (of a unit that is there), else -1; issues its copy.
    auto issue = [&](int j) -> int {
      const int e = __shfl_sync(0xffffffffu, e_cur, j & 31), pg = __shfl_sync(0xffffffffu, pg_cur, j & 31);
      const int at = e * HYQ_PAGE_ROWS + part * R::kRows;
      const bool in = (uint32_t)pg < (uint32_t)p.pv.n_pages, ok = e >= 0 && at < seg.len && in;
      const uint32_t n = done + (uint32_t)j;
      const int slot = n % kSlots;
      if (lane == slot) {  // copies that one thread issues complete one after another
        uint64_t* bar = &wb[slot];
        if (ok) {
          const uint32_t bytes = R::kTiles == 1 || at + 16 < seg.len ? R::kUnit : R::kTile;
          mbar_arrive_expect_tx(bar, bytes);
          bulk_g2s(ring + slot * R::kUnit, heads + (size_t)pg * ((size_t)p.HKV * R::kBlock), bytes, bar);
        } else {
          mbar_arrive_expect_tx(bar, 0);
          if (e >= 0 && !in) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        }
      }
      next_pages(j);
      return ok ? at : -1;
    };
    // Two halves (no lists): unit j into the slot, by the lane that holds its page.
    const uint32_t ctl = kept(smem_u32(&s_ctl[warp])), tiles = kept(smem_u32(ring)), query = kept(smem_u32(query_s[kq])),
                   scaled = kept(smem_u32(steps_s[kHalves == 1 ? 0 : tid >> 5]));
    constexpr uint32_t kFree = 8 * kSlots, kAt = 16 * kSlots;  // Ctl<2, kSlots>
    auto issue_at = [&](int j, uint32_t slot) {
      if (lane == (j & 31)) {
        const bool in = (uint32_t)pg_cur < (uint32_t)p.pv.n_pages;
        sts32(ctl + kAt + 4 * slot, (uint32_t)(in ? R::kRows * (w0 + warp + kWarps * j) : -1));
        mbar_expect_at(ctl + 8 * slot, in ? R::kUnit : 0);
        if (in)
          bulk_g2s_at(tiles + slot * R::kUnit, heads + (size_t)pg_cur * ((size_t)p.HKV * R::kBlock), R::kUnit, ctl + 8 * slot);
        else
          hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
      }
      next_pages(j);
    };
    int at_slot[kHalves == 1 ? kSlots : 1];  // one half: the slots' positions from the next unit's on
    if constexpr (kHalves == 1) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) at_slot[j] = j < nj && !dead ? issue(j) : -1;
    } else {
      if (half == 0 && !dead)
        for (int j = 0; j < min(kSlots, nj); ++j) issue_at(j, (done + j) % kSlots);
    }

    // ---- the query rows: warp r prepares row r of each of its half's tiles --
#pragma unroll
    for (int k = 0; k < kNW; ++k) {
      const int r = kRowsQ * (kq + k) + warp;
      prep_query_row<BK>(warp, lane, qv[k], bq_s(kq + k), rowc_s[kq + k], bz_s[kq + k]);
      if (lane == 0) lim_s[kq + k][warp] = r < seg.n_rows ? max(0, seg.len - p.n_q + 1 + token_of(r)) : seg.len;
    }
    __syncthreads();
    uint32_t bq[8][2];
    QConst qc;
    const int minlim = lim_s[0][0];  // the rows' tokens ascend
    PageState<kNW> st;
    if constexpr (NQ == 1) {
      load_query_consts(g, t, bq_s(0), rowc_s[0], bz_s[0], bq, qc);
    } else {
      if (tid < 32 * NQ) spread_query_consts(query_s[tid >> 5], lane, rowc_s[tid >> 5], bz_s[tid >> 5]);
      __syncthreads();
    }
    reset_state(st);

    // A wait ran out: flag it, let this warp's other copies (units j0 .. j1 - 1)
    // land before shared memory is used for anything else, and stop.
    auto give_up = [&](int j0, int j1) {
      if (lane == 0) {
        hyq_set_err(p.pv.err, HYQ_DEVERR_TIMEOUT);
        if (half == 0)
          for (int k = j0; k < nj && k < j1; ++k)
            (void)mbar_wait(&wb[(done + k) % kSlots], ((done + k) / kSlots) & 1u);
      }
      __syncwarp();
      dead = true;
    };
    if constexpr (kHalves == 1) {
      for (int j = 0; j < nj && !dead; ++j) {
        const uint32_t n = done + (uint32_t)j;
        const int slot = n % kSlots;
        if (__any_sync(0xffffffffu, !mbar_wait(&wb[slot], (n / kSlots) & 1u))) {
          give_up(j, j + kSlots);
          break;
        }
        const int at = at_slot[0];
        uint8_t* tb = ring + slot * R::kUnit;
        if (at >= 0) {
          if (at + R::kRows <= minlim) {
            q_tiles<BK, BV, R::kTiles>(tb, lane, bq, qc, st);
          } else {
            const int lim0 = lim_s[0][2 * t], lim1 = lim_s[0][2 * t + 1];
            for (int x = 0; x < R::kTiles && at + 16 * x < seg.len; ++x) {
              const int a = at + 16 * x;
              q_tiles<BK, BV, 1, true>(tb + x * R::kTile, lane, bq, qc, st, seg.len - a, lim0 - a, lim1 - a);
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k + 1 < kSlots; ++k) at_slot[k] = at_slot[k + 1];
        if (j + kSlots < nj) {
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          at_slot[kSlots - 1] = issue(j + kSlots);
        }
      }
    } else {
      uint32_t slot = done % kSlots, par = (done / kSlots) & 1u;
      for (int j = 0; j < nj && !dead; ++j) {
        if (!mbar_wait_warp(ctl + 8 * slot, par)) {
          give_up(j, j + kSlots - (j > 0 ? 1 : 0));
          break;
        }
        const int at = (int)lds32<kAt>(ctl + 4 * slot);
        const uint32_t tb = tiles + slot * R::kUnit;
        if (at >= 0) {
          if (at + R::kRows <= minlim)
            q_tile_pair<BK, BV, false>(tb, lane, query, 16, lim_s + kq, at, scaled, st);
          else
            q_tile_pair<BK, BV, true>(tb, lane, query, seg.len - at, lim_s + kq, at, scaled, st);
        }
        __syncwarp();
        if (half == 1) {
          if (lane == 0) mbar_arrive_at(ctl + kFree + 8 * slot);
        } else if (j > 0 && j - 1 + kSlots < nj) {
          // the slot of the unit before, which the other half has mostly left too
          const uint32_t s0 = slot ? slot - 1 : kSlots - 1, p0 = slot ? par : par ^ 1u;
          if (!mbar_wait_warp(ctl + kFree + 8 * s0, p0)) {
            give_up(j + 1, j - 1 + kSlots);
            break;
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          issue_at(j - 1 + kSlots, s0);
        }
        if (++slot == kSlots) slot = 0, par ^= 1u;
      }
    }
    done += nj;

    // ---- the block's partial, a query tile at a time -------------------------
    __syncwarp();
    const int n_rows = seg.n_rows;
    const bool whole = seg.w0 == 0 && seg.w1 == seg.n_units;
    float* pp = p.part + ((size_t)blockIdx.x * 2 + (seg.w0 == 0 ? 1 : 0)) * (NQ * kRowsQ * kPart);
    float* extra = kLeave == kOut ? nullptr : (kLeave == kRest ? p.rest : p.lse) +
                   ((size_t)seg.b * p.n_q * p.HQ + (size_t)seg.h * p.gq) * (kLeave == kRest ? kPart : 1);
    if (kHalves > 1) __syncthreads();  // both halves are done with the rings
#pragma unroll
    for (int k = 0; k < kNW; ++k)
      store_warp_partial<BV>(st, k, g, t, reinterpret_cast<float*>(ring + 4096 * (kq + k)), red_m[warp][kq + k],
                             red_l[warp][kq + k]);
    __syncthreads();
    // eight lanes a row: its weights 2^(m_w - M) and its sum
    if (tid < kRowsG * kWarps) {
      const int r = tid >> 3, w = tid & 7;
      const float mw = red_m[w][r >> 3][r & 7];
      float M = mw;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float wt = mw == -INFINITY ? 0.f : ex2(mw - M);
      float L = red_l[w][r >> 3][r & 7] * wt;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      s_wt[r][w] = wt;
      if (w == 0) {
        s_sum[r] = L;
        if (kLeave != kOut) s_top[r] = M;
        if (!whole && r < n_rows) {
          pp[r * kPart + HYQ_D] = M;
          pp[r * kPart + HYQ_D + 1] = L;
        }
      }
    }
    __syncthreads();
    // four elements of a row a thread (the warps' partials hold element d at d ^ (row / 2))
    for (int i = tid; i < min(kRowsG, n_rows) * (HYQ_D / 4); i += R::kBlockThreads) {  // (the bound: a known count)
      const int r = i >> 5, d = 4 * (i & 31), x = (r & 7) >> 1;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(smem + w * R::kWarpBytes + 4096 * (r >> 3) +
                                                          4 * ((r & 7) * HYQ_D + d));
        const float wt = s_wt[r][w];
        a.x = fmaf(wt, v.x, a.x), a.y = fmaf(wt, v.y, a.y), a.z = fmaf(wt, v.z, a.z), a.w = fmaf(wt, v.w, a.w);
      }
      if (x & 1) a = make_float4(a.y, a.x, a.w, a.z);
      if (x & 2) a = make_float4(a.z, a.w, a.x, a.y);
      if (whole && kLeave == kRest) {
        float* e = extra_row(extra, p.HQ, p.gq, seg.flat0 + r, kPart);
        *reinterpret_cast<float4*>(e + d) = a;
        if (d == 0) *reinterpret_cast<float2*>(e + HYQ_D) = make_float2(s_top[r], s_sum[r]);
      } else if (whole) {
        if (kLeave == kOutLse && d == 0) *extra_row(extra, p.HQ, p.gq, seg.flat0 + r, 1) = log_sum(s_top[r], s_sum[r]);
        const float L = s_sum[r], inv = L > 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<uint2*>(out_row(seg.out, p.HQ, p.gq, seg.flat0 + r) + d) =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
      } else {
        *reinterpret_cast<float4*>(pp + r * kPart + d) = a;
      }
    }
    __syncthreads();  // the rings are free again
    if (!whole) {
      // blocks that share this group: those holding its first and last unit
      const int64_t base = seg.base;
      const int c0 = run.sh.owner(base), c1 = run.sh.owner(base + seg.n_units - 1);
      if (tid == 0) {
        int32_t* ticket = p.tickets + ((size_t)seg.b * p.HKV + seg.h) * p.QT + seg.qt;
        int old;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(old) : "l"(ticket) : "memory");
        s_last = old == c1 - c0;
        if (s_last) *ticket = 0;
      }
      __syncthreads();
      if (s_last) {
        // part i: slot 0 of block c0 + i, where its run ends or goes through this
        // group; the first block, whose run holds the group's first unit, has it
        // in slot 1
        constexpr int kSlot = NQ * kRowsQ * kPart;
        join_parts<kHalves, kLeave>(p.part + (size_t)c0 * 2 * kSlot, kSlot, 2 * kSlot, c1 - c0 + 1, n_rows,
                                    smem, seg.out, p.HQ, p.gq, seg.flat0, extra);
      }
    }
    __syncthreads();  // the segment is done with
    // order this block's generic accesses to the rings before the next copies
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
}

// Query tiles that a group takes together: one, or four.  One by one, the
// groups of one KV head lie side by side and meet most of each other's reads in
// L2, and the group's start is shorter; four at a time the codes are unpacked half
// as often, and the last four may lack one.  64 / 8 heads, 4 / 6 / 7 / 8 / 11 / 12 tiles, us:
//                                            one by one                      by fours
//   8-bit codes, 8 sequences of up to 16001   88 / 112 / 128 / 165 / 194 / 215   68 / 116 / 116 / 115 / 164 / 164
//                32 of up to 2000             59 /  82 /  94 / 105 / 140 / 152   54 /  90 /  91 /  91 / 127 / 127
//                one of 32768                 39 /  53 /  57 /  64 /  83 /  94   37 /  58 /  57 /  58 /  77 /  77
//   4-bit codes, 8 of up to 16001             70 /  98 / 112 / 126 / 170 / 186   67 / 118 / 119 / 118 / 168 / 168
//                32 of up to 2000             53 /  74 /  85 /  95 / 127 / 137   53 /  89 /  90 /  90 / 125 / 125
//                one of 32768                 35 /  47 /  50 /  56 /  73 /  82   37 /  57 /  57 /  57 /  77 /  77
// so 8-bit codes take fours when at most one is lacking (three tiles: 64 against 67), and
// 4-bit codes full ones, from eight tiles on.  (Two at a time, one warp to a ring:
// between the two.)
int group_tiles(const hyq_config* c, int32_t n_q, bool blocks) {
  const int gq = c->num_q_heads / c->num_kv_heads, tiles = (n_q * gq + kRowsQ - 1) / kRowsQ;
  const int lack = (kMaxNQ - tiles % kMaxNQ) % kMaxNQ;
  const bool wide = hyq_bits_k(c) + hyq_bits_v(c) > 8;
  return !blocks && (wide ? lack <= 1 && tiles >= kMaxNQ : lack == 0 && tiles > kMaxNQ) ? kMaxNQ : 1;
}

template <int BK, int BV, int NQ, int kLeave>
cudaError_t launch(const Params& p, cudaStream_t s) {
  using R = Ring<BK, BV, NQ>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = hyq_once_per_device(done, [] {
    return cudaFuncSetAttribute(paged_kernel<BK, BV, NQ, kLeave>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                R::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  const int grid = R::kPerSm * hyq_num_sms();
  return hyq_launch_chained(paged_kernel<BK, BV, NQ, kLeave>, dim3(grid), R::kBlockThreads, R::kSmemBytes, s, p);
}

template <int BK, int BV>
cudaError_t launch_nq(const Params& p, int nq, cudaStream_t s) {
  if (p.rest) return nq == kMaxNQ ? launch<BK, BV, kMaxNQ, kRest>(p, s) : launch<BK, BV, 1, kRest>(p, s);
  if (p.lse) return nq == kMaxNQ ? launch<BK, BV, kMaxNQ, kOutLse>(p, s) : launch<BK, BV, 1, kOutLse>(p, s);
  return nq == kMaxNQ ? launch<BK, BV, kMaxNQ, kOut>(p, s) : launch<BK, BV, 1, kOut>(p, s);
}

// Partials of the largest grid: two slots of kMaxNQ query tiles on each SM
// (one tile a block takes two blocks an SM, which is less).
size_t part_bytes() { return hyq_align256((size_t)hyq_num_sms() * 2 * kMaxNQ * kRowsQ * kPart * 4); }

}  // namespace

// The partials first, at a size that only the device sets, then a ticket per
// group: calls of other shapes may share the workspace, since no call's
// partials lie where another's tickets are.
size_t hyq_paged_attention_ws_bytes(const hyq_config* c, int32_t batch, int32_t n_q) {
  const size_t groups = (size_t)batch * c->num_kv_heads * n_q;  // at most a group a token
  return part_bytes() + hyq_align256(groups * 4);
}

cudaError_t hyq_launch_paged_attention(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                       int32_t n_q, const void* q, int64_t ldq, const int32_t* sel, int32_t k_sel,
                                       void* out, float* lse, const SharedRows* shared, float* rest, void* ws,
                                       cudaStream_t s) {
  const int nq = group_tiles(c, n_q, sel != nullptr);
  Params p;
  p.pv = pv;
  p.seqs = seqs;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.sel = sel;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.part = static_cast<float*>(ws);
  p.tickets = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + part_bytes());
  p.batch = batch;
  p.n_q = n_q;
  p.HQ = c->num_q_heads;
  p.HKV = c->num_kv_heads;
  p.gq = c->num_q_heads / c->num_kv_heads;
  p.QT = sel ? n_q : (n_q * p.gq + nq * kRowsQ - 1) / (nq * kRowsQ);
  p.k_sel = k_sel;
  p.lse = lse;
  p.shared = shared ? *shared : SharedRows{};
  p.rest = rest;
  const int bk = hyq_bits_k(c), bv = hyq_bits_v(c);
  if (bk == 4) return bv == 4 ? launch_nq<4, 4>(p, nq, s) : launch_nq<4, 8>(p, nq, s);
  return bv == 4 ? launch_nq<8, 4>(p, nq, s) : launch_nq<8, 8>(p, nq, s);
}
