// Attention over the paged cache (hyq_paged_attention and its block-sparse
// form hyq_paged_attention_blocks).
//
// For each query token i of a sequence and query head h of a KV head,
//   out = sum_j 2^(x_j - M) v_j / sum_j 2^(x_j - M),  x_j = log2(e) q.k_j / sqrt(128),
// over the positions j that the token sees, k_j and v_j = c s + z from the
// pages: one pass with the running maximum and sum of a softmax (q_tile in
// hyq_qtile.cuh: codes as fp16 subnormals on mma.sync, scales and zeros
// applied outside).
//
// What bounds it: the cache is read once, 160 bytes per (position, KV head)
// for 4-bit codes, against 4 * 128 * g flops: HBM, then instruction issue.
//
// Work split: a group is one (sequence, KV head, tile of up to 8 query rows)
// and has ceil(len / 16) tiles of 16 rows.  The T tiles of all groups, laid
// end to end, are cut into equal runs, one per block (two blocks an SM), so
// that unlike lengths and single long sequences use the GPU alike and the
// launch does not depend on the lengths (they live on the device; a captured
// call stays valid as they grow).  A group inside one run is finished by its
// block; one that several runs share is joined from their partials
// (maximum, sum, accumulator) in run order by the last block to finish, an
// atomic ticket that nobody waits for.
#include "hyq_paged.cuh"
#include "hyq_qtile.cuh"

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRowsQ = HYQ_MAX_GQA;    // query rows per tile (MMA N)
constexpr int kPart = 2 + HYQ_D;       // m, l, acc[128] per query row
constexpr int kMinTiles = kWarps;      // tiles per block before work is split further
constexpr int kBlocksPerSm = 2;
constexpr int kMaxGrid = 1024;         // two blocks on each of up to 512 SMs

// Per-warp ring of tiles (bulk copies), as many as two blocks an SM allow.
template <int BK, int BV>
struct Ring : QFmt<BK, BV> {
  static constexpr int kSlots = BK + BV == 8 ? 4 : BK + BV == 12 ? 3 : 2;
  static constexpr int kWarpBytes = kSlots * QFmt<BK, BV>::kTile;
  static constexpr int kSmemBytes = kWarps * kWarpBytes;
  static_assert(kWarpBytes >= HYQ_MAX_GQA * HYQ_D * 4, "a warp's partial fits its ring");
};

struct Params {
  PageView pv;
  const int32_t* seqs;
  const __nv_bfloat16* q;
  int64_t ldq;
  const int32_t* sel;  // [batch][n_q][HKV][k_sel] or nullptr
  __nv_bfloat16* out;
  float* part;         // [grid][2][8][kPart]
  int32_t* tickets;    // [groups]
  int32_t batch, n_q, HQ, HKV, gq, QT, k_sel;
};

// Length of call row b (0 for a sequence out of range) and its tiles per group.
__device__ __forceinline__ int row_len(const Params& p, int b, int* seq) {
  const int s = page_seq(p.seqs, b, p.pv.n_seqs);
  *seq = s;
  if (s < 0) return 0;
  const int64_t cap = (int64_t)p.pv.max_blocks * HYQ_PAGE_ROWS;
  const int n = p.pv.lens[s];
  return n < 0 ? 0 : (int64_t)n > cap ? (int)cap : n;
}
__device__ __forceinline__ int row_tiles(const Params& p, int len) {
  if (!p.sel) return (len + 15) >> 4;
  return 4 * min(p.k_sel, (len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS);
}

template <int BK, int BV>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) paged_kernel(const Params p) {
  using R = Ring<BK, BV>;
  constexpr int kSlots = R::kSlots, kTile = R::kTile;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_cum[HYQ_PAGED_MAX_BATCH + 1];  // tiles per (KV head, query tile) of the rows before b
  __shared__ int64_t s_warp[kWarps];
  __shared__ __align__(16) uint32_t bq_s[4][kRowsQ][4][4];
  __shared__ float rowc_s[kRowsQ][4];
  __shared__ uint32_t bz_s[kRowsQ][4];
  __shared__ int lim_s[kRowsQ];
  __shared__ __align__(8) uint64_t bars[kWarps * kSlots];
  __shared__ float red_m[kWarps][kRowsQ], red_l[kWarps][kRowsQ];
  __shared__ float s_sum[kRowsQ];
  __shared__ int s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * R::kWarpBytes;
  uint64_t* wb = bars + warp * kSlots;
  if (lane < kSlots) mbar_init(&wb[lane], 1);
  mbar_fence_init();

  // ---- the rows' tiles, summed up: a block of 4 rows per thread -------------
  const int unit = p.HKV * p.QT;
  {
    int64_t w[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 4 * tid + i;
      int seq;
      const int len = b < p.batch ? row_len(p, b, &seq) : 0;
      if (b < p.batch && seq < 0 && blockIdx.x == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
      w[i] = row_tiles(p, len);
      sum += w[i];
      // a row without positions: its outputs are zero
      if (b < p.batch && w[i] == 0 && b % gridDim.x == blockIdx.x) {
        uint4* o = reinterpret_cast<uint4*>(p.out + (size_t)b * p.n_q * p.HQ * HYQ_D);
        for (int k = 0; k < p.n_q * p.HQ * (HYQ_D / 8); ++k) o[k] = make_uint4(0, 0, 0, 0);
      }
    }
    int64_t pre = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    if (lane == 31) s_warp[warp] = pre;
    __syncthreads();
    int64_t at = pre - sum;
    for (int i = 0; i < warp; ++i) at += s_warp[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * tid + i <= p.batch) s_cum[4 * tid + i] = at;
      at += w[i];
    }
    if (tid == kThreads - 1 && p.batch == HYQ_PAGED_MAX_BATCH) s_cum[HYQ_PAGED_MAX_BATCH] = at;
  }
  __syncthreads();
  const int64_t T = s_cum[p.batch] * unit;
  const int64_t nb = min((int64_t)gridDim.x, max((int64_t)1, T / kMinTiles));  // blocks that take part
  if ((int64_t)blockIdx.x >= nb) return;
  int64_t pos = T * blockIdx.x / nb;
  const int64_t end = T * (blockIdx.x + 1) / nb;

  // Lane i < kSlots fills slot i of the warp's ring (copies that one thread
  // issues complete one after another).  cur: position of its slot's tile,
  // whether it was copied, and the parity to wait for.
  uint32_t parity = 0, cur = 0;
  bool dead = false;

  while (pos < end) {
    // ---- the group at pos -----------------------------------------------
    int lo = 0, hi = p.batch;  // the last b with unit * s_cum[b] <= pos
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (s_cum[m] * unit <= pos) lo = m;
      else hi = m;
    }
    const int b = lo;
    const int W = (int)(s_cum[b + 1] - s_cum[b]);
    const int64_t off = pos - s_cum[b] * unit;
    const int grp = (int)(off / W), w0 = (int)(off - (int64_t)grp * W);
    const int w1 = (int)min((int64_t)W, w0 + (end - pos));
    const int h = grp / p.QT, qt = grp - h * p.QT;
    int seq;
    const int len = row_len(p, b, &seq);
    const int32_t* table = p.pv.table + (size_t)seq * p.pv.max_blocks;
    const int32_t* sel = p.sel ? p.sel + (((size_t)b * p.n_q + qt) * p.HKV + h) * p.k_sel : nullptr;
    const int n_rows = p.sel ? p.gq : min(kRowsQ, p.n_q * p.gq - kRowsQ * qt);
    const uint8_t* heads = p.pv.pool + (size_t)h * R::kBlock;  // this head's block of page 0
    const size_t page_bytes = (size_t)p.HKV * R::kBlock;

    // ---- this warp's tiles: w0 + warp, + 8, ... ---------------------------
    const int nj = w1 - w0 > warp ? (w1 - w0 - warp + kWarps - 1) / kWarps : 0;
    // Entry of the block list that tile j lies in (dense: the block itself);
    // -1 for one that must not be read.
    auto entry = [&](int j) -> int {
      if (j >= nj) return -1;
      const int x = (w0 + warp + kWarps * j) >> 2;
      if (!sel) return x;
      const int e = __ldg(sel + x), pe = x > 0 ? __ldg(sel + x - 1) : -1;
      if (e < 0) return -1;
      if ((x > 0 && pe < 0) || pe >= e || (int64_t)e * HYQ_PAGE_ROWS >= len) {
        hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        return -1;
      }
      return e;
    };
    auto page_of = [&](int e) -> int { return e >= 0 ? __ldg(table + e) : -1; };
    // Lane pipeline: page of its next tile, list entry of the one after.
    int e1 = -1, e2 = -1, pg1 = -1;
    auto issue = [&](int j) {  // lane j % kSlots
      const int x = (w0 + warp + kWarps * j) & 3;
      const int at = e1 * HYQ_PAGE_ROWS + 16 * x;
      bool ok = e1 >= 0 && at < len;
      if (ok && (pg1 < 0 || pg1 >= p.pv.n_pages)) {
        hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        ok = false;
      }
      if (ok) {
        uint64_t* bar = &wb[j % kSlots];
        mbar_arrive_expect_tx(bar, kTile);
        bulk_g2s(ring + (j % kSlots) * kTile, heads + (size_t)pg1 * page_bytes + x * kTile, kTile, bar);
        cur = ((uint32_t)at << 2) | 2u | parity;
        parity ^= 1u;
      } else {
        cur = 0;
      }
      e1 = e2;
      pg1 = page_of(e1);
      e2 = entry(j + 2 * kSlots);
    };
    if (lane < kSlots && !dead) {
      e1 = entry(lane);
      pg1 = page_of(e1);
      e2 = entry(lane + kSlots);
      if (lane < nj) issue(lane);
    }

    // ---- the query rows: warp r prepares row r ----------------------------
    {
      const int r = warp;
      const int flat = kRowsQ * qt + r;
      const int tok = p.sel ? qt : flat / p.gq, head = p.sel ? r : flat - tok * p.gq;
      uint2 v = make_uint2(0, 0);
      if (r < n_rows)
        v = __ldg(reinterpret_cast<const uint2*>(p.q + ((size_t)b * p.n_q + tok) * p.ldq +
                                                 (size_t)(h * p.gq + head) * HYQ_D + 4 * lane));
      prep_query_row<BK>(r, lane, v, bq_s, rowc_s, bz_s);
      if (lane == 0) lim_s[r] = r < n_rows ? max(0, len - p.n_q + 1 + tok) : len;
    }
    __syncthreads();
    uint32_t bq[8][2];
    QConst qc;
    load_query_consts(g, t, bq_s, rowc_s, bz_s, bq, qc);
    const int lim0 = lim_s[2 * t], lim1 = lim_s[2 * t + 1];
    const int minlim = lim_s[0];  // the rows' tokens ascend
    State st;
    reset_state(st);

    for (int j = 0; j < nj && !dead; ++j) {
      const int slot = j % kSlots;
      const uint32_t c = __shfl_sync(0xffffffffu, cur, slot);
      if (c & 2u) {
        const bool ok = mbar_wait(&wb[slot], c & 1u);
        if (__any_sync(0xffffffffu, !ok)) {
          // A copy did not arrive: flag it, let this warp's other copies land
          // before shared memory is used for anything else, and stop.
          if (lane == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_TIMEOUT);
          if (lane < kSlots && (cur & 2u)) (void)mbar_wait(&wb[lane], cur & 1u);
          __syncwarp();
          dead = true;
          break;
        }
        const int at = (int)(c >> 2);
        const uint8_t* tb = ring + slot * kTile;
        if (at + 16 <= minlim)
          q_tile<BK, BV, true>(tb, lane, 16, bq, qc, st);
        else
          q_tile<BK, BV, true, true>(tb, lane, len - at, bq, qc, st, lim0 - at, lim1 - at);
        __syncwarp();
      }
      if (lane == slot) {
        if (j + kSlots < nj) {
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          issue(j + kSlots);
        } else {
          cur = 0;
        }
      }
    }

    // ---- the block's partial ------------------------------------------------
    __syncwarp();
    store_warp_partial<BV>(st, qc, g, t, reinterpret_cast<float*>(ring), red_m[warp], red_l[warp]);
    __syncthreads();
    const bool whole = w0 == 0 && w1 == W;
    float* pp = p.part + ((size_t)blockIdx.x * 2 + (w0 == 0 ? 1 : 0)) * (kRowsQ * kPart);
    auto out_at = [&](int r) {
      const int flat = kRowsQ * qt + r;
      const int tok = p.sel ? qt : flat / p.gq, head = p.sel ? r : flat - tok * p.gq;
      return p.out + (((size_t)b * p.n_q + tok) * p.HQ + (size_t)h * p.gq + head) * HYQ_D;
    };
    for (int i = tid; i < n_rows * HYQ_D; i += kThreads) {
      const int r = i >> 7, d = i & (HYQ_D - 1);
      const float mw = lane < kWarps ? red_m[lane][r] : -INFINITY;
      float M = mw;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      M = __shfl_sync(0xffffffffu, M, 0);
      const float wt = mw == -INFINITY ? 0.f : ex2(mw - M);
      float L = lane < kWarps ? red_l[lane][r] * wt : 0.f;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      L = __shfl_sync(0xffffffffu, L, 0);
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        a = fmaf(__shfl_sync(0xffffffffu, wt, w),
                 reinterpret_cast<const float*>(smem + w * R::kWarpBytes)[r * HYQ_D + (d ^ (r >> 1))], a);
      if (whole) {
        out_at(r)[d] = __float2bfloat16_rn(L > 0.f ? a / L : 0.f);
      } else {
        pp[r * kPart + 2 + d] = a;
        if (d == 0) {
          pp[r * kPart + 0] = M;
          pp[r * kPart + 1] = L;
        }
      }
    }
    __syncthreads();  // the rings are free again
    if (!whole) {
      // blocks that share this group: those holding its first and last tile
      const int64_t base = s_cum[b] * unit + (int64_t)grp * W;
      const int c0 = (int)(((base + 1) * nb - 1) / T), c1 = (int)(((base + W) * nb - 1) / T);
      const size_t gi = ((size_t)b * p.HKV + h) * p.QT + qt;
      if (tid == 0) {
        int old;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(old) : "l"(p.tickets + gi) : "memory");
        s_last = old == c1 - c0;
        if (s_last) p.tickets[gi] = 0;
      }
      __syncthreads();
      if (s_last) {
        // part of block c: slot 1 when its run begins the group (c == c0 and
        // the run starts at or before it), else slot 0
        float* wts = reinterpret_cast<float*>(smem);  // [8][n] weights
        const int n = c1 - c0 + 1;
        auto part_of = [&](int c) {
          const bool first = T * c / nb <= base;
          return p.part + ((size_t)c * 2 + (first ? 1 : 0)) * (kRowsQ * kPart);
        };
        if (warp < n_rows) {
          float M = -INFINITY;
          for (int c = lane; c < n; c += 32) M = fmaxf(M, __ldcg(part_of(c0 + c) + warp * kPart));
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
          float L = 0.f;
          for (int c = lane; c < n; c += 32) {
            const float* e = part_of(c0 + c) + warp * kPart;
            const float m = __ldcg(e), wt = m == -INFINITY ? 0.f : ex2(m - M);
            wts[warp * n + c] = wt;
            L = fmaf(__ldcg(e + 1), wt, L);
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
          if (lane == 0) s_sum[warp] = L;
        }
        __syncthreads();
        for (int i = tid; i < n_rows * HYQ_D; i += kThreads) {
          const int r = i >> 7, d = i & (HYQ_D - 1);
          float a = 0.f;
#pragma unroll 8
          for (int c = 0; c < n; ++c) a = fmaf(__ldcg(part_of(c0 + c) + r * kPart + 2 + d), wts[r * n + c], a);
          const float L = s_sum[r];
          out_at(r)[d] = __float2bfloat16_rn(L > 0.f ? a / L : 0.f);
        }
        __syncthreads();
      }
    }
    // order this block's generic accesses to the rings before the next copies
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    pos += w1 - w0;
  }
}

int paged_grid() { return min(kBlocksPerSm * hyq_num_sms(), kMaxGrid); }

int query_tiles(const hyq_config* c, int32_t n_q, bool blocks) {
  const int gq = c->num_q_heads / c->num_kv_heads;
  return blocks ? n_q : (n_q * gq + kRowsQ - 1) / kRowsQ;
}

template <int BK, int BV>
cudaError_t launch(const Params& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = hyq_once_per_device(done, [] {
    return cudaFuncSetAttribute(paged_kernel<BK, BV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Ring<BK, BV>::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  paged_kernel<BK, BV><<<paged_grid(), kThreads, Ring<BK, BV>::kSmemBytes, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// The partials first, at a size that only the device sets, then a ticket per
// group: calls of other shapes may share the workspace, since no call's
// partials lie where another's tickets are.
size_t hyq_paged_attention_ws_bytes(const hyq_config* c, int32_t batch, int32_t n_q) {
  const size_t groups = (size_t)batch * c->num_kv_heads * n_q;  // n_q >= the dense query tiles
  return hyq_align256((size_t)paged_grid() * 2 * kRowsQ * kPart * 4) + hyq_align256(groups * 4);
}

cudaError_t hyq_launch_paged_attention(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                       int32_t n_q, const void* q, int64_t ldq, const int32_t* sel, int32_t k_sel,
                                       void* out, void* ws, cudaStream_t s) {
  Params p;
  p.pv = pv;
  p.seqs = seqs;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.sel = sel;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.part = static_cast<float*>(ws);
  p.tickets = reinterpret_cast<int32_t*>(static_cast<char*>(ws) +
                                         hyq_align256((size_t)paged_grid() * 2 * kRowsQ * kPart * 4));
  p.batch = batch;
  p.n_q = n_q;
  p.HQ = c->num_q_heads;
  p.HKV = c->num_kv_heads;
  p.gq = c->num_q_heads / c->num_kv_heads;
  p.QT = query_tiles(c, n_q, sel != nullptr);
  p.k_sel = k_sel;
  const int bk = hyq_bits_k(c), bv = hyq_bits_v(c);
  if (bk == 4) return bv == 4 ? launch<4, 4>(p, s) : launch<4, 8>(p, s);
  return bv == 4 ? launch<8, 4>(p, s) : launch<8, 8>(p, s);
}
