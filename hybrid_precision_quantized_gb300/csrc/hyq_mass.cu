// Accumulated attention weights of the paged cache (hyq_paged_accumulate): per KV
// head and position j
//   mass_j += sum over the query rows that see j of 2^(x_j - log2(e) lse),
//   x_j = log2(e) q.k_j / sqrt(128),
// with the logarithms lse of the rows' softmax sums given: one pass over the keys alone
// (their codes as fp16 subnormals on mma.sync, steps and zeros applied in
// float32, as in hyq_qtile.cuh).
//
// What bounds it: the keys are read once, 80 bytes per (position, KV head) for
// 4-bit codes, and 8 bytes of mass read and written: HBM for a few query rows (64 sequences of
// up to 32768, one token each: 178 us, 0.75 of the copy rate); instruction issue and latency (a
// product, an exponential and a sum per query row and position) for many (64 tokens of eight
// sequences of up to 8192: 119 us, 0.09 of the product rate).
//
// A group is one (sequence, KV head).  Its units (two 16-row tiles; with more than one tile
// of query rows a single one) go round the block's warps, each with a ring of asynchronous
// copies of its own, and a warp takes a unit against all query rows: a position's sum has one
// writer and one order, so there is nothing to join and results do not vary from run to run.
// The codes are unpacked once a unit and
// the query rows' operands read once for both tiles.  The pages of all groups, laid end to end,
// are cut into equal runs, a block each.
#include "hyq_paged.cuh"
#include "hyq_qtile.cuh"

namespace {

constexpr int kMaxWarps = 16;
constexpr int kCost = 4;   // pages that a group's fixed work is worth

struct Params {
  PageView pv;
  const int32_t* refs;
  const int32_t* seqs;
  const __nv_bfloat16* q;
  int64_t ldq;
  const float* lse;      // [batch][n_q][HQ]
  const int32_t* n_new;  // [batch] or nullptr
  float* mass;           // [n_pages][HKV][64]
  int32_t batch, n_q, HQ, HKV, gq, QT;
};

// A tile of eight query rows in shared memory.
struct __align__(16) Query {
  uint32_t bq[4][HYQ_MAX_GQA][4][4];
  float rowc[HYQ_MAX_GQA][4];
  uint32_t bz[HYQ_MAX_GQA][4];
  float nl[HYQ_MAX_GQA];  // -log2(e) lse; minus infinity for a row that gives nothing
  int lim[HYQ_MAX_GQA];  // positions that the row sees
};

template <int BK, int BV, int kTiles>
struct Unit {
  using F = QFmt<BK, BV>;
  static constexpr int kCodes = 256 * BK, kTile = kCodes + 256, kBytes = kTiles * kTile;  // of the keys alone
  static constexpr int kRows = 16 * kTiles, kPerPage = HYQ_PAGE_ROWS / kRows;
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(kLeft) : "memory");
}

// kSlots: units of a warp's ring.  (Bulk copies, of 1024 and 256 bytes here, were slower than a lane's 16 bytes each: 521
// against 318 us for 64 sequences of up to 32768, at that step.)
// kOne: one tile of query rows, whose operands stay in registers; more of them are read again for every unit, whose
// codes are then unpacked once for all.
template <int BK, int BV, int kSlots, bool kOne>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) mass_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  constexpr int kT = kOne ? 2 : 1;
  using U = Unit<BK, BV, kT>;
  constexpr int kRows = U::kRows, kPer = U::kPerPage;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_cum[HYQ_PAGED_MAX_BATCH + 1], s_warp[kMaxWarps];
  __shared__ __align__(16) int s_seq[HYQ_PAGED_MAX_BATCH];
  __shared__ int s_len[HYQ_PAGED_MAX_BATCH];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int n_threads = blockDim.x, n_warps = n_threads >> 5;
  uint8_t* ring = smem + warp * kSlots * U::kBytes;
  Query* query = reinterpret_cast<Query*>(smem + n_warps * kSlots * U::kBytes);  // [QT]
  chain_kernel();
  for (int b = tid; b < p.batch; b += n_threads) s_seq[b] = page_seq(p.seqs, b, p.pv.n_seqs);
  __syncthreads();
  {
    int64_t before = 0;
    for (int row0 = 0; row0 < p.batch; row0 += n_threads) {
      const int b = row0 + tid;
      int64_t w = 0;
      if (b < p.batch) {
        const int s = s_seq[b];
        bool bad = s < 0;
        for (int j = 0; p.seqs && j < b; ++j) bad |= s_seq[j] == s;  // listed before
        int64_t len = bad ? 0 : p.pv.lens[s];
        len = max((int64_t)0, min(len, (int64_t)p.pv.max_blocks * HYQ_PAGE_ROWS));
        if (bad && blockIdx.x == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        s_len[b] = (int)len;
        if (len) w = (len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS + kCost;
      }
      int64_t pre = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
      }
      __syncthreads();
      if (lane == 31) s_warp[warp] = pre;
      __syncthreads();
      int64_t at = before + pre - w;
      for (int i = 0; i < n_warps; ++i) {
        if (i < warp) at += s_warp[i];
        before += s_warp[i];
      }
      if (b < p.batch) s_cum[b] = at;
    }
    if (tid == 0) s_cum[p.batch] = before;
  }
  __syncthreads();
  const int64_t total = s_cum[p.batch] * p.HKV;
  int64_t pos = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  while (pos < end) {
    int lo = 0, hi = p.batch;  // the last b with HKV s_cum[b] <= pos
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (s_cum[m] * p.HKV <= pos) lo = m;
      else hi = m;
    }
    const int W = (int)(s_cum[lo + 1] - s_cum[lo]);
    const int64_t off = pos - s_cum[lo] * p.HKV;
    const int h = (int)(off / W), x0 = (int)(off - (int64_t)h * W), x1 = (int)min((int64_t)W, x0 + (end - pos));
    pos += x1 - x0;
    if (x1 <= kCost) continue;
    const int len = s_len[lo], fresh = len - (p.n_new ? p.n_new[lo] : p.n_q);
    const int32_t* table = p.pv.table + (size_t)s_seq[lo] * p.pv.max_blocks;
    // ---- this warp's units of kRows positions: u0, u0 + n_warps, ..; their pages 32 ahead --------
    const int u0 = kPer * max(0, x0 - kCost) + warp, u1 = min(kPer * (x1 - kCost), (len + kRows - 1) / kRows);
    const int nj = u1 > u0 ? (u1 - u0 + n_warps - 1) / n_warps : 0;
    auto page_of = [&](int j) -> int {  // of unit j, or -1 for one that is left out
      if (j >= nj) return -1;
      const int pg = table[(u0 + j * n_warps) / kPer];
      if ((uint32_t)pg >= (uint32_t)p.pv.n_pages) {
        hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        return -1;
      }
      if (p.refs[pg] > 1) {  // several sequences' positions
        hyq_set_err(p.pv.err, HYQ_DEVERR_PAGES);
        return -1;
      }
      return pg;
    };
    int pg_cur = page_of(lane), pg_nxt = page_of(32 + lane), round = 0;  // of units 32 round + lane, and 32 on
    auto page = [&](int j) { return __shfl_sync(0xffffffffu, (j >> 5) == round ? pg_cur : pg_nxt, j & 31); };  // this round's or the next's
    auto issue = [&](int j) {  // (a group of copies whether there are any or not)
      const int pg = j < nj ? page(j) : -1;
      if (pg >= 0) {
        const uint8_t* from = p.pv.pool + ((size_t)pg * p.HKV + h) * F::kBlock + kT * ((u0 + j * n_warps) % kPer) * F::kTile;
        const uint32_t to = smem_u32(ring) + (j % kSlots) * U::kBytes;
#pragma unroll
        for (int i = 0; i < (U::kBytes + 511) / 512; ++i) {
          const int x = 16 * lane + 512 * i, tile = x / U::kTile, at = x - tile * U::kTile;
          if (U::kBytes % 512 == 0 || x < U::kBytes) copy16(to + x, from + tile * F::kTile + (at < U::kCodes ? at : F::kKMeta + at - U::kCodes));
        }
      }
      copies_end();
    };
    auto weights = [&](int j, int pg) { return p.mass + ((size_t)pg * p.HKV + h) * HYQ_PAGE_ROWS + kRows * ((u0 + j * n_warps) % kPer); };
    auto held = [&](int j, int pg) {  // what this lane's position of unit j has so far
      return j < nj && pg >= 0 && lane < kRows && kRows * (u0 + j * n_warps) + lane < fresh ? weights(j, pg)[lane] : 0.f;
    };
#pragma unroll 1
    for (int j = 0; j < kSlots; ++j) issue(j);
    int pg = page(0);
    float old = held(0, pg);
    // ---- the query rows, a warp each ------------------------------------------------
    __syncthreads();
#pragma unroll 1
    for (int r0 = warp; r0 < p.QT * HYQ_MAX_GQA; r0 += 4 * n_warps) {
      uint2 v[4];
      float lse[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // four rows under way
        const int r = r0 + k * n_warps, tok = r / p.gq, head = h * p.gq + r - tok * p.gq;
        v[k] = make_uint2(0, 0), lse[k] = 0.f;
        if (tok < p.n_q) {
          v[k] = *reinterpret_cast<const uint2*>(p.q + ((size_t)lo * p.n_q + tok) * p.ldq + (size_t)head * HYQ_D + 4 * lane);
          lse[k] = p.lse[((size_t)lo * p.n_q + tok) * p.HQ + head];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + k * n_warps, tok = r / p.gq;
        if (r >= p.QT * HYQ_MAX_GQA) break;
        const int lim = tok < p.n_q ? max(0, len - p.n_q + 1 + tok) : 0;
        const uint32_t e = 0x7F807F80u, a = v[k].x & e, b = v[k].y & e;
        bool bad = (a >> 16) == 0x7F80u || (a & 0xFFFFu) == 0x7F80u || (b >> 16) == 0x7F80u || (b & 0xFFFFu) == 0x7F80u;
        bad |= !(fabsf(lse[k]) <= 3.402823466e38f);
        bad = __any_sync(0xffffffffu, bad);
        if (bad && lim > 0 && lane == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_SCORE);
        Query& qt = query[r / HYQ_MAX_GQA];
        prep_query_row<BK>(r & 7, lane, bad ? make_uint2(0, 0) : v[k], qt.bq, qt.rowc, qt.bz);
        if (lane == 0) qt.nl[r & 7] = bad || lim == 0 ? -INFINITY : lse[k] * -1.4426950408889634f, qt.lim[r & 7] = lim;
      }
    }
    __syncthreads();
    uint32_t bq1[8][2];
    QConst qc1;
    load_query_consts(g, t, query[0].bq, query[0].rowc, query[0].bz, bq1, qc1);
    const float nl1[2] = {query[0].nl[2 * t], query[0].nl[2 * t + 1]};
    const int minlim = len - p.n_q + 1;
    // ---- the units --------------------------------------------------------------------------
    for (int j = 0; j < nj; ++j) {
      const int at = kRows * (u0 + j * n_warps), pg_next = page(j + 1);
      copies_wait<kSlots - 1>();
      __syncwarp();
      const float next = held(j + 1, pg_next);
      float sums[2 * kT];  // of rows g, g + 8 of the tiles
#pragma unroll
      for (int i = 0; i < 2 * kT; ++i) sums[i] = 0.f;
      if (pg >= 0) {
        const bool all = at + kRows <= minlim;  // every row sees every position
        uint4 ma[kT], mb[kT];                   // steps and zeros of rows g, g + 8
        uint32_t kw[kT][BK == 4 ? 8 : 16];
#pragma unroll
        for (int i = 0; i < kT; ++i) {
          const uint8_t* tb = ring + (j % kSlots) * U::kBytes + i * U::kTile;
          load_words<BK == 4 ? 8 : 16>(tb, lane, kw[i]);
          ma[i] = *reinterpret_cast<const uint4*>(tb + U::kCodes + 16 * g);
          mb[i] = *reinterpret_cast<const uint4*>(tb + U::kCodes + 16 * (g + 8));
        }
        __syncwarp();
        issue(j + kSlots);  // the slot is free: everything is in registers
        // a tile's codes as fp16 subnormals, fragment of step ks
        auto fragment = [&](int i, int ks, uint32_t (&a)[4]) {
          if (BK == 4) {
            const uint32_t w = kw[i][ks], w8 = w >> 8;
            a[0] = w & 0x000F000Fu, a[1] = w & 0x00F000F0u, a[2] = w8 & 0x000F000Fu, a[3] = w8 & 0x00F000F0u;
          } else {
            const uint32_t wa = kw[i][BK == 4 ? 0 : 2 * ks], wb = kw[i][BK == 4 ? 0 : 2 * ks + 1];
            a[0] = wa & 0x00FF00FFu, a[1] = wb & 0x00FF00FFu, a[2] = odd_bytes(wa), a[3] = odd_bytes(wb);
          }
        };
        // what eight query rows give to a tile's positions
        auto give = [&](int i, auto step, const uint32_t (&bq)[8][2], const QConst& qc, float nl0, float nl1, const int* lim) {
          float C[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) C[q][0] = C[q][1] = C[q][2] = C[q][3] = 0.f;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) step(C[ks >> 1], ks, bq[ks][0], bq[ks][1]);
          const float2 a01 = half2_to_float2(ma[i].x), a23 = half2_to_float2(ma[i].y);
          const float2 b01 = half2_to_float2(mb[i].x), b23 = half2_to_float2(mb[i].y);
          float lg[4];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            lg[c] = qc.ksc[0][c] * fmaf(a01.x, C[0][c], fmaf(a01.y, C[1][c], fmaf(a23.x, C[2][c], a23.y * C[3][c])));
            lg[2 + c] = qc.ksc[1][c] * fmaf(b01.x, C[0][2 + c], fmaf(b01.y, C[1][2 + c], fmaf(b23.x, C[2][2 + c], b23.y * C[3][2 + c])));
          }
          mma_f16(lg, (t & 1) ? ma[i].w : ma[i].z, (t & 1) ? mb[i].w : mb[i].z, 0u, 0u, qc.bz, 0u);
          lg[0] = ex2(fmaf(lg[0], qc.inv[0], nl0)), lg[1] = ex2(fmaf(lg[1], qc.inv[1], nl1));
          lg[2] = ex2(fmaf(lg[2], qc.inv[0], nl0)), lg[3] = ex2(fmaf(lg[3], qc.inv[1], nl1));
          if (!all) {
            const int p0 = at + 16 * i + g, p1 = p0 + 8, l0 = lim[2 * t], l1 = lim[2 * t + 1];
            if (p0 >= l0) lg[0] = 0.f;
            if (p0 >= l1) lg[1] = 0.f;
            if (p1 >= l0) lg[2] = 0.f;
            if (p1 >= l1) lg[3] = 0.f;
          }
          sums[2 * i] += lg[0] + lg[1];
          sums[2 * i + 1] += lg[2] + lg[3];
        };
        if (kOne) {
#pragma unroll
          for (int i = 0; i < kT; ++i)
            give(i, [&](float (&C)[4], int ks, uint32_t b0, uint32_t b1) {
              uint32_t a[4];
              fragment(i, ks, a);
              mma_f16(C, a[0], a[1], a[2], a[3], b0, b1);
            }, bq1, qc1, nl1[0], nl1[1], query[0].lim);
        } else {
          uint32_t a[kT][8][4];
#pragma unroll
          for (int i = 0; i < kT; ++i)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) fragment(i, ks, a[i][ks]);
#pragma unroll 1
          for (int k = 0; k < p.QT; ++k) {
            uint32_t bq[8][2];
            QConst qc;
            load_query_consts(g, t, query[k].bq, query[k].rowc, query[k].bz, bq, qc);
            const float2 nl = *reinterpret_cast<const float2*>(&query[k].nl[2 * t]);
#pragma unroll
            for (int i = 0; i < kT; ++i)
              give(i, [&](float (&C)[4], int ks, uint32_t b0, uint32_t b1) {
                mma_f16(C, a[i][ks][0], a[i][ks][1], a[i][ks][2], a[i][ks][3], b0, b1);
              }, bq, qc, nl.x, nl.y, query[k].lim);
          }
        }
#pragma unroll
        for (int i = 0; i < 2 * kT; ++i) {
          sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 1);
          sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 2);
        }
        // row r of the unit: sums[r / 8] of the lanes 4 (r % 8) ..
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kT; ++i) {
          const float x = __shfl_sync(0xffffffffu, sums[i], 4 * (lane & 7));
          if (lane >> 3 == i) add = x;
        }
        if (lane < kRows && at + lane < len) weights(j, pg)[lane] = old + add;
      } else {
        issue(j + kSlots);
      }
      old = next, pg = pg_next;
      if ((j & 31) == 31) {
        pg_cur = pg_nxt;
        ++round;
        pg_nxt = page_of(32 * (round + 1) + lane);
      }
    }
    copies_wait<0>();
    __syncwarp();
  }
}

// Reads are what bounds a single tile of query rows: a ring holds four units where there is room, else two.
template <int BK, int BV, bool kOne>
cudaError_t launch_one(const Params& p, cudaStream_t s) {
  constexpr int kSlots = kOne && BK == 4 ? 4 : 2, kRoom = 208 * 1024, kRing = kSlots * Unit<BK, BV, kOne ? 2 : 1>::kBytes;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = hyq_once_per_device(done, [] {
    return cudaFuncSetAttribute(mass_kernel<BK, BV, kSlots, kOne>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
  });
  if (e != cudaSuccess) return e;
  const int query = p.QT * (int)sizeof(Query), fit = (kRoom - query) / kRing, warps = fit < kMaxWarps ? fit : kMaxWarps;
  return hyq_launch_chained(mass_kernel<BK, BV, kSlots, kOne>, dim3(hyq_num_sms()), 32 * warps, (size_t)warps * kRing + query, s, p);
}
template <int BK, int BV>
cudaError_t launch(const Params& p, cudaStream_t s) {
  return p.QT == 1 ? launch_one<BK, BV, true>(p, s) : launch_one<BK, BV, false>(p, s);
}

}  // namespace

cudaError_t hyq_launch_paged_accumulate(const hyq_config* c, const PageView& pv, const int32_t* refs,
                                        const int32_t* seqs, int32_t batch, int32_t n_q, const void* q, int64_t ldq,
                                        const float* lse, const int32_t* n_new, float* mass, cudaStream_t s) {
  Params p;
  p.pv = pv;
  p.refs = refs;
  p.seqs = seqs;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.lse = lse;
  p.n_new = n_new;
  p.mass = mass;
  p.batch = batch;
  p.n_q = n_q;
  p.HQ = c->num_q_heads;
  p.HKV = c->num_kv_heads;
  p.gq = p.HQ / p.HKV;
  p.QT = (n_q * p.gq + HYQ_MAX_GQA - 1) / HYQ_MAX_GQA;
  const int bk = hyq_bits_k(c), bv = hyq_bits_v(c);
  if (bk == 4) return bv == 4 ? launch<4, 4>(p, s) : launch<4, 8>(p, s);
  return bv == 4 ? launch<8, 4>(p, s) : launch<8, 8>(p, s);
}
