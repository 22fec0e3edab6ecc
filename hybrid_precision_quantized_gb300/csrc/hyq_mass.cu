// Accumulated attention weights of the paged cache (hyq_paged_accumulate): per KV
// head and position j
//   mass_j += sum over the query rows that see j of 2^(x_j - log2(e) lse),
//   x_j = log2(e) q.k_j / sqrt(128),
// with the logarithms lse of the rows' softmax sums given: one pass over the keys alone
// (their codes as fp16 subnormals on mma.sync, steps and zeros applied in
// float32, as in hyq_qtile.cuh).
//
// What bounds it: the keys are read once, 80 bytes per (position, KV head) for
// 4-bit codes, and 8 bytes of mass read and written: HBM for a few query rows; instruction
// issue (a product, an exponential and a sum per query row and position) for many.
//
// A group is one (sequence, KV head).  Its pages are taken whole by one warp
// each, for all query rows: a position's sum has one writer and one order, so there is
// nothing to join and results do not vary from run to run.  The pages of all
// groups, laid end to end, are cut into equal runs, a block each.
#include "hyq_paged.cuh"
#include "hyq_qtile.cuh"

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCost = 4;  // pages that a group's fixed work is worth

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
struct Query {
  uint32_t bq[4][HYQ_MAX_GQA][4][4];
  float rowc[HYQ_MAX_GQA][4];
  uint32_t bz[HYQ_MAX_GQA][4];
  float lse[HYQ_MAX_GQA];
  int lim[HYQ_MAX_GQA];  // positions that the row sees
};

template <int BK, int BV>
__global__ void __launch_bounds__(kThreads, 2) mass_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  extern __shared__ __align__(16) uint8_t smem[];
  Query* query = reinterpret_cast<Query*>(smem);  // [QT]
  __shared__ int64_t s_cum[HYQ_PAGED_MAX_BATCH + 1], s_warp[kWarps];
  __shared__ __align__(16) int s_seq[HYQ_PAGED_MAX_BATCH];
  __shared__ int s_len[HYQ_PAGED_MAX_BATCH];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  chain_kernel();
  for (int b = tid; b < p.batch; b += kThreads) s_seq[b] = page_seq(p.seqs, b, p.pv.n_seqs);
  __syncthreads();
  {
    int64_t before = 0;
    for (int row0 = 0; row0 < p.batch; row0 += kThreads) {
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
      for (int i = 0; i < kWarps; ++i) {
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
    const int u0 = max(0, x0 - kCost), u1 = x1 - kCost;
    if (u1 <= 0) continue;
    const int len = s_len[lo], fresh = len - (p.n_new ? p.n_new[lo] : p.n_q);
    const int32_t* table = p.pv.table + (size_t)s_seq[lo] * p.pv.max_blocks;
    // ---- the query rows, a warp each ------------------------------------------------
    __syncthreads();
    for (int r = warp; r < p.QT * HYQ_MAX_GQA; r += kWarps) {
      Query& qt = query[r / HYQ_MAX_GQA];
      const int r8 = r & 7, tok = r / p.gq, head = h * p.gq + r - tok * p.gq;
      uint2 v = make_uint2(0, 0);
      float lse = 0.f;
      int lim = 0;
      if (tok < p.n_q) {
        v = *reinterpret_cast<const uint2*>(p.q + ((size_t)lo * p.n_q + tok) * p.ldq + (size_t)head * HYQ_D + 4 * lane);
        lse = p.lse[((size_t)lo * p.n_q + tok) * p.HQ + head];
        lim = max(0, len - p.n_q + 1 + tok);
        const uint32_t e = 0x7F807F80u, a = v.x & e, b = v.y & e;
        bool bad = (a >> 16) == 0x7F80u || (a & 0xFFFFu) == 0x7F80u || (b >> 16) == 0x7F80u || (b & 0xFFFFu) == 0x7F80u;
        bad |= !(fabsf(lse) <= 3.402823466e38f);
        if (__any_sync(0xffffffffu, bad) && lim > 0) {  // its row alone gives nothing
          if (lane == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_SCORE);
          v = make_uint2(0, 0);
          lse = 0.f;
          lim = 0;
        }
      }
      prep_query_row<BK>(r8, lane, v, qt.bq, qt.rowc, qt.bz);
      if (lane == 0) qt.lse[r8] = lse, qt.lim[r8] = lim;
    }
    __syncthreads();
    const int minlim = len - p.n_q + 1;
    // ---- the pages, a warp each ---------------------------------------------------------
    for (int u = u0 + warp; u < u1; u += kWarps) {
      const int pg = table[u], at = u * HYQ_PAGE_ROWS;
      if ((uint32_t)pg >= (uint32_t)p.pv.n_pages) {
        if (lane == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        continue;
      }
      const uint8_t* blk = p.pv.pool + ((size_t)pg * p.HKV + h) * F::kBlock;
      float* mass = p.mass + ((size_t)pg * p.HKV + h) * HYQ_PAGE_ROWS;
      const int refs = p.refs[pg];
      if (refs > 1) {  // several sequences' positions
        if (lane == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_PAGES);
        continue;
      }
      const float old0 = mass[lane], old1 = mass[32 + lane];
      float sums[8];  // of rows g, g + 8 of each tile
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* tb = blk + i * F::kTile;
        uint32_t kw[BK == 4 ? 8 : 16];
        load_words<BK == 4 ? 8 : 16>(tb, lane, kw);
        const uint4 ma = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * g);
        const uint4 mb = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * (g + 8));
        const float2 a01 = half2_to_float2(ma.x), a23 = half2_to_float2(ma.y);
        const float2 b01 = half2_to_float2(mb.x), b23 = half2_to_float2(mb.y);
        const uint32_t za = (t & 1) ? ma.w : ma.z, zb = (t & 1) ? mb.w : mb.z;
        const int p0 = at + 16 * i + g, p1 = p0 + 8;
        const bool all = at + 16 * i + 16 <= minlim;
        float s0 = 0.f, s1 = 0.f;
        for (int k = 0; k < p.QT; ++k) {
          const Query& qt = query[k];
          uint32_t bq[8][2];
          QConst qc;
          load_query_consts(g, t, qt.bq, qt.rowc, qt.bz, bq, qc);
          float C[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) C[q][0] = C[q][1] = C[q][2] = C[q][3] = 0.f;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            if (BK == 4) {
              const uint32_t w = kw[ks], w8 = w >> 8;
              mma_f16(C[ks >> 1], w & 0x000F000Fu, w & 0x00F000F0u, w8 & 0x000F000Fu, w8 & 0x00F000F0u, bq[ks][0],
                      bq[ks][1]);
            } else {
              const uint32_t wa = kw[BK == 4 ? 0 : 2 * ks], wb = kw[BK == 4 ? 0 : 2 * ks + 1];
              mma_f16(C[ks >> 1], wa & 0x00FF00FFu, wb & 0x00FF00FFu, odd_bytes(wa), odd_bytes(wb), bq[ks][0], bq[ks][1]);
            }
          }
          float lg[4];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            lg[c] = qc.ksc[0][c] * fmaf(a01.x, C[0][c], fmaf(a01.y, C[1][c], fmaf(a23.x, C[2][c], a23.y * C[3][c])));
            lg[2 + c] = qc.ksc[1][c] * fmaf(b01.x, C[0][2 + c], fmaf(b01.y, C[1][2 + c], fmaf(b23.x, C[2][2 + c], b23.y * C[3][2 + c])));
          }
          mma_f16(lg, za, zb, 0u, 0u, qc.bz, 0u);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float nl = qt.lse[2 * t + c] * -1.4426950408889634f;
            const int lim = qt.lim[2 * t + c];
            const float e0 = ex2(fmaf(lg[c], qc.inv[c], nl)), e1 = ex2(fmaf(lg[2 + c], qc.inv[c], nl));
            const bool row = lim > 0;
            s0 += (all ? row : p0 < lim) ? e0 : 0.f;
            s1 += (all ? row : p1 < lim) ? e1 : 0.f;
          }
        }
        s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
        s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
        s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
        s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
        sums[2 * i] = s0, sums[2 * i + 1] = s1;
      }
      // row r of the page: sums[r / 8] of the lanes 4 (r % 8) ..; lane l writes rows l and 32 + l
      float add0 = 0.f, add1 = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = __shfl_sync(0xffffffffu, sums[j], 4 * (lane & 7)), y = __shfl_sync(0xffffffffu, sums[4 + j], 4 * (lane & 7));
        if (lane >> 3 == j) add0 = x, add1 = y;
      }
      if (at + lane < len) mass[lane] = (at + lane >= fresh ? 0.f : old0) + add0;
      if (at + 32 + lane < len) mass[32 + lane] = (at + 32 + lane >= fresh ? 0.f : old1) + add1;
    }
  }
}

template <int BK, int BV>
cudaError_t launch(const Params& p, cudaStream_t s) {
  const int bytes = p.QT * (int)sizeof(Query);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = hyq_once_per_device(done, [] {
    return cudaFuncSetAttribute(mass_kernel<BK, BV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                HYQ_PAGED_MAX_Q * (int)sizeof(Query));
  });
  if (e != cudaSuccess) return e;
  const int per_sm = bytes <= 80 * 1024 ? 2 : 1;
  return hyq_launch_chained(mass_kernel<BK, BV>, dim3(per_sm * hyq_num_sms()), kThreads, bytes, s, p);
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
