// Block choice from the bound records (hyq_paged_select).
//
// For a query token and KV head, with c_h the int8 codes of the group's query
// heads, the score of block j is
//   2^e_j sum_h sum_d max(c_hd lo_jd, c_hd hi_jd) = 2^e_j (A . hi_j + N . lo_j),
//   A = sum_h max(c_h, 0), N = sum_h min(c_h, 0):
// the largest term takes hi for a positive code and lo for a negative one, so
// the g heads fold into two vectors and a block costs 256 multiplications
// whatever g is.  All of it is integers, |sum| <= 8 * 128 * 127 * 127 < 2^24:
// exact, in any order, and so are ties.
//
// What bounds it: 260 bytes per (block, KV head) are read, with two products
// per byte; at one sequence the latency of the launch, the dependent loads
// (table, record) and the selection.
//
// One block scores a strided share of one list's blocks into the workspace:
// a warp has 16 records under way (eight lanes each, 16-byte loads), asked for
// before the query's codes are made.  The last block of the list to finish
// selects: the k-th largest key by 8-bit histograms from the highest bit in
// which the keys differ (two passes as a rule), then one ordered pass.
#include "hyq_paged.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 16;              // records that a warp has under way
constexpr int kPerIter = kWarps * kBatch;  // records scored per block and pass
constexpr int kPerSm = 4;               // resident blocks an SM
constexpr int kKeys = 8192;             // keys of a list held in shared memory (32 KB)

struct SelectParams {
  PageView pv;
  const int32_t* seqs;
  const __nv_bfloat16* q;
  int64_t ldq;
  int32_t* sel;
  uint32_t* keys;    // [lists][max_blocks]
  int32_t* tickets;  // [lists]
  int32_t batch, n_q, HQ, HKV, gq, k, n_first, n_last;
};

// Order-preserving image of a float.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int* s) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) t += s[i];
  return t;
}

// grid (shares, n_q * HKV, batch)
__global__ void __launch_bounds__(kThreads, kPerSm) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t s_keys[];  // kKeys
  __shared__ __align__(16) int16_t s_a[HYQ_D], s_n[HYQ_D];
  __shared__ float s_red[kWarps];
  __shared__ int s_cnt[kWarps], s_hist[256], s_pick[3];
  __shared__ uint32_t s_and[kWarps], s_or[kWarps];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  chain_kernel();
  const int b = blockIdx.z, tok = blockIdx.y / p.HKV, h = blockIdx.y - tok * p.HKV;
  const size_t list = ((size_t)b * p.n_q + tok) * p.HKV + h;
  const int seq = page_seq(p.seqs, b, p.pv.n_seqs);
  if (seq < 0 && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
  int64_t len = seq < 0 ? 0 : p.pv.lens[seq];
  len = min(max(len, (int64_t)0), (int64_t)p.pv.max_blocks * HYQ_PAGE_ROWS);
  const int64_t lim = max((int64_t)0, len - p.n_q + 1 + tok);
  const int nb = (int)((lim + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS);
  int32_t* sel = p.sel + list * p.k;
  auto query = [&] { return p.q + ((size_t)b * p.n_q + tok) * p.ldq + (size_t)h * p.gq * HYQ_D; };
  if (nb <= p.k) {  // every block that the token sees
    if (blockIdx.x == 0) {
      for (int i = tid; i < p.k; i += kThreads) sel[i] = i < nb ? i : -1;
      const __nv_bfloat16* q = query();
      bool odd = false;
      if (nb > 0)
        for (int i = tid; i < p.gq * HYQ_D; i += kThreads) odd |= !isfinite(__bfloat162float(q[i]));
      if (odd) hyq_set_err(p.pv.err, HYQ_DEVERR_SCORE);
    }
    return;
  }
  // ---- the first records: lane i < 16 holds the page of record i, eight lanes
  // then read a record each time, 16 elements a lane ---------------------------
  const int part = lane & 7, which = lane >> 3;  // record 4 x + which in step x
  const int32_t* table = p.pv.table + (size_t)seq * p.pv.max_blocks;
  uint32_t* keys = p.keys + list * p.pv.max_blocks;
  int j0 = blockIdx.x * kPerIter + warp * kBatch;
  auto page_at = [&](int j) { return lane < kBatch && j + lane < nb ? table[j + lane] : -1; };
  int page = page_at(j0), page_next = page_at(j0 + gridDim.x * kPerIter);
  int4 lo[kBatch / 4], hi[kBatch / 4];
  int ex[kBatch / 4];
  auto fetch = [&]() {
#pragma unroll
    for (int x = 0; x < kBatch / 4; ++x) {
      const int pg = __shfl_sync(0xffffffffu, page, 4 * x + which);
      lo[x] = hi[x] = make_int4(0, 0, 0, 0);
      ex[x] = INT32_MIN;  // no record
      if ((uint32_t)pg < (uint32_t)p.pv.n_pages) {
        const uint8_t* rec = p.pv.bounds + ((size_t)pg * p.HKV + h) * HYQ_BOUND_BYTES;
        lo[x] = reinterpret_cast<const int4*>(rec)[part];
        hi[x] = reinterpret_cast<const int4*>(rec + HYQ_D)[part];
        ex[x] = *reinterpret_cast<const int*>(rec + 2 * HYQ_D);
      }
    }
  };
  fetch();
  // ---- the query's codes: thread i < 128 holds element i of every head ------
  float x[HYQ_MAX_GQA], am = 0.f;
  const __nv_bfloat16* q = query();
  bool odd = false;
  if (tid < HYQ_D) {
#pragma unroll
    for (int r = 0; r < HYQ_MAX_GQA; ++r) {
      x[r] = r < p.gq ? __bfloat162float(q[r * HYQ_D + tid]) : 0.f;
      odd |= !isfinite(x[r]);
      am = fmaxf(am, fabsf(x[r]));
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  if (lane == 0) s_red[warp] = am;
  odd = __syncthreads_or(odd);
  if (tid < HYQ_D) {
    am = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float inv = pow2_int(min(-bound_exp(odd ? 0.f : am), 127));
    int pos = 0, neg = 0;
#pragma unroll
    for (int r = 0; r < HYQ_MAX_GQA; ++r) {
      const int c = odd ? 0 : __float2int_rn(x[r] * inv);
      pos += max(c, 0);
      neg += min(c, 0);
    }
    s_a[tid] = (int16_t)pos;
    s_n[tid] = (int16_t)neg;
  }
  if (odd && tid == 0 && blockIdx.x == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_SCORE);
  __syncthreads();
  int a[8], n[8];  // pairs of int16
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = reinterpret_cast<const int*>(s_a)[8 * part + i];
    n[i] = reinterpret_cast<const int*>(s_n)[8 * part + i];
  }
  // ---- scores -----------------------------------------------------------------
  for (; j0 < nb; j0 += gridDim.x * kPerIter) {
#pragma unroll
    for (int s = 0; s < kBatch / 4; ++s) {
      const int l[4] = {lo[s].x, lo[s].y, lo[s].z, lo[s].w}, u[4] = {hi[s].x, hi[s].y, hi[s].z, hi[s].w};
      int acc = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = __dp2a_lo(a[2 * i], u[i], acc);
        acc = __dp2a_hi(a[2 * i + 1], u[i], acc);
        acc = __dp2a_lo(n[2 * i], l[i], acc);
        acc = __dp2a_hi(n[2 * i + 1], l[i], acc);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      const int j = j0 + 4 * s + which;
      if (j < nb && part == 0) {
        const bool forced = j < p.n_first || j >= nb - p.n_last, ok = ex[s] != INT32_MIN;
        if (!ok) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
        // 0 and all ones lie outside the keys of finite scores
        keys[j] = forced ? 0xFFFFFFFFu : ok ? key_of((float)acc * pow2_int(min(max(ex[s], -126), 127))) : 0u;
      }
    }
    page = page_next;
    page_next = page_at(j0 + 2 * gridDim.x * kPerIter);
    if (j0 + gridDim.x * kPerIter < nb) fetch();
  }
  // ---- the last block of the list selects ------------------------------------
  __syncthreads();
  if (tid == 0) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(old) : "l"(p.tickets + list) : "memory");
    s_last = old == (int)gridDim.x - 1;
    if (s_last) p.tickets[list] = 0;
  }
  __syncthreads();
  if (!s_last) return;
  // A thread's keys are contiguous, so that ranks follow the block order.
  const int per = (nb + kThreads - 1) / kThreads, i0 = min(tid * per, nb), i1 = min(i0 + per, nb);
  const bool held = nb <= kKeys;
  uint32_t all_and = 0xFFFFFFFFu, all_or = 0u;
  int forced = 0;
  for (int i = tid; i < nb; i += kThreads) {
    const uint32_t u = __ldcg(keys + i);
    if (held) s_keys[i] = u;
    if (u == 0xFFFFFFFFu) {
      ++forced;
    } else {
      all_and &= u;
      all_or |= u;
    }
  }
  all_and = __reduce_and_sync(0xffffffffu, all_and);
  all_or = __reduce_or_sync(0xffffffffu, all_or);
  if (lane == 0) s_and[warp] = all_and, s_or[warp] = all_or;
  forced = block_sum(forced, s_cnt);  // its barriers publish s_and, s_or and s_keys
#pragma unroll
  for (int i = 0; i < kWarps; ++i) all_and &= s_and[i], all_or |= s_or[i];
  auto key = [&](int i) { return held ? s_keys[i] : __ldcg(keys + i); };
  // The bound v and the number `take` of keys equal to it that make `want`
  // selected keys among those not forced: digit by digit, `want` the keys still
  // to be found among those that agree with v above `shift`.
  int want = p.k - forced;
  uint32_t v = all_and;
  if (want <= 0) {
    v = 0xFFFFFFFEu;  // the forced blocks alone
  } else if (all_and != all_or) {
    const int top = 31 - __clz(all_and ^ all_or);
    v = all_and & ~((2u << top) - 1u);
    for (int high = top + 1; high > 0;) {
      const int shift = max(high - 8, 0);
      const uint32_t digits = (1u << (high - shift)) - 1u;
      for (int i = tid; i < 256; i += kThreads) s_hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < nb; i += kThreads) {
        const uint32_t u = key(i);
        if (u != 0xFFFFFFFFu && (high == 32 || (u >> high) == (v >> high))) atomicAdd(&s_hist[(u >> shift) & digits], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // lane l: digits 255 - 8 l .. 248 - 8 l, the largest first
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i] = s_hist[255 - 8 * lane - i];
        int pre = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += y;
        }
        int before = pre - sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < want && before + c[i] >= want) s_pick[0] = 255 - 8 * lane - i, s_pick[1] = before, s_pick[2] = c[i];
          before += c[i];
        }
      }
      __syncthreads();
      v |= (uint32_t)s_pick[0] << shift;
      want -= s_pick[1];
      const bool whole = s_pick[2] == want;
      high = shift;
      if (whole && shift > 0) {  // every key of this digit is selected: a bound just below them
        v -= 1u;
        want = 0;
        break;
      }
    }
  }
  // ranks: every key above v, and the first `want - above` equal to it
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t u = key(i);
    gt += u > v;
    eq += u == v && want > 0;  // want > 0: ties are left to take
  }
  const int above = block_sum(gt, s_cnt);
  // exclusive prefix of (gt, eq) over the threads
  int pg = gt, pe = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, pg, o), z = __shfl_up_sync(0xffffffffu, pe, o);
    if (lane >= o) pg += y, pe += z;
  }
  __syncthreads();
  if (lane == 31) s_cnt[warp] = pg, s_and[warp] = (uint32_t)pe;
  __syncthreads();
  int g0 = pg - gt, e0 = pe - eq;
  for (int i = 0; i < warp; ++i) g0 += s_cnt[i], e0 += (int)s_and[i];
  const int take = p.k - above;  // equal keys to take
  int at = g0 + min(e0, take), seen = e0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t u = key(i);
    if (u > v) {
      sel[at++] = i;
    } else if (u == v && want > 0) {
      if (seen < take) sel[at++] = i;
      ++seen;
    }
  }
}

int shares_of(int64_t lists, int32_t max_blocks) {
  // at most the blocks that are resident together (a second wave costs more
  // than longer shares: 256 lists of a thousand blocks 22.3 against 20.6 us), and
  // no more than there are passes
  const int64_t fill = kPerSm * (int64_t)hyq_num_sms() / lists;
  const int64_t most = (max_blocks + kPerIter - 1) / kPerIter;
  return (int)(fill < most ? (fill > 1 ? fill : 1) : most);
}

}  // namespace

// Tickets first at a size that only the batch limits set, then the keys.
static constexpr size_t kSelectLists = (size_t)HYQ_PAGED_MAX_BATCH * HYQ_PAGED_MAX_Q;

size_t hyq_paged_select_ws_bytes(const hyq_config* c, const hyq_pages* p, int32_t batch, int32_t n_q) {
  const size_t lists = (size_t)batch * n_q * c->num_kv_heads;
  return hyq_align256(kSelectLists * c->num_kv_heads * 4) + hyq_align256(lists * p->max_blocks * 4);
}

cudaError_t hyq_launch_paged_select(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                    int32_t n_q, const void* q, int64_t ldq, int32_t k, int32_t n_first,
                                    int32_t n_last, int32_t* sel, void* ws, cudaStream_t s) {
  SelectParams p;
  p.pv = pv;
  p.seqs = seqs;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.sel = sel;
  p.tickets = static_cast<int32_t*>(ws);
  p.keys = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + hyq_align256(kSelectLists * c->num_kv_heads * 4));
  p.batch = batch;
  p.n_q = n_q;
  p.HQ = c->num_q_heads;
  p.HKV = c->num_kv_heads;
  p.gq = c->num_q_heads / c->num_kv_heads;
  p.k = k;
  p.n_first = n_first;
  p.n_last = n_last;
  const int64_t lists = (int64_t)batch * n_q * p.HKV;
  const dim3 grid(shares_of(lists, pv.max_blocks), n_q * p.HKV, batch);
  return hyq_launch_chained(select_kernel, grid, kThreads, kKeys * 4, s, p);
}
