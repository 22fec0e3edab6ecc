// Eviction from the paged cache by accumulated attention weight (hyq_pages_evict).
//
// A sequence of n positions keeps k of them, per layer and KV head: the first
// n_first, the last n_last and, of the others, those of largest mass, ties to the lower
// position.  With w = k - n_last the kept positions below w stay where they are, those
// from w to n - n_last go to the free places below w (ascending to ascending), the
// last n_last go to [w, k) in order.  So a row moves only if it has to, a
// moved row is read and written once, and nothing is read after it has been written: the
// free places lie below w, what goes there at or behind it.
//
// Four launches: which sequences and how many pages (one block); the kept positions of
// every (layer, sequence, KV head) as a bit mask a page with the number kept before it;
// the free places, a block a page; the last n_last positions, which may overlap their
// new places and are therefore taken a page after another by one block, and the
// tables.  What bounds it: the mass is read once, each moved row read and written
// once, and of each page that changes the keys for its bounds: HBM for long
// prompts, latency (dependent launches and reads) for small calls.
#include "hyq_codes.cuh"
#include "hyq_f2.cuh"
#include "hyq_paged.cuh"

namespace {

constexpr int kPlanThreads = 1024;

// A row of the call as the plan leaves it.
struct Row {
  int32_t seq, n, k;  // k < 0: nothing to do
};
struct EvictWs {
  int64_t* cum;     // [batch + 1] pages below w of the rows before
  Row* row;         // [batch]
  uint64_t* mask;   // [n_layers][batch][HKV][max_blocks] kept positions below n - n_last
  int32_t* before;  // likewise: how many are kept in the pages before
};
size_t masks(const hyq_config* c, const hyq_pages* p, int32_t batch) {
  return (size_t)p->n_layers * batch * c->num_kv_heads * p->max_blocks;
}
EvictWs evict_ws(const hyq_config* c, const hyq_pages* p, int32_t batch, void* ws) {
  char* w = static_cast<char*>(ws);
  EvictWs r;
  r.cum = reinterpret_cast<int64_t*>(w);
  w += hyq_align256((batch + 1) * sizeof(int64_t));
  r.row = reinterpret_cast<Row*>(w);
  w += hyq_align256(batch * sizeof(Row));
  r.mask = reinterpret_cast<uint64_t*>(w);
  w += hyq_align256(masks(c, p, batch) * 8);
  r.before = reinterpret_cast<int32_t*>(w);
  return r;
}

struct Params {
  hyq_pages pages;
  const int32_t* seqs;
  const int32_t* keep;
  float* mass;  // [n_layers][n_pages][HKV][64]
  EvictWs ws;
  int32_t batch, n_first, n_last, HKV;
};

// One block; thread i handles call row i, warps look at the rows' pages.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Params p) {
  static_assert(HYQ_PAGED_MAX_BATCH <= kPlanThreads, "one row per thread");
  __shared__ int s_seq[kPlanThreads], s_n[kPlanThreads], s_k[kPlanThreads];
  __shared__ int64_t s_warp[kPlanThreads / 32];
  chain_kernel();
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
  const hyq_pages& pg = p.pages;
  s_seq[i] = i < p.batch ? page_seq(p.seqs, i, pg.n_seqs) : -1;
  __syncthreads();
  int n = 0, k = -1, err = 0;
  if (i < p.batch) {
    const int s = s_seq[i];
    bool bad = s < 0;
    for (int j = 0; p.seqs && j < i; ++j) bad |= s_seq[j] == s;
    k = p.keep[i];
    bad |= k < p.n_first + p.n_last;
    if (!bad) {
      n = pg.lens[s];
      bad = n < 0 || (int64_t)n > (int64_t)pg.max_blocks * HYQ_PAGE_ROWS;
    }
    if (bad) err = HYQ_DEVERR_INDEX;
    if (bad || n <= k) k = -1;
  }
  s_n[i] = n;
  s_k[i] = k;
  __syncthreads();
  for (int r = warp; r < p.batch; r += kPlanThreads / 32) {
    if (s_k[r] < 0) continue;
    const int32_t* table = pg.table + (size_t)s_seq[r] * pg.max_blocks;
    const int nb = (s_n[r] + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS, kb = (s_k[r] + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS;
    int e = 0;
    for (int j = lane; j < nb; j += 32) {
      const int page = table[j];
      if (page < 0 || page >= pg.n_pages) e |= HYQ_DEVERR_INDEX;
      else if (j < kb && pg.refs[page] > 1) e |= HYQ_DEVERR_PAGES;  // held by another sequence too
    }
    e = __reduce_or_sync(0xffffffffu, (unsigned)e);
    if (e && lane == 0) {
      s_k[r] = -1;
      hyq_set_err(pg.err, e);
    }
  }
  if (err) hyq_set_err(pg.err, err);
  __syncthreads();
  k = s_k[i];
  int64_t w = i < p.batch && k >= 0 ? (k - p.n_last + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS : 0, pre = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += y;
  }
  if (lane == 31) s_warp[warp] = pre;
  __syncthreads();
  int64_t at = pre - w;
  for (int j = 0; j < warp; ++j) at += s_warp[j];
  if (i < p.batch) {
    p.ws.cum[i] = at;
    if (i == p.batch - 1) p.ws.cum[p.batch] = at + w;
    p.ws.row[i] = Row{s_seq[i], n, k};
  }
}

// A mass as an integer above 0 that orders like it: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kPiece = 16;          // positions that a thread takes at a time
constexpr int kSmall = 8192;        // positions that a small block holds
static_assert(HYQ_PAGE_ROWS == 4 * kPiece, "four lanes a page");

// One block per (layer, row, KV head).  The threshold is found two bits at a time by counting the keys at and above
// three candidates: the keys stay in registers (read again for each pair of bits past the first 32768 positions), and
// counting needs no atomics, whose bins the exponents of masses share (by a histogram of eight bits at a time, a page a
// thread: 229 us for 4096 selections of 4160, with this NNN).
// kSelThreads threads hold kHeld pieces each.  Two sizes, three small blocks or a large one an SM, each for the
// sequences of its size (all in large ones: 975 us instead of NNN for the whole eviction of 16 x 4096 in 32 layers).
template <int kSelThreads, int kHeld>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const Params p) {
  constexpr int kSelWarps = kSelThreads / 32, kPass = kSelThreads * kPiece;  // positions of a pass
  __shared__ int s_count[2][3][kSelWarps], s_scan[kSelWarps];
  chain_kernel();
  const int h = blockIdx.x % p.HKV, b = blockIdx.x / p.HKV, layer = blockIdx.y, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const Row row = p.ws.row[b];
  if (row.k < 0) return;
  const int hi = row.n - p.n_last, w = row.k - p.n_last, want = w - p.n_first;  // of [n_first, hi)
  if ((hi <= kSmall) != (kHeld * kPass == kSmall)) return;  // the other size's
  const int32_t* table = p.pages.table + (size_t)row.seq * p.pages.max_blocks;
  const float* mass = p.mass + (size_t)layer * p.pages.n_pages * p.HKV * HYQ_PAGE_ROWS;
  // the keys of the piece that begins at `pos`; those that are not to be chosen from are 0 (no mass's key)
  auto keys = [&](int pos, uint32_t (&key)[kPiece]) {
    float4 v[kPiece / 4];
#pragma unroll
    for (int c = 0; c < kPiece / 4; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pos < hi) {
      const float4* at = reinterpret_cast<const float4*>(
          mass + ((size_t)table[pos / HYQ_PAGE_ROWS] * p.HKV + h) * HYQ_PAGE_ROWS + pos % HYQ_PAGE_ROWS);
#pragma unroll
      for (int c = 0; c < kPiece / 4; ++c) v[c] = at[c];
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const float x = i & 2 ? (i & 1 ? v[i >> 2].w : v[i >> 2].z) : (i & 1 ? v[i >> 2].y : v[i >> 2].x);
      key[i] = pos + i >= p.n_first && pos + i < hi ? mass_key(x) : 0u;
    }
  };
  uint32_t held[kHeld][kPiece];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) keys(k * kPass + kPiece * tid, held[k]);
  // the want-th largest key: the largest one that at least `want` keys reach
  uint32_t key = 0;
#pragma unroll 1
  for (int shift = 30; shift >= 0 && want > 0; shift -= 2) {
    const uint32_t c1 = key | 1u << shift, c2 = key | 2u << shift, c3 = key | 3u << shift;
    int n1 = 0, n2 = 0, n3 = 0;
    auto count = [&](const uint32_t (&x)[kPiece]) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) n1 += x[i] >= c1, n2 += x[i] >= c2, n3 += x[i] >= c3;
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (k * kPass < hi) count(held[k]);
    for (int pos = kHeld * kPass + kPiece * tid; pos < hi; pos += kPass) {
      uint32_t x[kPiece];
      keys(pos, x);
      count(x);
    }
    n1 = __reduce_add_sync(0xffffffffu, n1), n2 = __reduce_add_sync(0xffffffffu, n2), n3 = __reduce_add_sync(0xffffffffu, n3);
    int(&s)[3][kSelWarps] = s_count[(shift >> 1) & 1];
    if (lane == 0) s[0][warp] = n1, s[1][warp] = n2, s[2][warp] = n3;
    __syncthreads();
    const bool in = lane < kSelWarps;  // every warp sums up the warps' counts
    n1 = __reduce_add_sync(0xffffffffu, in ? s[0][lane] : 0), n2 = __reduce_add_sync(0xffffffffu, in ? s[1][lane] : 0);
    n3 = __reduce_add_sync(0xffffffffu, in ? s[2][lane] : 0);
    key = n3 >= want ? c3 : n2 >= want ? c2 : n1 >= want ? c1 : key;
  }
  // the mask: what lies above the key, and the first of those that equal it
  const size_t base = (((size_t)layer * p.batch + b) * p.HKV + h) * p.pages.max_blocks;
  int kept = 0, ties = 0;  // in the pieces before
  auto scan = [&](int v, int& before) {  // exclusive over the block, on top of `before`
    int pre = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = pre;
    __syncthreads();
    int at = before + pre - v;
    for (int k = 0; k < kSelWarps; ++k) {
      if (k < warp) at += s_scan[k];
      before += s_scan[k];
    }
    return at;
  };
  // how many of those that equal the key are kept: all above it are
  int above = 0;
  auto over = [&](const uint32_t (&x)[kPiece]) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) above += x[i] > key;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (k * kPass < hi) over(held[k]);
  for (int pos = kHeld * kPass + kPiece * tid; pos < hi; pos += kPass) {
    uint32_t x[kPiece];
    keys(pos, x);
    over(x);
  }
  int total = 0;
  (void)scan(above, total);
  const int left = want - total;
  auto finish = [&](int pos, const uint32_t (&x)[kPiece]) {  // (all threads)
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      gt |= (uint32_t)(want > 0 && x[i] > key) << i;
      eq |= (uint32_t)(want > 0 && x[i] == key && key != 0) << i;
    }
    const int nf = p.n_first - pos;
    if (nf > 0) gt |= nf >= kPiece ? (1u << kPiece) - 1 : (1u << nf) - 1;
    const int tie_at = scan(__popc(eq), ties);
    int drop = __popc(eq) - max(0, min(__popc(eq), left - tie_at));
    for (; drop > 0; --drop) eq &= ~(1u << (31 - __clz(eq)));
    const uint32_t m = pos < hi ? gt | eq : 0u;
    const int at = scan(__popc(m), kept);
    // four lanes' pieces are a page
    const uint32_t lo = m | __shfl_down_sync(0xffffffffu, m, 1) << 16, up = __shfl_down_sync(0xffffffffu, lo, 2);
    if ((lane & 3) == 0 && pos < hi) {
      p.ws.mask[base + pos / HYQ_PAGE_ROWS] = (uint64_t)lo | (uint64_t)up << 32;
      p.ws.before[base + pos / HYQ_PAGE_ROWS] = at;
    }
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (k * kPass < hi) finish(k * kPass + kPiece * tid, held[k]);
  for (int first = kHeld * kPass; first < hi; first += kPass) {
    uint32_t x[kPiece];
    keys(first + kPiece * tid, x);
    finish(first + kPiece * tid, x);
  }
}

// ---- rows ------------------------------------------------------------------------------
// One row of a 16-row tile, spread over a warp: its key codes as 32 words (of 4-bit codes the
// row's nibbles, low), its value codes a byte at a time, its steps and zeros.
template <int BK, int BV>
struct HeldRow {
  using F = QFmt<BK, BV>;
  static constexpr int kV = BV == 4 ? 2 : 4;
  uint32_t k, km;
  uint8_t v[kV];
  uint16_t vm;
  static __device__ __forceinline__ int key_word(int r, int lane) {
    const int t = lane & 3, u = BK == 4 ? lane >> 2 : 2 * (lane >> 2) + (r >> 3);
    return 512 * (u >> 2) + 16 * (4 * (r & 7) + t) + 4 * (u & 3);
  }
  static __device__ __forceinline__ int value_byte(int r, int lane, int i) {
    const int u = (lane >> 3) + 4 * i;
    return F::kVCode + 512 * (u >> 2) + 16 * (4 * (lane & 7) + ((r & 7) >> 1)) + 4 * (u & 3) + (r >> 3) + 2 * (r & 1);
  }
  static __device__ __forceinline__ int key_meta(int r, int lane) { return F::kKMeta + 16 * r + 4 * lane; }
  static __device__ __forceinline__ int value_meta(int r, int lane) {
    return F::kVMeta + 128 * (lane >> 2) + 16 * (r >> 1) + 4 * (lane & 3) + 2 * (r & 1);
  }
  __device__ __forceinline__ void load(const uint8_t* tile, int r, int lane) {
    k = *reinterpret_cast<const uint32_t*>(tile + key_word(r, lane));
    if (BK == 4) k = (k >> (4 * (r >> 3))) & 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = tile[value_byte(r, lane, i)];
    if (lane < 4) km = *reinterpret_cast<const uint32_t*>(tile + key_meta(r, lane));
    if (lane < 8) vm = *reinterpret_cast<const uint16_t*>(tile + value_meta(r, lane));
  }
  __device__ __forceinline__ void store(uint8_t* tile, int r, int lane) const {
    uint32_t* kw = reinterpret_cast<uint32_t*>(tile + key_word(r, lane));
    if (BK == 4) *kw = (*kw & ~(0x0F0F0F0Fu << (4 * (r >> 3)))) | k << (4 * (r >> 3));
    else *kw = k;
#pragma unroll
    for (int i = 0; i < kV; ++i) tile[value_byte(r, lane, i)] = v[i];
    if (lane < 4) *reinterpret_cast<uint32_t*>(tile + key_meta(r, lane)) = km;
    if (lane < 8) *reinterpret_cast<uint16_t*>(tile + value_meta(r, lane)) = vm;
  }
};

constexpr int kMoveThreads = 128;  // four warps: a 16-row tile of a page each
constexpr int kHold = 4;           // rows of a tile under way at a time

// Where the rows of one (layer, sequence, KV head) lie.
struct Place {
  uint8_t* pool;   // of (layer, page 0, head)
  float* mass;
  uint8_t* bounds;
  const int32_t* table;
  int HKV;
  template <int BK, int BV>
  __device__ __forceinline__ uint8_t* tile(int pos) const {
    return pool + (size_t)table[pos / HYQ_PAGE_ROWS] * HKV * QFmt<BK, BV>::kBlock + (pos % HYQ_PAGE_ROWS / 16) * QFmt<BK, BV>::kTile;
  }
  __device__ __forceinline__ float* weight(int pos) const {
    return mass + (size_t)table[pos / HYQ_PAGE_ROWS] * HKV * HYQ_PAGE_ROWS + pos % HYQ_PAGE_ROWS;
  }
};
template <int BK, int BV>
__device__ __forceinline__ Place place_of(const Params& p, const Row& row, int layer, int h) {
  const size_t block = (size_t)layer * p.pages.n_pages * p.HKV + h;
  return Place{p.pages.pool + block * QFmt<BK, BV>::kBlock, p.mass + block * HYQ_PAGE_ROWS,
               p.pages.bounds + block * HYQ_BOUND_BYTES, p.pages.table + (size_t)row.seq * p.pages.max_blocks, p.HKV};
}

// One warp: lane r < 16 names the position that comes to row r of the tile, or -1.  The rows go into the tile's
// copy `held` in shared memory, their masses are returned to lane r.
template <int BK, int BV>
__device__ __forceinline__ float gather_rows(const Place& pl, uint8_t* held, int lane, int from) {
  float weight = 0.f;
  if (lane < 16 && from >= 0) weight = *pl.weight(from);
  uint32_t todo = __ballot_sync(0xffffffffu, lane < 16 && from >= 0);
  while (todo) {
    HeldRow<BK, BV> x[kHold];
    int r[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      r[i] = todo ? __ffs(todo) - 1 : -1;
      todo &= todo - 1;
      const int src = __shfl_sync(0xffffffffu, from, r[i] < 0 ? 0 : r[i]);
      if (r[i] >= 0) x[i].load(pl.tile<BK, BV>(src), src % 16, lane);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r[i] >= 0) x[i].store(held, r[i], lane);
  }
  __syncwarp();
  return weight;
}
template <int BK, int BV>
__device__ __forceinline__ void copy_tile(uint8_t* to, const uint8_t* from, int lane) {
  constexpr int n = QFmt<BK, BV>::kTile / 16;
#pragma unroll
  for (int i = 0; i < (n + 31) / 32; ++i)
    if (32 * i + lane < n) reinterpret_cast<uint4*>(to)[32 * i + lane] = reinterpret_cast<const uint4*>(from)[32 * i + lane];
}

// One block: the bound record of a page's rows [0, rows) as they are held, from its tiles in shared memory.
template <int BK, int BV>
__device__ __forceinline__ void write_record(const uint8_t* page, int rows, uint8_t* rec, float* red /* [4] */) {
  using F = QFmt<BK, BV>;
  const int d = threadIdx.x;  // kMoveThreads = 128 elements
  float mn = INFINITY, mx = -INFINITY;
  // byte and nibble of element d in row 0 (4-bit: rows g, g + 8 share it)
  const int q = d >> 5;
  int at;
  if (BK == 4) {
    const int t = (d >> 3) & 3, u = 2 * q + ((d >> 2) & 1);
    at = 512 * (u >> 2) + 16 * t + 4 * (u & 3) + ((d >> 1) & 1) + 2 * (d & 1);
  } else {
    const int t = (d >> 2) & 3, u = 2 * (d >> 4), e = d & 3;
    at = 512 * (u >> 2) + 16 * t + 4 * (u & 3) + (e >> 1) + 2 * (e & 1);
  }
  for (int r = 0; r < rows; ++r) {
    const uint8_t* tile = page + (r >> 4) * F::kTile;
    const int i = r & 15;
    int c = tile[at + 64 * (i & 7) + (BK == 8 ? 4 * (i >> 3) : 0)];
    if (BK == 4) c = (c >> (4 * (i >> 3))) & 15;
    const __half* m = reinterpret_cast<const __half*>(tile + F::kKMeta + 16 * i);
    const float x = fmaf((float)c, __half2float(m[q]), __half2float(m[4 + q]));
    mn = fminf(mn, x);
    mx = fmaxf(mx, x);
  }
  float am = fmaxf(fabsf(mn), fabsf(mx));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  __syncthreads();
  if ((d & 31) == 0) red[d >> 5] = am;
  __syncthreads();
  am = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const int e = bound_exp(am);
  const float f = pow2_int(-e);
  rec[d] = (uint8_t)(int8_t)(int)floorf(mn * f);
  rec[HYQ_D + d] = (uint8_t)(int8_t)(int)ceilf(mx * f);
  if (d < 4) reinterpret_cast<int32_t*>(rec + 2 * HYQ_D)[d] = d == 0 ? e : 0;
}

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One warp: least and largest keys of a page, element by element, as they are held.
template <int BK, int BV>
struct Extremes {
  float lo[32], hi[32];  // of the lane's rows so far: elements 32 v + .. of its eight of each group v
  uint4 kc[BK / 2], ka, kb;

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < 32; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  }
  __device__ __forceinline__ void load(const uint8_t* tile, int lane) {
    using F = QFmt<BK, BV>;
#pragma unroll
    for (int i = 0; i < BK / 2; ++i) kc[i] = *reinterpret_cast<const uint4*>(tile + 512 * i + 16 * lane);
    ka = *reinterpret_cast<const uint4*>(tile + F::kKMeta + 16 * (lane >> 2));
    kb = *reinterpret_cast<const uint4*>(tile + F::kKMeta + 16 * ((lane >> 2) + 8));
  }
  // The tile's rows below vr (kAll: all sixteen).
  template <bool kAll>
  __device__ __forceinline__ void take(int lane, int vr) {
    const bool ina = (lane >> 2) < vr, inb = (lane >> 2) + 8 < vr;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      uint32_t xa[4], xb[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (BK == 4) {
          const uint32_t w = u4at(kc[v >> 1], 2 * (v & 1) + u), w8 = w >> 8;
          xa[2 * u] = low_codes(w), xa[2 * u + 1] = low_codes(w8);
          xb[2 * u] = high_codes(w), xb[2 * u + 1] = high_codes(w8);
        } else {
          const uint32_t wa = u4at(kc[BK == 4 ? 0 : v], 2 * u), wb = u4at(kc[BK == 4 ? 0 : v], 2 * u + 1);
          xa[2 * u] = even_codes(wa), xa[2 * u + 1] = odd_codes(wa);
          xb[2 * u] = even_codes(wb), xb[2 * u + 1] = odd_codes(wb);
        }
      }
      auto half = [&](uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(v & 1 ? w >> 16 : w & 0xFFFFu))); };
      const float sa = half(v < 2 ? ka.x : ka.y), za = half(v < 2 ? ka.z : ka.w);
      const float sb = half(v < 2 ? kb.x : kb.y), zb = half(v < 2 ? kb.z : kb.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 ca = *reinterpret_cast<const __half2*>(&xa[i]), cb = *reinterpret_cast<const __half2*>(&xb[i]);
        const float a[2] = {fmaf(__low2float(ca), sa, za), fmaf(__high2float(ca), sa, za)};
        const float b[2] = {fmaf(__low2float(cb), sb, zb), fmaf(__high2float(cb), sb, zb)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = 8 * v + 2 * i + e;
          lo[at] = fmin3(lo[at], kAll || ina ? a[e] : INFINITY, kAll || inb ? b[e] : INFINITY);
          hi[at] = fmax3(hi[at], kAll || ina ? a[e] : -INFINITY, kAll || inb ? b[e] : -INFINITY);
        }
      }
    }
  }
  // The record of what has been taken: lanes that differ in g exchange halves until each has four elements of all rows.
  __device__ __forceinline__ void write(uint8_t* rec, int lane) {
    auto halve = [&](int n, int bit) {  // of the first 2 n elements a lane keeps the half that its bit says
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) {
          const float l = __shfl_xor_sync(0xffffffffu, up ? lo[i] : lo[n + i], bit), h = __shfl_xor_sync(0xffffffffu, up ? hi[i] : hi[n + i], bit);
          lo[i] = fminf(up ? lo[n + i] : lo[i], l);
          hi[i] = fmaxf(up ? hi[n + i] : hi[i], h);
        }
    };
    halve(16, 16);
    halve(8, 8);
    halve(4, 4);
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) am = fmax3(am, fabsf(lo[i]), fabsf(hi[i]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    const int e = bound_exp(am), t = lane & 3, v = lane >> 3, i4 = (lane >> 2) & 1;
    const float f = pow2_int(-e);
    uint32_t l = 0, h = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l |= (uint32_t)(uint8_t)(int8_t)(int)floorf(lo[i] * f) << (8 * i);
      h |= (uint32_t)(uint8_t)(int8_t)(int)ceilf(hi[i] * f) << (8 * i);
    }
    const int at = 32 * v + (BK == 4 ? 8 * t + 4 * i4 : 16 * i4 + 4 * t);
    *reinterpret_cast<uint32_t*>(rec + at) = l;
    *reinterpret_cast<uint32_t*>(rec + HYQ_D + at) = h;
    if (lane < 4) reinterpret_cast<int32_t*>(rec + 2 * HYQ_D)[lane] = lane == 0 ? e : 0;
  }
};

// The free places below w: a warp takes one page of one (layer, row, KV head).  A tile without free places is read for its
// keys alone, straight into registers, the next one ahead.
template <int BK, int BV>
__global__ void __launch_bounds__(kMoveThreads) fill_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  __shared__ __align__(16) uint8_t s_tile[kMoveThreads / 32][F::kTile];
  chain_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* held = s_tile[warp];
  const int64_t per = (int64_t)p.HKV * p.pages.n_layers, items = p.ws.cum[p.batch] * per;
  for (int64_t it = (int64_t)blockIdx.x * (kMoveThreads / 32) + warp; it < items; it += (int64_t)gridDim.x * (kMoveThreads / 32)) {
    const int64_t x = items >> 32 ? it / per : (uint32_t)it / (uint32_t)per;
    const int lh = (int)(it - x * per), layer = lh / p.HKV, h = lh - layer * p.HKV;
    int b = 0, hi = p.batch;
    while (hi - b > 1) {
      const int m = (b + hi) >> 1;
      if (p.ws.cum[m] <= x) b = m;
      else hi = m;
    }
    const Row row = p.ws.row[b];
    const int j = (int)(x - p.ws.cum[b]), w = row.k - p.n_last, at = j * HYQ_PAGE_ROWS;
    const size_t base = (((size_t)layer * p.batch + b) * p.HKV + h) * p.pages.max_blocks;
    const int here = min(HYQ_PAGE_ROWS, w - at);  // its rows below w
    const uint64_t holes = ~p.ws.mask[base + j] & (here == 64 ? ~0ull : (1ull << here) - 1);
    if (!holes) continue;
    const Place pl = place_of<BK, BV>(p, row, layer, h);
    // the r-th free place takes the r-th kept position from w on, the (kw + r)-th of all
    const int nb = (row.n - p.n_last + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS, jw = w / HYQ_PAGE_ROWS;
    const uint64_t mw = jw < nb ? p.ws.mask[base + jw] & ((1ull << (w % HYQ_PAGE_ROWS)) - 1) : 0;
    const int kw = jw < nb ? p.ws.before[base + jw] + __popcll(mw) : 0;
    const int rank0 = kw + at - p.ws.before[base + j];  // of the page's first free place
    // a page with rows of the last n_last gets its record when they are there
    const bool record = at + HYQ_PAGE_ROWS <= w || p.n_last == 0;
    const int valid = min(HYQ_PAGE_ROWS, row.k - at);
    uint8_t* tile0 = pl.tile<BK, BV>(at);
    Extremes<BK, BV> x2;
    x2.reset();
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      uint8_t* tile = tile0 + i * F::kTile;
      const uint32_t mine = (uint32_t)(holes >> (16 * i)) & 0xFFFFu;
      if (mine) {
        int from = -1;
        if (lane < 16 && (mine >> lane) & 1) {
          const int rank = rank0 + __popcll(holes & ((1ull << (16 * i + lane)) - 1));
          int lo = jw, up = nb;  // the last page with `before` <= rank
          while (up - lo > 1) {
            const int m = (lo + up) >> 1;
            if (p.ws.before[base + m] <= rank) lo = m;
            else up = m;
          }
          uint64_t m = p.ws.mask[base + lo];
          for (int s = rank - p.ws.before[base + lo]; s > 0; --s) m &= m - 1;
          from = lo * HYQ_PAGE_ROWS + __ffsll(m) - 1;
        }
        copy_tile<BK, BV>(held, tile, lane);
        __syncwarp();
        const float weight = gather_rows<BK, BV>(pl, held, lane, from);
        copy_tile<BK, BV>(tile, held, lane);
        if (from >= 0) *pl.weight(at + 16 * i + lane) = weight;
      }
      if (record && 16 * i < valid) {
        x2.load(mine ? held : tile, lane);
        if (valid - 16 * i >= 16) x2.template take<true>(lane, 16);
        else x2.template take<false>(lane, valid - 16 * i);
      }
      __syncwarp();
    }
    if (record) x2.write(pl.bounds + (size_t)pl.table[j] * p.HKV * HYQ_BOUND_BYTES, lane);
  }
}

// The last n_last positions: a block takes one (layer, row, KV head), a page at a time.  Then the tables.
template <int BK, int BV>
__global__ void __launch_bounds__(kMoveThreads) shift_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  __shared__ __align__(16) uint8_t s_page[F::kBlock];
  __shared__ float s_red[4];
  chain_kernel();
  const int h = blockIdx.x % p.HKV, b = blockIdx.x / p.HKV, layer = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Row row = p.ws.row[b];
  if (row.k < 0) return;
  const Place pl = place_of<BK, BV>(p, row, layer, h);
  const int w = row.k - p.n_last, by = row.n - row.k, kb = (row.k + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS;
  for (int j = w / HYQ_PAGE_ROWS; j < kb && p.n_last > 0; ++j) {
    const int at = j * HYQ_PAGE_ROWS + 16 * warp, pos = at + lane;
    const int from = lane < 16 && pos >= w && pos < row.k ? pos + by : -1;
    uint8_t* tile = pl.tile<BK, BV>(at);
    uint8_t* held = s_page + warp * F::kTile;
    copy_tile<BK, BV>(held, tile, lane);
    __syncwarp();
    const float weight = gather_rows<BK, BV>(pl, held, lane, from);
    __syncthreads();  // all of the page's sources have been read: some lie in the page
    if (__any_sync(0xffffffffu, from >= 0)) copy_tile<BK, BV>(tile, held, lane);
    if (from >= 0) *pl.weight(pos) = weight;
    write_record<BK, BV>(s_page, min(HYQ_PAGE_ROWS, row.k - j * HYQ_PAGE_ROWS),
                         pl.bounds + (size_t)pl.table[j] * p.HKV * HYQ_BOUND_BYTES, s_red);
    __syncthreads();  // the stores are made before the next page's reads
  }
  if (layer == 0 && h == 0) {  // the other blocks have n and k from the plan
    const int nb = (row.n + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS;
    for (int j = kb + threadIdx.x; j < nb; j += kMoveThreads) atomicSub(p.pages.refs + pl.table[j], 1);
    if (threadIdx.x == 0) p.pages.lens[row.seq] = row.k;
  }
}

template <int BK, int BV>
cudaError_t launch(const Params& p, cudaStream_t s) {
  cudaError_t e = hyq_launch_chained(plan_kernel, dim3(1), kPlanThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  const dim3 heads(p.batch * p.HKV, p.pages.n_layers);
  e = hyq_launch_chained(select_kernel<256, 2>, heads, 256, 0, s, p);
  if (e != cudaSuccess) return e;
  if ((int64_t)p.pages.max_blocks * HYQ_PAGE_ROWS > kSmall) {  // longer sequences may be there
    e = hyq_launch_chained(select_kernel<512, 4>, heads, 512, 0, s, p);
    if (e != cudaSuccess) return e;
  }
  e = hyq_launch_chained(fill_kernel<BK, BV>, dim3(4 * hyq_num_sms()), kMoveThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  return hyq_launch_chained(shift_kernel<BK, BV>, heads, kMoveThreads, 0, s, p);
}

}  // namespace

size_t hyq_pages_evict_ws_bytes(const hyq_config* c, const hyq_pages* p, int32_t batch) {
  const size_t n = masks(c, p, batch);
  return hyq_align256((batch + 1) * sizeof(int64_t)) + hyq_align256(batch * sizeof(Row)) + hyq_align256(n * 8) +
         hyq_align256(n * 4);
}

cudaError_t hyq_launch_pages_evict(const hyq_config* c, const hyq_pages* p, const int32_t* seqs, int32_t batch,
                                   const int32_t* keep, int32_t n_first, int32_t n_last, float* mass, void* ws,
                                   cudaStream_t s) {
  Params q;
  q.pages = *p;
  q.seqs = seqs;
  q.keep = keep;
  q.mass = mass;
  q.ws = evict_ws(c, p, batch, ws);
  q.batch = batch;
  q.n_first = n_first;
  q.n_last = n_last;
  q.HKV = c->num_kv_heads;
  const int bk = hyq_bits_k(c), bv = hyq_bits_v(c);
  if (bk == 4) return bv == 4 ? launch<4, 4>(q, s) : launch<4, 8>(q, s);
  return bv == 4 ? launch<8, 4>(q, s) : launch<8, 8>(q, s);
}
