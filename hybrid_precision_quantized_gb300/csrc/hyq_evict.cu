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
// Launches: which sequences and how many pages (one block); the kept positions of
// every (layer, sequence, KV head) as a bit mask a page with the number kept before it;
// the free places, a warp a page; the last n_last positions, which may overlap their
// new places and are therefore taken a page after another by one block, and the
// tables; the bound records of the pages that received a row, a warp each.  What bounds it: the
// mass is read once, each moved row read and written once, and of each page that changes
// the keys for its bounds: in part HBM (2.9 TB/s of these bytes for 16 x 4096 in 32
// layers), in part dependent reads (page numbers, masks, rows) and the records'
// arithmetic; small calls are bound by the launches' latencies.
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
  int64_t* cum;     // [batch + 1] kept pages of the rows before
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
  int64_t w = i < p.batch && k >= 0 ? (k + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS : 0, pre = w;
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

// One block per (layer, row, KV head).  The threshold is found a bit at a time by counting the keys at and above a
// candidate: the keys stay in registers (read again for each bit past the first 32768 positions), and counting needs no
// atomics, whose bins the exponents of masses share (a histogram of eight bits at a time, a page a thread: 229 us
// for 4096 selections of 4160 in a cold launch, with this 43; 512 of up to 32512 took 86 and take 99).  Comparisons
// bound it: two bits by three candidates at a time took 474 and 243 us where whole evictions of 16 x 4096 in 32 layers and of
// eight prompts of up to 32768 in eight take 453 and 222.  Many positions receive nothing, and the threshold is among them:
// that is seen after four bits (143 to 45 us for the 4096 selections).
// kSelThreads threads hold kHeld pieces each.  Two sizes, three small blocks or a large one an SM, each for the
// sequences of its size (all in large ones: 975 us instead of 545 for an eviction of 16 x 4096 in
// 32 layers, when it took two bits at a time).
template <int kSelThreads, int kHeld>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const Params p) {
  constexpr int kSelWarps = kSelThreads / 32, kPass = kSelThreads * kPiece;  // positions of a pass
  __shared__ uint32_t s_count[2][kSelWarps], s_scan[2][kSelWarps];
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
  // a block's sum: the warps' sums, which every warp adds up; and that of the warps before `upto`
  auto sums = [&](const uint32_t* s, int upto) {
    const uint32_t x = lane < kSelWarps ? s[lane] : 0u;
    return make_uint2(__reduce_add_sync(0xffffffffu, x), __reduce_add_sync(0xffffffffu, lane < upto ? x : 0u));
  };
  uint32_t key = 0;
  auto reach = [&](uint32_t c, uint32_t* s) {  // how many keys are c or more
    int n = 0;
    auto count = [&](const uint32_t (&x)[kPiece]) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) n += x[i] >= c;
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (k * kPass < hi) count(held[k]);
    for (int pos = kHeld * kPass + kPiece * tid; pos < hi; pos += kPass) {
      uint32_t x[kPiece];
      keys(pos, x);
      count(x);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s[warp] = n;
    __syncthreads();
    return (int)sums(s, 0).x;
  };
  // the want-th largest key: the largest one that at least `want` keys reach
  int above = -1;
#pragma unroll 1
  for (int bit = 31; bit >= 0 && want > 0; --bit) {
    const uint32_t c = key | 1u << bit;
    const int n = reach(c, s_count[bit & 1]);
    if (n >= want) key = c;
    if (n == want) {  // just as many reach the candidate: no need to know the key itself
      key = c - 1;
      break;
    }
    if (bit == 28 && key == 0x80000000u) {  // [0, 2^-95): zeros as a rule, and then no further bit tells more
      const int more = reach(key + 1, s_scan[0]);
      if (more < want) {
        above = more;
        break;
      }
    }
  }
  // the mask: what lies above the key, and the first of those that equal it
  const size_t base = (((size_t)layer * p.batch + b) * p.HKV + h) * p.pages.max_blocks;
  // of those that equal the key, as many are kept as those above it leave
  if (above < 0) above = key == ~0u ? 0 : reach(key + 1, s_scan[0]);
  const int left = max(0, want - above);  // (none wanted: the key is 0)
  int above_before = 0, ties_before = 0, turn = 1;  // in the pieces before
  auto finish = [&](int pos, const uint32_t (&x)[kPiece]) {  // (all threads)
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      gt |= (uint32_t)(want > 0 && x[i] > key) << i;
      eq |= (uint32_t)(want > 0 && x[i] == key && key != 0) << i;
    }
    const int nf = p.n_first - pos;
    if (nf > 0) gt |= nf >= kPiece ? (1u << kPiece) - 1 : (1u << nf) - 1;
    // what the threads before have of both, a half word each (a pass has 2^14 positions at most)
    const uint32_t mine = (uint32_t)__popc(gt) | (uint32_t)__popc(eq) << 16;
    uint32_t pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    uint32_t* s = s_scan[turn];
    turn ^= 1;
    if (lane == 31) s[warp] = pre;
    __syncthreads();
    uint2 both = sums(s, warp);
    both.y += pre - mine;
    const int tie_at = ties_before + (int)(both.y >> 16), room = max(0, left - tie_at);
    const int at = above_before + (int)(both.y & 0xffffu) + min(tie_at, left);
    above_before += (int)(both.x & 0xffffu), ties_before += (int)(both.x >> 16);
    for (int drop = __popc(eq) - room; drop > 0; --drop) eq &= ~(1u << (31 - __clz(eq)));
    const uint32_t m = pos < hi ? gt | eq : 0u;
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
  uint64_t src = 0;  // the tile that the row comes from: all rows' table entries are read at once
  if (lane < 16 && from >= 0) {
    weight = *pl.weight(from);
    src = reinterpret_cast<uint64_t>(pl.tile<BK, BV>(from));
  }
  uint32_t todo = __ballot_sync(0xffffffffu, lane < 16 && from >= 0);
  while (todo) {
    HeldRow<BK, BV> x[kHold];
    int r[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      r[i] = todo ? __ffs(todo) - 1 : -1;
      todo &= todo - 1;
      const int at = r[i] < 0 ? 0 : r[i], row = __shfl_sync(0xffffffffu, from, at) & 15;
      const uint8_t* tile = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, src, at));
      if (r[i] >= 0) x[i].load(tile, row, lane);
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

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A lane's key codes of a 16-row tile, and steps and zeros of rows g and g + 8.
template <int BK>
struct Keys {
  uint4 kc[BK / 2], ka, kb;
};

// One warp: least and largest keys of a page, element by element, as they are held.
template <int BK, int BV>
struct Extremes {
  float lo[32], hi[32];  // of the lane's rows so far: elements 32 v + .. of its eight of each group v
  Keys<BK> next;         // the tile that is on its way

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < 32; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  }
  __device__ __forceinline__ void load(const uint8_t* tile, int lane) {
    using F = QFmt<BK, BV>;
#pragma unroll
    for (int i = 0; i < BK / 2; ++i) next.kc[i] = *reinterpret_cast<const uint4*>(tile + 512 * i + 16 * lane);
    next.ka = *reinterpret_cast<const uint4*>(tile + F::kKMeta + 16 * (lane >> 2));
    next.kb = *reinterpret_cast<const uint4*>(tile + F::kKMeta + 16 * ((lane >> 2) + 8));
  }
  // The tile's rows below vr (kAll: all sixteen).
  template <bool kAll>
  __device__ __forceinline__ void take(const Keys<BK>& k, int lane, int vr) {
    const bool ina = (lane >> 2) < vr, inb = (lane >> 2) + 8 < vr;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      uint32_t xa[4], xb[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (BK == 4) {
          const uint32_t w = u4at(k.kc[v >> 1], 2 * (v & 1) + u), w8 = w >> 8;
          xa[2 * u] = low_codes(w), xa[2 * u + 1] = low_codes(w8);
          xb[2 * u] = high_codes(w), xb[2 * u + 1] = high_codes(w8);
        } else {
          const uint32_t wa = u4at(k.kc[BK == 4 ? 0 : v], 2 * u), wb = u4at(k.kc[BK == 4 ? 0 : v], 2 * u + 1);
          xa[2 * u] = even_codes(wa), xa[2 * u + 1] = odd_codes(wa);
          xb[2 * u] = even_codes(wb), xb[2 * u + 1] = odd_codes(wb);
        }
      }
      auto half = [&](uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(v & 1 ? w >> 16 : w & 0xFFFFu))); };
      const float sa = half(v < 2 ? k.ka.x : k.ka.y), za = half(v < 2 ? k.ka.z : k.ka.w);
      const float sb = half(v < 2 ? k.kb.x : k.kb.y), zb = half(v < 2 ? k.kb.z : k.kb.w);
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

// A kept page of one (layer, row, KV head): item `it` of all.
struct Item {
  Row row;
  int b, layer, h, page;  // call row; page of the sequence
};
__device__ __forceinline__ Item item_of(const Params& p, const int64_t* cum, int64_t it) {
  const int64_t per = (int64_t)p.HKV * p.pages.n_layers, x = it >> 32 ? it / per : (uint32_t)it / (uint32_t)per;
  const int lh = (int)(it - x * per);
  Item r;
  r.layer = lh / p.HKV;
  r.h = lh - r.layer * p.HKV;
  int hi = p.batch;
  r.b = 0;
  while (hi - r.b > 1) {
    const int m = (r.b + hi) >> 1;
    if (cum[m] <= x) r.b = m;
    else hi = m;
  }
  r.row = p.ws.row[r.b];
  r.page = (int)(x - cum[r.b]);
  return r;
}
__device__ __forceinline__ size_t mask_of(const Params& p, const Item& it) {
  return (((size_t)it.layer * p.batch + it.b) * p.HKV + it.h) * p.pages.max_blocks;
}
// Its places below w that are free.
__device__ __forceinline__ uint64_t free_places(const Params& p, const Item& it) {
  const int here = it.row.k - p.n_last - it.page * HYQ_PAGE_ROWS;  // rows below w
  if (here <= 0) return 0;
  return ~p.ws.mask[mask_of(p, it) + it.page] & (here >= 64 ? ~0ull : (1ull << here) - 1);
}

// The free places below w: a warp takes a page.  (Its time is a chain of dependent reads; a block a page, a tile a warp,
// left three of four warps without work where a page has one free place: 385 against 184 us for 16 x 4096 in 32 layers, cold.)
template <int BK, int BV>
__global__ void __launch_bounds__(kMoveThreads) fill_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  constexpr int kWords = F::kTile / 16, kLoads = (kWords + 31) / 32;
  __shared__ __align__(16) uint8_t s_tile[kMoveThreads / 32][F::kTile];
  __shared__ int64_t s_cum[HYQ_PAGED_MAX_BATCH + 1];
  chain_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i <= p.batch; i += kMoveThreads) s_cum[i] = p.ws.cum[i];
  __syncthreads();
  uint8_t* held = s_tile[warp];
  const int64_t items = s_cum[p.batch] * p.HKV * p.pages.n_layers;
  for (int64_t it = (int64_t)blockIdx.x * (kMoveThreads / 32) + warp; it < items; it += (int64_t)gridDim.x * (kMoveThreads / 32)) {
    const Item x = item_of(p, s_cum, it);
    const uint64_t holes = free_places(p, x);
    if (!holes) continue;
    const Place pl = place_of<BK, BV>(p, x.row, x.layer, x.h);
    const size_t base = mask_of(p, x);
    // the r-th free place takes the r-th kept position from w on, the (kw + r)-th of all
    const int w = x.row.k - p.n_last, at = x.page * HYQ_PAGE_ROWS;
    const int nb = (x.row.n - p.n_last + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS, jw = w / HYQ_PAGE_ROWS;
    const uint64_t mw = jw < nb ? p.ws.mask[base + jw] & ((1ull << (w % HYQ_PAGE_ROWS)) - 1) : 0;
    const int rank0 = (jw < nb ? p.ws.before[base + jw] + __popcll(mw) : 0) + at - p.ws.before[base + x.page];
    uint8_t* tile = pl.tile<BK, BV>(at);
#pragma unroll 1
    for (int i = 0; i < 4; ++i, tile += F::kTile) {
      const uint32_t mine = (uint32_t)(holes >> (16 * i)) & 0xFFFFu;
      if (!mine) continue;
      uint4 v[kLoads];  // the tile arrives while its rows' sources are looked for
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        if (32 * k + lane < kWords) v[k] = reinterpret_cast<const uint4*>(tile)[32 * k + lane];
      const int r = 16 * i + lane;
      int from = -1;
      if (lane < 16 && (mine >> lane) & 1) {
        const int rank = rank0 + __popcll(holes & ((1ull << r) - 1));
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
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        if (32 * k + lane < kWords) reinterpret_cast<uint4*>(held)[32 * k + lane] = v[k];
      __syncwarp();
      const float weight = gather_rows<BK, BV>(pl, held, lane, from);
      copy_tile<BK, BV>(tile, held, lane);
      if (from >= 0) *pl.weight(at + r) = weight;
      __syncwarp();
    }
  }
}

// The records of pages that received a row, a warp each: their keys alone, straight into registers, a tile ahead.
template <int BK, int BV>
__global__ void __launch_bounds__(kMoveThreads, 4) record_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  __shared__ int64_t s_cum[HYQ_PAGED_MAX_BATCH + 1];
  chain_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i <= p.batch; i += kMoveThreads) s_cum[i] = p.ws.cum[i];
  __syncthreads();
  const int64_t items = s_cum[p.batch] * p.HKV * p.pages.n_layers;
  for (int64_t it = (int64_t)blockIdx.x * (kMoveThreads / 32) + warp; it < items; it += (int64_t)gridDim.x * (kMoveThreads / 32)) {
    const Item x = item_of(p, s_cum, it);
    const int at = x.page * HYQ_PAGE_ROWS, valid = min(HYQ_PAGE_ROWS, x.row.k - at);
    const bool shifted = p.n_last > 0 && at + HYQ_PAGE_ROWS > x.row.k - p.n_last;
    if (!shifted && !free_places(p, x)) continue;
    const Place pl = place_of<BK, BV>(p, x.row, x.layer, x.h);
    const uint8_t* tile = pl.tile<BK, BV>(at);
    Extremes<BK, BV> e;
    e.reset();
    e.load(tile, lane);
#pragma unroll 1
    for (int i = 0; 16 * i < valid; ++i) {
      Keys<BK> now = e.next;
      if (16 * (i + 1) < valid) e.load(tile + (i + 1) * F::kTile, lane);
      if (valid - 16 * i >= 16) e.template take<true>(now, lane, 16);
      else e.template take<false>(now, lane, valid - 16 * i);
    }
    e.write(pl.bounds + (size_t)pl.table[x.page] * p.HKV * HYQ_BOUND_BYTES, lane);
  }
}

// The last n_last positions: a block takes one (layer, row, KV head), a page at a time.  Then the tables.
template <int BK, int BV>
__global__ void __launch_bounds__(kMoveThreads) shift_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  __shared__ __align__(16) uint8_t s_page[F::kBlock];
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
    e = hyq_launch_chained(select_kernel<1024, 2>, heads, 1024, 0, s, p);
    if (e != cudaSuccess) return e;
  }
  e = hyq_launch_chained(fill_kernel<BK, BV>, dim3(12 * hyq_num_sms()), kMoveThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  e = hyq_launch_chained(shift_kernel<BK, BV>, heads, kMoveThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  return hyq_launch_chained(record_kernel<BK, BV>, dim3(4 * hyq_num_sms()), kMoveThreads, 0, s, p);
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
