// Page tables of the paged cache: taking, sharing, freeing and compacting pages
// (hyq_pages_reserve / _fork / _truncate / _compact).
//
// refs alone say which pages are free (refs = 0), so taking pages is a scan
// for the lowest free ones and freeing is a decrement; nothing else is kept.
// The tables are a few hundred kilobytes: those kernels are bound by latency
// (one block where an order decides, one launch where none does).  The page
// copies that reserve and compact bring with them are bound by HBM: each
// byte of a moved page is read and written once, by a kernel of its own over
// all layers that reads the list of copies from the workspace.
#include "hyq_paged.cuh"

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kScan = 16;  // pages per thread and pass of a scan

// Exclusive prefix of v over the block and the block's total.
struct Scan {
  int before, total;
};
__device__ __forceinline__ Scan block_scan(int v, int* s /* [kWarps] */) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int pre = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = pre;
  __syncthreads();
  int w = s[lane];  // kWarps = 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  const int below = warp ? __shfl_sync(0xffffffffu, w, (warp + 31) & 31) : 0;
  Scan r;
  r.before = below + pre - v;
  r.total = __shfl_sync(0xffffffffu, w, 31);
  return r;
}

// A thread's kScan consecutive refs from page `p0` on (0 past the pool), as a
// mask of the pages in use.
__device__ __forceinline__ uint32_t used_mask(const int32_t* refs, int p0, int n_pages) {
  uint32_t m = 0;
  if (p0 + kScan <= n_pages) {
#pragma unroll
    for (int i = 0; i < kScan / 4; ++i) {
      const int4 r = *reinterpret_cast<const int4*>(refs + p0 + 4 * i);
      m |= (r.x > 0 ? 1u : 0u) << (4 * i) | (r.y > 0 ? 2u : 0u) << (4 * i) | (r.z > 0 ? 4u : 0u) << (4 * i) |
           (r.w > 0 ? 8u : 0u) << (4 * i);
    }
  } else {
    for (int i = 0; i < kScan; ++i)
      if (p0 + i < n_pages && refs[p0 + i] > 0) m |= 1u << i;
  }
  return m;
}

// Workspace of a reserve: the copies, then the pages taken.
struct ReserveWs {
  int32_t* count;  // rows in the copy list (batch, or 0 when the call failed)
  int32_t* src;    // [HYQ_PAGED_MAX_BATCH] page copied for row i, -1 none
  int32_t* dst;
  int32_t* tiles;
  int32_t* take;   // [n_pages]
};
constexpr size_t kReserveHead = 256 + 3 * HYQ_PAGED_MAX_BATCH * 4;
__host__ __device__ __forceinline__ ReserveWs reserve_ws(void* ws) {
  char* w = static_cast<char*>(ws);
  ReserveWs r;
  r.count = reinterpret_cast<int32_t*>(w);
  r.src = reinterpret_cast<int32_t*>(w + 256);
  r.dst = r.src + HYQ_PAGED_MAX_BATCH;
  r.tiles = r.dst + HYQ_PAGED_MAX_BATCH;
  r.take = reinterpret_cast<int32_t*>(w + kReserveHead);
  return r;
}

constexpr int kTakeHeld = 4096;  // pages taken that are listed in shared memory

// One block; thread i handles call row i (batch <= kThreads).
__global__ void __launch_bounds__(kThreads) reserve_kernel(const hyq_pages p, const int32_t* seqs, int batch,
                                                           const int32_t* n_new, ReserveWs ws) {
  static_assert(HYQ_PAGED_MAX_BATCH <= kThreads, "one row per thread");
  __shared__ __align__(16) int s_seq[kThreads], s_last[kThreads];
  __shared__ int s_scan[kWarps], s_take[kTakeHeld];
  __shared__ int s_have[kThreads], s_need[kThreads], s_off[kThreads], s_copy[kThreads];
  chain_kernel();
  const int i = threadIdx.x;
  const bool row = i < batch;
  uint32_t used = used_mask(p.refs, i * kScan, p.n_pages);  // the scan's first pass, under way with the rows
  int err = 0, s = -1, len = 0, n = 0, have = 0, last = -1, old_refs = 0;
  int64_t need64 = 0;
  if (row) {
    s = page_seq(seqs, i, p.n_seqs);
    n = n_new ? n_new[i] : 1;
    if (s < 0 || n < 0) {
      err = HYQ_DEVERR_INDEX;
    } else {
      len = p.lens[s];
      have = (int)(((int64_t)len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS);
      need64 = ((int64_t)len + n + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS;
      if (len < 0 || have > p.max_blocks) {
        err = HYQ_DEVERR_INDEX;
      } else if (need64 > p.max_blocks || need64 - have > p.n_pages) {
        err = HYQ_DEVERR_PAGES;
      } else if (n > 0 && len % HYQ_PAGE_ROWS) {
        last = p.table[(size_t)s * p.max_blocks + have - 1];
        if (last < 0 || last >= p.n_pages) {
          err = HYQ_DEVERR_INDEX;
          last = -1;
        } else {
          old_refs = p.refs[last];
          if (old_refs <= 1) last = -1;  // its own page: written in place
        }
      }
    }
  }
  s_seq[i] = row ? s : -1;
  s_last[i] = last;
  __syncthreads();
  // the same sequence before this row; rows before it that leave the same page
  int rank = 0;
  if (row && s >= 0)
    for (int j = 0; j < i; j += 4) {
      const int4 a = *reinterpret_cast<const int4*>(s_seq + j), b = *reinterpret_cast<const int4*>(s_last + j);
      const int sj[4] = {a.x, a.y, a.z, a.w}, lj[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (j + k < i && sj[k] == s) err |= HYQ_DEVERR_INDEX;
        rank += j + k < i && last >= 0 && lj[k] == last;
      }
    }
  // as if in order: each leaves the page while another still holds it
  const bool copy = last >= 0 && old_refs - rank > 1;
  const int need = (int)need64;
  const int want = row && !err ? (copy ? 1 : 0) + need - have : 0;
  if (err) hyq_set_err(p.err, err);
  bool failed = __syncthreads_or(err);
  if (failed) {
    if (i == 0) *ws.count = 0;
    return;
  }
  const Scan sc = block_scan(want, s_scan);  // below 2^31: at most 1024 rows of at most n_pages each
  // the lowest free pages, listed in shared memory when they fit
  int32_t* take = sc.total <= kTakeHeld ? s_take : ws.take;
  int got = 0;
  for (int base = 0; base < p.n_pages && got < sc.total; base += kThreads * kScan) {
    const int p0 = base + i * kScan;
    const int in = min(max(p.n_pages - p0, 0), kScan);
    if (base > 0) used = used_mask(p.refs, p0, p.n_pages);
    uint32_t f = ~used & ((1u << in) - 1u);
    const Scan fs = block_scan(__popc(f), s_scan);
    int at = got + fs.before;
    for (; f && at < sc.total; f &= f - 1, ++at) take[at] = p0 + __ffs(f) - 1;
    got += fs.total;
  }
  failed = got < sc.total;
  s_have[i] = have;
  s_need[i] = row ? need : 0;
  s_off[i] = sc.before;
  s_copy[i] = copy;
  __syncthreads();  // the list and the rows are complete
  if (failed) {
    if (i == 0) {
      *ws.count = 0;
      hyq_set_err(p.err, HYQ_DEVERR_PAGES);
    }
    return;
  }
  if (i == 0) *ws.count = batch;
  if (row) {
    int32_t* table = p.table + (size_t)s * p.max_blocks;
    if (copy) {
      const int to = take[sc.before];
      ws.src[i] = last;
      ws.dst[i] = to;
      ws.tiles[i] = (len % HYQ_PAGE_ROWS + 15) / 16;
      table[have - 1] = to;
      p.refs[to] = 1;
      atomicSub(p.refs + last, 1);
    } else {
      ws.src[i] = -1;
    }
    p.lens[s] = len + n;
  }
  // the new pages of each row, a warp per row
  const int warp = i >> 5, lane = i & 31;
  for (int r = warp; r < batch; r += kWarps) {
    const int from = s_off[r] + s_copy[r], cnt = s_need[r] - s_have[r];
    int32_t* table = p.table + (size_t)s_seq[r] * p.max_blocks + s_have[r];
    for (int k = lane; k < cnt; k += 32) {
      const int to = take[from + k];
      table[k] = to;
      p.refs[to] = 1;
    }
  }
}

constexpr int kCopyThreads = 128;

// One block: `bytes` of a page's block for one KV head and layer (a multiple of
// 16) and its bound record, all loads of a thread ahead of its stores: a whole
// block of any code width is at most kDeep loads a thread.
constexpr int kDeep = 9;
static_assert(HYQ_QBLOCK_BYTES_BITS(8, 8) <= kDeep * 16 * kCopyThreads, "a block in one go");
static_assert(HYQ_BOUND_BYTES / 16 <= kCopyThreads, "a record in one go");
__device__ __forceinline__ void copy_block(uint8_t* dst, const uint8_t* src, int bytes, uint8_t* rec_dst,
                                           const uint8_t* rec_src) {
  const uint4* a = reinterpret_cast<const uint4*>(src);
  uint4* b = reinterpret_cast<uint4*>(dst);
  const int n = bytes / 16, i = threadIdx.x;
  uint4 v[kDeep], r;
#pragma unroll
  for (int k = 0; k < kDeep; ++k)
    if (i + k * kCopyThreads < n) v[k] = __ldcs(a + i + k * kCopyThreads);
  if (i < HYQ_BOUND_BYTES / 16) r = *(reinterpret_cast<const uint4*>(rec_src) + i);
#pragma unroll
  for (int k = 0; k < kDeep; ++k)
    if (i + k * kCopyThreads < n) b[i + k * kCopyThreads] = v[k];
  if (i < HYQ_BOUND_BYTES / 16) *(reinterpret_cast<uint4*>(rec_dst) + i) = r;
}
// a / b and the remainder, in 32 bits when they fit.
__device__ __forceinline__ int split(int64_t a, int b, int* rest) {
  const int q = a >> 32 ? (int)(a / b) : (int)((uint32_t)a / (uint32_t)b);
  *rest = (int)(a - (int64_t)q * b);
  return q;
}

// The copies of a reserve: an item is one (row, layer, KV head).
__global__ void __launch_bounds__(kCopyThreads) reserve_copy_kernel(const hyq_pages p, ReserveWs ws, int HKV,
                                                                    int block_bytes) {
  chain_kernel();
  const int n = *ws.count, per = p.n_layers * HKV;
  const int64_t items = (int64_t)n * per;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    int x;
    const int row = split(it, per, &x), layer = x / HKV, h = x - layer * HKV;
    const int src = ws.src[row];
    if (src < 0) continue;
    const size_t a = ((size_t)layer * p.n_pages + src) * HKV + h, b = ((size_t)layer * p.n_pages + ws.dst[row]) * HKV + h;
    copy_block(p.pool + b * block_bytes, p.pool + a * block_bytes, ws.tiles[row] * (block_bytes / 4),
               p.bounds + b * HYQ_BOUND_BYTES, p.bounds + a * HYQ_BOUND_BYTES);
  }
}

constexpr int kRowThreads = 128;

// One block per pair.
__global__ void __launch_bounds__(kRowThreads) fork_kernel(const hyq_pages p, const int32_t* src, const int32_t* dst,
                                                           int n) {
  chain_kernel();
  const int i = blockIdx.x, s = src[i], d = dst[i];
  bool bad = s < 0 || s >= p.n_seqs || d < 0 || d >= p.n_seqs;
  for (int j = threadIdx.x; j < n; j += kRowThreads) bad |= (j < i && dst[j] == d) || src[j] == d;
  bad = __syncthreads_or(bad);
  // A destination is written by its own pair alone and is no pair's source,
  // so these reads meet no other block's writes.
  int len = 0, held = 0;
  if (!bad) {
    len = p.lens[s];
    held = p.lens[d];
    bad = held != 0 || len < 0 || (int64_t)len > (int64_t)p.max_blocks * HYQ_PAGE_ROWS;
  }
  __syncthreads();  // every thread has read the lengths
  if (bad) {
    if (threadIdx.x == 0) hyq_set_err(p.err, HYQ_DEVERR_INDEX);
    return;
  }
  const int nb = (len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS;
  const int32_t* from = p.table + (size_t)s * p.max_blocks;
  int32_t* to = p.table + (size_t)d * p.max_blocks;
  for (int j = threadIdx.x; j < nb; j += kRowThreads) {
    const int page = from[j];
    to[j] = page;
    if (page >= 0 && page < p.n_pages) atomicAdd(p.refs + page, 1);
    else hyq_set_err(p.err, HYQ_DEVERR_INDEX);
  }
  if (threadIdx.x == 0) p.lens[d] = len;
}

// One block per sequence.
__global__ void __launch_bounds__(kRowThreads) truncate_kernel(const hyq_pages p, const int32_t* seqs,
                                                               const int32_t* new_lens, int n) {
  chain_kernel();
  const int i = blockIdx.x, s = seqs ? seqs[i] : i;
  bool bad = s < 0 || s >= p.n_seqs;
  if (seqs)
    for (int j = threadIdx.x; j < i; j += kRowThreads) bad |= seqs[j] == s;
  bad = __syncthreads_or(bad);
  const int to = new_lens ? new_lens[i] : 0;
  int len = 0;
  if (!bad) {
    len = p.lens[s];
    bad = to < 0 || to > len || (int64_t)len > (int64_t)p.max_blocks * HYQ_PAGE_ROWS;
  }
  __syncthreads();  // every thread has read the length
  if (bad) {
    if (threadIdx.x == 0) hyq_set_err(p.err, HYQ_DEVERR_INDEX);
    return;
  }
  const int b0 = (to + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS, b1 = (len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS;
  const int32_t* row = p.table + (size_t)s * p.max_blocks;
  for (int j = b0 + threadIdx.x; j < b1; j += kRowThreads) {
    const int page = row[j];
    if (page >= 0 && page < p.n_pages) atomicSub(p.refs + page, 1);
    else hyq_set_err(p.err, HYQ_DEVERR_INDEX);
  }
  if (threadIdx.x == 0) p.lens[s] = to;
}

// Workspace of a compaction.
struct CompactWs {
  int32_t* count;  // moves
  int32_t* src;    // [n_pages] pages at or past N in use, ascending
  int32_t* dst;    // [n_pages] free pages below N, ascending
  int32_t* map;    // [n_pages] new place of a page in use
};
CompactWs compact_ws(void* ws, int n_pages) {
  char* w = static_cast<char*>(ws);
  CompactWs r;
  r.count = reinterpret_cast<int32_t*>(w);
  r.src = reinterpret_cast<int32_t*>(w + 256);
  r.dst = r.src + n_pages;
  r.map = r.dst + n_pages;
  return r;
}

// One block: the number of pages in use N, the two lists, the map and the new refs.
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const hyq_pages p, int32_t* refs_out, CompactWs ws) {
  __shared__ int s_scan[kWarps];
  chain_kernel();
  const int tid = threadIdx.x, np = p.n_pages;
  constexpr int kPass = kThreads * kScan;
  int mine = 0;
  for (int base = 0; base < np; base += kPass) mine += __popc(used_mask(p.refs, base + tid * kScan, np));
  const int N = block_scan(mine, s_scan).total;
  int highs = 0, gaps = 0;
  for (int base = 0; base < np; base += kPass) {
    const int p0 = base + tid * kScan;
    const uint32_t used = used_mask(p.refs, p0, np);
    const int in = min(max(N - p0, 0), kScan);  // pages of this thread below N
    const uint32_t below = (1u << in) - 1u;
    uint32_t hi = used & ~below, gap = ~used & below;
    const Scan sh = block_scan(__popc(hi) | __popc(gap) << 16, s_scan);  // at most 2^14 each a pass
    int ah = highs + (sh.before & 0xFFFF), ag = gaps + (sh.before >> 16);
    for (; hi; hi &= hi - 1) ws.src[ah++] = p0 + __ffs(hi) - 1;
    for (; gap; gap &= gap - 1) ws.dst[ag++] = p0 + __ffs(gap) - 1;
    highs += sh.total & 0xFFFF;
    gaps += sh.total >> 16;
    for (int i = 0; i < kScan && p0 + i < np; ++i) {
      ws.map[p0 + i] = p0 + i;
      if (refs_out != p.refs && p0 + i < N) refs_out[p0 + i] = p.refs[p0 + i];
    }
  }
  if (tid == 0) *ws.count = highs;
  __syncthreads();  // the lists are complete
  for (int r = tid; r < highs; r += kThreads) {
    const int from = ws.src[r], to = ws.dst[r];
    ws.map[from] = to;
    refs_out[to] = p.refs[from];
  }
  __syncthreads();  // refs past N are read
  for (int q = N + tid; q < np; q += kThreads) refs_out[q] = 0;
}

// The table through the map, and the pages: an item is one (move, layer, KV head).
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const hyq_pages p, int32_t* table_out,
                                                                    CompactWs ws, int HKV, int block_bytes) {
  chain_kernel();
  const int64_t entries = (int64_t)p.n_seqs * p.max_blocks;
  for (int64_t x = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; x < entries;
       x += (int64_t)gridDim.x * kCopyThreads) {
    const int s = (int)(x / p.max_blocks), j = (int)(x - (int64_t)s * p.max_blocks);
    int page = p.table[x];
    if ((int64_t)j * HYQ_PAGE_ROWS < p.lens[s]) {
      if (page >= 0 && page < p.n_pages) page = ws.map[page];
      else hyq_set_err(p.err, HYQ_DEVERR_INDEX);
    }
    table_out[x] = page;
  }
  const int n = *ws.count, per = p.n_layers * HKV;
  const int64_t items = (int64_t)n * per;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    int x;
    const int m = split(it, per, &x), layer = x / HKV, h = x - layer * HKV;
    const size_t a = ((size_t)layer * p.n_pages + ws.src[m]) * HKV + h,
                 b = ((size_t)layer * p.n_pages + ws.dst[m]) * HKV + h;
    copy_block(p.pool + b * block_bytes, p.pool + a * block_bytes, block_bytes, p.bounds + b * HYQ_BOUND_BYTES,
               p.bounds + a * HYQ_BOUND_BYTES);
  }
}

int copy_grid(int64_t items) {
  const int64_t most = 12ll * hyq_num_sms();
  return (int)(items < 1 ? 1 : items < most ? items : most);
}

}  // namespace

size_t hyq_pages_reserve_ws_bytes(const hyq_pages* p) {
  return hyq_align256(kReserveHead) + hyq_align256((size_t)p->n_pages * 4);
}

cudaError_t hyq_launch_pages_reserve(const hyq_config* c, const hyq_pages* p, const int32_t* seqs, int32_t batch,
                                     const int32_t* n_new, void* ws, cudaStream_t s) {
  const ReserveWs w = reserve_ws(ws);
  cudaError_t e = hyq_launch_chained(reserve_kernel, dim3(1), kThreads, 0, s, *p, seqs, (int)batch, n_new, w);
  if (e != cudaSuccess) return e;
  return hyq_launch_chained(reserve_copy_kernel, dim3(copy_grid((int64_t)batch * p->n_layers * c->num_kv_heads)),
                            kCopyThreads, 0, s, *p, w, (int)c->num_kv_heads, (int)hyq_qblock_bytes(c));
}

cudaError_t hyq_launch_pages_fork(const hyq_pages* p, const int32_t* src, const int32_t* dst, int32_t n,
                                  cudaStream_t s) {
  return hyq_launch_chained(fork_kernel, dim3(n), kRowThreads, 0, s, *p, src, dst, (int)n);
}

cudaError_t hyq_launch_pages_truncate(const hyq_pages* p, const int32_t* seqs, const int32_t* new_lens, int32_t n,
                                      cudaStream_t s) {
  return hyq_launch_chained(truncate_kernel, dim3(n), kRowThreads, 0, s, *p, seqs, new_lens, (int)n);
}

size_t hyq_pages_compact_ws_bytes(const hyq_pages* p) { return 256 + hyq_align256((size_t)p->n_pages * 3 * 4); }

cudaError_t hyq_launch_pages_compact(const hyq_config* c, const hyq_pages* p, int32_t* table_out, int32_t* refs_out,
                                     void* ws, cudaStream_t s) {
  const CompactWs w = compact_ws(ws, p->n_pages);
  cudaError_t e = hyq_launch_chained(compact_plan_kernel, dim3(1), kThreads, 0, s, *p, refs_out ? refs_out : p->refs, w);
  if (e != cudaSuccess) return e;
  const int64_t half = ((int64_t)p->n_pages / 2 + 1) * p->n_layers * c->num_kv_heads;  // moves are at most n_pages / 2
  return hyq_launch_chained(compact_move_kernel, dim3(copy_grid(half)), kCopyThreads, 0, s, *p,
                            table_out ? table_out : p->table, w, (int)c->num_kv_heads, (int)hyq_qblock_bytes(c));
}
