// Quantised rows into the pages of their sequences (hyq_paged_append), with the
// bound records of the keys.
//
// Per group of 32 elements of a row (Quant_B of Algorithm 4): s the smallest
// FP16 value with qmax s >= max - min, z = FP16(min), codes nearest to
// (x - z) / s, decided exactly (hyq_qcode.cuh).  Reads 512 bytes per (row, KV
// head), writes 160 (4-bit codes), and 512 more with the dequantised rows.
//
// One block per (page that gets rows, KV head), one warp per (16-row tile, K
// or V): a lane holds the four elements of a row that share a code word, so a
// tile's words are assembled in registers, without shared memory.  Steps and
// zeros take a division each: eight rows are reduced together, the halves
// exchanged so that each of a group's eight lanes ends with one row's
// (min, max) (7 exchanges for 8 rows instead of 24) and derives that row's
// step, once per (row, group) instead of once per lane.
#include "hyq_paged.cuh"
#include "hyq_qcode.cuh"

namespace {

struct AppendParams {
  PageView pv;
  const int32_t* seqs;
  const int32_t* cu;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* k_hat;
  __nv_bfloat16* v_hat;
  int64_t ld;
  int32_t batch, n_rows, HKV;
};

// The rows that one page gets: rows [r0, r1) of the page, from row tok0 of
// the call's rows on.
struct PageRows {
  int page, r0, r1, tok0;
};

// First position and number of rows of call row i; n = 0 when there is
// nothing to write or the row must be left out (bad: for a reason to report).
struct CallRows {
  int seq, start, n, tok;
  bool bad;
};
__device__ __forceinline__ CallRows call_rows(const AppendParams& p, int i) {
  CallRows c;
  c.tok = p.cu ? __ldg(p.cu + i) : i;
  const int end = p.cu ? __ldg(p.cu + i + 1) : i + 1;
  c.n = end - c.tok;
  c.seq = page_seq(p.seqs, i, p.pv.n_seqs);
  c.start = 0;
  c.bad = c.seq < 0 || c.tok < 0 || end < c.tok || end > p.n_rows;
  if (!c.bad) {
    const int len = p.pv.lens[c.seq];
    c.start = len - c.n;
    c.bad = c.start < 0 || len < 0 || (int64_t)len > (int64_t)p.pv.max_blocks * HYQ_PAGE_ROWS;
  }
  if (c.bad) c.n = 0;
  return c;
}
__device__ __forceinline__ PageRows page_rows(const AppendParams& p, const CallRows& c, int nth) {
  const int blk = c.start / HYQ_PAGE_ROWS + nth, p0 = blk * HYQ_PAGE_ROWS;
  PageRows r;
  r.page = p.pv.table[(size_t)c.seq * p.pv.max_blocks + blk];
  r.r0 = max(0, c.start - p0);
  r.r1 = min(HYQ_PAGE_ROWS, c.start + c.n - p0);
  r.tok0 = c.tok + (p0 + r.r0 - c.start);
  if (r.page < 0 || r.page >= p.pv.n_pages) {
    hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
    r.r1 = r.r0;
  }
  return r;
}

// First of the four elements of a row that lane `lane` holds: the ones whose
// codes lie in one 32-bit word (K, 4-bit) or simply 4 lane .. 4 lane + 3.
// Group lane / 8 in both.
template <int T, int BITS>
__device__ __forceinline__ int first_element(int lane) {
  return T == 0 && BITS == 4 ? 8 * (lane & 3) + 32 * (lane >> 3) + 4 * ((lane >> 2) & 1) : 4 * lane;
}

__device__ __forceinline__ uint32_t u32_of(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __nv_bfloat162 bf2_of(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }

// (min, -max) of a lane's four elements, NaN if one is.
__device__ __forceinline__ uint32_t min_negmax(uint2 v) {
  const __nv_bfloat162 a = bf2_of(v.x), b = bf2_of(v.y);
  const __nv_bfloat162 mn = __hmin2_nan(a, b), mx = __hmax2_nan(a, b);
  const __nv_bfloat16 lo = __hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn));
  const __nv_bfloat16 hi = __hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx));
  return u32_of(__halves2bfloat162(lo, __hneg(hi)));
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) { return u32_of(__hmin2_nan(bf2_of(a), bf2_of(b))); }

// Step, zero and reciprocal of a group from (min, -max).  r = -1 marks a group
// that FP16 metadata cannot hold (or a NaN): codes, step and zero become 0.
struct GroupQ {
  uint32_t sz;  // FP16 step | zero << 16
  float r;
};
__device__ __forceinline__ GroupQ group_q(uint32_t mm, float qmax) {
  const float2 m = __bfloat1622float2(bf2_of(mm));
  const float mn = m.x, mx = -m.y;
  const __half sh = group_step(mn, mx, qmax), zh = __float2half_rn(mn);
  const float s = __half2float(sh), z = __half2float(zh);
  GroupQ o;
  if (isnan(m.x) || isnan(m.y) || isinf(s) || isinf(z)) {
    o.sz = 0u;
    o.r = -1.f;
  } else {
    o.sz = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(zh) << 16);
    o.r = s > 0.f ? __frcp_rn(s) : 0.f;
  }
  return o;
}

// Codes of a lane's four elements.  x becomes zeros when the group is marked.
__device__ __forceinline__ void codes4(uint2& v, uint32_t sz, float r, float qmax, float& s, float& z,
                                       uint32_t (&c)[4]) {
  if (r < 0.f) {
    v = make_uint2(0u, 0u);
    r = 0.f;
  }
  const float2 f = half2_to_float2(sz);
  s = f.x;
  z = f.y;
  const float2 a = __bfloat1622float2(bf2_of(v.x)), b = __bfloat1622float2(bf2_of(v.y));
  c[0] = code_of(a.x, z, r, s, qmax);
  c[1] = code_of(a.y, z, r, s, qmax);
  c[2] = code_of(b.x, z, r, s, qmax);
  c[3] = code_of(b.y, z, r, s, qmax);
}

// Metadata of (row r of the tile, group q).
template <int T>
__device__ __forceinline__ void store_meta(uint8_t* meta, int r, int q, uint32_t sz) {
  const int so = T == 0 ? 16 * r + 2 * q : 16 * (r >> 1) + 4 * q + 2 * (r & 1);
  *reinterpret_cast<uint16_t*>(meta + so) = (uint16_t)sz;
  *reinterpret_cast<uint16_t*>(meta + so + (T == 0 ? 8 : 128)) = (uint16_t)(sz >> 16);
}

__device__ __forceinline__ void store_hat(__nv_bfloat16* hat, const uint32_t (&c)[4], float s, float z) {
  const uint32_t lo = pack_bf16x2(fmaf((float)c[0], s, z), fmaf((float)c[1], s, z));
  const uint32_t hi = pack_bf16x2(fmaf((float)c[2], s, z), fmaf((float)c[3], s, z));
  *reinterpret_cast<uint2*>(hat) = make_uint2(lo, hi);
}

// Running bounds of a lane's four key elements (BF16 pairs).
struct Bounds4 {
  __nv_bfloat162 mn[2], mx[2];
};

// Rows `nm` (bits 0..15) of one tile, tensor T (0 = K, 1 = V): row i comes
// from src + i ld.  bnd: bounds of the rows taken (K).
template <int T, int BITS, int kTile, int kCode, int kMeta>
__device__ void tile_rows(uint8_t* tile, const __nv_bfloat16* src, int64_t ld, __nv_bfloat16* hat, int64_t ldh,
                          uint32_t nm, int lane, Bounds4& bnd, int32_t* err) {
  constexpr float qmax = BITS == 8 ? 255.f : 15.f;
  constexpr int kWords = T == 0 ? (BITS == 4 ? 8 : 1) : (BITS == 4 ? 8 : 16);
  const int e0 = first_element<T, BITS>(lane), q = lane >> 3, i8 = lane & 7;
  uint32_t w[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) w[k] = 0u;
  bool bad = false;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t hm = (nm >> (8 * half)) & 0xFFu;
    if (hm == 0) continue;
    uint2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = (hm >> i) & 1 ? __ldg(reinterpret_cast<const uint2*>(src + (8 * half + i) * ld + e0)) : make_uint2(0u, 0u);
    // eight rows' (min, -max): lane i8 of a group ends with row i8's
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = min_negmax(v[i]);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) {
      const bool up = i8 & o;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const uint32_t keep = up ? m[i + o] : m[i], give = up ? m[i] : m[i + o];
        m[i] = min2(keep, __shfl_xor_sync(0xffffffffu, give, o));
      }
    }
    const GroupQ gq = group_q(m[0], qmax);
    const bool mine = (hm >> i8) & 1;
    bad |= mine && gq.r < 0.f;
    if (mine) store_meta<T>(tile + kMeta, 8 * half + i8, q, gq.sz);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t sz = __shfl_sync(0xffffffffu, gq.sz, (lane & 24) | i);
      const float r = __shfl_sync(0xffffffffu, gq.r, (lane & 24) | i);
      if (!((hm >> i) & 1)) continue;  // the same for the whole warp
      float s, z;
      uint32_t c[4];
      codes4(v[i], sz, r, qmax, s, z, c);
      if (T == 0) {
        bnd.mn[0] = __hmin2(bnd.mn[0], bf2_of(v[i].x));
        bnd.mn[1] = __hmin2(bnd.mn[1], bf2_of(v[i].y));
        bnd.mx[0] = __hmax2(bnd.mx[0], bf2_of(v[i].x));
        bnd.mx[1] = __hmax2(bnd.mx[1], bf2_of(v[i].y));
      }
      if (hat) store_hat(hat + (8 * half + i) * ldh + e0, c, s, z);
      if (T == 0) {  // bytes: elements 0, 2, 1, 3
        const uint32_t word = c[0] | (c[2] << 8) | (c[1] << 16) | (c[3] << 24);
        if (BITS == 4)
          w[i % kWords] |= word << (4 * half);  // row i + 8 in the high nibbles of row i's word
        else
          *reinterpret_cast<uint32_t*>(tile + kCode + 512 * (lane >> 3) + 16 * (4 * i + (lane & 3)) +
                                       4 * (2 * ((lane >> 2) & 1) + half)) = word;
      } else if (BITS == 4) {  // row 2t + 8b + c: byte b + 2c of the words of t
        const int sh = 8 * (half + 2 * (i & 1));
        w[(2 * (i >> 1)) % kWords] |= (c[0] | (c[1] << 4)) << sh;
        w[(2 * (i >> 1) + 1) % kWords] |= (c[2] | (c[3] << 4)) << sh;
      } else {
        const int sh = 8 * (half + 2 * (i & 1));
#pragma unroll
        for (int k = 0; k < 4; ++k) w[(4 * (i >> 1) + k) % kWords] |= c[k] << sh;
      }
    }
  }
  if (T == 0 && BITS == 4) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(tile + kCode + 512 * (lane >> 4) + 16 * (4 * g + (lane & 3)) +
                                                  4 * ((lane >> 2) & 3));
      const uint32_t mask = ((nm >> g) & 1 ? 0x0F0F0F0Fu : 0u) | ((nm >> (g + 8)) & 1 ? 0xF0F0F0F0u : 0u);
      if (mask == 0u) continue;
      *dst = mask == 0xFFFFFFFFu ? w[g % kWords] : (*dst & ~mask) | w[g % kWords];
    }
  } else if (T == 1) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t mask = 0u;  // bytes b + 2c: rows 2t, 2t + 8, 2t + 1, 2t + 9
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((nm >> (2 * t + 8 * (j & 1) + (j >> 1))) & 1) mask |= 0xFFu << (8 * j);
      if (mask == 0u) continue;
      const int at = 16 * (4 * (lane & 7) + t);
      if (BITS == 4) {
        uint2* dst = reinterpret_cast<uint2*>(tile + kCode + 512 * (q >> 1) + at + 8 * (q & 1));
        uint2 x = make_uint2(w[(2 * t) % kWords], w[(2 * t + 1) % kWords]);
        if (mask != 0xFFFFFFFFu) {
          const uint2 old = *dst;
          x.x |= old.x & ~mask;
          x.y |= old.y & ~mask;
        }
        *dst = x;
      } else {
        uint4* dst = reinterpret_cast<uint4*>(tile + kCode + 512 * q + at);
        uint4 x = make_uint4(w[(4 * t) % kWords], w[(4 * t + 1) % kWords], w[(4 * t + 2) % kWords],
                             w[(4 * t + 3) % kWords]);
        if (mask != 0xFFFFFFFFu) {
          const uint4 old = *dst;
          x.x |= old.x & ~mask;
          x.y |= old.y & ~mask;
          x.z |= old.z & ~mask;
          x.w |= old.w & ~mask;
        }
        *dst = x;
      }
    }
  }
  if (bad) hyq_set_err(err, HYQ_DEVERR_QUANT_RANGE);
}

// One warp: the bound record of one (page, KV head) from the min / max of four
// elements per lane, joined with the present record unless `fresh`.  Codes at
// a coarser step follow from those at a finer one by an outward shift.
__device__ __forceinline__ void store_bounds(uint8_t* rec, int e0, const Bounds4& b, bool fresh) {
  float mn[4], mx[4], am = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = __bfloat1622float2(b.mn[i]), c = __bfloat1622float2(b.mx[i]);
    mn[2 * i] = a.x, mn[2 * i + 1] = a.y, mx[2 * i] = c.x, mx[2 * i + 1] = c.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) am = fmaxf(am, fmaxf(fabsf(mn[i]), fabsf(mx[i])));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  int e = bound_exp(am), oe = 0;
  uint32_t ol = 0u, oh = 0u;
  if (!fresh) {
    oe = *reinterpret_cast<const int32_t*>(rec + 256);
    ol = *reinterpret_cast<const uint32_t*>(rec + e0);
    oh = *reinterpret_cast<const uint32_t*>(rec + 128 + e0);
    e = max(e, oe);
  }
  __syncwarp();
  const float inv = ldexpf(1.f, -e);
  const int sh = min(max(e - oe, 0), 31);
  uint32_t l = 0u, h = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int lo = (int)floorf(mn[i] * inv), hi = (int)ceilf(mx[i] * inv);
    if (!fresh) {
      lo = min(lo, (int)(int8_t)(ol >> (8 * i)) >> sh);
      hi = max(hi, -(-(int)(int8_t)(oh >> (8 * i)) >> sh));
    }
    l |= ((uint32_t)lo & 0xFFu) << (8 * i);
    h |= ((uint32_t)hi & 0xFFu) << (8 * i);
  }
  *reinterpret_cast<uint32_t*>(rec + e0) = l;
  *reinterpret_cast<uint32_t*>(rec + 128 + e0) = h;
  if ((threadIdx.x & 31) == 0) *reinterpret_cast<int4*>(rec + 256) = make_int4(e, 0, 0, 0);
}

constexpr int kThreads = 256;  // 4 tiles x {K, V}

// grid (pages that the call may reach, KV heads' share): block x takes the
// x-th page that gets rows, in the order of the call's rows.
template <int BK, int BV>
__global__ void __launch_bounds__(kThreads) append_pages_kernel(const AppendParams p) {
  using F = QFmt<BK, BV>;
  __shared__ int s_warp[kThreads / 32];
  __shared__ PageRows s_rows;
  __shared__ bool s_found;
  __shared__ Bounds4 s_b[4][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // pages of the call rows 4 tid .. 4 tid + 3, summed up
  CallRows c[4];
  int n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = 0;
    if (4 * tid + i < p.batch) {
      c[i] = call_rows(p, 4 * tid + i);
      if (c[i].bad && blockIdx.x == 0 && blockIdx.y == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
      if (c[i].n > 0) n[i] = (c[i].start + c[i].n - 1) / HYQ_PAGE_ROWS - c[i].start / HYQ_PAGE_ROWS + 1;
    }
    sum += n[i];
  }
  int pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += y;
  }
  if (lane == 31) s_warp[warp] = pre;
  if (tid == 0) s_found = false;
  __syncthreads();
  int at = pre - sum;
  for (int i = 0; i < warp; ++i) at += s_warp[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int nth = (int)blockIdx.x - at;
    if (nth >= 0 && nth < n[i]) {
      s_rows = page_rows(p, c[i], nth);
      s_found = true;
    }
    at += n[i];
  }
  __syncthreads();
  if (!s_found) return;
  const PageRows r = s_rows;
  if (r.r1 <= r.r0) return;
  const int tile = warp & 3, T = warp >> 2;
  // rows of this tile: bits of [r0, r1) in [16 tile, 16 tile + 16)
  const int a = min(max(r.r0 - 16 * tile, 0), 16), z = min(max(r.r1 - 16 * tile, 0), 16);
  const uint32_t nm = ((1u << z) - 1u) & ~((1u << a) - 1u);
  const int64_t row0 = (int64_t)r.tok0 + 16 * tile - r.r0;  // call row of the tile's row 0 (may lie before tok0)
  for (int h = blockIdx.y; h < p.HKV; h += gridDim.y) {
    const size_t ph = (size_t)r.page * p.HKV + h;
    uint8_t* tp = p.pv.pool + ph * F::kBlock + tile * F::kTile;
    const int64_t ldh = (int64_t)p.HKV * HYQ_D;
    Bounds4 b;
    b.mn[0] = b.mn[1] = __floats2bfloat162_rn(INFINITY, INFINITY);
    b.mx[0] = b.mx[1] = __floats2bfloat162_rn(-INFINITY, -INFINITY);
    if (nm) {
      if (T == 0)
        tile_rows<0, BK, F::kTile, 0, F::kKMeta>(tp, p.k + row0 * p.ld + (int64_t)h * HYQ_D, p.ld,
                                                 p.k_hat ? p.k_hat + row0 * ldh + (int64_t)h * HYQ_D : nullptr, ldh,
                                                 nm, lane, b, p.pv.err);
      else
        tile_rows<1, BV, F::kTile, F::kVCode, F::kVMeta>(
            tp, p.v + row0 * p.ld + (int64_t)h * HYQ_D, p.ld,
            p.v_hat ? p.v_hat + row0 * ldh + (int64_t)h * HYQ_D : nullptr, ldh, nm, lane, b, p.pv.err);
    }
    if (T == 0) s_b[tile][lane] = b;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 1; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          b.mn[j] = __hmin2(b.mn[j], s_b[i][lane].mn[j]);
          b.mx[j] = __hmax2(b.mx[j], s_b[i][lane].mx[j]);
        }
      store_bounds(p.pv.bounds + ph * HYQ_BOUND_BYTES, first_element<0, BK>(lane), b, r.r0 == 0);
    }
    __syncthreads();
  }
}

// One row per sequence: grid (batch, HKV), warp 0 the key, warp 1 the value.
template <int BK, int BV>
__global__ void __launch_bounds__(64) append_one_kernel(const AppendParams p) {
  using F = QFmt<BK, BV>;
  const int h = blockIdx.y, T = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CallRows c = call_rows(p, blockIdx.x);
  if (c.bad && threadIdx.x == 0 && h == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
  if (c.n <= 0) return;
  const PageRows r = page_rows(p, c, 0);
  if (r.r1 <= r.r0) return;
  const size_t ph = (size_t)r.page * p.HKV + h;
  const int row = r.r0 & 15, q = lane >> 3;
  const float qmax = (T == 0 ? BK : BV) == 8 ? 255.f : 15.f;
  const int e0 = T == 0 ? first_element<0, BK>(lane) : first_element<1, BV>(lane);
  uint8_t* tile = p.pv.pool + ph * F::kBlock + (r.r0 >> 4) * F::kTile;
  uint2 v = __ldg(reinterpret_cast<const uint2*>((T == 0 ? p.k : p.v) + (int64_t)r.tok0 * p.ld + (int64_t)h * HYQ_D + e0));
  uint32_t m = min_negmax(v);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = min2(m, __shfl_xor_sync(0xffffffffu, m, o));
  const GroupQ gq = group_q(m, qmax);
  if (gq.r < 0.f) hyq_set_err(p.pv.err, HYQ_DEVERR_QUANT_RANGE);
  float s, z;
  uint32_t cd[4];
  codes4(v, gq.sz, gq.r, qmax, s, z, cd);
  __nv_bfloat16* hat = T == 0 ? p.k_hat : p.v_hat;
  if (hat) store_hat(hat + ((int64_t)r.tok0 * p.HKV + h) * HYQ_D + e0, cd, s, z);
  if (T == 0) {
    if ((lane & 7) == 0) store_meta<0>(tile + F::kKMeta, row, q, gq.sz);
    const uint32_t word = cd[0] | (cd[2] << 8) | (cd[1] << 16) | (cd[3] << 24);
    const int g = row & 7, half = row >> 3;
    if (BK == 4) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(tile + 512 * (lane >> 4) + 16 * (4 * g + (lane & 3)) + 4 * ((lane >> 2) & 3));
      *dst = (*dst & ~(0x0F0F0F0Fu << (4 * half))) | (word << (4 * half));
    } else {
      *reinterpret_cast<uint32_t*>(tile + 512 * (lane >> 3) + 16 * (4 * g + (lane & 3)) +
                                   4 * (2 * ((lane >> 2) & 1) + half)) = word;
    }
    Bounds4 b;
    b.mn[0] = b.mx[0] = bf2_of(v.x);
    b.mn[1] = b.mx[1] = bf2_of(v.y);
    store_bounds(p.pv.bounds + ph * HYQ_BOUND_BYTES, e0, b, r.r0 == 0);
  } else {
    if ((lane & 7) == 0) store_meta<1>(tile + F::kVMeta, row, q, gq.sz);
    const int t = (row & 7) >> 1, j = (row >> 3) + 2 * (row & 1);
    uint8_t* at = tile + F::kVCode + 16 * (4 * (lane & 7) + t) + j;
    if (BV == 4) {
      at += 512 * (q >> 1) + 8 * (q & 1);
      at[0] = (uint8_t)(cd[0] | (cd[1] << 4));
      at[4] = (uint8_t)(cd[2] | (cd[3] << 4));
    } else {
      at += 512 * q;
#pragma unroll
      for (int k = 0; k < 4; ++k) at[4 * k] = (uint8_t)cd[k];
    }
  }
}

template <int BK, int BV>
cudaError_t launch(const AppendParams& p, cudaStream_t s) {
  if (!p.cu) {
    append_one_kernel<BK, BV><<<dim3(p.batch, p.HKV), 64, 0, s>>>(p);
  } else {
    // a sequence with n rows reaches at most n / 64 + 2 pages
    const int pages = p.n_rows / HYQ_PAGE_ROWS + 2 * min(p.batch, p.n_rows);
    // every head its own block while that does not give far more blocks than
    // can be resident; then a block takes several heads in turn
    int hs = p.HKV;
    while (hs > 1 && (int64_t)pages * hs > 16 * hyq_num_sms()) hs = (hs + 1) / 2;
    append_pages_kernel<BK, BV><<<dim3(pages, hs), kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t hyq_launch_paged_append(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                    const int32_t* cu, int32_t n_rows, const void* k, const void* v, int64_t ld,
                                    void* k_hat, void* v_hat, cudaStream_t s) {
  const AppendParams p{pv,
                       seqs,
                       cu,
                       static_cast<const __nv_bfloat16*>(k),
                       static_cast<const __nv_bfloat16*>(v),
                       static_cast<__nv_bfloat16*>(k_hat),
                       static_cast<__nv_bfloat16*>(v_hat),
                       ld,
                       batch,
                       n_rows,
                       c->num_kv_heads};
  const int bk = hyq_bits_k(c), bv = hyq_bits_v(c);
  if (bk == 4) return bv == 4 ? launch<4, 4>(p, s) : launch<4, 8>(p, s);
  return bv == 4 ? launch<8, 4>(p, s) : launch<8, 8>(p, s);
}
