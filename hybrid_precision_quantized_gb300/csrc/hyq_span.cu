// Many query rows over one run of pages: cross attention (hyq_paged_cross_attention)
// and the shared part of hyq_paged_attention_shared.
//
// A segment is a run of positions [0, len) of one sequence and the query tokens
// that all see the whole of it; per KV head its query rows are (token, head)
// pairs, kRows of them to a block's tile.  For each row, in one pass,
//   M = max x_j, l = sum 2^(x_j - M), O = sum 2^(x_j - M) v_j,
//   x_j = log2(e) q.k_j / sqrt(128)
// on tcgen05: S = Q K^T and O += P V for 128 positions (two pages) at a time.
//
// The codes are taken to fp16 in shared memory once for all rows of a tile:
// c s + z is one fused multiply-add there, so a key or value element is off by half
// a step of fp16 (2^-11), and where fp16 is subnormal it is exact, for c s + z is a
// multiple of the same 2^-24 as s and z.  A row of queries is scaled by a power of
// two, which fp16 takes without rounding (BF16 has fewer bits; elements 2^-27 of
// the row's largest and less are rounded).  Probabilities are rounded to fp16, kept
// between 2^8 and 2^14 at the row's maximum so that the small ones are not lost.
#include "hyq_paged.cuh"
#include "hyq_tc.cuh"

namespace {

constexpr int kRows = 128;   // query rows of a tile (MMA M)
constexpr int kKeys = 128;   // positions of a unit: two pages (MMA N, and K of P V)
constexpr int kUnitPages = kKeys / HYQ_PAGE_ROWS;
constexpr int kThreads = 256;
constexpr int kCost = 4;     // units that a tile's fixed work is worth
constexpr int kRegion = 16384;           // 128 rows of 128 bytes, 128-byte swizzled
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256, kTmemCols = 512;
constexpr float kLog2Scale = 0.1275174307366466f;  // log2(e) / sqrt(128)
constexpr float kSlack = 6.f, kLift = 8.f;         // probabilities at the row's maximum: 2^kLift .. 2^(kLift + kSlack)

// Values beyond fp16: a unit in which c s + z may pass 65504 is taken times 2^-kFar.
template <int B>
constexpr int kFar = B == 4 ? 5 : 9;

struct Params {
  PageView pv;
  const int32_t* seqs;
  const int32_t* cu;     // cross: [n_seg + 1] tokens
  SharedRows shared;     // shared: the groups
  int32_t batch, n_q, n_seg, n_tokens;
  const __nv_bfloat16* q;
  int64_t ldq;
  __nv_bfloat16* out;
  float* part;           // [grid][2] parts
  struct Plan* plan;
  const float* rest;     // shared: partial results of the positions behind, [n_tokens][HQ][kPartFloats]
  int32_t HQ, HKV, gq;
};

// Part of a tile: [32][kRows] four elements each, then maximum and sum a row.
constexpr int kPart = kRows * (HYQ_D + 2);

// The units of all tiles laid end to end, cut into equal runs, a block each.
struct Shares {
  int64_t each, more;
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int owner(int64_t x) const {
    const int64_t wide = more * (each + 1);
    return (int)(x < wide ? x / (each + 1) : more + (x - wide) / each);
  }
};
struct Plan {
  Shares sh;
  int64_t cum[HYQ_PAGED_MAX_BATCH];  // units before segment i
  int32_t len[HYQ_PAGED_MAX_BATCH], t0[HYQ_PAGED_MAX_BATCH], rows[HYQ_PAGED_MAX_BATCH];
};

struct Seg {
  int len, t0, rows;  // positions, first token, query rows of a KV head
  int seq;
};
template <bool kShared>
__device__ __forceinline__ Seg segment(const Params& p, int i, bool report) {
  Seg s;
  if (kShared) {
    s.len = group_len(p.shared, p.pv, p.seqs, i, p.batch, p.n_q);
    const int b0 = p.shared.cu[i], b1 = p.shared.cu[i + 1];
    const bool ok = b0 >= (i == 0 ? 0 : p.shared.cu[i - 1]) && b0 <= b1 && b1 <= p.batch && (i > 0 || b0 == 0) &&
                    (i + 1 < p.n_seg || b1 == p.batch);
    if (report && (!ok || (s.len == 0 && b0 < b1 && p.shared.len[i] != 0))) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
    s.seq = s.len ? page_seq(p.seqs, b0, p.pv.n_seqs) : -1;
    s.t0 = s.len ? b0 * p.n_q : 0;
    s.rows = s.len ? (b1 - b0) * p.n_q * p.gq : 0;
    return s;
  }
  const int t0 = p.cu[i], t1 = p.cu[i + 1];
  const bool ok = t0 >= 0 && t0 <= t1 && t1 <= p.n_tokens;
  s.seq = page_seq(p.seqs, i, p.pv.n_seqs);
  if (report && (!ok || s.seq < 0)) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
  const int64_t cap = (int64_t)p.pv.max_blocks * HYQ_PAGE_ROWS;
  s.len = s.seq < 0 ? 0 : (int)max((int64_t)0, min((int64_t)p.pv.lens[s.seq], cap));
  s.t0 = t0;
  s.rows = ok ? (t1 - t0) * p.gq : 0;
  return s;
}
__device__ __forceinline__ int64_t units_of(int len) { return len ? (len + kKeys - 1) / kKeys + kCost : 0; }

// Byte offset of 16-byte chunk c of row r in a swizzled region.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// Place of position `key` of a unit among the columns of S: neighbours lie four
// rows apart, so that eight lanes' 16-byte stores of a key tile meet distinct banks.
__host__ __device__ constexpr int key_row(int key) { return (key & ~7) | ((key & 7) >> 1) | ((key & 1) << 2); }
__host__ __device__ constexpr int key_of(int row) { return (row & ~7) | ((row & 3) << 1) | ((row >> 2) & 1); }
// Element of the head dimension that column n of O holds (the rows of the value
// tile are ordered so that a stmatrix's eight rows meet distinct banks).
__host__ __device__ constexpr int elem_of(int n) { return (n & ~31) | ((n & 7) << 2) | ((n >> 3) & 3); }

__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes as an fp16 pair, exactly: their bits under 1024, less 1024.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {  // nibbles 0 and 4
  return hadd2_u((w & 0x000F000Fu) | 0x64006400u, 0xE400E400u);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {  // nibbles 1 and 5, which count 16 each
  return hfma2_u((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
}
__device__ __forceinline__ uint32_t even_codes(uint32_t w) {  // bytes 0 and 2
  return hadd2_u((w & 0x00FF00FFu) | 0x64006400u, 0xE400E400u);
}
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) {  // bytes 1 and 3
  return hadd2_u(__byte_perm(w, 0x64646464u, 0x4341), 0xE400E400u);
}
__device__ __forceinline__ uint32_t u4at(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// Halves 0 or 1 of a word, twice.
__device__ __forceinline__ uint32_t both(uint32_t w, int half) { return __byte_perm(w, 0, half ? 0x3232 : 0x1010); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether some c s + z of a group may leave fp16: `vr` rows of the tile at tb, this lane's rows.
template <int B>
__device__ __forceinline__ bool key_meta_far(const uint8_t* meta, int lane, int vr) {
  const uint32_t qmax = B == 4 ? 0x4B804B80u : 0x5BF85BF8u;  // 15, 255
  if (lane >= vr || lane >= 16) return false;
  const uint4 m = *reinterpret_cast<const uint4*>(meta + 16 * lane);
  const uint32_t a = hfma2_u(m.x, qmax, m.z) & 0x7FFF7FFFu, b = hfma2_u(m.y, qmax, m.w) & 0x7FFF7FFFu;
  const uint32_t top = __vmaxu2(a, b);
  return (top >> 16) >= 0x7C00u || (top & 0xFFFFu) >= 0x7C00u;
}
template <int B>
__device__ __forceinline__ bool value_meta_far(const uint8_t* meta, int lane, int vr) {
  const uint32_t qmax = B == 4 ? 0x4B804B80u : 0x5BF85BF8u;
  const int r = 2 * (lane >> 2);  // words: row pair, group
  uint32_t a = hfma2_u(*reinterpret_cast<const uint32_t*>(meta + 4 * lane), qmax,
                       *reinterpret_cast<const uint32_t*>(meta + 128 + 4 * lane)) & 0x7FFF7FFFu;
  return (r < vr && (a & 0xFFFFu) >= 0x7C00u) || (r + 1 < vr && (a >> 16) >= 0x7C00u);
}

// One warp: the 16 keys of a tile as fp16 rows row0 .. row0 + 15 of the key operand at `dst`
// (two regions of 64 elements).  Of 8-bit codes the four elements of each half of a
// group of 32 lie beside those of the other half (query rows are ordered alike).
template <int BK>
__device__ __forceinline__ void keys_to_half(const uint8_t* tb, const uint8_t* meta, int lane, uint8_t* dst, int row0,
                                             bool far) {
  const int g = lane >> 2, t = lane & 3;
  uint4 ma = *reinterpret_cast<const uint4*>(meta + 16 * g), mb = *reinterpret_cast<const uint4*>(meta + 16 * (g + 8));
  if (far) {
    const uint32_t f = (uint32_t)(15 - kFar<BK>) << 10, f2 = f | f << 16;
    ma = make_uint4(hmul2_u(ma.x, f2), hmul2_u(ma.y, f2), hmul2_u(ma.z, f2), hmul2_u(ma.w, f2));
    mb = make_uint4(hmul2_u(mb.x, f2), hmul2_u(mb.y, f2), hmul2_u(mb.z, f2), hmul2_u(mb.w, f2));
  }
  const int ra = key_row(row0 + g), rb = key_row(row0 + g + 8);
#pragma unroll
  for (int v = 0; v < 4; ++v) {  // group v: 16 bytes of each row
    uint32_t xa[4], xb[4];
    if (BK == 4) {
      const uint4 w4 = *reinterpret_cast<const uint4*>(tb + 512 * (v >> 1) + 16 * lane);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w = u4at(w4, 2 * (v & 1) + u), w8 = w >> 8;
        xa[2 * u] = low_codes(w), xa[2 * u + 1] = low_codes(w8);
        xb[2 * u] = high_codes(w), xb[2 * u + 1] = high_codes(w8);
      }
    } else {
      const uint4 w4 = *reinterpret_cast<const uint4*>(tb + 512 * v + 16 * lane);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t wa = u4at(w4, 2 * u), wb = u4at(w4, 2 * u + 1);
        xa[2 * u] = even_codes(wa), xa[2 * u + 1] = odd_codes(wa);
        xb[2 * u] = even_codes(wb), xb[2 * u + 1] = odd_codes(wb);
      }
    }
    const uint32_t sa = both(v < 2 ? ma.x : ma.y, v & 1), za = both(v < 2 ? ma.z : ma.w, v & 1);
    const uint32_t sb = both(v < 2 ? mb.x : mb.y, v & 1), zb = both(v < 2 ? mb.z : mb.w, v & 1);
    uint8_t* reg = dst + (v >> 1) * kRegion;
    const int c = 4 * (v & 1) + t;
    *reinterpret_cast<uint4*>(reg + swz(ra, c)) = make_uint4(hfma2_u(xa[0], sa, za), hfma2_u(xa[1], sa, za),
                                                             hfma2_u(xa[2], sa, za), hfma2_u(xa[3], sa, za));
    *reinterpret_cast<uint4*>(reg + swz(rb, c)) = make_uint4(hfma2_u(xb[0], sb, zb), hfma2_u(xb[1], sb, zb),
                                                             hfma2_u(xb[2], sb, zb), hfma2_u(xb[3], sb, zb));
  }
}

__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// The halves of a word about rows r, r + 1 that lie below vr.
__device__ __forceinline__ uint32_t halves_below(int r, int vr) {
  return (r < vr ? 0xFFFFu : 0u) | (r + 1 < vr ? 0xFFFF0000u : 0u);
}
// One warp: the 16 values of tile i of a page, transposed, as keys 16 i .. 16 i + 15 of the value operand's region
// `dst` (rows: elements in the order of elem_of); rows from vr on are zero.
template <int BV>
__device__ __forceinline__ void values_to_half(const uint8_t* tb, const uint8_t* meta, int lane, uint32_t dst, int i,
                                               int vr, bool far) {
  const int g = lane >> 2, t = lane & 3;
  uint4 s[2], z[2];  // of rows 2t + 8b and the next, groups 0 .. 3
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    s[b] = *reinterpret_cast<const uint4*>(meta + 16 * (t + 4 * b));
    z[b] = *reinterpret_cast<const uint4*>(meta + 128 + 16 * (t + 4 * b));
    const uint32_t in = halves_below(2 * t + 8 * b, vr);
    s[b] = make_uint4(s[b].x & in, s[b].y & in, s[b].z & in, s[b].w & in);
    z[b] = make_uint4(z[b].x & in, z[b].y & in, z[b].z & in, z[b].w & in);
    if (far) {
      const uint32_t f = (uint32_t)(15 - kFar<BV>) << 10, f2 = f | f << 16;
      s[b] = make_uint4(hmul2_u(s[b].x, f2), hmul2_u(s[b].y, f2), hmul2_u(s[b].z, f2), hmul2_u(s[b].w, f2));
      z[b] = make_uint4(hmul2_u(z[b].x, f2), hmul2_u(z[b].y, f2), hmul2_u(z[b].z, f2), hmul2_u(z[b].w, f2));
    }
  }
  // matrix m of a store: element 4 g + c of a group of 32, c = c0 + (m >> 1), keys of half m & 1; lane l gives the
  // address of row l & 7 of matrix l >> 3
  const int mb = (lane >> 3) & 1, mc = lane >> 4, r8 = lane & 7;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
#pragma unroll
    for (int c0 = 0; c0 < 4; c0 += 2) {
      uint32_t x[4];
      if (BV == 4) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(tb + 512 * (q >> 1) + 16 * lane);
        const uint32_t w = u4at(w4, 2 * (q & 1) + (c0 >> 1)), w8 = w >> 8;
        x[0] = low_codes(w), x[1] = low_codes(w8), x[2] = high_codes(w), x[3] = high_codes(w8);
      } else {
        const uint4 w4 = *reinterpret_cast<const uint4*>(tb + 512 * q + 16 * lane);
        const uint32_t wa = u4at(w4, c0), wb = u4at(w4, c0 + 1);
        x[0] = even_codes(wa), x[1] = odd_codes(wa), x[2] = even_codes(wb), x[3] = odd_codes(wb);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) x[m] = hfma2_u(x[m], u4at(s[m & 1], q), u4at(z[m & 1], q));
      const int n = 32 * q + 8 * (c0 + mc) + r8;
      stmatrix_x4(dst + swz(n, 2 * i + mb), x[0], x[1], x[2], x[3]);
    }
  }
}

// One warp: query row r of a tile as fp16 in the order of the keys' elements, scaled by a power of two, and the
// factor of its products (log2 units); v: the lane's elements 4 lane ..  A row that is not finite becomes NaN.
template <int BK>
__device__ __forceinline__ void query_to_half(uint2 v, int lane, uint8_t* dst, int r, float* factor) {
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
  float am = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y)));
  const bool nan = a.x != a.x || a.y != a.y || b.x != b.x || b.y != b.y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  const bool bad = __any_sync(0xffffffffu, nan) || !(am <= 3.402823466e38f);
  // 2^(e - 1) <= am < 2^e; subnormal queries count as 2^-126
  const int e = am > 0.f ? max((__float_as_int(am) >> 23) - 126, -125) : 14;
  // two steps: 2^(14 - e) alone may leave float32
  const float s1 = __int_as_float((127 + (14 - e) / 2) << 23), s2 = __int_as_float((127 + (14 - e) - (14 - e) / 2) << 23);
  uint2 w = make_uint2(pack_f16x2(a.x * s1 * s2, a.y * s1 * s2), pack_f16x2(b.x * s1 * s2, b.y * s1 * s2));
  if (bad) w = make_uint2(0x7FFF7FFFu, 0x7FFF7FFFu);
  const int vg = lane >> 3, el = BK == 4 ? 4 * lane : 32 * vg + 8 * (lane & 3) + 4 * ((lane >> 2) & 1);
  *reinterpret_cast<uint2*>(dst + (el >> 6) * kRegion + swz(r, (el & 63) >> 3) + 2 * (el & 7)) = w;
  // past 2^88 logits differ by more than any exponent holds, or not at all; below 2^-100 they are all alike
  if (lane == 0) *factor = bad ? 1.f : kLog2Scale * __int_as_float((127 + max(-100, min(e - 14, 88))) << 23);
}

// Shared memory of the block.
template <int BK, int BV>
struct Smem {
  static constexpr int kQ = 0, kK = kQ + 2 * kRegion, kV = kK + 2 * kRegion, kRaw = kV + 2 * kRegion;
  static constexpr int kBytes = kRaw + kUnitPages * QFmt<BK, BV>::kBlock + 1024;
};

template <int BK, int BV, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) span_kernel(const Params p) {
  using F = QFmt<BK, BV>;
  using M = Smem<BK, BV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full, done;
  __shared__ uint32_t s_tmem;
  __shared__ int64_t s_warp[kThreads / 32], s_pos, s_end;
  __shared__ Shares s_sh;
  __shared__ struct {
    int64_t base, x0, x1;
    int len, t0, rows, seq, W, grp;
  } s_seg;
  __shared__ float s_factor[kRows];
  __shared__ int s_valid[kUnitPages];
  constexpr int kPer = (HYQ_PAGED_MAX_BATCH + kThreads - 1) / kThreads;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&full, 1);
    mbar_init(&done, 1);
    mbar_fence_init();
  }
  if (warp == 0) tc_alloc(&s_tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  chain_kernel();

  // ---- the segments, kPer neighbours a thread ------------------------------------
  Seg seg[kPer];
  int64_t cum[kPer + 1];
  {
    int64_t w = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = tid * kPer + k;
      seg[k] = Seg{0, 0, 0, -1};
      if (i < p.n_seg) seg[k] = segment<kShared>(p, i, blockIdx.x == 0);
      cum[k] = w;
      w += (int64_t)p.HKV * ((seg[k].rows + kRows - 1) / kRows) * units_of(seg[k].len);
    }
    cum[kPer] = w;
    int64_t pre = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    if (lane == 31) s_warp[warp] = pre;
    __syncthreads();
    int64_t before = pre - w, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += s_warp[i];
      total += s_warp[i];
    }
#pragma unroll
    for (int k = 0; k <= kPer; ++k) cum[k] += before;
    if (tid == 0) {
      const int64_t nb = max((int64_t)1, min((int64_t)gridDim.x, total));
      s_sh.each = total / nb;
      s_sh.more = total - s_sh.each * nb;
      s_pos = s_sh.begin(min((int64_t)blockIdx.x, nb));
      s_end = s_sh.begin(min((int64_t)blockIdx.x + 1, nb));
      if (blockIdx.x == 0) p.plan->sh = s_sh;
    }
    if (blockIdx.x == 0)
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        if (i < p.n_seg) {
          p.plan->cum[i] = cum[k];
          p.plan->len[i] = seg[k].len;
          p.plan->t0[i] = seg[k].t0;
          p.plan->rows[i] = seg[k].rows;
        }
      }
  }
  __syncthreads();
  uint32_t nfull = 0, ndone = 0;  // phases waited for
  bool dead = false;

  while (true) {
    // ---- the tile that the run meets next ------------------------------------------
    const int64_t pos = s_pos, end = s_end;
    __syncthreads();
    if (pos >= end) break;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (cum[k] <= pos && pos < cum[k + 1]) {
        const int W = (int)units_of(seg[k].len);
        const int64_t off = pos - cum[k];
        const int grp = (int)(off / W);
        const int64_t x0 = off - (int64_t)grp * W, x1 = min((int64_t)W, x0 + (end - pos));
        s_seg.base = cum[k] + (int64_t)grp * W + kCost;
        s_seg.x0 = x0, s_seg.x1 = x1;
        s_seg.len = seg[k].len, s_seg.t0 = seg[k].t0, s_seg.rows = seg[k].rows, s_seg.seq = seg[k].seq;
        s_seg.W = W, s_seg.grp = grp;
        s_pos = pos + (x1 - x0);
      }
    __syncthreads();
    const int w0 = max(0, (int)s_seg.x0 - kCost), w1 = (int)s_seg.x1 - kCost, n_units = s_seg.W - kCost;
    if (w1 <= 0) continue;  // the fixed work alone: the next block's
    const int n_mt = (s_seg.rows + kRows - 1) / kRows, h = s_seg.grp / n_mt, mt = s_seg.grp - h * n_mt;
    const int row0 = mt * kRows, n_rows = min(kRows, s_seg.rows - row0), len = s_seg.len;
    const int32_t* table = p.pv.table + (size_t)s_seg.seq * p.pv.max_blocks;
    // ---- the query rows ---------------------------------------------------------------
    for (int r = warp; r < kRows; r += kThreads / 32) {
      uint2 v = make_uint2(0, 0);
      if (r < n_rows) {
        const int tok = (row0 + r) / p.gq;
        v = *reinterpret_cast<const uint2*>(p.q + (size_t)(s_seg.t0 + tok) * p.ldq +
                                            (size_t)(h * p.gq + row0 + r - tok * p.gq) * HYQ_D + 4 * lane);
      }
      query_to_half<BK>(v, lane, sm + M::kQ, r, s_factor + r);
    }
    float m = -INFINITY, l = 0.f;
    int vfar = 0;  // O is held times 2^-kFar
    __syncthreads();
    const float f = s_factor[tid & (kRows - 1)];
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);

    for (int u = w0; u < w1 && !dead; ++u) {
      // ---- the unit's pages ------------------------------------------------------------
      if (tid == 0) {
        uint32_t bytes = 0;
        int page[kUnitPages];
        for (int k = 0; k < kUnitPages; ++k) {
          const int blk = u * kUnitPages + k, left = len - blk * HYQ_PAGE_ROWS;
          page[k] = left > 0 ? table[blk] : -1;
          const bool in = (uint32_t)page[k] < (uint32_t)p.pv.n_pages;
          if (left > 0 && !in) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
          s_valid[k] = in ? min(left, HYQ_PAGE_ROWS) : 0;
          bytes += in ? F::kBlock : 0;
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        mbar_arrive_expect_tx(&full, bytes);
        for (int k = 0; k < kUnitPages; ++k)
          if (s_valid[k])
            bulk_g2s(sm + M::kRaw + k * F::kBlock, p.pv.pool + ((size_t)page[k] * p.HKV + h) * F::kBlock, F::kBlock, &full);
      }
      __syncthreads();
      if (!mbar_wait(&full, nfull & 1u)) dead = true;
      ++nfull;
      // ---- codes to fp16: a tile of 16 rows a warp -------------------------------------
      const int pg = warp >> 2, ti = warp & 3, vr = s_valid[pg] - 16 * ti;
      const uint8_t* tb = sm + M::kRaw + pg * F::kBlock + ti * F::kTile;
      const bool kf = !dead && key_meta_far<BK>(tb + F::kKMeta, lane, vr);
      const bool vf = !dead && value_meta_far<BV>(tb + F::kVMeta, lane, vr);
      const bool kfar = __syncthreads_or(kf);
      const int vnew = __syncthreads_or(vf) | vfar;
      if (__syncthreads_or(dead)) {
        dead = true;
        if (tid == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_TIMEOUT);
        break;
      }
      keys_to_half<BK>(tb, tb + F::kKMeta, lane, sm + M::kK, 64 * pg + 16 * ti, kfar);
      values_to_half<BV>(tb + F::kVCode, tb + F::kVMeta, lane, smem_u32(sm + M::kV) + pg * kRegion, ti, vr, vnew);
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        const uint32_t idesc = tc_idesc(0, 0, kRows, kKeys);
        for (int k = 0; k < 8; ++k)
          tc_mma_f16(tmem + kColS, tc_desc_sw128(smem_u32(sm + M::kQ) + (k >> 2) * kRegion + 32 * (k & 3)),
                     tc_desc_sw128(smem_u32(sm + M::kK) + (k >> 2) * kRegion + 32 * (k & 3)), idesc, k > 0);
        tc_commit(&done);
      }
      if (!mbar_wait(&done, ndone & 1u)) dead = true;
      ++ndone;
      if (__syncthreads_or(dead)) {
        dead = true;
        if (tid == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_TIMEOUT);
        break;
      }
      tc_fence_after();
      // ---- softmax: a row a thread --------------------------------------------------------
      if (tid < kRows) {
        const int v0 = s_valid[0], v1 = s_valid[1];
        const bool whole = v0 == HYQ_PAGE_ROWS && v1 == HYQ_PAGE_ROWS;
        // the maximum is kept as a product, in units of unscaled keys, and taken off before the factor is applied:
        // a large logit's rounding then cannot come out as an exponent
        const float up = kfar ? (float)(1 << kFar<BK>) : 1.f, fac = f * up;
        auto load = [&](int c, float (&x)[32]) {
          uint32_t r[32];
          tc_ld32(t_lane + kColS + 32 * c, r);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] = __uint_as_float(r[i]);
            if (!whole && key_of(32 * (c & 1) + i) >= (c < 2 ? v0 : v1)) x[i] = -INFINITY;
          }
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float x[32];
          load(c, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, x[i]);
        }
        const float top = mx * up;
        float corr = 1.f;
        if ((top - m) * f > kSlack) {
          corr = ex2((m - top) * f);
          m = top;
          l *= corr;
        }
        if (vnew && !vfar) corr *= 1.f / (float)(1 << kFar<BV>);
        if (u > w0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            tc_ld32(t_lane + kColO + 32 * c, r);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * corr);
            tc_st32(t_lane + kColO + 32 * c, r);
          }
        }
        const float nm = m == -INFINITY ? 0.f : -m / up;
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x[32];
            load(c + k, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[i] = ex2(fmaf(x[i] + nm, fac, kLift));
              l += x[i];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)  // positions 2 i, 2 i + 1
              w[16 * k + i] = pack_f16x2(x[key_row(2 * i)], x[key_row(2 * i + 1)]);
          }
          tc_st32(t_lane + kColP + 16 * c, w);
        }
        tc_wait_st();
      }
      vfar = vnew;
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        const uint32_t idesc = tc_idesc(0, 0, kRows, HYQ_D);
        for (int k = 0; k < 8; ++k)
          tc_mma_f16_ts(tmem + kColO, tmem + kColP + 8 * k,
                        tc_desc_sw128(smem_u32(sm + M::kV) + (k >> 2) * kRegion + 32 * (k & 3)), idesc, u > w0 || k > 0);
        tc_commit(&done);
      }
      if (!mbar_wait(&done, ndone & 1u)) dead = true;
      ++ndone;
      tc_fence_after();
      if (__syncthreads_or(dead)) {
        dead = true;
        if (tid == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_TIMEOUT);
      }
    }
    // ---- the tile's result, or this run's part of it --------------------------------------
    if (tid < kRows && !dead) {
      const bool whole = !kShared && w0 == 0 && w1 == n_units;
      const float scale = vfar ? (float)(1 << kFar<BV>) : 1.f, inv = whole ? (l > 0.f ? scale / l : l) : scale;
      float* part = p.part + ((size_t)blockIdx.x * 2 + (w0 == 0 ? 1 : 0)) * kPart;
      const int tok = (row0 + tid) / p.gq;
      __nv_bfloat16* out = p.out + ((size_t)(s_seg.t0 + tok) * p.HQ + h * p.gq + row0 + tid - tok * p.gq) * HYQ_D;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t r[32];
        tc_ld32(t_lane + kColO + 32 * q, r);
        tc_wait_ld();
        if (tid < n_rows) {
          float x[32];  // in the order of the elements
#pragma unroll
          for (int i = 0; i < 32; ++i) x[elem_of(i)] = __uint_as_float(r[i]) * inv;
          if (whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(out + 32 * q + 8 * c) =
                  make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                             pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<float4*>(part + ((8 * q + c) * kRows + tid) * 4) =
                  make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          }
        }
        __syncwarp();
      }
      if (!whole && tid < n_rows)
        *reinterpret_cast<float2*>(part + kRows * HYQ_D + 2 * tid) = make_float2(m * f - kLift, l);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  __syncthreads();
  if (warp == 0) tc_dealloc(tmem, kTmemCols);
}

// The parts of a row in run order, then (shared) what its own positions gave; eight rows of a KV head a block,
// a thread four elements.
constexpr int kJoinThreads = 256;
template <bool kShared>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Params p) {
  chain_kernel();
  const int lane = threadIdx.x & 31, d4 = 4 * (threadIdx.x >> 5) + (lane >> 3);
  const int64_t per = ((int64_t)p.n_tokens * p.gq + 7) / 8, items = per * p.HKV;
  const Plan& plan = *p.plan;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int h = (int)(it / per);
    const int64_t R = (it - h * per) * 8 + (lane & 7);
    if (R >= (int64_t)p.n_tokens * p.gq) continue;
    const int tok = (int)(R / p.gq), head = (int)(R - (int64_t)tok * p.gq);
    int i, len = 0;
    if (kShared) {
      i = p.n_seg ? group_of(p.shared, tok / p.n_q) : 0;
      if (p.n_seg) len = shared_len(p.shared, p.pv, p.seqs, tok / p.n_q, p.batch, p.n_q);
    } else {
      i = 0;
      int hi = p.n_seg;
      while (hi - i > 1) {
        const int mid = (i + hi) >> 1;
        if (p.cu[mid] <= tok) i = mid;
        else hi = mid;
      }
      if (p.cu[i] > tok || tok >= p.cu[i + 1] || p.cu[i] < 0 || p.cu[i + 1] > p.n_tokens) continue;  // nobody's token
      len = plan.len[i];
    }
    float top = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, float4 v) {
      const float mx = fmaxf(top, ml.x), ref = mx == -INFINITY ? 0.f : mx, c0 = ex2(top - ref), c1 = ex2(ml.x - ref);
      top = mx;
      L = fmaf(L, c0, ml.y * c1);
      a.x = fmaf(a.x, c0, v.x * c1), a.y = fmaf(a.y, c0, v.y * c1), a.z = fmaf(a.z, c0, v.z * c1),
      a.w = fmaf(a.w, c0, v.w * c1);
    };
    if (len > 0) {
      const int r = (tok - plan.t0[i]) * p.gq + head, mt = r / kRows, rr = r - mt * kRows;
      const int n_mt = (plan.rows[i] + kRows - 1) / kRows, n_units = (int)units_of(len) - kCost;
      const int64_t base = plan.cum[i] + ((int64_t)h * n_mt + mt) * (n_units + kCost) + kCost;
      const int c0 = plan.sh.owner(base), c1 = plan.sh.owner(base + n_units - 1);
      if (!kShared && c0 == c1) continue;  // written by its block
      for (int c = c0; c <= c1; ++c) {
        const float* part = p.part + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * kPart;
        add(__ldcg(reinterpret_cast<const float2*>(part + kRows * HYQ_D) + rr),
            __ldcg(reinterpret_cast<const float4*>(part) + d4 * kRows + rr));
      }
    }
    if (kShared) {
      const float* e = p.rest + ((size_t)tok * p.HQ + h * p.gq + head) * kPartFloats;
      add(*reinterpret_cast<const float2*>(e + HYQ_D), *(reinterpret_cast<const float4*>(e) + d4));
    }
    const float inv = L > 0.f ? 1.f / L : L;
    *reinterpret_cast<uint2*>(p.out + ((size_t)tok * p.HQ + h * p.gq + head) * HYQ_D + 4 * d4) =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
}

template <int BK, int BV, bool kShared>
cudaError_t launch(const Params& p, cudaStream_t s) {
  constexpr int bytes = Smem<BK, BV>::kBytes;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = hyq_once_per_device(done, [] {
    return cudaFuncSetAttribute(span_kernel<BK, BV, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  if (e != cudaSuccess) return e;
  const int sms = hyq_num_sms();
  e = hyq_launch_chained(span_kernel<BK, BV, kShared>, dim3(sms), kThreads, bytes, s, p);
  if (e != cudaSuccess) return e;
  const int64_t items = ((int64_t)p.n_tokens * p.gq + 7) / 8 * p.HKV;
  return hyq_launch_chained(join_kernel<kShared>, dim3((int)(items < 8 * sms ? items : 8 * sms)), kJoinThreads, 0, s, p);
}

template <bool kShared>
cudaError_t launch_bits(const hyq_config* c, const Params& p, cudaStream_t s) {
  const int bk = hyq_bits_k(c), bv = hyq_bits_v(c);
  if (bk == 4) return bv == 4 ? launch<4, 4, kShared>(p, s) : launch<4, 8, kShared>(p, s);
  return bv == 4 ? launch<8, 4, kShared>(p, s) : launch<8, 8, kShared>(p, s);
}

size_t plan_bytes() { return hyq_align256(sizeof(Plan)); }
size_t parts_bytes() { return hyq_align256((size_t)hyq_num_sms() * 2 * kPart * 4); }
size_t rest_bytes(const hyq_config* c, int32_t batch, int32_t n_q) {
  return hyq_align256((size_t)batch * n_q * c->num_q_heads * kPartFloats * 4);
}

Params params(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch, const void* q, int64_t ldq,
              void* out, void* ws) {
  Params p = {};
  p.pv = pv;
  p.seqs = seqs;
  p.batch = batch;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.plan = static_cast<Plan*>(ws);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + plan_bytes());
  p.HQ = c->num_q_heads;
  p.HKV = c->num_kv_heads;
  p.gq = p.HQ / p.HKV;
  return p;
}

// The attention's own workspace lies before the rows' results, at the size of its largest call: its tickets, which stay
// zero between calls, then have one place whatever the call's size.
size_t attention_bytes(const hyq_config* c) {
  return hyq_paged_attention_ws_bytes(c, HYQ_PAGED_MAX_BATCH, HYQ_PAGED_MAX_Q);
}

}  // namespace

size_t hyq_paged_shared_ws_bytes(const hyq_config* c, int32_t batch, int32_t n_q) {
  return plan_bytes() + parts_bytes() + attention_bytes(c) + rest_bytes(c, batch, n_q);
}
size_t hyq_paged_cross_ws_bytes(const hyq_config* c, int32_t batch) {
  return plan_bytes() + parts_bytes() + hyq_paged_attention_ws_bytes(c, batch, 1);
}

cudaError_t hyq_launch_paged_shared(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                    int32_t n_q, const SharedRows& shared, const void* q, int64_t ldq, void* out,
                                    void* ws, cudaStream_t s) {
  Params p = params(c, pv, seqs, batch, q, ldq, out, ws);
  char* own = static_cast<char*>(ws) + plan_bytes() + parts_bytes();
  float* rest = reinterpret_cast<float*>(own + attention_bytes(c));
  p.n_q = n_q;
  p.n_tokens = batch * n_q;
  p.shared = shared;
  p.n_seg = shared.n;
  p.rest = rest;
  const cudaError_t e = hyq_launch_paged_attention(c, pv, seqs, batch, n_q, q, ldq, nullptr, 0, out, nullptr, &p.shared,
                                                   rest, own, s);
  if (e != cudaSuccess) return e;
  return launch_bits<true>(c, p, s);
}

cudaError_t hyq_launch_paged_cross(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                   const int32_t* cu_q, int32_t n_tokens, const void* q, int64_t ldq, void* out,
                                   void* ws, cudaStream_t s) {
  if (!cu_q)  // a token a sequence: the last position sees them all
    return hyq_launch_paged_attention(c, pv, seqs, batch, 1, q, ldq, nullptr, 0, out, nullptr, nullptr, nullptr,
                                      static_cast<char*>(ws) + plan_bytes() + parts_bytes(), s);
  Params p = params(c, pv, seqs, batch, q, ldq, out, ws);
  p.n_q = 1;
  p.n_tokens = n_tokens;
  p.cu = cu_q;
  p.n_seg = batch;
  return launch_bits<false>(c, p, s);
}
