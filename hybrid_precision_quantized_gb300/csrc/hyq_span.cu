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
//
// What bounds it: 4 x 128 x 128 x 128 flops a job (128 query rows and a unit) are 1024 cycles
// of the tensor cores; the kernel takes about three times that (2000 tokens of four
// sequences of up to 16001, 8-bit codes: 824 us, 0.40 of the product rate; one sequence of
// 32768 for 64 requests: 0.19 of the rate for the whole call).  Each role waits for its own
// dependent instructions and for the one before it (products, exponentials, products),
// two jobs in flight; tensor cores are busy a third of the time, issue slots a half.
// Few query rows: the codes are read once, and the fixed work of a block (its tiles, the
// query rows, the join of parts) is most of the time.
#include <type_traits>

#include "hyq_codes.cuh"
#include "hyq_f2.cuh"
#include "hyq_paged.cuh"
#include "hyq_tc.cuh"

namespace {

constexpr int kRows = 128;   // query rows of a product (MMA M)
constexpr int kPair = 2 * kRows;  // of a tile
constexpr int kKeys = 128;   // positions of a unit: two pages (MMA N, and K of P V)
constexpr int kUnitPages = kKeys / HYQ_PAGE_ROWS;
constexpr int kCost = 6;     // jobs (128 rows of a unit) that a tile's fixed work is worth
constexpr int kRegion = 16384;  // 128 rows of 128 bytes, 128-byte swizzled
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;  // two of each
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
  struct Plan* plan;
  struct Split* split;   // [grid]
  struct Entry* list;    // [grid][HYQ_PAGED_MAX_BATCH]
  float* part;           // [grid][2] parts of tiles
  float* half;           // [grid][2] states of 128 rows
  const float* rest;     // shared: partial results of the positions behind, [n_tokens][HQ][kPartFloats]
  int32_t HQ, HKV, gq;
};

// Part of a tile: [32][kPair] four elements each, then maximum and sum a row.
constexpr int kPart = kPair * (HYQ_D + 2);

// The jobs of all tiles laid end to end (a tile's begin with kCost that are not there), cut into equal runs, a
// block each; a unit of a pair is its first job's block's.
struct Shares {
  int64_t each, more;
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int owner(int64_t x) const {
    const int64_t wide = more * (each + 1), y = x < wide ? x : x - wide, d = x < wide ? each + 1 : each;
    const int64_t q = ((y | d) >> 32) == 0 ? (int64_t)((uint32_t)y / (uint32_t)d) : y / d;
    return (int)(x < wide ? q : more + q);
  }
};
struct Plan {
  Shares sh;
  int64_t cum[HYQ_PAGED_MAX_BATCH];  // jobs before segment i
  int32_t len[HYQ_PAGED_MAX_BATCH], t0[HYQ_PAGED_MAX_BATCH], rows[HYQ_PAGED_MAX_BATCH];
};

// The tile whose first units are a block's and the others the next blocks'; n_rows is 0 when there is none.
struct Split {
  int64_t base;  // its first job behind the fixed work
  int32_t t0, row0, n_rows, h, nt, units;
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
__device__ __forceinline__ int n_units(int len) { return (len + kKeys - 1) / kKeys; }
// Jobs of one KV head: whole pairs, then the rows that are left.
__device__ __forceinline__ int64_t head_slots(int len, int rows) {
  if (len <= 0 || rows <= 0) return 0;
  const int U = n_units(len), n = (rows + kPair - 1) / kPair, left = rows - (n - 1) * kPair;
  return (int64_t)(n - 1) * (kCost + 2 * U) + kCost + (left > kRows ? 2 : 1) * U;
}
// First unit that begins at or behind job x of a tile with nt jobs a unit.
__device__ __forceinline__ int unit_from(int x, int nt) { return max(0, (x - kCost + nt - 1) / nt); }
// Whether block c has units of the tile whose first job (behind the fixed work) is `base`.
__device__ __forceinline__ bool holds(const Shares& sh, int c, int64_t base, int nt, int U) {
  const int64_t a = max((int64_t)0, sh.begin(c) - base), b = min((int64_t)nt * U, sh.begin(c + 1) - base);
  return a < b && (a + nt - 1) >> (nt - 1) < (b + nt - 1) >> (nt - 1);  // (nt is 1 or 2)
}

// Byte offset of 16-byte chunk c of row r in a swizzled region.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// Place of position `key` of a unit among the columns of S: neighbours lie four
// rows apart, so that eight lanes' 16-byte stores of a key tile meet distinct banks.
__host__ __device__ constexpr int key_row(int key) { return (key & ~7) | ((key & 7) >> 1) | ((key & 1) << 2); }
__host__ __device__ constexpr int key_of(int row) { return (row & ~7) | ((row & 3) << 1) | ((row >> 2) & 1); }
// Element of the head dimension that column n of O holds (the rows of the value
// tile are ordered so that a stmatrix's eight rows meet distinct banks).
__host__ __device__ constexpr int elem_of(int n) { return (n & ~31) | ((n & 7) << 2) | ((n >> 3) & 3); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__device__ __forceinline__ uint4 mul4(const uint4& v, uint32_t f) {
  return make_uint4(hmul2_u(v.x, f), hmul2_u(v.y, f), hmul2_u(v.z, f), hmul2_u(v.w, f));
}
template <int B>
__device__ __forceinline__ uint32_t far_scale() {  // 2^-kFar, twice
  const uint32_t f = (uint32_t)(15 - kFar<B>) << 10;
  return f | f << 16;
}

// Whether a step and zero (two of each) may take c s + z out of fp16: the largest code's, as bits without sign.
template <int B>
__device__ __forceinline__ uint32_t largest(uint32_t s, uint32_t z) {
  return hfma2_u(s, B == 4 ? 0x4B804B80u : 0x5BF85BF8u, z) & 0x7FFF7FFFu;  // 15, 255
}
__device__ __forceinline__ bool leaves_fp16(uint32_t most) { return (most >> 16) >= 0x7C00u || (most & 0xFFFFu) >= 0x7C00u; }

// The keys of a 16-row tile of codes in a warp's registers.
template <int BK, int BV>
struct KeyTile {
  using F = QFmt<BK, BV>;
  uint4 kc[BK / 2];  // code words, 512 bytes of the region each
  uint4 ka, kb;      // steps and zeros of rows g, g + 8

  __device__ __forceinline__ void load(const uint8_t* tb, int lane) {
    const int g = lane >> 2;
#pragma unroll
    for (int i = 0; i < BK / 2; ++i) kc[i] = *reinterpret_cast<const uint4*>(tb + 512 * i + 16 * lane);
    ka = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * g);
    kb = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * (g + 8));
  }
  // The keys as fp16 rows row0 .. row0 + 15 of the key operand at `dst` (two regions of 64 elements).  Of 8-bit codes
  // the four elements of each half of a group of 32 lie beside those of the other half (query rows are ordered alike).
  __device__ __forceinline__ void store(uint8_t* dst, int lane, int row0, bool is_far) {
    const int g = lane >> 2, t = lane & 3;
    if (__builtin_expect(is_far, 0)) ka = mul4(ka, far_scale<BK>()), kb = mul4(kb, far_scale<BK>());
    const int x = key_row(g);  // (row0 is a multiple of 8; row g + 8 lies 8 rows on, swizzled alike)
    uint8_t* at = dst + 128 * (row0 + x);
    // groups 2 i and 2 i + 1: 16 bytes of each row apiece.  (Rolled: see the waits.)
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint32_t xa[4], xb[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (BK == 4) {
            const uint32_t w = u4at(kc[0], 2 * v + u), w8 = w >> 8;
            xa[2 * u] = low_codes(w), xa[2 * u + 1] = low_codes(w8);
            xb[2 * u] = high_codes(w), xb[2 * u + 1] = high_codes(w8);
          } else {
            const uint32_t wa = u4at(kc[BK == 4 ? 0 : v], 2 * u), wb = u4at(kc[BK == 4 ? 0 : v], 2 * u + 1);
            xa[2 * u] = even_codes(wa), xa[2 * u + 1] = odd_codes(wa);
            xb[2 * u] = even_codes(wb), xb[2 * u + 1] = odd_codes(wb);
          }
        }
        const uint32_t sa = both(ka.x, v), za = both(ka.z, v), sb = both(kb.x, v), zb = both(kb.z, v);
        uint8_t* to = at + (((4 * v + t) ^ x) << 4);
        *reinterpret_cast<uint4*>(to) = make_uint4(hfma2_u(xa[0], sa, za), hfma2_u(xa[1], sa, za),
                                                   hfma2_u(xa[2], sa, za), hfma2_u(xa[3], sa, za));
        *reinterpret_cast<uint4*>(to + 1024) = make_uint4(hfma2_u(xb[0], sb, zb), hfma2_u(xb[1], sb, zb),
                                                          hfma2_u(xb[2], sb, zb), hfma2_u(xb[3], sb, zb));
      }
      at += kRegion;
      ka.x = ka.y, ka.z = ka.w, kb.x = kb.y, kb.z = kb.w;
      if (BK == 4) kc[0] = kc[1];
      else kc[0] = kc[BK / 2 - 2], kc[1] = kc[BK / 2 - 1];
    }
  }
};

// Its values.
template <int BK, int BV>
struct ValueTile {
  using F = QFmt<BK, BV>;
  uint4 vc[BV / 2];
  uint4 vs[2], vz[2];  // steps and zeros of rows 2t + 8b and the next, groups 0 .. 3

  __device__ __forceinline__ void load(const uint8_t* tb, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int i = 0; i < BV / 2; ++i) vc[i] = *reinterpret_cast<const uint4*>(tb + F::kVCode + 512 * i + 16 * lane);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      vs[b] = *reinterpret_cast<const uint4*>(tb + F::kVMeta + 16 * (t + 4 * b));
      vz[b] = *reinterpret_cast<const uint4*>(tb + F::kVMeta + 128 + 16 * (t + 4 * b));
    }
  }
  // The values, transposed, as keys 16 i .. 16 i + 15 of the value operand's region `dst` (rows: elements in the
  // order of elem_of); rows from vr on are zero.
  __device__ __forceinline__ void store(uint32_t dst, int lane, int i, int vr, bool is_far) {
    const int t = lane & 3;
    if (__builtin_expect(vr < 16, 0)) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t in = halves_below(2 * t + 8 * b, vr);
        vs[b] = make_uint4(vs[b].x & in, vs[b].y & in, vs[b].z & in, vs[b].w & in);
        vz[b] = make_uint4(vz[b].x & in, vz[b].y & in, vz[b].z & in, vz[b].w & in);
      }
    }
    if (__builtin_expect(is_far, 0)) {
#pragma unroll
      for (int b = 0; b < 2; ++b) vs[b] = mul4(vs[b], far_scale<BV>()), vz[b] = mul4(vz[b], far_scale<BV>());
    }
    // matrix m of a store: element 4 g + c of a group of 32, c = c0 + (m >> 1), keys of half m & 1; lane l gives the
    // address of row l & 7 of matrix l >> 3
    const int mb = (lane >> 3) & 1, mc = lane >> 4, r8 = lane & 7;
    const uint32_t at = dst + 128 * (8 * mc + r8) + (((2 * i + mb) ^ r8) << 4);
    uint32_t to = at;
#pragma unroll 1
    for (int i2 = 0; i2 < 2; ++i2) {  // groups 2 i2 and 2 i2 + 1
#pragma unroll
      for (int v = 0; v < 2; ++v) {
#pragma unroll
        for (int c0 = 0; c0 < 4; c0 += 2) {
          uint32_t x[4];
          if (BV == 4) {
            const uint32_t w = u4at(vc[0], 2 * v + (c0 >> 1)), w8 = w >> 8;
            x[0] = low_codes(w), x[1] = low_codes(w8), x[2] = high_codes(w), x[3] = high_codes(w8);
          } else {
            const uint32_t wa = u4at(vc[BV == 4 ? 0 : v], c0), wb = u4at(vc[BV == 4 ? 0 : v], c0 + 1);
            x[0] = even_codes(wa), x[1] = odd_codes(wa), x[2] = even_codes(wb), x[3] = odd_codes(wb);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) x[m] = hfma2_u(x[m], v ? vs[m & 1].y : vs[m & 1].x, v ? vz[m & 1].y : vz[m & 1].x);
          stmatrix_x4(to + 128 * (32 * v + 8 * c0), x[0], x[1], x[2], x[3]);
        }
      }
      to += 128 * 64;
#pragma unroll
      for (int b = 0; b < 2; ++b) vs[b].x = vs[b].z, vs[b].y = vs[b].w, vz[b].x = vz[b].z, vz[b].y = vz[b].w;
      if (BV == 4) vc[0] = vc[1];
      else vc[0] = vc[BV / 2 - 2], vc[1] = vc[BV / 2 - 1];
    }
  }
};

// ---- roles --------------------------------------------------------------------------------
// The block's warps work apart and meet at mbarriers:
//   softmax  two groups of four warps, a query row a thread: group t works on jobs t, t + 2, .. of a tile
//   codes    four warps for keys, four for values: a tile's query rows, then page by page the codes to fp16, 16 rows a
//            warp
//   mma      two warps, one thread of each issues: S = Q K^T; O += P V
//   copy     the tiles of the block's run, one after another, and their pages
//   scan     whether a page has rows beyond fp16
// A tile of more than 128 query rows is a pair: each unit is two jobs, one for each half of the
// rows, so that one half's products overlap the other's exponentials.  A smaller tile's
// units are one job each and alternate between the groups, whose states are joined at the end.
constexpr int kKeyWarp = 8, kValueWarp = 12, kMmaWarp = 16, kPvWarp = 17, kCopyWarp = 18, kScanWarp = 19, kThreads = 20 * 32;
constexpr int kTiles = 4;   // tiles of the run that are known ahead
constexpr int kVPages = 3;  // pages of values in fp16

// Shared memory of the block.
template <int BK, int BV>
struct Smem {
  static constexpr int kQ = 0, kK = kQ + 4 * kRegion, kV = kK + 4 * kRegion, kRaw = kV + kVPages * kRegion;
  static constexpr int kSlots = (227 * 1024 - 6 * 1024 - kRaw) / QFmt<BK, BV>::kBlock;  // pages of codes
  static constexpr int kBytes = kRaw + kSlots * QFmt<BK, BV>::kBlock + 1024;
  static_assert(kSlots >= 2, "two pages under way");
};

// A tile: units [w0, w1) of query rows row0 .. of KV head h of a segment.
struct Tile {
  const int32_t* table;
  int w0, w1;            // w1 == 0: no tile is left
  int len, t0, row0, n_rows, h;
  int pair, whole;       // more than 128 rows; all of its units are this block's
};
// A segment that the block's run meets.
struct Entry {
  int64_t cum;
  int32_t len, t0, rows, seq;
};

// The query rows of a tile as fp16 in the order of the keys' elements, each scaled by a power of two, and the factors of
// their products (log2 units).  A row that is not finite becomes NaN.  Eight warps, two rows of each at a time, a lane
// eight elements of one.
template <int BK>
__device__ __noinline__ void load_queries(const Params& p, const Tile& t, int warp, int lane, uint8_t* dst, float* factor) {
  constexpr int kAhead = 4;  // pairs of rows under way, and as many in hand
  const int half = lane >> 4, l = lane & 15;
  const int rows = (t.n_rows + 31) & ~31;  // (no warp looks at the rows behind: their products are their own)
  const int dt = 16 / p.gq, dh = 16 - dt * p.gq;
  int tok = (t.row0 + 2 * warp + half) / p.gq, head = t.row0 + 2 * warp + half - tok * p.gq;
  const __nv_bfloat16* q = p.q + (size_t)t.t0 * p.ldq + (size_t)t.h * p.gq * HYQ_D + 8 * l;
  auto fetch = [&](int r0, uint4 (&v)[kAhead]) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      v[k] = make_uint4(0, 0, 0, 0);
      if (r0 + 16 * k + half < t.n_rows) v[k] = *reinterpret_cast<const uint4*>(q + (size_t)tok * p.ldq + head * HYQ_D);
      tok += dt, head += dh;
      if (head >= p.gq) head -= p.gq, ++tok;
    }
  };
  uint4 v[kAhead], next[kAhead];
  fetch(2 * warp, v);
#pragma unroll 1
  for (int r0 = 2 * warp; r0 < rows; r0 += 16 * kAhead) {
    fetch(r0 + 16 * kAhead, next);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = r0 + 16 * k + half;
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u4at(v[k], i) << 16);
        x[2 * i + 1] = __uint_as_float(u4at(v[k], i) & 0xFFFF0000u);
      }
      float am = 0.f, z = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[i])), z = fmaf(x[i], 0.f, z);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      const bool bad = (__ballot_sync(0xffffffffu, z != 0.f) >> (16 * half)) & 0xFFFFu;  // (NaN: infinities too)
      // 2^(e - 1) <= am < 2^e; subnormal queries count as 2^-126
      const int e = am > 0.f ? max((__float_as_int(am) >> 23) - 126, -125) : 14;
      // two steps: 2^(14 - e) alone may leave float32
      const float s1 = __int_as_float((127 + (14 - e) / 2) << 23), s2 = __int_as_float((127 + (14 - e) - (14 - e) / 2) << 23);
      uint4 w = make_uint4(pack_f16x2(x[0] * s1 * s2, x[1] * s1 * s2), pack_f16x2(x[2] * s1 * s2, x[3] * s1 * s2),
                           pack_f16x2(x[4] * s1 * s2, x[5] * s1 * s2), pack_f16x2(x[6] * s1 * s2, x[7] * s1 * s2));
      if (bad) w = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
      uint8_t* to = dst + (r / kRows) * 2 * kRegion + (l >> 3) * kRegion;
      const int rr = r % kRows;
      if (BK == 4) {
        *reinterpret_cast<uint4*>(to + swz(rr, l & 7)) = w;
      } else {  // elements 32 v + 16 i + 4 t lie at 32 v + 8 t + 4 i
        const int c = 4 * ((l >> 2) & 1) + 2 * (l & 1), h8 = 8 * ((l >> 1) & 1);
        *reinterpret_cast<uint2*>(to + swz(rr, c) + h8) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2*>(to + swz(rr, c + 1) + h8) = make_uint2(w.z, w.w);
      }
      // past 2^88 logits differ by more than any exponent holds, or not at all; below 2^-100 they are all alike
      if (l == 0) factor[r] = bad ? 1.f : kLog2Scale * __int_as_float((127 + max(-100, min(e - 14, 88))) << 23);
      v[k] = next[k];
    }
  }
}

struct Bars {
  uint64_t raw_full[8], raw_seen[8], raw_empty[8];
  uint64_t k_full[2], k_empty[2], v_full[kVPages], v_empty[kVPages];
  uint64_t q_full, q_empty;
  uint64_t tile_full[kTiles], tile_empty[kTiles];
  uint64_t s_full[2], s_free[2], p_full[2], o_full[2], o_empty[2], joined, drained;
};
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done;
}

template <int BK, int BV, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) span_kernel(const __grid_constant__ Params p) {
  using F = QFmt<BK, BV>;
  using M = Smem<BK, BV>;
  constexpr int kSlots = M::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) Bars bar;
  __shared__ uint32_t s_tmem;
  __shared__ int64_t s_warp[kThreads / 32];
  __shared__ int64_t s_pos, s_end;
  __shared__ int s_first;
  __shared__ Tile s_tile[kTiles];
  __shared__ float s_factor[2][2 * kRows];
  __shared__ int s_valid[8];  // rows of the page in a slot
  // Of the last pages: their rows, whether the keys are taken down (bit 8), the values (bit 9).  Pages are scanned
  // ahead of the softmax by the slots and two units at most.
  __shared__ volatile uint32_t s_page[16];
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  constexpr int kPer = (HYQ_PAGED_MAX_BATCH + kThreads - 1) / kThreads;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kSlots; ++i) mbar_init(&bar.raw_full[i], 1), mbar_init(&bar.raw_seen[i], 1), mbar_init(&bar.raw_empty[i], 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], 4), mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.s_full[i], 1), mbar_init(&bar.s_free[i], 1), mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_full[i], 1), mbar_init(&bar.o_empty[i], 4);
    }
    for (int i = 0; i < kVPages; ++i) mbar_init(&bar.v_full[i], 4), mbar_init(&bar.v_empty[i], 1);
    for (int i = 0; i < kTiles; ++i) mbar_init(&bar.tile_full[i], 1), mbar_init(&bar.tile_empty[i], 19);
    mbar_init(&bar.q_full, 8), mbar_init(&bar.q_empty, 1);
    mbar_init(&bar.joined, 4), mbar_init(&bar.drained, 2);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tc_alloc(&s_tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  chain_kernel();

  // ---- the segments, kPer neighbours a thread; those of this block's run are listed ---------
  Entry* list = p.list + (size_t)blockIdx.x * HYQ_PAGED_MAX_BATCH;
  {
    Seg seg[kPer];
    int64_t cum[kPer + 1], w = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = tid * kPer + k;
      seg[k] = Seg{0, 0, 0, -1};
      if (i < p.n_seg) seg[k] = segment<kShared>(p, i, blockIdx.x == 0);
      cum[k] = w;
      w += (int64_t)p.HKV * head_slots(seg[k].len, seg[k].rows);
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
    const int64_t nb = max((int64_t)1, min((int64_t)gridDim.x, total));
    Shares sh;
    sh.each = total / nb;
    sh.more = total - sh.each * nb;
    const int64_t pos = sh.begin(min((int64_t)blockIdx.x, nb)), end = sh.begin(min((int64_t)blockIdx.x + 1, nb));
    if (tid == 0) {
      s_pos = pos, s_end = end;
      if (blockIdx.x == 0) p.plan->sh = sh;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = tid * kPer + k;
      if (i >= p.n_seg) break;
      if (cum[k] < end && cum[k + 1] > pos) list[i] = Entry{cum[k], seg[k].len, seg[k].t0, seg[k].rows, seg[k].seq};
      else if (cum[k] < end) list[i].rows = 0;
      if (cum[k] <= pos && pos < cum[k + 1]) s_first = i;
      if (blockIdx.x == 0) {
        p.plan->cum[i] = cum[k];
        p.plan->len[i] = seg[k].len;
        p.plan->t0[i] = seg[k].t0;
        p.plan->rows[i] = seg[k].rows;
      }
    }
  }
  __syncthreads();

  // The code of all roles has to stay in the SM's instruction cache together: a wait is a few instructions, and the
  // loops are rolled.  One that runs out leaves a flag, which is reported at the end.
  auto wait = [&](uint64_t& b, uint32_t parity) {
#pragma unroll 1
    for (int it = 0; it < (1 << 22); ++it) {
      if (mbar_try(&b, parity & 1u)) return true;
      if (*abort_flag) return false;
    }
    *abort_flag = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t& b, uint32_t parity) { return (bool)__all_sync(0xffffffffu, wait(b, parity)); };

  if (warp == kCopyWarp) {
    // ---------------- the run's tiles and their pages ---------------------------------------
    int64_t pos = s_pos;
    const int64_t end = s_end;
    int i = pos < end ? s_first : 0;
    uint32_t n_tile = 0, n_page = 0;
    Split cut;
    cut.n_rows = 0;
    bool ok = true;
    while (ok) {
      Tile t;
      t.w1 = 0;
      while (pos < end) {  // a tile of which the run has more than fixed work
        const Entry e = list[i];
        const int U = n_units(e.len);
        const int64_t per = head_slots(e.len, e.rows);
        if (e.rows == 0 || pos >= e.cum + per * p.HKV) {
          ++i;
          continue;
        }
        const int h = (int)((pos - e.cum) / per);
        const int64_t off = pos - e.cum - per * h;
        const int n_mt = (e.rows + kPair - 1) / kPair, mt = (int)min((int64_t)n_mt - 1, off / (kCost + 2 * U));
        const int n_rows = min(kPair, e.rows - mt * kPair), nt = n_rows > kRows ? 2 : 1;
        const int64_t x0 = off - (int64_t)mt * (kCost + 2 * U);
        const int W = kCost + nt * U, x1 = (int)min((int64_t)W, x0 + (end - pos));
        pos += x1 - x0;
        const int a = unit_from((int)x0, nt), b = unit_from(x1, nt);
        if (a >= b) continue;
        if (a == 0 && b < U)
          cut = Split{e.cum + per * h + (int64_t)mt * (kCost + 2 * U) + kCost, e.t0, mt * kPair, n_rows, h, nt, U};
        t = Tile{p.pv.table + (size_t)e.seq * p.pv.max_blocks, a, b, e.len, e.t0, mt * kPair, n_rows, h, nt == 2, a == 0 && b == U};
        break;
      }
      const uint32_t slot = n_tile % kTiles;
      ok = wait_warp(bar.tile_empty[slot], (n_tile / kTiles) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        s_tile[slot] = t;
        mbar_arrive(&bar.tile_full[slot]);
      }
      __syncwarp();
      ++n_tile;
      if (t.w1 == 0) break;
      const int p0 = t.w0 * kUnitPages, np = min(t.w1 * kUnitPages, (t.len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS) - p0;
      const uint8_t* heads = p.pv.pool + (size_t)t.h * F::kBlock;
      int cur = lane < np ? t.table[p0 + lane] : -1, nxt = 32 + lane < np ? t.table[p0 + 32 + lane] : -1;
      for (int j = 0; j < np; ++j) {
        const int pg = __shfl_sync(0xffffffffu, cur, j & 31);
        const uint32_t sl = n_page % kSlots;
        ok = wait_warp(bar.raw_empty[sl], (n_page / kSlots) ^ 1);
        if (!ok) break;
        if (lane == sl) {  // copies that one thread issues complete one after another
          const bool in = (uint32_t)pg < (uint32_t)p.pv.n_pages;
          if (!in) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
          s_valid[sl] = in ? min(HYQ_PAGE_ROWS, t.len - (p0 + j) * HYQ_PAGE_ROWS) : 0;
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          mbar_arrive_expect_tx(&bar.raw_full[sl], in ? F::kBlock : 0);
          if (in) bulk_g2s(sm + M::kRaw + sl * F::kBlock, heads + (size_t)pg * p.HKV * F::kBlock, F::kBlock, &bar.raw_full[sl]);
        }
        __syncwarp();
        ++n_page;
        if ((j & 31) == 31) {
          cur = nxt;
          nxt = j + 33 + lane < np ? t.table[p0 + j + 33 + lane] : -1;
        }
      }
    }
    if (lane == 0) p.split[blockIdx.x] = cut;
    if (!ok)  // copies in flight land before the block's shared memory goes
      for (uint32_t n = n_page > kSlots ? n_page - kSlots : 0; n < n_page; ++n)
        (void)mbar_wait(&bar.raw_full[n % kSlots], (n / kSlots) & 1u);
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ---------------- products ---------------------------------------------------------------
    // Each warp's flow is uniform and one lane issues: a product of 128 x 128 x 16 takes 64 cycles, and descriptors
    // put together by a single thread took longer than that.  P takes the place of S, so the next S of a group waits
    // for the product that reads P, and is itself the sign that all products of the group so far are done.
    constexpr uint64_t kStep = kRegion >> 4;
    const bool one = lane == 0, pv = warp == kPvWarp;
    auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    uint32_t n_tile = 0, kn = 0, sn[2] = {0, 0}, on[2] = {0, 0};
    bool ok = true;
    while (true) {
      ok = wait_warp(bar.tile_full[n_tile % kTiles], n_tile / kTiles);
      if (!ok) break;
      const Tile& tile = s_tile[n_tile % kTiles];
      const int w0 = same(tile.w0), w1 = same(tile.w1), len = same(tile.len), pair = same(tile.pair);
      if (w1 == 0) break;
      const int jobs = (w1 - w0) << pair;
      if (!pv) {
        const uint64_t dQ = tc_desc_sw128(smem_u32(sm + M::kQ)), dK = tc_desc_sw128(smem_u32(sm + M::kK));
        ok = wait_warp(bar.q_full, n_tile);
#pragma unroll 1
        for (int j = 0; ok && j < jobs; ++j) {
          const int t = j & 1, u = w0 + (j >> pair);
          if (!pair || t == 0) ok = wait_warp(bar.k_full[kn & 1], kn >> 1);
          ok = ok && wait_warp(bar.s_free[t], sn[t]++ ^ 1);
          if (!ok) break;
          tc_fence_after();
          const bool half = u * kKeys + HYQ_PAGE_ROWS >= len;  // one page
          const uint32_t idesc = half ? tc_idesc(0, 0, kRows, HYQ_PAGE_ROWS) : tc_idesc(0, 0, kRows, kKeys);
          const uint64_t a = dQ + (pair ? t : 0) * 2 * kStep, b = dK + (kn & 1) * 2 * kStep;
          if (one) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint64_t off = (k >> 2) * kStep + 2 * (k & 3);
              tc_mma_f16(tmem + kColS + kKeys * t, a + off, b + off, idesc, k > 0);
            }
            tc_commit(&bar.s_full[t]);
            if (!pair || t == 1) tc_commit(&bar.k_empty[kn & 1]);
            if (j + 1 == jobs) tc_commit(&bar.q_empty);
          }
          if (!pair || t == 1) ++kn;
        }
      } else {
        const uint64_t dV = tc_desc_sw128(smem_u32(sm + M::kV));
#pragma unroll 1
        for (int j = 0; ok && j < jobs; ++j) {
          const int t = j & 1, u = w0 + (j >> pair);
          const int pages = u * kKeys + HYQ_PAGE_ROWS >= len ? 1 : 2;
          if (j < 2) ok = wait_warp(bar.o_empty[t], on[t] ^ 1);
          ok = ok && wait_warp(bar.p_full[t], sn[t]++);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < pages; ++k) {
            const uint32_t n = kn + k, sl = n % kVPages;
            if (!pair || t == 0) {
              ok = wait_warp(bar.v_full[sl], n / kVPages);
              if (!ok) break;
              tc_fence_after();
            }
            const uint64_t b = dV + sl * kStep;
            const uint32_t a = tmem + kColS + kKeys * t + 32 * k;
            if (one) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                tc_mma_f16_ts(tmem + kColO + HYQ_D * t, a + 8 * x, b + 2 * x, tc_idesc(0, 0, kRows, HYQ_D),
                              j >= 2 || k > 0 || x > 0);
              if (!pair || t == 1) tc_commit(&bar.v_empty[sl]);
            }
          }
          if (!ok) break;
          if (one) {
            tc_commit(&bar.s_free[t]);
            if (j + 2 >= jobs) tc_commit(&bar.o_full[t]);
          }
          if (j + 2 >= jobs) ++on[t];
          if (!pair || t == 1) kn += pages;
        }
      }
      if (!ok) break;
      __syncwarp();
      if (one) mbar_arrive(&bar.tile_empty[n_tile % kTiles]);
      ++n_tile;
    }
    if (one) {
      tc_commit(&bar.drained);  // every product has finished
      (void)mbar_wait(&bar.drained, 0);
    }
    __syncwarp();
  } else if (warp >= kKeyWarp && warp < kMmaWarp) {
    // ---------------- query rows and codes ----------------------------------------------------
    // A page whose c s + z may leave fp16 is taken down; values then stay so to the end of the tile, whose O has one scale.
    auto codes = [&](auto kind) {
      constexpr bool kIsKeys = decltype(kind)::value;
      const int cw = warp & 3;
      uint32_t n_tile = 0, n_page = 0, kn = 0;
      while (wait_warp(bar.tile_full[n_tile % kTiles], n_tile / kTiles)) {
        const Tile& t = s_tile[n_tile % kTiles];
        const int last = (t.len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS, end = min(t.w1 * kUnitPages, last);
        int pg = t.w0 * kUnitPages;
        if (t.w1 == 0 || !wait_warp(bar.q_empty, n_tile ^ 1)) return;
        load_queries<BK>(p, t, warp - kKeyWarp, lane, sm + M::kQ, s_factor[n_tile & 1]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.q_full);
          mbar_arrive(&bar.tile_empty[n_tile % kTiles]);
        }
#pragma unroll 1
        for (; pg < end; ++pg, ++n_page) {
          const uint32_t sl = n_page % kSlots;
          if (!wait_warp(bar.raw_seen[sl], n_page / kSlots)) return;
          (void)mbar_try(&bar.raw_full[sl], (n_page / kSlots) & 1u);  // (it is: what the copy brought is visible)
          const uint32_t info = s_page[n_page & 15];
          typename std::conditional<kIsKeys, KeyTile<BK, BV>, ValueTile<BK, BV>>::type x;
          x.load(sm + M::kRaw + sl * F::kBlock + cw * F::kTile, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.raw_empty[sl]);
          if constexpr (kIsKeys) {
            const uint32_t ks = kn & 1, k = pg & 1;
            if (k == 0 && !wait_warp(bar.k_empty[ks], (kn >> 1) ^ 1)) return;
            x.store(sm + M::kK + ks * 2 * kRegion, lane, HYQ_PAGE_ROWS * k + 16 * cw, info & 0x100);
            fence_proxy_async_smem();
            __syncwarp();
            if (k == 1 || pg + 1 == last) {
              if (lane == 0) mbar_arrive(&bar.k_full[ks]);
              ++kn;
            }
          } else {
            const uint32_t vs = n_page % kVPages;
            if (!wait_warp(bar.v_empty[vs], (n_page / kVPages) ^ 1)) return;
            x.store(smem_u32(sm + M::kV) + vs * kRegion, lane, cw, (int)(info & 0xFF) - 16 * cw, info & 0x200);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.v_full[vs]);
          }
        }
        ++n_tile;
      }
    };
    if (warp < kValueWarp) codes(std::true_type{});
    else codes(std::false_type{});
  } else if (warp == kScanWarp) {
    // ---------------- rows beyond fp16 --------------------------------------------------------------
    uint32_t n_tile = 0, n_page = 0;
    bool ok = true;
    while (ok && wait_warp(bar.tile_full[n_tile % kTiles], n_tile / kTiles)) {
      const Tile& t = s_tile[n_tile % kTiles];
      int pages = min(t.w1 * kUnitPages, (t.len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS) - t.w0 * kUnitPages;
      if (t.w1 == 0) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.tile_empty[n_tile % kTiles]);
      ++n_tile;
      bool vfar = false;
#pragma unroll 1
      for (; pages > 0; --pages, ++n_page) {
        const uint32_t sl = n_page % kSlots;
        ok = wait_warp(bar.raw_full[sl], n_page / kSlots);
        if (!ok) break;
        const int valid = s_valid[sl];
        uint32_t km = 0, vm = 0;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {  // lane: words of row lane / 2 and of row pair lane / 4
          const uint8_t* tb = sm + M::kRaw + sl * F::kBlock + i * F::kTile;
          const uint32_t* k = reinterpret_cast<const uint32_t*>(tb + F::kKMeta) + 4 * (lane >> 1) + (lane & 1);
          const uint32_t* v = reinterpret_cast<const uint32_t*>(tb + F::kVMeta) + lane;
          const int r = valid - 16 * i;
          if ((lane >> 1) < r) km = __vmaxu2(km, largest<BK>(k[0], k[2]));
          vm = __vmaxu2(vm, largest<BV>(v[0], v[32]) & halves_below(2 * (lane >> 2), r));
        }
        const bool kf = __any_sync(0xffffffffu, leaves_fp16(km));
        vfar |= __any_sync(0xffffffffu, leaves_fp16(vm)) != 0;
        if (lane == 0) {
          s_page[n_page & 15] = (uint32_t)valid | (uint32_t)kf << 8 | (uint32_t)vfar << 9;
          mbar_arrive(&bar.raw_seen[sl]);
        }
        __syncwarp();
      }
    }
  } else {
    // ---------------- softmax: a query row a thread ---------------------------------------------
    const int t = warp >> 2, rr = tid & (kRows - 1);
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = t_lane + kColS + kKeys * t, tO = t_lane + kColO + HYQ_D * t;
    uint32_t n_tile = 0, n_page = 0, sn = 0, on = 0, joins = 0;
    bool ok = true;
    while (true) {
      ok = wait_warp(bar.tile_full[n_tile % kTiles], n_tile / kTiles);
      if (!ok) break;
      const Tile tile = s_tile[n_tile % kTiles];
      if (tile.w1 == 0) break;
      const int U = tile.w1 - tile.w0, jobs = tile.pair ? U : (U + 1 - t) / 2;
      const int r = rr + (tile.pair ? kRows * t : 0);
      const bool idle = (r & ~31) >= tile.n_rows;  // no row of the warp is one
      float m = -INFINITY, l = 0.f, f = 1.f;
      bool far = false;
      for (int j = 0; j < jobs; ++j) {
        ok = wait_warp(bar.s_full[t], sn++);
        if (!ok) break;
        if (idle) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_full[t]);
          continue;
        }
        tc_fence_after();
        if (j == 0) f = s_factor[n_tile & 1][r];
        const int u = tile.pair ? j : 2 * j + t;
        const bool one = (tile.w0 + u) * kKeys + HYQ_PAGE_ROWS >= tile.len;  // one page
        const uint32_t i0 = s_page[(n_page + 2 * u) & 15], i1 = one ? i0 & 0x200 : s_page[(n_page + 2 * u + 1) & 15];
        const int v0 = i0 & 0xFF, v1 = i1 & 0xFF, chunks = one ? 2 : 4;
        const bool far0 = i0 & 0x200, far1 = i1 & 0x200, full = v0 == HYQ_PAGE_ROWS && v1 == HYQ_PAGE_ROWS;
        const float up0 = i0 & 0x100 ? (float)(1 << kFar<BK>) : 1.f, up1 = i1 & 0x100 ? (float)(1 << kFar<BK>) : 1.f;
        auto load = [&](int c, float (&x)[32]) {
          uint32_t y[32];
          tc_ld32(tS + 32 * c, y);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(y[i]);
          if (__builtin_expect(!full, 0)) {
            const int v = (c < 2 ? v0 : v1) - 32 * (c & 1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (key_of(i) >= v) x[i] = -INFINITY;
          }
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          float x[32];
          load(c, x);
          float y[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < 32; i += 8) {
            y[0] = fmax3(y[0], x[i], x[i + 1]);
            y[1] = fmax3(y[1], x[i + 2], x[i + 3]);
            if (i + 4 < 32) {
              y[2] = fmax3(y[2], x[i + 4], x[i + 5]);
              y[3] = fmax3(y[3], x[i + 6], x[i + 7]);
            }
          }
          mx = fmaxf(mx, fmax3(fmaxf(y[0], y[1]), y[2], y[3]) * (c < 2 ? up0 : up1));
        }
        // The reference stands at a maximum that may lag by kSlack, in units of products.
        float corr = 1.f;
        if ((mx - m) * f > kSlack) {
          corr = ex2((m - mx) * f);
          m = mx;
          l *= corr;
        }
        if (far1 && !far) corr *= 1.f / (float)(1 << kFar<BV>);
        far = far1;
        if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {  // (the products so far are done: S came after them)
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t y[32];
            tc_ld32(tO + 32 * c, y);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * corr);
            tc_st32(tO + 32 * c, y);
          }
        }
        // Probabilities; they take the place of products that have been read.  Of rows whose logits are large the
        // reference is taken off before the factor is applied: its rounding would come out as an exponent.
        const float ref = m == -INFINITY ? 0.f : m;  // (nothing is seen yet, or the row is NaN)
        auto probs = [&](auto large) {
          constexpr bool kLarge = decltype(large)::value;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            const bool low = far1 && !far0 && c < 2;  // of values that are not taken down in a unit whose others are
            const float up = c < 2 ? up0 : up1, lift = low ? kLift - kFar<BV> : kLift;
            const uint64_t nm2 = f2_splat(kLarge ? -ref / up : fmaf(-ref, f, lift)),
                           fac2 = f2_splat(f * up), lift2 = f2_splat(lift);
            float x[32];
            load(c, x);
            uint64_t acc[2] = {0, 0};
            uint32_t w[16];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              float e[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint64_t y = f2_pack(x[8 * b + 2 * i], x[8 * b + 2 * i + 1]);
                y = kLarge ? f2_fma(f2_add(y, nm2), fac2, lift2) : f2_fma(y, fac2, nm2);
                e[2 * i] = ex2(f2_lo(y)), e[2 * i + 1] = ex2(f2_hi(y));
                acc[i & 1] = f2_add(acc[i & 1], f2_pack(e[2 * i], e[2 * i + 1]));
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)  // positions 2 i, 2 i + 1
                w[4 * b + i] = pack_f16x2(e[key_row(2 * i)], e[key_row(2 * i + 1)]);
            }
            acc[0] = f2_add(acc[0], acc[1]);
            const float sum = f2_lo(acc[0]) + f2_hi(acc[0]);
            l += low ? sum * (float)(1 << kFar<BV>) : sum;
            tc_st16(tS + 16 * c, w);
          }
        };
        if (__builtin_expect(__any_sync(0xffffffffu, fabsf(ref * f) > 4096.f), 0)) probs(std::true_type{});
        else probs(std::false_type{});
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[t]);
      }
      if (!ok) break;
      n_page += min(tile.w1 * kUnitPages, (tile.len + HYQ_PAGE_ROWS - 1) / HYQ_PAGE_ROWS) - tile.w0 * kUnitPages;
      // ---- the tile's result, or this run's part of it -----------------------------------------
      const bool two = !tile.pair && U > 1;  // both groups have a state of the same rows
      if (jobs) {
        ok = wait_warp(bar.o_full[t], on++);
        if (!ok) break;
        tc_fence_after();
      }
      float* half = p.half + ((size_t)blockIdx.x * 2 + (joins & 1)) * (kPart / 2);
      if (two && t == 1 && !idle) {  // group 1 hands its state over
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t y[32];
          tc_ld32(tO + 32 * q, y);
          tc_wait_ld();
          if (r < tile.n_rows) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(half + ((8 * q + c) * kRows + r) * 4) = make_uint4(y[c], y[8 + c], y[16 + c], y[24 + c]);
          }
          __syncwarp();
        }
        if (r < tile.n_rows)
          *reinterpret_cast<float2*>(half + kRows * HYQ_D + 2 * r) = make_float2(m * f - kLift, far ? -l : l);
      }
      if (two && t == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.joined);
      }
      if (two && t == 0) {
        ok = wait_warp(bar.joined, joins);
        if (!ok) break;
      }
      if (two) ++joins;
      if (jobs && !idle && (tile.pair || t == 0)) {
        // the group's own state and, with weights, the other group's and that of the rows' own positions
        float M0 = m * f - kLift, w0 = far ? (float)(1 << kFar<BV>) : 1.f, w1 = 0.f, w2 = 0.f, L = l;
        const int tok = tile.t0 + (tile.row0 + r) / p.gq, head = tile.h * p.gq + (tile.row0 + r) % p.gq;
        const bool row = r < tile.n_rows;
        if (two && row) {
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(half + kRows * HYQ_D) + r);
          const bool far2 = ml.y < 0.f;
          const float top = fmaxf(M0, ml.x), ref = top == -INFINITY ? 0.f : top, a = ex2(M0 - ref), b = ex2(ml.x - ref);
          L = L * a + fabsf(ml.y) * b;
          w0 *= a;
          w1 = b * (far2 ? (float)(1 << kFar<BV>) : 1.f);
          M0 = top;
        }
        const float* rest = nullptr;
        bool write = row;
        if (kShared && tile.whole && row) {
          write = shared_len(p.shared, p.pv, p.seqs, tok / p.n_q, p.batch, p.n_q) > 0;  // (else the join's)
          rest = p.rest + ((size_t)tok * p.HQ + head) * kPartFloats;
          const float2 ml = *reinterpret_cast<const float2*>(rest + HYQ_D);
          const float top = fmaxf(M0, ml.x), ref = top == -INFINITY ? 0.f : top, a = ex2(M0 - ref), b = ex2(ml.x - ref);
          L = L * a + ml.y * b;
          w0 *= a, w1 *= a, w2 = b;
        }
        if (tile.whole) {
          const float inv = L > 0.f ? 1.f / L : L;
          w0 *= inv, w1 *= inv, w2 *= inv;
        }
        float* part = p.part + ((size_t)blockIdx.x * 2 + (tile.w0 == 0 ? 1 : 0)) * kPart;
        __nv_bfloat16* out = p.out + ((size_t)tok * p.HQ + head) * HYQ_D;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t y[32];
          tc_ld32(tO + 32 * q, y);
          tc_wait_ld();
          if (write) {
            float x[32];  // in the order of the elements
#pragma unroll
            for (int i = 0; i < 32; ++i) x[elem_of(i)] = __uint_as_float(y[i]) * w0;
            if (two) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(half) + (8 * q + c) * kRows + r);
                x[4 * c] = fmaf(v.x, w1, x[4 * c]), x[4 * c + 1] = fmaf(v.y, w1, x[4 * c + 1]);
                x[4 * c + 2] = fmaf(v.z, w1, x[4 * c + 2]), x[4 * c + 3] = fmaf(v.w, w1, x[4 * c + 3]);
              }
            }
            if (kShared && tile.whole) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float4 v = *(reinterpret_cast<const float4*>(rest) + 8 * q + c);
                x[4 * c] = fmaf(v.x, w2, x[4 * c]), x[4 * c + 1] = fmaf(v.y, w2, x[4 * c + 1]);
                x[4 * c + 2] = fmaf(v.z, w2, x[4 * c + 2]), x[4 * c + 3] = fmaf(v.w, w2, x[4 * c + 3]);
              }
            }
            if (tile.whole) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4*>(out + 32 * q + 8 * c) =
                    make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                               pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
            } else {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<float4*>(part + ((8 * q + c) * kPair + r) * 4) =
                    make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            }
          }
          __syncwarp();
        }
        if (!tile.whole && row) *reinterpret_cast<float2*>(part + kPair * HYQ_D + 2 * r) = make_float2(M0, L);
      }
      if (jobs) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.o_empty[t]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.tile_empty[n_tile % kTiles]);
      ++n_tile;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_abort) hyq_set_err(p.pv.err, HYQ_DEVERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tc_dealloc(tmem, kTmemCols);
  }
}

constexpr int kJoinThreads = 256;
// Four elements of a row, summed up over parts.
struct Joined {
  float top = -INFINITY, L = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);

  __device__ __forceinline__ void add(float2 ml, float4 v) {
    const float mx = fmaxf(top, ml.x), ref = mx == -INFINITY ? 0.f : mx, c0 = ex2(top - ref), c1 = ex2(ml.x - ref);
    top = mx;
    L = fmaf(L, c0, ml.y * c1);
    a.x = fmaf(a.x, c0, v.x * c1), a.y = fmaf(a.y, c0, v.y * c1), a.z = fmaf(a.z, c0, v.z * c1),
    a.w = fmaf(a.w, c0, v.w * c1);
  }
  // Blocks c0 .. c1 of a tile, row r of it; eight parts under way.
  __device__ __forceinline__ void parts(const Params& p, const Shares& sh, int c0, int c1, int64_t base, int nt, int U, int r,
                                        int d4) {
    constexpr int kHold = 8;
    for (int c = c0; c <= c1; c += kHold) {
      float2 ml[kHold];
      float4 v[kHold];
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const float* part = p.part + ((size_t)(c + k) * 2 + (c + k == c0 ? 1 : 0)) * kPart;
        // (a run that ends before a pair's second half of a unit may have nothing of the tile)
        const bool in = c + k <= c1 && holds(sh, c + k, base, nt, U);
        ml[k] = in ? __ldcg(reinterpret_cast<const float2*>(part + kPair * HYQ_D) + r) : make_float2(-INFINITY, 0.f);
        v[k] = in ? __ldcg(reinterpret_cast<const float4*>(part) + d4 * kPair + r) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kHold; ++k) add(ml[k], v[k]);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* out) const {
    const float inv = L > 0.f ? 1.f / L : L;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
};

// Shared: the parts of a row in run order, then what its own positions gave; eight rows of a KV head a block, a thread
// four elements.  Rows that the span kernel has finished are left out.
__global__ void __launch_bounds__(kJoinThreads) join_shared_kernel(const __grid_constant__ Params p) {
  chain_kernel();
  const int lane = threadIdx.x & 31, d4 = 4 * (threadIdx.x >> 5) + (lane >> 3);
  // (the query rows of all heads are fewer than 2^31)
  const uint32_t rows = (uint32_t)p.n_tokens * p.gq, per = (rows + 7) / 8, items = per * p.HKV;
  const Plan& plan = *p.plan;
  for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int h = (int)(it / per);
    const uint32_t R = (it - h * per) * 8 + (lane & 7);
    if (R >= rows) continue;
    const int tok = (int)(R / p.gq), head = (int)(R - (uint32_t)tok * p.gq);
    const int i = p.n_seg ? group_of(p.shared, tok / p.n_q) : 0;
    const int len = p.n_seg ? shared_len(p.shared, p.pv, p.seqs, tok / p.n_q, p.batch, p.n_q) : 0;
    Joined sum;
    if (len > 0) {
      const int U = n_units(len), r = (tok - plan.t0[i]) * p.gq + head, mt = r / kPair, rr = r - mt * kPair;
      const int nt = min(kPair, plan.rows[i] - mt * kPair) > kRows ? 2 : 1;
      const int64_t base = plan.cum[i] + h * head_slots(len, plan.rows[i]) + (int64_t)mt * (kCost + 2 * U) + kCost;
      const int c0 = plan.sh.owner(base), c1 = plan.sh.owner(base + (int64_t)nt * (U - 1));
      if (c0 == c1) continue;  // written by its block
      sum.parts(p, plan.sh, c0, c1, base, nt, U, rr, d4);
    }
    const float* e = p.rest + ((size_t)tok * p.HQ + h * p.gq + head) * kPartFloats;
    sum.add(*reinterpret_cast<const float2*>(e + HYQ_D), *(reinterpret_cast<const float4*>(e) + d4));
    sum.store(p.out + ((size_t)tok * p.HQ + h * p.gq + head) * HYQ_D + 4 * d4);
  }
}

// Cross: eight rows of a tile that several blocks share, found where its first block has noted it; and zeros for the
// tokens of empty sequences.
__global__ void __launch_bounds__(kJoinThreads) join_cross_kernel(const __grid_constant__ Params p) {
  chain_kernel();
  const int lane = threadIdx.x & 31, d4 = 4 * (threadIdx.x >> 5) + (lane >> 3), c0 = blockIdx.x;
  const Split tile = p.split[c0];
  const int r = 8 * blockIdx.y + (lane & 7);
  if (r < tile.n_rows) {
    const Shares sh = p.plan->sh;
    Joined sum;
    sum.parts(p, sh, c0, sh.owner(tile.base + (int64_t)tile.nt * (tile.units - 1)), tile.base, tile.nt, tile.units, r, d4);
    const int tok = (tile.row0 + r) / p.gq, head = tile.h * p.gq + tile.row0 + r - tok * p.gq;
    sum.store(p.out + ((size_t)(tile.t0 + tok) * p.HQ + head) * HYQ_D + 4 * d4);
  }
  for (int i = blockIdx.x; i < p.n_seg; i += gridDim.x) {
    if (p.plan->len[i] > 0) continue;
    const size_t n = (size_t)(p.plan->rows[i] / p.gq) * p.HQ * (HYQ_D / 8);  // (whole tokens)
    uint4* out = reinterpret_cast<uint4*>(p.out + (size_t)p.plan->t0[i] * p.HQ * HYQ_D);
    for (size_t x = blockIdx.y * kJoinThreads + threadIdx.x; x < n; x += (size_t)gridDim.y * kJoinThreads)
      out[x] = make_uint4(0, 0, 0, 0);
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
  if (!kShared)
    return hyq_launch_chained(join_cross_kernel, dim3(sms, kPair / 8), kJoinThreads, 0, s, p);
  const int64_t items = ((int64_t)p.n_tokens * p.gq + 7) / 8 * p.HKV;
  return hyq_launch_chained(join_shared_kernel, dim3((int)(items < 8 * sms ? items : 8 * sms)), kJoinThreads, 0, s, p);
}

template <bool kShared>
cudaError_t launch_bits(const hyq_config* c, const Params& p, cudaStream_t s) {
  const int bk = hyq_bits_k(c), bv = hyq_bits_v(c);
  if (bk == 4) return bv == 4 ? launch<4, 4, kShared>(p, s) : launch<4, 8, kShared>(p, s);
  return bv == 4 ? launch<8, 4, kShared>(p, s) : launch<8, 8, kShared>(p, s);
}

size_t plan_bytes() { return hyq_align256(sizeof(Plan)) + hyq_align256((size_t)hyq_num_sms() * sizeof(Split)); }
size_t list_bytes() { return hyq_align256((size_t)hyq_num_sms() * HYQ_PAGED_MAX_BATCH * sizeof(Entry)); }
size_t parts_bytes() { return list_bytes() + hyq_align256((size_t)hyq_num_sms() * 3 * kPart * 4); }
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
  p.split = reinterpret_cast<Split*>(static_cast<char*>(ws) + hyq_align256(sizeof(Plan)));
  p.list = reinterpret_cast<Entry*>(static_cast<char*>(ws) + plan_bytes());
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + plan_bytes() + list_bytes());
  p.half = p.part + (size_t)hyq_num_sms() * 2 * kPart;
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
