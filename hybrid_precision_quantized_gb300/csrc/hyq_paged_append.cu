// Quantised rows into the pages of their sequences (hyq_paged_append), with the
// bound records of the keys.
//
// Per group of 32 elements of a row (Quant_B of Algorithm 4): s the smallest
// FP16 value with qmax s >= max - min, z = FP16(min), codes nearest to
// (x - z) / s, decided exactly (exact_code4).  Reads 512 bytes per (row, KV
// head), writes 160 (4-bit codes), and 512 more with the dequantised rows.
//
// One warp per (page that gets rows, KV head, K or V), working through the
// page's 16-row tiles.  A lane holds eight elements (one 16-byte load) of the
// rows 2t, 2t + 1, 2t + 8, 2t + 9 for two t: those whose codes share words in
// either fragment order, so that a tile's words are assembled in registers,
// without barriers; the next tile's rows come into shared memory meanwhile, each
// lane's own part; a key warp carries the page's bounds.
// Steps and reciprocals are costly: the rows are reduced together, halves
// exchanged, so that each of a group's four lanes ends with two rows' (min, max)
// and derives their steps, once per (row, group) instead of once per lane.
//
// What bounds it: instruction issue (81 per row and tensor at 16 warps an SM) and
// the last round of blocks; prompts of 30 thousand rows of 8 KV heads with the rows
// read back take 62 us, 0.76 of the copy rate.  A block lives about 15 us, so
// its start counts: a call row a thread and the page's number asked for
// after the first rows took 5 us off.  Slower than blocks of eight warps with a page
// each: 24 warps an SM with the rows read twice from shared memory (+6 us), blocks of
// four warps (+12), half pages of values a block (+3), resident blocks
// whose warps go from page to page (+8, and +3 with the values' tiles levelling the
// warps' shares).
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
// the call's rows on; the page's entry in the table.
struct PageRows {
  const int32_t* entry;
  int r0, r1, tok0;
};

// First position and number of rows of call row i; n = 0 when there is
// nothing to write or the row must be left out (bad: for a reason to report).
struct CallRows {
  int seq, start, n, tok;
  bool bad;
};
__device__ __forceinline__ CallRows call_rows(const AppendParams& p, int i) {
  CallRows c;
  c.tok = p.cu ? p.cu[i] : i;
  const int end = p.cu ? p.cu[i + 1] : i + 1;
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
  r.entry = p.pv.table + (size_t)c.seq * p.pv.max_blocks + blk;
  r.r0 = max(0, c.start - p0);
  r.r1 = min(HYQ_PAGE_ROWS, c.start + c.n - p0);
  r.tok0 = c.tok + (p0 + r.r0 - c.start);
  return r;
}
// The page is in the pool (reported if it is not).
__device__ __forceinline__ bool page_ok(const AppendParams& p, int page) {
  const bool ok = page >= 0 && page < p.pv.n_pages;
  if (!ok) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
  return ok;
}

__device__ __forceinline__ uint32_t u32_of(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __nv_bfloat162 bf2_of(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) { return u32_of(__hmin2_nan(bf2_of(a), bf2_of(b))); }
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return u32_of(__hmax2_nan(bf2_of(a), bf2_of(b))); }

// (min, -max) of a lane's eight elements, NaN if one is.
__device__ __forceinline__ uint32_t min_negmax(uint4 v) {
  const uint32_t mn = min2(min2(v.x, v.y), min2(v.z, v.w));
  const uint32_t nx = max2(max2(v.x, v.y), max2(v.z, v.w)) ^ 0x80008000u;
  return min2(__byte_perm(mn, nx, 0x5410), __byte_perm(mn, nx, 0x7632));
}

// Step, zero and reciprocal of a group from (min, -max).  The sign of r tells
// how the codes are found: r >= 0, the group's extremes lie within half a step
// of codes 0 and qmax, so no code needs a clamp; r < 0, one may (|r| is the
// reciprocal); -infinity, a group that FP16 metadata cannot hold (or a NaN):
// codes, step and zero are 0.
struct GroupQ {
  uint32_t sz;  // FP16 step | zero << 16
  float r;
};
// A code argument t = fl(fl(x - z) r) is off by at most 2^-24 (difference),
// 2^-23 (reciprocal) and 2^-24 (product) of its size: below 2^-17 for codes up to
// 15 and 2^-13 up to 255.  An argument that far from a midpoint rounds to the
// right code; the others are decided exactly.
template <int BITS>
struct Near {
  static constexpr float kTie = BITS == 4 ? 0.5f - 0x1p-17f : 0.5f - 0x1p-13f;
  static constexpr float kMax = BITS == 4 ? 15.f : 255.f;
  static constexpr float kInv = BITS == 4 ? 0x1.111112p-4f : 0x1.010102p-8f;  // 1 / kMax, rounded up
};
template <int BITS>
__device__ __forceinline__ GroupQ group_q(uint32_t mm) {
  constexpr float qmax = Near<BITS>::kMax;
  const float2 m = __bfloat1622float2(bf2_of(mm));
  const float mn = m.x, mx = -m.y;
  // s: the smallest FP16 value with qmax s >= d, d = mx - mn rounded up (qmax s
  // is exact in float32, so no such product lies between mx - mn and d).  The
  // rounded-up quotient is at most one FP16 step too large.
  const float d = __fsub_ru(mx, mn);
  uint32_t sb = __half_as_ushort(__float2half_ru(__fmul_ru(d, Near<BITS>::kInv)));
  if (sb > 0 && __fmul_rn(__half2float(__ushort_as_half((unsigned short)(sb - 1))), qmax) >= d) --sb;
  const float s = __half2float(__ushort_as_half((unsigned short)sb));
  const __half zh = __float2half_rn(mn);
  const float z = __half2float(zh);
  GroupQ o;
  if (isnan(m.x) || isnan(m.y) || isinf(s) || isinf(z)) {
    o.sz = 0u;
    o.r = -INFINITY;
  } else {
    o.sz = sb | ((uint32_t)__half_as_ushort(zh) << 16);
    float r = 0.f;
    if (s > 0.f) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    const float tl = __fmul_rn(__fsub_rn(mn, z), r), th = __fmul_rn(__fsub_rn(mx, z), r);
    o.r = tl > -0.5f && th < qmax + 0.5f ? r : -r;
  }
  return o;
}
__device__ __forceinline__ bool marked(float r) { return r == -INFINITY; }

// The code of x from its argument t: rint(t), and near the midpoint
// m = (k + 1/2) s the sign of x - z - m, in float32 without a rounding that
// counts.  m is exact (9 + 11 bits).  x - z = a + e with a = fl(x - z) and e its
// error (a two-sum); a lies within a factor of two of m there, so a - m is exact
// and x - z > m just when a - m > -e.  Ties go to the even code.
template <int BITS>
__device__ __forceinline__ float exact_code4(float x, float z, float s, float t) {
  float c = rintf(t);
  if (fabsf(__fsub_rn(t, c)) > Near<BITS>::kTie) {
    const float k = floorf(t), m = __fmul_rn(__fadd_rn(k, 0.5f), s);
    const float a = __fsub_rn(x, z), bb = __fsub_rn(a, x);
    const float e = __fsub_rn(__fsub_rn(x, __fsub_rn(a, bb)), __fadd_rn(z, bb));
    const float d = __fsub_rn(a, m);
    const bool odd = __float2int_rz(k) & 1;
    c = d > -e || (d == -e && odd) ? __fadd_rn(k, 1.f) : k;
  }
  return fminf(fmaxf(c, 0.f), Near<BITS>::kMax);
}

// The codes of the two elements of w, decided exactly (r < 0: with clamps).
// Out of line: about one row in 25 has such an element (the midpoints that a
// coarse BF16 grid meets).
template <int BITS>
__device__ __noinline__ float2 exact_pair(uint32_t w, float s, float z, float r) {
  if (marked(r)) return make_float2(0.f, 0.f);
  const float2 x = __bfloat1622float2(bf2_of(w));
  const float ra = fabsf(r);
  return make_float2(exact_code4<BITS>(x.x, z, s, __fmul_rn(__fsub_rn(x.x, z), ra)),
                     exact_code4<BITS>(x.y, z, s, __fmul_rn(__fsub_rn(x.y, z), ra)));
}

// Codes of a lane's eight elements: -c as float pairs and, for packing, as the
// low bytes of b (the bits of 1.5 * 2^23 + c).  v becomes zeros in a marked group.
struct Codes8 {
  uint64_t nc[4];
  uint32_t b[8];
};
template <int BITS>
__device__ __forceinline__ Codes8 codes8(uint4& v, float s, float z, float r) {
  Codes8 o;
  const uint64_t nz2 = f2_splat(-z), r2 = f2_splat(r), m2 = f2_splat(kMagic), no2 = f2_splat(-1.f);
  float far = 0.f;
  // distance of an element pair's arguments from their codes
  auto code_pair = [&](int k) {
    const uint32_t w = (&v.x)[k];
    const uint64_t x = (uint64_t)(w << 16) | ((uint64_t)(w & 0xFFFF0000u) << 32);
    const uint64_t y = f2_add(x, nz2), b = f2_fma(y, r2, m2);
    o.nc[k] = f2_fma(b, no2, m2);
    o.b[2 * k] = lo32(b), o.b[2 * k + 1] = hi32(b);
    const uint64_t d = f2_fma(y, r2, o.nc[k]);
    return fmaxf(fabsf(f2_lo(d)), fabsf(f2_hi(d)));
  };
#pragma unroll
  for (int k = 0; k < 4; ++k) far = fmaxf(far, code_pair(k));
  if (r < 0.f || far > Near<BITS>::kTie) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (code_pair(k) > Near<BITS>::kTie || r < 0.f) {
        const float2 c = exact_pair<BITS>((&v.x)[k], s, z, r);
        o.nc[k] = f2_pack(-c.x, -c.y);
        o.b[2 * k] = __float_as_uint(__fadd_rn(c.x, kMagic));
        o.b[2 * k + 1] = __float_as_uint(__fadd_rn(c.y, kMagic));
      }
    }
    if (marked(r)) v = make_uint4(0u, 0u, 0u, 0u);
  }
  return o;
}

// Bytes: the codes of elements 0, 2, 1, 3 of four (the order of a key word).
__device__ __forceinline__ uint32_t key_word(const uint32_t* b) {
  return __byte_perm(__byte_perm(b[0], b[2], 0x0040), __byte_perm(b[1], b[3], 0x0040), 0x5410);
}
// w with its byte `at` replaced by the low byte of x.
template <int at>
__device__ __forceinline__ uint32_t put_byte(uint32_t w, uint32_t x) {
  return __byte_perm(w, x, (0x3210u & ~(0xFu << (4 * at))) | (0x4u << (4 * at)));
}
__device__ __forceinline__ uint32_t put_byte(uint32_t w, uint32_t x, int at) {  // at: a constant after unrolling
  return at == 0 ? put_byte<0>(w, x) : at == 1 ? put_byte<1>(w, x) : at == 2 ? put_byte<2>(w, x) : put_byte<3>(w, x);
}

// Metadata of (row r of the tile, group q).
template <int T>
__device__ __forceinline__ void store_meta(uint8_t* meta, int r, int q, uint32_t sz) {
  const int so = T == 0 ? 16 * r + 2 * q : 16 * (r >> 1) + 4 * q + 2 * (r & 1);
  *reinterpret_cast<uint16_t*>(meta + so) = (uint16_t)sz;
  *reinterpret_cast<uint16_t*>(meta + so + (T == 0 ? 8 : 128)) = (uint16_t)(sz >> 16);
}

__device__ __forceinline__ void store_hat(__nv_bfloat16* hat, const Codes8& c, float s, float z) {
  const uint64_t ns2 = f2_splat(-s), z2 = f2_splat(z);
  uint4 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t x = f2_fma(c.nc[k], ns2, z2);
    (&o.x)[k] = pack_bf16x2(f2_lo(x), f2_hi(x));
  }
  *reinterpret_cast<uint4*>(hat) = o;
}

// Running bounds of a lane's eight key elements (BF16 pairs).
struct Bounds8 {
  uint32_t mn[4], mx[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 4; ++k) mn[k] = 0x7F807F80u, mx[k] = 0xFF80FF80u;  // +inf, -inf
  }
  __device__ __forceinline__ void take(const uint4& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mn[k] = u32_of(__hmin2(bf2_of(mn[k]), bf2_of((&v.x)[k])));
      mx[k] = u32_of(__hmax2(bf2_of(mx[k]), bf2_of((&v.x)[k])));
    }
  }
};

__device__ __forceinline__ void merge_store(uint2* dst, uint2 x, uint32_t mask) {
  if (mask != 0xFFFFFFFFu) {
    const uint2 old = *dst;
    x.x = (old.x & ~mask) | (x.x & mask);
    x.y = (old.y & ~mask) | (x.y & mask);
  }
  *dst = x;
}

// Row of step j of a lane, less 2 (lane / 16): rows 2t, 2t + 1, 2t + 8, 2t + 9 for
// t = lane / 16 and lane / 16 + 2.
__device__ __forceinline__ constexpr int step_row(int j) { return 4 * (j >> 2) + 8 * ((j >> 1) & 1) + (j & 1); }

// A lane's elements of the rows `nm` (bits 0..15) of a tile on their way to shared
// memory: step j to stage + 512 j, row i from src + i ld.  Each lane reads what
// it fetched itself, so no barrier is needed.
__device__ __forceinline__ void fetch_rows(uint32_t stage, const __nv_bfloat16* src, int64_t ld, uint32_t nm, int lane) {
  const int row0 = 2 * (lane >> 4);
  src += row0 * ld + 8 * (lane & 15);
  nm >>= row0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if ((nm >> step_row(j)) & 1)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(stage + 512 * j), "l"(src + step_row(j) * ld)
                   : "memory");
}

// Rows `nm` (bits 0..15) of one tile, tensor T (0 = K, 1 = V), that fetch_rows
// brought.  bnd: bounds of the rows taken (K).  Returns whether a group could not
// be held.
template <int T, int BITS, int kCode, int kMeta>
__device__ __forceinline__ bool tile_rows(uint8_t* tile, const uint8_t* stage, __nv_bfloat16* hat, int64_t ldh,
                                          uint32_t nm, int lane, Bounds8& bnd) {
  const int hw = lane >> 4, c = lane & 15, q = c >> 2, t4 = c & 3;
  // row of step j = 4 tt + 2 b + odd: 2 (2 tt + hw) + 8 b + odd
  const int row0 = 2 * hw;
  if (hat) hat += row0 * ldh + 8 * c;
  const uint32_t mine = nm >> row0;  // bit 4 tt + 8 b + odd: the lane's rows
  uint4 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = make_uint4(0u, 0u, 0u, 0u);
    if ((mine >> step_row(j)) & 1) v[j] = *reinterpret_cast<const uint4*>(stage + 512 * j);
  }
  // ---- steps and zeros: lane t4 of a group ends with steps 2 t4 and 2 t4 + 1 --
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = min_negmax(v[j]);
#pragma unroll
  for (int o = 2; o >= 1; o >>= 1) {
    const bool up = t4 & o;
#pragma unroll
    for (int i = 0; i < 2 * o; ++i) {
      const uint32_t keep = up ? m[i + 2 * o] : m[i], give = up ? m[i] : m[i + 2 * o];
      m[i] = min2(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  GroupQ gq[2];
  bool bad = false;
#pragma unroll
  for (int odd = 0; odd < 2; ++odd) {
    gq[odd] = group_q<BITS>(m[odd]);
    const int row = 4 * (t4 >> 1) + 8 * (t4 & 1) + odd;
    if ((mine >> row) & 1) {
      bad |= marked(gq[odd].r);
      store_meta<T>(tile + kMeta, row0 + row, q, gq[odd].sz);
    }
  }
  // ---- codes (rolled: the unrolled tile does not fit the instruction cache) ---
#pragma unroll 1
  for (int tt = 0; tt < 2; ++tt) {
    const uint32_t tm = mine >> (4 * tt);  // bits 0, 1, 8, 9
    uint32_t kw[2][2][2] = {};             // K: [odd][word][b]
    uint32_t vw[2][4] = {};                // V: [half of the elements][word]
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = j >> 1, odd = j & 1, from = (lane & 28) | (2 * tt + b);
      const uint32_t sz = __shfl_sync(0xffffffffu, gq[odd].sz, from);
      const float r = __shfl_sync(0xffffffffu, gq[odd].r, from);
      const float2 f = half2_to_float2(sz);
      uint4& x = v[j];
      const Codes8 cd = codes8<BITS>(x, f.x, f.y, r);
      if ((tm >> (8 * b + odd)) & 1) {
        if (T == 0) bnd.take(x);
        if (hat) store_hat(hat + (4 * tt + 8 * b + odd) * ldh, cd, f.x, f.y);
      }
      if (T == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w) kw[odd][w][b] = key_word(cd.b + 4 * w);
      } else {
        const int at = b + 2 * odd;  // row 2t + 8b + odd: byte b + 2 odd of the words
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (BITS == 4) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t* e = cd.b + 4 * half + 2 * w;
              vw[half][w] = put_byte(vw[half][w], (e[1] << 4) + e[0], at);
            }
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) vw[half][w] = put_byte(vw[half][w], cd.b[4 * half + w], at);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j + 4];
    if (T == 0) {
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        const int g = row0 + 4 * tt + odd;  // rows g and g + 8
        const bool lo = (tm >> odd) & 1, hi = (tm >> (8 + odd)) & 1;
        if (BITS == 4) {  // row g + 8 in the high nibbles of row g's words
          const uint2 x = make_uint2(kw[odd][0][0] | kw[odd][0][1] << 4, kw[odd][1][0] | kw[odd][1][1] << 4);
          if (lo || hi)
            merge_store(reinterpret_cast<uint2*>(tile + kCode + 512 * (q >> 1) + 16 * (4 * g + t4) + 8 * (q & 1)), x,
                        (lo ? 0x0F0F0F0Fu : 0u) | (hi ? 0xF0F0F0F0u : 0u));
        } else {  // a word of row g, then one of row g + 8
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint8_t* dst = tile + kCode + 512 * q + 16 * (4 * g + 2 * (c & 1) + w) + 8 * ((c >> 1) & 1);
            if (lo && hi)
              *reinterpret_cast<uint2*>(dst) = make_uint2(kw[odd][w][0], kw[odd][w][1]);
            else if (lo || hi)
              *reinterpret_cast<uint32_t*>(dst + (hi ? 4 : 0)) = kw[odd][w][hi ? 1 : 0];
          }
        }
      }
    } else {
      const uint32_t mask = ((tm & 1) ? 0xFFu : 0u) | ((tm >> 8) & 1 ? 0xFF00u : 0u) | ((tm & 2) ? 0xFF0000u : 0u) |
                            ((tm >> 9) & 1 ? 0xFF000000u : 0u);
      const int t = 2 * tt + hw;
      if (mask) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int at = 16 * (4 * (2 * t4 + half) + t);
          if (BITS == 4) {
            merge_store(reinterpret_cast<uint2*>(tile + kCode + 512 * (q >> 1) + at + 8 * (q & 1)),
                        make_uint2(vw[half][0], vw[half][1]), mask);
          } else {
            uint2* dst = reinterpret_cast<uint2*>(tile + kCode + 512 * q + at);
            merge_store(dst, make_uint2(vw[half][0], vw[half][1]), mask);
            merge_store(dst + 1, make_uint2(vw[half][2], vw[half][3]), mask);
          }
        }
      }
    }
  }
  return bad;
}

// One warp: the bound record of one (page, KV head) from the min / max of eight
// elements per lane (both half-warps hold the same elements: the first
// stores), joined with the present record unless `fresh`.  Codes at a coarser
// step follow from those at a finer one by an outward shift.
__device__ __forceinline__ void store_bounds(uint8_t* rec, int lane, const Bounds8& b, bool fresh) {
  float mn[8], mx[8], am = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = __bfloat1622float2(bf2_of(b.mn[k])), y = __bfloat1622float2(bf2_of(b.mx[k]));
    mn[2 * k] = x.x, mn[2 * k + 1] = x.y, mx[2 * k] = y.x, mx[2 * k + 1] = y.y;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) am = fmaxf(am, fmaxf(fabsf(mn[k]), fabsf(mx[k])));
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  const int c = lane & 15;
  int e = bound_exp(am), oe = 0;
  uint2 ol = make_uint2(0u, 0u), oh = ol;
  if (!fresh) {
    oe = *reinterpret_cast<const int32_t*>(rec + 256);
    ol = *reinterpret_cast<const uint2*>(rec + 8 * c);
    oh = *reinterpret_cast<const uint2*>(rec + 128 + 8 * c);
    e = max(e, oe);
  }
  __syncwarp();
  const float inv = pow2_int(min(max(-e, -126), 127));
  const int sh = min(max(e - oe, 0), 31);
  uint32_t l[2] = {0u, 0u}, h[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    int lo = (int)floorf(mn[k] * inv), hi = (int)ceilf(mx[k] * inv);
    if (!fresh) {
      const uint32_t wl = k < 4 ? ol.x : ol.y, wh = k < 4 ? oh.x : oh.y;
      lo = min(lo, (int)(int8_t)(wl >> (8 * (k & 3))) >> sh);
      hi = max(hi, -(-(int)(int8_t)(wh >> (8 * (k & 3))) >> sh));
    }
    l[k >> 2] |= ((uint32_t)lo & 0xFFu) << (8 * (k & 3));
    h[k >> 2] |= ((uint32_t)hi & 0xFFu) << (8 * (k & 3));
  }
  if (lane < 16) {
    *reinterpret_cast<uint2*>(rec + 8 * c) = make_uint2(l[0], l[1]);
    *reinterpret_cast<uint2*>(rec + 128 + 8 * c) = make_uint2(h[0], h[1]);
    if (lane == 0) *reinterpret_cast<int4*>(rec + 256) = make_int4(e, 0, 0, 0);
  }
}

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStageBytes = kWarps * 2 * 4096;

// One warp: rows r of a page, keys (T = 0) or values of KV head h.  stage: two tiles'
// worth of shared memory.
template <int BK, int BV>
__device__ __forceinline__ void append_page(const AppendParams& p, const PageRows& r, int h, int T, uint8_t* stage, int lane) {
  using F = QFmt<BK, BV>;
  const int page = *r.entry;  // not waited for before the first rows are on their way
  const int64_t ldh = (int64_t)p.HKV * HYQ_D;
  const __nv_bfloat16* src = (T == 0 ? p.k : p.v) + (int64_t)h * HYQ_D;
  __nv_bfloat16* hat = T == 0 ? p.k_hat : p.v_hat;
  if (hat) hat += (int64_t)h * HYQ_D;
  Bounds8 b;
  b.clear();
  bool bad = false;
  // The next tile's rows are on their way while one is worked on (11% faster).
  stage += 16 * lane;
  auto rows_of = [&](int tile) -> uint32_t {  // rows of the tile: bits of [r0, r1) in [16 tile, 16 tile + 16)
    const int a = max(r.r0 - 16 * tile, 0), z = min(r.r1 - 16 * tile, 16);
    return ((1u << z) - 1u) & ~((1u << a) - 1u);
  };
  const int64_t tok = (int64_t)r.tok0 - r.r0;  // call row of the page's row 0 (may lie before the call's first)
  auto fetch = [&](int tile) {
    if (16 * tile < r.r1)
      fetch_rows(smem_u32(stage) + 4096 * (tile & 1), src + (tok + 16 * tile) * p.ld, p.ld, rows_of(tile), lane);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  fetch(r.r0 >> 4);
  if (!page_ok(p, page)) {
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    return;
  }
  const size_t ph = (size_t)page * p.HKV + h;
  uint8_t* block = p.pv.pool + ph * F::kBlock;
#pragma unroll 1
  for (int tile = r.r0 >> 4; 16 * tile < r.r1; ++tile) {
    fetch(tile + 1);
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    uint8_t* tp = block + tile * F::kTile;
    const uint8_t* from = stage + 4096 * (tile & 1);
    __nv_bfloat16* to = hat ? hat + (tok + 16 * tile) * ldh : nullptr;
    if (T == 0)
      bad |= tile_rows<0, BK, 0, F::kKMeta>(tp, from, to, ldh, rows_of(tile), lane, b);
    else
      bad |= tile_rows<1, BV, F::kVCode, F::kVMeta>(tp, from, to, ldh, rows_of(tile), lane, b);
  }
  if (bad) hyq_set_err(p.pv.err, HYQ_DEVERR_QUANT_RANGE);
  if (T == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // the half-warps' rows
      b.mn[k] = u32_of(__hmin2(bf2_of(b.mn[k]), bf2_of(__shfl_xor_sync(0xffffffffu, b.mn[k], 16))));
      b.mx[k] = u32_of(__hmax2(bf2_of(b.mx[k]), bf2_of(__shfl_xor_sync(0xffffffffu, b.mx[k], 16))));
    }
    store_bounds(p.pv.bounds + ph * HYQ_BOUND_BYTES, lane, b, r.r0 == 0);
  }
}

// A block's pages: the `per` from page `first` on among those that the call's rows get, in
// the order of the rows.  Returns how many there are in all.  A row a thread (the
// loads of several rows in one thread would follow one another), 256 rows at a time.
__device__ __forceinline__ int find_pages(const AppendParams& p, int first, int per, PageRows* s_rows, int* s_warp) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kWarps) s_rows[tid].r0 = s_rows[tid].r1 = 0;  // no rows
  int before = 0;
  for (int row0 = 0; row0 < p.batch; row0 += kThreads) {
    const int row = row0 + tid;
    CallRows c;
    int n = 0;
    if (row < p.batch) {
      c = call_rows(p, row);
      if (c.bad && blockIdx.x == 0 && blockIdx.y == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
      if (c.n > 0) n = (c.start + c.n - 1) / HYQ_PAGE_ROWS - c.start / HYQ_PAGE_ROWS + 1;
    }
    int pre = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    if (row0 > 0) __syncthreads();  // the sums of the 256 rows before have been read
    if (lane == 31) s_warp[warp] = pre;
    __syncthreads();
    int at = before + pre - n;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) at += s_warp[i];
      before += s_warp[i];
    }
    for (int j = max(at - first, 0); j < per && first + j - at < n; ++j) s_rows[j] = page_rows(p, c, first + j - at);
  }
  __syncthreads();
  return before;
}

// The blocks take turns: when some of the call's rows are bad, the others may
// share rows and reach more pages than the grid was made for.  Out of line, so
// that the ordinary call's code is as if this were not (prompts in 62.4 us;
// 63.8 with the turns in a loop of the kernel).
template <int BK, int BV>
__device__ __noinline__ void append_in_turns(const AppendParams& p, int hb, uint8_t* s_stage, PageRows* s_rows,
                                             int* s_warp) {
  const int warp = threadIdx.x >> 5, per = kWarps / hb, h = blockIdx.y * hb + warp % hb;
  for (int first = (int)blockIdx.x * per;; first += (int)gridDim.x * per) {
    __syncthreads();  // the rows of the turn before have been read
    const int pages = find_pages(p, first, per, s_rows, s_warp);
    const PageRows r = s_rows[warp / hb];
    if (r.r1 > r.r0 && h < p.HKV) append_page<BK, BV>(p, r, h, blockIdx.z, s_stage + 8192 * warp, threadIdx.x & 31);
    if (first + (int)gridDim.x * per >= pages) break;
  }
}

// grid (pages that the call may reach / (8 / hb), KV heads / hb, {K, V}), with
// hb = 1, 2, 4 or 8 heads a block: a block takes 8 / hb pages that get rows, in
// the order of the call's rows, a warp for each (page, head).  Keys and values
// in blocks of their own: the warps of a block run the same code (5% faster).
template <int BK, int BV>
__global__ void __launch_bounds__(kThreads, 2) append_pages_kernel(const __grid_constant__ AppendParams p, int hb) {
  extern __shared__ __align__(16) uint8_t s_stage[];  // [kWarps][2][4096]
  __shared__ int s_warp[kThreads / 32];
  __shared__ PageRows s_rows[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  chain_kernel();
  const int per = kWarps / hb, first = (int)blockIdx.x * per;
  const int pages = find_pages(p, first, per, s_rows, s_warp);
  if (pages > (int)gridDim.x * per) return append_in_turns<BK, BV>(p, hb, s_stage, s_rows, s_warp);
  const int h = blockIdx.y * hb + warp % hb, T = blockIdx.z;
  const PageRows r = s_rows[warp / hb];
  if (r.r1 <= r.r0 || h >= p.HKV) return;
  append_page<BK, BV>(p, r, h, T, s_stage + 8192 * warp, lane);
}

// One row per sequence: a warp per (sequence, KV head), the key in its first
// half and the value in its second, eight elements a lane.
// grid (batch, KV heads / kHeadsOne)
constexpr int kHeadsOne = 4;

template <int BK, int BV>
__global__ void __launch_bounds__(32 * kHeadsOne) append_one_kernel(const AppendParams p) {
  using F = QFmt<BK, BV>;
  const int lane = threadIdx.x & 31, h = blockIdx.y * kHeadsOne + (threadIdx.x >> 5);
  chain_kernel();
  const CallRows cr = call_rows(p, blockIdx.x);
  if (cr.bad && threadIdx.x == 0 && blockIdx.y == 0) hyq_set_err(p.pv.err, HYQ_DEVERR_INDEX);
  if (cr.n <= 0 || h >= p.HKV) return;
  const PageRows pr = page_rows(p, cr, 0);
  const int T = lane >> 4, c = lane & 15, q = c >> 2, t4 = c & 3, row = pr.r0 & 15;
  uint4 v = *reinterpret_cast<const uint4*>((T == 0 ? p.k : p.v) + (int64_t)pr.tok0 * p.ld + (int64_t)h * HYQ_D + 8 * c);
  const int page = *pr.entry;
  if (!page_ok(p, page)) return;
  const size_t ph = (size_t)page * p.HKV + h;
  uint8_t* tile = p.pv.pool + ph * F::kBlock + (pr.r0 >> 4) * F::kTile;
  uint32_t m = min_negmax(v);
  m = min2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = min2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const GroupQ gq = (T == 0 ? BK : BV) == 4 ? group_q<4>(m) : group_q<8>(m);
  if (marked(gq.r)) hyq_set_err(p.pv.err, HYQ_DEVERR_QUANT_RANGE);
  const float2 f = half2_to_float2(gq.sz);
  const Codes8 cd = (T == 0 ? BK : BV) == 4 ? codes8<4>(v, f.x, f.y, gq.r) : codes8<8>(v, f.x, f.y, gq.r);
  __nv_bfloat16* hat = T == 0 ? p.k_hat : p.v_hat;
  if (hat) store_hat(hat + ((int64_t)pr.tok0 * p.HKV + h) * HYQ_D + 8 * c, cd, f.x, f.y);
  if (T == 0) {
    if (t4 == 0) store_meta<0>(tile + F::kKMeta, row, q, gq.sz);
    const int g = row & 7, b = row >> 3;
    const uint32_t w0 = key_word(cd.b), w1 = key_word(cd.b + 4);
    if (BK == 4) {
      merge_store(reinterpret_cast<uint2*>(tile + 512 * (q >> 1) + 16 * (4 * g + t4) + 8 * (q & 1)),
                  make_uint2(w0 << (4 * b), w1 << (4 * b)), 0x0F0F0F0Fu << (4 * b));
    } else {
      uint8_t* dst = tile + 512 * q + 16 * (4 * g + 2 * (c & 1)) + 8 * ((c >> 1) & 1) + 4 * b;
      *reinterpret_cast<uint32_t*>(dst) = w0;
      *reinterpret_cast<uint32_t*>(dst + 16) = w1;
    }
  } else {
    if (t4 == 0) store_meta<1>(tile + F::kVMeta, row, q, gq.sz);
    const int t = (row & 7) >> 1;
    uint8_t* dst = tile + F::kVCode + 16 * (8 * t4 + t) + (row >> 3) + 2 * (row & 1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint8_t* at = dst + 64 * half;
      if (BV == 4) {
        at += 512 * (q >> 1) + 8 * (q & 1);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t* e = cd.b + 4 * half + 2 * w;
          at[4 * w] = (uint8_t)((e[1] << 4) + e[0]);
        }
      } else {
        at += 512 * q;
#pragma unroll
        for (int w = 0; w < 4; ++w) at[4 * w] = (uint8_t)cd.b[4 * half + w];
      }
    }
  }
  // the key half's bounds, in both halves (store_bounds takes the whole warp)
  Bounds8 bnd;
#pragma unroll
  for (int k = 0; k < 4; ++k) bnd.mn[k] = bnd.mx[k] = __shfl_sync(0xffffffffu, (&v.x)[k], c);
  store_bounds(p.pv.bounds + ph * HYQ_BOUND_BYTES, lane, bnd, pr.r0 == 0);
}

template <int BK, int BV>
cudaError_t launch(const AppendParams& p, cudaStream_t s) {
  if (!p.cu)
    return hyq_launch_chained(append_one_kernel<BK, BV>, dim3(p.batch, (p.HKV + kHeadsOne - 1) / kHeadsOne),
                              32 * kHeadsOne, 0, s, p);
  // a sequence with n rows reaches at most n / 64 + 2 pages
  const int pages = p.n_rows / HYQ_PAGE_ROWS + 2 * min(p.batch, p.n_rows);
  const int hb = p.HKV >= 8 ? 8 : p.HKV > 2 ? 4 : p.HKV, per = kWarps / hb;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = hyq_once_per_device(done, [] {
    return cudaFuncSetAttribute(append_pages_kernel<BK, BV>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes);
  });
  if (e != cudaSuccess) return e;
  return hyq_launch_chained(append_pages_kernel<BK, BV>, dim3((pages + per - 1) / per, (p.HKV + hb - 1) / hb, 2), kThreads,
                            kStageBytes, s, p, hb);
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
