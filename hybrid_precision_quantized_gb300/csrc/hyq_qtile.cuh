// Attention over quantised tiles on the warp-level tensor cores, shared by the
// decode kernels: the online-softmax state of the query heads of one KV head,
// the query operands, and one 16-row tile's two products (see hyq_decode.cu
// for the method).
#pragma once

#include <math.h>

#include <type_traits>

#include "hyq_common.cuh"

namespace {

// log2(e) / sqrt(128): logits are kept in the base-2 domain.
constexpr float kScale = 0.1275174307366466f;

// Online-softmax state of one warp for the two heads (2t, 2t+1) a thread owns.
// Logits live in a scaled base-2 domain, lambda' = 2^sigma log2(e) q.k / sqrt(d)
// with one sigma per query head (QConst), chosen so that the per-group query
// sums fit the fp16 operand of the zero-point product; p = 2^((lambda' - m) 2^-sigma).
struct State {
  float m[2];       // running maximum (scaled domain)
  float nm[2];      // -m 2^-sigma (0 while m = -inf)
  float l[2];       // running sum of this thread's probabilities
  float acc[8][4];  // PV accumulators in units of 2^-24
  float zd[4];      // sum_j p_j z_jq: rows g < 4 = group g, columns heads 2t, 2t+1
};

// 2^x on the special-function unit, one instruction (relative error about
// 2^-22; 2^-inf = 0, results below 2^-126 flush to 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Online-softmax update of the two heads (2t, 2t+1) this thread owns with the
// logits of tokens (g, g+8); returns the probabilities p[2r + j].  The
// accumulators are rescaled only when some head's running max moved (the
// factor is exactly 1 otherwise).
// kLazy: first test (one warp vote) whether any logit of the tile exceeds its
// head's running maximum; if none does, the maximum stays, the correction is
// 1 and no cross-lane maximum is needed (the full path would give the same
// bits).  It pays off on long per-warp runs of tiles (one block per
// sequence and KV head), not on short ones, where early tiles move the maximum.
template <bool kLazy>
__device__ __forceinline__ void softmax_update(const float (&lg)[4], State& st, float (&p)[4],
                                               const float (&inv)[2]) {
  if (kLazy) {
    bool above = false;
#pragma unroll
    for (int j = 0; j < 2; ++j) above |= fmaxf(lg[j], lg[2 + j]) > st.m[j];
    if (!__any_sync(0xffffffffu, above)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[j] = ex2(fmaf(lg[j], inv[j], st.nm[j]));
        p[2 + j] = ex2(fmaf(lg[2 + j], inv[j], st.nm[j]));
        st.l[j] += p[j] + p[2 + j];
      }
      return;
    }
  }
  float corr[2];
  bool moved = false;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float tm = fmaxf(lg[j], lg[2 + j]);
    tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 4));
    tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 8));
    tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
    const float mn = fmaxf(st.m[j], tm);
    const float nm = (mn == -INFINITY) ? 0.f : -mn * inv[j];
    moved |= mn != st.m[j];
    corr[j] = ex2(fmaf(st.m[j], inv[j], nm));
    p[j] = ex2(fmaf(lg[j], inv[j], nm));
    p[2 + j] = ex2(fmaf(lg[2 + j], inv[j], nm));
    st.l[j] = fmaf(st.l[j], corr[j], p[j] + p[2 + j]);
    st.m[j] = mn;
    st.nm[j] = nm;
  }
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        st.acc[mt][j] *= corr[j];
        st.acc[mt][2 + j] *= corr[j];
      }
      st.zd[j] *= corr[j];
    }
  }
}

// Binary exponent e of a finite x > 0 with x = f 2^e, f in [0.5, 1)
// (subnormals included), 2^k for k in [-126, 127], and the clamp to that range.
__device__ __forceinline__ int exp_of(float x) {
  const int b = __float_as_int(x) >> 23;
  return b != 0 ? b - 126 : (__float_as_int(x * 16777216.f) >> 23) - 150;
}
__device__ __forceinline__ int clamp_exp(int k) { return min(max(k, -126), 127); }
__device__ __forceinline__ float pow2i(int k) { return __int_as_float((clamp_exp(k) + 127) << 23); }
__device__ __forceinline__ bool pos_finite(float x) { return x > 0.f && x <= 3.402823466e38f; }

// Per-block constants of the quantised path.
struct QConst {
  float ksc[2][2];  // scaled-domain factor of the code products [token g (x1) | g+8 (x16 codes)][head 2t + j]
  float inv[2];     // 2^-sigma of heads 2t, 2t+1
  float kss[2];     // scaled-domain factor of the BF16 products 2^sigma log2(e) / sqrt(d), heads 2t, 2t+1
  // B fragment of the zero-point product for head g: the scaled query sums
  // 2^sigma log2(e)/sqrt(d) sum(q over group) of groups 2(t&1), 2(t&1)+1 as
  // an fp16 pair, their high parts for t < 2 and the remainders for t >= 2
  // (hi + lo carries 22 bits).
  uint32_t bz;
};

// The two codes of bytes 1 and 3 of w as the low bytes of two 16-bit halves.
__device__ __forceinline__ uint32_t odd_bytes(uint32_t w) { return __byte_perm(w, 0u, 0x4341); }

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// `n` 32-bit words of a code region: word u of this lane at
// 512 (u / 4) + 16 lane + 4 (u % 4).
template <int n>
__device__ __forceinline__ void load_words(const uint8_t* region, int lane, uint32_t (&w)[n]) {
#pragma unroll
  for (int i = 0; i < n / 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(region + 512 * i + 16 * lane);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
}

__device__ __forceinline__ uint32_t u4c(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One 16-row quantised tile at `tb` (byte layout QFmt<BK, BV>), `vr` valid
// rows.  The codes enter the fp16 MMAs as subnormals c * 2^-24.  4-bit: the
// low nibble of a byte as c * 2^-24, the high nibble, masked in place, as
// 16 c * 2^-24; in both code orders the high nibbles are exactly fragment
// rows g+8 (K: tokens g+8; V: output rows g+8), so the factor 16 is a
// per-row constant: folded into ksc[1] for K and into the epilogue for V.
// 8-bit: bytes 0 and 2 of a word by one AND, bytes 1 and 3 by one byte
// permute, each a fragment register of two codes.  bq holds the query as
// fp16, scaled by 2^e.
//   logit = sum_q s_q (q.c)_q  (per-group code products scaled in fp32)
//         + sum_q z_q (sum q)_q (one MMA: the zero pairs against qc.bz)
//   out  += sum_j (p_j s_jq) c_jd  (P^T scaled by the V scale pairs in fp16)
//         + sum_j p_j z_jq          (one MMA: the V zero pairs against P^T)
// (the fixed-batch cache; q_tiles and q_tile_pair are the pages' forms)
template <int BK, int BV, bool kLazy>
__device__ __forceinline__ void q_tile(const uint8_t* tb, int lane, int vr, const uint32_t (&bq)[8][2],
                                       const QConst& qc, State& st) {
  using F = QFmt<BK, BV>;
  const int g = lane >> 2, t = lane & 3;
  float C[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) C[q][0] = C[q][1] = C[q][2] = C[q][3] = 0.f;
  if (BK == 4) {
    uint32_t kw[8];
    load_words<8>(tb, lane, kw);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t w = kw[ks], w8 = w >> 8;
      mma_f16(C[ks >> 1], w & 0x000F000Fu, w & 0x00F000F0u, w8 & 0x000F000Fu, w8 & 0x00F000F0u, bq[ks][0],
              bq[ks][1]);
    }
  } else {
    uint32_t kw[16];  // k-step ks: word 2ks (token g), 2ks + 1 (token g + 8)
    load_words<16>(tb, lane, kw);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t w0 = kw[2 * ks], w1 = kw[2 * ks + 1];
      mma_f16(C[ks >> 1], w0 & 0x00FF00FFu, w1 & 0x00FF00FFu, odd_bytes(w0), odd_bytes(w1), bq[ks][0], bq[ks][1]);
    }
  }
  // K metadata of tokens g and g+8: four scales, then four zeros.
  const uint4 ma = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * g);
  const uint4 mb = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * (g + 8));
  const float2 a01 = half2_to_float2(ma.x), a23 = half2_to_float2(ma.y);
  const float2 b01 = half2_to_float2(mb.x), b23 = half2_to_float2(mb.y);
  float lg[4];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    lg[c] = qc.ksc[0][c] * fmaf(a01.x, C[0][c], fmaf(a01.y, C[1][c], fmaf(a23.x, C[2][c], a23.y * C[3][c])));
    lg[2 + c] = qc.ksc[1][c] *
                fmaf(b01.x, C[0][2 + c], fmaf(b01.y, C[1][2 + c], fmaf(b23.x, C[2][2 + c], b23.y * C[3][2 + c])));
  }
  // + sum_q z_q (scaled query sum)_q: the A fragment's k slots 2t, 2t+1 are
  // groups 2(t&1), 2(t&1)+1 (high parts of the sums for t < 2, remainders
  // for t >= 2), so a lane passes the zero pair of those groups.
  mma_f16(lg, (t & 1) ? ma.w : ma.z, (t & 1) ? mb.w : mb.z, 0u, 0u, qc.bz, 0u);
  // A vertical-line position (held in BF16 elsewhere) has NaN key steps in
  // the stream: its logit is NaN, and the row is left out.
#pragma unroll
  for (int i = 0; i < 4; ++i) lg[i] = lg[i] != lg[i] ? -INFINITY : lg[i];
  if (vr < 16) {
    if (g >= vr) lg[0] = lg[1] = -INFINITY;
    if (g + 8 >= vr) lg[2] = lg[3] = -INFINITY;
  }
  float p[4];
  softmax_update<kLazy>(lg, st, p, qc.inv);
  // P^T fragments in fp16: tokens (2t, 2t+1) and (2t+8, 2t+9) of head g.
  const uint32_t pt0 = movmatrix_trans(pack_f16x2(p[0], p[1]));
  const uint32_t pt1 = movmatrix_trans(pack_f16x2(p[2], p[3]));
  const uint8_t* vm = tb + F::kVMeta;
  // V scale pairs of tokens (2t, 2t+1) and (2t+8, 2t+9), groups 0..3.
  const uint4 sv0 = *reinterpret_cast<const uint4*>(vm + 16 * t);
  const uint4 sv1 = *reinterpret_cast<const uint4*>(vm + 16 * (t + 4));
  // sum_j p_j z_jq on the tensor core: A rows = groups (g < 4), k = tokens.
  uint32_t z0 = 0u, z1 = 0u;
  if (g < 4) {
    z0 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * t + 4 * g);
    z1 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * (t + 4) + 4 * g);
  }
  mma_f16(st.zd, z0, 0u, z1, 0u, pt0, pt1);
  uint32_t vw[BV == 4 ? 8 : 16];
  load_words<BV == 4 ? 8 : 16>(tb + F::kVCode, lane, vw);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // B operand (tokens x heads) of group q: p * s in packed fp16.
    const uint32_t b0 = hmul2_u32(pt0, u4c(sv0, q)), b1 = hmul2_u32(pt1, u4c(sv1, q));
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {  // m-tile 2q + mm lies in group q
      if (BV == 4) {
        const uint32_t x = vw[2 * q + mm], x8 = x >> 8;
        mma_f16(st.acc[2 * q + mm], x & 0x000F000Fu, x & 0x00F000F0u, x8 & 0x000F000Fu, x8 & 0x00F000F0u, b0, b1);
      } else {  // m-tile mt: words 2mt (fragment rows g) and 2mt + 1 (rows g + 8)
        const uint32_t y0 = vw[2 * (2 * q + mm)], y1 = vw[2 * (2 * q + mm) + 1];
        mma_f16(st.acc[2 * q + mm], y0 & 0x00FF00FFu, y1 & 0x00FF00FFu, odd_bytes(y0), odd_bytes(y1), b0, b1);
      }
    }
  }
}

// ---- pages ----------------------------------------------------------------------
// A probability enters the value product in fp16, and so does its product with the
// value step: both are kept at the upper end of what fp16 holds, whatever the
// values' size, so that the small ones are not lost below it.  (With p at most 1 and
// p s as it came, an output made of rows 12 nats below one large and empty row was off by
// 0.28 of its size for 8-bit values of standard deviation 0.3 and by more than its
// size from 0.1 down, for 4-bit ones by 0.11 at 0.02; now by 0.002, its rounding to BF16.)
//
// p.  The reference that a row's logits are taken from stands below a logit near
// the row's maximum, so that p comes near 2^15.  It may lag: it moves (and the
// accumulators are rescaled) only when some p would pass 2^top, top = 15, and then
// to where that p is 2^(top - kSlack).  The first maximum of a row is seldom its
// last, so without the slack short runs of tiles rescale at most of their tiles (4-bit
// codes, 64 query rows a KV head, 32 sequences of up to 2000: 99 us with a slack of 2, 90
// with 6; p is rounded to half a step of fp16 down to 2^-23 of the row's largest).
// Each row's reference moves for its own logits alone: its result does not depend
// on the rows that share its tile.  Sums and zero-point terms are of the same p.
//
// p s.  A warp takes the steps times a power of two 2^F >= 1 such that the
// largest that it has met lies below 2: p s stays within 65504.  When a larger one
// comes, F falls, to where that step lies in [0.5, 1), and the accumulators with
// it.  Steps from 2 on (values that span 30, or 510 with 8-bit codes) lower top
// instead: a step made smaller could leave fp16, beside others that are not large.
// One lane scales each word of a tile's steps, in shared memory, before all read
// them (one sequence of 1000 positions: 9.37 us without any of this, 9.57 with it,
// 9.61 when each lane scaled the eight words that it read; drafts of 8-bit codes 65.5,
// 66.8, 67.9).
constexpr float kSlack = 6.f;

// Of N query tiles and one warp, for the heads (2t, 2t+1) that a thread owns.
template <int N>
struct PageState {
  float nm[N][2];      // minus the reference in log2 units (kNoMax before the first)
  float l[N][2];       // running sums of this thread's probabilities
  float acc[N][8][4];  // value products in units of 2^-24 2^F
  float zd[N][4];      // sum_j p_j z_jq: rows g < 4 = group g, columns heads 2t, 2t+1
  uint32_t lim;        // the largest step that F and top allow (its bits, twice)
  float top;
};
constexpr float kNoMax = 3.402823466e38f;  // finite: a masked logit less it is still minus infinity

template <int N>
__device__ __forceinline__ void reset_state(PageState<N>& st) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    st.nm[k][0] = st.nm[k][1] = kNoMax;
    st.l[k][0] = st.l[k][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) st.acc[k][mt][0] = st.acc[k][mt][1] = st.acc[k][mt][2] = st.acc[k][mt][3] = 0.f;
    st.zd[k][0] = st.zd[k][1] = st.zd[k][2] = st.zd[k][3] = 0.f;
  }
  st.lim = 0x03FF03FFu;  // subnormal steps: F = 15
  st.top = 15.f;
}

// A step's bits ascend with its value.  The limit of F >= 0 has the exponent
// field 15 - F (the steps below 2 2^-F), that of a lowered top 30 - top.
constexpr uint32_t kLimitF0 = 0x3FFFu;
__device__ __forceinline__ bool above_limit(uint32_t steps, uint32_t lim) { return __vmaxu2(steps, lim) != lim; }
// The largest of all lanes' steps.
__device__ __forceinline__ uint32_t most_step(uint32_t steps) {
  return __reduce_max_sync(0xffffffffu, max(steps & 0xFFFFu, steps >> 16));
}
// 2^F, twice in fp16.
__device__ __forceinline__ uint32_t step_scale(uint32_t lim) { return __vmaxu2(0x7BFF7BFFu - lim, 0x3C003C00u); }
// 2^F of one limit (one half) over 2^F of another.
__device__ __forceinline__ float scale_ratio(uint32_t a, uint32_t b) {
  return __int_as_float(0x3F800000 + (int)((min(b, kLimitF0) - min(a, kLimitF0)) << 13));
}
// The limit for a step `most`: one above the present limit comes to lie in [0.5, 1) times 2^F.
// Returns the change of F, which the value products take; top falls by `fell`.
template <int N>
__device__ __forceinline__ float raise_limit(uint32_t most, PageState<N>& st, float& fell) {
  const uint32_t was = st.lim & 0xFFFFu, lim = most > was ? min((most | 0x3FFu) + 0x400u, 0x7BFFu) : was;
  st.lim = lim * 0x00010001u;
  const float top = (float)(30 - (int)(max(lim, kLimitF0) >> 10));
  fell = st.top - top;
  st.top = top;
  return scale_ratio(lim, was);
}

// Query tile k's part of a raise: the reference of head 2t + j moves if one of its logits (tm: the
// lane's largest, times inv = 2^-sigma) lies more than top above it, and by what top fell.
template <int N>
__device__ __forceinline__ void raise_head(PageState<N>& st, int k, int j, float tm, float inv, float fell, float fc) {
  tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 4));
  tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 8));
  tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
  // inv is a power of two: the products are exact, and the sum rounded down keeps
  // the largest p within 2^(top - kSlack)
  const float old = st.nm[k][j], low = old - fell;
  const float nm = fmaf(tm, inv, low) > st.top ? __fadd_rd(fmaxf(st.top - kSlack, 0.f), -tm * inv) : low;
  const float corr = ex2(nm - old), ca = corr * fc;
  st.nm[k][j] = nm;
  st.l[k][j] *= corr;
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    st.acc[k][mt][j] *= ca;
    st.acc[k][mt][2 + j] *= ca;
  }
  st.zd[k][j] *= corr;
}

// The halves of a word about rows r, r + 1 that lie below vr.
__device__ __forceinline__ uint32_t rows_below(int r, int vr) {
  return (r < vr ? 0xFFFFu : 0u) | (r + 1 < vr ? 0xFFFF0000u : 0u);
}

// q_tile's products for NT adjacent tiles of a page: the tiles' independent chains
// overlap, and reference and steps are tested once for all of them.
//
// kRows: the tile may lie at the end of what some query row sees, and its
// rows past `vr` may hold anything (a page is reused without being cleared):
// heads 2t, 2t+1 see the first vh0, vh1 rows, and the value metadata of
// the rows past vr, which could be infinite or NaN, is taken as zero (their
// probabilities are zero, and so must be their products).  Otherwise every row is
// seen by every query row.  A NaN logit is its query's own and goes on to its output.
template <int BK, int BV, int NT, bool kRows = false>
__device__ __forceinline__ void q_tiles(uint8_t* tb0, int lane, const uint32_t (&bq)[8][2], const QConst& qc,
                                        PageState<1>& st, int vr = 16, int vh0 = 16, int vh1 = 16) {
  using F = QFmt<BK, BV>;
  static_assert(!kRows || NT == 1, "rows are left out of one tile at a time");
  const int g = lane >> 2, t = lane & 3;
  float lg[NT][4];
  uint32_t step[NT];  // the steps of rows 2g, 2g + 1 and group t
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint8_t* tb = tb0 + n * F::kTile;
    float C[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) C[q][0] = C[q][1] = C[q][2] = C[q][3] = 0.f;
    if (BK == 4) {
      uint32_t kw[8];
      load_words<8>(tb, lane, kw);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t w = kw[ks], w8 = w >> 8;
        mma_f16(C[ks >> 1], w & 0x000F000Fu, w & 0x00F000F0u, w8 & 0x000F000Fu, w8 & 0x00F000F0u, bq[ks][0],
                bq[ks][1]);
      }
    } else {
      uint32_t kw[16];
      load_words<16>(tb, lane, kw);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t w0 = kw[2 * ks], w1 = kw[2 * ks + 1];
        mma_f16(C[ks >> 1], w0 & 0x00FF00FFu, w1 & 0x00FF00FFu, odd_bytes(w0), odd_bytes(w1), bq[ks][0], bq[ks][1]);
      }
    }
    const uint4 ma = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * g);
    const uint4 mb = *reinterpret_cast<const uint4*>(tb + F::kKMeta + 16 * (g + 8));
    const float2 a01 = half2_to_float2(ma.x), a23 = half2_to_float2(ma.y);
    const float2 b01 = half2_to_float2(mb.x), b23 = half2_to_float2(mb.y);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      lg[n][c] =
          qc.ksc[0][c] * fmaf(a01.x, C[0][c], fmaf(a01.y, C[1][c], fmaf(a23.x, C[2][c], a23.y * C[3][c])));
      lg[n][2 + c] = qc.ksc[1][c] * fmaf(b01.x, C[0][2 + c],
                                         fmaf(b01.y, C[1][2 + c], fmaf(b23.x, C[2][2 + c], b23.y * C[3][2 + c])));
    }
    mma_f16(lg[n], (t & 1) ? ma.w : ma.z, (t & 1) ? mb.w : mb.z, 0u, 0u, qc.bz, 0u);
    if (kRows) {
      if (g >= vh0) lg[n][0] = -INFINITY;
      if (g >= vh1) lg[n][1] = -INFINITY;
      if (g + 8 >= vh0) lg[n][2] = -INFINITY;
      if (g + 8 >= vh1) lg[n][3] = -INFINITY;
    }
    step[n] = *reinterpret_cast<const uint32_t*>(tb + F::kVMeta + 4 * lane);
    if (kRows) step[n] &= rows_below(2 * g, vr);
  }
  // ---- reference and steps ---------------------------------------------------
  float x[NT][4];  // logits less the reference, in log2 units
  uint32_t steps = step[0];
#pragma unroll
  for (int n = 1; n < NT; ++n) steps = __vmaxu2(steps, step[n]);
  const uint32_t most = most_step(steps);
  bool above = most > (st.lim >> 16);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[n][i] = fmaf(lg[n][i], qc.inv[i & 1], st.nm[0][i & 1]);
    above |= fmaxf(fmaxf(x[n][0], x[n][1]), fmaxf(x[n][2], x[n][3])) > st.top;
  }
  if (__any_sync(0xffffffffu, above)) {
    float fell;
    const float fc = raise_limit(most, st, fell);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float tm = fmaxf(lg[0][j], lg[0][2 + j]);
#pragma unroll
      for (int n = 1; n < NT; ++n) tm = fmaxf(tm, fmaxf(lg[n][j], lg[n][2 + j]));
      raise_head(st, 0, j, tm, qc.inv[j], fell, fc);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        x[n][j] = fmaf(lg[n][j], qc.inv[j], st.nm[0][j]);
        x[n][2 + j] = fmaf(lg[n][2 + j], qc.inv[j], st.nm[0][j]);
      }
    }
  }
  // the steps times 2^F, in their place: a lane's own word, read by all below
  const uint32_t f2 = step_scale(st.lim);
#pragma unroll
  for (int n = 0; n < NT; ++n)
    *reinterpret_cast<uint32_t*>(tb0 + n * F::kTile + F::kVMeta + 4 * lane) = hmul2_u32(step[n], f2);
  __syncwarp();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint8_t* tb = tb0 + n * F::kTile;
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ex2(x[n][i]);
    st.l[0][0] += p[0] + p[2];
    st.l[0][1] += p[1] + p[3];
    const uint32_t pt0 = movmatrix_trans(pack_f16x2(p[0], p[1]));
    const uint32_t pt1 = movmatrix_trans(pack_f16x2(p[2], p[3]));
    const uint8_t* vm = tb + F::kVMeta;
    const uint4 sv0 = *reinterpret_cast<const uint4*>(vm + 16 * t);
    const uint4 sv1 = *reinterpret_cast<const uint4*>(vm + 16 * (t + 4));
    // rows g < 4 carry the zeros of group g; rows 4 .. 7 repeat them and are not used
    uint32_t z0 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * t + 4 * (g & 3));
    uint32_t z1 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * (t + 4) + 4 * (g & 3));
    if (kRows) {  // (the steps of those rows are zero already)
      z0 &= rows_below(2 * t, vr);
      z1 &= rows_below(2 * t + 8, vr);
    }
    mma_f16(st.zd[0], z0, 0u, z1, 0u, pt0, pt1);
    uint32_t vw[BV == 4 ? 8 : 16];
    load_words<BV == 4 ? 8 : 16>(tb + F::kVCode, lane, vw);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t b0 = hmul2_u32(pt0, u4c(sv0, q)), b1 = hmul2_u32(pt1, u4c(sv1, q));
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        if (BV == 4) {
          const uint32_t x = vw[2 * q + mm], x8 = x >> 8;
          mma_f16(st.acc[0][2 * q + mm], x & 0x000F000Fu, x & 0x00F000F0u, x8 & 0x000F000Fu, x8 & 0x00F000F0u, b0, b1);
        } else {
          const uint32_t y0 = vw[2 * (2 * q + mm)], y1 = vw[2 * (2 * q + mm) + 1];
          mma_f16(st.acc[0][2 * q + mm], y0 & 0x00FF00FFu, y1 & 0x00FF00FFu, odd_bytes(y0), odd_bytes(y1), b0, b1);
        }
      }
    }
  }
}

// q_tile_pair: two tiles of query rows at once, their operands in shared
// memory, laid out so that a lane's parts lie at constant offsets from two
// addresses (the loop has no registers to spare for more):
//   [0, 2048)     bq_s, 16 bytes per k-step pair and lane
//   [2048, 2112)  per t: the code-product factor and 2^-sigma of head 2t, then of 2t + 1
//   [2112, 2240)  per lane: the zero-point fragment
constexpr int kPairQuery = 2240;  // bytes of a query tile

// The lane's constants of a query tile from what prep_query_row left.
__device__ __forceinline__ void spread_query_consts(uint8_t* query, int lane, const float (&rowc_s)[HYQ_MAX_GQA][4],
                                                    const uint32_t (&bz_s)[HYQ_MAX_GQA][4]) {
  const int g = lane >> 2, t = lane & 3;
  const float *a = rowc_s[2 * t], *b = rowc_s[2 * t + 1];
  if (g == 0) *reinterpret_cast<float4*>(query + 2048 + 16 * t) = make_float4(a[0], a[2], b[0], b[2]);
  *reinterpret_cast<uint32_t*>(query + 2112 + 4 * lane) = bz_s[g][t];
}

// Loads from a shared memory address in a register, at a constant offset.  (An
// address formed from a shared variable's name costs three instructions and a
// special register each time that the compiler forms it anew.)
template <int kOff>
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a), "n"(kOff));
  return v;
}
template <int kOff>
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1 + %2];\n" : "=r"(v) : "r"(a), "n"(kOff));
  return v;
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(a), "r"(v) : "memory");
}

// One 16-row tile at address `tb` for two query tiles: a tile's codes are unpacked
// and its scales converted once for both.  query: address of the first query tile's
// operands; scaled: 128 bytes of the warp's own (two warps read a tile, each with
// an F of its own).  kRows as in q_tiles, with lim_s[k] the rows that query
// tile k's heads see, less `at`.
template <int BK, int BV, bool kRows>
__device__ __forceinline__ void q_tile_pair(uint32_t tb, int lane, uint32_t query, int vr,
                                            const int (*lim_s)[HYQ_MAX_GQA], int at, uint32_t scaled, PageState<2>& st) {
  using F = QFmt<BK, BV>;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t tl = tb + 16 * lane, tg = tb + 16 * g, tt = tb + 16 * t, tz = tt + 4 * (g & 3);
  const uint32_t qa = query + 16 * lane, qt = query + 16 * t, qz = query + 4 * lane;
  float lg[2][4];
  const uint4 ma = lds128<F::kKMeta>(tg), mb = lds128<F::kKMeta + 128>(tg);
  // group by group, each scaled as soon as its two products are there: few
  // accumulators are alive at a time
  auto key_group = [&](auto group) {
    constexpr int q = decltype(group)::value;
    const uint4 w = lds128<512 * (BK == 8 ? q : q >> 1)>(tl);
    const uint4 b0 = lds128<512 * q>(qa), b1 = lds128<kPairQuery + 512 * q>(qa);
    float C[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) C[k][0] = C[k][1] = C[k][2] = C[k][3] = 0.f;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t x0, x1, x2, x3;
      if (BK == 4) {
        const uint32_t v = u4c(w, 2 * (q & 1) + hf), v8 = v >> 8;
        x0 = v & 0x000F000Fu, x1 = v & 0x00F000F0u, x2 = v8 & 0x000F000Fu, x3 = v8 & 0x00F000F0u;
      } else {
        const uint32_t w0 = u4c(w, 2 * hf), w1 = u4c(w, 2 * hf + 1);
        x0 = w0 & 0x00FF00FFu, x1 = w1 & 0x00FF00FFu, x2 = odd_bytes(w0), x3 = odd_bytes(w1);
      }
      mma_f16(C[0], x0, x1, x2, x3, hf ? b0.z : b0.x, hf ? b0.w : b0.y);
      mma_f16(C[1], x0, x1, x2, x3, hf ? b1.z : b1.x, hf ? b1.w : b1.y);
    }
    // the group's steps of tokens g and g + 8
    const float2 fa = half2_to_float2(q < 2 ? ma.x : ma.y), fb = half2_to_float2(q < 2 ? mb.x : mb.y);
    const float sa = q & 1 ? fa.y : fa.x, sb = q & 1 ? fb.y : fb.x;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        lg[k][c] = q == 3 ? sa * C[k][c] : fmaf(sa, C[k][c], lg[k][c]);
        lg[k][2 + c] = q == 3 ? sb * C[k][2 + c] : fmaf(sb, C[k][2 + c], lg[k][2 + c]);
      }
  };
  key_group(std::integral_constant<int, 3>{});
  key_group(std::integral_constant<int, 2>{});
  key_group(std::integral_constant<int, 1>{});
  key_group(std::integral_constant<int, 0>{});
  const uint32_t za = (t & 1) ? ma.w : ma.z, zb = (t & 1) ? mb.w : mb.z;
  float x[2][4];  // logits less the reference, in log2 units
  uint32_t step = lds32<F::kVMeta>(tb + 4 * lane);  // of rows 2g, 2g + 1 and group t
  if (kRows) step &= rows_below(2 * g, vr);
  bool above = above_limit(step, st.lim);
  auto logits = [&](auto tile) {
    constexpr int k = decltype(tile)::value;
    float(&l)[4] = lg[k];
    const uint4 c = lds128<kPairQuery * k + 2048>(qt);
    const float f0 = __uint_as_float(c.x), f1 = __uint_as_float(c.z);
    constexpr float kHigh = BK == 4 ? 0.0625f : 1.f;  // 4-bit tokens g + 8 carry 16 c
    l[0] *= f0, l[1] *= f1, l[2] *= f0 * kHigh, l[3] *= f1 * kHigh;
    mma_f16(l, za, zb, 0u, 0u, lds32<kPairQuery * k + 2112>(qz), 0u);
    if (kRows) {
      const int v0 = lim_s[k][2 * t] - at, v1 = lim_s[k][2 * t + 1] - at;
      if (g >= v0) l[0] = -INFINITY;
      if (g >= v1) l[1] = -INFINITY;
      if (g + 8 >= v0) l[2] = -INFINITY;
      if (g + 8 >= v1) l[3] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k][i] = fmaf(l[i], __uint_as_float(i & 1 ? c.w : c.y), st.nm[k][i & 1]);
    above |= fmaxf(fmaxf(x[k][0], x[k][1]), fmaxf(x[k][2], x[k][3])) > st.top;
  };
  logits(std::integral_constant<int, 0>{});
  logits(std::integral_constant<int, 1>{});
  if (__any_sync(0xffffffffu, above)) {
    float fell;
    const float fc = raise_limit(most_step(step), st, fell);
    auto raise = [&](auto tile) {
      constexpr int k = decltype(tile)::value;
      const uint4 c = lds128<kPairQuery * k + 2048>(qt);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float inv = __uint_as_float(j ? c.w : c.y);
        raise_head(st, k, j, fmaxf(lg[k][j], lg[k][2 + j]), inv, fell, fc);
        x[k][j] = fmaf(lg[k][j], inv, st.nm[k][j]);
        x[k][2 + j] = fmaf(lg[k][2 + j], inv, st.nm[k][j]);
      }
    };
    raise(std::integral_constant<int, 0>{});
    raise(std::integral_constant<int, 1>{});
  }
  sts32(scaled + 4 * lane, hmul2_u32(step, step_scale(st.lim)));
  uint32_t pt0[2], pt1[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ex2(x[k][i]);
    st.l[k][0] += p[0] + p[2];
    st.l[k][1] += p[1] + p[3];
    pt0[k] = movmatrix_trans(pack_f16x2(p[0], p[1]));
    pt1[k] = movmatrix_trans(pack_f16x2(p[2], p[3]));
  }
  __syncwarp();  // the scaled steps are there
  const uint4 sv0 = lds128<0>(scaled + 16 * t), sv1 = lds128<64>(scaled + 16 * t);
  // rows g < 4 carry the zeros of group g; rows 4 .. 7 repeat them and are not used
  uint32_t z0 = lds32<F::kVMeta + 128>(tz), z1 = lds32<F::kVMeta + 192>(tz);
  if (kRows) {  // (the steps of those rows are zero already)
    z0 &= rows_below(2 * t, vr);
    z1 &= rows_below(2 * t + 8, vr);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) mma_f16(st.zd[k], z0, 0u, z1, 0u, pt0[k], pt1[k]);
  auto value_group = [&](auto group) {
    constexpr int q = decltype(group)::value;
    const uint4 w = lds128<F::kVCode + 512 * (BV == 8 ? q : q >> 1)>(tl);
    uint32_t b0[2], b1[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) b0[k] = hmul2_u32(pt0[k], u4c(sv0, q)), b1[k] = hmul2_u32(pt1[k], u4c(sv1, q));
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {
      uint32_t x0, x1, x2, x3;
      if (BV == 4) {
        const uint32_t v = u4c(w, 2 * (q & 1) + mm), v8 = v >> 8;
        x0 = v & 0x000F000Fu, x1 = v & 0x00F000F0u, x2 = v8 & 0x000F000Fu, x3 = v8 & 0x00F000F0u;
      } else {
        const uint32_t y0 = u4c(w, 2 * mm), y1 = u4c(w, 2 * mm + 1);
        x0 = y0 & 0x00FF00FFu, x1 = y1 & 0x00FF00FFu, x2 = odd_bytes(y0), x3 = odd_bytes(y1);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) mma_f16(st.acc[k][2 * q + mm], x0, x1, x2, x3, b0[k], b1[k]);
    }
  };
  value_group(std::integral_constant<int, 0>{});
  value_group(std::integral_constant<int, 1>{});
  value_group(std::integral_constant<int, 2>{});
  value_group(std::integral_constant<int, 3>{});
}

// A query row's operands: its fp16 B fragments (bq_s), scaled by an exact
// power of two 2^qe so that max |q| lies in [2^13, 2^14), stored in the order
// lane (g, t) reads them; and its constants: sigma (its largest scaled group
// sum 2^sigma log2(e)/sqrt(d) |sum q| below 2^13, and sigma <= 23 -
// exponent(max |q|), which bounds the scaled logits), the code-product
// factors (rowc_s) and the zero-point fragments (bz_s).  One warp per row r;
// v: the lane's four BF16 query elements 4 lane .. 4 lane + 3.
template <int BK>
__device__ __forceinline__ void prep_query_row(int r, int lane, uint2 v, uint32_t (&bq_s)[4][HYQ_MAX_GQA][4][4],
                                               float (&rowc_s)[HYQ_MAX_GQA][4], uint32_t (&bz_s)[HYQ_MAX_GQA][4]) {
  const float2 x01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
  const float2 x23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
  const float x[4] = {x01.x, x01.y, x23.x, x23.y};
  float gs = (x[0] + x[1]) + (x[2] + x[3]);  // group lane / 8
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) gs += __shfl_xor_sync(0xffffffffu, gs, o);
  float am = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  float gm = fabsf(gs * kScale);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  const int qe = pos_finite(am) ? clamp_exp(14 - exp_of(am)) : 14;
  const float gmb = fmaxf(gm, am * 0.0009765625f);  // 2^-10 max |q|
  const int sg = pos_finite(gmb) ? clamp_exp(13 - exp_of(gmb)) : 13;
  const float qscale = pow2i(qe);
#pragma unroll
  for (int hp = 0; hp < 2; ++hp) {
    const int e = 4 * lane + 2 * hp;  // pair (e, e + 1) -> lane t, k-step ks, half hh
    const int hh = (e >> 1) & 1;
    const int tt = BK == 4 ? (e >> 3) & 3 : (e >> 2) & 3;
    const int ks = BK == 4 ? 2 * (e >> 5) + ((e >> 2) & 1) : e >> 4;
    bq_s[ks >> 1][r][tt][2 * (ks & 1) + hh] = pack_f16x2(x[2 * hp] * qscale, x[2 * hp + 1] * qscale);
  }
  const float kss = kScale * pow2i(sg);
  const float s0 = __shfl_sync(0xffffffffu, gs, 0) * kss, s1 = __shfl_sync(0xffffffffu, gs, 8) * kss;
  const float s2 = __shfl_sync(0xffffffffu, gs, 16) * kss, s3 = __shfl_sync(0xffffffffu, gs, 24) * kss;
  if (lane < 4) {  // lane = t of the reading thread
    const float y0 = (lane & 1) ? s2 : s0, y1 = (lane & 1) ? s3 : s1;
    const float h0 = __half2float(__float2half_rn(y0)), h1 = __half2float(__float2half_rn(y1));
    bz_s[r][lane] = lane < 2 ? pack_f16x2(h0, h1) : pack_f16x2(y0 - h0, y1 - h1);
  }
  if (lane == 0) {
    const float k0 = kScale * 4096.f * (pow2i(12 - qe) * pow2i(sg));  // 2^(24 - qe) alone can leave float32
    rowc_s[r][0] = k0;
    rowc_s[r][1] = BK == 4 ? k0 * 0.0625f : k0;  // 4-bit tokens g+8 carry 16 c
    rowc_s[r][2] = pow2i(-sg);
    rowc_s[r][3] = kss;
  }
}

// B fragments of q in the permuted k order of the key codes (k-step ks covers
// elements e + {0,1} and e + {2,3}, e = 8(t + 4(ks/2)) + 4(ks%2) for 4-bit
// keys, e = 16 ks + 4t for 8-bit keys) and the constants of a lane's heads.
__device__ __forceinline__ void load_query_consts(int g, int t, const uint32_t (&bq_s)[4][HYQ_MAX_GQA][4][4],
                                                  const float (&rowc_s)[HYQ_MAX_GQA][4],
                                                  const uint32_t (&bz_s)[HYQ_MAX_GQA][4], uint32_t (&bq)[8][2],
                                                  QConst& qc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(&bq_s[i][g][t][0]);
    bq[2 * i][0] = v.x, bq[2 * i][1] = v.y, bq[2 * i + 1][0] = v.z, bq[2 * i + 1][1] = v.w;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    qc.ksc[0][j] = rowc_s[2 * t + j][0];
    qc.ksc[1][j] = rowc_s[2 * t + j][1];
    qc.inv[j] = rowc_s[2 * t + j][2];
    qc.kss[j] = rowc_s[2 * t + j][3];
  }
  qc.bz = bz_s[g][t];
}

__device__ __forceinline__ void reset_state(State& st) {
  st.m[0] = st.m[1] = -INFINITY;
  st.nm[0] = st.nm[1] = 0.f;
  st.l[0] = st.l[1] = 0.f;
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) st.acc[mt][0] = st.acc[mt][1] = st.acc[mt][2] = st.acc[mt][3] = 0.f;
  st.zd[0] = st.zd[1] = st.zd[2] = st.zd[3] = 0.f;
}

// A warp's partial result to shared memory: acc[head][128] with the
// zero-point terms in wpart ([8 heads][128] = 4 KB; element d of head hd at
// hd*128 + (d ^ (hd/2)), so that the 32 lanes' stores of one accumulator
// fall in 32 banks), what the probabilities are relative to (m: log2 units) and
// their sum per head.  unit: of the accumulators, times 2^24.
template <int BV>
__device__ __forceinline__ void store_partial(const float (&acc)[8][4], const float (&zd)[4], float (&l)[2], float m0,
                                              float m1, float unit, int g, int t, float* wpart,
                                              float (&red_m)[HYQ_MAX_GQA], float (&red_l)[HYQ_MAX_GQA]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], o);
  // sum_j p_j z_jq of heads 2t, 2t+1 sits in lane (q, t): gather all four groups.
  float zt[4][2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    zt[q][0] = __shfl_sync(0xffffffffu, zd[0], 4 * q + t);
    zt[q][1] = __shfl_sync(0xffffffffu, zd[1], 4 * q + t);
  }
  // Accumulator (m-tile u, ci) of thread (g, t): element 32(u/2) + 4g +
  // 2(u%2) + (ci >> 1), head 2t + (ci & 1); with 4-bit values the rows
  // ci >= 2 carry 16 c.
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int ci = 0; ci < 4; ++ci) {
      const int d = 32 * (u >> 1) + 4 * g + 2 * (u & 1) + (ci >> 1), hd = 2 * t + (ci & 1);
      const float f = (BV == 4 && ci >= 2) ? unit / 16.f : unit;
      wpart[hd * HYQ_D + (d ^ t)] = fmaf(acc[u][ci], f, zt[u >> 1][ci & 1]);
    }
  if (g == 0) {
    red_m[2 * t] = m0, red_m[2 * t + 1] = m1;
    red_l[2 * t] = l[0], red_l[2 * t + 1] = l[1];
  }
}
template <int BV>
__device__ __forceinline__ void store_warp_partial(State& st, const QConst& qc, int g, int t, float* wpart,
                                                   float (&red_m)[HYQ_MAX_GQA], float (&red_l)[HYQ_MAX_GQA]) {
  float m[2];  // back to log2 units
#pragma unroll
  for (int j = 0; j < 2; ++j) m[j] = st.m[j] == -INFINITY ? -INFINITY : st.m[j] * qc.inv[j];
  store_partial<BV>(st.acc, st.zd, st.l, m[0], m[1], HYQ_F16_SUB_SCALE, g, t, wpart, red_m, red_l);
}
// Query tile k of a warp.
template <int BV, int N>
__device__ __forceinline__ void store_warp_partial(PageState<N>& st, int k, int g, int t, float* wpart,
                                                   float (&red_m)[HYQ_MAX_GQA], float (&red_l)[HYQ_MAX_GQA]) {
  float m[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) m[j] = st.nm[k][j] == kNoMax ? -INFINITY : -st.nm[k][j];
  const float unit = HYQ_F16_SUB_SCALE * scale_ratio(kLimitF0, st.lim & 0xFFFFu);
  store_partial<BV>(st.acc[k], st.zd[k], st.l[k], m[0], m[1], unit, g, t, wpart, red_m, red_l);
}

}  // namespace
