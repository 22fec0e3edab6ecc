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
//
// kRows: the tile may lie at the end of what some query row sees, and its
// rows past `vr` may hold anything (a page is reused without being cleared):
// heads 2t, 2t+1 see the first vh[0], vh[1] rows, and the value metadata of
// the rows past vr, which could be infinite or NaN, is taken as zero (their
// probabilities are zero, and so must be their products).
template <int BK, int BV, bool kLazy, bool kRows = false>
__device__ __forceinline__ void q_tile(const uint8_t* tb, int lane, int vr, const uint32_t (&bq)[8][2],
                                       const QConst& qc, State& st, int vh0 = 16, int vh1 = 16) {
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
  // the stream: its logit is NaN, and the row is left out.  Pages (kRows) hold no
  // such rows: there a NaN is the query's own and goes on to its output.
  if (!kRows) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lg[i] = lg[i] != lg[i] ? -INFINITY : lg[i];
  }
  if (kRows) {
    if (g >= vh0) lg[0] = -INFINITY;
    if (g >= vh1) lg[1] = -INFINITY;
    if (g + 8 >= vh0) lg[2] = -INFINITY;
    if (g + 8 >= vh1) lg[3] = -INFINITY;
  } else if (vr < 16) {
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
  uint4 sv0 = *reinterpret_cast<const uint4*>(vm + 16 * t);
  uint4 sv1 = *reinterpret_cast<const uint4*>(vm + 16 * (t + 4));
  // sum_j p_j z_jq on the tensor core: A rows = groups (g < 4), k = tokens.
  uint32_t z0 = 0u, z1 = 0u;
  if (g < 4) {
    z0 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * t + 4 * g);
    z1 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * (t + 4) + 4 * g);
  }
  if (kRows) {
    // the halves of the pair (2t, 2t+1), and of (2t+8, 2t+9), that lie below vr
    const uint32_t k0 = (2 * t < vr ? 0xFFFFu : 0u) | (2 * t + 1 < vr ? 0xFFFF0000u : 0u);
    const uint32_t k1 = (2 * t + 8 < vr ? 0xFFFFu : 0u) | (2 * t + 9 < vr ? 0xFFFF0000u : 0u);
    sv0.x &= k0, sv0.y &= k0, sv0.z &= k0, sv0.w &= k0, z0 &= k0;
    sv1.x &= k1, sv1.y &= k1, sv1.z &= k1, sv1.w &= k1, z1 &= k1;
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

// The running maximum of q_tiles and q_tile_pair is a reference that may lag:
// it moves (and the accumulators are rescaled) only when a logit passes it by
// more than kSlack<BV> in log2 units.  A probability is then at most 2^kSlack,
// and p s still fits fp16: s is at most 2 * 65504 / qmax, 8734 for 4-bit and 514
// for 8-bit values.  The first maximum of a row is seldom its last, so without
// the slack short runs of tiles rescale at most of their tiles.  Each row's
// maximum moves for its own logits alone: its result does not depend on the rows
// that share its tile.
template <int BV>
constexpr float kSlack = BV == 4 ? 2.f : 6.f;
// The slack in the scaled domain of a row with inv = 2^-sigma.
template <int BV>
__device__ __forceinline__ float slack_of(float inv) {
  return kSlack<BV> * __int_as_float((254 << 23) - __float_as_int(inv));
}

// q_tile for NT adjacent tiles, every row seen by every query row and no row
// left out by NaN steps: the tiles' independent chains overlap, and the
// running maximum is tested once for all of them.
template <int BK, int BV, int NT>
__device__ __forceinline__ void q_tiles(const uint8_t* tb0, int lane, const uint32_t (&bq)[8][2], const QConst& qc,
                                        State& st) {
  using F = QFmt<BK, BV>;
  const int g = lane >> 2, t = lane & 3;
  float lg[NT][4];
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
  }
  // ---- running maximum ------------------------------------------------------
  float tm[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    tm[j] = fmaxf(lg[0][j], lg[0][2 + j]);
#pragma unroll
    for (int n = 1; n < NT; ++n) tm[j] = fmaxf(tm[j], fmaxf(lg[n][j], lg[n][2 + j]));
  }
  if (__any_sync(0xffffffffu, tm[0] > st.m[0] + slack_of<BV>(qc.inv[0]) || tm[1] > st.m[1] + slack_of<BV>(qc.inv[1]))) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      tm[j] = fmaxf(tm[j], __shfl_xor_sync(0xffffffffu, tm[j], 4));
      tm[j] = fmaxf(tm[j], __shfl_xor_sync(0xffffffffu, tm[j], 8));
      tm[j] = fmaxf(tm[j], __shfl_xor_sync(0xffffffffu, tm[j], 16));
      const float mn = tm[j] > st.m[j] + slack_of<BV>(qc.inv[j]) ? tm[j] : st.m[j];
      const float nm = mn == -INFINITY ? 0.f : -mn * qc.inv[j];
      const float corr = ex2(fmaf(st.m[j], qc.inv[j], nm));
      st.m[j] = mn;
      st.nm[j] = nm;
      st.l[j] *= corr;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        st.acc[mt][j] *= corr;
        st.acc[mt][2 + j] *= corr;
      }
      st.zd[j] *= corr;
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint8_t* tb = tb0 + n * F::kTile;
    float p[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      p[j] = ex2(fmaf(lg[n][j], qc.inv[j], st.nm[j]));
      p[2 + j] = ex2(fmaf(lg[n][2 + j], qc.inv[j], st.nm[j]));
      st.l[j] += p[j] + p[2 + j];
    }
    const uint32_t pt0 = movmatrix_trans(pack_f16x2(p[0], p[1]));
    const uint32_t pt1 = movmatrix_trans(pack_f16x2(p[2], p[3]));
    const uint8_t* vm = tb + F::kVMeta;
    const uint4 sv0 = *reinterpret_cast<const uint4*>(vm + 16 * t);
    const uint4 sv1 = *reinterpret_cast<const uint4*>(vm + 16 * (t + 4));
    // rows g < 4 carry the zeros of group g; rows 4 .. 7 repeat them and are not used
    const uint32_t z0 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * t + 4 * (g & 3));
    const uint32_t z1 = *reinterpret_cast<const uint32_t*>(vm + 128 + 16 * (t + 4) + 4 * (g & 3));
    mma_f16(st.zd, z0, 0u, z1, 0u, pt0, pt1);
    uint32_t vw[BV == 4 ? 8 : 16];
    load_words<BV == 4 ? 8 : 16>(tb + F::kVCode, lane, vw);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t b0 = hmul2_u32(pt0, u4c(sv0, q)), b1 = hmul2_u32(pt1, u4c(sv1, q));
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        if (BV == 4) {
          const uint32_t x = vw[2 * q + mm], x8 = x >> 8;
          mma_f16(st.acc[2 * q + mm], x & 0x000F000Fu, x & 0x00F000F0u, x8 & 0x000F000Fu, x8 & 0x00F000F0u, b0, b1);
        } else {
          const uint32_t y0 = vw[2 * (2 * q + mm)], y1 = vw[2 * (2 * q + mm) + 1];
          mma_f16(st.acc[2 * q + mm], y0 & 0x00FF00FFu, y1 & 0x00FF00FFu, odd_bytes(y0), odd_bytes(y1), b0, b1);
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
struct PairState {
  float nm[2][2];       // minus the running maximum in log2 units (kNoMax before the first)
  float l[2][2];        // running sums of this thread's probabilities
  float acc[2][8][4];   // as in State
  float zd[2][4];       // sum_j p_j z_jq: rows g < 4, as in State
};
constexpr float kNoMax = 1e30f;  // above any slack, and finite: a masked logit less it is still minus infinity

__device__ __forceinline__ void reset_pair(PairState& st) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    st.nm[k][0] = st.nm[k][1] = kNoMax;
    st.l[k][0] = st.l[k][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) st.acc[k][mt][0] = st.acc[k][mt][1] = st.acc[k][mt][2] = st.acc[k][mt][3] = 0.f;
    st.zd[k][0] = st.zd[k][1] = st.zd[k][2] = st.zd[k][3] = 0.f;
  }
}

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

// One 16-row tile at address `tb` for two query tiles: a tile's codes are unpacked
// and its scales converted once for both.  query: address of the first query tile's
// operands.  kRows as in q_tile, with lim_s[k] the rows that query
// tile k's heads see, less `at`.
template <int BK, int BV, bool kRows>
__device__ __forceinline__ void q_tile_pair(uint32_t tb, int lane, uint32_t query, int vr,
                                            const int (*lim_s)[HYQ_MAX_GQA], int at, PairState& st) {
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
  float x[2][4];  // lambda 2^-sigma - max, in log2 units
  bool above = false;
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
    above |= fmaxf(fmaxf(x[k][0], x[k][1]), fmaxf(x[k][2], x[k][3])) > kSlack<BV>;
  };
  logits(std::integral_constant<int, 0>{});
  logits(std::integral_constant<int, 1>{});
  if (__any_sync(0xffffffffu, above)) {
    auto raise = [&](auto tile) {
      constexpr int k = decltype(tile)::value;
      const uint4 c = lds128<kPairQuery * k + 2048>(qt);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float inv = __uint_as_float(j ? c.w : c.y);
        float tm = fmaxf(lg[k][j], lg[k][2 + j]);
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 4));
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 8));
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
        // inv is a power of two: the product is exact
        const float old = st.nm[k][j], nm = fmaf(tm, inv, old) > kSlack<BV> ? -tm * inv : old;
        const float corr = ex2(nm - old);
        st.nm[k][j] = nm;
        st.l[k][j] *= corr;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          st.acc[k][mt][j] *= corr;
          st.acc[k][mt][2 + j] *= corr;
        }
        st.zd[k][j] *= corr;
        x[k][j] = fmaf(lg[k][j], inv, nm);
        x[k][2 + j] = fmaf(lg[k][2 + j], inv, nm);
      }
    };
    raise(std::integral_constant<int, 0>{});
    raise(std::integral_constant<int, 1>{});
  }
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
  uint4 sv0 = lds128<F::kVMeta>(tt), sv1 = lds128<F::kVMeta + 64>(tt);
  // rows g < 4 carry the zeros of group g; rows 4 .. 7 repeat them and are not used
  uint32_t z0 = lds32<F::kVMeta + 128>(tz), z1 = lds32<F::kVMeta + 192>(tz);
  if (kRows) {
    const uint32_t k0 = (2 * t < vr ? 0xFFFFu : 0u) | (2 * t + 1 < vr ? 0xFFFF0000u : 0u);
    const uint32_t k1 = (2 * t + 8 < vr ? 0xFFFFu : 0u) | (2 * t + 9 < vr ? 0xFFFF0000u : 0u);
    sv0.x &= k0, sv0.y &= k0, sv0.z &= k0, sv0.w &= k0, z0 &= k0;
    sv1.x &= k1, sv1.y &= k1, sv1.z &= k1, sv1.w &= k1, z1 &= k1;
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

// Query tile k of a pair as a State, for store_warp_partial.
__device__ __forceinline__ State pair_state(const PairState& p, int k, const QConst& qc) {
  State st;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    st.m[j] = p.nm[k][j] == kNoMax ? -INFINITY : -p.nm[k][j] / qc.inv[j];
    st.l[j] = p.l[k][j];
    st.zd[j] = p.zd[k][j];
    st.nm[j] = st.zd[2 + j] = 0.f;
  }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) st.acc[mt][i] = p.acc[k][mt][i];
  return st;
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
    const float k0 = kScale * pow2i(clamp_exp(24 - qe)) * pow2i(sg);
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
// fall in 32 banks), the maximum (log2 units) and the sum per head.
template <int BV>
__device__ __forceinline__ void store_warp_partial(State& st, const QConst& qc, int g, int t, float* wpart,
                                                   float (&red_m)[HYQ_MAX_GQA], float (&red_l)[HYQ_MAX_GQA]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) st.l[j] += __shfl_xor_sync(0xffffffffu, st.l[j], o);
  // sum_j p_j z_jq of heads 2t, 2t+1 sits in lane (q, t): gather all four groups.
  float zt[4][2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    zt[q][0] = __shfl_sync(0xffffffffu, st.zd[0], 4 * q + t);
    zt[q][1] = __shfl_sync(0xffffffffu, st.zd[1], 4 * q + t);
  }
  // Accumulator (m-tile u, ci) of thread (g, t): element 32(u/2) + 4g +
  // 2(u%2) + (ci >> 1), head 2t + (ci & 1); with 4-bit values the rows
  // ci >= 2 carry 16 c.
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int ci = 0; ci < 4; ++ci) {
      const int d = 32 * (u >> 1) + 4 * g + 2 * (u & 1) + (ci >> 1), hd = 2 * t + (ci & 1);
      const float f = (BV == 4 && ci >= 2) ? HYQ_F16_SUB_SCALE / 16.f : HYQ_F16_SUB_SCALE;
      wpart[hd * HYQ_D + (d ^ t)] = fmaf(st.acc[u][ci], f, zt[u >> 1][ci & 1]);
    }
  if (g == 0)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      red_m[2 * t + j] = st.m[j] == -INFINITY ? -INFINITY : st.m[j] * qc.inv[j];  // back to log2 units
      red_l[2 * t + j] = st.l[j];
    }
}

}  // namespace
