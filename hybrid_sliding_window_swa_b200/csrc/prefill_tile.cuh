// prefill_tile.cuh -- per-tile pieces shared by the prefill kernels: the online-softmax step of
// one 128-key tile for one query row (one thread per TMEM lane), the output epilogue, and the
// cp.async loader for rolling-buffer rows.
//
// Math ("Sliding Window Attention (SWA) no riron to jisso", section "formal definition",
// eqs. (1)-(5)): row i's weights are softmax_j(q_i . k_j / sqrt(d)) over the keys of its band;
// the step keeps the running maximum in the exp2 domain and rescales O only when the maximum
// grows by more than 2^kTau, so P = 2^(s * scale * log2 e - m) stays below 2^kTau.
#pragma once
#include "common.cuh"
#include "kv_quant.cuh"

namespace hswa {
namespace {

constexpr int BM = 128;     // query rows per tile
constexpr int BN = 128;     // keys per tile
constexpr float kTau = 8.0f;  // lazy rescale threshold (log2 units): P stays <= 2^8

// Tuning parameters (compile-time):
//  HSWA_POLY_PER8           pairs of scores in every 8 whose exponential runs on the FMA pipe
//  HSWA_SOFTMAX_SINGLE_PASS 1: keep all 128 scores of a row in registers (one TMEM read);
//                           0: read S twice (row maximum, then exponentials), fewer registers
//  HSWA_SOFTMAX_REGS / HSWA_PRODUCER_REGS  setmaxnreg split (2 * 128 * a + 128 * b <= 384 * 168)
//  HSWA_UNIT_TBLOCK         prefill unit order: query tiles per block (0: the whole chunk)
//  HSWA_UNIT_SERPENTINE     1: CTAs take the rounds of units in alternating directions
#ifndef HSWA_POLY_PER8
#define HSWA_POLY_PER8 0
#endif
#ifndef HSWA_SOFTMAX_SINGLE_PASS
#define HSWA_SOFTMAX_SINGLE_PASS 1
#endif
#ifndef HSWA_SOFTMAX_REGS
#define HSWA_SOFTMAX_REGS 208
#endif
#ifndef HSWA_PRODUCER_REGS
#define HSWA_PRODUCER_REGS 88
#endif
#ifndef HSWA_UNIT_TBLOCK
#define HSWA_UNIT_TBLOCK 1
#endif
#ifndef HSWA_UNIT_SERPENTINE
#define HSWA_UNIT_SERPENTINE 1
#endif
static_assert(2 * 128 * HSWA_SOFTMAX_REGS + 128 * HSWA_PRODUCER_REGS <= 384 * 168, "register split");
#define HSWA_STR2(x) #x
#define HSWA_STR(x) HSWA_STR2(x)

__device__ __forceinline__ constexpr bool use_poly(int pair) { return (pair & 7) >= 8 - HSWA_POLY_PER8; }

// Modified scores of a call (hswa_score_mod), as a kernel takes them.
struct ScoreParams {
  float softcap;           // 0: none
  float cap_in, cap_log2;  // 2 log2(e) scale / cap, cap log2 e
  float poly_max;          // raw scores up to this magnitude take the polynomial (0: none do)
  float poly[6];           // cap log2(e) tanh(x scale / cap) = x (poly[0] + poly[1] x^2 + ...)
  float near_max;          // the same with three terms for |x| up to near_max = 0.35 (large caps: 0.125) cap / scale
  float near[3];
  const float* slope;      // [Hq] distance slopes, or null
  const int64_t* key_begin;  // [B][n_q], or null
  const int64_t* key_end;
};

inline void fill_score_params(const hswa_score_mod& m, double scale, ScoreParams* sp) {
  *sp = ScoreParams{};
  sp->softcap = m.softcap;
  sp->slope = m.dist_slope;
  sp->key_begin = m.key_begin;
  sp->key_end = m.key_end;
  if (m.softcap > 0.f) {
    const double log2e = 1.4426950408889634, c1 = scale / (double)m.softcap;
    sp->cap_in = (float)(2.0 * log2e * c1);
    sp->cap_log2 = (float)(log2e * m.softcap);
    // tanh(u) = u T(u^2) on |u| <= 1: interpolation at the 6 Chebyshev nodes of u^2 in [0, 1], off by at
    // most 5e-7. The powers of u's factor are folded into the coefficients, for caps whose folded
    // coefficients and powers stay well inside the fp32 range (c1 = scale / cap from 8e-8, the largest cap, to 100).
    const double T[6] = {0.9999993948006503,  -0.33328951370216614, 0.1328072064598301,
                         -0.05158598840417456, 0.01672085517953942, -0.0030582290375864097};
    // Three terms on |u| <= 0.35, off by at most 1e-6. Both errors are the cap's share of a score's, so caps above
    // 1 / 6e-4 of the scale (147 for d = 128) take neither: there the first three terms of the series serve on
    // |u| <= 1/8, off by 2.1e-7 of the value, and only larger scores go through the exponential.
    const double N[3] = {0.9999971183259196, -0.3329087359461866, 0.12394375936961438};
    const double S[3] = {1.0, -1.0 / 3.0, 2.0 / 15.0};
    const bool large = c1 < 6e-4;
    if (c1 <= 100.0) {
      sp->near_max = (float)((large ? 0.125 : 0.35) / c1);
      if (!large) sp->poly_max = (float)(1.0 / c1);
      double f = log2e * m.softcap * c1;
      for (int i = 0; i < 6; ++i, f *= c1 * c1) {
        if (!large) sp->poly[i] = (float)(T[i] * f);
        if (i < 3) sp->near[i] = (float)((large ? S[i] : N[i]) * f);
      }
    }
  }
}

// Largest magnitude of a row's raw scores (NaN ignored).
template <int N>
__device__ __forceinline__ float abs_max(const uint32_t (&v)[N]) {
  float m0 = 0.f, m1 = 0.f, m2 = 0.f, m3 = 0.f;
#pragma unroll
  for (int k = 0; k < N; k += 8) {
    m0 = fmax3(m0, fabsf(__uint_as_float(v[k])), fabsf(__uint_as_float(v[k + 1])));
    m1 = fmax3(m1, fabsf(__uint_as_float(v[k + 2])), fabsf(__uint_as_float(v[k + 3])));
    m2 = fmax3(m2, fabsf(__uint_as_float(v[k + 4])), fabsf(__uint_as_float(v[k + 5])));
    m3 = fmax3(m3, fabsf(__uint_as_float(v[k + 6])), fabsf(__uint_as_float(v[k + 7])));
  }
  return fmaxf(fmax3(m0, m1, m2), m3);
}

// The N raw scores of a row -> z log2(e), z = cap tanh(s / cap) - slope |i - j|. c_q: the query's own
// column (its position minus that of column 0), so column k is |c_q - k| away.
// The cap costs what tanh costs: through exponential and reciprocal it is two more MUFU operations per
// score, on the unit that the softmax itself loads most. While every score of the warp stays within the
// cap (|s| <= cap), the degree-11 polynomial on the FMA pipe replaces them: 7 packed multiply-adds per pair;
// within near_max a degree-5 one does, 4 per pair.
// Bias: on a tile wholly before the warp's queries |c_q - k| = c_q - k, two packed operations per pair.
// am: abs_max(v), used with a cap.
template <int N>
__device__ __forceinline__ void modify_scores(uint32_t (&v)[N], const ScoreParams& sp, float sl2, float slope2,
                                              float c_q, float am) {
  if (sp.softcap > 0.f) {
    if (__all_sync(0xffffffffu, am <= sp.near_max)) {
      const uint64_t n0 = f2_pack(sp.near[0], sp.near[0]), n1 = f2_pack(sp.near[1], sp.near[1]),
                     n2 = f2_pack(sp.near[2], sp.near[2]);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const uint64_t x = f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
        const uint64_t t = f2_mul(x, x);
        float a, b;
        f2_unpack(f2_mul(x, f2_fma(f2_fma(n2, t, n1), t, n0)), a, b);
        v[k] = __float_as_uint(a);
        v[k + 1] = __float_as_uint(b);
      }
    } else if (__all_sync(0xffffffffu, am <= sp.poly_max)) {
      uint64_t c[6];
#pragma unroll
      for (int i = 0; i < 6; ++i) c[i] = f2_pack(sp.poly[i], sp.poly[i]);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const uint64_t x = f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
        const uint64_t t = f2_mul(x, x);
        uint64_t y = f2_fma(c[5], t, c[4]);
        y = f2_fma(y, t, c[3]);
        y = f2_fma(y, t, c[2]);
        y = f2_fma(y, t, c[1]);
        y = f2_fma(y, t, c[0]);
        y = f2_mul(x, y);
        float a, b;
        f2_unpack(y, a, b);
        v[k] = __float_as_uint(a);
        v[k + 1] = __float_as_uint(b);
      }
    } else {
      // scores of every size: each takes the form that is exact for it (for tiny ones the exponential's is not)
      const uint64_t n0 = f2_pack(sp.near[0], sp.near[0]), n1 = f2_pack(sp.near[1], sp.near[1]),
                     n2 = f2_pack(sp.near[2], sp.near[2]);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const float x0 = __uint_as_float(v[k]), x1 = __uint_as_float(v[k + 1]);
        const uint64_t x = f2_pack(x0, x1), t = f2_mul(x, x);
        float a, b;
        f2_unpack(f2_mul(x, f2_fma(f2_fma(n2, t, n1), t, n0)), a, b);
        v[k] = __float_as_uint(fabsf(x0) <= sp.near_max ? a : capped_log2(x0, sp.cap_in, sp.cap_log2));
        v[k + 1] = __float_as_uint(fabsf(x1) <= sp.near_max ? b : capped_log2(x1, sp.cap_in, sp.cap_log2));
      }
    }
    sl2 = 1.f;
  }
  if (sp.slope) {
    if (__all_sync(0xffffffffu, c_q >= (float)(N - 1))) {
      // x sl2 + slope2 (k - c_q), k - c_q exact
      const uint64_t s2 = f2_pack(sl2, sl2), b2 = f2_pack(slope2, slope2), two = f2_pack(2.f, 2.f);
      uint64_t d = f2_pack(-c_q, 1.f - c_q);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        float a, b;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), s2, f2_mul(d, b2)), a, b);
        v[k] = __float_as_uint(a);
        v[k + 1] = __float_as_uint(b);
        d = f2_add(d, two);
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        v[k] = __float_as_uint(fmaf(-slope2, fabsf(c_q - (float)k), __uint_as_float(v[k]) * sl2));
    }
  }
}

// One key tile of one query row. trow: this warp's TMEM lane base; S of the row in columns
// [s_col, s_col + 128), O in [o_col, o_col + D). Columns outside [c_lo, c_hi] are masked when
// `edge`. m_used / l: running maximum (log2 domain) and row sum; o_live: O already holds a
// partial sum (it is rescaled when the maximum moves). P is written over S as packed bf16;
// the caller waits for the TMEM stores and signals the MMA.
// MASK_MODE selects how edge tiles are masked (all give the same result):
//  0  per-column compares (faster where every tile is an edge tile, as in the narrow kernel);
//  1  integer sign arithmetic on every column (faster where edge tiles are few);
//  2  W = 128 with no row's band clipped at the sequence start (the narrow kernel's common tile):
//     before the diagonal a row keeps columns k > r, on the diagonal k <= r, so for warp w
//     (rows 32w .. 32w + 31) chunk w is the only chunk the band edge crosses and every other
//     chunk is wholly in or out for the whole warp. The warp loads chunk (w + c) & 3 into
//     register block c (rot = w), masks block 0 by lane and selects the other blocks whole;
//     `lower_edge` marks the tile before the diagonal. Single-pass softmax only.
//
// MOD: the scores are modified first (modify_scores) and come out in the log2 domain.
template <int D, int MASK_MODE, bool MOD = false>
__device__ __forceinline__ void softmax_tile(uint32_t trow, uint32_t s_col, uint32_t o_col, float sl2, bool edge,
                                             int c_lo, int c_hi, float& m_used, float& l, bool o_live,
                                             int rot = 0, bool lower_edge = false, const ScoreParams* sp = nullptr,
                                             float slope2 = 0.f, float c_q = 0.f) {
  static_assert(!MOD || HSWA_SOFTMAX_SINGLE_PASS, "modified scores need the single-pass softmax");
  static_assert(MASK_MODE != 2 || HSWA_SOFTMAX_SINGLE_PASS, "the rotated mask needs the single-pass softmax");
  constexpr bool BRANCH_FREE_MASK = MASK_MODE == 1;
  const int rc = MASK_MODE == 2 ? rot : 0;  // chunk rotation (0 folds away in the other modes)
#if HSWA_SOFTMAX_SINGLE_PASS
    // all 128 scores of the row: four TMEM loads, one wait
    uint32_t v[128];
    tmem_ld32_into<0>(trow + s_col + 32 * ((rc + 0) & 3), v);
    tmem_ld32_into<32>(trow + s_col + 32 * ((rc + 1) & 3), v);
    tmem_ld32_into<64>(trow + s_col + 32 * ((rc + 2) & 3), v);
    tmem_ld32_into<96>(trow + s_col + 32 * ((rc + 3) & 3), v);
    tmem_wait_ld();
    reg_fence_into<0>(v);
    reg_fence_into<32>(v);
    reg_fence_into<64>(v);
    reg_fence_into<96>(v);
    // MOD: `near` = capped scores without a bias, all of the warp's within near_max. The cap is monotone,
    // so the row maximum is taken on raw scores and capped alone, and the three-term polynomial goes into
    // the exponential's argument: 3 packed operations per pair. (Masked scores, -inf, come out as -inf:
    // the polynomial's highest coefficient is positive.)
    bool near = false;
    if constexpr (MOD) {
      float am = 0.f;
      if (sp->softcap > 0.f) {
        am = abs_max(v);
        near = __all_sync(0xffffffffu, am <= sp->near_max) && !sp->slope;
      }
      if (!near) {
        modify_scores(v, *sp, sl2, slope2, c_q, am);
        sl2 = 1.f;
      }
    }
    if (MASK_MODE == 2) {
      // block 0 = chunk rot: the lower edge keeps j > lane, the diagonal keeps j <= lane
      const int lane = threadIdx.x & 31;
      if (lower_edge) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j <= lane) v[j] = 0xFF800000u;
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j > lane) v[j] = 0xFF800000u;
      }
#pragma unroll
      for (int c = 1; c < 4; ++c) {
        // chunk rot + c lies above the warp's rows (kept before the diagonal, dropped on it);
        // a wrapped chunk lies below them
        const bool out = lower_edge ? (rc + c > 3) : (rc + c <= 3);
#pragma unroll
        for (int j = 32 * c; j < 32 * c + 32; ++j) v[j] = out ? 0xFF800000u : v[j];
      }
    } else if (edge) {
      if (BRANCH_FREE_MASK) {
        // the sign of (k - c_lo) | (c_hi - k) is set exactly outside [c_lo, c_hi] (positions
        // stay below 2^31 - 256, so neither difference overflows)
        const int nlo = -c_lo;
#pragma unroll
        for (int k = 0; k < 128; ++k) {
          const uint32_t m = (uint32_t)(((k + nlo) | (c_hi - k)) >> 31);
          v[k] = (v[k] & ~m) | (0xFF800000u & m);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 128; ++k)
          if (k < c_lo || k > c_hi) v[k] = __float_as_uint(-INFINITY);
      }
    }
    float m0 = __uint_as_float(v[0]), m1 = __uint_as_float(v[1]);
    float m2 = __uint_as_float(v[2]), m3 = __uint_as_float(v[3]);
#pragma unroll
    for (int k = 4; k < 124; k += 8) {
      m0 = fmax3(m0, __uint_as_float(v[k + 0]), __uint_as_float(v[k + 1]));
      m1 = fmax3(m1, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
      m2 = fmax3(m2, __uint_as_float(v[k + 4]), __uint_as_float(v[k + 5]));
      m3 = fmax3(m3, __uint_as_float(v[k + 6]), __uint_as_float(v[k + 7]));
    }
    m0 = fmax3(m0, __uint_as_float(v[124]), __uint_as_float(v[125]));
    m1 = fmax3(m1, __uint_as_float(v[126]), __uint_as_float(v[127]));
    const float mx = fmaxf(fmax3(m0, m1, m2), m3);
    float m_tile = mx * sl2;
    if constexpr (MOD) {
      if (near) m_tile = mx == -INFINITY ? mx : mx * fmaf(fmaf(sp->near[2], mx * mx, sp->near[1]), mx * mx, sp->near[0]);
    }
    float alpha = 1.f;
    bool resc = false;
    if (m_tile > m_used + kTau) {
      if (m_used != -INFINITY) {
        alpha = ex2_approx(m_used - m_tile);
        resc = true;
      }
      l *= alpha;
      m_used = m_tile;
    }
    if (__any_sync(0xffffffffu, resc) && o_live) {
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(trow + o_col + c0, o);
        tmem_wait_ld();
        reg_fence32(o);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
        tmem_st32(trow + o_col + c0, o);
      }
      tmem_wait_st();
    }
    if constexpr (MOD) {
      if (near) {
        const float mo = (m_used == -INFINITY) ? 0.f : m_used;
        const uint64_t n0 = f2_pack(sp->near[0], sp->near[0]), n1 = f2_pack(sp->near[1], sp->near[1]),
                       n2 = f2_pack(sp->near[2], sp->near[2]), neg = f2_pack(-mo, -mo);
        uint64_t ac[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const uint64_t x = f2_pack(__uint_as_float(v[c0 + k]), __uint_as_float(v[c0 + k + 1]));
            const uint64_t t = f2_mul(x, x);
            float e0, e1;
            f2_unpack(f2_fma(x, f2_fma(f2_fma(n2, t, n1), t, n0), neg), e0, e1);
            e0 = ex2_approx(e0);
            e1 = ex2_approx(e1);
            ac[(k >> 1) & 3] = f2_add(ac[(k >> 1) & 3], f2_pack(e0, e1));
            pk[k >> 1] = pack_bf16x2(e0, e1);
          }
          tmem_st16(trow + s_col + 16 * (c0 >> 5), pk);
        }
        float a0, a1, b0, b1, d0, d1, f0, f1;
        f2_unpack(ac[0], a0, a1);
        f2_unpack(ac[1], b0, b1);
        f2_unpack(ac[2], d0, d1);
        f2_unpack(ac[3], f0, f1);
        l += ((a0 + a1) + (b0 + b1)) + ((d0 + d1) + (f0 + f1));
        return;
      }
    }
    // P = 2^(s * scale * log2 e - m) in place, packed to bf16 and stored over S
    const float moff = (m_used == -INFINITY) ? 0.f : m_used;
    const uint64_t scale2 = f2_pack(sl2, sl2);
    const uint64_t neg2 = f2_pack(-moff, -moff);
    uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int c0 = 0; c0 < BN; c0 += 32) {
      uint32_t pk[16];
      if (MASK_MODE == 2 && c0 > 0) {
        // a block wholly outside every row's band: P = 0 without exponentials
        const bool out = lower_edge ? (rc + (c0 >> 5) > 3) : (rc + (c0 >> 5) <= 3);
        if (out) {
#pragma unroll
          for (int k = 0; k < 16; ++k) pk[k] = 0u;
          tmem_st16(trow + s_col + 16 * (((c0 >> 5) + rc) & 3), pk);
          continue;
        }
      }
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        const int pair = (c0 + k) >> 1;
        const uint64_t x = f2_fma(f2_pack(__uint_as_float(v[c0 + k]), __uint_as_float(v[c0 + k + 1])), scale2, neg2);
        uint64_t e;
        if (use_poly(pair)) {
          e = exp2_poly_x2(x);
        } else {
          float x0, x1;
          f2_unpack(x, x0, x1);
          e = f2_pack(ex2_approx(x0), ex2_approx(x1));
        }
        acc[pair & 3] = f2_add(acc[pair & 3], e);
        float e0, e1;
        f2_unpack(e, e0, e1);
        pk[k >> 1] = pack_bf16x2(e0, e1);
      }
      tmem_st16(trow + s_col + 16 * (((c0 >> 5) + rc) & 3), pk);
    }
#else
    // pass 1: row maximum, 64 scores at a time
    float mx = -INFINITY;
#pragma unroll
    for (int h2 = 0; h2 < BN; h2 += 64) {
      uint32_t va[32], vb[32];
      tmem_ld32(trow + s_col + h2, va);
      tmem_ld32(trow + s_col + h2 + 32, vb);
      tmem_wait_ld();
      reg_fence32(va);
      reg_fence32(vb);
      if (edge) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t ma = (uint32_t)(((h2 + k - c_lo) | (c_hi - h2 - k)) >> 31);
          const uint32_t mb = (uint32_t)(((h2 + 32 + k - c_lo) | (c_hi - h2 - 32 - k)) >> 31);
          va[k] = (va[k] & ~ma) | (0xFF800000u & ma);
          vb[k] = (vb[k] & ~mb) | (0xFF800000u & mb);
        }
      }
      float m0 = mx, m1 = __uint_as_float(va[0]), m2 = __uint_as_float(vb[0]);
#pragma unroll
      for (int k = 1; k < 31; k += 2) {
        m0 = fmax3(m0, __uint_as_float(va[k]), __uint_as_float(va[k + 1]));
        m1 = fmax3(m1, __uint_as_float(vb[k]), __uint_as_float(vb[k + 1]));
      }
      m2 = fmax3(m2, __uint_as_float(va[31]), __uint_as_float(vb[31]));
      mx = fmax3(m0, m1, m2);
    }
    const float m_tile = mx * sl2;
    float alpha = 1.f;
    bool resc = false;
    if (m_tile > m_used + kTau) {
      if (m_used != -INFINITY) {
        alpha = ex2_approx(m_used - m_tile);
        resc = true;
      }
      l *= alpha;
      m_used = m_tile;
    }
    if (__any_sync(0xffffffffu, resc) && o_live) {
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(trow + o_col + c0, o);
        tmem_wait_ld();
        reg_fence32(o);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
        tmem_st32(trow + o_col + c0, o);
      }
      tmem_wait_st();
    }
    // pass 2: P = 2^(s * scale * log2 e - m), 32 columns at a time, the next chunk's TMEM
    // load in flight while this one is exponentiated, packed and stored over S.
    const float moff = (m_used == -INFINITY) ? 0.f : m_used;
    const uint64_t scale2 = f2_pack(sl2, sl2);
    const uint64_t neg2 = f2_pack(-moff, -moff);
    uint64_t acc[4] = {0, 0, 0, 0};
    uint32_t buf[2][32];
    tmem_ld32(trow + s_col, buf[0]);
    tmem_wait_ld();
    reg_fence32(buf[0]);
#pragma unroll
    for (int c = 0; c < BN / 32; ++c) {
      uint32_t(&cur)[32] = buf[c & 1];
      if (c + 1 < BN / 32) tmem_ld32(trow + s_col + 32 * (c + 1), buf[(c + 1) & 1]);
      const int c0 = 32 * c;
      if (edge) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t m = (uint32_t)(((c0 + k - c_lo) | (c_hi - c0 - k)) >> 31);
          cur[k] = (cur[k] & ~m) | (0xFF800000u & m);
        }
      }
      uint32_t pk[16];
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        const int pair = (c0 + k) >> 1;
        const uint64_t x = f2_fma(f2_pack(__uint_as_float(cur[k]), __uint_as_float(cur[k + 1])), scale2, neg2);
        uint64_t e;
        if (use_poly(pair)) {
          e = exp2_poly_x2(x);
        } else {
          float x0, x1;
          f2_unpack(x, x0, x1);
          e = f2_pack(ex2_approx(x0), ex2_approx(x1));
        }
        acc[pair & 3] = f2_add(acc[pair & 3], e);
        float e0, e1;
        f2_unpack(e, e0, e1);
        pk[k >> 1] = pack_bf16x2(e0, e1);
      }
      tmem_st16(trow + s_col + (c0 >> 1), pk);
      if (c + 1 < BN / 32) {
        tmem_wait_ld();
        reg_fence32(buf[(c + 1) & 1]);
      }
    }
#endif
    float a0, a1, b0, b1, c0_, c1_, d0, d1;
    f2_unpack(acc[0], a0, a1);
    f2_unpack(acc[1], b0, b1);
    f2_unpack(acc[2], c0_, c1_);
    f2_unpack(acc[3], d0, d1);
    l += ((a0 + a1) + (b0 + b1)) + ((c0_ + c1_) + (d0 + d1));
}

// Epilogue of one query tile: O / l -> bf16, staged per warp (its 32 rows x 128 B, 128-byte
// swizzle, 4 KB at `stage`) and written by one TMA store per 64-column half into the output
// map at (column, head h, row0 .. row0 + 31, batch b); rows past n_q fall outside the map.
// MAY_BE_EMPTY: a row with l = 0 saw no key (its O columns may never have been written) and gives zeros.
template <int D, bool MAY_BE_EMPTY = false>
__device__ __forceinline__ void store_output(uint32_t trow, uint32_t o_col, float l, uint8_t* stage, int lane,
                                             const CUtensorMap* tm_o, int h, int row0, int b, int n_q) {
  const float inv = 1.f / l;
  const bool none = MAY_BE_EMPTY && l == 0.f;
#pragma unroll
  for (int dh = 0; dh < D / 64; ++dh) {
    if (lane == 0) bulk_wait_read_all();  // the previous store from this buffer has read it
    __syncwarp();
#pragma unroll
    for (int c0 = 0; c0 < 64; c0 += 32) {
      uint32_t o[32];
      tmem_ld32(trow + o_col + dh * 64 + c0, o);
      tmem_wait_ld();
      reg_fence32(o);
      uint32_t pk[16];
#pragma unroll
      for (int k = 0; k < 32; k += 2)
        pk[k >> 1] = pack_bf16x2(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv);
      if (none) {
#pragma unroll
        for (int k = 0; k < 16; ++k) pk[k] = 0u;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int chunk = (c0 >> 3) + x;
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((chunk ^ (lane & 7)) << 4)) =
            make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row0 < n_q) {  // a box wholly past the chunk end is not issued
      tma_store_4d(tm_o, stage, dh * 64, h, row0, b);
      bulk_commit_group();
    }
  }
}

// The epilogue without staging: each thread writes its row's O / l (zeros when l = 0) with 16-byte stores.
// The columns of every group of eight hold the dims 0 4 1 5 2 6 3 7 (i4x8_bf16_perm).
template <int D>
__device__ __forceinline__ void store_output_direct(uint32_t trow, uint32_t o_col, float l, uint16_t* row, bool live) {
  const float inv = 1.f / l;
  const bool none = l == 0.f;
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += 32) {
    uint32_t o[32];
    tmem_ld32(trow + o_col + c0, o);
    tmem_wait_ld();
    reg_fence32(o);
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      // dims k, k + 1 of a group of eight are 0 2 | 4 6 | 1 3 | 5 7
      const int c = (k & ~7) + ((k & 2) << 1) + ((k & 4) >> 2);
      pk[k >> 1] = none ? 0u : pack_bf16x2(__uint_as_float(o[c]) * inv, __uint_as_float(o[c + 2]) * inv);
    }
    if (live) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        reinterpret_cast<uint4*>(row + c0)[x] = make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
    }
  }
}

// store_output for a caller whose next MMA waits for O's TMEM columns: all D columns of the row
// are read into registers first, `o_free` gets this thread's arrival (the columns may be
// overwritten from then on), and the packing, staging and TMA stores follow.
template <int D>
__device__ __forceinline__ void store_output_release(uint32_t trow, uint32_t o_col, float l, uint8_t* stage, int lane,
                                                     const CUtensorMap* tm_o, int h, int row0, int b, int n_q,
                                                     uint64_t* o_free) {
  uint32_t o[D];
  tmem_ld32_into<0>(trow + o_col, o);
  tmem_ld32_into<32>(trow + o_col + 32, o);
  if constexpr (D == 128) {
    tmem_ld32_into<64>(trow + o_col + 64, o);
    tmem_ld32_into<96>(trow + o_col + 96, o);
  }
  tmem_wait_ld();
  reg_fence_into<0>(o);
  reg_fence_into<32>(o);
  if constexpr (D == 128) {
    reg_fence_into<64>(o);
    reg_fence_into<96>(o);
  }
  tc_fence_before();
  mbar_arrive(o_free);
  const float inv = 1.f / l;
#pragma unroll
  for (int dh = 0; dh < D / 64; ++dh) {
    if (lane == 0) bulk_wait_read_all();  // the previous store from this buffer has read it
    __syncwarp();
#pragma unroll
    for (int c0 = 0; c0 < 64; c0 += 32) {
      uint32_t pk[16];
#pragma unroll
      for (int k = 0; k < 32; k += 2)
        pk[k >> 1] = pack_bf16x2(__uint_as_float(o[dh * 64 + c0 + k]) * inv,
                                 __uint_as_float(o[dh * 64 + c0 + k + 1]) * inv);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int chunk = (c0 >> 3) + x;
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((chunk ^ (lane & 7)) << 4)) =
            make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row0 < n_q) {  // a box wholly past the chunk end is not issued
      tma_store_4d(tm_o, stage, dh * 64, h, row0, b);
      bulk_commit_group();
    }
  }
}

// Rolling-buffer rows of one key tile with cp.async (any W and chunk start), one warp:
// positions kb .. kb + 127 come from slot pos mod W of the ring at `ring_rows` (W rows of d),
// rows whose position the ring does not hold ([held_lo, held_hi) holds) or a bad ring are
// zero-filled. Layout of dst: [D / 64 blocks][128 rows][128 B], 128-byte swizzle, consecutive
// 64-dim blocks blk_stride bytes apart (16 KB for one tile; a tile inside a taller operand
// leaves room for the other rows).
template <int D>
__device__ __forceinline__ void ring_rows_cpasync(const uint16_t* ring_rows, bool ok, int held_lo, int held_hi,
                                                  int W, uint8_t* dst, int kb, int lane, int blk_stride = BM * 128) {
  const uint32_t sdst = smem_u32(dst);
  constexpr int CH = D / 8;  // 16-byte chunks per row
  for (int idx = lane; idx < BN * CH; idx += 32) {
    const int r = idx / CH;
    const int c = idx % CH;
    const int pos = kb + r;
    const bool held = ok && pos >= held_lo && pos < held_hi;
    const uint16_t* src = held ? ring_rows + (int64_t)(pos % W) * D + c * 8 : ring_rows;
    const int blk = c >> 3, cc = c & 7;
    const uint32_t off = blk * blk_stride + r * 128 + ((cc ^ (r & 7)) << 4);
    cp_async_16(sdst + off, src, held ? 16u : 0u);
  }
  cp_async_wait_all();
  fence_proxy_async_smem();
  __syncwarp();
}

// Two E4M3 codes (the low 16 bits of x) -> their fp32 values times `scale`, packed to bf16x2
// (the E4M3 -> f16 step is exact; the product rounds once to fp32 and once to bf16).
__device__ __forceinline__ uint32_t e4m3x2_scaled_bf16x2(uint32_t x, float scale) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(x));
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return pack_bf16x2(lo * scale, hi * scale);
}

// ring_rows_cpasync for a ring of FP8 E4M3 codes: the held rows are dequantized (code value times
// `scale`) to bf16 in the tile's swizzled layout; the others are zero. One warp, plain loads
// (four 16-byte loads in flight per lane); the caller fences and signals as for the cp.async path.
template <int D>
__device__ __forceinline__ void ring_rows_fp8(const uint8_t* ring_rows, bool ok, int held_lo, int held_hi, int W,
                                              float scale, uint8_t* dst, int kb, int lane, int blk_stride = BM * 128) {
  constexpr int CH8 = D / 16;           // 16-code chunks per row
  constexpr int TOTAL = BN * CH8;       // chunks per tile
  constexpr int BATCH = 4;
  static_assert(TOTAL % (32 * BATCH) == 0, "tile chunks");
  for (int base = 0; base < TOTAL; base += 32 * BATCH) {
    uint4 x[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int idx = base + u * 32 + lane;
      const int r = idx / CH8, c = idx % CH8;
      const int pos = kb + r;
      const bool held = ok && pos >= held_lo && pos < held_hi;
      x[u] = held ? __ldg(reinterpret_cast<const uint4*>(ring_rows + (int64_t)(pos % W) * D + c * 16))
                  : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int idx = base + u * 32 + lane;
      const int r = idx / CH8, c = idx % CH8;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = e4m3x2_scaled_bf16x2(w[i], scale);
        o[2 * i + 1] = e4m3x2_scaled_bf16x2(w[i] >> 16, scale);
      }
      // codes 16c .. 16c + 15 -> bf16 chunks 2c and 2c + 1 of the row
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int cc = 2 * c + h;
        const int blk = cc >> 3, ch = cc & 7;
        *reinterpret_cast<uint4*>(dst + blk * blk_stride + r * 128 + ((ch ^ (r & 7)) << 4)) =
            make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
      }
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Eight 4-bit codes (a word) -> 16 bytes of bf16 values code * step + lo, dims in order. Each code is
// planted in the mantissa of 128 (bf16 128 + code, exact), 128 is subtracted (exact) and one bf16x2
// fused multiply-add rounds once.
__device__ __forceinline__ uint4 i4x8_bf16(uint32_t w, __nv_bfloat162 step, __nv_bfloat162 lo) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t z = (w >> (8 * i)) & 0xFFu;
    const uint32_t pair = ((z * 0x1001u) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&pair), __nv_bfloat162(128.f, 128.f));
    const __nv_bfloat162 y = __hfma2(c, step, lo);
    o[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The same with the eight dims in the order 0 4 1 5 2 6 3 7, as one mask takes them from the word.
__device__ __forceinline__ uint4 i4x8_bf16_perm(uint32_t w, __nv_bfloat162 step, __nv_bfloat162 lo) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&pair), __nv_bfloat162(128.f, 128.f));
    const __nv_bfloat162 y = __hfma2(c, step, lo);
    o[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void i4_pair_bf162(uint32_t pair, __nv_bfloat162& step, __nv_bfloat162& lo) {
  const uint32_t s = __byte_perm(pair, pair, 0x1010), l = __byte_perm(pair, pair, 0x3232);
  step = *reinterpret_cast<const __nv_bfloat162*>(&s);
  lo = *reinterpret_cast<const __nv_bfloat162*>(&l);
}

// ring_rows_fp8 for a 4-bit ring block (W rows of codes, then the pairs).
template <int D>
__device__ __forceinline__ void ring_rows_i4(const uint8_t* block, bool ok, int held_lo, int held_hi, int W,
                                             uint8_t* dst, int kb, int lane, int blk_stride = BM * 128) {
  constexpr int CPR = D / 32;  // 16-byte chunks of codes per row
  constexpr int TOTAL = BN * CPR;
  constexpr int BATCH = 4;
  static_assert(TOTAL % (32 * BATCH) == 0, "tile chunks");
  const uint32_t* pairs = reinterpret_cast<const uint32_t*>(block + (int64_t)W * (D / 2));
  for (int base = 0; base < TOTAL; base += 32 * BATCH) {
    uint4 x[BATCH];
    uint32_t pr[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int idx = base + u * 32 + lane;
      const int r = idx / CPR, c = idx % CPR;
      const int pos = kb + r;
      const bool held = ok && pos >= held_lo && pos < held_hi;
      const int slot = held ? pos % W : 0;
      x[u] = held ? __ldg(reinterpret_cast<const uint4*>(block + (int64_t)slot * (D / 2) + c * 16))
                  : make_uint4(0, 0, 0, 0);
      pr[u] = held ? __ldg(pairs + slot) : 0u;
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int idx = base + u * 32 + lane;
      const int r = idx / CPR, c = idx % CPR;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      __nv_bfloat162 step, lo;
      i4_pair_bf162(pr[u], step, lo);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int cc = 4 * c + i;  // 16-byte chunk of the row in bf16
        *reinterpret_cast<uint4*>(dst + (cc >> 3) * blk_stride + r * 128 + (((cc & 7) ^ (r & 7)) << 4)) =
            i4x8_bf16(w[i], step, lo);
      }
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace
}  // namespace hswa
