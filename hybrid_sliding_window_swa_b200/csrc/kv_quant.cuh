// kv_quant.cuh -- one row of a 4-bit pool: d codes and the row's (step, minimum).
//
// A row x[0 .. d) (one token, one KV head, K or V; bf16) is held as
//   lo   = min x                                      (a bf16, exactly)
//   step = bf16((max x - min x) * fp32(1 / 15))
//   code = clamp(rint((x - lo) * fp32(1 / step)), 0, 15)   (0 where step is 0)
// in fp32 with one rounding per operation, and stands for fp32(code * step + lo). Steps below 2^-120
// (whose reciprocal would leave the fp32 range) are held as 0, so such a row stands for its minimum.
// A row with a NaN or an infinity, or whose range passes the fp32 range, is held as NaN throughout.
//
// Code 2i is the low nibble of byte i, code 2i + 1 the high one. The (step, lo) pairs follow the
// codes of a block: a block is the 64 rows of one (page, KV head) or the W rows of one ring row:
//   [rows][d / 2] code bytes, then [rows] pairs of bf16 (step in the low half), padded to 16 bytes.
#pragma once
#include "common.cuh"

namespace hswa {

__host__ __device__ constexpr int64_t i4_block_bytes(int64_t rows, int d) {
  return rows * (d / 2) + ((rows * 4 + 15) / 16) * 16;
}

// The packed (step, lo) of a row and the reciprocal its codes use. `finite`: every entry is finite.
__device__ __forceinline__ uint32_t i4_params(float lo, float hi, bool finite, float& inv) {
  const float range = hi - lo;
  if (!finite || !(range <= 3.402823466e38f)) {
    inv = 0.f;
    return 0x7FFF7FFFu;
  }
  const uint32_t lo16 = __float_as_uint(lo) >> 16;  // lo is a bf16 value
  uint32_t st = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(range, 0.06666667f)));
  const float step = __uint_as_float(st << 16);
  if (step >= 7.5231638e-37f) {  // 2^-120
    inv = __frcp_rn(step);
  } else {
    inv = 0.f;
    st = 0u;
  }
  return st | (lo16 << 16);
}

__device__ __forceinline__ uint32_t i4_code(float x, float lo, float inv) {
  const uint32_t c = __float2uint_rn(__fmul_rn(__fsub_rn(x, lo), inv));  // negative and NaN give 0
  return c < 15u ? c : 15u;
}

// Eight consecutive entries (four bf16 pairs) -> 32 bits of codes.
__device__ __forceinline__ uint32_t i4_pack8(const uint32_t (&w)[4], float lo, float inv) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r |= i4_code(__uint_as_float(w[i] << 16), lo, inv) << (8 * i);
    r |= i4_code(__uint_as_float(w[i] & 0xFFFF0000u), lo, inv) << (8 * i + 4);
  }
  return r;
}

// Running minimum / maximum / finiteness over bf16 pairs.
struct RowRange {
  float lo = INFINITY, hi = -INFINITY;
  bool finite = true;
  __device__ __forceinline__ void add(uint32_t w) {
    const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xFFFF0000u);
    lo = fminf(lo, fminf(a, b));
    hi = fmaxf(hi, fmaxf(a, b));
    // exponent all ones in either half
    finite = finite && (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
  }
  // Combine over the aligned groups of LANES lanes given by `mask`.
  template <int LANES>
  __device__ __forceinline__ void reduce(unsigned mask) {
#pragma unroll
    for (int s = 1; s < LANES; s <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(mask, lo, s));
      hi = fmaxf(hi, __shfl_xor_sync(mask, hi, s));
      finite = __shfl_xor_sync(mask, finite ? 1 : 0, s) != 0 && finite;
    }
  }
};

// Address of a row's codes and of its pair inside a block of `rows` rows.
template <int D>
__device__ __forceinline__ uint8_t* i4_codes(uint8_t* block, int64_t row) {
  return block + row * (D / 2);
}
template <int D>
__device__ __forceinline__ uint32_t* i4_pair(uint8_t* block, int64_t rows, int64_t row) {
  return reinterpret_cast<uint32_t*>(block + rows * (D / 2)) + row;
}

}  // namespace hswa
