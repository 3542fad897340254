// rope.cu -- rotary positions over several axes, alone and together with the commit into the pool.
//
// A token has a position p_a on each axis a (one axis for text; time, height and width for images
// and video). Pair i of a head's first rot_dim entries is turned by theta_i = p_{axis(i)} f_i:
//   (x, y) -> (x cos theta_i - y sin theta_i, y cos theta_i + x sin theta_i)
// with pairs (i, i + rot_dim / 2) or (2i, 2i + 1); the other entries pass unchanged.
//
// What bounds it: every byte of q and k is read and written once (HBM). The angle is the delicate
// part: p f reaches 10^6 radians and more, where fp32 would keep two digits of the fraction of a
// turn, so it is taken in fp64 as a number of turns, p (f / 2 pi), its nearest whole number is
// subtracted, and only the remaining fraction of a turn goes to an fp32 sine and cosine
// (error about 2^-24). A block computes the table of its tokens once and all heads read it from
// shared memory: one sine per 2 (Hq + Hkv) entries, and 16-byte loads and stores for the rest.
#include "common.cuh"
#include "internal.h"
#include "kv_place.cuh"
#include "kv_quant.cuh"

namespace hswa {
namespace {

constexpr int RT = 256;  // threads per block

struct RopeParams {
  double turns[64];  // inv_freq / (2 pi)
  uint8_t axis[64];
  int rot, interleaved;
  int64_t n;           // tokens
  const int64_t* pos;  // [n_axes][n]
  int Hq, Hkv;
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* k;
  uint16_t* k_out;     // may be null in a commit
  const uint16_t* v;   // commit only
  CommitDst dst;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 16-byte chunks of entries a and b hold the partners (half style), or a then b hold whole pairs.
__device__ __forceinline__ void rotate_unit(uint4& A, uint4& B, const float* cs, const float* sn, bool pairs) {
  uint32_t a[4] = {A.x, A.y, A.z, A.w}, b[4] = {B.x, B.y, B.z, B.w};
  if (pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = bf_lo(a[i]), y = bf_hi(a[i]), c = cs[i], s = sn[i];
      a[i] = pack_bf16x2(x * c - y * s, y * c + x * s);
      const float x2 = bf_lo(b[i]), y2 = bf_hi(b[i]), c2 = cs[4 + i], s2 = sn[4 + i];
      b[i] = pack_bf16x2(x2 * c2 - y2 * s2, y2 * c2 + x2 * s2);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = bf_lo(a[i]), y0 = bf_lo(b[i]), x1 = bf_hi(a[i]), y1 = bf_hi(b[i]);
      const float c0 = cs[2 * i], s0 = sn[2 * i], c1 = cs[2 * i + 1], s1 = sn[2 * i + 1];
      a[i] = pack_bf16x2(x0 * c0 - y0 * s0, x1 * c1 - y1 * s1);
      b[i] = pack_bf16x2(y0 * c0 + x0 * s0, y1 * c1 + x1 * s1);
    }
  }
  A = make_uint4(a[0], a[1], a[2], a[3]);
  B = make_uint4(b[0], b[1], b[2], b[3]);
}

// FMT: 0 no commit, 1 bf16 pool, 2 FP8 pool, 3 4-bit pool. A thread handles a unit of 16 entries of
// one (token, head) row, as two 16-byte chunks; unit u uses frequencies 8u .. 8u + 7. The D / 16
// threads of a row are neighbours, so a 4-bit row finds its range by shuffles.
template <int D, int FMT>
__global__ void __launch_bounds__(RT) rope_kernel(const __grid_constant__ RopeParams p, int tpb) {
  constexpr int UPR = D / 16;  // units per row
  __shared__ float cs[4 * 64], sn[4 * 64];
  const int64_t n0 = (int64_t)blockIdx.x * tpb;
  const int nt = (int)min((int64_t)tpb, p.n - n0);
  // a thread keeps its unit of the row (and so its chunks and frequencies) and walks rows (token, head),
  // two at a time, the next two being read while these are turned; the first two are on their way while
  // the table is made
  const int heads = p.Hq + p.Hkv + (FMT ? p.Hkv : 0);
  const int total = nt * heads;
  const bool pairs = p.interleaved != 0;
  const int u = threadIdx.x % UPR;
  const bool rotated = u < (p.rot >> 4);
  const int c0 = rotated && !pairs ? u : 2 * u;
  const int c1 = rotated && !pairs ? u + (p.rot >> 4) : 2 * u + 1;
  const unsigned group = ((1u << UPR) - 1u) << ((threadIdx.x & 31) & ~(UPR - 1));
  constexpr int STEP = RT / UPR;
  constexpr int BATCH = 2;
  int t = 0, h = threadIdx.x / UPR;  // of the next row to read
  uint4 nA[BATCH], nB[BATCH];
  int nt_[BATCH], nh[BATCH];
  auto read = [&](int r) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      while (h >= heads) {
        h -= heads;
        ++t;
      }
      nt_[k] = t;
      nh[k] = h;
      if (r + k * STEP < total) {
        const int64_t n = n0 + t;
        const uint16_t* src = h < p.Hq ? p.q + (n * p.Hq + h) * D
                              : h < p.Hq + p.Hkv ? p.k + (n * p.Hkv + (h - p.Hq)) * D
                                                 : p.v + (n * p.Hkv + (h - p.Hq - p.Hkv)) * D;
        nA[k] = reinterpret_cast<const uint4*>(src)[c0];
        nB[k] = reinterpret_cast<const uint4*>(src)[c1];
      }
      h += STEP;
    }
  };
  read(threadIdx.x / UPR);
  const int half = p.rot >> 1;
  for (int i = threadIdx.x; i < nt * half; i += RT) {
    const int tk = i / half, f = i - tk * half;
    const double turns = (double)p.pos[(int64_t)p.axis[f] * p.n + n0 + tk] * p.turns[f];
    const float frac = (float)(turns - rint(turns));  // in [-1/2, 1/2]
    float s, c;
    sincospif(2.f * frac, &s, &c);
    cs[tk * 64 + f] = c;
    sn[tk * 64 + f] = s;
  }
  __syncthreads();
  for (int r = threadIdx.x / UPR; r < total; r += BATCH * STEP) {
    uint4 A[BATCH], B[BATCH];
    int tt[BATCH], hh[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      A[k] = nA[k];
      B[k] = nB[k];
      tt[k] = nt_[k];
      hh[k] = nh[k];
    }
    read(r + BATCH * STEP);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (r + k * STEP >= total) break;  // the same for the whole row
      const int64_t n = n0 + tt[k];
      const bool is_q = hh[k] < p.Hq, is_k = !is_q && hh[k] < p.Hq + p.Hkv;
      const int g = is_q ? 0 : (is_k ? hh[k] - p.Hq : hh[k] - p.Hq - p.Hkv);
      if (rotated && (is_q || is_k)) rotate_unit(A[k], B[k], cs + tt[k] * 64 + 8 * u, sn + tt[k] * 64 + 8 * u, pairs);
      uint16_t* out = is_q ? p.q_out + (n * p.Hq + hh[k]) * D : is_k && p.k_out ? p.k_out + (n * p.Hkv + g) * D : nullptr;
      if (out) {
        reinterpret_cast<uint4*>(out)[c0] = A[k];
        reinterpret_cast<uint4*>(out)[c1] = B[k];
      }
      if constexpr (FMT != 0) {
        if (is_q) continue;
        const int b = (int)(n / p.dst.n_tok), tok = (int)(n - (int64_t)b * p.dst.n_tok);
        int64_t block, row;
        if (!commit_place(p.dst, b, tok, g, block, row)) continue;  // the same for the whole row
        const int64_t rows = p.dst.is_swa ? p.dst.W : 64;
        uint8_t* base = is_k ? p.dst.k : p.dst.v;
        if constexpr (FMT == 1) {
          uint4* d = reinterpret_cast<uint4*>(base + (block * rows + row) * D * 2);
          d[c0] = A[k];
          d[c1] = B[k];
        } else if constexpr (FMT == 2) {
          const float inv = (is_k ? p.dst.inv_k : p.dst.inv_v)[g];
          uint2* d = reinterpret_cast<uint2*>(base + (block * rows + row) * D);
          auto q8 = [inv](const uint4& x) {
            return make_uint2((uint32_t)pack_e4m3x2(bf_lo(x.x) * inv, bf_hi(x.x) * inv) |
                                  ((uint32_t)pack_e4m3x2(bf_lo(x.y) * inv, bf_hi(x.y) * inv) << 16),
                              (uint32_t)pack_e4m3x2(bf_lo(x.z) * inv, bf_hi(x.z) * inv) |
                                  ((uint32_t)pack_e4m3x2(bf_lo(x.w) * inv, bf_hi(x.w) * inv) << 16));
          };
          d[c0] = q8(A[k]);
          d[c1] = q8(B[k]);
        } else {
          const uint32_t a[4] = {A[k].x, A[k].y, A[k].z, A[k].w}, bb[4] = {B[k].x, B[k].y, B[k].z, B[k].w};
          RowRange rr;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            rr.add(a[x]);
            rr.add(bb[x]);
          }
          rr.reduce<UPR>(group);
          float inv;
          const uint32_t pair = i4_params(rr.lo, rr.hi, rr.finite, inv);
          uint8_t* blk = base + block * i4_block_bytes(rows, D);
          uint32_t* d = reinterpret_cast<uint32_t*>(i4_codes<D>(blk, row));
          d[c0] = i4_pack8(a, rr.lo, inv);
          d[c1] = i4_pack8(bb, rr.lo, inv);
          if (u == 0) *i4_pair<D>(blk, rows, row) = pair;
        }
      }
    }
  }
}

}  // namespace

int launch_rope(const RopeLaunch& L, cudaStream_t stream) {
  RopeParams p{};
  const hswa_rope_desc& R = *L.rope;
  for (int i = 0; i < R.rot_dim / 2; ++i) {
    p.turns[i] = R.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    p.axis[i] = R.axis[i];
  }
  p.rot = R.rot_dim;
  p.interleaved = R.interleaved;
  p.n = L.n;
  p.pos = L.pos;
  p.Hq = L.Hq;
  p.Hkv = L.Hkv;
  p.q = L.q;
  p.q_out = L.q_out;
  p.k = L.k;
  p.k_out = L.k_out;
  p.v = L.v;
  int fmt = 0, sms = L.sms;
  if (L.pool) {
    const hswa_pool_desc& D = L.pool->desc;
    fill_commit_dst(L.pool, L.layer, L.n_tok, L.seq_ids, L.start_pos, L.page_table, L.pt_stride, &p.dst);
    fmt = D.kv_format == HSWA_KV_BF16 ? 1 : D.kv_format == HSWA_KV_FP8_E4M3 ? 2 : 3;
  }
  // tokens per block: the table of a block serves all its heads, so more tokens only amortise the
  // block's fixed cost; a short call takes one token per block to use every SM
  const int tpb = L.n >= (int64_t)sms * 8 ? 4 : 1;
  const int64_t blocks = (L.n + tpb - 1) / tpb;
  if (blocks > 0x7fffffff) {
    set_error("rope: too many tokens");
    return HSWA_ERR_UNSUPPORTED_SHAPE;
  }
#define HSWA_ROPE(DD)                                                              \
  switch (fmt) {                                                                   \
    case 0: rope_kernel<DD, 0><<<(int)blocks, RT, 0, stream>>>(p, tpb); break;     \
    case 1: rope_kernel<DD, 1><<<(int)blocks, RT, 0, stream>>>(p, tpb); break;     \
    case 2: rope_kernel<DD, 2><<<(int)blocks, RT, 0, stream>>>(p, tpb); break;     \
    default: rope_kernel<DD, 3><<<(int)blocks, RT, 0, stream>>>(p, tpb); break;    \
  }
  if (L.d == 128) {
    HSWA_ROPE(128)
  } else {
    HSWA_ROPE(64)
  }
#undef HSWA_ROPE
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("rope: launch failed: %s", cudaGetErrorString(e));
    return HSWA_ERR_CUDA;
  }
  return HSWA_OK;
}

}  // namespace hswa
