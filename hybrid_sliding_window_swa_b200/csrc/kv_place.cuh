// kv_place.cuh -- where one (sequence, token, KV head) row of a commit goes in the pool.
#pragma once
#include "common.cuh"

namespace hswa {

// The destination of a commit into one layer (device pointers of the pool, by value in a launch).
struct CommitDst {
  uint8_t* k;  // ring or page region of the pool, K and V
  uint8_t* v;
  const int64_t* start_pos;   // [n_seqs]
  const int32_t* seq_ids;     // SWA layers
  const int32_t* page_table;  // full layers
  int pt_stride;
  int is_swa, W, n_swa, layer, max_seqs, Hkv, n_tok;
  int64_t pages;
  const float* inv_k;  // FP8 pools: reciprocal scales of the layer
  const float* inv_v;
  int* err;
};

// Where a row goes: `block` indexes the (ring row, KV head) or (page, KV head) block, `row` the row
// inside it. False when the row is not written (superseded within the chunk, or out of bounds; the
// latter is recorded).
__device__ __forceinline__ bool commit_place(const CommitDst& c, int b, int t, int g, int64_t& block, int64_t& row) {
  const int64_t pos = c.start_pos[b] + t;
  if (c.is_swa) {
    if (t < c.n_tok - c.W) return false;  // overwritten later in the same chunk
    const int seq = c.seq_ids[b];
    if (seq < 0 || seq >= c.max_seqs || pos < 0) {
      record_error(c.err, HSWA_ERR_DEVICE_BOUNDS);
      return false;
    }
    block = ((int64_t)seq * c.n_swa + c.layer) * c.Hkv + g;
    row = pos % c.W;
  } else {
    const int64_t lp = pos >> 6;
    if (pos < 0 || lp >= c.pt_stride) {
      record_error(c.err, HSWA_ERR_DEVICE_BOUNDS);
      return false;
    }
    const int32_t page = c.page_table[(int64_t)b * c.pt_stride + lp];
    if (page < 0 || page >= c.pages) {
      record_error(c.err, HSWA_ERR_DEVICE_BOUNDS);
      return false;
    }
    block = ((int64_t)c.layer * c.pages + page) * c.Hkv + g;
    row = pos & 63;
  }
  return true;
}

}  // namespace hswa
