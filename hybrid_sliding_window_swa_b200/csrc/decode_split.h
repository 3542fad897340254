// decode_split.h -- how a decode call cuts its cached keys into splits, from the sizes the host knows.
#pragma once
#include <stdint.h>

namespace hswa {

#ifndef HSWA_DECODE_SPLIT
#define HSWA_DECODE_SPLIT 8192
#endif
constexpr int SPLIT = HSWA_DECODE_SPLIT;  // cached keys per split (tuning parameter, multiple of KB)
static_assert(SPLIT % 64 == 0, "splits start on page boundaries");

constexpr int64_t kExtCtas = 296;  // two CTAs on each of 148 SMs

// The most cached keys the rows of a sequence see (the first row of a full ring: all slots but the one that its own
// key takes).
inline int64_t max_cached(int window, int64_t max_ctx_len) {
  return window > 0 && max_ctx_len >= window ? window - 1 : max_ctx_len;
}

// Largest split count of any sequence for these arguments.
inline int64_t max_splits(int window, int64_t max_ctx_len, int split = SPLIT) {
  const int64_t nsp = (max_cached(window, max_ctx_len) + split - 1) / split;
  return nsp < 1 ? 1 : nsp;
}

// Keys per split of an extended launch (4-bit pools, modified scores). One sequence: as many equal splits as
// fill the resident CTAs once (a second round would pay the start and the merge of an item again: 104 us
// against 89 us for 256K tokens). Several sequences, whose lengths may differ: about four items per CTA if
// all were of the largest length, but at least 2048 keys (an item costs some 4 us besides its reads) unless
// one round would not be full. At most 8192 keys, as in the other launches.
inline int ext_split(int n_seqs, int Hkv, int window, int64_t max_ctx_len) {
  const int64_t cached = max_cached(window, max_ctx_len);
  const int64_t pairs = (int64_t)n_seqs * Hkv > 0 ? (int64_t)n_seqs * Hkv : 1;
  auto cut = [&](int64_t n) { return (cached + n - 1) / n; };
  int64_t split = cut(kExtCtas / pairs > 1 ? kExtCtas / pairs : 1);
  if (n_seqs > 1) {
    const int64_t fine = cut((4 * kExtCtas + pairs - 1) / pairs);
    const int64_t least = split < 2048 ? split : 2048;
    split = fine > least ? fine : least;
  }
  // a context of a few pages is one split: its 4 warps walk 8 blocks in less than a merge and its launch
  // take (400 keys: 10.2 us a call against 12.3 with splits of 256; 613 keys: 12.3 against 11.7)
  if (cached <= 512) return 512;
  split = (split + 63) / 64 * 64;
  return (int)(split < 256 ? 256 : (split > SPLIT ? SPLIT : split));
}

// What hybrid_decode_workspace_size promises for extended launches: at least the items of any call with at
// most these sequences and this context length, and growing with both (the exact count need not: fewer
// sequences may be cut finer).
inline int64_t ext_items_bound(int n_seqs, int Hkv, int64_t max_ctx_len) {
  const int64_t pairs = (int64_t)n_seqs * Hkv;
  const int64_t coarse = pairs * max_splits(0, max_ctx_len, SPLIT), fine = pairs * max_splits(0, max_ctx_len, 2048);
  const int64_t least = kExtCtas + pairs > fine ? kExtCtas + pairs : fine;
  const int64_t finest = pairs * max_splits(0, max_ctx_len, 256);
  int64_t cut = 4 * kExtCtas + pairs < least ? 4 * kExtCtas + pairs : least;
  if (cut > finest) cut = finest;
  return coarse > cut ? coarse : cut;
}

// 4-bit pools: is a whole item given to a team of warps? That takes contexts that are never split (a team reads
// its sequence to the end and nothing merges), short ones, and many items.
// Measured (us a call, 4 warps per item / a team;
// d = 128, 8 KV heads): 296 sequence-heads of 128 keys x 32 rows 19.1 / 14.5, 2048 of them 75.6 / 53.4; 384 keys
// x 32 rows 24.0 / 23.9 and 120 / 105, x 16 rows 19.1 / 19.2 and 84.9 / 78.9; 512 keys x 16 rows 95 / 110, x 8
// rows 16.4 / 14.9 and 66.3 / 63.0. With up to 32 sequences the other way has no plan kernel either and wins
// with few items (256 of 128 keys x 32 rows: 12.7 / 14.2).
inline bool i4_teams(int n_seqs, int Hkv, int rows, int window, int64_t max_ctx_len) {
  if (max_splits(window, max_ctx_len, ext_split(n_seqs, Hkv, window, max_ctx_len)) != 1) return false;
  return max_cached(window, max_ctx_len) <= (rows <= 8 ? 512 : 384) &&
         (int64_t)n_seqs * Hkv > (n_seqs > 32 ? 256 : 2 * kExtCtas);
}

}  // namespace hswa
