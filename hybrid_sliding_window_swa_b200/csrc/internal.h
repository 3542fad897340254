// internal.h -- host-side pool object and kernel launch interfaces of libhswa.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/hswa.h"

struct hswa_pool {
  hswa_pool_desc desc;
  int device;        // the CUDA device current at kv_pool_create; every call must run with it current
  int sms;           // its multiprocessor count
  int smem_optin;    // its largest opt-in shared memory per block (bytes)
  uint8_t* base;
  size_t bytes_swa, bytes_full, bytes_scales;
  bool fp8;          // entries are FP8 E4M3 codes (1 byte) instead of bf16 (2 bytes)
  bool i4;           // rows are 4-bit codes with a (step, minimum) pair, see kv_quant.cuh
  int esize;         // bytes per element (bf16 and FP8 pools)
  int64_t ring_blk;  // bytes of one (sequence, layer, KV head) ring block and of one (page, KV head)
  int64_t page_blk;  // block, K or V
  // element arrays (uint16_t for bf16 pools; for FP8 pools the same addresses hold bytes, see *8)
  uint16_t* ring_k;  // [max_seqs][n_swa][Hkv][W][d]
  uint16_t* ring_v;
  uint16_t* page_k;  // [n_full][pages][Hkv][page_size][d]
  uint16_t* page_v;
  uint8_t* ring_k8;  // the same regions as bytes
  uint8_t* ring_v8;
  uint8_t* page_k8;
  uint8_t* page_v8;
  float* scales;     // FP8: [4][n_layers][Hkv] = K scale, V scale, 1/K scale, 1/V scale (device)
  int* err;          // device error word
  bool ring_tma;     // W is a multiple of 128: ring tiles can be fetched with one TMA box
  CUtensorMap tm_ring_k, tm_ring_v;
  bool page_tma;
  CUtensorMap tm_page_k, tm_page_v;
  bool page_tma8;                     // FP8 pools with head_dim 128: pages as byte tiles
  CUtensorMap tm_page_k8, tm_page_v8; // [page_rows][64][128] bytes, 64-row boxes, 128-byte swizzle
};

namespace hswa {

// Thread-local error message of the ABI layer.
void set_error(const char* fmt, ...);

// HSWA_OK when the calling thread's current CUDA device is the pool's device; otherwise
// HSWA_ERR_INVALID_ARG with a message naming `who` (nothing may be launched for the call).
int check_device(const hswa_pool* pool, const char* who);

// The multiprocessor count of the current device (looked up once per device); HSWA_ERR_CUDA on failure.
int current_sms(const char* who, int* sms);

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per kernel and device: `done` is the kernel's own
// static bit mask over devices (devices past 63 set it every time).
#define HSWA_SET_SMEM(kernel, bytes, device)                                                          \
  do {                                                                                                \
    static std::atomic<unsigned long long> done{0};                                                   \
    const unsigned long long bit = (device) < 64 ? 1ull << (device) : 0ull;                           \
    if (!(done.load(std::memory_order_relaxed) & bit) || !bit) {                                      \
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(bytes));        \
      done.fetch_or(bit, std::memory_order_relaxed);                                                  \
    }                                                                                                 \
  } while (0)

// Encode a 2-5 dimensional bf16 tiled tensor map with 128-byte swizzle.
// dims/strides: innermost first; strides in bytes for dims 1.. (dim 0 is contiguous).
bool make_tmap_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                    const uint64_t* strides_bytes, const uint32_t* box);
// The same for 1-byte elements (FP8 codes), 128-byte swizzle.
bool make_tmap_u8(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                  const uint32_t* box);

int launch_append(const hswa_pool* pool, int layer, int n_seqs, const int32_t* seq_ids,
                  const int64_t* start_pos, int n_tok, const uint16_t* k, const uint16_t* v,
                  const int32_t* page_table, int pt_stride, cudaStream_t stream);

// Launch with programmatic dependence on the launch before it in the stream.
template <typename K, typename... A>
inline cudaError_t launch_dependent(K kernel, int grid, int block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The destination of a commit into `layer`, as the commit kernels take it.
void fill_commit_dst(const hswa_pool* pool, int layer, int n_tok, const int32_t* seq_ids, const int64_t* start_pos,
                     const int32_t* page_table, int pt_stride, struct CommitDst* out);

struct RopeLaunch {
  const hswa_rope_desc* rope;
  int d, sms;
  int64_t n;           // tokens
  const int64_t* pos;  // [n_axes][n]
  int Hq, Hkv;
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* k;
  uint16_t* k_out;
  // with a commit (pool not null)
  const hswa_pool* pool;
  int layer, n_tok;
  const uint16_t* v;
  const int32_t* seq_ids;
  const int64_t* start_pos;
  const int32_t* page_table;
  int pt_stride;
};
int launch_rope(const RopeLaunch& L, cudaStream_t stream);

int launch_gather_ring(const hswa_pool* pool, int layer, int dst, const int32_t* src, cudaStream_t stream);

int launch_selftest_wait(int* err, uint64_t limit_ns, cudaStream_t stream);

// Sliding window W = 1: o = v of each query head's KV head (k, q and the ring are not read).
int launch_window1(const hswa_pool* pool, const uint16_t* v, uint16_t* o, int B, int n_q, int Hq, int Hkv, int d,
                   cudaStream_t stream);

int launch_window_safe_len(const int64_t* m, const int64_t* c, const uint32_t* valid, int W, int n_req,
                           int64_t* out, cudaStream_t stream);

struct PrefillLaunch {
  // problem
  int B, n_q, Hq, Hkv, d;
  int window;  // >= 1 for SWA, 0 for full causal
  const int64_t* start_pos;  // device, may be null (all zero)
  const int32_t* seq_ids;    // SWA ring rows
  const int32_t* page_table; // full layers
  int pt_stride;
  uint16_t* o;
  // pool
  const hswa_pool* pool;
  int ring_layer;      // SWA layer index within the ring (SWA)
  int full_layer;      // full layer index within the paged pool (full)
  int layer;           // pool layer index (selects the FP8 scales)
  // tensor maps built by the ABI layer
  CUtensorMap tm_q, tm_k, tm_v;  // tm_k/tm_v: chunk K/V (SWA) or pages (full)
  CUtensorMap tm_o;              // output, stored 32 rows x 64 columns per TMA box
  const hswa_score_mod* mod;     // null: plain scores
  void* workspace;               // with key ranges: prefill_mod_bytes(B, n_q)
};

// Workspace of a prefill with key ranges: per query tile its bounds (16 bytes) and its place in the order.
inline size_t prefill_mod_bytes(int B, int n_q) {
  return (((size_t)B * (((size_t)n_q + 127) / 128) * 20) + 255) & ~(size_t)255;
}

int launch_prefill(const PrefillLaunch& L, cudaStream_t stream);
// Sliding-window prefill with 1 <= W <= 129 (the band of a query tile spans at most two key tiles).
int launch_prefill_narrow(const PrefillLaunch& L, cudaStream_t stream);

struct DecodeLaunch {
  int n_seqs, n_qt, Hq, Hkv, d;
  int layer;   // pool layer index (selects the FP8 scales)
  int window;  // >= 1 SWA (ring), 0 full (pages)
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint16_t* o;
  const int64_t* ctx_len;
  int64_t max_ctx_len;
  const int32_t* seq_ids;
  const int32_t* page_table;
  int pt_stride;
  const hswa_pool* pool;
  int ring_layer, full_layer;
  const hswa_score_mod* mod;  // null: plain scores
  bool ext;                   // 4-bit pool or score modifications: splits of ext_split keys
  void* workspace;
  size_t ws_bytes;
};

// What the size query returns: enough for any call with at most these sequences and this context length.
size_t decode_workspace_bound(int n_seqs, int n_qt, int Hq, int Hkv, int d, int64_t max_ctx_len);
size_t decode_workspace_bytes(int n_seqs, int n_qt, int Hq, int Hkv, int d, int window, int64_t max_ctx_len, bool ext);
// Dynamic shared memory of the split merge for these arguments (0 when no sequence can have two splits).
size_t decode_merge_smem_bytes(int n_seqs, int n_qt, int Hq, int Hkv, int window, int64_t max_ctx_len);
// Work items a call may have at most (a split of one KV head of one sequence each).
int64_t decode_max_items(int n_seqs, int Hkv, int window, int64_t max_ctx_len, bool ext);

// Argument checks shared by hybrid_decode_fwd and hybrid_decode_fwd_noalloc (messages name `who`).
// On HSWA_OK, *L is filled except for workspace/ws_bytes and *need is the scratch the call uses;
// L->n_seqs == 0 means there is nothing to launch.
int prepare_decode(hswa_pool* pool, const char* who, int layer, const uint16_t* q, const uint16_t* k_new,
                   const uint16_t* v_new, uint16_t* o, int n_seqs, int n_q_per_seq, const int64_t* ctx_len,
                   int64_t max_ctx_len, const int32_t* seq_ids, const int32_t* page_table, int pt_stride,
                   int n_q_heads, const hswa_score_mod* mod, DecodeLaunch* L, size_t* need);
int launch_decode(const DecodeLaunch& L, cudaStream_t stream);

}  // namespace hswa
