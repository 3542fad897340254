// decode_i4.cuh -- the decode step over a 4-bit pool (included by decode.cu, which holds the work
// list, the parameters and the merge of the splits).
//
// Math. A cached row stands for code * step + lo (kv_quant.cuh), so with k = step_k c + lo_k:
//   q . k = step_k (q . c) + lo_k sum(q),      o = sum_j p_j v_j = sum_j (p_j step_j) c_j + sum_j p_j lo_j.
// Both products therefore run on the codes themselves. An f16 with exponent field 0 is a subnormal:
// its value is its mantissa times 2^-24. A code masked out of its word is such a number, code * 2^-24
// for the low nibble of a byte and code * 2^-20 for the high one, without any conversion: five integer
// instructions turn a 32-bit word of eight codes into four f16 pairs of an MMA operand. The two
// factors are powers of two and are folded into Q (whose entries at odd dims are staged divided by 16)
// and, for O, into the output.
//
// Orientation. S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16: keys (and dims of V) fill the 16
// rows, query rows come in groups of 8 columns, so a step of one token with 8 heads per KV head wastes
// nothing. The codes go from shared memory to A fragments as they lie:
//   K  lane (g, t) reads 16 bytes (D = 128) of key pi(g): 32 dims, whose order inside the dot product
//      is free as long as Q is staged in the same order;
//   V  lane (g, t) reads the bytes of its 16 dims (16 g ..) of keys t, 4 + (t ^ 1), 8 + t, 12 + (t ^ 1);
//      two keys' words are interleaved by a byte permute, then masked. pi (the order of the 16 keys
//      along S^T's rows) makes these the keys 2t, 2t+1, 2t+8, 2t+9 of the P^T fragment; neighbours in
//      it differ in parity, so the K reads are free of bank conflicts and the V reads two-way (64-byte
//      rows).
// P (times the key's V step) is rounded to f16 (11 bits; an fp32 sum keeps l and sum p lo) and turned
// from accumulator to operand layout by movmatrix.
// f16 range: Q is staged with its row maximum at 2^14 .. 2^15 and the factor kept in fp32. The weights are
// p = 2^(z - off), where each query row's offset, a whole number, is held so that p step stays below 2^15: it moves
// when that might be passed, to the place where the largest p step is at most 2^7, and l, sum p lo and O are
// rescaled (O, l and sum p lo carry the same factor, which cancels in the end). Only keys that the row sees count:
// another token of the step may see values of any size. P keeps its 11 bits down to 2^-21 of the row's largest
// p step (for V steps of 2^-89 to 2^100; beyond them the small weights leave the fp32 or the f16 range). A minimum
// counts as a step of 2^-20 of its size, and a step as at least 2^-89, which keeps sum p lo and l finite.
//
// What bounds it. 2 (d / 2 + 4) bytes per key and KV head. Up to 8 rows the reads do: 5.2 TB/s while the items
// of a 256K-token sequence run (70 us the call; its 285 MB take 43 us). With 32 rows the instruction dispatch
// does: integer 40%, MMA 40%, fp32 14% of the cycles (ncu), which add up; neither more warps nor more
// registers nor issuing the next block's S among the V products moved it.
//
// Structure: 4 consumer warps and a producer warp per CTA, two CTAs per SM, taking items from the work
// list. A block is one 64-key page: (codes, pairs) of K and of V are contiguous, one bulk copy each
// (ring rows: the codes in one or two runs, the pairs row by row with cp.async), several blocks ahead, across items. The
// producer also hands over the item's geometry and its Q rows. The warps take blocks in turn (for more
// than 16 rows in pairs, half the rows each), 32 keys at a time so that enough independent MMAs are
// in flight, and merge their softmax states at the end of the item.
// A stage is read by whichever warp its block falls to, so a block is awaited only once it has been issued
// (stage_ring.h). Waits are bounded; a failing wait makes its warp return and the others run out theirs.

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Arrive on the barrier when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// mma_f16 with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The count of issued blocks (stage_ring.h), written by the producer and read by the consumers.
__device__ __forceinline__ void set_issued(uint32_t* word, uint32_t n) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(word)), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t get_issued(const uint32_t* word) {
  uint32_t n;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(n) : "r"(smem_u32(word)) : "memory");
  return n;
}

// Wait (bounded, the whole warp) until `block` has been issued; `seen` is the count last read.
template <int NS>
__device__ __forceinline__ bool wait_issued(const uint32_t* word, uint32_t block, uint32_t& seen, int* err) {
  if (StageRing<NS>::may_wait(seen, block)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    seen = __shfl_sync(0xffffffffu, get_issued(word), 0);
    if (StageRing<NS>::may_wait(seen, block)) return true;
    if ((it & 255u) == 0) {
      const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
      if (late) record_error(err, HSWA_ERR_TIMEOUT);
      if (__any_sync(0xffffffffu, late || read_error(err) != 0)) return false;
    }
  }
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// What a row's (step, minimum) pair counts as a step, and the whole number above the log2 of such a count.
__device__ __forceinline__ float i4_size(uint32_t pair) {
  return fmaxf(__uint_as_float(pair << 16), fabsf(__uint_as_float(pair & 0xFFFF0000u)) * 9.5367432e-7f);
}
__device__ __forceinline__ float i4_log2(float size) { return (float)(max(__float_as_int(size) >> 23, 38) - 126); }

// 4 consumer warps, two CTAs per SM, 32 keys of a warp in flight. Measured against (us, 256K-token sequence /
// mixed batch with drafts, cold L2; here 78 / 655): 6 warps 78 / 1001 (its 128 registers spill), 8 warps in
// one CTA 113 / 721, 12 warps 115 / 1014, 16 keys in flight 111 / 752, 64 keys 111 / 655.
constexpr int I4_WARPS = 4;
constexpr int I4_CTAS = 2;
constexpr int I4_KU = 2;  // 16-key groups
constexpr int I4_THREADS = (I4_WARPS + 1) * 32;
constexpr float I4_NO_OFF = -3e38f;  // the offset of a row that has seen no key: any key moves it

// One work item as the producer hands it to the consumers.
struct I4Item {
  int item, s, g, L;
  int a, b;              // cached keys [a, b) of this split
  int n_cached, n_blk;   // blocks of cached keys, blocks with the new tokens
  int nsp;               // splits of the sequence
  uint32_t cnt0;         // blocks before its first one (their place in the stage ring)
  int lo_min, lo_max;    // over the rows: smallest and largest first visible position
  int hi_min, hi_max;    // smallest and largest end of the visible ranges
  int row_lo[8], row_hi[8];  // per new token
};

// SOLO: many short items of one split each (the ring of a large batch), where most of an item's ~9.5 us went into
// its hand-over, the merge of the warps' states and the waits of warps without a block. A team
// of RG warps takes a whole item, its rows divided, so that no states are merged and the teams of a CTA do not
// wait for one another; items are (sequence, KV head) in order, without a plan kernel.
template <int D, int NT, int RG, bool SOLO>
struct I4Smem {
  static constexpr int ROWS = 8 * NT * RG;
  static constexpr int TEAMS = SOLO ? I4_WARPS / RG : 1;
  static constexpr int SLOTS = 2 * TEAMS;  // items handed out ahead
  static constexpr int BLK = (int)i4_block_bytes(64, D);
  static constexpr int STAGE = 2 * BLK;
  static constexpr int Q_BYTES = ROWS * D * 2;
  static constexpr int AREA_STRIDE = D + 4;  // floats
  static constexpr int Q_OFF = 0;
  static constexpr int AREA_OFF = Q_OFF + SLOTS * Q_BYTES;
  static constexpr int AREAS = SOLO ? 0 : I4_WARPS / RG;  // one per warp of a row group
  static constexpr int ML_OFF = AREA_OFF + AREAS * ROWS * AREA_STRIDE * 4;
  // offset, l, sum p lo per (warp, row), then per row
  static constexpr int ROW_OFF = ML_OFF + (SOLO ? 0 : (3 * I4_WARPS * ROWS + 3 * ROWS) * 4);  // per row: token, output offset
  static constexpr int ITEM_OFF = ROW_OFF + 2 * ROWS * 4;
  static constexpr int MAX_NS = 32;
  static constexpr int BAR_OFF = (ITEM_OFF + SLOTS * (int)sizeof(I4Item) + 15) / 16 * 16;
  static constexpr int STAGE_OFF = (BAR_OFF + (2 * MAX_NS + 2 * SLOTS + 1) * 8 + 16 + 127) / 128 * 128;
  // as many blocks in flight as the shared memory of I4_CTAS CTAs per SM allows
  static constexpr int FIT = (227 * 1024 / I4_CTAS - 1024 - STAGE_OFF) / STAGE;
  static constexpr int NS = FIT < MAX_NS ? FIT : MAX_NS;
  static constexpr int BYTES = STAGE_OFF + NS * STAGE;
  static_assert(NS >= 4, "blocks in flight");
  using Ring = StageRing<NS>;
};

template <int D, int NT, int RG, int MODE, bool SOLO>
__global__ void __launch_bounds__(I4_THREADS, I4_CTAS) decode_i4_kernel(DecParams p) {
  constexpr bool MOD = MODE != PLAIN;
  using SM = I4Smem<D, NT, RG, SOLO>;
  constexpr int ROWS = SM::ROWS;
  constexpr int NS = SM::NS;
  constexpr int SLOTS = SM::SLOTS, TEAMS = SM::TEAMS;
  using Ring = typename SM::Ring;
  constexpr int KW = I4_WARPS / RG / TEAMS;  // warps that share an item's row group
  constexpr int KU = I4_KU;
  constexpr int NW = D / 32;           // 32-bit words of K codes per lane
  constexpr int MT = D / 16;           // m-tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::BAR_OFF);
  uint64_t* empty = full + SM::MAX_NS;
  uint64_t* item_full = empty + SM::MAX_NS;
  uint64_t* item_empty = item_full + SLOTS;
  uint64_t* cons = item_empty + SLOTS;
  int* go = reinterpret_cast<int*>(cons + 1);
  uint32_t* issued = reinterpret_cast<uint32_t*>(go + 1);  // blocks issued, see stage_ring.h
  I4Item* items = reinterpret_cast<I4Item*>(smem + SM::ITEM_OFF);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  WsHeader* hdr = reinterpret_cast<WsHeader*>(p.ws);

  // what the producer needs first is read before the barriers are set up
  const bool fixed = SOLO || p.small;  // items are worked out here, not read from a plan
  const int err0 = fixed && tid == 0 ? read_error(p.err) : 0;
  int sp_L = 0, sp_body = 0, sp_excl = 0, sp_total = 0;
  if (!SOLO && p.small && warp == I4_WARPS) {
    const SmallPlan sp(p);
    sp_L = sp.L;
    sp_body = sp.body;
    sp_excl = sp.excl;
    sp_total = sp.total;
  }
  int* row_tok = reinterpret_cast<int*>(smem + SM::ROW_OFF);  // new token of a query row
  int* row_out = row_tok + ROWS;  // its place in the output, from (sequence, first token, first head of g)
  for (int r = tid; r < ROWS; r += I4_THREADS) {
    const int t = r < p.R ? r / p.G : 0;
    row_tok[r] = t;
    row_out[r] = (t * p.Hq + (r - t * p.G)) * D;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 33);  // the producer's 32 lanes and its byte count
      mbar_init(&empty[i], RG);  // the warps that read a block
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], I4_WARPS / TEAMS);
    }
    mbar_init(cons, I4_WARPS);
    *issued = 0;
    fence_barrier_init();
  }
  grid_go();    // the merge may take its place; it waits for this grid's end before it reads
  grid_wait();  // the work list
  if (tid == 0) *go = (fixed ? err0 : read_error(p.err)) == 0;
  __syncthreads();
  if (!*go) return;  // a pending device error: skip the work

  if (warp == I4_WARPS) {
    // ------------------------------------------------------------ producer
    const PlanView pv(p.ws, p.n_seqs);
    int total, body_total;
    if constexpr (SOLO) {
      body_total = 0;
      total = p.n_seqs * p.Hkv;
    } else if (p.small) {
      body_total = sp_total;
      total = (sp_total + p.n_seqs) * p.Hkv;
    } else {
      body_total = hdr->body_total;
      total = hdr->total_items;
    }
    uint32_t cnt = 0;  // blocks issued
    int it = 0, ends = 0;
    bool ok = true;
    for (;; ++it) {
      const int slot = it % SLOTS;
      if (!(ok = warp_wait(&item_empty[slot], ((it / SLOTS) & 1) ^ 1, p.err))) break;
      int item = 0;
      if (fixed) {
        item = blockIdx.x + it * (int)gridDim.x;
      } else {
        if (lane == 0) item = atomicAdd(&hdr->counter, 1);
        item = __shfl_sync(0xffffffffu, item, 0);
      }
      I4Item& I = items[slot];
      if (item >= total || item < 0) {
        if (lane == 0) {
          I.item = -1;
          mbar_arrive(&item_full[slot]);
        }
        if (++ends == TEAMS) break;  // every team has been told
        continue;
      }
      const int g = item % p.Hkv;
      const int sc = item / p.Hkv;
      int s, c, L, nsp;
      if constexpr (SOLO) {
        s = sc;
        c = 0;
        L = (int)safe_len(p, s);
        nsp = 1;
      } else if (p.small) {
        if (sc < body_total) {
          // the last sequence whose prefix is not past sc (those without body splits share a prefix
          // with their successor)
          s = 31 - __clz(__ballot_sync(0xffffffffu, lane < p.n_seqs && sp_excl <= sc));
          c = sc - __shfl_sync(0xffffffffu, sp_excl, s);
        } else {
          s = sc - body_total;
          c = -1;
        }
        L = __shfl_sync(0xffffffffu, sp_L, s);
        nsp = __shfl_sync(0xffffffffu, sp_body, s) + 1;
      } else if (sc < body_total) {
        int lo = 0, hi = p.n_seqs;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (pv.prefix[mid] <= sc) lo = mid; else hi = mid;
        }
        s = pv.order[lo];
        c = sc - pv.prefix[lo];
      } else {
        s = pv.tail[sc - body_total];
        c = -1;
      }
      if (!fixed) {
        L = (int)safe_len(p, s);
        nsp = n_splits_x<true>(p, s, L);
      }
      int64_t klo64, khi64;
      cached_range<true>(p, s, L, klo64, khi64);
      const int klo = (int)klo64, khi = (int)khi64;
      if (c < 0) c = nsp - 1;
      const int a = klo + c * p.split;
      const int b = khi - a > p.split ? a + p.split : khi;  // (a + split may pass 2^31)
      const int n_cached = b > a ? (b - a + 63) / 64 : 0;
      const int n_blk = n_cached + (c == nsp - 1 ? 1 : 0);
      // visible range of each new token's rows, by lane
      int rlo = 0, rhi = 0x7fffffff;
      row_range(p, s, L, lane < p.n_qt ? lane : 0, rlo, rhi);
      // (a row may see nothing)
      int lo_min = rhi > rlo ? rlo : 0x7fffffff, hi_max = rhi > rlo ? rhi : 0, lo_max = rlo, hi_min = rhi;
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) {
        lo_min = min(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, x));
        lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, x));
        hi_min = min(hi_min, __shfl_xor_sync(0xffffffffu, hi_min, x));
        hi_max = max(hi_max, __shfl_xor_sync(0xffffffffu, hi_max, x));
      }
      if (lane < 8) {
        I.row_lo[lane] = rlo;
        I.row_hi[lane] = rhi;
      }
      __syncwarp();
      if (lane == 0) {
        I.item = item;
        I.s = s;
        I.g = g;
        I.L = L;
        I.a = a;
        I.b = b;
        I.n_cached = n_cached;
        I.n_blk = n_blk;
        I.nsp = nsp;
        I.cnt0 = cnt;
        I.lo_min = lo_min;
        I.lo_max = lo_max;
        I.hi_min = hi_min;
        I.hi_max = hi_max;
        const uint32_t row_bytes = p.G * D * 2;
        mbar_arrive_expect_tx(&item_full[slot], p.n_qt * row_bytes);
        uint8_t* dst = smem + SM::Q_OFF + slot * SM::Q_BYTES;
        for (int t = 0; t < p.n_qt; ++t)
          bulk_load(dst + t * row_bytes, p.q + (((int64_t)s * p.n_qt + t) * p.Hq + g * p.G) * D, row_bytes,
                    &item_full[slot]);
      }
      // sources
      int64_t ring_block = -1;
      if (p.window > 0 && n_cached > 0) {
        const int seq = p.seq_ids[s];
        if (seq < 0 || seq >= p.max_seqs) {
          if (lane == 0) record_error(p.err, HSWA_ERR_DEVICE_BOUNDS);
        } else {
          ring_block = ((int64_t)seq * p.n_swa + p.ring_layer) * p.Hkv + g;
        }
      }
      const int32_t* pt_row = p.page_table ? p.page_table + (int64_t)s * p.pt_stride : nullptr;
      int my_page = -1;
      for (int kb = 0; kb < n_blk; ++kb, ++cnt) {
        const int st = Ring::stage(cnt);
        if (p.window <= 0 && (kb & 31) == 0) {
          const int lp = (a >> 6) + kb + lane;
          my_page = kb + lane < n_cached && lp < p.pt_stride ? pt_row[lp] : -1;
        }
        if (!(ok = warp_wait(&empty[st], Ring::parity(cnt) ^ 1, p.err))) break;
        if (lane == 0) set_issued(issued, cnt + 1);
        uint8_t* ks = smem + SM::STAGE_OFF + st * SM::STAGE;
        uint8_t* vs = ks + SM::BLK;
        if (kb < n_cached && p.window <= 0) {
          const int page = __shfl_sync(0xffffffffu, my_page, kb & 31);
          if (page >= 0 && page < p.pages) {
            if (lane == 0) {
              const int64_t off = (((int64_t)p.full_layer * p.pages + page) * p.Hkv + g) * SM::BLK;
              mbar_arrive_expect_tx(&full[st], 2 * SM::BLK);
              bulk_load(ks, p.src_k8 + off, SM::BLK, &full[st]);
              bulk_load(vs, p.src_v8 + off, SM::BLK, &full[st]);
            }
          } else {
            // rows that stand for zero
            if (lane == 0) record_error(p.err, HSWA_ERR_DEVICE_BOUNDS);
            for (int r = lane; r < 64; r += 32) {
              *i4_pair<D>(ks, 64, r) = 0u;
              *i4_pair<D>(vs, 64, r) = 0u;
            }
            fence_proxy_async_smem();
            if (lane == 0) mbar_arrive(&full[st]);
          }
          mbar_arrive(&full[st]);
        } else if (kb < n_cached) {
          const int pos0 = a + kb * 64;
          const int nvalid = min(64, b - pos0);
          if (ring_block >= 0) {
            const uint8_t* rk = p.src_k8 + ring_block * p.blk_bytes;
            const uint8_t* rv = p.src_v8 + ring_block * p.blk_bytes;
            const int slot0 = pos0 % p.window;
            auto wrap = [&](int r) {
              int x = slot0 + r;
              if (x >= p.window) x = p.window >= 64 ? x - p.window : x % p.window;
              return x;
            };
            // codes: one run of slots, or two where the ring wraps (nvalid < W); pairs are 4-byte copies
            if (lane == 0) {
              const int n0 = min(nvalid, p.window - slot0);
              mbar_arrive_expect_tx(&full[st], nvalid * D);  // K and V
              bulk_load(ks, rk + (int64_t)slot0 * (D / 2), n0 * (D / 2), &full[st]);
              bulk_load(vs, rv + (int64_t)slot0 * (D / 2), n0 * (D / 2), &full[st]);
              if (n0 < nvalid) {
                bulk_load(ks + n0 * (D / 2), rk, (nvalid - n0) * (D / 2), &full[st]);
                bulk_load(vs + n0 * (D / 2), rv, (nvalid - n0) * (D / 2), &full[st]);
              }
            }
            const int64_t pair0 = (int64_t)p.window * (D / 2);
            for (int r = lane; r < nvalid; r += 32) {
              const int64_t off = pair0 + (int64_t)wrap(r) * 4;
              cp_async_4(smem_u32(i4_pair<D>(ks, 64, r)), rk + off);
              cp_async_4(smem_u32(i4_pair<D>(vs, 64, r)), rv + off);
            }
          } else {
            for (int r = lane; r < 64; r += 32) {
              *i4_pair<D>(ks, 64, r) = 0u;
              *i4_pair<D>(vs, 64, r) = 0u;
            }
            if (lane == 0) mbar_arrive(&full[st]);
          }
          fence_proxy_async_smem();
          cp_async_arrive(&full[st]);
        } else {
          // the new tokens, as the cache will hold them: D / 8 lanes per row
          constexpr int LPR = D / 8;
          constexpr int RPP = 32 / LPR;  // rows per pass
          const unsigned group = ((1u << LPR) - 1u) << (lane & ~(LPR - 1));
          const int ch = lane % LPR;
          for (int r0 = 0; r0 < p.n_qt; r0 += RPP) {
            const int r = r0 + lane / LPR;
            const bool live = r < p.n_qt;
            const int64_t row = ((int64_t)s * p.n_qt + (live ? r : 0)) * p.Hkv + g;
            const uint4 xk = __ldg(reinterpret_cast<const uint4*>(p.k_new + row * D) + ch);
            const uint4 xv = __ldg(reinterpret_cast<const uint4*>(p.v_new + row * D) + ch);
            const uint32_t wk[4] = {xk.x, xk.y, xk.z, xk.w}, wv[4] = {xv.x, xv.y, xv.z, xv.w};
            RowRange ak, av;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ak.add(wk[i]);
              av.add(wv[i]);
            }
            ak.reduce<LPR>(group);
            av.reduce<LPR>(group);
            float ik, iv;
            const uint32_t pk = i4_params(ak.lo, ak.hi, ak.finite, ik), pv2 = i4_params(av.lo, av.hi, av.finite, iv);
            if (live) {
              reinterpret_cast<uint32_t*>(i4_codes<D>(ks, r))[ch] = i4_pack8(wk, ak.lo, ik);
              reinterpret_cast<uint32_t*>(i4_codes<D>(vs, r))[ch] = i4_pack8(wv, av.lo, iv);
              if (ch == 0) {
                *i4_pair<D>(ks, 64, r) = pk;
                *i4_pair<D>(vs, 64, r) = pv2;
              }
            }
          }
          fence_proxy_async_smem();
          if (lane == 0) mbar_arrive(&full[st]);
          mbar_arrive(&full[st]);
        }
      }
      if (!ok) break;
    }
    if (!ok) {
      // copies in flight must land before the CTA may end (bounded; the error word is already set)
      const uint32_t first = cnt > (uint32_t)NS ? cnt - NS : 0;
      for (uint32_t x = first; x < cnt; ++x) (void)mbar_wait_limit(&full[Ring::stage(x)], Ring::parity(x), nullptr, kWaitLimitNs);
      for (int x = it >= SLOTS ? it - SLOTS + 1 : 0; x <= it; ++x)
        (void)mbar_wait_limit(&item_full[x % SLOTS], (x / SLOTS) & 1, nullptr, 10000000ull);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g8 = lane >> 2, t4 = lane & 3;
  const int rg = RG == 2 ? warp & 1 : 0;
  const int pos = RG == 2 ? warp >> 1 : warp;
  const int kw = SOLO ? 0 : pos;
  const int row0 = rg * 8 * NT;
  // key of S^T row g8 within a 16-key group (row g8 + 8: + 8), see the header comment
  const int pi0 = (g8 & 1) ? 4 + ((g8 >> 1) ^ 1) : g8 >> 1;
  float* m_w = reinterpret_cast<float*>(smem + SM::ML_OFF);  // [KW][ROWS] offsets (-inf: no key seen)
  float* l_w = m_w + I4_WARPS * ROWS;
  float* b_w = l_w + I4_WARPS * ROWS;
  float* m_all = b_w + I4_WARPS * ROWS;
  float* l_all = m_all + ROWS;
  float* b_all = l_all + ROWS;
  float* area = reinterpret_cast<float*>(smem + SM::AREA_OFF);  // [AREAS][ROWS][AREA_STRIDE]
  uint32_t ncons = 0;
  uint32_t n_issued = 0;  // as last read
  auto cons_sync = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(cons);
    return warp_wait(cons, (ncons++) & 1, p.err);
  };

  for (int it = SOLO ? pos : 0;; it += TEAMS) {
    const int slot = it % SLOTS;
    if (!warp_wait(&item_full[slot], (it / SLOTS) & 1, p.err)) return;
    const I4Item& I = items[slot];
    if (I.item < 0) return;
    const uint32_t cnt = I.cnt0;
    const int L = I.L, ia = I.a, ib = I.b, n_cached = I.n_cached, n_blk = I.n_blk;

    // ---- Q fragments: lane (g8, t4) holds dims [t4 D/4, +D/4) of row g8 of each n-tile
    uint32_t qf[NT][NW][4];
    float c1[NT][2], c2[NT][2];  // score = c1 (acc * step + lo * c2)
    float slope[NT][2];
    int r_pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g8;
      const bool live = r < p.R;
      const uint4* src = reinterpret_cast<const uint4*>(smem + SM::Q_OFF + slot * SM::Q_BYTES + r * (D * 2)) +
                         t4 * (D / 32);
      uint32_t w[4 * NW];
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const uint4 x = live ? src[i] : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
      }
      float mx = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NW; ++i) {
        const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xFFFF0000u);
        mx = fmaxf(mx, fmaxf(fabsf(x0), fabsf(x1)));
        sum += x0 + x1;
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      int e = (__float_as_int(mx) >> 23) - 127;
      e = e < -110 ? -110 : (e > 115 ? 115 : e);
      const float f_lo = pow2i(14 - e), f_hi = f_lo * 0.0625f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        // dims 8i .. 8i + 7: w[4i + j] holds dims 2j, 2j + 1
        auto lo = [&](int j) { return __uint_as_float(w[4 * i + j] << 16) * f_lo; };
        auto hi = [&](int j) { return __uint_as_float(w[4 * i + j] & 0xFFFF0000u) * f_hi; };
        qf[nt][i][0] = pack_f16x2(lo(0), lo(2));
        qf[nt][i][1] = pack_f16x2(hi(0), hi(2));
        qf[nt][i][2] = pack_f16x2(lo(1), lo(3));
        qf[nt][i][3] = pack_f16x2(hi(1), hi(3));
      }
      // scores from the accumulator: acc * 2^(e - 14 + 24) * step + lo * sum(q), times the softmax scale
      const float a1 = (MOD ? p.scale_nat : p.scale_log2) * pow2i(e + 10), a2 = sum * pow2i(-e - 10);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        c1[nt][c] = __shfl_sync(0xffffffffu, a1, (2 * t4 + c) * 4);
        c2[nt][c] = __shfl_sync(0xffffffffu, a2, (2 * t4 + c) * 4);
        if constexpr (MOD) {
          const int rr = row0 + nt * 8 + 2 * t4 + c;
          const int tok = row_tok[rr];
          r_pos[nt][c] = L + tok;
          slope[nt][c] = p.slope && rr < p.R ? p.slope[I.g * p.G + rr % p.G] * 1.4426950408889634f : 0.f;
        }
      }
    }

    float o[MT][NT][4];
    float off[NT][2], l[NT][2], bs[NT][2];
    float ws[NT][2];  // sum of the weights as V takes them (p step) since they last left O, see below
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        off[nt][c] = I4_NO_OFF;
        l[nt][c] = 0.f;
        bs[nt][c] = 0.f;
        ws[nt][c] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    uint32_t n_done = 0;     // blocks this warp has added to O
    const int lo_min = I.lo_min, lo_max = I.lo_max, hi_min = I.hi_min, hi_max = I.hi_max;

    for (int kb = kw; kb < n_blk; kb += KW) {
      const uint32_t cb = cnt + kb;
      const int st = Ring::stage(cb);
      if (!wait_issued<NS>(issued, cb, n_issued, p.err) || !warp_wait(&full[st], Ring::parity(cb), p.err)) return;
      uint8_t* ks = smem + SM::STAGE_OFF + st * SM::STAGE;
      uint8_t* vs = ks + SM::BLK;
      const bool is_new = kb >= n_cached;
      const int kbase = is_new ? L : ia + kb * 64;
      const int kend = min(is_new ? L + p.n_qt : ib, hi_max);  // no key any row sees at or past this
      const bool edge = kbase + 64 > min(kend, hi_min) || kbase < lo_max;
#pragma unroll 1
      for (int k0 = 0; k0 < 64; k0 += 16 * KU) {
        if (edge && (kbase + k0 >= kend || kbase + k0 + 16 * KU <= lo_min)) continue;  // nothing here
        // ---- S^T = K Q^T, KU groups of 16 keys
        float acc[KU][NT][4];
        uint32_t kp[KU][2], vp[KU][2];
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          const int key0 = k0 + 16 * u;
          uint32_t wl[NW], wh[NW];
          const uint8_t* a0 = i4_codes<D>(ks, key0 + pi0) + t4 * (D / 8);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(a0), y = *reinterpret_cast<const uint4*>(a0 + 8 * (D / 2));
            wl[0] = x.x; wl[1] = x.y; wl[2] = x.z; wl[3] = x.w;
            wh[0] = y.x; wh[1] = y.y; wh[2] = y.z; wh[3] = y.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(a0), y = *reinterpret_cast<const uint2*>(a0 + 8 * (D / 2));
            wl[0] = x.x; wl[1] = x.y;
            wh[0] = y.x; wh[1] = y.y;
          }
          kp[u][0] = *i4_pair<D>(ks, 64, key0 + pi0);
          kp[u][1] = *i4_pair<D>(ks, 64, key0 + pi0 + 8);
          vp[u][0] = *i4_pair<D>(vs, 64, key0 + pi0);
          vp[u][1] = *i4_pair<D>(vs, 64, key0 + pi0 + 8);
#pragma unroll
          for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t x = wl[i] >> (8 * h), y = wh[i] >> (8 * h);
              const uint32_t a0 = x & 0x000F000Fu, a1 = y & 0x000F000Fu, a2 = x & 0x00F000F0u, a3 = y & 0x00F000F0u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (i == 0 && h == 0)
                  mma_f16_zero(acc[u][nt], a0, a1, a2, a3, qf[nt][0][0], qf[nt][0][1]);
                else
                  mma_f16(acc[u][nt], a0, a1, a2, a3, qf[nt][i][2 * h], qf[nt][i][2 * h + 1]);
              }
            }
        }
        if (edge) {  // rows no query row sees may hold anything: they stand for zero
#pragma unroll
          for (int u = 0; u < KU; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int key = kbase + k0 + 16 * u + pi0 + 8 * k;
              if (key >= kend || key < lo_min) kp[u][k] = vp[u][k] = 0u;
            }
        }
        // ---- scores in the log2 domain, masks
#pragma unroll
        for (int u = 0; u < KU; ++u) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float ksf = __uint_as_float(kp[u][k] << 16), klf = __uint_as_float(kp[u][k] & 0xFFFF0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float z = fmaf(acc[u][nt][2 * k + c], ksf, klf * c2[nt][c]);
                if constexpr (MOD) {
                  const int key = kbase + k0 + 16 * u + pi0 + 8 * k;
                  z *= c1[nt][c];
                  z = MODE == LARGE_CAP || p.softcap > 0.f ? capped_score<MODE>(z, p.cap_in, p.cap_log2) : z * 1.4426950408889634f;
                  if (p.slope) z = fmaf(-slope[nt][c], (float)abs(r_pos[nt][c] - key), z);
                }
                acc[u][nt][2 * k + c] = z;
              }
          }
        }
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int tok = row_tok[row0 + nt * 8 + 2 * t4 + c];
              const int r_lo = I.row_lo[tok], r_hi = min(I.row_hi[tok], kend);
#pragma unroll
              for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int key = kbase + k0 + 16 * u + pi0 + 8 * k;
                  if (key < r_lo || key >= r_hi) acc[u][nt][2 * k + c] = -INFINITY;
                }
            }
        }
        // Does a row's largest score go with the largest step of this lane's keys? (More than needed where they are
        // two keys, or the step is one that the row does not see; which rows have to move is looked at below.)
        float size = 0.f;
#pragma unroll
        for (int u = 0; u < KU; ++u) size = fmax3(size, i4_size(vp[u][0]), i4_size(vp[u][1]));
        const float room = 15.f - i4_log2(size);
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(acc[0][nt][c], acc[0][nt][2 + c]);
#pragma unroll
            for (int u = 1; u < KU; ++u) mx = fmax3(mx, acc[u][nt][c], acc[u][nt][2 + c]);
            move = move || (MOD ? mx - off[nt][c] : fmaf(mx, c1[nt][c], -off[nt][c])) > room;
          }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = -INFINITY;  // the largest log2 (p step) but for the offset
#pragma unroll
              for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float lq = i4_log2(i4_size(vp[u][k]));
                  mx = fmaxf(mx, MOD ? acc[u][nt][2 * k + c] + lq : fmaf(acc[u][nt][2 * k + c], c1[nt][c], lq));
                }
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
              if (mx - off[nt][c] > 15.f) {  // the same in the row's lanes
                const float to = ceilf(mx) - 7.f;
                const float f = ex2_approx(off[nt][c] - to);
                off[nt][c] = to;
                l[nt][c] *= f;
                bs[nt][c] *= f;
                ws[nt][c] *= f;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  o[i][nt][c] *= f;
                  o[i][nt][2 + c] *= f;
                }
              }
            }
        }
        // ---- softmax weights, O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          uint32_t pb[NT][2];
          const float vsf[2] = {__uint_as_float(vp[u][0] << 16), __uint_as_float(vp[u][1] << 16)};
          const float vlf[2] = {__uint_as_float(vp[u][0] & 0xFFFF0000u), __uint_as_float(vp[u][1] & 0xFFFF0000u)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
            // the two rows of a lane together (packed operations: half the instructions)
            uint64_t l2 = f2_pack(l[nt][0], l[nt][1]), b2 = f2_pack(bs[nt][0], bs[nt][1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float e[2];
#pragma unroll
              for (int c = 0; c < 2; ++c)
                e[c] = ex2_approx(MOD ? acc[u][nt][2 * k + c] - off[nt][c]
                                      : fmaf(acc[u][nt][2 * k + c], c1[nt][c], -off[nt][c]));
              const uint64_t e2 = f2_pack(e[0], e[1]);
              l2 = f2_add(l2, e2);
              b2 = f2_fma(e2, f2_pack(vlf[k], vlf[k]), b2);
              const uint64_t w2 = f2_mul(e2, f2_pack(vsf[k], vsf[k]));
              f2_unpack(w2, w[2 * k], w[2 * k + 1]);
              if constexpr (!SOLO) f2_unpack(f2_add(f2_pack(ws[nt][0], ws[nt][1]), w2), ws[nt][0], ws[nt][1]);
            }
            f2_unpack(l2, l[nt][0], l[nt][1]);
            f2_unpack(b2, bs[nt][0], bs[nt][1]);
            pb[nt][0] = movmatrix_t(pack_f16x2(w[0], w[1]));
            pb[nt][1] = movmatrix_t(pack_f16x2(w[2], w[3]));
          }
          // this lane's dims [g8 D/8, +D/8) of keys t4, 4 + (t4 ^ 1) and the same + 8
          const uint8_t* v0 = i4_codes<D>(vs, k0 + 16 * u + t4) + g8 * (D / 16);
          const uint8_t* v1 = i4_codes<D>(vs, k0 + 16 * u + 4 + (t4 ^ 1)) + g8 * (D / 16);
          constexpr int VW = D / 64;  // words per key
          uint32_t vw[4][VW];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint8_t* src = ((j & 1) ? v1 : v0) + (j >> 1) * 8 * (D / 2);
            if constexpr (VW == 2) {
              const uint2 x = *reinterpret_cast<const uint2*>(src);
              vw[j][0] = x.x;
              vw[j][1] = x.y;
            } else {
              vw[j][0] = *reinterpret_cast<const uint32_t*>(src);
            }
          }
#pragma unroll
          for (int h = 0; h < VW; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              // four dims (8h + 4q ..) of the two key pairs
              const uint32_t u0 = __byte_perm(vw[0][h], vw[1][h], q ? 0x7632u : 0x5410u);
              const uint32_t u1 = __byte_perm(vw[2][h], vw[3][h], q ? 0x7632u : 0x5410u);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t x0 = u0 >> (8 * y), x1 = u1 >> (8 * y);
                const uint32_t a0 = x0 & 0x000F000Fu, a1 = x0 & 0x00F000F0u;
                const uint32_t a2 = x1 & 0x000F000Fu, a3 = x1 & 0x00F000F0u;
                const int i = 4 * h + 2 * q + y;  // dims 2i (rows 0-7) and 2i + 1 (rows 8-15) of this lane's
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(o[i][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
              }
            }
        }
      }
      // Every 4 blocks, move the codes' mean out of O: sum P c is 7.5 sum p step plus a small rest, and the
      // tensor core's accumulation truncates, so over thousands of keys the rest (all that is left after
      // sum p lo is added) lost 0.2% of its size to the large common part. Any S may be taken from O as long
      // as the same S is added to sum p lo; S = 7.5 (sum p step since the last time), the rows' own weights: a
      // step of which a row sees little (a far larger V row of weight 0) must not enter its O. (A team's contexts
      // of at most 512 keys stay below 2^-17 of the sum without that: 32 accumulations.)
      if (!SOLO && (++n_done & 3u) == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float d = ws[nt][c];
            ws[nt][c] = 0.f;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
            const float S = 7.5f * d;
            bs[nt][c] = fmaf(0.125f, S, bs[nt][c]);  // the 8 lanes of a row are summed at the end
            const float se = S * 5.9604645e-8f, so = S * 9.5367432e-7f;  // 2^-24, 2^-20
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][nt][c] -= se;
              o[i][nt][2 + c] -= so;
            }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // ---- merge the warps' states
    const int s = I.s, hg = I.g, nsp = I.nsp, item = I.item;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
          bs[nt][c] += __shfl_xor_sync(0xffffffffu, bs[nt][c], x);
        }
    if constexpr (SOLO) {
      // the whole row is here: lane (g8, t4) holds dims [g8 D/8, +D/8) of rows 2 t4 and 2 t4 + 1
      uint16_t* out = p.o + ((int64_t)s * p.n_qt * p.Hq + hg * p.G) * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = row0 + nt * 8 + 2 * t4 + c;
          const float inv = l[nt][c] == 0.f ? 0.f : 1.f / l[nt][c];  // (a row that sees nothing: 0)
          const float b0 = bs[nt][c];
          uint32_t w[MT];
#pragma unroll
          for (int i = 0; i < MT; ++i)
            w[i] = pack_bf16x2(fmaf(o[i][nt][c], 16777216.f, b0) * inv,
                               fmaf(o[i][nt][2 + c], 1048576.f, b0) * inv);
          if (r < p.R) {
            uint4* dst = reinterpret_cast<uint4*>(out + row_out[r] + g8 * (D / 8));
#pragma unroll
            for (int i = 0; i < MT; i += 4) dst[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      continue;
    }
    if (it > 0 && !cons_sync()) return;  // the previous item's output has been read
    if (lane == 0) mbar_arrive(&item_empty[slot]);
    if (g8 == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = row0 + nt * 8 + 2 * t4 + c;
          m_w[kw * ROWS + r] = off[nt][c] == I4_NO_OFF ? -INFINITY : off[nt][c];
          l_w[kw * ROWS + r] = l[nt][c];
          b_w[kw * ROWS + r] = bs[nt][c];
        }
    }
    if (!cons_sync()) return;
    if (tid < ROWS) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < KW; ++w) M = fmaxf(M, m_w[w * ROWS + tid]);
      const float Mo = M == -INFINITY ? 0.f : M;
      float ls = 0.f, bb = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float f = ex2_approx(m_w[w * ROWS + tid] - Mo);
        ls += l_w[w * ROWS + tid] * f;
        bb += b_w[w * ROWS + tid] * f;
      }
      m_all[tid] = M;
      l_all[tid] = nsp == 1 ? (ls == 0.f ? 0.f : 1.f / ls) : ls;  // (a row that sees nothing: 0)
      b_all[tid] = bb;
    }
    {
      float f[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = row0 + nt * 8 + 2 * t4 + c;
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < KW; ++w) M = fmaxf(M, m_w[w * ROWS + r]);
          f[nt][c] = M == -INFINITY ? 0.f : ex2_approx(off[nt][c] - M);
        }
      // O^T accumulators: dims 2i hold 2^-24, dims 2i + 1 hold 2^-20 of the sum
      {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = row0 + nt * 8 + 2 * t4 + c;
            float* dst = area + (kw * ROWS + r) * SM::AREA_STRIDE + g8 * (D / 8);
#pragma unroll
            for (int i = 0; i < MT; i += 2) {
              const float4 y = make_float4(o[i][nt][c] * f[nt][c] * 16777216.f, o[i][nt][2 + c] * f[nt][c] * 1048576.f,
                                     o[i + 1][nt][c] * f[nt][c] * 16777216.f,
                                     o[i + 1][nt][2 + c] * f[nt][c] * 1048576.f);
              *reinterpret_cast<float4*>(dst + 2 * i) = y;
            }
          }
      }
      if (!cons_sync()) return;
    }
    // ---- output: bf16 rows when the sequence has one split, else this item's partial
    auto merged4 = [&](int r, int c) -> float4 {
      const float bb = b_all[r];
      float4 x = make_float4(bb, bb, bb, bb);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(area + (w * ROWS + r) * SM::AREA_STRIDE + c);
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
      }
      return x;
    };
    float* part = reinterpret_cast<float*>(p.ws + p.part_off + (size_t)item * p.part_bytes);
    uint16_t* out = p.o + ((int64_t)s * p.n_qt * p.Hq + hg * p.G) * D;
#pragma unroll 4
    for (int idx = tid; idx < p.R * (D / 4); idx += I4_WARPS * 32) {
      const int r = idx / (D / 4), c = (idx % (D / 4)) * 4;
      float4 x = merged4(r, c);
      if (nsp == 1) {
        const float inv = l_all[r];
        x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        uint2 pk;
        pk.x = pack_bf16x2(x.x, x.y);
        pk.y = pack_bf16x2(x.z, x.w);
        *reinterpret_cast<uint2*>(out + row_out[r] + c) = pk;
      } else {
        *reinterpret_cast<float4*>(part + r * D + c) = x;
      }
    }
    if (nsp > 1) {
      for (int r = tid; r < p.R; r += I4_WARPS * 32) {
        part[p.R * D + r] = m_all[r];
        part[p.R * D + p.R + r] = l_all[r];
      }
    }
  }
}
