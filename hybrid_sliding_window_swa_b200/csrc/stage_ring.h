// stage_ring.h -- a ring of NS stages for copied blocks, read by several readers, each its own blocks.
//
// A barrier of shared memory is awaited by the parity of a phase, so a wait tells a phase from its neighbours only:
// a reader that waits for block b while block b - NS, another reader's, is still on its way into the same stage
// passes at once, since block b - 2 NS had the parity it asks for. Copies to scattered places land in any order, so
// the readers' own progress does not rule that out. Therefore the producer counts the blocks it has issued: it
// issues block b when the stage's readers have released block b - NS, which they did after it had landed, so from
// then on the stage's barrier is in b's phase or past it, and b's reader may wait by parity. (A stage of its own
// for every reader would do as well, but the producer, which issues in order, then stands still for the slowest
// reader: 256 rings of 128 slots x 4 tokens 63.8 us against 60.8.)
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define HSWA_HD __host__ __device__ __forceinline__
#else
#define HSWA_HD inline
#endif

namespace hswa {

template <int NS>
struct StageRing {
  static HSWA_HD int stage(uint32_t block) { return (int)(block % NS); }
  static HSWA_HD uint32_t parity(uint32_t block) { return (block / NS) & 1u; }
  // `issued` blocks have been issued: may the reader of `block` wait for it by parity?
  static HSWA_HD bool may_wait(uint32_t issued, uint32_t block) { return (int32_t)(issued - block) > 0; }
};

}  // namespace hswa
