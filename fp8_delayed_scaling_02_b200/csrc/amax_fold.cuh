// The end of every delayed-scaling call, shared by the kernels that write an
// FP8 tensor: block amax -> one atomic per block -> ticket -> the last block
// folds the ring.
#pragma once

#include "common.cuh"
#include "fp8_ring.cuh"

namespace fp8ds {

// Three modes: fold (history set, amax_out null), local (amax_out set: the
// last block writes the grid's amax and scale_inv and does not fold; the
// fold follows after a cross-rank MAX of the amax) and fixed scale (both
// null: current scaling's cast pass).
struct RingArgs {
  float* history;
  int32_t* idx;
  float* scale;
  float* scale_inv;
  uint32_t* scratch;
  float* amax_out;
};

// Block-reduce the per-thread amax, publish it with one atomicMax, draw a
// ticket; the last of the `nblocks` blocks working on this ring folds it.
// Must be called by every thread of the block.
// The ring's history and idx are not written until the last block runs, so
// each block reads them early (prefetch_ring at kernel start, one lane per
// word) and the fold itself needs no dependent global reads besides the
// amax word.
struct RingCache {
  float hist;  // history[threadIdx.x] for threads 0..15
  int idx;     // read by thread 16
};

__device__ __forceinline__ RingCache prefetch_ring(const RingArgs& ring) {
  RingCache c{0.0f, 0};
  if (ring.history == nullptr || ring.amax_out != nullptr) return c;  // no fold in this call
  if (threadIdx.x < kHistoryLen) c.hist = ring.history[threadIdx.x];
  if (threadIdx.x == kHistoryLen) c.idx = *ring.idx;
  return c;
}

// Adds a block's amax m (>= 0) to the ring's amax word and draws the block's
// ticket (its arrival number among the blocks on this ring).  No fence: the
// max is an atom that returns only once the word holds the block's amax, and
// the ticket's address is computed from that return (bit 31 of a
// non-negative float's bits: 0 at run time, opaque to the compiler), so the
// ticket cannot be issued before the amax update is performed in L2.  The
// block that draws the last ticket exchanges the amax word only after that
// ticket returned -- after every other block's ticket, hence after every
// other block's amax update, was performed at the same L2 location.  Every
// global atomic a block issued earlier (the TMA producer's tile claims) must
// have returned before the block's final barrier for the same reason.  A
// release-ordered ticket would wait for the block's own output stores to
// complete; without it a 12.6M-element bf16 row quantize takes 8.6 instead of
// 9.0 us on B200.
__device__ __forceinline__ unsigned publish_amax_take_ticket(uint32_t* scratch, float m) {
  uint32_t old, dep, t;
  asm volatile("atom.relaxed.gpu.global.max.u32 %0, [%1], %2;" : "=r"(old) : "l"(scratch), "r"(__float_as_uint(m))
               : "memory");
  asm volatile("shr.u32 %0, %1, 31;" : "=r"(dep) : "r"(old));
  asm volatile("atom.relaxed.gpu.global.add.u32 %0, [%1], 1;" : "=r"(t) : "l"(scratch + 1 + dep) : "memory");
  return t;
}

// One thread's end of its block's work on a ring: the block's amax m goes in,
// and the block with the last of `nblocks` tickets clears the scratch words
// and folds (or, in local mode, writes the amax out).  hist holds the 16
// history values as they were at launch, idx the slot to write; s_used is the
// scale the call multiplied by.
template <int FMT>
__device__ __forceinline__ void commit_block_amax(float m, const RingArgs& ring, float s_used, float* hist, int idx,
                                                  const unsigned nblocks) {
  // (A single 64-bit compare-and-swap carrying amax and ticket was tried:
  // hundreds of blocks finishing together made its retries quadratic.)
  const unsigned t = publish_amax_take_ticket(ring.scratch, m);
  if (t != nblocks - 1) return;
  uint32_t bits;
  asm volatile("atom.relaxed.gpu.global.exch.b32 %0, [%1], 0;" : "=r"(bits) : "l"(ring.scratch) : "memory");
  const float a = __uint_as_float(bits);
  asm volatile("st.relaxed.gpu.global.u32 [%0], 0;" ::"l"(ring.scratch + 1) : "memory");
  asm volatile("st.relaxed.gpu.global.u32 [%0], 0;" ::"l"(ring.scratch + 2) : "memory");  // tile counter
  if (ring.amax_out != nullptr) {
    // Local mode: this rank's amax for the cross-rank MAX; the scale the
    // call used is already known, so its inverse is published now.
    *ring.amax_out = a;
    *ring.scale_inv = __frcp_rn(s_used);
    return;
  }
  ring_commit<FMT>(a, hist, idx, ring.history, ring.idx, ring.scale, ring.scale_inv, s_used);
}

template <int FMT, int NT = 256>
__device__ __forceinline__ void amax_ticket_fold(float amax, const RingArgs& ring, float s_used,
                                                 const RingCache& rc, const unsigned nblocks) {
  __shared__ float warp_max[NT / 32];
  __shared__ float hist_s[kHistoryLen];
  __shared__ int idx_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if (lane == 0) warp_max[warp] = amax;
  if (threadIdx.x < kHistoryLen) hist_s[threadIdx.x] = rc.hist;
  if (threadIdx.x == kHistoryLen) idx_s = rc.idx;
  __syncthreads();
  if (ring.history == nullptr && ring.amax_out == nullptr) {
    // Fixed scale: no amax to publish; the last block clears the scratch
    // words (the tile counter is shared by every kernel that claims tiles).
    if (threadIdx.x == 0) {
      unsigned t;
      asm volatile("atom.relaxed.gpu.global.add.u32 %0, [%1], 1;" : "=r"(t) : "l"(ring.scratch + 1) : "memory");
      if (t == nblocks - 1) {
        asm volatile("st.relaxed.gpu.global.u32 [%0], 0;" ::"l"(ring.scratch + 1) : "memory");
        asm volatile("st.relaxed.gpu.global.u32 [%0], 0;" ::"l"(ring.scratch + 2) : "memory");
      }
    }
    return;
  }
  if (threadIdx.x == 0) {
    float m = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) m = fmaxf(m, warp_max[w]);
    commit_block_amax<FMT>(m, ring, s_used, hist_s, idx_s, nblocks);
  }
}

}  // namespace fp8ds
