// Pieces shared by the kernels that stream a large bf16 matrix through an LDS
// ring filled by direct-to-LDS loads: waits, barrier, the ring's loop, and the
// tile layouts whose reads are free of bank conflicts.
#pragma once

#include "qlora_common.h"

namespace qlora {

__host__ __device__ static inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// X tile: row t, 16-byte piece c (columns 8c..8c+7).  Rows t, t+1, t+2, t+3,
// t+8, .. t+11 put a given 32-byte unit in 8 different bank groups.
__device__ __forceinline__ uint32_t swtg(int t, int c) {
  const int f = (t & 3) | (((t >> 3) & 1) << 2);
  return (uint32_t)(t * 256 + ((((c >> 1) ^ f)) << 5) + ((c & 1) << 4));
}
// Y planes: row q holds 64 tokens (128 B) in 16-byte chunks of 8 tokens.
__device__ __forceinline__ uint32_t swy(int q, int chunk) {
  return (uint32_t)(q * 128 + ((chunk ^ ((q >> 1) & 7)) << 4));
}

// s_waitcnt vmcnt(N) with the other counters unconstrained
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// The same with the wave's LDS reads done too (lgkmcnt(0)): in front of a
// barrier behind which another wave may load into what they read.  The compiler
// waits for a read where its value is used, which may be behind the barrier.
template <int N>
__device__ __forceinline__ void wait_vmcnt_lds() {
  static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
}

// One direct-to-LDS load of 16 bytes per lane: lane l writes bytes
// 16 l .. 16 l + 15 of the 1 KB block at `blk`.
__device__ __forceinline__ void dma16(brsrc_t r, uint8_t* blk, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)blk, 16, voff, 0, 0, 0);
}

// 16-byte chunk c (0..7) of row `row` in a tile of 128-byte rows sits at
// slot c ^ (row % 8): 16x16x32 fragment reads and 1 KB block writes are free
// of bank conflicts.
__device__ __forceinline__ uint32_t sw128(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

// Workgroup barrier without __syncthreads' memory fence, which the compiler
// lowers to a wait for every load in flight (the whole ring).  The ring's
// own vmcnt wait makes this wave's loads of the stage complete, the barrier
// makes every wave's, and LDS needs no cache maintenance; the empty asm
// statements keep the compiler from moving memory accesses across it.
__device__ __forceinline__ void ring_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The ring: stage s lives in buffer s % NS; step s waits for stage s (and for
// its own reads of stage s - 1), issues stage s + NS - 1 into the buffer of stage s - 1 (free after the barrier)
// and computes stage s.  Loads are issued unconditionally: stages past the
// end read only out-of-range offsets (zeros, no memory traffic) into buffers
// nobody reads again.  So before the wait of step s exactly the stages
// s .. s + NS - 2 are in flight, and since loads retire in order, allowing
// the later stages' loads to stay outstanding leaves stage s complete (LMIN:
// the loads every wave issues per stage; waves that issue more only wait
// longer).  A conditional issue would make the compiler wait for every load
// in flight where the paths meet, so the steady-state loop runs whole rings
// and the remaining steps follow it.  The final wait keeps late loads from
// writing LDS after the workgroup has ended.
template <int NS, int LMIN, typename Issue, typename Compute>
__device__ __forceinline__ void ring_run(int nst, uint8_t* const (&buf)[NS], Issue issue, Compute compute) {
  static_assert(NS >= 3 && NS <= 4, "ring depth");
#pragma unroll
  for (int u = 0; u < NS - 1; ++u) issue(u, buf[u]);
  auto step = [&](int s, int u) {
    wait_vmcnt_lds<LMIN * (NS - 2)>();
    ring_barrier();
    issue(s + NS - 1, buf[(u + NS - 1) % NS]);
    compute(buf[u]);
  };
  const int full = nst - nst % NS;
  for (int s0 = 0; s0 < full; s0 += NS) {
#pragma unroll
    for (int u = 0; u < NS; ++u) step(s0 + u, u);
  }
#pragma unroll
  for (int u = 0; u < NS - 1; ++u)
    if (full + u < nst) step(full + u, u);
  wait_vmcnt<0>();
}

// CH 16-byte chunks (8 CH k) per token row and stage: chunk c of row r
// sits at slot c ^ (r % CH), so 16x16x32 fragment reads are conflict-free.
template <int CH>
__device__ __forceinline__ uint32_t swch(int row, int c) {
  return (uint32_t)(row * (16 * CH) + ((c ^ (row & (CH - 1))) << 4));
}

}  // namespace qlora
