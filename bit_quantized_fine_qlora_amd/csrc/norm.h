// Shared by the norm's forward and backward kernels: how a row is held.
#pragma once

#include "rows.h"

namespace qlora {

constexpr int64_t kNormMaxWidth = 16384;

// A row is held by NW waves, VPT pieces of 8 values a thread: piece i of
// thread t is at column 8 (t + 64 NW i); 512 NW VPT >= n.
//   up to   512 values  1 wave, 1 piece a thread
//   up to  1024         1 wave, 2 pieces: no barrier (65536 x 1000 bf16 rms
//                       forward 48 us, 59 us with 2 waves of one and a barrier
//                       a row; backward 90 and 91 us)
//   up to  2048         4 waves, 1 piece, and
//   up to  4096         8 waves, 1 piece: with half the waves and two pieces the
//                       backward's gradient sums and rows in flight leave too
//                       few waves a CU (16384 x 1500 bf16 layer 40 us, 51 us
//                       so; 4096 x 4096 28 and 35 us); the forward alone would
//                       gain by it (29 and 25 us; 17 and 15 us)
//   up to  8192         forward 8 waves, 2 pieces (8192 x 8192 bf16 layer 49 us,
//                       70 us with 16 waves of one), backward 16 waves, 1 piece
//                       (8192 x 5120 layer 51 us, 53 us with 8 waves of two;
//                       8192 x 8192 81 and 80 us)
//   up to 16384         8 waves, 4 pieces
template <bool kBwd, typename F>
static void norm_shape(int64_t n, F f) {
  using std::integral_constant;
#define QLORA_SHAPE(NW_, VPT_) f(integral_constant<int, NW_>{}, integral_constant<int, VPT_>{})
  if (n <= 512) QLORA_SHAPE(1, 1);
  else if (n <= 1024) QLORA_SHAPE(1, 2);
  else if (n <= 2048) QLORA_SHAPE(4, 1);
  else if (n <= 4096) QLORA_SHAPE(8, 1);
  else if (n > 8192) QLORA_SHAPE(8, 4);
  else if constexpr (kBwd) QLORA_SHAPE(16, 1);
  else QLORA_SHAPE(8, 2);
#undef QLORA_SHAPE
}

// Rows of a workgroup: four waves of a row each where one wave holds a row.
__host__ __device__ constexpr int norm_rows(int nw) { return nw == 1 ? 4 : 1; }

// This thread's pieces of a row: load_row sends out the loads, finish_row,
// where the values are used, leaves zeros past the row's end (load_piece8,
// finish_piece8).  Rows of fewer than 8 values come one by one.
template <int XT, int VPT>
__device__ __forceinline__ void load_row(const RowSrc& s, int64_t row, int n, int t, int threads,
                                         Raw8<XT> (&r)[VPT]) {
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = load_piece8<XT>(s, row, n, 8 * (t + threads * i));
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = Raw8<XT>{};
    if (t == 0) r[0] = load_tail8<XT>(s, row, n, 0, n);
  }
}
template <int XT, int VPT>
__device__ __forceinline__ void finish_row(int n, int t, int threads, Raw8<XT> (&r)[VPT]) {
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = finish_piece8<XT>(r[i], n, 8 * (t + threads * i));
  }
}

// Sum of a value over the NW waves that share a row, the waves' sums added in
// 64 bits; every wave gets it.  Slots are taken in turn, as in row_sums below.
template <int NW>
__device__ __forceinline__ double row_sum64(float v, float (&red)[2][NW], int& turn, int wave) {
  v = wave_sum(v);
  if constexpr (NW == 1) {
    return (double)v;
  } else {
    auto& slot = red[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) slot[wave] = v;
    __syncthreads();
    double s = (double)slot[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) s += (double)slot[i];
    return s;
  }
}

// v^(-1/2): the hardware's 64-bit estimate, good to about 2^-23, and one Newton
// step, r + r (1 - v r^2) / 2; at 0 and infinity, where the step has no value,
// the estimate itself.
__device__ __forceinline__ float inverse_root(double v) {
  const double r = __builtin_amdgcn_rsq(v);
  const double e = __builtin_fma(-v * r, r, 1.0);
  return (float)(e == e ? __builtin_fma(0.5 * r, e, r) : r);
}

// Sums of K values over the NW waves that share a row; every wave gets them.
// Calls take the two slots of `red` in turn: a wave writes a slot again only
// after the barrier of the call between, which no wave reaches before it has
// read the slot.
template <int NW, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (&red)[2][K][NW], int& turn, int wave) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (NW > 1) {
    auto& slot = red[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) slot[k][wave] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = slot[k][0];
#pragma unroll
      for (int i = 1; i < NW; ++i) v[k] += slot[k][i];
    }
  }
}

}  // namespace qlora
