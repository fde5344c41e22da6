// One tile of a down product: 128 token rows of a large bf16 matrix times a
// rank-R operand, streamed through an LDS ring (u = x A^T, v = g B).
#pragma once

#include "ring.h"

namespace qlora {

namespace sk {
constexpr int DT = 128;   // down: tokens per workgroup (32 per wave)
constexpr int DCH = 8;    // down: 16-byte chunks per token row and stage (8 CH k)
constexpr int TJ = 128;   // token: columns per workgroup (32 per wave)
constexpr int TS = 64;    // token: tokens per stage
}  // namespace sk

// kYT: Y is given as [k][q] (B itself, R = 16 RB ranks, rows past yrows
// read as zero) instead of [q][k]; its stage tile keeps that layout (KS rows
// of 32 RB bytes, loaded as contiguous 1 KB blocks) and the MFMA operand is
// read transposed with ds_read_b64_tr_b16, so v = g B needs no copy of B^T.
// kPartRank: then R may also be a smaller multiple of 8, and the tile's columns
// from R on read as zero.  dst: this split's M x R sums.
template <int RB, int NS, int CH, bool kYT, bool kPartRank>
__device__ __forceinline__ void skinny_down_tile(const uint16_t* __restrict__ X, int64_t M, int64_t K,
                                                 const uint16_t* __restrict__ Y, int R, float* __restrict__ dst,
                                                 int64_t kc, int64_t yrows, int64_t t0, int split) {
  static_assert(CH == 8 || CH == 16, "row chunks per stage");
  static_assert(!kYT || CH == 8, "transposed rank operand: 64 k per stage");
  constexpr int KS = 8 * CH;               // k per stage
  constexpr int RPB = 64 / CH;             // rows per 1 KB load block
  constexpr int XPW = 32 / RPB;            // X blocks per wave (its 32 token rows)
  // Rank rows: 16 RB rows of CH chunks, in 1 KB blocks, YPW per wave (every
  // wave issues the same number of loads; blocks past the rank rows read
  // zeros into the padding)
  constexpr int YBLK = (16 * RB) / RPB;
  constexpr int YPW = YBLK >= 4 ? YBLK / 4 : 1;
  constexpr int XB = sk::DT * 16 * CH;     // 128 token rows x KS k
  constexpr int YB = 4 * YPW * 1024;
  constexpr int STAGE = XB + YB;
  __shared__ __align__(16) uint8_t s0[STAGE];
  __shared__ __align__(16) uint8_t s1[STAGE];
  __shared__ __align__(16) uint8_t s2[NS > 2 ? STAGE : 16];
  __shared__ __align__(16) uint8_t s3[NS > 3 ? STAGE : 16];
  uint8_t* const buf4[4] = {s0, s1, s2, s3};
  uint8_t* buf[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) buf[i] = buf4[i];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15;
  const int lq = lane >> 4;
  const int64_t kbeg = (int64_t)split * kc;
  const int64_t kend = (kbeg + kc < K) ? kbeg + kc : K;
  const int nst = (int)cdiv(kend - kbeg, KS);
  const uint32_t xbytes = (uint32_t)(M * K * 2);
  const uint32_t ybytes = (uint32_t)((int64_t)R * (kYT ? yrows : K) * 2);
  const brsrc_t rx = make_rsrc(X, xbytes);
  const brsrc_t ry = make_rsrc(Y, ybytes);
  // A 1 KB load block holds RPB rows: lane l lands in row l / CH of the
  // block at slot l % CH, which holds chunk (l % CH) ^ (row % CH) (swch).
  const int drow = lane / CH;
  const int dslot = lane % CH;
  constexpr int LMIN = XPW + YPW;
  auto issue = [&](int s, uint8_t* stg) {
    const int64_t kb = kbeg + (int64_t)s * KS;
#pragma unroll
    for (int b = 0; b < XPW; ++b) {  // this wave's token rows 32 w .. 32 w + 31
      const int row = 32 * wave + RPB * b + drow;
      const int64_t k = kb + 8 * (dslot ^ (row & (CH - 1)));
      const int64_t t = t0 + row;
      dma16(rx, stg + (32 * wave + RPB * b) * (16 * CH), (k < kend && t < M) ? (uint32_t)((t * K + k) * 2) : xbytes);
    }
#pragma unroll
    for (int j = 0; j < YPW; ++j) {
      const int blk = wave + 4 * j;
      if constexpr (kYT) {
        // rows kb + 1024 / (32 RB) blk .. of B, 2 RB lanes a row (KS rows in all)
        const int row = (1024 / (32 * RB)) * blk + lane / (2 * RB);
        const int64_t k = kb + row;
        const int c = lane % (2 * RB);
        const bool ok = k < kend && row < KS && (!kPartRank || 8 * c < R);
        dma16(ry, stg + XB + blk * 1024, ok ? (uint32_t)((k * R + 8 * c) * 2) : ybytes);
      } else {
        const int q = RPB * blk + drow;
        const int64_t k = kb + 8 * (dslot ^ (q & (CH - 1)));
        dma16(ry, stg + XB + blk * 1024, (k < kend && q < R) ? (uint32_t)(((int64_t)q * K + k) * 2) : ybytes);
      }
    }
  };
  f32x4 acc[2][RB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < RB; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const uint8_t* stg) {
#pragma unroll
    for (int kk = 0; kk < CH / 4; ++kk) {
      u32x4 bq[RB];
#pragma unroll
      for (int cb = 0; cb < RB; ++cb) {
        if constexpr (kYT) {
          // k rows 32 kk + 8 lq + 4 h + lr / 4, ranks 16 cb + 4 (lr % 4) .. + 3
          const uint8_t* src = stg + XB + (32 * kk + 8 * lq + (lr >> 2)) * (32 * RB) + 2 * (16 * cb + 4 * (lr & 3));
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)src);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 4 * (32 * RB)));
          const u32x2 l2 = __builtin_bit_cast(u32x2, lo);
          const u32x2 h2 = __builtin_bit_cast(u32x2, hi);
          bq[cb] = u32x4{l2[0], l2[1], h2[0], h2[1]};
        } else {
          bq[cb] = *reinterpret_cast<const u32x4*>(stg + XB + swch<CH>(16 * cb + lr, 4 * kk + lq));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(stg + swch<CH>(32 * wave + 16 * i + lr, 4 * kk + lq));
#pragma unroll
        for (int cb = 0; cb < RB; ++cb) acc[i][cb] = mfma16x16x32(a, bq[cb], acc[i][cb]);
      }
    }
  };
  ring_run<NS, LMIN>(nst, buf, issue, compute);

  // lane holds tokens 32 w + 16 i + 4 lq + e, rank 16 cb + lr
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int cb = 0; cb < RB; ++cb) {
      const int q = 16 * cb + lr;
      if (q >= R) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t t = t0 + 32 * wave + 16 * i + 4 * lq + e;
        if (t < M) dst[t * R + q] = acc[i][cb][e];
      }
    }
}

}  // namespace qlora
