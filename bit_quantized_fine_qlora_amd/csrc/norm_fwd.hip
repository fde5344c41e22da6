// Layer norm and RMS norm of the rows of an M x n tensor.
//   layer: mean = sum x / n, rstd = (sum (x - mean)^2 / n + eps)^(-1/2)
//   rms:   mean = 0,         rstd = (sum x^2 / n + eps)^(-1/2)
//   y = (x - mean) rstd w + b
// A row stays in registers between its uses, so x is read from memory once;
// the variance is the mean of squared differences (a second pass over the
// registers), not a difference of means.  From a wave's sum on the statistics
// are in 64 bits and each of them is rounded to fp32 once: in fp32 throughout,
// rstd's error was half as large again (0.75 against 0.49 units of 2^-24 in
// the mean square at 8192 values, 0.45 being the last rounding's) at the same
// time.  With a checkpoint asked for, y is also written in 8 bits while it is
// in registers, which saves the packing kernel's read.  Bound by HBM (operands
// that no cache holds): 8192 x 8192 bf16 rms 50 us (268 MB, 5.4 TB/s; a plain
// copy moves 5.0-5.3), with the checkpoint 65-67 us (338 MB), layer with a bias
// 49 and 64 us.  2049 x 5001 fp32, two rows a workgroup, is not: rms 22 us,
// layer 23 us (82 MB, 3.6-3.7 TB/s).
#include "norm.h"

namespace qlora {

struct NormFwdArgs {
  int n;
  int64_t M;
  float eps;
  double inv_n;
  const void* x;
  const void* w;
  const void* b;  // may be null
  void* y;
  float* mean;
  float* rstd;
  int8_t* codes;  // checkpoint of y, may be null (bf16 only)
  uint8_t* scales;
};

// Persistent workgroups walk the rows; the next row's loads go out before
// the current row is reduced.  kKeepBias: the bias stays in registers.  Loaded
// in each row it is waited for after the next row's loads, which go out before
// it, and makes every row wait for those.
template <bool kLayer, bool kKeepBias, int XT, int WT, int NW, int VPT>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void norm_fwd_kernel(NormFwdArgs a) {
#pragma clang fp contract(off)  // the same roundings in every instantiation
  __shared__ float red[2][NW];
  int turn = 0;
  constexpr int TPR = 64 * NW;
  const int wave = (int)threadIdx.x >> 6;
  const int t = NW == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * norm_rows(NW);
  const RowSrc src{a.x, nullptr};
  int64_t row = (int64_t)blockIdx.x * norm_rows(NW) + (NW == 1 ? wave : 0);
  if (row >= a.M) return;  // a whole workgroup, or (NW = 1, no barriers) a wave
  Raw8<WT> w[VPT], bias[kKeepBias ? VPT : 1];
  load_row<WT, VPT>(RowSrc{a.w, nullptr}, 0, a.n, t, TPR, w);
  finish_row<WT, VPT>(a.n, t, TPR, w);
  if constexpr (kKeepBias) {
    load_row<WT, VPT>(RowSrc{a.b, nullptr}, 0, a.n, t, TPR, bias);
    finish_row<WT, VPT>(a.n, t, TPR, bias);
  }
  Raw8<XT> next[VPT];
  load_row<XT, VPT>(src, row, a.n, t, TPR, next);
  for (; row < a.M; row += step) {
    Raw8<XT> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = next[i];
    finish_row<XT, VPT>(a.n, t, TPR, r);
    // unconditional (see load_piece8); after the last row this row again, from the cache
    load_row<XT, VPT>(src, row + step < a.M ? row + step : row, a.n, t, TPR, next);
    float mean = 0.0f;
    if constexpr (kLayer) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float v[8];
        raw_to_f32<XT>(r[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[j];
      }
      mean = (float)(row_sum64<NW>(s, red, turn, wave) * a.inv_n);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = 8 * (t + TPR * i);
      float v[8];
      raw_to_f32<XT>(r[i], v);
      float q = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float d = v[j];
        if constexpr (kLayer) d = col + j < a.n ? d - mean : 0.0f;
        q = __builtin_fmaf(d, d, q);
      }
      s += q;
    }
    const float rstd = inverse_root(row_sum64<NW>(s, red, turn, wave) * a.inv_n + (double)a.eps);
    if (t == 0) {
      a.rstd[row] = rstd;
      if constexpr (kLayer) a.mean[row] = mean;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = 8 * (t + TPR * i);
      float v[8], wv[8];
      raw_to_f32<XT>(r[i], v);
      raw_to_f32<WT>(w[i], wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (kLayer ? v[j] - mean : v[j]) * rstd;
      if (!kKeepBias && !a.b) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= wv[j];
      } else {
        float bv[8];
        if constexpr (kKeepBias) {
          raw_to_f32<WT>(bias[i], bv);
        } else {
          load_row<WT, 1>(RowSrc{a.b, nullptr}, 0, a.n, t + TPR * i, 0, bias);
          finish_row<WT, 1>(a.n, t + TPR * i, 0, bias);
          raw_to_f32<WT>(bias[0], bv);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf(v[j], wv[j], bv[j]);
      }
      store8<XT>(a.y, row, a.n, col, v);
      if constexpr (XT == kBf16) {
        if (a.codes) {
          // past the row's end w and b are zeros, but 0 times a non-finite
          // mean or rstd is not
          u32x4 y = round_bf16x8(v);
          if (col + 8 > a.n) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + j >= a.n) y[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
          }
          ckpt_store8(a.codes, a.scales, row, a.n, col, y);
        }
      }
    }
  }
}

template <bool kLayer, int XT, int WT>
static void norm_fwd_typed(const NormFwdArgs& a, hipStream_t stream) {
  norm_shape<false>(a.n, [&](auto nw, auto vpt) {
    constexpr int NW = decltype(nw)::value, VPT = decltype(vpt)::value;
    const int64_t wgs = (a.M + norm_rows(NW) - 1) / norm_rows(NW);
    const int64_t most = (int64_t)device_cus() * (NW == 1 ? 16 : NW == 4 ? 8 : 4);
    const dim3 grid((unsigned)(wgs < most ? wgs : most)), block(NW == 1 ? 256 : 64 * NW);
    // A layer norm's bias is kept where the registers are enough (8192 x 8192
    // bf16 50 us, 57 us loading it in each row; 16384 x 1500 bf16 29 and 36 us).
    constexpr bool kKeep = kLayer && VPT < 4;
    if (kKeep && a.b)
      hipLaunchKernelGGL((norm_fwd_kernel<kLayer, kKeep, XT, WT, NW, VPT>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((norm_fwd_kernel<kLayer, false, XT, WT, NW, VPT>), grid, block, 0, stream, a);
  });
}

void launch_norm_fwd(int layer, int x_type, int w_f32, int64_t M, int64_t n, float eps, const void* x, const void* w,
                     const void* b, void* y, float* mean, float* rstd, int8_t* codes, uint8_t* scales,
                     hipStream_t stream) {
  const NormFwdArgs a{(int)n, M, eps, 1.0 / (double)n, x, w, b, y, mean, rstd, codes, scales};
  if (x_type == kF32) layer ? norm_fwd_typed<true, kF32, kF32>(a, stream) : norm_fwd_typed<false, kF32, kF32>(a, stream);
  else if (w_f32) layer ? norm_fwd_typed<true, kBf16, kF32>(a, stream) : norm_fwd_typed<false, kBf16, kF32>(a, stream);
  else layer ? norm_fwd_typed<true, kBf16, kBf16>(a, stream) : norm_fwd_typed<false, kBf16, kBf16>(a, stream);
}

}  // namespace qlora
