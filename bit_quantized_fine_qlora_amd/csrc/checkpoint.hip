// Activation checkpoints in 8 bits: a bf16 M x n tensor kept as 8-bit
// integers with a power-of-two scale for each 32 values of a row (the format
// is stated at ckpt_encode8), 33/32 bytes a value instead of 2.  "QLoRA:
// Efficient Fine-Tuning" leaves activations as what grows with the batch once
// weights, optimizer state and gradients have shrunk; the adapted linear
// layer saves one tensor of that size, its input, and reads it in one place
// of the backward pass (grad_A).
//
// Both kernels move 8 values a lane and are bound by HBM: packing reads 2
// bytes and writes 33/32 a value, restoring the reverse: 8192 x 8192 36-39 us
// each (203 MB, 5.2-5.6 TB/s; a plain copy moves 5.0-5.3).  More loads in flight a
// thread, non-temporal loads and fewer or more workgroups measured 0 to 10 %
// slower.
#include "rows.h"

namespace qlora {

// Thread = 8 values; 16 lanes = 128 columns = 4 scale bytes.  Pieces are
// counted over rows padded to 128 columns, so that the quad of lanes that
// shares a block never crosses a row.
__global__ __launch_bounds__(256) void checkpoint_pack_kernel(int64_t M, int n, const uint16_t* __restrict__ x,
                                                              int8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  const int per_row = (int)(ckpt_pitch(n) / 4) * 16;  // 8-value pieces of a padded row
  const int64_t total = M * per_row;
  const RowSrc src{x, nullptr};
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int col = (int)(i - row * per_row) * 8;
    Raw8<kBf16> r;
    r.w = u32x4{0u, 0u, 0u, 0u};
    if (col + 8 <= n)
      r = load_full8<kBf16>(src, row, n, col);
    else if (col < n)
      r = load_tail8<kBf16>(src, row, n, col, n - col);
    ckpt_store8(codes, scales, row, n, col, r.w);
  }
}

__global__ __launch_bounds__(256) void checkpoint_unpack_kernel(int64_t M, int n, const int8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales,
                                                                uint16_t* __restrict__ x) {
  const int per_row = (n + 7) / 8;
  const int64_t total = M * per_row;
  const RowSrc src{codes, scales};
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int col = (int)(i - row * per_row) * 8;
    Raw8<kCkpt8> r;
    if (col + 8 <= n)
      r = load_full8<kCkpt8>(src, row, n, col);
    else
      r = load_tail8<kCkpt8>(src, row, n, col, n - col);
    float v[8];
    raw_to_f32<kCkpt8>(r, v);
    store8<kBf16>(x, row, n, col, v);
  }
}

static unsigned stream_grid(int64_t pieces) {
  const int64_t want = (pieces + 255) / 256, most = (int64_t)device_cus() * 32;
  return (unsigned)(want < most ? want : most);
}

void launch_checkpoint_pack(int64_t M, int64_t n, const uint16_t* x, int8_t* codes, uint8_t* scales,
                            hipStream_t stream) {
  hipLaunchKernelGGL(checkpoint_pack_kernel, dim3(stream_grid(M * (ckpt_pitch(n) / 4) * 16)), dim3(256), 0, stream, M,
                     (int)n, x, codes, scales);
}

void launch_checkpoint_unpack(int64_t M, int64_t n, const int8_t* codes, const uint8_t* scales, uint16_t* x,
                              hipStream_t stream) {
  hipLaunchKernelGGL(checkpoint_unpack_kernel, dim3(stream_grid(M * ((n + 7) / 8))), dim3(256), 0, stream, M, (int)n,
                     codes, scales, x);
}

}  // namespace qlora
