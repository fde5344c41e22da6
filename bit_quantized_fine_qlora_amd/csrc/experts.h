// Launchers of the experts' products (experts.hip).
#pragma once

#include "qlora_common.h"

namespace qlora {

// A factor (u or v) to be summed from `splits` M x R partials: fp32 out and
// bf16 planes, either may be null.
struct FactorJob {
  const float* part;
  int splits;
  float* out;
  uint16_t* planes;
};

bool experts_gemm_fits(int64_t M, int64_t E, int64_t N);
size_t experts_gemm_ws_bytes(int64_t M, int64_t E, int64_t N, int64_t K);
void launch_experts_gemm(bool bwd, const int32_t* offsets, int64_t E, const uint16_t* act, const uint8_t* codes,
                         const uint8_t* absmax8, const float* c2, const uint16_t* lora_a, const float* lora_b,
                         uint16_t* out, int64_t M, int64_t K, int64_t n, int64_t m, int r, float s, void* ws,
                         const Nf4Table& tab, hipStream_t stream);
size_t experts_stream_ws_bytes(int64_t M, int64_t E, int64_t N, int64_t K);
bool experts_stream_takes(int64_t M, int64_t E, int64_t N, int64_t K);
void launch_experts_stream(const int32_t* offsets, int64_t E, const uint16_t* x, const uint8_t* codes,
                           const uint8_t* absmax8, const float* c2, const uint16_t* B, const float* u, int usplits,
                           float* u_out, uint16_t* h, int64_t M, int64_t n, int64_t m, int r, float s, void* ws,
                           const Nf4Table& tab, hipStream_t stream);
int experts_down_splits(int64_t M, int64_t E, int64_t K, int R);
void launch_experts_down(const uint16_t* X, const int32_t* offsets, int64_t M, int64_t E, int64_t K, const uint16_t* Y,
                         bool yt, int64_t yrows, int R, float* part, int splits, hipStream_t stream);
void launch_experts_prepare(const uint16_t* g, uint16_t* gout, const uint16_t* B, uint16_t* bout, int64_t M, int64_t E,
                            int64_t m, int R, int64_t ld, hipStream_t stream);
size_t experts_planes_bytes(int64_t M, int R);
void launch_experts_factor(const FactorJob* jobs, int count, const int32_t* offsets, int64_t M, int64_t E, int R,
                           hipStream_t stream);
bool experts_token_fits(int64_t M, int64_t E, int64_t J);
size_t experts_token_ws_bytes(int64_t M, int64_t J, int R);
void launch_experts_token(const uint16_t* x, const uint16_t* vplanes, uint16_t* grad_A, float* part_a,
                          const uint16_t* g, int64_t g_ld, const uint16_t* uplanes, uint16_t* grad_B, float* part_b,
                          const int32_t* offsets, int64_t M, int64_t E, int64_t n, int64_t m, int R, float s,
                          hipStream_t stream);

}  // namespace qlora
