// Tensor table and launchers of the optimizer step over many tensors (adamw.hip).
#pragma once

#include "qlora_common.h"

namespace qlora {

// state: 0 fp32 moments, 1 moments in 8 bits.  grad: 0 bf16, 1 fp32.
struct AdamWTensor {
  int64_t count;
  float* p;
  uint16_t* p16;  // may be null
  const void* g;
  void* m;
  void* v;
  float* md;
  float* vd;
  int64_t chunk;  // first chunk
  int32_t grad, state;
};

int64_t adamw_chunks(int64_t count);
size_t adamw_plan_bytes(int64_t chunks, int64_t tensors);
constexpr int kPlanPerLaunch = 40;  // table entries in one launch's arguments (3.2 KB)
// Entries first .. first + count - 1 of a plan, count at most kPlanPerLaunch.
void launch_adamw_plan(const AdamWTensor* ts, int64_t first, int count, int64_t tensors, int64_t chunks, void* plan,
                       hipStream_t stream);
void launch_adamw_step(void* plan, int64_t tensors, int64_t chunks, double lr, double beta1, double beta2, double eps,
                       double weight_decay, int64_t step, const float* clip, const uint64_t* seed,
                       hipStream_t stream);
void launch_grad_clip(void* plan, int64_t tensors, int64_t chunks, double max_norm, float* out, hipStream_t stream);
void launch_moment8_values(int is_signed, int64_t count, const uint8_t* codes, const float* steps, float* out,
                           hipStream_t stream);

}  // namespace qlora
