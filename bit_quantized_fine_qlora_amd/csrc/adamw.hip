// The optimizer step over any number of tensors in one launch: Adam with
// decoupled weight decay, moments in 8 or 32 bits, gradients in bf16 or fp32,
// and the gradients' norm with the factor that holds it to a maximum.
// "QLoRA & 4-bit Fine-Tuning", Innovation 3 (optimizer state is what is left
// to shrink once the weight has 4 bits) and "QLoRA: Efficient Fine-Tuning",
// memory-layout figure (Adam moments for the adapters only).
//
// Per element, with f the clip factor (1 without):
//   g <- f g;  m <- b1 m + (1 - b1) g;  v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v / (1 - b2^t)) + eps)
// The weight takes lr wd p and its update in one subtraction: 1 - lr wd as a
// factor in fp32 would be a multiple of 2^-24, 1.3 % off for a decay of 2e-6
// and no decay at all below 3e-8, the same in every step.
//
// A moment in 8 bits.  Blocks of 128 consecutive elements share one fp32 step
// d; a code stands for a square, so that its values are dense near zero and
// 2 / k apart relative to themselves:
//   m: sign (bit 7) and k in 0 .. 127, value +-k^2 d, d = fp32(max |m| / 127^2)
//   v: its root is kept, k in 0 .. 255, root = k^2 d, value root^2,
//      d = fp32(max root / 255^2); a v that is not 0 takes no k below 1, so
//      that no element divides its first moment by eps alone
// d below 2^-126 counts as 0 (the whole block is 0).  Each value takes the
// nearest of them, the lower of two as near, or (kDrawn, v only) one of the two
// about it, drawn so that the mean is the value.  Nearest codes stop v's running
// average: a step moves it by 1 - b2 of itself, 0.1 %, and neighbours are 4 / k,
// 1.6 % at least, apart, so a root whose gradients fall to a fifth beside others
// that do not stays where it was (3.9 times too large 4000 steps later; drawn
// codes 0.99 times).  m moves by 10 % a step and takes the nearest.  The new moments and that choice
// are formed in 64 bits: what a code is then depends on the operands alone
// and not on an order of fp32 operations, and fp64 multiplies and adds run at
// the fp32 rate here.  The weight's update reads the moments before their
// rounding.
//
// All of it is bound by memory: 16 bytes an element with 8-bit moments (p
// read and written, the bf16 gradient, the bf16 copy, codes read and
// written) and 1/8 byte of steps, 28 with 32-bit ones.  Measured: 41.9 million
// elements in 448 tensors, 8 bits, 119-143 us by card (4.7-5.7 TB/s); 84.9
// million 236-264 us (5.2-5.8 TB/s), with drawn codes as long to 16 % longer
// (alone 151 us against 130, among other steps 156 and 156); 6.1 million in 97
// tensors of odd sizes, 32 bits and fp32 gradients, 30 us (183 MB, 6.1 TB/s,
// part of it out of the memory-side cache).
//
// The plan.  A step's tensors stay the same over a training run, so their
// table is written to device memory once: header, room for the norm's partial
// sums, one entry a tensor, and for each chunk of 2048 elements the tensor it
// belongs to.  A workgroup takes one chunk, so a step is one launch whatever
// the number of tensors (a table in the kernel's arguments holds 64).
#include <cmath>

#include "adamw.h"
#include "rows.h"

namespace qlora {

constexpr int kChunk = 2048;        // elements of a workgroup: 8 a thread
constexpr int kMomentBlock = 128;   // 16 lanes
constexpr int kNormGroups = 2048;   // workgroups of the norm's first pass at most

struct PlanView {
  int64_t* header;      // chunks, tensors
  double* partial;      // kNormGroups
  AdamWTensor* tensors;
  uint32_t* owner;      // tensor of each chunk
};

static __host__ __device__ PlanView plan_view(void* plan, int64_t tensors) {
  uint8_t* b = static_cast<uint8_t*>(plan);
  PlanView v;
  v.header = reinterpret_cast<int64_t*>(b);
  v.partial = reinterpret_cast<double*>(b + 256);
  v.tensors = reinterpret_cast<AdamWTensor*>(b + 256 + kNormGroups * sizeof(double));
  v.owner = reinterpret_cast<uint32_t*>(v.tensors + tensors);
  return v;
}

int64_t adamw_chunks(int64_t count) { return (count + kChunk - 1) / kChunk; }
size_t adamw_plan_bytes(int64_t chunks, int64_t tensors) {
  return 256 + kNormGroups * sizeof(double) + (size_t)tensors * sizeof(AdamWTensor) + (size_t)chunks * sizeof(uint32_t);
}

struct PlanArgs {
  AdamWTensor t[kPlanPerLaunch];
  int first, count;          // tensors first .. first + count - 1
  int64_t tensors, chunks;   // of the whole plan
};

// One workgroup a tensor: its entry and the owners of its chunks.
__global__ __launch_bounds__(256) void adamw_plan_kernel(PlanArgs a, void* plan) {
  const PlanView v = plan_view(plan, a.tensors);
  const AdamWTensor& t = a.t[blockIdx.x];
  const uint32_t id = (uint32_t)(a.first + (int)blockIdx.x);
  if (threadIdx.x == 0) {
    v.tensors[id] = t;
    if (id == 0) {
      v.header[0] = a.chunks;
      v.header[1] = a.tensors;
    }
  }
  const int64_t n = (t.count + kChunk - 1) / kChunk;
  for (int64_t c = threadIdx.x; c < n; c += 256) v.owner[t.chunk + c] = id;
}

void launch_adamw_plan(const AdamWTensor* ts, int64_t first, int count, int64_t tensors, int64_t chunks, void* plan,
                       hipStream_t stream) {
  PlanArgs a{};
  a.first = (int)first;
  a.count = count;
  a.tensors = tensors;
  a.chunks = chunks;
  for (int k = 0; k < count; ++k) a.t[k] = ts[k];
  hipLaunchKernelGGL(adamw_plan_kernel, dim3((unsigned)count), dim3(256), 0, stream, a, plan);
}

// 8 consecutive gradient values from element e on, of which the tensor has
// `left` (the rest are 0).
__device__ __forceinline__ void load_grad8(const AdamWTensor& t, int64_t e, int64_t left, float (&g)[8]) {
  if (t.grad == kBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(t.g) + e;
    if (left >= 8) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[2 * j] = bf16_lo_to_f32(w[j]);
        g[2 * j + 1] = bf16_hi_to_f32(w[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = j < left ? __uint_as_float((uint32_t)p[j] << 16) : 0.0f;
    }
  } else {
    const float* p = static_cast<const float*>(t.g) + e;
    if (left >= 8) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[j] = a[j];
        g[j + 4] = b[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = j < left ? p[j] : 0.0f;
    }
  }
}

__device__ __forceinline__ void load_f32x8(const float* p, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[j + 4] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.0f;
  }
}

__device__ __forceinline__ void store_f32x8(float* p, int64_t left, const float (&v)[8]) {
  if (left >= 8) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = v[j];
  }
}

__device__ __forceinline__ u32x2 load_codes8(const uint8_t* p, int64_t left) {
  if (left >= 8) return *reinterpret_cast<const u32x2*>(p);
  u32x2 w = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return w;
}

__device__ __forceinline__ void store_codes8(uint8_t* p, int64_t left, const u32x2& w) {
  if (left >= 8) {
    *reinterpret_cast<u32x2*>(p) = w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
}

// Maximum over the 16 lanes of a DPP row (one block of a moment); every lane
// gets it.
__device__ __forceinline__ double row_max(double v) {
  auto step = [&](auto ctrl) {
    const u32x2 b = __builtin_bit_cast(u32x2, v);
    u32x2 o;
    o[0] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[0], decltype(ctrl)::value, 0xF, 0xF, true);
    o[1] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[1], decltype(ctrl)::value, 0xF, 0xF, true);
    v = __builtin_fmax(v, __builtin_bit_cast(double, o));
  };
  using std::integral_constant;
  step(integral_constant<int, 0x121>{});  // row_ror:1
  step(integral_constant<int, 0x122>{});  // row_ror:2
  step(integral_constant<int, 0x124>{});  // row_ror:4
  step(integral_constant<int, 0x128>{});  // row_ror:8
  return v;
}

// The k whose square is nearest to x = value / d, given an fp32 approximation
// of x: floor(sqrt) is k or, next to a square, one off either way, and the
// exact comparison with k^2 + k + 1/2 (16 bits and a half) settles which.
__device__ __forceinline__ float root_floor(float x) { return __builtin_floorf(__builtin_amdgcn_sqrtf(x)); }

// The value of code k of a second moment with step d.
__device__ __forceinline__ double root_code(float k, double d) {
  const double root = (double)(k * k) * d;
  return root * root;
}

struct AdamWConst {
  double b1, c1, b2, c2;  // beta, 1 - beta
  float f1, g1, f2, g2;   // the same in fp32
  float decay;            // lr wd
  float step_size;        // lr / (1 - b1^t)
  float inv_bc2;          // 1 / (1 - b2^t)
  float inv_root_bc2;     // its root
  float eps;
};

// kDrawn: element 2048 c + i of the plan (chunk c) takes word i % 4 of
// Philox4x32-10 at the 64-bit counter 2^33 step + 512 c + i / 4 under the seed:
// 2 calls for a thread's 8 elements.
template <bool kDrawn>
__global__ __launch_bounds__(256) void adamw_step_kernel(void* plan, int64_t tensors, AdamWConst c,
                                                         const float* __restrict__ clip, uint64_t seed,
                                                         uint64_t counter) {
  const PlanView pv = plan_view(plan, tensors);
  // Read first and tested last, so that its latency is not added to the others'.
  // Not finite: gradients without a finite norm, no step.
  const float factor = clip ? clip[1] : 1.0f;
  const AdamWTensor T = pv.tensors[pv.owner[blockIdx.x]];
  const int64_t e = ((int64_t)blockIdx.x - T.chunk) * kChunk + 8 * (int)threadIdx.x;
  const int64_t left = T.count - e;  // lanes past the end stay for the blocks' maxima
  float g[8], p[8];
  if (T.state == 0) {
    if (left <= 0) return;
    float m[8], v[8];
    load_grad8(T, e, left, g);
    load_f32x8(T.p + e, left, p);
    load_f32x8(static_cast<const float*>(T.m) + e, left, m);
    load_f32x8(static_cast<const float*>(T.v) + e, left, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = g[j] * factor;
      m[j] = __builtin_fmaf(c.f1, m[j], c.g1 * x);
      v[j] = __builtin_fmaf(c.f2, v[j], c.g2 * x * x);
      const float u = c.step_size * (m[j] / (__builtin_sqrtf(v[j] * c.inv_bc2) + c.eps));
      p[j] -= __builtin_fmaf(c.decay, p[j], u);
    }
    if (!(__builtin_fabsf(factor) < __builtin_inff())) return;
    store_f32x8(static_cast<float*>(T.m) + e, left, m);
    store_f32x8(static_cast<float*>(T.v) + e, left, v);
  } else {
    const int64_t have = left > 0 ? left : 0;
    const int64_t at = left > 0 ? e : 0;
    load_grad8(T, at, have, g);
    load_f32x8(T.p + at, have, p);
    const u32x2 mw = load_codes8(static_cast<const uint8_t*>(T.m) + at, have);
    const u32x2 vw = load_codes8(static_cast<const uint8_t*>(T.v) + at, have);
    const double md = (double)T.md[at / kMomentBlock], vd = (double)T.vd[at / kMomentBlock];
    double m[8], v[8], mtop = 0.0, vtop = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double x = (double)g[j] * (double)factor;
      const uint32_t mc = mw[j >> 2] >> (8 * (j & 3)), vc = vw[j >> 2] >> (8 * (j & 3));
      const float mk = (float)(mc & 127u), vk = (float)(vc & 255u);
      const double old = (double)((mc & 128u) ? -mk * mk : mk * mk) * md;
      const double root = (double)(vk * vk) * vd;
      m[j] = c.b1 * old + c.c1 * x;
      v[j] = c.b2 * (root * root) + c.c2 * (x * x);
      mtop = __builtin_fmax(mtop, __builtin_fabs(m[j]));
      vtop = __builtin_fmax(vtop, v[j]);
    }
    mtop = row_max(mtop);
    vtop = row_max(vtop);
    constexpr float kTiny = 1.17549435e-38f;  // 2^-126
    float dm = (float)(mtop / (127.0 * 127.0)), dv = (float)(__builtin_sqrt(vtop) / (255.0 * 255.0));
    dm = dm < kTiny ? 0.0f : dm;
    dv = dv < kTiny ? 0.0f : dv;
    const float im = dm > 0.0f ? 1.0f / dm : 0.0f;
    // Roots are taken in fp32 as parts of the block's largest, of squares scaled
    // to 2^126 at most, so that neither a small block nor a small element beside
    // a large one leaves fp32's range (down to 2^-126 of the largest); where the
    // largest is past 2^125, whose reciprocals are not normal numbers, the
    // quotient's parts are scaled too.  (The largest is 255^2 steps.)
    const float big = (float)__builtin_sqrt(vtop);
    const double iv = vtop > 0.0 ? 0x1p126 / vtop : 0.0;
    const float sc = big * c.inv_root_bc2 > 0x1p125f ? 0.25f : 1.0f;
    const float to_denom = big * sc * c.inv_root_bc2, eps = __builtin_fmaxf(c.eps * sc, 0x1p-126f);
    const float step_size = c.step_size * sc;
    u32x2 mo = {0u, 0u}, vo = {0u, 0u};
    u32x4 draw[2] = {};
    if constexpr (kDrawn) {
      const uint64_t at = counter + (uint64_t)blockIdx.x * (kChunk / 4) + 2 * threadIdx.x;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        draw[i] = philox4x32_10((uint32_t)(at + i), (uint32_t)((at + i) >> 32), (uint32_t)seed, (uint32_t)(seed >> 32));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double am = __builtin_fabs(m[j]);
      const float mf = (float)am;
      float k = root_floor(mf * im);
      k += am > (double)(k * k + k + 0.5f) * (double)dm ? 1.0f : 0.0f;
      uint32_t mc = (uint32_t)__builtin_fminf(k, 127.0f);
      mc = dm > 0.0f ? mc : 0u;
      mc |= (m[j] < 0.0 && mc) ? 128u : 0u;
      const float root = __builtin_amdgcn_sqrtf((float)(v[j] * iv)) * 0x1p-63f;
      if constexpr (kDrawn) {
        k = root_floor(root * (255.0f * 255.0f));
        // Next to a code (1e-4 of the way to the next at most, at k = 255) k may be
        // one off either way: v then takes that code whatever the word, which moves
        // the mean by less than 1e-8 of the way.  (With k put right 160-166 us
        // instead of 152 for 41.9 million elements.)
        const double lo = root_code(k, (double)dv), hi = root_code(k + 1.0f, (double)dv);
        const double part = ((double)draw[j >> 2][j & 3] + 0.5) * 0x1p-32;
        k += v[j] - lo > (hi - lo) * part ? 1.0f : 0.0f;
      } else {
        k = root_floor(root * (255.0f * 255.0f));
        const double border = (double)(k * k + k + 0.5f) * (double)dv;
        k += v[j] > border * border ? 1.0f : 0.0f;
      }
      uint32_t vc = (uint32_t)__builtin_fminf(k, 255.0f);
      vc = vc == 0u && v[j] > 0.0 ? 1u : vc;
      vc = dv > 0.0f ? vc : 0u;
      mo[j >> 2] |= mc << (8 * (j & 3));
      vo[j >> 2] |= vc << (8 * (j & 3));
      const float denom = __builtin_fmaf(root, to_denom, eps);
      const float u = step_size * ((m[j] < 0.0 ? -mf : mf) * __builtin_amdgcn_rcpf(denom));
      p[j] -= __builtin_fmaf(c.decay, p[j], u);
    }
    if (left <= 0 || !(__builtin_fabsf(factor) < __builtin_inff())) return;
    store_codes8(static_cast<uint8_t*>(T.m) + e, left, mo);
    store_codes8(static_cast<uint8_t*>(T.v) + e, left, vo);
    if ((threadIdx.x & 15) == 0) {
      T.md[e / kMomentBlock] = dm;
      T.vd[e / kMomentBlock] = dv;
    }
  }
  store_f32x8(T.p + e, left, p);
  if (T.p16) {
    const u32x4 w = round_bf16x8(p);
    if (left >= 8) {
      *reinterpret_cast<u32x4*>(T.p16 + e) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) T.p16[e + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

void launch_adamw_step(void* plan, int64_t tensors, int64_t chunks, double lr, double beta1, double beta2, double eps,
                       double weight_decay, int64_t step, const float* clip, const uint64_t* seed,
                       hipStream_t stream) {
  AdamWConst c;
  const double bc1 = 1.0 - std::pow(beta1, (double)step), bc2 = 1.0 - std::pow(beta2, (double)step);
  c.b1 = beta1;
  c.c1 = 1.0 - beta1;
  c.b2 = beta2;
  c.c2 = 1.0 - beta2;
  c.f1 = (float)c.b1;
  c.g1 = (float)c.c1;
  c.f2 = (float)c.b2;
  c.g2 = (float)c.c2;
  c.decay = (float)(lr * weight_decay);
  c.step_size = (float)(lr / bc1);
  c.inv_bc2 = (float)(1.0 / bc2);
  c.inv_root_bc2 = (float)std::sqrt(1.0 / bc2);
  c.eps = (float)eps;
  const dim3 grid((unsigned)chunks), block(256);
  if (seed)
    hipLaunchKernelGGL(adamw_step_kernel<true>, grid, block, 0, stream, plan, tensors, c, clip, *seed,
                       (uint64_t)step << 33);
  else
    hipLaunchKernelGGL(adamw_step_kernel<false>, grid, block, 0, stream, plan, tensors, c, clip, 0ull, 0ull);
}

// ---------------------------------------------------------------------------
// The gradients' norm: squares and sums in 64 bits, each workgroup's chunks
// and then the workgroups' sums in a fixed order.  Bound by the read: 84 MB of
// bf16 gradients in 448 tensors 21-31 us by card (2.7-4.0 TB/s), 2-5 us for the
// second launch.  A chunk's owner, its tensor's entry and its gradient are read
// one after the other.  The gradient's address comes out of the table, so its
// loads are flat ones, which count with the scalar reads too: a look into the
// table waits for every load in flight, and four chunks at once or the table
// read ahead were no faster.
// ---------------------------------------------------------------------------

// Sum over the workgroup's 256 threads, in thread 0.
__device__ __forceinline__ double group_sum(double v) {
  __shared__ double part[4];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(256) void grad_norm_kernel(void* plan, int64_t tensors) {
  const PlanView pv = plan_view(plan, tensors);
  const int64_t chunks = pv.header[0];
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const AdamWTensor& T = pv.tensors[pv.owner[c]];
    const int64_t e = (c - T.chunk) * kChunk + 8 * (int)threadIdx.x;
    if (e >= T.count) continue;
    float g[8];
    load_grad8(T, e, T.count - e, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)g[j] * (double)g[j];
  }
  s = group_sum(s);
  if (threadIdx.x == 0) pv.partial[blockIdx.x] = s;
}

// out[0] = norm, out[1] = min(1, max_norm / (norm + 1e-6)), NaN where the norm
// is not finite.
__global__ __launch_bounds__(256) void grad_clip_kernel(void* plan, int64_t tensors, int groups, double max_norm,
                                                        float* __restrict__ out) {
  const PlanView pv = plan_view(plan, tensors);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kNormGroups / 256; ++i) {
    const int k = 256 * i + (int)threadIdx.x;
    s += k < groups ? pv.partial[k] : 0.0;
  }
  s = group_sum(s);
  if (threadIdx.x == 0) {
    const double norm = __builtin_sqrt(s);
    const double f = max_norm / (norm + 1e-6);
    const bool finite = norm < __builtin_inf();
    out[0] = (float)norm;
    out[1] = finite ? (float)(f < 1.0 ? f : 1.0) : __builtin_nanf("");
  }
}

void launch_grad_clip(void* plan, int64_t tensors, int64_t chunks, double max_norm, float* out, hipStream_t stream) {
  const int groups = (int)(chunks < kNormGroups ? chunks : kNormGroups);
  hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)groups), dim3(256), 0, stream, plan, tensors);
  hipLaunchKernelGGL(grad_clip_kernel, dim3(1), dim3(256), 0, stream, plan, tensors, groups, max_norm, out);
}

// The fp32 values that a moment's codes stand for.  41.9 million: 36-44 us
// (211 MB, 4.8-5.8 TB/s).
template <bool kSigned>
__global__ __launch_bounds__(256) void moment8_values_kernel(int64_t count, const uint8_t* __restrict__ codes,
                                                             const float* __restrict__ steps,
                                                             float* __restrict__ out) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (e >= count) return;
  const u32x2 w = load_codes8(codes + e, count - e);
  const double d = (double)steps[e / kMomentBlock];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t c = (w[j >> 2] >> (8 * (j & 3))) & 255u;
    if (kSigned) {
      const float k = (float)(c & 127u);
      v[j] = (float)((double)((c & 128u) ? -k * k : k * k) * d);
    } else {
      const double root = (double)((float)c * (float)c) * d;
      v[j] = (float)(root * root);
    }
  }
  store_f32x8(out + e, count - e, v);
}

void launch_moment8_values(int is_signed, int64_t count, const uint8_t* codes, const float* steps, float* out,
                           hipStream_t stream) {
  const unsigned grid = (unsigned)((count + kChunk - 1) / kChunk);
  if (is_signed)
    hipLaunchKernelGGL(moment8_values_kernel<true>, dim3(grid), dim3(256), 0, stream, count, codes, steps, out);
  else
    hipLaunchKernelGGL(moment8_values_kernel<false>, dim3(grid), dim3(256), 0, stream, count, codes, steps, out);
}

}  // namespace qlora
