// Preference loss (paired log ratios) of packed sequences, from their logits,
// and its gradient.
//   lse_t  = log sum_v exp(x_tv),  lp_t = x_t,label(t) - lse_t   (scored tokens)
//   lp_s   = sum of lp_t over sequence s
//   z_i    = beta ((lp_2i - ref_2i) - (lp_2i+1 - ref_2i+1))      (pair i)
//   loss   = mean_i [-(1 - e) log sigma(z_i) - e log sigma(-z_i)]
//   dloss/dlp_2i = c_i = beta / P (e sigma(z_i) - (1 - e) sigma(-z_i)) = -dloss/dlp_2i+1
//   grad_tv = c_t (1[v = label(t)] - exp(x_tv - lse_t))
// The gradient of a token needs its pair's z, a sum over all tokens of both
// sequences, so the logits are read twice: once for the row sums, in one pass
// with a running maximum, and once, element by element, for the gradient.
// Rows whose label is negative are neither read nor scored; their gradient is
// written as zeros.  With thousands of rows both passes are bound by HBM: 8
// pairs, 6144 x 131072 bf16 logits, 60 % of the tokens scored: rows 154-172 us
// (966 MB, 5.6-6.3 TB/s), sequences 8 us, gradient 431-453 us (2.58 GB, 5.7-6.0
// TB/s; a plain copy moves 5.0-5.3).  The logits' loads carry the non-temporal
// hint: 188 us and 486 us without, on the card of the slower figures.  With
// fewer the row pass is not, a workgroup to a row and no load in flight while
// it adds: 5 pairs, 1501 x 50021 fp32, 904 rows scored, 48-60 us (181 MB, 3.0-3.8
// TB/s), the same with rows of 50048; as many bytes in bf16, 3002 x 50021, 52 us;
// 6001 x 50021 fp32, 3530 scored, 173 us (706 MB, 4.1 TB/s).  The gradient of the
// first takes 74-81 us (481 MB, 5.9-6.5 TB/s).
#include <algorithm>

#include "rows.h"

namespace qlora {

constexpr float kLog2e = 1.4426950408889634f;

// Running maximum m and sum s of exp(x - m).  m = -inf means nothing finite
// yet: differences are then taken from 0, so that exp(-inf) adds nothing.
struct MaxSum {
  float m, s;
};

__device__ __forceinline__ float exp_from(float x, float m) { return __builtin_amdgcn_exp2f((x - m) * kLog2e); }

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  MaxSum o;
  o.m = a.m > b.m ? a.m : b.m;
  const float base = o.m == -INFINITY ? 0.0f : o.m;
  o.s = a.s * exp_from(a.m, base) + b.s * exp_from(b.m, base);
  return o;
}

template <int N>
__device__ __forceinline__ void add_values(MaxSum& a, const float (&v)[N]) {
  float m = a.m;
#pragma unroll
  for (int j = 0; j < N; ++j) m = __builtin_fmaxf(m, v[j]);
  const float base = m == -INFINITY ? 0.0f : m;
  float s = a.s * exp_from(a.m, base);
#pragma unroll
  for (int j = 0; j < N; ++j) s += exp_from(v[j], base);
  a.m = m;
  a.s = s;
}

struct PrefRowArgs {
  const void* logits;
  int64_t T;
  int V;
  const int64_t* labels;
  int splits;      // workgroups to a row
  int chunk;       // vocabulary entries of each, a multiple of 2048
  MaxSum* part;    // [T][splits], where splits > 1
  float* lse;      // [T]
  float* lp;       // [T]
  float* coef;     // [T], cleared here; may be null
  uint32_t* ticket;  // cleared here
};

// The token counts: its label is not negative.
__device__ __forceinline__ bool scored(int64_t label) { return label >= 0; }

template <int XT>
__device__ __forceinline__ float logit_at(const void* logits, int64_t t, int V, int64_t v) {
  if constexpr (XT == kBf16)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[t * V + v] << 16);
  else
    return static_cast<const float*>(logits)[t * V + v];
}

// lse and lp of a row from its maximum and sum.  A label past the vocabulary
// gives NaN and reads nothing.
template <int XT>
__device__ __forceinline__ float finish_row(const PrefRowArgs& a, int64_t t, int64_t label, MaxSum r) {
  const float lse = r.m + __builtin_logf(r.s);
  a.lse[t] = lse;
  return label < a.V ? logit_at<XT>(a.logits, t, a.V, label) - lse : NAN;
}

// Workgroup = one chunk of one row.
template <int XT>
__global__ __launch_bounds__(256) void pref_rows_kernel(PrefRowArgs a) {
  constexpr int U = 4;             // pieces of 8 values in flight per thread
  constexpr int kPiece = 256 * 8;  // values of the workgroup's pieces
  __shared__ MaxSum red[4];
  const int tid = (int)threadIdx.x;
  if (blockIdx.x == 0 && tid == 0 && a.ticket) *a.ticket = 0u;
  const RowSrc src{a.logits, nullptr};
  const int64_t items = a.T * a.splits;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t t = item / a.splits;
    const int sp = (int)(item - t * a.splits);
    const int64_t label = a.labels[t];
    if (sp == 0 && tid == 0) {
      if (a.coef) a.coef[t] = 0.0f;
      if (a.splits > 1 || !scored(label)) {  // a row of chunks is finished with its sequence
        a.lse[t] = 0.0f;
        a.lp[t] = 0.0f;
      }
    }
    if (!scored(label)) continue;
    const int v0 = sp * a.chunk;
    const int v1 = v0 + a.chunk < a.V ? v0 + a.chunk : a.V;
    MaxSum r{-INFINITY, 0.0f};
    const int full = v0 + (v1 - v0) / 8 * 8;  // whole pieces end here
    // batches of U pieces a thread; in the last one the pieces past the end
    // read the chunk's first piece and count as -inf
    for (int b0 = v0; b0 < full; b0 += kPiece * U) {
      Raw8<XT> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = b0 + 8 * tid + kPiece * u;
        raw[u] = load_full8<XT, XT == kBf16>(src, t, a.V, b < full ? b : v0);
      }
      float v[8 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw_to_f32<XT>(raw[u], *reinterpret_cast<float(*)[8]>(v + 8 * u));
      if (b0 + kPiece * U > full) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[8 * u + j] = b0 + 8 * tid + kPiece * u < full ? v[8 * u + j] : -INFINITY;
      }
      add_values(r, v);
    }
    if (full + tid < v1) {
      const float v[1] = {logit_at<XT>(a.logits, t, a.V, full + tid)};
      add_values(r, v);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) r = join(r, MaxSum{__shfl_xor(r.m, d, 64), __shfl_xor(r.s, d, 64)});
    __syncthreads();  // the previous item's red has been read
    if ((tid & 63) == 0) red[tid >> 6] = r;
    __syncthreads();
    if (tid == 0) {
      r = join(join(red[0], red[1]), join(red[2], red[3]));
      if (a.splits == 1)
        a.lp[t] = finish_row<XT>(a, t, label, r);
      else
        a.part[item] = r;
    }
  }
}

// ---------------------------------------------------------------------------
// sequences and pairs
// ---------------------------------------------------------------------------
struct PrefSeqArgs {
  int64_t T;
  int V;
  int64_t count;           // sequences, or pairs
  const int32_t* offsets;  // [sequences + 1]
  const int64_t* labels;
  const void* logits;
  int splits, group;
  const MaxSum* part;
  float* lse;
  float* lp;               // [T], from the row kernel where rows are whole
  float* logps;            // [sequences]
  // pairs only
  const float* ref;        // [sequences], or null (zeros)
  float beta, smoothing, inv_pairs;
  float* coef;             // [T]
  float* pair_loss;        // [pairs]
  float* loss;             // [1]
  uint32_t* ticket;
};

// Workgroup = one sequence (kPairs false) or one pair of sequences 2i (the
// preferred one) and 2i + 1: joins the row chunks, adds up the tokens'
// log-probabilities, and for a pair forms its loss term and the coefficient
// of each of its tokens.  Where rows are chunked, `group` lanes (a power of
// two that covers the chunks, at most a wave) join a token's chunks, so that
// few tokens of many chunks still wait for memory once.  Sums over tokens are
// in 64 bits: a margin is a small difference of sums that grow with the
// sequences' lengths.  The last workgroup to finish adds the pairs' terms in
// order.
constexpr int kSeqWaves = 16;
template <int XT, bool kPairs>
__global__ __launch_bounds__(64 * kSeqWaves) void pref_seq_kernel(PrefSeqArgs a) {
  __shared__ double red[2][kSeqWaves];
  __shared__ int last;
  const int tid = (int)threadIdx.x, wave = tid >> 6;
  constexpr int S = kPairs ? 2 : 1, kThreads = 64 * kSeqWaves;
  const int sub = tid & (a.group - 1), per_pass = kThreads / a.group;
  PrefRowArgs ra{};
  ra.logits = a.logits;
  ra.V = a.V;
  ra.lse = a.lse;
  ra.lp = a.lp;
  auto block_sum = [&](double v, double* slot) {
    v = wave_sum(v);
    if ((tid & 63) == 0) slot[wave] = v;
    __syncthreads();
    double o = slot[0];
#pragma unroll
    for (int w = 1; w < kSeqWaves; ++w) o += slot[w];
    return o;
  };
  float only = 0.0f;  // the term of the only pair
  for (int64_t i = blockIdx.x; i < a.count; i += gridDim.x) {
    double lp[S];
    int64_t lo[S], hi[S];
    const float rc = kPairs && a.ref ? a.ref[2 * i] : 0.0f, rr = kPairs && a.ref ? a.ref[2 * i + 1] : 0.0f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      // offsets come from the device: held within the tokens there are
      const int64_t o0 = a.offsets[S * i + k], o1 = a.offsets[S * i + k + 1];
      lo[k] = o0 < 0 ? 0 : o0 < a.T ? o0 : a.T;
      hi[k] = o1 < lo[k] ? lo[k] : o1 < a.T ? o1 : a.T;
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      double s = 0.0;
      if (a.splits == 1) {
        for (int64_t t = lo[k] + tid; t < hi[k]; t += kThreads) s += (double)a.lp[t];
      } else {
        for (int64_t t0 = lo[k]; t0 < hi[k]; t0 += per_pass) {
          const int64_t t = t0 + tid / a.group;
          const bool in = t < hi[k];
          MaxSum r{-INFINITY, 0.0f};
          const int64_t label = in ? a.labels[t] : -1;
          if (scored(label))
            for (int c = sub; c < a.splits; c += a.group) r = join(r, a.part[t * a.splits + c]);
          for (int d = a.group >> 1; d; d >>= 1) r = join(r, MaxSum{__shfl_xor(r.m, d, 64), __shfl_xor(r.s, d, 64)});
          if (sub == 0 && scored(label)) s += (double)finish_row<XT>(ra, t, label, r);
        }
      }
      lp[k] = block_sum(s, red[k]);
      if (tid == 0) a.logps[S * i + k] = (float)lp[k];
    }
    if constexpr (kPairs) {
      // 64 bits up to z, whose terms may be large and their difference small;
      // its logistic function in 32
      const float z = (float)((double)a.beta * ((lp[0] - rc) - (lp[1] - rr)));
      const float e = a.smoothing;
      const float t = expf(-__builtin_fabsf(z)), near = 1.0f / (1.0f + t), far = t / (1.0f + t), l = log1pf(t);
      const float up = z >= 0.0f ? near : far, down = z >= 0.0f ? far : near;  // sigma(z), sigma(-z)
      const float su = l + __builtin_fmaxf(-z, 0.0f), sd = l + __builtin_fmaxf(z, 0.0f);  // their -log
      const float c = a.beta * a.inv_pairs * (e * up - (1.0f - e) * down);
      // an infinite margin makes one of the logarithms infinite: where its factor is 0 it does not count
      only = (e == 1.0f ? 0.0f : (1.0f - e) * su) + (e == 0.0f ? 0.0f : e * sd);
      if (tid == 0) a.pair_loss[i] = only;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        for (int64_t t = lo[k] + tid; t < hi[k]; t += kThreads)
          if (scored(a.labels[t])) a.coef[t] = k ? -c : c;
    }
    __syncthreads();  // red and the rows' log-probabilities have been read
  }
  if constexpr (kPairs) {
    if (a.count == 1) {
      if (tid == 0) *a.loss = only;
      return;
    }
    if (tid == 0) {
      __threadfence();  // this workgroup's terms before its count
      last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
      __threadfence();
    }
    __syncthreads();
    if (last) {
      double s = 0.0;
      for (int64_t i = tid; i < a.count; i += kThreads)
        s += (double)__hip_atomic_load(a.pair_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s = block_sum(s, red[0]);
      if (tid == 0) *a.loss = (float)(s * (double)a.inv_pairs);
    }
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
struct PrefGradArgs {
  const void* logits;
  int64_t T;
  int V;
  const int64_t* labels;
  const float* lse;
  const float* coef;
  float scale;
  void* grad;  // may be logits itself
  int splits, chunk;
};

// Workgroup = one chunk of one row; every element depends on itself alone.
// Rows go from the last to the first: the forward pass has just left the last
// ones in the last-level cache (8 us of the 486 above).
template <int XT>
__global__ __launch_bounds__(256) void pref_grad_kernel(PrefGradArgs a) {
  constexpr int U = 4, kPiece = 256 * 8;
  const int tid = (int)threadIdx.x;
  const RowSrc src{a.logits, nullptr};
  const int64_t items = a.T * a.splits;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t item = items - 1 - it;
    const int64_t t = item / a.splits;
    const int v0 = (int)(item - t * a.splits) * a.chunk;
    const int v1 = v0 + a.chunk < a.V ? v0 + a.chunk : a.V;
    const int64_t label = a.labels[t];
    const float c = scored(label) ? a.coef[t] * a.scale : 0.0f;
    const int full = v0 + (v1 - v0) / 8 * 8;
    if (c == 0.0f) {
      const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int b = v0 + 8 * tid; b < full; b += kPiece) store8<XT>(a.grad, t, a.V, b, z);
      if (full + tid < v1) {
        if constexpr (XT == kBf16) static_cast<uint16_t*>(a.grad)[t * a.V + full + tid] = 0;
        else static_cast<float*>(a.grad)[t * a.V + full + tid] = 0.0f;
      }
      continue;
    }
    const float lse = a.lse[t];
    const int at = label < a.V ? (int)label : -1;
    auto grad8 = [&](const Raw8<XT>& raw, int col) {
      float v[8];
      raw_to_f32<XT>(raw, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = -c * exp_from(v[j], lse);
      if ((unsigned)(at - col) < 8u) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j == at) v[j] += c;
      }
      store8<XT>(a.grad, t, a.V, col, v);
    };
    for (int b0 = v0; b0 < full; b0 += kPiece * U) {
      Raw8<XT> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int col = b0 + 8 * tid + kPiece * u;
        raw[u] = load_full8<XT, XT == kBf16>(src, t, a.V, col < full ? col : v0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int col = b0 + 8 * tid + kPiece * u;
        if (col < full) grad8(raw[u], col);
      }
    }
    if (full + tid < v1) {
      const int col = full + tid;
      float v = -c * exp_from(logit_at<XT>(a.logits, t, a.V, col), lse);
      if (col == at) v += c;
      if constexpr (XT == kBf16)
        static_cast<uint16_t*>(a.grad)[t * a.V + col] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
      else
        static_cast<float*>(a.grad)[t * a.V + col] = v;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct PrefSplit {
  int splits, chunk;
};
static PrefSplit pref_chunks(int64_t V, int64_t chunk) {
  chunk = (chunk + 2047) / 2048 * 2048;
  return PrefSplit{(int)((V + chunk - 1) / chunk), (int)chunk};
}
// Where rows are few, chunks of whole 2048 entries that give every CU four
// workgroups; one chunk a row otherwise.
static PrefSplit pref_row_split(int64_t T, int64_t V) {
  const int64_t want = ((int64_t)device_cus() * 4 + T - 1) / T;
  return pref_chunks(V, (V + want - 1) / want);
}
// The gradient takes chunks of 8192 entries at most, one batch of loads a
// workgroup: it writes as much as it reads, and with short workgroups the
// rows that are read and written at a time lie closer together (6144 x 131072
// bf16: 453 us in chunks of 6000 to 12000 entries, 486 us by whole rows, 505
// us in chunks of 3000; 1501 x 50021 fp32: 74 us, 116 us in chunks of 16384).
static PrefSplit pref_grad_split(int64_t T, int64_t V) {
  return pref_chunks(V, std::min(pref_row_split(T, V).chunk, 8192));
}

struct PrefWs {
  size_t part, lp, pair_loss, ticket, total;
};
static PrefWs pref_ws(int64_t T, int64_t V, int64_t pairs) {
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  const PrefSplit p = pref_row_split(T, V);
  PrefWs w;
  w.part = 0;
  w.lp = up(p.splits > 1 ? (size_t)T * p.splits * sizeof(MaxSum) : 0);
  w.pair_loss = w.lp + up((size_t)T * sizeof(float));
  w.ticket = w.pair_loss + up((size_t)pairs * sizeof(float));
  w.total = w.ticket + 256;
  return w;
}
size_t pref_ws_bytes(int64_t T, int64_t V, int64_t pairs) { return pref_ws(T, V, pairs).total; }

static unsigned capped(int64_t items) { return (unsigned)(items < ((int64_t)1 << 22) ? items : (int64_t)1 << 22); }

// pairs: 0 for the sequences' log-probabilities alone.
void launch_pref_fwd(int type, int64_t T, int64_t V, int64_t seqs, int64_t pairs, const void* logits,
                     const int64_t* labels, const int32_t* offsets, const float* ref, float beta, float smoothing,
                     float* loss, float* logps, float* lse, float* coef, void* workspace, hipStream_t stream) {
  const PrefSplit p = pref_row_split(T, V);
  const PrefWs w = pref_ws(T, V, pairs);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* ticket = reinterpret_cast<uint32_t*>(ws + w.ticket);
  PrefRowArgs r{logits, T, (int)V, labels, p.splits, p.chunk, reinterpret_cast<MaxSum*>(ws + w.part), lse,
                reinterpret_cast<float*>(ws + w.lp), pairs ? coef : nullptr, pairs ? ticket : nullptr};
  const dim3 grid(capped(T * p.splits));
  if (type == kBf16) hipLaunchKernelGGL(pref_rows_kernel<kBf16>, grid, dim3(256), 0, stream, r);
  else hipLaunchKernelGGL(pref_rows_kernel<kF32>, grid, dim3(256), 0, stream, r);
  int group = 1;
  while (group < p.splits && group < 64) group *= 2;
  PrefSeqArgs s{T, (int)V, pairs ? pairs : seqs, offsets, labels, logits, p.splits, group, r.part, lse, r.lp, logps, ref,
                beta, smoothing, pairs ? 1.0f / (float)pairs : 0.0f, coef,
                reinterpret_cast<float*>(ws + w.pair_loss), loss, ticket};
  const dim3 sgrid(capped(s.count));
  if (pairs) {
    if (type == kBf16) hipLaunchKernelGGL((pref_seq_kernel<kBf16, true>), sgrid, dim3(64 * kSeqWaves), 0, stream, s);
    else hipLaunchKernelGGL((pref_seq_kernel<kF32, true>), sgrid, dim3(64 * kSeqWaves), 0, stream, s);
  } else {
    if (type == kBf16) hipLaunchKernelGGL((pref_seq_kernel<kBf16, false>), sgrid, dim3(64 * kSeqWaves), 0, stream, s);
    else hipLaunchKernelGGL((pref_seq_kernel<kF32, false>), sgrid, dim3(64 * kSeqWaves), 0, stream, s);
  }
}

void launch_pref_grad(int type, int64_t T, int64_t V, const void* logits, const int64_t* labels, const float* lse,
                      const float* coef, float scale, void* grad, hipStream_t stream) {
  const PrefSplit p = pref_grad_split(T, V);
  PrefGradArgs g{logits, T, (int)V, labels, lse, coef, scale, grad, p.splits, p.chunk};
  const dim3 grid(capped(T * p.splits));
  if (type == kBf16) hipLaunchKernelGGL(pref_grad_kernel<kBf16>, grid, dim3(256), 0, stream, g);
  else hipLaunchKernelGGL(pref_grad_kernel<kF32>, grid, dim3(256), 0, stream, g);
}

}  // namespace qlora
