// Backward of the layer norm and RMS norm, with the reduction of the weights'
// gradients.  With xh = (x - mean) rstd, d = g w, p = sum d xh / n and
// q = sum d / n (q = 0 for rms), per row:
//   grad_x = rstd (d - q - xh p)
// and over the rows grad_w = sum g xh, grad_b = sum g.  A row of x and g stays
// in registers between the two uses, so each is read once; x may be its 8-bit
// checkpoint, restored in registers.  The weights' gradients add up in
// registers too: a workgroup walks many rows, a thread always holding the same
// columns, and writes one fp32 partial row at its end, which a second small
// kernel adds up in a fixed order (5 us at 256 rows of 8192).  Bound by HBM
// (operands that no cache holds, both launches): 8192 x 8192 bf16 rms 78 us (403
// MB, 5.2 TB/s; a plain copy moves 5.0-5.3), layer 81 us, from the 8-bit
// checkpoint 64 and 67 us (338 MB), 16384 x 4096 fp32 layer 151 us (805 MB, 5.3
// TB/s); without the weights' gradients 73, 73, 59 (rms) and 146 us.  2049 x 5001
// fp32 layer, 8 rows a workgroup, is not: 34 us (123 MB and 20 MB of partial
// rows, 4.2 TB/s), 25 us without the weights' gradients.
#include "norm.h"

namespace qlora {

// Ends what the compiler knows of a piece's registers, so that it restores the
// values from them again after the row's sums instead of keeping all of them
// (in fp32) through the sums.
template <int XT>
__device__ __forceinline__ void forget(Raw8<XT>& r) {
  if constexpr (XT == kBf16) asm volatile("" : "+v"(r.w));
  else if constexpr (XT == kF32) asm volatile("" : "+v"(r.v));
  else asm volatile("" : "+v"(r.k), "+v"(r.c));
}

struct NormBwdArgs {
  int layer;  // kLayer kernels also serve rms with a bias: mean = q = 0 then
  int n;
  int64_t M;
  float inv_n;
  RowSrc x;
  const void* g;
  const void* w;
  const float* mean;
  const float* rstd;
  void* gx;
  float* part;  // [gridDim.x][accs][pitch] fp32 sums of each workgroup's rows
  int pitch;
};

// kAcc: also sum grad_w (and, with kLayer, grad_b).
template <bool kLayer, bool kAcc, int XT, int WT, int NW, int VPT>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void norm_bwd_kernel(NormBwdArgs a) {
#pragma clang fp contract(off)  // the same roundings in every instantiation
  constexpr int GT = XT == kCkpt8 ? kBf16 : XT;
  constexpr int ACC = kAcc ? (kLayer ? 2 : 1) : 0;
  constexpr int K = kLayer ? 2 : 1;
  // the next row's loads go out ahead of this row's sums, except where the
  // widest rows leave no registers for it
  constexpr bool kAhead = VPT < 4;
  __shared__ float red[2][K][NW];
  constexpr int TPR = 64 * NW;
  const int wave = (int)threadIdx.x >> 6;
  const int t = NW == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * norm_rows(NW);
  const RowSrc gsrc{a.g, nullptr}, wsrc{a.w, nullptr};
  Raw8<WT> w[VPT];
  load_row<WT, VPT>(wsrc, 0, a.n, t, TPR, w);
  finish_row<WT, VPT>(a.n, t, TPR, w);
  float acc[ACC ? ACC : 1][VPT][8];
#pragma unroll
  for (int c = 0; c < ACC; ++c)
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[c][i][j] = 0.0f;
  int turn = 0;
  int64_t row = (int64_t)blockIdx.x * norm_rows(NW) + (NW == 1 ? wave : 0);
  Raw8<XT> xn[VPT];
  Raw8<GT> gn[VPT];
  // Where 8 or 16 waves share a row, its statistics are loaded ahead of its x
  // and g: loads are waited for in order, and after the next row's loads they
  // would make every row wait for all of those before its barrier (8192 x 8192
  // bf16 rms from a checkpoint 64 us, 69 us so; 8192 x 5120 rms 50 and 56 us;
  // 2049 x 5001 fp32 rms 32 and 35; only many long fp32 rows are slower, 8192 x
  // 8192 rms 152 and 148).  Elsewhere, with more rows in flight a CU, they are
  // loaded where they are used (131072 x 500 rms 82 us, 85 us with them first;
  // 32768 x 2048 rms 81 and 84).
  constexpr bool kStatsFirst = kAhead && NW > 4;
  float mean_n = 0.0f, rstd_n = 0.0f;
  auto load_stats = [&](int64_t at) {
    if constexpr (kLayer) mean_n = a.layer ? a.mean[at] : 0.0f;
    rstd_n = a.rstd[at];
  };
  if (kAhead && row < a.M) {
    if constexpr (kStatsFirst) load_stats(row);
    load_row<XT, VPT>(a.x, row, a.n, t, TPR, xn);
    load_row<GT, VPT>(gsrc, row, a.n, t, TPR, gn);
  }
  for (; row < a.M; row += step) {
    Raw8<XT> xr[VPT];
    Raw8<GT> gr[VPT];
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        xr[i] = xn[i];
        gr[i] = gn[i];
      }
    } else {
      load_row<XT, VPT>(a.x, row, a.n, t, TPR, xr);
      load_row<GT, VPT>(gsrc, row, a.n, t, TPR, gr);
    }
    finish_row<XT, VPT>(a.n, t, TPR, xr);
    finish_row<GT, VPT>(a.n, t, TPR, gr);
    float mean = mean_n, rstd = rstd_n;
    if constexpr (kAhead) {
      const int64_t ahead = row + step < a.M ? row + step : row;  // unconditional, as in the forward
      if constexpr (kStatsFirst) load_stats(ahead);
      load_row<XT, VPT>(a.x, ahead, a.n, t, TPR, xn);
      load_row<GT, VPT>(gsrc, ahead, a.n, t, TPR, gn);
    }
    if constexpr (!kStatsFirst) {
      load_stats(row);
      mean = mean_n;
      rstd = rstd_n;
    }
    float s[K];
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float x[8], g[8], wv[8];
      raw_to_f32<XT>(xr[i], x);
      raw_to_f32<GT>(gr[i], g);
      raw_to_f32<WT>(w[i], wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (kLayer ? x[j] - mean : x[j]) * rstd;
        const float d = g[j] * wv[j];
        s[0] = __builtin_fmaf(d, xh, s[0]);
        if constexpr (kLayer) s[1] += d;
        if constexpr (ACC > 0) acc[0][i][j] = __builtin_fmaf(g[j], xh, acc[0][i][j]);
        if constexpr (ACC > 1) acc[1][i][j] += g[j];
      }
    }
    row_sums<NW, K>(s, red, turn, wave);
    if constexpr (VPT == 4) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        forget<XT>(xr[i]);
        forget<GT>(gr[i]);
      }
    }
    const float p = s[0] * a.inv_n;
    const float q = kLayer && a.layer ? s[K - 1] * a.inv_n : 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float x[8], g[8], wv[8], o[8];
      raw_to_f32<XT>(xr[i], x);
      raw_to_f32<GT>(gr[i], g);
      raw_to_f32<WT>(w[i], wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (kLayer ? x[j] - mean : x[j]) * rstd;
        float d = g[j] * wv[j];
        if constexpr (kLayer) d -= q;
        o[j] = rstd * __builtin_fmaf(-xh, p, d);
      }
      store8<GT>(a.gx, row, a.n, 8 * (t + TPR * i), o);
    }
  }
  if constexpr (ACC > 0) {
    if constexpr (NW == 1) {
      __shared__ float sum[4][512 * VPT];  // the four waves' sums, added in wave order
#pragma unroll
      for (int c = 0; c < ACC; ++c) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[wave][8 * (t + 64 * i) + j] = acc[c][i][j];
        __syncthreads();
        for (int col = (int)threadIdx.x; col < a.n; col += 256)
          a.part[((int64_t)blockIdx.x * ACC + c) * a.pitch + col] =
              ((sum[0][col] + sum[1][col]) + sum[2][col]) + sum[3][col];
      }
    } else {
#pragma unroll
      for (int c = 0; c < ACC; ++c)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int col = 8 * (t + TPR * i);
          float* dst = a.part + ((int64_t)blockIdx.x * ACC + c) * a.pitch + col;
          if (col < a.pitch) {
            *reinterpret_cast<f32x4*>(dst) = f32x4{acc[c][i][0], acc[c][i][1], acc[c][i][2], acc[c][i][3]};
            *reinterpret_cast<f32x4*>(dst + 4) = f32x4{acc[c][i][4], acc[c][i][5], acc[c][i][6], acc[c][i][7]};
          }
        }
    }
  }
}

// grad_w and grad_b: the workgroups' partial rows added up.  Workgroup = 64
// columns of one of the two: 16 groups of 16 threads take every 16th part
// each, 4 columns a thread and 8 parts in flight, and the groups' sums are
// added in group order.
__global__ __launch_bounds__(256) void norm_param_sum_kernel(const float* __restrict__ part, int parts, int accs,
                                                             int n, int pitch, int w_f32, void* __restrict__ gw,
                                                             void* __restrict__ gb) {
  __shared__ f32x4 sum[16][17];
  const int tid = (int)threadIdx.x, lane = tid & 15, group = tid >> 4;
  const int tiles = (n + 63) / 64;
  const int c = (int)blockIdx.x / tiles;
  const int col = (int)(blockIdx.x % tiles) * 64 + 4 * lane;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (col < pitch) {
    for (int k0 = group; k0 < parts; k0 += 16 * 8) {
      f32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = k0 + 16 * u < parts ? k0 + 16 * u : group;
        v[u] = *reinterpret_cast<const f32x4*>(part + ((int64_t)k * accs + c) * pitch + col);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (k0 + 16 * u < parts) s += v[u];
    }
  }
  sum[group][lane] = s;
  __syncthreads();
  if (tid < 64) {
    const int o = (int)(blockIdx.x % tiles) * 64 + tid;
    if (o < n) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) v += sum[k][tid >> 2][tid & 3];
      void* out = c ? gb : gw;
      if (w_f32) static_cast<float*>(out)[o] = v;
      else static_cast<uint16_t*>(out)[o] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int64_t norm_max_width() { return kNormMaxWidth; }

// Workgroups of the backward pass, each one partial row of each gradient.
// More of them hide more of a row's latency and cost a partial row each,
// written and read in fp32, as much as about two rows of x, g and grad_x: two
// a CU for rows of 4096 values once each has 16 rows (16384 x 4096 fp32 layer
// 151 us, 156 us with one a CU; 4096 x 4096 bf16 rms from a checkpoint 23 and
// 24 us, but from bf16 26 and 24 us), one a CU for longer ones (2049 x 5001
// fp32 layer 34 us, 39 us with two; 8192 x 8192 bf16 layer 81 and 85 us), eight
// a CU where a wave takes a row of two pieces (65536 x 1000 bf16 rms 90 us, with
// four 89; 65536 x 1024 fp32 layer 159 us, with four 149).
static int64_t norm_bwd_groups(int64_t M, int64_t n) {
  int64_t groups = 0;
  norm_shape<true>(n, [&](auto nw, auto vpt) {
    constexpr int NW = decltype(nw)::value, VPT = decltype(vpt)::value;
    const int64_t want = (M + norm_rows(NW) - 1) / norm_rows(NW), cus = device_cus();
    const int64_t per_cu = NW == 1 ? 4 * VPT : NW == 4 ? 4 : n > 4096 || M < 16 * cus ? 1 : 2;
    groups = want < per_cu * cus ? want : per_cu * cus;
  });
  return groups;
}

static int norm_pitch(int64_t n) { return (int)((n + 7) / 8 * 8); }

// Gradients that the kernels sum: the layer norm's kernel sums both or none.
static int norm_sums(int layer, int accs) { return accs == 0 ? 0 : layer ? 2 : accs; }

size_t norm_bwd_ws_bytes(int layer, int64_t M, int64_t n, int accs) {
  return (size_t)norm_bwd_groups(M, n) * (size_t)norm_sums(layer, accs) * (size_t)norm_pitch(n) * sizeof(float);
}

template <bool kLayer, bool kAcc, int XT, int WT>
static void norm_bwd_shaped(const NormBwdArgs& a, hipStream_t stream) {
  norm_shape<true>(a.n, [&](auto nw, auto vpt) {
    constexpr int NW = decltype(nw)::value, VPT = decltype(vpt)::value;
    hipLaunchKernelGGL((norm_bwd_kernel<kLayer, kAcc, XT, WT, NW, VPT>), dim3((unsigned)norm_bwd_groups(a.M, a.n)),
                       dim3(NW == 1 ? 256 : 64 * NW), 0, stream, a);
  });
}

template <int XT, int WT>
static void norm_bwd_typed(const NormBwdArgs& a, int sums, hipStream_t stream) {
  if (a.layer || sums == 2)
    sums ? norm_bwd_shaped<true, true, XT, WT>(a, stream) : norm_bwd_shaped<true, false, XT, WT>(a, stream);
  else
    sums ? norm_bwd_shaped<false, true, XT, WT>(a, stream) : norm_bwd_shaped<false, false, XT, WT>(a, stream);
}

// accs: 0 none of the weights' gradients, 1 grad_w, 2 grad_w and grad_b.
void launch_norm_bwd(int layer, int x_type, int w_f32, int64_t M, int64_t n, const void* x, const uint8_t* x_scales,
                     const void* g, const void* w, const float* mean, const float* rstd, void* gx, int accs, void* gw,
                     void* gb, float* part, hipStream_t stream) {
  const int pitch = norm_pitch(n), sums = norm_sums(layer, accs);
  const NormBwdArgs a{layer, (int)n, M, 1.0f / (float)n, RowSrc{x, x_scales}, g, w, mean, rstd, gx, part, pitch};
  if (x_type == kF32) norm_bwd_typed<kF32, kF32>(a, sums, stream);
  else if (x_type == kBf16) w_f32 ? norm_bwd_typed<kBf16, kF32>(a, sums, stream) : norm_bwd_typed<kBf16, kBf16>(a, sums, stream);
  else w_f32 ? norm_bwd_typed<kCkpt8, kF32>(a, sums, stream) : norm_bwd_typed<kCkpt8, kBf16>(a, sums, stream);
  if (accs) {
    const int tiles = (int)((n + 63) / 64);
    hipLaunchKernelGGL(norm_param_sum_kernel, dim3((unsigned)(tiles * accs)), dim3(256), 0, stream, part,
                       (int)norm_bwd_groups(M, n), sums, (int)n, pitch, w_f32, gw, gb);
  }
}

}  // namespace qlora
