// The adapted linear layer of many experts: rows in order of their expert,
// expert e's being offsets[e] .. offsets[e + 1] - 1 (device memory, so that a
// router's result never visits the host):
//   u = x A_e^T,  h = x W'_e^T + s u B_e^T
//   v = g B_e,    grad_x = g W'_e + s v A_e,  grad_A_e = s v^T x,  grad_B_e = s g^T u
// "QLoRA: Efficient Fine-Tuning", Step 3 (Eq. 3) and Step 4 (Eq. 5) for each
// expert's rows; W'_e is rows e m .. (e + 1) m - 1 of one stacked weight.
//
// Every kernel cuts each expert's rows into tiles of its own size, numbers
// the tiles through all experts, and lets a workgroup find its tile from the
// offsets by itself (find_span): no launch lays a plan out first, and the
// host, which does not know the offsets, launches for the most tiles that
// they can make (rows / tile + one for each expert that can have a row);
// workgroups past the last tile end at once.  A tile then is a tile of the
// dense kernels on shifted operands: rows past the expert's last read as zero
// and are not written.
#include <type_traits>

#include "experts.h"
#include "gemm_tile.h"
#include "skinny.h"

namespace qlora {

// ---------------------------------------------------------------------------
// Tiles of ragged rows
// ---------------------------------------------------------------------------
struct ExpertRows {
  const int32_t* offsets;  // E + 1
  int E;
  int M;
};

struct Span {
  int e;      // expert
  int row0;   // its first row
  int rows;   // its rows
  int tile;   // tile of this expert
  int tiles;  // of how many
  int slot;   // tiles before this one that belong to experts with more than one
};

__device__ __forceinline__ int wave_scan_max(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, 64);
    v = lane >= d && o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ int wave_scan_add(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, 64);
    v += lane >= d ? o : 0;
  }
  return v;
}

// 64 experts at a time, one a lane.  Offsets are held within 0 .. M and below
// none before them, so that every row belongs to one expert at most whatever
// they hold, and the tiles of all experts are as few as the host assumes.
struct ExpertScan {
  int first = 0;               // expert of lane 0
  int end = 0;                 // last row + 1 of the experts before
  int tiles = 0, slots = 0;    // of the experts before
  int row0 = 0, rows = 0, t = 0, t_incl = 0, s_incl = 0;  // of this lane's expert, and with those of the lanes below

  __device__ __forceinline__ static int held(int v, int M) { return v < 0 ? 0 : v > M ? M : v; }
  __device__ __forceinline__ void begin(const ExpertRows& r) {
    first = tiles = slots = 0;
    end = held(r.offsets[0], r.M);
  }
  __device__ __forceinline__ void load(const ExpertRows& r, int bt) {
    const int lane = threadIdx.x & 63;
    const int e = first + lane;
    int last = held(r.offsets[e < r.E ? e + 1 : r.E], r.M);
    last = wave_scan_max(last > end ? last : end);
    const int prev = __shfl_up(last, 1, 64);
    row0 = lane ? prev : end;
    rows = e < r.E ? last - row0 : 0;
    t = (rows + bt - 1) / bt;
    t_incl = wave_scan_add(t);
    s_incl = wave_scan_add(t > 1 ? t : 0);
  }
  __device__ __forceinline__ void next(const ExpertRows& r) {
    first += 64;
    end = __builtin_amdgcn_readlane(row0 + rows, 63);
    tiles += __builtin_amdgcn_readlane(t_incl, 63);
    slots += __builtin_amdgcn_readlane(s_incl, 63);
  }
  __device__ __forceinline__ Span span(int lane, int tile) const {
    Span s;
    s.e = first + lane;
    s.row0 = __builtin_amdgcn_readlane(row0, lane);
    s.rows = __builtin_amdgcn_readlane(rows, lane);
    s.tiles = __builtin_amdgcn_readlane(t, lane);
    s.tile = tile;
    s.slot = slots + __builtin_amdgcn_readlane(s_incl, lane) - (s.tiles > 1 ? s.tiles : 0) + tile;
    return s;
  }
};

// The tile of bt rows that pick(number of tiles) names, found by every wave
// for itself; false where pick names none.
template <typename Pick>
__device__ __forceinline__ bool find_span(const ExpertRows& r, int bt, Pick pick, Span& s) {
  ExpertScan k;
  k.begin(r);
  k.load(r, bt);
  if (r.E > 64) {
    while (k.first + 64 < r.E) {
      k.next(r);
      k.load(r, bt);
    }
  }
  const int total = k.tiles + __builtin_amdgcn_readlane(k.t_incl, 63);
  const int item = __builtin_amdgcn_readfirstlane(pick(total));
  if (item < 0 || item >= total) return false;
  if (r.E > 64) {
    k.begin(r);
    k.load(r, bt);
    while (k.tiles + __builtin_amdgcn_readlane(k.t_incl, 63) <= item) {
      k.next(r);
      k.load(r, bt);
    }
  }
  const uint64_t after = __ballot(k.tiles + k.t_incl > item);
  const int lane = __builtin_ctzll(after);
  const int before = k.tiles + __builtin_amdgcn_readlane(k.t_incl - k.t, lane);
  s = k.span(lane, item - before);
  return true;
}

// Expert e's rows and tiles (its first).
__device__ __forceinline__ Span expert_span(const ExpertRows& r, int bt, int e) {
  ExpertScan k;
  k.begin(r);
  k.load(r, bt);
  while (e >= k.first + 64) {
    k.next(r);
    k.load(r, bt);
  }
  return k.span(e - k.first, 0);
}

// Most tiles of bt rows that M rows of E experts make.
static inline int64_t most_tiles(int64_t M, int64_t E, int64_t bt) { return M / bt + (E < M ? E : M); }

// ---------------------------------------------------------------------------
// h and grad_x: the dense GEMM's tile on an expert's operands
// ---------------------------------------------------------------------------
template <bool kBwd, bool kPieces>
__global__ __launch_bounds__(lg2::kThreads) void experts_gemm_kernel(GemmArgs p, ExpertRows er, Nf4Table tab) {
  using T = lg2::Tile<kBwd>;
  __shared__ __align__(16) uint8_t sw0[T::W];
  __shared__ __align__(16) uint8_t sw1[T::W];
  __shared__ __align__(16) uint8_t sa0[lg2::ATILEB];
  __shared__ __align__(16) uint8_t sa1[lg2::ATILEB];
  __shared__ uint32_t lds_word;
  const lg2::Lds lds{{sw0, sw1}, {sa0, sa1}};
  const int tid = threadIdx.x;
  int k0 = 0, ks = (int)((p.K + lg2::BK - 1) / lg2::BK);
  bool lora = true;
  int bid = (int)blockIdx.x;
  if (kPieces) {
    const int piece = bid % p.pieces;
    bid /= p.pieces;
    const int nk = ks;
    k0 = piece * nk / p.pieces;
    ks = (piece + 1) * nk / p.pieces - k0;
    lora = piece == p.pieces - 1;
  }
  // Row tiles are numbered through the experts, feature tiles fastest; each
  // XCD (workgroup number mod 8) takes a run of neighbouring tiles.
  int tile_f = 0;
  Span s;
  const bool found = find_span(er, lg2::BT, [&](int total) {
    const int tiles = total * p.tiles_f;
    int item = bid;
    if (!kPieces) {
      const int run = (tiles + 7) >> 3;
      item = (bid >> 3) < run ? (bid & 7) * run + (bid >> 3) : tiles;
    }
    tile_f = item % p.tiles_f;
    return item < tiles ? item / p.tiles_f : -1;
  }, s);
  if (!found) return;
  const int64_t cells = p.wm * p.wn;
  const int64_t block0 = s.e * (cells / kBlock);
  p.act += s.row0 * p.K;
  p.codes += s.e * (cells / 2);
  p.absmax8 += block0;
  p.c2 += block0 / kGroupBlocks;
  const uint32_t skew = (uint32_t)(block0 % kGroupBlocks);
  p.lora_a += (int64_t)s.e * p.N * p.r;
  p.lora_b += (int64_t)s.row0 * p.r;
  p.out += s.row0 * p.N;
  p.M = s.rows;
  const int64_t f0 = (int64_t)tile_f * lg2::BF;
  const int64_t t0 = (int64_t)s.tile * lg2::BT;
  if (tid >= 64 * lg2::kMfmaWaves)
    gemm_producer<kBwd>(p, tab, lds, tid - 64 * lg2::kMfmaWaves, f0, t0, k0, ks, lora, 0, &lds_word, skew);
  else
    gemm_consumer<kBwd, kPieces, true>(p, lds, tid, f0, t0, k0, ks, lora, 0, &lds_word);
}

// Finishes tiles that ran as K pieces: out = bf16(piece 0 + piece 1 + ...), in
// the consumer's [wave][i][j][lane] order, 256 items of 4 features a workgroup.
template <bool kBwd>
__global__ __launch_bounds__(256) void experts_pieces_kernel(GemmArgs p, ExpertRows er) {
  constexpr int WF = kBwd ? 64 : 128;
  constexpr int WT = 128 * 64 / WF;
  constexpr int NI = WF / 16, NJ = WT / 16;
  constexpr int kItems = lg2::BF * lg2::BT / 4;
  const int tile = (int)blockIdx.x / (kItems / 256);
  const int rem = ((int)blockIdx.x % (kItems / 256)) * 256 + (int)threadIdx.x;
  Span s;
  if (!find_span(er, lg2::BT, [&](int total) { return tile < total * p.tiles_f ? tile / p.tiles_f : -1; }, s)) return;
  const int wave = rem / (NI * NJ * 64);
  const int ij = (rem / 64) % (NI * NJ);
  const int lane = rem % 64;
  const int i = ij / NJ, j = ij % NJ;
  const int64_t t = (int64_t)s.tile * lg2::BT + (wave / (lg2::BF / WF)) * WT + 16 * j + (lane & 15);
  const int64_t f = (int64_t)(tile % p.tiles_f) * lg2::BF + (wave % (lg2::BF / WF)) * WF + 16 * i + 4 * (lane >> 4);
  if (t >= s.rows || f >= p.N) return;
  const float* slot = p.piece_out + (size_t)tile * p.pieces * kItems * 4 + (size_t)rem * 4;
  f32x4 v = *reinterpret_cast<const f32x4*>(slot);
  for (int q = 1; q < p.pieces; ++q) v += *reinterpret_cast<const f32x4*>(slot + (size_t)q * kItems * 4);
  uint16_t* dst = p.out + (s.row0 + t) * p.N + f;
  const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  if ((p.N & 3) == 0) {
    *reinterpret_cast<u32x2*>(dst) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (f + e < p.N) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// K pieces of a GEMM with at most `tiles` tiles: as for the dense layer, up to
// a workgroup a CU, with at least 8 K steps to a piece.
static int experts_pieces(int64_t tiles, int64_t K) {
  const int64_t nk = cdiv(K, lg2::BK);
  int64_t pc = device_cus() / tiles;
  if (pc > 16) pc = 16;
  while (pc > 1 && nk / pc < 8) --pc;
  return pc < 1 ? 1 : (int)pc;
}

static int64_t gemm_tiles(int64_t M, int64_t E, int64_t N) { return most_tiles(M, E, lg2::BT) * cdiv(N, lg2::BF); }

bool experts_gemm_fits(int64_t M, int64_t E, int64_t N) { return gemm_tiles(M, E, N) < ((int64_t)1 << 24); }

size_t experts_gemm_ws_bytes(int64_t M, int64_t E, int64_t N, int64_t K) {
  const int64_t tiles = gemm_tiles(M, E, N);
  const int pc = experts_pieces(tiles, K);
  return pc > 1 ? (size_t)(tiles * pc) * lg2::BF * lg2::BT * sizeof(float) : 0;
}

// bwd: act = g (M x K, K = m or m rounded up to 64 with zero columns), out =
// grad_x; otherwise act = x, out = h.  ws: experts_gemm_ws_bytes.
void launch_experts_gemm(bool bwd, const int32_t* offsets, int64_t E, const uint16_t* act, const uint8_t* codes,
                         const uint8_t* absmax8, const float* c2, const uint16_t* lora_a, const float* lora_b,
                         uint16_t* out, int64_t M, int64_t K, int64_t n, int64_t m, int r, float s, void* ws,
                         const Nf4Table& tab, hipStream_t stream) {
  GemmArgs p{};
  p.act = act; p.codes = codes; p.absmax8 = absmax8; p.c2 = c2; p.lora_a = lora_a; p.lora_b = lora_b; p.out = out;
  p.M = M; p.K = K; p.N = bwd ? n : m; p.wn = n; p.wm = m; p.r = r; p.s = s;
  p.tiles_f = (int)cdiv(p.N, lg2::BF);
  const ExpertRows er{offsets, (int)E, (int)M};
  const int64_t tiles = gemm_tiles(M, E, p.N);
  const dim3 block(lg2::kThreads);
  p.pieces = experts_pieces(tiles, K);
  if (p.pieces > 1) {
    p.piece_out = static_cast<float*>(ws);
    const dim3 grid((unsigned)(tiles * p.pieces)), rgrid((unsigned)(tiles * (lg2::BF * lg2::BT / 4 / 256)));
    if (bwd) {
      hipLaunchKernelGGL((experts_gemm_kernel<true, true>), grid, block, 0, stream, p, er, tab);
      hipLaunchKernelGGL(experts_pieces_kernel<true>, rgrid, dim3(256), 0, stream, p, er);
    } else {
      hipLaunchKernelGGL((experts_gemm_kernel<false, true>), grid, block, 0, stream, p, er, tab);
      hipLaunchKernelGGL(experts_pieces_kernel<false>, rgrid, dim3(256), 0, stream, p, er);
    }
    return;
  }
  const dim3 grid((unsigned)(cdiv(tiles, 8) * 8));
  if (bwd)
    hipLaunchKernelGGL((experts_gemm_kernel<true, false>), grid, block, 0, stream, p, er, tab);
  else
    hipLaunchKernelGGL((experts_gemm_kernel<false, false>), grid, block, 0, stream, p, er, tab);
}

// ---------------------------------------------------------------------------
// u = x A_e^T and v = g B_e
// ---------------------------------------------------------------------------

// Y: A, E x [R][K], or (kYT) B, E x [yrows][R].
template <int RB, bool kYT>
__global__ __launch_bounds__(256) void experts_down_kernel(const uint16_t* __restrict__ X, ExpertRows er, int64_t K,
                                                           const uint16_t* __restrict__ Y, int R,
                                                           float* __restrict__ part, int64_t kc, int64_t yrows) {
  Span s;
  if (!find_span(er, sk::DT, [&](int) { return (int)blockIdx.x; }, s)) return;
  skinny_down_tile<RB, 3, 8, kYT, true>(X + s.row0 * K, s.rows, K, Y + s.e * (yrows * R), R,
                                        part + ((int64_t)blockIdx.y * er.M + s.row0) * R, kc, yrows,
                                        (int64_t)s.tile * sk::DT, (int)blockIdx.y);
}

static inline int rank_blocks(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

int experts_down_splits(int64_t M, int64_t E, int64_t K, int R) {
  const int64_t slots = (int64_t)(rank_blocks(R) <= 4 ? 2 : 1) * device_cus();
  int64_t want = cdiv(slots, most_tiles(M, E, sk::DT));
  const int64_t most = cdiv(K, 512);
  if (want > most) want = most;
  if (want > 64) want = 64;
  return (int)cdiv(K, cdiv(cdiv(K, want), 128) * 128);
}

// part: splits x M x R.  yt: Y holds R ranks a row (R a multiple of 8).
void launch_experts_down(const uint16_t* X, const int32_t* offsets, int64_t M, int64_t E, int64_t K, const uint16_t* Y,
                         bool yt, int64_t yrows, int R, float* part, int splits, hipStream_t stream) {
  const int64_t kc = cdiv(cdiv(K, splits), 128) * 128;
  const ExpertRows er{offsets, (int)E, (int)M};
  const dim3 grid((unsigned)most_tiles(M, E, sk::DT), (unsigned)splits);
  auto go = [&](auto rb) {
    constexpr int RB = decltype(rb)::value;
    if (yt)
      hipLaunchKernelGGL((experts_down_kernel<RB, true>), grid, dim3(256), 0, stream, X, er, K, Y, R, part, kc, yrows);
    else
      hipLaunchKernelGGL((experts_down_kernel<RB, false>), grid, dim3(256), 0, stream, X, er, K, Y, R, part, kc, K);
  };
  using std::integral_constant;
  switch (rank_blocks(R)) {
    case 1: go(integral_constant<int, 1>{}); break;
    case 2: go(integral_constant<int, 2>{}); break;
    case 4: go(integral_constant<int, 4>{}); break;
    default: go(integral_constant<int, 8>{}); break;
  }
}

// B_e^T (R x ld, zeros from column m on) of every expert, for ranks whose rows
// of B are not whole 16-byte pieces.
__global__ __launch_bounds__(256) void experts_transpose_kernel(const uint16_t* __restrict__ B, int64_t m, int R,
                                                                int64_t ld, int64_t count,
                                                                uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // over E x R x ld
  if (i >= count) return;
  const int64_t f = i % ld, eq = i / ld;
  const int64_t e = eq / R, q = eq % R;
  out[i] = f < m ? B[(e * m + f) * R + q] : (uint16_t)0;
}

void launch_experts_transpose(const uint16_t* B, int64_t E, int64_t m, int R, int64_t ld, uint16_t* out,
                              hipStream_t stream) {
  const int64_t count = E * R * ld;
  hipLaunchKernelGGL(experts_transpose_kernel, dim3((unsigned)cdiv(count, 256)), dim3(256), 0, stream, B, m, R, ld,
                     count, out);
}

// Sums the splits of u or v in order: fp32 out (may be null) and, for the
// products over rows, bf16 hi and lo planes [M][16 RB] with zero ranks from R
// on (planes may be null).  Rows outside every expert are left alone.
__global__ __launch_bounds__(256) void experts_factor_kernel(FactorJob a, FactorJob b, ExpertRows er, int R, int RP) {
  const FactorJob j = blockIdx.y ? b : a;
  const int i = (int)(blockIdx.x * 256 + threadIdx.x);  // rank pairs of all rows (fewer than 2^29)
  const int row = i / (RP / 2);
  const int q = i % (RP / 2) * 2;
  // the rows that belong to an expert: offsets[0] .. the largest offset
  int top = 0;
  for (int e = threadIdx.x & 63; e <= er.E; e += 64) {
    const int o = er.offsets[e];
    top = o > top ? o : top;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const int o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
  }
  const int low = er.offsets[0];
  if (row >= er.M || row < low || row >= top) return;
  float v[2] = {0.0f, 0.0f};
  const int64_t stride = (int64_t)er.M * R;
  const float* src = j.part + (int64_t)row * R + q;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (q + c < R) {
      float s = 0.0f;
      for (int k = 0; k < j.splits; k += 8) {
        float w[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] = k + x < j.splits ? src[(k + x) * stride + c] : 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x) s += w[x];
      }
      v[c] = s;
      if (j.out) j.out[(int64_t)row * R + q + c] = s;
    }
  if (!j.planes) return;
  float h0, l0, h1, l1;
  split_bf16(v[0], h0, l0);
  split_bf16(v[1], h1, l1);
  uint16_t* p = j.planes + (int64_t)row * RP + q;
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(h0, h1);
  *reinterpret_cast<uint32_t*>(p + (int64_t)er.M * RP) = pack_bf16x2(l0, l1);
}

size_t experts_planes_bytes(int64_t M, int R) { return (size_t)M * 16 * rank_blocks(R) * 4; }

// jobs: 1 or 2
void launch_experts_factor(const FactorJob* jobs, int count, const int32_t* offsets, int64_t M, int64_t E, int R,
                           hipStream_t stream) {
  const int RP = 16 * rank_blocks(R);
  const ExpertRows er{offsets, (int)E, (int)M};
  const dim3 grid((unsigned)cdiv(M * (RP / 2), 256), (unsigned)count);
  hipLaunchKernelGGL(experts_factor_kernel, grid, dim3(256), 0, stream, jobs[0], jobs[count - 1], er, R, RP);
}

// ---------------------------------------------------------------------------
// grad_A_e = s v^T x, grad_B_e = s g^T u: products over an expert's rows
// ---------------------------------------------------------------------------
// A workgroup takes 128 columns of x (or g) and all ranks, and walks one
// chunk of an expert's rows in stages of 64 through an LDS ring: the rows in
// their own layout and both planes of the factor, read transposed as MFMA
// operands.  An expert whose rows are one chunk gets its gradient from here;
// of more chunks each leaves fp32 sums in a slot, which experts_sum_kernel
// adds in order (it also writes the zeros of experts without rows).
struct TokenJob {
  const uint16_t* X;   // M x ld
  int64_t J, ld;       // columns that count, row length
  const uint16_t* P;   // planes of the factor
  uint16_t* out;       // E x [R][J] (rank_major) or E x [J][R]
  float* part;         // slots x J R, in out's order
  int tiles;           // column tiles
  int chunk;           // rows
  bool rank_major;
};

struct TokenArgs {
  TokenJob job[2];
  int first;           // workgroups of job 0
  ExpertRows er;
  int R;
  float s;
};

// Plane row t holds RB units of 16 ranks (32 bytes).  The eight rows of one
// transposed read (t, t + 1, t + 2, t + 3 and those plus 8) take one unit each;
// they fall into different banks where row bits that do not move the address
// by less than 256 bytes flip the unit, or with one unit a row the row.
template <int RB>
__device__ __forceinline__ int plane_flip(int t) {
  const int f = (t & 3) | (((t >> 3) & 1) << 2);
  return RB == 8 ? f : RB == 4 ? f >> 1 : RB == 2 ? f >> 2 : 0;
}
template <int RB>
__device__ __forceinline__ int plane_row(int t) {
  return RB == 1 ? t ^ (((t >> 3) & 1) << 2) : t;
}

template <int RB, int NS>
__global__ __launch_bounds__(256) void experts_token_kernel(TokenArgs a) {
  constexpr int XB = sk::TS * 256;       // 64 rows x 128 columns
  constexpr int PB = sk::TS * 32 * RB;   // one plane: 64 rows x 16 RB ranks
  constexpr int STAGE = XB + 2 * PB;
  __shared__ __align__(16) uint8_t s0[STAGE];
  __shared__ __align__(16) uint8_t s1[STAGE];
  __shared__ __align__(16) uint8_t s2[STAGE];
  __shared__ __align__(16) uint8_t s3[NS > 3 ? STAGE : 16];
  uint8_t* const buf4[4] = {s0, s1, s2, s3};
  uint8_t* buf[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) buf[i] = buf4[i];
  const int which = (int)blockIdx.x >= a.first ? 1 : 0;
  const TokenJob& job = a.job[which];
  const int bid = (int)blockIdx.x - (which ? a.first : 0);
  Span sp;
  if (!find_span(a.er, job.chunk, [&](int) { return bid / job.tiles; }, sp)) return;
  const int R = a.R;
  const int64_t J = job.J, ld = job.ld;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15;
  const int lq = lane >> 4;
  const int64_t j0 = (int64_t)(bid % job.tiles) * sk::TJ;
  const int tbeg = sp.tile * job.chunk;
  const int tend = tbeg + job.chunk < sp.rows ? tbeg + job.chunk : sp.rows;
  const int nst = (tend - tbeg + sk::TS - 1) / sk::TS;
  const uint32_t xbytes = (uint32_t)(sp.rows * ld * 2);
  // both planes behind one buffer: fewer than 2^22 rows of 256 bytes at most
  const uint32_t plane = (uint32_t)a.er.M * (32u * RB);
  const uint32_t pbytes = plane + (uint32_t)sp.rows * (32u * RB);
  const brsrc_t rx = make_rsrc(job.X + sp.row0 * ld, xbytes);
  const brsrc_t rp = make_rsrc(job.P + (int64_t)sp.row0 * (16 * RB), pbytes);
  const int xrow = lane >> 4;
  const int slot = lane & 15;
  constexpr int LMIN = 4 + RB;
  auto issue = [&](int s, uint8_t* stg) {
    const int tb = tbeg + s * sk::TS;
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // rows 16 w .. 16 w + 15 of the stage, 4 a load (swtg)
      const int blk = 4 * wave + b;
      const int row = 4 * blk + xrow;
      const int f = (row & 3) | (((row >> 3) & 1) << 2);
      const int c = ((((slot >> 1) ^ f)) << 1) | (slot & 1);
      const int64_t j = j0 + 8 * c;
      dma16(rx, stg + blk * 1024, (tb + row < tend && j < ld) ? (uint32_t)(((tb + row) * ld + j) * 2) : xbytes);
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {  // 1 KB blocks 4 b + w of the two planes (2 RB blocks each)
      const int id = 4 * b + wave;
      const int pl = id / (2 * RB);
      const int pos = (id % (2 * RB)) * 64 + lane;  // 16-byte piece of the plane's tile
      const int row = plane_row<RB>(pos / (2 * RB));
      const int unit = ((pos % (2 * RB)) >> 1) ^ plane_flip<RB>(row);
      dma16(rp, stg + XB + pl * PB + (id % (2 * RB)) * 1024,
            tb + row < tend ? pl * plane + (uint32_t)((tb + row) * (32 * RB) + unit * 32 + (pos & 1) * 16) : pbytes);
    }
  };
  f32x4 acc[2][RB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < RB; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int tr_row = lr >> 2;
  const int tr_c = lr & 3;
  auto read_tr = [](const uint8_t* p0, const uint8_t* p1) -> u32x4 {
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p0));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p1));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };
  auto compute = [&](const uint8_t* stg) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      // lanes 4 r + c of each 16-lane group address row r, columns 4 c .. 4 c + 3
      const int t = 32 * kk + 8 * lq + tr_row;
      u32x4 x[2];
#pragma unroll
      for (int ib = 0; ib < 2; ++ib) {
        const int c = 2 * (2 * wave + ib) + (tr_c >> 1);
        x[ib] = read_tr(stg + swtg(t, c) + (tr_c & 1) * 8, stg + swtg(t + 4, c) + (tr_c & 1) * 8);
      }
#pragma unroll
      for (int cb = 0; cb < RB; ++cb) {
        const int o0 = plane_row<RB>(t) * (32 * RB) + ((cb ^ plane_flip<RB>(t)) << 5) + 8 * tr_c;
        const int o1 = plane_row<RB>(t + 4) * (32 * RB) + ((cb ^ plane_flip<RB>(t + 4)) << 5) + 8 * tr_c;
        const u32x4 yh = read_tr(stg + XB + o0, stg + XB + o1);
        const u32x4 yl = read_tr(stg + XB + PB + o0, stg + XB + PB + o1);
#pragma unroll
        for (int ib = 0; ib < 2; ++ib) {
          acc[ib][cb] = mfma16x16x32(x[ib], yh, acc[ib][cb]);
          acc[ib][cb] = mfma16x16x32(x[ib], yl, acc[ib][cb]);
        }
      }
    }
  };
  ring_run<NS, LMIN>(nst, buf, issue, compute);

  // lane holds columns 32 w + 16 ib + 4 lq + e, rank 16 cb + lr
  const bool whole = sp.tiles == 1;
  uint16_t* out = job.out + sp.e * (J * R);
  float* part = job.part + sp.slot * (J * R);
#pragma unroll
  for (int cb = 0; cb < RB; ++cb) {
    const int q = 16 * cb + lr;
    if (q >= R) continue;
#pragma unroll
    for (int ib = 0; ib < 2; ++ib) {
      const int64_t j = j0 + 32 * wave + 16 * ib + 4 * lq;
      const f32x4 v = acc[ib][cb];
      if (job.rank_major) {  // J is a multiple of 64
        if (j >= J) continue;
        if (whole)
          *reinterpret_cast<u32x2*>(out + q * J + j) =
              u32x2{pack_bf16x2(a.s * v[0], a.s * v[1]), pack_bf16x2(a.s * v[2], a.s * v[3])};
        else
          *reinterpret_cast<f32x4*>(part + q * J + j) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (j + e >= J) break;
          if (whole)
            out[(j + e) * R + q] = (uint16_t)(pack_bf16x2(a.s * v[e], 0.0f) & 0xFFFFu);
          else
            part[(j + e) * R + q] = v[e];
        }
      }
    }
  }
}

constexpr int kSumCells = 4096;  // of a workgroup

__global__ __launch_bounds__(256) void experts_sum_kernel(TokenArgs a) {
  const TokenJob& job = a.job[blockIdx.z];
  const int64_t cells = job.J * a.R;
  const int64_t i0 = (int64_t)blockIdx.x * kSumCells;
  if (i0 >= cells) return;
  const Span sp = expert_span(a.er, job.chunk, (int)blockIdx.y);
  if (sp.tiles == 1) return;
  uint16_t* out = job.out + sp.e * cells;
  const float* part = job.part + sp.slot * cells;
  const int64_t i1 = i0 + kSumCells < cells ? i0 + kSumCells : cells;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
    float s = 0.0f;
    for (int k = 0; k < sp.tiles; k += 8) {
      float w[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) w[x] = k + x < sp.tiles ? part[(k + x) * cells + i] : 0.0f;
#pragma unroll
      for (int x = 0; x < 8; ++x) s += w[x];
    }
    out[i] = (uint16_t)(pack_bf16x2(a.s * s, 0.0f) & 0xFFFFu);
  }
}

// Rows of a chunk: enough workgroups for a few rounds of the chip (rows of
// experts differ, so one round would end with the longest), but no fewer than
// 256 rows, below which the sums weigh as much as the rows.
static int token_chunk(int64_t M, int64_t J, int R) {
  const int64_t want = (int64_t)3 * (rank_blocks(R) <= 2 ? 2 : 1) * device_cus();
  int64_t c = cdiv(cdiv(M * cdiv(J, sk::TJ), want), 64) * 64;
  return (int)(c < 256 ? 256 : c);
}

// Experts of more than one chunk have fewer than 2 M / chunk chunks in all.
size_t experts_token_ws_bytes(int64_t M, int64_t J, int R) {
  return (size_t)(2 * M / token_chunk(M, J, R)) * J * R * sizeof(float);
}

bool experts_token_fits(int64_t M, int64_t E, int64_t J) { return most_tiles(M, E, 256) * cdiv(J, sk::TJ) < ((int64_t)1 << 30); }

void launch_experts_token(const uint16_t* x, const uint16_t* vplanes, uint16_t* grad_A, float* part_a,
                          const uint16_t* g, int64_t g_ld, const uint16_t* uplanes, uint16_t* grad_B, float* part_b,
                          const int32_t* offsets, int64_t M, int64_t E, int64_t n, int64_t m, int R, float s,
                          hipStream_t stream) {
  TokenArgs a{};
  a.job[0] = TokenJob{x, n, n, vplanes, grad_A, part_a, (int)cdiv(n, sk::TJ), token_chunk(M, n, R), true};
  a.job[1] = TokenJob{g, m, g_ld, uplanes, grad_B, part_b, (int)cdiv(m, sk::TJ), token_chunk(M, m, R), false};
  a.er = ExpertRows{offsets, (int)E, (int)M};
  a.R = R;
  a.s = s;
  a.first = (int)(most_tiles(M, E, a.job[0].chunk) * a.job[0].tiles);
  const dim3 grid((unsigned)(a.first + most_tiles(M, E, a.job[1].chunk) * a.job[1].tiles));
  switch (rank_blocks(R)) {
    case 1: hipLaunchKernelGGL((experts_token_kernel<1, 3>), grid, dim3(256), 0, stream, a); break;
    case 2: hipLaunchKernelGGL((experts_token_kernel<2, 3>), grid, dim3(256), 0, stream, a); break;
    case 4: hipLaunchKernelGGL((experts_token_kernel<4, 4>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((experts_token_kernel<8, 3>), grid, dim3(256), 0, stream, a); break;
  }
  const int64_t most = (n > m ? n : m) * R;
  hipLaunchKernelGGL(experts_sum_kernel, dim3((unsigned)cdiv(most, kSumCells), (unsigned)E, 2), dim3(256), 0, stream,
                     a);
}

}  // namespace qlora
