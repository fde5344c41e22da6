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

// Inclusive scans over the wave's lanes of values that are not negative, by
// DPP row shifts and broadcasts (lanes without a source get 0).
template <typename Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
  auto step = [&](auto ctrl, auto rows) {
    v = op(v, __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false));
  };
  using std::integral_constant;
  step(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});  // row_shr:1
  step(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});  // row_shr:2
  step(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});  // row_shr:4
  step(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});  // row_shr:8
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // row_bcast:15 into rows 1 and 3
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // row_bcast:31 into rows 2 and 3
  return v;
}
__device__ __forceinline__ int wave_scan_max(int v) {
  return wave_scan(v, [](int a, int b) { return a > b ? a : b; });
}
__device__ __forceinline__ int wave_scan_add(int v) {
  return wave_scan(v, [](int a, int b) { return a + b; });
}

// 64 experts at a time, one a lane, the next 64 offsets on their way.  Offsets
// are held within 0 .. M and below none before them, so that every row belongs
// to one expert at most whatever they hold, and the tiles of all experts are as
// few as the host assumes.  kMany: more than 64 experts (1024 x 4096 x 512,
// 40000 rows: 1160 us, its bytes some 290; with a second pass over all offsets,
// and none on their way, 1340.  One form for all numbers costs 64 x 1024 x 2048 1 us of 55).
template <bool kMany>
struct ExpertScan {
  int first = 0;               // expert of lane 0
  int end = 0;                 // last row + 1 of the experts before
  int tiles = 0, slots = 0;    // of the experts before
  int row0 = 0, rows = 0, t = 0;  // of this lane's expert
  int t_incl = 0, s_incl = 0;     // with those of the lanes below

  int ahead = 0;  // offset behind this lane's expert of the 64 that are loaded next
  // Lane k: what comes before the experts from 64 k on (of those passed; 64
  // lanes hold 4096 experts), so that a second look at any 64 is one step.
  int k_end = 0, k_tiles = 0, k_slots = 0;

  __device__ __forceinline__ static int held(int v, int M) { return v < 0 ? 0 : v > M ? M : v; }
  __device__ __forceinline__ void fetch(const ExpertRows& r, int from) {
    const int e = from + (threadIdx.x & 63);
    ahead = r.offsets[e < r.E ? e + 1 : r.E];
  }
  __device__ __forceinline__ void begin(const ExpertRows& r) {
    first = tiles = slots = 0;
    fetch(r, 0);
    end = held(r.offsets[0], r.M);
  }
  __device__ __forceinline__ void load(const ExpertRows& r, int bt) {
    const int lane = threadIdx.x & 63;
    int last = held(ahead, r.M);
    if (kMany) {
      if (first + 64 < r.E) fetch(r, first + 64);
      if (lane == first >> 6) {
        k_end = end;
        k_tiles = tiles;
        k_slots = slots;
      }
    }
    last = wave_scan_max(last > end ? last : end);
    row0 = __builtin_amdgcn_update_dpp(end, last, 0x138, 0xF, 0xF, false);  // wave_shr:1, `end` into lane 0
    rows = first + lane < r.E ? last - row0 : 0;
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
  // Back to the last of the 64s passed whose lane has `before` at most `want`.
  __device__ __forceinline__ void again(const ExpertRows& r, int bt, int before, int want) {
    const int lane = threadIdx.x & 63;
    const int k = 63 - __builtin_clzll(__ballot(lane <= first >> 6 && before <= want));
    if (k != first >> 6) {
      first = 64 * k;
      end = __builtin_amdgcn_readlane(k_end, k);
      tiles = __builtin_amdgcn_readlane(k_tiles, k);
      slots = __builtin_amdgcn_readlane(k_slots, k);
      fetch(r, first);
      load(r, bt);
    }
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
template <bool kMany, typename Pick>
__device__ __forceinline__ bool find_span_of(const ExpertRows& r, int bt, Pick pick, Span& s) {
  ExpertScan<kMany> k;
  k.begin(r);
  k.load(r, bt);
  while (kMany && k.first + 64 < r.E) {
    k.next(r);
    k.load(r, bt);
  }
  const int total = k.tiles + __builtin_amdgcn_readlane(k.t_incl, 63);
  const int item = __builtin_amdgcn_readfirstlane(pick(total));
  if (item < 0 || item >= total) return false;
  if (kMany) k.again(r, bt, k.k_tiles, item);
  const uint64_t after = __ballot(k.tiles + k.t_incl > item);
  const int lane = __builtin_ctzll(after);
  const int before = k.tiles + __builtin_amdgcn_readlane(k.t_incl - k.t, lane);
  s = k.span(lane, item - before);
  return true;
}
template <typename Pick>
__device__ __forceinline__ bool find_span(const ExpertRows& r, int bt, Pick pick, Span& s) {
  return r.E > 64 ? find_span_of<true>(r, bt, pick, s) : find_span_of<false>(r, bt, pick, s);
}

// The same with the tiles numbered whole ones first and then each expert's
// ragged last one: a launch then ends with its short tiles.  pick(whole,
// ragged) names a tile of whole + ragged.
template <bool kMany, typename Pick>
__device__ __forceinline__ bool find_whole_first_of(const ExpertRows& r, int bt, Pick pick, Span& s) {
  auto counts = [&](const ExpertScan<kMany>& k, int& w, int& g) {  // of the lanes up to this one
    const int whole = k.rows / bt;
    g = __popcll(__ballot(k.t > whole) & (~0ull >> (63 - (threadIdx.x & 63))));
    w = k.t_incl - g;
  };
  ExpertScan<kMany> k;
  k.begin(r);
  k.load(r, bt);
  int w, g, whole = 0, ragged = 0, k_whole = 0;
  for (;;) {
    if (kMany && (int)(threadIdx.x & 63) == k.first >> 6) k_whole = whole;
    counts(k, w, g);
    whole += __builtin_amdgcn_readlane(w, 63);
    ragged += __builtin_amdgcn_readlane(g, 63);
    if (!kMany || k.first + 64 >= r.E) break;
    k.next(r);
    k.load(r, bt);
  }
  const int item = __builtin_amdgcn_readfirstlane(pick(whole, ragged));
  if (item < 0 || item >= whole + ragged) return false;
  const bool last = item >= whole;
  int want = last ? item - whole : item;  // among the tiles of its kind
  if (kMany) {
    const int before = last ? k.k_tiles - k_whole : k_whole;
    k.again(r, bt, before, want);
    want -= __builtin_amdgcn_readlane(before, k.first >> 6);
    counts(k, w, g);
  }
  const int lane = __builtin_ctzll(__ballot((last ? g : w) > want));
  const int full = __builtin_amdgcn_readlane(k.rows / bt, lane);
  s = k.span(lane, last ? full : want - (__builtin_amdgcn_readlane(w, lane) - full));
  return true;
}
template <typename Pick>
__device__ __forceinline__ bool find_span_whole_first(const ExpertRows& r, int bt, Pick pick, Span& s) {
  return r.E > 64 ? find_whole_first_of<true>(r, bt, pick, s) : find_whole_first_of<false>(r, bt, pick, s);
}

// Expert e's rows and tiles (its first).
__device__ __forceinline__ Span expert_span(const ExpertRows& r, int bt, int e) {
  ExpertScan<true> k;
  k.begin(r);
  k.load(r, bt);
  while (e >= k.first + 64) {
    k.next(r);
    k.load(r, bt);
  }
  return k.span(e - k.first, 0);
}

// The rows that belong to an expert: offsets[0] .. the largest offset, within
// 0 .. M.
__device__ __forceinline__ void live_rows(const ExpertRows& r, int& low, int& top) {
  top = 0;
  for (int e = threadIdx.x & 63; e <= r.E; e += 64) {
    const int o = r.offsets[e];
    top = o > top ? o : top;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const int o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
  }
  top = top < r.M ? top : r.M;
  low = ExpertScan<false>::held(r.offsets[0], r.M);
}

// Most tiles of bt rows that M rows of E experts make.
static inline int64_t most_tiles(int64_t M, int64_t E, int64_t bt) { return M / bt + (E < M ? E : M); }

// ---------------------------------------------------------------------------
// h and grad_x: the dense GEMM's tile on an expert's operands
// ---------------------------------------------------------------------------
// 2 rows N K operations against N K / 2 bytes of weights an expert: bound by
// the matrix units from some 100 rows an expert on.  Measured, r = 16, x 8 of
// 14336 x 4096 and 8192 rows (962 GFLOP): h 890-1030 us by card, grad_x 890-1050
// us, 0.92-1.08 PFLOP/s; one dense layer of these sizes takes 770-850 and
// 730-815 us on the same cards, the difference being the experts' ragged tiles.
// 64 of 1024 x 2048 and 6000 ragged rows (25 GFLOP, 104 MB): 47 us, of which 14
// go without any step of K (launch, finding the tile, first loads, epilogue)
// and 31 are a chain of LDS reads, dequantization and MFMA in tiles of mostly
// one expert's rows.
//
// Ragged tiles.  An expert's last tile has 1 .. 256 rows; its consumers take
// the least of 64, 128, 192 and 256 rows that holds them, all waves sharing
// whatever height it is (64 x 1024 x 2048: 56 us with heights of 128 and 256
// only, 49 with these; 16 x 4096 x 4096, 192 rows an expert: 116 and 104).  As
// a launch of their own the ragged tiles took as long (885 + 133 us against
// 1030), and a tile of 128 x 128 twice to a compute unit more (64 x 1024 x
// 2048: 62 us against 53 at that time; 8 x 14336 x 4096: 1267 against 1030).
//
// Few tiles run as K pieces, as in the dense layer: a piece to each of `slots`
// workgroups (0: no pieces), with at least 8 K steps.  How many tiles there are
// is only known here, so where there may be enough of them to go without, both
// kernels are launched, and one of them ends at once (a kernel that could do
// either would not have the registers).  8 x 4096 x 14336, 192 rows an expert:
// 333 us without pieces, 228 with them (207 with the heights above).
__device__ __forceinline__ int pieces_of(int tiles, int slots, int nk) {
  int p = slots / (tiles > 0 ? tiles : 1);
  p = p < 16 ? p : 16;
  p = p < nk / 8 ? p : nk / 8;
  return p > 1 ? p : 1;
}

template <bool kBwd, bool kPieces, bool kTail = false>
__global__ __launch_bounds__(lg2::kThreads) void experts_gemm_kernel(GemmArgs p, ExpertRows er, Nf4Table tab,
                                                                     int slots) {
  using T = lg2::Tile<kBwd>;
  __shared__ __align__(16) uint8_t sw0[T::W];
  __shared__ __align__(16) uint8_t sw1[T::W];
  __shared__ __align__(16) uint8_t sa0[lg2::ATILEB];
  __shared__ __align__(16) uint8_t sa1[lg2::ATILEB];
  __shared__ uint32_t lds_word;
  const lg2::Lds lds{{sw0, sw1}, {sa0, sa1}};
  const int tid = threadIdx.x;
  const int nk = (int)((p.K + lg2::BK - 1) / lg2::BK);
  // Row tiles are numbered through the experts, feature tiles fastest; each
  // XCD (workgroup number mod 8) takes a run of neighbouring tiles, of the
  // whole ones first and then of the ragged ones.  As pieces: workgroup
  // piece + pieces tile.
  const int bid = (int)blockIdx.x;
  int tile_f = 0, pieces = 1;
  Span s;
  const bool found = find_span_whole_first(er, lg2::BT, [&](int whole, int ragged) {
    const int first = whole * p.tiles_f, second = ragged * p.tiles_f;
    int item;
    pieces = pieces_of(first + second, slots, nk);
    if (kPieces != (pieces > 1)) return -1;
    if (kPieces) {
      item = bid / pieces;
      if (item >= first + second) return -1;
    } else {
      const int run = (first + 7) >> 3, run2 = (second + 7) >> 3;
      const int k = (bid >> 3) - run;
      if (k < 0) {
        item = (bid & 7) * run + (bid >> 3);
        if (item >= first) return -1;
      } else {
        item = (bid & 7) * run2 + k;
        if (k >= run2 || item >= second) return -1;
        item += first;
      }
    }
    tile_f = item % p.tiles_f;
    return item / p.tiles_f;
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
  pieces = kPieces ? __builtin_amdgcn_readfirstlane(pieces) : 1;
  tile_f = __builtin_amdgcn_readfirstlane(tile_f);
  const int piece = kPieces ? bid % pieces : 0;
  const int k0 = piece * nk / pieces, ks = (piece + 1) * nk / pieces - k0;
  const bool lora = piece == pieces - 1;
  const int64_t f0 = (int64_t)tile_f * lg2::BF;
  const int64_t t0 = (int64_t)s.tile * lg2::BT;
  const int64_t left = p.M - t0;
  if (tid >= 64 * lg2::kMfmaWaves)
    gemm_producer<kBwd>(p, tab, lds, tid - 64 * lg2::kMfmaWaves, f0, t0, k0, ks, lora, 0, &lds_word, skew);
  else if (left > 192)
    gemm_consumer<kBwd, kPieces, false, lg2::BT, true, kTail>(p, lds, tid, f0, t0, k0, ks, lora, 0, &lds_word);
  else if (left > 128)
    gemm_consumer<kBwd, kPieces, false, 192, true, kTail>(p, lds, tid, f0, t0, k0, ks, lora, 0, &lds_word);
  else if (left > 64)
    gemm_consumer<kBwd, kPieces, false, 128, true, kTail>(p, lds, tid, f0, t0, k0, ks, lora, 0, &lds_word);
  else
    gemm_consumer<kBwd, kPieces, false, 64, true, kTail>(p, lds, tid, f0, t0, k0, ks, lora, 0, &lds_word);
}

// Finishes tiles that ran as K pieces: out = bf16(piece 0 + piece 1 + ...), in
// the consumer's [wave][i][j][lane] order, 256 items of 4 features a workgroup.
template <bool kBwd, int kRows>
__device__ __forceinline__ void experts_pieces_tile(const GemmArgs& p, const Span& s, int tile, int rem) {
  constexpr int WF = WaveTile<kBwd, kRows>::F, WT = WaveTile<kBwd, kRows>::T;
  constexpr int NI = WF / 16, NJ = WT / 16;
  const int wave = rem / (NI * NJ * 64);
  const int ij = (rem / 64) % (NI * NJ);
  const int lane = rem % 64;
  const int i = ij / NJ, j = ij % NJ;
  const int64_t t = (int64_t)s.tile * lg2::BT + (wave / (lg2::BF / WF)) * WT + 16 * j + (lane & 15);
  const int64_t f = (int64_t)(tile % p.tiles_f) * lg2::BF + (wave % (lg2::BF / WF)) * WF + 16 * i + 4 * (lane >> 4);
  if (wave >= lg2::kMfmaWaves || t >= s.rows || f >= p.N) return;
  constexpr size_t kSlot = (size_t)lg2::BF * lg2::BT;
  const float* slot = p.piece_out + (size_t)tile * p.pieces * kSlot + (size_t)rem * 4;
  f32x4 v = *reinterpret_cast<const f32x4*>(slot);
  for (int q = 1; q < p.pieces; ++q) v += *reinterpret_cast<const f32x4*>(slot + (size_t)q * kSlot);
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

template <bool kBwd>
__global__ __launch_bounds__(256) void experts_pieces_kernel(GemmArgs p, ExpertRows er, int slots) {
  constexpr int kGroups = lg2::BF * lg2::BT / 4 / 256;
  const int tile = (int)blockIdx.x / kGroups;
  const int rem = ((int)blockIdx.x % kGroups) * 256 + (int)threadIdx.x;
  Span s;
  int pieces = 1;
  const bool found = find_span_whole_first(er, lg2::BT, [&](int whole, int ragged) {
    pieces = pieces_of((whole + ragged) * p.tiles_f, slots, (int)((p.K + lg2::BK - 1) / lg2::BK));
    return pieces > 1 ? tile / p.tiles_f : -1;
  }, s);
  if (!found) return;
  p.pieces = __builtin_amdgcn_readfirstlane(pieces);
  const int left = s.rows - s.tile * lg2::BT;
  if (left > 192)
    experts_pieces_tile<kBwd, 256>(p, s, tile, rem);
  else if (left > 128)
    experts_pieces_tile<kBwd, 192>(p, s, tile, rem);
  else if (left > 64)
    experts_pieces_tile<kBwd, 128>(p, s, tile, rem);
  else
    experts_pieces_tile<kBwd, 64>(p, s, tile, rem);
}

static int64_t gemm_tiles(int64_t M, int64_t E, int64_t N) { return most_tiles(M, E, lg2::BT) * cdiv(N, lg2::BF); }

// Fewer than 2^32 threads in a launch.
bool experts_gemm_fits(int64_t M, int64_t E, int64_t N) { return gemm_tiles(M, E, N) < ((int64_t)1 << 22); }

// Workgroups for K pieces: none where there will hardly be as few tiles as
// half the CUs (the bound counts a ragged tile to every expert), or where K is
// too short for two.
static int pieces_slots(int64_t M, int64_t E, int64_t N, int64_t K) {
  return gemm_tiles(M, E, N) <= device_cus() && cdiv(K, lg2::BK) >= 16 ? device_cus() : 0;
}

// Work items in pieces, at most: as many as slots, and 16 (or one for 8 K
// steps) to a tile.
static int64_t pieces_items(int64_t M, int64_t E, int64_t N, int64_t K) {
  const int64_t slots = pieces_slots(M, E, N, K), most = cdiv(K, lg2::BK) / 8;
  const int64_t all = gemm_tiles(M, E, N) * (most < 16 ? most : 16);
  return all < slots ? all : slots;
}

size_t experts_gemm_ws_bytes(int64_t M, int64_t E, int64_t N, int64_t K) {
  return (size_t)pieces_items(M, E, N, K) * lg2::BF * lg2::BT * sizeof(float);
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
  const int slots = pieces_slots(M, E, p.N, K);
  const dim3 block(lg2::kThreads);
  // the runs of whole and of ragged tiles are each rounded up to 8
  const int64_t wgs = cdiv(tiles, 8) * 8 + 8;
  const dim3 grid((unsigned)wgs);
  const bool tail = K % lg2::BK != 0;  // of the backward only: n is a multiple of 64
  if (!slots || 2 * tiles > slots) {
    if (tail)
      hipLaunchKernelGGL((experts_gemm_kernel<true, false, true>), grid, block, 0, stream, p, er, tab, slots);
    else if (bwd)
      hipLaunchKernelGGL((experts_gemm_kernel<true, false>), grid, block, 0, stream, p, er, tab, slots);
    else
      hipLaunchKernelGGL((experts_gemm_kernel<false, false>), grid, block, 0, stream, p, er, tab, slots);
  }
  if (!slots) return;
  p.piece_out = static_cast<float*>(ws);
  // at most half the slots in tiles
  const dim3 pgrid((unsigned)pieces_items(M, E, p.N, K));
  const dim3 rgrid((unsigned)((tiles < slots / 2 ? tiles : slots / 2) * (lg2::BF * lg2::BT / 4 / 256)));
  if (bwd) {
    if (tail)
      hipLaunchKernelGGL((experts_gemm_kernel<true, true, true>), pgrid, block, 0, stream, p, er, tab, slots);
    else
      hipLaunchKernelGGL((experts_gemm_kernel<true, true>), pgrid, block, 0, stream, p, er, tab, slots);
    hipLaunchKernelGGL(experts_pieces_kernel<true>, rgrid, dim3(256), 0, stream, p, er, slots);
  } else {
    hipLaunchKernelGGL((experts_gemm_kernel<false, true>), pgrid, block, 0, stream, p, er, tab, slots);
    hipLaunchKernelGGL(experts_pieces_kernel<false>, rgrid, dim3(256), 0, stream, p, er, slots);
  }
}

// s u (or s v) of row `row` (none past `rows`), ranks q .. q + 7, as bf16 hi + lo; the
// partials are summed in order, and the sum goes to u_out.
__device__ __forceinline__ void lora_rows(const float* part, int splits, int64_t stride, int64_t row, bool ok, int R,
                                          int q, float s, float* u_out, u32x4& hi, u32x4& lo) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  const int have = ok ? R - q : 0;
  const float* src = part + row * R + q;
  if (have >= 8 && (R & 3) == 0) {
    for (int k = 0; k < splits; ++k, src += stride) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(src), b = *reinterpret_cast<const f32x4*>(src + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += a[i];
        v[i + 4] += b[i];
      }
    }
  } else if (have > 0) {
    for (int k = 0; k < splits; ++k, src += stride) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < have) v[i] += src[i];
    }
  }
  if (u_out) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < have) u_out[row * R + q + i] = v[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float h0, l0, h1, l1;
    split_bf16(s * v[2 * i], h0, l0);
    split_bf16(s * v[2 * i + 1], h1, l1);
    hi[i] = pack_bf16x2(h0, h1);
    lo[i] = pack_bf16x2(l0, l1);
  }
}

// ---------------------------------------------------------------------------
// h where experts have few rows: weights straight into MFMA operands
// ---------------------------------------------------------------------------
// Every weight is read for a few rows, so the codes' bytes bound it.  A wave
// takes 32 features, dequantizes a code's 8 weights right where the MFMA wants
// them (a lane holds one 64-weight block of one feature, so one scale and one
// table serve it for 8 MFMA steps) and never writes weights to LDS; only x goes
// through it, shared by the workgroup's 128 features.  8 x 14336 x 4096 (235 MB
// of codes, 16 rows): 64-65 us, 3.6 TB/s; the codes' loads alone take 54 us
// (4.4 TB/s), with x and the barriers 59.  Loads arranged to 64 contiguous
// bytes a row and swapped between lanes took 69 us, non-temporal loads 67.  All
// workgroups are resident and end together, and lora_rows then adds u's K splits
// (8 here) one trip to memory after the other, behind B's loads: nothing hides
// these.
//
// Whole calls, us, tiles of 16 rows / tiles of 32 / the GEMM, by rows an expert
// (r = 16):
//                            16               32               48
//    8 x 14336 x 4096    67  74 109      102  77 107     152 118 107
//    8 x 4096 x 14336    64  69 119      108  80 123     154 136 127
//   16 x 4096 x 4096     38  42  60       63  45  60      87  72  60
//   64 x 1024 x 2048     25  28  38       38  30  38      52  44  39
// so tiles of 16 rows up to 16 rows an expert on average, of 32 up to 32, then
// the GEMM.  Tiles of 64 and 128 rows were no better than it anywhere above.
// The average is what the host knows.  All rows in k of the experts, forward
// calls, us, balanced / k of them hold all rows / a call of those k alone:
//    64 x 1024 x 2048, 2048 rows (32 on average): 32 /  k 2  31 /  40,  k 8  29 /  41
//    the same, 2560 rows (40, the GEMM):          40 /  k 2  59 /  43,  k 8  57 /  43
//    8 x 14336 x 4096, 256 rows (32):             78 /  k 1  73 /  60,  k 2  72 /  61
//    the same, 320 rows (40, the GEMM):          111 /  k 1  97 /  75,  k 2  80 /  72
//    1024 x 4096 x 512, 32000 rows (31):         747 /  k 8 651 / 164,  k 64 672 / 174
//    the same, 40000 rows (39, the GEMM):       1158 /  k 8 642 / 209,  k 64 655 / 225
// so a skew costs little at 64 experts, and up to four times at 1024, on both
// sides of the rule: streamed, busy experts' weights are read for every 32 rows;
// in the GEMM, workgroups are launched for the other experts' tiles.
struct StreamArgs {
  const uint16_t* x;        // M x K
  const uint8_t* codes;
  const uint8_t* absmax8;
  const float* c2;
  const uint16_t* B;        // E x N x R
  const float* u;           // usplits x M x R partials of u
  int usplits;
  float* u_out;             // M x R or null
  uint16_t* h;              // M x N
  float* part;              // ksplits x M x N, used with ksplits > 1
  int ksplits;
  int64_t K, N;
  int R;
  float s;
  int groups;               // feature groups
};

// TB: blocks of 16 rows in a tile.
template <int TB>
__global__ __launch_bounds__(256, 4) void experts_stream_kernel(StreamArgs p, ExpertRows er, Nf4Table tab) {
  constexpr int NW = 4;                  // waves
  constexpr int NF = 2;                  // blocks of 16 features of a wave
  constexpr int BT = 16 * TB;
  constexpr int STAGE = BT * 512;        // 256 k of each row
  constexpr int XL = TB * 8 / NW;        // 1 KB loads of x per wave and stage
  constexpr int CL = 4 * NF;             // loads of a piece of codes
  static_assert(TB * 8 % NW == 0, "loads of x");
  __shared__ __align__(16) uint8_t s0[STAGE];
  __shared__ __align__(16) uint8_t s1[STAGE];
  uint8_t* const buf[2] = {s0, s1};
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15;
  const int g = lane >> 4;
  // items: expert, feature group, row tile (fastest), so that the tiles that
  // read the same weights follow each other; a run of them to each XCD
  int item = 0;
  Span sp;
  const bool found = find_span(er, BT, [&](int total) {
    const int items = total * p.groups;
    const int run = (items + 7) >> 3;
    item = ((int)blockIdx.x & 7) * run + ((int)blockIdx.x >> 3);
    return ((int)blockIdx.x >> 3) < run && item < items ? item / p.groups : -1;
  }, sp);
  if (!found) return;
  const int local = item - (item / p.groups - sp.tile) * p.groups;  // among the expert's items
  const int fg = local / sp.tiles;
  const int tile = local % sp.tiles;
  const int split = (int)blockIdx.y;
  const int64_t K = p.K;
  const int pieces = (int)cdiv(K, 256);
  const int pb = split * pieces / p.ksplits, pe = (split + 1) * pieces / p.ksplits;
  const int nst = pe - pb;
  const int t0 = tile * BT;

  const int64_t cells = p.N * K;
  const int64_t block0 = sp.e * (cells / kBlock);
  const uint32_t skew = (uint32_t)(block0 % kGroupBlocks);
  const uint32_t cbytes = (uint32_t)(cells / 2), abytes = (uint32_t)(cells / kBlock);
  const uint32_t xbytes = (uint32_t)(sp.rows * K * 2);
  const brsrc_t rx = make_rsrc(p.x + sp.row0 * K, xbytes);
  const brsrc_t rc = make_rsrc(p.codes + sp.e * (cells / 2), cbytes);
  const brsrc_t ra = make_rsrc(p.absmax8 + block0, abytes);
  const brsrc_t rs = make_rsrc(p.c2 + block0 / kGroupBlocks, (abytes + skew + kGroupBlocks - 1) / kGroupBlocks * 4);

  // x: a 1 KB load holds 2 rows of 256 k.  The 16-byte chunk of k = 64 g + 8 q
  // sits at 16 (g % 2) + ((8 (g / 2) + q) ^ (t % 16)) of row t: a 16-byte read
  // serves half of lane group g's rows together with the other half of group
  // g + 1's, which then take different banks.
  auto issue_x = [&](int s, uint8_t* stg) {
#pragma unroll
    for (int b = 0; b < XL; ++b) {
      const int blk = wave * XL + b;
      const int row = 2 * blk + (lane >> 5);
      const int c = (lane & 31) ^ (row & 15);  // slot -> 16 (g % 2) + 8 (g / 2) + q
      const int64_t k = (int64_t)(pb + s) * 256 + 64 * ((c >> 4) | ((c >> 2) & 2)) + 8 * (c & 7);
      const bool live = s < nst && k < K && t0 + row < sp.rows;
      dma16(rx, stg + blk * 1024, live ? (uint32_t)(((t0 + row) * K + k) * 2) : xbytes);
    }
  };
  // codes: a lane takes one 64-weight block of feature row lr for each of the
  // wave's two 16-feature blocks and piece of 256 k: k = 64 g .. 64 g + 63.
  // MFMA step q then pairs k = 64 g + 8 q .. + 7 of both operands.
  const int64_t f0 = (int64_t)fg * (16 * NF * NW) + 16 * NF * wave;
  const uint32_t cbase = (uint32_t)(((f0 + lr) * K + (int64_t)pb * 256 + 64 * g) / 2);
  const uint32_t crow = (uint32_t)(16 * K / 2);
  struct Piece {
    u32x4 c[NF][2];
    uint32_t a[NF];
    float s[NF];
  };
  auto load = [&](int s, Piece& P) {
#pragma unroll
    for (int b = 0; b < NF; ++b) {
      const uint32_t off = s < nst ? cbase + b * crow + (uint32_t)s * 128 : cbytes;
      P.c[b][0] = bload128(rc, off);
      P.c[b][1] = bload128(rc, off + 16);
      const uint32_t blk = off / (kBlock / 2);
      P.a[b] = bload8(ra, blk);
      P.s[b] = __uint_as_float(bload32(rs, ((blk + skew) >> 8) << 2));
    }
  };
  f32x4 acc[NF][TB];
#pragma unroll
  for (int b = 0; b < NF; ++b)
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the reads of x run one MFMA step ahead
  auto compute = [&](const uint8_t* stg, const Piece& P) {
    u32x4 xf[2][TB];
    auto read = [&](int q) {
#pragma unroll
      for (int t = 0; t < TB; ++t)
        xf[q & 1][t] = *reinterpret_cast<const u32x4*>(stg + (16 * t + lr) * 512 + (g & 1) * 256 +
                                                       (((8 * (g >> 1) + q) ^ lr) << 4));
    };
    read(0);
    MagLut L[NF];
#pragma unroll
    for (int b = 0; b < NF; ++b) L[b] = make_mag_lut(tab, e4m3_decode(P.a[b]) * P.s[b]);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q < 7) read(q + 1);
      if (TB > 1) __builtin_amdgcn_sched_barrier(0);
      u32x4 w[NF];
#pragma unroll
      for (int b = 0; b < NF; ++b) {
        uint32_t o[4];
        mag_dequant8(L[b], P.c[b][q >> 2][q & 3], o);
        w[b] = u32x4{o[0], o[1], o[2], o[3]};
      }
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < NF; ++b) acc[b][t] = mfma16x16x32(w[b], xf[q & 1][t], acc[b][t]);
    }
  };
  // Two stages of x and two pieces of codes: while one is multiplied the next
  // is on its way.  A step begins when the wave's loads of its x have landed
  // (loads complete in order and only the piece's codes were issued after them;
  // the empty asm keeps the order of issue) and all waves have read the stage
  // before, which is then loaded anew.  Steps past the end load nothing.
  auto fence = []() { asm volatile("" ::: "memory"); };
  Piece P[2];
  issue_x(0, buf[0]);
  fence();
  load(0, P[0]);
  fence();
  auto step = [&](int s, int u) {
    wait_vmcnt_lds<CL>();
    ring_barrier();
    issue_x(s + 1, buf[u ^ 1]);
    fence();
    load(s + 1, P[u ^ 1]);
    fence();
    compute(buf[u], P[u]);
  };
  int st = 0;
  for (; st + 1 < nst; st += 2) {
    step(st, 0);
    step(st + 1, 1);
  }
  if (st < nst) step(st, 0);
  wait_vmcnt<0>();

  // lane holds features f0 + 16 b + 4 g + e of row t0 + 16 t + lr.  The LoRA
  // term, in the first K split: ranks 32 at a time, s u as bf16 hi + lo.
  const int R = p.R;
  if (split == 0) {
    const uint16_t* B = p.B + sp.e * (p.N * R);
    for (int q0 = 0; q0 < R; q0 += 32) {
      u32x4 w[NF];
#pragma unroll
      for (int b = 0; b < NF; ++b) {
        const int64_t f = f0 + 16 * b + lr;
        const int q = q0 + 8 * g;
        if (f < p.N && (R & 7) == 0 && q + 8 <= R) {
          w[b] = *reinterpret_cast<const u32x4*>(B + f * R + q);
        } else {
          w[b] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (f < p.N && q + i < R) w[b][i >> 1] |= (uint32_t)B[f * R + q + i] << (16 * (i & 1));
        }
      }
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int row = t0 + 16 * t + lr;
        u32x4 hi, lo;
        lora_rows(p.u, p.usplits, (int64_t)er.M * R, sp.row0 + row, row < sp.rows, R, q0 + 8 * g, p.s,
                  fg == 0 && wave == 0 ? p.u_out : nullptr, hi, lo);
#pragma unroll
        for (int b = 0; b < NF; ++b) {
          acc[b][t] = mfma16x16x32(w[b], hi, acc[b][t]);
          acc[b][t] = mfma16x16x32(w[b], lo, acc[b][t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int row = t0 + 16 * t + lr;
    if (row >= sp.rows) continue;
#pragma unroll
    for (int b = 0; b < NF; ++b) {
      const int64_t f = f0 + 16 * b + 4 * g;
      if (f >= p.N) continue;
      const f32x4 v = acc[b][t];
      const int64_t o = (int64_t)(sp.row0 + row) * p.N + f;
      if (p.ksplits > 1) {
        float* dst = p.part + (int64_t)split * er.M * p.N + o;
        if ((p.N & 3) == 0) {
          *reinterpret_cast<f32x4*>(dst) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (f + e < p.N) dst[e] = v[e];
        }
      } else {
        const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if ((p.N & 3) == 0) {
          *reinterpret_cast<u32x2*>(p.h + o) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (f + e < p.N) p.h[o + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
}

// h = bf16(sum of the K splits, in order), 4 values a thread, for the rows that belong to an
// expert.
__global__ __launch_bounds__(256) void experts_stream_sum_kernel(StreamArgs p, ExpertRows er) {
  int low, top;
  live_rows(er, low, top);
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int64_t end = (int64_t)top * p.N;
  if (i + 4 <= (int64_t)low * p.N || i >= end) return;
  const int64_t stride = (int64_t)er.M * p.N;
  const int64_t from = (int64_t)low * p.N;
  if (i >= from && i + 4 <= end && (stride & 3) == 0) {
    f32x4 v = *reinterpret_cast<const f32x4*>(p.part + i);
    for (int k = 1; k < p.ksplits; ++k) v += *reinterpret_cast<const f32x4*>(p.part + k * stride + i);
    *reinterpret_cast<u32x2*>(p.h + i) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    return;
  }
  for (int e = 0; e < 4; ++e) {
    if (i + e < from || i + e >= end) continue;
    float v = p.part[i + e];
    for (int k = 1; k < p.ksplits; ++k) v += p.part[k * stride + i + e];
    p.h[i + e] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  }
}

// Features go to workgroups of 4 waves, 32 a wave; K is split where the
// workgroups would not fill the compute units four times, each split at least
// two pieces of 256.
struct StreamPlan {
  int tb;       // 16-row blocks of a tile, 0: the GEMM takes the call
  int groups;   // of 128 features
  int ksplits;
};

constexpr int kStreamWaves = 4;

static StreamPlan stream_plan(int64_t M, int64_t E, int64_t N, int64_t K) {
  const int64_t rows = cdiv(M, E < M ? E : M);  // of an expert, if all have as many
  StreamPlan s{};
  s.tb = rows <= 16 ? 1 : rows <= 32 ? 2 : 0;
  s.ksplits = 1;
  if (!s.tb) return s;
  s.groups = (int)cdiv(N, 32 * kStreamWaves);
  const int64_t items = most_tiles(M, E, 16 * s.tb) * s.groups;
  int64_t ks = 4 * (int64_t)device_cus() / items;
  const int64_t most = cdiv(K, 256) / 2;
  ks = ks > most ? most : ks;
  ks = ks > 8 ? 8 : ks;
  s.ksplits = ks < 1 ? 1 : (int)ks;
  return s;
}

size_t experts_stream_ws_bytes(int64_t M, int64_t E, int64_t N, int64_t K) {
  const StreamPlan s = stream_plan(M, E, N, K);
  return s.tb && s.ksplits > 1 ? (size_t)s.ksplits * M * N * sizeof(float) : 0;
}
bool experts_stream_takes(int64_t M, int64_t E, int64_t N, int64_t K) { return stream_plan(M, E, N, K).tb != 0; }

void launch_experts_stream(const int32_t* offsets, int64_t E, const uint16_t* x, const uint8_t* codes,
                           const uint8_t* absmax8, const float* c2, const uint16_t* B, const float* u, int usplits,
                           float* u_out, uint16_t* h, int64_t M, int64_t n, int64_t m, int r, float s, void* ws,
                           const Nf4Table& tab, hipStream_t stream) {
  const StreamPlan plan = stream_plan(M, E, m, n);
  const StreamArgs p{x,     codes, absmax8, c2, B, u, usplits, u_out, h, static_cast<float*>(ws), plan.ksplits,
                     n,     m,     r,       s,  plan.groups};
  const ExpertRows er{offsets, (int)E, (int)M};
  const int64_t items = most_tiles(M, E, 16 * plan.tb) * plan.groups;
  const dim3 grid((unsigned)(cdiv(items, 8) * 8), (unsigned)plan.ksplits), block(64 * kStreamWaves);
  if (plan.tb == 1)
    hipLaunchKernelGGL((experts_stream_kernel<1>), grid, block, 0, stream, p, er, tab);
  else
    hipLaunchKernelGGL((experts_stream_kernel<2>), grid, block, 0, stream, p, er, tab);
  if (plan.ksplits > 1)
    hipLaunchKernelGGL(experts_stream_sum_kernel, dim3((unsigned)cdiv(M * m, 1024)), dim3(256), 0, stream, p, er);
}

// ---------------------------------------------------------------------------
// u = x A_e^T and v = g B_e
// ---------------------------------------------------------------------------
// One read of x or g, which bounds it; the dense layer's tile of 128 rows on
// an expert's rows.  K is split until there is a workgroup to each compute
// unit, and experts_factor_kernel adds the splits in order.  8192 rows, r = 16:
// u of 4096 columns 16 us (67 MB, 4.2 TB/s), v of 14336 columns 46 us (235 MB,
// 5.1 TB/s; with splits for two workgroups to a unit 56, for half of them 58);
// 4096 rows of 8192 columns, r = 64: 22 us (3.0 TB/s).

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
  int64_t want = device_cus() / most_tiles(M, E, sk::DT);  // one round, a workgroup to a compute unit
  const int64_t most = cdiv(K, 512);
  if (want > most) want = most;
  if (want > 64) want = 64;
  if (want < 1) want = 1;
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

// What the kernels cannot read as it stands, in one launch: rows of g whose
// length is not a multiple of 8, copied to rows of ld = m rounded up to 64 with
// zeros behind; and B_e^T (R x ld, zeros from column m on) of every expert, for
// ranks whose rows of B are not whole 16-byte pieces.  Either may be null.
__global__ __launch_bounds__(256) void experts_prepare_kernel(const uint16_t* __restrict__ g, int64_t gcount,
                                                              uint16_t* __restrict__ gout,
                                                              const uint16_t* __restrict__ B, int64_t bcount,
                                                              uint16_t* __restrict__ bout, int64_t m, int R,
                                                              int64_t ld, int64_t gblocks) {
  if ((int64_t)blockIdx.x < gblocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // over M x ld
    if (i >= gcount) return;
    const int64_t t = i / ld, f = i % ld;
    gout[i] = f < m ? g[t * m + f] : (uint16_t)0;
  } else {
    int64_t i = ((int64_t)blockIdx.x - gblocks) * 256 + threadIdx.x;  // over E x R x ld
    for (; i < bcount; i += ((int64_t)gridDim.x - gblocks) * 256) {
      const int64_t f = i % ld, eq = i / ld;
      const int64_t e = eq / R, q = eq % R;
      bout[i] = f < m ? B[(e * m + f) * R + q] : (uint16_t)0;
    }
  }
}

void launch_experts_prepare(const uint16_t* g, uint16_t* gout, const uint16_t* B, uint16_t* bout, int64_t M, int64_t E,
                            int64_t m, int R, int64_t ld, hipStream_t stream) {
  const int64_t gcount = gout ? M * ld : 0, bcount = bout ? E * R * ld : 0;
  const int64_t gblocks = cdiv(gcount, 256), bblocks = cdiv(bcount, 256);  // gcount < 2^30
  const int64_t blocks = gblocks + (bblocks < (1 << 20) ? bblocks : 1 << 20);
  if (blocks)
    hipLaunchKernelGGL(experts_prepare_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, g, gcount, gout, B, bcount,
                       bout, m, R, ld, gblocks);
}

// Sums the splits of u or v in order: fp32 out (may be null) and, for the
// products over rows, bf16 hi and lo planes [M][16 RB] with zero ranks from R
// on (planes may be null).  Rows outside every expert are left alone.  8192
// rows of 16 ranks, 3 splits: 4-5 us, its launch and one trip to memory.
__global__ __launch_bounds__(256) void experts_factor_kernel(FactorJob a, FactorJob b, ExpertRows er, int R, int RP) {
  const FactorJob j = blockIdx.y ? b : a;
  const int i = (int)(blockIdx.x * 256 + threadIdx.x);  // rank pairs of all rows (fewer than 2^29)
  const int row = i / (RP / 2);
  const int q = i % (RP / 2) * 2;
  int low, top;
  live_rows(er, low, top);
  if (row < low || row >= top) return;
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
// adds in order (it also writes the zeros of experts without rows; where no
// expert can have two chunks, it is not needed).  Bound by the read of x and
// g.  Both products in one launch, 8192 rows of 4096 and 14336 columns, r = 16:
// 56 us and 5 us for the sums (302 MB, 5.0 TB/s); 4096 rows of 28672 and 8192
// columns, r = 64: 70 us and 8 us (3.9 TB/s).
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
  int single;          // every expert's rows are one chunk: a row of workgroups to each expert, also to those
                       // without rows, whose zeros they write
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

template <int RB, int NS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void experts_token_kernel(TokenArgs a) {
  constexpr int ROW = 64 * WAVES;        // bytes of a row of the stage: 32 columns a wave
  constexpr int XB = sk::TS * ROW;       // 64 rows
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
  if (a.single) {
    sp = expert_span(a.er, job.chunk, bid / job.tiles);
    sp.tiles = 1;
  } else if (!find_span(a.er, job.chunk, [&](int) { return bid / job.tiles; }, sp)) {
    return;
  }
  const int R = a.R;
  const int64_t J = job.J, ld = job.ld;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15;
  const int lq = lane >> 4;
  const int64_t j0 = (int64_t)(bid % job.tiles) * (32 * WAVES);
  const int tbeg = sp.tile * job.chunk;
  const int tend = tbeg + job.chunk < sp.rows ? tbeg + job.chunk : sp.rows;
  const int nst = (tend - tbeg + sk::TS - 1) / sk::TS;
  const uint32_t xbytes = (uint32_t)(sp.rows * ld * 2);
  // both planes behind one buffer: fewer than 2^22 rows of 256 bytes at most
  const uint32_t plane = (uint32_t)a.er.M * (32u * RB);
  const uint32_t pbytes = plane + (uint32_t)sp.rows * (32u * RB);
  const brsrc_t rx = make_rsrc(job.X + sp.row0 * ld, xbytes);
  const brsrc_t rp = make_rsrc(job.P + (int64_t)sp.row0 * (16 * RB), pbytes);
  constexpr int XR = 16 / WAVES;         // rows of a 1 KB load
  const int xrow = lane / (4 * WAVES);
  const int slot = lane % (4 * WAVES);
  static_assert(4 * RB % WAVES == 0, "blocks of the planes");
  constexpr int PL = 4 * RB / WAVES;     // loads of the planes per wave
  constexpr int LMIN = 4 + PL;
  auto issue = [&](int s, uint8_t* stg) {
    const int tb = tbeg + s * sk::TS;
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // XR rows a load; 32-byte unit u of a row at u ^ f, as in swtg
      const int blk = 4 * wave + b;
      const int row = XR * blk + xrow;
      const int f = (row & 3) | (((row >> 3) & 1) << 2);
      const int c = ((((slot >> 1) ^ f)) << 1) | (slot & 1);
      const int64_t j = j0 + 8 * c;
      dma16(rx, stg + blk * 1024, (tb + row < tend && j < ld) ? (uint32_t)(((tb + row) * ld + j) * 2) : xbytes);
    }
#pragma unroll
    for (int b = 0; b < PL; ++b) {  // 1 KB blocks of the two planes (2 RB blocks each)
      const int id = WAVES * b + wave;
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
  auto xat = [](int t, int c) -> uint32_t {
    const int f = (t & 3) | (((t >> 3) & 1) << 2);
    return (uint32_t)(t * ROW + (((c >> 1) ^ f) << 5) + ((c & 1) << 4));
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
        x[ib] = read_tr(stg + xat(t, c) + (tr_c & 1) * 8, stg + xat(t + 4, c) + (tr_c & 1) * 8);
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

constexpr int kSumCells = 1024;  // of a workgroup, 4 a thread

__global__ __launch_bounds__(256) void experts_sum_kernel(TokenArgs a) {
  const TokenJob& job = a.job[blockIdx.z];
  const int64_t cells = job.J * a.R;
  const int64_t i = (int64_t)blockIdx.x * kSumCells + 4 * (int)threadIdx.x;
  if ((int64_t)blockIdx.x * kSumCells >= cells) return;
  const Span sp = expert_span(a.er, job.chunk, (int)blockIdx.y);
  if (sp.tiles == 1 || i >= cells) return;
  uint16_t* out = job.out + sp.e * cells + i;
  const float* part = job.part + sp.slot * cells + i;
  if ((cells & 3) == 0) {
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < sp.tiles; k += 4) {
      f32x4 w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)  // the loads go out together; what is past the end is loaded again and not added
        w[x] = *reinterpret_cast<const f32x4*>(part + (k + x < sp.tiles ? k + x : k) * cells);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (k + x < sp.tiles) s += w[x];
    }
    *reinterpret_cast<u32x2*>(out) =
        u32x2{pack_bf16x2(a.s * s[0], a.s * s[1]), pack_bf16x2(a.s * s[2], a.s * s[3])};
    return;
  }
  for (int e = 0; e < 4 && i + e < cells; ++e) {
    float s = 0.0f;
    for (int k = 0; k < sp.tiles; ++k) s += part[k * cells + e];
    out[e] = (uint16_t)(pack_bf16x2(a.s * s, 0.0f) & 0xFFFFu);
  }
}

// Waves of a workgroup, 32 columns each: at 64 ranks, where the planes of a
// stage are as large as 128 columns of it, 8.
static int token_waves(int R) { return rank_blocks(R) == 4 ? 8 : 4; }

// Rows of a chunk: a workgroup to each compute unit, if all experts had whole
// chunks, but no fewer than 256 rows, below which the sums weigh as much as
// the rows.  4 x 8192 x 28672, 4096 rows, 64 ranks: 70 us and 8 us for the
// sums, with chunks of half 81 and 15, of a third 91 and 17; 8 x 14336 x 4096,
// 8192 rows, 16 ranks: 56 us, half 59, a third 58, 5 us for the sums each.
static int token_chunk(int64_t M, int64_t J, int R) {
  const int64_t c = cdiv(cdiv(M * cdiv(J, 32 * token_waves(R)), device_cus()), 64) * 64;
  return (int)(c < 256 ? 256 : c);
}

// Experts of more than one chunk have fewer than 2 M / chunk chunks in all.
size_t experts_token_ws_bytes(int64_t M, int64_t J, int R) {
  return (size_t)(2 * M / token_chunk(M, J, R)) * J * R * sizeof(float);
}

// Fewer than 2^32 threads in the launches of the products (two jobs, 512 threads at most) and of their sums.
bool experts_token_fits(int64_t M, int64_t E, int64_t J) {
  return (M / 256 + E) * cdiv(J, 128) < ((int64_t)1 << 22) && J < ((int64_t)1 << 27);
}

void launch_experts_token(const uint16_t* x, const uint16_t* vplanes, uint16_t* grad_A, float* part_a,
                          const uint16_t* g, int64_t g_ld, const uint16_t* uplanes, uint16_t* grad_B, float* part_b,
                          const int32_t* offsets, int64_t M, int64_t E, int64_t n, int64_t m, int R, float s,
                          hipStream_t stream) {
  TokenArgs a{};
  const int tj = 32 * token_waves(R);
  a.job[0] = TokenJob{x, n, n, vplanes, grad_A, part_a, (int)cdiv(n, tj), token_chunk(M, n, R), true};
  a.job[1] = TokenJob{g, m, g_ld, uplanes, grad_B, part_b, (int)cdiv(m, tj), token_chunk(M, m, R), false};
  a.er = ExpertRows{offsets, (int)E, (int)M};
  a.R = R;
  a.s = s;
  a.single = M <= a.job[0].chunk && M <= a.job[1].chunk;
  auto wgs = [&](const TokenJob& j) { return (a.single ? E : most_tiles(M, E, j.chunk)) * j.tiles; };
  a.first = (int)wgs(a.job[0]);
  const dim3 grid((unsigned)(a.first + wgs(a.job[1])));
  switch (rank_blocks(R)) {
    case 1: hipLaunchKernelGGL((experts_token_kernel<1, 3, 4>), grid, dim3(256), 0, stream, a); break;
    case 2: hipLaunchKernelGGL((experts_token_kernel<2, 3, 4>), grid, dim3(256), 0, stream, a); break;
    case 4: hipLaunchKernelGGL((experts_token_kernel<4, 3, 8>), grid, dim3(512), 0, stream, a); break;
    default: hipLaunchKernelGGL((experts_token_kernel<8, 3, 4>), grid, dim3(256), 0, stream, a); break;
  }
  if (a.single) return;
  const int64_t most = (n > m ? n : m) * R;
  hipLaunchKernelGGL(experts_sum_kernel, dim3((unsigned)cdiv(most, kSumCells), (unsigned)E, 2), dim3(256), 0, stream,
                     a);
}

}  // namespace qlora
