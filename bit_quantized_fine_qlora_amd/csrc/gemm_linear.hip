// The two large-token GEMMs of the adapted linear layer (the tile itself is in
// gemm_tile.h): work items, the K split of few tiles and of a short last
// round, and the launches.
//   forward   h      = x W'^T + s u B^T   (K = n, output features = rows of W0)
//   backward  grad_x = g W'   + s v A     (K = m, output features = columns of W0)
#include "gemm_tile.h"

namespace qlora {

// kPieces: few-tile mode (every tile as p.pieces K pieces), a separate
// instantiation so that the other kernels' register allocation is untouched;
// kTail (K not a multiple of 64) likewise.
template <bool kBwd, bool kPieces, bool kSkip, bool kTail = false>
__global__ __launch_bounds__(lg2::kThreads) void linear_gemm_kernel(GemmArgs p, Nf4Table tab) {
  using T = lg2::Tile<kBwd>;
  __shared__ __align__(16) uint8_t sw0[T::W];
  __shared__ __align__(16) uint8_t sw1[T::W];
  __shared__ __align__(16) uint8_t sa0[lg2::ATILEB];
  __shared__ __align__(16) uint8_t sa1[lg2::ATILEB];
  __shared__ uint32_t lds_word;
  const lg2::Lds lds{{sw0, sw1}, {sa0, sa1}};
  const int tid = threadIdx.x;
  const int nk = (int)((p.K + lg2::BK - 1) / lg2::BK);
  // work item -> tile and K range: full tiles first (XCD-aware order), then
  // the K halves of the split tiles, which run in the last round
  int tile, k0 = 0, ks = nk, split = 0;
  bool lora = true;
  if (kPieces) {
    const int piece = (int)blockIdx.x % p.pieces;
    tile = (int)blockIdx.x / p.pieces;
    k0 = piece * nk / p.pieces;
    ks = (piece + 1) * nk / p.pieces - k0;
    lora = piece == p.pieces - 1;
  } else if ((int)blockIdx.x < p.full_tiles) {
    tile = xcd_remap_l(blockIdx.x, p.full_tiles);
  } else {
    const int w = (int)blockIdx.x - p.full_tiles;
    const int half = w & 1;
    tile = p.full_tiles + (w >> 1);
    split = (w >> 1) + 1;
    k0 = half ? nk / 2 : 0;
    ks = half ? nk - nk / 2 : nk / 2;
    lora = half != 0;
  }
  const int tile_f = tile % p.tiles_f;
  const int tile_t = tile / p.tiles_f;
  const int64_t f0 = (int64_t)tile_f * lg2::BF;
  const int64_t t0 = (int64_t)tile_t * lg2::BT;
  // wave-uniform role split; both roles pass the same number of barriers
  if (tid >= 64 * lg2::kMfmaWaves)
    gemm_producer<kBwd>(p, tab, lds, tid - 64 * lg2::kMfmaWaves, f0, t0, k0, ks, lora, split, &lds_word);
  else
    gemm_consumer<kBwd, kPieces, kSkip, lg2::BT, false, kTail>(p, lds, tid, f0, t0, k0, ks, lora, split, &lds_word);
}

__global__ void zero_u32_kernel(uint32_t* p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0u;
}

// Compute units of the current device (256 when no device answers).
int device_cus() {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (!cached[dev]) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cached[dev] = v;
  }
  return cached[dev];
}

// Few tiles (at most half the CUs, e.g. 33..256 tokens at 4096 - 14336
// features): every tile runs as P K pieces, P = min(CUs / tiles, 16) with
// at least 8 K steps per piece, so up to all CUs stream the weight.  With
// P >= 3 the P fp32 tile sums (tiles P 2^18 <= CUs 2^18 bytes) are added in
// piece order by a separate pass, so the result does not depend on which
// piece ends first.  With P = 2 the two halves meet through the K-split
// hand-off instead (commutative, so also order-free): no second pass, and
// half the fp32 traffic (the 70B block's k and v forwards: 128 tiles).
constexpr int kMaxPieces = 16;
static int64_t tiles_of(int64_t M, int64_t N) { return ((N + lg2::BF - 1) / lg2::BF) * ((M + lg2::BT - 1) / lg2::BT); }
static int few_tile_pieces(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = tiles_of(M, N);
  const int cus = device_cus();
  const int64_t nk = (K + lg2::BK - 1) / lg2::BK;
  if (tiles * 2 > cus) return 1;
  int64_t pc = cus / tiles;
  if (pc > kMaxPieces) pc = kMaxPieces;
  while (pc > 1 && nk / pc < 8) --pc;
  return (int)pc;
}
int gemm_pieces(int64_t M, int64_t N, int64_t K) {
  const int pc = few_tile_pieces(M, N, K);
  return pc == 2 ? 1 : pc;
}

// Tiles split in two K halves that meet through the hand-off: every tile
// when the few-tile mode would use two pieces; otherwise, when the tile
// count leaves at most half a round for the last pass, those last tiles:
// with T tiles on C CUs (one workgroup per CU), the last T mod C <= C/2
// tiles become 2 (T mod C) half-length work items, so the last round fills
// the chip for half the time instead of half the chip for the full time.
// Either way the two halves of a tile run in the same round.
int gemm_split_tiles(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = tiles_of(M, N);
  const int cus = device_cus();
  const int64_t rem = tiles % cus;
  const int64_t nk = (K + lg2::BK - 1) / lg2::BK;
  if (nk < 8) return 0;
  if (tiles * 2 <= cus) return few_tile_pieces(M, N, K) == 2 ? (int)tiles : 0;
  if (tiles < cus || rem == 0 || rem > cus / 2) return 0;
  return (int)rem;
}

// Finishes a few-tile GEMM: out = bf16(((piece 0 + piece 1) + ...) + add).
// Thread g takes fragment item g % 16384 (4 features of one token) of tile
// g / 16384 from every piece's slot, in the consumer's [wave][i][j][lane]
// order, so that the slot reads are whole 1 KB rows.
template <bool kBwd>
__global__ __launch_bounds__(256) void reduce_pieces_kernel(GemmArgs p) {
  constexpr int WF = kBwd ? 64 : 128;
  constexpr int WT = 128 * 64 / WF;
  constexpr int NI = WF / 16, NJ = WT / 16;
  constexpr int kItems = lg2::BF * lg2::BT / 4;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int tile = (int)(g / kItems);
  const int rem = (int)(g % kItems);
  const int wave = rem / (NI * NJ * 64);
  const int ij = (rem / 64) % (NI * NJ);
  const int lane = rem % 64;
  const int i = ij / NJ, j = ij % NJ;
  const int64_t t = (int64_t)(tile / p.tiles_f) * lg2::BT + (wave / (lg2::BF / WF)) * WT + 16 * j + (lane & 15);
  const int64_t f = (int64_t)(tile % p.tiles_f) * lg2::BF + (wave % (lg2::BF / WF)) * WF + 16 * i + 4 * (lane >> 4);
  if (tile >= p.tiles_f * p.tiles_t || t >= p.M || f >= p.N) return;
  const float* slot = p.piece_out + (size_t)tile * p.pieces * kItems * 4 + (size_t)rem * 4;
  f32x4 v = *reinterpret_cast<const f32x4*>(slot);
  for (int q = 1; q < p.pieces; ++q) v += *reinterpret_cast<const f32x4*>(slot + (size_t)q * kItems * 4);
  const int64_t o = t * p.N + f;
  if ((p.N & 3) == 0) {
    if (p.add) v += *reinterpret_cast<const f32x4*>(p.add + o);
    *reinterpret_cast<u32x2*>(p.out + o) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (f + e >= p.N) break;
    const float a = v[e] + (p.add ? p.add[o + e] : 0.0f);
    p.out[o + e] = (uint16_t)(pack_bf16x2(a, 0.0f) & 0xFFFFu);
  }
}

size_t gemm_split_ws_bytes(int64_t M, int64_t N, int64_t K) {
  const int pc = gemm_pieces(M, N, K);
  if (pc > 1) return (size_t)pc * tiles_of(M, N) * lg2::BF * lg2::BT * sizeof(float);
  const size_t ns = (size_t)gemm_split_tiles(M, N, K);
  if (!ns) return 0;
  return ns * lg2::BF * lg2::BT * sizeof(float) + (((2 * ns + 1) * sizeof(uint32_t) + 255) / 256) * 256;
}

// Byte offset, inside the split workspace, of the give-up word of a GEMM
// whose last round is split in K, or -1 when the GEMM has no hand-off.
int64_t gemm_giveup_offset(int64_t M, int64_t N, int64_t K) {
  if (gemm_pieces(M, N, K) > 1) return -1;
  const int64_t ns = gemm_split_tiles(M, N, K);
  if (!ns) return -1;
  return ns * lg2::BF * lg2::BT * (int64_t)sizeof(float) + 2 * ns * (int64_t)sizeof(uint32_t);
}

// The hand-off words of a GEMM on split_ws (none without a split or with K
// pieces), for the kernel before it to clear.
SyncZero gemm_split_sync(int64_t M, int64_t N, int64_t K, void* split_ws) {
  SyncZero z;
  if (!split_ws || gemm_pieces(M, N, K) > 1) return z;
  const int64_t ns = gemm_split_tiles(M, N, K);
  if (!ns) return z;
  z.p = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(split_ws) + (size_t)ns * lg2::BF * lg2::BT * sizeof(float));
  z.n = (int)(2 * ns + 1);
  return z;
}

template <bool kPieces>
static void launch_gemm_kernel(bool bwd, bool skip, dim3 grid, const GemmArgs& p, const Nf4Table& tab,
                               hipStream_t stream) {
  const dim3 block(lg2::kThreads);
  if (bwd && p.K % lg2::BK != 0) {
    if (skip)
      hipLaunchKernelGGL((linear_gemm_kernel<true, kPieces, true, true>), grid, block, 0, stream, p, tab);
    else
      hipLaunchKernelGGL((linear_gemm_kernel<true, kPieces, false, true>), grid, block, 0, stream, p, tab);
  } else if (bwd) {
    if (skip)
      hipLaunchKernelGGL((linear_gemm_kernel<true, kPieces, true>), grid, block, 0, stream, p, tab);
    else
      hipLaunchKernelGGL((linear_gemm_kernel<true, kPieces, false>), grid, block, 0, stream, p, tab);
  } else {
    if (skip)
      hipLaunchKernelGGL((linear_gemm_kernel<false, kPieces, true>), grid, block, 0, stream, p, tab);
    else
      hipLaunchKernelGGL((linear_gemm_kernel<false, kPieces, false>), grid, block, 0, stream, p, tab);
  }
}

// split_ws: gemm_split_ws_bytes(M, N, K) bytes (16-byte aligned), or null to
// run every tile whole.  sync_zeroed: the words of gemm_split_sync were
// cleared by an earlier kernel on the stream (else a small launch clears them).
static void launch_linear_gemm(bool bwd, const GemmArgs& a, void* split_ws, const Nf4Table& tab,
                               hipStream_t stream, bool sync_zeroed) {
  GemmArgs p = a;
  p.tiles_f = (int)((p.N + lg2::BF - 1) / lg2::BF);
  p.tiles_t = (int)((p.M + lg2::BT - 1) / lg2::BT);
  const int tiles = p.tiles_f * p.tiles_t;
  const int pc = split_ws ? gemm_pieces(p.M, p.N, p.K) : 1;
  if (pc > 1) {
    p.pieces = pc;
    p.piece_out = static_cast<float*>(split_ws);
    p.full_tiles = tiles;
    p.nsplit = 0;
    p.partial = nullptr;
    p.split_sync = nullptr;
    launch_gemm_kernel<true>(bwd, p.M % lg2::BT != 0, dim3(tiles * pc), p, tab, stream);
    const unsigned rblocks = (unsigned)tiles * (lg2::BF * lg2::BT / 4 / 256);
    if (bwd)
      hipLaunchKernelGGL(reduce_pieces_kernel<true>, dim3(rblocks), dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL(reduce_pieces_kernel<false>, dim3(rblocks), dim3(256), 0, stream, p);
    return;
  }
  const int ns = split_ws ? gemm_split_tiles(p.M, p.N, p.K) : 0;
  p.full_tiles = tiles - ns;
  p.nsplit = ns;
  p.partial = nullptr;
  p.split_sync = nullptr;
  if (ns) {
    p.partial = static_cast<float*>(split_ws);
    p.split_sync = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(split_ws) +
                                               (size_t)ns * lg2::BF * lg2::BT * sizeof(float));
    if (!sync_zeroed)
      hipLaunchKernelGGL(zero_u32_kernel, dim3((2 * ns + 1 + 255) / 256), dim3(256), 0, stream, p.split_sync,
                         2 * ns + 1);
  }
  const int grid = tiles + ns;
  launch_gemm_kernel<false>(bwd, p.M % lg2::BT != 0, dim3(grid), p, tab, stream);
}

void launch_fwd_gemm(const uint16_t* x, const uint8_t* codes, const uint8_t* absmax8, const float* c2,
                     const uint16_t* B, const float* u, uint16_t* h, int64_t M, int64_t n, int64_t m, int r,
                     float s, void* split_ws, const Nf4Table& tab, hipStream_t stream, bool sync_zeroed) {
  GemmArgs p{};
  p.act = x; p.codes = codes; p.absmax8 = absmax8; p.c2 = c2; p.lora_a = B; p.lora_b = u; p.out = h;
  p.M = M; p.K = n; p.N = m; p.wn = n; p.wm = m; p.r = r; p.s = s;
  launch_linear_gemm(false, p, split_ws, tab, stream, sync_zeroed);
}

// g is M x m_pad (m_pad = m, or m rounded up to 64 with zero columns when
// m % 8 != 0, so every 16-byte chunk of the tensor is whole).
// add: M x n fp32 added to the result before its rounding, or null; r = 0
// runs no LoRA steps.
void launch_dgrad_gemm(const uint16_t* g, const uint8_t* codes, const uint8_t* absmax8, const float* c2,
                       const uint16_t* A, const float* v, uint16_t* gx, int64_t M, int64_t n, int64_t m,
                       int64_t m_pad, int r, float s, void* split_ws, const Nf4Table& tab, hipStream_t stream,
                       const float* add, bool sync_zeroed) {
  GemmArgs p{};
  p.act = g; p.codes = codes; p.absmax8 = absmax8; p.c2 = c2; p.lora_a = A; p.lora_b = v; p.out = gx; p.add = add;
  p.M = M; p.K = m_pad; p.N = n; p.wn = n; p.wm = m; p.r = r; p.s = s;
  launch_linear_gemm(true, p, split_ws, tab, stream, sync_zeroed);
}

}  // namespace qlora
