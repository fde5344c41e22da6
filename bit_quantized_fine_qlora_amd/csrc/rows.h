// Pieces shared by the row-wise training operators (norm, 8-bit checkpoints,
// preference loss): 8 values of a row in registers, the 8-bit checkpoint
// format, and sums over a workgroup.
//
// Rows have any length, so a row's 8-value pieces need not be 16-byte
// aligned; global memory takes vector accesses at any alignment of the
// element, and the types below only tell the compiler so.
#pragma once

#include <type_traits>

#include "qlora_common.h"

namespace qlora {

// types of a row operand, as the C ABI numbers them
constexpr int kBf16 = 0, kF32 = 1, kCkpt8 = 2;

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef f32x8 f32x8_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// Length of a checkpoint's row of scale bytes: one per 32 values, rounded up
// to a multiple of 4 (the bytes past ceil(n / 32) are zero).
__host__ __device__ static inline int64_t ckpt_pitch(int64_t n) { return (n + 127) / 128 * 4; }

// ---------------------------------------------------------------------------
// 8 values in registers, as they were loaded
// ---------------------------------------------------------------------------
template <int XT>
struct Raw8;
template <>
struct Raw8<kBf16> {
  u32x4 w;
};
template <>
struct Raw8<kF32> {
  f32x8 v;
};
template <>
struct Raw8<kCkpt8> {
  u32x2 k;
  uint32_t c;
};

// One row operand: its base and, for a checkpoint, the scale bytes' base.
struct RowSrc {
  const void* p;
  const uint8_t* scales;
};

// kNt: with the non-temporal hint, for operands that are read once.  Not for
// fp32, whose 8 values are two loads: the hint drops the line between them
// (1501 x 50021 logits: loss 56 us with it and 50 us without, gradient 98 and
// 83 us).
template <bool kNt, typename T>
__device__ __forceinline__ T load_as(const void* p) {
  if constexpr (kNt) return __builtin_nontemporal_load(static_cast<const T*>(p));
  else return *static_cast<const T*>(p);
}

// Values col .. col + 7 of a row, all of which the row has.
template <int XT, bool kNt = false>
__device__ __forceinline__ Raw8<XT> load_full8(const RowSrc& s, int64_t row, int n, int col) {
  const int64_t e = row * n + col;
  Raw8<XT> r;
  if constexpr (XT == kBf16) {
    r.w = load_as<kNt, u32x4_any>(static_cast<const uint16_t*>(s.p) + e);
  } else if constexpr (XT == kF32) {
    r.v = load_as<kNt, f32x8_any>(static_cast<const float*>(s.p) + e);
  } else {
    r.k = load_as<kNt, u32x2_any>(static_cast<const uint8_t*>(s.p) + e);
    r.c = s.scales[row * ckpt_pitch(n) + (col >> 5)];
  }
  return r;
}

// The same for a piece that may cross or lie past the row's end, in two parts.
// load_piece8 always loads: a load under a branch would make the compiler wait
// for every load in flight where the paths meet.  A piece that crosses the end
// reads the row's last 8 values, one past it the first 8 (so n must be at
// least 8); finish_piece8, where the values are used, moves the former into
// place and clears what the row does not have.
template <int XT>
__device__ __forceinline__ Raw8<XT> load_piece8(const RowSrc& s, int64_t row, int n, int col) {
  const int from = col + 8 <= n ? col : col < n ? n - 8 : 0;
  if constexpr (XT == kCkpt8) {
    Raw8<XT> r;
    r.k = *reinterpret_cast<const u32x2_any*>(static_cast<const uint8_t*>(s.p) + row * n + from);
    r.c = s.scales[row * ckpt_pitch(n) + (col < n ? col >> 5 : 0)];
    return r;
  } else {
    return load_full8<XT>(s, row, n, from);
  }
}

template <int XT>
__device__ __forceinline__ Raw8<XT> finish_piece8(Raw8<XT> r, int n, int col) {
  if (col + 8 <= n) return r;
  const int by = col < n ? col + 8 - n : 8;  // values to move down by
  if constexpr (XT == kBf16) {
    u32x4 w = r.w;
    w = by & 8 ? u32x4{0u, 0u, 0u, 0u} : w;
    w = by & 4 ? u32x4{w[2], w[3], 0u, 0u} : w;
    w = by & 2 ? u32x4{w[1], w[2], w[3], 0u} : w;
    const u32x4 h = {w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
    r.w = by & 1 ? h : w;
  } else if constexpr (XT == kF32) {
#pragma unroll
    for (int d = 8; d; d >>= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) r.v[j] = by & d ? (j + d < 8 ? r.v[(j + d) & 7] : 0.0f) : r.v[j];
  } else {
    const uint64_t k = by & 8 ? 0ull : ((uint64_t)r.k[1] << 32 | r.k[0]) >> (8 * by);
    r.k = u32x2{(uint32_t)k, (uint32_t)(k >> 32)};
    r.c = by & 8 ? 0u : r.c;
  }
  return r;
}

// The first `count` (1..7) of 8 values from `col` on, the rest zero.
template <int XT>
__device__ __forceinline__ Raw8<XT> load_tail8(const RowSrc& s, int64_t row, int n, int col, int count) {
  const int64_t e = row * n + col;
  Raw8<XT> r;
  if constexpr (XT == kBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(s.p) + e;
    r.w = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < count) r.w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
  } else if constexpr (XT == kF32) {
    const float* p = static_cast<const float*>(s.p) + e;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = j < count ? p[j < count ? j : 0] : 0.0f;
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(s.p) + e;
    r.k = u32x2{0u, 0u};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < count) r.k[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    r.c = s.scales[row * ckpt_pitch(n) + (col >> 5)];
  }
  return r;
}

// ---------------------------------------------------------------------------
// The 8-bit checkpoint of a bf16 row.  A block of 32 consecutive values keeps
// 8-bit integers k and one byte c; the value is k 2^(c - 127).  With E the
// exponent field of the block's largest magnitude, c = max(E, 7) - 6, which
// puts that magnitude at 64 <= |k| < 128 (below for E < 7: steps under
// 2^-126 are not used), and k = x 2^(127 - c) rounded half to even and held
// within +-127.  A power-of-two step costs up to a factor of two against
// largest / 127, and a block of 32 instead of a row wins more than that back
// where some channels are far larger than others; in exchange both
// directions are exact scalings: a restored value is a bf16 number, so a
// kernel that restores in registers sees the same bits as one that reads the
// restored tensor, and the 8-bit mantissa of the largest values loses one bit.
// c = 255 marks a block with an infinity or NaN: k = 0 throughout, and
// 0 times the infinite scale restores the whole block as NaN.
// ---------------------------------------------------------------------------

// Codes (4 to a word) and scale byte of 8 bf16 values; 4 lanes that are
// neighbours in a quad hold one block's 32 values and get the same c.
__device__ __forceinline__ void ckpt_encode8(const u32x4& w, u32x2& k, uint32_t& c) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[j] & 0x7FFF7FFFu));
  uint32_t top = m[0] > m[1] ? m[0] : m[1];
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true);  // quad lanes 1 0 3 2
  top = top > o ? top : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true);  // quad lanes 2 3 0 1
  top = top > o ? top : o;
  const uint32_t e = top >> 7;
  c = e == 255u ? 255u : (e > 7u ? e : 7u) - 6u;
  const float inv = __uint_as_float((254u - c) << 23);  // 2^(127 - c)
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = (j & 1) ? bf16_hi_to_f32(w[j >> 1]) : bf16_lo_to_f32(w[j >> 1]);
    // the product is exact; adding 1.5 2^23 rounds it half to even and leaves
    // the integer in the sum's low byte
    b[j] = __float_as_uint(__builtin_amdgcn_fmed3f(x * inv, -127.0f, 127.0f) + 12582912.0f);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    k[h] = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u) |
           __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
  if (c == 255u) k = u32x2{0u, 0u};
}

__device__ __forceinline__ float ckpt_scale(uint32_t c) { return __uint_as_float(c << 23); }  // 2^(c - 127)

// Restoring 4 codes: a byte of ckpt_biased(word) is k + 127, and k 2^(c - 127)
// = fma(k + 127, scale, -127 scale), exactly: the unsigned byte conversion
// runs at full rate where the signed one takes twice as long, and with a bias
// of 127 the last term is finite for every scale that a finite block has.
__device__ __forceinline__ uint32_t ckpt_biased(uint32_t word) { return (word ^ 0x80808080u) - 0x01010101u; }
__device__ __forceinline__ float ckpt_value(uint32_t biased, int j, float scale, float offset) {
  return __builtin_fmaf((float)((biased >> (8 * j)) & 0xFFu), scale, offset);
}

template <int XT>
__device__ __forceinline__ void raw_to_f32(const Raw8<XT>& r, float (&v)[8]) {
  if constexpr (XT == kBf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo_to_f32(r.w[j]);
      v[2 * j + 1] = bf16_hi_to_f32(r.w[j]);
    }
  } else if constexpr (XT == kF32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r.v[j];
  } else {
    const float s = ckpt_scale(r.c), o = -127.0f * s;
    const uint32_t b[2] = {ckpt_biased(r.k[0]), ckpt_biased(r.k[1])};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = ckpt_value(b[j >> 2], j & 3, s, o);
  }
}

__device__ __forceinline__ u32x4 round_bf16x8(const float (&v)[8]) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// Stores the first min(8, n - col) of 8 values (none past the row's end),
// rounded to bf16 where XT is; a piece that crosses the end goes out as 4, 2
// and 1 values.
template <int XT>
__device__ __forceinline__ void store8(void* base, int64_t row, int n, int col, const float (&v)[8]) {
  typedef uint32_t u32_any __attribute__((aligned(2)));
  typedef u32x2 u32x2_b __attribute__((aligned(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef f32x2 f32x2_any __attribute__((aligned(4)));
  if (col >= n) return;
  const int64_t e = row * n + col;
  if constexpr (XT == kBf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + e;
    u32x4 w = round_bf16x8(v);
    if (col + 8 <= n) {
      *reinterpret_cast<u32x4_any*>(p) = w;
    } else {
      if ((n - col) & 4) {
        *reinterpret_cast<u32x2_b*>(p) = u32x2{w[0], w[1]};
        w[0] = w[2];
        w[1] = w[3];
        p += 4;
      }
      if ((n - col) & 2) {
        *reinterpret_cast<u32_any*>(p) = w[0];
        w[0] = w[1];
        p += 2;
      }
      if ((n - col) & 1) *p = (uint16_t)w[0];
    }
  } else {
    float* p = static_cast<float*>(base) + e;
    f32x4 a = {v[0], v[1], v[2], v[3]};
    const f32x4 b = {v[4], v[5], v[6], v[7]};
    if (col + 8 <= n) {
      *reinterpret_cast<f32x4_any*>(p) = a;
      *reinterpret_cast<f32x4_any*>(p + 4) = b;
    } else {
      if ((n - col) & 4) {
        *reinterpret_cast<f32x4_any*>(p) = a;
        a = b;
        p += 4;
      }
      if ((n - col) & 2) {
        *reinterpret_cast<f32x2_any*>(p) = f32x2{a[0], a[1]};
        a[0] = a[2];
        p += 2;
      }
      if ((n - col) & 1) *p = a[0];
    }
  }
}

// Encodes and stores 8 bf16 values (zeros past the row's end) of the
// checkpoint row; the 4 lanes of a quad hold neighbouring pieces, and lanes
// up to the padded row length take part.
__device__ __forceinline__ void ckpt_store8(int8_t* codes, uint8_t* scales, int64_t row, int n, int col,
                                            const u32x4& w) {
  u32x2 k;
  uint32_t c;
  ckpt_encode8(w, k, c);
  if (col + 8 <= n) {
    *reinterpret_cast<u32x2_any*>(codes + row * n + col) = k;
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (col + j < n) codes[row * n + col + j] = (int8_t)(k[j >> 2] >> (8 * (j & 3)));
  }
  const int64_t pitch = ckpt_pitch(n);
  if ((col & 31) == 0 && (col >> 5) < pitch) scales[row * pitch + (col >> 5)] = (uint8_t)(col < n ? c : 0u);
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------

// Sum over the wave's 64 lanes by DPP row shifts and broadcasts; every lane
// gets it.  The order is fixed.
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](auto ctrl, auto rows) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, decltype(rows)::value,
                                                    0xF, false));
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});  // row_shr:1
  add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});  // row_shr:2
  add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});  // row_shr:4
  add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});  // row_shr:8
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // row_bcast:15 into rows 1 and 3
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // row_bcast:31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

}  // namespace qlora
