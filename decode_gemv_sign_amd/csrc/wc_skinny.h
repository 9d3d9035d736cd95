// wc_skinny.h — products of weight rows with a few columns on the matrix
// cores, shared by the 4-bit GEMV (wc_fp4.hip) and the mixture-of-experts
// layer (wc_moe.hip).
//
// One v_mfma_f32_16x16x32_bf16 multiplies 16 weight rows with up to 16 input
// rows over 32 columns.  Lane l = r + 16 h gives 8 values of weight row r and
// 8 values of input row r, and receives sums of input row r with weight rows
// 4h .. 4h + 3.  The two operands only have to put the same column at the same
// (h, element) place, so a wave's step of 128 columns (four of these) may take
// its columns in the order in which they load best:
//   4-bit weights  lane h owns columns 32h .. 32h + 31 of the step, one group:
//                  16 bytes of codes and one scale, a single wide load
//   BF16 weights   instance j owns columns 32j .. 32j + 31, lane h 8 of them,
//                  so that every load covers 64 contiguous bytes of each row
#pragma once

#include "wc_common.h"
#include "wc_fp4.h"

namespace wc {

constexpr int kRowTile = 16;   // weight rows, and input rows, per MFMA
constexpr int kStep = 128;     // columns per wave step

enum WeightKind { kBf16 = 0, kFp4 = 1 };

typedef __bf16 mfma_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 mfma_bf16x8 __attribute__((ext_vector_type(8)));
typedef float mfma_f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ inline mfma_f32x4 mfma16(u32x4 a, u32x4 b, mfma_f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mfma_bf16x8, a),
                                                 __builtin_bit_cast(mfma_bf16x8, b), c, 0, 0, 0);
}

// The scale 2^(e - 127) as the conversion instructions take it: they use the
// exponent field alone, so e = 0 is 2^-127 and e = 255 gives NaN.
__device__ inline float fp4_scale(uint32_t e) { return __uint_as_float(e << 23); }

// 8 codes (low nibble first) times their scale, as 8 BF16 values: four
// conversions, exact within BF16's range.
__device__ inline u32x4 fp4_expand(uint32_t codes, float scale) {
  u32x4 w;
  w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return w;
}

__device__ inline uint16_t bf16_of(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// 8 BF16 values at p, of which the first `left` exist (the rest are 0, and
// are not read).  Rows of an odd length start at any 2-byte address.
__device__ inline u32x4 load8(const uint16_t* __restrict__ p, int left) {
  if (left >= 8) return *(const u32x4_any*)p;
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < left) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
  return v;
}

// A lane's view of a weight row and of an input row.
struct WeightRow {
  const uint8_t* data;    // 4-bit: the lane's first group; BF16: the lane's first value
  const uint8_t* scales;  // 4-bit: the lane's first scale
};

// Row `row` of an array of rows of `cols` columns.
template <int KIND>
__device__ inline WeightRow weight_row(const void* data, const uint8_t* scales, uint64_t row,
                                       uint32_t cols) {
  const uint32_t h = (uint32_t)lane_id() >> 4;
  WeightRow w;
  if constexpr (KIND == kFp4) {
    const uint64_t groups = WC_FP4_GROUPS(cols);
    w.data = (const uint8_t*)data + (row * groups + h) * 16u;
    w.scales = scales + row * groups + h;
  } else {
    w.data = (const uint8_t*)((const uint16_t*)data + row * cols + 8u * h);
    w.scales = nullptr;
  }
  return w;
}

// A lane's weights of one step.
template <int KIND>
struct WeightStep {
  u32x4 v[KIND == kFp4 ? 1 : 4];
  uint32_t e;
};

template <int KIND>
__device__ inline void load_weights(const WeightRow& w, uint32_t step, uint32_t cols,
                                    WeightStep<KIND>& s) {
  const bool whole = (step + 1) * kStep <= cols;  // the same for all lanes
  const uint32_t h = (uint32_t)lane_id() >> 4;
  if constexpr (KIND == kFp4) {
    const bool in = whole || step * kStep + 32u * h < cols;  // padding nibbles are 0
    if (in) {
      s.v[0] = __builtin_nontemporal_load((const u32x4*)(w.data + (size_t)step * 64u));
      s.e = w.scales[step * 4u];
    } else {
      s.v[0] = u32x4{0, 0, 0, 0};
      s.e = 127;
    }
  } else {
    const uint16_t* p = (const uint16_t*)w.data + (size_t)step * kStep;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int left = (int)cols - (int)(step * kStep + 32u * j + 8u * h);
      s.v[j] = whole ? *(const u32x4_any*)(p + 32 * j) : load8(p + 32 * j, left);
    }
  }
}

// A lane's values of one input row in one step, in the weights' column order;
// x points at the row.
template <int KIND>
__device__ inline void load_inputs(const uint16_t* __restrict__ x, uint32_t step, uint32_t cols,
                                   u32x4 v[4]) {
  const bool whole = (step + 1) * kStep <= cols;
  const uint32_t h = (uint32_t)lane_id() >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t c = step * kStep + (KIND == kFp4 ? 32u * h + 8u * j : 32u * j + 8u * h);
    v[j] = whole ? *(const u32x4_any*)(x + c) : load8(x + c, (int)cols - (int)c);
  }
}

// Instance j's weight operand.
template <int KIND>
__device__ inline u32x4 weight_operand(const WeightStep<KIND>& s, int j) {
  if constexpr (KIND == kFp4)
    return fp4_expand(s.v[0][j], fp4_scale(s.e));
  else
    return s.v[j];
}

// Software pipeline over n steps with D slots: step q + D - 1 is loaded just
// before step q is used.  Past the end the last step is loaded again, so the
// loads in flight are the same on every path.
template <int D, typename Slot, typename Load, typename Use>
__device__ inline void step_ring(uint32_t n, Load&& load, Use&& use) {
  if (n == 0) return;
  Slot s[D];
#pragma unroll
  for (int i = 0; i < D - 1; ++i) load((uint32_t)i < n ? (uint32_t)i : n - 1u, s[i]);
  for (uint32_t q = 0; q < n; q += D) {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      const uint32_t next = q + i + D - 1;
      load(next < n ? next : n - 1u, s[(i + D - 1) % D]);
      if (q + i >= n) return;
      use(q + i, s[i]);
    }
  }
}

}  // namespace wc
