// wc_fp4.hip — BF16 matrices as 4-bit codes with a power-of-two scale per 32
// columns: encode, read-back, and matrix-vector products (include/wc_fp4.h
// defines the format).
#include "wc_launch.h"
#include "wc_skinny.h"

namespace wc {

// The biased exponent of a group's scale from the largest |w| (BF16 bits
// without the sign): the smallest e >= 1 with |w| <= 7 * 2^(e - 127).
// |w| = 1.m * 2^(E - 127) is within 7 * 2^(E - 2 - 127) exactly when
// 1.m <= 1.75, that is m <= 0x60.
__device__ inline uint32_t fp4_exponent(uint32_t top) {
  const int e = (int)(top >> 7) - 2 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  return top >= 0x7F80u ? 255u : (uint32_t)(e < 1 ? 1 : e);
}

// 8 BF16 values / 2^(e - 127) to the nearest code, ties to even (the
// instruction's rounding; above 6 it gives 6, and no value is above 7).
__device__ inline uint32_t fp4_pack8(u32x4 w, uint32_t e) {
  const float s = fp4_scale(e);
  // whole dwords first: a bit cast of a vector's element reads element 0
  const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mfma_bf16x2, w0), s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mfma_bf16x2, w1), s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mfma_bf16x2, w2), s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mfma_bf16x2, w3), s, 3);
  if (e == 253u) {  // code 6 (4 * 2^126) is past BF16: it becomes 5
    const uint32_t six = c >> 2 & c >> 1 & ~c & 0x11111111u;
    c -= six;
  }
  return e == 255u ? 0u : c;
}

__device__ inline uint32_t max_abs8(u32x4 w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  return m;
}

// A lane codes 8 columns; the four lanes of a group share their maximum.
// Blocks walk the rows' pieces of 8 columns, `pieces` = 4 G per row.
__global__ __launch_bounds__(kBlockThreads) void k_fp4_encode(const uint16_t* __restrict__ w,
                                                              uint64_t rows, uint32_t cols,
                                                              uint32_t groups,
                                                              uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  const uint64_t total = rows * groups * 4u;
  const uint64_t stride = (uint64_t)gridDim.x * kBlockThreads;
  // whole quads of lanes share a group, and total is a multiple of 4
  for (uint64_t p = (uint64_t)blockIdx.x * kBlockThreads + threadIdx.x; p < total; p += stride) {
    const uint64_t row = p / (groups * 4u);
    const uint32_t c = (uint32_t)(p - row * (groups * 4u)) * 8u;
    const u32x4 v = load8(w + row * cols + c, (int)cols - (int)c);
    uint32_t m = max_abs8(v);
    const uint32_t a = (uint32_t)__shfl_xor((int)m, 1, kWave);
    m = m > a ? m : a;
    const uint32_t b = (uint32_t)__shfl_xor((int)m, 2, kWave);
    m = m > b ? m : b;
    const uint32_t e = fp4_exponent(m);
    ((uint32_t*)codes)[p] = fp4_pack8(v, e);
    if ((p & 3u) == 0) scales[p / 4u] = (uint8_t)e;
  }
}

__global__ __launch_bounds__(kBlockThreads) void k_fp4_decode(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              uint64_t rows, uint32_t cols,
                                                              uint32_t groups,
                                                              uint16_t* __restrict__ out) {
  const uint64_t total = rows * groups * 4u;
  const uint64_t stride = (uint64_t)gridDim.x * kBlockThreads;
  for (uint64_t p = (uint64_t)blockIdx.x * kBlockThreads + threadIdx.x; p < total; p += stride) {
    const uint64_t row = p / (groups * 4u);
    const uint32_t c = (uint32_t)(p - row * (groups * 4u)) * 8u;
    const u32x4 v = fp4_expand(((const uint32_t*)codes)[p], fp4_scale(scales[p / 4u]));
    uint16_t* o = out + row * cols + c;
    if (c + 8u <= cols) {
      *(u32x4_any*)o = v;
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 7; ++i)
        if (c + i < cols) o[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  }
}

struct Fp4Args {
  const uint8_t* codes;
  const uint8_t* scales;
  const uint16_t* x;
  float* y;
  uint64_t rows;
  uint32_t cols, batch, steps;
};

// 16 rows per block; its waves take every WPB-th step of 128 columns and add
// their sums in LDS in wave order.  NT tiles of 16 input rows per wave; input
// rows past the batch repeat the last one and are not stored.
template <int NT, int WPB>
__global__ __launch_bounds__(kWave * WPB) void k_fp4_gemv(Fp4Args a) {
  __shared__ mfma_f32x4 part[WPB][NT][kWave];
  const int lane = lane_id(), wave = wave_in_block();
  const uint32_t r = (uint32_t)lane & 15u;
  const uint64_t row0 = (uint64_t)blockIdx.x * kRowTile;
  const uint64_t row = row0 + r < a.rows ? row0 + r : a.rows - 1u;
  const uint32_t b0 = blockIdx.y * (kRowTile * NT);
  const WeightRow w = weight_row<kFp4>(a.codes, a.scales, row, a.cols);
  const uint16_t* x[NT];
  mfma_f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t b = b0 + 16u * t + r;
    x[t] = a.x + (uint64_t)(b < a.batch ? b : a.batch - 1u) * a.cols;
    acc[t] = mfma_f32x4{0, 0, 0, 0};
  }
  struct Slot {
    WeightStep<kFp4> w;
    u32x4 x[NT][4];
  };
  const uint32_t n = a.steps > (uint32_t)wave ? (a.steps - 1u - (uint32_t)wave) / WPB + 1u : 0u;
  step_ring<2, Slot>(
      n,
      [&](uint32_t q, Slot& s) {
        const uint32_t step = q * WPB + (uint32_t)wave;
        load_weights<kFp4>(w, step, a.cols, s.w);
#pragma unroll
        for (int t = 0; t < NT; ++t) load_inputs<kFp4>(x[t], step, a.cols, s.x[t]);
      },
      [&](uint32_t, const Slot& s) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 op = weight_operand<kFp4>(s.w, j);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[t] = mfma16(op, s.x[t][j], acc[t]);
        }
      });
#pragma unroll
  for (int t = 0; t < NT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < NT * kWave; i += kWave * WPB) {
    const uint32_t t = i / kWave, l = i % kWave;
    mfma_f32x4 s = part[0][t][l];
#pragma unroll
    for (int v = 1; v < WPB; ++v) s += part[v][t][l];
    const uint32_t b = b0 + 16u * t + (l & 15u);
    const uint64_t y0 = row0 + 4u * (l >> 4);
    if (b < a.batch) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (y0 + k < a.rows) a.y[(uint64_t)b * a.rows + y0 + k] = s[k];
    }
  }
}

namespace {

int fp4_shape_ok(uint64_t rows, uint64_t cols) {
  if (cols > WC_FP4_MAX_COLS) return WC_E_SIZE;
  if (cols && rows >= (1ull << 40) / cols) return WC_E_SIZE;
  return WC_OK;
}

int launched() { return hipGetLastError() == hipSuccess ? WC_OK : WC_E_HIP; }

uint32_t piece_blocks(uint64_t pieces) {
  const uint64_t b = (pieces + kBlockThreads - 1) / kBlockThreads;
  const uint64_t most = (uint64_t)cu_count() * 16u;
  return (uint32_t)(b < most ? b : most);
}

}  // namespace
}  // namespace wc

extern "C" int wc_fp4_encode(const uint16_t* d_w, uint64_t rows, uint64_t cols, uint8_t* d_codes,
                             uint8_t* d_scales, void* stream) {
  if (const int v = wc::fp4_shape_ok(rows, cols)) return v;
  if (rows == 0 || cols == 0) return WC_OK;
  if (!d_w || !wc::aligned16(d_w) || !d_codes || !wc::aligned16(d_codes) || !d_scales) return WC_E_ARG;
  const uint32_t groups = (uint32_t)WC_FP4_GROUPS(cols);
  wc::k_fp4_encode<<<wc::piece_blocks(rows * groups * 4u), wc::kBlockThreads, 0, (hipStream_t)stream>>>(
      d_w, rows, (uint32_t)cols, groups, d_codes, d_scales);
  return wc::launched();
}

extern "C" int wc_fp4_decode(const uint8_t* d_codes, const uint8_t* d_scales, uint64_t rows,
                             uint64_t cols, uint16_t* d_out, void* stream) {
  if (const int v = wc::fp4_shape_ok(rows, cols)) return v;
  if (rows == 0 || cols == 0) return WC_OK;
  if (!d_out || !wc::aligned16(d_out) || !d_codes || !wc::aligned16(d_codes) || !d_scales)
    return WC_E_ARG;
  const uint32_t groups = (uint32_t)WC_FP4_GROUPS(cols);
  wc::k_fp4_decode<<<wc::piece_blocks(rows * groups * 4u), wc::kBlockThreads, 0, (hipStream_t)stream>>>(
      d_codes, d_scales, rows, (uint32_t)cols, groups, d_out);
  return wc::launched();
}

extern "C" int wc_fp4_gemv(const uint8_t* d_codes, const uint8_t* d_scales, uint64_t rows,
                           uint64_t cols, const uint16_t* d_x, uint32_t batch, float* d_y,
                           void* stream) {
  if (batch < 1 || batch > WC_MAX_BATCH) return WC_E_UNSUPPORTED;
  if (const int v = wc::fp4_shape_ok(rows, cols)) return v;
  if (rows == 0) return WC_OK;
  if (!d_y || ((uintptr_t)d_y & 3u)) return WC_E_ARG;
  if (cols && (!d_codes || !wc::aligned16(d_codes) || !d_scales || !d_x || !wc::aligned16(d_x)))
    return WC_E_ARG;
  const uint64_t row_blocks = (rows + wc::kRowTile - 1) / wc::kRowTile;
  if (row_blocks >= (1ull << 31)) return WC_E_SIZE;
  wc::Fp4Args a = {d_codes, d_scales, d_x, d_y, rows, (uint32_t)cols, batch,
                   (uint32_t)((cols + wc::kStep - 1) / wc::kStep)};
  hipStream_t s = (hipStream_t)stream;
  const dim3 block(wc::kWave * 8);
  if (batch <= 16)
    wc::k_fp4_gemv<1, 8><<<dim3((uint32_t)row_blocks, 1), block, 0, s>>>(a);
  else if (batch <= 32)
    wc::k_fp4_gemv<2, 8><<<dim3((uint32_t)row_blocks, 1), block, 0, s>>>(a);
  else
    wc::k_fp4_gemv<4, 8><<<dim3((uint32_t)row_blocks, (batch + 63u) / 64u), block, 0, s>>>(a);
  return wc::launched();
}
