// wc_skinny.h — products of weight rows with a few input rows on the matrix
// cores, shared by the 4-bit GEMV (wc_fp4.hip) and the mixture-of-experts
// layer (wc_moe.hip).
//
// One v_mfma_f32_16x16x32_bf16 multiplies 16 weight rows with 16 input rows
// over 32 columns.  Lane r + 16 h gives 8 values of weight row r and 8 values of
// input row r, and receives the sums of input row r with weight rows 4h .. 4h+3.
// The two operands only have to put the same column at the same (h, element)
// place, so any order of the columns will do.
//
// Loads in that lane order are slow: neighbouring lanes touch 16 different rows,
// and the vector L1 then takes 64 cycles for a wave's 1 KB load (measured: 65,
// bytes and dwords the same), where four neighbouring lanes on 64 contiguous
// bytes take 17.  At 1 KB of 4-bit codes per 64 cycles and as much again for the
// scales a compute unit gets 8 bytes per cycle, which bound the first form of
// these kernels at about half of HBM's rate.  So lane 4b + j (+ 16 h) loads piece
// j of row 4b + i in load i, for i = 0 .. 3, and the four registers are
// transposed inside each quad of lanes by DPP: register j then holds piece j of
// row r = 4b + i, as the MFMA wants it.
//
// Columns go by steps:
//   4-bit weights  512 columns: piece (h, j) is the group of columns
//                  128 h + 32 j .., one 16-byte load; four blocks j of four MFMAs
//   BF16 weights   128 columns: piece (h, j) is columns 32 h + 8 j ..; one block
#pragma once

#include <type_traits>

#include "wc_common.h"
#include "wc_fp4.h"

namespace wc {

constexpr uint32_t kRowTile = 16;  // weight rows, and input rows, per MFMA

enum WeightKind {
  kBf16 = 0,
  kFp4 = 1,
  kBf16Any = 2,  // BF16 rows that start at any 2-byte address
};
template <int KIND>
constexpr uint32_t kBlocks = KIND == kFp4 ? 4u : 1u;  // blocks of a step
template <int KIND>
constexpr uint32_t kStepCols = 128u * kBlocks<KIND>;

typedef __bf16 mfma_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 mfma_bf16x8 __attribute__((ext_vector_type(8)));
typedef float mfma_f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef __amdgpu_buffer_rsrc_t buffer;

__device__ __forceinline__ mfma_f32x4 mfma16(u32x4 a, u32x4 b, mfma_f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mfma_bf16x8, a),
                                                 __builtin_bit_cast(mfma_bf16x8, b), c, 0, 0, 0);
}

// The scale 2^(e - 127) as the conversion instructions take it: they use the
// exponent field alone, so e = 0 is 2^-127 and e = 255 gives NaN.
__device__ __forceinline__ float fp4_scale(uint32_t e) { return __uint_as_float(e << 23); }

// 8 codes (low nibble first) times their scale, as 8 BF16 values: four
// conversions, exact within BF16's range.
__device__ __forceinline__ u32x4 fp4_expand(uint32_t codes, float scale) {
  u32x4 w;
  w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return w;
}

__device__ __forceinline__ uint16_t bf16_of(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// f(0), .., f(N - 1) with constant arguments: registers indexed by them stay
// registers.
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// Inputs that the kernels can read: rows that start at 16-byte boundaries, or, of a
// length that rules this out, at any 2-byte address.
inline bool rows_aligned(const void* x, uint64_t cols) {
  return x && ((uintptr_t)x & (cols % 8u ? 1u : 15u)) == 0;
}

// ---- loads -------------------------------------------------------------------

// Bytes [0, n) from p on (wave-uniform).  What a load asks for past them reads as
// 0 and touches no memory; kNowhere is such an offset for every buffer here.
__device__ __forceinline__ buffer buffer_of(const void* p, uint32_t n) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)n, 0x00027000);
}
constexpr uint32_t kNowhere = 0xFFFFFF00u;
template <bool ONCE = false>  // ONCE: what nothing reads again; the caches let it go first
__device__ __forceinline__ u32x4 load16(buffer b, uint32_t lane_off, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)lane_off, (int)off, ONCE ? 2 : 0));
}
// 16 bytes per lane into LDS at dst + 16 * lane.  Buffer loads, as the compiler
// waits for all loads where a register load was followed by one through a
// pointer into LDS.
__device__ __forceinline__ void load16_lds(buffer b, uint8_t* dst, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void_t*)dst, 16, (int)lane_off, (int)off, 0, 0);
}

// Values c .. c + 7 of a row of `cols` BF16 values (cols >= 1); what lies past
// the row is 0.  Rows of an odd length start at any 2-byte address.  A piece that
// the row's end cuts is taken from the row's last 8 values and shifted down, so
// that every piece is one load within the row.
__device__ inline u32x4 load8(const uint16_t* __restrict__ row, uint32_t c, uint32_t cols) {
  if (cols < 8u) {  // the same for all lanes
    uint32_t e[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) e[i] = row[i < cols ? i : cols - 1u];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) e[i] = c + i < cols ? e[i] : 0u;  // c is a multiple of 8
    return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
  }
  const uint32_t from = c < cols - 8u ? c : cols - 8u, off = c - from;
  const u32x4 v = *(const u32x4_any*)(row + from);
  uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  if (off >= 4u) {
    lo = hi;
    hi = 0;
  }
  const uint32_t sh = 16u * (off & 3u);
  lo = lo >> sh | (hi << 1) << (63u - sh);
  hi >>= sh;
  if (off >= 8u) lo = hi = 0;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// a of the lanes with `up` set and b of the others change places across PERM.
template <int PERM>
__device__ __forceinline__ void quad_swap(u32x4& a, u32x4& b, bool up) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = a[k], y = b[k];
    const uint32_t xs = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, PERM, 0xF, 0xF, true);
    const uint32_t ys = (uint32_t)__builtin_amdgcn_mov_dpp((int)y, PERM, 0xF, 0xF, true);
    a[k] = up ? ys : x;
    b[k] = up ? y : xs;
  }
}

// v[j] of lane 4b + i <- v[i] of lane 4b + j.
__device__ __forceinline__ void quad_transpose(u32x4 v[4]) {
  const bool odd = lane_id() & 1, high = lane_id() & 2;
  quad_swap<0xB1>(v[0], v[1], odd);  // lanes 1 0 3 2
  quad_swap<0xB1>(v[2], v[3], odd);
  quad_swap<0x4E>(v[0], v[2], high);  // lanes 2 3 0 1
  quad_swap<0x4E>(v[1], v[3], high);
}

// ---- weights -----------------------------------------------------------------

// Where a lane's pieces stand in a tile of 16 rows of `cols` columns: the same for
// every tile of an array.
template <int KIND>
struct WeightLane {
  uint32_t cols, row_bytes, groups;
  uint32_t off[4];     // piece lane & 3 of row 4b + i
  uint32_t scale_off;  // kFp4: of the lane's MFMA row r, from group 4 h on

  __device__ __forceinline__ explicit WeightLane(uint32_t c) : cols(c) {
    const uint32_t lane = (uint32_t)lane_id(), r = lane & 15u, h = lane >> 4;
    groups = (uint32_t)WC_FP4_GROUPS(c);
    row_bytes = KIND == kFp4 ? groups * 16u : c * 2u;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) off[i] = ((r & ~3u) + i) * row_bytes + 64u * h + 16u * (r & 3u);
    scale_off = r * groups + 4u * h;
  }
};

// Rows row0 .. row0 + 15 of an array of `rows` rows (all of it wave-uniform).
// Sums of rows past the end come out as 0, or as another row's, and are not used.
template <int KIND>
struct WeightTile {
  const uint8_t* data;
  const uint8_t* scales;
  uint32_t n;  // rows that exist, up to 16

  __device__ __forceinline__ WeightTile(const void* d, const uint8_t* s, uint64_t row0, uint64_t rows,
                                        const WeightLane<KIND>& l) {
    n = rows - row0 < 16u ? (uint32_t)(rows - row0) : 16u;
    data = (const uint8_t*)d + row0 * l.row_bytes;
    scales = KIND == kFp4 ? s + row0 * l.groups : nullptr;
  }
};

// A lane's weights of one step; kFp4: with the scales of its four groups.
struct WeightStep {
  u32x4 v[4];
  uint32_t e;
};

// TAIL: the row's last step, of which some columns do not exist: they read as 0.
// ONCE: for weights that no other tile of inputs needs.  It pays in the MoE
// kernels, where an expert's matrices are one tile's (128 experts, 16 tokens, 4-bit:
// 127 us without, 114 with; 32 experts, BF16, 2 tokens: 81 and 75; 64 experts, BF16,
// 64 tokens: 170 and 157).  The 4-bit GEMV goes without: its matrices may still be in
// the card's memory-side cache (24576 x 6144, batch 1: 17.6 us without, 18.5 with;
// from HBM 20.4 and 19.0).
template <int KIND, bool TAIL, bool ONCE = false>
__device__ __forceinline__ void load_weights(const WeightLane<KIND>& l, const WeightTile<KIND>& w,
                                             uint32_t step, WeightStep& s) {
  const uint32_t lane = (uint32_t)lane_id(), r = lane & 15u, h = lane >> 4, j = lane & 3u;
  if constexpr (KIND == kFp4) {
    const buffer b = buffer_of(w.data, w.n * l.row_bytes);  // rows past the end read as 0
    const bool in = !TAIL || step * 16u + 4u * h + j < l.groups;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.v[i] = load16<ONCE>(b, in ? l.off[i] : kNowhere, step * 256u);
    const uint8_t* scales = w.scales + (r < w.n ? l.scale_off : 4u * h) + step * 16u;
    if constexpr (TAIL) {
      s.e = 0;
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (step * 16u + 4u * h + k < l.groups) s.e |= (uint32_t)scales[k] << (8u * k);
    } else {
      s.e = *(const u32_any*)scales;
    }
  } else if constexpr (KIND == kBf16) {
    const buffer b = buffer_of(w.data, w.n * l.row_bytes);
    const bool in = !TAIL || step * 128u + 32u * h + 8u * j < l.cols;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.v[i] = load16<ONCE>(b, in ? l.off[i] : kNowhere, step * 256u);
  } else {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t q = (r & ~3u) + i;
      const uint16_t* row = (const uint16_t*)(w.data + (uint64_t)(q < w.n ? q : w.n - 1u) * l.row_bytes);
      const uint32_t c = step * 128u + 32u * h + 8u * j;
      s.v[i] = TAIL ? load8(row, c, l.cols) : *(const u32x4_any*)(row + c);
    }
  }
}

// Operand k (0 .. 3) of block j, after quad_transpose(s.v).
template <int KIND>
__device__ __forceinline__ u32x4 weight_operand(const WeightStep& s, int j, int k) {
  if constexpr (KIND == kFp4) {
    const uint32_t e = j == 0 ? s.e << 23 : j == 1 ? s.e << 15 : j == 2 ? s.e << 7 : s.e >> 1;
    return fp4_expand(s.v[j][k], __uint_as_float(e & 0x7F800000u));
  } else {
    return s.v[k];
  }
}

// n steps, U at a time: the loads of U steps go out together, then the steps are
// used; the other waves of the compute unit have theirs in flight meanwhile.
// Loading a step ahead of its use measured slower where a wave has few steps: past
// the end such a pipeline either loads for nothing (each load costs its address
// cycles) or branches, and then every wait is for all loads.
template <int U, typename Slot, typename Load, typename Use>
__device__ __forceinline__ void step_batch(uint32_t q, Load&& load, Use&& use) {
  Slot s[U];
  each<U>([&](auto i) __attribute__((always_inline)) { load(q + i, s[i]); });
  __builtin_amdgcn_sched_barrier(0);  // no load moves down among the uses
  each<U>([&](auto i) __attribute__((always_inline)) { use(s[i]); });
}
template <int U, typename Slot, typename Load, typename Use>
__device__ __forceinline__ void step_batches(uint32_t n, Load&& load, Use&& use) {
  uint32_t q = 0;
  for (; q + U <= n; q += U) step_batch<U, Slot>(q, load, use);
  const uint32_t left = n - q;
  each<U>([&](auto i) __attribute__((always_inline)) {
    if constexpr (i > 0)
      if (left == (uint32_t)i) step_batch<i, Slot>(q, load, use);
  });
}

// ---- inputs ------------------------------------------------------------------

// First column of a lane's block j in a step.
template <int KIND>
__device__ __forceinline__ uint32_t input_col(int j) {
  const uint32_t h = (uint32_t)lane_id() >> 4;
  return KIND == kFp4 ? 128u * h + 32u * (uint32_t)j : 32u * h;
}

// Up to 16 input rows.
//   full   loads i = 0 .. 3 take piece lane & 3 of input row 4b + i, and after
//          quad_transpose register k is operand k, with input row r in column r
//   QUAD   up to four input rows: one load, lane 4 b + k has piece k of row b.
//          Operand k multiplies it whole, into sums of its own, of which column
//          4 b + k is what it should be (Sums below): no transposition
// ANY: rows that start at any 2-byte address.
template <bool QUAD, bool ANY>
struct InputTile {
  static constexpr int kLoads = QUAD ? 1 : 4;
  const uint16_t* base;  // wave-uniform
  uint32_t bytes, cols;
  uint32_t row[kLoads];  // the input rows that the lane loads

  // The first n of the rows at x, of c columns each; row_of(i) is the input row
  // for column i of the product.
  template <typename F>
  __device__ __forceinline__ InputTile(const uint16_t* x, uint32_t n, uint32_t c, F&& row_of)
      : base(x), bytes(n * c * 2u), cols(c) {
    const uint32_t r = (uint32_t)lane_id() & 15u;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) row[i] = row_of(QUAD ? r >> 2 : (r & ~3u) + (uint32_t)i);
  }
};

template <bool QUAD>
struct InputBlock {
  u32x4 v[QUAD ? 1 : 4];
};

template <int KIND, bool TAIL, bool QUAD, bool ANY>
__device__ __forceinline__ void load_inputs(const InputTile<QUAD, ANY>& x, uint32_t step, int j,
                                            InputBlock<QUAD>& s) {
  const uint32_t c = input_col<KIND>(j) + 8u * ((uint32_t)lane_id() & 3u);
  const uint32_t at = step * kStepCols<KIND> + c;
#pragma unroll
  for (int i = 0; i < (QUAD ? 1 : 4); ++i) {
    if constexpr (ANY) {
      const uint16_t* row = x.base + (uint64_t)x.row[i] * x.cols;
      s.v[i] = TAIL ? load8(row, at, x.cols) : *(const u32x4_any*)(row + at);
    } else {
      const bool in = !TAIL || at < x.cols;
      s.v[i] = load16(buffer_of(x.base, x.bytes), in ? (x.row[i] * x.cols + c) * 2u : kNowhere,
                      step * kStepCols<KIND> * 2u);
    }
  }
}

template <bool QUAD>
struct Sums {
  mfma_f32x4 v[QUAD ? 4 : 1];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < (QUAD ? 4 : 1); ++j) v[j] = mfma_f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void add(u32x4 weights, const InputBlock<QUAD>& x, int k) {
    v[QUAD ? k : 0] = mfma16(weights, x.v[QUAD ? 0 : k], v[QUAD ? k : 0]);
  }
  // Sums of input row b in every column of quad b (full: of row n in column n).
  __device__ __forceinline__ mfma_f32x4 total() const {
    if constexpr (!QUAD) {
      return v[0];
    } else {
      const uint32_t j = (uint32_t)lane_id() & 3u;
      mfma_f32x4 t;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float s = j == 0 ? v[0][k] : j == 1 ? v[1][k] : j == 2 ? v[2][k] : v[3][k];
        s += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), 0xB1, 0xF, 0xF, true));
        s += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), 0x4E, 0xF, 0xF, true));
        t[k] = s;
      }
      return t;
    }
  }
};

}  // namespace wc
