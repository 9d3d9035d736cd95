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
// Blocks walk the rows' pieces of 8 columns, 4 G per row.  Bound by HBM:
// 24576 x 6144 in 66 us, 382 MB at 5.8 TB/s (a plain copy of 2 GiB: 4.9); 73 us with
// loads that leave the weights, which nothing reads again, in the caches.  Four loads
// in flight per lane took longer.  1000 x 4100: 4.2 us, of which 2.4 are an empty
// kernel's.
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
    const uint16_t* from = w + row * cols;
    const u32x4 v =
        c + 8u <= cols ? (u32x4)__builtin_nontemporal_load((const u32x4_any*)(from + c)) : load8(from, c, cols);
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

// A lane rebuilds 8 columns.  Bound by HBM: 24576 x 6144 in 72 us with all 387 MB to and
// from there, 5.4 TB/s (75 with stores that stay in the caches); 57 right after
// k_fp4_encode, whose codes are then still in the memory-side cache.  1000 x 4100: 4.0 us.
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
      __builtin_nontemporal_store((u32x4_any)v, (u32x4_any*)o);
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
  uint64_t rows;    // of this launch
  uint64_t stride;  // floats from one input's outputs to the next one's
  uint32_t cols, batch;
};

// y = W x, the codes rebuilt as BF16 operands (exact: a magnitude has two bits)
// and summed in fp32 by the matrix cores.  16 rows per block, up to 16 input rows
// (QUAD: up to 4, each input loaded once, with no transposition; Sums in
// wc_skinny.h).  Each wave takes a run
// of the steps, and their sums are added in LDS in wave order.  Input rows past
// the batch repeat the last one and are not stored.  ANY: rows of inputs that do
// not start at 16-byte boundaries.
// At one to four inputs it is bound by memory.  24576 x 6144, batch 1: 80 MB from HBM in
// 20.5 us, 3.9 TB/s (6.2 is the most a read-only kernel reached from there); 17 where
// the memory-side cache holds them (three such matrices in turn).  14336 x 4096, batch 4:
// 32 MB in 10.1 us, cached 8.4, of which 2.4 are an empty kernel's.  A small call is
// launch and one trip to memory: 1024 x 4096 in 4.2 us, cached 3.7.  At 5 to 16 the
// inputs' loads and their transposition count as much as the codes: 5003 rows, batch
// 16: 4096 columns 8.9 us, 4104 (a short last step) 10.6, 4100 (rows at 8-byte
// boundaries besides) 11.9, 4101 13.6; cached 7.2, 8.5, 10.3 and 11.9.  Loading several
// steps at once, or as a pipeline, took longer at every size: the loads are bound by
// their address cycles, not by their latency.
template <bool QUAD, bool ANY>
__global__ __launch_bounds__(kWave * 16) void k_fp4_gemv(Fp4Args a) {
  extern __shared__ mfma_f32x4 part[];  // [waves][kWave]
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t waves = blockDim.x / kWave;
  const uint64_t row0 = (uint64_t)blockIdx.x * kRowTile;
  const uint32_t b0 = blockIdx.y * kRowTile;
  const uint32_t nb = a.batch - b0 < kRowTile ? a.batch - b0 : kRowTile;
  const WeightLane<kFp4> lw(a.cols);
  const WeightTile<kFp4> w(a.codes, a.scales, row0, a.rows, lw);
  const InputTile<QUAD, ANY> x(a.x + (uint64_t)b0 * a.cols, nb, a.cols,
                               [&](uint32_t i) { return i < nb ? i : nb - 1u; });
  Sums<QUAD> acc;
  acc.clear();
  struct Slot {
    WeightStep w;
    InputBlock<QUAD> x[4];
  };
  auto use = [&](Slot& s) __attribute__((always_inline)) {
    quad_transpose(s.w.v);
    each<4>([&](auto j) __attribute__((always_inline)) {
      if constexpr (!QUAD) quad_transpose(s.x[j].v);
      each<4>([&](auto k) __attribute__((always_inline)) {
        acc.add(weight_operand<kFp4>(s.w, j, k), s.x[j], k);
      });
    });
  };
  const uint32_t whole = a.cols / kStepCols<kFp4>;
  const uint32_t steps = (a.cols + kStepCols<kFp4> - 1u) / kStepCols<kFp4>;
  const uint32_t s0 = wave * steps / waves, s1 = (wave + 1u) * steps / waves;
  step_batches<1, Slot>(
      (s1 < whole ? s1 : whole) - s0,
      [&](uint32_t q, Slot& s) __attribute__((always_inline)) {
        load_weights<kFp4, false>(lw, w, s0 + q, s.w);
        each<4>([&](auto j) __attribute__((always_inline)) {
          load_inputs<kFp4, false>(x, s0 + q, j, s.x[j]);
        });
      },
      use);
  if (s1 > whole && s1 > s0) {  // the short last step
    Slot s;
    load_weights<kFp4, true>(lw, w, whole, s.w);
    each<4>([&](auto j) __attribute__((always_inline)) { load_inputs<kFp4, true>(x, whole, j, s.x[j]); });
    use(s);
  }
  part[wave * kWave + lane] = acc.total();
  __syncthreads();
  if (wave == 0) {
    mfma_f32x4 s = part[lane];
    for (uint32_t v = 1; v < waves; ++v) s += part[v * kWave + lane];
    const uint32_t n = lane & 15u, b = b0 + (QUAD ? n >> 2 : n);
    const uint64_t y0 = row0 + 4u * (lane >> 4);
    if (b < a.batch && !(QUAD && (n & 3u))) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (y0 + k < a.rows) a.y[b * a.stride + y0 + k] = s[k];
    }
  }
}

// Larger batches: MT x 16 weight rows by NT x 16 input rows per block, each of
// its waves a run of the steps.  The inputs come to the wave's own part of LDS, by
// buffer loads into LDS, D / 2 blocks of 128 columns (wc_skinny.h) at a time and as
// many ahead: load i of a tile takes, lane 4b + k (+ 16 h), piece k of input row
// 4b + i, so quads read 64 contiguous bytes, and the operand reads do the
// transposition; 16 bytes of padding after every load put the pieces that one
// operand read takes at a time in different banks.  Two blocks at a time are the
// two halves of the cache lines of the inputs, which one at a time are mostly
// fetched twice (8192 x 8192, batch 32: 14.2 us against 16.2); the larger tiles
// take one, as LDS has to hold two such blocks per compute unit (24576 x 6144,
// batch 64: 43.9 against 48.6).  Nothing is shared between waves until the end, so
// there is no barrier for their loads to wait at.
// 6144 x 24576, batch 32: 83 MB in 28 to 33 us where the memory-side cache holds the
// codes, 38 from HBM.  Without the inputs' loads it took 22 (cached), without the
// codes' 31, without the products as long: it waits for the inputs, 1.5 MB from L2 per
// compute unit, and its 192 blocks leave a quarter of the units idle.  4096 x 4096,
// batch 256: 18.6 us, 460 TFLOP/s, of which the blocks' first loads and the launch are
// about 5.
constexpr uint32_t kWideLoad = 1024u + 16u;
constexpr uint32_t kWideWaves = 4;

// Loads before it are issued before loads after it.
__device__ __forceinline__ void load_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int MT, int NT, int D>
__global__ __launch_bounds__(kWave * kWideWaves) void k_fp4_wide(Fp4Args a) {
  constexpr uint32_t kBuf = NT * 4u * kWideLoad;
  constexpr int P = D / 2;
  constexpr int kCodeLoads = 5;  // of a step of a tile: four of codes, one of scales
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // [kWideWaves][D][kBuf], then the sums
  const uint32_t lane = (uint32_t)lane_id(), kg = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u, h = lane >> 4;
  const uint64_t row0 = (uint64_t)blockIdx.x * (kRowTile * MT);
  const uint32_t b0 = blockIdx.y * (kRowTile * NT);
  uint8_t* const mine = lds + kg * (D * kBuf);
  const uint32_t steps = (a.cols + kStepCols<kFp4> - 1u) / kStepCols<kFp4>;
  const uint32_t whole = a.cols / kStepCols<kFp4>;
  const uint32_t s0 = kg * steps / kWideWaves, s1 = (kg + 1u) * steps / kWideWaves;
  // the lane's places in the inputs: at most 64 rows of 32 MiB
  const uint32_t nb = a.batch - b0 < NT * 16u ? a.batch - b0 : NT * 16u;
  const uint16_t* const x0 = a.x + (uint64_t)b0 * a.cols;
  const uint32_t c0 = 128u * h + 8u * (lane & 3u);
  uint32_t x[NT * 4];  // in bytes
  each<NT * 4>([&](auto i) __attribute__((always_inline)) {
    const uint32_t b = (i / 4u) * 16u + (r & ~3u) + i % 4u;
    x[i] = ((b < nb ? b : nb - 1u) * a.cols + c0) * 2u;
  });
  // blocks j .. j + P - 1; the two halves of a cache line one after the other
  auto stage = [&](uint32_t s, auto j) __attribute__((always_inline)) {
    const buffer from = buffer_of(x0, nb * a.cols * 2u);
    each<NT * 4 * P>([&](auto i) __attribute__((always_inline)) {
      load16_lds(from, mine + ((j + i % P) % D) * kBuf + (i / P) * kWideLoad, x[i / P],
                 s * (kStepCols<kFp4> * 2u) + 64u * (j + i % P));
    });
  };
  const WeightLane<kFp4> lw(a.cols);
  WeightStep w[MT];
  // tiles past the last row repeat the first one and are not stored
  auto codes = [&](uint32_t s, auto tail, WeightStep* to) __attribute__((always_inline)) {
    each<MT>([&](auto m) __attribute__((always_inline)) {
      const uint64_t at = row0 + 16u * m;
      const WeightTile<kFp4> t(a.codes, a.scales, at < a.rows ? at : row0, a.rows, lw);
      load_weights<kFp4, tail>(lw, t, s, to[m]);
    });
  };
  mfma_f32x4 acc[MT][NT];
  each<MT * NT>([&](auto i) __attribute__((always_inline)) { acc[i / NT][i % NT] = mfma_f32x4{0, 0, 0, 0}; });
  auto use = [&](auto j) __attribute__((always_inline)) {
    const uint8_t* in = mine + (j % D) * kBuf + (r & 3u) * kWideLoad + (4u * (r >> 2) + 16u * h) * 16u;
    each<4>([&](auto k) __attribute__((always_inline)) {
      u32x4 xs[NT];
      each<NT>([&](auto t) __attribute__((always_inline)) { xs[t] = *(const u32x4*)(in + t * 4u * kWideLoad + 16u * k); });
      each<MT>([&](auto m) __attribute__((always_inline)) {
        const u32x4 op = weight_operand<kFp4>(w[m], j, k);
        each<NT>([&](auto t) __attribute__((always_inline)) { acc[m][t] = mfma16(op, xs[t], acc[m][t]); });
      });
    });
  };
  // A whole step, and (MORE) the loads of the one after it.
  auto step = [&](uint32_t s, auto more) __attribute__((always_inline)) {
    each<MT>([&](auto m) __attribute__((always_inline)) { quad_transpose(w[m].v); });
    WeightStep next[MT];
    each<4>([&](auto j) __attribute__((always_inline)) {
      if constexpr (j % P == 0) {
        // blocks j .. j + P - 1 are in when no load is left but those of the next
        // step's codes, which at j == P were asked for after them
        wait_vm<(more && j == P ? MT * kCodeLoads : 0)>();
        wait_lgkm0();  // the buffers to fill have been read
        wave_lds_sync();
        constexpr int kTo = j + P;
        if constexpr (kTo < 4) stage(s, std::integral_constant<int, kTo>{});
        if constexpr (kTo >= 4 && more) stage(s + 1u, std::integral_constant<int, kTo - 4>{});
        load_fence();
      }
      if constexpr (j == 0 && more) {
        codes(s + 1u, std::false_type{}, next);
        load_fence();
      }
      use(j);
    });
    if constexpr (more) each<MT>([&](auto m) __attribute__((always_inline)) { w[m] = next[m]; });
  };
  const uint32_t end = s1 < whole ? s1 : whole;
  if (s0 < end) {
    codes(s0, std::false_type{}, w);
    load_fence();
    stage(s0, std::integral_constant<int, 0>{});
    load_fence();
    for (uint32_t s = s0; s + 1u < end; ++s) step(s, std::true_type{});
    step(end - 1u, std::false_type{});
  }
  if (s1 > whole && s0 < s1) {  // the short last step; cols is a multiple of 8: a piece is in or out
    codes(whole, std::true_type{}, w);
    each<MT>([&](auto m) __attribute__((always_inline)) { quad_transpose(w[m].v); });
    each<4>([&](auto j) __attribute__((always_inline)) {
      const uint32_t c = whole * kStepCols<kFp4> + 32u * j;
      wait_lgkm0();
      each<NT * 4>([&](auto i) __attribute__((always_inline)) {
        *(u32x4*)(mine + (j % D) * kBuf + i * kWideLoad + 16u * lane) =
            c + c0 < a.cols ? *(const u32x4*)((const uint8_t*)(x0 + c) + x[i]) : u32x4{0, 0, 0, 0};
      });
      wait_lgkm0();
      wave_lds_sync();
      use(j);
    });
  }
  // the waves' sums, in order
  __syncthreads();
  mfma_f32x4* const part = (mfma_f32x4*)lds;  // [kWideWaves][MT][NT][kWave]
  each<MT * NT>([&](auto i) __attribute__((always_inline)) {
    part[(kg * MT * NT + i) * kWave + lane] = acc[i / NT][i % NT];
  });
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < MT * NT * kWave; i += kWave * kWideWaves) {
    mfma_f32x4 s = part[i];
#pragma unroll
    for (uint32_t v = 1; v < kWideWaves; ++v) s += part[v * (MT * NT * kWave) + i];
    const uint32_t l = i % kWave, t = i / kWave % NT, m = i / (kWave * NT);
    const uint32_t b = b0 + 16u * t + (l & 15u);
    const uint64_t y0 = row0 + 16u * m + 4u * (l >> 4);
    if (b < a.batch) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (y0 + k < a.rows) a.y[b * a.stride + y0 + k] = s[k];
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

// Waves per block: the blocks of a compute unit, all resident at once, share 16
// (at up to 128 registers), and no wave is without a step.
template <bool QUAD>
void launch_rows(const Fp4Args& a, uint32_t row_blocks, uint32_t batch_blocks, hipStream_t s) {
  const uint32_t steps = (a.cols + kStepCols<kFp4> - 1u) / kStepCols<kFp4>;
  const uint32_t per_cu = (row_blocks + cu_count() - 1u) / cu_count();
  uint32_t waves = per_cu < 16u ? 16u / per_cu : 1u;
  waves = waves < steps ? waves : (steps ? steps : 1u);
  const dim3 grid(row_blocks, batch_blocks);
  const size_t lds = waves * kWave * sizeof(mfma_f32x4);
  if (a.cols % 8u == 0)
    k_fp4_gemv<QUAD, false><<<grid, kWave * waves, lds, s>>>(a);
  else
    k_fp4_gemv<QUAD, true><<<grid, kWave * waves, lds, s>>>(a);
}

template <int MT, int NT, int D>
void launch_wide(const Fp4Args& a, hipStream_t s) {
  const uint32_t row_blocks = (uint32_t)((a.rows + MT * 16u - 1u) / (MT * 16u));
  const size_t in = (size_t)kWideWaves * D * NT * 4u * kWideLoad, sums = (size_t)kWideWaves * MT * NT * 1024u;
  k_fp4_wide<MT, NT, D><<<dim3(row_blocks, (a.batch + 16u * NT - 1u) / (16u * NT)), kWave * kWideWaves,
                           in > sums ? in : sums, s>>>(a);
}

// Every block reads the inputs of its batch tiles whole, so the largest tile whose
// blocks fill five eighths of the compute units is the fastest: 64 rows by 64 inputs
// against 64 by 32 at 8192 x 8192: batch 128 30.6 us and 34.1, batch 64 (128 blocks
// of the larger) 25.6 and 19.8; 64 by 32 against 32 by 32 at 14336 x 4096, batch 32:
// 13.9 and 16.2, at 8192 x 8192 (128 of the larger) 18.0 and 14.2; 32 by 32
// against 32 by 16 at 4096 x 4096: batch 64 8.3 and 8.9, batch 32 (128) 7.5 and 6.3.
uint32_t wide_blocks(const Fp4Args& a, uint32_t mt, uint32_t nt) {
  return (uint32_t)((a.rows + 16u * mt - 1u) / (16u * mt)) * ((a.batch + 16u * nt - 1u) / (16u * nt));
}
uint32_t wide_enough() { return cu_count() * 5u / 8u; }

void launch_wide_for(const Fp4Args& a, hipStream_t s) {
  if (a.batch > 32 && wide_blocks(a, 4, 4) >= wide_enough())
    launch_wide<4, 4, 2>(a, s);
  else if (a.batch > 16 && wide_blocks(a, 4, 2) >= wide_enough())
    launch_wide<4, 2, 2>(a, s);
  else if (a.batch > 16 && wide_blocks(a, 2, 2) >= wide_enough())
    launch_wide<2, 2, 4>(a, s);
  else
    launch_wide<2, 1, 4>(a, s);
}

void launch_gemv(const Fp4Args& a, hipStream_t s) {
  const uint32_t row_blocks = (uint32_t)((a.rows + kRowTile - 1u) / kRowTile);
  if (a.batch <= 4)
    launch_rows<true>(a, row_blocks, 1, s);
  else if (a.cols % 8u || (a.batch <= 16 && wide_blocks(a, 2, 1) < wide_enough()))
    launch_rows<false>(a, row_blocks, (a.batch + 15u) / 16u, s);
  else
    launch_wide_for(a, s);
}

// Most rows of one launch: a grid has fewer than 2^32 threads in x, and k_fp4_wide of
// 32 rows takes 8 for a row (k_fp4_gemv, which has one wave per block by then, 4).
constexpr uint64_t kLaunchRows = 1ull << 28;

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
  if (cols && (!d_codes || !wc::aligned16(d_codes) || !d_scales || !wc::rows_aligned(d_x, cols)))
    return WC_E_ARG;
  if (rows >= (1ull << 35)) return WC_E_SIZE;  // cols 0
  for (uint64_t r = 0; r < rows; r += wc::kLaunchRows) {
    const uint64_t n = rows - r < wc::kLaunchRows ? rows - r : wc::kLaunchRows;
    wc::launch_gemv({d_codes + WC_FP4_CODE_BYTES(r, cols), d_scales + WC_FP4_SCALE_BYTES(r, cols), d_x,
                     d_y + r, n, rows, (uint32_t)cols, batch}, (hipStream_t)stream);
    if (const int v = wc::launched()) return v;
  }
  return WC_OK;
}
