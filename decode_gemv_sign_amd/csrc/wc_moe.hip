// wc_moe.hip — a whole mixture-of-experts layer for up to 64 tokens in three
// launches (include/wc_moe.h defines the operator):
//   k_moe_router   logits of every token and expert (matrix cores)
//   k_moe_gate_up  every block chooses the experts again from the logits
//                  (a few waves' work, cheaper than a launch), then works on its
//                  share of the (expert, 16 intermediate rows) tiles: gate and up
//                  products, silu(gate) * up * weight into the workspace
//   k_moe_down     16 output rows per block: the sum over all chosen experts,
//                  kept in the block (or in two or four that split the experts
//                  where the rows are too few for the card), so that nothing is
//                  added through memory in an order that could change
// Each expert's set of tokens is one 64-bit mask, which is what bounds the
// number of tokens of a call.
#include "wc_launch.h"
#include "wc_moe.h"
#include "wc_skinny.h"

namespace wc {

constexpr uint32_t kMoeExperts = WC_MOE_MAX_EXPERTS;
constexpr uint32_t kMoePlaces = WC_MOE_MAX_TOKENS * WC_MOE_MAX_TOP_K;  // (token, choice) pairs
constexpr uint32_t kRouterWaves = 8;
constexpr uint32_t kMaxSplits = 4;   // column splits of the router
constexpr uint32_t kUpWaves = 12;    // waves per block of k_moe_gate_up, one block per compute unit
constexpr uint32_t kDownWaves = 16;  // and of k_moe_down
constexpr uint32_t kMaxParts = 4;    // blocks of k_moe_down on the same rows

// The products take an expert's tokens in units: in k_moe_gate_up of up to 16,
// and of no more than its LDS holds inputs for; in k_moe_down of up to 8, each as
// a high and a low part.
constexpr uint32_t kUpInputs = 128u * 1024u;  // bytes of LDS
constexpr uint32_t kDownTokens = 8;

struct MoeUnit {
  uint16_t expert;
  uint16_t place;  // of its first token among the chosen pairs
  uint16_t count;  // its tokens
  uint16_t pair;   // k_moe_gate_up: 0 for an expert's only unit, else 1; k_moe_down:
                   // 1 and 2 for two units that go together, else 0
};

// The choice, as k_moe_down needs it.
struct MoeRoute {
  uint32_t units;
  MoeUnit unit[kMoePlaces];
  uint8_t token[kMoePlaces];  // by place
};

struct MoeArgs {
  const uint16_t* x;
  const uint16_t* router;
  const float* bias;
  const void* gu;
  const uint8_t* gu_scales;
  const void* dn;
  const uint8_t* dn_scales;
  uint16_t* y;
  int32_t* ids;
  float* weights;
  float* logits;      // [splits][tokens][experts]: sums over a split of the columns
  MoeRoute* route;
  uint16_t* act;      // operands of k_moe_down (act_at below)
  uint32_t* arrived;  // blocks of k_moe_down that are done, by row tile
  float* partial;     // their sums, [row tile][part][tokens][16]
  uint32_t tokens, hidden, inter, experts, top_k, scoring, renorm;
  uint32_t splits;      // of the router's columns
  uint32_t up_tokens;   // most tokens of a unit of k_moe_gate_up
  uint32_t up_inputs;   // tokens whose inputs its LDS holds
  uint32_t act_blocks;  // of 128 columns per unit: inter rounded up to whole steps, the rest 0
  uint32_t down_fp4;    // the order of the columns in a step
  uint32_t parts;       // blocks of k_moe_down on the same rows
  float scale;
};

// Byte offsets in the caller's workspace.
struct MoeWork {
  size_t logits, route, act, arrived, partial, total;
};

inline uint32_t moe_blocks(uint32_t cols, uint32_t step_cols) {  // of 128 columns, in whole steps
  return (cols + step_cols - 1u) / step_cols * (step_cols / 128u);
}

// Most tokens of a unit of k_moe_gate_up: what its LDS holds in whole 4-bit steps.
inline uint32_t moe_up_tokens(uint32_t hidden) {
  const uint32_t n = kUpInputs / (moe_blocks(hidden, kStepCols<kFp4>) * 256u);
  return n > 16u ? 16u : n;
}

inline MoeWork moe_work(const wc_moe_shape& s) {
  MoeWork m;
  const uint64_t tiles = (s.hidden + 15u) / 16u;
  m.logits = 0;
  m.route = pad16(m.logits + 4ull * kMaxSplits * s.tokens * s.experts);
  m.act = pad16(m.route + sizeof(MoeRoute));
  // 512 bytes a pair and block; whole 4-bit steps, so that the size does not go by the kind
  m.arrived = m.act + 512ull * s.tokens * s.top_k * moe_blocks(s.inter, kStepCols<kFp4>);
  m.partial = pad16(m.arrived + 4u * tiles);
  m.total = m.partial + 64ull * kMaxParts * s.tokens * tiles;
  return m;
}

// Columns of a row go to the lanes of the matrix operands in pieces of 8
// (wc_skinny.h): piece q of a row is piece k of lanes h in a block.
struct Piece {
  uint32_t block, k, h;
};
template <bool FP4>
__device__ __forceinline__ Piece piece_of(uint32_t q) {
  return FP4 ? Piece{(q >> 6) * 4u + (q >> 2 & 3u), q & 3u, q >> 4 & 3u} : Piece{q >> 4, q & 3u, q >> 2 & 3u};
}

// Where pieces of the operands of `count` rows stand, in pieces: [block][k][h][row],
// so that what 64 lanes ask for at a time is contiguous and no larger than the
// rows there are.
__device__ __forceinline__ uint32_t operand_at(uint32_t block, uint32_t k, uint32_t h, uint32_t count, uint32_t row) {
  return ((block * 4u + k) * 4u + h) * count + row;
}

// `act` of a unit of k_moe_down: 2 * count rows, of token i the high part at 2 i
// and the low part at 2 i + 1.
__device__ __forceinline__ u32x4* act_of(const MoeArgs& a, const MoeUnit& u) {
  return (u32x4*)a.act + (uint64_t)u.place * (32u * a.act_blocks);
}

// ---- router ------------------------------------------------------------------

// Block = 16 experts x 16 tokens x a split of the columns, a run of steps per wave.
// The router is small (128 x 4096: 1 MB): what it takes is launch and one trip to
// memory, 3.6 us with 64 experts of 2048 columns and 5 with 128 of 4096, so the
// columns are spread over blocks until a wave has one step.
template <bool ANY>
__global__ __launch_bounds__(kWave * kRouterWaves) void k_moe_router(MoeArgs a) {
  __shared__ mfma_f32x4 part[kRouterWaves][kWave];
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u;
  const uint32_t e0 = blockIdx.x * kRowTile, t0 = blockIdx.y * kRowTile;
  // the counters that k_moe_down's blocks count in
  if (blockIdx.y == 0 && blockIdx.z == 0)
    for (uint32_t i = blockIdx.x * (kWave * kRouterWaves) + threadIdx.x; i < (a.hidden + 15u) / 16u;
         i += gridDim.x * (kWave * kRouterWaves))
      a.arrived[i] = 0;
  constexpr int kKind = ANY ? kBf16Any : kBf16;
  const WeightLane<kKind> lw(a.hidden);
  const WeightTile<kKind> w(a.router, nullptr, e0, a.experts, lw);
  const InputTile<false, ANY> x(a.x, a.tokens, a.hidden,
                                [&](uint32_t i) { return t0 + i < a.tokens ? t0 + i : a.tokens - 1u; });
  mfma_f32x4 acc = {0, 0, 0, 0};
  struct Slot {
    WeightStep w;
    InputBlock<false> x;
  };
  auto use = [&](Slot& s) __attribute__((always_inline)) {
    quad_transpose(s.w.v);
    quad_transpose(s.x.v);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc = mfma16(s.w.v[k], s.x.v[k], acc);
  };
  const uint32_t whole = a.hidden / kStepCols<kKind>;
  const uint32_t at = blockIdx.z * kRouterWaves + wave, waves = a.splits * kRouterWaves;
  const uint32_t s0 = at * whole / waves, s1 = (at + 1u) * whole / waves;
  step_batches<2, Slot>(
      s1 - s0,
      [&](uint32_t q, Slot& s) __attribute__((always_inline)) {
        load_weights<kKind, false>(lw, w, s0 + q, s.w);
        load_inputs<kKind, false>(x, s0 + q, 0, s.x);
      },
      use);
  if (at == waves - 1u && whole * kStepCols<kKind> < a.hidden) {
    Slot s;
    load_weights<kKind, true>(lw, w, whole, s.w);
    load_inputs<kKind, true>(x, whole, 0, s.x);
    use(s);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    mfma_f32x4 s = part[0][lane];
#pragma unroll
    for (int v = 1; v < kRouterWaves; ++v) s += part[v][lane];
    if (t0 + r < a.tokens) {
      float* o = a.logits + ((uint64_t)blockIdx.z * a.tokens + t0 + r) * a.experts;
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t ee = e0 + 4u * (lane >> 4) + k;
        if (ee < a.experts) o[ee] = s[k];
      }
    }
  }
}

// ---- choice of the experts -----------------------------------------------------

// Reductions over the 16 lanes of a row, by rotations, or (WIDE) over the wave:
// every lane gets the result, with the same bits.
template <bool WIDE, typename F>
__device__ inline uint32_t row_reduce(uint32_t v, F&& f) {
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));  // row_ror:8
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));  // row_ror:4
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));  // row_ror:2
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));  // row_ror:1
  if constexpr (WIDE) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16, kWave));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32, kWave));
  }
  return v;
}
template <bool WIDE>
__device__ inline uint32_t row_max(uint32_t v) {
  return row_reduce<WIDE>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <bool WIDE>
__device__ inline uint32_t row_min(uint32_t v) {
  return row_reduce<WIDE>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <bool WIDE>
__device__ inline uint32_t row_or(uint32_t v) {
  return row_reduce<WIDE>(v, [](uint32_t a, uint32_t b) { return a | b; });
}
template <bool WIDE>
__device__ inline float row_sum(float v) {
  return __uint_as_float(row_reduce<WIDE>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// An unsigned key in the order of the values: -inf lowest (but above 0, the
// key of what cannot be chosen), NaN highest, -0 and +0 the same.
__device__ inline uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ inline float key_value(uint32_t k) {
  return __uint_as_float(k == 0xFFFFFFFFu ? k : k >> 31 ? k & 0x7FFFFFFFu : ~k);
}

struct MoeChoice {
  uint64_t mask[kMoeExperts];        // tokens of each expert
  uint16_t first[kMoeExperts];       // its first place among the chosen pairs
  MoeUnit unit[kMoePlaces];          // units of k_moe_gate_up
  uint32_t units;
  int16_t id[kMoePlaces];            // by [token][choice]
  float weight[kMoePlaces];
  float place_weight[kMoePlaces];    // by place
  uint8_t place_token[kMoePlaces];
};

// The choice of one token by 16 lanes, four tokens side by side in a wave, or
// (WIDE) by 64: lane r holds PER experts, r and every kLanes-th after it.
// t >= tokens does nothing but keep step.
template <int PER, bool WIDE>
__device__ inline void choose(const MoeArgs& a, uint32_t t, MoeChoice& c) {
  constexpr uint32_t kLanes = WIDE ? 64u : 16u;
  const uint32_t r = (uint32_t)lane_id() & (kLanes - 1u);
  const bool real = t < a.tokens;
  float logit[PER], score[PER], more[kMaxSplits][PER];
  uint32_t key[PER];
#pragma unroll
  for (uint32_t s = 0; s < kMaxSplits; ++s) {  // all loads together
    const float* row = a.logits + ((uint64_t)(s < a.splits ? s : 0u) * a.tokens + (real ? t : 0u)) * a.experts;
#pragma unroll
    for (int i = 0; i < PER; ++i) more[s][i] = row[r + kLanes * i < a.experts ? r + kLanes * i : 0u];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    logit[i] = more[0][i];
#pragma unroll
    for (uint32_t s = 1; s < kMaxSplits; ++s)
      if (s < a.splits) logit[i] += more[s][i];
  }
  if (a.scoring == WC_MOE_SOFTMAX) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t k = r + kLanes * i < a.experts ? order_key(logit[i]) : 0u;
      top = top > k ? top : k;
    }
    const float most = key_value(row_max<WIDE>(top));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      score[i] = expf(logit[i] - most);
      if (r + kLanes * i < a.experts) sum += score[i];
    }
    sum = row_sum<WIDE>(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] = 1.0f / (1.0f + expf(-logit[i]));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t e = r + kLanes * i;
    if (a.bias) {
      const float b = a.bias[e < a.experts ? e : 0u];
      key[i] = b == -INFINITY ? 0u : order_key(score[i] + b);
    } else {
      key[i] = order_key(logit[i]);
    }
    if (e >= a.experts) key[i] = 0;
  }
  float sum = 0.0f, mine = 0.0f;  // lane j keeps choice j
  int my_id = -1;
  for (uint32_t j = 0; j < a.top_k; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = top > key[i] ? top : key[i];
    top = row_max<WIDE>(top);
    uint32_t at = 0xFFFFu;  // the lowest expert with that key
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == top) at = r + kLanes * i;
    at = row_min<WIDE>(at);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (r + kLanes * i == at) {
        w = __float_as_uint(score[i]);
        key[i] = 0;
      }
    const float v = __uint_as_float(row_or<WIDE>(w));
    if (top != 0) {  // 0: nothing left to choose
      sum += v;
      if (r == j) {
        mine = v;
        my_id = (int)at;
      }
    }
  }
  if (a.renorm) mine = sum == 0.0f ? 0.0f : mine / sum;
  mine *= a.scale;
  if (real && r < a.top_k) {
    c.id[t * a.top_k + r] = (int16_t)my_id;
    c.weight[t * a.top_k + r] = my_id < 0 ? 0.0f : mine;
    if (my_id >= 0) atomicOr((unsigned long long*)&c.mask[my_id], 1ull << t);  // order does not matter
  }
}

// Units of up to `size` of an expert's tokens, at `at` and after; `pairs`: for
// k_moe_down.
__device__ inline void fill_units(MoeUnit* unit, uint32_t at, uint32_t e, uint32_t first, uint32_t n,
                                  uint32_t size, bool pairs) {
  for (uint32_t m = 0; m < n; m += size) {
    const bool second = m / size & 1u, one = !second && m + size >= n;
    unit[at++] = MoeUnit{(uint16_t)e, (uint16_t)(first + m), (uint16_t)(n - m < size ? n - m : size),
                         (uint16_t)(!pairs ? n > size : one ? 0 : second ? 2 : 1)};
  }
}

// The whole block: every token's choice, then the experts' places and units.
// `route`: where k_moe_down's part goes, or null.
__device__ inline void choose_all(const MoeArgs& a, MoeChoice& c, MoeRoute* route) {
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  for (uint32_t e = threadIdx.x; e < a.experts; e += kWave * kUpWaves) c.mask[e] = 0;
  __syncthreads();
  if (a.experts <= 64u) {
    for (uint32_t t = 4u * wave; t < a.tokens; t += 4u * kUpWaves) choose<4, false>(a, t + (lane >> 4), c);
  } else if (a.experts <= 128u) {
    for (uint32_t t = 4u * wave; t < a.tokens; t += 4u * kUpWaves) choose<8, false>(a, t + (lane >> 4), c);
  } else {
    for (uint32_t t = wave; t < a.tokens; t += kUpWaves) choose<8, true>(a, t, c);
  }
  __syncthreads();
  if (wave == 0) {
    uint32_t places = 0, units = 0, down = 0;
    for (uint32_t e0 = 0; e0 < a.experts; e0 += kWave) {
      const uint32_t e = e0 + lane;
      const uint32_t n = e < a.experts ? (uint32_t)__popcll(c.mask[e]) : 0u;
      const uint32_t nu = (n + a.up_tokens - 1u) / a.up_tokens, nd = (n + kDownTokens - 1u) / kDownTokens;
      const uint32_t pb = wave_excl_scan_u32(n), ub = wave_excl_scan_u32(nu | nd << 16);
      const uint32_t first = places + pb;
      if (e < a.experts) c.first[e] = (uint16_t)first;
      fill_units(c.unit, units + (ub & 0xFFFFu), e, first, n, a.up_tokens, false);
      if (route) fill_units(route->unit, down + (ub >> 16), e, first, n, kDownTokens, true);
      const uint32_t all = wave_total(nu | nd << 16);
      places += wave_total(n);
      units += all & 0xFFFFu;
      down += all >> 16;
    }
    if (lane == 0) {
      c.units = units;
      if (route) route->units = down;
    }
  }
  __syncthreads();
  for (uint32_t p = threadIdx.x; p < a.tokens * a.top_k; p += kWave * kUpWaves) {
    const int id = c.id[p];
    if (id >= 0) {
      const uint32_t t = p / a.top_k;
      const uint32_t at = c.first[id] + (uint32_t)__popcll(c.mask[id] & ((1ull << t) - 1ull));
      c.place_weight[at] = c.weight[p];
      c.place_token[at] = (uint8_t)t;
      if (route) route->token[at] = (uint8_t)t;
    }
    if (route) {
      if (a.ids) a.ids[p] = id;
      if (a.weights) a.weights[p] = c.weight[p];
    }
  }
  __syncthreads();
}

// ---- gate and up ---------------------------------------------------------------

// A block's share of the tiles (unit, 16 rows of gate and the same 16 of up) is
// one run of them, unit by unit, which it takes in as few parts as the inputs of
// their tokens fit LDS, mostly one.  The inputs come there in operand order; then
// the steps of all the part's tiles are shared out evenly: each wave takes one run
// of steps, and a tile that several waves worked on is joined in LDS, in wave
// order.  A wave loads one step ahead: its runs are long, and past the end it does
// not load.
// The weights of experts with one unit of tokens pass the caches by; those of more
// units do not, as the next tile reads them again (64 tokens, 8 experts of 2048 x 4096,
// 2 each: 122 us for the layer, 129 if they do).
// Bound by HBM where there are many weights (bytes fetched, by the counters): BF16, 32
// experts of 2048 x 4096, 2 tokens, 4 each: 235 MB in 46 us, 5.1 TB/s; 64 experts of
// 1024 x 2048, 64 tokens: 540 MB in 100 us, 5.4 TB/s; 4-bit, 128 experts of 1024 x 4096,
// 16 tokens: 343 MB in 68 us, 5.1 TB/s.  One token of 64 experts of 1408 x 2048, 4-bit:
// 19 MB in 14 us, most of it the launch, the choice, which every block makes before its
// first load of weights, and the inputs.
template <int KIND>
__global__ __launch_bounds__(kWave * kUpWaves, 3) void k_moe_gate_up(MoeArgs a) {
  __shared__ MoeChoice c;
  extern __shared__ __attribute__((aligned(16))) u32x4 inputs[];  // then sums[kUpWaves][2][2][kWave]
  mfma_f32x4* const sums = (mfma_f32x4*)inputs;
  choose_all(a, c, blockIdx.x == 0 ? a.route : nullptr);
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u, h = lane >> 4;
  constexpr bool kIsFp4 = KIND == kFp4;
  constexpr int kB = kBlocks<KIND>;
  const uint32_t tiles = (a.inter + kRowTile - 1u) / kRowTile, items = c.units * tiles;
  const uint32_t whole = a.hidden / kStepCols<KIND>;
  const uint32_t steps = (a.hidden + kStepCols<KIND> - 1u) / kStepCols<KIND>;
  const WeightLane<KIND> lw(a.hidden);
  const uint32_t end = (blockIdx.x + 1u) * items / gridDim.x;

  // The tile's sums g and u, for the unit's tokens: into act.
  auto finish = [&](const MoeUnit& unit, uint32_t tile, mfma_f32x4 g, mfma_f32x4 u) __attribute__((always_inline)) {
    if (r >= unit.count) return;
    const uint32_t place = unit.place + r, rank = place - c.first[unit.expert];
    const uint32_t n = (uint32_t)__popcll(c.mask[unit.expert]);
    const uint32_t m0 = rank / kDownTokens * kDownTokens;  // its unit of k_moe_down
    const uint32_t rows = 2u * (n - m0 < kDownTokens ? n - m0 : kDownTokens);
    uint2* const act = (uint2*)act_of(a, MoeUnit{0, (uint16_t)(c.first[unit.expert] + m0), 0, 0});
    auto put = [&](uint32_t col, uint2 hi, uint2 lo) __attribute__((always_inline)) {
      const Piece p = a.down_fp4 ? piece_of<true>(col >> 3) : piece_of<false>(col >> 3);
      const uint32_t at = 2u * operand_at(p.block, p.k, p.h, rows, 2u * (rank - m0)) + (col >> 2 & 1u);
      act[at] = hi;
      act[at + 2u] = lo;
    };
    const float weight = c.place_weight[place];
    const uint32_t i0 = tile * kRowTile + 4u * h;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // weight * silu(gate) * up, as the sum of two BF16 (16 bits of it).  A finite v that
      // rounds past BF16's range keeps its largest number and leaves the rest to the low part.
      const float v = i0 + k < a.inter ? g[k] / (1.0f + expf(-g[k])) * u[k] * weight : 0.0f;
      hi[k] = bf16_of(v);
      if ((hi[k] & 0x7FFFu) == 0x7F80u && fabsf(v) < INFINITY) --hi[k];
      const float rest = v - __uint_as_float(hi[k] << 16);
      lo[k] = rest == rest ? bf16_of(rest) : 0u;  // v infinite or NaN: the high part says so
    }
    put(i0, uint2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16}, uint2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16});
    if (tile + 1u == tiles)
      for (uint32_t i = i0 + kRowTile; i < a.act_blocks * 128u; i += kRowTile) put(i, uint2{0, 0}, uint2{0, 0});
  };

  for (uint32_t item = blockIdx.x * items / gridDim.x; item < end;) {
    const uint32_t item0 = item, unit0 = item0 / tiles, place0 = c.unit[unit0].place;
    uint32_t unit1 = unit0 + 1u;  // the part's units: all that the block has, or that fit
    while (unit1 * tiles < end && c.unit[unit1].place + c.unit[unit1].count - place0 <= a.up_inputs) ++unit1;
    item = end < unit1 * tiles ? end : unit1 * tiles;
    const uint32_t total = (item - item0) * steps;
    const uint32_t f0 = wave * total / kUpWaves, f1 = (wave + 1u) * total / kUpWaves;
    const uint64_t rows = (uint64_t)a.experts * 2u * a.inter;
    const uint32_t pieces = steps * kB * 16u;  // of a token's inputs
    mfma_f32x4 g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
    mfma_f32x4 g0 = g, u0 = u;  // of the wave's first tile, when it is not the last
    uint32_t done = 0;          // whether that is so
    // the next step to load: unit, tile, step; and to use
    const uint32_t first = item0 + f0 / steps;
    uint32_t lu = first / tiles, lt = first - lu * tiles, ls = f0 % steps;
    uint32_t uu = lu, ut = lt, us = ls;
    const bool starts = ls == 0;  // the first tile has no steps before this wave
    auto advance = [&](uint32_t& unit, uint32_t& tile, uint32_t& step) __attribute__((always_inline)) {
      if (++step < steps) return;
      step = 0;
      if (++tile < tiles) return;
      tile = 0;
      ++unit;
    };
    struct Slot {
      WeightStep g, u;
    };
    auto load = [&](Slot& s) __attribute__((always_inline)) {
      const uint64_t e = (uint32_t)__builtin_amdgcn_readfirstlane((int)c.unit[lu].expert);
      const uint64_t row = e * 2u * a.inter + lt * kRowTile;
      const WeightTile<KIND> wg(a.gu, a.gu_scales, row, rows, lw);
      const WeightTile<KIND> wu(a.gu, a.gu_scales, row + a.inter, rows, lw);
      if (ls >= whole) {
        load_weights<KIND, true>(lw, wg, ls, s.g);
        load_weights<KIND, true>(lw, wu, ls, s.u);
      } else if (c.unit[lu].pair == 0) {
        load_weights<KIND, false, true>(lw, wg, ls, s.g);
        load_weights<KIND, false, true>(lw, wu, ls, s.u);
      } else {
        load_weights<KIND, false>(lw, wg, ls, s.g);
        load_weights<KIND, false>(lw, wu, ls, s.u);
      }
      advance(lu, lt, ls);
    };
    auto use = [&](Slot& s) __attribute__((always_inline)) {
      const MoeUnit unit = c.unit[uu];
      const u32x4* in = inputs + (unit.place - place0) * pieces;
      const uint32_t mine = r < unit.count ? r : unit.count - 1u;  // columns past the tokens repeat the last one
      quad_transpose(s.g.v);
      quad_transpose(s.u.v);
      each<kB>([&](auto j) __attribute__((always_inline)) {
        each<4>([&](auto k) __attribute__((always_inline)) {
          const u32x4 x = in[operand_at(us * kB + j, k, h, unit.count, mine)];
          g = mfma16(weight_operand<KIND>(s.g, j, k), x, g);
          u = mfma16(weight_operand<KIND>(s.u, j, k), x, u);
        });
      });
      if (us + 1u == steps) {  // the tile's last step
        if (starts || done) {
          finish(unit, ut, g, u);
        } else {
          g0 = g;
          u0 = u;
        }
        done = 1;
        g = u = mfma_f32x4{0, 0, 0, 0};
      }
      advance(uu, ut, us);
    };
    Slot now, next;
    if (f0 < f1) load(now);  // on its way while the inputs come in
    // inputs, unit by unit as [block][k][h][token]
    for (uint32_t un = unit0; un < unit1; ++un) {
      const MoeUnit unit = c.unit[un];
      u32x4* in = inputs + (unit.place - place0) * pieces;
      for (uint32_t i = threadIdx.x; i < pieces * unit.count; i += kWave * kUpWaves) {
        const uint32_t t = i / pieces, q = i - t * pieces;
        const uint16_t* row = a.x + (uint64_t)c.place_token[unit.place + t] * a.hidden;
        const Piece p = piece_of<kIsFp4>(q);
        in[operand_at(p.block, p.k, p.h, unit.count, t)] =
            8u * q + 8u <= a.hidden ? *(const u32x4_any*)(row + 8u * q) : load8(row, 8u * q, a.hidden);
      }
    }
    __syncthreads();
    if (f0 < f1) {
      // a step is loaded while the one before it is used
      for (uint32_t f = f0 + 1u; f < f1; ++f) {
        load(next);
        __builtin_amdgcn_sched_barrier(0);
        use(now);
        now = next;
      }
      use(now);
    }
    // Tiles shared with other waves: sums[wave][0] is the wave's part of its first
    // tile, [1] of its last one.  Tile t's steps t * steps .. are those of waves
    // w0 .. w1, and w1 joins them.
    __syncthreads();
    if (f1 > f0) {
      const bool ended = us == 0;  // its last tile is whole, or ends here
      if (!starts && done) {
        sums[(wave * 4u + 0u) * kWave + lane] = g0;
        sums[(wave * 4u + 1u) * kWave + lane] = u0;
      }
      if (!ended) {
        const uint32_t slot = !starts && !done ? 0u : 2u;  // the first tile itself, or a later one
        sums[(wave * 4u + slot) * kWave + lane] = g;
        sums[(wave * 4u + slot + 1u) * kWave + lane] = u;
      }
    }
    __syncthreads();
    if (f1 > f0 && !starts && done) {
      const uint32_t t = f0 / steps;
      // the first wave with a step of tile t: the last w with w * total / kUpWaves <= t * steps
      uint32_t w0 = wave;
      while (w0 > 0 && w0 * total / kUpWaves > t * steps) --w0;
      mfma_f32x4 sg = {0, 0, 0, 0}, su = {0, 0, 0, 0};
      for (uint32_t v = w0; v <= wave; ++v) {
        const uint32_t v0 = v * total / kUpWaves;
        if (v0 == (v + 1u) * total / kUpWaves) continue;  // no steps
        const uint32_t slot = v0 > t * steps ? 0u : 2u;  // inside its first tile, or at the tile's start or before
        sg += sums[(v * 4u + slot) * kWave + lane];
        su += sums[(v * 4u + slot + 1u) * kWave + lane];
      }
      const uint32_t un = (item0 + t) / tiles;
      finish(c.unit[un], item0 + t - un * tiles, sg, su);
    }
    __syncthreads();
  }
}

// ---- down ----------------------------------------------------------------------

// 16 rows of y per block, or per a.parts blocks.  Steps are (unit, columns) in unit
// order, a run of them per part, and of that per wave; an expert's units go two by
// two, taking turns at the same columns, so that its weights come from memory once
// for 16 tokens (64 tokens, 8 of 64 experts each: 60 us and 1.08 times the weights'
// bytes, against 63 and 1.44); units without a second one pass the caches by (58).  Lane column n takes the high part of token
// n & 7 of the unit, or (n >= 8) the low part.  When a unit is done, its sums go to
// the wave's own [token][16] array in LDS; at the end these are added over the
// waves, and over the parts by the last block to arrive, in order both.
// BF16, 2 tokens as above: 118 MB fetched in 21.3 us, 5.6 TB/s; 4-bit, 16 tokens: 174 MB
// in 38 to 44 us; one token: 10 MB in 7.7 us.  12 waves took the same as 16; the
// operands of the activations loaded by quads and transposed here instead of stored
// in operand order by k_moe_gate_up spilled registers and took longer.
template <int KIND, int U>
__global__ __launch_bounds__(kWave * kDownWaves) void k_moe_down(MoeArgs a) {
  extern __shared__ __attribute__((aligned(16))) float ysum[];  // [kDownWaves][tokens][16]
  __shared__ MoeUnit unit[kMoePlaces];
  __shared__ uint8_t token[kMoePlaces];
  __shared__ uint32_t before;
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u, h = lane >> 4;
  const uint32_t units = a.route->units, pairs = a.tokens * a.top_k;
  for (uint32_t j = threadIdx.x; j < pairs; j += kWave * kDownWaves) {  // there are no more units than pairs
    unit[j] = a.route->unit[j];
    token[j] = a.route->token[j];
  }
  float* const mine = ysum + wave * a.tokens * 16u;
  for (uint32_t j = threadIdx.x; j < kDownWaves * a.tokens * 4u; j += kWave * kDownWaves)
    ((mfma_f32x4*)ysum)[j] = mfma_f32x4{0, 0, 0, 0};
  __syncthreads();

  const uint32_t row0 = blockIdx.x * kRowTile;
  mfma_f32x4 acc = {0, 0, 0, 0}, other = acc;
  uint32_t now = 0xFFFFFFFFu, then = now;  // the units in acc and in other
  auto flush = [&](mfma_f32x4& acc, uint32_t which) __attribute__((always_inline)) {
    if (which == 0xFFFFFFFFu) return;
    const MoeUnit un = unit[which];
    // lane r < 8 adds the sum of its token's low parts (lane r + 8) to that of the high parts.
    // Where the latter is infinite or NaN it is the result: an infinite weight times a
    // low part of 0 or of the other sign would make it NaN.
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float s = acc[k];
      const float low = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x128, 0xF, 0xF, false));
      acc[k] = fabsf(s) < INFINITY ? s + low : s;
    }
    if (r < un.count) {
      mfma_f32x4* o = (mfma_f32x4*)(mine + token[un.place + r] * 16u) + h;
      *o += acc;
    }
  };
  constexpr int kB = kBlocks<KIND>;
  struct Slot {
    WeightStep w;
    u32x4 x[kB][4];
    uint32_t unit;
  };
  const WeightLane<KIND> lw(a.inter);
  const uint32_t whole = a.inter / kStepCols<KIND>;
  const uint32_t per = a.act_blocks / kB;  // steps of a unit, a short last one among them
  const uint32_t waves = a.parts * kDownWaves, at = blockIdx.y * kDownWaves + wave;
  const uint32_t s0 = at * (units * per) / waves;
  const uint32_t s1 = (at + 1u) * (units * per) / waves;
  uint32_t lu = s0 / per, ls = s0 - lu * per;  // the next step to load
  if (s0 < s1 && unit[lu].pair) {
    const uint32_t first = lu + 1u - unit[lu].pair, at = s0 - first * per;
    lu = first + (at & 1u);
    ls = at >> 1;
  }
  step_batches<U, Slot>(
      s1 - s0,
      [&](uint32_t, Slot& s) __attribute__((always_inline)) {
        const MoeUnit un = unit[lu];
        const uint64_t e = (uint32_t)__builtin_amdgcn_readfirstlane((int)un.expert);
        const WeightTile<KIND> w(a.dn, a.dn_scales, e * a.hidden + row0, (uint64_t)a.experts * a.hidden, lw);
        if (ls >= whole)
          load_weights<KIND, true>(lw, w, ls, s.w);
        else if (un.pair == 0)
          load_weights<KIND, false, true>(lw, w, ls, s.w);
        else
          load_weights<KIND, false>(lw, w, ls, s.w);
        const uint32_t i = r & 7u, last = un.count - 1u;  // columns past the tokens repeat the last one
        const u32x4* x = act_of(a, un) + 2u * (i < last ? i : last) + (r >> 3);
        each<4 * kB>([&](auto q) __attribute__((always_inline)) {
          s.x[q / 4][q % 4] = x[operand_at(ls * kB + q / 4, q % 4, h, 2u * un.count, 0)];
        });
        s.unit = lu;
        if (un.pair == 1u) {
          ++lu;
        } else if (++ls == per) {
          ++lu;
          ls = 0;
        } else if (un.pair == 2u) {
          --lu;
        }
      },
      [&](Slot& s) __attribute__((always_inline)) {
        if (s.unit != now) {
          const mfma_f32x4 last = acc;
          if (s.unit == then) {
            acc = other;
          } else {
            flush(other, then);
            acc = mfma_f32x4{0, 0, 0, 0};
          }
          other = last;
          then = now;
          now = s.unit;
        }
        quad_transpose(s.w.v);
        each<kB>([&](auto j) __attribute__((always_inline)) {
          each<4>([&](auto k) __attribute__((always_inline)) {
            acc = mfma16(weight_operand<KIND>(s.w, j, k), s.x[j][k], acc);
          });
        });
      });
  flush(other, then);
  flush(acc, now);
  __syncthreads();
  const uint32_t n = a.tokens * 16u;
  float* const parts = a.partial + (uint64_t)blockIdx.x * a.parts * n;
  for (uint32_t i = threadIdx.x; i < n; i += kWave * kDownWaves) {
    float s = 0.0f;
    for (uint32_t v = 0; v < kDownWaves; ++v) s += ysum[v * n + i];
    if (a.parts == 1u) {
      const uint32_t o = row0 + i % 16u;
      if (o < a.hidden) a.y[(uint64_t)(i / 16u) * a.hidden + o] = bf16_of(s);
    } else {
      __hip_atomic_store(&parts[blockIdx.y * n + i], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (a.parts == 1u) return;
  // The sums are stored and loaded as agent-scope atomics, which go past the
  // caches that the card's dies do not share; a wait for the stores then orders
  // them before the arrival.  (A fence would write back the whole L2: 85 us.)
  wait_vm<0>();
  __syncthreads();
  if (threadIdx.x == 0)
    before = __hip_atomic_fetch_add(&a.arrived[blockIdx.x], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (before + 1u != a.parts) return;
  for (uint32_t i = threadIdx.x; i < n; i += kWave * kDownWaves) {
    float s = 0.0f;
    for (uint32_t v = 0; v < a.parts; ++v)
      s += __hip_atomic_load(&parts[v * n + i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t o = row0 + i % 16u;
    if (o < a.hidden) a.y[(uint64_t)(i / 16u) * a.hidden + o] = bf16_of(s);
  }
}

namespace {

int moe_shape_ok(const wc_moe_shape* s) {
  if (!s) return WC_E_ARG;
  if (s->tokens < 1 || s->tokens > WC_MOE_MAX_TOKENS) return WC_E_UNSUPPORTED;
  if (s->experts < 1 || s->experts > WC_MOE_MAX_EXPERTS) return WC_E_UNSUPPORTED;
  if (s->top_k < 1 || s->top_k > WC_MOE_MAX_TOP_K || s->top_k > s->experts) return WC_E_UNSUPPORTED;
  if (s->hidden < 1 || s->hidden > WC_MOE_MAX_DIM || s->inter < 1 || s->inter > WC_MOE_MAX_DIM)
    return WC_E_UNSUPPORTED;
  static_assert(WC_MOE_MAX_DIM * 2u <= 128u * 1024u, "one token's inputs fit k_moe_gate_up's LDS");
  if (s->scoring > WC_MOE_SIGMOID || (s->flags & ~WC_MOE_RENORM)) return WC_E_ARG;
  return WC_OK;
}

int experts_ok(const wc_moe_experts* e) {
  if (!e || e->kind > WC_MOE_FP4) return WC_E_ARG;
  if (!e->d_data || !aligned16(e->d_data)) return WC_E_ARG;
  if (e->kind == WC_MOE_FP4 && !e->d_scales) return WC_E_ARG;
  return WC_OK;
}

}  // namespace
}  // namespace wc

extern "C" size_t wc_moe_workspace_bytes(const wc_moe_shape* shape) {
  return wc::moe_shape_ok(shape) == WC_OK ? wc::moe_work(*shape).total : 0;
}

extern "C" int wc_moe(const wc_moe_shape* shape, const uint16_t* d_x, const uint16_t* d_router,
                      const float* d_bias, const wc_moe_experts* gate_up,
                      const wc_moe_experts* down, uint16_t* d_y, int32_t* d_ids, float* d_weights,
                      void* d_work, size_t work_bytes, void* stream) {
  if (const int v = wc::moe_shape_ok(shape)) return v;
  if (const int v = wc::experts_ok(gate_up)) return v;
  if (const int v = wc::experts_ok(down)) return v;
  if (!wc::rows_aligned(d_x, shape->hidden) || !d_router || !wc::aligned16(d_router)) return WC_E_ARG;
  if (!d_y || ((uintptr_t)d_y & 1u)) return WC_E_ARG;
  if (((uintptr_t)d_bias | (uintptr_t)d_ids | (uintptr_t)d_weights) & 3u) return WC_E_ARG;
  if (!d_work || !wc::aligned16(d_work)) return WC_E_ARG;
  const wc::MoeWork m = wc::moe_work(*shape);
  if (work_bytes < m.total) return WC_E_SIZE;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* work = (uint8_t*)d_work;
  wc::MoeArgs a = {};
  a.x = d_x;
  a.router = d_router;
  a.bias = d_bias;
  a.gu = gate_up->d_data;
  a.gu_scales = gate_up->d_scales;
  a.dn = down->d_data;
  a.dn_scales = down->d_scales;
  a.y = d_y;
  a.ids = d_ids;
  a.weights = d_weights;
  a.logits = (float*)(work + m.logits);
  a.route = (wc::MoeRoute*)(work + m.route);
  a.act = (uint16_t*)(work + m.act);
  a.tokens = shape->tokens;
  a.hidden = shape->hidden;
  a.inter = shape->inter;
  a.experts = shape->experts;
  a.top_k = shape->top_k;
  a.scoring = shape->scoring;
  a.renorm = shape->flags & WC_MOE_RENORM;
  a.scale = shape->scale;

  a.arrived = (uint32_t*)(work + m.arrived);
  a.partial = (float*)(work + m.partial);
  a.up_tokens = wc::moe_up_tokens(a.hidden);
  a.down_fp4 = down->kind == WC_MOE_FP4;
  a.act_blocks = wc::moe_blocks(a.inter, a.down_fp4 ? wc::kStepCols<wc::kFp4> : wc::kStepCols<wc::kBf16>);
  const uint32_t row_blocks = (a.hidden + 15u) / 16u, cus = wc::cu_count();
  a.parts = 1;
  // rows too few for the card, and at least some steps for every wave
  const uint64_t steps = (uint64_t)a.tokens * a.top_k * a.act_blocks / (a.down_fp4 ? 4u : 1u);
  while (a.parts < wc::kMaxParts && 4u * row_blocks * a.parts < 3u * cus &&
         steps >= 4u * wc::kDownWaves * a.parts)
    a.parts *= 2u;

  // one step per wave up to 4096 columns: the router is small, its loads should go out together
  const uint32_t router_steps = (a.hidden + 127u) / 128u;
  a.splits = (router_steps + wc::kRouterWaves - 1u) / wc::kRouterWaves;
  if (a.splits > wc::kMaxSplits) a.splits = wc::kMaxSplits;
  const dim3 router_grid((a.experts + 15u) / 16u, (a.tokens + 15u) / 16u, a.splits);
  const bool any = a.hidden % 8u != 0;  // rows that do not start at 16-byte boundaries
  if (any)
    wc::k_moe_router<true><<<router_grid, wc::kWave * wc::kRouterWaves, 0, s>>>(a);
  else
    wc::k_moe_router<false><<<router_grid, wc::kWave * wc::kRouterWaves, 0, s>>>(a);
  if (hipGetLastError() != hipSuccess) return WC_E_HIP;

  // tiles there are at least when every pair has an expert of its own, or all share
  const uint32_t pairs = a.tokens * a.top_k;
  const uint64_t items = (uint64_t)pairs * ((a.inter + 15u) / 16u);
  const uint32_t blocks = (uint32_t)(items < cus ? items : cus);
  const size_t sums = (size_t)wc::kUpWaves * 4u * wc::kWave * sizeof(wc::mfma_f32x4);
  const uint32_t token_bytes = 256u *
      wc::moe_blocks(a.hidden, gate_up->kind == WC_MOE_FP4 ? wc::kStepCols<wc::kFp4> : wc::kStepCols<wc::kBf16>);
  a.up_inputs = wc::kUpInputs / token_bytes;
  if (a.up_inputs > pairs) a.up_inputs = pairs;
  const size_t in = (size_t)a.up_inputs * token_bytes;
  const size_t lds_up = in > sums ? in : sums;
  const dim3 up_block(wc::kWave * wc::kUpWaves);
  if (gate_up->kind == WC_MOE_FP4)
    wc::k_moe_gate_up<wc::kFp4><<<blocks, up_block, lds_up, s>>>(a);
  else if (any)
    wc::k_moe_gate_up<wc::kBf16Any><<<blocks, up_block, lds_up, s>>>(a);
  else
    wc::k_moe_gate_up<wc::kBf16><<<blocks, up_block, lds_up, s>>>(a);
  if (hipGetLastError() != hipSuccess) return WC_E_HIP;

  const size_t lds = (size_t)wc::kDownWaves * a.tokens * 16u * sizeof(float);
  const dim3 block(wc::kWave * wc::kDownWaves), grid(row_blocks, a.parts);
  if (a.down_fp4)
    wc::k_moe_down<wc::kFp4, 1><<<grid, block, lds, s>>>(a);
  else if (a.inter % 8u)
    wc::k_moe_down<wc::kBf16Any, 2><<<grid, block, lds, s>>>(a);
  else
    wc::k_moe_down<wc::kBf16, 2><<<grid, block, lds, s>>>(a);
  return hipGetLastError() == hipSuccess ? WC_OK : WC_E_HIP;
}
