// wc_moe.hip — a whole mixture-of-experts layer for up to 64 tokens in three
// launches (include/wc_moe.h defines the operator):
//   k_moe_router   logits of every token and expert (matrix cores)
//   k_moe_gate_up  every block chooses the experts again from the logits
//                  (a few waves' work, cheaper than a launch), then walks
//                  (expert, 16 intermediate rows) items: gate and up products,
//                  silu(gate) * up * weight into the workspace
//   k_moe_down     16 output rows per block: the sum over all chosen experts,
//                  kept in the block, so that nothing is added through memory
//                  and the result does not depend on which block ends first
// Each expert's set of tokens is one 64-bit mask, which is what bounds the
// number of tokens of a call.
#include "wc_launch.h"
#include "wc_moe.h"
#include "wc_skinny.h"

namespace wc {

constexpr uint32_t kMoeExperts = WC_MOE_MAX_EXPERTS;
constexpr uint32_t kMoePlaces = WC_MOE_MAX_TOKENS * WC_MOE_MAX_TOP_K;  // (token, choice) pairs
constexpr uint32_t kRouterWaves = 16;
constexpr uint32_t kUpWaves = 4;     // waves per block of k_moe_gate_up
constexpr uint32_t kDownWaves = 16;  // and of k_moe_down

// The products take an expert's tokens in units: of up to 32 in k_moe_gate_up,
// of up to 8 in k_moe_down.
constexpr uint32_t kUpTokens = 32;
constexpr uint32_t kDownTokens = 8;
constexpr uint32_t kUpUnits = kMoeExperts + kMoePlaces / kUpTokens;
constexpr uint32_t kDownUnits = kMoeExperts + kMoePlaces / kDownTokens;

struct MoeUnit {
  uint16_t expert;
  uint16_t place;  // of its first token among the chosen pairs
  uint16_t count;  // its tokens
};

// The choice, as k_moe_down needs it.
struct MoeRoute {
  uint32_t units;
  MoeUnit unit[kDownUnits];
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
  float* logits;  // [tokens][experts]
  MoeRoute* route;
  uint16_t* act;  // operands of k_moe_down: by unit, block, k, lane (act_at below)
  uint32_t tokens, hidden, inter, experts, top_k, scoring, renorm;
  uint32_t act_blocks;  // of 128 columns per unit: inter rounded up to whole steps, the rest 0
  uint32_t down_fp4;    // the order of the columns in a step
  uint32_t most_units;  // bound of MoeRoute::units
  float scale;
};

// Byte offsets in the caller's workspace.
struct MoeWork {
  size_t logits, route, act, total;
};

// Units of k_moe_down at most: every chosen expert's first, and one more for
// every kDownTokens further pairs.
inline uint32_t moe_units(const wc_moe_shape& s, uint32_t size) {
  const uint32_t pairs = s.tokens * s.top_k;
  return (pairs < s.experts ? pairs : s.experts) + (s.tokens > size ? pairs / size : 0u);
}

inline uint32_t moe_act_blocks(uint32_t inter, uint32_t step_cols) {
  return (inter + step_cols - 1u) / step_cols * (step_cols / 128u);
}

inline MoeWork moe_work(const wc_moe_shape& s) {
  MoeWork m;
  m.logits = 0;
  m.route = pad16(m.logits + 4ull * s.tokens * s.experts);
  m.act = pad16(m.route + sizeof(MoeRoute));
  // 4 KB a block; whole 4-bit steps, so that the size does not go by the kind
  m.total = m.act + 4096ull * moe_units(s, kDownTokens) * moe_act_blocks(s.inter, kStepCols<kFp4>);
  return m;
}

// Where column c of a unit's input row n stands in `act`: as the lanes of
// k_moe_down hold it (wc_skinny.h), so that its loads are contiguous.
__device__ __forceinline__ uint64_t act_at(const MoeArgs& a, uint32_t unit, uint32_t n, uint32_t c) {
  const uint32_t block = a.down_fp4 ? (c >> 9) * 4u + (c >> 5 & 3u) : c >> 7;
  const uint32_t h = a.down_fp4 ? c >> 7 & 3u : c >> 5 & 3u;
  return (((uint64_t)unit * a.act_blocks + block) * 4u + (c >> 3 & 3u)) * 512u + (n + 16u * h) * 8u + (c & 7u);
}

// ---- router ------------------------------------------------------------------

// Block = 16 experts x 16 tokens, a run of steps per wave.
template <bool ANY>
__global__ __launch_bounds__(kWave * kRouterWaves) void k_moe_router(MoeArgs a) {
  __shared__ mfma_f32x4 part[kRouterWaves][kWave];
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u;
  const uint32_t e0 = blockIdx.x * kRowTile, t0 = blockIdx.y * kRowTile;
  constexpr int kKind = ANY ? kBf16Any : kBf16;
  const WeightTile<kKind> w(a.router, nullptr, e0, a.experts, a.hidden);
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
  const uint32_t s0 = wave * whole / kRouterWaves, s1 = (wave + 1u) * whole / kRouterWaves;
  step_batches<2, Slot>(
      s1 - s0,
      [&](uint32_t q, Slot& s) __attribute__((always_inline)) {
        load_weights<kKind, false>(w, s0 + q, s.w);
        load_inputs<kKind, false>(x, s0 + q, 0, s.x);
      },
      use);
  if (wave == kRouterWaves - 1u && whole * kStepCols<kKind> < a.hidden) {
    Slot s;
    load_weights<kKind, true>(w, whole, s.w);
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
      float* o = a.logits + (uint64_t)(t0 + r) * a.experts;
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
  uint64_t mask[kMoeExperts];     // tokens of each expert
  uint16_t first[kMoeExperts];    // its first place among the chosen pairs
  uint16_t down_first[kMoeExperts];  // and its first unit of k_moe_down
  MoeUnit unit[kUpUnits];         // units of k_moe_gate_up
  uint32_t units, down_units;
  float weight[kMoePlaces];       // by [token][choice]
  int16_t id[kMoePlaces];
  float place_weight[kMoePlaces]; // by place
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
  const float* row = a.logits + (uint64_t)(real ? t : 0u) * a.experts;
  float logit[PER], score[PER];
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) logit[i] = row[r + kLanes * i < a.experts ? r + kLanes * i : 0u];
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

// One unit of up to `size` of an expert's tokens, at `at` and after.
__device__ inline void fill_units(MoeUnit* unit, uint32_t at, uint32_t e, uint32_t first, uint32_t n,
                                  uint32_t size) {
  for (uint32_t m = 0; m < n; m += size)
    unit[at++] = MoeUnit{(uint16_t)e, (uint16_t)(first + m), (uint16_t)(n - m < size ? n - m : size)};
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
      // three sums of at most 1024 in one scan: places, and units of both kinds
      const uint32_t nu = (n + kUpTokens - 1u) / kUpTokens, nd = (n + kDownTokens - 1u) / kDownTokens;
      const uint32_t before = wave_excl_scan_u32(n | nd << 12 | nu << 24);
      const uint32_t first = places + (before & 0xFFFu);
      if (e < a.experts) {
        c.first[e] = (uint16_t)first;
        c.down_first[e] = (uint16_t)(down + (before >> 12 & 0xFFFu));
      }
      fill_units(c.unit, units + (before >> 24), e, first, n, kUpTokens);
      if (route) fill_units(route->unit, down + (before >> 12 & 0xFFFu), e, first, n, kDownTokens);
      const uint32_t all = wave_total(n | nd << 12 | nu << 24);
      places += all & 0xFFFu;
      down += all >> 12 & 0xFFFu;
      units += all >> 24;
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

// One item: 16 rows of gate and the same 16 of up of one expert, with NT tiles
// of 16 of a unit's tokens; wave `part` of SPLIT takes its run of steps.
template <int KIND, bool ANY, int NT, int U>
__device__ __forceinline__ void gate_up_item(const MoeArgs& a, const MoeChoice& c, const MoeUnit& unit,
                                             uint32_t row0, uint32_t part, uint32_t split,
                                             mfma_f32x4 g[NT], mfma_f32x4 u[NT]) {
  const uint64_t base = (uint64_t)unit.expert * 2u * a.inter;
  // rows past `inter` repeat the last one: sums that are not used
  const WeightTile<KIND> wg(a.gu, a.gu_scales, base + row0, base + a.inter, a.hidden);
  const WeightTile<KIND> wu(a.gu, a.gu_scales, base + a.inter + row0, base + 2u * a.inter, a.hidden);
  auto input = [&](int t) __attribute__((always_inline)) {
    return InputTile<false, ANY>(a.x, a.tokens, a.hidden, [&](uint32_t i) {
      const uint32_t m = 16u * (uint32_t)t + i;  // columns past the unit's tokens repeat its last one
      return (uint32_t)c.place_token[unit.place + (m < unit.count ? m : unit.count - 1u)];
    });
  };
  const InputTile<false, ANY> x0 = input(0), x1 = input(NT - 1);
#pragma unroll
  for (int t = 0; t < NT; ++t) g[t] = u[t] = mfma_f32x4{0, 0, 0, 0};
  constexpr int kB = kBlocks<KIND>;
  struct Slot {
    WeightStep g, u;
    InputBlock<false> x[NT][kB];
  };
  auto use = [&](Slot& s) __attribute__((always_inline)) {
    quad_transpose(s.g.v);
    quad_transpose(s.u.v);
    each<kB>([&](auto j) __attribute__((always_inline)) {
      each<NT>([&](auto t) __attribute__((always_inline)) { quad_transpose(s.x[t][j].v); });
      each<4>([&](auto k) __attribute__((always_inline)) {
        const u32x4 og = weight_operand<KIND>(s.g, j, k), ou = weight_operand<KIND>(s.u, j, k);
        each<NT>([&](auto t) __attribute__((always_inline)) {
          g[t] = mfma16(og, s.x[t][j].v[k], g[t]);
          u[t] = mfma16(ou, s.x[t][j].v[k], u[t]);
        });
      });
    });
  };
  auto load = [&](auto tail, uint32_t step, Slot& s) __attribute__((always_inline)) {
    load_weights<KIND, tail>(wg, step, s.g);
    load_weights<KIND, tail>(wu, step, s.u);
    each<kB>([&](auto j) __attribute__((always_inline)) {
      load_inputs<KIND, tail>(x0, step, j, s.x[0][j]);
      if constexpr (NT == 2) load_inputs<KIND, tail>(x1, step, j, s.x[1][j]);
    });
  };
  const uint32_t whole = a.hidden / kStepCols<KIND>;
  const uint32_t steps = (a.hidden + kStepCols<KIND> - 1u) / kStepCols<KIND>;
  const uint32_t s0 = part * steps / split, s1 = (part + 1u) * steps / split;
  step_batches<U, Slot>(
      (s1 < whole ? s1 : whole) - s0,
      [&](uint32_t q, Slot& s) __attribute__((always_inline)) { load(std::false_type{}, s0 + q, s); }, use);
  if (s1 > whole && s1 > s0) {  // the short last step
    Slot s;
    load(std::true_type{}, whole, s);
    use(s);
  }
}

// MANY: more than 16 tokens in the call, so units may fill two tiles.
// SPLIT waves share an item; the block works on kUpWaves / SPLIT of them.
template <int KIND, bool ANY, bool MANY, uint32_t SPLIT>
__global__ __launch_bounds__(kWave * kUpWaves, MANY ? 2 : 3) void k_moe_gate_up(MoeArgs a) {
  constexpr int NT = MANY ? 2 : 1;
  constexpr uint32_t kItems = kUpWaves / SPLIT;
  __shared__ MoeChoice c;
  __shared__ mfma_f32x4 sums[kUpWaves][2 * NT][kWave];
  choose_all(a, c, blockIdx.x == 0 ? a.route : nullptr);
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t slot = wave / SPLIT, part = wave % SPLIT;
  const uint32_t tiles = (a.inter + kRowTile - 1) / kRowTile, items = c.units * tiles;
  for (uint32_t base = blockIdx.x * kItems; base < items; base += gridDim.x * kItems) {
    const uint32_t item = base + slot;
    const bool on = item < items;
    const MoeUnit unit = c.unit[on ? item / tiles : 0u];
    const uint32_t row0 = item % tiles * kRowTile;
    if (on) {
      if (NT == 1 || unit.count <= 16u) {
        mfma_f32x4 g[1], u[1];
        gate_up_item<KIND, ANY, 1, KIND == kFp4 ? 1 : 2>(a, c, unit, row0, part, SPLIT, g, u);
        sums[wave][0][lane] = g[0];
        sums[wave][1][lane] = u[0];
      } else {
        mfma_f32x4 g[NT], u[NT];
        gate_up_item<KIND, ANY, NT, 1>(a, c, unit, row0, part, SPLIT, g, u);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          sums[wave][2 * t][lane] = g[t];
          sums[wave][2 * t + 1][lane] = u[t];
        }
      }
    }
    __syncthreads();
    // wave `part` of an item finishes its tiles part, part + SPLIT, ..
    for (uint32_t t = part; on && 16u * t < unit.count; t += SPLIT) {
      mfma_f32x4 sg = sums[slot * SPLIT][2 * t][lane], su = sums[slot * SPLIT][2 * t + 1][lane];
#pragma unroll
      for (uint32_t v = 1; v < SPLIT; ++v) {
        sg += sums[slot * SPLIT + v][2 * t][lane];
        su += sums[slot * SPLIT + v][2 * t + 1][lane];
      }
      const uint32_t m = 16u * t + (lane & 15u);
      if (m < unit.count) {
        const uint32_t place = unit.place + m, rank = place - c.first[unit.expert];
        const uint32_t to = c.down_first[unit.expert] + rank / kDownTokens, n = rank % kDownTokens;
        const float p = c.place_weight[place];
        const uint32_t i0 = row0 + 4u * (lane >> 4);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // weight * silu(gate) * up, as the sum of two BF16 (16 bits of it)
          const float h = i0 + k < a.inter ? sg[k] / (1.0f + expf(-sg[k])) * su[k] * p : 0.0f;
          hi[k] = bf16_of(h);
          const float rest = h - __uint_as_float(hi[k] << 16);
          lo[k] = rest == rest ? bf16_of(rest) : 0u;  // h infinite or NaN: the high part says so
        }
        *(uint2*)(a.act + act_at(a, to, n, i0)) = uint2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
        *(uint2*)(a.act + act_at(a, to, n + 8u, i0)) = uint2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
        if (row0 + kRowTile >= a.inter) {
          for (uint32_t i = i0 + kRowTile; i < a.act_blocks * 128u; i += kRowTile) {
            *(uint2*)(a.act + act_at(a, to, n, i)) = uint2{0, 0};
            *(uint2*)(a.act + act_at(a, to, n + 8u, i)) = uint2{0, 0};
          }
        }
      }
    }
    __syncthreads();
  }
}

// ---- down ----------------------------------------------------------------------

// 16 rows of y per block.  Steps are (unit, 128 columns) in unit order, a run of
// them per wave.  A unit's high parts are columns 0..7 of the products, its low
// parts columns 8..15.  When the unit changes, the sums go to the wave's own
// [token][16] array in LDS; at the end these are added over the waves.
template <int KIND, int U>
__global__ __launch_bounds__(kWave * kDownWaves) void k_moe_down(MoeArgs a) {
  extern __shared__ __attribute__((aligned(16))) float ysum[];  // [kDownWaves][tokens][16]
  __shared__ MoeUnit unit[kDownUnits];
  __shared__ uint8_t token[kMoePlaces];
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u, h = lane >> 4;
  const uint32_t units = a.route->units;
  for (uint32_t j = threadIdx.x; j < a.most_units; j += kWave * kDownWaves) unit[j] = a.route->unit[j];
  for (uint32_t j = threadIdx.x; j < a.tokens * a.top_k; j += kWave * kDownWaves) token[j] = a.route->token[j];
  float* const mine = ysum + wave * a.tokens * 16u;
  for (uint32_t j = threadIdx.x; j < kDownWaves * a.tokens * 4u; j += kWave * kDownWaves)
    ((mfma_f32x4*)ysum)[j] = mfma_f32x4{0, 0, 0, 0};
  __syncthreads();

  const uint32_t row0 = blockIdx.x * kRowTile;
  mfma_f32x4 acc = {0, 0, 0, 0};
  uint32_t now = 0xFFFFFFFFu;  // the unit in acc
  auto flush = [&]() __attribute__((always_inline)) {
    if (now == 0xFFFFFFFFu) return;
    const MoeUnit un = unit[now];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float s = acc[k];
      acc[k] = s + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x128, 0xF, 0xF, false));
    }
    if (r < un.count) {
      mfma_f32x4* o = (mfma_f32x4*)(mine + token[un.place + r] * 16u) + h;
      *o += acc;
    }
    acc = mfma_f32x4{0, 0, 0, 0};
  };
  constexpr int kB = kBlocks<KIND>;
  struct Slot {
    WeightStep w;
    u32x4 x[kB][4];
    uint32_t unit;
  };
  auto use = [&](Slot& s) __attribute__((always_inline)) {
    if (s.unit != now) {
      flush();
      now = s.unit;
    }
    quad_transpose(s.w.v);
    each<kB>([&](auto j) __attribute__((always_inline)) {
      each<4>([&](auto k) __attribute__((always_inline)) {
        acc = mfma16(weight_operand<KIND>(s.w, j, k), s.x[j][k], acc);
      });
    });
  };
  const uint32_t whole = a.inter / kStepCols<KIND>;
  const uint32_t per = a.act_blocks / kB;  // steps of a unit, a short last one among them
  const uint32_t steps = units * per;
  const uint32_t s0 = (uint32_t)((uint64_t)wave * steps / kDownWaves);
  const uint32_t s1 = (uint32_t)((uint64_t)(wave + 1u) * steps / kDownWaves);
  uint32_t lu = s0 / per, ls = s0 - lu * per;  // the next step to load
  step_batches<U, Slot>(
      s1 - s0,
      [&](uint32_t, Slot& s) __attribute__((always_inline)) {
        const uint64_t e = (uint32_t)__builtin_amdgcn_readfirstlane((int)unit[lu].expert);
        const WeightTile<KIND> w(a.dn, a.dn_scales, e * a.hidden + row0, (e + 1u) * a.hidden, a.inter);
        if (ls < whole)
          load_weights<KIND, false>(w, ls, s.w);
        else
          load_weights<KIND, true>(w, ls, s.w);
        const u32x4* x = (const u32x4*)a.act + ((uint64_t)lu * a.act_blocks + ls * kB) * (4u * kWave) + lane;
        each<4 * kB>([&](auto i) __attribute__((always_inline)) { s.x[i / 4][i % 4] = x[i * kWave]; });
        s.unit = lu;
        const bool wrap = ls + 1u == per;
        lu += wrap ? 1u : 0u;
        ls = wrap ? 0u : ls + 1u;
      },
      use);
  flush();
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < a.tokens * 16u; i += kWave * kDownWaves) {
    float s = 0.0f;
    for (uint32_t v = 0; v < kDownWaves; ++v) s += ysum[v * a.tokens * 16u + i];
    const uint32_t t = i / 16u, o = row0 + i % 16u;
    if (o < a.hidden) a.y[(uint64_t)t * a.hidden + o] = bf16_of(s);
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
  if (s->scoring > WC_MOE_SIGMOID || (s->flags & ~WC_MOE_RENORM)) return WC_E_ARG;
  return WC_OK;
}

int experts_ok(const wc_moe_experts* e) {
  if (!e || e->kind > WC_MOE_FP4) return WC_E_ARG;
  if (!e->d_data || !aligned16(e->d_data)) return WC_E_ARG;
  if (e->kind == WC_MOE_FP4 && !e->d_scales) return WC_E_ARG;
  return WC_OK;
}

template <int KIND, bool ANY>
void launch_gate_up(const MoeArgs& a, uint32_t units, hipStream_t s) {
  constexpr uint32_t kSplit = 4;
  const dim3 block(kWave * kUpWaves);
  const uint64_t items = (uint64_t)units * ((a.inter + 15u) / 16u);
  const uint64_t most = (uint64_t)cu_count() * 3u;
  auto blocks = [&](uint32_t per) {
    const uint64_t b = (items + per - 1u) / per;
    return (uint32_t)(b < most ? b : most);
  };
  if (a.tokens > 16u)
    k_moe_gate_up<KIND, ANY, true, kSplit><<<blocks(kUpWaves / kSplit), block, 0, s>>>(a);
  else
    k_moe_gate_up<KIND, ANY, false, kSplit><<<blocks(kUpWaves / kSplit), block, 0, s>>>(a);
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
  if (!d_x || !wc::aligned16(d_x) || !d_router || !wc::aligned16(d_router)) return WC_E_ARG;
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

  const dim3 router_grid((a.experts + 15u) / 16u, (a.tokens + 15u) / 16u);
  if (a.hidden % 8u)
    wc::k_moe_router<true><<<router_grid, wc::kWave * wc::kRouterWaves, 0, s>>>(a);
  else
    wc::k_moe_router<false><<<router_grid, wc::kWave * wc::kRouterWaves, 0, s>>>(a);
  if (hipGetLastError() != hipSuccess) return WC_E_HIP;

  const uint32_t up_units = wc::moe_units(*shape, wc::kUpTokens);
  a.most_units = wc::moe_units(*shape, wc::kDownTokens);
  a.down_fp4 = down->kind == WC_MOE_FP4;
  a.act_blocks = wc::moe_act_blocks(a.inter, a.down_fp4 ? wc::kStepCols<wc::kFp4> : wc::kStepCols<wc::kBf16>);
  const bool any = a.hidden % 8u != 0;  // rows that do not start at 16-byte boundaries
  if (gate_up->kind == WC_MOE_FP4)
    any ? wc::launch_gate_up<wc::kFp4, true>(a, up_units, s) : wc::launch_gate_up<wc::kFp4, false>(a, up_units, s);
  else
    any ? wc::launch_gate_up<wc::kBf16Any, true>(a, up_units, s)
        : wc::launch_gate_up<wc::kBf16, false>(a, up_units, s);
  if (hipGetLastError() != hipSuccess) return WC_E_HIP;

  const uint32_t row_blocks = (a.hidden + 15u) / 16u;
  const size_t lds = (size_t)wc::kDownWaves * a.tokens * 16u * sizeof(float);
  const dim3 block(wc::kWave * wc::kDownWaves);
  if (down->kind == WC_MOE_FP4)
    wc::k_moe_down<wc::kFp4, 1><<<row_blocks, block, lds, s>>>(a);
  else if (a.inter % 8u)
    wc::k_moe_down<wc::kBf16Any, 2><<<row_blocks, block, lds, s>>>(a);
  else
    wc::k_moe_down<wc::kBf16, 2><<<row_blocks, block, lds, s>>>(a);
  return hipGetLastError() == hipSuccess ? WC_OK : WC_E_HIP;
}
