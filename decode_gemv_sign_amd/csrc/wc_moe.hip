// wc_moe.hip — a whole mixture-of-experts layer for up to 64 tokens in three
// launches (include/wc_moe.h defines the operator):
//   k_moe_router   logits of every token and expert (matrix cores)
//   k_moe_gate_up  every block chooses the experts again from the logits
//                  (a few waves' work, cheaper than a launch), then walks
//                  (expert, 16 intermediate rows) items: gate and up products,
//                  silu(gate) * up * weight as BF16 into the workspace
//   k_moe_down     16 output rows per block: the sum over all chosen experts
//                  in registers, so that nothing is added through memory and
//                  the result does not depend on which block ends first
// Each expert's set of tokens is one 64-bit mask, which is what bounds the
// number of tokens of a call.
#include "wc_launch.h"
#include "wc_moe.h"
#include "wc_skinny.h"

namespace wc {

constexpr uint32_t kMoeExperts = WC_MOE_MAX_EXPERTS;
constexpr uint32_t kMoePlaces = WC_MOE_MAX_TOKENS * WC_MOE_MAX_TOP_K;  // (token, choice) pairs
constexpr int kMoeWaves = 8;  // waves per block of all three kernels

// What k_moe_down needs to know of the choice: the experts that some token
// chose, in index order, each with its tokens and its first row of `act`.
struct MoeRoute {
  uint32_t count;
  uint32_t reserved[3];
  uint64_t mask[kMoeExperts];
  uint32_t expert[kMoeExperts];
  uint32_t first[kMoeExperts];
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
  float* logits;   // [splits][tokens][experts] partial sums
  MoeRoute* route;
  uint16_t* act;   // BF16 [chosen pairs][act_stride]
  uint32_t tokens, hidden, inter, experts, top_k, scoring, renorm;
  uint32_t splits, split_steps;  // router: column splits, steps of each
  uint32_t act_stride;
  float scale;
};

// Byte offsets in the caller's workspace.
struct MoeWork {
  size_t logits, route, act, total;
  uint32_t splits, split_steps, act_stride;
};

inline MoeWork moe_work(const wc_moe_shape& s) {
  MoeWork m;
  const uint32_t steps = (s.hidden + kStep - 1) / kStep;
  // one step per wave and block: the router is a few hundred KB, so what
  // counts is that its loads go out together
  m.splits = (steps + kMoeWaves - 1) / kMoeWaves;
  if (m.splits > 8u) m.splits = 8u;
  m.split_steps = (steps + m.splits - 1) / m.splits;
  m.act_stride = (s.inter + 7u) & ~7u;
  m.logits = 0;
  m.route = pad16(m.logits + 4ull * m.splits * s.tokens * s.experts);
  m.act = pad16(m.route + sizeof(MoeRoute));
  m.total = pad16(m.act + 2ull * s.tokens * s.top_k * m.act_stride);
  return m;
}

// ---- router ------------------------------------------------------------------

// Block = 16 experts x 16 tokens x one split of the columns; the waves take
// the split's steps in turn.
__global__ __launch_bounds__(kWave * kMoeWaves) void k_moe_router(MoeArgs a) {
  __shared__ mfma_f32x4 part[kMoeWaves][kWave];
  const int lane = lane_id(), wave = wave_in_block();
  const uint32_t r = (uint32_t)lane & 15u;
  const uint32_t e0 = blockIdx.x * kRowTile, t0 = blockIdx.y * kRowTile, split = blockIdx.z;
  const uint32_t e = e0 + r < a.experts ? e0 + r : a.experts - 1u;
  const uint32_t t = t0 + r < a.tokens ? t0 + r : a.tokens - 1u;
  const WeightRow w = weight_row<kBf16>(a.router, nullptr, e, a.hidden);
  const uint16_t* x = a.x + (uint64_t)t * a.hidden;
  const uint32_t steps = (a.hidden + kStep - 1) / kStep;
  const uint32_t s0 = split * a.split_steps;
  const uint32_t s1 = s0 + a.split_steps < steps ? s0 + a.split_steps : steps;
  mfma_f32x4 acc = {0, 0, 0, 0};
  for (uint32_t s = s0 + (uint32_t)wave; s < s1; s += kMoeWaves) {
    WeightStep<kBf16> ws;
    u32x4 xs[4];
    load_weights<kBf16>(w, s, a.hidden, ws);
    load_inputs<kBf16>(x, s, a.hidden, xs);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = mfma16(ws.v[j], xs[j], acc);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    mfma_f32x4 s = part[0][lane];
#pragma unroll
    for (int v = 1; v < kMoeWaves; ++v) s += part[v][lane];
    if (t0 + r < a.tokens) {
      float* o = a.logits + ((uint64_t)split * a.tokens + t0 + r) * a.experts;
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t ee = e0 + 4u * ((uint32_t)lane >> 4) + k;
        if (ee < a.experts) o[ee] = s[k];
      }
    }
  }
}

// ---- choice of the experts -----------------------------------------------------

__device__ inline uint32_t wave_max_u32(uint32_t v) {
  auto take = [&](uint32_t o) { v = v > o ? v : o; };
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));  // row_shr:1
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));  // row_shr:2
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));  // row_shr:4
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));  // row_shr:8
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));  // row_bcast:15
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}

// An unsigned key in the order of the values: -inf lowest (but above 0, the
// key of what cannot be chosen), NaN highest, -0 and +0 the same.
__device__ inline uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

struct MoeChoice {
  uint64_t mask[kMoeExperts];    // tokens of each expert
  uint32_t first[kMoeExperts];   // its first place among the chosen pairs
  uint16_t active[kMoeExperts];  // experts with tokens, in index order
  float pair_weight[kMoePlaces];   // by place: the weight, and the token
  uint8_t pair_token[kMoePlaces];
  float weight[kMoePlaces];        // by [token][choice]
  int16_t id[kMoePlaces];
  uint32_t count;                  // experts with tokens
};

// One token's choice by one wave: lane l holds experts l, l + 64, ..
template <int PER>
__device__ inline void choose(const MoeArgs& a, uint32_t t, MoeChoice& c) {
  const uint32_t lane = (uint32_t)lane_id();
  float logit[PER], score[PER];
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t e = lane + 64u * i;
    logit[i] = 0.0f;
    for (uint32_t s = 0; s < a.splits; ++s)
      if (e < a.experts) logit[i] += a.logits[((uint64_t)s * a.tokens + t) * a.experts + e];
  }
  if (a.scoring == WC_MOE_SOFTMAX) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64u * i < a.experts) {
        const uint32_t k = order_key(logit[i]);
        top = top > k ? top : k;
      }
    top = wave_max_u32(top);
    // the largest logit back from its key (NaN stays NaN)
    const float most = __uint_as_float(top == 0xFFFFFFFFu ? top : top >> 31 ? top & 0x7FFFFFFFu : ~top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      score[i] = expf(logit[i] - most);
      if (lane + 64u * i < a.experts) sum += score[i];
    }
    sum = wave_sum_f32(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] = 1.0f / (1.0f + expf(-logit[i]));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t e = lane + 64u * i;
    key[i] = 0;
    if (e < a.experts) {
      if (a.bias) {
        const float b = a.bias[e];
        key[i] = b == -INFINITY ? 0u : order_key(score[i] + b);
      } else {
        key[i] = order_key(logit[i]);
      }
    }
  }
  float sum = 0.0f, mine = 0.0f;  // lane j keeps choice j
  int my_id = -1;
  for (uint32_t j = 0; j < a.top_k; ++j) {
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = top > key[i] ? top : key[i];
    top = wave_max_u32(top);
    if (top == 0) break;  // nothing left to choose
    int id = -1;
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (id < 0) {
        const uint64_t at = __ballot(key[i] == top);
        if (at) {
          const int l = __ffsll((unsigned long long)at) - 1;
          id = l + 64 * i;
          w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(score[i]), l));
          if ((int)lane == l) key[i] = 0;
        }
      }
    }
    sum += w;
    if (lane == j) {
      mine = w;
      my_id = id;
    }
  }
  if (a.renorm) mine = sum == 0.0f ? 0.0f : mine / sum;
  mine *= a.scale;
  if (lane < a.top_k) {
    c.id[t * a.top_k + lane] = (int16_t)my_id;
    c.weight[t * a.top_k + lane] = my_id < 0 ? 0.0f : mine;
    if (my_id >= 0) atomicOr((unsigned long long*)&c.mask[my_id], 1ull << t);  // order does not matter
  }
}

// The whole block: every token's choice, then the experts' places.
__device__ inline void choose_all(const MoeArgs& a, MoeChoice& c) {
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  for (uint32_t e = threadIdx.x; e < a.experts; e += kWave * kMoeWaves) c.mask[e] = 0;
  __syncthreads();
  for (uint32_t t = wave; t < a.tokens; t += kMoeWaves) {
    if (a.experts <= 128u)
      choose<2>(a, t, c);
    else
      choose<8>(a, t, c);
  }
  __syncthreads();
  if (wave == 0) {
    uint32_t places = 0, active = 0;
    for (uint32_t e0 = 0; e0 < a.experts; e0 += kWave) {
      const uint32_t e = e0 + lane;
      const uint64_t m = e < a.experts ? c.mask[e] : 0ull;
      const uint32_t n = (uint32_t)__popcll(m);
      const uint32_t before = wave_excl_scan_u32(n);
      const uint64_t some = __ballot(n != 0);
      if (e < a.experts) c.first[e] = places + before;
      if (n) c.active[active + (uint32_t)__popcll(some & ((1ull << lane) - 1ull))] = (uint16_t)e;
      places += wave_total(n);
      active += (uint32_t)__popcll(some);
    }
    if (lane == 0) c.count = active;
  }
  __syncthreads();
  for (uint32_t p = threadIdx.x; p < a.tokens * a.top_k; p += kWave * kMoeWaves) {
    const int id = c.id[p];
    if (id >= 0) {
      const uint32_t t = p / a.top_k;
      const uint32_t at = c.first[id] + (uint32_t)__popcll(c.mask[id] & ((1ull << t) - 1ull));
      c.pair_weight[at] = c.weight[p];
      c.pair_token[at] = (uint8_t)t;
    }
  }
  __syncthreads();
}

// ---- gate and up ---------------------------------------------------------------

// One item: 16 rows of gate and the same 16 of up of one expert, NT tiles of 16
// of its tokens from its token m0 on.  The waves take the steps in turn.
template <int KIND, int NT>
__device__ inline void gate_up_item(const MoeArgs& a, const MoeChoice& c, uint32_t e, uint32_t row0,
                                    uint32_t m0, mfma_f32x4* part) {
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u;
  const uint32_t first = c.first[e], n = (uint32_t)__popcll(c.mask[e]);
  const uint32_t row = row0 + r < a.inter ? row0 + r : a.inter - 1u;
  const uint64_t base = (uint64_t)e * 2u * a.inter;
  const WeightRow wg = weight_row<KIND>(a.gu, a.gu_scales, base + row, a.hidden);
  const WeightRow wu = weight_row<KIND>(a.gu, a.gu_scales, base + a.inter + row, a.hidden);
  const uint16_t* x[NT];
  mfma_f32x4 g[NT], u[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t m = m0 + 16u * t + r;  // columns past the expert's tokens repeat its last one
    x[t] = a.x + (uint64_t)c.pair_token[first + (m < n ? m : n - 1u)] * a.hidden;
    g[t] = u[t] = mfma_f32x4{0, 0, 0, 0};
  }
  struct Slot {
    WeightStep<KIND> g, u;
    u32x4 x[NT][4];
  };
  const uint32_t steps = (a.hidden + kStep - 1) / kStep;
  const uint32_t count = steps > wave ? (steps - 1u - wave) / kMoeWaves + 1u : 0u;
  step_ring<2, Slot>(
      count,
      [&](uint32_t q, Slot& s) {
        const uint32_t step = q * kMoeWaves + wave;
        load_weights<KIND>(wg, step, a.hidden, s.g);
        load_weights<KIND>(wu, step, a.hidden, s.u);
#pragma unroll
        for (int t = 0; t < NT; ++t) load_inputs<KIND>(x[t], step, a.hidden, s.x[t]);
      },
      [&](uint32_t, const Slot& s) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 og = weight_operand<KIND>(s.g, j), ou = weight_operand<KIND>(s.u, j);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            g[t] = mfma16(og, s.x[t][j], g[t]);
            u[t] = mfma16(ou, s.x[t][j], u[t]);
          }
        }
      });
  __syncthreads();  // the previous item's sums have been read
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    part[((uint32_t)wave * NT + t) * 2u * kWave + lane] = g[t];
    part[((uint32_t)wave * NT + t) * 2u * kWave + kWave + lane] = u[t];
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < NT * kWave; i += kWave * kMoeWaves) {
    const uint32_t t = i / kWave, l = i % kWave;
    mfma_f32x4 sg = {0, 0, 0, 0}, su = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kMoeWaves; ++v) {
      sg += part[(v * NT + t) * 2u * kWave + l];
      su += part[(v * NT + t) * 2u * kWave + kWave + l];
    }
    const uint32_t m = m0 + 16u * t + (l & 15u);
    if (m < n) {
      const float p = c.pair_weight[first + m];
      uint16_t* o = a.act + (uint64_t)(first + m) * a.act_stride;
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t i0 = row0 + 4u * (l >> 4) + k;
        const float h = sg[k] / (1.0f + expf(-sg[k])) * su[k] * p;
        if (i0 < a.inter) o[i0] = bf16_of(h);
      }
    }
  }
}

template <int KIND, int NT>
__global__ __launch_bounds__(kWave * kMoeWaves) void k_moe_gate_up(MoeArgs a) {
  __shared__ MoeChoice c;
  __shared__ mfma_f32x4 part[kMoeWaves * NT * 2 * kWave];
  choose_all(a, c);
  if (blockIdx.x == 0) {
    for (uint32_t p = threadIdx.x; p < a.tokens * a.top_k; p += kWave * kMoeWaves) {
      if (a.ids) a.ids[p] = c.id[p];
      if (a.weights) a.weights[p] = c.weight[p];
    }
    if (threadIdx.x == 0) a.route->count = c.count;
    for (uint32_t j = threadIdx.x; j < c.count; j += kWave * kMoeWaves) {
      const uint32_t e = c.active[j];
      a.route->expert[j] = e;
      a.route->mask[j] = c.mask[e];
      a.route->first[j] = c.first[e];
    }
  }
  const uint32_t tiles = (a.inter + kRowTile - 1) / kRowTile;
  for (uint32_t it = blockIdx.x; it < c.count * tiles; it += gridDim.x) {
    const uint32_t e = c.active[it / tiles], row0 = it % tiles * kRowTile;
    const uint32_t n = (uint32_t)__popcll(c.mask[e]);
    if (NT == 1 || n <= 16u)
      gate_up_item<KIND, 1>(a, c, e, row0, 0, part);
    else if (NT == 2 || n <= 32u)
      gate_up_item<KIND, 2>(a, c, e, row0, 0, part);
    else
      gate_up_item<KIND, NT>(a, c, e, row0, 0, part);
  }
}

// ---- down ----------------------------------------------------------------------

// 16 rows of y per block, NT tiles of 16 tokens.  A wave's steps are
// (expert, 128 columns) in expert order, every kMoeWaves-th of them.  A step's
// products go to sums of their own, and a token's column is added only where
// the token chose the expert: columns of other tokens hold products with
// some row of `act` that mean nothing, NaN possibly.
template <int KIND, int NT>
__global__ __launch_bounds__(kWave * kMoeWaves) void k_moe_down(MoeArgs a) {
  __shared__ mfma_f32x4 part[kMoeWaves][NT][kWave];
  __shared__ uint64_t mask[kMoeExperts];
  __shared__ uint32_t expert[kMoeExperts], first[kMoeExperts];
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 15u;
  const uint32_t count = a.route->count;
  for (uint32_t j = threadIdx.x; j < count; j += kWave * kMoeWaves) {
    mask[j] = a.route->mask[j];
    expert[j] = a.route->expert[j];
    first[j] = a.route->first[j];
  }
  __syncthreads();
  const uint32_t row0 = blockIdx.x * kRowTile;
  const uint32_t row = row0 + r < a.hidden ? row0 + r : a.hidden - 1u;
  mfma_f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = mfma_f32x4{0, 0, 0, 0};
  struct Slot {
    WeightStep<KIND> w;
    u32x4 x[NT][4];
    uint64_t mask;
  };
  const uint32_t per = (a.inter + kStep - 1) / kStep;  // steps per expert
  const uint32_t steps = count * per;
  const uint32_t n = steps > wave ? (steps - 1u - wave) / kMoeWaves + 1u : 0u;
  step_ring<2, Slot>(
      n,
      [&](uint32_t q, Slot& s) {
        const uint32_t f = q * kMoeWaves + wave, j = f / per, step = f - j * per;
        const uint32_t e = expert[j], p0 = first[j];
        s.mask = mask[j];
        load_weights<KIND>(weight_row<KIND>(a.dn, a.dn_scales, (uint64_t)e * a.hidden + row, a.inter),
                           step, a.inter, s.w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if ((s.mask >> (16 * t) & 0xFFFFull) == 0) continue;
          // the row of the lane's token; of some other one where it has none
          const uint32_t tok = 16u * t + r;
          const uint32_t rank = (uint32_t)__popcll(s.mask & ((1ull << tok) - 1ull));
          const uint32_t most = (uint32_t)__popcll(s.mask) - 1u;
          load_inputs<KIND>(a.act + (uint64_t)(p0 + (rank < most ? rank : most)) * a.act_stride, step,
                            a.inter, s.x[t]);
        }
      },
      [&](uint32_t, const Slot& s) {
        mfma_f32x4 sum[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) sum[t] = mfma_f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 op = weight_operand<KIND>(s.w, j);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (s.mask >> (16 * t) & 0xFFFFull) sum[t] = mfma16(op, s.x[t][j], sum[t]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bool on = s.mask >> (16u * t + r) & 1ull;
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[t][k] += on ? sum[t][k] : 0.0f;
        }
      });
#pragma unroll
  for (int t = 0; t < NT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < NT * kWave; i += kWave * kMoeWaves) {
    const uint32_t t = i / kWave, l = i % kWave;
    mfma_f32x4 s = part[0][t][l];
#pragma unroll
    for (int v = 1; v < kMoeWaves; ++v) s += part[v][t][l];
    const uint32_t tok = 16u * t + (l & 15u);
    if (tok < a.tokens) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t h = row0 + 4u * (l >> 4) + k;
        if (h < a.hidden) a.y[(uint64_t)tok * a.hidden + h] = bf16_of(s[k]);
      }
    }
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

template <int KIND>
void launch_gate_up(const MoeArgs& a, uint32_t blocks, hipStream_t s) {
  const dim3 block(kWave * kMoeWaves);
  if (a.tokens <= 16)
    k_moe_gate_up<KIND, 1><<<blocks, block, 0, s>>>(a);
  else if (a.tokens <= 32)
    k_moe_gate_up<KIND, 2><<<blocks, block, 0, s>>>(a);
  else
    k_moe_gate_up<KIND, 4><<<blocks, block, 0, s>>>(a);
}

template <int KIND>
void launch_down(const MoeArgs& a, uint32_t blocks, hipStream_t s) {
  const dim3 block(kWave * kMoeWaves);
  if (a.tokens <= 16)
    k_moe_down<KIND, 1><<<blocks, block, 0, s>>>(a);
  else if (a.tokens <= 32)
    k_moe_down<KIND, 2><<<blocks, block, 0, s>>>(a);
  else
    k_moe_down<KIND, 4><<<blocks, block, 0, s>>>(a);
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
  a.splits = m.splits;
  a.split_steps = m.split_steps;
  a.act_stride = m.act_stride;

  const dim3 router_grid((a.experts + 15u) / 16u, (a.tokens + 15u) / 16u, m.splits);
  wc::k_moe_router<<<router_grid, wc::kWave * wc::kMoeWaves, 0, s>>>(a);
  if (hipGetLastError() != hipSuccess) return WC_E_HIP;

  const uint32_t most = a.tokens * a.top_k < a.experts ? a.tokens * a.top_k : a.experts;
  const uint64_t items = (uint64_t)most * ((a.inter + 15u) / 16u);
  const uint64_t resident = (uint64_t)wc::cu_count() * 4u;
  const uint32_t blocks = (uint32_t)(items < resident ? items : resident);
  if (gate_up->kind == WC_MOE_FP4)
    wc::launch_gate_up<wc::kFp4>(a, blocks, s);
  else
    wc::launch_gate_up<wc::kBf16>(a, blocks, s);
  if (hipGetLastError() != hipSuccess) return WC_E_HIP;

  const uint32_t row_blocks = (a.hidden + 15u) / 16u;
  if (down->kind == WC_MOE_FP4)
    wc::launch_down<wc::kFp4>(a, row_blocks, s);
  else
    wc::launch_down<wc::kBf16>(a, row_blocks, s);
  return hipGetLastError() == hipSuccess ? WC_OK : WC_E_HIP;
}
