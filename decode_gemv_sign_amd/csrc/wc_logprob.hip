// wc_logprob.hip — log probabilities of given tokens, entropy and top alternatives
// of rows of logits in one pass over them (include/wc_logprob.h).
#include "wc_launch.h"
#include "wc_logprob.h"
#include "wc_skinny.h"

namespace wc {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMine = 16;               // logits of a lane's batch
constexpr uint32_t kBatch = kMine * kWave;  // of a wave's
constexpr uint32_t kSingly = 6;  // keys that are put into a list one by one, faster than a merge
constexpr uint32_t kManyWaves = 4, kFewWaves = 16;  // of a block: see cut_scores

// Running sums of a row: m the largest logit, and with t = (x - m) log2(e), s = sum 2^t
// and w = sum t 2^t; lse = m + log s and the entropy (log2 s - w / s) ln 2, which loses
// nothing where one token is nearly certain.  m = -inf: nothing but -inf so far.
struct Sums3 {
  float m = -INFINITY, s = 0, w = 0;
  // Both over the larger of the two offsets.
  __device__ __forceinline__ void join(float om, float os, float ow) {
    const float top = fmaxf(m, om);
    // below -300 the factor is 0, which must not meet an infinite distance
    const float d = m == -INFINITY ? 0.0f : fmaxf((m - top) * kLog2e, -300.0f);
    const float od = om == -INFINITY ? 0.0f : fmaxf((om - top) * kLog2e, -300.0f);
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(d);
    const float of = om == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(od);
    w = (w + s * d) * f + (ow + os * od) * of;
    s = s * f + os * of;  // a NaN stays one
    m = top;
  }
  __device__ __forceinline__ void add(const float x[kMine], float top) {
    if (__ballot(top > m)) join(top, 0, 0);
    const float o = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const float t = (x[i] - o) * kLog2e, e = __builtin_amdgcn_exp2f(t);
      s += e;
      w = fmaf(fmaxf(t, -300.0f), e, w);  // -inf: 0 times a number
    }
  }
  __device__ __forceinline__ void join_wave() {
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) join(__shfl_xor(m, o, kWave), __shfl_xor(s, o, kWave), __shfl_xor(w, o, kWave));
  }
};

// Keys order logits as the alternatives are: by value, then by the lower index; NaN
// first, 0 for none.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 is 0
  const uint32_t v = x != x ? 0xFFFFFFFFu : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return (uint64_t)v << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t v = (uint32_t)(k >> 32);
  return __uint_as_float(v & 0x80000000u ? v ^ 0x80000000u : ~v);  // NaN: some NaN
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~(uint32_t)k; }

__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {  // lane: wave-uniform
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)k, lane);
}

// The wave's values sorted over its lanes, falling (none of them NaN).
template <typename T>
__device__ __forceinline__ T wave_sorted(T v) {
  const uint32_t lane = (uint32_t)lane_id();
#pragma unroll
  for (uint32_t k = 2; k <= (uint32_t)kWave; k *= 2) {
#pragma unroll
    for (uint32_t j = k / 2; j > 0; j /= 2) {
      const T other = __shfl_xor(v, (int)j, kWave);
      const bool larger = !(lane & j) == !(lane & k);  // this lane keeps the larger one
      v = (v > other) == larger ? v : other;
    }
  }
  return v;
}

// The largest `top` keys seen, in lanes 0 .. top - 1, falling.
struct Best {
  uint64_t list = 0, least = 0;  // least: the last one's, 0 while there are fewer
  uint32_t top;

  // Keys of lanes in `mask`, one after the other.
  __device__ __forceinline__ void insert(uint64_t key, uint64_t mask) {
    const uint32_t lane = (uint32_t)lane_id();
    while (mask) {
      const int from = __ffsll((unsigned long long)mask) - 1;
      mask &= mask - 1;
      const uint64_t k = lane_key(key, from);
      if (k <= least) continue;
      const uint32_t at = (uint32_t)__popcll(__ballot(list > k));
      const uint64_t up = (uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(list >> 32), 0x138, 0xF, 0xF, false) << 32 |
                          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)list, 0x138, 0xF, 0xF, false);  // one lane up
      list = lane < at ? list : lane == at ? k : up;
      least = lane_key(list, (int)top - 1);
    }
  }
  // A key per lane (0: none) at once: both lists falling, one of them turned round, are a
  // sequence that a merge's last steps sort.
  __device__ __forceinline__ void merge(uint64_t key) {
    const uint32_t lane = (uint32_t)lane_id();
    key = (uint64_t)wave_sorted((unsigned long long)key);
    const uint64_t turned = (uint64_t)__shfl_xor((unsigned long long)key, kWave - 1, kWave);
    list = list > turned ? list : turned;
#pragma unroll
    for (int j = kWave / 2; j > 0; j /= 2) {
      const uint64_t other = (uint64_t)__shfl_xor((unsigned long long)list, j, kWave);
      list = (list > other) == !(lane & (uint32_t)j) ? list : other;
    }
    least = lane_key(list, (int)top - 1);
  }
};

struct Scores {
  const void* x;
  uint64_t stride;
  const int64_t* tokens;
  float *logprob, *entropy;
  int32_t* ids;
  float* top_logprob;
  float* sums;     // [rows][parts][4]: m, s, w
  uint64_t* keys;  // [rows][top][parts]
  uint32_t rows, vocab, top, parts, part;  // part: logits of one, a multiple of a block's batches
};

template <bool F32>
__device__ __forceinline__ float logit_at(const Scores& a, uint64_t row, uint64_t i) {
  if constexpr (F32) return ((const float*)a.x)[row * a.stride + i];
  return __uint_as_float((uint32_t)((const uint16_t*)a.x)[row * a.stride + i] << 16);
}

// What a row's sums and keys give.  One wave; sums in every lane.
template <bool F32>
__device__ __forceinline__ void finish(const Scores& a, uint32_t row, const Sums3& t, const Best& best) {
  const uint32_t lane = (uint32_t)lane_id();
  const float log_s = __builtin_amdgcn_logf(t.s), off = t.m == -INFINITY ? 0.0f : t.m;
  const bool bad = t.s != t.s;
  auto log_of = [&](float x) __attribute__((always_inline)) {
    return x == -INFINITY ? -INFINITY : ((x - off) * kLog2e - log_s) * kLn2;
  };
  if (lane == 0) {
    const int64_t token = a.tokens[row];
    const bool in = (uint64_t)token < (uint64_t)a.vocab;
    a.logprob[row] = bad || !in ? NAN : log_of(logit_at<F32>(a, row, in ? (uint64_t)token : 0u));
    a.entropy[row] = bad ? NAN : t.s == 0.0f ? 0.0f : (log_s - t.w / t.s) * kLn2;
  }
  if (lane < a.top) {
    const uint64_t at = (uint64_t)row * a.top + lane;
    a.ids[at] = best.list ? (int32_t)key_index(best.list) : -1;
    a.top_logprob[at] = best.list ? (bad ? NAN : log_of(key_value(best.list))) : -INFINITY;
  }
}

// One pass: a wave takes every NW-th batch of its part of the row, keeps the sums per
// lane and the largest `top` keys in its lanes.  Without alternatives it is bound by
// memory: 2048 rows of 100000 BF16 logits in 86 us, 4.8 TB/s (100003, whose rows start at
// any 2-byte address: 98; both in a graph, from HBM).  With 20 of them it is bound by
// instructions, 320 vector ones for a batch of 16 logits per lane, 162 without
// alternatives: 132 us (100003: 133 to 143).  That keys are found in a batch is likely
// throughout, as each wave has a list of its own; the waves share the least value that
// counts.  One or two waves to a row find fewer but wait for their loads (152 and 149 us
// where this took 147), and loads two batches ahead took longer (164).
template <bool F32, bool TOP, uint32_t NW>
__global__ __launch_bounds__(kWave* NW) void k_token_logprobs(Scores a) {
  __shared__ uint64_t room[NW][2 * kWave];
  __shared__ float sums[NW][3];
  __shared__ float shared_least;  // some wave has `top` keys of this value or larger ones
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t row = blockIdx.x / a.parts, part = blockIdx.x - row * a.parts;
  const uint32_t from = part * a.part;  // below vocab (cut_scores)
  const uint32_t end = a.vocab - from < a.part ? a.vocab : from + a.part;
  constexpr uint32_t kEach = F32 ? 4u : 8u;  // logits of a load
  constexpr int kLoads = kMine / kEach;
  const uint8_t* const base = (const uint8_t*)a.x + (uint64_t)row * a.stride * (F32 ? 4u : 2u);
  struct Slot {
    u32x4 v[kLoads];
  };
  auto load = [&](uint32_t at, Slot& s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      s.v[i] = *(const u32x4_any*)(base + (uint64_t)at * (F32 ? 4u : 2u) + (i * kWave + lane) * 16u);
  };
  auto values = [&](const Slot& s, float x[kMine]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
          x[4 * i + j] = __uint_as_float(s.v[i][j]);
        } else {
          x[8 * i + 2 * j] = __uint_as_float(s.v[i][j] << 16);
          x[8 * i + 2 * j + 1] = __uint_as_float(s.v[i][j] & 0xFFFF0000u);
        }
      }
  };
  auto index = [&](uint32_t at, int i) __attribute__((always_inline)) {
    return at + ((uint32_t)i / kEach * kWave + lane) * kEach + (uint32_t)i % kEach;
  };

  Sums3 t;
  Best best;
  best.top = a.top;
  if constexpr (TOP) {
    if (threadIdx.x == 0) shared_least = -INFINITY;
    __syncthreads();
  }
  volatile float* const others = &shared_least;
  float least = -INFINITY;  // larger ones may be among the best
  auto use = [&](uint32_t at, const float x[kMine]) __attribute__((always_inline)) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kMine; ++i) top = fmaxf(top, x[i]);
    t.add(x, top);
    if constexpr (TOP) {
      const bool nan = t.s != t.s;
      // Fewer than `top` so far, or a batch in which half the lanes have better ones (rising
      // rows): at least `top` of its logits are as large as the top-th of the lanes' largest.
      // 2048 x 100003 BF16 that rise along the row, 20 alternatives: 676 us with this bar,
      // 1581 with the list's least alone; random rows took 133 in the same calls with either.
      const uint32_t lanes = (uint32_t)__popcll(__ballot(top > least));
      if (!best.least || (lanes >= (uint32_t)kWave / 2 && lanes >= a.top && !__ballot(nan))) {
        const float enough = __int_as_float(
            __builtin_amdgcn_readlane(__float_as_int(wave_sorted(__ballot(nan) ? -INFINITY : top)), (int)a.top - 1));
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const bool take = !(x[i] < enough) && x[i] != -INFINITY;
          const uint64_t mask = __ballot(take);
          if (!mask) continue;
          const uint32_t to = n + (uint32_t)__popcll(mask & ((1ull << lane) - 1ull));
          if (take && to < kWave) room[wave][to] = key_of(x[i], index(at, i));
          n += (uint32_t)__popcll(mask);
        }
        wave_lds_sync();
        const uint64_t first = lane < n ? room[wave][lane] : 0u;
        wave_lds_sync();
        best.merge(first);
        if (n > (uint32_t)kWave) {  // many equal ones
          uint32_t m = 0;
#pragma unroll 1
          for (int i = 0; i < kMine; ++i) {
            float y = x[0];
#pragma unroll
            for (int j = 1; j < kMine; ++j) y = i == j ? x[j] : y;
            const bool take = !(y < enough) && y != -INFINITY;
            const uint64_t mask = __ballot(take), k = key_of(y, index(at, i));
            const uint32_t to = m + (uint32_t)__popcll(mask & ((1ull << lane) - 1ull));
            m += (uint32_t)__popcll(mask);
            best.insert(k, __ballot(take && to >= (uint32_t)kWave && k > best.least));
          }
        }
      } else if (lanes || __ballot(nan)) {
        uint32_t n = 0;
#pragma unroll
        for (int g = 0; g < kMine; g += 4) {
          bool any = false;
#pragma unroll
          for (int i = g; i < g + 4; ++i) any = any || !(x[i] <= least);
          if (!__ballot(any)) continue;
#pragma unroll
          for (int i = g; i < g + 4; ++i) {
            const bool take = !(x[i] <= least);
            const uint64_t mask = __ballot(take);
            if (!mask) continue;
            const uint64_t k = key_of(x[i], index(at, i));
            const uint32_t to = n + (uint32_t)__popcll(mask & ((1ull << lane) - 1ull));
            if (take && to < (uint32_t)kWave) room[wave][to] = k;
            n += (uint32_t)__popcll(mask);
            if (n > (uint32_t)kWave) best.insert(k, __ballot(take && to >= (uint32_t)kWave && k > best.least));
          }
        }
        wave_lds_sync();
        const uint64_t k = lane < n ? room[wave][lane] : 0u;
        wave_lds_sync();
        if (n <= kSingly)
          best.insert(k, __ballot(k > best.least));
        else
          best.merge(k);
      }
      // Keys that follow have larger indices than the wave's own: equal values are no
      // better.  Of equal values of another wave they may have lower ones.
      const float mine = best.least ? key_value(best.least) : -INFINITY, other = *others;
      if (lane == 0 && mine > other) *others = mine;  // any wave's will do
      const int32_t below = __float_as_int(other) + (other > 0.0f ? -1 : 1);  // the next lower number
      least = other > -INFINITY && other != 0.0f ? fmaxf(mine, __int_as_float(below)) : mine;
      least = mine != mine ? mine : least;
    }
  };

  uint32_t at = from + wave * kBatch;
  if (at + kBatch <= end) {
    Slot now;
    load(at, now);
    while (at + kBatch <= end) {
      const uint32_t next = at + NW * kBatch;
      const Slot s = now;
      if (next + kBatch <= end) load(next, now);
      float x[kMine];
      values(s, x);
      use(at, x);
      at = next;
    }
  }
  if (at < end) {  // the short last one
    float x[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const uint32_t k = index(at, i);
      x[i] = logit_at<F32>(a, row, k < end ? k : end - 1u);
      x[i] = k < end ? x[i] : -INFINITY;
    }
    use(at, x);
  }
  t.join_wave();
  if (lane == 0) {
    sums[wave][0] = t.m;
    sums[wave][1] = t.s;
    sums[wave][2] = t.w;
  }
  if constexpr (TOP) room[wave][kWave + lane] = lane < a.top ? best.list : 0u;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (uint32_t i = 1; i < NW; ++i) t.join(sums[i][0], sums[i][1], sums[i][2]);
  if constexpr (TOP) {
#pragma unroll
    for (uint32_t i = 1; i < NW; ++i) {
      const uint64_t k = room[i][kWave + lane];
      best.insert(k, __ballot(k > best.least));
    }
  }
  if (a.parts == 1) {
    finish<F32>(a, row, t, best);
    return;
  }
  if (lane == 0) {
    float* const to = a.sums + 4u * ((uint64_t)row * a.parts + part);
    to[0] = t.m;
    to[1] = t.s;
    to[2] = t.w;
  }
  if (TOP && lane < a.top) a.keys[((uint64_t)row * a.top + lane) * a.parts + part] = best.list;
}

// The parts of a row, joined by one wave.
template <bool F32>
__global__ __launch_bounds__(kWave) void k_join_logprobs(Scores a) {
  const uint32_t lane = (uint32_t)lane_id(), row = blockIdx.x;
  Sums3 t;
  if (lane < a.parts) {  // parts <= kWave
    const float* const from = a.sums + 4u * ((uint64_t)row * a.parts + lane);
    t.m = from[0];
    t.s = from[1];
    t.w = from[2];
  }
  t.join_wave();
  Best best;
  best.top = a.top;
  const uint32_t n = a.top * a.parts;
  const uint64_t* const keys = a.keys + (uint64_t)row * n;  // the parts' best first
  if (n) best.merge(lane < n ? keys[lane] : 0u);
  for (uint32_t i = kWave; i < n; i += kWave) {
    const uint64_t k = i + lane < n ? keys[i + lane] : 0u;
    best.insert(k, __ballot(k > best.least));
  }
  finish<F32>(a, row, t, best);
}

namespace {

// Enough rows to fill the card have a block of four waves each.  Fewer have one of 16,
// up to eight batches a wave, in one launch, and longer ones are split into parts of whole
// batches and joined by a second.  fp32, 5 alternatives, whole / split, us in a graph (from
// Python; a second launch is 5 us of host time):
//   logits        1 row                     4 rows      32 rows                  256 rows
//   8000     9.3 / 11.0 (14 / 18)      9.8 / 11.5   10.1 / 12.2 (14 / 18)   11.3 / 14.6
//   32000   13.5 / 11.0 (14 / 18)     14.3 / 11.8   15.5 / 13.1 (15 / 18)   18.1 / 22.5
//   64000   17.3 / 11.5 (17 / 18)     18.0 / 12.2   19.0 / 14.6 (18 / 18)   22.7 / 26.7
//   128256  23.3 / 11.8 (23 / 18)     24.1 / 13.1   25.5 / 17.5 (25 / 18)   32.3 / 34.8
//   152064  24.8 / 12.0 (25 / 18)     26.0 / 13.4   27.5 / 20.6 (26 / 19)   36.4 / 39.8
// So the limit of eight batches is right for calls from Python up to 64000 logits and for
// 256 rows; in a graph, few rows past 16000 are faster split.
struct ScoreCut {
  uint32_t waves, parts, part;
};
int cut_scores(const wc_logprob_shape* s, ScoreCut* cut) {
  if (!s || s->vocab < 1u || s->vocab >= (1u << 31)) return WC_E_ARG;
  if (s->kind > WC_LOGITS_F32) return WC_E_ARG;
  if (s->top > WC_LOGPROB_MAX_TOP) return WC_E_UNSUPPORTED;
  const uint32_t step = kManyWaves * kBatch, steps = (s->vocab + step - 1u) / step;
  const bool few = s->rows < 2u * cu_count() && s->vocab <= kFewWaves * kBatch * 8u;
  uint32_t n = s->rows && !few ? (4u * cu_count() + s->rows - 1u) / s->rows : 1u;
  n = n < (uint32_t)kWave ? n : (uint32_t)kWave;
  n = n < steps ? n : steps;
  cut->waves = few ? kFewWaves : kManyWaves;
  cut->part = (steps + n - 1u) / n * step;
  cut->parts = (s->vocab - 1u) / cut->part + 1u;
  if ((uint64_t)s->rows * cut->parts >= (1ull << 24)) return WC_E_SIZE;  // a grid of fewer than 2^32 threads
  return WC_OK;
}
uint64_t score_bytes(const wc_logprob_shape* s, uint32_t parts) {
  return parts == 1u ? 0u : (uint64_t)s->rows * parts * (16u + 8u * s->top);
}

template <bool F32, bool TOP>
void launch_scores_of(const Scores& a, uint32_t waves, hipStream_t s) {
  const uint32_t blocks = a.rows * a.parts;
  if (waves == kFewWaves)
    k_token_logprobs<F32, TOP, kFewWaves><<<blocks, kWave * kFewWaves, 0, s>>>(a);
  else
    k_token_logprobs<F32, TOP, kManyWaves><<<blocks, kWave * kManyWaves, 0, s>>>(a);
}
template <bool F32>
void launch_scores(const Scores& a, uint32_t waves, hipStream_t s) {
  if (a.top)
    launch_scores_of<F32, true>(a, waves, s);
  else
    launch_scores_of<F32, false>(a, waves, s);
  if (a.parts > 1u) k_join_logprobs<F32><<<a.rows, kWave, 0, s>>>(a);
}

}  // namespace
}  // namespace wc

extern "C" size_t wc_token_logprobs_workspace_bytes(const wc_logprob_shape* shape) {
  wc::ScoreCut cut;
  if (wc::cut_scores(shape, &cut)) return 0;
  return wc::score_bytes(shape, cut.parts);
}

extern "C" int wc_token_logprobs(const wc_logprob_shape* shape, const void* d_logits, const int64_t* d_tokens,
                                 float* d_logprobs, float* d_entropy, int32_t* d_top_ids, float* d_top_logprobs,
                                 void* d_work, size_t work_bytes, void* stream) {
  wc::ScoreCut cut;
  if (const int v = wc::cut_scores(shape, &cut)) return v;
  const bool f32 = shape->kind == WC_LOGITS_F32;
  if (shape->stride >= (1ull << 40)) return WC_E_SIZE;
  if (shape->rows > 1u && shape->stride < shape->vocab) return WC_E_ARG;
  if (shape->rows == 0) return WC_OK;
  if (!d_logits || ((uintptr_t)d_logits & (f32 ? 3u : 1u)) || !d_tokens || ((uintptr_t)d_tokens & 7u)) return WC_E_ARG;
  if (!d_logprobs || ((uintptr_t)d_logprobs & 3u) || !d_entropy || ((uintptr_t)d_entropy & 3u)) return WC_E_ARG;
  if (shape->top && (!d_top_ids || ((uintptr_t)d_top_ids & 3u) || !d_top_logprobs || ((uintptr_t)d_top_logprobs & 3u)))
    return WC_E_ARG;
  const uint64_t need = wc::score_bytes(shape, cut.parts);
  if (need) {
    if (!d_work || !wc::aligned16(d_work)) return WC_E_ARG;
    if (work_bytes < need) return WC_E_SIZE;
  }
  wc::Scores a;
  a.x = d_logits;
  a.stride = shape->stride;
  a.tokens = d_tokens;
  a.logprob = d_logprobs;
  a.entropy = d_entropy;
  a.ids = d_top_ids;
  a.top_logprob = d_top_logprobs;
  a.sums = (float*)d_work;
  a.keys = (uint64_t*)((uint8_t*)d_work + (uint64_t)shape->rows * cut.parts * 16u);
  a.rows = shape->rows;
  a.vocab = shape->vocab;
  a.top = shape->top;
  a.parts = cut.parts;
  a.part = cut.part;
  if (f32)
    wc::launch_scores<true>(a, cut.waves, (hipStream_t)stream);
  else
    wc::launch_scores<false>(a, cut.waves, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? WC_OK : WC_E_HIP;
}
