// wc_prompt.hip — causal attention of whole prompts, packed one after the other
// (include/wc_attn.h).
#include "wc_attn.h"
#include "wc_launch.h"
#include "wc_skinny.h"

namespace wc {

typedef float mfma_f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

__device__ __forceinline__ mfma_f32x16 mfma32(u32x4 a, u32x4 b, mfma_f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(mfma_bf16x8, a),
                                                 __builtin_bit_cast(mfma_bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, mfma_bf16x2));
}

struct Prompt {
  const uint16_t *q, *k, *v;
  const int32_t* starts;
  uint16_t* out;
  float* lse;  // may be null
  uint64_t tokens;
  uint32_t q_stride, k_stride, v_stride;
  uint32_t seqs, heads, kv_heads, group, window;
  float scale;   // times log2(e), not 0
  float masked;  // a score whose weight is 0: -inf, or +inf where scale is negative
};

// A block takes 32 queries of one head per wave and walks the tiles of 64 tokens
// that they attend to, from the last one down.
//
// Keys times queries: 32 tokens are the rows of v_mfma_f32_32x32x16_bf16 and the
// queries its columns, so that a lane receives the scores of its query (lane % 32)
// with 16 of the 32 tokens (lane / 32 has the other half).  These are, rounded to
// BF16, the second product's operand as they stand, as the order in which tokens
// are summed over is free: the values' operand takes tokens in the same order, by
// LDS reads that transpose (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 numbers
// and receive a column each).  The second product has the head's columns as rows,
// so that the running maximum and sum of a query stay in its lane pair.
//
// That rounding of the weights (not of their sum) is as large as the outputs' own:
// 2.3e-3 of the norm from 64 bits where fp32 weights are 1.7e-3 away.  Weights as the
// sum of two BF16 numbers would close that, with half as many products more on the unit
// that bounds the kernel: 16384 tokens 2.88 ms against 2.14 in the same run, 12 prompts
// to 2048 172 us against 145.
//
// Weights are exp2(s - offset), the offset a value near the query's largest score so
// far: it is set at its first tile, and moves (and the tile is done once more) only
// when the weights of a tile add up to more than kMost.  So a step looks for no
// maximum, and nothing crosses lanes.
constexpr float kMost = 65536.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kStepTokens = 64;

// The place of a tile's 16-byte pieces in LDS.  Rows are padded to a power of two,
// and the pieces of a row change places so that what a wave reads at a time lies in
// different banks: 16 rows at one piece (keys), 4 pieces in each of 4 rows (values).
template <int G>
struct Place {
  static constexpr uint32_t kRow = G == 1 ? 64u : G == 2 ? 128u : G <= 4 ? 256u : 512u;  // bytes
  static constexpr uint32_t kPieces = kRow / 16u;
  static constexpr uint32_t kRowsPerBank = kRow >= 256u ? 1u : 256u / kRow;
  static constexpr uint32_t kTile = kStepTokens * kRow;
  static constexpr uint32_t kMask = (kPieces < 16u ? kPieces : 16u) - 1u;
  __device__ static __forceinline__ uint32_t key(uint32_t row) { return row / kRowsPerBank & kMask; }
  __device__ static __forceinline__ uint32_t value(uint32_t row) { return row / kRowsPerBank << 2 & kMask; }
};

// 16384 tokens, 32 heads of 128: 2.06 ms in a graph (1.97 to 2.2 from card to card and
// run to run), 1066 TFLOP/s where a library product of 8192^3 reached 1184, with the
// matrix cores busy half of the time at the 2.0 GHz that the card then keeps; the rest is
// exponentials (141 vector instructions for 32 products) and waiting for operands and for
// the other wave of the SIMD.  Operands are read a group of four products ahead, and the
// products of the two halves of a tile alternate, as one waits for the one before it on
// the same sums.  (Of runs at 2.0 ms: chained 2.1, weights of one half between the
// products of the other 2.1, three tiles in LDS 2.04, waves of other priorities no
// change.)  launch_prompt_of has the block shapes' figures.
//
// Head dims past 128 have one wave to a SIMD (up to 456 registers) and rows of 512 bytes in
// LDS whatever their length: 16384 tokens of heads of 160 4.2 ms, 192 4.6, 224 5.0, 256
// 5.6, at 655 to 790 TFLOP/s.
template <int G, int NW>
__global__ __launch_bounds__(kWave* NW, G <= 4 ? 2 : 1) void k_prompt(Prompt a) {
  using P = Place<G>;
  constexpr uint32_t D = 32u * G, kRows = 32u * NW;
  constexpr int kSteps = 2 * G;  // MFMAs over the head's columns
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // [2][keys, values][kTile]
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint32_t r = lane & 31u, h = lane >> 5;

  // head, then (sequence, rows) of this block
  const uint32_t n = blockIdx.x % a.heads, kv = n % a.kv_heads, head = kv * a.group + n / a.kv_heads;
  uint32_t left = blockIdx.x / a.heads, start = 0, len = 0, row0 = 0;
  bool found = false;
  for (uint32_t s0 = 0; s0 < a.seqs && !found; s0 += kWave) {
    const uint32_t s = s0 + lane;
    int64_t from = 0, to = 0;
    if (s < a.seqs) {
      const int64_t t = (int64_t)a.tokens, x = a.starts[s], y = a.starts[s + 1];
      from = x < 0 ? 0 : x > t ? t : x;
      to = y < from ? from : y > t ? t : y;
    }
    const uint32_t tiles = (uint32_t)((to - from + kRows - 1) / kRows), before = wave_excl_scan_u32(tiles);
    const uint64_t hit = __ballot(left >= before && left < before + tiles);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      start = (uint32_t)__builtin_amdgcn_readlane((int)from, at);
      len = (uint32_t)__builtin_amdgcn_readlane((int)to, at) - start;
      const uint32_t t = left - (uint32_t)__builtin_amdgcn_readlane((int)before, at);
      row0 = ((uint32_t)__builtin_amdgcn_readlane((int)tiles, at) - 1u - t) * kRows;  // the longest first
      found = true;
    } else {
      left -= (uint32_t)__builtin_amdgcn_readlane((int)(before + tiles), kWave - 1);
    }
  }
  if (!found) return;

  // the wave's queries: rows past the end repeat the last one
  const uint32_t w0 = row0 + 32u * wave;
  const uint32_t pos = w0 + r < len ? w0 + r : len - 1u;
  const bool real = w0 + r < len;
  u32x4 q[kSteps];
  {
    const uint16_t* from = a.q + (uint64_t)(start + pos) * a.q_stride + head * D + 8u * h;
    each<kSteps>([&](auto i) __attribute__((always_inline)) { q[i] = *(const u32x4*)(from + 16 * i); });
  }
  const uint32_t end = row0 + kRows < len ? row0 + kRows : len;
  const int32_t last = (int32_t)((end - 1u) / kStepTokens);
  const auto first_of = [&](uint32_t p) { return a.window && p >= a.window ? (int32_t)((p - a.window + 1u) / kStepTokens) : 0; };
  const int32_t first = first_of(row0);
  // tiles that some query of this wave attends to (none where it has no query)
  const uint32_t w1 = w0 + 31u < end ? w0 + 31u : end - 1u;
  const int32_t mine_last = w0 < end ? (int32_t)(w1 / kStepTokens) : -1, mine_first = first_of(w0);

  // A load brings 1 KB, kLoadRows rows; a wave takes every NW-th of a tile's.  The
  // places of the pieces repeat after a period of its loads, so that the lane's
  // offsets are few.  Rows past the sequence and pieces past the head read as 0.
  constexpr uint32_t kLoads = P::kTile / 1024u, kLoadRows = 64u / P::kPieces;
  constexpr uint32_t kPeriod = kLoadRows * NW / P::kRowsPerBank % (P::kMask + 1u) ? 2u : 1u;
  static_assert(kLoadRows * NW * kPeriod / P::kRowsPerBank % (P::kMask + 1u) == 0 || kLoads <= NW, "period");
  uint32_t k_off[kPeriod], v_off;
  each<kPeriod>([&](auto i) __attribute__((always_inline)) {
    const uint32_t row = kLoadRows * wave + lane / P::kPieces, slot = lane % P::kPieces;
    const uint32_t kp = slot ^ P::key(row + kLoadRows * NW * i), vp = slot ^ P::value(row);
    k_off[i] = kp * 8u < D ? row * a.k_stride * 2u + kp * 16u : kNowhere;
    v_off = vp * 8u < D ? row * a.v_stride * 2u + vp * 16u : kNowhere;
  });
  auto stage = [&](int32_t tile, uint32_t to) __attribute__((always_inline)) {
    each<(kLoads + NW - 1) / NW>([&](auto i) __attribute__((always_inline)) {
      if (kLoads >= NW || wave < kLoads) {
        const uint32_t t0 = (uint32_t)tile * kStepTokens + kLoadRows * NW * i;
        const uint32_t rows = t0 < len ? (len - t0 < kStepTokens ? len - t0 : kStepTokens) : 0u;
        const uint64_t at = t0 < len ? start + t0 : start;
        load16_lds(buffer_of(a.k + at * a.k_stride + kv * D, rows * a.k_stride * 2u),
                   lds + to + (wave + NW * i) * 1024u, k_off[i % kPeriod], 0);
        load16_lds(buffer_of(a.v + at * a.v_stride + kv * D, rows * a.v_stride * 2u),
                   lds + to + P::kTile + (wave + NW * i) * 1024u, v_off, 0);
      }
    });
  };

  float m = -INFINITY, off = 0, sum = 0;
  mfma_f32x16 acc[G];
  int32_t later[3] = {-1, -1, -1};  // a wave has at most one tile at its queries and two at their windows
  each<G>([&](auto g) __attribute__((always_inline)) {
    each<16>([&](auto i) __attribute__((always_inline)) { acc[g][+i] = 0; });
  });

  // The lane's places in a tile: rows of keys (pieces by exclusive or), and of values.
  const uint32_t k_at = r * P::kRow + (h ^ P::key(r)) * 16u;
  const uint32_t v_row = 4u * h + (lane >> 2 & 3u), v_piece = 2u * (lane >> 4 & 1u) + (lane >> 1 & 1u);
  const uint32_t v_at = v_row * P::kRow + (v_piece ^ P::value(v_row)) * 16u + 8u * (lane & 1u);
  static_assert(P::kRow >= 256u || P::kMask < 8u, "");

  // Keys of 32 tokens (t), columns 16 i ..
  auto key_operand = [&](uint32_t from, int t, int i) __attribute__((always_inline)) {
    return *(const u32x4*)(lds + from + 32 * t * P::kRow + (k_at ^ 32u * i));
  };
  // Values of columns 32 g .. of 16 tokens (chunk c), in the scores' order.
  auto value_operand = [&](uint32_t from, int g, int c) __attribute__((always_inline)) {
    u32x4 x;
    each<2>([&](auto j) __attribute__((always_inline)) {
      const uint8_t* at = lds + from + (16 * c + 8 * j) * P::kRow + (v_at ^ 64u * g);
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at);
      const uint2 z = __builtin_bit_cast(uint2, y);
      x[2 * j] = z.x;
      x[2 * j + 1] = z.y;
    });
    return x;
  };

  auto step = [&](int32_t tile, uint32_t k) __attribute__((always_inline)) {
    const uint32_t t0 = (uint32_t)tile * kStepTokens, v = k + P::kTile;
    // some query does not attend to some token
    const bool edge = t0 + kStepTokens - 1u > w0 || (a.window && w1 >= a.window && t0 <= w1 - a.window);
    mfma_f32x16 s[2];
    float part;
    // Each query goes by its own sums alone: one that has no score to take as its offset
    // (NaN, or -inf throughout) does not keep the others from moving theirs.
    bool need = m == -INFINITY, set = false, full = __ballot(need);
    for (;;) {  // once more where a query's offset has to move, which it does at most once
      // operands a group of four products ahead
      u32x4 keys[2][4];
      auto load_keys = [&](auto j) __attribute__((always_inline)) {
        each<4>([&](auto n) __attribute__((always_inline)) { keys[j % 2][n] = key_operand(k, n % 2, 2 * j + n / 2); });
      };
      load_keys(std::integral_constant<int, 0>{});
      each<2>([&](auto t) __attribute__((always_inline)) {
        each<16>([&](auto i) __attribute__((always_inline)) { s[t][+i] = 0; });
      });
      each<G>([&](auto j) __attribute__((always_inline)) {
        if constexpr (j + 1 < G) load_keys(std::integral_constant<int, j + 1>{});
        __builtin_amdgcn_sched_barrier(0);
        each<4>([&](auto n) __attribute__((always_inline)) { s[n % 2] = mfma32(keys[j % 2][n], q[2 * j + n / 2], s[n % 2]); });
        __builtin_amdgcn_sched_barrier(0);
      });
      if (edge) {
        int32_t ahead = (int32_t)(pos - t0 - 4u * h);  // of the query, from the lane's first token
        asm volatile("" : "+v"(ahead));                // what follows is not kept over the tiles
        each<2>([&](auto t) __attribute__((always_inline)) {
          each<16>([&](auto i) __attribute__((always_inline)) {
            const int32_t d = ahead - (32 * t + 8 * (i / 4) + i % 4);
            const bool ok = d >= 0 && (!a.window || (uint32_t)d < a.window);
            s[t][+i] = ok ? s[t][+i] : a.masked;
          });
        });
      }
      if (full) {
        float top = -INFINITY;
        each<2>([&](auto t) __attribute__((always_inline)) {
          each<16>([&](auto i) __attribute__((always_inline)) { top = fmaxf(top, s[t][+i] * a.scale); });
        });
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        // queries that need not move keep theirs: no query's bits depend on another's
        const float now = need ? top : m, to = now == -INFINITY ? 0.0f : now;
        const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(off - to);
        m = now;
        off = to;
        set = set || need;
        sum *= f;
        each<G>([&](auto g) __attribute__((always_inline)) { acc[g] *= f; });
      }
      part = 0;
      each<2>([&](auto t) __attribute__((always_inline)) {
        each<16>([&](auto i) __attribute__((always_inline)) {
          s[t][+i] = __builtin_amdgcn_exp2f(fmaf(s[t][+i], a.scale, -off));
          part += s[t][+i];
        });
      });
      need = !set && !(part <= kMost);
      full = __ballot(need);
      if (!full) break;
      const int other = __shfl_xor((int)need, 32, kWave);
      need = need || other;
    }
    sum += part;
    u32x4 values[2][G], w[4];
    auto load_values = [&](auto c) __attribute__((always_inline)) {
      each<G>([&](auto g) __attribute__((always_inline)) { values[c % 2][g] = value_operand(v, g, c); });
    };
    load_values(std::integral_constant<int, 0>{});
    each<2>([&](auto t) __attribute__((always_inline)) {
      each<8>([&](auto i) __attribute__((always_inline)) {
        w[2 * t + i / 4][i % 4] = bf16_pair(s[t][2 * i], s[t][2 * i + 1]);
      });
    });
    if (edge) {
      // a value that is not finite must not reach the queries that do not attend to
      // it: the tile's second product is left for the end
      uint32_t odd = 0, from = v + 16u * lane;
      asm volatile("" : "+v"(from));
      each<P::kTile / 1024>([&](auto i) __attribute__((always_inline)) {
        const u32x4 x = *(const u32x4*)(lds + from + 1024 * i);
        each<4>([&](auto j) __attribute__((always_inline)) { odd |= (x[+j] & 0x7FFF7FFFu) + 0x00800080u; });
      });
      if (__ballot(odd & 0x80008000u)) {
        later[2] = later[1];
        later[1] = later[0];
        later[0] = tile;
        return;
      }
    }
    each<4>([&](auto c) __attribute__((always_inline)) {
      if constexpr (c + 1 < 4) load_values(std::integral_constant<int, c + 1>{});
      __builtin_amdgcn_sched_barrier(0);
      each<G>([&](auto g) __attribute__((always_inline)) { acc[g] = mfma32(values[c % 2][g], w[c], acc[g]); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  stage(last, 0);
  for (int32_t tile = last; tile >= first; tile -= 2) {
    each<2>([&](auto b) __attribute__((always_inline)) {
      const int32_t now = tile - b;
      if (now < first) return;
      wait_vm<0>();
      __syncthreads();  // this tile is in, and the other buffer has been read
      if (now > first) stage(now - 1, (b ^ 1) * 2u * P::kTile);
      if (now <= mine_last && now >= mine_first) step(now, b * 2u * P::kTile);
    });
  }

  // The products left: token by token, those that the lane's query attends to.
  each<3>([&](auto z) __attribute__((always_inline)) {
    if (later[z] < 0) return;
    for (uint32_t t = 0; t < kStepTokens; ++t) {
      const uint32_t p = (uint32_t)later[z] * kStepTokens + t;
      if (p >= len) break;
      const uint16_t* from = a.k + (uint64_t)(start + p) * a.k_stride + kv * D + 8u * h;
      float x = 0;
      each<kSteps>([&](auto i) __attribute__((always_inline)) {
        const u32x4 key = *(const u32x4*)(from + 16 * i);
        each<4>([&](auto j) __attribute__((always_inline)) {
          x = fmaf(__uint_as_float(key[+j] << 16), __uint_as_float(q[i][+j] << 16), x);
          x = fmaf(__uint_as_float(key[+j] & 0xFFFF0000u), __uint_as_float(q[i][+j] & 0xFFFF0000u), x);
        });
      });
      x += __shfl_xor(x, 32, kWave);
      const bool ok = p <= pos && (!a.window || pos - p < a.window);
      x = __builtin_amdgcn_exp2f(x * a.scale - off);
      const uint16_t* value = a.v + (uint64_t)(start + p) * a.v_stride + kv * D + 4u * h;
      each<G>([&](auto g) __attribute__((always_inline)) {
        each<16>([&](auto i) __attribute__((always_inline)) {
          const float y = __uint_as_float((uint32_t)value[32 * g + 8 * (i / 4) + i % 4] << 16);
          acc[g][+i] = ok ? fmaf(x, y, acc[g][+i]) : acc[g][+i];
        });
      });
    }
  });

  sum += __shfl_xor(sum, 32, kWave);
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (!real) return;
  const uint64_t row = (uint64_t)(start + pos) * a.heads + head;
  each<G>([&](auto g) __attribute__((always_inline)) {
    each<4>([&](auto i) __attribute__((always_inline)) {
      uint2 o;
      o.x = bf16_pair(acc[g][4 * i] * by, acc[g][4 * i + 1] * by);
      o.y = bf16_pair(acc[g][4 * i + 2] * by, acc[g][4 * i + 3] * by);
      *(uint2*)(a.out + row * D + 32u * g + 8u * i + 4u * h) = o;
    });
  });
  if (a.lse && h == 0)
    a.lse[row] = sum == 0.0f ? -INFINITY : (m == -INFINITY ? sum : (m + __builtin_amdgcn_logf(sum)) * kLn2);
}

namespace {

int launched() { return hipGetLastError() == hipSuccess ? WC_OK : WC_E_HIP; }

// Tiles of `rows` queries that any division of the tokens among the sequences needs.
uint64_t prompt_tiles(const wc_prompt_shape* s, uint32_t rows) { return s->tokens / rows + s->seqs; }

template <int G, int NW>
int launch_prompt(const Prompt& a, const wc_prompt_shape* p, hipStream_t s) {
  const uint64_t blocks = prompt_tiles(p, 32u * NW) * a.heads;
  if (blocks * kWave * NW >= (1ull << 32)) return WC_E_SIZE;
  constexpr uint32_t lds = 4u * Place<G>::kTile;
  static bool done[64] = {false};
  int dev = 0;
  if (lds > 65536u && hipGetDevice(&dev) == hipSuccess && (dev < 0 || dev >= 64 || !done[dev])) {
    if (hipFuncSetAttribute((const void*)k_prompt<G, NW>, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
      return WC_E_HIP;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  k_prompt<G, NW><<<(uint32_t)blocks, kWave * NW, lds, s>>>(a);
  return launched();
}

// Blocks of 8 waves (one to a compute unit) read keys and values half as often, of 4 (two)
// have fewer rows past the diagonal.  32 heads on 8, us in a graph with 4 / 8 waves:
//   head dim                 32          64          96          128
//   1 x 16384 tokens      863 / 883  1240 / 1388  1883 / 1865  2176 / 2100
//   3 x 8192              705 / 739   978 / 1181  1492 / 1540  1739 / 1689
//   1 x 8192              234 / 247   336 / 380    480 / 509    563 / 564
//   4 x 4096              271 / 293   363 / 428    535 / 576    629 / 641
//   1 x 4096               79 / 92    100 / 110    145 / 142    169 / 157
//   8 x 2048              144 / 157   188 / 237    272 / 300    310 / 336
// The rule was made for heads of 128, where it gains up to 7% and loses up to 2.  From 4096
// tokens on heads of 96 lie between a gain of 2% and a loss of 8, those of 32 and 64 lose 2
// to 21.
template <int G>
int launch_prompt_of(const Prompt& a, const wc_prompt_shape* p, hipStream_t s) {
  if constexpr (G <= 4)
    if (p->tokens / p->seqs >= 4096u && prompt_tiles(p, 256) * a.heads >= 2u * cu_count()) return launch_prompt<G, 8>(a, p, s);
  return launch_prompt<G, 4>(a, p, s);
}

}  // namespace
}  // namespace wc

extern "C" int wc_prompt_attention(const wc_prompt_shape* shape, const uint16_t* d_q, const uint16_t* d_k,
                                   const uint16_t* d_v, const int32_t* d_starts, uint16_t* d_out, float* d_lse,
                                   void* stream) {
  if (!shape) return WC_E_ARG;
  const wc_prompt_shape& s = *shape;
  if (s.head_dim < 32u || s.head_dim > WC_ATTN_MAX_DIM || s.head_dim % 32u) return WC_E_ARG;
  if (s.kv_heads < 1u || s.heads < 1u || s.heads > WC_ATTN_MAX_HEADS || s.heads % s.kv_heads) return WC_E_ARG;
  if (s.tokens >= (1ull << 31) || s.seqs >= (1u << 31)) return WC_E_SIZE;
  const uint64_t most = 1ull << 24;
  if (s.q_stride >= most || s.k_stride >= most || s.v_stride >= most) return WC_E_SIZE;
  const uint64_t row = (uint64_t)s.heads * s.head_dim, kv_row = (uint64_t)s.kv_heads * s.head_dim;
  if (s.q_stride % 8u || s.k_stride % 8u || s.v_stride % 8u) return WC_E_ARG;
  if (s.tokens > 1u && (s.q_stride < row || s.k_stride < kv_row || s.v_stride < kv_row)) return WC_E_ARG;
  if (s.tokens == 0 || s.seqs == 0) return WC_OK;
  if (!d_q || !wc::aligned16(d_q) || !d_k || !wc::aligned16(d_k) || !d_v || !wc::aligned16(d_v)) return WC_E_ARG;
  if (!d_starts || ((uintptr_t)d_starts & 3u) || !d_out || !wc::aligned16(d_out) || ((uintptr_t)d_lse & 3u))
    return WC_E_ARG;
  // a factor that makes every score 0 without making a mask's infinity NaN: fp32's least number
  // (the largest score then counts as 2^-21)
  const float scale = s.scale == 0.0f ? 0x1p-149f : s.scale * wc::kLog2e;
  // the strides are the lengths of the buffers' rows too: those of one token may be anything
  const bool one = s.tokens == 1u;
  const wc::Prompt a = {d_q, d_k, d_v, d_starts, d_out, d_lse, s.tokens, (uint32_t)s.q_stride,
                        (uint32_t)(one ? kv_row : s.k_stride), (uint32_t)(one ? kv_row : s.v_stride), s.seqs, s.heads,
                        s.kv_heads, s.heads / s.kv_heads, s.window, scale, scale < 0.0f ? INFINITY : -INFINITY};
  const hipStream_t st = (hipStream_t)stream;
  switch (s.head_dim / 32u) {
    case 1: return wc::launch_prompt_of<1>(a, shape, st);
    case 2: return wc::launch_prompt_of<2>(a, shape, st);
    case 3: return wc::launch_prompt_of<3>(a, shape, st);
    case 4: return wc::launch_prompt_of<4>(a, shape, st);
    case 5: return wc::launch_prompt_of<5>(a, shape, st);
    case 6: return wc::launch_prompt_of<6>(a, shape, st);
    case 7: return wc::launch_prompt_of<7>(a, shape, st);
    default: return wc::launch_prompt_of<8>(a, shape, st);
  }
}
