// wc_cache.hip — a cache of keys and values in 4 bits: append, read-back, and
// attention of a sequence's newest tokens over it (include/wc_attn.h defines the
// operators and the cache's layout).
#include "wc_attn.h"
#include "wc_launch.h"
#include "wc_skinny.h"

namespace wc {

constexpr uint32_t kTokens = 32;  // of a tile

struct Cache {
  uint8_t* data;
  uint32_t pages, page_tiles, heads, groups;
  __host__ __device__ uint32_t dim() const { return 32u * groups; }
  __host__ __device__ uint32_t tile_bytes() const { return 34u * dim(); }
  // Tile `tile` of the page (both in range) of one head.
  __device__ __forceinline__ uint8_t* at(uint32_t page, uint32_t head, uint32_t tile) const {
    return data + (((uint64_t)page * heads + head) * page_tiles + tile) * tile_bytes();
  }
};

// Places in a tile, in bytes: of the 8 codes of keys in part p (0 .. 3) of group g
// of token t, of the pair n (0 .. 15) of codes of values, and of the scales.
__device__ __forceinline__ uint32_t key_row(uint32_t t) { return 4u * (t >> 3) + (t & 3u); }
__device__ __forceinline__ uint32_t key_place(uint32_t groups, uint32_t t, uint32_t g, uint32_t p) {
  const uint32_t quad = g & ~3u, w = groups - quad < 4u ? groups - quad : 4u;
  return 4u * ((t >> 2 & 1u) * 64u * groups + quad * 64u + (16u * p + key_row(t)) * w + (g & 3u));
}
__device__ __forceinline__ uint32_t value_place(uint32_t groups, uint32_t t, uint32_t g, uint32_t n) {
  const uint32_t pair = g & ~1u, w = groups - pair < 2u ? 1u : 2u;
  return 512u * (groups + pair) + ((16u * (t >> 3) + n) * w + (g & 1u)) * 8u + (t & 7u);
}
__device__ __forceinline__ uint32_t key_scale_place(uint32_t groups, uint32_t t, uint32_t g) {
  return 1024u * groups + (2u * key_row(t) + (t >> 2 & 1u)) * groups + g;
}
__device__ __forceinline__ uint32_t value_scale_place(uint32_t groups, uint32_t t, uint32_t g) {
  return 1056u * groups + ((t >> 3) * groups + g) * 8u + (t & 7u);
}

// Append and read-back take W tokens of one head per block, in two phases joined in
// LDS: rows (a lane has 8 columns of a token) and places in the tiles.  What a token has
// in a tile lies scattered, 64 single bytes for 128 columns of values, and a store or
// load of single bytes takes as long as one of dwords; so four tokens whose slots are
// an aligned four of a tile are taken together, a dword for each pair of columns.
// 8192 tokens of 8 heads of 128: 11.6 us to append (42.5 MB, 3.7 TB/s) and 10.0 to read;
// bytes alone took 24.5 and 15.9.  W is 32, or 4 where that leaves compute units without a
// block (32 tokens: 3.5 and 3.4 us, of which 2.4 are an empty kernel's; windows of 32 took
// 4.8 and 4.7).
constexpr uint32_t kManyTokens = 32, kFewTokens = 4;

template <uint32_t W>
struct Window {
  const uint8_t* tile[W];  // null: no such slot
  uint8_t place[W];        // in the tile
  bool four[W];            // the token's aligned four is in the window, in order

  // Called by the whole block; a barrier has to follow.
  __device__ __forceinline__ void open(const Cache& c, const int64_t* slots, uint64_t token0, uint32_t n,
                                       uint32_t head) {
    const uint32_t i = threadIdx.x;
    if (i >= W) return;  // part of the first wave
    const int64_t slot = i < n ? slots[token0 + i] : -1;
    const bool in = (uint64_t)slot < (uint64_t)c.pages * c.page_tiles * kTokens;
    const uint32_t t = in ? (uint32_t)(slot >> 5) : 0u;  // below 2^31 (cache_ok)
    const uint32_t page = t / c.page_tiles, p = (uint32_t)slot & 3u;
    tile[i] = in ? c.at(page, head, t - page * c.page_tiles) : nullptr;
    place[i] = (uint8_t)(slot & 31);
    // lane i - p holds slot - p, and the three after it follow
    bool runs = in;
#pragma unroll
    for (int o = 1; o < 4; ++o) {
      const int64_t next = __shfl_down((long long)slot, o, (int)W);
      runs = runs && i + o < n && next == slot + o;
    }
    const uint64_t heads = __ballot(runs && p == 0u);
    four[i] = in && i >= p && (heads >> (i - p) & 1u);
  }
};

template <int G, uint32_t W>
__global__ __launch_bounds__(kBlockThreads) void k_cache_append(Cache c, const uint16_t* __restrict__ k,
                                                                uint64_t k_stride,
                                                                const uint16_t* __restrict__ v,
                                                                uint64_t v_stride,
                                                                const int64_t* __restrict__ slots,
                                                                uint64_t tokens) {
  constexpr uint32_t kParts = 4u * G, kUnits = 2u * kParts * W;  // parts of a row: 8 columns each
  constexpr int kRounds = (kUnits + kBlockThreads - 1) / kBlockThreads;
  __shared__ Window<W> w;
  __shared__ uint32_t codes[2][W][kParts];
  __shared__ uint8_t scales[2][W][G];
  const uint32_t head = blockIdx.x % c.heads;
  const uint64_t token0 = (uint64_t)(blockIdx.x / c.heads) * W;
  const uint32_t n = tokens - token0 < W ? (uint32_t)(tokens - token0) : W;
  u32x4 x[kRounds];
  each<kRounds>([&](auto i) __attribute__((always_inline)) {
    const uint32_t u = (i * kBlockThreads + threadIdx.x) % kUnits;  // whole quads of lanes share a group
    const uint32_t part = u % kParts, t = u / kParts % W;
    const uint64_t row = token0 + (t < n ? t : n - 1u);
    x[i] = *(const u32x4*)((u / (kParts * W) ? v + row * v_stride : k + row * k_stride) + head * 32u * G + 8u * part);
  });
  w.open(c, slots, token0, n, head);
  each<kRounds>([&](auto i) __attribute__((always_inline)) {
    const uint32_t u = (i * kBlockThreads + threadIdx.x) % kUnits;  // past the last: the same again
    const uint32_t part = u % kParts, t = u / kParts % W, kind = u / (kParts * W);
    uint32_t m = max_abs8(x[i]);
    const uint32_t a = (uint32_t)__shfl_xor((int)m, 1, kWave);
    m = m > a ? m : a;
    const uint32_t b = (uint32_t)__shfl_xor((int)m, 2, kWave);
    m = m > b ? m : b;
    const uint32_t e = fp4_exponent(m);
    codes[kind][t][part] = fp4_pack8(x[i], e);
    if (part % 4u == 0) scales[kind][t][part / 4u] = (uint8_t)e;
  });
  __syncthreads();
  // keys: a part of a quad of groups
  constexpr uint32_t kQuads = (G + 3) / 4;
  for (uint32_t u = threadIdx.x; u < W * 4u * kQuads; u += kBlockThreads) {
    const uint32_t p = u % 4u, quad = u / 4u % kQuads * 4u, t = u / (4u * kQuads);
    if (!w.tile[t]) continue;
    uint32_t* const to = (uint32_t*)(w.tile[t] + key_place(G, w.place[t], quad, p));
    if (G % 4 == 0) {
      *(u32x4*)to = u32x4{codes[0][t][4u * quad + p], codes[0][t][4u * quad + 4u + p],
                          codes[0][t][4u * quad + 8u + p], codes[0][t][4u * quad + 12u + p]};
    } else {
      for (uint32_t i = 0; i < 4u && quad + i < (uint32_t)G; ++i) to[i] = codes[0][t][4u * (quad + i) + p];
    }
  }
  // values: four bytes of a token, or one of four tokens
  for (uint32_t u = threadIdx.x; u < W * kParts; u += kBlockThreads) {
    const uint32_t part = u % kParts, g = part / 4u, t = u / kParts;
    if (!w.tile[t]) continue;
    uint8_t* const to = (uint8_t*)w.tile[t];
    if (w.four[t]) {
      const uint32_t at = w.place[t] & 3u, t0 = t - at;  // this lane: pair 4 (part % 4) + at
      uint32_t y = 0;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) y |= (codes[1][t0 + i][part] >> (8u * at) & 0xFFu) << (8u * i);
      *(uint32_t*)(to + value_place(G, w.place[t0], g, 4u * (part % 4u) + at)) = y;
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        to[value_place(G, w.place[t], g, 4u * (part % 4u) + i)] = (uint8_t)(codes[1][t][part] >> (8u * i));
    }
  }
  for (uint32_t u = threadIdx.x; u < W * G * 2u; u += kBlockThreads) {
    const uint32_t g = u % G, t = u / G % W, kind = u / (G * W);
    if (!w.tile[t]) continue;
    uint8_t* const to = (uint8_t*)w.tile[t];
    to[kind ? value_scale_place(G, w.place[t], g) : key_scale_place(G, w.place[t], g)] = scales[kind][t][g];
  }
}

template <int G, uint32_t W>
__global__ __launch_bounds__(kBlockThreads) void k_cache_read(Cache c, const int64_t* __restrict__ slots,
                                                              uint64_t tokens, uint16_t* __restrict__ k,
                                                              uint16_t* __restrict__ v) {
  constexpr uint32_t kParts = 4u * G;
  __shared__ Window<W> w;
  __shared__ __attribute__((aligned(4))) uint8_t codes[W][kParts * 4u];  // of values
  const uint32_t head = blockIdx.x % c.heads;
  const uint64_t token0 = (uint64_t)(blockIdx.x / c.heads) * W;
  const uint32_t n = tokens - token0 < W ? (uint32_t)(tokens - token0) : W;
  w.open(c, slots, token0, n, head);
  __syncthreads();
  for (uint32_t u = threadIdx.x; u < W * kParts; u += kBlockThreads) {
    const uint32_t part = u % kParts, g = part / 4u, t = u / kParts;
    if (!w.tile[t]) continue;
    if (w.four[t]) {
      const uint32_t at = w.place[t] & 3u, t0 = t - at;
      const uint32_t x = *(const uint32_t*)(w.tile[t] + value_place(G, w.place[t0], g, 4u * (part % 4u) + at));
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) codes[t0 + i][4u * part + at] = (uint8_t)(x >> (8u * i));
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        codes[t][4u * part + i] = w.tile[t][value_place(G, w.place[t], g, 4u * (part % 4u) + i)];
    }
  }
  __syncthreads();
  for (uint32_t u = threadIdx.x; u < 2u * kParts * W; u += kBlockThreads) {
    const uint32_t part = u % kParts, g = part / 4u, t = u / kParts % W, kind = u / (kParts * W);
    if (t >= n) continue;
    uint32_t x = 0, e = 255u;  // NaN
    if (const uint8_t* const from = w.tile[t]) {
      x = kind ? *(const uint32_t*)&codes[t][4u * part]
               : *(const uint32_t*)(from + key_place(G, w.place[t], g, part % 4u));
      e = from[kind ? value_scale_place(G, w.place[t], g) : key_scale_place(G, w.place[t], g)];
    }
    const uint64_t at = ((token0 + t) * c.heads + head) * (32u * G) + 8u * part;
    *(u32x4*)((kind ? v : k) + at) = fp4_expand(x, fp4_scale(e));
  }
}

// ---- attention ---------------------------------------------------------------
//
// A block takes up to 16 queries (columns) of one sequence that share a head of
// keys, and a share of the sequence's tiles; its waves take the tiles in turn and
// join their sums at the end.  Keys times queries: one MFMA has 16 tokens as rows
// and 32 columns of the head; a lane receives the scores of 4 tokens with its query
// (column lane % 16).  The tokens are assigned to the rows so that after two of
// them a lane has the scores of the 8 tokens whose values it holds, which is the
// second product's operand as it stands: nothing crosses lanes.  Values times
// weights: rows are columns of the head, the 32 tokens are summed over; the cache
// holds for each lane the codes of its pair of columns for 8 tokens.
//
// The weights exp(s - m) go into the product as the sum of two BF16 numbers: one
// would be off by as much as the outputs' own rounding, 16 bits of it add nothing
// to that.  The second costs nothing where at most 8 columns are used (DUP): columns
// 8 .. 15 repeat the queries and take the low parts.
//
// 4 sequences of 65536 tokens, 8 heads of 128 (8 queries each): 285 MB in 57 us, 5.0 TB/s
// (a copy of 2 GiB: 4.9), and 4.8 for the join.  32 sequences of 128 to 8192 tokens: 70 MB
// in 20.5 us, of which 6 are the lengths, the pages and the first tiles, one after the
// other, and the waves' joining.  Keys and values have one set of registers each: the
// next tile's keys are asked for when the scores are made, its values when they are
// used (two sets took twice the registers, and half of the waves: 24.5 us).  The scores
// of a step are not looked through for a maximum across lanes.
//
// m is a value near the largest score so far, per query: it moves (and the sums are
// scaled) only when a score passes it by more than kSlack, so that a step needs no
// exchange between lanes.  Weights are then up to 2^kSlack, far inside fp32 and
// BF16.
constexpr uint32_t kAttnWaves = 4;
// Of a block that has a whole sequence: as many as its LDS holds the sums of.
template <int G, bool WHOLE>
constexpr uint32_t kWavesOf = WHOLE ? (G <= 4 ? 16u : 8u) : kAttnWaves;
constexpr float kSlack = 16.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct CacheAttn {
  Cache c;
  const uint16_t* q;
  uint64_t q_stride;
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;
  float* lse;   // may be null
  float* part;  // [head of keys][column tile][share + seqs blocks][columns][dim]
  float2* top;  // [..][columns]: m and the sum of weights
  uint32_t seqs, news, heads, group, width;
  uint32_t window;             // kNoWindow where there is none
  uint32_t col_tiles, share;   // share: see Shares
  float scale;                 // times log2(e)
};
constexpr uint32_t kNoWindow = 0x7FFFFFC0u;  // past any length

// The tiles of a sequence that its queries attend to.  A sequence without any counts
// as one of them, for the block that writes its empty result.
struct Span {
  int32_t len = 0;
  uint32_t first = 0, end = 0;
  __device__ __forceinline__ Span() {}
  __device__ __forceinline__ Span(const CacheAttn& a, uint32_t seq) {
    const int32_t n = a.lengths[seq];
    len = n > 0 ? n : 0;
    const uint32_t cap = a.width * a.c.page_tiles;  // at most 2^25 (attn_cut)
    end = ((uint32_t)len + 31u) / 32u;
    end = end < cap ? end : cap;
    const int32_t lo = len - (int32_t)a.news + 1 - (int32_t)a.window;
    first = lo > 0 ? (uint32_t)lo / 32u : 0u;
    first = first < end ? first : end;
  }
  __device__ __forceinline__ uint32_t count() const { return end > first ? end - first : 1u; }
};

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// Inclusive prefix sum across the wave (DPP shifts within rows of 16 lanes, then rows).
__device__ __forceinline__ uint32_t wave_upto(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);
  return v;
}

// How the blocks of a head are shared out: per = all sequences' tiles / a.share, and a
// sequence gets the fewest blocks that leave none more than per tiles.  So sequences of
// any lengths load the card evenly, with at most a.share + a.seqs blocks, and a block
// has one sequence (blocks that took equal runs of all tiles, with several sequences
// where they are short, measured 29.6 us where this takes 20.8; 32 sequences up to 8192
// tokens).  Each wave works this out from the lengths, 64 sequences at a time.
struct Shares {
  Span span;              // the lane's sequence, seq0 + lane
  uint32_t blocks, upto;  // its blocks, and those up to its last
  uint32_t seq0 = 0, per;
  __device__ __forceinline__ explicit Shares(const CacheAttn& a) {
    const uint32_t lane = (uint32_t)lane_id();
    span = lane < a.seqs ? Span(a, lane) : Span();
    uint32_t total = wave_total(lane < a.seqs ? span.count() : 0u);
    for (uint32_t s = kWave; s < a.seqs; s += kWave)
      total += wave_total(s + lane < a.seqs ? Span(a, s + lane).count() : 0u);
    per = ((total + a.share - 1u) / a.share + kAttnWaves - 1u) / kAttnWaves * kAttnWaves;
    count(a, 0);
  }
  __device__ __forceinline__ void count(const CacheAttn& a, uint32_t base) {
    blocks = seq0 + (uint32_t)lane_id() < a.seqs ? (span.count() + per - 1u) / per : 0u;
    upto = base + wave_upto(blocks);
  }
  __device__ __forceinline__ bool next(const CacheAttn& a) {
    const uint32_t base = lane_value(upto, kWave - 1);
    seq0 += kWave;
    if (seq0 >= a.seqs) return false;
    span = seq0 + (uint32_t)lane_id() < a.seqs ? Span(a, seq0 + (uint32_t)lane_id()) : Span();
    count(a, base);
    return true;
  }
  // The lane with the sequence of block b; -1: there is no such block.  Wave-uniform.
  __device__ __forceinline__ int owner(const CacheAttn& a, uint32_t b) {
    do {
      const uint64_t hit = __ballot(b < upto);
      if (hit) return __ffsll((unsigned long long)hit) - 1;
    } while (next(a));
    return -1;
  }
  __device__ __forceinline__ int find(const CacheAttn& a, uint32_t seq) {
    while (seq >= seq0 + kWave) next(a);
    return (int)(seq - seq0);
  }
};

// N dwords at byte `off` (4 N bytes aligned for N = 1, 2, 4).
template <int N>
__device__ __forceinline__ void load_dwords(buffer b, uint32_t off, uint32_t* to) {
  if constexpr (N >= 4) {
    const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
    each<4>([&](auto i) __attribute__((always_inline)) { to[i] = x[+i]; });
    load_dwords<N - 4>(b, off + 16u, to + 4);
  } else if constexpr (N >= 2) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, (int)off, 0, 0));
    to[0] = x[0];
    to[1] = x[1];
    load_dwords<N - 2>(b, off + 8u, to + 2);
  } else if constexpr (N == 1) {
    to[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(b, (int)off, 0, 0);
  }
}

// A lane's keys of a tile, and their scales (byte half G + g).
template <int G>
struct KeyRegs {
  uint32_t codes[2][G], scales[(2 * G + 3) / 4];
  __device__ __forceinline__ void load(buffer b, uint32_t lane) {
    const uint32_t r = lane & 15u;
    each<2>([&](auto half) __attribute__((always_inline)) {
      each<(G + 3) / 4>([&](auto z) __attribute__((always_inline)) {
        constexpr int w = G - 4 * z < 4 ? G - 4 * z : 4;
        load_dwords<w>(b, lane * (w * 4u) + half * 256u * G + z * 1024u, &codes[half][4 * z]);
      });
    });
    const uint32_t off = 1024u * G + r * 2u * G;
    if constexpr (G % 2 == 0) {
      load_dwords<G / 2>(b, off, scales);
    } else {
      each<(2 * G + 3) / 4>([&](auto i) __attribute__((always_inline)) {
        scales[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, (int)(off + 4u * i), 0, 0);
        if constexpr (2 * i + 1 < G)
          scales[i] |= (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, (int)(off + 4u * i + 2u), 0, 0) << 16;
      });
    }
  }
};

// A lane's values: its pair of columns of each group for 8 tokens, and their scales.
template <int G>
struct ValueRegs {
  uint32_t codes[G][2], scales[G][2];
  __device__ __forceinline__ void load(buffer b, uint32_t lane) {
    const uint32_t h = lane >> 4;
    each<(G + 1) / 2>([&](auto p) __attribute__((always_inline)) {
      constexpr int w = 2 * p + 1 < G ? 4 : 2;
      load_dwords<w>(b, 512u * G + p * 1024u + lane * (w * 4u), codes[2 * p]);
    });
    load_dwords<2 * G>(b, 1056u * G + h * 8u * G, scales[0]);
  }
};

// Byte b (constant) of w as a scale.
template <int B>
__device__ __forceinline__ float scale_of(uint32_t w) {
  const uint32_t e = B == 0 ? w << 23 : B == 1 ? w << 15 : B == 2 ? w << 7 : w >> 1;
  return __uint_as_float(e & 0x7F800000u);
}

template <int B>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, B));
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, mfma_bf16x2));
}

// 0xFF in the bytes of x that are 0xFF, else 0.
__device__ __forceinline__ uint32_t bytes_ff(uint32_t x) {
  const uint32_t t = x & ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return (t >> 7) * 0xFFu;
}

// WHOLE: a block has a whole sequence, nothing is left to join.
template <int G, bool DUP, bool WHOLE>
__global__ __launch_bounds__(kWave * (kWavesOf<G, WHOLE>), G <= 4 ? 4 : 2) void k_cache_attention(CacheAttn a) {
  constexpr uint32_t D = 32u * G, kCols = DUP ? 8u : 16u, kWaves = (kWavesOf<G, WHOLE>);
  constexpr uint32_t kHeld = 4u * kCols;  // lanes whose sums are kept
  __shared__ mfma_f32x4 sums[kWaves][G][2][kHeld];
  __shared__ float tops[kWaves][16], totals[kWaves][16];
  const uint32_t wave = (uint32_t)wave_in_block();
  const uint32_t kv = blockIdx.x % a.c.heads, rest = blockIdx.x / a.c.heads;
  const uint32_t ct = rest % a.col_tiles, block = rest / a.col_tiles;
  const uint32_t lane = (uint32_t)lane_id(), h = lane >> 4;
  uint32_t seq = block, blocks = 1, share = 0;  // share: which one of the sequence's
  int32_t len;
  uint32_t first, end;
  if constexpr (WHOLE) {
    const Span span(a, seq);
    len = span.len;
    first = span.first;
    end = span.end;
  } else {
    Shares shares(a);
    const int owner = shares.owner(a, block);
    if (owner < 0) return;
    seq = shares.seq0 + (uint32_t)owner;
    blocks = lane_value(shares.blocks, owner);
    share = block - (lane_value(shares.upto, owner) - blocks);
    len = (int32_t)lane_value((uint32_t)shares.span.len, owner);
    first = lane_value(shares.span.first, owner);
    end = lane_value(shares.span.end, owner);
  }
  const uint32_t most_tiles = (end - first + blocks - 1u) / blocks, tile0 = first + share * most_tiles;
  const uint32_t tiles = tile0 < end ? (end - tile0 < most_tiles ? end - tile0 : most_tiles) : 0u;

  // The pages of 64 tiles, one per lane, and of the next 64; ~0 where there is none.
  auto pages = [&](uint32_t i) __attribute__((always_inline)) {
    return i + lane < tiles ? (uint32_t)a.table[(uint64_t)seq * a.width + (tile0 + i + lane) / a.c.page_tiles] : ~0u;
  };
  // (a whole sequence's first pages do not wait for its length)
  uint32_t page_of = ~0u;
  if (WHOLE && a.window == kNoWindow)
    page_of = lane < a.width * a.c.page_tiles ? (uint32_t)a.table[(uint64_t)seq * a.width + lane / a.c.page_tiles] : ~0u;
  else
    page_of = pages(0);
  uint32_t ahead = tiles > (uint32_t)kWave ? pages(kWave) : ~0u;
  uint32_t in_page = (tile0 + wave) % a.c.page_tiles;  // the next tile's place
  const uint32_t in_step = kWaves % a.c.page_tiles;
  // the lane's query; columns past the last repeat it
  const uint32_t cols = a.news * a.group;
  uint32_t col = ct * kCols + (lane & (kCols - 1u));
  col = col < cols ? col : cols - 1u;
  const uint32_t qi = col / a.group, head = kv * a.group + col - qi * a.group;
  const int32_t hi = len - (int32_t)a.news + (int32_t)qi;  // its position
  u32x4 q[G];
  {
    const uint16_t* from = a.q + ((uint64_t)seq * a.news + qi) * a.q_stride + (uint64_t)head * D + 8u * h;
    each<G>([&](auto g) __attribute__((always_inline)) { q[g] = *(const u32x4*)(from + 32 * g); });
  }

  float m = -INFINITY, off = 0, sum = 0;  // off: m, or 0 while there is none
  uint32_t spoilt = 0;                    // groups in which the query attends to a value that is NaN
  mfma_f32x4 acc[G][2];
  each<G>([&](auto g) __attribute__((always_inline)) { acc[g][0] = acc[g][1] = mfma_f32x4{0, 0, 0, 0}; });

  // The wave's tiles are wave, wave + kWaves, ..  Past the last one and where there
  // is no page loads bring 0 and touch no memory.
  auto next_of = [&](uint32_t i, bool& bad) __attribute__((always_inline)) {
    const uint32_t page = lane_value(page_of, (int)(i % kWave));
    bad = page >= a.c.pages;
    const bool none = bad || i >= tiles;
    const uint64_t tile = ((uint64_t)(none ? 0u : page) * a.c.heads + kv) * a.c.page_tiles + in_page;
    in_page += in_step;
    in_page = in_page >= a.c.page_tiles ? in_page - a.c.page_tiles : in_page;
    return buffer_of(a.c.data + tile * a.c.tile_bytes(), none ? 0u : a.c.tile_bytes());
  };
  KeyRegs<G> k;
  ValueRegs<G> v;
  bool bad = false;
  if (wave < tiles) {
    const buffer t = next_of(wave, bad);
    k.load(t, lane);
    v.load(t, lane);
  }
  for (uint32_t i = wave; i < tiles; i += kWaves) {
    if ((i + kWaves) / kWave != i / kWave) {
      page_of = ahead;
      ahead = pages((i / kWave + 2u) * kWave);
    }
    const int32_t p0 = (int32_t)((tile0 + i) * 32u);
    bool next_bad;
    const buffer next = next_of(i + kWaves, next_bad);
    // some query does not attend to some token (wave-uniform)
    const bool edge = bad || p0 + 31 > len - (int32_t)a.news || p0 <= len - 1 - (int32_t)a.window;
    float s[8];
    each<2>([&](auto half) __attribute__((always_inline)) {
      mfma_f32x4 x = {0, 0, 0, 0};
      each<G>([&](auto g) __attribute__((always_inline)) {
        constexpr int at = half * G + g;
        x = mfma16(fp4_expand(k.codes[half][g], scale_of<at % 4>(k.scales[at / 4])), q[g], x);
      });
      each<4>([&](auto j) __attribute__((always_inline)) { s[4 * half + j] = x[+j] * a.scale; });
    });
    __builtin_amdgcn_sched_barrier(0);
    k.load(next, lane);
    if (edge) {
      uint32_t mine[2] = {0, 0}, any[2] = {0, 0};  // tokens that this query, that some query attends to
      each<8>([&](auto j) __attribute__((always_inline)) {
        const int32_t p = p0 + (int32_t)(8u * h) + j;
        const bool ok = (uint32_t)(hi - p) < a.window;
        s[j] = bad ? NAN : s[j];
        s[j] = ok ? s[j] : -INFINITY;
        mine[j / 4] |= ok ? 0xFFu << (8 * (j % 4)) : 0u;
        any[j / 4] |= (uint32_t)(len - 1 - p) < a.window + a.news - 1u ? 0xFFu << (8 * (j % 4)) : 0u;
      });
      // What no query attends to may hold anything and becomes 0.  A NaN scale stands
      // for 32 NaN values: they become 0 too, and the group is NaN at the end for the
      // queries that attend to it.
      each<G>([&](auto g) __attribute__((always_inline)) {
        each<2>([&](auto j) __attribute__((always_inline)) {
          const uint32_t nan = bytes_ff(v.scales[g][j]);
          spoilt |= nan & mine[j] ? 1u << g : 0u;
          v.codes[g][j] &= any[j] & ~nan;
          v.scales[g][j] &= any[j] & ~nan;
        });
      });
    }
    float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
    if (__ballot(top > m + kSlack)) {
      top = fmaxf(top, __shfl_xor(top, 16, kWave));
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      // queries that need not move keep theirs: no query's bits depend on another's
      const float now = top > m + kSlack ? top : m, to = now == -INFINITY ? 0.0f : now;
      const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(off - to);
      m = now;
      off = to;
      sum *= f;
      each<G>([&](auto g) __attribute__((always_inline)) {
        acc[g][0] *= f;
        acc[g][1] *= f;
      });
    }
    each<8>([&](auto j) __attribute__((always_inline)) {
      s[j] = __builtin_amdgcn_exp2f(s[j] - off);
      sum += s[j];
    });
    u32x4 high, low;
    each<4>([&](auto j) __attribute__((always_inline)) {
      const uint32_t x = bf16_pair(s[2 * j], s[2 * j + 1]);
      high[+j] = x;
      low[+j] = bf16_pair(s[2 * j] - __uint_as_float(x << 16), s[2 * j + 1] - __uint_as_float(x & 0xFFFF0000u));
    });
    if constexpr (DUP) high = lane & 8u ? low : high;
    each<G>([&](auto g) __attribute__((always_inline)) {
      uint32_t d[8];
      each<2>([&](auto j) __attribute__((always_inline)) {
        each<4>([&](auto n) __attribute__((always_inline)) {
          d[4 * j + n] = fp4_pair<n>(v.codes[g][j], scale_of<n>(v.scales[g][j]));
        });
      });
      u32x4 even, odd;  // columns of the lane's pair
      each<4>([&](auto j) __attribute__((always_inline)) {
        even[+j] = __builtin_amdgcn_perm(d[2 * j + 1], d[2 * j], 0x05040100u);
        odd[+j] = __builtin_amdgcn_perm(d[2 * j + 1], d[2 * j], 0x07060302u);
      });
      acc[g][0] = mfma16(even, high, acc[g][0]);
      acc[g][1] = mfma16(odd, high, acc[g][1]);
      if constexpr (!DUP) {
        acc[g][0] = mfma16(even, low, acc[g][0]);
        acc[g][1] = mfma16(odd, low, acc[g][1]);
      }
    });
    __builtin_amdgcn_sched_barrier(0);
    v.load(next, lane);
    bad = next_bad;
  }
  // a query at a position past the table attends to itself, which is not there
  if (hi >= 0 && (uint32_t)hi / 32u >= a.width * a.c.page_tiles) sum = NAN;

  sum += __shfl_xor(sum, 16, kWave);
  sum += __shfl_xor(sum, 32, kWave);
  if (__ballot(spoilt)) {
    spoilt |= (uint32_t)__shfl_xor((int)spoilt, 16, kWave);
    spoilt |= (uint32_t)__shfl_xor((int)spoilt, 32, kWave);
    each<G>([&](auto g) __attribute__((always_inline)) {
      if (spoilt >> g & 1u) acc[g][0] = acc[g][1] = mfma_f32x4{NAN, NAN, NAN, NAN};
    });
  }
  // The waves' sums, on the largest of their offsets, in order.
  if (lane < 16u) tops[wave][lane] = m;
  __syncthreads();
  float most = -INFINITY;
  each<kWaves>([&](auto i) __attribute__((always_inline)) { most = fmaxf(most, tops[i][lane & 15u]); });
  const float scale = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - most);  // without an offset all is 0 or NaN
  if (lane < 16u) totals[wave][lane] = sum * scale;
  const uint32_t held = DUP ? 8u * h + (lane & 7u) : lane;
  each<G>([&](auto g) __attribute__((always_inline)) {
    mfma_f32x4 x = acc[g][0] * scale, y = acc[g][1] * scale;
    if constexpr (DUP) {  // the products with the low parts are 8 lanes further
      each<4>([&](auto i) __attribute__((always_inline)) {
        x[+i] += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x[+i]), 0x128, 0xF, 0xF, true));
        y[+i] += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(y[+i]), 0x128, 0xF, 0xF, true));
      });
    }
    // the lane's columns of the group in order: 8 h .. 8 h + 7
    if (!DUP || !(lane & 8u)) {
      sums[wave][g][0][held] = mfma_f32x4{x[0], y[0], x[1], y[1]};
      sums[wave][g][1][held] = mfma_f32x4{x[2], y[2], x[3], y[3]};
    }
  });
  __syncthreads();
  const uint64_t at = (((uint64_t)kv * a.col_tiles + ct) * (a.share + a.seqs) + block) * kCols;
  for (uint32_t i = threadIdx.x; i < G * 2u * kHeld; i += kWaves * kWave) {
    const uint32_t l = i % kHeld, c = l % kCols;
    // of group i / (2 kHeld), its half p: 4 columns from 32 g + 8 (l / kCols) + 4 p on
    const uint32_t to = (i / (2u * kHeld)) * 32u + l / kCols * 8u + i / kHeld % 2u * 4u;
    mfma_f32x4 x = {0, 0, 0, 0};
    float total = 0;
    each<kWaves>([&](auto n) __attribute__((always_inline)) {
      x += (&sums[n][0][0][0])[i];
      total += totals[n][c];
    });
    const uint32_t mine = ct * kCols + c;
    if (mine >= cols) continue;
    const uint32_t qj = mine / a.group;
    const uint64_t row = ((uint64_t)seq * a.news + qj) * a.heads + kv * a.group + mine - qj * a.group;
    if (blocks == 1u) {
      const float by = total == 0.0f ? 0.0f : 1.0f / total;
      uint2 o;
      o.x = bf16_pair(x[0] * by, x[1] * by);
      o.y = bf16_pair(x[2] * by, x[3] * by);
      *(uint2*)(a.out + row * D + to) = o;
    } else {
      *(mfma_f32x4*)(a.part + (at + c) * D + to) = x;
    }
    if (i < kCols) {
      float top = -INFINITY;
      each<kWaves>([&](auto n) __attribute__((always_inline)) { top = fmaxf(top, tops[n][c]); });
      if (blocks != 1u)
        a.top[at + c] = make_float2(top, total);
      else if (a.lse)
        a.lse[row] = total == 0.0f ? -INFINITY : (top == -INFINITY ? total : (top + __builtin_amdgcn_logf(total)) * kLn2);
    }
  }
}

// The shares of a query's sequence, joined by a block: D / 4 lanes take a share's sums,
// four shares' loads go out together.
template <int G>
__global__ __launch_bounds__(kBlockThreads) void k_cache_join(CacheAttn a, uint32_t cols_of_tile) {
  constexpr uint32_t D = 32u * G, kLanes = D / 4u, kSets = kBlockThreads / kLanes, kWaves = kBlockThreads / kWave;
  __shared__ float2 both[kWaves];
  __shared__ mfma_f32x4 sums[kSets][kLanes];
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block();
  const uint64_t row = blockIdx.x;
  const uint32_t head = (uint32_t)(row % a.heads), token = (uint32_t)(row / a.heads);
  const uint32_t seq = token / a.news, qi = token - seq * a.news;
  Shares shares(a);
  const int owner = shares.find(a, seq);
  const uint32_t n = lane_value(shares.blocks, owner), block0 = lane_value(shares.upto, owner) - n;
  if (n == 1u) return;
  const uint32_t kv = head / a.group, col = qi * a.group + head - kv * a.group;
  const uint32_t ct = col / cols_of_tile;
  const uint64_t from = (((uint64_t)kv * a.col_tiles + ct) * (a.share + a.seqs) + block0) * cols_of_tile +
                        (col - ct * cols_of_tile);
  auto place = [&](uint32_t s) __attribute__((always_inline)) { return from + (uint64_t)s * cols_of_tile; };
  float most = -INFINITY, total = 0;
  for (uint32_t s = threadIdx.x; s < n; s += kBlockThreads) most = fmaxf(most, a.top[place(s)].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, kWave));
  if (lane == 0) both[wave].x = most;
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < kWaves; ++i) most = fmaxf(most, both[i].x);
  for (uint32_t s = threadIdx.x; s < n; s += kBlockThreads) {
    const float2 t = a.top[place(s)];
    total += t.x == -INFINITY ? t.y : __builtin_amdgcn_exp2f(t.x - most) * t.y;  // t.y is 0 or NaN there
  }
  total = wave_sum_f32(total);
  if (lane == 0) both[wave].y = total;
  const uint32_t set = threadIdx.x / kLanes, mine = threadIdx.x - set * kLanes;
  mfma_f32x4 x = {0, 0, 0, 0};
  if (set < kSets) {
    for (uint32_t s0 = set; s0 < n; s0 += 4u * kSets) {
      float w[4];
      mfma_f32x4 y[4];
      each<4>([&](auto i) __attribute__((always_inline)) {
        const bool in = s0 + kSets * i < n;
        const uint64_t at = place(in ? s0 + kSets * i : s0);
        const float t = a.top[at].x;
        w[i] = in && t != -INFINITY ? __builtin_amdgcn_exp2f(t - most) : 0.0f;
        y[i] = *(const mfma_f32x4*)(a.part + at * D + 4u * mine);
      });
      each<4>([&](auto i) __attribute__((always_inline)) { x += w[i] * y[i]; });
    }
    sums[set][mine] = x;
  }
  __syncthreads();
  total = 0;
#pragma unroll
  for (uint32_t i = 0; i < kWaves; ++i) total += both[i].y;
  if (set == 0) {
#pragma unroll
    for (uint32_t i = 1; i < kSets; ++i) x += sums[i][mine];
    const float by = total == 0.0f ? 0.0f : 1.0f / total;
    uint2 o;
    o.x = bf16_pair(x[0] * by, x[1] * by);
    o.y = bf16_pair(x[2] * by, x[3] * by);
    *(uint2*)(a.out + row * D + 4u * mine) = o;
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[row] = total == 0.0f ? -INFINITY : (most == -INFINITY ? total : (most + __builtin_amdgcn_logf(total)) * kLn2);
}

namespace {

int launched() { return hipGetLastError() == hipSuccess ? WC_OK : WC_E_HIP; }

int cache_ok(const wc_fp4_cache* c) {
  if (!c || !c->d_data || !aligned16(c->d_data)) return WC_E_ARG;
  if (c->head_dim < 32u || c->head_dim > WC_ATTN_MAX_DIM || c->head_dim % 32u) return WC_E_ARG;
  if (c->kv_heads < 1u || c->kv_heads > WC_ATTN_MAX_HEADS) return WC_E_ARG;
  if (c->page_size < 32u || c->page_size > (1u << 20) || c->page_size % 32u) return WC_E_ARG;
  if (c->pages < 1u) return WC_E_ARG;
  if (c->pages >= (1ull << 31) || c->pages * c->page_size >= (1ull << 36)) return WC_E_SIZE;
  return WC_OK;
}
Cache cache_of(const wc_fp4_cache* c) {
  return {c->d_data, (uint32_t)c->pages, c->page_size / 32u, c->kv_heads, c->head_dim / 32u};
}

// launch(first token, tokens, blocks, W) for windows of W tokens, a block for each and
// each head, in launches of fewer than 2^32 threads.
template <typename F>
int each_windows(uint64_t tokens, uint32_t heads, F&& launch) {
  const bool few = tokens / kManyTokens * heads < cu_count();
  const uint64_t most = (1ull << 23) / heads * kManyTokens;
  for (uint64_t t = 0; t < tokens; t += most) {
    const uint64_t n = tokens - t < most ? tokens - t : most;
    if (few)
      launch(t, n, (uint32_t)((n + kFewTokens - 1u) / kFewTokens * heads), std::integral_constant<uint32_t, kFewTokens>{});
    else
      launch(t, n, (uint32_t)((n + kManyTokens - 1u) / kManyTokens * heads), std::integral_constant<uint32_t, kManyTokens>{});
    if (const int v = launched()) return v;
  }
  return WC_OK;
}

// f(groups) with the number of groups as a constant.
template <typename F>
void by_groups(uint32_t groups, F&& f) {
  switch (groups) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 5: f(std::integral_constant<int, 5>{}); break;
    case 6: f(std::integral_constant<int, 6>{}); break;
    case 7: f(std::integral_constant<int, 7>{}); break;
    default: f(std::integral_constant<int, 8>{}); break;
  }
}

// How a call is cut: columns of a tile, tiles of columns, and Shares' share.
struct Cut {
  uint32_t cols, col_tiles, share;
  uint64_t blocks;  // of a head of keys and a tile of columns
  bool whole;       // a block for each sequence
};
int attn_cut(const wc_fp4_cache* c, const wc_fp4_attention_shape* s, Cut* cut) {
  if (!s || s->new_tokens < 1u || s->new_tokens > WC_ATTN_MAX_NEW) return WC_E_UNSUPPORTED;
  if (s->heads < 1u || s->heads > WC_ATTN_MAX_HEADS || s->heads % c->kv_heads) return WC_E_ARG;
  const uint64_t cap = (uint64_t)s->table_width * (c->page_size / 32u);
  if (cap > (1ull << 25)) return WC_E_SIZE;  // positions below 2^30
  const uint32_t cols = s->new_tokens * (s->heads / c->kv_heads);
  cut->cols = cols <= 8u ? 8u : 16u;
  cut->col_tiles = (cols + cut->cols - 1u) / cut->cols;
  uint64_t tiles = cap ? cap : 1u;  // of a sequence, at most
  if (s->window) {
    const uint64_t most = ((uint64_t)s->window + s->new_tokens - 1u + 30u) / 32u + 1u;
    tiles = most < tiles ? most : tiles;
  }
  const uint64_t all = tiles * s->seqs, rows = (uint64_t)c->kv_heads * cut->col_tiles;
  if (all >= (1ull << 30) || (uint64_t)s->seqs * s->new_tokens * s->heads >= (1ull << 24)) return WC_E_SIZE;
  // Whole sequences where a wave has at most four tiles of them and half of the card has
  // a block, or where it has one: a block alone draws little from memory.  us in a graph,
  // whole / split and joined, 32 heads on 8 of 128:
  //   whole by the rule   1 x 500 8.2 / 9.5, 16 x 1000 12.2 / 14.0, 16 x 2000 17.9 / 18.6,
  //                       32 x 2000 20.0 / 25.5, 64 x 2000 38.8 / 36.1
  //   split by the rule   1 x 1000 10.2 / 9.5, 1 x 1500 12.9 / 9.8, 1 x 2048 15.5 / 10.3,
  //                       4 x 2000 15.8 / 11.4, 8 x 2000 16.2 / 14.3, 32 x 4000 34.1 / 37.1
  // and 16 x 1000 of other head dims 7.1 / 10.9 (32), 8.3 / 11.5 (64), 13.7 / 16.1 (160),
  // 15.7 / 18.1 (256).  The lengths are on the device, so the rule goes by what the table
  // or the window allows: 16 x 1000 in a table of 2048 pages of 64 take the split, 14.6.
  const uint64_t waves = c->head_dim <= 128u ? 16u : 8u;
  cut->whole = tiles <= waves || (tiles <= 4u * waves && rows * s->seqs >= cu_count() / 2u);
  // four blocks to a compute unit (32 sequences to 8192: 27.2 us; three 28.6, two 32.1, six 29.1)
  uint64_t share = (4u * cu_count() + rows - 1u) / rows;
  share = share > s->seqs + share / 4u ? share - s->seqs : share / 4u + 1u;  // with seqs blocks more the card is full
  const uint64_t most = (all + kAttnWaves - 1u) / kAttnWaves;  // a tile for each wave
  share = share < most ? share : most;
  cut->share = cut->whole ? 0u : share ? (uint32_t)share : 1u;
  cut->blocks = cut->share + s->seqs;
  if (cut->blocks * rows >= (1ull << 22)) return WC_E_SIZE;  // grids of fewer than 2^32 threads
  return WC_OK;
}
uint64_t attn_partials(const wc_fp4_cache* c, const Cut& cut) {
  return cut.whole ? 0u : (uint64_t)c->kv_heads * cut.col_tiles * cut.blocks * cut.cols;
}

template <int G>
void launch_attention(const CacheAttn& a, const Cut& cut, hipStream_t s) {
  const uint32_t blocks = a.c.heads * cut.col_tiles * (uint32_t)cut.blocks;
  if (cut.whole) {
    constexpr uint32_t kThreads = kWave * (kWavesOf<G, true>);
    if (cut.cols == 8u)
      k_cache_attention<G, true, true><<<blocks, kThreads, 0, s>>>(a);
    else
      k_cache_attention<G, false, true><<<blocks, kThreads, 0, s>>>(a);
    return;
  }
  if (cut.cols == 8u)
    k_cache_attention<G, true, false><<<blocks, kWave * kAttnWaves, 0, s>>>(a);
  else
    k_cache_attention<G, false, false><<<blocks, kWave * kAttnWaves, 0, s>>>(a);
  k_cache_join<G><<<a.seqs * a.news * a.heads, kBlockThreads, 0, s>>>(a, cut.cols);
}

}  // namespace
}  // namespace wc

extern "C" int wc_fp4_cache_append(const wc_fp4_cache* cache, const uint16_t* d_k, uint64_t k_stride,
                                   const uint16_t* d_v, uint64_t v_stride, const int64_t* d_slots,
                                   uint64_t tokens, void* stream) {
  if (const int v = wc::cache_ok(cache)) return v;
  const uint64_t row = (uint64_t)cache->kv_heads * cache->head_dim;
  if (tokens >= (1ull << 31) || k_stride >= (1ull << 31) || v_stride >= (1ull << 31)) return WC_E_SIZE;
  if (k_stride % 8u || v_stride % 8u || (tokens > 1u && (k_stride < row || v_stride < row))) return WC_E_ARG;
  if (tokens == 0) return WC_OK;
  if (!d_k || !wc::aligned16(d_k) || !d_v || !wc::aligned16(d_v) || !d_slots || ((uintptr_t)d_slots & 7u))
    return WC_E_ARG;
  const wc::Cache c = wc::cache_of(cache);
  return wc::each_windows(tokens, c.heads, [&](uint64_t t, uint64_t n, uint32_t blocks, auto w) {
    wc::by_groups(c.groups, [&](auto g) {
      wc::k_cache_append<decltype(g)::value, decltype(w)::value><<<blocks, wc::kBlockThreads, 0, (hipStream_t)stream>>>(
          c, d_k + t * k_stride, k_stride, d_v + t * v_stride, v_stride, d_slots + t, n);
    });
  });
}

extern "C" int wc_fp4_cache_read(const wc_fp4_cache* cache, const int64_t* d_slots, uint64_t tokens,
                                 uint16_t* d_k, uint16_t* d_v, void* stream) {
  if (const int v = wc::cache_ok(cache)) return v;
  if (tokens >= (1ull << 31)) return WC_E_SIZE;
  if (tokens == 0) return WC_OK;
  if (!d_k || !wc::aligned16(d_k) || !d_v || !wc::aligned16(d_v) || !d_slots || ((uintptr_t)d_slots & 7u))
    return WC_E_ARG;
  const wc::Cache c = wc::cache_of(cache);
  const uint64_t row = (uint64_t)cache->kv_heads * cache->head_dim;
  return wc::each_windows(tokens, c.heads, [&](uint64_t t, uint64_t n, uint32_t blocks, auto w) {
    wc::by_groups(c.groups, [&](auto g) {
      wc::k_cache_read<decltype(g)::value, decltype(w)::value><<<blocks, wc::kBlockThreads, 0, (hipStream_t)stream>>>(
          c, d_slots + t, n, d_k + t * row, d_v + t * row);
    });
  });
}

extern "C" size_t wc_fp4_attention_workspace_bytes(const wc_fp4_cache* cache,
                                                   const wc_fp4_attention_shape* shape) {
  wc::Cut cut;
  if (wc::cache_ok(cache) || wc::attn_cut(cache, shape, &cut)) return 0;
  const uint64_t n = wc::attn_partials(cache, cut);
  return n * (cache->head_dim + 2u) * 4u;
}

extern "C" int wc_fp4_attention(const wc_fp4_cache* cache, const wc_fp4_attention_shape* shape,
                                const uint16_t* d_q, const int32_t* d_table, const int32_t* d_lengths,
                                uint16_t* d_out, float* d_lse, void* d_work, size_t work_bytes,
                                void* stream) {
  if (const int v = wc::cache_ok(cache)) return v;
  wc::Cut cut;
  if (const int v = wc::attn_cut(cache, shape, &cut)) return v;
  if (shape->seqs == 0) return WC_OK;
  const uint64_t row = (uint64_t)shape->heads * cache->head_dim;
  if (shape->q_stride >= (1ull << 31)) return WC_E_SIZE;
  if (shape->q_stride % 8u || ((uint64_t)shape->seqs * shape->new_tokens > 1u && shape->q_stride < row))
    return WC_E_ARG;
  if (!d_q || !wc::aligned16(d_q) || !d_out || !wc::aligned16(d_out) || ((uintptr_t)d_lse & 3u)) return WC_E_ARG;
  if (!d_lengths || ((uintptr_t)d_lengths & 3u)) return WC_E_ARG;
  if (shape->table_width && (!d_table || ((uintptr_t)d_table & 3u))) return WC_E_ARG;
  const uint64_t n = wc::attn_partials(cache, cut);
  if (n) {
    if (!d_work || !wc::aligned16(d_work)) return WC_E_ARG;
    if (work_bytes < n * (cache->head_dim + 2u) * 4u) return WC_E_SIZE;
  }
  wc::CacheAttn a;
  a.c = wc::cache_of(cache);
  a.q = d_q;
  a.q_stride = shape->q_stride;
  a.table = d_table;
  a.lengths = d_lengths;
  a.out = d_out;
  a.lse = d_lse;
  a.part = (float*)d_work;
  a.top = (float2*)(a.part + n * cache->head_dim);
  a.seqs = shape->seqs;
  a.news = shape->new_tokens;
  a.heads = shape->heads;
  a.group = shape->heads / cache->kv_heads;
  a.width = shape->table_width;
  a.window = shape->window && shape->window < wc::kNoWindow ? shape->window : wc::kNoWindow;
  a.col_tiles = cut.col_tiles;
  a.share = cut.share;
  a.scale = shape->scale * wc::kLog2e;
  wc::by_groups(a.c.groups, [&](auto g) { wc::launch_attention<decltype(g)::value>(a, cut, (hipStream_t)stream); });
  return wc::launched();
}
