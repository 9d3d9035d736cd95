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

// A lane's 8 columns of a token's keys or values.
struct RowPart {
  uint64_t token;
  uint32_t head, group, part;
  bool values;
  __device__ __forceinline__ RowPart(uint64_t u, uint32_t per, const Cache& c) {
    token = u / per;
    uint32_t r = (uint32_t)(u - token * per);
    part = r & 3u;
    r >>= 2;
    group = r % c.groups;
    r /= c.groups;
    values = r >= c.heads;
    head = values ? r - c.heads : r;
  }
};
__device__ __forceinline__ bool slot_in(const Cache& c, int64_t slot) {
  return (uint64_t)slot < (uint64_t)c.pages * c.page_tiles * kTokens;
}
__device__ __forceinline__ uint8_t* slot_tile(const Cache& c, int64_t slot, uint32_t head) {
  const uint32_t tile = (uint32_t)(slot >> 5);  // below 2^31 (cache_ok)
  const uint32_t page = tile / c.page_tiles;
  return c.at(page, head, tile - page * c.page_tiles);
}

__global__ __launch_bounds__(kBlockThreads) void k_cache_append(Cache c, const uint16_t* __restrict__ k,
                                                                uint64_t k_stride,
                                                                const uint16_t* __restrict__ v,
                                                                uint64_t v_stride,
                                                                const int64_t* __restrict__ slots,
                                                                uint64_t tokens) {
  const uint32_t per = 8u * c.heads * c.groups;
  const uint64_t total = tokens * per, stride = (uint64_t)gridDim.x * kBlockThreads;
  // whole quads of lanes share a group, and total is a multiple of 4
  for (uint64_t u = (uint64_t)blockIdx.x * kBlockThreads + threadIdx.x; u < total; u += stride) {
    const RowPart r(u, per, c);
    const uint64_t col = (uint64_t)r.head * c.dim() + 32u * r.group + 8u * r.part;
    const u32x4 x = *(const u32x4*)((r.values ? v + r.token * v_stride : k + r.token * k_stride) + col);
    const int64_t slot = slots[r.token];
    uint32_t m = max_abs8(x);
    const uint32_t a = (uint32_t)__shfl_xor((int)m, 1, kWave);
    m = m > a ? m : a;
    const uint32_t b = (uint32_t)__shfl_xor((int)m, 2, kWave);
    m = m > b ? m : b;
    if (!slot_in(c, slot)) continue;  // the same for the quad
    const uint32_t e = fp4_exponent(m), codes = fp4_pack8(x, e), t = (uint32_t)slot & 31u;
    uint8_t* const to = slot_tile(c, slot, r.head);
    if (r.values) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        to[value_place(c.groups, t, r.group, 4u * r.part + i)] = (uint8_t)(codes >> (8u * i));
      if (r.part == 0) to[value_scale_place(c.groups, t, r.group)] = (uint8_t)e;
    } else {
      *(uint32_t*)(to + key_place(c.groups, t, r.group, r.part)) = codes;
      if (r.part == 0) to[key_scale_place(c.groups, t, r.group)] = (uint8_t)e;
    }
  }
}

__global__ __launch_bounds__(kBlockThreads) void k_cache_read(Cache c, const int64_t* __restrict__ slots,
                                                              uint64_t tokens, uint16_t* __restrict__ k,
                                                              uint16_t* __restrict__ v) {
  const uint32_t per = 8u * c.heads * c.groups;
  const uint64_t total = tokens * per, stride = (uint64_t)gridDim.x * kBlockThreads;
  for (uint64_t u = (uint64_t)blockIdx.x * kBlockThreads + threadIdx.x; u < total; u += stride) {
    const RowPart r(u, per, c);
    const int64_t slot = slots[r.token];
    uint32_t codes = 0, e = 255u;  // NaN
    if (slot_in(c, slot)) {
      const uint32_t t = (uint32_t)slot & 31u;
      const uint8_t* const from = slot_tile(c, slot, r.head);
      if (r.values) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          codes |= (uint32_t)from[value_place(c.groups, t, r.group, 4u * r.part + i)] << (8u * i);
        e = from[value_scale_place(c.groups, t, r.group)];
      } else {
        codes = *(const uint32_t*)(from + key_place(c.groups, t, r.group, r.part));
        e = from[key_scale_place(c.groups, t, r.group)];
      }
    }
    const uint64_t at = (r.token * c.heads + r.head) * c.dim() + 32u * r.group + 8u * r.part;
    *(u32x4*)((r.values ? v : k) + at) = fp4_expand(codes, fp4_scale(e));
  }
}

// ---- attention ---------------------------------------------------------------
//
// A block takes up to 16 queries (columns) of one sequence that share a head of
// keys, and a chunk of the sequence's tiles; its waves take the tiles in turn and
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
// m is a value near the largest score so far, per query: it moves (and the sums are
// scaled) only when a score passes it by more than kSlack, so that a step needs no
// exchange between lanes.  Weights are then up to 2^kSlack, far inside fp32 and
// BF16.
constexpr uint32_t kAttnWaves = 4;
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
  float* part;  // [(seq, kv head, column tile)][split][columns][dim]
  float2* top;  // [..][split][columns]: m and the sum of weights
  uint32_t seqs, news, heads, group, width, window;
  uint32_t col_tiles, splits, chunk;  // chunk: tiles of a split
  float scale;                        // times log2(e)
};

// Which tiles of a sequence are read, and by how many splits.
struct Span {
  int32_t len;
  uint32_t first, end, splits;
  __device__ __forceinline__ Span(const CacheAttn& a, uint32_t seq) {
    const int32_t n = a.lengths[seq];
    len = n > 0 ? n : 0;
    const uint32_t cap = a.width * a.c.page_tiles;  // below 2^26 (attn_ok)
    end = ((uint32_t)len + 31u) / 32u;
    end = end < cap ? end : cap;
    const int64_t lo = a.window ? (int64_t)len - a.news - a.window + 1 : 0;
    first = lo > 0 ? (uint32_t)(lo / 32) : 0u;
    first = first < end ? first : end;
    splits = (end - first + a.chunk - 1u) / a.chunk;
    splits = splits ? splits : 1u;
  }
};

template <int G>
struct TileRegs {
  uint32_t k[2][G];
  uint32_t ks[(2 * G + 3) / 4];
  uint32_t v[G][2];
  uint32_t vs[G][2];

  __device__ __forceinline__ void load(const uint8_t* t) {
    const uint32_t lane = (uint32_t)lane_id(), r = lane & 15u, h = lane >> 4;
    each<2>([&](auto half) __attribute__((always_inline)) {
      each<(G + 3) / 4>([&](auto z) __attribute__((always_inline)) {
        constexpr int w = G - 4 * z < 4 ? G - 4 * z : 4;
        const uint8_t* p = t + (half * 64u * G + z * 256u + lane * w) * 4u;
        if constexpr (w == 4) {
          const u32x4 x = *(const u32x4*)p;
          each<4>([&](auto i) __attribute__((always_inline)) { k[half][4 * z + i] = x[+i]; });
        } else if constexpr (w == 2) {
          const uint2 x = *(const uint2*)p;
          k[half][4 * z] = x.x;
          k[half][4 * z + 1] = x.y;
        } else {
          each<w>([&](auto i) __attribute__((always_inline)) { k[half][4 * z + i] = ((const uint32_t*)p)[i]; });
        }
      });
    });
    const uint8_t* s = t + 1024u * G + r * 2u * G;
    if constexpr (G % 2 == 0) {
      each<G / 2>([&](auto i) __attribute__((always_inline)) { ks[i] = ((const uint32_t*)s)[i]; });
    } else {
      each<(2 * G + 3) / 4>([&](auto i) __attribute__((always_inline)) {
        const uint32_t hi = 2 * i + 1 < G ? ((const uint16_t*)s)[2 * i + 1 < G ? 2 * i + 1 : 0] : 0u;
        ks[i] = ((const uint16_t*)s)[2 * i] | hi << 16;
      });
    }
    each<(G + 1) / 2>([&](auto p) __attribute__((always_inline)) {
      const uint8_t* from = t + 512u * G + p * 1024u;
      if constexpr (2 * p + 1 < G) {
        const u32x4 x = *(const u32x4*)(from + lane * 16u);
        v[2 * p][0] = x[0];
        v[2 * p][1] = x[1];
        v[2 * p + 1][0] = x[2];
        v[2 * p + 1][1] = x[3];
      } else {
        const uint2 x = *(const uint2*)(from + lane * 8u);
        v[2 * p][0] = x.x;
        v[2 * p][1] = x.y;
      }
    });
    each<G>([&](auto g) __attribute__((always_inline)) {
      const uint2 x = *(const uint2*)(t + 1056u * G + h * 8u * G + g * 8u);
      vs[g][0] = x.x;
      vs[g][1] = x.y;
    });
  }

  // Values of the tokens that are not in `keep` (bytes 0xFF or 0) become 0.
  __device__ __forceinline__ void keep_values(const uint32_t keep[2]) {
    each<G>([&](auto g) __attribute__((always_inline)) {
      each<2>([&](auto i) __attribute__((always_inline)) {
        v[g][i] &= keep[i];
        vs[g][i] = (vs[g][i] & keep[i]) | (0x7F7F7F7Fu & ~keep[i]);
      });
    });
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

// Values of group g for the lane's 8 tokens: the even and the odd column of its pair.
template <int G>
__device__ __forceinline__ void value_operands(const TileRegs<G>& t, int g, u32x4& even, u32x4& odd) {
  uint32_t d[8];
  each<2>([&](auto i) __attribute__((always_inline)) {
    each<4>([&](auto b) __attribute__((always_inline)) {
      d[4 * i + b] = fp4_pair<b>(t.v[g][i], scale_of<b>(t.vs[g][i]));
    });
  });
  each<4>([&](auto j) __attribute__((always_inline)) {
    even[+j] = __builtin_amdgcn_perm(d[2 * j + 1], d[2 * j], 0x05040100u);
    odd[+j] = __builtin_amdgcn_perm(d[2 * j + 1], d[2 * j], 0x07060302u);
  });
}

template <int G, bool DUP>
__global__ __launch_bounds__(kWave* kAttnWaves) void k_cache_attention(CacheAttn a) {
  constexpr uint32_t D = 32u * G, kCols = DUP ? 8u : 16u;
  __shared__ mfma_f32x4 sums[kAttnWaves][G][2][kWave];
  __shared__ float2 tops[kAttnWaves][16];
  const uint32_t lane = (uint32_t)lane_id(), wave = (uint32_t)wave_in_block(), h = lane >> 4;
  uint32_t b = blockIdx.x;
  const uint32_t kv = b % a.c.heads;
  b /= a.c.heads;
  const uint32_t ct = b % a.col_tiles;
  b /= a.col_tiles;
  const uint32_t split = b % a.splits, seq = b / a.splits;
  const Span sp(a, seq);
  if (split >= sp.splits) return;
  const uint32_t tile0 = sp.first + split * a.chunk;
  const uint32_t tile1 = tile0 + a.chunk < sp.end ? tile0 + a.chunk : sp.end;

  // the lane's query; columns past the last repeat it
  const uint32_t cols = a.news * a.group;
  uint32_t col = ct * kCols + (lane & (kCols - 1u));
  const bool real = col < cols;
  col = real ? col : cols - 1u;
  const uint32_t qi = col / a.group, head = kv * a.group + col - qi * a.group;
  const int32_t hi = sp.len - (int32_t)a.news + (int32_t)qi;  // its position
  const int64_t lo = a.window ? (int64_t)hi - a.window + 1 : 0;
  u32x4 q[G];
  {
    const uint16_t* from = a.q + ((uint64_t)seq * a.news + qi) * a.q_stride + (uint64_t)head * D + 8u * h;
    each<G>([&](auto g) __attribute__((always_inline)) { q[g] = *(const u32x4*)(from + 32 * g); });
  }
  // positions that every query attends to, and that some query does
  const int64_t all0 = a.window ? (int64_t)sp.len - a.window : 0, all1 = (int64_t)sp.len - a.news;
  const int64_t any0 = a.window ? (int64_t)sp.len - a.news - a.window + 1 : 0;

  float m = -INFINITY, off = 0, sum = 0;  // off: m, or 0 while there is none
  mfma_f32x4 acc[G][2];
  each<G>([&](auto g) __attribute__((always_inline)) { acc[g][0] = acc[g][1] = mfma_f32x4{0, 0, 0, 0}; });

  uint32_t pages = 0;  // of the wave's next 64 tiles, one per lane
  bool bad = false, bad_next = false;
  auto fetch = [&](uint32_t i, TileRegs<G>& t) __attribute__((always_inline)) {  // the wave's i-th tile
    if (i % kWave == 0) {
      const uint32_t mine = tile0 + wave + (i + lane) * kAttnWaves;
      pages = mine < tile1 ? (uint32_t)a.table[(uint64_t)seq * a.width + mine / a.c.page_tiles] : 0u;
    }
    const uint32_t tile = tile0 + wave + i * kAttnWaves;
    uint32_t page = (uint32_t)__builtin_amdgcn_readlane((int)pages, (int)(i % kWave));
    bad_next = page >= a.c.pages;
    page = bad_next ? 0u : page;
    t.load(a.c.at(page, kv, tile % a.c.page_tiles));
  };

  auto step = [&](uint32_t tile, TileRegs<G>& t) __attribute__((always_inline)) {
    const int64_t p0 = (int64_t)tile * 32;
    const bool edge = bad || p0 < all0 || p0 + 31 > all1;  // wave-uniform
    float s[8];
    each<2>([&](auto half) __attribute__((always_inline)) {
      mfma_f32x4 x = {0, 0, 0, 0};
      each<G>([&](auto g) __attribute__((always_inline)) {
        constexpr int at = half * G + g;
        x = mfma16(fp4_expand(t.k[half][g], scale_of<at % 4>(t.ks[at / 4])), q[g], x);
      });
      each<4>([&](auto i) __attribute__((always_inline)) { s[4 * half + i] = x[+i] * a.scale; });
    });
    if (edge) {
      uint32_t keep[2] = {0, 0};
      each<8>([&](auto i) __attribute__((always_inline)) {
        const int64_t p = p0 + 8u * h + i;
        s[i] = bad ? NAN : s[i];
        s[i] = p <= hi && p >= lo ? s[i] : -INFINITY;
        keep[i / 4] |= !bad && p < sp.len && p >= any0 ? 0xFFu << (8 * (i % 4)) : 0u;
      });
      t.keep_values(keep);
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
    each<8>([&](auto i) __attribute__((always_inline)) {
      s[i] = __builtin_amdgcn_exp2f(s[i] - off);
      sum += s[i];
    });
    u32x4 high, low;
    each<4>([&](auto j) __attribute__((always_inline)) {
      const uint32_t x = bf16_pair(s[2 * j], s[2 * j + 1]);
      high[+j] = x;
      low[+j] = bf16_pair(s[2 * j] - __uint_as_float(x << 16), s[2 * j + 1] - __uint_as_float(x & 0xFFFF0000u));
    });
    if constexpr (DUP) high = lane & 8u ? low : high;
    auto product = [&](const TileRegs<G>& from, bool take) __attribute__((always_inline)) {
      each<G>([&](auto g) __attribute__((always_inline)) {
        u32x4 even, odd;
        value_operands<G>(from, g, even, odd);
        mfma_f32x4 x = mfma16(even, high, acc[g][0]), y = mfma16(odd, high, acc[g][1]);
        if constexpr (!DUP) {
          x = mfma16(even, low, x);
          y = mfma16(odd, low, y);
        }
        each<4>([&](auto i) __attribute__((always_inline)) {
          acc[g][0][+i] = take ? x[+i] : acc[g][0][+i];
          acc[g][1][+i] = take ? y[+i] : acc[g][1][+i];
        });
      });
    };
    if (edge && a.news > 1) {
      // a value that is not finite must not reach the queries that do not attend to it
      bool odd_one = false;
      each<G>([&](auto g) __attribute__((always_inline)) {
        each<2>([&](auto i) __attribute__((always_inline)) {
          each<4>([&](auto b) __attribute__((always_inline)) {
            odd_one = odd_one || (t.vs[g][i] >> (8 * b) & 0xFFu) >= 253u;
          });
        });
      });
      if (__ballot(odd_one)) {
        for (uint32_t j = 0; j < a.news; ++j) {  // each query by itself
          const int64_t at = (int64_t)sp.len - a.news + j, from = a.window ? at - a.window + 1 : 0;
          uint32_t keep[2] = {0, 0};
          each<8>([&](auto i) __attribute__((always_inline)) {
            const int64_t p = p0 + 8u * h + i;
            keep[i / 4] |= p <= at && p >= from ? 0xFFu << (8 * (i % 4)) : 0u;
          });
          TileRegs<G> mine = t;
          mine.keep_values(keep);
          product(mine, qi == j);
        }
        return;
      }
    }
    product(t, true);
  };

  const uint32_t mine = tile0 + wave < tile1 ? (tile1 - tile0 - wave + kAttnWaves - 1u) / kAttnWaves : 0u;
  if (mine) {
    TileRegs<G> now;
    fetch(0, now);
    for (uint32_t i = 0; i + 1u < mine; ++i) {
      TileRegs<G> next;
      bad = bad_next;
      fetch(i + 1u, next);
      step(tile0 + wave + i * kAttnWaves, now);
      now = next;
    }
    bad = bad_next;
    step(tile0 + wave + (mine - 1u) * kAttnWaves, now);
  }
  // a query at a position past the table attends to itself, which is not there
  if (hi >= 0 && (uint64_t)hi >= (uint64_t)a.width * a.c.page_tiles * 32u) sum = NAN;

  sum += __shfl_xor(sum, 16, kWave);
  sum += __shfl_xor(sum, 32, kWave);
  each<G>([&](auto g) __attribute__((always_inline)) {
    // the lane's columns of the group in order: 8 h .. 8 h + 7
    sums[wave][g][0][lane] = mfma_f32x4{acc[g][0][0], acc[g][1][0], acc[g][0][1], acc[g][1][1]};
    sums[wave][g][1][lane] = mfma_f32x4{acc[g][0][2], acc[g][1][2], acc[g][0][3], acc[g][1][3]};
  });
  if (lane < 16u) tops[wave][lane] = make_float2(m, sum);
  __syncthreads();
  float most = -INFINITY, total = 0, w[kAttnWaves];
  each<kAttnWaves>([&](auto i) __attribute__((always_inline)) { most = fmaxf(most, tops[i][lane & 15u].x); });
  each<kAttnWaves>([&](auto i) __attribute__((always_inline)) {
    const float2 t = tops[i][lane & 15u];
    w[i] = t.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(t.x - most);
    // a NaN sum counts although its wave has no largest score
    total += t.x == -INFINITY ? (t.y != t.y ? t.y : 0.0f) : w[i] * t.y;
  });
  const bool whole = sp.splits == 1u;
  const float by = total == 0.0f ? 0.0f : 1.0f / total;
  const bool stores = real && (!DUP || !(lane & 8u));
  const uint64_t row = ((uint64_t)seq * a.news + qi) * a.heads + head;
  const uint64_t at = ((((uint64_t)seq * a.c.heads + kv) * a.col_tiles + ct) * a.splits + split) * kCols +
                      (lane & (kCols - 1u));
  for (uint32_t g = wave; g < (uint32_t)G; g += kAttnWaves) {
    mfma_f32x4 x[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    each<kAttnWaves>([&](auto i) __attribute__((always_inline)) {
      each<2>([&](auto p) __attribute__((always_inline)) {
        mfma_f32x4 y = sums[i][g][p][lane];
        if constexpr (DUP) y += sums[i][g][p][lane ^ 8u];
        x[p] += w[i] * y;
      });
    });
    if (!stores) continue;
    if (whole) {
      u32x4 o;
      each<4>([&](auto j) __attribute__((always_inline)) {
        o[+j] = bf16_pair(x[j / 2][2 * (j % 2)] * by, x[j / 2][2 * (j % 2) + 1] * by);
      });
      *(u32x4*)(a.out + row * D + 32u * g + 8u * h) = o;
    } else {
      mfma_f32x4* to = (mfma_f32x4*)(a.part + at * D + 32u * g + 8u * h);
      to[0] = x[0];
      to[1] = x[1];
    }
  }
  if (wave == 0 && h == 0 && stores) {
    if (!whole)
      a.top[at] = make_float2(most, total);
    else if (a.lse)
      a.lse[row] = total == 0.0f ? -INFINITY : (most == -INFINITY ? total : (most + __builtin_amdgcn_logf(total)) * kLn2);
  }
}

// The splits of each query, joined: a wave takes one, a lane D / 64 columns or fewer.
template <int G>
__global__ __launch_bounds__(kBlockThreads) void k_cache_join(CacheAttn a, uint32_t cols_of_tile) {
  constexpr uint32_t D = 32u * G;
  const uint32_t lane = (uint32_t)lane_id();
  const uint64_t row = (uint64_t)blockIdx.x * (kBlockThreads / kWave) + (uint32_t)wave_in_block();
  if (row >= (uint64_t)a.seqs * a.news * a.heads) return;
  const uint32_t head = (uint32_t)(row % a.heads);
  const uint64_t token = row / a.heads;
  const uint32_t seq = (uint32_t)(token / a.news), qi = (uint32_t)(token - (uint64_t)seq * a.news);
  const Span sp(a, seq);
  if (sp.splits == 1u) return;
  const uint32_t kv = head / a.group, col = qi * a.group + head - kv * a.group;
  const uint32_t ct = col / cols_of_tile;
  const uint64_t at = (((uint64_t)seq * a.c.heads + kv) * a.col_tiles + ct) * a.splits * cols_of_tile +
                      (col - ct * cols_of_tile);
  float most = -INFINITY, total = 0;
  for (uint32_t s = lane; s < sp.splits; s += kWave) most = fmaxf(most, a.top[at + (uint64_t)s * cols_of_tile].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, kWave));
  float x[(D + 63) / 64] = {};
  for (uint32_t s = 0; s < sp.splits; ++s) {
    const float2 t = a.top[at + (uint64_t)s * cols_of_tile];
    const float w = t.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(t.x - most);
    total += t.x == -INFINITY ? (t.y != t.y ? t.y : 0.0f) : w * t.y;
    const float* from = a.part + (at + (uint64_t)s * cols_of_tile) * D;
#pragma unroll
    for (uint32_t i = 0; i < (D + 63) / 64; ++i)
      if (64u * i + lane < D) x[i] += w * from[64u * i + lane];
  }
  const float by = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
  for (uint32_t i = 0; i < (D + 63) / 64; ++i)
    if (64u * i + lane < D) a.out[row * D + 64u * i + lane] = bf16_of(x[i] * by);
  if (lane == 0 && a.lse)
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

uint32_t part_blocks(uint64_t units) {
  const uint64_t b = (units + kBlockThreads - 1) / kBlockThreads, most = (uint64_t)cu_count() * 16u;
  return (uint32_t)(b < most ? b : most);
}

// How a call is cut: columns of a tile, tiles of columns, tiles of a split.
struct Cut {
  uint32_t cols, col_tiles, chunk, splits;
  uint64_t blocks() const { return (uint64_t)col_tiles * splits; }  // per sequence and head of keys
};
int attn_cut(const wc_fp4_cache* c, const wc_fp4_attention_shape* s, Cut* cut) {
  if (!s || s->new_tokens < 1u || s->new_tokens > WC_ATTN_MAX_NEW) return WC_E_UNSUPPORTED;
  if (s->heads < 1u || s->heads > WC_ATTN_MAX_HEADS || s->heads % c->kv_heads) return WC_E_ARG;
  const uint64_t cap = (uint64_t)s->table_width * (c->page_size / 32u);
  if (cap >= (1ull << 26)) return WC_E_SIZE;  // positions below 2^31
  const uint32_t cols = s->new_tokens * (s->heads / c->kv_heads);
  cut->cols = cols <= 8u ? 8u : 16u;
  cut->col_tiles = (cols + cut->cols - 1u) / cut->cols;
  uint64_t tiles = cap;
  if (s->window) {
    const uint64_t most = ((uint64_t)s->window + s->new_tokens - 1u + 30u) / 32u + 1u;
    tiles = most < cap ? most : cap;
  }
  const uint64_t rows = (uint64_t)s->seqs * c->kv_heads * cut->col_tiles;
  uint64_t chunk = (tiles * rows + 4u * cu_count() - 1u) / (4u * cu_count());
  chunk = chunk < 4u ? 4u : (chunk > 64u ? 64u : (chunk + 3u) & ~3ull);
  cut->chunk = (uint32_t)chunk;
  cut->splits = (uint32_t)((tiles + chunk - 1u) / chunk);
  if (!cut->splits) cut->splits = 1u;
  if (rows * cut->splits >= (1ull << 24)) return WC_E_SIZE;  // a grid of fewer than 2^32 threads
  return WC_OK;
}
uint64_t attn_partials(const wc_fp4_cache* c, const wc_fp4_attention_shape* s, const Cut& cut) {
  return cut.splits == 1u ? 0u : (uint64_t)s->seqs * c->kv_heads * cut.blocks() * cut.cols;
}

template <int G>
void launch_attention(const CacheAttn& a, const Cut& cut, hipStream_t s) {
  const uint32_t blocks = a.seqs * a.c.heads * cut.col_tiles * cut.splits;
  if (cut.cols == 8u)
    k_cache_attention<G, true><<<blocks, kWave * kAttnWaves, 0, s>>>(a);
  else
    k_cache_attention<G, false><<<blocks, kWave * kAttnWaves, 0, s>>>(a);
  if (cut.splits > 1u) {
    const uint32_t rows = a.seqs * a.news * a.heads;
    k_cache_join<G><<<(rows + 3u) / 4u, kBlockThreads, 0, s>>>(a, cut.cols);
  }
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
  wc::k_cache_append<<<wc::part_blocks(tokens * row / 4u), wc::kBlockThreads, 0, (hipStream_t)stream>>>(
      wc::cache_of(cache), d_k, k_stride, d_v, v_stride, d_slots, tokens);
  return wc::launched();
}

extern "C" int wc_fp4_cache_read(const wc_fp4_cache* cache, const int64_t* d_slots, uint64_t tokens,
                                 uint16_t* d_k, uint16_t* d_v, void* stream) {
  if (const int v = wc::cache_ok(cache)) return v;
  if (tokens >= (1ull << 31)) return WC_E_SIZE;
  if (tokens == 0) return WC_OK;
  if (!d_k || !wc::aligned16(d_k) || !d_v || !wc::aligned16(d_v) || !d_slots || ((uintptr_t)d_slots & 7u))
    return WC_E_ARG;
  const uint64_t row = (uint64_t)cache->kv_heads * cache->head_dim;
  wc::k_cache_read<<<wc::part_blocks(tokens * row / 4u), wc::kBlockThreads, 0, (hipStream_t)stream>>>(
      wc::cache_of(cache), d_slots, tokens, d_k, d_v);
  return wc::launched();
}

extern "C" size_t wc_fp4_attention_workspace_bytes(const wc_fp4_cache* cache,
                                                   const wc_fp4_attention_shape* shape) {
  wc::Cut cut;
  if (wc::cache_ok(cache) || wc::attn_cut(cache, shape, &cut)) return 0;
  const uint64_t n = wc::attn_partials(cache, shape, cut);
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
  const uint64_t n = wc::attn_partials(cache, shape, cut);
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
  a.window = shape->window;
  a.col_tiles = cut.col_tiles;
  a.splits = cut.splits;
  a.chunk = cut.chunk;
  a.scale = shape->scale * wc::kLog2e;
  const hipStream_t s = (hipStream_t)stream;
  switch (a.c.groups) {
    case 1: wc::launch_attention<1>(a, cut, s); break;
    case 2: wc::launch_attention<2>(a, cut, s); break;
    case 3: wc::launch_attention<3>(a, cut, s); break;
    case 4: wc::launch_attention<4>(a, cut, s); break;
    case 5: wc::launch_attention<5>(a, cut, s); break;
    case 6: wc::launch_attention<6>(a, cut, s); break;
    case 7: wc::launch_attention<7>(a, cut, s); break;
    default: wc::launch_attention<8>(a, cut, s); break;
  }
  return wc::launched();
}
