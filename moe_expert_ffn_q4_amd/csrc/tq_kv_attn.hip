// tq_kv_attn.hip -- softmax attention over the paged 4-bit key/value cache.
//
// The products run on the fp16 matrix cores with exact operands. A nibble n becomes the fp16
// integer n - 8 in two instructions per pair (its bits under the exponent of 1024, less 1032). A
// key tile of 16 tokens times one block of 32 dimensions is one 16x16x32 product per block, with
// the queries (each row times a power of two, split into fp16 hi + lo for fp32 queries) as the
// other operand; a block's product is multiplied by the block's fp16 scale in fp32. The result
// holds, in lane l, column l % 16 (a query row) and the tokens 4 (l / 16) + 0..3, which is the
// layout of the A operand of the second product: weights stay in the lane that formed them, are
// multiplied by the values' scale of each block and rounded to fp16 (hi + lo as two rows of the
// operand for fp32 and fp16 activations).
#include "tq_kv.h"
#include "tq_kv_device.h"
#include "tq_launch.h"

namespace tq {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x3a4 __attribute__((ext_vector_type(3), aligned(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kGrid = 512;       // workgroups of a full launch: two per compute unit
constexpr int kMinSteps = 4;     // key steps (32 tokens) per workgroup at least: one per wave
constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kSlack = 7.f;    // see step()

// ---- the step's work as one line of units -----------------------------------------------------
// An item is a query tile (up to NCOL columns: tokens x heads of one kv head) of a request; the
// units of an item are the 32-token steps of its request. All items' units form one line, cut
// into equal shares, one a workgroup, so ragged batches load the chip evenly. The lengths live on
// the device, so every workgroup forms the prefix sums over the requests itself.
struct Request {
  int r, row0, fresh, len, first_pos;  // rows row0 .. row0 + fresh, tokens of the sequence
  int tiles, steps;                    // query tiles, units per item
};

struct TileShape {
  int tokens, splits;  // tokens of a query tile; or, for groups wider than a tile, tiles per token
};

template <int NCOL>
__device__ __forceinline__ TileShape tile_shape(int group) {
  TileShape t;
  t.tokens = group <= NCOL ? NCOL / group : 1;
  t.splits = group <= NCOL ? 1 : (group + NCOL - 1) / NCOL;
  return t;
}

__device__ __forceinline__ int seen_from(const AttnArgs &a, int pos) {
  return a.window ? max(0, pos - a.window + 1) : 0;
}

__device__ __forceinline__ Request request(const AttnArgs &a, const TileShape &ts, int r) {
  Request q;
  q.r = r;
  q.row0 = min(max(a.cu_new[r], 0), a.rows);
  q.fresh = max(min(a.cu_new[r + 1], a.rows) - q.row0, 0);
  q.len = (int)min((int64_t)max(a.seq_len[r], 0), (int64_t)a.max_blocks << a.g.page_shift);
  q.first_pos = q.len - q.fresh;
  q.tiles = (q.fresh + ts.tokens - 1) / ts.tokens * ts.splits;
  q.steps = max(1, (q.len + 31) / 32 - seen_from(a, q.first_pos) / 32);
  return q;
}

__device__ __forceinline__ int64_t units_of(const AttnArgs &a, const Request &q) {
  return (int64_t)a.g.heads * q.tiles * q.steps;
}

struct Place {
  int64_t total, per;  // units of all requests, units per workgroup
  int r;               // the request that holds the wanted unit
  int64_t base;        // its first unit
};

// Called by every thread of the workgroup. `unit_of(per)`: the wanted unit.
template <typename F>
__device__ __forceinline__ Place locate(const AttnArgs &a, const TileShape &ts, F unit_of) {
  __shared__ int64_t sums[kWaves];
  __shared__ int64_t found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int n = (a.requests + kThreads - 1) / kThreads;
  const int r0 = min(a.requests, tid * n), r1 = min(a.requests, r0 + n);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += units_of(a, request(a, ts, r));
  int64_t incl = mine;
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 63) sums[wave] = incl;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  Place p;
  p.total = 0;
  int64_t base = incl - mine;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) base += sums[w];
    p.total += sums[w];
  }
  p.per = max((int64_t)kMinSteps, (p.total + a.grid - 1) / a.grid);
  const int64_t u = unit_of(p.per);
  if (u >= base && u < base + mine) {
    for (int r = r0; r < r1; ++r) {
      const int64_t m = units_of(a, request(a, ts, r));
      if (u < base + m) {
        found[0] = r;
        found[1] = base;
        break;
      }
      base += m;
    }
  }
  __syncthreads();
  p.r = (int)found[0];
  p.base = found[1];
  return p;
}

// ---- operands ---------------------------------------------------------------------------------

// Four tokens (or dimensions) pairs of one dword of quants as fp16 integers n - 8:
// low nibbles of bytes (0, 2), of bytes (1, 3), high nibbles of both pairs.
__device__ __forceinline__ void unpack(uint32_t w, f16x2 out[4]) {
  const uint32_t u = w >> 8;
  const f16x2 low = {(_Float16)-1032.f, (_Float16)-1032.f};
  const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  const f16x2 high = {(_Float16)-72.f, (_Float16)-72.f};
  out[0] = __builtin_bit_cast(f16x2, (w & 0x000F000Fu) | 0x64006400u) + low;
  out[1] = __builtin_bit_cast(f16x2, (u & 0x000F000Fu) | 0x64006400u) + low;
  out[2] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (w & 0x00F000F0u) | 0x64006400u), sixteenth, high);
  out[3] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (u & 0x00F000F0u) | 0x64006400u), sixteenth, high);
}

__device__ __forceinline__ f16x8 join(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The lane's share of one 16-token tile.
template <int NB>
struct TileRegs {
  uint32_t k[NB], v[NB];          // quants: one dword per block
  uint32_t ks[2 * NB], vs[2 * NB];  // fp16 scales [block][4 tokens]
};

template <int NB>
__device__ __forceinline__ void load_quants(const uint8_t *p, int lane, uint32_t *out) {
  typedef __attribute__((address_space(1))) const u32x2a4 *g2;
  typedef __attribute__((address_space(1))) const u32x3a4 *g3;
  if constexpr (NB == 2) {
    const u32x2a4 w = *(g2)(p + lane * 8);
    out[0] = w[0];
    out[1] = w[1];
  } else if constexpr (NB == 3) {
    const u32x3a4 w = *(g3)(p + lane * 12);
    for (int i = 0; i < 3; ++i) out[i] = w[i];
  } else {
#pragma unroll
    for (int c = 0; c < NB / 4; ++c) {
      const u32x4 w = gload(p + c * 1024 + lane * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[4 * c + i] = w[i];
    }
  }
}

template <int NB>
__device__ __forceinline__ void load_scales(const uint8_t *p, int g, uint32_t *out) {
  typedef __attribute__((address_space(1))) const u32x2 *g2;
  p += g * 8 * NB;
  if constexpr (NB % 2 == 0) {
#pragma unroll
    for (int c = 0; c < NB / 2; ++c) {
      const u32x4 w = gload(p + 16 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[4 * c + i] = w[i];
    }
  } else {
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      const u32x2 w = *(g2)(p + 8 * c);
      out[2 * c] = w[0];
      out[2 * c + 1] = w[1];
    }
  }
}

template <int NB>
__device__ __forceinline__ void load_tile(const uint8_t *p, int lane, TileRegs<NB> &t) {
  constexpr int kQuant = 256 * NB, kHalf = 288 * NB;
  load_quants<NB>(p, lane, t.k);
  load_scales<NB>(p + kQuant, lane >> 4, t.ks);
  load_quants<NB>(p + kHalf, lane, t.v);
  load_scales<NB>(p + kHalf + kQuant, lane >> 4, t.vs);
}

// The scale of token 4 g + r of block b as fp32 (folds into mixed-precision FMAs).
__device__ __forceinline__ float scale_of(const uint32_t *s, int b, int r) {
  const f16x2 h = __builtin_bit_cast(f16x2, s[2 * b + (r >> 1)]);
  return (float)h[r & 1];
}

__device__ __forceinline__ float row_swap8(float v) {  // lane l's value from lane l ^ 8 of its row of 16
  const int i = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, 0x128, 0xF, 0xF, false));
}

// Query columns of an item: column c is token tok0 + c / group of the request, head
// head0 + c % group; or one token and heads head0 + c for groups wider than the tile.
struct Columns {
  int tok0, head0, count;
  int per;  // heads per token in the tile
};

template <int NCOL>
__device__ __forceinline__ Columns columns(const AttnArgs &a, const TileShape &ts, const Request &q,
                                           int kvh, int tile) {
  Columns c;
  if (ts.splits == 1) {
    c.tok0 = tile * ts.tokens;
    c.head0 = kvh * a.group;
    c.per = a.group;
    c.count = min(ts.tokens, q.fresh - c.tok0) * a.group;
  } else {
    const int part = tile % ts.splits;
    c.tok0 = tile / ts.splits;
    c.head0 = kvh * a.group + part * NCOL;
    c.per = NCOL;
    c.count = min(NCOL, a.group - part * NCOL);
  }
  return c;
}

// ---- the kernel ---------------------------------------------------------------------------------

template <typename A, int NB, bool SPLIT>
struct Attn {
  typedef typename A::type T;
  static constexpr int NCOL = SPLIT ? 8 : 16;  // query columns of a tile
  static constexpr int D = 32 * NB;
  static constexpr int kPart = NCOL * (D + 2);  // floats of a partial result: m, l, O
  static constexpr int kMergeBlocks = NB < 4 ? NB : 4;  // blocks merged over the waves at a time

  struct State {
    f32x4 o[2 * NB];  // rows 4 g + r (query columns), columns l % 16: dimension 32 b + 16 half + l % 16
    float m, l;       // of column l % 16: reference exponent (shared by the lane groups), this lane's sum
  };

  // One step of 32 tokens. Reference exponent: weights are p = 2^(s - m) with m such that p times
  // the value's scale stays below 2^15, the fp16 range, whatever the scales are; m only moves when
  // a lane would pass that (kSlack binades of slack over the 2^8 it is set to), so the exchange
  // between lane groups and the rescaling of O are rare. `l` sums p in the same reference.
  template <bool MASK>
  static __device__ __forceinline__ void step(const TileRegs<NB> (&t)[2], const f16x8 (&qf)[NB],
                                              float qs, int lo, int hi, int any_lo, int any_hi,
                                              int t0, int lane, State &st) {
    const int g = lane >> 4;
    float s[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f16x2 n[4];
        unpack(t[i].k[b], n);
        const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(n[0], n[1], n[2], n[3]), qf[b],
                                                               f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(scale_of(t[i].ks, b, r), d[r], acc[r]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[r];
        if constexpr (SPLIT) v += row_swap8(v);  // hi and lo columns of one query
        if constexpr (MASK) {
          const int tok = t0 + 16 * i + 4 * g + r;
          v = tok >= lo && tok < hi ? v : -INFINITY;
        }
        s[4 * i + r] = v;
      }
    }
    // largest |scale| of the lane's tokens, as fp16 bits (their order is the magnitudes')
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) {
        uint32_t w = t[i].vs[j] & 0x7FFF7FFFu;
        if constexpr (MASK) {  // scales of tokens that no column sees may be anything
          const int tok = t0 + 16 * i + 4 * g + 2 * (j & 1);
          if (tok < any_lo || tok >= any_hi) w &= 0xFFFF0000u;
          if (tok + 1 < any_lo || tok + 1 >= any_hi) w &= 0x0000FFFFu;
        }
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, w));
      }
    const int expo = (int)(most[0] > most[1] ? most[0] : most[1]) >> 10;  // scale < 2^(expo - 14)
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
    float want = fmaf(mx, qs, (float)(expo - 22));
    if (__any(want > st.m + kSlack)) {
      want = fmaxf(want, __shfl_xor(want, 16));
      want = fmaxf(want, __shfl_xor(want, 32));
      const float m = fmaxf(st.m, want);
      const float alpha = __builtin_amdgcn_exp2f(st.m - m);
      st.m = m;
      st.l *= alpha;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float f = __shfl(alpha, 4 * g + r);
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) st.o[j][r] *= f;
      }
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(fmaf(s[i], qs, -st.m));
      st.l += p[i];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f16x8 w;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = scale_of(t[i >> 2].vs, b, i & 3);
        float x = fmaf(p[i], d, 0.f);
        if constexpr (MASK) x = s[i] == -INFINITY ? 0.f : x;  // 0 times a scale that is not a number
        const _Float16 h = (_Float16)x;
        if constexpr (SPLIT) w[i] = lane & 8 ? (_Float16)(x - (float)h) : h;
        else w[i] = h;
      }
      f16x2 n0[4], n1[4];
      unpack(t[0].v[b], n0);
      unpack(t[1].v[b], n1);
      st.o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, join(n0[0], n0[1], n1[0], n1[1]), st.o[2 * b], 0, 0, 0);
      st.o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, join(n0[2], n0[3], n1[2], n1[3]), st.o[2 * b + 1], 0, 0, 0);
    }
  }

  static __device__ __forceinline__ void store_out(const AttnArgs &a, const Request &q, const Columns &c,
                                                   int col, int d, float v) {
    const int tok = col / c.per, head = c.head0 + col - tok * c.per;
    T *out = (T *)a.out.data + (int64_t)(q.row0 + c.tok0 + tok) * a.out.row_stride + (int64_t)head * a.out.head_stride;
    out[d] = A::from(v);
  }
  static __device__ __forceinline__ void store_lse(const AttnArgs &a, const Request &q, const Columns &c,
                                                   int col, float m, float l) {
    if (!a.lse) return;
    const int tok = col / c.per, head = c.head0 + col - tok * c.per;
    a.lse[(int64_t)(q.row0 + c.tok0 + tok) * (a.group * a.g.heads) + head] =
        l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
  }

  // The units [v0, v1) of an item's `steps`, by the whole workgroup.
  static __device__ void segment(const AttnArgs &a, const TileShape &ts, const Request &q, int kvh,
                                 int tile, int v0, int v1, float *part, float *lds) {
    const int lane = threadIdx.x & 63, wave = wave_index(), g = lane >> 4;
    const Columns cs = columns<NCOL>(a, ts, q, kvh, tile);
    // tokens that the tile's columns see: all together, and this lane's column
    const int last_tok = cs.tok0 + (cs.count - 1) / cs.per;
    const int any_lo = seen_from(a, q.first_pos + cs.tok0);
    const int any_hi = max(q.first_pos + last_tok + 1, 0);
    const int all_lo = seen_from(a, q.first_pos + last_tok), all_hi = max(q.first_pos + cs.tok0 + 1, 0);
    const int col = min(SPLIT ? lane & 7 : lane & 15, cs.count - 1);
    const int tok = cs.tok0 + col / cs.per, head = cs.head0 + col % cs.per;
    const int pos = q.first_pos + tok, lo = seen_from(a, pos), hi = max(pos + 1, 0);
    // the query: dimensions 32 b + 4 g + 0..3 and 16 more, times a power of two
    const T *qp = (const T *)a.q.data + (int64_t)(q.row0 + tok) * a.q.row_stride + (int64_t)head * a.q.head_stride;
    f16x8 qf[NB];
    float qs;
    {
      float v[8 * NB], most = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[8 * b + i] = A::load(qp + 32 * b + 4 * g + (i & 3) + 16 * (i >> 2));
          most = fmaxf(most, fabsf(v[8 * b + i]));
        }
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
      const int e = most > 0.f && most < INFINITY ? min(15 - __builtin_amdgcn_frexp_expf(most), 100) : 0;
      qs = ldexpf(a.scale, -e);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = ldexpf(v[8 * b + i], e);
          const _Float16 h = (_Float16)x;
          if constexpr (SPLIT) qf[b][i] = lane & 8 ? (_Float16)(x - (float)h) : h;
          else qf[b][i] = h;
        }
    }
    State st;
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) st.o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    st.m = kLowest;
    st.l = 0.f;
    // the tile's own steps: the item's units are spread over them (a tile of early tokens has fewer)
    const int s0 = any_lo / 32, n = max(0, (any_hi + 31) / 32 - s0);
    const int from = s0 + (int)((int64_t)v0 * n / q.steps), to = s0 + (int)((int64_t)v1 * n / q.steps);
    const int32_t *table = a.block_table + (int64_t)q.r * a.max_blocks;
    const int last_block = ((q.len + a.g.page_tokens - 1) >> a.g.page_shift) - 1;
    const uint8_t *head_data = a.g.data + (int64_t)kvh * a.g.head_bytes;
    // A tile's address; a page outside the cache reads page 0 (its tokens are masked below).
    auto page_of = [&](int t) { return table[min(t >> a.g.page_shift, last_block)]; };
    auto tile_at = [&](int t, int page) {
      const int64_t ok = page >= 0 && page < a.g.pages ? page : 0;
      return head_data + ok * a.g.page_bytes + (int64_t)((t & (a.g.page_tokens - 1)) >> 4) * a.g.tile_bytes;
    };
    TileRegs<NB> cur[2], next[2];
    int s = from + wave;
    int page0 = 0, page1 = 0;
    if (s < to) {
      page0 = page_of(32 * s);
      page1 = page_of(32 * s + 16);
      load_tile<NB>(tile_at(32 * s, page0), lane, cur[0]);
      load_tile<NB>(tile_at(32 * s + 16, page1), lane, cur[1]);
    }
    while (s < to) {
      const int s1 = s + kWaves;
      int np0 = 0, np1 = 0;
      if (s1 < to) {
        np0 = page_of(32 * s1);
        np1 = page_of(32 * s1 + 16);
        load_tile<NB>(tile_at(32 * s1, np0), lane, next[0]);
        load_tile<NB>(tile_at(32 * s1 + 16, np1), lane, next[1]);
      }
      const int t0 = 32 * s;
      const bool bad0 = page0 < 0 || page0 >= a.g.pages, bad1 = page1 < 0 || page1 >= a.g.pages;
      if (t0 >= all_lo && t0 + 32 <= all_hi && !bad0 && !bad1) {
        step<false>(cur, qf, qs, lo, hi, any_lo, any_hi, t0, lane, st);
      } else {
        const int l0 = bad0 ? t0 + 16 : 0, h0 = bad1 ? t0 + 16 : 0x7FFFFFFF;
        step<true>(cur, qf, qs, max(lo, l0), min(hi, h0), max(any_lo, l0), min(any_hi, h0), t0, lane, st);
      }
      cur[0] = next[0];
      cur[1] = next[1];
      page0 = np0;
      page1 = np1;
      s = s1;
    }
    // join the waves: sums over the lane groups, then O in runs of up to 128 dimensions
    st.l += __shfl_xor(st.l, 16);
    st.l += __shfl_xor(st.l, 32);
    float *lm = lds, *ll = lds + kWaves * NCOL, *lo_ = lds + 2 * kWaves * NCOL;
    __syncthreads();
    if (lane < NCOL) {
      lm[wave * NCOL + lane] = st.m;
      ll[wave * NCOL + lane] = st.l;
    }
    constexpr int kRun = 32 * kMergeBlocks;
#pragma unroll
    for (int b0 = 0; b0 < NB; b0 += kMergeBlocks) {
      if (b0) __syncthreads();
#pragma unroll
      for (int j = 0; j < 2 * kMergeBlocks; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v = st.o[2 * b0 + j][r];
          if constexpr (SPLIT) v += __shfl_xor(v, 32);
          const int row = 4 * g + r;
          if (row < NCOL) lo_[(wave * NCOL + row) * kRun + 16 * j + (lane & 15)] = v;
        }
      __syncthreads();
      for (int i = threadIdx.x; i < NCOL * kRun; i += kThreads) {
        const int c = i / kRun, d = i - c * kRun;
        if (c >= cs.count) continue;
        float m = lm[c], l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, lm[w * NCOL + c]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(lm[w * NCOL + c] - m);
          l = fmaf(f, ll[w * NCOL + c], l);
          o = fmaf(f, lo_[(w * NCOL + c) * kRun + d], o);
        }
        if (part) {
          part[2 * NCOL + c * D + 32 * b0 + d] = o;
          if (b0 == 0 && d == 0) {
            part[c] = m;
            part[NCOL + c] = l;
          }
        } else {
          store_out(a, q, cs, c, 32 * b0 + d, l == 0.f ? 0.f : o / l);
          if (b0 == 0 && d == 0) store_lse(a, q, cs, c, m, l);
        }
      }
    }
  }
};

// Workgroup w takes the units [w per, (w + 1) per). Items that it holds whole are finished here;
// of the others, at most one begun before its share (part 2 w) and one that ends behind it
// (part 2 w + 1), it leaves partial results for k_kv_join. Bound by HBM (1.125 bytes per key and
// value element pair).
template <typename A, int NB, bool SPLIT>
__global__ __launch_bounds__(kThreads, NB <= 4 ? 2 : 1) void k_kv_attn(AttnArgs a) {
  typedef Attn<A, NB, SPLIT> X;
  __shared__ float lds[2 * kWaves * X::NCOL + kWaves * X::NCOL * 32 * X::kMergeBlocks];
  const TileShape ts = tile_shape<X::NCOL>(a.group);
  const int w = blockIdx.x;
  const Place pl = locate(a, ts, [&](int64_t per) { return w * per; });
  if (pl.r < 0) return;
  int64_t u = w * pl.per;
  const int64_t end = min(pl.total, u + pl.per);
  Request q = request(a, ts, pl.r);
  int64_t base = pl.base;
  while (u < end) {
    int64_t in = u - base;
    while (in >= units_of(a, q)) {  // on to the next request (one without new tokens has no units)
      base += units_of(a, q);
      q = request(a, ts, q.r + 1);
      in = u - base;
    }
    const int64_t item = in / q.steps;
    const int kvh = (int)(item / q.tiles), tile = (int)(item - (int64_t)kvh * q.tiles);
    const int v0 = (int)(in - item * q.steps), v1 = (int)min((int64_t)q.steps, v0 + (end - u));
    float *part = nullptr;
    if (v0 > 0 || v1 < q.steps) part = a.parts + (int64_t)(2 * w + (v0 == 0)) * X::kPart;
    X::segment(a, ts, q, kvh, tile, v0, v1, part, lds);
    u += v1 - v0;
  }
}

// Workgroup w joins the parts of the item whose first part workgroup w of k_kv_attn left, if it
// left one: part 2 w + 1 and the parts 2 w' of the following workgroups up to the item's end.
template <typename A, int NB, bool SPLIT>
__global__ __launch_bounds__(kThreads) void k_kv_join(AttnArgs a) {
  typedef Attn<A, NB, SPLIT> X;
  const TileShape ts = tile_shape<X::NCOL>(a.group);
  const int w = blockIdx.x;
  const Place pl = locate(a, ts, [&](int64_t per) { return (w + 1) * per - 1; });
  if (pl.r < 0) return;
  const Request q = request(a, ts, pl.r);
  const int64_t e = (w + 1) * pl.per, in = e - 1 - pl.base, item = in / q.steps;
  const int64_t start = pl.base + item * q.steps, stop = start + q.steps;
  if (start < w * pl.per || stop <= e) return;
  const int kvh = (int)(item / q.tiles), tile = (int)(item - (int64_t)kvh * q.tiles);
  const Columns cs = columns<X::NCOL>(a, ts, q, kvh, tile);
  const int last = (int)((stop - 1) / pl.per);  // workgroup with the item's last units
  const float *first = a.parts + (int64_t)(2 * w + 1) * X::kPart;
  auto part = [&](int i) { return i == w ? first : a.parts + (int64_t)(2 * i) * X::kPart; };
  for (int i = threadIdx.x; i < cs.count * X::D; i += kThreads) {
    const int c = i / X::D, d = i - c * X::D;
    float m = kLowest, l = 0.f, o = 0.f;
    for (int p = w; p <= last; ++p) {
      const float *x = part(p);
      const float pm = x[c], n = fmaxf(m, pm);
      const float f = __builtin_amdgcn_exp2f(m - n), h = __builtin_amdgcn_exp2f(pm - n);
      l = fmaf(l, f, h * x[X::NCOL + c]);
      o = fmaf(o, f, h * x[2 * X::NCOL + c * X::D + d]);
      m = n;
    }
    X::store_out(a, q, cs, c, d, l == 0.f ? 0.f : o / l);
    if (d == 0) X::store_lse(a, q, cs, c, m, l);
  }
}

template <typename A, int NB, bool SPLIT>
int launch(const AttnArgs &a, hipStream_t s) {
  k_kv_attn<A, NB, SPLIT><<<dim3(a.grid), kThreads, 0, s>>>(a);
  if (a.grid > 1) k_kv_join<A, NB, SPLIT><<<dim3(a.grid - 1), kThreads, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename A, bool SPLIT>
int launch_dim(const AttnArgs &a, hipStream_t s) {
  switch (a.g.nb) {
    case 2: return launch<A, 2, SPLIT>(a, s);
    case 3: return launch<A, 3, SPLIT>(a, s);
    case 4: return launch<A, 4, SPLIT>(a, s);
    default: return launch<A, 8, SPLIT>(a, s);
  }
}

bool split_type(int type) { return type != TQ_BF16; }

}  // namespace

size_t kv_attention_workspace(int type, int64_t head_dim, int grid) {
  const int ncol = split_type(type) ? 8 : 16;
  return (size_t)grid * 2 * ncol * (head_dim + 2) * 4;
}

int kv_attention_grid(int type, int64_t kv_heads, int64_t head_dim, int64_t group, int64_t rows,
                      int64_t requests, int64_t max_len) {
  (void)head_dim;
  // an upper bound of the units: every row a tile of its own over the longest sequence
  const int64_t ncol = split_type(type) ? 8 : 16;
  (void)requests;
  const int64_t tiles = rows * (group <= ncol ? 1 : (group + ncol - 1) / ncol);
  const int64_t steps = max_len / 32 + 2;
  const double units = (double)tiles * (double)kv_heads * (double)steps;
  const double most = units / kMinSteps + 1;
  return most < kGrid ? (int)most : kGrid;
}

int launch_kv_attention(int type, const AttnArgs &a, hipStream_t s) {
  return type == TQ_F32 ? launch_dim<ActF32, true>(a, s)
         : type == TQ_BF16 ? launch_dim<ActBF16, false>(a, s) : launch_dim<ActF16, true>(a, s);
}

}  // namespace tq
