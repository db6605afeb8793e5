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
#include <atomic>

#include "tq_kv.h"
#include "tq_kv_device.h"
#include "tq_launch.h"
#include "tq_mfma.h"

namespace tq {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3a4 __attribute__((ext_vector_type(3), aligned(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
// Workgroups per compute unit, from registers (168 or 256 a lane) and LDS (37 or 74 KB at head_dim
// 128 and 256); a full launch has just as many, all of them resident at once.
constexpr int resident(int nb) { return nb <= 4 ? 3 : 2; }
constexpr int kComputeUnits = 256;
#ifndef KV_ITEM
#define KV_ITEM 16
#endif
#ifndef KV_MIN
#define KV_MIN 8
#endif
constexpr int kMinUnits = KV_MIN;     // units per workgroup at least
constexpr int kItemUnits = KV_ITEM;    // what an item costs beside its steps (queries, merge, output)
constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kSlack = 2.f;    // see step()

// ---- the step's work as one line of units -----------------------------------------------------
// An item is a query tile (up to NCOL columns: tokens x heads of one kv head) of a request; its
// units are the 32-token steps of its request and kItemUnits for what it costs beside them. All
// items' units form one line, cut into equal shares, one a workgroup, so ragged batches load the
// chip evenly; a share of an item's units is the same share of its steps. The lengths live on the
// device, so every workgroup forms the prefix sums over the requests itself.
struct Request {
  int r, row0, fresh, len, first_pos;  // rows row0 .. row0 + fresh, tokens of the sequence
  int tiles, units;                    // query tiles, units per item
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
  q.units = kItemUnits + max(0, (q.len + 31) / 32 - seen_from(a, q.first_pos) / 32);
  return q;
}

__device__ __forceinline__ int64_t units_of(const AttnArgs &a, const Request &q) {
  return (int64_t)a.g.heads * q.tiles * q.units;
}

// a / b for 0 <= a < 2^53, 0 < b < 2^31 (a 64-bit integer division takes over a hundred
// instructions; the quotient of the doubles is off by less than one).
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  int64_t q = (int64_t)((double)a / (double)b);
  const int64_t r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

struct Place {
  int64_t total, per;  // units of all requests, units per workgroup
  int r;               // the request that holds the wanted unit
  int64_t base;        // its first unit
};

// A value that is the same in all lanes, as a scalar (LDS reads are per lane to the compiler, and
// everything derived from the place would then be computed per lane).
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

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
  p.total = uniform64(p.total);
  p.per = max((int64_t)kMinUnits, quotient(p.total + a.grid - 1, a.grid));
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
  p.r = __builtin_amdgcn_readfirstlane((int)found[0]);
  p.base = uniform64(found[1]);
  return p;
}

// ---- operands ---------------------------------------------------------------------------------

// Constants of unpack(), in registers: with the masks as scalars and the exponent as a vector
// register, mask and exponent are one v_and_or_b32 (an instruction takes one literal or scalar).
struct Unpack {
  uint32_t low, high, exponent;
  __device__ __forceinline__ Unpack() : low(0x000F000Fu), high(0x00F000F0u), exponent(0x64006400u) {
    asm("" : "+s"(low), "+s"(high), "+v"(exponent));
  }
};

// The nibbles of one dword of quants as fp16 integers n - 8: the bits of a nibble under the exponent
// of 1024 are 1024 + n, those of a high nibble 1024 + 16 n. Low nibbles of bytes (0, 2), of bytes
// (1, 3), high nibbles of both pairs. (As fp16 subnormals n 2^-24, by masks alone, the products
// lose up to ten bits: the matrix cores align a product by its operands' exponent fields. Measured
// on this kernel: 3e-4 of the terms' magnitude against 3e-7.)
__device__ __forceinline__ void unpack(const Unpack &k, uint32_t w, uint32_t out[4]) {
  const uint32_t u = w >> 8;
  const f16x2 low = {(_Float16)-1032.f, (_Float16)-1032.f};
  const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  const f16x2 high = {(_Float16)-72.f, (_Float16)-72.f};
  auto half2 = [](uint32_t v) { return __builtin_bit_cast(f16x2, v); };
  out[0] = __builtin_bit_cast(uint32_t, half2((w & k.low) | k.exponent) + low);
  out[1] = __builtin_bit_cast(uint32_t, half2((u & k.low) | k.exponent) + low);
  out[2] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(half2((w & k.high) | k.exponent), sixteenth, high));
  out[3] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(half2((u & k.high) | k.exponent), sixteenth, high));
}

__device__ __forceinline__ f16x8 join(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(f16x8, u32x4{a, b, c, d});
}

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Bytes of one step (two tiles), and the LDS-DMA loads that fetch a tile: whole waves of 16 bytes
// a lane, then the rest.
template <int NB>
struct Step {
  static constexpr int kTile = 576 * NB, kBytes = 2 * kTile;
  static constexpr int kFull = kTile / 1024, kRest = kTile % 1024 / 16;
  static constexpr int kLoads = 2 * (kFull + (kRest ? 1 : 0));
};

// One tile into LDS at `to` (the same for the wave), in kLoads / 2 loads.
template <int NB>
__device__ __forceinline__ void fetch_tile(const uint8_t *p, int lane, uint32_t to) {
  typedef Step<NB> S;
  p += lane * 16;
#pragma unroll
  for (int i = 0; i < S::kFull; ++i) load_lds16(p + 1024 * i, to + 1024 * i);
  if (S::kRest && lane < S::kRest) load_lds16(p + 1024 * S::kFull, to + 1024 * S::kFull);
}

// Waits until at most `ahead` steps' loads are outstanding.
template <int NB, int MOST>
__device__ __forceinline__ void wait_steps(int ahead) {
  if constexpr (MOST == 0) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  } else {
    if (ahead >= MOST) asm volatile("s_waitcnt vmcnt(%0)" : : "i"(MOST * Step<NB>::kLoads) : "memory");
    else wait_steps<NB, MOST - 1>(ahead);
  }
}

template <int NB>
__device__ __forceinline__ void read_quants(const uint8_t *p, int lane, uint32_t *out) {
  if constexpr (NB == 2) {
    const u32x2 w = *(const u32x2 *)(p + lane * 8);
    out[0] = w[0];
    out[1] = w[1];
  } else if constexpr (NB == 3) {
    const u32x3a4 w = *(const u32x3a4 *)(p + lane * 12);
#pragma unroll
    for (int i = 0; i < 3; ++i) out[i] = w[i];
  } else {
#pragma unroll
    for (int c = 0; c < NB / 4; ++c) {
      const u32x4 w = *(const u32x4 *)(p + c * 1024 + lane * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[4 * c + i] = w[i];
    }
  }
}

template <int NB>
__device__ __forceinline__ void read_scales(const uint8_t *p, int g, uint32_t *out) {
  p += g * 8 * NB;
  if constexpr (NB % 2 == 0) {
#pragma unroll
    for (int c = 0; c < NB / 2; ++c) {
      const u32x4 w = *(const u32x4 *)(p + 16 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[4 * c + i] = w[i];
    }
  } else {
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      const u32x2 w = *(const u32x2 *)(p + 8 * c);
      out[2 * c] = w[0];
      out[2 * c + 1] = w[1];
    }
  }
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
  static constexpr int kPart = NCOL * (D + 2);  // floats of a partial result: m, l, O (16-byte aligned)
  static constexpr int kMergeBlocks = NB < 4 ? NB : 4;  // blocks merged over the waves at a time
  static constexpr int kAhead = NB == 2 ? 2 : 1;        // steps that a wave has on their way
  static constexpr int kRing = kWaves * (kAhead + 1) * Step<NB>::kBytes;
  static constexpr int kMerge = (2 * kWaves * NCOL + kWaves * NCOL * 32 * kMergeBlocks) * 4;
  static constexpr int kLds = kRing > kMerge ? kRing : kMerge;

  struct State {
    f32x4 o[2 * NB];  // rows 4 g + r (query columns), columns l % 16: dimension 32 b + 16 half + l % 16
    float m, l;       // of column l % 16: reference exponent (shared by the lane groups), this lane's sum
    int top;          // every value scale so far is below 2^(top - 15) (the same for the wave)
  };

  // p times a value's scale as an fp16 operand: one term, or for SPLIT the second term in the rows
  // of the second terms (`second` 1).
  static __device__ __forceinline__ _Float16 weight(float p, float d, float second) {
    float x = fmaf(p, d, 0.f);
    if constexpr (SPLIT) {
      // Both terms from one fp32 value: where the compiler rounds the exact product to fp16 for one
      // of them and its fp32 rounding for the other, near a tie they are an fp16 step apart.
      asm("" : "+v"(x));
      const _Float16 h = (_Float16)x;
      return (_Float16)fmaf(-(float)h, second, x);
    }
    return (_Float16)x;
  }

  // One step of 32 tokens. Reference exponent: weights are p = 2^(s - m) with m such that p times
  // the value's scale stays below 2^15, the fp16 range, whatever the scales are: m >= s + top - 28 - kSlack
  // for every token, where top (1, 2, 4, 8 or 16 by one mask test on the scales' exponents, exact
  // above 16) bounds the scales. m is set without the slack and moves only when a token passes it,
  // so the exchange between lane groups and the rescaling of O are rare. `l` sums p in the same
  // reference. `mask` (the same for the wave): some token of the step is hidden from some column.
  static __device__ __forceinline__ void step(const uint8_t *at, const f16x8 (&qf)[NB], float qs,
                                              bool mask, int lo, int hi, int any_lo, int any_hi,
                                              int t0, int lane, float second, State &st) {
    constexpr int kTile = Step<NB>::kTile, kQuant = 256 * NB, kHalf = 288 * NB;
    const Unpack uk;
    const int g = lane >> 4;
    float s[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t kq[NB], ks[2 * NB];
      read_quants<NB>(at + i * kTile, lane, kq);
      read_scales<NB>(at + i * kTile + kQuant, g, ks);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t n[4];
        unpack(uk, kq[b], n);
        const f32x4 d = mfma(join(n[0], n[1], n[2], n[3]), qf[b], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(scale_of(ks, b, r), d[r], acc[r]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[r];
        if constexpr (SPLIT) v += row_swap8(v);  // hi and lo columns of one query
        s[4 * i + r] = v;
      }
      if constexpr (NB == 8) __builtin_amdgcn_sched_barrier(0);  // the tiles one by one: registers
    }
    uint32_t vs[2][2 * NB];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_scales<NB>(at + i * kTile + kHalf + kQuant, g, vs[i]);
    // the scales' bits together: they have a bit of exponent 16, 8, 4 ... exactly if one has it
    uint32_t any_scale = 0;
    bool odd_scales = false;
    if (!mask) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) any_scale |= vs[i][j];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
        s[i] = tok >= lo && tok < hi ? s[i] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // scales of tokens that no column sees may be anything: 0
          const int tok = t0 + 16 * i + 4 * g + 2 * j;
          const uint32_t keep = (tok >= any_lo && tok < any_hi ? 0xFFFFu : 0u) |
                                (tok + 1 >= any_lo && tok + 1 < any_hi ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int b = 0; b < NB; ++b) any_scale |= vs[i][2 * b + j] &= keep;
        }
      odd_scales = __any((any_scale & 0x7C00u) == 0x7C00u || (any_scale & 0x7C000000u) == 0x7C000000u);
    }
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
    auto over = [&](int top) {  // exponents of top and more, for top a power of two up to 16
      const uint32_t bits = 0x7C00u & ~((uint32_t)(top - 1) << 10);
      return (any_scale & (bits | bits << 16)) != 0;
    };
    float want = fmaf(mx, qs, (float)(st.top - 28));
    if (__any(over(min(st.top, 16)) || want > st.m + kSlack)) {
      while (st.top < 16 && __any(over(st.top))) st.top *= 2;
      if (__any(over(16))) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j) {
            most = max(most, vs[i][j] & 0x7C00u);
            most = max(most, vs[i][j] >> 16 & 0x7C00u);
          }
        int e = (int)(most >> 10) + 1;
        e = max(e, __shfl_xor(e, 16));
        e = max(e, __shfl_xor(e, 32));
        st.top = max(st.top, __builtin_amdgcn_readfirstlane(e));
      }
      want = fmaf(mx, qs, (float)(st.top - 28));
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
    uint32_t vq[2][NB];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_quants<NB>(at + i * kTile + kHalf, lane, vq[i]);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f16x8 w;
      if (odd_scales) {  // a hidden token's scale may be no number: 0 times it must stay 0
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t d2 = opaque(vs[i >> 2][2 * b + (i >> 1 & 1)]);
          const float d = half_bits_to_float(i & 1 ? d2 >> 16 : d2);
          w[i] = weight(p[i], s[i] == -INFINITY ? 0.f : d, second);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = weight(p[i], scale_of(vs[i >> 2], b, i & 3), second);
      }
      uint32_t n0[4], n1[4];
      unpack(uk, vq[0][b], n0);
      unpack(uk, vq[1][b], n1);
      st.o[2 * b] = mfma(w, join(n0[0], n0[1], n1[0], n1[1]), st.o[2 * b]);
      st.o[2 * b + 1] = mfma(w, join(n0[2], n0[3], n1[2], n1[3]), st.o[2 * b + 1]);
    }
  }

  // Column `col` of a tile whose first row of q is `row`, first head head0, with `per` heads a token.
  static __device__ __forceinline__ void store_out(const AttnArgs &a, int row, int head0, int per,
                                                   int col, int d, float v) {
    const int tok = col / per, head = head0 + col - tok * per;
    T *out = (T *)a.out.data + (int64_t)(row + tok) * a.out.row_stride + (int64_t)head * a.out.head_stride;
    out[d] = A::from(v);
  }
  static __device__ __forceinline__ void store_lse(const AttnArgs &a, int row, int head0, int per,
                                                   int col, float m, float l) {
    if (!a.lse) return;
    const int tok = col / per, head = head0 + col - tok * per;
    a.lse[(int64_t)(row + tok) * (a.group * a.g.heads) + head] =
        l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
  }

  // The units [v0, v1) of an item, by the whole workgroup.
  static __device__ void segment(const AttnArgs &a, const TileShape &ts, const Request &q, int kvh,
                                 int tile, int v0, int v1, int done, int share_units, float *part,
                                 uint8_t *lds) {
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
    State st;
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) st.o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    st.m = kLowest;
    st.l = 0.f;
    st.top = 1;
    // the tile's own steps: the item's units are spread over them (a tile of early tokens has fewer)
    const int s0 = any_lo / 32, n = max(0, (any_hi + 31) / 32 - s0);
    // A wave that is ahead steps back: priority 3 in the first quarter of the workgroup's share, then
    // 2, 1, 0. (Issue goes to the oldest wave first: without it the first workgroups of a compute
    // unit ended after 31 us where the last took 50 us, alone on their SIMDs at the end.)
    int level = 0, next_level = 0;
    auto step_back = [&](int i) {
      if (i < next_level) return;
      if (level == 0) __builtin_amdgcn_s_setprio(3);
      else if (level == 1) __builtin_amdgcn_s_setprio(2);
      else if (level == 2) __builtin_amdgcn_s_setprio(1);
      else __builtin_amdgcn_s_setprio(0);
      ++level;
      next_level = level == 4 ? 0x7FFFFFFF : (level * share_units / 4 - done) / kWaves;
    };
    const double share = (double)n / (double)q.units;  // exact where it has to be: 0 at 0, n at units
    auto step_at = [&](int v) { return s0 + (v == q.units ? n : (int)(v * share)); };
    const int from = step_at(v0), to = step_at(v1);
    const int32_t *table = a.block_table + (int64_t)q.r * a.max_blocks;
    const int last_block = ((q.len + a.g.page_tokens - 1) >> a.g.page_shift) - 1;
    const uint8_t *head_data = a.g.data + (int64_t)kvh * a.g.head_bytes;
    // A tile's address; a page outside the cache reads page 0 (its tokens are masked below).
    // (constant address space: a scalar load, which does not count among the fetches in flight)
    auto page_of = [&](int t) {
      typedef __attribute__((address_space(4))) const int32_t *scalar;
      return ((scalar)(uintptr_t)table)[__builtin_amdgcn_readfirstlane(min(t >> a.g.page_shift, last_block))];
    };
    const unsigned pages = (unsigned)a.g.pages;
    auto tile_at = [&](int t, int page) {
      const int64_t ok = (unsigned)page < pages ? page : 0;
      return head_data + ok * a.g.page_bytes + (int64_t)((t & (a.g.page_tokens - 1)) >> 4) * a.g.tile_bytes;
    };
    // Steps from + wave, from + wave + kWaves, ...: kAhead steps of the wave are on their way into
    // its own ring in LDS (no barriers: a wave waits for its own loads only).
    const int steps = to - from > wave ? (to - from - wave + kWaves - 1) / kWaves : 0;
    const uint8_t *ring = lds + wave * (kAhead + 1) * Step<NB>::kBytes;
    const uint32_t ring_at = lds_address(ring);
    const float second = lane & 8 ? 1.f : 0.f;
    auto token_of = [&](int i) { return 32 * (from + wave + i * kWaves); };
    int fp0 = 0, fp1 = 0;  // pages of the next step to fetch
    if (steps > 0) {
      fp0 = page_of(token_of(0));
      fp1 = page_of(token_of(0) + 16);
    }
    unsigned bad_pages = 0;  // two bits for each place of the ring
    auto fetch = [&](int i) {
      const int t = token_of(i), place = i % (kAhead + 1);
      const uint32_t at = ring_at + (uint32_t)place * Step<NB>::kBytes;
      const unsigned bad = ((unsigned)fp0 >= pages) | ((unsigned)fp1 >= pages) << 1;
      bad_pages = (bad_pages & ~(3u << (2 * place))) | bad << (2 * place);
      const uint8_t *p0 = tile_at(t, fp0), *p1 = tile_at(t + 16, fp1);
      const int tn = token_of(i + 1);
      fp0 = page_of(tn);
      fp1 = page_of(tn + 16);
      fetch_tile<NB>(p0, lane, at);
      fetch_tile<NB>(p1, lane, at + Step<NB>::kTile);
    };
    for (int i = 0; i < kAhead && i < steps; ++i) fetch(i);
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
    for (int i = 0; i < steps; ++i) {
      // the step that takes the place of the last one read, whose reads have all returned
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const unsigned bad = bad_pages >> (2 * (i % (kAhead + 1))) & 3u;
      step_back(i);
      if (i + kAhead < steps) fetch(i + kAhead);
      wait_steps<NB, kAhead>(steps - 1 - i);
      const uint8_t *at = ring + (i % (kAhead + 1)) * Step<NB>::kBytes;
      const int t0 = token_of(i);
      const bool inner = t0 >= all_lo && t0 + 32 <= all_hi;
      const int l0 = bad & 1 ? t0 + 16 : 0, h0 = bad & 2 ? t0 + 16 : 0x7FFFFFFF;
      step(at, qf, qs, !inner || bad, max(lo, l0), min(hi, h0), max(any_lo, l0), min(any_hi, h0), t0, lane,
           second, st);
    }
    int id = threadIdx.x;  // formed anew: addresses below are not to be kept through the loop above
    asm volatile("" : "+v"(id));
    const int l16 = id & 15, grp = id >> 4 & 3;
    // join the waves: sums over the lane groups, then O in runs of up to 128 dimensions
    st.l += __shfl_xor(st.l, 16);
    st.l += __shfl_xor(st.l, 32);
    float *lm = (float *)lds, *ll = lm + kWaves * NCOL, *lo_ = lm + 2 * kWaves * NCOL;
    __syncthreads();
    if ((id & 63) < NCOL) {
      lm[wave * NCOL + l16] = st.m;
      ll[wave * NCOL + l16] = st.l;
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
          const int row = 4 * grp + r;
          if (row < NCOL) lo_[(wave * NCOL + row) * kRun + 16 * j + l16] = v;
        }
      __syncthreads();
      for (int i = id; i < NCOL * kRun; i += kThreads) {
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
          store_out(a, q.row0 + cs.tok0, cs.head0, cs.per, c, 32 * b0 + d, l == 0.f ? 0.f : o / l);
          if (b0 == 0 && d == 0) store_lse(a, q.row0 + cs.tok0, cs.head0, cs.per, c, m, l);
        }
      }
    }
    __syncthreads();  // the next segment's fetches go where these sums were
  }
};

// What k_kv_join needs of the item whose first part a workgroup left (parts 0: none).
struct JoinItem {
  int parts, row, head0, per, count;
};

// Workgroup w takes the units [w per, (w + 1) per). Items that it holds whole are finished here;
// of the others, at most one begun before its share (part 2 w) and one that ends behind it
// (part 2 w + 1), it leaves partial results for k_kv_join. Bound by HBM (1.125 bytes per key and
// value element pair).
template <typename A, int NB, bool SPLIT>
__global__ __launch_bounds__(kThreads, resident(NB)) void k_kv_attn(AttnArgs a) {
  typedef Attn<A, NB, SPLIT> X;
  extern __shared__ __align__(16) uint8_t attn_lds[];
  const TileShape ts = tile_shape<X::NCOL>(a.group);
  // neighbouring shares on one XCD: query tiles of one request read the same keys through one L2
  const int w = a.grid % 8 ? (int)blockIdx.x : (int)(blockIdx.x % 8 * (a.grid / 8) + blockIdx.x / 8);
  const Place pl = locate(a, ts, [&](int64_t per) { return w * per; });
  JoinItem join = {0, 0, 0, 0, 0};
  int64_t u = w * pl.per;
  const int64_t end = pl.r < 0 ? u : min(pl.total, u + pl.per);
  Request q = request(a, ts, max(pl.r, 0));
  int64_t base = pl.base;
  while (u < end) {
    int64_t in = u - base;
    while (in >= units_of(a, q)) {  // on to the next request (one without new tokens has no units)
      base += units_of(a, q);
      q = request(a, ts, q.r + 1);
      in = u - base;
    }
    const int64_t item = quotient(in, q.units);
    const int kvh = (int)quotient(item, q.tiles), tile = (int)(item - (int64_t)kvh * q.tiles);
    const int v0 = (int)(in - item * q.units), v1 = (int)min((int64_t)q.units, v0 + (end - u));
    float *part = nullptr;
    if (v0 > 0 || v1 < q.units) part = a.parts + (int64_t)(2 * w + (v0 == 0)) * X::kPart;
    if (v0 == 0 && v1 < q.units) {
      const Columns cs = columns<X::NCOL>(a, ts, q, kvh, tile);
      const int64_t last = base + (item + 1) * q.units - 1;
      join = {(int)(last / pl.per) - w + 1, q.row0 + cs.tok0, cs.head0, cs.per, cs.count};
    }
    X::segment(a, ts, q, kvh, tile, v0, v1, (int)min(u - w * pl.per, (int64_t)1 << 28), (int)min(pl.per, (int64_t)1 << 28), part, attn_lds);
    u += v1 - v0;
  }
  if (threadIdx.x == 0) ((JoinItem *)a.joins)[w] = join;
}

// Workgroup (w, y) joins the item whose first part workgroup w of k_kv_attn left: part 2 w + 1 and
// the parts 2 w' of the following workgroups. A thread takes four dimensions of a column and every
// fourth part. Bound by latency: the parts' references, sums and outputs are read eight parts at a
// time, at once.
constexpr int kJoinUnits = 128, kJoinGroups = 4;

template <typename A, int NB, bool SPLIT>
__global__ __launch_bounds__(kJoinUnits * kJoinGroups) void k_kv_join(AttnArgs a) {
  typedef Attn<A, NB, SPLIT> X;
  constexpr int kRuns = X::D / 4, kBatch = 8;
  __shared__ f32x4 other_o[kJoinGroups - 1][kJoinUnits];
  __shared__ float other_m[kJoinGroups - 1][kJoinUnits], other_l[kJoinGroups - 1][kJoinUnits];
  const int w = blockIdx.x, unit = threadIdx.x % kJoinUnits, group = threadIdx.x / kJoinUnits;
  const int i = blockIdx.y * kJoinUnits + unit;
  const JoinItem item = ((const JoinItem *)a.joins)[w];
  if (item.parts == 0 || (int)blockIdx.y * kJoinUnits >= item.count * kRuns) return;
  const int c = i / kRuns, d = (i - c * kRuns) * 4;
  const bool live = c < item.count;
  float m = kLowest, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  auto join = [&](float pm, float pl, f32x4 po) {
    const float top = fmaxf(m, pm);
    const float f = __builtin_amdgcn_exp2f(m - top), h = __builtin_amdgcn_exp2f(pm - top);
    l = fmaf(l, f, h * pl);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = fmaf(o[j], f, h * po[j]);
    m = top;
  };
  for (int at = group; live && at < item.parts; at += kBatch * kJoinGroups) {
    float pm[kBatch], pl[kBatch];
    f32x4 po[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int n = at + k * kJoinGroups;
      if (n >= item.parts) break;
      const float *p = a.parts + (int64_t)(2 * (w + n) + (n == 0)) * X::kPart;
      pm[k] = p[c];
      pl[k] = p[X::NCOL + c];
      po[k] = *(const f32x4 *)(p + 2 * X::NCOL + c * X::D + d);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (at + k * kJoinGroups >= item.parts) break;
      join(pm[k], pl[k], po[k]);
    }
  }
  if (group > 0) {
    other_m[group - 1][unit] = m;
    other_l[group - 1][unit] = l;
    other_o[group - 1][unit] = o;
  }
  __syncthreads();
  if (group > 0 || !live) return;
#pragma unroll
  for (int k = 0; k < kJoinGroups - 1; ++k) join(other_m[k][unit], other_l[k][unit], other_o[k][unit]);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    X::store_out(a, item.row, item.head0, item.per, c, d + j, l == 0.f ? 0.f : o[j] / l);
  if (d == 0) X::store_lse(a, item.row, item.head0, item.per, c, m, l);
}

template <typename A, int NB, bool SPLIT>
int launch(const AttnArgs &args, hipStream_t s) {
  AttnArgs a = args;
  a.joins = a.parts + (int64_t)a.grid * 2 * Attn<A, NB, SPLIT>::kPart;
  constexpr int kLds = Attn<A, NB, SPLIT>::kLds;
  if (kLds > 64 * 1024) {  // once a device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return -1;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
      if (hipFuncSetAttribute(reinterpret_cast<const void *>(&k_kv_attn<A, NB, SPLIT>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, kLds) != hipSuccess)
        return -1;
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  k_kv_attn<A, NB, SPLIT><<<dim3(a.grid), kThreads, kLds, s>>>(a);
  constexpr int kUnits = Attn<A, NB, SPLIT>::NCOL * 8 * NB;  // units of an item
  if (a.grid > 1)
    k_kv_join<A, NB, SPLIT><<<dim3(a.grid - 1, (kUnits + kJoinUnits - 1) / kJoinUnits), kJoinUnits * kJoinGroups, 0, s>>>(a);
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
  return (size_t)grid * (2 * ncol * (head_dim + 2) * 4 + sizeof(JoinItem));
}

int kv_attention_grid(int type, int64_t kv_heads, int64_t head_dim, int64_t group, int64_t rows,
                      int64_t requests, int64_t max_len) {
  // an upper bound of the units: every row a tile of its own over the longest sequence
  const int64_t ncol = split_type(type) ? 8 : 16;
  (void)requests;
  const int64_t tiles = rows * (group <= ncol ? 1 : (group + ncol - 1) / ncol);
  const int64_t steps = max_len / 32 + 2 + kItemUnits;
  const double units = (double)tiles * (double)kv_heads * (double)steps;
  const double most = units / kMinUnits + 1;
  const int full = kComputeUnits * resident((int)(head_dim / 32));
  return most < full ? (int)most : full;
}

int launch_kv_attention(int type, const AttnArgs &a, hipStream_t s) {
  return type == TQ_F32 ? launch_dim<ActF32, true>(a, s)
         : type == TQ_BF16 ? launch_dim<ActBF16, false>(a, s) : launch_dim<ActF16, true>(a, s);
}

}  // namespace tq
