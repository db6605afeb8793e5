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
constexpr int kMinUnits = 8;  // units per workgroup at least
// What an item costs beside its steps (queries, merge, output), in steps of k_kv_attn and k_kv_wide.
constexpr int item_units(bool wide) { return wide ? 5 : 16; }
constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kSlack = 2.f;    // see step()

// A request with more query columns a kv head (new tokens x heads) than this goes to k_kv_wide, which
// is launched beside k_kv_attn from an average of as many a request (the lengths live on the device;
// the launch costs about 8 us where no request is for it). Two tiles of 16 columns cost k_kv_attn
// as much issue as k_kv_wide's workgroup costs for up to 128.
constexpr int kWideCols = 32;
// Query tiles of 16 columns that a wave of k_kv_wide takes (registers: two do not fit beside two
// terms of an fp32 query or beside head_dim 256 without scratch).
constexpr int wide_tiles(bool f32, int nb) { return nb == 8 || (f32 && nb == 4) ? 1 : 2; }
// Workgroups of k_kv_wide per compute unit (registers: 256 a lane up to head_dim 128, 512 for 256).
constexpr int resident_wide(int nb) { return nb <= 4 ? 2 : 1; }

bool split_type(int type) { return type != TQ_BF16; }

bool wide_launch(int64_t group, int64_t rows, int64_t requests) { return rows * group > kWideCols * requests; }

// ---- the step's work as one line of units -----------------------------------------------------
// An item is a query tile (up to NCOL columns: tokens x heads of one kv head) of a request; its
// units are the 32-token steps of its request and item_units for what it costs beside them. All
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

// WIDE: of the requests with more than wide_cols query columns a kv head, else of the others; a
// request of the other class has no tiles.
template <bool WIDE>
__device__ __forceinline__ Request request(const AttnArgs &a, const TileShape &ts, int r) {
  Request q;
  q.r = r;
  q.row0 = min(max(a.cu_new[r], 0), a.rows);
  q.fresh = max(min(a.cu_new[r + 1], a.rows) - q.row0, 0);
  q.len = (int)min((int64_t)max(a.seq_len[r], 0), (int64_t)a.max_blocks << a.g.page_shift);
  q.first_pos = q.len - q.fresh;
  const bool wide = (int64_t)q.fresh * a.group > a.wide_cols;
  q.tiles = wide == WIDE ? (q.fresh + ts.tokens - 1) / ts.tokens * ts.splits : 0;
  q.units = item_units(WIDE) + max(0, (q.len + 31) / 32 - seen_from(a, q.first_pos) / 32);
  return q;
}

__device__ __forceinline__ int64_t units_of(const AttnArgs &a, const Request &q) {
  return (int64_t)a.g.heads * q.tiles * q.units;
}

// a / b for 0 <= a, 0 < b < 2^31 (a 64-bit integer division takes over a hundred instructions; the
// quotient of the doubles is off by one at most below 2^53, by little more above).
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  int64_t q = (int64_t)((double)a / (double)b), r = a - q * b;
  for (; r < 0; r += b) --q;
  for (; r >= b; r -= b) ++q;
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
template <bool WIDE, typename F>
__device__ __forceinline__ Place locate(const AttnArgs &a, const TileShape &ts, F unit_of) {
  __shared__ int64_t sums[kWaves];
  __shared__ int64_t found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int n = (a.requests + kThreads - 1) / kThreads;
  const int r0 = min(a.requests, tid * n), r1 = min(a.requests, r0 + n);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += units_of(a, request<WIDE>(a, ts, r));
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
      const int64_t m = units_of(a, request<WIDE>(a, ts, r));
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

// ---- softmax over steps -----------------------------------------------------------------------

// Running results of CT query tiles of 16 columns.
template <int NB, int CT>
struct State {
  f32x4 o[CT][2 * NB];  // rows 4 g + r (columns of the tile), columns l % 16: dimension 32 b + 16 half + l % 16
  float m[CT], l[CT];   // of column l % 16: reference exponent (shared by the lane groups), this lane's sum
  int top;              // every value scale so far is below 2^(top - 15) (the same for the wave)

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < CT; ++c) {
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) o[c][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      m[c] = kLowest;
      l[c] = 0.f;
    }
    top = 1;
  }
};

// The bits of a step's value scales together: they have a bit of exponent 16, 8, 4 ... exactly if
// one of them has it. With `mask`, scales of tokens outside any_lo .. any_hi (which no column sees and
// which may be anything) become 0, and `odd` says whether one may be no number.
template <int NB>
__device__ __forceinline__ uint32_t scale_bits(uint32_t (&vs)[2][2 * NB], bool mask, int any_lo, int any_hi,
                                               int t0, int g, bool &odd) {
  uint32_t bits = 0;
  odd = false;
  if (!mask) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) bits |= vs[i][j];
    return bits;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tok = t0 + 16 * i + 4 * g + 2 * j;
      const uint32_t keep = (tok >= any_lo && tok < any_hi ? 0xFFFFu : 0u) |
                            (tok + 1 >= any_lo && tok + 1 < any_hi ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int b = 0; b < NB; ++b) bits |= vs[i][2 * b + j] &= keep;
    }
  odd = __any((bits & 0x7C00u) == 0x7C00u || (bits & 0x7C000000u) == 0x7C000000u);
  return bits;
}

// Logits s (of the lane's 8 tokens, times qs) to weights p = 2^(s - m), in place, with the sums and
// outputs so far brought to the same reference m: such that p times the value's scale stays below
// 2^15, the fp16 range, whatever the scales are. m >= s + top - 28 - kSlack for every token, where
// top (1, 2, 4, 8 or 16 by one mask test on the scales' exponents, exact above 16) bounds the scales.
// m is set without the slack and moves only when a token passes it, so the exchange between lane
// groups and the rescaling of O are rare.
template <int NB, int CT>
__device__ __forceinline__ void weigh(float (&s)[CT][8], const float (&qs)[CT], const uint32_t (&vs)[2][2 * NB],
                                      uint32_t bits, int g, State<NB, CT> &st) {
  auto over = [&](int top) {  // exponents of top and more, for top a power of two up to 16
    const uint32_t b = 0x7C00u & ~((uint32_t)(top - 1) << 10);
    return (bits & (b | b << 16)) != 0;
  };
  float mx[CT];
  bool move = over(min(st.top, 16));
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    mx[c] = s[c][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx[c] = fmaxf(mx[c], s[c][i]);
    move |= fmaf(mx[c], qs[c], (float)(st.top - 28)) > st.m[c] + kSlack;
  }
  if (__any(move)) {
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
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      float want = fmaf(mx[c], qs[c], (float)(st.top - 28));
      want = fmaxf(want, __shfl_xor(want, 16));
      want = fmaxf(want, __shfl_xor(want, 32));
      const float m = fmaxf(st.m[c], want);
      const float alpha = __builtin_amdgcn_exp2f(st.m[c] - m);
      st.m[c] = m;
      st.l[c] *= alpha;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float f = __shfl(alpha, 4 * g + r);
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) st.o[c][j][r] *= f;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[c][i] = __builtin_amdgcn_exp2f(fmaf(s[c][i], qs[c], -st.m[c]));
      st.l[c] += s[c][i];
    }
}

// Scale of token i (of the lane's 8) of block b, taken as 0 where the column (which sees lo .. hi)
// does not see the token: its bits may be no number, and 0 times it must stay 0. Its own copy of
// the bits, so that the usual path keeps its half-register operands.
__device__ __forceinline__ float odd_scale(const uint32_t *vs, int b, int i, int t0, int g, int lo, int hi) {
  const uint32_t d2 = opaque(vs[2 * b + (i >> 1 & 1)]);
  const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
  return tok >= lo && tok < hi ? half_bits_to_float(i & 1 ? d2 >> 16 : d2) : 0.f;
}

// The power of two that a query row with largest magnitude `most` is multiplied by.
__device__ __forceinline__ int query_exponent(float most) {
  return most > 0.f && most < INFINITY ? min(15 - __builtin_amdgcn_frexp_expf(most), 100) : 0;
}

// The softmax scale for a query times 2^e; not 0, which times a hidden token's -infinity would be no number.
__device__ __forceinline__ float query_scale(float scale, int e) { return fmaxf(ldexpf(scale, -e), 1.17549435e-38f); }

// Column `col` of a tile whose first row of q is `row`, first head head0, with `per` heads a token.
template <typename A>
__device__ __forceinline__ void store_out(const AttnArgs &a, int row, int head0, int per, int col, int d,
                                          float v) {
  const int tok = col / per, head = head0 + col - tok * per;
  typename A::type *out = (typename A::type *)a.out.data + (int64_t)(row + tok) * a.out.row_stride +
                          (int64_t)head * a.out.head_stride;
  out[d] = A::from(v);
}
__device__ __forceinline__ void store_lse(const AttnArgs &a, int row, int head0, int per, int col, float m,
                                          float l) {
  if (!a.lse) return;
  const int tok = col / per, head = head0 + col - tok * per;
  a.lse[(int64_t)(row + tok) * (a.group * a.g.heads) + head] =
      l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

// A wave that is ahead steps back: priority 3 in the first quarter of the workgroup's share, then 2,
// 1, 0. Issue goes to the oldest wave first: without it the first workgroups of a compute unit ended
// after 31 us where the last took 50 us (k_kv_wide: 400 and 540), alone on their SIMDs at the end.
struct StepBack {
  int done, share, stride;  // units done before this segment, of the share; units from step to step
  int level = 0, next = 0;

  __device__ __forceinline__ void at(int i) {
    if (i < next) return;
    do {
      if (level == 0) __builtin_amdgcn_s_setprio(3);
      else if (level == 1) __builtin_amdgcn_s_setprio(2);
      else if (level == 2) __builtin_amdgcn_s_setprio(1);
      else __builtin_amdgcn_s_setprio(0);
      ++level;
      next = level >= 4 ? 0x7FFFFFFF : ((int)((int64_t)level * share / 4) - done) / stride;
    } while (i >= next);
  }
};

// ---- few columns: waves share an item's steps ----------------------------------------------------

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

  static constexpr bool kWide = false;
  typedef A Act;

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

  // One step of 32 tokens; `mask` (the same for the wave): some token is hidden from some column.
  static __device__ __forceinline__ void step(const uint8_t *at, const f16x8 (&qf)[NB], float qs,
                                              bool mask, int lo, int hi, int any_lo, int any_hi,
                                              int t0, int lane, float second, State<NB, 1> &st) {
    constexpr int kTile = Step<NB>::kTile, kQuant = 256 * NB, kHalf = 288 * NB;
    const Unpack uk;
    const int g = lane >> 4;
    float s[1][8];
    // Software pipeline, kept by the scheduling barriers: everything the products need is read at
    // once, and a product's results are scaled while the next one is multiplied.
    constexpr int kTiles = NB == 8 ? 1 : 2;  // tiles read at once (registers)
    uint32_t vs[2][2 * NB];
#pragma unroll
    for (int i0 = 0; i0 < 2; i0 += kTiles) {
      uint32_t kq[kTiles][NB], ks[kTiles][2 * NB];
      f32x4 d[2];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        read_quants<NB>(at + (i0 + i) * kTile, lane, kq[i]);
        read_scales<NB>(at + (i0 + i) * kTile + kQuant, g, ks[i]);
      }
      if (kTiles == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) read_scales<NB>(at + i * kTile + kHalf + kQuant, g, vs[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n <= kTiles * NB; ++n) {  // product n: tile i0 + n / NB, block n % NB
        if (n < kTiles * NB) {
          uint32_t q[4];
          unpack(uk, kq[n / NB][n % NB], q);
          d[n & 1] = mfma(join(q[0], q[1], q[2], q[3]), qf[n % NB], f32x4{0.f, 0.f, 0.f, 0.f});
          __builtin_amdgcn_sched_barrier(0);
        }
        if (n > 0) {
          const int i = (n - 1) / NB, b = (n - 1) % NB;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[0][4 * (i0 + i) + r] = fmaf(scale_of(ks[i], b, r), d[(n - 1) & 1][r], b ? s[0][4 * (i0 + i) + r] : 0.f);
        }
      }
    }
    uint32_t vq[2][NB];  // read before the softmax
    if (kTiles == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i) read_quants<NB>(at + i * kTile + kHalf, lane, vq[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) read_scales<NB>(at + i * kTile + kHalf + kQuant, g, vs[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (SPLIT) {  // hi and lo columns of one query
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0][i] += row_swap8(s[0][i]);
    }
    if (mask) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
        s[0][i] = tok >= lo && tok < hi ? s[0][i] : -INFINITY;
      }
    }
    bool odd;
    const uint32_t bits = scale_bits<NB>(vs, mask, any_lo, any_hi, t0, g, odd);
    const float qs1[1] = {qs};
    weigh<NB, 1>(s, qs1, vs, bits, g, st);
    const float (&p)[8] = s[0];
    if (kTiles == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) read_quants<NB>(at + i * kTile + kHalf, lane, vq[i]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f16x8 w;
      if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = weight(p[i], odd_scale(vs[i >> 2], b, i, t0, g, lo, hi), second);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = weight(p[i], scale_of(vs[i >> 2], b, i & 3), second);
      }
      uint32_t n0[4], n1[4];
      unpack(uk, vq[0][b], n0);
      unpack(uk, vq[1][b], n1);
      st.o[0][2 * b] = mfma(w, join(n0[0], n0[1], n1[0], n1[1]), st.o[0][2 * b]);
      st.o[0][2 * b + 1] = mfma(w, join(n0[2], n0[3], n1[2], n1[3]), st.o[0][2 * b + 1]);
    }
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
    State<NB, 1> st;
    st.clear();
    // the tile's own steps: the item's units are spread over them (a tile of early tokens has fewer)
    const int s0 = any_lo / 32, n = max(0, (any_hi + 31) / 32 - s0);
    StepBack back{done, share_units, kWaves};
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
      const int e = query_exponent(most);
      qs = query_scale(a.scale, e);
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
      back.at(i);
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
    st.l[0] += __shfl_xor(st.l[0], 16);
    st.l[0] += __shfl_xor(st.l[0], 32);
    float *lm = (float *)lds, *ll = lm + kWaves * NCOL, *lo_ = lm + 2 * kWaves * NCOL;
    __syncthreads();
    if ((id & 63) < NCOL) {
      lm[wave * NCOL + l16] = st.m[0];
      ll[wave * NCOL + l16] = st.l[0];
    }
    constexpr int kRun = 32 * kMergeBlocks;
#pragma unroll
    for (int b0 = 0; b0 < NB; b0 += kMergeBlocks) {
      if (b0) __syncthreads();
#pragma unroll
      for (int j = 0; j < 2 * kMergeBlocks; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v = st.o[0][2 * b0 + j][r];
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
          store_out<A>(a, q.row0 + cs.tok0, cs.head0, cs.per, c, 32 * b0 + d, l == 0.f ? 0.f : o / l);
          if (b0 == 0 && d == 0) store_lse(a, q.row0 + cs.tok0, cs.head0, cs.per, c, m, l);
        }
      }
    }
    __syncthreads();  // the next segment's fetches go where these sums were
  }
};

// ---- many columns: waves share an item's keys and values -----------------------------------------

// A workgroup takes 64 CT query columns, 16 CT a wave. Each wave unpacks a quarter of a step (one
// tile of keys or of values) into LDS in the matrix cores' operand layout, so a nibble is unpacked
// once for 64 CT columns, and all waves read all of it. Two stages and one barrier a step: behind it,
// a wave unpacks its part of the next step, asks for the raw quants of the second after it, and multiplies.
// Bound by vector issue, so the values' scales are applied where it costs least: for bf16
// activations to the values, once, as they are unpacked (rounded to fp16, 2^-12 of a value, against
// 2^-9 in the output; a tile's values are brought to [0, 8) by a power of two, which the softmax
// weights take up); for fp32 and fp16 to the weights, which then enter as two fp16 terms.
template <typename A, int NB, bool SPLIT>
struct Wide {
  typedef A Act;
  typedef typename A::type T;
  static constexpr bool kWide = true;
  static constexpr int CT = wide_tiles(sizeof(T) == 4, NB);
  static constexpr int NCOL = kWaves * 16 * CT;
  static constexpr int D = 32 * NB;
  static constexpr int kPart = NCOL * (D + 2);
  static constexpr int kQueryTerms = sizeof(T) == 4 ? 2 : 1;  // fp16 and bf16 queries are one term
  // offsets in a stage: key operands, value operands, scales, then what Header holds
  static constexpr int kValues = 2048 * NB, kScales = 4096 * NB, kHeader = 4224 * NB;
  static constexpr int kStage = kHeader + 128;
  static constexpr int kLds = 2 * kStage;

  struct Header {  // of a step's two tiles
    int exponent[2][4];   // the values of tokens 4 g + 0..3 are stored times 2^-exponent
    uint32_t odd[2][4];   // a scale among them is no number
    uint32_t no_page[2];  // the tile's page is outside the cache
  };

  struct Raw {
    uint32_t q[NB], s[2 * NB];  // the lane's share of a tile's key or value quants, its tokens' scales
    uint32_t no_page;
  };

  static __device__ __forceinline__ void load(const uint8_t *p, int lane, Raw &r) {
    typedef __attribute__((address_space(1))) const u32x2 *g2;
    typedef __attribute__((address_space(1))) const u32x3a4 *g3;
    if constexpr (NB == 2) {
      const u32x2 w = *(g2)(p + lane * 8);
      r.q[0] = w[0];
      r.q[1] = w[1];
    } else if constexpr (NB == 3) {
      const u32x3a4 w = *(g3)(p + lane * 12);
#pragma unroll
      for (int i = 0; i < 3; ++i) r.q[i] = w[i];
    } else {
#pragma unroll
      for (int c = 0; c < NB / 4; ++c) {
        const u32x4 w = gload(p + c * 1024 + lane * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.q[4 * c + i] = w[i];
      }
    }
    p += 256 * NB + (lane >> 4) * 8 * NB;
    if constexpr (NB % 2 == 0) {
#pragma unroll
      for (int c = 0; c < NB / 2; ++c) {
        const u32x4 w = gload(p + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.s[4 * c + i] = w[i];
      }
    } else {
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        const u32x2 w = *(g2)(p + 8 * c);
        r.s[2 * c] = w[0];
        r.s[2 * c + 1] = w[1];
      }
    }
  }

  // Tile i of the step as operands into a stage.
  static __device__ __forceinline__ void unpack_into(uint8_t *stage, bool values, int i, int lane, const Raw &r) {
    const Unpack uk;
    const int g = lane >> 4;
    Header *head = (Header *)(stage + kHeader);
    if ((lane & 15) == 0) {
      uint8_t *to = stage + kScales + ((values ? 2 : 0) + i) * 32 * NB + g * 8 * NB;
#pragma unroll
      for (int c = 0; c < NB; ++c) *(u32x2 *)(to + 8 * c) = u32x2{r.s[2 * c], r.s[2 * c + 1]};
    }
    if (!values) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t n[4];
        unpack(uk, r.q[b], n);
        *(u32x4 *)(stage + (i * NB + b) * 1024 + lane * 16) = u32x4{n[0], n[1], n[2], n[3]};
      }
      if (lane == 0) head->no_page[i] = r.no_page;
      return;
    }
    f16x2 d[2 * NB];
    if constexpr (!SPLIT) {
      typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
      uint32_t raw[2 * NB];
      auto exponent = [&]() {
        u16x2 most = {0, 0};
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
          most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, raw[j] & 0x7C007C00u));
        return max((int)most[0], (int)most[1]) >> 10;
      };
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) raw[j] = r.s[j];
      int top = exponent();
      const bool odd = top == 31;
      if (__any(odd)) {  // not numbers as 0 here, and the columns that see them afterwards: see_odd()
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
          if ((raw[j] & 0x7C00u) == 0x7C00u) raw[j] &= 0xFFFF0000u;
          if ((raw[j] & 0x7C000000u) == 0x7C000000u) raw[j] &= 0x0000FFFFu;
        }
        top = exponent();
      }
      const int e = top - 14;  // scales below 2^e, e -14 .. 16
      const _Float16 f = (_Float16)ldexpf(1.f, -e);
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) d[j] = __builtin_bit_cast(f16x2, raw[j]) * f16x2{f, f};
      if ((lane & 15) == 0) {
        head->odd[i][g] = odd;
        head->exponent[i][g] = e;
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t n[4];
      unpack(uk, r.q[b], n);
      if constexpr (!SPLIT) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          n[k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, n[k]) * d[2 * b + (k & 1)]);
      }
      uint8_t *v = stage + kValues + 2 * b * 1024 + lane * 16 + 8 * i;
      *(u32x2 *)v = u32x2{n[0], n[1]};
      *(u32x2 *)(v + 1024) = u32x2{n[2], n[3]};
    }
  }

  template <typename F>
  static __device__ __forceinline__ void weights(const float (&p)[8], F scale, f16x8 &w0, f16x8 &w1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = scale(i);
      float x = fmaf(p[i], d, 0.f);
      if constexpr (SPLIT) {
        asm("" : "+v"(x));  // both terms from one fp32 value
        w0[i] = (_Float16)x;
        w1[i] = (_Float16)(x - (float)w0[i]);
      } else {
        w0[i] = (_Float16)x;
      }
    }
  }

  static __device__ __forceinline__ void step(const uint8_t *stage, const f16x8 (&qf)[CT][kQueryTerms][NB],
                                              const float (&qs)[CT], bool mask, const int (&lo)[CT],
                                              const int (&hi)[CT], int any_lo, int any_hi, int t0, int lane,
                                              State<NB, CT> &st, int (&odd)[CT]) {
    const int g = lane >> 4;
    float s[CT][8];
    // Software pipeline, kept by the scheduling barriers (left alone, the compiler reads, waits,
    // multiplies and waits again, operand by operand): the operands of kRead products ahead are
    // read, and a product's results are scaled while the next ones are multiplied.
    constexpr int kProducts = 2 * NB, kRead = kQueryTerms == 2 ? 2 : 4;
    uint32_t ks[2][2 * NB];
    f16x8 k[kProducts];
    f32x4 d[2][CT];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_scales<NB>(stage + kScales + i * 32 * NB, g, ks[i]);
#pragma unroll
    for (int n = 0; n < kRead; ++n) k[n] = *(const f16x8 *)(stage + n * 1024 + lane * 16);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n <= kProducts; ++n) {  // product n: tile n / NB, block n % NB
      if (n < kProducts) {
        if (n + kRead < kProducts) k[n + kRead] = *(const f16x8 *)(stage + (n + kRead) * 1024 + lane * 16);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          d[n & 1][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int t = kQueryTerms - 1; t >= 0; --t) d[n & 1][c] = mfma(k[n], qf[c][t][n % NB], d[n & 1][c]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (n > 0) {
        const int i = (n - 1) / NB, b = (n - 1) % NB;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[c][4 * i + r] = fmaf(scale_of(ks[i], b, r), d[(n - 1) & 1][c][r], b ? s[c][4 * i + r] : 0.f);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (mask) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
          s[c][i] = tok >= lo[c] && tok < hi[c] ? s[c][i] : -INFINITY;
        }
    }
    if constexpr (SPLIT) scaled_weights(stage, s, qs, mask, lo, hi, any_lo, any_hi, t0, lane, st);
    else scaled_values(stage, s, qs, mask, lo, hi, t0, lane, st, odd);
  }

  static __device__ __forceinline__ void scaled_weights(const uint8_t *stage, float (&s)[CT][8], const float (&qs)[CT],
                                                        bool mask, const int (&lo)[CT], const int (&hi)[CT],
                                                        int any_lo, int any_hi, int t0, int lane, State<NB, CT> &st) {
    const int g = lane >> 4;
    uint32_t vs[2][2 * NB];
#pragma unroll
    for (int i = 0; i < 2; ++i) read_scales<NB>(stage + kScales + (2 + i) * 32 * NB, g, vs[i]);
    bool odd;
    const uint32_t bits = scale_bits<NB>(vs, mask, any_lo, any_hi, t0, g, odd);
    weigh<NB, CT>(s, qs, vs, bits, g, st);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const f16x8 v0 = *(const f16x8 *)(stage + kValues + 2 * b * 1024 + lane * 16);
      const f16x8 v1 = *(const f16x8 *)(stage + kValues + (2 * b + 1) * 1024 + lane * 16);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        f16x8 w0, w1;
        if (odd) weights(s[c], [&](int i) { return odd_scale(vs[i >> 2], b, i, t0, g, lo[c], hi[c]); }, w0, w1);
        else weights(s[c], [&](int i) { return scale_of(vs[i >> 2], b, i & 3); }, w0, w1);
        st.o[c][2 * b] = mfma(w0, v0, st.o[c][2 * b]);
        st.o[c][2 * b + 1] = mfma(w0, v1, st.o[c][2 * b + 1]);
        if constexpr (SPLIT) {
          st.o[c][2 * b] = mfma(w1, v0, st.o[c][2 * b]);
          st.o[c][2 * b + 1] = mfma(w1, v1, st.o[c][2 * b + 1]);
        }
      }
    }
  }

  // Weights p = 2^(s - m + e) for values times 2^-e: m is moved where a weight would pass 2^15 and then
  // set so that the largest is 2^8 (see weigh()); the sums take p 2^-e.
  static __device__ __forceinline__ void scaled_values(const uint8_t *stage, float (&s)[CT][8], const float (&qs)[CT],
                                                       bool mask, const int (&lo)[CT], const int (&hi)[CT], int t0,
                                                       int lane, State<NB, CT> &st, int (&odd)[CT]) {
    const int g = lane >> 4;
    const Header *head = (const Header *)(stage + kHeader);
    f16x8 v[2 * NB];  // read before the softmax
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) v[j] = *(const f16x8 *)(stage + kValues + j * 1024 + lane * 16);
    const float e[2] = {(float)head->exponent[0][g], (float)head->exponent[1][g]};
    __builtin_amdgcn_sched_barrier(0);
    const float back[2] = {__builtin_amdgcn_exp2f(-e[0]), __builtin_amdgcn_exp2f(-e[1])};
    bool move = false;
    float want[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      float mx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mx[i] = fmaf(fmaxf(fmaxf(s[c][4 * i], s[c][4 * i + 1]), fmaxf(s[c][4 * i + 2], s[c][4 * i + 3])), qs[c], e[i]);
      want[c] = fmaxf(mx[0], mx[1]) - 8.f;
      move |= want[c] > st.m[c] + 7.f;
    }
    if (__any(move)) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        float w = fmaxf(want[c], __shfl_xor(want[c], 16));
        w = fmaxf(w, __shfl_xor(w, 32));
        const float m = fmaxf(st.m[c], w);
        const float alpha = __builtin_amdgcn_exp2f(st.m[c] - m);
        st.m[c] = m;
        st.l[c] *= alpha;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float f = __shfl(alpha, 4 * g + r);
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j) st.o[c][j][r] *= f;
        }
      }
    }
    f16x8 w[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const float off[2] = {e[0] - st.m[c], e[1] - st.m[c]};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[c][i], qs[c], off[i >> 2]));
        st.l[c] = fmaf(p, back[i >> 2], st.l[c]);
        w[c][i] = (_Float16)p;
      }
    }
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
      for (int c = 0; c < CT; ++c) st.o[c][j] = mfma(w[c], v[j], st.o[c][j]);
    if (__any(head->odd[0][g] | head->odd[1][g])) see_odd(stage, mask, lo, hi, t0, g, odd);
  }

  // Bit b of odd[c]: the lane's column sees one of the lane's tokens whose block b has a scale that is no
  // number (its values entered as 0; finish() makes the column's outputs of the block no numbers).
  static __device__ __forceinline__ void see_odd(const uint8_t *stage, bool mask, const int (&lo)[CT],
                                                 const int (&hi)[CT], int t0, int g, int (&odd)[CT]) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
      const uint8_t *scales = stage + kScales + (2 + (i >> 2)) * 32 * NB + g * 8 * NB + 2 * (i & 3);
      int bits = 0;
      for (int b = 0; b < NB; ++b) bits |= (*(const uint16_t *)(scales + 8 * b) & 0x7C00u) == 0x7C00u ? 1 << b : 0;
#pragma unroll
      for (int c = 0; c < CT; ++c) odd[c] |= !mask || (tok >= lo[c] && tok < hi[c]) ? bits : 0;
    }
  }

  // The units [v0, v1) of an item, by the whole workgroup.
  static __device__ void segment(const AttnArgs &a, const TileShape &ts, const Request &q, int kvh, int tile,
                                 int v0, int v1, int done, int share_units, float *part, uint8_t *lds) {
    StepBack back{done, share_units, 1};
    const int lane = threadIdx.x & 63, wave = wave_index(), g = lane >> 4;
    const Columns cs = columns<NCOL>(a, ts, q, kvh, tile);
    const int last_tok = cs.tok0 + (cs.count - 1) / cs.per;
    const int any_lo = seen_from(a, q.first_pos + cs.tok0), any_hi = max(q.first_pos + last_tok + 1, 0);
    // this wave's columns (none: it unpacks only), and what they see: all together, and each
    const int c0 = wave * 16 * CT, mine = min(cs.count - c0, 16 * CT);
    const int tok_a = cs.tok0 + min(c0, cs.count - 1) / cs.per;
    const int tok_b = cs.tok0 + (min(c0 + 16 * CT, cs.count) - 1) / cs.per;
    const int mine_lo = seen_from(a, q.first_pos + tok_a), mine_hi = max(q.first_pos + tok_b + 1, 0);
    const int all_lo = seen_from(a, q.first_pos + tok_b), all_hi = max(q.first_pos + tok_a + 1, 0);
    const int s0 = any_lo / 32, n = max(0, (any_hi + 31) / 32 - s0);
    const double share = (double)n / (double)q.units;
    auto step_at = [&](int v) { return s0 + (v == q.units ? n : (int)(v * share)); };
    const int from = step_at(v0), steps = step_at(v1) - from;
    const int32_t *table = a.block_table + (int64_t)q.r * a.max_blocks;
    const int last_block = ((q.len + a.g.page_tokens - 1) >> a.g.page_shift) - 1;
    const unsigned pages = (unsigned)a.g.pages;
    const bool values = wave >= 2;
    const int half = wave & 1;  // the tile of a step that this wave unpacks
    const uint8_t *head_data = a.g.data + (int64_t)kvh * a.g.head_bytes + (values ? a.g.half_bytes : 0);
    auto page_of = [&](int t) {
      typedef __attribute__((address_space(4))) const int32_t *scalar;
      return ((scalar)(uintptr_t)table)[__builtin_amdgcn_readfirstlane(min(t >> a.g.page_shift, last_block))];
    };
    auto token_of = [&](int i) { return 32 * (from + min(i, steps - 1)) + 16 * half; };  // past the end the last again
    Raw raw0, raw1;
    int next_page = 0;
    auto fetch = [&](int i, Raw &raw) {
      const int t = token_of(i), page = next_page;
      next_page = page_of(token_of(i + 1));
      const int64_t ok = (unsigned)page < pages ? page : 0;
      raw.no_page = (unsigned)page >= pages;
      load(head_data + ok * a.g.page_bytes + (int64_t)((t & (a.g.page_tokens - 1)) >> 4) * a.g.tile_bytes, lane, raw);
    };
    if (steps > 0) {
      next_page = page_of(token_of(0));
      fetch(0, raw0);
      fetch(1, raw1);
    }
    f16x8 qf[CT][kQueryTerms][NB];
    float qs[CT];
    int lo[CT], hi[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int col = min(c0 + 16 * c + (lane & 15), cs.count - 1);
      const int tok = cs.tok0 + col / cs.per, head = cs.head0 + col % cs.per, pos = q.first_pos + tok;
      lo[c] = seen_from(a, pos);
      hi[c] = max(pos + 1, 0);
      const T *qp = (const T *)a.q.data + (int64_t)(q.row0 + tok) * a.q.row_stride + (int64_t)head * a.q.head_stride;
      // read twice rather than kept: the values beside everything else would spill
      auto element = [&](int b, int i) { return A::load(qp + 32 * b + 4 * g + (i & 3) + 16 * (i >> 2)); };
      float most = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(element(b, i)));
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
      const int e = query_exponent(most);
      qs[c] = query_scale(a.scale, e);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = ldexpf(element(b, i), e);
          const _Float16 h = (_Float16)x;
          qf[c][0][b][i] = h;
          if constexpr (kQueryTerms == 2) qf[c][1][b][i] = (_Float16)(x - (float)h);
        }
      }
    }
    State<NB, CT> st;
    st.clear();
    int odd[CT] = {};
    if (steps > 0) {
      unpack_into(lds, values, half, lane, raw0);
      fetch(2, raw0);
    }
    auto turn = [&](int i, Raw &raw) {  // raw: of step i + 1
      back.at(i);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      uint8_t *stage = lds + (i & 1) * kStage;
      if (i + 1 < steps) {
        unpack_into(lds + kStage - (i & 1) * kStage, values, half, lane, raw);
        fetch(i + 3, raw);
      }
      const int t0 = 32 * (from + i);
      if (mine <= 0 || t0 >= mine_hi || t0 + 32 <= mine_lo) return;
      const Header *head = (const Header *)(stage + kHeader);
      const bool bad0 = __builtin_amdgcn_readfirstlane(head->no_page[0]), bad1 = __builtin_amdgcn_readfirstlane(head->no_page[1]);
      const bool inner = t0 >= all_lo && t0 + 32 <= all_hi && !bad0 && !bad1;
      const int l0 = bad0 ? t0 + 16 : 0, h0 = bad1 ? t0 + 16 : 0x7FFFFFFF;
      int lo1[CT], hi1[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        lo1[c] = max(lo[c], l0);
        hi1[c] = min(hi[c], h0);
      }
      step(stage, qf, qs, !inner, lo1, hi1, max(mine_lo, l0), min(mine_hi, h0), t0, lane, st, odd);
    };
    for (int i = 0; i < steps; i += 2) {
      turn(i, raw1);
      if (i + 1 < steps) turn(i + 1, raw0);
    }
    const int l16 = lane & 15;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      float l = st.l[c];
      l += __shfl_xor(l, 16);
      l += __shfl_xor(l, 32);
      int nan_blocks = odd[c] | __shfl_xor(odd[c], 16);
      nan_blocks |= __shfl_xor(nan_blocks, 32);
      const int own = c0 + 16 * c + l16;
      if (g == 0 && own < cs.count) {
        if (part) {
          part[own] = st.m[c];
          part[NCOL + own] = l;
        } else {
          store_lse(a, q.row0 + cs.tok0, cs.head0, cs.per, own, st.m[c], l);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float sum = __shfl(l, 4 * g + r), inv = sum == 0.f ? 0.f : 1.f / sum;
        const int col = c0 + 16 * c + 4 * g + r, nans = __shfl(nan_blocks, 4 * g + r);
        if (col >= cs.count) continue;
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
          const float v = nans >> (j >> 1) & 1 ? NAN : st.o[c][j][r];
          if (part) part[2 * NCOL + col * D + 16 * j + l16] = v;
          else store_out<A>(a, q.row0 + cs.tok0, cs.head0, cs.per, col, 16 * j + l16, v * inv);
        }
      }
    }
    __syncthreads();  // the next segment's first steps go where this one's last may still be read
  }
};

// What k_kv_join needs of the item whose first part a workgroup left (parts 0: none).
struct JoinItem {
  int parts, row, head0, per, count;
};

// Workgroup w takes the units [w per, (w + 1) per) of the class's items. Items that it holds whole
// are finished here; of the others, at most one begun before its share (part 2 w) and one that ends
// behind it (part 2 w + 1), it leaves partial results for k_kv_join.
template <typename X>
__device__ __forceinline__ void take_share(AttnArgs &a, uint8_t *lds) {
  const TileShape ts = tile_shape<X::NCOL>(a.group);
  // neighbouring shares on one XCD: query tiles of one request read the same keys through one L2
  const int w = a.grid % 8 ? (int)blockIdx.x : (int)(blockIdx.x % 8 * (a.grid / 8) + blockIdx.x / 8);
  const Place pl = locate<X::kWide>(a, ts, [&](int64_t per) { return w * per; });
  JoinItem join = {0, 0, 0, 0, 0};
  int64_t u = w * pl.per;
  const int64_t end = pl.r < 0 ? u : min(pl.total, u + pl.per);
  Request q = request<X::kWide>(a, ts, max(pl.r, 0));
  int64_t base = pl.base;
  while (u < end) {
    int64_t in = u - base;
    while (in >= units_of(a, q)) {  // on to the next request (some have no units)
      base += units_of(a, q);
      q = request<X::kWide>(a, ts, q.r + 1);
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
    X::segment(a, ts, q, kvh, tile, v0, v1, (int)min(u - w * pl.per, (int64_t)1 << 28),
               (int)min(pl.per, (int64_t)1 << 28), part, lds);
    u += v1 - v0;
  }
  if (threadIdx.x == 0) ((JoinItem *)a.joins)[w] = join;
}

// Bound by HBM (1.125 bytes per key and value element pair) and, close to it, by vector issue: 64
// requests to 8192 tokens, 64 + 8 heads of 128, bf16: 75 us, 4.0 TB/s, vector issue 0.6 of the time;
// one request of 131072 tokens fp16, whose weights are two terms: 50 us, 3.0 TB/s. Below some 100000
// (token, kv head) pairs bound by latency: 4096 tokens of 8 heads fp32 13.6 us.
template <typename A, int NB, bool SPLIT>
__global__ __launch_bounds__(kThreads, resident(NB)) void k_kv_attn(AttnArgs a) {
  extern __shared__ __align__(16) uint8_t attn_lds[];
  take_share<Attn<A, NB, SPLIT>>(a, attn_lds);
}

// Bound by vector issue and the waits between it: four pieces of 1024 tokens over up to 8192, 32 + 8
// heads of 128, bf16, take 515 to 540 us, 0.5 PFLOP/s; of a wave's 290 vector instructions a step 32
// are matrix products; issue takes half of the time, the matrix cores are busy for a fifth.
template <typename A, int NB, bool SPLIT>
__global__ __launch_bounds__(kThreads, resident_wide(NB)) void k_kv_wide(AttnArgs a) {
  extern __shared__ __align__(16) uint8_t attn_lds[];
  take_share<Wide<A, NB, SPLIT>>(a, attn_lds);
}

// Workgroup (w, y) joins the item whose first part workgroup w of k_kv_attn left: part 2 w + 1 and
// the parts 2 w' of the following workgroups. A thread takes four dimensions of a column and, of
// k_kv_attn's parts (up to hundreds of a long sequence), every fourth; k_kv_wide's items have few
// parts. Bound by latency: the parts' references, sums and outputs are read eight parts at a time,
// at once (64 requests 5 us, the 768 parts of one long sequence 6 us).
constexpr int kJoinThreads = 512;

template <typename X>
__global__ __launch_bounds__(kJoinThreads) void k_kv_join(AttnArgs a) {
  constexpr int kJoinGroups = X::kWide ? 1 : 4, kJoinUnits = kJoinThreads / kJoinGroups;
  constexpr int kRuns = X::D / 4, kBatch = 8;
  __shared__ f32x4 other_o[kJoinGroups][kJoinUnits];
  __shared__ float other_m[kJoinGroups][kJoinUnits], other_l[kJoinGroups][kJoinUnits];
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
  if constexpr (kJoinGroups > 1) {
    if (group > 0) {
      other_m[group][unit] = m;
      other_l[group][unit] = l;
      other_o[group][unit] = o;
    }
    __syncthreads();
  }
  if (group > 0 || !live) return;
#pragma unroll
  for (int k = 1; k < kJoinGroups; ++k) join(other_m[k][unit], other_l[k][unit], other_o[k][unit]);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    store_out<typename X::Act>(a, item.row, item.head0, item.per, c, d + j, l == 0.f ? 0.f : o[j] / l);
  if (d == 0) store_lse(a, item.row, item.head0, item.per, c, m, l);
}

// The kernel `K` over X's items with `grid` workgroups, then their join.
template <typename X, void (*K)(AttnArgs)>
int launch_class(const AttnArgs &args, int grid, hipStream_t s) {
  AttnArgs a = args;
  a.grid = grid;
  a.joins = a.parts + (int64_t)grid * 2 * X::kPart;
  if (X::kLds > 64 * 1024) {  // once a device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return -1;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
      if (hipFuncSetAttribute(reinterpret_cast<const void *>(K), hipFuncAttributeMaxDynamicSharedMemorySize,
                              X::kLds) != hipSuccess)
        return -1;
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  K<<<dim3(grid), kThreads, X::kLds, s>>>(a);
  constexpr int kThreadsOfItem = X::NCOL * X::D / 4 * (X::kWide ? 1 : 4);
  if (grid > 1)
    k_kv_join<X><<<dim3(grid - 1, (kThreadsOfItem + kJoinThreads - 1) / kJoinThreads), kJoinThreads, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename A, int NB, bool SPLIT>
int launch(const AttnArgs &args, hipStream_t s) {
  AttnArgs a = args;
  const bool wide = wide_launch(a.group, a.rows, a.requests);
  a.wide_cols = wide ? kWideCols : INT32_MAX;
  if (wide) {
    const int rc = launch_class<Wide<A, NB, SPLIT>, k_kv_wide<A, NB, SPLIT>>(a, kComputeUnits * resident_wide(NB), s);
    if (rc) return rc;
  }
  return launch_class<Attn<A, NB, SPLIT>, k_kv_attn<A, NB, SPLIT>>(a, a.grid, s);
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

}  // namespace

size_t kv_attention_workspace(int type, int64_t head_dim, int64_t group, int64_t rows, int64_t requests, int grid) {
  auto bytes = [&](int64_t workgroups, int64_t columns) {
    return (size_t)(workgroups * (2 * columns * (head_dim + 2) * 4 + (int64_t)sizeof(JoinItem)));
  };
  const size_t few = bytes(grid, split_type(type) ? 8 : 16);
  const int nb = (int)(head_dim / 32), columns = kWaves * 16 * wide_tiles(type == TQ_F32, nb);
  const size_t many = wide_launch(group, rows, requests) ? bytes(kComputeUnits * resident_wide(nb), columns) : 0;
  return few > many ? few : many;
}

int kv_attention_grid(int type, int64_t kv_heads, int64_t head_dim, int64_t group, int64_t rows, int64_t max_len) {
  // an upper bound of the units: every row a tile of its own over the longest sequence
  const int64_t ncol = split_type(type) ? 8 : 16;
  const int64_t tiles = rows * (group <= ncol ? 1 : (group + ncol - 1) / ncol);
  const int64_t steps = max_len / 32 + 2 + item_units(false);
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
