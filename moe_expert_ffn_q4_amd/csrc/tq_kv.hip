// tq_kv.hip -- the step plan, the append and the read-back of the paged 4-bit key/value cache.
#include "tq_kv.h"
#include "tq_kv_device.h"
#include "tq_launch.h"

namespace tq {

namespace {

constexpr int kThreads = 256;

int launch_status() { return hipGetLastError() == hipSuccess ? 0 : -1; }

// ---- plan -----------------------------------------------------------------------------------

// Index of the run that holds i: off[0] <= ... <= off[n], off[r] <= i < off[r + 1].
__device__ __forceinline__ int run_of(const int32_t *off, int n, int i) {
  int lo = 0, hi = n;  // first index > i lies in (lo, hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Prefix sums over the requests of new tokens, needed pages and released pages; then every row,
// needed page and released page finds its request by bisection. Bound by latency (two dependent
// reads, the scan's barriers, the bisection: 4.2 us for 8 requests, 9.8 us for 512 and 16384 rows):
// each workgroup repeats the scan of at most 4096 requests from L2 rather than wait for another
// one's, so a step is a single launch. Nothing reads what another workgroup of the launch writes:
// pages on the stack above free_count are read from the ended requests' table rows, which the launch
// leaves alone.
__global__ __launch_bounds__(kThreads) void k_kv_plan(PlanArgs a) {
  extern __shared__ int32_t plan_lds[];
  __shared__ int64_t wave_sum[3][kThreads / 64];
  __shared__ int bad_lds;
  const int R = a.requests, tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  int32_t *cu = plan_lds, *need = cu + R + 1, *rel = need + R + 1;
  const int P = 1 << a.page_shift;
  const bool managed = a.free_pages != nullptr;
  if (tid == 0) bad_lds = 0;
  const int per = (R + kThreads - 1) / kThreads, r0 = min(R, tid * per), r1 = min(R, r0 + per);
  int64_t s[3] = {0, 0, 0};
  int bad = 0;
  auto request = [&](int r, int64_t v[3]) {
    const int kv = a.kv_len[r], nw = a.new_len[r];
    v[0] = v[1] = v[2] = 0;
    if (kv < 0 || nw < -1) {
      bad |= 8;
      return;
    }
    const int64_t have = ((int64_t)kv + P - 1) >> a.page_shift;
    const int64_t after = ((int64_t)kv + max(nw, 0) + P - 1) >> a.page_shift;
    if (after > a.max_blocks) bad |= 4;
    if (nw < 0) {
      v[2] = managed ? have : 0;
    } else {
      v[0] = nw;
      v[1] = managed ? after - have : 0;
    }
  };
  for (int r = r0; r < r1; ++r) {
    int64_t v[3];
    request(r, v);
    for (int i = 0; i < 3; ++i) s[i] += v[i];
  }
  int64_t incl[3];
  for (int i = 0; i < 3; ++i) {
    int64_t x = s[i];
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    incl[i] = x;
    if (lane == 63) wave_sum[i][wave] = x;
  }
  __syncthreads();
  int64_t total[3], base[3];
  for (int i = 0; i < 3; ++i) {
    total[i] = 0;
    base[i] = incl[i] - s[i];
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) base[i] += wave_sum[i][w];
      total[i] += wave_sum[i][w];
    }
  }
  const int64_t fc = managed ? a.free_count[0] : 0;
  if (managed && (fc < 0 || fc > a.pages || fc + total[2] > a.pages)) bad |= 8;
  else if (managed && total[1] > fc + total[2]) bad |= 1;
  if (total[0] > a.rows) bad |= 2;
  if (bad) atomicOr(&bad_lds, bad);
  __syncthreads();
  bad = bad_lds;
  const int first = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
  if (first == 0) {
    a.status[0] = bad;
    if (a.free_count_out) a.free_count_out[0] = (int32_t)(bad ? (managed ? a.free_count[0] : 0) : fc + total[2] - total[1]);
  }
  if (bad) {
    for (int r = first; r <= R; r += step) {
      a.cu_new[r] = 0;
      if (r < R) a.seq_len[r] = max(a.kv_len[r], 0);
    }
    for (int t = first; t < a.rows; t += step) a.slots[t] = a.positions[t] = a.requests_of[t] = -1;
    return;
  }
  for (int r = r0; r < r1; ++r) {
    cu[r] = (int32_t)base[0];
    need[r] = (int32_t)base[1];
    rel[r] = (int32_t)base[2];
    int64_t v[3];
    request(r, v);
    for (int i = 0; i < 3; ++i) base[i] += v[i];
  }
  if (tid == 0) {
    cu[R] = (int32_t)total[0];
    need[R] = (int32_t)total[1];
    rel[R] = (int32_t)total[2];
  }
  __syncthreads();
  auto have_of = [&](int r) { return (int)(((int64_t)a.kv_len[r] + P - 1) >> a.page_shift); };
  auto stack = [&](int i) -> int32_t {  // 0 <= i < fc + total[2]
    if (i < fc) return a.free_pages[i];
    i -= (int)fc;
    const int r = run_of(rel, R, i);
    return a.block_table[(int64_t)r * a.max_blocks + (i - rel[r])];
  };
  const int top = (int)(fc + total[2]);
  for (int r = first; r <= R; r += step) {
    a.cu_new[r] = cu[r];
    if (r < R) {
      const int nw = a.new_len[r];
      a.seq_len[r] = nw < 0 ? 0 : a.kv_len[r] + nw;
    }
  }
  for (int t = first; t < a.rows; t += step) {
    int slot = -1, pos = -1, r = -1;
    if (t < cu[R]) {
      r = run_of(cu, R, t);
      const int kv = a.kv_len[r];
      pos = kv + (t - cu[r]);
      const int col = pos >> a.page_shift, have = (int)(((int64_t)kv + P - 1) >> a.page_shift);
      const int32_t page = managed && col >= have ? stack(top - 1 - (need[r] + col - have))
                                                  : a.block_table[(int64_t)r * a.max_blocks + col];
      if (page >= 0 && page < a.pages) slot = (page << a.page_shift) + (pos & (P - 1));
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
    a.requests_of[t] = r;
  }
  for (int j = first; j < need[R]; j += step) {
    const int r = run_of(need, R, j);
    a.block_table[(int64_t)r * a.max_blocks + have_of(r) + (j - need[r])] = stack(top - 1 - j);
  }
  for (int j = first; j < rel[R]; j += step) a.free_pages[fc + j] = stack((int)fc + j);
}

// ---- append ---------------------------------------------------------------------------------

// v of the lane N to the right within its row of 16 (rotating), without LDS.
template <int N>
__device__ __forceinline__ float row_rotate(float v) {
  const int i = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, 0x120 + N, 0xF, 0xF, false));
}
// v of lane ^ N (1 or 2).
template <int N>
__device__ __forceinline__ uint32_t quad_swap(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, N == 1 ? 0xB1 : 0x4E, 0xF, 0xF, false);
}

// W pairs of a head turned by cosine and sine t[0..W): runs e0 and e1 of W elements each; interleaved:
// the runs follow each other and hold the pairs side by side. In T's arithmetic.
template <typename F, typename C, int W>
__device__ __forceinline__ void turn_pairs(F (&lo)[W], F (&hi)[W], const C *t, bool interleaved) {
  if (interleaved) {
    F v[2 * W];
#pragma unroll
    for (int k = 0; k < 2 * W; ++k) v[k] = k < W ? lo[k] : hi[k - W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const F x0 = v[2 * k], x1 = v[2 * k + 1], c = t[k].x, s = t[k].y;
      v[2 * k] = x0 * c - x1 * s;
      v[2 * k + 1] = x0 * s + x1 * c;
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
      lo[k] = v[k];
      hi[k] = v[W + k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const F x0 = lo[k], x1 = hi[k], c = t[k].x, s = t[k].y;
      lo[k] = x0 * c - x1 * s;
      hi[k] = x0 * s + x1 * c;
    }
  }
}

// One workgroup: `rb` rows x `hg` kv heads (and their share of the q heads). The rows' sines and
// cosines are formed once per workgroup in fp64 (an fp32 angle is off by 0.03 rad at position
// 500000) and kept in LDS. Keys are turned in fp64 and rounded to fp32 once, so that the 4-bit
// rounding that follows is the definition's; queries, of which there are several times as many, are
// turned in fp32 (fp64 conversions and products took half of the kernel's time: 120 us for 8192 rows
// of 64 + 16 heads). q heads go from global memory to global memory, k and v heads into LDS as fp32,
// from where sixteen lanes round a block of 32 (lane c holds its values c and c + 16, the two
// nibbles of one byte). W pairs are turned per thread step, 16 bytes of a run where the rows allow.
// 8192 rows bf16, 64 + 16 heads of 128: 77 us, 4.0 TB/s of 311 MB; vector issue takes half of it and
// the waves wait for memory and at the two barriers for most of the rest. One row: 6 us, of latency.
template <typename A, int W, int NB>
__global__ __launch_bounds__(kThreads) void k_kv_append(AppendArgs a, int rb, int hg) {
  typedef typename A::type T;
  constexpr int D = 32 * NB, kUnits = D / (2 * W);  // thread steps per head
  extern __shared__ double2 append_lds[];
  __shared__ int slot_lds[16];
  const int tid = threadIdx.x, pairs = a.inv_freq ? a.pairs : 0;
  const int row0 = blockIdx.x * rb, rows = min(rb, a.rows - row0);
  const int h0 = blockIdx.y * hg, heads = min(hg, a.g.heads - h0);
  const int q0 = (int)((int64_t)a.q.heads * blockIdx.y / gridDim.y);
  const int qn = (int)((int64_t)a.q.heads * (blockIdx.y + 1) / gridDim.y) - q0;
  double2 *turn = append_lds;                      // [rb][pairs]: cosine, sine
  float2 *turn32 = (float2 *)(turn + rb * pairs);  // the same in fp32
  float *stage = (float *)(turn32 + ((rb * pairs + 1) & ~1));  // [rb][k heads, v heads][D]
  if (tid < rows) {
    const int slot = a.slots[row0 + tid];
    slot_lds[tid] = slot >= 0 && (slot >> a.g.page_shift) < a.g.pages ? slot : -1;
  }
  __syncthreads();
  for (int i = tid; i < rows * pairs; i += kThreads) {
    const int row = i / pairs, p = i - row * pairs;
    if (slot_lds[row] < 0) continue;
    int axis = 0;
    while (axis < 3 && p >= a.section_end[axis]) ++axis;
    const double angle = (double)a.positions[axis * a.axis_stride + row0 + row] * (double)a.inv_freq[p];
    double si, co;
    sincos(angle, &si, &co);
    turn[i] = make_double2(co, si);
    turn32[i] = make_float2((float)co, (float)si);
  }
  __syncthreads();
  // the two runs of W elements of a head's step u: W pairs, or 2 W elements that stay
  auto runs = [&](int u, int np, int &e0, int &e1) {
    const bool turned = u * W < np;
    e0 = turned ? (a.interleaved ? 2 * u * W : u * W) : 2 * np + (u * W - np) * 2;
    e1 = e0 + (turned && !a.interleaved ? np : W);
    return turned;
  };
  for (int i = tid; i < rows * 2 * heads * kUnits; i += kThreads) {
    const int u = i % kUnits, rest = i / kUnits, row = rest / (2 * heads), j = rest - row * 2 * heads;
    if (slot_lds[row] < 0) continue;
    const bool is_v = j >= heads;
    const int head = h0 + (is_v ? j - heads : j);
    const T *x = (const T *)(is_v ? a.v.data : a.k.data) +
                 (row0 + row) * (is_v ? a.v.row_stride : a.k.row_stride) + head * (is_v ? a.v.head_stride : a.k.head_stride);
    int e0, e1;
    const bool turned = runs(u, is_v ? 0 : pairs, e0, e1);
    float lo[W], hi[W];
    load_run<A, W, (W > 1)>(x + e0, lo);
    load_run<A, W, (W > 1)>(x + e1, hi);
    if (turned) {
      double dlo[W], dhi[W];
#pragma unroll
      for (int k = 0; k < W; ++k) {
        dlo[k] = lo[k];
        dhi[k] = hi[k];
      }
      turn_pairs<double, double2, W>(dlo, dhi, turn + row * pairs + u * W, a.interleaved);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        lo[k] = (float)dlo[k];
        hi[k] = (float)dhi[k];
      }
    }
    float *y = stage + (row * 2 * heads + j) * D;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      y[e0 + k] = lo[k];
      y[e1 + k] = hi[k];
    }
  }
  for (int i = tid; i < rows * qn * kUnits; i += kThreads) {
    const int u = i % kUnits, rest = i / kUnits, row = rest / qn, head = q0 + rest - row * qn;
    if (slot_lds[row] < 0) continue;
    const T *x = (const T *)a.q.data + (row0 + row) * a.q.row_stride + head * a.q.head_stride;
    T *y = (T *)a.q_out.data + (row0 + row) * a.q_out.row_stride + head * a.q_out.head_stride;
    int e0, e1;
    const bool turned = runs(u, pairs, e0, e1);
    float lo[W], hi[W];
    load_run<A, W, (W > 1)>(x + e0, lo);
    load_run<A, W, (W > 1)>(x + e1, hi);
    if (turned) turn_pairs<float, float2, W>(lo, hi, turn32 + row * pairs + u * W, a.interleaved);
    if constexpr (W > 1) {
      store_run_past<A, W>(y + e0, lo);
      store_run_past<A, W>(y + e1, hi);
    } else {
      y[e0] = A::from(lo[0]);
      y[e1] = A::from(hi[0]);
    }
  }
  __syncthreads();
  // a group of sixteen lanes takes a row's head, block by block
  const int lane = tid & 63, c = lane & 15, sh = lane & 48, pairs_of = rows * 2 * heads;
  for (int i0 = wave_index() * 4; i0 < pairs_of; i0 += kThreads / 16) {
    const int i = min(i0 + (lane >> 4), pairs_of - 1);  // the ballots below take whole waves
    const int row = i / (2 * heads), j = i - row * 2 * heads;
    const int slot = slot_lds[row];
    const bool live = slot >= 0 && i == i0 + (lane >> 4), is_v = j >= heads;
    const int tok = slot & 15;
    const float *x = stage + (row * 2 * heads + j) * D;
    uint8_t *tile = a.g.data + (live ? tile_of_slot(a.g, slot, h0 + (is_v ? j - heads : j)) : 0) + (is_v ? 288 * NB : 0);
    // the lane's byte of value quants, or (every fourth lane) its dword of key quants, of block 0
    constexpr int kWords = NB < 4 ? NB : 4;
    uint8_t *to = tile + (is_v ? ((tok >> 2) * 16 + c) * kWords * 4 + quant_place(tok) : ((c >> 2) * 16 + tok) * kWords * 4);
    _Float16 *to_scale = (_Float16 *)(tile + 256 * NB) + (tok >> 2) * NB * 4 + (tok & 3);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float lo = slot >= 0 ? x[32 * b + c] : 0.f, hi = slot >= 0 ? x[32 * b + c + 16] : 0.f;
      float most = fmaxf(fabsf(lo), fabsf(hi));
      const bool odd = !(fabsf(lo) < INFINITY) || !(fabsf(hi) < INFINITY);
      most = fmaxf(most, row_rotate<8>(most));
      most = fmaxf(most, row_rotate<4>(most));
      most = fmaxf(most, row_rotate<2>(most));
      most = fmaxf(most, row_rotate<1>(most));
      auto group = [&](bool v) { return (unsigned)(__ballot(v) >> sh) & 0xFFFFu; };
      const unsigned in_lo = group(fabsf(lo) == most), in_hi = group(fabsf(hi) == most);
      const unsigned neg_lo = group(lo < 0.f), neg_hi = group(hi < 0.f), any_odd = group(odd);
      // sign of the first value of largest magnitude: values 0..15 are the lo ones
      const unsigned in = in_lo ? in_lo : in_hi, neg = in_lo ? neg_lo : neg_hi;
      const bool negative = (neg & in & (0u - in)) != 0;
      const float want = fminf(most * 0.125f, 65504.f);
      _Float16 d = (_Float16)(negative ? want : -want);
      if (any_odd) d = __builtin_bit_cast(_Float16, (uint16_t)0x7E00);
      const float df = (float)d, inv = __builtin_amdgcn_rcpf(df), h = 0.5f * fabsf(df);
      const bool none = any_odd || df == 0.f;
      // nearest even of v / d, exactly: v - n d is exact in fp32 (n has 4 bits, d 11), so its
      // comparison with d / 2 settles what the approximate reciprocal may have missed
      auto nibble = [&](float v) -> uint32_t {
        float n = fminf(fmaxf(rintf(v * inv), -9.f), 9.f);
        const float r = fmaf(-n, df, v);
        const float m = n + ((r < 0.f) == (df < 0.f) ? 1.f : -1.f);  // the neighbour on r's side
        if (fabsf(r) > h || (fabsf(r) == h && ((int)n & 1))) n = m;
        return none ? 8u : (uint32_t)(8 + (int)fminf(fmaxf(n, -8.f), 7.f));
      };
      const uint32_t byte = nibble(lo) | nibble(hi) << 4;
      uint32_t word = byte << (8 * quant_place(c));
      word |= quad_swap<1>(word);
      word |= quad_swap<2>(word);
      if (!live) continue;
      constexpr int kChunk = 64 * kWords * 4;
      uint8_t *at = to + (b / kWords) * kChunk + (b % kWords) * 4;
      if (is_v) *at = (uint8_t)byte;
      else if ((c & 3) == 0) *(uint32_t *)at = word;
      if (c == 0) to_scale[4 * b] = d;
    }
  }
}

// ---- read -----------------------------------------------------------------------------------

// One thread: eight neighbouring values of one row and head, keys and values, so that a wave stores
// whole lines. The quants (of a value row: a byte of each of sixteen dwords a block, which four
// tokens share) come through LDS, fetched 16 bytes a lane: read byte by byte from global memory, the
// loads' address work took the whole time (66 cycles an instruction; 119 us for 65536 rows). Bound by
// HBM: 65536 rows bf16 of 8 heads of 128 take 64 us, 5.4 TB/s of 344 MB.
template <typename A, int NB>
__global__ __launch_bounds__(kThreads) void k_kv_read(ReadArgs a, int rows_per_wg) {
  typedef typename A::type T;
  constexpr int kUnits = NB * 4, kWords = NB < 4 ? NB : 4, kHeads = kThreads / kUnits, kPieces = NB * 4;
  __shared__ u32x4 quads[kHeads][kPieces + 1];  // a row's head: the dwords of its four tokens' value quants
  __shared__ uint32_t keys[kHeads][kPieces + 1];  // its key quants [chunk][i / 4][word]
  const int row0 = blockIdx.x * rows_per_wg;
  const int n = min(rows_per_wg, a.rows - row0) * a.g.heads;  // heads of rows
  const int u = threadIdx.x % kUnits, mine = threadIdx.x / kUnits;  // also the piece that the thread fetches
  const int b = u >> 2, half = u >> 1 & 1, f = u & 1;
  const int chunk = b / kWords, word = b - chunk * kWords;
  for (int i0 = 0; i0 < n; i0 += kHeads) {
    const int i = i0 + mine;
    const bool live = mine < kHeads && i < n;
    const int r = live ? i / a.g.heads : 0, row = row0 + r, h = live ? i - r * a.g.heads : 0;
    const int slot = a.slots[row], tok = slot & 15;
    const bool there = slot >= 0 && (slot >> a.g.page_shift) < a.g.pages;
    float kd = 0.f, vd = 0.f;
    if (i0) __syncthreads();
    if (live && there) {
      const uint8_t *tile = a.g.data + tile_of_slot(a.g, slot, h);
      const int scale_at = ((tok >> 2) * NB + b) * 4 + (tok & 3);
      if (a.k) {
        keys[mine][u] = ((const uint32_t *)tile)[(u / kWords * 16 + tok) * kWords + u % kWords];
        kd = (float)((const _Float16 *)(tile + 256 * NB))[scale_at];
      }
      if (a.v) {
        constexpr int kChunk = kWords * 4;  // pieces of a chunk
        quads[mine][u] = gload(tile + 288 * NB + ((u / kChunk * 4 + (tok >> 2)) * kChunk + u % kChunk) * 16);
        vd = (float)((const _Float16 *)(tile + 544 * NB))[scale_at];
      }
    }
    __syncthreads();
    if (!live) continue;
    const int64_t out = ((int64_t)row * a.g.heads + h) * (32 * NB) + 8 * u;
    auto give = [&](void *dst, const uint32_t (&byte)[8], float d) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = there ? d * (float)((int)(byte[k] >> (4 * half) & 15u) - 8) : 0.f;
      store_run_past<A, 8>((T *)dst + out, v);
    };
    uint32_t byte[8];
    if (a.k) {
      const uint32_t *q = &keys[mine][(chunk * 4 + 2 * f) * kWords + word];
      const uint32_t w0 = q[0], w1 = q[kWords];
#pragma unroll
      for (int k = 0; k < 8; ++k) byte[k] = ((k < 4 ? w0 : w1) >> (8 * quant_place(k))) & 0xFFu;
      give(a.k, byte, kd);
    }
    if (a.v) {
      const uint8_t *q = (const uint8_t *)&quads[mine][0] + 4 * ((chunk * 16 + 8 * f) * kWords + word) + quant_place(tok & 3);
#pragma unroll
      for (int k = 0; k < 8; ++k) byte[k] = q[4 * kWords * k];
      give(a.v, byte, vd);
    }
  }
}

template <typename A, int NB>
int launch_append(const AppendArgs &a, hipStream_t s) {
  constexpr int kRun = 16 / (int)sizeof(typename A::type);  // elements of a 16-byte run
  const int pairs = a.inv_freq ? a.pairs : 0;
  auto lds = [&](int rb, int hg) { return rb * (pairs * 24 + 16 + 2 * hg * a.head_dim * 4); };
  // few rows: one row and head per workgroup (latency); many: up to four rows and eight heads, which
  // share a row's sines, within 20 KB of LDS, so that registers and not LDS bound the workgroups of a
  // compute unit (8192 rows of 64 + 16 heads of 128: 81 us with two rows in 20 KB, 87 us with four in
  // 39 KB; 1501 rows of head_dim 64, which stay within it: 15.7 us with four rows, 17.4 us with two)
  int rb = 1, hg = 1;
  if ((int64_t)a.rows * a.g.heads > 1024) {
    hg = a.g.heads < 8 ? a.g.heads : 8;
    for (rb = 4; rb > 1 && lds(rb, hg) > 20 * 1024;) rb >>= 1;
  }
  const dim3 grid((a.rows + rb - 1) / rb, (a.g.heads + hg - 1) / hg);
  auto fits = [](const HeadRows &h) {
    return h.data == nullptr || ((uintptr_t)h.data % 16 == 0 && h.row_stride % kRun == 0 && h.head_stride % kRun == 0);
  };
  if (pairs % kRun == 0 && fits(a.k) && fits(a.v) && fits(a.q) && fits(a.q_out))
    k_kv_append<A, kRun, NB><<<grid, kThreads, lds(rb, hg), s>>>(a, rb, hg);
  else
    k_kv_append<A, 1, NB><<<grid, kThreads, lds(rb, hg), s>>>(a, rb, hg);
  return launch_status();
}

template <typename A, int NB>
int launch_read(const ReadArgs &a, hipStream_t s) {
  // few rows: a workgroup per row; many: enough rows for each thread to take four units
  const int per_row = a.g.heads * NB * 4;
  const int most = (4 * kThreads + per_row - 1) / per_row;
  const int rows = clampi(a.rows / 1024, 1, most);
  k_kv_read<A, NB><<<dim3((a.rows + rows - 1) / rows), kThreads, 0, s>>>(a, rows);
  return launch_status();
}

template <typename A>
int append_dim(const AppendArgs &a, hipStream_t s) {
  switch (a.g.nb) {
    case 2: return launch_append<A, 2>(a, s);
    case 3: return launch_append<A, 3>(a, s);
    case 4: return launch_append<A, 4>(a, s);
    default: return launch_append<A, 8>(a, s);
  }
}

template <typename A>
int read_dim(const ReadArgs &a, hipStream_t s) {
  switch (a.g.nb) {
    case 2: return launch_read<A, 2>(a, s);
    case 3: return launch_read<A, 3>(a, s);
    case 4: return launch_read<A, 4>(a, s);
    default: return launch_read<A, 8>(a, s);
  }
}

}  // namespace

int launch_kv_plan(const PlanArgs &a, hipStream_t s) {
  const int work = a.rows > a.requests ? a.rows : a.requests;
  const int grid = clampi((work + 2 * kThreads - 1) / (2 * kThreads), 1, 64);
  k_kv_plan<<<dim3(grid), kThreads, (size_t)3 * (a.requests + 1) * 4, s>>>(a);
  return launch_status();
}

int launch_kv_append(int type, const AppendArgs &a, hipStream_t s) {
  return type == TQ_F32 ? append_dim<ActF32>(a, s)
         : type == TQ_BF16 ? append_dim<ActBF16>(a, s) : append_dim<ActF16>(a, s);
}

int launch_kv_read(int type, const ReadArgs &a, hipStream_t s) {
  return type == TQ_F32 ? read_dim<ActF32>(a, s)
         : type == TQ_BF16 ? read_dim<ActBF16>(a, s) : read_dim<ActF16>(a, s);
}

}  // namespace tq
