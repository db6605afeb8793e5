// tq_kv.h -- the paged 4-bit key/value cache: layout and host-side launchers (internal to libtq).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"

namespace tq {

// ---- layout ---------------------------------------------------------------------------------
// A page holds, per kv head, page_tokens / 16 tiles of 16 tokens. A tile is
//   key quants | key scales | value quants | value scales.
// A row (one token of one head) is NB = head_dim / 32 blocks of 32 values, w = d * (n - 8) with d
// fp16 and n 0..15 (TQ_Q4_0's values). One byte of quants holds a block's values i and i + 16
// (low and high nibble, i < 16). The bytes are ordered for the attention kernel's matrix-core
// operands: one 16-byte load per lane (head_dim 128) is the lane's share of four key (or value)
// operands, a wave reads 1 KiB in one run, and the two bytes 0 and 2 (or 1 and 3) of a dword are
// neighbours along the contracted dimension.
//   keys    [chunk][i / 4][token][word][P[i % 4]]       block = chunk * words + word
//   values  [chunk][token / 4][i][word][P[token % 4]]
//   scales  [token / 4][block][token % 4]
// P = (0, 2, 1, 3); words = min(NB, 4).
struct KvGeom {
  int nb, words;           // blocks per row, words (blocks) per chunk
  int heads, page_tokens, page_shift;  // kv heads; page_tokens = 1 << page_shift
  int quant_bytes, half_bytes, tile_bytes;  // key quants, key quants + scales, whole tile
  int64_t head_bytes, page_bytes;           // one head's tiles in a page, a page
  int64_t pages;
  uint8_t *data;
};

inline KvGeom kv_geom(const tq_kv_cache &c) {
  KvGeom g{};
  g.nb = (int)(c.head_dim / 32);
  g.words = g.nb < 4 ? g.nb : 4;
  g.heads = (int)c.kv_heads;
  g.page_tokens = (int)c.page_tokens;
  while ((1 << g.page_shift) < g.page_tokens) ++g.page_shift;
  g.quant_bytes = 256 * g.nb;
  g.half_bytes = g.quant_bytes + 32 * g.nb;
  g.tile_bytes = 2 * g.half_bytes;
  g.head_bytes = (int64_t)(g.page_tokens / 16) * g.tile_bytes;
  g.page_bytes = g.head_bytes * g.heads;
  g.pages = c.pages;
  g.data = (uint8_t *)c.data;
  return g;
}

// Strided rows of heads: element (row, head, i) at data + row * row_stride + head * head_stride + i.
struct HeadRows {
  void *data;
  int64_t row_stride, head_stride;
  int heads;
};

struct PlanArgs {
  int requests, max_blocks, rows, page_shift, pages;
  const int32_t *kv_len, *new_len;
  int32_t *block_table, *free_pages;
  const int32_t *free_count;
  int32_t *cu_new, *seq_len, *slots, *positions, *requests_of, *free_count_out, *status;
};

struct AppendArgs {
  KvGeom g;
  int rows, head_dim;
  const int32_t *slots;
  HeadRows k, v, q, q_out;
  const float *inv_freq;  // null: no rotation
  const int32_t *positions;
  int64_t axis_stride;
  int pairs, interleaved;
  int section_end[4];  // pair p takes its position from the first axis a with p < section_end[a]
};

struct ReadArgs {
  KvGeom g;
  int rows, head_dim;
  const int32_t *slots;
  void *k, *v;  // [rows][heads][head_dim]
};

struct AttnArgs {
  KvGeom g;
  int rows, requests, max_blocks, group, grid;
  int wide_cols;  // set by the launch
  int window;     // tokens a row sees, itself included; 0: all
  float scale;    // softmax scale times log2(e)
  HeadRows q, out;
  float *lse;     // [rows][q heads] or null
  const int32_t *block_table, *seq_len, *cu_new;
  float *parts;   // partial results (workspace)
  void *joins;    // behind them: the items to join
};

// Each returns 0 when everything was enqueued, -1 on a HIP launch error. `type` is TQ_F32,
// TQ_BF16 or TQ_F16.
int launch_kv_plan(const PlanArgs &a, hipStream_t s);
int launch_kv_append(int type, const AppendArgs &a, hipStream_t s);
int launch_kv_read(int type, const ReadArgs &a, hipStream_t s);
size_t kv_attention_workspace(int type, int64_t head_dim, int64_t group, int64_t rows, int64_t requests, int grid);
// Workgroups of the attention launch (each takes an equal share of the step's key tiles).
int kv_attention_grid(int type, int64_t kv_heads, int64_t head_dim, int64_t group, int64_t rows, int64_t max_len);
int launch_kv_attention(int type, const AttnArgs &a, hipStream_t s);

}  // namespace tq
