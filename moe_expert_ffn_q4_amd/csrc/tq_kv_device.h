// tq_kv_device.h -- device helpers shared by the key/value cache kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq_device.h"
#include "tq_kv.h"

namespace tq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Activation types: loads to fp32 and stores from fp32 (one nearest-even rounding).
struct ActF32 {
  typedef float type;
  static __device__ __forceinline__ float load(const type *p) { return *p; }
  static __device__ __forceinline__ type from(float v) { return v; }
};
struct ActBF16 {
  typedef __bf16 type;
  static __device__ __forceinline__ float load(const type *p) { return (float)*p; }
  static __device__ __forceinline__ type from(float v) { return (__bf16)v; }
};
struct ActF16 {
  typedef _Float16 type;
  static __device__ __forceinline__ float load(const type *p) { return (float)*p; }
  static __device__ __forceinline__ type from(float v) { return (_Float16)v; }
};

// N consecutive elements at p, in one access where VEC (p aligned to N elements).
template <typename A, int N, bool VEC>
__device__ __forceinline__ void load_run(const typename A::type *p, float *v) {
  typedef typename A::type run __attribute__((ext_vector_type(N)));
  if constexpr (VEC) {
    const run r = *(const run *)p;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (float)r[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = A::load(p + i);
  }
}
template <typename A, int N, bool VEC>
__device__ __forceinline__ void store_run(typename A::type *p, const float *v) {
  typedef typename A::type run __attribute__((ext_vector_type(N)));
  if constexpr (VEC) {
    run r;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = A::from(v[i]);
    *(run *)p = r;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = A::from(v[i]);
  }
}

// The same for N elements of 16 bytes or more that nothing reads back soon: past the caches, whose
// lines the stores would push out (65536 rows of k_kv_read: 93 -> 65 us).
template <typename A, int N>
__device__ __forceinline__ void store_run_past(typename A::type *p, const float *v) {
  typedef typename A::type run __attribute__((ext_vector_type(N)));
  struct pieces {
    u32x4 at[sizeof(run) / 16];
  };
  run r;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = A::from(v[i]);
  const pieces s = __builtin_bit_cast(pieces, r);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(run) / 16); ++i) __builtin_nontemporal_store(s.at[i], (u32x4 *)p + i);
}

// The place (0..3) of index i % 4 within a dword of quants: 0, 2, 1, 3.
__device__ __forceinline__ int quant_place(int i) { return ((i & 1) << 1) | ((i >> 1) & 1); }

// First byte of the tile that holds a slot (0 <= slot < pages * page_tokens) for kv head h.
__device__ __forceinline__ int64_t tile_of_slot(const KvGeom &g, int slot, int h) {
  const int page = slot >> g.page_shift, in = (slot & (g.page_tokens - 1)) >> 4;
  return (int64_t)page * g.page_bytes + (int64_t)h * g.head_bytes + (int64_t)in * g.tile_bytes;
}

// Dword of quants (within a tile's key or value quants): `four` indexes the groups of four that
// share a dword (keys: i / 4, values: token / 4), `sixteen` the other index (keys: token, values: i).
__device__ __forceinline__ int quant_word(const KvGeom &g, int block, int four, int sixteen) {
  const int w = g.words, chunk = block / w;
  return ((chunk * 4 + four) * 16 + sixteen) * w + block - chunk * w;
}

}  // namespace tq
