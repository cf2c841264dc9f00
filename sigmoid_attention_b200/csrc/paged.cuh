// paged.cuh -- arguments of the paged-cache kernels (pages.cu, paged_few.cu,
// paged_many.cu).
#pragma once

#include "common.cuh"

namespace sigattn {

constexpr int kMaxPagedLen = 1 << 24;  // tokens of one sequence (max_pages * page_size)
constexpr int kMaxPagedGroup = 128;    // query heads per key/value head

struct PagedReserve {
  const int *cached, *fresh;  // [B]
  int* table;                 // [B][max_pages]
  const int* free_pages;
  const int* free_count;
  int* free_count_out;
  int *cu, *kv, *slots, *positions;
  int B, max_pages, page_shift, num_pages, rows;
  int max_new;  // most new tokens of one sequence
  int* ws;
};

struct PagedRelease {
  const int *kv, *keep;  // [B]; keep may be null
  const int* table;
  int* free_pages;
  const int* free_count;
  int* free_count_out;
  int* kv_out;  // [B]; may be null
  int B, max_pages, page_shift, num_pages;
  int* ws;
};

struct PagedWrite {
  const __nv_bfloat16 *k, *v, *q;
  __nv_bfloat16 *k_cache, *v_cache, *q_out;
  long long k_stride, v_stride, q_stride, q_out_stride;
  const int *slots, *positions, *pair_axis;
  const float* inv_freq;
  int axes, pairs, adjacent, rows, Hq, Hkv, d, page_shift, num_pages;
  int shares;  // warps per token (set by the launcher)
  int* ws;
};

struct PagedAttend {
  const __nv_bfloat16 *q, *k_cache, *v_cache;
  __nv_bfloat16* o;
  long long q_stride;
  const int *cu, *kv, *table;
  int B, Hq, Hkv, max_q, total, max_pages, page_shift, num_pages, d, causal;
  int lone;      // most units per CTA that are shared out by single query tiles (paged_many.cu)
  float cut;     // what a row of a part costs to add up, in units of work
  float* parts;  // partial sums of tiles cut over CTAs, two places per CTA
  int* ws;
};

// CTAs of a paged attention call at most (the workspace holds two parts each).
constexpr int kMaxPagedCtas = 152;
// PagedAttend::cut. Measured, per setting 0 / kFewCut / 5 kFewCut: one token of 8
// query rows over 36663 keys 25.7 / 16.4 / 19.1 us, of 16 over 131072 52.4 / 36.3 /
// 44.5 us; per 1/2 / 1 / 2 / 4 kManyCut: 200 tokens of 8 heads over 4000 keys 26.9 /
// 25.2 / 26.7 / 28.1 us, 200 of one head over 60000 58.7 / 56.2 / 58.6 / 68.5, 700 of
// 4 heads over 1500 23.8 / 21.4 / 21.5 / 22.7 (and 0 in pairs: 34 tokens of 7 heads
// over 29856 keys 84 us, with it 41).
constexpr float kFewCut = 0.02f, kManyCut = 0.003f;
// PagedAttend::lone, at d = 64. Single tiles against pairs: 200 tokens of 8 heads
// over 4000 keys 25 / 36 us, 300 tokens of 8 heads 11.8 / 15.7, 500 tokens of 8
// heads over 5000 keys (d = 128, 16 units) 32 / 42 and over 10000 43 / 53; beyond
// that a pair's better use of each key block wins: 1000 tokens over 30000 keys 162
// / 141 us, and at d = 64 500 tokens over 10000 (16 units) 36 / 35, 30000 79 / 65.
constexpr int kLoneUnits = 16;
// Query rows per key/value head (G * new tokens) up to which paged_few.cu serves;
// beyond, paged_many.cu. Measured, few / many, 16 texts of 2000 keys, 8 heads: d = 64,
// 32 rows 21.7 / 30.9 us, 50 28.9 / 31.7, 64 31.3 / 31.6; d = 128, 17 rows 30.3 / 32.6, 32
// 33.5 / 32.1, 50 38.5 / 33.0, 64 43.5 / 33.0 (each thread's weights and the products'
// columns grow with the rows).
constexpr int few_rows(int d) { return d == 64 ? 64 : 32; }

// One pair in one word (x1 low, x2 high) turned by (cos, sin) = cs.
__device__ __forceinline__ uint32_t turn_word(uint32_t w, float2 cs) {
  const float x1 = __uint_as_float(w << 16), x2 = __uint_as_float(w & 0xffff0000u);
  return pack_bf16x2(x1 * cs.x - x2 * cs.y, x2 * cs.x + x1 * cs.y);
}

// Two pairs: first members in the halves of x, second members in those of y.
__device__ __forceinline__ void turn_words(uint32_t& x, uint32_t& y, float2 lo, float2 hi) {
  const float x1 = __uint_as_float(x << 16), x2 = __uint_as_float(y << 16);
  const float z1 = __uint_as_float(x & 0xffff0000u), z2 = __uint_as_float(y & 0xffff0000u);
  x = pack_bf16x2(x1 * lo.x - x2 * lo.y, z1 * hi.x - z2 * hi.y);
  y = pack_bf16x2(x2 * lo.x + x1 * lo.y, z2 * hi.x + z1 * hi.y);
}

}  // namespace sigattn
