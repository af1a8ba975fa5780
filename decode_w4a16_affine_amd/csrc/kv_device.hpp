// Device helpers of the paged 8-bit key/value cache (include/w4a16_kv.h): the
// scale rule, encoding and decoding of codes, and the argument structs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm_device.hpp"
#include "w4a16_kv.h"

namespace w4k {

constexpr float kKvMinScale = 0x1p-100f;

// Scale of a page and head from the bit pattern of its largest magnitude (bf16
// bits without sign, so integer order is the order of magnitudes with
// infinity and NaN on top), as fp32.  a / 127 resp. a / 448 in fp32 (correctly
// rounded), then up to the next bf16 number resp. power of two.  The exact
// quotient lies on the same side of every bf16 number b as its fp32 rounding:
// a and 127 b are multiples of one ulp of b's 8 significant bits, so where
// they differ they differ by over 2^-16 of a.  Non-finite magnitudes give NaN.
template <int TYPE>
__device__ __forceinline__ float kv_scale_of(uint32_t amax_bits) {
  if (amax_bits >= 0x7F80u) return __builtin_nanf("");
  const float a = bf16_lo(amax_bits);
  uint32_t u;
  if constexpr (TYPE == W4A16_KV_INT8)
    u = (__float_as_uint(a / 127.0f) + 0xFFFFu) & 0xFFFF0000u;
  else
    u = (__float_as_uint(a / 448.0f) + 0x7FFFFFu) & 0x7F800000u;
  return fmaxf(__uint_as_float(u), kKvMinScale);
}

// Nearest code of y (|y| <= 127 resp. 448 up to rounding), ties to even.
template <int TYPE>
__device__ __forceinline__ uint32_t kv_encode(float y) {
  if constexpr (TYPE == W4A16_KV_INT8)
    return (uint32_t)(int)rintf(y) & 0xFFu;
  else
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, 0.0f, 0, false) & 0xFFu;
}

// Code in byte B of a word as fp32 (exact).
template <int TYPE, int B>
__device__ __forceinline__ float kv_decode(uint32_t w) {
  if constexpr (TYPE == W4A16_KV_INT8)
    return (float)(int8_t)(w >> (8 * B));
  else
    return __builtin_amdgcn_cvt_f32_fp8((int)w, B);
}

// A page and head's scale is NaN: its codes are 0 (int8 has no other answer).
template <int TYPE>
__device__ __forceinline__ uint32_t kv_code_of(float x, float scale) {
  return scale == scale ? kv_encode<TYPE>(x / scale) : 0u;
}

struct KvCache {
  uint8_t* k;
  uint8_t* v;
  uint16_t* ks;
  uint16_t* vs;
  int pages, heads, page_shift;
};

struct KvAttnArgs {
  KvCache c;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* token_start;
  uint16_t* out;
  float scale_log2;      // |scale| * log2(e): softmax in base 2
  uint32_t q_sign;       // sign bits of two bf16 if scale < 0, else 0
  int width, window, tokens, requests, max_new, max_len, q_heads, group;
  uint32_t group_inverse;      // ceil(2^16 / group): see kv_token_of
  bool split;                  // requests of few rows take the split form (else all take tiles)
  bool by_token;               // its partial results lie by the step's tokens (else by request)
  // requests of few rows: log2 of the entries a chunk, chunks a row at most, row
  // groups a cache head, new tokens a request at most
  int chunk_shift, chunks, row_groups, split_tokens;
  // requests of many: parts of the cache that a row's workgroups share, entries a part
  int parts, part;
};

// Launchers (kv_attention.hip, once per head size).
#define W4K_DECLARE_KV(D)                                                                     \
  hipError_t kv_attention_d##D(int type, const KvAttnArgs& a, void* workspace, hipStream_t st);
W4K_DECLARE_KV(64)
W4K_DECLARE_KV(128)
W4K_DECLARE_KV(256)
#undef W4K_DECLARE_KV

// Row / group for 0 <= row < 1024 (group <= 64): the product exceeds the
// quotient by less than row / 2^16 < 1 / group.
__device__ __forceinline__ int kv_token_of(const KvAttnArgs& a, int row) {
  return (int)((uint32_t)row * a.group_inverse >> 16);
}

constexpr int kKvMaxChunks = 128;     // chunks of a row at most
constexpr int kKvSplitRows = 64;      // requests of at most this many rows a cache head take the split form

// A row and chunk's partial result: D floats of output, then these (the
// maximum and four waves' sums).  Rows lie as in `out`, or as split_tokens tokens a
// request where that is less (a step of many prompts' tokens): the rows that can
// take the split form are at most either.
constexpr int kKvPartStats = 5;
inline size_t kv_partials(const KvAttnArgs& a) {
  const size_t by_request = (size_t)a.requests * a.split_tokens;
  return a.split && a.chunks > 1 ? (a.by_token ? (size_t)a.tokens : by_request) * a.q_heads * a.chunks : 0;
}
// Row of the partial results of row out_row of `out`, which is of request r with first token row `first`.
__device__ __forceinline__ size_t kv_part_row(const KvAttnArgs& a, int out_row, int r, int first) {
  return a.by_token ? (size_t)out_row : out_row + ((int64_t)r * a.split_tokens - first) * a.q_heads;
}

// The tile form: waves of a workgroup, of which `share` take the same 32 rows
// (two for D = 256, where the output of 32 rows alone would take 128 registers of a
// wave), and its rows.  A row and part's partial result: D floats, maximum, sum.
constexpr int kKvTile = 64;           // cache entries at once
constexpr int kKvTileCols = 2;        // 16-row pieces a wave (or the waves that share rows)
constexpr int kKvTileStats = 2;
constexpr int kv_tile_share(int D) { return D == 256 ? 2 : 1; }
constexpr int kv_tile_waves(int D, int type) { return D == 256 && type == W4A16_KV_INT8 ? 8 : 4; }
constexpr int kv_tile_rows(int D, int type) { return kv_tile_waves(D, type) / kv_tile_share(D) * kKvTileCols * 16; }
inline size_t kv_tile_partials(const KvAttnArgs& a) {
  return a.parts > 1 ? (size_t)a.tokens * a.q_heads * a.parts : 0;
}

// The workspace, in floats: the split form's results, their statistics (up to a
// multiple of 16 bytes), the tile form's results and statistics.
inline size_t kv_split_floats(const KvAttnArgs& a, int D) {
  return kv_partials(a) * D + (kv_partials(a) * kKvPartStats + 3) / 4 * 4;
}
inline size_t kv_workspace_floats(const KvAttnArgs& a, int D) {
  return kv_split_floats(a, D) + kv_tile_partials(a) * (D + kKvTileStats);
}

}  // namespace w4k
