// What the two forms of the cache attention share: conversions of codes to
// matrix operands, rows and their masks, the softmax step.
#pragma once

#include "kv_device.hpp"

namespace w4k {

typedef __bf16 kv_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 kv_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 kv_f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 kv_f16x2 __attribute__((ext_vector_type(2)));
typedef float kv_f32x4 __attribute__((ext_vector_type(4)));
typedef float kv_f32x2 __attribute__((ext_vector_type(2)));
// 16 codes; a plain vector: arrays of the HIP struct type end up in scratch memory
typedef uint32_t kv_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t kv_u32x2 __attribute__((ext_vector_type(2)));

// lambdas over register arrays must be inlined for these to stay in registers
#define W4K_INLINE __attribute__((always_inline))

constexpr float kKvNone = -3e38f;     // running maximum before any entry
constexpr int kKvJoinThreads = 256;   // of the kernels that join partial results

// 16 codes from the cache, past the caches' reuse order: the cache streams
// through once, and whole lines fetched this way reach 5.9 TB/s where ordinary
// loads reach 5.4 (12 x 105k entries, 8 heads of 128, loads alone).
__device__ __forceinline__ kv_u32x4 kv_load(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const kv_u32x4*>(p));
}

// Four codes as two words of two bf16 (exact).
template <int TYPE>
__device__ __forceinline__ uint2 kv_bf16_of4(uint32_t w) {
  uint2 o;
  if constexpr (TYPE == W4A16_KV_INT8) {
    // integers up to 128 have 8 significant bits: the upper halves of their fp32 form
    o.x = __builtin_amdgcn_perm(__float_as_uint(kv_decode<TYPE, 1>(w)), __float_as_uint(kv_decode<TYPE, 0>(w)),
                                0x07060302u);
    o.y = __builtin_amdgcn_perm(__float_as_uint(kv_decode<TYPE, 3>(w)), __float_as_uint(kv_decode<TYPE, 2>(w)),
                                0x07060302u);
  } else {
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
  }
  return o;
}

// Four codes as two words of two fp16 (exact).
template <int TYPE>
__device__ __forceinline__ uint2 kv_f16_of4(uint32_t w) {
  uint2 o;
  if constexpr (TYPE == W4A16_KV_INT8) {
    // code + 128 in the low byte of the fp16 number 1024, then minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const kv_f16x2 bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    o.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(kv_f16x2, __builtin_amdgcn_perm(u, 0x64646464u, 0x00050004u)) + bias);
    o.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(kv_f16x2, __builtin_amdgcn_perm(u, 0x64646464u, 0x00070006u)) + bias);
  } else {
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
  }
  return o;
}

template <int TYPE>
__device__ __forceinline__ kv_bf16x8 kv_bf16_of8(uint32_t a, uint32_t b) {
  const uint2 x = kv_bf16_of4<TYPE>(a), y = kv_bf16_of4<TYPE>(b);
  return __builtin_bit_cast(kv_bf16x8, make_uint4(x.x, x.y, y.x, y.y));
}

template <int TYPE>
__device__ __forceinline__ kv_f16x8 kv_f16_of8(uint32_t a, uint32_t b) {
  const uint2 x = kv_f16_of4<TYPE>(a), y = kv_f16_of4<TYPE>(b);
  return __builtin_bit_cast(kv_f16x8, make_uint4(x.x, x.y, y.x, y.y));
}

// Requests whose rows within the step's bound (max_new tokens, which is what the
// launch is sized by) are few take the split form, the others tiles: one rule for
// the kernels of both forms and for their joins.
__device__ __forceinline__ bool kv_few_rows(const KvAttnArgs& a, int n) {
  return a.split && min(n, a.max_new) * a.group <= kKvSplitRows;
}

// Where the rows of one workgroup lie: shared by the split kernel and the join.
struct KvRows {
  int n, first, seq;      // new tokens, first token row, length of the request
  int live;               // tokens that have a row: at most max_new, and rows of q
  int begin, end;         // cache entries any of the group's rows attends
};

// The rows of tokens i0 .. i1 of request r (the last one clipped to its tokens).
__device__ __forceinline__ KvRows kv_rows_of(const KvAttnArgs& a, int r, int i0, int i1) {
  KvRows k;
  k.first = a.token_start[r];
  k.n = a.token_start[r + 1] - k.first;
  k.seq = a.seq_lens[r];
  const long long held = (long long)a.width << a.c.page_shift;
  const long long pos0 = (long long)k.seq - k.n;      // of token 0
  k.live = (int)min((long long)min(k.n, a.max_new), (long long)a.tokens - k.first);
  const long long hi = pos0 + min(i1, k.live - 1);      // (entries of tokens without a row may hold anything)
  // 0 <= begin <= end <= max_len where anything is attended, and begin = max(end, 0) where
  // nothing is: whatever the lengths and the window, tiles are counted from a number
  // that a few of them more do not carry past 32 bits
  k.end = (int)max(min(min(hi + 1, (long long)a.max_len), held), 0LL);
  k.begin = a.window > 0 ? (int)min(max(pos0 + i0 - a.window + 1, 0LL), (long long)k.end) : 0;
  return k;
}

__device__ __forceinline__ int kv_shared_entries(const KvSharedArgs& a) {
  return min(max(a.shared_len[0], 0), a.max_shared);
}
// Of these rows' entries those behind the shared ones.
__device__ __forceinline__ void kv_keep_own(const KvSharedArgs& a, KvRows& k) {
  const int shared = kv_shared_entries(a);
  k.end = min(k.end, shared + a.max_own);
  k.begin = min(shared, k.end);
}

// The last request that begins at or before token t.
__device__ __forceinline__ int kv_request_of(const KvAttnArgs& a, int t) {
  int r = 0;
  for (int count = a.requests; count > 1;) {
    const int step = count >> 1;
    if (a.token_start[r + step] <= t) r += step;
    count -= step;
  }
  return r;
}
// Positions of a batch's tokens.  Each lane of a wave holds one request (of more than 64, every
// step-th one's first token): one round of loads and a search across lanes, where a search through
// memory waits for a load at each of its steps.
struct KvOwners {
  int step, start, base;      // base: with one request a lane, what a token's position exceeds its row by
};
__device__ __forceinline__ KvOwners kv_owners(const KvAttnArgs& a) {
  KvOwners o;
  o.step = (a.requests + kWave - 1) / kWave;
  const int r = min((int)(threadIdx.x & (kWave - 1)) * o.step, a.requests - 1);
  o.start = a.token_start[r];
  o.base = o.step == 1 ? (int)((uint32_t)a.seq_lens[r] - (uint32_t)a.token_start[r + 1]) : 0;
  return o;
}
// The last of the first `shared` entries that token t attends, or -1 (by a whole wave).
__device__ __forceinline__ int kv_last_shared(const KvAttnArgs& a, const KvOwners& o, int t, int shared) {
  int l = 0;      // the last lane whose request begins at or before t
  for (int count = (a.requests + o.step - 1) / o.step; count > 1;) {
    const int half = count >> 1;
    if (__shfl(o.start, l + half) <= t) l += half;
    count -= half;
  }
  long long base = __shfl(o.base, l);
  if (o.step > 1) {
    int r = l * o.step;
    for (int count = min(o.step, a.requests - r); count > 1;) {
      const int half = count >> 1;
      if (a.token_start[r + half] <= t) r += half;
      count -= half;
    }
    base = (long long)a.seq_lens[r] - a.token_start[r + 1];
  }
  return (int)max(min(base + t, shared - 1LL), -1LL);
}

// The parts of the cache (a.part entries each) that rows of the tile form attend.
struct KvParts {
  int first, count;
};
__device__ __forceinline__ KvParts kv_parts_of(const KvAttnArgs& a, const KvRows& rows) {
  if (a.parts <= 1) return KvParts{0, 1};
  const int first = rows.begin / a.part;
  return KvParts{first, max(rows.end - 1, rows.begin) / a.part - first + 1};
}

// One lane's part of the rows it shares: entries lo .. hi of the cache.
template <int NC>
struct KvLaneRows {
  int hi[NC], lo[NC];
};

// For a number that a block entered by few waves computes with: made opaque
// inside the block, so that the compiler cannot move the block's selects in
// front of the branch (it did, and they were over a third of a tile's vector
// instructions).
__device__ __forceinline__ int kv_opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The largest of the values that lanes x, x + 16, x + 32 and x + 48 hold, to all
// four: a swap of a register with its copy sets the values of two rows of lanes
// side by side, without a way through LDS.
__device__ __forceinline__ float kv_max_of_groups(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// One tile's softmax step for a lane, in two parts: the scores s of its 4 NP
// entries (first entry j) for NC rows become the tile's largest logit of each row
// (kv_tile_max) and, once the running maximum is known, fp16 weights
// (kv_weights).  ks: key scale times the logits' scale (>= 0); vs: value
// scale; whole: no entry of the tile is masked for any row; page_ok: this
// lane's entries have a page.
template <int NC, int NP>
__device__ __forceinline__ void kv_tile_max(kv_f32x4 (&s)[NC][NP], const KvLaneRows<NC>& rows, int j, float ks,
                                            float lv, bool whole, bool page_ok, float (&tile_top)[NC]) {
  // entry e of the lane's 4 NP is attended by row c iff first <= e <= last
  if (!whole) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int first = kv_opaque(rows.lo[c] - j), last = kv_opaque(page_ok ? rows.hi[c] - j : -1);
#pragma unroll
      for (int e = 0; e < 4 * NP; ++e)
        s[c][e / 4][e % 4] = e >= first && e <= last ? s[c][e / 4][e % 4] : -__builtin_inff();
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float top = s[c][0][0];
#pragma unroll
    for (int e = 1; e + 1 < 4 * NP; e += 2)      // maxima of three
      top = fmaxf(fmaxf(top, s[c][e / 4][e % 4]), s[c][(e + 1) / 4][(e + 1) % 4]);
    top = fmaxf(top, s[c][NP - 1][3]);
    top = top > kKvNone ? __builtin_fmaf(top, ks, lv) : kKvNone;
    tile_top[c] = kv_max_of_groups(top);
  }
}

// The running maximum moves only when a row's logits exceed it by 8, and most
// tiles leave the sums as they are (a factor of exactly 1, also for the rows
// beside one that moves).  Weights are held times 2^6 (sums and output alike, so
// it divides out): at most 2^14, inside fp16's 65504, while entries of 2^-30 of the
// largest weight still count (without the factor those below 2^-25 vanished:
// a million of them beside one large entry are 3% of the answer).
constexpr float kKvWeightLog2 = 6.0f;
__device__ __forceinline__ float kv_new_max(float m, float top) { return top > m + 8.0f ? top : m; }

// Weights under the maxima m (already the new ones); l *= fade, += the tile's sum.
template <int NC, int NP>
__device__ __forceinline__ void kv_weights(kv_f32x4 (&s)[NC][NP], const KvLaneRows<NC>& rows, int j, float ks, float lv,
                                           float rv, bool whole, bool page_ok, const float (&m)[NC],
                                           const float (&fade)[NC], float (&l)[NC], kv_f16x8 (&w)[NC][NP / 2]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const float shift = lv + kKvWeightLog2 - m[c];
    float p[4 * NP], sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4 * NP; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[c][e / 4][e % 4], ks, shift));
    // masked entries are exactly 0 also where the page's scales are 0 or NaN
    float value_inverse = rv;
    if (!whole) {
      const int first = kv_opaque(rows.lo[c] - j), last = kv_opaque(page_ok ? rows.hi[c] - j : -1);
#pragma unroll
      for (int e = 0; e < 4 * NP; ++e) p[e] = e >= first && e <= last ? p[e] : 0.0f;
      value_inverse = first < 4 * NP && last >= 0 && first <= last ? rv : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4 * NP; ++e) sum += p[e];
    l[c] = __builtin_fmaf(l[c], fade[c], sum * value_inverse);
#pragma unroll
    for (int h = 0; h < NP / 2; ++h) {
      uint32_t pk[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const kv_f32x2 pair = {p[8 * h + 2 * i], p[8 * h + 2 * i + 1]};
        pk[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, kv_f16x2));
      }
      w[c][h] = __builtin_bit_cast(kv_f16x8, make_uint4(pk[0], pk[1], pk[2], pk[3]));
    }
  }
}

// E4M3 codes of entries that no row attends (never filled, or a page's next use)
// may be NaN, and 0 * NaN must not enter the sums: the bytes of 16 value codes
// that stand for entries `skip` .. `left` - 1 of them.
__device__ __forceinline__ kv_u32x4 kv_existing_bytes(int skip, int left) {
  auto below = [](int k) { return k >= 4 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << (8 * k)) - 1u; };
  auto bytes = [&](int b) { return below(left - 4 * b) & ~below(skip - 4 * b); };
  return kv_u32x4{bytes(0), bytes(1), bytes(2), bytes(3)};
}

// Products with N operands that lie in LDS, each read AHEAD of its use: left to
// itself the compiler read each into the registers of the one before, and a
// wave waited out LDS's latency for every one (in the tile form 1080 cycles a
// tile instead of 780 for 16 operands of two products each).
template <int AHEAD, int N, class Load, class Use>
__device__ __forceinline__ void kv_stream_operands(Load&& load, Use&& use) {
  decltype(load(0)) f[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) f[i] = load(i);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    use(i, f[i % AHEAD]);
    if (i + AHEAD < N) f[i % AHEAD] = load(i + AHEAD);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// 16 queries' elements with the sign of the logits' scale (so that ks >= 0)
__device__ __forceinline__ kv_bf16x8 kv_query8(const uint16_t* p, uint32_t sign) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  u = make_uint4(u.x ^ sign, u.y ^ sign, u.z ^ sign, u.w ^ sign);
  return __builtin_bit_cast(kv_bf16x8, u);
}

// What the sums are multiplied with at the end: 1 / l, and 0 for a row that
// attends nothing (one more fp32 rounding than a division, far below bf16's).
__device__ __forceinline__ float kv_inverse(float l) { return l != 0.0f ? 1.0f / l : 0.0f; }

__device__ __forceinline__ void kv_store4(uint16_t* out, kv_f32x4 v, float inverse) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<bf16x4*>(out) = __builtin_convertvector(v * inverse, bf16x4);
}

}  // namespace w4k
