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

constexpr int kKvTile = 64;           // cache entries a wave takes at once
constexpr float kKvNone = -3e38f;     // running maximum before any entry

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

// Where the rows of one workgroup lie: shared by the split kernel and the join.
struct KvRows {
  int n, first, seq;      // new tokens, first token row, length of the request
  int begin, end;         // cache entries any of the group's rows attends
};

// Rows [row0, row0 + rows) of request r (rows counted token by token, G a token).
__device__ __forceinline__ KvRows kv_rows_of(const KvAttnArgs& a, int r, int row0, int rows) {
  KvRows k;
  k.first = a.token_start[r];
  k.n = a.token_start[r + 1] - k.first;
  k.seq = a.seq_lens[r];
  const int last = min(row0 + rows, min(k.n, a.max_new) * a.group) - 1;
  const long long held = (long long)a.width << a.c.page_shift;
  const int lo = k.seq - k.n + row0 / a.group, hi = k.seq - k.n + last / a.group;
  k.end = (int)min((long long)min(hi + 1, a.max_len), held);
  k.begin = a.window > 0 ? max(0, lo - a.window + 1) : 0;
  return k;
}

// One lane's part of the rows it shares: entries lo .. hi of the cache.
template <int NC>
struct KvLaneRows {
  int hi[NC], lo[NC];
};

// One tile's softmax step for a lane: scores s of its 16 entries (first entry
// j) and NC rows become fp16 weights; the running maximum m, sum l and the
// factor `fade` for what was summed before are updated.  ks: key scale times
// the logits' scale (>= 0), vs: value scale; whole: no entry of the tile is
// masked for any row; page_ok: this lane's entries have a page.
//
// The maximum moves only when a row's logits exceed it by 2^3: weights then stay
// below 2^8, far inside fp16, and most tiles leave the sums as they are (a
// factor of exactly 1, also for the rows beside one that moves).
constexpr float kKvSlack = 8.0f;

template <int NC>
__device__ __forceinline__ void kv_softmax_step(kv_f32x4 (&s)[NC][4], const KvLaneRows<NC>& rows, int j, float ks,
                                                float vs, bool whole, bool page_ok, float (&m)[NC], float (&l)[NC],
                                                float (&fade)[NC], kv_f16x8 (&w)[NC][2]) {
  const float lv = __builtin_amdgcn_logf(vs), rv = __builtin_amdgcn_rcpf(vs);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    // entry e of the 16 is attended by row c iff first <= e <= last
    const int first = rows.lo[c] - j, last = page_ok ? rows.hi[c] - j : -1;
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        s[c][e / 4][e % 4] = e >= first && e <= last ? s[c][e / 4][e % 4] : -__builtin_inff();
    }
    float top = fmaxf(fmaxf(s[c][0][0], s[c][0][1]), s[c][0][2]);
    top = fmaxf(fmaxf(top, s[c][0][3]), s[c][1][0]);
    top = fmaxf(fmaxf(top, s[c][1][1]), s[c][1][2]);
    top = fmaxf(fmaxf(top, s[c][1][3]), s[c][2][0]);
    top = fmaxf(fmaxf(top, s[c][2][1]), s[c][2][2]);
    top = fmaxf(fmaxf(top, s[c][2][3]), s[c][3][0]);
    top = fmaxf(fmaxf(top, s[c][3][1]), fmaxf(s[c][3][2], s[c][3][3]));
    top = top > kKvNone ? __builtin_fmaf(top, ks, lv) : kKvNone;
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m_new = top > m[c] + kKvSlack ? top : m[c];
    fade[c] = __builtin_amdgcn_exp2f(m[c] - m_new);
    m[c] = m_new;
    const float shift = lv - m_new;
    float p[16], sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[c][e / 4][e % 4], ks, shift));
    // masked entries are exactly 0 also where the page's scales are 0 or NaN
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 16; ++e) p[e] = e >= first && e <= last ? p[e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) sum += p[e];
    const bool any = whole || (first <= 15 && last >= 0 && first <= last);
    l[c] = l[c] * fade[c] + (any ? sum * rv : 0.0f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
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

// E4M3 codes of entries that hold nothing may be NaN, and 0 * NaN must not
// enter the sums: the bytes of 16 value codes that stand for existing entries.
__device__ __forceinline__ uint4 kv_existing_bytes(int left) {
  auto bytes = [&](int b) {
    const int k = left - 4 * b;
    return k >= 4 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
  };
  return make_uint4(bytes(0), bytes(1), bytes(2), bytes(3));
}
__device__ __forceinline__ uint4 kv_and(uint4 a, uint4 b) {
  return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}

// 16 queries' elements with the sign of the logits' scale (so that ks >= 0)
__device__ __forceinline__ kv_bf16x8 kv_query8(const uint16_t* p, uint32_t sign) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  u = make_uint4(u.x ^ sign, u.y ^ sign, u.z ^ sign, u.w ^ sign);
  return __builtin_bit_cast(kv_bf16x8, u);
}

__device__ __forceinline__ void kv_store4(uint16_t* out, kv_f32x4 v, float l) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = f32_to_bf16(l != 0.0f ? v[i] / l : 0.0f);
  *reinterpret_cast<uint2*>(out) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
}

}  // namespace w4k
