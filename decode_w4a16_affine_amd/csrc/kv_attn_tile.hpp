// Attention over the paged 8-bit cache for requests of many new tokens
// (prompts and prompt chunks).
//
// A workgroup of four waves takes 128 rows of one request and cache head (as
// many whole tokens' query heads as fit), 32 a wave, and walks the cache in
// tiles of 64 entries.  The products, the order of a lane's entries, the
// softmax and the arithmetic are those of the split form (kv_attn_split.hpp);
// what differs is where the operands come from: here a tile's codes serve 128
// rows, so each is loaded and converted once, by the thread whose place in a
// matrix operand it has, and put into LDS as a finished 16-bit operand (16
// bytes a lane, in lane order: reads and writes are free of bank conflicts).
// Two LDS buffers: the codes of the next tile are loaded into registers before
// the current one is multiplied and converted after it, one barrier a tile.
#pragma once

#include "kv_attn_common.hpp"

namespace w4k {

constexpr int kKvTile = 64;           // cache entries at once
constexpr int kKvTileWaves = 4;
constexpr int kKvTileCols = 2;                                     // 16-row pieces a wave
constexpr int kKvTileRows = kKvTileWaves * kKvTileCols * 16;

// Workgroup u -> request and first token.  Request r owns the numbers from
// floor(token_start[r] / TT) + r on: at least ceil(n / TT) of them, and they
// grow with r, so a search finds the owner without a prefix sum of tiles.
__device__ __forceinline__ int kv_tile_owner(const int32_t* token_start, int requests, int tt, int u) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, count = requests;         // the owner is in [lo, lo + count)
  while (count > 1) {
    const int step = (count + kWave - 1) / kWave;
    const int at = lo + lane * step;
    const bool past = lane * step >= count || token_start[at] / tt + at > u;
    const uint64_t no = __ballot(past);
    const int first = no ? __builtin_ctzll(no) : kWave;     // lanes before it begin at or before u
    if (first == 0) return -1;
    lo += (first - 1) * step;
    count = min(step, requests - lo);
  }
  return lo;
}

template <int D, int TYPE>
__global__ __launch_bounds__(kKvTileWaves * kWave) void kv_tile_kernel(KvAttnArgs a) {
  constexpr int NC = kKvTileCols;
  constexpr int KC = D / 64;          // 16-byte pieces of a key a lane holds
  constexpr int DT = D / 16;          // 16-row pieces of the output
  constexpr int VW = DT / kKvTileWaves;   // of which a wave loads
  __shared__ kv_u32x4 s_k[2][4 * 2 * KC * kWave];      // [piece t][sum step][lane]
  __shared__ kv_u32x4 s_v[2][DT * 2 * kWave];          // [piece d][sum step][lane]
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int x = lane & 15, g = lane >> 4;
  const int tt = kv_token_of(a, kKvTileRows);
  const int u = gridDim.x - 1 - blockIdx.x;        // later tokens attend more: they go first
  const int kh = blockIdx.y;
  const int r = __builtin_amdgcn_readfirstlane(kv_tile_owner(a.token_start, a.requests, tt, u));
  if (r < 0) return;
  const int i0 = (u - a.token_start[r] / tt - r) * tt;
  const int n = a.token_start[r + 1] - a.token_start[r];
  const int live_tokens = min(min(n, a.max_new), a.tokens - a.token_start[r]);
  if ((long long)n * a.group <= kKvSplitRows || i0 < 0 || i0 >= live_tokens || a.token_start[r] < 0) return;
  const int here = min(tt, live_tokens - i0);       // the workgroup's tokens
  const int live = here * a.group;                  // and rows
  const KvRows rows = kv_rows_of(a, r, i0, i0 + here - 1);
  const int shift = a.c.page_shift, P = 1 << shift;

  // this wave's rows
  const int wrow = wave * NC * 16;
  kv_bf16x8 q[NC][2 * KC];
  KvLaneRows<NC> lr;
  int64_t out_at[NC];
  const int pos0 = rows.seq - rows.n + i0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int row = min(wrow + 16 * c + x, live - 1);
    const int i = kv_token_of(a, row), h = kh * a.group + row - i * a.group;
    const int64_t t = rows.first + i0 + i;
    const bool ok = wrow + 16 * c + x < live;
    lr.hi[c] = ok ? min(pos0 + i, rows.end - 1) : -1;
    lr.lo[c] = a.window > 0 ? pos0 + i - a.window + 1 : 0;
    out_at[c] = ok ? (t * a.q_heads + h) * D : -1;
    const uint16_t* qp = a.q + t * a.q_stride + (size_t)h * D + 16 * g;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      q[c][2 * k] = kv_query8(qp + 64 * k, a.q_sign);
      q[c][2 * k + 1] = kv_query8(qp + 64 * k + 8, a.q_sign);
    }
  }
  // entries that some row of the wave attends, and those that every row does
  const int first_pos = pos0 + kv_token_of(a, min(wrow, live - 1));
  const int last_pos = pos0 + kv_token_of(a, min(wrow + NC * 16, live) - 1);
  const int any_hi = wrow < live ? min(last_pos, rows.end - 1) : -1;
  const int any_lo = a.window > 0 ? first_pos - a.window + 1 : 0;
  const int all_hi = min(first_pos, rows.end - 1);
  const int all_lo = a.window > 0 ? last_pos - a.window + 1 : 0;

  kv_f32x4 o[NC][DT];
  float m[NC], l[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    m[c] = kKvNone;
    l[c] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[c][d] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // the codes, scales and page of a tile that this thread loads
  const int32_t* table = a.table + (size_t)r * a.width;
  kv_u32x4 kc[KC], vc[VW];
  float ks, vs;
  bool page_ok;
  auto load = [&](int j0) {
    auto page_of = [&](int b) {
      const int j = j0 + 16 * b;
      const int page = j < rows.end ? table[j >> shift] : -1;
      return page >= 0 && page < a.c.pages ? page : -1;
    };
    const int kp = page_of(x >> 2), vp = page_of(g);
    const size_t kph = (size_t)max(kp, 0) * a.c.heads + kh, vph = (size_t)max(vp, 0) * a.c.heads + kh;
    const uint8_t* ka = a.c.k + (kph * P + ((j0 + 16 * (x >> 2)) & (P - 1)) + 4 * wave + (x & 3)) * D + 16 * g;
    const uint8_t* va = a.c.v + (vph * D + 16 * VW * wave + x) * P + ((j0 + 16 * g) & (P - 1));
#pragma unroll
    for (int k = 0; k < KC; ++k) kc[k] = *reinterpret_cast<const kv_u32x4*>(ka + 64 * k);
#pragma unroll
    for (int d = 0; d < VW; ++d) vc[d] = *reinterpret_cast<const kv_u32x4*>(va + (size_t)d * 16 * P);
    ks = bf16_lo(a.c.ks[vph]) * a.scale_log2;
    vs = bf16_lo(a.c.vs[vph]);
    vs = vs < kKvMinScale ? kKvMinScale : vs;     // 0 in a page that was never begun; NaN stays
    page_ok = vp >= 0;
    if (TYPE == W4A16_KV_FP8 && (j0 + kKvTile > rows.end || !__all(page_ok))) {
      const kv_u32x4 mask = kv_existing_bytes(page_ok ? rows.end - (j0 + 16 * g) : 0);
#pragma unroll
      for (int d = 0; d < VW; ++d) vc[d] = vc[d] & mask;
    }
  };
  auto store = [&](int b) {
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      s_k[b][((wave * KC + k) * 2) * kWave + lane] =
          __builtin_bit_cast(kv_u32x4, kv_bf16_of8<TYPE>(kc[k].x, kc[k].y));
      s_k[b][((wave * KC + k) * 2 + 1) * kWave + lane] =
          __builtin_bit_cast(kv_u32x4, kv_bf16_of8<TYPE>(kc[k].z, kc[k].w));
    }
#pragma unroll
    for (int d = 0; d < VW; ++d) {
      s_v[b][((wave * VW + d) * 2) * kWave + lane] = __builtin_bit_cast(kv_u32x4, kv_f16_of8<TYPE>(vc[d].x, vc[d].y));
      s_v[b][((wave * VW + d) * 2 + 1) * kWave + lane] =
          __builtin_bit_cast(kv_u32x4, kv_f16_of8<TYPE>(vc[d].z, vc[d].w));
    }
  };

  int j0 = rows.begin & ~(kKvTile - 1);
  if (j0 < rows.end) {
    load(j0);
    store(0);
  }
  __syncthreads();
  for (int b = 0; j0 < rows.end; j0 += kKvTile, b ^= 1) {
    const float ks_now = ks, vs_now = vs;
    const bool ok_now = page_ok;
    const bool more = j0 + kKvTile < rows.end;
    if (more) load(j0 + kKvTile);
    if (j0 <= any_hi && j0 + kKvTile > any_lo) {
      const bool whole = __all(ok_now) && j0 + kKvTile - 1 <= all_hi && j0 >= all_lo;
      kv_f32x4 s[NC][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int c = 0; c < NC; ++c) s[c][t] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 2 * KC; ++k) {
          const kv_bf16x8 f = __builtin_bit_cast(kv_bf16x8, s_k[b][(t * 2 * KC + k) * kWave + lane]);
#pragma unroll
          for (int c = 0; c < NC; ++c) s[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, q[c][k], s[c][t], 0, 0, 0);
        }
      }
      float fade[NC], top[NC];
      kv_f16x8 w[NC][2];
      const float lv = __builtin_amdgcn_logf(vs_now), rv = __builtin_amdgcn_rcpf(vs_now);
      kv_tile_max<NC, 4>(s, lr, j0 + 16 * g, ks_now, lv, whole, ok_now, top);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float m_new = kv_new_max(m[c], top[c]);
        fade[c] = __builtin_amdgcn_exp2f(m[c] - m_new);
        m[c] = m_new;
      }
      kv_weights<NC, 4>(s, lr, j0 + 16 * g, ks_now, lv, rv, whole, ok_now, m, fade, l, w);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (__any(fade[c] != 1.0f))
#pragma unroll
          for (int d = 0; d < DT; ++d) o[c][d] *= fade[c];
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const kv_f16x8 f = __builtin_bit_cast(kv_f16x8, s_v[b][(d * 2 + h) * kWave + lane]);
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, w[c][h], o[c][d], 0, 0, 0);
        }
    }
    if (more) store(b ^ 1);
    __syncthreads();
  }

#pragma unroll
  for (int c = 0; c < NC; ++c) {
    l[c] += __shfl_xor(l[c], 16);
    l[c] += __shfl_xor(l[c], 32);
    if (out_at[c] < 0) continue;
    const float inverse = kv_inverse(l[c]);
#pragma unroll
    for (int d = 0; d < DT; ++d) kv_store4(a.out + out_at[c] + 16 * d + 4 * g, o[c][d], inverse);
  }
}

}  // namespace w4k
