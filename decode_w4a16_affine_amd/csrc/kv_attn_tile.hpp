// Attention over the paged 8-bit cache for requests of many new tokens
// (prompts and prompt chunks).
//
// A workgroup takes 128 rows of one request and cache head (64 for D = 256 with
// E4M3 codes; as many whole tokens' query heads as fit) and walks the cache in
// tiles of 64 entries.  The products, the softmax and the arithmetic are those of
// the split form (kv_attn_split.hpp); what differs is how the work is cut.  Here
// a tile's codes serve all rows, so each is loaded and converted once, by the
// thread whose place in a matrix operand it has, and put into LDS as a finished
// 16-bit operand (16 bytes a lane, in lane order: reads and writes are free of
// bank conflicts).  Lane (x, g) = (l % 16, l / 16) scores entries 16 g .. + 15 of the
// tile: rows 4 b + i of piece t of the key operand are entries 16 b + 4 t + i.
//
// D = 64, 128: a wave has 32 rows.  Keys and values have two buffers; the next
// tile's codes are loaded before this one is multiplied and converted after it,
// one barrier a tile.  (One buffer and two barriers: 686 us instead of 634 for
// four prompt chunks of 200 to 2000 tokens behind up to 12000, 32 heads of 128.)
// D = 256: the output of 32 rows would take 128 registers of a wave, so two waves
// share them: each scores half of the entries (pieces t = 2 h, 2 h + 1, whose
// weights are operand h of the second product), they agree on the maxima and
// exchange weights through LDS, and each multiplies all 64 weights with the
// values of its half of the head's elements.  One buffer and two barriers: before
// the first, the waves score and publish maxima; between them they write
// weights, this tile's values and the next tile's keys.  (One wave for 32 rows:
// 246 us where two took 166, before operands were read ahead; a prompt of 4099
// tokens, 10 heads of 256.)  With int8 codes the conversions need registers that
// only eight waves (two pieces each to convert instead of four) leave; four
// reloaded the queries from scratch memory every tile (515 us where eight took 207,
// at that time).
//
// Bound and measured.  The matrix products are 2 x 32 instructions of 16 cycles a
// wave and tile, 1024 cycles; beside them a wave issues about 340 vector
// instructions a tile for heads of 128, 1370 cycles, and reads 32 KB from LDS.  Four
// prompt chunks of 200 to 2000 tokens behind up to 12000, 32 heads of 128 over 8,
// int8: 600 us, 850 TFLOP/s; by counters the SIMDs' vector units are busy for 46% of
// the launch and the matrix units for 35%, LDS for 26% without a bank conflict: two
// waves a SIMD, which registers limit it to, hardly overlap the two.  (Most of the
// vector work is the softmax's, not the conversions': eight waves for heads of 128,
// 256 rows, halve these and took the same time, and 30% more where workgroups are
// few.)  A tile of a lone workgroup takes 1.65 us for heads of 128 and 1.8 for 256
// (the products alone 0.43), of two that share a CU 2.1 and 2.25.  A prompt of 4099
// tokens, 10 heads of 256 over 2, E4M3: 131 us, 660 TFLOP/s, as long as the 65 tiles
// of its last rows take, while a workgroup walks 33 on average (vector 28%, matrix
// 27%).  The same in int8: 165 us; eight waves of 254 registers leave room for one
// workgroup a CU, of which there are 328 for 256 CUs.
#pragma once

#include "kv_attn_common.hpp"

namespace w4k {

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
__global__ __launch_bounds__(kv_tile_waves(D, TYPE) * kWave, 2) void kv_tile_kernel(KvAttnArgs a,
                                                                                             float* part_o,
                                                                                             float* part_ml) {
  constexpr int NC = kKvTileCols, W = kv_tile_waves(D, TYPE), HS = kv_tile_share(D);
  constexpr int KC = D / 64;              // 16-byte pieces of a key a lane multiplies
  constexpr int NP = 4 / HS;              // 16-entry pieces of a tile that a wave scores
  constexpr int DT = D / 16, DH = DT / HS;  // 16-row pieces of the output, and those a wave owns
  constexpr int KU = 4 * KC, VU = DT;     // 64-lane pieces of a tile's keys and values
  constexpr int KL = KU / W, VL = VU / W;   // of which a wave loads
  static_assert(KU % W == 0 && VU % W == 0 && KC % KL == 0, "each wave loads the same");
  constexpr int NB = HS == 1 ? 2 : 1;       // buffers
  constexpr int AHEAD = D == 256 ? 3 : 4;   // operands read ahead of their products, as registers allow
  __shared__ kv_u32x4 s_k[NB][KU * 2 * kWave];      // [piece t][sum step][lane]
  __shared__ kv_u32x4 s_v[NB][VU * 2 * kWave];      // [piece d][sum step][lane]
  __shared__ kv_u32x4 s_p[HS == 2 ? W : 1][NC][kWave];      // a wave's weights as an operand
  __shared__ float s_m[W][NC * 16];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int x = lane & 15, g = lane >> 4;
  const int half = HS == 2 ? wave & 1 : 0;
  const int tt = kv_token_of(a, kv_tile_rows(D, TYPE));
  // Heads run fastest: a head's workgroups share an XCD's L2 (eight heads), and
  // the last tokens, which attend most, go first for every head (with a head's
  // tiles together, the last head's long ones began late: 770 us instead of 638).
  const int kh = blockIdx.x % a.c.heads;
  const int u = (gridDim.x - 1 - blockIdx.x) / a.c.heads;
  const int r = __builtin_amdgcn_readfirstlane(kv_tile_owner(a.token_start, a.requests, tt, u));
  if (r < 0) return;
  const int i0 = (u - a.token_start[r] / tt - r) * tt;
  const int n = a.token_start[r + 1] - a.token_start[r];
  const int live_tokens = min(min(n, a.max_new), a.tokens - a.token_start[r]);
  if (kv_few_rows(a, n) || i0 < 0 || i0 >= live_tokens || a.token_start[r] < 0) return;
  const int here = min(tt, live_tokens - i0);       // the workgroup's tokens
  const int live = here * a.group;                  // and rows
  const KvRows rows = kv_rows_of(a, r, i0, i0 + here - 1);
  const int shift = a.c.page_shift, P = 1 << shift;
  // the part of the cache (all of it if a.parts is 1) that this workgroup walks
  const KvParts parts = kv_parts_of(a, rows);
  const int part = blockIdx.y;
  if (part >= parts.count) return;
  const int part_begin = (parts.first + part) * a.part;
  const int part_end = (int)min((long long)part_begin + a.part, (long long)rows.end);

  // this pair of waves' rows
  const int wrow = wave / HS * NC * 16;
  kv_bf16x8 q[NC][2 * KC];
  KvLaneRows<NC> lr;
  int out_at[NC];
  const int pos0 = rows.seq - rows.n + i0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int row = min(wrow + 16 * c + x, live - 1);
    const int i = kv_token_of(a, row), h = kh * a.group + row - i * a.group;
    const int t = rows.first + i0 + i;
    const bool ok = wrow + 16 * c + x < live;
    lr.hi[c] = ok ? min(pos0 + i, rows.end - 1) : -1;
    lr.lo[c] = a.window > 0 ? pos0 + i - a.window + 1 : 0;
    out_at[c] = ok ? t * a.q_heads + h : -1;
    const uint16_t* qp = a.q + t * a.q_stride + (size_t)h * D + 16 * g;
#pragma unroll
    for (int k = 0; k < 2 * KC; ++k) q[c][k] = kv_query8(qp + 64 * (k >> 1) + 8 * (k & 1), a.q_sign);
  }
  // entries that some row of the pair attends, and those that every row does
  const int first_pos = pos0 + kv_token_of(a, min(wrow, live - 1));
  const int last_pos = pos0 + kv_token_of(a, min(wrow + NC * 16, live) - 1);
  const int any_hi = wrow < live ? min(last_pos, rows.end - 1) : -1;
  const int any_lo = a.window > 0 ? first_pos - a.window + 1 : 0;
  const int all_hi = min(first_pos, rows.end - 1);
  const int all_lo = a.window > 0 ? last_pos - a.window + 1 : 0;

  kv_f32x4 o[NC][DH];
  float m[NC], l[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    m[c] = kKvNone;
    l[c] = 0.0f;
#pragma unroll
    for (int d = 0; d < DH; ++d) o[c][d] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // Pages of a tile: lane (x, g) needs that of 16-entry block x / 4 for its keys
  // and of block g for its values and scores.  They are read two tiles ahead of
  // their use and checked only there, so that nothing waits for them.
  const int32_t* table = a.table + (size_t)r * a.width;
  struct Pages {
    int k, v;
  };
  auto pages = [&](int j0) W4K_INLINE {
    return Pages{table[min((j0 + 16 * (x >> 2)) >> shift, a.width - 1)], table[min((j0 + 16 * g) >> shift, a.width - 1)]};
  };
  auto checked = [&](int j0, Pages p) W4K_INLINE {
    return Pages{j0 + 16 * (x >> 2) < rows.end && p.k >= 0 && p.k < a.c.pages ? p.k : -1,
                 j0 + 16 * g < rows.end && p.v >= 0 && p.v < a.c.pages ? p.v : -1};
  };
  // What of an address does not change over the tiles is one number a lane; a
  // wave's units of keys lie within one piece of 16 entries (KL divides KC)
  const uint32_t head_bytes = (uint32_t)D << shift;      // one head's codes of a page
  const uint32_t page_bytes = (uint32_t)a.c.heads * head_bytes;      // <= 2^10 * 2^16
  const uint8_t* const k_lane = a.c.k + (size_t)kh * head_bytes + 4 * (wave * KL / KC) * D + 64 * (wave * KL % KC) +
                                (x & 3) * D + 16 * g;
  const uint8_t* const v_lane = a.c.v + (size_t)kh * head_bytes + ((16 * wave * VL + x) << shift);
  kv_u32x4 kc[KL], vc[VL];
  auto load_keys = [&](int j0, int page) W4K_INLINE {
    const uint8_t* ka = k_lane + (uint64_t)(uint32_t)max(page, 0) * page_bytes + ((j0 + 16 * (x >> 2)) & (P - 1)) * D;
#pragma unroll
    for (int i = 0; i < KL; ++i) kc[i] = *reinterpret_cast<const kv_u32x4*>(ka + 64 * i);
  };
  auto load_values = [&](int j0, int page) W4K_INLINE {
    const uint8_t* va = v_lane + (uint64_t)(uint32_t)max(page, 0) * page_bytes + ((j0 + 16 * g) & (P - 1));
#pragma unroll
    for (int i = 0; i < VL; ++i) vc[i] = *reinterpret_cast<const kv_u32x4*>(va + (16 * i << shift));
  };
  float ks, vs;
  auto load_scales = [&](int page) W4K_INLINE {
    const uint32_t at = (uint32_t)max(page, 0) * (uint32_t)a.c.heads + kh;
    ks = bf16_lo(a.c.ks[at]) * a.scale_log2;
    vs = bf16_lo(a.c.vs[at]);
  };
  auto put_keys = [&](int b) W4K_INLINE {
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      const int unit = wave * KL + i;
      s_k[b][unit * 2 * kWave + lane] = __builtin_bit_cast(kv_u32x4, kv_bf16_of8<TYPE>(kc[i].x, kc[i].y));
      s_k[b][(unit * 2 + 1) * kWave + lane] = __builtin_bit_cast(kv_u32x4, kv_bf16_of8<TYPE>(kc[i].z, kc[i].w));
    }
  };
  auto put_values = [&](int b, int j0, int page) W4K_INLINE {
    // E4M3 codes of entries that no row attends may be NaN, which weights of 0
    // would not hide: where the tile has such entries, their codes become 0
    if (TYPE == W4A16_KV_FP8 && !(j0 >= rows.begin && j0 + kKvTile <= rows.end && __all(page >= 0))) {
      const int first = kv_opaque(j0 + 16 * g);
      const kv_u32x4 exist = kv_existing_bytes(rows.begin - first, page >= 0 ? rows.end - first : 0);
#pragma unroll
      for (int i = 0; i < VL; ++i) vc[i] = vc[i] & exist;
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int unit = wave * VL + i;
      s_v[b][unit * 2 * kWave + lane] = __builtin_bit_cast(kv_u32x4, kv_f16_of8<TYPE>(vc[i].x, vc[i].y));
      s_v[b][(unit * 2 + 1) * kWave + lane] = __builtin_bit_cast(kv_u32x4, kv_f16_of8<TYPE>(vc[i].z, vc[i].w));
    }
  };

  int j0 = max(part_begin, rows.begin & ~(kKvTile - 1));
  int page = -1;                  // of this tile's values
  Pages next = {-1, -1}, after = {-1, -1};
  if (j0 < part_end) {
    const Pages first = checked(j0, pages(j0));
    next = checked(j0 + kKvTile, pages(j0 + kKvTile));
    after = pages(j0 + 2 * kKvTile);
    page = first.v;
    load_keys(j0, first.k);
    load_values(j0, page);
    load_scales(page);
    put_keys(0);
    if constexpr (HS == 1)
      put_values(0, j0, page);
    else
      load_keys(j0 + kKvTile, next.k);
  }
  __syncthreads();
  for (int b = 0; j0 < part_end; j0 += kKvTile, b ^= NB - 1) {
    const bool active = j0 <= any_hi && j0 + kKvTile > any_lo;      // of this pair's rows
    const int jl = j0 + 16 * g + 8 * half;       // this lane's first entry
    const bool ok = page >= 0;
    const bool whole = __all(page >= 0) && j0 + kKvTile - 1 <= all_hi && j0 >= all_lo;
    const float vs_now = vs < kKvMinScale ? kKvMinScale : vs;       // 0 in a page never begun; NaN stays
    const float ks_now = ks, lv = __builtin_amdgcn_logf(vs_now), rv = __builtin_amdgcn_rcpf(vs_now);
    const Pages second = checked(j0 + 2 * kKvTile, after);
    after = pages(j0 + 3 * kKvTile);
    if constexpr (HS == 1) {
      load_keys(j0 + kKvTile, next.k);
      load_values(j0 + kKvTile, next.v);
      load_scales(next.v);
    }
    kv_f32x4 s[NC][NP];
    float top[NC];
    if (active) {
#pragma unroll
      for (int t = 0; t < NP; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c) s[c][t] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      kv_stream_operands<AHEAD, NP * 2 * KC>(
          [&](int i) W4K_INLINE { return s_k[b][(2 * half * 2 * KC + i) * kWave + lane]; },
          [&](int i, kv_u32x4 f) W4K_INLINE {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              s[c][i / (2 * KC)] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(kv_bf16x8, f), q[c][i % (2 * KC)], s[c][i / (2 * KC)], 0, 0, 0);
          });
      kv_tile_max<NC, NP>(s, lr, jl, ks_now, lv, whole, ok, top);
      if constexpr (HS == 2) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (g == 0) s_m[wave][16 * c + x] = top[c];
      }
    }
    if constexpr (HS == 2) __syncthreads();
    kv_f16x8 w[NC][NP / 2];
    if (active) {
      float fade[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if constexpr (HS == 2) top[c] = fmaxf(top[c], s_m[wave ^ 1][16 * c + x]);
        const float m_new = kv_new_max(m[c], top[c]);
        fade[c] = __builtin_amdgcn_exp2f(m[c] - m_new);
        m[c] = m_new;
      }
      kv_weights<NC, NP>(s, lr, jl, ks_now, lv, rv, whole, ok, m, fade, l, w);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if constexpr (HS == 2) s_p[wave][c][lane] = __builtin_bit_cast(kv_u32x4, w[c][0]);
        if (__any(fade[c] != 1.0f))
#pragma unroll
          for (int d = 0; d < DH; ++d) o[c][d] *= fade[c];
      }
    }
    if constexpr (HS == 2) {
      put_values(0, j0, page);
      put_keys(0);                               // of the next tile
      load_values(j0 + kKvTile, next.v);
      load_scales(next.v);
      __syncthreads();
      load_keys(j0 + 2 * kKvTile, second.k);
    }
    if (active) {
      kv_f16x8 p[NC][2];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          p[c][h] = HS == 1 ? w[c][h % (NP / 2)] : __builtin_bit_cast(kv_f16x8, s_p[(wave & ~1) + h][c][lane]);
      kv_stream_operands<AHEAD, DH * 2>(
          [&](int i) W4K_INLINE { return s_v[b][(half * DH * 2 + i) * kWave + lane]; },
          [&](int i, kv_u32x4 f) W4K_INLINE {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              o[c][i / 2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(kv_f16x8, f), p[c][i % 2],
                                                                   o[c][i / 2], 0, 0, 0);
          });
    }
    if constexpr (HS == 1) {
      put_keys(b ^ 1);
      put_values(b ^ 1, j0 + kKvTile, next.v);
      __syncthreads();
    }
    page = next.v;
    next = second;
  }

  // a row's sum over both waves
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    l[c] += __shfl_xor(l[c], 16);
    l[c] += __shfl_xor(l[c], 32);
    if (HS == 2 && g == 0) s_m[wave][16 * c + x] = l[c];
  }
  if constexpr (HS == 2) __syncthreads();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (out_at[c] < 0) continue;
    const float sum = HS == 1 ? l[c] : s_m[wave & ~1][16 * c + x] + s_m[wave | 1][16 * c + x];
    const int d0 = 16 * DH * half + 4 * g;
    if (parts.count == 1) {
      const float inverse = kv_inverse(sum);
      uint16_t* out = a.out + (size_t)out_at[c] * D + d0;
#pragma unroll
      for (int d = 0; d < DH; ++d) kv_store4(out + 16 * d, o[c][d], inverse);
    } else {
      const size_t at = (size_t)out_at[c] * a.parts + part;
#pragma unroll
      for (int d = 0; d < DH; ++d) *reinterpret_cast<kv_f32x4*>(part_o + at * D + d0 + 16 * d) = o[c][d];
      if (g == 0 && half == 0) {
        part_ml[kKvTileStats * at] = m[c];
        part_ml[kKvTileStats * at + 1] = sum;
      }
    }
  }
}

// Joins the parts of a row in their order: D / 4 threads a row (bound by two reads
// from L2, one after the other: 4 us).  Rows that lie
// in one part are written already, those of requests of few rows are not the
// tiles'.
template <int D, int TYPE>
__global__ __launch_bounds__(kKvJoinThreads) void kv_tile_join_kernel(KvAttnArgs a, const float* part_o,
                                                                      const float* part_ml) {
  const int row = blockIdx.x * (kKvJoinThreads / (D / 4)) + threadIdx.x / (D / 4);      // of `out`
  const int d = 4 * (threadIdx.x % (D / 4));
  const int t = row / a.q_heads;
  if (t >= a.tokens || t < a.token_start[0]) return;
  int r = 0;                                                    // the last request that begins at or before t
  for (int count = a.requests; count > 1;) {
    const int step = count >> 1;
    if (a.token_start[r + step] <= t) r += step;
    count -= step;
  }
  const int n = a.token_start[r + 1] - a.token_start[r], i = t - a.token_start[r];
  if (a.token_start[r] < 0 || i >= min(n, a.max_new) || kv_few_rows(a, n)) return;
  // the rows of its workgroup
  const int tt = kv_token_of(a, kv_tile_rows(D, TYPE)), i0 = i / tt * tt;
  const int here = min(tt, min(min(n, a.max_new), a.tokens - a.token_start[r]) - i0);
  const KvParts parts = kv_parts_of(a, kv_rows_of(a, r, i0, i0 + here - 1));
  if (parts.count <= 1) return;
  const size_t at = (size_t)row * a.parts;
  // eight parts at a time, so that their loads do not wait for each other (the
  // last one's are repeated, with factor 0)
  constexpr int U = 8;
  const kv_f32x2* ml = reinterpret_cast<const kv_f32x2*>(part_ml) + at;
  float top = kKvNone;
  for (int p0 = 0; p0 < parts.count; p0 += U)
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[min(p0 + u, parts.count - 1)][0]);
  float sum_l = 0.0f;
  kv_f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int p0 = 0; p0 < parts.count; p0 += U) {
    kv_f32x2 s[U];
    kv_f32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = min(p0 + u, parts.count - 1);
      s[u] = ml[p];
      v[u] = *reinterpret_cast<const kv_f32x4*>(part_o + (at + p) * D + d);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p0 + u >= parts.count) break;
      const float f = __builtin_amdgcn_exp2f(s[u][0] - top);
      sum_l = __builtin_fmaf(s[u][1], f, sum_l);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(v[u][e], f, sum[e]);
    }
  }
  kv_store4(a.out + (size_t)row * D + d, sum, kv_inverse(sum_l));
}

}  // namespace w4k
