// Attention over the paged 8-bit cache for requests of few new tokens (decode
// and verify): the cache is streamed once, split over workgroups along its
// length.
//
// Rows.  Request r with n new tokens has n * G rows a cache head (G query heads
// share it); a workgroup takes NC * 16 of them as the columns of the matrix
// products, so every key and value is loaded once for all of them.
//
// Products, transposed so that nothing is exchanged between lanes:
//   S^T [64 entries x 16 rows] = K Q^T     v_mfma_f32_16x16x32_bf16, A = K
//   O^T [D x 16 rows]         += V^T P^T   v_mfma_f32_16x16x32_f16,  A = V^T
// (operand layout of both: lane l supplies A[l % 16][8 (l / 16) .. +7] and
// B[8 (l / 16) .. +7][l % 16] and receives C[4 (l / 16) + i][l % 16]).  The
// sum index of a product may be permuted and its A rows assigned freely, which
// is used twice, with x = l % 16 and g = l / 16:
//   * keys: matrix row 4 b + i of piece t is entry 16 b + 4 t + i of the tile, so
//     lane (x, g) receives the scores of entries 16 g .. 16 g + 15 for row x,
//     four a piece.  A lane loads 16 contiguous codes of an entry: 64 c + 16 g
//     .. + 15 of the head for c < D / 64, the two halves of which enter two
//     products; the queries are loaded in the same order;
//   * values: those 16 entries are then exactly what lane (x, g) must supply of
//     P^T, and the matching A operand is 16 contiguous codes of row d = 16 dt + x
//     of the page (tokens are innermost in v).
// So a lane's 16 entries lie in one page (pages hold a multiple of 16), one
// key scale and one value scale serve all its scores, and neither scores nor
// weights pass through LDS.
//
// Arithmetic.  Key codes are exact in bf16 and the queries are bf16: the dot
// products are fp32 sums of exact products.  With u_j = s_j * (key scale *
// scale * log2 e) + log2(value scale) the weights w_j = 2^(u_j - m), m the
// running maximum of u, contain the value scale, so O = sum w_j * code_j needs
// no scaling of codes, and the softmax sum is l = sum w_j / (value scale).
// w in [0, 1] is rounded to fp16 for the second product (2^-12 relative; bf16
// would add 2^-9, as much as the output's own rounding); value codes are exact
// in fp16.  m, l and O are fp32.
//
// Split.  Workgroups take chunks of the cache at fixed positions (multiples of
// a.chunk, which depends on max_len alone) and the four waves of one take the
// chunk's 64-entry tiles in turn; the partial (m, l, O) of the waves are joined
// in wave order, those of chunks in chunk order by kv_join_kernel.  So a row's
// result depends on its entries and position alone: it is bitwise the same in
// any batch and for any number of candidates.
#pragma once

#include "kv_attn_common.hpp"

namespace w4k {

constexpr int kKvSplitWaves = 4;

template <int D, int TYPE, int NC>
__global__ __launch_bounds__(kKvSplitWaves * kWave) void kv_split_kernel(KvAttnArgs a, float* part_o, float* part_ml) {
  constexpr int KC = D / 64;          // 16-byte pieces of a key a lane holds
  constexpr int DT = D / 16;          // 16-row pieces of the output
  constexpr int RS = D + 4;           // floats between rows in LDS
  __shared__ float s_o[kKvSplitWaves][16 * RS];
  __shared__ float s_m[kKvSplitWaves][NC * 16], s_l[kKvSplitWaves][NC * 16];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int x = lane & 15, g = lane >> 4;
  const int r = blockIdx.x;
  const int kh = blockIdx.y / a.row_groups, row0 = (blockIdx.y % a.row_groups) * (NC * 16);
  const KvRows rows = kv_rows_of(a, r, row0, NC * 16);
  const int live = min(rows.n, a.max_new) * a.group;       // rows of the request
  if (rows.n * a.group > kKvSplitRows || row0 >= live) return;
  const int chunk = rows.begin / a.chunk + (int)blockIdx.z;
  const int c_end = min((chunk + 1) * a.chunk, rows.end);
  const int c_begin = max(chunk * a.chunk, rows.begin) & ~(kKvTile - 1);
  if (c_begin >= c_end && (blockIdx.z > 0 || rows.end > rows.begin)) return;
  const int shift = a.c.page_shift, P = 1 << shift;

  // this lane's rows: queries (in the keys' order) and positions
  kv_bf16x8 q[NC][2 * KC];
  KvLaneRows<NC> lr;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int row = min(row0 + 16 * c + x, live - 1);
    const int i = row / a.group, t = rows.first + i, h = kh * a.group + row % a.group;
    const bool ok = row0 + 16 * c + x < live && t >= 0 && t < a.tokens;
    lr.hi[c] = ok ? min(rows.seq - rows.n + i, rows.end - 1) : -1;
    lr.lo[c] = a.window > 0 ? rows.seq - rows.n + i - a.window + 1 : 0;
    const uint16_t* qp = a.q + (ok ? (size_t)t * a.q_stride + (size_t)h * D : 0) + 16 * g;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      q[c][2 * k] = kv_query8(qp + 64 * k, a.q_sign);
      q[c][2 * k + 1] = kv_query8(qp + 64 * k + 8, a.q_sign);
    }
  }
  // positions that every row of the group attends need no mask
  const int all_hi = min(rows.seq - rows.n + row0 / a.group, rows.end - 1);
  const int all_lo = a.window > 0 ? rows.seq - rows.n + (min(row0 + NC * 16, live) - 1) / a.group - a.window + 1 : 0;

  kv_f32x4 o[NC][DT];
  float m[NC], l[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    m[c] = kKvNone;
    l[c] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[c][d] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int32_t* table = a.table + (size_t)r * a.width;
  // tiles go to the waves by position, whatever part of the chunk is attended
  constexpr int kStep = kKvSplitWaves * kKvTile;
  int j0 = chunk * a.chunk + wave * kKvTile;
  if (j0 < c_begin) j0 += (c_begin - j0 + kStep - 1) / kStep * kStep;
  for (; j0 < c_end; j0 += kStep) {
    // the pages of the entries this lane loads keys of (block x / 4) and scores (block g)
    auto page_of = [&](int b) {
      const int j = j0 + 16 * b;
      const int page = j < rows.end ? table[j >> shift] : -1;
      return page >= 0 && page < a.c.pages ? page : -1;
    };
    const int kp = page_of(x >> 2), vp = page_of(g);
    const bool whole = __all(kp >= 0 && vp >= 0) && j0 + kKvTile - 1 <= all_hi && j0 >= all_lo;
    const size_t kph = (size_t)max(kp, 0) * a.c.heads + kh, vph = (size_t)max(vp, 0) * a.c.heads + kh;
    const uint8_t* ka = a.c.k + (kph * P + ((j0 + 16 * (x >> 2)) & (P - 1)) + (x & 3)) * D + 16 * g;
    const uint8_t* va = a.c.v + (vph * D + x) * P + ((j0 + 16 * g) & (P - 1));
    uint4 kc[4][KC], vc[DT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int k = 0; k < KC; ++k) kc[t][k] = *reinterpret_cast<const uint4*>(ka + 4 * t * D + 64 * k);
#pragma unroll
    for (int d = 0; d < DT; ++d) vc[d] = *reinterpret_cast<const uint4*>(va + (size_t)d * 16 * P);
    const float ks = bf16_lo(a.c.ks[vph]) * a.scale_log2;
    float vs = bf16_lo(a.c.vs[vph]);
    vs = vs < kKvMinScale ? kKvMinScale : vs;     // 0 in a page that was never begun; NaN stays

    kv_f32x4 s[NC][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int c = 0; c < NC; ++c) s[c][t] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const kv_bf16x8 a0 = kv_bf16_of8<TYPE>(kc[t][k].x, kc[t][k].y), a1 = kv_bf16_of8<TYPE>(kc[t][k].z, kc[t][k].w);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          s[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, q[c][2 * k], s[c][t], 0, 0, 0);
          s[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, q[c][2 * k + 1], s[c][t], 0, 0, 0);
        }
      }
    }
    float fade[NC];
    kv_f16x8 w[NC][2];
    kv_softmax_step<NC>(s, lr, j0 + 16 * g, ks, vs, whole, vp >= 0, m, l, fade, w);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (__any(fade[c] != 1.0f))
#pragma unroll
        for (int d = 0; d < DT; ++d) o[c][d] *= fade[c];
    if (TYPE == W4A16_KV_FP8 && !whole) {
      const uint4 mask = kv_existing_bytes(vp >= 0 ? rows.end - (j0 + 16 * g) : 0);
#pragma unroll
      for (int d = 0; d < DT; ++d) vc[d] = kv_and(vc[d], mask);
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const kv_f16x8 a0 = kv_f16_of8<TYPE>(vc[d].x, vc[d].y), a1 = kv_f16_of8<TYPE>(vc[d].z, vc[d].w);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, w[c][0], o[c][d], 0, 0, 0);
        o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, w[c][1], o[c][d], 0, 0, 0);
      }
    }
  }

  // join the waves: a common maximum, then the sums in wave order
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    l[c] += __shfl_xor(l[c], 16);
    l[c] += __shfl_xor(l[c], 32);
    if (g == 0) {
      s_m[wave][16 * c + x] = m[c];
      s_l[wave][16 * c + x] = l[c];
    }
  }
  __syncthreads();
  const bool single = rows.begin / a.chunk == max(rows.end - 1, rows.begin) / a.chunk;     // one chunk holds all
  const int max_rows = a.split_tokens * a.group;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float top = kKvNone;
#pragma unroll
    for (int v = 0; v < kKvSplitWaves; ++v) top = fmaxf(top, s_m[v][16 * c + x]);
    const float fade = __builtin_amdgcn_exp2f(m[c] - top);
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<kv_f32x4*>(&s_o[wave][x * RS + 16 * d + 4 * g]) = o[c][d] * fade;
    __syncthreads();
    // four neighbouring elements of a row a thread and step
    for (int e = threadIdx.x; e < 16 * (D / 4); e += kKvSplitWaves * kWave) {
      const int rr = e / (D / 4), d = 4 * (e % (D / 4)), row = row0 + 16 * c + rr;
      if (row >= live) continue;
      float mm = kKvNone, ll = 0.0f;
#pragma unroll
      for (int v = 0; v < kKvSplitWaves; ++v) mm = fmaxf(mm, s_m[v][16 * c + rr]);
      kv_f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < kKvSplitWaves; ++v) {
        ll += s_l[v][16 * c + rr] * __builtin_amdgcn_exp2f(s_m[v][16 * c + rr] - mm);
        sum += *reinterpret_cast<const kv_f32x4*>(&s_o[v][rr * RS + d]);
      }
      if (single) {
        const int t = rows.first + row / a.group;
        if (t < 0 || t >= a.tokens) continue;
        kv_store4(a.out + ((size_t)t * a.q_heads + kh * a.group + row % a.group) * D + d, sum, ll);
      } else {
        const size_t at = (((size_t)r * a.c.heads + kh) * max_rows + row) * a.chunks + blockIdx.z;
        *reinterpret_cast<kv_f32x4*>(part_o + at * D + d) = sum;
        if (d == 0) {
          part_ml[2 * at] = mm;
          part_ml[2 * at + 1] = ll;
        }
      }
    }
    __syncthreads();
  }
}

// Joins the chunks of one row (grid: request, cache head, row) in chunk order:
// D / 4 threads hold four elements each of one slice of the chunks, the slices'
// sums are added in slice order.  Rows whose group lies in one chunk are
// already written.
constexpr int kKvJoinThreads = 256;
constexpr int kKvMaxChunks = 256;

template <int D, int NC>
__global__ __launch_bounds__(kKvJoinThreads) void kv_join_kernel(KvAttnArgs a, const float* part_o,
                                                                 const float* part_ml) {
  constexpr int S = kKvJoinThreads / (D / 4);
  __shared__ float s_f[kKvMaxChunks];
  __shared__ float s_w[kKvJoinThreads / kWave];
  __shared__ kv_f32x4 s_o[kKvJoinThreads];
  const int max_rows = a.split_tokens * a.group;
  const int r = blockIdx.x, kh = blockIdx.y, row = blockIdx.z;
  const int row0 = row / (NC * 16) * (NC * 16);
  const KvRows rows = kv_rows_of(a, r, row0, NC * 16);
  if (rows.n * a.group > kKvSplitRows || row >= min(rows.n, a.max_new) * a.group) return;
  const int first = rows.begin / a.chunk, count = max(rows.end - 1, rows.begin) / a.chunk - first + 1;
  if (count <= 1) return;
  const size_t at = (((size_t)r * a.c.heads + kh) * max_rows + row) * a.chunks;
  // one thread a chunk (count <= kKvMaxChunks = the block's threads); threads
  // and slices go by the chunk's place in the cache, not by the group's first
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int mc = ((int)threadIdx.x - first) & (kKvJoinThreads - 1);
  const bool mine = mc < count;
  const float m = mine ? part_ml[2 * (at + mc)] : kKvNone;
  const float l = mine ? part_ml[2 * (at + mc) + 1] : 0.0f;
  float top = m;
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  if (lane == 0) s_w[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kKvJoinThreads / kWave; ++w) top = fmaxf(top, s_w[w]);
  const float f = __builtin_amdgcn_exp2f(m - top);
  s_f[mc] = mine ? f : 0.0f;
  float sum_l = mine ? l * f : 0.0f;
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) sum_l += __shfl_xor(sum_l, off);
  __syncthreads();
  if (lane == 0) s_w[wave] = sum_l;
  __syncthreads();
  float ll = 0.0f;
#pragma unroll
  for (int w = 0; w < kKvJoinThreads / kWave; ++w) ll += s_w[w];
  const int slice = threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4));
  kv_f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = (slice - first) & (S - 1); c < count; c += S) {
    const kv_f32x4 v = *reinterpret_cast<const kv_f32x4*>(part_o + (at + c) * D + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(v[i], s_f[c], sum[i]);
  }
  s_o[threadIdx.x] = sum;
  __syncthreads();
  if (slice > 0) return;
#pragma unroll
  for (int s = 1; s < S; ++s) sum += s_o[s * (D / 4) + threadIdx.x];
  const int t = rows.first + row / a.group;
  if (t < 0 || t >= a.tokens) return;
  kv_store4(a.out + ((size_t)t * a.q_heads + kh * a.group + row % a.group) * D + d, sum, ll);
}

}  // namespace w4k
