// Attention over the paged 8-bit cache for requests of few new tokens (decode
// and verify): the cache is streamed once, split over workgroups along its
// length.
//
// Rows.  Request r with n new tokens has n * G rows a cache head (G query heads
// share it); a workgroup takes NC * 16 of them as the columns of the matrix
// products, so every key and value is loaded once for all of them.
//
// Products, transposed so that no score or weight changes lanes:
//   S^T [T entries x 16 rows] = K Q^T      v_mfma_f32_16x16x32_bf16, A = K
//   O^T [D x 16 rows]        += V^T P^T    v_mfma_f32_16x16x32_f16,  A = V^T
// (operand layout of both: lane l supplies A[l % 16][8 (l / 16) .. +7] and
// B[8 (l / 16) .. +7][l % 16] and receives C[4 (l / 16) + i][l % 16]).  A wave's
// tile is T = 32 entries.  The sum index of a product may be permuted and its A rows
// assigned freely, which is used twice, with x = l % 16, g = l / 16, E = T / 4:
//   * keys: matrix row 4 b + i of piece t is entry E b + 4 t + i of the tile, so
//     lane (x, g) receives the scores of entries E g .. E g + E - 1 for row x,
//     four a piece.  Its 16 codes 64 c + 16 g .. + 15 of a key enter two
//     products; the queries are loaded in the same order;
//   * values: those E entries are then exactly what lane (x, g) must supply of
//     P^T, and the matching A operand is E contiguous codes of row d = 16 dt + x
//     of the page (tokens are innermost in v).
// So a lane's entries lie in one page (pages hold a multiple of 16) and one
// key scale and one value scale serve all its scores.
//
// Arithmetic.  Key codes are exact in bf16 and the queries are bf16: the dot
// products are fp32 sums of exact products.  With u_j = s_j * (key scale *
// scale * log2 e) + log2(value scale) the weights w_j = 2^(u_j - m), m the
// running maximum of u, contain the value scale, so O = sum w_j * code_j needs
// no scaling of codes, and the softmax sum is l = sum w_j / (value scale).  w
// (times a constant, see kv_new_max) is rounded to fp16 for the second product (2^-12 relative; bf16
// would add 2^-9, as much as the output's own rounding); value codes are exact
// in fp16.  m, l and O are fp32.
//
// Workgroup.  Its four waves take T entries each of a step of 4 T: each
// multiplies its own keys, the waves agree on the step's maximum (16 rows'
// maxima a wave through LDS), put their weights into LDS as finished operands,
// and then each wave multiplies all weights of the step with the values of its
// own quarter of the head's elements.  So the output is never summed over
// waves, and a wave holds D / 4 of it.
//
// Loads.  A wave loads keys and values in memory order, 1024 consecutive bytes
// an instruction where pages allow, a step ahead, into registers; they pass
// through T D bytes of LDS of the wave's own (keys, then values) into operand
// order.  (Loading operands straight from the cache, 16 rows of 64 bytes an
// instruction, kept the L1 busy four times as long and halved whole lines
// between two fetches: 3 x 105k entries, 8 heads of 128, 128 us against 113.)
// What a load brings is first touched a step later: converting a scale or
// checking a page number where it is loaded waits for all loads before it
// (48 decode requests 67 us instead of 63, see below).
//
// Split.  A workgroup takes one chunk of the cache, cut at fixed positions
// (multiples of 2^a.chunk_shift, which depends on max_len alone): its (m, l, O)
// begin anew, and kv_join_kernel adds them in chunk order.  A row's result
// depends on its entries and position alone: it is bitwise the same in any
// batch and for any number of candidates (a masked entry or step adds exact
// zeros and leaves the maximum).
//
// Bound and measured, both kernels and their launches: the cache's bytes once.
// 3 requests of 90001 to 120001 entries, 8 heads of 128, int8, 4 query heads
// each: 645 MB, 114 us, 5.7 TB/s (the loads alone 5.9).  48 of 300 to 6000, E4M3,
// pages of 32: 313 MB, 60 us, 5.2 TB/s.  With less to read, the start of a
// workgroup (3 us until its first entries arrive) and the latency of its steps: one
// token in 717 entries, a step a workgroup, 6.3 us and the join 3.6.  16 verify
// batches of 2 to 6 tokens in 1000 to 9000 entries, 10 heads of 256 over 2, 70 MB: 25.6
// us and the join 4.5.  A workgroup that has entries lives 18 us on average there (by
// its wave cycles), for four steps of 128 entries and 12 to 30 rows; its waves wait for
// 37% of that, and vector, matrix and LDS units are busy for 18, 7 and 10% of the 25.6
// us.  What makes up the 8 us between that life and the kernel's has not been measured.
#pragma once

#include <type_traits>

#include "kv_attn_common.hpp"

namespace w4k {

constexpr int kKvSplitWaves = 4;
constexpr int kKvSplitTile = 32;                   // entries a wave takes at once (T above)
constexpr int kKvSplitAhead = 2;                    // operands read from LDS ahead of their products
constexpr int kKvGridRequests = 32768;             // requests on the grid's y axis (more go to z)

// Waves per SIMD that the registers have to allow: what they do without spilling
// (a reload of a spilled register would wait for the loads in flight).
constexpr int kv_split_occupancy(int D, int NC) { return D == 256 ? 2 : D == 128 || NC == 2 ? 3 : 4; }

// Queries stay in LDS where a third wave a SIMD, or the products' operands, need
// their registers (16 requests of 16 tokens, 4 query heads of 128: 71 us instead of
// 79); with D = 256 there is room to read those of the next piece ahead.
constexpr bool kv_split_queries_in_lds(int D, int NC) { return NC == 2 && D >= 128; }

// What the waves of a workgroup share.
template <int D, int NC>
struct KvSplitShared {
  static constexpr int W = kKvSplitWaves;
  kv_u32x4 stage[W][kKvSplitTile * D / (16 * kWave) * kWave];      // a wave's keys, then its values
  kv_u32x4 p[W][NC][kWave];                                        // the step's weights as operands
  kv_u32x4 q[kv_split_queries_in_lds(D, NC) ? NC * 2 * (D / 64) : 0][kWave];
  float m[W][NC * 16], l[W][NC * 16];
};

// Behind shared entries (Args = KvSharedArgs) a request's own ones alone are taken; over them
// (KvPrefixArgs) the rows of all requests are taken as if they were one's, each with its own
// last entry.  Both give partial results, which another kernel joins.
// r: the request (PREFIX: 0); block: its cache head, rows and chunk.
template <int D, int TYPE, int NC, class Args>
__device__ __forceinline__ void kv_split_body(const Args& a, KvSplitShared<D, NC>& shared, int block, int r, float* part_o,
                                              float* part_ml) {
  constexpr bool SHARED = kv_behind_shared<Args>, PREFIX = kv_over_shared<Args>;
  constexpr int W = kKvSplitWaves;
  constexpr int T = kKvSplitTile, E = T / 4, STEP = W * T;
  constexpr int NP = T / 16;                       // pieces of scores
  constexpr bool Q_LDS = kv_split_queries_in_lds(D, NC);
  constexpr int QB = D == 256 ? 2 : 1;             // pieces of queries in registers
  constexpr int KC = D / 64;                       // 16-byte pieces of a key a lane multiplies
  constexpr int DW = D / 16 / W;                   // 16-row pieces of the output a wave owns
  constexpr int LD = T * D / (16 * kWave);         // 16-byte loads a lane and step, keys and values each
  auto& s_stage = shared.stage;
  auto& s_p = shared.p;
  auto& s_q = shared.q;
  auto& s_m = shared.m;
  auto& s_l = shared.l;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int x = lane & 15, g = lane >> 4;
  // Workgroups go to the eight XCDs in turn.  Heads run fastest, then row
  // groups, then a request's chunks, so that every request is spread over all
  // XCDs (with requests fastest, those of ragged batches were unevenly loaded)
  if (r >= a.requests) return;
  int chunk_shift = a.chunk_shift;
  if constexpr (PREFIX) chunk_shift = a.part_shift;
  const int kh = block % a.c.heads;
  block /= a.c.heads;
  const int row0 = block % a.row_groups * (NC * 16);
  block /= a.row_groups;                                   // which of the request's chunks
  const int shift = a.c.page_shift, P = 1 << shift;
  const int32_t* table = a.table + (size_t)r * a.width;
  // Pages of a step's 16-entry blocks, block x in lane (x, g); others fetch them
  // from there.  They are looked up whatever the request's length (beyond it
  // they are masked), so the first step's do not wait for the length.
  auto pages = [&](int j0) W4K_INLINE {
    return table[min((j0 + 16 * x) >> shift, a.width - 1)];
  };
  auto checked = [&](int j0, int page) W4K_INLINE {
    return (j0 + 16 * x) >> shift < a.width && page >= 0 && page < a.c.pages ? page : -1;
  };
  int page = 0, page_after = 0;
  int page_of = -1;      // SHARED: where the page that is looked up first begins, if shared_len is its bound
  if constexpr (SHARED) {
    page_of = block == 0 ? a.max_shared & ~(STEP - 1) : ((a.max_shared >> chunk_shift) + block) << chunk_shift;
    if (a.width > 0) page = pages(page_of);
  } else if (a.window == 0 && a.width > 0) {
    page = pages(block << chunk_shift);
  }
  const int i_first = kv_token_of(a, row0), i_last = kv_token_of(a, row0 + NC * 16 - 1);
  KvRows rows;
  int last = -1;      // PREFIX: the last entry that token `lane` attends (there are at most 64)
  if constexpr (PREFIX) {
    const KvOwners owners = kv_owners(a);
    rows.first = a.token_start[0];
    rows.n = a.token_start[a.requests] - rows.first;
    rows.live = min(rows.n, a.tokens - rows.first);
    if (rows.first < 0 || row0 >= rows.live * a.group) return;
    const int entries = (int)min((long long)kv_shared_entries(a), (long long)a.width << shift);
    last = kv_last_shared(a, owners, rows.first + min(lane, rows.live - 1), entries);
    if (lane >= rows.live) last = -1;
    int end = lane >= i_first && lane <= i_last ? last + 1 : 0;
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) end = max(end, __shfl_xor(end, off));
    rows.end = __builtin_amdgcn_readfirstlane(end);
    rows.begin = rows.seq = 0;
    if (rows.end == 0) return;
  } else {
    rows = kv_rows_of(a, r, i_first, i_last);
    if (!kv_few_rows(a, rows.n)) return;
  }
  const int live = rows.live * a.group;                    // rows of the request
  if (row0 >= live) return;
  if constexpr (SHARED) {
    kv_keep_own(a, rows);
    if (rows.begin >= rows.end) return;
  }
  const int first = rows.begin >> chunk_shift;              // the group's first chunk
  const int at_begin = (first + block) << chunk_shift;
  const int at_end = (int)min((long long)at_begin + (1LL << chunk_shift), (long long)rows.end);
  if (block > 0 && at_begin >= at_end) return;

  // No load stands under a condition: entries without a page read page 0 instead
  // (in the L2 after the first) and are masked, so the waits for loads count
  // exactly and the next step's stay in flight through this one.
  // (What the loops below derive from an opaque number is computed anew each
  // step; kept over the steps it would take thirty registers.)
  constexpr int KP = D / 16, KR = kWave / KP;      // 16-byte pieces a key, keys an instruction
  constexpr int VR = D / W;                        // rows of values a wave owns
  const uint32_t page_head_bytes = (uint32_t)D << shift;      // one head's codes of a page, keys or values
  auto page_offset = [&](int page) W4K_INLINE {
    return (uint64_t)(uint32_t)max(page, 0) * ((uint64_t)a.c.heads * page_head_bytes);
  };
  auto lane_value = [](uint64_t v, int from) W4K_INLINE {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), from) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, from);
  };
  const uint8_t* const k_head = a.c.k + (size_t)kh * page_head_bytes;
  const uint8_t* const v_head = a.c.v + (size_t)kh * page_head_bytes + (size_t)(VR * wave << shift);
  kv_u32x4 kc[LD], vc[LD];
  uint16_t ks, vs;      // bits, converted where used: a conversion here would wait for the loads
  bool page_ok;
  const int my_block = (T * wave + E * g) >> 4;    // of this lane's scores
  // keys: piece 64 i + lane of the wave's T keys is lane's i-th
  auto load_keys = [&](int j0, int page) W4K_INLINE {
    const uint64_t off = page_offset(page);
#pragma unroll
    for (int b = 0; b < T / 16; ++b) {
      const int j = j0 + T * wave + 16 * b;
      const uint8_t* ka = k_head + lane_value(off, T / 16 * wave + b) + (j & (P - 1)) * D;
#pragma unroll
      for (int i = 0; i < 16 / KR; ++i) kc[b * (16 / KR) + i] = kv_load(ka + 16 * lane + 1024 * i);
    }
    const int sp = __shfl(page, my_block);
    page_ok = sp >= 0;
    const uint32_t sph = (uint32_t)max(sp, 0) * (uint32_t)a.c.heads + kh;      // pages * heads < 2^32: see the host's check
    ks = a.c.ks[sph];
    vs = a.c.vs[sph];
  };
  // Values: a wave's VR rows of the step, page by page, each row of a page a
  // power of two of pieces (16-entry blocks).  The bits of a piece's number
  // 64 i + lane are (page, row, block in page), so what depends on i and on the
  // lane are disjoint parts of them.
  const int bs = min(shift - 4, __builtin_ctz(STEP / 16));    // log2 of a page's blocks in the step
  const int pps = __builtin_ctz(VR) + bs;                     // log2 of a page's pieces
  const int in_page = (1 << pps) - 1;
  const int lane_page_0 = lane >> pps, lane_row = (lane & in_page) >> bs, lane_blk = lane & ((1 << bs) - 1);
  const int value_lane = lane_row * P + lane_blk * 16;
  auto load_values = [&](int j0, int page) W4K_INLINE {
    const uint64_t off = page_offset(page);
    const uint8_t* const v0 = v_head + (j0 & (P - 1));
    if (pps >= 6) {       // a page's pieces fill an instruction: one page for all lanes
#pragma unroll
      for (int i = 0; i < LD; ++i)
        vc[i] = kv_load(v0 + lane_value(off, (i * kWave >> pps) << bs) + ((i * kWave & in_page) >> bs << shift) +
                        value_lane);
    } else {
      const int lane_page = kv_opaque(lane >> pps);
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int at = ((i * kWave >> pps) + lane_page) << bs;
        const uint64_t o = (uint64_t)(uint32_t)__shfl((int)(off >> 32), at) << 32 | (uint32_t)__shfl((int)off, at);
        vc[i] = kv_load(v0 + o + value_lane);
      }
    }
  };
  // Their places in LDS (numbers of 16-byte units), permuted so that the writes
  // in memory order and the reads in operand order both spread over the banks:
  // piece p of key r lies at KP r + (p ^ key_turn(r)), block b of value row r at
  // VR b + (r ^ value_turn(b)); the turns are linear over xor, so a lane's
  // places are one number of its own combined with constants of i.
  auto key_turn = [](int r) W4K_INLINE {
    // (r mod 4 and r / E are what tells the keys apart that 16 lanes read at once)
    return D == 64 ? (r >> 1 & 1) | (r >> 2 & 2) : (r & 3) | (r >> 1 & (D == 128 ? 4 : 12));
  };
  auto value_turn = [](int b) W4K_INLINE { return (b & 1) << 2 | (b & 2) | (b >> 2 & 1); };
  kv_u32x4* const stage = s_stage[wave];
  const int key_put = lane ^ key_turn(lane / KP);                  // KP r + p = lane for i = 0
  const int key_row = E * (x >> 2) + (x & 3);                      // operand row x of piece t = 0
  int key_get[KC];
#pragma unroll
  for (int k = 0; k < KC; ++k) key_get[k] = KP * key_row + ((4 * k + g) ^ key_turn(key_row));
  const int lane_block = (lane_page_0 << bs) + lane_blk;
  const int value_put_0 = VR * lane_block + (lane_row ^ value_turn(lane_block));
  const int get_block = E * g >> 4;                                // of tile v = 0
  const int value_get = VR * get_block + (x ^ value_turn(get_block));
  auto put_keys = [&]() W4K_INLINE {
#pragma unroll
    for (int i = 0; i < LD; ++i) stage[i * kWave + (key_put ^ key_turn(i * KR))] = kc[i];
  };
  auto put_values = [&](int j0, int page) W4K_INLINE {
    // E4M3 codes of entries that no row attends may be NaN, which weights of 0
    // would not hide: where the step has such entries, their codes become 0
    if (TYPE == W4A16_KV_FP8 &&
        !(j0 >= rows.begin && j0 + STEP <= rows.end && __all(page >= 0 || x >= STEP / 16))) {
      const int lane_first = kv_opaque(lane_block);
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int block = (i * kWave >> pps << bs) + lane_first;
        const int at = j0 + 16 * block;
        vc[i] = vc[i] & kv_existing_bytes(rows.begin - at, __shfl(page, block) >= 0 ? rows.end - at : 0);
      }
    }
    const int value_put = kv_opaque(value_put_0);
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int block = i * kWave >> pps << bs, row = (i * kWave & in_page) >> bs;
      stage[value_put ^ (VR * block + (row ^ value_turn(block)))] = vc[i];
    }
  };
  int j0 = max(at_begin, rows.begin & ~(STEP - 1));
  if (SHARED ? j0 != page_of : a.window > 0 && rows.begin < rows.end) page = pages(j0);
  page = checked(j0, page);

  // this lane's rows: queries (in the keys' order) and positions
  kv_bf16x8 q[Q_LDS ? 1 : NC][2 * KC];
  KvLaneRows<NC> lr;
  int out_at[NC];      // row of `out` (tokens * query heads < 2^31: see the host's check), or -1
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int row = min(row0 + 16 * c + x, live - 1);
    const int i = kv_token_of(a, row), t = rows.first + i, h = kh * a.group + row - i * a.group;
    const bool ok = row0 + 16 * c + x < live && t >= 0 && t < a.tokens;
    out_at[c] = ok ? t * a.q_heads + h : -1;
    if constexpr (PREFIX) {
      const int mine = __shfl(last, i);
      lr.hi[c] = ok ? mine : -1;
    } else {
      lr.hi[c] = ok ? min(rows.seq - rows.n + i, rows.end - 1) : -1;
    }
    lr.lo[c] = SHARED ? rows.begin : a.window > 0 ? rows.seq - rows.n + i - a.window + 1 : 0;
    const uint16_t* qp = a.q + (ok ? (size_t)t * a.q_stride + (size_t)h * D : 0) + 16 * g;
    if constexpr (Q_LDS) {      // the waves share the rows: each puts a quarter of the pieces (read after a barrier)
#pragma unroll
      for (int k = 0; k < 2 * KC / W; ++k) {
        const int kk = wave + W * k;
        s_q[c * 2 * KC + kk][lane] =
            __builtin_bit_cast(kv_u32x4, kv_query8(qp + 64 * (kk >> 1) + 8 * (kk & 1), a.q_sign));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2 * KC; ++k) q[c][k] = kv_query8(qp + 64 * (k >> 1) + 8 * (k & 1), a.q_sign);
    }
  }
  if constexpr (Q_LDS) __syncthreads();
  // positions that every row of the group attends need no mask
  int all_hi = min(rows.seq - rows.n + i_first, rows.end - 1);
  if constexpr (PREFIX) {
    all_hi = lane >= i_first && lane <= min(i_last, rows.live - 1) ? last : rows.end - 1;
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) all_hi = min(all_hi, __shfl_xor(all_hi, off));
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);
  }
  const int all_lo = SHARED         ? rows.begin
                     : a.window > 0 ? rows.seq - rows.n + min(i_last, rows.live - 1) - a.window + 1
                                    : 0;

  kv_f32x4 o[NC][DW];
  float m[NC], l[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    m[c] = kKvNone;
    l[c] = 0.0f;
#pragma unroll
    for (int d = 0; d < DW; ++d) o[c][d] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const bool single =      // one chunk holds all
      !SHARED && !PREFIX && first == max(rows.end - 1, rows.begin) >> chunk_shift;
  if (j0 < at_end) {
    load_keys(j0, page);
    load_values(j0, page);
    page_after = pages(j0 + STEP);
  }
  // one step; more: another one follows in this block
  auto step = [&](auto more_c) W4K_INLINE {
    constexpr bool more = decltype(more_c)::value;
    const int jw = j0 + T * wave, jl = jw + E * g;      // the wave's and this lane's first entry
    const bool whole = __all(page_ok) && jw + T - 1 <= all_hi && jw >= all_lo;
    const bool ok_now = page_ok;
    put_keys();
    const float ks_now = bf16_lo(ks) * a.scale_log2, vs_page = bf16_lo(vs);
    const float vs_now = vs_page < kKvMinScale ? kKvMinScale : vs_page;      // 0 in a page never begun; NaN stays
    int page_next = 0;
    if constexpr (more) {
      page_next = checked(j0 + STEP, page_after);
      page_after = pages(j0 + 2 * STEP);
      load_keys(j0 + STEP, page_next);
    }
    kv_f32x4 s[NC][NP];
#pragma unroll
    for (int t = 0; t < NP; ++t)
#pragma unroll
      for (int c = 0; c < NC; ++c) s[c][t] = kv_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    kv_bf16x8 qk[Q_LDS ? QB : 1][NC][2];
    auto read_queries = [&](int k) W4K_INLINE {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          qk[k % QB][c][h] = __builtin_bit_cast(kv_bf16x8, s_q[c * 2 * KC + 2 * k + h][lane]);
    };
    if constexpr (Q_LDS && QB == 2) read_queries(0);
    kv_stream_operands<kKvSplitAhead, KC * NP>(
        [&](int i) W4K_INLINE { return stage[key_get[i / NP] + 4 * (i % NP) * KP]; },
        [&](int i, kv_u32x4 kk) W4K_INLINE {
          const int k = i / NP, t = i % NP;
          if constexpr (Q_LDS)
            if (t == 0 && k + QB - 1 < KC) read_queries(k + QB - 1);
          const kv_bf16x8 a0 = kv_bf16_of8<TYPE>(kk.x, kk.y), a1 = kv_bf16_of8<TYPE>(kk.z, kk.w);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            s[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, Q_LDS ? qk[k % QB][c][0] : q[c][2 * k], s[c][t], 0, 0, 0);
            s[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, Q_LDS ? qk[k % QB][c][1] : q[c][2 * k + 1], s[c][t], 0, 0, 0);
          }
        });
    const float lv = __builtin_amdgcn_logf(vs_now), rv = __builtin_amdgcn_rcpf(vs_now);
    float top[NC], fade[NC];
    kv_tile_max<NC, NP>(s, lr, jl, ks_now, lv, whole, ok_now, top);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (g == 0) s_m[wave][16 * c + x] = top[c];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float all = kKvNone;
#pragma unroll
      for (int w = 0; w < W; ++w) all = fmaxf(all, s_m[w][16 * c + x]);
      const float m_new = kv_new_max(m[c], all);
      fade[c] = __builtin_amdgcn_exp2f(m[c] - m_new);
      m[c] = m_new;
    }
    kv_f16x8 w[NC][1];
    kv_weights<NC, NP>(s, lr, jl, ks_now, lv, rv, whole, ok_now, m, fade, l, w);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      s_p[wave][c][lane] = __builtin_bit_cast(kv_u32x4, w[c][0]);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (__any(fade[c] != 1.0f))
#pragma unroll
        for (int d = 0; d < DW; ++d) o[c][d] *= fade[c];
    put_values(j0, page);
    if constexpr (more) {
      load_values(j0 + STEP, page_next);
      page = page_next;
    }
    __syncthreads();
    constexpr int VB = T / 16;               // blocks a tile
    kv_f16x8 p[2][NC];                       // weights of two tiles: the next one's are read ahead
#pragma unroll
    for (int c = 0; c < NC; ++c) p[0][c] = __builtin_bit_cast(kv_f16x8, s_p[0][c][lane]);
    kv_stream_operands<kKvSplitAhead, W * DW>(
        [&](int i) W4K_INLINE {             // this lane's 8 entries of the row: half of a 16-byte unit
          const int v = i / DW, d = i % DW;
          return reinterpret_cast<const kv_u32x2*>(
              &stage[(value_get ^ value_turn(VB * v)) + VB * v * VR + 16 * d])[g & 1];
        },
        [&](int i, kv_u32x2 vv) W4K_INLINE {
          const int v = i / DW, d = i % DW;
          if (d == 0 && v + 1 < W)
#pragma unroll
            for (int c = 0; c < NC; ++c) p[(v + 1) % 2][c] = __builtin_bit_cast(kv_f16x8, s_p[v + 1][c][lane]);
          const kv_f16x8 av = kv_f16_of8<TYPE>(vv.x, vv.y);
#pragma unroll
          for (int c = 0; c < NC; ++c)
            o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, p[v % 2][c], o[c][d], 0, 0, 0);
        });
  };
  for (; j0 + STEP < at_end; j0 += STEP) step(std::true_type{});
  if (j0 < at_end) step(std::false_type{});      // (none where nothing is attended: zeros)

  // the chunk's result: the output itself where one chunk holds all
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    l[c] += __shfl_xor(l[c], 16);
    l[c] += __shfl_xor(l[c], 32);
  }
  if (single) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (g == 0) s_l[wave][16 * c + x] = l[c];
    __syncthreads();
  }
  const int d0 = 16 * DW * wave + 4 * g;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (out_at[c] < 0) continue;
    if (single) {
      const float inverse =
          kv_inverse(((s_l[0][16 * c + x] + s_l[1][16 * c + x]) + s_l[2][16 * c + x]) + s_l[3][16 * c + x]);
      uint16_t* out = a.out + (size_t)out_at[c] * D + d0;
#pragma unroll
      for (int d = 0; d < DW; ++d) kv_store4(out + 16 * d, o[c][d], inverse);
    } else {
      const size_t at = SHARED || PREFIX ? (size_t)out_at[c] * (a.parts + a.chunks) + (SHARED ? a.parts : 0) + block
                                         : kv_part_row(a, out_at[c], r, rows.first) * a.chunks + block;
#pragma unroll
      for (int d = 0; d < DW; ++d) *reinterpret_cast<kv_f32x4*>(part_o + at * D + d0 + 16 * d) = o[c][d];
      if (g == 0) {
        part_ml[kKvPartStats * at + 1 + wave] = l[c];     // the waves' sums, added by the join
        if (wave == 0) part_ml[kKvPartStats * at] = m[c];
      }
    }
  }
}

template <int D, int TYPE, int NC>
__global__ __launch_bounds__(kKvSplitWaves * kWave, kv_split_occupancy(D, NC)) void kv_split_kernel(
    KvAttnArgs a, float* part_o, float* part_ml) {
  __shared__ KvSplitShared<D, NC> shared;
  kv_split_body<D, TYPE, NC>(a, shared, blockIdx.x, blockIdx.z * kKvGridRequests + blockIdx.y, part_o, part_ml);
}

// Joins the chunks of one row (grid: cache head and row, request) in chunk order:
// D / 4 threads hold four elements each of one slice of the chunks, the slices'
// sums are added in slice order.  Rows whose group lies in one chunk are
// already written.  Bound by the launch and three reads that wait for each other:
// 2.7 to 4.8 us in the cases above, 6.9 for 96 rows of up to 118 chunks.
template <int D, int NC>
__global__ __launch_bounds__(kKvJoinThreads) void kv_join_kernel(KvAttnArgs a, const float* part_o,
                                                                 const float* part_ml) {
  constexpr int S = kKvJoinThreads / (D / 4);
  static_assert(kKvMaxChunks <= kKvJoinThreads, "one thread a chunk");
  __shared__ float s_f[kKvJoinThreads];
  __shared__ float s_w[2][kKvJoinThreads / kWave];
  __shared__ kv_f32x4 s_o[kKvJoinThreads];
  const int max_rows = a.split_tokens * a.group;
  const int r = blockIdx.z * kKvGridRequests + blockIdx.y;
  if (r >= a.requests) return;
  const int kh = blockIdx.x / max_rows, row = blockIdx.x % max_rows;
  const int row0 = row / (NC * 16) * (NC * 16);
  const KvRows rows = kv_rows_of(a, r, kv_token_of(a, row0), kv_token_of(a, row0 + NC * 16 - 1));
  if (!kv_few_rows(a, rows.n) || row >= rows.live * a.group) return;
  const int first = rows.begin >> a.chunk_shift;
  const int count = (max(rows.end - 1, rows.begin) >> a.chunk_shift) - first + 1;
  if (count <= 1) return;
  const int i = kv_token_of(a, row), t = rows.first + i;
  if (t < 0 || t >= a.tokens) return;
  const int out_row = t * a.q_heads + kh * a.group + row - i * a.group;
  const size_t at = kv_part_row(a, out_row, r, rows.first) * a.chunks;
  // one thread a chunk (count <= kKvMaxChunks = the block's threads); threads
  // and slices go by the chunk's place in the cache, not by the group's first
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int mc = ((int)threadIdx.x - first) & (kKvJoinThreads - 1);
  const bool mine = mc < count;
  const float* ml = part_ml + kKvPartStats * (at + (mine ? mc : 0));
  float m = ml[0], l = ((ml[1] + ml[2]) + ml[3]) + ml[4];
  // a slice's first chunks do not wait for the factors
  const int slice = threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4));
  const int c0 = (slice - first) & (S - 1);
  const float* po = part_o + at * D + d;
  kv_f32x4 v0 = {0.0f, 0.0f, 0.0f, 0.0f}, v1 = v0;
  if (c0 < count) v0 = *reinterpret_cast<const kv_f32x4*>(po + (size_t)c0 * D);
  if (c0 + S < count) v1 = *reinterpret_cast<const kv_f32x4*>(po + (size_t)(c0 + S) * D);
  m = mine ? m : kKvNone;
  float top = m;
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  if (lane == 0) s_w[0][wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kKvJoinThreads / kWave; ++w) top = fmaxf(top, s_w[0][w]);
  const float f = __builtin_amdgcn_exp2f(m - top);
  s_f[mc] = mine ? f : 0.0f;
  float sum_l = mine ? l * f : 0.0f;
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) sum_l += __shfl_xor(sum_l, off);
  if (lane == 0) s_w[1][wave] = sum_l;
  __syncthreads();
  float ll = 0.0f;
#pragma unroll
  for (int w = 0; w < kKvJoinThreads / kWave; ++w) ll += s_w[1][w];
  kv_f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](kv_f32x4 v, int c) W4K_INLINE {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(v[i], s_f[c], sum[i]);
  };
  if (c0 < count) add(v0, c0);
  if (c0 + S < count) add(v1, c0 + S);
  for (int c = c0 + 2 * S; c < count; c += S) add(*reinterpret_cast<const kv_f32x4*>(po + (size_t)c * D), c);
  s_o[threadIdx.x] = sum;
  __syncthreads();
  if (slice > 0) return;
#pragma unroll
  for (int s = 1; s < S; ++s) sum += s_o[s * (D / 4) + threadIdx.x];
  kv_store4(a.out + (size_t)out_row * D + d, sum, kv_inverse(ll));
}

}  // namespace w4k
