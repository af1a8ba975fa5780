// C ABI of the paged 8-bit key/value cache (include/w4a16_kv.h), and the plan,
// append and dequant kernels.  The attention is in kv_attention.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv_device.hpp"
#include "kv_host.hpp"

namespace w4k {

namespace {

constexpr int kKvThreads = 256;
constexpr int kKvWaves = kKvThreads / kWave;
constexpr int kKvMaxLen = 1 << 29;

__device__ __forceinline__ int kv_length(int n) { return min(max(n, 0), kKvMaxLen); }

// ---------------------------------------------------------------------------
// plan.  A block takes kKvWaves requests, one a wave; the grid's y axis shares
// the columns and tokens of each.  The exclusive sums up to the block's first
// request are a reduction over all earlier lengths (a few strided loads a
// thread, from L2), so one launch does everything and no block waits for
// another.  Bound by its one launch and three dependent loads: 40 requests of
// 248 columns 3.6 us, 701 of 956 columns with 13k new tokens 5.3 (2.7 MB).  (The
// reduction grows with the square of the requests: of a whole call's time nothing
// shows up to 4096 requests, 32768 take 64 us, 262144 2.8 ms.)
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kKvThreads) void kv_plan_kernel(const int32_t* __restrict__ ctx_lens,
                                                             const int32_t* __restrict__ new_lens,
                                                             const int32_t* __restrict__ free_pages, int num_free,
                                                             int32_t* __restrict__ table, int width,
                                                             int32_t* __restrict__ seq_lens,
                                                             int32_t* __restrict__ token_start,
                                                             int32_t* __restrict__ slot_map,
                                                             int32_t* __restrict__ pages_used, int requests,
                                                             int tokens, int page_shift) {
  __shared__ int s_new[kKvWaves], s_need[kKvWaves];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int P = 1 << page_shift;
  const int r0 = blockIdx.x * kKvWaves;
  auto pages_of = [&](int n) { return (n + P - 1) >> page_shift; };
  int sum_new = 0, sum_need = 0;
  for (int r = threadIdx.x; r < r0; r += kKvThreads) {
    const int c = kv_length(ctx_lens[r]), n = kv_length(new_lens[r]);
    sum_new += n;
    sum_need += pages_of(c + n) - pages_of(c);
  }
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) {
    sum_new += __shfl_xor(sum_new, off);
    sum_need += __shfl_xor(sum_need, off);
  }
  if (lane == 0) {
    s_new[wave] = sum_new;
    s_need[wave] = sum_need;
  }
  __syncthreads();
  int start = 0, first = 0;
#pragma unroll
  for (int w = 0; w < kKvWaves; ++w) {
    start += s_new[w];
    first += s_need[w];
  }
  int c = 0, n = 0, held = 0, need = 0;
  const int r = r0 + wave;
  for (int x = r0; x <= r && x < requests; ++x) {   // this block's earlier requests
    start += n;
    first += need;
    c = kv_length(ctx_lens[x]);
    n = kv_length(new_lens[x]);
    held = pages_of(c);
    need = pages_of(c + n) - held;
  }
  const int step = gridDim.y * kWave, at = blockIdx.y * kWave + lane;
  if (r < requests) {
    if (at == 0) {
      seq_lens[r] = c + n;
      token_start[r] = start;
    }
    // entry b of the request's row: its own, the next free page, or none
    auto fresh = [&](int b) {
      const long long f = (long long)first + (b - held);
      return b < held + need && f < num_free ? free_pages[f] : -1;
    };
    int32_t* row = table + (size_t)r * width;
    for (int b = held + at; b < width; b += step) row[b] = fresh(b);
    for (int i = at; i < n; i += step) {
      const long long t = (long long)start + i;
      if (t >= tokens) break;
      const int b = (c + i) >> page_shift;
      const int page = b >= width ? -1 : b < held ? row[b] : fresh(b);
      // (a page number of 2^31 / P or more is outside every cache: no slot, rather than one
      // that wraps into another page)
      slot_map[t] = page >= 0 && page <= 0x7FFFFFFF >> page_shift ? (page << page_shift) + ((c + i) & (P - 1)) : -1;
    }
  }
  // the wave of the last request knows the totals
  if (r == requests - 1 || (requests == 0 && wave == 0)) {
    const int total = start + n;
    if (at == 0) {
      token_start[requests] = total;
      pages_used[0] = first + need;
    }
    for (long long t = (long long)total + at; t < tokens; t += step) slot_map[t] = -1;
  }
}

// ---------------------------------------------------------------------------
// append.  Codes are nearest(x / scale), the scale a rule on the largest |x| of
// the run (see kv_device.hpp), so a run is read for its maximum and then encoded;
// a thread keeps the first four tokens it read, and short runs are read once.  A
// block looks at `span` consecutive tokens for one cache head, keys
// or values (grid y), and quantizes every run that begins among them: the
// largest magnitude of the run (an integer maximum of bf16 bits), the scale,
// then the codes.  A run lies in one page, so its threads alone write that page
// and head.  A single run is the whole block's; several (single tokens of
// many requests) go to the block's waves in turn, without barriers.
// Bound: HBM for prompts, 3 bytes a number: 11.8k tokens, 8 heads of 128, 72 MB,
// 23 us, 3.2 TB/s (a block waits for its maximum before it writes).  Values of runs
// over 64 tokens are read again for each 64 of them that are turned: in pages of 128
// and 256 the same prompts take 30 and 31 us.  Single tokens: the launch and four
// dependent loads (the slot, the run's slots, the row and the old scale, the
// value words that the token shares with others): 64 requests 5.7 us, 24 verify
// batches 5.1.
// ---------------------------------------------------------------------------

// Codes of four bf16 entries under factor f = 1 / scale (0 where the scale is NaN).
// FP8: f is exact.  INT8: y = x f errs by less than 2^-15; a quotient of two
// 8-bit numbers of at most 127 is a tie (k + 1/2) or at least 2^-10 away from one,
// so y rounded to a multiple of 2^-13 rounds like the quotient itself.
template <int TYPE>
__device__ __forceinline__ uint32_t kv_codes4(float a, float b, float c, float d, float f, bool ok) {
  uint32_t w;
  if constexpr (TYPE == W4A16_KV_INT8) {
    const float grid = 0x1.8p10f;      // ulp 2^-13
    auto code = [&](float x) { return (uint32_t)(int)rintf((x * f + grid) - grid) & 0xFFu; };
    w = code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
  } else {
    w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a * f, b * f, 0, false);
    w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * f, d * f, (int)w, true);
  }
  return ok ? w : 0u;
}

// The four codes of a word encoded again for a larger scale (code * old / new:
// the product is exact, and the division is one, since 15-bit numerators can
// lie closer to a tie than the grid above).  Rare, and not inlined: the kernel's
// code is fetched anew for every launch of a decode step.
template <int TYPE>
__device__ __attribute__((noinline)) uint32_t kv_again4(uint32_t w, float old_s, float s) {
  return kv_code_of<TYPE>(kv_decode<TYPE, 0>(w) * old_s, s) | kv_code_of<TYPE>(kv_decode<TYPE, 1>(w) * old_s, s) << 8 |
         kv_code_of<TYPE>(kv_decode<TYPE, 2>(w) * old_s, s) << 16 |
         kv_code_of<TYPE>(kv_decode<TYPE, 3>(w) * old_s, s) << 24;
}

// Four tokens' (page offsets 4 w .. + 3) eight elements from d on, as loaded.
struct KvQuad {
  uint4 t[4];
};

constexpr int kKvTurnWords = 16;       // words (of four tokens) of a row turned through LDS at once

// One run: n entries from token row xr on, into slots slot .. slot + n - 1, by
// threads tid of N (the block, or one wave).  The work is cut into quads of
// four tokens by the page's offsets and eight elements, so that a thread holds
// whole words of the values' rows.
template <int D, int TYPE, int N>
__device__ void kv_append_run(const uint16_t* xr, int64_t stride, int n, int slot, bool is_v, int head, const KvCache& c,
                              int tid, uint32_t* s_max, uint32_t (*s_turn)[kKvTurnWords + 1]) {
  constexpr int DG = D / 8;
  const int P = 1 << c.page_shift, off = slot & (P - 1);
  const size_t ph = (size_t)(slot >> c.page_shift) * c.heads + head;
  uint16_t* scale_at = (is_v ? c.vs : c.ks) + ph;
  const float old_s = off > 0 ? bf16_lo(*scale_at) : 0.0f;
  const int w0 = off >> 2, words = ((off + n + 3) >> 2) - w0, quads = words * DG;
  auto load = [&](int q) {
    KvQuad u;
    const int t = 4 * (w0 + q / DG) - off;
    const uint16_t* at = xr + t * stride + q % DG * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u.t[i] = make_uint4(0u, 0u, 0u, 0u);
      if (q < quads && t + i >= 0 && t + i < n) u.t[i] = *reinterpret_cast<const uint4*>(at + i * stride);
    }
    return u;
  };
  uint32_t big = 0;
  auto largest = [&](const KvQuad& u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {u.t[i].x, u.t[i].y, u.t[i].z, u.t[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) big = max(big, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    }
  };
  const KvQuad kept = load(tid);      // (the first of a thread is not loaded again)
  largest(kept);
  for (int q = tid + N; q < quads; q += N) largest(load(q));
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, o));
  if constexpr (N > kWave) {
    if ((tid & (kWave - 1)) == 0) s_max[tid / kWave] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < N / kWave; ++w) big = max(big, s_max[w]);
  }
  float s = kv_scale_of<TYPE>(big);
  bool grown = false;
  if (off > 0) {
    if (!(s <= old_s))        // larger, or either is NaN
      grown = old_s == old_s;
    else
      s = old_s;
    if (!(old_s == old_s)) s = old_s;
  }
  if (tid == 0) *scale_at = (uint16_t)(__float_as_uint(s) >> 16);     // (every thread has read the old one)
  const bool ok = s == s;
  const float f = 1.0f / s;
  auto each_quad = [&](auto&& use) {
    KvQuad u = kept;
    for (int q = tid; q < quads;) {
      use(q, u);
      q += N;
      if (q < quads) u = load(q);
    }
  };
  if (!is_v) {
    uint8_t* page = c.k + ph * P * D;
    if (grown)
      for (int e = tid; e < off * (D / 4); e += N) {
        uint32_t* w = reinterpret_cast<uint32_t*>(page) + e;
        *w = kv_again4<TYPE>(*w, old_s, s);
      }
    each_quad([&](int q, const KvQuad& u) {
      const int tok = 4 * (w0 + q / DG), d = q % DG * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint2 o;
        o.x = kv_codes4<TYPE>(bf16_lo(u.t[i].x), bf16_hi(u.t[i].x), bf16_lo(u.t[i].y), bf16_hi(u.t[i].y), f, ok);
        o.y = kv_codes4<TYPE>(bf16_lo(u.t[i].z), bf16_hi(u.t[i].z), bf16_lo(u.t[i].w), bf16_hi(u.t[i].w), f, ok);
        if (tok + i >= off && tok + i < off + n) *reinterpret_cast<uint2*>(page + (size_t)(tok + i) * D + d) = o;
      }
    });
    return;
  }
  uint8_t* page = c.v + ph * P * D;
  // Puts a row's word: all of it inside the run, or only its bytes (one on the
  // run's border keeps the others, those before the run encoded again if the
  // scale grew).
  auto put = [&](int d, int tok, uint32_t fresh) {
    uint32_t* w = reinterpret_cast<uint32_t*>(page + (size_t)d * P + tok);
    if (tok < off || tok + 4 > off + n) {
      const uint32_t old = *w, kept_codes = grown && tok < off ? kv_again4<TYPE>(old, old_s, s) : old;
      uint32_t o = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o |= (tok + j < off ? kept_codes : tok + j < off + n ? fresh : old) & 0xFFu << (8 * j);
      fresh = o;
    }
    *w = fresh;
  };
  // the eight rows' words of a quad
  auto turned = [&](const KvQuad& u, uint32_t (&o)[8]) {
    const uint32_t w[4][4] = {{u.t[0].x, u.t[0].y, u.t[0].z, u.t[0].w},
                              {u.t[1].x, u.t[1].y, u.t[1].z, u.t[1].w},
                              {u.t[2].x, u.t[2].y, u.t[2].z, u.t[2].w},
                              {u.t[3].x, u.t[3].y, u.t[3].z, u.t[3].w}};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[2 * j] = kv_codes4<TYPE>(bf16_lo(w[0][j]), bf16_lo(w[1][j]), bf16_lo(w[2][j]), bf16_lo(w[3][j]), f, ok);
      o[2 * j + 1] = kv_codes4<TYPE>(bf16_hi(w[0][j]), bf16_hi(w[1][j]), bf16_hi(w[2][j]), bf16_hi(w[3][j]), f, ok);
    }
  };
  if constexpr (N > kWave) {
    // through LDS, so that a row's words leave side by side (and one token's by as many threads as it has rows)
    for (int v0 = 0; v0 < words; v0 += kKvTurnWords) {
      const int count = min(words - v0, kKvTurnWords);
      each_quad([&](int q, const KvQuad& u) {
        const int w = q / DG - v0, d = q % DG * 8;
        if (w < 0 || w >= count) return;
        uint32_t o[8];
        turned(u, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) s_turn[d + j][w] = o[j];
      });
      __syncthreads();
      for (int e = tid; e < count * D; e += N) {
        const bool full = count == kKvTurnWords;
        const int d = full ? e / kKvTurnWords : e % D, w = full ? e % kKvTurnWords : e / D;
        put(d, 4 * (w0 + v0 + w), s_turn[d][w]);
      }
      __syncthreads();
    }
  } else {
    each_quad([&](int q, const KvQuad& u) {
      uint32_t o[8];
      turned(u, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) put(q % DG * 8 + j, 4 * (w0 + q / DG), o[j]);
    });
  }
  if (grown)      // the words wholly before the run
    for (int e = tid; e < w0 * D; e += N) {
      uint32_t* w = reinterpret_cast<uint32_t*>(page + (size_t)(e / w0) * P) + e % w0;
      *w = kv_again4<TYPE>(*w, old_s, s);
    }
}

template <int D, int TYPE>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(const uint16_t* __restrict__ k, int64_t k_stride,
                                                               const uint16_t* __restrict__ v, int64_t v_stride,
                                                               const int32_t* __restrict__ slot_map, KvCache c,
                                                               int tokens, int span) {
  __shared__ uint32_t s_max[kKvWaves];
  __shared__ int s_len[kKvWaves];
  __shared__ uint32_t s_turn[D][kKvTurnWords + 1];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const uint16_t* x = (is_v ? v : k) + (size_t)head * D;
  const int64_t stride = is_v ? v_stride : k_stride;
  const int P = 1 << c.page_shift;
  const int64_t slots = (int64_t)c.pages << c.page_shift;
  const int t0 = blockIdx.x * span;
  // lane i of every wave looks at token t0 + i: does a run begin there?
  int slot = -1;
  bool begins = false;
  if (lane < span && t0 + lane < tokens) {
    slot = slot_map[t0 + lane];
    const int prev = t0 + lane > 0 ? slot_map[t0 + lane - 1] : -1;
    begins = slot >= 0 && slot < slots && ((slot & (P - 1)) == 0 || prev != slot - 1);
  }
  uint64_t runs = __ballot(begins);
  if (runs == 0) return;
  if ((runs & (runs - 1)) == 0) {
    // one run: thread i looks at its entry i
    const int i0 = __builtin_ctzll(runs), first = __shfl(slot, i0);
    const int t = t0 + i0 + (int)threadIdx.x;
    bool in_run = (first & (P - 1)) + (int)threadIdx.x < P && t < tokens;
    if (in_run) in_run = slot_map[t] == first + (int)threadIdx.x;
    const uint64_t no = ~__ballot(in_run);
    if (lane == 0) s_len[wave] = no ? __builtin_ctzll(no) : kWave;
    __syncthreads();
    int n = 0;
    for (int w = 0; w < kKvWaves; ++w) {
      n += s_len[w];
      if (s_len[w] < kWave) break;
    }
    kv_append_run<D, TYPE, kKvThreads>(x + (t0 + i0) * stride, stride, n, first, is_v, head, c, threadIdx.x, s_max,
                                       s_turn);
    return;
  }
  for (int r = 0; runs; ++r, runs &= runs - 1) {
    if (r % kKvWaves != wave) continue;
    const int i0 = __builtin_ctzll(runs), first = __shfl(slot, i0);
    int n = 0;
    for (bool more = true; more; n += kWave) {      // 64 entries at a time
      const int i = n + lane, t = t0 + i0 + i;
      bool in_run = (first & (P - 1)) + i < P && t < tokens;
      if (in_run) in_run = slot_map[t] == first + i;
      const uint64_t no = ~__ballot(in_run);
      if (no) {
        n += __builtin_ctzll(no) - kWave;
        more = false;
      }
    }
    kv_append_run<D, TYPE, kWave>(x + (t0 + i0) * stride, stride, n, first, is_v, head, c, lane, s_max, s_turn);
  }
}

// ---------------------------------------------------------------------------
// dequant: block (page, head, keys or values); four codes a thread and step.
// Bandwidth bound, four of five bytes are written: past the caches' reuse order
// (ordinary stores pushed the cache's own pages out of the L2: append and dequant
// of 11.8k tokens 57 us instead of 43, 4.5 TB/s).
// ---------------------------------------------------------------------------
typedef float kv_f32x4 __attribute__((ext_vector_type(4)));

template <int D, int TYPE>
__global__ __launch_bounds__(kKvThreads) void kv_dequant_kernel(KvCache c, const int32_t* __restrict__ pages,
                                                                float* __restrict__ k_out,
                                                                float* __restrict__ v_out) {
  const int P = 1 << c.page_shift;
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int page = pages[blockIdx.x];
  const bool ok = page >= 0 && page < c.pages;
  const size_t ph = ok ? (size_t)page * c.heads + head : 0;
  const float s = ok ? bf16_lo((is_v ? c.vs : c.ks)[ph]) : __builtin_nanf("");
  float* out = (is_v ? v_out : k_out) + ((size_t)blockIdx.x * c.heads + head) * P * D;
  if (!is_v) {
    const uint32_t* in = reinterpret_cast<const uint32_t*>(c.k + ph * P * D);
    for (int e = threadIdx.x; e < P * D / 4; e += kKvThreads) {
      const uint32_t w = ok ? in[e] : 0;
      const kv_f32x4 v = {kv_decode<TYPE, 0>(w) * s, kv_decode<TYPE, 1>(w) * s, kv_decode<TYPE, 2>(w) * s,
                    kv_decode<TYPE, 3>(w) * s};
      __builtin_nontemporal_store(v, reinterpret_cast<kv_f32x4*>(out) + e);
    }
  } else {
    // 4 x 4 pieces: four rows' words of four tokens in, four tokens' float4 of four rows out
    const uint8_t* in = c.v + ph * P * D;
    for (int e = threadIdx.x; e < P * D / 16; e += kKvThreads) {
      const int d = 4 * (e % (D / 4)), tok = 4 * (e / (D / 4));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = ok ? *reinterpret_cast<const uint32_t*>(in + (size_t)(d + i) * P + tok) : 0;
      auto put = [&](auto bc) {
        constexpr int B = decltype(bc)::value;
        const kv_f32x4 v = {kv_decode<TYPE, B>(w[0]) * s, kv_decode<TYPE, B>(w[1]) * s, kv_decode<TYPE, B>(w[2]) * s,
                      kv_decode<TYPE, B>(w[3]) * s};
        __builtin_nontemporal_store(v, reinterpret_cast<kv_f32x4*>(out + (size_t)(tok + B) * D + d));
      };
      put(std::integral_constant<int, 0>{});
      put(std::integral_constant<int, 1>{});
      put(std::integral_constant<int, 2>{});
      put(std::integral_constant<int, 3>{});
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// calls f with the cache's head size and type as constants
template <class F>
void with_cache_form(const w4a16_kv_cache_t* c, F&& f) {
  using std::integral_constant;
  auto typed = [&](auto d) {
    if (c->type == W4A16_KV_INT8)
      f(d, integral_constant<int, W4A16_KV_INT8>{});
    else
      f(d, integral_constant<int, W4A16_KV_FP8>{});
  };
  if (c->dim == 64)
    typed(integral_constant<int, 64>{});
  else if (c->dim == 128)
    typed(integral_constant<int, 128>{});
  else
    typed(integral_constant<int, 256>{});
}

w4a16_status_t check_attention(const w4a16_kv_cache_t* cache, int tokens, int requests, int max_new, int max_len,
                               int window, int q_heads) {
  const w4a16_status_t st = check_cache(cache);
  if (st != W4A16_OK) return st;
  if (tokens < 0 || requests < 0 || max_new < 0 || max_len < 0 || window < 0 || q_heads < 1) return W4A16_ERR_SHAPE;
  if (tokens > W4A16_KV_MAX_TOKENS || requests > W4A16_KV_MAX_REQUESTS || max_len > kKvMaxLen) return W4A16_ERR_SHAPE;
  if (q_heads % cache->heads || (int64_t)tokens * q_heads > 0x7FFFFFFFLL) return W4A16_ERR_SHAPE;
  if (q_heads / cache->heads > W4A16_KV_MAX_GROUP) return W4A16_ERR_UNSUPPORTED;
  // the tiles' grid (at least 64 rows each) within the launch limit of 2^32 threads
  const int64_t tiles = tokens / (64 / (q_heads / cache->heads)) + requests;
  if (tiles * cache->heads > (1 << 22)) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// The launch parameters of an attention call from its (checked) sizes.
// Chunks of the cache (one workgroup each): they depend on max_len alone, so a
// row's sums do not depend on the batch.  A workgroup needs 3 us to begin and
// about 1 us for each step of 128 entries, and a row and chunk costs D + 5
// floats written and read again: short chunks answer sooner, long ones stream
// better.  Measured (us, chunks of 128 / 256 / 512 / 1024): one request of 717
// entries 8.8 / 11.2 / 15.7 / 17.6; 96 with a window of 512 in up to 3101
// 16.1 / 15.1 / 15.2 / 17.4; 48 of up to 6001 84.2 / 70.2 / 63.3 / 63.3; 16
// verify batches of up to 9006 37.4 / 33.4 / 31.0 / 42.8.
KvAttnArgs attention_args(const w4a16_kv_cache_t* cache, int tokens, int requests, int max_new, int max_len,
                          int window, int q_heads) {
  KvAttnArgs a{};
  a.c = device_cache(cache);
  // (a window of 2^30 hides nothing from lengths up to 2^29, and leaves room for what is
  // subtracted from it)
  a.window = window < 1 << 30 ? window : 1 << 30;
  a.tokens = tokens;
  a.requests = requests;
  a.max_new = max_new;
  a.max_len = max_len;
  a.q_heads = q_heads;
  a.group = q_heads / cache->heads;
  a.group_inverse = (65536u + a.group - 1) / a.group;
  a.split_tokens = max_new < kKvSplitRows / a.group ? max_new : kKvSplitRows / a.group;
  // A call of one request of many new tokens is a prompt: without the launches
  // for requests of few it is 9 us shorter (it may still bring few, as tiles).
  a.split = requests > 1 || (int64_t)max_new * a.group <= kKvSplitRows;
  a.by_token = tokens <= (int64_t)requests * a.split_tokens;
  const int rows = a.split_tokens * a.group;
  a.row_groups = rows <= 16 ? 1 : (rows + 31) / 32;
  a.chunk_shift = max_len <= 1024 ? 7 : max_len <= 4096 ? 8 : max_len <= 16384 ? 9 : 10;
  auto in_chunks = [&](long long n) { return (n + (1LL << a.chunk_shift) - 1) >> a.chunk_shift; };
  while (in_chunks(max_len) > kKvMaxChunks - 1) ++a.chunk_shift;     // (a window may add one)
  long long chunks = in_chunks(max_len);
  // a window's rows attend window + split_tokens - 1 entries at most
  const long long in_window = in_chunks((long long)a.window + a.split_tokens - 2) + 1;
  if (window > 0 && in_window < chunks) chunks = in_window;
  a.chunks = chunks > 1 ? (int)chunks : 1;
  // Where prompts bring fewer workgroups than the card holds (512, two a CU), the
  // cache is cut into parts that share their rows: their tiles run side by side, and
  // a join adds the parts (uncut, 100 tokens behind 8000 entries, 32 heads of 128 over
  // 8: 211 us instead of 44).  Each row and part costs D + 2 floats written and read
  // again, so a part has six tiles at least.  Measured (us, at least 4 / 6 / 8): 64
  // tokens behind 8000, 10 heads of 256 over 2, 41.6 / 34.9 / 36.8; two of 103 behind
  // 1373, 16 heads of 128 over 2, 27.1 / 29.2 / 34.7.  For 1024 workgroups instead of
  // 512: 1000 behind 8000, 32 heads of 128 over 8, 199 instead of 187.
  a.parts = 1;
  a.part = kKvMaxLen + kKvTile;      // all
  if (requests > 0 && (int64_t)max_new * a.group > kKvSplitRows) {
    const int tile_tokens = kv_tile_rows(cache->dim, cache->type) / a.group;
    const int64_t workgroups = (int64_t)(tokens / tile_tokens + requests) * cache->heads;
    const int64_t reach = (int64_t)a.window + tile_tokens - 1;      // entries of a window's workgroup
    const int64_t span = window > 0 && reach < max_len ? reach : max_len;
    const int64_t wanted = std::min<int64_t>(512 / workgroups, span / (6 * kKvTile));
    if (wanted > 1) {
      a.part = (int)((span + wanted * kKvTile - 1) / (wanted * kKvTile)) * kKvTile;
      // (a window's entries may begin inside a part)
      a.parts = (int)std::min<int64_t>((max_len + a.part - 1) / a.part, (span + a.part - 2) / a.part + 1);
    }
  }
  return a;
}

size_t attention_workspace(const KvAttnArgs& a, int dim) {
  return kv_workspace_floats(a, dim) * sizeof(float);
}

}  // namespace

}  // namespace w4k

using namespace w4k;

extern "C" {

w4a16_status_t w4a16_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* free_pages,
                             int num_free, int32_t* block_table, int width, int32_t* seq_lens, int32_t* token_start,
                             int32_t* slot_map, int32_t* pages_used, int requests, int tokens, int page,
                             void* stream) {
  if (!page_supported(page)) return W4A16_ERR_UNSUPPORTED;
  if (requests < 0 || requests > W4A16_KV_MAX_REQUESTS || tokens < 0 || tokens > W4A16_KV_MAX_TOKENS ||
      num_free < 0 || width < 0 || width > W4A16_KV_MAX_WIDTH)
    return W4A16_ERR_SHAPE;
  if (!token_start || !pages_used) return W4A16_ERR_NULL;
  if (requests > 0 && (!ctx_lens || !new_lens || !seq_lens)) return W4A16_ERR_NULL;
  if ((num_free > 0 && !free_pages) || (tokens > 0 && !slot_map) || (requests > 0 && width > 0 && !block_table))
    return W4A16_ERR_NULL;
  for (const void* p : {(const void*)ctx_lens, (const void*)new_lens, (const void*)free_pages,
                        (const void*)block_table, (const void*)seq_lens, (const void*)token_start,
                        (const void*)slot_map, (const void*)pages_used})
    if (!kv_aligned(p, 4)) return W4A16_ERR_ALIGN;
  // enough blocks a request for the longest row of columns or (as far as the
  // host can tell) tokens, 16 a lane; the whole grid bounded
  const int gx = requests > 0 ? (requests + kKvWaves - 1) / kKvWaves : 1;
  int gy = (int)(((long long)(tokens > width ? tokens : width) + kWave * 16 - 1) / (kWave * 16));
  const int most = 4096 / gx;
  gy = gy > most ? most : gy;
  gy = gy < 1 ? 1 : gy;
  hipLaunchKernelGGL(kv_plan_kernel, dim3(gx, gy), dim3(kKvThreads), 0, (hipStream_t)stream, ctx_lens, new_lens,
                     free_pages, num_free, block_table, width, seq_lens, token_start, slot_map, pages_used, requests,
                     tokens, __builtin_ctz((unsigned)page));
  return kv_launched(hipGetLastError());
}

w4a16_status_t w4a16_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                               const int32_t* slot_map, const w4a16_kv_cache_t* cache, int tokens, void* stream) {
  w4a16_status_t st = check_cache(cache);
  if (st != W4A16_OK) return st;
  if (tokens < 0 || tokens > W4A16_KV_MAX_TOKENS) return W4A16_ERR_SHAPE;
  const int64_t row = (int64_t)cache->heads * cache->dim;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 || k_stride > (1LL << 40) ||
      v_stride > (1LL << 40))
    return W4A16_ERR_SHAPE;
  if (tokens == 0 || cache->pages == 0) return W4A16_OK;
  st = check_cache_pointers(cache);
  if (st != W4A16_OK) return st;
  if (!k || !v || !slot_map) return W4A16_ERR_NULL;
  if (!kv_aligned(k, 16) || !kv_aligned(v, 16) || !kv_aligned(slot_map, 4)) return W4A16_ERR_ALIGN;
  // Tokens a block looks at: one while blocks are few, more where most tokens
  // continue a run.  Measured (us, 1 / 4 / 16 / 64 tokens, 8 heads of 128): 11.8k tokens of
  // three prompts in pages of 64, 210 / 41 / 31 / 23; 2000 of one, 43 / 15 / 8 / 11; 700
  // verify batches of 5, 52 / 39 / 25 / 30.  The rule knows tokens, not runs, and
  // single tokens of many requests want fewer: 64 of them 5 / 7 / 21 / 79, 512 23 / 14 /
  // 21 / 69, 4000 156 / 68 / 72 / 101.
  const int span = tokens <= 256 ? 1 : tokens <= 4096 ? 16 : 64;
  with_cache_form(cache, [&](auto d, auto type) {
    hipLaunchKernelGGL((kv_append_kernel<decltype(d)::value, decltype(type)::value>),
                       dim3((unsigned)((tokens + span - 1) / span), 2 * cache->heads), dim3(kKvThreads), 0,
                       (hipStream_t)stream, k, k_stride, v, v_stride, slot_map, device_cache(cache), tokens, span);
  });
  return kv_launched(hipGetLastError());
}

size_t w4a16_kv_attention_workspace_bytes(int tokens, int requests, int max_new, int max_len, int window, int q_heads,
                                          const w4a16_kv_cache_t* cache) {
  if (check_attention(cache, tokens, requests, max_new, max_len, window, q_heads) != W4A16_OK) return 0;
  if (tokens == 0 || requests == 0 || max_new == 0) return 0;
  return attention_workspace(attention_args(cache, tokens, requests, max_new, max_len, window, q_heads), cache->dim);
}

w4a16_status_t w4a16_kv_attention(const uint16_t* q, int64_t q_stride, const w4a16_kv_cache_t* cache,
                                  const int32_t* block_table, int width, const int32_t* seq_lens,
                                  const int32_t* token_start, uint16_t* out, float scale, int window, int tokens,
                                  int requests, int max_new, int max_len, int q_heads, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  w4a16_status_t st = check_attention(cache, tokens, requests, max_new, max_len, window, q_heads);
  if (st != W4A16_OK) return st;
  if (width < 0 || width > W4A16_KV_MAX_WIDTH || q_stride < (int64_t)q_heads * cache->dim || q_stride % 8 || q_stride > (1LL << 40))
    return W4A16_ERR_SHAPE;
  if (tokens == 0 || requests == 0 || max_new == 0) return W4A16_OK;
  if (cache->pages == 0) return W4A16_ERR_SHAPE;      // masked entries are read from page 0
  st = check_cache_pointers(cache);
  if (st != W4A16_OK) return st;
  if (!q || !out || !seq_lens || !token_start || (width > 0 && !block_table)) return W4A16_ERR_NULL;
  if (!kv_aligned(q, 16) || !kv_aligned(out, 16) || !kv_aligned(block_table, 4) || !kv_aligned(seq_lens, 4) ||
      !kv_aligned(token_start, 4))
    return W4A16_ERR_ALIGN;
  KvAttnArgs a = attention_args(cache, tokens, requests, max_new, max_len, window, q_heads);
  const size_t need = attention_workspace(a, cache->dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  if (!kv_aligned(workspace, 16)) return W4A16_ERR_ALIGN;
  a.q = q;
  a.q_stride = q_stride;
  a.table = block_table;
  a.width = width;
  a.seq_lens = seq_lens;
  a.token_start = token_start;
  a.out = out;
  a.scale_log2 = __builtin_fabsf(scale) * 1.44269504088896340736f;
  a.q_sign = scale < 0.0f ? 0x80008000u : 0u;
  hipStream_t s = (hipStream_t)stream;
  switch (cache->dim) {
    case 64: return kv_launched(kv_attention_d64(cache->type, a, workspace, s));
    case 128: return kv_launched(kv_attention_d128(cache->type, a, workspace, s));
    default: return kv_launched(kv_attention_d256(cache->type, a, workspace, s));
  }
}

w4a16_status_t w4a16_kv_dequant(const w4a16_kv_cache_t* cache, const int32_t* pages, int count, float* k_out,
                                float* v_out, void* stream) {
  w4a16_status_t st = check_cache(cache);
  if (st != W4A16_OK) return st;
  if (count < 0 || count > W4A16_KV_MAX_DEQUANT) return W4A16_ERR_SHAPE;      // (2^32 threads on a grid's axis)
  if (count == 0) return W4A16_OK;
  st = check_cache_pointers(cache);
  if (st != W4A16_OK) return st;
  if (!pages || !k_out || !v_out) return W4A16_ERR_NULL;
  if (!kv_aligned(pages, 4) || !kv_aligned(k_out, 16) || !kv_aligned(v_out, 16)) return W4A16_ERR_ALIGN;
  with_cache_form(cache, [&](auto d, auto type) {
    hipLaunchKernelGGL((kv_dequant_kernel<decltype(d)::value, decltype(type)::value>),
                       dim3((unsigned)count, 2 * cache->heads), dim3(kKvThreads), 0, (hipStream_t)stream,
                       device_cache(cache), pages, k_out, v_out);
  });
  return kv_launched(hipGetLastError());
}

}  // extern "C"
