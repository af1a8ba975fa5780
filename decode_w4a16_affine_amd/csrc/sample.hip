// Sampling from logits (w4a16_sample of include/w4a16_step.h).
//
// With C = (falling logit, rising index) as one 64-bit number every limit is "the tokens up
// to some C": top_k's is the C of the k-th token, top_p's that of the first token at which
// the running sum of weights reaches its share.  So nothing is sorted: a histogram over
// buckets of logits (1 / 12 of a temperature or 1 / 18 wide) tells which buckets the limits lie in, and
// only those buckets' tokens are looked at one by one.
//
// Launches.  scan: a workgroup reads a chunk of 8192 logits into registers; its largest
// logit and its histogram, or (rows without limits) each wave's largest and sum of weights.
// cut: a workgroup a row adds the chunks' histograms and finds the buckets lo .. hi that the
// limits lie in.  collect: reads the logits again and lists the tokens of these buckets; where
// the chunks are few each of its workgroups makes the cut for itself (kCutAlone), and
// where min_p is the first limit it adds up what that keeps and lists nothing.  draw: a
// workgroup a row finds the last kept token among the listed ones, adds the kept weights of
// each chunk, picks a chunk and looks up the token in it (without limits: a wave's 1024
// logits).  A call without limits has scan and draw alone.  A row whose chunks list
// thousands of tokens (flat rows, ties) is gone through by waves, a chunk each, from the lists
// or, where a list is too short, from the logits.
//
// Weights exp((logit - largest) / temperature) are computed in fp64 and added as integers of
// 2^-e (e = 62 - log2 N for a row: its sum stays below 2^63), or in a fixed order: sums do not
// depend on the order in which atomics arrive, and the answer is always the same.
// (fp32 would be off by 2^-24 of the larger weights at every border between the tokens,
// of which a row has up to 2^20.)
//
// What bounds it.  Many rows: the scan, at the rate of its fp64 weights or of memory, whichever is
// slower (256 rows of 262144 fp32 without limits: 57 us for 268 MB, 4.7 TB/s, and 7 for the
// draw; of bf16 the same together 58; 48 rows of bf16 with top_p and min_p: 12.5 for 25 MB and every
// weight, cut 7.0, collect 9.8, draw 18).  One row: the latency of the stages behind each other, each with two or
// three trips to memory (262144 fp32, top_k and top_p: scan 4.0, collect with its cut 9.8, draw 8.3).
// A draw's workgroup has a CU to itself and is bound by its own instructions: what one wave can do
// it does alone, 11 us before instead of 8.3, and 25 instead of 18 for the 48.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_host.hpp"
#include "w4a16_step.h"

namespace w4k {

namespace {

// lambdas over register arrays must be inlined for these to stay in registers
#define W4K_INLINE __attribute__((always_inline))

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / kWave;
constexpr int kSampleBins = 2048;
constexpr int kScanThreads = 512;
constexpr int kScanWaves = kScanThreads / kWave;
constexpr int kLane = 16;                             // logits a lane holds
constexpr int kChunk = kScanThreads * kLane;          // and a workgroup
constexpr int kSub = kWave * kLane;                    // a wave
constexpr int kChunks = W4A16_SAMPLE_MAX_N / kChunk;
constexpr int kBuckets = 256;
constexpr float kBucketsPerUnit = 12.0f;              // of (logit / temperature)
// For lower temperatures buckets are not narrower than 1 / 18 of a logit, 14 logits for all of them: tokens that top_k
// keeps lie that far apart whatever their weights (262144 normal logits of deviation 3, temperature 0.1, the
// first 50: 22 us, with 1 / 120 159).
constexpr float kMaxInverse = 1.5f;
// Up to a workgroup for each CU collect makes the cut itself, side by side, and a launch is saved (8 rows of 262144
// with top_k and top_p 33.3 us in a graph, with a cut of its own 34.6; 16 rows 38.0 and 37.9, 24 43.6 and 41.5).
constexpr int kCutAlone = 256;
constexpr int kListed = 2048;                         // tokens of a chunk that are listed at most
constexpr int kSmallK = 512;                          // limits of so few tokens need no weights from the scan
constexpr int kCutScale = 42;                         // sums of a row's buckets (2^20 weights below 2^63)
constexpr int kChunkScale = 49;                       // a chunk's weights are multiples of 2^-49 (8192 of them below 2^63)
// A bucket of a chunk: its tokens times 2^50, and their weights, multiples of 2^-36 (8192 below 2^50).  Its limits
// are found with a margin for that, and what a weight is off by, 2^-37 of the largest, divides among the tokens'
// borders: one in 10^6 rows or fewer would draw a neighbour.
constexpr int kBinScale = 36, kBinCount = 50;
constexpr double kBinUnit = 0x1p-36;
constexpr int kSorted = 1024;                         // listed tokens that are sorted at most
constexpr int kHeld = 8;                              // listed tokens that a thread of the draw holds
static_assert(kChunk == 1 << (62 - kChunkScale) && kChunk <= 1 << (kBinCount - kBinScale - 1), "sums fit");
static_assert(kSub == kSampleThreads && kChunks * kScanWaves <= kSampleThreads && kBuckets <= kScanThreads &&
                  kSorted == kSampleThreads,
              "a thread each");

// (2^f - 1) / f for |f| <= 1/2: the polynomial through it at the nine Chebyshev points, which leaves 2^f off by
// 2^-44.6 of it.
struct SampleSeries {
  double c[9] = {6.931471805599453e-01,  2.402265069581299e-01,  5.5504108664760424e-02,
                 9.618129159402558e-03,  1.3333558179043112e-03, 1.5403455852453838e-04,
                 1.525268684626772e-05, 1.3255224878668817e-06, 1.0203121063391729e-07};
};
struct SampleArgs {
  const void* logits;
  int64_t stride;
  const float *uniforms, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* share;
  int M, N;
  int log2_scale;      // weights are multiples of 2^-log2_scale
  // of these rows (see sample_places)
  int chunks;
  int list_threads;    // of the draw, for each chunk's list: a power of two
  // rows without limits: a wave's tokens of the scan (`subs` of 1024 a row)
  int subs;
  float* sub_top;      // [M][subs] largest logit, NaN if it has one
  double* sub_mass;    // [M][subs] weights, of this one's
  // others
  float* top;          // [M][chunks] largest logit of a chunk, NaN if it has one
  uint64_t* kept;      // [M][chunks] weights of the buckets in front of lo, of a row's
  uint64_t* bins;      // [M][chunks][kBuckets] tokens and weights of a chunk's buckets, of its largest logit
  uint32_t* listed;    // [M][chunks] tokens in lo .. hi
  uint2* list;         // [M][chunks][kListed] these: logit, token
  struct SampleCut* cut;      // [M]
  SampleSeries series;        // for the scan: literals would be loaded anew for each weight
};

// Where a row's limits lie.
struct SampleCut {
  int lo, hi;          // buckets
  int before;          // tokens in front of lo
  int min_p_alone;     // top_k and top_p end behind hi: nothing is listed, `kept` is of all that min_p keeps
  uint64_t total;      // all weights, as kept (SampleArgs)
  double least;        // (logit - largest) / temperature of min_p
};

// A row's parameters.
struct SampleRow {
  bool greedy;         // the largest logit is the only one kept
  double t, inv_t;     // temperature, and 1 / it
  int k;               // 0: no limit
  float top_p, min_p;  // >= 1, 0: no limit
};

__device__ __forceinline__ SampleRow sample_row(const SampleArgs& a, int r) {
  SampleRow p;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  p.greedy = !(t > 0.0f) || !a.uniforms;
  // (an estimate and two steps of Newton's: to 2^-51 of it, without a division's special cases)
  p.t = (double)fminf(fmaxf(t, 0x1p-149f), 3.402823466e38f);
  double inv = __builtin_amdgcn_rcp(p.t);
  inv = __builtin_fma(__builtin_fma(-p.t, inv, 1.0), inv, inv);
  p.inv_t = __builtin_fma(__builtin_fma(-p.t, inv, 1.0), inv, inv);
  p.k = a.top_k ? a.top_k[r] : 0;
  p.k = p.k > 0 && p.k < a.N ? p.k : 0;
  p.top_p = a.top_p ? a.top_p[r] : 1.0f;
  p.top_p = p.top_p < 1.0f ? p.top_p : 1.0f;
  p.min_p = a.min_p ? a.min_p[r] : 0.0f;
  p.min_p = p.min_p > 0.0f ? p.min_p : 0.0f;
  p.greedy |= p.top_p <= 0.0f || p.min_p > 1.0f;
  return p;
}
__device__ __forceinline__ bool sample_limited(const SampleRow& p) {
  return !p.greedy && (p.k || p.top_p < 1.0f || p.min_p > 0.0f);
}
// Few tokens are kept at most: all in the buckets up to the k-th token's are listed, and the
// scan counts without computing weights.
__device__ __forceinline__ bool sample_few(const SampleRow& p) { return p.k && p.k <= kSmallK; }

__device__ __forceinline__ float sample_load(const float* p) { return *p; }
__device__ __forceinline__ float sample_load(const uint16_t* p) { return bf16_lo(*p); }

// Larger logits have larger numbers (-0 and 0, which are equal, the same one).
__device__ __forceinline__ uint32_t sample_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u >> 31 ? ~u : u | 0x80000000u;
}
// Position in the order of falling logits: smaller comes first.  (And the logit back.)
__device__ __forceinline__ uint64_t sample_order(float v, int i) { return (uint64_t)~sample_key(v) << 32 | (uint32_t)i; }

__device__ __forceinline__ float sample_logit(uint64_t c) {
  const uint32_t key = ~(uint32_t)(c >> 32);
  return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key);
}

// (logit - top) / temperature: 0 for the largest also where that is infinite
__device__ __forceinline__ double sample_log_weight(float v, float top, double inv_t) {
  return v == top ? 0.0 : ((double)v - (double)top) * inv_t;
}
typedef uint32_t sample_u32x2 __attribute__((ext_vector_type(2)));
// 2^(t + scale) for t <= 0, below t = -1000 as there.  2^t = 2^n 2^f with |f| <= 1/2.  n + scale appears in the low
// bits of a sum with 1.5 * 2^52 and is added to the exponent's: conversions to and from fp64, rint and ldexp take
// four times as long as a sum (256 tempered rows of 262144: 70 us with them, 64 without).  It holds for normal results,
// so for scales from kLeastScale on.  (Further down the exponent is carried past its end: 2^-1036 came out as -2^1012
// where a chunk's factor had the scale -36 and a chunk lay 684 temperatures below the row's largest logit.)
constexpr int kLeastScale = -21;
static_assert(62 - 20 - kChunkScale >= kLeastScale && W4A16_SAMPLE_MAX_N == 1 << 20, "log2_scale - kChunkScale");
__device__ __forceinline__ double sample_exp2(double t, int scale, const SampleSeries& series = SampleSeries{}) {
  t = fmax(t, -1000.0);
  const double to_int = 0x1.8p52 + (double)scale, shifted = t + to_int, f = t - (shifted - to_int);
  double y = series.c[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) y = __builtin_fma(y, f, series.c[i]);
  y = __builtin_fma(y, f, 1.0);
  sample_u32x2 u = __builtin_bit_cast(sample_u32x2, y);
  u[1] += (uint32_t)__double_as_longlong(shifted) << 20;
  return __builtin_bit_cast(double, u);
}
constexpr double kLog2E = 1.4426950408889634074;
// A weight times 2^log2_scale
__device__ __forceinline__ double sample_weight(float v, float top, double inv_t, int log2_scale) {
  return sample_exp2(sample_log_weight(v, top, inv_t) * kLog2E, log2_scale);
}
// A weight held in integers: it appears in the low bits of 2^52 and it (at most 2^50).
__device__ __forceinline__ uint64_t sample_units(double w) {
  return (uint64_t)__double_as_longlong(w + 0x1p52) & 0xFFFFFFFFFFFFFull;
}

// A logit's bucket counted from any fixed one; grows with the logit.  (A sum with 1.5 * 2^23 is rounded
// to an integer; far logits share the outermost ones.)
__device__ __forceinline__ float sample_bucket_scale(double inv_t) {
  return kBucketsPerUnit * fminf((float)inv_t, kMaxInverse);
}
__device__ __forceinline__ int sample_bucket(float v, float scale) {
  return __float_as_int(__builtin_amdgcn_fmed3f(__builtin_fmaf(v, scale, 0x1.8p23f), 0x1p23f, 0x1.fffffep23f));
}
// Counted down from the one of a row's or chunk's largest logit, and the last one for all behind it.
__device__ __forceinline__ int sample_below(int top_bucket, float v, float scale) {
  return min(top_bucket - sample_bucket(v, scale), kBuckets - 1);
}

// 16 bytes of logits at any place that their type allows
struct __attribute__((packed, aligned(2))) SampleWords {
  uint32_t w[4];
};
__device__ __forceinline__ void sample_load_some(const float* p, float (&v)[4]) {
  const SampleWords u = *reinterpret_cast<const SampleWords*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u.w[i]);
}
__device__ __forceinline__ void sample_load_some(const uint16_t* p, float (&v)[8]) {
  const SampleWords u = *reinterpret_cast<const SampleWords*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u.w[i]), v[2 * i + 1] = bf16_hi(u.w[i]);
}
// `count` logits from token i on, -infinity past the row's end
template <int COUNT, class T>
__device__ __forceinline__ void sample_load_row(const T* row, int i, int N, float* v) {
  if (i + COUNT <= N) {
    float x[COUNT];
    sample_load_some(row + i, x);
#pragma unroll
    for (int e = 0; e < COUNT; ++e) v[e] = x[e];
  } else {
#pragma unroll
    for (int e = 0; e < COUNT; ++e) v[e] = i + e < N ? sample_load(row + i + e) : -__builtin_inff();
  }
}
// The lane's logits of a chunk: pieces of V in a row.
template <class T>
constexpr int kPiece = 16 / sizeof(T);
template <class T>
__device__ __forceinline__ int sample_token(int chunk, int x) {
  constexpr int V = kPiece<T>;
  return chunk * kChunk + ((threadIdx.x / kWave * (kLane / V) + x / V) * kWave + (threadIdx.x & (kWave - 1))) * V + x % V;
}
template <class T>
__device__ __forceinline__ void sample_load_chunk(const T* row, int chunk, int N, float (&v)[kLane]) {
  constexpr int V = kPiece<T>;
  if ((chunk + 1) * kChunk <= N) {      // (no load under a condition)
    const T* const p = row + sample_token<T>(chunk, 0);
#pragma unroll
    for (int x = 0; x < kLane; x += V) {
      float some[V];
      sample_load_some(p + x * kWave, some);
#pragma unroll
      for (int e = 0; e < V; ++e) v[x + e] = some[e];
    }
  } else {
#pragma unroll
    for (int x = 0; x < kLane; x += V) sample_load_row<V>(row, sample_token<T>(chunk, x), N, v + x);
  }
}

// Eight in a row, of a thread of the draw.
constexpr int kDrawLane = kChunk / kSampleThreads;
template <class T>
__device__ __forceinline__ void sample_load_eight(const T* row, int i, int N, float (&v)[kDrawLane]) {
  constexpr int V = kDrawLane <= kPiece<T> ? kDrawLane : kPiece<T>;
#pragma unroll
  for (int e = 0; e < kDrawLane; e += V) sample_load_row<V>(row, i + e, N, v + e);
}

// A wave's running sums: rows of 16 lanes by shifts within them, then their last lanes' to the rows behind.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t sample_from_lane(uint32_t v) {
  // (of lanes that have no source, or are not of ROWS, 0)
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, ROWS == 0xF);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t sample_from_lane(uint64_t v) {
  return (uint64_t)sample_from_lane<CTRL, ROWS>((uint32_t)(v >> 32)) << 32 | sample_from_lane<CTRL, ROWS>((uint32_t)v);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double sample_from_lane(double v) {
  return __longlong_as_double((long long)sample_from_lane<CTRL, ROWS>((uint64_t)__double_as_longlong(v)));
}
template <class V>
__device__ __forceinline__ V sample_row_scan(V v) {
  v += sample_from_lane<0x111, 0xF>(v);
  v += sample_from_lane<0x112, 0xF>(v);
  v += sample_from_lane<0x114, 0xF>(v);
  v += sample_from_lane<0x118, 0xF>(v);
  return v;
}
template <class V>
__device__ __forceinline__ V sample_wave_scan(V v) {
  v = sample_row_scan(v);
  v += sample_from_lane<0x142, 0xA>(v);      // lane 15 to the second row, lane 47 to the fourth
  v += sample_from_lane<0x143, 0xC>(v);      // lane 31 to the upper half
  return v;
}
__device__ __forceinline__ uint32_t sample_of_lane(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ uint64_t sample_of_lane(uint64_t v, int lane) {
  return (uint64_t)sample_of_lane((uint32_t)(v >> 32), lane) << 32 | sample_of_lane((uint32_t)v, lane);
}
// A wave's sum, in a fixed order.
__device__ __forceinline__ double sample_wave_sum(double v) {
  return __longlong_as_double((long long)sample_of_lane((uint64_t)__double_as_longlong(sample_wave_scan(v)), kWave - 1));
}

// What a row's workgroup of the draw shares.
struct SampleShared {
  uint64_t bins[kSampleBins];
  uint64_t waves[kSampleWaves];
  uint64_t found[2];
  uint32_t few;
  uint64_t chunk[2 * kWave];      // kept weights
  uint32_t listed[2 * kWave], place[2 * kWave];
  // what its first wave makes of the row, so that others do not: sixteen waves on four SIMDs take
  // sixteen cycles for an instruction, one takes four
  float top, top_p;
  double inv_t;
  int special, far, k, picked;
  SampleCut cut;
  uint64_t base, all, left;
  uint32_t all_listed;
  float tops[kSampleWaves], sub_top;      // of rows without limits
};

// Sums over the block's first `waves` waves (the others only wait): of threads before this one, and of all.
__device__ __forceinline__ uint64_t sample_scan(uint64_t v, uint64_t& before, int waves, SampleShared& sh) {
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  __syncthreads();      // (sh.waves may still be read from a scan before)
  uint64_t sum = 0;
  if (wave < waves) {
    sum = sample_wave_scan(v);
    if (lane == kWave - 1) sh.waves[wave] = sum;
  }
  __syncthreads();
  // each row of lanes scans the waves' sums
  static_assert(kSampleWaves == 16, "a lane of a row each");
  const uint64_t upto = sample_row_scan((lane & 15) < waves ? sh.waves[lane & 15] : (uint64_t)0);
  before = (wave ? sample_of_lane(upto, wave - 1) : 0) + sum - v;
  return sample_of_lane(upto, 15);
}

// The number that lane i ^ J holds, without a way through LDS.
template <int J>
__device__ __forceinline__ uint32_t sample_across(uint32_t v) {
  const int x = (int)v;
  if constexpr (J == 1) return (uint32_t)__builtin_amdgcn_update_dpp(x, x, 0xB1, 0xF, 0xF, false);
  if constexpr (J == 2) return (uint32_t)__builtin_amdgcn_update_dpp(x, x, 0x4E, 0xF, 0xF, false);
  if constexpr (J == 4) {      // 7 - i of each eight, then 3 - i of each four
    const int y = __builtin_amdgcn_update_dpp(x, x, 0x141, 0xF, 0xF, false);
    return (uint32_t)__builtin_amdgcn_update_dpp(y, y, 0x1B, 0xF, 0xF, false);
  }
  if constexpr (J == 8) return (uint32_t)__builtin_amdgcn_update_dpp(x, x, 0x128, 0xF, 0xF, false);      // turned by 8 of 16
  // a swap with its own copy leaves the lane's number in one and the other's in the other
  if constexpr (J == 16) {
    auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? s[0] : s[1];
  }
  if constexpr (J == 32) {
    auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32) ? s[0] : s[1];
  }
}
template <int J>
__device__ __forceinline__ uint64_t sample_exchange(uint64_t c, bool up) {
  const uint64_t other = (uint64_t)sample_across<J>((uint32_t)(c >> 32)) << 32 | sample_across<J>((uint32_t)c);
  return (other < c) == (up == ((threadIdx.x & J) == 0)) ? other : c;
}
template <int J>
__device__ __forceinline__ uint64_t sample_merge(uint64_t c, bool up) {
  c = sample_exchange<J>(c, up);
  if constexpr (J > 1) c = sample_merge<J / 2>(c, up);
  return c;
}
// Sorts the threads' numbers, the smallest to thread 0, by compare and exchange (bitonic);
// n: a power of two of threads that have one, at least a wave's.
__device__ __forceinline__ uint64_t sample_sort(uint64_t c, int n, uint64_t* s_swap) {
  const int i = threadIdx.x;
  const bool in = __builtin_amdgcn_readfirstlane(i) < n;      // (whole waves)
  if (in) {
    c = sample_merge<1>(c, (i & 2) == 0);
    c = sample_merge<2>(c, (i & 4) == 0);
    c = sample_merge<4>(c, (i & 8) == 0);
    c = sample_merge<8>(c, (i & 16) == 0);
    c = sample_merge<16>(c, (i & 32) == 0);
    c = sample_merge<32>(c, (i & 64) == 0);
  }
  for (int k = 2 * kWave; k <= n; k <<= 1) {
    const bool up = (i & k) == 0;
    for (int j = k >> 1; j >= kWave; j >>= 1) {
      __syncthreads();
      s_swap[i] = c;
      __syncthreads();
      const uint64_t other = s_swap[i ^ j];
      c = (other < c) == (up == ((i & j) == 0)) ? other : c;
    }
    if (in) c = sample_merge<32>(c, up);
  }
  return c;
}

// The first C (in order) at which the running sum of `measure` reaches target >= 1, of tokens in lo .. hi
// (others do not count); `otherwise` if it does not.  visit(f) calls f(C, measure)
// for the thread's tokens, measure_of(C) is measure() again.  Bins over lo .. hi tell which of them has it;
// a bin of few tokens is sorted, another one is divided again.
template <class Visit, class Measure>
__device__ __forceinline__ uint64_t sample_select(Visit&& visit, Measure&& measure_of, uint64_t target, uint64_t lo,
                                                  uint64_t hi, uint64_t otherwise, SampleShared& sh) {
  constexpr int SCAN = 4, EACH = kSampleBins / (SCAN * kWave);      // waves that scan the bins, bins a thread
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  uint64_t base = 0;      // the sum in front of lo
  for (;;) {
    const uint64_t range = hi - lo;
    const int bits = range ? 64 - __builtin_clzll(range) : 0, shift = bits > 11 ? bits - 11 : 0;
    static_assert(kSampleBins == 1 << 11, "the shift");
    __syncthreads();
    sh.bins[tid] = 0, sh.bins[tid + kSampleThreads] = 0;
    if (tid == 0) sh.found[0] = 0, sh.found[1] = 0, sh.few = 0;
    __syncthreads();
    visit([&](uint64_t c, auto&& measure) W4K_INLINE {
      if (c >= lo && c <= hi) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[(c - lo) >> shift]), measure());
    });
    __syncthreads();
    uint64_t sum = 0, before;
    if (wave < SCAN)
      for (int i = 0; i < EACH; ++i) sum += sh.bins[EACH * tid + i];
    const uint64_t all = sample_scan(sum, before, SCAN, sh);
    if (base + all < target) return otherwise;
    before += base;
    if (wave < SCAN && before < target && before + sum >= target) {      // one thread's
      int at = EACH * tid;
      while (before + sh.bins[at] < target) before += sh.bins[at++];
      sh.found[0] = at;
      sh.found[1] = before;
    }
    __syncthreads();
    lo += sh.found[0] << shift;
    hi = lo + ((1ull << shift) - 1) < hi ? lo + ((1ull << shift) - 1) : hi;
    base = sh.found[1];
    if (shift == 0) return lo;
    // the bin's tokens, in order, if they are few
    visit([&](uint64_t c, auto&&) W4K_INLINE {
      if (c < lo || c > hi) return;
      const uint32_t at = atomicAdd(&sh.few, 1u);
      if (at < kSorted) sh.bins[at] = c;
    });
    __syncthreads();
    const int n = (int)sh.few;
    if (n > kSorted) {      // equal logits among them: not between lo and hi, but where they are
      if (tid == 0) sh.found[0] = hi, sh.found[1] = lo;
      __syncthreads();
      uint64_t least = ~0ull, most = 0;
      visit([&](uint64_t c, auto&&) W4K_INLINE {
        if (c < lo || c > hi) return;
        least = c < least ? c : least;
        most = c > most ? c : most;
      });
      if (least <= most) {
        atomicMin(reinterpret_cast<unsigned long long*>(&sh.found[0]), least);
        atomicMax(reinterpret_cast<unsigned long long*>(&sh.found[1]), most);
      }
      __syncthreads();
      lo = sh.found[0], hi = sh.found[1];
      continue;
    }
    int threads = kWave;
    while (threads < n) threads <<= 1;
    const uint64_t c = sample_sort(tid < n ? sh.bins[tid] : ~0ull, threads, sh.bins + kSampleThreads);
    const uint64_t m = tid < n ? measure_of(c) : 0;
    sample_scan(m, before, threads / kWave, sh);
    before += base;
    if (m && before < target && before + m >= target) sh.found[0] = c;
    __syncthreads();
    return sh.found[0];
  }
}

// A row's largest logit (NaN if it has one) from its chunks': every wave goes through all,
// two a lane; their loads come first, so that others can be on their way beside them.
static_assert(kChunks <= 2 * kWave, "two chunks a lane");
struct SampleTops {
  float top[2];
};
__device__ __forceinline__ SampleTops sample_tops(const SampleArgs& a, int r) {
  const int lane = threadIdx.x & (kWave - 1);
  SampleTops t;
#pragma unroll
  for (int i = 0; i < 2; ++i) t.top[i] = a.top[(size_t)r * a.chunks + min(lane + i * kWave, a.chunks - 1)];
  return t;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float sample_max_row(float v) {
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xF, false)));
}
// The largest of a wave's numbers (fmaxf leaves NaN out).
__device__ __forceinline__ float sample_wave_max(float v) {
  v = sample_max_row<0x111, 0xF>(v);
  v = sample_max_row<0x112, 0xF>(v);
  v = sample_max_row<0x114, 0xF>(v);
  v = sample_max_row<0x118, 0xF>(v);
  v = sample_max_row<0x142, 0xA>(v);
  v = sample_max_row<0x143, 0xC>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1));
}
__device__ __forceinline__ float sample_row_top(const SampleTops& t) {
  if (__any(t.top[0] != t.top[0] || t.top[1] != t.top[1])) return __builtin_nanf("");
  return sample_wave_max(fmaxf(t.top[0], t.top[1]));
}

// ---------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(kScanThreads, 8) void sample_scan_kernel(SampleArgs a) {
  __shared__ uint64_t s_bins[kBuckets];
  __shared__ float s_top[kScanWaves];
  const int chunk = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const T* const row = static_cast<const T*>(a.logits) + r * a.stride;
  float v[kLane];
  sample_load_chunk(row, chunk, a.N, v);
  const SampleRow p = sample_row(a, r);
  const size_t at = (size_t)r * a.chunks + chunk;
  // the largest logit (fmaxf leaves NaN out)
  float top = -__builtin_inff();
  bool nan = false;
#pragma unroll
  for (int x = 0; x < kLane; ++x) {
    top = fmaxf(top, v[x]);
    nan |= v[x] != v[x];
  }
  top = sample_wave_max(top);
  // f(logit, weight times 2^scale), four at a time: more would take too many registers.  Where the
  // largest logit is moderate one fma gives the exponent, off by 2^-41 for all alike.
  const double inv_t = p.inv_t * kLog2E;
  auto weights = [&](int log2_scale, auto&& f) W4K_INLINE {
    const double away = -(double)top * inv_t;
    if (away < 4096.0 && away > -4096.0) {
#pragma unroll
      for (int x = 0; x < kLane; ++x) {
        f(v[x], sample_exp2(__builtin_fma((double)v[x], inv_t, away), log2_scale, a.series));
        if (x % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int x = 0; x < kLane; ++x) {
        float y = v[x];
        asm("" : "+v"(y));      // (both sides' conversions in front of the branch would take all registers)
        f(y, sample_exp2(sample_log_weight(y, top, p.inv_t) * kLog2E, log2_scale, a.series));
        if (x % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // Without limits every wave is for itself: it computes while others wait for their logits, and nothing waits
  // for the last of them (256 rows of 262144: 57 us, with a chunk's sums behind a barrier 65).
  if (!sample_limited(p)) {
    double sum = 0.0;
    if (!p.greedy && top > -__builtin_inff()) weights(0, [&](float, double w) W4K_INLINE { sum += w; });
    sum = sample_wave_sum(sum);
    nan = __any(nan);
    if (lane == 0) {
      a.sub_top[at * kScanWaves + wave] = nan ? __builtin_nanf("") : top;
      a.sub_mass[at * kScanWaves + wave] = sum;
    }
    return;
  }
  if (tid < kBuckets) s_bins[tid] = 0;
  if (lane == 0) s_top[wave] = top;
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int w = 0; w < kScanWaves; ++w) top = fmaxf(top, s_top[w]);
  if (!nan && top > -__builtin_inff()) {
    const float scale = sample_bucket_scale(p.inv_t);
    const int top_bucket = sample_bucket(top, scale);
    if (sample_few(p)) {
#pragma unroll
      for (int x = 0; x < kLane; ++x) {      // (the upper half of a bucket)
        const int b = sample_below(top_bucket, v[x], scale);
        if (b < kBuckets - 1) atomicAdd(reinterpret_cast<uint32_t*>(&s_bins[b]) + 1, 1u << (kBinCount - 32));
      }
    } else {
      // The last bucket's weights are added up first and its tokens not counted (they are the rest):
      // it may have most of a chunk, whose additions would wait for each other.
      uint64_t rest = 0;
      weights(kBinScale, [&](float x, double w) W4K_INLINE {
        const uint64_t units = sample_units(w);
        const int b = sample_below(top_bucket, x, scale);
        if (b < kBuckets - 1)
          atomicAdd(reinterpret_cast<unsigned long long*>(&s_bins[b]), units + (1ull << kBinCount));
        else
          rest += units;
      });
      rest = sample_wave_scan(rest);
      if (lane == kWave - 1 && rest) atomicAdd(reinterpret_cast<unsigned long long*>(&s_bins[kBuckets - 1]), rest);
    }
  }
  __syncthreads();
  if (tid < kBuckets) a.bins[at * kBuckets + tid] = s_bins[tid];
  if (tid == 0) a.top[at] = nan ? __builtin_nanf("") : top;
}

// ---------------------------------------------------------------------------
// collect
// ---------------------------------------------------------------------------
constexpr int kAtOnce = 16;        // chunks whose buckets are added at once
constexpr int kSlices = kScanThreads / kBuckets;
constexpr int kAhead = kAtOnce / kSlices;      // of which a thread has this many
__device__ __forceinline__ double sample_bin_mass(uint64_t bin) {
  return __longlong_as_double((long long)((bin & ((1ull << kBinCount) - 1)) | 0x433ull << 52)) - 0x1p52;
}

// The buckets that a row's limits lie in, by one workgroup of kScanThreads threads.
struct SampleCutShared {
  uint64_t bins[kAtOnce][kBuckets];
  double factor[kChunks];
  int shift[kChunks];
  double mass[kBuckets];
  uint32_t count[kBuckets];
  uint64_t waves[3][kBuckets / kWave];
  int first[3];
  SampleCut cut;
};
struct SampleCutLoads {
  uint64_t bin[kAhead];
};
__device__ __forceinline__ void sample_cut_load(const SampleArgs& a, int r, int c0, SampleCutLoads& l) {
  const int b = threadIdx.x % kBuckets, slice = threadIdx.x / kBuckets;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    l.bin[i] = a.bins[((size_t)r * a.chunks + min(c0 + i * kSlices + slice, a.chunks - 1)) * kBuckets + b];
}
__device__ __forceinline__ SampleCut sample_find_cut(const SampleArgs& a, int r, const SampleRow& p, const SampleTops& tops,
                                                    float top, SampleCutLoads& l, SampleCutShared& sh) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int b = tid % kBuckets, slice = tid / kBuckets;
  const float scale = sample_bucket_scale(p.inv_t);
  const int top_bucket = sample_bucket(top, scale);
  // the bucket of the least weight, by fp32 arithmetic on its edge
  int edge_at = kBuckets;
  double least = -__builtin_inf();
  if (p.min_p > 0.0f) {
    least = log((double)p.min_p);
    const float edge = (float)((double)top + least * p.t);
    edge_at = sample_below(top_bucket, fminf(fmaxf(edge, -3e38f), top), scale);
  }
  if (tid < kWave) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = lane + i * kWave;
      if (c >= a.chunks) break;
      // (a chunk of -infinity alone has no weights; its tokens lie in the last bucket)
      const float t = tops.top[i];
      sh.factor[c] = t > -__builtin_inff() ? sample_weight(t, top, p.inv_t, 0) * kBinUnit : 0.0;
      sh.shift[c] = t > -__builtin_inff() ? min(top_bucket - sample_bucket(t, scale), kBuckets) : kBuckets;
    }
  }
  if (tid < 3) sh.first[tid] = kBuckets - 1;
  // a row's bucket: those of its chunks, shifted by their largest logits; what lies behind is the last one's
  double mass = 0.0, behind = 0.0;
  uint32_t count = 0;
  for (int c0 = 0; c0 < a.chunks; c0 += kAtOnce) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) sh.bins[i * kSlices + slice][b] = l.bin[i];
    if (c0 + kAtOnce < a.chunks) sample_cut_load(a, r, c0 + kAtOnce, l);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int in = i * kSlices + slice, c = c0 + in;
      if (c >= a.chunks) break;
      const int shift = sh.shift[c], from = b - shift;
      const double factor = sh.factor[c];
      if (from >= 0 && b < kBuckets - 1) {
        const uint64_t x = sh.bins[in][from];
        mass = __builtin_fma(sample_bin_mass(x), factor, mass);
        count += (uint32_t)(x >> kBinCount);
      }
      if (b + shift >= kBuckets - 1) behind = __builtin_fma(sample_bin_mass(sh.bins[in][b]), factor, behind);
    }
  }
  // (bins is free: the second slice's sums)
  __syncthreads();
  double* const s_part = reinterpret_cast<double*>(sh.bins);
  if (slice == 1) s_part[b] = mass, s_part[kBuckets + b] = behind, sh.count[b] = count;
  static_assert(kSlices == 2, "the sums of two");
  __syncthreads();
  uint64_t units = 0, counted = 0;
  if (slice == 0) {
    auto in_units = [&](double m) { return (uint64_t)__builtin_rint(__builtin_ldexp(m, kCutScale)); };
    units = sample_wave_scan(in_units(mass + s_part[b]));
    const uint64_t units_behind = sample_wave_scan(in_units(behind + s_part[kBuckets + b]));
    counted = sample_wave_scan((uint64_t)(count + sh.count[b]));
    if (lane == kWave - 1) sh.waves[0][wave] = units, sh.waves[1][wave] = counted, sh.waves[2][wave] = units_behind;
  }
  __syncthreads();
  // sums over the buckets up to this one
  uint64_t total_units = 0;
#pragma unroll
  for (int w = 0; w < kBuckets / kWave; ++w) {
    total_units += sh.waves[0][w] + sh.waves[2][w];
    if (w < wave) units += sh.waves[0][w], counted += sh.waves[1][w];
  }
  if (b == kBuckets - 1) units = total_units, counted = a.N;
  auto mass_of = [&](uint64_t u) { return __builtin_ldexp((double)u, -kCutScale); };
  const double upto = mass_of(units), total = mass_of(total_units);
  if (slice == 0) sh.mass[b] = upto, sh.count[b] = (uint32_t)counted;
  // the first bucket at which each limit may lie; the last one if none does
  auto first_of = [&](bool reached, int which) {
    const uint64_t there = __ballot(reached);
    if (there && lane == 0) atomicMin(&sh.first[which], wave * kWave + __builtin_ctzll(there));
  };
  if (slice == 0 && p.k) first_of(counted >= (uint64_t)p.k, 0);
  __syncthreads();
  const int k_at = p.k ? sh.first[0] : kBuckets;
  const bool few = sample_few(p);
  if (slice == 0 && !few && p.top_p < 1.0f) {
    // Sums are exact to 2^-24 (2^-37 times 8192 for each of 128 chunks at worst, 2^-28 where errors
    // cancel), beside a total of at least 1: a border that near leaves both buckets open.  The weights
    // that top_k keeps end somewhere in its bucket.
    const double fewest = p.k ? (k_at ? sh.mass[k_at - 1] : 0.0) : total, most = p.k ? sh.mass[k_at] : total;
    first_of(upto + 0x1p-16 >= p.top_p * fewest, 1);
    first_of(upto >= p.top_p * most + 0x1p-16, 2);
  }
  __syncthreads();
  int lo = k_at, hi = k_at;
  bool min_p_alone = false;
  if (few) {
    lo = 0;
  } else {
    if (p.top_p < 1.0f) {
      lo = min(lo, sh.first[1]);
      hi = p.k ? k_at : sh.first[2];      // (with top_k, its sum is needed exactly)
    }
    if (p.min_p > 0.0f) {      // one bucket to either side of the edge's
      min_p_alone = edge_at + 1 < lo || (!p.k && p.top_p >= 1.0f);
      if (min_p_alone) hi = edge_at + 1;
      lo = min(lo, edge_at - 1);
    }
  }
  lo = max(lo, 0), hi = min(hi, kBuckets - 1);
  return SampleCut{lo, hi, lo ? (int)sh.count[lo - 1] : 0, min_p_alone,
                   (uint64_t)__builtin_rint(__builtin_ldexp(total, a.log2_scale)), least};
}

__global__ __launch_bounds__(kScanThreads) void sample_cut_kernel(SampleArgs a) {
  __shared__ SampleCutShared sh;
  const int r = blockIdx.x;
  const SampleTops tops = sample_tops(a, r);
  SampleCutLoads l;
  sample_cut_load(a, r, 0, l);
  const SampleRow p = sample_row(a, r);
  if (!sample_limited(p)) return;
  const float top = sample_row_top(tops);
  if (!(top > -__builtin_inff())) return;
  const SampleCut cut = sample_find_cut(a, r, p, tops, top, l, sh);
  if (threadIdx.x == 0) a.cut[r] = cut;
}

// CUT: every workgroup of a row finds its buckets by itself, instead of a launch before this one.
template <class T, bool CUT>
__global__ __launch_bounds__(kScanThreads) void sample_collect_kernel(SampleArgs a) {
  struct Empty {};
  __shared__ std::conditional_t<CUT, SampleCutShared, Empty> sh;
  __shared__ uint32_t s_listed;
  __shared__ double s_sum[kScanWaves];
  __shared__ uint64_t s_units[kScanWaves];
  const int chunk = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const T* const row = static_cast<const T*>(a.logits) + r * a.stride;
  const size_t at = (size_t)r * a.chunks + chunk;
  // all loads of the launch at once
  const SampleTops tops = sample_tops(a, r);
  SampleCutLoads l;
  SampleCut cut;
  if constexpr (CUT)
    sample_cut_load(a, r, 0, l);
  else
    cut = a.cut[r];
  const uint64_t own_bin = a.bins[at * kBuckets + tid % kBuckets];
  const float own_top = a.top[at];
  float v[kLane];
  sample_load_chunk(row, chunk, a.N, v);
  const SampleRow p = sample_row(a, r);
  if (!sample_limited(p)) return;
  const float top = sample_row_top(tops);
  if (!(top > -__builtin_inff())) return;
  if (tid == 0) s_listed = 0;
  if constexpr (CUT) {
    cut = sample_find_cut(a, r, p, tops, top, l, sh);
    if (chunk == 0 && tid == 0) a.cut[r] = cut;
  }
  __syncthreads();
  const float scale = sample_bucket_scale(p.inv_t);
  const int top_bucket = sample_bucket(top, scale);
  // The lane's tokens in lo .. hi, and their places in the chunk's list; of the last bucket's only those that have a
  // weight (masked logits do not, and nothing is drawn behind them: 262144 of which 200 are not masked, top_k
  // 1000: 22 us, with all listed 672).
  float lowest = -__builtin_inff();
  if (cut.hi == kBuckets - 1 && top < __builtin_inff())
    lowest = (float)((double)top - (a.log2_scale + 2) / (p.inv_t * kLog2E));
  uint32_t mine = 0;
#pragma unroll
  for (int x = 0; x < kLane; ++x) {
    const int below = sample_below(top_bucket, v[x], scale);
    mine |= (below >= cut.lo && below <= cut.hi && v[x] >= lowest && sample_token<T>(chunk, x) < a.N ? 1u : 0u) << x;
  }
  uint64_t units = 0;      // min_p alone: the weights of these tokens that it keeps
  if (cut.min_p_alone) {
#pragma unroll
    for (int x = 0; x < kLane; ++x) {
      const double log_weight = sample_log_weight(v[x], top, p.inv_t);
      if (mine >> x & 1 && log_weight >= cut.least)
        units += (uint64_t)__builtin_rint(sample_exp2(log_weight * kLog2E, a.log2_scale));
      if (x % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
    units = sample_wave_scan(units);
  } else if (__any(mine)) {
    const uint32_t count = __builtin_popcount(mine), upto = sample_wave_scan(count);
    uint32_t slot = 0;
    if (lane == kWave - 1) slot = atomicAdd(&s_listed, upto);
    slot = (uint32_t)__builtin_amdgcn_readlane((int)slot, kWave - 1) + upto - count;
#pragma unroll
    for (int x = 0; x < kLane; ++x) {
      if (mine >> x & 1) {
        if (slot < kListed)
          a.list[at * kListed + slot] = make_uint2(__float_as_uint(v[x]), (uint32_t)sample_token<T>(chunk, x));
        ++slot;
      }
    }
  }
  // weights of the chunk's buckets in front of lo
  double sum = 0.0;
  if (!sample_few(p) && tid < kBuckets && own_top > -__builtin_inff() &&
      tid + top_bucket - sample_bucket(own_top, scale) < cut.lo)
    sum = sample_bin_mass(own_bin);
  sum = sample_wave_sum(sum);
  if (lane == kWave - 1) s_sum[wave] = sum, s_units[wave] = units;
  __syncthreads();
  if (tid == 0) {
    units = s_units[0];
    for (int w = 1; w < kScanWaves; ++w) sum += s_sum[w], units += s_units[w];
    a.kept[at] = units + (own_top > -__builtin_inff()
                     ? (uint64_t)__builtin_rint(sum * sample_weight(own_top, top, p.inv_t, a.log2_scale - kBinScale))
                     : 0);
    a.listed[at] = s_listed;
  }
}

// ---------------------------------------------------------------------------
// draw
// ---------------------------------------------------------------------------
// What the launches before left of a row, in its workgroup's first wave.
__device__ __forceinline__ void sample_begin(const SampleArgs& a, int r, SampleShared& sh) {
  const int lane = threadIdx.x & (kWave - 1);
  const size_t at0 = (size_t)r * a.chunks;
  // all loads at once: what is read one after the other costs a microsecond or two each
  const SampleTops tops = sample_tops(a, r);
  uint32_t listed[2];
  uint64_t kept[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const size_t c = at0 + min(lane + i * kWave, a.chunks - 1);
    listed[i] = a.listed[c];
    kept[i] = a.kept[c];
  }
  const SampleCut cut = a.cut[r];
  const SampleRow p = sample_row(a, r);
  const float top = sample_row_top(tops);
  const bool special = !(top > -__builtin_inff());
  if (special) {
    // the first chunk that has a NaN
    int chunk = 0;
#pragma unroll
    for (int i = 1; i >= 0; --i) {
      const uint64_t has = __ballot(lane + i * kWave < a.chunks && tops.top[i] != tops.top[i]);
      if (has) chunk = i * kWave + __builtin_ctzll(has);
    }
    if (lane == 0) sh.picked = chunk, sh.few = ~0u;
  } else {
    bool over = false;
    uint64_t base = 0;
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = lane + i * kWave;
      if (c >= a.chunks) listed[i] = 0, kept[i] = 0;
      over |= listed[i] > (uint32_t)min(kListed, a.list_threads * kHeld);
      if (sample_few(p)) kept[i] = 0;
      sh.chunk[c] = kept[i], sh.listed[c] = listed[i];
      base += sample_of_lane(sample_wave_scan(kept[i]), kWave - 1);
      const uint32_t upto = sample_wave_scan(listed[i]);
      sh.place[c] = all + upto - listed[i];
      all += sample_of_lane(upto, kWave - 1);
    }
    const bool far = __any(over);
    if (lane == 0) {
      sh.base = base, sh.all_listed = all, sh.cut = cut;
      sh.far = far;
      sh.k = p.k ? p.k - cut.before : 0;
      sh.top_p = p.top_p;
    }
  }
  if (lane == 0) {
    sh.top = top, sh.inv_t = p.inv_t;
    sh.special = special;
  }
}

// The token that has the rest of a target behind the tokens before it, of a piece of weights 2^-kChunkScale of its
// largest logit's.
__device__ __forceinline__ uint64_t sample_rest(uint64_t left, float piece_top, float top, double inv_t, int log2_scale,
                                                uint64_t in_piece) {
  const uint64_t target =
      (uint64_t)fmin((double)left / sample_weight(piece_top, top, inv_t, log2_scale - kChunkScale), 0x1p63);
  return target < in_piece ? target : in_piece - 1;
}
__device__ __forceinline__ double sample_piece_weight(float v, float piece_top, double to_log2) {
  return piece_top == __builtin_inff() ? v == piece_top ? __builtin_ldexp(1.0, kChunkScale) : 0.0
                                       : sample_exp2(((double)v - (double)piece_top) * to_log2, kChunkScale);
}
// Of the sum of weights the part in front of the drawn token: floor(u * total).
__device__ __forceinline__ uint64_t sample_target(float u, uint64_t total) {
  const double at = (double)u * (double)total;
  const uint64_t target = at > 0.0 ? at < 9e18 ? (uint64_t)at : ~0ull : 0;
  return target < total ? target : total - 1;
}

// A row without limits, or its largest logit.
template <class T>
__device__ __forceinline__ void sample_draw_free(const SampleArgs& a, int r, const SampleRow& p, const T* row, float u,
                                                 float sub_top, double sub_mass, SampleShared& sh) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const float most = sample_wave_max(sub_top);
  if (lane == 0) sh.tops[wave] = most;
  if (tid == 0) sh.few = ~0u, sh.picked = kSampleThreads;
  const bool nan = __syncthreads_or(sub_top != sub_top);
  const float top = nan ? __builtin_nanf("") : sample_wave_max(sh.tops[lane % kSampleWaves]);
  if (p.greedy || !(top > -__builtin_inff())) {
    const uint64_t has = __ballot(nan ? sub_top != sub_top : sub_top == top);
    if (has && lane == 0) atomicMin(&sh.picked, wave * kWave + __builtin_ctzll(has));
    __syncthreads();
    const int i = sh.picked * kSub + tid;
    const float v = i < a.N ? sample_load(row + i) : -__builtin_inff();
    const uint64_t here = __ballot(i < a.N && (nan ? v != v : v == top));
    if (here && lane == 0) atomicMin(&sh.few, (uint32_t)(i + __builtin_ctzll(here)));
    __syncthreads();
    if (tid == 0) {
      a.tokens[r] = top == -__builtin_inff() ? -1 : (int)sh.few;
      if (a.share) a.share[r] = nan ? top : top == -__builtin_inff() ? 0.0f : 1.0f;
    }
    return;
  }
  const uint64_t sum = sub_top > -__builtin_inff()
                           ? (uint64_t)__builtin_rint(sub_mass * sample_weight(sub_top, top, p.inv_t, a.log2_scale))
                           : 0;
  uint64_t before;
  const uint64_t total = sample_scan(sum, before, kSampleWaves, sh), target = sample_target(u, total);
  if (before <= target && before + sum > target) sh.picked = tid, sh.left = target - before, sh.sub_top = sub_top;
  __syncthreads();
  const int i = sh.picked * kSub + tid;
  const float piece_top = sh.sub_top;
  const float v = i < a.N ? sample_load(row + i) : -__builtin_inff();
  const uint64_t w = sample_units(sample_piece_weight(v, piece_top, p.inv_t * kLog2E));
  const uint64_t in_piece = sample_scan(w, before, kSampleWaves, sh);
  const uint64_t rest = sample_rest(sh.left, piece_top, top, p.inv_t, a.log2_scale, in_piece);
  if (before <= rest && before + w > rest) {
    a.tokens[r] = i;
    // (of the weight itself: a small one's integer has few digits)
    if (a.share) a.share[r] = (float)(sample_weight(v, top, p.inv_t, a.log2_scale) / (double)total);
  }
}

template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ SampleShared sh;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const T* const row = static_cast<const T*>(a.logits) + r * a.stride;
  const size_t at0 = (size_t)r * a.chunks;
  // `threads` threads a chunk for its listed tokens; the first of each is on its way from the start
  const int threads = a.list_threads;
  const int list_chunk = tid / threads, list_at = tid & (threads - 1);
  const uint2* const list = a.list + (at0 + min(list_chunk, a.chunks - 1)) * kListed + list_at;
  const uint2 first_entry = *list;
  const size_t sub = (size_t)r * a.subs + min(tid, a.subs - 1);
  const float sub_top = a.sub_top[sub];
  const double sub_mass = a.sub_mass[sub];
  const float u = a.uniforms ? a.uniforms[r] : 0.0f;
  if (const SampleRow p = sample_row(a, r); !sample_limited(p)) {
    sample_draw_free(a, r, p, row, u, tid < a.subs ? sub_top : -__builtin_inff(), sub_mass, sh);
    return;
  }
  if (wave == 0) sample_begin(a, r, sh);
  __syncthreads();
  const float top = sh.top;
  const double inv_t = sh.inv_t;
  if (sh.special) {
    const bool none = top == -__builtin_inff();
    uint32_t at = ~0u;
    if (!none) {
      const int chunk = sh.picked;
      for (int i = kChunk * chunk + tid; i < min(kChunk * (chunk + 1), a.N); i += kSampleThreads) {
        const float v = sample_load(row + i);
        if (v != v) at = min(at, (uint32_t)i);
      }
    }
    if (at != ~0u) atomicMin(&sh.few, at);
    __syncthreads();
    if (tid == 0) {
      a.tokens[r] = none ? -1 : (int)sh.few;
      if (a.share) a.share[r] = none ? 0.0f : top;
    }
    return;
  }
  auto weight = [&](float v) { return (uint64_t)__builtin_rint(sample_weight(v, top, inv_t, a.log2_scale)); };
  auto weight_of = [&](uint64_t c) { return weight(sample_logit(c)); };
  uint64_t last = sample_order(-__builtin_inff(), W4A16_SAMPLE_MAX_N);      // the last C that is kept (0: no listed token is)
  uint64_t before;
  const bool far = sh.far;      // some chunk lists more than its threads hold
  const int k = sh.k;
  const float top_p = sh.top_p;
  const uint64_t base = sh.base;
  const uint32_t all_listed = sh.all_listed;
  const SampleCut cut = sh.cut;
  const float scale = sample_bucket_scale(inv_t);
  const int top_bucket = sample_bucket(top, scale);
  const bool min_p = cut.least > -__builtin_inf();
  bool check_min_p = min_p;      // (behind last it need not be)
  const int count = list_chunk < a.chunks ? (int)sh.listed[list_chunk] : 0;
  uint64_t c[kHeld];
  auto order = [&](uint2 e) { return sample_order(__uint_as_float(e.x), (int)e.y); };
  if (!far) {
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      c[e] = ~0ull;
      if (list_at + e * threads < count) c[e] = order(e ? list[e * threads] : first_entry);
    }
  }
  if (cut.min_p_alone) {
    // nothing is listed
  } else if (!far && all_listed <= kSorted) {
    // in order: the limits are numbers of tokens
    const int n = (int)all_listed;
    int sorted = kWave;
    while (sorted < n) sorted <<= 1;
#pragma unroll
    for (int e = 0; e < kHeld; ++e)
      if (c[e] != ~0ull) sh.bins[sh.place[list_chunk] + list_at + e * threads] = c[e];
    __syncthreads();
    const uint64_t mine = sample_sort(tid < n ? sh.bins[tid] : ~0ull, sorted, sh.bins + kSampleThreads);
    check_min_p = false;
    bool kept = tid < n;
    uint64_t w = 0;
    if (kept) {
      w = weight_of(mine);
      if (min_p) kept = sample_log_weight(sample_logit(mine), top, inv_t) >= cut.least;
    }
    if (k) kept = kept && tid < k;
    if (top_p < 1.0f) {
      // (of what top_k keeps)
      const uint64_t sum = sample_scan(!k || tid < k ? w : 0, before, sorted / kWave, sh);
      const uint64_t all = k ? base + sum : cut.total;
      kept = kept && (base + before < (uint64_t)__builtin_ceil((double)top_p * (double)all) || base + before == 0);
    }
    const int keep = __syncthreads_count(kept);
    if (tid == keep - 1) sh.found[0] = mine;
    if (kept) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.chunk[(uint32_t)mine / kChunk]), w);
    __syncthreads();
    last = keep ? sh.found[0] : 0;
  } else {
    uint64_t w[kHeld];
    if (!far) {
#pragma unroll
      for (int e = 0; e < kHeld; ++e) w[e] = c[e] != ~0ull ? weight_of(c[e]) : 0;
    }
    // calls f(C, its weight as a function) for the thread's tokens of a chunk, a wave's: those listed, or (of a chunk
    // that has more of them than its list holds) those in lo .. hi
    auto visit_chunk = [&](int chunk, auto&& f) W4K_INLINE {
      const int n = (int)sh.listed[chunk];
      constexpr int AHEAD = 4;      // loads on their way
      if (n <= kListed) {
        const uint2* const from = a.list + (at0 + chunk) * kListed;
        uint2 next[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) next[e] = from[min(lane + e * kWave, kListed - 1)];
        for (int i = lane; i < n; i += kWave) {
          const uint2 entry = next[0];
#pragma unroll
          for (int e = 0; e + 1 < AHEAD; ++e) next[e] = next[e + 1];
          next[AHEAD - 1] = from[min(i + AHEAD * kWave, kListed - 1)];
          const float v = __uint_as_float(entry.x);
          f(sample_order(v, (int)entry.y), [&]() W4K_INLINE { return weight(v); });
        }
      } else {
        const int first = chunk * kChunk + lane, end = min((chunk + 1) * kChunk, a.N);
        float next[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) next[e] = sample_load(row + min(first + e * kWave, a.N - 1));
        for (int i = first; i < end; i += kWave) {
          const float v = next[0];
#pragma unroll
          for (int e = 0; e + 1 < AHEAD; ++e) next[e] = next[e + 1];
          next[AHEAD - 1] = sample_load(row + min(i + AHEAD * kWave, a.N - 1));
          const int b = sample_below(top_bucket, v, scale);
          if (b >= cut.lo && b <= cut.hi) f(sample_order(v, i), [&]() W4K_INLINE { return weight(v); });
        }
      }
    };
    // ... of the row
    auto visit = [&](auto&& f) W4K_INLINE {
      if (far) {
        for (int i = wave; i < a.chunks; i += kSampleWaves) visit_chunk(i, f);
      } else {
#pragma unroll
        for (int e = 0; e < kHeld; ++e)
          if (c[e] != ~0ull) f(c[e], [&]() W4K_INLINE { return w[e]; });
      }
    };
    // All of them lie between the logits that bound the buckets lo .. hi, with half a bucket more at both ends
    // (far logits share the outermost buckets: there, anywhere).
    uint64_t lo = 0, hi = ~0ull;
    const float high = __int_as_float(top_bucket - cut.lo) + 1.0f, low = __int_as_float(top_bucket - cut.hi) - 1.0f;
    if (high < 0x1.fffffep23f && low > 0x1p23f && cut.hi < kBuckets - 1) {
      lo = sample_order(fminf((high - 0x1.8p23f) / scale, top), 0);
      hi = sample_order((low - 0x1.8p23f) / scale, -1);
    }
    // (fewer than k are listed where top_p ends in front of the k-th)
    if (k && all_listed >= (uint32_t)k)
      last = sample_select(
          [&](auto&& f) W4K_INLINE {
            visit([&](uint64_t c, auto&&) W4K_INLINE { f(c, []() W4K_INLINE { return (uint64_t)1; }); });
          },
          [](uint64_t) { return (uint64_t)1; }, (uint64_t)k, lo, hi, last, sh);
    if (top_p < 1.0f) {
      const uint64_t limit = last;
      uint64_t all = cut.total;
      if (k) {
        uint64_t sum = 0;
        visit([&](uint64_t c, auto&& w) W4K_INLINE { sum += c <= limit ? w() : 0; });
        all = base + sample_scan(sum, before, kSampleWaves, sh);
      }
      const uint64_t target = (uint64_t)__builtin_ceil((double)top_p * (double)all);
      if (target <= base && base > 0)
        last = 0;
      else
        last = sample_select(visit, weight_of, target > base ? target - base : 1, lo, min(hi, limit), limit, sh);
    }
    // the kept weights of each chunk, by its wave or the threads that hold its list
    // (additions of one token each to few sums would wait for each other)
    auto kept_weight = [&](uint64_t c, uint64_t w) W4K_INLINE {
      return c <= last && (!min_p || sample_log_weight(sample_logit(c), top, inv_t) >= cut.least) ? w : 0;
    };
    if (far) {
      for (int i = wave; i < a.chunks; i += kSampleWaves) {
        uint64_t sum = 0;
        visit_chunk(i, [&](uint64_t c, auto&& w) W4K_INLINE { sum += c <= last ? kept_weight(c, w()) : 0; });
        sum = sample_wave_scan(sum);
        if (lane == kWave - 1) sh.chunk[i] += sum;
      }
    } else {
      uint64_t sum = 0;
#pragma unroll
      for (int e = 0; e < kHeld; ++e) sum += c[e] != ~0ull ? kept_weight(c[e], w[e]) : 0;
      sum = sample_wave_scan(sum);
      const int part = min(threads, kWave);
      const uint64_t earlier = __shfl((unsigned long long)sum, max(lane - part, 0));
      sum -= lane >= part ? earlier : 0;
      if ((lane & (part - 1)) == part - 1 && list_chunk < a.chunks && sum)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.chunk[list_chunk]), sum);
    }
    __syncthreads();
  }
  // the chunk: the first whose running sum exceeds u * total, that is its whole part
  if (wave == 0) {
    uint64_t sum[2], upto[2], total = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] = lane + i * kWave < a.chunks ? sh.chunk[lane + i * kWave] : 0;
      upto[i] = total + sample_wave_scan(sum[i]);
      total = sample_of_lane(upto[i], kWave - 1);
    }
    const uint64_t target = sample_target(u, total);
    if (lane == 0) sh.picked = 0, sh.left = 0, sh.all = total;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (upto[i] - sum[i] <= target && upto[i] > target) sh.picked = lane + i * kWave, sh.left = target - (upto[i] - sum[i]);
  }
  __syncthreads();
  const int chunk = sh.picked;
  const float chunk_top = a.top[at0 + chunk];      // (kept, as the chunk has a kept token)
  // its tokens, eight a thread
  constexpr int V = kDrawLane;
  const int i0 = chunk * kChunk + tid * V;
  float v[V];
  sample_load_eight(row, i0, a.N, v);
  const float last_v = sample_logit(last);
  const int last_i = (int)(uint32_t)last;
  const double to_log2 = inv_t * kLog2E;
  uint64_t w[V], sum = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    // (tokens of whole buckets come in front of every listed one)
    bool kept = last ? v[e] > last_v || (v[e] == last_v && i0 + e <= last_i) : sample_below(top_bucket, v[e], scale) < cut.lo;
    if (check_min_p)
      kept = kept && (sample_below(top_bucket, v[e], scale) < cut.lo || sample_log_weight(v[e], top, inv_t) >= cut.least);
    w[e] = 0;
    if (kept) w[e] = sample_units(sample_piece_weight(v[e], chunk_top, to_log2));
    sum += w[e];
  }
  const uint64_t in_chunk = sample_scan(sum, before, kSampleWaves, sh);
  const uint64_t target = sample_rest(sh.left, chunk_top, top, inv_t, a.log2_scale, in_chunk);
  if (before <= target && before + sum > target) {
    int e = 0;
#pragma unroll
    for (int i = 0; i + 1 < V; ++i)
      if (e == i && before + w[i] <= target) before += w[i], ++e;
    float drawn = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) drawn = e == i ? v[i] : drawn;
    a.tokens[r] = i0 + e;
    if (a.share) a.share[r] = (float)(sample_weight(drawn, top, inv_t, a.log2_scale) / (double)sh.all);
  }
}

bool sample_sizes(int M, int N) {
  return M >= 0 && M <= W4A16_SAMPLE_MAX_ROWS && N >= 0 && N <= W4A16_SAMPLE_MAX_N;
}

__global__ __launch_bounds__(256) void sample_none_kernel(SampleArgs a) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= a.M) return;
  a.tokens[r] = -1;
  if (a.share) a.share[r] = 0.0f;
}

int sample_chunks(int N) { return (N + kChunk - 1) / kChunk; }

// Rows that go through the launches together: a chunk takes 18.5 KB of workspace.
int sample_rows_at_once(int M, int N) {
  const int most = 8192 / sample_chunks(N);
  return M < most ? M : most;
}

// Places of `rows` rows' arrays in the workspace; the bytes they take.
size_t sample_places(SampleArgs& a, uintptr_t ws, int rows) {
  a.chunks = sample_chunks(a.N);
  a.subs = a.chunks * kScanWaves;
  a.list_threads = kSampleThreads;
  while (a.list_threads * a.chunks > kSampleThreads) a.list_threads >>= 1;
  const size_t n = (size_t)rows * a.chunks;
  size_t at = 0;
  auto take = [&](auto*& p, size_t count) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(ws + at);
    at += (count * sizeof(*p) + 15) / 16 * 16;
  };
  take(a.list, n * kListed);
  take(a.bins, n * kBuckets);
  take(a.sub_mass, n * kScanWaves);
  take(a.kept, n);
  take(a.cut, rows);
  take(a.top, n);
  take(a.sub_top, n * kScanWaves);
  take(a.listed, n);
  return at;
}

template <class T>
void sample_launch(SampleArgs a, void* ws, hipStream_t st) {
  const int at_once = sample_rows_at_once(a.M, a.N);
  const bool limits = a.top_k || a.top_p || a.min_p;
  const int M = a.M;
  for (int r = 0; r < M; r += at_once) {
    a.M = M - r < at_once ? M - r : at_once;
    sample_places(a, (uintptr_t)ws, at_once);
    const dim3 grid(a.chunks, a.M);
    hipLaunchKernelGGL(sample_scan_kernel<T>, grid, dim3(kScanThreads), 0, st, a);
    if (limits && a.chunks * a.M <= kCutAlone) {
      hipLaunchKernelGGL((sample_collect_kernel<T, true>), grid, dim3(kScanThreads), 0, st, a);
    } else if (limits) {
      hipLaunchKernelGGL(sample_cut_kernel, dim3(a.M), dim3(kScanThreads), 0, st, a);
      hipLaunchKernelGGL((sample_collect_kernel<T, false>), grid, dim3(kScanThreads), 0, st, a);
    }
    hipLaunchKernelGGL(sample_draw_kernel<T>, dim3(a.M), dim3(kSampleThreads), 0, st, a);
    // the next rows
    a.logits = static_cast<const T*>(a.logits) + a.M * a.stride;
    a.tokens += a.M;
    for (const float** p : {&a.uniforms, &a.temperature, &a.top_p, &a.min_p})
      if (*p) *p += a.M;
    if (a.top_k) a.top_k += a.M;
    if (a.share) a.share += a.M;
  }
}

}  // namespace

}  // namespace w4k

using namespace w4k;

extern "C" {

size_t w4a16_sample_workspace_bytes(int M, int N) {
  if (!sample_sizes(M, N) || M == 0 || N == 0) return 0;
  SampleArgs a{};
  a.N = N;
  return sample_places(a, 0, sample_rows_at_once(M, N));
}

w4a16_status_t w4a16_sample(const void* logits, int in_dtype, int64_t stride, const float* uniforms,
                            const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                            int32_t* tokens, float* share, void* workspace, size_t workspace_bytes, int M, int N,
                            void* stream) {
  if (in_dtype != W4A16_OUT_BF16 && in_dtype != W4A16_OUT_F32) return W4A16_ERR_UNSUPPORTED;
  if (!sample_sizes(M, N) || stride < N || stride > (1LL << 40)) return W4A16_ERR_SHAPE;
  if (M == 0) return W4A16_OK;
  if (!tokens || (N > 0 && !logits)) return W4A16_ERR_NULL;
  if (!kv_aligned(logits, in_dtype == W4A16_OUT_F32 ? 4 : 2)) return W4A16_ERR_ALIGN;
  for (const void* p : {(const void*)uniforms, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                        (const void*)min_p, (const void*)tokens, (const void*)share})
    if (!kv_aligned(p, 4)) return W4A16_ERR_ALIGN;
  const size_t need = w4a16_sample_workspace_bytes(M, N);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  if (!kv_aligned(workspace, 16)) return W4A16_ERR_ALIGN;
  SampleArgs a{};
  a.logits = logits;
  a.stride = stride;
  a.uniforms = uniforms;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.share = share;
  a.M = M;
  a.N = N;
  a.log2_scale = 62;
  for (int n = N - 1; n > 0; n >>= 1) --a.log2_scale;
  hipStream_t st = (hipStream_t)stream;
  if (N == 0)
    hipLaunchKernelGGL(sample_none_kernel, dim3((M + 255) / 256), dim3(256), 0, st, a);
  else if (in_dtype == W4A16_OUT_F32)
    sample_launch<float>(a, workspace, st);
  else
    sample_launch<uint16_t>(a, workspace, st);
  return kv_launched(hipGetLastError());
}

}  // extern "C"
