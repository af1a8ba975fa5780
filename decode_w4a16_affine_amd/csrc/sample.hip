// Sampling from logits (w4a16_sample of include/w4a16_step.h).
//
// With C = (falling logit, rising index) as one 64-bit number every limit is "the tokens up
// to some C": top_k's is the C of the k-th token, top_p's that of the first token at which
// the running sum of weights reaches its share.  So nothing is sorted: a histogram over
// buckets of logits (1 / 8 of a temperature wide) tells which buckets the limits lie in, and
// only those buckets' tokens are looked at one by one.
//
// Launches.  scan: a workgroup reads a chunk of 8192 logits into registers; its largest
// logit, and either the sum of its weights (rows without limits) or its histogram.  cut: a
// workgroup a row adds the histograms and finds the buckets lo .. hi that the limits
// lie in.  collect: reads the logits again and lists the tokens of these buckets.  draw: a
// workgroup a row finds the last kept token among the listed ones, adds the kept weights
// of each chunk, picks a chunk and looks up the token in it.  A call without limits skips cut
// and collect.  A row whose lists overflow (thousands of tokens of a chunk in one bucket: ties)
// is left to one workgroup, which finds the limits digit by digit from the logits themselves.
//
// Weights exp((logit - largest) / temperature) are computed in fp64 and added as integers of
// 2^-e (e = 62 - log2 N for a row: its sum stays below 2^63), or in a fixed order: sums do not
// depend on the order in which atomics arrive, and the answer is always the same.
// (fp32 would be off by 2^-24 of the larger weights at every border between the tokens,
// of which a row has up to 2^20.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_host.hpp"
#include "w4a16_step.h"

namespace w4k {

namespace {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / kWave;
constexpr int kSampleSub = 1024;      // tokens whose weights are summed together before the draw
constexpr int kSampleSubs = W4A16_SAMPLE_MAX_N / kSampleSub;
constexpr int kSampleBins = 2048;
constexpr int kScanThreads = 512;
constexpr int kScanWaves = kScanThreads / kWave;
constexpr int kLane = 16;                             // logits a lane holds
constexpr int kChunk = kScanThreads * kLane;          // and a workgroup
constexpr int kChunks = W4A16_SAMPLE_MAX_N / kChunk;
constexpr int kBuckets = 256;
constexpr float kBucketsPerUnit = 8.0f;               // of (logit / temperature)
constexpr int kListed = 1024;                         // tokens of a chunk that are listed at most
constexpr int kSmallK = 512;                          // limits of so few tokens need no weights from the scan
constexpr int kChunkScale = 49;                       // a chunk's weights are multiples of 2^-49 (8192 of them below 2^63)
static_assert(kChunk == 1 << (62 - kChunkScale) && kChunks <= kSampleThreads && kBuckets <= kScanThreads, "");
static_assert(kSampleSub == kSampleThreads && kSampleSubs <= kSampleThreads, "one thread a token, or a piece");

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
  float* top;          // [M][chunks] largest logit of a chunk, NaN if it has one
  uint32_t* top_at;    // [M][chunks] its first token, or the first NaN
  double* mass;        // [M][chunks] rows without limits: weights, of a chunk's largest logit
  uint64_t* kept;      // [M][chunks] others: weights of the buckets in front of lo, of a row's
  uint64_t* bins;      // [M][chunks][kBuckets] weights of a chunk's buckets, of its largest logit
  uint32_t* counts;    // [M][chunks][kBuckets] tokens of a chunk's buckets
  uint64_t* total;     // [M][chunks] weights of a chunk
  uint32_t* listed;    // [M][chunks] tokens in lo .. hi
  uint2* list;         // [M][chunks][kListed] these: logit, token
  struct SampleCut* cut;      // [M]
};

// Where a row's limits lie.
struct SampleCut {
  int lo, hi;          // buckets
  int before;          // tokens in front of lo
  int min_p_alone;     // top_k and top_p end behind hi
  uint64_t total;      // all weights, of the row's largest logit
};

// A row's parameters.
struct SampleRow {
  bool greedy;         // the largest logit is the only one kept
  double inv_t;        // 1 / temperature
  int k;               // 0: no limit
  float top_p, min_p;  // >= 1, 0: no limit
};

__device__ __forceinline__ SampleRow sample_row(const SampleArgs& a, int r) {
  SampleRow p;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  p.greedy = !(t > 0.0f) || !a.uniforms;
  p.inv_t = 1.0 / (double)fminf(t, 3.402823466e38f);
  p.k = a.top_k ? a.top_k[r] : 0;
  p.k = p.k > 0 && p.k < a.N ? p.k : 0;
  p.top_p = a.top_p ? a.top_p[r] : 1.0f;
  p.top_p = p.top_p < 1.0f ? p.top_p : 1.0f;
  p.min_p = a.min_p ? a.min_p[r] : 0.0f;
  p.min_p = p.min_p > 0.0f ? p.min_p : 0.0f;
  p.greedy |= p.top_p <= 0.0f || p.min_p > 1.0f;
  return p;
}
__device__ __forceinline__ bool sample_limited(const SampleRow& p) { return p.k || p.top_p < 1.0f || p.min_p > 0.0f; }
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
// Position in the order of falling logits: smaller comes first.
__device__ __forceinline__ uint64_t sample_order(float v, int i) { return (uint64_t)~sample_key(v) << 32 | (uint32_t)i; }

__device__ __forceinline__ double sample_log_weight(float v, float top, double inv_t) {
  return v == top ? 0.0 : ((double)v - (double)top) * inv_t;
}
// The weight times 2^log2_scale.  2^t = 2^n 2^f with |f| <= 1/2, the latter by its Taylor series to
// f^11: off by 2^-47 of it (the rest of the series 2^-47, t's rounding 2^-47 where t is above -64).
__device__ __forceinline__ double sample_weight(float v, float top, double inv_t, int log2_scale) {
  const double t = fmax(sample_log_weight(v, top, inv_t) * 1.4426950408889634074, -1000.0);
  const double n = __builtin_rint(t), f = t - n;
  double y = 4.4455382718708101e-10;
  y = __builtin_fma(y, f, 7.0549116208011209e-09);
  y = __builtin_fma(y, f, 1.0178086009239696e-07);
  y = __builtin_fma(y, f, 1.3215486790144305e-06);
  y = __builtin_fma(y, f, 1.5252733804059838e-05);
  y = __builtin_fma(y, f, 1.5403530393381606e-04);
  y = __builtin_fma(y, f, 1.3333558146428441e-03);
  y = __builtin_fma(y, f, 9.6181291076284769e-03);
  y = __builtin_fma(y, f, 5.5504108664821576e-02);
  y = __builtin_fma(y, f, 2.4022650695910071e-01);
  y = __builtin_fma(y, f, 6.9314718055994529e-01);
  y = __builtin_fma(y, f, 1.0);
  return __builtin_ldexp(y, (int)n + log2_scale);
}
// The same rounded to an integer, for scales up to 2^49: it appears in the low bits of 2^52 and it.
__device__ __forceinline__ uint64_t sample_units(float v, float top, double inv_t) {
  return (uint64_t)__double_as_longlong(sample_weight(v, top, inv_t, kChunkScale) + 0x1p52) & 0xFFFFFFFFFFFFFull;
}

// A logit's bucket counted from any fixed one; grows with the logit.  (Far logits share
// the outermost ones.)
__device__ __forceinline__ float sample_bucket_scale(double inv_t) {
  return fminf(kBucketsPerUnit * (float)inv_t, 0x1p100f);
}
__device__ __forceinline__ int sample_bucket(float v, float scale) {
  return (int)__builtin_floorf(fminf(fmaxf(v * scale, -0x1p23f), 0x1p23f));
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
#pragma unroll
  for (int x = 0; x < kLane; x += V) sample_load_row<V>(row, sample_token<T>(chunk, x), N, v + x);
}

// Sums over the block's threads.  Values of threads before this one, and of all (returned).
__device__ __forceinline__ uint64_t sample_scan(uint64_t v, uint64_t& before, uint64_t (&s_waves)[kSampleWaves]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  uint64_t sum = v;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const uint64_t o = __shfl_up((unsigned long long)sum, off);
    if (lane >= off) sum += o;
  }
  __syncthreads();      // (s_waves may still be read from a scan before)
  if (lane == kWave - 1) s_waves[wave] = sum;
  __syncthreads();
  uint64_t total = 0, earlier = 0;
#pragma unroll
  for (int w = 0; w < kSampleWaves; ++w) {
    if (w == wave) earlier = total;
    total += s_waves[w];
  }
  before = earlier + sum - v;
  return total;
}

struct SampleShared {
  uint64_t bins[kSampleBins];
  uint64_t waves[kSampleWaves];
  uint64_t found[2];
  uint64_t chunk[kChunks];      // kept weights
  uint32_t listed[kChunks];
};

// The first C (in order) at which the running sum of `measure` reaches target, 1 <=
// target <= the sum over all.  visit(f) calls f(C, measure) for the thread's tokens.
template <class Visit>
__device__ uint64_t sample_select(Visit&& visit, uint64_t target, SampleShared& sh) {
  // digits of C: 11, 11 and 10 bits of the logit, 12 (always 0), 10 and 10 of the index
  constexpr int shifts[5] = {53, 42, 32, 10, 0};
  uint64_t prefix = 0, base = 0;      // C's digits so far; the sum in front of them
  int known = 64;                     // bits below which C is not known yet
#pragma unroll 1
  for (int d = 0; d < 5; ++d) {
    const int shift = shifts[d];
    for (int b = threadIdx.x; b < kSampleBins; b += kSampleThreads) sh.bins[b] = 0;
    __syncthreads();
    visit([&](uint64_t c, uint64_t measure) {
      if (known == 64 || c >> known == prefix >> known)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[(c >> shift) & (kSampleBins - 1)]), measure);
    });
    __syncthreads();
    const uint64_t v0 = sh.bins[2 * threadIdx.x], v1 = sh.bins[2 * threadIdx.x + 1];
    uint64_t before;
    sample_scan(v0 + v1, before, sh.waves);
    before += base;
    if (before < target && before + v0 + v1 >= target) {      // one thread's
      const bool second = before + v0 < target;
      sh.found[0] = 2 * threadIdx.x + second;
      sh.found[1] = before + (second ? v0 : 0);
    }
    __syncthreads();
    prefix |= sh.found[0] << shift;
    base = sh.found[1];
    known = d == 2 ? 20 : shift;
    __syncthreads();
  }
  return prefix;
}

// A row's chunks: its largest logit and that one's token, or its first NaN's.
struct SampleTop {
  float top;
  uint32_t at;
};
__device__ __forceinline__ SampleTop sample_row_top(const SampleArgs& a, int r) {
  // every wave goes through all chunks (up to 128: two a lane)
  const int lane = threadIdx.x & (kWave - 1);
  float top = -__builtin_inff();
  uint32_t at = ~0u, nan = ~0u;
  for (int c = lane; c < a.chunks; c += kWave) {
    const float v = a.top[(size_t)r * a.chunks + c];
    const uint32_t i = a.top_at[(size_t)r * a.chunks + c];
    if (v != v)
      nan = min(nan, i);
    else if (v > top || at == ~0u)
      top = v, at = i;
  }
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) {
    const float v = __shfl_xor(top, off);
    const uint32_t i = (uint32_t)__shfl_xor((int)at, off);
    nan = min(nan, (uint32_t)__shfl_xor((int)nan, off));
    if (v > top || (v == top && i < at)) top = v, at = i;
  }
  return nan != ~0u ? SampleTop{__builtin_nanf(""), nan} : SampleTop{top, at};
}

// ---------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(kScanThreads) void sample_scan_kernel(SampleArgs a) {
  __shared__ uint64_t s_bins[kBuckets];
  __shared__ uint32_t s_counts[kBuckets];
  __shared__ float s_top[kScanWaves];
  __shared__ uint32_t s_at[kScanWaves];
  __shared__ double s_sum[kScanWaves];
  const int chunk = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const T* const row = static_cast<const T*>(a.logits) + r * a.stride;
  float v[kLane];
  sample_load_chunk(row, chunk, a.N, v);
  const SampleRow p = sample_row(a, r);
  if (tid < kBuckets) s_bins[tid] = 0, s_counts[tid] = 0;
  const size_t at = (size_t)r * a.chunks + chunk;
  // the largest logit (fmaxf leaves NaN out), and the first token that has it or is NaN
  float top = v[0];
  bool nan = false;
#pragma unroll
  for (int x = 0; x < kLane; ++x) {
    top = fmaxf(top, v[x]);
    nan |= v[x] != v[x];
  }
  top = top == top ? top : -__builtin_inff();
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  if (lane == 0) s_top[wave] = top;
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int w = 0; w < kScanWaves; ++w) top = fmaxf(top, s_top[w]);
  uint32_t first = ~0u;
#pragma unroll
  for (int x = kLane - 1; x >= 0; --x)      // (a lane's tokens grow with x)
    if (nan ? v[x] != v[x] : v[x] == top) first = sample_token<T>(chunk, x);
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) first = min(first, (uint32_t)__shfl_xor((int)first, off));
  if (lane == 0) s_at[wave] = first;
  double sum = 0.0;
  if (!p.greedy && !nan && top > -__builtin_inff()) {
    if (!sample_limited(p)) {
#pragma unroll
      for (int x = 0; x < kLane; ++x) sum += sample_weight(v[x], top, p.inv_t, 0);
#pragma unroll
      for (int off = kWave / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    } else {
      const float scale = sample_bucket_scale(p.inv_t);
      const int top_bucket = sample_bucket(top, scale);
      const bool few = sample_few(p);
      uint64_t units = 0;
#pragma unroll
      for (int x = 0; x < kLane; ++x) {
        const int b = sample_below(top_bucket, v[x], scale);
        const uint64_t w = few ? 0 : sample_units(v[x], top, p.inv_t);
        units += w;
        // (what the last bucket has is the rest)
        if (b < kBuckets - 1) {
          atomicAdd(&s_counts[b], 1u);
          if (!few) atomicAdd(reinterpret_cast<unsigned long long*>(&s_bins[b]), w);
        }
      }
#pragma unroll
      for (int off = kWave / 2; off > 0; off >>= 1) units += __shfl_xor((unsigned long long)units, off);
      sum = __longlong_as_double((long long)units);
    }
  }
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 0; w < kScanWaves; ++w) first = min(first, s_at[w]);
    a.top[at] = nan ? __builtin_nanf("") : top;
    a.top_at[at] = first;
    double all = 0.0;
    uint64_t units = 0;
#pragma unroll
    for (int w = 0; w < kScanWaves; ++w) {
      all += s_sum[w];
      units += (uint64_t)__double_as_longlong(s_sum[w]);
    }
    a.mass[at] = all;
    a.total[at] = units;
  }
  if (sample_limited(p) && tid < kBuckets) {
    a.counts[at * kBuckets + tid] = s_counts[tid];
    if (!sample_few(p)) a.bins[at * kBuckets + tid] = s_bins[tid];
  }
}

// ---------------------------------------------------------------------------
// cut: a thread a bucket
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kBuckets) void sample_cut_kernel(SampleArgs a) {
  __shared__ double s_factor[kChunks];
  __shared__ int s_shift[kChunks];
  __shared__ double s_waves[kBuckets / kWave];
  __shared__ uint32_t s_counts[kBuckets / kWave];
  __shared__ double s_mass[kBuckets];
  __shared__ uint32_t s_count[kBuckets];
  __shared__ int s_first[4];
  const int r = blockIdx.x, b = threadIdx.x, lane = b & (kWave - 1), wave = b / kWave;
  const SampleRow p = sample_row(a, r);
  const SampleTop row = sample_row_top(a, r);
  if (p.greedy || !sample_limited(p) || !(row.top > -__builtin_inff())) return;
  const bool few = sample_few(p);
  const float scale = sample_bucket_scale(p.inv_t);
  const int top_bucket = sample_bucket(row.top, scale);
  double total = 0.0;
  for (int c = b; c < a.chunks; c += kBuckets) {
    const float top = a.top[(size_t)r * a.chunks + c];
    // (a chunk of -infinity alone has no weights; its tokens lie in the last bucket)
    s_factor[c] = top > -__builtin_inff() ? sample_weight(top, row.top, p.inv_t, 0) : 0.0;
    s_shift[c] = top > -__builtin_inff() ? min(top_bucket - sample_bucket(top, scale), kBuckets) : kBuckets;
  }
  if (b < 4) s_first[b] = kBuckets - 1;
  __syncthreads();
  double mass = 0.0;
  uint32_t count = 0;
  for (int c = 0; c < a.chunks; ++c) {
    const size_t at = (size_t)r * a.chunks + c;
    if (!few) total += __builtin_ldexp((double)a.total[at], -kChunkScale) * s_factor[c];
    const int from = b - s_shift[c];
    if (from < 0 || b == kBuckets - 1) continue;
    count += a.counts[at * kBuckets + from];
    if (!few) mass += __builtin_ldexp((double)a.bins[at * kBuckets + from], -kChunkScale) * s_factor[c];
  }
  // sums over the buckets up to this one, in a fixed order
  double upto = mass;
  uint32_t counted = count;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const double m = __shfl_up(upto, off);
    const uint32_t n = (uint32_t)__shfl_up((int)counted, off);
    if (lane >= off) upto += m, counted += n;
  }
  if (lane == kWave - 1) s_waves[wave] = upto, s_counts[wave] = counted;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += s_waves[w], counted += s_counts[w];
  if (b == kBuckets - 1) upto = total, counted = a.N;
  s_mass[b] = upto, s_count[b] = counted;
  __syncthreads();
  // the first bucket at which each limit may lie; the last one if none does
  if (p.k && counted >= (uint32_t)p.k) atomicMin(&s_first[0], b);
  __syncthreads();
  const int k_at = p.k ? s_first[0] : kBuckets;
  int lo = k_at, hi = k_at;
  bool min_p_alone = false;
  if (few) {
    lo = 0;
  } else {
    if (p.top_p < 1.0f) {
      // Sums are exact to 2^-40: a border that near leaves both buckets open.  The weights that top_k
      // keeps end somewhere in its bucket.
      const double least = p.k ? (k_at ? s_mass[k_at - 1] : 0.0) : total, most = p.k ? s_mass[k_at] : total;
      if (upto * (1.0 + 0x1p-40) >= p.top_p * least) atomicMin(&s_first[1], b);
      if (upto >= p.top_p * most * (1.0 + 0x1p-40)) atomicMin(&s_first[2], b);
      __syncthreads();
      lo = min(lo, s_first[1]);
      hi = p.k ? k_at : s_first[2];      // (with top_k, its sum is needed exactly)
    }
    if (p.min_p > 0.0f) {
      // the bucket of the least weight, by fp32 arithmetic on its edge: one to either side
      const float edge = (float)((double)row.top + log((double)p.min_p) / p.inv_t);
      const int at = sample_below(top_bucket, fminf(fmaxf(edge, -3e38f), row.top), scale);
      min_p_alone = at + 1 < lo || (!p.k && p.top_p >= 1.0f);
      if (min_p_alone) hi = at + 1;
      lo = min(lo, at - 1);
    }
  }
  lo = max(lo, 0), hi = min(hi, kBuckets - 1);
  if (b == 0)
    a.cut[r] = SampleCut{lo, hi, lo ? (int)s_count[lo - 1] : 0, min_p_alone,
                         (uint64_t)__builtin_rint(__builtin_ldexp(total, a.log2_scale))};
}

// ---------------------------------------------------------------------------
// collect
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(kScanThreads) void sample_collect_kernel(SampleArgs a) {
  __shared__ uint32_t s_count;
  __shared__ double s_sum[kScanWaves];
  const int chunk = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const SampleRow p = sample_row(a, r);
  if (p.greedy || !sample_limited(p)) return;
  const T* const row = static_cast<const T*>(a.logits) + r * a.stride;
  float v[kLane];
  sample_load_chunk(row, chunk, a.N, v);
  const SampleTop top = sample_row_top(a, r);
  if (!(top.top > -__builtin_inff())) return;
  const SampleCut cut = a.cut[r];
  if (tid == 0) s_count = 0;
  __syncthreads();
  const size_t at = (size_t)r * a.chunks + chunk;
  const float scale = sample_bucket_scale(p.inv_t);
  const int top_bucket = sample_bucket(top.top, scale);
#pragma unroll
  for (int x = 0; x < kLane; ++x) {
    const int i = sample_token<T>(chunk, x), b = sample_below(top_bucket, v[x], scale);
    const bool mine = b >= cut.lo && b <= cut.hi && i < a.N;
    const uint64_t all = __ballot(mine);
    if (!all) continue;
    uint32_t slot = 0;
    if (lane == __builtin_ctzll(all)) slot = atomicAdd(&s_count, (uint32_t)__builtin_popcountll(all));
    slot = (uint32_t)__shfl((int)slot, __builtin_ctzll(all)) + __builtin_popcountll(all & ((1ull << lane) - 1));
    if (mine && slot < kListed) a.list[at * kListed + slot] = make_uint2(__float_as_uint(v[x]), (uint32_t)i);
  }
  // weights of the chunk's buckets in front of lo
  const float chunk_top = a.top[at];
  double sum = 0.0;
  if (!sample_few(p) && tid < kBuckets && chunk_top > -__builtin_inff() &&
      tid + top_bucket - sample_bucket(chunk_top, scale) < cut.lo)
    sum = __builtin_ldexp((double)a.bins[at * kBuckets + tid], -kChunkScale);
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kScanWaves; ++w) sum += s_sum[w];
    a.kept[at] = chunk_top > -__builtin_inff()
                     ? (uint64_t)__builtin_rint(sum * sample_weight(chunk_top, top.top, p.inv_t, a.log2_scale))
                     : 0;
    a.listed[at] = s_count;
  }
}

// ---------------------------------------------------------------------------
// draw
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ SampleShared sh;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const T* const row = static_cast<const T*>(a.logits) + r * a.stride;
  const SampleRow p = sample_row(a, r);
  const SampleTop first = sample_row_top(a, r);
  const float top = first.top;
  if (p.greedy || !(top > -__builtin_inff())) {
    if (tid == 0) {
      a.tokens[r] = top == -__builtin_inff() ? -1 : (int)first.at;
      if (a.share) a.share[r] = top != top ? top : top == -__builtin_inff() ? 0.0f : 1.0f;
    }
    return;
  }
  auto weight = [&](float v) { return (uint64_t)__builtin_rint(sample_weight(v, top, p.inv_t, a.log2_scale)); };
  const size_t at0 = (size_t)r * a.chunks;
  uint64_t last = ~0ull;      // the last C that top_k and top_p keep
  int sure = kBuckets;        // buckets in front of it are kept whole
  const double least = p.min_p > 0.0f ? log((double)p.min_p) : -__builtin_inf();
  const float scale = sample_bucket_scale(p.inv_t);
  const int top_bucket = sample_bucket(top, scale);
  if (!sample_limited(p)) {
    if (tid < a.chunks) {
      const float chunk_top = a.top[at0 + tid];
      sh.chunk[tid] = chunk_top > -__builtin_inff()
                          ? (uint64_t)__builtin_rint(a.mass[at0 + tid] * sample_weight(chunk_top, top, p.inv_t, a.log2_scale))
                          : 0;
    }
    __syncthreads();
  } else {
    const SampleCut cut = a.cut[r];
    uint64_t kept = 0;
    int listed = 0;
    if (tid < a.chunks) {
      listed = (int)a.listed[at0 + tid];
      kept = sample_few(p) ? 0 : a.kept[at0 + tid];
      sh.listed[tid] = min(listed, kListed);
      sh.chunk[tid] = kept;
    }
    const bool overflow = __syncthreads_or(listed > kListed);
    // tokens whose order decides: those listed, or all of the row behind `sure` whole buckets
    sure = overflow ? 0 : cut.lo;
    if (overflow && tid < a.chunks) sh.chunk[tid] = 0, kept = 0;
    uint64_t before;
    const uint64_t base = sample_scan(kept, before, sh.waves);      // (and a barrier)
    auto visit = [&](auto&& f) {
      if (overflow) {
        for (int i = tid; i < a.N; i += kSampleThreads) f(sample_load(row + i), i);
      } else {
        for (int c = wave; c < a.chunks; c += kSampleWaves)
          for (int j = lane; j < (int)sh.listed[c]; j += kWave) {
            const uint2 e = a.list[(at0 + c) * kListed + j];
            f(__uint_as_float(e.x), (int)e.y);
          }
      }
    };
    bool none = false;      // no listed token is kept
    const bool others = overflow || !cut.min_p_alone;
    if (p.k && others) {
      const int64_t k = p.k - (overflow ? 0 : cut.before);
      uint64_t count = 0;
      visit([&](float, int) { ++count; });
      // (fewer are listed where top_p ends in front of the k-th)
      if ((int64_t)sample_scan(count, before, sh.waves) >= k)
        last = sample_select([&](auto&& f) { visit([&](float v, int i) { f(sample_order(v, i), 1); }); }, (uint64_t)k, sh);
    }
    if (p.top_p < 1.0f && others) {
      const uint64_t limit = last;
      uint64_t sum = 0;
      visit([&](float v, int i) { sum += sample_order(v, i) <= limit ? weight(v) : 0; });
      sum = sample_scan(sum, before, sh.waves);
      const uint64_t all = p.k || overflow ? base + sum : cut.total;
      const uint64_t target = (uint64_t)__builtin_ceil((double)p.top_p * (double)all);
      if (target <= base && base > 0)
        none = true;
      else if (target - base < sum)
        last = sample_select(
            [&](auto&& f) {
              visit([&](float v, int i) {
                const uint64_t c = sample_order(v, i);
                if (c <= limit) f(c, weight(v));
              });
            },
            target > base ? target - base : 1, sh);
    }
    if (none) last = 0;
    visit([&](float v, int i) {
      if (sample_order(v, i) <= last && sample_log_weight(v, top, p.inv_t) >= least)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.chunk[i / kChunk]), weight(v));
    });
    __syncthreads();
  }
  // the chunk: the first whose running sum exceeds u * total, that is its whole part
  uint64_t before;
  uint64_t sum = tid < a.chunks ? sh.chunk[tid] : 0;
  const uint64_t total = sample_scan(sum, before, sh.waves);
  const double at = (double)a.uniforms[r] * (double)total;
  uint64_t target = at > 0.0 ? at < 9e18 ? (uint64_t)at : ~0ull : 0;
  target = target < total ? target : total - 1;
  if (tid == 0) sh.found[0] = 0, sh.found[1] = 0;
  __syncthreads();
  if (before <= target && before + sum > target) sh.found[0] = tid, sh.found[1] = target - before;
  __syncthreads();
  const int chunk = (int)sh.found[0];
  const uint64_t into = sh.found[1];
  const float chunk_top = a.top[at0 + chunk];      // (kept, as the chunk has a kept token)
  // its tokens, eight a thread
  constexpr int V = kChunk / kSampleThreads;
  const int i0 = chunk * kChunk + tid * V;
  float v[V];
  sample_load_row<V <= kPiece<T> ? V : kPiece<T>>(row, i0, a.N, v);
  if constexpr (V > kPiece<T>) sample_load_row<kPiece<T>>(row, i0 + kPiece<T>, a.N, v + kPiece<T>);
  uint64_t w[V];
  sum = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const bool kept = sample_limited(p) ? sample_below(top_bucket, v[e], scale) < sure ||
                                              (sample_order(v[e], i0 + e) <= last &&
                                               sample_log_weight(v[e], top, p.inv_t) >= least)
                                        : true;
    w[e] = kept ? sample_units(v[e], chunk_top, p.inv_t) : 0;
    sum += w[e];
  }
  const uint64_t in_chunk = sample_scan(sum, before, sh.waves);
  target = (uint64_t)fmin((double)into / sample_weight(chunk_top, top, p.inv_t, a.log2_scale - kChunkScale), 0x1p63);
  target = target < in_chunk ? target : in_chunk - 1;
  if (before <= target && before + sum > target) {
    int e = 0;
#pragma unroll
    for (int i = 0; i + 1 < V; ++i)
      if (e == i && before + w[i] <= target) before += w[i], ++e;
    float drawn = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) drawn = e == i ? v[i] : drawn;
    a.tokens[r] = i0 + e;
    // (of the weight itself: a small one's integer has few digits)
    if (a.share) a.share[r] = (float)(sample_weight(drawn, top, p.inv_t, a.log2_scale) / (double)total);
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

// Rows that go through the launches together: a chunk takes 11.5 KB of workspace.
int sample_rows_at_once(int M, int N) {
  const int most = 16384 / sample_chunks(N);
  return M < most ? M : most;
}

// Places of `rows` rows' arrays in the workspace; the bytes they take.
size_t sample_places(SampleArgs& a, uintptr_t ws, int rows) {
  a.chunks = sample_chunks(a.N);
  const size_t n = (size_t)rows * a.chunks;
  size_t at = 0;
  auto take = [&](auto*& p, size_t count) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(ws + at);
    at += (count * sizeof(*p) + 15) / 16 * 16;
  };
  take(a.list, n * kListed);
  take(a.bins, n * kBuckets);
  take(a.counts, n * kBuckets);
  take(a.mass, n);
  take(a.kept, n);
  take(a.total, n);
  take(a.cut, rows);
  take(a.top, n);
  take(a.top_at, n);
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
    if (limits) {
      hipLaunchKernelGGL(sample_cut_kernel, dim3(a.M), dim3(kBuckets), 0, st, a);
      hipLaunchKernelGGL(sample_collect_kernel<T>, grid, dim3(kScanThreads), 0, st, a);
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
