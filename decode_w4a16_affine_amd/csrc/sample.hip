// Sampling from logits (w4a16_sample of include/w4a16_step.h).
//
// A workgroup takes a row.  With C = (falling logit, rising index) as one 64-bit
// number every limit is "the tokens up to some C": top_k's is the C of the k-th
// token, top_p's that of the first token at which the running sum of weights reaches
// its share.  Both are found digit by digit (a histogram of counts or weights of the
// tokens that agree with the digits so far), without sorting.
//
// Weights exp((logit - largest) / temperature) are computed in fp64 and held as
// integers of 2^-e (e = 62 - log2 N: a row's sum stays below 2^63): sums do not depend on
// their order, so histograms may be filled by atomics and the answer is always the same.
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
};

// A row's parameters.
struct SampleRow {
  bool greedy;
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
  return p;
}

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
// The weight times 2^log2_scale
__device__ __forceinline__ double sample_weight(float v, float top, double inv_t, int log2_scale) {
  return __builtin_ldexp(exp(sample_log_weight(v, top, inv_t)), log2_scale);
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
  uint32_t key[kSampleWaves], nan[kSampleWaves];
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

template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_row_kernel(SampleArgs a) {
  __shared__ SampleShared sh;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const T* const row = static_cast<const T*>(a.logits) + r * a.stride;
  const SampleRow p = sample_row(a, r);
  auto result = [&](int token, float share) {
    if (tid == 0) {
      a.tokens[r] = token;
      if (a.share) a.share[r] = share;
    }
  };
  // the largest logit, and the first NaN
  uint32_t key = 0, nan = ~0u;
  for (int i = tid; i < a.N; i += kSampleThreads) {
    const float v = sample_load(row + i);
    if (v != v)
      nan = min(nan, (uint32_t)i);
    else
      key = max(key, sample_key(v));
  }
  for (int off = kWave / 2; off > 0; off >>= 1) {
    key = max(key, (uint32_t)__shfl_xor((int)key, off));
    nan = min(nan, (uint32_t)__shfl_xor((int)nan, off));
  }
  if (lane == 0) sh.key[wave] = key, sh.nan[wave] = nan;
  __syncthreads();
  for (int w = 0; w < kSampleWaves; ++w) key = max(key, sh.key[w]), nan = min(nan, sh.nan[w]);
  const float top = __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key);
  if (nan != ~0u) return result((int)nan, __builtin_nanf(""));
  if (key <= sample_key(-__builtin_inff())) return result(-1, 0.0f);

  auto weight = [&](float v) { return (uint64_t)__builtin_rint(sample_weight(v, top, p.inv_t, a.log2_scale)); };
  auto visit = [&](auto&& f) {
    for (int i = tid; i < a.N; i += kSampleThreads) f(sample_load(row + i), i);
  };
  auto count_of = [&](auto&& f) {
    visit([&](float v, int i) { f(sample_order(v, i), 1); });
  };
  // the last C that is kept
  uint64_t last = ~0ull;
  if (p.greedy || p.top_p <= 0.0f || p.min_p > 1.0f)
    last = sample_select(count_of, 1, sh);
  else {
    if (p.k) last = sample_select(count_of, (uint64_t)p.k, sh);
    if (p.top_p < 1.0f) {
      const uint64_t limit = last;
      uint64_t sum = 0, before;
      visit([&](float v, int i) { sum += sample_order(v, i) <= limit ? weight(v) : 0; });
      const uint64_t total = sample_scan(sum, before, sh.waves);
      const uint64_t target = (uint64_t)__builtin_ceil((double)p.top_p * (double)total);
      last = sample_select(
          [&](auto&& f) {
            visit([&](float v, int i) {
              const uint64_t c = sample_order(v, i);
              if (c <= limit) f(c, weight(v));
            });
          },
          target < 1 ? 1 : target > total ? total : target, sh);
    }
  }
  if (p.greedy) return result((int)(uint32_t)last, 1.0f);
  const double least = p.min_p > 0.0f && p.min_p <= 1.0f ? log((double)p.min_p) : -__builtin_inf();
  auto kept_weight = [&](float v, int i) {
    return sample_order(v, i) <= last && sample_log_weight(v, top, p.inv_t) >= least ? weight(v) : 0;
  };
  // weights of pieces of kSampleSub tokens, a wave a piece
  const int subs = (a.N + kSampleSub - 1) / kSampleSub;
  __syncthreads();
  for (int s = wave; s < subs; s += kSampleWaves) {
    uint64_t sum = 0;
    for (int i = s * kSampleSub + lane; i < min((s + 1) * kSampleSub, a.N); i += kWave)
      sum += kept_weight(sample_load(row + i), i);
    for (int off = kWave / 2; off > 0; off >>= 1) sum += __shfl_xor((unsigned long long)sum, off);
    if (lane == 0) sh.bins[s] = sum;
  }
  __syncthreads();
  uint64_t before;
  uint64_t sum = tid < subs ? sh.bins[tid] : 0;
  const uint64_t total = sample_scan(sum, before, sh.waves);
  // the first running sum above u * total is the first above its whole part
  const double at = (double)a.uniforms[r] * (double)total;
  uint64_t target = at > 0.0 ? at < 9e18 ? (uint64_t)at : ~0ull : 0;
  target = target < total ? target : total - 1;
  if (before <= target && before + sum > target) sh.found[0] = tid, sh.found[1] = before;
  __syncthreads();
  const int sub = (int)sh.found[0];
  const uint64_t base = sh.found[1];
  const int i = sub * kSampleSub + tid;
  sum = i < a.N ? kept_weight(sample_load(row + i), i) : 0;
  sample_scan(sum, before, sh.waves);
  before += base;
  if (before <= target && before + sum > target) {
    a.tokens[r] = i;
    // (of the weight itself: a small one's integer has few digits)
    if (a.share) a.share[r] = (float)(sample_weight(sample_load(row + i), top, p.inv_t, a.log2_scale) / (double)total);
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

}  // namespace

}  // namespace w4k

using namespace w4k;

extern "C" {

size_t w4a16_sample_workspace_bytes(int M, int N) {
  (void)M, (void)N;
  return 0;
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
  SampleArgs a{logits, stride, uniforms, temperature, top_p, min_p, top_k, tokens, share, M, N, 62};
  for (int n = N - 1; n > 0; n >>= 1) --a.log2_scale;
  hipStream_t st = (hipStream_t)stream;
  if (N == 0)
    hipLaunchKernelGGL(sample_none_kernel, dim3((M + 255) / 256), dim3(256), 0, st, a);
  else if (in_dtype == W4A16_OUT_F32)
    hipLaunchKernelGGL(sample_row_kernel<float>, dim3(M), dim3(kSampleThreads), 0, st, a);
  else
    hipLaunchKernelGGL(sample_row_kernel<uint16_t>, dim3(M), dim3(kSampleThreads), 0, st, a);
  return kv_launched(hipGetLastError());
}

}  // extern "C"
