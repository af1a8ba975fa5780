// Attention over the paged 8-bit cache (include/w4a16_kv.h).  Compiled once per
// head size (W4K_D = 64, 128, 256).
#include "kv_attn_split.hpp"
#include "kv_device.hpp"

namespace w4k {

namespace {

// The request of token row t: the last r with token_start[r] <= t (empty
// requests share their start with the next one), or -1.
__device__ __forceinline__ int kv_request_of(const int32_t* token_start, int requests, int t) {
  int lo = 0, hi = requests;      // token_start[lo] <= t < token_start[hi] when a request holds t
  if (t < token_start[0] || t >= token_start[requests]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (token_start[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One wave a token row and query head.  Lane j scores cache entry j0 + j, the
// wave keeps the running maximum and sum of the softmax (each step rescales
// what was summed under the old maximum), and each lane sums its D / 64
// output elements over the 64 entries.
template <int D, int TYPE>
__global__ __launch_bounds__(kWave) void kv_attention_row_kernel(KvAttnArgs a) {
  constexpr int E = D / kWave;
  __shared__ float qs[D];
  __shared__ float ps[kWave];
  __shared__ int pg[kWave];
  const int lane = threadIdx.x;
  const int h = blockIdx.x % a.q_heads;
  const int t = blockIdx.x / a.q_heads;
  const int r = kv_request_of(a.token_start, a.requests, t);
  if (r < 0) return;
  const int n = a.token_start[r + 1] - a.token_start[r];
  const int i = t - a.token_start[r];
  if (i >= a.max_new || n * a.group <= kKvSplitRows) return;
  const int kh = h / a.group;
  const int pos = a.seq_lens[r] - n + i;
  const int end = (int)min((long long)min(pos + 1, a.max_len), (long long)a.width << a.c.page_shift);
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  for (int e = lane; e < D; e += kWave) qs[e] = bf16_lo(a.q[(size_t)t * a.q_stride + h * D + e]) * a.scale_log2;
  __syncthreads();
  const int P = 1 << a.c.page_shift;
  float m = -3e38f, l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int j0 = begin; j0 < end; j0 += kWave) {
    const int j = j0 + lane;
    float s = -__builtin_inff(), vs = 0.0f;
    int page = -1;
    if (j < end) {
      page = a.table[(size_t)r * a.width + (j >> a.c.page_shift)];
      if (page < 0 || page >= a.c.pages) page = -1;
    }
    if (page >= 0) {
      const size_t ph = (size_t)page * a.c.heads + kh;
      const uint32_t* kp = reinterpret_cast<const uint32_t*>(a.c.k + (ph * P + (j & (P - 1))) * D);
      float dot = 0.0f;
      for (int e = 0; e < D / 4; ++e) {
        const uint32_t w = kp[e];
        dot = __builtin_fmaf(qs[4 * e], kv_decode<TYPE, 0>(w), dot);
        dot = __builtin_fmaf(qs[4 * e + 1], kv_decode<TYPE, 1>(w), dot);
        dot = __builtin_fmaf(qs[4 * e + 2], kv_decode<TYPE, 2>(w), dot);
        dot = __builtin_fmaf(qs[4 * e + 3], kv_decode<TYPE, 3>(w), dot);
      }
      s = dot * bf16_lo(a.c.ks[ph]);
      vs = bf16_lo(a.c.vs[ph]);
    }
    float top = s;
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    const float m_new = fmaxf(m, top);
    const float fade = exp2f(m - m_new);
    m = m_new;
    const float p = page >= 0 ? exp2f(s - m) : 0.0f;
    l = l * fade + p;
    ps[lane] = page >= 0 ? p * vs : 0.0f;
    pg[lane] = page;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= fade;
    for (int x = 0; x < kWave; ++x) {
      if (pg[x] < 0) continue;
      const size_t ph = (size_t)pg[x] * a.c.heads + kh;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t w = a.c.v[(ph * D + lane + e * kWave) * P + ((j0 + x) & (P - 1))];
        o[e] = __builtin_fmaf(ps[x], kv_decode<TYPE, 0>(w), o[e]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) l += __shfl_xor(l, off);
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[((size_t)t * a.q_heads + h) * D + lane + e * kWave] = (uint16_t)f32_to_bf16(l != 0.0f ? o[e] / l : 0.0f);
}

template <int TYPE>
hipError_t kv_attention_typed(const KvAttnArgs& a, void* workspace, hipStream_t st) {
  constexpr int D = W4K_D;
  float* part_o = static_cast<float*>(workspace);
  float* part_ml = part_o + kv_partials(a) * D;
  const dim3 grid(a.requests, a.c.heads * a.row_groups, a.chunks);
  const int rows = a.split_tokens * a.group;
  auto split = [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    hipLaunchKernelGGL((kv_split_kernel<D, TYPE, NC>), grid, dim3(kKvSplitWaves * kWave), 0, st, a, part_o, part_ml);
    if (a.chunks > 1)
      hipLaunchKernelGGL((kv_join_kernel<D, NC>), dim3(a.requests, a.c.heads, rows), dim3(kKvJoinThreads), 0, st, a,
                         part_o, part_ml);
  };
  if (rows <= 16)
    split(std::integral_constant<int, 1>{});
  else
    split(std::integral_constant<int, 2>{});
  if ((int64_t)a.max_new * a.group > kKvSplitRows)
    hipLaunchKernelGGL((kv_attention_row_kernel<D, TYPE>), dim3((unsigned)((size_t)a.tokens * a.q_heads)), dim3(kWave),
                       0, st, a);
  return hipGetLastError();
}

}  // namespace

#define W4K_CAT_(a, b) a##b
#define W4K_CAT(a, b) W4K_CAT_(a, b)

hipError_t W4K_CAT(kv_attention_d, W4K_D)(int type, const KvAttnArgs& a, void* workspace, hipStream_t st) {
  return type == W4A16_KV_INT8 ? kv_attention_typed<W4A16_KV_INT8>(a, workspace, st)
                               : kv_attention_typed<W4A16_KV_FP8>(a, workspace, st);
}

}  // namespace w4k
