// Norms of queries and keys for each head with the position rotation
// (w4a16_qk_norm_rope of include/w4a16_step.h).
//
// D / 8 lanes hold a head, 8 elements each, so a wave has 8, 4 or 2 heads of a
// token at once.  The rotation pairs elements rot / 2 apart, so lane l takes two
// pieces of four that are pairs of each other, 4 l .. + 3 and rot / 2 + 4 l .. + 3, and no
// element changes lanes (neighbouring pairs: the 8 elements in a row).  Lanes past the
// rotated elements take 8 in a row.  The sum of squares goes over D / 8 lanes by row
// operations, in a fixed order.
//
// A lane's four pairs are the same in every head: their sines are computed once a
// token and wave.  The angle in turns is position * frequency / 2 pi in fp64 (a far
// position has thousands of turns, whose fraction fp32 would lose), its
// fraction's sine and cosine in fp32.
//
// Bound and measured: rows read and written once.  11801 tokens of 40 heads of 128,
// 242 MB: 47 us, 5.2 TB/s (a copy of 2 GiB: 4.9); 4099 of 20 with positions of
// three axes, 42 MB: 10.5 us, 4.0 TB/s.  A step of 48 tokens takes 3.2 us in a graph: one launch and
// two loads that wait for each other (positions and rows).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_host.hpp"
#include "w4a16_step.h"

namespace w4k {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWaves = kRopeThreads / kWave;
constexpr int kRopeFill = 2048;      // waves that share a step's heads

struct RopeArgs {
  const uint16_t *q, *k, *qw, *kw;
  uint16_t *qo, *ko;
  int64_t qs, ks, qos, kos;
  const float* inv_freq;
  const int32_t* positions;
  int tokens, q_heads, heads, rot;       // heads: queries' and keys'
  int parts, span;                       // waves a token, wave-fuls of heads a wave
  int axes, end[W4A16_ROPE_MAX_AXES - 1];      // end[a]: the first pair past axis a's section
  float eps, offset;
};

typedef float rope_f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 rope_bf16x4 __attribute__((ext_vector_type(4)));

template <int CTRL>
__device__ __forceinline__ float rope_add_row(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// The sum over each L = 8, 16 or 32 lanes, to all of them.
template <int L>
__device__ __forceinline__ float rope_sum(float v) {
  v = rope_add_row<0xB1>(v);        // neighbours
  v = rope_add_row<0x4E>(v);        // pairs
  v = rope_add_row<0x141>(v);       // fours (the mirror of 8 lanes)
  if constexpr (L >= 16) v = rope_add_row<0x140>(v);      // eights (the mirror of 16)
  if constexpr (L >= 32) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return v;
}

// 1 / sqrt(v).  The instruction takes a subnormal v (rows below 2^-63) for 0: TINY brings small ones up by an even power
// of two.  An eps of kRopeTiny or more leaves none, and in its kernels the question would cost 1 to 2%.
constexpr float kRopeTiny = 0x1p-100f;
template <bool TINY>
__device__ __forceinline__ float rope_rsq(float v) {
  const bool small = TINY && v < kRopeTiny;
  return __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v) * (small ? 0x1p32f : 1.0f);
}

__device__ __forceinline__ rope_f32x4 rope_f32(uint2 u) {
  return rope_f32x4{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
}
__device__ __forceinline__ uint2 rope_bf16(rope_f32x4 v) {
  return __builtin_bit_cast(uint2, __builtin_convertvector(v, rope_bf16x4));
}

// NORM: kRopeNormTiny with an eps below kRopeTiny.
constexpr int kRopeNorm = 1, kRopeNormTiny = 2;
template <int D, int NORM, bool PAIRS>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
  constexpr int L = D / 8, HEADS = kWave / L;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l = lane % L;
  const int w = blockIdx.x * kRopeWaves + wave;
  const int t = w / a.parts;
  if (t >= a.tokens) return;
  const bool turns = 8 * l < a.rot;
  // the lane's two pieces of four elements
  const int at0 = PAIRS || !turns ? 8 * l : 4 * l;
  const int at1 = PAIRS || !turns ? 8 * l + 4 : a.rot / 2 + 4 * l;
  const int first = (w - t * a.parts) * a.span * HEADS, last = min(first + a.span * HEADS, a.heads);
  const uint16_t* const q = a.q + t * a.qs;
  const uint16_t* const k = a.k + t * a.ks;
  auto load = [&](int h, uint2 (&x)[2]) {
    h = min(h, a.heads - 1);      // (lanes past the last head compute it again and do not store)
    const uint16_t* p = h < a.q_heads ? q + h * D : k + (h - a.q_heads) * D;
    x[0] = *reinterpret_cast<const uint2*>(p + at0);
    x[1] = *reinterpret_cast<const uint2*>(p + at1);
  };
  uint2 next[2];
  load(first + lane / L, next);
  rope_f32x4 factor[2][2];      // of queries and keys
  if constexpr (NORM != 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint16_t* p = i ? a.kw : a.qw;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint2 u = p ? *reinterpret_cast<const uint2*>(p + (j ? at1 : at0)) : make_uint2(0x3F803F80u, 0x3F803F80u);
        factor[i][j] = p ? rope_f32(u) + a.offset : rope_f32(u);
      }
    }
  }
  float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (turns) {
    const float4 f = *reinterpret_cast<const float4*>(a.inv_freq + 4 * l);
    const float freq[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int axis = 0;
      if (a.axes > 1) {
        const int i = 4 * l + e;
        axis = (i >= a.end[0]) + (a.axes > 2 && i >= a.end[1]) + (a.axes > 3 && i >= a.end[2]);
      }
      const double turn = (double)a.positions[(size_t)axis * a.tokens + t] * (double)freq[e] * 0.15915494309189533577;
      sincospif(2.0f * (float)(turn - __builtin_rint(turn)), &s[e], &c[e]);
    }
  }
  for (int h0 = first; h0 < last; h0 += HEADS) {
    const int h = h0 + lane / L;
    rope_f32x4 x[2] = {rope_f32(next[0]), rope_f32(next[1])};
    if (h0 + HEADS < last) load(h + HEADS, next);
    const bool is_q = h < a.q_heads;
    if constexpr (NORM != 0) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = __builtin_fmaf(x[j][e], x[j][e], sum);
      const float r = rope_rsq<NORM == kRopeNormTiny>(rope_sum<L>(sum) * (1.0f / D) + a.eps);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = x[j][e] * r * (is_q ? factor[0][j][e] : factor[1][j][e]);
    }
    rope_f32x4 y[2] = {x[0], x[1]};
    if (turns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (PAIRS) {
          const int j = e / 2, i = e % 2 * 2;
          y[j][i] = __builtin_fmaf(x[j][i], c[e], -(x[j][i + 1] * s[e]));
          y[j][i + 1] = __builtin_fmaf(x[j][i], s[e], x[j][i + 1] * c[e]);
        } else {
          y[0][e] = __builtin_fmaf(x[0][e], c[e], -(x[1][e] * s[e]));
          y[1][e] = __builtin_fmaf(x[0][e], s[e], x[1][e] * c[e]);
        }
      }
    }
    if (h < a.heads) {
      uint16_t* p = is_q ? a.qo + t * a.qos + h * D : a.ko + t * a.kos + (h - a.q_heads) * D;
      *reinterpret_cast<uint2*>(p + at0) = rope_bf16(y[0]);
      *reinterpret_cast<uint2*>(p + at1) = rope_bf16(y[1]);
    }
  }
}

template <int D>
void rope_launch(const RopeArgs& a, int flags, hipStream_t st) {
  const unsigned blocks = (unsigned)(((int64_t)a.tokens * a.parts + kRopeWaves - 1) / kRopeWaves);
  auto go = [&](auto norm, auto pairs) {
    hipLaunchKernelGGL((rope_kernel<D, decltype(norm)::value, decltype(pairs)::value>), dim3(blocks),
                       dim3(kRopeThreads), 0, st, a);
  };
  const bool pairs = flags & W4A16_ROPE_INTERLEAVED;
  auto with_pairs = [&](auto norm) { pairs ? go(norm, std::true_type{}) : go(norm, std::false_type{}); };
  using std::integral_constant;
  if (!(flags & W4A16_ROPE_NORM))
    with_pairs(integral_constant<int, 0>{});
  else if (a.eps >= kRopeTiny)
    with_pairs(integral_constant<int, kRopeNorm>{});
  else
    with_pairs(integral_constant<int, kRopeNormTiny>{});
}

bool rope_stride(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0 && stride <= (1LL << 40); }

}  // namespace

}  // namespace w4k

using namespace w4k;

extern "C" {

w4a16_status_t w4a16_qk_norm_rope(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                  const uint16_t* q_weight, const uint16_t* k_weight, float weight_offset,
                                  const float* inv_freq, const int32_t* positions, const int* sections, int axes,
                                  uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out, int64_t k_out_stride,
                                  float eps, int flags, int tokens, int q_heads, int k_heads, int dim, int rot,
                                  void* stream) {
  if ((dim != 64 && dim != 128 && dim != 256) || flags & ~(W4A16_ROPE_NORM | W4A16_ROPE_INTERLEAVED))
    return W4A16_ERR_UNSUPPORTED;
  if (tokens < 0 || tokens > W4A16_KV_MAX_TOKENS || q_heads < 0 || q_heads > (1 << 16) || k_heads < 0 ||
      k_heads > (1 << 16) || rot < 0 || rot > dim || rot % 8)
    return W4A16_ERR_SHAPE;
  if (axes < 1 || axes > W4A16_ROPE_MAX_AXES) return W4A16_ERR_UNSUPPORTED;
  RopeArgs a{};
  if (axes > 1) {
    if (!sections) return W4A16_ERR_NULL;
    int64_t pairs = 0;
    for (int i = 0; i < axes; ++i) {
      if (sections[i] < 0) return W4A16_ERR_SHAPE;
      pairs += sections[i];
      if (pairs > rot / 2) return W4A16_ERR_SHAPE;
      if (i < W4A16_ROPE_MAX_AXES - 1) a.end[i] = (int)pairs;
    }
    if (pairs != rot / 2) return W4A16_ERR_SHAPE;
  }
  const bool has_q = q_heads > 0, has_k = k_heads > 0;
  if ((has_q && (!rope_stride(q_stride, (int64_t)q_heads * dim) || !rope_stride(q_out_stride, (int64_t)q_heads * dim))) ||
      (has_k && (!rope_stride(k_stride, (int64_t)k_heads * dim) || !rope_stride(k_out_stride, (int64_t)k_heads * dim))))
    return W4A16_ERR_SHAPE;
  if (tokens == 0 || (!has_q && !has_k)) return W4A16_OK;
  if ((has_q && (!q || !q_out)) || (has_k && (!k || !k_out)) || (rot > 0 && (!inv_freq || !positions)))
    return W4A16_ERR_NULL;
  for (const void* p : {(const void*)q, (const void*)k, (const void*)q_out, (const void*)k_out, (const void*)q_weight,
                        (const void*)k_weight, (const void*)inv_freq})
    if (!kv_aligned(p, 16)) return W4A16_ERR_ALIGN;
  if (!kv_aligned(positions, 4)) return W4A16_ERR_ALIGN;
  a.q = q, a.k = k, a.qw = q_weight, a.kw = k_weight;
  a.qo = q_out, a.ko = k_out;
  a.qs = q_stride, a.ks = k_stride, a.qos = q_out_stride, a.kos = k_out_stride;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.heads = q_heads + k_heads;
  a.rot = rot;
  a.axes = axes;
  a.eps = eps;
  a.offset = weight_offset;
  // Wave-fuls of heads a wave: one while waves are few, so that a small step is spread over
  // the card; more where they share their token's sines.  Measured (us in a graph, for at least 2048 /
  // 8192 / 16384 waves): 4099 tokens of 20 heads of 128 with three axes 10.6 / 13.6 / 16.7, 1500 of
  // 40 8.8 / 11.9 / 11.8, 11801 of 40 48.0 / 47.5 / 46.7.
  // Shares are made even (1500 of 40: 8.2 instead of 8.8).
  const int fulls = (a.heads + kWave * 8 / dim - 1) / (kWave * 8 / dim);
  const int64_t waves = (int64_t)tokens * fulls;
  a.span = waves <= kRopeFill ? 1 : (int)(waves / kRopeFill) < fulls ? (int)(waves / kRopeFill) : fulls;
  a.parts = (fulls + a.span - 1) / a.span;
  a.span = (fulls + a.parts - 1) / a.parts;
  hipStream_t st = (hipStream_t)stream;
  switch (dim) {
    case 64: rope_launch<64>(a, flags, st); break;
    case 128: rope_launch<128>(a, flags, st); break;
    default: rope_launch<256>(a, flags, st); break;
  }
  return kv_launched(hipGetLastError());
}

}  // extern "C"
