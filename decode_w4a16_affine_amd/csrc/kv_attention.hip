// Attention over the paged 8-bit cache (include/w4a16_kv.h).  Compiled once per
// head size (W4K_D = 64, 128, 256).
#include "kv_attn_split.hpp"
#include "kv_attn_tile.hpp"
#include "kv_device.hpp"

namespace w4k {

namespace {

template <int TYPE>
hipError_t kv_attention_typed(const KvAttnArgs& a, void* workspace, hipStream_t st) {
  constexpr int D = W4K_D;
  float* part_o = static_cast<float*>(workspace);
  float* part_ml = part_o + kv_partials(a) * D;
  float* tile_o = part_o + kv_split_floats(a, D);
  float* tile_ml = tile_o + kv_tile_partials(a) * D;
  const int rows = a.split_tokens * a.group;
  const unsigned ry = a.requests < kKvGridRequests ? a.requests : kKvGridRequests;
  const unsigned rz = (a.requests + kKvGridRequests - 1) / kKvGridRequests;
  auto split = [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    hipLaunchKernelGGL((kv_split_kernel<D, TYPE, NC>), dim3(a.c.heads * a.row_groups * a.chunks, ry, rz),
                       dim3(kKvSplitWaves * kWave), 0, st, a, part_o, part_ml);
    if (a.chunks > 1)
      hipLaunchKernelGGL((kv_join_kernel<D, NC>), dim3(a.c.heads * rows, ry, rz), dim3(kKvJoinThreads), 0, st, a,
                         part_o, part_ml);
  };
  if (a.split) {
    if (rows <= 16)
      split(std::integral_constant<int, 1>{});
    else
      split(std::integral_constant<int, 2>{});
  }
  if ((int64_t)a.max_new * a.group > kKvSplitRows) {
    const int64_t tiles = a.tokens / (kv_tile_rows(D, TYPE) / a.group) + a.requests;
    hipLaunchKernelGGL((kv_tile_kernel<D, TYPE>), dim3((unsigned)(tiles * a.c.heads), a.parts),
                       dim3(kv_tile_waves(D, TYPE) * kWave), 0, st, a, tile_o, tile_ml);
    if (a.parts > 1) {
      constexpr int rows_a_block = kKvJoinThreads / (D / 4);
      hipLaunchKernelGGL((kv_tile_join_kernel<D, TYPE>),
                         dim3((unsigned)(((int64_t)a.tokens * a.q_heads + rows_a_block - 1) / rows_a_block)),
                         dim3(kKvJoinThreads), 0, st, a, tile_o, tile_ml);
    }
  }
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
