// Attention behind entries that a batch's requests share (w4a16_kv_attention_shared of
// include/w4a16_step.h).  Compiled once per head size (W4K_D = 64, 128, 256).
#include "kv_attn_split.hpp"
#include "kv_attn_tile.hpp"
#include "kv_device.hpp"

namespace w4k {

namespace {

template <int D, int TYPE>
__global__ __launch_bounds__(kv_tile_waves(D, TYPE) * kWave, 2) void kv_shared_tile_kernel(KvSharedArgs a,
                                                                                         float* part_o,
                                                                                         float* part_ml) {
  kv_tile_body<D, TYPE>(a, part_o, part_ml);
}

template <int D, int TYPE, int NC>
__global__ __launch_bounds__(kKvSplitWaves * kWave, kv_split_occupancy(D, NC)) void kv_shared_split_kernel(
    KvSharedArgs a, float* part_o, float* part_ml) {
  kv_split_body<D, TYPE, NC>(a, part_o, part_ml);
}

template <int D, int TYPE, int NC>
__global__ __launch_bounds__(kKvSplitWaves * kWave, kv_split_occupancy(D, NC)) void kv_prefix_split_kernel(
    KvPrefixArgs a, float* part_o, float* part_ml) {
  kv_split_body<D, TYPE, NC>(a, part_o, part_ml);
}

template <int TYPE>
hipError_t kv_shared_typed(const KvSharedArgs& a, void* workspace, hipStream_t st) {
  constexpr int D = W4K_D;
  float* part_o = static_cast<float*>(workspace);
  float* part_ml = part_o + kv_shared_partials(a) * D;
  const int rows = a.split_tokens * a.group;
  const unsigned ry = a.requests < kKvGridRequests ? a.requests : kKvGridRequests;
  const unsigned rz = (a.requests + kKvGridRequests - 1) / kKvGridRequests;
  if (a.part_shift > 0 && a.parts > 0) {
    KvPrefixArgs p{a};
    const int all_rows = a.tokens * a.group;
    p.row_groups = all_rows <= 16 ? 1 : (all_rows + 31) / 32;
    const dim3 grid(a.c.heads * p.row_groups * a.parts), block(kKvSplitWaves * kWave);
    if (all_rows <= 16)
      hipLaunchKernelGGL((kv_prefix_split_kernel<D, TYPE, 1>), grid, block, 0, st, p, part_o, part_ml);
    else
      hipLaunchKernelGGL((kv_prefix_split_kernel<D, TYPE, 2>), grid, block, 0, st, p, part_o, part_ml);
  } else if (a.parts > 0) {
    const int tt = kv_tile_rows(D, TYPE) / a.group;
    hipLaunchKernelGGL((kv_shared_tile_kernel<D, TYPE>), dim3((unsigned)((a.tokens + tt - 1) / tt * a.c.heads), a.parts),
                       dim3(kv_tile_waves(D, TYPE) * kWave), 0, st, a, part_o, part_ml);
  }
  if (a.chunks > 0) {
    const dim3 grid(a.c.heads * a.row_groups * a.chunks, ry, rz);
    if (rows <= 16)
      hipLaunchKernelGGL((kv_shared_split_kernel<D, TYPE, 1>), grid, dim3(kKvSplitWaves * kWave), 0, st, a, part_o, part_ml);
    else
      hipLaunchKernelGGL((kv_shared_split_kernel<D, TYPE, 2>), grid, dim3(kKvSplitWaves * kWave), 0, st, a, part_o, part_ml);
  }
  hipLaunchKernelGGL((kv_shared_join_kernel<D>), dim3(a.c.heads * rows, ry, rz), dim3(kKvJoinThreads), 0, st, a, part_o,
                     part_ml);
  return hipGetLastError();
}

}  // namespace

#define W4K_CAT_(a, b) a##b
#define W4K_CAT(a, b) W4K_CAT_(a, b)

hipError_t W4K_CAT(kv_shared_d, W4K_D)(int type, const KvSharedArgs& a, void* workspace, hipStream_t st) {
  return type == W4A16_KV_INT8 ? kv_shared_typed<W4A16_KV_INT8>(a, workspace, st)
                               : kv_shared_typed<W4A16_KV_FP8>(a, workspace, st);
}

}  // namespace w4k
