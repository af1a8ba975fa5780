// Attention behind entries that a batch's requests share (w4a16_kv_attention_shared of
// include/w4a16_step.h).  Compiled once per head size (W4K_D = 64, 128, 256).
//
// softmax over (shared, own) entries is joined from both sides' (maximum, sum, output): the
// shared entries are attended by all requests' rows at once, in the form that their number
// makes the better one (kv_shared.hip), a request's own by its rows alone, in the split
// form; kv_shared_join_kernel adds the parts of each row.
//
// Bound and measured (in a graph).  64 single tokens, 32 heads of 128 over 8, E4M3, behind 8000
// shared and up to 2000 own entries, 148 MB: 52 us, of which the join takes 5.7 (14 MB of
// partial results written and read again).  The tiles' registers leave the own entries' workgroups two a
// CU where three stream better: in launches of their own the tiles took 26 and the others 32.
// (w4a16_kv_attention reads 1.2 GB for that.)  24 behind 100001, int8, 229 MB: 80 us; 96 of a
// tile's 128 rows, a quarter of the units idle.  8 behind 1501, 10 heads of 256 over 2: 12.4 us.
#include "kv_attn_split.hpp"
#include "kv_attn_tile.hpp"
#include "kv_device.hpp"

namespace w4k {

namespace {

// Shared entries and the requests' own in one launch: the workgroups of the shared ones, which take
// longer, begin first, and the others fill up the card.
struct KvTurn {
  int over, of;      // workgroup `of` of the shared entries' (over) or of the own ones
};
__device__ __forceinline__ KvTurn kv_turn(int block, int over) {
  return block < over ? KvTurn{1, block} : KvTurn{0, block - over};
}

// `over` workgroups of shared entries (x tiles' or chunks', heads fastest), `own` of the rest (own_x a request).
template <int D, int TYPE, int NC>
__global__ __launch_bounds__(kv_tile_waves(D, TYPE) * kWave, 2) void kv_shared_tile_kernel(KvSharedArgs a, int over, int over_x,
                                                                                         int own, int own_x,
                                                                                         float* part_o,
                                                                                         float* part_ml) {
  __shared__ union {
    KvTileShared<D, TYPE> tile;
    KvSplitShared<D, NC> split;
  } shared;
  const KvTurn turn = kv_turn(blockIdx.x, over);
  if (turn.over) {
    kv_tile_body<D, TYPE>(a, shared.tile, turn.of % over_x, over_x, turn.of / over_x, part_o, part_ml);
  } else {
    if (threadIdx.x >= kKvSplitWaves * kWave) return;      // (whole waves)
    kv_split_body<D, TYPE, NC>(a, shared.split, turn.of % own_x, turn.of / own_x, part_o, part_ml);
  }
}

template <int D, int TYPE, int NCP, int NC>
__global__ __launch_bounds__(kKvSplitWaves * kWave, kv_split_occupancy(D, NCP)) void kv_shared_split_kernel(
    KvPrefixArgs p, int over, int own, int own_x, int row_groups, float* part_o, float* part_ml) {
  __shared__ union {
    KvSplitShared<D, NCP> over;
    KvSplitShared<D, NC> own;
  } shared;
  const KvTurn turn = kv_turn(blockIdx.x, over);
  if (turn.over) {
    kv_split_body<D, TYPE, NCP>(p, shared.over, turn.of, 0, part_o, part_ml);
  } else {
    KvSharedArgs a = p;
    a.row_groups = row_groups;
    kv_split_body<D, TYPE, NC>(a, shared.own, turn.of % own_x, turn.of / own_x, part_o, part_ml);
  }
}

template <int TYPE>
hipError_t kv_shared_typed(const KvSharedArgs& a, void* workspace, hipStream_t st) {
  constexpr int D = W4K_D;
  float* part_o = static_cast<float*>(workspace);
  float* part_ml = part_o + kv_shared_partials(a) * D;
  const int rows = a.split_tokens * a.group, all_rows = a.tokens * a.group;
  const int own_x = a.c.heads * a.row_groups * a.chunks, own = own_x * a.requests;
  if (a.part_shift > 0) {
    KvPrefixArgs p{a};
    p.row_groups = all_rows <= 16 ? 1 : (all_rows + 31) / 32;
    const int over = a.c.heads * p.row_groups * a.parts;
    auto go = [&](auto ncp, auto nc) {
      hipLaunchKernelGGL((kv_shared_split_kernel<D, TYPE, decltype(ncp)::value, decltype(nc)::value>), dim3(over + own),
                         dim3(kKvSplitWaves * kWave), 0, st, p, over, own, own_x, a.row_groups, part_o, part_ml);
    };
    using std::integral_constant;
    if (rows > 16)
      go(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    else if (all_rows > 16)
      go(integral_constant<int, 2>{}, integral_constant<int, 1>{});
    else
      go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  } else if (a.parts + a.chunks > 0) {
    const int tt = kv_tile_rows(D, TYPE) / a.group;
    const int over_x = (a.tokens + tt - 1) / tt * a.c.heads, over = over_x * a.parts;
    const dim3 grid(over + own), block(kv_tile_waves(D, TYPE) * kWave);
    if (rows <= 16)
      hipLaunchKernelGGL((kv_shared_tile_kernel<D, TYPE, 1>), grid, block, 0, st, a, over, over_x, own, own_x, part_o, part_ml);
    else
      hipLaunchKernelGGL((kv_shared_tile_kernel<D, TYPE, 2>), grid, block, 0, st, a, over, over_x, own, own_x, part_o, part_ml);
  }
  const unsigned ry = a.requests < kKvGridRequests ? a.requests : kKvGridRequests;
  const unsigned rz = (a.requests + kKvGridRequests - 1) / kKvGridRequests;
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
