// C ABI of the attention behind shared entries (w4a16_kv_attention_shared of
// include/w4a16_step.h): argument checks and launch parameters.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv_host.hpp"
#include "w4a16_step.h"

namespace w4k {

namespace {

constexpr int kMaxEntries = 1 << 28;
constexpr int kSplitSteps = 768;     // of 128 entries and 32 rows
constexpr int kOwnFill = 2048;       // workgroups of the requests' own entries
constexpr int kSplitFill = 512;      // workgroups of the split form
constexpr int kPartTiles = 4;        // tiles of a part at least
constexpr int kPartFill = 48;        // workgroups of fewer tiles, if there are fewer
constexpr int kOwnOfTile = 256;      // own entries that take as long as a tile of shared ones

w4a16_status_t check_shared(const w4a16_kv_cache_t* cache, int tokens, int requests, int max_new, int max_shared,
                            int max_own, int q_heads) {
  const w4a16_status_t st = check_cache(cache);
  if (st != W4A16_OK) return st;
  if (tokens < 0 || requests < 0 || max_new < 0 || max_shared < 0 || max_own < 0 || q_heads < 1) return W4A16_ERR_SHAPE;
  if (tokens > W4A16_KV_MAX_TOKENS || requests > W4A16_KV_MAX_REQUESTS || max_shared > kMaxEntries ||
      max_own > kMaxEntries)
    return W4A16_ERR_SHAPE;
  if (q_heads % cache->heads || (int64_t)tokens * q_heads > 0x7FFFFFFFLL) return W4A16_ERR_SHAPE;
  const int group = q_heads / cache->heads;
  if (group > W4A16_KV_MAX_GROUP || (int64_t)max_new * group > kKvSplitRows) return W4A16_ERR_UNSUPPORTED;
  // the tiles' grid (at least 64 rows each) within the launch limit of 2^32 threads
  const int64_t tiles = tokens / (64 / group) + requests;
  if (tiles * cache->heads > (1 << 22)) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// The launch parameters of a call from its (checked) sizes, all of them above 0.
KvSharedArgs shared_args(const w4a16_kv_cache_t* cache, int tokens, int requests, int max_new, int max_shared,
                         int max_own, int q_heads) {
  KvSharedArgs a{};
  a.c = device_cache(cache);
  a.tokens = tokens;
  a.requests = requests;
  a.max_new = max_new;
  a.max_len = 2 * kMaxEntries;
  a.max_shared = max_shared;
  a.max_own = max_own;
  a.q_heads = q_heads;
  a.group = q_heads / cache->heads;
  a.group_inverse = (65536u + a.group - 1) / a.group;
  a.split_tokens = max_new;
  a.split = true;
  a.by_token = true;
  const int rows = a.split_tokens * a.group;
  a.row_groups = rows <= 16 ? 1 : (rows + 31) / 32;
  // Chunks of a request's own entries, which may begin inside one: of one step while the workgroups
  // are few.  Measured behind 8000, 32 heads of 128 over 8 (us in a graph, at most 512 / 1024 / 2048 / 4096): 64
  // requests with up to 2000 of their own 56.2 / 56.2 / 55.4 / 59.9, 24 33.0 / 32.0 / 32.4 / 36.3, 16 with up to
  // 8000 58.1 / 49.5 / 48.3 / 50.0.
  const int64_t own_groups = (int64_t)requests * cache->heads * a.row_groups;
  a.chunk_shift = 7;
  auto in_chunks = [&](int64_t n) { return (n + (1LL << a.chunk_shift) - 1) >> a.chunk_shift; };
  while (in_chunks(max_own) > kKvMaxChunks - 1 || own_groups * (max_own >> a.chunk_shift) > kOwnFill) ++a.chunk_shift;
  a.chunks = max_own > 0 ? (int)in_chunks(max_own) + 1 : 0;
  // The form over the shared entries.  The split form's workgroup has 32 rows and a step of 128
  // entries, short ones side by side; the tile form converts an entry once for 128 rows.  The
  // split form takes 64 rows, or more (up to 128) while its steps are few.  Measured (us in a graph, split / tile):
  // 70 rows of 256 over 2 heads behind 1000 entries 13.3 / 16.6, 4000 16.0 / 21.8, 12000 24.3 / 26.6,
  // 50000 50.7 / 44.3; 120 of 64 over 4 behind 1000 10.6 / 12.7, 8000 14.5 / 16.4; 96 of 128 over 8
  // behind 8000 22.3 / 24.7, 100001 149 / 73.
  a.part = kKvTile;
  const int rows_shared = tokens <= kWave ? tokens * a.group : kKvMaxSharedRows + 1;
  const int64_t groups = (int64_t)cache->heads * ((rows_shared + 31) / 32);
  if (max_shared > 0 && (rows_shared <= kKvSplitRows || (rows_shared <= kKvMaxSharedRows &&
                                                         groups * ((max_shared + 127) / 128) <= kSplitSteps))) {
    // Chunks of one step while their workgroups are fewer than the card holds (us, 256 / 512 / 1024 at most):
    // 16 rows behind 100001, 8 heads of 128, 54.7 / 43.7 / 52.7; 64 behind 8000 18.4 / 20.0 / 24.8.
    a.part_shift = 7;
    while ((max_shared - 1) >> a.part_shift >= kKvMaxParts || groups * (max_shared >> a.part_shift) > kSplitFill)
      ++a.part_shift;
    a.part = 1 << a.part_shift;
    a.parts = (max_shared + a.part - 1) >> a.part_shift;
  } else if (max_shared > 0) {
    // Parts for a workgroup a CU, so that the requests' own run beside them, and for one in two where these take as
    // long all the same: fewer partial results (32 heads of 128 over 8, 2 / 1 / 0.5 a CU in us: 64 single tokens
    // behind 8000 and up to 2000 of their own, 512 entries a tile, 65 / 61 / 55.5; 24 of them 35 / 35 / 32.4; 64 behind
    // 30000, 136 a tile, 90 / 79.5 / 107; behind 8000 with up to 20 of their own 40.5 / 36.7 / 41).  Two where tiles
    // are many (24 behind 100001 75 / 90 / 164), which eight waves of heads of 256 leave no room for.  Each
    // row and part costs D + 5 floats written and read again: four tiles at least (us, 2 / 3 / 4 / 6: 64
    // tokens of 16 requests behind 6000, 16 heads of 64 over 4, 18.8 / 18.0 / 18.2 / 19.8), fewer where that
    // makes less than 48 workgroups (64 tokens behind 500, 10 heads of 256 over 2, 18.4 instead of 27.3; behind 4000,
    // where they are more, parts of one tile gain nothing: 26.5 and 26.0).
    const int tile_tokens = kv_tile_rows(cache->dim, cache->type) / a.group;
    const int64_t workgroups = (int64_t)((tokens + tile_tokens - 1) / tile_tokens) * cache->heads;
    const int64_t tiles = workgroups * (max_shared / kKvTile);
    const int64_t own = (int64_t)requests * max_own * cache->heads;
    const int64_t fill = own >= kOwnOfTile * tiles                                              ? 128
                         : tiles > 256 * 32 && kv_tile_waves(cache->dim, cache->type) == 4 ? 512
                                                                                           : 256;
    const int64_t few = std::min<int64_t>(kPartFill / workgroups, (max_shared + kKvTile - 1) / kKvTile);
    const int64_t wanted =
        std::min<int64_t>({fill / workgroups, std::max<int64_t>(max_shared / (kPartTiles * kKvTile), few), kKvMaxParts});
    const int64_t parts = wanted > 1 ? wanted : 1;
    a.part = (int)((max_shared + parts * kKvTile - 1) / (parts * kKvTile)) * kKvTile;
    a.parts = (max_shared + a.part - 1) / a.part;
  }
  return a;
}

// The launch: workgroups over shared entries (of at least 64 rows) and of the requests' own.
bool shared_launch_fits(const KvSharedArgs& a) {
  const int64_t over = (int64_t)(a.tokens / (64 / a.group) + 1) * a.c.heads * a.parts;
  const int64_t own = (int64_t)a.c.heads * a.row_groups * a.chunks * a.requests;
  return over + own <= (1 << 22);      // (of up to 512 threads, 2^32 of which are a launch's limit)
}

size_t shared_workspace(const KvSharedArgs& a, int dim) {
  return kv_shared_partials(a) * (dim + kKvPartStats) * sizeof(float);
}

}  // namespace

}  // namespace w4k

using namespace w4k;

extern "C" {

size_t w4a16_kv_attention_shared_workspace_bytes(int tokens, int requests, int max_new, int max_shared, int max_own,
                                                 int q_heads, const w4a16_kv_cache_t* cache) {
  if (check_shared(cache, tokens, requests, max_new, max_shared, max_own, q_heads) != W4A16_OK) return 0;
  if (tokens == 0 || requests == 0 || max_new == 0) return 0;
  const KvSharedArgs a = shared_args(cache, tokens, requests, max_new, max_shared, max_own, q_heads);
  return shared_launch_fits(a) ? shared_workspace(a, cache->dim) : 0;
}

w4a16_status_t w4a16_kv_attention_shared(const uint16_t* q, int64_t q_stride, const w4a16_kv_cache_t* cache,
                                         const int32_t* block_table, int width, const int32_t* seq_lens,
                                         const int32_t* token_start, const int32_t* shared_len, uint16_t* out,
                                         float scale, int tokens, int requests, int max_new, int max_shared,
                                         int max_own, int q_heads, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  w4a16_status_t st = check_shared(cache, tokens, requests, max_new, max_shared, max_own, q_heads);
  if (st != W4A16_OK) return st;
  if (width < 0 || width > W4A16_KV_MAX_WIDTH || q_stride < (int64_t)q_heads * cache->dim || q_stride % 8 ||
      q_stride > (1LL << 40))
    return W4A16_ERR_SHAPE;
  if (tokens == 0 || requests == 0 || max_new == 0) return W4A16_OK;
  if (cache->pages == 0) return W4A16_ERR_SHAPE;      // masked entries are read from page 0
  st = check_cache_pointers(cache);
  if (st != W4A16_OK) return st;
  if (!q || !out || !seq_lens || !token_start || !shared_len || (width > 0 && !block_table)) return W4A16_ERR_NULL;
  if (!kv_aligned(q, 16) || !kv_aligned(out, 16) || !kv_aligned(block_table, 4) || !kv_aligned(seq_lens, 4) ||
      !kv_aligned(token_start, 4) || !kv_aligned(shared_len, 4))
    return W4A16_ERR_ALIGN;
  KvSharedArgs a = shared_args(cache, tokens, requests, max_new, max_shared, max_own, q_heads);
  if (!shared_launch_fits(a)) return W4A16_ERR_SHAPE;
  const size_t need = shared_workspace(a, cache->dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  if (!kv_aligned(workspace, 16)) return W4A16_ERR_ALIGN;
  a.q = q;
  a.q_stride = q_stride;
  a.table = block_table;
  a.width = width;
  a.seq_lens = seq_lens;
  a.token_start = token_start;
  a.shared_len = shared_len;
  a.out = out;
  a.scale_log2 = __builtin_fabsf(scale) * 1.44269504088896340736f;
  a.q_sign = scale < 0.0f ? 0x80008000u : 0u;
  hipStream_t s = (hipStream_t)stream;
  switch (cache->dim) {
    case 64: return kv_launched(kv_shared_d64(cache->type, a, workspace, s));
    case 128: return kv_launched(kv_shared_d128(cache->type, a, workspace, s));
    default: return kv_launched(kv_shared_d256(cache->type, a, workspace, s));
  }
}

}  // extern "C"
