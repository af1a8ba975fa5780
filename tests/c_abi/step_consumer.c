/*
 * include/w4a16_step.h from C99: every entry point is linked and called with
 * arguments that it refuses (or has no work for) before anything reaches a GPU,
 * and a workspace size is what the header says.  Exit status 0 and a line "ok"
 * on success.
 */
#include <stdio.h>

#include "w4a16_step.h"

#define EXPECT(call, status)                                                          \
  do {                                                                                \
    int got_ = (int)(call);                                                           \
    if (got_ != (int)(status)) {                                                      \
      fprintf(stderr, "%s:%d: status %d (%s)\n", __FILE__, __LINE__, got_,            \
              w4a16_status_str((w4a16_status_t)got_));                                \
      return 1;                                                                       \
    }                                                                                 \
  } while (0)

int main(void) {
  static uint16_t bf16[512];
  static int32_t i32[16];
  static float f32[256];
  const int sections[3] = {16, 8, 8};
  w4a16_kv_cache_t c = {0, 0, 0, 0, W4A16_KV_FP8, 8, 2, 64, 128};
  EXPECT(w4a16_qk_norm_rope(bf16, 64, bf16, 64, 0, 0, 0.0f, f32, i32, sections, 3, bf16, 64, bf16, 64, 1e-6f,
                            W4A16_ROPE_NORM | W4A16_ROPE_INTERLEAVED, 0, 1, 1, 64, 64, 0), W4A16_OK);
  EXPECT(w4a16_qk_norm_rope(0, 64, bf16, 64, 0, 0, 0.0f, f32, i32, 0, 1, bf16, 64, bf16, 64, 1e-6f, 0, 1, 1, 1, 64,
                            64, 0), W4A16_ERR_NULL);
  EXPECT(w4a16_qk_norm_rope(bf16, 64, bf16, 64, 0, 0, 0.0f, f32, i32, 0, W4A16_ROPE_MAX_AXES + 1, bf16, 64, bf16, 64,
                            1e-6f, 0, 1, 1, 1, 64, 64, 0), W4A16_ERR_UNSUPPORTED);
  EXPECT(w4a16_kv_attention_shared(bf16, 512, &c, i32, 4, i32, i32, i32, bf16, 0.1f, 1, 1, 1, 64, 64, 4, 0, 0, 0),
         W4A16_ERR_NULL);
  EXPECT(w4a16_kv_attention_shared(bf16, 512, &c, i32, 4, i32, i32, i32, bf16, 0.1f, 0, 1, 1, 64, 64, 4, 0, 0, 0),
         W4A16_OK);
  EXPECT(w4a16_kv_attention_shared(bf16, 512, &c, i32, 4, i32, i32, i32, bf16, 0.1f, 40, 1, 33, 64, 64, 4, 0, 0, 0),
         W4A16_ERR_UNSUPPORTED);
  EXPECT(w4a16_sample(f32, W4A16_OUT_F32, 8, f32, f32, i32, f32, f32, i32, f32, 0, 0, 1, 8, 0), W4A16_ERR_WORKSPACE);
  EXPECT(w4a16_sample(f32, W4A16_OUT_F32, 7, f32, f32, i32, f32, f32, i32, f32, 0, 0, 1, 8, 0), W4A16_ERR_SHAPE);
  EXPECT(w4a16_sample(0, W4A16_OUT_BF16, 8, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 8, 0), W4A16_OK);
  EXPECT(w4a16_sample_workspace_bytes(1, W4A16_SAMPLE_MAX_N + 1) != 0, 0);
  EXPECT(w4a16_sample_workspace_bytes(W4A16_SAMPLE_MAX_ROWS, 1) != 0, 1);
  /* 6 rows; one chunk of 128 for 64 shared entries, two for 64 own: 133 floats each */
  if (w4a16_kv_attention_shared_workspace_bytes(3, 3, 1, 64, 64, 2, &c) != 3u * 2u * 3u * 133u * 4u) {
    fprintf(stderr, "workspace: %lu bytes\n",
            (unsigned long)w4a16_kv_attention_shared_workspace_bytes(3, 3, 1, 64, 64, 2, &c));
    return 1;
  }
  puts("ok");
  return 0;
}
