/*
 * include/w4a16_kv.h from C99: every entry point is linked and called with
 * arguments that it refuses (or has no work for) before anything reaches a GPU,
 * and the workspace size of a small decode step is what the header says.
 * Exit status 0 and a line "ok" on success.
 */
#include <stdio.h>

#include "w4a16_kv.h"

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
  static uint16_t bf16[256];
  static int32_t i32[16];
  static float f32[256];
  w4a16_kv_cache_t c = {0, 0, 0, 0, W4A16_KV_FP8, 8, 2, 64, 128};
  EXPECT(w4a16_kv_plan(i32, i32, i32, 1, i32, 2, i32, i32, i32, i32, 1, 1, 48, 0), W4A16_ERR_UNSUPPORTED);
  EXPECT(w4a16_kv_plan(i32, i32, i32, 1, i32, W4A16_KV_MAX_WIDTH + 1, i32, i32, i32, i32, 1, 1, 64, 0),
         W4A16_ERR_SHAPE);
  EXPECT(w4a16_kv_plan(0, i32, i32, 1, i32, 2, i32, i32, i32, i32, 1, 1, 64, 0), W4A16_ERR_NULL);
  EXPECT(w4a16_kv_append(bf16, 256, bf16, 256, i32, &c, 1, 0), W4A16_ERR_NULL);
  EXPECT(w4a16_kv_append(bf16, 256, bf16, 256, i32, &c, 0, 0), W4A16_OK);
  EXPECT(w4a16_kv_append(bf16, 255, bf16, 256, i32, &c, 1, 0), W4A16_ERR_SHAPE);
  EXPECT(w4a16_kv_attention(bf16, 512, &c, i32, 4, i32, i32, bf16, 0.1f, 0, 1, 1, 1, 64, 4, 0, 0, 0), W4A16_ERR_NULL);
  EXPECT(w4a16_kv_attention(bf16, 512, &c, i32, 4, i32, i32, bf16, 0.1f, 0, 0, 1, 1, 64, 4, 0, 0, 0), W4A16_OK);
  c.dim = 96;
  EXPECT(w4a16_kv_dequant(&c, i32, 1, f32, f32, 0), W4A16_ERR_UNSUPPORTED);
  c.dim = 128;
  EXPECT(w4a16_kv_dequant(&c, i32, W4A16_KV_MAX_DEQUANT, f32, f32, 0), W4A16_ERR_NULL);
  EXPECT(w4a16_kv_dequant(&c, i32, 0, f32, f32, 0), W4A16_OK);
  /* 3 tokens of 4 query heads in 4 chunks of 128 entries: 133 floats a row and chunk */
  if (w4a16_kv_attention_workspace_bytes(3, 3, 1, 512, 0, 4, &c) != 3u * 4u * 4u * 133u * 4u) {
    fprintf(stderr, "workspace: %lu bytes\n",
            (unsigned long)w4a16_kv_attention_workspace_bytes(3, 3, 1, 512, 0, 4, &c));
    return 1;
  }
  puts("ok");
  return 0;
}
