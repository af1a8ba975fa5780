// Host-only stand-ins for the attention launchers of the key/value cache, so
// that its C-ABI translation unit (csrc/kv.hip) can be built under the address
// and undefined-behaviour sanitizers and its argument checks and launch sizes
// exercised without a GPU.  Every stand-in reports a refused launch.
#include <hip/hip_runtime.h>

#include "kv_device.hpp"

namespace w4k {

#define W4K_STUB_KV(D) \
  hipError_t kv_attention_d##D(int, const KvAttnArgs&, void*, hipStream_t) { return hipErrorInvalidValue; }
W4K_STUB_KV(64)
W4K_STUB_KV(128)
W4K_STUB_KV(256)

}  // namespace w4k
