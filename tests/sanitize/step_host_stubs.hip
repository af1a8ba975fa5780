// Host-only stand-ins for the launchers of the attention behind shared entries, so that its C-ABI
// translation unit (csrc/kv_shared.hip) can be built under the address and undefined-behaviour
// sanitizers without a GPU.  Every stand-in reports a refused launch.
#include <hip/hip_runtime.h>

#include "kv_device.hpp"

namespace w4k {

#define W4K_STUB_SHARED(D) \
  hipError_t kv_shared_d##D(int, const KvSharedArgs&, void*, hipStream_t) { return hipErrorInvalidValue; }
W4K_STUB_SHARED(64)
W4K_STUB_SHARED(128)
W4K_STUB_SHARED(256)

}  // namespace w4k
