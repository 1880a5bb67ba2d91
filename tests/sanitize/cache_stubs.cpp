// Stand-ins for the cache's kernel launchers in the CPU-only sanitizer build
// of the validation layer: no device is present, and attention kernels ask for
// scratch as if four workgroups were in flight.
#include <hip/hip_runtime_api.h>

#include "../../hadamard_rotation_preprocessing_amd/csrc/cache.h"

namespace hr {
int launch_cache_append(const CacheAppendArgs&, int, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_cache_update(const CacheUpdateArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_cache_compact(const CacheCompactArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_cache_attn(const CacheAttnKey&, const CacheAttnArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int cache_attn_workers(const CacheAttnKey&, int* workers) {
    *workers = 4;
    return 0;
}
}  // namespace hr
