// The cache's kernel launchers, replaced: which attention kernel a call takes is
// noted instead.  As cache_stubs.cpp otherwise.
#include <hip/hip_runtime_api.h>

#include "../../hadamard_rotation_preprocessing_amd/csrc/cache.h"

static hr::CacheAttnKey last;

// 1: a workgroup's waves take different keys of the same rows; 8: different rows
extern "C" int chosen_waves() { return last.wr; }

namespace hr {
int launch_cache_append(const CacheAppendArgs&, int, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_cache_update(const CacheUpdateArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_cache_compact(const CacheCompactArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_cache_attn(const CacheAttnKey& k, const CacheAttnArgs&, void*) {
    last = k;
    return static_cast<int>(hipErrorNoDevice);
}
int cache_attn_workers(const CacheAttnKey&, int* workers) {
    *workers = 4;
    return 0;
}
}  // namespace hr
