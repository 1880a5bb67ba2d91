// Stand-ins for the launchers of the eviction and of the latent cache in the
// CPU-only sanitizer build of the validation layer: no device is present, and the
// kernels ask for scratch as if four workgroups were in flight.
#include <hip/hip_runtime_api.h>

#include "../../hadamard_rotation_preprocessing_amd/csrc/evict.h"
#include "../../hadamard_rotation_preprocessing_amd/csrc/latent.h"

namespace hr {
int launch_cache_weights(const CacheWeightsArgs&, int, void*) { return static_cast<int>(hipErrorNoDevice); }
int cache_weights_workers(int, int* workers) {
    *workers = 4;
    return 0;
}
int launch_cache_evict(const CacheEvictArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_latent_append(const LatentPagesArgs&, int, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_latent_read(const LatentPagesArgs&, int, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_latent_attn(const LatentAttnKey&, const LatentAttnArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int launch_latent_prompt(const LatentPromptArgs&, void*) { return static_cast<int>(hipErrorNoDevice); }
int latent_attn_workers(const LatentAttnKey&, int* workers) {
    *workers = 4;
    return 0;
}
}  // namespace hr
