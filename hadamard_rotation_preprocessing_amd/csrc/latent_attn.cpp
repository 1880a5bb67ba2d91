// Dispatch of the latent attention kernels by dimension and groups.
#include <hip/hip_runtime_api.h>

#include "latent.h"

namespace hr {

int latent_attn_256_1(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream);
int latent_attn_256_2(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream);
int latent_attn_512_1(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream);
int latent_attn_512_2(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream);
int latent_attn_512_4(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream);

namespace {
int by_shape(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream) {
    if (k.d == 256 && k.ng == 1) return latent_attn_256_1(k, a, workers, stream);
    if (k.d == 256 && k.ng == 2) return latent_attn_256_2(k, a, workers, stream);
    if (k.d == 512 && k.ng == 1) return latent_attn_512_1(k, a, workers, stream);
    if (k.d == 512 && k.ng == 2) return latent_attn_512_2(k, a, workers, stream);
    if (k.d == 512 && k.ng == 4) return latent_attn_512_4(k, a, workers, stream);
    return static_cast<int>(hipErrorInvalidValue);
}
}  // namespace

int launch_latent_attn(const LatentAttnKey& k, const LatentAttnArgs& a, void* stream) { return by_shape(k, &a, nullptr, stream); }
int latent_attn_workers(const LatentAttnKey& k, int* workers) { return by_shape(k, nullptr, workers, nullptr); }

}  // namespace hr
