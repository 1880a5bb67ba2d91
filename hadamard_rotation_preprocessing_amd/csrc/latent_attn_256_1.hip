// Latent attention kernels for latents of 256 in 1 group.
#include "latent_attn.h"

namespace hr {
int latent_attn_256_1(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream) {
    return pick_scales<256, 1>(k, a, workers, stream);
}
}  // namespace hr
