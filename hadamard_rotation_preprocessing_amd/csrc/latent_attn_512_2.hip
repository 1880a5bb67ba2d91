// Latent attention kernels for latents of 512 in 2 groups.
#include "latent_attn.h"

namespace hr {
int latent_attn_512_2(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream) {
    return pick_scales<512, 2>(k, a, workers, stream);
}
}  // namespace hr
