// Latent attention kernels for latents of 512 in 4 groups.
#include "latent_attn.h"

namespace hr {
int latent_attn_512_4(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream) {
    return pick_scales<512, 4>(k, a, workers, stream);
}
}  // namespace hr
