// Attention kernels of the paged 4-bit cache for heads of 256.
#include "cache_attn.h"

namespace hr {
int cache_attn_256(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    if (k.ng == 1) return pick_scales<256, 1>(k, a, workers, stream);
    if (k.ng == 2) return pick_scales<256, 2>(k, a, workers, stream);
    if (k.ng == 4) return pick_scales<256, 4>(k, a, workers, stream);
    if (k.ng == 8) return pick_scales<256, 8>(k, a, workers, stream);
    return static_cast<int>(hipErrorInvalidValue);
}
}  // namespace hr
