// Attention kernels of the paged 4-bit cache for heads of 64.
#include "cache_attn.h"

namespace hr {
int cache_attn_64(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    if (k.ng == 1) return pick_scales<64, 1>(k, a, workers, stream);
    if (k.ng == 2) return pick_scales<64, 2>(k, a, workers, stream);
    return static_cast<int>(hipErrorInvalidValue);
}
}  // namespace hr
