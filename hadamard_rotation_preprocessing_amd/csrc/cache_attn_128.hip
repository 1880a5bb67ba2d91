// Attention kernels of the paged 4-bit cache for heads of 128.
#include "cache_attn.h"

namespace hr {
int cache_attn_128(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    if (k.ng == 1) return pick_scales<128, 1>(k, a, workers, stream);
    if (k.ng == 2) return pick_scales<128, 2>(k, a, workers, stream);
    if (k.ng == 4) return pick_scales<128, 4>(k, a, workers, stream);
    return static_cast<int>(hipErrorInvalidValue);
}
}  // namespace hr
