// Dispatch of the cache's attention kernels by head dimension.
#include <hip/hip_runtime_api.h>

#include "cache.h"

namespace hr {

int cache_attn_64(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream);
int cache_attn_128(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream);
int cache_attn_256(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream);

namespace {
int by_dim(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    if (k.d == 64) return cache_attn_64(k, a, workers, stream);
    if (k.d == 128) return cache_attn_128(k, a, workers, stream);
    return cache_attn_256(k, a, workers, stream);
}
}  // namespace

int launch_cache_attn(const CacheAttnKey& k, const CacheAttnArgs& a, void* stream) { return by_dim(k, &a, nullptr, stream); }
int cache_attn_workers(const CacheAttnKey& k, int* workers) { return by_dim(k, nullptr, workers, nullptr); }

}  // namespace hr
