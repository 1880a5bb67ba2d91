// Argument structs shared by the eviction's host layer (evict_api.cpp) and its
// kernels (evict_weights.hip, evict_pages.hip).  Plain data only.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "cache.h"

namespace hr {

struct CacheEvictArgs {
    uint8_t* pool;
    const int32_t* table;
    const int32_t* lens;
    float* weights;
    int32_t* new_table;
    int32_t* new_lens;
    int32_t* refs;
    int32_t* status;
    int32_t* work;
    CachePage pg;
    int64_t layers, n_pages, width;
    int32_t rows, max_pages;
    int32_t budget, sinks, recent;
};

struct CacheWeightsArgs {
    const void* q;
    const uint8_t* pool;
    const float* lse;
    float* weights;
    uint8_t* work;
    int64_t q_st, q_sh;        // element strides
    int64_t width;
    CachePage pg;
    CacheSeqs sq;
    float scale;               // of the scores
    float norm;                // 1 / sqrt(d) (rotate)
    float decay;
    int32_t hq, rep;           // query heads; query heads per kv head
    int32_t causal, window, rotate;
    int32_t workers;           // workgroups
    int32_t few;               // row tiles of the kernel of few rows, or 0: that of many
};

// Launchers: 0 or a hipError_t.
int launch_cache_weights(const CacheWeightsArgs& a, int bf16, void* stream);
// workgroups that hr_cache_weights keeps in flight on the current device
int cache_weights_workers(int few, int* workers);
int launch_cache_evict(const CacheEvictArgs& a, void* stream);

// bytes of scratch: the numbering of the sequences' work; a row's factor and
// log-sum-exp, and its query as pairs of float16; and in the kernel of many rows two
// partial sums of a block of up to 256 keys for each workgroup, of which there are at
// most kWeightsParts
constexpr int kWeightsParts = 512;
constexpr int64_t cache_weights_first(int64_t seqs) { return ((seqs + 1) * 8 + 15) / 16 * 16; }
constexpr int64_t cache_weights_bytes(int64_t seqs, int64_t tokens, int32_t q_heads, int d, int few) {
    return cache_weights_first(seqs) + (tokens * q_heads * 8 + 15) / 16 * 16 + tokens * q_heads * d * 4 +
           (few == 0 ? int64_t{kWeightsParts} * 2 * 256 * 4 : 0);
}
// int32 words of scratch
constexpr int64_t cache_evict_words(int64_t n_pages, int64_t rows) { return 3 * n_pages + rows + 16; }

}  // namespace hr
