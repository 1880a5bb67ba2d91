// Argument structs shared by the cache's host layer (cache_api.cpp) and its
// kernels (cache_attn_*.hip, cache_pages.hip).  Plain data only.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace hr {

// A page's layout, resolved (offsets inside a head's part of a page).
struct CachePage {
    int32_t hkv, d, ng;        // kv heads, head dimension, groups per vector
    int32_t page, logp;        // positions of a page
    int32_t sym, sf32;         // symmetric codes; float32 scales (else bfloat16)
    int32_t kc, vc, ks, vs, kz, vz;
    int64_t head_bytes, page_bytes;
};

// The sequences of a call.  n(b) = cu[b + 1] - cu[b], or tokens / rows.
struct CacheSeqs {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;         // nullable
    int32_t rows, max_pages;
    int32_t tokens;
    int32_t per;               // tokens / rows (cu == NULL)
    int64_t n_pages;
};

struct CacheAppendArgs {
    uint8_t* pool;
    const void* k;
    const void* v;
    int64_t k_st, k_sh, v_st, v_sh;   // element strides
    CachePage pg;
    CacheSeqs sq;
    float norm;                // 1 / sqrt(d)
    int32_t rotate;
    int32_t units;             // blocks of positions (an upper bound)
};

struct CacheAttnArgs {
    const void* q;
    void* out;
    float* lse;                // nullable
    const uint8_t* pool;
    float* work;               // partial results
    int64_t q_st, q_sh, o_st, o_sh;   // element strides
    CachePage pg;
    CacheSeqs sq;
    float scale;               // of the scores
    float norm;                // 1 / sqrt(d) (rotate)
    int32_t hq, rep;           // query heads; query heads per kv head
    int32_t causal, window, rotate;
    int32_t workers;           // workgroups
    int32_t step, over;        // a unit's rows = step rep + over (set with the kernel)
};

// Which attention kernel a call takes.
struct CacheAttnKey {
    int32_t d, ng, sf32;       // of the cache
    int32_t wide;              // float32 activations
    int32_t rt, wr;            // row tiles of a wave, waves along the rows
};

struct CacheUpdateArgs {
    uint8_t* pool;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* parents;
    const int32_t* grow;
    int32_t* new_table;
    int32_t* new_lens;
    int32_t* refs;
    int32_t* status;
    int32_t* work;
    int64_t layers, n_pages, page_bytes;
    int32_t rows, max_pages, new_rows, page;
};

struct CacheCompactArgs {
    uint8_t* pool;
    uint8_t* into;             // nullable: within the pool
    const int32_t* table;
    const int32_t* lens;
    int32_t* new_table;
    int32_t* refs;
    int32_t* status;
    int32_t* work;
    int64_t layers, n_pages, into_pages, page_bytes;
    int32_t rows, max_pages, page;
};

// Launchers: 0 or a hipError_t.
int launch_cache_append(const CacheAppendArgs& a, int bf16, void* stream);
int launch_cache_update(const CacheUpdateArgs& a, void* stream);
int launch_cache_compact(const CacheCompactArgs& a, void* stream);
int launch_cache_attn(const CacheAttnKey& k, const CacheAttnArgs& a, void* stream);
// workgroups that an attention kernel keeps in flight on the current device
int cache_attn_workers(const CacheAttnKey& k, int* workers);

// int32 words of scratch
constexpr int64_t cache_update_words(int64_t n_pages, int64_t new_rows) { return 4 * n_pages + 4 * new_rows + 16; }
constexpr int64_t cache_compact_words(int64_t n_pages) { return 5 * n_pages + 16; }

// hr_cache_update and hr_cache_compact of pages of any kind (cache_api.cpp).
int cache_update(void* pool, int64_t layers, int64_t n_pages, const CachePage& pg, const int32_t* table, const int32_t* lens,
                 int64_t rows, int64_t max_pages, const int32_t* parents, const int32_t* grow, int64_t new_rows, int32_t* new_table,
                 int32_t* new_lens, int32_t* refs, int32_t* status, void* work, int64_t work_bytes, void* stream);
int cache_compact(void* pool, int64_t layers, int64_t n_pages, const CachePage& pg, const int32_t* table, const int32_t* lens,
                  int64_t rows, int64_t max_pages, void* into, int64_t into_pages, int32_t* new_table, int32_t* refs,
                  int32_t* status, void* work, int64_t work_bytes, void* stream);

// Message and status of a failing call on this thread (api.cpp).
int set_error(int status, const char* text);

}  // namespace hr
