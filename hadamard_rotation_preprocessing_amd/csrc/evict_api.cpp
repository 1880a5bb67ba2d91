// C-ABI entry points of the eviction (include/hadarot_evict.h): argument
// validation.  Every check runs before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include <cmath>

#include "../../include/hadarot_evict.h"
#include "cache_check.h"
#include "evict.h"

namespace {

int check_width(int64_t width, int64_t max_pages, int page) {
    if (width < max_pages * page || width >= (int64_t{1} << 31))
        return fail(HR_EINVAL, "width = %lld must be at least max_pages * page_size = %lld and below 2^31", (long long)width,
                    (long long)(max_pages * page));
    return HR_OK;
}

// Row tiles of the kernel of few rows for a call, by the rows (new tokens x query heads
// of a kv head) that a sequence has by the caller's bound, or without one in the mean; 0
// for the kernel of many rows.  Queries in registers and keys streaming past take 34 us
// for 4 rows where the keys of a block in registers and rows through LDS take 90 us
// (24 sequences of up to 32768, 8 heads of 128); more rows than two tiles need several
// passes over the keys there, and one here.
int few_tiles(int64_t tokens, int rep, int64_t seqs, int64_t max_q) {
    const int64_t n = max_q > 0 ? (max_q < tokens ? max_q : tokens) : seqs > 0 ? (tokens + seqs - 1) / seqs : tokens;
    return n * rep <= 16 ? 1 : n * rep <= 32 ? 2 : 0;
}

}  // namespace

extern "C" {

int hr_cache_weights_work(int dtype, int64_t tokens, int32_t q_heads, const hr_cache_spec* spec, int64_t rows, int64_t max_q,
                          int64_t* bytes) {
    hr::CachePage pg;
    int st = check_spec(spec, &pg);
    if (st) return st;
    if (!bytes) return fail(HR_EINVAL, "bytes is NULL");
    if ((st = check_attention_sizes(dtype, tokens, q_heads, pg, max_q))) return st;
    if (rows < 0 || rows > kMaxCount) return fail(HR_EINVAL, "rows = %lld must be in 0..2^30", (long long)rows);
    *bytes = tokens == 0 ? 0 : hr::cache_weights_bytes(rows, tokens, q_heads, pg.d, few_tiles(tokens, q_heads / pg.hkv, rows, max_q));
    return ok();
}

int hr_cache_weights(const void* q, int64_t q_stride_token, int64_t q_stride_head, int dtype, int64_t tokens, int32_t q_heads,
                     const void* pool, int64_t n_pages, const hr_cache_spec* spec, const hr_cache_seqs* seqs, const float* lse,
                     float scale, int causal, int64_t window, int rotate, float decay, float* weights, int64_t width,
                     int64_t max_q, void* work, int64_t work_bytes, void* stream) {
    hr::CacheWeightsArgs a{};
    int st = check_spec(spec, &a.pg);
    if (st) return st;
    if ((st = check_attention_sizes(dtype, tokens, q_heads, a.pg, max_q)) || (st = check_seqs(seqs, a.pg, n_pages, tokens, &a.sq)) ||
        (st = check_reach(seqs, a.pg.page)) || (st = check_mask(scale, causal, window)))
        return st;
    if (!(decay >= 0.0f) || !std::isfinite(decay)) return fail(HR_EINVAL, "decay must be finite and not negative");
    if ((st = check_width(width, seqs->max_pages, a.pg.page))) return st;
    if (tokens == 0) return ok();
    int64_t qb;
    if ((st = check_rows(q, "q", q_stride_token, q_stride_head, tokens, q_heads, a.pg.d, dtype, &qb)) ||
        (st = check_ptr(pool, "pool", 16)) || (st = check_ptr(lse, "lse", 4)) || (st = check_ptr(weights, "weights", 4)))
        return st;
    a.few = few_tiles(tokens, q_heads / a.pg.hkv, seqs->rows, max_q);
    const int64_t need = hr::cache_weights_bytes(seqs->rows, tokens, q_heads, a.pg.d, a.few);
    if ((st = check_ptr(work, "work", 16))) return st;
    if (work_bytes < need) return fail(HR_EINVAL, "work_bytes = %lld: %lld are needed", (long long)work_bytes, (long long)need);
    const Range r[] = {{"weights", weights, size_of(size_of(seqs->rows, a.pg.hkv), width, 4), true},
                       {"work", work, need, true},
                       {"q", q, qb, false},
                       {"lse", lse, tokens * q_heads * 4, false},
                       {"pool", pool, size_of(n_pages, a.pg.page_bytes), false},
                       {"table", seqs->table, seqs->rows * seqs->max_pages * 4, false},
                       {"lens", seqs->lens, seqs->rows * 4, false},
                       {"cu_q", seqs->cu_q, (seqs->rows + 1) * 4, false}};
    if ((st = check_overlap(r, 8))) return st;
    int workers;
    const int e = hr::cache_weights_workers(a.few, &workers);
    if (e != 0) return fail(HR_EDEVICE, "device query failed: %s", hipGetErrorString(static_cast<hipError_t>(e)));
    a.q = q;
    a.pool = static_cast<const uint8_t*>(pool);
    a.lse = lse;
    a.weights = weights;
    a.work = static_cast<uint8_t*>(work);
    a.q_st = q_stride_token;
    a.q_sh = q_stride_head;
    a.width = width;
    a.norm = static_cast<float>(1.0 / sqrt(static_cast<double>(a.pg.d)));
    a.scale = scale > 0.0f ? scale : a.norm;
    a.decay = decay;
    a.hq = q_heads;
    a.rep = q_heads / a.pg.hkv;
    a.causal = causal != 0;
    a.window = window >= (int64_t{1} << 31) ? 0 : static_cast<int32_t>(window);
    a.rotate = rotate != 0;
    a.workers = workers;
    return launched(hr::launch_cache_weights(a, dtype == HR_BF16, stream));
}

int hr_cache_evict_work(int64_t n_pages, int64_t rows, int64_t* bytes) {
    if (!bytes) return fail(HR_EINVAL, "bytes is NULL");
    int st = check_pages(n_pages, 1);
    if (st) return st;
    if (rows < 0 || rows > kMaxCount) return fail(HR_EINVAL, "rows = %lld must be in 0..2^30", (long long)rows);
    *bytes = hr::cache_evict_words(n_pages, rows) * 4;
    return ok();
}

int hr_cache_evict(void* pool, int64_t layers, int64_t n_pages, const hr_cache_spec* spec, const int32_t* table,
                   const int32_t* lens, int64_t rows, int64_t max_pages, float* weights, int64_t width, int64_t budget,
                   int64_t sinks, int64_t recent, int32_t* new_table, int32_t* new_lens, int32_t* refs, int32_t* status,
                   void* work, int64_t work_bytes, void* stream) {
    hr::CachePage pg;
    int st = check_spec(spec, &pg);
    if (st) return st;
    if ((st = check_pages(n_pages, layers)) || (st = check_table(rows, max_pages, pg.page, "rows")) ||
        (st = check_counted(rows, max_pages, "rows")) || (st = check_width(width, max_pages, pg.page)))
        return st;
    if (budget <= 0 || budget >= (int64_t{1} << 31)) return fail(HR_EINVAL, "budget = %lld must be positive and below 2^31", (long long)budget);
    if (sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
        return fail(HR_EINVAL, "sinks = %lld and recent = %lld must not be negative, and together at most budget = %lld", (long long)sinks,
                    (long long)recent, (long long)budget);
    if ((st = check_ptr(pool, "pool", 16)) || (st = check_ptr(refs, "refs", 4)) || (st = check_ptr(status, "status", 4))) return st;
    if (rows > 0 && ((st = check_ptr(table, "table", 4)) || (st = check_ptr(lens, "lens", 4)) ||
                     (st = check_ptr(weights, "weights", 4)) || (st = check_ptr(new_table, "new_table", 4)) ||
                     (st = check_ptr(new_lens, "new_lens", 4))))
        return st;
    const int64_t need = hr::cache_evict_words(n_pages, rows) * 4;
    if ((st = check_ptr(work, "work", 16))) return st;
    if (work_bytes < need) return fail(HR_EINVAL, "work_bytes = %lld: %lld are needed", (long long)work_bytes, (long long)need);
    const int64_t wide = size_of(size_of(layers, rows, pg.hkv), width, 4);
    const Range r[] = {{"pool", pool, size_of(layers, n_pages, pg.page_bytes), true},
                       {"weights", weights, wide, true},
                       {"new_table", new_table, rows * max_pages * 4, true},
                       {"new_lens", new_lens, rows * 4, true},
                       {"refs", refs, n_pages * 4, true},
                       {"status", status, 16, true},
                       {"work", work, need, true},
                       {"table", table, rows * max_pages * 4, false},
                       {"lens", lens, rows * 4, false}};
    if ((st = check_overlap(r, 9))) return st;
    hr::CacheEvictArgs a{};
    a.pool = static_cast<uint8_t*>(pool);
    a.table = table;
    a.lens = lens;
    a.weights = weights;
    a.new_table = new_table;
    a.new_lens = new_lens;
    a.refs = refs;
    a.status = status;
    a.work = static_cast<int32_t*>(work);
    a.pg = pg;
    a.layers = layers;
    a.n_pages = n_pages;
    a.width = width;
    a.rows = static_cast<int32_t>(rows);
    a.max_pages = static_cast<int32_t>(max_pages);
    a.budget = static_cast<int32_t>(budget);
    a.sinks = static_cast<int32_t>(sinks);
    a.recent = static_cast<int32_t>(recent);
    return launched(hr::launch_cache_evict(a, stream));
}

}  // extern "C"
