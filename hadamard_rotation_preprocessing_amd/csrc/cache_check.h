// Checks of arguments that the C entry points of the paged 4-bit caches share:
// pointers, sizes, overlaps, page records, page tables, sequences and strided
// rows.  Every one runs on the host, before anything is enqueued.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <cmath>

#include "../../include/hadarot_cache.h"
#include "cache.h"

namespace {

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return hr::set_error(status, buf);
}

int ok() { return hr::set_error(HR_OK, ""); }

int launched(int e) {
    if (e != 0) return fail(HR_EDEVICE, "kernel launch failed: %s", hipGetErrorString(static_cast<hipError_t>(e)));
    return ok();
}

bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// No count of rows, pages, tokens or heads above these; every index then stays
// within 31 bits.  Products with strides and page sizes need not stay within 63:
// size_of and sum_of hold them at the largest.
constexpr int64_t kMaxCount = int64_t{1} << 30;
constexpr int64_t kMaxHeads = 1 << 16;
// workgroups of 256 threads of a launch (a grid holds fewer than 2^32 threads)
constexpr int64_t kMaxGrid = 1 << 24;
constexpr int64_t kMaxKeys = int64_t{1} << 31;

int64_t size_of(int64_t a, int64_t b, int64_t c = 1) {   // a b c, none negative
    int64_t r;
    if (__builtin_mul_overflow(a, b, &r) || __builtin_mul_overflow(r, c, &r)) return INT64_MAX;
    return r;
}
int64_t sum_of(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_add_overflow(a, b, &r) ? INT64_MAX : r;
}

int check_ptr(const void* p, const char* name, size_t align) {
    if (!p) return fail(HR_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align) return fail(HR_EINVAL, "%s is not %zu-byte aligned", name, align);
    return HR_OK;
}

struct Range {
    const char* name;
    const void* p;
    int64_t bytes;
    bool written;
};

// No written range may overlap another one.
int check_overlap(const Range* r, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j) {
            if (!r[i].p || !r[j].p || !(r[i].written || r[j].written) || r[i].bytes <= 0 || r[j].bytes <= 0) continue;
            const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].p), b = reinterpret_cast<uintptr_t>(r[j].p);
            // (by distance: an end may lie past the last address)
            if (a < b ? b - a < static_cast<uintptr_t>(r[i].bytes) : a - b < static_cast<uintptr_t>(r[j].bytes))
                return fail(HR_EINVAL, "%s overlaps %s", r[i].name, r[j].name);
        }
    return HR_OK;
}

int check_spec(const hr_cache_spec* s, hr::CachePage* p) {
    if (!s) return fail(HR_EINVAL, "cache spec is NULL");
    if (s->kv_heads <= 0 || s->kv_heads > kMaxHeads)
        return fail(HR_EINVAL, "kv_heads = %d must be in 1..%lld", s->kv_heads, (long long)kMaxHeads);
    if (s->head_dim <= 0) return fail(HR_EINVAL, "head_dim = %d must be positive", s->head_dim);
    if (s->head_dim != 64 && s->head_dim != 128 && s->head_dim != 256)
        return fail(HR_EUNSUPPORTED, "head_dim = %d: 64, 128 and 256 are implemented", s->head_dim);
    if (s->page_size <= 0) return fail(HR_EINVAL, "page_size = %d must be positive", s->page_size);
    if (!is_pow2(s->page_size) || s->page_size < 16 || s->page_size > 256)
        return fail(HR_EUNSUPPORTED, "page_size = %d: powers of two from 16 to 256 are implemented", s->page_size);
    const hr_qspec& q = s->q;
    if (q.format == HR_Q_MXFP4 || q.format == HR_Q_NVFP4)
        return fail(HR_EUNSUPPORTED, "the cache holds INT groups: MXFP4 and NVFP4 pages are not implemented");
    if (q.format != HR_Q_INT) return fail(HR_EINVAL, "quantizer format %d is not HR_Q_INT", q.format);
    if (q.bits != 4) return fail(HR_EUNSUPPORTED, "bits = %d: only 4-bit codes are implemented", q.bits);
    if (q.sym != 0 && q.sym != 1) return fail(HR_EINVAL, "sym must be 0 or 1");
    if (q.scale_dtype != HR_F32 && q.scale_dtype != HR_BF16)
        return fail(HR_EINVAL, "INT scales must be HR_F32 or HR_BF16");
    if (q.group_size <= 0 || s->head_dim % q.group_size)
        return fail(HR_EINVAL, "group_size %d does not divide head_dim = %d", q.group_size, s->head_dim);
    if (!is_pow2(q.group_size) || q.group_size < 32)
        return fail(HR_EUNSUPPORTED, "group_size %d: powers of two from 32 to head_dim are implemented", q.group_size);
    memset(p, 0, sizeof *p);
    p->hkv = s->kv_heads;
    p->d = s->head_dim;
    p->ng = s->head_dim / q.group_size;
    p->page = s->page_size;
    while ((1 << p->logp) < p->page) ++p->logp;
    p->sym = q.sym;
    p->sf32 = q.scale_dtype == HR_F32;
    const int64_t codes = int64_t{p->page} * p->d / 2;
    const int64_t scales = up(int64_t{p->page} * p->ng * (p->sf32 ? 4 : 2), 16);
    const int64_t zeros = p->sym ? 0 : up(int64_t{p->page} * p->ng / 2, 16);
    p->vc = static_cast<int32_t>(codes);
    p->ks = static_cast<int32_t>(2 * codes);
    p->vs = static_cast<int32_t>(2 * codes + scales);
    p->kz = p->sym ? 0 : static_cast<int32_t>(2 * codes + 2 * scales);
    p->vz = p->sym ? 0 : static_cast<int32_t>(2 * codes + 2 * scales + zeros);
    p->head_bytes = up(2 * (codes + scales + zeros), 128);
    p->page_bytes = p->head_bytes * p->hkv;
    return HR_OK;
}

int check_pages(int64_t n_pages, int64_t layers) {
    if (n_pages <= 0 || n_pages > kMaxCount) return fail(HR_EINVAL, "n_pages = %lld must be in 1..2^30", (long long)n_pages);
    if (layers <= 0 || layers > (1 << 20)) return fail(HR_EINVAL, "layers = %lld must be in 1..2^20", (long long)layers);
    return HR_OK;
}

int check_table(int64_t rows, int64_t max_pages, int page, const char* name) {
    if (rows < 0 || rows > kMaxCount) return fail(HR_EINVAL, "%s = %lld must be in 0..2^30", name, (long long)rows);
    if (max_pages <= 0 || max_pages * page >= (int64_t{1} << 31))
        return fail(HR_EINVAL, "max_pages = %lld must be positive and hold fewer than 2^31 positions", (long long)max_pages);
    if (rows * max_pages > (int64_t{1} << 40)) return fail(HR_EINVAL, "page table too large");
    return HR_OK;
}

// A table whose entries are counted (holders of a page, pages handed out): the
// kernels do that in 31 bits.
int check_counted(int64_t rows, int64_t max_pages, const char* name) {
    if (rows * max_pages >= (int64_t{1} << 31))
        return fail(HR_EUNSUPPORTED, "%s x max_pages = %lld x %lld must be below 2^31", name, (long long)rows, (long long)max_pages);
    return HR_OK;
}

int check_seqs(const hr_cache_seqs* s, const hr::CachePage& pg, int64_t n_pages, int64_t tokens, hr::CacheSeqs* o) {
    if (!s) return fail(HR_EINVAL, "seqs is NULL");
    int st;
    if ((st = check_pages(n_pages, 1))) return st;
    if ((st = check_table(s->rows, s->max_pages, pg.page, "rows"))) return st;
    if (s->rows == 0 && tokens > 0) return fail(HR_EINVAL, "%lld tokens of no rows", (long long)tokens);
    if (tokens == 0) return HR_OK;
    if (!s->cu_q && tokens % s->rows)
        return fail(HR_EINVAL, "tokens = %lld is not a multiple of rows = %lld and cu_q is NULL", (long long)tokens,
                    (long long)s->rows);
    if ((st = check_ptr(s->table, "table", 4)) || (st = check_ptr(s->lens, "lens", 4))) return st;
    if (s->cu_q && (st = check_ptr(s->cu_q, "cu_q", 4))) return st;
    o->table = s->table;
    o->lens = s->lens;
    o->cu = s->cu_q;
    o->rows = static_cast<int32_t>(s->rows);
    o->max_pages = static_cast<int32_t>(s->max_pages);
    o->tokens = static_cast<int32_t>(tokens);
    o->per = static_cast<int32_t>(tokens / s->rows);
    o->n_pages = n_pages;
    return HR_OK;
}

// For kernels that look some tiles past a sequence's end: positions there are still ints.
int check_reach(const hr_cache_seqs* s, int page) {
    constexpr int64_t most = (int64_t{1} << 31) - (1 << 16);
    if (s->max_pages * page > most)
        return fail(HR_EUNSUPPORTED, "max_pages = %lld hold more than 2^31 - 2^16 positions", (long long)s->max_pages);
    return HR_OK;
}

int check_tokens(int dtype, int64_t tokens) {
    if (dtype != HR_F32 && dtype != HR_BF16) return fail(HR_EINVAL, "dtype %d is not HR_F32 or HR_BF16", dtype);
    if (tokens < 0 || tokens > kMaxCount) return fail(HR_EINVAL, "tokens = %lld must be in 0..2^30", (long long)tokens);
    return HR_OK;
}

// A strided [tokens, heads, d] tensor: rows 16-byte aligned, and strides that
// do not make two rows overlap.
int check_rows(const void* p, const char* name, int64_t st, int64_t sh, int64_t tokens, int64_t heads, int d, int dtype,
               int64_t* bytes) {
    int e;
    if ((e = check_ptr(p, name, 16))) return e;
    const int64_t es = dtype == HR_F32 ? 4 : 2;
    if (st < 0 || sh < 0 || st > (int64_t{1} << 40) || sh > (int64_t{1} << 40))
        return fail(HR_EINVAL, "%s strides must be in 0..2^40", name);
    if ((tokens > 1 && st * es % 16) || (heads > 1 && sh * es % 16))
        return fail(HR_EINVAL, "%s rows are not 16-byte aligned (strides %lld, %lld)", name, (long long)st, (long long)sh);
    if ((heads > 1 && sh < d) || (tokens > 1 && st < d))
        return fail(HR_EINVAL, "%s strides %lld, %lld are smaller than a row of %d", name, (long long)st, (long long)sh, d);
    *bytes = size_of(sum_of(size_of(tokens - 1, st), (heads - 1) * sh + d), es);
    return HR_OK;
}

// Rows of [tokens, heads] may not share elements where they are written: one
// of the two strides has to span the whole of the other dimension.
int check_distinct(const char* name, int64_t st, int64_t sh, int64_t tokens, int64_t heads, int d) {
    if (tokens <= 1 || heads <= 1) return HR_OK;
    if (st >= (heads - 1) * sh + d || sh >= sum_of(size_of(tokens - 1, st), d)) return HR_OK;
    return fail(HR_EINVAL, "%s strides %lld, %lld make rows overlap", name, (long long)st, (long long)sh);
}

int check_attention_sizes(int dtype, int64_t tokens, int32_t q_heads, const hr::CachePage& pg, int64_t max_q) {
    int st;
    if ((st = check_tokens(dtype, tokens))) return st;
    if (q_heads <= 0 || q_heads > kMaxHeads) return fail(HR_EINVAL, "q_heads = %d must be in 1..%lld", q_heads, (long long)kMaxHeads);
    if (q_heads % pg.hkv) return fail(HR_EINVAL, "q_heads = %d is not a multiple of kv_heads = %d", q_heads, pg.hkv);
    if (max_q < 0) return fail(HR_EINVAL, "max_q = %lld is negative", (long long)max_q);
    if (tokens * q_heads >= (int64_t{1} << 31)) return fail(HR_EINVAL, "tokens * q_heads must be below 2^31");
    return HR_OK;
}

int check_mask(float scale, int causal, int64_t window) {
    if (!(scale >= 0.0f) || !std::isfinite(scale)) return fail(HR_EINVAL, "scale must be positive and finite (0: 1 / sqrt(head_dim))");
    if (window < 0) return fail(HR_EINVAL, "window = %lld is negative", (long long)window);
    if (window > 0 && !causal) return fail(HR_EINVAL, "a window needs causal attention");
    return HR_OK;
}

}  // namespace
