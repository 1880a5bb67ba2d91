// C-ABI entry points of the paged 4-bit cache (include/hadarot_cache.h):
// argument validation, the page layout, and the choice of kernels.  Every
// check runs before anything is enqueued.
#include <hip/hip_runtime_api.h>
#include <math.h>
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

// The new tokens that a sequence of the call has, for the choice of a kernel: the
// caller's bound, or without one the mean (which they are where cu_q is NULL).
// One token in each of 64 sequences of up to 32768 positions: 94 us, where all
// tokens counted as one sequence's took 313.  A prompt among 63 single tokens (4000
// positions, 32 heads over 8 of 128), few-row kernel against shared, us: 128 tokens
// 93, 98; 512 166, 360; 1400 (rows by the mean: shared) 314, 415.
int64_t new_tokens(int64_t tokens, int64_t seqs, int64_t max_q) {
    if (max_q > 0) return max_q < tokens ? max_q : tokens;
    return seqs > 0 ? (tokens + seqs - 1) / seqs : tokens;
}

// The kernel of a call, by its query rows (query heads per kv head x new tokens
// of a sequence at most) and its scores at most (query rows x keys; the lengths
// are on the device, so keys are what the table or the window allows).
// Few rows: a workgroup's waves take different keys of the same 16 or 32 rows
// (32: one group per vector, heads up to 128; the registers of more do not fit).
// Many: the waves take different rows of the same keys, whose operands they
// share, 256 or 128 to a workgroup.  Measured, few-row kernel against shared, us:
//   rows of a sequence (32 sequences, 8000 keys, 8 kv heads; bfloat16, heads of
//   128): one group 32: 86, 206; 64: 134, 211; 128: 246, 218.  float32 64: 262,
//   413; 128: 489, 448.  Groups of 32 (4 kv heads) 28: 102, 124; 42: 142, 129;
//   56: 174, 131.  Heads of 256 (16 sequences, 4000 keys) 32: 63, 105; 64: 95, 126.
//   scores of all heads (millions), 1 sequence of 8000 keys if nothing else is
//   said: one group 8: 31, 42; 33: 53, 59 and (4 of 4000 keys) 56, 59; 66: 81, 76;
//   134: 136, 112.  float32 13: 43, 72; 17 (2 of 4100 keys): 50, 68; 33: 77, 102;
//   67: 137, 151.  Groups of 32 7: 38, 57; 14: 56, 57; 17: 63, 61.  Heads of 256 8:
//   44, 86; 33: 91, 105.
// So heads of 256 (64 rows, 33 million scores) and float32 calls (67 million) go to
// the shared kernel somewhat before it is the faster one.
void attn_key(const hr::CachePage& pg, int dtype, int64_t tokens, int32_t q_heads, int64_t seqs, int64_t max_q, int64_t keys,
              hr::CacheAttnKey* k) {
    memset(k, 0, sizeof *k);
    const int64_t rows = new_tokens(tokens, seqs, max_q) * (q_heads / pg.hkv);
    k->d = pg.d;
    k->ng = pg.ng;
    k->sf32 = pg.sf32;
    k->wide = dtype == HR_F32;
    const bool two = !k->wide && pg.d <= 128 && pg.ng == 1, light = k->wide || two;
    if (rows <= (light ? 96 : 32) || tokens * q_heads < (int64_t{1} << (light ? 25 : 23)) / (keys > 0 ? keys : 1)) {
        k->rt = rows > 16 && two ? 2 : 1;
        k->wr = 1;
    } else {
        k->rt = k->wide || pg.d == 256 ? 1 : 2;
        k->wr = 8;
    }
}

int attn_sizes(int dtype, int64_t tokens, int32_t q_heads, const hr::CachePage& pg, int64_t max_q) {
    int st;
    if ((st = check_tokens(dtype, tokens))) return st;
    if (q_heads <= 0 || q_heads > kMaxHeads) return fail(HR_EINVAL, "q_heads = %d must be in 1..%lld", q_heads, (long long)kMaxHeads);
    if (q_heads % pg.hkv) return fail(HR_EINVAL, "q_heads = %d is not a multiple of kv_heads = %d", q_heads, pg.hkv);
    if (max_q < 0) return fail(HR_EINVAL, "max_q = %lld is negative", (long long)max_q);
    if (tokens * q_heads >= (int64_t{1} << 31)) return fail(HR_EINVAL, "tokens * q_heads must be below 2^31");
    return HR_OK;
}

int attn_work_bytes(const hr::CacheAttnKey& k, int* workers, int64_t* bytes) {
    const int e = hr::cache_attn_workers(k, workers);
    if (e != 0) return fail(HR_EDEVICE, "occupancy query failed: %s", hipGetErrorString(static_cast<hipError_t>(e)));
    // two partial results per workgroup, rows of d sums, a maximum and a sum of
    // exponentials each, and a record of the unit that it leaves unfinished
    *bytes = int64_t{*workers} * (2 * (16 * k.rt * k.wr) * (k.d + 4) * 4 + 32);
    return HR_OK;
}

}  // namespace

extern "C" {

int hr_cache_page_layout(const hr_cache_spec* spec, hr_cache_page* out) {
    hr::CachePage p;
    int st = check_spec(spec, &p);
    if (st) return st;
    if (!out) return fail(HR_EINVAL, "out is NULL");
    out->page_bytes = p.page_bytes;
    out->head_bytes = p.head_bytes;
    out->k_codes = p.kc;
    out->v_codes = p.vc;
    out->k_scales = p.ks;
    out->v_scales = p.vs;
    out->k_zeros = p.kz;
    out->v_zeros = p.vz;
    return ok();
}

int hr_cache_append(void* pool, int64_t n_pages, const hr_cache_spec* spec, const hr_cache_seqs* seqs, const void* k,
                    int64_t k_stride_token, int64_t k_stride_head, const void* v, int64_t v_stride_token,
                    int64_t v_stride_head, int dtype, int64_t tokens, int rotate, void* stream) {
    hr::CacheAppendArgs a{};
    int st = check_spec(spec, &a.pg);
    if (st) return st;
    if ((st = check_tokens(dtype, tokens)) || (st = check_seqs(seqs, a.pg, n_pages, tokens, &a.sq))) return st;
    if (tokens == 0) return ok();
    int64_t kb, vb;
    if ((st = check_ptr(pool, "pool", 16)) ||
        (st = check_rows(k, "k", k_stride_token, k_stride_head, tokens, a.pg.hkv, a.pg.d, dtype, &kb)) ||
        (st = check_rows(v, "v", v_stride_token, v_stride_head, tokens, a.pg.hkv, a.pg.d, dtype, &vb)))
        return st;
    const Range r[] = {{"pool", pool, size_of(n_pages, a.pg.page_bytes), true},
                       {"k", k, kb, false},
                       {"v", v, vb, false},
                       {"table", seqs->table, seqs->rows * seqs->max_pages * 4, false},
                       {"lens", seqs->lens, seqs->rows * 4, false},
                       {"cu_q", seqs->cu_q, (seqs->rows + 1) * 4, false}};
    if ((st = check_overlap(r, 6))) return st;
    a.pool = static_cast<uint8_t*>(pool);
    a.k = k;
    a.v = v;
    a.k_st = k_stride_token;
    a.k_sh = k_stride_head;
    a.v_st = v_stride_token;
    a.v_sh = v_stride_head;
    a.norm = static_cast<float>(1.0 / sqrt(static_cast<double>(a.pg.d)));
    a.rotate = rotate != 0;
    const int64_t block = 1024 / a.pg.d;  // positions that a wave takes
    const int64_t units = tokens / block + 2 * seqs->rows;
    if (units * ((a.pg.hkv + 3) / 4) >= kMaxGrid) return fail(HR_EUNSUPPORTED, "too many rows, tokens and heads for one launch");
    a.units = static_cast<int32_t>(units);
    return launched(hr::launch_cache_append(a, dtype == HR_BF16, stream));
}

int hr_cache_attention_work(int dtype, int64_t tokens, int32_t q_heads, const hr_cache_spec* spec, int64_t rows,
                            int64_t max_q, int64_t* bytes) {
    hr::CachePage pg;
    int st = check_spec(spec, &pg);
    if (st) return st;
    if (!bytes) return fail(HR_EINVAL, "bytes is NULL");
    if ((st = attn_sizes(dtype, tokens, q_heads, pg, max_q))) return st;
    if (rows < 0 || rows > kMaxCount) return fail(HR_EINVAL, "rows = %lld must be in 0..2^30", (long long)rows);
    *bytes = 0;
    if (tokens == 0) return ok();
    hr::CacheAttnKey key;
    // what suffices for any length and window: of the kernels of no keys and of
    // all that there can be
    int64_t need[2];
    for (int i = 0; i < 2; ++i) {
        int workers;
        attn_key(pg, dtype, tokens, q_heads, rows, max_q, i ? kMaxKeys : 0, &key);
        if ((st = attn_work_bytes(key, &workers, &need[i]))) return st;
    }
    *bytes = need[0] > need[1] ? need[0] : need[1];
    return ok();
}

int hr_cache_attention(const void* q, int64_t q_stride_token, int64_t q_stride_head, int dtype, int64_t tokens,
                       int32_t q_heads, const void* pool, int64_t n_pages, const hr_cache_spec* spec,
                       const hr_cache_seqs* seqs, float scale, int causal, int64_t window, int rotate, void* out,
                       int64_t out_stride_token, int64_t out_stride_head, float* lse, int64_t max_q, void* work,
                       int64_t work_bytes, void* stream) {
    hr::CacheAttnArgs a{};
    int st = check_spec(spec, &a.pg);
    if (st) return st;
    if ((st = attn_sizes(dtype, tokens, q_heads, a.pg, max_q)) ||
        (st = check_seqs(seqs, a.pg, n_pages, tokens, &a.sq)))
        return st;
    if (!(scale >= 0.0f) || !std::isfinite(scale)) return fail(HR_EINVAL, "scale must be positive and finite (0: 1 / sqrt(head_dim))");
    if (window < 0) return fail(HR_EINVAL, "window = %lld is negative", (long long)window);
    if (window > 0 && !causal) return fail(HR_EINVAL, "a window needs causal attention");
    if (tokens == 0) return ok();
    int64_t qb, ob;
    if ((st = check_rows(q, "q", q_stride_token, q_stride_head, tokens, q_heads, a.pg.d, dtype, &qb)) ||
        (st = check_rows(out, "out", out_stride_token, out_stride_head, tokens, q_heads, a.pg.d, dtype, &ob)) ||
        (st = check_distinct("out", out_stride_token, out_stride_head, tokens, q_heads, a.pg.d)) ||
        (st = check_ptr(pool, "pool", 16)) || (lse && (st = check_ptr(lse, "lse", 4))))
        return st;
    const bool in_place = q == out && q_stride_token == out_stride_token && q_stride_head == out_stride_head;
    // in place is safe: the rows of a unit are read by the workgroups that
    // work on it alone, and written by the last of them or, where the unit is
    // cut over several, by the joining launch
    Range r[] = {{"out", out, ob, true},
                 {"lse", lse, lse ? tokens * q_heads * 4 : 0, true},
                 {"q", in_place ? nullptr : q, qb, false},
                 {"pool", pool, size_of(n_pages, a.pg.page_bytes), false},
                 {"table", seqs->table, seqs->rows * seqs->max_pages * 4, false},
                 {"lens", seqs->lens, seqs->rows * 4, false},
                 {"cu_q", seqs->cu_q, (seqs->rows + 1) * 4, false},
                 {"work", nullptr, 0, true}};
    if ((st = check_overlap(r, 7))) return st;
    int64_t keys = int64_t{seqs->max_pages} << a.pg.logp;
    if (window > 0 && window < keys - tokens) keys = window + new_tokens(tokens, seqs->rows, max_q);
    hr::CacheAttnKey key;
    attn_key(a.pg, dtype, tokens, q_heads, seqs->rows, max_q, keys, &key);
    int workers;
    int64_t need;
    if ((st = attn_work_bytes(key, &workers, &need))) return st;
    if ((st = check_ptr(work, "work", 16))) return st;
    if (work_bytes < need)
        return fail(HR_EINVAL, "work_bytes = %lld: %lld are needed", (long long)work_bytes, (long long)need);
    r[0].written = r[1].written = false;   // (compared above)
    r[2].p = q;
    r[7] = {"work", work, need, true};
    if ((st = check_overlap(r, 8))) return st;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.pool = static_cast<const uint8_t*>(pool);
    a.work = static_cast<float*>(work);
    a.q_st = q_stride_token;
    a.q_sh = q_stride_head;
    a.o_st = out_stride_token;
    a.o_sh = out_stride_head;
    a.norm = static_cast<float>(1.0 / sqrt(static_cast<double>(a.pg.d)));
    a.scale = scale > 0.0f ? scale : a.norm;
    a.hq = q_heads;
    a.rep = q_heads / a.pg.hkv;
    a.causal = causal != 0;
    a.window = window >= (int64_t{1} << 31) ? 0 : static_cast<int32_t>(window);
    a.rotate = rotate != 0;
    a.workers = workers;
    return launched(hr::launch_cache_attn(key, a, stream));
}

int hr_cache_update_work(int64_t n_pages, int64_t new_rows, int64_t* bytes) {
    if (!bytes) return fail(HR_EINVAL, "bytes is NULL");
    int st = check_pages(n_pages, 1);
    if (st) return st;
    if (new_rows < 0 || new_rows > kMaxCount) return fail(HR_EINVAL, "new_rows = %lld must be in 0..2^30", (long long)new_rows);
    *bytes = hr::cache_update_words(n_pages, new_rows) * 4;
    return ok();
}

int hr_cache_update(void* pool, int64_t layers, int64_t n_pages, const hr_cache_spec* spec, const int32_t* table,
                    const int32_t* lens, int64_t rows, int64_t max_pages, const int32_t* parents, const int32_t* grow,
                    int64_t new_rows, int32_t* new_table, int32_t* new_lens, int32_t* refs, int32_t* status, void* work,
                    int64_t work_bytes, void* stream) {
    hr::CachePage pg;
    int st = check_spec(spec, &pg);
    if (st) return st;
    if ((st = check_pages(n_pages, layers)) || (st = check_table(rows, max_pages, pg.page, "rows")) ||
        (st = check_table(new_rows, max_pages, pg.page, "new_rows")) || (st = check_counted(rows, max_pages, "rows")) ||
        (st = check_counted(new_rows, max_pages, "new_rows")))
        return st;
    if ((st = check_ptr(pool, "pool", 16)) || (st = check_ptr(refs, "refs", 4)) || (st = check_ptr(status, "status", 4)))
        return st;
    if (rows > 0 && ((st = check_ptr(table, "table", 4)) || (st = check_ptr(lens, "lens", 4)))) return st;
    if (new_rows > 0 && ((st = check_ptr(parents, "parents", 4)) || (st = check_ptr(grow, "grow", 4)) ||
                         (st = check_ptr(new_table, "new_table", 4)) || (st = check_ptr(new_lens, "new_lens", 4))))
        return st;
    const int64_t need = hr::cache_update_words(n_pages, new_rows) * 4;
    if ((st = check_ptr(work, "work", 16))) return st;
    if (work_bytes < need) return fail(HR_EINVAL, "work_bytes = %lld: %lld are needed", (long long)work_bytes, (long long)need);
    const Range r[] = {{"pool", pool, size_of(layers, n_pages, pg.page_bytes), true},
                       {"new_table", new_table, new_rows * max_pages * 4, true},
                       {"new_lens", new_lens, new_rows * 4, true},
                       {"refs", refs, n_pages * 4, true},
                       {"status", status, 16, true},
                       {"work", work, need, true},
                       {"table", table, rows * max_pages * 4, false},
                       {"lens", lens, rows * 4, false},
                       {"parents", parents, new_rows * 4, false},
                       {"grow", grow, new_rows * 4, false}};
    if ((st = check_overlap(r, 10))) return st;
    hr::CacheUpdateArgs a{};
    a.pool = static_cast<uint8_t*>(pool);
    a.table = table;
    a.lens = lens;
    a.parents = parents;
    a.grow = grow;
    a.new_table = new_table;
    a.new_lens = new_lens;
    a.refs = refs;
    a.status = status;
    a.work = static_cast<int32_t*>(work);
    a.layers = layers;
    a.n_pages = n_pages;
    a.page_bytes = pg.page_bytes;
    a.rows = static_cast<int32_t>(rows);
    a.max_pages = static_cast<int32_t>(max_pages);
    a.new_rows = static_cast<int32_t>(new_rows);
    a.page = pg.page;
    return launched(hr::launch_cache_update(a, stream));
}

int hr_cache_compact_work(int64_t n_pages, int64_t* bytes) {
    if (!bytes) return fail(HR_EINVAL, "bytes is NULL");
    int st = check_pages(n_pages, 1);
    if (st) return st;
    *bytes = hr::cache_compact_words(n_pages) * 4;
    return ok();
}

int hr_cache_compact(void* pool, int64_t layers, int64_t n_pages, const hr_cache_spec* spec, const int32_t* table,
                     const int32_t* lens, int64_t rows, int64_t max_pages, void* into, int64_t into_pages,
                     int32_t* new_table, int32_t* refs, int32_t* status, void* work, int64_t work_bytes, void* stream) {
    hr::CachePage pg;
    int st = check_spec(spec, &pg);
    if (st) return st;
    if ((st = check_pages(n_pages, layers)) || (st = check_table(rows, max_pages, pg.page, "rows")) ||
        (st = check_counted(rows, max_pages, "rows")))
        return st;
    if (into && (into_pages <= 0 || into_pages > kMaxCount))
        return fail(HR_EINVAL, "into_pages = %lld must be in 1..2^30", (long long)into_pages);
    if ((st = check_ptr(pool, "pool", 16)) || (into && (st = check_ptr(into, "into", 16))) ||
        (st = check_ptr(refs, "refs", 4)) || (st = check_ptr(status, "status", 4)))
        return st;
    if (rows > 0 && ((st = check_ptr(table, "table", 4)) || (st = check_ptr(lens, "lens", 4)) ||
                     (st = check_ptr(new_table, "new_table", 4))))
        return st;
    const int64_t need = hr::cache_compact_words(n_pages) * 4;
    if ((st = check_ptr(work, "work", 16))) return st;
    if (work_bytes < need) return fail(HR_EINVAL, "work_bytes = %lld: %lld are needed", (long long)work_bytes, (long long)need);
    const Range r[] = {{"pool", pool, size_of(layers, n_pages, pg.page_bytes), true},
                       {"into", into, into ? size_of(layers, into_pages, pg.page_bytes) : 0, true},
                       {"new_table", new_table, rows * max_pages * 4, true},
                       {"refs", refs, (into ? into_pages : n_pages) * 4, true},
                       {"status", status, 16, true},
                       {"work", work, need, true},
                       {"table", table, rows * max_pages * 4, false},
                       {"lens", lens, rows * 4, false}};
    if ((st = check_overlap(r, 8))) return st;
    hr::CacheCompactArgs a{};
    a.pool = static_cast<uint8_t*>(pool);
    a.into = static_cast<uint8_t*>(into);
    a.table = table;
    a.lens = lens;
    a.new_table = new_table;
    a.refs = refs;
    a.status = status;
    a.work = static_cast<int32_t*>(work);
    a.layers = layers;
    a.n_pages = n_pages;
    a.into_pages = into ? into_pages : n_pages;
    a.page_bytes = pg.page_bytes;
    a.rows = static_cast<int32_t>(rows);
    a.max_pages = static_cast<int32_t>(max_pages);
    a.page = pg.page;
    return launched(hr::launch_cache_compact(a, stream));
}

}  // extern "C"
