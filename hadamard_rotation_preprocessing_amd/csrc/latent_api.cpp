// C-ABI entry points of the latent cache (include/hadarot_latent.h): argument
// validation, the page layout, and the choice of kernels.  Every check runs
// before anything is enqueued.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <cmath>

#include "../../include/hadarot_latent.h"
#include "cache_check.h"
#include "latent.h"

namespace {

int check_latent(const hr_latent_spec* s, hr::LatentPage* p) {
    if (!s) return fail(HR_EINVAL, "latent spec is NULL");
    if (s->latent_dim <= 0) return fail(HR_EINVAL, "latent_dim = %d must be positive", s->latent_dim);
    if (s->latent_dim != 256 && s->latent_dim != 512)
        return fail(HR_EUNSUPPORTED, "latent_dim = %d: 256 and 512 are implemented", s->latent_dim);
    if (s->rope_dim <= 0) return fail(HR_EINVAL, "rope_dim = %d must be positive", s->rope_dim);
    if (s->rope_dim != hr::kRope) return fail(HR_EUNSUPPORTED, "rope_dim = %d: 64 is implemented", s->rope_dim);
    // page size, format, bits, symmetry and scales are those of a cache of keys
    // with as many dimensions (256 at most)
    hr_cache_spec like{1, 256, s->page_size, s->q};
    if (s->q.format == HR_Q_INT) {
        const int32_t g = s->q.group_size;
        if (g <= 0 || s->latent_dim % g) return fail(HR_EINVAL, "group_size %d does not divide latent_dim = %d", g, s->latent_dim);
        if (!is_pow2(g) || g < 128) return fail(HR_EUNSUPPORTED, "group_size %d: powers of two from 128 to latent_dim are implemented", g);
        like.q.group_size = 128;
    }
    hr::CachePage c;
    const int st = check_spec(&like, &c);
    if (st) return st;
    memset(p, 0, sizeof *p);
    p->d = s->latent_dim;
    p->ng = s->latent_dim / s->q.group_size;
    p->page = c.page;
    p->logp = c.logp;
    p->sym = c.sym;
    p->sf32 = c.sf32;
    const int64_t codes = int64_t{p->page} * p->d / 2;
    const int64_t scales = up(int64_t{p->page} * p->ng * (p->sf32 ? 4 : 2), 16);
    const int64_t zeros = p->sym ? 0 : up(int64_t{p->page} * p->ng / 2, 16);
    p->scales = static_cast<int32_t>(codes);
    p->zeros = p->sym ? 0 : static_cast<int32_t>(codes + scales);
    p->rope = static_cast<int32_t>(codes + scales + zeros);
    p->page_bytes = up(codes + scales + zeros + int64_t{p->page} * hr::kRope * 2, 128);
    return HR_OK;
}

// A cache of keys whose pages have the same positions: for the checks of tables
// and sequences.
hr::CachePage like(const hr::LatentPage& p) {
    hr::CachePage c{};
    c.hkv = 1;
    c.d = p.d;
    c.page = p.page;
    c.logp = p.logp;
    c.page_bytes = p.page_bytes;
    return c;
}

int check_heads(int64_t tokens, int32_t heads, int64_t max_q) {
    if (heads <= 0 || heads > kMaxHeads) return fail(HR_EINVAL, "heads = %d must be in 1..%lld", heads, (long long)kMaxHeads);
    if (max_q < 0) return fail(HR_EINVAL, "max_q = %lld is negative", (long long)max_q);
    if (tokens * heads >= (int64_t{1} << 31)) return fail(HR_EINVAL, "tokens * heads must be below 2^31");
    return HR_OK;
}

// The kernel of a call, by the query rows (new tokens x heads) of a sequence.
void attn_key(const hr::LatentPage& pg, int dtype, int64_t tokens, int32_t heads, int64_t seqs, int64_t max_q, hr::LatentAttnKey* k) {
    memset(k, 0, sizeof *k);
    const int64_t n = max_q > 0 ? (max_q < tokens ? max_q : tokens) : seqs > 0 ? (tokens + seqs - 1) / seqs : tokens;
    const int64_t rows = n * heads;
    k->d = pg.d;
    k->ng = pg.ng;
    k->sf32 = pg.sf32;
    k->wide = dtype == HR_F32;
    k->rt = rows <= 32 || k->wide ? 1 : 2;
    k->wr = rows <= 16 ? 1 : 2;
}

int attn_work(const hr::LatentAttnKey& k, int64_t seqs, int64_t rows, int* workers, int64_t* bytes) {
    const int e = hr::latent_attn_workers(k, workers);
    if (e != 0) return fail(HR_EDEVICE, "occupancy query failed: %s", hipGetErrorString(static_cast<hipError_t>(e)));
    *bytes = hr::latent_work_bytes(k, seqs, rows, *workers);
    return HR_OK;
}

int check_scale(float scale, bool zero) {
    if (!(scale >= 0.0f) || !std::isfinite(scale) || (scale == 0.0f && !zero))
        return fail(HR_EINVAL, zero ? "scale must be positive and finite (0: 1 / sqrt(nope + 64))" : "scale must be positive and finite");
    return HR_OK;
}

// Whether rows of da elements at a and of db at b, with the same stride, lie in
// columns of their own.
bool beside(const void* a, int64_t da, const void* b, int64_t db, int64_t sa, int64_t sb, int dtype) {
    if (sa != sb) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const uintptr_t es = dtype == HR_F32 ? 4 : 2, apart = (x < y ? y - x : x - y) / es;
    const uintptr_t left = static_cast<uintptr_t>(x < y ? da : db), right = static_cast<uintptr_t>(x < y ? db : da);
    return apart >= left && apart + right <= static_cast<uintptr_t>(sa);
}

}  // namespace

extern "C" {

int hr_latent_page_layout(const hr_latent_spec* spec, hr_latent_page* out) {
    hr::LatentPage p;
    int st = check_latent(spec, &p);
    if (st) return st;
    if (!out) return fail(HR_EINVAL, "out is NULL");
    out->page_bytes = p.page_bytes;
    out->codes = 0;
    out->scales = p.scales;
    out->zeros = p.zeros;
    out->rope = p.rope;
    return ok();
}

int hr_latent_append(void* pool, int64_t n_pages, const hr_latent_spec* spec, const hr_cache_seqs* seqs, const void* c,
                     int64_t c_stride, const void* rope, int64_t rope_stride, int dtype, int64_t tokens, int rotate,
                     void* stream) {
    hr::LatentPagesArgs a{};
    int st = check_latent(spec, &a.pg);
    if (st) return st;
    if ((st = check_tokens(dtype, tokens)) || (st = check_seqs(seqs, like(a.pg), n_pages, tokens, &a.sq))) return st;
    if (tokens == 0) return ok();
    int64_t cb, rb;
    if ((st = check_ptr(pool, "pool", 16)) || (st = check_rows(c, "c", c_stride, 0, tokens, 1, a.pg.d, dtype, &cb)) ||
        (st = check_rows(rope, "rope", rope_stride, 0, tokens, 1, hr::kRope, dtype, &rb)))
        return st;
    const Range r[] = {{"pool", pool, size_of(n_pages, a.pg.page_bytes), true},
                       {"c", c, cb, false},
                       {"rope", rope, rb, false},
                       {"table", seqs->table, seqs->rows * seqs->max_pages * 4, false},
                       {"lens", seqs->lens, seqs->rows * 4, false},
                       {"cu_q", seqs->cu_q, (seqs->rows + 1) * 4, false}};
    if ((st = check_overlap(r, 6))) return st;
    a.pool = static_cast<uint8_t*>(pool);
    a.c_in = c;
    a.rope_in = rope;
    a.c_st = c_stride;
    a.r_st = rope_stride;
    a.norm = static_cast<float>(1.0 / sqrt(static_cast<double>(a.pg.d)));
    a.rotate = rotate != 0;
    const int64_t block = 1024 / a.pg.d;  // positions that a wave takes
    const int64_t units = tokens / block + 2 * seqs->rows;
    if (units / 4 >= kMaxGrid) return fail(HR_EUNSUPPORTED, "too many rows and tokens for one launch");
    a.units = static_cast<int32_t>(units);
    return launched(hr::launch_latent_append(a, dtype == HR_BF16, stream));
}

int hr_latent_read(const void* pool, int64_t n_pages, const hr_latent_spec* spec, const hr_cache_seqs* seqs, void* c,
                   int64_t c_stride, void* rope, int64_t rope_stride, int dtype, int64_t positions, int rotate, void* stream) {
    hr::LatentPagesArgs a{};
    int st = check_latent(spec, &a.pg);
    if (st) return st;
    if (dtype != HR_F32 && dtype != HR_BF16) return fail(HR_EINVAL, "dtype %d is not HR_F32 or HR_BF16", dtype);
    if (positions < 0 || positions > kMaxCount)
        return fail(HR_EINVAL, "positions = %lld must be in 0..2^30", (long long)positions);
    if ((st = check_seqs(seqs, like(a.pg), n_pages, positions, &a.sq))) return st;
    if (positions == 0) return ok();
    if (positions * (a.pg.d / 16) / 256 >= kMaxGrid) return fail(HR_EUNSUPPORTED, "too many positions for one launch");
    int64_t cb, rb;
    if ((st = check_ptr(pool, "pool", 16)) || (st = check_rows(c, "c", c_stride, 0, positions, 1, a.pg.d, dtype, &cb)) ||
        (st = check_rows(rope, "rope", rope_stride, 0, positions, 1, hr::kRope, dtype, &rb)))
        return st;
    // c and rope may be columns of one matrix
    Range r[] = {{"c", c, cb, true},
                 {"rope", beside(c, a.pg.d, rope, hr::kRope, c_stride, rope_stride, dtype) ? nullptr : rope, rb, true},
                 {"pool", pool, size_of(n_pages, a.pg.page_bytes), false},
                 {"table", seqs->table, seqs->rows * seqs->max_pages * 4, false},
                 {"lens", seqs->lens, seqs->rows * 4, false},
                 {"cu_q", seqs->cu_q, (seqs->rows + 1) * 4, false}};
    if ((st = check_overlap(r, 6))) return st;
    r[0].p = nullptr;
    r[1].p = rope;
    if ((st = check_overlap(r, 6))) return st;
    a.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
    a.c_out = c;
    a.rope_out = rope;
    a.c_st = c_stride;
    a.r_st = rope_stride;
    a.norm = static_cast<float>(1.0 / sqrt(static_cast<double>(a.pg.d)));
    a.rotate = rotate != 0;
    return launched(hr::launch_latent_read(a, dtype == HR_BF16, stream));
}

int hr_latent_attention_work(int dtype, int64_t tokens, int32_t heads, const hr_latent_spec* spec, int64_t rows, int64_t max_q,
                             int64_t* bytes) {
    hr::LatentPage pg;
    int st = check_latent(spec, &pg);
    if (st) return st;
    if (!bytes) return fail(HR_EINVAL, "bytes is NULL");
    if ((st = check_tokens(dtype, tokens)) || (st = check_heads(tokens, heads, max_q))) return st;
    if (rows < 0 || rows > kMaxCount) return fail(HR_EINVAL, "rows = %lld must be in 0..2^30", (long long)rows);
    *bytes = 0;
    if (tokens == 0) return ok();
    hr::LatentAttnKey key;
    attn_key(pg, dtype, tokens, heads, rows, max_q, &key);
    int workers;
    if ((st = attn_work(key, rows, tokens * heads, &workers, bytes))) return st;
    return ok();
}

int hr_latent_attention(const void* q, int64_t q_stride_token, int64_t q_stride_head, const void* q_rope,
                        int64_t q_rope_stride_token, int64_t q_rope_stride_head, int dtype, int64_t tokens, int32_t heads,
                        const void* pool, int64_t n_pages, const hr_latent_spec* spec, const hr_cache_seqs* seqs, float scale,
                        int causal, int rotate, void* out, int64_t out_stride_token, int64_t out_stride_head, float* lse,
                        int64_t max_q, void* work, int64_t work_bytes, void* stream) {
    hr::LatentAttnArgs a{};
    int st = check_latent(spec, &a.pg);
    if (st) return st;
    if ((st = check_tokens(dtype, tokens)) || (st = check_heads(tokens, heads, max_q)) ||
        (st = check_seqs(seqs, like(a.pg), n_pages, tokens, &a.sq)) || (st = check_reach(seqs, a.pg.page)) ||
        (st = check_scale(scale, false)))
        return st;
    if (tokens == 0) return ok();
    int64_t qb, rb, ob;
    if ((st = check_rows(q, "q", q_stride_token, q_stride_head, tokens, heads, a.pg.d, dtype, &qb)) ||
        (st = check_rows(q_rope, "q_rope", q_rope_stride_token, q_rope_stride_head, tokens, heads, hr::kRope, dtype, &rb)) ||
        (st = check_rows(out, "out", out_stride_token, out_stride_head, tokens, heads, a.pg.d, dtype, &ob)) ||
        (st = check_distinct("out", out_stride_token, out_stride_head, tokens, heads, a.pg.d)) ||
        (st = check_ptr(pool, "pool", 16)) || (lse && (st = check_ptr(lse, "lse", 4))))
        return st;
    hr::LatentAttnKey key;
    attn_key(a.pg, dtype, tokens, heads, seqs->rows, max_q, &key);
    int workers;
    int64_t need;
    if ((st = attn_work(key, seqs->rows, tokens * heads, &workers, &need))) return st;
    if ((st = check_ptr(work, "work", 16))) return st;
    if (work_bytes < need)
        return fail(HR_EINVAL, "work_bytes = %lld: %lld are needed", (long long)work_bytes, (long long)need);
    // out may share memory with q or q_rope (be q itself, or lie beside q_rope in
    // one tensor): both are read whole before out is written
    const Range r[] = {{"out", out, ob, true},
                       {"lse", lse, lse ? tokens * heads * 4 : 0, true},
                       {"work", work, need, true},
                       {"pool", pool, size_of(n_pages, a.pg.page_bytes), false},
                       {"table", seqs->table, seqs->rows * seqs->max_pages * 4, false},
                       {"lens", seqs->lens, seqs->rows * 4, false},
                       {"cu_q", seqs->cu_q, (seqs->rows + 1) * 4, false}};
    const Range w[] = {{"work", work, need, true},
                       {"lse", lse, lse ? tokens * heads * 4 : 0, true},
                       {"q", q, qb, false},
                       {"q_rope", q_rope, rb, false}};
    if ((st = check_overlap(r, 7)) || (st = check_overlap(w, 4))) return st;
    a.q = q;
    a.q_rope = q_rope;
    a.out = out;
    a.lse = lse;
    a.pool = static_cast<const uint8_t*>(pool);
    a.work = static_cast<uint8_t*>(work);
    a.q_st = q_stride_token;
    a.q_sh = q_stride_head;
    a.r_st = q_rope_stride_token;
    a.r_sh = q_rope_stride_head;
    a.o_st = out_stride_token;
    a.o_sh = out_stride_head;
    a.scale = scale;
    a.norm = static_cast<float>(1.0 / sqrt(static_cast<double>(a.pg.d)));
    a.heads = heads;
    a.causal = causal != 0;
    a.rotate = rotate != 0;
    a.workers = workers;
    return launched(hr::launch_latent_attn(key, a, stream));
}

int hr_latent_prompt_attention(const void* q, int64_t q_stride_token, int64_t q_stride_head, const void* k,
                               int64_t k_stride_token, int64_t k_stride_head, const void* v, int64_t v_stride_token,
                               int64_t v_stride_head, const void* rope, int64_t rope_stride, int dtype, int64_t tokens,
                               int64_t positions, int32_t heads, int32_t nope, const int32_t* cu_q, const int32_t* cu_k,
                               int64_t rows, float scale, int causal, void* out, int64_t out_stride_token,
                               int64_t out_stride_head, float* lse, void* stream) {
    int st;
    if ((st = check_tokens(dtype, tokens)) || (st = check_heads(tokens, heads, 0))) return st;
    if (dtype != HR_BF16) return fail(HR_EUNSUPPORTED, "prompts over expanded keys take HR_BF16 only");
    if (positions < 0 || positions > kMaxCount)
        return fail(HR_EINVAL, "positions = %lld must be in 0..2^30", (long long)positions);
    if (nope <= 0) return fail(HR_EINVAL, "nope = %d must be positive", nope);
    if (nope != 64 && nope != 128) return fail(HR_EUNSUPPORTED, "nope = %d: 64 and 128 are implemented", nope);
    if (rows < 0 || rows > kMaxCount) return fail(HR_EINVAL, "rows = %lld must be in 0..2^30", (long long)rows);
    if (rows == 0 && (tokens > 0 || positions > 0))
        return fail(HR_EINVAL, "%lld tokens and %lld positions of no rows", (long long)tokens, (long long)positions);
    if ((st = check_scale(scale, true))) return st;
    if (tokens == 0) return ok();
    int64_t qb, kb = 0, vb = 0, rb = 0, ob;
    if ((st = check_ptr(cu_q, "cu_q", 4)) || (st = check_ptr(cu_k, "cu_k", 4)) ||
        (st = check_rows(q, "q", q_stride_token, q_stride_head, tokens, heads, nope + hr::kRope, dtype, &qb)) ||
        (st = check_rows(out, "out", out_stride_token, out_stride_head, tokens, heads, nope, dtype, &ob)) ||
        (st = check_distinct("out", out_stride_token, out_stride_head, tokens, heads, nope)) || (lse && (st = check_ptr(lse, "lse", 4))))
        return st;
    if (positions > 0 && ((st = check_rows(k, "k", k_stride_token, k_stride_head, positions, heads, nope, dtype, &kb)) ||
                          (st = check_rows(v, "v", v_stride_token, v_stride_head, positions, heads, nope, dtype, &vb)) ||
                          (st = check_rows(rope, "rope", rope_stride, 0, positions, 1, hr::kRope, dtype, &rb))))
        return st;
    const int64_t blocks = tokens / 128 + rows;
    if (size_of(blocks, heads) >= kMaxGrid) return fail(HR_EUNSUPPORTED, "too many rows, tokens and heads for one launch");
    const Range r[] = {{"out", out, ob, true},
                       {"lse", lse, lse ? tokens * heads * 4 : 0, true},
                       {"q", q, qb, false},
                       {"k", k, kb, false},
                       {"v", v, vb, false},
                       {"rope", rope, rb, false},
                       {"cu_q", cu_q, (rows + 1) * 4, false},
                       {"cu_k", cu_k, (rows + 1) * 4, false}};
    if ((st = check_overlap(r, 8))) return st;
    hr::LatentPromptArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.rope = static_cast<const uint16_t*>(rope);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q_st = q_stride_token;
    a.q_sh = q_stride_head;
    a.k_st = k_stride_token;
    a.k_sh = k_stride_head;
    a.v_st = v_stride_token;
    a.v_sh = v_stride_head;
    a.r_st = rope_stride;
    a.o_st = out_stride_token;
    a.o_sh = out_stride_head;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.tokens = static_cast<int32_t>(tokens);
    a.positions = static_cast<int32_t>(positions);
    a.rows = static_cast<int32_t>(rows);
    a.heads = heads;
    a.nope = nope;
    a.scale = scale > 0.0f ? scale : static_cast<float>(1.0 / sqrt(static_cast<double>(nope + hr::kRope)));
    a.causal = causal != 0;
    return launched(hr::launch_latent_prompt(a, stream));
}

int hr_latent_update(void* pool, int64_t layers, int64_t n_pages, const hr_latent_spec* spec, const int32_t* table,
                     const int32_t* lens, int64_t rows, int64_t max_pages, const int32_t* parents, const int32_t* grow,
                     int64_t new_rows, int32_t* new_table, int32_t* new_lens, int32_t* refs, int32_t* status, void* work,
                     int64_t work_bytes, void* stream) {
    hr::LatentPage pg;
    int st = check_latent(spec, &pg);
    if (st) return st;
    return hr::cache_update(pool, layers, n_pages, like(pg), table, lens, rows, max_pages, parents, grow, new_rows, new_table, new_lens,
                            refs, status, work, work_bytes, stream);
}

int hr_latent_compact(void* pool, int64_t layers, int64_t n_pages, const hr_latent_spec* spec, const int32_t* table,
                      const int32_t* lens, int64_t rows, int64_t max_pages, void* into, int64_t into_pages, int32_t* new_table,
                      int32_t* refs, int32_t* status, void* work, int64_t work_bytes, void* stream) {
    hr::LatentPage pg;
    int st = check_latent(spec, &pg);
    if (st) return st;
    return hr::cache_compact(pool, layers, n_pages, like(pg), table, lens, rows, max_pages, into, into_pages, new_table, refs, status,
                             work, work_bytes, stream);
}

}  // extern "C"
