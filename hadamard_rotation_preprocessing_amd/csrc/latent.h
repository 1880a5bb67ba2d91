// Argument structs shared by the latent cache's host layer (latent_api.cpp) and
// its kernels (latent_pages.hip, latent_attn_*.hip, latent_prompt.hip).  Plain
// data only.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "cache.h"

namespace hr {

constexpr int kRope = 64;      // elements of a rotary key

// A page's layout, resolved.
struct LatentPage {
    int32_t d, ng;             // latent dimension, groups per vector
    int32_t page, logp;        // positions of a page
    int32_t sym, sf32;         // symmetric codes; float32 scales (else bfloat16)
    int32_t scales, zeros, rope;   // offsets of the sections (codes: 0)
    int64_t page_bytes;
};

struct LatentPagesArgs {       // append and read
    uint8_t* pool;
    const void* c_in;          // append
    const void* rope_in;
    void* c_out;               // read
    void* rope_out;
    int64_t c_st, r_st;        // element strides
    LatentPage pg;
    CacheSeqs sq;
    float norm;                // 1 / sqrt(d)
    int32_t rotate;
    int32_t units;             // append: blocks of positions (an upper bound)
};

struct LatentAttnArgs {
    const void* q;
    const void* q_rope;
    void* out;
    float* lse;                // nullable
    const uint8_t* pool;
    uint8_t* work;
    int64_t q_st, q_sh, r_st, r_sh, o_st, o_sh;   // element strides
    LatentPage pg;
    CacheSeqs sq;
    float scale;               // of the scores
    float norm;                // 1 / sqrt(d) (rotate)
    int32_t heads;
    int32_t causal, rotate;
    int32_t workers;           // workgroups
};

// Which attention kernel a call takes: 16 rt wr query rows of a sequence to a
// workgroup, in waves of 16 rt.
struct LatentAttnKey {
    int32_t d, ng, sf32;
    int32_t wide;              // float32 activations
    int32_t rt, wr;
};

struct LatentPromptArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* rope;
    uint16_t* out;
    float* lse;                // nullable
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, r_st, o_st, o_sh;   // element strides
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t tokens, positions, rows, heads, nope;
    float scale;
    int32_t causal;
};

// Launchers: 0 or a hipError_t.
int launch_latent_append(const LatentPagesArgs& a, int bf16, void* stream);
int launch_latent_read(const LatentPagesArgs& a, int bf16, void* stream);
int launch_latent_attn(const LatentAttnKey& k, const LatentAttnArgs& a, void* stream);
int launch_latent_prompt(const LatentPromptArgs& a, void* stream);
// workgroups that an attention kernel keeps in flight on the current device
int latent_attn_workers(const LatentAttnKey& k, int* workers);

// The scratch of an attention over `seqs` sequences with `rows` query rows: the
// numbering of the sequences' work, and where each workgroup begins; the queries as operands, with 16 bytes more for
// each row; the sums of each row; and two partial sums for each workgroup.
constexpr int64_t latent_first_bytes(int64_t seqs) { return ((seqs + 1) * 8 + 15) / 16 * 16; }
constexpr int64_t latent_start_bytes(int workers) { return (int64_t{workers} * 4 + 4 + 15) / 16 * 16; }
constexpr int64_t latent_work_bytes(const LatentAttnKey& k, int64_t seqs, int64_t rows, int workers) {
    const int terms = k.wide ? 2 : 1, rope_terms = k.wide ? 3 : 1;
    return latent_first_bytes(seqs) + latent_start_bytes(workers) + rows * (16 + 2 * (terms * k.d + rope_terms * kRope) + 4 * (k.d + 4)) +
           int64_t{workers} * 2 * (16 * k.rt * k.wr) * (k.d + 4) * 4;
}

}  // namespace hr
