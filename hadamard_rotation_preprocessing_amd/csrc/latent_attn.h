// Latent attention over the paged 4-bit cache (hr_latent_attention): kernels for
// one latent dimension and number of groups, instantiated by latent_attn_*.hip.
//
// Mathematics.  A latent c = s (k - z) (codes k, zero point z, scale s of its
// group) is the key and the value of all heads.  Codes less zero points are small
// integers, float16 exactly, so scores are matrix products over them, one for each
// group, with float32 scales on the results, and one over the rotary keys in
// bfloat16.  For the values the scales go into the probabilities, for each group
// apart: P_g = exp(w - m) s_g, and O_g = P_g (k - z) is a matrix product over the
// same integers.
//   The softmax is taken in one pass.  Its reference m only keeps exponentials in
// float32's range, so it moves when one passes 2^kFar.  P_g goes into the product
// as float16 in a power of two of its row and group, which moves when a value would
// pass 2^kTop: it follows the largest exp(w - m) s_g that the row has seen, so what
// a row does not see has no part in it, and scales of any size keep their bits.
//
// Layout.  A workgroup takes M = 16 RT WR query rows (new tokens x heads) of a
// sequence, and 64 keys a step.  Scores are formed transposed, S^T = C Q^T, by WR x
// 4 waves: a wave takes 16 keys (A operand: packed codes made into float16 in its
// registers, straight from memory) and 16 RT rows (B operand, in registers
// throughout).  The operands go to LDS too, where the second product finds them:
// O^T = C^T P^T, for which every wave takes all M rows and its share of the
// dimensions, so that the sums are spread over the workgroup.  C^T comes out of LDS
// by transposing reads (ds_read_b64_tr_b16), P^T by way of LDS from the waves that
// made it, its 32 keys of a matrix step in the order 4 g + i, 16 + 4 g + i of the
// registers of two score tiles.
//   Elements of eight of a vector stand in the order 0 4 1 5 2 6 3 7 throughout:
// that of the nibbles of a word under two masks.
//
// Split.  latent_query rotates the queries, turns them into operands in the scratch
// and numbers the work: a unit is a block of M rows of a sequence, an item 64 keys of
// it, and every workgroup takes an equal, contiguous run of all items.  A row's sums
// are left in the scratch, for units that are cut in parts, and latent_finish joins
// the parts in key order, divides, rotates back and rounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "cache_vectors.h"
#include "latent.h"
#include "plan.h"

namespace hr {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfloat8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLow = -3.0e38f;      // reference of a row that has seen nothing
constexpr float kFar = 0x1p20f;       // largest exponential before the reference moves
constexpr float kTop = 0x1p15f;       // largest probability in its unit (float16 ends at 65504)
constexpr int kSet = 8;               // log2 of the largest one when a unit is set
constexpr int kUnit = 126;            // units are 2^-kUnit .. 2^kUnit
constexpr int kQTop = 14;             // a query's largest element is below 2^kQTop in float16

__device__ __forceinline__ float4v mfma_f16(uint4v a, uint4v b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ float4v mfma_bf16(uint4v a, uint4v b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bfloat8, a), __builtin_bit_cast(bfloat8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pk_sub(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, a) - __builtin_bit_cast(half2v, b));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    half2v h;
    h.x = static_cast<_Float16>(a);
    h.y = static_cast<_Float16>(b);
    return __builtin_bit_cast(uint32_t, h);
}
// two floats as pairs of float16: hi, and what it loses of them
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
    asm("" : "+v"(a), "+v"(b));   // (as values: no contraction with the products that made them)
    hi = pack_f16(a, b);
    const half2v h = __builtin_bit_cast(half2v, hi);
    lo = pack_f16(a - static_cast<float>(h.x), b - static_cast<float>(h.y));
}
// bf16 (finite or not) from float32, nearest even, NaN kept
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
// 2^e of an integer e in -126 .. 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <int D_, int NG_, bool WIDE_, int RT_, int WR_>
struct Cfg {
    static constexpr int D = D_, NG = NG_, RT = RT_, WR = WR_;
    static constexpr bool WIDE = WIDE_;
    static constexpr int WK = 4, WAVES = WR * WK, THREADS = 64 * WAVES;
    static constexpr int KEYS = 16 * WK;           // of a step
    static constexpr int TILES = RT * WR, M = 16 * TILES;
    static constexpr int T = WIDE ? 2 : 1;         // float16 terms of a query and a probability
    static constexpr int TR = WIDE ? 3 : 1;        // bfloat16 terms of a rotary query
    static constexpr int KS = D / 32, KG = KS / NG, G = D / NG;
    static constexpr int DW = D / WAVES, DT = DW / 16;   // dimensions of a wave in the second product
    static constexpr int VS = 2 * D + 32;          // bytes of a key's operands in LDS
    static constexpr int PS = 2 * KEYS + 16;       // bytes of a row's probabilities
    static constexpr int QS = 2 * (T * D + TR * kRope);   // bytes of a row's query in the scratch
    static constexpr int RS = D + 4;               // floats of a row's sums
    static constexpr int WGS = WR == 1 ? 2 : 1;    // workgroups of a CU
};

// A sequence of the call, clamped so that nothing leaves its buffer.
struct Seq {
    int start, n, len;
};
__device__ __forceinline__ int cu_at(const CacheSeqs& s, int b) {
    const int c = s.cu ? s.cu[b] : b * s.per;
    return min(max(c, 0), s.tokens);
}
__device__ __forceinline__ Seq seq_at(const CacheSeqs& s, int logp, int b) {
    Seq r;
    r.start = cu_at(s, b);
    r.n = max(cu_at(s, b + 1) - r.start, 0);
    r.len = static_cast<int>(min(static_cast<int64_t>(max(s.lens[b], 0)), static_cast<int64_t>(s.max_pages) << logp));
    return r;
}
// items of a unit of a sequence, and its units
template <class C>
__device__ __forceinline__ int items_of(const Seq& s) { return static_cast<int>((static_cast<int64_t>(s.len) + C::KEYS - 1) / C::KEYS); }
template <class C>
__device__ __forceinline__ int units_of(const Seq& s, int heads) {
    return static_cast<int>((static_cast<int64_t>(s.n) * heads + C::M - 1) / C::M);
}
// the first item of workgroup w of n, of `total`
__device__ __forceinline__ int64_t begin_of(int64_t total, int w, int n) { return total * w / n; }

// How many workgroups take part: not so many that joining their parts costs more
// than it saves.
constexpr int kLeast = 4;              // items of a workgroup
__device__ __forceinline__ int used_workers(int64_t total, int workers) {
    const int64_t n = (total + kLeast - 1) / kLeast;
    return static_cast<int>(n < workers ? (n > 1 ? n : 1) : workers);
}

// 16 dimensions of four keys out of LDS: lane m of 16 gives the address of its four
// dimensions 4 (m % 4) of key m / 4, and gets dimension m of the four keys.
__device__ __forceinline__ uint2v transposed(const uint8_t* p) {
    typedef short4v __attribute__((address_space(3)))* Lds;
    return __builtin_bit_cast(uint2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
}

// The scratch.
template <class C>
struct Work {
    int64_t* first;      // [rows + 1]: items before those of a sequence
    float* factor;       // [query rows]: of a score's products with codes
    uint8_t* query;
    float* whole;        // [query rows][RS]: sums, the reference, and the sum of exponentials
    float* part;         // [workers][2][M][RS]
    __device__ __forceinline__ Work(const LatentAttnArgs& a) {
        const int64_t rows = static_cast<int64_t>(a.sq.tokens) * a.heads;
        first = reinterpret_cast<int64_t*>(a.work);
        uint8_t* p = a.work + latent_first_bytes(a.sq.rows);
        factor = reinterpret_cast<float*>(p);
        query = p + rows * 16;
        whole = reinterpret_cast<float*>(query + rows * C::QS);
        part = whole + rows * C::RS;
    }
};

// ---------------------------------------------------------------------------
// queries

template <class C, class In>
__global__ void __launch_bounds__(256) latent_query(const LatentAttnArgs a) {
    constexpr int D = C::D, LPV = D / 16, R = kRope / LPV;
    const Work<C> work(a);
    if (blockIdx.x == 0) {     // the numbering of items
        __shared__ int64_t sums[256];
        int64_t before = 0;
        for (int r0 = 0; r0 < a.sq.rows; r0 += 256) {
            int64_t v = 0;
            if (r0 + static_cast<int>(threadIdx.x) < a.sq.rows) {
                const Seq s = seq_at(a.sq, a.pg.logp, r0 + threadIdx.x);
                v = static_cast<int64_t>(items_of<C>(s)) * units_of<C>(s, a.heads);
            }
            sums[threadIdx.x] = v;
            __syncthreads();
            for (int x = 1; x < 256; x *= 2) {
                const int64_t y = static_cast<int>(threadIdx.x) >= x ? sums[threadIdx.x - x] : 0;
                __syncthreads();
                sums[threadIdx.x] += y;
                __syncthreads();
            }
            if (r0 + static_cast<int>(threadIdx.x) < a.sq.rows) work.first[r0 + threadIdx.x + 1] = before + sums[threadIdx.x];
            before += sums[255];
            __syncthreads();
        }
        if (threadIdx.x == 0) work.first[0] = 0;
    }
    const int64_t row = (int64_t{blockIdx.x} * 256 + threadIdx.x) / LPV, total = static_cast<int64_t>(a.sq.tokens) * a.heads;
    const int lane = threadIdx.x & 63, e = lane % LPV;
    const uint32_t at = static_cast<uint32_t>(min(row, total - 1)), t = at / a.heads, h = at % a.heads;
    float x[16];
    load16(static_cast<const In*>(a.q) + t * a.q_st + h * a.q_sh + 16 * e, x);
    const In* rp = static_cast<const In*>(a.q_rope) + t * a.r_st + h * a.r_sh + R * e;
    if (a.rotate) hadamard<D>(x, lane, a.norm);
    float top = fabsf(x[0]);
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
    top = over_lanes<LPV>(top, [](float p, float q) { return fmaxf(p, q); });
    int unit = 0;
    if (top > 0.0f && top < __builtin_inff()) unit = min(max(kQTop - 1 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), -110), 110);
    if (row >= total) return;
    uint8_t* to = work.query + row * C::QS;
#pragma unroll
    for (int j = 0; j < 16; j += 8) {
        uint4v hi, lo;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t p, q;
            split_f16(__builtin_ldexpf(x[j + k], unit), __builtin_ldexpf(x[j + k + 4], unit), p, q);
            hi[k] = p;
            lo[k] = q;
        }
        reinterpret_cast<uint4v*>(to)[(16 * e + j) / 8] = hi;
        if constexpr (C::WIDE) reinterpret_cast<uint4v*>(to + 2 * D)[(16 * e + j) / 8] = lo;
    }
    uint16_t* rope = reinterpret_cast<uint16_t*>(to + 2 * C::T * D) + R * e;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if constexpr (C::WIDE) {
            float v = rp[i];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t b = to_bf16(v);
                rope[k * kRope + i] = static_cast<uint16_t>(b);
                v -= bf2f(b);
            }
        } else {
            rope[i] = rp[i];
        }
    }
    if (e == 0) work.factor[row] = __builtin_ldexpf(a.scale * kLog2e, -unit);
}

// ---------------------------------------------------------------------------
// the sums

// What a wave holds of 16 keys before it works on them.
template <class C>
struct Raw {
    uint4v codes[C::KS / 4];   // of key lane & 15: the lane group's quarter of every group
    uint4v rope[2];
    uint32_t scales[4 * C::NG];   // of keys 4 g .. 4 g + 3 (two to a word if bfloat16)
    uint32_t zeros;            // of key lane & 15, a nibble for each group
};

template <class C>
__device__ __forceinline__ void load_keys(const LatentAttnArgs& a, int page, int t0, Raw<C>& w) {
    constexpr int D = C::D, NG = C::NG;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const uint8_t* base = a.pool + page * a.pg.page_bytes;
    const int off = t0 & (a.pg.page - 1);
    const uint8_t* codes = base + (off + m) * (D / 2) + g * (C::G / 8);
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int i = 0; i < C::KG / 4; ++i) w.codes[q * (C::KG / 4) + i] = *reinterpret_cast<const uint4v*>(codes + q * (C::G / 2) + 16 * i);
#pragma unroll
    for (int i = 0; i < 2; ++i) w.rope[i] = *reinterpret_cast<const uint4v*>(base + a.pg.rope + (off + m) * (2 * kRope) + 64 * i + 16 * g);
    if (a.pg.sf32) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(base + a.pg.scales) + (off + 4 * g) * NG;
#pragma unroll
        for (int i = 0; i < 4 * NG; ++i) w.scales[i] = s[i];
    } else {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(base + a.pg.scales) + (off + 4 * g) * NG / 2;
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) w.scales[i] = s[i];
    }
    w.zeros = 0;
    if (!a.pg.sym) {
        const uint8_t* z = base + a.pg.zeros + (off + m) * NG / 2;
        if constexpr (NG == 4) w.zeros = *reinterpret_cast<const uint16_t*>(z);
        else if constexpr (NG == 2) w.zeros = *z;
        else w.zeros = *z >> (4 * (m & 1));
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::WGS * C::WAVES / 4) latent_sums(const LatentAttnArgs a) {
    constexpr int D = C::D, NG = C::NG, RT = C::RT, T = C::T, M = C::M;
    __shared__ __attribute__((aligned(16))) uint8_t values[C::KEYS * C::VS];
    __shared__ __attribute__((aligned(16))) uint8_t probs[T * NG * M * C::PS];
    __shared__ float top[C::WK * M];           // of a wave's keys, for each row
    __shared__ float top_g[C::WK * M * NG];
    __shared__ float shift[M * NG];            // what a row's sums are multiplied by
    __shared__ int units[M * NG];              // log2 of a row's units
    __shared__ int moved;
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wk = wave % C::WK, wr = wave / C::WK;
    const Work<C> work(a);
    const LatentPage& pg = a.pg;
    const int64_t total = work.first[a.sq.rows];
    const int used = used_workers(total, gridDim.x);
    if (static_cast<int>(blockIdx.x) >= used) return;
    const int64_t end = begin_of(total, blockIdx.x + 1, used);
    int64_t item = begin_of(total, blockIdx.x, used);
    if (tid == 0) moved = 0;
    const float f0 = a.scale * kLog2e;
    while (item < end) {
        int lo = 0, hi = a.sq.rows - 1;        // the last sequence that begins at or before this item
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (work.first[mid] <= item) lo = mid;
            else hi = mid - 1;
        }
        const Seq s = seq_at(a.sq, pg.logp, lo);
        const int per = items_of<C>(s);
        const int64_t in_seq = item - work.first[lo];
        const int rb = static_cast<int>(in_seq / per), k0 = static_cast<int>(in_seq % per);
        const int k1 = static_cast<int>(min(static_cast<int64_t>(per), k0 + end - item));
        item += k1 - k0;
        const int32_t* table = a.sq.table + static_cast<int64_t>(lo) * a.sq.max_pages;
        const int rows = s.n * a.heads, r0 = rb * M, first = s.len - s.n;
        const int64_t row_at = static_cast<int64_t>(s.start) * a.heads;

        // the wave's rows as B operands
        uint4v query[RT][T][C::KS], rope[RT][C::TR][2];
        float factor[RT];
        int pos[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = min(r0 + (wr * RT + rt) * 16 + m, rows - 1);
            const uint8_t* q = work.query + (row_at + r) * C::QS;
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int ks = 0; ks < C::KS; ++ks)
                    query[rt][t][ks] = *reinterpret_cast<const uint4v*>(q + 2 * (t * D + (ks / C::KG) * C::G + g * (C::G / 4) + 8 * (ks % C::KG)));
#pragma unroll
            for (int t = 0; t < C::TR; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) rope[rt][t][i] = *reinterpret_cast<const uint4v*>(q + 2 * (T * D + t * kRope + 32 * i + 8 * g));
            factor[rt] = work.factor[row_at + r];
            pos[rt] = a.causal ? min(first + r / a.heads, s.len - 1) : s.len - 1;   // the last key that the row sees
        }
        const int last_row = min(r0 + M, rows) - 1;
        const int limit = a.causal ? min(max(first + last_row / a.heads + 1, 0), s.len) : s.len;
        // the first key that not all of the wave's rows see
        const int all = a.causal ? min(first + min(r0 + wr * 16 * RT, rows - 1) / a.heads + 1, s.len) : s.len;

        float4v acc[C::TILES][C::DT];
#pragma unroll
        for (int x = 0; x < C::TILES; ++x)
#pragma unroll
            for (int d = 0; d < C::DT; ++d) acc[x][d] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        float ref[RT], sum[RT];
        int unit[RT][NG];                      // log2
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            ref[rt] = kLow;
            sum[rt] = 0.0f;
#pragma unroll
            for (int q = 0; q < NG; ++q) unit[rt][q] = -kUnit;
        }

        const auto page_at = [&](int t0) {     // of the wave's keys from t0; -1: none are there
            if (t0 >= limit) return -1;
            const int p = table[t0 >> pg.logp];
            return p >= 0 && p < a.sq.n_pages ? p : -1;
        };
        Raw<C> raw;
        const int end_key = min(k1 * C::KEYS, limit);
        int t0 = k0 * C::KEYS + 16 * wk;
        int page = __builtin_amdgcn_readfirstlane(page_at(t0)), next = __builtin_amdgcn_readfirstlane(page_at(t0 + C::KEYS));
        if (page >= 0) load_keys<C>(a, page, t0, raw);
        __syncthreads();

        for (; t0 - 16 * wk < end_key; t0 += C::KEYS) {
            // scores, and the operands to LDS
            float4v w[RT], wrope[RT];
            float scale[4][NG];
            const bool here = page >= 0;
            if (here) {
                const uint32_t f0c = 0x64006400u ^ (pg.sym ? 0x00080008u : 0u), f1c = 0x54005400u ^ (pg.sym ? 0x00800080u : 0u);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        const int x = i * NG + q;
                        scale[i][q] = pg.sf32 ? __uint_as_float(raw.scales[x])
                                              : __uint_as_float((x & 1) ? raw.scales[x / 2] & 0xFFFF0000u : raw.scales[x / 2] << 16);
                    }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    wrope[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int t = C::TR - 1; t >= 0; --t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) wrope[rt] = mfma_bf16(raw.rope[i], rope[rt][t][i], wrope[rt]);
                }
                uint8_t* to = values + (16 * wk + m) * C::VS + g * (C::G / 4) * 2;
#pragma unroll
                for (int q = 0; q < NG; ++q) {
                    const uint32_t z = pg.sym ? 8u : (raw.zeros >> (4 * q)) & 15u;
                    const uint32_t z0 = 0x64006400u + z * 0x00010001u, z1 = 0x54005400u + z * 0x00100010u;
                    float4v c[RT];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) c[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < C::KG; ++i) {
                        const int ks = q * C::KG + i;
                        uint32_t x = raw.codes[ks / 4][ks % 4];
                        uint4v k;
                        k.x = pk_sub((x & 0x000F000Fu) ^ f0c, z0);
                        k.y = pk_sub((x & 0x00F000F0u) ^ f1c, z1);
                        x >>= 8;
                        k.z = pk_sub((x & 0x000F000Fu) ^ f0c, z0);
                        k.w = pk_sub((x & 0x00F000F0u) ^ f1c, z1);
                        // (waves of the same keys write half of the operands each)
                        if (C::WR == 1 || ks * C::WR / C::KS == wr) *reinterpret_cast<uint4v*>(to + 2 * (q * C::G + 8 * i)) = k;
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            if constexpr (C::WIDE) c[rt] = mfma_f16(k, query[rt][T - 1][ks], c[rt]);
                            c[rt] = mfma_f16(k, query[rt][0][ks], c[rt]);
                        }
                    }
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[rt][i] = q ? __builtin_fmaf(c[rt][i], scale[i][q], w[rt][i]) : c[rt][i] * scale[i][0];
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[rt][i] = __builtin_fmaf(w[rt][i], factor[rt], wrope[rt][i] * f0);
            } else {
                // keys that are not there: no probability, and finite operands
                uint8_t* to = values + (16 * wk + m) * C::VS + g * (D / 4) * 2;
#pragma unroll
                for (int ks = 0; ks < C::KS; ++ks)
                    if (C::WR == 1 || ks * C::WR / C::KS == wr) *reinterpret_cast<uint4v*>(to + 16 * ks) = uint4v{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int q = 0; q < NG; ++q) scale[i][q] = 0.0f;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[rt][i] = -__builtin_inff();
            }
            const int key = t0 + 4 * g;
            const bool full = here && t0 + 16 <= all;
            if (!full) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key + i > pos[rt]) w[rt][i] = -__builtin_inff();
            }
            // the next keys
            page = next;
            next = __builtin_amdgcn_readfirstlane(page_at(t0 + 2 * C::KEYS));
            if (page >= 0) load_keys<C>(a, page, t0 + C::KEYS, raw);

            // probabilities in their units, to LDS
            float more[RT];
            bool far = false;
            const auto put = [&]() {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    float p[4];
                    more[rt] = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[i] = __builtin_amdgcn_exp2f(w[rt][i] - ref[rt]);
                        more[rt] += p[i];
                        far = far || !(p[i] <= kFar);
                    }
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        float x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[i] = __builtin_ldexpf(p[i] * scale[i][q], -unit[rt][q]);
                            // (an unseen key's scale may be anything)
                            if (!full && key + i > pos[rt]) x[i] = 0.0f;
                            far = far || !(x[i] <= kTop);
                        }
                        // keys 16 wk + 4 g + i stand at 8 g + 4 (wk & 1) + i of their 32
                        uint8_t* to = probs + (q * M + (wr * RT + rt) * 16 + m) * C::PS + (wk / 2) * 64 + 16 * g + 8 * (wk & 1);
                        if constexpr (C::WIDE) {
                            uint2v hi, lost;
                            uint32_t h, l;
                            split_f16(x[0], x[1], h, l);
                            hi.x = h;
                            lost.x = l;
                            split_f16(x[2], x[3], h, l);
                            hi.y = h;
                            lost.y = l;
                            *reinterpret_cast<uint2v*>(to) = hi;
                            *reinterpret_cast<uint2v*>(to + NG * M * C::PS) = lost;
                        } else {
                            *reinterpret_cast<uint2v*>(to) = uint2v{pack_f16(x[0], x[1]), pack_f16(x[2], x[3])};
                        }
                    }
                }
            };
            put();
            if (__any(far) && lane == 0) moved = 1;
            __syncthreads();
            if (moved) {
                // references and units follow the largest of what the rows see
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    float x = fmaxf(fmaxf(w[rt][0], w[rt][1]), fmaxf(w[rt][2], w[rt][3]));
                    x = fmaxf(x, __shfl_xor(x, 16));
                    x = fmaxf(x, __shfl_xor(x, 32));
                    if (g == 0) top[wk * M + (wr * RT + rt) * 16 + m] = x;
                }
                __syncthreads();
                if (tid == 0) moved = 0;
                int fall[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const int r = (wr * RT + rt) * 16 + m;
                    const float x = fmaxf(fmaxf(top[r], top[M + r]), fmaxf(top[2 * M + r], top[3 * M + r]));
                    const float was = ref[rt];
                    // (a whole number, so that what follows from it is exact)
                    if (x < __builtin_inff()) ref[rt] = fmaxf(was, ceilf(x));
                    fall[rt] = static_cast<int>(fmaxf(was - ref[rt], -4000.0f));
                    sum[rt] = __builtin_ldexpf(sum[rt], fall[rt]);
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_exp2f(w[rt][i] - ref[rt]);
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        float y = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (full || key + i <= pos[rt]) y = fmaxf(y, p[i] * scale[i][q]);
                        y = fmaxf(y, __shfl_xor(y, 16));
                        y = fmaxf(y, __shfl_xor(y, 32));
                        if (g == 0) top_g[(wk * M + r) * NG + q] = y;
                    }
                }
                __syncthreads();
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const int r = (wr * RT + rt) * 16 + m;
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        float y = 0.0f;
#pragma unroll
                        for (int x = 0; x < C::WK; ++x) y = fmaxf(y, top_g[(x * M + r) * NG + q]);
                        const int old = unit[rt][q] + fall[rt];
                        const int now = max(old, (static_cast<int>(__float_as_uint(y) >> 23) & 255) - 127 - kSet);
                        unit[rt][q] = min(max(now, -kUnit), kUnit);
                        if (wk == 0 && g == 0) shift[r * NG + q] = __builtin_ldexpf(1.0f, max(old - unit[rt][q], -4000));
                    }
                }
                put();
                __syncthreads();
#pragma unroll
                for (int x = 0; x < C::TILES; ++x) {
                    const float f = shift[(16 * x + m) * NG + wave * C::DW / C::G];
#pragma unroll
                    for (int d = 0; d < C::DT; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[x][d][i] *= f;
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) sum[rt] += more[rt];

            // sums of the wave's dimensions over all rows
            const uint8_t* pr = probs + (wave * C::DW / C::G * M + m) * C::PS + 16 * g;
            const uint8_t* va = values + (4 * g + m / 4) * C::VS + (wave * C::DW + 4 * (m % 4)) * 2;
#pragma unroll
            for (int k = 0; k < C::KEYS / 32; ++k) {
                uint4v p[T][C::TILES];
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int x = 0; x < C::TILES; ++x) p[t][x] = *reinterpret_cast<const uint4v*>(pr + (t * NG * M + 16 * x) * C::PS + 64 * k);
#pragma unroll
                for (int d = 0; d < C::DT; ++d) {
                    const uint2v v0 = transposed(va + (32 * k) * C::VS + 32 * d), v1 = transposed(va + (32 * k + 16) * C::VS + 32 * d);
                    const uint4v v = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
                    for (int x = 0; x < C::TILES; ++x)
#pragma unroll
                        for (int t = T - 1; t >= 0; --t) acc[x][d] = mfma_f16(v, p[t][x], acc[x][d]);
                }
            }
            __syncthreads();
        }

        // the segment's sums: rows of the unit if it is whole, else one of the
        // workgroup's two parts
        const bool whole = k0 == 0 && k1 == per;
        float* out = whole ? work.whole + (row_at + r0) * C::RS
                           : work.part + (static_cast<int64_t>(blockIdx.x) * 2 + (k0 > 0 ? 0 : 1)) * M * C::RS;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = (wr * RT + rt) * 16 + m;
            float l = sum[rt];
            l += __shfl_xor(l, 16);
            l += __shfl_xor(l, 32);
            if (g == 0) {
                top[wk * M + r] = l;
                if (wk == 0) {
#pragma unroll
                    for (int q = 0; q < NG; ++q) units[r * NG + q] = unit[rt][q];
                    if (r0 + r < rows) out[static_cast<int64_t>(r) * C::RS + D] = ref[rt];
                }
            }
        }
        __syncthreads();
        if (tid < M && r0 + tid < rows)
            out[static_cast<int64_t>(tid) * C::RS + D + 1] = (top[tid] + top[M + tid]) + (top[2 * M + tid] + top[3 * M + tid]);
#pragma unroll
        for (int x = 0; x < C::TILES; ++x) {
            const int r = 16 * x + m, e = units[r * NG + wave * C::DW / C::G];
            if (r0 + r < rows)
#pragma unroll
                for (int d = 0; d < C::DT; ++d) {
                    float4v v = acc[x][d];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = __builtin_ldexpf(v[i], e);
                    *reinterpret_cast<float4v*>(out + static_cast<int64_t>(r) * C::RS + wave * C::DW + 16 * d + 4 * g) = v;
                }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// the results

// A workgroup takes one row: eight (or 16) groups of D / 16 lanes take its parts in
// turn, and the first of them adds what they have, in their order.
template <class C, class Out>
__global__ void __launch_bounds__(256) latent_finish(const LatentAttnArgs a, int workers) {
    constexpr int D = C::D, LPV = D / 16, GROUPS = 256 / LPV;
    __shared__ __attribute__((aligned(16))) float sums[GROUPS][D];
    __shared__ float refs[GROUPS], exps[GROUPS];
    const Work<C> work(a);
    const int group = threadIdx.x / LPV, e = threadIdx.x % LPV, lane = threadIdx.x & 63;
    const int64_t total = work.first[a.sq.rows];
    const int used = used_workers(total, workers);
    const int64_t rows = static_cast<int64_t>(a.sq.tokens) * a.heads;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int t = static_cast<int>(static_cast<uint32_t>(row) / a.heads), h = static_cast<int>(static_cast<uint32_t>(row) % a.heads);
        int lo = 0, hi = a.sq.rows - 1;            // the last sequence that begins at or before this token
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (cu_at(a.sq, mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        const Seq s = seq_at(a.sq, a.pg.logp, lo);
        const int per = items_of<C>(s);
        const int64_t r = row - static_cast<int64_t>(s.start) * a.heads;
        const int64_t u0 = work.first[lo] + r / C::M * per, u1 = u0 + per;
        const bool there = t >= s.start && t < s.start + s.n && per > 0;   // (else no workgroup had this row)
        float v[16] = {}, ref = kLow, l = 0.0f;
        const auto add = [&](const float* p) {
            const float pl = p[D + 1];
            if (!(pl == 0.0f)) {
                const float pr = p[D], now = fmaxf(ref, pr);
                const float f0 = __builtin_amdgcn_exp2f(ref - now), f1 = __builtin_amdgcn_exp2f(pr - now);
                l = l * f0 + pl * f1;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = v[i] * f0 + p[16 * e + i] * f1;
                ref = now;
            }
        };
        int groups = 1;
        if (there) {
            const int w0 = static_cast<int>(((u0 + 1) * used - 1) / total);
            if (begin_of(total, w0 + 1, used) >= u1) {
                if (group == 0) add(work.whole + row * C::RS);
            } else {
                groups = GROUPS;
                for (int w = w0 + group; w < used && begin_of(total, w, used) < u1; w += GROUPS) {
                    const int slot = begin_of(total, w, used) > u0 ? 0 : 1;
                    add(work.part + ((static_cast<int64_t>(w) * 2 + slot) * C::M + r % C::M) * C::RS);
                }
            }
        }
        if (groups > 1) {                          // (the same for the whole workgroup)
            __syncthreads();
            if (group > 0) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4v*>(&sums[group][16 * e + i]) = float4v{v[i], v[i + 1], v[i + 2], v[i + 3]};
                if (e == 0) {
                    refs[group] = ref;
                    exps[group] = l;
                }
            }
            __syncthreads();
            if (group == 0)
                for (int x = 1; x < GROUPS; ++x) {
                    if (exps[x] == 0.0f) continue;
                    const float now = fmaxf(ref, refs[x]);
                    const float f0 = __builtin_amdgcn_exp2f(ref - now), f1 = __builtin_amdgcn_exp2f(refs[x] - now);
                    l = l * f0 + exps[x] * f1;
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = v[i] * f0 + sums[x][16 * e + i] * f1;
                    ref = now;
                }
        }
        if (group > 0) continue;
        const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
        // back to the elements' own order
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i / 8 * 8 + (i % 2) * 4 + (i % 8) / 2] = l == 0.0f ? 0.0f : v[i] * inverse;
        if (a.rotate) hadamard<D>(y, lane, a.norm);
        Out* out = static_cast<Out*>(a.out) + t * a.o_st + h * a.o_sh + 16 * e;
#pragma unroll
        for (int i = 0; i < 16; i += 16 / sizeof(Out)) {
            uint4v x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(Out) == 2) x[j] = to_bf16(y[i + 2 * j]) | (to_bf16(y[i + 2 * j + 1]) << 16);
                else x[j] = __float_as_uint(y[i + j]);
            }
            *reinterpret_cast<uint4v*>(out + i) = x;
        }
        if (a.lse && e == 0) a.lse[row] = l == 0.0f ? -__builtin_inff() : (ref + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
}

template <class C>
int attn_launch(const LatentAttnArgs& a, hipStream_t s) {
    const int64_t rows = int64_t{a.sq.tokens} * a.heads, threads = rows * (C::D / 16);
    const dim3 query(static_cast<uint32_t>((threads + 255) / 256)), finish(static_cast<uint32_t>(rows < (1 << 20) ? rows : 1 << 20));
    if constexpr (C::WIDE) hipLaunchKernelGGL((latent_query<C, float>), query, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((latent_query<C, uint16_t>), query, dim3(256), 0, s, a);
    hipLaunchKernelGGL((latent_sums<C>), dim3(a.workers), dim3(C::THREADS), 0, s, a);
    if constexpr (C::WIDE) hipLaunchKernelGGL((latent_finish<C, float>), finish, dim3(256), 0, s, a, a.workers);
    else hipLaunchKernelGGL((latent_finish<C, uint16_t>), finish, dim3(256), 0, s, a, a.workers);
    return static_cast<int>(hipGetLastError());
}

// workgroups in flight on the current device, asked for once
template <class C>
int attn_workers(int* workers) {
    static std::atomic<int> known[kMaxDevices];
    int dev;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return static_cast<int>(e);
    int n = dev < kMaxDevices ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        int cus;
        e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
        if (e != hipSuccess) return static_cast<int>(e);
        n = C::WGS * cus;
        if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
    }
    *workers = n;
    return 0;
}

template <class C>
int attn_do(const LatentAttnArgs* a, int* workers, void* stream) {
    if (workers) return attn_workers<C>(workers);
    return attn_launch<C>(*a, static_cast<hipStream_t>(stream));
}

template <int D, int NG>
int pick_rows(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream) {
    if (k.wide) return k.wr == 1 ? attn_do<Cfg<D, NG, true, 1, 1>>(a, workers, stream) : attn_do<Cfg<D, NG, true, 1, 2>>(a, workers, stream);
    if (k.rt == 1) return k.wr == 1 ? attn_do<Cfg<D, NG, false, 1, 1>>(a, workers, stream) : attn_do<Cfg<D, NG, false, 1, 2>>(a, workers, stream);
    return attn_do<Cfg<D, NG, false, 2, 2>>(a, workers, stream);
}

}  // namespace
}  // namespace hr
