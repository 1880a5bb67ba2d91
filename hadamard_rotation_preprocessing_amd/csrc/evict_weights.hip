// Attention weights added up over the paged 4-bit cache (hr_cache_weights).
//
// Mathematics.  With a key k = s (c - z) a score is the sum over its groups of
// s (q . (c - z)): a matrix product over small integers, which float16 holds
// exactly, and a float32 scale on its results.  The log-sum-exp is given, so that
// a weight is one exponential, and a position's sum over the rows of its kv head
// (new tokens x query heads) is a sum over the rows of a result tile: the queries
// are the A operand and the keys the B operand of v_mfma_f32_16x16x32_f16, so that
// a lane holds four rows of one key.  The result is float32, and so must the
// scores be: a query is the sum of two float16 (22 bits) in a power of two of its
// row, two matrix products for each step.
//
// Layout.  weights_query rotates the queries once and leaves them in the scratch
// in the order of a lane's operand, kv head by kv head, with each row's scale and
// log-sum-exp.
//
// Many rows (chunks of prompts): a workgroup of weights_add takes the keys of a block
// of one kv head of one sequence, 16 KT of them to a wave, as operands in registers,
// and passes over the rows that see some of them, kRows at a time through LDS, shared
// by its four waves; two buffers, and the next rows on their way.  Blocks are numbered
// over all sequences and kv heads; where they do not go into the workgroups evenly,
// their rows are numbered, a workgroup takes an equal run of those, and weights_join
// adds up the blocks that were cut.  Two chunks of 2048 tokens against 8192 positions,
// 32 heads over 8 of 128: the whole call 503 to 513 us, of which weights_query is 22 and
// weights_join 5 (480 GFLOP with the two products counted, 950 TFLOP/s).  By counters
// the matrix instructions are 42% of weights_add's cycles, the vector ones 48% (of 112
// cycles for a tile 64 are exponentials), LDS is active for 32% of them and 10% are
// conflicts; waves wait a fifth of their time.  Steps to this form, each beside the one
// before (on a day when the last took 566 us): no rows on their way 702 us; with them, and
// a branch for each absent tile, 681; one tile of keys at a time 586, two 581;
// neighbouring work on one die 566.
//
// Few rows (steps): weights_few, below.  24 sequences of up to 32768, one token each:
// 34 us for 74 MB, 2.2 TB/s.  Waves wait 60% of their time, and vector instructions are
// 47% of the cycles: for 64 keys a wave has 16 loads (codes, and a scale, a zero point
// and a weight of 2, 1 and 4 bytes for each of 16 keys, the same in four lane groups) and
// 4 stores under way.  A window saves nothing here: tiles that no row sees are loaded and
// multiplied too (24 of 32768, all of it or a window of 4096: 155 us both).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "cache_vectors.h"
#include "evict.h"

namespace hr {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef int int4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 32;     // rows of a stage
constexpr int kItem = 64;     // keys of a block of weights_few: four tiles of 16, one of each on its way
// Stages that the keys' way into registers and the sums' way out cost.  (With 1 or 4 for
// 2 one chunk of 64 tokens behind 3936, 32 heads over 8, takes 29 or 27 us for 27, three
// of 777 tokens of up to 900, 8 over 2 of 64, 34 or 33 for 32.)
constexpr int kSetUp = 2;
// Of work to a workgroup: with less there are fewer workgroups.  (With 1 the latter take
// 34 us for 32, and four chunks of 100 tokens behind 900, 8 heads over 2, 24 for 31;
// with 16 50 and 44.)
constexpr int kLeast = 4;
constexpr int kTop = 14;      // a row's largest query element is below 2^kTop in float16

__device__ __forceinline__ float4v mfma(uint4v a, uint4v b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pk_sub(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, a) - __builtin_bit_cast(half2v, b));
}
// two floats as pairs of float16: hi, and what it loses of them
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
    asm("" : "+v"(a), "+v"(b));   // (as values: no contraction with the products that made them)
    half2v h, l;
    h.x = static_cast<_Float16>(a);
    h.y = static_cast<_Float16>(b);
    l.x = static_cast<_Float16>(a - static_cast<float>(h.x));
    l.y = static_cast<_Float16>(b - static_cast<float>(h.y));
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, l);
}

__device__ __forceinline__ int cu_at(const CacheSeqs& s, int b) {
    const int c = s.cu ? s.cu[b] : b * s.per;
    return min(max(c, 0), s.tokens);
}

template <int D>
struct Shape {
    static constexpr int KT = D == 256 ? 2 : 4;      // 16-key tiles of a wave
    static constexpr int KEYS = 4 * 16 * KT;         // of a block
    static constexpr int STRIDE = 4 * D + 32;        // bytes of a row in LDS: hi, lo, and a shift of eight banks
};

// A sequence: its tokens from `start`, its positions, and the position of its first
// new token (which may lie before 0).
struct Seq {
    int start, n, len, first;
};
__device__ __forceinline__ Seq seq_of(const CacheWeightsArgs& a, int b) {
    Seq s;
    s.start = cu_at(a.sq, b);
    s.n = max(cu_at(a.sq, b + 1) - s.start, 0);
    s.len = static_cast<int>(min(static_cast<int64_t>(max(a.sq.lens[b], 0)), static_cast<int64_t>(a.sq.max_pages) << a.pg.logp));
    s.first = s.len - s.n;
    return s;
}

// The rows of a kv head that see some key of [j0, j0 + keys): from p0, a multiple of
// kRows, to p1; their stages.
__device__ __forceinline__ int stages_of(const CacheWeightsArgs& a, const Seq& s, int64_t j0, int keys, int64_t& p0, int64_t& p1) {
    p0 = 0;
    p1 = static_cast<int64_t>(s.n) * a.rep;
    if (a.causal) {
        p0 = max(j0 - s.first, int64_t{0}) * a.rep;
        if (a.window) p1 = min(p1, (j0 + keys - 1 - s.first + a.window) * a.rep);
    }
    p0 = p0 / kRows * kRows;
    return p1 > p0 ? static_cast<int>((p1 - p0 + kRows - 1) / kRows) : 0;
}

typedef const int32_t __attribute__((address_space(4)))* ConstInts;

// the last of first[0 .. n - 1], ascending, that is at most `item`, by the whole wave
__device__ __forceinline__ int last_at_most(const int64_t* first, int n, int64_t item) {
    const int lane = threadIdx.x & 63;
    int lo = 0, end = n;
    while (end - lo > 1) {
        const int step = (end - lo + 63) / 64, at = lo + lane * step;
        const int k = __popcll(__ballot(at < end && first[at < end ? at : lo] <= item));
        lo += (k > 0 ? k - 1 : 0) * step;
        end = min(lo + step, end);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// ---------------------------------------------------------------------------
// the queries

// What a row needs beside its query: the factor of its products with codes (the
// score's scale, in powers of e turned to powers of 2, over the row's unit) and its
// log-sum-exp in powers of 2.
struct RowScale {
    float factor, lse;
};
// Whether a row's log-sum-exp is -inf (as inf here): it is left out by selection, as
// its scores may be NaN.
__device__ __forceinline__ bool adds_nothing(const RowScale& r) { return r.lse == __builtin_inff(); }

// Rows (t, i) of q, as [kv head][token][query head of it][hi, lo][D] float16.
// Elements of eight stand in the order 0 4 1 5 2 6 3 7, that of the codes' operands.
template <int D, class T>
__global__ void __launch_bounds__(256) weights_query(const CacheWeightsArgs a, uint32_t* out, RowScale* rows, int64_t* first_of) {
    constexpr int LPV = D / 16;
    if (blockIdx.x == 0) {       // the numbering of the work
        __shared__ int64_t sums[4], counts[256];
        constexpr int KEYS = Shape<D>::KEYS;
        // `lanes` threads to a sequence, as many as there are for each
        int lanes = 64;
        while (lanes > 1 && 256 / lanes < a.sq.rows) lanes /= 2;
        const int at_once = 256 / lanes, part = threadIdx.x % lanes;
        // a thread's part of the stages of a sequence's head, and the most of one block
        const auto stages = [&](const Seq& s, int& most) {
            int64_t mine = 0, p0, p1;
            if (s.n > 0)
                for (int64_t j0 = static_cast<int64_t>(part) * KEYS; j0 < s.len; j0 += lanes * KEYS) {
                    const int w = kSetUp + stages_of(a, s, j0, KEYS, p0, p1);
                    mine += w;
                    most = max(most, w);
                }
            return mine;
        };
        bool whole = true;
        if (!a.few) {
            int64_t work = 0, blocks = 0;
            int most = 0;
            for (int i = threadIdx.x / lanes; i < a.sq.rows; i += at_once) {
                const Seq s = seq_of(a, i);
                work += stages(s, most) * a.pg.hkv;
                if (s.n > 0 && part == 0) blocks += (static_cast<int64_t>(s.len) + KEYS - 1) / KEYS * a.pg.hkv;
            }
#pragma unroll
            for (int x = 1; x < 64; x *= 2) {
                work += __shfl_xor(work, x);
                blocks += __shfl_xor(blocks, x);
                most = max(most, __shfl_xor(most, x));
            }
            if ((threadIdx.x & 63) == 0) {
                counts[threadIdx.x / 64] = work;
                counts[4 + threadIdx.x / 64] = blocks;
                counts[8 + threadIdx.x / 64] = most;
            }
            __syncthreads();
            work = counts[0] + counts[1] + counts[2] + counts[3];
            blocks = counts[4] + counts[5] + counts[6] + counts[7];
            const int64_t heaviest = max(max(counts[8], counts[9]), max(counts[10], counts[11]));
            whole = 4 * heaviest * ((blocks + a.workers - 1) / a.workers) * a.workers <= 5 * work;
            __syncthreads();
        }
        int64_t before = 0;
        for (int r0 = 0; r0 < a.sq.rows; r0 += 256) {
            const int r = r0 + threadIdx.x;
            int64_t v = 0;
            if (whole) {                      // in blocks of keys
                if (r < a.sq.rows) {
                    const Seq s = seq_of(a, r);
                    const int keys = a.few ? kItem : KEYS;
                    if (s.n > 0) v = (static_cast<int64_t>(s.len) + keys - 1) / keys * a.pg.hkv;
                }
            } else {                          // in stages
                int most = 0;
                for (int i = threadIdx.x / lanes; i < 256 && r0 + i < a.sq.rows; i += at_once) {
                    int64_t n = stages(seq_of(a, r0 + i), most);
                    for (int x = 1; x < lanes; x *= 2) n += __shfl_xor(n, x);
                    if (part == 0) counts[i] = n * a.pg.hkv;
                }
                __syncthreads();
                if (r < a.sq.rows) v = counts[threadIdx.x];
            }
            for (int x = 1; x < 64; x *= 2) {
                const int64_t y = __shfl_up(v, x);
                if ((threadIdx.x & 63) >= x) v += y;
            }
            __syncthreads();
            if ((threadIdx.x & 63) == 63) sums[threadIdx.x / 64] = v;
            __syncthreads();
            for (int x = 0; x < 4; ++x)
                if (x < static_cast<int>(threadIdx.x / 64)) v += sums[x];
            if (r < a.sq.rows) first_of[r + 1] = before + v;
            before += sums[0] + sums[1] + sums[2] + sums[3];
        }
        if (threadIdx.x == 0) first_of[0] = whole && !a.few ? -1 : 0;     // (and how it is numbered)
    }
    const int64_t v = (int64_t{blockIdx.x} * 256 + threadIdx.x) / LPV;
    const int64_t total = int64_t{a.sq.tokens} * a.hq;
    const int lane = threadIdx.x & 63, e = lane % LPV;
    const int64_t at = min(v, total - 1);
    const int64_t t = at / a.hq;
    const int i = static_cast<int>(at % a.hq), h = i / a.rep;
    float x[16];
    load16(static_cast<const T*>(a.q) + t * a.q_st + i * a.q_sh + 16 * e, x);
    if (a.rotate) hadamard<D>(x, lane, a.norm);
    float top = fabsf(x[0]);
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
    top = over_lanes<LPV>(top, [](float p, float q) { return fmaxf(p, q); });
    int unit = 0;
    if (top > 0.0f && top < __builtin_inff()) unit = min(kTop - 1 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), 110);   // (from -114)
    const int64_t r = (int64_t{h} * a.sq.tokens + t) * a.rep + i % a.rep;
    if (v >= total) return;
    uint32_t* to = out + r * D;       // hi: D / 2 words, then lo
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
        reinterpret_cast<uint4v*>(to + D / 2)[(16 * e + j) / 8] = lo;
    }
    if (e == 0) {
        const float lse = a.lse[at];
        rows[r].factor = __builtin_ldexpf(a.scale * kLog2e, -unit);
        rows[r].lse = lse == -__builtin_inff() ? __builtin_inff() : lse * kLog2e;
    }
}

// ---------------------------------------------------------------------------
// the sums

// A row of a stage, as its keys see it: they lie in [lo, hi).
struct RowInfo {
    float factor, lse;
    int lo, hi;
};

// a value that all lanes have, as the compiler cannot see
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uni(int64_t v) {
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(uni(static_cast<int>(v >> 32)))) << 32 |
                                static_cast<uint32_t>(uni(static_cast<int>(v))));
}

// The work of all sequences and kv heads, in stages: a block of keys has kSetUp and
// those of its rows.  Workgroup `worker` takes [begin, end) of it.  Where whole blocks
// go into the workgroups evenly (the longest takes at most 5/4 of the mean) the work
// is numbered in blocks, one each, and first_of[0] is -1: workgroups then keep step
// and share the queries in their caches (two chunks of 2048 tokens against 8192: 518 us,
// 537 in stages, evenly); where not, a few blocks with many rows are the work of all (two
// chunks of 269 tokens against 447, 7 heads of one kv head: 93 us whole, 31 in stages).
struct Range {
    int64_t begin, end;
};
__device__ __forceinline__ Range range_of(const CacheWeightsArgs& a, int64_t total, bool whole, int worker) {
    const int64_t n = min(max(whole ? total : total / kLeast, int64_t{1}), static_cast<int64_t>(a.workers));
    if (worker >= n) return {total, total};
    return {total * worker / n, total * (worker + 1) / n};
}

// The block that `item` belongs to: its sequence, kv head, first key and work, and what
// of its work lies before item.  All lanes of a wave ask for the same.
struct Block {
    Seq s;
    int b, h, work;
    int64_t j0, at;
};
template <int KEYS>
__device__ __forceinline__ Block block_of(const CacheWeightsArgs& a, const int64_t* first_of, bool whole, int64_t item) {
    Block k;
    k.b = last_at_most(first_of, a.sq.rows, item);
    k.s = seq_of(a, k.b);
    const int64_t before = max(first_of[k.b], int64_t{0}), heads = (first_of[k.b + 1] - before) / a.pg.hkv;   // work of a head
    k.h = static_cast<int>((item - before) / heads);
    k.at = (item - before) % heads;
    k.work = 1;
    if (whole) {
        k.j0 = k.at * KEYS;
        k.at = 0;
        return k;
    }
    const int lane = threadIdx.x & 63;
    for (k.j0 = 0;; k.j0 += 64 * KEYS) {
        int64_t p0, p1;
        const int64_t j0 = k.j0 + static_cast<int64_t>(lane) * KEYS;
        const int mine = j0 < k.s.len ? kSetUp + stages_of(a, k.s, j0, KEYS, p0, p1) : 0;
        int64_t upto = mine;
#pragma unroll
        for (int x = 1; x < 64; x *= 2) {
            const int64_t y = __shfl_up(upto, x);
            if (lane >= x) upto += y;
        }
        const uint64_t past = __ballot(upto > k.at);
        if (past) {
            const int l = __ffsll(static_cast<unsigned long long>(past)) - 1;
            k.work = __shfl(mine, l);
            k.at -= __shfl(upto, l) - k.work;
            k.j0 += static_cast<int64_t>(l) * KEYS;
            return k;
        }
        k.at -= __shfl(upto, 63);
        if (k.j0 + 64 * KEYS >= k.s.len) return k;     // (never: the numbering has the item)
    }
}

template <int D, int NG>
__global__ void __launch_bounds__(256) weights_add(const CacheWeightsArgs a, const uint32_t* query, const RowScale* scales, const int64_t* first_of, float* parts) {
    using S = Shape<D>;
    constexpr int KT = S::KT, KG = D / 32 / NG;
    __shared__ __attribute__((aligned(16))) uint8_t stages_[2][kRows * S::STRIDE];
    __shared__ __attribute__((aligned(16))) RowInfo infos[2][kRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
    const CachePage& pg = a.pg;
    // neighbouring work, which reads the same queries, on the same die
    const int worker = a.workers % 8 ? blockIdx.x : blockIdx.x % 8 * (a.workers / 8) + blockIdx.x / 8;
    const bool by_block = uni(first_of[0]) < 0;
    const Range range = range_of(a, uni(first_of[a.sq.rows]), by_block, worker);
    for (int64_t item = range.begin; item < range.end;) {
        Block k = block_of<S::KEYS>(a, first_of, by_block, item);
        k.s = {uni(k.s.start), uni(k.s.n), uni(k.s.len), uni(k.s.first)};
        k.work = uni(k.work);
        const int b = uni(k.b), h = uni(k.h), j0 = uni(static_cast<int>(k.j0)), n = k.s.n, len = k.s.len, first = k.s.first, start = k.s.start;
        const int u0 = uni(static_cast<int>(k.at)), u1 = static_cast<int>(min(static_cast<int64_t>(k.work), u0 + range.end - item));
        item += max(u1 - u0, 1);
        const int32_t* table = a.sq.table + static_cast<int64_t>(b) * a.sq.max_pages;

        // the wave's keys: B operands of c - z, and their scales
        uint4v key[KT][D / 32];
        float scale[KT][NG];
        bool there[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const int t0 = j0 + (wave * KT + kt) * 16;
            const int page = t0 < len ? table[t0 >> pg.logp] : -1;
            there[kt] = page >= 0 && page < a.sq.n_pages;
            if (!there[kt]) {              // (worked on all the same, and not added)
#pragma unroll
                for (int i = 0; i < D / 32; ++i) key[kt][i] = uint4v{0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < NG; ++q) scale[kt][q] = 0.0f;
                continue;
            }
            const int off = (t0 & (pg.page - 1)) + m;
            const uint8_t* base = a.pool + page * pg.page_bytes + h * pg.head_bytes;
            const uint8_t* codes = base + pg.kc + off * (D / 2);
#pragma unroll
            for (int q = 0; q < NG; ++q) {
                const int at = off * NG + q;
                scale[kt][q] = pg.sf32 ? reinterpret_cast<const float*>(base + pg.ks)[at]
                                       : bf2f(reinterpret_cast<const uint16_t*>(base + pg.ks)[at]);
                const uint32_t z = pg.sym ? 8u : (base[pg.kz + at / 2] >> (4 * (at & 1))) & 15u;
                // ORed with 1024 (at bit 4: 64) a code c is the float16 1024 + c (64 + c)
                const uint32_t f0 = 0x64006400u ^ (pg.sym ? 0x00080008u : 0u), f1 = 0x54005400u ^ (pg.sym ? 0x00800080u : 0u);
                const uint32_t z0 = 0x64006400u + z * 0x00010001u, z1 = 0x54005400u + z * 0x00100010u;
#pragma unroll
                for (int i = 0; i < KG; ++i) {
                    uint32_t w = reinterpret_cast<const uint32_t*>(codes)[q * (D / NG / 8) + g * KG + i];
                    uint4v k;
                    k.x = pk_sub((w & 0x000F000Fu) ^ f0, z0);
                    k.y = pk_sub((w & 0x00F000F0u) ^ f1, z1);
                    w >>= 8;
                    k.z = pk_sub((w & 0x000F000Fu) ^ f0, z0);
                    k.w = pk_sub((w & 0x00F000F0u) ^ f1, z1);
                    key[kt][q * KG + i] = k;
                }
            }
        }
        float sum[KT] = {}, sums[KT] = {};
        const int64_t rows = static_cast<int64_t>(n) * a.rep;
        const int64_t at = (static_cast<int64_t>(h) * a.sq.tokens + start) * a.rep;   // the rows' place in `query`
        int64_t p0, p1;                // the rows that see some key of the block; of them, this workgroup's
        stages_of(a, k.s, j0, S::KEYS, p0, p1);
        if (!by_block) {
            p1 = min(p1, p0 + static_cast<int64_t>(max(u1 - kSetUp, 0)) * kRows);
            p0 += static_cast<int64_t>(max(u0 - kSetUp, 0)) * kRows;
        }
        int stages = 0;
        // the next rows are on their way while these are worked on
        constexpr int LOADS = kRows * D / 4 / 256;          // of 16 bytes
        uint4v ahead[LOADS];
        RowScale rs{};
        const auto load = [&](int64_t p) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int x = i * 256 + tid, r = x / (D / 4), c = x % (D / 4);
                ahead[i] = reinterpret_cast<const uint4v*>(query + (at + min(p + r, rows - 1)) * D)[c];
            }
            rs = scales[at + min(p + lane % kRows, rows - 1)];   // (every wave asks about them, below)
        };
        if (p0 < p1) load(p0);
        for (int64_t p = p0; p < p1; p += kRows) {
            uint8_t* stage = stages_[stages & 1];
            RowInfo* info = infos[stages & 1];
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int x = i * 256 + tid, r = x / (D / 4), c = x % (D / 4);
                *reinterpret_cast<uint4v*>(stage + r * S::STRIDE + c * 16) = ahead[i];
            }
            if (tid < kRows) {
                RowInfo ri;
                const int pos = first + static_cast<int>(static_cast<uint32_t>(min(p + tid, rows - 1)) / a.rep);
                ri.factor = rs.factor;
                ri.lse = rs.lse;
                ri.lo = a.window ? max(pos - a.window + 1, 0) : 0;
                ri.hi = p + tid < rows && !adds_nothing(rs) ? (a.causal ? min(pos + 1, len) : len) : 0;
                info[tid] = ri;
            }
            const bool some_out = __any(adds_nothing(rs));
            // (two buffers: the last readers of this one are before the last barrier)
            __syncthreads();
            if (p + kRows < p1) load(p + kRows);
            // whether every row of the stage is there, adds something and sees every key of the block
            const int pos0 = first + static_cast<int>(static_cast<uint32_t>(p) / a.rep);
            const int pos1 = first + static_cast<int>(static_cast<uint32_t>(min(p + kRows, rows) - 1) / a.rep);
            const bool full = !some_out && p + kRows <= rows && j0 + S::KEYS <= len && (!a.causal || j0 + S::KEYS - 1 <= pos0) &&
                              (!a.window || j0 > pos1 - a.window);
            const auto tiles = [&](auto FULL) __attribute__((always_inline)) {
#pragma unroll
                for (int rt = 0; rt < kRows / 16; ++rt) {
                    uint4v qh[D / 32], ql[D / 32];
                    const uint8_t* row = stage + (rt * 16 + m) * S::STRIDE;
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int i = 0; i < KG; ++i) {
                            const int c = 2 * (q * (D / NG) + g * (D / NG / 4) + 8 * i);
                            qh[q * KG + i] = *reinterpret_cast<const uint4v*>(row + c);
                            ql[q * KG + i] = *reinterpret_cast<const uint4v*>(row + 2 * D + c);
                        }
                    RowInfo ri[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) ri[i] = info[rt * 16 + 4 * g + i];
// (two tiles at a time: no matrix instruction waits for the one before it)
#pragma unroll
                    for (int kt = 0; kt < KT; kt += 2) {
                        float4v w[2];
#pragma unroll
                        for (int q = 0; q < NG; ++q) {
                            float4v c[2];
                            c[0] = c[1] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int i = 0; i < KG; ++i) {
#pragma unroll
                                for (int x = 0; x < 2; ++x) c[x] = mfma(ql[q * KG + i], key[kt + x][q * KG + i], c[x]);
#pragma unroll
                                for (int x = 0; x < 2; ++x) c[x] = mfma(qh[q * KG + i], key[kt + x][q * KG + i], c[x]);
                            }
#pragma unroll
                            for (int x = 0; x < 2; ++x)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    w[x][i] = q ? __builtin_fmaf(c[x][i], scale[kt + x][q], w[x][i]) : c[x][i] * scale[kt + x][0];
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int j = j0 + (wave * KT + kt + x) * 16 + m;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float e = __builtin_amdgcn_exp2f(__builtin_fmaf(w[x][i], ri[i].factor, -ri[i].lse));
                                if constexpr (!decltype(FULL)::value) e = j >= ri[i].lo && j < ri[i].hi ? e : 0.0f;
                                sums[kt + x] += e;
                            }
                        }
                    }
                }
            };
            if (full) tiles(std::true_type());
            else tiles(std::false_type());
            // sums of 16 stages apart, so that a long sum loses less
            if (++stages % 16 == 0) {
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    sum[kt] += sums[kt];
                    sums[kt] = 0.0f;
                }
            }
        }
        __syncthreads();                   // (the next block's rows)
        const bool whole = u0 == 0 && u1 == k.work;
        float* out = a.weights + (static_cast<int64_t>(b) * pg.hkv + h) * a.width;
        float* part = parts + (static_cast<int64_t>(worker) * 2 + (u0 == 0)) * S::KEYS;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            float v = there[kt] ? sum[kt] + sums[kt] : 0.0f;
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            const int j = j0 + (wave * KT + kt) * 16 + m;
            if (g == 0 && !whole) part[(wave * KT + kt) * 16 + m] = v;
            if (g == 0 && whole && j < len) out[j] = (j < first ? a.decay * out[j] : 0.0f) + v;
        }
    }
}

// Sums of a block that several workgroups took: parts[w][1] of the one that began it,
// parts[w][0] of those after it, in their order.
template <int D>
__global__ void __launch_bounds__(Shape<D>::KEYS) weights_join(const CacheWeightsArgs a, const int64_t* first_of, const float* parts) {
    constexpr int KEYS = Shape<D>::KEYS;
    if (first_of[0] < 0) return;           // (whole blocks)
    const int64_t total = first_of[a.sq.rows];
    const int worker = blockIdx.x;
    const Range mine = range_of(a, total, false, worker);
    if (mine.begin == mine.end || mine.end == total) return;
    const Block k = block_of<KEYS>(a, first_of, false, mine.end);
    if (k.at == 0 || mine.end - k.at < mine.begin) return;     // no block is cut here, or it began before
    const int64_t end = mine.end - k.at + k.work;
    const int t = threadIdx.x;
    float sum = parts[(static_cast<int64_t>(worker) * 2 + 1) * KEYS + t];
    for (int w = worker + 1;; ++w) {
        sum += parts[static_cast<int64_t>(w) * 2 * KEYS + t];
        if (range_of(a, total, false, w).end >= end) break;
    }
    const int64_t j = k.j0 + t;
    float* out = a.weights + (static_cast<int64_t>(k.b) * a.pg.hkv + k.h) * a.width;
    if (j < k.s.len) out[j] = (j < k.s.first ? a.decay * out[j] : 0.0f) + sum;
}

// ---------------------------------------------------------------------------
// few rows
//
// With up to 32 rows of a kv head (single tokens, drafts) the queries stay in
// registers and the keys stream past them: every wave takes an equal, contiguous run
// of all key blocks of all kv heads and sequences, numbered by weights_query, whatever
// the lengths, and no wave waits for another.  The loads of the next kItem keys are on
// their way throughout.

template <int N>
__device__ __forceinline__ void buffer_words(__amdgpu_buffer_rsrc_t r, int lane_at, int at, uint32_t* w) {
    if constexpr (N == 1) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, lane_at, at, 0);
    } else if constexpr (N == 2) {
        const uint2v x = __builtin_bit_cast(uint2v, __builtin_amdgcn_raw_buffer_load_b64(r, lane_at, at, 0));
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4v x = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(r, lane_at + 4 * i, at, 0));
            w[i] = x.x;
            w[i + 1] = x.y;
            w[i + 2] = x.z;
            w[i + 3] = x.w;
        }
    }
}

// What a lane holds of a tile of 16 keys on its way: of key lane & 15 a quarter of each
// group's codes, the scales and zero points, and the weight.
template <int D, int NG>
struct Tile {
    uint32_t codes[D / 32], scales[NG], zeros, weight;
};

template <int D, int NG, int RT>
__global__ void __launch_bounds__(256) weights_few(const CacheWeightsArgs a, const uint32_t* query, const RowScale* scales, const int64_t* first_of) {
    constexpr int KG = D / 32 / NG, G = D / NG;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const CachePage& pg = a.pg;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6)), waves = gridDim.x * 4;
    const int64_t total = ((const int64_t __attribute__((address_space(4)))*)(first_of))[a.sq.rows];
    int64_t item = total * wave / waves;
    const int64_t end = total * (wave + 1) / waves;
    if (item >= end) return;
    int b = last_at_most(first_of, a.sq.rows, item);
    const uint32_t flip0 = pg.sym ? 0x00080008u : 0u, flip1 = pg.sym ? 0x00800080u : 0u;
    const uint32_t f0 = 0x64006400u ^ flip0, f1 = 0x54005400u ^ flip1;
    while (item < end) {
        const auto first_item = (const int64_t __attribute__((address_space(4)))*)(first_of);
        while (first_item[b + 1] <= item) ++b;
        const ConstInts cu = (ConstInts)(a.sq.cu), lens = (ConstInts)(a.sq.lens);
        const int start = min(max(a.sq.cu ? cu[b] : b * a.sq.per, 0), a.sq.tokens);
        const int n = max(min(max(a.sq.cu ? cu[b + 1] : (b + 1) * a.sq.per, 0), a.sq.tokens) - start, 0);
        const int len = static_cast<int>(min(static_cast<int64_t>(max(lens[b], 0)), static_cast<int64_t>(a.sq.max_pages) << pg.logp));
        const int blocks = static_cast<int>((static_cast<int64_t>(len) + kItem - 1) / kItem);
        const int64_t in_row = item - first_item[b];
        const int h = static_cast<int>(in_row / blocks), k0 = static_cast<int>(in_row % blocks);
        const int k1 = static_cast<int>(min(static_cast<int64_t>(blocks), k0 + end - item));   // blocks k0 .. k1 - 1 of the head
        item += k1 - k0;
        const int first = len - n, rows = n * a.rep;
        const ConstInts table = (ConstInts)(a.sq.table + static_cast<int64_t>(b) * a.sq.max_pages);
        const int64_t at = (static_cast<int64_t>(h) * a.sq.tokens + start) * a.rep;   // the rows' place in `query`
        float* out = a.weights + (static_cast<int64_t>(b) * pg.hkv + h) * a.width;
        // (more rows than one pass takes: the passes after the first add to it)
        for (int r0 = 0; r0 < rows; r0 += 16 * RT) {
            uint4v qh[RT][D / 32], ql[RT][D / 32];
            float factor[RT][4], lse[RT][4];
            int from[RT][4], to[RT][4];            // the keys that a row sees
            int all_from = 0, all_to = len;        // and those that all rows do
            bool some_out = false;                 // whether one of the lane's rows adds nothing
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint32_t* q = query + (at + min(r0 + 16 * rt + m, rows - 1)) * D;
#pragma unroll
                for (int x = 0; x < NG; ++x)
#pragma unroll
                    for (int i = 0; i < KG; ++i) {
                        const int c = (x * G + g * (G / 4) + 8 * i) / 8;
                        qh[rt][x * KG + i] = reinterpret_cast<const uint4v*>(q)[c];
                        ql[rt][x * KG + i] = reinterpret_cast<const uint4v*>(q + D / 2)[c];
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = r0 + 16 * rt + 4 * g + i;
                    const RowScale rs = scales[at + min(r, rows - 1)];
                    const int pos = first + min(r, rows - 1) / a.rep;
                    factor[rt][i] = rs.factor;
                    lse[rt][i] = r < rows ? rs.lse : __builtin_inff();
                    to[rt][i] = r < rows && !adds_nothing(rs) ? (a.causal ? min(pos + 1, len) : len) : 0;
                    some_out = some_out || adds_nothing(rs);
                    from[rt][i] = a.window ? max(pos - a.window + 1, 0) : 0;
                }
            }
            if (a.causal) all_to = min(first + r0 / a.rep + 1, len);
            if (a.window) all_from = max(first + (min(r0 + 16 * RT, rows) - 1) / a.rep - a.window + 1, 0);
            const bool whole = r0 + 16 * RT <= rows && !__any(some_out);

            Tile<D, NG> tile[4];
            int page[4], next[4];                  // of the tile in a place, and of the one after it
            const int upto = static_cast<int>(min(static_cast<int64_t>(k1) * kItem, static_cast<int64_t>(len)));   // the run's end
            const auto page_of = [&](int t) __attribute__((always_inline)) { return t < upto ? table[t >> pg.logp] : -1; };
            const auto load = [&](auto X, int t) __attribute__((always_inline)) {
                const bool here = static_cast<uint32_t>(page[X]) < static_cast<uint64_t>(a.sq.n_pages);
                const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                    const_cast<uint8_t*>(a.pool + (here ? page[X] : 0) * pg.page_bytes + h * pg.head_bytes), 0, here ? static_cast<int>(pg.head_bytes) : 0, 0x00020000);
                const int off = t & (pg.page - 1);
                Tile<D, NG>& w = tile[X];
                if constexpr (NG == 1) {
                    buffer_words<D / 32>(r, m * (D / 2) + g * (D / 8), pg.kc + off * (D / 2), w.codes);
                } else {
#pragma unroll
                    for (int x = 0; x < NG; ++x) buffer_words<KG>(r, m * (D / 2) + g * (G / 8) + x * (G / 2), pg.kc + off * (D / 2), w.codes + x * KG);
                }
                if (pg.sf32) {
                    buffer_words<NG>(r, 4 * m * NG, pg.ks + off * NG * 4, w.scales);
                } else {
#pragma unroll
                    for (int x = 0; x < NG; ++x)
                        w.scales[x] = static_cast<uint32_t>(static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, 2 * (m * NG + x), pg.ks + off * NG * 2, 0))) << 16;
                }
                // (symmetric: some bytes, not looked at)
                const int zl = m * NG / 2, zs = pg.kz + off * NG / 2;
                if constexpr (NG <= 2) w.zeros = static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(r, zl, zs, 0));
                else if constexpr (NG == 4) w.zeros = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, zl, zs, 0));
                else w.zeros = __builtin_amdgcn_raw_buffer_load_b32(r, zl, zs, 0);
                const int j = t + m;
                w.weight = __float_as_uint(j < upto ? out[j] : 0.0f);
            };
            const auto work = [&](auto X, int t) __attribute__((always_inline)) {
                const Tile<D, NG>& w = tile[X];
                const bool here = static_cast<uint32_t>(page[X]) < static_cast<uint64_t>(a.sq.n_pages);
                float sum = 0.0f;
                if (here) {
                    float4v s[RT];
#pragma unroll
                    for (int x = 0; x < NG; ++x) {
                        const uint32_t z = pg.sym ? 8u : (w.zeros >> (4 * (NG == 1 ? m & 1 : x))) & 15u;
                        const uint32_t z0 = 0x64006400u + z * 0x00010001u, z1 = 0x54005400u + z * 0x00100010u;
                        float4v c[RT];
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) c[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int i = 0; i < KG; ++i) {
                            uint32_t v = w.codes[x * KG + i];
                            uint4v k;
                            k.x = pk_sub((v & 0x000F000Fu) ^ f0, z0);
                            k.y = pk_sub((v & 0x00F000F0u) ^ f1, z1);
                            v >>= 8;
                            k.z = pk_sub((v & 0x000F000Fu) ^ f0, z0);
                            k.w = pk_sub((v & 0x00F000F0u) ^ f1, z1);
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) {
                                c[rt] = mfma(ql[rt][x * KG + i], k, c[rt]);
                                c[rt] = mfma(qh[rt][x * KG + i], k, c[rt]);
                            }
                        }
                        const float sc = __uint_as_float(w.scales[x]);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) s[rt][i] = x ? __builtin_fmaf(c[rt][i], sc, s[rt][i]) : c[rt][i] * sc;
                    }
                    const bool full = whole && t >= all_from && t + 16 <= all_to;
                    const int j = t + m;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][i], factor[rt][i], -lse[rt][i]));
                            if (!full) e = j >= from[rt][i] && j < to[rt][i] ? e : 0.0f;
                            sum += e;
                        }
                    sum += __shfl_xor(sum, 16);
                    sum += __shfl_xor(sum, 32);
                }
                const int j = t + m;
                const float old = __uint_as_float(w.weight);
                if (g == 0 && j < len) out[j] = (r0 > 0 ? old : j < first ? a.decay * old : 0.0f) + sum;
            };
            const int t0 = k0 * kItem;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                page[x] = page_of(t0 + 16 * x);
                next[x] = page_of(t0 + 16 * x + kItem);
            }
            typedef std::integral_constant<int, 0> P0;
            typedef std::integral_constant<int, 1> P1;
            typedef std::integral_constant<int, 2> P2;
            typedef std::integral_constant<int, 3> P3;
            load(P0(), t0);
            load(P1(), t0 + 16);
            load(P2(), t0 + 32);
            load(P3(), t0 + 48);
            const auto turn = [&](auto X, int t) __attribute__((always_inline)) {
                if (t < len) work(X, t);
                page[X] = next[X];
                load(X, t + kItem);
                next[X] = page_of(t + 2 * kItem);
            };
            for (int k = k0; k < k1; ++k) {
                const int t = k * kItem;
                turn(P0(), t);
                turn(P1(), t + 16);
                turn(P2(), t + 32);
                turn(P3(), t + 48);
            }
        }
    }
}

template <int D, class T>
void query_launch(const CacheWeightsArgs& a, uint32_t* out, RowScale* rows, int64_t* first_of, hipStream_t s) {
    const int64_t threads = int64_t{a.sq.tokens} * a.hq * (D / 16);
    hipLaunchKernelGGL((weights_query<D, T>), dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0, s, a, out, rows, first_of);
}

template <int D, int NG>
void add_launch(const CacheWeightsArgs& a, int bf16, hipStream_t s) {
    int64_t* first_of = reinterpret_cast<int64_t*>(a.work);
    RowScale* rows = reinterpret_cast<RowScale*>(a.work + cache_weights_first(a.sq.rows));
    uint32_t* query = reinterpret_cast<uint32_t*>(a.work + cache_weights_first(a.sq.rows) + (int64_t{a.sq.tokens} * a.hq * 8 + 15) / 16 * 16);
    if (bf16) query_launch<D, uint16_t>(a, query, rows, first_of, s);
    else query_launch<D, float>(a, query, rows, first_of, s);
    if (a.few == 0) {
        float* parts = reinterpret_cast<float*>(query + int64_t{a.sq.tokens} * a.hq * D);
        hipLaunchKernelGGL((weights_add<D, NG>), dim3(a.workers), dim3(256), 0, s, a, query, rows, first_of, parts);
        hipLaunchKernelGGL((weights_join<D>), dim3(a.workers), dim3(Shape<D>::KEYS), 0, s, a, first_of, parts);
    } else if (a.few == 1) hipLaunchKernelGGL((weights_few<D, NG, 1>), dim3(a.workers), dim3(256), 0, s, a, query, rows, first_of);
    else hipLaunchKernelGGL((weights_few<D, NG, 2>), dim3(a.workers), dim3(256), 0, s, a, query, rows, first_of);
}

}  // namespace

int cache_weights_workers(int few, int* workers) {
    int dev, cus;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    // With few rows, four to a compute unit with one tile of rows and two with two: what
    // fits at once with heads of 64 and 128 in one or two groups (24 sequences of up to 32768
    // and single tokens, 128: 38 us, with three 42; of 8000 and 8 new tokens 72, with one
    // 118).  Kernels of more registers run a second round: single tokens with heads of 128
    // in groups of 32 take 68 us where three take 59, of 256 65 where three take 54, and of
    // 256 in groups of 64 or 32 80 and 118 where two take 78 and 115.
    if (e == hipSuccess) *workers = few == 0 ? (2 * cus < kWeightsParts ? 2 * cus : kWeightsParts) : (few == 2 ? 2 : 4) * cus;
    return static_cast<int>(e);
}

int launch_cache_weights(const CacheWeightsArgs& a, int bf16, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int d = a.pg.d, ng = a.pg.ng;
    if (d == 64 && ng == 1) add_launch<64, 1>(a, bf16, s);
    else if (d == 64 && ng == 2) add_launch<64, 2>(a, bf16, s);
    else if (d == 128 && ng == 1) add_launch<128, 1>(a, bf16, s);
    else if (d == 128 && ng == 2) add_launch<128, 2>(a, bf16, s);
    else if (d == 128 && ng == 4) add_launch<128, 4>(a, bf16, s);
    else if (d == 256 && ng == 1) add_launch<256, 1>(a, bf16, s);
    else if (d == 256 && ng == 2) add_launch<256, 2>(a, bf16, s);
    else if (d == 256 && ng == 4) add_launch<256, 4>(a, bf16, s);
    else if (d == 256 && ng == 8) add_launch<256, 8>(a, bf16, s);
    else return static_cast<int>(hipErrorInvalidValue);
    return static_cast<int>(hipGetLastError());
}

}  // namespace hr
