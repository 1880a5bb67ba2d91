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
// log-sum-exp.  A workgroup of weights_add takes the keys of a block of one kv head
// of one sequence, 16 KT of them to a wave, as operands in registers, and passes
// over all rows that see some of them, kRows at a time through LDS, shared by its
// four waves.  Blocks are numbered over all sequences and kv heads, and workgroups
// take them in turn.  Nothing is joined afterwards.
#include <hip/hip_runtime.h>
#include <stdint.h>

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

// ---------------------------------------------------------------------------
// the queries

// What a row needs beside its query: the factor of its products with codes (the
// score's scale, in powers of e turned to powers of 2, over the row's unit) and its
// log-sum-exp in powers of 2.
struct RowScale {
    float factor, lse;
};

// Rows (t, i) of q, as [kv head][token][query head of it][hi, lo][D] float16.
// Elements of eight stand in the order 0 4 1 5 2 6 3 7, that of the codes' operands.
template <int D, class T>
__global__ void __launch_bounds__(256) weights_query(const CacheWeightsArgs a, uint32_t* out, RowScale* rows) {
    constexpr int LPV = D / 16;
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
    if (top > 0.0f && top < __builtin_inff()) unit = min(max(kTop - 1 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), -110), 110);
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

template <int D>
struct Shape {
    static constexpr int KT = D == 256 ? 2 : 4;      // 16-key tiles of a wave
    static constexpr int KEYS = 4 * 16 * KT;         // of a block
    static constexpr int STRIDE = 4 * D + 16;        // bytes of a row in LDS: hi, lo, and a shift of four banks
};

template <int D, int NG>
__global__ void __launch_bounds__(256) weights_add(const CacheWeightsArgs a, const uint32_t* query, const RowScale* scales) {
    using S = Shape<D>;
    constexpr int KT = S::KT, KG = D / 32 / NG;
    __shared__ __attribute__((aligned(16))) uint8_t stage[kRows * S::STRIDE];
    __shared__ __attribute__((aligned(16))) RowInfo info[kRows];
    __shared__ int64_t first_of[257];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
    const CachePage& pg = a.pg;
    int64_t mine = blockIdx.x;             // this workgroup's next block among those of rows r0 and on
    for (int r0 = 0; r0 < a.sq.rows; r0 += 256) {
        // the blocks of 256 rows, numbered
        int64_t n_blocks = 0;
        if (r0 + tid < a.sq.rows && cu_at(a.sq, r0 + tid + 1) > cu_at(a.sq, r0 + tid)) {
            const int64_t len = min(static_cast<int64_t>(max(a.sq.lens[r0 + tid], 0)), static_cast<int64_t>(a.sq.max_pages) << pg.logp);
            n_blocks = (len + S::KEYS - 1) / S::KEYS * pg.hkv;
        }
        __syncthreads();
        first_of[tid + 1] = n_blocks;
        if (tid == 0) first_of[0] = 0;
        __syncthreads();
        for (int x = 1; x < 256; x *= 2) {
            const int64_t y = tid + 1 > x ? first_of[tid + 1 - x] : 0;
            __syncthreads();
            first_of[tid + 1] += y;
            __syncthreads();
        }
        const int64_t total = first_of[256];
        for (; mine < total; mine += gridDim.x) {
            int lo = 0, hi = 255;          // the last row whose blocks begin at or before this one
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (first_of[mid] <= mine) lo = mid;
                else hi = mid - 1;
            }
            const int b = r0 + lo;
            const int start = cu_at(a.sq, b), n = cu_at(a.sq, b + 1) - start;
            const int len = static_cast<int>(min(static_cast<int64_t>(max(a.sq.lens[b], 0)), static_cast<int64_t>(a.sq.max_pages) << pg.logp));
            const int blocks = static_cast<int>((static_cast<int64_t>(len) + S::KEYS - 1) / S::KEYS);
            const int64_t in_row = mine - first_of[lo];
            const int h = static_cast<int>(in_row / blocks), j0 = static_cast<int>(in_row % blocks) * S::KEYS;
            const int first = len - n;     // position of the first new token (may lie before 0)
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
                if (!there[kt]) continue;
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
            float sum[KT] = {}, part[KT] = {};
            const int64_t rows = static_cast<int64_t>(n) * a.rep;
            const int64_t at = (static_cast<int64_t>(h) * a.sq.tokens + start) * a.rep;   // the rows' place in `query`
            int64_t p0 = 0, p1 = rows;     // rows that see some key of the block
            if (a.causal) {
                p0 = max(static_cast<int64_t>(j0) - first, int64_t{0}) * a.rep;
                if (a.window) p1 = min(p1, (static_cast<int64_t>(j0) + S::KEYS - 1 - first + a.window) * a.rep);
            }
            int stages = 0;
            for (int64_t p = p0 / kRows * kRows; p < p1; p += kRows) {
                __syncthreads();
                constexpr int WORDS = kRows * D / 4;            // 16 bytes each
#pragma unroll
                for (int i = 0; i < WORDS / 256; ++i) {
                    const int x = i * 256 + tid, r = x / (D / 4), c = x % (D / 4);
                    const uint4v v = reinterpret_cast<const uint4v*>(query + (at + min(p + r, rows - 1)) * D)[c];
                    *reinterpret_cast<uint4v*>(stage + r * S::STRIDE + c * 16) = v;
                }
                if (tid < kRows) {
                    RowInfo ri;
                    const int64_t r = min(p + tid, rows - 1);
                    const RowScale rs = scales[at + r];
                    const int pos = first + static_cast<int>(static_cast<uint32_t>(r) / a.rep);
                    ri.factor = rs.factor;
                    ri.lse = rs.lse;
                    ri.lo = a.window ? max(pos - a.window + 1, 0) : 0;
                    ri.hi = p + tid < rows ? (a.causal ? min(pos + 1, len) : len) : 0;
                    info[tid] = ri;
                }
                __syncthreads();
                // whether every row of the stage is there and sees every key of the block
                const int pos0 = first + static_cast<int>(static_cast<uint32_t>(p) / a.rep);
                const int pos1 = first + static_cast<int>(static_cast<uint32_t>(min(p + kRows, rows) - 1) / a.rep);
                const bool full = p + kRows <= rows && j0 + S::KEYS <= len && (!a.causal || j0 + S::KEYS - 1 <= pos0) &&
                                  (!a.window || j0 > pos1 - a.window);
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
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        if (!there[kt]) continue;
                        float4v w = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int q = 0; q < NG; ++q) {
                            float4v c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int i = 0; i < KG; ++i) {
                                c = mfma(ql[q * KG + i], key[kt][q * KG + i], c);
                                c = mfma(qh[q * KG + i], key[kt][q * KG + i], c);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = q ? __builtin_fmaf(c[i], scale[kt][q], w[i]) : c[i] * scale[kt][0];
                        }
                        const int j = j0 + (wave * KT + kt) * 16 + m;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float e = __builtin_amdgcn_exp2f(__builtin_fmaf(w[i], ri[i].factor, -ri[i].lse));
                            if (!full) e = j >= ri[i].lo && j < ri[i].hi ? e : 0.0f;
                            part[kt] += e;
                        }
                    }
                }
                // sums of 16 stages apart, so that a long sum loses less
                if (++stages % 16 == 0) {
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        sum[kt] += part[kt];
                        part[kt] = 0.0f;
                    }
                }
            }
            float* out = a.weights + (static_cast<int64_t>(b) * pg.hkv + h) * a.width;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                float v = sum[kt] + part[kt];
                v += __shfl_xor(v, 16);
                v += __shfl_xor(v, 32);
                const int j = j0 + (wave * KT + kt) * 16 + m;
                if (g == 0 && j < len) out[j] = (j < first ? a.decay * out[j] : 0.0f) + v;
            }
        }
        mine -= total;
    }
}

template <int D, class T>
void query_launch(const CacheWeightsArgs& a, uint32_t* out, RowScale* rows, hipStream_t s) {
    const int64_t threads = int64_t{a.sq.tokens} * a.hq * (D / 16);
    hipLaunchKernelGGL((weights_query<D, T>), dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0, s, a, out, rows);
}

template <int D, int NG>
void add_launch(const CacheWeightsArgs& a, int bf16, hipStream_t s) {
    RowScale* rows = reinterpret_cast<RowScale*>(a.work);
    uint32_t* query = reinterpret_cast<uint32_t*>(a.work + (int64_t{a.sq.tokens} * a.hq * 8 + 15) / 16 * 16);
    if (bf16) query_launch<D, uint16_t>(a, query, rows, s);
    else query_launch<D, float>(a, query, rows, s);
    hipLaunchKernelGGL((weights_add<D, NG>), dim3(a.workers), dim3(256), 0, s, a, query, rows);
}

}  // namespace

int cache_weights_workers(int* workers) {
    int dev, cus;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e == hipSuccess) *workers = 4 * cus;
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
