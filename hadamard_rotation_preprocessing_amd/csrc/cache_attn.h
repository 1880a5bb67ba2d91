// Attention over the paged 4-bit cache (hr_cache_attention): kernels for one
// head dimension, instantiated by cache_attn_64/128/256.hip.
//
// Mathematics.  With a key k = s (c - z) (codes c, zero point z, scale s of
// its group) a score is q . k = sum over groups of s (q . c - z sum(q)): the
// matrix product runs over the integer codes, and scale and zero point are
// applied to its 16 x 16 results.  The softmax is taken in one pass: a running
// maximum m, l = sum exp(w - m) and o = sum exp(w - m) v, rescaled when m
// grows.  With one group per vector the value's scale multiplies the
// probability, so that o is a matrix product over the integers c - z too;
// with several groups it multiplies the values.
//
// Layout.  No tile is staged: a wave turns the packed codes it has loaded into
// operands of v_mfma_f32_16x16x32_f16 in its registers.
//   Scores are formed transposed, S^T = K Q^T: the codes are the A operand
//   (lane l: key l & 15), the queries the B operand.  The result has the query
//   in the lane (l & 15) and four consecutive keys 4 (l >> 4) + r in its
//   registers, so a query's statistics are one value per lane, and two 16-key
//   results are the B operand of O^T = V^T P^T as they stand: its eight k slots
//   of lane group g are the keys 4g + r and 16 + 4g + r.
//   For V^T (A operand: dimension in the lane, keys in the slots) a lane loads
//   the same 32-bit word of its eight keys' rows; v_perm_b32 puts the same byte
//   of two keys side by side, and one AND leaves two keys' codes of one
//   dimension.
// A nibble in the low bits of a half is a float16 subnormal, c 2^-24 (at bit 4:
// c 2^-20), exactly, and so are differences of two: the codes become operands
// without a conversion.  The matrix unit aligns a subnormal's products by its
// exponent field, so these keep some ten bits less of a sum: measured, 4e-6 to
// 7e-6 of a result's norm against 1e-6, far below bfloat16's 1.7e-3.  float32
// activations and scaled values (several groups) take ordinary numbers
// instead: ORed with 1024 (at bit 4: 64), c is the float16 1024 + c, and a
// subtraction leaves c or c - z.  Queries and probabilities are scaled by
// powers of two to use float16's range, and the sums are float32.
//
// Split.  A unit is a kv head of a sequence with a block of its query rows
// (new tokens x query heads of that kv head).  Units are cut into items of as
// many keys as a workgroup's waves take at once, and every workgroup takes an
// equal, contiguous run of all items, whatever the lengths; partial results
// are joined in key order by cache_attn_join.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "cache.h"
#include "plan.h"

namespace hr {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float4v mfma(uint4v a, uint4v b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pk_sub(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, a) - __builtin_bit_cast(half2v, b));
}
__device__ __forceinline__ uint32_t pk_mul(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, a) * __builtin_bit_cast(half2v, b));
}
__device__ __forceinline__ uint32_t pk_fma(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2v, a), __builtin_bit_cast(half2v, b),
                                                                  __builtin_bit_cast(half2v, c)));
}
// two floats -> two float16 (nearest even), the first in the low half
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    half2v h;
    h.x = static_cast<_Float16>(a);
    h.y = static_cast<_Float16>(b);
    return __builtin_bit_cast(uint32_t, h);
}
__device__ __forceinline__ float lo_f32(uint32_t h) { return static_cast<float>(__builtin_bit_cast(half2v, h).x); }
__device__ __forceinline__ float hi_f32(uint32_t h) { return static_cast<float>(__builtin_bit_cast(half2v, h).y); }

// sum and maximum over the four lane groups of a query (lanes l, l + 16, ...)
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float max_groups(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

// bf16 (finite or not) from float32, nearest even, NaN kept
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

constexpr float kLow = -3.0e38f;      // running maximum of nothing
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPExp = 9;              // probabilities are at most 2^kSlack and carry 2^kPExp in float16
constexpr float kSlack = 6.0f;        // how far (log2) a score may pass the running maximum before it moves
constexpr int kSExp = 8;              // value scales (several groups) carry 2^kSExp

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
    r.len = min(max(s.lens[b], 0), s.max_pages << logp);
    return r;
}

// Key ranges of query rows [r0, r1) of a sequence: [lo, hi) holds every key
// that some row sees, [flo, fhi) those that all rows see.
struct Span {
    int lo, hi, flo, fhi;
};
__device__ __forceinline__ Span span_of(const CacheAttnArgs& a, const Seq& s, int r0, int r1) {
    Span p;
    const int first = s.len - s.n + r0 / a.rep, last = s.len - s.n + (r1 - 1) / a.rep;
    p.hi = a.causal ? min(max(last + 1, 0), s.len) : s.len;
    p.fhi = a.causal ? min(max(first + 1, 0), s.len) : s.len;
    p.lo = a.window ? max(first - a.window + 1, 0) : 0;
    p.flo = a.window ? max(last - a.window + 1, 0) : 0;
    return p;
}

template <int D_, int NG_, bool SF32_, bool WIDE_, int RT_, int WR_>
struct Cfg {
    static constexpr int D = D_, NG = NG_, RT = RT_, WR = WR_, WT = 4 / WR_;
    static constexpr bool SF32 = SF32_, WIDE = WIDE_;
    static constexpr int KS = D / 32;              // matrix steps over a vector
    static constexpr int KG = KS / NG;             // of one group
    static constexpr int DT = D / 16;              // dimension tiles of O^T
    static constexpr int VW = D == 256 ? 2 : 1;    // 32-bit words of a V row per lane (64: half a word)
    static constexpr int ROWS = 16 * RT * WR;      // query rows of a unit
    static constexpr int KEYS = 32 * WT;           // keys of an item
    static constexpr int ES = SF32 ? 4 : 2;
    static constexpr int KSW = NG * ES;            // 32-bit words of four positions' scales
    static constexpr int ZW = (NG + 1) / 2;        // 32-bit words of four positions' zero points (one group: 16 bits)
    static constexpr int VSN = NG == 1 ? KSW : 8;  // words of value scales per 16 (one group) or 32 keys
    static constexpr int P = WIDE ? 2 : 1;         // float16 terms of an operand
    static constexpr bool SUBK = !WIDE;            // subnormal codes of K
    static constexpr bool SUBV = !WIDE && NG == 1; // and of V
};

// What a wave holds of 32 keys before it works on them.
template <class C>
struct Raw {
    uint32_t k[2][C::KS];
    uint32_t ks[2][C::KSW];
    uint32_t kz[2][C::ZW];
    uint32_t v[8][C::VW];
    uint32_t vs[C::NG == 1 ? 2 : 8][C::NG == 1 ? C::KSW : 1];
    uint32_t vz[C::NG == 1 ? 2 : 8];
    int here;   // bit a: subtile a's page is present
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2v x = *reinterpret_cast<const uint2v*>(p);
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4v x = *reinterpret_cast<const uint4v*>(p + 4 * i);
            w[i] = x.x;
            w[i + 1] = x.y;
            w[i + 2] = x.z;
            w[i + 3] = x.w;
        }
    }
}

// Loads 32 keys from t0 (a multiple of 16).  Pages outside the pool are
// read as page 0 and marked absent; t0 is below the table's last position.
template <class C>
__device__ __forceinline__ void load_keys(const CacheAttnArgs& a, const int32_t* table, int h, int t0, Raw<C>& w) {
    constexpr int D = C::D, NG = C::NG;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    w.here = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int t = t0 + 16 * s;
        const int slot = min(t >> a.pg.logp, a.sq.max_pages - 1);
        int page = table[slot];
        if (static_cast<uint32_t>(page) < static_cast<uint64_t>(a.sq.n_pages)) w.here |= 1 << s;
        else page = 0;
        const uint8_t* base = a.pool + page * a.pg.page_bytes + h * a.pg.head_bytes;
        const int off = t & (a.pg.page - 1);
        // keys: a lane holds D/4 dimensions of key m, one run with one group,
        // eight of every 32 with several (a matrix step is then one group's)
        const uint8_t* kp = base + a.pg.kc + (off + m) * (D / 2);
        if constexpr (NG == 1) {
            load_words<C::KS>(kp + g * (D / 8), w.k[s]);
        } else {
#pragma unroll
            for (int i = 0; i < C::KS; ++i) load_words<1>(kp + i * 16 + g * 4, &w.k[s][i]);
        }
        load_words<C::KSW>(base + a.pg.ks + (off + 4 * g) * (NG * C::ES), w.ks[s]);
        if (!a.pg.sym) {
            const uint8_t* zp = base + a.pg.kz + (off + 4 * g) * NG / 2;
            if constexpr (NG == 1) w.kz[s][0] = *reinterpret_cast<const uint16_t*>(zp);
            else load_words<C::ZW>(zp, w.kz[s]);
        }
        // values: D/16 dimensions of keys 4g + r
        const uint8_t* vp = base + a.pg.vc + (off + 4 * g) * (D / 2) + m * (D / 32);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (D == 64) w.v[4 * s + r][0] = *reinterpret_cast<const uint16_t*>(vp + r * (D / 2));
            else load_words<C::VW>(vp + r * (D / 2), w.v[4 * s + r]);
        }
        if constexpr (NG == 1) {
            load_words<C::KSW>(base + a.pg.vs + (off + 4 * g) * C::ES, w.vs[s]);
            if (!a.pg.sym) w.vz[s] = *reinterpret_cast<const uint16_t*>(base + a.pg.vz + (off + 4 * g) / 2);
        } else {
            const int gi = m / (16 / NG);  // the lane's group
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int at = (off + 4 * g + r) * NG + gi;
                if constexpr (C::SF32) w.vs[4 * s + r][0] = *reinterpret_cast<const uint32_t*>(base + a.pg.vs + 4 * at);
                else w.vs[4 * s + r][0] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(base + a.pg.vs + 2 * at)) << 16;
                if (!a.pg.sym) w.vz[4 * s + r] = (base[a.pg.vz + at / 2] >> (4 * (at & 1))) & 15u;
            }
        }
    }
}

// scale r (of word-packed float32 or bfloat16 scales)
template <bool SF32>
__device__ __forceinline__ float scale_at(const uint32_t* w, int i) {
    if constexpr (SF32) return __uint_as_float(w[i]);
    return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

// Four operand words of eight codes: (0,4) (1,5) (2,6) (3,7).  Subnormal: in
// units of 2^-24, the second and fourth word with a factor of 16.
template <bool SUB>
__device__ __forceinline__ uint4v code_operand(uint32_t w) {
    uint4v f;
    if constexpr (!SUB) {
        f.x = pk_sub((w & 0x000F000Fu) | 0x64006400u, 0x64006400u);
        f.y = pk_sub((w & 0x00F000F0u) | 0x54005400u, 0x54005400u);
        w >>= 8;
        f.z = pk_sub((w & 0x000F000Fu) | 0x64006400u, 0x64006400u);
        f.w = pk_sub((w & 0x00F000F0u) | 0x54005400u, 0x54005400u);
        return f;
    }
    f.x = w & 0x000F000Fu;
    f.y = w & 0x00F000F0u;
    w >>= 8;
    f.z = w & 0x000F000Fu;
    f.w = w & 0x00F000F0u;
    return f;
}

// The state of a wave's rows: queries as operands and the running softmax.
template <class C>
struct Rows {
    uint4v q[C::RT][C::P][C::KS];
    float qsum[C::RT][C::NG];   // sum of a group's queries (as float16), over the whole vector, in raw units
    float c[C::RT];             // log2 units of one unit of a raw score
    float slack[C::RT];         // kSlack in raw units
    int lim[C::RT], lo[C::RT];  // keys [lo, lim) are seen
    float m[C::RT], mc[C::RT];  // running maximum, raw and in log2 units
    float l[C::RT];             // sum of exponentials (this lane's keys)
    float4v o[C::RT][C::DT];
    int e;                      // exponent of the value scales in o
};

// Loads rows r0 + 16 rt + (lane & 15) of kv head h, rotates them and makes
// them operands.  Rows past the sequence's repeat its last one.
template <class C, class T>
__device__ void load_rows(const CacheAttnArgs& a, const Seq& s, int h, int r0, Rows<C>& w) {
    constexpr int D = C::D, N = D / 4;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        const int row = min(r0 + 16 * rt + n, s.n * a.rep - 1);
        const int tok = row / a.rep, hh = row - tok * a.rep;
        const T* p = static_cast<const T*>(a.q) + static_cast<int64_t>(s.start + tok) * a.q_st +
                     static_cast<int64_t>(h * a.rep + hh) * a.q_sh;
        const int pos = s.len - s.n + tok;
        w.lim[rt] = a.causal ? min(pos + 1, s.len) : s.len;
        w.lo[rt] = a.window ? pos - a.window + 1 : 0;
        float v[N];
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const int at = C::NG == 1 ? g * N + i * 8 : i * 32 + g * 8;
            if constexpr (sizeof(T) == 2) {
                uint32_t x[4];
                load_words<4>(reinterpret_cast<const uint8_t*>(p + at), x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[8 * i + 2 * j] = __uint_as_float(x[j] << 16);
                    v[8 * i + 2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
                }
            } else {
                uint32_t x[8];
                load_words<8>(reinterpret_cast<const uint8_t*>(p + at), x);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[8 * i + j] = __uint_as_float(x[j]);
            }
        }
        if (a.rotate) {
            // H over the dimension's bits: those inside the lane, then the two
            // that are the lane group's
#pragma unroll
            for (int st = 1; st < N; st *= 2)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (!(j & st)) {
                        const float x = v[j], y = v[j + st];
                        v[j] = x + y;
                        v[j + st] = x - y;
                    }
#pragma unroll
            for (int st = 16; st < 64; st *= 2)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float y = __shfl_xor(v[j], st);
                    v[j] = (lane & st) ? y - v[j] : v[j] + y;
                }
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] *= a.norm;
        }
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) top = fmaxf(top, fabsf(v[j]));
        top = max_groups(top);
        // the largest element at 2^10 .. 2^11 of float16; rows of infinities
        // keep their exponent (they give NaN all the same)
        int e = 0;
        if (top > 0.0f && top < __builtin_inff()) e = min(max(11 - (static_cast<int>(__float_as_uint(top) >> 23) - 126), -100), 100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        w.c[rt] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + (C::SUBK ? 24 : 0) - e) << 23);
        w.slack[rt] = kSlack / w.c[rt];
        float sum[C::NG];
#pragma unroll
        for (int i = 0; i < C::NG; ++i) sum[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < C::KS; ++i) {
            // order of code_operand; with subnormal codes the elements of
            // its second and fourth word lose the 16 that the codes there
            // carry, and the unit 2^-24 stays in the raw scores: c has its
            // inverse.
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = C::SUBK && (j & 1) ? up * 0.0625f : up;
                const float x = v[8 * i + j] * f, y = v[8 * i + j + 4] * f;
                hi[j] = pack_f16(x, y);
                float back = lo_f32(hi[j]) + hi_f32(hi[j]);
                if constexpr (C::WIDE) {
                    lo[j] = pack_f16(x - lo_f32(hi[j]), y - hi_f32(hi[j]));
                    back += lo_f32(lo[j]) + hi_f32(lo[j]);
                }
                sum[C::NG == 1 ? 0 : i / C::KG] += C::SUBK && (j & 1) ? back * 16.0f : back;
            }
            w.q[rt][0][i] = uint4v{hi[0], hi[1], hi[2], hi[3]};
            if constexpr (C::WIDE) w.q[rt][1][i] = uint4v{lo[0], lo[1], lo[2], lo[3]};
        }
#pragma unroll
        for (int i = 0; i < C::NG; ++i) w.qsum[rt][i] = sum_groups(sum[i]) * (C::SUBK ? 0x1p-24f : 1.0f);
        w.m[rt] = kLow;
        w.mc[rt] = kLow;
        w.l[rt] = 0.0f;
#pragma unroll
        for (int j = 0; j < C::DT; ++j) w.o[rt][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    w.e = -100;
}

// One step over 32 keys.  MASK: some of them are not seen by every row.
template <class C, bool MASK>
__device__ __forceinline__ void step(const CacheAttnArgs& a, Raw<C>& w, int t0, Rows<C>& st) {
    constexpr int NG = C::NG, RT = C::RT;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const bool sym = a.pg.sym;
    if (sym) {  // two's complement nibbles: c + 8, zero point 8
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < C::KS; ++i) w.k[s][i] ^= 0x88888888u;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int i = 0; i < C::VW; ++i) w.v[t][i] ^= 0x88888888u;
    }
    // raw scores: sc[rt][4 s + r] of key t0 + 16 s + 4 g + r
    float sc[RT][8];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            float4v acc[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = gi * C::KG; i < (gi + 1) * C::KG; ++i) {
                const uint4v f = code_operand<C::SUBK>(w.k[s][i]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    acc[rt] = mfma(f, st.q[rt][0][i], acc[rt]);
                    if constexpr (C::WIDE) acc[rt] = mfma(f, st.q[rt][1][i], acc[rt]);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float ks = scale_at<C::SF32>(w.ks[s], r * NG + gi);
                const int nib = r * NG + gi;
                const float kz = sym ? 8.0f : static_cast<float>((w.kz[s][nib / 8] >> (4 * (nib & 7))) & 15u);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float x = fmaf(-kz, st.qsum[rt][gi], acc[rt][r]);
                    if constexpr (NG == 1) sc[rt][4 * s + r] = x * ks;
                    else sc[rt][4 * s + r] = gi == 0 ? x * ks : fmaf(x, ks, sc[rt][4 * s + r]);
                }
            }
        }
    }
    bool seen[RT][8];
    if constexpr (MASK) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = t0 + 16 * s + 4 * g + r;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    seen[rt][4 * s + r] = ((w.here >> s) & 1) && t < st.lim[rt] && t >= st.lo[rt];
                    if (!seen[rt][4 * s + r]) sc[rt][4 * s + r] = -__builtin_inff();
                }
            }
    }
    // value scales of the lane's keys; those that no row of the wave may see
    // (past the sequence or on an absent page) are not looked at
    float vs[8];
    uint32_t nz[8];   // several groups: zero points
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if constexpr (NG == 1) vs[t] = scale_at<C::SF32>(w.vs[t / 4], t & 3);
        else vs[t] = __uint_as_float(w.vs[t][0]);
        if constexpr (MASK) {
            bool any = false;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) any |= seen[rt][t];
            // (several groups: the scale goes into the operand that all 16
            // queries share, so it must be dropped only if none sees the key)
            if constexpr (NG == 1) {
                if (!any) vs[t] = 0.0f;
            } else if (__ballot(any) == 0) {
                vs[t] = 0.0f;
            }
        }
    }
    // the exponent of the value scales: grows to cover the largest
    float big = 0.0f;
#pragma unroll
    for (int t = 0; t < 8; ++t) big = fmaxf(big, fabsf(vs[t]) < __builtin_inff() ? fabsf(vs[t]) : 0.0f);
    const float cover = __uint_as_float(static_cast<uint32_t>(127 + st.e) << 23);
    if (__any(big > cover)) {
        big = max_groups(big);
#pragma unroll
        for (int x = 1; x < 16; x *= 2) big = fmaxf(big, __shfl_xor(big, x));
        const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 126, -100), 127);
        const int eu = __builtin_amdgcn_readfirstlane(e);
        const float f = ldexpf(1.0f, st.e - eu);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int j = 0; j < C::DT; ++j) st.o[rt][j] *= f;
        st.e = eu;
    }
    const float down = ldexpf(1.0f, (NG == 1 ? kPExp : kSExp) - st.e);
#pragma unroll
    for (int t = 0; t < 8; ++t) vs[t] *= down;
    if constexpr (NG > 1) {
#pragma unroll
        for (int t = 0; t < 8; ++t) nz[t] = sym ? 8u : w.vz[t];
        // a scale that is not finite must reach the queries that see its key
        // and no others: it leaves the shared operand, and their probability
        // becomes NaN instead
        bool odd = false;
#pragma unroll
        for (int t = 0; t < 8; ++t) odd |= !(fabsf(vs[t]) < __builtin_inff());
        if (__any(odd)) {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                int bad = !(fabsf(vs[t]) < __builtin_inff());
                if (bad) vs[t] = 0.0f;
#pragma unroll
                for (int x = 1; x < 16; x *= 2) bad |= __shfl_xor(bad, x);
                if (bad) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        if (sc[rt][t] > -__builtin_inff()) sc[rt][t] = __builtin_nanf("");
                }
            }
        }
    }
    // softmax: probabilities as operands
    uint4v ph[RT], pl[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        float top = sc[rt][0];
#pragma unroll
        for (int t = 1; t < 8; ++t) top = fmaxf(top, sc[rt][t]);
        if (__any(top > st.m[rt] + st.slack[rt])) {
            top = fmaxf(max_groups(top), st.m[rt]);
            const float mc = top > kLow ? top * st.c[rt] : kLow;
            const float f = exp2f(st.mc[rt] - mc);
            st.m[rt] = top;
            st.mc[rt] = mc;
            st.l[rt] *= f;
#pragma unroll
            for (int j = 0; j < C::DT; ++j) st.o[rt][j] *= f;
        }
        float p[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float x = __builtin_amdgcn_exp2f(fmaf(sc[rt][t], st.c[rt], -st.mc[rt]));
            if constexpr (MASK)
                if (!seen[rt][t]) x = 0.0f;   // (a row that has seen nothing yet has no usable m)
            st.l[rt] += x;
            if constexpr (NG == 1) p[t] = x * vs[t];
            else p[t] = x * static_cast<float>(1 << kPExp);
            if constexpr (MASK && NG == 1)
                if (!seen[rt][t]) p[t] = 0.0f;   // (nor may another row's infinite scale reach this one)
        }
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hw[i] = pack_f16(p[2 * i], p[2 * i + 1]);
            if constexpr (C::WIDE) lw[i] = pack_f16(p[2 * i] - lo_f32(hw[i]), p[2 * i + 1] - hi_f32(hw[i]));
        }
        ph[rt] = uint4v{hw[0], hw[1], hw[2], hw[3]};
        if constexpr (C::WIDE) pl[rt] = uint4v{lw[0], lw[1], lw[2], lw[3]};
    }
    // zero points of key pairs, in the low and in the second nibble
    uint32_t z0[4], z1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (NG == 1) {
            if (sym) {
                z0[i] = 0x00080008u;
            } else {
                const uint32_t u = w.vz[i / 2] >> (8 * (i & 1));
                z0[i] = ((u << 12) | u) & 0x000F000Fu;
            }
        } else {
            z0[i] = nz[2 * i] | (nz[2 * i + 1] << 16);
        }
        z1[i] = z0[i] << 4;
        if constexpr (!C::SUBV) {
            z0[i] |= 0x64006400u;
            z1[i] |= 0x54005400u;
        }
    }
    uint32_t s0[4], s1[4];   // several groups: the pairs' scales, and what float16 loses of them
    if constexpr (NG > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s0[i] = pack_f16(vs[2 * i], vs[2 * i + 1]);
            if constexpr (C::WIDE && C::SF32) s1[i] = pack_f16(vs[2 * i] - lo_f32(s0[i]), vs[2 * i + 1] - hi_f32(s0[i]));
        }
    }
    // O^T += V^T P^T, two dimensions a byte
#pragma unroll
    for (int b = 0; b < (C::D == 64 ? 2 : 4 * C::VW); ++b) {
        const uint32_t sel = 0x0C040C00u + 0x00010001u * (b & 3);
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __builtin_amdgcn_perm(w.v[2 * i + 1][b / 4], w.v[2 * i][b / 4], sel);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t f[4], fl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = x[i] & (half ? 0x00F000F0u : 0x000F000Fu);
                if constexpr (!C::SUBV) f[i] |= half ? 0x54005400u : 0x64006400u;
                f[i] = pk_sub(f[i], half ? z1[i] : z0[i]);
                if constexpr (NG > 1) {
                    const uint32_t d = f[i];
                    f[i] = pk_mul(d, s0[i]);
                    if constexpr (C::WIDE) {
                        fl[i] = pk_fma(d, s0[i], f[i] ^ 0x80008000u);
                        if constexpr (C::SF32) fl[i] = pk_fma(d, s1[i], fl[i]);
                    }
                }
            }
            const uint4v av = {f[0], f[1], f[2], f[3]};
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float4v& o = st.o[rt][2 * b + half];
                o = mfma(av, ph[rt], o);
                if constexpr (C::WIDE) {
                    o = mfma(av, pl[rt], o);
                    if constexpr (NG > 1) o = mfma(uint4v{fl[0], fl[1], fl[2], fl[3]}, ph[rt], o);
                }
            }
        }
    }
}

// A wave's share of keys [k0, k1) (k0 a multiple of 32) of a unit: every WT-th
// 32 of them.
template <class C>
__device__ __forceinline__ void walk(const CacheAttnArgs& a, const int32_t* table, int h, const Span& sp, int k0, int k1,
                                     int wt, Rows<C>& st) {
    k0 = max(k0, sp.lo & ~31);
    k1 = min(k1, sp.hi);
    for (int t = k0 + 32 * wt; t < k1; t += 32 * C::WT) {
        Raw<C> w;
        load_keys<C>(a, table, h, t, w);
        if (t >= sp.flo && t + 32 <= sp.fhi && w.here == 3) step<C, false>(a, w, t, st);
        else step<C, true>(a, w, t, st);
    }
}

// Writes a wave's finished rows, or its part of them to the scratch.
// o: sums in value units relative to m (raw scores times c = log2 units).
template <class C, class T>
__device__ __forceinline__ void put_rows(const CacheAttnArgs& a, const Seq& s, int h, int r0, const Rows<C>& st, float* part,
                                         int part_row) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        const int row = r0 + 16 * rt + n;
        if (row >= s.n * a.rep) continue;
        const float m2 = st.mc[rt], l = st.l[rt];
        if (part) {
            float* p = part + static_cast<int64_t>(part_row + 16 * rt + n) * (C::D + 2);
            if (g == 0) {
                p[0] = l > 0.0f || l != l ? m2 : kLow;
                p[1] = l;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < C::DT; j += 2)
                    *reinterpret_cast<float2*>(p + 2 + (4 * g + r) * C::DT + j) = make_float2(st.o[rt][j][r], st.o[rt][j + 1][r]);
            continue;
        }
        const int tok = row / a.rep, hh = row - tok * a.rep;
        const int64_t t = s.start + tok;
        const int64_t head = h * a.rep + hh;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T* p = static_cast<T*>(a.out) + t * a.o_st + head * a.o_sh;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < C::DT; j += 4) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = st.o[rt][j + i][r] * inv;
                T* to = p + (4 * g + r) * C::DT + j;
                if constexpr (sizeof(T) == 2)
                    *reinterpret_cast<uint2v*>(to) =
                        uint2v{to_bf16(x[0]) | (to_bf16(x[1]) << 16), to_bf16(x[2]) | (to_bf16(x[3]) << 16)};
                else *reinterpret_cast<float4v*>(to) = float4v{x[0], x[1], x[2], x[3]};
            }
        if (a.lse && g == 0) a.lse[t * a.hq + head] = l == 0.0f ? -__builtin_inff() : (m2 + __log2f(l)) * 0.6931471805599453f;
    }
}

// Ends a wave's rows: sums over the lane groups, and o in value units.
template <class C>
__device__ __forceinline__ void settle(Rows<C>& st) {
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        st.l[rt] = sum_groups(st.l[rt]);
        const int f = (C::SUBV ? 24 : C::NG > 1 ? -kSExp : 0) - kPExp + st.e;
#pragma unroll
        for (int j = 0; j < C::DT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) st.o[rt][j][r] = ldexpf(st.o[rt][j][r], C::SUBV && (j & 1) ? f - 4 : f);
    }
}

// Joins the waves that took different keys of the same rows: all get the
// common maximum, then halves add up through LDS.  The result is wave 0's.
template <class C>
__device__ __forceinline__ void join_waves(Rows<C>& st, float* lds) {
    static_assert(C::WT == 4 && C::WR == 1, "four waves along the keys");
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    float* ml = lds;                                       // [4][RT * 16]
    float* buf = lds + 4 * C::RT * 16;                     // [2][RT][DT][64] float4
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt)
        if (g == 0) ml[wave * C::RT * 16 + rt * 16 + n] = st.mc[rt];
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        float top = kLow;
        for (int x = 0; x < 4; ++x) top = fmaxf(top, ml[x * C::RT * 16 + rt * 16 + n]);
        const float f = exp2f(st.mc[rt] - top);
        st.mc[rt] = top;
        st.l[rt] *= f;
#pragma unroll
        for (int j = 0; j < C::DT; ++j) st.o[rt][j] *= f;
    }
    constexpr int W = C::RT * (C::DT * 4 + 1) * 64;        // floats of one wave's rows
    for (int half = 2; half >= 1; half /= 2) {
        if (wave >= half && wave < 2 * half) {
            float* p = buf + (wave - half) * W + lane;
#pragma unroll
            for (int rt = 0; rt < C::RT; ++rt) {
#pragma unroll
                for (int j = 0; j < C::DT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[((rt * C::DT + j) * 4 + r) * 64] = st.o[rt][j][r];
                p[(C::RT * C::DT * 4 + rt) * 64] = st.l[rt];
            }
        }
        __syncthreads();
        if (wave < half) {
            const float* p = buf + wave * W + lane;
#pragma unroll
            for (int rt = 0; rt < C::RT; ++rt) {
#pragma unroll
                for (int j = 0; j < C::DT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) st.o[rt][j][r] += p[((rt * C::DT + j) * 4 + r) * 64];
                st.l[rt] += p[(C::RT * C::DT * 4 + rt) * 64];
            }
        }
        __syncthreads();
    }
}

template <class C>
constexpr int join_floats() {
    return C::WT == 1 ? 1 : 4 * C::RT * 16 + 2 * C::RT * (C::DT * 4 + 1) * 64;
}

// Rows [r0, r0 + ROWS) of kv head h of a sequence over the keys [k0, k1);
// part: where a partial result goes (else the rows are finished here).
template <class C, class T>
__device__ __forceinline__ void segment(const CacheAttnArgs& a, const Seq& s, int b, int h, int r0, int k0, int k1,
                                        float* part, float* lds) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wave % C::WR, wt = wave / C::WR;
    const int row = r0 + wr * 16 * C::RT;
    const int rows = min(row + 16 * C::RT, s.n * a.rep);
    if (C::WT == 1 && row >= rows) return;   // (no barriers along the rows)
    Rows<C> st;
    load_rows<C, T>(a, s, h, row, st);
    const Span sp = span_of(a, s, row, rows);
    walk<C>(a, a.sq.table + static_cast<int64_t>(b) * a.sq.max_pages, h, sp, k0, k1, wt, st);
    settle<C>(st);
    if constexpr (C::WT > 1) {
        join_waves<C>(st, lds);
        if (wave == 0) put_rows<C, T>(a, s, h, row, st, part, row - r0);
    } else {
        put_rows<C, T>(a, s, h, row, st, part, row - r0);
    }
}

// The items of a sequence: heads x row blocks x blocks of keys, at least one
// block of keys so that rows that see nothing are written too.
struct Items {
    int first, blocks, rbs;   // first key (a multiple of 32), key blocks, row blocks
    int64_t total;
};
template <class C>
__device__ __forceinline__ Items items_of(const CacheAttnArgs& a, const Seq& s) {
    Items it;
    it.rbs = (s.n * a.rep + C::ROWS - 1) / C::ROWS;
    it.first = 0;
    it.blocks = 1;
    if (s.n > 0) {
        const Span sp = span_of(a, s, 0, s.n * a.rep);
        it.first = min(sp.lo, sp.hi) & ~31;
        it.blocks = max((sp.hi - it.first + C::KEYS - 1) / C::KEYS, 1);
    }
    it.total = static_cast<int64_t>(a.pg.hkv) * it.rbs * it.blocks;
    return it;
}

// All items of the call, and the sequence that holds item `want` with the
// items before it.  Every thread of the workgroup takes part.
struct Place {
    int64_t total, before;
    int b;
};
template <class C, class F>
__device__ __forceinline__ Place place(const CacheAttnArgs& a, int64_t* lds, F want_of) {
    const int tid = threadIdx.x;
    int64_t sum = 0;
    for (int b = tid; b < a.sq.rows; b += 256) sum += items_of<C>(a, seq_at(a.sq, a.pg.logp, b)).total;
    // total over the workgroup
    for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
    __syncthreads();
    if ((tid & 63) == 0) lds[tid >> 6] = sum;
    __syncthreads();
    Place p;
    p.total = lds[0] + lds[1] + lds[2] + lds[3];
    const int64_t want = want_of(p.total);
    int64_t base = 0;
    p.b = a.sq.rows;
    p.before = p.total;
    for (int c = 0; c < a.sq.rows; c += 256) {
        const int b = c + tid;
        const int64_t own = b < a.sq.rows ? items_of<C>(a, seq_at(a.sq, a.pg.logp, b)).total : 0;
        int64_t inc = own;
        for (int x = 1; x < 64; x *= 2) {
            const int64_t y = __shfl_up(inc, x);
            if ((tid & 63) >= x) inc += y;
        }
        __syncthreads();
        if ((tid & 63) == 63) lds[tid >> 6] = inc;
        if (tid == 0) lds[4] = -1;
        __syncthreads();
        for (int x = 0; x < (tid >> 6); ++x) inc += lds[x];
        const int64_t chunk = lds[0] + lds[1] + lds[2] + lds[3];
        if (want >= base + inc - own && want < base + inc) {
            lds[4] = b;
            lds[5] = base + inc - own;
        }
        __syncthreads();
        if (lds[4] >= 0) {
            p.b = static_cast<int>(lds[4]);
            p.before = lds[5];
            break;
        }
        base += chunk;
    }
    __syncthreads();
    return p;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// How many workgroups share `total` items: at most one each.
__device__ __forceinline__ int64_t sharers(const CacheAttnArgs& a, int64_t total) {
    return total < a.workers ? (total > 0 ? total : 1) : a.workers;
}
// First item of workgroup w of nw.
__device__ __forceinline__ int64_t first_item(int64_t w, int64_t nw, int64_t total) { return w * total / nw; }

// The workgroup that holds item u.
__device__ __forceinline__ int64_t holder(int64_t u, int64_t nw, int64_t total) {
    int64_t w = u * nw / total;
    while (w + 1 < nw && first_item(w + 1, nw, total) <= u) ++w;
    while (w > 0 && first_item(w, nw, total) > u) --w;
    return w;
}

// Split form: workgroup w takes items [first_item(w), first_item(w + 1)).  A
// unit that it does not hold whole goes to scratch slot 2 w + 1 if it begins
// here, else 2 w.
template <class C, class T>
__global__ void __launch_bounds__(256) cache_attn_split(const CacheAttnArgs a) {
    __shared__ float lds[join_floats<C>() > 16 ? join_floats<C>() : 16];
    int64_t i0 = 0, i1 = 0;
    const Place p = place<C>(a, reinterpret_cast<int64_t*>(lds), [&](int64_t total) {
        const int64_t nw = sharers(a, total);
        if (blockIdx.x >= nw) return total;
        i0 = first_item(blockIdx.x, nw, total);
        i1 = first_item(blockIdx.x + 1, nw, total);
        return i0;
    });
    i0 = uniform64(i0);
    i1 = uniform64(i1);
    int64_t before = uniform64(p.before);
    for (int b = __builtin_amdgcn_readfirstlane(p.b); b < a.sq.rows && i0 < i1; ++b) {
        const Seq s = seq_at(a.sq, a.pg.logp, b);
        const Items it = items_of<C>(a, s);
        while (i0 < i1 && i0 < before + it.total) {
            const int64_t at = i0 - before;
            const int unit = static_cast<int>(at / it.blocks), k = static_cast<int>(at % it.blocks);
            const int64_t left = i1 - i0;
            const int end = left < it.blocks - k ? k + static_cast<int>(left) : it.blocks;
            const int h = unit / it.rbs, rb = unit % it.rbs;
            float* part = nullptr;
            if (k > 0 || end < it.blocks)
                part = a.work + (2 * static_cast<int64_t>(blockIdx.x) + (k == 0 ? 1 : 0)) * (C::ROWS * (C::D + 2));
            segment<C, T>(a, s, b, h, rb * C::ROWS, it.first + k * C::KEYS, it.first + end * C::KEYS, part, lds);
            i0 += end - k;
        }
        before += it.total;
    }
}

// Joins the parts of units that were cut: a workgroup for a row, its four
// waves along the parts, the lanes along the dimensions.
template <class C, class T>
__global__ void __launch_bounds__(256) cache_attn_join(const CacheAttnArgs a) {
    constexpr int D = C::D, E = D / 64;
    __shared__ int64_t lds[8];
    __shared__ float sm[4], sl[4], so[4][D];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    for (int64_t id = blockIdx.x; id < static_cast<int64_t>(a.sq.tokens) * a.hq; id += gridDim.x) {
        const int64_t token = id / a.hq;
        const int head = static_cast<int>(id % a.hq), h = head / a.rep;
        // the token's sequence: the last one that starts at or before it
        int b = 0;
        if (a.sq.cu) {
            int hi = a.sq.rows - 1;
            while (b < hi) {
                const int mid = (b + hi + 1) / 2;
                if (cu_at(a.sq, mid) <= token) b = mid;
                else hi = mid - 1;
            }
        } else {
            b = static_cast<int>(min(token / a.sq.per, static_cast<int64_t>(a.sq.rows - 1)));
        }
        const Seq s = seq_at(a.sq, a.pg.logp, b);
        if (token < s.start || token >= s.start + s.n) continue;
        const Items it = items_of<C>(a, s);
        // items before the sequence, and of the call
        int64_t sum = 0, pre = 0;
        for (int x = tid; x < a.sq.rows; x += 256) {
            const int64_t t = items_of<C>(a, seq_at(a.sq, a.pg.logp, x)).total;
            sum += t;
            if (x < b) pre += t;
        }
        for (int x = 1; x < 64; x *= 2) {
            sum += __shfl_xor(sum, x);
            pre += __shfl_xor(pre, x);
        }
        __syncthreads();
        if (lane == 0) {
            lds[wave] = sum;
            lds[4 + wave] = pre;
        }
        __syncthreads();
        const int64_t total = lds[0] + lds[1] + lds[2] + lds[3], before = lds[4] + lds[5] + lds[6] + lds[7];
        const int64_t nw = sharers(a, total);
        const int row = static_cast<int>(token - s.start) * a.rep + head % a.rep;
        const int rb = row / C::ROWS;
        const int64_t u0 = before + (static_cast<int64_t>(h) * it.rbs + rb) * it.blocks, u1 = u0 + it.blocks - 1;
        const int64_t w0 = holder(u0, nw, total), w1 = holder(u1, nw, total);
        if (w0 == w1) continue;   // finished by its workgroup
        const float* base = a.work + static_cast<int64_t>(row % C::ROWS) * (D + 2);
        float m = kLow, l = 0.0f, o[E];
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.0f;
        for (int64_t w = w0 + wave; w <= w1; w += 4) {
            const float* p = base + (2 * w + (w == w0 ? 1 : 0)) * (C::ROWS * (D + 2));
            const float pm = p[0], pl = p[1];
            const float top = fmaxf(m, pm);
            const float f = exp2f(m - top), pf = exp2f(pm - top);
            l = l * f + pl * pf;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = o[i] * f + p[2 + lane * E + i] * pf;
            m = top;
        }
        if (lane == 0) {
            sm[wave] = m;
            sl[wave] = l;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) so[wave][lane * E + i] = o[i];
        __syncthreads();
        float top = kLow;
        for (int x = 0; x < 4; ++x) top = fmaxf(top, sm[x]);
        l = 0.0f;
        for (int x = 0; x < 4; ++x) l += sl[x] * exp2f(sm[x] - top);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T* out = static_cast<T*>(a.out) + token * a.o_st + static_cast<int64_t>(head) * a.o_sh;
        if (tid < D) {
            float x = 0.0f;
            for (int y = 0; y < 4; ++y) x += so[y][tid] * exp2f(sm[y] - top);
            x *= inv;
            if constexpr (sizeof(T) == 2) out[tid] = static_cast<T>(to_bf16(x));
            else out[tid] = x;
        }
        if (a.lse && tid == 0)
            a.lse[token * a.hq + head] = l == 0.0f ? -__builtin_inff() : (top + __log2f(l)) * 0.6931471805599453f;
    }
}

// Whole form: a workgroup for each unit.  Unit u of a head belongs to the last
// sequence b with floor(cu(b) rep / ROWS) + b <= u; a sequence has at most
// as many units as that bound leaves it.
template <class C, class T>
__global__ void __launch_bounds__(256) cache_attn_whole(const CacheAttnArgs a) {
    const int u = blockIdx.x % a.units, h = blockIdx.x / a.units;
    auto first = [&](int b) { return static_cast<int64_t>(cu_at(a.sq, b)) * a.rep / C::ROWS + b; };
    int b = 0, hi = a.sq.rows - 1;
    while (b < hi) {
        const int mid = (b + hi + 1) / 2;
        if (first(mid) <= u) b = mid;
        else hi = mid - 1;
    }
    const Seq s = seq_at(a.sq, a.pg.logp, b);
    const int64_t rbs = (static_cast<int64_t>(s.n) * a.rep + C::ROWS - 1) / C::ROWS;
    // the last row blocks see the most keys: they go first
    const int64_t rb = rbs - 1 - (u - first(b));
    if (rb < 0 || rb >= rbs) return;
    segment<C, T>(a, s, b, h, static_cast<int>(rb) * C::ROWS, 0, s.len, nullptr, nullptr);
}

template <class C, class T>
int split_workers(int* workers) {
    static std::atomic<int> slots[kMaxDevices];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= kMaxDevices) return static_cast<int>(hipErrorInvalidDevice);
    int n = slots[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        int cus = 0, per = 0;
        if ((e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return static_cast<int>(e);
        if ((e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, cache_attn_split<C, T>, 256, 0)) != hipSuccess)
            return static_cast<int>(e);
        n = cus * (per > 0 ? per : 1);
        slots[dev].store(n, std::memory_order_relaxed);
    }
    *workers = n;
    return 0;
}

// One kernel family: launches it, or with workers set only asks how many
// workgroups it keeps in flight.
template <class C, class T>
int family(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    if (workers) return split_workers<C, T>(workers);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (k.split) {
        hipLaunchKernelGGL((cache_attn_split<C, T>), dim3(a->workers), dim3(256), 0, s, *a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return static_cast<int>(e);
        const int64_t rows = static_cast<int64_t>(a->sq.tokens) * a->hq;
        hipLaunchKernelGGL((cache_attn_join<C, T>), dim3(static_cast<uint32_t>(rows < (1 << 20) ? rows : 1 << 20)), dim3(256),
                           0, s, *a);
    } else if constexpr (C::WR == 4) {
        hipLaunchKernelGGL((cache_attn_whole<C, T>), dim3(static_cast<uint32_t>(a->units) * a->pg.hkv), dim3(256), 0, s, *a);
    } else {
        return static_cast<int>(hipErrorInvalidValue);
    }
    return static_cast<int>(hipGetLastError());
}

template <int D, int NG, bool SF32>
int pick_shape(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    if (k.wide) {
        if (k.wr == 1) return family<Cfg<D, NG, SF32, true, 1, 1>, float>(k, a, workers, stream);
        return family<Cfg<D, NG, SF32, true, 1, 4>, float>(k, a, workers, stream);
    }
    if (k.rt == 1 && k.wr == 1) return family<Cfg<D, NG, SF32, false, 1, 1>, uint16_t>(k, a, workers, stream);
    if constexpr (D == 256) {
        return family<Cfg<D, NG, SF32, false, 1, 4>, uint16_t>(k, a, workers, stream);
    } else {
        if (k.wr == 1) return family<Cfg<D, NG, SF32, false, 2, 1>, uint16_t>(k, a, workers, stream);
        return family<Cfg<D, NG, SF32, false, 2, 4>, uint16_t>(k, a, workers, stream);
    }
}

template <int D, int NG>
int pick_scales(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    return k.sf32 ? pick_shape<D, NG, true>(k, a, workers, stream) : pick_shape<D, NG, false>(k, a, workers, stream);
}

}  // namespace
}  // namespace hr
