// Attention over the paged 4-bit cache (hr_cache_attention): kernels for one
// head dimension, instantiated by cache_attn_64/128/256.hip.
//
// Mathematics.  With a key k = s (c - z) (codes c, zero point z, scale s of
// its group) a score is q . k = sum over groups of s (q . c - z sum(q)): the
// matrix product runs over the integer codes, with one more step for
// z . -sum(q), and s is applied to its 16 x 16 results.  The softmax is taken
// in one pass: a running maximum m, l = sum exp(w - m) and o = sum exp(w - m) v.
// m only has to keep the exponentials in range, so it moves when one passes
// 2^kSlack, and everything is rescaled then: the test is on the exponentials
// themselves, and scores are not formed otherwise.  With one group per vector
// the value's scale multiplies the probability, so that o is a matrix product
// over the integers c - z too; with several groups it multiplies the values.
//
// Layout.  With few rows no tile is staged: a wave turns the packed codes it has
// loaded into operands of v_mfma_f32_16x16x32_f16 in its registers.  With many
// rows the waves take different rows of the same keys, and an operand is made
// once for all of them, in LDS (see Tile).
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
// many keys as a workgroup takes at once, and every workgroup takes an equal,
// contiguous run of all items, whatever the lengths; partial results are joined
// in key order by cache_attn_join.  Where there are units enough the kernel of many
// rows shares them out whole instead (kCut).
//
// What bounds it.  Few rows: the bytes of the cache, and at small sizes some ten
// microseconds for the chain from the lengths to the first keys, the merge of the
// waves and the joining launch.  One token in each of 16 sequences of 2048
// positions, 32 kv heads of 128 (140 MB): 39 us, 3.6 TB/s where a large copy has
// 4.95 (28 us); 24 sequences of up to 32768, 8 kv heads (132 MB): 42 us; one of 331:
// 16 us.  Heads of 256 do not fit the registers with several groups (16 sequences of
// 4000, 8 kv heads: 41 us with one group, 60, 115 and 252 with groups of 128, 64 and
// 32, which spill 12 to 284 registers; 376 with float32 scales, 490).
// Many rows: neither unit alone, see Tile.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "cache.h"
#include "plan.h"

namespace hr {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfloat8 __attribute__((ext_vector_type(8)));
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

// Two floats as pairs of float16: hi, and what it loses of them.  They pass an
// empty asm as values: a product would be rounded to float16 in one instruction
// where it makes hi, and through float32 where lo takes hi from it, which in one
// of some thousand elements are neighbouring numbers, 2^-11 apart.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
    asm("" : "+v"(a), "+v"(b));
    hi = pack_f16(a, b);
    lo = pack_f16(a - lo_f32(hi), b - hi_f32(hi));
}

// The value of lane ^ X inside 32 lanes: a swizzle, whose pattern is in the
// instruction (a general shuffle would hold its addresses in registers).
template <int X>
__device__ __forceinline__ uint32_t swizzle_xor(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(v), (X << 10) | 0x1F));
}
template <int X>
__device__ __forceinline__ float swizzle_xor(float v) {
    return __uint_as_float(swizzle_xor<X>(__float_as_uint(v)));
}
// f over the values of lanes l and l + 32, and over those of rows of 16 lanes
// 2 i and 2 i + 1: one register exchange each
template <class F>
__device__ __forceinline__ float over_halves(float v, F f) {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
template <class F>
__device__ __forceinline__ float over_rows(float v, F f) {
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
struct Sum {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
// over the four lane groups of a query (lanes l, l + 16, ...)
__device__ __forceinline__ float sum_groups(float v) { return over_halves(over_rows(v, Sum()), Sum()); }
__device__ __forceinline__ float max_groups(float v) { return over_halves(over_rows(v, Max()), Max()); }
// over the wave
__device__ __forceinline__ float max_wave(float v) {
    v = fmaxf(v, swizzle_xor<1>(v));
    v = fmaxf(v, swizzle_xor<2>(v));
    v = fmaxf(v, swizzle_xor<4>(v));
    v = fmaxf(v, swizzle_xor<8>(v));
    return max_groups(v);
}

// bf16 (finite or not) from float32, nearest even, NaN kept
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// The phases of a step stay in order: left alone, the scheduler forms all
// operands of a step at once, and spills.
#define HR_PHASE() __builtin_amdgcn_sched_barrier(0)
// A rare case stays a branch, instead of being computed always and selected.
#define HR_BRANCH() asm volatile("")

constexpr float kLow = -3.0e38f;      // running maximum of nothing
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPExp = 9;              // probabilities are at most 2^kSlack and carry 2^kPExp in float16
constexpr int kSlack = 6;             // how far (log2) a score may pass the running maximum before it moves
constexpr int kSExp = 8;              // value scales (several groups) carry 2^kSExp
constexpr int kFar = 32;              // value scales outside 2^-kFar .. 2^kFar are set aside
constexpr int kNoUnit = -10000;       // the unit of value scales before the first of them

// Integers read at an address that is the same in all lanes: through the scalar
// cache, into scalar registers.
typedef const int32_t __attribute__((address_space(4)))* ConstInts;

// A sequence of the call, clamped so that nothing leaves its buffer.  UNI: b is
// the same in all lanes.
struct Seq {
    int start, n, len;
};
template <bool UNI>
__device__ __forceinline__ int int_at(const int32_t* p, int64_t i) {
    if constexpr (UNI) return ((ConstInts)(p))[i];
    return p[i];
}
template <bool UNI>
__device__ __forceinline__ int cu_at(const CacheSeqs& s, int b) {
    const int c = s.cu ? int_at<UNI>(s.cu, b) : b * s.per;
    return min(max(c, 0), s.tokens);
}
template <bool UNI>
__device__ __forceinline__ Seq seq_at(const CacheSeqs& s, int logp, int b) {
    Seq r;
    r.start = cu_at<UNI>(s, b);
    r.n = max(cu_at<UNI>(s, b + 1) - r.start, 0);
    r.len = min(max(int_at<UNI>(s.lens, b), 0), s.max_pages << logp);
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
    static constexpr int D = D_, NG = NG_, RT = RT_, WR = WR_;
    static constexpr bool SF32 = SF32_, WIDE = WIDE_;
    static constexpr bool SHARED = WR > 1;         // keys become operands once for all waves
    static constexpr int THREADS = SHARED ? 64 * WR : 256;
    static constexpr int WT = SHARED ? 1 : 4;      // waves along the keys
    static constexpr int KS = D / 32;              // matrix steps over a vector
    static constexpr int KG = KS / NG;             // of one group
    static constexpr int DT = D / 16;              // dimension tiles of O^T
    static constexpr int VW = D == 256 ? 2 : 1;    // 32-bit words of a V row per lane (64: half a word)
    static constexpr int ROWS = 16 * RT * WR;      // query rows of a unit
    static constexpr int P = WIDE ? 2 : 1;         // float16 terms of an operand
    // shared: 32-key tiles of a pass, so that two passes' operands fit LDS
    static constexpr int TILES = P * D <= 128 ? 4 : P * D == 256 ? 2 : 1;
    static constexpr int KEYS = SHARED ? 32 * TILES : 32 * WT;  // keys of an item
    static constexpr int ES = SF32 ? 4 : 2;
    static constexpr int KSW = NG * ES;            // 32-bit words of four positions' scales
    static constexpr int WAVES = D == 64 && NG == 1 && RT == 1 && !SHARED ? 3 : 2;   // waves per SIMD
    static constexpr bool SUBK = !WIDE;            // subnormal codes of K
    static constexpr bool SUBV = !WIDE && NG == 1; // and of V
    static constexpr bool VLO = WIDE && NG > 1;    // scaled values as pairs of float16
    // How far (log2) value scales may lie below their unit, and scaled keys below
    // 2^12, and keep their bits in float16.  Values: scales carry 2^kSExp, down to
    // float16's smallest normal number, 2^-14, or for pairs to 2^-3; where they are
    // in probabilities, of which those far below 1 lose bits anyway, 2^14 or 2^10.
    static constexpr int VEXP = NG == 1 && !SHARED ? kPExp : kSExp;
    static constexpr int VRANGE = NG == 1 && !SHARED ? (WIDE ? 10 : 14) : (WIDE ? 10 : 21);
    static constexpr int KRANGE = WIDE ? 13 : 24;
};

// A workgroup's note of the segment it works on, in LDS, for sweep_rows.
struct Todo {
    int aside;               // whether it sets keys aside (0 between segments)
    int b, h, r0, k0, k1;
    float c;                 // of the rows, with shared operands
    float* part;             // where its rows go (nullptr: they are finished)
    float* spare;            // for the parts of rows that are finished but for such keys
    __device__ __forceinline__ void set(int b_, int h_, int r, int from, int to, float scale, float* p, float* sp) {
        b = b_;
        h = h_;
        r0 = r;
        k0 = from;
        k1 = to;
        c = scale;
        part = p;
        spare = sp;
    }
};

// What a wave holds of 32 keys before it works on them.
template <class C>
struct Raw {
    uint32_t k[2][C::KS];
    uint32_t ks[2][C::KSW];
    uint32_t kz[2];          // zero points of key m, a nibble for each group
    uint32_t v[8][C::VW];
    uint32_t vs[C::NG == 1 ? 2 : 8][C::NG == 1 ? C::KSW : 1];
    uint32_t vz[C::NG == 1 ? 2 : 8];
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

// The pages of the 16-key subtiles at t0 and t0 + 16 (uniform over the wave; t0
// a multiple of 16), out of range where absent.  A constant-address load, so
// that it goes through the scalar cache and leaves the vector loads' count.
struct Pages {
    int p[2];
};
__device__ __forceinline__ Pages pages_at(const CacheAttnArgs& a, const int32_t* table, int t0) {
    const ConstInts tab = (ConstInts)(table);
    Pages r;
    const int last = a.sq.max_pages - 1;
    r.p[0] = tab[min(t0 >> a.pg.logp, last)];
    r.p[1] = tab[min((t0 + 16) >> a.pg.logp, last)];
    return r;
}
__device__ __forceinline__ bool present(const CacheAttnArgs& a, int page) {
    return static_cast<uint32_t>(page) < static_cast<uint32_t>(a.sq.n_pages);   // (at most 2^30)
}

// The value of a lane offset as it stands here: sums with constants formed from
// it stay beside their load, as its immediate offset, instead of each holding
// a register throughout the loop.
#define HR_KEEP(v) asm volatile("" : "+v"(v))

// N words (or 1 or 2 bytes) from a buffer: a descriptor and an offset that are
// the same in all lanes, plus the lane's offset.
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
__device__ __forceinline__ uint32_t buffer_u16(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    return static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, lane_at, at, 0));
}
__device__ __forceinline__ uint32_t buffer_u8(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    return static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(r, lane_at, at, 0));
}

// A head's part of a page; an absent page's has no bytes, so that its loads give
// zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t head_buffer(const CacheAttnArgs& a, int page, int h) {
    const bool here = present(a, page);
    const uint8_t* base = a.pool + (here ? page : 0) * a.pg.page_bytes + h * a.pg.head_bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, here ? static_cast<int>(a.pg.head_bytes) : 0, 0x00020000);
}

// The values of subtile s, at position off of their page: D/16 dimensions of
// keys 4 g + r, their scales and zero points.
template <class C, class W>
__device__ __forceinline__ void load_values(const CacheAttnArgs& a, __amdgpu_buffer_rsrc_t r, int off, int s, W& w) {
    constexpr int D = C::D, NG = C::NG;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int vc = a.pg.vc + off * (D / 2), vs = a.pg.vs + off * (NG * C::ES), vz = a.pg.vz + off * NG / 2;
    int vl = 4 * g * (D / 2) + m * (D / 32);
    HR_KEEP(vl);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (D == 64) w.v[4 * s + i][0] = buffer_u16(r, vl + i * (D / 2), vc);
        else buffer_words<C::VW>(r, vl + i * (D / 2), vc, w.v[4 * s + i]);
    }
    if constexpr (NG == 1) {
        buffer_words<C::KSW>(r, 4 * g * C::ES, vs, w.vs[s]);
        w.vz[s] = buffer_u16(r, 2 * g, vz);
    } else {
        int at = 4 * g * NG + m / (16 / NG);  // the lane's group of key 4g
        HR_KEEP(at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (C::SF32) buffer_words<1>(r, 4 * at + 4 * i * NG, vs, w.vs[4 * s + i]);
            else w.vs[4 * s + i][0] = buffer_u16(r, 2 * at + 2 * i * NG, vs);
            w.vz[4 * s + i] = buffer_u8(r, at / 2 + i * (NG / 2), vz);
        }
    }
}

// Loads 32 keys from t0.
template <class C>
__device__ __forceinline__ void load_keys(const CacheAttnArgs& a, const Pages& pages, int h, int t0, Raw<C>& w) {
    constexpr int D = C::D, NG = C::NG;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const __amdgpu_buffer_rsrc_t r = head_buffer(a, pages.p[s], h);
        const int off = (t0 + 16 * s) & (a.pg.page - 1);
        const int kc = a.pg.kc + off * (D / 2), ks = a.pg.ks + off * (NG * C::ES), kz = a.pg.kz + off * NG / 2;
        // keys: a lane holds D/4 dimensions of key m, one run with one group,
        // eight of every 32 with several (a matrix step is then one group's)
        int kl = m * (D / 2) + g * (NG == 1 ? D / 8 : 4);
        HR_KEEP(kl);
        if constexpr (NG == 1) {
            buffer_words<C::KS>(r, kl, kc, w.k[s]);
        } else {
#pragma unroll
            for (int i = 0; i < C::KS; ++i) buffer_words<1>(r, kl + i * 16, kc, &w.k[s][i]);
        }
        buffer_words<C::KSW>(r, 4 * g * NG * C::ES, ks, w.ks[s]);
        if constexpr (NG == 1) w.kz[s] = buffer_u8(r, m / 2, kz);
        else if constexpr (NG == 2) w.kz[s] = buffer_u8(r, m, kz);
        else if constexpr (NG == 4) w.kz[s] = buffer_u16(r, 2 * m, kz);
        else buffer_words<1>(r, 4 * m, kz, &w.kz[s]);
        load_values<C>(a, r, off, s, w);
    }
}

// scale r (of word-packed float32 or bfloat16 scales)
template <bool SF32>
__device__ __forceinline__ float scale_at(const uint32_t* w, int i) {
    if constexpr (SF32) return __uint_as_float(w[i]);
    return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

// Symmetric codes are two's complement nibbles: flipping the top bit gives
// c + 8 with zero point 8.  Where there is no section of zero points the loads
// above read codes instead (offset 0), and are masked away here.
struct Zeros {
    uint32_t flip;         // 8 in both halves, or 0
    uint32_t mask, fixed;  // zero point = (what was read & mask) | fixed, in both halves
};
__device__ __forceinline__ Zeros zeros_of(const CacheAttnArgs& a) {
    Zeros z;
    z.flip = a.pg.sym ? 0x00080008u : 0u;
    z.mask = a.pg.sym ? 0u : 0x000F000Fu;
    z.fixed = z.flip;
    return z;
}

// Four operand words of eight codes: (0,4) (1,5) (2,6) (3,7).  Subnormal: in
// units of 2^-24, the second and fourth word with a factor of 16.  CENTRED:
// less the zero point, z0 = it twice, z1 = 16 times that; of ordinary numbers
// the float16 1024 + z and 64 + z.
template <bool SUB, bool CENTRED>
__device__ __forceinline__ uint4v code_operand(uint32_t w, uint32_t flip, uint32_t z0, uint32_t z1) {
    const uint32_t f0 = SUB ? flip : flip | 0x64006400u, f1 = SUB ? flip << 4 : flip << 4 | 0x54005400u;
    uint4v f;
    f.x = (w & 0x000F000Fu) ^ f0;
    f.y = (w & 0x00F000F0u) ^ f1;
    w >>= 8;
    f.z = (w & 0x000F000Fu) ^ f0;
    f.w = (w & 0x00F000F0u) ^ f1;
    if constexpr (CENTRED) {
        f.x = pk_sub(f.x, z0);
        f.y = pk_sub(f.y, z1);
        f.z = pk_sub(f.z, z0);
        f.w = pk_sub(f.w, z1);
    }
    return f;
}

// The operands of V^T of 32 keys: pair() gives the two dimensions of byte b of
// the lane's words, each over the lane's eight keys.
template <class C, bool SCALED>
struct Values {
    static constexpr bool SUB = !C::WIDE && !SCALED;   // subnormal codes
    uint32_t f0, f1;          // XORed into the masked codes
    uint32_t z0[4], z1[4];    // zero points of key pairs, for the low and the high nibble
    uint32_t s0[4], s1[4];    // SCALED: the pairs' scales, and what float16 loses of them

    // vs: SCALED only, scales times a power of two
    template <class W>
    __device__ __forceinline__ Values(const Zeros& zs, const W& w, const float (&vs)[8]) {
        const int lane = threadIdx.x & 63;
        f0 = SUB ? zs.flip : zs.flip | 0x64006400u;
        f1 = SUB ? zs.flip << 4 : zs.flip << 4 | 0x54005400u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t u;
            if constexpr (C::NG == 1) {
                u = w.vz[i / 2] >> (8 * (i & 1));
                u |= u << 12;
            } else {
                const int gi = (lane & 15) / (16 / C::NG);
                u = (w.vz[2 * i] | (w.vz[2 * i + 1] << 16)) >> (4 * (gi & 1));
            }
            z0[i] = (u & zs.mask) | zs.fixed;
            z1[i] = z0[i] << 4;
            if constexpr (!SUB) {
                z0[i] |= 0x64006400u;
                z1[i] |= 0x54005400u;
            }
            if constexpr (SCALED) {
                if constexpr (C::WIDE && C::SF32) split_f16(vs[2 * i], vs[2 * i + 1], s0[i], s1[i]);
                else s0[i] = pack_f16(vs[2 * i], vs[2 * i + 1]);
            }
        }
    }
    // x: the byte of the four key pairs, side by side
    template <class W>
    __device__ __forceinline__ void bytes(const W& w, int b, uint32_t (&x)[4]) const {
        const uint32_t sel = 0x0C040C00u + 0x00010001u * (b & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __builtin_amdgcn_perm(w.v[2 * i + 1][b / 4], w.v[2 * i][b / 4], sel);
    }
    __device__ __forceinline__ uint4v operand(const uint32_t (&x)[4], int half, uint4v* lo) const {
        uint4v f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t d = pk_sub(half ? (x[i] & 0x00F000F0u) ^ f1 : (x[i] & 0x000F000Fu) ^ f0, half ? z1[i] : z0[i]);
            if constexpr (!SCALED) {
                f[i] = d;
            } else {
                f[i] = pk_mul(d, s0[i]);
                if constexpr (C::WIDE) {
                    (*lo)[i] = pk_fma(d, s0[i], f[i] ^ 0x80008000u);
                    if constexpr (C::SF32) (*lo)[i] = pk_fma(d, s1[i], (*lo)[i]);
                }
            }
        }
        return f;
    }
};
template <class C>
__device__ __forceinline__ constexpr int value_bytes() {
    return C::D == 64 ? 2 : 4 * C::VW;
}

// The state of a wave's rows: queries as operands and the running softmax.
template <class C>
struct Rows {
    uint4v q[C::RT][C::P][C::KS];
    uint4v qz[C::RT][C::SUBK && !C::SHARED ? C::NG : 1];  // -sum(q) of a group as an operand (subnormal codes)
    float c;                    // log2 units of one raw score unit, of rows in the common unit
    int own;                    // kOwnUnit if some row of the wave is not, else 0
    int unit[C::SHARED && C::WIDE ? C::RT : 1];   // shared, float32: scores are times 2^-unit
    int lim[C::RT], lo[C::RT];  // keys [lo, lim) are seen
    float mc[C::RT];            // running maximum, log2 units
    float l[C::RT];             // sum of exponentials (this lane's keys)
    float4v o[C::RT][C::DT];
    int e;                      // unit of the value scales in o
    float big, small;           // few rows: the largest and smallest of them in that unit
    // shared operands: scores start from start[] = kPExp - mc (from: in all four
    // registers of a matrix operand); lsum is the sum of exponentials as a
    // matrix result
    float start[C::SHARED ? C::RT : 1];
    float4v from[C::SHARED ? C::RT : 1], lsum[C::SHARED ? C::RT : 1];
};

// What the makers of a tile's key operands note of it (see Passes): bits 0 and 1
// absent subtiles, kOwnUnit (added by the waves), the rest the keys' exponent.
enum { kOwnUnit = 4, kShiftBits = 3 };

// The sign matrix of the index bits that a lane's eight elements and its lane
// group make (5 of them, H_32) as the A operand of a bfloat16 product: row m of
// half a is the element 8 (m >> 2) + 4 a + (m & 3), so that the product leaves
// every result in the lane and register of its input.
__device__ __forceinline__ uint4v hadamard32(int a) {
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int j = 4 * a + (m & 3);
    // bit i of byte j: parity of i & j
    uint32_t s = (j & 1 ? 0xAAu : 0u) ^ (j & 2 ? 0xCCu : 0u) ^ (j & 4 ? 0xF0u : 0u);
    if (__popc((m >> 2) & g) & 1) s ^= 0xFFu;
    uint4v f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = 0x3F803F80u | ((s >> (2 * i) & 1u) << 15) | ((s >> (2 * i + 1) & 1u) << 31);
    return f;
}

// Loads rows r0 + 16 rt + (lane & 15) of kv head h, rotates them and makes
// them operands.  Rows past the sequence's repeat its last one.  units: for the
// exponents of the wave's 16 RT rows against the common one.
template <class C, class T>
__device__ __forceinline__ void load_rows(const CacheAttnArgs& a, const Seq& s, int h, int r0, Rows<C>& w, float* lds, int* units) {
    constexpr int D = C::D, N = D / 4;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    float v[C::RT][N];
    float top[C::RT];   // a row's largest element
    // shared operands: the scores' factor is a fraction, which goes into the rows,
    // and a power of two, so that the keys' scales are taken as they are
    const float factor = a.scale * kLog2e;
    const float fraction = C::SHARED ? __builtin_amdgcn_frexp_mantf(factor) : 1.0f;
    const uint4v h0 = hadamard32(0), h1 = hadamard32(1);
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        const int row = min(r0 + 16 * rt + n, s.n * a.rep - 1);
        const int tok = row / a.rep, hh = row - tok * a.rep;
        const T* p = static_cast<const T*>(a.q) + static_cast<int64_t>(s.start + tok) * a.q_st +
                     static_cast<int64_t>(h * a.rep + hh) * a.q_sh;
        const int pos = s.len - s.n + tok;
        w.lim[rt] = a.causal ? min(pos + 1, s.len) : s.len;
        w.lo[rt] = a.window ? pos - a.window + 1 : 0;
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const int at = C::NG == 1 ? g * N + i * 8 : i * 32 + g * 8;
            if constexpr (sizeof(T) == 2) {
                uint32_t x[4];
                load_words<4>(reinterpret_cast<const uint8_t*>(p + at), x);
                if (a.rotate) {
                    // bfloat16 times +-1 is exact, and the sums are float32
                    const uint4v in = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float4v out = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bfloat8, y ? h1 : h0), __builtin_bit_cast(bfloat8, in),
                            float4v{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[rt][8 * i + 4 * y + j] = out[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[rt][8 * i + 2 * j] = __uint_as_float(x[j] << 16);
                        v[rt][8 * i + 2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
                    }
                }
            } else {
                uint32_t x[8];
                load_words<8>(reinterpret_cast<const uint8_t*>(p + at), x);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[rt][8 * i + j] = __uint_as_float(x[j]);
            }
        }
        if (a.rotate) {
            // H over the dimension's bits.  bfloat16 rows have those of the
            // eight elements and of the lane group from the products above, and
            // want those of the run; float32 rows want all.
#pragma unroll
            for (int st = sizeof(T) == 2 ? 8 : 1; st < N; st *= 2)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (!(j & st)) {
                        const float x = v[rt][j], y = v[rt][j + st];
                        v[rt][j] = x + y;
                        v[rt][j + st] = x - y;
                    }
            if constexpr (sizeof(T) == 4) {
                // (+ in the lower of two lanes, lower - upper in the other)
                const uint32_t s0 = (lane & 16) << 27, s1 = (lane & 32) << 26;
                const auto diff0 = [s0](float x, float y) { return x + __uint_as_float(__float_as_uint(y) ^ s0); };
                const auto diff1 = [s1](float x, float y) { return x + __uint_as_float(__float_as_uint(y) ^ s1); };
#pragma unroll
                for (int j = 0; j < N; ++j) v[rt][j] = over_halves(over_rows(v[rt][j], diff0), diff1);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) v[rt][j] *= a.norm;
        }
        if constexpr (C::SHARED) {
#pragma unroll
            for (int j = 0; j < N; ++j) v[rt][j] *= fraction;
        }
        float own = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) own = fmaxf(own, fabsf(v[rt][j]));
        own = max_groups(own);
        top[rt] = own < __builtin_inff() ? own : 0.0f;   // (a row of infinities or NaN scales nothing: it gives NaN all the same)
    }
    // A power of two puts the largest element of the wave's rows at 2^5 .. 2^6 (a
    // group's sum then stays in float16's range); with shared operands, of the
    // workgroup's at 2 .. 4: their scaled keys, which carry c, have range to spare
    // too.  A row that is not much smaller shares that unit: float16 loses nothing
    // above 2^-25, which is 2^-16 of a row's largest element at a distance of
    // 2^RANGE (pairs: 2^-22).  Other rows have a unit of their own, put right in
    // their scores, so that a result does not depend on the rows beside it.  The
    // scores of pairs in shared operands are put right in any case.
    constexpr int TO = C::SHARED ? 2 : 6, RANGE = !C::WIDE ? 10 : C::SHARED ? 0 : 8;
    const auto exponent = [](float x) { return min(max(TO - (static_cast<int>(__float_as_uint(x) >> 23) - 126), -100), 100); };
    float all = top[0];
#pragma unroll
    for (int rt = 1; rt < C::RT; ++rt) all = fmaxf(all, top[rt]);
    all = max_wave(all);
    if constexpr (C::SHARED) {
        __syncthreads();
        if (lane == 0) lds[threadIdx.x >> 6] = all;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C::WR; ++i) all = fmaxf(all, lds[i]);
        __syncthreads();
    }
    const int common = __builtin_amdgcn_readfirstlane(all > 0.0f ? exponent(all) : 0);
    int e[C::RT];
    bool others = false;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        e[rt] = top[rt] > 0.0f ? exponent(top[rt]) : common;
        if (e[rt] - common <= RANGE) e[rt] = common;
        others |= e[rt] != common;
        if constexpr (C::SHARED && C::WIDE) w.unit[rt] = e[rt] - common;
        else if (g == 0) units[16 * rt + n] = e[rt] - common;
    }
    w.own = !(C::SHARED && C::WIDE) && __any(others) ? kOwnUnit : 0;
    if constexpr (C::SHARED) w.c = ldexpf(1.0f, __builtin_amdgcn_frexp_expf(factor) - common);
    else w.c = factor * __uint_as_float(static_cast<uint32_t>(127 + (C::SUBK ? 24 : 0) - common) << 23);
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e[rt]) << 23);
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
                const float f = C::SUBK && !C::SHARED && (j & 1) ? up * 0.0625f : up;
                const float x = v[rt][8 * i + j] * f, y = v[rt][8 * i + j + 4] * f;
                if constexpr (C::WIDE) split_f16(x, y, hi[j], lo[j]);
                else hi[j] = pack_f16(x, y);
                if constexpr (C::SUBK && !C::SHARED) {
                    const float back = lo_f32(hi[j]) + hi_f32(hi[j]);
                    sum[C::NG == 1 ? 0 : i / C::KG] += (j & 1) ? back * 16.0f : back;
                }
            }
            w.q[rt][0][i] = uint4v{hi[0], hi[1], hi[2], hi[3]};
            if constexpr (C::WIDE) w.q[rt][1][i] = uint4v{lo[0], lo[1], lo[2], lo[3]};
        }
        if constexpr (C::SUBK && !C::SHARED) {
            // the zero point's operand has z in k slots 0 and 1 of lane group
            // 0: -sum(q) there as two float16
#pragma unroll
            for (int i = 0; i < C::NG; ++i) {
                const float t = -sum_groups(sum[i]);
                uint32_t hi, lo;
                split_f16(t, 0.0f, hi, lo);
                w.qz[rt][i] = uint4v{g == 0 ? (hi & 0xFFFFu) | (lo << 16) : 0u, 0u, 0u, 0u};
            }
        }
        w.mc[rt] = kLow;
        w.l[rt] = 0.0f;
        if constexpr (C::SHARED) {
            constexpr float s = kPExp;
            w.start[rt] = s;
            w.from[rt] = float4v{s, s, s, s};
            w.lsum[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int j = 0; j < C::DT; ++j) w.o[rt][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    w.e = kNoUnit;
}

// Raw scores of 32 keys, in log2 units once multiplied by mul:
// x[rt][4 s + r] is key 16 s + 4 g + r.
template <class C>
__device__ __forceinline__ void scores(const Zeros& zs, const Raw<C>& w, const Rows<C>& st, float (&x)[C::RT][8],
                                       float (&mul)[8]) {
    constexpr int NG = C::NG, RT = C::RT;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            HR_PHASE();
            // zero point of key m, in the low and in the second nibble
            const uint32_t z = NG == 1 ? w.kz[s] >> (4 * (lane & 1)) : w.kz[s] >> (4 * gi);
            float4v acc[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t z0 = (((z << 16) | (z & 0xFFFFu)) & zs.mask) | zs.fixed, z1 = 0;
            if constexpr (C::SUBK) {
                const uint4v za = {lane < 16 ? z0 : 0u, 0u, 0u, 0u};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) acc[rt] = mfma(za, st.qz[rt][gi], acc[rt]);
            } else {
                z1 = (z0 << 4) | 0x54005400u;
                z0 |= 0x64006400u;
            }
#pragma unroll
            for (int i = gi * C::KG; i < (gi + 1) * C::KG; ++i) {
                const uint4v f = code_operand<C::SUBK, !C::SUBK>(w.k[s][i], zs.flip, z0, z1);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    acc[rt] = mfma(f, st.q[rt][0][i], acc[rt]);
                    if constexpr (C::WIDE) acc[rt] = mfma(f, st.q[rt][1][i], acc[rt]);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float ks = scale_at<C::SF32>(w.ks[s], r * NG + gi) * st.c;
                if constexpr (NG == 1) mul[4 * s + r] = ks;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    if constexpr (NG == 1) x[rt][4 * s + r] = acc[rt][r];
                    else x[rt][4 * s + r] = gi == 0 ? acc[rt][r] * ks : fmaf(acc[rt][r], ks, x[rt][4 * s + r]);
                }
            }
        }
    }
    if constexpr (NG > 1) {
#pragma unroll
        for (int t = 0; t < 8; ++t) mul[t] = 1.0f;
    }
}

// One step of the softmax: x becomes exp2(x mul - mc), moving the running
// maximum first if one of them would pass 2^kSlack.  (Unseen keys have -inf
// and a finite mul.)
template <class C>
__device__ __forceinline__ void exponentials(Rows<C>& st, int rt, float (&x)[8], const float (&mul)[8]) {
    float p[8], top = 0.0f;
#pragma unroll
    for (int t = 0; t < 8; ++t) p[t] = __builtin_amdgcn_exp2f(fmaf(x[t], mul[t], -st.mc[rt]));
#pragma unroll
    for (int t = 0; t < 8; ++t) top = fmaxf(top, p[t]);
    if (__any(top > static_cast<float>(1 << kSlack))) {
        top = kLow;
#pragma unroll
        for (int t = 0; t < 8; ++t) top = fmaxf(top, x[t] * mul[t]);
        const float mc = fmaxf(max_groups(top), st.mc[rt]);
        const float f = exp2f(st.mc[rt] - mc);
        st.mc[rt] = mc;
        st.l[rt] *= f;
#pragma unroll
        for (int j = 0; j < C::DT; ++j) st.o[rt][j] *= f;
        // (the products rounded as mc is: beside it an unrounded one of 2^30 may be
        // 2^6 larger)
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma clang fp contract(off)
            p[t] = __builtin_amdgcn_exp2f(x[t] * mul[t] - mc);
        }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        st.l[rt] += p[t];
        x[t] = p[t];
    }
}

// Scores to probabilities as an operand (hi, and lo for pairs of float16): one
// group: times the value scales vs.
template <class C>
__device__ __forceinline__ void probabilities(Rows<C>& st, int rt, float (&x)[8], const float (&mul)[8], const float (&vs)[8],
                                              uint4v& hi, uint4v& lo) {
    exponentials<C>(st, rt, x, mul);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) p[j] = x[2 * i + j] * (C::NG == 1 ? vs[2 * i + j] : C::SHARED ? vs[0] : static_cast<float>(1 << kPExp));
        uint32_t h, l = 0;
        if constexpr (C::WIDE) split_f16(p[0], p[1], h, l);
        else h = pack_f16(p[0], p[1]);
        hi[i] = h;
        lo[i] = l;
    }
}

// The unit of value scales.  o is held in units of 2^e of them, and a scale takes
// part in a float16 operand if its exponent is in [e - VRANGE, e].  With shared
// operands the unit moves with the scales of a pass, and o with it, exactly.  A
// few-row wave takes the one of its first step throughout, and goes through its
// keys again with a unit for every step if some scale was not in it (a branch that
// moves the unit in every step's code takes 8% of a single token's time).
// Keys whose scales are too far from the others' for one unit, beyond 2^kFar either
// way, or not finite are set aside: left out of the step, and taken one at a time
// when the segment is done, in float32 throughout (sweep_rows).  So a key that a
// row does not see has no influence on it, whatever its scale is, and one that it
// sees costs the others no bits.  Whether a key is set aside depends on the scales
// of its step (pass) alone, not on those before it: the sweep finds the same keys.
// (Within 2^kFar no move of the unit lets a sum overflow.)
// A token of R3's cache: 43 us; 118 and 145 with one scale in 20000 and in 1000 2^28
// times the others', 2400 with all of them anywhere from 1 to 2^30.
__device__ __forceinline__ int exponent(float x) {   // |x| < 2^exponent(x); x finite
    return static_cast<int>((__float_as_uint(x) >> 23) & 0xFFu) - 126;
}
__device__ __forceinline__ float power(int e) {      // 2^e, -126 <= e <= 128 (infinite)
    return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}
// The unit for exponents from lo to hi, at most RANGE apart: those in its middle.
template <int RANGE>
__device__ __forceinline__ int unit_for(int lo, int hi) {
    return min(max(hi + (RANGE - (hi - lo)) / 2, RANGE - kFar), kFar);
}
template <int RANGE>
__device__ __forceinline__ bool set_aside(float x, int lo) {
    x = fabsf(x);
    return x != 0.0f && !(x >= power(lo - 1) && x < power(min(lo + RANGE, kFar)));
}
template <class C>
__device__ __forceinline__ void set_unit(Rows<C>& st, int e) {
    if (st.e != kNoUnit) {
        const float f = ldexpf(1.0f, st.e - e);
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
            for (int j = 0; j < C::DT; ++j) st.o[rt][j] *= f;
    }
    st.e = e;
}
__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b) {   // of both halves
    typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, a), __builtin_bit_cast(ushort2v, b)));
}
// Over the lanes that hold a wave's value scales (one group: 16 have the same).
template <class C>
__device__ __forceinline__ float max_scales(float v) {
    return C::NG == 1 ? max_groups(v) : max_wave(v);
}
// The exponents of the wave's scales, but for those that are 0, or not within
// 2^kFar (some: there are such).  hi < lo: there are no others.
template <class C>
__device__ __forceinline__ void exponents_of(const float (&vs)[8], int& lo, int& hi, bool& some) {
    // the smallest as an integer, less 1: a zero is the largest then
    float big = 0.0f;
    uint32_t small = ~0u;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        big = __builtin_elementwise_maximum(big, fabsf(vs[t]));   // (keeps a NaN)
        small = min(small, __float_as_uint(fabsf(vs[t])) - 1u);
    }
    some = __any(!(big < 0x1p32f) || small < 0x2F000000u - 1u);   // 2^-33
    if (some) {
        HR_BRANCH();
        big = 0.0f, small = ~0u;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float x = fabsf(vs[t]);
            const bool in = x >= 0x1p-33f && x < 0x1p32f;
            big = fmaxf(big, in ? x : 0.0f);
            small = min(small, in ? __float_as_uint(x) - 1u : ~0u);
        }
    }
    // both in one word: the exponent fields, of the smallest 255 less it
    uint32_t both = __float_as_uint(big) >> 23 << 16 | (small == ~0u ? 0u : 255u - ((small + 1u) >> 23));
    if constexpr (C::NG > 1) {
        both = max_u16(both, swizzle_xor<1>(both));
        both = max_u16(both, swizzle_xor<2>(both));
        both = max_u16(both, swizzle_xor<4>(both));
        both = max_u16(both, swizzle_xor<8>(both));
    }
    const auto most = [](float x, float y) { return __uint_as_float(max_u16(__float_as_uint(x), __float_as_uint(y))); };
    both = __builtin_amdgcn_readfirstlane(__float_as_uint(over_halves(over_rows(__uint_as_float(both), most), most)));
    hi = static_cast<int>(both >> 16) - 126;
    lo = 129 - static_cast<int>(both & 0xFFFFu);
}
// The keys of 32, key 16 (t / 4) + 4 g + t % 4 in element t of lane group g, of
// which some lane says that they are out.
__device__ __forceinline__ uint32_t keys_of(const bool (&out)[8]) {
    uint32_t keys = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const uint64_t who = __ballot(out[t]);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (who >> (16 * g) & 0xFFFFu) keys |= 1u << (16 * (t / 4) + 4 * g + t % 4);
    }
    return __builtin_amdgcn_readfirstlane(keys);
}
// The value scales of a few-row step, and those of keys past the last that is
// seen, or on an absent page, whatever they are, as `none`.
template <class C, class W>
__device__ __forceinline__ void step_scales(const W& w, float (&vs)[8]) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if constexpr (C::NG == 1) vs[t] = scale_at<C::SF32>(w.vs[t / 4], t & 3);
        else vs[t] = __uint_as_float(C::SF32 ? w.vs[t][0] : w.vs[t][0] << 16);
    }
}
__device__ __forceinline__ void drop_unseen(const CacheAttnArgs& a, const Pages& pages, int t0, int end, float none, float (&vs)[8]) {
    const int g = (threadIdx.x & 63) >> 4;
    const bool here[2] = {present(a, pages.p[0]), present(a, pages.p[1])};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const int key = t0 + 16 * (t / 4) + 4 * g + t % 4;
        vs[t] = key < end && here[t / 4] ? vs[t] : none;
    }
}
// The keys that such a step sets aside, and the exponents lo to hi of the others.
template <class C>
__device__ __forceinline__ uint32_t aside_of(const float (&vs)[8], int& lo, int& hi) {
    bool some, out[8];
    exponents_of<C>(vs, lo, hi, some);
    if (hi < lo) lo = hi = 0;
    if (!some && hi - lo <= C::VRANGE) return 0;
    hi = min(hi, lo + C::VRANGE);
#pragma unroll
    for (int t = 0; t < 8; ++t) out[t] = set_aside<C::VRANGE>(vs[t], lo);
    return keys_of(out);
}

// One step over 32 keys; mask: some of them are not seen by every row; units: of
// the wave's rows.  MOVES: the unit of the value scales is the step's own, and flag
// is set if keys are set aside.
template <class C, bool MOVES>
__device__ __forceinline__ void step(const CacheAttnArgs& a, const Raw<C>& w, const Pages& pages, bool mask, int end, int* flag,
                                     const int* units, int t0, Rows<C>& st) {
    constexpr int NG = C::NG, RT = C::RT;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const Zeros zs = zeros_of(a);
    float x[RT][8], mul[8];
    scores<C>(zs, w, st, x, mul);
    HR_PHASE();
    if (st.own) {
        HR_BRANCH();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int unit = -units[16 * rt + (lane & 15)];
#pragma unroll
            for (int t = 0; t < 8; ++t) x[rt][t] = ldexpf(x[rt][t], unit);
        }
    }
    // value scales in their unit (several groups: they go into the operand that
    // all 16 queries share)
    float vs[8];
    step_scales<C>(w, vs);
    if (mask) {
        // unseen scores become -inf, whatever they are
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int key = t0 + 16 * (t / 4) + 4 * g + t % 4;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const bool seen = present(a, pages.p[t / 4]) && key < st.lim[rt] && key >= st.lo[rt];
                x[rt][t] = seen ? x[rt][t] * mul[t] : -__builtin_inff();
            }
            mul[t] = 1.0f;
        }
        if constexpr (!MOVES) drop_unseen(a, pages, t0, end, ldexpf(1.0f, st.e - 1), vs);   // (one in the unit)
    }
    if constexpr (MOVES) {
        int lo, hi;
        drop_unseen(a, pages, t0, end, 0.0f, vs);
        const uint32_t aside = aside_of<C>(vs, lo, hi);
        if (!(hi <= st.e && lo >= st.e - C::VRANGE)) set_unit<C>(st, unit_for<C::VRANGE>(lo, hi));
        if (aside) {
            HR_BRANCH();
            *flag = 1;
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (aside >> (16 * (t / 4) + 4 * g + t % 4) & 1) {
                    vs[t] = 0.0f;
                    mul[t] = 1.0f;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) x[rt][t] = -__builtin_inff();
                }
        }
    }
    const float down = ldexpf(1.0f, C::VEXP - st.e);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        vs[t] *= down;
        if constexpr (!MOVES) {
            st.big = __builtin_elementwise_maximum(st.big, fabsf(vs[t]));   // (keeps a NaN)
            st.small = fminf(st.small, fabsf(vs[t]));
        }
    }
    uint4v ph[RT], pl[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        HR_PHASE();
        probabilities<C>(st, rt, x[rt], mul, vs, ph[rt], pl[rt]);
    }
    // O^T += V^T P^T, two dimensions a byte
    const Values<C, (NG > 1)> values(zs, w, vs);
#pragma unroll
    for (int b = 0; b < value_bytes<C>(); ++b) {
        HR_PHASE();
        uint32_t y[4];
        values.bytes(w, b, y);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint4v vl;
            const uint4v vh = values.operand(y, half, &vl);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float4v& o = st.o[rt][2 * b + half];
                o = mfma(vh, ph[rt], o);
                if constexpr (C::WIDE) o = mfma(vh, pl[rt], o);
                if constexpr (C::VLO) o = mfma(vl, ph[rt], o);
            }
        }
    }
}

// A wave's share of keys [k0, k1) (k0 a multiple of 32) of a unit: every WT-th
// 32 of them.  The next step's keys are loaded before a step is computed, and
// the pages of the one after it are looked up; start() is called before the
// rows are loaded, so that the first keys are on their way meanwhile.
template <class C>
struct Walk {
    static constexpr int S = 32 * C::WT;
    const int32_t* table;
    int h, t, end;
    Pages now, next;
    Raw<C> w;

    __device__ __forceinline__ void start(const CacheAttnArgs& a, const Span& sp, int k0, int k1, int wt) {
        t = max(k0, sp.lo & ~31) + 32 * wt;
        end = min(k1, sp.hi);
        if (t >= end) return;
        now = pages_at(a, table, t);
        next = pages_at(a, table, t + S);
        load_keys<C>(a, now, h, t, w);
    }
    // A unit that the first step's scales are in, with room above and below.
    __device__ __forceinline__ int first_unit(const CacheAttnArgs& a) const {
        float vs[8], big = 0.0f;
        step_scales<C>(w, vs);
        drop_unseen(a, now, t, end, 0.0f, vs);
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(vs[i]));
        const int hi = __builtin_amdgcn_readfirstlane(exponent(max_scales<C>(big)));
        return min(max((hi < -kFar ? 0 : hi) + C::VRANGE / 3, C::VRANGE - kFar), kFar);
    }
    template <bool MOVES>
    __device__ __forceinline__ void run(const CacheAttnArgs& a, const Span& sp, int* flag, const int* units, Rows<C>& st) {
        if (t >= end) return;
        while (true) {
            Raw<C> n;
            const bool more = t + S < end;
            if (more) load_keys<C>(a, next, h, t + S, n);
            const Pages after = pages_at(a, table, t + 2 * S);
            const bool all = t >= sp.flo && t + 32 <= sp.fhi && present(a, now.p[0]) && present(a, now.p[1]);
            step<C, MOVES>(a, w, now, !all, end, flag, units, t, st);
            if (!more) return;
            t += S;
            w = n;
            now = next;
            next = after;
        }
    }
};

// Four neighbouring elements of an output row.
template <class T>
__device__ __forceinline__ void store4(T* to, float4v x) {
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2v*>(to) = uint2v{to_bf16(x[0]) | (to_bf16(x[1]) << 16), to_bf16(x[2]) | (to_bf16(x[3]) << 16)};
    else *reinterpret_cast<float4v*>(to) = x;
}
__device__ __forceinline__ float log_sum(float m2, float l) {
    return l == 0.0f ? -__builtin_inff() : (m2 + __log2f(l)) * 0.6931471805599453f;
}
// A part of a row in the scratch: d sums, the maximum (log2 units), the sum of
// exponentials, padded to 16 bytes.
template <class C>
constexpr int part_stride() {
    return C::D + 4;
}

// Writes a wave's finished rows, or its part of them to the scratch.
template <class C, class T>
__device__ __forceinline__ void put_rows(const CacheAttnArgs& a, const Seq& s, int h, int r0, const Rows<C>& st, float* part,
                                         int part_row) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        const int row = r0 + 16 * rt + n;
        if (row >= s.n * a.rep) continue;
        const float l = st.l[rt];
        if (part) {
            float* p = part + (part_row + 16 * rt + n) * part_stride<C>();
            if (g == 0) {
                p[C::D] = l > 0.0f || l != l ? st.mc[rt] : kLow;
                p[C::D + 1] = l;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < C::DT; j += 4)
                    *reinterpret_cast<float4v*>(p + (4 * g + r) * C::DT + j) =
                        float4v{st.o[rt][j][r], st.o[rt][j + 1][r], st.o[rt][j + 2][r], st.o[rt][j + 3][r]};
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
                float4v x;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = st.o[rt][j + i][r] * inv;
                store4<T>(p + (4 * g + r) * C::DT + j, x);
            }
        if (a.lse && g == 0) a.lse[t * a.hq + head] = log_sum(st.mc[rt], l);
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

// Joins the four waves that took different keys of the same rows and writes
// the rows, or their part to the scratch (to `spare` for rows that are finished
// here but for keys set aside; returns whether there are such): maxima first,
// then every wave's sums through LDS in a few rows at a time, 16 threads to a row.
template <class C>
constexpr int join_floats() {
    return 2 * 4 * 16 + 4 * 16 * (C::D + 4);
}
template <class C, class T>
__device__ __forceinline__ bool join_waves(const CacheAttnArgs& a, const Seq& s, int h, int r0, Rows<C>& st, float* part,
                                           float* spare, const int* flag, float* lds) {
    static_assert(C::WT == 4 && C::WR == 1, "four waves along the keys");
    constexpr int D = C::D, LD = D + 4;                    // (rows 16 bytes apart in the banks)
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, g = lane >> 4;
    float* ml = lds;                                       // [2][4][16]: maxima, sums
    float* so = lds + 128;                                 // [4][16][LD]
    bool aside = false;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        const int rows = min(s.n * a.rep - r0 - 16 * rt, 16);
        if (rows <= 0) break;
        __syncthreads();
        if (rt == 0) {
            // (every wave has set it that will, and the next segment's may be
            // set only after the barrier below)
            aside = __builtin_amdgcn_readfirstlane(*flag) != 0;
            if (aside && !part) part = spare;
        }
        if (g == 0) {
            ml[wave * 16 + n] = st.mc[rt];
            ml[64 + wave * 16 + n] = st.l[rt];
        }
        if (n < rows) {
            float* p = so + (wave * 16 + n) * LD + 4 * g * C::DT;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < C::DT; j += 4)
                    *reinterpret_cast<float4v*>(p + r * C::DT + j) =
                        float4v{st.o[rt][j][r], st.o[rt][j + 1][r], st.o[rt][j + 2][r], st.o[rt][j + 3][r]};
        }
        __syncthreads();
        const int row = tid >> 4, i = tid & 15;            // 16 threads to a row
        if (row < rows) {
            float top = kLow, l = 0.0f, f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) top = fmaxf(top, ml[x * 16 + row]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                f[x] = exp2f(ml[x * 16 + row] - top);
                l += f[x] * ml[64 + x * 16 + row];
            }
            const int at = r0 + 16 * rt + row, tok = at / a.rep;
            const int64_t t = s.start + tok, head = h * a.rep + at - tok * a.rep;
            const float inv = part ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
            float* pp = part + (16 * rt + row) * part_stride<C>();
            T* po = static_cast<T*>(a.out) + t * a.o_st + head * a.o_sh;
#pragma unroll
            for (int j = 0; j < D; j += 64) {
                float4v v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int x = 0; x < 4; ++x) v += *reinterpret_cast<const float4v*>(so + (x * 16 + row) * LD + j + 4 * i) * f[x];
                v *= inv;
                if (part) *reinterpret_cast<float4v*>(pp + j + 4 * i) = v;
                else store4<T>(po + j + 4 * i, v);
            }
            if (i == 0) {
                if (part) {
                    pp[D] = l > 0.0f || l != l ? top : kLow;
                    pp[D + 1] = l;
                } else if (a.lse) {
                    a.lse[t * a.hq + head] = log_sum(top, l);
                }
            }
        }
    }
    return aside;
}

// ---------------------------------------------------------------------------
// Many rows: shared operands.  Eight waves have 16 or 32 rows each, one after
// the other of the same unit.  For every pass of TILES x 32 keys some of the
// waves turn the keys' or the values' codes of a tile into operands in LDS,
// scaled: k by its scales and a power of two (the rest of the factor that gives log2
// units is in the queries), v by its scales and one, the unit of the pass (VEXP).
// That is done once for all rows, and leaves a row's wave for each score one
// exponential, half a maximum and half a conversion:
//   - the running maximum is the start value of the matrix product, so that
//     its result is the exponent (kPExp - mc + score) itself;
//   - the sum of exponentials is a matrix product with ones.
// 2 prompts of 2048 tokens behind 6144 keys, 32 heads over 8 of 128: 560 us, 860
// TFLOP/s of scores and values, where a large bfloat16 matrix product has 1216
// (395 us); with operands made anew for every four waves it was 755.  By the
// counters the matrix units are busy 39% of the time (SQ_VALU_MFMA_BUSY_CYCLES over
// the busy cycles of all SIMDs), the waves wait 36% of theirs (SQ_WAIT_ANY over
// SQ_WAVE_CYCLES), and there are 3.4 other vector instructions for a matrix
// instruction: neither unit is full.  A workgroup fills a CU (132 kB of LDS, 256
// registers a lane), so nothing runs while its waves wait for each other at the end
// of a pass.
// Two passes' operands are in LDS: a pass is made while the one before it is
// computed.  The waves that make values do so first (their scales are looked
// at again at the end of a pass), those that make keys last: the two of a SIMD
// are one of each, so that its matrix unit and its vector unit both have work.
// Scaled operands s (c - z) are rounded to float16 for bfloat16 activations: with
// bfloat16 scales (8 bits) that is exact but for |c - z| of 9, 11, 13 and 15 (4 bits
// more), and then each element's own, of 2^-12 at most; float32 scales are rounded
// with their elements (keys) or before them (values).  The sum of exponentials is
// that of the probabilities as they are multiplied, 11 bits each, so what rounding
// does to all of a row cancels; the log-sum-exp errs by 2^-12 at most.  Scales
// applied to the results and probabilities instead, in float32, took 755 us for the
// call above and do not change its error, 1.70e-3 (1.66e-3 of it bfloat16's own
// rounding); with scales times the scores' factor rounded for a whole key it was
// 1.99e-3.  float32 activations take pairs of float16 throughout.

template <class C>
struct Tile {
    uint4v k[C::P][2 * C::KS][64];
    uint4v v[C::P][C::DT][64];
};
template <class C>
struct Passes {
    Tile<C> tile[2][C::TILES];
    // of a tile: keys (bit s: subtile s is on an absent page; 2^kShiftBits x shift:
    // they are times 2^-shift, extreme scales), keys that are set aside for their own
    // scales, and for their values', -
    uint4v note[2][C::TILES];
    uint2v range[2][C::TILES];  // exponents lo, hi of a tile's value scales
    Todo todo;
    float top[C::WR];
    int unit[C::WR][16 * C::RT];   // exponents of the rows' units (bfloat16 activations)
};
template <class C>
constexpr int lds_floats() {
    if constexpr (C::SHARED) return static_cast<int>(sizeof(Passes<C>)) / 4;
    // (and the units of each wave's rows, and a Todo)
    else return join_floats<C>() + 4 * 16 * C::RT + 4 + static_cast<int>(sizeof(Todo)) / 4;
}

template <class C>
__device__ __forceinline__ Todo* todo_at(float* lds) {
    if constexpr (C::SHARED) return &reinterpret_cast<Passes<C>*>(lds)->todo;
    else return reinterpret_cast<Todo*>(lds + join_floats<C>() + 4 * 16 * C::RT);
}

// Codes and scales of a tile's keys: key m in the lane.
template <class C>
struct RawK {
    uint32_t k[2][C::KS];
    uint32_t ks[2][(C::NG * C::ES + 3) / 4];
    uint32_t kz[2];
};
// Codes and scales of its values: keys 4 g + r of a subtile.
template <class C>
struct RawV {
    uint32_t v[8][C::VW];
    uint32_t vs[C::NG == 1 ? 2 : 8][C::NG == 1 ? C::KSW : 1];
    uint32_t vz[C::NG == 1 ? 2 : 8];
};

template <class C>
__device__ __forceinline__ void load_raw(const CacheAttnArgs& a, const Pages& pages, int h, int t0, RawK<C>& w) {
    constexpr int D = C::D, NG = C::NG;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const __amdgpu_buffer_rsrc_t r = head_buffer(a, pages.p[s], h);
        const int off = (t0 + 16 * s) & (a.pg.page - 1);
        const int kc = a.pg.kc + off * (D / 2), ks = a.pg.ks + off * (NG * C::ES), kz = a.pg.kz + off * NG / 2;
        int kl = m * (D / 2) + g * (NG == 1 ? D / 8 : 4);
        HR_KEEP(kl);
        if constexpr (NG == 1) {
            buffer_words<C::KS>(r, kl, kc, w.k[s]);
        } else {
#pragma unroll
            for (int i = 0; i < C::KS; ++i) buffer_words<1>(r, kl + i * 16, kc, &w.k[s][i]);
        }
        if constexpr (NG * C::ES == 2) w.ks[s][0] = buffer_u16(r, 2 * m, ks);
        else buffer_words<NG * C::ES / 4>(r, NG * C::ES * m, ks, w.ks[s]);
        if constexpr (NG == 1) w.kz[s] = buffer_u8(r, m / 2, kz);
        else if constexpr (NG == 2) w.kz[s] = buffer_u8(r, m, kz);
        else if constexpr (NG == 4) w.kz[s] = buffer_u16(r, 2 * m, kz);
        else buffer_words<1>(r, 4 * m, kz, &w.kz[s]);
    }
}

template <class C>
__device__ __forceinline__ void load_raw(const CacheAttnArgs& a, const Pages& pages, int h, int t0, RawV<C>& w) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
        load_values<C>(a, head_buffer(a, pages.p[s], h), (t0 + 16 * s) & (a.pg.page - 1), s, w);
}

// The scales of a tile's keys (times c), and the power of two that they are
// divided by.  c - z is at most 15: scales of 2^-13 .. 2^12 keep within float16, and
// a tile of others is moved there.  Larger keys among small ones are set aside,
// and their scales become 0.
template <class C>
__device__ __forceinline__ int key_unit(const RawK<C>& w, int t0, int end, float c, float (&ks)[2][C::NG], uint32_t& aside) {
    constexpr int NG = C::NG;
    const int m = threadIdx.x & 15;
    float top[2];                            // the key's largest
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        top[s] = 0.0f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            ks[s][gi] = t0 + 16 * s + m < end ? scale_at<C::SF32>(w.ks[s], gi) * c : 0.0f;
            top[s] = __builtin_elementwise_maximum(top[s], fabsf(ks[s][gi]));   // (keeps a NaN)
        }
    }
    aside = 0;
    const float most = __builtin_elementwise_maximum(top[0], top[1]);
    if (!__any(!(most <= 4096.0f)) && __any(most >= 0x1p-13f)) return 0;
    HR_BRANCH();
    float big = 0.0f, small = __builtin_inff();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (top[s] < __builtin_inff()) big = fmaxf(big, top[s]);
        if (top[s] > 0.0f) small = fminf(small, top[s]);
    }
    big = max_wave(big);
    small = -max_wave(-small);
    int e = 0;
    if (big > 4096.0f) e = max(min(exponent(big), exponent(small) + C::KRANGE) - 12, 0);
    else if (big > 0.0f && big < 0x1p-13f) e = exponent(big);
    e = __builtin_amdgcn_readfirstlane(e);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const bool out = !(top[s] <= 4096.0f) && !(e + 12 < 128 && top[s] < power(e + 12));
        aside |= static_cast<uint32_t>(__ballot(out) & 0xFFFFu) << (16 * s);   // (a key's four lanes agree)
        if (out) {
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) ks[s][gi] = 0.0f;
        }
    }
    return e;
}

// Makes the key operands of a tile.  (c: log2 units of a product with the
// queries as they are held.)
template <class C>
__device__ __forceinline__ void make_keys(const CacheAttnArgs& a, const RawK<C>& w, const Pages& pages, int t0, int end, float c,
                                          Tile<C>& tile, uint32_t* note, int* flag) {
    constexpr int NG = C::NG;
    const int lane = threadIdx.x & 63;
    const Zeros zs = zeros_of(a);
    float ks[2][NG];
    uint32_t aside;
    const int e = key_unit<C>(w, t0, end, c, ks, aside);
    if (aside) *flag = 1;
    if (e != 0) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) ks[s][gi] = ldexpf(ks[s][gi], -e);
    }
    const int special = (present(a, pages.p[0]) ? 0 : 1) | (present(a, pages.p[1]) ? 0 : 2) | e * (1 << kShiftBits);
    if (lane == 0) *reinterpret_cast<uint2v*>(note) = uint2v{static_cast<uint32_t>(special), aside};
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < C::KS; ++i) {
            const int gi = i / C::KG;
            const uint32_t z = NG == 1 ? w.kz[s] >> (4 * (lane & 1)) : w.kz[s] >> (4 * gi);
            uint32_t z0 = (((z << 16) | (z & 0xFFFFu)) & zs.mask) | zs.fixed;
            const uint32_t z1 = (z0 << 4) | 0x54005400u;
            z0 |= 0x64006400u;
            uint32_t hi, lo = 0;
            if constexpr (C::WIDE || C::SF32) split_f16(ks[s][gi], ks[s][gi], hi, lo);
            else hi = pack_f16(ks[s][gi], ks[s][gi]);   // (exact)
            const uint4v d = code_operand<false, true>(w.k[s][i], zs.flip, z0, z1);
            uint4v f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (what float16 loses of a float32 scale would be lost of all the
                // key's elements at once, and move its score by up to 2^-11)
                if constexpr (!C::WIDE && C::SF32) f[j] = pk_fma(d[j], hi, pk_mul(d[j], lo));
                else f[j] = pk_mul(d[j], hi);
            }
            tile.k[0][s * C::KS + i][lane] = f;
            if constexpr (C::WIDE) {
                uint4v fl;
#pragma unroll
                for (int j = 0; j < 4; ++j) fl[j] = pk_fma(d[j], lo, pk_fma(d[j], hi, f[j] ^ 0x80008000u));
                tile.k[1][s * C::KS + i][lane] = fl;
            }
        }
}

// Value scales of a tile; those past the sequence or on an absent page are 0.
template <class C>
__device__ __forceinline__ void value_scales(const CacheAttnArgs& a, const RawV<C>& w, const Pages& pages, int t0, int end,
                                             float (&vs)[8]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if constexpr (C::NG == 1) vs[t] = scale_at<C::SF32>(w.vs[t / 4], t & 3);
        else vs[t] = __uint_as_float(C::SF32 ? w.vs[t][0] : w.vs[t][0] << 16);
        if (t0 + 16 * (t / 4) + 4 * g + t % 4 >= end || !present(a, pages.p[t / 4])) vs[t] = 0.0f;
    }
}

// Makes the value operands of a tile, times 2^(kSExp - e).  check: some scales may
// not be in the unit, which begins at exponent lo.
template <class C>
__device__ __forceinline__ void make_values(const CacheAttnArgs& a, const RawV<C>& w, const Pages& pages, int t0, int end, int e,
                                            bool check, int lo, Tile<C>& tile, uint32_t* set_aside_at, int* flag) {
    const int lane = threadIdx.x & 63;
    float vs[8];
    value_scales<C>(a, w, pages, t0, end, vs);
    uint32_t aside = 0;
    if (check) {
        HR_BRANCH();
        bool out[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            out[t] = set_aside<C::VRANGE>(vs[t], lo);
            if (out[t]) vs[t] = 0.0f;
        }
        aside = keys_of(out);
        if (aside) *flag = 1;
    }
    if (lane == 0) *set_aside_at = aside;
    const float down = ldexpf(1.0f, kSExp - e);
#pragma unroll
    for (int t = 0; t < 8; ++t) vs[t] *= down;
    const Values<C, true> values(zeros_of(a), w, vs);
#pragma unroll
    for (int b = 0; b < value_bytes<C>(); ++b) {
        HR_PHASE();
        uint32_t y[4];
        values.bytes(w, b, y);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint4v vl;
            tile.v[0][2 * b + half][lane] = values.operand(y, half, &vl);
            if constexpr (C::WIDE) tile.v[1][2 * b + half][lane] = vl;
        }
    }
}

// Operands of a tile on their way from LDS: GROUP of them at a time, while the
// products of the group before them run.
template <class C>
struct Fetch {
    static constexpr int GROUP = 4;
    uint4v f[C::P][GROUP];
    __device__ __forceinline__ void keys(const Tile<C>& tile, int first) {
#pragma unroll
        for (int p = 0; p < C::P; ++p)
#pragma unroll
            for (int i = 0; i < GROUP; ++i)
                if (first + i < 2 * C::KS) f[p][i] = tile.k[p][first + i][threadIdx.x & 63];
    }
    __device__ __forceinline__ void values(const Tile<C>& tile, int first) {
#pragma unroll
        for (int p = 0; p < C::P; ++p)
#pragma unroll
            for (int i = 0; i < GROUP; ++i) f[p][i] = tile.v[p][first + i][threadIdx.x & 63];
    }
};

// The scores of a tile, in log2 units.
template <class C>
__device__ __forceinline__ void raw_scores(const Tile<C>& tile, int special, const int* units, const Rows<C>& st,
                                           float4v (&x)[C::RT][2]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 2 * C::RT; ++i) {
        float4v& y = x[i / 2][i % 2];
        y = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < C::KS; ++j) y = mfma(tile.k[0][i % 2 * C::KS + j][lane], st.q[i / 2][0][j], y);
        if ((special & ~3) != 0) {   // (extreme scales or rows: their unit is not 1)
            HR_BRANCH();
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = ldexpf(y[r], (special >> kShiftBits) - units[i / 2 * 16 + (lane & 15)]);
        }
    }
}

// Moves the running maxima to what the scores of a tile have, where that is more,
// and the sums with them; the scores become exponents, kPExp less what they lie
// below the maximum.  (Of the scores themselves: as a product that starts from
// kPExp - mc, a score far above mc has lost bits of its own.)  Whether some row has
// not seen a key yet.
template <class C>
__device__ __forceinline__ bool move_maximum(float4v (&x)[C::RT][2], Rows<C>& st) {
    bool left = false;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        float w = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < 8; ++k) w = fmaxf(w, x[rt][k / 4][k % 4]);
        w = max_groups(w);
        const bool fresh = st.mc[rt] == kLow, any = w > -__builtin_inff();
        if (fresh && !any) left = true;
        const float mc = any && (fresh || w > st.mc[rt]) ? w : st.mc[rt];
        const float f = fresh ? 1.0f : exp2f(st.mc[rt] - mc);   // (nothing to scale before the first key)
        if (mc != st.mc[rt]) st.start[rt] = kPExp - mc;
        st.mc[rt] = mc;
        st.from[rt] = float4v{st.start[rt], st.start[rt], st.start[rt], st.start[rt]};
        st.lsum[rt] *= f;
#pragma unroll
        for (int j = 0; j < C::DT; ++j) st.o[rt][j] *= f;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) x[rt][s][r] = x[rt][s][r] - mc + kPExp;
    }
    return __any(left);
}

// One step over a tile.  special: what the makers noted of it, aside: keys that
// are left out; units: of the wave's rows; unset: some row has not seen a
// key yet.
template <class C>
__device__ __forceinline__ void tile_step(const Tile<C>& tile, int special, uint32_t aside, const int* units, int t0, const Span& sp,
                                          Rows<C>& st, bool& unset) {
    constexpr int RT = C::RT, GROUP = Fetch<C>::GROUP;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    // scores as exponents: the products start from kPExp - mc.  (Not so for float32
    // activations, where it would cost the sums bits, and extreme scales and rows,
    // whose unit is not 1: it is added at the end.)
    const bool late = C::WIDE || (special & ~3) != 0;
    if (late) {
        HR_BRANCH();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) st.from[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    float4v acc[RT][2];
    Fetch<C> now, next;
    now.keys(tile, 0);
#pragma unroll
    for (int first = 0; first < 2 * C::KS; first += GROUP) {
        HR_PHASE();
        if (first + GROUP < 2 * C::KS) next.keys(tile, first + GROUP);
        else next.values(tile, 0);
#pragma unroll
        for (int i = first; i < first + GROUP && i < 2 * C::KS; ++i) {
            const int s = i / C::KS, k = i % C::KS;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                acc[rt][s] = mfma(now.f[0][i - first], st.q[rt][0][k], k == 0 ? st.from[rt] : acc[rt][s]);
                if constexpr (C::WIDE) {
                    acc[rt][s] = mfma(now.f[0][i - first], st.q[rt][1][k], acc[rt][s]);
                    acc[rt][s] = mfma(now.f[1][i - first], st.q[rt][0][k], acc[rt][s]);
                }
            }
        }
        now = next;
    }
    HR_PHASE();
    if (late) {
        HR_BRANCH();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int unit = (special >> kShiftBits) - (C::WIDE ? st.unit[rt] : units[16 * rt + (lane & 15)]);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[rt][k / 4][k % 4] = ldexpf(acc[rt][k / 4][k % 4], unit);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) st.from[rt] = float4v{st.start[rt], st.start[rt], st.start[rt], st.start[rt]};
    }
    const bool all = t0 >= sp.flo && t0 + 32 <= sp.fhi && (special & 3) == 0 && aside == 0;
    float p[RT][8], top = 0.0f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            p[rt][k] = __builtin_amdgcn_exp2f(late ? acc[rt][k / 4][k % 4] + st.start[rt] : acc[rt][k / 4][k % 4]);
            top = fmaxf(top, p[rt][k]);
        }
    if (!all || unset || __any(top > static_cast<float>(1 << (kPExp + kSlack)))) {
        HR_BRANCH();
        if constexpr (!C::WIDE)
            if (!late) raw_scores<C>(tile, special, units, st, acc);
        if (!all) {
            // unseen scores become -inf, whatever they are
            HR_BRANCH();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = 16 * (k / 4) + 4 * g + k % 4, key = t0 + at;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const bool seen = !(special >> (k / 4) & 1) && !(aside >> at & 1) && key < st.lim[rt] && key >= st.lo[rt];
                    if (!seen) acc[rt][k / 4][k % 4] = -__builtin_inff();
                }
            }
        }
        unset = move_maximum<C>(acc, st);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int k = 0; k < 8; ++k) p[rt][k] = __builtin_amdgcn_exp2f(acc[rt][k / 4][k % 4]);
    }
    uint4v ph[RT], pl[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t h, l = 0;
            if constexpr (C::WIDE) split_f16(p[rt][2 * k], p[rt][2 * k + 1], h, l);
            else h = pack_f16(p[rt][2 * k], p[rt][2 * k + 1]);
            ph[rt][k] = h;
            pl[rt][k] = l;
        }
    const uint4v ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        st.lsum[rt] = mfma(ones, ph[rt], st.lsum[rt]);
        if constexpr (C::WIDE) st.lsum[rt] = mfma(ones, pl[rt], st.lsum[rt]);
    }
#pragma unroll
    for (int first = 0; first < C::DT; first += GROUP) {
        HR_PHASE();
        if (first + GROUP < C::DT) next.values(tile, first + GROUP);
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float4v& o = st.o[rt][first + i];
                o = mfma(now.f[0][i], ph[rt], o);
                if constexpr (C::WIDE) {
                    o = mfma(now.f[0][i], pl[rt], o);
                    o = mfma(now.f[1][i], ph[rt], o);
                }
            }
        now = next;
    }
    HR_PHASE();
}

// The same for two row tiles, one half a step behind the other, so that the
// exponentials of one are formed while the matrix unit works for the other.
// Everything else (keys that some rows do not see, extreme scales, a maximum
// that moves) is in one branch between the scores and the values.
#define HR_GROUP(what, n) __builtin_amdgcn_sched_group_barrier(what, n, 0)
enum { kMatrix = 0x8, kLdsRead = 0x100, kTranscendental = 0x400 };
__device__ __forceinline__ uint4v exponentials(const float4v (&acc)[2]) {
    uint4v ph;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        ph[k] = pack_f16(__builtin_amdgcn_exp2f(acc[k / 2][2 * k % 4]), __builtin_amdgcn_exp2f(acc[k / 2][2 * k % 4 + 1]));
    return ph;
}
template <class C>
__device__ __forceinline__ void pair_step(const Tile<C>& tile, int special, uint32_t aside, const int* units, int t0, const Span& sp,
                                          Rows<C>& st, bool& unset) {
    constexpr int N = C::DT;   // operands of keys, and of values
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const uint4v ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
    uint4v k[N], v[N];
    float4v acc[2][2];
    HR_PHASE();
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = tile.k[0][i][lane];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int i = 0; i < C::KS; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                acc[rt][s] = mfma(k[s * C::KS + i], st.q[rt][0][i], i == 0 ? st.from[rt] : acc[rt][s]);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = tile.v[0][i][lane];
    uint4v p0 = exponentials(acc[0]);
    asm volatile("" : "+v"(p0));   // (here, and not after the branch)
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, acc[i / 8][i / 4 % 2][i % 4]);
    HR_GROUP(kLdsRead, N);
    HR_GROUP(kMatrix, N + 2);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        HR_GROUP(kTranscendental, 8 / N);
        HR_GROUP(kMatrix, 1);
        HR_GROUP(kLdsRead, 1);
    }
    const bool all = t0 >= sp.flo && t0 + 32 <= sp.fhi && (special | aside) == 0;
    if (!all || unset || __any(top > static_cast<float>(kPExp + kSlack))) {
        HR_BRANCH();
        raw_scores<C>(tile, special, units, st, acc);
        if (!all) {
            // unseen scores become -inf, whatever they are
            HR_BRANCH();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = 16 * (i / 4) + 4 * g + i % 4, key = t0 + at;
#pragma unroll
                for (int rt = 0; rt < 2; ++rt) {
                    float& x = reinterpret_cast<float*>(&acc[rt][i / 4])[i % 4];
                    if ((special >> (i / 4) & 1) || (aside >> at & 1) || key >= st.lim[rt] || key < st.lo[rt]) x = -__builtin_inff();
                }
            }
        }
        unset = move_maximum<C>(acc, st);
        p0 = exponentials(acc[0]);
    }
    st.lsum[0] = mfma(ones, p0, st.lsum[0]);
#pragma unroll
    for (int i = 0; i < N; ++i) st.o[0][i] = mfma(v[i], p0, st.o[0][i]);
    const uint4v p1 = exponentials(acc[1]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        HR_GROUP(kMatrix, 1);
        HR_GROUP(kTranscendental, 8 / N);
    }
    st.lsum[1] = mfma(ones, p1, st.lsum[1]);
#pragma unroll
    for (int i = 0; i < N; ++i) st.o[1][i] = mfma(v[i], p1, st.o[1][i]);
    HR_PHASE();
}

// The exponents of a pass's value scales: those of its tiles, if they fit one
// unit, else those from the largest of the tiles' smallest on (one odd key in a
// tile, large or small, is then the one that is set aside).
template <class C>
struct PassScales {
    int lo = 1000, hi = -1000, vote = -1000;
    __device__ __forceinline__ void add(int l, int h) {
        lo = min(lo, l);
        hi = max(hi, h);
        if (h >= l) vote = max(vote, l);
    }
    __device__ __forceinline__ void settle() {
        if (hi < lo) lo = hi = 0;
        if (hi - lo > C::VRANGE) {
            lo = vote;
            hi = min(hi, lo + C::VRANGE);
        }
    }
};

// What a wave makes for the passes, besides computing: keys or values of tile
// `tile`, or nothing.  (Each is a loop of its own, so that a wave holds only
// what it loads, and no value of a load on its way passes through a branch.)
enum { kMakeKeys, kMakeValues, kMakeNothing };

template <class C, int ROLE>
__device__ __forceinline__ void passes(const CacheAttnArgs& a, const int32_t* table, int h, int tile, int begin, int end, const Span& sp,
                                       Rows<C>& st, Passes<C>& ps) {
    constexpr int S = 32 * C::TILES, N = C::TILES;
    const int lane = threadIdx.x & 63, mine = 32 * tile;
    std::conditional_t<ROLE == kMakeKeys, RawK<C>, RawV<C>> w;
    Pages now, next = pages_at(a, table, min(begin + mine, max(end - 1, 0) & ~15));
    // the tile of the pass at t, and the pages of the next.  Past the end there
    // is no page, so that nothing is read.
    const auto load = [&](int t) {
        if constexpr (ROLE == kMakeNothing) return;
        now = next;
        if (t + mine >= end) now.p[0] = now.p[1] = -1;
        load_raw<C>(a, now, h, t + mine, w);
        next = pages_at(a, table, min(t + S + mine, max(end - 1, 0) & ~15));
    };
    int own_lo = 0, own_hi = 0;         // of the tile that was announced last
    bool some = false;
    const auto announce = [&](int t, int buf) {   // the value scales' exponents of the loaded tile
        if constexpr (ROLE == kMakeValues) {
            float vs[8];
            value_scales<C>(a, w, now, t + mine, end, vs);
            exponents_of<C>(vs, own_lo, own_hi, some);
            if (lane == 0) ps.range[buf][tile] = uint2v{static_cast<uint32_t>(own_lo), static_cast<uint32_t>(own_hi)};
        }
    };
    const int* units = ps.unit[threadIdx.x >> 6];
    int made = kNoUnit;                 // the unit of the pass made last
    const auto make = [&](int t, int buf) {
        PassScales<C> sc;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint2v r = ps.range[buf][i];
            sc.add(__builtin_amdgcn_readfirstlane(static_cast<int>(r.x)), __builtin_amdgcn_readfirstlane(static_cast<int>(r.y)));
        }
        if (!(sc.hi <= made && sc.lo >= made - C::VRANGE)) {
            HR_BRANCH();
            sc.settle();
            if (!(sc.hi <= made && sc.lo >= made - C::VRANGE)) made = unit_for<C::VRANGE>(sc.lo, sc.hi);
        }
        [[maybe_unused]] uint32_t* note = reinterpret_cast<uint32_t*>(&ps.note[buf][tile]);
        if constexpr (ROLE == kMakeKeys) {
            if (t + mine < end) make_keys<C>(a, w, now, t + mine, end, st.c, ps.tile[buf][tile], note, &ps.todo.aside);
        } else if constexpr (ROLE == kMakeValues) {
            const bool check = some || own_hi > sc.hi || own_lo < sc.lo;
            if (t + mine < end)
                make_values<C>(a, w, now, t + mine, end, made, check, sc.lo, ps.tile[buf][tile], note + 2, &ps.todo.aside);
        }
    };
    load(begin);
    announce(begin, 0);
    __syncthreads();
    make(begin, 0);
    load(begin + S);
    announce(begin + S, 1);
    __syncthreads();
    bool unset = true;
    int buf = 0;
    for (int t = begin; t < end; t += S, buf ^= 1) {
        const int e = made;             // of this pass; make() may move it for the next
        if constexpr (ROLE != kMakeKeys) {
            make(t + S, buf ^ 1);
            load(t + 2 * S);
        }
        if (e != st.e) set_unit<C>(st, e);
        // (tiles that no row of the wave sees are left out)
        const int first = max(sp.lo - t, 0) >> 5, stop = (min(min(end, sp.hi) - t, S) + 31) >> 5;
#pragma unroll 1
        for (int i = first; i < stop; ++i) {
            const uint4v note = ps.note[buf][i];
            const int special = __builtin_amdgcn_readfirstlane(static_cast<int>(note.x)) | st.own, t0 = t + 32 * i;
            const uint32_t aside = __builtin_amdgcn_readfirstlane(note.y | note.z);
            if constexpr (C::RT == 2) pair_step<C>(ps.tile[buf][i], special, aside, units, t0, sp, st, unset);
            else tile_step<C>(ps.tile[buf][i], special, aside, units, t0, sp, st, unset);
        }
        if constexpr (ROLE == kMakeKeys) {
            make(t + S, buf ^ 1);
            load(t + 2 * S);
        }
        // (the exponents of the next pass were read above by every wave before
        // its own barrier, those after it go to this pass's place)
        announce(t + 2 * S, buf);
        __syncthreads();
    }
}

// One key that was set aside, at base + ... of its page, for one row (the wave's;
// the same in all lanes): its score from its own elements s (c - z), one step of
// the softmax on the row's part, p s (c - z) added.  A lane has D / 64 dimensions.
template <class C, class T>
__device__ __forceinline__ void aside_row(const CacheAttnArgs& a, const Seq& s, int h, int row, const uint8_t* base, int off, int key,
                                          float* p) {
    constexpr int D = C::D, NG = C::NG, E = D / 64;
    const int lane = threadIdx.x & 63;
    const int tok = row / a.rep, hh = row - tok * a.rep, pos = s.len - s.n + tok;
    if (a.causal && (key > pos || (a.window && key <= pos - a.window))) return;
    const T* from = static_cast<const T*>(a.q) + static_cast<int64_t>(s.start + tok) * a.q_st +
                    static_cast<int64_t>(h * a.rep + hh) * a.q_sh + lane * E;
    float q[E], k[E], v[E], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if constexpr (sizeof(T) == 2) q[i] = __uint_as_float(static_cast<uint32_t>(from[i]) << 16);
        else q[i] = from[i];
    }
    if (a.rotate) {
#pragma unroll
        for (int x = 1; x < E; x *= 2)
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (!(i & x)) {
                    const float u = q[i], w = q[i + x];
                    q[i] = u + w;
                    q[i + x] = u - w;
                }
        for (int x = 1; x < 64; x *= 2)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float o = __shfl_xor(q[i], x);
                q[i] = lane & x ? o - q[i] : o + q[i];
            }
#pragma unroll
        for (int i = 0; i < E; ++i) q[i] *= a.norm;
    }
    const auto elements = [&](int codes, int scales, int zeros, float (&to)[E]) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int dim = lane * E + i, at = off * NG + dim / (D / NG);
            uint32_t c = base[codes + off * (D / 2) + dim / 2] >> (4 * (dim & 1)) & 15u;
            const uint32_t z = a.pg.sym ? 8u : base[zeros + at / 2] >> (4 * (at & 1)) & 15u;
            if (a.pg.sym) c ^= 8u;
            const float scale = C::SF32 ? reinterpret_cast<const float*>(base + scales)[at]
                                        : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base + scales)[at]) << 16);
            to[i] = scale * static_cast<float>(static_cast<int>(c) - static_cast<int>(z));
        }
    };
    elements(a.pg.kc, a.pg.ks, a.pg.kz, k);
    elements(a.pg.vc, a.pg.vs, a.pg.vz, v);
#pragma unroll
    for (int i = 0; i < E; ++i) sum = fmaf(q[i], k[i], sum);
    for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
    float w = sum * (a.scale * kLog2e);
    asm("" : "+v"(w));                     // (rounded, as the maximum is that it is compared with)
    const float was = p[D];
    const float mc = fmaxf(was, w), f = exp2f(was - mc), pr = exp2f(w - mc);
    const float l = fmaf(p[D + 1], f, pr);
#pragma unroll
    for (int i = 0; i < E; ++i) p[lane * E + i] = fmaf(p[lane * E + i], f, pr * v[i]);
    p[D] = mc;                             // (every lane its own copy of these two)
    p[D + 1] = l;
}

// The keys of a segment that were set aside, for the rows' parts at `part`, a row
// to a wave at a time; last: the rows are finished here.  A function of its own,
// that is called: inlined, what it needs takes registers in the loops before it
// (10% of a step's time, and where none are free many times that).
typedef const CacheAttnArgs __attribute__((address_space(4)))* ConstArgs;
template <class C, class T>
__device__ __attribute__((noinline)) void sweep_rows(ConstArgs args, Todo* todo) {
    const CacheAttnArgs& a = *(const CacheAttnArgs*)(args);
    constexpr int WAVES = C::THREADS / 64, D = C::D, E = D / 64, TILES = C::SHARED ? C::TILES : 1;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int b = __builtin_amdgcn_readfirstlane(todo->b), h = __builtin_amdgcn_readfirstlane(todo->h);
    const int r0 = __builtin_amdgcn_readfirstlane(todo->r0), k0 = todo->k0, k1 = todo->k1;
    const float c = todo->c;
    const bool last = todo->part == nullptr;
    float* part = last ? todo->spare : todo->part;
    const Seq s = seq_at<true>(a.sq, a.pg.logp, b);
    const int rows = min(s.n * a.rep - r0, C::ROWS);
    const Span sp = span_of(a, s, r0, r0 + rows);
    const int32_t* table = a.sq.table + static_cast<int64_t>(b) * a.sq.max_pages;
    const int begin = __builtin_amdgcn_readfirstlane(max(k0, sp.lo & ~31)), end = __builtin_amdgcn_readfirstlane(min(k1, sp.hi));
    __threadfence_block();
    __syncthreads();                       // (the parts were written by other waves)
    for (int t = begin; t < end; t += 32 * TILES) {
        PassScales<C> sc;
        for (int turn = C::SHARED ? 0 : 1; turn < 2; ++turn) {   // with shared operands the pass's unit first
            for (int t0 = t; t0 < min(t + 32 * TILES, end); t0 += 32) {
                const Pages pages = pages_at(a, table, t0);
                RawV<C> rv;
                load_raw<C>(a, pages, h, t0, rv);
                float vs[8];
                uint32_t aside;
                if constexpr (C::SHARED) {
                    value_scales<C>(a, rv, pages, t0, end, vs);
                    if (turn == 0) {
                        int lo, hi;
                        bool some;
                        exponents_of<C>(vs, lo, hi, some);
                        sc.add(lo, hi);
                        continue;
                    }
                    bool out[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) out[x] = set_aside<C::VRANGE>(vs[x], sc.lo);
                    RawK<C> rk;
                    load_raw<C>(a, pages, h, t0, rk);
                    float ks[2][C::NG];
                    key_unit<C>(rk, t0, end, c, ks, aside);
                    aside = __builtin_amdgcn_readfirstlane(aside) | keys_of(out);
                } else {
                    int lo, hi;
                    step_scales<C>(rv, vs);
                    drop_unseen(a, pages, t0, end, 0.0f, vs);
                    aside = aside_of<C>(vs, lo, hi);
                }
                while (aside) {
                    const int i = __builtin_ctz(aside), key = t0 + i, page = i < 16 ? pages.p[0] : pages.p[1];
                    aside &= aside - 1;
                    if (key >= end || !present(a, page)) continue;
                    const uint8_t* base = a.pool + page * a.pg.page_bytes + h * a.pg.head_bytes;
                    for (int row = wave; row < rows; row += WAVES)
                        aside_row<C, T>(a, s, h, r0 + row, base, key & (a.pg.page - 1), key, part + row * part_stride<C>());
                }
            }
            if (turn == 0) sc.settle();
        }
    }
    if (last) {
        for (int row = wave; row < rows; row += WAVES) {
            const float* p = part + row * part_stride<C>();
            const int tok = (r0 + row) / a.rep;
            const int64_t t = s.start + tok, head = h * a.rep + (r0 + row) - tok * a.rep;
            const float l = p[D + 1], inv = l == 0.0f ? 0.0f : 1.0f / l;
            T* to = static_cast<T*>(a.out) + t * a.o_st + head * a.o_sh + lane * E;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = p[lane * E + i] * inv;
                if constexpr (sizeof(T) == 2) to[i] = static_cast<uint16_t>(to_bf16(x));
                else to[i] = x;
            }
            if (a.lse && lane == 0) a.lse[t * a.hq + head] = log_sum(p[D], l);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) todo->aside = 0;
    __syncthreads();
}

// Rows [r0, r0 + ROWS) of kv head h of a sequence over the keys [k0, k1);
// part: where a partial result goes (else the rows are finished here); spare: for
// one of a segment that sets keys aside.
template <class C, class T>
__device__ __forceinline__ void shared_segment(const CacheAttnArgs& a, const Seq& s, int b, int h, int r0, int k0, int k1,
                                               float* part, float* spare, float* lds) {
    constexpr int N = C::TILES;
    Passes<C>& ps = *reinterpret_cast<Passes<C>*>(lds);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t* table = a.sq.table + static_cast<int64_t>(b) * a.sq.max_pages;
    const int row = r0 + wave * 16 * C::RT, last = s.n * a.rep;
    const Span all = span_of(a, s, r0, min(r0 + C::ROWS, last));
    Span sp = {0, 0, 0, 0};
    if (row < last) sp = span_of(a, s, row, min(row + 16 * C::RT, last));
    const int begin = max(k0, all.lo & ~31), end = min(k1, all.hi);
    Rows<C> st;
    load_rows<C, T>(a, s, h, row, st, ps.top, ps.unit[wave]);
    if (threadIdx.x == 0) ps.todo.set(b, h, r0, k0, k1, st.c, part, spare);
    if (wave < N) passes<C, kMakeKeys>(a, table, h, wave, begin, end, sp, st, ps);
    else if (wave < 2 * N) passes<C, kMakeValues>(a, table, h, wave - N, begin, end, sp, st, ps);
    else passes<C, kMakeNothing>(a, table, h, 0, begin, end, sp, st, ps);
    // to value units, as the other kernels leave them
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        st.l[rt] = ldexpf(st.lsum[rt][0], -kPExp);
#pragma unroll
        for (int j = 0; j < C::DT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) st.o[rt][j][r] = ldexpf(st.o[rt][j][r], st.e - kPExp - kSExp);
    }
    const bool aside = __builtin_amdgcn_readfirstlane(ps.todo.aside) != 0;
    if (aside && !part) part = spare;
    put_rows<C, T>(a, s, h, row, st, part, row - r0);
    if (aside) {
        HR_BRANCH();
        sweep_rows<C, T>((ConstArgs)(__builtin_amdgcn_kernarg_segment_ptr()), &ps.todo);
    }
}

// Rows [r0, r0 + ROWS) of kv head h of a sequence over the keys [k0, k1);
// part: where a partial result goes (else the rows are finished here); spare: for
// one of a segment that sets keys aside.
template <class C, class T>
__device__ __forceinline__ void segment(const CacheAttnArgs& a, const Seq& s, int b, int h, int r0, int k0, int k1,
                                        float* part, float* spare, float* lds) {
    if constexpr (C::SHARED) {
        shared_segment<C, T>(a, s, b, h, r0, k0, k1, part, spare, lds);
    } else {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const Span sp = span_of(a, s, r0, min(r0 + C::ROWS, s.n * a.rep));
        Rows<C> st;
        Walk<C> keys;
        keys.table = a.sq.table + static_cast<int64_t>(b) * a.sq.max_pages;
        keys.h = h;
        keys.start(a, sp, k0, k1, wave);
        int* units = reinterpret_cast<int*>(lds + join_floats<C>()) + wave * 16 * C::RT;
        Todo* todo = todo_at<C>(lds);
        if (threadIdx.x == 0) todo->set(b, h, r0, k0, k1, 0.0f, part, spare);
        load_rows<C, T>(a, s, h, r0, st, lds, units);
        if (keys.t < keys.end) {
            st.e = keys.first_unit(a);
            st.big = 0.0f;
            st.small = 0x1p126f;
            keys.template run<false>(a, sp, nullptr, units, st);
            if (__any(!(st.big < power(C::VEXP) && st.small >= power(C::VEXP - C::VRANGE - 1)))) {
                HR_BRANCH();
                st.e = kNoUnit;
#pragma unroll
                for (int rt = 0; rt < C::RT; ++rt) {
                    st.mc[rt] = kLow;
                    st.l[rt] = 0.0f;
#pragma unroll
                    for (int j = 0; j < C::DT; ++j) st.o[rt][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
                }
                keys.start(a, sp, k0, k1, wave);
                keys.template run<true>(a, sp, &todo->aside, units, st);
            }
        }
        settle<C>(st);
        if (join_waves<C, T>(a, s, h, r0, st, part, spare, &todo->aside, lds)) {
            HR_BRANCH();
            sweep_rows<C, T>((ConstArgs)(__builtin_amdgcn_kernarg_segment_ptr()), todo);
        }
    }
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// A walk over the row blocks of a sequence: their rows and the keys that they
// see.  (Tokens are counted along, as a division for each block would cost more
// than the rest.)
template <class C>
__device__ __forceinline__ uint32_t row_blocks(const CacheAttnArgs& a, const Seq& s) {
    return (static_cast<uint32_t>(s.n) * static_cast<uint32_t>(a.rep) + C::ROWS - 1) / C::ROWS;
}
template <class C>
struct RowBlocks {
    int rep, step, over;      // ROWS = step rep + over
    int past, len, last;      // keys before the new tokens (may be negative), all keys, the last token
    int window;
    bool causal;
    int tok, rem;             // the token of the block's first row, and how far the row is into it
    int first, blocks;        // first key (a multiple of 32), key blocks (at least one, so that rows that see nothing are written)
    __device__ __forceinline__ RowBlocks(const CacheAttnArgs& a, const Seq& s, uint32_t i) {
        rep = a.rep;
        step = a.step;
        over = a.over;
        past = s.len - s.n;
        len = s.len;
        last = s.n - 1;
        window = a.window;
        causal = a.causal != 0;
        tok = rem = 0;
        if (i > 0) {
            const uint32_t r0 = i * C::ROWS;
            tok = static_cast<int>(r0 / static_cast<uint32_t>(rep));
            rem = static_cast<int>(r0) - tok * rep;
        }
        see();
    }
    __device__ __forceinline__ void next() {
        tok += step;
        rem += over;
        if (rem >= rep) {
            rem -= rep;
            ++tok;
        }
        see();
    }
    __device__ __forceinline__ void see() {
        const int x = rem + over;   // the last row's token: ceil((rem + ROWS) / rep) - 1 past tok
        const int to = min(tok + step + (x > 0 ? 1 : 0) + (x > rep ? 1 : 0) - 1, last);
        const int hi = causal ? min(max(past + to + 1, 0), len) : len;
        const int lo = window ? max(past + tok - window + 1, 0) : 0;
        first = min(lo, hi) & ~31;
        blocks = max((hi - first + C::KEYS - 1) / C::KEYS, 1);
    }
};

// Work is counted in items.  For each kv head and row block a unit has kSetup
// items that stand for its start and end, then one for each block of keys.
// (few rows: 7 us against 1.7 for a block; many: with 1, 2, 3, 4 items one sequence
// of 64 tokens behind 8000 keys took 112, 71, 56, 55 us, and other calls the same
// within 5%)
constexpr int kSetup = 4;
// the items of row blocks [i, n) for one kv head; most: the largest unit
template <class C>
__device__ __forceinline__ int64_t items_of(const CacheAttnArgs& a, const Seq& s, uint32_t i, uint32_t n, int* most) {
    if (i >= n) return 0;
    RowBlocks<C> rb(a, s, i);
    int64_t sum = rb.blocks + kSetup;
    *most = max(*most, rb.blocks + kSetup);
    for (++i; i < n; ++i) {
        rb.next();
        sum += rb.blocks + kSetup;
        *most = max(*most, rb.blocks + kSetup);
    }
    return sum;
}

// f over the values of this lane and those before it, by moves between lanes
// (a general shuffle goes through LDS); 0 is f's identity.
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t moved(int64_t v) {
    const uint32_t lo = moved<CTRL, ROWS>(static_cast<int>(v)), hi = moved<CTRL, ROWS>(static_cast<int>(v >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}
template <class V, class F>
__device__ __forceinline__ V scan_wave(V v, F f) {
    v = f(v, moved<0x111, 0xF>(v));   // the lane 1, 2, 4, 8 before, in a row of 16
    v = f(v, moved<0x112, 0xF>(v));
    v = f(v, moved<0x114, 0xF>(v));
    v = f(v, moved<0x118, 0xF>(v));
    v = f(v, moved<0x142, 0xA>(v));   // a row's last lane to the row after it, in the second and fourth
    v = f(v, moved<0x143, 0xC>(v));   // lane 31 to the upper half
    return v;
}
struct Add {
    __device__ __forceinline__ int64_t operator()(int64_t x, int64_t y) const { return x + y; }
};
struct Most {
    __device__ __forceinline__ int operator()(int x, int y) const { return max(x, y); }
};

// Sums of N values over the workgroup's threads before this one, and over all;
// the largest of another (N = 2).
template <int THREADS, int N>
__device__ __forceinline__ void scan_items(int64_t (&v)[2], int64_t (&all)[2], int* most, int64_t* lds) {
    constexpr int W = THREADS / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t inc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) inc[i] = scan_wave(v[i], Add());
    int m = 0;
    if constexpr (N == 2) m = scan_wave(*most, Most());
    __syncthreads();
    if (lane == 63) {
#pragma unroll
        for (int i = 0; i < N; ++i) lds[i * W + wave] = inc[i];
        if constexpr (N == 2) lds[2 * W + wave] = m;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        int64_t before = 0;
        all[i] = 0;
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const int64_t y = lds[i * W + x];
            if (x < wave) before += y;
            all[i] += y;
        }
        v[i] = before + inc[i] - v[i];
    }
    if constexpr (N == 2) {
#pragma unroll
        for (int x = 0; x < W; ++x) *most = max(*most, static_cast<int>(lds[2 * W + x]));
    }
}

// How the items are shared out: every workgroup of the first nw has `share`,
// and the first `rest` of them one more.
struct Shares {
    int64_t total, share, rest;
    __device__ __forceinline__ int64_t first(int64_t w) const { return w * share + min(w, rest); }
    // the workgroup that holds item u
    __device__ __forceinline__ int64_t holder(int64_t u) const {
        const int64_t longer = rest * (share + 1);
        return u < longer ? u / (share + 1) : rest + (u - longer) / share;
    }
};
__device__ __forceinline__ Shares shares_of(int64_t total, int workers) {
    const uint32_t nw = total < workers ? static_cast<uint32_t>(max(total, int64_t{1})) : workers;
    Shares sh;
    sh.total = total;
    sh.share = total < (int64_t{1} << 31) ? static_cast<int64_t>(static_cast<uint32_t>(total) / nw) : total / nw;
    sh.rest = total - sh.share * nw;
    return sh;
}

// What cutting costs a workgroup, in items: a second unit's start and end, and
// the joining launch.  Always cut, by this rule and always whole, us: 4 prompts of
// 512 tokens (32 heads over 8 of 128) 67, 52, 53; 8 of 256 behind 744 keys (heads of
// 64) 56, 48, 50; 1 of 512 behind 7488 keys 116, 116, 296; 8 of 2048 behind 6144
// 2147, 2138, 2329.
constexpr int kCut = 8;

// Workgroup w: its items [i0, i1), the sequence b that holds the first and the
// items before that sequence.  Every thread takes part.  whole: units are not
// cut, as sharing them out whole is no longer for the workgroup that has most;
// each counts as one item then.
struct Place {
    Shares sh;
    int64_t i0, i1, before;
    int b;
    bool whole;
    Seq s;                // sequence b
};
template <class C>
__device__ __forceinline__ Place place(const CacheAttnArgs& a, int64_t* lds) {
    constexpr int OUT = 3 * C::THREADS / 64, N = C::SHARED ? 2 : 1;
    const int tid = threadIdx.x;
    // few sequences: 2^per threads for each, with a part of its row blocks
    int per = 0;
    while (per < 6 && a.sq.rows <= C::THREADS >> (per + 1)) ++per;
    const int nth = tid >> per, part = tid & ((1 << per) - 1), step = C::THREADS >> per;
    Place p;
    Seq s = {0, 0, 0};
    int most = 0;
    int64_t total[2] = {0, 0}, own[2], pre[2], all[2];
    const auto items = [&](int b) {
        own[0] = own[1] = 0;
        uint32_t n = 0;
        if (b < a.sq.rows) {
            s = seq_at<false>(a.sq, a.pg.logp, b);
            n = row_blocks<C>(a, s);
            const uint32_t each = (n + (1u << per) - 1) >> per, i = part * each;
            own[0] = items_of<C>(a, s, i, min(i + each, n), &most);
        }
        if (__any(n > 1))
            for (int x = 1; x < 1 << per; x *= 2) own[0] += __shfl_xor(own[0], x);
        if (part == 0) own[1] = static_cast<int64_t>(n) * a.pg.hkv;
        pre[0] = own[0] = part == 0 ? own[0] * a.pg.hkv : 0;
        pre[1] = own[1];
        scan_items<C::THREADS, N>(pre, all, &most, lds);
    };
    // (a call of no more sequences than threads is scanned once)
    for (int c = 0; c < a.sq.rows; c += step) {
        items(c + nth);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            pre[i] += total[i];
            total[i] += all[i];
        }
    }
    p.sh = shares_of(uniform64(total[0]), a.workers);
    p.whole = false;
    if constexpr (N == 2) {
        const Shares whole = shares_of(uniform64(total[1]), a.workers);
        p.whole = (whole.share + (whole.rest > 0 ? 1 : 0)) * __builtin_amdgcn_readfirstlane(most) <= p.sh.share + kCut;
        if (p.whole) p.sh = whole;
    }
    const int64_t w = blockIdx.x;
    p.i0 = min(p.sh.first(w), p.sh.total);
    p.i1 = min(p.sh.first(w + 1), p.sh.total);
    if (tid == 0) lds[OUT] = -1;
    int64_t base[2] = {0, 0};
    for (int c = 0; c < a.sq.rows; c += step) {
        if (a.sq.rows > step) {
            items(c + nth);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                pre[i] += base[i];
                base[i] += all[i];
            }
        }
        __syncthreads();
        const int64_t at = p.whole ? pre[1] : pre[0];
        if (p.i0 >= at && p.i0 < at + (p.whole ? own[1] : own[0])) {
            lds[OUT] = c + nth;
            lds[OUT + 1] = at;
            lds[OUT + 2] = s.start;
            lds[OUT + 3] = static_cast<int64_t>(s.n) << 32 | static_cast<uint32_t>(s.len);
        }
        __syncthreads();
        if (lds[OUT] >= 0) break;
    }
    p.b = lds[OUT] >= 0 ? __builtin_amdgcn_readfirstlane(static_cast<int>(lds[OUT])) : a.sq.rows;
    p.before = uniform64(lds[OUT + 1]);
    const int64_t nl = uniform64(lds[OUT + 3]);
    p.s = {__builtin_amdgcn_readfirstlane(static_cast<int>(lds[OUT + 2])), static_cast<int>(nl >> 32), static_cast<int>(nl)};
    __syncthreads();
    return p;
}

// Where item `at` of a sequence is: its kv head, row block and unit's first
// item; each: the items of a kv head.  Every lane of the wave takes part.
struct Found {
    int h;
    uint32_t rb;
    int64_t first, each;
};
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {   // (of small numbers, mostly)
    return x < (int64_t{1} << 31) && y < (int64_t{1} << 31) ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
}
template <class C>
__device__ __forceinline__ Found find_item(const CacheAttnArgs& a, const Seq& s, uint32_t n, int64_t at, bool whole) {
    Found f;
    if (whole) {
        f.each = n;
        f.h = static_cast<int>(divide(at, n));
        f.rb = static_cast<uint32_t>(at - f.h * f.each);
        f.first = at;
        return f;
    }
    if (n == 1) {
        f.each = RowBlocks<C>(a, s, 0).blocks + kSetup;
        f.h = static_cast<int>(divide(at, f.each));
        f.rb = 0;
        f.first = f.h * f.each;
        return f;
    }
    int most = 0;
    const uint32_t part = (n + 63) / 64, i = min((threadIdx.x & 63) * part, n);
    const int64_t own = items_of<C>(a, s, i, min(i + part, n), &most), inc = scan_wave(own, Add());
    f.each = uniform64(__shfl(inc, 63));
    f.h = static_cast<int>(divide(at, f.each));
    at -= f.h * f.each;
    // the lane that has it, and from there on
    const uint64_t who = __ballot(at >= inc - own && at < inc);
    const int l = who ? __builtin_ctzll(who) : 0;
    f.rb = __builtin_amdgcn_readfirstlane(__shfl(i, l));
    f.first = uniform64(__shfl(inc - own, l));
    RowBlocks<C> rb(a, s, f.rb);
    while (f.first + rb.blocks + kSetup <= at) {
        f.first += rb.blocks + kSetup;
        ++f.rb;
        rb.next();
    }
    f.first += f.h * f.each;
    return f;
}

// What the joining launch needs of a unit that begins in a workgroup and goes
// on in the next ones.
struct Cut {
    int start, n;    // the sequence's first token and number of tokens
    int h, r0;       // kv head, first query row
    int last;        // the workgroup that ends it; -1: nothing to join
};

// Split form: workgroup w takes an equal share of all items.  A unit that it
// does not hold whole goes to scratch slot 2 w + 1 if it begins here, else 2 w.
template <class C, class T>
__global__ void __launch_bounds__(C::THREADS, C::WAVES) cache_attn_split(const CacheAttnArgs a) {
    __shared__ float4v lds4[lds_floats<C>() / 4 + 1];
    float* lds = reinterpret_cast<float*>(lds4);
    if (threadIdx.x == 0) todo_at<C>(lds)->aside = 0;
    const Place p = place<C>(a, reinterpret_cast<int64_t*>(lds));
    int64_t i0 = p.i0;
    const int64_t i1 = p.i1;
    int64_t before = p.before;
    constexpr int SLOT = C::ROWS * part_stride<C>();
    Cut* cuts = reinterpret_cast<Cut*>(a.work + static_cast<int64_t>(a.workers) * 2 * SLOT);
    Cut cut = {0, 0, 0, 0, -1};
    for (int b = p.b; b < a.sq.rows && i0 < i1; ++b) {
        const Seq s = b == p.b ? p.s : seq_at<true>(a.sq, a.pg.logp, b);
        const uint32_t n = row_blocks<C>(a, s);
        if (n == 0) continue;
        Found f = find_item<C>(a, s, n, i0 - before, p.whole);
        int64_t unit = before + f.first;
        for (int h = f.h; h < a.pg.hkv && i0 < i1; ++h, f.rb = 0) {
            RowBlocks<C> rb(a, s, f.rb);
            for (uint32_t i = f.rb; i < n && i0 < i1; ++i) {
                const int size = p.whole ? 1 : rb.blocks + kSetup;
                const int from = static_cast<int>(i0 - unit), to = static_cast<int>(min(i1 - unit, static_cast<int64_t>(size)));
                const int k = p.whole ? 0 : max(from - kSetup, 0), end = p.whole ? rb.blocks : to - kSetup;
                if (end > k) {           // (else only items of the unit's start)
                    const int r0 = static_cast<int>(i * C::ROWS);
                    // (a unit that ends here leaves the second slot free, which a
                    // unit that goes on takes after it)
                    float* part = nullptr;
                    float* spare = a.work + (2 * static_cast<int64_t>(blockIdx.x) + 1) * SLOT;
                    if (k > 0 || end < rb.blocks) part = spare - (k == 0 ? 0 : SLOT);
                    if (k == 0 && end < rb.blocks) cut = {s.start, s.n, h, r0, static_cast<int>(p.sh.holder(unit + size - 1))};
                    segment<C, T>(a, s, b, h, r0, rb.first + k * C::KEYS, rb.first + end * C::KEYS, part, spare, lds);
                }
                i0 = unit + to;
                unit += size;
                rb.next();
            }
        }
        before += f.each * a.pg.hkv;
    }
    if (threadIdx.x == 0) cuts[blockIdx.x] = cut;
}

// Joins the parts of units that were cut, in the order of their keys:
// blockIdx.x = w takes the unit that begins in workgroup w, a wave for a row.
// D / 4 lanes read a part, four dimensions each, the others the next ones, and
// four parts are on their way at a time.
template <class C, class T>
__global__ void __launch_bounds__(256) cache_attn_join(const CacheAttnArgs a) {
    constexpr int D = C::D, L = D / 4, AT = 64 / L, PS = part_stride<C>(), SLOT = C::ROWS * PS;
    const Cut* cuts = reinterpret_cast<const Cut*>(a.work + static_cast<int64_t>(a.workers) * 2 * SLOT);
    const Cut cut = cuts[blockIdx.x];
    const int lane = threadIdx.x & 63, row = blockIdx.y * 4 + (threadIdx.x >> 6);
    const int at = cut.r0 + row;
    if (cut.last < 0 || row >= C::ROWS || at >= cut.n * a.rep) return;
    const int parts = cut.last - static_cast<int>(blockIdx.x) + 1;
    const float* first = a.work + 2 * static_cast<int64_t>(blockIdx.x) * SLOT + row * PS;
    float m = kLow, l = 0.0f;
    float4v o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = lane / L; p0 < parts; p0 += 4 * AT) {
        float4v x[4];
        float2 ml[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = min(p0 + i * AT, parts - 1);
            const float* from = first + (2 * static_cast<int64_t>(p) + (p == 0 ? 1 : 0)) * SLOT;
            x[i] = *reinterpret_cast<const float4v*>(from + lane % L * 4);
            ml[i] = *reinterpret_cast<const float2*>(from + D);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p0 + i * AT >= parts) break;
            const float top = fmaxf(m, ml[i].x), f = exp2f(m - top), pf = exp2f(ml[i].x - top);
            l = l * f + ml[i].y * pf;
            o = o * f + x[i] * pf;
            m = top;
        }
    }
#pragma unroll
    for (int x = L; x < 64; x *= 2) {
        const float om = __shfl_xor(m, x), ol = __shfl_xor(l, x);
        const float4v oo = {__shfl_xor(o[0], x), __shfl_xor(o[1], x), __shfl_xor(o[2], x), __shfl_xor(o[3], x)};
        const float top = fmaxf(m, om), f = exp2f(m - top), pf = exp2f(om - top);
        l = l * f + ol * pf;
        o = o * f + oo * pf;
        m = top;
    }
    const int tok = at / a.rep;
    const int64_t t = cut.start + tok, head = cut.h * a.rep + at - tok * a.rep;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (lane < L) store4<T>(static_cast<T*>(a.out) + t * a.o_st + head * a.o_sh + 4 * lane, o * inv);
    if (a.lse && lane == 0) a.lse[t * a.hq + head] = log_sum(m, l);
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
        if ((e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, cache_attn_split<C, T>, C::THREADS, 0)) != hipSuccess)
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
int family(const CacheAttnArgs* a, int* workers, void* stream) {
    if (workers) return split_workers<C, T>(workers);
    hipStream_t s = static_cast<hipStream_t>(stream);
    CacheAttnArgs args = *a;
    args.step = C::ROWS / a->rep;
    args.over = C::ROWS % a->rep;
    hipLaunchKernelGGL((cache_attn_split<C, T>), dim3(a->workers), dim3(C::THREADS), 0, s, args);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return static_cast<int>(e);
    hipLaunchKernelGGL((cache_attn_join<C, T>), dim3(a->workers, C::ROWS / 4), dim3(256), 0, s, args);
    return static_cast<int>(hipGetLastError());
}

template <int D, int NG, bool SF32>
int pick_shape(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    if (k.wide) {
        if (k.wr == 1) return family<Cfg<D, NG, SF32, true, 1, 1>, float>(a, workers, stream);
        return family<Cfg<D, NG, SF32, true, 1, 8>, float>(a, workers, stream);
    }
    if (k.wr == 1) {
        if constexpr (D <= 128 && NG == 1)
            if (k.rt == 2) return family<Cfg<D, NG, SF32, false, 2, 1>, uint16_t>(a, workers, stream);
        return family<Cfg<D, NG, SF32, false, 1, 1>, uint16_t>(a, workers, stream);
    }
    return family<Cfg<D, NG, SF32, false, D == 256 ? 1 : 2, 8>, uint16_t>(a, workers, stream);
}

template <int D, int NG>
int pick_scales(const CacheAttnKey& k, const CacheAttnArgs* a, int* workers, void* stream) {
    return k.sf32 ? pick_shape<D, NG, true>(k, a, workers, stream) : pick_shape<D, NG, false>(k, a, workers, stream);
}

}  // namespace
}  // namespace hr
