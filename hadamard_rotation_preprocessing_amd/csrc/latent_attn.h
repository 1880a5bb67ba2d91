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
//   The softmax is taken in one pass.  P_g goes into the product as float16, one for
// bfloat16 activations (11 bits, of which the result keeps 8) and a pair for float32, so its
// reference m follows the largest exp(w - m) s_g that the row has seen: probabilities
// are at most 2^kTop, 2^kSet when the reference is set, and what a row does not see
// has no part in it.  Where scales are below 2^-92 or above 2^100 float32's own range
// ends (the sum of exponentials is in the same units).
//
// Layout.  A workgroup takes M = 16 RT WR query rows (new tokens x heads) of a
// sequence, and 32 keys a step, in waves of two kinds that work side by side, one step
// apart, with one barrier a step:
//   2 WR score waves form S^T = C Q^T (A operand: 16 keys out of LDS; B operand: 16 RT
//   rows, in registers throughout) and put probabilities into LDS;
//   4 value waves turn the packed codes of the step after into float16 operands in
//   LDS, and add O^T += C^T P^T of the step before for all M rows, a quarter of the
//   dimensions each.  C^T comes out of the same operands by transposing reads
//   (ds_read_b64_tr_b16).  The codes are on their way from memory for kAhead steps.
// A SIMD has a wave of each kind, so that one's matrix steps run while the other is at
// its exponentials or codes.  P^T's 32 keys stand in the order 4 g + i, 16 + 4 g + i of
// the registers of two score tiles.  Elements of eight of a vector stand in the order
// 0 4 1 5 2 6 3 7 throughout: that of the nibbles of a word under two masks.
//
// Split.  latent_query rotates the queries, turns them into operands in the scratch
// and numbers the work: a unit is a block of M rows of a sequence, an item 64 keys of
// it, and every workgroup takes an equal, contiguous run of all items.  A row's sums
// are left in the scratch, for units that are cut in parts, and latent_finish joins
// the parts in key order, divides, rotates back and rounds.
//
// Measured.  32 sequences of up to 32768, one token, 128 heads, latents of 512 in four
// groups: latent_query 7 us, latent_sums 145 us (465 TFLOP/s, 1.55 us a step of 32 keys
// and 64 rows), latent_finish 15 us; the call 164 us.  By counters the matrix units are
// busy 20% of the cycles, the vector units 30%, LDS 24% (and 4% with conflicts), and waves
// wait 54% of their time: two waves a SIMD, of two kinds that meet at a barrier each step,
// and chains of LDS writes, transposing reads and matrix steps in each.  Registers allow
// no third: this kernel takes all 256 and spills 45 (all those of 64 rows and latents of
// 512 spill 32 to 46, the float32 ones 7 to 27; those of latents of 256 none).  128 heads
// are two units of 64 rows, which load and unpack every code twice.  Tried: waves of one
// kind, each with scores and values, 517 us for the whole call where this form takes 165;
// sixteen waves with half the registers 2.44 us a step; codes turned into operands in
// registers by every wave, without LDS, 1.99 us a step.
// One sequence of 331, 16 heads: 4.0, 13.2 and 4.5 us, of which most is latency: three
// workgroups take part, one of them with items of set-up alone.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

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
constexpr float kTop = 0x1p15f;       // largest probability (float16 ends at 65504)
constexpr int kSet = 8;               // log2 of the largest one when a reference is set
constexpr int kLeastRef = -100;       // how far (log2) a reference may lie below the largest score
constexpr float kMostExp = 0x1p110f;  // largest exponential
constexpr int kBatch = 4;             // operands of scores loaded at once
constexpr int kAhead = 3;             // steps that keys are loaded ahead (as many as there are buffers)
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
// floor(log2(v)) of v >= 0 that is a normal number (-127 of smaller ones, 128 of larger)
__device__ __forceinline__ int exponent(float v) { return static_cast<int>((__float_as_uint(v) >> 23) & 255) - 127; }

// Matrix steps stay in order, with the loads of the operands of kBatch of them ahead.
// (Measured with 512 in four groups: without these barriers to the scheduler the kernels
// spill as many registers, or up to 6 fewer, and a server's step takes 163 us for 165.)
#define HR_PHASE() __builtin_amdgcn_sched_barrier(0)
// The kernel's lambdas hold its registers: one that is called would keep them in memory.
#define HR_INLINE __attribute__((always_inline))

template <int D_, int NG_, bool SF32_, bool WIDE_, int RT_, int WR_>
struct Cfg {
    static constexpr int D = D_, NG = NG_, RT = RT_, WR = WR_;
    static constexpr bool SF32 = SF32_, WIDE = WIDE_;
    static constexpr int WK = 2, SCORES = WR * WK, VALUES = 4, THREADS = 64 * (SCORES + VALUES);   // waves
    static constexpr int KEYS = 16 * WK;           // of a step
    static constexpr int TILES = RT * WR, M = 16 * TILES;
    static constexpr int T = WIDE ? 2 : 1;         // float16 terms of a query and a probability
    static constexpr int TR = WIDE ? 3 : 1;        // bfloat16 terms of a rotary query
    static constexpr int KS = D / 32, G = D / NG, KG = KS / NG;
    static constexpr int DW = D / VALUES, DT = DW / 16;   // dimensions of a value wave
    static constexpr int LK = 64 / (KEYS / VALUES);       // lanes that share a key's codes
    static constexpr int CW = D / 8 / LK;          // words of codes of a lane
    static constexpr int VS = 2 * (D + kRope) + 32;       // bytes of a key's operands in LDS (64 banks of 4: an eighth more than a multiple of all)
    static constexpr int PS = 2 * KEYS + 16;       // bytes of a row's probabilities
    static constexpr int QS = 2 * (T * D + TR * kRope);   // bytes of a row's query in the scratch
    static constexpr int RS = D + 4;               // floats of a row's sums
};

// Integers read at an address that is the same in all lanes: through the scalar
// cache, into scalar registers.
typedef const int32_t __attribute__((address_space(4)))* ConstInts;
typedef const int64_t __attribute__((address_space(4)))* ConstLongs;

// A sequence of the call, clamped so that nothing leaves its buffer.  UNI: b is the same
// in all lanes.
struct Seq {
    int start, n, len;
};
template <bool UNI>
__device__ __forceinline__ int int_at(const int32_t* p, int b) {
    if constexpr (UNI) return ((ConstInts)(p))[b];
    else return p[b];
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
    r.len = static_cast<int>(min(static_cast<int64_t>(max(int_at<UNI>(s.lens, b), 0)), static_cast<int64_t>(s.max_pages) << logp));
    return r;
}
// items of a unit of a sequence, and its units.  An item is kItem keys; a unit that has
// any counts kSetUp items more, before them, for what it costs beside its keys.  (32
// sequences of up to 32768 and 128 heads take 162 us with 6, 219 with 0, 168 with 3 and
// 165 with 12; 8 sequences of 2000, 40 new tokens, 32 heads 127, 129, 126 and 137; one
// sequence the same with all of them.)
constexpr int kItem = 64, kSetUp = 6;
__device__ __forceinline__ int items_of(const Seq& s) {
    return s.len > 0 ? static_cast<int>((static_cast<int64_t>(s.len) + kItem - 1) / kItem) + kSetUp : 0;
}
template <class C>
__device__ __forceinline__ int units_of(const Seq& s, int heads) {
    return static_cast<int>((static_cast<int64_t>(s.n) * heads + C::M - 1) / C::M);
}
// the first item of workgroup w of n, of `total`
__device__ __forceinline__ int64_t begin_of(int64_t total, int w, int n) { return total * w / n; }

// How many workgroups take part: not so many that joining their parts costs more
// than it saves.  (16 heads, one sequence of 331, 1000, 4096 and 32768: 24, 26, 30 and 37
// us with 4; 21, 24, 25 and 42 with 1; 22, 23, 31 and 42 with 2; 27, 31, 34 and 40 with 8.)
constexpr int kLeast = 4;              // items of a workgroup
__device__ __forceinline__ int used_workers(int64_t total, int workers) {
    const int64_t n = (total + kLeast - 1) / kLeast;
    return static_cast<int>(n < workers ? (n > 1 ? n : 1) : workers);
}

// The run of items that a workgroup takes: neighbouring runs, which are of the same
// sequences, on the same XCD (workgroups go to the XCDs in turn), so that row blocks of
// the same keys find them in its L2.
constexpr int kXcds = 8;
__device__ __forceinline__ int worker_of(int block, int n) { return n % kXcds ? block : block % kXcds * (n / kXcds) + block / kXcds; }

__device__ __forceinline__ float max_groups(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
// N floats (a multiple of 4)
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* v) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4v x = *reinterpret_cast<const float4v*>(p + i);
        v[i] = x.x;
        v[i + 1] = x.y;
        v[i + 2] = x.z;
        v[i + 3] = x.w;
    }
}

// In LDS a key's operands stand in runs of 64 bytes, four lanes' 16 bytes, whose order
// within run r is g ^ swizzle(r): so that the lanes that write a key, a run each, reach
// banks of their own.
__device__ __forceinline__ constexpr int swizzle(int r) { return (r >> 1) & 3; }

// 16 dimensions of four keys out of LDS: lane m of 16 gives the address of its four
// dimensions 4 (m % 4) of key m / 4, and gets dimension m of the four keys.
__device__ __forceinline__ uint2v transposed(const uint8_t* p) {
    typedef short4v __attribute__((address_space(3)))* Lds;
    return __builtin_bit_cast(uint2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
}

constexpr int kFew = 32;               // parts of a row that a lane group joins by itself

// The scratch.
template <class C>
struct Work {
    int64_t* first;      // [rows + 1]: items before those of a sequence
    int32_t* start;      // [workers + 1]: the sequence that a workgroup's items begin in; whether some rows have many parts
    float* factor;       // [query rows][4]: of a row's scores, and of its products with rotary keys before
    uint8_t* query;
    float* whole;        // [query rows][RS]: sums, the reference, and the sum of exponentials
    float* part;         // [workers][2][M][RS]
    __device__ __forceinline__ Work(const LatentAttnArgs& a) {
        const int64_t rows = static_cast<int64_t>(a.sq.tokens) * a.heads;
        first = reinterpret_cast<int64_t*>(a.work);
        uint8_t* p = a.work + latent_first_bytes(a.sq.rows);
        start = reinterpret_cast<int32_t*>(p);
        p += latent_start_bytes(a.workers);
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
        __shared__ int64_t sums[4], firsts[257];     // (of the first 256 sequences)
        __shared__ int longest;
        if (threadIdx.x == 0) {
            firsts[0] = work.first[0] = 0;
            longest = 0;
        }
        int64_t before = 0;
        for (int r0 = 0; r0 < a.sq.rows; r0 += 256) {
            const int r = r0 + threadIdx.x;
            int64_t v = 0;
            int per = 0;
            if (r < a.sq.rows) {
                const Seq s = seq_at<false>(a.sq, a.pg.logp, r);
                per = items_of(s);
                v = static_cast<int64_t>(per) * units_of<C>(s, a.heads);
                if (v == 0) per = 0;
            }
            for (int x = 1; x < 64; x *= 2) {
                const int64_t y = __shfl_up(v, x);
                if ((threadIdx.x & 63) >= x) v += y;
            }
            __syncthreads();
            if ((threadIdx.x & 63) == 63) sums[threadIdx.x / 64] = v;
            if (per > longest) atomicMax(&longest, per);
            __syncthreads();
            for (int x = 0; x < 4; ++x) {
                if (x < static_cast<int>(threadIdx.x / 64)) v += sums[x];
            }
            if (r < a.sq.rows) work.first[r + 1] = before + v;
            if (r0 == 0) firsts[threadIdx.x + 1] = v;
            before += sums[0] + sums[1] + sums[2] + sums[3];
        }
        __threadfence_block();
        __syncthreads();
        // the sequence that each workgroup begins in
        const int used = used_workers(before, a.workers);
        for (int w = threadIdx.x; w < used; w += 256) {
            const int64_t item = begin_of(before, w, used);
            int lo = 0, hi = a.sq.rows - 1;    // the last sequence that begins at or before the item
            while (lo < hi) {
                const int mid = lo + (hi - lo + 1) / 2;
                if ((mid <= 256 ? firsts[mid] : work.first[mid]) <= item) lo = mid;
                else hi = mid - 1;
            }
            work.start[w] = lo;
        }
        // whether a unit may have more than kFew parts: it touches that many runs of
        // total / used items
        if (threadIdx.x == 0) work.start[a.workers] = static_cast<int64_t>(longest) * used > static_cast<int64_t>(kFew - 2) * before;
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
    // products with rotary keys are put in the same unit, which has to leave them in range
    float rtop = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) rtop = fmaxf(rtop, fabsf(sizeof(In) == 2 ? bf2f(static_cast<uint32_t>(rp[i])) : static_cast<float>(rp[i])));
    rtop = over_lanes<LPV>(rtop, [](float p, float q) { return fmaxf(p, q); });
    const int most = min(100 - exponent(rtop), 110);
    int unit = 0;
    if (top > 0.0f && top < __builtin_inff()) unit = min(kQTop - 1 - exponent(top), most);   // (from -114)
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
    if (e == 0) {
        work.factor[4 * row] = __builtin_ldexpf(a.scale * kLog2e, -unit);
        work.factor[4 * row + 1] = __builtin_ldexpf(1.0f, unit);
    }
}

// ---------------------------------------------------------------------------
// the sums

// What a lane of a value wave holds of a key on its way: codes of CW / 4 runs of 32
// elements with their groups' scales and zero points, and a part of the rotary key.
template <class C>
struct Raw {
    uint4v codes[C::CW / 4], rope;
    uint32_t scale[C::CW / 4], zero[C::CW / 4];
};

template <class C>
struct Lds {
    __attribute__((aligned(16))) uint8_t keys[3][C::KEYS * C::VS];
    __attribute__((aligned(16))) uint8_t probs[2][C::T * C::NG * C::M * C::PS];
    __attribute__((aligned(16))) float scales[3][C::KEYS * C::NG];
    float top[C::WK * C::M], shift[C::M];
    int there[3][C::WK];       // whether a step's 16 keys have a page
    int moved[3];              // whether a reference moves after a step
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 2) latent_sums(const LatentAttnArgs a) {
    constexpr int D = C::D, NG = C::NG, RT = C::RT, T = C::T, M = C::M;
    __shared__ Lds<C> lds;
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool scoring = wave < C::SCORES;
    const int wk = wave % C::WK, wr = wave / C::WK;      // of a score wave
    const int vw = wave - C::SCORES;                     // of a value wave
    const Work<C> work(a);
    const LatentPage& pg = a.pg;
    const ConstLongs before = (ConstLongs)(work.first);
    const int64_t total = before[a.sq.rows];
    const int used = used_workers(total, gridDim.x);
    const int worker = worker_of(blockIdx.x, gridDim.x);
    if (worker >= used) return;
    const int64_t end = begin_of(total, worker + 1, used);
    int64_t item = begin_of(total, worker, used);
    int lo = ((ConstInts)(work.start))[worker];
    while (item < end) {
        while (before[lo + 1] <= item) ++lo;
        const Seq s = seq_at<true>(a.sq, pg.logp, lo);
        const int per = items_of(s);
        const int64_t in_seq = item - before[lo];
        const int rb = static_cast<int>(in_seq / per), i0 = static_cast<int>(in_seq % per);
        const int i1 = static_cast<int>(min(static_cast<int64_t>(per), i0 + end - item));
        item += i1 - i0;
        if (i1 <= kSetUp) continue;            // none of the unit's keys
        const int k0 = max(i0 - kSetUp, 0), k1 = i1 - kSetUp;
        const int len = s.len, rows = s.n * a.heads, r0 = rb * M, first = len - s.n;
        const int64_t row_at = static_cast<int64_t>(s.start) * a.heads;
        const int last_row = min(r0 + M, rows) - 1;
        const int limit = a.causal ? min(max(first + last_row / a.heads + 1, 0), len) : len;   // no row sees keys past it
        const int steps = (min(k1 * (kItem), limit) - k0 * kItem + C::KEYS - 1) / C::KEYS;     // (may be negative)
        const bool whole = k0 == 0 && i1 == per;
        float* out = whole ? work.whole + (row_at + r0) * C::RS
                           : work.part + (static_cast<int64_t>(worker) * 2 + (k0 > 0 ? 0 : 1)) * M * C::RS;
        const int key0 = k0 * kItem;
        __syncthreads();                       // (the last segment's readers are done)
        if (tid < 3) lds.moved[tid] = 0;

        if (scoring) {
            // the wave's rows as B operands
            uint4v query[RT][T][C::KS], rope[RT][C::TR][2];
            float factor[RT], rfactor[RT];
            int pos[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int r = min(r0 + (wr * RT + rt) * 16 + m, rows - 1);
                const uint8_t* q = work.query + (row_at + r) * C::QS;
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks) query[rt][t][ks] = *reinterpret_cast<const uint4v*>(q + 2 * (t * D + 32 * ks + 8 * g));
#pragma unroll
                for (int t = 0; t < C::TR; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) rope[rt][t][i] = *reinterpret_cast<const uint4v*>(q + 2 * (T * D + t * kRope + 32 * i + 8 * g));
                factor[rt] = work.factor[4 * (row_at + r)];
                rfactor[rt] = work.factor[4 * (row_at + r) + 1];
                pos[rt] = a.causal ? min(first + r / a.heads, len - 1) : len - 1;   // the last key that the row sees
            }
            // the first key that not all of the wave's rows see
            const int all = a.causal ? min(first + min(r0 + wr * 16 * RT, rows - 1) / a.heads + 1, len) : len;
            float ref[RT], sum[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                ref[rt] = kLow;
                sum[rt] = 0.0f;
            }
            __syncthreads();                   // (the first keys are there)
            int b3 = 0;
            for (int i = 0; i < steps; ++i) {
                const uint8_t* keys = lds.keys[b3] + (16 * wk + m) * C::VS;
                float scale[4][NG];
                load_floats<4 * NG>(lds.scales[b3] + (16 * wk + 4 * g) * NG, &scale[0][0]);
                // operands: two of the rotary key, then the codes'; kBatch of them are on
                // their way while as many are worked on
                float4v w[RT], c[RT];
                uint4v k[2][kBatch];
                const auto operand = [&](int x) HR_INLINE { return *reinterpret_cast<const uint4v*>(keys + (x < 2 ? 2 * D + 64 * x + 16 * g : 64 * (x - 2) + 16 * (g ^ swizzle(x - 2)))); };
                constexpr int ALL = C::KS + 2;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) w[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int x = 0; x < kBatch; ++x) k[0][x] = operand(x);
#pragma unroll
                for (int x0 = 0; x0 < ALL; x0 += kBatch) {
                    HR_PHASE();
#pragma unroll
                    for (int x = x0 + kBatch; x < x0 + 2 * kBatch && x < ALL; ++x) k[x / kBatch % 2][x % kBatch] = operand(x);
#pragma unroll
                    for (int x = x0; x < x0 + kBatch && x < ALL; ++x) {
                        const uint4v kx = k[x / kBatch % 2][x % kBatch];
                        if (x < 2) {
#pragma unroll
                            for (int t = C::TR - 1; t >= 0; --t)
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt) w[rt] = mfma_bf16(kx, rope[rt][t][x], w[rt]);
                            if (x == 1)
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                                    for (int y = 0; y < 4; ++y) w[rt][y] *= rfactor[rt];
                        } else {
                            const int ks = x - 2, q = ks / C::KG;
                            if (ks % C::KG == 0)
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt) c[rt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int t = T - 1; t >= 0; --t)
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt) c[rt] = mfma_f16(kx, query[rt][t][ks], c[rt]);
                            if (ks % C::KG == C::KG - 1)
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                                    for (int y = 0; y < 4; ++y) w[rt][y] = __builtin_fmaf(c[rt][y], scale[y][q], w[rt][y]);
                        }
                    }
                }
                HR_PHASE();
                const int t0 = key0 + i * C::KEYS + 16 * wk, key = t0 + 4 * g;
                const bool here = lds.there[b3][wk] != 0, full = here && t0 + 16 <= all;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[rt][x] *= factor[rt];
                if (!full) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const int bound = here ? pos[rt] : -1;
#pragma unroll
                        for (int x = 0; x < 4; ++x) w[rt][x] = key + x > bound ? -__builtin_inff() : w[rt][x];
                    }
                    // an unseen key's scale may be any bits (infinities are NaN here), and its
                    // probability is 0: what is multiplied by it is finite (a key that is seen
                    // has a NaN score then)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int q = 0; q < NG; ++q) scale[x][q] = fminf(scale[x][q], 0x1.fffffep127f);
                }
                // probabilities, to LDS: keys 16 wk + 4 g + x stand at 8 g + 4 wk + x
                uint8_t* to = lds.probs[i & 1] + (wr * 16 * RT + m) * C::PS + 16 * g + 8 * wk;
                float more[RT];
                const auto put = [&]() HR_INLINE {
                    float most = 0.0f, largest = 0.0f;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        float p[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) p[x] = __builtin_amdgcn_exp2f(w[rt][x] - ref[rt]);
                        more[rt] = (p[0] + p[1]) + (p[2] + p[3]);
                        largest = fmaxf(fmaxf(largest, more[rt]), 0.0f);
#pragma unroll
                        for (int q = 0; q < NG; ++q) {
                            float v[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) v[x] = p[x] * scale[x][q];
                            most = fmaxf(fmaxf(most, v[0]), v[1]);
                            most = fmaxf(fmaxf(most, v[2]), v[3]);
                            uint8_t* p16 = to + (q * M + 16 * rt) * C::PS;
                            if constexpr (C::WIDE) {
                                uint2v hi, lost;
                                uint32_t h, l;
                                split_f16(v[0], v[1], h, l);
                                hi.x = h;
                                lost.x = l;
                                split_f16(v[2], v[3], h, l);
                                hi.y = h;
                                lost.y = l;
                                *reinterpret_cast<uint2v*>(p16) = hi;
                                *reinterpret_cast<uint2v*>(p16 + NG * M * C::PS) = lost;
                            } else {
                                *reinterpret_cast<uint2v*>(p16) = uint2v{pack_f16(v[0], v[1]), pack_f16(v[2], v[3])};
                            }
                        }
                    }
                    return most > kTop || largest > kMostExp;
                };
                if (__any(put()) && lane == 0) lds.moved[b3] = 1;
                __syncthreads();
                if (lds.moved[b3]) {
                    // references follow the largest of what the rows see
                    float p[RT][4], base[RT];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        float x = fmaxf(fmaxf(w[rt][0], w[rt][1]), fmaxf(w[rt][2], w[rt][3]));
                        x = max_groups(x);
                        if (g == 0) lds.top[wk * M + (wr * RT + rt) * 16 + m] = x;
                    }
                    __syncthreads();
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const int r = (wr * RT + rt) * 16 + m;
                        base[rt] = ceilf(fmaxf(lds.top[r], lds.top[M + r]));   // (a whole number: factors are exact)
#pragma unroll
                        for (int x = 0; x < 4; ++x) p[rt][x] = __builtin_amdgcn_exp2f(w[rt][x] - base[rt]);
                    }
                    __syncthreads();
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        float y = 0.0f;
#pragma unroll
                        for (int q = 0; q < NG; ++q)
#pragma unroll
                            for (int x = 0; x < 4; ++x) y = fmaxf(y, p[rt][x] * scale[x][q]);
                        y = max_groups(y);
                        if (g == 0) lds.top[wk * M + (wr * RT + rt) * 16 + m] = y;
                    }
                    __syncthreads();
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const int r = (wr * RT + rt) * 16 + m;
                        const float y = fmaxf(lds.top[r], lds.top[M + r]), was = ref[rt];
                        if (base[rt] > kLow && base[rt] < __builtin_inff())
                            ref[rt] = fmaxf(was, base[rt] + static_cast<float>(max(exponent(y) - kSet, kLeastRef)));
                        const float f = __builtin_amdgcn_exp2f(was - ref[rt]);
                        sum[rt] *= f;
                        if (wk == 0 && g == 0) lds.shift[r] = f;
                    }
                    put();
                    __syncthreads();
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) sum[rt] += more[rt];
                b3 = b3 == 2 ? 0 : b3 + 1;
            }
            __syncthreads();                   // (the value waves' last step)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int r = (wr * RT + rt) * 16 + m;
                const float l = sum_groups(sum[rt]);
                if (g == 0) {
                    lds.top[wk * M + r] = l;
                    if (wk == 0 && r0 + r < rows) out[static_cast<int64_t>(r) * C::RS + D] = ref[rt];
                }
            }
            __syncthreads();
            if (tid < M && r0 + tid < rows) out[static_cast<int64_t>(tid) * C::RS + D + 1] = lds.top[tid] + lds.top[M + tid];
        } else {
            // keys of the wave: 8 vw + lane / LK, LK lanes to a key
            const int kk = (C::KEYS / C::VALUES) * vw + lane / C::LK, part = lane % C::LK;
            const ConstInts table = (ConstInts)(a.sq.table + static_cast<int64_t>(lo) * a.sq.max_pages);
            const int slots = a.sq.max_pages - 1;
            // the page of the 16 keys that the wave's are of in step i; absent past the
            // sequence's end
            const auto page_of = [&](int i) HR_INLINE {
                const int t = key0 + i * C::KEYS + (C::KEYS / C::VALUES) * vw / 16 * 16;
                return i < steps && t < len ? table[min(t >> pg.logp, slots)] : -1;
            };
            // a lane's offsets from its wave's first key
            const int ko = lane / C::LK, co = ko * (D / 2) + 16 * part, ro = ko * (2 * kRope) + 16 * part;
            const auto group_of = [&](int x) HR_INLINE { return (part + C::LK * x) * 32 / C::G; };
            const auto load = [&](int page, int i, Raw<C>& w) HR_INLINE {
                const int t = key0 + i * C::KEYS + (C::KEYS / C::VALUES) * vw, off = t & (pg.page - 1);
                // (an absent page has no bytes: its loads give zeros)
                const bool here = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.sq.n_pages);
                const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.pool + (here ? page : 0) * pg.page_bytes), 0,
                                                                                   here ? static_cast<int>(pg.page_bytes) : 0, 0x00020000);
#pragma unroll
                for (int x = 0; x < C::CW / 4; ++x) {
                    w.codes[x] = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(r, co + 16 * C::LK * x, off * (D / 2), 0));
                    const int at = ko * NG + group_of(x);
                    if constexpr (C::SF32) w.scale[x] = __builtin_amdgcn_raw_buffer_load_b32(r, 4 * at, pg.scales + off * NG * 4, 0);
                    else w.scale[x] = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, 2 * at, pg.scales + off * NG * 2, 0));
                    // (symmetric: some byte, not looked at)
                    w.zero[x] = static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(r, at / 2, pg.zeros + off * NG / 2, 0));
                }
                w.rope = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(r, ro, pg.rope + off * (2 * kRope), 0));
            };
            // operands of a step
            const uint32_t f0c = 0x64006400u ^ (pg.sym ? 0x00080008u : 0u), f1c = 0x54005400u ^ (pg.sym ? 0x00800080u : 0u);
            // operands of 8 of the lane's elements: word n of its codes
            const auto store_word = [&](const Raw<C>& w, int n, uint8_t* to) HR_INLINE {
                const int x = n / 4, y = n % 4, run = part + C::LK * x, at = ko * NG + group_of(x);
                const uint32_t z = pg.sym ? 8u : (w.zero[x] >> (4 * (at & 1))) & 15u;
                const uint32_t z0 = 0x64006400u + z * 0x00010001u, z1 = 0x54005400u + z * 0x00100010u;
                uint32_t c = w.codes[x][y];
                uint4v k;
                k.x = pk_sub((c & 0x000F000Fu) ^ f0c, z0);
                k.y = pk_sub((c & 0x00F000F0u) ^ f1c, z1);
                c >>= 8;
                k.z = pk_sub((c & 0x000F000Fu) ^ f0c, z0);
                k.w = pk_sub((c & 0x00F000F0u) ^ f1c, z1);
                *reinterpret_cast<uint4v*>(to + 64 * run + 16 * (y ^ swizzle(part))) = k;
            };
            // and what belongs to them
            const auto store_rest = [&](const Raw<C>& w, int page, int b, uint8_t* to) HR_INLINE {
                if (lane == 0) lds.there[b][vw / 2] = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.sq.n_pages);   // (waves of the same 16 keys say the same)
#pragma unroll
                for (int x = 0; x < C::CW / 4; ++x)
                    if ((part + C::LK * x) * 32 % C::G == 0) {
                        // (the scale of an infinite latent is infinite, and its codes say nothing: NaN)
                        const float s = __uint_as_float(C::SF32 ? w.scale[x] : w.scale[x] << 16);
                        lds.scales[b][kk * NG + group_of(x)] = fabsf(s) == __builtin_inff() ? __builtin_nanf("") : s;
                    }
                *reinterpret_cast<uint4v*>(to + 2 * D + 16 * part) = w.rope;
            };
            float4v acc[C::TILES][C::DT];
#pragma unroll
            for (int x = 0; x < C::TILES; ++x)
#pragma unroll
                for (int d = 0; d < C::DT; ++d) acc[x][d] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
            const uint32_t grp = vw * C::DW / C::G;
            // Sums of the wave's dimensions over all rows, of the step in buffers b and p;
            // between its matrix steps, word by word, the operands of the codes in w go to
            // buffer `into`: one keeps the matrix unit, the other vector unit and LDS busy.
            const auto add = [&](int b, int p, bool moved, const Raw<C>& w, int into) HR_INLINE {
                if (moved) {
#pragma unroll
                    for (int x = 0; x < C::TILES; ++x) {
                        const float f = lds.shift[16 * x + m];
#pragma unroll
                        for (int d = 0; d < C::DT; ++d)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[x][d][i] *= f;
                    }
                }
                const uint8_t* pr = lds.probs[p] + (grp * M + m) * C::PS + 16 * g;
                const uint8_t* va = lds.keys[b] + (4 * g + m / 4) * C::VS + vw * C::DW * 2 + m % 2 * 8;
                uint8_t* to = lds.keys[into] + kk * C::VS;
                uint4v pb[T][C::TILES], v[2];
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int x = 0; x < C::TILES; ++x) pb[t][x] = *reinterpret_cast<const uint4v*>(pr + (t * NG * M + 16 * x) * C::PS);
                const auto operand = [&](int d) HR_INLINE {
                    // (dimensions 16 d + 4 (m % 4) of the wave's: half a 16-byte part of run d / 2)
                    const int at = d / 2 * 64 + 16 * ((d % 2 * 2 + m % 4 / 2) ^ swizzle(vw * (C::DW / 32) + d / 2));
                    const uint2v v0 = transposed(va + at), v1 = transposed(va + 16 * C::VS + at);
                    return uint4v{v0.x, v0.y, v1.x, v1.y};
                };
                v[0] = operand(0);
#pragma unroll
                for (int d = 0; d < C::DT; ++d) {
                    if (d + 1 < C::DT) v[(d + 1) & 1] = operand(d + 1);
                    HR_PHASE();
#pragma unroll
                    for (int t = T - 1; t >= 0; --t)
#pragma unroll
                        for (int x = 0; x < C::TILES; ++x) acc[x][d] = mfma_f16(v[d & 1], pb[t][x], acc[x][d]);
                    store_word(w, d, to);
                    HR_PHASE();
                }
            };
            static_assert(C::CW == C::DT, "a word for each tile of dimensions");
            // A step's codes have a place in raw that depends on its number alone, and the
            // loop is unrolled: a load on its way cannot be moved to another register.
            Raw<C> raw[kAhead];
            int page[kAhead], next[kAhead];    // of the step in a place, and of the one after it
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                page[x] = page_of(x);
                next[x] = page_of(x + kAhead);
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) load(page[x], x, raw[x]);
            // the loads of the step that takes place X after one that has been stored
            const auto reload = [&](auto X, int i) HR_INLINE {
                page[X] = next[X];
                load(page[X], i, raw[X]);
                next[X] = page_of(i + kAhead);
            };
            const auto store = [&](auto X, int i) HR_INLINE {
                uint8_t* to = lds.keys[X] + kk * C::VS;
                store_rest(raw[X], page[X], X, to);
#pragma unroll
                for (int n = 0; n < C::CW; ++n) store_word(raw[X], n, to);
                reload(X, i + kAhead);
            };
            typedef std::integral_constant<int, 0> P0;
            typedef std::integral_constant<int, 1> P1;
            typedef std::integral_constant<int, 2> P2;
            store(P0(), 0);
            __syncthreads();
            store(P1(), 1);
            bool moved = false;
            // the end of the interval in which scores are formed in buffer b
            const auto meet = [&](int b) HR_INLINE {
                __syncthreads();
                moved = lds.moved[b] != 0;
                if (moved) {
                    __syncthreads();
                    __syncthreads();
                    __syncthreads();
                    __syncthreads();
                }
            };
            if (steps > 0) meet(0);
            // an interval: the scores of step i are formed, in buffer B, the step before is
            // added and the one after stored
            const auto interval = [&](auto B, int i) HR_INLINE {
                constexpr int next_b = (B + 1) % 3;
                if (vw == 0 && lane == 0) lds.moved[next_b] = 0;
                store_rest(raw[next_b], page[next_b], next_b, lds.keys[next_b] + kk * C::VS);
                add((B + 2) % 3, (i + 1) & 1, moved, raw[next_b], next_b);
                reload(std::integral_constant<int, next_b>(), i + 1 + kAhead);
                if (i < steps) meet(B);
            };
            for (int i = 1; i <= steps; i += 3) {
                interval(P1(), i);
                if (i + 1 <= steps) interval(P2(), i + 1);
                if (i + 2 <= steps) interval(P0(), i + 2);
            }
            __syncthreads();
            // the segment's sums
#pragma unroll
            for (int x = 0; x < C::TILES; ++x) {
                const int r = 16 * x + m;
                if (r0 + r < rows)
#pragma unroll
                    for (int d = 0; d < C::DT; ++d)
                        *reinterpret_cast<float4v*>(out + static_cast<int64_t>(r) * C::RS + vw * C::DW + 16 * d + 4 * g) = acc[x][d];
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// the results

// What a group of D / 16 lanes adds up of a row's sums, 16 elements to a lane.
struct Joined {
    float v[16] = {}, ref = kLow, l = 0.0f;
    __device__ __forceinline__ void add(const float (&x)[16], float xr, float xl) {
        // (a part that saw nothing has the reference kLow, and sums of 0)
        const float now = fmaxf(ref, xr), f0 = __builtin_amdgcn_exp2f(ref - now), f1 = __builtin_amdgcn_exp2f(xr - now);
        l = l * f0 + xl * f1;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] * f0 + x[i] * f1;
        ref = now;
    }
};

// Where a row's sums are: `whole`, or in `parts` parts from workgroup w0 on.
struct Where {
    int parts, w0;
    int64_t u0;                // the first item of the unit's keys
    int in_unit, left;         // the row's place in its unit, and the unit's rows
};
template <class C, bool UNI>
__device__ __forceinline__ Where where_of(const LatentAttnArgs& a, const Work<C>& work, int64_t total, int used, int64_t row) {
    const int t = static_cast<int>(static_cast<uint32_t>(row) / a.heads);
    int lo = 0, hi = a.sq.rows - 1;                // the last sequence that begins at or before this token
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (cu_at<UNI>(a.sq, mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    const Seq s = seq_at<UNI>(a.sq, a.pg.logp, lo);
    Where w{0, 0, 0, 0, 0};
    const int per = items_of(s);
    if (t < s.start || t >= s.start + s.n || per == 0) return w;   // (no workgroup had this row)
    const int64_t r = row - static_cast<int64_t>(s.start) * a.heads;
    w.in_unit = static_cast<int>(r % C::M);
    w.left = static_cast<int>(min(static_cast<int64_t>(C::M), static_cast<int64_t>(s.n) * a.heads - (r - w.in_unit)));
    w.u0 = (UNI ? ((ConstLongs)(work.first))[lo] : work.first[lo]) + r / C::M * per + kSetUp;
    const int64_t last = w.u0 + per - kSetUp - 1;
    w.w0 = static_cast<int>(((w.u0 + 1) * used - 1) / total);
    w.parts = static_cast<int>(((last + 1) * used - 1) / total) - w.w0 + 1;
    return w;
}

template <class C, class Out>
__device__ __forceinline__ void finish_row(const LatentAttnArgs& a, int64_t row, const Joined& j) {
    constexpr int LPV = C::D / 16;
    const int e = threadIdx.x % LPV, lane = threadIdx.x & 63;
    const int t = static_cast<int>(static_cast<uint32_t>(row) / a.heads), h = static_cast<int>(static_cast<uint32_t>(row) % a.heads);
    const float inverse = 1.0f / j.l;
    // back to the elements' own order
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i / 8 * 8 + (i % 2) * 4 + (i % 8) / 2] = j.l == 0.0f ? 0.0f : j.v[i] * inverse;
    if (a.rotate) hadamard<C::D>(y, lane, a.norm);
    Out* out = static_cast<Out*>(a.out) + t * a.o_st + h * a.o_sh + 16 * e;
#pragma unroll
    for (int i = 0; i < 16; i += 16 / sizeof(Out)) {
        uint4v x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(Out) == 2) x[k] = to_bf16(y[i + 2 * k]) | (to_bf16(y[i + 2 * k + 1]) << 16);
            else x[k] = __float_as_uint(y[i + k]);
        }
        *reinterpret_cast<uint4v*>(out + i) = x;
    }
    if (a.lse && e == 0) a.lse[row] = j.l == 0.0f ? -__builtin_inff() : (j.ref + __builtin_amdgcn_logf(j.l)) * 0.6931471805599453f;
}

// Rows of few parts are joined by a group of D / 16 lanes each, the first workgroups'; a
// row of many by a workgroup of its own, whose groups take its parts in turn and whose
// first group adds what they have.  Either way a row's sums are added in one order, that
// of its keys, or that of the groups and of its keys in them.
template <class C, class Out>
__global__ void __launch_bounds__(256) latent_finish(const LatentAttnArgs a) {
    constexpr int D = C::D, LPV = D / 16, GROUPS = 256 / LPV;
    __shared__ __attribute__((aligned(16))) float sums[GROUPS][D];
    __shared__ float refs[GROUPS], exps[GROUPS];
    const Work<C> work(a);
    const int group = threadIdx.x / LPV, e = threadIdx.x % LPV;
    const int64_t total = ((ConstLongs)(work.first))[a.sq.rows];
    const int used = used_workers(total, a.workers);
    const int64_t rows = static_cast<int64_t>(a.sq.tokens) * a.heads;
    const auto part = [&](const Where& w, int i) {
        const int p = w.w0 + i, slot = begin_of(total, p, used) > w.u0 ? 0 : 1;
        return work.part + ((static_cast<int64_t>(p) * 2 + slot) * C::M + w.in_unit) * C::RS;
    };
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * GROUPS; row0 < rows; row0 += static_cast<int64_t>(gridDim.x) * GROUPS) {
        const int64_t row = row0 + group;
        // (most often the rows are of one unit, neighbours there)
        Where w = where_of<C, true>(a, work, total, used, row0);
        if (w.in_unit + group < w.left) w.in_unit += group;
        else w = where_of<C, false>(a, work, total, used, min(row, rows - 1));
        if (row >= rows || w.parts > kFew) continue;
        Joined j;
        for (int i0 = 0; i0 < w.parts; i0 += 4) {
            float x[4][16], xr[4], xl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = min(i0 + i, w.parts - 1);
                const float* p = w.parts == 1 ? work.whole + row * C::RS : part(w, n);
#pragma unroll
                for (int k = 0; k < 16; k += 4) load_floats<4>(p + 16 * e + k, x[i] + k);
                xr[i] = p[D];
                xl[i] = p[D + 1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i0 + i < w.parts) j.add(x[i], xr[i], xl[i]);
        }
        finish_row<C, Out>(a, row, j);
    }
    if (!((ConstInts)(work.start))[a.workers]) return;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const Where w = where_of<C, true>(a, work, total, used, row);
        if (w.parts <= kFew) continue;             // (the same for the whole workgroup)
        Joined j;
        for (int i = group; i < w.parts; i += GROUPS) {
            const float* p = part(w, i);
            float x[16];
#pragma unroll
            for (int k = 0; k < 16; k += 4) load_floats<4>(p + 16 * e + k, x + k);
            j.add(x, p[D], p[D + 1]);
        }
        __syncthreads();
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4v*>(&sums[group][16 * e + i]) = float4v{j.v[i], j.v[i + 1], j.v[i + 2], j.v[i + 3]};
            if (e == 0) {
                refs[group] = j.ref;
                exps[group] = j.l;
            }
        }
        __syncthreads();
        if (group > 0) continue;
        for (int x = 1; x < GROUPS; ++x) {
            float v[16];
            load_floats<16>(&sums[x][16 * e], v);
            j.add(v, refs[x], exps[x]);
        }
        finish_row<C, Out>(a, row, j);
    }
}

// workgroups that join: for rows of few parts, and enough for rows of many
inline int64_t finish_grid(int64_t rows, int groups) {
    const int64_t few = (rows + groups - 1) / groups, many = rows < 1024 ? rows : 1024;
    return few > (1 << 20) ? 1 << 20 : few > many ? few : many;
}

template <class C>
int attn_launch(const LatentAttnArgs& a, hipStream_t s) {
    const int64_t rows = int64_t{a.sq.tokens} * a.heads, threads = rows * (C::D / 16);
    const dim3 query(static_cast<uint32_t>((threads + 255) / 256)), finish(static_cast<uint32_t>(finish_grid(rows, 256 / (C::D / 16))));
    if constexpr (C::WIDE) hipLaunchKernelGGL((latent_query<C, float>), query, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((latent_query<C, uint16_t>), query, dim3(256), 0, s, a);
    hipLaunchKernelGGL((latent_sums<C>), dim3(a.workers), dim3(C::THREADS), 0, s, a);
    if constexpr (C::WIDE) hipLaunchKernelGGL((latent_finish<C, float>), finish, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((latent_finish<C, uint16_t>), finish, dim3(256), 0, s, a);
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
        n = cus;
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

template <int D, int NG, bool SF32>
int pick_rows(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream) {
    if (k.wide) return k.wr == 1 ? attn_do<Cfg<D, NG, SF32, true, 1, 1>>(a, workers, stream) : attn_do<Cfg<D, NG, SF32, true, 1, 2>>(a, workers, stream);
    if (k.rt == 1) return k.wr == 1 ? attn_do<Cfg<D, NG, SF32, false, 1, 1>>(a, workers, stream) : attn_do<Cfg<D, NG, SF32, false, 1, 2>>(a, workers, stream);
    return attn_do<Cfg<D, NG, SF32, false, 2, 2>>(a, workers, stream);
}

template <int D, int NG>
int pick_scales(const LatentAttnKey& k, const LatentAttnArgs* a, int* workers, void* stream) {
    return k.sf32 ? pick_rows<D, NG, true>(k, a, workers, stream) : pick_rows<D, NG, false>(k, a, workers, stream);
}

}  // namespace
}  // namespace hr
