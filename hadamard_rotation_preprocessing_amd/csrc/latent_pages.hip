// Writing latents into the paged 4-bit cache and taking them out of it
// (hr_latent_append, hr_latent_read).
//
// Both are one pass over the data: D / 16 lanes share a latent, 16 consecutive
// elements each, as in cache_vectors.h, and the same lanes take the rotary key.
// The floor is the bytes; what comes next is the instruction stream of the
// transform and the codes, which by counters takes the vector units nearly all of their
// cycles.  Measured: 32768 latents of 512 appended in 16.8 us (50 MB, 3.0 TB/s), single
// tokens of 64 sequences in 9 us a call, 4.9 us of it in the kernel; 24 sequences of up to
// 32768 read in 55 us (192 MB, 3.5 TB/s), 76 us a call where inputs and outputs change from
// call to call.  Over two sets of inputs in turn the append takes 18.6 us, and 12.6 without
// the rotation; the read 52 us into the same buffers, and 41 without it (4.7 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache_index.h"
#include "cache_vectors.h"
#include "latent.h"

namespace hr {
namespace {

// bf16 (finite or not) from float32, nearest even, NaN kept
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// ---------------------------------------------------------------------------
// append
//
// A wave takes 1024 / D consecutive positions of a sequence, aligned to that
// number, so that it owns every byte of zero points it writes.

template <int D, int G, bool SYM, class T>
__global__ void __launch_bounds__(256) latent_append(const LatentPagesArgs a) {
    constexpr int LPV = D / 16, POS = 64 / LPV, LANES = G / 16, NG = D / G, R = kRope / LPV;
    const int lane = threadIdx.x & 63;
    const int u = static_cast<int>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (u >= a.units) return;
    const AppendBlock blk = append_block<POS>(a.sq, a.pg.logp, u);
    if (!blk.any) return;
    const int page = a.sq.table[static_cast<int64_t>(blk.b) * a.sq.max_pages + (blk.p0 >> a.pg.logp)];
    if (static_cast<uint32_t>(page) >= static_cast<uint64_t>(a.sq.n_pages)) return;
    uint8_t* base = a.pool + page * a.pg.page_bytes;
    const int pos = blk.p0 + lane / LPV, off = pos & (a.pg.page - 1), e = lane % LPV;
    const bool mine = blk.holds(pos);
    const int64_t tok = blk.token(pos);
    float v[16];
    load16(static_cast<const T*>(a.c_in) + tok * a.c_st + 16 * e, v);
    const T* rp = static_cast<const T*>(a.rope_in) + tok * a.r_st + R * e;
    uint32_t rope[R / 2];
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
        if constexpr (sizeof(T) == 2) rope[i] = reinterpret_cast<const uint32_t*>(rp)[i];
        else rope[i] = to_bf16(rp[2 * i]) | (to_bf16(rp[2 * i + 1]) << 16);
    }
    if (a.rotate) hadamard<D>(v, lane, a.norm);
    uint32_t scale, zero = 0;
    const uint2v w = quantize<LANES, SYM>(v, a.pg.sf32, &scale, &zero);
    const int at = off * NG + e / LANES;
    if (mine) {
        *reinterpret_cast<uint2v*>(base + off * (D / 2) + 8 * e) = w;
#pragma unroll
        for (int i = 0; i < R / 2; ++i) reinterpret_cast<uint32_t*>(base + a.pg.rope + off * (2 * kRope))[e * (R / 2) + i] = rope[i];
        if (e % LANES == 0) {
            if (a.pg.sf32) reinterpret_cast<uint32_t*>(base + a.pg.scales)[at] = scale;
            else reinterpret_cast<uint16_t*>(base + a.pg.scales)[at] = static_cast<uint16_t>(scale);
        }
    }
    if constexpr (!SYM) {
        // two zero points to a byte: the other one belongs to the next group, or
        // with one group to the next position, G / 16 lanes on
        const uint32_t other = __shfl_xor(zero, LANES);
        const bool others = __shfl_xor(static_cast<int>(mine), LANES) != 0;
        uint8_t* zp = base + a.pg.zeros + at / 2;
        if (e % LANES == 0) {
            if (mine && others) {
                if (!(at & 1)) *zp = static_cast<uint8_t>(zero | (other << 4));
            } else if (mine) {
                const uint32_t old = *zp;
                *zp = static_cast<uint8_t>((at & 1) ? (old & 15u) | (zero << 4) : (old & 0xF0u) | zero);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// read
//
// A wave takes 1024 / D output rows.

template <int D, int NG, class T>
__global__ void __launch_bounds__(256) latent_read(const LatentPagesArgs a) {
    constexpr int LPV = D / 16, LANES = LPV / NG, R = kRope / LPV;
    const int64_t p = (int64_t{blockIdx.x} * 256 + threadIdx.x) / LPV;
    const int lane = threadIdx.x & 63, e = lane % LPV;
    const int at = static_cast<int>(min(p, static_cast<int64_t>(a.sq.tokens) - 1));
    const auto cu = [&](int b) { return index_min(index_max(a.sq.cu ? a.sq.cu[b] : b * a.sq.per, 0), a.sq.tokens); };
    int lo = 0, hi = a.sq.rows - 1;       // the last row that begins at or before this place
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (cu(mid) <= at) lo = mid;
        else hi = mid - 1;
    }
    const int pos = max(at - cu(lo), 0);
    const int64_t cap = static_cast<int64_t>(a.sq.max_pages) << a.pg.logp;
    int page = -1;
    if (pos < min(static_cast<int64_t>(max(a.sq.lens[lo], 0)), cap))
        page = a.sq.table[static_cast<int64_t>(lo) * a.sq.max_pages + (pos >> a.pg.logp)];
    const bool here = static_cast<uint32_t>(page) < static_cast<uint64_t>(a.sq.n_pages);
    float v[16] = {};
    uint32_t rope[R / 2] = {};
    if (here) {
        const uint8_t* base = a.pool + page * a.pg.page_bytes;
        const int off = pos & (a.pg.page - 1), g = off * NG + e / LANES;
        const uint2v w = *reinterpret_cast<const uint2v*>(base + off * (D / 2) + 8 * e);
        const float s = a.pg.sf32 ? reinterpret_cast<const float*>(base + a.pg.scales)[g]
                                  : bf2f(reinterpret_cast<const uint16_t*>(base + a.pg.scales)[g]);
        const int z = a.pg.sym ? 8 : (base[a.pg.zeros + g / 2] >> (4 * (g & 1))) & 15;
        const uint32_t flip = a.pg.sym ? 0x88888888u : 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = static_cast<float>(static_cast<int>(((w[i / 8] ^ flip) >> (4 * (i % 8))) & 15u) - z) * s;
#pragma unroll
        for (int i = 0; i < R / 2; ++i) rope[i] = reinterpret_cast<const uint32_t*>(base + a.pg.rope + off * (2 * kRope))[e * (R / 2) + i];
    }
    if (a.rotate) hadamard<D>(v, lane, a.norm);
    if (p >= a.sq.tokens) return;
    T* c = static_cast<T*>(a.c_out) + p * a.c_st + 16 * e;
    T* r = static_cast<T*>(a.rope_out) + p * a.r_st + R * e;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint4v x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = to_bf16(v[8 * i + 2 * j]) | (to_bf16(v[8 * i + 2 * j + 1]) << 16);
            reinterpret_cast<uint4v*>(c)[i] = x;
        }
#pragma unroll
        for (int i = 0; i < R / 2; ++i) reinterpret_cast<uint32_t*>(r)[i] = rope[i];
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            uint4v x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = __float_as_uint(v[i + j]);
            reinterpret_cast<uint4v*>(c)[i / 4] = x;
        }
#pragma unroll
        for (int i = 0; i < R / 2; ++i) {
            r[2 * i] = bf2f(rope[i] & 0xFFFFu);
            r[2 * i + 1] = bf2f(rope[i] >> 16);
        }
    }
}

template <int D, int G, class T>
void append_launch(const LatentPagesArgs& a, hipStream_t s) {
    const dim3 grid((static_cast<uint32_t>(a.units) + 3) / 4);
    if (a.pg.sym) hipLaunchKernelGGL((latent_append<D, G, true, T>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((latent_append<D, G, false, T>), grid, dim3(256), 0, s, a);
}
template <int D, int NG, class T>
void read_launch(const LatentPagesArgs& a, hipStream_t s) {
    const int64_t threads = int64_t{a.sq.tokens} * (D / 16);
    hipLaunchKernelGGL((latent_read<D, NG, T>), dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0, s, a);
}

// f.template operator()<D, NG>() for the page's shape
template <class F>
int by_shape(const LatentPage& pg, F f) {
    if (pg.d == 512 && pg.ng == 4) f.template operator()<512, 4>();
    else if (pg.d == 512 && pg.ng == 2) f.template operator()<512, 2>();
    else if (pg.d == 512 && pg.ng == 1) f.template operator()<512, 1>();
    else if (pg.d == 256 && pg.ng == 2) f.template operator()<256, 2>();
    else if (pg.d == 256 && pg.ng == 1) f.template operator()<256, 1>();
    else return static_cast<int>(hipErrorInvalidValue);
    return static_cast<int>(hipGetLastError());
}

struct Append {
    const LatentPagesArgs& a;
    int bf16;
    hipStream_t s;
    template <int D, int NG>
    void operator()() const {
        if (bf16) append_launch<D, D / NG, uint16_t>(a, s);
        else append_launch<D, D / NG, float>(a, s);
    }
};
struct Read {
    const LatentPagesArgs& a;
    int bf16;
    hipStream_t s;
    template <int D, int NG>
    void operator()() const {
        if (bf16) read_launch<D, NG, uint16_t>(a, s);
        else read_launch<D, NG, float>(a, s);
    }
};

}  // namespace

int launch_latent_append(const LatentPagesArgs& a, int bf16, void* stream) {
    return by_shape(a.pg, Append{a, bf16, static_cast<hipStream_t>(stream)});
}
int launch_latent_read(const LatentPagesArgs& a, int bf16, void* stream) {
    return by_shape(a.pg, Read{a, bf16, static_cast<hipStream_t>(stream)});
}

}  // namespace hr
