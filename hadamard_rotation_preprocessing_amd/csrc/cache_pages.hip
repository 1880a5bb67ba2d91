// Writing the paged 4-bit cache (hr_cache_append) and moving its pages
// (hr_cache_update, hr_cache_compact).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache.h"
#include "cache_index.h"
#include "codes.h"

namespace hr {
namespace {

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// append
//
// A wave takes the K and V vectors of one kv head at 1024 / D consecutive
// positions of a sequence, aligned to that number, so that it owns every byte
// of zero points it writes.  D / 16 lanes share a vector, 16 consecutive
// elements each: four bits of the Hadamard transform are inside the lane, the
// other two to four are lane bits, and a group of 32 to 256 elements is 2 to
// 16 consecutive lanes.  The stages go in the order of the index bits.
//
// Every element is read once and every code written once, so the floor is the
// copy of those bytes; what comes next is the instruction stream, 700 vector
// instructions for a lane's 32 elements.  32768 tokens x 32 heads of 128 (683 MB):
// 155 us, 4.4 TB/s where a large copy has 4.95; with selections in the lane
// stages and codes packed one by one (820 instructions) it was 175.  One token of
// each of 64 sequences: 6 us, the launch and the chain of loads to the page.

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// the value of lane ^ X (X = 1, 2, 4, 8, inside 16 lanes)
template <int X>
__device__ __forceinline__ float lane_xor(float v) {
    if constexpr (X == 1) return dpp<0xB1>(v);         // quad_perm [1,0,3,2]
    if constexpr (X == 2) return dpp<0x4E>(v);         // quad_perm [2,3,0,1]
    if constexpr (X == 4) return dpp<0x141>(dpp<0x1B>(v));  // quad_perm [3,2,1,0], then the row's half mirrored: ^ 3 ^ 7
    return dpp<0x128>(v);                               // row_ror 8
}

template <int LANES, class F>
__device__ __forceinline__ float over_lanes(float v, F f) {
    if constexpr (LANES >= 2) v = f(v, lane_xor<1>(v));
    if constexpr (LANES >= 4) v = f(v, lane_xor<2>(v));
    if constexpr (LANES >= 8) v = f(v, lane_xor<4>(v));
    if constexpr (LANES >= 16) v = f(v, lane_xor<8>(v));
    return v;
}

// (a product with 1 or -1 is exact, and costs less than a selection; the move
// between lanes is part of the addition)
template <int X>
__device__ __forceinline__ void lane_stage(float (&v)[16], int lane) {
#pragma clang fp contract(off)
    const float sign = (lane & X) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = lane_xor<X>(v[i]) + v[i] * sign;
}

template <int D>
__device__ __forceinline__ void hadamard(float (&v)[16], int lane, float norm) {
#pragma unroll
    for (int s = 1; s < 16; s *= 2)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (!(i & s)) {
                const float x = v[i], y = v[i + s];
                v[i] = x + y;
                v[i + s] = x - y;
            }
    lane_stage<1>(v, lane);
    lane_stage<2>(v, lane);
    if constexpr (D >= 128) lane_stage<4>(v, lane);
    if constexpr (D >= 256) lane_stage<8>(v, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= norm;
}

template <class T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4v x = reinterpret_cast<const uint4v*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(x[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4v x = reinterpret_cast<const uint4v*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(x[j]);
        }
    }
}

// The codes of 16 elements y: quotient(y) is y / s, rounded to an integer.
// Codes are packed as float32, four of them to an integer below 2^16; symmetric
// ones with 8 added, which an XOR takes back.
template <bool SYM, class Q>
__device__ __forceinline__ uint2v pack_codes(const float (&v)[16], float z, Q quotient) {
#pragma clang fp contract(off)
    uint2v w;
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
        uint32_t half[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const float q = quotient(v[i + 4 * j + k]);
                const float c = __builtin_amdgcn_fmed3f(q + z, 0.0f, 15.0f);   // (NaN: 0)
                sum = k == 3 ? c : __builtin_fmaf(sum, 16.0f, c);
            }
            half[j] = static_cast<uint32_t>(sum);
        }
        w[i / 8] = (half[1] << 16 | half[0]) ^ (SYM ? 0x88888888u : 0u);
    }
    return w;
}

// Quantizes the lane's 16 elements: scale s = range / steps of the group,
// stored (f32 or nearest-even bf16), codes from the stored scale.  A group with
// a NaN has a NaN scale, so that whoever reads it sees one.  y / s is the
// correctly rounded quotient: one division gives r = 1 / s, and with t = y r the
// remainder fma(-t, s, y) is exact, so fma(remainder, r, t) rounds to y / s (P.
// Markstein, IBM J. Res. Dev. 34, 1990).  That keeps every code equal to the
// definition's, ties included, at two more instructions than a product with the
// reciprocal.  Where r or the remainder could leave the normal numbers, and for
// scales that are not finite, each element is divided.
template <int LANES, bool SYM>
__device__ __forceinline__ uint2v quantize(const float (&v)[16], bool sf32, uint32_t* scale, uint32_t* zero) {
#pragma clang fp contract(off)
    float s, z = 0.0f;
    bool nan;
    if constexpr (SYM) {
        float top = fabsf(v[0]);
#pragma unroll
        for (int i = 1; i < 16; ++i) top = __builtin_elementwise_maximum(top, fabsf(v[i]));   // (keeps a NaN)
        nan = top != top;
        top = over_lanes<LANES>(top, [](float a, float b) { return fmaxf(a, b); });
        s = top / 7.0f;
    } else {
        float lo = fminf(v[0], 0.0f), hi = __builtin_elementwise_maximum(v[0], 0.0f);
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            lo = fminf(lo, v[i]);
            hi = __builtin_elementwise_maximum(hi, v[i]);
        }
        nan = hi != hi;
        lo = over_lanes<LANES>(lo, [](float a, float b) { return fminf(a, b); });
        hi = over_lanes<LANES>(hi, [](float a, float b) { return fmaxf(a, b); });
        s = (hi - lo) / 15.0f;
        z = lo;
    }
    if (s == 0.0f) s = 1.0f;
    const bool odd = __any(nan || !(s >= 0x1p-64f && s <= 0x1p64f));
    if (odd && over_lanes<LANES>(nan ? 1.0f : 0.0f, [](float a, float b) { return fmaxf(a, b); }) != 0.0f)
        s = __uint_as_float(0x7FC00000u);
    if (sf32) {
        *scale = __float_as_uint(s);
    } else {
        *scale = f2bf(s);
        s = bf2f(*scale);
    }
    if constexpr (SYM) {
        z = 8.0f;
    } else {
        z = fminf(fmaxf(rintf(-z / s), 0.0f), 15.0f);
        *zero = static_cast<uint32_t>(static_cast<int>(z));
    }
    if (odd) return pack_codes<SYM>(v, z, [s](float y) { return rintf(y / s); });
    const float r = 1.0f / s;
    return pack_codes<SYM>(v, z, [s, r](float y) {
        const float t = y * r;
        return rintf(__builtin_fmaf(__builtin_fmaf(-t, s, y), r, t));
    });
}

template <int D, int G, bool SYM, class T>
__global__ void __launch_bounds__(256) cache_append(const CacheAppendArgs a) {
    constexpr int LPV = D / 16, POS = 64 / LPV, LANES = G / 16, NG = D / G;
    const int lane = threadIdx.x & 63;
    // four heads of a block of positions to a workgroup
    const int groups = (a.pg.hkv + 3) / 4;
    const int h = static_cast<int>(blockIdx.x % groups) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = blockIdx.x / groups;
    if (h >= a.pg.hkv) return;
    const AppendBlock blk = append_block<POS>(a.sq, a.pg.logp, u);
    if (!blk.any) return;
    const int page = a.sq.table[static_cast<int64_t>(blk.b) * a.sq.max_pages + (blk.p0 >> a.pg.logp)];
    if (static_cast<uint32_t>(page) >= static_cast<uint64_t>(a.sq.n_pages)) return;
    uint8_t* base = a.pool + page * a.pg.page_bytes + h * a.pg.head_bytes;
    const int pos = blk.p0 + lane / LPV, off = pos & (a.pg.page - 1), e = lane % LPV;
    const bool mine = blk.holds(pos);
    const int64_t tok = blk.token(pos);
    float k[16], v[16];
    load16(static_cast<const T*>(a.k) + tok * a.k_st + h * a.k_sh + 16 * e, k);
    load16(static_cast<const T*>(a.v) + tok * a.v_st + h * a.v_sh + 16 * e, v);
    if (a.rotate) hadamard<D>(k, lane, a.norm);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        uint32_t scale, zero = 0;
        const uint2v w = quantize<LANES, SYM>(x ? v : k, a.pg.sf32, &scale, &zero);
        const int g = e / LANES, at = off * NG + g;
        if (mine) {
            *reinterpret_cast<uint2v*>(base + (x ? a.pg.vc : a.pg.kc) + off * (D / 2) + 8 * e) = w;
            if (e % LANES == 0) {
                uint8_t* sp = base + (x ? a.pg.vs : a.pg.ks);
                if (a.pg.sf32) reinterpret_cast<uint32_t*>(sp)[at] = scale;
                else reinterpret_cast<uint16_t*>(sp)[at] = static_cast<uint16_t>(scale);
            }
        }
        if constexpr (!SYM) {
            // two zero points to a byte: the other one belongs to the next
            // group, or with one group to the next position, G / 16 lanes on
            const uint32_t other = __shfl_xor(zero, LANES);
            const bool others = __shfl_xor(static_cast<int>(mine), LANES) != 0;
            uint8_t* zp = base + (x ? a.pg.vz : a.pg.kz) + at / 2;
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
}

template <int D, int G, class T>
int append_launch(const CacheAppendArgs& a, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(a.units) * ((a.pg.hkv + 3) / 4));
    if (a.pg.sym) hipLaunchKernelGGL((cache_append<D, G, true, T>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((cache_append<D, G, false, T>), grid, dim3(256), 0, s, a);
    return static_cast<int>(hipGetLastError());
}

template <int D, class T>
int append_group(const CacheAppendArgs& a, hipStream_t s) {
    const int g = D / a.pg.ng;
    if (g == 32) return append_launch<D, 32, T>(a, s);
    if (g == 64) return append_launch<D, 64, T>(a, s);
    if constexpr (D >= 128)
        if (g == 128) return append_launch<D, 128, T>(a, s);
    if constexpr (D >= 256)
        if (g == 256) return append_launch<D, 256, T>(a, s);
    return static_cast<int>(hipErrorInvalidValue);
}

template <class T>
int append_dim(const CacheAppendArgs& a, hipStream_t s) {
    if (a.pg.d == 64) return append_group<64, T>(a, s);
    if (a.pg.d == 128) return append_group<128, T>(a, s);
    return append_group<256, T>(a, s);
}

// ---------------------------------------------------------------------------
// update and compact
//
// Both count the holders of every page from the table itself (integer
// additions, so the order of the atomics does not matter) and number the free
// or live pages in ascending order.  One workgroup does that, its counters in
// LDS where the pool's pages fit (kPlanPages) and in the scratch otherwise; a
// second launch writes the new table and copies the pages.  The plan is a few
// dependent passes over some ten thousand integers: in LDS it takes 5 to 9 us,
// where counting by one launch and scanning by another took 20 to 25 with the
// gaps between them (14 us with 256 rows of 128 pages over 12000).  Counters in the
// scratch cost a pass over global memory by that one workgroup for each of these
// passes: whole calls of 256 rows of 128 pages over 12288, 12289, 16384, 65536 and
// 262144 pages take 19, 35, 47, 136 and 415 us (update), and 20, 37 and 260 us over
// 12288, 12289 and 65536 (compact).  The copies are bound by memory: 100 MB in 19
// us, 400 MB in 70 to 77, 5.3 to 5.7 TB/s.

constexpr int kScan = 1024;        // threads of the planning workgroup
constexpr int kPlanPages = 12288;  // pages whose three counters fit LDS

// exclusive sum of v over the workgroup's kScan threads, and the total
__device__ __forceinline__ int scan_wg(int v, int* total, int* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) {
        const int y = __shfl_up(inc, x);
        if (lane >= x) inc += y;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int x = 0; x < kScan / 64; ++x) {
        const int y = lds[x];
        if (x < wave) before += y;
        all += y;
    }
    *total = all;
    return before + inc - v;
}

// What row i of the new table takes from the old one.
struct Kept {
    const int32_t* row;   // the parent's entries
    int before, after;    // lengths
    int kept, held;       // pages inherited, pages of the new length
    int last;             // slot of the page that it goes on in, or -1
};
__device__ __forceinline__ Kept kept_of(const CacheUpdateArgs& a, int i) {
    Kept k;
    const int p = a.parents[i];
    const bool has = p >= 0 && p < a.rows;
    k.row = a.table + static_cast<int64_t>(has ? p : 0) * a.max_pages;
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page;
    k.before = has ? static_cast<int>(min(static_cast<int64_t>(max(a.lens[p], 0)), cap)) : 0;
    k.after = static_cast<int>(min(max(static_cast<int64_t>(k.before) + a.grow[i], int64_t{0}), cap));
    k.held = (k.after + a.page - 1) / a.page;
    k.kept = min((k.before + a.page - 1) / a.page, k.held);
    k.last = k.after > k.before && k.before % a.page > 0 ? k.before / a.page : -1;
    return k;
}
__device__ __forceinline__ int page_in(int32_t page, int64_t n) {
    return page >= 0 && page < n ? page : -1;
}

// Entries of the table are taken by groups of 16 lanes, a row each at a time.
constexpr int kRowLanes = 16;

// The plan of an update: which row copies its last page (copies[i], the page
// or -1), the number base[i] of free pages handed out before row i's, the free
// pages in ascending order as far as they are needed, the copies (from, to)
// with their number, refs and status.
template <bool LDS>
__global__ void __launch_bounds__(kScan) update_plan(const CacheUpdateArgs a, int32_t* base, int32_t* copies, int32_t* free_list,
                                                     int32_t* moves, int32_t* counters) {
    extern __shared__ int32_t counts[];
    __shared__ int lds[kScan / 64];
    const int n = static_cast<int>(a.n_pages), tid = threadIdx.x;
    int32_t* held = LDS ? counts : counters;       // entries of the new rows that inherit a page
    int32_t* writers = held + n;                   // rows that go on in it
    int32_t* lowest = writers + n;                 // the lowest of them
    for (int p = tid; p < n; p += kScan) {
        held[p] = 0;
        writers[p] = 0;
        lowest[p] = 0x7FFFFFFF;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = tid / kRowLanes; i < a.new_rows; i += kScan / kRowLanes) {
        const Kept k = kept_of(a, i);
#pragma unroll 4
        for (int j = tid % kRowLanes; j < k.kept; j += kRowLanes) {
            const int p = page_in(k.row[j], n);
            if (p < 0) continue;
            atomicAdd(held + p, 1);
            if (j == k.last) {
                atomicAdd(writers + p, 1);
                atomicMin(lowest + p, i);
            }
        }
    }
    __threadfence_block();
    __syncthreads();
    int need = 0, done = 0, total;
    for (int c = 0; c < a.new_rows; c += kScan) {
        const int i = c + tid;
        int mine = 0, copy = -1;
        if (i < a.new_rows) {
            const Kept k = kept_of(a, i);
            if (k.last >= 0) {
                const int p = page_in(k.row[k.last], n);
                if (p >= 0 && !(lowest[p] == i && held[p] == writers[p])) copy = p;
            }
            mine = (copy >= 0) + k.held - k.kept;
            copies[i] = copy;
        }
        const int before = scan_wg(mine, &total, lds);
        if (i < a.new_rows) base[i] = need + before;
        need += total;
    }
    // free pages: a thread numbers a run of neighbouring pages.  (writers is
    // no longer needed and takes the counts of the rows that copy.)
    __syncthreads();
    for (int p = tid; p < n; p += kScan) writers[p] = 0;
    __threadfence_block();
    __syncthreads();
    const int run = (n + kScan - 1) / kScan, p0 = min(tid * run, n), p1 = min(p0 + run, n);
    int mine = 0;
    for (int p = p0; p < p1; ++p) mine += held[p] == 0;
    int found;
    int rank = scan_wg(mine, &found, lds);
    for (int p = p0; p < p1; ++p)
        if (held[p] == 0) {
            if (rank < need) {
                free_list[rank] = p;
                lowest[p] = -1;          // handed out
            }
            ++rank;
        }
    __threadfence_block();
    for (int c = 0; c < a.new_rows; c += kScan) {
        const int i = c + tid;
        int at = 0, src = -1;
        if (i < a.new_rows) {            // (this thread's own stores of the first loop)
            at = base[i];
            src = copies[i];
            if (src >= 0) atomicAdd(writers + src, 1);
        }
        const bool does = src >= 0 && at < found;
        const int m = done + scan_wg(does, &total, lds);   // (its barriers make the free pages visible)
        if (does) {
            moves[2 * m] = src;
            moves[2 * m + 1] = free_list[at];
        }
        done += total;
    }
    __threadfence_block();
    __syncthreads();
    for (int p = tid; p < n; p += kScan) a.refs[p] = lowest[p] < 0 ? 1 : held[p] - writers[p];
    if (tid == 0) {
        const int given = min(need, found), used = n - found + given;
        a.status[0] = used;
        a.status[1] = need - given;
        a.status[2] = done;
        moves[2 * int64_t{a.new_rows}] = done;
        a.status[3] = n - used;
        base[a.new_rows] = found;
    }
}

// Copies bytes [b0, b1) of a page (multiples of 16), eight loads on their way
// in every thread.
constexpr int kChunk = 256 * 8 * 16;
__device__ __forceinline__ void copy_chunk(const uint8_t* from, uint8_t* to, int64_t b0, int64_t bytes) {
    const int64_t at = b0 + threadIdx.x * 16;
    if (b0 + kChunk <= bytes) {
        uint4v x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_nontemporal_load(reinterpret_cast<const uint4v*>(from + at + i * 4096));
#pragma unroll
        for (int i = 0; i < 8; ++i) __builtin_nontemporal_store(x[i], reinterpret_cast<uint4v*>(to + at + i * 4096));
    } else {
        for (int64_t i = at; i < bytes; i += 4096)
            *reinterpret_cast<uint4v*>(to + i) = *reinterpret_cast<const uint4v*>(from + i);
    }
}

// Copies pages: workgroup b of n takes every n-th chunk of a page of one layer.
__device__ __forceinline__ void copy_pages(const uint8_t* from, int64_t from_pages, uint8_t* to, int64_t to_pages, int64_t bytes,
                                           int64_t layers, const int32_t* moves, int n_moves, int b, int n) {
    const int64_t chunks = (bytes + kChunk - 1) / kChunk, units = n_moves * layers * chunks;
    for (int64_t u = b; u < units; u += n) {
        const int64_t page = u / chunks, m = page / layers, l = page % layers;
        copy_chunk(from + (l * from_pages + moves[2 * m]) * bytes, to + (l * to_pages + moves[2 * m + 1]) * bytes,
                   u % chunks * kChunk, bytes);
    }
}
constexpr int kCopyGrid = 1024;  // workgroups that copy: 16 waves with eight loads each on a CU

// The first `rows` workgroups write the new table, a row each at a time; the
// others copy.
__global__ void __launch_bounds__(256) update_write(const CacheUpdateArgs a, const int32_t* base, const int32_t* copies,
                                                    const int32_t* free_list, const int32_t* moves, int rows) {
    if (static_cast<int>(blockIdx.x) >= rows) {
        copy_pages(a.pool, a.n_pages, a.pool, a.n_pages, a.page_bytes, a.layers, moves, moves[2 * int64_t{a.new_rows}], blockIdx.x - rows,
                   gridDim.x - rows);
        return;
    }
    const int found = base[a.new_rows];
    for (int i = blockIdx.x; i < a.new_rows; i += rows) {
        const int at = base[i];
        const bool copy = copies[i] >= 0;
        const Kept k = kept_of(a, i);
        int32_t* row = a.new_table + static_cast<int64_t>(i) * a.max_pages;
        for (int j = threadIdx.x; j < a.max_pages; j += 256) {
            int p = -1;
            if (j < k.kept && !(copy && j == k.last)) {
                p = page_in(k.row[j], a.n_pages);
            } else if (j < k.held) {
                const int64_t f = at + (j < k.kept ? int64_t{0} : static_cast<int64_t>(copy) + j - k.kept);
                p = f < found ? free_list[f] : -1;
            }
            row[j] = p;
        }
        if (threadIdx.x == 0) a.new_lens[i] = k.after;
    }
}

__device__ __forceinline__ int held_pages(const CacheCompactArgs& a, int i) {
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page;
    const int64_t len = min(static_cast<int64_t>(max(a.lens[i], 0)), cap);
    return static_cast<int>((len + a.page - 1) / a.page);
}

// The plan of a compaction: to[p], the new place of page p or -1; the moves
// (from, to) with their number; refs and status.
template <bool LDS>
__global__ void __launch_bounds__(kScan) compact_plan(const CacheCompactArgs a, int32_t* to, int32_t* moves, int32_t* counters) {
    extern __shared__ int32_t counts[];
    __shared__ int lds[kScan / 64];
    const int n = static_cast<int>(a.n_pages), places = static_cast<int>(a.into_pages), tid = threadIdx.x;
    int32_t* held = LDS ? counts : counters;     // entries of the table that hold a page
    int32_t* holes = held + n;                   // free places below the number of live pages
    for (int p = tid; p < n; p += kScan) held[p] = 0;
    for (int p = tid; p < places; p += kScan) a.refs[p] = 0;
    __threadfence_block();
    __syncthreads();
    for (int i = tid / kRowLanes; i < a.rows; i += kScan / kRowLanes) {
        const int k = held_pages(a, i);
        const int32_t* row = a.table + static_cast<int64_t>(i) * a.max_pages;
#pragma unroll 4
        for (int j = tid % kRowLanes; j < k; j += kRowLanes) {
            const int p = page_in(row[j], n);
            if (p >= 0) atomicAdd(held + p, 1);
        }
    }
    __threadfence_block();
    __syncthreads();
    // a thread numbers a run of neighbouring pages
    const int run = (n + kScan - 1) / kScan, p0 = min(tid * run, n), p1 = min(p0 + run, n);
    int mine = 0, live;
    for (int p = p0; p < p1; ++p) mine += held[p] > 0;
    const int live_before = scan_wg(mine, &live, lds);
    int moved;
    if (a.into) {
        moved = min(live, places);
        int rank = live_before;
        for (int p = p0; p < p1; ++p) {
            int t = -1;
            if (held[p] > 0 && rank++ < places) {
                t = rank - 1;
                a.refs[t] = held[p];
                moves[2 * t] = p;
                moves[2 * t + 1] = t;
            }
            to[p] = t;
        }
    } else {
        // holes below `live`: as many as live pages at and above it
        const int free_before = p0 - live_before;
        int rank = free_before;
        for (int p = p0; p < min(p1, live); ++p)
            if (held[p] == 0) holes[rank++] = p;
        mine = 0;
        for (int p = max(p0, live); p < p1; ++p) mine += held[p] > 0;
        rank = scan_wg(mine, &moved, lds);       // (its barriers make the holes visible)
        __threadfence_block();
        __syncthreads();
        for (int p = p0; p < p1; ++p) {
            int t = -1;
            if (held[p] > 0) {
                t = p;
                if (p >= live) {
                    t = holes[rank];
                    moves[2 * rank] = p;
                    moves[2 * rank + 1] = t;
                    ++rank;
                }
                a.refs[t] = held[p];
            }
            to[p] = t;
        }
    }
    if (tid == 0) {
        const int placed = a.into ? moved : live;
        a.status[0] = live;
        a.status[1] = live - placed;
        a.status[2] = moved;
        a.status[3] = places - placed;
        moves[2 * int64_t{n}] = moved;
    }
}

// The first `rows` workgroups write the new table, a row each; the others copy
// the pages, a chunk of a page of one layer at a time.
__global__ void __launch_bounds__(256) compact_write(const CacheCompactArgs a, const int32_t* to, const int32_t* moves, int rows) {
    if (static_cast<int>(blockIdx.x) < rows) {
        for (int i = blockIdx.x; i < a.rows; i += rows) {
            const int held = held_pages(a, i);
            const int64_t at = static_cast<int64_t>(i) * a.max_pages;
            for (int j = threadIdx.x; j < a.max_pages; j += 256) {
                const int p = j < held ? page_in(a.table[at + j], a.n_pages) : -1;
                a.new_table[at + j] = p < 0 ? -1 : to[p];
            }
        }
        return;
    }
    copy_pages(a.pool, a.n_pages, a.into ? a.into : a.pool, a.into_pages, a.page_bytes, a.layers, moves, moves[2 * a.n_pages],
               blockIdx.x - rows, gridDim.x - rows);
}

// Launches a planning kernel: in LDS if its counters fit, else in the scratch.
template <class A, class... P>
int plan(void (*in_lds)(A, P...), void (*in_scratch)(A, P...), int words, const A& a, hipStream_t s, P... args) {
    const size_t bytes = static_cast<size_t>(words) * a.n_pages * 4;
    if (a.n_pages <= kPlanPages) {
        if (bytes > 65536) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(in_lds), hipFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(bytes));
            if (e != hipSuccess) return static_cast<int>(e);
        }
        hipLaunchKernelGGL(in_lds, dim3(1), dim3(kScan), bytes, s, a, args...);
    } else {
        hipLaunchKernelGGL(in_scratch, dim3(1), dim3(kScan), 0, s, a, args...);
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_cache_append(const CacheAppendArgs& a, int bf16, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    return bf16 ? append_dim<uint16_t>(a, s) : append_dim<float>(a, s);
}

int launch_cache_update(const CacheUpdateArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    int32_t* base = a.work;                       // new_rows + 1
    int32_t* copies = base + a.new_rows + 1;      // new_rows
    int32_t* moves = copies + a.new_rows;         // 2 new_rows + 1
    int32_t* free_list = moves + 2 * int64_t{a.new_rows} + 1;
    const int e = plan(update_plan<true>, update_plan<false>, 3, a, s, base, copies, free_list, moves, free_list + a.n_pages);
    if (e || a.new_rows == 0) return e;
    const int rows = a.new_rows < 4096 ? a.new_rows : 4096;
    hipLaunchKernelGGL(update_write, dim3(static_cast<uint32_t>(rows + kCopyGrid)), dim3(256), 0, s, a, base, copies, free_list, moves,
                       rows);
    return static_cast<int>(hipGetLastError());
}

int launch_cache_compact(const CacheCompactArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    int32_t* to = a.work;
    int32_t* moves = to + a.n_pages;              // 2 n_pages + 1
    const int e = plan(compact_plan<true>, compact_plan<false>, 2, a, s, to, moves, moves + 2 * a.n_pages + 1);
    if (e) return e;
    const int rows = a.rows < 4096 ? a.rows : 4096;
    hipLaunchKernelGGL(compact_write, dim3(static_cast<uint32_t>(rows + kCopyGrid)), dim3(256), 0, s, a, to, moves, rows);
    return static_cast<int>(hipGetLastError());
}

}  // namespace hr
