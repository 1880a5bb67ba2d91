// Writing the paged 4-bit cache (hr_cache_append) and moving its pages
// (hr_cache_update, hr_cache_compact).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache.h"
#include "cache_index.h"
#include "cache_plan.h"
#include "cache_vectors.h"
#include "codes.h"

namespace hr {
namespace {

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
