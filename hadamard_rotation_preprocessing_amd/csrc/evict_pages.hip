// Eviction from the paged 4-bit cache (hr_cache_evict): the plan of its pages,
// the choice of positions, and their moves.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache_plan.h"
#include "evict.h"

namespace hr {
namespace {

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// the plan
//
// As in update and compact one workgroup counts the holders of every page from
// the table (integer additions: their order does not matter), finds which rows
// are over their budget and how many pages each needs, numbers the free pages,
// and writes the new table.

struct Row {
    const int32_t* table;
    int len, held;      // positions, pages of them
};
__device__ __forceinline__ Row row_of(const CacheEvictArgs& a, int i) {
    Row r;
    r.table = a.table + static_cast<int64_t>(i) * a.max_pages;
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.pg.page;
    r.len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[i], 0)), cap));
    r.held = static_cast<int>((static_cast<int64_t>(r.len) + a.pg.page - 1) / a.pg.page);
    return r;
}

// sums and prefixes over the kRowLanes lanes of a row
__device__ __forceinline__ uint32_t row_ballot(bool v) {
    const int first = (threadIdx.x & 63) / kRowLanes * kRowLanes;
    return static_cast<uint32_t>(__ballot(v) >> first) & ((1u << kRowLanes) - 1);
}

// need[i]: pages that row i needs; afterwards the number of free pages handed
// out before row i's, or -1 for a row that stays as it is.
template <bool LDS>
__global__ void __launch_bounds__(kScan) evict_plan(const CacheEvictArgs a, int32_t* need, int32_t* free_list, int32_t* counters) {
    extern __shared__ int32_t counts[];
    __shared__ int lds[kScan / 64];
    const int n = static_cast<int>(a.n_pages), tid = threadIdx.x, lane = tid % kRowLanes;
    int32_t* held = LDS ? counts : counters;   // entries of the old table that hold a page
    int32_t* after = held + n;                 // of the new one
    for (int p = tid; p < n; p += kScan) {
        held[p] = 0;
        after[p] = 0;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = tid / kRowLanes; i < a.rows; i += kScan / kRowLanes) {
        const Row r = row_of(a, i);
#pragma unroll 4
        for (int j = lane; j < r.held; j += kRowLanes) {
            const int p = page_in(r.table[j], n);
            if (p >= 0) atomicAdd(held + p, 1);
        }
    }
    __threadfence_block();
    __syncthreads();
    const int stay = (a.budget + a.pg.page - 1) / a.pg.page;
    for (int i = tid / kRowLanes; i < a.rows; i += kScan / kRowLanes) {
        const Row r = row_of(a, i);
        int mine = -1;
        if (r.len > a.budget) {
            mine = 0;
            bool whole = true;
            for (int j = lane; j < r.held; j += kRowLanes) {
                const int p = page_in(r.table[j], n);
                whole = whole && p >= 0;
                mine += p >= 0 && j < stay && held[p] > 1;
            }
            // (the row's lanes are all here: its length is theirs)
#pragma unroll
            for (int x = 1; x < kRowLanes; x *= 2) {
                mine += __shfl_xor(mine, x);
                whole = whole & (__shfl_xor(static_cast<int>(whole), x) != 0);
            }
            if (!whole) mine = -1;
        }
        if (lane == 0) need[i] = mine;
    }
    // free pages: a thread numbers a run of neighbouring pages
    const int run = (n + kScan - 1) / kScan, p0 = min(tid * run, n), p1 = min(p0 + run, n);
    int mine = 0, found;
    for (int p = p0; p < p1; ++p) mine += held[p] == 0;
    int rank = scan_wg(mine, &found, lds);     // (its barriers make need visible)
    for (int p = p0; p < p1; ++p)
        if (held[p] == 0) free_list[rank++] = p;
    __threadfence_block();
    __syncthreads();
    int wanted = 0, done = 0, total;
    for (int c = 0; c < a.rows; c += kScan) {
        const int i = c + tid;
        const int w = i < a.rows ? need[i] : -1;
        const int at = wanted + scan_wg(max(w, 0), &total, lds);
        const bool does = w == 0 || (w > 0 && at + w <= found);
        if (i < a.rows) {
            need[i] = does ? at : -1;
            a.new_lens[i] = does ? a.budget : row_of(a, i).len;
        }
        wanted += total;
        scan_wg(does, &total, lds);
        done += total;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = tid / kRowLanes; i < a.rows; i += kScan / kRowLanes) {
        const Row r = row_of(a, i);
        int at = need[i];
        const int keep = at >= 0 ? stay : r.held;
        int32_t* row = a.new_table + static_cast<int64_t>(i) * a.max_pages;
        for (int j0 = 0; j0 < a.max_pages; j0 += kRowLanes) {
            const int j = j0 + lane;
            int p = j < keep ? page_in(r.table[j], n) : -1;
            const bool fresh = at >= 0 && p >= 0 && held[p] > 1;
            const uint32_t all = row_ballot(fresh);
            if (fresh) p = free_list[at + __popc(all & ((1u << lane) - 1))];
            if (at >= 0) at += __popc(all);
            if (j < a.max_pages) row[j] = p;
            if (p >= 0) atomicAdd(after + p, 1);
        }
    }
    __threadfence_block();
    __syncthreads();
    mine = 0;
    for (int p = tid; p < n; p += kScan) {
        const int k = after[p];
        a.refs[p] = k;
        mine += k > 0;
    }
    scan_wg(mine, &total, lds);
    if (tid == 0) {
        a.status[0] = total;
        a.status[1] = max(wanted - found, 0);
        a.status[2] = done;
        a.status[3] = n - total;
    }
}

// ---------------------------------------------------------------------------
// choice and moves
//
// A workgroup takes a kv head of a row of one layer.  It finds the weight of the
// last position that stays by a radix selection (three histograms of 11, 11 and
// 10 bits over the weights' bits, in an order that follows their size), and then
// passes over the positions in chunks: a prefix sum gives what stays its place,
// the sources of a chunk's destinations are listed in LDS, and its vectors move,
// kMove positions at a time: all loads, a barrier, all stores.  A destination is
// never past its source, and the sources of the next kMove lie past all of these,
// so that loads of one step need not wait for the stores of the one before.
//
// Measured: 32 rows of up to 16384 cut to 4096, 4 layers of 8 heads of 128: evict_plan 19
// us, evict_move 165 to 176 us, which read 289 MB and write 173 MB by counters, 2.7 TB/s
// (of 374 MB that the moves and the selection need): positions that stay are scattered,
// so that a read is 64 bytes of a key's or value's codes.  Waves wait 80% of their time: a
// step's loads take 12 us (512 positions of each of 320 workgroups) however they are
// issued.  Four rows of 1100 cut to 1024, 2 layers: 6 and 16 us, of which the selection is 5
// and each of two steps 5.  The selection needs nothing of the plan, and waits for it.
// Tried: weights held in registers through the passes, the first histogram in copies,
// eight parts a thread, two workgroups of half the threads a compute unit, the rows over
// budget first, non-temporal loads: 165 to 173 us, and 18 to 20 for the few rows.

constexpr int kThreads = 1024;
constexpr int kPer = 4;                     // positions of a thread in a chunk
constexpr int kChunk = kThreads * kPer;
constexpr int kBins = 2048;

// A number whose unsigned order is that of the weights: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// exclusive sum over the workgroup, and the total
__device__ __forceinline__ uint32_t scan_all(uint32_t v, uint32_t* total, uint32_t* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t inc = v;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) {
        const uint32_t y = __shfl_up(inc, x);
        if (lane >= x) inc += y;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = inc;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int x = 0; x < kThreads / 64; ++x) {
        const uint32_t y = lds[x];
        if (x < wave) before += y;
        all += y;
    }
    *total = all;
    return before + inc - v;
}

struct Lds {
    uint32_t hist[kBins];
    int32_t src[kChunk];
    uint32_t scan[kThreads / 64];
    uint32_t bin, above;
};

// The rank of the k-th largest of w[lo, hi) (k from 1), and how many of those
// with exactly that rank stay.
__device__ __forceinline__ uint32_t select(const float* w, int lo, int hi, int k, int* ties, Lds& s) {
    uint32_t prefix = 0;      // the bits found so far
    int left = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        const int known = shift + bits;
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
        __syncthreads();
        for (uint32_t j = lo + threadIdx.x; j < static_cast<uint32_t>(hi); j += kThreads) {
            const uint32_t r = rank_of(w[j]);
            if (known == 32 || (r >> known) == (prefix >> known)) atomicAdd(&s.hist[(r >> shift) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        // the bin in which the count from the top reaches `left`: two bins a
        // thread, the largest first
        const int b1 = kBins - 1 - 2 * threadIdx.x, b0 = b1 - 1;
        const uint32_t n1 = s.hist[b1], n0 = s.hist[b0];
        uint32_t total;
        const uint32_t before = scan_all(n1 + n0, &total, s.scan);
        const uint32_t want = static_cast<uint32_t>(left);
        if (before < want && before + n1 >= want) {
            s.bin = b1;
            s.above = before;
        } else if (before + n1 < want && before + n1 + n0 >= want) {
            s.bin = b0;
            s.above = before + n1;
        }
        __syncthreads();
        prefix |= s.bin << shift;
        left -= static_cast<int>(s.above);
    }
    *ties = left;
    return prefix;
}

// N bytes of a vector's scales or zero points
template <int N>
struct Bytes {
    uint8_t b[N] __attribute__((aligned(N < 16 ? N : 16)));
    __device__ __forceinline__ void load(const uint8_t* p) { __builtin_memcpy(b, __builtin_assume_aligned(p, N < 16 ? N : 16), N); }
    __device__ __forceinline__ void store(uint8_t* p) const { __builtin_memcpy(__builtin_assume_aligned(p, N < 16 ? N : 16), b, N); }
};

// D: head dimension, SB: bytes of a vector's scales, ZN: zero points of a vector
// (0 if symmetric)
template <int D, int SB, int ZN>
__global__ void __launch_bounds__(kThreads) evict_move(const CacheEvictArgs a, const int32_t* done, int64_t units) {
    __shared__ Lds s;
    constexpr int PARTS = D / 16;                  // 16-byte parts of a position's codes, K and V
    constexpr int MOVE = 4 * kThreads / PARTS;     // positions of a step: four parts a thread
    const int tid = threadIdx.x;
    const CachePage& pg = a.pg;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int h = static_cast<int>(u % pg.hkv), row = static_cast<int>(u / pg.hkv % a.rows);
        const int64_t layer = u / pg.hkv / a.rows;
        if (done[row] < 0) continue;               // (the same for the whole workgroup)
        const Row r = row_of(a, row);
        float* w = a.weights + ((layer * a.rows + row) * pg.hkv + h) * a.width;
        const int32_t* to_table = a.new_table + static_cast<int64_t>(row) * a.max_pages;
        uint8_t* base = a.pool + layer * a.n_pages * pg.page_bytes + h * pg.head_bytes;
        const int lo = a.sinks, hi = r.len - a.recent, k = a.budget - a.sinks - a.recent;
        int ties = 0;
        uint32_t last = 0xFFFFFFFFu;
        bool some = k > 0;
        if (some) last = select(w, lo, hi, k, &ties, s);
        int before_all = 0, ties_all = 0;          // destinations and ties of the chunks before
        for (uint32_t c = 0; c < static_cast<uint32_t>(r.len); c += kChunk) {
            // what stays: more than the last weight, or as much and among the first `ties`
            uint32_t more = 0, same = 0;
            const uint32_t j0 = c + kPer * tid;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint32_t j = j0 + i;
                if (j >= static_cast<uint32_t>(r.len)) break;
                if (j < static_cast<uint32_t>(lo) || j >= static_cast<uint32_t>(hi)) more |= 1u << i;
                else if (some) {
                    const uint32_t x = rank_of(w[j]);
                    if (x > last) more |= 1u << i;
                    else if (x == last) same |= 1u << i;
                }
            }
            uint32_t total;
            const uint32_t sum = scan_all(__popc(more) | (__popc(same) << 16), &total, s.scan);
            int tie = ties_all + static_cast<int>(sum >> 16);
            int at = static_cast<int>(sum & 0xFFFFu) + min(tie, ties) - min(ties_all, ties);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                bool stays = (more >> i) & 1;
                if ((same >> i) & 1) stays = tie++ < ties;
                if (stays) s.src[at++] = static_cast<int>(j0) + i;
            }
            const int here = static_cast<int>(total & 0xFFFFu) + min(ties_all + static_cast<int>(total >> 16), ties) - min(ties_all, ties);
            ties_all += static_cast<int>(total >> 16);
            __syncthreads();
            for (int d0 = 0; d0 < here; d0 += MOVE) {
                const int nm = min(MOVE, here - d0);
                uint4v x[4];
                uint8_t *from[4], *to[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int part = tid % PARTS, d = i * (kThreads / PARTS) + tid / PARTS;
                    from[i] = to[i] = nullptr;
                    if (d < nm) {
                        const int src = s.src[d0 + d], dst = before_all + d0 + d;
                        const int p = r.table[src >> pg.logp], t = to_table[dst >> pg.logp];
                        constexpr int HALF = PARTS / 2;
                        const int sec = part < HALF ? pg.kc : pg.vc, in = part % HALF * 16;
                        if (p != t || src != dst) {
                            from[i] = base + p * pg.page_bytes + sec + (src & (pg.page - 1)) * (D / 2) + in;
                            to[i] = base + t * pg.page_bytes + sec + (dst & (pg.page - 1)) * (D / 2) + in;
                            x[i] = *reinterpret_cast<const uint4v*>(from[i]);
                        }
                    }
                }
                // scales, zero points and weights: a thread for a position
                Bytes<SB> ks, vs;
                Bytes<ZN <= 1 ? 1 : ZN / 2> kz, vz;
                float weight = 0.0f;
                const bool mine = tid < nm;
                bool moves = false;
                int src = 0, dst = 0;
                uint8_t *pf = nullptr, *pt = nullptr;
                if (mine) {
                    src = s.src[d0 + tid];
                    dst = before_all + d0 + tid;
                    const int p = r.table[src >> pg.logp], t = to_table[dst >> pg.logp];
                    pf = base + p * pg.page_bytes;
                    pt = base + t * pg.page_bytes;
                    moves = p != t || src != dst;
                    const int off = src & (pg.page - 1);
                    ks.load(pf + pg.ks + off * SB);
                    vs.load(pf + pg.vs + off * SB);
                    if constexpr (ZN >= 2) {
                        kz.load(pf + pg.kz + off * (ZN / 2));
                        vz.load(pf + pg.vz + off * (ZN / 2));
                    } else if constexpr (ZN == 1) {
                        kz.b[0] = (pf[pg.kz + off / 2] >> (4 * (off & 1))) & 15;
                        vz.b[0] = (pf[pg.vz + off / 2] >> (4 * (off & 1))) & 15;
                    }
                    weight = w[src];
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (to[i]) *reinterpret_cast<uint4v*>(to[i]) = x[i];
                uint32_t zn = 0;
                if constexpr (ZN == 1) zn = kz.b[0] | (vz.b[0] << 8);
                if (mine) {
                    const int off = dst & (pg.page - 1);
                    if (moves) {
                        ks.store(pt + pg.ks + off * SB);
                        vs.store(pt + pg.vs + off * SB);
                        if constexpr (ZN >= 2) {
                            kz.store(pt + pg.kz + off * (ZN / 2));
                            vz.store(pt + pg.vz + off * (ZN / 2));
                        }
                        w[dst] = weight;
                    }
                    if constexpr (ZN == 1) s.hist[tid] = zn;   // (the histogram is no longer needed)
                }
                if constexpr (ZN == 1) {
                    // two positions to a byte: the even one's thread writes it, or the
                    // odd one's where that is the step's first; a half that belongs to
                    // no position of the step stays as it is
                    __syncthreads();
                    if (mine && (!(dst & 1) || tid == 0)) {
                        const int off = dst & (pg.page - 1);
                        const bool pair = !(dst & 1) && tid + 1 < nm;
                        const uint32_t other = pair ? s.hist[tid + 1] : 0;
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            uint8_t* z = pt + (v ? pg.vz : pg.kz) + off / 2;
                            const uint32_t me = (zn >> (8 * v)) & 15u, ot = (other >> (8 * v)) & 15u;
                            if (pair) *z = static_cast<uint8_t>(me | (ot << 4));
                            else if (dst & 1) *z = static_cast<uint8_t>((*z & 15u) | (me << 4));
                            else *z = static_cast<uint8_t>((*z & 0xF0u) | me);
                        }
                    }
                }
            }
            before_all += here;
            __syncthreads();
        }
    }
}

template <int D, int SB>
void move_zeros(const CacheEvictArgs& a, const int32_t* done, int64_t units, dim3 grid, hipStream_t s) {
    constexpr int MOST = D / 32;
    const int zn = a.pg.sym ? 0 : a.pg.ng;
    if (zn == 0) hipLaunchKernelGGL((evict_move<D, SB, 0>), grid, dim3(kThreads), 0, s, a, done, units);
    if (zn == 1) hipLaunchKernelGGL((evict_move<D, SB, 1>), grid, dim3(kThreads), 0, s, a, done, units);
    if constexpr (MOST >= 2)
        if (zn == 2) hipLaunchKernelGGL((evict_move<D, SB, 2>), grid, dim3(kThreads), 0, s, a, done, units);
    if constexpr (MOST >= 4)
        if (zn == 4) hipLaunchKernelGGL((evict_move<D, SB, 4>), grid, dim3(kThreads), 0, s, a, done, units);
    if constexpr (MOST >= 8)
        if (zn == 8) hipLaunchKernelGGL((evict_move<D, SB, 8>), grid, dim3(kThreads), 0, s, a, done, units);
}

template <int D>
void move_scales(const CacheEvictArgs& a, const int32_t* done, int64_t units, dim3 grid, hipStream_t s) {
    const int sb = a.pg.ng * (a.pg.sf32 ? 4 : 2);
    if (sb == 2) move_zeros<D, 2>(a, done, units, grid, s);
    if (sb == 4) move_zeros<D, 4>(a, done, units, grid, s);
    if (sb == 8) move_zeros<D, 8>(a, done, units, grid, s);
    if constexpr (D >= 128)
        if (sb == 16) move_zeros<D, 16>(a, done, units, grid, s);
    if constexpr (D >= 256)
        if (sb == 32) move_zeros<D, 32>(a, done, units, grid, s);
}

constexpr int64_t kMoveGrid = 1 << 20;

}  // namespace

int launch_cache_evict(const CacheEvictArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    int32_t* need = a.work;                       // rows
    int32_t* free_list = need + a.rows;           // n_pages
    const int e = plan(evict_plan<true>, evict_plan<false>, 2, a, s, need, free_list, free_list + a.n_pages);
    if (e || a.rows == 0) return e;
    const int64_t units = a.layers * a.rows * a.pg.hkv;
    const dim3 grid(static_cast<uint32_t>(units < kMoveGrid ? units : kMoveGrid));
    if (a.pg.d == 64) move_scales<64>(a, need, units, grid, s);
    else if (a.pg.d == 128) move_scales<128>(a, need, units, grid, s);
    else move_scales<256>(a, need, units, grid, s);
    return static_cast<int>(hipGetLastError());
}

}  // namespace hr
