// Which tokens and positions a wave of cache_append takes: index arithmetic
// alone, so that it can be compiled and checked without a device.
#pragma once

#include <stdint.h>

#include "cache.h"

#ifdef __HIP__
#define HR_INDEX __host__ __device__ __forceinline__
#else
#define HR_INDEX inline
#endif

namespace hr {

HR_INDEX int index_min(int a, int b) { return a < b ? a : b; }
HR_INDEX int index_max(int a, int b) { return a > b ? a : b; }

// The positions that block u of POS takes: [p0, p0 + POS) of sequence b, and
// what its tokens are.
struct AppendBlock {
    int b, start, n;   // the sequence, its first token, its number of tokens
    int first, len;    // position of its first new token (may lie before 0), positions
    int p0;            // the block's first position
    bool any;          // whether a new token lies in it; nothing is read or written if not

    // whether position p holds a new token
    HR_INDEX bool holds(int p) const { return p >= index_max(first, 0) && p < len; }
    // the token of position p, or of the nearest one that holds a token (any only)
    HR_INDEX int token(int p) const { return start + index_min(index_max(p - first, 0), n - 1); }
};

template <int POS>
HR_INDEX AppendBlock append_block(const CacheSeqs& sq, int logp, int u) {
    const auto cu = [&](int b) { return index_min(index_max(sq.cu ? sq.cu[b] : b * sq.per, 0), sq.tokens); };
    AppendBlock k;
    // the last b with floor(cu(b) / POS) + 2 b <= u, a bound that leaves every
    // sequence at least the blocks it touches
    k.b = 0;
    int hi = sq.rows - 1;
    while (k.b < hi) {
        const int mid = (k.b + hi + 1) / 2;
        if (cu(mid) / POS + 2 * mid <= u) k.b = mid;
        else hi = mid - 1;
    }
    k.start = cu(k.b);
    k.n = index_max(cu(k.b + 1) - k.start, 0);
    k.len = index_min(index_max(sq.lens[k.b], 0), sq.max_pages << logp);
    k.first = k.len - k.n;
    // (a sequence without new tokens has blocks as well; compared in blocks, as
    // a position past the longest table's last one may not fit an int)
    const int nth = u - (k.start / POS + 2 * k.b), block = index_max(k.first, 0) / POS;
    k.any = k.n > 0 && k.len > 0 && nth >= 0 && nth <= (k.len - 1) / POS - block;
    k.p0 = k.any ? (block + nth) * POS : 0;
    return k;
}

}  // namespace hr
