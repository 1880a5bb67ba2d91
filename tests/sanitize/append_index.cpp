// The index arithmetic of cache_append without a device: every block of every
// call below reads tokens of its own sequence only, and the new positions of a
// sequence are taken exactly once, by the token that belongs there.
#include <stdio.h>

#include <random>
#include <vector>

#include "../../hadamard_rotation_preprocessing_amd/csrc/cache_index.h"

namespace {

int errors = 0;

template <int POS>
void check(const std::vector<int>& lens, const std::vector<int>& cu, bool use_cu, int max_pages, int logp) {
    hr::CacheSeqs s{};
    s.lens = lens.data();
    s.rows = static_cast<int32_t>(lens.size());
    s.tokens = cu.back();
    s.per = s.tokens / s.rows;
    s.cu = use_cu ? cu.data() : nullptr;
    s.max_pages = max_pages;
    std::vector<std::vector<int>> got(lens.size());
    for (size_t b = 0; b < lens.size(); ++b) got[b].assign(size_t{1} * max_pages << logp, -1);
    const int units = s.tokens / POS + 2 * s.rows;
    for (int u = 0; u < units; ++u) {
        const hr::AppendBlock k = hr::append_block<POS>(s, logp, u);
        if (!k.any) continue;
        for (int i = 0; i < POS; ++i) {
            const int p = k.p0 + i, t = k.token(p);
            if (t < cu[k.b] || t >= cu[k.b + 1]) {
                printf("POS %d row %d (length %d, tokens %d..%d): reads token %d\n", POS, k.b, lens[k.b], cu[k.b], cu[k.b + 1], t);
                ++errors;
            }
            if (!k.holds(p)) continue;
            if (got[k.b][p] != -1) ++errors, printf("POS %d row %d position %d twice\n", POS, k.b, p);
            got[k.b][p] = t;
        }
    }
    for (size_t b = 0; b < lens.size(); ++b) {
        const int len = std::min(std::max(lens[b], 0), max_pages << logp), n = cu[b + 1] - cu[b];
        for (size_t p = 0; p < got[b].size(); ++p) {
            const int pos = static_cast<int>(p), want = pos < len && pos >= len - n ? cu[b] + pos - (len - n) : -1;
            if (got[b][p] != want) ++errors, printf("POS %d row %zu position %d: token %d, not %d\n", POS, b, pos, got[b][p], want);
        }
    }
}

void all(const std::vector<int>& lens, const std::vector<int>& news, int max_pages = 8, int logp = 4) {
    std::vector<int> cu(1, 0);
    bool same = true;
    for (int n : news) cu.push_back(cu.back() + n), same &= n == news[0];
    for (int use_cu = same ? 0 : 1; use_cu < 2; ++use_cu) {
        check<4>(lens, cu, use_cu, max_pages, logp);
        check<8>(lens, cu, use_cu, max_pages, logp);
        check<16>(lens, cu, use_cu, max_pages, logp);
    }
}

// The longest table there can be: its last positions, and no block past them.
void far() {
    const int len = 0x7FFFFFF0, cu[] = {0, 3}, lens[] = {len};
    hr::CacheSeqs s{};
    s.lens = lens;
    s.cu = cu;
    s.rows = 1;
    s.tokens = 3;
    s.max_pages = len >> 4;
    int taken = 0;
    for (int u = 0; u < 3 / 8 + 2 + 4; ++u) {
        const hr::AppendBlock k = hr::append_block<8>(s, 4, u);
        if (!k.any) continue;
        if (k.p0 < len - 16 || k.p0 > len - 8) ++errors, printf("block at %d\n", k.p0);
        for (int i = 0; i < 8; ++i) taken += k.holds(k.p0 + i);
    }
    if (taken != 3) ++errors, printf("%d of 3 taken\n", taken);
}

}  // namespace

int main() {
    all({100, 50}, {0, 3});                      // an idle sequence first
    all({1, 7, 100, 33}, {0, 0, 0, 5});          // several
    all({31, 50, 9}, {2, 0, 3});                 // between others
    all({31, 50, 9}, {2, 3, 0});                 // last
    all({5, 0, 3, 128}, {0, 0, 0, 0});           // no new token at all
    all({0, 4, 0}, {6, 7, 0});                   // more new tokens than positions
    all({3000, -5, 20}, {4, 1, 0});              // lengths beyond the table and below zero
    far();
    std::mt19937 rng(1);
    for (int i = 0; i < 3000; ++i) {
        const int rows = 1 + rng() % 7;
        std::vector<int> lens(rows), news(rows);
        for (int b = 0; b < rows; ++b) {
            lens[b] = rng() % 140;
            news[b] = rng() % 3 ? rng() % 40 : 0;
        }
        all(lens, news);
    }
    printf("%d errors\n", errors);
    return errors != 0;
}
