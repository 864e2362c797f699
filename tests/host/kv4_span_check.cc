// Host build of the 4-bit cache's tile and mask arithmetic
// (io_aware_exact_21_b200/csrc/kv4_span.cuh) against the definition in 64 bits:
// query position qp sees key k when k < nk, and under a causal mask k <= qp, and
// under a window k > qp - window.  Lengths run up to 2^31 - 1, windows as well, and
// the sanitiser for signed overflow is on.  Prints "ok" and exits 0, or names the
// first violation and exits 1.
#include <algorithm>
#include <cstdio>
#include <cstdint>
#include <vector>

#define __device__
#define __forceinline__ inline
#include "kv4_span.cuh"

namespace {

int failures = 0;

void fail(const char* what, int64_t a, int64_t b, int64_t c, int64_t d) {
    if (failures++ < 10)
        std::printf("FAIL %s (%lld %lld %lld %lld)\n", what, static_cast<long long>(a), static_cast<long long>(b),
                    static_cast<long long>(c), static_cast<long long>(d));
}

bool sees(int64_t qp, int64_t k, int64_t nk, int causal, int64_t window) {
    return k >= 0 && k < nk && (!causal || k <= qp) && (window <= 0 || k > qp - window);
}

void check(int nk, int nq, int causal, int window) {
    constexpr int T = 64;
    const int tiles = fa::kv4_tile_count(nk, T);
    if (tiles != (static_cast<int64_t>(nk) + T - 1) / T) fail("tile count", nk, tiles, 0, 0);
    const int t0 = fa::kv4_first_tile(nk, nq, window, T);
    if (t0 < 0 || (nk > 0 && t0 >= tiles)) fail("first tile outside", nk, nq, window, t0);
    const int first = nk - nq, last = nk - 1;
    // no key below the first tile is seen (its last one, by the first query)
    if (t0 > 0 && sees(first, static_cast<int64_t>(t0) * T - 1, nk, causal, window)) fail("first tile", nk, nq, window, t0);
    std::vector<int> at;            // tiles looked at: the ends, and about the borders of what is seen
    for (int64_t k : {int64_t{0}, int64_t{nk} - 1, int64_t{first}, int64_t{first} - window, int64_t{last} - window})
        for (int64_t t = k / T - 2; t <= k / T + 2; ++t)
            if (t >= 0 && t < tiles) at.push_back(static_cast<int>(t));
    std::sort(at.begin(), at.end());
    at.erase(std::unique(at.begin(), at.end()), at.end());
    for (int qp = first; qp <= last; ++qp) {
        const int lo = fa::kv4_key_lo(qp, window), hi = fa::kv4_key_hi(qp, nk, causal);
        for (int t : at)
            for (int e = 0; e < T; ++e) {
                const int64_t k = static_cast<int64_t>(t) * T + e;
                if ((k >= lo && k < hi) != sees(qp, k, nk, causal, window)) fail("key range", nk, qp, window, k);
            }
    }
    for (int t : at) {
        const int k0 = t * T;
        bool all = true;
        for (int e = 0; e < T; ++e) {
            bool one = false;
            for (int qp = first; qp <= last; ++qp) {
                const bool s = sees(qp, static_cast<int64_t>(k0) + e, nk, causal, window);
                one |= s;
                all &= s;
            }
            if (k0 + e >= 0 && fa::kv4_unseen(k0 + e, nk, first, last, causal, window) == one)
                fail("unseen", nk, nq, window, k0 + e);
        }
        if (!all && !fa::kv4_tile_masked(k0, T, nk, first, last, causal, window)) fail("masked", nk, nq, window, k0);
    }
}

}  // namespace

int main() {
    constexpr int kMax = 2147483647;
    std::vector<int> lens;
    for (int n = 0; n <= 200; ++n) lens.push_back(n);
    for (int n = 0; n < 140; ++n) lens.push_back(kMax - n);
    for (int nk : lens)
        for (int nq : {1, 3, 64, 100}) {
            check(nk, nq, 0, 0);
            check(nk, nq, 1, 0);
            for (int w : {1, 2, 63, 64, 65, 1000, kMax - 200, kMax - 64, kMax - 8, kMax - 1, kMax}) check(nk, nq, 1, w);
        }
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
