// kv4_span.cuh -- which key tiles of a 4-bit cache a sequence has and what a
// block of query rows sees of them.  A cache may hold up to 2^31 - 8 rows, so no
// sum here goes past a row that exists: positions are below 2^31, a query's
// position qp lies in [-Nq, nk), a tile starts at k0 < nk, and a window is below
// 2^31.
#pragma once

namespace fa {

__device__ __forceinline__ int kv4_tile_count(int keys, int tile) { return keys / tile + (keys % tile != 0); }

// First tile that the last nq positions of nk rows need under a window.
__device__ __forceinline__ int kv4_first_tile(int nk, int nq, int window, int tile) {
    if (window <= 0) return 0;
    const long long first = static_cast<long long>(nk) - nq - window + 1;
    return first > 0 ? static_cast<int>(first / tile) : 0;
}

// The keys that query position qp sees are [lo, hi).
__device__ __forceinline__ int kv4_key_lo(int qp, int window) {
    return window > 0 && qp >= window ? qp - window + 1 : 0;
}
__device__ __forceinline__ int kv4_key_hi(int qp, int nk, int causal) { return causal && qp < nk ? qp + 1 : nk; }

// Whether some query of positions [first, last] does not see some key of the tile
// at k0, and whether no one of them sees `key`.
__device__ __forceinline__ bool kv4_tile_masked(int k0, int tile, int nk, int first, int last, int causal,
                                                int window) {
    return nk - k0 < tile || (causal && k0 + (tile - 1) > first) || (window > 0 && last - k0 >= window);
}
__device__ __forceinline__ bool kv4_unseen(int key, int nk, int first, int last, int causal, int window) {
    return key >= nk || (causal && key > last) || (window > 0 && first - key >= window);
}

}  // namespace fa
