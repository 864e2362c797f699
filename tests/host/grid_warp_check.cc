// Host build of the warp numbering of the kernels with a warp to each (row, head)
// (grid_warp in io_aware_exact_21_b200/csrc/schedule.cuh): a grid of 256-thread
// CTAs gives each warp its own number, in order, up to the largest grid that the
// host launches, past 2^27 warps (2^32 threads) too.  Prints "ok" and exits 0, or
// names the first violation and exits 1.
#include <algorithm>
#include <cstdint>
#include <cstdio>

#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
struct Dim3 {
    unsigned x = 0, y = 1, z = 1;
};
static Dim3 blockIdx, gridDim, threadIdx, blockDim;
static inline void __syncthreads() {}

#include "schedule.cuh"

int main() {
    blockDim.x = 256;
    const int64_t last = fa::kMaxGridWarps / 8;
    const int64_t from[] = {0, (int64_t{1} << 24) - 3, (int64_t{1} << 27) - 3, (int64_t{1} << 27) + 12345, last - 6};
    for (int64_t f : from)
        for (int64_t b = f; b < f + 6; ++b)
            for (unsigned t = 0; t < 256; ++t) {
                blockIdx.x = static_cast<unsigned>(b);
                threadIdx.x = t;
                if (static_cast<int64_t>(fa::grid_warp()) != b * 8 + t / 32) {
                    std::printf("FAIL block %lld thread %u: warp %lld\n", static_cast<long long>(b), t,
                                static_cast<long long>(fa::grid_warp()));
                    return 1;
                }
            }
    std::puts("ok");
    return 0;
}
