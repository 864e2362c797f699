/* Plain C caller of the 4-bit cache's entry points: compiles against
 * include/fa.h alone and exercises their host-side argument checks (nothing
 * reaches a GPU). */
#include <stdio.h>
#include "fa.h"

#define CHECK(expr, want)                                                        \
    do {                                                                         \
        int got_ = (int)(expr);                                                  \
        if (got_ != (want)) {                                                    \
            printf("FAIL %s: got %d want %d\n", #expr, got_, (want));            \
            return 1;                                                            \
        }                                                                        \
    } while (0)

int main(void) {
    void* p = (void*)(size_t)0x10000;          /* never dereferenced */
    void* odd = (void*)(size_t)0x10008;
    float* f = (float*)p;
    const int* n = (const int*)p;
    /* B, N, Hkv, Nk, d */
    CHECK(fa_quantize_kv4(p, p, p, p, p, p, 2, 0, 3, 64, 128, NULL, NULL, NULL, 0), FA_OK);
    CHECK(fa_quantize_kv4(NULL, p, p, p, p, p, 2, 4, 3, 64, 128, NULL, NULL, NULL, 0), FA_ERR_NULLPTR);
    CHECK(fa_quantize_kv4(p, p, p, p, p, p, 2, 4, 3, 64, 96, NULL, NULL, NULL, 0), FA_ERR_UNSUPPORTED_D);
    CHECK(fa_quantize_kv4(p, p, p, p, p, p, 2, 4, 3, 60, 128, NULL, NULL, NULL, 0), FA_ERR_BAD_SHAPE);
    CHECK(fa_quantize_kv4(p, p, p, p, p, p, 2, 4, 3, 64, 128, n, NULL, n, 0), FA_ERR_BAD_SHAPE);
    CHECK(fa_quantize_kv4(odd, p, p, p, p, p, 2, 4, 3, 64, 128, NULL, n, NULL, 0), FA_ERR_MISALIGNED);
    CHECK(fa_dequantize_kv4(p, p, p, p, p, p, 2, 0, 3, 64, 128, NULL, NULL, NULL, 0), FA_OK);
    CHECK(fa_dequantize_kv4(p, p, p, NULL, p, p, 2, 4, 3, 64, 128, NULL, NULL, NULL, 0), FA_ERR_NULLPTR);
    CHECK(fa_dequantize_kv4(p, p, odd, p, p, p, 2, 4, 3, 64, 64, NULL, NULL, NULL, 0), FA_ERR_MISALIGNED);
    /* B, H, Hkv, Nq, Nk, d, scale, causal, window, seqlens_k, num_splits, workspace */
    CHECK(fa_fwd_kv4(p, p, p, p, p, p, f, 2, 6, 3, 0, 512, 128, 0.1f, 1, 0, NULL, 1, NULL, 0, 0), FA_OK);
    CHECK(fa_fwd_kv4(p, p, p, p, p, p, f, 2, 7, 3, 1, 512, 128, 0.1f, 1, 0, NULL, 1, p, 1 << 30, 0), FA_ERR_BAD_SHAPE);
    CHECK(fa_fwd_kv4(p, p, p, p, p, p, f, 2, 6, 3, 1, 512, 128, 0.1f, 1, 0, NULL, 33, p, 1 << 30, 0), FA_ERR_BAD_SHAPE);
    CHECK(fa_fwd_kv4(p, p, p, p, p, p, f, 2, 6, 3, 1, 512, 128, 0.f, 1, 0, NULL, 1, p, 1 << 30, 0), FA_ERR_BAD_SCALE);
    CHECK(fa_fwd_kv4(p, p, p, p, p, p, f, 2, 6, 3, 1, 512, 128, 0.1f, 0, 9, NULL, 1, p, 1 << 30, 0), FA_ERR_BAD_MASK);
    CHECK(fa_fwd_kv4(p, p, p, p, p, p, f, 2, 6, 3, 1, 512, 128, 0.1f, 1, 0, NULL, 4, NULL, 0, 0), FA_ERR_WORKSPACE);
    CHECK(fa_fwd_kv4(p, p, p, p, p, p, f, 2, 6, 3, 1, 512, 128, 0.1f, 1, 0, NULL, 4, odd, 1 << 30, 0), FA_ERR_MISALIGNED);
    /* one key split: two partial results of 8 query rows to each of 6 items */
    CHECK(fa_fwd_kv4_workspace_size(2, 6, 3, 1, 512, 128, 0, 1), 2 * 6 * 8 * 130 * 4);
    CHECK(fa_fwd_kv4_workspace_size(2, 7, 3, 1, 512, 128, 0, 1), 0);
    printf("ok\n");
    return 0;
}
