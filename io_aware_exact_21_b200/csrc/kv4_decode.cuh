// kv4_decode.cuh -- attention of a few query rows over the 4-bit key/value
// cache (kv4_rows.cuh has the format), split along the keys.
//
// With code c, scale s and zero z of a cache row, and x_ij the score of query
// row i and key j in base 2,
//     x_ij = scale log2(e) s^k_j (sum_c q_ic c^k_jc - z^k_j sum_c q_ic),
//     O_i  = sum_j p_ij s^v_j (c^v_j - z^v_j) / sum_j p_ij,  p_ij = 2^(x_ij - m_i).
// The codes enter the matrix products as they are: a nibble in the low bits of
// a 16-bit word is the fp16 subnormal c 2^-24, one nibble further up c 2^-20,
// and tensor cores multiply subnormals exactly.  So unpacking is one AND a
// pair of codes and one shift for every four pairs, with no conversion; the
// powers of two go into q (its channels at the upper nibbles carry 1/16) and
// into the last scaling of O.  The scales and zeros apply to the small fp32
// score tile: scale after the product, s^v folded into p.
//
// Roundings.  q is scaled by a power of two per row so that its largest element
// lies in [2^14, 2^15) and held in fp16, which is exact for elements down to 2^-24
// of that one and off by 2^-25 of the row's largest below it.  w = p s^v is scaled
// by a power of two and rounded to fp16, the two-byte operand that the product
// needs: by 2^-11 (bf16: 2^-8) or, where it is small, by 2^-21 of the largest w of
// its query row.  The power of two is one for the warp, from the largest s^v of its
// keys so far, while the s^v of all keys that its rows can see lie within 2^10 of
// that: then each row's largest w stays above 2^-4 (p is 1 at the row's reference),
// and fp16's step is at most 2^-24.  Where a scale lies farther off, a large row that
// a mask hides from another query, or whose p is next to nothing, would push the w
// that count out of fp16; from there on each query row has a power of two of its own,
// from the largest w it has met (kv4_attend).  Looking for such scales costs a vote a
// tile: 1 to 3 % of the time, 5 % of the shortest calls.
// The zeros are one more row of the second product, so the same rounded weights
// multiply c and z, and an error of theirs goes with |c - z|; with the weights as they
// were before the rounding it went with c, eight times as far where most codes stand
// next to z.  (The products are exact, but the tensor core takes an fp16 subnormal for
// a number of 2^-14 when it lines products up to add them, and cuts what lies 2^-23
// below the largest: up to 2^-13 of the largest w of 16 keys, in units of a code.  z is
// cut as c is.  In the scores, sums of q c, it is 2^-13 of the largest |q| of 16
// channels: nothing for q's eight bits while its elements are within 2^6 of each
// other, 1e-3 of the LSE where one is 100 times the rest.  All codes at a byte's high
// half would make both 2^-17, for 2 more shifts to 8 codes: 44.9 us for 42.9 with
// the scores' alone at B 16, 47.6 with both.)  Everything else is fp32, the row sums
// take the unrounded p.
//
// What bounds it: with R = Nq * H / Hkv query rows to a key/value head the
// cache is D + 4 bytes a token and head for 4 R D operations, so up to a dozen
// rows HBM is the limit if the instructions per code stay few.  mma.sync
// rather than tcgen05: its operands come from registers, where the codes are
// unpacked, while tcgen05 would have them written back to shared or tensor
// memory as 16-bit words first, four times the cache's bytes.
//
// A warp takes whole key tiles, through its own stage of bulk copies, with its
// own reference and sums, and waits for no other warp; what several warps have
// of the same rows is put together at the end, within a cluster
// (kv4_cluster_kernel) or by a second kernel (kv4_decode_kernel and
// kv4_merge_kernel).
//
// Measured on one B200 at 16 requests x 16 heads, one query each, caches of
// 4096 to 8192 rows, d = 128 (208 MB, 31.7 us at the measured copy rate): 43 to 45
// us on different boards with the merge, which is 3 of them.  The same with the arithmetic left out 34
// us, with the loads left out 33 us; so both sides matter, and an instruction
// less a code has been worth more than anything else: 64 us with a tile of 32
// keys, cp.async and a maximum looked for in each tile; 47 us with equal ranges
// and the maximum only where a tile's sum asks for it; 45 us with ldmatrix in
// place of byte permutes.  More warps with fewer registers (16 of 128 an SM:
// 46 us against 43 without the merge), deeper stages (44 against 43) and 8-bit
// products (their mma.sync is slower here than the 16-bit one) did not pay.
//
// Per tile: S^T = C^k q^T with 16 keys x 8 query rows to an mma (the codes are
// the A operand), p from it in registers, transposed by movmatrix into the B
// operand of O^T += C^v p^T, whose A operand, two keys' codes in a register,
// comes from a transposing ldmatrix over the bytes of the tile.  Which channel
// sits at which mma index is free as long as q agrees, so of K each lane reads
// whole words of codes, the D/4 channels of lane % 4.
#pragma once

#include "decode_kernel.cuh"
#include "kv4_rows.cuh"
#include "kv4_span.cuh"

namespace fa {

struct Kv4DecodeParams {
    const __nv_bfloat16* q;      // [B, Nq, H, D]
    const uint8_t* codes[2];     // K, V: [B, Hkv, Nk, D / 2]
    const uint16_t* words[2];    // [B, Hkv, Nk]
    __nv_bfloat16* o;            // [B, Nq, H, D]
    float* lse;                  // [B, H, Nq]
    float* o_part;               // [2 ranges, ROWS, D] partial outputs, see kv4_span
    float2* ml_part;             // [2 ranges, ROWS] their references and sums, base 2
    const int* seqlens_k;        // [B] or nullptr
    int B, H, Hkv, G, Nq, Nk;    // G = H / Hkv
    int causal, window;
    int row_blocks;              // blocks of ROWS query rows to a (sequence, kv head)
    int ranges;                  // ranges the work is cut into at most
    float scale_log2;
    int* error_word;
    uint64_t timeout_ns;
    int fault_skip;              // test hook: the first K tile of each warp is left unloaded
};

template <int D, int NT>
struct Kv4DecCfg {
    static constexpr int BN = 64;                         // keys a tile
    static constexpr int ROWS = 8 * NT;                   // query rows a warp
    static constexpr int WARPS = 4;                       // a CTA
    static constexpr int MIN_CTAS = NT == 1 ? 3 : 2;      // an SM: 168 and 255 registers a thread
    static constexpr int MT = BN / 16;                    // mma key tiles
    static constexpr int ROWB = D / 2;                    // bytes of a row's codes
    static constexpr int TILE = BN * ROWB;                // K or V codes of a tile
    static constexpr int WORDB = BN * 2;
    // a warp's shared memory: V codes (swizzled, so 1024-byte aligned); K codes,
    // K words, V words; (scale, zero) of K, scales of V, zeros of V as 16-bit words
    static constexpr int OFF_K = TILE;
    static constexpr int OFF_WORDS = OFF_K + TILE;
    static constexpr int OFF_SCALES = OFF_WORDS + 2 * WORDB;
    static constexpr int OFF_ROWS = OFF_SCALES + BN * 14;               // [ROWS] Kv4RowScale
    static constexpr int WARP_BYTES = (OFF_ROWS + ROWS * 12 + 1023) / 1024 * 1024;
    static constexpr int OFF_BAR = WARPS * WARP_BYTES;                  // [WARPS][2]: K, V
    static constexpr int OFF_MISC = OFF_BAR + WARPS * 16;
    static constexpr int SMEM = OFF_MISC + WARPS * 12 + 16 + 1024;
    static constexpr int OSTRIDE = D + 4;                 // floats a row of a partial output in shared memory
    static_assert(TILE % 1024 == 0 && OFF_WORDS % 16 == 0 && WORDB % 16 == 0, "copies and swizzle");
    static_assert(ROWS * (OSTRIDE + 2) * 4 <= OFF_ROWS, "a warp leaves its partial result in its memory");
};

// p may grow to this before its reference moves: 2^8 times s^v below 2^7 is in fp16
constexpr float kKv4Over = 256.f;
constexpr float kNoRef = 3.4028234e38f;   // minus the reference before the first score: any score then is over

// Where the V scales of a warp's keys differ by more than kKv4Spread powers of
// two: a query row's largest w, in units of 2^8, up to the last tile, minus the
// reference that it is relative to (kNoRef: no key yet), and the power k that the
// row's w and sums are scaled by in those units.
constexpr int kKv4Spread = 10;
constexpr uint32_t kKv4Unseen = 0x10000u;   // in place of the word of a V row that no query sees: s, z = 0
struct Kv4RowScale {
    float largest, minus_ref;
    int k;
    __device__ __forceinline__ void take(float w, float nm) {
        largest = fmaxf(minus_ref == kNoRef ? 0.f : largest * ex2(nm - minus_ref), w);
        minus_ref = nm;
    }
};

// The power that brings the largest w into [2^13, 2^14); the limits keep p 2^k and
// 2^-k within fp32.
__device__ __forceinline__ int kv4_row_power(const Kv4RowScale& r) {
    return min(max(r.largest > 0.f ? 140 - static_cast<int>(__float_as_uint(r.largest) >> 23) : r.k, -112), 119);
}
__device__ __forceinline__ float kv4_pow2(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

__device__ __forceinline__ void mma_f16(float2 (&c)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0].x), "+f"(c[0].y), "+f"(c[1].x), "+f"(c[1].y)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float2 (&c)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0].x), "=f"(c[0].y), "=f"(c[1].x), "=f"(c[1].y)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// {low: a, high: b} as fp16
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

constexpr uint32_t kNibLo = 0x000f000fu, kNibHi = 0x00f000f0u;

// Keys of a 16-key tile at mma index g (and, 4 further, g + 8) of the score
// product.  It follows from the second product, whose operand ldmatrix brings
// in transposed: four keys of a byte column to a lane, whose codes of keys
// (0, 2) and (1, 3) of the four pair up under the masks.  The order of the
// rows that ldmatrix is given (kv4_v_key) is chosen so that eight of them, and
// two K rows, fall into different banks.
__device__ __forceinline__ int kv4_key(int g) { return (g & 3) | ((g >> 2) << 3); }
__device__ __forceinline__ int kv4_v_key(int i) { return (i & 8) | ((i & 7) >> 1) | ((i & 1) << 2); }

// Two 16 x 16 byte matrices (keys x byte columns), transposed: registers 0, 1
// hold columns lane / 4 and lane / 4 + 8 of the first, keys 4 (lane % 4) .. + 3.
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t row) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(row)
                 : "memory");
}

struct Kv4Span {
    int nk, t0, n;      // used keys, first key tile and tiles of a sequence
};

template <int BN>
__device__ __forceinline__ Kv4Span kv4_span(const Kv4DecodeParams& p, int b) {
    Kv4Span s;
    s.nk = p.seqlens_k ? min(max(p.seqlens_k[b], 0), p.Nk) : p.Nk;
    s.t0 = kv4_first_tile(s.nk, p.Nq, p.window, BN);
    s.n = kv4_tile_count(s.nk, BN) - s.t0;
    return s;
}

// Row of [B * Nq * H] of query row r of kv head hk, and its place in lse.
__device__ __forceinline__ size_t kv4_out_row(const Kv4DecodeParams& p, int b, int hk, int r, size_t& lse_at) {
    const int i = r / p.G, h = hk * p.G + r - i * p.G;
    lse_at = (static_cast<size_t>(b) * p.H + h) * p.Nq + i;
    return (static_cast<size_t>(b) * p.Nq + i) * p.H + h;
}

// A query row's sum of partial results, held by a warp: D / 32 channels a
// lane, the reference M (base 2) and the sum L.
template <int D>
struct Kv4Row {
    float a[D / 32], M, L;
    __device__ __forceinline__ Kv4Row() : M(-INFINITY), L(0.f) {
#pragma unroll
        for (int e = 0; e < D / 32; ++e) a[e] = 0.f;
    }
    // Adds the partial result with reference and sum `ml` and the lane's channels v.
    __device__ __forceinline__ void take(float2 ml, const float* v) {
        if (ml.x == -INFINITY && !isnan(ml.y)) return;      // no key of this row
        const float m = fmaxf(M, ml.x);
        const float w0 = M == -INFINITY ? 0.f : ex2(M - m), w1 = ex2(ml.x - m);
        L = (M == -INFINITY ? L : L * w0) + ml.y * w1;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) a[e] = fmaf(v[e], w1, a[e] * w0);
        M = m;
    }
    __device__ __forceinline__ void store(const Kv4DecodeParams& p, int b, int hk, int r) const {
        const int lane = lane_id();
        size_t lse_at;
        const size_t row = kv4_out_row(p, b, hk, r, lse_at);
        const bool some = !(L == 0.f);                      // a NaN sum stays NaN
        const float inv = some ? 1.f / L : 0.f;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + lane * (D / 32));
#pragma unroll
        for (int e = 0; e < D / 64; ++e) dst[e] = pack_bf16(a[2 * e] * inv, a[2 * e + 1] * inv);
        if (lane == 0) p.lse[lse_at] = some ? (M + __log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
};

// What a warp has of an item: O^T in mma fragments ([m][nt][mma row g8 / g8 + 8],
// query rows 2 t4 + {0, 1}), the sums of p s^v z likewise (mma rows 0 .. 7 alike,
// for the even channels, and 8 .. 15), the lane's sums of p, minus the reference
// (kNoRef: none), the exponent that O and za are scaled by, with a power of each
// row's own besides where `wide` is set (OFF_ROWS).
template <int D, int NT>
struct Kv4Acc {
    float2 o[D / 16][NT][2], za[NT][2];
    float2 l[NT], nm[NT];
    uint32_t ev;                    // biased exponent of the largest V scale
    bool wide;
};

// One warp's attention over `count` key tiles (from tile `first` on) of kv head
// hk of sequence b, for query rows r0 .. r0 + nrows - 1.  `ring` is the warp's
// shared memory, bar_k its two barriers, `phase` their phase.  False when a
// wait gave up.
template <int D, int NT>
__device__ __forceinline__ bool kv4_attend(const Kv4DecodeParams& p, const CUtensorMap* tm_v, Kv4Acc<D, NT>& acc,
                                           uint8_t* ring, uint64_t* bar_k,
                                           uint32_t& phase, const WaitCtl& wc, int b, int hk, int r0, int nrows,
                                           int nk, int first, int count) {
    using C = Kv4DecCfg<D, NT>;
    const int lane = lane_id(), g8 = lane >> 2, t4 = lane & 3;
    const float kNegInf = -INFINITY;
    uint64_t* bar_v = bar_k + 1;
    float2* sck = reinterpret_cast<float2*>(ring + C::OFF_SCALES);
    float* scv = reinterpret_cast<float*>(sck + C::BN);
    uint16_t* zv = reinterpret_cast<uint16_t*>(scv + C::BN);
    const int qpos0 = nk - p.Nq;                             // key position of query 0
    const int64_t row0 = (static_cast<int64_t>(b) * p.Hkv + hk) * p.Nk + static_cast<int64_t>(first) * C::BN;
    const int room = p.Nk - first * C::BN;
    // loads of tile i: K with both words, and V (rows to be read are a multiple of 8)
    auto load_k = [&](int i) {
        if (lane == 0) {
            const uint32_t rows = min(C::BN, room - i * C::BN);
            const int64_t row = row0 + i * C::BN;
            mbar_arrive_expect_tx(bar_k, rows * (C::ROWB + 4));
            bulk_load(ring + C::OFF_K, p.codes[0] + row * C::ROWB, rows * C::ROWB, bar_k);
            bulk_load(ring + C::OFF_WORDS, p.words[0] + row, rows * 2, bar_k);
            bulk_load(ring + C::OFF_WORDS + C::WORDB, p.words[1] + row, rows * 2, bar_k);
        }
    };
    auto load_v = [&](int i) {
        if (lane == 0) {            // rows past the cache's room come as zeros
            mbar_arrive_expect_tx(bar_v, C::TILE);
            tma_load_3d(ring, tm_v, bar_v, 0, (first + i) * (C::TILE / 128), b * p.Hkv + hk);
        }
    };
    // this lane's row for ldmatrix (its first 16-byte chunk; two chunks on the
    // address differs in bit 5): the tile lies in 128-byte lines of 2 or 4 keys,
    // whose chunks are exchanged by the line's index
    constexpr int KPL = 128 / C::ROWB;                       // keys a line
    const int v_key = kv4_v_key(lane & 15);
    const uint32_t v_at = smem_u32(ring) + v_key / KPL * 128 +
                          ((((v_key % KPL) * (8 / KPL)) | (lane >> 4)) ^ (v_key / KPL)) * 16;
    const int kkey = kv4_key(g8);
    // the keys of the lane's code pairs in the second product: these two and the
    // two that are 4 further
    const uint16_t* zv_at = zv + (t4 >> 1) * 8 + (t4 & 1) * 2;
    if (count > 0) {
        if (!p.fault_skip) load_k(0);
        load_v(0);
    }

    // ------------------------------------- queries as B fragments --
    // Row nt * 8 + g8, channels t4 * D/4 ..: of word w (8 codes), pair u of
    // k-step pairs: codes (2u, 2u + 4) plain and (2u + 1, 2u + 5) times 1/16.
    constexpr int W = D / 32;
    uint32_t qf[NT][W][2][2];
    float2 sq[NT], rf[NT];          // of rows nt * 8 + 2 t4 + {0, 1}: sum of q and the score factor
    int hi[NT][2], lo[NT][2];       // their allowed keys are [lo, hi)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int rr = nt * 8 + g8;
        uint4 raw[W];
        const bool have = rr < nrows;
        const int qi = (r0 + rr) / p.G;
        const size_t qrow = have ? (static_cast<size_t>(b) * p.Nq + qi) * p.H + hk * p.G + (r0 + rr) - qi * p.G : 0;
#pragma unroll
        for (int w = 0; w < W; ++w)
            raw[w] = have ? *reinterpret_cast<const uint4*>(p.q + qrow * D + t4 * (D / 4) + w * 8) : make_uint4(0, 0, 0, 0);
        uint32_t top = 0;           // largest magnitude, as bf16 bits (NaN and infinity on top)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7fffu, (v[j] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top >> 7), 14);             // biased exponent
        const float qs = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);   // 2^(14 - (e - 127))
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f[8] = {bf16_lo(raw[w].x) * qs, bf16_hi(raw[w].x) * qs, bf16_lo(raw[w].y) * qs,
                                bf16_hi(raw[w].y) * qs, bf16_lo(raw[w].z) * qs, bf16_hi(raw[w].z) * qs,
                                bf16_lo(raw[w].w) * qs, bf16_hi(raw[w].w) * qs};
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += f[j];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                qf[nt][w][u][0] = pack_f16(f[2 * u], f[2 * u + 4]);
                qf[nt][w][u][1] = pack_f16(f[2 * u + 1] * 0.0625f, f[2 * u + 5] * 0.0625f);
            }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // a query with NaN or infinity has NaN scores (through its sum; the factor
        // stays finite), which the masks replace: without a key it has O = 0
        sum = e >= 255 ? NAN : sum * -5.9604644775390625e-8f;          // -2^-24, as the codes
        const float f = e >= 255 ? 1.f : ldexpf(p.scale_log2, e - 117);    // / (qs 2^-24)
        sq[nt].x = __shfl_sync(0xffffffffu, sum, 8 * t4);
        sq[nt].y = __shfl_sync(0xffffffffu, sum, 8 * t4 + 4);
        rf[nt].x = __shfl_sync(0xffffffffu, f, 8 * t4);
        rf[nt].y = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int qp = qpos0 + (r0 + min(nt * 8 + 2 * t4 + j, nrows - 1)) / p.G;
            hi[nt][j] = kv4_key_hi(qp, nk, p.causal);
            lo[nt][j] = kv4_key_lo(qp, p.window);
        }
    }
    const int qp_first = qpos0 + r0 / p.G, qp_last = qpos0 + (r0 + nrows - 1) / p.G;

    float2 (&oacc)[D / 16][NT][2] = acc.o;
    float2 (&za)[NT][2] = acc.za;
    float2 (&l)[NT] = acc.l, (&nm)[NT] = acc.nm;
    // O and za of a nt times f
    auto scale_rows = [&](int nt, float2 f) {
        za[nt][0] = fmul2(za[nt][0], f);
        za[nt][1] = fmul2(za[nt][1], f);
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
            oacc[m][nt][0] = fmul2(oacc[m][nt][0], f);
            oacc[m][nt][1] = fmul2(oacc[m][nt][1], f);
        }
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int m = 0; m < D / 16; ++m) oacc[m][nt][0] = oacc[m][nt][1] = make_float2(0.f, 0.f);
        l[nt] = za[nt][0] = za[nt][1] = make_float2(0.f, 0.f);
        nm[nt] = make_float2(kNoRef, kNoRef);
    }
    uint32_t& ev = acc.ev;
    ev = 6;
    uint32_t low = 0xffffu;         // the smallest V word so far
    bool& wide = acc.wide;
    wide = false;
    Kv4RowScale* rows = reinterpret_cast<Kv4RowScale*>(ring + C::OFF_ROWS) + 2 * t4;    // of this lane's rows

    for (int i = 0; i < count; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_k, phase, wc))) return false;
        const uint8_t* st = ring + C::OFF_K;
        const int k0 = (first + i) * C::BN;

        // ---- scales and zeros: a key a lane
        const bool masked = kv4_tile_masked(k0, C::BN, nk, qp_first, qp_last, p.causal, p.window);
        {
            const uint16_t* ws = reinterpret_cast<const uint16_t*>(ring + C::OFF_WORDS);
            uint32_t wk[C::BN / 32], wv[C::BN / 32], top = 0, bot = 0xffffu;
#pragma unroll
            for (int kk = 0; kk < C::BN / 32; ++kk) {
                wk[kk] = ws[kk * 32 + lane];
                wv[kk] = ws[C::BN + kk * 32 + lane];
                // rows that no query sees may hold anything
                if (masked && kv4_unseen(k0 + kk * 32 + lane, nk, qp_first, qp_last, p.causal, p.window))
                    wv[kk] = kKv4Unseen;
                if (wv[kk] != kKv4Unseen) {
                    top = max(top, wv[kk]);
                    bot = min(bot, wv[kk]);
                }
            }
            if (__any_sync(0xffffffffu, top >= (ev + 1) << 7 || bot < low)) {
                // a larger or a smaller scale than any before, or a NaN
                top = 0;
                bot = low;
#pragma unroll
                for (int kk = 0; kk < C::BN / 32; ++kk) {
                    if (wv[kk] == kKv4Unseen) continue;
                    if (wv[kk] >= 0x7f80u) {        // acts through the row's score
                        wk[kk] = kKv4NaN;
                        wv[kk] = kKv4Unseen;
                        continue;
                    }
                    top = max(top, wv[kk]);
                    bot = min(bot, wv[kk]);
                }
                top = __reduce_max_sync(0xffffffffu, top) >> 7;
                low = __reduce_min_sync(0xffffffffu, bot);
                if (!wide && static_cast<int>(max(top, ev)) - static_cast<int>(low >> 7) > kKv4Spread) {
                    // from here on a power for each row; its largest w so far, if
                    // it has met a key, is about that of the largest scale
                    wide = true;
                    if (g8 == 0) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float w = ldexpf(1.f, static_cast<int>(ev) - 135);
                            const int k = 141 - static_cast<int>(ev);
                            rows[nt * 8] = {w, nm[nt].x, k};
                            rows[nt * 8 + 1] = {w, nm[nt].y, k};
                        }
                    }
                    ev = 141;           // units of 2^8
                }
                if (!wide && top > ev) {        // O goes down with the new factor
                    const float d = __uint_as_float((127u - min(top - ev, 127u)) << 23);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) scale_rows(nt, make_float2(d, d));
                    ev = top;
                }
            }
            const float vnorm = __uint_as_float((260u - ev) << 23);     // 2^(6 - (ev - 127))
#pragma unroll
            for (int kk = 0; kk < C::BN / 32; ++kk) {
                sck[kk * 32 + lane] = make_float2(__uint_as_float((wk[kk] & 0xfff0u) << 16),
                                                  __uint_as_float(0x4b000000u | (wk[kk] & 15u)) - 8388608.f);
                scv[kk * 32 + lane] = __uint_as_float((wv[kk] & 0xfff0u) << 16) * vnorm;
                zv[kk * 32 + lane] = static_cast<uint16_t>(wv[kk] & 15u);       // fp16: z 2^-24, as the codes
            }
        }
        __syncwarp();

        // ---- scores, and p = 2^(x - reference).  A lane's sum over the tile tells
        // when a score has passed the reference by so much that p s^v could
        // leave fp16: then the scores are formed again (they are not kept), the
        // reference moves to their maximum, and p is taken anew.
        float2 e[C::MT][NT][2], ts[NT];
        for (bool move = false;; move = true) {
            float2 (&s)[C::MT][NT][2] = e;
            // ---- S^T = C^k q^T: keys x 8 NT rows
#pragma unroll
            for (int m = 0; m < C::MT; ++m) {
                uint32_t ka[W], kb[W];
                const uint8_t* ra = st + (m * 16 + kkey) * C::ROWB + t4 * (W * 4);
                const uint8_t* rb = ra + 4 * C::ROWB;
                if constexpr (D == 128) {
                    const uint4 u = *reinterpret_cast<const uint4*>(ra), v = *reinterpret_cast<const uint4*>(rb);
                    ka[0] = u.x; ka[1] = u.y; ka[2] = u.z; ka[3] = u.w;
                    kb[0] = v.x; kb[1] = v.y; kb[2] = v.z; kb[3] = v.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(ra), v = *reinterpret_cast<const uint2*>(rb);
                    ka[0] = u.x; ka[1] = u.y;
                    kb[0] = v.x; kb[1] = v.y;
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t u = ka[w], v = kb[w], u8 = u >> 8, v8 = v >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (w == 0)
                            mma_f16_first(s[m][nt], u & kNibLo, v & kNibLo, u & kNibHi, v & kNibHi, qf[nt][w][0][0],
                                          qf[nt][w][0][1]);
                        else
                            mma_f16(s[m][nt], u & kNibLo, v & kNibLo, u & kNibHi, v & kNibHi, qf[nt][w][0][0],
                                    qf[nt][w][0][1]);
                        mma_f16(s[m][nt], u8 & kNibLo, v8 & kNibLo, u8 & kNibHi, v8 & kNibHi, qf[nt][w][1][0],
                                qf[nt][w][1][1]);
                    }
                }
            }
            // ---- scores (over the row factor rf) and masks
#pragma unroll
            for (int m = 0; m < C::MT; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float2 sz = sck[m * 16 + half * 4 + kkey];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        s[m][nt][half] = fmul2(ffma2(make_float2(sz.y, sz.y), sq[nt], s[m][nt][half]),
                                               make_float2(sz.x, sz.x));
                }
            if (masked) {
#pragma unroll
                for (int m = 0; m < C::MT; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int key = k0 + m * 16 + half * 4 + kkey;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (key >= hi[nt][0] || key < lo[nt][0]) s[m][nt][half].x = kNegInf;
                            if (key >= hi[nt][1] || key < lo[nt][1]) s[m][nt][half].y = kNegInf;
                        }
                    }
            }

            if (move) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float2 mx = s[0][nt][0];
#pragma unroll
                    for (int m = 0; m < C::MT; ++m)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            mx.x = fmaxf(mx.x, s[m][nt][half].x);
                            mx.y = fmaxf(mx.y, s[m][nt][half].y);
                        }
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) {
                        mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, o));
                        mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, o));
                    }
                    // the reference never falls; -inf (nothing yet) leaves none
                    float2 n2 = fmul2(mx, make_float2(-rf[nt].x, -rf[nt].y));
                    n2 = make_float2(fminf(n2.x, nm[nt].x), fminf(n2.y, nm[nt].y));
                    const float2 a = make_float2(nm[nt].x == kNoRef ? 0.f : ex2(n2.x - nm[nt].x),
                                                 nm[nt].y == kNoRef ? 0.f : ex2(n2.y - nm[nt].y));
                    nm[nt] = n2;
                    l[nt] = fmul2(l[nt], a);
                    scale_rows(nt, a);
                }
            }
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                ts[nt] = make_float2(0.f, 0.f);
#pragma unroll
                for (int m = 0; m < C::MT; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float2 y = ffma2(s[m][nt][half], rf[nt], nm[nt]);
                        e[m][nt][half] = make_float2(ex2(y.x), ex2(y.y));
                        ts[nt] = fadd2(ts[nt], e[m][nt][half]);
                    }
                over = over || ts[nt].x > kKv4Over || ts[nt].y > kKv4Over;
            }
            if (move || !__any_sync(0xffffffffu, over)) break;
        }
        __syncwarp();               // K may be loaded again
        if (i + 1 < count) load_k(i + 1);
        if (__builtin_expect(wide, 0)) {
            // ---- each row's power: its largest w to [2^13, 2^14), p takes the power
            float2 mx[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mx[nt] = make_float2(0.f, 0.f);
#pragma unroll
                for (int m = 0; m < C::MT; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float sv = scv[m * 16 + half * 4 + kkey];
                        mx[nt].x = fmaxf(mx[nt].x, e[m][nt][half].x * sv);
                        mx[nt].y = fmaxf(mx[nt].y, e[m][nt][half].y * sv);
                    }
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) {
                    mx[nt].x = fmaxf(mx[nt].x, __shfl_xor_sync(0xffffffffu, mx[nt].x, o));
                    mx[nt].y = fmaxf(mx[nt].y, __shfl_xor_sync(0xffffffffu, mx[nt].y, o));
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                Kv4RowScale r[2] = {rows[nt * 8], rows[nt * 8 + 1]};
                r[0].take(mx[nt].x, nm[nt].x);
                r[1].take(mx[nt].y, nm[nt].y);
                const int k[2] = {kv4_row_power(r[0]), kv4_row_power(r[1])};
                const int up[2] = {k[0] - r[0].k, k[1] - r[1].k};
                if (__any_sync(0xffffffffu, up[0] != 0 || up[1] != 0)) {      // in two steps, up to 2^+-250
                    scale_rows(nt, make_float2(kv4_pow2(up[0] / 2), kv4_pow2(up[1] / 2)));
                    scale_rows(nt, make_float2(kv4_pow2(up[0] - up[0] / 2), kv4_pow2(up[1] - up[1] / 2)));
                }
#pragma unroll
                for (int m = 0; m < C::MT; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        e[m][nt][half] = fmul2(e[m][nt][half], make_float2(kv4_pow2(k[0]), kv4_pow2(k[1])));
                __syncwarp();
                if (g8 == 0) {
                    rows[nt * 8] = {r[0].largest, r[0].minus_ref, k[0]};
                    rows[nt * 8 + 1] = {r[1].largest, r[1].minus_ref, k[1]};
                }
            }
        }
        // ---- p s^v as the B fragments of the second product
        uint32_t pf[C::MT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) l[nt] = fadd2(l[nt], ts[nt]);
#pragma unroll
        for (int m = 0; m < C::MT; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float sv = scv[m * 16 + half * 4 + kkey];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 w = fmul2(e[m][nt][half], make_float2(sv, sv));
                    pf[m][nt][half] = transpose8x8(pack_f16(w.x, w.y));
                }
            }
        // ---- za += Z (p s^v)^T: the zeros, at the places of a byte's low code and
        // of its high one, so that the products lose the same as those of O
#pragma unroll
        for (int m = 0; m < C::MT; ++m) {
            const uint32_t z0 = *reinterpret_cast<const uint32_t*>(zv_at + m * 16);
            const uint32_t z1 = *reinterpret_cast<const uint32_t*>(zv_at + m * 16 + 4);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(za[nt], z0, z0 << 4, z1, z1 << 4, pf[m][nt][0], pf[m][nt][1]);
        }
        // ---- O^T += C^v (p s^v)^T
        if (!__all_sync(0xffffffffu, mbar_wait(bar_v, phase, wc))) return false;
#pragma unroll
        for (int m = 0; m < C::MT; ++m)
#pragma unroll
            for (int c2 = 0; c2 < D / 64; ++c2) {          // two chunks of 16 bytes
                uint32_t v[4];
                load_transposed(v, (v_at ^ ((c2 ? 32u : 0u) | (D == 64 && (m & 1) ? 64u : 0u))) + m * 16 * C::ROWB);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t u = v[k], u8 = u >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(oacc[c2 * 4 + k][nt], u & kNibLo, u & kNibHi, u8 & kNibLo, u8 & kNibHi, pf[m][nt][0],
                                pf[m][nt][1]);
                }
            }
        __syncwarp();               // and V
        if (i + 1 < count) load_v(i + 1);
        phase ^= 1;
    }

    return true;
}

// Hands each of the warp's query rows to put(row, values, reference, sum): a
// lane has channels 16 m + 2 g8 + {0, 1}, m < D / 16, of two rows of each nt.
// O is left as it is (relative to the reference).
template <int D, int NT, typename Put>
__device__ __forceinline__ void kv4_each_row(Kv4Acc<D, NT>& acc, const uint8_t* ring, int nrows, const Put& put) {
    const int t4 = lane_id() & 3;
    const Kv4RowScale* rows = reinterpret_cast<const Kv4RowScale*>(ring + Kv4DecCfg<D, NT>::OFF_ROWS);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
            acc.l[nt].x += __shfl_xor_sync(0xffffffffu, acc.l[nt].x, o);
            acc.l[nt].y += __shfl_xor_sync(0xffffffffu, acc.l[nt].y, o);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = nt * 8 + 2 * t4 + j;
            if (r >= nrows) continue;
            // undoes vnorm, and the row's power
            const float back = ldexpf(1.f, static_cast<int>(acc.ev) - 133 - (acc.wide ? rows[r].k : 0));
            const float z0 = j ? acc.za[nt][0].y : acc.za[nt][0].x, z1 = j ? acc.za[nt][1].y : acc.za[nt][1].x;
            const float n1 = j ? acc.nm[nt].y : acc.nm[nt].x;
            float a[D / 8];
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {      // codes times 2^-24, and 2^-20
                a[2 * m] = ((j ? acc.o[m][nt][0].y : acc.o[m][nt][0].x) - z0) * 16777216.f * back;
                a[2 * m + 1] = ((j ? acc.o[m][nt][1].y : acc.o[m][nt][1].x) - z1) * 1048576.f * back;
            }
            put(r, a, n1 == kNoRef ? -INFINITY : -n1, j ? acc.l[nt].y : acc.l[nt].x);
        }
    }
}

// After a wait that gave up: lets the copies in flight land before the CTA exits.
__device__ __forceinline__ void kv4_drain(uint64_t* bar_k, uint32_t phase, int* error_word) {
    if (lane_id() == 0) {
        volatile int no_abort = 0;
        const WaitCtl dw{&no_abort, error_word, 200000000ull};
        mbar_wait(bar_k, phase, dw);
        mbar_wait(bar_k, phase ^ 1, dw);        // the next tile's K, where V gave up
        mbar_wait(bar_k + 1, phase, dw);
    }
}

// ------------------------------------------------ few tiles: a cluster an item --
// An item (sequence, kv head, block of query rows) to each cluster of CTAs, its
// tiles in equal parts to the warps of the cluster.  The warps of a CTA put
// their results together in shared memory, the CTAs in distributed shared
// memory: no second kernel and no workspace.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 4 bytes of the shared memory of the cluster's CTA `rank`, at this CTA's address `p`.
__device__ __forceinline__ float cluster_load(const float* p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <int D, int NT>
__global__ void __launch_bounds__(Kv4DecCfg<D, NT>::WARPS * 32, Kv4DecCfg<D, NT>::MIN_CTAS)
kv4_cluster_kernel(const __grid_constant__ CUtensorMap tm_v, const Kv4DecodeParams p) {
    using C = Kv4DecCfg<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem_1024(smem_raw);
    const int warp = threadIdx.x >> 5, lane = lane_id(), g8 = lane >> 2;
    const int ctas = cluster_size(), rank = cluster_rank();
    uint64_t* bar_k = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * 2;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    if (lane == 0) {
        mbar_init(bar_k, 1);
        mbar_init(bar_k + 1, 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) *abort_flag = 0;
    const int per = p.Hkv * p.row_blocks;
    const int id = blockIdx.x / ctas;
    const int b = id / per, item = id - b * per, hk = item / p.row_blocks;
    const int r0 = (item - hk * p.row_blocks) * C::ROWS, nrows = min(C::ROWS, p.Nq * p.G - r0);
    const Kv4Span sp = kv4_span<C::BN>(p, b);
    const int all = ctas * C::WARPS, me = rank * C::WARPS + warp;
    const int t0 = static_cast<int>(static_cast<int64_t>(sp.n) * me / all);
    const int t1 = static_cast<int>(static_cast<int64_t>(sp.n) * (me + 1) / all);
    __syncthreads();
    const WaitCtl wc{abort_flag, p.error_word, p.timeout_ns};
    uint32_t phase = 0;
    Kv4Acc<D, NT> acc;
    const bool ok = kv4_attend<D, NT>(p, &tm_v, acc, smem + warp * C::WARP_BYTES, bar_k, phase, wc, b, hk, r0, nrows, sp.nk,
                                      sp.t0 + t0, t1 - t0);
    if (!ok) kv4_drain(bar_k, phase, p.error_word);
    auto partial = [&](int w) { return reinterpret_cast<float*>(smem + w * C::WARP_BYTES); };   // [ROWS][OSTRIDE]
    auto stats = [&](int w) { return partial(w) + C::ROWS * C::OSTRIDE; };                      // [ROWS][2]
    kv4_each_row<D, NT>(acc, smem + warp * C::WARP_BYTES, nrows, [&](int r, const float (&a)[D / 8], float ref, float l) {
        float2* dst = reinterpret_cast<float2*>(partial(warp) + r * C::OSTRIDE + 2 * g8);
#pragma unroll
        for (int m = 0; m < D / 16; ++m) dst[8 * m] = make_float2(a[2 * m], a[2 * m + 1]);
        if (g8 == 0) *reinterpret_cast<float2*>(stats(warp) + 2 * r) = make_float2(ref, l);
    });
    __syncthreads();
    constexpr int V = D / 32;
    for (int r = warp; r < nrows; r += C::WARPS) {
        Kv4Row<D> sum;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w)
            sum.take(make_float2(stats(w)[2 * r], stats(w)[2 * r + 1]), partial(w) + r * C::OSTRIDE + lane * V);
        if (ctas == 1) {
            sum.store(p, b, hk, r0 + r);
        } else {            // over warp 0's row, which no other warp reads
            __syncwarp();
#pragma unroll
            for (int e = 0; e < V; ++e) partial(0)[r * C::OSTRIDE + lane * V + e] = sum.a[e];
            if (lane == 0) *reinterpret_cast<float2*>(stats(0) + 2 * r) = make_float2(sum.M, sum.L);
        }
    }
    if (ctas == 1) return;
    cluster_barrier();
    for (int r = me; r < nrows; r += all) {
        Kv4Row<D> sum;
        for (int c = 0; c < ctas; ++c) {
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = cluster_load(partial(0) + r * C::OSTRIDE + lane * V + e, c);
            sum.take(make_float2(cluster_load(stats(0) + 2 * r, c), cluster_load(stats(0) + 2 * r + 1, c)), v);
        }
        sum.store(p, b, hk, r0 + r);
    }
    cluster_barrier();      // the CTAs' memory stays until all have read it
}

// ------------------------------------------------------ many tiles: ranges --
// The work is the sequence of all key tiles of all items, `per` items to a
// sequence.  Sequences differ in length, and only the device knows them, so the
// tiles are cut into equal ranges, one a warp; a range's ends may lie inside an
// item, which then has partial results: that of the item's first tiles in slot 1
// of their range, all others in slot 0 of theirs (a range has at most one each).
// To start an item (queries, first loads, a partial result) takes a warp about
// as long as a tile, so an item counts for kKv4Start tiles more than it has, and
// its first tiles are such as have no keys.  32 requests of 0 to 8192 rows, 32
// heads over 8, d 128: 32.8 us (34.1 without, 33.1 with two).
constexpr int kKv4Start = 1;
__device__ __forceinline__ int kv4_weight(int n) { return n > 0 ? n + kKv4Start : 0; }

// The cut of `total` tiles (below 2^31) into ranges of q or, the first rem,
// q + 1 tiles; fewer ranges than p.ranges when there are fewer tiles.
struct Kv4Cut {
    int ranges, q, rem;
    __device__ __forceinline__ Kv4Cut(const Kv4DecodeParams& p, int total) {
        ranges = max(1, min(p.ranges, total));
        q = total / ranges;
        rem = total - q * ranges;
    }
    __device__ __forceinline__ int start(int c) const { return c * q + min(c, rem); }
    __device__ __forceinline__ int range_of(int x) const {
        const int cut = rem * (q + 1);
        return x < cut ? x / (q + 1) : rem + (x - cut) / q;
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(Kv4DecCfg<D, NT>::WARPS * 32, Kv4DecCfg<D, NT>::MIN_CTAS)
kv4_decode_kernel(const __grid_constant__ CUtensorMap tm_v, const Kv4DecodeParams p) {
    using C = Kv4DecCfg<D, NT>;
    // the merge launched after this grid may be scheduled now
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem_1024(smem_raw);
    const int warp = threadIdx.x >> 5, lane = lane_id(), g8 = lane >> 2;
    const int per = p.Hkv * p.row_blocks;
    uint64_t* bar_k = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * 2;
    int* sh_b = reinterpret_cast<int*>(smem + C::OFF_MISC);
    int* sh_base = sh_b + C::WARPS;
    int* sh_sum = sh_base + C::WARPS;
    volatile int* abort_flag = sh_sum + C::WARPS;
    if (lane == 0) {
        mbar_init(bar_k, 1);
        mbar_init(bar_k + 1, 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) *abort_flag = 0;

    // ---------------------------------------------- this warp's tiles --
    // tiles [x, x_end) of the sequence; b is the sequence of tile x and `base`
    // its first tile.  A thread looks at B / THREADS sequences.
    const int each = (p.B + C::WARPS * 32 - 1) / (C::WARPS * 32);
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * each), b1 = min(p.B, b0 + each);
    int sum = 0;
    for (int i = b0; i < b1; ++i) sum += kv4_weight(kv4_span<C::BN>(p, i).n);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh_sum[warp] = incl;
    __syncthreads();
    int total = 0, at = incl - sum;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
        if (w < warp) at += sh_sum[w];
        total += sh_sum[w];
    }
    total *= per;
    at *= per;
    const Kv4Cut cut(p, total);
    const int range = blockIdx.x * C::WARPS + warp;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
        const int xw = cut.start(blockIdx.x * C::WARPS + w);
        if (at <= xw && xw < at + sum * per) {
            int first = at;
            for (int i = b0; i < b1; ++i) {
                const int next = first + kv4_weight(kv4_span<C::BN>(p, i).n) * per;
                if (xw < next) {
                    sh_b[w] = i;
                    sh_base[w] = first;
                    break;
                }
                first = next;
            }
        }
    }
    __syncthreads();
    if (range >= cut.ranges || total == 0) return;      // from here on each warp is on its own
    int x = cut.start(range);
    const int x_end = cut.start(range + 1);
    int b = sh_b[warp];
    int base = sh_base[warp];
    const WaitCtl wc{abort_flag, p.error_word, p.timeout_ns};
    uint32_t phase = 0;
    while (x < x_end) {
        const Kv4Span sp = kv4_span<C::BN>(p, b);
        if (sp.n == 0) {
            ++b;
            continue;
        }
        const int weight = kv4_weight(sp.n);
        const int item = (x - base) / weight;
        const int at_item = x - base - item * weight;
        const int take = min(weight - at_item, x_end - x);
        const int tile0 = max(0, at_item - kKv4Start);
        const int count = max(0, at_item + take - kKv4Start) - tile0;
        x += take;
        const int seq = b;
        if (x - base == weight * per) {
            base = x;
            ++b;
        }
        if (count == 0) continue;
        const int hk = item / p.row_blocks;
        const int r0 = (item - hk * p.row_blocks) * C::ROWS, nrows = min(C::ROWS, p.Nq * p.G - r0);
        Kv4Acc<D, NT> acc;
        if (!kv4_attend<D, NT>(p, &tm_v, acc, smem + warp * C::WARP_BYTES, bar_k, phase, wc, seq, hk, r0, nrows, sp.nk,
                               sp.t0 + tile0, count)) {
            kv4_drain(bar_k, phase, p.error_word);
            return;
        }
        const bool whole = count == sp.n;
        kv4_each_row<D, NT>(acc, smem + warp * C::WARP_BYTES, nrows, [&](int r, const float (&a)[D / 8], float ref, float l) {
            if (whole) {
                const bool some = !(l == 0.f);      // a NaN sum stays NaN
                const float inv = some ? 1.f / l : 0.f;
                size_t lse_at;
                const size_t row = kv4_out_row(p, seq, hk, r0 + r, lse_at);
                uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + 2 * g8);
#pragma unroll
                for (int m = 0; m < D / 16; ++m) dst[8 * m] = pack_bf16(a[2 * m] * inv, a[2 * m + 1] * inv);
                if (g8 == 0) p.lse[lse_at] = some ? (ref + __log2f(l)) * 0.6931471805599453f : -INFINITY;
            } else {
                const size_t at_row = (static_cast<size_t>(range) * 2 + (tile0 == 0)) * C::ROWS + r;
                float2* dst = reinterpret_cast<float2*>(p.o_part + at_row * D + 2 * g8);
#pragma unroll
                for (int m = 0; m < D / 16; ++m) dst[8 * m] = make_float2(a[2 * m], a[2 * m + 1]);
                if (g8 == 0) p.ml_part[at_row] = make_float2(ref, l);
            }
        });
    }
}

// Merges the partial results of the items that lie in several ranges, and
// writes the outputs of sequences without keys.  A CTA to a query row; its
// warps share the ranges.
constexpr int kKv4MergeWarps = 16;      // at most

template <int D, int NT>
__global__ void __launch_bounds__(kKv4MergeWarps * 32)
kv4_merge_kernel(const Kv4DecodeParams p) {
    using C = Kv4DecCfg<D, NT>;
    constexpr int V = D / 32;                   // channels a lane
    constexpr int AHEAD = 4;                    // partials read at once
    __shared__ float sm_a[kKv4MergeWarps][D];
    __shared__ float2 sm_ml[kKv4MergeWarps];
    const int lane = lane_id(), warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int per = p.Hkv * p.row_blocks;
    const int rows = p.Nq * p.G;
    const int r = blockIdx.x % rows, bh = blockIdx.x / rows;
    const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
    const int item = hk * p.row_blocks + r / C::ROWS;
    int total = 0, at = 0;
    for (int i = lane; i < p.B; i += 32) {
        const int w = kv4_weight(kv4_span<C::BN>(p, i).n);
        total += w;
        if (i < b) at += w;
    }
    total = __reduce_add_sync(0xffffffffu, total) * per;
    at = __reduce_add_sync(0xffffffffu, at) * per;
    const int n = kv4_span<C::BN>(p, b).n;
    at += item * kv4_weight(n);
    const Kv4Cut cut(p, total);
    const int c0 = n > 0 ? cut.range_of(at + kKv4Start) : 0, c1 = n > 0 ? cut.range_of(at + kv4_weight(n) - 1) : 0;
    // launched as a programmatic dependent of the kernel above: from here on
    // its results are complete.  Every thread waits, so that this grid does not
    // end before that one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n > 0 && c0 == c1) return;              // written by the range's own warp
    Kv4Row<D> sum;
    if (n > 0) {
        auto slot = [&](int c) { return (static_cast<size_t>(c) * 2 + (c == c0)) * C::ROWS + r % C::ROWS; };
        for (int c = c0 + warp; c <= c1; c += AHEAD * warps) {
            float v[AHEAD][V];
            float2 ml[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const size_t from = slot(min(c + warps * i, c1));
                ml[i] = c + warps * i <= c1 ? p.ml_part[from] : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[i][e] = p.o_part[from * D + lane * V + e];
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) sum.take(ml[i], v[i]);
        }
        const int used = min(warps, c1 - c0 + 1);
#pragma unroll
        for (int e = 0; e < V; ++e) sm_a[warp][lane * V + e] = sum.a[e];
        if (lane == 0) sm_ml[warp] = make_float2(sum.M, sum.L);
        __syncthreads();
        if (warp != 0) return;
        for (int w = 1; w < used; ++w) sum.take(sm_ml[w], &sm_a[w][lane * V]);
    } else if (warp != 0) {
        return;
    }
    sum.store(p, b, hk, r);
}

}  // namespace fa
