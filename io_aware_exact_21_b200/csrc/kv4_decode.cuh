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
// Roundings: q is scaled by a power of two per row so that its largest
// element lies in [2^14, 2^15) and held in fp16, which is exact for elements
// down to 2^-24 of that one and off by 2^-25 of the row's largest below it;
// p s^v is scaled likewise by the largest s^v of the warp's keys so far and
// rounded to fp16 (2^-11; the two-byte operand the product needs, finer than
// bf16's 2^-8).  Everything else is fp32, the row sums take the unrounded p.
//
// What bounds it: with R = Nq * H / Hkv query rows to a key/value head the
// cache is D + 4 bytes a token and head for 4 R D operations, so up to a few
// dozen rows HBM is the limit if the instructions per code stay few.  mma.sync
// rather than tcgen05: its operands come from registers, where the codes are
// unpacked, while tcgen05 would have them written back to shared or tensor
// memory as 16-bit words first, four times the cache's bytes.
//
// One warp is on its own: it takes every WARPS-th tile of 32 keys of the
// CTA's range through its own ring of cp.async stages, with its own running
// maximum and sums, so the key loop has no CTA barrier; the warps' results
// merge once at the end, the splits' in combine_kernel.
//
// Per tile: S^T = C^k q^T with 16 keys x 8 query rows to an mma (the codes are
// the A operand), p from it in registers, transposed by movmatrix into the B
// operand of O^T += C^v p^T, whose A operand pairs two keys' codes by byte
// permutes.  Which channel sits at which mma index is free as long as q (or
// the store of O) agrees, so each lane reads whole words of codes: for K the
// D/4 channels of lane % 4, for V the D/8 channels of lane / 4.
#pragma once

#include "decode_kernel.cuh"
#include "kv4_rows.cuh"

namespace fa {

struct Kv4DecodeParams {
    const __nv_bfloat16* q;      // [B, Nq, H, D]
    const uint8_t* codes[2];     // K, V: [B, Hkv, Nk, D / 2]
    const uint16_t* words[2];    // [B, Hkv, Nk]
    __nv_bfloat16* o;            // [B, Nq, H, D]
    float* lse;                  // [B, H, Nq]
    float* o_part;               // nsplit > 1: [nsplit, B * Nq, H, D]
    float* lse_part;             // nsplit > 1: [nsplit, H, B * Nq], base 2
    const int* seqlens_k;        // [B] or nullptr
    int B, H, Hkv, G, Nq, Nk;    // G = H / Hkv
    int causal, window, nsplit, row_blocks;
    float scale_log2;
};

template <int D, int NT>
struct Kv4DecCfg {
    static constexpr int BN = 32;                         // keys a tile
    static constexpr int ROWS = 8 * NT;                   // query rows a CTA
    static constexpr int WARPS = NT == 1 ? 8 : 4;
    static constexpr int MIN_CTAS = NT == 1 ? 2 : 3;
    static constexpr int NSTAGE = 3;
    static constexpr int ROWB = D / 2;                    // bytes of a row's codes
    static constexpr int TILE = BN * ROWB;                // K or V codes of a tile
    static constexpr int WORDB = BN * 2;
    static constexpr int STAGE = 2 * TILE + 2 * WORDB;
    static constexpr int RING = NSTAGE * STAGE;           // a warp's
    static constexpr int SCALES = 2 * BN * 8;             // a warp's (scale, zero) of K and V
    static constexpr int OFF_SCALES = WARPS * RING;
    static constexpr int OFF_STATS = OFF_SCALES + WARPS * SCALES;   // max and sum [WARPS][ROWS]
    static constexpr int SMEM = OFF_STATS + 2 * WARPS * ROWS * 4;
    static constexpr int OSTRIDE = D + 4;                 // floats a row of the merge area
    static_assert(WARPS * ROWS * OSTRIDE * 4 <= OFF_STATS, "the merge reuses ring and scales");
    static_assert(STAGE % 16 == 0, "16-byte copies");
};

// 16 bytes of shared memory from global memory, `bytes` of them copied and the
// rest zero (0: nothing is read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Shared-memory row of key k (0 .. 31) of a V tile.  The PV product wants keys
// 2t, 2t + 1, 2t + 8, 2t + 9 on lane t of each four; this order (with 16-byte
// chunks exchanged in every other pair of 64-byte rows) makes the four lanes'
// reads of one of them fall into different banks.
__device__ __forceinline__ int kv4_v_row(int k) {
    return (k & 24) | ((k & 1) << 2) | ((k >> 1) & 3);
}
template <int D>
__device__ __forceinline__ int kv4_v_chunk(int row, int chunk) {
    return D == 128 ? chunk ^ (row & 2) : chunk;
}

template <int D, int NT>
__global__ void __launch_bounds__(Kv4DecCfg<D, NT>::WARPS * 32, Kv4DecCfg<D, NT>::MIN_CTAS)
kv4_decode_kernel(const Kv4DecodeParams p) {
    using C = Kv4DecCfg<D, NT>;
    // the merge launched after this grid may be scheduled now
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = lane_id();
    const int g8 = lane >> 2, t4 = lane & 3;
    const float kNegInf = -INFINITY;

    // CTA = (sequence, kv head, split, block of query rows), the last fastest
    int id = blockIdx.x;
    const int rb = id % p.row_blocks;
    id /= p.row_blocks;
    const int split = id % p.nsplit;
    id /= p.nsplit;
    const int hk = id % p.Hkv;
    const int b = id / p.Hkv;
    const int r0 = rb * C::ROWS;                          // first of the CTA's query rows
    const int nrows = min(C::ROWS, p.Nq * p.G - r0);
    const int nk = p.seqlens_k ? min(max(p.seqlens_k[b], 0), p.Nk) : p.Nk;
    const int qpos0 = nk - p.Nq;                          // key position of query 0
    const int rows_q = p.B * p.Nq;

    int tb = 0, te = 0;
    if (!decode_split_range(nk, p.Nq, p.causal, p.window, C::BN, p.nsplit, split, tb, te)) {
        for (int e = threadIdx.x; e < nrows; e += C::WARPS * 32) {
            const int i = (r0 + e) / p.G, h = hk * p.G + (r0 + e) % p.G;
            if (p.nsplit > 1)
                p.lse_part[(static_cast<size_t>(split) * p.H + h) * rows_q + b * p.Nq + i] = kNegInf;
            else
                p.lse[(static_cast<size_t>(b) * p.H + h) * p.Nq + i] = kNegInf;
        }
        if (p.nsplit == 1)
            for (int e = threadIdx.x; e < nrows * (D / 8); e += C::WARPS * 32) {
                const int r = r0 + e / (D / 8);
                const size_t row = (static_cast<size_t>(b) * p.Nq + r / p.G) * p.H + hk * p.G + r % p.G;
                *reinterpret_cast<uint4*>(p.o + row * D + (e % (D / 8)) * 8) = make_uint4(0, 0, 0, 0);
            }
        return;
    }

    // -------------------------------------------------- the warp's ring --
    const size_t head = static_cast<size_t>(b) * p.Hkv + hk;
    const uint8_t* kc = p.codes[0] + head * p.Nk * C::ROWB;
    const uint8_t* vc = p.codes[1] + head * p.Nk * C::ROWB;
    const uint16_t* kw = p.words[0] + head * p.Nk;
    const uint16_t* vw = p.words[1] + head * p.Nk;
    uint8_t* ring = smem + warp * C::RING;
    const uint32_t ring_a = smem_u32(ring);
    auto load_tile = [&](int tile, int slot) {
        const int k0 = tile * C::BN;
        const uint32_t dst = ring_a + slot * C::STAGE;
        constexpr int CH = C::ROWB / 16;                  // 16-byte chunks a row
#pragma unroll
        for (int j = 0; j < C::BN * CH / 32; ++j) {
            const int idx = lane + 32 * j;
            const int key = idx / CH, chunk = idx % CH;
            const int bytes = k0 + key < nk ? 16 : 0;
            const size_t off = bytes ? static_cast<size_t>(k0 + key) * C::ROWB + chunk * 16 : 0;
            cp_async16(dst + idx * 16, kc + off, bytes);
            const int vr = kv4_v_row(key);
            cp_async16(dst + C::TILE + vr * C::ROWB + kv4_v_chunk<D>(vr, chunk) * 16, vc + off, bytes);
        }
        if (lane < 8) {                                   // words: 8 keys a copy, K on lanes 0-3, V on 4-7
            const int key = (lane & 3) * 8;
            const int bytes = max(0, min(16, 2 * (nk - k0 - key)));
            const uint16_t* src = (lane < 4 ? kw : vw) + (bytes ? k0 + key : 0);
            cp_async16(dst + 2 * C::TILE + (lane >> 2) * C::WORDB + key * 2, src, bytes);
        }
    };
    const int first = tb + warp;
    const int ntile = first < te ? (te - first + C::WARPS - 1) / C::WARPS : 0;
#pragma unroll
    for (int s = 0; s < C::NSTAGE - 1; ++s) {
        if (s < ntile) load_tile(first + s * C::WARPS, s);
        cp_async_commit();
    }

    // ----------------------------------------- queries as B fragments --
    // Row nt * 8 + g8, channels t4 * D/4 ..: of word w (8 codes), pair u of
    // k-step pairs: codes (2u, 2u + 4) plain and (2u + 1, 2u + 5) times 1/16.
    constexpr int W = D / 32;
    uint32_t qf[NT][W][2][2];
    float sq[NT][2], rf[NT][2];     // of rows nt * 8 + 2 t4 + {0, 1}: sum of q and the score factor
    int hi[NT][2], lo[NT][2];       // their allowed keys are [lo, hi)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int rr = nt * 8 + g8;
        uint4 raw[W];
        const bool have = rr < nrows;
        const size_t qrow = have ? (static_cast<size_t>(b) * p.Nq + (r0 + rr) / p.G) * p.H + hk * p.G + (r0 + rr) % p.G : 0;
#pragma unroll
        for (int w = 0; w < W; ++w)
            raw[w] = have ? *reinterpret_cast<const uint4*>(p.q + qrow * D + t4 * (D / 4) + w * 8) : make_uint4(0, 0, 0, 0);
        uint32_t top = 0;               // largest magnitude, as bf16 bits (NaN and infinity on top)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t x[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(x[j] & 0x7fffu, (x[j] >> 16) & 0x7fffu));
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
        sum *= 5.9604644775390625e-8f;                                 // 2^-24, as the codes
        const float f = e >= 255 ? NAN : ldexpf(p.scale_log2, e - 117);    // / (qs 2^-24)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sq[nt][j] = __shfl_sync(0xffffffffu, sum, (2 * t4 + j) * 4);
            rf[nt][j] = __shfl_sync(0xffffffffu, f, (2 * t4 + j) * 4);
            const int r = nt * 8 + 2 * t4 + j;
            const int qp = qpos0 + (r0 + r) / p.G;
            hi[nt][j] = p.causal ? min(nk, qp + 1) : nk;
            lo[nt][j] = p.window > 0 ? max(0, qp - p.window + 1) : 0;
        }
    }
    const int qp_first = qpos0 + r0 / p.G, qp_last = qpos0 + (r0 + nrows - 1) / p.G;

    float oacc[D / 16][NT][4];
    float mu[NT][2], l[NT][2], za[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[m][nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            mu[nt][j] = kNegInf;
            l[nt][j] = 0.f;
            za[nt][j] = 0.f;
        }
    }
    uint32_t ev = 14;                   // biased exponent of the largest V scale so far
    float2* sck = reinterpret_cast<float2*>(smem + C::OFF_SCALES + warp * C::SCALES);
    float2* scv = sck + C::BN;

    for (int i = 0; i < ntile; ++i) {
        if (i + C::NSTAGE - 1 < ntile)
            load_tile(first + (i + C::NSTAGE - 1) * C::WARPS, (i + C::NSTAGE - 1) % C::NSTAGE);
        cp_async_commit();
        cp_async_wait<C::NSTAGE - 1>();
        __syncwarp();
        const uint8_t* st = ring + (i % C::NSTAGE) * C::STAGE;
        const int k0 = (first + i * C::WARPS) * C::BN;

        // ---- scales and zeros: lane = key
        float dscale;                   // 2^(old - new) exponent of the V scaling
        {
            const uint16_t* ws = reinterpret_cast<const uint16_t*>(st + 2 * C::TILE);
            uint32_t wk = ws[lane], wv = ws[C::BN + lane];
            if (wv >= 0x7f80u) {        // a row that holds NaN or infinity: it acts through its score
                wk = kKv4NaN;
                wv = 0;
            }
            const uint32_t e_new = max(ev, __reduce_max_sync(0xffffffffu, wv >> 7));
            dscale = __uint_as_float((127u - min(e_new - ev, 127u)) << 23);
            ev = e_new;
            const float vs = __uint_as_float((wv & 0xfff0u) << 16) * __uint_as_float((268u - ev) << 23);
            sck[lane] = make_float2(__uint_as_float((wk & 0xfff0u) << 16),
                                    __uint_as_float(0x4b000000u | (wk & 15u)) - 8388608.f);
            scv[lane] = make_float2(vs, __uint_as_float(0x4b000000u | (wv & 15u)) - 8388608.f);
        }
        __syncwarp();

        // ---- S^T = C^k q^T: 32 keys x 8 NT rows
        float s[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[m][nt][e] = 0.f;
            uint32_t ka[W], kb[W];
            const uint8_t* ra = st + (m * 16 + g8) * C::ROWB + t4 * (W * 4);
            const uint8_t* rbp = ra + 8 * C::ROWB;
            if constexpr (D == 128) {
                const uint4 a = *reinterpret_cast<const uint4*>(ra), bb = *reinterpret_cast<const uint4*>(rbp);
                ka[0] = a.x; ka[1] = a.y; ka[2] = a.z; ka[3] = a.w;
                kb[0] = bb.x; kb[1] = bb.y; kb[2] = bb.z; kb[3] = bb.w;
            } else {
                const uint2 a = *reinterpret_cast<const uint2*>(ra), bb = *reinterpret_cast<const uint2*>(rbp);
                ka[0] = a.x; ka[1] = a.y;
                kb[0] = bb.x; kb[1] = bb.y;
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t x = ka[w], y = kb[w], x8 = x >> 8, y8 = y >> 8;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(s[m][nt], x & kNibLo, y & kNibLo, x & kNibHi, y & kNibHi, qf[nt][w][0][0], qf[nt][w][0][1]);
                    mma_f16(s[m][nt], x8 & kNibLo, y8 & kNibLo, x8 & kNibHi, y8 & kNibHi, qf[nt][w][1][0], qf[nt][w][1][1]);
                }
            }
        }
        // ---- scores (over the row factor rf) and masks
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float2 sz = sck[m * 16 + half * 8 + g8];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        s[m][nt][half * 2 + j] = fmaf(-sz.y, sq[nt][j], s[m][nt][half * 2 + j]) * sz.x;
            }
        if (k0 + C::BN > nk || (p.causal && k0 + C::BN - 1 > qp_first) ||
            (p.window > 0 && k0 <= qp_last - p.window)) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = k0 + m * 16 + (e >> 1) * 8 + g8;
                        if (key >= hi[nt][e & 1] || key < lo[nt][e & 1]) s[m][nt][e] = kNegInf;
                    }
        }
        // ---- running maximum
        float alpha[NT][2];
        bool change = dscale != 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float mx = fmaxf(fmaxf(s[0][nt][j], s[0][nt][2 + j]), fmaxf(s[1][nt][j], s[1][nt][2 + j]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                alpha[nt][j] = 1.f;
                if (mx > mu[nt][j]) {
                    alpha[nt][j] = ex2((mu[nt][j] - mx) * rf[nt][j]);     // 0 from -inf
                    mu[nt][j] = mx;
                    change = true;
                }
            }
        if (__any_sync(0xffffffffu, change)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    l[nt][j] *= alpha[nt][j];
                    alpha[nt][j] *= dscale;
                    za[nt][j] *= alpha[nt][j];
                }
#pragma unroll
                for (int m = 0; m < D / 16; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) oacc[m][nt][e] *= alpha[nt][e & 1];
            }
        }
        // ---- p, and p s^v as the B fragments of the second product
        uint32_t pf[2][NT][2];
        float nm[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) nm[nt][j] = mu[nt][j] == kNegInf ? 0.f : -mu[nt][j] * rf[nt][j];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float2 sz = scv[m * 16 + half * 8 + g8];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float e = ex2(fmaf(s[m][nt][half * 2 + j], rf[nt][j], nm[nt][j]));
                        l[nt][j] += e;
                        w[j] = e * sz.x;
                        za[nt][j] = fmaf(w[j], sz.y, za[nt][j]);
                    }
                    pf[m][nt][half] = transpose8x8(pack_f16(w[0], w[1]));
                }
            }
        // ---- O^T += C^v (p s^v)^T
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            constexpr int VW = D / 64;                     // words of codes a lane and key
            uint32_t v[4][VW];                             // keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int row = m * 16 + (kk >> 1) * 8 + (kk & 1) * 4 + t4;     // kv4_v_row
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2*>(
                        st + C::TILE + row * C::ROWB + kv4_v_chunk<D>(row, g8 >> 1) * 16 + (g8 & 1) * 8);
                    v[kk][0] = x.x;
                    v[kk][VW - 1] = x.y;
                } else {
                    v[kk][0] = *reinterpret_cast<const uint32_t*>(st + C::TILE + row * C::ROWB + g8 * 4);
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int up = 0; up < 2; ++up) {           // codes 0-3, then 4-7 of the word
                    const uint32_t sel = up ? 0x7632u : 0x5410u;
                    const uint32_t x = __byte_perm(v[0][w], v[1][w], sel), y = __byte_perm(v[2][w], v[3][w], sel);
                    const uint32_t x8 = x >> 8, y8 = y >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(oacc[w * 4 + up * 2][nt], x & kNibLo, x & kNibHi, y & kNibLo, y & kNibHi,
                                pf[m][nt][0], pf[m][nt][1]);
                        mma_f16(oacc[w * 4 + up * 2 + 1][nt], x8 & kNibLo, x8 & kNibHi, y8 & kNibLo, y8 & kNibHi,
                                pf[m][nt][0], pf[m][nt][1]);
                    }
                }
        }
        __syncwarp();                   // the stage may be loaded again
    }

    // -------------------------------------------------- merge of the warps --
    cp_async_wait<0>();
    float* sm_m = reinterpret_cast<float*>(smem + C::OFF_STATS);       // [WARPS][ROWS], base 2
    float* sm_l = sm_m + C::WARPS * C::ROWS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], o);
                za[nt][j] += __shfl_xor_sync(0xffffffffu, za[nt][j], o);
            }
            mu[nt][j] = mu[nt][j] == kNegInf ? kNegInf : mu[nt][j] * rf[nt][j];
            if (g8 == 0) {
                sm_m[warp * C::ROWS + nt * 8 + 2 * t4 + j] = mu[nt][j];
                sm_l[warp * C::ROWS + nt * 8 + 2 * t4 + j] = l[nt][j];
            }
        }
    __syncthreads();                    // also: every warp is done with its ring
    float* so = reinterpret_cast<float*>(smem);            // [WARPS][ROWS][OSTRIDE]
    const float back = ldexpf(1.f, static_cast<int>(ev) - 141);       // undoes 2^(14 - (ev - 127))
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = nt * 8 + 2 * t4 + j;
            float M = kNegInf;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) M = fmaxf(M, sm_m[w * C::ROWS + r]);
            const float f = mu[nt][j] == kNegInf && !isnan(l[nt][j]) ? 0.f : ex2(mu[nt][j] - M) * back;
            float* dst = so + (warp * C::ROWS + r) * C::OSTRIDE + g8;
            // channel g8 * D/8 + n sits at n * 8 + g8: eight lanes, eight banks
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
                dst[(2 * m) * 8] = fmaf(oacc[m][nt][j], 16777216.f, -za[nt][j]) * f;       // 2^24
                dst[(2 * m + 1) * 8] = fmaf(oacc[m][nt][2 + j], 1048576.f, -za[nt][j]) * f;    // 2^20
            }
        }
    __syncthreads();
    for (int e = threadIdx.x; e < nrows * (D / 2); e += C::WARPS * 32) {
        const int r = e / (D / 2), c2 = (e % (D / 2)) * 2;
        const int at = (c2 % (D / 8)) * 8 + c2 / (D / 8);
        float M = kNegInf, L = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) M = fmaxf(M, sm_m[w * C::ROWS + r]);
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
            const float mw = sm_m[w * C::ROWS + r], lw = sm_l[w * C::ROWS + r];
            L += mw == kNegInf && !isnan(lw) ? 0.f : lw * ex2(mw - M);
            a0 += so[(w * C::ROWS + r) * C::OSTRIDE + at];
            a1 += so[(w * C::ROWS + r) * C::OSTRIDE + at + 8];
        }
        const bool some = !(L == 0.f);              // NaN stays NaN
        const float inv = some ? 1.f / L : 0.f;
        const float lse2 = some ? M + __log2f(L) : kNegInf;
        const int i = (r0 + r) / p.G, h = hk * p.G + (r0 + r) % p.G;
        const size_t row = static_cast<size_t>(b) * p.Nq + i;
        if (p.nsplit == 1) {
            *reinterpret_cast<uint32_t*>(p.o + (row * p.H + h) * D + c2) = pack_bf16(a0 * inv, a1 * inv);
            if (c2 == 0) p.lse[(static_cast<size_t>(b) * p.H + h) * p.Nq + i] = lse2 * 0.6931471805599453f;
        } else {
            *reinterpret_cast<float2*>(p.o_part + ((static_cast<size_t>(split) * rows_q + row) * p.H + h) * D + c2) =
                make_float2(a0 * inv, a1 * inv);
            if (c2 == 0) p.lse_part[(static_cast<size_t>(split) * p.H + h) * rows_q + row] = lse2;
        }
    }
}

}  // namespace fa
