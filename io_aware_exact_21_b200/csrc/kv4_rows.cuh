// kv4_rows.cuh -- the 4-bit key/value cache: its number format, and the
// kernels that write new rows into it and read rows back.
//
// A cache row is one token of one key/value head, x of D channels.  With
//     hi = max(0, max x),  lo = min(0, min x),
//     s  = the smallest number with 4 significant bits that has
//          15 s >= hi - lo (and is at least 2^-126),
//     z  = floor(-lo / s + 1/2)                                 (0 .. 15),
//     c  = min(15, floor(x / s + 1/2) + z)                      (0 .. 15)
// it stands for s (c - z), at most s / 2 away from x.  s has 4 significant
// bits and |c - z| <= 15 has 4, so every value is a bf16 number: reading a
// row back, and attention over the rows read back, round nothing.  s is bf16
// with its low four mantissa bits zero, and those four bits hold z: one
// 16-bit word a row, 4 + 16/D bits a value.  A row that holds NaN or infinity
// gets s = NaN and reads back as NaN.
//
// Both kernels move each byte once and compute little, so HBM bounds them:
// 2 D bytes of bf16 against D / 2 + 2 of cache for a row.  A row's D / 8
// lanes hold 8 channels each (one 16-byte access of the bf16 side, one 4-byte
// access of the codes); a warp takes consecutive tokens of one head, so that
// its cache rows lie next to each other, and starts all its loads before it
// uses the first.
#pragma once

#include "sm100.cuh"

namespace fa {

constexpr uint32_t kKv4NaN = 0x7fc0u;     // the word of a row that holds NaN or infinity

// Where the rows of a write or read sit: row i of sequence b, i < n_b, is
// cache row starts[b] + i.  n_b is N, or lens[b] where that is smaller; with
// cu_seqlens the rows are packed and n_b is cu_seqlens[b + 1] - cu_seqlens[b].
struct Kv4Place {
    const int* cu_seqlens;   // or nullptr
    const int* starts;       // or nullptr (all 0)
    const int* lens;         // or nullptr (all N)
    int B, N, H;             // N: rows a sequence; packed: all rows
    int Nk;                  // cache rows a sequence has room for
    int from_window;         // > 0 (fixed length, no starts): row 0 of the bf16 side is the first
    int from_queries;        //   that the attention call's queries read (kv4_first_row), N the room there
};

// For attention under a sliding window: the first cache row that the last
// `from_queries` positions of a sequence of n rows read, in whole 128-key tiles.
__device__ __forceinline__ int kv4_first_row(const Kv4Place& w, int n) {
    if (w.from_window <= 0) return 0;
    const int64_t first = static_cast<int64_t>(n) - w.from_queries - w.from_window + 1;
    return first > 0 ? static_cast<int>(first) / 128 * 128 : 0;
}

// The cache rows of sequence b that such a call uses.
__device__ __forceinline__ int kv4_used(const Kv4Place& w, int b) {
    return w.lens ? min(max(w.lens[b], 0), w.Nk) : w.Nk;
}

// Sequence and cache row of row r of the [rows, H, D] side; false when r
// belongs to no sequence or its cache row does not exist.
__device__ __forceinline__ bool kv4_place(const Kv4Place& w, int64_t r, int64_t rows, int& b, int& pos) {
    if (r >= rows) return false;
    int64_t i;
    if (w.cu_seqlens) {
        if (w.B <= 0 || r >= w.cu_seqlens[w.B] || r < w.cu_seqlens[0]) return false;
        int lo = 0, hi = w.B;                 // cu[lo] <= r < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (w.cu_seqlens[mid] <= r) lo = mid;
            else hi = mid;
        }
        b = lo;
        i = r - w.cu_seqlens[b];
    } else {
        b = static_cast<int>(static_cast<uint32_t>(r) / static_cast<uint32_t>(w.N));   // rows < 2^31
        i = r - static_cast<int64_t>(b) * w.N;
        if (w.from_window > 0) {
            const int n = kv4_used(w, b);
            i += kv4_first_row(w, n);
            if (i >= n) return false;
        } else if (i >= (w.lens ? min(w.lens[b], w.N) : w.N)) {
            return false;
        }
    }
    const int64_t at = (w.starts ? w.starts[b] : 0) + i;
    pos = static_cast<int>(at);
    return at >= 0 && at < w.Nk;
}

__device__ __forceinline__ uint32_t bf2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t bf2_min_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// {low: max x, high: -min x} of 8 channels (one bf16 pair a word); NaN where x has one.
__device__ __forceinline__ uint32_t kv4_extremes(const uint4& x) {
    const uint32_t up = bf2_max_nan(bf2_max_nan(x.x, x.y), bf2_max_nan(x.z, x.w));
    const uint32_t dn = bf2_min_nan(bf2_min_nan(x.x, x.y), bf2_min_nan(x.z, x.w)) ^ 0x80008000u;
    return bf2_max_nan(__byte_perm(up, dn, 0x5410), __byte_perm(up, dn, 0x7632));
}

// The same of whole rows, each held by LANES neighbouring lanes, a row of each
// of ITER steps: lane c of a group returns those of step c % ITER.  The lanes
// halve the steps they hold with each exchange (ITER - 1 of them, not
// log2(LANES) for every step).
template <int LANES, int ITER>
__device__ __forceinline__ uint32_t kv4_row_extremes(const uint4 (&x)[ITER]) {
    uint32_t m[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it) m[it] = kv4_extremes(x[it]);
    const int lane = lane_id();
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        if (o < ITER) {
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < ITER / 2 / o; ++i) {
                const uint32_t keep = upper ? m[2 * i + 1] : m[2 * i], send = upper ? m[2 * i] : m[2 * i + 1];
                m[i] = bf2_max_nan(keep, __shfl_xor_sync(0xffffffffu, send, o));
            }
        } else {
            m[0] = bf2_max_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        }
    }
    return m[0];
}

// How a row is rounded: x * inv + base cut to an integer is 128 + c.
struct Kv4Scale {
    float inv, base;
    uint32_t word;
    bool clamp;         // c = 16 can come out
};

// s: with r = hi - lo rounded up to fp32 (halved, so that it cannot overflow),
// r (1 - 2^-21) / 15 rounded up to 4 significant bits is s or the number below
// it, which 15 s >= r tells apart: 15 s is an fp32 number, so it compares with
// r as with the exact difference.
//
// c: x / s is either exactly half-way between two integers or at least 2^-10
// away from that (8 bits over 4 bits), while x * (1 / s) + z errs by less than
// 2^-17; so adding 1/2 + 2^-11 before cutting the fraction gives the nearest
// integer with exact ties upwards.  c = 16 needs hi / s and -lo / s both
// half-way and 15 together.
__device__ __forceinline__ Kv4Scale kv4_scale(uint32_t m) {
    m = bf2_max_nan(m, 0u);
    const float hi = __uint_as_float(m << 16), neg_lo = __uint_as_float(m & 0xffff0000u);
    const float r = __fmaf_ru(hi, 0.5f, 0.5f * neg_lo);
    uint32_t sb = (__float_as_uint(r * (0.13333333f * (1.f - 1.f / 2097152.f))) + 0x000fffffu) & 0xfff00000u;
    sb = max(sb + (7.5f * __uint_as_float(sb) < r ? 0x00100000u : 0u), 0x00800000u);
    Kv4Scale s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.inv) : "f"(__uint_as_float(sb)));
    constexpr float kHalfUp = 0.5f + 1.f / 2048.f;
    const uint32_t zb = __float_as_uint(fmaf(neg_lo, s.inv, 128.f + kHalfUp));
    s.base = __uint_as_float(zb & 0xffff0000u) + kHalfUp;           // 128 + z + 1/2 and a little
    s.word = hi <= 3.4e38f && neg_lo <= 3.4e38f ? (sb | (zb & 0x000f0000u)) >> 16 : kKv4NaN;
    s.clamp = fmaf(hi, s.inv, s.base) >= 144.f;
    return s;
}

// Codes of 8 channels.  128 + c has c in the third byte of its fp32 pattern,
// from where byte permutes collect it.
__device__ __forceinline__ uint32_t kv4_encode(const uint4& x, float inv, float base, bool clamp) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    float2 c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = ffma2(make_float2(__uint_as_float(xs[j] << 16), __uint_as_float(xs[j] & 0xffff0000u)),
                     make_float2(inv, inv), make_float2(base, base));
    if (clamp) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = make_float2(fminf(c[j].x, 143.9f), fminf(c[j].y, 143.9f));
    }
    auto third = [](float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0062); };
    const uint32_t even = __byte_perm(third(c[0].x, c[1].x), third(c[2].x, c[3].x), 0x5410);
    const uint32_t odd = __byte_perm(third(c[0].y, c[1].y), third(c[2].y, c[3].y), 0x5410);
    return even + odd * 16u;
}

// The 8 channels of a word of codes as bf16.  128 + c - (128 + z) and the
// product with s are exact.
__device__ __forceinline__ uint4 kv4_decode(uint32_t codes, uint32_t word) {
    const uint32_t s2 = (word & 0xfff0u) * 0x00010001u;
    const uint32_t z2 = (0xc300u | (word & 15u)) * 0x00010001u;       // -(128 + z), twice
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t byte = (codes >> (8 * j)) & 0xffu;
        const uint32_t c2 = ((byte * 4097u) & 0x000f000fu) | 0x43004300u;   // 128 + c, low and high code
        uint32_t d, v;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(c2), "r"(z2));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(d), "r"(s2));
        r[j] = v;
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

struct Kv4Params {
    Kv4Place place;
    int64_t rows;                  // rows of the bf16 side
    __nv_bfloat16* x[2];           // K, V: [rows, H, D]
    uint8_t* codes[2];             // [B, H, Nk, D / 2]
    uint16_t* words[2];            // [B, H, Nk]
    int poison;                    // reading for attention: see kv4_read_kernel
    int* back_lens;                // or nullptr: for from_window, the rows read back of each sequence
};

constexpr int kKv4Warps = 8;

// Tokens that one warp takes: ITER steps of the 32 / (D / 8) rows it holds at once.
template <int D, int ITER>
__host__ __device__ constexpr int kv4_tokens() { return ITER * (32 / (D / 8)); }

// What a warp works on: tokens first .. first + TOK - 1 of head h.
struct Kv4Unit {
    int64_t first;
    int h, left;        // left: how many of the tokens exist
};

template <int TOK>
__device__ __forceinline__ Kv4Unit kv4_unit(const Kv4Params& p) {
    const uint32_t unit = blockIdx.x * kKv4Warps + (threadIdx.x >> 5);    // the host keeps units below 2^31
    const uint32_t chunk = unit / static_cast<uint32_t>(p.place.H);
    const int64_t first = static_cast<int64_t>(chunk) * TOK;
    const int64_t left = p.rows - first;
    return {first, static_cast<int>(unit - chunk * p.place.H), static_cast<int>(left < TOK ? left : TOK)};
}

// Row of the cache arrays of a unit's token; below 0 where it is not taken.
__device__ __forceinline__ int64_t kv4_row(const Kv4Params& p, const Kv4Unit& u, int token) {
    int b, pos;
    if (token >= u.left || !kv4_place(p.place, u.first + token, p.rows, b, pos)) return -1;
    return (static_cast<int64_t>(b) * p.place.H + u.h) * p.place.Nk + pos;
}

// Writes bf16 rows into the cache.  blockIdx.y selects K or V.
//
// Instructions bound it as soon as there are many a value (the integer pipe
// does half of them): a row's scale is found by one lane, not by all that hold
// the row, and the row's extremes come to that lane by exchanges that halve
// what a lane holds.  At 0.69 GB read and written (106 us at the copy rate):
// 221 us with the library's correctly rounded division and reciprocal by every
// lane, 155 us with approximations that are exact here, 126 us with a lane to a
// token, 112 us with the halving exchanges, packed products and addresses that
// advance by a step.
// Rows that are not taken are not read: their places are looked up before the loads
// (16 sequences of 128 to 4096 rows in a padded buffer of 4096, 32 heads, d 128: 151
// us, 206 with every row read; packed, where every row counts, as before; one token a
// sequence 0.1 us more, the loads wait for the look).
template <int D, int ITER>
__global__ void __launch_bounds__(kKv4Warps * 32)
kv4_write_kernel(const Kv4Params p) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES, TOK = kv4_tokens<D, ITER>();
    const Kv4Unit u = kv4_unit<TOK>(p);
    if (u.left <= 0) return;
    const int lane = lane_id(), sub = lane / LANES, c8 = lane % LANES;
    const int64_t row = kv4_row(p, u, c8 % ITER * ROWS + sub);
    const uint32_t take = __ballot_sync(0xffffffffu, row >= 0) >> (sub * LANES);    // bit it: of step it
    const __nv_bfloat16* x = (blockIdx.y ? p.x[1] : p.x[0]) + ((u.first + sub) * p.place.H + u.h) * D + c8 * 8;
    const int64_t step = static_cast<int64_t>(ROWS) * p.place.H * D;
    uint4 v[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it)
        v[it] = take >> it & 1 ? __ldcs(reinterpret_cast<const uint4*>(x + it * step)) : make_uint4(0, 0, 0, 0);
    if (__all_sync(0xffffffffu, row < 0)) return;
    const Kv4Scale s = kv4_scale(kv4_row_extremes<LANES, ITER>(v));
    const bool clamp = __any_sync(0xffffffffu, s.clamp);
    if (row >= 0 && c8 < ITER) (blockIdx.y ? p.words[1] : p.words[0])[row] = static_cast<uint16_t>(s.word);
    uint8_t* codes = (blockIdx.y ? p.codes[1] : p.codes[0]) + c8 * 4;
    const int64_t mine = row * (D / 2);
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        const int from = sub * LANES + it;
        const float inv = __shfl_sync(0xffffffffu, s.inv, from);
        const float base = __shfl_sync(0xffffffffu, s.base, from);
        const int64_t to = __shfl_sync(0xffffffffu, mine, from);
        const uint32_t c = kv4_encode(v[it], inv, base, clamp);
        if (to >= 0) *reinterpret_cast<uint32_t*>(codes + to) = c;
    }
}

// Reads cache rows back as bf16.  poison (attention's own use): a token whose
// K or V row is NaN becomes K = NaN, V = 0, so that it reaches the scores of
// the queries that see it and no product of the others (0 * NaN).  Under a window
// only the rows that the queries read are brought back, to the front of a buffer
// with room for those alone; back_lens takes their number.
template <int D, int ITER>
__global__ void __launch_bounds__(kKv4Warps * 32)
kv4_read_kernel(const Kv4Params p) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES, TOK = kv4_tokens<D, ITER>();
    if (p.back_lens && blockIdx.y == 0) {       // (the grid has a thread to each row of the buffer at least)
        const int64_t b = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
        if (b < p.place.B) {
            const int n = kv4_used(p.place, static_cast<int>(b));
            p.back_lens[b] = n - kv4_first_row(p.place, n);
        }
    }
    const Kv4Unit u = kv4_unit<TOK>(p);
    if (u.left <= 0) return;
    const int lane = lane_id(), sub = lane / LANES, c8 = lane % LANES;
    const uint8_t* codes = (blockIdx.y ? p.codes[1] : p.codes[0]) + c8 * 4;
    const uint16_t* words = blockIdx.y ? p.words[1] : p.words[0];
    const uint16_t* other = blockIdx.y ? p.words[0] : p.words[1];
    // a token a lane: its row, and the row's word
    const int64_t row = lane < TOK ? kv4_row(p, u, lane) : -1;
    const int64_t mine = row * (D / 2);
    uint32_t c[ITER];
    bool taken[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        const int64_t from = __shfl_sync(0xffffffffu, mine, it * ROWS + sub);
        taken[it] = from >= 0;
        c[it] = taken[it] ? *reinterpret_cast<const uint32_t*>(codes + from) : 0u;
    }
    uint32_t word = 0;
    if (row >= 0) {
        word = words[row];
        if (p.poison && (word >= 0x7f80u || other[row] >= 0x7f80u)) word = blockIdx.y == 0 ? kKv4NaN : 0u;
    }
    __nv_bfloat16* x = (blockIdx.y ? p.x[1] : p.x[0]) + ((u.first + sub) * p.place.H + u.h) * D + c8 * 8;
    const int64_t step = static_cast<int64_t>(ROWS) * p.place.H * D;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        const uint32_t w = __shfl_sync(0xffffffffu, word, it * ROWS + sub);
        if (taken[it]) *reinterpret_cast<uint4*>(x + it * step) = kv4_decode(c[it], w);
    }
}

}  // namespace fa
