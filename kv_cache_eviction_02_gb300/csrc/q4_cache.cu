// Cache in 4 bits: prompts quantised as a whole, rows quantised into pages, both read back.
//
// A group's step is the smallest s of four significant bits, 2^-126 at least, with 15 s >= hi - lo, where
// lo = min(0, least value) and hi = max(0, largest): four bits, so that s m is exact in bf16 (the step
// is at most an eighth larger than it need be). With M = floor(F / s), F the type's largest number, the zero
// code is k = min(M, -lo / s) and a value's m = x / s, both to the nearest (halves toward zero) and m within
// -k .. min(15 - k, M). x / s is x times a reciprocal of s that is too small by about 2^-20: halves fall
// toward zero as they should, and the quotient of a 16-bit value by a step of four bits is at least 2^-12
// (relative) away from a half unless it is one, so no other value changes sides; fp32 values are put right by the
// exact remainder x - s m.
//
// Bound by HBM: one layer's 128K prompt of bf16 (8 heads of d 128) packed and read back 226 us, 6.1 TB/s; four ragged
// prompts of 32K (fp16) read back 93.5 us, 6.7 TB/s. Each of four lanes works out one row's steps (each for itself: 289 us), and
// values come back in 16-bit arithmetic, which is exact (in fp32: 122 us for the latter). A thread takes 8 channels of the four
// tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of a tile, whose codes fill whole words of K and of V: rows come in 16-byte
// loads and leave as full 32-byte sectors, no shared memory between.
#include <type_traits>

#include "q4.cuh"

namespace kve {
namespace {

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: x + kMagic rounds x to a whole number in the low bits

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T> __device__ __forceinline__ float largest();
template <> __device__ __forceinline__ float largest<float>() { return 3.4028234663852886e38f; }
template <> __device__ __forceinline__ float largest<__nv_bfloat16>() { return 3.3895313892515355e38f; }
template <> __device__ __forceinline__ float largest<__half>() { return 65504.f; }

// 8 neighbouring channels as they lie in memory.
template <typename T> struct Eight {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void zero() {
        for (auto &x : w) x = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ float at(int e) const { return to_f(reinterpret_cast<const T *>(w)[e]); }
    __device__ __forceinline__ void range(float *lo, float *hi) const {
        if constexpr (sizeof(T) == 2) {
            using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            const T2 *x = reinterpret_cast<const T2 *>(w);
            const T2 l = __hmin2_nan(__hmin2_nan(x[0], x[1]), __hmin2_nan(x[2], x[3]));
            const T2 h = __hmax2_nan(__hmax2_nan(x[0], x[1]), __hmax2_nan(x[2], x[3]));
            *lo = min_nan(to_f(l.x), to_f(l.y));
            *hi = max_nan(to_f(h.x), to_f(h.y));
        } else {
            *lo = *hi = at(0);
#pragma unroll
            for (int e = 1; e < 8; ++e) {
                *lo = min_nan(*lo, at(e));
                *hi = max_nan(*hi, at(e));
            }
        }
    }
};

// x / s rounded to a whole number, as a float (halves toward zero); r a little below 1 / s.
template <bool EXACT> __device__ __forceinline__ float nearest(float x, float s, float r) {
    float m = fmaf(x, r, kMagic) - kMagic;
    if (EXACT) {
        const float rest = fmaf(-m, s, x);  // exact: m s is next to x
        if (fabsf(rest) > 0.5f * s) m += copysignf(1.f, rest);
    }
    return m;
}

// The codes of four rows of 8 values, in the low nibbles of n, and their groups' parameters. The G / 8 lanes that share
// the four groups are neighbours and all call: each of four lanes works out one row's step for all of them.
template <typename T, int G>
__device__ __forceinline__ void quantise(const Eight<T> (&x)[4], uint32_t (&n)[4][8], unsigned short (&p)[4]) {
    constexpr bool EXACT = sizeof(T) == 4;
    float lo[4], hi[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t].range(&lo[t], &hi[t]);
    const int lane = threadIdx.x & 31;
    const bool up2 = lane & 2, up1 = lane & 1;  // this lane's row: lane % 4
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float sl = up2 ? lo[i] : lo[i + 2], sh = up2 ? hi[i] : hi[i + 2];
        lo[i] = min_nan(up2 ? lo[i + 2] : lo[i], __shfl_xor_sync(0xffffffffu, sl, 2));
        hi[i] = max_nan(up2 ? hi[i + 2] : hi[i], __shfl_xor_sync(0xffffffffu, sh, 2));
    }
    const float sl = up1 ? lo[0] : lo[1], sh = up1 ? hi[0] : hi[1];
    float l = min_nan(up1 ? lo[1] : lo[0], __shfl_xor_sync(0xffffffffu, sl, 1));
    float h = max_nan(up1 ? hi[1] : hi[0], __shfl_xor_sync(0xffffffffu, sh, 1));
#pragma unroll
    for (int o = 4; o < G / 8; o <<= 1) {
        l = min_nan(l, __shfl_xor_sync(0xffffffffu, l, o));
        h = max_nan(h, __shfl_xor_sync(0xffffffffu, h, o));
    }
    l = min_nan(l, 0.f);
    h = max_nan(h, 0.f);
    // an infinity or a NaN (a range above fp32's largest number is none): no step, codes do not matter
    const bool bad = !(fmaxf(h, -l) <= largest<float>() && l == l);
    // 15 s >= h - l: from a quotient that is too small, up by at most two of the numbers of four bits. h - l is
    // rounded up, which leaves the answer as it is, since 15 s is exact.
    const float down = fmaxf(h, -l) > 0x1p100f ? 0x1p-8f : 1.f;
    const float d = fmaxf(__fsub_ru(h * down, l * down), 15 * 0x1p-126f);
    float s = __uint_as_float(__float_as_uint(d * 0.06666665f) & 0xFFF00000u);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (15.f * s < d) s = __uint_as_float(__float_as_uint(s) + 0x00100000u);
    s *= down < 1.f ? 0x1p8f : 1.f;
    float r = bad ? 0.f : rcp_approx(s) * (1.f - 0x1p-20f), most = 15.f;
    if (15.f * s > largest<T>()) {  // whole numbers whose values the type still holds
        most = fminf(floorf(largest<T>() * r), 15.f);
        if ((most + 1.f) * s <= largest<T>()) most += 1.f;
    }
    const float k = bad ? 0.f : fminf(nearest<EXACT>(-l, s, r), most);
    // parameter, zero code, highest code; and whether a code may have to be raised (15 s above the largest number)
    const uint32_t mine = (bad ? (uint32_t)kQ4Nan : __float_as_uint(s) >> 16 | (uint32_t)k) |
                          (uint32_t)fminf(15.f, k + most) << 16;
    const bool raise = __any_sync(0xffffffffu, most < 15.f);
    auto codes = [&](auto both) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t y = __shfl_sync(0xffffffffu, mine, (lane & ~3) | t);
            const float rt = __shfl_sync(0xffffffffu, r, (lane & ~3) | t);
            p[t] = (unsigned short)y;
            const float st = __uint_as_float((y & 0xFFF0u) << 16);
            // kMagic + k, + the highest code: its bits are 0x4B400000 + the number
            const float zero = __uint_as_float(0x4B400000u + (y & 15u)), top = __uint_as_float(0x4B400000u + (y >> 16));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = x[t].at(e);
                float c = EXACT ? nearest<true>(v, st, rt) + zero : fmaf(v, rt, zero);
                if (decltype(both)::value) c = fmaxf(c, kMagic);
                n[t][e] = __float_as_uint(fminf(c, top));
            }
        }
    };
    if (raise) codes(std::true_type{});
    else codes(std::false_type{});
}

// bytes c | (c + 2) << 4 for channels c = 0, 1, 4, 5 of K, c | (c + 1) << 4 for c = 0, 2, 4, 6 of V
template <bool IS_V> __device__ __forceinline__ void pairs(const uint32_t (&n)[8], uint32_t (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = IS_V ? 2 * i : (i & 1) + 4 * (i >> 1);
        b[i] = n[c] + (n[c + (IS_V ? 1 : 2)] << 4);
    }
}
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Quantises 8 channels (ch .. ch + 7) of the four tokens {2 j, 2 j + 1, 2 j + 8, 2 j + 9} of a tile into it. A
// warp may hold lanes of K and of V: what they do together comes before they part.
template <typename T, int D, int G>
__device__ __forceinline__ void store_quad(const Eight<T> (&x)[4], int j, int ch, bool is_v, uint8_t *tile) {
    constexpr int NG = D / G;
    uint32_t n[4][8], b[4][4];
    unsigned short p[4];
    quantise<T, G>(x, n, p);
    if (is_v) {
#pragma unroll
        for (int t = 0; t < 4; ++t) pairs<true>(n[t], b[t]);
        const int r = (ch & 8) >> 1, w = ch >> 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint32_t *>(tile + q4_codes(D) + q4_word<D>((r + i) * 4 + j, w)) =
                bytes4(b[0][i], b[2][i], b[1][i], b[3][i]);
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) pairs<false>(n[t], b[t]);
        const int lane = ch >> 3 & 3, w = ch >> 5 << 1;
#pragma unroll
        for (int u = 0; u < 2; ++u)  // tokens 2 j + u and 2 j + u + 8
            *reinterpret_cast<uint2 *>(tile + q4_word<D>((2 * j + u) * 4 + lane, w)) =
                make_uint2(bytes4(b[u][0], b[u + 2][0], b[u][1], b[u + 2][1]),
                           bytes4(b[u][2], b[u + 2][2], b[u][3], b[u + 2][3]));
    }
    if (ch % G == 0) {
        unsigned short *params = reinterpret_cast<unsigned short *>(
            tile + 2 * q4_codes(D) + (is_v ? q4_params(D, G) : 0));
#pragma unroll
        for (int t = 0; t < 4; ++t) params[(2 * j + (t & 1) + 8 * (t >> 1)) * NG + ch / G] = p[t];
    }
}

constexpr int kQ4Threads = 256;

// Threads of a tile: D / 8 for its channels, 4 for its quads of tokens, K and V apart. Which tile of the grid's row.
template <int D> __device__ __forceinline__ int tile_of(int *j, int *ch, bool *is_v) {
    const unsigned i = threadIdx.x;
    *ch = (int)(i % (D / 8)) * 8;
    *j = (int)(i / (D / 8) & 3);
    *is_v = i / (D / 2) & 1;
    return (int)(blockIdx.x * (kQ4Threads / D) + i / D);
}

// ---- a prompt as a whole ---------------------------------------------------------------------------
template <typename T, int D, int G>
__global__ void __launch_bounds__(kQ4Threads) q4_pack_kernel(Q4Cache C) {
    pg_wait_prior();
    pg_launch_dependents();
    int j, ch;
    bool is_v;
    const int tile = tile_of<D>(&j, &ch, &is_v), s = blockIdx.y, h = blockIdx.z;
    const int len = C.len ? pg_clamp(__ldg(C.len + s), 0, C.D.n) : C.D.n;
    if (tile >= (len + kQ4Tile - 1) / kQ4Tile) return;  // (whole warps: a tile's threads are a multiple of 32)
    const T *src = static_cast<const T *>(is_v ? C.V : C.K) +
                   (is_v ? s * C.v0 + h * C.v1 : s * C.s0 + h * C.s1) + ch;
    const long long row = is_v ? C.v2 : C.s2;
    Eight<T> x[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int tok = tile * kQ4Tile + 2 * j + (t & 1) + 8 * (t >> 1);
        x[t].zero();
        if (tok < len) x[t].load(src + tok * row);
    }
    store_quad<T, D, G>(x, j, ch, is_v, C.cache + (((size_t)s * C.D.Hkv + h) * C.Q.ptiles + tile) * q4_tile_bytes(D, G));
}

// ---- rows into pages -------------------------------------------------------------------------------
__device__ __forceinline__ uint8_t *page_tile(const Q4Cache &C, int slot, int h, int bytes) {
    const int page = slot >> C.D.lgP;
    return C.cache + ((((size_t)page * C.D.Hkv + h) << (C.D.lgP - 4)) + ((slot & (C.D.P - 1)) >> 4)) * bytes;
}
// a slot of the caller's; one outside the pool is recorded and skipped
__device__ __forceinline__ int slot_of(const Q4Cache &C, int i) {
    const int slot = __ldg(C.slots + i);
    if (slot >= C.D.npages << C.D.lgP) {
        atomicOr(C.err, KVE_DEVERR_BADPAGE);
        return -1;
    }
    return slot;
}

// 8 channels of four rows, row t of them the token slot[t] % 16 of a tile (none where slot[t] < 0): byte by byte, so that
// a tile's other tokens stay as they are.
template <typename T, int D, int G>
__device__ __forceinline__ void store_rows(const Q4Cache &C, const Eight<T> (&x)[4], const int (&slot)[4], int h, int ch,
                                           bool is_v) {
    uint32_t n[4][8], b[4];
    unsigned short p[4];
    quantise<T, G>(x, n, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (slot[i] < 0) continue;
        const int t = slot[i] & 15;
        uint8_t *tile = page_tile(C, slot[i], h, q4_tile_bytes(D, G));
        if (is_v) {
            pairs<true>(n[i], b);
            uint8_t *w = tile + q4_codes(D) + ((t & 1) << 1) + (t >> 3);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                w[q4_word<D>((((ch & 8) >> 1) + y) * 4 + ((t & 7) >> 1), ch >> 4)] = (uint8_t)b[y];
        } else {
            pairs<false>(n[i], b);
            uint8_t *w = tile + q4_word<D>((t & 7) * 4 + (ch >> 3 & 3), ch >> 5 << 1) + (t >> 3);
#pragma unroll
            for (int y = 0; y < 4; ++y) w[2 * y] = (uint8_t)b[y];
        }
        if (ch % G == 0)
            *reinterpret_cast<unsigned short *>(tile + 2 * q4_codes(D) + (is_v ? q4_params(D, G) : 0) +
                                                2 * (t * (D / G) + ch / G)) = p[i];
    }
}

// The threads of a tile (tile_of) take 16 rows that stand behind one another in the batch. Rows that fill a tile of the
// cache (16 consecutive slots) are written as one by the threads of the 16 in which they begin, as whole words; other
// rows byte by byte (64 prompts of up to 2000 rows, fp16, 8 heads of d 128, with their reading back: all of them byte by
// byte 232 us, so 177; 131 with the steps and the way back as they are now).
template <typename T, int D, int G>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(Q4Cache C) {
    pg_wait_prior();
    pg_launch_dependents();
    int j, ch;
    bool is_v;
    const int win = tile_of<D>(&j, &ch, &is_v), h = blockIdx.y, lane = threadIdx.x & 31;
    if (win >= (C.D.rows + 15) / 16) return;  // (whole warps)
    const int i0 = win * 16;
    // slots of the 16 rows before, of these, and of the 16 behind: bit p of the masks is row i0 - 16 + p
    auto at = [&](int i) { return i >= 0 && i < C.D.rows ? slot_of(C, i) : -1; };
    const int sa = at(i0 - 16 + lane), sb = lane < 16 ? at(i0 + 16 + lane) : -1;
    const int pa = __shfl_up_sync(0xffffffffu, sa, 1), last = __shfl_sync(0xffffffffu, sa, 31);
    int pb = __shfl_up_sync(0xffffffffu, sb, 1);
    if (lane == 0) pb = last;
    auto follows = [](int s, int before) { return s >= 0 && (s & 15) != 0 && before >= 0 && s == before + 1; };
    unsigned long long run = __ballot_sync(0xffffffffu, lane > 0 && follows(sa, pa)) |
                             (unsigned long long)__ballot_sync(0xffffffffu, follows(sb, pb)) << 32;
    run &= run >> 1;
    run &= run >> 2;
    run &= run >> 4;  // of 8 rows
    run &= run >> 7;  // of 15
    const unsigned full = __ballot_sync(0xffffffffu, sa >= 0 && (sa & 15) == 0) & (unsigned)(run >> 1);
    unsigned long long covered = full;
    covered |= covered << 1;
    covered |= covered << 2;
    covered |= covered << 4;
    covered |= covered << 8;
    const T *src = static_cast<const T *>(is_v ? C.V : C.K) + h * (is_v ? C.v1 : C.s1) + ch;
    const long long row = is_v ? C.v2 : C.s2;
    Eight<T> x[4];
    if (full >> 16) {
        const int first = __ffs(full >> 16) - 1;
        const int slot = __shfl_sync(0xffffffffu, sa, 16 + first);
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t].load(src + (i0 + first + 2 * j + (t & 1) + 8 * (t >> 1)) * row);
        store_quad<T, D, G>(x, j, ch, is_v, page_tile(C, slot, h, q4_tile_bytes(D, G)));
    }
    const unsigned there = __ballot_sync(0xffffffffu, sa >= 0) >> 16;
    if ((there & ~(unsigned)(covered >> 16) & 0xFFFFu) == 0) return;
    int slot[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int i = j + 4 * t;
        slot[t] = __shfl_sync(0xffffffffu, sa, 16 + i);
        if (covered >> (16 + i) & 1) slot[t] = -1;
        x[t].zero();
        if (slot[t] >= 0) x[t].load(src + (i0 + i) * row);
    }
    store_rows<T, D, G>(C, x, slot, h, ch, is_v);
}

// ---- reading back ----------------------------------------------------------------------------------
template <typename T, int D, int G, bool PAGES>
__global__ void __launch_bounds__(kQ4Threads) q4_unpack_kernel(Q4Cache C) {
    pg_wait_prior();
    pg_launch_dependents();
    constexpr int NG = D / G;
    int j, ch;
    bool is_v;
    const int tile = tile_of<D>(&j, &ch, &is_v), s = blockIdx.y, h = blockIdx.z, t0 = tile * kQ4Tile;
    const int len = C.len ? pg_clamp(__ldg(C.len + s), 0, C.rows) : C.rows;
    if (tile >= (len + kQ4Tile - 1) / kQ4Tile) return;
    const uint8_t *src;
    if (PAGES) {
        const int page = pg_page(C.table + (size_t)s * C.width, t0, C.D.lgP, C.D.npages, C.err);
        src = page_tile(C, (page << C.D.lgP) + (t0 & (C.D.P - 1)), h, q4_tile_bytes(D, G));
    } else {
        src = C.cache + (((size_t)s * C.D.Hkv + h) * C.Q.ptiles + tile) * q4_tile_bytes(D, G);
    }
    const uint8_t *codes = src + (is_v ? q4_codes(D) : 0);
    const unsigned short *params = reinterpret_cast<const unsigned short *>(
        src + 2 * q4_codes(D) + (is_v ? q4_params(D, G) : 0)) + ch / G;
    // K: w[0], w[1] and w[2], w[3] of tokens 2 j and 2 j + 1 (with + 8); V: w[i] of channels 2 i, 2 i + 1
    uint32_t w[4], p[4];
    if (is_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __ldg(reinterpret_cast<const uint32_t *>(codes + q4_word<D>((((ch & 8) >> 1) + i) * 4 + j, ch >> 4)));
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(
                codes + q4_word<D>((2 * j + u) * 4 + (ch >> 3 & 3), ch >> 5 << 1)));
            w[2 * u] = x.x;
            w[2 * u + 1] = x.y;
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) p[t] = __ldg(params + (2 * j + (t & 1) + 8 * (t >> 1)) * NG);
    Eight<T> out[4];  // of tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9
    if constexpr (sizeof(T) == 2) {
        if (is_v) {
            const Q4Codes<T> of0(p[0] | p[1] << 16), of1(p[2] | p[3] << 16);
            uint32_t *o[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) o[t] = reinterpret_cast<uint32_t *>(out[t].w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = of0.low(w[i]), b = of0.high(w[i]), c = of1.low(w[i] >> 8), d = of1.high(w[i] >> 8);
                o[0][i] = __byte_perm(a, b, 0x5410);
                o[1][i] = __byte_perm(a, b, 0x7632);
                o[2][i] = __byte_perm(c, d, 0x5410);
                o[3][i] = __byte_perm(c, d, 0x7632);
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const Q4Codes<T> of(p[t] * 0x10001u);
                const uint32_t x = w[2 * (t & 1)] >> (t & 2 ? 8 : 0), y = w[2 * (t & 1) + 1] >> (t & 2 ? 8 : 0);
                out[t].w[0] = make_uint4(of.low(x), of.high(x), of.low(y), of.high(y));
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float step = __uint_as_float((p[t] & 0xFFF0u) << 16), off = 8388608.f + (float)(p[t] & 15u);
            float *x = reinterpret_cast<float *>(out[t].w);
            auto value = [&](uint32_t word, int bit) {  // 2^23 + n, less 2^23 + k: exact
                return (__uint_as_float((word >> bit & 15u) | 0x4B000000u) - off) * step;
            };
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = is_v ? value(w[e >> 1], (t >> 1) * 8 + (t & 1) * 16 + (e & 1) * 4)
                            : value(w[2 * (t & 1) + (e >> 2)], (t >> 1) * 8 + (e & 1) * 16 + (e & 2) * 2);
        }
    }
    T *dst = static_cast<T *>(is_v ? C.Vo : C.Ko) + (is_v ? s * C.v0 + h * C.v1 : s * C.s0 + h * C.s1) + ch;
    const long long row = is_v ? C.v2 : C.s2;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int tok = t0 + 2 * j + (t & 1) + 8 * (t >> 1);
        if (tok >= len) continue;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(dst + tok * row)[i] = out[t].w[i];
    }
}

// ---- host ------------------------------------------------------------------------------------------
template <typename F> cudaError_t by_type(int dtype, F f) {
    if (dtype == KVE_F32) return f(float{});
    return dtype == KVE_BF16 ? f(__nv_bfloat16{}) : f(__half{});
}
template <int V> using Int = std::integral_constant<int, V>;
template <typename F> cudaError_t by_sizes(const Q4Shape &Q, F f) {
    if (Q.d == 128)
        return Q.group == 32 ? f(Int<128>{}, Int<32>{})
                             : (Q.group == 64 ? f(Int<128>{}, Int<64>{}) : f(Int<128>{}, Int<128>{}));
    if (Q.d == 64) return Q.group == 32 ? f(Int<64>{}, Int<32>{}) : f(Int<64>{}, Int<64>{});
    return f(Int<32>{}, Int<32>{});
}
// blocks of kQ4Threads / d tiles
unsigned q4_blocks(long long tiles, int d) { return (unsigned)((tiles + kQ4Threads / d - 1) / (kQ4Threads / d)); }

}  // namespace

cudaError_t launch_q4_pack(const Q4Cache &C, cudaStream_t st) {
    const dim3 grid(q4_blocks(C.Q.ptiles, C.D.d), C.count, C.D.Hkv);
    return by_type(C.D.dtype, [&](auto t) {
        return by_sizes(C.Q, [&](auto d, auto g) {
            return pg_launch(q4_pack_kernel<decltype(t), decltype(d)::value, decltype(g)::value>, grid, kQ4Threads, 0,
                             true, st, C);
        });
    });
}

cudaError_t launch_q4_append(const Q4Cache &C, cudaStream_t st) {
    const dim3 grid(q4_blocks((C.D.rows + 15) / 16, C.D.d), C.D.Hkv);
    return by_type(C.D.dtype, [&](auto t) {
        return by_sizes(C.Q, [&](auto d, auto g) {
            return pg_launch(q4_append_kernel<decltype(t), decltype(d)::value, decltype(g)::value>, grid, kQ4Threads, 0,
                             true, st, C);
        });
    });
}

cudaError_t launch_q4_unpack(const Q4Cache &C, cudaStream_t st) {
    const dim3 grid(q4_blocks((C.rows + kQ4Tile - 1) / kQ4Tile, C.D.d), C.count, C.D.Hkv);
    return by_type(C.D.dtype, [&](auto t) {
        return by_sizes(C.Q, [&](auto d, auto g) {
            constexpr int D = decltype(d)::value, G = decltype(g)::value;
            auto kern = C.table ? q4_unpack_kernel<decltype(t), D, G, true>
                                : q4_unpack_kernel<decltype(t), D, G, false>;
            return pg_launch(kern, grid, kQ4Threads, 0, true, st, C);
        });
    });
}

}  // namespace kve
