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
// Bound by HBM. A thread takes 8 channels of the four tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of a tile, whose codes fill
// whole words of K and of V: rows come in 16-byte loads and leave as full 32-byte sectors, no shared memory between.
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

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    alignas(16) T v[8];
    reinterpret_cast<uint4 *>(v)[0] = __ldg(reinterpret_cast<const uint4 *>(p));
    if (sizeof(T) == 4)
        reinterpret_cast<uint4 *>(v)[sizeof(T) / 4] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_f(v[e]);
}

// x / s rounded to a whole number, as a float (halves toward zero); r a little below 1 / s.
template <bool EXACT> __device__ __forceinline__ float nearest(float x, float s, float r) {
    float m = fmaf(x, r, kMagic) - kMagic;
    if (EXACT) {
        const float rest = fmaf(-m, s, x);  // exact: m s is next to x
        if (fabsf(rest) > 0.5f * s) m += copysignf(1.f, rest);
    }
    return m;
}

// The codes of 8 values, in the low nibbles of n, and the group's parameter. The G / 8 lanes that share a group
// are neighbours and all call.
template <typename T, int G>
__device__ __forceinline__ unsigned short quantise8(float (&x)[8], uint32_t (&n)[8]) {
    constexpr bool EXACT = sizeof(T) == 4;
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = min_nan(lo, x[e]);
        hi = max_nan(hi, x[e]);
    }
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    lo = min_nan(lo, 0.f);
    hi = max_nan(hi, 0.f);
    const bool bad = !(hi - lo <= 3.4e38f) && !(fmaxf(hi, -lo) <= largest<float>() && lo == lo);
    if (bad) {  // an infinity or a NaN (a range above fp32's largest number is none)
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = 0;
        return kQ4Nan;
    }
    // 15 s >= hi - lo: from a quotient that is too small, up by at most two of the numbers of four bits. hi - lo is
    // rounded up, which leaves the answer as it is, since 15 s is exact.
    const float down = fmaxf(hi, -lo) > 0x1p100f ? 0x1p-8f : 1.f;
    const float t = fmaxf(__fsub_ru(hi * down, lo * down), 15 * 0x1p-126f);
    float s = __uint_as_float(__float_as_uint(t * 0.06666665f) & 0xFFF00000u);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (15.f * s < t) s = __uint_as_float(__float_as_uint(s) + 0x00100000u);
    s *= down < 1.f ? 0x1p8f : 1.f;
    const float r = rcp_approx(s) * (1.f - 0x1p-20f);
    float most = 15.f;
    if (15.f * s > largest<T>()) {  // whole numbers whose values the type still holds
        most = fminf(floorf(largest<T>() * r), 15.f);
        if ((most + 1.f) * s <= largest<T>()) most += 1.f;
    }
    const float k = fminf(nearest<EXACT>(-lo, s, r), most), top = fminf(15.f, k + most);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float y;
        if (EXACT) y = nearest<true>(x[e], s, r) + (kMagic + k);
        else y = fmaf(x[e], r, kMagic + k);
        n[e] = __float_as_uint(fminf(fmaxf(y, kMagic), kMagic + top));  // 0x4B400000 + code
    }
    return (unsigned short)(__float_as_uint(s) >> 16 | (uint32_t)k);
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
__device__ __forceinline__ void store_quad(float (&x)[4][8], int j, int ch, bool is_v, uint8_t *tile) {
    constexpr int NG = D / G;
    uint32_t n[4][8], b[4][4];
    unsigned short p[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) p[t] = quantise8<T, G>(x[t], n[t]);
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

// Threads of a tile: D / 8 for its channels, 4 for its quads of tokens, K and V apart.
template <int D> __device__ __forceinline__ long long tile_of(long long i, int *j, int *ch, bool *is_v) {
    constexpr int C = D / 8;
    *ch = (int)(i % C) * 8;
    i /= C;
    *j = (int)(i & 3);
    *is_v = (i >> 2) & 1;
    return i >> 3;
}

// ---- a prompt as a whole ---------------------------------------------------------------------------
template <typename T, int D, int G>
__global__ void __launch_bounds__(kQ4Threads) q4_pack_kernel(Q4Cache C) {
    pg_wait_prior();
    pg_launch_dependents();
    const long long items = (long long)C.count * C.D.Hkv * C.Q.ptiles * D;  // 8 D / 8 threads a tile
    const long long step = (long long)gridDim.x * kQ4Threads;
    // (whole warps stay: a tile's threads are a multiple of 32)
    for (long long i = (long long)blockIdx.x * kQ4Threads + threadIdx.x; i < items; i += step) {
        int j, ch;
        bool is_v;
        const long long at = tile_of<D>(i, &j, &ch, &is_v);
        const long long unit = pg_div(at, C.Q.ptiles);
        const int tile = (int)(at - unit * C.Q.ptiles), s = (int)(unit / C.D.Hkv), h = (int)(unit - (long long)s * C.D.Hkv);
        const int len = C.len ? pg_clamp(__ldg(C.len + s), 0, C.D.n) : C.D.n;
        if (tile * kQ4Tile >= len) continue;
        const T *src = static_cast<const T *>(is_v ? C.V : C.K) +
                       (is_v ? s * C.v0 + h * C.v1 : s * C.s0 + h * C.s1) + ch;
        const long long row = is_v ? C.v2 : C.s2;
        float x[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int tok = tile * kQ4Tile + 2 * j + (t & 1) + 8 * (t >> 1);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[t][e] = 0.f;
            if (tok < len) load8(src + tok * row, x[t]);
        }
        uint8_t *dst = C.cache + (size_t)at * q4_tile_bytes(D, G);
        store_quad<T, D, G>(x, j, ch, is_v, dst);
    }
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

// A thread per row and 8 channels of K or V.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(Q4Cache C) {
    pg_wait_prior();
    pg_launch_dependents();
    constexpr int LPR = D / 8;
    const long long i = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
    const int ch = (int)(i % LPR) * 8;
    const bool is_v = (i / LPR) & 1;
    const long long at = pg_div(i / LPR >> 1, C.D.Hkv);
    const int h = (int)((i / LPR >> 1) - at * C.D.Hkv), row = (int)min(at, (long long)C.D.rows);
    int slot = -1;
    float x[8] = {};
    if (row < C.D.rows) slot = slot_of(C, row);
    if (slot >= 0)
        load8(static_cast<const T *>(is_v ? C.V : C.K) + row * (is_v ? C.v2 : C.s2) +
                  h * (is_v ? C.v1 : C.s1) + ch, x);
    uint8_t *tile = page_tile(C, max(slot, 0), h, q4_tile_bytes(D, G));
    // (lanes of a warp may be of K and of V, and of rows without a slot: the shuffles are among a group's lanes)
    uint32_t n[8], b[4];
    const unsigned short p = quantise8<T, G>(x, n);
    if (slot < 0) return;
    const int t = slot & 15;
    uint8_t *codes = tile + (is_v ? q4_codes(D) : 0);
    if (is_v) {
        pairs<true>(n, b);
        const int byte = ((t & 1) << 1) + (t >> 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            codes[q4_word<D>((((ch & 8) >> 1) + i) * 4 + ((t & 7) >> 1), ch >> 4) + byte] = (uint8_t)b[i];
    } else {
        pairs<false>(n, b);
        uint8_t *w = codes + q4_word<D>((t & 7) * 4 + (ch >> 3 & 3), ch >> 5 << 1) + (t >> 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[2 * i] = (uint8_t)b[i];
    }
    if (ch % G == 0)
        *reinterpret_cast<unsigned short *>(tile + 2 * q4_codes(D) + (is_v ? q4_params(D, G) : 0) +
                                            2 * (t * (D / G) + ch / G)) = p;
}

// ---- reading back ----------------------------------------------------------------------------------
__device__ __forceinline__ float value(uint32_t word, int bit, float s, float off) {
    // 2^23 + n, minus 2^23 + k: exact
    return (__uint_as_float((word >> bit & 15u) | 0x4B000000u) - off) * s;
}

template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    alignas(16) T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = from_f<T>(x[e]);
    reinterpret_cast<uint4 *>(p)[0] = reinterpret_cast<uint4 *>(v)[0];
    if (sizeof(T) == 4) reinterpret_cast<uint4 *>(p)[1] = reinterpret_cast<uint4 *>(v)[sizeof(T) / 4];
}

template <typename T, int D, int G, bool PAGES>
__global__ void __launch_bounds__(kQ4Threads) q4_unpack_kernel(Q4Cache C) {
    pg_wait_prior();
    pg_launch_dependents();
    constexpr int NG = D / G;
    const int tiles = (C.rows + kQ4Tile - 1) / kQ4Tile;
    const long long items = (long long)C.count * C.D.Hkv * tiles * D;
    const long long step = (long long)gridDim.x * kQ4Threads;
    for (long long i = (long long)blockIdx.x * kQ4Threads + threadIdx.x; i < items; i += step) {
        int j, ch;
        bool is_v;
        const long long at = tile_of<D>(i, &j, &ch, &is_v), unit = pg_div(at, tiles);
        const int tile = (int)(at - unit * tiles), s = (int)(unit / C.D.Hkv), h = (int)(unit - (long long)s * C.D.Hkv);
        const int len = C.len ? pg_clamp(__ldg(C.len + s), 0, C.rows) : C.rows, t0 = tile * kQ4Tile;
        if (t0 >= len) continue;
        const uint8_t *src;
        if (PAGES) {
            const int page = pg_page(C.table + (size_t)s * C.width, t0, C.D.lgP, C.D.npages, C.err);
            src = page_tile(C, (page << C.D.lgP) + (t0 & (C.D.P - 1)), h, q4_tile_bytes(D, G));
        } else {
            src = C.cache + ((size_t)unit * C.Q.ptiles + tile) * q4_tile_bytes(D, G);
        }
        const uint8_t *codes = src + (is_v ? q4_codes(D) : 0);
        const unsigned short *params = reinterpret_cast<const unsigned short *>(
            src + 2 * q4_codes(D) + (is_v ? q4_params(D, G) : 0));
        // w[t][i]: the byte of token t (in the order 2 j, 2 j + 1, 2 j + 8, 2 j + 9) of pair i, in its low 8 bits
        uint32_t w[4][4];
        if (is_v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = __ldg(reinterpret_cast<const uint32_t *>(
                    codes + q4_word<D>((((ch & 8) >> 1) + i) * 4 + j, ch >> 4)));
                w[0][i] = x;
                w[2][i] = x >> 8;
                w[1][i] = x >> 16;
                w[3][i] = x >> 24;
            }
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint2 x = __ldg(reinterpret_cast<const uint2 *>(
                    codes + q4_word<D>((2 * j + u) * 4 + (ch >> 3 & 3), ch >> 5 << 1)));
                w[u][0] = x.x;
                w[u + 2][0] = x.x >> 8;
                w[u][1] = x.x >> 16;
                w[u + 2][1] = x.x >> 24;
                w[u][2] = x.y;
                w[u + 2][2] = x.y >> 8;
                w[u][3] = x.y >> 16;
                w[u + 2][3] = x.y >> 24;
            }
        }
        T *dst = static_cast<T *>(is_v ? C.Vo : C.Ko) + (is_v ? s * C.v0 + h * C.v1 : s * C.s0 + h * C.s1) + ch;
        const long long row = is_v ? C.v2 : C.s2;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int tok = 2 * j + (t & 1) + 8 * (t >> 1);
            if (t0 + tok >= len) continue;
            const uint32_t p = __ldg(params + tok * NG + ch / G);
            const float step = __uint_as_float((p & 0xFFF0u) << 16);
            const float off = 8388608.f + (float)(p & 15u);
            float x[8];
            float lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = value(w[t][i], 0, step, off);
                hi[i] = value(w[t][i], 4, step, off);
            }
            if (is_v) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = lo[i];
                    x[2 * i + 1] = hi[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[(i & 1) + 4 * (i >> 1)] = lo[i];
                    x[(i & 1) + 4 * (i >> 1) + 2] = hi[i];
                }
            }
            store8(dst + (t0 + tok) * row, x);
        }
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
unsigned q4_blocks(long long items, int most) {
    const long long blocks = (items + kQ4Threads - 1) / kQ4Threads;
    return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_q4_pack(const Q4Cache &C, cudaStream_t st) {
    const long long items = (long long)C.count * C.D.Hkv * C.Q.ptiles * C.D.d;
    return by_type(C.D.dtype, [&](auto t) {
        return by_sizes(C.Q, [&](auto d, auto g) {
            return pg_launch(q4_pack_kernel<decltype(t), decltype(d)::value, decltype(g)::value>,
                             q4_blocks(items, kPgSms * 64), kQ4Threads, 0, true, st, C);
        });
    });
}

cudaError_t launch_q4_append(const Q4Cache &C, cudaStream_t st) {
    const long long items = (long long)C.D.rows * C.D.Hkv * 2 * (C.D.d / 8);
    return by_type(C.D.dtype, [&](auto t) {
        return by_sizes(C.Q, [&](auto d, auto g) {
            return pg_launch(q4_append_kernel<decltype(t), decltype(d)::value, decltype(g)::value>,
                             q4_blocks(items, 0x7fffffff), kQ4Threads, 0, true, st, C);
        });
    });
}

cudaError_t launch_q4_unpack(const Q4Cache &C, cudaStream_t st) {
    const long long items = (long long)C.count * C.D.Hkv * ((C.rows + kQ4Tile - 1) / kQ4Tile) * C.D.d;
    return by_type(C.D.dtype, [&](auto t) {
        return by_sizes(C.Q, [&](auto d, auto g) {
            constexpr int D = decltype(d)::value, G = decltype(g)::value;
            auto kern = C.table ? q4_unpack_kernel<decltype(t), D, G, true>
                                : q4_unpack_kernel<decltype(t), D, G, false>;
            return pg_launch(kern, q4_blocks(items, kPgSms * 64), kQ4Threads, 0, true, st, C);
        });
    });
}

}  // namespace kve
