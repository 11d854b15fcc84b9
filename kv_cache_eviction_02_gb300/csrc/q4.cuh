// Cache in 4 bits: its layout, and what the kernels that write, read and attend to it share (q4_*.cu).
//
// A row of a KV head is held in groups of G channels, each as whole numbers m of 16 neighbouring ones and a
// step s of four significant bits, for the values s m. s m has at most 8 significant bits, so it is
// exact in bf16 (and in fp16 wherever that reaches), and a product of two operands that the tensor cores take is
// a product with the value itself. Codes n = m + k are 0 .. 15; a group's parameter is s as bf16, whose last four
// bits are 0, with k in them (0x7FF0, a NaN: the group stands for NaN).
//
// Codes lie in the order in which the warps of q4_attn.cu read them: a tile of 16 tokens is one contiguous block
// [K codes][V codes][K parameters][V parameters], read by one bulk copy. A lane's word for 16 channels is the A
// operand of an m16n8k16 product: a nibble at bit 0 or 4 of each half is the fp16 number n 2^-24 or n 2^-20 as it
// stands (below fp16's normal numbers, which the tensor cores multiply exactly), so a word takes four ANDs
// and one shift. Every byte of a word belongs to one token, so tokens of a tile can be written apart.
//   K: lane 4 r + j (r < 8, j < 4), words 2 c, 2 c + 1: channels 32 c + 8 j .. + 7 of tokens r (bytes 0 and 2) and
//      r + 8 (bytes 1 and 3); channels e, e + 2 (e = 0, 1 mod 4) in the low and high nibble of a byte
//   V: lane 4 r + j, word c: channels 16 c + 2 r (low nibble) and + 1 (high) of tokens 2 j (byte 0), 2 j + 8 (1),
//      2 j + 1 (2), 2 j + 9 (3)
//   parameters: [16 tokens][groups]
// A lane's words lie in pieces of 16 bytes (8 with d_head 32), lane after lane.
#pragma once

#include <type_traits>

#include "pages_ptx.cuh"

namespace kve {

constexpr int kQ4Tile = 16;  // tokens
__host__ __device__ constexpr int q4_codes(int d) { return 8 * d; }              // bytes, K or V of a tile
__host__ __device__ constexpr int q4_params(int d, int group) { return 32 * (d / group); }
__host__ __device__ constexpr int q4_tile_bytes(int d, int group) {
    return 2 * (q4_codes(d) + q4_params(d, group));
}
// byte offset of word w of a lane among its K (or V) codes
template <int D> __host__ __device__ constexpr int q4_word(int lane, int w) {
    constexpr int per = D == 32 ? 8 : 16;
    return (w >> 2) * 512 + lane * per + (w & 3) * 4;
}

template <int D> __host__ __device__ constexpr int q4_lane(int lane) { return lane * (D == 32 ? 8 : 16); }

constexpr unsigned short kQ4Nan = 0x7FF0;

// A 4-bit array as the kernels see it: tiles [block][KV head][tiles_per_block], a block being a prompt or a page.
struct Q4Shape {
    int d, group, tile;  // bytes per tile
    int ptiles;          // tiles per prompt and KV head
    bool wide;           // prompts are read back into 16-bit arrays first, for many row tiles
};

// Calls of the cache's own kernels.
struct Q4Cache {
    PgDims D;
    Q4Shape Q;
    const void *K, *V;  // 16-bit or fp32 rows
    void *Ko, *Vo;
    long long s0, s1, s2;  // strides (elements) of prompt or request, head, row; V's
    long long v0, v1, v2;
    uint8_t *cache;
    const int32_t *table, *len, *slots;
    int count, width, rows;  // prompts or requests, table entries each, rows that the arrays have
    unsigned *err;
};
cudaError_t launch_q4_pack(const Q4Cache &C, cudaStream_t st);
cudaError_t launch_q4_append(const Q4Cache &C, cudaStream_t st);
cudaError_t launch_q4_unpack(const Q4Cache &C, cudaStream_t st);

// Sizes and splits of an attention call over 4-bit arrays; its partial results are joined by launch_pg_join.
// A.Kp is the prompts' array, A.K the pages'.
bool q4_dims(const KvePgShape *sh, int group, PgDims *D, Q4Shape *Q, const char **why);
PgWorkspace q4_ws_layout(const PgDims &D, const Q4Shape &Q);
unsigned long long q4_segs(const PgDims &D);
template <typename T>  // partial results over the prompts, or over the own rows of requests with many new ones
cudaError_t launch_q4_tc(const PgDims &D, const Q4Shape &Q, const PgAttn &A, bool own, cudaStream_t st);
extern template cudaError_t launch_q4_tc<__nv_bfloat16>(const PgDims &, const Q4Shape &, const PgAttn &, bool, cudaStream_t);
extern template cudaError_t launch_q4_tc<__half>(const PgDims &, const Q4Shape &, const PgAttn &, bool, cudaStream_t);
cudaError_t launch_q4_lines(const PgDims &D, const Q4Shape &Q, const PgAttn &A, cudaStream_t st);

// ---- device helpers --------------------------------------------------------------------------------
// one contiguous block into shared memory; addresses and size are multiples of 16 bytes
__device__ __forceinline__ void q4_bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(tc::smem_u32(bar))
        : "memory");
}

// A lane's words of a tile's K or V codes (shared-memory addresses, the lane's own offset among them).
template <int D> __device__ __forceinline__ void q4_words(uint32_t at, uint32_t (&w)[D / 16]) {
    if constexpr (D == 32) {
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                         : "r"(at + i * 512)
                         : "memory");
    }
}
// The parameters of a token: NG of 16 bits in (NG + 1) / 2 words.
template <int NG> __device__ __forceinline__ void q4_params_of(uint32_t at, uint32_t (&w)[(NG + 1) / 2]) {
    if constexpr (NG == 4)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    else if constexpr (NG == 2)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
    else
        asm volatile("{\n\t.reg .u16 x;\n\tld.shared.u16 x, [%1];\n\tcvt.u32.u16 %0, x;\n\t}" : "=r"(w[0]) : "r"(at) : "memory");
}

// Codes as values of a 16-bit type, two at a time: p2 holds the parameters of the two, low() takes the nibbles at bits 0
// and 16, high() those at bits 4 and 20. Exact, but for fp16: values below its normal numbers round once, those above its
// largest are infinities.
template <typename T> struct Q4Codes;
template <> struct Q4Codes<__nv_bfloat16> {
    uint32_t s, k;
    __device__ __forceinline__ explicit Q4Codes(uint32_t p2, bool = true) : s(p2 & 0xFFF0FFF0u), k((p2 & 0x000F000Fu) | 0x43004300u) {}
    __device__ __forceinline__ uint32_t of(uint32_t low_nibbles) const {
        const uint32_t x = (low_nibbles & 0x000F000Fu) | 0x43004300u;  // 128 + n
        const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x),
                                                 *reinterpret_cast<const __nv_bfloat162 *>(&k)),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&s));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    __device__ __forceinline__ uint32_t low(uint32_t x) const { return of(x); }
    __device__ __forceinline__ uint32_t high(uint32_t x) const { return of(x >> 4); }
};
template <> struct Q4Codes<__half> {
    // a code at bits 4 to 7 of 64's mantissa is 64 + n; step = a e, a of four bits below 2 and e a power of two: (64 + n) a - (64 + k) a
    // has 11 bits at most and only the product with e can round. zero: 0, or NaN where e is none
    uint32_t a, c, e, zero;
    __device__ __forceinline__ static __half2 h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
    __device__ __forceinline__ static uint32_t u(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }
    // Whether fp16 does not have the power of two of a parameter, least .. most, in either half of the words of which
    // y is the maximum of beyond(word).
    static constexpr uint32_t kLeast = 103u << 23, kMost = 142u << 23, kNone = 255u << 23;  // 2^-24, 2^15; NaN's
    __device__ __forceinline__ static uint32_t beyond(uint32_t p2) {  // (a borrow leaves its half far outside)
        return (p2 & 0x7F807F80u) - (kLeast >> 16) * 0x10001u;
    }
    __device__ __forceinline__ static bool far(uint32_t y) {
        constexpr uint32_t span = ((kMost - kLeast) >> 16) * 0x10001u;
        return __vmaxu2(y, span) != span;
    }
    // check: the parameters may be such ones
    __device__ __forceinline__ explicit Q4Codes(uint32_t p2, bool check = true) {
        a = (p2 & 0x00700070u) << 3 | 0x3C003C00u;
        const uint32_t e0 = p2 << 16 & 0x7F800000u, e1 = p2 & 0x7F800000u;
        e = u(__floats2half2_rn(__uint_as_float(e0), __uint_as_float(e1)));
        // a takes what lies below the least power of two or, above the largest, a factor of two, with which every code
        // but 0 is an infinity (0 stays 0). NaN steps keep their infinite e.
        if (check && far(beyond(p2))) {
            auto rest = [](uint32_t x) { return x < kLeast ? __uint_as_float(x) * 0x1p24f : (x > kMost ? 2.f : 1.f); };
            auto held = [](uint32_t x) { return __uint_as_float(x == kNone ? x : min(max(x, kLeast), kMost)); };
            a = u(__hmul2(h2(a), __floats2half2_rn(rest(e0), rest(e1))));
            e = u(__floats2half2_rn(held(e0), held(e1)));
        }
        c = u(__hmul2(h2((p2 << 4 & 0x00F000F0u) | 0xD400D400u), h2(a)));  // -(64 + k) a
        zero = check ? u(__hmul2(h2(e), h2(0u))) : 0u;
    }
    __device__ __forceinline__ uint32_t high(uint32_t x) const {
        return u(__hfma2(__hfma2(h2((x & 0x00F000F0u) | 0x54005400u), h2(a), h2(c)), h2(e), h2(zero)));
    }
    __device__ __forceinline__ uint32_t low(uint32_t x) const { return high(x << 4); }
};

// The same of all parameters of N tokens, NG each: whether Q4Codes have to look at them one by one. All lanes call.
template <typename T, int NG, int N> __device__ __forceinline__ bool q4_any_far(const uint32_t (&p)[N][(NG + 1) / 2]) {
    if constexpr (std::is_same<T, __half>::value) {
        uint32_t y = 0;
#pragma unroll
        for (int t = 0; t < N; t += NG == 1 ? 2 : 1)
#pragma unroll
            for (int i = 0; i < (NG + 1) / 2; ++i)
                y = __vmaxu2(y, Q4Codes<T>::beyond(NG == 1 ? __byte_perm(p[t][0], p[(t + 1) % N][0], 0x5410) : p[t][i]));
        return __any_sync(0xffffffffu, Q4Codes<T>::far(y));
    }
    return false;
}

}  // namespace kve
