// Cache in 4 bits: attention over prompts and pages by warps, a lane's codes as tensor-core operands as they stand.
//
// Few query rows (a decode step's g heads per KV head) read all of a cache: bound by HBM, then by the
// instructions that a code costs. The products run transposed, S^T = K Q^T and O^T += V^T P^T, as
// m16n8k16 fragments of fp16 numbers whose A operand is the cache's own words (q4.cuh): no code is converted, a
// nibble is the number n 2^-24 or n 2^-20. With a group's step and zero code taken out of the sums,
//   q.k = sum over groups of s_g (q_g.n_g - k_g sum q_g),   o_c = sum over tokens of (p_t s_t,g) (n_t,c - k_t,g),
// a score is a product per group, times s in fp32, and the terms of the zero codes are products too: A holds k_g of
// the 16 tokens, B the sums of q (as two fp16 numbers, off by 2^-22), or the same weights p s as the codes'.
// Queries are carried as fp16 after their row's largest entry is brought to 2^7 .. 2^8 (bf16 and fp16 entries keep all
// their bits down to 2^-17 of the largest, smaller ones are off by 2^-28 of it; fp32 ones are two fp16
// numbers). Weights p s are fp32 numbers rounded once to fp16, half a step (fp32: two fp16 numbers).
//
// Work is dealt out as in pages_own.cu: units (request or prompt, KV head, 8 or 16 query rows) and their tiles of 16
// tokens in one line, equal shares for all CTAs (one per SM) and in them for their warps, a ring of tiles per warp that
// runs on across units. A tile is one contiguous block: one bulk copy by one lane. Pieces of a unit that several
// warps of a CTA have seen are joined in shared memory, so a CTA hands on one partial result of a unit.
//
// One request behind 128K rows (32/8 heads of d 128, groups of 32, 151 MB): 44.5 us, of which the set-up until the first
// product takes 3.5, the tiles 32 (4.8 TB/s), the join 8. 64 requests with caches of up to 16K rows (groups of 64, 572
// MB): 122 us, 4.7 TB/s, 295 instructions a tile and warp, the logic unit busy for 0.54 of the time and a warp's own
// dependent instructions most of the rest: 12 warps an SM are what the registers hold. What was measured and not
// kept: 16 warps with spills (59 -> 60 us), codes made normal numbers for bf16 too (V's 43 -> 47 us, K's and V's 53),
// units of 16 query rows (109 -> 121), shifts as multiplications (124 -> 136), the join in this kernel by tickets (43 ->
// 69: waits on atomics, and few warps for the join).
#include <type_traits>

#include "q4.cuh"

namespace kve {
namespace {

// Weights p s are fp16 numbers, carried up to 2^15 of a reference m that all groups of a row share: it is set 2^7 below
// the largest, of the row's tokens and groups. That holds every group's bits as long as the steps of each token's groups
// lie within 2^12 (fp32: 2^10) of one another and are not below 2^-32 less that, since no group's largest weight is then
// further below: nothing above 2^-20 (2^-22) of it is lost. Tokens whose steps lie further apart raise m by their least
// step only, as far as 2^-80 of the largest, so that their weights may be any fp32 numbers, and are brought to 2^7 .. 2^8
// group by group, a tile at a time, and the products back into the sums (V's groups 2^20 apart: 64 caches 260 us for
// 122, one request behind 128K 91 for 44.5). Groups of zeros would be such steps, on every token of a head that is
// padded: those that a piece of a unit has only seen as zeros stay out of it (138 and 50 us). If one comes alive after
// all, m may stand too high for it, and all further tiles of the piece take the longer way.
constexpr float kLnUp = 7.f, kLnGrow = 15.f, kLnLeastStep = 0x1p-32f, kLnFar = 0x1p-80f, kLnZeroStep = 0x1p-126f;

// The tensor cores cut the sums' bits at 2^-24 of the largest product's exponent, which for a number as it stands in the
// cache counts as 2^-14: to 2^-17 of a product of V's. That is enough for outputs of bf16 (2^-9). For fp16 and fp32 V's
// codes (for fp32 K's too) are made normal numbers n - k, by one subtraction from 1024 + n.
enum { kLnBf16, kLnF16, kLnF32 };

// A unit's set-up (its queries, its pages' numbers, a first tile from memory, its result) takes a warp as long as some
// tiles: so many that it counts for in the line, before its own (4 requests of a few own rows behind 16K rows: without,
// the one CTA with all the own rows ends 6 us after the others; 25.5 -> 20.0 us).
constexpr int kLnPad = 3;

constexpr int kLnStage = 2;  // tiles per ring place: at most, of one unit
// One CTA per SM, of as many warps as its registers hold, and a ring of what shared memory has room for.
template <int D, int G, int NT, int MODE> struct Ln {
    static constexpr int WARPS = NT == 2 && D == 128 ? 8 : 12, THREADS = 32 * WARPS, RB = 8 * NT;
    static constexpr int TB = q4_tile_bytes(D, G), SB = kLnStage * TB;
    static constexpr int ROW = D + 4;                    // floats per row of a piece in shared memory
    static constexpr int PIECE = RB * ROW * 4 + RB * 8;  // o [RB][ROW], (m, l) [RB]
    static constexpr int FIT = ((227 * 1024 - 12 * 1024) / WARPS - PIECE) / SB, NST = FIT < 6 ? FIT : 6;
    static constexpr int WARP = NST * SB + PIECE;        // bytes per warp: ring, first piece
    static constexpr int SMEM = WARPS * WARP + 128;
    static_assert(NST >= 2 && PIECE <= NST * SB && SB % 16 == 0 && PIECE % 16 == 0);
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same onto zeros
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                     uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}
__device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float y;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int NG> __device__ __forceinline__ void steps_of(const uint32_t (&w)[(NG + 1) / 2], float (&s)[NG]) {
#pragma unroll
    for (int g = 0; g < NG; ++g)
        s[g] = __uint_as_float((g & 1 ? w[g >> 1] : w[g >> 1] << 16) & 0xFFF00000u);
}
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u, k1024 = 0x64006400u;

template <int D, int G, int NT, int MODE>
__global__ void __launch_bounds__(Ln<D, G, NT, MODE>::THREADS, 1)
    q4_line_kernel(PgDims D_, PgAttn A, PgOwn W, int ptiles) {
    using L = Ln<D, G, NT, MODE>;
    constexpr int NST = L::NST, TB = L::TB, SB = L::SB, RB = L::RB, WARPS = L::WARPS, THREADS = L::THREADS;
    constexpr bool F32 = MODE == kLnF32, KC = F32, VC = MODE != kLnBf16;  // codes less their zero codes, of K and of V
    constexpr int NG = D / G, KW = D / 16, PW = (NG + 1) / 2, NS = F32 ? 2 : 1;
    constexpr float kApart = F32 ? 0x1p10f : 0x1p12f;  // how far steps lie apart at most
    constexpr int kFresh = 1 << NG;
    constexpr bool PAIR = NT == 1;  // two tiles at once: one alone leaves the warps waiting for its products
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ long long csum[THREADS + 1];
    __shared__ int usum[THREADS + 1];
    __shared__ uint64_t bars[WARPS][NST];
    __shared__ int piece_unit[2 * WARPS], piece_rows[2 * WARPS];  // of a warp's first and last piece: -1 or what joins
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane & 3;
    if (lane < NST) tc::mbar_init(&bars[warp][lane], 1);
    if (lane < 2) piece_unit[2 * warp + lane] = -1;
    if (threadIdx.x == 0) s_abort = 0;
    tc::mbar_fence_init();
    if (D_.np == 0) pg_wait_prior();  // first kernel of its call (else the prompts' has waited)
    pg_launch_dependents();

    const int e0 = F32 || D_.line ? 0 : D_.S, ents = D_.S + D_.R - e0;  // the line's first entity, and how many
    auto entity = [&](int e, int *cr, int *nb) {
        int len, first, nq, rows;
        pg_unit_entity<F32>(D_, A, e + e0, &len, &first, &nq, &rows, cr, nb);
    };
    PgShare sh{};
    long long X0, x = 0;
    int n = 0, e = 0, unit = 0;  // tiles of this warp; where they begin: entity, tiles into it, units before it
    auto mine = [&]() {
        X0 = blockIdx.x * sh.cpw;
        const long long all = min(sh.total - X0, sh.cpw);  // of the CTA
        if (all <= 0) return;
        const long long from = pg_div(all * warp, WARPS);
        n = (int)(pg_div(all * (warp + 1), WARPS) - from);
        X0 += from;
    };
    if (ents <= 32) {  // every warp by itself, an entity per lane
        int cr = 0, nb = 0;
        if (lane < ents) entity(lane, &cr, &nb);
        const int us = nb * D_.Hkv;
        const long long cs = (long long)(cr + kLnPad) * us;
        long long c = cs;
        int u = us;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, c, o);
            const int z = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) {
                c += y;
                u += z;
            }
        }
        const int longest = __reduce_max_sync(0xffffffffu, nb > 0 ? cr : 0);
        sh.total = __shfl_sync(0xffffffffu, c, 31);
        sh.cpw = pg_per_share(sh.total, gridDim.x, longest);
        if (blockIdx.x == 0 && warp == 0) {
            if (lane < ents) {
                W.base[lane] = c - cs;
                W.unit[lane] = u - us;
            }
            if (lane == 0) *W.cpw = sh.cpw;
        }
        mine();
        e = __popc(__ballot_sync(0xffffffffu, c <= X0)) & 31;
        x = X0 - __shfl_sync(0xffffffffu, c - cs, e);
        unit = __shfl_sync(0xffffffffu, u - us, e);
    } else {
        sh = pg_share<THREADS, 1>(ents, D_.Hkv, csum, usum, W, entity, kLnPad);
        mine();
        pg_share_find<THREADS>(csum, usum, sh, X0, &e, &x, &unit);
    }
    __syncthreads();  // s_abort and the pieces' marks are set
    PgCursor<F32> cc;
    if (n > 0) {
        cc.enter(D_, A, e + e0);
        auto tiles = [&]() { return (long long)(cc.cr + kLnPad) * cc.nb * D_.Hkv; };
        while (x >= tiles()) {
            x -= tiles();
            unit += cc.nb * D_.Hkv;
            cc.enter(D_, A, cc.e + 1);
        }
        const int u = (int)pg_div(x, cc.cr + kLnPad);
        cc.c = (int)(x - (long long)u * (cc.cr + kLnPad)) - kLnPad;
        cc.kh = u / cc.nb;
        cc.rb = u - cc.kh * cc.nb;
        unit += u;
        if (cc.c < 0) {  // the share begins in the unit's set-up
            n += cc.c;
            cc.c = 0;
        }
    }
    if (n > 0) {
        PgCursor<F32> ca = cc;  // runs ahead: the tiles to load

        uint8_t *ring = smem + warp * L::WARP;
        uint64_t *bar = bars[warp];
        volatile int *abort_flag = &s_abort;
        // ---- queries of a unit ----
        constexpr int QW = F32 ? 2 : 1;
        uint4 raw[NT][D / 32][QW];        // this lane's channels 32 c + 8 j .. of query row lane / 4 of each block
        uint32_t qf[NT][NS][KW][2];       // B operand of S^T
        uint32_t zq[NT][2];               // minus the sums of q over groups 2 (j & 1), + 1
        float fc[NT][2];                  // from the products to log2 units, for this lane's columns 2 j, + 1
        float o[NT][KW][4], z[NT][4], m[NT][2], l[NT][2];
        int see[NT][2], see_least = 0, rows, row0;  // tokens that columns see; the tiles that all of them see whole
        const float k1 = kLog2e * rsqrtf((float)D);
        int dead;  // groups of V that were zeros in all tiles so far; kFresh: before the first, -1: one came alive
        uint32_t zmask[NG], rmask[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            zmask[g] = (j & 1) == g >> 1 ? (g & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
            rmask[g] = lane >> 2 == g ? ~0u : 0u;
        }
        auto ask_q = [&]() {
            rows = cc.rows;
            row0 = cc.rb * RB;
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                const int rr = row0 + 8 * b + (lane >> 2), t = rr < rows ? rr / D_.g : 0;
                const size_t at = (cc.first + t) * A.q_row +
                                  (size_t)(cc.kh * D_.g + (rr < rows ? rr - t * D_.g : 0)) * D + j * 8;
                const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(A.q) + at * (F32 ? 4 : 2));
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
#pragma unroll
                    for (int i = 0; i < QW; ++i) {
                        raw[b][c][i] = make_uint4(0, 0, 0, 0);
                        if (rr < rows) raw[b][c][i] = __ldg(p + c * (F32 ? 8 : 4) + i);
                    }
            }
        };
        auto begin = [&]() {  // of a unit, or of this warp's part of one, when its queries are there
            see_least = 0x7fffffff;
            dead = kFresh;
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(raw[b]);
                auto value = [&](int i) {
                    if (F32) return __uint_as_float(w[i]);
                    if (MODE == kLnF16) {
                        const float2 f = unpack(w[i >> 1]);
                        return i & 1 ? f.y : f.x;
                    }
                    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
                };
                float most = 0.f;
                if (F32) {
#pragma unroll
                    for (int i = 0; i < D / 4; ++i) most = fmaxf(most, fabsf(value(i)));
                } else {  // magnitudes as whole numbers, two at a time
                    uint32_t x = 0;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) x = __vmaxu2(x, w[i] & 0x7FFF7FFFu);
                    x = max(x >> 16, x & 0xFFFFu);
                    most = MODE == kLnF16 ? unpack(x).x : __uint_as_float(x << 16);
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const int ex = most == 0.f ? 127 : min(max((int)(__float_as_uint(most) >> 23), 27), 230);
                const float up = __uint_as_float((261 - ex) << 23);               // 2^(7 - exponent)
                const float back = k1 * __uint_as_float((KC ? ex - 7 : ex + 17) << 23);  // 1 / up, with 2^24 for K's codes
#pragma unroll
                for (int e = 0; e < 2; ++e) fc[b][e] = __shfl_sync(0xffffffffu, back, (2 * j + e) * 4);
#pragma unroll
                for (int k = 0; k < KW; ++k)  // 4 channels of this word's
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float f = h ? up * 0.0625f : up;  // (the second pair's codes stand 2^4 higher)
                        float a = value(4 * k + 2 * h) * f, c = value(4 * k + 2 * h + 1) * f;
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            const uint32_t y = pack(a, c);
                            qf[b][i][k][h] = y;
                            const float2 r = unpack(y);
                            a -= r.x;
                            c -= r.y;
                        }
                    }
                if (!KC) {  // sums over groups: a product with ones (and 2^4 for the second pairs)
                    constexpr uint32_t k1 = 0x3C003C00u, k16 = 0x4C004C00u;
                    float sum[NG];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float c[4];
#pragma unroll
                        for (int k = g * G / 16; k < (g + 1) * G / 16; ++k) {
                            const uint32_t(&f)[2] = qf[b][0][k];
                            if (k == g * G / 16) mma0(c, k1, k1, k16, k16, f[0], f[1]);
                            else mma(c, k1, k1, k16, k16, f[0], f[1]);
                        }
                        // column lane / 4, which lanes with j = lane / 8 hold
                        const float s0 = __shfl_sync(0xffffffffu, c[0], lane >> 3);
                        const float s1 = __shfl_sync(0xffffffffu, c[1], lane >> 3);
                        sum[g] = -(lane & 4 ? s1 : s0);
                    }
                    const float a = NG > 2 && (j & 1) ? sum[NG > 2 ? 2 : 0] : (j & 1 ? 0.f : sum[0]);
                    const float c = NG > 2 && (j & 1) ? sum[NG > 2 ? 3 : 0] : (j & 1 || NG == 1 ? 0.f : sum[NG > 1 ? 1 : 0]);
                    const uint32_t y = pack(a, c);
                    const float2 r = unpack(y);
                    zq[b][0] = j < 2 ? y : 0u;
                    zq[b][1] = j < 2 ? pack(a - r.x, c - r.y) : 0u;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int qr = row0 + 8 * b + j * 2 + e;
                    see[b][e] = qr >= rows ? 0 : (cc.e < D_.S ? cc.len : cc.len - cc.nq + 1 + qr / D_.g);
                    if (qr < rows) see_least = min(see_least, see[b][e]);
                    m[b][e] = kPgNoMax;
                    l[b][e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) z[b][e] = 0.f;
#pragma unroll
                for (int k = 0; k < KW; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[b][k][e] = 0.f;
            }
            see_least = max(__reduce_min_sync(0xffffffffu, see_least), 0) / kQ4Tile;
        };
        // ---- tiles on their way ----
        // A stage is a pair of tiles, the even one first, or one where a piece begins or ends between them. A request's
        // pages are asked for 32 at a time, a lane each, and 32 ahead of those in use: the table's answer (a trip to L2)
        // is not waited for.
        const int tpp = D_.lgP - 4, tmask = (1 << tpp) - 1;  // tiles per page: log2, less one
        const uint32_t page_bytes = ((uint32_t)D_.Hkv << tpp) * TB;
        auto stage_of = [&](int c, int end) { return min(kLnStage - (c & 1), end - c); };
        int fill = 0, togo = n, end = min(ca.cr, ca.c + n);  // of the piece that is being loaded
        const uint8_t *base;
        int pages = 0, ahead = 0, page0 = 0;  // this lane's page of the 32 from page0 on, and of the next 32
        auto ask_pages = [&](int from) {
            const int p = from + lane;
            if (p > (ca.cr - 1) >> tpp) return 0;
            return __ldg(A.table + (size_t)(ca.e - D_.S) * D_.maxp + p);
        };
        auto enter = [&]() {  // the piece to load
            if (ca.e < D_.S) {
                base = static_cast<const uint8_t *>(A.Kp) + ((size_t)ca.e * D_.Hkv + ca.kh) * ptiles * TB;
            } else {
                base = static_cast<const uint8_t *>(A.K) + ((size_t)ca.kh << tpp) * TB;
                page0 = (ca.c >> tpp) & ~31;
                pages = ask_pages(page0);
                ahead = ask_pages(page0 + 32);
            }
        };
        auto load = [&]() {
            const int t = stage_of(ca.c, end);
            const uint8_t *src = base, *src1 = nullptr;
            if (ca.e < D_.S) {
                src += (size_t)ca.c * TB;
            } else {
                if ((ca.c >> tpp) - page0 == 32) {
                    page0 += 32;
                    pages = ahead;
                    ahead = ask_pages(page0 + 32);
                }
                auto page_at = [&](int c) {
                    return base + (size_t)pg_page_id(__shfl_sync(0xffffffffu, pages, (c >> tpp) & 31), D_.npages, A.err) *
                                      page_bytes;
                };
                src = page_at(ca.c) + (ca.c & tmask) * TB;
                if (tmask == 0 && t == 2) src1 = page_at(ca.c + 1);
            }
            if (tc::elect_one()) {
                tc::mbar_expect_tx(&bar[fill], t * TB);
                q4_bulk_load(ring + fill * SB, src, src1 ? TB : t * TB, &bar[fill]);
                if (src1) q4_bulk_load(ring + fill * SB + TB, src1, TB, &bar[fill]);
            }
            if (++fill == NST) fill = 0;
            ca.c += t;
            togo -= t;
            if (ca.c == end && (togo -= kLnPad) > 0) {
                --ca.c;
                ca.next(D_, A);
                end = min(ca.cr, togo);
                enter();
            }
        };
        ask_q();
        enter();
#pragma unroll 1
        for (int i = 0; i < NST - 1 && togo > 0; ++i) load();
        begin();

        int slot = 0, left = n;  // ring place of this stage; tiles that are not done
        int starts = cc.c;       // the piece's first tile of its unit
        uint32_t phase = 0;
        const uint32_t ring_at = tc::smem_u32(ring);
        const uint32_t codes_at = q4_lane<D>(lane), param_at = 2 * q4_codes(D) + (lane >> 2) * (2 * NG);
#pragma unroll 1
        while (left > 0) {
            if (togo > 0) load();
            const int nt = stage_of(cc.c, min(cc.cr, cc.c + left));
            if (!tc::mbar_wait_warp(&bar[slot], phase, abort_flag, A.err)) break;
            uint32_t tile = ring_at + slot * SB;
            if (++slot == NST) {
                slot = 0;
                phase ^= 1;
            }
            int tok = cc.c * kQ4Tile + (lane >> 2);
            // false: nothing done, since steps lie apart, which a masked tile alone takes
            auto work = [&](auto tiles, auto masked) {
                constexpr int TT = decltype(tiles)::value;
                constexpr bool MASK = decltype(masked)::value, ALONE = MASK && TT == 1;
                // scores: 16 tokens x 8 query rows per tile and block, a group at a time
                float s[TT][NT][4];
                {
                    uint32_t kw[TT][KW], kp[TT][2][PW];
                    float sk[TT][2][NG];
#pragma unroll
                    for (int i = 0; i < TT; ++i) {
                        q4_words<D>(tile + i * TB + codes_at, kw[i]);
                        q4_params_of<NG>(tile + i * TB + param_at, kp[i][0]);
                        q4_params_of<NG>(tile + i * TB + param_at + 16 * NG, kp[i][1]);
                    }
#pragma unroll
                    for (int i = 0; i < TT; ++i) {
                        steps_of<NG>(kp[i][0], sk[i][0]);
                        steps_of<NG>(kp[i][1], sk[i][1]);
                    }
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float c[TT][NT][4];
                        uint32_t kc[TT][4];  // 1024 + zero code, of both tokens and of codes 2^4 higher
#pragma unroll
                        for (int i = 0; i < TT; ++i) {
                            if (KC) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t x = __byte_perm(kp[i][h][g >> 1], 0, g & 1 ? 0x3232 : 0x1010);
                                    kc[i][h] = (x & kLow) | k1024;
                                    kc[i][h + 2] = (x << 4 & kHigh) | k1024;
                                }
                                continue;
                            }
                            const uint32_t z0 = (NG == 4 && (j & 1) ? kp[i][0][PW - 1] : kp[i][0][0]) & kLow;
                            const uint32_t z1 = (NG == 4 && (j & 1) ? kp[i][1][PW - 1] : kp[i][1][0]) & kLow;
#pragma unroll
                            for (int b = 0; b < NT; ++b)
                                mma0(c[i][b], z0, z1, z0, z1, zq[b][0] & zmask[g], zq[b][1] & zmask[g]);
                        }
#pragma unroll
                        for (int k = g * G / 16; k < (g + 1) * G / 16; ++k)
#pragma unroll
                            for (int i = 0; i < TT; ++i) {
                                const uint32_t x = kw[i][k], h = x >> 8;
                                uint32_t a0 = x & kLow, a1 = h & kLow, a2 = x & kHigh, a3 = h & kHigh;
                                if (KC) {
                                    a0 = minus(a0 | k1024, kc[i][0]);
                                    a1 = minus(a1 | k1024, kc[i][1]);
                                    a2 = minus(a2 | k1024, kc[i][2]);
                                    a3 = minus(a3 | k1024, kc[i][3]);
                                }
#pragma unroll
                                for (int b = 0; b < NT; ++b)
#pragma unroll
                                    for (int y = 0; y < NS; ++y) {
                                        const uint32_t(&f)[2] = qf[b][y][k];
                                        if (KC && k == g * G / 16 && y == 0) mma0(c[i][b], a0, a1, a2, a3, f[0], f[1]);
                                        else mma(c[i][b], a0, a1, a2, a3, f[0], f[1]);
                                    }
                            }
#pragma unroll
                        for (int i = 0; i < TT; ++i)
#pragma unroll
                            for (int b = 0; b < NT; ++b)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    s[i][b][e] = g == 0 ? sk[i][e >> 1][0] * c[i][b][e]
                                                        : fmaf(sk[i][e >> 1][g], c[i][b][e], s[i][b][e]);
                    }
                }
                uint32_t vw[TT][KW], vp[TT][2][PW];
                float sv[TT][2][NG], least[TT][2], far = 0.f;
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    q4_words<D>(tile + i * TB + codes_at + q4_codes(D), vw[i]);
                    q4_params_of<NG>(tile + i * TB + param_at + q4_params(D, G), vp[i][0]);
                    q4_params_of<NG>(tile + i * TB + param_at + q4_params(D, G) + 16 * NG, vp[i][1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // (groups that hold no number are left out)
                        steps_of<NG>(vp[i][h], sv[i][h]);
                        float hi = kLnLeastStep, lo = sv[i][h][0];
                        if constexpr (NG == 4) {
                            hi = tc::max3(tc::max3(hi, sv[i][h][0], sv[i][h][1]), sv[i][h][2], sv[i][h][3]);
                            lo = fminf(min3(lo, sv[i][h][1], sv[i][h][2]), sv[i][h][3]);
                        } else if constexpr (NG == 2) {
                            hi = tc::max3(hi, sv[i][h][0], sv[i][h][1]);
                            lo = fminf(lo, sv[i][h][1]);
                        } else {
                            hi = fmaxf(hi, lo);
                        }
                        far = fmaxf(far, fmaf(-kApart, lo, hi));
                        least[i][h] = lg2_approx(hi);
                    }
                }
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < TT; ++i) {
                            s[i][b][e] *= fc[b][e];
                            s[i][b][e + 2] *= fc[b][e];
                            if (MASK) {
                                if (tok + 16 * i >= see[b][e]) s[i][b][e] = -INFINITY;
                                if (tok + 16 * i + 8 >= see[b][e]) s[i][b][e + 2] = -INFINITY;
                            }
                        }
                float mt[NT][2];
                auto grows = [&]() {
                    bool grow = false;
#pragma unroll
                    for (int b = 0; b < NT; ++b)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int i = 0; i < TT; ++i) {
                                const float x = fmaxf(s[i][b][e] + least[i][0], s[i][b][e + 2] + least[i][1]);
                                mt[b][e] = i == 0 ? x : fmaxf(mt[b][e], x);
                            }
                            grow = grow || mt[b][e] > m[b][e] + kLnGrow;
                        }
                    return grow;
                };
                bool grow = grows(), apart = far > 0.f;
                grow = __any_sync(0xffffffffu, grow || apart || dead != 0);
                if (grow && (__any_sync(0xffffffffu, apart) || dead != 0)) {
                    // again, without tokens that nobody sees and dead groups
                    bool seen[TT][2];
                    uint32_t some = 0;  // groups that are not zero
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            seen[i][h] = !MASK;
                            if (MASK)
#pragma unroll
                                for (int b = 0; b < NT; ++b)
                                    seen[i][h] = seen[i][h] || tok + 16 * i + 8 * h < max(see[b][0], see[b][1]);
#pragma unroll
                            for (int g = 0; g < NG; ++g)
                                if (seen[i][h] && !(sv[i][h][g] <= kLnZeroStep)) some |= 1u << g;
                        }
                    some = __reduce_or_sync(0xffffffffu, some);
                    int now = dead == kFresh ? (int)(~some & (kFresh - 1)) : dead;
                    if (now > 0 && (now & some)) now = -1;
                    apart = now < 0;
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float hi = kLnLeastStep, lo = INFINITY;
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                hi = seen[i][h] ? fmaxf(hi, sv[i][h][g]) : hi;
                                lo = now > 0 && (now >> g & 1) ? lo : fminf(lo, sv[i][h][g]);
                            }
                            const bool x = seen[i][h] && lo * kApart < hi;
                            apart = apart || x;
                            least[i][h] = lg2_approx(x ? fmaxf(fmaxf(lo, hi * kLnFar), kLnFar) : hi);
                        }
                    apart = __any_sync(0xffffffffu, apart);
                    if (!ALONE && apart) return false;
                    dead = now;
                    grow = __any_sync(0xffffffffu, grows());
                }
                if (grow) {
#pragma unroll
                    for (int b = 0; b < NT; ++b)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = mt[b][e];
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                            const float mn = fmaxf(m[b][e], x - kLnUp), f = tc::ex2_approx(m[b][e] - mn);
                            m[b][e] = mn;
                            l[b][e] *= f;
                            z[b][e] *= f;
#pragma unroll
                            for (int k = 0; k < KW; ++k) {
                                o[b][k][e] *= f;
                                o[b][k][e + 2] *= f;
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < TT; ++i)
#pragma unroll
                    for (int b = 0; b < NT; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[i][b][e] = tc::ex2_approx(s[i][b][e] - m[b][e & 1]);
                            l[b][e & 1] += s[i][b][e];
                        }
                // zero codes of the tokens, group by row: those of group lane / 4
                uint32_t v0[TT], v1[TT];
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    v0[i] = transpose8(NG == 4 && (j & 1) ? vp[i][0][PW - 1] : vp[i][0][0]) & kLow;
                    v1[i] = transpose8(NG == 4 && (j & 1) ? vp[i][1][PW - 1] : vp[i][1][0]) & kLow;
                }
                auto v_operand = [&](int i, int k, uint32_t k0, uint32_t k1, uint32_t(&a)[4]) {
                    const uint32_t x = vw[i][k], h = x >> 8;
                    a[0] = x & kLow;
                    a[1] = x & kHigh;
                    a[2] = h & kLow;
                    a[3] = h & kHigh;
                    if (VC) {
                        a[0] = minus(a[0] | k1024, k0 | k1024);
                        a[1] = minus(a[1] | k1024, k0 << 4 | k1024);
                        a[2] = minus(a[2] | k1024, k1 | k1024);
                        a[3] = minus(a[3] | k1024, k1 << 4 | k1024);
                    }
                };
                if (ALONE && apart) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const uint32_t k0 = VC ? __shfl_sync(0xffffffffu, v0[0], g * 4 + j) : 0u;
                        const uint32_t k1 = VC ? __shfl_sync(0xffffffffu, v1[0], g * 4 + j) : 0u;
                        uint32_t pf[NT][NS][2];
                        float down[NT][2], zero[NT][2];
#pragma unroll
                        for (int b = 0; b < NT; ++b) {
                            float a[4], up[2];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                a[e] = tok + 8 * (e >> 1) >= see[b][e & 1] ? 0.f : s[0][b][e] * sv[0][e >> 1][g];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = fmaxf(a[e], a[e + 2]);
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                                const uint32_t ex = min(max(__float_as_uint(x) >> 23, 8u), 254u);
                                up[e] = __uint_as_float((261 - ex) << 23);  // 2^(7 - exponent)
                                down[b][e] = __uint_as_float((ex - 7) << 23);
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float x = a[2 * h] * up[0], y = a[2 * h + 1] * up[1];
#pragma unroll
                                for (int n = 0; n < NS; ++n) {
                                    const uint32_t w = pack(x, y);
                                    pf[b][n][h] = transpose8(w);
                                    const float2 r = unpack(w);
                                    x -= r.x;
                                    y -= r.y;
                                }
                            }
                            zero[b][0] = zero[b][1] = 0.f;
                            if (!VC) {
                                float c[4];
                                mma0(c, v0[0] & rmask[g], 0u, v1[0] & rmask[g], 0u, pf[b][0][0], pf[b][0][1]);
                                zero[b][0] = __shfl_sync(0xffffffffu, c[0], g * 4 + j);
                                zero[b][1] = __shfl_sync(0xffffffffu, c[1], g * 4 + j);
                            }
                        }
#pragma unroll
                        for (int k = g * G / 16; k < (g + 1) * G / 16; ++k) {
                            uint32_t a[4];
                            v_operand(0, k, k0, k1, a);
#pragma unroll
                            for (int b = 0; b < NT; ++b) {
                                float c[4];
                                mma0(c, a[0], a[1], a[2], a[3], pf[b][0][0], pf[b][0][1]);
                                if (NS == 2) mma(c, a[0], a[1], a[2], a[3], pf[b][NS - 1][0], pf[b][NS - 1][1]);
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    o[b][k][e] = fmaf(c[e] - zero[b][e], down[b][e], o[b][k][e]);
                                    o[b][k][e + 2] = fmaf(fmaf(-16.f, zero[b][e], c[e + 2]), down[b][e], o[b][k][e + 2]);
                                }
                            }
                        }
                    }
                    return true;
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t pf[TT][NT][NS][2], k0[TT], k1[TT];
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int b = 0; b < NT; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float a = s[i][b][2 * h] * sv[i][h][g], c = s[i][b][2 * h + 1] * sv[i][h][g];
                                if (MASK) {  // (a row that the query must not see may hold anything)
                                    if (tok + 16 * i + 8 * h >= see[b][0]) a = 0.f;
                                    if (tok + 16 * i + 8 * h >= see[b][1]) c = 0.f;
                                }
#pragma unroll
                                for (int y = 0; y < NS; ++y) {
                                    const uint32_t x = pack(a, c);
                                    pf[i][b][y][h] = transpose8(x);
                                    const float2 r = unpack(x);
                                    a -= r.x;
                                    c -= r.y;
                                }
                            }
#pragma unroll
                    for (int i = 0; i < TT; ++i) {
                        if (VC) {
                            k0[i] = __shfl_sync(0xffffffffu, v0[i], g * 4 + j);
                            k1[i] = __shfl_sync(0xffffffffu, v1[i], g * 4 + j);
                        } else {
#pragma unroll
                            for (int b = 0; b < NT; ++b)
                                mma(z[b], v0[i] & rmask[g], 0u, v1[i] & rmask[g], 0u, pf[i][b][0][0], pf[i][b][0][1]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int k = g * G / 16; k < (g + 1) * G / 16; ++k) {
                            uint32_t a[4];
                            v_operand(i, k, VC ? k0[i] : 0u, VC ? k1[i] : 0u, a);
#pragma unroll
                            for (int b = 0; b < NT; ++b)
#pragma unroll
                                for (int y = 0; y < NS; ++y)
                                    mma(o[b][k], a[0], a[1], a[2], a[3], pf[i][b][y][0], pf[i][b][y][1]);
                        }
                }
                return true;
            };
            // tiles that all rows see whole, then the others
            const int whole = min(nt, see_least - cc.c);
            using One = std::integral_constant<int, 1>;
            using Two = std::integral_constant<int, PAIR ? 2 : 1>;
            if (!(PAIR && whole == 2 && work(Two{}, std::false_type{}))) {
#pragma unroll 1
                for (int i = 0; i < nt; ++i, tile += TB, tok += kQ4Tile)
                    if (PAIR || i >= whole || !work(One{}, std::false_type{})) work(One{}, std::true_type{});
            }
            left -= nt;
            const bool last = left == 0 || (cc.c + nt == cc.cr && left <= kLnPad), ends = last || cc.c + nt == cc.cr;
            // The zero codes' sums leave the codes' every few tiles: both grow with all weights, their difference only
            // as the values do, and the tensor cores cut the bits off that a large sum has no room for.
            if (!VC && (ends || (left & 2))) {
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const float zero = __shfl_sync(0xffffffffu, z[b][e], g * 4 + j);
#pragma unroll
                            for (int k = g * G / 16; k < (g + 1) * G / 16; ++k) {
                                o[b][k][e] -= zero;
                                o[b][k][e + 2] = fmaf(-16.f, zero, o[b][k][e + 2]);
                            }
                        }
#pragma unroll
                for (int b = 0; b < NT; ++b) z[b][0] = z[b][1] = 0.f;
            }
            if (ends) {  // the piece
                const long long seg = (long long)unit + blockIdx.x;
                // one that does not hold all of its unit waits for the other warps' pieces: a warp's last one where its
                // ring was, which is empty now, one before it, its first, behind the ring
                const bool open = starts > 0 || cc.c + nt < cc.cr;
                uint8_t *to = last ? ring : ring + NST * SB;
                if (open && lane == 0) {
                    piece_unit[2 * warp + last] = unit;
                    piece_rows[2 * warp + last] = min(RB, rows - row0);
                }
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = l[b][e];
                        x += __shfl_xor_sync(0xffffffffu, x, 4);
                        x += __shfl_xor_sync(0xffffffffu, x, 8);
                        x += __shfl_xor_sync(0xffffffffu, x, 16);
                        const int qr = 8 * b + j * 2 + e;
                        float2 *ml = reinterpret_cast<float2 *>(to + RB * L::ROW * 4) + qr;
                        float *dst = reinterpret_cast<float *>(to) + qr * L::ROW;
                        if (!open) {
                            // (row starts that are no sums of lengths can ask for more places than there are)
                            if (row0 + qr >= rows || (unsigned long long)seg >= W.segs) continue;
                            const size_t row = (size_t)seg * W.seg_rows + qr;
                            ml = W.ml + row;
                            dst = W.o + row * D;
                        }
                        if (lane < 4) *ml = make_float2(m[b][e], x);
                        dst += (lane >> 2) * 2;
#pragma unroll
                        for (int k = 0; k < KW; ++k)  // channels 16 k + 2 (lane / 4), + 1
                            *reinterpret_cast<float2 *>(dst + 16 * k) =
                                make_float2(o[b][k][e] * (VC ? 1.f : 0x1p24f), o[b][k][e + 2] * (VC ? 0.0625f : 0x1p20f));
                    }
                ++unit;
            }
            __syncwarp();  // the stage's readers are done: the next issue may overwrite it
            cc.c += nt;
            if (cc.c == cc.cr && (left -= kLnPad) > 0) {
                --cc.c;
                cc.next(D_, A);
                starts = 0;
                ask_q();
                begin();
            }
        }
        if (s_abort) {  // copies still in flight land before the block ends
            for (int k = 0; k < NST; ++k) {
                tc::mbar_drain(&bar[k], 0);
                tc::mbar_drain(&bar[k], 1);
            }
        }
    }
    // pieces of one unit stand behind one another
    __syncthreads();
    for (int a = 0, z; a < 2 * WARPS; a = z) {
        const int unit = piece_unit[a];
        z = a + 1;
        if (unit < 0) continue;
        while (z < 2 * WARPS && (piece_unit[z] == unit || piece_unit[z] < 0)) ++z;
        const long long seg = (long long)unit + blockIdx.x;
        const int rows = piece_rows[a];
        if ((unsigned long long)seg >= W.segs) continue;
        for (int i = threadIdx.x; i < rows * (D / 4); i += THREADS) {
            const int qr = i / (D / 4), col = i % (D / 4) * 4;
            float M = kPgNoMax, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p = a; p < z; ++p) {
                if (piece_unit[p] < 0) continue;
                const uint8_t *at = smem + (p >> 1) * L::WARP + (p & 1 ? 0 : NST * SB);
                const float2 ml = reinterpret_cast<const float2 *>(at + RB * L::ROW * 4)[qr];
                const float4 v = *reinterpret_cast<const float4 *>(at + (qr * L::ROW + col) * 4);
                const float mn = fmaxf(M, ml.x), f = exp2f(M - mn), w = exp2f(ml.x - mn);
                M = mn;
                sum = fmaf(w, ml.y, sum * f);
                acc = make_float4(fmaf(w, v.x, acc.x * f), fmaf(w, v.y, acc.y * f), fmaf(w, v.z, acc.z * f),
                                  fmaf(w, v.w, acc.w * f));
            }
            const size_t row = (size_t)seg * W.seg_rows + qr;
            if (col == 0) W.ml[row] = make_float2(M, sum);
            *reinterpret_cast<float4 *>(W.o + row * D + col) = acc;
        }
    }
    pg_end_after_prior();
}

// ---- host ------------------------------------------------------------------------------------------
// Prompts of more than one row tile are read back into 16-bit arrays of the workspace (one layer's, up to kQ4WideMost
// bytes), which the kernel of pages_tc.cu then takes as they are: the operands are made once instead of once per
// one or two row tiles, on an SM whose issue slots the softmax of two row tiles needs.
constexpr long long kQ4WideMost = 1LL << 32;
// Prompts of 16-bit types with more than kQ4LineRows query rows go to tcgen05 (unless all there is to do is short), as
// do the own rows of a request with more than kQ4FewRows query rows and kQ4FewScores scores where there are at least
// kQ4FewUnits requests times KV heads: a line's warps read the codes once for every 8 query rows, the tensor cores for
// 128, but a CTA takes its time whatever it holds. By lines and on tcgen05, us (32/8 heads of d 128, bf16): behind 16K
// rows 16 query rows a head 20 and 31, 32 rows 54 and 31, 64 rows 98 and 34; behind 128K rows 32 rows 241 and 121, 128
// rows 959 and 128; behind 256 rows 8 requests 11.8 and 18.1, 64 requests 18.0 and 18.2. Own rows of 64 requests, `new`
// new rows: 10 and 392 rows 53 and 49, 16 and 1024 96 and 85, 32 and 512 108 and 82, 64 and 2048 398 and 263; of 8
// requests: 16 and 1024 21 and 30, 64 and 2048 55 and 65, 16 and 4096 33 and 59.
constexpr int kQ4LineRows = 16, kQ4FewRows = 32, kQ4FewScores = 32768, kQ4FewUnits = 128;

int ln_ctas(const PgDims &D) {
    const int rb = pg_unit_rows(D);
    const long long rows = (long long)D.max_new * D.g;
    long long chunks = (long long)D.R * D.Hkv * ((rows + rb - 1) / rb) * ((D.cap() + kPgChunk - 1) / kPgChunk);
    if (D.line)
        chunks += (long long)D.S * D.Hkv * ((D.group_rows() * D.g + rb - 1) / rb) * ((D.n + kPgChunk - 1) / kPgChunk);
    return (int)(chunks < D.own_sms ? chunks : D.own_sms);
}

template <int D, int G, int NT, int MODE>
cudaError_t go(const PgDims &D_, const Q4Shape &Q, const PgAttn &A, cudaStream_t st) {
    using L = Ln<D, G, NT, MODE>;
    return pg_launch(q4_line_kernel<D, G, NT, MODE>, ln_ctas(D_), L::THREADS, L::SMEM, true, st, D_, A, A.own, Q.ptiles);
}
template <int D, int G> cudaError_t by_type(const PgDims &D_, const Q4Shape &Q, const PgAttn &A, cudaStream_t st) {
    if (D_.dtype == KVE_F32) return go<D, G, 2, kLnF32>(D_, Q, A, st);
    return D_.dtype == KVE_BF16 ? go<D, G, 1, kLnBf16>(D_, Q, A, st) : go<D, G, 1, kLnF16>(D_, Q, A, st);
}

}  // namespace

bool q4_dims(const KvePgShape *sh, int group, PgDims *D, Q4Shape *Q, const char **why) {
    if (!pg_dims(sh, D, why)) return false;
    if ((group != 32 && group != 64 && group != 128) || group > D->d)
        return (*why = "group must be 32, 64 or 128, at most d_head"), false;
    if (D->P < kQ4Tile) return (*why = "page_size must be 16 or more"), false;
    Q->d = D->d;
    Q->group = group;
    Q->tile = q4_tile_bytes(D->d, group);
    Q->ptiles = (D->n + kQ4Tile - 1) / kQ4Tile;
    Q->wide = false;
    D->direct = D->prompt_own = false;
    D->np = D->ns = 0;
    D->own_sms = kPgSms;
    D->line = D->n > 0;
    D->pad = kLnPad;
    if (D->dtype == KVE_F32) return true;
    D->unit_rows = 8;
    D->few_rows = kQ4FewRows;
    D->few_scores = D->R * D->Hkv >= kQ4FewUnits ? kQ4FewScores : 0x7fffffff;
    auto ctas = [](const PgDims &D, bool own) {  // per KV head, of a split: launched, and those that hold rows
        const long long of = own ? D.R : D.S;
        const long long per = (long long)pg_tile_rows(D) * pg_pairs(D, own ? D.max_new : D.group_rows());
        const long long most = of * pg_tc_blocks(D, own), all = D.rows / per + of;
        return std::make_pair(most, most < all ? most : all);
    };
    if (D->n > 0 && D->group_rows() * D->g > kQ4LineRows && !pg_short_prompts(*D)) {
        D->line = false;
        const long long bytes = 4LL * D->S * D->Hkv * D->n * D->d;  // K and V
        Q->wide = D->group_rows() > pg_tile_rows(*D) && bytes <= kQ4WideMost;
        const auto c = ctas(*D, false);
        pg_tiles_split(D->Hkv * c.second, D->n, &D->np, &D->psplit);
        if (D->Hkv * c.first * D->np < kPgShare) D->own_sms = (int)(kPgSms - D->Hkv * c.first * D->np);
    }
    if (pg_many_new(*D)) pg_tiles_split(D->Hkv * ctas(*D, true).second, D->cap(), &D->ns, &D->ssplit);
    return true;
}

unsigned long long q4_segs(const PgDims &D) {
    const long long busy = D.R < D.rows ? D.R : D.rows, rb = pg_unit_rows(D);
    long long units = D.Hkv * ((long long)D.rows * D.g / rb + busy);
    if (D.line) units += D.Hkv * ((long long)D.rows * D.g / rb + (D.S < D.rows ? D.S : D.rows));
    return units + ln_ctas(D);
}

PgWorkspace q4_ws_layout(const PgDims &D, const Q4Shape &Q) {
    PgWorkspace W{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~size_t(255);
        return at;
    };
    const size_t rows = (size_t)D.rows * D.Hq * (D.np + D.ns);
    W.part_ml = take(sizeof(float2) * rows);
    W.part_o = take(sizeof(float) * rows * D.d);
    const size_t segs = (size_t)q4_segs(D) * pg_seg_rows(D);
    W.own_ml = take(sizeof(float2) * segs);
    W.own_o = take(sizeof(float) * segs * D.d);
    W.own_base = take(sizeof(long long) * (D.S + D.R));
    W.own_unit = take(sizeof(int) * (D.S + D.R));
    W.own_cpw = take(sizeof(long long));
    const size_t wide = Q.wide ? 2 * (size_t)D.S * D.Hkv * D.n * D.d : 0;
    W.k16 = take(wide);
    W.v16 = take(wide);
    W.total = off;
    return W;
}

cudaError_t launch_q4_lines(const PgDims &D, const Q4Shape &Q, const PgAttn &A, cudaStream_t st) {
    if (Q.d == 128)
        return Q.group == 32 ? by_type<128, 32>(D, Q, A, st)
                             : (Q.group == 64 ? by_type<128, 64>(D, Q, A, st) : by_type<128, 128>(D, Q, A, st));
    if (Q.d == 64) return Q.group == 32 ? by_type<64, 32>(D, Q, A, st) : by_type<64, 64>(D, Q, A, st);
    return by_type<32, 32>(D, Q, A, st);
}

}  // namespace kve
