// The kernel of pages_tc.cu on tcgen05, whose K and V come from 16-bit arrays (G = 0) or from a cache in 4 bits in
// groups of G channels (q4.cuh). What differs then: a raw tile arrives as it lies (bulk copies of 64 tokens), and
// warps turn its codes into the operands that TMA would have brought (all that are neither the products' nor a softmax's:
// three, with one row tile per CTA four more less the one that sends for the tiles): n - k from 128 + n (bf16) or 64 +
// n (fp16), exactly, times the step, which is exact too, since s m has 8 significant bits. K's words hold 8
// channels of a token, a 16-byte store; V's hold tokens side by side, and stmatrix turns them, which leaves the
// 8 even channels of every 16 before the 8 odd ones: the epilogue puts O's columns back in order.
//
// One row tile behind 128K rows (8 KV heads, groups of 32): bf16 133 us, fp16 156, 2.4 to 2.9 us a tile of 128 tokens, which
// the makers bound (without their work 81 us): a warp takes 2200 cycles for 16 tokens' K and V. More makers (4 -> 6) or raw halves (3 -> 6) changed
// nothing; makers in functions of their own did, which leaves the softmax its registers (two row tiles: 384 -> 233 us).
#pragma once

#include <cudaTypedefs.h>

#include "q4.cuh"

namespace kve {
namespace {

__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void mbar_inval(uint64_t *bar) {
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

template <typename T> struct PtIsHalf { static constexpr bool value = false; };
template <> struct PtIsHalf<__half> { static constexpr bool value = true; };
template <typename T> __device__ __forceinline__ uint32_t pt_pack(float a, float b);
template <> __device__ __forceinline__ uint32_t pt_pack<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pt_pack<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Shared memory: QT row tiles, then the K/V ring (K_0, V_0, K_1, ...), with 4 bits three raw halves of a tile, then
// barriers.
template <int D, int QT, int G> struct PtLayout {
    static constexpr int KB = D / 64;  // 128-byte column blocks of a row
    static constexpr uint32_t TILE = KB * 16384;
    static constexpr int SLOTS = G ? (D == 128 ? 4 : 8)
                                   : (D == 128 ? (QT == 2 ? 5 : 6) : (QT == 2 ? 11 : 12));
    static constexpr uint32_t RING = QT * TILE, RAW = RING + SLOTS * TILE;
    static constexpr int RAWS = G ? (QT == 1 || D == 64 ? 6 : 3) : 0, HALF = G ? 4 * q4_tile_bytes(D, G ? G : 32) : 0;
    static constexpr uint32_t BAR = (RAW + RAWS * HALF + 127) / 128 * 128;
    static constexpr int NBAR = 1 + 2 * SLOTS + 9 + 2 * RAWS;
    static constexpr size_t SMEM = BAR + 512 + 1024;
    static_assert(NBAR * 8 + 16 <= 512 && SMEM <= 227 * 1024);
    // (the epilogue's rows of O)
    static_assert(4 * QT * 32 * (D + 4) * 4 <= SLOTS * TILE + RAWS * HALF);
};
struct PtDesc {
    uint64_t q, k, v;  // of row tile 0 and of ring place 0 as K and as V
};
template <int QT, int G> constexpr int pt_threads() { return (4 + 4 * QT + (G && QT == 1 ? 4 : 0)) * 32; }
template <int QT> constexpr int pt_makers() { return QT == 1 ? 6 : 3; }  // warps that make operands

struct PtArgs {
    PgDims D;
    int nrt, tt;  // row tiles (or pairs) per prompt and KV head, new rows per tile
    float k1;
    const int32_t *plen, *q_start, *len, *table;
    const void *q, *K, *V;  // and row_req: for the own rows
    long long q_row;
    const int32_t *row_req;
    float2 *part_ml;
    float *part_o;
    unsigned *err;
    const uint8_t *codes;  // 4 bits: the prompts' array, or with OWN the pages
    int ptiles;
};

// Own rows of the prompt's requests whose tables hold at most 32 rows, a warp per row and head: query rows
// first, first + step, ... below `end` of the prompt's, into split np of the partial results. Each lane looks up
// one of them (request, tokens that it sees), then for each row one of its tokens' pages, a row ahead: what is
// left of a row is its K/V's way from memory.
template <typename T, int E>
__device__ __forceinline__ void pt_own_rows(const PtArgs &A, int s, int kh, int tok0, int first, int end,
                                            int step, int lane) {
    const PgDims &D = A.D;
    constexpr int d = 32 * E;
    for (; first < end; first += 32 * step) {
        const int rr = first + lane * step;
        int tok = 0, h = 0, r = 0, see = 0;
        bool mine = false;  // the row is its request's
        if (rr < end) {
            tok = tok0 + rr / D.g;
            h = kh * D.g + rr % D.g;
            r = __ldg(A.row_req + tok);
            if (r >= s * D.F && r < (s + 1) * D.F) {
                const int start = pg_start(A.q_start, r, D.rows);
                const int nq = pg_start(A.q_start, r + 1, D.rows) - start;
                mine = tok >= start && tok - start < min(nq, D.max_new);
                see = pg_clamp(__ldg(A.len + r), 0, D.cap()) - nq + 1 + (tok - start);
            }
        }
        unsigned todo = __ballot_sync(0xffffffffu, mine);
        auto pages = [&](int i) {  // of row i's tokens, one per lane
            const int ri = __shfl_sync(0xffffffffu, r, i), n = __shfl_sync(0xffffffffu, see, i);
            return lane < n ? pg_page(A.table + (size_t)ri * D.maxp, lane, D.lgP, D.npages, A.err) : 0;
        };
        int next = todo ? pages(__ffs(todo) - 1) : 0;
        while (todo) {
            const int i = __ffs(todo) - 1, page = next;
            todo &= todo - 1;
            const int ti = __shfl_sync(0xffffffffu, tok, i), hi = __shfl_sync(0xffffffffu, h, i);
            const int n = __shfl_sync(0xffffffffu, see, i);
            float q[E], M = kPgNoMax, L = 0.f, acc[E];
            row_cols<T, E>(static_cast<const T *>(A.q) + ti * A.q_row + (size_t)hi * d + lane * E, q);
            if (todo) next = pages(__ffs(todo) - 1);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.f;
            for (int t0 = 0; t0 < n; t0 += 8) {
                float k[8][E], v[8][E], x[8], Mn = M;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int p = __shfl_sync(0xffffffffu, page, (t0 + j) & 31);
#pragma unroll
                    for (int e = 0; e < E; ++e) k[j][e] = v[j][e] = 0.f;
                    if (t0 + j < n) {
                        const size_t at =
                            ((((size_t)p * D.Hkv + kh) << D.lgP) + ((t0 + j) & (D.P - 1))) * d + lane * E;
                        row_cols<T, E>(static_cast<const T *>(A.K) + at, k[j]);
                        row_cols<T, E>(static_cast<const T *>(A.V) + at, v[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float y = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) y = fmaf(q[e], k[j][e], y);
                    x[j] = t0 + j < n ? warp_sum(y) * A.k1 : -INFINITY;  // (the same in every lane)
                    Mn = fmaxf(Mn, x[j]);
                }
                const float f = exp2f(M - Mn);
                M = Mn;
                L *= f;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float w = exp2f(x[j] - M);
                    L += w;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[j][e], acc[e]);
                }
            }
            const size_t row = ((size_t)D.np * D.rows + ti) * D.Hq + hi;
            if (lane == 0) A.part_ml[row] = make_float2(M, L);
#pragma unroll
            for (int e = 0; e < E; ++e) A.part_o[row * d + lane * E + e] = acc[e];
        }
    }
}

// Barriers of a CTA, in shared memory.
template <int D, int QT, int G> struct PtBars {
    uint64_t *q_full, *rfull, *rempty, *s_full, *p_half, *p_full, *o_done, *drain, *o_final, *raw_full, *raw_empty;
    __device__ explicit PtBars(uint64_t *b) {
        constexpr int S = PtLayout<D, QT, G>::SLOTS;
        q_full = b;
        rfull = b + 1;
        rempty = rfull + S;
        s_full = rempty + S;
        p_half = s_full + 2;
        p_full = p_half + 2;
        o_done = p_full + 2;
        drain = o_done + 1;
        o_final = drain + 1;
        raw_full = o_final + 1;
        raw_empty = raw_full + PtLayout<D, QT, G>::RAWS;
    }
};

// Matrix descriptors advance by adding to the address field (16-byte units): building one per product
// costs the issuing thread about 150 cycles, more than the product's 64 (measured: 8 products of
// 128 x 128 x 16 took 1200 cycles with descriptors built in place, 514 with added offsets).
//
// S(i) = Q_t K_i^T into S buffer `sb`. With two row tiles sb = t; with one, the buffers alternate and
// S(i + 1) is computed while the softmax of S(i) runs. A thread's MMAs run in issue order, so the
// product that read P from these columns is done before they are overwritten.
template <typename T, int D, int QT, int G>
__device__ __forceinline__ void pt_issue_s(const PtDesc &d, uint32_t tmem, int t, int sb, int i) {
    using L = PtLayout<D, QT, G>;
    constexpr uint32_t id = tc::idesc_f16kind(128, 128, 0, !PtIsHalf<T>::value);
    const int slot = (2 * i) % L::SLOTS;
    tc::fence_after_sync();
    const uint64_t q = d.q + (uint32_t)t * (L::TILE / 16), k = d.k + (uint32_t)slot * (L::TILE / 16);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const uint32_t o = ((s >> 2) * 16384 + (s & 3) * 32) / 16;
        tc::mma_bf16(tmem + sb * 128, q + o, k + o, id, s > 0);
    }
}

// O_t += P(i) V_i, P from S buffer `sb`; the first half of the tokens goes as soon as its weights are
// stored, while the softmax is still at the second. half_ready: the first half is known to be there.
template <typename T, int D, int QT, int G>
__device__ __forceinline__ bool pt_issue_pv(const PtBars<D, QT, G> &B, const PtDesc &d, uint32_t tmem,
                                            int t, int sb, uint32_t p_phase, int i, bool half_ready,
                                            volatile int *abort_flag, unsigned *err) {
    using L = PtLayout<D, QT, G>;
    constexpr uint32_t id = tc::idesc_f16kind(128, D, 1, !PtIsHalf<T>::value);
    const int slot = (2 * i + 1) % L::SLOTS;
    const uint64_t v = d.v + (uint32_t)slot * (L::TILE / 16);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (!(half == 0 && half_ready) &&
            !tc::mbar_wait(half ? &B.p_full[sb] : &B.p_half[sb], p_phase, abort_flag, err))
            return false;
        tc::fence_after_sync();
#pragma unroll
        for (int s = 4 * half; s < 4 * half + 4; ++s)  // 16 tokens: 8 TMEM columns of P, 16 V rows
            tc::mma_bf16_ts(tmem + 256 + t * D, tmem + sb * 128 + 8 * s, v + s * (2048 / 16), id,
                            (i > 0 || s > 0) ? 1u : 0u);
    }
    return true;
}

// Waits until item c of the ring (K_i: 2 i, V_i: 2 i + 1) has landed.
template <typename T, int D, int QT, int G>
__device__ __forceinline__ bool pt_landed(const PtBars<D, QT, G> &B, int c, volatile int *abort_flag,
                                          unsigned *err) {
    constexpr int S = PtLayout<D, QT, G>::SLOTS;
    return tc::mbar_wait(&B.rfull[c % S], (c / S) & 1, abort_flag, err);
}

// One row tile: S is double-buffered, so a tile's scores are two ahead.
template <typename T, int D, int QT, int G>
__device__ __forceinline__ bool pt_issue_one(const PtBars<D, QT, G> &B, const PtDesc &d, uint32_t tmem,
                                             int ntl, volatile int *abort_flag, unsigned *err) {
    constexpr int S = PtLayout<D, QT, G>::SLOTS;
    auto scores = [&](int i) {
        if (!pt_landed<T, D, QT, G>(B, 2 * i, abort_flag, err)) return false;
        pt_issue_s<T, D, QT, G>(d, tmem, 0, i & 1, i);
        tc::mma_commit(&B.s_full[i & 1]);
        tc::mma_commit(&B.rempty[(2 * i) % S]);
        return true;
    };
    bool ok = true;
    for (int i = 0; ok && i < 2 && i < ntl; ++i) ok = scores(i);
    for (int i = 0; ok && i < ntl; ++i) {
        ok = pt_landed<T, D, QT, G>(B, 2 * i + 1, abort_flag, err) &&
             pt_issue_pv<T, D, QT, G>(B, d, tmem, 0, i & 1, (i >> 1) & 1, i, false, abort_flag, err);
        if (!ok) break;
        tc::mma_commit(B.o_done);
        if (i == ntl - 1) tc::mma_commit(B.o_final);
        tc::mma_commit(&B.rempty[(2 * i + 1) % S]);
        if (i + 2 < ntl) ok = scores(i + 2);
    }
    return ok;
}

// Two row tiles, in strict turn: [P_0 V, S_0 next], [P_1 V, S_1 next]. The turns keep the softmax
// groups half a period apart, one computing weights while the other's products run (a thread per tile
// let them fall into step and both wait: 3400 cycles a period instead of 2650). A commit holds the
// issuing thread until the products before it are nearly done and a wait on a barrier that has
// completed costs it 75 cycles, so there is one commit a turn, and what can be tested for the next
// turn is tested before it. A tile's s_full then stands for everything before it: the ring places of
// K_(i+1) and V_i (released by the softmax of tile 1) and the previous product into O.
template <typename T, int D, int QT, int G>
__device__ __forceinline__ bool pt_issue_two(const PtBars<D, QT, G> &B, const PtDesc &d, uint32_t tmem,
                                             int ntl, volatile int *abort_flag, unsigned *err) {
    constexpr int S = PtLayout<D, QT, G>::SLOTS;
    if (!pt_landed<T, D, QT, G>(B, 0, abort_flag, err)) return false;
    for (int t = 0; t < 2; ++t) {
        pt_issue_s<T, D, QT, G>(d, tmem, t, t, 0);
        tc::mma_commit(&B.s_full[t]);
    }
    bool v_ready = false, p_ready = false;
    for (int i = 0; i < ntl; ++i) {
        const bool more = i + 1 < ntl;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t == 0 && !v_ready && !pt_landed<T, D, QT, G>(B, 2 * i + 1, abort_flag, err))
                return false;
            if (!pt_issue_pv<T, D, QT, G>(B, d, tmem, t, t, i & 1, i, p_ready, abort_flag, err))
                return false;
            if (t == 0 && more && !pt_landed<T, D, QT, G>(B, 2 * i + 2, abort_flag, err)) return false;
            if (more) pt_issue_s<T, D, QT, G>(d, tmem, t, t, i + 1);
            p_ready = t == 0 ? mbar_test(&B.p_half[1], i & 1) : mbar_test(&B.p_half[0], (i + 1) & 1);
            if (t == 1)
                v_ready = more && mbar_test(&B.rfull[(2 * i + 3) % S], ((2 * i + 3) / S) & 1);
            if (more) tc::mma_commit(&B.s_full[t]);
        }
    }
    tc::mma_commit(B.o_final);
    return true;
}

// Softmax of one row tile by 4 warps (warp lg owns TMEM lanes 32 lg .. 32 lg + 31, a thread one
// row). DB: one row tile, S(i) in buffer i % 2, whose barriers complete every second tile.
// see0: with OWN, the tokens that the first new row sees (each later one sees one more).
template <typename T, int D, int QT, int G, bool OWN, bool DB>
__device__ __forceinline__ void pt_softmax(const PtArgs &A, const PtBars<D, QT, G> &B, uint8_t *sm,
                                           uint32_t tmem, int warp, int lane, int row0, int nrow,
                                           int tok0, int kh, int t0, int t1, int see0, int ntl,
                                           int sp, volatile int *abort_flag) {
    using L = PtLayout<D, QT, G>;
    const int t = DB ? 0 : (warp - 4) >> 2, lg = warp & 3;
    const int r = lg * 32 + lane, g = A.D.g;
    const int first = row0 + t * A.tt * g;              // the tile's first row of the prompt
    const int rr = first + r;
    const bool valid = r < A.tt * g && rr < nrow;
    const int see = OWN ? min(t1, see0 + rr / g) : t1;  // this row's end
    const uint32_t lane_off = (uint32_t)(lg * 32) << 16;
    const uint32_t o_col = tmem + lane_off + 256 + t * D;
    float m = kPgNoMax, l = 0.f;
    bool ok = true;
    for (int i = 0; i < ntl; ++i) {
        const int sb = DB ? (i & 1) : t;
        const uint32_t s_col = tmem + lane_off + sb * 128;
        if (!tc::mbar_wait_warp(&B.s_full[sb], DB ? ((i >> 1) & 1) : (i & 1), abort_flag, A.err)) {
            ok = false;
            break;
        }
        tc::fence_after_sync();
        if (!DB && t == 1 && r == 0) {
            tc::mbar_arrive(&B.rempty[(2 * i) % L::SLOTS]);
            if (i > 0) tc::mbar_arrive(&B.rempty[(2 * i - 1) % L::SLOTS]);
        }
        float s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(s_col + c * 32, s[c]);
        tc::tmem_wait_ld();
        const int nv = t1 - (t0 + i * 128);         // tokens of this tile
        const int nvr = OWN ? see - (t0 + i * 128) : nv;  // of which the row sees
        if (nvr < 128) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (c * 32 + e >= nvr) s[c][e] = -INFINITY;
        }
        if (G == 0 && nv < 128) {
            // V rows behind the last token: zeros, whatever the array holds there
            const int vc = 2 * i + 1, slot = vc % L::SLOTS;
            if (!tc::mbar_wait_warp(&B.rfull[slot], (vc / L::SLOTS) & 1, abort_flag, A.err)) {
                ok = false;
                break;
            }
            uint8_t *v = sm + L::RING + slot * L::TILE;
            for (int e = nv * 8 + lane; e < 128 * 8; e += 32)
#pragma unroll
                for (int kb = 0; kb < L::KB; ++kb)
                    *reinterpret_cast<uint4 *>(v + kb * 16384 + e * 16) = make_uint4(0, 0, 0, 0);
            tc::fence_proxy_async_smem();
        }
        // weights of a half from its scores: p = 2^(s k1 - m), rounded to the type of V (half a step,
        // like V's own entries; ex2.approx is off by 2^-22 of p); their sum takes p before the rounding
        float pk[32], l0, l1;
        auto half_weights = [&](const float (&x)[32], const float (&y)[32]) {
            const uint64_t k1_2 = tc::pk2(A.k1, A.k1), negm_2 = tc::pk2(-m, -m);
            uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float u0 = j < 16 ? x[(2 * j) & 31] : y[(2 * j) & 31];
                const float u1 = j < 16 ? x[(2 * j + 1) & 31] : y[(2 * j + 1) & 31];
                float x0, x1;
                tc::upk2(tc::fma2(tc::pk2(u0, u1), k1_2, negm_2), x0, x1);
                const float p0 = tc::ex2_approx(x0), p1 = tc::ex2_approx(x1);
                sum2[j & 3] = tc::add2(sum2[j & 3], tc::pk2(p0, p1));
                pk[j] = __uint_as_float(pt_pack<T>(p0, p1));
            }
            float a[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) tc::upk2(sum2[k], a[2 * k], a[2 * k + 1]);
            return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
        };
        // The first half goes ahead with the maximum of the tiles before, beside the search for this
        // tile's: a weight may exceed 1 by up to 2^8 before the row is rescaled anyway, and only a
        // larger growth (rare after the first tiles) makes the half anew from S, still in TMEM.
        l0 = half_weights(s[0], s[1]);
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2) m4[c] = tc::max3(m4[c], s[c][e], s[c][e + 1]);
        const float mt = tc::max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * A.k1;
        const float mn = fmaxf(m, PtIsHalf<T>::value ? mt - kPgHalfUp : mt);
        // rows of the tile that hold no query carry whatever shared memory held: they never rescale
        const bool grow = valid && mn > m + kPgRescale;
        // tcgen05.ld/st are warp-collective: the whole warp rescales when one of its rows does
        if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? tc::ex2_approx(m - mn) : 1.f;
            if (grow) m = mn;
            l *= f;
            if (i > 0) {  // O holds the product before (s_full says so with two tiles)
                if (DB && !tc::mbar_wait_warp(B.o_done, (i - 1) & 1, abort_flag, A.err)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tc::tmem_ld32(o_col + c * 32, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= f;
                    tc::tmem_st32(o_col + c * 32, o);
                }
            }
            tc::tmem_ld32(s_col, s[0]);
            tc::tmem_ld32(s_col + 32, s[1]);
            tc::tmem_wait_ld();
            if (nvr < 64) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e >= nvr) s[e >> 5][e & 31] = -INFINITY;
            }
            l0 = half_weights(s[0], s[1]);
        }
        tc::tmem_st32(s_col, pk);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&B.p_half[sb]);
        l1 = half_weights(s[2], s[3]);
        tc::tmem_st32(s_col + 32, pk);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&B.p_full[sb]);
        l += l0 + l1;
    }
    // the last product of all: O is done and the ring is free
    if (__all_sync(0xffffffffu, ok && tc::mbar_wait(B.o_final, 0, abort_flag, A.err))) {
        tc::fence_after_sync();
        // O leaves through the ring, which is free now: a thread's row into shared memory (rows 16
        // bytes apart in the banks), then whole rows to the workspace, 16 bytes a lane. Straight from
        // the threads, every store would touch 32 lines.
        const int d = A.D.d, rows = min(32, min(A.tt * g, nrow - first) - lg * 32);
        float *st = reinterpret_cast<float *>(sm + L::RING) + (warp - 4) * (32 * (D + 4));
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc::tmem_ld32(o_col + c * 32, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int x = G ? (e >> 2) * 16 + (e & 3) * 2 : 4 * e;  // (4 bits: even channels before odd ones)
                *reinterpret_cast<float4 *>(st + lane * (D + 4) + c * 32 + 4 * e) =
                    make_float4(o[x], o[x + (G ? 8 : 1)], o[x + (G ? 1 : 2)], o[x + (G ? 9 : 3)]);
            }
        }
        __syncwarp();
        const size_t place =  // of this lane's row
            ((size_t)(OWN ? A.D.np + sp : sp) * A.D.rows + tok0 + rr / g) * A.D.Hq + kh * g + rr % g;
        const int lpr = d / 4, col = (lane % lpr) * 4;  // lanes per row: 32, 16 or 8
#pragma unroll 8
        for (int x0 = 0; x0 < rows; x0 += 32 / lpr) {
            const int x = x0 + lane / lpr;
            const size_t to = __shfl_sync(0xffffffffu, place, x & 31);
            if (x < rows)
                *reinterpret_cast<float4 *>(A.part_o + to * d + col) =
                    *reinterpret_cast<const float4 *>(st + x * (D + 4) + col);
        }
        if (valid) A.part_ml[place] = make_float2(m, l);
    }
}

// (a function of its own where other roles would take registers from it)
template <typename T, int D, int QT, int G, bool OWN, bool DB, typename... P>
__device__ __noinline__ void pt_softmax_apart(const PtArgs &A, uint64_t *bars, P... p) {
    pt_softmax<T, D, QT, G, OWN, DB>(A, PtBars<D, QT, G>(bars), p...);
}

// ---- 4 bits ----------------------------------------------------------------------------------------
// The raw tiles, halves of 64 tokens at a time, as far as there are tokens (warp 0).
template <int D, int QT, int G, bool OWN> struct PtRaw {
    using L = PtLayout<D, QT, G>;
    const PtArgs &A;
    int s, kh, t0, t1, halves, next = 0;
    __device__ __forceinline__ PtRaw(const PtArgs &A, int s, int kh, int t0, int t1)
        : A(A), s(s), kh(kh), t0(t0), t1(t1), halves(2 * ((t1 - t0 + 127) / 128)) {}
    // Sends for halves: those before `must` have to be, those before `may` where there is room.
    __device__ __forceinline__ bool upto(const PtBars<D, QT, G> &B, uint8_t *sm, int must, int may, int lane,
                                         volatile int *abort_flag) {
        for (; next < halves && next < may; ++next) {
            const int place = next % L::RAWS;
            const uint32_t phase = ((next / L::RAWS) & 1) ^ 1;
            if (next >= must) {
                if (!__all_sync(0xffffffffu, mbar_test(&B.raw_empty[place], phase))) return true;
            } else if (!tc::mbar_wait_warp(&B.raw_empty[place], phase, abort_flag, A.err)) {
                return false;
            }
            send(B, sm, place, lane);
        }
        return true;
    }
    __device__ __forceinline__ void send(const PtBars<D, QT, G> &B, uint8_t *sm, int place, int lane) {
        const int tb = q4_tile_bytes(A.D.d, G), tpp = A.D.lgP - 4;
        const int first = (t0 + next * 64) >> 4, n = max(0, min(4, ((t1 + 15) >> 4) - first));
        uint8_t *to = sm + L::RAW + place * L::HALF;
        if (lane == 0) tc::mbar_expect_tx(&B.raw_full[place], n * tb);
        __syncwarp();
        if (n == 0) return;  // (the second half of a last tile: the phase ends without bytes)
        if (!OWN) {
            if (tc::elect_one())
                q4_bulk_load(to, A.codes + (((size_t)s * A.D.Hkv + kh) * A.ptiles + first) * tb, n * tb,
                             &B.raw_full[place]);
            return;
        }
        const int tile = first + (lane & 3);
        unsigned long long at = 0;
        if (lane < n)
            at = (((unsigned long long)pg_page(A.table + (size_t)s * A.D.maxp, tile << 4, A.D.lgP, A.D.npages, A.err) *
                       A.D.Hkv + kh) << tpp) + (tile & ((1 << tpp) - 1));
        for (int i = 0; i < n;) {  // tiles of one page lie side by side
            const unsigned long long x = __shfl_sync(0xffffffffu, at, i);
            const int run = min(n - i, (1 << tpp) - ((first + i) & ((1 << tpp) - 1)));
            if (tc::elect_one()) q4_bulk_load(to + i * tb, A.codes + x * tb, run * tb, &B.raw_full[place]);
            i += run;
        }
    }
    // copies still in flight land before the CTA goes on (at once on the normal path)
    __device__ __forceinline__ void drain(const PtBars<D, QT, G> &B, int lane) const {
        if (lane == 0)
            for (int c = next - L::RAWS < 0 ? 0 : next - L::RAWS; c < next; ++c)
                tc::mbar_drain(&B.raw_full[c % L::RAWS], (c / L::RAWS) & 1);
    }
};

// 16 tokens of K into rows row0 .. of a ring place, as TMA lays them down.
template <typename T, int DR, int G>
__device__ __forceinline__ void pt_k_tile(uint32_t raw, uint32_t place, int row0, int lane) {
    constexpr int NG = DR / G, PW = (NG + 1) / 2;
    const int r = lane >> 2, j = lane & 3;
    uint32_t w[DR / 16], p[2][PW];
    q4_words<DR>(raw + q4_lane<DR>(lane), w);
#pragma unroll
    for (int h = 0; h < 2; ++h) q4_params_of<NG>(raw + 2 * q4_codes(DR) + (r + 8 * h) * 2 * NG, p[h]);
    auto make = [&](auto check) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Q4Codes<T> of(__byte_perm(p[h][g >> 1], 0, g & 1 ? 0x3232 : 0x1010), check);
                const int row = row0 + r + 8 * h;
#pragma unroll
                for (int c = g * G / 32; c < (g + 1) * G / 32; ++c) {
                    const uint32_t x = w[2 * c] >> (8 * h), y = w[2 * c + 1] >> (8 * h);
                    const uint32_t v[4] = {of.low(x), of.high(x), of.low(y), of.high(y)};
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                     place + (c >> 1) * 16384 + tc::sw128_offset(row, (c & 1) * 4 + j)),
                                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                 : "memory");
                }
            }
    };
    if (q4_any_far<T, NG>(p)) make(std::true_type{});
    else make(std::false_type{});
}
// 16 tokens of V, of which the first `have` are there; the others' rows are zeros.
template <typename T, int DR, int G, bool WHOLE>
__device__ __forceinline__ void pt_v_tile(uint32_t raw, uint32_t place, int row0, int have, int lane) {
    constexpr int NG = DR / G, PW = (NG + 1) / 2;
    const int j = lane & 3;
    uint32_t w[DR / 16], p[4][PW], there[2];
    q4_words<DR>(raw + q4_codes(DR) + q4_lane<DR>(lane), w);
#pragma unroll
    for (int t = 0; t < 4; ++t)  // tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9
        q4_params_of<NG>(raw + 2 * q4_codes(DR) + q4_params(DR, G) + (2 * j + (t & 1) + 8 * (t >> 1)) * 2 * NG, p[t]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        there[h] = (2 * j + 8 * h < have ? 0xFFFFu : 0u) | (2 * j + 8 * h + 1 < have ? 0xFFFF0000u : 0u);
    const int to = lane >> 3, row = row0 + (to >> 1) * 8 + (lane & 7);
    auto make = [&](auto check) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const Q4Codes<T> of0(__byte_perm(p[0][g >> 1], p[1][g >> 1], g & 1 ? 0x7632 : 0x5410), check);
            const Q4Codes<T> of1(__byte_perm(p[2][g >> 1], p[3][g >> 1], g & 1 ? 0x7632 : 0x5410), check);
#pragma unroll
            for (int c = g * G / 16; c < (g + 1) * G / 16; ++c) {
                const uint32_t x = w[c], y = x >> 8;
                uint32_t v[4] = {of0.low(x), of0.high(x), of1.low(y), of1.high(y)};
                if (!WHOLE) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] &= there[i >> 1];
                }
                asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(
                                 place + (c >> 2) * 16384 + tc::sw128_offset(row, (2 * c + (to & 1)) & 7)),
                             "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                             : "memory");
            }
        }
    };
    if (q4_any_far<T, NG>(p)) make(std::true_type{});
    else make(std::false_type{});
}
// K and V of ntl tiles of 128 tokens (n tokens there): K of both halves, then V. The makers take turns at the 16-token
// tiles; one of them may also be the one that sends for the raw halves.
template <typename T, int D, int DR, int QT, int G, bool OWN, bool SENDS>
__device__ __noinline__ void pt_make_of(const PtArgs &A, uint64_t *bars, uint8_t *sm, int part, int lane, int s, int kh,
                                        int t0, int t1, volatile int *abort_flag) {
    using L = PtLayout<D, QT, G>;
    constexpr int MAKERS = pt_makers<QT>();
    const PtBars<D, QT, G> B(bars);
    PtRaw<D, QT, G, OWN> raw(A, s, kh, t0, t1);
    unsigned *err = A.err;
    const uint32_t base = tc::smem_u32(sm);
    const int n = t1 - t0, ntl = (n + 127) / 128;
    for (int c = 0; c < 2 * ntl; ++c) {
        const int slot = c % L::SLOTS;
        if (SENDS && !raw.upto(B, sm, (c | 1) + 1, (c | 1) + L::RAWS, lane, abort_flag)) break;
        if (!tc::mbar_wait_warp(&B.rempty[slot], ((c / L::SLOTS) & 1) ^ 1, abort_flag, err)) break;
        const uint32_t to = base + L::RING + slot * L::TILE;
        bool ok = true;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            const int h = (c & ~1) + half, place = h % L::RAWS;
            ok = tc::mbar_wait_warp(&B.raw_full[place], (h / L::RAWS) & 1, abort_flag, err);
            if (!ok) break;
#pragma unroll 1
            for (int i = (part + MAKERS - (2 * c + half) * 4 % MAKERS) % MAKERS; i < 4; i += MAKERS) {
                const uint32_t from = base + L::RAW + place * L::HALF + i * q4_tile_bytes(DR, G);
                const int row0 = half * 64 + i * 16;
                const int have = n - (c >> 1) * 128 - row0;
                if (!(c & 1)) pt_k_tile<T, DR, G>(from, to, row0, lane);
                else if (have >= 16) pt_v_tile<T, DR, G, true>(from, to, row0, have, lane);
                else pt_v_tile<T, DR, G, false>(from, to, row0, have, lane);
            }
            if (c & 1) {
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&B.raw_empty[place]);
            }
            if (SENDS) ok = raw.upto(B, sm, 0, h + 1 + L::RAWS, lane, abort_flag);
        }
        if (!ok) break;
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&B.rfull[slot]);
    }
    if (SENDS) raw.drain(B, lane);
}
template <typename T, int D, int QT, int G, bool OWN, bool SENDS>
__device__ __forceinline__ void pt_make(const PtArgs &A, uint64_t *bars, uint8_t *sm, int part, int lane, int s, int kh,
                                        int t0, int t1, volatile int *abort_flag) {
    if constexpr (D == 64 && G == 32) {
        if (A.D.d == 32) {
            pt_make_of<T, D, 32, QT, G, OWN, SENDS>(A, bars, sm, part, lane, s, kh, t0, t1, abort_flag);
            return;
        }
    }
    pt_make_of<T, D, D, QT, G, OWN, SENDS>(A, bars, sm, part, lane, s, kh, t0, t1, abort_flag);
}

// Tiles of 64 columns made for d_head 32 have 32 that nothing writes: zeros, of the ring that a round finds. (Q has zeros
// there, but 0 times what an epilogue left may be NaN. A function of its own: inlined, it took registers.)
__device__ __noinline__ void pt_clear(uint8_t *ring, uint32_t bytes) {
    for (uint32_t i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
        *reinterpret_cast<uint4 *>(ring + i) = make_uint4(0, 0, 0, 0);
}

// Warps: 0 TMA, 1 MMA, 2-3 own rows of short tables, then 4 softmax warps per row tile, with 4 bits
// and one row tile then 4 that make operands.
template <typename T, int D, int QT, int G, bool OWN>
__global__ void __launch_bounds__(pt_threads<QT, G>(), 1)
    pg_prompt_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PtArgs A) {
    using L = PtLayout<D, QT, G>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // what needs no input first: under programmatic launch it overlaps the end of the kernel before
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    const PtBars<D, QT, G> B(bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::NBAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + L::NBAR + 1);
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::fence_before_sync();
    } else if (warp == 0 && lane == 0) {
        if (G == 0) {
            tc::tma_prefetch_desc(&tm_k);
            tc::tma_prefetch_desc(&tm_v);
        }
        tc::tma_prefetch_desc(&tm_q);
        *abort_flag = 0;
    }
    if constexpr (D == 64 && G == 32)
        if (A.D.d == 32) pt_clear(sm + L::RING, L::SLOTS * L::TILE);
    if (!OWN) pg_wait_prior();  // (with OWN the call's first kernel has waited)
    pg_launch_dependents();
    // the row tiles of a (prompt or request, KV head, split) are adjacent: they meet in L2 on its K/V
    int b = blockIdx.x;
    const int rt0 = b % A.nrt;
    b /= A.nrt;
    const int nsplit = OWN ? A.D.ns : A.D.np;
    const int sp = b % nsplit;
    b /= nsplit;
    const int kh = b % A.D.Hkv, s = b / A.D.Hkv;  // prompt or request
    const int tok0 = pg_start(A.q_start, OWN ? s : s * A.D.F, A.D.rows);
    const int tok1 = pg_start(A.q_start, OWN ? s + 1 : (s + 1) * A.D.F, A.D.rows);
    int end;
    if (OWN) end = pg_clamp(__ldg(A.len + s), 0, A.D.cap());
    else end = A.plen ? pg_clamp(__ldg(A.plen + s), 0, A.D.n) : A.D.n;
    const int per = A.tt * A.D.g, see0 = end - (tok1 - tok0) + 1;
    int nrow = (tok1 - tok0) * A.D.g;
    if (OWN) {
        nrow = min(tok1 - tok0, A.D.max_new) * A.D.g;
        if (!pg_on_tc(A.D, nrow, end)) nrow = 0;  // pages_own.cu's
    }
    const int all = nrow;  // query rows, with or without tokens of this split
    // warps 2 and 3, once: the own rows of this CTA's row blocks, shared with the other splits
    bool own_done = OWN || QT == 2 || !A.D.prompt_own || (warp != 2 && warp != 3);
    auto own_rows = [&]() {
        for (int rt = rt0; rt * QT * per < all; rt += A.nrt) {
            const int first = rt * QT * per + 2 * sp + warp - 2, end = min(all, (rt + 1) * QT * per);
            if (D == 128) pt_own_rows<T, 4>(A, s, kh, tok0, first, end, 2 * nsplit, lane);
            else if (A.D.d == 64) pt_own_rows<T, 2>(A, s, kh, tok0, first, end, 2 * nsplit, lane);
            else pt_own_rows<T, 1>(A, s, kh, tok0, first, end, 2 * nsplit, lane);
        }
        own_done = true;
    };
    const int step = OWN ? A.D.ssplit : A.D.psplit;
    const int t0 = sp * step, t_end = min(end, t0 + step);
    if (t_end <= t0) nrow = 0;

    // there can be more row blocks than the launch has places for: a prompt with more than four times its
    // even share of the rows, or with a request that was refused for packing more than max_new
    for (int rt = rt0; rt * QT * per < nrow; rt += A.nrt) {
        const int row0 = rt * QT * per;
        const int nqt = QT == 2 && row0 + per < nrow ? 2 : 1;
        // with OWN, no further than its last row sees (one token at least: every split that the join
        // counts has a result)
        int t1 = t_end;
        if (OWN) {
            const int last = (min(nrow, row0 + QT * per) - 1) / A.D.g;
            t1 = max(t0 + 1, min(t_end, see0 + last));
        }
        const int ntl = (t1 - t0 + 127) / 128;
        // softmax warps with a valid row, per tile
        auto warps_of = [&](int t) { return (min(per, nrow - row0 - t * per) + 31) / 32; };
        if (threadIdx.x == 0) {
            tc::mbar_init(B.q_full, 1);
            for (int i = 0; i < L::SLOTS; ++i) {
                tc::mbar_init(&B.rfull[i], G ? pt_makers<QT>() : 1);
                tc::mbar_init(&B.rempty[i], 1);
            }
            for (int t = 0; t < 2; ++t) {
                tc::mbar_init(&B.s_full[t], 1);
                tc::mbar_init(&B.p_half[t], 32 * warps_of(nqt == 2 ? t : 0));
                tc::mbar_init(&B.p_full[t], 32 * warps_of(nqt == 2 ? t : 0));
            }
            tc::mbar_init(B.o_done, 1);
            tc::mbar_init(B.drain, 1);
            tc::mbar_init(B.o_final, 1);
            for (int i = 0; i < L::RAWS; ++i) {
                tc::mbar_init(&B.raw_full[i], 1);
                tc::mbar_init(&B.raw_empty[i], pt_makers<QT>());
            }
            tc::mbar_fence_init();
        }
        __syncthreads();
        tc::fence_after_sync();
        const uint32_t tmem = *tmem_slot;

        if (warp == 0) {
            // ---- TMA producer ----
            if (lane == 0) {
                tc::mbar_expect_tx(B.q_full, (uint32_t)(nqt * L::KB * per * 128));
                for (int t = 0; t < nqt; ++t)
                    for (int kb = 0; kb < L::KB; ++kb)
                        tc::tma_load_3d(sm + t * L::TILE + kb * 16384, &tm_q, 64 * kb, kh * A.D.g,
                                    tok0 + (rt * QT + t) * A.tt, B.q_full);
            }
            int issued = 0;
            if constexpr (G != 0) {
                if constexpr (QT == 1) {
                    PtRaw<D, QT, G, OWN> raw(A, s, kh, t0, t1);
                    raw.upto(B, sm, raw.halves, raw.halves, lane, abort_flag);
                    raw.drain(B, lane);
                } else {
                    pt_make<T, D, QT, G, OWN, true>(A, bars, sm, 0, lane, s, kh, t0, t1, abort_flag);
                }
            } else if (OWN) {
                // a tile is up to 128 / box boxes of box = min(page, 128) rows; the lanes look up 32
                // at a time, one lane issues (TMA takes uniform operands)
                const int lgB = A.D.lgP < 7 ? A.D.lgP : 7;
                for (int c = 0; c < 2 * ntl; ++c) {
                    const int slot = c % L::SLOTS, tb = t0 + (c >> 1) * 128;
                    if (!tc::mbar_wait_warp(&B.rempty[slot], ((c / L::SLOTS) & 1) ^ 1, abort_flag,
                                            A.err))
                        break;
                    const int boxes = (min(128, t1 - tb) + (1 << lgB) - 1) >> lgB;
                    if (lane == 0)
                        tc::mbar_expect_tx(&B.rfull[slot], (uint32_t)(boxes * L::KB * 128) << lgB);
                    __syncwarp();
                    for (int b0 = 0; b0 < boxes; b0 += 32) {
                        const int j = tb + ((b0 + lane) << lgB);
                        int row = 0;
                        if (b0 + lane < boxes)
                            row = ((pg_page(A.table + (size_t)s * A.D.maxp, j, A.D.lgP, A.D.npages,
                                            A.err) * A.D.Hkv + kh) << A.D.lgP) + (j & (A.D.P - 1));
                        for (int x = 0; x < min(32, boxes - b0); ++x) {
                            const int y = __shfl_sync(0xffffffffu, row, x);
                            if (tc::elect_one())
                                for (int kb = 0; kb < L::KB; ++kb)
                                    tc::tma_load_2d(sm + L::RING + slot * L::TILE + kb * 16384 +
                                                        ((b0 + x) << lgB) * 128,
                                                    (c & 1) ? &tm_v : &tm_k, 64 * kb, y,
                                                    &B.rfull[slot]);
                        }
                    }
                    issued = c + 1;
                }
            } else if (lane == 0) {
                for (int c = 0; c < 2 * ntl; ++c) {
                    const int slot = c % L::SLOTS;
                    if (!tc::mbar_wait(&B.rempty[slot], ((c / L::SLOTS) & 1) ^ 1, abort_flag,
                                       A.err))
                        break;
                    tc::mbar_expect_tx(&B.rfull[slot], L::TILE);
                    for (int kb = 0; kb < L::KB; ++kb)
                        tc::tma_load_4d(sm + L::RING + slot * L::TILE + kb * 16384,
                                    (c & 1) ? &tm_v : &tm_k, 64 * kb, t0 + (c >> 1) * 128, kh, s,
                                    &B.rfull[slot]);
                    issued = c + 1;
                }
            }
            if (lane == 0) {
                // copies still in flight land before the CTA goes on (at once on the normal path)
                tc::mbar_drain(B.q_full, 0);
                for (int c = issued - L::SLOTS < 0 ? 0 : issued - L::SLOTS; G == 0 && c < issued; ++c)
                    tc::mbar_drain(&B.rfull[c % L::SLOTS], (c / L::SLOTS) & 1);
            }
        } else if (warp == 1) {
            if (tc::elect_one()) {  // ---- MMA issuer ----
                const uint32_t base = tc::smem_u32(sm);
                const PtDesc d{tc::sdesc_sw128(base, 16, 1024),
                               tc::sdesc_sw128(base + L::RING, 16, 1024),
                               tc::sdesc_sw128(base + L::RING, 16384, 1024)};
                if (tc::mbar_wait(B.q_full, 0, abort_flag, A.err)) {
                    if (QT == 2 && nqt == 2)
                        pt_issue_two<T, D, QT, G>(B, d, tmem, ntl, abort_flag, A.err);
                    else
                        pt_issue_one<T, D, QT, G>(B, d, tmem, ntl, abort_flag, A.err);
                }
                // every product issued has completed before the tiles or the TMEM are reused
                tc::mma_commit(B.drain);
                tc::mbar_drain(B.drain, 0);
            }
        } else if (G != 0 && (warp == 2 || warp == 3 || (QT == 1 && warp >= 8))) {
            if constexpr (G != 0)
                pt_make<T, D, QT, G, OWN, false>(A, bars, sm, QT == 2 ? warp - 1 : (warp < 4 ? warp - 2 : warp - 6), lane, s, kh, t0, t1,
                                                 abort_flag);
        } else if (warp >= 4) {
            const int t = (warp - 4) >> 2;
            if (t < nqt && (warp & 3) < warps_of(t)) {
                if (G != 0 && nqt == 1)
                    pt_softmax_apart<T, D, QT, G, OWN, true>(A, bars, sm, tmem, warp, lane, row0, nrow, tok0, kh, t0, t1,
                                                             see0, ntl, sp, abort_flag);
                else if (G != 0 && QT == 2)
                    pt_softmax_apart<T, D, QT, G, OWN, false>(A, bars, sm, tmem, warp, lane, row0, nrow, tok0, kh, t0, t1,
                                                              see0, ntl, sp, abort_flag);
                else if (nqt == 1)
                    pt_softmax<T, D, QT, G, OWN, true>(A, B, sm, tmem, warp, lane, row0, nrow, tok0, kh,
                                                    t0, t1, see0, ntl, sp, abort_flag);
                else if (QT == 2)
                    pt_softmax<T, D, QT, G, OWN, false>(A, B, sm, tmem, warp, lane, row0, nrow, tok0,
                                                     kh, t0, t1, see0, ntl, sp, abort_flag);
            }
        } else if (!OWN && QT == 1 && !own_done) {
            own_rows();
        }
        tc::fence_before_sync();
        if ((rt + A.nrt) * QT * per >= nrow) break;
        // another round (the fence waits for the stores of the one before, so not after the last): the ring's
        // plain reads and writes before the next TMA loads
        if constexpr (D == 64 && G == 32) {
            if (A.D.d == 32) {
                __syncthreads();  // (the epilogues have read their rows)
                pt_clear(sm + L::RING, L::SLOTS * L::TILE);
            }
        }
        tc::fence_proxy_async_smem();
        __syncthreads();
        tc::fence_after_sync();
        if (*abort_flag) break;
        if (threadIdx.x == 0)
            for (int i = 0; i < L::NBAR; ++i) mbar_inval(bars + i);
    }
    if (!OWN && QT == 1 && !own_done) own_rows();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(*tmem_slot, 512);
    if (OWN) pg_end_after_prior();
}

// ---- host ------------------------------------------------------------------------------------------
// Everything of a launch but K's and V's maps.
template <int QT> PtArgs pt_args(const PgDims &D_, const PgAttn &A, bool own) {
    PtArgs P{};
    P.D = D_;
    P.tt = pg_tile_rows(D_);
    P.nrt = pg_tc_blocks(D_, own);
    P.k1 = kLog2e / sqrtf((float)D_.d);
    P.plen = A.plen;
    P.q_start = A.q_start;
    P.len = A.len;
    P.table = A.table;
    P.q = A.q;
    P.q_row = A.q_row;
    P.K = A.K;
    P.V = A.V;
    P.row_req = A.row_req;
    P.part_ml = A.part_ml;
    P.part_o = A.part_o;
    P.err = A.err;
    return P;
}
inline bool pt_q_map(CUtensorMap *tq, bool f16, const PgDims &D_, const PgAttn &A) {
    const cuuint64_t qd[3] = {(cuuint64_t)D_.d, (cuuint64_t)D_.Hq, (cuuint64_t)D_.rows};
    const long long qs[2] = {D_.d, A.q_row};
    const cuuint32_t qb[3] = {64, (cuuint32_t)D_.g, (cuuint32_t)pg_tile_rows(D_)};
    return pg_tmap(tq, f16, A.q, 3, qd, qs, qb);
}
template <typename T, int D, int QT, int G, bool OWN>
cudaError_t pt_launch(const PgDims &D_, const PtArgs &P, const CUtensorMap &tq, const CUtensorMap &tk,
                      const CUtensorMap &tv, cudaStream_t st) {
    const long long ctas = (long long)(OWN ? D_.R : D_.S) * D_.Hkv * (OWN ? D_.ns : D_.np) * P.nrt;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return pg_launch(pg_prompt_tc_kernel<T, D, QT, G, OWN>, (unsigned)ctas, pt_threads<QT, G>(),
                     PtLayout<D, QT, G>::SMEM, true, st, tq, tk, tv, P);
}

}  // namespace
}  // namespace kve
