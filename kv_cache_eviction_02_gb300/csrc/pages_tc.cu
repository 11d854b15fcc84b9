// Shared-prompt decoding on the 5th-generation tensor cores (tcgen05, sm_103a): attention of all
// rows behind a prompt over the prompt's K/V, bf16 or fp16. d_head 32 runs as 64: the boxes reach behind
// the arrays' rows, where TMA fills in zeros.
//
// The rows of a prompt's requests (new rows x g query heads of a KV head) are stacked into 128-row
// tiles, so the prompt's K/V stream from HBM once per tile or pair of tiles, however many requests
// share it. One CTA takes one or two row tiles of one prompt and KV head over a split of the tokens:
//   S_t = Q_t K^T (128 rows x 128 tokens) into TMEM, the softmax of a row in one thread (running
//   maximum, rescale of O only when it grew by 2^8), P as 16-bit pairs back into TMEM over S, and
//   O_t += P_t V with P read from TMEM and V as the MN-major B operand.
// Tiles come by TMA straight from the caller's strided arrays: Q as {d, g heads, rows} boxes, K and V
// as {d, 128 tokens} boxes of a {d, tokens, heads, prompts} map, rows behind the map filled with
// zeros. Rows between a prompt's own length and the map's end may hold anything: their scores are
// masked, and the softmax warps write zeros over their V rows in shared memory before they hand P on.
// Few rows (lookahead: 4 trajectories x 4 heads): bound by HBM; many (hundreds): by the tensor pipe.
//
// The same kernel (OWN) takes the own rows of requests that add many rows at once: K and V as boxes of
// the request's pages, scores masked at each row's own position.
#include <cudaTypedefs.h>

#include "pages_ptx.cuh"

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

// Shared memory: QT row tiles, then the K/V ring (K_0, V_0, K_1, ...), then barriers.
template <int D, int QT> struct PtLayout {
    static constexpr int KB = D / 64;  // 128-byte column blocks of a row
    static constexpr uint32_t TILE = KB * 16384;
    static constexpr int SLOTS = D == 128 ? (QT == 2 ? 5 : 6) : (QT == 2 ? 11 : 12);
    static constexpr uint32_t RING = QT * TILE, BAR = RING + SLOTS * TILE;
    static constexpr int NBAR = 1 + 2 * SLOTS + 9;
    static constexpr size_t SMEM = BAR + 512 + 1024;
};
struct PtDesc {
    uint64_t q, k, v;  // of row tile 0 and of ring place 0 as K and as V
};
template <int QT> constexpr int pt_threads() { return (4 + 4 * QT) * 32; }

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
template <int D, int QT> struct PtBars {
    uint64_t *q_full, *rfull, *rempty, *s_full, *p_half, *p_full, *o_done, *drain, *o_final;
    __device__ explicit PtBars(uint64_t *b) {
        constexpr int S = PtLayout<D, QT>::SLOTS;
        q_full = b;
        rfull = b + 1;
        rempty = rfull + S;
        s_full = rempty + S;
        p_half = s_full + 2;
        p_full = p_half + 2;
        o_done = p_full + 2;
        drain = o_done + 1;
        o_final = drain + 1;
    }
};

// Matrix descriptors advance by adding to the address field (16-byte units): building one per product
// costs the issuing thread about 150 cycles, more than the product's 64 (measured: 8 products of
// 128 x 128 x 16 took 1200 cycles with descriptors built in place, 514 with added offsets).
//
// S(i) = Q_t K_i^T into S buffer `sb`. With two row tiles sb = t; with one, the buffers alternate and
// S(i + 1) is computed while the softmax of S(i) runs. A thread's MMAs run in issue order, so the
// product that read P from these columns is done before they are overwritten.
template <typename T, int D, int QT>
__device__ __forceinline__ void pt_issue_s(const PtDesc &d, uint32_t tmem, int t, int sb, int i) {
    using L = PtLayout<D, QT>;
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
template <typename T, int D, int QT>
__device__ __forceinline__ bool pt_issue_pv(const PtBars<D, QT> &B, const PtDesc &d, uint32_t tmem,
                                            int t, int sb, uint32_t p_phase, int i, bool half_ready,
                                            volatile int *abort_flag, unsigned *err) {
    using L = PtLayout<D, QT>;
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
template <typename T, int D, int QT>
__device__ __forceinline__ bool pt_landed(const PtBars<D, QT> &B, int c, volatile int *abort_flag,
                                          unsigned *err) {
    constexpr int S = PtLayout<D, QT>::SLOTS;
    return tc::mbar_wait(&B.rfull[c % S], (c / S) & 1, abort_flag, err);
}

// One row tile: S is double-buffered, so a tile's scores are two ahead.
template <typename T, int D, int QT>
__device__ __forceinline__ bool pt_issue_one(const PtBars<D, QT> &B, const PtDesc &d, uint32_t tmem,
                                             int ntl, volatile int *abort_flag, unsigned *err) {
    constexpr int S = PtLayout<D, QT>::SLOTS;
    auto scores = [&](int i) {
        if (!pt_landed<T, D, QT>(B, 2 * i, abort_flag, err)) return false;
        pt_issue_s<T, D, QT>(d, tmem, 0, i & 1, i);
        tc::mma_commit(&B.s_full[i & 1]);
        tc::mma_commit(&B.rempty[(2 * i) % S]);
        return true;
    };
    bool ok = true;
    for (int i = 0; ok && i < 2 && i < ntl; ++i) ok = scores(i);
    for (int i = 0; ok && i < ntl; ++i) {
        ok = pt_landed<T, D, QT>(B, 2 * i + 1, abort_flag, err) &&
             pt_issue_pv<T, D, QT>(B, d, tmem, 0, i & 1, (i >> 1) & 1, i, false, abort_flag, err);
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
template <typename T, int D, int QT>
__device__ __forceinline__ bool pt_issue_two(const PtBars<D, QT> &B, const PtDesc &d, uint32_t tmem,
                                             int ntl, volatile int *abort_flag, unsigned *err) {
    constexpr int S = PtLayout<D, QT>::SLOTS;
    if (!pt_landed<T, D, QT>(B, 0, abort_flag, err)) return false;
    for (int t = 0; t < 2; ++t) {
        pt_issue_s<T, D, QT>(d, tmem, t, t, 0);
        tc::mma_commit(&B.s_full[t]);
    }
    bool v_ready = false, p_ready = false;
    for (int i = 0; i < ntl; ++i) {
        const bool more = i + 1 < ntl;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t == 0 && !v_ready && !pt_landed<T, D, QT>(B, 2 * i + 1, abort_flag, err))
                return false;
            if (!pt_issue_pv<T, D, QT>(B, d, tmem, t, t, i & 1, i, p_ready, abort_flag, err))
                return false;
            if (t == 0 && more && !pt_landed<T, D, QT>(B, 2 * i + 2, abort_flag, err)) return false;
            if (more) pt_issue_s<T, D, QT>(d, tmem, t, t, i + 1);
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
template <typename T, int D, int QT, bool OWN, bool DB>
__device__ __forceinline__ void pt_softmax(const PtArgs &A, const PtBars<D, QT> &B, uint8_t *sm,
                                           uint32_t tmem, int warp, int lane, int row0, int nrow,
                                           int tok0, int kh, int t0, int t1, int see0, int ntl,
                                           int sp, volatile int *abort_flag) {
    using L = PtLayout<D, QT>;
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
        if (nv < 128) {
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
            for (int e = 0; e < 8; ++e)
                *reinterpret_cast<float4 *>(st + lane * (D + 4) + c * 32 + 4 * e) =
                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
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

// Warps: 0 TMA, 1 MMA, 2-3 own rows of short tables, then 4 softmax warps per row tile.
template <typename T, int D, int QT, bool OWN>
__global__ void __launch_bounds__(pt_threads<QT>(), 1)
    pg_prompt_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, PtArgs A) {
    using L = PtLayout<D, QT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // what needs no input first: under programmatic launch it overlaps the end of the kernel before
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    const PtBars<D, QT> B(bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::NBAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + L::NBAR + 1);
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::fence_before_sync();
    } else if (warp == 0 && lane == 0) {
        tc::tma_prefetch_desc(&tm_k);
        tc::tma_prefetch_desc(&tm_v);
        tc::tma_prefetch_desc(&tm_q);
        *abort_flag = 0;
    }
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
                tc::mbar_init(&B.rfull[i], 1);
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
            if (OWN) {
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
                for (int c = issued - L::SLOTS < 0 ? 0 : issued - L::SLOTS; c < issued; ++c)
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
                        pt_issue_two<T, D, QT>(B, d, tmem, ntl, abort_flag, A.err);
                    else
                        pt_issue_one<T, D, QT>(B, d, tmem, ntl, abort_flag, A.err);
                }
                // every product issued has completed before the tiles or the TMEM are reused
                tc::mma_commit(B.drain);
                tc::mbar_drain(B.drain, 0);
            }
        } else if (warp >= 4) {
            const int t = (warp - 4) >> 2;
            if (t < nqt && (warp & 3) < warps_of(t)) {
                if (nqt == 1)
                    pt_softmax<T, D, QT, OWN, true>(A, B, sm, tmem, warp, lane, row0, nrow, tok0, kh,
                                                    t0, t1, see0, ntl, sp, abort_flag);
                else if (QT == 2)
                    pt_softmax<T, D, QT, OWN, false>(A, B, sm, tmem, warp, lane, row0, nrow, tok0,
                                                     kh, t0, t1, see0, ntl, sp, abort_flag);
            }
        } else if (!OWN && QT == 1 && !own_done) {
            own_rows();
        }
        tc::fence_before_sync();
        if ((rt + A.nrt) * QT * per >= nrow) break;
        // another round (the fence waits for the stores of the one before, so not after the last): the ring's
        // plain reads and writes before the next TMA loads
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
template <typename T, int D, int QT, bool OWN>
cudaError_t go(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    using L = PtLayout<D, QT>;
    constexpr bool f16 = PtIsHalf<T>::value;
    const int tt = pg_tile_rows(D_);
    const cuuint64_t d = D_.d, one = 1;
    CUtensorMap tq, tk, tv;
    const cuuint64_t qd[3] = {d, (cuuint64_t)D_.Hq, (cuuint64_t)D_.rows};
    const long long qs[2] = {D_.d, A.q_row};
    const cuuint32_t qb[3] = {64, (cuuint32_t)D_.g, (cuuint32_t)tt};
    // the prompt's {columns, tokens, heads, prompts}, or the pool's {columns, rows}
    const cuuint64_t kd[4] = {d, OWN ? (cuuint64_t)D_.npages * D_.Hkv * D_.P : (cuuint64_t)D_.n,
                              OWN ? one : (cuuint64_t)D_.Hkv, OWN ? one : (cuuint64_t)D_.S};
    const long long ks[3] = {OWN ? D_.d : A.p_tok, A.p_head, A.p_prompt};
    const cuuint32_t kb[4] = {64, OWN && D_.P < 128 ? (cuuint32_t)D_.P : 128u, 1, 1};
    const int rank = OWN ? 2 : 4;
    if (!pg_tmap(&tq, f16, A.q, 3, qd, qs, qb) ||
        !pg_tmap(&tk, f16, OWN ? A.K : A.Kp, rank, kd, ks, kb) ||
        !pg_tmap(&tv, f16, OWN ? A.V : A.Vp, rank, kd, ks, kb))
        return cudaErrorInvalidValue;
    PtArgs P{};
    P.D = D_;
    P.tt = tt;
    P.nrt = pg_tc_blocks(D_, OWN);
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
    const long long ctas = (long long)(OWN ? D_.R : D_.S) * D_.Hkv * (OWN ? D_.ns : D_.np) * P.nrt;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return pg_launch(pg_prompt_tc_kernel<T, D, QT, OWN>, (unsigned)ctas, pt_threads<QT>(), L::SMEM,
                     true, st, tq, tk, tv, P);
}

template <typename T, bool OWN>
cudaError_t by_shape(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    const int qt = pg_pairs(D, OWN ? D.max_new : D.group_rows());
    if (D.d == 128) return qt == 2 ? go<T, 128, 2, OWN>(D, A, st) : go<T, 128, 1, OWN>(D, A, st);
    return qt == 2 ? go<T, 64, 2, OWN>(D, A, st) : go<T, 64, 1, OWN>(D, A, st);
}

}  // namespace

bool pg_tmap(CUtensorMap *map, bool f16, const void *base, int rank, const cuuint64_t *dims,
             const long long *strides, const cuuint32_t *box) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!fn) return false;
    cuuint64_t bytes[4];
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = (cuuint64_t)strides[i] * 2;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
              const_cast<void *>(base), dims, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_pg_prompt_tc(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_shape<__nv_bfloat16, false>(D, A, st)
                               : by_shape<__half, false>(D, A, st);
}

cudaError_t launch_pg_own_tc(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_shape<__nv_bfloat16, true>(D, A, st)
                               : by_shape<__half, true>(D, A, st);
}

}  // namespace kve
