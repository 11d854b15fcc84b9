// Shared-prompt decoding on the 5th-generation tensor cores (tcgen05, sm_103a): attention of all
// rows behind a prompt over the prompt's K/V, bf16 or fp16, d_head 64 or 128.
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
#include <cudaTypedefs.h>

#include "pages.cuh"
#include "tc_common.cuh"

namespace kve {
namespace {

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
        "r"(tc::smem_u32(bar))
        : "memory");
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
    static constexpr int NBAR = 1 + 2 * SLOTS + 8;
    static constexpr size_t SMEM = BAR + 512 + 1024;
};
template <int QT> constexpr int pt_threads() { return (4 + 4 * QT) * 32; }
constexpr float kPtRescale = 8.f;

struct PtArgs {
    PgDims D;
    int nrt, tt;  // row tiles (or pairs) per prompt and KV head, new rows per tile
    float k1;
    const int32_t *plen, *q_start;
    float2 *part_ml;
    float *part_o;
    unsigned *err;
};

// Barriers of a CTA, in shared memory.
template <int D, int QT> struct PtBars {
    uint64_t *q_full, *rfull, *rempty, *s_full, *p_full, *o_done, *drain, *o_final;
    __device__ explicit PtBars(uint64_t *b) {
        constexpr int S = PtLayout<D, QT>::SLOTS;
        q_full = b;
        rfull = b + 1;
        rempty = rfull + S;
        s_full = rempty + S;
        p_full = s_full + 2;
        o_done = p_full + 2;
        drain = o_done + 2;
        o_final = drain + 1;
    }
};

// S(i) = Q_t K_i^T into S buffer `sb`. With two row tiles sb = t and K_i is released after the last;
// with one, the buffers alternate and S(i + 1) is computed while the softmax of S(i) runs. MMAs run
// in issue order, so the product that read P from these columns is done before they are overwritten.
template <typename T, int D, int QT>
__device__ __forceinline__ bool pt_issue_s(const PtBars<D, QT> &B, uint32_t base, uint32_t tmem,
                                           int t, int sb, int i, bool wait, bool last,
                                           volatile int *abort_flag, unsigned *err) {
    using L = PtLayout<D, QT>;
    constexpr uint32_t id = tc::idesc_f16kind(128, 128, 0, !PtIsHalf<T>::value);
    const int c = 2 * i, slot = c % L::SLOTS;
    if (wait && !tc::mbar_wait(&B.rfull[slot], (c / L::SLOTS) & 1, abort_flag, err)) return false;
    tc::fence_after_sync();
    const uint32_t q = base + t * L::TILE, k = base + L::RING + slot * L::TILE;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const uint32_t o = (s >> 2) * 16384 + (s & 3) * 32;
        tc::mma_bf16(tmem + sb * 128, tc::sdesc_sw128(q + o, 16, 1024),
                     tc::sdesc_sw128(k + o, 16, 1024), id, s > 0);
    }
    tc::mma_commit(&B.s_full[sb]);
    if (last) tc::mma_commit(&B.rempty[slot]);
    return true;
}

// O_t += P(i) V_i, P from S buffer `sb`.
template <typename T, int D, int QT>
__device__ __forceinline__ bool pt_issue_pv(const PtBars<D, QT> &B, uint32_t base, uint32_t tmem,
                                            int t, int sb, uint32_t p_phase, int i, bool wait,
                                            bool last, bool final, volatile int *abort_flag,
                                            unsigned *err) {
    using L = PtLayout<D, QT>;
    constexpr uint32_t id = tc::idesc_f16kind(128, D, 1, !PtIsHalf<T>::value);
    const int c = 2 * i + 1, slot = c % L::SLOTS;
    if (wait && !tc::mbar_wait(&B.rfull[slot], (c / L::SLOTS) & 1, abort_flag, err)) return false;
    if (!tc::mbar_wait(&B.p_full[sb], p_phase, abort_flag, err)) return false;
    tc::fence_after_sync();
    const uint32_t v = base + L::RING + slot * L::TILE;
#pragma unroll
    for (int s = 0; s < 8; ++s)  // 16 tokens per step: 8 TMEM columns of P, 16 rows of V
        tc::mma_bf16_ts(tmem + 256 + t * D, tmem + sb * 128 + 8 * s,
                        tc::sdesc_sw128(v + s * 2048, 16384, 1024), id, (i > 0 || s > 0) ? 1u : 0u);
    tc::mma_commit(&B.o_done[t]);
    if (final) tc::mma_commit(B.o_final);
    if (last) tc::mma_commit(&B.rempty[slot]);
    return true;
}

// Softmax of one row tile by 4 warps (warp lg owns TMEM lanes 32 lg .. 32 lg + 31, a thread one
// row). DB: one row tile, S(i) in buffer i % 2, whose barriers complete every second tile.
template <typename T, int D, int QT, bool DB>
__device__ __forceinline__ void pt_softmax(const PtArgs &A, const PtBars<D, QT> &B, uint8_t *sm,
                                           uint32_t tmem, int warp, int lane, int row0, int nrow,
                                           int tok0, int kh, int t0, int t1, int ntl, int sp,
                                           volatile int *abort_flag) {
    using L = PtLayout<D, QT>;
    const int t = DB ? 0 : (warp - 4) >> 2, lg = warp & 3;
    const int r = lg * 32 + lane, g = A.D.g;
    const int first = row0 + t * A.tt * g;              // the tile's first row of the prompt
    const int rr = first + r;
    const bool valid = r < A.tt * g && rr < nrow;
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
        float s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(s_col + c * 32, s[c]);
        tc::tmem_wait_ld();
        const int nv = t1 - (t0 + i * 128);  // tokens of this tile
        if (nv < 128) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (c * 32 + e >= nv) s[c][e] = -INFINITY;
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
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2) m4[c] = tc::max3(m4[c], s[c][e], s[c][e + 1]);
        const float mt = tc::max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
        const float mn = fmaxf(m, mt * A.k1);
        // rows of the tile that hold no query carry whatever shared memory held: they never rescale
        const bool rescale = valid && mn > m + kPtRescale;
        const float f = (rescale && i > 0) ? tc::ex2_approx(m - mn) : 1.f;
        if (rescale) m = mn;
        const uint64_t k1_2 = tc::pk2(A.k1, A.k1), negm_2 = tc::pk2(-m, -m);
        uint64_t lsum2[4] = {0, 0, 0, 0};
        // p = 2^(s k1 - m) <= 2^8, rounded to the type of V (half a step, like V's own entries); the
        // sum l takes p before the rounding
        float pk[2][32];
#pragma unroll
        for (int j = 0; j < 64; ++j) {
            float x0, x1;
            tc::upk2(tc::fma2(tc::pk2(s[j >> 4][(2 * j) & 31], s[j >> 4][(2 * j + 1) & 31]), k1_2,
                              negm_2),
                     x0, x1);
            const float p0 = tc::ex2_approx(x0), p1 = tc::ex2_approx(x1);
            lsum2[j & 3] = tc::add2(lsum2[j & 3], tc::pk2(p0, p1));
            pk[j >> 5][j & 31] = __uint_as_float(pt_pack<T>(p0, p1));
        }
        float a[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::upk2(lsum2[k], a[2 * k], a[2 * k + 1]);
        l = fmaf(l, f, ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7])));
        // tcgen05.ld/st are warp-collective: the whole warp rescales when one of its rows does
        if (__any_sync(0xffffffffu, f != 1.f)) {
            if (!tc::mbar_wait_warp(&B.o_done[t], (i - 1) & 1, abort_flag, A.err)) {
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
        tc::tmem_st32(s_col, pk[0]);
        tc::tmem_st32(s_col + 32, pk[1]);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&B.p_full[sb]);
    }
    if (__all_sync(0xffffffffu,
                   ok && (DB ? tc::mbar_wait(B.o_final, 0, abort_flag, A.err)
                             : tc::mbar_wait(&B.o_done[t], (ntl - 1) & 1, abort_flag, A.err)))) {
        tc::fence_after_sync();
        const size_t at =
            ((size_t)sp * A.D.rows + tok0 + (valid ? rr / g : 0)) * A.D.Hq + kh * g +
            (valid ? rr % g : 0);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc::tmem_ld32(o_col + c * 32, o);
            tc::tmem_wait_ld();
            if (valid) {
                float4 *dst = reinterpret_cast<float4 *>(A.part_o + at * D + c * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
        }
        if (valid) A.part_ml[at] = make_float2(m, l);
    }
}

// Warps: 0 TMA, 1 MMA, 2-3 idle, then 4 softmax warps per row tile.
template <typename T, int D, int QT>
__global__ void __launch_bounds__(pt_threads<QT>(), 1)
    pg_prompt_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, PtArgs A) {
    using L = PtLayout<D, QT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the row tiles of a (prompt, KV head, split) are adjacent: they meet in L2 on its K/V
    int b = blockIdx.x;
    const int rt0 = b % A.nrt;
    b /= A.nrt;
    const int sp = b % A.D.np;
    b /= A.D.np;
    const int kh = b % A.D.Hkv, s = b / A.D.Hkv;
    const int tok0 = pg_start(A.q_start, s * A.D.F, A.D.rows);
    const int tok1 = pg_start(A.q_start, (s + 1) * A.D.F, A.D.rows);
    const int nrow = (tok1 - tok0) * A.D.g, per = A.tt * A.D.g;
    const int end = A.plen ? pg_clamp(__ldg(A.plen + s), 0, A.D.n) : A.D.n;
    const int t0 = sp * A.D.psplit, t1 = min(end, t0 + A.D.psplit);
    const int ntl = (t1 - t0 + 127) / 128;
    if (ntl <= 0 || rt0 * QT * per >= nrow) return;

    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    const PtBars<D, QT> B(bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::NBAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + L::NBAR + 1);
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::fence_before_sync();
    }
    if (threadIdx.x == 0) *abort_flag = 0;

    // the launch has tiles for max_new rows a request; a request refused for packing more leaves
    // more rows to go through
    for (int rt = rt0; rt * QT * per < nrow; rt += A.nrt) {
        const int row0 = rt * QT * per;
        const int nqt = QT == 2 && row0 + per < nrow ? 2 : 1;
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
                tc::mbar_init(&B.p_full[t], 32 * warps_of(nqt == 2 ? t : 0));
                tc::mbar_init(&B.o_done[t], 1);
            }
            tc::mbar_init(B.drain, 1);
            tc::mbar_init(B.o_final, 1);
            tc::mbar_fence_init();
        }
        __syncthreads();
        tc::fence_after_sync();
        const uint32_t tmem = *tmem_slot;

        if (warp == 0) {
            if (lane == 0) {  // ---- TMA producer ----
                tc::mbar_expect_tx(B.q_full, (uint32_t)(nqt * L::KB * per * 128));
                for (int t = 0; t < nqt; ++t)
                    for (int kb = 0; kb < L::KB; ++kb)
                        tma_load_3d(sm + t * L::TILE + kb * 16384, &tm_q, 64 * kb, kh * A.D.g,
                                    tok0 + (rt * QT + t) * A.tt, B.q_full);
                int issued = 0;
                for (int c = 0; c < 2 * ntl; ++c) {
                    const int slot = c % L::SLOTS;
                    if (!tc::mbar_wait(&B.rempty[slot], ((c / L::SLOTS) & 1) ^ 1, abort_flag,
                                       A.err))
                        break;
                    tc::mbar_expect_tx(&B.rfull[slot], L::TILE);
                    for (int kb = 0; kb < L::KB; ++kb)
                        tma_load_4d(sm + L::RING + slot * L::TILE + kb * 16384,
                                    (c & 1) ? &tm_v : &tm_k, 64 * kb, t0 + (c >> 1) * 128, kh, s,
                                    &B.rfull[slot]);
                    issued = c + 1;
                }
                // copies still in flight land before the CTA goes on (at once on the normal path)
                tc::mbar_drain(B.q_full, 0);
                for (int c = issued - L::SLOTS < 0 ? 0 : issued - L::SLOTS; c < issued; ++c)
                    tc::mbar_drain(&B.rfull[c % L::SLOTS], (c / L::SLOTS) & 1);
            }
        } else if (warp == 1) {
            if (lane == 0) {  // ---- MMA issuer ----
                const uint32_t base = tc::smem_u32(sm);
                bool ok = tc::mbar_wait(B.q_full, 0, abort_flag, A.err);
                if (nqt == 1) {
                    for (int i = 0; ok && i < 2 && i < ntl; ++i)
                        ok = pt_issue_s<T, D, QT>(B, base, tmem, 0, i & 1, i, true, true,
                                                  abort_flag, A.err);
                    for (int i = 0; ok && i < ntl; ++i) {
                        ok = pt_issue_pv<T, D, QT>(B, base, tmem, 0, i & 1, (i >> 1) & 1, i, true,
                                                   true, i == ntl - 1, abort_flag, A.err);
                        if (ok && i + 2 < ntl)
                            ok = pt_issue_s<T, D, QT>(B, base, tmem, 0, i & 1, i + 2, true, true,
                                                      abort_flag, A.err);
                    }
                } else {
                    for (int t = 0; ok && t < 2; ++t)
                        ok = pt_issue_s<T, D, QT>(B, base, tmem, t, t, 0, t == 0, t == 1,
                                                  abort_flag, A.err);
                    for (int i = 0; ok && i < ntl; ++i)
                        for (int t = 0; ok && t < 2; ++t) {
                            ok = pt_issue_pv<T, D, QT>(B, base, tmem, t, t, i & 1, i, t == 0, t == 1,
                                                       false, abort_flag, A.err);
                            if (ok && i + 1 < ntl)
                                ok = pt_issue_s<T, D, QT>(B, base, tmem, t, t, i + 1, t == 0, t == 1,
                                                          abort_flag, A.err);
                        }
                }
                // every product issued has completed before the tiles or the TMEM are reused
                tc::mma_commit(B.drain);
                tc::mbar_drain(B.drain, 0);
            }
        } else if (warp >= 4) {
            const int t = (warp - 4) >> 2;
            if (t < nqt && (warp & 3) < warps_of(t)) {
                if (nqt == 1)
                    pt_softmax<T, D, QT, true>(A, B, sm, tmem, warp, lane, row0, nrow, tok0, kh, t0,
                                               t1, ntl, sp, abort_flag);
                else if (QT == 2)
                    pt_softmax<T, D, QT, false>(A, B, sm, tmem, warp, lane, row0, nrow, tok0, kh, t0,
                                                t1, ntl, sp, abort_flag);
            }
        }
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        if (*abort_flag) break;
        if (threadIdx.x == 0)
            for (int i = 0; i < L::NBAR; ++i) mbar_inval(bars + i);
    }
    if (warp == 1) tc::tmem_dealloc(*tmem_slot, 512);
}

// ---- host ------------------------------------------------------------------------------------------
bool tmap(CUtensorMap *map, bool f16, const void *base, int rank, const cuuint64_t *dims,
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

template <typename T, int D, int QT>
cudaError_t go(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    using L = PtLayout<D, QT>;
    constexpr bool f16 = PtIsHalf<T>::value;
    const int tt = pg_tile_rows(D_);
    CUtensorMap tq, tk, tv;
    const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)D_.Hq, (cuuint64_t)D_.rows};
    const long long qs[2] = {D, A.q_row};
    const cuuint32_t qb[3] = {64, (cuuint32_t)D_.g, (cuuint32_t)tt};
    const cuuint64_t kd[4] = {(cuuint64_t)D, (cuuint64_t)D_.n, (cuuint64_t)D_.Hkv,
                              (cuuint64_t)D_.S};
    const long long ks[3] = {A.p_tok, A.p_head, A.p_prompt};
    const cuuint32_t kb[4] = {64, 128, 1, 1};
    if (!tmap(&tq, f16, A.q, 3, qd, qs, qb) || !tmap(&tk, f16, A.Kp, 4, kd, ks, kb) ||
        !tmap(&tv, f16, A.Vp, 4, kd, ks, kb))
        return cudaErrorInvalidValue;
    PtArgs P{};
    P.D = D_;
    P.tt = tt;
    P.nrt = (int)((D_.group_rows() + (long long)tt * QT - 1) / ((long long)tt * QT));
    P.k1 = kLog2e / sqrtf((float)D);
    P.plen = A.plen;
    P.q_start = A.q_start;
    P.part_ml = A.part_ml;
    P.part_o = A.part_o;
    P.err = A.err;
    const long long ctas = (long long)D_.S * D_.Hkv * D_.np * P.nrt;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = pg_prompt_tc_kernel<T, D, QT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)L::SMEM);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)ctas, pt_threads<QT>(), L::SMEM, st>>>(tq, tk, tv, P);
    return cudaGetLastError();
}

template <typename T>
cudaError_t by_shape(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    const int qt = pg_prompt_pairs(D);
    if (D.d == 128) return qt == 2 ? go<T, 128, 2>(D, A, st) : go<T, 128, 1>(D, A, st);
    return qt == 2 ? go<T, 64, 2>(D, A, st) : go<T, 64, 1>(D, A, st);
}

}  // namespace

cudaError_t launch_pg_prompt_tc(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_shape<__nv_bfloat16>(D, A, st) : by_shape<__half>(D, A, st);
}

}  // namespace kve
