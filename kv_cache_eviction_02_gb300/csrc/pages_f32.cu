// Shared-prompt decoding, fp32: attention over the prompts and the requests' own rows in one launch,
// with warp-level matrix products.
//
// The work of all prompts and all requests stands in one line: entities (the prompts, then the
// requests), of each its units (KV head, block of 16 query rows), of each its chunks of 16 tokens; every
// warp takes the same number of consecutive chunks and leaves one partial result per unit it has seen a
// piece of, at place (unit index + warp index). (pages_own.cu deals out the own rows of 16-bit types in
// the same way.)
//
// The products run on the tensor cores as sums of three tf32 products: x = hi + lo, hi of 11 and lo of
// the next 11 bits, x y = hi hi + hi lo + lo hi up to 2^-21 |x y| (fp32 carries 2^-24; the errors of d
// products of either sign add up to less than the rounding of their fp32 sum). They are taken transposed,
// S^T = K Q^T and O^T = V^T P^T in m16n8k8 fragments: 16 tokens (or output columns) on the wide side, 8
// query rows on the narrow one. The tensor cores' own sums are kept short: the scores in three
// accumulators, O of each chunk in fresh ones that are then added to the running O in fp32. A
// lookahead step over 32K rows (8 KV heads of d 128, 268 MB) takes 58 us, 4.6 TB/s: bound by the
// instructions of 8 warps per SM and their latencies, 1.5 times the time of its bytes (d 128: 255 registers
// and 114 bytes of spills a thread, 64 and 32 none. FFMA with a lane per
// D/32 columns 143 us; 6 warps with whole chunks in the ring and 4-byte fragment loads 88).
// Everything else is fp32; the factor log2 e / sqrt d is carried as two floats, since its rounding would
// shift every score the same way.
#include <type_traits>

#include "pages.cuh"

namespace kve {
namespace {

constexpr int kF3Warps = kPgF32Warps, kF3Threads = 32 * kF3Warps;
constexpr int kF3Tok = kPgChunk, kF3Rows = kPgF32Rows, kF3NT = kF3Rows / 8;

// A warp's ring holds K and V of a chunk as items of their own (K_0, V_0, K_1, ...): K's place is free as
// soon as the scores are there, so 3 items keep as many bytes on their way as two whole chunks would, and
// leave room for 8 warps. Fragments are read 16 bytes a lane: the order of the d products is free, so the
// four columns that a lane reads of K (and of Q) at once serve two k-steps, and the order of the output
// columns is too, so those of V serve two m-tiles. Row pitches put the rows that 8 lanes read at once into
// different banks: K's 64 bytes apart (2 rows x 4 lanes), V's 32 (4 rows x 2 lanes).
template <int D> constexpr int f3_slots() { return D == 128 ? 3 : (D == 64 ? 5 : 7); }  // odd
template <int D> constexpr int f3_kpitch() { return D + 16; }
template <int D> constexpr int f3_vpitch() { return D + 8; }
template <int D> constexpr int f3_item() { return kF3Tok * f3_kpitch<D>(); }  // floats
template <int D> constexpr int f3_smem() { return kF3Warps * f3_slots<D>() * f3_item<D>() * 4; }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on) {
    // src-size 0 fills the 16 bytes with zeros: rows behind the last token hold anything
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// x = hi + lo, hi rounded to tf32 (the tensor cores read the upper 19 bits of lo).
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kF3Threads, 1) pg_f32_kernel(PgDims D_, PgAttn A, PgOwn W) {
    constexpr int NS = f3_slots<D>(), SF = f3_item<D>(), NT = kF3NT;
    constexpr int AHEAD = (NS - 1) / 2;  // chunks asked for before the current one
    constexpr int KP = f3_kpitch<D>(), VP = f3_vpitch<D>();
    extern __shared__ __align__(16) float sm[];
    __shared__ long long csum[kF3Threads + 1];
    __shared__ int usum[kF3Threads + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pg_wait_prior();
    pg_launch_dependents();
    const PgShare sh = pg_share<kF3Threads>(
        D_.S + D_.R, D_.Hkv, csum, usum, W, [&](int e, int *cr, int *nb) {
            int len, first, nq, rows;
            pg_unit_entity<true>(D_, A, e, &len, &first, &nq, &rows, cr, nb);
        });
    const int w = blockIdx.x * kF3Warps + warp;
    const long long X0 = w * sh.cpw;
    const int n = (int)min(sh.total - X0, sh.cpw);  // chunks of this warp
    if (n <= 0) return;
    PgCursor<true> cc;
    int unit;
    {
        long long x;
        int e;
        pg_share_find<kF3Threads>(csum, usum, sh, X0, &e, &x, &unit);
        cc.enter(D_, A, e);
        while (x >= (long long)cc.cr * cc.nb * D_.Hkv) {
            x -= (long long)cc.cr * cc.nb * D_.Hkv;
            unit += cc.nb * D_.Hkv;
            cc.enter(D_, A, cc.e + 1);
        }
        const int u = (int)pg_div(x, cc.cr);
        cc.c = (int)(x - (long long)u * cc.cr);
        cc.kh = u / cc.nb;
        cc.rb = u - cc.kh * cc.nb;
        unit += u;
    }
    PgCursor<true> ca = cc;  // runs ahead: the chunks to load

    float *ring = sm + warp * (NS * SF);
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    // lane t (mod 16) looks after token t of a chunk: where it lies is asked a chunk before it is loaded,
    // so the answer of the block table is not waited for
    struct Where {
        const float *K, *V;  // of row 0
        long long step;      // elements from one row to the next
        int page, at;        // own rows: its page and the row in it; prompts: -, row. at < 0: no such token
        bool own;
    };
    auto where = [&]() -> Where {
        const int j = ca.c * kF3Tok + (lane & (kF3Tok - 1));
        Where x{static_cast<const float *>(A.K), static_cast<const float *>(A.V), D, 0,
                j < ca.len ? j : -1, ca.e >= D_.S};
        if (!x.own) {
            const long long base = ca.e * A.p_prompt + ca.kh * A.p_head;
            x.K = static_cast<const float *>(A.Kp) + base;
            x.V = static_cast<const float *>(A.Vp) + base;
            x.step = A.p_tok;
        } else if (x.at >= 0) {
            x.page = __ldg(A.table + (size_t)(ca.e - D_.S) * D_.maxp + (j >> D_.lgP));
            x.at = (ca.kh << D_.lgP) + (j & (D_.P - 1));
        }
        return x;
    };
    // the row that a lane's token lies in (below 2^31 in either array), -1 behind the last one
    auto row_of = [&](const Where &x) {
        return x.own && x.at >= 0
                   ? pg_page_id(x.page, D_.npages, A.err) * (D_.Hkv << D_.lgP) + x.at
                   : x.at;
    };
    auto load = [&](int place, const float *rows, long long step, int row, int pitch) {
        // 8 lanes a row, 128 bytes at a time
        const uint32_t dst = ring_s + (uint32_t)(place * SF + (lane >> 3) * pitch + (lane & 7) * 4) * 4;
#pragma unroll
        for (int i = 0; i < kF3Tok / 4; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, 4 * i + (lane >> 3));
            const float *src = rows + (r < 0 ? 0 : r) * step + (lane & 7) * 4;
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                cp16(dst + (4 * i * pitch + 32 * c) * 4, src + 32 * c, r >= 0);
        }
    };
    float q[NT][D / 8][2];  // B operand of S^T: query row lane / 4 of each block
    // this lane's query rows 2 (lane % 4), + 1 of each block; output columns 32 (j / 2) + 4 (lane / 4) +
    // 2 (j % 2), + 1
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    int see[NT][2], live;                     // tokens they see; the unit's rows
    auto begin = [&]() {                      // of a unit, or of this warp's part of one
        const int row0 = cc.rb * kF3Rows;
        live = min(kF3Rows, cc.rows - row0);
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            const int rr = row0 + 8 * b + (lane >> 2), t = rr < cc.rows ? rr / D_.g : 0;
            const float4 *qp = reinterpret_cast<const float4 *>(
                                   static_cast<const float *>(A.q) + (cc.first + t) * A.q_row +
                                   (size_t)(cc.kh * D_.g + (rr < cc.rows ? rr - t * D_.g : 0)) * D) +
                               (lane & 3);
#pragma unroll
            for (int p = 0; p < D / 16; ++p) {
                const float4 x = rr < cc.rows ? __ldg(qp + 4 * p) : make_float4(0.f, 0.f, 0.f, 0.f);
                q[b][2 * p][0] = x.x;
                q[b][2 * p][1] = x.y;
                q[b][2 * p + 1][0] = x.z;
                q[b][2 * p + 1][1] = x.w;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int qr = row0 + 8 * b + (lane & 3) * 2 + e;
                see[b][e] = qr >= cc.rows ? 0
                                          : (cc.e < D_.S ? cc.len : cc.len - cc.nq + 1 + qr / D_.g);
                m[b][e] = kPgNoMax;
                l[b][e] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[b][j][e] = 0.f;
        }
    };
    int asked = 1;
    Where x0 = where(), x1 = x0;
    begin();  // its loads of Q run beside the table's
    auto ask = [&]() {
        if (asked < n) {
            ca.next(D_, A);
            x1 = where();
            ++asked;
        }
    };
    ask();
    // chunk i + AHEAD goes into the places of V_(i-1) and K_i; a group of copies per item, empty ones
    // behind the last
    int fill = 0, row = -1;
    auto load_k = [&](int chunk) {
        if (chunk < n) {
            row = row_of(x0);
            load(fill, x0.K, x0.step, row, KP);
        }
        cp_commit();
        if (++fill == NS) fill = 0;
    };
    auto load_v = [&](int chunk) {
        if (chunk < n) {
            load(fill, x0.V, x0.step, row, VP);
            x0 = x1;
            ask();
        }
        cp_commit();
        if (++fill == NS) fill = 0;
    };
#pragma unroll 1
    for (int i = 0; i < AHEAD; ++i) {
        load_k(i);
        load_v(i);
    }
    const double k1 = 1.4426950408889634074 / sqrt((double)D);
    const float k_hi = (float)k1, k_lo = (float)(k1 - (double)k_hi);
    int slot = 0;
    // one chunk; NB: blocks of query rows that hold one
    auto chunk = [&](int i, auto nb) {
        constexpr int NB = decltype(nb)::value;
        cp_wait<NS - 1>();
        __syncwarp();
        const float *ks = ring + slot * SF + (lane >> 2) * KP + (lane & 3) * 4;
        if (++slot == NS) slot = 0;
        // S^T, in three accumulators: hi hi of even and of odd steps, and the rest
        float s0[NB][4], s1[NB][4], s2[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) s0[b][e] = s1[b][e] = s2[b][e] = 0.f;
#pragma unroll
        for (int p = 0; p < D / 16; ++p) {
            const float4 x = *reinterpret_cast<const float4 *>(ks + 16 * p);
            const float4 y = *reinterpret_cast<const float4 *>(ks + 8 * KP + 16 * p);
            const float a[2][4] = {{x.x, y.x, x.y, y.y}, {x.z, y.z, x.w, y.w}};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split(a[k][e], hi[e], lo[e]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t h0, l0, h1, l1;
                    split(q[b][2 * p + k][0], h0, l0);
                    split(q[b][2 * p + k][1], h1, l1);
                    mma1688(k ? s1[b] : s0[b], hi, h0, h1);
                    mma1688(s2[b], hi, l0, l1);
                    mma1688(s2[b], lo, h0, h1);
                }
            }
        }
        __syncwarp();  // K's readers are done: V of a later chunk goes there
        load_v(i + AHEAD);
        const int tok = cc.c * kF3Tok + (lane >> 2);
        uint32_t ph[NB][2][2], pl[NB][2][2];  // B operand of O^T: tokens 8 x .. 8 x + 7
        float f[NB][2];                       // what the rows' O and l shrink by
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float a = (s0[b][e] + s1[b][e]) + s2[b][e];
                float c = (s0[b][e + 2] + s1[b][e + 2]) + s2[b][e + 2];
                a = tok < see[b][e] ? a : -INFINITY;
                c = tok + 8 < see[b][e] ? c : -INFINITY;
                float x = fmaxf(a, c);
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                const float mn = x == -INFINITY ? m[b][e] : fmaxf(m[b][e], fmaf(x, k_hi, x * k_lo));
                f[b][e] = exp2f(m[b][e] - mn);
                m[b][e] = mn;
                // s log2 e / sqrt d - m with one rounding near the result
                p[e] = a == -INFINITY ? 0.f : exp2f(fmaf(a, k_hi, fmaf(a, k_lo, -mn)));
                p[e + 2] = c == -INFINITY ? 0.f : exp2f(fmaf(c, k_hi, fmaf(c, k_lo, -mn)));
                l[b][e] = fmaf(l[b][e], f[b][e], p[e] + p[e + 2]);
            }
            // from (token lane / 4, row 2 (lane % 4) + e) to (token lane % 4 + 4 h, row lane / 4)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int from = ((lane & 3) + 4 * h) * 4 + (lane >> 3);
                    const float even = __shfl_sync(0xffffffffu, p[2 * x], from);
                    const float odd = __shfl_sync(0xffffffffu, p[2 * x + 1], from);
                    split(lane & 4 ? odd : even, ph[b][x][h], pl[b][x][h]);
                }
        }
        cp_wait<NS - 1>();
        __syncwarp();
        const float *vs = ring + slot * SF + (lane & 3) * VP + (lane >> 2) * 4;
        if (++slot == NS) slot = 0;
#pragma unroll
        for (int jj = 0; jj < D / 32; ++jj) {
            float t[2][NB][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[k][b][e] = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4 v = *reinterpret_cast<const float4 *>(vs + 8 * x * VP + 32 * jj);
                const float4 w = *reinterpret_cast<const float4 *>(vs + (8 * x + 4) * VP + 32 * jj);
                const float a[2][4] = {{v.x, v.y, w.x, w.y}, {v.z, v.w, w.z, w.w}};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split(a[k][e], hi[e], lo[e]);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        mma1688(t[k][b], lo, ph[b][x][0], ph[b][x][1]);
                        mma1688(t[k][b], hi, pl[b][x][0], pl[b][x][1]);
                        mma1688(t[k][b], hi, ph[b][x][0], ph[b][x][1]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[b][2 * jj + k][e] = fmaf(o[b][2 * jj + k][e], f[b][e & 1], t[k][b][e]);
        }
    };
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        load_k(i + AHEAD);
        if (i > 0 && cc.c == 0) begin();
        if (live > 8) chunk(i, std::integral_constant<int, 2>());
        else chunk(i, std::integral_constant<int, 1>());
        if (i == n - 1 || cc.c == cc.cr - 1) {  // the piece ends
            const long long seg = (long long)unit + w;
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[b][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    const int qr = 8 * b + (lane & 3) * 2 + e;
                    // (row starts that are no sums of lengths can ask for more places than there are)
                    if (qr >= live || (unsigned long long)seg >= W.segs) continue;
                    const size_t row = (size_t)seg * W.seg_rows + qr;
                    if (lane < 4) W.ml[row] = make_float2(m[b][e], x);
                    float4 *dst = reinterpret_cast<float4 *>(W.o + row * D) + (lane >> 2);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
                        dst[8 * j] = make_float4(o[b][2 * j][e], o[b][2 * j][e + 2],
                                                 o[b][2 * j + 1][e], o[b][2 * j + 1][e + 2]);
                }
            ++unit;
        }
        if (i + 1 < n) cc.next(D_, A);
        __syncwarp();  // V's readers are done: K of a later chunk goes there
    }
}

template <int D> cudaError_t go(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    return pg_launch(pg_f32_kernel<D>, pg_own_ctas(D_), kF3Threads, f3_smem<D>(), true, st, D_, A,
                     A.own);
}

}  // namespace

cudaError_t launch_pg_f32(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.d == 128 ? go<128>(D, A, st) : (D.d == 64 ? go<64>(D, A, st) : go<32>(D, A, st));
}

}  // namespace kve
