// Shared-prompt decoding, fp32: attention over the prompts and the requests' own rows on the CUDA cores,
// in one launch.
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
// accumulators, O of each chunk in fresh ones that are then added to the running O in fp32. (FFMA with a
// lane per D/32 columns took 4 times the instructions: a lookahead step over 32K rows 143 us.)
// Everything else is fp32; the factor log2 e / sqrt d is carried as two floats, since its rounding would
// shift every score the same way.
#include "pages.cuh"

namespace kve {
namespace {

constexpr int kF3Warps = kPgF32Warps, kF3Threads = 32 * kF3Warps;
constexpr int kF3Tok = kPgF32Chunk, kF3Rows = kPgF32Rows, kF3NT = kF3Rows / 8;

// Rows in shared memory are padded so that the fragments' reads fall into 32 different banks: K's by 4
// floats (8 tokens x 4 columns), V's by 8 (4 tokens x 8 columns).
template <int D> constexpr int f3_stages() { return D == 128 ? 2 : (D == 64 ? 4 : 6); }
template <int D> constexpr int f3_stage_floats() { return kF3Tok * (2 * D + 12); }
template <int D> constexpr int f3_smem() {
    return kF3Warps * f3_stages<D>() * f3_stage_floats<D>() * 4;
}

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

// Where a warp stands in the line of chunks.
struct Cursor {
    int e, len, first, rows, nq;  // entity, its tokens, its first packed row, its query rows per KV head
    int cr, nb;                   // chunks per unit, row blocks
    int kh, rb, c;                // KV head, row block, chunk of the unit
    __device__ __forceinline__ void enter(const PgDims &D, const PgAttn &A, int entity) {
        e = entity;
        pg_f32_entity(D, A, e, &len, &first, &nq, &rows, &cr, &nb);
        kh = rb = c = 0;
    }
    // to the next chunk; only called when there is one
    __device__ __forceinline__ void next(const PgDims &D, const PgAttn &A) {
        if (++c < cr) return;
        c = 0;
        if (++rb < nb) return;
        rb = 0;
        if (++kh < D.Hkv) return;
        do enter(D, A, e + 1);
        while ((cr == 0 || nb == 0) && e + 1 < D.S + D.R);
    }
};

template <int D>
__global__ void __launch_bounds__(kF3Threads, 1) pg_f32_kernel(PgDims D_, PgAttn A, PgOwn W) {
    constexpr int NST = f3_stages<D>(), SF = f3_stage_floats<D>(), NT = kF3NT;
    constexpr int KP = D + 4, VP = D + 8;  // floats from one row to the next
    extern __shared__ __align__(16) float sm[];
    __shared__ long long csum[kF3Threads + 1];
    __shared__ int usum[kF3Threads + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pg_wait_prior();
    pg_launch_dependents();
    const PgShare sh = pg_share<kF3Threads>(
        D_.S + D_.R, D_.Hkv, csum, usum, W, [&](int e, int *cr, int *nb) {
            int len, first, nq, rows;
            pg_f32_entity(D_, A, e, &len, &first, &nq, &rows, cr, nb);
        });
    const int w = blockIdx.x * kF3Warps + warp;
    const long long X0 = w * sh.cpw;
    const int n = (int)min(sh.total - X0, sh.cpw);  // chunks of this warp
    if (n <= 0) return;
    Cursor cc;
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
    Cursor ca = cc;  // runs ahead: the chunks to load

    float *ring = sm + warp * (NST * SF);
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    // lane t (mod 16) looks after token t of a chunk: where it lies is asked two chunks before it is
    // loaded, so the answer of the block table is not waited for
    struct Where {
        long long base;  // prompts: the element offset of the head's first row
        int page, at;    // at: -1 behind the last token
        bool own;
    };
    auto where = [&]() -> Where {
        const int j = ca.c * kF3Tok + (lane & (kF3Tok - 1));
        Where x{0, 0, j < ca.len ? j : -1, ca.e >= D_.S};
        if (!x.own) {
            x.base = ca.e * A.p_prompt + ca.kh * A.p_head;
        } else if (x.at >= 0) {
            x.page = __ldg(A.table + (size_t)(ca.e - D_.S) * D_.maxp + (j >> D_.lgP));
            x.at = (ca.kh << D_.lgP) + (j & (D_.P - 1));
        }
        return x;
    };
    auto load = [&](int place, const Where &x) {
        constexpr int WPR = D / 4, RPI = 32 / WPR;  // 16-byte words per row, rows per instruction
        const float *Kb = static_cast<const float *>(x.own ? A.K : A.Kp);
        const float *Vb = static_cast<const float *>(x.own ? A.V : A.Vp);
        long long o = -1;
        if (x.at >= 0)
            o = x.own ? ((long long)pg_page_id(x.page, D_.npages, A.err) * (D_.Hkv << D_.lgP) + x.at) * D
                      : x.base + x.at * A.p_tok;
        const uint32_t dst = ring_s + (uint32_t)(place * SF * 4 + (lane % WPR) * 16);
#pragma unroll
        for (int i = 0; i < kF3Tok / RPI; ++i) {
            const int row = i * RPI + lane / WPR;
            const long long r = __shfl_sync(0xffffffffu, o, row);
            const long long at = (r < 0 ? 0 : r) + (lane % WPR) * 4;
            cp16(dst + row * KP * 4, Kb + at, r >= 0);
            cp16(dst + (kF3Tok * KP + row * VP) * 4, Vb + at, r >= 0);
        }
    };
    float q[NT][D / 8][2];                    // B operand of S^T: query row lane / 4 of each block
    float o[NT][D / 16][4], m[NT][2], l[NT][2];  // this lane's query rows 2 (lane % 4), + 1
    int see[NT][2], live;                     // tokens they see; the unit's rows
    auto begin = [&]() {                      // of a unit, or of this warp's part of one
        const int row0 = cc.rb * kF3Rows;
        live = min(kF3Rows, cc.rows - row0);
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            const int rr = row0 + 8 * b + (lane >> 2), t = rr < cc.rows ? rr / D_.g : 0;
            const float *qp = static_cast<const float *>(A.q) + (cc.first + t) * A.q_row +
                              (size_t)(cc.kh * D_.g + (rr < cc.rows ? rr - t * D_.g : 0)) * D +
                              (lane & 3);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                q[b][k][0] = rr < cc.rows ? __ldg(qp + 8 * k) : 0.f;
                q[b][k][1] = rr < cc.rows ? __ldg(qp + 8 * k + 4) : 0.f;
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
    int asked = 1, ahead = 0;
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
#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) {
        if (ahead < n) {
            load(ahead++, x0);
            x0 = x1;
            ask();
        }
        cp_commit();
    }
    const double k1 = 1.4426950408889634074 / sqrt((double)D);
    const float k_hi = (float)k1, k_lo = (float)(k1 - (double)k_hi);
    int slot = 0, fill = NST - 1;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        if (ahead < n) {
            load(fill, x0);
            ++ahead;
            x0 = x1;
            ask();
        }
        cp_commit();
        if (++fill == NST) fill = 0;
        if (i > 0 && cc.c == 0) begin();
        cp_wait<NST - 1>();
        __syncwarp();
        const float *ks = ring + slot * SF, *vs = ks + kF3Tok * KP;
        if (++slot == NST) slot = 0;
        const int nb = live > 8 ? 2 : 1;  // blocks with a row
        // S^T, in three accumulators: hi hi of even and of odd steps, and the rest
        float s0[NT][4], s1[NT][4], s2[NT][4];
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) s0[b][e] = s1[b][e] = s2[b][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                split(ks[((lane >> 2) + 8 * (e & 1)) * KP + 8 * k + 4 * (e >> 1) + (lane & 3)], hi[e],
                      lo[e]);
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                if (b >= nb) break;
                uint32_t h0, l0, h1, l1;
                split(q[b][k][0], h0, l0);
                split(q[b][k][1], h1, l1);
                mma1688(k & 1 ? s1[b] : s0[b], hi, h0, h1);
                mma1688(s2[b], hi, l0, l1);
                mma1688(s2[b], lo, h0, h1);
            }
        }
        const int tok = cc.c * kF3Tok + (lane >> 2);
        uint32_t ph[NT][2][2], pl[NT][2][2];  // B operand of O^T: tokens 8 x .. 8 x + 7
        float f[NT][2];                       // what the rows' O and l shrink by
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            if (b >= nb) break;
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
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            float t[NT][4];
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) t[b][e] = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    split(vs[(8 * x + 4 * (e >> 1) + (lane & 3)) * VP + 16 * j + 8 * (e & 1) +
                             (lane >> 2)],
                          hi[e], lo[e]);
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    if (b >= nb) break;
                    mma1688(t[b], lo, ph[b][x][0], ph[b][x][1]);
                    mma1688(t[b], hi, pl[b][x][0], pl[b][x][1]);
                    mma1688(t[b], hi, ph[b][x][0], ph[b][x][1]);
                }
            }
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                if (b >= nb) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[b][j][e] = fmaf(o[b][j][e], f[b][e & 1], t[b][e]);
            }
        }
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
                    float *dst = W.o + row * D + (lane >> 2);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        dst[16 * j] = o[b][j][e];
                        dst[16 * j + 8] = o[b][j][e + 2];
                    }
                }
            ++unit;
        }
        if (i + 1 < n) cc.next(D_, A);
        __syncwarp();  // the chunk's readers are done: the next issue may overwrite it
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
