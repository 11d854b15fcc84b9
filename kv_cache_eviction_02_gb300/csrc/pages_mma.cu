// Shared-prompt decoding, 16-bit types: attention of the requests' own rows (and of prompts whose
// heads the tcgen05 kernel does not take) with warp-level matrix products.
//
// Own rows are read by g query heads of one or a few new rows, so a request and KV head have 1 to a
// few dozen query rows over its K/V: bound by HBM, with 2 g flops per byte at one new row. The
// products run as m16n8k16 fragments in registers: 16 query rows meet 16 tokens per step and warp,
// which a 128-row tcgen05 tile would leave almost empty, and the weights P go from the accumulator
// of S = Q K^T straight into the A fragment of P V without touching shared memory.
#include "pages.cuh"

namespace kve {
namespace {

constexpr int kMmThreads = 128, kMmWarps = 4, kMmTok = 16;  // tokens per warp and step

template <int D> constexpr int mm_stages() { return D == 128 ? 3 : 4; }
template <int D> constexpr int mm_stage_bytes() { return kMmTok * D * 2 * 2; }  // K and V
template <int D> constexpr int mm_smem() { return kMmWarps * mm_stages<D>() * mm_stage_bytes<D>(); }

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
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                 uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two weights as a 16-bit pair. A weight is at most 2^8 (see kMmRescale) and rounds to half a step
// of the type, as V's own entries did; their sum l is taken in fp32 before the rounding.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-byte chunk c of a row of D 16-bit values, placed so that the 8 rows of an ldmatrix matrix fall
// into 8 different groups of banks.
template <int D> __device__ __forceinline__ uint32_t mm_off(int row, int c) {
    const int x = D >= 64 ? (row & 7) : ((row >> 1) & 3);
    return (uint32_t)(row * (D * 2) + ((c ^ x) << 4));
}

constexpr float kMmRescale = 8.f;  // O is rescaled when a row's maximum grew by more than 2^8

// RW = 1: the CTA's 4 warps share 16 query rows and split the tokens, 16 at a time, each with a ring
// of its own (no barrier in the loop); their results are joined in shared memory at the end.
// RW = 4: each warp has 16 rows of its own and the ring's 64 tokens per step serve all 4.
template <typename T, int D, int RW, bool OWN>
__global__ void __launch_bounds__(kMmThreads, 2)
    pg_attn_mma_kernel(PgDims D_, PgAttn A, int nblk) {
    constexpr int NST = mm_stages<D>(), SB = mm_stage_bytes<D>(), CPR = D / 8;  // chunks per row
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float2 sml[kMmWarps][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nsplit = OWN ? D_.ns : D_.np;
    int b = blockIdx.x;
    const int sp = b % nsplit;
    b /= nsplit;
    const int rb0 = b % nblk;
    b /= nblk;
    const int kh = b % D_.Hkv, u = b / D_.Hkv;
    const int r0 = OWN ? u : u * D_.F, r1 = OWN ? u + 1 : r0 + D_.F;
    const int tok0 = pg_start(A.q_start, r0, D_.rows), tok1 = pg_start(A.q_start, r1, D_.rows);
    const int nrow = (tok1 - tok0) * D_.g;
    int end;
    if (OWN) end = pg_clamp(__ldg(A.len + u), 0, D_.cap());
    else end = A.plen ? pg_clamp(__ldg(A.plen + u), 0, D_.n) : D_.n;
    const int step = OWN ? D_.ssplit : D_.psplit;
    const int t0 = sp * step, t1 = min(end, t0 + step);
    if (t0 >= t1 || rb0 * 16 * RW >= nrow) return;

    const T *Kb = static_cast<const T *>(OWN ? A.K : A.Kp);
    const T *Vb = static_cast<const T *>(OWN ? A.V : A.Vp);
    if (!OWN) {
        Kb += u * A.p_prompt + kh * A.p_head;
        Vb += u * A.p_prompt + kh * A.p_head;
    }
    const int32_t *trow = A.table + (size_t)(OWN ? u : 0) * D_.maxp;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const int iters = (t1 - t0 + 63) / 64;
    const float k1 = kLog2e * rsqrtf((float)D);

    // the element offset of token j's row (lanes 0-15 hold a step's 16 tokens); -1 behind the end
    auto row_of = [&](int j) -> long long {
        if (j >= t1) return -1;
        if (OWN) {
            const int page = pg_page(trow, j, D_.lgP, D_.npages, A.err);
            return (long long)((((size_t)page * D_.Hkv + kh) << D_.lgP) + (j & (D_.P - 1))) * D;
        }
        return (long long)j * A.p_tok;
    };
    // this warp's 16 tokens of step `it` into its ring: consecutive lanes take a row's chunks
    auto load = [&](int it, long long at) {
        const uint32_t dst = ring + (uint32_t)((warp * NST + it % NST) * SB);
        constexpr int RPI = 32 / CPR;  // rows per instruction
        const int c = lane % CPR;
#pragma unroll
        for (int i = 0; i < kMmTok / RPI; ++i) {
            const int row = i * RPI + lane / CPR;
            const long long o = __shfl_sync(0xffffffffu, at, row);
            const uint32_t d = dst + mm_off<D>(row, c);
            cp16(d, Kb + (o < 0 ? 0 : o) + c * 8, o >= 0);
            cp16(d + SB / 2, Vb + (o < 0 ? 0 : o) + c * 8, o >= 0);
        }
    };

    for (int rb = rb0; rb * 16 * RW < nrow; rb += nblk) {
        // Q fragments: this lane's rows lane / 4 and lane / 4 + 8
        uint32_t qf[D / 16][4];
        int see[2], tokr[2], hr[2];
        bool live[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int rr = rb * 16 * RW + (RW > 1 ? warp * 16 : 0) + (lane >> 2) + 8 * x;
            live[x] = rr < nrow;
            tokr[x] = tok0 + (live[x] ? rr / D_.g : 0);
            hr[x] = kh * D_.g + (live[x] ? rr % D_.g : 0);
            see[x] = !live[x] ? t0
                              : (OWN ? min(t1, end - (tok1 - tok0) + 1 + (tokr[x] - tok0)) : t1);
            const T *qp = static_cast<const T *>(A.q) + tokr[x] * A.q_row + (size_t)hr[x] * D +
                          (lane & 3) * 2;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][x] = live[x] ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * k)) : 0u;
                qf[k][x + 2] =
                    live[x] ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * k + 8)) : 0u;
            }
        }
        float o[D / 8][4], m[2] = {kPgNoMax, kPgNoMax}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

        const int mine = t0 + warp * kMmTok + (lane & 15);
        long long at = row_of(mine);
#pragma unroll
        for (int it = 0; it < NST - 1; ++it) {
            if (it < iters) load(it, at);
            cp_commit();
            at = row_of(mine + (it + 1) * 64);
        }
        for (int it = 0; it < iters; ++it) {
            if (it + NST - 1 < iters) load(it + NST - 1, at);
            cp_commit();
            at = row_of(mine + (it + NST) * 64);  // for the next step's load
            cp_wait<NST - 1>();
            if (RW == 1) __syncwarp();
            else __syncthreads();
#pragma unroll 1
            for (int w = RW == 1 ? warp : 0; w < (RW == 1 ? warp + 1 : kMmWarps); ++w) {
                const int tb = t0 + it * 64 + w * kMmTok;
                if (tb >= t1) break;
                const uint32_t ks = ring + (uint32_t)((w * NST + it % NST) * SB), vs = ks + SB / 2;
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                {
                    const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t kf[4];
                        ldsm4(ks + mm_off<D>(row, 2 * k + half), kf);
                        mma16816<T>(s[0], qf[k], kf[0], kf[1]);
                        mma16816<T>(s[1], qf[k], kf[2], kf[3]);
                    }
                }
                // scores in the log2 domain, the row's maximum over the 4 lanes that share it
                float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int x = e >> 1, tok = tb + n * 8 + (lane & 3) * 2 + (e & 1);
                        s[n][e] = tok < see[x] ? s[n][e] * k1 : -INFINITY;
                        mt[x] = fmaxf(mt[x], s[n][e]);
                    }
                bool grow = false;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 1));
                    mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 2));
                    grow = grow || mt[x] > m[x] + kMmRescale;
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float mn = fmaxf(m[x], mt[x]), f = ex2(m[x] - mn);
                        m[x] = mn;
                        l[x] *= f;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            o[j][2 * x] *= f;
                            o[j][2 * x + 1] *= f;
                        }
                    }
                }
                uint32_t pf[4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float p0 = ex2(s[n][2 * x] - m[x]), p1 = ex2(s[n][2 * x + 1] - m[x]);
                        l[x] += p0 + p1;
                        pf[2 * n + x] = pack2<T>(p0, p1);
                    }
                {
                    const int row = lane & 15, half = lane >> 4;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t vf[4];
                        ldsm4t(vs + mm_off<D>(row, 2 * j + half), vf);
                        mma16816<T>(o[2 * j], pf, vf[0], vf[1]);
                        mma16816<T>(o[2 * j + 1], pf, vf[2], vf[3]);
                    }
                }
            }
            if (RW == 1) __syncwarp();
            else __syncthreads();
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        }
        const size_t base = (size_t)(OWN ? D_.np + sp : sp) * D_.rows;
        if (RW > 1) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!live[x]) continue;
                const size_t row = (base + tokr[x]) * D_.Hq + hr[x];
                if ((lane & 3) == 0) A.part_ml[row] = make_float2(m[x], l[x]);
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2 *>(A.part_o + row * D + 8 * j + (lane & 3) * 2) =
                        make_float2(o[j][2 * x], o[j][2 * x + 1]);
            }
            __syncthreads();
        } else {
            // join the 4 warps: O_w scaled to the common maximum, summed in warp order
            cp_wait<0>();
            if ((lane & 3) == 0) {
                sml[warp][lane >> 2] = make_float2(m[0], l[0]);
                sml[warp][(lane >> 2) + 8] = make_float2(m[1], l[1]);
            }
            __syncthreads();
            float *om = reinterpret_cast<float *>(smem);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = (lane >> 2) + 8 * x;
                float M = sml[0][row].x;
#pragma unroll
                for (int w = 1; w < kMmWarps; ++w) M = fmaxf(M, sml[w][row].x);
                const float f = ex2(m[x] - M);
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2 *>(om + (warp * 16 + row) * D + 8 * j +
                                                (lane & 3) * 2) =
                        make_float2(o[j][2 * x] * f, o[j][2 * x + 1] * f);
            }
            __syncthreads();
            for (int e = threadIdx.x; e < 16 * D / 4; e += kMmThreads) {
                const int row = e / (D / 4), c = e % (D / 4) * 4, rr = rb * 16 + row;
                if (rr >= nrow) break;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kMmWarps; ++w) {
                    const float4 p = *reinterpret_cast<const float4 *>(om + (w * 16 + row) * D + c);
                    v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
                }
                const size_t at2 = (base + tok0 + rr / D_.g) * D_.Hq + kh * D_.g + rr % D_.g;
                *reinterpret_cast<float4 *>(A.part_o + at2 * D + c) = v;
                if (c == 0) {
                    float M = sml[0][row].x, L = 0.f;
                    for (int w = 1; w < kMmWarps; ++w) M = fmaxf(M, sml[w][row].x);
                    for (int w = 0; w < kMmWarps; ++w) L += sml[w][row].y * ex2(sml[w][row].x - M);
                    A.part_ml[at2] = make_float2(M, L);
                }
            }
            __syncthreads();
        }
    }
}

template <typename T, int D, int RW, bool OWN>
cudaError_t go(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    const long long rows = (OWN ? (long long)D_.max_new : D_.group_rows()) * D_.g;
    const long long nblk = (rows + 16 * RW - 1) / (16 * RW);
    const long long ctas = (long long)(OWN ? D_.R : D_.S) * D_.Hkv * nblk * (OWN ? D_.ns : D_.np);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = pg_attn_mma_kernel<T, D, RW, OWN>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         mm_smem<D>());
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)ctas, kMmThreads, mm_smem<D>(), st>>>(D_, A, (int)nblk);
    return cudaGetLastError();
}

template <typename T, int D, bool OWN>
cudaError_t rows_rule(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    const long long rows = (OWN ? (long long)D_.max_new : D_.group_rows()) * D_.g;
    return rows > 16 ? go<T, D, 4, OWN>(D_, A, st) : go<T, D, 1, OWN>(D_, A, st);
}

template <typename T, bool OWN>
cudaError_t by_head(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.d == 128 ? rows_rule<T, 128, OWN>(D, A, st)
                      : (D.d == 64 ? rows_rule<T, 64, OWN>(D, A, st)
                                   : rows_rule<T, 32, OWN>(D, A, st));
}

}  // namespace

cudaError_t launch_pg_own_mma(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_head<__nv_bfloat16, true>(D, A, st)
                               : by_head<__half, true>(D, A, st);
}

cudaError_t launch_pg_prompt_mma(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_head<__nv_bfloat16, false>(D, A, st)
                               : by_head<__half, false>(D, A, st);
}

}  // namespace kve
