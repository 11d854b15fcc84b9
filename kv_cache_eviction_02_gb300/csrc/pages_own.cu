// Shared-prompt decoding, 16-bit types: attention of the requests' own rows, and over short prompts, with
// warp-level matrix products.
//
// Own rows are read by g query heads of one or a few new rows, so a request and KV head have 1 to a
// few dozen query rows over its K/V: bound by HBM, with 2 g flops per byte at one new row. The products
// run transposed, S^T = K Q^T and O^T += V^T P^T, as m16n8k16 fragments in registers: 16 tokens (or 16
// output columns) on the wide side and 8 query rows on the narrow one, which fits a decode step's 4 to
// 8 query heads where a 128-row tcgen05 tile would be almost empty. The weights go from the accumulator
// of S^T to the B operand of V^T P^T by an 8 x 8 transpose in registers.
//
// Work is dealt to warps, not blocks. A unit is (request or prompt, KV head, block of 8 or 16 query rows), a
// chunk 16 of its tokens; the chunks of all units stand in one line (request, then KV head, then row block)
// and every warp takes the same number of consecutive ones, however the lengths lie. A warp's ring of
// chunks (TMA boxes of the pages, swizzled for ldmatrix) runs on across the units it passes, so HBM sees
// no pause at a unit's end, and no warp waits for another. Each piece of a unit that a warp has seen
// becomes one partial result at place (unit index + warp index), which no other piece has; the join finds
// a unit's pieces from the same arithmetic, in order.
//
// 256 requests of up to 1024 own rows (8 KV heads of d 128, 542 MB): 91 us, 6.0 TB/s of DRAM, 0.88 of what a
// copy reaches. A warp has a chunk done every 4100 cycles, of which it waits 2400 for memory: 1824 warps with
// one or two chunks of 8 KB on their way each (two blocks per SM of three stages: 102 us, 5.4 TB/s).
#include <cudaTypedefs.h>

#include <type_traits>

#include "pages_ptx.cuh"

namespace kve {
namespace {

constexpr int kMmThreads = 32 * kPgOwnWarps, kMmTok = kPgChunk;  // tokens per chunk

// Three blocks per SM for units of 8 query rows (d_head 128: two stages; 256 requests behind 8K rows 137 us
// with two blocks of three stages, 130 so), two for 16, whose fragments take the registers.
template <int D, int NT> constexpr int mm_stages() { return D == 128 ? (NT == 1 ? 2 : 3) : 4; }
// A row takes at least 128 bytes: a box must start on a multiple of them, and one of page size 1 is a
// single row. With d_head 32 the boxes reach behind the rows, where TMA fills in zeros.
template <int D> constexpr int mm_row_bytes() { return D == 32 ? 128 : D * 2; }
template <int D> constexpr int mm_stage_bytes() { return kMmTok * mm_row_bytes<D>() * 2; }  // K and V
template <int D, int NT> constexpr int mm_smem() {
    return kPgOwnWarps * mm_stages<D, NT>() * mm_stage_bytes<D>() + 1024;
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
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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
// Two weights as a 16-bit pair. A weight is at most 2^8 (fp16: 2^15; see kPgRescale) and rounds to half a step
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

// Where TMA puts 16-byte word c of a chunk's row: column blocks of 64 values one after the other, in
// each 128-byte rows swizzled so that 8 rows of a word fall into different banks.
__device__ __forceinline__ uint32_t mm_off(int row, int c) {
    return (uint32_t)((c >> 3) * (kMmTok * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// NT: blocks of 8 query rows per unit. RB = 8 NT is the unit's rows. MODE: what a warp takes, its share of the
// requests' units, of the prompts' and the requests', or all of one request and KV head.
enum { kOwn, kLine, kDirect };
template <typename T, int D, int NT, int MODE>
__global__ void __launch_bounds__(kMmThreads, NT == 1 ? 3 : 2)
    pg_own_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                  PgDims D_, PgAttn A, PgOwn W) {
    constexpr int NST = mm_stages<D, NT>(), SB = mm_stage_bytes<D>(), RB = 8 * NT;
    constexpr bool LINE = MODE == kLine, DIRECT = MODE == kDirect;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ long long csum[kMmThreads + 1];  // chunks before each thread's requests
    __shared__ int usum[kMmThreads + 1];        // units before them
    __shared__ uint64_t bars[kPgOwnWarps][NST];
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane < NST) tc::mbar_init(&bars[warp][lane], 1);
    if (threadIdx.x == 0) {
        s_abort = 0;
        tc::tma_prefetch_desc(&tm_k);
        tc::tma_prefetch_desc(&tm_v);
        if (MODE != kOwn) {
            tc::tma_prefetch_desc(&tm_kp);
            tc::tma_prefetch_desc(&tm_vp);
        }
    }
    tc::mbar_fence_init();
    if (D_.np == 0) pg_wait_prior();  // first kernel of its call (else the prompt's has waited)
    pg_launch_dependents();

    const int w = blockIdx.x * kPgOwnWarps + warp;
    int n = 0, unit = 0;  // chunks of this warp; the index of its first unit
    PgCursor<false> cc;
    int prompt = 0, plen = 0, pchunks = 0;  // kDirect: chunks c < pchunks are the prompt's
    if constexpr (DIRECT) {
        __syncthreads();  // the barriers and s_abort are set
        cc.rows = cc.rb = 0;
        const int blocks = pg_direct_blocks(D_), u = w / blocks;
        if (u < D_.R * D_.Hkv) {
            const int r = u / D_.Hkv;
            cc.enter(D_, A, D_.S + r);
            cc.kh = u - r * D_.Hkv;
            cc.rb = w - u * blocks;
            prompt = r / D_.F;
            plen = A.plen ? pg_clamp(__ldg(A.plen + prompt), 0, D_.n) : D_.n;
            pchunks = (plen + kMmTok - 1) / kMmTok;
            n = pchunks + cc.cr;
        }
    } else {
        const PgShare sh = pg_share<kMmThreads>(
            D_.R + (LINE ? D_.S : 0), D_.Hkv, csum, usum, W, [&](int e, int *cr, int *nb) {
                int len, first, nq, rows;
                pg_unit_entity<false>(D_, A, e + (LINE ? 0 : D_.S), &len, &first, &nq, &rows, cr, nb);
            });
        const long long X0 = w * sh.cpw;
        n = (int)min(sh.total - X0, sh.cpw);
        if (n > 0) {
            long long x;
            int e;
            pg_share_find<kMmThreads>(csum, usum, sh, X0, &e, &x, &unit);
            cc.enter(D_, A, e + (LINE ? 0 : D_.S));
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
    }
    if (DIRECT ? cc.rb * RB < cc.rows : n > 0) {
        PgCursor<false> ca = cc;  // runs ahead: the addresses of the chunks to load

        uint8_t *ring = smem + warp * NST * SB;
        uint64_t *bar = bars[warp];
        volatile int *abort_flag = &s_abort;
        // (rsqrtf is off by 2 units in the last place at most, ex2.approx below by 2^-22 of the weight: far below
        // the weights' rounding to 16 bits)
        const float k1 = kLog2e * rsqrtf((float)D);
        uint32_t qf[NT][D / 16][2];  // B operand of S^T: query row lane / 4 of each block
        float o[NT][D / 16][4], m[NT][2], l[NT][2];  // this lane's query rows 2 (lane % 4), + 1
        int see[NT][2], rows, row0;  // tokens they see; query rows of the entity, the unit's first
        auto begin = [&]() {         // of a unit, or of this warp's part of one
            rows = cc.rows;
            row0 = cc.rb * RB;
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                const int rr = row0 + 8 * b + (lane >> 2), t = rr < rows ? rr / D_.g : 0;
                const T *qp = static_cast<const T *>(A.q) + (cc.first + t) * A.q_row +
                              (size_t)(cc.kh * D_.g + (rr < rows ? rr - t * D_.g : 0)) * D +
                              (lane & 3) * 2;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qf[b][k][0] =
                        rr < rows ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * k)) : 0u;
                    qf[b][k][1] =
                        rr < rows ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * k + 8)) : 0u;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int qr = row0 + 8 * b + (lane & 3) * 2 + e;
                    see[b][e] = qr >= rows ? 0
                                           : (LINE && cc.e < D_.S ? cc.len : cc.len - cc.nq + 1 + qr / D_.g);
                    m[b][e] = kPgNoMax;
                    l[b][e] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[b][j][e] = 0.f;
            }
        };
        // A chunk is 16 / box boxes of box = min(page, 16) rows, one per lane. Where a chunk's pages lie
        // is asked two chunks before they are loaded: the answer of the table (a trip to L2) is not
        // waited for. at: the box's row within its page and head, -1 behind the request's last page; a
        // prompt's chunk is one box (one of each column block): its prompt, its first token and its head.
        const int lgB = D_.lgP < 4 ? D_.lgP : 4, boxes = kMmTok >> lgB;
        const int page_rows = D_.Hkv << D_.lgP;
        const uint32_t box_bytes = (uint32_t)(mm_row_bytes<D>() * 2) << lgB;
        // a box of 16 rows brings all column blocks, [block][row][64 values]; smaller ones one block
        const int zs = lgB < 4 && D > 64 ? D / 64 : 1;
        struct Where {
            int page, at, head;  // head: -1 for pages
        };
        auto where = [&]() -> Where {
            if (LINE && ca.e < D_.S) return Where{ca.e, ca.c * kMmTok, ca.kh};
            if (DIRECT && ca.c < pchunks) return Where{prompt, ca.c * kMmTok, ca.kh};
            const int j = (ca.c - pchunks) * kMmTok + (lane << lgB);
            if (lane >= boxes || j >= ca.len) return Where{0, -1, -1};
            return Where{__ldg(A.table + (size_t)(ca.e - D_.S) * D_.maxp + (j >> D_.lgP)),
                         (ca.kh << D_.lgP) + (j & (D_.P - 1)), -1};
        };
        auto load = [&](int place, Where x) {
            if (MODE != kOwn && x.head >= 0) {
                if (tc::elect_one()) {
                    uint8_t *k = ring + place * SB;
                    tc::mbar_expect_tx(&bar[place], SB);
                    for (int z = 0; z < (D == 128 ? 2 : 1); ++z) {
                        tc::tma_load_4d(k + z * (kMmTok * 128), &tm_kp, 64 * z, x.at, x.head, x.page,
                                    &bar[place]);
                        tc::tma_load_4d(k + SB / 2 + z * (kMmTok * 128), &tm_vp, 64 * z, x.at, x.head, x.page,
                                    &bar[place]);
                    }
                }
                __syncwarp();
                return;
            }
            int row = -1;
            if (x.at >= 0) row = pg_page_id(x.page, D_.npages, A.err) * page_rows + x.at;
            const int used = __popc(__ballot_sync(0xffffffffu, row >= 0));
            uint8_t *k = ring + place * SB;
            if (tc::elect_one()) tc::mbar_expect_tx(&bar[place], used * box_bytes);
            for (int b = 0; b < used; ++b) {  // one lane issues: TMA takes uniform operands
                const int y = __shfl_sync(0xffffffffu, row, b);
                if (tc::elect_one()) {
                    for (int z = 0; z < zs; ++z) {
                        tc::tma_load_3d(k + z * (kMmTok * 128), &tm_k, 0, y, z, &bar[place]);
                        tc::tma_load_3d(k + SB / 2 + z * (kMmTok * 128), &tm_v, 0, y, z, &bar[place]);
                    }
                }
                k += 128 << lgB;
            }
        };
        int asked = 1, ahead = 0;  // chunks asked for, chunks issued
        Where x0 = where(), x1{0, -1, -1};
        begin();  // its loads of Q run beside the table's
        auto ask = [&]() {
            if (asked < n) {
                if (DIRECT) ++ca.c;
                else ca.next(D_, A);
                x1 = where();
                ++asked;
            }
        };
        ask();
#pragma unroll 1
        for (int i = 0; i < NST - 1 && ahead < n; ++i) {
            load(ahead++, x0);
            x0 = x1;
            ask();
        }

        int slot = 0, fill = NST - 1;  // ring places of this chunk and of the one to issue
        uint32_t phase = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (ahead < n) {
                load(fill, x0);
                ++ahead;
                x0 = x1;
                ask();
            }
            if (++fill == NST) fill = 0;
            if (!DIRECT && i > 0 && cc.c == 0) begin();
            if (!tc::mbar_wait_warp(&bar[slot], phase, abort_flag, A.err)) break;
            const bool pre = DIRECT && cc.c < pchunks;  // a chunk of the prompt, which all rows see
            const int tb = (cc.c - (pre ? 0 : pchunks)) * kMmTok, len = pre ? plen : cc.len;
            const uint32_t ks = tc::smem_u32(ring + slot * SB), vs = ks + SB / 2;
            if (tb + kMmTok > len) {
                // V rows behind the last token hold anything (their weights are 0): zeros instead
                for (int e = (len - tb) * (D / 8) + lane; e < kMmTok * (D / 8); e += 32)
                    *reinterpret_cast<uint4 *>(ring + slot * SB + SB / 2 +
                                               mm_off(e / (D / 8), e % (D / 8))) =
                        make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();  // before TMA writes there again
                __syncwarp();
            }
            if (++slot == NST) {
                slot = 0;
                phase ^= 1;
            }
            // S^T: 16 tokens x 8 query rows per block
            float s[NT][4];
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[b][e] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t kf[4];
                ldsm4(ks + mm_off(lane & 15, 2 * k + (lane >> 4)), kf);
#pragma unroll
                for (int b = 0; b < NT; ++b) mma16816<T>(s[b], kf, qf[b][k][0], qf[b][k][1]);
            }
            uint32_t pf[NT][2];
            const int tok = tb + (lane >> 2);
            constexpr float UP = std::is_same<T, __half>::value ? kPgHalfUp : 0.f;
            bool grow = false;
            float mt[NT][2];
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // scores in the log2 domain, maximum over the tokens
                    const int end = pre ? plen : see[b][e];
                    s[b][e] = tok < end ? s[b][e] * k1 : -INFINITY;
                    s[b][e + 2] = tok + 8 < end ? s[b][e + 2] * k1 : -INFINITY;
                    float x = fmaxf(s[b][e], s[b][e + 2]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    mt[b][e] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    grow = grow || mt[b][e] > m[b][e] + (kPgRescale + UP);
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mn = fmaxf(m[b][e], mt[b][e] - UP), f = tc::ex2_approx(m[b][e] - mn);
                        m[b][e] = mn;
                        l[b][e] *= f;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            o[b][j][e] *= f;
                            o[b][j][e + 2] *= f;
                        }
                    }
            }
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int x = 0; x < 2; ++x) {  // tokens 0-7, 8-15
                    const float p0 = tc::ex2_approx(s[b][2 * x] - m[b][0]);
                    const float p1 = tc::ex2_approx(s[b][2 * x + 1] - m[b][1]);
                    l[b][0] += p0;
                    l[b][1] += p1;
                    pf[b][x] = transpose8(pack2<T>(p0, p1));
                }
            // O^T: 16 output columns x 8 query rows per block
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t vf[4];
                ldsm4t(vs + mm_off((lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1)), vf);
#pragma unroll
                for (int b = 0; b < NT; ++b) mma16816<T>(o[b][j], vf, pf[b][0], pf[b][1]);
            }
            if (!DIRECT && (i == n - 1 || cc.c == cc.cr - 1)) {  // the piece ends
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
                        if (row0 + qr >= rows || (unsigned long long)seg >= W.segs) continue;
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
            if (DIRECT) ++cc.c;
            else if (i + 1 < n) cc.next(D_, A);
            __syncwarp();  // the chunk's readers are done: the next issue may overwrite it
        }
        if (DIRECT && !s_abort) {
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[b][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    const int qr = row0 + 8 * b + (lane & 3) * 2 + e, t = qr / D_.g, tok = cc.first + t;
                    if (qr >= rows || __ldg(A.row_req + tok) != cc.e - D_.S) continue;
                    const float inv = x > 0.f ? 1.f / x : 0.f;
                    const long long row = (long long)tok * D_.Hq + cc.kh * D_.g + (qr - t * D_.g);
                    T *dst = static_cast<T *>(A.out) + row * D + (lane >> 2);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        dst[16 * j] = from_f<T>(o[b][j][e] * inv);
                        dst[16 * j + 8] = from_f<T>(o[b][j][e + 2] * inv);
                    }
                    if (A.lse && lane < 4) A.lse[row] = x == 0.f ? -INFINITY : (m[b][e] + log2f(x)) * kLn2;
                }
        }
        if (s_abort) {  // copies still in flight land before the block ends
            for (int k = 0; k < NST; ++k) {
                tc::mbar_drain(&bar[k], 0);
                tc::mbar_drain(&bar[k], 1);
            }
        }
    }
    pg_end_after_prior();
}

template <typename T, int D, int NT, int MODE>
cudaError_t go(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    const bool f16 = std::is_same<T, __half>::value;
    CUtensorMap tk, tv;
    // {64 columns, rows of the pool, column blocks}
    constexpr int blocks = D == 128 ? 2 : 1;
    const bool whole = D_.P >= kMmTok;
    const cuuint64_t dims[3] = {D == 32 ? 32 : 64, (cuuint64_t)D_.npages * D_.Hkv * D_.P, blocks};
    const long long stride[2] = {D, 64};
    const cuuint32_t box[3] = {64, (cuuint32_t)(whole ? kMmTok : D_.P), whole ? blocks : 1};
    if (!pg_tmap(&tk, f16, A.K, 3, dims, stride, box) ||
        !pg_tmap(&tv, f16, A.V, 3, dims, stride, box))
        return cudaErrorInvalidValue;
    CUtensorMap pk = tk, pv = tv;
    if (MODE != kOwn && D_.n > 0) {
        const cuuint64_t pd[4] = {D, (cuuint64_t)D_.n, (cuuint64_t)D_.Hkv, (cuuint64_t)D_.S};
        const long long ps[3] = {A.p_tok, A.p_head, A.p_prompt};
        const cuuint32_t pb[4] = {64, kMmTok, 1, 1};
        if (!pg_tmap(&pk, f16, A.Kp, 4, pd, ps, pb) || !pg_tmap(&pv, f16, A.Vp, 4, pd, ps, pb))
            return cudaErrorInvalidValue;
    }
    return pg_launch(pg_own_kernel<T, D, NT, MODE>, pg_own_ctas(D_), kMmThreads, mm_smem<D, NT>(), true, st, tk,
                     tv, pk, pv, D_, A, A.own);
}

template <typename T, int D> cudaError_t by_rows(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    const bool one = pg_unit_rows(D_) == 8;
    if (D_.direct) return one ? go<T, D, 1, kDirect>(D_, A, st) : go<T, D, 2, kDirect>(D_, A, st);
    if (D_.line) return one ? go<T, D, 1, kLine>(D_, A, st) : go<T, D, 2, kLine>(D_, A, st);
    return one ? go<T, D, 1, kOwn>(D_, A, st) : go<T, D, 2, kOwn>(D_, A, st);
}

template <typename T> cudaError_t by_head(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.d == 128 ? by_rows<T, 128>(D, A, st)
                      : (D.d == 64 ? by_rows<T, 64>(D, A, st) : by_rows<T, 32>(D, A, st));
}

}  // namespace

cudaError_t launch_pg_own16(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_head<__nv_bfloat16>(D, A, st) : by_head<__half>(D, A, st);
}

}  // namespace kve
