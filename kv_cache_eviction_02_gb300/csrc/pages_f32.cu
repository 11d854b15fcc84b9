// Shared-prompt decoding, fp32: attention over the prompts and the requests' own rows on the CUDA cores,
// in one launch.
//
// The work of all prompts and all requests stands in one line: entities (the prompts, then the
// requests), of each its units (KV head, block of 16 query rows), of each its chunks of 8 tokens; every
// warp takes the same number of consecutive chunks and leaves one partial result per unit it has seen a
// piece of, at place (unit index + warp index). (pages_own.cu deals out the own rows of 16-bit types in
// the same way.)
//
// Within a warp a lane owns D/32 columns of K, V, Q and O, so a token's row is one shared-memory read
// without bank conflicts and Q and O stay in registers. For 4 query rows and 8 tokens the lanes' 32
// partial dot products are summed by recursive halving (31 exchanges in all), which leaves the score of
// (row, token) in lane 8 row + token; weights go back to all lanes through 512 bytes of shared memory.
// Sums of d products in a tree of 32, everything fp32; the factor log2 e / sqrt d is carried as two
// floats, since its rounding would shift every score the same way. Bound by HBM up to 8 query rows per
// KV head, by FFMA issue at 16.
#include "pages.cuh"

namespace kve {
namespace {

constexpr int kF3Threads = 32 * kPgOwnWarps, kF3Tok = kPgF32Chunk, kF3Rows = kPgF32Rows;

template <int D> constexpr int f3_stages() { return D == 128 ? 3 : 6; }
template <int D> constexpr int f3_stage_floats() { return 2 * kF3Tok * D; }  // K and V
template <int D> constexpr int f3_smem() {
    return kPgOwnWarps * (f3_stages<D>() * f3_stage_floats<D>() + kF3Tok * kF3Rows) * 4;
}
constexpr float kF3Rescale = 8.f;  // O is rescaled when a row's maximum grew by more than 2^8

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

template <int E> struct Cols { float v[E]; };
template <int E> __device__ __forceinline__ Cols<E> cols(const float *p) {
    Cols<E> c;
    if (E == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        c.v[0] = x.x;
        c.v[1 % E] = x.y;
        c.v[2 % E] = x.z;
        c.v[3 % E] = x.w;
    } else if (E == 2) {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        c.v[0] = x.x;
        c.v[1 % E] = x.y;
    } else {
        c.v[0] = *p;
    }
    return c;
}

// Sums 32 values over the 32 lanes: lane L is left with the sum of value L.
__device__ __forceinline__ float halve(float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
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
__global__ void __launch_bounds__(kF3Threads, 2) pg_f32_kernel(PgDims D_, PgAttn A, PgOwn W) {
    constexpr int NST = f3_stages<D>(), SF = f3_stage_floats<D>(), E = D / 32, NG = kF3Rows / 4;
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
    const int w = blockIdx.x * kPgOwnWarps + warp;
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

    float *ring = sm + warp * (NST * SF + kF3Tok * kF3Rows), *ps = ring + NST * SF;
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    // lane t (mod 8) looks after token t of a chunk: where it lies is asked two chunks before it is
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
        const uint32_t dst = ring_s + (uint32_t)(place * SF * 4 + lane * 16);
#pragma unroll
        for (int i = 0; i < kF3Tok / RPI; ++i) {
            const long long r = __shfl_sync(0xffffffffu, o, i * RPI + lane / WPR);
            const long long at = (r < 0 ? 0 : r) + (lane % WPR) * 4;
            cp16(dst + i * 512, Kb + at, r >= 0);
            cp16(dst + i * 512 + kF3Tok * D * 4, Vb + at, r >= 0);
        }
    };
    float q[kF3Rows][E], o[kF3Rows][E];  // this lane's columns of the unit's 16 rows
    float m[NG], l[NG];                  // of row lane / 8 of each group of 4
    int see[NG], live;                   // tokens the row sees; the unit's rows
    auto begin = [&]() {                 // of a unit, or of this warp's part of one
        const int row0 = cc.rb * kF3Rows;
        live = min(kF3Rows, cc.rows - row0);
#pragma unroll
        for (int r = 0; r < kF3Rows; ++r) {
#pragma unroll
            for (int x = 0; x < E; ++x) q[r][x] = o[r][x] = 0.f;
            if (r < live) {
                const int t = (row0 + r) / D_.g, h = cc.kh * D_.g + row0 + r - t * D_.g;
                const Cols<E> c = cols<E>(static_cast<const float *>(A.q) +
                                          (cc.first + t) * A.q_row + (size_t)h * D + lane * E);
#pragma unroll
                for (int x = 0; x < E; ++x) q[r][x] = c.v[x];
            }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int r = row0 + g * 4 + (lane >> 3);
            see[g] = cc.e < D_.S ? cc.len : cc.len - cc.nq + 1 + r / D_.g;
            if (r >= cc.rows) see[g] = 0;
            m[g] = kPgNoMax;
            l[g] = 0.f;
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
        const float *ks = ring + slot * SF + lane * E, *vs = ks + kF3Tok * D;
        if (++slot == NST) slot = 0;
        const int tok = cc.c * kF3Tok + (lane & 7);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g * 4 >= live) break;
            float part[32];
#pragma unroll
            for (int t = 0; t < kF3Tok; ++t) {
                const Cols<E> k = cols<E>(ks + t * D);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float a = q[g * 4 + r][0] * k.v[0];
#pragma unroll
                    for (int x = 1; x < E; ++x) a = fmaf(q[g * 4 + r][x], k.v[x], a);
                    part[r * 8 + t] = a;
                }
            }
            const float dot = halve(part);  // (by all lanes)
            const float s = tok < see[g] ? dot : -INFINITY;
            float smax = s;
#pragma unroll
            for (int x = 1; x < 8; x <<= 1)
                smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, x));
            const float mt = fmaf(smax, k_hi, smax * k_lo);
            const bool grow = mt > m[g] + kF3Rescale;
            if (__any_sync(0xffffffffu, grow)) {
                const float mn = fmaxf(m[g], mt), f = exp2f(m[g] - mn);
                m[g] = mn;
                l[g] *= f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float fr = __shfl_sync(0xffffffffu, f, r * 8);
#pragma unroll
                    for (int x = 0; x < E; ++x) o[g * 4 + r][x] *= fr;
                }
            }
            // s log2 e / sqrt d - m with one rounding near the result
            const float p = s == -INFINITY ? 0.f : exp2f(fmaf(s, k_hi, fmaf(s, k_lo, -m[g])));
            l[g] += p;
            ps[(lane & 7) * kF3Rows + g * 4 + (lane >> 3)] = p;
        }
        __syncwarp();
#pragma unroll
        for (int t = 0; t < kF3Tok; ++t) {
            const Cols<E> v = cols<E>(vs + t * D);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g * 4 >= live) break;
                const float4 p = *reinterpret_cast<const float4 *>(ps + t * kF3Rows + g * 4);
                const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int x = 0; x < E; ++x) o[g * 4 + r][x] = fmaf(pr[r], v.v[x], o[g * 4 + r][x]);
            }
        }
        if (i == n - 1 || cc.c == cc.cr - 1) {  // the piece ends
            const long long seg = (long long)unit + w;
            // (row starts that are no sums of lengths can ask for more places than there are)
            if (seg < W.segs) {
                const size_t at = (size_t)seg * W.seg_rows;
#pragma unroll
                for (int r = 0; r < kF3Rows; ++r)
                    if (r < live) {
                        float *dst = W.o + (at + r) * D + lane * E;
#pragma unroll
                        for (int x = 0; x < E; ++x) dst[x] = o[r][x];
                    }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float x = l[g];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    const int r = g * 4 + (lane >> 3);
                    if ((lane & 7) == 0 && r < live) W.ml[at + r] = make_float2(m[g], x);
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
