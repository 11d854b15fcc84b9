// Shared-prompt decoding on the CUDA cores: the page planner, the paged append, the attention of
// fp32 inputs and the kernel that joins the partial results of an attention call.
#include "pages.cuh"

namespace kve {

// Splits of the prompt and of the requests' own rows.
//   Prompt on tcgen05: one CTA per SM, so the split count that minimises
//     ceil(items * splits / 152) * (tiles per split + 4): a CTA's set-up and the partial result that
//     it writes and the join reads cost about four tiles.
//   Elsewhere: enough CTAs to fill the GPU a few times, at least 128 tokens each.
// Own rows are split by the table's width, since lengths are known on the device only; the CTAs of
// splits that a request does not reach return at once.
static void pg_split(PgDims *D) {
    auto split = [](long long items, long long n, long long ctas, long long least, int *count,
                    int *len) {
        long long want = (ctas + items - 1) / items;
        const long long most = (n + least - 1) / least;
        if (want > most) want = most;
        if (want > 64) want = 64;
        if (want < 1) want = 1;
        const long long per = ((n + want - 1) / want + 127) / 128 * 128;
        *len = (int)per;
        *count = (int)((n + per - 1) / per);
    };
    const long long prow = D->group_rows() * D->g, orow = (long long)D->max_new * D->g;
    D->np = 0;
    D->psplit = 128;
    if (D->n > 0 && pg_prompt_tc(*D)) {
        const long long per = (long long)pg_tile_rows(*D) * pg_prompt_pairs(*D);
        const long long items = (long long)D->S * D->Hkv * ((D->group_rows() + per - 1) / per);
        const long long tiles = (D->n + 127LL) / 128;
        long long best = -1, len = 1;
        for (long long p = 1; p <= 64 && p <= tiles; ++p) {
            const long long waves = (items * p + 151) / 152, t = (tiles + p - 1) / p;
            const long long cost = waves * (t + 4);
            if (best < 0 || cost < best) {
                best = cost;
                len = t;
            }
        }
        D->psplit = (int)(len * 128);
        D->np = (int)((tiles + len - 1) / len);
    } else if (D->n > 0) {
        split((long long)D->S * D->Hkv * ((prow + 15) / 16), D->n, 152 * 8, 128, &D->np,
              &D->psplit);
    }
    split((long long)D->R * D->Hkv * ((orow + 15) / 16), D->cap(), 152 * 8, 256, &D->ns,
          &D->ssplit);
}

// ---- sizes ---------------------------------------------------------------------------------------
bool pg_dims(const KvePgShape *sh, PgDims *D, const char **why) {
    constexpr long long kMax30 = 1LL << 30, kMax31 = 1LL << 31;
    *why = nullptr;
    if (!sh) return (*why = "null shape"), false;
    if (sh->n_prompts < 1 || sh->fan < 1 || sh->n_q_heads < 1 || sh->n_kv_heads < 1 ||
        sh->n_prefix < 0 || sh->n_pages < 1 || sh->max_pages < 1 || sh->n_rows < 1 ||
        sh->max_new < 1)
        return (*why = "sizes must be positive (n_prefix may be 0)"), false;
    if (sh->dtype != KVE_F32 && sh->dtype != KVE_BF16 && sh->dtype != KVE_F16)
        return (*why = "dtype must be KVE_F32, KVE_BF16 or KVE_F16"), false;
    if (sh->n_q_heads % sh->n_kv_heads != 0 || sh->n_q_heads / sh->n_kv_heads > 128)
        return (*why = "n_q_heads must be a multiple of n_kv_heads, at most 128 times it"), false;
    if (sh->d_head != 32 && sh->d_head != 64 && sh->d_head != 128)
        return (*why = "d_head must be 32, 64 or 128"), false;
    if (sh->page_size < 1 || sh->page_size > 256 || (sh->page_size & (sh->page_size - 1)))
        return (*why = "page_size must be a power of two, 1 to 256"), false;
    if ((long long)sh->n_prompts * sh->fan > 16384)
        return (*why = "n_prompts * fan must be at most 16384"), false;
    if (sh->n_rows > kMax30 || sh->n_prefix > kMax30 ||
        (long long)sh->n_pages * sh->page_size > kMax30 ||
        (long long)sh->max_pages * sh->page_size > kMax30)
        return (*why = "n_rows, n_prefix, n_pages * page_size and max_pages * page_size must be "
                       "at most 2^30"),
               false;
    if ((long long)sh->n_rows * sh->n_q_heads >= kMax31 ||
        (long long)sh->n_pages * sh->page_size * sh->n_kv_heads >= kMax31)
        return (*why = "n_rows * n_q_heads and n_pages * n_kv_heads * page_size must be below 2^31"),
               false;
    if ((long long)sh->n_prompts * sh->n_kv_heads > 65535)
        return (*why = "n_prompts * n_kv_heads must be at most 65535"), false;
    D->S = sh->n_prompts;
    D->F = sh->fan;
    D->R = D->S * D->F;
    D->Hq = sh->n_q_heads;
    D->Hkv = sh->n_kv_heads;
    D->g = D->Hq / D->Hkv;
    D->d = sh->d_head;
    D->n = sh->n_prefix;
    D->P = sh->page_size;
    D->lgP = 0;
    while ((1 << D->lgP) < D->P) ++D->lgP;
    D->npages = sh->n_pages;
    D->maxp = sh->max_pages;
    D->rows = sh->n_rows;
    D->max_new = sh->max_new < sh->n_rows ? sh->max_new : sh->n_rows;
    D->dtype = sh->dtype;
    pg_split(D);
    return true;
}

PgWorkspace pg_ws_layout(const PgDims &D) {
    PgWorkspace W{};
    const size_t rows = (size_t)D.rows * D.Hq * (D.np + D.ns);
    W.part_ml = 0;
    W.part_o = (sizeof(float2) * rows + 255) & ~size_t(255);
    W.total = (W.part_o + sizeof(float) * rows * D.d + 255) & ~size_t(255);
    return W;
}

namespace {

// ---- page planner ----------------------------------------------------------------------------------
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b, unsigned cap) {
    return min(a + b, cap);
}

// Inclusive scan over the block of two values at a time, each saturating at its cap (saturating
// addition of non-negative numbers is associative). tot: two values per warp.
__device__ __forceinline__ uint2 block_scan2(uint2 v, uint2 cap, uint2 *tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned a = __shfl_up_sync(0xffffffffu, v.x, o);
        const unsigned b = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) {
            v.x = sat_add(v.x, a, cap.x);
            v.y = sat_add(v.y, b, cap.y);
        }
    }
    if (nw == 1) return v;
    __syncthreads();  // tot may still be read from the last scan
    if (lane == 31) tot[warp] = v;
    __syncthreads();
    uint2 before = make_uint2(0, 0);
    for (int w = 0; w < warp; ++w) {
        before.x = sat_add(before.x, tot[w].x, cap.x);
        before.y = sat_add(before.y, tot[w].y, cap.y);
    }
    v.x = sat_add(v.x, before.x, cap.x);
    v.y = sat_add(v.y, before.y, cap.y);
    return v;
}

// One step of the page planner. Every CTA of the launch's one cluster scans all requests by itself
// (two scans: rows and returned pages, then wanted pages of the requests not refused so far) and
// keeps, per request, the end of its rows and its offset into the ring; the rows, 128 at a time,
// and the finished requests are then shared out over the cluster's warps. A row finds its request
// in shared memory and its page in the table (an old page) or straight in the ring (a new one), so
// nothing waits for another CTA's stores; the row that opens a new page writes it to the table.
// Lengths and the pool are written by the first CTA after a cluster barrier, when every CTA has
// read them, so both may be updated in place.
// Bound by latency: a chain of about ten dependent memory and barrier steps.
__global__ void __launch_bounds__(1024)
    pg_plan_kernel(PgPlanArgs A, int R, int lgP, int npages, int maxp, int nrows, int max_new) {
    extern __shared__ unsigned sh_plan[];
    unsigned *row_end = sh_plan;                            // [R]
    int *off = reinterpret_cast<int *>(sh_plan + R);        // [R] ring offset, -1: refused
    __shared__ uint2 tot[32];
    __shared__ unsigned carry[3];  // rows, returned pages, wanted pages of the tiles before
    __shared__ int s_refused;
    __shared__ unsigned s_taken;
    const int P = 1 << lgP;
    const int cap = maxp << lgP;
    const int n_free = pg_clamp(A.pool_in[1], 0, npages);
    const int head = (unsigned)A.pool_in[0] < (unsigned)npages ? A.pool_in[0] : 0;
    if (threadIdx.x == 0) {
        carry[0] = carry[1] = carry[2] = 0;
        s_refused = 0;
        s_taken = 0;
    }
    __syncthreads();
    const uint2 cap1 = make_uint2((unsigned)nrows + 1u, (unsigned)npages + 1u);
    const uint2 cap2 = make_uint2((unsigned)npages + 1u, 1u);
    for (int base = 0; base < R; base += blockDim.x) {
        const int r = base + threadIdx.x;
        int nw = 0, old = 0;
        if (r < R) {
            nw = A.new_len[r];
            old = A.len_in[r];
        }
        const bool bad_len = old < 0 || old > cap;
        const int have = bad_len ? 0 : (old + P - 1) >> lgP;
        const unsigned add = nw > 0 ? min((unsigned)nw, cap1.x) : 0u;
        const unsigned freed = nw < 0 ? (unsigned)have : 0u;
        const unsigned c0 = carry[0], c1 = carry[1], c2 = carry[2];
        uint2 s = block_scan2(make_uint2(add, freed), cap1, tot);
        s.x = sat_add(s.x, c0, cap1.x);
        s.y = sat_add(s.y, c1, cap1.y);
        bool bad = nw != 0 && bad_len;
        unsigned want = 0;
        if (nw > 0) {
            bad = bad || nw > max_new || s.x > (unsigned)nrows || (long long)old + nw > cap;
            if (!bad) want = (unsigned)(((old + nw + P - 1) >> lgP) - have);
        }
        uint2 w = block_scan2(make_uint2(want, 0), cap2, tot);
        w.x = sat_add(w.x, c2, cap2.x);
        if (want > 0 && w.x > (unsigned)n_free) bad = true;
        if (r < R) {
            row_end[r] = s.x;
            off[r] = bad ? -1 : (int)(nw < 0 ? s.y - freed : w.x - want);
            if (bad) atomicAdd(&s_refused, 1);
            if (!bad && want > 0) atomicMax(&s_taken, w.x);
        }
        __syncthreads();  // every thread has read the carries
        if (threadIdx.x == blockDim.x - 1) {
            carry[0] = s.x;
            carry[1] = s.y;
            carry[2] = w.x;
        }
        __syncthreads();
    }

    const int lane = threadIdx.x & 31;
    const int warps = (blockDim.x >> 5) * gridDim.x;
    const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    // rows: 128 consecutive ones per warp
    for (int row0 = warp * 128; row0 < nrows; row0 += warps * 128) {
        int first = 0, hi = R;  // the request of the warp's first row: the first with an end beyond
        while (first < hi) {
            const int mid = (first + hi) >> 1;
            if (row_end[mid] <= (unsigned)row0) first = mid + 1;
            else hi = mid;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = row0 + k * 32 + lane;
            if (row >= nrows) continue;
            int r = first;
            if (r < R && row_end[r] <= (unsigned)row) {  // gallop, then halve
                int b = 1;
                while (r + b < R && row_end[r + b] <= (unsigned)row) b <<= 1;
                int lo = r + (b >> 1) + 1, up = min(r + b, R);
                while (lo < up) {
                    const int mid = (lo + up) >> 1;
                    if (row_end[mid] <= (unsigned)row) lo = mid + 1;
                    else up = mid;
                }
                r = lo;
            }
            int req = -1, pos = -1, slot = -1;
            if (r < R && off[r] >= 0) {
                const int old = A.len_in[r], have = (old + P - 1) >> lgP;
                req = r;
                pos = old + row - (int)(r > 0 ? row_end[r - 1] : 0u);
                const int j = pos >> lgP;
                int page;
                if (j < have) {
                    page = A.table[(size_t)r * maxp + j];
                } else {
                    int at = head + off[r] + (j - have);  // < 2 npages
                    if (at >= npages) at -= npages;
                    page = A.free_pages[at];
                    if ((pos & (P - 1)) == 0) A.table[(size_t)r * maxp + j] = page;
                }
                if ((unsigned)page < (unsigned)npages) slot = (page << lgP) + (pos & (P - 1));
            }
            A.row_req[row] = req;
            A.row_pos[row] = pos;
            A.slot_map[row] = slot;
        }
    }
    // finished requests: their pages go behind the ring's free ones (places that no row reads)
    for (int r = warp; r < R; r += warps) {
        if (A.new_len[r] >= 0 || off[r] < 0) continue;
        const int have = (A.len_in[r] + P - 1) >> lgP;
        for (int j = lane; j < have; j += 32) {
            const long long at = (long long)head + n_free + off[r] + j;
            A.free_pages[at % npages] = A.table[(size_t)r * maxp + j];
        }
    }
    if (gridDim.x > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::
                         : "memory");
    } else {
        __syncthreads();
    }
    if (blockIdx.x != 0) return;
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
        const int nw = A.new_len[r], old = A.len_in[r];
        A.q_start[r] = (int)min(r > 0 ? row_end[r - 1] : 0u, (unsigned)nrows);
        A.len_out[r] = off[r] < 0 ? old : (nw < 0 ? 0 : old + nw);
    }
    if (threadIdx.x == 0) {
        A.q_start[R] = (int)min(row_end[R - 1], (unsigned)nrows);
        int at = head + (int)s_taken;
        if (at >= npages) at -= npages;
        A.pool_out[0] = at;
        A.pool_out[1] = (int)min((unsigned)n_free - s_taken + carry[1], (unsigned)npages);
        A.pool_out[2] = (int)min(row_end[R - 1], (unsigned)nrows);
        A.pool_out[3] = s_refused;
    }
}

// ---- paged append ----------------------------------------------------------------------------------
// One 16-byte word of K and of V per thread and step: consecutive threads take consecutive words of
// a row (all heads), so reads are whole rows and writes whole head rows of a page. Bound by HBM.
__global__ void __launch_bounds__(256)
    pg_append_kernel(const uint4 *__restrict__ K_new, const uint4 *__restrict__ V_new,
                     long long k_row, long long v_row, const int32_t *__restrict__ slots,
                     uint4 *__restrict__ K, uint4 *__restrict__ V, int rows, int Hkv, int lgv,
                     int lgP, int nslots, unsigned *err) {
    const int vpr = Hkv << lgv;  // words per row
    const long long total = (long long)rows * vpr;
    for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < total;
         e += (long long)gridDim.x * blockDim.x) {
        const int row = (int)(e / vpr), c = (int)(e - (long long)row * vpr);
        const int slot = __ldg(slots + row);
        if (slot < 0) continue;
        if (slot >= nslots) {
            if (c == 0) atomicOr(err, KVE_DEVERR_BADPAGE);
            continue;
        }
        const uint4 k = __ldg(K_new + row * k_row + c), v = __ldg(V_new + row * v_row + c);
        const int page = slot >> lgP, o = slot & ((1 << lgP) - 1);
        const size_t dst = (((((size_t)page * Hkv + (c >> lgv)) << lgP) + o) << lgv) +
                           (c & ((1 << lgv) - 1));
        K[dst] = k;
        V[dst] = v;
    }
}

// ---- attention on the CUDA cores -------------------------------------------------------------------
constexpr int kSimtRows = 16, kSimtTok = 32, kSimtThreads = 128;

// One CTA: 16 rows (row = (row of the batch, query head of the KV head), heads fastest) of one
// prompt and KV head over a split of the prompt, or of one request and KV head over a split of its
// own rows. Eight threads share a row: each scores 4 of a tile's 32 tokens and holds D/8 of the
// row's output columns; fp32 throughout, running maximum and sum in the log2 domain.
// Blocks 0 .. prompt_ctas - 1 take the prompt's part, the others the requests'.
template <int D>
__global__ void __launch_bounds__(kSimtThreads)
    pg_attn_simt_kernel(PgDims D_, PgAttn A, int prompt_ctas, int prompt_blocks, int own_blocks) {
    constexpr int LD = D + 4, WPR = D / 4, NC = D / 32;
    __shared__ __align__(16) float qs[kSimtRows][LD], ks[kSimtTok][LD], vs[kSimtTok][LD];
    __shared__ float ps[kSimtRows][kSimtTok + 1];
    const bool own = (int)blockIdx.x >= prompt_ctas;
    int b = own ? blockIdx.x - prompt_ctas : blockIdx.x;
    const int nsplit = own ? D_.ns : D_.np, nblk = own ? own_blocks : prompt_blocks;
    const int sp = b % nsplit;
    b /= nsplit;
    const int rb0 = b % nblk;
    b /= nblk;
    const int kh = b % D_.Hkv, u = b / D_.Hkv;  // prompt or request
    const int r0 = own ? u : u * D_.F, r1 = own ? u + 1 : r0 + D_.F;
    const int tok0 = pg_start(A.q_start, r0, D_.rows), tok1 = pg_start(A.q_start, r1, D_.rows);
    const int nrow = (tok1 - tok0) * D_.g;
    if (rb0 * kSimtRows >= nrow) return;
    // tokens of this split, and what the first row sees of them
    int end, see0;
    if (own) {
        end = pg_clamp(__ldg(A.len + u), 0, D_.cap());
        see0 = end - (tok1 - tok0) + 1;
    } else {
        end = A.plen ? pg_clamp(__ldg(A.plen + u), 0, D_.n) : D_.n;
        see0 = end;
    }
    const int step = own ? D_.ssplit : D_.psplit;
    const int t0 = sp * step, t1 = min(end, t0 + step);
    if (t0 >= t1) return;

    const int row = threadIdx.x >> 3, sub = threadIdx.x & 7;
    const float k1 = kLog2e * rsqrtf((float)D);
    const float *Kb = static_cast<const float *>(own ? A.K : A.Kp);
    const float *Vb = static_cast<const float *>(own ? A.V : A.Vp);
    // the launch has blocks for max_new rows a request; a request refused for packing more leaves
    // more rows to go through
    for (int rb = rb0; rb * kSimtRows < nrow; rb += nblk) {
        const int rr = rb * kSimtRows + row;
        const bool live = rr < nrow;
        const int tok = tok0 + (live ? rr / D_.g : 0), h = kh * D_.g + (live ? rr % D_.g : 0);
        const int see = own ? min(t1, see0 + (tok - tok0)) : t1;
        __syncthreads();  // the last tile's readers are done
        for (int e = threadIdx.x; e < kSimtRows * D; e += kSimtThreads) {
            const int i = e / D, c = e % D, ri = rb * kSimtRows + i;
            float v = 0.f;
            if (ri < nrow)
                v = static_cast<const float *>(A.q)[(tok0 + ri / D_.g) * A.q_row +
                                                    (size_t)(kh * D_.g + ri % D_.g) * D + c];
            qs[i][c] = v;
        }
        float m = kPgNoMax, l = 0.f, acc[NC * 4];
#pragma unroll
        for (int i = 0; i < NC * 4; ++i) acc[i] = 0.f;
        for (int t = t0; t < t1; t += kSimtTok) {
            __syncthreads();
            for (int e = threadIdx.x; e < kSimtTok * WPR; e += kSimtThreads) {
                const int i = e / WPR, c = (e % WPR) * 4, j = t + i;
                float4 kw = make_float4(0.f, 0.f, 0.f, 0.f), vw = kw;
                if (j < t1) {
                    size_t at;
                    if (own) {
                        const int page = pg_page(A.table + (size_t)u * D_.maxp, j, D_.lgP,
                                                 D_.npages, A.err);
                        at = ((((size_t)page * D_.Hkv + kh) << D_.lgP) + (j & (D_.P - 1))) * D;
                    } else {
                        at = u * A.p_prompt + kh * A.p_head + j * A.p_tok;
                    }
                    kw = __ldg(reinterpret_cast<const float4 *>(Kb + at + c));
                    vw = __ldg(reinterpret_cast<const float4 *>(Vb + at + c));
                }
                *reinterpret_cast<float4 *>(&ks[i][c]) = kw;
                *reinterpret_cast<float4 *>(&vs[i][c]) = vw;
            }
            __syncthreads();
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 q = *reinterpret_cast<const float4 *>(&qs[row][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 k = *reinterpret_cast<const float4 *>(&ks[sub + 8 * i][c]);
                    s[i] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[i]))));
                }
            }
            float mt = m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = t + sub + 8 * i < see ? s[i] * k1 : -INFINITY;
                mt = fmaxf(mt, s[i]);
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
            const float f = exp2f(m - mt);
            m = mt;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = exp2f(s[i] - m);
                sum += p;
                ps[row][sub + 8 * i] = p;
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = fmaf(l, f, sum);
#pragma unroll
            for (int i = 0; i < NC * 4; ++i) acc[i] *= f;
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < kSimtTok; ++i) {
                const float p = ps[row][i];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(&vs[i][sub * 4 + 32 * c]);
                    acc[4 * c] = fmaf(p, v.x, acc[4 * c]);
                    acc[4 * c + 1] = fmaf(p, v.y, acc[4 * c + 1]);
                    acc[4 * c + 2] = fmaf(p, v.z, acc[4 * c + 2]);
                    acc[4 * c + 3] = fmaf(p, v.w, acc[4 * c + 3]);
                }
            }
        }
        if (!live) continue;
        const size_t at = ((size_t)(own ? D_.np + sp : sp) * D_.rows + tok) * D_.Hq + h;
        if (sub == 0) A.part_ml[at] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            *reinterpret_cast<float4 *>(A.part_o + at * D + sub * 4 + 32 * c) =
                make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
    }
}

// ---- joining the partial results ---------------------------------------------------------------------
// One warp per (row, query head): with M = max_s m_s over the row's prompt and own splits,
// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s, in split order.
template <typename T, int D>
__global__ void __launch_bounds__(256) pg_join_kernel(PgDims D_, PgAttn A) {
    constexpr int E = D / 32;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (w >= (long long)D_.rows * D_.Hq) return;
    const int tok = (int)(w / D_.Hq);
    const int r = __ldg(A.row_req + tok);
    if (r < 0 || r >= D_.R) return;
    const int first = __ldg(A.q_start + r);
    if (tok < first || tok >= __ldg(A.q_start + r + 1)) return;
    const int u = r / D_.F;
    const int plen = A.plen ? pg_clamp(__ldg(A.plen + u), 0, D_.n) : D_.n;
    const int len = pg_clamp(__ldg(A.len + r), 0, D_.cap());
    const int np = D_.np > 0 ? (plen + D_.psplit - 1) / D_.psplit : 0;
    const int nsp = np + (len + D_.ssplit - 1) / D_.ssplit;
    const size_t step = (size_t)D_.rows * D_.Hq;
    // split s lies at place s (prompt) or D_.np + s - np (own rows)
    float M = kPgNoMax;
    for (int s = lane; s < nsp; s += 32)
        M = fmaxf(M, A.part_ml[(size_t)(s < np ? s : s - np + D_.np) * step + w].x);
    M = warp_max(M);
    float L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int s0 = 0; s0 < nsp; s0 += 32) {
        float wt = 0.f, lw = 0.f;
        if (s0 + lane < nsp) {
            const int s = s0 + lane;
            const float2 ml = A.part_ml[(size_t)(s < np ? s : s - np + D_.np) * step + w];
            wt = exp2f(ml.x - M);
            lw = wt * ml.y;
        }
        L += warp_sum(lw);
        const int cnt = min(32, nsp - s0);
#pragma unroll 4
        for (int j = 0; j < cnt; ++j) {
            const int s = s0 + j;
            const float f = __shfl_sync(0xffffffffu, wt, j);
            const float *o = A.part_o +
                             ((size_t)(s < np ? s : s - np + D_.np) * step + w) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(f, o[e], acc[e]);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    T *dst = static_cast<T *>(A.out) + (size_t)w * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = from_f<T>(acc[e] * inv);
    if (A.lse && lane == 0) A.lse[w] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t attn_simt(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    const long long pb = (D_.group_rows() * D_.g + kSimtRows - 1) / kSimtRows;
    const long long ob = ((long long)D_.max_new * D_.g + kSimtRows - 1) / kSimtRows;
    const long long pc = (long long)D_.S * D_.Hkv * pb * D_.np;
    const long long oc = (long long)D_.R * D_.Hkv * ob * D_.ns;
    if (pc + oc > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    pg_attn_simt_kernel<D><<<(unsigned)(pc + oc), kSimtThreads, 0, st>>>(D_, A, (int)pc, (int)pb,
                                                                         (int)ob);
    return cudaGetLastError();
}

template <typename T>
cudaError_t join(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    const long long warps = (long long)D.rows * D.Hq;
    const unsigned ctas = (unsigned)((warps + 7) / 8);
    if (D.d == 128) pg_join_kernel<T, 128><<<ctas, 256, 0, st>>>(D, A);
    else if (D.d == 64) pg_join_kernel<T, 64><<<ctas, 256, 0, st>>>(D, A);
    else pg_join_kernel<T, 32><<<ctas, 256, 0, st>>>(D, A);
    return cudaGetLastError();
}

}  // namespace

// ---- launchers -----------------------------------------------------------------------------------
cudaError_t launch_pg_plan(const PgDims &D, const PgPlanArgs &A, cudaStream_t st) {
    // one warp for the smallest steps (no barrier to wait for), up to 1024 threads, then up to 8
    // CTAs of a cluster: a CTA per 4096 rows
    long long work = D.R > (D.rows + 3) / 4 ? D.R : (D.rows + 3) / 4;
    int threads = 32;
    while (threads < 1024 && threads < work) threads <<= 1;
    int ctas = 1;
    while (ctas < 8 && (long long)ctas * 4096 < D.rows) ctas <<= 1;
    const size_t smem = 2 * sizeof(int) * (size_t)D.R;
    cudaError_t e = cudaFuncSetAttribute(pg_plan_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, 131072);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pg_plan_kernel, A, D.R, D.lgP, D.npages, D.maxp, D.rows,
                              D.max_new);
}

cudaError_t launch_pg_append(const PgDims &D, const void *K_new, const void *V_new,
                             long long k_row, long long v_row, const int32_t *slots, void *K,
                             void *V, unsigned *err, cudaStream_t st) {
    const int es = (int)dtype_size(D.dtype), words = D.d * es / 16;  // 4, 8, 16 or 32
    int lgv = 0;
    while ((1 << lgv) < words) ++lgv;
    const long long total = (long long)D.rows * D.Hkv * words;
    long long blocks = (total + 255) / 256;
    if (blocks > 152 * 64) blocks = 152 * 64;
    pg_append_kernel<<<(unsigned)blocks, 256, 0, st>>>(
        static_cast<const uint4 *>(K_new), static_cast<const uint4 *>(V_new), k_row * es / 16,
        v_row * es / 16, slots, static_cast<uint4 *>(K), static_cast<uint4 *>(V), D.rows, D.Hkv,
        lgv, D.lgP, D.npages << D.lgP, err);
    return cudaGetLastError();
}

cudaError_t launch_pg_attention(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    if (D.dtype == KVE_F32) {
        cudaError_t e = D.d == 128 ? attn_simt<128>(D, A, st)
                                   : (D.d == 64 ? attn_simt<64>(D, A, st) : attn_simt<32>(D, A, st));
        return e != cudaSuccess ? e : join<float>(D, A, st);
    }
    cudaError_t e = cudaSuccess;
    if (D.n > 0) e = pg_prompt_tc(D) ? launch_pg_prompt_tc(D, A, st) : launch_pg_prompt_mma(D, A, st);
    if (e == cudaSuccess) e = launch_pg_own_mma(D, A, st);
    if (e != cudaSuccess) return e;
    return D.dtype == KVE_BF16 ? join<__nv_bfloat16>(D, A, st) : join<__half>(D, A, st);
}

}  // namespace kve
