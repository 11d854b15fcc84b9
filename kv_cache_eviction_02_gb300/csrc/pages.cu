// Shared-prompt decoding on the CUDA cores: the page planner, the paged append, the attention of
// fp32 inputs and the kernel that joins the partial results of an attention call.
#include "pages.cuh"

namespace kve {

// How an attention call is split.
//   Prompt, 16-bit types (one CTA per SM): the split count that minimises
//     ceil(items * splits / 152) * (tiles per split + 4): a CTA's set-up and the partial result that
//     it writes and the join reads cost about four tiles. A short prompt leaves SMs over; the own
//     rows' kernel then runs on those beside it (with blocks for all SMs, the last of its equal shares
//     would begin when the prompt's kernel has ended: 51 instead of 41 us for 64 answers behind 164
//     rows). Holding a long prompt's kernel back to a share of the SMs so that both end together was
//     no faster than one after the other (256 requests behind 8K rows: 139 and 137 us): own rows need
//     all SMs' buffers in flight to reach the HBM rate.
//   fp32: enough CTAs to fill the GPU a few times, at least 128 tokens each; own rows by the table's
//     width, since lengths are known on the device only (the CTAs of splits that a request does not
//     reach return at once). 16-bit own rows are dealt out on the device (pages_own.cu).
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
    D->np = D->ns = 0;
    D->psplit = 128;
    D->ssplit = 256;
    D->own_sms = kPgSms;
    if (D->dtype == KVE_F32) {
        if (D->n > 0)
            split((long long)D->S * D->Hkv * ((prow + 15) / 16), D->n, kPgSms * 8, 128, &D->np,
                  &D->psplit);
        split((long long)D->R * D->Hkv * ((orow + 15) / 16), D->cap(), kPgSms * 8, 256, &D->ns,
              &D->ssplit);
    } else if (D->n > 0) {
        const long long pairs = pg_prompt_pairs(*D), per = pg_tile_rows(*D) * pairs;
        const long long most = D->S * ((D->group_rows() + per - 1) / per);  // launched per KV head
        const long long all = D->rows / per + D->S;                         // of which hold rows
        const long long items = D->Hkv * (most < all ? most : all);
        const long long tiles = (D->n + 127LL) / 128;
        long long best = -1, len = 1;
        for (long long p = 1; p <= 64 && p <= tiles; ++p) {
            const long long waves = (items * p + kPgSms - 1) / kPgSms, t = (tiles + p - 1) / p;
            const long long cost = waves * (t + 4);
            if (best < 0 || cost < best) {
                best = cost;
                len = t;
            }
        }
        D->psplit = (int)(len * 128);
        D->np = (int)((tiles + len - 1) / len);
        // (the prompt's kernel starts first)
        const long long ctas = D->Hkv * most * D->np;
        if (ctas < kPgShare) D->own_sms = (int)(kPgSms - ctas);
    }
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
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~size_t(255);
        return at;
    };
    const bool f32 = D.dtype == KVE_F32;
    const size_t rows = (size_t)D.rows * D.Hq * (D.np + (f32 ? D.ns : 0));
    W.part_ml = take(sizeof(float2) * rows);
    W.part_o = take(sizeof(float) * rows * D.d);
    const size_t segs = f32 ? 0 : (size_t)pg_own_segs(D) * pg_seg_rows(D);
    W.own_ml = take(sizeof(float2) * segs);
    W.own_o = take(sizeof(float) * segs * D.d);
    W.own_base = take(f32 ? 0 : sizeof(long long) * D.R);
    W.own_unit = take(f32 ? 0 : sizeof(int) * D.R);
    W.own_cpw = take(f32 ? 0 : sizeof(long long));
    W.total = off;
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
// keeps, per request, the end of its rows, its length and its offset into the ring in shared memory;
// rows and finished requests are then shared out over the cluster's warps. A row finds its request in
// shared memory and its page in the table (an old page) or straight in the ring (a new one), so
// nothing waits for another CTA's stores; the row that opens a new page writes it to the table. Those
// loads are never of cells that the launch writes: old table entries stay, and returned pages go
// behind the ring's free window.
// Lengths and the pool are written by the first CTA behind a cluster barrier that every CTA reaches
// when it has read them, so both may be updated in place.
// Bound by latency: launch, the loads of the lengths, two scans, one dependent load per batch of rows.
// Four rows per lane are looked up before the first is stored, so their loads overlap.
constexpr int kPlanUnroll = 4;

// The first request whose rows end behind `row`, searched from `from` on.
__device__ __forceinline__ int plan_find(const unsigned *row_end, int from, int R, unsigned row) {
    int lo = from, b = 1;  // gallop, then halve
    if (lo >= R || row_end[lo] > row) return lo;
    while (lo + b < R && row_end[lo + b] <= row) b <<= 1;
    int up = min(lo + b, R);
    lo += (b >> 1) + 1;
    while (lo < up) {
        const int mid = (lo + up) >> 1;
        if (row_end[mid] <= row) lo = mid + 1;
        else up = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(1024)
    pg_plan_kernel(PgPlanArgs A, int R, int lgP, int npages, int maxp, int nrows, int max_new) {
    extern __shared__ unsigned sh_plan[];
    unsigned *row_end = sh_plan;                           // [R]
    int *len = reinterpret_cast<int *>(sh_plan + R);       // [R] as it was
    int *off = len + R;  // [R] ring offset of its new pages; -1: refused; -2 - offset: finished
    __shared__ uint2 tot[32];
    __shared__ unsigned carry[3];  // rows, returned pages, wanted pages of the tiles before
    __shared__ int s_refused;
    __shared__ unsigned s_taken;
    const int P = 1 << lgP;
    const int cap = maxp << lgP;
    const int head_in = A.pool_in[0], free_in = A.pool_in[1];
    int nw = 0, old = 0;
    if ((int)threadIdx.x < R) {
        nw = A.new_len[threadIdx.x];
        old = A.len_in[threadIdx.x];
    }
    if (threadIdx.x == 0) {
        carry[0] = carry[1] = carry[2] = 0;
        s_refused = 0;
        s_taken = 0;
    }
    const int n_free = pg_clamp(free_in, 0, npages);
    const int head = (unsigned)head_in < (unsigned)npages ? head_in : 0;
    const uint2 cap1 = make_uint2((unsigned)nrows + 1u, (unsigned)npages + 1u);
    const uint2 cap2 = make_uint2((unsigned)npages + 1u, 1u);
    __syncthreads();
    for (int base = 0; base < R; base += blockDim.x) {
        const int r = base + threadIdx.x;
        if (base > 0 && r < R) {
            nw = A.new_len[r];
            old = A.len_in[r];
        }
        if (r >= R) nw = old = 0;
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
            len[r] = old;
            off[r] = bad ? -1 : (nw < 0 ? -2 - (int)(s.y - freed) : (int)(w.x - want));
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
    if (gridDim.x > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");

    const int lane = threadIdx.x & 31;
    const int warps = (blockDim.x >> 5) * gridDim.x;
    const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    // rows: 32 consecutive ones per warp and step, `warps * 32` apart
    for (int base = warp * 32; base < nrows; base += warps * 32 * kPlanUnroll) {
        int req[kPlanUnroll], pos[kPlanUnroll], page[kPlanUnroll];
        long long cell[kPlanUnroll];  // the table cell of a new page
#pragma unroll
        for (int k = 0; k < kPlanUnroll; ++k) {
            const int row0 = base + k * warps * 32, row = row0 + lane;
            req[k] = pos[k] = page[k] = -1;
            cell[k] = -1;
            if (row0 >= nrows) continue;
            int lo = 0, up = R;  // the same search in every lane: the request of the first row
            while (lo < up) {
                const int mid = (lo + up) >> 1;
                if (row_end[mid] <= (unsigned)row0) lo = mid + 1;
                else up = mid;
            }
            const int r = plan_find(row_end, lo, R, (unsigned)row);
            if (r < R && off[r] >= 0) {
                const int was = len[r], have = (was + P - 1) >> lgP;
                req[k] = r;
                pos[k] = was + row - (int)(r > 0 ? row_end[r - 1] : 0u);
                const int j = pos[k] >> lgP;
                const size_t at = (size_t)r * maxp + j;
                int ring = head + off[r] + (j - have);  // < 2 npages
                if (ring >= npages) ring -= npages;
                page[k] = __ldg(j < have ? A.table + at : A.free_pages + ring);
                if (j >= have && (pos[k] & (P - 1)) == 0) cell[k] = (long long)at;
            }
        }
#pragma unroll
        for (int k = 0; k < kPlanUnroll; ++k) {
            const int row = base + k * warps * 32 + lane;
            if (row >= nrows) continue;
            A.row_req[row] = req[k];
            A.row_pos[row] = pos[k];
            A.slot_map[row] = (unsigned)page[k] < (unsigned)npages
                                  ? (page[k] << lgP) + (pos[k] & (P - 1))
                                  : -1;
            if (cell[k] >= 0) A.table[cell[k]] = page[k];
        }
    }
    // finished requests: their pages go behind the ring's free ones (places that no row reads)
    for (int r0 = warp * 32; r0 < R; r0 += warps * 32) {
        unsigned done = __ballot_sync(0xffffffffu, r0 + lane < R && off[r0 + lane] < -1);
        for (; done; done &= done - 1) {
            const int r = r0 + __ffs(done) - 1;
            const int have = (len[r] + P - 1) >> lgP;
            for (int j = lane; j < have; j += 32) {
                const long long at = (long long)head + n_free + (-2 - off[r]) + j;
                A.free_pages[at % npages] = __ldg(A.table + (size_t)r * maxp + j);
            }
        }
    }
    if (gridDim.x > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (blockIdx.x != 0) return;
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
        const unsigned first = r > 0 ? row_end[r - 1] : 0u;
        A.q_start[r] = (int)min(first, (unsigned)nrows);
        A.len_out[r] = off[r] == -1 ? len[r] : (off[r] < 0 ? 0 : len[r] + (int)(row_end[r] - first));
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
template <int D, bool OWN>
__device__ __forceinline__ void attn_simt_block(const PgDims &D_, const PgAttn &A, int nblk) {
    constexpr int LD = D + 4, WPR = D / 4, NC = D / 32;
    __shared__ __align__(16) float qs[kSimtRows][LD], ks[kSimtTok][LD], vs[kSimtTok][LD];
    __shared__ float ps[kSimtRows][kSimtTok + 1];
    const int nsplit = OWN ? D_.ns : D_.np;
    int b = blockIdx.x;
    const int sp = b % nsplit;
    b /= nsplit;
    const int rb0 = b % nblk;
    b /= nblk;
    const int kh = b % D_.Hkv, u = b / D_.Hkv;  // prompt or request
    const int r0 = OWN ? u : u * D_.F, r1 = OWN ? u + 1 : r0 + D_.F;
    const int tok0 = pg_start(A.q_start, r0, D_.rows), tok1 = pg_start(A.q_start, r1, D_.rows);
    const int nrow = (tok1 - tok0) * D_.g;
    if (rb0 * kSimtRows >= nrow) return;
    // tokens of this split, and what the first row sees of them
    int end, see0;
    if (OWN) {
        end = pg_clamp(__ldg(A.len + u), 0, D_.cap());
        see0 = end - (tok1 - tok0) + 1;
    } else {
        end = A.plen ? pg_clamp(__ldg(A.plen + u), 0, D_.n) : D_.n;
        see0 = end;
    }
    const int step = OWN ? D_.ssplit : D_.psplit;
    const int t0 = sp * step, t1 = min(end, t0 + step);
    if (t0 >= t1) return;

    const int row = threadIdx.x >> 3, sub = threadIdx.x & 7;
    const float k1 = kLog2e * rsqrtf((float)D);
    const float *Kb = static_cast<const float *>(OWN ? A.K : A.Kp);
    const float *Vb = static_cast<const float *>(OWN ? A.V : A.Vp);
    // the launch has blocks for max_new rows a request; a request refused for packing more leaves
    // more rows to go through
    for (int rb = rb0; rb * kSimtRows < nrow; rb += nblk) {
        const int rr = rb * kSimtRows + row;
        const bool live = rr < nrow;
        const int tok = tok0 + (live ? rr / D_.g : 0), h = kh * D_.g + (live ? rr % D_.g : 0);
        const int see = OWN ? min(t1, see0 + (tok - tok0)) : t1;
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
                    if (OWN) {
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
        const size_t at = ((size_t)(OWN ? D_.np + sp : sp) * D_.rows + tok) * D_.Hq + h;
        if (sub == 0) A.part_ml[at] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            *reinterpret_cast<float4 *>(A.part_o + at * D + sub * 4 + 32 * c) =
                make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
    }
}

template <int D, bool OWN>
__global__ void __launch_bounds__(kSimtThreads) pg_attn_simt_kernel(PgDims D_, PgAttn A, int nblk) {
    if (!OWN || D_.n == 0) pg_wait_prior();  // first kernel of its call
    pg_launch_dependents();
    attn_simt_block<D, OWN>(D_, A, nblk);
    if (OWN) pg_wait_prior();
}

// ---- joining the partial results ---------------------------------------------------------------------
// One warp per (row, query head): with M = max_s m_s over the row's partial results s (prompt splits,
// then own rows in order), out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s, in that order whatever
// order they were made in. Bound by latency: which partial results a row has is worked out before the
// kernels that make them have ended, and eight of them are on their way at a time.
template <typename T, int D>
__device__ __forceinline__ void join_row(const PgDims &D_, const PgAttn &A) {
    constexpr int E = D / 32, U = 8;
    constexpr bool F32 = sizeof(T) == 4;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const bool in = w < (long long)D_.rows * D_.Hq;
    const int tok = in ? (int)(w / D_.Hq) : 0;
    int r = in ? __ldg(A.row_req + tok) : -1;
    if (r >= D_.R) r = -1;
    int len = 0, first = 0, nq = 0, cr = 0, nb = 0, plen = 0;
    if (r >= 0) {
        pg_own_request(D_, A, r, &len, &first, &nq, &cr, &nb);
        plen = A.plen ? pg_clamp(__ldg(A.plen + r / D_.F), 0, D_.n) : D_.n;
    }
    const bool mine = r >= 0 && tok >= first && tok - first < min(nq, D_.max_new);
    pg_wait_prior();
    pg_launch_dependents();
    if (!mine) return;
    const int h = (int)(w - (long long)tok * D_.Hq);
    const int np = D_.np > 0 ? (plen + D_.psplit - 1) / D_.psplit : 0;
    const long long step = (long long)D_.rows * D_.Hq;
    int nsp;
    long long seg = 0;
    if (F32) {
        nsp = np + (len + D_.ssplit - 1) / D_.ssplit;
    } else {
        const int rb = pg_unit_rows(D_);
        const int rr = (tok - first) * D_.g + h % D_.g, u = h / D_.g * nb + rr / rb;
        const long long cpw = *A.own.cpw, x = A.own.base[r] + (long long)u * cr;
        const long long w0 = x / cpw, w1 = cr > 0 ? (x + cr - 1) / cpw : w0 - 1;
        const long long at = A.own.unit[r] + u + w0;
        // as many pieces as there are places (all of them when the row starts are sums of lengths)
        const long long have = at + (w1 - w0 + 1) <= A.own.segs ? w1 - w0 + 1 : A.own.segs - at;
        nsp = np + (int)(have > 0 ? have : 0);
        seg = at * A.own.seg_rows + (rr & (rb - 1));
    }
    auto row_of = [&](int s) -> long long {  // the partial result's row in its arrays
        if (s < np) return s * step + w;
        return F32 ? (long long)(s - np + D_.np) * step + w
                   : seg + (long long)(s - np) * A.own.seg_rows;
    };
    auto o_of = [&](int s) {
        return (F32 || s < np ? A.part_o : A.own.o) + row_of(s) * D + lane * E;
    };
    auto ml_of = [&](int s) { return (F32 || s < np ? A.part_ml : A.own.ml)[row_of(s)]; };
    float v[U][E];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[j][e] = 0.f;
            if (s0 + j < nsp) {
                const float *o = o_of(s0 + j);
                if (E == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(o);
                    v[j][0] = x.x;
                    v[j][E > 1 ? 1 : 0] = x.y;
                    v[j][E > 2 ? 2 : 0] = x.z;
                    v[j][E > 3 ? 3 : 0] = x.w;
                } else if (E == 2) {
                    const float2 x = *reinterpret_cast<const float2 *>(o);
                    v[j][0] = x.x;
                    v[j][E > 1 ? 1 : 0] = x.y;
                } else {
                    v[j][0] = *o;
                }
            }
        }
    };
    fetch(0);
    float2 ml = make_float2(kPgNoMax, 0.f);
    if (lane < nsp) ml = ml_of(lane);
    float M = ml.x;
    for (int s = lane + 32; s < nsp; s += 32) M = fmaxf(M, ml_of(s).x);
    M = warp_max(M);
    float L = 0.f, acc[E], wt = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int s0 = 0; s0 < nsp; s0 += U) {
        if ((s0 & 31) == 0) {  // the weights of 32 partial results, one per lane
            if (s0 > 0) ml = s0 + lane < nsp ? ml_of(s0 + lane) : make_float2(kPgNoMax, 0.f);
            wt = s0 + lane < nsp ? exp2f(ml.x - M) : 0.f;
            L += warp_sum(wt * ml.y);
        }
        if (s0 > 0) fetch(s0);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float f = __shfl_sync(0xffffffffu, wt, (s0 + j) & 31);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(f, v[j][e], acc[e]);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    T *dst = static_cast<T *>(A.out) + (size_t)w * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = from_f<T>(acc[e] * inv);
    if (A.lse && lane == 0) A.lse[w] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <typename T, int D>
__global__ void __launch_bounds__(128) pg_join_kernel(PgDims D_, PgAttn A) {
    join_row<T, D>(D_, A);
}

template <int D, bool OWN>
cudaError_t attn_simt(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    const long long rows = (OWN ? (long long)D_.max_new : D_.group_rows()) * D_.g;
    const long long nblk = (rows + kSimtRows - 1) / kSimtRows;
    const long long ctas = (long long)(OWN ? D_.R : D_.S) * D_.Hkv * nblk * (OWN ? D_.ns : D_.np);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return pg_launch(pg_attn_simt_kernel<D, OWN>, (unsigned)ctas, kSimtThreads, 0, true, st, D_, A,
                     (int)nblk);
}

template <bool OWN> cudaError_t simt(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.d == 128 ? attn_simt<128, OWN>(D, A, st)
                      : (D.d == 64 ? attn_simt<64, OWN>(D, A, st) : attn_simt<32, OWN>(D, A, st));
}

template <typename T> cudaError_t join(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    const unsigned ctas = (unsigned)(((long long)D.rows * D.Hq + 3) / 4);
    auto kern = D.d == 128 ? pg_join_kernel<T, 128>
                           : (D.d == 64 ? pg_join_kernel<T, 64> : pg_join_kernel<T, 32>);
    return pg_launch(kern, ctas, 128, 0, true, st, D, A);
}

}  // namespace

// ---- launchers -----------------------------------------------------------------------------------
cudaError_t launch_pg_plan(const PgDims &D, const PgPlanArgs &A, cudaStream_t st) {
    // one warp for the smallest steps (no barrier to wait for), up to 1024 threads, then up to 8
    // CTAs of a cluster: a CTA per 4096 rows
    const int work = D.R > D.rows ? D.R : D.rows;
    int threads = 32;
    while (threads < 1024 && threads < work) threads <<= 1;
    int ctas = 1;
    while (ctas < 8 && (long long)ctas * 4096 < D.rows) ctas <<= 1;
    const size_t smem = 3 * sizeof(int) * (size_t)D.R;
    if (smem > 40 * 1024) {  // with the static arrays above 48 KB
        cudaError_t e = cudaFuncSetAttribute(
            pg_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * 4 * 16384);
        if (e != cudaSuccess) return e;
    }
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

cudaError_t launch_pg_prompt(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    if (D.dtype == KVE_F32) return simt<false>(D, A, st);
    return launch_pg_prompt_tc(D, A, st);
}

cudaError_t launch_pg_own(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_F32 ? simt<true>(D, A, st) : launch_pg_own16(D, A, st);
}

cudaError_t launch_pg_join(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    if (D.dtype == KVE_F32) return join<float>(D, A, st);
    return D.dtype == KVE_BF16 ? join<__nv_bfloat16>(D, A, st) : join<__half>(D, A, st);
}

}  // namespace kve
