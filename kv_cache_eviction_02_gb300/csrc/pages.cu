// Shared-prompt decoding: sizes and splits, the page planner, the paged append, and the kernel that joins
// the partial results of an attention call.
#include "pages.cuh"

namespace kve {

// How an attention call is split.
//   Prompt, 16-bit types (one CTA per SM): the split count that minimises
//     ceil(items * splits / 152) * (tiles per split + 4): a CTA's set-up and the partial result that
//     it writes and the join reads cost about four tiles. One number for all prompts, from n_prefix: of
//     prompts much shorter than that, the CTAs of splits behind their end return at once, and a long one
//     among many short ones keeps its few splits (lengths are known on the device only). A short prompt
//     leaves SMs over; the own rows' kernel then runs on those beside it (with blocks for all SMs, the last
//     of its equal shares would begin when the prompt's kernel has ended: figures at kPgShare). Holding a
//     long prompt's kernel back to a share of the SMs so that both end together was no faster than one
//     after the other: own rows need all SMs' buffers in flight to reach the HBM rate.
//   Own rows of requests with many new rows: the same by the table's width, since lengths are known on
//     the device only (the CTAs of splits that a request does not reach return at once).
//   Other own rows, and all of fp32: dealt out on the device (pages_own.cu, pages_f32.cu).
static void pg_split(PgDims *D) {
    auto tiles_split = [](long long items, long long n, int *count, int *len) {
        const long long tiles = (n + 127) / 128;
        long long best = -1, per = 1;
        // the most splits that w rounds of the SMs hold, for the first few w
        for (long long w = (items + kPgSms - 1) / kPgSms, last = w + 12; w <= last; ++w) {
            long long p = w * kPgSms / items;
            if (p > 64) p = 64;
            if (p > tiles) p = tiles;
            const long long t = (tiles + p - 1) / p, cost = w * (t + 4);
            if (best < 0 || cost < best) {
                best = cost;
                per = t;
            }
            if (p == tiles || p == 64) break;
        }
        *len = (int)(per * 128);
        *count = (int)((tiles + per - 1) / per);
    };
    D->own_sms = kPgSms;
    D->np = D->ns = 0;
    D->psplit = 128;
    D->ssplit = 256;
    D->direct = pg_direct(*D);
    D->prompt_own = false;
    D->line = D->n > 0;
    if (D->dtype == KVE_F32 || D->direct) return;
    if (D->n > 0) {
        const int pairs = pg_pairs(*D, D->group_rows());
        const long long per = pg_tile_rows(*D) * pairs;
        const long long most = (long long)D->S * pg_tc_blocks(*D, false);  // launched per KV head
        const long long all = D->rows / per + D->S;                        // of which hold rows
        const long long items = D->Hkv * (most < all ? most : all);
        tiles_split(items, D->n, &D->np, &D->psplit);
        // two warps per CTA, beside its tiles: a row takes 1 us and 1.3 for every 8 tokens, a tile 0.6, and there
        // are 3 besides (measured: 16 prompts of 2K rows with 4 requests of up to 32 own rows 115 us so, 33 with
        // a launch for the own rows; 4 of 32K 93 and 107)
        const long long rows = D->group_rows() * D->g < 128 ? D->group_rows() * D->g : 128;
        const long long own = (rows + 2 * D->np - 1) / (2 * D->np) * (10 + 13 * ((D->cap() + 7) / 8));
        D->prompt_own = pairs == 1 && D->cap() <= kPgFewOwn && !pg_many_new(*D) &&
                        own <= 30 + 6 * (D->psplit / 128);
        D->line = !D->prompt_own && pg_short_prompts(*D);
        if (D->line) {
            D->np = 0;
        } else {  // (the prompt's kernel starts first)
            const long long ctas = D->Hkv * most * D->np;
            if (ctas < kPgShare) D->own_sms = (int)(kPgSms - ctas);
        }
    }
    if (D->prompt_own) {
        D->ns = 1;
        D->ssplit = D->cap();
    } else if (pg_many_new(*D)) {
        const long long per = pg_tile_rows(*D) * pg_pairs(*D, D->max_new);
        const long long most = (long long)D->R * pg_tc_blocks(*D, true), all = D->rows / per + D->R;
        tiles_split(D->Hkv * (most < all ? most : all), D->cap(), &D->ns, &D->ssplit);
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
    if ((long long)sh->n_prompts * sh->n_kv_heads > 65535 || sh->n_q_heads > 65535)
        return (*why = "n_prompts * n_kv_heads and n_q_heads must be at most 65535"), false;
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
    const size_t rows = (size_t)D.rows * D.Hq * (D.np + D.ns);
    W.part_ml = take(sizeof(float2) * rows);
    W.part_o = take(sizeof(float) * rows * D.d);
    const size_t segs = D.prompt_own || D.direct ? 0 : (size_t)pg_own_segs(D) * pg_seg_rows(D);
    W.own_ml = take(sizeof(float2) * segs);
    W.own_o = take(sizeof(float) * segs * D.d);
    W.own_base = take(sizeof(long long) * (D.S + D.R));
    W.own_unit = take(sizeof(int) * (D.S + D.R));
    W.own_cpw = take(sizeof(long long));
    W.total = off;
    return W;
}

namespace {

// ---- page planner ----------------------------------------------------------------------------------
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b, unsigned cap) {
    return min(a + b, cap);
}

// Rows, returned pages and wanted pages; sums saturate at their caps (saturating addition of
// non-negative numbers is associative).
struct PlanSum {
    unsigned rows, back, want;
};
__device__ __forceinline__ PlanSum plan_add(PlanSum a, PlanSum b, PlanSum cap) {
    return PlanSum{sat_add(a.rows, b.rows, cap.rows), sat_add(a.back, b.back, cap.back),
                   sat_add(a.want, b.want, cap.want)};
}
__device__ __forceinline__ PlanSum plan_scan_warp(PlanSum v, PlanSum cap) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const PlanSum u{__shfl_up_sync(0xffffffffu, v.rows, o), __shfl_up_sync(0xffffffffu, v.back, o),
                        __shfl_up_sync(0xffffffffu, v.want, o)};
        if (lane >= o) v = plan_add(v, u, cap);
    }
    return v;
}
// Inclusive scan over the block; every warp scans the warps' totals by itself.
__device__ __forceinline__ PlanSum plan_scan(PlanSum v, PlanSum cap, PlanSum *tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    v = plan_scan_warp(v, cap);
    if (nw == 1) return v;
    if (lane == 31) tot[warp] = v;
    __syncthreads();
    const PlanSum t = plan_scan_warp(lane < nw ? tot[lane] : PlanSum{0, 0, 0}, cap);
    if (warp > 0)
        v = plan_add(v,
                     PlanSum{__shfl_sync(0xffffffffu, t.rows, warp - 1),
                             __shfl_sync(0xffffffffu, t.back, warp - 1),
                             __shfl_sync(0xffffffffu, t.want, warp - 1)},
                     cap);
    return v;
}

// The first request whose rows end behind `row`: the whole warp searches for one row, 32 steps at a
// time.
__device__ __forceinline__ int plan_find_warp(const unsigned *row_end, int R, unsigned row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = R;  // the answer is in lo .. lo + n
    while (n > 0) {
        const int step = (n + 31) >> 5, at = (lane + 1) * step - 1;
        const bool beyond = at < n && row_end[lo + at] <= row;
        const int k = __popc(__ballot_sync(0xffffffffu, beyond));
        lo += k * step;
        n = min(step - 1, n - k * step);
    }
    return lo;
}
// The same for one lane, from request `from` (not behind the answer) on: gallop, then halve.
__device__ __forceinline__ int plan_find(const unsigned *row_end, int from, int R, unsigned row) {
    int lo = from, b = 1;
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

// One step of the page planner. Every CTA scans all requests by itself and keeps, per request, the end
// of its rows, its length and its offset into the ring in shared memory; rows and finished requests are
// then shared out over all CTAs' warps. A row finds its request in shared memory and its page in the
// table (an old page) or straight in the ring (a new one), so nothing waits for another CTA's stores;
// the row that opens a new page writes it to the table. Those loads are never of cells that the launch
// writes: old table entries stay, and returned pages go behind the ring's free window.
// One scan serves all: whether a request is too long, or adds too much, is known before it; one whose
// rows pass n_rows makes every later one with rows pass too, so its wanted pages disturb nobody.
// Lengths and the pool may be updated in place: up to 4096 rows one CTA does everything, above that they
// are written by a second launch of one CTA, which scans beside the first and writes when it has ended.
// Bound by latency: launch, the loads of the lengths, the scan, one dependent load per row. V rows in
// a row per lane: 1 for small steps (more warps, shorter), 4 above 1024 rows (a fourth of the searches,
// 16-byte stores).
template <int V>
__global__ void __launch_bounds__(1024)
    pg_plan_kernel(PgPlanArgs A, int R, int lgP, int npages, int maxp, int nrows, int max_new,
                   bool vec, bool do_rows, bool do_lens) {
    extern __shared__ unsigned sh_plan[];
    unsigned *row_end = sh_plan;                      // [R]
    int *len = reinterpret_cast<int *>(sh_plan + R);  // [R] as it was
    int *off = len + R;  // [R] ring offset of its new pages; -1: refused; -2 - offset: finished
    __shared__ PlanSum tot[32], carry;  // carry: of the requests before this round
    __shared__ int s_refused;
    __shared__ unsigned s_taken;
    const int P = 1 << lgP;
    const int cap = maxp << lgP;
    if (do_rows) pg_wait_prior();  // (a second launch starts when the first has waited)
    pg_launch_dependents();
    const int head_in = A.pool_in[0], free_in = A.pool_in[1];
    int nw = 0, old = 0;
    if ((int)threadIdx.x < R) {
        nw = A.new_len[threadIdx.x];
        old = A.len_in[threadIdx.x];
    }
    if (threadIdx.x == 0) {
        carry = PlanSum{0, 0, 0};
        s_refused = 0;
        s_taken = 0;
    }
    const int n_free = pg_clamp(free_in, 0, npages);
    const int head = (unsigned)head_in < (unsigned)npages ? head_in : 0;
    const PlanSum caps{(unsigned)nrows + 1u, (unsigned)npages + 1u, (unsigned)npages + 1u};
    __syncthreads();
    for (int base = 0; base < R; base += blockDim.x) {
        const int r = base + threadIdx.x;
        if (base > 0) {
            nw = r < R ? A.new_len[r] : 0;
            old = r < R ? A.len_in[r] : 0;
        }
        const bool bad_len = old < 0 || old > cap;
        const int have = bad_len ? 0 : (old + P - 1) >> lgP;
        PlanSum v{0, 0, 0};
        bool bad = nw != 0 && bad_len;
        if (nw > 0) {
            v.rows = min((unsigned)nw, caps.rows);
            bad = bad || nw > max_new || (long long)old + nw > cap;
            if (!bad) v.want = (unsigned)(((old + nw + P - 1) >> lgP) - have);
        } else if (nw < 0) {
            v.back = (unsigned)have;
        }
        const PlanSum s = plan_add(plan_scan(v, caps, tot), carry, caps);
        if (nw > 0 && (s.rows > (unsigned)nrows || (v.want > 0 && s.want > (unsigned)n_free)))
            bad = true;
        if (r < R) {
            row_end[r] = s.rows;
            len[r] = old;
            off[r] = bad ? -1 : (nw < 0 ? -2 - (int)(s.back - v.back) : (int)(s.want - v.want));
            if (bad) atomicAdd(&s_refused, 1);
            if (!bad && v.want > 0) atomicMax(&s_taken, s.want);
        }
        __syncthreads();  // every thread has read the carry
        if (threadIdx.x == blockDim.x - 1) carry = s;
        __syncthreads();
    }
    const int lane = threadIdx.x & 31;
    const int warps = (blockDim.x >> 5) * gridDim.x;
    const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    for (int base = warp * 32 * V; do_rows && base < nrows; base += warps * 32 * V) {
        int r = plan_find_warp(row_end, R, (unsigned)base);
        const int row0 = base + lane * V;
        r = plan_find(row_end, r, R, (unsigned)row0);
        int req[V], pos[V], page[V];
        long long cell[V];  // the table cell of a new page, -1: none
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const unsigned row = row0 + k;
            req[k] = pos[k] = page[k] = -1;
            cell[k] = -1;
            if (k > 0)
                while (r < R && row_end[r] <= row) ++r;
            if (r >= R || off[r] < 0) continue;
            const int was = len[r], have = (was + P - 1) >> lgP;
            req[k] = r;
            pos[k] = was + (int)(row - (r > 0 ? row_end[r - 1] : 0u));
            const int j = pos[k] >> lgP;
            const size_t at = (size_t)r * maxp + j;
            int ring = head + off[r] + (j - have);  // < 2 npages
            if (ring >= npages) ring -= npages;
            page[k] = __ldg(j < have ? A.table + at : A.free_pages + ring);
            if (j >= have && (pos[k] & (P - 1)) == 0) cell[k] = (long long)at;
        }
        int slot[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            slot[k] = (unsigned)page[k] < (unsigned)npages ? (page[k] << lgP) + (pos[k] & (P - 1))
                                                           : -1;
            if (cell[k] >= 0) A.table[cell[k]] = page[k];
        }
        if (V == 4 && vec && row0 + V <= nrows) {
            *reinterpret_cast<int4 *>(A.row_req + row0) =
                make_int4(req[0], req[1 % V], req[2 % V], req[3 % V]);
            *reinterpret_cast<int4 *>(A.row_pos + row0) =
                make_int4(pos[0], pos[1 % V], pos[2 % V], pos[3 % V]);
            *reinterpret_cast<int4 *>(A.slot_map + row0) =
                make_int4(slot[0], slot[1 % V], slot[2 % V], slot[3 % V]);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (row0 + k >= nrows) break;
                A.row_req[row0 + k] = req[k];
                A.row_pos[row0 + k] = pos[k];
                A.slot_map[row0 + k] = slot[k];
            }
        }
    }
    // finished requests: their pages go behind the ring's free ones (places that no row reads)
    for (int r0 = warp * 32; do_rows && r0 < R; r0 += warps * 32) {
        unsigned done = __ballot_sync(0xffffffffu, r0 + lane < R && off[r0 + lane] < -1);
        for (; done; done &= done - 1) {
            const int r = r0 + __ffs(done) - 1;
            const int have = (len[r] + P - 1) >> lgP;
            for (int j0 = lane; j0 < have; j0 += 256) {  // 8 loads of the table on their way at a time
                int page[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    page[k] = j0 + 32 * k < have ? __ldg(A.table + (size_t)r * maxp + j0 + 32 * k) : 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const unsigned at =
                        (unsigned)head + (unsigned)n_free + (unsigned)(-2 - off[r]) + j0 + 32 * k;
                    if (j0 + 32 * k < have) A.free_pages[at % (unsigned)npages] = page[k];
                }
            }
        }
    }
    if (!do_lens) return;
    if (!do_rows) pg_wait_prior();  // the first launch has read the lengths
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
        A.pool_out[1] = (int)min((unsigned)n_free - s_taken + carry.back, (unsigned)npages);
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
    pg_wait_prior();
    pg_launch_dependents();
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

// ---- joining the partial results ---------------------------------------------------------------------
// One warp per (row, query head): with M = max_s m_s over its partial results s (prompt splits, then own
// rows in order), out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s, in that order whatever order they
// were made in. Few rows are bound by latency: which partial results there are is worked out before the
// kernels that make them have ended, and eight are on their way at a time. Many are bound by reading
// them from L2. (A warp for all heads of a KV head, to share the search, was slower: 28 against 22 us
// for 21K rows and heads.)
// What the partial results of a row's heads have in common, read before the kernels that make them have
// ended; `where` then says where those of a head lie: two runs, the prompt's and the own rows', each with its
// first row, the rows from one to the next, and how many there are.
template <bool F32> struct PgFound {
    int r, first, nq, len, cr, nb, pfirst, pcr, pnb;
    int np, nd;  // splits of its prompt and, if dense, of its own rows
    bool mine;   // the row has a place
    bool dense;  // own rows by the tcgen05 kernel: splits of [splits][rows][Hq], like the prompt's
    struct Runs {
        const float *po, *oo;
        const float2 *pm, *om;
        long long prow, pstep, orow, ostep;
        int np, no;
    };
    __device__ __forceinline__ PgFound(const PgDims &D, const PgAttn &A, int tok, bool on) {
        r = on ? __ldg(A.row_req + tok) : -1;
        if (r >= D.R) r = -1;
        int x0, x1;
        int plen = 0;
        len = first = nq = cr = nb = pfirst = pcr = pnb = 0;
        if (r >= 0) {
            const int p = r / D.F;
            pg_unit_entity<F32>(D, A, D.S + r, &len, &first, &nq, &x0, &cr, &nb);
            if (D.line) pg_unit_entity<F32>(D, A, p, &plen, &pfirst, &x0, &x1, &pcr, &pnb);
            else if (!F32) plen = A.plen ? pg_clamp(__ldg(A.plen + p), 0, D.n) : D.n;
        }
        nq = min(nq, D.max_new);
        mine = r >= 0 && tok >= first && tok - first < nq;
        dense = !F32 && (D.prompt_own || pg_on_tc((long long)nq * D.g, len));
        np = D.np == 0 ? 0 : (plen + D.psplit - 1) / D.psplit;
        nd = dense ? (len + D.ssplit - 1) / D.ssplit : 0;
    }
    __device__ __forceinline__ Runs where(const PgDims &D, const PgAttn &A, int tok, int h, int kh) const {
        const int hk = h - kh * D.g;
        const long long row = (long long)tok * D.Hq + h, step = (long long)D.rows * D.Hq;
        Runs x;
        const bool line = F32 || D.line;
        x.po = line ? A.own.o : A.part_o;
        x.oo = dense ? A.part_o : A.own.o;
        x.pm = line ? A.own.ml : A.part_ml;
        x.om = dense ? A.part_ml : A.own.ml;
        x.prow = row;
        x.pstep = step;
        x.orow = D.np * step + row;
        x.ostep = step;
        x.np = np;
        x.no = nd;
        // pieces of a unit: query row rr of entity e
        auto pieces = [&](int e, int rr, int chunks, int blocks, long long *at_row, int *count) {
            const int lg = F32 || pg_unit_rows(D) == 16 ? 4 : 3, u = kh * blocks + (rr >> lg);
            const long long c = A.own.base[e] + (long long)u * chunks, cpw = *A.own.cpw;
            const long long w0 = pg_div(c, cpw), w1 = chunks > 0 ? pg_div(c + chunks - 1, cpw) : w0 - 1;
            const long long at = A.own.unit[e] + u + w0;
            // as many as there are places (all, when the row starts are sums of lengths)
            *count = at < 0 ? 0 : (int)max(min(w1 - w0 + 1, (long long)A.own.segs - at), 0LL);
            *at_row = at * A.own.seg_rows + (rr & ((1 << lg) - 1));
        };
        if (!dense) {
            pieces((line ? D.S : 0) + r, (tok - first) * D.g + hk, cr, nb, &x.orow, &x.no);
            x.ostep = A.own.seg_rows;
        }
        if (D.line) {
            pieces(r / D.F, (tok - pfirst) * D.g + hk, pcr, pnb, &x.prow, &x.np);
            x.pstep = A.own.seg_rows;
        }
        return x;
    }
};

// W: warps per row and head, 1 or all 4 of the block, which then take turns of U results and are joined in
// shared memory, in order.
template <typename T, int D, int U, int W>
__global__ void __launch_bounds__(128) pg_join_kernel(PgDims D_, PgAttn A) {
    constexpr int E = D / 32;
    constexpr bool F32 = sizeof(T) == 4;
    const int tok = blockIdx.x, lane = threadIdx.x & 31, w = W == 1 ? 0 : threadIdx.x >> 5;
    const int h = W == 1 ? blockIdx.y * 4 + (threadIdx.x >> 5) : blockIdx.y;
    const PgFound<F32> at(D_, A, tok, h < D_.Hq);
    const bool mine = at.mine;
    const int kh = h / D_.g;
    const long long row = (long long)tok * D_.Hq + h;
    float M = kPgNoMax, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    pg_wait_prior();
    pg_launch_dependents();
    if (!mine) return;
    const auto x = at.where(D_, A, tok, h, kh);
    const int np = x.np, nsp = np + x.no;
    // U at a time: a running maximum over the groups, in order
    for (int s0 = U * w; s0 < nsp; s0 += U * W) {
        float v[U][E];
        float2 ml[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int s = s0 + j;
            ml[j] = make_float2(kPgNoMax, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) v[j][e] = 0.f;
            if (s < nsp) {
                const long long pr = s < np ? x.prow + s * x.pstep : x.orow + (s - np) * x.ostep;
                const float *o = (s < np ? x.po : x.oo) + pr * D + lane * E;
                ml[j] = (s < np ? x.pm : x.om)[pr];
                if (E == 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(o);
                    v[j][0] = y.x;
                    v[j][1 % E] = y.y;
                    v[j][2 % E] = y.z;
                    v[j][3 % E] = y.w;
                } else if (E == 2) {
                    const float2 y = *reinterpret_cast<const float2 *>(o);
                    v[j][0] = y.x;
                    v[j][1 % E] = y.y;
                } else {
                    v[j][0] = *o;
                }
            }
        }
        float Mn = M;
#pragma unroll
        for (int j = 0; j < U; ++j) Mn = fmaxf(Mn, ml[j].x);
        const float f = exp2f(M - Mn);
        M = Mn;
        L *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float wt = exp2f(ml[j].x - M);
            L = fmaf(wt, ml[j].y, L);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, v[j][e], acc[e]);
        }
    }
    if constexpr (W > 1) {
        __shared__ float part[W][E + 2][32];
        if (w > 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) part[w][e][lane] = acc[e];
            part[w][E][lane] = M;
            part[w][E + 1][lane] = L;
        }
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int x = 1; x < W; ++x) {
            const float mx = part[x][E][lane], Mn = fmaxf(M, mx), f = exp2f(M - Mn), fx = exp2f(mx - Mn);
            M = Mn;
            L = fmaf(fx, part[x][E + 1][lane], L * f);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(fx, part[x][e][lane], acc[e] * f);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    alignas(16) T out[E];
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = from_f<T>(acc[e] * inv);
    T *dst = static_cast<T *>(A.out) + (size_t)row * D + lane * E;
    if (sizeof(out) == 16) *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(out);
    else if (sizeof(out) == 8) *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(out);
    else
#pragma unroll
        for (int e = 0; e < E; ++e) dst[e] = out[e];
    if (A.lse && lane == 0) A.lse[row] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

// The same for many rows of d_head 32 and 64: a warp joins four heads of a row (2 or 4 at a time, 4 columns a
// lane), so that the steps to find their results, which wait for one another, are taken once for four (92K
// rows and heads: 45 -> 22 us with d_head 32; with 128, where the four take turns, it was slower: 15 -> 17).
template <typename T, int D>
__global__ void __launch_bounds__(128) pg_join_many_kernel(PgDims D_, PgAttn A) {
    constexpr bool F32 = sizeof(T) == 4;
    static_assert(D < 128);
    constexpr int LANES = D / 4, PAR = 32 / LANES, N = 4 / PAR;  // lanes per head, heads at a time, turns
    constexpr int U = 8 / N;                                     // results on their way per head
    const int lane = threadIdx.x & 31, sub = lane / LANES, col = lane % LANES * 4;
    const int quads = (D_.Hq + 3) / 4;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int tok = (int)pg_div(w, quads), h0 = (int)(w - (long long)tok * quads) * 4;
    const PgFound<F32> at(D_, A, tok, tok < D_.rows);
    int kh[N];
#pragma unroll
    for (int i = 0; i < N; ++i)  // (heads behind the last: not stored)
        kh[i] = min(h0 + i * PAR + sub, D_.Hq - 1) / D_.g;
    pg_wait_prior();
    pg_launch_dependents();
    if (!at.mine) return;
    typename PgFound<F32>::Runs x[N];
    float M[N], L[N];
    float4 acc[N];
    int most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = at.where(D_, A, tok, min(h0 + i * PAR + sub, D_.Hq - 1), kh[i]);
        most = max(most, x[i].np + x[i].no);
        M[i] = kPgNoMax;
        L[i] = 0.f;
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int s0 = 0; s0 < most; s0 += U) {
        float4 v[N][U];
        float2 ml[N][U];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int s = s0 + j, np = x[i].np;
                v[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                ml[i][j] = make_float2(kPgNoMax, 0.f);
                if (s < np + x[i].no) {
                    const long long r =
                        s < np ? x[i].prow + s * x[i].pstep : x[i].orow + (s - np) * x[i].ostep;
                    v[i][j] = *reinterpret_cast<const float4 *>((s < np ? x[i].po : x[i].oo) + r * D + col);
                    ml[i][j] = (s < np ? x[i].pm : x[i].om)[r];
                }
            }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float Mn = M[i];
#pragma unroll
            for (int j = 0; j < U; ++j) Mn = fmaxf(Mn, ml[i][j].x);
            const float f = exp2f(M[i] - Mn);
            M[i] = Mn;
            L[i] *= f;
            acc[i] = make_float4(acc[i].x * f, acc[i].y * f, acc[i].z * f, acc[i].w * f);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const float wt = exp2f(ml[i][j].x - Mn);
                L[i] = fmaf(wt, ml[i][j].y, L[i]);
                acc[i] = make_float4(fmaf(wt, v[i][j].x, acc[i].x), fmaf(wt, v[i][j].y, acc[i].y),
                                     fmaf(wt, v[i][j].z, acc[i].z), fmaf(wt, v[i][j].w, acc[i].w));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int h = h0 + i * PAR + sub;
        if (h >= D_.Hq) continue;
        const float inv = L[i] > 0.f ? 1.f / L[i] : 0.f;
        alignas(16) T out[4] = {from_f<T>(acc[i].x * inv), from_f<T>(acc[i].y * inv),
                                from_f<T>(acc[i].z * inv), from_f<T>(acc[i].w * inv)};
        const long long row = (long long)tok * D_.Hq + h;
        T *dst = static_cast<T *>(A.out) + row * D + col;
        if (sizeof(out) == 16) *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(out);
        else *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(out);
        if (A.lse && col == 0) A.lse[row] = L[i] > 0.f ? (M[i] + log2f(L[i])) * kLn2 : -INFINITY;
    }
}

template <typename T, int D> cudaError_t join_d(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    // few rows: all warps of a block for one, 8 partial results on their way in each (lookahead over 32K
    // rows of fp32, 152 pieces a row: the join 20 -> 12 us); many: fewer instructions
    const bool alone = (long long)D_.rows * D_.Hq <= kPgSms * 8;
    const bool few = (long long)D_.rows * D_.Hq < kPgSms * 32;
    auto kern = pg_join_kernel<T, D, 8, 1>;
    if constexpr (D < 128) {
        if (!few) {
            const long long warps = (long long)D_.rows * ((D_.Hq + 3) / 4);
            return pg_launch(pg_join_many_kernel<T, D>, (unsigned)((warps + 3) / 4), 128, 0, true, st, D_,
                             A);
        }
    } else {
        if (!few) kern = pg_join_kernel<T, D, 4, 1>;
    }
    if (alone) kern = pg_join_kernel<T, D, 8, 4>;
    return pg_launch(kern, dim3(D_.rows, alone ? D_.Hq : (D_.Hq + 3) / 4), 128, 0, true, st, D_, A);
}

template <typename T> cudaError_t join(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.d == 128 ? join_d<T, 128>(D, A, st)
                      : (D.d == 64 ? join_d<T, 64>(D, A, st) : join_d<T, 32>(D, A, st));
}

}  // namespace

// ---- launchers -----------------------------------------------------------------------------------
cudaError_t launch_pg_plan(const PgDims &D, const PgPlanArgs &A, cudaStream_t st) {
    // one warp for the smallest steps (no barrier to wait for), up to 1024 threads; above 4096 rows a
    // CTA per 2048, on all SMs, and a second launch for the lengths (256K rows of 256 requests: one CTA
    // 119 us, 8 of a cluster 21 us)
    const int work = D.R > D.rows ? D.R : D.rows;
    int threads = 32;
    while (threads < 1024 && threads < work) threads <<= 1;
    const bool many = D.rows > 4096;
    int ctas = many ? (D.rows + 2047) / 2048 : 1;
    if (ctas > kPgSms) ctas = kPgSms;
    const bool vec = (reinterpret_cast<uintptr_t>(A.row_req) | reinterpret_cast<uintptr_t>(A.row_pos) |
                      reinterpret_cast<uintptr_t>(A.slot_map)) % 16 == 0;
    // (small steps do without a change of the limit, a call into the driver)
    const size_t bytes = 3 * sizeof(int) * (size_t)D.R;
    const PgSmem smem(bytes, bytes > 40 * 1024 ? 3 * sizeof(int) * 16384 : bytes);
    auto go = [&](auto kern, int grid, int block, bool rows, bool lens) {
        return pg_launch(kern, grid, block, smem, true, st, A, D.R, D.lgP, D.npages, D.maxp, D.rows,
                         D.max_new, vec, rows, lens);
    };
    if (D.rows <= 1024) return go(pg_plan_kernel<1>, 1, threads, true, true);
    cudaError_t e = go(pg_plan_kernel<4>, ctas, threads, true, !many);
    int few = 32;
    while (few < 1024 && few < D.R) few <<= 1;
    return e == cudaSuccess && many ? go(pg_plan_kernel<1>, 1, few, false, true) : e;
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
    return pg_launch(pg_append_kernel, (unsigned)blocks, 256, 0, true, st,
                     static_cast<const uint4 *>(K_new), static_cast<const uint4 *>(V_new),
                     k_row * es / 16, v_row * es / 16, slots, static_cast<uint4 *>(K),
                     static_cast<uint4 *>(V), D.rows, D.Hkv, lgv, D.lgP, D.npages << D.lgP, err);
}

cudaError_t launch_pg_own(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    if (D.dtype == KVE_F32) return launch_pg_f32(D, A, st);
    if (D.prompt_own) return cudaSuccess;
    const cudaError_t e = launch_pg_own16(D, A, st);
    return e == cudaSuccess && D.ns > 0 ? launch_pg_own_tc(D, A, st) : e;
}

cudaError_t launch_pg_join(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    if (D.dtype == KVE_F32) return join<float>(D, A, st);
    return D.dtype == KVE_BF16 ? join<__nv_bfloat16>(D, A, st) : join<__half>(D, A, st);
}

}  // namespace kve
