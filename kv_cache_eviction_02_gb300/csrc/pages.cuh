// Shared-prompt decoding: internal declarations of the page planner, the paged append and the
// attention over one shared prompt cache plus each request's own pages (pages*.cu).
#pragma once

#include <cuda.h>

#include "kve_internal.cuh"

namespace kve {

// Sizes of one call (KvePgShape) and how its attention is split.
struct PgDims {
    int S, F, R;               // prompts, requests per prompt, requests
    int Hq, Hkv, g, d;
    int n;                     // prompt rows held per (prompt, KV head)
    int P, lgP, npages, maxp;  // page size (a power of two), pages in the pool, table width
    int rows, max_new, dtype;
    int np, psplit;            // 16-bit types: prompt splits and their tokens (0 without a prompt)
    int ns, ssplit;            // pg_many_new: splits of a request's own rows and their tokens
    int own_sms;               // SMs for the kernel that deals out units
    bool line;                 // that kernel takes the prompts too (fp32; 16-bit types: short work)
    bool direct;               // it does all, a warp per request and KV head
    bool prompt_own;           // the prompt's kernel does the own rows too (split np)
    // rows behind one prompt, when no request packs more than max_new
    __host__ __device__ long long group_rows() const {
        return (long long)F * max_new < rows ? (long long)F * max_new : rows;
    }
    __host__ __device__ int cap() const { return maxp * P; }
};

constexpr int kPgSms = 152;    // GB300
// A prompt kernel of fewer CTAs than this has its SMs left out of the own rows' grid (pg_split). Grid over the SMs
// left, and over all, us (32/8 heads of d 128, bf16; prompt CTAs in brackets): 64 requests of up to 1023 own rows
// behind 164 rows 36.1 and 43.0 [16], behind 512 36.4 and 42.9 [32], behind 1000 39.6 and 44.5 [64]; 64 of up to
// 255 behind 1000 20.6 and 22.6 [64]; but 256 of up to 1023 behind 164 105 and 107 [64], behind 300 129 and 109
// [96], 2 x 213 behind 10 rows (40/8 heads) 177 and 168 [80]: with own rows for much longer than the prompt the SMs
// left out are missed. Few requests (16) and other prompts: within 5 % of one another. (A rule by the two
// kernels' times instead of one number would take both.)
constexpr int kPgShare = 100;

// Units of 8 or 16 query rows (fp32: 16), chunks of 16 tokens, dealt out to the warps of pages_own.cu
// (16-bit types) or pages_f32.cu.
constexpr long long kPgDirectMost = 1 << 20;  // most chunks of a call without partial results
constexpr int kPgChunk = 16, kPgOwnWarps = 4, kPgF32Warps = 8, kPgF32Rows = 16;

// Workspace carve-up (byte offsets, 256-aligned): partial results [splits][rows][Hq] (m in log2 and l;
// o [d] fp32) over the prompt and over the own rows of requests with many new rows; the pieces of units
// [segs][seg_rows], with what the join needs to find them.
struct PgWorkspace {
    size_t part_ml, part_o;
    size_t own_ml, own_o, own_base, own_unit, own_cpw;
    size_t total;
};

bool pg_dims(const KvePgShape *sh, PgDims *D, const char **why);
PgWorkspace pg_ws_layout(const PgDims &D);

// The kernel on tcgen05 (16-bit types): new rows per 128-row tile (whole groups of query heads), and row
// tiles per CTA for `rows` new rows. Two tiles share one K/V stream and take turns on the tensor pipe; an
// odd small number of tiles runs one per CTA, since a half-empty pair would leave the pipe idle in its
// turn.
inline int pg_tile_rows(const PgDims &D) { return 128 / D.g; }
inline int pg_pairs(const PgDims &D, long long rows) {
    const long long tiles = (rows + pg_tile_rows(D) - 1) / pg_tile_rows(D);
    return tiles % 2 == 0 || tiles >= 9 ? 2 : 1;
}
// Row blocks (one or two tiles) that the launch has places for, per prompt or request: as many as it can
// have, and no more than four times its even share (with max_new far above what most requests add, nearly
// all of them would come to nothing).
inline int pg_tc_blocks(const PgDims &D, bool own) {
    const long long rows = own ? D.max_new : D.group_rows(), of = own ? D.R : D.S;
    const long long per = (long long)pg_tile_rows(D) * pg_pairs(D, rows);
    const long long most = (rows + per - 1) / per, share = 4 * ((D.rows + per * of - 1) / (per * of));
    return (int)(most < share ? most : share);
}
// A request with more query rows per KV head than kPgFewRows (the warps of pages_own.cu would read its K/V
// more than twice) and more than kPgFewScores scores has its own rows done on tcgen05, where a CTA costs
// several microseconds whatever it does; the others go to pages_own.cu. The choice is made per request on
// the device, so a batch of both runs both kernels. On tcgen05, and by warps, us, of whole calls behind 1000 rows
// (bf16, up to `new` new rows): 32/8 heads of d 128, 64 requests: new 16 and 256 own rows (17K scores at
// most) 69 and 58, 32 and 64 (12K) 72 and 69, 32 and 256 (37K) 89 and 92, 64 and 64 (33K) 118 and 130, 64 and 512
// (147K) 152 and 223; 40/8 of d 64: 9 and 256 (12K) 45 and 40, 16 and 128 (12K) 46 and 47, 32 and 64 (15K)
// 66 and 72, 32 and 512 (87K) 93 and 131. Eight requests alone are better off with warps until about 40K scores
// (32/8 heads, 9 and 512: 28 and 19; 32 and 128: 25 and 25; 64 and 512: 36 and 45). With at most 32 query rows
// tcgen05 is never ahead (64 requests of up to 8 new rows, 32/8 heads: 1024 own rows 104 and 95, 4096 278 and 278;
// of 4, 8/1 heads: 4096 own rows 67 and 48); with 64 it is (8 new rows, 8/1 heads, 4096: 71 and 82).
constexpr int kPgFewRows = 32, kPgFewScores = 12288;
__host__ __device__ inline bool pg_on_tc(long long rows, int len) {
    return rows > kPgFewRows && rows * len > kPgFewScores;
}
__host__ __device__ inline bool pg_many_new(const PgDims &D) {
    return D.dtype != KVE_F32 && pg_on_tc((long long)D.max_new * D.g, D.cap());
}

// Tables of at most this many rows behind a prompt of a 16-bit type (the lookahead's trajectories): two idle
// warps of the prompt's kernel work out the own rows, a launch less (16K lookahead step: with a kernel of their
// own 23.3 us, in the join, which cannot start beside the prompt's CTAs, 20.5, so 16.4).
constexpr int kPgFewOwn = 32;
// Query rows of a unit: 8 when no request has more, else 16 (the rows of a unit share its K/V loads; more
// than 16 would not leave registers for two blocks per SM).
__host__ __device__ inline int pg_unit_rows(const PgDims &D) {
    return D.dtype != KVE_F32 && (long long)D.max_new * D.g <= 8 ? 8 : 16;
}
// 16-bit types: the warps of pages_own.cu take the prompts too when all there is to do is short, so that a
// call has one launch less and no tcgen05 kernel, which costs several microseconds whatever it does (a step of
// 4 requests behind 11 rows 12.0 -> 8.7 us); not with long own rows, where the prompt's kernel
// hides behind them (172 requests of up to 268 own rows, 23K chunks: 26.7 us, in one line 24.6; 64 of up to
// 1875, 60K: 54 and 59). The prompt's kernel, and one line, by the prompt's rows (32/8 heads of d 128, up to 60 own
// rows): 4 requests 128 rows 8.8 and 7.5, 256 9.0 and 8.3, 400 9.6 and 9.5, 700 9.9 and 11.5; 64 requests 128
// 15.9 and 13.0, 256 15.9 and 15.1, 400 16.3 and 18.6. By the prompts' chunks (250 rows, 8 requests each): 512 11.1
// and 9.5, 2048 13.4 and 13.1, 4096 19.1 and 16.9, 8192 25.5 and 27.5.
inline bool pg_short_prompts(const PgDims &D) {
    const int rb = pg_unit_rows(D);
    auto chunks = [&](long long of, long long rows, int tokens) {  // at most
        return of * D.Hkv * ((rows * D.g + rb - 1) / rb) * ((tokens + kPgChunk - 1) / kPgChunk);
    };
    return D.n <= 256 && chunks(D.S, D.group_rows(), D.n) <= 2048 &&
           chunks(D.R, D.max_new, D.cap()) <= 24576;
}
// Very short work of 16-bit types: a warp takes all that a block of query rows of one request and KV head sees,
// prompt and own rows, and writes the output, so a call is one launch without partial results (183 requests
// behind 11 rows, up to 16 own ones: 16.8 -> 7.3 us; 687 of up to 57 new rows behind 2 rows 361 -> 168). A lone
// warp takes 0.5 to 0.8 us a chunk of d_head 128, half that of 64 and 32, and two launches 9 us: 8 requests of up
// to 143 own rows 9.0 us, so 12.0; more warps than the SMs hold hide that (253 requests of up to 157 own rows 61
// -> 38 us; 256 with 200 and 121 rows, 24 chunks, 33 and 34). (With fp32, 1.2 us a chunk and more, it paid for
// next to nothing.)
__host__ __device__ inline int pg_direct_blocks(const PgDims &D) {  // row blocks per request and KV head
    const int rb = pg_unit_rows(D);
    return (int)(((long long)D.max_new * D.g + rb - 1) / rb);
}
inline bool pg_direct(const PgDims &D) {
    const long long chunks = (D.n + kPgChunk - 1) / kPgChunk + (D.cap() + kPgChunk - 1) / kPgChunk;
    const long long units = (long long)D.R * D.Hkv * pg_direct_blocks(D);
    const int most = units > kPgSms * 12 ? 20 : (D.d == 128 ? 7 : 11);
    return D.dtype != KVE_F32 && chunks <= most && units * chunks <= kPgDirectMost;
}
// Rows of a unit that can hold a query, CTAs of the kernel that deals out units (three per SM, two for units
// of 16 rows, fp32 one; fewer when there cannot be a chunk for each warp), and the places its pieces need.
inline int pg_seg_rows(const PgDims &D) {
    // (a prompt's rows may be all there are: a refused request can pack more than max_new)
    const long long rows = (long long)(D.line ? D.rows : D.max_new) * D.g;
    return rows < pg_unit_rows(D) ? (int)rows : pg_unit_rows(D);
}
inline int pg_own_ctas(const PgDims &D) {
    if (D.direct) return (D.R * D.Hkv * pg_direct_blocks(D) + kPgOwnWarps - 1) / kPgOwnWarps;
    const int rb = pg_unit_rows(D);
    long long rows = (long long)D.max_new * D.g;
    long long chunks =
        (long long)D.R * D.Hkv * ((rows + rb - 1) / rb) * ((D.cap() + kPgChunk - 1) / kPgChunk);
    if (D.line)
        chunks += (long long)D.S * D.Hkv * ((D.group_rows() * D.g + rb - 1) / rb) *
                  ((D.n + kPgChunk - 1) / kPgChunk);
    const int warps = D.dtype == KVE_F32 ? kPgF32Warps : kPgOwnWarps;
    const long long ctas = (chunks + warps - 1) / warps, most = D.own_sms * (D.dtype == KVE_F32 ? 1 : (rb == 8 ? 3 : 2));
    return (int)(ctas < most ? ctas : most);
}
inline long long pg_own_segs(const PgDims &D) {
    const long long busy = D.R < D.rows ? D.R : D.rows;
    long long units = D.Hkv * ((long long)D.rows * D.g / pg_unit_rows(D) + busy);
    if (D.line || D.dtype == KVE_F32)  // (fp32: without a prompt they are counted all the same, with no chunks)
        units += D.Hkv * ((long long)D.rows * D.g / pg_unit_rows(D) + (D.S < D.rows ? D.S : D.rows));
    return units + (long long)pg_own_ctas(D) * (D.dtype == KVE_F32 ? kPgF32Warps : kPgOwnWarps);
}

// Where the pieces lie: the chunks of entity e (request e; with the prompts in the line prompt e, then request
// e - S; fp32 always) start at base[e] in the line of all chunks and its units at unit[e]; every warp has cpw chunks; the piece of
// unit u that warp w saw is at place u + w, seg_rows rows each.
struct PgOwn {
    float2 *ml;
    float *o;
    long long *base, *cpw;
    int *unit;
    unsigned long long segs;
    int seg_rows;
};

// Device pointers of one attention call. Strides in elements.
struct PgAttn {
    const void *q;
    long long q_row;
    const void *Kp, *Vp;
    long long p_prompt, p_head, p_tok;
    const int32_t *plen;  // may be null: every prompt has D.n rows
    const void *K, *V;
    const int32_t *table, *len, *q_start, *row_req;
    void *out;
    float *lse;  // may be null
    float2 *part_ml;
    float *part_o;
    PgOwn own;
    unsigned *err;
};

struct PgPlanArgs {
    const int32_t *new_len, *len_in, *pool_in;
    int32_t *free_pages, *table, *len_out, *pool_out, *q_start, *row_req, *row_pos, *slot_map;
};

cudaError_t launch_pg_plan(const PgDims &D, const PgPlanArgs &A, cudaStream_t st);
cudaError_t launch_pg_append(const PgDims &D, const void *K_new, const void *V_new,
                             long long k_row, long long v_row, const int32_t *slots, void *K,
                             void *V, unsigned *err, cudaStream_t st);
cudaError_t launch_pg_prompt_tc(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_own_tc(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_f32(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_own16(const PgDims &D, const PgAttn &A, cudaStream_t st);
// Tensor map of a 16-bit array: rank dims, strides (elements) of all but the innermost, a box of
// 128 bytes in the innermost, 128-byte swizzle. Boxes land on multiples of 128 bytes.
bool pg_tmap(CUtensorMap *map, bool f16, const void *base, int rank, const cuuint64_t *dims,
             const long long *strides, const cuuint32_t *box);
// the stages of pg_attention: partial results over the prompt (16-bit types: launch_pg_prompt_tc), over
// the requests' own rows (fp32: and over the prompt), and their join
cudaError_t launch_pg_own(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_join(const PgDims &D, const PgAttn &A, cudaStream_t st);

constexpr float kPgNoMax = -3e38f;  // running maximum before any visible token

// 16-bit types: a row is rescaled when its maximum has grown by 2^kPgRescale, so weights reach that. fp16
// weights are carried kPgHalfUp powers of two higher (its largest number is just below 2^16): a weight is
// then off by half a step or, below 2^-21 of the largest, by 2^-32 of it, where 2^-25 would let many small
// ones vanish together. The reference stored as m is lower by as much.
constexpr float kPgRescale = 8.f, kPgHalfUp = 7.f;

// ---- device helpers --------------------------------------------------------------------------------
// The device arrays are the caller's: every index read from them is brought into range before it
// becomes an address.
__device__ __forceinline__ int pg_clamp(int v, int lo, int hi) { return min(max(v, lo), hi); }

__device__ __forceinline__ int pg_start(const int32_t *q_start, int r, int rows) {
    return pg_clamp(__ldg(q_start + r), 0, rows);
}

// An entity of the line of units: prompt e < S with the rows of all its requests, or request e - S: its
// tokens, first packed row, packed rows, query rows per KV head that have a place (a request: not those beyond
// max_new), chunks per unit and row blocks (none for what runs on tcgen05).
template <bool F32>
__device__ __forceinline__ void pg_unit_entity(const PgDims &D, const PgAttn &A, int e, int *len,
                                               int *first, int *nq, int *rows, int *cr, int *nb) {
    const bool own = e >= D.S;
    const int r0 = own ? e - D.S : e * D.F, r1 = own ? r0 + 1 : r0 + D.F;
    if (own) *len = pg_clamp(__ldg(A.len + r0), 0, D.cap());
    else *len = A.plen ? pg_clamp(__ldg(A.plen + e), 0, D.n) : D.n;
    *first = pg_start(A.q_start, r0, D.rows);
    *nq = max(0, pg_start(A.q_start, r1, D.rows) - *first);
    *rows = (own ? min(*nq, D.max_new) : *nq) * D.g;
    *cr = (*len + kPgChunk - 1) / kPgChunk;
    const int lg = F32 || pg_unit_rows(D) == 16 ? 4 : 3;
    *nb = *cr > 0 ? (*rows + (1 << lg) - 1) >> lg : 0;  // (without tokens no units: warps step over it)
    if (!F32 && (own ? pg_on_tc(*rows, *len) : !D.line)) *nb = 0;
}

// Where a warp stands in the line of chunks.
template <bool F32> struct PgCursor {
    int e, len, first, rows, nq;  // entity, its tokens, its first packed row, its query rows per KV head
    int cr, nb;                   // chunks per unit, row blocks
    int kh, rb, c;                // KV head, row block, chunk of the unit
    __device__ __forceinline__ void enter(const PgDims &D, const PgAttn &A, int entity) {
        e = entity;
        pg_unit_entity<F32>(D, A, e, &len, &first, &nq, &rows, &cr, &nb);
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

__device__ __forceinline__ long long pg_div(long long a, long long b) {  // of non-negative numbers
    if (((unsigned long long)(a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
    return a / b;
}

// Equal shares of the line of chunks. All threads of the block: sums chunks and units of n entities
// (thread t of q consecutive ones; csum[t], usum[t]: those before its), shares the chunks out evenly over
// the launch's warps, and lets block 0 write down what the join needs. A share is at least a 16th of the
// longest unit, up to 4 chunks: smaller ones would leave more pieces to join than they save.
struct PgShare {
    long long total, cpw;  // chunks in all, chunks per warp
    int q;                 // entities per thread
};
template <int THREADS, typename F>
__device__ __forceinline__ PgShare pg_share(int n, int Hkv, long long *csum, int *usum,
                                            const PgOwn &W, F entity) {
    const int lane = threadIdx.x & 31, q = (n + THREADS - 1) / THREADS;
    const int a = min(n, (int)threadIdx.x * q), z = min(n, a + q);
    long long cs = 0;
    int us = 0, longest = 0;
    for (int e = a; e < z; ++e) {
        int cr, nb;
        entity(e, &cr, &nb);
        cs += (long long)cr * nb * Hkv;
        us += nb * Hkv;
        if (nb > 0) longest = max(longest, cr);
    }
    __shared__ int s_longest;
    if (threadIdx.x == 0) s_longest = 0;
    csum[threadIdx.x + 1] = cs;
    usum[threadIdx.x + 1] = us;
    if (threadIdx.x == 0) {
        csum[0] = 0;
        usum[0] = 0;
    }
    __syncthreads();
    atomicMax(&s_longest, longest);
    constexpr int K = THREADS / 32;
    if (threadIdx.x < 32) {  // lane l scans entries K l + 1 .. K l + K
        long long c4[K], ct = 0;
        int u4[K], ut = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            c4[i] = ct += csum[K * lane + 1 + i];
            u4[i] = ut += usum[K * lane + 1 + i];
        }
        long long cb = ct;
        int ub = ut;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, cb, o);
            const int y = __shfl_up_sync(0xffffffffu, ub, o);
            if (lane >= o) {
                cb += x;
                ub += y;
            }
        }
#pragma unroll
        for (int i = 0; i < K; ++i) {
            csum[K * lane + 1 + i] = cb - ct + c4[i];
            usum[K * lane + 1 + i] = ub - ut + u4[i];
        }
    }
    __syncthreads();
    PgShare s;
    s.total = csum[THREADS];
    s.q = q;
    const int nw = gridDim.x * (THREADS / 32);
    s.cpw = max(max(1LL, pg_div(s.total + nw - 1, nw)), min(4LL, (s_longest + 15) / 16LL));
    if (blockIdx.x == 0) {
        cs = csum[threadIdx.x];
        us = usum[threadIdx.x];
        for (int e = a; e < z; ++e) {
            int cr, nb;
            entity(e, &cr, &nb);
            W.base[e] = cs;
            W.unit[e] = us;
            cs += (long long)cr * nb * Hkv;
            us += nb * Hkv;
        }
        if (threadIdx.x == 0) *W.cpw = s.cpw;
    }
    return s;
}
// The first entity of the group that holds chunk X, X counted from there, and the units before it.
template <int THREADS>
__device__ __forceinline__ void pg_share_find(const long long *csum, const int *usum,
                                              const PgShare &s, long long X, int *e, long long *x,
                                              int *unit) {
    constexpr int K = THREADS / 32;
    const int lane = threadIdx.x & 31;
    int grp = 0;  // the last with csum <= X
#pragma unroll
    for (int i = 0; i < K; ++i)
        grp += __popc(__ballot_sync(0xffffffffu, csum[K * lane + 1 + i] <= X));
    *e = grp * s.q;
    *x = X - csum[grp];
    *unit = usum[grp];
}

// E consecutive columns of a row of K, V or q (E = 4: 8 bytes of a 16-bit type).
template <typename T, int E> __device__ __forceinline__ void row_cols(const T *p, float (&v)[E]) {
    if (sizeof(T) * E == 8) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
        const T *y = reinterpret_cast<const T *>(&x);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = to_f(y[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = to_f(__ldg(p + e));
    }
}

// Programmatic dependent launch: a dependent kernel of the same call may start when every block of the
// one before it has called pg_launch_dependents(), and reads its results after pg_wait_prior(). Of a
// kernel that reads nothing of the one before it the last block waits all the same before it ends, so its
// own end implies the end of the kernel before it, and what follows in the stream waits for all of the
// call. (The other blocks leave their SMs to the next ones.)
__device__ __forceinline__ void pg_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pg_wait_prior() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void pg_end_after_prior() {
    if (blockIdx.x == gridDim.x - 1) pg_wait_prior();
}

// A page id of the caller's table; one outside the pool is recorded and read as page 0.
__device__ __forceinline__ int pg_page_id(int page, int npages, unsigned *err) {
    if ((unsigned)page >= (unsigned)npages) {
        atomicOr(err, KVE_DEVERR_BADPAGE);
        page = 0;
    }
    return page;
}
// The page that holds own row `pos` of a request.
__device__ __forceinline__ int pg_page(const int32_t *trow, int pos, int lgP, int npages,
                                       unsigned *err) {
    return pg_page_id(__ldg(trow + (pos >> lgP)), npages, err);
}

// Dynamic shared memory of a launch, and the most that any launch of its kernel takes. A kernel's limit is one
// for all threads of the process: set to what the launch at hand takes, it would fail the larger launch of another
// thread that stands between its own setting and its launch.
struct PgSmem {
    size_t bytes, most;
    PgSmem(size_t bytes) : bytes(bytes), most(bytes) {}
    PgSmem(size_t bytes, size_t most) : bytes(bytes), most(most) {}
};

// Launches `kern` on `st`, as a dependent of the kernel before it if asked.
template <typename... P, typename... Q>
cudaError_t pg_launch(void (*kern)(P...), dim3 grid, unsigned block, PgSmem smem, bool dependent,
                      cudaStream_t st, Q &&...args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem.bytes;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = dependent ? 1 : 0;
    if (smem.most > 40 * 1024) {  // with the static arrays above 48 KB
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem.most);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

}  // namespace kve
