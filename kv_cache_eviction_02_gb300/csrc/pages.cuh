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
    int np, psplit;            // prompt splits and their tokens (0 without a prompt)
    int ns, ssplit;            // fp32: splits of a request's own rows and their tokens
    int own_sms;               // 16-bit types: SMs for the own rows' kernel
    // rows behind one prompt, when no request packs more than max_new
    __host__ __device__ long long group_rows() const {
        return (long long)F * max_new < rows ? (long long)F * max_new : rows;
    }
    __host__ __device__ int cap() const { return maxp * P; }
};

constexpr int kPgSms = 152;    // GB300
constexpr int kPgShare = 100;  // most SMs the prompt's kernel takes beside the own rows' one

// Own rows of 16-bit types: units of 8 or 16 query rows, chunks of 16 tokens (pages_own.cu).
constexpr int kPgChunk = 16, kPgOwnWarps = 4;

// Workspace carve-up (byte offsets, 256-aligned): partial results [splits][rows][Hq] (m in log2 and l;
// o [d] fp32) over the prompt and, fp32 only, over the own rows' splits; 16-bit types: the pieces of
// own rows [segs][seg_rows], with what the join needs to find them.
struct PgWorkspace {
    size_t part_ml, part_o;
    size_t own_ml, own_o, own_base, own_unit, own_cpw;
    size_t total;
};

bool pg_dims(const KvePgShape *sh, PgDims *D, const char **why);
PgWorkspace pg_ws_layout(const PgDims &D);

// The prompt's kernel on tcgen05 (16-bit types): new rows per 128-row tile (whole groups of query
// heads), and row tiles per CTA. Two tiles share one K/V stream and take turns on the tensor pipe; an
// odd small number of tiles runs one per CTA, since a half-empty pair would leave the pipe idle in its
// turn.
inline int pg_tile_rows(const PgDims &D) { return 128 / D.g; }
inline int pg_prompt_pairs(const PgDims &D) {
    const long long tiles = (D.group_rows() + pg_tile_rows(D) - 1) / pg_tile_rows(D);
    return tiles % 2 == 0 || tiles >= 9 ? 2 : 1;
}
// Query rows of a unit of own rows: 8 when no request has more, else 16 (the rows of a unit share its
// K/V loads; more than 16 would not leave registers for two blocks per SM).
__host__ __device__ inline int pg_unit_rows(const PgDims &D) {
    return (long long)D.max_new * D.g <= 8 ? 8 : 16;
}
// Rows of a unit that can hold a query, CTAs of the own rows' kernel (two per SM, fewer when the tables
// cannot hold a chunk for each warp), and the places its pieces need.
inline int pg_seg_rows(const PgDims &D) {
    const long long rows = (long long)D.max_new * D.g;
    return rows < pg_unit_rows(D) ? (int)rows : pg_unit_rows(D);
}
inline int pg_own_ctas(const PgDims &D) {
    const int rb = pg_unit_rows(D);
    const long long units = (long long)D.R * D.Hkv * (((long long)D.max_new * D.g + rb - 1) / rb);
    const long long ctas = (units * ((D.cap() + kPgChunk - 1) / kPgChunk) + kPgOwnWarps - 1) /
                           kPgOwnWarps;
    return (int)(ctas < 2 * D.own_sms ? ctas : 2 * D.own_sms);
}
inline long long pg_own_segs(const PgDims &D) {
    const long long busy = D.R < D.rows ? D.R : D.rows;
    return D.Hkv * ((long long)D.rows * D.g / pg_unit_rows(D) + busy) +
           (long long)pg_own_ctas(D) * kPgOwnWarps;
}

// Where the own rows' pieces lie: request r's chunks start at base[r] in the line of all chunks and its
// units at unit[r]; every warp has cpw chunks; the piece of unit u that warp w saw is at place u + w,
// seg_rows rows each.
struct PgOwn {
    float2 *ml;
    float *o;
    long long *base, *cpw;
    int *unit;
    long long segs;
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
cudaError_t launch_pg_own16(const PgDims &D, const PgAttn &A, cudaStream_t st);
// Tensor map of a 16-bit array: rank dims, strides (elements) of all but the innermost, a box of at
// most 128 bytes (swizzled by 128, or by 64 bytes) in the innermost.
bool pg_tmap(CUtensorMap *map, bool f16, const void *base, int rank, const cuuint64_t *dims,
             const long long *strides, const cuuint32_t *box, bool swizzle64);
// the three stages of pg_attention: partial results over the prompt, over the requests' own rows, and
// their join
cudaError_t launch_pg_prompt(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_own(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_join(const PgDims &D, const PgAttn &A, cudaStream_t st);

constexpr float kPgNoMax = -3e38f;  // running maximum before any visible token

// ---- device helpers --------------------------------------------------------------------------------
// The device arrays are the caller's: every index read from them is brought into range before it
// becomes an address.
__device__ __forceinline__ int pg_clamp(int v, int lo, int hi) { return min(max(v, lo), hi); }

__device__ __forceinline__ int pg_start(const int32_t *q_start, int r, int rows) {
    return pg_clamp(__ldg(q_start + r), 0, rows);
}

// A request's own rows: how many lie in its pages, its packed rows, and (16-bit types) its chunks per
// unit and its row blocks. Rows beyond max_new have no place.
__device__ __forceinline__ void pg_own_request(const PgDims &D, const PgAttn &A, int r, int *len,
                                               int *first, int *nq, int *cr, int *nb) {
    *len = pg_clamp(__ldg(A.len + r), 0, D.cap());
    *first = pg_start(A.q_start, r, D.rows);
    *nq = max(0, pg_start(A.q_start, r + 1, D.rows) - *first);
    *cr = (*len + kPgChunk - 1) / kPgChunk;
    const int rb = pg_unit_rows(D);
    *nb = (min(*nq, D.max_new) * D.g + rb - 1) / rb;
}

// Programmatic dependent launch: a dependent kernel of the same call may start when every block of the
// one before it has called pg_launch_dependents(), and reads its results after pg_wait_prior(). Every
// block of a dependent kernel calls pg_wait_prior() before it ends, so its own end implies the end of
// the kernel before it, and what follows in the stream waits for all of the call.
__device__ __forceinline__ void pg_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pg_wait_prior() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
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

// Launches `kern` on `st`, as a dependent of the kernel before it if asked. All of these kernels ask for
// the same split of the SM's memory (all of it shared memory): an SM changes its split only when it is
// empty, so kernels that differ in it could not overlap, and with the default split the own rows' kernel
// found room for one block on some SMs and ran in two waves (35 instead of 22 us for 64 answers).
template <typename... P, typename... Q>
cudaError_t pg_launch(void (*kern)(P...), unsigned grid, unsigned block, size_t smem, bool dependent,
                      cudaStream_t st, Q &&...args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = dependent ? 1 : 0;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess && smem > 48 * 1024)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

}  // namespace kve
