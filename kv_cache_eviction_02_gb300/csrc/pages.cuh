// Shared-prompt decoding: internal declarations of the page planner, the paged append and the
// attention over one shared prompt cache plus each request's own pages (pages*.cu).
#pragma once

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
    int ns, ssplit;            // splits of a request's own rows and their tokens
    // rows behind one prompt, when no request packs more than max_new
    __host__ __device__ long long group_rows() const {
        return (long long)F * max_new < rows ? (long long)F * max_new : rows;
    }
    __host__ __device__ int cap() const { return maxp * P; }
};

struct PgWorkspace {
    size_t part_ml, part_o;  // [np + ns][rows][Hq] float2 (m in log2, l) and [..][d] fp32
    size_t total;
};

bool pg_dims(const KvePgShape *sh, PgDims *D, const char **why);
PgWorkspace pg_ws_layout(const PgDims &D);

// The prompt's kernel on tcgen05 takes 16-bit types and d_head 64 or 128: new rows per 128-row tile
// (whole groups of query heads), and row tiles per CTA. Two tiles share one K/V stream and take turns
// on the tensor pipe; an odd small number of tiles runs one per CTA, since a half-empty pair would
// leave the pipe idle in its turn.
inline bool pg_prompt_tc(const PgDims &D) { return D.dtype != KVE_F32 && D.d >= 64; }
inline int pg_tile_rows(const PgDims &D) { return 128 / D.g; }
inline int pg_prompt_pairs(const PgDims &D) {
    const long long tiles = (D.group_rows() + pg_tile_rows(D) - 1) / pg_tile_rows(D);
    return tiles % 2 == 0 || tiles >= 9 ? 2 : 1;
}

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
cudaError_t launch_pg_prompt_mma(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_own_mma(const PgDims &D, const PgAttn &A, cudaStream_t st);
cudaError_t launch_pg_attention(const PgDims &D, const PgAttn &A, cudaStream_t st);

constexpr float kPgNoMax = -3e38f;  // running maximum before any visible token

// ---- device helpers --------------------------------------------------------------------------------
// The device arrays are the caller's: every index read from them is brought into range before it
// becomes an address.
__device__ __forceinline__ int pg_clamp(int v, int lo, int hi) { return min(max(v, lo), hi); }

__device__ __forceinline__ int pg_start(const int32_t *q_start, int r, int rows) {
    return pg_clamp(__ldg(q_start + r), 0, rows);
}

// The page that holds own row `pos` of a request; an id outside the pool is recorded and read as
// page 0.
__device__ __forceinline__ int pg_page(const int32_t *trow, int pos, int lgP, int npages,
                                       unsigned *err) {
    int page = __ldg(trow + (pos >> lgP));
    if ((unsigned)page >= (unsigned)npages) {
        atomicOr(err, KVE_DEVERR_BADPAGE);
        page = 0;
    }
    return page;
}

}  // namespace kve
