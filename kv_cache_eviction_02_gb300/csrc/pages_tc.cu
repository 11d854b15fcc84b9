// Shared-prompt decoding on the 5th-generation tensor cores (tcgen05, sm_103a): attention of all
// rows behind a prompt over the prompt's K/V, bf16 or fp16. d_head 32 runs as 64: the boxes reach behind
// the arrays' rows, where TMA fills in zeros.
//
// The rows of a prompt's requests (new rows x g query heads of a KV head) are stacked into 128-row
// tiles, so the prompt's K/V stream from HBM once per tile or pair of tiles, however many requests
// share it. One CTA takes one or two row tiles of one prompt and KV head over a split of the tokens:
//   S_t = Q_t K^T (128 rows x 128 tokens) into TMEM, the softmax of a row in one thread (running
//   maximum, rescale of O only when it grew by 2^8), P as 16-bit pairs back into TMEM over S, and
//   O_t += P_t V with P read from TMEM and V as the MN-major B operand.
// Tiles come by TMA straight from the caller's strided arrays: Q as {d, g heads, rows} boxes, K and V
// as {d, 128 tokens} boxes of a {d, tokens, heads, prompts} map, rows behind the map filled with
// zeros. Rows between a prompt's own length and the map's end may hold anything: their scores are
// masked, and the softmax warps write zeros over their V rows in shared memory before they hand P on.
// Few rows (lookahead: 4 trajectories x 4 heads): bound by HBM; many (hundreds): by the tensor pipe.
//
// The same kernel (OWN) takes the own rows of requests that add many rows at once: K and V as boxes of
// the request's pages, scores masked at each row's own position.
#include "pages_tc.cuh"

namespace kve {
namespace {

// ---- host ------------------------------------------------------------------------------------------
template <typename T, int D, int QT, bool OWN>
cudaError_t go(const PgDims &D_, const PgAttn &A, cudaStream_t st) {
    constexpr bool f16 = PtIsHalf<T>::value;
    const cuuint64_t d = D_.d, one = 1;
    CUtensorMap tq, tk, tv;
    // the prompt's {columns, tokens, heads, prompts}, or the pool's {columns, rows}
    const cuuint64_t kd[4] = {d, OWN ? (cuuint64_t)D_.npages * D_.Hkv * D_.P : (cuuint64_t)D_.n,
                              OWN ? one : (cuuint64_t)D_.Hkv, OWN ? one : (cuuint64_t)D_.S};
    const long long ks[3] = {OWN ? D_.d : A.p_tok, A.p_head, A.p_prompt};
    const cuuint32_t kb[4] = {64, OWN && D_.P < 128 ? (cuuint32_t)D_.P : 128u, 1, 1};
    const int rank = OWN ? 2 : 4;
    if (!pt_q_map(&tq, f16, D_, A) ||
        !pg_tmap(&tk, f16, OWN ? A.K : A.Kp, rank, kd, ks, kb) ||
        !pg_tmap(&tv, f16, OWN ? A.V : A.Vp, rank, kd, ks, kb))
        return cudaErrorInvalidValue;
    return pt_launch<T, D, QT, 0, OWN>(D_, pt_args<QT>(D_, A, OWN), tq, tk, tv, st);
}

template <typename T, bool OWN>
cudaError_t by_shape(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    const int qt = pg_pairs(D, OWN ? D.max_new : D.group_rows());
    if (D.d == 128) return qt == 2 ? go<T, 128, 2, OWN>(D, A, st) : go<T, 128, 1, OWN>(D, A, st);
    return qt == 2 ? go<T, 64, 2, OWN>(D, A, st) : go<T, 64, 1, OWN>(D, A, st);
}

}  // namespace

bool pg_tmap(CUtensorMap *map, bool f16, const void *base, int rank, const cuuint64_t *dims,
             const long long *strides, const cuuint32_t *box) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!fn) return false;
    cuuint64_t bytes[4];
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = (cuuint64_t)strides[i] * 2;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
              const_cast<void *>(base), dims, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_pg_prompt_tc(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_shape<__nv_bfloat16, false>(D, A, st)
                               : by_shape<__half, false>(D, A, st);
}

cudaError_t launch_pg_own_tc(const PgDims &D, const PgAttn &A, cudaStream_t st) {
    return D.dtype == KVE_BF16 ? by_shape<__nv_bfloat16, true>(D, A, st)
                               : by_shape<__half, true>(D, A, st);
}

}  // namespace kve
