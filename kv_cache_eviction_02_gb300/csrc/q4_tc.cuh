// Cache in 4 bits on the 5th-generation tensor cores: attention of many query rows over a prompt, or over a request's
// own pages, by the kernel of pages_tc.cuh with its operands made from codes. (A type per translation unit: they
// compile beside one another.)
#pragma once

#include "pages_tc.cuh"

namespace kve {
namespace {

template <typename T, int D, int QT, int G, bool OWN>
cudaError_t go(const PgDims &D_, const Q4Shape &Q, const PgAttn &A, cudaStream_t st) {
    CUtensorMap tq;
    if (!pt_q_map(&tq, PtIsHalf<T>::value, D_, A)) return cudaErrorInvalidValue;
    PtArgs P = pt_args<QT>(D_, A, OWN);
    P.codes = static_cast<const uint8_t *>(OWN ? A.K : A.Kp);
    P.ptiles = Q.ptiles;
    return pt_launch<T, D, QT, G, OWN>(D_, P, tq, tq, tq, st);
}
template <typename T, int G, bool OWN>
cudaError_t by_shape(const PgDims &D, const Q4Shape &Q, const PgAttn &A, cudaStream_t st) {
    const int qt = pg_pairs(D, OWN ? D.max_new : D.group_rows());
    if (D.d == 128) return qt == 2 ? go<T, 128, 2, G, OWN>(D, Q, A, st) : go<T, 128, 1, G, OWN>(D, Q, A, st);
    if constexpr (G <= 64) return qt == 2 ? go<T, 64, 2, G, OWN>(D, Q, A, st) : go<T, 64, 1, G, OWN>(D, Q, A, st);
    return cudaErrorInvalidValue;
}
template <typename T, bool OWN> cudaError_t by_group(const PgDims &D, const Q4Shape &Q, const PgAttn &A, cudaStream_t st) {
    return Q.group == 32 ? by_shape<T, 32, OWN>(D, Q, A, st)
                         : (Q.group == 64 ? by_shape<T, 64, OWN>(D, Q, A, st) : by_shape<T, 128, OWN>(D, Q, A, st));
}

}  // namespace

template <typename T> cudaError_t launch_q4_tc(const PgDims &D, const Q4Shape &Q, const PgAttn &A, bool own, cudaStream_t st) {
    return own ? by_group<T, true>(D, Q, A, st) : by_group<T, false>(D, Q, A, st);
}

}  // namespace kve
