// qlin_w4_api.hip -- the extern "C" entry points of the 4-bit weight
// operators declared in include/qlin.h: argument checks, then one launch
// sequence on the caller's stream.  No allocation, no synchronisation, no
// state.
#include <hip/hip_runtime.h>

#include "../../include/qlin.h"
#include "w4_launch.hpp"

namespace {

inline bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p) % a != 0; }

inline int launch_status(hipError_t e) { return e == hipSuccess ? QLIN_OK : QLIN_ERR_LAUNCH; }

constexpr int64_t kMaxDim = 1 << 20;    // N (rows of W) and K: indexes of scale groups stay in 32 bits
constexpr int64_t kMaxPitch = 1 << 20;  // bytes of a code row: a workgroup has fewer than 4096 rows, offsets in them fit 32 bits

inline bool bad_flag(int dtype) { return dtype != QLIN_DT_BF16 && dtype != QLIN_DT_FP16; }

// shape and pointer rules every 4-bit weight shares; N counts the rows of W
int check_shape(int64_t M, int64_t N, int64_t K, int64_t group) {
    if (M < 1 || M > QLIN_MAX_M_PREFILL || N < 1 || N > kMaxDim || K < 32 || K > kMaxDim || K % 32 != 0)
        return QLIN_ERR_SHAPE;
    if (group < 32 || group % 32 != 0 || K % group != 0) return QLIN_ERR_SHAPE;
    return QLIN_OK;
}

inline bool weight_misaligned(const uint8_t* w, int64_t ldw, const void* ws) {
    return misaligned(w, 16) || ldw % 16 != 0 || misaligned(ws, 2);
}

}  // namespace

extern "C" {

int qlin_gemv_w4(const void* x, int64_t ldx, int64_t M, int64_t K, int dtype,
                 const uint8_t* w, int64_t ldw, int64_t N, const void* ws, const uint8_t* wz, int64_t group,
                 const void* bias, void* y, int64_t ldy, void* stream) {
    if (bad_flag(dtype)) return QLIN_ERR_ARG;
    if (!x || !w || !ws || !y) return QLIN_ERR_NULL;
    const int rc = check_shape(M, N, K, group);
    if (rc != QLIN_OK) return rc;
    if (ldx < K || ldw < K / 2 || ldw > kMaxPitch || ldy < N) return QLIN_ERR_STRIDE;
    if (misaligned(x, 16) || ldx % 8 != 0 || weight_misaligned(w, ldw, ws) || misaligned(y, 2) ||
        (bias && misaligned(bias, 2)))
        return QLIN_ERR_ALIGN;
    const qlin::W4LinearArgs a{dtype, (const uint16_t*)x, ldx, M,
                               {w, ldw, N, K, (const uint16_t*)ws, wz, group},
                               (const uint16_t*)bias, (uint16_t*)y, ldy};
    return launch_status(qlin::launch_gemv_w4(a, (hipStream_t)stream));
}

size_t qlin_gemv_w4_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_shape(M, N, K, 32) != QLIN_OK) return 0;
    return qlin::w4_bwd_workspace_bytes(M, N, K);
}

int qlin_gemv_w4_bwd(const void* dy, int64_t lddy, int64_t M, int64_t N, int dtype,
                     const uint8_t* w, int64_t ldw, int64_t K, const void* ws, const uint8_t* wz, int64_t group,
                     void* dx, int64_t lddx, void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_flag(dtype)) return QLIN_ERR_ARG;
    if (!dy || !w || !ws || !dx) return QLIN_ERR_NULL;
    const int rc = check_shape(M, N, K, group);
    if (rc != QLIN_OK) return rc;
    if (lddy < N || ldw < K / 2 || ldw > kMaxPitch || lddx < K) return QLIN_ERR_STRIDE;
    if (misaligned(dy, 16) || lddy % 8 != 0 || weight_misaligned(w, ldw, ws) || misaligned(dx, 2))
        return QLIN_ERR_ALIGN;
    const size_t need = qlin::w4_bwd_workspace_bytes(M, N, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return QLIN_ERR_WORKSPACE;
    if (need > 0 && misaligned(workspace, 16)) return QLIN_ERR_ALIGN;
    const qlin::W4BwdArgs a{dtype, (const uint16_t*)dy, lddy, M, {w, ldw, N, K, (const uint16_t*)ws, wz, group},
                            (uint16_t*)dx, lddx, (float*)workspace};
    return launch_status(qlin::launch_gemv_w4_bwd(a, (hipStream_t)stream));
}

int qlin_glu_w4(const void* x, int64_t ldx, int64_t M, int64_t K, int dtype,
                const uint8_t* w13, int64_t ldw, int64_t I, const void* s13, const uint8_t* z13, int64_t group,
                int act, void* y, int64_t ldy, void* gu, int64_t ldgu, void* stream) {
    if (bad_flag(dtype) || (act != QLIN_ACT_SILU && act != QLIN_ACT_GELU_TANH)) return QLIN_ERR_ARG;
    if (!x || !w13 || !s13 || !y) return QLIN_ERR_NULL;
    if (I < 1 || I > kMaxDim / 2) return QLIN_ERR_SHAPE;
    const int rc = check_shape(M, 2 * I, K, group);
    if (rc != QLIN_OK) return rc;
    if (ldx < K || ldw < K / 2 || ldw > kMaxPitch || ldy < I || (gu && ldgu < 2 * I)) return QLIN_ERR_STRIDE;
    if (misaligned(x, 16) || ldx % 8 != 0 || weight_misaligned(w13, ldw, s13) || misaligned(y, 2) ||
        (gu && misaligned(gu, 2)))
        return QLIN_ERR_ALIGN;
    const qlin::W4GluArgs a{dtype, (const uint16_t*)x, ldx, M, {w13, ldw, 2 * I, K, (const uint16_t*)s13, z13, group},
                            I, act, (uint16_t*)y, ldy, (uint16_t*)gu, ldgu, nullptr, 0};
    return launch_status(qlin::launch_glu_w4(a, (hipStream_t)stream));
}

int qlin_glu_w4_bwd(const void* dy, int64_t lddy, int64_t M, int64_t I, int dtype, int act,
                    const void* x, int64_t ldx, const void* gu, int64_t ldgu,
                    const uint8_t* w13, int64_t ldw, int64_t K, const void* s13, const uint8_t* z13, int64_t group,
                    void* dgu, int64_t lddgu, void* dx, int64_t lddx,
                    void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_flag(dtype) || (act != QLIN_ACT_SILU && act != QLIN_ACT_GELU_TANH)) return QLIN_ERR_ARG;
    if (!dy || (!x && !gu) || !w13 || !s13 || !dgu) return QLIN_ERR_NULL;
    if (I < 1 || I > kMaxDim / 2) return QLIN_ERR_SHAPE;
    const int rc = check_shape(M, 2 * I, K, group);
    if (rc != QLIN_OK) return rc;
    if (lddy < I || (gu ? ldgu < 2 * I : ldx < K) || ldw < K / 2 || ldw > kMaxPitch || lddgu < 2 * I || (dx && lddx < K))
        return QLIN_ERR_STRIDE;
    if (gu == dgu && ldgu != lddgu && M > 1) return QLIN_ERR_STRIDE;  // a row written before another is read
    if (misaligned(dy, 2) || (gu ? misaligned(gu, 2) : misaligned(x, 16) || ldx % 8 != 0) ||
        weight_misaligned(w13, ldw, s13) || misaligned(dgu, 16) || lddgu % 8 != 0 || (dx && misaligned(dx, 2)))
        return QLIN_ERR_ALIGN;
    const size_t need = dx ? qlin::w4_bwd_workspace_bytes(M, 2 * I, K) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return QLIN_ERR_WORKSPACE;
    if (need > 0 && misaligned(workspace, 16)) return QLIN_ERR_ALIGN;
    const qlin::W4Weight wt{w13, ldw, 2 * I, K, (const uint16_t*)s13, z13, group};
    hipStream_t st = (hipStream_t)stream;
    hipError_t e;
    if (gu) {
        const qlin::W4GateBwdArgs a{dtype, (const uint16_t*)dy, lddy, M, I, act, (const uint16_t*)gu, ldgu,
                                    (uint16_t*)dgu, lddgu};
        e = qlin::launch_gate_bwd(a, st);
    } else {
        const qlin::W4GluArgs a{dtype, (const uint16_t*)x, ldx, M, wt, I, act, nullptr, 0, (uint16_t*)dgu, lddgu,
                                (const uint16_t*)dy, lddy};
        e = qlin::launch_glu_w4(a, st);
    }
    if (e != hipSuccess || !dx) return launch_status(e);
    const qlin::W4BwdArgs b{dtype, (const uint16_t*)dgu, lddgu, M, wt, (uint16_t*)dx, lddx, (float*)workspace};
    return launch_status(qlin::launch_gemv_w4_bwd(b, st));
}

}  // extern "C"
