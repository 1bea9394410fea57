// qlin_i8ffn_api.hip -- the extern "C" entry points of the INT8 feed-forward
// operators declared in include/qlin.h: argument checks, then one launch
// sequence on the caller's stream.  No allocation, no synchronisation, no
// state.
#include <hip/hip_runtime.h>

#include "../../include/qlin.h"
#include "i8ffn_launch.hpp"

namespace {

inline bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p) % a != 0; }

inline int launch_status(hipError_t e) { return e == hipSuccess ? QLIN_OK : QLIN_ERR_LAUNCH; }

constexpr int64_t kMaxK = 131072;       // |sum of K products of codes| < 2^31
constexpr int64_t kMaxWidth = 1 << 20;  // I of the gated front
constexpr int64_t kMaxPitch = 1 << 30;  // elements of any row pitch: rows x pitch x bytes stays far inside 63 bits
constexpr int64_t kMaxE = 1024, kMaxTopk = 16;

inline bool bad_type(int dtype, int act) {
    return (dtype != QLIN_DT_BF16 && dtype != QLIN_DT_FP16) || (act != QLIN_ACT_SILU && act != QLIN_ACT_GELU_TANH);
}

inline bool bad_reduction(int64_t K) { return K < 16 || K > kMaxK || K % 16 != 0; }

bool bad_moe_shape(int64_t M, int64_t H, int64_t I, int64_t topk, int64_t E) {
    return M < 1 || M > QLIN_MAX_M_PREFILL || bad_reduction(H) || bad_reduction(I) || E < 1 || E > kMaxE || topk < 1 ||
           topk > kMaxTopk;
}

}  // namespace

extern "C" {

int qlin_glu_i8(const void* x, int64_t ldx, int64_t M, int64_t K, int dtype,
                const int8_t* w13, int64_t ldw, int64_t I, const float* s13, int ws_per_row, int act,
                int8_t* xq, int64_t ldxq, float* xs, void* y, int64_t ldy, void* stream) {
    if (bad_type(dtype, act) || (ws_per_row != 0 && ws_per_row != 1)) return QLIN_ERR_ARG;
    if (!x || !w13 || !s13 || !xq || !xs || !y) return QLIN_ERR_NULL;
    if (M < 1 || M > QLIN_MAX_M_PREFILL || I < 1 || I > kMaxWidth || bad_reduction(K)) return QLIN_ERR_SHAPE;
    if (ldx < K || ldw < K || ldxq < K || ldy < I || ldx > kMaxPitch || ldw > kMaxPitch || ldxq > kMaxPitch ||
        ldy > kMaxPitch)
        return QLIN_ERR_STRIDE;
    if (misaligned(x, 16) || ldx % 8 != 0 || misaligned(w13, 16) || ldw % 16 != 0 || misaligned(s13, 4) ||
        misaligned(xq, 16) || ldxq % 16 != 0 || misaligned(xs, 4) || misaligned(y, 2))
        return QLIN_ERR_ALIGN;
    const qlin::I8GluArgs a{dtype, (const uint16_t*)x, ldx, M, K, w13, ldw, I, s13, ws_per_row, act,
                            xq, ldxq, xs, (uint16_t*)y, ldy};
    return launch_status(qlin::launch_glu_i8(a, (hipStream_t)stream));
}

size_t qlin_moe_ffn_i8_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t topk, int64_t E) {
    if (bad_moe_shape(M, H, I, topk, E)) return 0;
    return qlin::moe_ffn_i8_workspace_bytes(M, H, I, topk, E);
}

int qlin_moe_ffn_i8(const void* x, int64_t ldx, int64_t M, int64_t H, int dtype,
                    const float* logits, int64_t ldl, int64_t E, int64_t topk, int route,
                    const int8_t* w13, int64_t ldw13, const float* s13, int64_t I,
                    const int8_t* w2, int64_t ldw2, const float* s2, int act,
                    int32_t* ids, float* gw, void* y, int64_t ldy,
                    void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_type(dtype, act) || (route != QLIN_ROUTE_SELECTED && route != QLIN_ROUTE_ALL)) return QLIN_ERR_ARG;
    if (!x || !w13 || !s13 || !w2 || !s2 || !ids || !gw || !y) return QLIN_ERR_NULL;
    if (bad_moe_shape(M, H, I, topk, E) || (logits && topk > E)) return QLIN_ERR_SHAPE;
    if (ldx < H || (logits && ldl < E) || ldw13 < H || ldw2 < I || ldy < H || ldx > kMaxPitch ||
        (logits && ldl > kMaxPitch) || ldw13 > kMaxPitch || ldw2 > kMaxPitch || ldy > kMaxPitch)
        return QLIN_ERR_STRIDE;
    if (misaligned(x, 16) || ldx % 8 != 0 || misaligned(logits, 4) || misaligned(w13, 16) || ldw13 % 16 != 0 ||
        misaligned(s13, 4) || misaligned(w2, 16) || ldw2 % 16 != 0 || misaligned(s2, 4) || misaligned(ids, 4) ||
        misaligned(gw, 4) || misaligned(y, 2))
        return QLIN_ERR_ALIGN;
    if (!workspace || workspace_bytes < qlin::moe_ffn_i8_workspace_bytes(M, H, I, topk, E)) return QLIN_ERR_WORKSPACE;
    if (misaligned(workspace, 16)) return QLIN_ERR_ALIGN;
    const qlin::I8MoeArgs a{dtype, (const uint16_t*)x, ldx, M, H, logits, ldl, E, topk, route, w13, ldw13, s13, I,
                            w2, ldw2, s2, act, ids, gw, (uint16_t*)y, ldy, (uint8_t*)workspace};
    return launch_status(qlin::launch_moe_ffn_i8(a, (hipStream_t)stream));
}

}  // extern "C"
