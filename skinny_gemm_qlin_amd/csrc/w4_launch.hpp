// w4_launch.hpp -- internal interface of the 4-bit weight operators between
// the C-ABI layer (qlin_w4_api.hip) and the kernels.  Arguments are validated.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qlin {

// The weight matrix: codes [N][ldw] (bytes), scales [N][K / group], zero
// points [N][K / group] or null (8 everywhere).
struct W4Weight {
    const uint8_t* w; int64_t ldw; int64_t N; int64_t K;
    const uint16_t* ws; const uint8_t* wz; int64_t group;
};

struct W4LinearArgs {  // y = x W^T + bias
    int dtype; const uint16_t* x; int64_t ldx; int64_t M; W4Weight w;
    const uint16_t* bias; uint16_t* y; int64_t ldy;
};

struct W4BwdArgs {  // dx = dy W
    int dtype; const uint16_t* dy; int64_t lddy; int64_t M; W4Weight w;
    uint16_t* dx; int64_t lddx; float* part;  // part: workspace of w4_bwd_workspace_bytes
};

struct W4GluArgs {  // g, u = x W^T (w.N = 2 I); dy null: y = act(g) u, gu (optional); else dgu
    int dtype; const uint16_t* x; int64_t ldx; int64_t M; W4Weight w; int64_t I; int act;
    uint16_t* y; int64_t ldy; uint16_t* gu; int64_t ldgu;
    const uint16_t* dy; int64_t lddy;  // backward: gradient of y; gu then receives [dg, du]
};

struct W4GateBwdArgs {  // dgu = [dy u act'(g), dy act(g)] from the kept gu
    int dtype; const uint16_t* dy; int64_t lddy; int64_t M; int64_t I; int act;
    const uint16_t* gu; int64_t ldgu; uint16_t* dgu; int64_t lddgu;
};

hipError_t launch_gemv_w4(const W4LinearArgs& a, hipStream_t st);
hipError_t launch_glu_w4(const W4GluArgs& a, hipStream_t st);
hipError_t launch_gemv_w4_bwd(const W4BwdArgs& a, hipStream_t st);
hipError_t launch_gate_bwd(const W4GateBwdArgs& a, hipStream_t st);
size_t w4_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K);

}  // namespace qlin
