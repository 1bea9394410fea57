// i8ffn_launch.hpp -- internal interface of the INT8 feed-forward operators
// (gated front, routed expert layer) between the C-ABI layer
// (qlin_i8ffn_api.hip) and the kernels.  Arguments are validated.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qlin {

struct I8GluArgs {  // y = act(g) u, [g, u] = x W13^T; codes and scales of x go to xq, xs
    int dtype; const uint16_t* x; int64_t ldx; int64_t M; int64_t K;
    const int8_t* w13; int64_t ldw; int64_t I; const float* s13; int ws_step; int act;
    int8_t* xq; int64_t ldxq; float* xs; uint16_t* y; int64_t ldy;
};

struct I8MoeArgs {  // logits null: ids and gw are inputs
    int dtype; const uint16_t* x; int64_t ldx; int64_t M; int64_t H;
    const float* logits; int64_t ldl; int64_t E; int64_t topk; int route;
    const int8_t* w13; int64_t ldw13; const float* s13; int64_t I;
    const int8_t* w2; int64_t ldw2; const float* s2; int act;
    int32_t* ids; float* gw; uint16_t* y; int64_t ldy; uint8_t* workspace;
};

hipError_t launch_glu_i8(const I8GluArgs& a, hipStream_t st);
hipError_t launch_moe_ffn_i8(const I8MoeArgs& a, hipStream_t st);
size_t moe_ffn_i8_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t topk, int64_t E);

}  // namespace qlin
