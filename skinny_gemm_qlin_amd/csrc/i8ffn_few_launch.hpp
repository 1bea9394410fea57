// i8ffn_few_launch.hpp -- entry points of the kernels for up to 16 tokens, one
// translation unit per 16-bit type.
#pragma once
#include "i8ffn_launch.hpp"

namespace qlin {

struct I8FewRegions {  // of the layer's workspace
    int8_t* xq; float* xs; uint16_t* h; int8_t* hq; float* hs; void* list;
};

size_t few_list_bytes();
hipError_t few_glu_bf16(const I8GluArgs& a, hipStream_t st);
hipError_t few_glu_fp16(const I8GluArgs& a, hipStream_t st);
hipError_t few_moe_bf16(const I8MoeArgs& a, const I8FewRegions& r, hipStream_t st);
hipError_t few_moe_fp16(const I8MoeArgs& a, const I8FewRegions& r, hipStream_t st);

}  // namespace qlin
