// i8ffn_few_bf16.hip -- the INT8 feed-forward kernels for up to 16 tokens, bf16.
#include "i8ffn_few_impl.hpp"

namespace qlin {

size_t few_list_bytes() { return sizeof(FewList); }
hipError_t few_glu_bf16(const I8GluArgs& a, hipStream_t st) { return few_glu<kBf16>(a, st); }
hipError_t few_moe_bf16(const I8MoeArgs& a, const I8FewRegions& r, hipStream_t st) { return few_moe<kBf16>(a, r, st); }

}  // namespace qlin
