// i8ffn_few_fp16.hip -- the INT8 feed-forward kernels for up to 16 tokens, fp16.
#include "i8ffn_few_impl.hpp"

namespace qlin {

hipError_t few_glu_fp16(const I8GluArgs& a, hipStream_t st) { return few_glu<kFp16>(a, st); }
hipError_t few_moe_fp16(const I8MoeArgs& a, const I8FewRegions& r, hipStream_t st) { return few_moe<kFp16>(a, r, st); }

}  // namespace qlin
