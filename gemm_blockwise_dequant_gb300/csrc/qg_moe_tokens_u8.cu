// qg_moe_tokens_u8.cu -- the few-token expert products for 8-bit codes (qg_moe_tokens.cuh).
#include "qg_moe_tokens.cuh"

namespace qg {
namespace moe {
template cudaError_t launch_experts<8>(const Args &a, cudaStream_t s);
template bool experts_fit<8>(int K, int bs, bool zp);
}  // namespace moe
}  // namespace qg
