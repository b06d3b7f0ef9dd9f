// qg_moe_tokens_u2.cu -- the few-token expert products for 2-bit codes (qg_moe_tokens.cuh).
#include "qg_moe_tokens.cuh"

namespace qg {
namespace moe {
template cudaError_t launch_experts<2>(const Args &a, cudaStream_t s);
template bool experts_fit<2>(int K, int bs, bool zp);
}  // namespace moe
}  // namespace qg
