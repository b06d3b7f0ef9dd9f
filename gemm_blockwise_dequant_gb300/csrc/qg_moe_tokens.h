// qg_moe_tokens.h -- what the translation units of the few-token MoE layer share.
#pragma once

#include "qg_internal.h"

namespace qg {
namespace moe {

constexpr int kMaxPairs = 1024, kMaxExperts = 512;

// One of the two products over the experts.
struct Args {
    int fc;                 // 1: SwiGLU of both halves; 2: plain
    const void *src;        // fc 1: [T][K] activations; fc 2: [P][K] fp32
    int src_dtype;
    const int32_t *ids;     // [P]
    int P, k, E;
    const uint8_t *w;       // [E][N][K * bits / 8]
    const uint16_t *scales, *zp, *bias;  // zp, bias: or null
    int N, K, bs, interleaved;
    float *out;             // fc 1: [P][N / 2]; fc 2: [P][N]
    int *status;            // or null
    int most_rows;          // that can meet at one expert, were every token's choices different
    int terms;              // fp16 values that an activation enters as: 1 or 2, each with a row (and an MMA column) of its own
    int room;               // rows of activations that fit (filled in at the launch)
};
template <int BITS>
cudaError_t launch_experts(const Args &a, cudaStream_t s);
// A row of K activations fits the kernel's shared memory.
template <int BITS>
bool experts_fit(int K, int bs, bool zp);

}  // namespace moe
}  // namespace qg
