// qg_lora_tc.h -- launches of the adapters' tensor-core contractions (qg_lora_tc.cu).
#pragma once

#include "qg_lora_common.cuh"

namespace qg {

struct ShrinkTc {
    LoraProblem p;
    float *sums;             // [T][rank]: V (unscaled) or G (scaled)
    const float *V;          // backward: the forward pass's V, for its largest values
    float *tile_max;         // [2][CTAs]: largest sum and largest V of a CTA's rows; or null
    int *tile_adapter;       // [CTAs] or null
    TermsOut terms;          // bf16, backward: the terms of G and V
    int bwd, bf16, cs;
    int n, steps, stages, w_bytes;  // filled in by the launch
    unsigned *fault;
};

struct TermsTc {
    LoraProblem p;
    const float *skinny[2];  // G, V
    uint16_t *terms;         // [2][terms][T][rank]
    const float *tile_max;
    const int *tile_adapter;
    int parts;
};

struct WgradTc {
    LoraProblem p;
    void *out[2];            // dA, dB
    int g_dtype, accumulate;
    const float *tile_max;   // of the shrink launch before it
    const int *tile_adapter;
    int parts;               // its CTAs
    int cols[2], tiles[2], n, cs, stages;  // filled in by the launch
    unsigned *fault;
};

bool lora_tc_available();
int shrink_tc_tiles(int T, int S);
cudaError_t launch_shrink_tc(ShrinkTc q, const void *in, int64_t ld, const void *w, cudaStream_t s);
size_t wgrad_tc_terms_bytes(int T, int r);  // room for the 16-bit terms of G and V
int wgrad_tc_terms(bool bf16, int g_dtype); // how many each
// bf16: the terms are there; fp16: they are made from G and V with the tiles' largest values.
cudaError_t launch_wgrad_tc(WgradTc q, const float *G, const float *V, uint16_t *terms, const void *x, int64_t ldx, const void *dy, int64_t lddy, bool bf16,
                            cudaStream_t s);

}  // namespace qg
