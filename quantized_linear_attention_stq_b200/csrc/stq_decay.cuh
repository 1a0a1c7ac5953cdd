// stq_decay.cuh -- declarations shared by the kernels of decayed linear attention (fp32 state pool).
#pragma once

#include "stq_internal.cuh"

namespace stq {

struct DecayParams {
    float *states;        // [state_slots][H][d][d]
    const int32_t *slots; // [B]
    const void *q, *k, *v;  // [B][H][T][d]
    const float *alpha;   // [B][H][T]
    const int32_t *lens;  // [B] or null: every prompt has T tokens
    float *o;             // [B][H][T][d]
    int32_t *status;
    int32_t state_slots, B, H, T;
    // a prompt cut into segments (one: the whole prompt, records and products are null)
    float *records;   // [B][H][segments][d][d]: a segment's own sum, then the state before it
    float *products;  // [B][H][segments]: the product of a segment's decays
    int32_t segments, seg_tokens;
};

// Token by token, any d and input type.
cudaError_t launch_decay_serial(const DecayParams &p, int d, int in_bf16, bool sums, cudaStream_t s);
// Chunks of kDecayChunk tokens on the tensor cores, bf16 inputs, any d; cudaErrorNotSupported where no
// tensor map can be made. seg_tokens is a multiple of kDecayChunk.
// Both: with `sums`, the segments' own sums and products go to records and products, and nothing else
// is written; without, the outputs and final states are, from the states before the segments.
constexpr int kDecayChunk = 128;
cudaError_t launch_decay_chunk(const DecayParams &p, int d, bool sums, cudaStream_t s);

#ifdef __CUDACC__
// Tokens of request b; -1 for a length outside [0, T].
__device__ __forceinline__ int prompt_length(const DecayParams &p, int b)
{
    const int n = p.lens ? p.lens[b] : p.T;
    return n < 0 || n > p.T ? -1 : n;
}
#endif

}  // namespace stq
