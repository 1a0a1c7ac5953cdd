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
    float2 *products; // [B][H][segments]: the product of a segment's decays, as Product::packed gives it
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
// A product of many decays, m 2^e: over thousands of tokens it may leave fp32's range, and fp64's, while
// what it is multiplied with is zero, small or large enough for the result to stay within. settle() is due
// after every 128 decays at most: m stays so far from fp64's ends that a product of 128 decays, which fits
// fp32, leaves it within (one that is below 2^-500 has left nothing of an fp32 state).
struct Product {
    double m = 1.0;
    int e = 0;
    __device__ __forceinline__ void settle()
    {
        const unsigned field = (unsigned)__double2hiint(m) >> 20 & 0x7FFu;  // m's exponent + 1023
        if (field - 523u > 1000u && m != 0.0 && isfinite(m)) {
            int up;
            m = frexp(m, &up);
            e = min(max(e + up, -(1 << 30)), 1 << 30);
        }
    }
    // (x, 0) for a product that a normal fp32 number x rounds (or zero, or not finite); else (a, e), a e-th
    // power of two apart
    __device__ __forceinline__ float2 packed() const
    {
        int up = 0;
        const bool plain = m == 0.0 || !isfinite(m);
        const double a = plain ? m : frexp(m, &up);
        const int all = e + up;
        const float x = (float)ldexp(a, all);
        if (plain || (fabsf(x) >= 1.17549435e-38f && fabsf(x) <= 3.402823466e38f)) return make_float2(x, __int_as_float(0));
        return make_float2((float)a, __int_as_float(all));
    }
};
// product * S + x
__device__ __forceinline__ float carry(float2 product, float S, float x)
{
    const int e = __float_as_int(product.y);
    return e == 0 ? fmaf(product.x, S, x) : (float)ldexp((double)product.x * S, e) + x;
}

// Tokens of request b; -1 for a length outside [0, T].
__device__ __forceinline__ int prompt_length(const DecayParams &p, int b)
{
    const int n = p.lens ? p.lens[b] : p.T;
    return n < 0 || n > p.T ? -1 : n;
}
#endif

}  // namespace stq
