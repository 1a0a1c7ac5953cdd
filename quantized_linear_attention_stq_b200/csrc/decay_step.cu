// decay_step.cu -- linear attention with a decay per head, without the delta term, on an fp32 state
// pool (contract in include/stq.h): one token (stq_decay_step) and the token-by-token prompt form.
//
//   S <- alpha S + k v^T ;  o = S^T q      (readout after the update)
//
// One token. Bound by HBM: a head's state is read and written once (8 d^2 bytes), with 5 d^2
// operations. One CTA per (request, head) keeps the whole state in registers between its load and
// its store, all loads of a thread in flight at once; a warp's lanes hold consecutive columns, so
// rows move in whole 128-byte lines and the readout is a sum over the CTA's row groups.
//
// Token by token (fp32 inputs, most bf16 ones of d = 16, short prompts). The state of a block of columns stays in registers for the
// whole prompt (columns of S are independent of each other); tokens are staged through shared memory 16 or
// 32 at a time. A column's rows are spread over SL lanes, joined by shuffles per token. Bound by the FMAs,
// three to an entry and token (32 heads of 2048 tokens of d = 128: 269 us, of which 89 at the FMAs' rate).
//
// Segments. Where there are too few heads to fill the GPU, prompts are cut into segments: a first
// pass over all but the last makes each segment's own sum (from an empty state) and the product of its
// decays, a join turns these into the states before the segments, and the main pass then runs all
// segments at once. The first pass costs a part of the main one, so a cut has to win more than that.
#include <cmath>

#include "../../include/stq.h"
#include "stream_order.cuh"
#include "stq_decay.cuh"

namespace stq {
namespace {

// Four inputs as they lie in memory.
template <int IN_BF16>
struct Raw4 {
    uint2 r;
    __device__ __forceinline__ void load(const void *base, size_t idx)
    {
        r = *reinterpret_cast<const uint2 *>(reinterpret_cast<const __nv_bfloat16 *>(base) + idx);
    }
    __device__ __forceinline__ float4 value() const
    {
        return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                           __uint_as_float(r.y & 0xFFFF0000u));
    }
};
template <>
struct Raw4<0> {
    float4 r;
    __device__ __forceinline__ void load(const void *base, size_t idx)
    {
        r = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + idx);
    }
    __device__ __forceinline__ float4 value() const { return r; }
};

template <int D>
struct StepCfg {
    static constexpr int C4 = D / 4;                                  // float4 columns of a row
    static constexpr int NT = D * C4 < 256 ? D * C4 : 256;            // threads
    static constexpr int RG = NT / C4;                                // rows of one pass
    static constexpr int NR = D / RG;                                 // passes
};

template <int D, int IN_BF16>
__global__ void __launch_bounds__(StepCfg<D>::NT) decay_step_kernel(const DecayParams p)
{
    using S = StepCfg<D>;
    __shared__ float4 part[S::RG][S::C4];
    __shared__ float qs[D], ks[D];
    const int tid = threadIdx.x, c = tid % S::C4, rg = tid / S::C4;
    wait_for_stream();
    const size_t tile = blockIdx.x;  // (request, head)
    const int b = (int)(tile / (unsigned)p.H), h = (int)(tile - (size_t)b * p.H);
    const int slot = p.slots[b];
    if (slot < 0 || slot >= p.state_slots) {
        if (tid == 0) flag(p.status, kFlagBounds);
        return;
    }
    float4 *st = reinterpret_cast<float4 *>(p.states + ((size_t)slot * p.H + h) * (D * D)) + (size_t)rg * S::C4 + c;
    float4 s[S::NR];
#pragma unroll
    for (int i = 0; i < S::NR; ++i) s[i] = __ldcs(st + (size_t)i * S::RG * S::C4);
    for (int i = tid; i < D; i += S::NT) {
        qs[i] = load_in<IN_BF16>(p.q, tile * D + i);
        ks[i] = load_in<IN_BF16>(p.k, tile * D + i);
    }
    Raw4<IN_BF16> rv;
    rv.load(p.v, tile * D + 4 * c);
    const float4 v = rv.value();
    const float a = p.alpha[tile];
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < S::NR; ++i) {
        const int row = rg + i * S::RG;
        const float kk = ks[row], qq = qs[row];
        s[i].x = fmaf(a, s[i].x, kk * v.x);
        s[i].y = fmaf(a, s[i].y, kk * v.y);
        s[i].z = fmaf(a, s[i].z, kk * v.z);
        s[i].w = fmaf(a, s[i].w, kk * v.w);
        __stcs(st + (size_t)i * S::RG * S::C4, s[i]);
        acc.x = fmaf(qq, s[i].x, acc.x);
        acc.y = fmaf(qq, s[i].y, acc.y);
        acc.z = fmaf(qq, s[i].z, acc.z);
        acc.w = fmaf(qq, s[i].w, acc.w);
    }
    // a state entry that is not finite may meet a zero query entry: 0 * it is NaN, so it is tested here
    float bad = 0.f;
#pragma unroll
    for (int i = 0; i < S::NR; ++i)
        bad += (s[i].x - s[i].x) + (s[i].y - s[i].y) + (s[i].z - s[i].z) + (s[i].w - s[i].w);
    part[rg][c] = acc;
    __syncthreads();
    if (tid < S::C4) {
        float4 t = part[0][c];
#pragma unroll
        for (int r = 1; r < S::RG; ++r) {
            const float4 x = part[r][c];
            t.x += x.x;
            t.y += x.y;
            t.z += x.z;
            t.w += x.w;
        }
        bad += (t.x - t.x) + (t.y - t.y) + (t.z - t.z) + (t.w - t.w);
        *reinterpret_cast<float4 *>(p.o + tile * D + 4 * c) = t;
    }
    if (bad != 0.f) flag(p.status, kFlagNonfinite);  // x - x is 0 for a finite x, NaN otherwise
}

template <int D, int CW>
struct SerialCfg {
    static constexpr int SL = D >= 32 ? 8 : 4;                     // lanes sharing a column
    static constexpr int RW = D / SL;                              // rows of a thread
    // Columns of a CTA. One column to a thread: few heads are spread over more SMs by 16 than by 32, and as many CTAs
    // fill the GPU (d = 32, 77 tokens: 15 heads 5.5 and 7.2 us, 148 heads 7.2 and 7.4, 190 heads 9.4 and 11.5).
    static constexpr int CB = CW == 1 ? 16 : D < 64 ? D : 64;
    static constexpr int NT = CB / CW * SL;
    // Tokens staged at a time, by what 48 KB of shared memory hold of q, k and (one column to a thread) o's parts
    static constexpr int TB = CW == 4 || D == 128 ? 16 : 32;
};

template <int D, int IN_BF16, int SUMS, int CW>
__global__ void __launch_bounds__(SerialCfg<D, CW>::NT) decay_serial_kernel(const DecayParams p)
{
    using S = SerialCfg<D, CW>;
    __shared__ __align__(16) float qs[SUMS ? 1 : S::TB][D], ks[S::TB][D];
    // with one column to a thread o is summed behind the tokens, from a part of every lane (a pitch of SL + 1
    // keeps the lanes' writes and reads on different banks)
    constexpr int PARTS = CW == 1 && !SUMS ? S::SL + 1 : 1;
    __shared__ __align__(16) float vs[S::TB][S::CB], os[S::TB][S::CB * PARTS];
    __shared__ float as[S::TB];
    const int tid = threadIdx.x, r = tid % S::SL, cl = tid / S::SL * CW;
    const int seg = blockIdx.x / (D / S::CB), c0 = blockIdx.x % (D / S::CB) * S::CB;
    const size_t tile = blockIdx.y + (size_t)blockIdx.z * gridDim.y;  // (request, head)
    wait_for_stream();
    if (tile >= (size_t)p.B * p.H) return;
    const int b = (int)(tile / (unsigned)p.H), h = (int)(tile - (size_t)b * p.H);
    const int slot = p.slots[b];
    const int len = prompt_length(p, b);
    if (slot < 0 || slot >= p.state_slots || len < 0) {
        if (tid == 0) flag(p.status, kFlagBounds);
        return;
    }
    const int64_t from = (int64_t)seg * p.seg_tokens;
    if (from >= len) return;
    const int end = len - (int)from < p.seg_tokens ? len : (int)from + p.seg_tokens;
    if (SUMS && end == len) return;  // the state behind the last segment is the main pass's
    float *pool = p.states + ((size_t)slot * p.H + h) * (D * D) + c0 + cl;
    float *record = p.records ? p.records + (tile * p.segments + seg) * (D * D) + c0 + cl : nullptr;
    const float *before = p.segments > 1 ? record : pool;
    // rows of a thread: groups of 4, SL groups apart, so that the lanes' 16-byte reads of k and q are adjacent
    auto row = [&](int i) { return (size_t)((i / 4 * S::SL + r) * 4 + i % 4) * D; };
    float s[S::RW][CW];
#pragma unroll
    for (int i = 0; i < S::RW; ++i)
#pragma unroll
        for (int c = 0; c < CW; ++c) s[i][c] = SUMS ? 0.f : before[row(i) + c];
    const size_t base = tile * (size_t)p.T;
    Product upto;
    // a block's inputs are loaded a block ahead
    constexpr int NQ = (S::TB * D / 4 + S::NT - 1) / S::NT, NV = (S::TB * S::CB / 4 + S::NT - 1) / S::NT;
    static_assert(S::TB <= S::NT, "a thread has one decay of a block at most");
    Raw4<IN_BF16> rq[NQ], rk[NQ], rv[NV];
    float ra = 1.f;
    auto fetch = [&](int t0) {
        const int n = end - t0 < S::TB ? end - t0 : S::TB;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int i = 4 * (tid + x * S::NT);
            if (i < n * D) {
                if (!SUMS) rq[x].load(p.q, (base + t0) * D + i);
                rk[x].load(p.k, (base + t0) * D + i);
            }
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int i = 4 * (tid + x * S::NT);
            if (i < n * S::CB) rv[x].load(p.v, (base + t0 + i / S::CB) * D + c0 + i % S::CB);
        }
        if (tid < n) ra = p.alpha[base + t0 + tid];
    };
    fetch((int)from);
    for (int t0 = (int)from; t0 < end; t0 += S::TB) {
        const int n = end - t0 < S::TB ? end - t0 : S::TB;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int i = 4 * (tid + x * S::NT);
            if (i < n * D) {
                if (!SUMS) *reinterpret_cast<float4 *>(&qs[0][0] + i) = rq[x].value();
                *reinterpret_cast<float4 *>(&ks[0][0] + i) = rk[x].value();
            }
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int i = 4 * (tid + x * S::NT);
            if (i < n * S::CB) *reinterpret_cast<float4 *>(&vs[0][0] + i) = rv[x].value();
        }
        if (tid < n) as[tid] = ra;
        if (end - t0 > S::TB) fetch(t0 + S::TB);
        __syncthreads();
#pragma unroll(CW == 1 ? 8 : 2)
        for (int t = 0; t < n; ++t) {
            const float a = as[t];
            float v[CW], acc[CW];
            if constexpr (CW == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&vs[t][cl]);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
            } else {
                v[0] = vs[t][cl];
            }
#pragma unroll
            for (int c = 0; c < CW; ++c) acc[c] = 0.f;
            if (SUMS) upto.m *= a;
#pragma unroll
            for (int i = 0; i < S::RW; i += 4) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&ks[t][(i / 4 * S::SL + r) * 4]);
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < CW; ++c) s[i + e][c] = fmaf(a, s[i + e][c], kk[e] * v[c]);
                if constexpr (!SUMS) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(&qs[t][(i / 4 * S::SL + r) * 4]);
                    const float qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int c = 0; c < CW; ++c) acc[c] = fmaf(qq[e], s[i + e][c], acc[c]);
                }
            }
            if constexpr (!SUMS && CW == 1) os[t][cl * PARTS + r] = acc[0];
            if constexpr (!SUMS && CW == 4) {
                // four sums over eight lanes: a lane keeps half of its columns at a step
                const bool hi = r & 4, odd = r & 2;
                float x = hi ? acc[2] : acc[0], y = hi ? acc[3] : acc[1];
                x += __shfl_xor_sync(0xffffffffu, hi ? acc[0] : acc[2], 4);
                y += __shfl_xor_sync(0xffffffffu, hi ? acc[1] : acc[3], 4);
                float z = odd ? y : x;
                z += __shfl_xor_sync(0xffffffffu, odd ? x : y, 2);
                z += __shfl_xor_sync(0xffffffffu, z, 1);
                if (!(r & 1)) os[t][cl + (r >> 1)] = z;
            }
        }
        __syncthreads();
        if constexpr (SUMS) {
            upto.settle();
            continue;
        }
        float bad = 0.f;
        for (int i = 4 * tid; i < n * S::CB; i += 4 * S::NT) {
            float4 x;
            if constexpr (CW == 4) {
                x = *reinterpret_cast<const float4 *>(&os[0][0] + i);
            } else {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float *part = &os[0][0] + (i + e) * PARTS;
                    y[e] = part[0] + part[1] + (part[2] + part[3]);
                    if constexpr (S::SL == 8) y[e] += part[4] + part[5] + (part[6] + part[7]);
                }
                x = make_float4(y[0], y[1], y[2], y[3]);
            }
            bad += (x.x - x.x) + (x.y - x.y) + (x.z - x.z) + (x.w - x.w);
            *reinterpret_cast<float4 *>(p.o + (base + t0 + i / S::CB) * D + c0 + i % S::CB) = x;
        }
        if (bad != 0.f) flag(p.status, kFlagNonfinite);
        // os is next written behind the next block's staging barrier, so no third barrier is needed
    }
    if (!SUMS && end != len) return;
    float *to = SUMS ? record : pool, bad = 0.f;
#pragma unroll
    for (int i = 0; i < S::RW; ++i)
#pragma unroll
        for (int c = 0; c < CW; ++c) {
            to[row(i) + c] = s[i][c];
            bad += s[i][c] - s[i][c];
        }
    if (bad != 0.f) flag(p.status, kFlagNonfinite);
    if (SUMS && tid == 0 && c0 == 0) p.products[tile * p.segments + seg] = upto.packed();
}

// records[j] <- the state before segment j, for the segments that the prompt has. A thread per four
// entries goes along the segments; its loads of JOIN segments are in flight at once.
constexpr int JOIN = 8;
__global__ void __launch_bounds__(256) decay_join_kernel(const DecayParams p, const int d)
{
    wait_for_stream();
    const int n4 = d * d / 4, per = (n4 + 255) / 256;
    const int64_t tile = blockIdx.x / per;
    const int i = blockIdx.x % per * 256 + threadIdx.x;
    const int b = (int)(tile / p.H), h = (int)(tile - (int64_t)b * p.H);
    const int slot = p.slots[b], len = prompt_length(p, b);
    if (i >= n4 || slot < 0 || slot >= p.state_slots || len <= 0) return;
    const int n = (int)(((int64_t)len + p.seg_tokens - 1) / p.seg_tokens);
    float4 S = reinterpret_cast<const float4 *>(p.states + ((size_t)slot * p.H + h) * d * d)[i];
    float4 *rec = reinterpret_cast<float4 *>(p.records + (size_t)tile * p.segments * d * d) + i;
    const float2 *prod = p.products + tile * p.segments;
    for (int j0 = 0; j0 < n; j0 += JOIN) {
        float4 x[JOIN];
        float2 a[JOIN];
#pragma unroll
        for (int j = 0; j < JOIN; ++j)
            if (j0 + j < n - 1) {  // the last segment has no sum of its own
                x[j] = rec[(size_t)(j0 + j) * n4];
                a[j] = prod[j0 + j];
            }
        int far = 0;
#pragma unroll
        for (int j = 0; j < JOIN; ++j)
            if (j0 + j < n - 1) far |= __float_as_int(a[j].y);
        if (far == 0) {  // the usual case, free of branches along the states
#pragma unroll
            for (int j = 0; j < JOIN; ++j)
                if (j0 + j < n) {
                    rec[(size_t)(j0 + j) * n4] = S;
                    if (j0 + j < n - 1)
                        S = make_float4(fmaf(a[j].x, S.x, x[j].x), fmaf(a[j].x, S.y, x[j].y), fmaf(a[j].x, S.z, x[j].z),
                                        fmaf(a[j].x, S.w, x[j].w));
                }
            continue;
        }
        for (int j = j0; j < j0 + JOIN && j < n; ++j) {
            const float4 sum = rec[(size_t)j * n4];
            rec[(size_t)j * n4] = S;
            if (j < n - 1)
                S = make_float4(carry(prod[j], S.x, sum.x), carry(prod[j], S.y, sum.y), carry(prod[j], S.z, sum.z),
                                carry(prod[j], S.w, sum.w));
        }
    }
}

template <int D>
cudaError_t step(const DecayParams &p, int in_bf16, cudaStream_t s)
{
    const unsigned grid = (unsigned)((size_t)p.B * p.H);
    return launch_early(in_bf16 ? decay_step_kernel<D, 1> : decay_step_kernel<D, 0>, dim3(grid), StepCfg<D>::NT, 0, s, p);
}

template <int D, int IN_BF16, int CW>
cudaError_t serial(const DecayParams &p, bool sums, cudaStream_t s)
{
    using S = SerialCfg<D, CW>;
    const size_t tiles = (size_t)p.B * p.H;
    const unsigned gy = (unsigned)(tiles < 32768 ? tiles : 32768);
    const dim3 grid((unsigned)p.segments * (D / S::CB), gy, (unsigned)((tiles + gy - 1) / gy));
    return launch_early(sums ? decay_serial_kernel<D, IN_BF16, 1, CW> : decay_serial_kernel<D, IN_BF16, 0, CW>, grid, S::NT,
                        0, s, p);
}

template <int D, int CW>
cudaError_t serial(const DecayParams &p, int in_bf16, bool sums, cudaStream_t s)
{
    return in_bf16 ? serial<D, 1, CW>(p, sums, s) : serial<D, 0, CW>(p, sums, s);
}

// Four columns to a thread feed the FMAs from a quarter of the shared memory's reads, one to a thread
// makes four times the warps. With four and with one, 100 tokens: d = 128, 40 heads 28.4 and 29.6 us, 64 heads 28.4
// and 38.7; d = 64, 80 heads 18.9 and 17.8, 128 heads 19.0 and 23.1; d = 32, 200 heads 15.5 and 11.8, 256 heads 15.6
// and 14.9, 400 heads 18.7 and 22.1.
bool serial_wide(const DecayParams &p, int d)
{
    return (int64_t)p.B * p.H * p.segments * d > 50 * 128;
}

cudaError_t decay_join(const DecayParams &p, int d, cudaStream_t s)
{
    const int64_t grid = (int64_t)p.B * p.H * ((d * d / 4 + 255) / 256);
    return launch_early(decay_join_kernel, dim3((unsigned)grid), 256, 0, s, p, d);
}

// How a prompt is done: by chunks or token by token, in how many segments of how many tokens.
struct Split {
    bool chunk;
    int segments, seg_tokens;
};

constexpr int kSMs = 148;            // the workspace's size must not depend on the device in use
constexpr int kMostSegments = 1024;  // the join goes along them

// Whether a prompt goes by chunks, given its heads (over all requests) and whether it may be cut into segments. A
// chunk takes its time however few of its tokens there are, and a round of heads over the SMs takes it whole;
// token by token the time goes with the tokens, and with the heads only where they are many. Measured, us token by
// token / by chunks:
//   d = 128, from 32 tokens on: 128 heads 18.9 / 13.1, 512 heads 52 / 49 (32 tokens). Where heads are few the
//     latency of a token is all there is: 1 to 16 heads 10 / 13 (64 tokens), 14.0 / 13.1 (96); 32 heads 11.5 / 13.0
//     (48), 14.4 / 13.0 (64).
//   d = 64, from 64 on: 1 head 6.8 / 7.6, 64 heads 8.8 / 8.1, 512 heads 30.0 / 30.2.
//   d = 32, from 104 on: 1 head 6.5 / 7.0 (96), 8.2 / 7.1 (127), 256 heads 13.8 / 14.8 and 17.7 / 15.0; 400 heads 22
//     / 22 (112), 35 / 30 (192); 512 heads 36 / 38 (192), 47 / 39 (256); 1024 heads 66 / 70 (256), 98 / 94 (384).
//   d = 16: a chunk takes nearly d = 64's time for a sixteenth of its state, so token by token, 1024 heads 115 / 190 (1024
//     tokens), 110 heads 150 / 194 (8192), 16 heads 182 / 266 (65536); but 1 to 148 heads 9.1 / 6.7 (128) and
//     9.8 / 9.4 (256), and 1 head 50 / 36 (32768), 91 / 49 (65536). Without a cut a token takes 0.05 us, a chunk 2.7,
//     with up to two rounds of heads; 512 heads 85 / 106 (1024).
bool by_chunks(int64_t tiles, int T, int d, int in_bf16, bool cut)
{
    if (!in_bf16) return false;
    switch (d) {
        case 16:
            if (!cut) return T >= 128 && tiles <= 2 * kSMs;
            return (T >= 128 && T <= 256 && tiles <= kSMs) || (T >= 24576 && tiles <= 2);
        case 32: return T >= (tiles <= 256 ? 104 : tiles <= 448 ? 128 : 224);
        case 64: return T >= 64;
        default: return T >= (tiles < 24 ? 88 : tiles < 48 ? 56 : 32);
    }
}

// The most segments that a prompt of T tokens, or of fewer, is cut in by chunks and token by token. Neither falls
// with T: the workspace is sized for both, so that one made for the longest prompt serves every shorter one.
int most_chunk_segments(int64_t tiles, int T, int in_bf16)
{
    // A cut wins by filling the rounds of CTAs better: `gain` of a round for every chunk of the prompt, against
    // the best of no cut and one round. Each round more costs a CTA's start and end in both passes, 5.25
    // chunks' time. Two rounds beside that cover the rounding of chunks to segments (all choices of the
    // model below that have up to 4096 chunks are within the limit).
    const int64_t chunks = ((int64_t)T + kDecayChunk - 1) / kDecayChunk;
    if (!in_bf16 || chunks < 6 || tiles > 197) return 1;
    const int whole = (int)(tiles + kSMs - 1) / kSMs, one = kSMs / (int)tiles < 64 ? kSMs / (int)tiles : 64;
    const double gain = (one > 1 ? 1.5 / one : whole) - 1.5 * (double)tiles / kSMs;
    const double n = (whole + floor(((gain > 0.0 ? gain * (double)chunks : 0.0) + 12.0) / 5.25)) * kSMs / (double)tiles;
    const int64_t most = chunks < 64 ? chunks : 64;
    return n < (double)most ? (n > 1.0 ? (int)n : 1) : (int)most;
}

int most_serial_segments(int64_t tiles, int T, int d, int in_bf16)
{
    const int64_t ctas = tiles * (d > 64 ? d / 64 : 1);
    // CTAs to an SM (512 heads of 1024 tokens of d = 16: 165 us with 4, 152 with 8, 119 with 12)
    const int64_t want = d <= 32 ? 12 : 8;
    // bf16 prompts of d > 16 that go token by token are too short for a cut
    if (T < 128 || ctas > want * kSMs / 2 || (in_bf16 && d > 16)) return 1;
    int64_t n = want * kSMs / ctas;
    n = n < T / 64 ? n : T / 64;
    return (int)(n < kMostSegments ? n : kMostSegments);
}

Split split(int B, int H, int T, int d, int in_bf16, bool cut)
{
    const int64_t tiles = (int64_t)B * H;
    Split r{by_chunks(tiles, T, d, in_bf16, cut), 1, T};
    const int64_t most = !cut ? 1 : r.chunk ? most_chunk_segments(tiles, T, in_bf16) : most_serial_segments(tiles, T, d, in_bf16);
    if (r.chunk) {
        // One CTA to an SM: rounds of CTAs, each its chunks and 3.5 chunks' time of start and end (20 us; 5.5
        // us a chunk). The first pass takes half of the main one's time, the join 1.5 chunks' and 0.15 a
        // segment.
        const int64_t chunks = ((int64_t)T + kDecayChunk - 1) / kDecayChunk, ctas = tiles;
        double best = 0.0;
        int64_t per = chunks;
        for (int64_t n = 1; n <= most; ++n) {
            const int64_t c = (chunks + n - 1) / n;
            if ((chunks + c - 1) / c != n) continue;  // fewer segments of this length do
            double t = (double)((ctas * n + kSMs - 1) / kSMs) * ((double)c + 3.5);
            if (n > 1) t += 0.5 * (double)((ctas * (n - 1) + kSMs - 1) / kSMs) * ((double)c + 3.5) + 1.5 + 0.15 * n;
            if (n == 1 || t < best) best = t, per = c;
        }
        r.segments = (int)((chunks + per - 1) / per);
        r.seg_tokens = (int)(per * kDecayChunk < 0x7fffffff ? per * kDecayChunk : 0x7fffff80);
        return r;
    }
    if (most == 1) return r;
    const int64_t per = (((int64_t)T + most - 1) / most + 31) / 32 * 32;
    r.segments = (int)((T + per - 1) / per);
    r.seg_tokens = (int)per;
    return r;
}

// Bytes of the records and products of so many segments a prompt.
size_t split_bytes(int segments, int B, int H, int d)
{
    return segments > 1 ? (size_t)B * H * segments * ((size_t)d * d + 2) * sizeof(float) : 0;
}

}  // namespace

cudaError_t launch_decay_serial(const DecayParams &p, int d, int in_bf16, bool sums, cudaStream_t s)
{
    const bool wide = serial_wide(p, d);
    switch (d) {
        case 16: return serial<16, 1>(p, in_bf16, sums, s);
        case 32: return wide ? serial<32, 4>(p, in_bf16, sums, s) : serial<32, 1>(p, in_bf16, sums, s);
        case 64: return wide ? serial<64, 4>(p, in_bf16, sums, s) : serial<64, 1>(p, in_bf16, sums, s);
        default: return wide ? serial<128, 4>(p, in_bf16, sums, s) : serial<128, 1>(p, in_bf16, sums, s);
    }
}

}  // namespace stq

namespace {

bool decay_aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) % 16) == 0; }

// Arguments that both forms share; `work` is false for a call without any.
stq_status check_decay(int32_t B, int32_t H, int32_t T, int32_t d, int32_t in_dtype, const float *states,
                       int32_t state_slots, const int32_t *slots, const void *q, const void *k, const void *v,
                       const float *alpha, const float *o, bool *work)
{
    *work = false;
    if (B < 0 || H < 1 || T < 0 || state_slots < 0 || (in_dtype != STQ_F32 && in_dtype != STQ_BF16))
        return STQ_ERR_INVALID_ARG;
    if (!(d == 16 || d == 32 || d == 64 || d == 128)) return STQ_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return STQ_OK;
    if (!states || !slots || !q || !k || !v || !alpha || !o) return STQ_ERR_INVALID_ARG;
    if (!decay_aligned(states) || !decay_aligned(q) || !decay_aligned(k) || !decay_aligned(v) || !decay_aligned(o) ||
        (reinterpret_cast<uintptr_t>(alpha) % 4) || (reinterpret_cast<uintptr_t>(slots) % 4))
        return STQ_ERR_INVALID_ARG;
    if (B > 2147483647 / H) return STQ_ERR_UNSUPPORTED;
    *work = true;
    return STQ_OK;
}

stq::DecayParams decay_params(int32_t B, int32_t H, int32_t T, float *states, int32_t state_slots,
                              const int32_t *slots, const void *q, const void *k, const void *v, const float *alpha,
                              const int32_t *lens, float *o, int32_t *dev_status)
{
    stq::DecayParams p{};
    p.B = B;
    p.H = H;
    p.T = T;
    p.states = states;
    p.state_slots = state_slots;
    p.slots = slots;
    p.q = q;
    p.k = k;
    p.v = v;
    p.alpha = alpha;
    p.lens = lens;
    p.o = o;
    p.status = dev_status;
    return p;
}

}  // namespace

extern "C" stq_status stq_decay_step(int32_t B, int32_t H, int32_t d, int32_t in_dtype, float *states,
                                     int32_t state_slots, const int32_t *slots, const void *q, const void *k,
                                     const void *v, const float *alpha, float *o, int32_t *dev_status, void *stream)
{
    bool work;
    const stq_status st = check_decay(B, H, 1, d, in_dtype, states, state_slots, slots, q, k, v, alpha, o, &work);
    if (st != STQ_OK || !work) return st;
    const stq::DecayParams p =
        decay_params(B, H, 1, states, state_slots, slots, q, k, v, alpha, nullptr, o, dev_status);
    const int bf = in_dtype == STQ_BF16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (d) {
        case 16: e = stq::step<16>(p, bf, s); break;
        case 32: e = stq::step<32>(p, bf, s); break;
        case 64: e = stq::step<64>(p, bf, s); break;
        default: e = stq::step<128>(p, bf, s); break;
    }
    return e == cudaSuccess ? STQ_OK : STQ_ERR_CUDA;
}

extern "C" size_t stq_decay_prefill_workspace_bytes(int32_t B, int32_t H, int32_t T, int32_t d, int32_t in_dtype)
{
    if (B < 1 || H < 1 || T < 1 || B > 2147483647 / H || (in_dtype != STQ_F32 && in_dtype != STQ_BF16)) return 0;
    if (!(d == 16 || d == 32 || d == 64 || d == 128)) return 0;
    const int bf = in_dtype == STQ_BF16, c = stq::most_chunk_segments((int64_t)B * H, T, bf);
    const int s = stq::most_serial_segments((int64_t)B * H, T, d, bf);
    return stq::split_bytes(c > s ? c : s, B, H, d);
}

extern "C" stq_status stq_decay_prefill(int32_t B, int32_t H, int32_t T, int32_t d, int32_t in_dtype, float *states,
                                        int32_t state_slots, const int32_t *slots, const void *q, const void *k,
                                        const void *v, const float *alpha, const int32_t *lens, float *o,
                                        void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    bool work;
    const stq_status st = check_decay(B, H, T, d, in_dtype, states, state_slots, slots, q, k, v, alpha, o, &work);
    if (st != STQ_OK || !work) return st;
    if (reinterpret_cast<uintptr_t>(lens) % 4) return STQ_ERR_INVALID_ARG;
    const int bf = in_dtype == STQ_BF16;
    const size_t need = stq_decay_prefill_workspace_bytes(B, H, T, d, in_dtype);
    if (workspace && need && (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256))
        return STQ_ERR_INVALID_ARG;
    const stq::Split cut = stq::split(B, H, T, d, bf, workspace != nullptr);
    stq::DecayParams p = decay_params(B, H, T, states, state_slots, slots, q, k, v, alpha, lens, o, dev_status);
    p.segments = cut.segments;
    p.seg_tokens = cut.seg_tokens;
    if (cut.segments > 1) {
        p.records = static_cast<float *>(workspace);
        p.products = reinterpret_cast<float2 *>(p.records + (size_t)B * H * cut.segments * d * d);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto pass = [&](bool sums) {
        cudaError_t e = cut.chunk ? stq::launch_decay_chunk(p, d, sums, s) : cudaErrorNotSupported;
        if (e == cudaErrorNotSupported) e = stq::launch_decay_serial(p, d, bf, sums, s);
        return e;
    };
    cudaError_t e = cudaSuccess;
    if (cut.segments > 1) {
        e = pass(true);
        if (e == cudaSuccess) e = stq::decay_join(p, d, s);
    }
    if (e == cudaSuccess) e = pass(false);
    return e == cudaSuccess ? STQ_OK : STQ_ERR_CUDA;
}
