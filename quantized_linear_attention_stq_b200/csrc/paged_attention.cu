// paged_attention.cu -- attention of one new token per request over a paged key-value cache
// (stq_paged_attention; contract in include/stq.h).
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - m),  m = max_t scale q.k_t
//
// One pass over the cache with the running maximum and sum of the softmax: a tile's scores raise
// the maximum from m to m', what was summed so far is scaled by exp(m - m'). Exponentials are taken
// in base 2, with scale * log2(e) multiplied into the scores. Bound by HBM: every cached key and
// value is read once for all the query heads that share it.
//
// bf16 caches go through the warp-level matrix instructions (16 query rows x 16 keys): with one new
// token a unit has 16 rows at most, an eighth of what a tcgen05 tile is tall, and the products are
// a small part of the time that the bytes take. Weights enter the second product as bf16 terms
// whose sum is the fp32 weight, so that o keeps fp32's accuracy. fp32 caches go through fp32 FMAs.
#include "../../include/stq.h"
#include "stq_paged.cuh"
#include "stream_order.cuh"

namespace stq {
namespace {

using namespace paged;

constexpr int NTA = 128;
constexpr int KT = 32;  // keys staged at a time
static_assert(TK % KT == 0, "a tile is a whole number of stages");

// Where a block stands on the line of tiles.
struct Cursor {
    long long begin, end;  // its share
    long long total;
    int b;                 // request of `begin`
    long long before;      // tiles (per unit) of the requests before b
};

// The block's share: the total by one pass over the lengths, then the request that `begin` falls in.
// `first_tile` is written by block 0. Called by all threads; ends with a barrier.
__device__ __forceinline__ Cursor find_share(const Params &p, int units)
{
    __shared__ long long red[NTA / 32];
    __shared__ Cursor cur;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const bool writer = blockIdx.x == 0;
    if (p.B <= NTA) {  // one look at the lengths does
        bool bad = false;
        const int nt = tid < p.B ? tiles_of(cached_length(p, tid, &bad)) : 0;
        if (bad && writer) flag(p.status, kFlagBounds);
        long long x = nt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) red[w] = x;
        __syncthreads();
        long long upto = x, all = 0;
#pragma unroll
        for (int i = 0; i < NTA / 32; ++i) {
            if (i < w) upto += red[i];
            all += red[i];
        }
        const long long mine = upto - nt, total = all * units;
        const int C = busy_blocks(total, gridDim.x), c = min((int)blockIdx.x, C);
        const long long begin = share_begin(total, c, C), end = share_begin(total, min(c + 1, C), C);
        if (writer && tid < p.B) p.first_tile[tid] = mine;
        if (writer && tid == 0) p.first_tile[p.B] = all;
        const bool here = tid < p.B && mine * units <= begin && begin < upto * units;  // of one thread at most
        if (here) cur = Cursor{begin, end, total, tid, mine};
        if (!__syncthreads_or(here) && tid == 0) cur = Cursor{begin, end, total, p.B, all};
        __syncthreads();
        return cur;
    }
    long long sum = 0;
    for (int b0 = 0; b0 < p.B; b0 += NTA) {
        const int b = b0 + tid;
        bool bad = false;
        const int nt = b < p.B ? tiles_of(cached_length(p, b, &bad)) : 0;
        if (bad && writer) flag(p.status, kFlagBounds);
        sum += nt;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) red[w] = sum;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < NTA / 32; ++i) total += red[i];
    total *= units;
    const int C = busy_blocks(total, gridDim.x), c = min((int)blockIdx.x, C);
    const long long begin = share_begin(total, c, C), end = share_begin(total, min(c + 1, C), C);
    __syncthreads();
    long long before = 0;
    if (tid == 0) {
        cur.begin = begin;
        cur.end = end;
        cur.total = total;
        cur.b = p.B;
    }
    for (int b0 = 0; b0 < p.B; b0 += NTA) {
        const int b = b0 + tid;
        bool bad;
        const int nt = b < p.B ? tiles_of(cached_length(p, b, &bad)) : 0;
        long long x = nt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) red[w] = x;
        __syncthreads();
        long long upto = before + x, all = before;
#pragma unroll
        for (int i = 0; i < NTA / 32; ++i) {
            if (i < w) upto += red[i];
            all += red[i];
        }
        const long long mine = upto - nt;
        if (writer && b < p.B) p.first_tile[b] = mine;
        if (b < p.B && mine * units <= begin && begin < upto * units) {
            cur.b = b;
            cur.before = mine;
        }
        before = all;
        __syncthreads();
        if (!writer && (begin >= end || before * units > begin)) break;
    }
    if (writer && tid == 0) p.first_tile[p.B] = before;
    __syncthreads();
    return cur;
}

template <int D, int GT>
struct SimtSmem {
    float q[GT][D];
    float k[2][KT][D + 4];
    float v[2][KT][D];
    long long at[3][KT];  // where a stage's keys stand; -1: none
    float s[4][GT][KT];  // partial scores of the four quarters of d
    float p[GT][KT];
    float corr[GT], m[GT], l[GT];
    static_assert(2 * KT * (D + 4) >= GT * D, "the joined sums fit where the keys were");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// One unit's tiles [t0, t1): scores by quarters of d (a lane per key, a warp per quarter), softmax
// by rows, products by (columns, key class). Copies run a stage ahead, the look-up of the pages one
// further. Leaves the sums in acc, joined over the key classes, in shared memory (sums[GT][D]), and m, l.
template <int D, int GT>
__device__ __forceinline__ void simt_unit(const Params &p, SimtSmem<D, GT> &sm, int b, int hk, int rt, int len,
                                          int t0, int t1, float *sums)
{
    constexpr int C4 = D / 4, PARTS = NTA / C4;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int c4 = tid % C4, part = tid / C4;
    const int rows = min(GT, p.group - rt * ROWS);
    const size_t q0 = ((size_t)b * p.Hq + (size_t)hk * p.group + rt * ROWS) * D;
    const int32_t *row = p.table + (size_t)b * p.W;
    const int first = t0 * TK, last = min(len, t1 * TK), N = (last - first + KT - 1) / KT;
    auto look_up = [&](int n) {  // warp 0: the places of stage n's keys
        // unsigned: the look-up runs up to 94 tokens past the last, which may be close to int32's end
        const unsigned t = (unsigned)first + (unsigned)(n * KT + lane);
        long long at = -1;
        if (t < (unsigned)last) {
            const int pg = row[t / (unsigned)p.page];
            if (pg >= 0 && pg < p.num_pages)
                at = (((long long)pg * p.Hkv + hk) * p.page + t % (unsigned)p.page) * D;
            else
                flag(p.status, kFlagBounds);
        }
        sm.at[n % 3][lane] = at;
    };
    auto copy = [&](int n) {
#pragma unroll
        for (int x = 0; x < KT * C4 / NTA; ++x) {
            const int i = tid + x * NTA, r = i / C4, c = 4 * (i % C4);
            const long long at = sm.at[n % 3][r];
            const long long from = at < 0 ? 0 : at + c;
            cp16(smem_u32(&sm.k[n & 1][r][c]), (const float *)p.k_pages + from, at >= 0);
            cp16(smem_u32(&sm.v[n & 1][r][c]), (const float *)p.v_pages + from, at >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();  // the unit before has been read out
    if (w == 0) {
        look_up(0);
        look_up(1);
    }
    for (int i = tid; i < GT * D; i += NTA) (&sm.q[0][0])[i] = i < rows * D ? ((const float *)p.q)[q0 + i] : 0.f;
    if (tid < GT) {
        sm.m[tid] = -INFINITY;
        sm.l[tid] = 0.f;
    }
    float acc[GT][4];
#pragma unroll
    for (int g = 0; g < GT; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][e] = 0.f;
    __syncthreads();
    copy(0);
    for (int n = 0; n < N; ++n) {
        if (n + 1 < N) {
            copy(n + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const float(*ks)[D + 4] = sm.k[n & 1];
        const float(*vs)[D] = sm.v[n & 1];
        {  // scores: lane = key, warp = quarter of d
            float s[GT];
#pragma unroll
            for (int g = 0; g < GT; ++g) s[g] = 0.f;
#pragma unroll
            for (int c = 0; c < C4 / 4; ++c) {
                const int col = (w * (C4 / 4) + c) * 4;
                const float4 kk = *reinterpret_cast<const float4 *>(&ks[lane][col]);
#pragma unroll
                for (int g = 0; g < GT; ++g) {
                    const float4 qq = *reinterpret_cast<const float4 *>(&sm.q[g][col]);
                    s[g] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[g]))));
                }
            }
#pragma unroll
            for (int g = 0; g < GT; ++g) sm.s[w][g][lane] = s[g];
        }
        if (w == 0) look_up(n + 2);
        __syncthreads();
        for (int g = w; g < GT; g += NTA / 32) {
            float s = (sm.s[0][g][lane] + sm.s[1][g][lane]) + (sm.s[2][g][lane] + sm.s[3][g][lane]);
            s = sm.at[n % 3][lane] >= 0 ? s * p.scale2 : -INFINITY;
            float top = s;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float m0 = sm.m[g], m1 = fmaxf(m0, top);
            const float base = m1 == -INFINITY ? 0.f : m1;  // nothing to weigh yet
            const float e = exp2f(s - base), corr = exp2f(m0 - base);
            float sum = e;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            sm.p[g][lane] = e;
            __syncwarp();
            if (lane == 0) {
                sm.m[g] = m1;
                sm.corr[g] = corr;
                sm.l[g] = fmaf(sm.l[g], corr, sum);
            }
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            const float c = sm.corr[g];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[g][e] *= c;
        }
#pragma unroll 4
        for (int r = part; r < KT; r += PARTS) {
            const float4 vv = *reinterpret_cast<const float4 *>(&vs[r][4 * c4]);
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                const float e = sm.p[g][r];
                acc[g][0] = fmaf(e, vv.x, acc[g][0]);
                acc[g][1] = fmaf(e, vv.y, acc[g][1]);
                acc[g][2] = fmaf(e, vv.z, acc[g][2]);
                acc[g][3] = fmaf(e, vv.w, acc[g][3]);
            }
        }
        __syncthreads();  // the stage is overwritten next
    }
    // join the key classes, one class at a time (a fixed order)
    for (int r = 0; r < PARTS; ++r) {
        __syncthreads();
        if (part == r)
#pragma unroll
            for (int g = 0; g < GT; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &x = sums[g * D + 4 * c4 + e];
                    x = r == 0 ? acc[g][e] : x + acc[g][e];
                }
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------------------------
// bf16 caches
// ---------------------------------------------------------------------------------------------
constexpr int SUB = 16;  // keys of a warp's step; the block's four warps take a tile's four quarters
static_assert(TK == SUB * (NTA / 32), "a tile is one step of every warp");

// How the three bf16 terms of the weights (h + m + l, 24 significand bits) are laid on the 16 rows:
// rows of the query tile that a group leaves free take further terms of the same rows, whose
// scores are computed alongside.
//   group <= 4: rows 0..3 h, 4..7 m, 8..11 l   one product
//   group <= 8: rows 0..7 h, 8..15 m; then l   two products
//   else:       three products
template <int GROUP>
struct Terms {
    static constexpr int PERIOD = GROUP;  // row % PERIOD is the query head
    static constexpr int PRODUCTS = GROUP == 4 ? 1 : GROUP == 8 ? 2 : 3;
};

// Blocks on an SM, by shared memory and registers.
constexpr int mma_blocks(int d) { return d == 128 ? 2 : d == 64 ? 3 : 4; }

template <int D>
struct MmaCfg {
    static constexpr int CH = D / 8;                   // 16-byte chunks of a row
    static constexpr int HALF = SUB * D * 2;           // bytes of a step's keys (or values)
    static constexpr int STAGES = D == 128 ? 3 : 4;
    static constexpr int WARP_BYTES = STAGES * 2 * HALF;
    static constexpr int RING = (NTA / 32) * WARP_BYTES;
    static constexpr int SUMS = (NTA / 32) * ROWS * (D + 4) * 4;  // the warps' sums, where the ring was
    static constexpr int MAIN = RING > SUMS ? RING : SUMS;
    static constexpr int OUT = ROWS * D * 4;
    static constexpr int SMEM = MAIN + OUT + (NTA / 32 + 1) * ROWS * 2 * 4 + (NTA / 32) * STAGES * 4;
};

// Byte offset of chunk c of row r: rows of 128 bytes or more are swizzled by r % 8, shorter ones by
// their 128-byte line, so that 8 rows' same chunk falls on 8 different 16-byte banks.
template <int D>
__device__ __forceinline__ uint32_t row_chunk(int r, int c)
{
    constexpr int CH = MmaCfg<D>::CH, PER = CH >= 8 ? 1 : 8 / CH, MASK = (CH >= 8 ? 8 : CH) - 1;
    return (uint32_t)(r * CH + (c ^ ((r / PER) & MASK))) * 16u;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf2(float x, float y)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// What rounding (x, y) to the packed bf16 pair v leaves over.
__device__ __forceinline__ void rest2(uint32_t v, float &x, float &y)
{
    x -= __uint_as_float(v << 16);
    y -= __uint_as_float(v & 0xFFFF0000u);
}

// One unit's tiles [t0, t1): every warp takes its 16 keys of each tile through its own ring of
// asynchronous copies and keeps its own maximum, sum and products; joined at the end into
// sums[ROWS][D], m, l (shared memory).
template <int D, int GROUP>
__device__ __forceinline__ void mma_unit(const Params &p, uint8_t *smem, int b, int hk, int rt, int len, int t0, int t1,
                                         float *sums, float *m_out, float *l_out)
{
    using M = MmaCfg<D>;
    using T = Terms<GROUP>;
    constexpr int KS = D / 16, NT = D / 8, PC = SUB * M::CH / 32;  // k steps, column tiles, copies of a lane
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, r = lane >> 2, qd = lane & 3;
    const int rows = min(ROWS, p.group - rt * ROWS);
    const uint32_t ring = smem_u32(smem) + (uint32_t)w * M::WARP_BYTES;
    float *wm = l_out + ROWS, *wl = wm + (NTA / 32) * ROWS;  // the warps' maxima and sums
    volatile uint32_t *masks = reinterpret_cast<uint32_t *>(wl + (NTA / 32) * ROWS) + w * M::STAGES;
    __syncthreads();  // the unit before has been read out

    uint32_t qa[KS][4];
    {
        const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.q + ((size_t)b * p.Hq + (size_t)hk * p.group + rt * ROWS) * D;
        const int g0 = r % T::PERIOD, g1 = (r + 8) % T::PERIOD;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = 16 * k + 8 * h + 2 * qd;
                qa[k][2 * h] = g0 < rows ? *reinterpret_cast<const uint32_t *>(q + g0 * D + col) : 0u;
                qa[k][2 * h + 1] = g1 < rows ? *reinterpret_cast<const uint32_t *>(q + g1 * D + col) : 0u;
            }
    }
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // of rows r and r + 8; sums per lane

    const int32_t *row = p.table + (size_t)b * p.W;
    const int steps = t1 - t0;
    const size_t head = (size_t)hk * p.page;
    // the page of this lane's key (lanes 16.. repeat 0..) at a step; -1 behind the end
    auto page_at = [&](int j) {
        const int t = (t0 + j) * TK + w * SUB + (lane & 15);
        return j < steps && t < len ? row[t / p.page] : -1;
    };
    // copy a step's keys and values into ring slot `slot`
    auto fetch = [&](int j, int slot, int pg) {
        const int t = (t0 + j) * TK + w * SUB + (lane & 15);
        const bool in = j < steps && t < len, live = in && pg >= 0 && pg < p.num_pages;
        if (in && !live) flag(p.status, kFlagBounds);
        const uint32_t mask = __ballot_sync(0xffffffffu, live);
        const size_t at = live ? ((size_t)pg * p.Hkv * p.page + head + t % p.page) * D : 0;
        if (lane == 0) masks[slot] = mask & 0xffffu;
        const uint32_t dst = ring + (uint32_t)slot * (2 * M::HALF);
#pragma unroll
        for (int i = 0; i < PC; ++i) {
            const int c = i * 32 + lane, kr = c / M::CH, ch = c % M::CH;
            const size_t src = __shfl_sync(0xffffffffu, (unsigned long long)at, kr) + ch * 8;
            const bool ok = (mask >> kr) & 1u;
            cp16(dst + row_chunk<D>(kr, ch), (const __nv_bfloat16 *)p.k_pages + src, ok);
            cp16(dst + M::HALF + row_chunk<D>(kr, ch), (const __nv_bfloat16 *)p.v_pages + src, ok);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    int pg = page_at(0);
#pragma unroll
    for (int j = 0; j < M::STAGES - 1; ++j) {
        const int next = page_at(j + 1);
        fetch(j, j, pg);
        pg = next;
    }
    int slot = 0;
    for (int j = 0; j < steps; ++j) {
        const int next = page_at(j + M::STAGES);
        asm volatile("cp.async.wait_group %0;" ::"n"(M::STAGES - 2) : "memory");
        __syncwarp();
        const uint32_t mask = masks[slot];
        const uint32_t kb = ring + (uint32_t)slot * (2 * M::HALF), vb = kb + M::HALF;
        // scores of 16 keys: two column tiles of 8, even and odd k steps in chains of their own
        float s[2][2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[h][n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t f[4];  // keys 0..7 (chunks 2k, 2k + 1), keys 8..15
            ldsm4(f, kb + row_chunk<D>((lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)));
            mma16816(s[k & 1][0], qa[k], f[0], f[1]);
            mma16816(s[k & 1][1], qa[k], f[2], f[3]);
        }
        float x[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool live = (mask >> (8 * n + 2 * qd + (e & 1))) & 1u;
                x[n][e] = live ? (s[0][n][e] + s[1][n][e]) * p.scale2 : -INFINITY;
            }
        float u0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        float u1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, d));
            u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, d));
        }
        const float n0 = fmaxf(m0, u0), n1 = fmaxf(m1, u1);
        const float c0 = n0 == -INFINITY ? 1.f : exp2f(m0 - n0), c1 = n1 == -INFINITY ? 1.f : exp2f(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= c0;
        l1 *= c1;
        const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            x[n][0] = exp2f(x[n][0] - b0);
            x[n][1] = exp2f(x[n][1] - b0);
            x[n][2] = exp2f(x[n][2] - b1);
            x[n][3] = exp2f(x[n][3] - b1);
            l0 += x[n][0] + x[n][1];
            l1 += x[n][2] + x[n][3];
        }
        // the weights' terms as rows of the first operand: keys 0..7 in a[0], a[1], keys 8..15 in a[2], a[3]
        uint32_t ta[3][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float &y0 = x[n][2 * h], &y1 = x[n][2 * h + 1];
                const uint32_t t0b = bf2(y0, y1);
                rest2(t0b, y0, y1);
                const uint32_t t1b = bf2(y0, y1);
                rest2(t1b, y0, y1);
                const uint32_t t2b = bf2(y0, y1);
                const int at = 2 * n + h;
                if constexpr (GROUP == 4) {
                    ta[0][at] = h == 0 ? (r < 4 ? t0b : t1b) : (r < 4 ? t2b : 0u);
                } else if constexpr (GROUP == 8) {
                    ta[0][at] = h == 0 ? t0b : t1b;
                    ta[1][at] = h == 0 ? t2b : 0u;
                } else {
                    ta[0][at] = t0b;
                    ta[1][at] = t1b;
                    ta[2][at] = t2b;
                }
            }
        // Products of one step go to sums of their own, which are added to the running ones by fp32
        // FMAs with the rescaling: the matrix instruction truncates the sum it is given, and over a
        // long cache that bias adds up (500,001 keys: 4.3e-6 of the result, against 6e-7 this way).
        constexpr int NB = NT < 4 ? NT : 4;  // column tiles at a time, so that the terms' chains overlap
#pragma unroll
        for (int n = 0; n < NT; n += NB) {
            float y[NB][4];
            uint32_t f[NB / 2][4];  // columns 8n.. : keys 0..7, 8..15; columns 8n + 8.. : the same
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) ldsm4t(f[i], vb + row_chunk<D>(lane & 15, n + 2 * i + (lane >> 4)));
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[i][e] = 0.f;
#pragma unroll
            for (int t = T::PRODUCTS - 1; t >= 0; --t)
#pragma unroll
                for (int i = 0; i < NB; ++i) mma16816(y[i], ta[t], f[i / 2][2 * (i & 1)], f[i / 2][2 * (i & 1) + 1]);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                acc[n + i][0] = fmaf(acc[n + i][0], c0, y[i][0]);
                acc[n + i][1] = fmaf(acc[n + i][1], c0, y[i][1]);
                acc[n + i][2] = fmaf(acc[n + i][2], c1, y[i][2]);
                acc[n + i][3] = fmaf(acc[n + i][3], c1, y[i][3]);
            }
        }
        __syncwarp();  // every lane has read the slot that is filled next
        const int fill = slot == 0 ? M::STAGES - 1 : slot - 1;
        fetch(j + M::STAGES - 1, fill, pg);
        pg = next;
        slot = slot + 1 == M::STAGES ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    __syncthreads();  // the rings are done with
    float *ws = reinterpret_cast<float *>(smem) + w * (ROWS * (D + 4));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2 *>(ws + r * (D + 4) + 8 * n + 2 * qd) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2 *>(ws + (r + 8) * (D + 4) + 8 * n + 2 * qd) = make_float2(acc[n][2], acc[n][3]);
    }
    if (qd == 0) {
        wm[w * ROWS + r] = m0;
        wm[w * ROWS + r + 8] = m1;
        wl[w * ROWS + r] = l0;
        wl[w * ROWS + r + 8] = l1;
    }
    __syncthreads();
    // join the four warps, and the terms that lie on rows of their own
    const float *all = reinterpret_cast<const float *>(smem);
    constexpr int TERM_ROWS = GROUP == 4 ? 3 : GROUP == 8 ? 2 : 1;
    for (int i = tid; i < rows * D; i += NTA) {
        const int g = i / D, c = i % D;
        float m = wm[g];
#pragma unroll
        for (int v = 1; v < NTA / 32; ++v) m = fmaxf(m, wm[v * ROWS + g]);
        const float base = m == -INFINITY ? 0.f : m;
        float sum = 0.f, l = 0.f;
#pragma unroll
        for (int v = 0; v < NTA / 32; ++v) {
            const float e = exp2f(wm[v * ROWS + g] - base);
            float part = 0.f;
#pragma unroll
            for (int t = TERM_ROWS - 1; t >= 0; --t) part += all[(v * ROWS + g + t * GROUP) * (D + 4) + c];
            sum = fmaf(e, part, sum);
            l = fmaf(e, wl[v * ROWS + g], l);
        }
        sums[i] = sum;
        if (c == 0) {
            m_out[g] = m;
            l_out[g] = l;
        }
    }
    __syncthreads();
}

// Writes a finished unit's output, or a piece of it for the join.
template <int D>
__device__ __forceinline__ void finish(const Params &p, int b, int hk, int rt, const float *sums, const float *m,
                                       const float *l, int piece)
{
    const int rows = min(ROWS, p.group - rt * ROWS);
    if (piece >= 0) {
        float *out = p.pieces + ((size_t)blockIdx.x * 2 + piece) * ROWS * (D + 2);
        for (int i = threadIdx.x; i < rows * D; i += NTA) out[i] = sums[i];
        for (int i = threadIdx.x; i < rows; i += NTA) {
            out[ROWS * D + i] = m[i];
            out[ROWS * D + ROWS + i] = l[i];
        }
        return;
    }
    float *o = p.o + ((size_t)b * p.Hq + (size_t)hk * p.group + rt * ROWS) * D;
    bool bad = false;
    for (int i = threadIdx.x; i < rows * D; i += NTA) {
        const float t = l[i / D];
        const float x = t == 0.f ? 0.f : sums[i] / t;
        bad |= !(fabsf(x) <= 3.402823466e38f);
        o[i] = x;
    }
    if (bad) flag(p.status, kFlagNonfinite);
}

// Calls unit(b, hk, rt, len, first tile, end tile, piece) for the block's work.
template <class Unit>
__device__ __forceinline__ void walk(const Params &p, Unit unit)
{
    wait_for_stream();
    const int units = p.Hkv * p.row_tiles;
    if (!p.split) {
        const int u = blockIdx.x % units, b = blockIdx.x / units;
        bool bad;
        const int len = cached_length(p, b, &bad);
        if (bad && threadIdx.x == 0) flag(p.status, kFlagBounds);
        unit(b, u / p.row_tiles, u % p.row_tiles, len, 0, tiles_of(len), -1);
        return;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up; it waits
    const Cursor cur = find_share(p, units);
    long long at = cur.begin, before = cur.before;
    for (int b = cur.b; at < cur.end; ++b) {
        bool bad;
        const int len = cached_length(p, b, &bad), nt = tiles_of(len);
        const long long r0 = before * units;  // the request's first tile
        while (at < cur.end && at < r0 + (long long)nt * units) {
            const int u = (int)((at - r0) / nt);
            const long long s = r0 + (long long)u * nt, e = s + nt, stop = e < cur.end ? e : cur.end;
            unit(b, u / p.row_tiles, u % p.row_tiles, len, (int)(at - s), (int)(stop - s),
                 at == s && stop == e ? -1 : s < cur.begin ? 0 : 1);
            at = stop;
        }
        before += nt;
    }
}

template <int D, int GT>
__global__ void __launch_bounds__(NTA) paged_simt_kernel(const Params p)
{
    extern __shared__ __align__(16) uint8_t raw[];
    SimtSmem<D, GT> &sm = *reinterpret_cast<SimtSmem<D, GT> *>(raw);
    float *sums = &sm.k[0][0][0];  // a unit's sums are joined where its keys were
    walk(p, [&](int b, int hk, int rt, int len, int t0, int t1, int piece) {
        simt_unit<D, GT>(p, sm, b, hk, rt, len, t0, t1, sums);
        finish<D>(p, b, hk, rt, sums, sm.m, sm.l, piece);
    });
}

template <int D, int GROUP>
__global__ void __launch_bounds__(NTA, mma_blocks(D)) paged_mma_kernel(const Params p)
{
    extern __shared__ __align__(128) uint8_t raw[];
    float *sums = reinterpret_cast<float *>(raw + MmaCfg<D>::MAIN), *m = sums + ROWS * D, *l = m + ROWS;
    walk(p, [&](int b, int hk, int rt, int len, int t0, int t1, int piece) {
        mma_unit<D, GROUP>(p, raw, b, hk, rt, len, t0, t1, sums, m, l);
        finish<D>(p, b, hk, rt, sums, m, l, piece);
    });
}

// Joins the pieces of the units that were cut, and zeroes the rows of requests without tokens. One
// block per (request, query head): d columns x NTJ / d classes of pieces, joined in a fixed order.
constexpr int NTJ = 256;
__global__ void __launch_bounds__(NTJ) paged_join_kernel(const Params p, int d, int most_blocks)
{
    __shared__ float weight[kMaxBlocks], red[NTJ], lsum[NTJ];
    __shared__ float4 sums[NTJ];
    // started while the attention kernel runs; every thread waits for its end, so that what follows
    // on the stream follows both
    wait_for_stream();
    const int units = p.Hkv * p.row_tiles;
    const int row = blockIdx.x % p.Hq, b = blockIdx.x / p.Hq, tid = threadIdx.x;
    const int hk = row / p.group, g = row % p.group, rt = g / ROWS, r = g % ROWS;
    const long long f0 = p.first_tile[b], nt = p.first_tile[b + 1] - f0, total = p.first_tile[p.B] * units;
    float *o = p.o + ((size_t)b * p.Hq + row) * d;
    if (nt == 0) {
        if (tid < d) o[tid] = 0.f;
        return;
    }
    const int blocks = busy_blocks(total, most_blocks);
    const long long s = f0 * units + (hk * p.row_tiles + rt) * nt;
    const int c0 = block_of(total, s, blocks), n = block_of(total, s + nt - 1, blocks) - c0 + 1;
    if (n == 1) return;  // finished by that block
    // the unit goes on behind the first block's share, and began before the others'
    const size_t stride = (size_t)ROWS * (d + 2);
    const float *first = p.pieces + (size_t)c0 * 2 * stride;
    auto piece = [&](int i) { return first + (i == 0 ? stride : 2 * stride * i); };
    if (n <= 32) {
        // few pieces: a warp has the weights of all, and no load waits for another (1 request of 1000
        // tokens: 10.0 us so far, 9.1 this way, with the attention)
        const int c = tid % d, cls = tid / d, classes = NTJ / d, lane = tid & 31;
        const float mi = lane < n ? piece(lane)[ROWS * d + r] : -INFINITY;
        const float li = lane < n ? piece(lane)[ROWS * d + ROWS + r] : 0.f;
        float x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = cls + k * classes < n ? piece(cls + k * classes)[r * d + c] : 0.f;
        float m = mi;
#pragma unroll
        for (int h = 16; h > 0; h >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, h));
        const float w = exp2f(mi - (m == -INFINITY ? 0.f : m));
        float l = w * li, sum = 0.f;
#pragma unroll
        for (int h = 16; h > 0; h >>= 1) l += __shfl_xor_sync(0xffffffffu, l, h);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, (cls + k * classes) & 31);
            if (cls + k * classes < n) sum = fmaf(wk, x[k], sum);
        }
        red[tid] = sum;
        __syncthreads();
        if (tid < d) {
            for (int i = 1; i < classes; ++i) sum += red[i * d + tid];
            const float out = l == 0.f ? 0.f : sum / l;
            if (!(fabsf(out) <= 3.402823466e38f)) flag(p.status, kFlagNonfinite);
            o[tid] = out;
        }
        return;
    }
    float m = -INFINITY;
    for (int i = tid; i < n; i += NTJ) m = fmaxf(m, weight[i] = piece(i)[ROWS * d + r]);
    red[tid] = m;
    __syncthreads();
#pragma unroll
    for (int h = NTJ / 2; h > 0; h >>= 1) {
        if (tid < h) red[tid] = fmaxf(red[tid], red[tid + h]);
        __syncthreads();
    }
    const float base = red[0] == -INFINITY ? 0.f : red[0];
    __syncthreads();
    float l = 0.f;
    for (int i = tid; i < n; i += NTJ) {
        weight[i] = exp2f(weight[i] - base);
        l = fmaf(weight[i], piece(i)[ROWS * d + ROWS + r], l);
    }
    lsum[tid] = l;
    __syncthreads();
    // four columns to a thread: sixteen bytes of eight pieces are on their way at a time
    const int c4s = d / 4, c4 = tid % c4s, cls = tid / c4s, classes = NTJ / c4s;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = cls; i < n; i += classes) {
        const float4 x = *reinterpret_cast<const float4 *>(piece(i) + r * d + 4 * c4);
        const float w = weight[i];
        sum = make_float4(fmaf(w, x.x, sum.x), fmaf(w, x.y, sum.y), fmaf(w, x.z, sum.z), fmaf(w, x.w, sum.w));
    }
    sums[tid] = sum;
    __syncthreads();
#pragma unroll
    for (int h = NTJ / 2; h > 0; h >>= 1) {
        if (tid < h) {
            lsum[tid] += lsum[tid + h];
            if (h >= c4s) {
                const float4 x = sums[tid + h];
                sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
                sums[tid] = sum;
            }
        }
        __syncthreads();
    }
    if (tid < c4s) {
        const float l = lsum[0];
        const float out[4] = {sum.x / l, sum.y / l, sum.z / l, sum.w / l};
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = l == 0.f ? 0.f : out[e];
            bad |= !(fabsf(x) <= 3.402823466e38f);
            o[4 * tid + e] = x;
        }
        if (bad) flag(p.status, kFlagNonfinite);
    }
}

template <class Kernel>
cudaError_t launch_one(Kernel kernel, const Params &p, unsigned grid, int bytes, cudaStream_t s)
{
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, dim3(grid), NTA, bytes, s, p);
}

template <int D>
cudaError_t launch_d(const Params &p, int in_bf16, unsigned grid, cudaStream_t s)
{
    const int g = p.group;
    if (in_bf16) {
        constexpr int bytes = MmaCfg<D>::SMEM;
        return g <= 4   ? launch_one(paged_mma_kernel<D, 4>, p, grid, bytes, s)
               : g <= 8 ? launch_one(paged_mma_kernel<D, 8>, p, grid, bytes, s)
                        : launch_one(paged_mma_kernel<D, 16>, p, grid, bytes, s);
    }
    // fp32 rows in classes of 1, 4 and 16: the FMAs of the class's rows are made whatever the group is. 16 requests of
    // 500 to 8000 tokens, two key-value heads of d = 128: groups of 1 and 2 to 4 take 32 and 36 to 38 us, of 5 to 16 81
    // to 85 (a class of 8 would bring 5 to 8 to 56; not built)
    return g <= 1   ? launch_one(paged_simt_kernel<D, 1>, p, grid, (int)sizeof(SimtSmem<D, 1>), s)
           : g <= 4 ? launch_one(paged_simt_kernel<D, 4>, p, grid, (int)sizeof(SimtSmem<D, 4>), s)
                    : launch_one(paged_simt_kernel<D, 16>, p, grid, (int)sizeof(SimtSmem<D, 16>), s);
}

cudaError_t launch_attention(const Params &p, int d, int in_bf16, unsigned grid, cudaStream_t s)
{
    switch (d) {
        case 16: return launch_d<16>(p, in_bf16, grid, s);
        case 32: return launch_d<32>(p, in_bf16, grid, s);
        case 64: return launch_d<64>(p, in_bf16, grid, s);
        default: return launch_d<128>(p, in_bf16, grid, s);
    }
}

}  // namespace
}  // namespace stq

namespace {
bool attn_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t prefix_bytes(int32_t B) { return ((size_t)B + 1) * 8 / 256 * 256 + 256; }
}  // namespace

extern "C" size_t stq_paged_attention_workspace_bytes(int32_t B, int32_t q_heads, int32_t d, int32_t kv_heads)
{
    if (B < 1 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 || d < 1) return 0;
    return prefix_bytes(B) + (size_t)stq::paged::kMaxBlocks * 2 * stq::paged::ROWS * ((size_t)d + 2) * 4;
}

extern "C" stq_status stq_paged_attention(int32_t B, int32_t q_heads, int32_t kv_heads, int32_t d, int32_t dtype,
                                          int32_t page_size, int32_t num_pages, int32_t table_width, const void *q,
                                          const void *k_pages, const void *v_pages, const int32_t *table,
                                          const int32_t *lens, float scale, float *o, void *workspace,
                                          size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    if (B < 0 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || page_size < 1 || num_pages < 0 ||
        table_width < 0 || (dtype != STQ_F32 && dtype != STQ_BF16))
        return STQ_ERR_INVALID_ARG;
    const float scale2 = scale * 1.4426950408889634f;
    if (!(scale2 - scale2 == 0.f)) return STQ_ERR_INVALID_ARG;
    if (!(d == 16 || d == 32 || d == 64 || d == 128)) return STQ_ERR_UNSUPPORTED;
    if (B == 0) return STQ_OK;
    if (!q || !lens || !o || (table_width > 0 && (!table || !k_pages || !v_pages))) return STQ_ERR_INVALID_ARG;
    if (!attn_aligned(q, 16) || !attn_aligned(k_pages, 16) || !attn_aligned(v_pages, 16) || !attn_aligned(o, 16) ||
        !attn_aligned(table, 4) || !attn_aligned(lens, 4))
        return STQ_ERR_INVALID_ARG;
    if (workspace && (workspace_bytes < stq_paged_attention_workspace_bytes(B, q_heads, d, kv_heads) ||
                      !attn_aligned(workspace, 256)))
        return STQ_ERR_INVALID_ARG;
    const int64_t span = (int64_t)table_width * page_size;
    const int group = q_heads / kv_heads, row_tiles = (group + stq::paged::ROWS - 1) / stq::paged::ROWS;
    if (B > 2147483647 / q_heads || span > 0x7fffffff - stq::paged::TK) return STQ_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return STQ_ERR_CUDA;
    stq::paged::Params p{};
    p.q = q;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.table = table;
    p.lens = lens;
    p.o = o;
    p.status = dev_status;
    p.scale2 = scale2;
    p.B = B;
    p.Hq = q_heads;
    p.Hkv = kv_heads;
    p.group = group;
    p.row_tiles = row_tiles;
    p.W = table_width;
    p.page = page_size;
    p.num_pages = num_pages;
    p.split = workspace != nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t units = (int64_t)B * kv_heads * row_tiles;
    int64_t grid = units;
    if (p.split) {
        p.first_tile = static_cast<long long *>(workspace);
        p.pieces = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + prefix_bytes(B));
        const int64_t most = units * ((span + stq::paged::TK - 1) / stq::paged::TK);
        // the blocks that fit at a time, by their registers (fp32, more than four rows) and shared memory
        grid = (dtype == STQ_BF16 ? stq::mma_blocks(d) : group > 4 ? 2 : d == 128 ? 3 : 4) * (int64_t)sms;
        if (grid > stq::paged::kMaxBlocks) grid = stq::paged::kMaxBlocks;
        if (grid > most) grid = most > 0 ? most : 1;
    }
    if (stq::launch_attention(p, d, dtype == STQ_BF16, (unsigned)grid, s) != cudaSuccess) return STQ_ERR_CUDA;
    if (!p.split) return STQ_OK;
    const cudaError_t e =
        stq::launch_early(stq::paged_join_kernel, dim3((unsigned)((int64_t)B * q_heads)), stq::NTJ, 0, s, p, d, (int)grid);
    return e == cudaSuccess ? STQ_OK : STQ_ERR_CUDA;
}
