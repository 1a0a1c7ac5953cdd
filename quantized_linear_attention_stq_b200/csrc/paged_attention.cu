// paged_attention.cu -- attention of one new token per request over a paged key-value cache
// (stq_paged_attention; contract in include/stq.h).
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - m),  m = max_t scale q.k_t
//
// One pass over the cache with the running maximum and sum of the softmax: a tile's scores raise
// the maximum from m to m', what was summed so far is scaled by exp(m - m'). Exponentials are taken
// in base 2, with scale * log2(e) multiplied into the scores. Bound by HBM: every cached key and
// value is read once for all the query heads that share it.
#include "../../include/stq.h"
#include "stq_paged.cuh"

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
    const long long begin = share_begin(total, blockIdx.x, gridDim.x);
    const long long end = share_begin(total, blockIdx.x + 1, gridDim.x);
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
    float k[KT][D + 4];
    float v[KT][D];
    float s[4][GT][KT];  // partial scores of the four quarters of d
    float p[GT][KT];
    float corr[GT], m[GT], l[GT];
    static_assert(KT * (D + 4) >= GT * D, "the joined sums fit where the keys were");
};

// One unit's tiles [t0, t1): scores by quarters of d (a lane per key, a warp per quarter), softmax
// by rows, products by (columns, key class). Leaves the sums in acc, joined over the key classes, in
// shared memory (sums[GT][D]), and m, l.
template <int D, int GT, int IN_BF16>
__device__ __forceinline__ void simt_unit(const Params &p, SimtSmem<D, GT> &sm, int b, int hk, int rt, int len,
                                          int t0, int t1, float *sums)
{
    constexpr int C4 = D / 4, PARTS = NTA / C4;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int c4 = tid % C4, part = tid / C4;
    const int rows = min(GT, p.group - rt * ROWS);
    const size_t q0 = ((size_t)b * p.Hq + (size_t)hk * p.group + rt * ROWS) * D;
    __syncthreads();  // the unit before has been read out
    for (int i = tid; i < GT * D; i += NTA) (&sm.q[0][0])[i] = i < rows * D ? load_in<IN_BF16>(p.q, q0 + i) : 0.f;
    if (tid < GT) {
        sm.m[tid] = -INFINITY;
        sm.l[tid] = 0.f;
    }
    float acc[GT][4];
#pragma unroll
    for (int g = 0; g < GT; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][e] = 0.f;
    const int32_t *row = p.table + (size_t)b * p.W;
    const int first = t0 * TK, last = min(len, t1 * TK);
    for (int k0 = first; k0 < last; k0 += KT) {
        __syncthreads();
        for (int i = tid; i < KT * C4; i += NTA) {
            const int r = i / C4, c = i % C4, t = k0 + r;
            float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
            float live = 0.f;
            if (t < last) {
                const int pg = row[t / p.page];
                if (pg >= 0 && pg < p.num_pages) {
                    const size_t at = (((size_t)pg * p.Hkv + hk) * p.page + t % p.page) * D + 4 * c;
                    if constexpr (IN_BF16) {
                        const uint2 a = *reinterpret_cast<const uint2 *>((const __nv_bfloat16 *)p.k_pages + at);
                        const uint2 e = *reinterpret_cast<const uint2 *>((const __nv_bfloat16 *)p.v_pages + at);
                        kk = make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u),
                                         __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xFFFF0000u));
                        vv = make_float4(__uint_as_float(e.x << 16), __uint_as_float(e.x & 0xFFFF0000u),
                                         __uint_as_float(e.y << 16), __uint_as_float(e.y & 0xFFFF0000u));
                    } else {
                        kk = *reinterpret_cast<const float4 *>((const float *)p.k_pages + at);
                        vv = *reinterpret_cast<const float4 *>((const float *)p.v_pages + at);
                    }
                    live = 1.f;
                } else {
                    flag(p.status, kFlagBounds);
                }
            }
            *reinterpret_cast<float4 *>(&sm.k[r][4 * c]) = kk;
            *reinterpret_cast<float4 *>(&sm.v[r][4 * c]) = vv;
            if (c == 0) sm.k[r][D] = live;  // in the row's padding
        }
        __syncthreads();
        {  // scores: lane = key, warp = quarter of d
            float s[GT];
#pragma unroll
            for (int g = 0; g < GT; ++g) s[g] = 0.f;
#pragma unroll
            for (int c = 0; c < C4 / 4; ++c) {
                const int col = (w * (C4 / 4) + c) * 4;
                const float4 kk = *reinterpret_cast<const float4 *>(&sm.k[lane][col]);
#pragma unroll
                for (int g = 0; g < GT; ++g) {
                    const float4 qq = *reinterpret_cast<const float4 *>(&sm.q[g][col]);
                    s[g] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[g]))));
                }
            }
#pragma unroll
            for (int g = 0; g < GT; ++g) sm.s[w][g][lane] = s[g];
        }
        __syncthreads();
        for (int g = w; g < GT; g += NTA / 32) {
            float s = (sm.s[0][g][lane] + sm.s[1][g][lane]) + (sm.s[2][g][lane] + sm.s[3][g][lane]);
            s = sm.k[lane][D] != 0.f ? s * p.scale2 : -INFINITY;
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
        for (int r = part; r < KT; r += PARTS) {
            const float4 vv = *reinterpret_cast<const float4 *>(&sm.v[r][4 * c4]);
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                const float e = sm.p[g][r];
                acc[g][0] = fmaf(e, vv.x, acc[g][0]);
                acc[g][1] = fmaf(e, vv.y, acc[g][1]);
                acc[g][2] = fmaf(e, vv.z, acc[g][2]);
                acc[g][3] = fmaf(e, vv.w, acc[g][3]);
            }
        }
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

// Writes a finished unit's output, or a piece of it for the join.
template <int D>
__device__ __forceinline__ void finish(const Params &p, int b, int hk, int rt, int len, const float *sums,
                                       const float *m, const float *l, int piece)
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

template <int D, int GT, int IN_BF16>
__global__ void __launch_bounds__(NTA) paged_simt_kernel(const Params p)
{
    extern __shared__ __align__(16) uint8_t raw[];
    SimtSmem<D, GT> &sm = *reinterpret_cast<SimtSmem<D, GT> *>(raw);
    float *sums = &sm.k[0][0];  // a unit's sums are joined where its keys were
    const int units = p.Hkv * p.row_tiles;
    if (!p.split) {
        const int u = blockIdx.x % units, b = blockIdx.x / units;
        bool bad;
        const int len = cached_length(p, b, &bad);
        if (bad && threadIdx.x == 0) flag(p.status, kFlagBounds);
        simt_unit<D, GT, IN_BF16>(p, sm, b, u / p.row_tiles, u % p.row_tiles, len, 0, tiles_of(len), sums);
        finish<D>(p, b, u / p.row_tiles, u % p.row_tiles, len, sums, sm.m, sm.l, -1);
        return;
    }
    const Cursor cur = find_share(p, units);
    long long at = cur.begin, before = cur.before;
    for (int b = cur.b; at < cur.end; ++b) {
        bool bad;
        const int len = cached_length(p, b, &bad), nt = tiles_of(len);
        const long long r0 = before * units;  // the request's first tile
        while (at < cur.end && at < r0 + (long long)nt * units) {
            const int u = (int)((at - r0) / nt);
            const long long s = r0 + (long long)u * nt, e = s + nt, stop = e < cur.end ? e : cur.end;
            simt_unit<D, GT, IN_BF16>(p, sm, b, u / p.row_tiles, u % p.row_tiles, len, (int)(at - s), (int)(stop - s),
                                      sums);
            const bool whole = at == s && stop == e;
            finish<D>(p, b, u / p.row_tiles, u % p.row_tiles, len, sums, sm.m, sm.l, whole ? -1 : s < cur.begin ? 0 : 1);
            at = stop;
        }
        before += nt;
    }
}

// Joins the pieces of the units that were cut, and zeroes the rows of requests without tokens.
// One block per (request, query head), a thread per column.
__global__ void __launch_bounds__(128) paged_join_kernel(const Params p, int d, int blocks)
{
    const int units = p.Hkv * p.row_tiles;
    const int row = blockIdx.x % p.Hq, b = blockIdx.x / p.Hq;
    const int hk = row / p.group, g = row % p.group, rt = g / ROWS, r = g % ROWS, c = threadIdx.x;
    const long long f0 = p.first_tile[b], nt = p.first_tile[b + 1] - f0, total = p.first_tile[p.B] * units;
    float *o = p.o + ((size_t)b * p.Hq + row) * d;
    if (nt == 0) {
        if (c < d) o[c] = 0.f;
        return;
    }
    const long long s = f0 * units + (hk * p.row_tiles + rt) * nt;
    const int c0 = block_of(total, s, blocks), c1 = block_of(total, s + nt - 1, blocks);
    if (c0 == c1 || c >= d) return;
    const size_t stride = (size_t)ROWS * (d + 2);
    // the first block's piece goes on behind its share unless the unit began before it
    auto piece = [&](int blk) {
        const int which = s < share_begin(total, blk, blocks) ? 0 : 1;
        return p.pieces + ((size_t)blk * 2 + which) * stride;
    };
    float m = -INFINITY;
    for (int blk = c0; blk <= c1; ++blk)
        if (share_begin(total, blk, blocks) < share_begin(total, blk + 1, blocks))
            m = fmaxf(m, piece(blk)[ROWS * d + r]);
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f, l = 0.f;
    for (int blk = c0; blk <= c1; ++blk)
        if (share_begin(total, blk, blocks) < share_begin(total, blk + 1, blocks)) {
            const float *x = piece(blk);
            const float e = exp2f(x[ROWS * d + r] - base);
            sum = fmaf(e, x[r * d + c], sum);
            l = fmaf(e, x[ROWS * d + ROWS + r], l);
        }
    const float out = l == 0.f ? 0.f : sum / l;
    if (!(fabsf(out) <= 3.402823466e38f)) flag(p.status, kFlagNonfinite);
    o[c] = out;
}

template <int D, int GT>
cudaError_t launch_simt(const Params &p, int in_bf16, unsigned grid, cudaStream_t s)
{
    const auto kernel = in_bf16 ? paged_simt_kernel<D, GT, 1> : paged_simt_kernel<D, GT, 0>;
    constexpr int bytes = (int)sizeof(SimtSmem<D, GT>);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, NTA, bytes, s>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_group(const Params &p, int in_bf16, unsigned grid, cudaStream_t s)
{
    const int g = p.group;
    return g <= 1 ? launch_simt<D, 1>(p, in_bf16, grid, s)
         : g <= 4 ? launch_simt<D, 4>(p, in_bf16, grid, s)
                  : launch_simt<D, 16>(p, in_bf16, grid, s);
}

cudaError_t launch_attention(const Params &p, int d, int in_bf16, unsigned grid, cudaStream_t s)
{
    switch (d) {
        case 16: return launch_group<16>(p, in_bf16, grid, s);
        case 32: return launch_group<32>(p, in_bf16, grid, s);
        case 64: return launch_group<64>(p, in_bf16, grid, s);
        default: return launch_group<128>(p, in_bf16, grid, s);
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
        table_width < 0 || (dtype != STQ_F32 && dtype != STQ_BF16) || !(scale - scale == 0.f))
        return STQ_ERR_INVALID_ARG;
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
    p.scale2 = scale * 1.4426950408889634f;
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
        grid = 4 * (int64_t)sms;
        if (grid > stq::paged::kMaxBlocks) grid = stq::paged::kMaxBlocks;
        if (grid > most) grid = most > 0 ? most : 1;
    }
    if (stq::launch_attention(p, d, dtype == STQ_BF16, (unsigned)grid, s) != cudaSuccess) return STQ_ERR_CUDA;
    if (!p.split) return STQ_OK;
    stq::paged_join_kernel<<<(unsigned)((int64_t)B * q_heads), 128, 0, s>>>(p, d, (int)grid);
    return cudaGetLastError() == cudaSuccess ? STQ_OK : STQ_ERR_CUDA;
}
