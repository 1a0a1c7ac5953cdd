// pages.cu -- the paged key-value cache's bookkeeping on the GPU (contract in include/stq.h): pages
// for the new tokens of a batch (stq_page_plan) and the write of their keys and values
// (stq_page_write).
//
// Plan. With page size ps, request b holds P(len_b) pages, P(n) = ceil(n / ps), and asks for
// P(len_b + new_b) - P(len_b) more. Two prefix sums over the requests, of new tokens and of asked
// pages, give every request its place in the slot map and in the free list, so the result does not
// depend on the order in which threads run. Bound by launch and memory latency, not by bytes. A small
// plan is one block's. A large one is that of many blocks, each of which makes the sums for itself and
// writes its part of the table and of the slot map; the first also writes the lengths, the starts and the
// list's head, unless these are updated in place and the other blocks still read them. Then a second
// launch of one block writes them: it starts beside the first, makes its sums, and waits before it writes.
//
// Write. A row of a token's keys (all heads) is contiguous on the way in; each head's part goes to
// its own page rows. 16-byte copies, four in flight per thread; bound by HBM.
#include "../../include/stq.h"
#include "stq_internal.cuh"
#include "stream_order.cuh"

namespace stq {
namespace {

constexpr int NTP = 1024;
constexpr int kPlanOneBlock = 4096;

struct PlanParams {
    int32_t *table;
    const int32_t *lens, *fresh, *free_pages, *free_head;
    int32_t *slot_map, *starts, *lens_out, *head_out, *status;
    int32_t B, W, page, F, N;
    int fill;    // this launch writes the table and the slot map
    int commit;  // the first block of this launch writes the lengths, the starts and the list's head
};

// Inclusive prefix sums of a pair of 64-bit counts over the CTA; *total gets the CTA's sums.
__device__ __forceinline__ longlong2 scan_pair(longlong2 x, longlong2 *warp_sums, longlong2 *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x.x, d), b = __shfl_up_sync(0xffffffffu, x.y, d);
        if (lane >= d) {
            x.x += a;
            x.y += b;
        }
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    if (w == 0) {
        longlong2 y = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long a = __shfl_up_sync(0xffffffffu, y.x, d), b = __shfl_up_sync(0xffffffffu, y.y, d);
            if (lane >= d) {
                y.x += a;
                y.y += b;
            }
        }
        warp_sums[lane] = y;
    }
    __syncthreads();
    if (w > 0) {
        x.x += warp_sums[w - 1].x;
        x.y += warp_sums[w - 1].y;
    }
    *total = warp_sums[31];
    __syncthreads();
    return x;
}

// Slot of row `row` of page pg; -1 (and the bounds flag) for a page whose slots are not int32.
__device__ __forceinline__ int slot_of(int pg, int row, int page, int32_t *status)
{
    const long long slot = (long long)pg * page + row;
    if (pg >= 0 && slot <= 0x7fffffffLL) return (int)slot;
    flag(status, kFlagBounds);
    return -1;
}

// The last of n ascending starts that is at or before i.
__device__ __forceinline__ int find_start(const int *start, int n, long long i)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(NTP) page_plan_kernel(const PlanParams p)
{
    __shared__ longlong2 warp_sums[32];
    // of the requests of one round, NTP at a time:
    __shared__ int token0[NTP];  // slot-map index of the first new token
    __shared__ int held[NTP];    // tokens before, or -1: it gets no slots
    __shared__ int page0[NTP];   // pages asked for by the round's requests before it
    __shared__ int taken;        // pages taken by the requests served so far
    const int tid = threadIdx.x;
    // A launch that writes the table waits for all that was before the call. Of two launches, the first lets the
    // second start only behind that wait, and writes none of the lengths, counts and list head that the second
    // then reads at once; the status word that it may flag before its own wait is only ever OR-ed into.
    if (p.fill) wait_for_stream();
    if (!p.commit) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool commits = p.commit && blockIdx.x == 0;
    const int head = *p.free_head;
    const bool bad_head = head < 0 || head > p.F;
    const long long avail = bad_head ? 0 : p.F - head;
    const bool speaks = commits;  // one block of a call reports what it finds
    long long tok_base = 0, page_base = 0;
    if (tid == 0) {
        taken = 0;
        if (bad_head && speaks) flag(p.status, kFlagBounds);
    }
    const int step = (int)gridDim.x * NTP, at = (int)blockIdx.x * NTP + tid;
    for (int b0 = 0; b0 < p.B; b0 += NTP) {
        const int b = b0 + tid, nb = min(NTP, p.B - b0);
        int len = 0, add = 0, need = 0;
        bool ok = false;
        if (b < p.B) {
            len = p.lens[b];
            add = p.fresh[b];
            // counts and positions are int32: a row may span more, a request may not hold more
            ok = len >= 0 && add >= 0 && (long long)len + add <= min((long long)p.W * p.page, 0x7fffffffLL);
            add = max(add, 0);
            if (ok)
                need = (int)(((long long)len + add + p.page - 1) / p.page - ((long long)len + p.page - 1) / p.page);
        }
        longlong2 total;
        const longlong2 upto = scan_pair(make_longlong2(add, need), warp_sums, &total);
        const long long tok = tok_base + upto.x - add, pg = page_base + upto.y - need;
        // the sums were made while the first launch ran; what it reads is written behind its end
        if (!p.fill) wait_for_stream();
        if (b < p.B) {
            // its pages are on the list, and its tokens in the slot map
            const bool fits = ok && (need == 0 || pg + need <= avail) && tok + add <= p.N;
            token0[tid] = (int)min(tok, (long long)p.N);
            held[tid] = fits ? len : -1;
            page0[tid] = (int)min(upto.y - need, 0x7fffffffLL);
            if (fits && need > 0) atomicMax(&taken, (int)(pg + need));
            if (!fits && speaks) flag(p.status, kFlagBounds);
            if (commits) {
                p.starts[b] = token0[tid];
                p.lens_out[b] = fits ? len + add : len;
            }
        }
        const long long end = min(tok_base + total.x, (long long)p.N);
        __syncthreads();
        if (p.fill) {
            // the list's pages of this round: those of one request go to its row, in order
            const long long pages = min(total.y, avail - page_base);
            for (long long i = at; i < pages; i += step) {
                const int r = find_start(page0, nb, i);
                if (held[r] >= 0) {
                    const int now = (int)(((long long)held[r] + p.page - 1) / p.page);
                    p.table[(size_t)(b0 + r) * p.W + now + (int)(i - page0[r])] = p.free_pages[head + page_base + i];
                }
            }
            for (long long i = tok_base + at; i < end; i += step) {
                const int r = find_start(token0, nb, i);
                int slot = -1;
                if (held[r] >= 0) {
                    const int pos = held[r] + (int)(i - token0[r]), k = pos / p.page;
                    const int now = (int)(((long long)held[r] + p.page - 1) / p.page);
                    // a page it held before, or one just taken (its entry may not be written yet)
                    const int pgid = k < now ? p.table[(size_t)(b0 + r) * p.W + k]
                                             : p.free_pages[head + page_base + page0[r] + (k - now)];
                    slot = slot_of(pgid, pos - k * p.page, p.page, p.status);
                }
                p.slot_map[i] = slot;
            }
        }
        __syncthreads();
        tok_base = end;
        page_base += total.y;
    }
    if (p.fill)
        for (long long i = tok_base + at; i < p.N; i += step) p.slot_map[i] = -1;
    if (!p.fill) wait_for_stream();
    if (commits && tid == 0) {
        p.starts[p.B] = (int)tok_base;
        *p.head_out = bad_head ? head : head + taken;
    }
}

struct WriteParams {
    uint8_t *k_pages, *v_pages;
    const int32_t *slot_map;
    const uint8_t *k, *v;
    int64_t k_stride, v_stride;  // bytes between tokens
    int32_t *status;
    int64_t pieces;              // 16-byte pieces of one of k, v
    int32_t heads, page, row_pieces, head_pieces;
    int64_t slots;               // pages * page
};

constexpr int NTW = 256, PIECES = 2;  // threads; pieces of k, and of v, of a thread

// A block takes NTW * PIECES pieces in a row, so that one 64-bit division serves them all.
__global__ void __launch_bounds__(NTW) page_write_kernel(const WriteParams p)
{
    wait_for_stream();
    const int64_t base = (int64_t)blockIdx.x * (NTW * PIECES), t0 = base / p.row_pieces;
    const unsigned rest = (unsigned)(base - t0 * p.row_pieces) + threadIdx.x;
    uint4 a[PIECES], b[PIECES];
    size_t dst[PIECES];
    bool live[PIECES];
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const unsigned j = rest + u * NTW, dt = j / (unsigned)p.row_pieces, c = j - dt * (unsigned)p.row_pieces;
        const int64_t t = t0 + dt;
        live[u] = base + threadIdx.x + u * NTW < p.pieces;
        if (!live[u]) continue;
        const int slot = p.slot_map[t];
        if (slot < 0 || slot >= p.slots) {
            if (slot != -1) flag(p.status, kFlagBounds);
            live[u] = false;
            continue;
        }
        const unsigned h = c / (unsigned)p.head_pieces, x = c - h * (unsigned)p.head_pieces;
        const int pg = slot / p.page, off = slot - pg * p.page;
        dst[u] = ((((size_t)pg * p.heads + h) * p.page + off) * p.head_pieces + x) * 16;
        a[u] = __ldcs(reinterpret_cast<const uint4 *>(p.k + t * p.k_stride + (size_t)c * 16));
        b[u] = __ldcs(reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + (size_t)c * 16));
    }
#pragma unroll
    for (int u = 0; u < PIECES; ++u)
        if (live[u]) {
            *reinterpret_cast<uint4 *>(p.k_pages + dst[u]) = a[u];
            *reinterpret_cast<uint4 *>(p.v_pages + dst[u]) = b[u];
        }
}

}  // namespace
}  // namespace stq

namespace {
bool page_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
}  // namespace

extern "C" stq_status stq_page_plan(int32_t B, int32_t table_width, int32_t page_size, int32_t *table,
                                    const int32_t *lens, const int32_t *fresh, const int32_t *free_pages,
                                    int32_t num_free, const int32_t *free_head, int32_t *slot_map,
                                    int32_t slot_map_size, int32_t *starts, int32_t *lens_out, int32_t *head_out,
                                    int32_t *dev_status, void *stream)
{
    if (B < 0 || table_width < 0 || page_size < 1 || num_free < 0 || slot_map_size < 0) return STQ_ERR_INVALID_ARG;
    if (!free_head || !head_out || !starts) return STQ_ERR_INVALID_ARG;
    if ((slot_map_size > 0 && !slot_map) || (num_free > 0 && !free_pages)) return STQ_ERR_INVALID_ARG;
    if (B > 0 && (!lens || !fresh || !lens_out || (table_width > 0 && !table))) return STQ_ERR_INVALID_ARG;
    for (const void *ptr : {(const void *)table, (const void *)lens, (const void *)fresh, (const void *)free_pages,
                            (const void *)free_head, (const void *)slot_map, (const void *)starts,
                            (const void *)lens_out, (const void *)head_out})
        if (!page_aligned(ptr, 4)) return STQ_ERR_INVALID_ARG;
    stq::PlanParams p{table,    lens,       fresh, free_pages,  free_head, slot_map, starts,        lens_out,
                      head_out, dev_status, B,     table_width, page_size, num_free, slot_map_size, 1,  1};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the slot map's size bounds the work: one block up to kPlanOneBlock entries
    if (slot_map_size <= stq::kPlanOneBlock) {
        return stq::launch_early(stq::page_plan_kernel, dim3(1), stq::NTP, 0, s, p) == cudaSuccess ? STQ_OK : STQ_ERR_CUDA;
    }
    const int blocks = (slot_map_size + stq::NTP - 1) / stq::NTP;
    auto apart = [](const int32_t *x, int64_t nx, const int32_t *y, int64_t ny) { return x + nx <= y || y + ny <= x; };
    bool in_place = !apart(head_out, 1, free_head, 1);
    for (const int32_t *in : {lens, fresh})
        in_place = in_place || !apart(lens_out, B, in, B) || !apart(starts, (int64_t)B + 1, in, B) || !apart(head_out, 1, in, B);
    in_place = in_place || !apart(lens_out, B, free_head, 1) || !apart(starts, (int64_t)B + 1, free_head, 1);
    p.commit = !in_place;
    if (stq::launch_early(stq::page_plan_kernel, dim3(blocks < 296 ? blocks : 296), stq::NTP, 0, s, p) != cudaSuccess)
        return STQ_ERR_CUDA;
    if (!in_place) return STQ_OK;
    p.fill = 0;
    p.commit = 1;
    return stq::launch_early(stq::page_plan_kernel, dim3(1), stq::NTP, 0, s, p) == cudaSuccess ? STQ_OK : STQ_ERR_CUDA;
}

extern "C" stq_status stq_page_write(int32_t N, int32_t kv_heads, int32_t d, int32_t dtype, int32_t page_size,
                                     int32_t num_pages, void *k_pages, void *v_pages, const int32_t *slot_map,
                                     const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                                     int32_t *dev_status, void *stream)
{
    if (N < 0 || kv_heads < 1 || page_size < 1 || num_pages < 0 || (dtype != STQ_F32 && dtype != STQ_BF16))
        return STQ_ERR_INVALID_ARG;
    if (!(d == 16 || d == 32 || d == 64 || d == 128)) return STQ_ERR_UNSUPPORTED;
    if (N == 0) return STQ_OK;
    if (!k_pages || !v_pages || !slot_map || !k || !v) return STQ_ERR_INVALID_ARG;
    const int64_t size = dtype == STQ_BF16 ? 2 : 4, row = (int64_t)kv_heads * d;
    if (!page_aligned(k_pages, 16) || !page_aligned(v_pages, 16) || !page_aligned(k, 16) || !page_aligned(v, 16) ||
        !page_aligned(slot_map, 4) || k_stride < row || v_stride < row || k_stride * size % 16 != 0 ||
        v_stride * size % 16 != 0)
        return STQ_ERR_INVALID_ARG;
    if (row * size / 16 > 0x7fffffff || (int64_t)num_pages * page_size > 0x7fffffff) return STQ_ERR_UNSUPPORTED;
    stq::WriteParams p{};
    p.k_pages = static_cast<uint8_t *>(k_pages);
    p.v_pages = static_cast<uint8_t *>(v_pages);
    p.slot_map = slot_map;
    p.k = static_cast<const uint8_t *>(k);
    p.v = static_cast<const uint8_t *>(v);
    p.k_stride = k_stride * size;
    p.v_stride = v_stride * size;
    p.status = dev_status;
    p.heads = kv_heads;
    p.page = page_size;
    p.head_pieces = (int)(d * size / 16);
    p.row_pieces = kv_heads * p.head_pieces;
    p.pieces = (int64_t)N * p.row_pieces;
    p.slots = (int64_t)num_pages * page_size;
    const int64_t blocks = (p.pieces + stq::NTW * stq::PIECES - 1) / (stq::NTW * stq::PIECES);
    if (blocks > 0x7fffffff) return STQ_ERR_UNSUPPORTED;
    const cudaError_t e =
        stq::launch_early(stq::page_write_kernel, dim3((unsigned)blocks), stq::NTW, 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? STQ_OK : STQ_ERR_CUDA;
}
