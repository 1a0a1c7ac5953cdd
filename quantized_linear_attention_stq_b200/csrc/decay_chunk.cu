// decay_chunk.cu -- prompts of decayed linear attention in chunks of 128 tokens on the tensor cores
// (bf16 inputs; stq_decay_prefill, contract in include/stq.h).
//
// Inside a chunk, with b_t = prod_{r<=t} alpha_r, e_s = prod_{r>s} alpha_r, D_ts = prod_{s<r<=t} alpha_r
// and S the state before the chunk:
//   o_t = b_t S^T q_t + sum_{s<=t} D_ts (q_t.k_s) v_s        S <- b_C S + sum_s (e_s k_s) v_s^T
// that is, four products on [token][d] tiles:
//   scores Q K^T,   O = Q S,   P V with P = D o scores,   dS = (e K)^T V
//
// A CTA goes along one (request, head), or one segment of it. Q, K and V come by TMA and enter the
// products as they are. What is not a bf16 input (S, P, e K) enters as three bf16 terms h + m + l, which
// carry fp32's 24 significand bits: P and (e K)^T from Tensor Memory, as first operands, S from shared
// memory. S itself stays in registers in fp32 (its sum with b_C S is an ordinary fma; only dS is summed
// by the tensor cores). Decays are multiplied up, never divided: D_ts is the product of the decays from
// the end of s's group of 16 tokens, of whole groups and up to t in t's group, so a decay of zero or a
// product that underflows is as exact as any other. These partial products, b, e and the chunk's whole product
// are made in fp64 and rounded once (an error of theirs would repeat in every chunk of a constant decay). D_ts
// is multiplied from the partial ones in fp32, rounded seven times at most; inside a group of 16 it is a running
// fp32 product, rounded 14 times at most. Neither error goes into the state.
//
// Roles: warps 0-7 turn scores into P, add b O and P V and write o (two warps to each 32 rows, on
// alternate groups of 16 columns of P and halves of O's columns); warps 8-15 keep S and write its terms;
// warps 16-23 make e K, 16 tokens at a time, four warps to a group of tokens (for sums only, warps 0-7 do,
// too; with all 24 the state's warps came late to dS, 5 % of the time of 16 heads of 65521 tokens); warp 24 issues the TMA loads, warp 25 the MMAs, warp 26
// makes the products of the decays. Products are issued as scores, dS, O, P V: P is made while dS and O
// run, dS is read while O does (P V then takes its columns of Tensor Memory), S's terms for the next
// chunk are made from the end of O on, o is read while the next scores run. Roles meet at mbarriers only,
// each waited for with a limit; a barrier's next phase needs its waiter's progress, so no wait can miss
// its phase.
//
// Bound by the power limit: 16 x 16 heads of 8192 tokens of d = 128 take 760 to 800 us in a second's run, at
// 1.6 GHz, and 650 to 670 in 20 passes; their tensor work alone would take 496 and 415 us at cuBLAS's rates, their
// bytes 415. A chunk takes 8140 cycles, and the tensor pipe is active for 5120 of them (counters of that case). 16
// heads of 65521 tokens, in nine segments: 475 to 515 us in a second's run, 420 in 20 passes, of which the main pass
// takes 289, the first 104 and the join 7 (floor 206 us of bytes).
//
// A group of 16 scores (16 fp32 columns of Tensor Memory) is replaced in place by the h and m terms of
// its 16 entries of P (8 columns each); the l terms have columns of their own.
#include "../../include/stq.h"
#include "prefill_common.cuh"
#include "stq_decay.cuh"
#include "stream_order.cuh"
#include "tensor_map.cuh"

namespace stq {
namespace {

constexpr int CT = kDecayChunk;         // tokens of a chunk
constexpr int NTC = 896;                // threads
constexpr uint32_t BOX = CT * 128;      // a [128 tokens][64 columns] bf16 box
// Tensor Memory columns: scores, then P's h and m terms; its l terms; O; dS, then P V; slots of e K's terms
constexpr uint32_t TM_SC = 0, TM_L = 128, TM_O = 192, TM_DS = 320, TM_KT = 448, KT_COLS = 24;

// Decay products of a chunk, and inside groups of 16 tokens; read two and four at a time in every stage.
struct alignas(16) ChunkGates {
    float alpha[CT];
    float b[CT], e[CT];
    float upto[CT], behind[CT];  // the group's up to the token, and behind it
    float group[8];
    double all;
};

// Loads of q, k, v landed; k free; v free; gates made / free; scores done; P made; O done; P V done; o read; e K's slots full / free; dS done / read; S's terms made; end.
enum { FQ, FK, FV = FK + 3, KE = FV + 3, VE = KE + 3, GA = VE + 3, GF = GA + 2, SC = GF + 2, PF, QS, OF, OFF, KTF, KTE = KTF + 8, DS = KTE + 8, DSF = DS + 2, SF = DSF + 2, END, NBAR };

template <int STAGES>
struct ChunkMisc {
    unsigned long long bars[NBAR];
    ChunkGates g[STAGES];
    uint32_t tmem;
};

template <int KB, int SUMS>
struct ChunkCfg {
    static constexpr uint32_t QB = KB * BOX;            // bytes of a q, k or v tile
    static constexpr int KS = SUMS ? 3 : 1;             // stages of k
    static constexpr int VS = SUMS ? 3 : 2;             // stages of v
    static constexpr int GS = SUMS ? 2 : 1;             // stages of the decays' products, and dS's of columns
    static constexpr uint32_t K = 0;
    static constexpr uint32_t V = K + KS * QB;
    static constexpr uint32_t Q = V + VS * QB;
    static constexpr uint32_t ST = Q + (SUMS ? 0 : QB); // three terms of S: [KB][64 KB rows][64 columns]
    static constexpr uint32_t SA = KB * 64 * 128;       // ... bytes of 64 columns
    static constexpr uint32_t STB = KB * SA;            // ... of a term
    // [32 rows][32 columns] of o for each of 8 warps: the chunk's v for d = 128, where P V is done with it
    static constexpr uint32_t O = KB == 2 ? V : ST + (SUMS ? 0 : 3 * STB);
    static constexpr uint32_t OB = KB == 2 ? QB : 0;    // ... from one stage to the next
    static constexpr uint32_t MISC = ST + (SUMS ? 0 : 3 * STB) + (SUMS || KB == 2 ? 0 : 8 * 4096);
    static constexpr uint32_t SMEM = MISC + sizeof(ChunkMisc<GS>);
    static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");
    static constexpr int SLOTS = SUMS ? 8 : 2;          // of e K
    static constexpr uint32_t KT = SUMS ? 0 : TM_KT;
};

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int t, int tile, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(t), "r"(tile), "r"(bar)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}

// Sixteen rows of eight columns: lane l gives rows l / 4 (r[0], r[2]) and l / 4 + 8, columns l % 4 and 4 + l % 4.
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%4], {%0, %1, %2, %3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(taddr)
                 : "memory");
}

// The largest magnitude of three; NaN where one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight columns of this thread's lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// The same sixteen columns as pf::tmem_ld16, not there before tmem_wait_ld16.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// Four transposed 8 x 8 matrices of 16-bit entries from shared memory.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tma_prefetch(const CUtensorMap *map, int x, int t, int tile)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(t), "r"(tile)
                 : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *map, uint32_t src, int x, int t, int tile)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(t),
                 "r"(tile), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// D[tmem] (+)= A[smem] * B[smem], one of several products of the same A in a row: the first (0) leaves A in
// the tensor core's buffer, the others take it from there, the last (2) lets it go.
template <int TURN>
__device__ __forceinline__ void mma_same_a(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (TURN == 0)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16.collector::a::fill [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else if constexpr (TURN == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16.collector::a::use [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16.collector::a::lastuse [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// A thread's registers beyond or below those of the launch, by whole groups of four warps: 256 threads at
// 96, 256 at 88, 256 at 40 and 128 at 56 are the 896 at 72 that the launch has.
template <int N>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of a converged warp; known to the compiler as one (MMAs issued under `lane == 0` took at least
// 96 cycles each here, under elect 44 to 108).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

template <int KB, int SUMS>
__global__ void __launch_bounds__(NTC, 1)
    decay_chunk_kernel(const __grid_constant__ DecayParams p, const int d, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mo)
{
    using M = ChunkCfg<KB, SUMS>;
    constexpr int KS = M::KS, VS = M::VS, GS = M::GS;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    ChunkMisc<M::GS> &ms = *reinterpret_cast<ChunkMisc<M::GS> *>(sm + M::MISC);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    wait_for_stream();
    // (request, head), segment of the prompt
    const int64_t item = blockIdx.x;
    const int seg = (int)(item % p.segments);
    const int64_t tile = item / p.segments;
    const int b = (int)(tile / p.H), h = (int)(tile - (int64_t)b * p.H);
    const int slot = p.slots[b], len = prompt_length(p, b);
    if (slot < 0 || slot >= p.state_slots || len < 0) {
        if (tid == 0) flag(p.status, kFlagBounds);
        return;
    }
    const int chunks = (int)(((int64_t)len + CT - 1) / CT), seg_chunks = p.seg_tokens / CT;
    const int64_t n0l = (int64_t)seg * seg_chunks;
    if (n0l >= chunks) return;
    const int n0 = (int)n0l, N = min(chunks - n0, seg_chunks);
    const bool last = n0 + N == chunks;
    if (SUMS && last) return;  // the state behind the last segment is the main pass's

    auto bar = [&](int i) { return smem_u32(&ms.bars[i]); };
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            int count = 1;
            if (i >= KE && i < KE + 3) count = SUMS ? 16 : 8;
            if (i >= GF && i < GF + 2) count = 24;
            if (i >= VE && i < VE + 3) count = SUMS ? 1 : 8;
            if (i == PF || i == OFF || i == DSF || i == DSF + 1 || i == SF) count = 8;
            if (i >= KTF && i < KTF + 8) count = 4;
            mbar_init(bar(i), count);
        }
        fence_mbar_init();
    }
    if (warp == 25) umma::tmem_alloc(smem_u32(&ms.tmem), 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = ms.tmem;
    const int quarter = warp & 3;
    auto ds_at = [](int n) { return TM_DS - n % GS * 128; };  // dS's columns (sums have O's free)
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);  // this warp's lanes
    // a wait that gave up ends its role; the other roles' waits then give up too
    bool ok = true;
    auto wait = [&](int i, int phase) {  // of a warp
        const uint32_t at = bar(i), parity = (uint32_t)phase & 1u;
        if (!__all_sync(0xffffffffu, mbar_try_wait(at, parity))) ok = ok && pf::wait_bar(at, parity, p.status);
        return ok;
    };
    auto once = [&](int i, int phase) {  // of one thread
        if (ok && !mbar_wait_bounded(bar(i), (uint32_t)phase & 1u)) {
            ok = false;
            flag(p.status, kFlagTimeout);
        }
        return ok;
    };
    auto arrive = [&](int i) {  // of a warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    // Terms of e K, tokens 16 j .. 16 j + 15 of chunk n: a row of Tensor Memory per entry of k, two tokens
    // to a column, which is how transposed 8 x 8 matrices lie in a warp's registers. Rows of v behind the
    // prompt's end hold other tokens and are zeroed here, before the MMAs of these tokens.
    // The terms are made before the slot is waited for: a slot's way back and forth bounds dS. A warp makes
    // those of 16 of its quarter's 32 entries of k (x: which). A slot is always filled by the same warps: who
    // waits for it to be free has then seen it free before.
    auto make_ek = [&](int n, int j) {
        const int slot_ = j % M::SLOTS, use = (8 * n + j) / M::SLOTS;
        const int left = len - (n0 + n) * CT - 16 * j;  // tokens of the group that the prompt has
        uint32_t hh[2][4], mm[2][4], ll[2][4];
        if (quarter < 2 * KB) {
            const int tok = 16 * j + (lane & 7) + (lane >> 4) * 8, c8 = 4 * (quarter & 1) + (lane >> 3 & 1);
            const uint32_t k = sb + M::K + (n % KS) * M::QB + (quarter >> 1) * BOX;
            const ChunkGates &g = ms.g[n % GS];
            const float2 e[2] = {*reinterpret_cast<const float2 *>(&g.e[16 * j + 2 * (lane & 3)]),
                                 *reinterpret_cast<const float2 *>(&g.e[16 * j + 8 + 2 * (lane & 3)])};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t r[4];
                ldmatrix4_trans(k + umma::sw128_chunk(tok, c8 + 2 * x), r);
                if (left < 16)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int u = left - 8 * (i >> 1) - 2 * (lane & 3);
                        r[i] = u >= 2 ? r[i] : u == 1 ? r[i] & 0xFFFFu : 0u;
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    pf::split3_pair(__fmul2_rn(make_float2(__uint_as_float(r[i] << 16),
                                                           __uint_as_float(r[i] & 0xFFFF0000u)), e[i >> 1]),
                                    hh[x][i], mm[x][i], ll[x][i]);
            }
        }
        if (use > 0 && !wait(KTE + slot_, use - 1)) return;
        umma::fence_after_sync();
        if (quarter < 2 * KB) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t to = tl + ((uint32_t)(16 * x) << 16) + M::KT + slot_ * KT_COLS;
                tmem_st_16x8(to, hh[x]);
                tmem_st_16x8(to + 8, mm[x]);
                tmem_st_16x8(to + 16, ll[x]);
            }
            tmem_wait_st();
        }
        if (left < 16) {
            if (!wait(FV + n % VS, n / VS)) return;
            const int u = 4 * quarter + (lane >> 3);  // four rows of a warp
            if (u >= left)
                for (int x = 0; x < KB; ++x)
                    *reinterpret_cast<uint4 *>(sm + M::V + (n % VS) * M::QB + x * BOX + umma::sw128_chunk(16 * j + u, lane & 7)) =
                        make_uint4(0u, 0u, 0u, 0u);
            umma::fence_proxy_async();
        }
        umma::fence_before_sync();
        arrive(KTF + slot_);
    };
    // ... of groups j = first, first + step, ... of a chunk
    auto make_chunk = [&](int n, int first, int step) {
        if (!wait(GA + n % GS, n / GS) || !wait(FK + n % KS, n / KS)) return;
#pragma unroll 1
        for (int j = first; j < 8 && ok; j += step) make_ek(n, j);
        if (ok) arrive(KE + n % KS);
    };

    if (warp < 8) {
        regs_up<96>();
        // ---- P, o -----------------------------------------------------------------------------
        if constexpr (SUMS) {
            for (int n = 0; n < N && ok; ++n) {
                make_chunk(n, warp >> 2, 4);
                arrive(GF + n % GS);
            }
        } else {
            const int t = 32 * quarter + lane, sub = warp >> 2, l16 = lane & 15, top = 2 * quarter + 1;
            const bool hi = lane >= 16;
            const uint32_t z[16] = {}, z8[8] = {};
            for (int c = top + 1 + sub; c < 8; c += 2)  // tokens behind the row's: zero in every chunk
                tmem_st8(tl + TM_L + 8 * c, z8);
            float most = 0.f;
            for (int n = 0; n < N; ++n) {
                const int t0 = (n0 + n) * CT;
                if (!wait(GA, n)) break;
                const ChunkGates &g = ms.g[0];
                const float bt = g.b[t], upto = g.upto[t];
                if (!wait(SC, n)) break;
                umma::fence_after_sync();
                for (int c = top + 1 + sub; c < 8; c += 2) tmem_st16(tl + TM_SC + 16 * c, z);
                // The topmost group: of the two halves of the rows one has its diagonal there. The other has
                // nothing (sub 0), or all of the group below its own (sub 1).
                int c = top - sub;
                uint32_t next[16];  // scores, loaded a group ahead
                {
                    float D = 0.f, x[16];
                    uint32_t v[16];
                    tmem_ld16_async(tl + TM_SC + 16 * c, v);
                    tmem_wait_ld16(v);
                    if (c >= 2) tmem_ld16_async(tl + TM_SC + 16 * (c - 2), next);
                    const bool diag = hi == (sub == 0);
#pragma unroll
                    for (int i = 15; i >= 0; --i) {
                        if (i < 15) D *= g.alpha[16 * c + i + 1];
                        if (i >= l16) D = 1.f;
                        const float w = diag ? D : g.behind[16 * c + i] * upto;
                        x[i] = (diag ? i > l16 : sub == 0) ? 0.f : __uint_as_float(v[i]) * w;
                    }
                    uint32_t hm[16], ll[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) pf::split3_pair(make_float2(x[2 * i], x[2 * i + 1]), hm[i], hm[8 + i], ll[i]);
                    tmem_st16(tl + TM_SC + 16 * c, hm);
                    tmem_st8(tl + TM_L + 8 * c, ll);
                }
                float w = hi ? upto * g.group[top - 1] : upto;
                if (sub && quarter) w *= g.group[top - 2];
#pragma unroll 1
                for (c -= 2; c >= 0; c -= 2) {
                    float v[16];
                    tmem_wait_ld16(next);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(next[i]);
                    if (c >= 2) tmem_ld16_async(tl + TM_SC + 16 * (c - 2), next);
                    uint32_t hm[16], ll[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&g.behind[16 * c + i]);
                        const float2 w2 = make_float2(w, w);
                        pf::split3_pair(__fmul2_rn(make_float2(v[i], v[i + 1]), __fmul2_rn(make_float2(f.x, f.y), w2)),
                                        hm[i / 2], hm[8 + i / 2], ll[i / 2]);
                        pf::split3_pair(__fmul2_rn(make_float2(v[i + 2], v[i + 3]), __fmul2_rn(make_float2(f.z, f.w), w2)),
                                        hm[i / 2 + 1], hm[8 + i / 2 + 1], ll[i / 2 + 1]);
                    }
                    tmem_st16(tl + TM_SC + 16 * c, hm);
                    tmem_st8(tl + TM_L + 8 * c, ll);
                    if (c >= 2) w *= g.group[c] * g.group[c - 1];
                }
                tmem_wait_st();
                umma::fence_before_sync();
                arrive(PF);
                arrive(GF + n % GS);
                if (n > 0) {  // the tile of the chunk before has left shared memory: v may be loaded there
                    if (lane == 0) tma_stores_read();
                    arrive(VE + (n - 1) % VS);
                }

                if (!wait(OF, n)) break;
                umma::fence_after_sync();
                const int c0 = 32 * KB * sub;
                float o[KB][32];
#pragma unroll
                for (int cc = 0; cc < KB; ++cc) {
                    umma::tmem_ld32(tl + TM_O + c0 + 32 * cc, o[cc]);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {  // (16 at a time spill where o has all its 64 columns)
                        float x[8];
                        tmem_ld8(tl + TM_DS + c0 + 32 * cc + i, x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[cc][i + e] = fmaf(bt, o[cc][i + e], x[e]);
                    }
                }
                umma::fence_before_sync();
                arrive(OFF);
                // through shared memory, by TMA, where the prompt has all of the warp's rows
                const bool whole = t0 + 32 * quarter + 32 <= len;
                const uint32_t tile_o = M::O + (n & 1) * M::OB + warp * 4096;
#pragma unroll
                for (int cc = 0; cc < KB; ++cc) {
                    const int at = c0 + 32 * cc;
                    if (at >= d) break;
                    if (t0 + t < len)
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            if (i < 16 || d > 16) most = max_abs3(most, o[cc][i], o[cc][i + 1]);
                    if (whole) {
                        if (cc > 0) {
                            if (lane == 0) tma_stores_read();
                            __syncwarp();
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(sm + tile_o + umma::sw128_chunk(lane, i / 4)) =
                                make_float4(o[cc][i], o[cc][i + 1], o[cc][i + 2], o[cc][i + 3]);
                        umma::fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) tma_store(&mo, sb + tile_o, at, t0 + 32 * quarter, (int)tile);
                    } else if (t0 + t < len) {
                        float *dst = p.o + (tile * p.T + t0 + t) * d + at;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (i < 16 || d > 16)
                                *reinterpret_cast<float4 *>(dst + i) = make_float4(o[cc][i], o[cc][i + 1], o[cc][i + 2], o[cc][i + 3]);
                    }
                }
            }
            if (lane == 0) tma_stores_read();
            if (!(most <= 3.402823466e38f)) flag(p.status, kFlagNonfinite);
        }
    } else if (warp < 16) {
        regs_up<88>();
        // ---- S ----------------------------------------------------------------------------------
        constexpr int SC_ = 32 * KB;  // columns of a thread
        const int i = 32 * quarter + lane, c0 = SC_ * (warp >> 2 & 1);
        const int cols = i < d ? min(SC_, d - c0) : 0;
        float *record = p.records ? p.records + ((tile * p.segments + seg) * d + i) * d + c0 : nullptr;
        float *pool = p.states + (((int64_t)slot * p.H + h) * d + i) * d + c0;
        float S[SC_];
        {
            const float *from = p.segments > 1 ? record : pool;
#pragma unroll
            for (int c = 0; c < SC_; c += 4) {
                const float4 x = !SUMS && c < cols ? *reinterpret_cast<const float4 *>(from + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                S[c] = x.x;
                S[c + 1] = x.y;
                S[c + 2] = x.z;
                S[c + 3] = x.w;
            }
        }
        auto put_state = [&]() {
            if (quarter < 2 * KB) {
                uint8_t *st = sm + M::ST + (c0 >> 6) * M::SA;
#pragma unroll
                for (int c = 0; c < SC_ / 8; ++c) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = S[8 * c + e];
                    pf::store_split3(st, st + M::STB, st + 2 * M::STB, umma::sw128_chunk(i, (c0 >> 3 & 7) + c), x);
                }
            }
            umma::fence_proxy_async();
            arrive(SF);
        };
        Product upto;  // the segment's decay
        if (!SUMS) put_state();
        for (int n = 0; n < N && ok; ++n) {
            if (!wait(GA + n % GS, n / GS)) break;
            const float bc = (float)ms.g[n % GS].all;
            if (SUMS) upto.m *= ms.g[n % GS].all;
            arrive(GF + n % GS);
            if (SUMS) upto.settle();
            if (!wait(DS + n % GS, n / GS)) break;
            umma::fence_after_sync();
#pragma unroll
            for (int c = 0; c < SC_; c += 16) {
                float x[16];
                pf::tmem_ld16(tl + ds_at(n) + c0 + c, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) S[c + e] = fmaf(bc, S[c + e], x[e]);
            }
            umma::fence_before_sync();
            arrive(DSF + n % GS);
            if (!SUMS && n + 1 < N) {
                if (!wait(QS, n)) break;
                put_state();
            }
        }
        if (ok && (SUMS || last)) {
            float *to = SUMS ? record : pool;
            bool bad = false;
#pragma unroll
            for (int c = 0; c < SC_; c += 4)
                if (c < cols) {
                    *reinterpret_cast<float4 *>(to + c) = make_float4(S[c], S[c + 1], S[c + 2], S[c + 3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) bad |= !(fabsf(S[c + e]) <= 3.402823466e38f);
                }
            if (bad) flag(p.status, kFlagNonfinite);
            if (SUMS && tid == 256) p.products[tile * p.segments + seg] = upto.packed();
        }
    } else if (warp < 24) {
        regs_down<40>();
        // ---- e K ----------------------------------------------------------------------------
        for (int n = 0; n < N && ok; ++n) {
            const int x = warp >> 2 & 1;
            SUMS ? make_chunk(n, 2 + x, 4) : make_chunk(n, x, 2);
            arrive(GF + n % GS);
        }
    } else if (regs_down<56>(); warp == 24) {
        // ---- TMA ----------------------------------------------------------------------------
        if (elect_one()) {
            auto load = [&](uint32_t to, const CUtensorMap *map, int n, int full) {
                mbar_arrive_expect_tx(bar(full), M::QB);
                for (int x = 0; x < KB; ++x)
                    tma_box(sb + to + x * BOX, map, 64 * x, (n0 + n) * CT, (int)tile, bar(full));
            };
            int nq = 0, nk = 0, nv = 0;  // loads issued
            for (int n = 0; n < N; ++n) {
                if (n >= VS && !once(VE + n % VS, n / VS - 1)) break;
                load(M::V + n % VS * M::QB, &mv, n, FV + n % VS);
                ++nv;
                if (n >= KS && !once(KE + n % KS, n / KS - 1)) break;
                if (!SUMS && n >= 1 && !once(SC, n - 1)) break;
                load(M::K + n % KS * M::QB, &mk, n, FK + n % KS);
                ++nk;
                if constexpr (!SUMS) {
                    if (n + 1 < N)  // the next chunk to L2: these loads start late
                        for (int x = 0; x < KB; ++x) {
                            tma_prefetch(&mk, 64 * x, (n0 + n + 1) * CT, (int)tile);
                            tma_prefetch(&mq, 64 * x, (n0 + n + 1) * CT, (int)tile);
                        }
                    if (n >= 1 && !once(QS, n - 1)) break;  // the scores were done before
                    load(M::Q, &mq, n, FQ);
                    ++nq;
                }
            }
            // no copy is in flight when the CTA ends, also where a wait gave up
            if (nq) mbar_wait_bounded(bar(FQ), (uint32_t)(nq - 1) & 1u);
            for (int n = nk - KS < 0 ? 0 : nk - KS; n < nk; ++n) mbar_wait_bounded(bar(FK + n % KS), (uint32_t)(n / KS) & 1u);
            for (int n = nv - VS < 0 ? 0 : nv - VS; n < nv; ++n) mbar_wait_bounded(bar(FV + n % VS), (uint32_t)(n / VS) & 1u);
        }
    } else if (warp == 25) {
        // ---- MMA ----------------------------------------------------------------------------
        if (elect_one()) {
            const uint32_t cols = KB == 2 ? 128 : d;  // of v
            const int steps = KB == 2 ? 8 : d / 16;   // of 16 entries of q and k
            const uint32_t id_sc = umma::idesc_bf16(128, 128, 0, 0), id_d = umma::idesc_bf16(128, 0, 0, 1) | (cols >> 3) << 17;
            uint64_t dq = umma::smem_desc(sb + M::Q, 16, 1024), dk = umma::smem_desc(sb + M::K, 16, 1024),
                           dv = umma::smem_desc(sb + M::V, BOX, 1024), ds = umma::smem_desc(sb + M::ST, M::SA, 1024);
            for (int n = 0; n < N; ++n) {
                // (kept from making all tiles' descriptors before the loop, which is more than its registers)
                asm volatile("" : "+l"(dq), "+l"(dk), "+l"(dv), "+l"(ds));
                const uint64_t kn = dk + n % KS * (M::QB >> 4), vn = dv + n % VS * (M::QB >> 4);
                if constexpr (!SUMS) {
                    // P of the chunk before is used up when its P V is done
                    if (!once(FK + n % KS, n / KS) || !once(FQ, n) || (n > 0 && !once(OF, n - 1))) break;
                    umma::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 4 * KB; ++kk)
                        if (kk < steps)
                            umma::mma_bf16(tmem + TM_SC, dq + (((kk >> 2) * BOX + (kk & 3) * 32) >> 4),
                                           kn + (((kk >> 2) * BOX + (kk & 3) * 32) >> 4), id_sc, kk != 0);
                    umma::mma_commit(bar(SC));
                }
                if (!once(FV + n % VS, n / VS) || (n >= GS && !once(SUMS ? DSF + n % GS : OFF, n / GS - 1))) break;
                auto o_step = [&](int kk) {
                    const uint64_t a = dq + (((kk >> 2) * BOX + (kk & 3) * 32) >> 4), s = ds + (kk * 2048 >> 4);
                    mma_same_a<0>(tmem + TM_O, a, s + (2 * M::STB >> 4), id_d, kk != 0);
                    mma_same_a<1>(tmem + TM_O, a, s + (M::STB >> 4), id_d, 1);
                    mma_same_a<2>(tmem + TM_O, a, s, id_d, 1);
                };
                // rows d.. of dS are not read
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    const int slot_ = j % M::SLOTS, use = (8 * n + j) / M::SLOTS;
                    if (!once(KTF + slot_, use)) break;
                    umma::fence_after_sync();
                    const uint32_t a = tmem + M::KT + slot_ * KT_COLS;
                    const uint64_t v = vn + j * (2048 >> 4);
                    mma_ts(tmem + ds_at(n), a + 16, v, id_d, j != 0);
                    mma_ts(tmem + ds_at(n), a + 8, v, id_d, 1);
                    mma_ts(tmem + ds_at(n), a, v, id_d, 1);
                    umma::mma_commit(bar(KTE + slot_));
                    // Steps of O between the groups of dS: a slot's way back and forth takes longer than the other
                    // slot's products. The last steps are left for the time in which dS is read.
                    if (!SUMS && j < 5 && j < steps) {
                        if (j == 0 && !once(SF, n)) break;
                        umma::fence_after_sync();
                        o_step(j);
                    }
                }
                if (!ok) break;
                umma::mma_commit(bar(DS + n % GS));
                if constexpr (SUMS) {
                    umma::mma_commit(bar(VE + n % VS));
                } else {
#pragma unroll 1
                    for (int kk = 5; kk < steps; ++kk) o_step(kk);
                    umma::mma_commit(bar(QS));
                    if (!once(PF, n) || !once(DSF, n)) break;
                    umma::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) mma_ts(tmem + TM_DS, tmem + TM_L + 8 * kk, vn + (kk * 2048 >> 4), id_d, kk != 0);
#pragma unroll
                    for (int kk = 0; kk < 16; ++kk)
                        mma_ts(tmem + TM_DS, tmem + TM_SC + 16 * (kk & 7) + (kk < 8 ? 8 : 0), vn + ((kk & 7) * 2048 >> 4), id_d, 1);
                    umma::mma_commit(bar(OF));
                }
            }
            // what was issued is over before Tensor Memory is given back, also where a wait gave up
            umma::mma_commit(bar(END));
            mbar_wait_bounded(bar(END), 0);
        }
    } else if (warp == 26) {
        // ---- products of the decays: four tokens to a lane, four lanes to a group ----------------
        const float *alpha = p.alpha + tile * p.T;
        float next[4];
        auto load = [&](int n) {
            const int t = (n0 + n) * CT + 4 * lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i] = n < N && i < len - t ? alpha[t + i] : 1.f;
        };
        load(0);
        for (int n = 0; n < N; ++n) {
            const float a[4] = {next[0], next[1], next[2], next[3]};
            load(n + 1);
            double pre = (double)a[0] * a[1] * a[2] * a[3], suf = pre;
            // inclusive over the group's lanes, from the left and from the right
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, pre, o, 4), z = __shfl_down_sync(0xffffffffu, suf, o, 4);
                if ((lane & 3) >= o) pre *= y;
                if ((lane & 3) + o < 4) suf *= z;
            }
            const double group = __shfl_sync(0xffffffffu, pre, 3, 4);
            pre = __shfl_up_sync(0xffffffffu, pre, 1, 4);
            suf = __shfl_down_sync(0xffffffffu, suf, 1, 4);
            if ((lane & 3) == 0) pre = 1.0;
            if ((lane & 3) == 3) suf = 1.0;
            // the same over the groups
            double left = group, right = group;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, left, o), z = __shfl_down_sync(0xffffffffu, right, o);
                if (lane >= o) left *= y;
                if (lane + o < 32) right *= z;
            }
            const double all = __shfl_sync(0xffffffffu, left, 31);
            left = __shfl_up_sync(0xffffffffu, left, 4);
            right = __shfl_down_sync(0xffffffffu, right, 4);
            if (lane < 4) left = 1.0;
            if (lane >= 28) right = 1.0;
            if (n >= GS && !wait(GF + n % GS, n / GS - 1)) break;
            ChunkGates &to = ms.g[n % GS];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pre *= a[i];
                to.alpha[4 * lane + i] = a[i];
                to.upto[4 * lane + i] = (float)pre;
                to.b[4 * lane + i] = (float)(left * pre);
            }
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                to.behind[4 * lane + i] = (float)suf;
                to.e[4 * lane + i] = (float)(suf * right);
                suf *= a[i];
            }
            if ((lane & 3) == 0) to.group[lane >> 2] = (float)group;
            if (lane == 0) to.all = all;
            arrive(GA + n % GS);
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 25) umma::tmem_dealloc(tmem, 512);
}

template <int KB, int SUMS>
cudaError_t launch(const DecayParams &p, int d, cudaStream_t s)
{
    const EncodeTiled enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    // q, k, v as boxes of 128 tokens x 64 columns, o of 32 x 32; what lies outside the tensor is read as zeros
    // and not written
    CUtensorMap map[4];
    const void *at[4] = {p.q, p.k, p.v, p.o};
    for (int i = 0; i < 4; ++i) {
        const cuuint64_t row = (cuuint64_t)d * (i < 3 ? 2 : 4);
        const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p.T, (cuuint64_t)p.B * p.H};
        const cuuint64_t strides[2] = {row, row * p.T};
        const cuuint32_t box[3] = {i < 3 ? 64u : 32u, i < 3 ? (cuuint32_t)CT : 32u, 1}, estr[3] = {1, 1, 1};
        if (enc(&map[i], i < 3 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                const_cast<void *>(at[i]), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorNotSupported;
    }
    auto kernel = decay_chunk_kernel<KB, SUMS>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ChunkCfg<KB, SUMS>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.B * p.H * p.segments;
    if (grid > 0x7fffffff) return cudaErrorNotSupported;
    return launch_early(kernel, dim3((unsigned)grid), NTC, ChunkCfg<KB, SUMS>::SMEM, s, p, d, map[0], map[1], map[2], map[3]);
}

}  // namespace

cudaError_t launch_decay_chunk(const DecayParams &p, int d, bool sums, cudaStream_t s)
{
    if (d <= 64) return sums ? launch<1, 1>(p, d, s) : launch<1, 0>(p, d, s);
    return sums ? launch<2, 1>(p, d, s) : launch<2, 0>(p, d, s);
}

}  // namespace stq
