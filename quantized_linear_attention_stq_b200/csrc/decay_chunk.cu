// decay_chunk.cu -- prompts of decayed linear attention in chunks of 128 tokens on the tensor cores
// (bf16 inputs; stq_decay_prefill, contract in include/stq.h).
//
// Inside a chunk, with b_t = prod_{r<=t} alpha_r, e_s = prod_{r>s} alpha_r, D_ts = prod_{s<r<=t} alpha_r
// and S the state before the chunk:
//   o_t = b_t S^T q_t + sum_{s<=t} D_ts (q_t.k_s) v_s        S <- b_C S + sum_s k_s (e_s v_s)^T
// that is, four products on [token][d] tiles:
//   scores Q K^T,   O1 = Q S,   O2 = P V with P = D o scores,   dS = K^T (e V)
//
// The columns of S are independent of each other, so a CTA takes 64 of them for one (request, head):
// for d = 128 two CTAs share a head, and its q and k tiles meet in L2. S stays in registers (fp32, a row
// per thread). Everything that is not a bf16 input enters its product as three bf16 terms h + m + l,
// which carry fp32's 24 significand bits; decays are multiplied up directly, never divided, so a decay
// of zero or a product that underflows is as exact as any other. Products over a chunk are made in
// fp64 and rounded once (an error of theirs would repeat in every chunk of a constant decay).
//
// Roles: warps 0-3 turn scores into P (a row per thread, kept in Tensor Memory as the first operand)
// and write o; warps 4-7 scale V, keep S and write its terms; warp 8 issues the TMA loads, warp 9 the
// MMAs, warp 10 makes the chunk's decay products. A chunk's products are issued as scores, dS, O1, O2,
// so that dS of the next chunk needs nothing of the P of this one; K is free after dS, a chunk before
// Q and V are. Roles meet at mbarriers only, each waited for with a limit; a barrier's next phase
// needs its waiter's progress, so no wait can miss its phase (those of the TMA warp therefore come in
// two, for even and odd chunks).
#include "../../include/stq.h"
#include "prefill_common.cuh"
#include "stq_decay.cuh"
#include "tensor_map.cuh"

namespace stq {
namespace {

constexpr int CT = kDecayChunk;         // tokens of a chunk
constexpr int NTC = 352;                // threads
constexpr uint32_t BOX = CT * 128;      // a [128 tokens][64 columns] bf16 box
// Tensor Memory columns
constexpr uint32_t TM_SC = 0, TM_O1 = 128, TM_O2 = 192, TM_DS = 256, TM_P = 320;

// Barriers: loads of q, k, v landed; decays made / used by the rows' / by the state's warps; scores done; P made; e V made; dS done / read;
// terms of S made; O1 done; O2 done; o read; end. Those with 0 and 1 are of even and odd chunks.
enum { FQ0, FQ1, FK0, FK1, FV0, FV1, GA0, GA1, GF0, GF1, EF, SC, PF, VP, DS0, DS1, DSF, SF, QS0, QS1, OF0, OF1, OFF, END, NBAR };

struct ChunkGates {
    float alpha[CT + 4];  // zeros behind the chunk's
    float b[CT];
};

struct ChunkMisc {
    unsigned long long bars[NBAR];
    alignas(16) ChunkGates g[2];  // of the rows' warps; those of the state's warps follow
    float e[CT];
    double all;
    uint32_t tmem;
};

template <int KB>
struct ChunkCfg {
    static constexpr uint32_t QB = KB * BOX;            // bytes of a q (or k) tile
    static constexpr uint32_t Q = 0;                    // two stages (of k where only sums are computed)
    static constexpr uint32_t K = 2 * QB;
    static constexpr uint32_t V = K + QB;               // two stages
    static constexpr uint32_t VT = V + 2 * BOX;         // three terms of e V
    static constexpr uint32_t ST = VT + 3 * BOX;        // three terms of S: [64 KB rows][64 columns]
    static constexpr uint32_t STB = KB * 64 * 128;
    static constexpr uint32_t MISC = ST + 3 * STB;
    static constexpr uint32_t SMEM = MISC + sizeof(ChunkMisc);
    static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");
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

// Up to 32 floats (the first n) to a row of o.
__device__ __forceinline__ void store_o(float *dst, const float (&x)[32], int n, bool wide)
{
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
        if (c >= n) return;
        if (wide) {
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c), "f"(x[c]),
                         "f"(x[c + 1]), "f"(x[c + 2]), "f"(x[c + 3]), "f"(x[c + 4]), "f"(x[c + 5]), "f"(x[c + 6]),
                         "f"(x[c + 7])
                         : "memory");
        } else {
            *reinterpret_cast<float4 *>(dst + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
            *reinterpret_cast<float4 *>(dst + c + 4) = make_float4(x[c + 4], x[c + 5], x[c + 6], x[c + 7]);
        }
    }
}

template <int KB, int SUMS>
__global__ void __launch_bounds__(NTC, 1)
    decay_chunk_kernel(const __grid_constant__ DecayParams p, const int d, const int wide,
                       const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv)
{
    using M = ChunkCfg<KB>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    ChunkMisc &ms = *reinterpret_cast<ChunkMisc *>(sm + M::MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // (request, head), half of the columns, segment of the prompt
    const int half = blockIdx.x % KB;
    const int64_t item = blockIdx.x / KB;
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
        for (int i = 0; i < NBAR; ++i)
            mbar_init(bar(i), i == PF || i == VP || i == DSF || i == SF || i == OFF ? 128
                              : i == GA0 || i == GA1                                ? 32
                              : i == GF0 || i == GF1 || i == EF                     ? 4
                                                                                    : 1);
        fence_mbar_init();
    }
    if (warp == 9) umma::tmem_alloc(smem_u32(&ms.tmem), 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = ms.tmem;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);  // this warp's lanes
    // a wait that gave up ends its role; the other roles' waits then give up too
    bool ok = true;
    auto wait = [&](int i, int phase) { return ok = ok && pf::wait_bar(bar(i), (uint32_t)phase & 1u, p.status); };
    auto once = [&](int i, int phase) {  // of one thread
        if (ok && !mbar_wait_bounded(bar(i), (uint32_t)phase & 1u)) {
            ok = false;
            flag(p.status, kFlagTimeout);
        }
        return ok;
    };

    if (warp < 4) {
        // ---- scores -> P; o -----------------------------------------------------------------
        if constexpr (!SUMS) {
            const int t = tid;
            {
                uint32_t z[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = 0u;
                for (int cb = warp + 1; cb < 4; ++cb)  // tokens behind the row's: zero in every chunk
                    for (int x = 0; x < 3; ++x) tmem_st16(tl + TM_P + 64 * x + 16 * cb, z);
            }
            bool bad = false;
            for (int n = 0; n < N; ++n) {
                const int t0 = (n0 + n) * CT, st = n & 1;
                if (!wait(GA0 + st, n >> 1)) break;
                const ChunkGates &g = ms.g[st];
                const float bt = g.b[t];
                if (!wait(SC, n)) break;
                umma::fence_after_sync();
                float D = 0.f;
#pragma unroll 1
                for (int cb = warp; cb >= 0; --cb) {
                    float v[32];
                    umma::tmem_ld32(tl + TM_SC + 32 * cb, v);
                    uint32_t hh[16], mm[16], ll[16];
                    const bool diag = cb == warp;
                    float right = g.alpha[32 * cb + 32];  // the decay of the token right of the group of four
#pragma unroll
                    for (int e = 28; e >= 0; e -= 4) {
                        const float4 al = *reinterpret_cast<const float4 *>(&g.alpha[32 * cb + e]);
                        const float next[4] = {al.y, al.z, al.w, right};
                        right = al.x;
                        float x[4];
#pragma unroll
                        for (int i = 3; i >= 0; --i) {
                            D *= next[i];
                            if (diag && e + i >= lane) D = e + i == lane ? 1.f : 0.f;
                            x[i] = diag && e + i > lane ? 0.f : v[e + i] * D;
                        }
                        pf::split3_pair(make_float2(x[0], x[1]), hh[e / 2], mm[e / 2], ll[e / 2]);
                        pf::split3_pair(make_float2(x[2], x[3]), hh[e / 2 + 1], mm[e / 2 + 1], ll[e / 2 + 1]);
                    }
                    tmem_st16(tl + TM_P + 16 * cb, hh);
                    tmem_st16(tl + TM_P + 64 + 16 * cb, mm);
                    tmem_st16(tl + TM_P + 128 + 16 * cb, ll);
                }
                tmem_wait_st();
                umma::fence_before_sync();
                mbar_arrive(bar(PF));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(GF0 + st));

                if (!wait(OF0 + st, n >> 1)) break;
                umma::fence_after_sync();
                float *dst = p.o + (tile * p.T + t0 + t) * d + 64 * half;
                const bool live = t0 + t < len;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    float x[32], y[32];
                    umma::tmem_ld32(tl + TM_O1 + c, x);
                    umma::tmem_ld32(tl + TM_O2 + c, y);
                    if (c == 32) {
                        umma::fence_before_sync();
                        mbar_arrive(bar(OFF));
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        x[e] = fmaf(bt, x[e], y[e]);
                        bad |= live && c + e < d && !(fabsf(x[e]) <= 3.402823466e38f);
                    }
                    if (live) store_o(dst + c, x, d - c, wide);
                }
            }
            if (bad) flag(p.status, kFlagNonfinite);
        }
    } else if (warp < 8) {
        // ---- e V, S -------------------------------------------------------------------------
        const int i = tid - 128;  // token of the chunk; row of S
        const int cols = i < d ? min(64, d) : 0;
        float *record = p.records ? p.records + ((tile * p.segments + seg) * d + i) * d + 64 * half : nullptr;
        float *pool = p.states + (((int64_t)slot * p.H + h) * d + i) * d + 64 * half;
        float S[64];
        {
            const float *from = p.segments > 1 ? record : pool;
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 x = !SUMS && c < cols ? *reinterpret_cast<const float4 *>(from + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                S[c] = x.x;
                S[c + 1] = x.y;
                S[c + 2] = x.z;
                S[c + 3] = x.w;
            }
        }
        auto put_state = [&]() {
            if (i < 64 * KB)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = S[8 * c + e];
                    pf::store_split3(sm + M::ST, sm + M::ST + M::STB, sm + M::ST + 2 * M::STB, umma::sw128_chunk(i, c), x);
                }
            umma::fence_proxy_async();
            mbar_arrive(bar(SF));
        };
        double all = 1.0;   // the chunk's product
        double upto = 1.0;  // the segment's
        auto scale_v = [&](int n) {
            const int t0 = (n0 + n) * CT, st = n & 1;
            if (!wait(GA0 + st, n >> 1)) return;
            const float ef = ms.e[i];
            all = ms.all;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(EF));
            if (!wait(FV0 + st, n >> 1)) return;
            uint8_t *vt = sm + M::VT, *v = sm + M::V + st * BOX;
            const bool live = i < len - t0;
            if (len - t0 < CT) {
                // rows behind the prompt's end hold other tokens: zero, also in the tiles the MMAs read
                if (!wait(SUMS ? FK0 + st : FK0, SUMS ? n >> 1 : n)) return;
                uint8_t *k = sm + (SUMS ? M::Q + st * M::QB : M::K);
                if (!live)
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        *reinterpret_cast<uint4 *>(v + umma::sw128_chunk(i, c)) = make_uint4(0u, 0u, 0u, 0u);
                        for (int x = 0; x < KB; ++x)
                            *reinterpret_cast<uint4 *>(k + x * BOX + umma::sw128_chunk(i, c)) = make_uint4(0u, 0u, 0u, 0u);
                    }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t off = umma::sw128_chunk(i, c);
                float x[8];
                pf::bf16x8_to_f32(*reinterpret_cast<const uint4 *>(v + off), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = live ? x[e] * ef : 0.f;
                pf::store_split3(vt, vt + BOX, vt + 2 * BOX, off, x);
            }
            umma::fence_proxy_async();
            mbar_arrive(bar(VP));
        };
        if (!SUMS) put_state();
        scale_v(0);
        for (int n = 0; n < N && ok; ++n) {
            const float bc = (float)all;
            upto *= all;
            if (!wait(DS0 + (n & 1), n >> 1)) break;
            umma::fence_after_sync();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x[32];
                umma::tmem_ld32(tl + TM_DS + 32 * c, x);
#pragma unroll
                for (int e = 0; e < 32; ++e) S[32 * c + e] = fmaf(bc, S[32 * c + e], x[e]);
            }
            umma::fence_before_sync();
            mbar_arrive(bar(DSF));
            if (n + 1 == N) break;
            scale_v(n + 1);
            if (!SUMS) {
                if (!wait(QS0 + (n & 1), n >> 1)) break;
                put_state();
            }
        }
        if (ok && (SUMS || last)) {
            float *to = SUMS ? record : pool;
            bool bad = false;
#pragma unroll
            for (int c = 0; c < 64; c += 4)
                if (c < cols) {
                    *reinterpret_cast<float4 *>(to + c) = make_float4(S[c], S[c + 1], S[c + 2], S[c + 3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) bad |= !(fabsf(S[c + e]) <= 3.402823466e38f);
                }
            if (bad) flag(p.status, kFlagNonfinite);
            if (SUMS && i == 0 && half == 0) p.products[tile * p.segments + seg] = (float)upto;
        }
    } else if (warp == 8) {
        // ---- TMA ----------------------------------------------------------------------------
        if (lane == 0) {
            int nq[2] = {0, 0}, nk[2] = {0, 0}, nv[2] = {0, 0};  // loads issued on each barrier
            for (int n = 0; n < N; ++n) {
                const int t0 = (n0 + n) * CT, st = n & 1;
                if constexpr (SUMS) {
                    if (n >= 2 && !once(DS0 + st, (n - 2) >> 1)) break;
                    mbar_arrive_expect_tx(bar(FK0 + st), M::QB);
                    for (int x = 0; x < KB; ++x)
                        tma_box(sb + M::Q + st * M::QB + x * BOX, &mk, 64 * x, t0, (int)tile, bar(FK0 + st));
                    ++nk[st];
                } else {
                    if (n >= 2 && !once(QS0 + st, (n - 2) >> 1)) break;
                    mbar_arrive_expect_tx(bar(FQ0 + st), M::QB);
                    for (int x = 0; x < KB; ++x)
                        tma_box(sb + M::Q + st * M::QB + x * BOX, &mq, 64 * x, t0, (int)tile, bar(FQ0 + st));
                    ++nq[st];
                    if (n >= 1 && !once(DS0 + (st ^ 1), (n - 1) >> 1)) break;
                    mbar_arrive_expect_tx(bar(FK0), M::QB);
                    for (int x = 0; x < KB; ++x) tma_box(sb + M::K + x * BOX, &mk, 64 * x, t0, (int)tile, bar(FK0));
                    ++nk[0];
                    if (n >= 2 && !once(OF0 + st, (n - 2) >> 1)) break;
                }
                mbar_arrive_expect_tx(bar(FV0 + st), BOX);
                tma_box(sb + M::V + st * BOX, &mv, 64 * half, t0, (int)tile, bar(FV0 + st));
                ++nv[st];
            }
            // no copy is in flight when the CTA ends, also where a wait gave up
            for (int st = 0; st < 2; ++st) {
                if (nq[st]) mbar_wait_bounded(bar(FQ0 + st), (uint32_t)(nq[st] - 1) & 1u);
                if (nk[st]) mbar_wait_bounded(bar(FK0 + st), (uint32_t)(nk[st] - 1) & 1u);
                if (nv[st]) mbar_wait_bounded(bar(FV0 + st), (uint32_t)(nv[st] - 1) & 1u);
            }
        }
    } else if (warp == 9) {
        // ---- MMA ----------------------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t ID_SC = umma::idesc_bf16(128, 128, 0, 0), ID_DS = umma::idesc_bf16(128, 64, 1, 1),
                               ID_O = umma::idesc_bf16(128, 64, 0, 1);
            for (int n = 0; n < N; ++n) {
                const int st = n & 1;
                const uint32_t q = sb + M::Q + st * M::QB, k = SUMS ? q : sb + M::K, v = sb + M::V + st * BOX;
                if (!once(SUMS ? FK0 + st : FK0, SUMS ? n >> 1 : n)) break;
                if constexpr (!SUMS) {
                    if (!once(FQ0 + st, n >> 1)) break;
                    umma::fence_after_sync();  // the scores before were read: PF was waited for
#pragma unroll
                    for (int kk = 0; kk < 4 * KB; ++kk)
                        umma::mma_bf16(tmem + TM_SC, umma::smem_desc(q + (kk >> 2) * BOX + (kk & 3) * 32, 16, 1024),
                                       umma::smem_desc(k + (kk >> 2) * BOX + (kk & 3) * 32, 16, 1024), ID_SC, kk != 0);
                    umma::mma_commit(bar(SC));
                }
                if (!once(VP, n)) break;
                if (n > 0 && !once(DSF, n - 1)) break;
                umma::fence_after_sync();
                // rows 64.. of dS are not read where d <= 64 (the tile behind k stands in for their k)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                    for (int x = 0; x < 3; ++x)
                        umma::mma_bf16(tmem + TM_DS, umma::smem_desc(k + kk * 2048, BOX, 1024),
                                       umma::smem_desc(sb + M::VT + x * BOX + kk * 2048, 16, 1024), ID_DS, (kk | x) != 0);
                umma::mma_commit(bar(DS0 + st));
                if constexpr (!SUMS) {
                    if (!once(SF, n)) break;
                    if (n > 0 && !once(OFF, n - 1)) break;
                    umma::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 4 * KB; ++kk)
#pragma unroll
                        for (int x = 0; x < 3; ++x)
                            umma::mma_bf16(tmem + TM_O1, umma::smem_desc(q + (kk >> 2) * BOX + (kk & 3) * 32, 16, 1024),
                                           umma::smem_desc(sb + M::ST + x * M::STB + kk * 2048, 16, 1024), ID_O, (kk | x) != 0);
                    umma::mma_commit(bar(QS0 + st));
                    if (!once(PF, n)) break;
                    umma::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                        for (int x = 0; x < 3; ++x)
                            mma_ts(tmem + TM_O2, tmem + TM_P + 64 * x + 8 * kk, umma::smem_desc(v + kk * 2048, 16, 1024),
                                   ID_O, (kk | x) != 0);
                    umma::mma_commit(bar(OF0 + st));
                }
            }
            // what was issued is over before Tensor Memory is given back, also where a wait gave up
            umma::mma_commit(bar(END));
            mbar_wait_bounded(bar(END), 0);
        }
    } else {
        // ---- products of the decays -----------------------------------------------------------
        const float *alpha = p.alpha + tile * p.T;
        float next[4];
        auto load = [&](int n) {
            const int t = (n0 + n) * CT + 4 * lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i] = n < N && i < len - t ? alpha[t + i] : 1.f;
        };
        if (lane < 4) ms.g[0].alpha[CT + lane] = ms.g[1].alpha[CT + lane] = 0.f;
        load(0);
        for (int n = 0; n < N; ++n) {
            const int st = n & 1;
            const float a[4] = {next[0], next[1], next[2], next[3]};
            load(n + 1);
            const double p1 = (double)a[0] * a[1], p2 = p1 * a[2], p3 = p2 * a[3];
            const double s2 = a[3], s1 = s2 * a[2], s0 = s1 * a[1];
            double pre = p3, suf = p3;  // inclusive over the lanes from the left and from the right
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, pre, o), z = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane >= o) pre *= y;
                if (lane + o < 32) suf *= z;
            }
            const double all = __shfl_sync(0xffffffffu, pre, 31);
            pre = __shfl_up_sync(0xffffffffu, pre, 1);
            suf = __shfl_down_sync(0xffffffffu, suf, 1);
            if (lane == 0) pre = 1.0;
            if (lane == 31) suf = 1.0;
            if (!SUMS && n >= 2 && !wait(GF0 + st, (n - 2) >> 1)) break;
            if (n >= 1 && !wait(EF, n - 1)) break;
            ChunkGates &g = ms.g[st];
            *reinterpret_cast<float4 *>(&g.alpha[4 * lane]) = make_float4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<float4 *>(&g.b[4 * lane]) =
                make_float4((float)(pre * a[0]), (float)(pre * p1), (float)(pre * p2), (float)(pre * p3));
            *reinterpret_cast<float4 *>(&ms.e[4 * lane]) =
                make_float4((float)(suf * s0), (float)(suf * s1), (float)(suf * s2), (float)suf);
            if (lane == 0) ms.all = all;
            mbar_arrive(bar(GA0 + st));
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 9) umma::tmem_dealloc(tmem, 512);
}

template <int KB, int SUMS>
cudaError_t launch(const DecayParams &p, int d, cudaStream_t s)
{
    const EncodeTiled enc = encode_tiled();
    CUtensorMap map[3];
    const void *in[3] = {p.q, p.k, p.v};
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p.T, (cuuint64_t)p.B * p.H};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * p.T};
    const cuuint32_t box[3] = {64, CT, 1}, estr[3] = {1, 1, 1};
    for (int i = 0; i < 3; ++i)
        if (!enc || enc(&map[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(in[i]), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorNotSupported;
    auto kernel = decay_chunk_kernel<KB, SUMS>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ChunkCfg<KB>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.B * p.H * p.segments * KB;
    if (grid > 0x7fffffff) return cudaErrorNotSupported;
    const int wide = reinterpret_cast<uintptr_t>(p.o) % 32 == 0;
    kernel<<<(unsigned)grid, NTC, ChunkCfg<KB>::SMEM, s>>>(p, d, wide, map[0], map[1], map[2]);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_chunk(const DecayParams &p, int d, bool sums, cudaStream_t s)
{
    if (d <= 64) return sums ? launch<1, 1>(p, d, s) : launch<1, 0>(p, d, s);
    return sums ? launch<2, 1>(p, d, s) : launch<2, 0>(p, d, s);
}

}  // namespace stq
