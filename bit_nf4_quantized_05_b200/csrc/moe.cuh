// moe.cuh -- a mixture-of-experts layer over NF4 experts for a few tokens:
//
//   l = x R^T, p = softmax(l), the top_k experts of each token with weights w
//   a_e = act(x Wg_e^T) . (x Wu_e^T),   out = sum_j w_j a_{e_j} Wd_{e_j}^T (+ residual)
//
// Three kernels, each launched while the one before it drains:
//   nf4_moe_router_kernel         the logits, summed in fp64
//   nf4_moe_experts_kernel<false> routing (every CTA for itself: the logits are
//                                 a few KB), then a_e of the chosen experts
//   nf4_moe_experts_kernel<true>  the down products, their weighted sum
// The experts' codes are nearly all the bytes: 3 H F / 2 per chosen expert.
//
// A token chooses an expert at most once, so routing is a bit mask of tokens
// per expert (an order-free OR, so the result does not depend on timing). An
// expert's tokens are cut into chunks of 8 (the columns of one MMA) and
// numbered as slots, expert by expert; the work items are (chunk, 64 weight
// rows): 32 gate rows and the 32 up rows of the same features, or 64 down rows.
//
// An item belongs to a group of GW = 4, 8 or 16 warps (16 / GW groups a CTA,
// each with its own barrier, so that one computes while another joins its
// sums). The warps split k in steps of 128 elements: warp w takes steps w, w +
// GW, ... A step is 64 rows x 64 bytes of codes, brought by TMA into the warp's
// own ring of two slots, one step ahead across items. As in the streaming
// kernel of the linear layer, a code byte becomes two bf16 levels by one byte
// permute and one conflict-free shared load, the products run on mma.sync with
// the tokens as its 8 columns (16 x 8 x 16; a tcgen05 tile would spend 128 rows
// on at most 8 tokens and need the operand written to shared memory), and a
// 64-element block's fp32 partial is multiplied by its scale once.
#pragma once

#include "decode_stream.cuh"
#include "epilogue.cuh"

namespace nf4 {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMoeChunk = 8;                       // tokens of one work item
// chunks: every expert's last one may be partly filled
constexpr int kMoeMaxChunks = kMoeMaxExperts + kMoeMaxSlots / kMoeChunk;
constexpr int kMoeWarps = 16;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMoeRows = 64;                       // weight rows of one item
constexpr int kMoeStepBytes = 64;                  // code bytes of one row in a step: 2 blocks
constexpr int kMoeSlotBytes = kMoeRows * kMoeStepBytes;
constexpr int kMoeRing = 2;

// The table holds bf16(1.4367 level), and every scale carries the factor that
// takes it back. bf16 hits some multiples of the 16 levels better than others:
// over the codes of normally distributed weights the rounding is 0.078% of a
// weight in the mean square at this factor (found by a search over [1, 2)),
// against 0.136% for bf16(level) itself.
constexpr float kMoeLevelUp = 1.4367f;
constexpr float kMoeLevelDown = 0.69603324f;

struct MoeChunk {
    uint16_t expert;
    uint16_t slot0;      // first slot
    uint16_t n;          // tokens, 1..8
    uint16_t pad;
};

// What routing leaves in the workspace for the down kernel.
struct MoeRoute {
    int nchunks;
    int pad[3];
    MoeChunk chunk[kMoeMaxChunks];
    float weight[kMoeMaxSlots];           // by slot
    uint16_t slot_of[kMoeMaxSlots];       // by token * top_k + j
};

struct MoeArgs {
    int M, E, top_k, H, F;
    int act, renorm;
    const uint16_t *x;            // [M, H]
    const uint16_t *router;       // [E, H]
    const uint16_t *residual;     // [M, H] or null
    uint16_t *out;                // [M, H]
    int32_t *ids;                 // [M, top_k] or null
    float *weights;               // [M, top_k] or null
    // scales of the expert weight of this launch (gate_up or down)
    const float *absmax;
    const uint8_t *q8;
    const float *cg;
    int dq, bshift;
    // workspace
    double *logits;               // [M, E]
    MoeRoute *route;
    uint16_t *a;                  // [slots, F] bf16
    float *y;                     // [slots, H] weighted down products
    int *done;                    // [H / 64] items finished of each stripe of out
};

// ---------------------------------------------------------------------------
// Router logits in fp64: which experts a token takes is decided by comparing
// them, and a product of two bf16 values is exact in fp64, so sums that differ
// only in their order practically never swap two experts. A CTA forms 4 tokens
// x 4 experts, its 8 warps splitting H.
// ---------------------------------------------------------------------------
constexpr int kMrThreads = 256;
constexpr int kMrTokens = 4, kMrExperts = 4;

__device__ __forceinline__ void bf16_to_f64(const uint4 &v, double (&d)[8]) {
    float f[8];
    bf16_unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = static_cast<double>(f[i]);
}

__global__ void __launch_bounds__(kMrThreads)
nf4_moe_router_kernel(const MoeArgs a) {
    __shared__ double part[kMrThreads / 32][kMrTokens * kMrExperts];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < a.H / kMoeRows; i += kMrThreads) a.done[i] = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = static_cast<int>(blockIdx.x) * kMrExperts, m0 = static_cast<int>(blockIdx.y) * kMrTokens;
    double acc[kMrTokens][kMrExperts] = {};
    for (int k = threadIdx.x * 8; k < a.H; k += kMrThreads * 8) {
        double w[kMrExperts][8];
#pragma unroll
        for (int j = 0; j < kMrExperts; ++j)
            if (e0 + j < a.E)
                bf16_to_f64(__ldg(reinterpret_cast<const uint4 *>(a.router + static_cast<int64_t>(e0 + j) * a.H + k)), w[j]);
#pragma unroll
        for (int i = 0; i < kMrTokens; ++i) {
            if (m0 + i >= a.M) break;
            double x[8];
            bf16_to_f64(*reinterpret_cast<const uint4 *>(a.x + static_cast<int64_t>(m0 + i) * a.H + k), x);
#pragma unroll
            for (int j = 0; j < kMrExperts; ++j)
                if (e0 + j < a.E)
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[i][j] = fma(x[c], w[j][c], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < kMrTokens; ++i)
#pragma unroll
        for (int j = 0; j < kMrExperts; ++j) {
            double v = acc[i][j];
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) part[warp][i * kMrExperts + j] = v;
        }
    __syncthreads();
    if (threadIdx.x < kMrTokens * kMrExperts) {
        const int m = m0 + threadIdx.x / kMrExperts, e = e0 + threadIdx.x % kMrExperts;
        double v = 0.0;
        for (int w = 0; w < kMrThreads / 32; ++w) v += part[w][threadIdx.x];
        if (m < a.M && e < a.E) a.logits[static_cast<int64_t>(m) * a.E + e] = v;
    }
}

// ---------------------------------------------------------------------------
// Shared memory of the experts kernel, by absolute shared address (see the
// streaming kernel): the level table's rows take the even 128-byte halves of
// [65536, 131072), the groups' partial sums the odd halves; ring slots fill
// the space below and above; the header is at the window's start.
// ---------------------------------------------------------------------------
struct MoeHeader {
    uint64_t bars[kMoeWarps][kMoeRing];
    int abort_flag;
    int nchunks;
    int last[kMoeWarps];                          // by group
    int warp_slots[kMoeMaxExperts / 32], warp_chunks[kMoeMaxExperts / 32];
    MoeChunk chunk[kMoeMaxChunks];
    float weight[kMoeMaxSlots];                   // by slot
    uint16_t slot_of[kMoeMaxSlots];               // by token * top_k + j
    union {
        struct {                                  // while routing
            unsigned long long mask[kMoeMaxExperts];   // tokens of each expert
            float w[kMoeMaxSlots];                     // by token * top_k + j
            uint8_t id[kMoeMaxSlots];
        };
    };
    uint8_t token[kMoeMaxSlots];                  // by slot
    uint16_t slot0[kMoeMaxExperts];
};
static_assert(kMoeMaxExperts <= 256 && kMoeMaxTokens <= 64, "ids in a byte, tokens in a 64-bit mask");
constexpr int kMoeHeaderBytes = (sizeof(MoeHeader) + 1023) / 1024 * 1024;
static_assert(kMoeHeaderBytes <= 20 * 1024, "header");

// Routing of all tokens, by every thread of the CTA: the chosen experts with
// their weights, the chunks, and the slots. Larger logit first, ties to the
// lower index; a NaN counts as minus infinity (its weights are NaN all the same).
__device__ __forceinline__ void moe_route(const MoeArgs &a, MoeHeader *h) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const double ninf = -INFINITY;
    for (int e = threadIdx.x; e < kMoeMaxExperts; e += kMoeThreads) h->mask[e] = 0;
    __syncthreads();
    for (int m = warp; m < a.M; m += kMoeThreads / 32) {
        constexpr int kPer = kMoeMaxExperts / 32;
        double v[kPer];
        float ex[kPer];
        double top = ninf;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            v[i] = e < a.E ? __ldcg(a.logits + static_cast<int64_t>(m) * a.E + e) : ninf;
            if (isnan(v[i])) {
                nan = true;
                v[i] = ninf;
            }
            top = fmax(top, v[i]);
        }
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
        nan = __any_sync(0xffffffffu, nan) != 0;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            ex[i] = lane + 32 * i < a.E ? expf(static_cast<float>(v[i] - top)) : 0.0f;
            sum += ex[i];
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float chosen = 0.0f, mine = 0.0f;
        uint32_t taken = 0;                      // of this lane's experts
        int my_id = 0;
        for (int j = 0; j < a.top_k; ++j) {
            double b = ninf;
            int bi = 0x7fffffff;
            float be = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = lane + 32 * i;
                if (e < a.E && !((taken >> i) & 1u) && (bi == 0x7fffffff || v[i] > b)) {
                    b = v[i];
                    bi = e;
                    be = ex[i];
                }
            }
            for (int o = 16; o > 0; o >>= 1) {
                const double ob = __shfl_xor_sync(0xffffffffu, b, o);
                const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
                const float oe = __shfl_xor_sync(0xffffffffu, be, o);
                if (ob > b || (ob == b && oi < bi)) {
                    b = ob;
                    bi = oi;
                    be = oe;
                }
            }
            if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
            chosen += be;
            if (lane == j) {
                my_id = bi;
                mine = be;
            }
        }
        if (lane < a.top_k) {
            float w = mine / (a.renorm ? chosen : sum);
            if (nan) w = __int_as_float(0x7fffffff);
            const int i = m * a.top_k + lane;
            h->id[i] = static_cast<uint8_t>(my_id);
            h->w[i] = w;
            atomicOr(&h->mask[my_id], 1ull << m);
            if (blockIdx.x == 0) {
                if (a.ids) a.ids[i] = my_id;
                if (a.weights) a.weights[i] = w;
            }
        }
    }
    __syncthreads();
    // exclusive sums over the experts of their slots and chunks
    const int e = threadIdx.x;
    int n = 0, nc = 0, s_in = 0, c_in = 0;
    if (e < kMoeMaxExperts) {
        n = e < a.E ? __popcll(h->mask[e]) : 0;
        nc = (n + kMoeChunk - 1) / kMoeChunk;
        s_in = n;
        c_in = nc;
        for (int o = 1; o < 32; o <<= 1) {
            const int s = __shfl_up_sync(0xffffffffu, s_in, o), c = __shfl_up_sync(0xffffffffu, c_in, o);
            if (lane >= o) {
                s_in += s;
                c_in += c;
            }
        }
        if (lane == 31) {
            h->warp_slots[warp] = s_in;
            h->warp_chunks[warp] = c_in;
        }
    }
    __syncthreads();
    if (e < kMoeMaxExperts) {
        int s0 = s_in - n, c0 = c_in - nc;
        for (int w = 0; w < warp; ++w) {
            s0 += h->warp_slots[w];
            c0 += h->warp_chunks[w];
        }
        h->slot0[e] = static_cast<uint16_t>(s0);
        for (int i = 0; i < nc; ++i)
            h->chunk[c0 + i] = {static_cast<uint16_t>(e), static_cast<uint16_t>(s0 + i * kMoeChunk),
                                static_cast<uint16_t>(min(kMoeChunk, n - i * kMoeChunk)), 0};
        if (e == kMoeMaxExperts - 1) h->nchunks = c0 + nc;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.M * a.top_k; i += kMoeThreads) {
        const int m = i / a.top_k, id = h->id[i];
        const int s = h->slot0[id] + __popcll(h->mask[id] & ((1ull << m) - 1));
        h->token[s] = static_cast<uint8_t>(m);
        h->slot_of[i] = static_cast<uint16_t>(s);
        h->weight[s] = h->w[i];
    }
    __syncthreads();
}

template <int THREADS>
__device__ __forceinline__ void group_sync(int grp) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(THREADS) : "memory");
}

// A walk over a group's items: (chunk, tile) in steps of the number of groups.
struct MoeWalk {
    int chunk, tile;
    __device__ __forceinline__ void next(int dchunk, int dtile, int tiles) {
        chunk += dchunk;
        tile += dtile;
        if (tile >= tiles) {
            tile -= tiles;
            ++chunk;
        }
    }
};

// GW: warps of a group. PAIRS: 8-bit scales of 64-element blocks, an even number
// to a row, so that the two scales of a step are one aligned 16-bit load (the
// usual weight; the other scale forms take single loads).
template <bool DOWN, int GW, bool PAIRS>
__global__ void __launch_bounds__(kMoeThreads, 1)
nf4_moe_experts_kernel(const __grid_constant__ CUtensorMap tm_codes,   // u8, 64-byte swizzle; down: [rows, K/2], box
                                                                       // {64, 64}; gate_up: [2 E, F, K/2], box {64, 32, 2}
                       const MoeArgs a) {
    constexpr int kGroups = kMoeWarps / GW;
    extern __shared__ __align__(1024) uint8_t dsm[];
    const uint32_t sbase = smem_u32(dsm);
    const uint32_t low0 = (sbase + kMoeHeaderBytes + 1023u) & ~1023u;
    const uint32_t win_end = sbase + kDsDynBytes;
    const uint32_t nlow = low0 <= kDsLutAddr ? (kDsLutAddr - low0) / kMoeSlotBytes : 0u;
    const uint32_t nhigh = win_end >= kDsHighAddr ? (win_end - kDsHighAddr) / kMoeSlotBytes : 0u;
    if (low0 > kDsLutAddr || win_end < kDsHighAddr || nlow + nhigh < kMoeWarps * kMoeRing) {
        if (threadIdx.x == 0) record_status(NF4_ERR_CUDA);     // the fixed addresses are not ours
        return;
    }
    MoeHeader *hd = reinterpret_cast<MoeHeader *>(dsm);
    volatile int *abort_flag = &hd->abort_flag;
    uint8_t *lut_g = dsm + (kDsLutAddr - sbase);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = warp / GW, gw = warp % GW;
    const int g = lane >> 2, t = lane & 3;

    if (threadIdx.x == 0) {
        for (int w = 0; w < kMoeWarps; ++w)
            for (int s = 0; s < kMoeRing; ++s) mbar_init(&hd->bars[w][s], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_codes);
    }
    for (int idx = threadIdx.x; idx < 256 * 32; idx += kMoeThreads) {
        const int b = idx >> 5, l = idx & 31;
        *reinterpret_cast<uint32_t *>(lut_g + b * 256 + 4 * l) =
            bf16_pack(kMoeLevelUp * c_levels[b >> 4], kMoeLevelUp * c_levels[b & 15]);
    }
    griddep_wait();
    griddep_launch_dependents();
    if constexpr (!DOWN) {
        __syncthreads();
        moe_route(a, hd);
        if (blockIdx.x == 0) {
            MoeRoute *r = a.route;
            if (threadIdx.x == 0) r->nchunks = hd->nchunks;
            for (int i = threadIdx.x; i < hd->nchunks; i += kMoeThreads) r->chunk[i] = hd->chunk[i];
            for (int i = threadIdx.x; i < a.M * a.top_k; i += kMoeThreads) {
                r->weight[i] = hd->weight[i];
                r->slot_of[i] = hd->slot_of[i];
            }
        }
    } else {
        const MoeRoute *r = a.route;
        const int most = min(kMoeMaxChunks, a.M * a.top_k);
        if (threadIdx.x == 0) hd->nchunks = __ldcg(&r->nchunks);
        for (int i = threadIdx.x; i < most; i += kMoeThreads) {
            const uint2 v = __ldcg(reinterpret_cast<const uint2 *>(r->chunk) + i);
            *reinterpret_cast<uint2 *>(&hd->chunk[i]) = v;
        }
        for (int i = threadIdx.x; i < a.M * a.top_k; i += kMoeThreads) {
            hd->weight[i] = __ldcg(r->weight + i);
            hd->slot_of[i] = __ldcg(r->slot_of + i);
        }
        __syncthreads();
    }

    const int K = DOWN ? a.F : a.H;
    const int kblocks = K / kBlock;
    const int nkc = (kblocks + 1) / 2;                         // steps of an item
    const int tiles = DOWN ? a.H / kMoeRows : a.F / (kMoeRows / 2);
    const int nchunks = hd->nchunks;
    const int bpr = kblocks >> a.bshift;                       // scale blocks of a weight row
    const int stride = static_cast<int>(gridDim.x) * kGroups;
    const int first = static_cast<int>(blockIdx.x) + grp * static_cast<int>(gridDim.x);
    const int dchunk = stride / tiles, dtile = stride - dchunk * tiles;
    MoeWalk item{first / tiles, first % tiles};

    uint32_t slot[kMoeRing];
#pragma unroll
    for (int s = 0; s < kMoeRing; ++s) {
        const uint32_t i = static_cast<uint32_t>(warp * kMoeRing + s);
        slot[s] = i < nlow ? low0 + i * kMoeSlotBytes : kDsHighAddr + (i - nlow) * kMoeSlotBytes;
    }

    // ---- requests: one step ahead of the computation, across items. A warp
    // with gw >= nkc has no steps and only takes part in the joining of sums.
    const bool any = gw < nkc;
    int issued = 0, landed = 0;
    MoeWalk iw = item;
    int ikc = gw, ic1 = 0, ic2 = 0;                            // box coordinates of iw's item
    auto box_of = [&]() {
        if (iw.chunk >= nchunks) return;
        const int e = hd->chunk[iw.chunk].expert;
        ic1 = DOWN ? e * a.H + iw.tile * kMoeRows : iw.tile * (kMoeRows / 2);
        ic2 = 2 * e;
    };
    auto issue = [&]() {
        if (!any || iw.chunk >= nchunks || abort_raised(abort_flag)) return;
        if (lane == 0) {
            const int s = issued % kMoeRing;
            uint64_t *bar = &hd->bars[warp][s];
            fence_proxy_async_smem();      // the slot was read through the generic proxy
            mbar_arrive_expect_tx(bar, kMoeSlotBytes);
            if constexpr (DOWN) tma_load_2d(dsm + (slot[s] - sbase), &tm_codes, bar, ikc * kMoeStepBytes, ic1);
            else tma_load_3d(dsm + (slot[s] - sbase), &tm_codes, bar, ikc * kMoeStepBytes, ic1, ic2);
        }
        ++issued;
        ikc += GW;
        if (ikc >= nkc) {
            ikc = gw;
            iw.next(dchunk, dtile, tiles);
            box_of();
        }
    };

    // Which row of a 16-row tile lane group g reads: with 64-byte rows under
    // the 64-byte swizzle, rows {0,1,4,5} (and {2,3,6,7}) of one block take
    // all 32 banks once.
    const int prow = (g & 1) | ((g & 2) << 1) | ((g & 4) >> 1);

    // ---- operands of the next step: the raw scales of this lane's two rows
    // (rows prow and prow + 8 of tile t) and the activations of its token g.
    // Lanes beyond the chunk's tokens read its last token again: their columns
    // of the products are never stored. After the group's last item the cursor
    // stays where it is, so every load below is of something valid.
    MoeWalk nw = item;
    int nkc_at = gw;
    const uint16_t *nx = nullptr;                              // x (or a) at token g, element 16 t
    uint32_t nsb = 0;                                          // scale index of the first row; the second is 8 bpr on
    auto operands_of = [&]() {
        const MoeChunk c = hd->chunk[nw.chunk];
        const int sl = c.slot0 + min(g, c.n - 1);
        nx = (DOWN ? a.a + static_cast<int64_t>(sl) * K : a.x + static_cast<int64_t>(hd->token[sl]) * K) + 16 * t;
        const int row = DOWN ? c.expert * a.H + nw.tile * kMoeRows + 16 * t
                             : (c.expert * 2 + (t >> 1)) * a.F + nw.tile * (kMoeRows / 2) + 16 * (t & 1);
        nsb = static_cast<uint32_t>(row + prow) * static_cast<uint32_t>(bpr);
    };
    auto next_operands = [&]() {
        nkc_at += GW;
        if (nkc_at >= nkc) {
            MoeWalk w = nw;
            w.next(dchunk, dtile, tiles);
            if (w.chunk < nchunks) {
                nw = w;
                nkc_at = gw;
                operands_of();
            } else {
                nkc_at -= GW;
            }
        }
    };
    uint32_t raw[2][PAIRS ? 1 : 2];                            // [row][block]: q8 codes, or the absmax bits
    float grp_c[2][PAIRS ? 1 : 2];                             // their group constants
    auto load_scales = [&]() {
        const int b0 = 2 * nkc_at;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at = nsb + static_cast<uint32_t>(8 * i * bpr + (b0 >> a.bshift));
            if constexpr (PAIRS) {
                raw[i][0] = __ldg(reinterpret_cast<const uint16_t *>(a.q8 + at));
                grp_c[i][0] = __ldg(a.cg + (at >> 8));
            } else {
                // the second block of a step: its own scale, the same one (128-element
                // blocks), or, behind the row's last block, not used
                const uint32_t at1 = a.bshift || b0 + 1 >= kblocks ? at : at + 1;
                if (a.dq) {
                    raw[i][0] = __ldg(a.q8 + at);
                    raw[i][1] = __ldg(a.q8 + at1);
                    grp_c[i][0] = __ldg(a.cg + (at >> 8));
                    grp_c[i][1] = __ldg(a.cg + (at1 >> 8));
                } else {
                    raw[i][0] = __float_as_uint(__ldg(a.absmax + at));
                    raw[i][1] = __float_as_uint(__ldg(a.absmax + at1));
                }
            }
        }
    };
    // (c / 127 by its reciprocal: one rounding away, and the sums are not compared bit for bit)
    auto scale_of = [&](int i, int b) -> float {
        if constexpr (PAIRS) {
            const uint32_t q = b ? raw[i][0] >> 8 : raw[i][0] & 0xffu;
            return static_cast<float>(q) * (grp_c[i][0] * (kMoeLevelDown / 127.0f));
        } else {
            return a.dq ? static_cast<float>(raw[i][b]) * (grp_c[i][b] * (kMoeLevelDown / 127.0f))
                        : __uint_as_float(raw[i][b]) * kMoeLevelDown;
        }
    };
    uint4 xv[2][2];                                            // [block][half]
    auto load_x = [&](int b) {
        const int blk = min(2 * nkc_at + b, kblocks - 1);
        const uint4 *q = reinterpret_cast<const uint4 *>(nx + blk * kBlock);
        xv[b][0] = q[0];
        xv[b][1] = q[1];
    };

    const uint32_t lanew = (static_cast<uint32_t>(lane) << 2) | (1u << 16);
    const uint32_t swz = static_cast<uint32_t>((prow >> 1) & 3);
    const uint32_t code_row = static_cast<uint32_t>(prow) * kMoeStepBytes + 8u * (t & 1);
    const uint32_t code_chunk[2] = {((0u + (t >> 1)) ^ swz) << 4, ((2u + (t >> 1)) ^ swz) << 4};
    // this thread's place in the group's partial sums: lane's sums j and j + 8
    // for j = gw, gw + GW, ... < 8 (j = 4 tile + element)
    auto park = [&](int w, int j) {
        return reinterpret_cast<float *>(lut_g + ((grp * GW + w) * 16 + j) * 256 + 128 + 4 * lane);
    };

    // down: the item before's place in the count of its stripe, looked at one
    // item later, when the atomic has long returned
    int seen = -1, seen_tile = 0;
    auto combine = [&](int tile) {
        // every slot's share of these 64 columns is there: each token's top_k
        // of them are added in order
        const int gt = gw * 32 + lane;
        const int h = tile * kMoeRows + (gt & 63);
        for (int m = gt >> 6; m < a.M; m += GW / 2) {
            float v = 0.0f;
            for (int j = 0; j < a.top_k; ++j)
                v += __ldcg(a.y + static_cast<int64_t>(hd->slot_of[m * a.top_k + j]) * a.H + h);
            const int64_t o = static_cast<int64_t>(m) * a.H + h;
            if (a.residual) v += bf16_lo(a.residual[o]);
            const __nv_bfloat16 b = __float2bfloat16_rn(v);
            a.out[o] = *reinterpret_cast<const uint16_t *>(&b);
        }
    };

    box_of();
    issue();
    if (any && item.chunk < nchunks) {
        operands_of();
        load_scales();
        load_x(0);
        load_x(1);
    }

    for (; item.chunk < nchunks; item.next(dchunk, dtile, tiles)) {
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
        for (int kc = gw; kc < nkc; kc += GW) {
            float sc[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[i][b] = scale_of(i, b);
            next_operands();
            load_scales();
            issue();
            const int rs = landed % kMoeRing;
            if (mbar_wait_warp(&hd->bars[warp][rs], static_cast<uint32_t>(landed / kMoeRing) & 1u, abort_flag)) ++landed;
            const uint32_t cbase = slot[rs] + code_row + after_wait_zero();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (b == 1 && 2 * kc + 1 >= kblocks) break;    // an odd row's last step is one block
                uint2 cw[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi)
                        cw[i][hi] = ds_lds64(cbase + (16 * i + 8 * hi) * kMoeStepBytes + code_chunk[b]);
                float pp[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 &x4 = xv[b][q >> 1];
                    const uint32_t b0 = (q & 1) ? x4.z : x4.x, b1 = (q & 1) ? x4.w : x4.y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t wl = (q < 2) ? cw[i][0].x : cw[i][0].y;
                        const uint32_t wh = (q < 2) ? cw[i][1].x : cw[i][1].y;
                        uint32_t af[4];
                        if (q & 1) {
                            af[0] = ds_lut(ds_addr<2>(wl, lanew));
                            af[1] = ds_lut(ds_addr<2>(wh, lanew));
                            af[2] = ds_lut(ds_addr<3>(wl, lanew));
                            af[3] = ds_lut(ds_addr<3>(wh, lanew));
                        } else {
                            af[0] = ds_lut(ds_addr<0>(wl, lanew));
                            af[1] = ds_lut(ds_addr<0>(wh, lanew));
                            af[2] = ds_lut(ds_addr<1>(wl, lanew));
                            af[3] = ds_lut(ds_addr<1>(wh, lanew));
                        }
                        if (q == 0) ds_mma_zero(pp[i], af, b0, b1);
                        else mma_bf16_16816(pp[i], af, b0, b1);
                    }
                }
                load_x(b);              // the next step's, into the registers just read
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // rows prow and prow + 8 of tile i: lane (g, i) of this quad has their scales
                    const float s0 = __shfl_sync(0xffffffffu, sc[0][b], (lane & ~3) | i);
                    const float s1 = __shfl_sync(0xffffffffu, sc[1][b], (lane & ~3) | i);
                    acc[i][0] = fmaf(s0, pp[i][0], acc[i][0]);
                    acc[i][1] = fmaf(s0, pp[i][1], acc[i][1]);
                    acc[i][2] = fmaf(s1, pp[i][2], acc[i][2]);
                    acc[i][3] = fmaf(s1, pp[i][3], acc[i][3]);
                }
            }
            if (2 * kc + 1 >= kblocks) load_x(1);
            __syncwarp();               // every lane has read the slot
        }

        // ---- the group's k splits meet in the odd halves of the table rows,
        // and are added in warp order
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) *park(gw, i * 4 + e) = acc[i][e];
        if (DOWN && gw == 0 && lane == 0) hd->last[grp] = seen == nchunks - 1;
        group_sync<32 * GW>(grp);
        if (DOWN && hd->last[grp]) combine(seen_tile);
        const MoeChunk c = hd->chunk[item.chunk];
#pragma unroll
        for (int j = gw; j < 8; j += GW) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int w = 0; w < GW; ++w) {
                s0 += *park(w, j);
                s1 += *park(w, j + 8);
            }
            const int e = j & 3;
            const int rr = 16 * (j >> 2) + prow + 8 * (e >> 1), col = 2 * t + (e & 1);
            if (col < c.n) {
                if constexpr (!DOWN) {
                    // s0 is gate row rr, s1 up row rr
                    const __nv_bfloat16 v = __float2bfloat16_rn(act_value(s0, a.act) * s1);
                    a.a[static_cast<int64_t>(c.slot0 + col) * a.F + item.tile * (kMoeRows / 2) + rr] =
                        *reinterpret_cast<const uint16_t *>(&v);
                } else {
                    const float w = hd->weight[c.slot0 + col];
                    float *y = a.y + static_cast<int64_t>(c.slot0 + col) * a.H + item.tile * kMoeRows + rr;
                    __stcg(y, w * s0);
                    __stcg(y + 32, w * s1);
                }
            }
        }
        group_sync<32 * GW>(grp);        // the partials are free again, the products written
        if (DOWN) {
            seen_tile = item.tile;
            if (gw == 0 && lane == 0) {
                __threadfence();         // the group's products before the count
                seen = atomicAdd(a.done + item.tile, 1);
                __threadfence();
            }
        }
    }
    if (DOWN) {
        if (gw == 0 && lane == 0) hd->last[grp] = seen == nchunks - 1;
        group_sync<32 * GW>(grp);
        if (hd->last[grp]) combine(seen_tile);
    }
    // leave no copy in flight into shared memory that is about to be released
    // (after a normal end every copy has landed)
    if (lane == 0)
        for (int s = landed; s < issued; ++s)
            mbar_drain(&hd->bars[warp][s % kMoeRing], static_cast<uint32_t>(s / kMoeRing) & 1u);
    __syncwarp();
}

}  // namespace nf4
