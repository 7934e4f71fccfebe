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
// An item belongs to a group of 8 warps (two groups a CTA, each with its own
// barrier, so that one computes while the other joins its sums). The warps
// split k in steps of 128 elements: warp w takes steps w, w + 8, ... A step is
// 64 rows x 64 bytes of codes, brought by TMA into the warp's own ring of two
// slots, one step ahead across items. As in the streaming kernel of the linear
// layer, a code byte becomes two bf16 levels by one byte permute and one
// conflict-free shared load, the products run on mma.sync with the tokens as
// its 8 columns (16 x 8 x 16; a tcgen05 tile would spend 128 rows on at most 8
// tokens and need the operand written to shared memory), and a 64-element
// block's fp32 partial is multiplied by its scale once.
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
constexpr int kMoeGroups = 2;
constexpr int kMoeGroupWarps = 8;
constexpr int kMoeThreads = 32 * kMoeGroups * kMoeGroupWarps;
constexpr int kMoeRows = 64;                       // weight rows of one item
constexpr int kMoeStepBytes = 64;                  // code bytes of one row in a step: 2 blocks
constexpr int kMoeSlotBytes = kMoeRows * kMoeStepBytes;
constexpr int kMoeRing = 2;

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
    uint64_t bars[kMoeGroups * kMoeGroupWarps][kMoeRing];
    int abort_flag;
    int nchunks;
    int last[kMoeGroups];
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

__device__ __forceinline__ void group_sync(int grp) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * kMoeGroupWarps) : "memory");
}

// One position of a warp in its walk: step kc of work item `item`.
struct MoePos {
    int item, kc;
};

template <bool DOWN>
__global__ void __launch_bounds__(kMoeThreads, 1)
nf4_moe_experts_kernel(const __grid_constant__ CUtensorMap tm_codes,   // [rows, K/2] u8, box {64, 32}, 64-byte swizzle
                       const MoeArgs a) {
    extern __shared__ __align__(1024) uint8_t dsm[];
    const uint32_t sbase = smem_u32(dsm);
    const uint32_t low0 = (sbase + kMoeHeaderBytes + 1023u) & ~1023u;
    const uint32_t win_end = sbase + kDsDynBytes;
    const uint32_t nlow = low0 <= kDsLutAddr ? (kDsLutAddr - low0) / kMoeSlotBytes : 0u;
    const uint32_t nhigh = win_end >= kDsHighAddr ? (win_end - kDsHighAddr) / kMoeSlotBytes : 0u;
    constexpr uint32_t kSlots = kMoeGroups * kMoeGroupWarps * kMoeRing;
    if (low0 > kDsLutAddr || win_end < kDsHighAddr || nlow + nhigh < kSlots) {
        if (threadIdx.x == 0) record_status(NF4_ERR_CUDA);     // the fixed addresses are not ours
        return;
    }
    MoeHeader *hd = reinterpret_cast<MoeHeader *>(dsm);
    volatile int *abort_flag = &hd->abort_flag;
    uint8_t *lut_g = dsm + (kDsLutAddr - sbase);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = warp / kMoeGroupWarps, gw = warp % kMoeGroupWarps;
    const int g = lane >> 2, t = lane & 3;

    if (threadIdx.x == 0) {
        for (int w = 0; w < kMoeGroups * kMoeGroupWarps; ++w)
            for (int s = 0; s < kMoeRing; ++s) mbar_init(&hd->bars[w][s], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_codes);
    }
    for (int idx = threadIdx.x; idx < 256 * 32; idx += kMoeThreads) {
        const int b = idx >> 5, l = idx & 31;
        *reinterpret_cast<uint32_t *>(lut_g + b * 256 + 4 * l) = bf16_pack(c_levels[b >> 4], c_levels[b & 15]);
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
    const int nitems = hd->nchunks * tiles;
    const int stride = static_cast<int>(gridDim.x) * kMoeGroups;
    const int first = static_cast<int>(blockIdx.x) + grp * static_cast<int>(gridDim.x);
    const int bpr = kblocks >> a.bshift;                       // scale blocks of a weight row

    // first weight row of an item's two 32-row halves
    auto rows_of = [&](int item, int &r0, int &r1) {
        const int c = item / tiles, tile = item - c * tiles;
        const int e = hd->chunk[c].expert;
        if (DOWN) {
            r0 = e * a.H + tile * kMoeRows;
            r1 = r0 + kMoeRows / 2;
        } else {
            r0 = e * 2 * a.F + tile * (kMoeRows / 2);
            r1 = r0 + a.F;
        }
    };
    auto advance = [&](MoePos &p) {
        p.kc += kMoeGroupWarps;
        if (p.kc >= nkc) {
            p.kc = gw;
            p.item += stride;
        }
    };
    const bool any = gw < nkc;                                 // this warp has steps at all
    auto valid = [&](const MoePos &p) { return any && p.item < nitems; };

    uint32_t slot[kMoeRing];
#pragma unroll
    for (int s = 0; s < kMoeRing; ++s) {
        const uint32_t i = static_cast<uint32_t>(warp * kMoeRing + s);
        slot[s] = i < nlow ? low0 + i * kMoeSlotBytes : kDsHighAddr + (i - nlow) * kMoeSlotBytes;
    }
    int issued = 0, landed = 0;
    MoePos ip{first, gw};                                      // the next step to request
    auto issue = [&]() {
        if (!valid(ip) || abort_raised(abort_flag)) return;
        if (lane == 0) {
            int r0, r1;
            rows_of(ip.item, r0, r1);
            uint64_t *bar = &hd->bars[warp][issued % kMoeRing];
            uint8_t *dst = dsm + (slot[issued % kMoeRing] - sbase);
            fence_proxy_async_smem();      // the slot was read through the generic proxy
            mbar_arrive_expect_tx(bar, kMoeSlotBytes);
            tma_load_2d(dst, &tm_codes, bar, ip.kc * kMoeStepBytes, r0);
            tma_load_2d(dst + kMoeSlotBytes / 2, &tm_codes, bar, ip.kc * kMoeStepBytes, r1);
        }
        ++issued;
        advance(ip);
    };

    // Raw scales of a step for this lane's two rows: 16 t + prow and 8 more
    // (the rows whose sums the lane's quad forms in tile t).
    // Which row of a 16-row tile lane group g reads: with 64-byte rows under
    // the 64-byte swizzle, rows {0,1,4,5} (and {2,3,6,7}) of one block take
    // all 32 banks once.
    const int prow = (g & 1) | ((g & 2) << 1) | ((g & 4) >> 1);
    struct Raw {
        uint32_t s[2][2];       // [row][block]: q8 code, or the absmax bits
        float c[2][2];          // their group constants
    };
    auto load_scales = [&](const MoePos &p) -> Raw {
        Raw r;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                r.s[i][b] = 0u;
                r.c[i][b] = 0.0f;
            }
        if (!valid(p)) return r;
        int r0, r1;
        rows_of(p.item, r0, r1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = (t < 2 ? r0 : r1 - kMoeRows / 2) + 16 * t + prow + 8 * i;
            const int64_t rb = static_cast<int64_t>(row) * bpr;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int blk = 2 * p.kc + b;
                if (blk < kblocks) {
                    const int64_t at = rb + (blk >> a.bshift);
                    if (a.dq) {
                        r.s[i][b] = __ldg(a.q8 + at);
                        r.c[i][b] = __ldg(a.cg + (at >> 8));
                    } else {
                        r.s[i][b] = __float_as_uint(__ldg(a.absmax + at));
                    }
                }
            }
        }
        return r;
    };
    // the activations of a step: per block the 16 elements [16 t, 16 t + 16) of slot g's token
    auto load_x = [&](const MoePos &p, uint4 (&xv)[2][2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) xv[b][0] = xv[b][1] = make_uint4(0, 0, 0, 0);
        if (!valid(p)) return;
        const MoeChunk c = hd->chunk[p.item / tiles];
        if (g >= c.n) return;
        const uint16_t *row = DOWN ? a.a + static_cast<int64_t>(c.slot0 + g) * K
                                   : a.x + static_cast<int64_t>(hd->token[c.slot0 + g]) * K;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int blk = 2 * p.kc + b;
            if (blk < kblocks) {
                const uint4 *q = reinterpret_cast<const uint4 *>(row + blk * kBlock + 16 * t);
                xv[b][0] = q[0];
                xv[b][1] = q[1];
            }
        }
    };

    const uint32_t lanew = (static_cast<uint32_t>(lane) << 2) | (1u << 16);
    const uint32_t swz = static_cast<uint32_t>((prow >> 1) & 3);
    const uint32_t code_row = static_cast<uint32_t>(prow) * kMoeStepBytes + 8u * (t & 1);
    const uint32_t code_chunk[2] = {((0u + (t >> 1)) ^ swz) << 4, ((2u + (t >> 1)) ^ swz) << 4};

    issue();
    MoePos np{first, gw};                                      // the step whose operands are in flight
    Raw raw = load_scales(np);
    uint4 xn[2][2];
    load_x(np, xn);

    for (int item = first; item < nitems; item += stride) {
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
        for (int kc = gw; kc < nkc; kc += kMoeGroupWarps) {
            uint4 xc[2][2];
            float sc[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                xc[b][0] = xn[b][0];
                xc[b][1] = xn[b][1];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    // (c / 127 by its reciprocal: one rounding away, and the sums are not compared bit for bit)
                    sc[i][b] = a.dq ? static_cast<float>(raw.s[i][b]) * (raw.c[i][b] * (1.0f / 127.0f))
                                    : __uint_as_float(raw.s[i][b]);
            }
            advance(np);
            raw = load_scales(np);
            load_x(np, xn);
            issue();
            const int rs = landed % kMoeRing;
            if (mbar_wait_warp(&hd->bars[warp][rs], static_cast<uint32_t>(landed / kMoeRing) & 1u, abort_flag)) ++landed;
            const uint32_t cbase = slot[rs] + code_row + after_wait_zero();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint2 cw[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi)
                        cw[i][hi] = ds_lds64(cbase + (16 * i + 8 * hi) * kMoeStepBytes + code_chunk[b]);
                float pp[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 &xv = xc[b][q >> 1];
                    const uint32_t b0 = (q & 1) ? xv.z : xv.x, b1 = (q & 1) ? xv.w : xv.y;
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
            __syncwarp();               // every lane has read the slot
        }

        // ---- the group's k splits meet in the odd halves of the table rows,
        // and are added in warp order
        auto park = [&](int w, int j) {
            return reinterpret_cast<float *>(lut_g + (grp * 128 + w * 16 + j) * 256 + 128 + 4 * lane);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) *park(gw, i * 4 + e) = acc[i][e];
        group_sync(grp);
        const int ch = item / tiles, tile = item - ch * tiles;
        const MoeChunk c = hd->chunk[ch];
        float s0 = 0.0f, s1 = 0.0f;
        // thread (gw, lane) takes sums gw and gw + 8 of its lane: tile i = j / 4, element e = j % 4
#pragma unroll
        for (int w = 0; w < kMoeGroupWarps; ++w) {
            s0 += *park(w, gw);
            s1 += *park(w, gw + 8);
        }
        const int e = gw & 3, i0 = gw >> 2;
        const int rr = 16 * i0 + prow + 8 * (e >> 1), col = 2 * t + (e & 1);
        if constexpr (!DOWN) {
            // s0 is gate row rr, s1 up row rr
            if (col < c.n) {
                const __nv_bfloat16 v = __float2bfloat16_rn(act_value(s0, a.act) * s1);
                a.a[static_cast<int64_t>(c.slot0 + col) * a.F + tile * (kMoeRows / 2) + rr] =
                    *reinterpret_cast<const uint16_t *>(&v);
            }
            group_sync(grp);            // the partials are free again
        } else {
            const int h0 = tile * kMoeRows;
            if (col < c.n) {
                const float w = hd->weight[c.slot0 + col];
                float *y = a.y + static_cast<int64_t>(c.slot0 + col) * a.H + h0;
                __stcg(y + rr, w * s0);
                __stcg(y + rr + 32, w * s1);
            }
            __threadfence();
            group_sync(grp);
            const int gt = gw * 32 + lane;
            if (gt == 0) {
                const int seen = atomicAdd(a.done + tile, 1);
                __threadfence();
                hd->last[grp] = seen == hd->nchunks - 1;
            }
            group_sync(grp);
            if (hd->last[grp]) {
                // every slot's share of these 64 columns is there: each token's
                // top_k of them are added in order
                const int h = h0 + (gt & 63);
                for (int m = gt >> 6; m < a.M; m += 4) {
                    float v = 0.0f;
                    for (int j = 0; j < a.top_k; ++j)
                        v += __ldcg(a.y + static_cast<int64_t>(hd->slot_of[m * a.top_k + j]) * a.H + h);
                    const int64_t o = static_cast<int64_t>(m) * a.H + h;
                    if (a.residual) v += bf16_lo(a.residual[o]);
                    const __nv_bfloat16 b = __float2bfloat16_rn(v);
                    a.out[o] = *reinterpret_cast<const uint16_t *>(&b);
                }
            }
        }
    }
    // leave no copy in flight into shared memory that is about to be released
    // (after a normal end every copy has landed)
    if (lane == 0)
        for (int s = landed; s < issued; ++s)
            mbar_drain(&hd->bars[warp][s % kMoeRing], static_cast<uint32_t>(s / kMoeRing) & 1u);
    __syncwarp();
}

}  // namespace nf4
