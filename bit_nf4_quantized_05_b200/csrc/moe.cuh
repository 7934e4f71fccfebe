// moe.cuh -- a mixture-of-experts layer over NF4 experts for a few tokens:
//
//   l = x R^T, p = softmax(l), the top_k experts of each token with weights w
//   a_e = act(x Wg_e^T) . (x Wu_e^T),   out = sum_j w_j a_{e_j} Wd_{e_j}^T (+ residual)
//
// Two kernels, the second launched while the first drains:
//   nf4_moe_router_kernel    the logits, summed in fp64
//   nf4_moe_experts_kernel   routing (every CTA for itself: the logits are a few
//                            KB), a_e of the chosen experts, then the down
//                            products and their weighted sum
// The experts' codes are nearly all the bytes: 3 H F / 2 per chosen expert.
//
// A token chooses an expert at most once, so routing is a bit mask of tokens
// per expert (an order-free OR, so the result does not depend on timing). An
// expert's tokens are cut into chunks of 8 (the columns of one MMA) and
// numbered as slots, expert by expert; the work items are (chunk, 64 weight
// rows): 32 gate rows and the 32 up rows of the same features, or 64 down rows.
// Groups of warps take items from one counter, all gate-up items before the
// down items. A down item waits until its chunk's gate-up items are done; those
// were all taken before it by groups that are running and never wait, so the
// wait ends whatever part of the grid is resident. (As two kernels, the second
// one's start and the first one's last, uneven round cost 12 of 105 us for 16
// tokens at 6 of 64 experts of 2048 x 1408.)
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
//
// What bounds it: some 300 SM cycles per 4 KB of codes (4.0 TB/s over the card)
// against 178 at HBM's rate. The shared-memory pipe takes 235 to 268 wavefronts of
// them (128 table lookups, 32 for the codes, 16 shuffles of scales, operands, sums),
// but leaving out any one part saves an eighth at most. Around that, a call spends
// about 12 us on router, routing and the first codes, and one item's time at the
// uneven end: 24 us for one token at 8 of 64 experts (2048, 1024; 25 MB of codes);
// 171, 195 or 224 us for 4 tokens at 2 of 8 (5120, 13824), as they come to 5, 6 or 7
// different experts of 108 MB each; 94 us for 16 tokens at 6 of 64 (2048, 1408; 54
// experts, 241 MB).
#pragma once

#include <cstddef>
#include <type_traits>

#include "decode_stream.cuh"
#include "epilogue.cuh"
#include "moe_plan.cuh"

namespace nf4 {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
// chunks: every expert's last one may be partly filled
constexpr int kMoeMaxChunks = kMoeMaxExperts + kMoeMaxSlots / kMoeChunk;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMoeRows = 64;                       // weight rows of one item
constexpr int kMoeStepBytes = 64;                  // code bytes of one row in a step: 2 blocks
constexpr int kMoeSlotBytes = kMoeRows * kMoeStepBytes;
constexpr int kMoeRing = 2;

// The table holds T = bf16(1.4367 level), and every scale carries a factor that
// takes the multiple back. bf16 hits some multiples of the 16 levels better than others:
// over the codes of normally distributed weights in blocks of 64 the rounding is 0.078%
// of a weight in the mean square at this multiple (found by a search over [1, 2)), against
// 0.136% for bf16(level) itself; in blocks of 128, 0.083% against 0.144%. The factor is not
// 1 / 1.4367 (0.6960395) but the least-squares fit sum p level T / sum p T^2, p the
// frequencies of those codes in blocks of 64. For blocks of 128 the fit is 6e-5 higher,
// far inside bf16's 2^-8 of every result.
constexpr float kMoeLevelUp = 1.4367f;
constexpr float kMoeLevelDown = 0.69603324f;

struct MoeChunk {
    uint16_t expert;
    uint16_t slot0;      // first slot
    uint16_t n;          // tokens, 1..8
    uint16_t pad;
};

// Scales of one of the two expert weights.
struct MoeScales {
    const float *absmax;
    const uint8_t *q8;
    const float *cg;
    int dq, bshift;
};

// Counters of one call in the workspace, cleared by the router kernel.
struct MoeCounters {
    int claimed;                  // work items taken
    int gate_up_done;             // gate-up items finished
    int chunk_done[kMoeMaxChunks];    // by chunk
    int stripe_done[1];           // [H / 64] down items finished of each stripe of out
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
    MoeScales gate_up, down;
    // workspace
    int splits;                   // of H in the router kernel
    double *logits;               // [splits, M, E] partial sums
    MoeCounters *cnt;
    uint16_t *a;                  // [slots, F] bf16
    float *y;                     // [slots, H] weighted down products
};

// ---------------------------------------------------------------------------
// Router logits in fp64: which experts a token takes is decided by comparing
// them, and a product of two bf16 values is exact in fp64, so sums that differ
// only in their order practically never swap two experts. Bound by latency: a
// CTA forms 4 tokens x 4 experts over 1024 elements of H, 8 to a thread, so that
// every load is in flight at once, and the routing adds the splits in order.
// bf16 becomes fp64 by moving bits: the conversion instruction runs at a few
// results a clock and took 13 of this kernel's 15 us at H = 5120.
// ---------------------------------------------------------------------------
constexpr int kMrThreads = 128;
constexpr int kMrSplit = kMrThreads * 8;
constexpr int kMrTokens = 4, kMrExperts = 4;

// The fp64 value of the bf16 in the low half of b.
__device__ __forceinline__ double bf16_to_f64(uint32_t b) {
    const uint32_t mag = b & 0x7fffu, sign = (b & 0x8000u) << 16;
    if (mag < 0x80u)                                   // zero, or below the normal range
        return mag ? static_cast<double>(__uint_as_float(b << 16)) : __hiloint2double(static_cast<int>(sign), 0);
    // exponent bias 1023 for 127; all ones (infinity, NaN) stays all ones
    const uint32_t hi = (mag << 13) + (mag >= 0x7f80u ? 2u * (896u << 20) : 896u << 20);
    return __hiloint2double(static_cast<int>(hi | sign), 0);
}

__device__ __forceinline__ void bf16_to_f64(const uint4 &v, double (&d)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d[2 * i] = bf16_to_f64(w[i] & 0xffffu);
        d[2 * i + 1] = bf16_to_f64(w[i] >> 16);
    }
}

__global__ void __launch_bounds__(kMrThreads)
nf4_moe_router_kernel(const MoeArgs a) {
    constexpr int kOut = kMrTokens * kMrExperts;
    __shared__ double part[kMrThreads / 32][kOut];
    {
        // on the way into L2 while the kernel before finishes
        const int e = static_cast<int>(blockIdx.x) * kMrExperts + (threadIdx.x >> 5);
        const int k = static_cast<int>(blockIdx.z) * kMrSplit + (threadIdx.x & 31) * 32;
        if (e < a.E && k < a.H)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.router + static_cast<int64_t>(e) * a.H + k));
    }
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        int *c = reinterpret_cast<int *>(a.cnt);
        const int n = static_cast<int>(offsetof(MoeCounters, stripe_done) / 4) + a.H / kMoeRows;
        for (int i = threadIdx.x; i < n; i += kMrThreads) c[i] = 0;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = static_cast<int>(blockIdx.x) * kMrExperts, m0 = static_cast<int>(blockIdx.y) * kMrTokens;
    const int k = static_cast<int>(blockIdx.z) * kMrSplit + threadIdx.x * 8;
    double acc[kOut] = {};                             // [token][expert]
    if (k < a.H) {
        uint4 wv[kMrExperts], xv[kMrTokens];
#pragma unroll
        for (int j = 0; j < kMrExperts; ++j)           // rows behind the last are read as the last
            wv[j] = __ldg(reinterpret_cast<const uint4 *>(a.router + static_cast<int64_t>(min(e0 + j, a.E - 1)) * a.H + k));
#pragma unroll
        for (int i = 0; i < kMrTokens; ++i)
            xv[i] = *reinterpret_cast<const uint4 *>(a.x + static_cast<int64_t>(min(m0 + i, a.M - 1)) * a.H + k);
        double w[kMrExperts][8];
#pragma unroll
        for (int j = 0; j < kMrExperts; ++j) bf16_to_f64(wv[j], w[j]);
#pragma unroll
        for (int i = 0; i < kMrTokens; ++i) {
            if (m0 + i >= a.M) break;
            double x[8];
            bf16_to_f64(xv[i], x);
#pragma unroll
            for (int j = 0; j < kMrExperts; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[i * kMrExperts + j] = fma(x[c], w[j][c], acc[i * kMrExperts + j]);
        }
    }
    // sums over the warp: each step halves the sums a lane still holds; after
    // four, lane l has sum (l >> 1) of its pair
#pragma unroll
    for (int h = kOut / 2, o = 16; h >= 1; h >>= 1, o >>= 1)
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const bool up = (lane & o) != 0;
            const double keep = up ? acc[i + h] : acc[i], send = up ? acc[i] : acc[i + h];
            acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 1);
    if (!(lane & 1)) part[warp][lane >> 1] = acc[0];
    __syncthreads();
    if (threadIdx.x < kOut) {
        const int m = m0 + threadIdx.x / kMrExperts, e = e0 + threadIdx.x % kMrExperts;
        double v = 0.0;
        for (int w = 0; w < kMrThreads / 32; ++w) v += part[w][threadIdx.x];
        if (m < a.M && e < a.E) a.logits[(static_cast<int64_t>(blockIdx.z) * a.M + m) * a.E + e] = v;
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
    int last[kMoeWarps], ready[kMoeWarps];        // by group
    uint32_t claim[kMoeWarps][4];                 // by group: its items, a ring of four
    int start[kMoeWarps][2];                      // by group: its first two, as taken
    int warp_slots[kMoeMaxExperts / 32], warp_chunks[kMoeMaxExperts / 32];
    MoeChunk chunk[kMoeMaxChunks];
    float weight[kMoeMaxSlots];                   // by slot
    uint16_t slot_of[kMoeMaxSlots];               // by token * top_k + j
    unsigned long long mask[kMoeMaxExperts];      // tokens of each expert
    float w[kMoeMaxSlots];                        // by token * top_k + j
    uint8_t id[kMoeMaxSlots];
    uint8_t token[kMoeMaxSlots];                  // by slot
    uint16_t slot0[kMoeMaxExperts];
};
static_assert(kMoeMaxExperts * 12 <= kMoeSlotBytes, "keys and their high words in a ring slot");
static_assert(kMoeMaxExperts <= 256 && kMoeMaxTokens <= 64, "ids in a byte, tokens in a 64-bit mask");
constexpr int kMoeHeaderBytes = (sizeof(MoeHeader) + 1023) / 1024 * 1024;
static_assert(kMoeHeaderBytes <= 20 * 1024, "header");

// fp64 values as integers of the same order, all above 0; NaN as minus infinity.
__device__ __forceinline__ unsigned long long order_key(double v) {
    const unsigned long long b = isnan(v) ? 0xfff0000000000000ull : static_cast<unsigned long long>(__double_as_longlong(v));
    return (b >> 63 ? ~b : b | 1ull << 63) + 1ull;
}
__device__ __forceinline__ double key_value(unsigned long long key) {
    const unsigned long long b = key - 1ull;
    return __longlong_as_double(static_cast<long long>(b >> 63 ? b & ~(1ull << 63) : ~b));
}

// Routing of all tokens, by every thread of the CTA: the chosen experts with
// their weights, the chunks, and the slots. Larger logit first, ties to the
// lower index; a NaN counts as minus infinity (all weights of its token are NaN).
// A warp takes a token. A lane counts, for each of its experts, the keys above:
// by their high words, and by whole keys only where two of those are equal
// (8 rounds of a warp maximum over 64 experts took twice as long). The
// keys are where the warp's ring slots will be: kMoeMaxExperts of them, then
// their high words.
__device__ __forceinline__ void moe_route(const MoeArgs &a, MoeHeader *h, unsigned long long *key) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < kMoeMaxExperts; e += kMoeThreads) h->mask[e] = 0;
    __syncthreads();
    uint32_t *high = reinterpret_cast<uint32_t *>(key + kMoeMaxExperts);
    const int64_t split = static_cast<int64_t>(a.M) * a.E;
#pragma unroll 1
    for (int m = warp; m < a.M; m += kMoeThreads / 32) {
        bool nan = false;
#pragma unroll 1
        for (int e = lane; e < ((a.E + 3) & ~3); e += 32) {
            const double *l = a.logits + static_cast<int64_t>(m) * a.E + e;
            double v = 0.0;
            if (e < a.E) {
#pragma unroll 4
                for (int s = 0; s < a.splits; ++s) v += __ldcg(l + s * split);
            }
            nan |= isnan(v);
            key[e] = e < a.E ? order_key(v) : 0ull;
            high[e] = static_cast<uint32_t>(key[e] >> 32);
        }
        nan = __any_sync(0xffffffffu, nan) != 0;
        __syncwarp();
#pragma unroll 1
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = min(e0 + lane, a.E - 1);
            const uint32_t mine = high[e];
            int rank = 0, same = 0;
#pragma unroll 2
            for (int f = 0; f < a.E; f += 4) {
                const uint4 h4 = *reinterpret_cast<const uint4 *>(high + f);
                rank += (h4.x > mine) + (h4.y > mine) + (h4.z > mine) + (h4.w > mine);
                same += (h4.x == mine) + (h4.y == mine) + (h4.z == mine) + (h4.w == mine);
            }
            if (__any_sync(0xffffffffu, same > 1)) {
                rank = 0;
#pragma unroll 1
                for (int f = 0; f < a.E; ++f) rank += key[f] > key[e] || (key[f] == key[e] && f < e) ? 1 : 0;
            }
            if (e0 + lane < a.E && rank < a.top_k) h->id[m * a.top_k + rank] = static_cast<uint8_t>(e);
        }
        __syncwarp();
        const int my_id = h->id[m * a.top_k + min(lane, a.top_k - 1)];
        const double top = key_value(key[h->id[m * a.top_k]]);
        // (infinities propagate through the sum as in a softmax)
        const float ex = lane < a.top_k ? expf(static_cast<float>(key_value(key[my_id]) - top)) : 0.0f;
        float sum = 0.0f;
        if (a.renorm) {
            sum = ex;
        } else {
#pragma unroll 1
            for (int e = lane; e < a.E; e += 32) sum += expf(static_cast<float>(key_value(key[e]) - top));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane < a.top_k) {
            const float w = nan ? __int_as_float(0x7fffffff) : ex / sum;
            const int i = m * a.top_k + lane;
            h->w[i] = w;
            atomicOr(&h->mask[my_id], 1ull << m);
            if (blockIdx.x == 0) {
                if (a.ids) a.ids[i] = my_id;
                if (a.weights) a.weights[i] = w;
            }
        }
        __syncwarp();
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
#pragma unroll
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
}

template <int THREADS>
__device__ __forceinline__ void group_sync(int grp) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(THREADS) : "memory");
}

// A work item as one word: down (bit 31), chunk (bits 22..30), tile (bits 0..21).
constexpr uint32_t kMoeNoItem = 0xffffffffu;
__device__ __forceinline__ int item_chunk(uint32_t it) { return static_cast<int>((it >> 22) & 511u); }
__device__ __forceinline__ int item_tile(uint32_t it) { return static_cast<int>(it & 0x3fffffu); }
__device__ __forceinline__ bool item_down(uint32_t it) { return (it >> 31) != 0; }
static_assert(kMoeMaxChunks < 511, "chunk field, with the empty item apart");

__device__ __forceinline__ int load_acquire_gpu(const int *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// GW: warps of a group. PAIRS: 8-bit scales of 64-element blocks, an even number
// to a row, so that the two scales of a step are one aligned 16-bit load (the
// usual weight; the other scale forms take single loads).
template <int GW, bool PAIRS>
__global__ void __launch_bounds__(kMoeThreads, 1)
nf4_moe_experts_kernel(const __grid_constant__ CUtensorMap tm_gate_up,   // u8 [2 E, F, H/2], box {64, 32, 2}, 64-byte swizzle
                       const __grid_constant__ CUtensorMap tm_down,      // u8 [E H, F/2], box {64, 64}, 64-byte swizzle
                       const MoeArgs a) {
    constexpr int kGroups = kMoeWarps / GW;
    static_assert(kGroups * GW == kMoeWarps, "a group's barrier counts its warps");
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
        tma_prefetch_desc(&tm_gate_up);
        tma_prefetch_desc(&tm_down);
    }
    for (int idx = threadIdx.x; idx < 256 * 32; idx += kMoeThreads) {
        const int b = idx >> 5, l = idx & 31;
        *reinterpret_cast<uint32_t *>(lut_g + b * 256 + 4 * l) =
            bf16_pack(kMoeLevelUp * c_levels[b >> 4], kMoeLevelUp * c_levels[b & 15]);
    }
    griddep_wait();
    griddep_launch_dependents();

    uint32_t slot[kMoeRing];
#pragma unroll
    for (int s = 0; s < kMoeRing; ++s) {
        const uint32_t i = static_cast<uint32_t>(warp * kMoeRing + s);
        slot[s] = i < nlow ? low0 + i * kMoeSlotBytes : kDsHighAddr + (i - nlow) * kMoeSlotBytes;
    }

    // ---- items are taken by the group's first thread, two ahead of the one
    // being computed: the last step of an item already requests the next one's
    // data, and the atomic of the one after it is in flight meanwhile. The first
    // two are taken by the last warp, which has the fewest tokens to route, one
    // after the other, so that few items spread over the grid.
    const bool taker = gw == 0 && lane == 0;
    int taken = 0;
    if (warp == kMoeWarps - 1 && lane < kGroups) {
        const int c0 = atomicAdd(&a.cnt->claimed, 1);
        hd->start[lane][0] = c0;
        hd->start[lane][1] = atomicAdd(&a.cnt->claimed, c0 < 0 ? 0 : 1);
    }
    moe_route(a, hd, reinterpret_cast<unsigned long long *>(dsm + (slot[0] - sbase)));
    __syncthreads();
    const int nchunks = hd->nchunks;
    const int tiles_gu = a.F / (kMoeRows / 2), tiles_dn = a.H / kMoeRows;
    const int items_gu = nchunks * tiles_gu;
    auto item_of = [&](int i) -> uint32_t {
        const bool dn = i >= items_gu;
        if (dn) i -= items_gu;
        const int per = dn ? tiles_dn : tiles_gu;
        const int c = i / per;
        if (c >= nchunks) return kMoeNoItem;
        return (dn ? 1u << 31 : 0u) | static_cast<uint32_t>(c) << 22 | static_cast<uint32_t>(i - c * per);
    };
    if (taker) {
        hd->claim[grp][0] = item_of(hd->start[grp][0]);
        hd->claim[grp][1] = item_of(hd->start[grp][1]);
        taken = atomicAdd(&a.cnt->claimed, 1);
    }
    group_sync<32 * GW>(grp);
    int seq = 0;                                               // the current item is claim[seq % 4]
    uint32_t cur = hd->claim[grp][0];

    int issued = 0, landed = 0;
    // request one step's codes (kc-th 128 elements of the item's 64 rows)
    auto issue = [&](uint32_t it, int kc) {
        if (abort_raised(abort_flag)) return;
        if (lane == 0) {
            const int s = issued % kMoeRing;
            uint64_t *bar = &hd->bars[warp][s];
            uint8_t *dst = dsm + (slot[s] - sbase);
            const int e = hd->chunk[item_chunk(it)].expert, tile = item_tile(it);
            fence_proxy_async_smem();      // the slot was read through the generic proxy
            mbar_arrive_expect_tx(bar, kMoeSlotBytes);
            if (item_down(it)) tma_load_2d(dst, &tm_down, bar, kc * kMoeStepBytes, e * a.H + tile * kMoeRows);
            else tma_load_3d(dst, &tm_gate_up, bar, kc * kMoeStepBytes, tile * (kMoeRows / 2), 2 * e);
        }
        ++issued;
    };
    // the first step of this warp in an item whose rows have nkc steps; a warp
    // beyond the last one takes it too and leaves its products out of the sums
    auto first_step = [&](bool dn) { return min(gw, ((dn ? a.F : a.H) / kBlock + 1) / 2 - 1); };

    // Which row of a 16-row tile lane group g reads: with 64-byte rows under
    // the 64-byte swizzle, rows {0,1,4,5} (and {2,3,6,7}) of one block take
    // all 32 banks once.
    const int prow = (g & 1) | ((g & 2) << 1) | ((g & 4) >> 1);
    const uint32_t lanew = (static_cast<uint32_t>(lane) << 2) | (1u << 16);
    const uint32_t swz = static_cast<uint32_t>((prow >> 1) & 3);
    const uint32_t code_row = static_cast<uint32_t>(prow) * kMoeStepBytes + 8u * (t & 1);
    const uint32_t code_chunk[2] = {((0u + (t >> 1)) ^ swz) << 4, ((2u + (t >> 1)) ^ swz) << 4};
    // sum j (= 4 tile + element) of warp w of this group, this thread's lane
    auto park = [&](int w, int j) {
        return reinterpret_cast<float *>(lut_g + ((grp * GW + w) * 16 + j) * 256 + 128 + 4 * lane);
    };

    if (cur != kMoeNoItem) issue(cur, first_step(item_down(cur)));

    // ---- the items of one kind, to the group's last of them
    auto run = [&](auto down_c) {
        constexpr bool DOWN = decltype(down_c)::value;
        const MoeScales &sw = DOWN ? a.down : a.gate_up;
        const int K = DOWN ? a.F : a.H;
        const int kblocks = K / kBlock;
        const int nkc = (kblocks + 1) / 2;                     // steps of an item
        const int bpr = kblocks >> sw.bshift;                  // scale blocks of a weight row
        const int kc0 = first_step(DOWN);
        const bool real = gw < nkc;

        // down: the group waits until the activations of a chunk are complete
        // (one thread looks, with pauses: a thousand warps reading the same
        // counters would hold up the atomics that they wait for). True once all
        // chunks are known to be.
        auto wait_chunk = [&](int chunk) -> bool {
            if (taker) {
                const long long t0 = clock64();
                const long long lim = g_dbg_flag_wait_limit > 0 ? g_dbg_flag_wait_limit : kWaitLimitCycles;
                int st = 0;
                while (true) {
                    if (load_acquire_gpu(&a.cnt->gate_up_done) == items_gu) {
                        st = 1;
                        break;
                    }
                    if (load_acquire_gpu(&a.cnt->chunk_done[chunk]) == tiles_gu || abort_raised(abort_flag)) break;
                    if (clock64() - t0 > lim) {
                        record_status(NF4_ERR_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    __nanosleep(100);
                }
                hd->ready[grp] = st;
            }
            group_sync<32 * GW>(grp);        // the thread's acquire holds for the group's loads below
            return hd->ready[grp] != 0;
        };

        // operands of the next step: the raw scales of this lane's two rows
        // (rows prow and prow + 8 of tile t) and the activations of its token g.
        // Lanes beyond the chunk's tokens read its last token again: their
        // columns of the products are never stored.
        int nkc_at = kc0;
        const uint16_t *nx = nullptr;                          // x (or a) at token g, element 16 t
        uint32_t nsb = 0;                                      // scale index of the first row; the second is 8 bpr on
        auto operands_of = [&](uint32_t it) {
            const MoeChunk c = hd->chunk[item_chunk(it)];
            const int sl = c.slot0 + min(g, c.n - 1);
            nx = (DOWN ? a.a + static_cast<int64_t>(sl) * K : a.x + static_cast<int64_t>(hd->token[sl]) * K) + 16 * t;
            const int row = DOWN ? c.expert * a.H + item_tile(it) * kMoeRows + 16 * t
                                 : (c.expert * 2 + (t >> 1)) * a.F + item_tile(it) * (kMoeRows / 2) + 16 * (t & 1);
            nsb = static_cast<uint32_t>(row + prow) * static_cast<uint32_t>(bpr);
            nkc_at = kc0;
        };
        uint32_t raw[2][PAIRS ? 1 : 2];                        // [row][block]: q8 codes, or the absmax bits
        float grp_c[2][PAIRS ? 1 : 2];                         // their group constants
        auto load_scales = [&]() {
            const int b0 = 2 * nkc_at;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t at = nsb + static_cast<uint32_t>(8 * i * bpr + (b0 >> sw.bshift));
                if constexpr (PAIRS) {
                    raw[i][0] = __ldg(reinterpret_cast<const uint16_t *>(sw.q8 + at));
                    grp_c[i][0] = __ldg(sw.cg + (at >> 8));
                } else {
                    // the second block of a step: its own scale, the same one (128-element
                    // blocks), or, behind the row's last block, not used
                    const uint32_t at1 = sw.bshift || b0 + 1 >= kblocks ? at : at + 1;
                    if (sw.dq) {
                        raw[i][0] = __ldg(sw.q8 + at);
                        raw[i][1] = __ldg(sw.q8 + at1);
                        grp_c[i][0] = __ldg(sw.cg + (at >> 8));
                        grp_c[i][1] = __ldg(sw.cg + (at1 >> 8));
                    } else {
                        raw[i][0] = __float_as_uint(__ldg(sw.absmax + at));
                        raw[i][1] = __float_as_uint(__ldg(sw.absmax + at1));
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
                return sw.dq ? static_cast<float>(raw[i][b]) * (grp_c[i][b] * (kMoeLevelDown / 127.0f))
                             : __uint_as_float(raw[i][b]) * kMoeLevelDown;
            }
        };
        uint4 xv[2][2];                                        // [block][half]
        auto load_x = [&](int b) {
            const int blk = min(2 * nkc_at + b, kblocks - 1);
            const uint4 *q = reinterpret_cast<const uint4 *>(nx + blk * kBlock);
            xv[b][0] = q[0];
            xv[b][1] = q[1];
        };

        // down: the item before's place in the count of its stripe, looked at
        // one item later, when the atomic has long returned
        int seen = -1, seen_tile = 0;
        auto combine = [&](int tile) {
            // every slot's share of these 64 columns is there: each token's
            // top_k of them are added in order
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
        // the thread that counts the group's finished items (not the one that
        // takes them, whose atomics are on the way to the next)
        const bool counter = gw == GW - 1 && lane == 0;

        if (cur == kMoeNoItem || item_down(cur) != DOWN) return;
        bool all_done = !DOWN, fetched = false;

        while (cur != kMoeNoItem && item_down(cur) == DOWN) {
            const uint32_t nxt = hd->claim[grp][(seq + 1) & 3];
            if (!fetched) {
                operands_of(cur);
                load_scales();
                if (DOWN && !all_done) all_done = wait_chunk(item_chunk(cur));
                load_x(0);
                load_x(1);
            }
            fetched = all_done && nxt != kMoeNoItem && item_down(nxt) == DOWN;
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
            for (int kc = kc0; kc < nkc; kc += GW) {
                float sc[2][2];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) sc[i][b] = scale_of(i, b);
                // the next step: of this item, or the first of the next one (its
                // activations only when they are known to be complete)
                if (kc + GW < nkc) {
                    nkc_at += GW;
                    issue(cur, kc + GW);
                } else if (nxt != kMoeNoItem) {
                    issue(nxt, first_step(item_down(nxt)));
                    if (fetched) operands_of(nxt);
                }
                load_scales();
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

            // ---- the group's k splits meet in the odd halves of the table
            // rows, and are added in warp order
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) *park(gw, i * 4 + e) = real ? acc[i][e] : 0.0f;
            if (taker) {
                hd->claim[grp][(seq + 2) & 3] = item_of(taken);
                taken = atomicAdd(&a.cnt->claimed, 1);
            }
            if (DOWN && counter) hd->last[grp] = seen == nchunks - 1;
            group_sync<32 * GW>(grp);
            if (DOWN && hd->last[grp]) combine(seen_tile);
            const MoeChunk c = hd->chunk[item_chunk(cur)];
            const int tile = item_tile(cur);
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
                        // s0 is gate row rr, s1 up row rr; rounded to the down product's operand
                        const __nv_bfloat16 v = __float2bfloat16_rn(act_value(s0, a.act) * s1);
                        a.a[static_cast<int64_t>(c.slot0 + col) * a.F + tile * (kMoeRows / 2) + rr] =
                            *reinterpret_cast<const uint16_t *>(&v);
                    } else {
                        const float w = hd->weight[c.slot0 + col];
                        float *y = a.y + static_cast<int64_t>(c.slot0 + col) * a.H + tile * kMoeRows + rr;
                        __stcg(y, w * s0);
                        __stcg(y + 32, w * s1);
                    }
                }
            }
            group_sync<32 * GW>(grp);        // the partials are free again, the results written
            seen_tile = tile;
            if (counter) {
                __threadfence();             // the group's results before the counts
                if constexpr (DOWN) {
                    seen = atomicAdd(a.cnt->stripe_done + tile, 1);
                    __threadfence();         // the others' results after it
                } else if (!g_dbg_skip_flag_set) {
                    atomicAdd(&a.cnt->chunk_done[item_chunk(cur)], 1);
                    atomicAdd(&a.cnt->gate_up_done, 1);
                }
            }
            ++seq;
            cur = nxt;
        }
        if (DOWN) {
            if (counter) hd->last[grp] = seen == nchunks - 1;
            group_sync<32 * GW>(grp);
            if (hd->last[grp]) combine(seen_tile);
        }
    };
    run(std::integral_constant<bool, false>{});
    run(std::integral_constant<bool, true>{});
    // leave no copy in flight into shared memory that is about to be released
    // (after a normal end every copy has landed)
    if (lane == 0)
        for (int s = landed; s < issued; ++s)
            mbar_drain(&hd->bars[warp][s % kMoeRing], static_cast<uint32_t>(s / kMoeRing) & 1u);
    __syncwarp();
}

}  // namespace nf4
