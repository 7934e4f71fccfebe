// epilogue.cuh -- the element-wise end of the QLoRA layer and its gradient:
//
//   forward    z = (the layer's sum) + bias,  h = act(z) . mul + residual
//   backward   dz = dH . mul . act'(z),  dmul = dH . act(z),  dbias = sum_m dz
//
// z is kept in bf16 between the two (half the bytes of the fp32 sum, on a path bound by
// HBM): act and act' are off by up to 2^-8 |z| times |act'| and |act''|. Only a ReLU's
// derivative jumps, and the rounding of z does not change its sign.
//
// The forward part runs inside the kernels that produce the sum (the fused
// GEMM's and the decode kernel's output step), on the fp32 accumulator, before
// its one rounding to bf16. The backward part is the kernel below: its dz
// feeds the layer's backward products.
#pragma once

#include "nf4_common.cuh"

namespace nf4 {

struct EpiArgs {
    int act;                    // nf4_act
    const uint16_t *bias;       // [N] bf16 (optional)
    const uint16_t *mul;        // [M, N] bf16 (optional)
    const uint16_t *residual;   // [M, N] bf16 (optional)
    uint16_t *z;                // [M, N] bf16 pre-activation for the backward (optional)
};

// ---------------------------------------------------------------------------
// Activations in fp32. The logistic function comes from the hardware
// exponential and division: a few 2^-22 relative, and |z| 2^-23 more from the
// rounding of the exponential's argument (2^-16 at |z| = 100), far inside the
// bf16 rounding (2^-8) of every result; below z = -87.3, where it is under
// 2^-126, it is 0 (the division's range). Both GELU forms go through functions
// without a cancellation (1 + tanh, 1 + erf) for large negative z. NaN passes
// through every activation.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluTanhScale = 1.59576912160573f;    // 2 sqrt(2 / pi)
constexpr float kGeluTanhCubic = 0.044715f;

// Normal distribution function. With x = |z| / sqrt 2 and t = 1 / (1 + x / 2),
//   erfc(x) = t 2^(-x^2 log2(e) + Q(t)),
// the form of Press, Teukolsky, Vetterling and Flannery, Numerical Recipes, section
// 6.2 (erfcc); Q is a degree-7 Chebyshev fit of log2(erfc(x) e^(x^2) / t) over
// 0.08 <= t <= 1, made here. Relative error, with every operation rounded once: 1e-6 for
// z > -3; below, the rounding of the exponent (which grows as z^2) adds to it, 2e-6 down to
// -6, 3.3e-6 to -9, 8.5e-6 to -13 (beyond |z| = 32 both are 0 in fp32). One reciprocal,
// one exponential and eight multiply-adds.
__device__ __forceinline__ float normal_cdf(float z) {
    const float t = __fdividef(1.0f, fmaf(0.35355339059327376f, fabsf(z), 1.0f));
    float q = -0.27331653237342834f;
    q = fmaf(q, t, 1.0946335792541504f);
    q = fmaf(q, t, -1.4626392126083374f);
    q = fmaf(q, t, 0.5222470164299011f);
    q = fmaf(q, t, -0.06672894954681396f);
    q = fmaf(q, t, 0.5712890028953552f);
    q = fmaf(q, t, 1.4401801824569702f);
    q = fmaf(q, t, -1.8256661891937256f - 1.0f);        // the - 1 halves erfc
    const float tail = t * exp2f(fmaf(-0.72134752044448170f * z, z, q));
    return z < 0.0f ? tail : 1.0f - tail;
}

__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case NF4_ACT_RELU: return z < 0.0f ? 0.0f : z;
        case NF4_ACT_SILU: return z * logistic(z);
        // (1 + tanh(v / 2)) / 2 = logistic(v)
        case NF4_ACT_GELU_TANH:
            return z * logistic(kGeluTanhScale * fmaf(kGeluTanhCubic * z * z, z, z));
        case NF4_ACT_GELU: return z * normal_cdf(z);
        default: return z;
    }
}

__device__ __forceinline__ void act8(float (&f)[8], int act) {
    switch (act) {
#define NF4_ACT8(A_)                                      \
    case A_:                                              \
        _Pragma("unroll") for (int i = 0; i < 8; ++i) f[i] = act_value(f[i], A_); \
        break;
        NF4_ACT8(NF4_ACT_RELU)
        NF4_ACT8(NF4_ACT_SILU)
        NF4_ACT8(NF4_ACT_GELU_TANH)
        NF4_ACT8(NF4_ACT_GELU)
#undef NF4_ACT8
        default: break;
    }
}

// act(z) and act'(z)
__device__ __forceinline__ void act_pair(float z, int act, float &a, float &da) {
    switch (act) {
        case NF4_ACT_RELU:
            a = z < 0.0f ? 0.0f : z;
            da = z > 0.0f ? 1.0f : 0.0f;
            return;
        case NF4_ACT_SILU: {
            const float p = logistic(z);
            a = z * p;
            da = fmaf(a, 1.0f - p, p);
            return;
        }
        case NF4_ACT_GELU_TANH: {
            const float p = logistic(kGeluTanhScale * fmaf(kGeluTanhCubic * z * z, z, z));
            a = z * p;
            // p (1 - p) is zero in fp32 long before |z| = 100; the bound keeps z^2 finite
            const float zz = fminf(z * z, 1.0e4f);
            da = fmaf(a * (1.0f - p), kGeluTanhScale * fmaf(3.0f * kGeluTanhCubic, zz, 1.0f), p);
            return;
        }
        case NF4_ACT_GELU: {
            const float cdf = normal_cdf(z);
            a = z * cdf;
            da = fmaf(z, 0.39894228040143268f * __expf(-0.5f * z * z), cdf);
            return;
        }
        default:
            a = z;
            da = 1.0f;
    }
}

__device__ __forceinline__ void act_pair8(const float (&z)[8], int act, float (&a)[8], float (&da)[8]) {
    switch (act) {
#define NF4_ACT_PAIR8(A_)                                 \
    case A_:                                              \
        _Pragma("unroll") for (int i = 0; i < 8; ++i) act_pair(z[i], A_, a[i], da[i]); \
        break;
        NF4_ACT_PAIR8(NF4_ACT_RELU)
        NF4_ACT_PAIR8(NF4_ACT_SILU)
        NF4_ACT_PAIR8(NF4_ACT_GELU_TANH)
        NF4_ACT_PAIR8(NF4_ACT_GELU)
        default:
            NF4_ACT_PAIR8(NF4_ACT_NONE)
#undef NF4_ACT_PAIR8
    }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_at(const uint16_t *p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}
__device__ __forceinline__ uint32_t bf16_pack(float lo, float hi) {
    __nv_bfloat162 h2 = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h2);
}
__device__ __forceinline__ uint4 bf16_pack8(const float (&f)[8]) {
    return make_uint4(bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7]));
}
__device__ __forceinline__ void bf16_unpack8(const uint4 &v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

// ---------------------------------------------------------------------------
// dz = dH . mul . act'(z) (bf16, the operand of the backward's products),
// dmul = dH . act(z), dbias = sum over tokens of dz (summed in fp32 before the
// rounding of dz).
//
// Bound by HBM: reads dH, z (and mul), writes dz (and dmul), once. A CTA takes
// 128 columns (16 lanes of 8) and every (32 x splits)-th row from its own; the
// splits of one column stripe are a cluster, so the column sums meet in
// distributed shared memory and are added in a fixed order: one launch, no
// atomics, no workspace. A thread has two rows in flight. 225 us at 28672
// columns and 4096 tokens with mul and dmul (5.2 TB/s); 30 us at 5120 columns and
// 2048 tokens, where the grid is just over one wave. dz is null when there is neither activation nor mul
// (then dz is dH itself and only the column sums are formed).
// ---------------------------------------------------------------------------
constexpr int kEbThreads = 512;
constexpr int kEbCols = 128;
constexpr int kEbRows = kEbThreads / (kEbCols / 8);     // rows of one pass of a CTA
constexpr int kEbMaxSplits = 8;

struct EpiBwdArgs {
    int64_t M, N;
    int act;
    const uint16_t *dH, *z, *mul;   // z, mul optional
    uint16_t *dz, *dmul;            // optional
    void *dbias;                    // optional, bf16 or fp32
    int dbias_f32;
};

__global__ void __launch_bounds__(kEbThreads, 2)
qlora_epilogue_bwd_kernel(const EpiBwdArgs a) {
    __shared__ float part[kEbRows][kEbCols + 4];
    griddep_wait();
    griddep_launch_dependents();
    const int c8 = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int64_t col = static_cast<int64_t>(blockIdx.y) * kEbCols + c8 * 8;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kEbRows;
    float sum[8] = {};
    if (col < a.N) {
        // two rows in flight per thread
        for (int64_t m = static_cast<int64_t>(blockIdx.x) * kEbRows + r; m < a.M; m += 2 * step) {
            uint4 gv[2], zv[2], mv[2];
            bool ok[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t mi = m + i * step;
                ok[i] = mi < a.M;
                const int64_t o = (ok[i] ? mi : m) * a.N + col;
                gv[i] = *reinterpret_cast<const uint4 *>(a.dH + o);
                if (a.z) zv[i] = *reinterpret_cast<const uint4 *>(a.z + o);
                if (a.mul) mv[i] = *reinterpret_cast<const uint4 *>(a.mul + o);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok[i]) break;
                const int64_t o = (m + i * step) * a.N + col;
                float g[8];
                bf16_unpack8(gv[i], g);
                if (a.dz || a.dmul) {
                    float z[8] = {}, f[8], dm[8];
                    if (a.z) bf16_unpack8(zv[i], z);
                    act_pair8(z, a.act, dm, f);               // act, act'
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dm[e] *= g[e];
                        g[e] *= f[e];
                    }
                    if (a.mul) {
                        bf16_unpack8(mv[i], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[e] *= f[e];
                    }
                    if (a.dmul) *reinterpret_cast<uint4 *>(a.dmul + o) = bf16_pack8(dm);
                    if (a.dz) *reinterpret_cast<uint4 *>(a.dz + o) = bf16_pack8(g);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += g[e];
            }
        }
    }
    if (!a.dbias) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) part[r][c8 * 8 + e] = sum[e];
    __syncthreads();
    // the CTA's 32 row sums of each column, in row order
    float v = 0.0f;
    if (threadIdx.x < kEbCols) {
#pragma unroll
        for (int i = 0; i < kEbRows; ++i) v += part[i][threadIdx.x];
        part[0][threadIdx.x] = v;
    }
    // the grid's x dimension is one cluster: its CTAs' sums, in rank order
    cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x < kEbCols) {
        const int64_t n = static_cast<int64_t>(blockIdx.y) * kEbCols + threadIdx.x;
        const uint32_t own = smem_u32(&part[0][threadIdx.x]);
        for (uint32_t rk = 1; rk < gridDim.x; ++rk) {
            float w;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(mapa_shared(own, rk)) : "memory");
            v += w;
        }
        if (n < a.N) {
            if (a.dbias_f32) {
                static_cast<float *>(a.dbias)[n] = v;
            } else {
                const __nv_bfloat16 b = __float2bfloat16_rn(v);
                static_cast<uint16_t *>(a.dbias)[n] = *reinterpret_cast<const uint16_t *>(&b);
            }
        }
    }
    cluster_sync();       // no CTA leaves while its sums may still be read
}

}  // namespace nf4
