// Group norm with an activation, channels last: each token's C channels are
// normalised in G groups of D = C / G,
//
//     n = (x - mean) / sqrt(var + eps),  h = n weight + bias,
//     y = h act(gate),  or act(h) without a gate,
//
// and its gradient.  What follows a recurrence over heads: a group is a head,
// statistics stay within the token.
//
// Both directions are bound by memory: x (and gate) in and y out; x, gate and
// gy in and gx, ggate out.  A group is held in the registers of P threads (P a
// power of two up to a warp, or the whole block), VW elements per access and
// NI accesses each, so it is read once, the mean is exact before the squared
// differences are summed, and the gradient recomputes the statistics from the
// x it has to read anyway instead of loading stored ones.  A thread keeps its
// channels and walks over tokens: weight and bias are read once per block,
// and the gradient's sums over tokens stay in registers, one partial per
// block, added in a fixed order by a second kernel.  32768 tokens of 40 groups of
// 64 with a gate, bf16: 102 us (75 % of the copy rate), gradient 185 us (69 %).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace wkvb {

enum NormAct { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

template <typename IO>
struct NormArgs {
    const IO *x, *gate;          // [N, C]; gate may be NULL
    const float *weight, *bias;  // [C] or NULL (1, 0)
    IO *y;                       // forward
    const IO *gy;                // gradient
    IO *gx, *ggate;
    float *partial;              // [gridDim.x][2][C]: sums of gh n and gh
    long long N;
    int C, G, D, act;
    int gpb;     // groups per block
    int blocks;  // blocks along the tokens (gradient)
    float eps;
};

// VW elements as they lie in memory: what a thread holds of the tokens ahead
template <typename IO, int VW>
struct NormVec;

template <typename IO>
struct NormVec<IO, 1> {
    IO v;
    __device__ void load(const IO *p) { v = *p; }
    __device__ void zero() { v = static_cast<IO>(0.f); }
    __device__ void get(float *x) const { x[0] = static_cast<float>(v); }
    __device__ static void store(IO *p, const float *x) { *p = static_cast<IO>(x[0]); }
};
template <>
struct NormVec<float, 4> {
    float4 v;
    __device__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
    __device__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ void get(float *x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
    __device__ static void store(float *p, const float *x) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <>
struct NormVec<__nv_bfloat16, 8> {
    uint4 v;
    __device__ void load(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ void get(float *x) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static void store(__nv_bfloat16 *p, const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// e^-z and p = 1 / (1 + e^-z).  With bf16 I/O by the hardware's exponential
// and reciprocal: two instructions instead of about thirty, without which the
// arithmetic and not the memory is the bound.  e is off by some 2^-22 plus
// |z| 2^-24 of itself (the rounding of the exponential's argument): 2^-22 around
// 0, 2^-17 at |z| = 80.  Of p that is less: next to 1, e is small, and next to 0 p
// and what it multiplies are.  The outputs keep 2^-9, and gweight and gbias, fp32
// sums of such terms, weigh each by the activation it belongs to.  For fp32 by
// expf and the fast division (2 units in the last place; from z = -87.3 down
// p is 0 instead of 2^-126 and less).
template <typename IO>
__device__ __forceinline__ float norm_sigmoid(float z, float &e) {
    if constexpr (sizeof(IO) == 2) {
        e = ex2_approx(-1.4426950408889634f * z);
        return rcp_approx(1.f + e);
    } else {
        e = expf(-z);
        return __fdividef(1.f, 1.f + e);
    }
}

// f = act(z)
template <typename IO, int VW>
__device__ __forceinline__ void norm_act(const float (&z)[VW], int act, float (&f)[VW]) {
    float e;
    if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = z[i] * norm_sigmoid<IO>(z[i], e);
    } else if (act == kActSigmoid) {
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = norm_sigmoid<IO>(z[i], e);
    } else {
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = z[i];
    }
}
// and df = act'(z)
template <typename IO, int VW>
__device__ __forceinline__ void norm_act_grad(const float (&z)[VW], int act, float (&f)[VW],
                                              float (&df)[VW]) {
    if (act == kActNone) {
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = z[i], df[i] = 1.f;
        return;
    }
#pragma unroll
    for (int i = 0; i < VW; ++i) {
        float e;
        const float p = norm_sigmoid<IO>(z[i], e);
        const float m = z[i] < -80.f ? 1.f : e * p;  // 1 - p, not by a difference; e may be infinite
        f[i] = act == kActSilu ? z[i] * p : p;
        df[i] = act == kActSilu ? fmaf(f[i], m, p) : p * m;
    }
}

// Sum over the P threads of a group, the same in every one of them.  `red`:
// one float per warp, for P beyond a warp (the block then holds one group).
template <int P>
__device__ __forceinline__ float norm_sum(float v, float *red) {
    constexpr int kLanes = P < 32 ? P : 32;
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    if constexpr (P > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < P / 32; ++w) v += red[w];
    }
    return v;
}

// This thread's place: P lanes per group, a.gpb groups per token and block,
// tokens row, row + stride, ...  Threads beyond the last full token, and
// groups beyond G in the last block column, only take part in the shuffles.
template <int P, int VW>
struct NormPlace {
    int lane, c0, rows;  // lane in the group, its first channel, tokens per block step
    int row;             // token slot in the block
    bool on;
    template <typename A>
    __device__ explicit NormPlace(const A &a) {
        lane = static_cast<int>(threadIdx.x) % P;
        const int slot = static_cast<int>(threadIdx.x) / P;
        rows = max(1, static_cast<int>(blockDim.x) / (P * a.gpb));
        row = slot / a.gpb;
        const int grp = static_cast<int>(blockIdx.y) * a.gpb + slot % a.gpb;
        on = row < rows && grp < a.G;
        c0 = grp * a.D;
    }
};

// Reads one token's VW * NI elements of this thread.
template <typename IO, int VW, int P, int NI>
__device__ __forceinline__ void norm_read(NormVec<IO, VW> (&v)[NI], const IO *p, bool on, int lane, int D) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int d = (lane + i * P) * VW;
        if (on && d < D) v[i].load(p + d);
        else v[i].zero();
    }
}

// The group's mean and 1 / sqrt(var + eps); x becomes its difference to the mean
template <int VW, int P, int NI>
__device__ __forceinline__ float norm_center(float (&x)[NI][VW], int lane, int D, float inv_d, float eps,
                                             float *red) {
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) sum += x[i][e];
    const float mean = norm_sum<P>(sum, red) * inv_d;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const bool in = (lane + i * P) * VW < D;
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            x[i][e] = in ? x[i][e] - mean : 0.f;
            sq = fmaf(x[i][e], x[i][e], sq);
        }
    }
    return 1.f / sqrtf(norm_sum<P>(sq, red) * inv_d + eps);
}

// Tokens that a thread reads ahead of those it works on: as many registers as
// they cost, they are what keeps the memory busy (latency times bandwidth is
// about 45 KB an SM).
template <int VW, int NI>
constexpr int kNormAhead = VW * NI <= 8 ? 2 : 1;

template <typename IO, int VW, int P, int NI>
__global__ void __launch_bounds__(256, VW * NI > 8 ? 2 : 3) group_norm_kernel(const NormArgs<IO> a) {
    __shared__ float red[32];
    const NormPlace<P, VW> at(a);
    float wt[NI][VW], bs[NI][VW];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            const int d = (at.lane + i * P) * VW + e;
            const bool in = at.on && d < a.D;
            wt[i][e] = in && a.weight ? a.weight[at.c0 + d] : 1.f;
            bs[i][e] = in && a.bias ? a.bias[at.c0 + d] : 0.f;
        }
    const float inv_d = 1.f / static_cast<float>(a.D);
    constexpr int U = kNormAhead<VW, NI>;
    const long long stride = static_cast<long long>(gridDim.x) * at.rows, step = U * stride;
    const bool gated = a.gate != nullptr;
    NormVec<IO, VW> xv[U][NI], gv[U][NI];
    const auto read = [&](int u, long long row) {
        const bool on = at.on && row < a.N;
        const size_t off = static_cast<size_t>(on ? row : 0) * a.C + at.c0;
        norm_read<IO, VW, P, NI>(xv[u], a.x + off, on, at.lane, a.D);
        if (gated) norm_read<IO, VW, P, NI>(gv[u], a.gate + off, on, at.lane, a.D);
    };
    long long base = static_cast<long long>(blockIdx.x) * at.rows;
#pragma unroll
    for (int u = 0; u < U; ++u) read(u, base + at.row + u * stride);
    for (; base < a.N; base += step) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0 && base + u * stride >= a.N) break;
            const long long row = base + at.row + u * stride;
            const bool on = at.on && row < a.N;
            const size_t off = static_cast<size_t>(on ? row : 0) * a.C + at.c0;
            float x[NI][VW], gt[NI][VW];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                xv[u][i].get(x[i]);
                if (gated) gv[u][i].get(gt[i]);
            }
            read(u, row + step);
            const float rstd = norm_center<VW, P, NI>(x, at.lane, a.D, inv_d, a.eps, red);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int d = (at.lane + i * P) * VW;
                if (!(on && d < a.D)) continue;
                float f[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) x[i][e] = fmaf(x[i][e] * rstd, wt[i][e], bs[i][e]);
                if (gated) {
                    norm_act<IO, VW>(gt[i], a.act, f);
#pragma unroll
                    for (int e = 0; e < VW; ++e) x[i][e] *= f[e];
                } else {
                    norm_act<IO, VW>(x[i], a.act, f);
#pragma unroll
                    for (int e = 0; e < VW; ++e) x[i][e] = f[e];
                }
                NormVec<IO, VW>::store(a.y + off + d, x[i]);
            }
        }
    }
}

// gx = rstd (gn - mean(gn) - n mean(gn n)), gn = gh weight, with gh = gy
// act(gate) and ggate = gy h act'(gate), or gh = gy act'(h).
template <typename IO, int VW, int P, int NI>
__global__ void __launch_bounds__(256, VW * NI > 8 ? 1 : 2) group_norm_grad_kernel(const NormArgs<IO> a) {
    __shared__ float red[32];
    extern __shared__ float sums[];  // [2][rows][gpb * D]
    const NormPlace<P, VW> at(a);
    float wt[NI][VW], bs[NI][VW], gw[NI][VW] = {}, gb[NI][VW] = {};
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            const int d = (at.lane + i * P) * VW + e;
            const bool in = at.on && d < a.D;
            wt[i][e] = in && a.weight ? a.weight[at.c0 + d] : 1.f;
            bs[i][e] = in && a.bias ? a.bias[at.c0 + d] : 0.f;
        }
    const float inv_d = 1.f / static_cast<float>(a.D);
    constexpr int U = kNormAhead<VW, NI>;
    const long long stride = static_cast<long long>(gridDim.x) * at.rows, step = U * stride;
    const bool gated = a.gate != nullptr;
    NormVec<IO, VW> xv[U][NI], gv[U][NI], yv[U][NI];
    const auto read = [&](int u, long long row) {
        const bool on = at.on && row < a.N;
        const size_t off = static_cast<size_t>(on ? row : 0) * a.C + at.c0;
        norm_read<IO, VW, P, NI>(xv[u], a.x + off, on, at.lane, a.D);
        norm_read<IO, VW, P, NI>(yv[u], a.gy + off, on, at.lane, a.D);
        if (gated) norm_read<IO, VW, P, NI>(gv[u], a.gate + off, on, at.lane, a.D);
    };
    long long base = static_cast<long long>(blockIdx.x) * at.rows;
#pragma unroll
    for (int u = 0; u < U; ++u) read(u, base + at.row + u * stride);
    for (; base < a.N; base += step) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0 && base + u * stride >= a.N) break;
            const long long row = base + at.row + u * stride;
            const bool on = at.on && row < a.N;
            const size_t off = static_cast<size_t>(on ? row : 0) * a.C + at.c0;
            float x[NI][VW], gt[NI][VW], gy[NI][VW];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                xv[u][i].get(x[i]);
                yv[u][i].get(gy[i]);
                if (gated) gv[u][i].get(gt[i]);
            }
            read(u, row + step);
            const float spread = norm_center<VW, P, NI>(x, at.lane, a.D, inv_d, a.eps, red);
            // no token, no spread: with eps = 0 it would be infinite, and its
            // product with x = 0 would be NaN in the sums over tokens
            const float rstd = on ? spread : 0.f;
            float m1 = 0.f, m2 = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float f[VW], df[VW], h[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    x[i][e] *= rstd;
                    h[e] = fmaf(x[i][e], wt[i][e], bs[i][e]);
                }
                // threads without a token have x = gy = 0: they add nothing
                if (gated) {
                    norm_act_grad<IO, VW>(gt[i], a.act, f, df);
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        gt[i][e] = gy[i][e] * h[e] * df[e];
                        gy[i][e] *= f[e];
                    }
                } else {
                    norm_act_grad<IO, VW>(h, a.act, f, df);
#pragma unroll
                    for (int e = 0; e < VW; ++e) gy[i][e] *= df[e];
                }
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    gw[i][e] = fmaf(gy[i][e], x[i][e], gw[i][e]);
                    gb[i][e] += gy[i][e];
                    gy[i][e] *= wt[i][e];
                    m1 += gy[i][e];
                    m2 = fmaf(gy[i][e], x[i][e], m2);
                }
            }
            m1 = norm_sum<P>(m1, red) * inv_d;
            m2 = norm_sum<P>(m2, red) * inv_d;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int d = (at.lane + i * P) * VW;
                if (!(on && d < a.D)) continue;
#pragma unroll
                for (int e = 0; e < VW; ++e) x[i][e] = rstd * (gy[i][e] - m1 - x[i][e] * m2);
                NormVec<IO, VW>::store(a.gx + off + d, x[i]);
                if (gated) NormVec<IO, VW>::store(a.ggate + off + d, gt[i]);
            }
        }
    }
    if (a.partial == nullptr) return;
    // the block's sums: token slots added in order
    const int span = a.gpb * a.D, first = static_cast<int>(blockIdx.y) * span;
    if (at.on) {
        float *s = sums + static_cast<size_t>(at.row) * span + (at.c0 - first);
        float *t = s + static_cast<size_t>(at.rows) * span;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int d = (at.lane + i * P) * VW + e;
                if (d < a.D) s[d] = gw[i][e], t[d] = gb[i][e];
            }
    }
    __syncthreads();
    float *out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.C;
    for (int d = threadIdx.x; d < span && first + d < a.C; d += blockDim.x) {
        float w = 0.f, v = 0.f;
        for (int r = 0; r < at.rows; ++r) {
            w += sums[r * span + d];
            v += sums[(at.rows + r) * span + d];
        }
        out[first + d] = w;
        out[a.C + first + d] = v;
    }
}

// gweight, gbias: the blocks' sums added in a fixed order.  One block per 32
// columns of the [n][2 C] partials, 16 warps each adding every sixteenth one.
constexpr int kNormSumWarps = 16;
__global__ void __launch_bounds__(32 * kNormSumWarps)
    group_norm_sum_kernel(const float *partial, int n, int C, float *gweight, float *gbias) {
    __shared__ float part[kNormSumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * C)
#pragma unroll 8
        for (int i = warp; i < n; i += kNormSumWarps) s += partial[static_cast<size_t>(i) * 2 * C + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * C) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < kNormSumWarps; ++w) s += part[w][lane];
        if (c < C) {
            if (gweight != nullptr) gweight[c] = s;
        } else if (gbias != nullptr) {
            gbias[c - C] = s;
        }
    }
}

}  // namespace wkvb
