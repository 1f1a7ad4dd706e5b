// Gated delta rule, step by step: the kernel of single-token decoding, of
// short sequences, of fp32 and of sizes the chunked kernel does not take; and
// the two state sweeps of the gradient.
//
// A warp owns 4 CPL columns of one head's state, held in registers: lane
// 4 g + c holds columns CPL c .. and, of every 32 rows, the four rows
// 4g .. 4g+3, so a row of k in shared memory is read with one 16-byte access
// per four rows, free of bank conflicts.  Per step and state element: one
// multiply-add each for S^T k, S^T q and the update.  The decay costs next to
// none: registers hold S / c_t with one scalar per step, the product of the
// stage's decays so far, folded back into the registers once a stage (or at
// every step of a stage in which some c_t leaves [2^-24, 2^24]: an a_t of 0
// does and clears the state).  S^T q is taken before the update,
// o = S'^T q + (q.k) beta r: it is off the step's dependent chain.  With
// CPL = 4 both sums are reduced together over the eight lanes of a column:
// halves are exchanged (4 + 2 + 1 shuffles for eight sums, against 24 for full
// butterflies), and four shuffles hand the new residuals back.  CPL = 1, where
// there are so few heads that most of the SMs' sub-partitions would have no
// warp: a quarter of the multiply-adds per step, and plain butterflies.
//
// The steps' q, k and v come kRecSteps at a time, asynchronously, a stage
// ahead of their use: the loop never waits for memory.
//
// Bounds: a decoding step moves the state in and out and nothing else of
// weight (8 DK DV bytes a head); long sequences are bound by the latency of a
// step's sums and exchanges, and with many heads by the three multiply-adds
// per element, 3 DK DV / 128 cycles of an SM per step and head.  256 rows' next
// tokens, 32 heads of 128: 176 us, 6.1 TB/s; one row's: 4.7 us.  fp32 T=777, 18
// heads of 96 x 80: 166 us, 0.21 us a step.
#pragma once

#include "delta_common.cuh"
#include "ptx.cuh"

namespace wkvb {

// 16-byte asynchronous copies global -> shared
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last N groups have landed
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kRecSteps = 8;     // steps staged in shared memory at a time
constexpr float kRecSmall = 5.9604645e-8f;  // 2^-24
constexpr float kRecLarge = 16777216.f;     // 2^24

template <typename IO>
struct DeltaFwdArgs {
    const IO *q, *k, *v;
    const float *g, *beta;
    const float *s_in;  // [B, HV, DK, DV] or NULL
    IO *o;              // outputs (kOutputs), or
    float *r;           // residuals r_t [B, T, HV, DV] and
    float *starts;      // the state before each chunk [chunks][B, HV, DK, DV]
                        // (the gradient's sweep)
    float *s_out;       // [B, HV, DK, DV] or NULL
    float scale;
    DeltaSizes z;
};

template <typename IO>
struct DeltaRevArgs {
    const IO *q, *k, *go;
    const float *g, *beta;
    const float *gs_out;  // gradient of the last state or NULL
    IO *gv;
    float *du;            // D_t^T k_t [B, T, HV, DV]
    float *ends;          // gradient of the state after each chunk [chunks][B, HV, DK, DV]
    float *gs_in;         // gradient of s_in or NULL
    float scale;
    DeltaSizes z;
};

// Shared memory of one block: two stages of kRecSteps steps of q, k (rows
// beyond DK zero) and of one value tensor, as they are in memory, and the
// per-step scalars.
template <typename IO, int RPT, int COLS>
struct RecStage {
    static constexpr int kRows = 8 * RPT;
    alignas(16) IO q[2][kRecSteps][kRows];
    alignas(16) IO k[2][kRecSteps][kRows];
    alignas(16) IO x[2][kRecSteps][COLS];
    alignas(16) float4 step[kRecSteps];  // c: the product of the decays; 1 / c; beta; q.k
    float a[kRecSteps];
    float fold;                          // the whole stage's product
    int smooth;                          // every c is within [kRecSmall, kRecLarge]
};

// the state tile of one lane
template <int RPT, int CPL>
struct RecTile {
    float s[RPT][CPL];
};

template <int RPT>
__device__ __forceinline__ int rec_row(int r, int grp) {
    return 32 * (r >> 2) + 4 * grp + (r & 3);
}

template <int RPT, int CPL>
__device__ __forceinline__ void rec_load(RecTile<RPT, CPL> &t, const float *p, int grp, int col0, int DK,
                                         int DV) {
    const bool vec = CPL == 4 && DV % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int row = rec_row<RPT>(r, grp);
        if constexpr (CPL == 4)
            if (p != nullptr && row < DK && vec && col0 < DV) {
                const float4 x = *reinterpret_cast<const float4 *>(p + static_cast<size_t>(row) * DV + col0);
                t.s[r][0] = x.x, t.s[r][1] = x.y, t.s[r][2] = x.z, t.s[r][3] = x.w;
                continue;
            }
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            t.s[r][c] = (p != nullptr && row < DK && col0 + c < DV)
                            ? p[static_cast<size_t>(row) * DV + col0 + c] : 0.f;
    }
}

template <int RPT, int CPL>
__device__ __forceinline__ void rec_store(const RecTile<RPT, CPL> &t, float *p, int grp, int col0, int DK, int DV) {
    const bool vec = CPL == 4 && DV % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int row = rec_row<RPT>(r, grp);
        if (row >= DK) continue;
        if constexpr (CPL == 4)
            if (vec && col0 < DV) {
                *reinterpret_cast<float4 *>(p + static_cast<size_t>(row) * DV + col0) =
                    make_float4(t.s[r][0], t.s[r][1], t.s[r][2], t.s[r][3]);
                continue;
            }
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            if (col0 + c < DV) p[static_cast<size_t>(row) * DV + col0 + c] = t.s[r][c];
    }
}

__device__ __forceinline__ float rec_xor(float x, int s) { return __shfl_xor_sync(0xffffffffu, x, s); }

// Sums of x and y, CPL = 4, over the eight lanes that share columns (lane bits
// 2..4).  Returns one finished sum: of x in lanes with bit 4 clear, of y in the
// others, for column rec_col<4>(lane).
template <int CPL>
__device__ __forceinline__ int rec_col(int lane) {
    return CPL == 4 ? (lane >> 2) & 3 : 0;
}
__device__ __forceinline__ float rec_reduce2(const float (&x)[4], const float (&y)[4], int lane) {
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = (b4 ? y[i] : x[i]) + rec_xor(b4 ? x[i] : y[i], 16);
    const float g0 = rec_xor(b3 ? z[0] : z[2], 8), g1 = rec_xor(b3 ? z[1] : z[3], 8);
    const float w0 = (b3 ? z[2] : z[0]) + g0, w1 = (b3 ? z[3] : z[1]) + g1;
    return (b2 ? w1 : w0) + rec_xor(b2 ? w0 : w1, 4);
}

// Sum of x alone.  CPL = 4: every lane ends with column rec_col's; CPL = 1:
// with its only column's.
template <int CPL>
__device__ __forceinline__ float rec_reduce1(const float (&x)[CPL], int lane) {
    const bool b3 = lane & 8, b2 = lane & 4;
    float z;
    if constexpr (CPL == 4) {
        const float g0 = rec_xor(b3 ? x[0] : x[2], 8), g1 = rec_xor(b3 ? x[1] : x[3], 8);
        const float w0 = (b3 ? x[2] : x[0]) + g0, w1 = (b3 ? x[3] : x[1]) + g1;
        z = (b2 ? w1 : w0) + rec_xor(b2 ? w0 : w1, 4);
    } else {
        const float w = x[0] + rec_xor(x[0], 8);
        z = w + rec_xor(w, 4);
    }
    return z + rec_xor(z, 16);
}

// the lane's columns' values, each from a lane (bit 4 clear) that holds it
template <int CPL>
__device__ __forceinline__ void rec_spread(float z, int lane, float (&u)[CPL]) {
#pragma unroll
    for (int j = 0; j < CPL; ++j) u[j] = __shfl_sync(0xffffffffu, z, 4 * j + (lane & 3));
}

// four rows of a staged q or k
__device__ __forceinline__ void rec_four(const float *p, float *x) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void rec_four(const __nv_bfloat16 *p, float *x) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

// Brings stages of kRecSteps steps in: q, k and the value tensor's columns
// cb .. by asynchronous 16-byte copies where bases and rows are multiples of
// them, element by element otherwise; the scalars in registers.
template <typename IO, int RPT, int NT, int COLS>
struct RecFeed {
    RecStage<IO, RPT, COLS> &sm;
    const IO *q, *k, *x;
    const float *g, *beta;
    const DeltaSizes &z;
    int b, hv, cb;
    bool vec;
    float g1, b1;  // the next stage's, in threads 0 .. kRecSteps - 1
    // this thread's 16-byte pieces of one step's q and k, and of one stage's x
    static constexpr int W = 16 / sizeof(IO);
    static constexpr int PK = (2 * 8 * RPT / W + NT - 1) / NT;
    static constexpr int PX = COLS / W, NX = (kRecSteps * PX + NT - 1) / NT;
    const IO *src[PK];  // at step 0
    uint32_t dst[PK];
    size_t key_step, val_step;

    __device__ RecFeed(RecStage<IO, RPT, COLS> &s, const IO *q_, const IO *k_, const IO *x_, const float *g_,
                       const float *beta_, const DeltaSizes &z_, int b_, int hv_, int cb_)
        : sm(s), q(q_), k(k_), x(x_), g(g_), beta(beta_), z(z_), b(b_), hv(hv_), cb(cb_), g1(0.f), b1(0.f) {
        const uintptr_t any = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                              reinterpret_cast<uintptr_t>(x);
        vec = any % 16 == 0 && z.DK % W == 0 && z.DV % W == 0;
        key_step = static_cast<size_t>(z.HK) * z.DK, val_step = static_cast<size_t>(z.HV) * z.DV;
        const size_t row = token_offset(b, 0, hv / z.group, z.T, z.HK, z.DK);
        const int pk = z.DK / W;
#pragma unroll
        for (int p = 0; p < PK; ++p) {
            const int i = threadIdx.x + p * NT, e = (i < pk ? i : i - pk) * W;
            src[p] = i >= 2 * pk ? nullptr : (i < pk ? q : k) + row + e;
            dst[p] = smem_addr(i < pk ? &sm.q[0][0][e] : &sm.k[0][0][i < 2 * pk ? e : 0]);
        }
        for (int i = threadIdx.x; i < static_cast<int>(sizeof(sm.q) / 4); i += NT) {
            reinterpret_cast<uint32_t *>(sm.q)[i] = 0;
            reinterpret_cast<uint32_t *>(sm.k)[i] = 0;
        }
        __syncthreads();
    }
    // starts a stage's copies: steps t0 .. t0 + n - 1 into buffer s
    __device__ __forceinline__ void start(int s, int t0, int n) {
        if (threadIdx.x < n) {
            const size_t o = (static_cast<size_t>(b) * z.T + t0 + threadIdx.x) * z.HV + hv;
            g1 = g[o], b1 = beta[o];
        }
        if (vec) {
            constexpr uint32_t kRowBytes = 8 * RPT * sizeof(IO), kStageBytes = kRecSteps * kRowBytes;
#pragma unroll
            for (int p = 0; p < PK; ++p) {
                if (src[p] == nullptr) continue;
                const IO *from = src[p] + t0 * key_step;
                const uint32_t to = dst[p] + s * kStageBytes;
#pragma unroll
                for (int t = 0; t < kRecSteps; ++t)
                    if (t < n) {
                        cp_async16(to + t * kRowBytes, from);
                        from += key_step;
                    }
            }
            const IO *v = x + token_offset(b, t0, hv, z.T, z.HV, z.DV) + cb;
#pragma unroll
            for (int p = 0; p < NX; ++p) {
                const int i = threadIdx.x + p * NT, t = i / PX, e = i % PX * W;
                if (t < n && cb + e < z.DV) cp_async16(smem_addr(&sm.x[s][t][e]), v + t * val_step + e);
            }
        } else {
            for (int t = 0; t < n; ++t) {
                const size_t o = token_offset(b, t0 + t, hv / z.group, z.T, z.HK, z.DK);
                for (int i = threadIdx.x; i < z.DK; i += NT) sm.q[s][t][i] = q[o + i], sm.k[s][t][i] = k[o + i];
                const size_t v = token_offset(b, t0 + t, hv, z.T, z.HV, z.DV) + cb;
                for (int i = threadIdx.x; i < COLS; i += NT)
                    if (cb + i < z.DV) sm.x[s][t][i] = x[v + i];
            }
        }
        cp_async_commit();
    }
    // e^x to a float's precision
    static __device__ __forceinline__ float exp_of(double x) {
        const float hi = static_cast<float>(x), e = expf(hi);
        return hi > -200.f ? fmaf(e, static_cast<float>(x - hi), e) : e;
    }
    // The scalars of the stage started last become this one's; c_t includes
    // a_t and what came before it, or in the reverse sweep what comes after
    // step t without a_t.
    template <bool kReverse>
    __device__ __forceinline__ void scalars(int n) {
        if (threadIdx.x >= 32) return;
        const int t = threadIdx.x;
        // the decays' logarithms are summed, in double, so that a long run of
        // mild ones costs one rounding of an exponential a stage and not one a step
        double sum = t < n ? g1 : 0.f;
#pragma unroll
        for (int s = 1; s < kRecSteps; s *= 2) {
            const double other = kReverse ? __shfl_down_sync(0xffffffffu, sum, s) : __shfl_up_sync(0xffffffffu, sum, s);
            if (kReverse ? t + s < kRecSteps : t >= s) sum += other;
        }
        const float fold = exp_of(__shfl_sync(0xffffffffu, sum, kReverse ? 0 : kRecSteps - 1));
        if (kReverse) {
            sum = __shfl_down_sync(0xffffffffu, sum, 1);
            if (t == kRecSteps - 1) sum = 0.0;
        }
        const float c = exp_of(sum);
        const bool fine = t >= kRecSteps || (c >= kRecSmall && c <= kRecLarge);
        const int smooth = __all_sync(0xffffffffu, fine);
        if (t < kRecSteps) {
            sm.a[t] = t < n ? expf(g1) : 1.f;
            sm.step[t].x = c, sm.step[t].y = 1.f / c, sm.step[t].z = b1;
        }
        if (t == 0) sm.fold = fold, sm.smooth = smooth;
    }
    // q.k of the stage's steps, four lanes a step; for the whole block
    __device__ __forceinline__ void products(int s, int n) {
        const int t = threadIdx.x >> 2, c = threadIdx.x & 3;
        float d = 0.f;
        if (threadIdx.x < 32) {
#pragma unroll
            for (int i = 0; i < RPT / 2; ++i) {
                float x4[4], y4[4];
                rec_four(&sm.q[s][t][16 * i + 4 * c], x4);
                rec_four(&sm.k[s][t][16 * i + 4 * c], y4);
#pragma unroll
                for (int e = 0; e < 4; ++e) d = fmaf(x4[e], y4[e], d);
            }
            d += rec_xor(d, 1);
            d += rec_xor(d, 2);
            if (c == 0 && t < n) sm.step[t].w = d;
        }
    }
};

// RPT: rows per lane, 8 lanes deep (DK <= 8 RPT); NW: warps per block, each
// its own 4 CPL columns; kOutputs: writes o, else the gradient sweep's r and
// chunk states.  Grid: B * HV * ceil(DV / (4 CPL NW)) blocks, columns fastest.
template <typename IO, int RPT, int NW, int CPL, bool kOutputs>
__device__ __forceinline__ void delta_recurrent(const DeltaFwdArgs<IO> &a, RecStage<IO, RPT, 4 * CPL * NW> &sm,
                                                unsigned block) {
    constexpr int kCols = 4 * CPL * NW;
    const DeltaSizes &z = a.z;
    const int ncb = (z.DV + kCols - 1) / kCols;
    const int cb = static_cast<int>(block % ncb) * kCols;
    const long long bh = block / ncb;
    const int b = static_cast<int>(bh / z.HV), hv = static_cast<int>(bh % z.HV);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int grp = lane >> 2, cl = lane & 3;
    const int wc = warp * 4 * CPL;            // this warp's columns in the block's
    const int col0 = cb + wc + CPL * cl;
    const int j = rec_col<CPL>(lane);         // the column it finishes
    const bool writer = CPL == 4 || (lane & 12) == 0;  // of the lanes that finish the same
    const size_t per_state = static_cast<size_t>(z.DK) * z.DV;

    RecFeed<IO, RPT, 32 * NW, kCols> feed(sm, a.q, a.k, a.v, a.g, a.beta, z, b, hv, cb);
    feed.start(0, 0, min(kRecSteps, z.T));
    RecTile<RPT, CPL> S;
    rec_load<RPT, CPL>(S, a.s_in == nullptr ? nullptr : a.s_in + bh * per_state, grp, col0, z.DK, z.DV);
    const int oc = wc + CPL * cl + j;  // the column this lane finishes
    constexpr int kSums = CPL == 1 ? 2 : 1;  // independent sums per column
    // step t of the staged ones; the registers hold S / c, c and 1 / c in f
    const auto step = [&](int st, int t, size_t out, float4 f) {
        const float c0 = f.x;
        float k[RPT], sk[kSums][CPL] = {}, sq[kSums][CPL] = {};
#pragma unroll
        for (int r = 0; r < RPT; r += 4) {
            rec_four(&sm.k[st][t][rec_row<RPT>(r, grp)], &k[r]);
            float q[4] = {};
            if constexpr (kOutputs) rec_four(&sm.q[st][t][rec_row<RPT>(r, grp)], q);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    sk[e % kSums][c] = fmaf(S.s[r + e][c], k[r + e], sk[e % kSums][c]);
                    if constexpr (kOutputs) sq[e % kSums][c] = fmaf(S.s[r + e][c], q[e], sq[e % kSums][c]);
                }
        }
        if constexpr (kSums == 2) sk[0][0] += sk[1][0], sq[0][0] += sq[1][0];
        const float xt = to_f32(sm.x[st][t][oc]);
        float res, oq = 0.f, u[CPL], uj;
        if constexpr (kOutputs && CPL == 4) {
            const float sum = rec_reduce2(sk[0], sq[0], lane);
            res = xt - c0 * sum;  // of use where bit 4 is clear
            oq = c0 * sum;        // of use where it is set
        } else {
            res = xt - c0 * rec_reduce1<CPL>(sk[0], lane);
        }
        if constexpr (CPL == 4) {
            rec_spread<4>(f.z * res, lane, u);
            uj = j == 0 ? u[0] : j == 1 ? u[1] : j == 2 ? u[2] : u[3];
        } else {
            u[0] = uj = f.z * res;
        }
        if constexpr (kOutputs) {
            if constexpr (CPL == 1) oq = c0 * rec_reduce1<1>(sq[0], lane);
            if ((lane & 16) && writer && cb + oc < z.DV) from_f32(a.o + out, a.scale * fmaf(f.w, uj, oq));
        } else {
            if (!(lane & 16) && writer && cb + oc < z.DV) a.r[out] = res;
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) u[c] *= f.y;
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int c = 0; c < CPL; ++c) S.s[r][c] = fmaf(k[r], u[c], S.s[r][c]);
    };
    const auto decay = [&](float f) {
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int c = 0; c < CPL; ++c) S.s[r][c] *= f;
    };

    for (int t0 = 0, st = 0; t0 < z.T; t0 += kRecSteps, st ^= 1) {
        const int n = min(kRecSteps, z.T - t0);
        feed.template scalars<false>(n);
        const int left = z.T - t0 - kRecSteps;
        if (left > 0) {
            feed.start(st ^ 1, t0 + kRecSteps, min(kRecSteps, left));
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        if constexpr (kOutputs) {
            feed.products(st, n);
            __syncthreads();
        } else if (t0 % kDeltaChunk == 0) {
            const size_t heads = static_cast<size_t>(z.B) * z.HV;
            rec_store<RPT, CPL>(S, a.starts + ((t0 / kDeltaChunk) * heads + bh) * per_state, grp, col0, z.DK, z.DV);
        }
        size_t out = token_offset(b, t0, hv, z.T, z.HV, z.DV) + cb + oc;
        if (n == kRecSteps && sm.smooth) {
#pragma unroll CPL == 1 ? 4 : 1
            for (int t = 0; t < kRecSteps; ++t, out += feed.val_step) step(st, t, out, sm.step[t]);
            decay(sm.fold);
        } else {
            for (int t = 0; t < n; ++t, out += feed.val_step) {
                decay(sm.a[t]);
                step(st, t, out, make_float4(1.f, 1.f, sm.step[t].z, sm.step[t].w));
            }
        }
        __syncthreads();  // the stage is read
    }
    if (kOutputs && a.s_out != nullptr)
        rec_store<RPT, CPL>(S, a.s_out + bh * per_state, grp, col0, z.DK, z.DV);
}

// The reverse sweep: D is the gradient of the state, last step first.
//     D_t = D + scale q_t go_t^T,  du_t = D_t^T k_t,  gv_t = beta_t du_t,
//     D <- a_t (D_t - k_t gv_t^T)
// with the same column split, and du_t = D^T k_t + scale (q.k) go_t, so the
// one sum over rows is taken before the update.  Writes du, gv and, for every
// chunk, the gradient of the state after it.
template <typename IO, int RPT, int NW, int CPL>
__device__ __forceinline__ void delta_reverse(const DeltaRevArgs<IO> &a, RecStage<IO, RPT, 4 * CPL * NW> &sm,
                                              unsigned block) {
    constexpr int kCols = 4 * CPL * NW;
    const DeltaSizes &z = a.z;
    const int ncb = (z.DV + kCols - 1) / kCols;
    const int cb = static_cast<int>(block % ncb) * kCols;
    const long long bh = block / ncb;
    const int b = static_cast<int>(bh / z.HV), hv = static_cast<int>(bh % z.HV);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int grp = lane >> 2, cl = lane & 3, j = rec_col<CPL>(lane);
    const bool writer = CPL == 4 || (lane & 12) == 0;
    const int wc = warp * 4 * CPL;
    const int col0 = cb + wc + CPL * cl;
    const size_t per_state = static_cast<size_t>(z.DK) * z.DV;
    const size_t heads = static_cast<size_t>(z.B) * z.HV;

    RecFeed<IO, RPT, 32 * NW, kCols> feed(sm, a.q, a.k, a.go, a.g, a.beta, z, b, hv, cb);
    const int last = (z.T - 1) / kRecSteps * kRecSteps;
    feed.start(0, last, z.T - last);
    RecTile<RPT, CPL> D;
    rec_load<RPT, CPL>(D, a.gs_out == nullptr ? nullptr : a.gs_out + bh * per_state, grp, col0, z.DK, z.DV);
    const int oc = wc + CPL * cl + j;
    constexpr int kSums = CPL == 1 ? 2 : 1;
    const auto step = [&](int st, int t, size_t out, float4 f) {
        float k[RPT], q[RPT], sk[kSums][CPL] = {};
#pragma unroll
        for (int r = 0; r < RPT; r += 4) {
            rec_four(&sm.k[st][t][rec_row<RPT>(r, grp)], &k[r]);
            rec_four(&sm.q[st][t][rec_row<RPT>(r, grp)], &q[r]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < CPL; ++c) sk[e % kSums][c] = fmaf(D.s[r + e][c], k[r + e], sk[e % kSums][c]);
        }
        if constexpr (kSums == 2) sk[0][0] += sk[1][0];
        const float du = fmaf(a.scale * f.w, to_f32(sm.x[st][t][oc]), f.x * rec_reduce1<CPL>(sk[0], lane));
        const float w = f.z * du;
        if (!(lane & 16) && writer && cb + oc < z.DV) {
            a.du[out] = du;
            from_f32(a.gv + out, w);
        }
        float wj[CPL], gj[CPL];
        if constexpr (CPL == 4) rec_spread<4>(w, lane, wj);
        else wj[0] = w;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            wj[c] *= -f.y;
            gj[c] = a.scale * f.y * to_f32(sm.x[st][t][wc + CPL * cl + c]);
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int c = 0; c < CPL; ++c) D.s[r][c] = fmaf(k[r], wj[c], fmaf(q[r], gj[c], D.s[r][c]));
    };
    const auto decay = [&](float f) {
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int c = 0; c < CPL; ++c) D.s[r][c] *= f;
    };

    for (int t0 = last, st = 0; t0 >= 0; t0 -= kRecSteps, st ^= 1) {
        const int n = min(kRecSteps, z.T - t0);
        feed.template scalars<true>(n);
        if (t0 > 0) {
            feed.start(st ^ 1, t0 - kRecSteps, kRecSteps);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        feed.products(st, n);
        __syncthreads();
        if (t0 + n == z.T || (t0 + n) % kDeltaChunk == 0)
            rec_store<RPT, CPL>(D, a.ends + ((t0 / kDeltaChunk) * heads + bh) * per_state, grp, col0, z.DK, z.DV);
        size_t out = token_offset(b, t0 + n - 1, hv, z.T, z.HV, z.DV) + cb + oc;
        if (n == kRecSteps && sm.smooth) {
#pragma unroll CPL == 1 ? 4 : 1
            for (int t = kRecSteps - 1; t >= 0; --t, out -= feed.val_step) step(st, t, out, sm.step[t]);
            decay(sm.fold);
        } else {
            for (int t = n - 1; t >= 0; --t, out -= feed.val_step) {
                step(st, t, out, make_float4(1.f, 1.f, sm.step[t].z, sm.step[t].w));
                decay(sm.a[t]);
            }
        }
        __syncthreads();  // the stage is read
    }
    if (a.gs_in != nullptr)
        rec_store<RPT, CPL>(D, a.gs_in + bh * per_state, grp, col0, z.DK, z.DV);
}

template <typename IO, int RPT, int NW, int CPL>
__global__ void __launch_bounds__(32 * NW) delta_recurrent_kernel(const DeltaFwdArgs<IO> a) {
    __shared__ RecStage<IO, RPT, 4 * CPL * NW> sm;
    delta_recurrent<IO, RPT, NW, CPL, true>(a, sm, blockIdx.x);
}

// Both sweeps of the gradient at once: neither needs the other, and a step's
// latency is what bounds them.
template <typename IO, int RPT, int NW, int CPL>
__global__ void __launch_bounds__(32 * NW) delta_recurrent_sweeps_kernel(const DeltaFwdArgs<IO> f,
                                                                         const DeltaRevArgs<IO> r) {
    __shared__ RecStage<IO, RPT, 4 * CPL * NW> sm;
    const unsigned half = gridDim.x / 2;
    if (blockIdx.x < half) delta_recurrent<IO, RPT, NW, CPL, false>(f, sm, blockIdx.x);
    else delta_reverse<IO, RPT, NW, CPL>(r, sm, blockIdx.x - half);
}

}  // namespace wkvb
