// Gated delta rule over chunks of 64 steps on the tensor cores, bf16 I/O: the
// forward, and the two state sweeps of the gradient.
//
// With G the cumulative log decay inside the chunk, E_i = e^{G_i}, F_i =
// e^{G_last - G_i}, A_ij = e^{G_i - G_j} (i >= j) and S0 the state before it,
// the residuals r of the chunk's steps solve a unit triangular system, and
// everything else is a product:
//
//     L_ij = A_ij (k_i.k_j) beta_j  (i > j),   M_ij = A_ij (q_i.k_j) beta_j  (i >= j)
//     r = (I + L)^{-1} (V - E (K S0))
//     O = scale (E (Q S0) + M r),   S1 = E_last S0 + K^T (F beta r)
//
// Backwards in time, D1 the gradient of the state after the chunk:
//
//     L'_ij = beta_i A_ij (k_i.k_j)  (i > j),   X_ij = A_ij (q_i.k_j)  (i >= j)
//     du = (I + L')^{-T} (F (K D1) + scale X^T GO)
//     D0 = E_last D1 + Q^T (scale E GO) - K^T (E beta du)
//
// the same recurrence with other matrices.  Two kernels:
//
//   delta_prep_kernel, one block per chunk and head: all that does not need
//   the state.  K K^T, Q K^T, the decays, (I + L)^{-1} and its relatives, as
//   bf16 operand tiles in scratch memory, laid out as the chain's shared
//   memory wants them.
//
//   delta_chain(), one block per head (the kernels delta_forward_kernel and
//   delta_sweeps_kernel): only the products with the state
//   and what depends on them:
//
//       P = S0^T K^T;  x = V^T T^T + (a P) T^T;  S1 = e S0 + (b x)^T K
//
//   with per-step factors a, b (-E and F beta, or F and -E beta).  Column j of
//   the state meets only column j of V, so the state is kept transposed: a
//   lane of tensor memory is a column of S (an entry of v), every product of
//   the chain has the chunk's matrix as its shared-memory operand and the
//   lane's vector as its tensor-memory operand, and nothing moves between
//   lanes.  The part of x without the state is accumulated first, straight
//   from V's tile, while the chain waits for P.
//
//     warps 0-7   the chain; warp w reads lanes 32 (w % 4) .., warps 0-3 the
//                 first half of every product's columns, warps 4-7 the second.
//                 The state's fp32 value is in registers.
//     next four   off the chain: the output -- r again as an operand of M r,
//                 then scale (E (Q S0) + M r) --, or the stores of a sweep
//     then one    TMA: tiles, a chunk ahead
//     and one     issues every tcgen05.mma
//
// Precision: fp32 sums everywhere.  Operands that are not inputs (S, P, x, the
// inverse) enter as kParts bf16 parts, and of a product of two of them the
// part pairs that matter: three parts (all 24 bits, six pairs) where an fp32
// result leaves the kernel -- the state, or anything of the gradient --, two
// parts (16 bits, three pairs) where only o does, and in what reaches nothing
// but o: S in Q S0, M and r in M r.  16 bits leave the value that is rounded
// to o within 2^-16 of its terms' size, so that o is the rounding of the exact
// value for all but one element in some 300 (with M in one part its error was
// 1.3 to 1.4 times the rounding's).
//
// Bound: the chain of three dependent products per chunk with the loads and
// conversions between them, not bandwidth: 5200 cycles with 64 columns in two
// parts, 8100 with 128 in three, of which the tensor cores work 1500 and 3200.
// B=8 T=4096, 40 heads of 64: preparation 264 us, chain 540 us; B=1 T=16384, 32
// heads of 128 with the state: 154 and 1040 us (step by step: 3932 and 21924 in
// all).  Both sweeps of B=2 T=4096, 32 heads of 128: 303 us, for 870 MB of
// stores.
#pragma once

#include "delta_common.cuh"
#include "tcgen05.cuh"

namespace wkvb {

enum DeltaMode {
    kFwdOut,     // o and the last state
    kFwdStates,  // the gradient's first sweep: residuals and the chunks' states
    kReverse     // its second: du, gv and the gradients of the chunks' states
};

// Per-step factors of one chunk, at the end of its tiles.
struct ChunkScalars {
    float a[kDeltaChunk], b[kDeltaChunk];  // factors of P and of x
    float e_last;
};
constexpr int kScalarBytes = 1024;
constexpr int kTileBytes = 64 * 128;  // one 64 x 64 bf16 operand

// Scratch of one chunk and head for the chain: the inverse's parts, M's two where
// the mode has it, the scalars; for kReverse also (second buffer) the parts
// of scale X (I + L')^{-1} and of scale E Q.
template <int kParts, int kMode>
struct ChunkImage {
    static constexpr int kM = kParts * kTileBytes;
    static constexpr int kScalars = kM + (kMode == kFwdOut ? 2 * kTileBytes : 0);
    static constexpr int kBytes = kScalars + kScalarBytes;
};
__host__ __device__ constexpr int second_image_bytes(int ksub) { return 3 * (1 + ksub) * kTileBytes; }

// What a sweep leaves of `rows` steps or state rows of chunk and head `at`:
// [DV / 16][rows / 8][16 columns][8 rows], so that 16 columns of everything are
// one piece, DV rounded up.  The place of column dv's first eight; the next
// eights follow kSweepEight floats apart.
constexpr int kSweepCols = 16, kSweepEight = 8 * kSweepCols;
__host__ __device__ inline size_t sweep_floats(int64_t rows, int64_t DV) {
    return static_cast<size_t>(rows) * ((DV + kSweepCols - 1) / kSweepCols * kSweepCols);
}
__device__ __forceinline__ size_t sweep_at(const DeltaSizes &z, size_t at, int rows, int dv) {
    return at * sweep_floats(rows, z.DV) + static_cast<size_t>(dv / kSweepCols) * rows * kSweepCols +
           dv % kSweepCols * 8;
}

struct DeltaPrepArgs {
    const float *g, *beta;
    unsigned char *fwd, *rev, *rev2;  // images [chunks][B * HV]
    float scale;
    DeltaSizes z;
    int silent;  // for tests of the bounded waits: the chunk whose copies are not made, or -1
};

struct DeltaChainArgs {
    const unsigned char *img, *img2;  // images [chunks][B * HV]
    const float *s_in;                // [B, HV, DK, DV] or NULL; gs_out for kReverse
    __nv_bfloat16 *o;                 // kFwdOut
    float *s_out;                     // [B, HV, DK, DV] or NULL; gs_in for kReverse
    float *x;                         // sweeps: r or du, of 64 steps per chunk and head, and
    float *states;                    // S0 or D1, of DK rows: as sweep_at() says
    float scale;
    DeltaSizes z;
    int silent;  // for tests of the bounded waits: the chunk whose copies are not made, or -1
};

constexpr int kChLd = 68;  // floats per row of the 64 x 64 fp32 work matrices

// A chunk's cumulative log decays G_t, in double (64 terms down to -120 each;
// their differences go to fp32), and beta: steps 2 lane and 2 lane + 1 of one
// warp.  Steps beyond T have g = beta = 0.  Returns G of the last step.
__device__ __forceinline__ double delta_scan_g(const float *g, const float *beta, const DeltaSizes &z, int b,
                                               int hv, int t0, int lane, float (&bt)[2], double (&d)[2]) {
    const int n = min(kDeltaChunk, z.T - t0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        const size_t o = (static_cast<size_t>(b) * z.T + t0 + t) * z.HV + hv;
        bt[e] = t < n ? beta[o] : 0.f;
        d[e] = t < n ? delta_clamp_g(g[o]) : 0.f;
    }
    double run = d[0] + d[1];
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
        const double up = __shfl_up_sync(0xffffffffu, run, s);
        if (lane >= s) run += up;
    }
    d[0] = run - d[1], d[1] = run;
    return __shfl_sync(0xffffffffu, run, 31);
}

// byte offset of 16-byte piece `c` (0..7) of row `r` in a 128-byte-swizzled
// tile whose base is a multiple of 1024
__device__ __forceinline__ uint32_t swz128(int r, int c) {
    return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// Fragments of fp32 row-major matrices in shared memory (leading dimension
// kChLd) as N bf16 parts: A (16 x 16 at row r0, column c0)
template <int N>
struct FragA {
    uint32_t x[N][4];
    __device__ __forceinline__ void load(const float *m, int r0, int c0, int lane) {
        const int r = r0 + (lane >> 2), c = c0 + 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = *reinterpret_cast<const float2 *>(&m[(r + (i & 1) * 8) * kChLd + c + (i >> 1) * 8]);
            set(i, f.x, f.y);
        }
    }
    // C fragments of two neighbouring 8-column tiles, negated
    __device__ __forceinline__ void from_c(const float (&c0)[4], const float (&c1)[4]) {
        set(0, -c0[0], -c0[1]);
        set(1, -c0[2], -c0[3]);
        set(2, -c1[0], -c1[1]);
        set(3, -c1[2], -c1[3]);
    }
    __device__ __forceinline__ void set(int i, float a, float b) {
        uint32_t p[N];
        split_bf16<N>(a, b, p);
#pragma unroll
        for (int e = 0; e < N; ++e) x[e][i] = p[e];
    }
};
// ... and B (16 x 8 at row k0, column n0)
template <int N>
struct FragB {
    uint32_t x[N][2];
    __device__ __forceinline__ void load(const float *m, int k0, int n0, int lane) {
        const int k = k0 + 2 * (lane & 3), n = n0 + (lane >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t p[N];
            split_bf16<N>(m[(k + 8 * i) * kChLd + n], m[(k + 8 * i + 1) * kChLd + n], p);
#pragma unroll
            for (int e = 0; e < N; ++e) x[e][i] = p[e];
        }
    }
};
// C += A B over the part pairs that matter, small ones first
template <int N>
__device__ __forceinline__ void mma_split(float (&c)[4], const FragA<N> &a, const FragB<N> &b) {
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i) mma16816(c, a.x[i], b.x[s - i][0], b.x[s - i][1]);
}

// t = (I + l)^{-1} for a strictly lower triangular 64 x 64 l; a block of four
// warps, with a barrier at the end.  The 16 x 16 blocks of t above the
// diagonal ones are not written.
template <int N>
__device__ __forceinline__ void invert_unit_lower(const float *l, float *t, int warp, int lane) {
    {   // diagonal blocks: x_i = d_ic - sum_{k < i} l_ik x_k, one column per lane
        const int o = 16 * warp, c = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a0 = i == c ? 1.f : 0.f, a1 = 0.f;
#pragma unroll
            for (int k = 0; k < i; k += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(&l[(o + i) * kChLd + o + k]);
                a0 = fmaf(-f.x, x[k], a0);
                if (k + 1 < i) a1 = fmaf(-f.y, x[k + 1], a1);
                if (k + 2 < i) a0 = fmaf(-f.z, x[k + 2], a0);
                if (k + 3 < i) a1 = fmaf(-f.w, x[k + 3], a1);
            }
            x[i] = a0 + a1;
        }
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) t[(o + i) * kChLd + o + c] = x[i];
        }
    }
    __syncthreads();
    const int r = lane >> 2, c2 = 2 * (lane & 3);
    {   // blocks (1,0) and (3,2): -X_i L X_j, 8 columns per warp
        const int bi = 16 * (1 + 2 * (warp >> 1)), bj = bi - 16, n0 = bj + 8 * (warp & 1);
        FragA<N> fa;
        FragB<N> fb;
        float z[2][4] = {}, y[4] = {};
        fa.load(t, bi, bi, lane);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            fb.load(l, bi, bj + 8 * n, lane);
            mma_split<N>(z[n], fa, fb);
        }
        fa.from_c(z[0], z[1]);
        fb.load(t, bj, n0, lane);
        mma_split<N>(y, fa, fb);
        *reinterpret_cast<float2 *>(&t[(bi + r) * kChLd + n0 + c2]) = make_float2(y[0], y[1]);
        *reinterpret_cast<float2 *>(&t[(bi + r + 8) * kChLd + n0 + c2]) = make_float2(y[2], y[3]);
    }
    __syncthreads();
    {   // the lower left quarter: warp = (16-row block, 16-column half)
        const int m = warp >> 1, r0 = 32 + 16 * m, n0 = 16 * (warp & 1);
        FragA<N> fa;
        FragB<N> fb;
        float z[4][4] = {};
        for (int kb = 0; kb <= m; ++kb) {
            fa.load(t, r0, 32 + 16 * kb, lane);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                fb.load(l, 32 + 16 * kb, 8 * n, lane);
                mma_split<N>(z[n], fa, fb);
            }
        }
        float y[2][4] = {};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (16 * kb < n0) continue;  // X is lower triangular
            fa.from_c(z[2 * kb], z[2 * kb + 1]);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                fb.load(t, 16 * kb, n0 + 8 * n, lane);
                mma_split<N>(y[n], fa, fb);
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            *reinterpret_cast<float2 *>(&t[(r0 + r) * kChLd + n0 + 8 * n + c2]) = make_float2(y[n][0], y[n][1]);
            *reinterpret_cast<float2 *>(&t[(r0 + r + 8) * kChLd + n0 + 8 * n + c2]) = make_float2(y[n][2], y[n][3]);
        }
    }
    __syncthreads();
}

// A work matrix's lower triangle of 16 x 16 blocks as operand tiles, one per
// part, in the 128-byte-swizzled layout; what is above the diagonal within a
// diagonal block has to be zero already.  The blocks above are left: no
// product reads them.
template <int N>
__device__ __forceinline__ void write_lower(const float *m, unsigned char *dst, float scale, int tid) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int p = tid + 128 * e, i = p >> 3, c = p & 7;
        if ((c >> 1) > (i >> 4)) continue;
        float x[8];
        *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(&m[i * kChLd + 8 * c]);
        *reinterpret_cast<float4 *>(x + 4) = *reinterpret_cast<const float4 *>(&m[i * kChLd + 8 * c + 4]);
        uint32_t y[4][N];
#pragma unroll
        for (int q = 0; q < 4; ++q) split_bf16<N>(scale * x[2 * q], scale * x[2 * q + 1], y[q]);
#pragma unroll
        for (int q = 0; q < N; ++q)
            *reinterpret_cast<uint4 *>(dst + q * kTileBytes + swz128(i, c)) =
                make_uint4(y[0][q], y[1][q], y[2][q], y[3][q]);
    }
}

template <int KSUB, bool kGrad>
struct PrepSmem {
    union {
        alignas(1024) unsigned char kq[KSUB * 16384];  // per 64 columns: 64 rows of K, 64 of Q
        alignas(16) float t[64 * kChLd];               // then the inverse
    };
    alignas(16) float m[kGrad ? 64 * kChLd : 4];  // X
    alignas(16) float l[64 * kChLd];
    float ghi[kDeltaChunk], glo[kDeltaChunk];  // G_i as two floats
    float e[kDeltaChunk], f[kDeltaChunk], beta[kDeltaChunk];
    float e_last;
    uint64_t full;
    int dead;
};

// A 4 x 4 transposition among the four lanes of a quad: word j of lane c becomes
// word c of lane j.
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4], int lane) {
#pragma unroll
    for (int s = 1; s <= 2; s *= 2) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & s) continue;
            const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + s], s);
            (up ? x[i] : x[i + s]) = y;
        }
    }
}

// kGrad: both sweeps' images (kFwdStates and kReverse, three parts), else the
// forward's.  Grid: chunks * B * HV, heads fastest.
template <int KSUB, int kParts, bool kGrad>
__global__ void __launch_bounds__(128, kGrad ? (KSUB == 1 ? 4 : 3) : (KSUB == 1 ? 5 : 3))
    delta_prep_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const DeltaPrepArgs a) {
    using Smem = PrepSmem<KSUB, kGrad>;
    // (aligned by the declaration: with room for rounding, one block less fits
    // the SM)
    extern __shared__ __align__(1024) unsigned char tiles[];
    Smem &sm = *reinterpret_cast<Smem *>(tiles);
    const DeltaSizes &z = a.z;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const unsigned heads = static_cast<unsigned>(z.B) * z.HV, bh = blockIdx.x % heads;
    const int b = static_cast<int>(bh / z.HV), hv = static_cast<int>(bh % z.HV), hk = hv / z.group;
    const int t0 = static_cast<int>(blockIdx.x / heads) * kDeltaChunk;
    const bool silent = t0 / kDeltaChunk == a.silent;
    if (tid == 0) {
        sm.dead = 0;
        mbar_init(&sm.full, 1);
        fence_mbar_init();
        if (!silent) {
            mbar_arrive_expect_tx(&sm.full, KSUB * 16384);
#pragma unroll
            for (int s = 0; s < KSUB; ++s) {
                tma_load_4d(sm.kq + s * 16384, &map_k, &sm.full, 64 * s, hk, t0, b);
                tma_load_4d(sm.kq + s * 16384 + 8192, &map_q, &sm.full, 64 * s, hk, t0, b);
            }
        }
    }
    __syncthreads();
    if (w == 0) {  // the warp with the fewest products
        float bt[2];
        double d[2];
        const double last = delta_scan_g(a.g, a.beta, z, b, hv, t0, lane, bt, d);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            sm.ghi[t] = static_cast<float>(d[e]);
            sm.glo[t] = static_cast<float>(d[e] - sm.ghi[t]);
            sm.beta[t] = bt[e];
            sm.e[t] = expf(static_cast<float>(d[e]));
            sm.f[t] = expf(static_cast<float>(last - d[e]));
        }
        if (lane == 0) sm.e_last = expf(static_cast<float>(last));
    }
    // a copy that never lands leaves NaN behind, not old tiles' values
    const bool landed = mbar_wait(&sm.full, 0, &sm.dead);
    if (!landed && !silent && tid == 0) mbar_drain(&sm.full, 0);
    const float poison = landed ? 0.f : __int_as_float(0x7FC00000);

    // K K^T and Q K^T: this warp's 16 rows, columns up to the diagonal
    const int i0 = 16 * w, r = lane >> 2, c2 = 2 * (lane & 3);
    float kk[8][4] = {}, qk[8][4] = {};
    {
        const uint32_t kq = smem_addr(sm.kq);
        const int ksteps = (z.DK + 15) / 16;
#pragma unroll 1
        for (int s = 0; s < ksteps; ++s) {
            const uint32_t base = kq + (s >> 2) * 16384;
            const int ks = (s & 3) * 2;
            uint32_t ak[4], aq[4];
            const uint32_t ao = swz128(i0 + (lane & 15), ks + (lane >> 4));
            ldmatrix4(base + ao, ak);
            ldmatrix4(base + 8192 + ao, aq);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if (p > w) continue;  // warp-uniform
                uint32_t bb[4];
                ldmatrix4(base + swz128(16 * p + (lane & 7) + ((lane >> 4) << 3), ks + ((lane >> 3) & 1)), bb);
                mma16816(kk[2 * p], ak, bb[0], bb[1]);
                mma16816(kk[2 * p + 1], ak, bb[2], bb[3]);
                mma16816(qk[2 * p], aq, bb[0], bb[1]);
                mma16816(qk[2 * p + 1], aq, bb[2], bb[3]);
            }
        }
    }
    __syncthreads();
    // the decays.  Left of the diagonal block e^{G_i - G_j} = e^{G_i - G_ref}
    // e^{G_ref - G_j} with ref the block's first row: neither factor exceeds
    // 1, and there are 14 exponentials instead of 48.
    {
        const float rhi = sm.ghi[i0], rlo = sm.glo[i0];
        float er[2], fc[8][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = i0 + r + 8 * h;
            er[h] = expf((sm.ghi[i] - rhi) + (sm.glo[i] - rlo));
        }
#pragma unroll
        for (int p = 0; p < 6; ++p)
            if (p < 2 * w) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    fc[p][e] = expf((rhi - sm.ghi[8 * p + c2 + e]) + (rlo - sm.glo[8 * p + c2 + e]));
            }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p > 2 * w + 1) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = i0 + r + 8 * h, j = 8 * p + c2 + e;
                    float d;
                    if (p < 2 * w) d = er[h] * fc[p < 6 ? p : 0][e];
                    else d = i >= j ? expf((sm.ghi[i] - sm.ghi[j]) + (sm.glo[i] - sm.glo[j])) : 0.f;
                    kk[p][2 * h + e] = i > j ? d * kk[p][2 * h + e] + poison : 0.f;
                    qk[p][2 * h + e] = i >= j ? d * qk[p][2 * h + e] + poison : 0.f;
                }
        }
    }
    const auto put_l = [&](bool by_row) {  // L, or L'
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p > 2 * w + 1) continue;
            const int j = 8 * p + c2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = i0 + r + 8 * h;
                const float b0 = by_row ? sm.beta[i] : sm.beta[j], b1 = by_row ? b0 : sm.beta[j + 1];
                *reinterpret_cast<float2 *>(&sm.l[i * kChLd + j]) =
                    make_float2(b0 * kk[p][2 * h], b1 * kk[p][2 * h + 1]);
            }
        }
    };
    put_l(false);
    const size_t at = blockIdx.x;
    if constexpr (kGrad) {  // X
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p > 2 * w + 1) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2 *>(&sm.m[(i0 + r + 8 * h) * kChLd + 8 * p + c2]) =
                    make_float2(qk[p][2 * h], qk[p][2 * h + 1]);
        }
    } else {
        // M as two operand tiles, in 16-byte pieces: a quad's four lanes hold
        // four pieces of every part (two column blocks, two rows), a word each
        using Img = ChunkImage<kParts, kFwdOut>;
        unsigned char *img = a.fwd + at * Img::kBytes + Img::kM;
        const int piece = lane & 3;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (m > w) continue;  // warp-uniform
            uint32_t x[4][2], y[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = 2 * m + (e >> 1), h = 2 * (e & 1), j = 8 * p + c2;
                split_bf16<2>(sm.beta[j] * qk[p][h], sm.beta[j + 1] * qk[p][h + 1], x[e]);
                y[0][e] = x[e][0], y[1][e] = x[e][1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                quad_transpose(y[e], lane);
                *reinterpret_cast<uint4 *>(img + e * kTileBytes +
                                           swz128(i0 + r + 8 * (piece & 1), 2 * m + (piece >> 1))) =
                    make_uint4(y[e][0], y[e][1], y[e][2], y[e][3]);
            }
        }
    }
    if constexpr (kGrad) {  // scale E Q
        unsigned char *rev2 = a.rev2 + at * second_image_bytes(KSUB);
#pragma unroll
        for (int e = 0; e < 4 * KSUB; ++e) {
            const int p = tid + 128 * e, s = p >> 9, i = (p >> 3) & 63, c = p & 7;
            const uint4 v = *reinterpret_cast<const uint4 *>(sm.kq + s * 16384 + 8192 + swz128(i, c));
            const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
            const float f = a.scale * sm.e[i] + poison;
            uint32_t y[4][3];
#pragma unroll
            for (int q = 0; q < 4; ++q) split_bf16<3>(f * bf16_low(vv[q]), f * bf16_high(vv[q]), y[q]);
#pragma unroll
            for (int q = 0; q < 3; ++q)
                *reinterpret_cast<uint4 *>(rev2 + (3 + q * KSUB + s) * kTileBytes + swz128(i, c)) =
                    make_uint4(y[0][q], y[1][q], y[2][q], y[3][q]);
        }
    }
    __syncthreads();
    invert_unit_lower<kParts>(sm.l, sm.t, w, lane);
    if constexpr (!kGrad) {
        using Img = ChunkImage<kParts, kFwdOut>;
        unsigned char *img = a.fwd + at * Img::kBytes;
        write_lower<kParts>(sm.t, img, 1.f, tid);
        ChunkScalars *sc = reinterpret_cast<ChunkScalars *>(img + Img::kScalars);
        if (tid < kDeltaChunk) sc->a[tid] = -sm.e[tid], sc->b[tid] = sm.f[tid] * sm.beta[tid];
        if (tid == 0) sc->e_last = sm.e_last;
    } else {
        using Img = ChunkImage<3, kReverse>;
        unsigned char *fwd = a.fwd + at * Img::kBytes, *rev = a.rev + at * Img::kBytes;
        unsigned char *rev2 = a.rev2 + at * second_image_bytes(KSUB);
        write_lower<3>(sm.t, fwd, 1.f, tid);
        ChunkScalars *sc = reinterpret_cast<ChunkScalars *>(fwd + Img::kScalars);
        ChunkScalars *sr = reinterpret_cast<ChunkScalars *>(rev + Img::kScalars);
        if (tid < kDeltaChunk) {
            sc->a[tid] = -sm.e[tid], sc->b[tid] = sm.f[tid] * sm.beta[tid];
            sr->a[tid] = sm.f[tid], sr->b[tid] = -sm.e[tid] * sm.beta[tid];
        }
        if (tid == 0) sc->e_last = sr->e_last = sm.e_last;
        put_l(true);
        __syncthreads();
        invert_unit_lower<3>(sm.l, sm.t, w, lane);
        write_lower<3>(sm.t, rev, 1.f, tid);
        // X (I + L')^{-1}: this warp's 16 rows
        float x[8][4] = {};
        for (int kb = 0; kb <= w; ++kb) {
            FragA<3> fa;
            fa.load(sm.m, i0, 16 * kb, lane);
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                if (p > 2 * kb + 1) continue;
                FragB<3> fb;
                fb.load(sm.t, 16 * kb, 8 * p, lane);
                mma_split<3>(x[p], fa, fb);
            }
        }
        // into L's place: the barrier at the end of the inversion is behind
        // its last read
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p > 2 * w + 1) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2 *>(&sm.l[(i0 + r + 8 * h) * kChLd + 8 * p + c2]) =
                    make_float2(x[p][2 * h], x[p][2 * h + 1]);
        }
        __syncthreads();
        write_lower<3>(sm.l, rev2, a.scale, tid);
    }
}

// ---- the chain ------------------------------------------------------------------

// tensor memory columns (fp32: one per element; bf16 pairs: one per two)
constexpr uint32_t kTmP = 0;      // [64] P = S0^T K^T, then the parts of a P and of b x over it
constexpr uint32_t kTmQ = 64;     // [64] S0^T Q^T
constexpr uint32_t kTmDs = 96;    // [DK <= 128] the state's increment, from Q's second half on
constexpr uint32_t kTmX = 224;    // [64] x, then M r
constexpr uint32_t kTmThird = 288;  // [32] third parts of a P and of b x
constexpr uint32_t kTmS = 320;    // [3][64] S0: parts
constexpr uint32_t kTmCols = 512;
// r as two parts [2][32]: in S's third part's place, or over its first one
// (free once P and Q S are done)
template <int kParts>
constexpr uint32_t kTmR = kTmS + (kParts < 3 ? 128 : 0);

// columns of part `p` of steps 16 k .. 16 k + 15.  Each warp's parts lie where
// it alone has read P.
__device__ __forceinline__ constexpr uint32_t tm_parts(int k, int p) {
    return p < 2 ? kTmP + 32 * (k >> 1) + 16 * p + 8 * (k & 1) : kTmThird + 8 * k;
}

template <int KSUB, int kParts, int kMode>
struct ChainSmem {
    static constexpr int kBlock = kMode == kFwdOut ? 16384 : 8192;  // 64 rows of K (and of Q), 64 columns
    static constexpr int kImage = ChunkImage<kParts, kMode>::kBytes;
    static constexpr int kImage2 = kMode == kReverse ? second_image_bytes(KSUB) : 0;
    alignas(1024) unsigned char kq[2][KSUB * kBlock];
    alignas(1024) unsigned char v[2][16384];
    alignas(1024) unsigned char img2[kImage2 > 0 ? kImage2 : 1024];
    alignas(1024) unsigned char img[2][kImage];
    uint64_t kq_full[2], kq_empty[2], v_full[2], v_empty[2], t_full[2], t_empty[2], z_full, z_empty;
    uint64_t p_full, q_full, r_full, x_full, b_full, d_full, s_full;
    uint64_t q_read, m_full, o_full, s_read, x_free, drain;
    uint32_t tmem;
    int dead;
};

// Threads: eight chain warps, four output warps, a warp group whose first two
// warps load and issue.
constexpr int kChainThreads = 512;

// 16 consecutive steps of this thread's lane as operand parts
template <int N, typename At>
__device__ __forceinline__ void put_parts(const At &at, const float *x) {
    uint32_t y[N][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t p[N];
        split_bf16<N>(x[2 * i], x[2 * i + 1], p);
#pragma unroll
        for (int e = 0; e < N; ++e) y[e][i] = p[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) tmem_st8(at(e), y[e]);
}

template <int KSUB, int kParts, int kMode>
__device__ __forceinline__ void delta_chain(const CUtensorMap &map_q, const CUtensorMap &map_k,
                                            const CUtensorMap &map_v, const DeltaChainArgs &a,
                                            unsigned bh, unsigned char *raw) {
    using Smem = ChainSmem<KSUB, kParts, kMode>;
    using Img = ChunkImage<kParts, kMode>;
    constexpr bool kOut = kMode == kFwdOut, kRev = kMode == kReverse;
    constexpr int kLoadWarp = 12;
    // registers of 256 + 128 + 128 threads: together the launch's 512 * 128.
    // With all of DK = 128 in the chain's it needs more (1202 -> 1164 us for one
    // prompt of 16384 steps, 32 heads of 128), elsewhere the others do.
    constexpr bool kMore = kOut && KSUB == 2;
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const DeltaSizes &z = a.z;
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int b = static_cast<int>(bh / z.HV), hv = static_cast<int>(bh % z.HV), hk = hv / z.group;
    const int chunks = (z.T + kDeltaChunk - 1) / kDeltaChunk;
    const size_t per_state = static_cast<size_t>(z.DK) * z.DV, heads = static_cast<size_t>(z.B) * z.HV;
    const int vblocks = (z.DV + 63) / 64;
    volatile int *dead = &sm.dead;
    const auto chunk_at = [&](int c) { return kRev ? chunks - 1 - c : c; };

    if (tid == 0) {
        sm.dead = 0;
        for (int i = 0; i < 2; ++i) {
            for (uint64_t *p : {&sm.kq_full[i], &sm.kq_empty[i], &sm.v_full[i], &sm.v_empty[i], &sm.t_full[i]})
                mbar_init(p, 1);
            mbar_init(&sm.t_empty[i], 1 + 8 + (kOut ? 4 : 0));  // the last product, the scalars' readers
        }
        for (uint64_t *p : {&sm.z_full, &sm.z_empty, &sm.p_full, &sm.q_full, &sm.x_full, &sm.d_full, &sm.o_full, &sm.drain})
            mbar_init(p, 1);
        for (uint64_t *p : {&sm.r_full, &sm.b_full, &sm.s_full}) mbar_init(p, 256);
        for (uint64_t *p : {&sm.q_read, &sm.m_full, &sm.s_read, &sm.x_free}) mbar_init(p, 128);
        fence_mbar_init();
    }
    if (warp == kLoadWarp + 1) tmem_alloc(&sm.tmem, kTmCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);

    if (warp >= kLoadWarp) {
        regs_down<kMore ? 72 : 88>();
        if (warp == kLoadWarp && lane == 0) {
            // ---- TMA ----
            int nk = 0, nt = 0, nv = 0, nz = 0;  // copies issued
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1, ck = chunk_at(c), t0 = ck * kDeltaChunk;
                const uint32_t free = ((c >> 1) & 1) ^ 1;
                if (ck == a.silent) break;
                if (!mbar_wait_one(&sm.kq_empty[st], free, dead)) break;
                mbar_arrive_expect_tx(&sm.kq_full[st], KSUB * Smem::kBlock);
#pragma unroll
                for (int s = 0; s < KSUB; ++s) {
                    unsigned char *p = sm.kq[st] + s * Smem::kBlock;
                    tma_load_4d(p, &map_k, &sm.kq_full[st], 64 * s, hk, t0, b);
                    if constexpr (kOut) tma_load_4d(p + 8192, &map_q, &sm.kq_full[st], 64 * s, hk, t0, b);
                }
                ++nk;
                if (!mbar_wait_one(&sm.t_empty[st], free, dead)) break;
                mbar_arrive_expect_tx(&sm.t_full[st], Img::kBytes);
                bulk_load(sm.img[st], a.img + (ck * heads + bh) * Img::kBytes, Img::kBytes, &sm.t_full[st]);
                ++nt;
                if (!mbar_wait_one(&sm.v_empty[st], free, dead)) break;
                mbar_arrive_expect_tx(&sm.v_full[st], 8192 * vblocks);
                for (int s = 0; s < vblocks; ++s)
                    tma_load_4d(sm.v[st] + 8192 * s, &map_v, &sm.v_full[st], 64 * s, hv, t0, b);
                ++nv;
                if constexpr (kRev) {
                    if (!mbar_wait_one(&sm.z_empty, (c & 1) ^ 1, dead)) break;
                    mbar_arrive_expect_tx(&sm.z_full, Smem::kImage2);
                    bulk_load(sm.img2, a.img2 + (ck * heads + bh) * Smem::kImage2, Smem::kImage2, &sm.z_full);
                    ++nz;
                }
            }
            // the copies in flight land before the block ends
            const auto drain2 = [&](uint64_t *bar, int n) {
                for (int d = max(0, n - 2); d < n; ++d) mbar_drain(&bar[d & 1], (d >> 1) & 1);
            };
            drain2(sm.kq_full, nk), drain2(sm.t_full, nt), drain2(sm.v_full, nv);
            if (kRev && nz > 0) mbar_drain(&sm.z_full, (nz - 1) & 1);
        } else if (warp == kLoadWarp + 1) {
            // ---- tcgen05.mma ----
            // (the whole warp: see mma_ts)
            const auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, dead); };
            // columns beyond DK are zeros in K's tile and in S: full widths
            constexpr uint32_t i_64 = mma_idesc(64, false);
            constexpr uint32_t i_ds = mma_idesc(64 * KSUB, true);
            // lanes beyond 64 read the one block of a narrow V once more
            const uint32_t v_lbo = vblocks > 1 ? 8192 : 0;
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t half = (c >> 1) & 1, one = c & 1;
                const uint64_t kd = mma_smem_desc(smem_addr(sm.kq[st]), 16, 1024);
                const uint64_t kn = mma_smem_desc(smem_addr(sm.kq[st]), Smem::kBlock, 1024);
                const uint64_t vd = mma_smem_desc(smem_addr(sm.v[st]), v_lbo, 1024);
                const uint64_t td = mma_smem_desc(smem_addr(sm.img[st]), 16, 1024);
                const uint64_t zd = mma_smem_desc(smem_addr(sm.img2), 8192, 1024);
                // x (+)= operand T^T over one part of T, T lower triangular by
                // blocks of 16: forward T's rows are x's steps, and block
                // column k reaches rows 16 k and up; backwards its columns
                // are, and block row k reaches columns up to 16 k + 15
                const auto tri = [&](int k, uint64_t tile, auto &&issue) {
                    if constexpr (kRev)
                        issue(kTmX, desc_at(tile, k * 2048), mma_idesc(16 * (k + 1), true));
                    else
                        issue(kTmX + 16 * k, desc_at(tile, k * 2048 + k * 32), mma_idesc(64 - 16 * k, false));
                };
                const auto step = [](int k) { return kRev ? 3 - k : k; };  // the widest first
                if (!wait(&sm.kq_full[st], half)) break;
                if (!wait(&sm.s_full, one)) break;
                if (c > 0 && !wait(&sm.x_free, one ^ 1)) break;
                tc_fence_after();
                // An addition in the tensor cores cuts its result off, some
                // 4e-8 of it each time and always towards zero: the small
                // parts come first, so that few are made at full size.
                const auto with_state = [&](uint32_t d, uint32_t rows, int parts, uint32_t idesc) {
#pragma unroll
                    for (int p = parts - 1; p >= 0; --p)
#pragma unroll
                        for (int s = 0; s < 4 * KSUB; ++s)
                            mma_ts(tm + d, tm + kTmS + 64 * p + s * 8,
                                   desc_at(kd, rows + (s >> 2) * Smem::kBlock + (s & 3) * 32), idesc,
                                   p < parts - 1 || s > 0);
                };
                if constexpr (kOut && kParts == 2) {  // both at once, [K; Q] as one operand
                    with_state(kTmP, 0, 2, mma_idesc(128, false));
                    mma_commit(&sm.p_full);
                    mma_commit(&sm.q_full);
                } else {
                    with_state(kTmP, 0, kParts, i_64);
                    mma_commit(&sm.p_full);
                    if constexpr (kOut) {  // off the chain: S's first two parts
                        with_state(kTmQ, 8192, 2, i_64);
                        mma_commit(&sm.q_full);
                    }
                }
                // x without the state
                if (!wait(&sm.t_full[st], half)) break;
                if (!wait(&sm.v_full[st], half)) break;
                if constexpr (kRev)
                    if (!wait(&sm.z_full, one)) break;
                const auto base = [&](int p) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = step(j);
                        tri(k, desc_at(kRev ? zd : td, p * kTileBytes), [&](uint32_t d, uint64_t t, uint32_t i) {
                            mma_ss(tm + d, desc_at(vd, k * 2048), t, i | kMmaAmn, p < kParts - 1 || j > 0);
                        });
                    }
                };
#pragma unroll
                for (int p = kParts - 1; p > 0; --p) base(p);
                if (!wait(&sm.r_full, one)) break;
                tc_fence_after();
                // x += (a P) T^T over the part pairs that matter
#pragma unroll
                for (int w = kParts - 1; w >= 0; --w) {
                    if (w == 0) base(0);
#pragma unroll
                    for (int p = 0; p <= w; ++p)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = step(j);
                            tri(k, desc_at(td, (w - p) * kTileBytes), [&](uint32_t d, uint64_t t, uint32_t i) {
                                mma_ts(tm + d, tm + tm_parts(k, p), t, i, true);
                            });
                        }
                }
                if constexpr (!kRev) mma_commit(&sm.v_empty[st]);
                mma_commit(&sm.x_full);
                // the state's increment: K (and scale E Q) with DK as the N index
                if constexpr (kRev) {
#pragma unroll
                    for (int p = 2; p >= 0; --p)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ss(tm + kTmDs, desc_at(vd, k * 2048),
                                   desc_at(zd, (3 + p * KSUB) * kTileBytes + k * 2048), i_ds | kMmaAmn, p < 2 || k > 0);
                    mma_commit(&sm.v_empty[st]);
                    mma_commit(&sm.z_empty);
                }
                if (!wait(&sm.b_full, one)) break;
                if constexpr (kOut)
                    if (!wait(&sm.q_read, one)) break;
                tc_fence_after();
#pragma unroll
                for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(tm + kTmDs, tm + tm_parts(k, p), desc_at(kn, k * 2048), i_ds, kRev || p < kParts - 1 || k > 0);
                mma_commit(&sm.d_full);
                mma_commit(&sm.kq_empty[st]);
                if constexpr (kOut) {  // M r
                    if (!wait(&sm.m_full, one)) break;
                    tc_fence_after();
#pragma unroll
                    for (int w = 1; w >= 0; --w)
#pragma unroll
                        for (int p = 0; p <= w; ++p)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tri(k, desc_at(td, Img::kM + (w - p) * kTileBytes), [&](uint32_t d, uint64_t t, uint32_t i) {
                                    mma_ts(tm + d, tm + kTmR<kParts> + 32 * p + 8 * k, t, i, w == 0 || p + k > 0);
                                });
                    mma_commit(&sm.o_full);
                }
                mma_commit(&sm.t_empty[st]);
            }
            mma_commit(&sm.drain);  // nothing is in flight when tensor memory goes back
            mbar_drain(&sm.drain, 0);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---- the output ----
        regs_down<kMore ? 104 : 120>();
        if constexpr (kOut) {
            const int dv = 32 * (warp & 3) + lane;
            const uint32_t tl = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
            const bool on = dv < z.DV;
            const size_t step = static_cast<size_t>(z.HV) * z.DV;
            int c = 0;
            for (; c < chunks; ++c) {
                const uint32_t half = (c >> 1) & 1, one = c & 1;
                const ChunkScalars &sc = *reinterpret_cast<const ChunkScalars *>(sm.img[c & 1] + Img::kScalars);
                if (!mbar_wait(&sm.t_full[c & 1], half, dead)) break;
                if (!mbar_wait(&sm.q_full, one, dead)) break;
                tc_fence_after();
                float q[32];  // Q S's second half, before the increment takes its place
                tmem_ld32(tl + kTmQ + 32, q);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive(&sm.q_read);
                if (!mbar_wait(&sm.x_full, one, dead)) break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[32];
                    tmem_ld32(tl + kTmX + 32 * h, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        put_parts<2>([&](int p) { return tl + kTmR<kParts> + 32 * p + 8 * (2 * h + e); }, x + 16 * e);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sm.m_full);
                if (!mbar_wait(&sm.o_full, one, dead)) break;
                tc_fence_after();
                uint32_t out[32];
#pragma unroll
                for (int h = 1; h >= 0; --h) {
                    float x[32];
                    tmem_ld32(tl + kTmX + 32 * h, x);
                    if (h == 0) tmem_ld32(tl + kTmQ, q);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {  // the scalars hold -E
                        const int t = 32 * h + 2 * i;
                        out[t / 2] = pack_bf16(a.scale * fmaf(-sc.a[t], q[2 * i], x[2 * i]),
                                               a.scale * fmaf(-sc.a[t + 1], q[2 * i + 1], x[2 * i + 1]));
                    }
                }
                tc_fence_before();
                mbar_arrive(&sm.x_free);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.t_empty[c & 1]);
                const int t0 = c * kDeltaChunk, n = min(kDeltaChunk, z.T - t0);
                if (on) {
                    __nv_bfloat16 *op = a.o + token_offset(b, t0, hv, z.T, z.HV, z.DV) + dv;
                    const auto put = [&](int i) {
                        const __nv_bfloat162 two = *reinterpret_cast<const __nv_bfloat162 *>(&out[i / 2]);
                        op[i * step] = i & 1 ? __high2bfloat16(two) : __low2bfloat16(two);
                    };
                    if (n == kDeltaChunk) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) put(i);
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i < n) put(i);
                    }
                }
            }
            for (int t = c * kDeltaChunk; on && t < z.T; ++t)  // a wait gave up: what is missing becomes NaN
                a.o[token_offset(b, t, hv, z.T, z.HV, z.DV) + dv] = __float2bfloat16_rn(__int_as_float(0x7FC00000));
        } else {
            // what the gradient needs of a sweep: the chunk's first state (its
            // parts' sum) and its x
            const int dv = 32 * (warp & 3) + lane;
            const uint32_t tl = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
            const bool on = dv < z.DV;
            int c = 0;
            for (; c < chunks; ++c) {
                const uint32_t one = c & 1;
                const int ck = chunk_at(c);
                const size_t at = ck * heads + bh;
                float4 *sp = reinterpret_cast<float4 *>(a.states + sweep_at(z, at, z.DK, dv));
                float4 *xp = reinterpret_cast<float4 *>(a.x + sweep_at(z, at, kDeltaChunk, dv));
                if (!mbar_wait(&sm.s_full, one, dead)) break;
                tc_fence_after();
#pragma unroll 1
                for (int h = 0; h < 2 * KSUB; ++h) {
                    uint32_t y[3][16];
#pragma unroll
                    for (int p = 0; p < 3; ++p) tmem_ld16(tl + kTmS + 64 * p + 16 * h, y[p]);
                    tmem_wait_ld();
                    if (h + 1 == 2 * KSUB) {
                        tc_fence_before();
                        mbar_arrive(&sm.s_read);
                    }
                    const auto lo = [&](int i) { return bf16_low(y[0][i]) + (bf16_low(y[1][i]) + bf16_low(y[2][i])); };
                    const auto hi = [&](int i) { return bf16_high(y[0][i]) + (bf16_high(y[1][i]) + bf16_high(y[2][i])); };
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (on && 32 * h + 4 * i < z.DK)
                            sp[(4 * h + i / 2) * (kSweepEight / 4) + i % 2] = make_float4(lo(2 * i), hi(2 * i), lo(2 * i + 1), hi(2 * i + 1));
                }
                if (!mbar_wait(&sm.x_full, one, dead)) break;
                tc_fence_after();
                float x[64];
                tmem_ld32(tl + kTmX, x);
                tmem_ld32(tl + kTmX + 32, x + 32);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive(&sm.x_free);
                if (on) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        xp[(i / 2) * (kSweepEight / 4) + i % 2] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
            }
            for (; on && c < chunks; ++c) {  // a wait gave up: what is missing becomes NaN
                const size_t at = chunk_at(c) * heads + bh;
                const float nan = __int_as_float(0x7FC00000);
                for (int i = 0; i < z.DK; ++i) a.states[sweep_at(z, at, z.DK, dv) + (i >> 3) * kSweepEight + (i & 7)] = nan;
                for (int i = 0; i < kDeltaChunk; ++i)
                    a.x[sweep_at(z, at, kDeltaChunk, dv) + (i >> 3) * kSweepEight + (i & 7)] = nan;
            }
        }
    } else {
        // ---- the chain ----
        regs_up<kMore ? 168 : 152>();
        const int cg = warp >> 2;                    // half of the columns
        const int dv = 32 * (warp & 3) + lane;       // this thread's lane
        const uint32_t tl = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        constexpr int SC = 32 * KSUB;                // state rows (DK) per thread
        const int dk0 = SC * cg;
        const bool on = dv < z.DV;
        float S[SC];
        const float *s_in = a.s_in == nullptr ? nullptr : a.s_in + bh * per_state + dv;
#pragma unroll
        for (int i = 0; i < SC; ++i)
            S[i] = (s_in != nullptr && on && dk0 + i < z.DK) ? s_in[static_cast<size_t>(dk0 + i) * z.DV] : 0.f;
        const auto put_state = [&]() {  // S as an operand
#pragma unroll
            for (int h = 0; h < SC / 16; ++h)
                put_parts<kParts>([&](int p) { return tl + kTmS + 64 * p + (dk0 + 16 * h) / 2; }, &S[16 * h]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sm.s_full);
        };
        const auto keep_state = [&](float *p) {
            if (!on) return;
#pragma unroll
            for (int i = 0; i < SC; ++i)
                if (dk0 + i < z.DK) p[static_cast<size_t>(dk0 + i) * z.DV + dv] = S[i];
        };
        const auto put_steps = [&](const float (&x)[32]) {  // 32 steps as an operand
#pragma unroll
            for (int h = 0; h < 2; ++h)
                put_parts<kParts>([&](int p) { return tl + tm_parts(2 * cg + h, p); }, &x[16 * h]);
            tmem_wait_st();
            tc_fence_before();
        };
        put_state();
        bool ok = true;
        int c = 0;
        for (; c < chunks; ++c) {
            const uint32_t half = (c >> 1) & 1, one = c & 1;
            const ChunkScalars &sc = *reinterpret_cast<const ChunkScalars *>(sm.img[c & 1] + Img::kScalars);
            if (!(ok = mbar_wait(&sm.t_full[c & 1], half, dead))) break;
            if (!(ok = mbar_wait(&sm.p_full, one, dead))) break;
            tc_fence_after();
            float x[32];
            tmem_ld32(tl + kTmP + 32 * cg, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= sc.a[32 * cg + i];
            put_steps(x);
            mbar_arrive(&sm.r_full);
            if (!(ok = mbar_wait(&sm.x_full, one, dead))) break;
            tc_fence_after();
            tmem_ld32(tl + kTmX + 32 * cg, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= sc.b[32 * cg + i];
            put_steps(x);
            mbar_arrive(&sm.b_full);
            if (!(ok = mbar_wait(&sm.d_full, one, dead))) break;
            tc_fence_after();
            const float el = sc.e_last;
#pragma unroll
            for (int h = 0; h < SC / 32; ++h) {
                tmem_ld32(tl + kTmDs + dk0 + 32 * h, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) S[32 * h + i] = fmaf(el, S[32 * h + i], x[i]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.t_empty[c & 1]);  // the scalars are read
            if (c + 1 < chunks) {
                // r's parts lie over S's first one: M r has read them
                if constexpr (kOut && kParts == 3)
                    if (!(ok = mbar_wait(&sm.o_full, one, dead))) break;
                // ... and S is stored
                if constexpr (!kOut)
                    if (!(ok = mbar_wait(&sm.s_read, one, dead))) break;
                tc_fence_after();
                put_state();
            }
        }
        if (!ok) {  // a wait gave up: what is missing becomes NaN
            const float nan = __int_as_float(0x7FC00000);
#pragma unroll
            for (int i = 0; i < SC; ++i) S[i] = nan;
        }
        if (a.s_out != nullptr) keep_state(a.s_out + bh * per_state);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kLoadWarp + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_free(tm, kTmCols);
    }
}

// one block per head
template <int KSUB, int kParts>
__global__ void __launch_bounds__(kChainThreads, 1)
    delta_forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const DeltaChainArgs a) {
    extern __shared__ unsigned char raw[];
    delta_chain<KSUB, kParts, kFwdOut>(map_q, map_k, map_v, a, blockIdx.x, raw);
}

// Both sweeps of the gradient at once, one block per head each: neither needs
// the other, and there are often fewer heads than SMs.
template <int KSUB>
__global__ void __launch_bounds__(kChainThreads, 1)
    delta_sweeps_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ CUtensorMap map_go, const DeltaChainArgs f, const DeltaChainArgs r) {
    extern __shared__ unsigned char raw[];
    const unsigned heads = static_cast<unsigned>(f.z.B) * f.z.HV;
    if (blockIdx.x < heads) delta_chain<KSUB, 3, kFwdStates>(map_k, map_k, map_v, f, blockIdx.x, raw);
    else delta_chain<KSUB, 3, kReverse>(map_k, map_k, map_go, r, blockIdx.x - heads, raw);
}

}  // namespace wkvb
