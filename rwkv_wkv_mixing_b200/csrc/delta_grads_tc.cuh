// Gradients of the gated delta rule within one chunk on the tensor cores, bf16
// I/O: the formulas of delta_grads.cuh, from what the two sweeps left (S0, D1,
// r, du).  One block per chunk and key head, over the value heads that share
// it.
//
// tcgen05 products have 128 rows, a chunk 64 steps: two operands are stacked
// (rows 0-63 and 64-127), so that lane i of tensor memory ends with gq_i and
// lane 64 + i with gk_i:
//
//     R1 = [GO; W] S0^T     R2 = [GO; W] U^T     R3 = [Q; K] K^T
//     R4 = [ ; U] D1^T      [X; -Y] = [scale; -1] tril(A R2)
//     R5 = [X; -Y] K        R6 = [ ; X^T Q - Y^T K]
//     [gq; gk] = [scale E; -E] R1 + R5 + [0; F R4 + R6]
//
// W, U, S0 and D1 are fp32 and enter as three bf16 parts (six part pairs), for
// gg, an fp32 output of many terms; X and Y, which reach only gq and gk, as two.
// The products over DV take 16 columns at a time.  Their operands lie with a
// column (an entry of v) per row: the sweeps, where a lane is such a column,
// leave eight steps or state rows of it side by side, and what a thread
// converts are whole 16-byte pieces of operand; GO's tile is transposed.  A
// slice is copied to shared memory two slices ahead and converted while the
// one before it is multiplied.  16 warps convert and read out; one more copies,
// and one issues, alone so that its descriptors stay in registers.  gv = W goes
// out from the operand itself (its first part is the rounded value), 64 columns
// at a time.
//
// Bound: about 30000 cycles a head and chunk with DK = DV = 128, two thirds the
// eight slices' conversions (1300 cycles) and products (1100), which wait for
// one another, one third the read-out; 30 % of the issue slots, 25 % of the
// tensor cores.  B=2 T=4096, 32 heads of 128: 498 us (fp32 multiply-adds: 2140);
// B=8 T=1024, 12 heads of 64: 142 us (633).
#pragma once

#include "delta_chunk.cuh"

namespace wkvb {

struct DeltaTcGradArgs {
    const float *g, *beta;
    const float *r, *du, *starts, *ends;  // as the sweeps left them (sweep_at)
    __nv_bfloat16 *gq, *gk, *gv;          // gv by its tensor map
    float *gg, *gbeta;
    float scale;
    DeltaSizes z;
    int silent;  // as in DeltaPrepArgs
};

constexpr int kTcWorkers = 512, kTcGradThreads = kTcWorkers + 64;
constexpr int kTcPLd = 65;

constexpr int kTcCols = kSweepCols;  // columns of a slice

// A slice's operands: a row per column, 64 steps (or state rows) per 2 KB.
template <int KSUB>
struct TcTiles {
    unsigned char a[3][4096];         // parts of [GO; W]
    unsigned char u[3][2048];         // of U
    unsigned char s[3][KSUB * 2048];  // of S0
    unsigned char d[3][KSUB * 2048];  // of D1
};

template <int KSUB>
struct TcGradSmem {
    static constexpr int kOcts = 8 * KSUB;  // eights of state rows
    alignas(1024) unsigned char qk[KSUB][16384];  // per 64 columns: 64 rows of Q, 64 of K
    union {
        alignas(1024) TcTiles<KSUB> tiles[2];
        struct {
            alignas(1024) unsigned char xy[2][16384];  // then parts of [X; -Y]
            float p[128 * kTcPLd];                     // and P's sums over j < t
        };
    };
    alignas(1024) unsigned char go[2][8192];  // GO as it is in memory, 64 columns
    alignas(1024) unsigned char gv[8192];     // and gv
    // the next slices, fp32: eights of r, du, S0, D1
    alignas(16) float next[2][2 * 8 + 2 * kOcts][kTcCols][8];
    float ghi[kDeltaChunk], glo[kDeltaChunk], e[kDeltaChunk], f[kDeltaChunk], beta[kDeltaChunk];
    float to_last[kDeltaChunk];         // e^{G_l - G_j}, l the last step of j's sixteen
    float gbeta[kDeltaChunk];
    float rows[4][128], writes[4][64];  // the steps' terms with S0 and with D1, by quarter of the columns
    float p_quarter[3][128];            // P's sums over 16 columns
    float sums[8][kDeltaChunk];
    float part[kTcWorkers / 32];
    float e_last;
    uint64_t tile, full[2], ready[2], done[2], ready_xy, done_xy, drain;
    uint32_t tmem;
    int dead;
};

// Eight steps or state rows of one column
__device__ __forceinline__ void load_eight(const float (&p)[8], bool on, float (&x)[8]) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
    if (on) v = *reinterpret_cast<const float4 *>(&p[0]), w = *reinterpret_cast<const float4 *>(&p[4]);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
}
// ... and as operand parts: 16-byte piece c of row `row` of tiles `stride` apart
__device__ __forceinline__ void put_eight(unsigned char *tile, uint32_t stride, int row, int c, const float (&x)[8]) {
    uint32_t y[4][3];
#pragma unroll
    for (int q = 0; q < 4; ++q) split_bf16<3>(x[2 * q], x[2 * q + 1], y[q]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
        *reinterpret_cast<uint4 *>(tile + p * stride + swz128(row, c)) = make_uint4(y[0][p], y[1][p], y[2][p], y[3][p]);
}
// Eight values of every lane summed over half a warp: lane l ends with value
// (l >> 1) & 7's sum, two lanes each.
__device__ __forceinline__ float sum_eight(const float (&x)[8], int lane) {
    const bool b3 = lane & 8, b2 = lane & 4, b1 = lane & 2;
    float y[4], z[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (b3 ? x[4 + i] : x[i]) + __shfl_xor_sync(0xffffffffu, b3 ? x[i] : x[4 + i], 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) z[i] = (b2 ? y[2 + i] : y[i]) + __shfl_xor_sync(0xffffffffu, b2 ? y[i] : y[2 + i], 4);
    const float s = (b1 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, b1 ? z[0] : z[1], 2);
    return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

template <int KSUB>
__global__ void __launch_bounds__(kTcGradThreads, 1)
    delta_grads_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_go, const __grid_constant__ CUtensorMap map_gv,
                          const DeltaTcGradArgs a) {
    using Smem = TcGradSmem<KSUB>;
    extern __shared__ unsigned char raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    constexpr uint32_t kR1 = 0, kR2 = 128, kR3 = 192, kR6 = 128, kR4 = 256, kR5 = 384;
    const DeltaSizes &z = a.z;
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int heads = z.B * z.HV;
    const unsigned bk = blockIdx.x % (static_cast<unsigned>(z.B) * z.HK);
    const int chunk = static_cast<int>(blockIdx.x / (static_cast<unsigned>(z.B) * z.HK));
    const int b = static_cast<int>(bk / z.HK), hk = static_cast<int>(bk % z.HK);
    const int t0 = chunk * kDeltaChunk, n = min(kDeltaChunk, z.T - t0);
    const int slices = (z.DV + kTcCols - 1) / kTcCols, vblocks = (slices + 3) / 4;
    volatile int *dead = &sm.dead;

    if (tid == 0) {
        sm.dead = 0;
        for (uint64_t *p : {&sm.tile, &sm.full[0], &sm.full[1], &sm.done[0], &sm.done[1], &sm.done_xy, &sm.drain})
            mbar_init(p, 1);
        for (uint64_t *p : {&sm.ready[0], &sm.ready[1], &sm.ready_xy}) mbar_init(p, kTcWorkers);
        fence_mbar_init();
        mbar_arrive_expect_tx(&sm.tile, KSUB * 16384);
#pragma unroll
        for (int s = 0; s < KSUB; ++s) {
            tma_load_4d(sm.qk[s], &map_q, &sm.tile, 64 * s, hk, t0, b);
            tma_load_4d(sm.qk[s] + 8192, &map_k, &sm.tile, 64 * s, hk, t0, b);
        }
    }
    if (warp == 0) tmem_alloc(&sm.tmem, 512);
    // GO has one part: its half of the others is zero
    const auto clear = [&]() {
        static_assert(kTcWorkers == 512, "two tiles, two parts, 128 pieces");
        reinterpret_cast<uint4 *>(sm.tiles[tid >> 8].a[1 + (tid >> 7 & 1)])[tid & 127] = make_uint4(0, 0, 0, 0);
    };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);

    // this thread's lane of tensor memory and quarter of the columns
    const int cg = warp >> 2, row = 32 * (warp & 3) + lane, i = row & 63;
    const bool low = row < 64;
    const uint32_t tl = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    constexpr int kC = 16 * KSUB;
    float acc[kC] = {};  // gq or gk, columns kC cg ..
    // Starts the copies of slice q (counted over the heads), in one thread: few
    // and large, since each takes some 200 cycles to issue.
    const auto fetch = [&](int q) {
        const int gh = q / slices, sl = q % slices;
        const int hv = hk * z.group + gh, col = kTcCols * sl;
        const size_t at = static_cast<size_t>(chunk) * heads + b * z.HV + hv;
        const size_t step = sweep_at(z, at, kDeltaChunk, col), state = sweep_at(z, at, z.DK, col);
        const uint32_t steps = kDeltaChunk * kTcCols * 4, states = z.DK * kTcCols * 4;
        uint64_t *full = &sm.full[q & 1];
        mbar_arrive_expect_tx(full, 2 * (steps + states) + (sl % 4 == 0 ? 8192 : 0));
        if (sl % 4 == 0) tma_load_4d(sm.go[(gh * vblocks + sl / 4) & 1], &map_go, full, col, hv, t0, b);
        bulk_load(sm.next[q & 1][0], a.r + step, steps, full);
        bulk_load(sm.next[q & 1][8], a.du + step, steps, full);
        bulk_load(sm.next[q & 1][16], a.starts + state, states, full);
        bulk_load(sm.next[q & 1][16 + Smem::kOcts], a.ends + state, states, full);
    };
    if (warp == kTcWorkers / 32) {
        // ---- products ----
        // of one slice
        const auto issue = [&](TcTiles<KSUB> &t, bool first) {
            constexpr uint32_t i_s = mma_idesc(64 * KSUB, true) | kMmaAmn, i_64 = mma_idesc(64, true) | kMmaAmn;
            const uint64_t ad = mma_smem_desc(smem_addr(t.a), 2048, 1024);
            const uint64_t ud = mma_smem_desc(smem_addr(t.u), 2048, 1024);
            // U as rows 64 .. 127: what lies 2 KB before it gives the products of
            // lanes that nothing reads
            const uint64_t uh = mma_smem_desc(smem_addr(t.u) - 2048, 2048, 1024);
            const uint64_t sd = mma_smem_desc(smem_addr(t.s), 2048, 1024);
            const uint64_t dd = mma_smem_desc(smem_addr(t.d), 2048, 1024);
#pragma unroll
            for (int w = 2; w >= 0; --w)  // the small pairs first (delta_chunk.cuh)
#pragma unroll
                for (int p = 0; p <= w; ++p) {
                    const bool add = !first || w < 2 || p > 0;
                    mma_ss(tm + kR2, desc_at(ad, p * 4096), desc_at(ud, (w - p) * 2048), i_64, add);
                    mma_ss(tm + kR1, desc_at(ad, p * 4096), desc_at(sd, (w - p) * KSUB * 2048), i_s, add);
                    mma_ss(tm + kR4, desc_at(uh, p * 2048), desc_at(dd, (w - p) * KSUB * 2048), i_s, add);
                }
            if (first) {
                const uint64_t qd = mma_smem_desc(smem_addr(sm.qk), 16, 1024);
#pragma unroll
                for (int s = 0; s < 4 * KSUB; ++s) {
                    const uint32_t o = (s >> 2) * 16384 + (s & 3) * 32;
                    mma_ss(tm + kR3, desc_at(qd, o), desc_at(qd, o + 8192), mma_idesc(64, false), s > 0);
                }
            }
        };
        const auto wait = [&](uint64_t *bar, int n) { return mbar_wait(bar, n & 1, dead); };
        bool on = wait(&sm.tile, 0);
        int q = 0;
        for (int gh = 0; on && gh < z.group; ++gh) {
            for (int sl = 0; on && sl < slices; ++sl, ++q) {
                on = wait(&sm.ready[q & 1], q >> 1);
                tc_fence_after();
                if (q & 1) issue(sm.tiles[1], sl == 0);
                else issue(sm.tiles[0], sl == 0);
                mma_commit(&sm.done[q & 1]);
            }
            on = on && wait(&sm.ready_xy, gh);
            tc_fence_after();
            {
                    constexpr uint32_t i_k = mma_idesc(64 * KSUB, true);
                    const uint64_t xd = mma_smem_desc(smem_addr(sm.xy), 16, 1024);
                    const uint64_t qn = mma_smem_desc(smem_addr(sm.qk), 16384, 1024);
                    const uint64_t kn = desc_at(qn, 8192);
                    // transposed, X and -Y are lanes 64 .. 127 and what lies 8 KB
                    // before them the unread ones
                    const uint64_t xt = mma_smem_desc(smem_addr(sm.xy) - 8192, 8192, 1024);
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_ss(tm + kR5, desc_at(xd, p * 16384 + k * 32), desc_at(kn, k * 2048), i_k, p + k > 0);
                            mma_ss(tm + kR6, desc_at(xt, p * 16384 + k * 2048), desc_at(qn, k * 2048), i_k | kMmaAmn, p + k > 0);
                            mma_ss(tm + kR6, desc_at(xt, p * 16384 + 8192 + k * 2048), desc_at(kn, k * 2048), i_k | kMmaAmn, true);
                        }
            }
            mma_commit(&sm.done_xy);
        }
        // what is in flight ends before the block does
        mma_commit(&sm.drain);
        mbar_drain(&sm.drain, 0);
        __syncwarp();
    } else if (warp == kTcWorkers / 32 + 1) {
        // ---- copies ----
        const int all = chunk == a.silent ? 0 : z.group * slices;
        int q = 0;
        if (lane == 0) {
            for (; q < min(all, 2); ++q) fetch(q);
            for (; q < all; ++q) {
                if (!mbar_wait_one(&sm.ready[q & 1], ((q - 2) >> 1) & 1, dead)) break;
                fetch(q);
            }
            mbar_drain(&sm.tile, 0);
            for (int d = max(0, q - 2); d < q; ++d) mbar_drain(&sm.full[d & 1], (d >> 1) & 1);
        }
        __syncwarp();
    } else {
    const auto sync = [] { named_bar_sync(1, kTcWorkers); };
    int q = 0;  // slices so far
    // (a wait that gives up leaves `dead` set: the outputs become NaN at the end)
    mbar_wait(&sm.tile, 0, dead);
    for (int gh = 0; gh < z.group; ++gh) {
        const int hv = hk * z.group + gh;
        sync();  // the last head's shared values are read
        clear();
        if (warp == 0) {
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
                sm.to_last[t] = expf(static_cast<float>(__shfl_sync(0xffffffffu, d[1], lane | 7) - d[e]));
            }
            if (lane == 0) sm.e_last = expf(static_cast<float>(last));
        }
        sync();
        float inner = 0.f, gbeta = 0.f;  // <D1, S0>; du.r of one step (warps 0-3)
#pragma unroll 1
        for (int sl = 0; sl < slices; ++sl, ++q) {
            TcTiles<KSUB> &tl_ = sm.tiles[q & 1];
            const float(&next)[2 * 8 + 2 * Smem::kOcts][kTcCols][8] = sm.next[q & 1];
            mbar_wait(&sm.full[q & 1], (q >> 1) & 1, dead);
            if (q >= 2) mbar_wait(&sm.done[q & 1], ((q - 2) >> 1) & 1, dead);  // the tiles are read
            // half a warp takes the 16 columns of eight steps of r and du
            // (warps 0-3) or of eight rows of S0 and D1 (8-15); 4-7 take GO
            const int c = lane & 15, half = lane >> 4, col = kTcCols * sl + c;
            const bool in = col < z.DV;
            if (warp < 4) {
                // W of two slices ago has also gone out (before its readers' next arrival)
                if (q >= 2) mbar_wait(&sm.ready[(q - 1) & 1], ((q - 1) >> 1) & 1, dead);
                const int oct = 2 * warp + half;
                float x[8], y[8], dot[8];
                load_eight(next[oct][c], in, x);
                load_eight(next[8 + oct][c], in, y);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float bt = sm.beta[8 * oct + t];
                    dot[t] = x[t] * y[t];
                    x[t] *= bt;
                    y[t] *= bt;
                }
                put_eight(tl_.u[0], 2048, c, oct, x);
                put_eight(tl_.a[0] + 2048, 4096, c, oct, y);
                gbeta += sum_eight(dot, lane);
            } else if (warp < 8) {
                // transposed: 8 columns and 32 steps (four 8 x 8 blocks) a warp
                const int w = warp - 4;
                uint32_t g[4];
                ldmatrix4_trans(smem_addr(sm.go[(gh * vblocks + sl / 4) & 1]) +
                                    swz128(32 * (w >> 1) + lane, 2 * (sl & 3) + (w & 1)), g);
                stmatrix4(smem_addr(tl_.a[0]) + swz128(8 * (w & 1) + (lane & 7), 4 * (w >> 1) + (lane >> 3)), g);
            } else if (warp < 8 + 4 * KSUB) {
                const int oct = 2 * (warp - 8) + half;
                const bool on = in && 8 * oct < z.DK;
                float x[8], y[8];
                load_eight(next[16 + oct][c], on, x);
                load_eight(next[16 + Smem::kOcts + oct][c], on, y);
#pragma unroll
                for (int t = 0; t < 8; ++t) inner = fmaf(x[t], y[t], inner);
                put_eight(tl_.s[0] + (oct >> 3) * 2048, KSUB * 2048, c, oct & 7, x);
                put_eight(tl_.d[0] + (oct >> 3) * 2048, KSUB * 2048, c, oct & 7, y);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&sm.ready[q & 1]);
            if (warp >= 4 && warp < 8) {  // gv = W, transposed back
                const int w = warp - 4;
                mbar_wait(&sm.ready[q & 1], (q >> 1) & 1, dead);
                if (sl % 4 == 0) {  // the tile has left
                    if (warp == 4 && lane == 0) bulk_wait_read_all();
                    named_bar_sync(2, 128);
                }
                uint32_t g[4];
                // 16 steps of the 16 columns a warp
                ldmatrix4_trans(smem_addr(tl_.a[0]) + 2048 +
                                    swz128((lane & 7) + 8 * (lane >> 4), 2 * w + ((lane >> 3) & 1)), g);
                stmatrix4(smem_addr(sm.gv) + swz128(16 * w + (lane & 15), 2 * (sl & 3) + (lane >> 4)), g);
                if (sl % 4 == 3 || sl + 1 == slices) {
                    fence_proxy_async_smem();
                    named_bar_sync(2, 128);
                    if (warp == 4 && lane == 0) {
                        tma_store_4d(&map_gv, sm.gv, 64 * (sl / 4), hv, t0, b);
                        bulk_commit();
                    }
                }
            }
        }
        if (warp < 4 && (lane & 1) == 0) sm.gbeta[8 * (2 * warp + (lane >> 4)) + ((lane >> 1) & 7)] = gbeta;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, s);
        if (lane == 0) sm.part[warp] = inner;
        if (q >= 2) mbar_wait(&sm.done[q & 1], ((q - 2) >> 1) & 1, dead);
        mbar_wait(&sm.done[(q - 1) & 1], ((q - 1) >> 1) & 1, dead);
        tc_fence_after();
        sync();  // gv's senders have read the last W, too
        // X, -Y and P: row i of 64, columns 16 cg ..
        {
            float x[16], y[16];
            tmem_ld16(tl + kR2 + 16 * cg, x);
            tmem_ld16(tl + kR3 + 16 * cg, y);
            tmem_wait_ld();
            const float hi = sm.ghi[i], lo = sm.glo[i], f = low ? a.scale : -1.f;
            float sum = 0.f;
            const int first = i & 32, c0 = 16 * cg;  // of the warp's 32 steps, and of the columns
            if (first + 31 < c0) {  // above the diagonal (warp-uniform)
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = 0.f, sm.p[row * kTcPLd + c0 + e] = 0.f;
            } else if (first >= c0 + 16) {  // left of it: e^{G_i - G_l} e^{G_l - G_j}
                const float fi = f * expf((hi - sm.ghi[c0 + 15]) + (lo - sm.glo[c0 + 15]));
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[e] *= fi * sm.to_last[c0 + e];
                    sm.p[row * kTcPLd + c0 + e] = sum;
                    sum = fmaf(x[e], y[e], sum);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = c0 + e;
                    const bool in = low ? i >= j : i > j;
                    x[e] = in ? f * expf((hi - sm.ghi[j]) + (lo - sm.glo[j])) * x[e] : 0.f;
                    sm.p[row * kTcPLd + j] = sum;
                    sum += i > j ? x[e] * y[e] : 0.f;
                }
            }
            if (cg < 3) sm.p_quarter[cg][row] = sum;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t o[4][2];
#pragma unroll
                for (int q = 0; q < 4; ++q) split_bf16<2>(x[8 * c + 2 * q], x[8 * c + 2 * q + 1], o[q]);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    *reinterpret_cast<uint4 *>(sm.xy[p] + swz128(row, 2 * cg + c)) =
                        make_uint4(o[0][p], o[1][p], o[2][p], o[3][p]);
            }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sm.ready_xy);
        sync();
        // meanwhile P's columns: eight threads per step
        {
            const int t = tid & 63, q = tid >> 6;
            float s = 0.f;
#pragma unroll
            for (int r = 16 * q; r < 16 * q + 16; ++r) {
                float p = sm.p[r * kTcPLd + t];
#pragma unroll
                for (int c = 0; c < 3; ++c) p += t >= 16 * (c + 1) ? sm.p_quarter[c][r] : 0.f;
                s += (r & 63) >= t ? p : 0.f;
            }
            sm.sums[q][t] = s;
        }
        mbar_wait(&sm.done_xy, gh & 1, dead);
        tc_fence_after();
        // gq and gk, and their terms' products with q and k
        {
            const float f1 = low ? a.scale * sm.e[i] : -sm.e[i], f4 = sm.f[i];
            float read = 0.f, write = 0.f;
#pragma unroll
            for (int h = 0; h < KSUB; ++h) {
                const int c0 = kC * cg + 16 * h;
                float x[16], y[16];
                uint32_t kv[8];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        sm.qk[c0 >> 6] + (low ? 0 : 8192) + swz128(i, ((c0 & 63) >> 3) + c));
                    kv[4 * c] = v.x, kv[4 * c + 1] = v.y, kv[4 * c + 2] = v.z, kv[4 * c + 3] = v.w;
                }
                const auto k = [&](int e) { return e & 1 ? bf16_high(kv[e / 2]) : bf16_low(kv[e / 2]); };
                tmem_ld16(tl + kR1 + c0, x);
                tmem_ld16(tl + kR5 + c0, y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[e] *= f1;
                    read = fmaf(k(e), x[e], read);
                    acc[16 * h + e] += x[e] + y[e];
                }
                if (!low) {  // warp-uniform
                    tmem_ld16(tl + kR4 + c0, x);
                    tmem_ld16(tl + kR6 + c0, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        x[e] *= f4;
                        write = fmaf(k(e), x[e], write);
                        acc[16 * h + e] += x[e] + y[e];
                    }
                }
            }
            sm.rows[cg][row] = read;
            if (!low) sm.writes[cg][i] = write;
        }
        tc_fence_before();
        sync();
        if (warp == 0) {  // two steps per lane
            float inner_sum = lane < kTcWorkers / 32 ? sm.part[lane] : 0.f;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) inner_sum += __shfl_xor_sync(0xffffffffu, inner_sum, s);
            float w[2], r[2], s[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                w[e] = (sm.writes[0][t] + sm.writes[1][t]) + (sm.writes[2][t] + sm.writes[3][t]);
                r[e] = ((sm.rows[0][t] + sm.rows[1][t]) + (sm.rows[2][t] + sm.rows[3][t])) +
                       ((sm.rows[0][64 + t] + sm.rows[1][64 + t]) + (sm.rows[2][64 + t] + sm.rows[3][64 + t]));
                s[e] = ((sm.sums[0][t] + sm.sums[1][t]) + (sm.sums[2][t] + sm.sums[3][t])) +
                       ((sm.sums[4][t] + sm.sums[5][t]) + (sm.sums[6][t] + sm.sums[7][t]));
            }
            // sums over the writes before and the reads from a step on
            float before = w[0] + w[1], from = r[0] + r[1];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float x = __shfl_up_sync(0xffffffffu, before, d), y = __shfl_down_sync(0xffffffffu, from, d);
                if (lane >= d) before += x;
                if (lane + d < 32) from += y;
            }
            before = __shfl_up_sync(0xffffffffu, before, 1);
            if (lane == 0) before = 0.f;
            const float last = sm.e_last * inner_sum;
            const float after = __shfl_down_sync(0xffffffffu, from, 1);
            const float reads[2] = {from, r[1] + (lane < 31 ? after : 0.f)};
            const float writes[2] = {before, before + w[0]};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                if (t >= n) continue;
                const size_t o = (static_cast<size_t>(b) * z.T + t0 + t) * z.HV + hv;
                a.gg[o] = last + reads[e] + writes[e] + s[e];
                a.gbeta[o] = sm.gbeta[t];
            }
        }
    }
    if (i < n) {
        __nv_bfloat16 *p = (low ? a.gq : a.gk) + token_offset(b, t0 + i, hk, z.T, z.HK, z.DK);
#pragma unroll
        for (int c = 0; c < kC / 8; ++c) {
            const int col = kC * cg + 8 * c;
            if (col >= z.DK) continue;
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = pack_bf16(acc[8 * c + 2 * q], acc[8 * c + 2 * q + 1]);
            *reinterpret_cast<uint4 *>(p + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    if (warp == 4 && lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (*dead) {  // a wait gave up: everything of this block becomes NaN
        const float nan = __int_as_float(0x7FC00000);
        for (int e = tid; e < n * z.DK; e += kTcGradThreads) {
            const size_t o = token_offset(b, t0 + e / z.DK, hk, z.T, z.HK, z.DK) + e % z.DK;
            from_f32(a.gq + o, nan);
            from_f32(a.gk + o, nan);
        }
        // the value heads of a key head are neighbours
        for (long long e = tid; e < static_cast<long long>(n) * z.group; e += kTcGradThreads) {
            const size_t o = token_offset(b, t0 + static_cast<int>(e / z.group),
                                          hk * z.group + static_cast<int>(e % z.group), z.T, z.HV, 1);
            a.gg[o] = a.gbeta[o] = nan;
            for (int i = 0; i < z.DV; ++i) from_f32(a.gv + o * z.DV + i, nan);
        }
    }
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_free(tm, 512);
    }
}

}  // namespace wkvb
