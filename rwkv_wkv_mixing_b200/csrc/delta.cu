// C entry points of the gated delta rule: argument checks, the choice of
// kernel and its launches.  The declarations and their contracts are in
// include/wkv_b200.h.
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "delta_chunk.cuh"
#include "delta_grads.cuh"
#include "delta_grads_tc.cuh"
#include "delta_recurrent.cuh"
#include "host_checks.cuh"

using namespace wkvb;

namespace {

using bf16 = __nv_bfloat16;

// ---- test hook (see gated_delta_set_fault_injection) ----
std::atomic<int> g_fault_kernel{0}, g_fault_chunk{0};

int silent_chunk(int kernel) { return g_fault_kernel.load() == kernel ? g_fault_chunk.load() : -1; }

wkv_status check_delta(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK, int64_t DV,
                       bool *empty) {
    if (B < 0 || T < 0 || HK < 0 || HV < 0 || DK < 0 || DV < 0)
        return fail(WKV_ERR_INVALID_ARG,
                    "negative size (B=%lld T=%lld HK=%lld HV=%lld DK=%lld DV=%lld)",
                    static_cast<long long>(B), static_cast<long long>(T),
                    static_cast<long long>(HK), static_cast<long long>(HV),
                    static_cast<long long>(DK), static_cast<long long>(DV));
    if (HK == 0 ? HV != 0 : HV % HK != 0)
        return fail(WKV_ERR_INVALID_ARG, "HK must divide HV (HK=%lld HV=%lld)",
                    static_cast<long long>(HK), static_cast<long long>(HV));
    if (DK > kDeltaMaxDim || DV > kDeltaMaxDim)
        return fail(WKV_ERR_INVALID_ARG, "DK and DV are at most %d", kDeltaMaxDim);
    // T may be 0: the state passes through
    *empty = B == 0 || HV == 0 || DK == 0 || DV == 0;
    if (*empty) return WKV_OK;
    if (T > INT32_MAX - kDeltaChunk || B > INT32_MAX || HV > INT32_MAX)
        return fail(WKV_ERR_INVALID_ARG, "each of B, T, HV must be below 2^31 - %d", kDeltaChunk);
    // blocks of one launch: at most 8 column blocks, twice, or one per chunk,
    // per head (narrow ones only while they are few)
    const unsigned __int128 heads = static_cast<unsigned __int128>(B) * HV;
    if (heads * 16 > INT32_MAX || heads * ((T + kDeltaChunk - 1) / kDeltaChunk) > INT32_MAX)
        return fail(WKV_ERR_INVALID_ARG, "problem too large for one launch");
    return WKV_OK;
}

DeltaSizes sizes(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK, int64_t DV) {
    return {static_cast<int>(B),  static_cast<int>(T),  static_cast<int>(HK), static_cast<int>(HV),
            static_cast<int>(DK), static_cast<int>(DV), static_cast<int>(HV / HK)};
}

// How the recurrent kernels spread a head's columns: warps per block and
// columns per lane (a warp has four times as many).  Warps of one head in one
// block share its staged q and k; while there are fewer warps than SM
// sub-partitions, one-warp blocks spread them over more SMs (the staged rows
// then come from L2 several times).  Long fp32 sequences take warps of a
// quarter of the columns as long as these are few enough not to wait for one
// another: B=3 T=777, 6 heads of 96 x 80 166 against 284 us; B=4 T=2048, 8
// heads of 128 545 against 816 us.  (A few steps are bound by the state's
// loads, whose rows would be 16 bytes wide.)
enum class RecShape { kWide, kOne, kNarrow, kNarrowFour };

RecShape recurrent_shape(const DeltaSizes &z, int sms, size_t elem_bytes) {
    const int64_t warps = static_cast<int64_t>(z.B) * z.HV * ((z.DV + 15) / 16);
    if (elem_bytes == 4 && z.T > 16 && warps <= 4 * static_cast<int64_t>(sms))
        return warps <= sms ? RecShape::kNarrow : RecShape::kNarrowFour;
    return warps <= 2 * static_cast<int64_t>(sms) || z.DV <= 16 ? RecShape::kOne : RecShape::kWide;
}

unsigned recurrent_grid(const DeltaSizes &z, int cols) {
    return static_cast<unsigned>(static_cast<int64_t>(z.B) * z.HV * ((z.DV + cols - 1) / cols));
}

// launch(warps per block, columns per lane) of the problem's shape
template <typename IO, typename Launch>
wkv_status with_shape(const DeltaSizes &z, int sms, const Launch &launch) {
    cudaGetLastError();
    switch (recurrent_shape(z, sms, sizeof(IO))) {
        case RecShape::kWide: launch(std::integral_constant<int, 4>(), std::integral_constant<int, 4>()); break;
        case RecShape::kOne: launch(std::integral_constant<int, 1>(), std::integral_constant<int, 4>()); break;
        default:
            if constexpr (sizeof(IO) == 4) {
                if (recurrent_shape(z, sms, sizeof(IO)) == RecShape::kNarrow)
                    launch(std::integral_constant<int, 1>(), std::integral_constant<int, 1>());
                else
                    launch(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
            }
    }
    return launched();
}

// A lane holds 8, 12 or 16 rows of the state, for heads of at most 64, 96 and 128
// rows.  (What 12 save against 16: one token of 512 heads of 96 x 96 10.1 against
// 11.1 us, 24 steps of 256 heads in bf16 22.6 against 27.4, 400 in fp32 287
// against 352.)
template <typename IO>
wkv_status launch_recurrent(const DeltaFwdArgs<IO> &a, int sms, cudaStream_t s) {
    return with_shape<IO>(a.z, sms, [&](auto nw, auto cpl) {
        constexpr int NW = decltype(nw)::value, CPL = decltype(cpl)::value;
        const unsigned grid = recurrent_grid(a.z, 4 * CPL * NW);
        if (a.z.DK <= 64) delta_recurrent_kernel<IO, 8, NW, CPL><<<grid, 32 * NW, 0, s>>>(a);
        else if (a.z.DK <= 96) delta_recurrent_kernel<IO, 12, NW, CPL><<<grid, 32 * NW, 0, s>>>(a);
        else delta_recurrent_kernel<IO, 16, NW, CPL><<<grid, 32 * NW, 0, s>>>(a);
    });
}

template <typename IO>
wkv_status launch_recurrent_sweeps(const DeltaFwdArgs<IO> &f, const DeltaRevArgs<IO> &r, int sms, cudaStream_t s) {
    return with_shape<IO>(f.z, sms, [&](auto nw, auto cpl) {
        constexpr int NW = decltype(nw)::value, CPL = decltype(cpl)::value;
        const unsigned grid = 2 * recurrent_grid(f.z, 4 * CPL * NW);
        if (f.z.DK <= 64) delta_recurrent_sweeps_kernel<IO, 8, NW, CPL><<<grid, 32 * NW, 0, s>>>(f, r);
        else if (f.z.DK <= 96) delta_recurrent_sweeps_kernel<IO, 12, NW, CPL><<<grid, 32 * NW, 0, s>>>(f, r);
        else delta_recurrent_sweeps_kernel<IO, 16, NW, CPL><<<grid, 32 * NW, 0, s>>>(f, r);
    });
}

// ---- the chunked kernels --------------------------------------------------------
// A tensor map of a [B, T, H, D] bf16 tensor: boxes of 64 columns of one head
// over 64 steps; steps and columns beyond the tensor read as zero.
bool make_map(CUtensorMap *m, const void *p, const DeltaSizes &z, int H, int D) {
    const Driver &d = driver();
    if (d.encode_tiled == nullptr) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                          static_cast<cuuint64_t>(z.T), static_cast<cuuint64_t>(z.B)};
    cuuint64_t strides[3] = {row, row * H, row * H * z.T};
    cuuint32_t boxes[4] = {64, 1, kDeltaChunk, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return d.encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides,
                          boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 calls take the chunked kernels where a tensor map describes their
// tensors (bases and rows of multiples of 16 bytes).
bool chunked_sizes(int64_t T, int64_t HV, int64_t DK, int64_t DV, int elem_bytes) {
    return elem_bytes == 2 && DK % 8 == 0 && DV % 8 == 0 &&
           static_cast<unsigned __int128>(T) * HV * 256 < (static_cast<unsigned __int128>(1) << 40);
}

bool chunked_fits(const DeltaSizes &z, const void *q, const void *k, const void *v) {
    return chunked_sizes(z.T, z.HV, z.DK, z.DV, 2) && aligned(q, 16) && aligned(k, 16) && aligned(v, 16) &&
           driver().encode_tiled != nullptr;
}

// The forward does from some steps on: its two launches cost a few tens of
// steps.  Up to as many heads as SMs, chunked against step by step: 4 heads of
// 64, 16 and 14 us at 24 steps, 16 and 19 at 33; 32 heads of 128, 20 and 15, 20
// and 20, and 20 and 25 at 48.  With more heads a chunk's latency counts several
// times, the steps' too where a state is wide: 512 heads of 128, 65 and 66 us at
// 33 steps, 68 and 103 at 56; of 72 x 104, 53 and 53 at 33.  States of at most 64
// columns go on step by step for longer: 256 heads of 64, 27 and 28 at 48 steps;
// 512 heads, 43 and 36 at 48, 40 and 47 at 64; of 128 x 64, 55 and 58 at 56.
//
// The gradient does at any length: 34 against 39 us at one step of 4 heads of
// 64, 44 against 80 of 32 heads of 128, 421 against 521 of 2048 heads of 64 (41
// against 40 of 128 heads of 64 is the worst), and the more the longer.
bool chunked_forward(int64_t B, int64_t T, int64_t HV, int64_t DK, int64_t DV, int elem_bytes) {
    return T > (B * HV <= 148 || DV > 64 ? 32 : 56) && chunked_sizes(T, HV, DK, DV, elem_bytes);
}

size_t chunk_count(int64_t T) { return static_cast<size_t>((T + kDeltaChunk - 1) / kDeltaChunk); }

template <int KSUB, int kParts, bool kGrad>
wkv_status launch_prep(const DeltaPrepArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, int dev,
                       cudaStream_t s) {
    auto kern = delta_prep_kernel<KSUB, kParts, kGrad>;
    constexpr size_t smem = sizeof(PrepSmem<KSUB, kGrad>);
    static std::atomic<uint64_t> configured{0};
    const wkv_status st = allow_smem(kern, smem, dev, configured);
    if (st != WKV_OK) return st;
    cudaGetLastError();
    kern<<<static_cast<unsigned>(chunk_count(a.z.T) * a.z.B * a.z.HV), 128, smem, s>>>(mq, mk, a);
    return launched();
}

template <int KSUB, int kParts>
wkv_status launch_forward(const DeltaPrepArgs &p, const DeltaChainArgs &a, const CUtensorMap (&m)[3], int dev,
                          cudaStream_t s) {
    wkv_status st = launch_prep<KSUB, kParts, false>(p, m[0], m[1], dev, s);
    if (st != WKV_OK) return st;
    auto kern = delta_forward_kernel<KSUB, kParts>;
    constexpr size_t smem = sizeof(ChainSmem<KSUB, kParts, kFwdOut>) + 1024;
    static_assert(smem <= 232448, "shared memory of one block");
    static std::atomic<uint64_t> configured{0};
    if ((st = allow_smem(kern, smem, dev, configured)) != WKV_OK) return st;
    kern<<<static_cast<unsigned>(a.z.B) * a.z.HV, kChainThreads, smem, s>>>(m[0], m[1], m[2], a);
    return launched();
}

template <int KSUB>
wkv_status launch_gradient(const DeltaPrepArgs &p, const DeltaChainArgs &f, const DeltaChainArgs &r,
                           const DeltaTcGradArgs &g, const CUtensorMap (&m)[5], int dev, cudaStream_t s) {
    wkv_status st = launch_prep<KSUB, 3, true>(p, m[0], m[1], dev, s);
    if (st != WKV_OK) return st;
    auto kern = delta_sweeps_kernel<KSUB>;
    constexpr size_t smem =
        std::max(sizeof(ChainSmem<KSUB, 3, kFwdStates>), sizeof(ChainSmem<KSUB, 3, kReverse>)) + 1024;
    static_assert(smem <= 232448, "shared memory of one block");
    static std::atomic<uint64_t> configured{0};
    if ((st = allow_smem(kern, smem, dev, configured)) != WKV_OK) return st;
    kern<<<2u * static_cast<unsigned>(f.z.B) * f.z.HV, kChainThreads, smem, s>>>(m[1], m[2], m[3], f, r);
    auto grads = delta_grads_tc_kernel<KSUB>;
    constexpr size_t smem_g = sizeof(TcGradSmem<KSUB>) + 1024;
    static_assert(smem_g <= 232448, "shared memory of one block");
    static std::atomic<uint64_t> configured_g{0};
    if ((st = allow_smem(grads, smem_g, dev, configured_g)) != WKV_OK) return st;
    grads<<<static_cast<unsigned>(chunk_count(g.z.T) * g.z.B * g.z.HK), kTcGradThreads, smem_g, s>>>(m[0], m[1], m[3], m[4], g);
    return launched();
}

// the forward's scratch: one image per chunk and head
size_t forward_scratch(int64_t B, int64_t T, int64_t HV, bool with_state) {
    return chunk_count(T) * B * HV *
           (with_state ? ChunkImage<3, kFwdOut>::kBytes : ChunkImage<2, kFwdOut>::kBytes);
}

// dst = src, or zeros; the T = 0 call's only work
wkv_status copy_state(float *dst, const float *src, size_t bytes, cudaStream_t stream) {
    if (dst == nullptr || dst == src) return WKV_OK;
    const cudaError_t e = src != nullptr
                              ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, stream)
                              : cudaMemsetAsync(dst, 0, bytes, stream);
    return e == cudaSuccess ? WKV_OK : cuda_fail(e, "copy of the state");
}

// Bytes of a tensor; sizes without a limit (those of calls that compute
// nothing) end at 2^62, which no allocation holds.
size_t tensor_bytes(std::initializer_list<int64_t> sizes, size_t elem) {
    unsigned __int128 n = elem;
    for (const int64_t s : sizes)
        if (s == 0) return 0;
    for (const int64_t s : sizes) n = std::min<unsigned __int128>(n * s, static_cast<unsigned __int128>(1) << 62);
    return static_cast<size_t>(n);
}

// A call without value heads, or with heads of no width, has nothing but sums
// over nothing: those of its outputs that are not empty become zeros.
template <int N>
wkv_status zero_outputs(Buf (&bufs)[N], cudaStream_t stream) {
    bool any = false;
    for (Buf &b : bufs) {
        if (b.bytes == 0) b.p = nullptr;  // an empty tensor's pointer may be anything
        any = any || (b.written && b.p != nullptr);
    }
    if (!any) return WKV_OK;
    int dev = 0;
    wkv_status st = current_device(&dev);
    if (st != WKV_OK || (st = check_buffers(bufs, dev)) != WKV_OK) return st;
    for (const Buf &b : bufs) {
        if (!b.written || b.p == nullptr) continue;
        const cudaError_t e = cudaMemsetAsync(const_cast<void *>(b.p), 0, b.bytes, stream);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    }
    return WKV_OK;
}

template <typename IO>
wkv_status delta_forward(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK, int64_t DV,
                         const void *q, const void *k, const void *v, const float *g,
                         const float *beta, float scale, void *o, const float *s_in, float *s_out,
                         void *scratch, int64_t scratch_bytes, cudaStream_t stream) {
    set_last_error("");
    bool empty = false;
    wkv_status st = check_delta(B, T, HK, HV, DK, DV, &empty);
    if (st != WKV_OK) return st;
    const int64_t need = empty ? 0 : gated_delta_scratch(B, T, HV, DK, DV, sizeof(IO), s_out != nullptr);
    if (!empty && scratch_bytes < need)
        return fail(WKV_ERR_INVALID_ARG, "scratch has %lld bytes, %lld needed",
                    static_cast<long long>(scratch_bytes), static_cast<long long>(need));
    const size_t nk = tensor_bytes({B, T, HK, DK}, sizeof(IO)), nv = tensor_bytes({B, T, HV, DV}, sizeof(IO));
    const size_t ng = tensor_bytes({B, T, HV}, 4), ns = tensor_bytes({B, HV, DK, DV}, 4);
    const bool none = T == 0 || empty;
    Buf bufs[] = {{"q", q, nk, sizeof(IO), false, none},
                  {"k", k, nk, sizeof(IO), false, none},
                  {"v", v, nv, sizeof(IO), false, none},
                  {"g", g, ng, 4, false, none},
                  {"beta", beta, ng, 4, false, none},
                  {"o", o, nv, sizeof(IO), true, none},
                  {"s_in", s_in, ns, 4, false, true},
                  {"s_out", s_out, ns, 4, true, true},
                  {"scratch", need > 0 ? scratch : nullptr, static_cast<size_t>(need), 16, true, need == 0}};
    if (empty) return zero_outputs(bufs, stream);
    int dev = 0;
    if ((st = current_device(&dev)) != WKV_OK) return st;
    if ((st = check_buffers(bufs, dev, 6, 7)) != WKV_OK) return st;
    if (none) return copy_state(s_out, s_in, ns, stream);
    DeltaFwdArgs<IO> a{};
    a.q = static_cast<const IO *>(q), a.k = static_cast<const IO *>(k);
    a.v = static_cast<const IO *>(v), a.o = static_cast<IO *>(o);
    a.g = g, a.beta = beta, a.s_in = s_in, a.s_out = s_out, a.scale = scale;
    a.z = sizes(B, T, HK, HV, DK, DV);
    if constexpr (sizeof(IO) == 2) {
        CUtensorMap m[3];
        if (need > 0 && chunked_fits(a.z, q, k, v) && make_map(&m[0], q, a.z, a.z.HK, a.z.DK) &&
            make_map(&m[1], k, a.z, a.z.HK, a.z.DK) && make_map(&m[2], v, a.z, a.z.HV, a.z.DV)) {
            const DeltaPrepArgs p{g, beta, static_cast<unsigned char *>(scratch), nullptr, nullptr, scale, a.z, silent_chunk(1)};
            const DeltaChainArgs c{p.fwd, nullptr, s_in, a.o, s_out, nullptr, nullptr, scale, a.z, silent_chunk(2)};
            const bool small = a.z.DK <= 64;
            if (s_out == nullptr)
                return small ? launch_forward<1, 2>(p, c, m, dev, stream) : launch_forward<2, 2>(p, c, m, dev, stream);
            return small ? launch_forward<1, 3>(p, c, m, dev, stream) : launch_forward<2, 3>(p, c, m, dev, stream);
        }
    }
    return launch_recurrent<IO>(a, sm_count(dev), stream);
}

// The gradient's scratch: the states before each chunk, the gradients of the
// states after each chunk, the residuals r and du, and the sweeps' images or
// gq and gk of every value head.
struct Scratch {
    size_t starts, ends, r, du, fwd, rev, rev2, parts, bytes;
    Scratch(int64_t B, int64_t T, int64_t HV, int64_t DK, int64_t DV, int elem_bytes) {
        const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
        const size_t heads = static_cast<size_t>(B) * HV, images = chunk_count(T) * heads;
        const size_t rows = images * sweep_floats(kDeltaChunk, DV) * 4;
        const bool chunked = chunked_sizes(T, HV, DK, DV, elem_bytes);
        const size_t img = chunked ? ChunkImage<3, kReverse>::kBytes : 0;
        starts = 0;
        ends = up(images * sweep_floats(DK, DV) * 4);
        r = 2 * ends;
        du = r + up(rows);
        fwd = du + up(rows);
        rev = fwd + images * img;
        rev2 = rev + images * img;
        parts = rev2 + (chunked ? images * second_image_bytes(DK <= 64 ? 1 : 2) : 0);
        bytes = parts + (chunked ? 0 : up(heads * T * DK * 8));
    }
};

template <typename IO, int NC>
wkv_status launch_grads(const DeltaGradArgs<IO> &a, unsigned grid, int dev, cudaStream_t s) {
    auto kern = delta_grads_kernel<IO, NC>;
    static std::atomic<uint64_t> configured{0};
    const wkv_status st = allow_smem(kern, sizeof(GradStage), dev, configured);
    if (st != WKV_OK) return st;
    cudaGetLastError();
    kern<<<grid, kGradThreads, sizeof(GradStage), s>>>(a);
    return launched();
}

template <typename IO>
wkv_status delta_backward(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK, int64_t DV,
                          const void *q, const void *k, const void *v, const float *g,
                          const float *beta, float scale, const float *s_in, const void *go,
                          const float *gs_out, void *gq, void *gk, void *gv, float *gg,
                          float *gbeta, float *gs_in, void *scratch, int64_t scratch_bytes,
                          cudaStream_t stream) {
    set_last_error("");
    bool empty = false;
    wkv_status st = check_delta(B, T, HK, HV, DK, DV, &empty);
    if (st != WKV_OK) return st;
    const int64_t need = empty ? 0 : gated_delta_backward_scratch(B, T, HV, DK, DV, sizeof(IO));
    if (!empty && scratch_bytes < need)
        return fail(WKV_ERR_INVALID_ARG, "scratch has %lld bytes, %lld needed",
                    static_cast<long long>(scratch_bytes), static_cast<long long>(need));
    const size_t nk = tensor_bytes({B, T, HK, DK}, sizeof(IO)), nv = tensor_bytes({B, T, HV, DV}, sizeof(IO));
    const size_t ng = tensor_bytes({B, T, HV}, 4), ns = tensor_bytes({B, HV, DK, DV}, 4);
    const bool none = T == 0 || empty;
    Buf bufs[] = {{"q", q, nk, sizeof(IO), false, none},
                  {"k", k, nk, sizeof(IO), false, none},
                  {"v", v, nv, sizeof(IO), false, none},
                  {"g", g, ng, 4, false, none},
                  {"beta", beta, ng, 4, false, none},
                  {"go", go, nv, sizeof(IO), false, none},
                  {"s_in", s_in, ns, 4, false, true},
                  {"gs_out", gs_out, ns, 4, false, true},
                  {"gq", gq, nk, sizeof(IO), true, none},
                  {"gk", gk, nk, sizeof(IO), true, none},
                  {"gv", gv, nv, sizeof(IO), true, none},
                  {"gg", gg, ng, 4, true, none},
                  {"gbeta", gbeta, ng, 4, true, none},
                  {"gs_in", gs_in, ns, 4, true, true},
                  {"scratch", need > 0 ? scratch : nullptr, static_cast<size_t>(need), 16, true, need == 0}};
    if (empty) return zero_outputs(bufs, stream);
    int dev = 0;
    if ((st = current_device(&dev)) != WKV_OK) return st;
    if ((st = check_buffers(bufs, dev)) != WKV_OK) return st;
    if (none) return copy_state(gs_in, gs_out, ns, stream);
    const Scratch sc(B, T, HV, DK, DV, sizeof(IO));
    char *base = static_cast<char *>(scratch);
    float *starts = reinterpret_cast<float *>(base + sc.starts);
    float *ends = reinterpret_cast<float *>(base + sc.ends);
    float *r = reinterpret_cast<float *>(base + sc.r);
    float *du = reinterpret_cast<float *>(base + sc.du);
    const DeltaSizes z = sizes(B, T, HK, HV, DK, DV);
    const int sms = sm_count(dev);

    DeltaFwdArgs<IO> f{};
    f.q = static_cast<const IO *>(q), f.k = static_cast<const IO *>(k);
    f.v = static_cast<const IO *>(v);
    f.g = g, f.beta = beta, f.s_in = s_in, f.r = r, f.starts = starts, f.scale = scale, f.z = z;
    DeltaRevArgs<IO> rv{};
    rv.q = f.q, rv.k = f.k, rv.go = static_cast<const IO *>(go);
    rv.g = g, rv.beta = beta, rv.gs_out = gs_out, rv.gv = static_cast<IO *>(gv);
    rv.du = du, rv.ends = ends, rv.gs_in = gs_in, rv.scale = scale, rv.z = z;
    if constexpr (sizeof(IO) == 2) {
        CUtensorMap m[5];
        if (chunked_fits(z, q, k, v) && aligned(go, 16) && aligned(gq, 16) && aligned(gk, 16) && aligned(gv, 16) &&
            make_map(&m[0], q, z, z.HK, z.DK) && make_map(&m[1], k, z, z.HK, z.DK) &&
            make_map(&m[2], v, z, z.HV, z.DV) && make_map(&m[3], go, z, z.HV, z.DV) &&
            make_map(&m[4], gv, z, z.HV, z.DV)) {
            unsigned char *img = static_cast<unsigned char *>(scratch);
            const DeltaPrepArgs p{g, beta, img + sc.fwd, img + sc.rev, img + sc.rev2, scale, z, silent_chunk(1)};
            const DeltaChainArgs fa{p.fwd, nullptr, s_in, nullptr, nullptr, r, starts, scale, z, silent_chunk(2)};
            const DeltaChainArgs ra{p.rev, p.rev2, gs_out, nullptr, gs_in, du, ends, scale, z, silent_chunk(2)};
            const DeltaTcGradArgs tg{g, beta, r, du, starts, ends, static_cast<IO *>(gq), static_cast<IO *>(gk),
                                     static_cast<IO *>(gv), gg, gbeta, scale, z, silent_chunk(3)};
            return z.DK <= 64 ? launch_gradient<1>(p, fa, ra, tg, m, dev, stream)
                              : launch_gradient<2>(p, fa, ra, tg, m, dev, stream);
        }
    }
    if ((st = launch_recurrent_sweeps<IO>(f, rv, sms, stream)) != WKV_OK) return st;

    DeltaGradArgs<IO> ga{};
    ga.q = f.q, ga.k = f.k, ga.go = rv.go, ga.g = g, ga.beta = beta, ga.r = r, ga.du = du;
    ga.starts = starts, ga.ends = ends, ga.gq = static_cast<IO *>(gq);
    ga.gk = static_cast<IO *>(gk), ga.gg = gg, ga.gbeta = gbeta, ga.scale = scale, ga.z = z;
    // While there are fewer key heads' chunks than SMs, their value heads take a
    // block each and are added by another kernel: B=2 T=333, 6 heads of 80 x 72
    // on 3 key heads, 74 against 122 us.  Beyond, the blocks fill the SMs.
    const size_t blocks = chunk_count(T) * B * HK;
    const bool split = z.group > 1 && blocks <= static_cast<size_t>(sms) && sc.bytes > sc.parts;
    if (split) ga.parts = reinterpret_cast<float *>(base + sc.parts);
    const unsigned grid = static_cast<unsigned>(split ? blocks * z.group : blocks);
    st = z.DK <= 64 ? launch_grads<IO, 4>(ga, grid, dev, stream)
         : z.DK <= 96 ? launch_grads<IO, 6>(ga, grid, dev, stream) : launch_grads<IO, 8>(ga, grid, dev, stream);
    if (st != WKV_OK) return st;
    if (split) {
        const size_t n = static_cast<size_t>(B) * T * HK * DK;
        delta_grads_sum_kernel<IO><<<static_cast<unsigned>(std::min<size_t>((n + 255) / 256, 8 * sms)), 256, 0, stream>>>(ga);
    }
    return launched();
}

}  // namespace

extern "C" {

wkv_status gated_delta(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK, int64_t DV,
                       const float *q, const float *k, const float *v, const float *g,
                       const float *beta, float scale, float *o, const float *s_in, float *s_out,
                       void *scratch, int64_t scratch_bytes, cudaStream_t stream) {
    return delta_forward<float>(B, T, HK, HV, DK, DV, q, k, v, g, beta, scale, o, s_in, s_out,
                                scratch, scratch_bytes, stream);
}

wkv_status gated_delta_bf16(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK, int64_t DV,
                            const wkv_bf16_t *q, const wkv_bf16_t *k, const wkv_bf16_t *v,
                            const float *g, const float *beta, float scale, wkv_bf16_t *o,
                            const float *s_in, float *s_out, void *scratch,
                            int64_t scratch_bytes, cudaStream_t stream) {
    return delta_forward<bf16>(B, T, HK, HV, DK, DV, q, k, v, g, beta, scale, o, s_in, s_out,
                               scratch, scratch_bytes, stream);
}

wkv_status gated_delta_set_fault_injection(int kernel, int chunk) {
    set_last_error("");
    if (kernel < 0 || kernel > 3 || chunk < 0)
        return fail(WKV_ERR_INVALID_ARG, "kernel must be 0 .. 3, chunk >= 0");
    g_fault_kernel.store(kernel);
    g_fault_chunk.store(chunk);
    return WKV_OK;
}

int64_t gated_delta_scratch(int64_t B, int64_t T, int64_t HV, int64_t DK, int64_t DV, int elem_bytes,
                            int with_state) {
    bool empty = false;
    if (check_delta(B, T, HV, HV, DK, DV, &empty) != WKV_OK || empty ||
        !chunked_forward(B, T, HV, DK, DV, elem_bytes))
        return 0;
    return static_cast<int64_t>(forward_scratch(B, T, HV, with_state != 0));
}

int64_t gated_delta_backward_scratch(int64_t B, int64_t T, int64_t HV, int64_t DK, int64_t DV,
                                     int elem_bytes) {
    bool empty = false;
    if (check_delta(B, T, HV, HV, DK, DV, &empty) != WKV_OK || empty || T == 0) return 0;
    return static_cast<int64_t>(Scratch(B, T, HV, DK, DV, elem_bytes).bytes);
}

wkv_status gated_delta_backward(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK,
                                int64_t DV, const float *q, const float *k, const float *v,
                                const float *g, const float *beta, float scale, const float *s_in,
                                const float *go, const float *gs_out, float *gq, float *gk,
                                float *gv, float *gg, float *gbeta, float *gs_in, void *scratch,
                                int64_t scratch_bytes, cudaStream_t stream) {
    return delta_backward<float>(B, T, HK, HV, DK, DV, q, k, v, g, beta, scale, s_in, go, gs_out,
                                 gq, gk, gv, gg, gbeta, gs_in, scratch, scratch_bytes, stream);
}

wkv_status gated_delta_backward_bf16(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK,
                                     int64_t DV, const wkv_bf16_t *q, const wkv_bf16_t *k,
                                     const wkv_bf16_t *v, const float *g, const float *beta,
                                     float scale, const float *s_in, const wkv_bf16_t *go,
                                     const float *gs_out, wkv_bf16_t *gq, wkv_bf16_t *gk,
                                     wkv_bf16_t *gv, float *gg, float *gbeta, float *gs_in,
                                     void *scratch, int64_t scratch_bytes, cudaStream_t stream) {
    return delta_backward<bf16>(B, T, HK, HV, DK, DV, q, k, v, g, beta, scale, s_in, go, gs_out, gq,
                                gk, gv, gg, gbeta, gs_in, scratch, scratch_bytes, stream);
}

}  // extern "C"
