// Launchers of the backward kernels: the WKV recurrence's (wkv4_backward.cuh)
// and the token shift's (wkv4_shift_backward.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/wkv4.h"
#include "wkv4_backward.cuh"
#include "wkv4_launch.cuh"
#include "wkv4_shift_backward.cuh"

namespace wkv4 {

// Launch shape of the backward pass, from the sizes and the type alone (the
// workspace is sized from it): steps a chunk, CTAs a cluster, rounds.
struct BwdShape {
    int L, NC;
    int64_t rounds;
    int64_t rows(int64_t B) const { return B * NC; }  // partial sums a channel
};

static BwdShape bwd_shape(int64_t B, int64_t T, int64_t C, int dtype, bool gated) {
    BwdShape s;
    const int64_t tiles = (C + kBwdC - 1) / kBwdC * B;
    auto shape = [&](int L) {
        const int64_t ctas = std::max<int64_t>(1, (T + kBwdWarps * L - 1) / (kBwdWarps * L));
        s.L = L;
        // 8 CTAs a cluster at most, 16 where all of them fit the GPU at once or in
        // two waves of 3 an SM with one round: a round is a chain of latencies,
        // and the second makes k, v be read twice, but what wide clusters wait
        // for each other grows with their number.  bf16, gated, with 8 and 16:
        // B=1, T=2048, C=768 37.0, 16.3 us; B=4, T=2048, C=768 54.4, 49.2; B=4,
        // T=1536, C=2560 97.3, 100.4; B=4, T=2048, C=5120 241, 261.  No more of
        // them than the rounds need: a CTA without steps keeps its place all the same.
        const bool wide = tiles * kBwdMaxCtas <= 2 * 148 || (ctas <= kBwdMaxCtas && tiles * ctas <= 6 * 148);
        const int most = wide ? kBwdMaxCtas : 8;
        s.rounds = (ctas + most - 1) / most;
        s.NC = (int)((ctas + s.rounds - 1) / s.rounds);
    };
    // Steps a chunk: 32; in fp32 (twice the shared memory, so fewer CTAs an SM)
    // 16 unless the CTAs are few and walk several rounds, whose joins are then
    // spread over twice the steps (B=1, T=16384, C=2048: 346 us with 16, 233 with 32).
    shape(dtype == WKV4_F32 ? 16 : 32);
    if (dtype == WKV4_F32 && !gated && s.rounds > 1 && tiles * s.NC <= 2 * 148) shape(32);
    return s;
}

// Workspace: partial sums of gw, gu (one row a CTA of each cluster, none when
// one CTA a channel tile writes them itself), then the rounds' states.
static size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }
static size_t bwd_part_bytes(int64_t B, int64_t C, const BwdShape& s) {
    return s.rows(B) == 1 ? 0 : align16((size_t)2 * s.rows(B) * C * 4);
}

size_t backward_workspace(int64_t B, int64_t T, int64_t C, int dtype) {
    size_t most = 0;  // gated or not
    for (bool gated : {false, true}) {
        const BwdShape s = bwd_shape(B, T, C, dtype, gated);
        most = std::max(most, bwd_part_bytes(B, C, s) + (s.rounds > 1 ? (size_t)s.rounds * B * C * kSumBytes : 0));
    }
    return most;
}

static cudaError_t launch_column_sum(const float* part, float* o0, float* o1, float* o2, int n,
                                     int64_t rows, int64_t C, cudaStream_t stream) {
    const ColumnSumParams p{part, {o0, o1, o2}, rows, C};
    return launch_pdl(wkv4_column_sum_kernel, launch_grid(dim3((unsigned)((C + 31) / 32), (unsigned)n)),
                      dim3(256), 0, stream, p);
}

template <typename IO, int L, bool kGate, bool kOne>
static cudaError_t launch_backward_t(const BwdArgs& a, BwdParams& p, const BwdShape& sh) {
    using Lay = BwdLayout<IO, L, kGate>;
    auto kern = wkv4_backward_kernel<IO, L, kGate, kOne>;
    static DeviceFlags attr;
    cudaError_t e = ensure_smem_attr(attr, kern, Lay::bytes(kBwdMaxCtas));
    if (e != cudaSuccess) return e;
    if (sh.NC > 8) {
        static DeviceFlags wide;
        e = ensure_attr(wide, kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    const unsigned tiles = (unsigned)((a.C + kBwdC - 1) / kBwdC), threads = 32 * kBwdWarps;
    if constexpr (!kOne) {
        auto sum = wkv4_backward_summary_kernel<IO, L>;
        const size_t smem = kBwdWarps * (4 * Lay::kTile + kBwdC * kSumBytes);
        static DeviceFlags sattr;
        e = ensure_smem_attr(sattr, sum, smem);
        if (e != cudaSuccess) return e;
        e = launch_pdl(sum, launch_grid(dim3(tiles, (unsigned)sh.rounds, (unsigned)a.B)), dim3(threads),
                       smem, a.stream, p, sh.NC);
        if (e != cudaSuccess) return e;
        const int64_t BC = a.B * a.C;
        e = launch_pdl(wkv4_backward_prefix_kernel, launch_grid(dim3((unsigned)((BC + 127) / 128))),
                       dim3(128), 0, a.stream, p, (int64_t)sh.NC * kBwdWarps * L);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = launch_grid(dim3((unsigned)sh.NC, tiles, (unsigned)a.B));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = Lay::bytes(sh.NC);
    cfg.stream = a.stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)sh.NC;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) return e;
    if (sh.rows(a.B) > 1)
        e = launch_column_sum(p.part_w, a.gw, a.gu, nullptr, 2, sh.rows(a.B), a.C, a.stream);
    return e;
}

template <typename IO, int L, bool kGate>
static cudaError_t launch_backward_rounds(const BwdArgs& a, BwdParams& p, const BwdShape& sh) {
    return sh.rounds == 1 ? launch_backward_t<IO, L, kGate, true>(a, p, sh)
                          : launch_backward_t<IO, L, kGate, false>(a, p, sh);
}

template <typename IO>
static cudaError_t launch_backward_io(const BwdArgs& a, BwdParams& p, const BwdShape& sh) {
    if constexpr (sizeof(IO) == 4) {
        if (sh.L == 32) return launch_backward_rounds<IO, 32, false>(a, p, sh);
        return a.r ? launch_backward_rounds<IO, 16, true>(a, p, sh) : launch_backward_rounds<IO, 16, false>(a, p, sh);
    } else {
        return a.r ? launch_backward_rounds<IO, 32, true>(a, p, sh) : launch_backward_rounds<IO, 32, false>(a, p, sh);
    }
}

cudaError_t launch_backward(const BwdArgs& a) {
    const BwdShape sh = bwd_shape(a.B, a.T, a.C, a.dtype, a.r != nullptr);
    BwdParams p{};
    p.B = a.B;
    p.T = a.T;
    p.C = a.C;
    p.rounds = (int)sh.rounds;
    p.w = a.w;
    p.u = a.u;
    p.k = a.k;
    p.v = a.v;
    p.r = a.r;
    p.gy = a.gy;
    p.state_in = a.state_in;
    p.state_out = a.state_out;
    p.gstate_out = a.gstate_out;
    p.gk = a.gk;
    p.gv = a.gv;
    p.gr = a.gr;
    p.gstate_in = a.gstate_in;
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    if (sh.rows(a.B) > 1) {
        p.part_w = reinterpret_cast<float*>(ws);
        p.part_u = p.part_w + sh.rows(a.B) * a.C;
        ws += bwd_part_bytes(a.B, a.C, sh);
    } else {
        p.part_w = a.gw;
        p.part_u = a.gu;
    }
    if (sh.rounds > 1) {
        const int64_t n = sh.rounds * a.B * a.C;
        p.ck_p = reinterpret_cast<int*>(ws);
        p.ck_a = reinterpret_cast<float*>(ws + n * 4);
        p.ck_b = p.ck_a + n;
    }
    const size_t es = dtype_size(a.dtype);
    p.NC = sh.NC;
    p.vec_load = (a.C * es) % 16 == 0 && aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.gy, 16) &&
                 aligned(a.r, 16);
    p.vec_store = a.C % 2 == 0 && aligned(a.gk, 2 * es) && aligned(a.gv, 2 * es) && aligned(a.gr, 2 * es);
    p.wait_rounds = wait_rounds();
    p.mute = kMuteNone;
#ifdef WKV4_CHECKED
    // with WKV4_FAULT_RANK=R the injected fault silences the CTAs of rank R alone
    if (fault_plan().exchange) p.mute = env_int("WKV4_FAULT_RANK", kMuteAll);
#endif
    if (a.T == 0) {
        const int64_t n = a.B * a.C;
        return launch_pdl(wkv4_backward_no_steps_kernel, launch_grid(dim3((unsigned)((n + 127) / 128))),
                          dim3(128), 0, a.stream, p, a.gw, a.gu);
    }
    switch (a.dtype) {
        case WKV4_F32: return launch_backward_io<float>(a, p, sh);
        case WKV4_F16: return launch_backward_io<__half>(a, p, sh);
        default: return launch_backward_io<__nv_bfloat16>(a, p, sh);
    }
}

// ------------------------------------------------------------- token shift

// Runs of the token shift's backward pass: as many CTAs as the GPU holds at
// once, at least kShiftMinRun steps a run.
struct ShiftBwdShape {
    int V;
    int64_t run, yblocks;
    // A channel block's CTAs as one cluster: no second kernel (a short call is all
    // launches: B=2, T=65, C=768 29.8 -> 24.6 us of host time).  Clusters of 16
    // would leave SMs idle (B=4, T=1024, C=5120: 51.9 us against 46.4).
    bool one_cluster(int64_t B) const { return yblocks * B <= 8; }
};

// V: channels a thread at most (by alignment).  The wide form reads 512 bytes a
// warp and row instead of 256, which HBM likes better, and is taken where its
// fewer threads fill the GPU all the same (bf16: B=4, T=1024, C=5120 39.8 us
// against 47.1; B=2, T=65, C=768 5.5 against 4.7).
static ShiftBwdShape shift_bwd_shape(int64_t B, int64_t T, int64_t C, int V) {
    ShiftBwdShape s;
    s.V = V;
    const int64_t xb = (C + kShiftBwdX * V - 1) / (kShiftBwdX * V);
    const int64_t blocks = std::max<int64_t>(1, (int64_t)148 * shift_bwd_ctas(V) / std::max<int64_t>(1, xb * B));
    const int64_t runs = blocks * kShiftBwdY;
    s.run = std::max<int64_t>((T + runs - 1) / runs, kShiftMinRun);
    if (V == kShiftBwdWide && s.run == kShiftMinRun) return shift_bwd_shape(B, T, C, 4);
    s.run = std::max<int64_t>(s.run, (T + 65535ll * kShiftBwdY - 1) / (65535ll * kShiftBwdY));
    s.yblocks = (T + s.run * kShiftBwdY - 1) / (s.run * kShiftBwdY);
    return s;
}

size_t shift_backward_workspace(int64_t B, int64_t T, int64_t C, int n) {
    int64_t rows = 0;  // any channel width may be taken (it depends on type and alignment)
    for (int V : {1, 4, kShiftBwdWide}) {
        const ShiftBwdShape s = shift_bwd_shape(B, T, C, V);
        if (!s.one_cluster(B)) rows = std::max(rows, s.yblocks);
    }
    return (size_t)n * B * rows * C * 4;
}

template <typename IO, int V, int N>
static cudaError_t launch_shift_bwd_t(const ShiftBwdParams& p, const ShiftBwdShape& s, cudaStream_t stream) {
    auto kern = wkv4_token_shift_backward_kernel<IO, V, N>;
    const dim3 grid((unsigned)((p.C + kShiftBwdX * V - 1) / (kShiftBwdX * V)), (unsigned)s.yblocks, (unsigned)p.B);
    const bool one = s.one_cluster(p.B);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = launch_grid(grid);
    cfg.blockDim = dim3(kShiftBwdX, kShiftBwdY);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = (unsigned)s.yblocks;
    at[1].val.clusterDim.z = (unsigned)p.B;
    cfg.attrs = at;
    cfg.numAttrs = one ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename IO, int N>
static cudaError_t launch_shift_bwd_n(const ShiftBwdParams& p, const ShiftBwdShape& s, cudaStream_t stream) {
    if constexpr (sizeof(IO) == 2)
        if (s.V == kShiftBwdWide) return launch_shift_bwd_t<IO, kShiftBwdWide, N>(p, s, stream);
    return s.V == 4 ? launch_shift_bwd_t<IO, 4, N>(p, s, stream) : launch_shift_bwd_t<IO, 1, N>(p, s, stream);
}

template <typename IO>
static cudaError_t launch_shift_bwd_io(const ShiftBwdParams& p, const ShiftBwdShape& s, int n,
                                       cudaStream_t stream) {
    return n == 3 ? launch_shift_bwd_n<IO, 3>(p, s, stream) : launch_shift_bwd_n<IO, 2>(p, s, stream);
}

cudaError_t launch_shift_backward(const ShiftBwdArgs& a) {
    const int n = a.mix[2] ? 3 : 2;
    const size_t es = dtype_size(a.dtype);
    auto fits = [&](int V) {  // every row starts on V elements
        bool ok = a.C % V == 0 && aligned(a.x, V * es) && aligned(a.x_prev, V * es) && aligned(a.gx, V * es) &&
                  aligned(a.gx_prev, V * es) && aligned(a.gx_last, V * es);
        for (int i = 0; i < n; ++i) ok = ok && aligned(a.mix[i], 16) && aligned(a.g[i], V * es);
        return ok;
    };
    const int V = es == 2 && fits(kShiftBwdWide) ? kShiftBwdWide : fits(4) ? 4 : 1;
    const ShiftBwdShape s = shift_bwd_shape(a.B, a.T, a.C, V);
    ShiftBwdParams p{};
    p.B = a.B;
    p.T = a.T;
    p.C = a.C;
    p.x = a.x;
    p.x_prev = a.x_prev;
    p.gx_last = a.gx_last;
    p.gx = a.gx;
    p.gx_prev = a.gx_prev;
    for (int i = 0; i < n; ++i) {
        p.mix[i] = a.mix[i];
        p.g[i] = a.g[i];
    }
    for (int i = 0; i < n; ++i) p.gmix[i] = a.gmix[i];
    p.part = s.one_cluster(a.B) ? nullptr : static_cast<float*>(a.workspace);
    p.rows = a.B * s.yblocks;
    p.run = s.run;
    cudaError_t e;
    switch (a.dtype) {
        case WKV4_F32: e = launch_shift_bwd_io<float>(p, s, n, a.stream); break;
        case WKV4_F16: e = launch_shift_bwd_io<__half>(p, s, n, a.stream); break;
        default: e = launch_shift_bwd_io<__nv_bfloat16>(p, s, n, a.stream); break;
    }
    if (e != cudaSuccess || !p.part) return e;
    return launch_column_sum(p.part, a.gmix[0], a.gmix[1], a.gmix[2], n, p.rows, a.C, a.stream);
}

cudaError_t read_train_error(unsigned* bits, bool reset) { return read_error_word(bits, reset); }

}  // namespace wkv4
