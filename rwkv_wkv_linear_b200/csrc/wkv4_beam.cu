// Launchers of the beam search kernels (wkv4_beam.cuh).
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/wkv4.h"
#include "wkv4_beam.cuh"
#include "wkv4_launch.cuh"

namespace wkv4 {

template <typename IO>
static cudaError_t launch_beam_select_t(const BeamParams& p, int64_t G, int R, cudaStream_t stream) {
    auto kern = wkv4_beam_select_kernel<IO>;
    // the merge holds every unit's candidates
    const size_t cands = (size_t)p.K * p.S * p.n * sizeof(BeamCand);
    const size_t most = sizeof(BeamShared) + (size_t)kBeamMaxK * kBeamMaxN * sizeof(BeamCand);
    static DeviceFlags attr, wide;
    cudaError_t e = ensure_smem_attr(attr, kern, most);
    if (e != cudaSuccess) return e;
    if (R > 8) {
        e = ensure_attr(wide, kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = launch_grid(dim3((unsigned)(G * R)));
    cfg.blockDim = dim3(kBeamThreads);
    cfg.dynamicSmemBytes = sizeof(BeamShared) + std::max(cands, (size_t)kBeamPieces * 16);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)R;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_beam_select(const BeamArgs& a) {
    BeamParams p{};
    p.V = a.V;
    p.ld = a.ld;
    p.K = (int)a.K;
    p.n = (int)a.n;
    p.end_id = a.end_id;
    p.logits = a.logits;
    p.scores = a.scores;
    p.finished = a.finished;
    p.out_scores = a.out_scores;
    p.out_parents = a.out_parents;
    p.out_tokens = a.out_tokens;
    // CTAs a group: one a beam or one a 2048 logits, whichever are more, at most
    // 8 a cluster -- 16 (which a group of SMs may not have room for twice) while
    // the groups leave SMs idle otherwise: one request of 4 beams 8.4 us against
    // 9.9, 48 requests of 8 beams 33.3 us against 21.0 with 8.
    const int most = a.G * 16 <= 148 ? 16 : 8;
    int R = 1;
    while (R < most && (R < a.K || a.K * a.V >= 2 * R * 2048)) R *= 2;
    p.S = 1;
    while (p.S * 2 * a.K <= R) p.S *= 2;
    switch (a.dtype) {
        case WKV4_F32: return launch_beam_select_t<float>(p, a.G, R, a.stream);
        case WKV4_F16: return launch_beam_select_t<__half>(p, a.G, R, a.stream);
        default: return launch_beam_select_t<__nv_bfloat16>(p, a.G, R, a.stream);
    }
}

template <typename E, int N>
static cudaError_t launch_reorder_n(const ReorderArgs& a, const ReorderParams& p, int x) {
    const int y = 256 / x;
    // an empty pool still has new slot ids to write
    const dim3 grid((unsigned)std::max<int64_t>(1, (p.row + x - 1) / x),
                    (unsigned)std::max<int64_t>(1, (a.P + y * N - 1) / (y * N)), (unsigned)a.G);
    return launch_pdl(wkv4_state_reorder_kernel<E, N>, launch_grid(grid), dim3((unsigned)x, (unsigned)y), 0,
                      a.stream, p);
}

template <typename E>
static cudaError_t launch_reorder_t(const ReorderArgs& a, int64_t row_bytes) {
    ReorderParams p{a.P, a.S, row_bytes / (int64_t)sizeof(E), (int)a.K, a.pool, a.ids, a.parents, a.new_ids};
    int x = 32;  // threads along a row; the rest of the block along the planes
    while (x < 256 && x < p.row) x *= 2;
    // two planes a thread once there is more than a wave of CTAs: twice the rows
    // in flight (8 requests of 8 beams, 120 planes of 5120 fp32: 22.6 us against
    // 27.0 with one and 23.5 with four; a small pool 2.2, 2.4, 3.1)
    const int64_t ctas = (p.row + x - 1) / x * ((a.P + 256 / x - 1) / (256 / x)) * a.G;
    return ctas > 148 * 8 ? launch_reorder_n<E, 2>(a, p, x) : launch_reorder_n<E, 1>(a, p, x);
}

cudaError_t launch_state_reorder(const ReorderArgs& a) {
    const int64_t bytes = a.C * (int64_t)dtype_size(a.dtype);
    const uintptr_t mis = (uintptr_t)a.pool | (uintptr_t)bytes;
    if (mis % 16 == 0) return launch_reorder_t<uint4>(a, bytes);
    if (mis % 4 == 0) return launch_reorder_t<uint32_t>(a, bytes);
    return launch_reorder_t<uint16_t>(a, bytes);
}

cudaError_t read_beam_error(unsigned* bits, bool reset) { return read_error_word(bits, reset); }

}  // namespace wkv4
