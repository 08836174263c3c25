// Backward pass of the token shift.  Forward, for up to three mixes m_i,
//   out_i[b,t] = m_i x[b,t] + (1 - m_i) x[b,t-1],  x[b,-1] = x_prev[b],
// so with g_i the gradient of out_i
//   gx[b,t]    = sum_i m_i g_i[b,t] + sum_i (1 - m_i) g_i[b,t+1]   (t + 1 < T)
//              (+ gx_last[b] at t = T - 1: x_last = x[:, T-1] feeds the next call),
//   gx_prev[b] = sum_i (1 - m_i) g_i[b,0],
//   gm_i       = sum_{b,t} g_i[b,t] (x[b,t] - x[b,t-1]).
//
// An HBM stream: a thread owns V channels of one batch row and walks a run of
// steps with the row before in registers (x[t-1], and sum_i m_i g_i[t-1], which
// waits for the next row's share before it is stored), so every input is read
// once (plus one row a run) and gx written once.  Its rows come through a ring
// of kShiftBwdStages of its own in shared memory, filled by asynchronous
// copies: a thread waits for nobody, and what is in flight does not cost
// registers.  The gm_i partial sums of the CTA's runs are joined in shared
// memory.  Where the CTAs of one channel block are at most 8 they are one
// cluster and add up their sums through its shared memory; otherwise each
// writes a row and wkv4_column_sum_kernel adds the rows.  Both in a fixed
// order.  All arithmetic in fp32, rounded once at the stores.
#pragma once

#include <cooperative_groups.h>

#include "wkv4_device.cuh"
#include "wkv4_shift.cuh"  // load_f32

namespace wkv4 {

struct ShiftBwdParams {
    int64_t B, T, C;
    const void* x;
    const void* x_prev;   // [B][C] or NULL (zero)
    const float* mix[3];
    const void* g[3];     // gradients of the outputs
    const void* gx_last;  // [B][C] or NULL
    void* gx;
    void* gx_prev;        // [B][C] or NULL
    float* gmix[3];       // gm_i, written by the clusters themselves (part NULL), or
    float* part;          // [n][rows][C] partial sums of gm, row (b, y block)
    int64_t rows;
    int64_t run;          // steps a thread walks
};

constexpr int kShiftBwdX = 32;  // channel groups a CTA
constexpr int kShiftBwdY = 4;   // runs a CTA
template <typename IO> constexpr int kShiftBwdStages = sizeof(IO) == 2 ? 8 : 4;  // 32 KB of rows a CTA
constexpr int kShiftBwdCtas = 5;  // CTAs an SM (shared memory, and 96 registers a thread)

template <int kBytes>
__device__ __forceinline__ void shift_copy(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}

// V > 1: every row of every tensor starts on V elements.
template <typename IO, int V, int N>
__global__ void __launch_bounds__(kShiftBwdX* kShiftBwdY, kShiftBwdCtas)
    wkv4_token_shift_backward_kernel(const ShiftBwdParams p) {
    allow_dependents();
    grid_dependency_wait();
    constexpr bool kRing = V > 1;
    constexpr int kThreads = kShiftBwdX * kShiftBwdY, kPiece = V * (int)sizeof(IO);
    constexpr int kStages = kShiftBwdStages<IO>;
    const int64_t b = blockIdx.z;
    const int64_t c = ((int64_t)blockIdx.x * kShiftBwdX + threadIdx.x) * V;
    const int64_t t0 = ((int64_t)blockIdx.y * kShiftBwdY + threadIdx.y) * p.run;
    const int64_t t1 = min(p.T, t0 + p.run);
    __shared__ float red[N][kShiftBwdY][kShiftBwdX * V];
    // [stage][x, g_0 .. g_{N-1}][thread]
    __shared__ __align__(16) unsigned char ring[kRing ? kStages * (N + 1) * kThreads * kPiece : 16];
    const int tid = threadIdx.y * kShiftBwdX + threadIdx.x;
    float acc[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[i][j] = 0.f;
    if (c < p.C && t0 < t1 && in_range(c + V - 1, p.C) && in_range(b, p.B)) {
        const int64_t row = b * p.T;
        const IO* x = static_cast<const IO*>(p.x);
        // the run's rows, and the row after it for its share of the run's last
        const int rows = (int)(t1 - t0) + (t1 < p.T ? 1 : 0);
        int64_t next = (row + t0) * p.C + c;  // the next row to be copied
        int copied = 0;
        auto slot = [&](int stage, int which) { return ring + ((stage * (N + 1) + which) * kThreads + tid) * kPiece; };
        auto copy_row = [&](int stage) {
            if (copied < rows) {
                shift_copy<kPiece>(smem_u32(slot(stage, 0)), x + next);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    shift_copy<kPiece>(smem_u32(slot(stage, i + 1)), static_cast<const IO*>(p.g[i]) + next);
                next += p.C;
                ++copied;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if constexpr (kRing) {
#pragma unroll
            for (int s = 0; s < kStages; ++s) copy_row(s);
        }
        float m[N][V], xp[V], a[V];
#pragma unroll
        for (int i = 0; i < N; ++i) load_f32<V>(p.mix[i] + c, m[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) xp[j] = a[j] = 0.f;
        if (t0 > 0) {
            load_vec<IO, V>(x + (row + t0 - 1) * p.C + c, xp);
        } else if (p.x_prev) {
            load_vec<IO, V>(static_cast<const IO*>(p.x_prev) + b * p.C + c, xp);
        }
        IO* out = static_cast<IO*>(p.gx) + (row + t0) * p.C + c;  // row t - 1's gx goes to out - C
        int stage = 0;
#pragma unroll(kRing ? 1 : 4)
        for (int t = 0; t < rows; ++t) {
            float xt[V], g[N][V], own[V], prev[V];
            if constexpr (kRing) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
                load_vec<IO, V>(reinterpret_cast<const IO*>(slot(stage, 0)), xt);
#pragma unroll
                for (int i = 0; i < N; ++i) load_vec<IO, V>(reinterpret_cast<const IO*>(slot(stage, i + 1)), g[i]);
                copy_row(stage);
                stage = stage + 1 == kStages ? 0 : stage + 1;
            } else {
                load_vec<IO, V>(x + next, xt);
#pragma unroll
                for (int i = 0; i < N; ++i) load_vec<IO, V>(static_cast<const IO*>(p.g[i]) + next, g[i]);
                next += p.C;
            }
            // row t's shares: own = sum m g to gx[t], prev = sum (1 - m) g to gx[t - 1]
#pragma unroll
            for (int j = 0; j < V; ++j) {
                own[j] = m[0][j] * g[0][j];
                prev[j] = fmaf(-m[0][j], g[0][j], g[0][j]);
#pragma unroll
                for (int i = 1; i < N; ++i) {
                    own[j] = fmaf(m[i][j], g[i][j], own[j]);
                    prev[j] += fmaf(-m[i][j], g[i][j], g[i][j]);
                }
                a[j] += prev[j];
            }
            if (t > 0) {
                store_vec<IO, V>(out - p.C, a);
            } else if (t0 == 0 && p.gx_prev) {
                store_vec<IO, V>(static_cast<IO*>(p.gx_prev) + b * p.C + c, prev);
            }
            out += p.C;
            if (t < (int)(t1 - t0)) {  // (the row after the run counts in its own run)
#pragma unroll
                for (int j = 0; j < V; ++j) {
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i][j] = fmaf(g[i][j], xt[j] - xp[j], acc[i][j]);
                    xp[j] = xt[j];
                    a[j] = own[j];
                }
            }
        }
        if (t1 == p.T) {
            if (p.gx_last) {
                float gl[V];
                load_vec<IO, V>(static_cast<const IO*>(p.gx_last) + b * p.C + c, gl);
#pragma unroll
                for (int j = 0; j < V; ++j) a[j] += gl[j];
            }
            store_vec<IO, V>(out - p.C, a);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) red[i][threadIdx.y][j * kShiftBwdX + threadIdx.x] = acc[i][j];
    __syncthreads();
    const int64_t cb = (int64_t)blockIdx.x * kShiftBwdX * V;  // the CTA's first channel
    if (p.part) {
        const int64_t prow = b * gridDim.y + blockIdx.y;
        for (int q = tid; q < N * V * kShiftBwdX; q += kThreads) {
            const int i = q / (V * kShiftBwdX), x = q % (V * kShiftBwdX);
            const int64_t ch = cb + (int64_t)(x % kShiftBwdX) * V + x / kShiftBwdX;
            float s = 0.f;
#pragma unroll
            for (int y = 0; y < kShiftBwdY; ++y) s += red[i][y][x];
            if (ch < p.C) p.part[(i * p.rows + prow) * p.C + ch] = s;
        }
        return;
    }
    // the cluster: all (y, b) of this channel block; CTA r adds every CTA's runs
    // of its share of the columns
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int n = (int)cluster.num_blocks();
    cluster.sync();
    for (int q = tid + kThreads * (int)cluster.block_rank(); q < N * V * kShiftBwdX; q += kThreads * n) {
        const int i = q / (V * kShiftBwdX), x = q % (V * kShiftBwdX);
        const int64_t ch = cb + (int64_t)(x % kShiftBwdX) * V + x / kShiftBwdX;
        float s = 0.f;
        for (int r = 0; r < n; ++r) {
            const float* const at = cluster.map_shared_rank(&red[i][0][x], r);
#pragma unroll
            for (int y = 0; y < kShiftBwdY; ++y) s += at[y * kShiftBwdX * V];
        }
        if (ch < p.C) p.gmix[i][ch] = s;
    }
    cluster.sync();  // no CTA leaves while a peer may still read its sums
}

}  // namespace wkv4
