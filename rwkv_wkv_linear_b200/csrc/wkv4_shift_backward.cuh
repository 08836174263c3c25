// Backward pass of the token shift.  Forward, for up to three mixes m_i,
//   out_i[b,t] = m_i x[b,t] + (1 - m_i) x[b,t-1],  x[b,-1] = x_prev[b],
// so with g_i the gradient of out_i
//   gx[b,t]    = sum_i m_i g_i[b,t] + sum_i (1 - m_i) g_i[b,t+1]   (t + 1 < T)
//              (+ gx_last[b] at t = T - 1: x_last = x[:, T-1] feeds the next call),
//   gx_prev[b] = sum_i (1 - m_i) g_i[b,0],
//   gm_i       = sum_{b,t} g_i[b,t] (x[b,t] - x[b,t-1]).
//
// An HBM stream: a thread owns V channels of one batch row (as packed pairs) and
// walks a run of steps with the row before in registers (x[t-1], and
// sum_i m_i g_i[t-1], which waits for the next row's share before it is stored),
// so every input is read once (plus one row a run) and gx written once.  Its
// rows come through a ring of a few rows of its own in shared memory, filled by
// asynchronous copies: a thread waits for nobody, and what is in flight does not
// cost registers.  What counts for HBM is the bytes a warp reads in a row: with
// 8 channels of 16 bits (512 bytes) B=4, T=1024, C=5120 takes 39.8 us (5.3 TB/s
// of the 210 MB, the column sums' launch included), with 4 (256 bytes) 47.1,
// whatever the number of instructions.  The gm_i partial sums of the CTA's runs are joined in shared
// memory.  Where the CTAs of one channel block are at most 8 they are one
// cluster and add up their sums through its shared memory; otherwise each
// writes a row and wkv4_column_sum_kernel adds the rows.  Both in a fixed
// order.  All arithmetic in fp32, rounded once at the stores.
#pragma once

#include <cooperative_groups.h>

#include "wkv4_device.cuh"
#include "wkv4_chunk.cuh"  // packed f32x2
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
constexpr int kShiftBwdWide = 8;  // channels a thread of the wide form (16-bit types: 16 bytes a row)
// CTAs an SM, by shared memory and registers
__host__ __device__ constexpr int shift_bwd_ctas(int V) { return V == kShiftBwdWide ? 3 : 5; }
// rows of a thread in flight: 32 KB a CTA
__host__ __device__ constexpr int shift_bwd_stages(int piece) { return piece == 16 ? 4 : 8; }

template <int kBytes>
__device__ __forceinline__ void shift_copy(uint32_t dst, const void* src) {
    if constexpr (kBytes == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
    }
}

// V channels as packed pairs (V == 1: the upper half zero).
template <int V>
__device__ __forceinline__ void to_pairs(const float (&x)[V], f2 (&y)[(V + 1) / 2]) {
#pragma unroll
    for (int j = 0; j < (V + 1) / 2; ++j) y[j] = pk(x[2 * j], 2 * j + 1 < V ? x[2 * j + 1 < V ? 2 * j + 1 : 0] : 0.f);
}
template <typename IO, int V>
__device__ __forceinline__ void load_pairs(const IO* p, f2 (&y)[(V + 1) / 2]) {
    float x[V];
    load_vec<IO, V>(p, x);
    to_pairs(x, y);
}
template <typename IO, int V>
__device__ __forceinline__ void store_pairs(IO* p, const f2 (&y)[(V + 1) / 2]) {
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = j % 2 ? hi(y[j / 2]) : lo(y[j / 2]);
    store_vec<IO, V>(p, x);
}

// V > 1: every row of every tensor starts on V elements.
template <typename IO, int V, int N>
__global__ void __launch_bounds__(kShiftBwdX* kShiftBwdY, shift_bwd_ctas(V))
    wkv4_token_shift_backward_kernel(const ShiftBwdParams p) {
    allow_dependents();
    grid_dependency_wait();
    constexpr bool kRing = V > 1;
    constexpr int kThreads = kShiftBwdX * kShiftBwdY, kPiece = V * (int)sizeof(IO);
    constexpr int kStages = shift_bwd_stages(kPiece);
    const int64_t b = blockIdx.z;
    const int64_t c = ((int64_t)blockIdx.x * kShiftBwdX + threadIdx.x) * V;
    const int64_t t0 = ((int64_t)blockIdx.y * kShiftBwdY + threadIdx.y) * p.run;
    const int64_t t1 = min(p.T, t0 + p.run);
    __shared__ float red[N][kShiftBwdY][kShiftBwdX * V];
    // [stage][x, g_0 .. g_{N-1}][thread]
    __shared__ __align__(16) unsigned char ring[kRing ? kStages * (N + 1) * kThreads * kPiece : 16];
    const int tid = threadIdx.y * kShiftBwdX + threadIdx.x;
    constexpr int H = (V + 1) / 2;  // channel pairs (V == 1: the upper half idle)
    f2 acc[N][H];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < H; ++j) acc[i][j] = 0ull;
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
        f2 m[N][H], rest[N][H], xp[H], a[H];  // mixes, 1 - mixes
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float y[V];
            load_f32<V>(p.mix[i] + c, y);
            to_pairs(y, m[i]);
#pragma unroll
            for (int j = 0; j < H; ++j) rest[i][j] = fma2(m[i][j], pk(-1.f, -1.f), pk(1.f, 1.f));
        }
#pragma unroll
        for (int j = 0; j < H; ++j) xp[j] = a[j] = 0ull;
        if (t0 > 0) {
            load_pairs<IO, V>(x + (row + t0 - 1) * p.C + c, xp);
        } else if (p.x_prev) {
            load_pairs<IO, V>(static_cast<const IO*>(p.x_prev) + b * p.C + c, xp);
        }
        IO* out = static_cast<IO*>(p.gx) + (row + t0) * p.C + c;  // row t - 1's gx goes to out - C
        int stage = 0;
#pragma unroll(kRing ? 1 : 4)
        for (int t = 0; t < rows; ++t) {
            f2 xt[H], g[N][H];
            if constexpr (kRing) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
                load_pairs<IO, V>(reinterpret_cast<const IO*>(slot(stage, 0)), xt);
#pragma unroll
                for (int i = 0; i < N; ++i) load_pairs<IO, V>(reinterpret_cast<const IO*>(slot(stage, i + 1)), g[i]);
                copy_row(stage);
                stage = stage + 1 == kStages ? 0 : stage + 1;
            } else {
                load_pairs<IO, V>(x + next, xt);
#pragma unroll
                for (int i = 0; i < N; ++i) load_pairs<IO, V>(static_cast<const IO*>(p.g[i]) + next, g[i]);
                next += p.C;
            }
            // row t's share of gx[t - 1], sum (1 - m) g (of gx_prev for the first row)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < H; ++j) a[j] = fma2(rest[i][j], g[i][j], a[j]);
            if (t > 0) {
                store_pairs<IO, V>(out - p.C, a);
            } else if (t0 == 0 && p.gx_prev) {
                store_pairs<IO, V>(static_cast<IO*>(p.gx_prev) + b * p.C + c, a);
            }
            out += p.C;
            if (t < (int)(t1 - t0)) {  // (the row after the run counts in its own run)
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const f2 dx = fma2(xp[j], pk(-1.f, -1.f), xt[j]);
                    a[j] = mul2(m[0][j], g[0][j]);
#pragma unroll
                    for (int i = 1; i < N; ++i) a[j] = fma2(m[i][j], g[i][j], a[j]);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i][j] = fma2(g[i][j], dx, acc[i][j]);
                    xp[j] = xt[j];
                }
            }
        }
        if (t1 == p.T) {
            if (p.gx_last) {
                f2 gl[H];
                load_pairs<IO, V>(static_cast<const IO*>(p.gx_last) + b * p.C + c, gl);
#pragma unroll
                for (int j = 0; j < H; ++j) a[j] = add2(a[j], gl[j]);
            }
            store_pairs<IO, V>(out - p.C, a);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) red[i][threadIdx.y][j * kShiftBwdX + threadIdx.x] = j % 2 ? hi(acc[i][j / 2]) : lo(acc[i][j / 2]);
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
