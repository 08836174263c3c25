// Backward pass of the WKV recurrence (and of the gated one) for sm_100a.
//
// Forward, per batch row and channel (decay w, bonus u), A, D the numerator
// and denominator sums before step t:
//   Z_t = D_t + e^{u+k_t},  y_t = (A_t + e^{u+k_t} v_t) / Z_t,  out_t = s_t y_t,
//   A_{t+1} = e^w A_t + e^{k_t} v_t,  D_{t+1} = e^w D_t + e^{k_t},
// with s_t = sigmoid(r_t) (1 without a gate).  With g_t = s_t gout_t and
// al_t = g_t / Z_t the gradients of the sums run the same recurrence the
// other way,
//   P_t = dL/dA_t = al_t + e^w P_{t+1},  Q_t = dL/dD_t = -al_t y_t + e^w Q_{t+1},
// and
//   gv_t = e^{k_t} (e^u al_t + P_{t+1}),
//   gk_t = e^{k_t} (e^u al_t (v_t - y_t) + P_{t+1} v_t + Q_{t+1}),
//   gr_t = gout_t y_t s_t (1 - s_t),
//   gu   = sum_t e^{u+k_t} al_t (v_t - y_t),
//   gw   = sum_t e^w (P_{t+1} A_t + Q_{t+1} D_t).
// So there are two scans, one from each end, and the second needs the first.
//
// Layout.  A tile is 64 channels of one batch row; a warp owns L = 16 steps
// of it, a lane two adjacent channels (packed f32x2 arithmetic), a CTA NW
// warps, a cluster of NC CTAs a round of NC NW L steps.  A round's k, v, gout
// (and r) are copied to shared memory once and stay there:
//   1. each warp summarises its chunk (a, b, p) as the forward does;
//   2. the chunks are joined in the CTA (64 threads, a channel each), the
//      CTAs' aggregates read through cluster shared memory;
//   3. from the state at its start each warp walks its steps once more for
//      y_t, al_t (kept in fp32 in shared memory, over the gout and r rows
//      they replace), gr, and its share of gu and gw, then folds the chunk's
//      (P, Q) from its end;
//   4. the (P, Q) are joined the same way from the other end;
//   5. a last walk from the chunk's end writes gk, gv.
// One round covers T when NC NW L >= T: every input is read once and every
// gradient written once.  Longer sequences walk their rounds from the last to
// the first; a first kernel (wkv4_backward_summary_kernel) summarises k, v of
// every round and wkv4_backward_prefix_kernel turns that into the state at
// each round's start, so k and v are read twice.
//
// gw without the states of the last walk: inside a chunk of n steps
//   sum_t e^w (P_{t+1} A_t + Q_{t+1} D_t)
//     = sum_s al_s (A'_s - y_s D'_s) + P_n A'_n + Q_n D'_n,
// with A'_0 = D'_0 = 0, A'_{t+1} = e^w (A'_t + A_t) (the derivative of A by w
// since the chunk's start), so the ascending walk accumulates the sum and the
// chunk's end closes it.
//
// Numerics.  Forward states are (a, b, max) triples; (P, Q) is carried the
// same way, P = a 2^p, Q = b 2^p with p in fp64, scaled so that the larger of
// |a|, |b| is in [1, 2).  Within a chunk everything is held against the
// chunk's reference 2^{max k}, under the limits of the forward's
// fixed-reference path; (P, Q) may lie at most kFastStateLift above it.  Where
// a limit is passed a channel takes the exact per-step path (exact_backward_*:
// quadratic in the chunk's 16 steps, any range).  gw and gu are summed in
// fp32: a thread's steps, then the warps, then (wkv4_column_sum_kernel) the
// CTAs, in a fixed order.
#pragma once

#include <cooperative_groups.h>

#include "wkv4_chunk.cuh"

namespace wkv4 {

constexpr int kBwdL = 16;   // steps a warp chunk
constexpr int kBwdC = 64;   // channels a tile

struct BwdParams {
    int64_t B, T, C;
    int CGB;       // channel tiles a batch row
    int rounds;    // rounds of a cluster's steps
    const float* w;
    const float* u;
    const void* k;
    const void* v;
    const void* r;   // NULL: no gate
    const void* gy;
    const float* state_in;    // [3][B][C] or NULL
    const float* state_out;   // [3][B][C], read for its max when gstate_out is given
    const float* gstate_out;  // [3][B][C] or NULL (its max plane is not read)
    void* gk;
    void* gv;
    void* gr;
    float* gstate_in;  // [3][B][C] or NULL
    float* part_w;     // [rows][C] partial sums, row b NC + rank
    float* part_u;
    // rounds > 1: per round and channel the summary, then the state at the round's start
    float* ck_a;       // [rounds][B C]
    float* ck_b;
    double* ck_p;
    bool vec_load;     // every row starts on 16 bytes
    bool vec_store;    // channel pairs of gk, gv, gr may be stored as one access
};

// Shared memory of the backward kernel.  Per warp: k and v rows as loaded,
// then two fp32 planes [L][64] for al and y; gout is loaded into the end of
// the first plane and r into the end of the second, and the walk of step 3
// overwrites them (see kRawAt).
template <typename IO>
struct BwdLayout {
    static constexpr int kRow = kBwdC * (int)sizeof(IO);
    static constexpr int kTile = kBwdL * kRow;             // k or v rows of a warp
    static constexpr int kPlane = kBwdL * kBwdC * 4;       // al or y of a warp
    // The raw rows end where the plane ends.  fp32: the same bytes, row for
    // row.  16-bit: raw row j is at kPlane/2 + 128 j, plane row i at 256 i ..
    // 256 i + 255, which reaches raw rows j <= 2 i - 15 <= i for i < 16 only:
    // rows already read when steps are walked upwards (a group of 4 rows is
    // read by the whole warp before any of it is written).
    static constexpr int kRawAt = kPlane - kTile;
    static constexpr int kWarp = 2 * kTile + 2 * kPlane;
    int NW;
    __host__ __device__ size_t chunks() const { return (size_t)NW * kWarp; }
    // chunk summaries [NW][64]: p (fp64), a, b; then the CTA's two aggregates and the start triple
    __host__ __device__ size_t aggs() const { return chunks() + (size_t)NW * kBwdC * 16; }
    __host__ __device__ size_t bytes() const { return aggs() + 3 * (size_t)kBwdC * 16; }
};

// [n][64] triples in shared memory: p, then a, then b
struct Triples {
    double* p;
    float* a;
    float* b;
    __device__ __forceinline__ Triples(unsigned char* at, int n)
        : p(reinterpret_cast<double*>(at)),
          a(reinterpret_cast<float*>(at + (size_t)n * kBwdC * 8)),
          b(reinterpret_cast<float*>(at + (size_t)n * kBwdC * 12)) {}
    __device__ __forceinline__ St get(int i) const { return {a[i], b[i], p[i]}; }
    __device__ __forceinline__ void put(int i, St s) const {
        a[i] = s.a;
        b[i] = s.b;
        p[i] = s.p;
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's n rows of 64 channels from c0 of one [B][T][C] tensor (src: batch
// row b, step t0, channel 0) into shared memory; channels past C read as
// zero, rows past n are left.  vec: C and the base are multiples of 16 bytes,
// 16-byte asynchronous copies; otherwise element by element.
template <typename IO>
__device__ __forceinline__ void load_rows(unsigned char* dst, const IO* src, int64_t C, int64_t c0,
                                          int n, int lane, bool vec) {
    constexpr int kE = 16 / (int)sizeof(IO), kP = kBwdC / kE;  // elements a piece, pieces a row
    if (vec) {
        const uint32_t d = smem_u32(dst);
#pragma unroll
        for (int q = 0; q < kBwdL * kP / 32; ++q) {
            const int row = (q * 32 + lane) / kP, piece = (q * 32 + lane) % kP;
            const int64_t c = c0 + piece * kE;
            if (row < n) {
                const bool in = c < C;
                cp_async16(d + (uint32_t)(row * kBwdC * (int)sizeof(IO) + piece * 16),
                           src + (int64_t)row * C + (in ? c : 0), in ? 16 : 0);
            }
        }
    } else {
        IO* d = reinterpret_cast<IO*>(dst);
        for (int row = 0; row < n; ++row)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = lane + 32 * h;
                const int64_t c = c0 + j;
                d[row * kBwdC + j] = c < C ? src[(int64_t)row * C + c] : Io<IO>::from_f(0.f);
            }
    }
}

// (P, Q) with a common exponent: the larger magnitude brought to [1, 2).
__device__ __forceinline__ St scaled(float P, float Q, double p) {
    const float m = fmaxf(fabsf(P), fabsf(Q));
    const int e = ((__float_as_int(m) >> 23) & 0xff);
    if (m == 0.f) return empty_state();
    if (e == 0 || e == 255) return {P, Q, p};  // subnormal, or infinite / NaN: as it is
    const float s = __int_as_float((254 - e) << 23);
    return {P * s, Q * s, p + (double)(e - 127)};
}

// Gradients through the gate: g = s gout and, through the pointer, gr.
__device__ __forceinline__ float gate_grad(float gout, float y, float r, float& gr) {
    const float x = ex2(fminf(-r * kLog2e, 126.f));
    const float s = rcp_approx(1.f + x);
    const float g = gout * s;
    gr = g * y * (x * s);
    return g;
}

// One channel of one chunk for the exact per-step paths, in global memory.
template <typename IO>
struct ExactChunk {
    const IO* k;
    const IO* v;
    const IO* gy;
    const IO* r;      // NULL: no gate
    int64_t stride;
    int n;
    double w2, u2;
    St S;             // the state at the chunk's start
};

// The output y of step i from the state s before it, with 1 / Z = rz 2^{-q}
// and E = e^{u+k} / 2^q.
struct ExactOut {
    float y, rz, E;
    double q;
};
__device__ __forceinline__ ExactOut exact_out(const St& s, double x, float v, double u2) {
    const double q = fmax(s.p, u2 + x);
    const float f1 = ex2((float)(s.p - q)), f2 = ex2((float)(u2 + x - q));
    const float rz = 1.f / fmaf(f1, s.b, f2);
    return {fmaf(f1, s.a, f2 * v) * rz, rz, f2, q};
}

// Upward walk: gr, and the chunk's (P, Q) at its start from zero at its end.
template <typename IO>
__device__ __noinline__ St exact_backward_up(const ExactChunk<IO> c, IO* gr_out) {
    St s = c.S, acc = empty_state();
    for (int i = 0; i < c.n; ++i) {
        const int64_t o = (int64_t)i * c.stride;
        const float k = Io<IO>::to_f(c.k[o]), v = Io<IO>::to_f(c.v[o]);
        const ExactOut e = exact_out(s, (double)k * kLog2eD, v, c.u2);
        float g = Io<IO>::to_f(c.gy[o]);
        if (c.r) {
            float gr;
            g = gate_grad(g, e.y, Io<IO>::to_f(c.r[o]), gr);
            gr_out[o] = Io<IO>::from_f(gr);
        }
        const float al = g * e.rz;
        acc = combine(acc, scaled(al, -al * e.y, (double)i * c.w2 - e.q), 0.0);
        exact_update(s, k, v, c.w2);
    }
    return scaled(acc.a, acc.b, acc.p);
}

struct ExactGrads {
    St R;  // (P, Q) at the chunk's start
    float gw, gu;
};

// Downward walk from (P, Q) at the chunk's end: gk, gv and the chunk's whole
// gw, gu.  The state before each step is rebuilt from the chunk's start.
template <typename IO>
__device__ __noinline__ ExactGrads exact_backward_down(const ExactChunk<IO> c, St R, IO* gk_out,
                                                       IO* gv_out) {
    float gw = 0.f, gu = 0.f;
    for (int i = c.n - 1; i >= 0; --i) {
        St s = c.S;
        for (int j = 0; j < i; ++j) {
            const int64_t o = (int64_t)j * c.stride;
            exact_update(s, Io<IO>::to_f(c.k[o]), Io<IO>::to_f(c.v[o]), c.w2);
        }
        const int64_t o = (int64_t)i * c.stride;
        const float k = Io<IO>::to_f(c.k[o]), v = Io<IO>::to_f(c.v[o]);
        const double x = (double)k * kLog2eD;
        const ExactOut e = exact_out(s, x, v, c.u2);
        float g = Io<IO>::to_f(c.gy[o]);
        if (c.r) {
            float gr;
            g = gate_grad(g, e.y, Io<IO>::to_f(c.r[o]), gr);
        }
        const float al = g * e.rz, own = e.E * al;
        // the products are of the gradients' order; in fp64 their factors cannot overflow
        const double later = exp2(fmin(R.p + x, 1000.0));
        const float gut = own * (v - e.y);
        gv_out[o] = Io<IO>::from_f(own + (float)(later * R.a));
        gk_out[o] = Io<IO>::from_f(gut + (float)(later * ((double)R.a * v + R.b)));
        gu += gut;
        gw += (float)(exp2(fmin(R.p + s.p + c.w2, 1000.0)) *
                      ((double)R.a * s.a + (double)R.b * s.b));
        R = combine(R, scaled(al, -al * e.y, -e.q), c.w2);
        R = scaled(R.a, R.b, R.p);
    }
    return {R, gw, gu};
}

// Steps of a chunk starting at t.
__device__ __forceinline__ int chunk_steps(int64_t T, int64_t t, int most) {
    return (int)max((int64_t)0, min((int64_t)most, T - t));
}

// One pair's stores of a gradient row.
template <typename IO>
__device__ __forceinline__ void store_pair(IO* p, f2 x, bool vec, bool ok0, bool ok1) {
    if (vec && ok1) {
        Pair<IO>::store(p, x);
    } else {
        if (ok0) p[0] = Io<IO>::from_f(lo(x));
        if (ok1) p[1] = Io<IO>::from_f(hi(x));
    }
}

template <typename IO, bool kGate>
__global__ void __launch_bounds__(256, 2) wkv4_backward_kernel(const BwdParams p) {
    namespace cg = cooperative_groups;
    allow_dependents();
    grid_dependency_wait();
    using Lay = BwdLayout<IO>;
    constexpr int L = kBwdL;
    extern __shared__ __align__(16) unsigned char smem[];
    const int NW = blockDim.x >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int NC = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const Lay lay{NW};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = 2 * lane;
    const int64_t tile = blockIdx.x / NC;
    const int64_t b = tile / p.CGB, c0 = (tile - b * p.CGB) * kBwdC;
    const int64_t T = p.T, C = p.C, BC = p.B * C;
    const int Ts = NW * L;                    // steps of this CTA in a round
    const int64_t round_steps = (int64_t)NC * Ts;
    const int64_t c = c0 + col;
    const bool ok0 = c < C, ok1 = c + 1 < C;

    unsigned char* const wbase = smem + (size_t)warp * Lay::kWarp;
    const IO* const sk = reinterpret_cast<const IO*>(wbase);
    const IO* const sv = reinterpret_cast<const IO*>(wbase + Lay::kTile);
    unsigned char* const plane1 = wbase + 2 * Lay::kTile;
    unsigned char* const plane2 = plane1 + Lay::kPlane;
    const IO* const sg = reinterpret_cast<const IO*>(plane1 + Lay::kRawAt);
    const IO* const sr = reinterpret_cast<const IO*>(plane2 + Lay::kRawAt);
    float* const sal = reinterpret_cast<float*>(plane1);
    float* const sy = reinterpret_cast<float*>(plane2);
    const Triples chunk(smem + lay.chunks(), NW);
    const Triples aggF(smem + lay.aggs(), 1), aggR(smem + lay.aggs() + kBwdC * 16, 1),
        start(smem + lay.aggs() + 2 * kBwdC * 16, 1);

    // every global access below is (b T + t) C + c for t < T, c < C, or b C + c
    if (!in_range(b, p.B)) return;
    PairConsts cc;
    pair_consts(p.w, p.u, c, C, cc);

    // the 64 threads that join chunks and CTAs: a channel each
    const int jc = threadIdx.x;
    const bool joiner = jc < kBwdC;
    const bool jok = joiner && c0 + jc < C;
    const int64_t jch = b * C + c0 + jc;
    const double jw2 = jok ? (double)p.w[c0 + jc] * kLog2eD : 0.0;
    St Rcarry = empty_state();  // (P, Q) after the current round's last step
    if (jok && p.gstate_out)
        Rcarry = scaled(p.gstate_out[jch], p.gstate_out[BC + jch],
                        -(double)p.state_out[2 * BC + jch] * kLog2eD);

    f2 gw_sum = 0ull, gu_sum = 0ull;
    const f2 l2e = pk(kLog2e, kLog2e);

    for (int round = p.rounds - 1; round >= 0; --round) {
        const int64_t t_round = (int64_t)round * round_steps;
        const int64_t t_cta = t_round + (int64_t)rank * Ts;
        const int64_t t0 = t_cta + warp * L;
        const int n = chunk_steps(T, t0, L);
        const int64_t at = (b * T + t0) * C;  // element offset of the chunk's first row
        if (n > 0) {
            load_rows<IO>(wbase, static_cast<const IO*>(p.k) + at, C, c0, n, lane, p.vec_load);
            load_rows<IO>(wbase + Lay::kTile, static_cast<const IO*>(p.v) + at, C, c0, n, lane,
                          p.vec_load);
            cp_async_commit();
            load_rows<IO>(plane1 + Lay::kRawAt, static_cast<const IO*>(p.gy) + at, C, c0, n, lane,
                          p.vec_load);
            if constexpr (kGate)
                load_rows<IO>(plane2 + Lay::kRawAt, static_cast<const IO*>(p.r) + at, C, c0, n,
                              lane, p.vec_load);
        } else {
            cp_async_commit();
        }
        cp_async_commit();
        // the state at the round's start
        St carry = empty_state();
        if (jok) {
            if (p.rounds > 1) {
                const int64_t i = (int64_t)round * BC + jch;
                carry = {p.ck_a[i], p.ck_b[i], p.ck_p[i]};
            } else if (p.state_in) {
                carry = load_state_log2(p.state_in, BC, jch);
            }
        }
        cp_async_wait<1>();
        __syncwarp();

        // 1. the chunk's summary
        PairRef ref;
        St sum[2];
        chunk_phase1<IO, L>(ref, sk, sv, kBwdC, col, n, cc, sum);
        __syncthreads();  // the last round's suffixes have been read
        chunk.put(warp * kBwdC + col, sum[0]);
        chunk.put(warp * kBwdC + col + 1, sum[1]);
        __syncthreads();

        // 2. prefixes within the CTA, then over the cluster
        if (joiner) {
            St acc = empty_state();
            for (int q = 0; q < NW; ++q) {
                const St x = chunk.get(q * kBwdC + jc);
                chunk.put(q * kBwdC + jc, acc);
                acc = combine(acc, x, (double)chunk_steps(T, t_cta + q * L, L) * jw2);
            }
            aggF.put(jc, acc);
        }
        cluster.sync();
        if (joiner) {
            for (int q = 0; q < rank; ++q) {
                const St x{*cluster.map_shared_rank(aggF.a + jc, q),
                           *cluster.map_shared_rank(aggF.b + jc, q),
                           *cluster.map_shared_rank(aggF.p + jc, q)};
                carry = combine(carry, x, (double)chunk_steps(T, t_round + (int64_t)q * Ts, Ts) * jw2);
            }
            start.put(jc, carry);
        }
        __syncthreads();

        // 3. the chunk from the state at its start: y, al, gr, and (P, Q) of the chunk alone
        St S[2];
        bool fast[2];
        float a0[2], b0[2];
        const double before = (double)(chunk_steps(T, t_cta, warp * L));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            S[j] = combine(start.get(col + j), chunk.get(warp * kBwdC + col + j), before * cc.w2[j]);
            const double lift = S[j].p - (double)ref.kref[j];
            fast[j] = ref.fast[j] && lift <= (double)(kFastStateLift * kLog2e);
            const float sc = ex2((float)lift);
            a0[j] = S[j].a * sc;
            b0[j] = S[j].b * sc;
        }
        cp_async_wait<0>();
        __syncwarp();
        const f2 nref = pk(-ref.kref[0], -ref.kref[1]);
        f2 A = pk(a0[0], a0[1]), D = pk(b0[0], b0[1]);
        f2 Ap = 0ull, Dp = 0ull;  // derivatives by w since the chunk's start
        f2 gw = 0ull, gu = 0ull;
        IO* const gr = kGate ? static_cast<IO*>(p.gr) + at + c : nullptr;
#pragma unroll 1
        for (int q = 0; q < n; q += 4) {
            f2 gg[4], rr[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                gg[s] = Pair<IO>::load(sg + (q + s) * kBwdC + col);
                if constexpr (kGate) rr[s] = Pair<IO>::load(sr + (q + s) * kBwdC + col);
            }
            __syncwarp();  // the rows this group overwrites have been read by every lane
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int i = q + s;
                if (i < n) {
                    const f2 e = ex2_2(fma2(Pair<IO>::load(sk + i * kBwdC + col), l2e, nref));
                    const f2 v = Pair<IO>::load(sv + i * kBwdC + col);
                    const f2 ee = mul2(cc.eu, e);
                    const f2 rz = rcp2(add2(D, ee));
                    const f2 y = mul2(fma2(ee, v, A), rz);
                    const f2 ny = y ^ 0x8000000080000000ull;
                    f2 g = gg[s];
                    if constexpr (kGate) {
                        const f2 x0 = mul2(rr[s], pk(-kLog2e, -kLog2e));
                        const f2 x = pk(ex2(fminf(lo(x0), 126.f)), ex2(fminf(hi(x0), 126.f)));
                        const f2 sgm = rcp2(add2(pk(1.f, 1.f), x));
                        g = mul2(g, sgm);
                        store_pair(gr + (int64_t)i * C, mul2(mul2(g, y), mul2(x, sgm)), p.vec_store,
                                   ok0 && fast[0], ok1 && fast[1]);
                    }
                    const f2 al = mul2(g, rz);
                    *reinterpret_cast<f2*>(sal + i * kBwdC + col) = al;
                    *reinterpret_cast<f2*>(sy + i * kBwdC + col) = y;
                    gu = fma2(mul2(ee, al), add2(v, ny), gu);
                    gw = fma2(al, fma2(ny, Dp, Ap), gw);
                    const f2 t1 = mul2(cc.ew, A), t2 = mul2(cc.ew, D);
                    Ap = fma2(cc.ew, Ap, t1);
                    Dp = fma2(cc.ew, Dp, t2);
                    A = fma2(e, v, t1);
                    D = add2(t2, e);
                }
            }
        }
        f2 P = 0ull, Q = 0ull;
#pragma unroll 4
        for (int i = n - 1; i >= 0; --i) {
            const f2 al = *reinterpret_cast<const f2*>(sal + i * kBwdC + col);
            const f2 y = *reinterpret_cast<const f2*>(sy + i * kBwdC + col);
            P = fma2(cc.ew, P, al);
            Q = fma2(cc.ew, Q, mul2(al, y ^ 0x8000000080000000ull));
        }
        St loc[2];
        const float Pj[2] = {lo(P), hi(P)}, Qj[2] = {lo(Q), hi(Q)};
        auto exact_chunk = [&](int j) {
            return ExactChunk<IO>{static_cast<const IO*>(p.k) + at + c + j,
                                  static_cast<const IO*>(p.v) + at + c + j,
                                  static_cast<const IO*>(p.gy) + at + c + j,
                                  kGate ? static_cast<const IO*>(p.r) + at + c + j : nullptr,
                                  C, n, cc.w2[j], (double)cc.u[j] * kLog2eD, S[j]};
        };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (n == 0 || !(j ? ok1 : ok0)) {
                loc[j] = empty_state();
            } else if (fast[j]) {
                loc[j] = scaled(Pj[j], Qj[j], -(double)ref.kref[j]);
            } else {
                loc[j] = exact_backward_up<IO>(exact_chunk(j), gr + j);
            }
        }
        __syncthreads();  // the prefixes have been read
        chunk.put(warp * kBwdC + col, loc[0]);
        chunk.put(warp * kBwdC + col + 1, loc[1]);
        __syncthreads();

        // 4. suffixes within the CTA, then over the cluster
        if (joiner) {
            St acc = empty_state();
            for (int q = NW - 1; q >= 0; --q) {
                const St x = chunk.get(q * kBwdC + jc);
                chunk.put(q * kBwdC + jc, acc);
                // what comes after the chunk reaches its start through the chunk's own decay
                acc = combine(acc, x, (double)chunk_steps(T, t_cta + q * L, L) * jw2);
            }
            aggR.put(jc, acc);
        }
        cluster.sync();
        if (joiner) {
            for (int q = NC - 1; q >= 0; --q) {
                if (q == rank) start.put(jc, Rcarry);
                const St x{*cluster.map_shared_rank(aggR.a + jc, q),
                           *cluster.map_shared_rank(aggR.b + jc, q),
                           *cluster.map_shared_rank(aggR.p + jc, q)};
                Rcarry = combine(Rcarry, x, (double)chunk_steps(T, t_round + (int64_t)q * Ts, Ts) * jw2);
            }
        }
        __syncthreads();

        // 5. the last walk, downwards
        St R[2];
        bool fastR[2];
        float p0[2], q0[2];
        const int64_t t_next = t0 + L;
        const double after = (double)chunk_steps(T, t_next, (NW - 1 - warp) * L);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const St x = combine(start.get(col + j), chunk.get(warp * kBwdC + col + j), after * cc.w2[j]);
            R[j] = scaled(x.a, x.b, x.p);
            const double lift = R[j].p + (double)ref.kref[j];
            fastR[j] = fast[j] && lift <= (double)(kFastStateLift * kLog2e);
            const float sc = ex2((float)lift);
            p0[j] = R[j].a * sc;
            q0[j] = R[j].b * sc;
        }
        P = pk(p0[0], p0[1]);
        Q = pk(q0[0], q0[1]);
        gw = fma2(P, Ap, fma2(Q, Dp, gw));
        IO* const gk = static_cast<IO*>(p.gk) + at + c;
        IO* const gv = static_cast<IO*>(p.gv) + at + c;
#pragma unroll 4
        for (int i = n - 1; i >= 0; --i) {
            const f2 e = ex2_2(fma2(Pair<IO>::load(sk + i * kBwdC + col), l2e, nref));
            const f2 v = Pair<IO>::load(sv + i * kBwdC + col);
            const f2 al = *reinterpret_cast<const f2*>(sal + i * kBwdC + col);
            const f2 ny = *reinterpret_cast<const f2*>(sy + i * kBwdC + col) ^ 0x8000000080000000ull;
            const f2 ea = mul2(cc.eu, al);
            store_pair(gv + (int64_t)i * C, mul2(e, add2(ea, P)), p.vec_store, ok0 && fastR[0],
                       ok1 && fastR[1]);
            store_pair(gk + (int64_t)i * C, mul2(e, fma2(ea, add2(v, ny), fma2(P, v, Q))),
                       p.vec_store, ok0 && fastR[0], ok1 && fastR[1]);
            P = fma2(cc.ew, P, al);
            Q = fma2(cc.ew, Q, mul2(al, ny));
        }
        float gwj[2] = {lo(gw), hi(gw)}, guj[2] = {lo(gu), hi(gu)};
        const float Pe[2] = {lo(P), hi(P)}, Qe[2] = {lo(Q), hi(Q)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool ok = j ? ok1 : ok0;
            if (n > 0 && ok) {
                if (fastR[j]) {
                    R[j] = {Pe[j], Qe[j], -(double)ref.kref[j]};
                } else {
                    const ExactGrads x = exact_backward_down<IO>(exact_chunk(j), R[j], gk + j, gv + j);
                    R[j] = x.R;
                    gwj[j] = x.gw;
                    guj[j] = x.gu;
                }
            } else {
                gwj[j] = guj[j] = 0.f;
            }
            if (t0 == 0 && ok && p.gstate_in) {
                const int64_t ch = b * C + c + j;
                const double f = exp2(fmin(R[j].p + (double)p.state_in[2 * BC + ch] * kLog2eD, 1000.0));
                const float ga = (float)(f * R[j].a), gb = (float)(f * R[j].b);
                const float sa = p.state_in[ch], sb = p.state_in[BC + ch];
                p.gstate_in[ch] = ga;
                p.gstate_in[BC + ch] = gb;
                p.gstate_in[2 * BC + ch] = fmaf(sa, ga, sb * gb);
            }
        }
        gw_sum = add2(gw_sum, pk(gwj[0], gwj[1]));
        gu_sum = add2(gu_sum, pk(guj[0], guj[1]));
    }

    // the CTA's sums of gw, gu
    __syncthreads();
    float* const red = reinterpret_cast<float*>(smem + lay.chunks());  // [2][NW][64]
    *reinterpret_cast<f2*>(red + warp * kBwdC + col) = gw_sum;
    *reinterpret_cast<f2*>(red + (NW + warp) * kBwdC + col) = gu_sum;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kBwdC; i += blockDim.x) {
        const int which = i / kBwdC, ch = i % kBwdC;
        if (c0 + ch < C) {
            float s = 0.f;
            for (int q = 0; q < NW; ++q) s += red[(which * NW + q) * kBwdC + ch];
            (which ? p.part_u : p.part_w)[(b * NC + rank) * C + c0 + ch] = s;
        }
    }
    cluster.sync();  // no CTA leaves while a peer may still read its aggregates
}

// Summary of every round's k, v (several rounds): CTA (tile, round), each
// warp walking its NC chunks of L steps with the next chunk's rows in flight.
template <typename IO>
__global__ void __launch_bounds__(256) wkv4_backward_summary_kernel(const BwdParams p, int NC) {
    allow_dependents();
    grid_dependency_wait();
    constexpr int L = kBwdL, kTile = BwdLayout<IO>::kTile;
    extern __shared__ __align__(16) unsigned char smem[];
    const int NW = blockDim.x >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = 2 * lane;
    const int64_t tile = blockIdx.x, round = blockIdx.y;
    const int64_t b = tile / p.CGB, c0 = (tile - b * p.CGB) * kBwdC;
    const int64_t T = p.T, C = p.C, BC = p.B * C;
    const int64_t t_round = round * NC * NW * L, t_warp = t_round + (int64_t)warp * NC * L;
    if (!in_range(b, p.B)) return;
    PairConsts cc;
    pair_consts(p.w, p.u, c0 + col, C, cc);
    unsigned char* const buf = smem + (size_t)warp * 4 * kTile;  // two stages of k, v
    const Triples chunk(smem + (size_t)NW * 4 * kTile, NW);
    auto load = [&](int q) {
        const int64_t t = t_warp + (int64_t)q * L;
        const int n = q < NC ? chunk_steps(T, t, L) : 0;
        unsigned char* const d = buf + (q & 1) * 2 * kTile;
        if (n > 0) {
            const int64_t at = (b * T + t) * C;
            load_rows<IO>(d, static_cast<const IO*>(p.k) + at, C, c0, n, lane, p.vec_load);
            load_rows<IO>(d + kTile, static_cast<const IO*>(p.v) + at, C, c0, n, lane, p.vec_load);
        }
        cp_async_commit();
    };
    St acc[2] = {empty_state(), empty_state()};
    load(0);
    for (int q = 0; q < NC; ++q) {
        load(q + 1);
        cp_async_wait<1>();
        __syncwarp();
        const int n = chunk_steps(T, t_warp + (int64_t)q * L, L);
        const IO* const sk = reinterpret_cast<const IO*>(buf + (q & 1) * 2 * kTile);
        PairRef ref;
        St sum[2];
        chunk_phase1<IO, L>(ref, sk, sk + kTile / sizeof(IO), kBwdC, col, n, cc, sum);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = combine(acc[j], sum[j], (double)n * cc.w2[j]);
        __syncwarp();  // read by every lane before the stage is loaded again
    }
    chunk.put(warp * kBwdC + col, acc[0]);
    chunk.put(warp * kBwdC + col + 1, acc[1]);
    __syncthreads();
    const int jc = threadIdx.x;
    if (jc < kBwdC && c0 + jc < C) {
        const double w2 = (double)p.w[c0 + jc] * kLog2eD;
        St s = empty_state();
        for (int q = 0; q < NW; ++q)
            s = combine(s, chunk.get(q * kBwdC + jc),
                        (double)chunk_steps(T, t_round + (int64_t)q * NC * L, NC * L) * w2);
        const int64_t i = round * BC + b * C + c0 + jc;
        p.ck_a[i] = s.a;
        p.ck_b[i] = s.b;
        p.ck_p[i] = s.p;
    }
}

// The rounds' summaries -> the state at each round's start, in place.
__global__ void __launch_bounds__(128) wkv4_backward_prefix_kernel(const BwdParams p, int64_t round_steps) {
    allow_dependents();
    grid_dependency_wait();
    const int64_t BC = p.B * p.C;
    const int64_t ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (ch >= BC) return;
    const double w2 = (double)p.w[ch % p.C] * kLog2eD;
    St s = p.state_in ? load_state_log2(p.state_in, BC, ch) : empty_state();
    constexpr int kAhead = 8;  // rounds loaded at once: the chain waits for memory once per group
    for (int r0 = 0; r0 < p.rounds; r0 += kAhead) {
        St x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t i = (int64_t)(r0 + j) * BC + ch;
            if (r0 + j < p.rounds) x[j] = {p.ck_a[i], p.ck_b[i], p.ck_p[i]};
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (r0 + j < p.rounds) {
                const int64_t i = (int64_t)(r0 + j) * BC + ch;
                p.ck_a[i] = s.a;
                p.ck_b[i] = s.b;
                p.ck_p[i] = s.p;
                // every round but the last is whole, and nothing follows the last
                s = combine(s, x[j], (double)round_steps * w2);
            }
        }
    }
}

// out[j][c] = sum over rows of part[j][row][c]: up to three column sums, a CTA
// of 32 columns x 8 row groups, joined in a fixed order.
struct ColumnSumParams {
    const float* part;  // [n][rows][C]
    float* out[3];
    int64_t rows, C;
};

__global__ void __launch_bounds__(256) wkv4_column_sum_kernel(const ColumnSumParams p) {
    allow_dependents();
    grid_dependency_wait();
    __shared__ float red[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + x;
    const float* const part = p.part + (int64_t)blockIdx.y * p.rows * p.C;
    float s = 0.f;
    if (c < p.C) {
#pragma unroll 4
        for (int64_t r = y; r < p.rows; r += 8) s += part[r * p.C + c];
    }
    red[y][x] = s;
    __syncthreads();
    if (y == 0 && c < p.C) {
#pragma unroll
        for (int q = 1; q < 8; ++q) s += red[q][x];
        p.out[blockIdx.y][c] = s;
    }
}

}  // namespace wkv4
