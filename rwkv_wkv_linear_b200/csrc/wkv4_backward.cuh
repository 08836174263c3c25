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
// Layout.  A tile is 64 channels of one batch row; a warp owns L steps of it (32,
// or 16 in fp32, whose rows are twice as long), a lane two adjacent channels
// (packed f32x2 arithmetic), a CTA NW warps, a cluster of NC CTAs a round of
// NC NW L steps.  A round's k, v, gout (and r) are copied to shared memory once
// and stay there:
//   1. each warp summarises its chunk (a, b, p) as the forward does;
//   2. the chunks are joined in the CTA (64 threads, a channel each), the
//      CTAs' aggregates read through cluster shared memory;
//   3. from the state at its start each warp walks its steps once more for
//      y_t, al_t (kept in fp32 in tensor memory: al_t and -al_t y_t of a
//      channel pair are four columns of the lane), gr, and its share of gu and
//      gw, and folds the chunk's (P, Q) on the way;
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
// Numerics.  Sums are carried as (a, b, p): A = a 2^p, D = b 2^p with an integer
// p, so that joins scale by exact powers of two and no exponential or fp64
// enters them; the decay over n steps is a factor in (1/2, 1] and an integer
// exponent, worked out once a thread.  (P, Q) is carried the same way.
// Within a chunk everything is held against the chunk's reference 2^R,
// R = ceil(max k log2 e), under limits like those of the forward's
// fixed-reference path (kBwdRange, kBwdLift).  Where a limit is passed a
// channel takes the exact per-step path (exact_backward_*: quadratic in the
// chunk's steps, fp64 exponents).
//
// Masks.  Where no usual key came yet, a state is made of the keys that stand
// for a mask (-1e9, -1e30) alone, so their exponents count too, and they do not
// all fit 32 bits.  Exponents up to +-kNear (1.02e9 nats) are held as they are;
// keys and maxima beyond count as kNear, and from 2^50 on as one value further
// out, kStill, that a decay does not move: next to a max that large a decay is
// lost in the forward's fp64 as well.  So two steps' weights are told apart
// unless both keys lie past 1.02e9 nats on the same side of 2^50.
//
// gw and gu are summed in fp32: a thread's steps, then the warps, then
// (wkv4_column_sum_kernel) the CTAs, in a fixed order.
//
// What bounds it.  B=4, T=1024, C=5120, bf16, gated: 95.3 us for 294 MB (3.1 TB/s)
// and 161 warp instructions a step of 64 channels at 2.2 a clock and SM: issue,
// with 12 warps an SM (by shared memory and registers alike) to cover the
// instructions' latencies, not HBM.  A fourth CTA an SM costs more in spills
// than it hides; al, y in tensor memory instead of shared memory are what makes
// three fit.  B=1, T=16384, C=2048, fp32, with k, v read twice: 229 us for 940 MB
// (4.1 TB/s).  Short calls are a chain of latencies: B=1, T=48, C=768 5.9 us.
// Masked steps are not fast: with the last quarter of the 14B width's keys at
// -inf, or its first at -1e9, the exact path makes it 822 or 702 us.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "wkv4_chunk.cuh"

namespace wkv4 {

constexpr int kBwdC = 64;   // channels a tile
constexpr int kBwdWarps = 4;    // warps a CTA
constexpr int kBwdMaxCtas = 16;  // CTAs a cluster
constexpr int kBwdPitch = 68;   // sums a row of the chunks' (2 lanes a channel, 2 chunks each, meet no bank twice)
constexpr int kSumBytes = 12;   // a sum in memory: p, a, b
constexpr int kMuteNone = -1, kMuteAll = -2;

struct BwdParams {
    int64_t B, T, C;
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
    int* ck_p;         // [rounds][B C]
    float* ck_a;
    float* ck_b;
    uint32_t wait_rounds;  // limit of each bounded wait
    int mute;              // checked builds' fault injection: the rank that pushes no sums, kMuteNone or kMuteAll
    int NC;            // CTAs a cluster
    bool vec_load;     // every row of k, v, gout, r starts on 16 bytes
    bool vec_store;    // channel pairs of gk, gv, gr may be stored as one access
};

// Shared memory of the backward kernel: per warp the rows of k, v, gout (and
// r) as loaded, then the warps' chunk sums [NW], the sum after a round [2],
// four barriers and the tensor-memory base, and the other CTAs' sums [NC].
template <typename IO, int L, bool kGate>
struct BwdLayout {
    static constexpr int kTile = L * kBwdC * (int)sizeof(IO);  // one tensor's rows of a warp
    static constexpr int kWarp = (kGate ? 4 : 3) * kTile;
    static constexpr int kChunks = kBwdWarps * kWarp;
    static constexpr int kCarry = kChunks + kBwdWarps * kBwdPitch * kSumBytes;
    static constexpr int kBars = kCarry + 2 * kBwdC * kSumBytes;
    static constexpr int kPeers = kBars + 6 * 8;
    // al_t and -al_t y_t of a step's channel pair: 4 columns of tensor memory.
    // A CTA holds its columns from start to end, and an allocation that cannot
    // be met waits for another CTA's release.  None has to: a CTA of this
    // kernel takes at least its columns' share (of 512) of the SM's shared
    // memory, and of its registers, so whatever set of CTAs an SM takes on --
    // of this kernel and of the others that hold to either share -- needs no
    // more columns than there are.
    static constexpr int kColumns = 4 * L;
    static constexpr int kShare = kColumns * (228 * 1024 / 512) - 1024;  // (1 KB a CTA is the system's)
    __host__ __device__ static constexpr int bytes(int NC) {
        return kPeers + NC * kBwdC * kSumBytes > kShare ? kPeers + NC * kBwdC * kSumBytes : kShare;
    }
    // CTAs an SM that the shared memory allows, which the registers are shared by
    static constexpr int kCtas = 3 * (bytes(8) + 1024) <= 228 * 1024 ? 3 : 2;  // an SM
    static_assert(32 * kBwdWarps * 128 >= kColumns * (65536 / 512), "registers below the columns' share");
};

// Limits of the fixed-reference walk: the spread of a chunk's keys in nats
// (+ min(0, u)), so that 1 / Z <= 2^58, and how far the state before the chunk
// or the (P, Q) behind it may lie above the reference, in powers of two.
constexpr float kBwdRange = 40.f;
constexpr int kBwdLift = 63;
// Exponents (log2 units).  Decays carry one on by 2^20 in a chunk and 1.1e8 in a
// round, after which it is brought back to kReach.
constexpr int kNear = 1480000000;
constexpr int kReach = 1520000000;
constexpr int kStillFrom = 1650000000;  // from here on (in magnitude) a decay does not move it:
constexpr int kStill = 1700000000;      // exponents of 2^50 and more
constexpr int kNone = -1950000000;      // an empty sum's, below every other
constexpr double kStillD = 0x1p100;     // kStill as an fp64 exponent, which swallows decays by itself

// A = a 2^p, D = b 2^p.
struct Sum {
    float a, b;
    int p;
};
// 2^x = f 2^i
struct Decay {
    float f;
    int i;
};

__device__ __forceinline__ Sum empty_sum() { return {0.f, 0.f, kNone}; }
// 2^d, 0 below the normal range, d <= 127
__device__ __forceinline__ float pow2i(int d) { return __int_as_float(max(d + 127, 0) << 23); }
// 2^{low - high} (the distance may take all 32 bits)
__device__ __forceinline__ float pow2_below(int low, int high) {
    // bits of 1.0 less the distance in the exponent's place, as one multiply-add (B=4, T=1024, C=5120
    // 95.0 us against 95.5 with a shift and a subtraction)
    int r;
    asm("mad.lo.s32 %0, %1, -8388608, 1065353216;" : "=r"(r) : "r"((int)min((unsigned)high - (unsigned)low, 127u)));
    return __int_as_float(r);
}
__device__ __forceinline__ bool is_still(int p) { return abs(p) >= kStillFrom; }
// The exponent of a key or of a state's max.
__device__ __forceinline__ double key2(float k) {
    const double x = (double)k * kLog2eD;
    if (!(fabs(x) > (double)kNear) || isinf(k)) return x;
    return copysign(fabs(x) < 0x1p50 ? (double)kNear : kStillD, x);
}
// w in log2 units as two floats.  Decays faster than 2^-32768 a step are taken
// as that: nothing passes either, and n steps of it stay an integer exponent
// (likewise growth above 2^32768).
struct Rate {
    float hi, lo;
};
__device__ __forceinline__ Rate rate_of(float w) {
    const float hi = w * kLog2e;
    if (!(fabsf(hi) <= 32768.f)) return {hi > 0.f ? 32768.f : -32768.f, 0.f};
    constexpr float kLog2eLo = (float)(kLog2eD - (double)kLog2e);
    return {hi, fmaf(w, kLog2e, -hi) + w * kLog2eLo};
}
// e^{n w}: the product split exactly into its rounded value and the rest
__device__ __forceinline__ Decay decay_of(Rate r, int n) {
    const float x = (float)n * r.hi;
    const float c = ceilf(x);
    // (exp2f, not ex2.approx: the factor is applied once a chunk, and its error
    // grows with the number of chunks a slow decay remembers)
    return {exp2f((x - c) + (fmaf((float)n, r.hi, -x) + (float)n * r.lo)), (int)c};
}
__device__ __forceinline__ Sum decayed(Sum x, Decay d) {
    const bool still = is_still(x.p);
    const float f = still ? 1.f : d.f;
    return {x.a * f, x.b * f, still ? x.p : x.p + d.i};
}
// a 2^p, b 2^p with a fractional p
__device__ __forceinline__ Sum sum_of(float a, float b, double p) {
    if (a == 0.f && b == 0.f) return empty_sum();
    if (fabs(p) >= (double)kStillFrom) {
        if (p <= -INFINITY) return empty_sum();
        return {a, b, p < 0.0 ? -kStill : kStill};
    }
    const double c = p == p ? ceil(p) : 0.0;  // (a NaN goes on in a and b)
    const float f = exp2f((float)(p - c));
    return {a * f, b * f, (int)c};
}
__device__ __forceinline__ double exponent_of(int p) {
    if (!is_still(p)) return (double)p;
    return p > 0 ? kStillD : p >= -kStill ? -kStillD : kEmptyMax2;
}
__device__ __forceinline__ St st_of(Sum x) { return {x.a, x.b, exponent_of(x.p)}; }

// x, decayed by d, and y added.
__device__ __forceinline__ Sum join(Sum x, Sum y, Decay d) {
    const bool still = is_still(x.p);
    const int px = still ? x.p : x.p + d.i, p = max(px, y.p);
    const float fx = pow2_below(px, p) * (still ? 1.f : d.f), fy = pow2_below(y.p, p);
    return {fmaf(x.a, fx, y.a * fy), fmaf(x.b, fx, y.b * fy), p};
}

// x and y added.
__device__ __forceinline__ Sum join(Sum x, Sum y) {
    const int p = max(x.p, y.p);
    const float fx = pow2_below(x.p, p), fy = pow2_below(y.p, p);
    return {fmaf(x.a, fx, y.a * fy), fmaf(x.b, fx, y.b * fy), p};
}

// A lane's sum from another lane of the group of P that shares a channel.
template <int P>
__device__ __forceinline__ Sum lane_sum(Sum x, int from) {
    return {__shfl_sync(0xffffffffu, x.a, from, P), __shfl_sync(0xffffffffu, x.b, from, P),
            __shfl_sync(0xffffffffu, x.p, from, P)};
}

// The larger magnitude brought to [1, 2), and an exponent that decays have
// carried past kReach back to it.
__device__ __forceinline__ Sum scaled(float a, float b, int p) {
    const int e = (__float_as_int(fmaxf(fabsf(a), fabsf(b))) >> 23) & 0xff;
    if (e == 0 || e == 255 || is_still(p))  // zero, subnormal, infinite or NaN: as it is
        return a == 0.f && b == 0.f ? empty_sum() : Sum{a, b, p};
    const float s = __int_as_float((254 - e) << 23);
    return {a * s, b * s, min(max(p + e - 127, -kReach), kReach)};
}

// [n] sums in shared memory: p, then a, then b
struct Sums {
    int* p;
    float* a;
    float* b;
    __device__ __forceinline__ Sums(unsigned char* at, int n)
        : p(reinterpret_cast<int*>(at)),
          a(reinterpret_cast<float*>(at + (size_t)n * 4)),
          b(reinterpret_cast<float*>(at + (size_t)n * 8)) {}
    __device__ __forceinline__ Sum get(int i) const { return {a[i], b[i], p[i]}; }
    __device__ __forceinline__ void put(int i, Sum s) const {
        a[i] = s.a;
        b[i] = s.b;
        p[i] = s.p;
    }
    // columns i, i + 1 (i even)
    __device__ __forceinline__ void put2(int i, Sum s, Sum t) const {
        *reinterpret_cast<float2*>(a + i) = make_float2(s.a, t.a);
        *reinterpret_cast<float2*>(b + i) = make_float2(s.b, t.b);
        *reinterpret_cast<int2*>(p + i) = make_int2(s.p, t.p);
    }
    __device__ __forceinline__ void get2(int i, Sum (&s)[2]) const {
        const float2 x = *reinterpret_cast<const float2*>(a + i), y = *reinterpret_cast<const float2*>(b + i);
        const int2 z = *reinterpret_cast<const int2*>(p + i);
        s[0] = {x.x, y.x, z.x};
        s[1] = {x.y, y.y, z.y};
    }
};

// The sum written to entry i of the same array of the cluster's CTA `rank`,
// its 12 bytes completing on that CTA's barrier `bar`.
__device__ __forceinline__ void push_sum(const Sums& at, int i, Sum s, uint64_t* bar, int rank) {
    const uint32_t mb = mapa_u32(smem_u32(bar), (uint32_t)rank);
    auto put = [&](const void* p, uint32_t x) {
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                         mapa_u32(smem_u32(p), (uint32_t)rank)),
                     "r"(x), "r"(mb)
                     : "memory");
    };
    put(at.a + i, __float_as_uint(s.a));
    put(at.b + i, __float_as_uint(s.b));
    put(at.p + i, (uint32_t)s.p);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's n rows of 64 channels from c0 of N [B][T][C] tensors (src: the first
// row, channel 0) into shared memory, L rows a tensor one after another;
// channels past C read as zero, rows past n are left.  vec: every row starts
// on 16 bytes, 16-byte asynchronous copies; otherwise element by element, 8
// rows of every tensor in flight.
template <typename IO, int L, int N>
__device__ __forceinline__ void load_rows(unsigned char* dst, const IO* const (&src)[N], int64_t C, int c0,
                                          int n, int lane, bool vec) {
    constexpr int kE = 16 / (int)sizeof(IO), kP = kBwdC / kE;  // elements a piece, pieces a row
    constexpr int kTile = L * kBwdC * (int)sizeof(IO);
    if (vec) {
        constexpr int kR = 32 / kP;  // rows a pass of the warp
        const int row = lane / kP, piece = lane % kP;
        const int c = c0 + piece * kE;
        const int bytes = c < C ? 16 : 0;
        const uint32_t d = smem_u32(dst) + (uint32_t)(row * kBwdC * (int)sizeof(IO) + piece * 16);
        const int64_t o = (int64_t)row * C + (c < C ? c : 0);
#pragma unroll
        for (int h = 0; h < N; ++h) {
            const IO* s = src[h] + o;
#pragma unroll
            for (int q = 0; q < L / kR; ++q) {
                if (q * kR + row < n)
                    cp_async16(d + (uint32_t)(h * kTile + q * kR * kBwdC * (int)sizeof(IO)), s, bytes);
                s += (int64_t)kR * C;
            }
        }
    } else {
        IO* d = reinterpret_cast<IO*>(dst) + lane;
        const bool ok0 = c0 + lane < C, ok1 = c0 + lane + 32 < C;
        int64_t o = c0 + lane;
        constexpr int kG = 8;
#pragma unroll 1
        for (int q = 0; q < n; q += kG) {
            IO x[N][kG][2];
#pragma unroll
            for (int h = 0; h < N; ++h)
#pragma unroll
                for (int i = 0; i < kG; ++i) {
                    const IO* s = src[h] + o + (int64_t)i * C;
                    x[h][i][0] = ok0 && q + i < n ? s[0] : Io<IO>::from_f(0.f);
                    x[h][i][1] = ok1 && q + i < n ? s[32] : Io<IO>::from_f(0.f);
                }
#pragma unroll
            for (int h = 0; h < N; ++h)
#pragma unroll
                for (int i = 0; i < kG; ++i) {
                    d[(h * L + q + i) * kBwdC] = x[h][i][0];
                    d[(h * L + q + i) * kBwdC + 32] = x[h][i][1];
                }
            o += (int64_t)kG * C;
        }
    }
}

// The same with an fp64 exponent, for the exact paths.  (One that swallows decays
// would swallow the change of scale.)
__device__ __forceinline__ St scaled_st(float P, float Q, double p) {
    const Sum x = scaled(P, Q, 0);
    if (x.p == kNone) return empty_state();
    return fabs(p) >= (double)kStillFrom ? St{P, Q, p} : St{x.a, x.b, p + (double)x.p};
}

// min(x, most), NaN where x is (fminf would return `most`).
__device__ __forceinline__ float at_most(float x, float most) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(most));
    return y;
}

// Gradients through the gate: g = s gout and, through the pointer, gr.
__device__ __forceinline__ float gate_grad(float gout, float y, float r, float& gr) {
    const float x = ex2(at_most(-r * kLog2e, 126.f));
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

// The state after a step of exponent x.
__device__ __forceinline__ void exact_advance(St& s, double x, float v, double w2) {
    const double q = fmax(s.p + w2, x);
    const float f1 = ex2((float)(s.p + w2 - q)), f2 = ex2((float)(x - q));
    s.a = fmaf(f1, s.a, f2 * v);
    s.b = fmaf(f1, s.b, f2);
    s.p = q;
}
// A chunk's sums from the empty state, rows in shared memory.
template <typename IO>
__device__ __noinline__ St exact_summary(const IO* sk, const IO* sv, int n, double w2) {
    St s = empty_state();
    for (int i = 0; i < n; ++i) exact_advance(s, key2(Io<IO>::to_f(sk[i * kBwdC])), Io<IO>::to_f(sv[i * kBwdC]), w2);
    return s;
}

// Upward walk: gr, and the chunk's (P, Q) at its start from zero at its end.
template <typename IO>
__device__ __noinline__ St exact_backward_up(const ExactChunk<IO> c, IO* gr_out) {
    St s = c.S, acc = empty_state();
    for (int i = 0; i < c.n; ++i) {
        const int64_t o = (int64_t)i * c.stride;
        const double x = key2(Io<IO>::to_f(c.k[o]));
        const float v = Io<IO>::to_f(c.v[o]);
        const ExactOut e = exact_out(s, x, v, c.u2);
        float g = Io<IO>::to_f(c.gy[o]);
        if (c.r) {
            float gr;
            g = gate_grad(g, e.y, Io<IO>::to_f(c.r[o]), gr);
            gr_out[o] = Io<IO>::from_f(gr);
        }
        const float al = g * e.rz;
        acc = combine(acc, scaled_st(al, -al * e.y, (double)i * c.w2 - e.q), 0.0);
        exact_advance(s, x, v, c.w2);
    }
    return scaled_st(acc.a, acc.b, acc.p);
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
            exact_advance(s, key2(Io<IO>::to_f(c.k[o])), Io<IO>::to_f(c.v[o]), c.w2);
        }
        const int64_t o = (int64_t)i * c.stride;
        const float v = Io<IO>::to_f(c.v[o]);
        const double x = key2(Io<IO>::to_f(c.k[o]));
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
        R = combine(R, scaled_st(al, -al * e.y, -e.q), c.w2);
        R = scaled_st(R.a, R.b, R.p);
    }
    return {R, gw, gu};
}

__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_acquire() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Steps of a chunk starting at t.
__device__ __forceinline__ int chunk_steps(int T, int t, int most) { return max(0, min(most, T - t)); }

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

// A stored pair as floats.  bf16: the halves of a float's bits, two operations.
template <typename IO>
__device__ __forceinline__ f2 load_f2(const IO* p) {
    if constexpr (std::is_same<IO, __nv_bfloat16>::value) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
        return pku(x << 16, x & 0xffff0000u);
    } else {
        return Pair<IO>::load(p);
    }
}

constexpr f2 kSigns = 0x8000000080000000ull;

// A pair's decay and bonus.
//
// Step i of a chunk decays by ew[i % 4]: neighbouring floats about e^w whose
// running product stays within a rounding of e^{(i + 1) w}.  One float for
// every step would be off by up to 2^-25 a step in one direction, 32 times
// over along a chunk: the largest error of gw under slow decays.
struct BwdConsts {
    f2 ew[4], eu;
    float w[2], u[2];
    __device__ __forceinline__ static void decays(float w, float (&m)[4]) {
        // e^w = m0 + l, l the rest that m0 leaves out (known where e^w is near 1;
        // a fast decay is not applied often enough to need it)
        float m0 = expf(w), l = 0.f;
        if (fabsf(w) < 0.5f) {
            const float x = expm1f(w);
            m0 = 1.f + x;
            l = x - (m0 - 1.f);
        }
        float c = 0.f;  // what the product so far has left out
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c += l;
            m[i] = m0 + c;
            c -= m[i] - m0;
        }
    }
    __device__ __forceinline__ void load(const float* gw, const float* gu, int64_t c, int64_t C) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            w[j] = c + j < C ? __ldg(gw + c + j) : 0.f;
            u[j] = c + j < C ? __ldg(gu + c + j) : 0.f;
        }
    }
    __device__ __forceinline__ void derive() {
        float m[2][4];
        decays(w[0], m[0]);
        decays(w[1], m[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) ew[i] = pk(m[0][i], m[1][i]);
        eu = pk(expf(u[0]), expf(u[1]));
    }
};

// A pair's chunk reference (a whole power of two at or above its largest key)
// and whether each channel may be held against it.
struct BwdRef {
    float R[2];
    bool fast[2];
};

// The chunk's sums from the empty state (n >= 0 steps).
template <typename IO>
__device__ __forceinline__ void bwd_summary(const IO* sk, const IO* sv, int col, int n,
                                            const BwdConsts& cc, BwdRef& ref, Sum (&sum)[2]) {
    sum[0] = sum[1] = empty_sum();
    ref.fast[0] = ref.fast[1] = false;
    ref.R[0] = ref.R[1] = 0.f;
    if (n == 0) return;
    typename Pair<IO>::Raw mx = Pair<IO>::raw(sk + col), mn = mx;
#pragma unroll 8
    for (int i = 1; i < n; ++i) Pair<IO>::minmax(Pair<IO>::raw(sk + i * kBwdC + col), mx, mn);
    float kmax[2], kmin[2];
    Pair<IO>::bounds(mx, mn, kmax, kmin);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float R = ceilf(kmax[j] * kLog2e);
        ref.fast[j] = kmax[j] - kmin[j] <= kBwdRange + fminf(0.f, cc.u[j]) && cc.u[j] <= kFastMaxU &&
                      cc.w[j] <= kFastMaxW && fabsf(R) <= 4194304.f;
        ref.R[j] = fabsf(R) <= 4194304.f ? R : 0.f;
    }
    const f2 l2e = pk(kLog2e, kLog2e), nref = pk(-ref.R[0], -ref.R[1]);
    f2 A = 0ull, D = 0ull;
    auto step = [&](int i, int s) {
        const f2 e = ex2_2(fma2(load_f2<IO>(sk + i * kBwdC + col), l2e, nref));
        A = fma2(cc.ew[s], A, mul2(e, load_f2<IO>(sv + i * kBwdC + col)));
        D = fma2(cc.ew[s], D, e);
    };
    int q = 0;
#pragma unroll 2
    for (; q + 4 <= n; q += 4) {
#pragma unroll
        for (int s = 0; s < 4; ++s) step(q + s, s);
    }
#pragma unroll
    for (int s = 0; s < 3; ++s)
        if (q + s < n) step(q + s, s);
    const float Aj[2] = {lo(A), hi(A)}, Dj[2] = {lo(D), hi(D)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (ref.fast[j]) {  // D is a normal positive number: bring it to [1, 2)
            const int e = (__float_as_int(Dj[j]) >> 23) & 0xff;
            const float s = __int_as_float((254 - e) << 23);
            sum[j] = {Aj[j] * s, Dj[j] * s, (int)ref.R[j] + e - 127};
        } else {
            const St x = exact_summary<IO>(sk + col + j, sv + col + j, n, (double)cc.w[j] * kLog2eD);
            sum[j] = sum_of(x.a, x.b, x.p);
        }
    }
}

// One warp's chunk in shared memory.
template <typename IO>
struct BwdChunk {
    const IO* k;
    const IO* v;
    const IO* gy;
    const IO* r;
    uint32_t stash;  // tensor memory: al_t, -al_t y_t of the lane's pair, 4 columns a step
    int col, n;
};

// Warp-wide: 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
    // the wait is tied to the registers, so no use of them is scheduled before it
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// What the upward walk leaves: shares of gw, gu, the derivatives of A, D by w,
// and (P, Q) of the chunk alone times 2^kUpShift.
struct BwdUp {
    f2 gw, gu, Ap, Dp, P, Q;
};
// The weight e^{iw} of step i in the chunk's (P, Q) starts at 2^40, so that
// under a fast decay it stays a float as long as al (up to 2^58 g) can make up
// for it; 2^98 times a gradient of 2^29 is still in range.
constexpr int kUpShift = 40;

// Step 3.  kPlain: a whole chunk with every lane's two channels present, on the
// fixed-reference path and stored as pairs.
template <typename IO, int L, bool kGate, bool kPlain>
__device__ __forceinline__ void bwd_walk_up(const BwdChunk<IO>& ch, const BwdConsts& cc, f2 nref, f2 A,
                                            f2 D, IO* gr, int64_t C, bool vec, bool s0, bool s1, BwdUp& o) {
    const f2 l2e = pk(kLog2e, kLog2e), one = pk(1.f, 1.f), m1 = pk(-1.f, -1.f);
    f2 Ap = 0ull, Dp = 0ull, gw = 0ull, gu = 0ull, P = 0ull, Q = 0ull;
    f2 f = pk(0x1p40f, 0x1p40f);
#pragma unroll 1
    for (int q = 0; q < (kPlain ? L : ch.n); q += 4) {
        uint32_t st[16];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int i = q + s;
            if (kPlain || i < ch.n) {
                const f2 e = ex2_2(fma2(load_f2<IO>(ch.k + i * kBwdC + ch.col), l2e, nref));
                const f2 v = load_f2<IO>(ch.v + i * kBwdC + ch.col);
                const f2 ee = mul2(cc.eu, e);
                const f2 rz = rcp2(add2(D, ee));
                const f2 ny = mul2(mul2(fma2(ee, v, A), m1), rz);
                f2 g = load_f2<IO>(ch.gy + i * kBwdC + ch.col);
                if constexpr (kGate) {
                    const f2 x0 = mul2(load_f2<IO>(ch.r + i * kBwdC + ch.col), pk(-kLog2e, -kLog2e));
                    // (above 2^126 the gate is 0 to within its rounding, and x s stays finite)
                    const f2 x = pk(ex2(at_most(lo(x0), 126.f)), ex2(at_most(hi(x0), 126.f)));
                    const f2 sg = rcp2(add2(one, x));
                    g = mul2(g, sg);
                    const f2 grv = mul2(mul2(g, ny), mul2(x, sg)) ^ kSigns;
                    if constexpr (kPlain)
                        Pair<IO>::store(gr + (int64_t)i * C, grv);
                    else
                        store_pair(gr + (int64_t)i * C, grv, vec, s0, s1);
                }
                const f2 al = mul2(g, rz);
                const f2 nay = mul2(al, ny);
                st[4 * s] = (uint32_t)al;
                st[4 * s + 1] = (uint32_t)(al >> 32);
                st[4 * s + 2] = (uint32_t)nay;
                st[4 * s + 3] = (uint32_t)(nay >> 32);
                gu = fma2(mul2(ee, al), add2(v, ny), gu);
                gw = fma2(al, fma2(ny, Dp, Ap), gw);
                P = fma2(f, al, P);
                Q = fma2(f, nay, Q);
                f = mul2(f, cc.ew[s]);
                Ap = mul2(cc.ew[s], add2(Ap, A));
                Dp = mul2(cc.ew[s], add2(Dp, D));
                // (one rounding a step: where one key outweighs the rest, A and D
                // drift apart by it and y D' - A' is what they differ by)
                A = fma2(cc.ew[s], A, mul2(e, v));
                D = fma2(cc.ew[s], D, e);
            } else {
                st[4 * s] = st[4 * s + 1] = st[4 * s + 2] = st[4 * s + 3] = 0;
            }
        }
        __syncwarp();  // tensor-memory accesses are warp-collective
        tmem_st16(ch.stash + 4 * q, st);
    }
    tmem_wait_st();
    o = {gw, gu, Ap, Dp, P, Q};
}

// Step 5: gk, gv from (P, Q) at the chunk's end; (P, Q) at its start in P, Q.
// With h = e^u al + P and j = -e^u al y + Q: gv = e h, gk = e (h v + j).
template <typename IO, int L, bool kPlain>
__device__ __forceinline__ void bwd_walk_down(const BwdChunk<IO>& ch, const BwdConsts& cc, f2 nref, f2& P,
                                              f2& Q, IO* gk, IO* gv, int64_t C, bool vec, bool s0, bool s1) {
    const f2 l2e = pk(kLog2e, kLog2e);
    const int n = kPlain ? L : ch.n;
#pragma unroll 1
    for (int q = (n - 1) & ~7; q >= 0; q -= 8) {
        uint32_t st[32];
        __syncwarp();
        tmem_ld32(ch.stash + 4 * q, st);
#pragma unroll
        for (int s = 7; s >= 0; --s) {
            const int i = q + s;
            if (kPlain || i < n) {
                const f2 e = ex2_2(fma2(load_f2<IO>(ch.k + i * kBwdC + ch.col), l2e, nref));
                const f2 v = load_f2<IO>(ch.v + i * kBwdC + ch.col);
                const f2 al = pku(st[4 * s], st[4 * s + 1]), nay = pku(st[4 * s + 2], st[4 * s + 3]);
                const f2 h = fma2(cc.eu, al, P), j = fma2(cc.eu, nay, Q);
                const f2 xv = mul2(e, h), xk = mul2(e, fma2(h, v, j));
                if constexpr (kPlain) {
                    Pair<IO>::store(gv + (int64_t)i * C, xv);
                    Pair<IO>::store(gk + (int64_t)i * C, xk);
                } else {
                    store_pair(gv + (int64_t)i * C, xv, vec, s0, s1);
                    store_pair(gk + (int64_t)i * C, xk, vec, s0, s1);
                }
                P = fma2(cc.ew[s & 3], P, al);
                Q = fma2(cc.ew[s & 3], Q, nay);
            }
        }
    }
}

// gk of a step with nothing before it: y is v, so the step's own share of it (and
// of gu) is 0, not what the approximate reciprocal leaves of v - y, which may be
// all there is.  From (P, Q) behind it, against the reference 2^R.
template <typename IO>
__device__ __noinline__ IO first_step_gk(IO k, IO v, float R, float P, float Q) {
    return Io<IO>::from_f(ex2(fmaf(Io<IO>::to_f(k), kLog2e, -R)) * fmaf(P, Io<IO>::to_f(v), Q));
}

// kOne: T fits one round.  The loop over rounds and what lives across it fall
// away, and with them the spills at 168 registers (B=4, T=1024, C=5120, bf16,
// gated: 95.7 us against 105.6; B=8, T=1024, C=768, fp16: 34.4 against 37.3).
template <typename IO, int L, bool kGate, bool kOne>
__global__ void __launch_bounds__(32 * kBwdWarps, BwdLayout<IO, L, kGate>::kCtas) wkv4_backward_kernel(const BwdParams p) {
    namespace cg = cooperative_groups;
    allow_dependents();
    grid_dependency_wait();
    using Lay = BwdLayout<IO, L, kGate>;
    constexpr int NW = kBwdWarps, Ts = NW * L;  // steps of a chunk, of a CTA in a round
    constexpr int P = NW / 2;              // threads that join a channel's chunks, two chunks each
    constexpr unsigned kAll = 0xffffffffu;
    extern __shared__ __align__(16) unsigned char smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int NC = p.NC, rank = (int)cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = 2 * lane;
    const int c0 = (int)blockIdx.y * kBwdC;  // grid: the cluster's CTAs, channel tiles, batch rows
    const int T = (int)p.T, rounds = kOne ? 1 : p.rounds, last = rounds - 1;
    const int64_t C = p.C, BC = p.B * C;
    const int round_steps = NC * Ts;
    const int64_t c = c0 + col;
    const bool ok0 = c < C, ok1 = c + 1 < C;
    const int b = blockIdx.z;
    // every global access below is (b T + t) C + c for b < B, t < T, c < C, or b C + c
    if (!in_range(b, p.B)) return;

    unsigned char* const wbase = smem + warp * Lay::kWarp;
    const Sums chunk(smem + Lay::kChunks, NW * kBwdPitch);
    // CTA q's sums: those of the ranks below this one on the way up, above on the way down
    auto peer = [&](int q) { return Sums(smem + Lay::kPeers + q * (kBwdC * kSumBytes), kBwdC); };
    const Sums after(smem + Lay::kCarry, 2 * kBwdC);            // (P, Q) after a round, two in turn
    // barriers: the lower ranks' forward sums, the higher ranks' (P, Q), the two rows of `after`
    uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + Lay::kBars);
    uint32_t* const tslot = reinterpret_cast<uint32_t*>(bar + 4);
    // A bounded wait that runs out sets the CTA's flag and the error word: from then
    // on the CTA waits for, arms and pushes nothing (its results are reported
    // bad), and stays until the cluster's other CTAs are done, whose sums may
    // still be on their way to it.
    volatile int* const s_fail = reinterpret_cast<volatile int*>(tslot + 1);
    bool failed = false;  // as this thread knows it
    auto wait = [&](int which, uint32_t parity) {
        if (failed || mbar_wait_cluster_bounded(bar + which, parity, p.wait_rounds)) return;
        atomicOr(&g_device_error, kErrExchangeWait);
        failed = true;
        *s_fail = 1;
    };
    const bool muted = p.mute == rank || p.mute == kMuteAll;
    // a round's rows of this warp: k and v, then (a second group) gout and r
    auto load_round = [&](int round) {
        const int t0 = round * round_steps + rank * Ts + warp * L;
        const int n = chunk_steps(T, t0, L);
        const int64_t at = ((int64_t)b * T + t0) * C;
        const IO* const kv[2] = {static_cast<const IO*>(p.k) + at, static_cast<const IO*>(p.v) + at};
        load_rows<IO, L>(wbase, kv, C, c0, n, lane, p.vec_load);
        cp_async_commit();
        if constexpr (kGate) {
            const IO* const gr[2] = {static_cast<const IO*>(p.gy) + at, static_cast<const IO*>(p.r) + at};
            load_rows<IO, L>(wbase + 2 * Lay::kTile, gr, C, c0, n, lane, p.vec_load);
        } else {
            const IO* const g[1] = {static_cast<const IO*>(p.gy) + at};
            load_rows<IO, L>(wbase + 2 * Lay::kTile, g, C, c0, n, lane, p.vec_load);
        }
        cp_async_commit();
    };
    // a round's rows of this warp brought to L2 (32 lanes, 128 bytes each)
    auto prefetch_round = [&](int round) {
        constexpr int kLanes = 32 / L;
        const int t = round * round_steps + rank * Ts + warp * L + lane / kLanes;
        const int cl = c0 + (lane % kLanes) * (kBwdC / kLanes);
        if (t < T && cl < C) {
            const int64_t o = ((int64_t)b * T + t) * C + cl;
            prefetch_l2(static_cast<const IO*>(p.k) + o);
            prefetch_l2(static_cast<const IO*>(p.v) + o);
            prefetch_l2(static_cast<const IO*>(p.gy) + o);
            if constexpr (kGate) prefetch_l2(static_cast<const IO*>(p.r) + o);
        }
    };
    // w and u first: behind the rows' copies they would wait for them
    const int jc = threadIdx.x / P, part = threadIdx.x % P;
    const bool jok = c0 + jc < C;
    const float jw = jok ? __ldg(p.w + c0 + jc) : 0.f;
    BwdConsts cc;
    cc.load(p.w, p.u, c, C);
    if (threadIdx.x < 4) {  // each thread fences the barrier it has set up
        mbar_init(bar + threadIdx.x, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) *s_fail = 0;
    if (warp == 0) tmem_alloc(tslot, Lay::kColumns);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    // Every CTA's barriers are set up before a peer's sum may arrive.  (Relaxed:
    // each barrier has its own fence, and a release would wait for the rows.)
    cluster_arrive_relaxed();
    load_round(last);
    // the lane quarter of tensor memory that this warp reaches
    const uint32_t taddr = *tslot + ((uint32_t)warp << 21);
    BwdChunk<IO> ch{reinterpret_cast<const IO*>(wbase), reinterpret_cast<const IO*>(wbase + Lay::kTile),
                    reinterpret_cast<const IO*>(wbase + 2 * Lay::kTile),
                    reinterpret_cast<const IO*>(wbase + (kGate ? 3 : 2) * Lay::kTile), taddr, col, 0};

    cc.derive();
    // this thread's part in the joins: chunks 2 part, 2 part + 1 of channel jc,
    // and CTAs q0 .. q0 + qn - 1 of the cluster
    const Rate rate = rate_of(jw);
    const Decay dL = decay_of(rate, L), d2 = decay_of(rate, 2 * L), d4 = decay_of(rate, 4 * L),
                dT = decay_of(rate, Ts);
    const Decay d_before = decay_of(rate, 2 * part * L), d_after = decay_of(rate, (NW - 2 - 2 * part) * L);
    const int qn = (NC + P - 1) / P, q0 = min(part * qn, NC), q1 = min(q0 + qn, NC);
    // from the end of CTA min(q1, rank) - 1 to this CTA's start; from the start
    // of CTA max(q0, rank + 1) to this CTA's end
    const Decay d_up = decay_of(rate, (rank - min(q1, rank)) * Ts);
    const Decay d_down = decay_of(rate, (max(q0, rank + 1) - (rank + 1)) * Ts);
    cluster_wait_acquire();

    f2 gw_sum = 0ull, gu_sum = 0ull;
    // the rounds from the last to the first; (P, Q) goes from turn to turn through
    // the two rows of `after`
#pragma unroll 1
    for (int round = last; round >= 0; --round) {
        const int turn = last - round;
        const uint32_t parity = turn & 1;
        const bool handed = turn > 0;  // this round goes on from the one after it
        const int t0 = round * round_steps + rank * Ts + warp * L;
        const int n = ch.n = chunk_steps(T, t0, L);
        const int64_t at = ((int64_t)b * T + t0) * C;  // element offset of the chunk's first row
        const int64_t jch = (int64_t)b * C + c0 + jc;
        if (handed) {
            __syncwarp();  // the last round's rows have been read by every lane
            load_round(round);
            failed |= *s_fail != 0;  // (no thread waits between the last round's end and this one's first barrier)
        }
        if (threadIdx.x == 0 && !failed) {  // what this round's barriers will receive
            if (rank > 0) mbar_arrive_expect_tx(bar, (uint32_t)rank * kBwdC * kSumBytes);
            if (rank < NC - 1) mbar_arrive_expect_tx(bar + 1, (uint32_t)(NC - 1 - rank) * kBwdC * kSumBytes);
            if (rank > 0 && handed) mbar_arrive_expect_tx(bar + 2 + ((turn - 1) & 1), kBwdC * kSumBytes);
        }
        // the next round's rows while this one is waited for
        if (round > 0) prefetch_round(round - 1);
        // the state at the round's start
        Sum carry = empty_sum();
        if (jok && part == 0) {
            if (rounds > 1) {
                const int64_t i = (int64_t)round * BC + jch;
                carry = {p.ck_a[i], p.ck_b[i], p.ck_p[i]};
            } else if (p.state_in) {
                carry = sum_of(p.state_in[jch], p.state_in[BC + jch], key2(p.state_in[2 * BC + jch]));
            }
        }
        cp_async_wait<1>();
        __syncwarp();

        // 1. the chunk's summary
        BwdRef ref;
        {
            Sum sum[2];
            bwd_summary<IO>(ch.k, ch.v, col, n, cc, ref, sum);
            chunk.put2(warp * kBwdPitch + col, sum[0], sum[1]);
        }
        __syncthreads();

        // 2. the state at every chunk's start: a scan over the CTA's chunks, the
        // lower ranks' sums, and the state at the round's start
        {
            const int i0 = 2 * part * kBwdPitch + jc, i1 = i0 + kBwdPitch;
            const Sum x0 = chunk.get(i0);
            Sum y = join(x0, chunk.get(i1), dL);
            Sum o = lane_sum<P>(y, part - 1);
            if (part >= 1) y = join(o, y, d2);
            if constexpr (P == 4) {
                o = lane_sum<P>(y, part - 2);
                if (part >= 2) y = join(o, y, d4);
            }
            const Sum total = lane_sum<P>(y, P - 1);
            Sum ex = lane_sum<P>(y, part - 1);
            if (part == 0) ex = empty_sum();
            for (int q = rank + 1 + part; q < NC && !muted && !failed; q += P)
                push_sum(peer(rank), jc, total, bar, q);
            Sum s = carry;  // part 0: the round's start; the others: empty
            if (rank > 0) {
                wait(0, parity);
                for (int q = q0; q < min(q1, rank); ++q) s = join(s, peer(q).get(jc), dT);
                s = decayed(s, d_up);
#pragma unroll
                for (int h = 1; h < P; h *= 2) s = join(s, lane_sum<P>(s, part ^ h));
            } else {
                s = lane_sum<P>(s, 0);
            }
            const Sum S0 = join(s, ex, d_before);
            chunk.put(i0, S0);
            chunk.put(i1, join(S0, x0, dL));
        }
        __syncthreads();

        // 3. the chunk from the state at its start
        Sum S[2];
        chunk.get2(warp * kBwdPitch + col, S);
        bool fast[2];
        float a0[2], b0[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int lift = S[j].p - (int)ref.R[j];
            fast[j] = ref.fast[j] && lift <= kBwdLift;
            const float sc = pow2i(min(lift, 127));
            a0[j] = S[j].a * sc;
            b0[j] = S[j].b * sc;
        }
        cp_async_wait<0>();
        __syncwarp();
        const f2 nref = pk(-ref.R[0], -ref.R[1]);
        IO* const gr = kGate ? static_cast<IO*>(p.gr) + at + c : nullptr;
        BwdUp up;
        const bool plain = __all_sync(kAll, n == L && p.vec_store && ok1 && fast[0] && fast[1]);
        if (plain) {
            bwd_walk_up<IO, L, kGate, true>(ch, cc, nref, pk(a0[0], a0[1]), pk(b0[0], b0[1]), gr, C, true, true,
                                         true, up);
        } else {
            bwd_walk_up<IO, L, kGate, false>(ch, cc, nref, pk(a0[0], a0[1]), pk(b0[0], b0[1]), gr, C,
                                          p.vec_store, ok0 && fast[0], ok1 && fast[1], up);
        }
        auto exact_chunk = [&](int j) {
            return ExactChunk<IO>{static_cast<const IO*>(p.k) + at + c + j,
                                  static_cast<const IO*>(p.v) + at + c + j,
                                  static_cast<const IO*>(p.gy) + at + c + j,
                                  kGate ? static_cast<const IO*>(p.r) + at + c + j : nullptr,
                                  C, n, (double)cc.w[j] * kLog2eD, (double)cc.u[j] * kLog2eD, st_of(S[j])};
        };
        {
            Sum loc[2];
            const float Pj[2] = {lo(up.P), hi(up.P)}, Qj[2] = {lo(up.Q), hi(up.Q)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (n == 0 || !(j ? ok1 : ok0)) {
                    loc[j] = empty_sum();
                } else if (fast[j]) {
                    loc[j] = scaled(Pj[j], Qj[j], -(int)ref.R[j] - kUpShift);
                } else {
                    const St x = exact_backward_up<IO>(exact_chunk(j), gr + j);
                    const Sum y = sum_of(x.a, x.b, x.p);
                    loc[j] = scaled(y.a, y.b, y.p);
                }
            }
            chunk.put2(warp * kBwdPitch + col, loc[0], loc[1]);
        }
        __syncthreads();

        // 4. (P, Q) at every chunk's end, the same from the other side
        {
            const int i0 = 2 * part * kBwdPitch + jc, i1 = i0 + kBwdPitch;
            const Sum x1 = chunk.get(i1);
            Sum y = join(x1, chunk.get(i0), dL);
            Sum o = lane_sum<P>(y, part + 1);
            if (part < P - 1) y = join(o, y, d2);
            if constexpr (P == 4) {
                o = lane_sum<P>(y, part + 2);
                if (part < P - 2) y = join(o, y, d4);
            }
            const Sum total = lane_sum<P>(y, 0);
            Sum ex = lane_sum<P>(y, part + 1);
            if (part == P - 1) ex = empty_sum();
            failed |= *s_fail != 0;
            for (int q = rank - 1 - part; q >= 0 && !muted && !failed; q -= P)
                push_sum(peer(rank), jc, total, bar + 1, q);
            // (P, Q) after the round: what rank 0 found last round, or the last
            // state's, carried on to the end of the last round (as if the
            // recurrence ran on there: every chunk is a whole one to the joins)
            Sum s = empty_sum();
            if (part == P - 1) {
                if (handed) {
                    if (rank > 0) wait(2 + ((turn - 1) & 1), ((turn - 1) >> 1) & 1);
                    s = after.get(((turn - 1) & 1) * kBwdC + jc);
                } else if (jok && p.gstate_out) {
                    const Sum x = decayed(sum_of(p.gstate_out[jch], p.gstate_out[BC + jch],
                                                 -key2(p.state_out[2 * BC + jch])),
                                          decay_of(Rate{-rate.hi, -rate.lo}, rounds * round_steps - T));
                    s = scaled(x.a, x.b, x.p);
                }
            }
            if (rank < NC - 1) wait(1, parity);
            for (int q = q1 - 1; q >= max(q0, rank + 1); --q) s = join(s, peer(q).get(jc), dT);
            s = decayed(s, d_down);
#pragma unroll
            for (int h = 1; h < P; h *= 2) s = join(s, lane_sum<P>(s, part ^ h));
            if (rank == 0 && round > 0) {  // the round before goes on from this one's start
                const Sum x = join(s, total, dT), y0 = scaled(x.a, x.b, x.p);
                const int slot = (turn & 1) * kBwdC + jc;
                if (part == P - 1) after.put(slot, y0);
                for (int q = 1 + part; q < NC && !muted && !failed; q += P)
                    push_sum(after, slot, y0, bar + 2 + (turn & 1), q);
            }
            const Sum R1 = join(s, ex, d_after);
            chunk.put(i1, R1);
            chunk.put(i0, join(R1, x1, dL));
        }
        __syncthreads();

        // 5. the walk down
        Sum R[2];
        chunk.get2(warp * kBwdPitch + col, R);
        bool fastR[2];
        float p0[2], q0f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (n < L) R[j] = decayed(R[j], decay_of(rate_of(cc.w[j]), L - n));
            R[j] = scaled(R[j].a, R[j].b, R[j].p);
            const int lift = R[j].p + (int)ref.R[j];
            fastR[j] = fast[j] && lift <= kBwdLift;
            const float sc = pow2i(min(lift, 127));
            p0[j] = R[j].a * sc;
            q0f[j] = R[j].b * sc;
        }
        f2 Pw = pk(p0[0], p0[1]), Qw = pk(q0f[0], q0f[1]);
        const f2 gw = fma2(Pw, up.Ap, fma2(Qw, up.Dp, up.gw));
        IO* const gk = static_cast<IO*>(p.gk) + at + c;
        IO* const gv = static_cast<IO*>(p.gv) + at + c;
        if (plain && __all_sync(kAll, fastR[0] && fastR[1])) {
            bwd_walk_down<IO, L, true>(ch, cc, nref, Pw, Qw, gk, gv, C, true, true, true);
        } else {
            bwd_walk_down<IO, L, false>(ch, cc, nref, Pw, Qw, gk, gv, C, p.vec_store, ok0 && fastR[0],
                                     ok1 && fastR[1]);
            if (n == 1) {
                if (ok0 && fastR[0] && S[0].a == 0.f && S[0].b == 0.f) {
                    gk[0] = first_step_gk(ch.k[col], ch.v[col], ref.R[0], p0[0], q0f[0]);
                    up.gu = pk(0.f, hi(up.gu));
                }
                if (ok1 && fastR[1] && S[1].a == 0.f && S[1].b == 0.f) {
                    gk[1] = first_step_gk(ch.k[col + 1], ch.v[col + 1], ref.R[1], p0[1], q0f[1]);
                    up.gu = pk(lo(up.gu), 0.f);
                }
            }
        }
        float gwj[2] = {lo(gw), hi(gw)}, guj[2] = {lo(up.gu), hi(up.gu)};
        const float Pe[2] = {lo(Pw), hi(Pw)}, Qe[2] = {lo(Qw), hi(Qw)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool ok = n > 0 && (j ? ok1 : ok0);
            if (ok && !fastR[j]) {
                const ExactGrads x = exact_backward_down<IO>(exact_chunk(j), st_of(R[j]), gk + j, gv + j);
                R[j] = sum_of(x.R.a, x.R.b, x.R.p);
                gwj[j] = x.gw;
                guj[j] = x.gu;
            } else {
                R[j] = {Pe[j], Qe[j], -(int)ref.R[j]};
            }
            if (!ok) gwj[j] = guj[j] = 0.f;
            if (t0 == 0 && ok && p.gstate_in) {
                const int64_t sc = (int64_t)b * C + c + j;
                const double f = exp2(fmin(exponent_of(R[j].p) + key2(p.state_in[2 * BC + sc]), 1000.0));
                const float ga = (float)(f * R[j].a), gb = (float)(f * R[j].b);
                const float sa = p.state_in[sc], sb = p.state_in[BC + sc];
                p.gstate_in[sc] = ga;
                p.gstate_in[BC + sc] = gb;
                p.gstate_in[2 * BC + sc] = fmaf(sa, ga, sb * gb);
            }
        }
        gw_sum = add2(gw_sum, pk(gwj[0], gwj[1]));
        gu_sum = add2(gu_sum, pk(guj[0], guj[1]));
    }

    // the CTA's sums of gw, gu
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    float* const red = reinterpret_cast<float*>(smem);  // [2][NW][64], over the rows
    *reinterpret_cast<f2*>(red + warp * kBwdC + col) = gw_sum;
    *reinterpret_cast<f2*>(red + (NW + warp) * kBwdC + col) = gu_sum;
    const bool gave_up = __syncthreads_or(failed);
    for (int i = threadIdx.x; i < 2 * kBwdC; i += 32 * NW) {
        const int which = i / kBwdC, ci = i % kBwdC;
        if (c0 + ci < C) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < NW; ++q) s += red[(which * NW + q) * kBwdC + ci];
            (which ? p.part_u : p.part_w)[((int64_t)blockIdx.z * NC + rank) * C + c0 + ci] = s;
        }
    }
    // (the barriers above are behind every warp's last access to tensor memory)
    if (warp == 0) tmem_dealloc(*tslot, Lay::kColumns);
    // Every sum pushed to this CTA has been waited for, so it may leave -- unless
    // it gave up: then it leaves behind the others (a CTA that exits counts as
    // arrived, and each does, its waits being bounded).
    if (gave_up) {
        cluster_arrive_relaxed();
        cluster_wait_acquire();
    }
}

// Summary of every round's k, v (several rounds): CTA (tile, round), each
// warp walking its NC chunks of L steps with the next chunk's rows in flight.
template <typename IO, int L>
__global__ void __launch_bounds__(32 * kBwdWarps) wkv4_backward_summary_kernel(const BwdParams p, int NC) {
    allow_dependents();
    grid_dependency_wait();
    constexpr int NW = kBwdWarps, kTile = BwdLayout<IO, L, false>::kTile;
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = 2 * lane;
    const int round = blockIdx.y, b = blockIdx.z, c0 = (int)blockIdx.x * kBwdC, T = (int)p.T;
    const int64_t C = p.C, BC = p.B * C;
    const int t_warp = (round * NW + warp) * NC * L;
    if (!in_range(b, p.B)) return;
    BwdConsts cc;
    cc.load(p.w, p.u, c0 + col, C);
    unsigned char* const buf = smem + (size_t)warp * 4 * kTile;  // two stages of k, v
    const Sums chunk(smem + (size_t)NW * 4 * kTile, NW * kBwdC);
    auto load = [&](int q) {
        const int t = t_warp + q * L;
        const int n = q < NC ? chunk_steps(T, t, L) : 0;
        unsigned char* const d = buf + (q & 1) * 2 * kTile;
        const int64_t at = ((int64_t)b * T + t) * C;
        const IO* const kv[2] = {static_cast<const IO*>(p.k) + at, static_cast<const IO*>(p.v) + at};
        load_rows<IO, L>(d, kv, C, c0, n, lane, p.vec_load);
        cp_async_commit();
    };
    cc.derive();
    const Decay dL[2] = {decay_of(rate_of(cc.w[0]), L), decay_of(rate_of(cc.w[1]), L)};
    Sum acc[2] = {empty_sum(), empty_sum()};
    load(0);
    for (int q = 0; q < NC; ++q) {
        load(q + 1);
        cp_async_wait<1>();
        __syncwarp();
        const int n = chunk_steps(T, t_warp + q * L, L);
        const IO* const sk = reinterpret_cast<const IO*>(buf + (q & 1) * 2 * kTile);
        BwdRef ref;
        Sum sum[2];
        bwd_summary<IO>(sk, sk + kTile / sizeof(IO), col, n, cc, ref, sum);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = join(acc[j], sum[j], dL[j]);  // nothing follows a cut chunk
        __syncwarp();  // read by every lane before the stage is loaded again
    }
    chunk.put2(warp * kBwdC + col, acc[0], acc[1]);
    __syncthreads();
    const int jc = threadIdx.x;
    if (jc < kBwdC && c0 + jc < C) {
        const Decay d = decay_of(rate_of(p.w[c0 + jc]), NC * L);
        Sum s = empty_sum();
        for (int q = 0; q < NW; ++q) s = join(s, chunk.get(q * kBwdC + jc), d);
        const int64_t i = (int64_t)round * BC + (int64_t)b * C + c0 + jc;
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
    const Decay d = decay_of(rate_of(p.w[ch % p.C]), (int)round_steps);
    Sum s = empty_sum();
    if (p.state_in) s = sum_of(p.state_in[ch], p.state_in[BC + ch], key2(p.state_in[2 * BC + ch]));
    constexpr int kAhead = 8;  // rounds loaded at once: the chain waits for memory once per group
    for (int r0 = 0; r0 < p.rounds; r0 += kAhead) {
        Sum x[kAhead];
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
                s = join(s, x[j], d);
                s = scaled(s.a, s.b, s.p);
            }
        }
    }
}

// No steps: the state passes through, and its gradient with it (in the unit of
// the state given; the two maxima are the same where state_out is a copy).
__global__ void __launch_bounds__(128) wkv4_backward_no_steps_kernel(const BwdParams p, float* gw, float* gu) {
    allow_dependents();
    grid_dependency_wait();
    const int64_t BC = p.B * p.C;
    const int64_t ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (ch < p.C) gw[ch] = gu[ch] = 0.f;
    if (ch >= BC || !p.gstate_in) return;
    float ga = 0.f, gb = 0.f;
    if (p.gstate_out) {
        const float f = expf((float)((double)p.state_in[2 * BC + ch] - (double)p.state_out[2 * BC + ch]));
        ga = f * p.gstate_out[ch];
        gb = f * p.gstate_out[BC + ch];
    }
    p.gstate_in[ch] = ga;
    p.gstate_in[BC + ch] = gb;
    p.gstate_in[2 * BC + ch] = fmaf(p.state_in[ch], ga, p.state_in[BC + ch] * gb);
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
