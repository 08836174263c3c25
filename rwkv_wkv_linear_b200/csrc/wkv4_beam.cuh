// Beam search between two decode steps (sm_100a): the n best continuations of
// a group's K beams over the vocabulary, and the move of the beams' states in
// their slot pool.
//
// Selection.  With x_kv the logits of beam k and c_k its score so far, the
// candidates of a group are
//   s_kv = c_k + (x_kv - lse_k),  lse_k = log sum_v e^{x_kv},
// and the n largest of the K V are wanted, ties to the lowest k V + v.  One
// pass over the logits, one launch, no workspace: a cluster of R CTAs a group,
// the rows cut into segments (units) dealt to its CTAs.  Within a unit a
// thread keeps a running maximum and sum of exponentials (fp32 against its
// own reference, joined over threads and units in fp64), and the unit's n
// largest logits are found on the way:
//   * each thread's maximum over its first batch gives a bound: the n-th
//     largest of the 256 maxima is at most the unit's n-th largest logit.  It is
//     found among the maxima at or above a looser one, the least of the warps'
//     (n/8)-th largest;
//   * the 16-byte pieces with an element at or above the bound are kept in
//     shared memory (about n times the unit's batches on unordered data).  After
//     the pass the threads' maxima are those of the whole unit: the looser bound
//     taken from them once more leaves some two n of the pieces' elements, which
//     are ranked by counting;
//   * where either list overflows (many equal logits, or a first batch well below
//     the rest: a script-ordered vocabulary, its first tokens ruled out) the n
//     largest are found one by one, each a pass over the unit (the batch below
//     takes 340 us then).
// Logits of one row order like their scores, so only n a unit matter; the
// first CTA of the cluster receives the units' lists and sums through cluster
// shared memory and computes the scores in fp64.  The lists being in order, a
// candidate's rank is its place in its own plus what bisection finds before it
// in each other.
//
// What bounds it.  48 requests of 8 beams over 50277 bf16 logits, n = 16: 20.9 us
// for 38.6 MB (1.8 TB/s); 2 or 3 rows an SM, whose pass ends after about 12 us,
// the rest being the latencies of ranking, cluster barrier and merge.  (With an
// eighth of the exponentials on the FMA units it takes 21.1 us, with the looser
// first bound alone 22.3.)  One request of 4 beams, fp32: 8.6 us, the chain of
// latencies alone: three batches of loads are in flight a thread.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "wkv4_chunk.cuh"  // packed f32x2, Pair

namespace wkv4 {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamMaxN = 64;       // candidates a group
constexpr int kBeamMaxK = 32;       // beams a group: a lane of the merging warp each
constexpr int kBeamPieces = 1024;   // pieces with a candidate that a unit's list holds
constexpr int kBeamList = 1024;     // candidates a unit's list holds
constexpr int kBeamBatch = 4;       // 16-byte pieces a thread loads at once
constexpr float kBeamMaxScore = 2e9f;  // |score| of a live beam; beyond, fp64 sums no longer tell logits apart

struct BeamParams {
    int64_t V, ld;
    int K, n, S;           // beams, candidates, segments a row
    int end_id;
    const void* logits;    // [G K][ld]
    const float* scores;   // [G][K]
    const uint8_t* finished;  // [G][K] or NULL
    float* out_scores;     // [G][n]
    int32_t* out_parents;
    int32_t* out_tokens;
};

// Order of candidates within a row as one integer: larger logit first, then
// the lower token.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 as +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t beam_key(float x, uint32_t token) {
    return ((uint64_t)ordered(x) << 32) | (uint32_t)~token;
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}

// A unit's result, in the first CTA's shared memory.
struct BeamUnit {
    float ref;      // the unit's largest logit
    double sum;     // sum of e^{x - ref} over the unit (NaN: a NaN or +inf among the logits)
    int count;      // keys, at most n, in order
    uint64_t keys[kBeamMaxN];
};

struct alignas(16) BeamShared {
    BeamUnit units[kBeamMaxK];
    alignas(16) uint64_t list[kBeamList + 2];
    int32_t piece_at[kBeamPieces];
    uint64_t best[kBeamMaxN];
    double lse[kBeamMaxK];   // log-sum of a live beam's row, NaN: no candidates
    float score[kBeamMaxK];
    bool ended[kBeamMaxK];   // finished beams
    alignas(16) uint32_t top[kBeamThreads];  // the threads' first maxima at or above the loose bound
    uint32_t wbound[kBeamWarps];
    float wref[kBeamWarps];
    double wsum[kBeamWarps];
    uint64_t wkey[kBeamWarps];
    uint32_t bound;
    int tops, count, npieces;
    // then [kBeamPieces] pieces, or in the merge all candidates and those ranked
    __device__ __forceinline__ uint4* pieces() { return reinterpret_cast<uint4*>(this + 1); }
};

template <typename IO>
struct BeamVec {
    static constexpr int E = 16 / (int)sizeof(IO);  // elements of a 16-byte piece
    // two elements of a piece as floats
    __device__ __forceinline__ static f2 pair(const uint4& x, int h) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if constexpr (sizeof(IO) == 4) {
            return pku(w[2 * h], w[2 * h + 1]);
        } else if constexpr (std::is_same<IO, __nv_bfloat16>::value) {
            return pku(w[h] << 16, w[h] & 0xffff0000u);
        } else {
            return Pair<__half>::cvt(*reinterpret_cast<const __half2*>(&w[h]));
        }
    }
    // the piece's largest element (NaN left out)
    __device__ __forceinline__ static float max(const uint4& x) {
        if constexpr (sizeof(IO) == 4) {
            return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)),
                         fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
        } else {
            typedef typename Pair<IO>::Raw Raw;
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            Raw r[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) r[h] = *reinterpret_cast<const Raw*>(&w[h]);
            const f2 m = Pair<IO>::cvt(__hmax2(__hmax2(r[0], r[1]), __hmax2(r[2], r[3])));
            return fmaxf(lo(m), hi(m));
        }
    }
    __device__ __forceinline__ static uint4 neg_inf() {
        const uint32_t w = sizeof(IO) == 4                             ? 0xff800000u
                           : std::is_same<IO, __nv_bfloat16>::value ? 0xff80ff80u
                                                                       : 0xfc00fc00u;
        return make_uint4(w, w, w, w);
    }
};

// A live beam's score: finite and small enough that fp64 sums keep its logits apart.
__device__ __forceinline__ bool beam_alive(float score) { return fabsf(score) <= kBeamMaxScore; }

// The logits of one unit: `len` elements at p, the first being token v0.
template <typename IO>
struct BeamRow {
    const IO* p;
    int len;
    uint32_t v0;
    int head, nvec, tail;  // elements before the first whole 16 bytes, 16-byte pieces, elements after
    __device__ __forceinline__ BeamRow(const IO* p_, int len_, uint32_t v0_) : p(p_), len(len_), v0(v0_) {
        constexpr int E = BeamVec<IO>::E;
        head = min(len, (int)((16 - (int)((uintptr_t)p & 15)) & 15) / (int)sizeof(IO));
        nvec = (len - head) / E;
        tail = len - head - nvec * E;
    }
    // element that thread tid takes from the head and tail, or -1
    __device__ __forceinline__ int loose(int tid) const {
        return tid < head ? tid : tid < head + tail ? len - tail + (tid - head) : -1;
    }
    // index of element j of piece q
    __device__ __forceinline__ int at(int q, int j) const { return head + q * BeamVec<IO>::E + j; }
};

// A thread's largest logit and its sum of e^{x - max}, as two sums of packed
// pairs of 2^{x log2e - r} with r = max log2e rounded; nat() takes the rounding
// back, to first order: below 2^11 it is at most 2^-13, so that what is left out
// is under 2^-26.  From 2^11 on (masks, mostly) the difference is taken before
// it is scaled: the rounding of r would be a factor of its own there, and past
// 2^31 no float's.
struct BeamSum {
    float max = -INFINITY;
    float r = 0.f;  // 0 before any finite logit: a NaN among those still ends up in the sum
    f2 sum = 0ull;
    bool far = false;
    // max log2e - r, the rounding of r (at most 2^-24 of it)
    __device__ __forceinline__ float rest() const {
        return far || max == -INFINITY ? 0.f : fmaf(max, kLog2e, -r);
    }
    __device__ __forceinline__ void raise(float m) {
        if (m > max) {
            const float f = ex2((max - m) * kLog2e), e = rest();  // max = -inf: 0
            max = m;
            far = !(fabsf(m) < 0x1p11f);
            r = m * kLog2e;
            const float c = f * fmaf(rest() - e, 0.6931472f, 1.f);  // from the old rounding to the new
            sum = mul2(sum, pk(c, c));
        }
    }
    template <int N>
    __device__ __forceinline__ void add(const f2 (&x)[N]) {
        if (far) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                sum = add2(sum, pk(ex2((lo(x[i]) - max) * kLog2e), ex2((hi(x[i]) - max) * kLog2e)));
        } else {
            const f2 l2e = pk(kLog2e, kLog2e), nr = pk(-r, -r);
            f2 t[N];
#pragma unroll
            for (int i = 0; i < N; ++i) t[i] = ex2_2(fma2(x[i], l2e, nr));
#pragma unroll
            for (int h = 1; h < N; h *= 2)  // a tree: no chain of additions
#pragma unroll
                for (int i = 0; i + h < N; i += 2 * h) t[i] = add2(t[i], t[i + h]);
            sum = add2(sum, t[0]);
        }
    }
    // the sum relative to e^max itself: 2^{r - max log2e} = 1 - rest ln 2
    __device__ __forceinline__ float nat() const {
        const float s = lo(sum) + hi(sum);
        return fmaf(s, rest() * -0.6931472f, s);
    }
};

// log x for x >= 1/2 to about 2^-24: the exponent in fp64, log of the mantissa in
// [0.7, 1.4] in fp32 with what its rounding left out.
__device__ __forceinline__ double beam_log(double x) {
    if (!(x >= 0.5 && x < 1e300)) return log(x);
    const long long bits = __double_as_longlong(x) - 0x3fe6a09e667f3bcdll;  // of sqrt(1/2)
    const int e = (int)(bits >> 52);
    const double m = __longlong_as_double(__double_as_longlong(x) - ((long long)e << 52));
    const float f = (float)m;
    return (double)e * kLn2D + (double)(logf(f) + (float)(m - (double)f) / f);
}

// A partial sum against the reference `to` (its own reference -inf: it saw no
// finite logit, and is 0 or NaN).
__device__ __forceinline__ double beam_term(float ref, double sum, float to) {
    return ref == -INFINITY ? sum : sum * (double)expf(ref - to);
}

template <typename IO>
__device__ __forceinline__ void beam_load(const BeamRow<IO>& r, int batch, int tid, uint4 (&x)[kBeamBatch]) {
#pragma unroll
    for (int i = 0; i < kBeamBatch; ++i) {
        const int q = (batch * kBeamBatch + i) * kBeamThreads + tid;
        x[i] = q < r.nvec ? __ldcs(reinterpret_cast<const uint4*>(r.p + r.head) + q) : BeamVec<IO>::neg_inf();
    }
}

// The q-th largest of a warp's keys.
__device__ __forceinline__ uint32_t beam_warp_top(uint32_t key, int q) {
    uint32_t top = 0;
    for (; q > 0; --q) {
        top = __reduce_max_sync(0xffffffffu, key);
        const unsigned who = __ballot_sync(0xffffffffu, key == top);
        if ((int)(threadIdx.x & 31) == __ffs(who) - 1) key = 0;
    }
    return top;
}
// The least of the warps' bounds.
__device__ __forceinline__ uint32_t beam_least(const BeamShared& s) {
    uint32_t least = s.wbound[0];
#pragma unroll
    for (int q = 1; q < kBeamWarps; ++q) least = min(least, s.wbound[q]);
    return least;
}

// The n-th largest of the threads' keys (n <= 256).
__device__ __forceinline__ uint32_t beam_bound(BeamShared& s, uint32_t key, int n) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t top = beam_warp_top(key, (n + kBeamWarps - 1) / kBeamWarps);
    if (lane == 0) s.wbound[warp] = top;
    if (tid == 0) {
        s.tops = 0;
        s.count = 0;
        s.npieces = 0;
    }
    __syncthreads();
    const uint32_t loose = beam_least(s);
    // (equal keys need no order: the n-th largest value lies where those above
    // it are fewer than n and those at or above it n or more)
    s.top[tid] = 0;
    __syncwarp();
    int at = -1;
    if (key >= loose) at = atomicAdd(&s.tops, 1);
    __syncthreads();
    if (at >= 0) s.top[at] = key;
    __syncthreads();
    if (at >= 0) {
        const int tops = s.tops;
        int above = 0, equal = 0;
        const uint4* const top4 = reinterpret_cast<const uint4*>(s.top);
#pragma unroll 4
        for (int q = 0; q < (tops + 3) / 4; ++q) {
            const uint4 o = top4[q];
            above += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
            equal += (o.x == key) + (o.y == key) + (o.z == key) + (o.w == key);
        }
        if (above < n && above + equal >= n) s.bound = key;
    }
    __syncthreads();
    return s.bound;
}

// One unit: its sum and its n largest logits into `out` (the first CTA's
// shared memory), unless its beam is dead or finished: then its logits do not
// count.  All threads of the CTA; `ready` is called before the first write to
// `out`.
template <typename IO, typename Ready>
__device__ void beam_unit(BeamShared& s, const IO* p, int len, uint32_t v0, int n, const float* score,
                          const uint8_t* finished, BeamUnit* out, Ready ready) {
    typedef BeamVec<IO> V;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (finished && *finished) return;  // before the first load: its logits are not read
    const BeamRow<IO> row(p, len, v0);
    const int batches = (row.nvec + kBeamBatch * kBeamThreads - 1) / (kBeamBatch * kBeamThreads);
    uint4 x0[kBeamBatch], x1[kBeamBatch], x2[kBeamBatch];
    beam_load(row, 0, tid, x0);
    const int li = row.loose(tid);
    const float lx = li >= 0 ? Io<IO>::to_f(p[li]) : -INFINITY;
    beam_load(row, 1, tid, x1);
    beam_load(row, 2, tid, x2);
    if (!beam_alive(*score)) return;
    BeamSum sum;
    float m = lx;
#pragma unroll
    for (int i = 0; i < kBeamBatch; ++i) m = fmaxf(m, V::max(x0[i]));
    const float bound = key_value((uint64_t)beam_bound(s, ordered(m), n) << 32);
    float most = fmaxf(bound, -3.402823466e38f);  // (-inf is no candidate)

    auto take = [&](float x, int at) {
        if (x >= most) {
            const int slot = atomicAdd(&s.count, 1);
            if (slot < kBeamList) s.list[slot] = beam_key(x, v0 + (uint32_t)at);
        }
    };
    auto pass = [&](const uint4 (&x)[kBeamBatch], int b) {
        float top[kBeamBatch], most_here = -INFINITY;
#pragma unroll
        for (int i = 0; i < kBeamBatch; ++i) {
            top[i] = V::max(x[i]);
            most_here = fmaxf(most_here, top[i]);
        }
        sum.raise(most_here);
#pragma unroll
        for (int i = 0; i < kBeamBatch; ++i) {
            f2 y[V::E / 2];
#pragma unroll
            for (int h = 0; h < V::E / 2; ++h) y[h] = V::pair(x[i], h);
            sum.add(y);
            if (top[i] >= most) {
                const int slot = atomicAdd(&s.npieces, 1);
                if (slot < kBeamPieces) {
                    s.pieces()[slot] = x[i];
                    s.piece_at[slot] = (b * kBeamBatch + i) * kBeamThreads + tid;
                }
            }
        }
    };
    sum.raise(m);
    {
        const f2 x[1] = {pk(lx, -INFINITY)};
        sum.add(x);
    }
    if (li >= 0) take(lx, li);
    for (int b = 0; b < batches; b += 3) {
        pass(x0, b);
        beam_load(row, b + 3, tid, x0);
        if (b + 1 >= batches) break;
        pass(x1, b + 1);
        beam_load(row, b + 4, tid, x1);
        if (b + 2 >= batches) break;
        pass(x2, b + 2);
        beam_load(row, b + 5, tid, x2);
    }

    // the unit's sum: brought to one reference over a warp, then over the warps
    float ref = sum.max;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    // (a thread that saw no finite logit has the sum 0 or NaN)
    double d = sum.max == -INFINITY ? sum.nat() : sum.nat() * ex2((sum.max - ref) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) {
        s.wref[warp] = ref;
        s.wsum[warp] = d;
    }
    {
        const uint32_t top = beam_warp_top(ordered(sum.max), (n + kBeamWarps - 1) / kBeamWarps);
        if (lane == 0) s.wbound[warp] = top;
    }
    __syncthreads();
    // by now the threads' largest logits are those of the whole unit
    most = fmaxf(most, key_value((uint64_t)beam_least(s) << 32));
    const int pieces = s.npieces;
    for (int i = tid; i < min(pieces, kBeamPieces) * V::E; i += kBeamThreads)
        take(Io<IO>::to_f(reinterpret_cast<const IO*>(s.pieces())[i]), row.at(s.piece_at[i / V::E], i % V::E));
    ready();
    __syncthreads();
    const int count = pieces <= kBeamPieces ? s.count : kBeamList + 1;
    if (warp == kBeamWarps - 1) {  // (the first warps rank)
        const float r0 = lane < kBeamWarps ? s.wref[lane] : -INFINITY;
        float r = r0;
#pragma unroll
        for (int o = kBeamWarps / 2; o > 0; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
        double t = lane < kBeamWarps ? beam_term(r0, s.wsum[lane], r) : 0.0;
#pragma unroll
        for (int o = kBeamWarps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) {
            out->ref = r;
            out->sum = t;
        }
    }
    if (count <= kBeamList) {
        for (int i = tid; i < count; i += kBeamThreads) {
            const uint64_t key = s.list[i];
            int rank = 0;
            const ulonglong2* const list2 = reinterpret_cast<const ulonglong2*>(s.list);
#pragma unroll 8
            for (int q = 0; q < (count + 1) / 2; ++q) {
                const ulonglong2 o = list2[q];
                rank += (o.x > key) + ((2 * q + 1 < count) & (o.y > key));
            }
            if (rank < n) out->keys[rank] = key;
        }
        if (tid == 0) out->count = min(count, n);
    } else {
        // one by one, each the largest key below the last
        uint64_t last = ~0ull;
        int have = 0;
        for (; have < n; ++have) {
            uint64_t best = 0;
            for (int i = tid; i < len; i += kBeamThreads) {
                const float x = Io<IO>::to_f(p[i]);
                const uint64_t key = beam_key(x, v0 + (uint32_t)i);
                if (x > -INFINITY && key < last && key > best) best = key;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
                best = other > best ? other : best;
            }
            if (lane == 0) s.wkey[warp] = best;
            __syncthreads();
            for (int q = 0; q < kBeamWarps; ++q) best = s.wkey[q] > best ? s.wkey[q] : best;
            __syncthreads();
            if (best == 0) break;
            if (tid == 0) out->keys[have] = best;
            last = best;
        }
        if (tid == 0) out->count = have;
    }
    __syncthreads();  // the shared list is free for the next unit
}

// Integer order of doubles (larger first).
__device__ __forceinline__ uint64_t ordered64(double x) {  // (never 0 for a number)
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// A candidate of the merge: its score's integer order, and its place k V + v.
struct alignas(16) BeamCand {
    uint64_t key;
    uint32_t flat;
    float score;
};

template <typename IO>
__global__ void __launch_bounds__(kBeamThreads, 3) wkv4_beam_select_kernel(const BeamParams p) {
    namespace cg = cooperative_groups;
    allow_dependents();
    grid_dependency_wait();
    extern __shared__ __align__(16) unsigned char smem[];
    BeamShared& s = *reinterpret_cast<BeamShared*>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int R = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t g = blockIdx.x / (unsigned)R;
    BeamShared* const first = cluster.map_shared_rank(&s, 0);
    // every CTA of the cluster has started before its shared memory is written
    cluster.barrier_arrive();
    bool waited = false;
    auto ready = [&] {
        if (!waited) cluster.barrier_wait();
        waited = true;
    };
    const int units = p.K * p.S;
    for (int q = rank; q < units; q += R) {
        const int k = q / p.S, seg = q - k * p.S;
        const int64_t row = g * p.K + k;
        const int64_t v0 = p.V * seg / p.S, v1 = p.V * (seg + 1) / p.S;
        beam_unit<IO>(s, static_cast<const IO*>(p.logits) + row * p.ld + v0, (int)(v1 - v0), (uint32_t)v0,
                      p.n, p.scores + row, p.finished ? p.finished + row : nullptr, &first->units[q], ready);
    }
    ready();
    if (rank == 0 && tid < p.K) {
        const float score = p.scores[g * p.K + tid];
        const bool ended = p.finished && p.finished[g * p.K + tid];
        s.score[tid] = score;
        s.ended[tid] = ended;
    }
    cluster.sync();
    if (rank != 0) return;

    // the rows' log-sums
    if (tid < p.K) {
        double lse = (double)NAN;
        if (beam_alive(s.score[tid]) && !s.ended[tid]) {
            const BeamUnit* u = s.units + tid * p.S;
            float ref = -INFINITY;
            for (int q = 0; q < p.S; ++q) ref = fmaxf(ref, u[q].ref);
            double sum = 0.0;
            for (int q = 0; q < p.S; ++q) sum += beam_term(u[q].ref, u[q].sum, ref);
            lse = (double)ref + beam_log(sum);
            if (!isfinite(lse)) lse = (double)NAN;
        }
        s.lse[tid] = lse;
    }
    __syncthreads();
    // candidates: every unit's list, or a finished beam's one; best first, the rest 0
    BeamCand* const all = reinterpret_cast<BeamCand*>(s.pieces());  // [units][n], free now
    const int total = units * p.n;
    int found = 0;
    for (int e = tid; e < total; e += kBeamThreads) {
        const int q = e / p.n, j = e - q * p.n, k = q / p.S;
        const float score = s.score[k];
        BeamCand c{0, 0xffffffffu, -INFINITY};
        if (s.ended[k]) {
            if (j == 0 && q == k * p.S && beam_alive(score))
                c = {ordered64((double)score), (uint32_t)(k * p.V) + (uint32_t)p.end_id, score};
        } else if (s.lse[k] == s.lse[k] && j < s.units[q].count) {
            const uint64_t key = s.units[q].keys[j];
            const double x = (double)score + ((double)key_value(key) - s.lse[k]);
            c = {ordered64(x), (uint32_t)(k * p.V) + ~(uint32_t)key, (float)x};
        }
        all[e] = c;
        found += c.key != 0;
    }
    found = __reduce_add_sync(0xffffffffu, found);
    if (lane == 0) s.wkey[tid >> 5] = (uint64_t)found;
    __syncthreads();
    found = 0;
#pragma unroll
    for (int q = 0; q < kBeamWarps; ++q) found += (int)s.wkey[q];
    // a candidate's rank: its place in its own list and, by bisection, the
    // number before it in each other (equal scores: the lower unit's first).
    // `share` threads a candidate divide the other lists.
    int share = 1, span = 1;
    while (share < 32 && share < units && 2 * share * total <= kBeamThreads) share *= 2;
    while (2 * span <= p.n) span *= 2;
    const int have = min(found, p.n);
    const int64_t out = g * p.n;
    for (int e0 = 0; e0 < total; e0 += kBeamThreads / share) {
        const int e = e0 + tid / share;
        const BeamCand c = e < total ? all[e] : BeamCand{0, 0, 0.f};
        const int q = e / p.n;
        int before = 0;
        if (c.key != 0) {
            for (int o0 = tid & (share - 1); o0 < units; o0 += 4 * share) {
                int at[4] = {};  // four lists at a time
                for (int step = span; step > 0; step >>= 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int o = o0 + i * share, next = at[i] + step;
                        // (keys of numbers are below 2^64 - 1)
                        if (o < units && next <= p.n && all[o * p.n + next - 1].key >= c.key + (o >= q))
                            at[i] = next;
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) before += o0 + i * share == q ? e - q * p.n : at[i];
            }
        }
        for (int o = share / 2; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        if (c.key != 0 && before < p.n && (tid & (share - 1)) == 0) {
            const uint32_t k = c.flat / (uint32_t)p.V;
            p.out_scores[out + before] = c.score;
            p.out_parents[out + before] = (int32_t)k;
            p.out_tokens[out + before] = (int32_t)(c.flat - k * (uint32_t)p.V);
            s.best[before] = c.flat;
        }
    }
    if (have == p.n) return;
    // fewer candidates than n: the lowest entries not taken, at -inf
    __syncthreads();
    if (tid >= 32) return;
    int filled = have;
    for (uint32_t f = 0; filled < p.n; ++f) {
        bool taken = false;
        for (int i = lane; i < have; i += 32) taken |= s.best[i] == f;
        if (__any_sync(0xffffffffu, taken)) continue;
        if (lane == 0) {
            p.out_scores[out + filled] = -INFINITY;
            p.out_parents[out + filled] = (int32_t)(f / (uint32_t)p.V);
            p.out_tokens[out + filled] = (int32_t)(f % (uint32_t)p.V);
        }
        ++filled;
    }
}

// ------------------------------------------------------- state reordering
//
// Beam j of a group goes on from the state of beam parents[j].  States are
// rows of a pool of S slots in P planes, [P][S][C], the row of beam j in slot
// ids[j].  The first beam (lowest j) that goes on from a parent keeps the
// parent's slot; a parent's further children take the slots of the beams
// nobody goes on from, in ascending order of beam, and only those rows are
// copied.  A slot that is written is never read (nobody goes on from its
// beam), so copies need no order and no staging, and a second run with the
// same ids writes the same rows again.
//
// Bound by HBM: (K - parents that go on) rows of every plane read and
// written.  Every warp works out the group's assignment by itself from its K
// ids and parents (a lane a beam), then copies its part of the rows.  8 groups
// of 8 beams of which 5 go on, 120 planes of 5120 fp32: 22.6 us for 118 MB
// (5.2 TB/s); one group of 4 beams, 36 planes of 768: 2.2 us, a launch.
struct ReorderParams {
    int64_t P, S, row;   // planes, slots, elements (of the copied type) a row
    int K;
    void* pool;
    const int32_t* ids;      // [G][K]
    const int32_t* parents;  // [G][K]
    int32_t* new_ids;        // [G][K]
};

// N: planes a thread copies.
template <typename E, int N>
__global__ void __launch_bounds__(256) wkv4_state_reorder_kernel(const ReorderParams p) {
    allow_dependents();
    grid_dependency_wait();
    const int64_t g = blockIdx.z;
    const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
    const bool beam = lane < p.K;
    const int32_t id = beam ? p.ids[g * p.K + lane] : -1 - lane;
    const int32_t par = beam ? p.parents[g * p.K + lane] : 0;
    const unsigned all = 0xffffffffu, below = (1u << lane) - 1u;
    // (the warp-wide match outside any condition: every lane takes part)
    const bool shared = (__match_any_sync(all, id) & ~(1u << lane)) != 0;  // one beam a slot
    const bool whole = __all_sync(
        all, !beam || (!shared && id >= 0 && id < p.S && par >= 0 && par < p.K));
    const unsigned same = __match_any_sync(all, beam ? par : 32 + lane);
    const bool kept = !beam || (same & below) == 0;
    const unsigned moved = __ballot_sync(all, !kept);
    const unsigned has_child = __reduce_or_sync(all, beam && whole ? 1u << par : 0u);
    unsigned free = ~has_child & (p.K == 32 ? all : (1u << p.K) - 1u);
    int32_t dst = __shfl_sync(all, id, par & 31);
    const int32_t src = dst;
    // the q-th child without a slot takes the q-th free one
    for (unsigned left = moved; left && whole; left &= left - 1) {
        const int32_t slot = __shfl_sync(all, id, __ffs(free) - 1);
        if (lane == __ffs(left) - 1) dst = slot;
        free &= free - 1;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.y * blockDim.x + threadIdx.x < 32 && beam) {
        p.new_ids[g * p.K + lane] = whole ? dst : id;
        if (!whole && lane == 0) atomicOr(&g_device_error, kErrSlot);
    }
    if (!whole) return;  // a bad id or parent: the group is left as it is
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t plane0 = (int64_t)blockIdx.y * blockDim.y * N + threadIdx.y, step = p.S * p.row;
    E* const base = static_cast<E*>(p.pool) + plane0 * step + c;
    // four rows of every plane in flight a thread
    for (unsigned left = moved; left;) {
        int32_t from[4], to[4];
        E x[N][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int who = left ? __ffs(left) - 1 : -1;
            from[i] = __shfl_sync(all, src, who & 31);
            to[i] = __shfl_sync(all, dst, who & 31);
            if (who < 0 || c >= p.row || !in_range(from[i], p.S) || !in_range(to[i], p.S)) to[i] = -1;
            left &= left - 1;
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (to[i] >= 0 && plane0 + q * blockDim.y < p.P)
                    x[q][i] = base[q * blockDim.y * step + from[i] * p.row];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (to[i] >= 0 && plane0 + q * blockDim.y < p.P)
                    base[q * blockDim.y * step + to[i] * p.row] = x[q][i];
    }
}

}  // namespace wkv4
