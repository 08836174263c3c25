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
//     largest of the 256 maxima is at most the unit's n-th largest logit;
//   * elements at or above the bound go to a list in shared memory (about
//     n times the unit's batches on unordered data), whose n largest are
//     ranked by counting;
//   * a list that overflows (many equal logits) is dropped and the n largest
//     are found one by one, each a pass over the unit.
// Logits of one row order like their scores, so only n a unit matter; the
// first CTA of the cluster receives the units' lists and sums through cluster
// shared memory, computes the scores in fp64 and merges the lists' heads, one
// warp, a lane a unit.
//
// What bounds it: HBM reads of the logits, with one ex2 an element close
// behind (16 a clock and SM).
#pragma once

#include <cooperative_groups.h>

#include "wkv4_device.cuh"

namespace wkv4 {

constexpr int kBeamThreads = 256;
constexpr int kBeamMaxN = 64;       // candidates a group
constexpr int kBeamMaxK = 32;       // beams a group: a lane of the merging warp each
constexpr int kBeamList = 1024;     // elements a unit's list holds
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

struct BeamShared {
    BeamUnit units[kBeamMaxK];
    uint64_t list[kBeamList];
    uint64_t best[kBeamMaxN];
    float tmax[kBeamThreads];
    float wref[kBeamThreads / 32];
    double wsum[kBeamThreads / 32];
    uint64_t wkey[kBeamThreads / 32];
    float bound;
    int count;
};

template <typename IO>
struct BeamVec {
    static constexpr int E = 16 / (int)sizeof(IO);
    static constexpr int N = kBeamBatch * E;
};

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

// A thread's largest logit and its sum of e^{x - max}.  The difference is taken
// before it is scaled: it cannot overflow at the type's largest values, and
// near the maximum, where the terms that count are, it is exact.
struct BeamSum {
    float max = -INFINITY;
    float base = 0.f;  // max, or 0 before any finite logit (a NaN among those still ends up in the sum)
    float sum = 0.f;
    __device__ __forceinline__ void raise(float m) {
        if (m > max) {
            sum *= ex2((max - m) * kLog2e);  // max = -inf: 0 * 0
            max = base = m;
        }
    }
    __device__ __forceinline__ void add(float x) { sum += ex2((x - base) * kLog2e); }
};

template <typename IO>
__device__ __forceinline__ void beam_load(const BeamRow<IO>& r, int batch, int tid, uint4 (&x)[kBeamBatch]) {
#pragma unroll
    for (int i = 0; i < kBeamBatch; ++i) {
        const int q = (batch * kBeamBatch + i) * kBeamThreads + tid;
        if (q < r.nvec) x[i] = __ldcs(reinterpret_cast<const uint4*>(r.p + r.head) + q);
    }
}

// The pieces of one batch as floats (-inf past the end).
template <typename IO>
__device__ __forceinline__ void beam_unpack(const BeamRow<IO>& r, int batch, int tid,
                                            const uint4 (&x)[kBeamBatch], float (&f)[BeamVec<IO>::N]) {
    constexpr int E = BeamVec<IO>::E;
#pragma unroll
    for (int i = 0; i < kBeamBatch; ++i) {
        const bool in = (batch * kBeamBatch + i) * kBeamThreads + tid < r.nvec;
        IO t[E];
        *reinterpret_cast<uint4*>(t) = x[i];
#pragma unroll
        for (int j = 0; j < E; ++j) f[i * E + j] = in ? Io<IO>::to_f(t[j]) : -INFINITY;
    }
}

// A partial sum against the reference `to` (its own reference -inf: it saw no
// finite logit, and is 0 or NaN).
__device__ __forceinline__ double beam_term(float ref, double sum, float to) {
    return ref == -INFINITY ? sum : sum * exp((double)ref - (double)to);
}

__device__ __forceinline__ void beam_push(BeamShared& s, float x, uint32_t token) {
    const int at = atomicAdd(&s.count, 1);
    if (at < kBeamList) s.list[at] = beam_key(x, token);
}

// One unit: its sum and its n largest logits into `out` (the first CTA's
// shared memory).  All threads of the CTA.
template <typename IO>
__device__ void beam_unit(BeamShared& s, const IO* p, int len, uint32_t v0, int n, BeamUnit* out) {
    constexpr int E = BeamVec<IO>::E, N = BeamVec<IO>::N;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const BeamRow<IO> row(p, len, v0);
    const int batches = (row.nvec + kBeamBatch * kBeamThreads - 1) / (kBeamBatch * kBeamThreads);
    uint4 cur[kBeamBatch] = {}, nxt[kBeamBatch] = {};
    beam_load(row, 0, tid, cur);
    const int li = row.loose(tid);
    const float lx = li >= 0 ? Io<IO>::to_f(p[li]) : -INFINITY;
    beam_load(row, 1, tid, nxt);
    BeamSum sum;
    float f[N];
    beam_unpack(row, 0, tid, cur, f);
    float m = lx;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, f[j]);
    // the bound: the n-th largest of the threads' first maxima
    s.tmax[tid] = m;
    if (tid == 0) {
        s.count = 0;
        s.bound = -INFINITY;
    }
    __syncthreads();
    int above = 0;
#pragma unroll 8
    for (int q = 0; q < kBeamThreads; ++q) {
        const float o = s.tmax[q];
        above += o > m || (o == m && q < tid);
    }
    if (above == n - 1) s.bound = m;
    __syncthreads();
    const float bound = s.bound;

    auto take = [&](float x, int at) {
        if (x >= bound && x > -INFINITY) beam_push(s, x, v0 + (uint32_t)at);
    };
    sum.raise(m);
    sum.add(lx);
    if (li >= 0) take(lx, li);
    for (int b = 0;; ++b) {
#pragma unroll
        for (int j = 0; j < N; ++j) sum.add(f[j]);
        if (m >= bound && m > -INFINITY) {
#pragma unroll
            for (int j = 0; j < N; ++j) take(f[j], row.at((b * kBeamBatch + j / E) * kBeamThreads + tid, j % E));
        }
        if (b + 1 >= batches) break;
#pragma unroll
        for (int i = 0; i < kBeamBatch; ++i) cur[i] = nxt[i];
        beam_load(row, b + 2, tid, nxt);
        beam_unpack(row, b + 1, tid, cur, f);
        m = f[0];
#pragma unroll
        for (int j = 1; j < N; ++j) m = fmaxf(m, f[j]);
        sum.raise(m);
    }

    // the unit's sum: references joined over a warp, then over the warps
    float ref = sum.max;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    double d = beam_term(sum.max, (double)sum.sum, ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) {
        s.wref[warp] = ref;
        s.wsum[warp] = d;
    }
    __syncthreads();
    const int count = s.count;
    if (tid == 0) {
        float r = s.wref[0];
        for (int q = 1; q < kBeamThreads / 32; ++q) r = fmaxf(r, s.wref[q]);
        double t = 0.0;
        for (int q = 0; q < kBeamThreads / 32; ++q) t += beam_term(s.wref[q], s.wsum[q], r);
        out->ref = r;
        out->sum = t;
    }
    if (count <= kBeamList) {
        const int have = min(count, n);
        for (int i = tid; i < count; i += kBeamThreads) {
            const uint64_t key = s.list[i];
            int rank = 0;
            for (int q = 0; q < count; ++q) rank += s.list[q] > key;
            if (rank < n) out->keys[rank] = key;
        }
        if (tid == 0) out->count = have;
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
            for (int q = 0; q < kBeamThreads / 32; ++q) best = s.wkey[q] > best ? s.wkey[q] : best;
            __syncthreads();
            if (best == 0) break;
            if (tid == 0) out->keys[have] = best;
            last = best;
        }
        if (tid == 0) out->count = have;
    }
    __syncthreads();  // the shared list is free for the next unit
}

// A live beam's score: finite and small enough that fp64 sums keep its logits apart.
__device__ __forceinline__ bool beam_alive(float score) { return fabsf(score) <= kBeamMaxScore; }

// Integer order of doubles (larger first).
__device__ __forceinline__ uint64_t ordered64(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// Warp-wide largest of 64-bit values.
__device__ __forceinline__ uint64_t warp_max64(uint64_t x) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
    return ((uint64_t)hi << 32) | lo;
}

template <typename IO>
__global__ void __launch_bounds__(kBeamThreads) wkv4_beam_select_kernel(const BeamParams p) {
    namespace cg = cooperative_groups;
    allow_dependents();
    grid_dependency_wait();
    __shared__ BeamShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int R = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t g = blockIdx.x / R;
    BeamShared* const first = cluster.map_shared_rank(&s, 0);
    cluster.sync();  // every CTA of the cluster has started: its shared memory may be written
    const int units = p.K * p.S;
    for (int q = rank; q < units; q += R) {
        const int k = q / p.S, seg = q % p.S;
        const int64_t row = g * p.K + k;
        const float score = p.scores[row];
        if (!beam_alive(score) || (p.finished && p.finished[row])) continue;  // no logits of this beam count
        const int64_t v0 = p.V * seg / p.S, v1 = p.V * (seg + 1) / p.S;
        beam_unit<IO>(s, static_cast<const IO*>(p.logits) + row * p.ld + v0, (int)(v1 - v0), (uint32_t)v0,
                      p.n, &first->units[q]);
    }
    cluster.sync();
    if (rank != 0 || threadIdx.x >= 32) return;

    // the merge: lane q holds unit q of row k
    const int lane = threadIdx.x, k = lane / p.S;
    const bool mine = lane < units;
    const float score = mine ? p.scores[g * p.K + k] : -INFINITY;
    const bool alive = beam_alive(score);
    const bool done = alive && p.finished && p.finished[g * p.K + k];
    double lse = 0.0;
    int left = 0, at = 0;  // candidates left in the unit, the next one
    if (alive && !done) {
        // log-sum of the row over its units
        float ref = -INFINITY;
        for (int q = k * p.S; q < (k + 1) * p.S; ++q) ref = fmaxf(ref, s.units[q].ref);
        double sum = 0.0;
        for (int q = k * p.S; q < (k + 1) * p.S; ++q)
            sum += beam_term(s.units[q].ref, s.units[q].sum, ref);
        lse = (double)ref + log(sum);
        if (isfinite(lse)) left = s.units[lane].count;
    } else if (done && lane % p.S == 0) {
        left = 1;
    }
    const int64_t out = g * p.n;
    int have = 0;
    uint64_t next = 0;      // order of this unit's next candidate, 0: none
    uint32_t flat = 0;
    double val = 0.0;
    auto fetch = [&] {
        next = 0;
        if (left > 0) {
            uint32_t token = (uint32_t)p.end_id;
            val = (double)score;
            if (!done) {
                const uint64_t key = s.units[lane].keys[at];
                token = ~(uint32_t)key;
                val = (double)score + ((double)key_value(key) - lse);
            }
            flat = (uint32_t)(k * p.V) + token;
            next = ordered64(val);
            ++at;
            --left;
        }
    };
    fetch();
    for (; have < p.n; ++have) {
        const uint64_t top = warp_max64(next);
        if (top == 0) break;
        const uint32_t lowest = __reduce_min_sync(0xffffffffu, next == top ? flat : 0xffffffffu);
        if (next == top && flat == lowest) {
            p.out_scores[out + have] = (float)val;
            p.out_parents[out + have] = k;
            p.out_tokens[out + have] = (int32_t)(flat - (uint32_t)(k * p.V));
            s.best[have] = flat;
            fetch();
        }
        __syncwarp();
    }
    // fewer candidates than n: the lowest entries not taken, at -inf
    for (uint32_t f = 0; have < p.n; ++f) {
        bool taken = false;
        for (int i = lane; i < have; i += 32) taken |= s.best[i] == f;
        if (__any_sync(0xffffffffu, taken)) continue;
        if (lane == 0) {
            p.out_scores[out + have] = -INFINITY;
            p.out_parents[out + have] = (int32_t)(f / (uint32_t)p.V);
            p.out_tokens[out + have] = (int32_t)(f % (uint32_t)p.V);
            s.best[have] = f;
        }
        __syncwarp();
        ++have;
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
// ids and parents (a lane a beam), then copies its part of the rows.
struct ReorderParams {
    int64_t P, S, row;   // planes, slots, elements (of the copied type) a row
    int K;
    void* pool;
    const int32_t* ids;      // [G][K]
    const int32_t* parents;  // [G][K]
    int32_t* new_ids;        // [G][K]
};

template <typename E>
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
    const int64_t plane = (int64_t)blockIdx.y * blockDim.y + threadIdx.y;
    const bool in = c < p.row && plane < p.P;
    E* const base = static_cast<E*>(p.pool) + plane * p.S * p.row + c;
    // four rows in flight a thread
    for (unsigned left = moved; left;) {
        int32_t from[4], to[4];
        E x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int who = left ? __ffs(left) - 1 : -1;
            from[i] = __shfl_sync(all, src, who & 31);
            to[i] = __shfl_sync(all, dst, who & 31);
            if (who < 0) to[i] = -1;
            left &= left - 1;
            if (in && to[i] >= 0 && in_range(from[i], p.S)) x[i] = base[from[i] * p.row];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (in && to[i] >= 0 && in_range(to[i], p.S)) base[to[i] * p.row] = x[i];
    }
}

}  // namespace wkv4
