// logit_stream.cuh -- one pass over rows of logits that are not kept: the
// statistics of their softmax, and the places where their largest entries lie.
#pragma once

#include "logit_rows.cuh"

namespace gc {

// Vectors of a thread that are read ahead, and between two looks at the maximum:
// 2 left memory idle (log probabilities of 4096 x 131072 bf16: 175 us against
// 167), 8 cost a resident CTA.
constexpr int kBatch = 4;

// A thread's vectors come in units of kBatch: within unit u the TH threads read
// kBatch consecutive stretches of TH whole vectors.  Unit `full` is the first
// that is not complete, unit `full` + 1 the ragged vectors (thread 0 has the
// row's first, thread 1 its last).
template <int TH>
struct Units {
    int full;

    template <typename T>
    __device__ __forceinline__ explicit Units(const RowPart<T>& p) : full((p.i1 - p.i0) / (kBatch * TH)) {}

    __device__ __forceinline__ int count() const { return full + 2; }

    // The k-th vector of thread t's unit u, -1 if there is none.
    template <typename T>
    __device__ __forceinline__ int vector(const RowPart<T>& p, int u, int t, int k) const {
        if (u <= full) {
            const int v = p.i0 + (u * kBatch + k) * TH + t;
            return v < p.i1 ? v : -1;
        }
        if (k > 0) return -1;
        return t == 0 && p.v0 < p.i0 ? p.v0 : t == 1 && p.i1 < p.v1 ? p.i1 : -1;
    }
};

// Most units that a part of `vectors` vectors has.
constexpr int most_units(int vectors, int threads) { return vectors / (kBatch * threads) + 2; }

// The thread's statistics over its units; note(u, m) is called with each
// unit's largest entry.  The next unit's vectors are read into registers
// before the present one's arithmetic.  KEEP: the row will be read again soon,
// so its lines are not the first to leave L2.
template <int TH, bool ENTROPY, bool KEEP, typename T, typename Note>
__device__ __forceinline__ Stat stream_stats(const RowPart<T>& p, const Units<TH>& units, float c2, Note note) {
    Sums st{neg_inf(), 0, 0};
    const uint4* src = p.vectors() + p.i0 + threadIdx.x;
    int left = p.i1 - p.i0 - static_cast<int>(threadIdx.x);             // vectors at and after src
    uint4 next[kBatch];
    auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (k * TH < left) next[k] = KEEP ? __ldcg(src + k * TH) : __ldcs(src + k * TH);
        src += kBatch * TH;
    };
    fetch();
    float vm = neg_inf();
    const int edge = units.vector(p, units.full + 1, threadIdx.x, 0);
    if (edge >= 0) {
        const uint4 w[1] = {p.load(edge)};
        vm = batch_max<T>(w);
        accumulate<T, ENTROPY>(st, w, vm, c2);
    }
    note(units.full + 1, vm);
#pragma unroll 2
    for (int u = 0; u < units.full; ++u) {
        uint4 w[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) w[k] = next[k];
        left -= kBatch * TH;
        fetch();
        vm = batch_max<T>(w);
        note(u, vm);
        accumulate<T, ENTROPY>(st, w, vm, c2);
    }
    float um = neg_inf();
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        if (k * TH < left) {
            const uint4 w[1] = {next[k]};
            vm = batch_max<T>(w);
            um = max_nan(um, vm);
            accumulate<T, ENTROPY>(st, w, vm, c2);
        }
    }
    note(units.full, um);
    return finish(st);
}

// The statistics of a whole row that is not kept, the same in every thread of a
// CTA; TH threads read, those above take part in the barriers alone.
template <int TH, typename T>
__device__ __forceinline__ Stat whole_row_stats(const RowPart<T> p, StatSmem& sm, float c2) {
    Stat mine{neg_inf(), 0.0f, 0.0f};
    if (threadIdx.x < TH) mine = stream_stats<TH, false, true>(p, Units<TH>(p), c2, [](int, float) {});
    return block_stats<TH>(sm, mine, c2);
}

// Writes f(v, vector v) to the same places of `out` for every vector of the
// part, the next unit's vectors read before the present one's arithmetic.
// `out` may be the row itself.  go() is called once the first unit's vectors are
// on their way; false ends the call with nothing written.  Threads below TH call
// it.
template <int TH, typename T, typename Go, typename F>
__device__ __forceinline__ void stream_map(const RowPart<T>& p, T* out, Go go, F f) {
    constexpr int E = RowPart<T>::E;
    const bool same = row_shift(out) == p.shift;
    uint4* dst = reinterpret_cast<uint4*>(out - p.shift);
    auto store = [&](int v, uint4 w) {
        if (same && p.whole(v)) {
            __stcs(dst + v, w);
        } else {                            // ragged, or another alignment than the input's
            float x[E];
            Elem<T>::unpack(w, x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = p.index(v, e);
                if (i >= 0 && i < p.V) out[i] = Elem<T>::round_to(x[e]);
            }
        }
    };
    int v = p.i0 + threadIdx.x;
    uint4 next[kBatch];
    auto fetch = [&](int from) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (from + k * TH < p.i1) next[k] = __ldcs(p.vectors() + from + k * TH);
    };
    fetch(v);
    if (!go()) return;
    if (threadIdx.x == 0 && p.v0 < p.i0) store(p.v0, f(p.v0, p.load(p.v0)));
    if (threadIdx.x == 1 && p.i1 < p.v1) store(p.i1, f(p.i1, p.load(p.i1)));
    if (same) {                             // complete units without a look at their ends
#pragma unroll 2
        for (int u = (p.i1 - p.i0) / (kBatch * TH); u > 0; --u, v += kBatch * TH) {
            uint4 w[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) w[k] = next[k];
            fetch(v + kBatch * TH);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) __stcs(dst + v + k * TH, f(v + k * TH, w[k]));
        }
    }
    for (; v < p.i1; v += kBatch * TH) {
        uint4 w[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) w[k] = next[k];
        fetch(v + kBatch * TH);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (v + k * TH < p.i1) store(v + k * TH, f(v + k * TH, w[k]));
    }
}

template <int TH, typename T, typename F>
__device__ __forceinline__ void stream_map(const RowPart<T>& p, T* out, F f) {
    stream_map<TH>(p, out, []() { return true; }, f);
}

// Vectors per CTA of a kernel that maps rows piece by piece, `slots` CTAs
// resident at once: 1 to 8 units, the count with the smallest
// waves * (units + half a unit to start).
inline int map_part(int64_t N, int64_t V, int elem_bytes, int threads, int64_t slots) {
    const int E = 16 / elem_bytes;
    const int64_t vectors = (V + 2 * (E - 1)) / E, unit = kBatch * threads;
    int64_t best = -1;
    int part = 0;
    for (int u = 8; u >= 1; --u) {
        const int64_t tiles = (vectors + u * unit - 1) / (u * unit);
        const int64_t cost = ((N * tiles + slots - 1) / slots) * (2 * u + 1);
        if (best < 0 || cost < best) {
            best = cost;
            part = static_cast<int>(u * unit);
        }
    }
    return part;
}

// 1024 threads of a streaming kernel are resident per SM: four CTAs of 256, or
// eight of 128.  With more rows than there are places for CTAs of 256, CTAs of
// 128 hold a row each and overlap its join with seven others' reading (20
// alternatives: 1000 rows of 200 KB 34 us against 41, 4096 rows of 64 KB 60
// against 74); very long rows then run out of even waves (2000 rows of 800 KB:
// 293 against 253), and the threshold of many alternatives, the K-th largest
// of the threads' maxima, gets poor (4096 rows of 64 KB: K = 64 86 us against
// 97, K = 100 136 against 115).  With fewer rows than two for each SM, clusters share a row while the
// parts stay long: every CTA of a cluster pays for a join (16 rows of 256 KB:
// 14.4, 12.4, 10.4, 12.3 us in clusters of 1, 2, 4, 8).
constexpr int kStreamThreads = 1024;
constexpr int64_t kLongRowBytes = 512 * 1024;
constexpr int kManyTop = 64;
constexpr int64_t kMinPartBytes = 64 * 1024;

struct StreamGeometry {
    int threads, cluster, part;             // part: vectors per CTA
};

inline StreamGeometry stream_geometry(int64_t N, int64_t V, int elem_bytes, int K, int sms) {
    const int E = 16 / elem_bytes;
    const int64_t vectors = (V + E - 1 + E - 1) / E;        // any alignment of the row
    StreamGeometry g{256, 1, 0};
    if (N > sms * (kStreamThreads / 256)) {
        if (vectors * 16 <= kLongRowBytes && K <= kManyTop) g.threads = 128;
    } else {
        while (g.cluster < kMaxCluster && N * g.cluster * 2 <= 2 * sms && vectors * 16 >= 2 * g.cluster * kMinPartBytes)
            g.cluster *= 2;
    }
    g.part = static_cast<int>((vectors + g.cluster - 1) / g.cluster);
    return g;
}

}  // namespace gc
