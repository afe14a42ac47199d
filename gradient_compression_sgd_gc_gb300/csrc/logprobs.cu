// logprobs.cu -- log probabilities of given tokens with entropy and top
// alternatives, and their gradient.
//
//   y = x / tau;  lse = log sum exp(y);  logp = y[id] - lse
//   H = log s - u / s          (Stat's s and u, in base 2)
//   d = (g (onehot - p) - h p (log p + H)) / tau
//
// The forward pass reads each logit once from memory, the gradient reads and
// writes each once (rows with |lse| >= 1024 are read twice).
#include "logit_stream.cuh"

namespace gc {
namespace {

// ---------------------------------------------------------------- top alternatives

// Order of the alternatives: by value (NaN first, a zero of either sign the
// same), then by lowest index.  A 64-bit key holds both, larger is better.
__device__ __forceinline__ uint32_t value_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint64_t entry_of(uint32_t key, int index) {
    return (static_cast<uint64_t>(key) << 32) | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ int entry_index(uint64_t e) { return static_cast<int>(~static_cast<uint32_t>(e)); }

// The upper half of the keys of masked entries: -inf and the lowest values of
// both types.
constexpr uint32_t kMaskedTop = 0x0080u;
constexpr uint32_t kInfTop = 0xff80u;

// Entries that a CTA can collect (a run of rising logits puts all 8 elements of
// K vectors above the threshold), and units that it can look at again.
__host__ __device__ constexpr int candidate_cap(int K) { return 8 * K + 128; }
__host__ __device__ constexpr int hit_cap(int K) { return 2 * K + 128; }
constexpr int kPad = 4 * 32;                // after the entries, to fill their list up

struct TopSmem {
    int count, hits;                        // candidates, units collected
    uint32_t best;                          // largest key of a round (descend)
    int warp_count[kMaxRowWarps];
    int listed[kMaxCluster];                // entries in each CTA's list
};

// Dynamic shared memory of a CTA: the candidates, the cluster's sorted lists,
// the units to look at again, and the upper half of each unit's largest key.
struct TopBuffers {
    uint64_t* cand;
    uint64_t* list;
    uint32_t* hit;
    uint16_t* unit_key;

    __device__ __forceinline__ TopBuffers(unsigned char* smem, int K, int parts) {
        cand = reinterpret_cast<uint64_t*>(smem);
        list = cand + candidate_cap(K) + kPad;
        hit = reinterpret_cast<uint32_t*>(list + parts * K);
        unit_key = reinterpret_cast<uint16_t*>(hit + hit_cap(K));
    }
};

constexpr size_t top_bytes(int K, int parts, int threads, int units) {
    return sizeof(uint64_t) * (candidate_cap(K) + kPad + static_cast<size_t>(parts) * K) + sizeof(uint32_t) * hit_cap(K) +
           sizeof(uint16_t) * threads * units;
}

// More than any call takes: the most alternatives in the largest cluster, with
// the units of a whole fp32 row of the longest (whose CTAs have 256 threads).
constexpr size_t kMostTopBytes = top_bytes(GC_MAX_TOP, kMaxCluster, 256, most_units(GC_MAX_VOCAB / 4 + 2, 256));

// Calls f(key, index) for every entry of the part, by the thread that has it.
template <int TH, typename T, typename F>
__device__ __forceinline__ void for_entries(const RowPart<T>& p, F f) {
    constexpr int E = RowPart<T>::E;
    for (int v = p.v0 + threadIdx.x; v < p.v1; v += TH) {
        float x[E];
        Elem<T>::unpack(p.load(v), x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = p.index(v, e);
            if (i >= 0 && i < p.V) f(value_key(x[e]), i);
        }
    }
}

// Adds the entries of this CTA's part with keys up to `from`, best first, until
// `need` are found or none is left; equal keys in order of their index.  One
// distinct value a round, each of which reads the part again: for the masked
// entries and for ties at a known key.
template <int TH, typename T>
__device__ __noinline__ void descend(const RowPart<T> p, TopSmem& sm, uint64_t* cand, uint32_t from, int need) {
    constexpr int E = RowPart<T>::E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    while (need > 0) {
        if (threadIdx.x == 0) sm.best = 0;
        __syncthreads();
        uint32_t best = 0;                  // no key is 0
        for_entries<TH>(p, [&](uint32_t k, int) {
            if (k <= from && k > best) best = k;
        });
        best = __reduce_max_sync(0xffffffffu, best);
        if (lane == 0 && best) atomicMax(&sm.best, best);
        __syncthreads();
        best = sm.best;
        if (best == 0) return;              // the part has no more entries
        for (int base = p.v0; base < p.v1 && need > 0; base += TH) {
            const int v = base + threadIdx.x;
            unsigned hit = 0;
            if (v < p.v1) {
                float f[E];
                Elem<T>::unpack(p.load(v), f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = p.index(v, e);
                    if (value_key(f[e]) == best && i >= 0 && i < p.V) hit |= 1u << e;
                }
            }
            int incl = __popc(hit);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane == 31) sm.warp_count[warp] = incl;
            __syncthreads();
            int at = incl - __popc(hit), all = 0;
#pragma unroll
            for (int w = 0; w < TH / 32; ++w) {
                if (w < warp) at += sm.warp_count[w];
                all += sm.warp_count[w];
            }
            const int have = sm.count;
            for (; hit; hit &= hit - 1, ++at)
                if (at < need) cand[have + at] = entry_of(best, p.index(v, __ffs(hit) - 1));
            __syncthreads();
            if (threadIdx.x == 0) sm.count = have + min(all, need);
            need -= min(all, need);
            __syncthreads();
        }
        from = best - 1;
    }
}

// The K best entries of this CTA's part where too many are not below `low` to
// be collected: the K-th key by bisection between `low`, which K entries reach,
// and the largest key, a reading for each bit of their distance, then the
// entries above it and its first ties: some 20 readings of the part where the
// values lie close together, 35 at most (one key far above a plateau of ties).
template <int TH, typename T>
__device__ __noinline__ void exact_top(const RowPart<T> p, TopSmem& sm, uint64_t* cand, uint32_t low, uint32_t high, int K) {
    const int lane = threadIdx.x & 31;
    while (low < high) {
        const uint32_t mid = low + (high - low + 1) / 2;
        if (threadIdx.x == 0) sm.count = 0;
        __syncthreads();
        int n = 0;
        for_entries<TH>(p, [&](uint32_t k, int) { n += k >= mid; });
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0 && n) atomicAdd(&sm.count, n);
        __syncthreads();
        if (sm.count >= K) low = mid;
        else high = mid - 1;
        __syncthreads();
    }
    if (threadIdx.x == 0) sm.count = 0;
    __syncthreads();
    for_entries<TH>(p, [&](uint32_t k, int i) {
        if (k > low) cand[atomicAdd(&sm.count, 1)] = entry_of(k, i);     // fewer than K
    });
    __syncthreads();
    const int need = K - sm.count;
    __syncthreads();
    descend<TH>(p, sm, cand, low, need);
}

// The K best entries of this CTA's part, sorted, to list[rank][..] of the
// cluster's first CTA.  The K-th largest of the threads' maxima is no
// larger than the K-th largest entry, so what is not below it (in its upper 16
// bits) contains the K best: a few more than K entries, in the units whose
// maximum reaches it, which are read again.  Masked entries are left to
// descend(), which takes them in order of their index.
template <int TH, typename T>
__device__ void part_top(const RowPart<T>& p, const Units<TH>& units, TopSmem& sm, const TopBuffers& b, int K, float thread_max,
                         float part_max, unsigned rank) {
    constexpr int E = RowPart<T>::E;
    const int cap = candidate_cap(K), hits_cap = hit_cap(K);
    const uint32_t mine = value_key(thread_max) >> 16;
    if (threadIdx.x == 0) sm.count = sm.hits = 0;
    // the largest `top` that K threads reach: below the maximum, where it mostly
    // is, in steps growing by 8, then by bisection
    uint32_t high = value_key(part_max) >> 16, width = 64, top = 0;
    while (width < 65536) {
        top = high > width ? high - width : 0;
        if (__syncthreads_count(mine >= top) >= K) break;
        if (top == 0) break;
        high = top;
        width *= 8;
    }
    if (width >= 65536) top = 0;
    while (high - top > 0) {                // K threads reach top; high + 1 is untested or not reached
        const uint32_t t = top + (high - top + 1) / 2;
        if (__syncthreads_count(mine >= t) >= K) top = t;
        else high = t - 1;
    }
    const bool masked = top <= kMaskedTop;
    const uint32_t least = masked ? kMaskedTop + 1 : top;
    // as a value, which NaN is not below: the keys above that of +inf are NaN's
    const float least_value = key_value(min(least, kInfTop) << 16);
    if (mine >= least) {
        for (int u = 0; u < units.count(); ++u) {
            if (b.unit_key[u * TH + threadIdx.x] >= least) {
                const int at = atomicAdd(&sm.hits, 1);
                if (at < hits_cap) b.hit[at] = static_cast<uint32_t>(u) * TH + threadIdx.x;
            }
        }
    }
    __syncthreads();
    const int hits = sm.hits;
    if (hits <= hits_cap) {
        for (int i = threadIdx.x; i < hits * kBatch; i += TH) {
            const uint32_t h = b.hit[i / kBatch];
            const int v = units.vector(p, h / TH, h % TH, i % kBatch);
            if (v < 0) continue;
            float f[E];
            Elem<T>::unpack(p.load(v), f);
            unsigned found = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) found |= static_cast<unsigned>(!(f[e] < least_value)) << e;
            // as many rounds as the vector with the most has, mostly one
            for (; found; found &= found - 1) {
                const int which = __ffs(found) - 1;
                float x = f[0];
#pragma unroll
                for (int e = 1; e < E; ++e)
                    if (e == which) x = f[e];
                const int at = atomicAdd(&sm.count, 1);
                if (at < cap) b.cand[at] = entry_of(value_key(x), p.index(v, which));
            }
        }
    }
    __syncthreads();
    int n = sm.count;
    __syncthreads();
    if (hits > hits_cap || n > cap)         // many equal values, or large ones close together
        exact_top<TH>(p, sm, b.cand, least << 16, value_key(part_max), K);
    else if (n < K && masked)
        descend<TH>(p, sm, b.cand, ((kMaskedTop + 1) << 16) - 1, K - n);
    __syncthreads();
    n = sm.count;
    if (threadIdx.x == 0) st_remote(remote_smem(&sm.listed[rank], 0), static_cast<uint32_t>(min(n, K)));
    // ranks by counting, 2^share neighbouring threads to an entry, four entries
    // a step (the list is filled up with zeros, which are below every entry)
    int share = 0;
    while (share < 5 && (n << (share + 1)) <= TH) ++share;
    const int lanes = 1 << share, sub = threadIdx.x & (lanes - 1), padded = (n + 4 * lanes - 1) & ~(4 * lanes - 1);
    for (int i = n + threadIdx.x; i < padded; i += TH) b.cand[i] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += TH >> share) {
        const int i = i0 + (threadIdx.x >> share);
        if (__all_sync(0xffffffffu, i >= n)) continue;
        const uint64_t e = i < n ? b.cand[i] : 0;
        int r = 0;
        for (int j = sub; j < padded; j += 4 * lanes) {
#pragma unroll
            for (int k = 0; k < 4; ++k) r += b.cand[j + k * lanes] > e;
        }
        for (int o = 1; o < lanes; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        if (i < n && sub == 0 && r < K) st_remote(remote_smem(b.list + rank * K + r, 0), e);
    }
}

// ---------------------------------------------------------------- forward

struct LogprobArgs {
    RowArgs row;
    const void* ids;
    int id64, K;
    float* logprobs;
    float* entropy;
    float* lse;
    int32_t* top_ids;
    float* top_logprobs;
    int* status;
};

template <typename T, int TH, bool TOP>
__global__ void __launch_bounds__(TH, kStreamThreads / TH) k_token_logprobs(LogprobArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ StatSmem stat_smem;
    __shared__ TopSmem top_smem;
    const unsigned rank = cluster_rank(), parts = cluster_size();
    const int64_t n = blockIdx.x / parts;
    cluster_announce(parts);
    const RowPart<T> p(a.row, n, rank);
    const Units<TH> units(p);
    const TopBuffers top(smem_raw, a.K, parts);
    const float c2 = a.row.c2;
    const Stat mine = stream_stats<TH, true, false>(p, units, c2, [&](int u, float m) {
        if (TOP) top.unit_key[u * TH + threadIdx.x] = static_cast<uint16_t>(value_key(m) >> 16);
    });
    float x_id = 0.0f;
    bool have = false;
    if (rank == 0 && threadIdx.x == 0) {
        const int64_t id = load_id(a.ids, a.id64, n, a.row.V, a.status);
        have = id >= 0;
        if (have) x_id = Elem<T>::load_plain(p.row + id);
    }
    const Stat cta = block_stats<TH>(stat_smem, mine, c2);
    cluster_started(parts);
    if (threadIdx.x < 3) {
        const float v = threadIdx.x == 0 ? cta.m : threadIdx.x == 1 ? cta.s : cta.u;
        st_remote(remote_smem(&stat_smem.part[rank][threadIdx.x], 0), v);
    }
    if (TOP) part_top(p, units, top_smem, top, a.K, mine.m, cta.m, rank);
    cluster_join(parts);
    if (rank != 0) return;

    const Stat st = join_parts(stat_smem.part, parts, c2);
    const float ln_s = logf(st.s);
    if (threadIdx.x == 0) {
        a.logprobs[n] = have ? log_prob(st, ln_s, x_id, a.row) : 0.0f;
        if (a.entropy)
            a.entropy[n] = st.m == neg_inf() ? 0.0f : max_nan(0.0f, fmaf(-kLn2, st.u / st.s, ln_s));
        if (a.lse) a.lse[n] = row_lse(st, ln_s, a.row);
    }
    if (TOP) {
        // an entry's rank over the row: its rank in its own list and, by
        // bisection, the better entries of the other lists
        for (int i = threadIdx.x; i < static_cast<int>(parts) * a.K; i += TH) {
            const int c = i / a.K, r = i - c * a.K;
            if (r >= top_smem.listed[c]) continue;
            const uint64_t e = top.list[i];
            int g = r;
            for (int d = 0; d < static_cast<int>(parts); ++d) {
                if (d == c) continue;
                int lo = 0, hi = top_smem.listed[d];
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (top.list[d * a.K + mid] > e) lo = mid + 1;
                    else hi = mid;
                }
                g += lo;
            }
            if (g < a.K) {
                a.top_ids[n * a.K + g] = entry_index(e);
                a.top_logprobs[n * a.K + g] = log_prob(st, ln_s, key_value(static_cast<uint32_t>(e >> 32)), a.row);
            }
        }
    }
}

// ---------------------------------------------------------------- gradient

constexpr int kGradThreads = 256;
constexpr int kGradCtas = 4;                // resident per SM

struct LogprobGradArgs {
    RowArgs row;
    const void* ids;
    unsigned tiles;                         // CTAs per row
    int id64;
    const float* lse;
    const float* entropy;
    const float* g_logprobs;
    const float* g_entropy;
    void* out;
    int64_t ld_out;
    int* status;
};

// What a row's gradient is made of: d = p (k0 + k1 log p), and `token` more for
// the token.
template <typename T>
struct Slope {
    int64_t id;
    float token, k0, k1;

    __device__ __forceinline__ Slope(const LogprobGradArgs& a, int64_t n, bool entropy, int* status) {
        id = load_id(a.ids, a.id64, n, a.row.V, status);
        const float g = a.g_logprobs ? __ldg(a.g_logprobs + n) : 0.0f;
        const float h = entropy ? __ldg(a.g_entropy + n) : 0.0f;
        const float H = entropy ? __ldg(a.entropy + n) : 0.0f;
        token = g * a.row.inv_tau;
        k1 = -h * a.row.inv_tau;
        k0 = fmaf(k1, H, id >= 0 ? -token : 0.0f);
    }

    // The vector that holds the token, -1 without one.
    __device__ __forceinline__ int vector(const RowPart<T>& p) const {
        return id >= 0 ? static_cast<int>((id + p.shift) / Elem<T>::E) : -1;
    }

    __device__ __forceinline__ void add_token(const RowPart<T>& p, int v, float (&f)[Elem<T>::E]) const {
#pragma unroll
        for (int e = 0; e < Elem<T>::E; ++e)
            if (p.index(v, e) == id) f[e] += token;
    }
};

// The gradient of a row whose lse does not hold its sum, by one CTA: the row is
// read once more before, and nothing is written until then, so it may be in
// place.  2048 x 131072 bf16 of -1e9 take 280 us, where usual rows take 162; 300
// x 50001 fp32 34 and 19; one row of 131072 bf16 25 and 9.
template <typename T, bool ENTROPY>
__device__ __noinline__ void whole_row_grad(const LogprobGradArgs& a, int64_t n) {
    __shared__ StatSmem stat_smem;
    const RowPart<T> p(a.row, n, 0, kWholeRow);
    const float c2 = a.row.c2, inv_tau = a.row.inv_tau;
    const Stat st = whole_row_stats<kGradThreads>(p, stat_smem, c2);
    const Slope<T> slope(a, n, ENTROPY, a.status);
    const int v_id = slope.vector(p);
    const bool empty = st.m == neg_inf();
    const float ln_s = logf(st.s), inv_s = 1.0f / st.s;
    stream_map<kGradThreads>(p, static_cast<T*>(a.out) + n * a.ld_out, [&](int v, uint4 w) {
        float f[Elem<T>::E];
        Elem<T>::unpack(w, f);
#pragma unroll
        for (int e = 0; e < Elem<T>::E; ++e) {
            const float q = empty ? 0.0f : inv_s * exp2_fast(max_nan(exponent(f[e], st.m, c2), -150.0f));
            f[e] = q == 0.0f ? 0.0f : q * fmaf(slope.k1, fmaf(f[e] - st.m, inv_tau, -ln_s), slope.k0);
        }
        if (v == v_id) slope.add_token(p, v, f);
        return Elem<T>::pack(f);
    });
}

// One CTA per piece of a row, or one for a row whose lse does not hold its sum.
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kGradThreads, kGradCtas) k_token_logprobs_grad(const __grid_constant__ LogprobGradArgs a) {
    constexpr int E = Elem<T>::E;
    const int64_t n = blockIdx.x / a.tiles;
    const unsigned tile = blockIdx.x % a.tiles;
    const float lse = __ldg(a.lse + n), inv_tau = a.row.inv_tau;
    if (!lse_holds(lse)) {
        if (tile == 0) whole_row_grad<T, ENTROPY>(a, n);
        return;
    }
    const RowPart<T> p(a.row, n, tile);
    const Slope<T> slope(a, n, ENTROPY, tile == 0 ? a.status : nullptr);
    const int v_id = slope.vector(p);
    const float k0 = slope.k0, k1 = slope.k1;
    stream_map<kGradThreads>(p, static_cast<T*>(a.out) + n * a.ld_out, [&](int v, uint4 w) {
        float f[E];                         // masked entries at -2^60: p is 0 and log p finite
        Elem<T>::unpack(floored<T>(w), f);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            // log p = y - lse in natural units, so that neither the rounding of
            // lse * log2(e) nor that of 1 / temperature scales the row
            const uint64_t lp = log_prob_pair(pair(f[e], f[e + 1]), lse, inv_tau, a.row.inv_tau_low);
            float y0, y1;
            unpair(pair_mul(lp, pair(kLog2e, kLog2e)), y0, y1);
            const uint64_t d = ENTROPY ? pair_fma(lp, pair(k1, k1), pair(k0, k0)) : pair(k0, k0);
            unpair(pair_mul(pair(exp2_fast(y0), exp2_fast(y1)), d), f[e], f[e + 1]);
        }
        if (v == v_id) slope.add_token(p, v, f);
        return Elem<T>::pack(f);
    });
}

template <typename T, int TH>
int launch_logprobs(LogprobArgs a, int cluster, cudaStream_t s) {
    static_assert(kUnaskedSmem + sizeof(StatSmem) + sizeof(TopSmem) <= 48 * 1024, "static shared memory");
    if (a.K == 0) return launch_rows(k_token_logprobs<T, TH, false>, cluster, a.row.N, TH, 0, 0, a, s);
    return launch_rows(k_token_logprobs<T, TH, true>, cluster, a.row.N, TH,
                       top_bytes(a.K, cluster, TH, most_units(a.row.part, TH)), kMostTopBytes, a, s);
}

template <typename T>
int launch_logprobs(LogprobArgs a, int sms, cudaStream_t s) {
    const StreamGeometry g = stream_geometry(a.row.N, a.row.V, sizeof(T), a.K, sms);
    a.row.part = g.part;
    return g.threads == 128 ? launch_logprobs<T, 128>(a, g.cluster, s) : launch_logprobs<T, 256>(a, g.cluster, s);
}

template <typename T>
int launch_logprobs_grad(LogprobGradArgs a, int64_t slots, cudaStream_t s) {
    constexpr int E = Elem<T>::E;
    a.row.part = map_part(a.row.N, a.row.V, sizeof(T), kGradThreads, slots);
    const int64_t vectors = (a.row.V + 2LL * (E - 1)) / E, tiles = (vectors + a.row.part - 1) / a.row.part;
    if (a.row.N > 0x7fffffffLL / tiles) return GC_ERR_INVALID;
    a.tiles = static_cast<unsigned>(tiles);
    const unsigned grid = static_cast<unsigned>(a.row.N * tiles);
    if (a.g_entropy)
        k_token_logprobs_grad<T, true><<<grid, kGradThreads, 0, s>>>(a);
    else
        k_token_logprobs_grad<T, false><<<grid, kGradThreads, 0, s>>>(a);
    return launch_status();
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

int token_logprobs(const void* logits, gc_dtype dtype, int64_t ld, const void* ids, gc_id_type id_type, int64_t N, int64_t V,
                   double temperature, float* logprobs, float* entropy, float* lse, int K, int32_t* top_ids,
                   float* top_logprobs, int* d_status, gc_stream_t stream) {
    if (N < 0 || V < 1 || V > GC_MAX_VOCAB || ld < V || !valid_type(dtype) || !valid_id_type(id_type) ||
        !valid_temperature(temperature) || K < 0 || K > GC_MAX_TOP || K > V)
        return GC_ERR_INVALID;
    if (N == 0) return GC_OK;
    if (!logits || !ids || !logprobs || (K > 0 && (!top_ids || !top_logprobs))) return GC_ERR_INVALID;
    if (!aligned_to(logits, type_bytes(dtype)) || !aligned_to(ids, id_type == GC_I64 ? 8 : 4) || !aligned_to(logprobs, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(lse, 4) || !aligned_to(top_ids, 4) || !aligned_to(top_logprobs, 4) ||
        !aligned_to(d_status, 4))
        return GC_ERR_ALIGN;
    const int sms = grid_for(1);
    if (sms < 1) return GC_ERR_CUDA;
    LogprobArgs a;
    a.row.x = logits, a.row.ld = ld, a.row.N = N, a.row.V = static_cast<int>(V), a.row.part = 0;
    a.row.c2 = static_cast<float>(1.4426950408889634 / temperature);
    split_inverse(temperature, &a.row.inv_tau, &a.row.inv_tau_low);
    a.ids = ids, a.id64 = id_type == GC_I64, a.K = K;
    a.logprobs = logprobs, a.entropy = entropy, a.lse = lse, a.top_ids = top_ids, a.top_logprobs = top_logprobs;
    a.status = d_status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == GC_F32 ? launch_logprobs<float>(a, sms, s) : launch_logprobs<__nv_bfloat16>(a, sms, s);
}

int token_logprobs_grad(const void* logits, gc_dtype dtype, int64_t ld, const void* ids, gc_id_type id_type, int64_t N,
                        int64_t V, double temperature, const float* lse, const float* entropy, const float* g_logprobs,
                        const float* g_entropy, void* dlogits, int64_t ld_out, int* d_status, gc_stream_t stream) {
    if (N < 0 || V < 1 || V > kMaxMapped || ld < V || ld_out < V || !valid_type(dtype) || !valid_id_type(id_type) ||
        !valid_temperature(temperature))
        return GC_ERR_INVALID;
    if (N == 0) return GC_OK;
    if (!logits || !ids || !lse || !dlogits || (!g_logprobs && !g_entropy) || (g_entropy && !entropy)) return GC_ERR_INVALID;
    if (!aligned_to(logits, type_bytes(dtype)) || !aligned_to(dlogits, type_bytes(dtype)) ||
        !aligned_to(ids, id_type == GC_I64 ? 8 : 4) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) ||
        !aligned_to(g_logprobs, 4) || !aligned_to(g_entropy, 4) || !aligned_to(d_status, 4))
        return GC_ERR_ALIGN;
    const int sms = grid_for(1);
    if (sms < 1) return GC_ERR_CUDA;
    LogprobGradArgs a = {};
    a.row.x = logits, a.row.ld = ld, a.row.N = N, a.row.V = static_cast<int>(V);
    a.row.c2 = static_cast<float>(1.4426950408889634 / temperature);
    split_inverse(temperature, &a.row.inv_tau, &a.row.inv_tau_low);
    a.ids = ids, a.id64 = id_type == GC_I64;
    a.lse = lse, a.entropy = entropy, a.g_logprobs = g_logprobs, a.g_entropy = g_entropy;
    a.out = dlogits, a.ld_out = ld_out;
    a.status = d_status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == GC_F32 ? launch_logprobs_grad<float>(a, sms * kGradCtas, s)
                           : launch_logprobs_grad<__nv_bfloat16>(a, sms * kGradCtas, s);
}

}  // extern "C"
