// distill.cu -- distillation from a teacher's top logits: loss, gradient, and
// both in one pass.
//
//   q = softmax(t / tau) over the row's present entries,  p = softmax(x / tau)
//   loss = tau^2 sum_k q_k (log q_k - log p[id_k])
//   d_j  = w tau (p_j - sum_{k: id_k = j} q_k)
//
// The loss reads each logit once; the gradient reads and writes each once (rows
// with |lse| >= 1024 are read twice), and so does, in memory, the loss with its gradient: its second reading of a row
// comes from L2.
#include "logit_stream.cuh"

namespace gc {
namespace {

struct DistillArgs {
    RowArgs row;
    const int32_t* top_ids;
    const float* top_logits;
    int K;
    float tau;
    const float* weights;
    float* loss;
    float* lse;
    void* out;
    int64_t ld_out;
    int* status;
};

// A row's teacher entries: id (-1: absent, or no probability), q, log q.
struct Teacher {
    int id[GC_MAX_TOP];
    float q[GC_MAX_TOP], log_q[GC_MAX_TOP];
    bool mass;                              // whether any entry has probability
};

// By one warp, four entries a lane.
__device__ __forceinline__ void load_teacher(Teacher& t, const int32_t* ids, const float* logits, int K, int64_t V,
                                             float c2, int* status) {
    const int lane = threadIdx.x & 31;
    constexpr int kPer = GC_MAX_TOP / 32;
    int id[kPer];
    float x[kPer], m = neg_inf();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        id[i] = -1;
        x[i] = neg_inf();
        if (k < K) {
            id[i] = static_cast<int>(load_id(ids, k, V, status));
            x[i] = __ldg(logits + k);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (id[i] < 0) x[i] = neg_inf();
        m = max_nan(m, x[i]);
    }
    m = warp_max_nan(m);
    float e[kPer], y[kPer], z = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        y[i] = m == neg_inf() ? -150.0f : max_nan((x[i] - m) * c2, -150.0f);
        e[i] = exp2_fast(y[i]);
        z += e[i];
    }
    z = warp_sum(z);
    const float log2_z = log2f(z);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        if (k < K) {
            const float q = z == 0.0f ? 0.0f : e[i] / z;
            t.id[k] = q == 0.0f ? -1 : id[i];
            t.q[k] = q;
            t.log_q[k] = (y[i] - log2_z) * kLn2;
        }
    }
    if (lane == 0) t.mass = z != 0.0f;
}

// The entries of a teacher that lie in one part of the row, in their order.
constexpr int kOwnSlots = 512;
constexpr int kTwice = 1 << 31;             // of a slot: the id occurs more than once

struct Own {
    int id[GC_MAX_TOP];                     // to a multiple of 4: -1
    float q[GC_MAX_TOP];
    int slot[kOwnSlots];                    // a hash table of the ids (0: free, else id + 1)
};

// The slot of an id that has one, or the free slot where it belongs: at most 128
// of 512 are taken, so one of the two is met.
template <typename F>
__device__ __forceinline__ void probe(int id, F stop) {
    for (uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) >> 23; !stop(h); h = (h + 1) & (kOwnSlots - 1)) {
    }
}

// Collects the entries with ids in [lo, hi); returns their count.  By one warp.
__device__ __forceinline__ int collect_own(Own& own, const Teacher& t, int K, int lo, int hi) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kOwnSlots / 128; ++k)
        reinterpret_cast<int4*>(own.slot)[32 * k + lane] = make_int4(0, 0, 0, 0);
    reinterpret_cast<int4*>(own.id)[lane] = make_int4(-1, -1, -1, -1);
    __syncwarp();
    int n = 0;
    for (int k0 = 0; k0 < K; k0 += 32) {
        const int id = k0 + lane < K ? t.id[k0 + lane] : -1;
        const bool mine = id >= 0 && id >= lo && id < hi;
        const unsigned m = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const int at = n + __popc(m & ((1u << lane) - 1u));
            own.id[at] = id;
            own.q[at] = t.q[k0 + lane];
            probe(id, [&](uint32_t h) {
                const int old = atomicCAS(&own.slot[h], 0, id + 1);
                if (old == 0) return true;
                if ((old & ~kTwice) != id + 1) return false;
                atomicOr(&own.slot[h], kTwice);
                return true;
            });
        }
        n += __popc(m);
    }
    __syncwarp();
    return n;
}

// The sum of q over the entries with entry k's id, for the first of them; the
// others return a negative number.  A teacher's ids seldom repeat.
__device__ __forceinline__ float merged_q(const Own& own, int k, int n) {
    const int id = own.id[k];
    bool twice = false;
    probe(id, [&](uint32_t h) {
        twice = own.slot[h] < 0;
        return (own.slot[h] & ~kTwice) == id + 1;
    });
    if (!twice) return own.q[k];
    float q = 0.0f;
    for (int j = 0; j < n; j += 4) {
        const int4 four = *reinterpret_cast<const int4*>(&own.id[j]);
        const int ids[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ids[i] != id) continue;
            if (j + i < k) return -1.0f;
            q += own.q[j + i];
        }
    }
    return q;
}

// The student's logits at a row's teacher entries, four a lane.
template <typename T>
__device__ __forceinline__ void load_student(const Teacher& t, const T* row, int K, float (&x)[GC_MAX_TOP / 32]) {
#pragma unroll
    for (int i = 0; i < GC_MAX_TOP / 32; ++i) {
        const int k = (threadIdx.x & 31) + 32 * i;
        x[i] = k < K && t.id[k] >= 0 ? Elem<T>::load_before(row + t.id[k]) : 0.0f;
    }
}

// A row's loss, by one warp.
__device__ __forceinline__ float row_loss(const Teacher& t, const float (&x)[GC_MAX_TOP / 32], const Stat& st, float ln_s,
                                          const DistillArgs& a) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < GC_MAX_TOP / 32; ++i) {
        const int k = (threadIdx.x & 31) + 32 * i;
        if (k < a.K && t.id[k] >= 0) sum += t.q[k] * (t.log_q[k] - log_prob(st, ln_s, x[i], a.row));
    }
    sum = warp_sum(sum);
    return t.mass ? sum * (a.tau * a.tau) : 0.0f;
}

// ---------------------------------------------------------------- loss

template <typename T, int TH>
__global__ void __launch_bounds__(TH, kStreamThreads / TH) k_distill_loss(DistillArgs a) {
    __shared__ StatSmem stat_smem;
    __shared__ Teacher teacher;
    const unsigned rank = cluster_rank(), parts = cluster_size();
    const int64_t n = blockIdx.x / parts;
    cluster_announce(parts);
    const RowPart<T> p(a.row, n, rank);
    const Units<TH> units(p);
    const Stat mine = stream_stats<TH, false, false>(p, units, a.row.c2, [](int, float) {});
    float x[GC_MAX_TOP / 32];
    if (rank == 0 && threadIdx.x < 32) {
        load_teacher(teacher, a.top_ids + n * a.K, a.top_logits + n * a.K, a.K, a.row.V, a.row.c2, a.status);
        __syncwarp();
        load_student(teacher, p.row, a.K, x);
    }
    const Stat cta = block_stats<TH>(stat_smem, mine, a.row.c2);
    cluster_started(parts);
    if (threadIdx.x < 3) {
        const float v = threadIdx.x == 0 ? cta.m : threadIdx.x == 1 ? cta.s : 0.0f;
        st_remote(remote_smem(&stat_smem.part[rank][threadIdx.x], 0), v);
    }
    cluster_join(parts);
    if (rank != 0 || threadIdx.x >= 32) return;
    const Stat st = join_parts(stat_smem.part, parts, a.row.c2);
    const float ln_s = logf(st.s);
    const float loss = row_loss(teacher, x, st, ln_s, a);
    if (threadIdx.x == 0) {
        a.loss[n] = loss;
        if (a.lse) a.lse[n] = row_lse(st, ln_s, a.row);
    }
}

// ---------------------------------------------------------------- loss and gradient

// A cluster works on a row, a contiguous part per CTA: first the part's
// statistics, then, once the cluster has joined them, the part's gradient, for
// which the part is read from L2 again.  The rows under work on all SMs are a
// fraction of L2, so memory sees each logit once.  A warp of its own takes the
// teacher's side: entries, loss, and the corrections of the few gradients that
// have a q.
constexpr int kRowThreads = 256;
constexpr int kTeacherThreads = kRowThreads + 32;
constexpr int kStepCtas = 4;                // resident per SM

// Barrier 1: the row's threads arrive, the teacher's warp waits for them.
__device__ __forceinline__ void rows_arrive() { asm volatile("bar.arrive 1, %0;" ::"n"(kTeacherThreads) : "memory"); }
__device__ __forceinline__ void teacher_wait() { asm volatile("bar.sync 1, %0;" ::"n"(kTeacherThreads) : "memory"); }
// Barrier 2: both wait for each other.
__device__ __forceinline__ void entries_ready() { asm volatile("bar.sync 2, %0;" ::"n"(kTeacherThreads) : "memory"); }

// Writes g p = gs 2^(c2 (x - m)) over a part of a row; zeros where it has none.
template <typename T>
__device__ __forceinline__ void map_gradient(const RowPart<T>& p, T* out, bool none, float gs, float m, float c2) {
    constexpr int E = Elem<T>::E;
    const uint64_t minus_m = pair(-m, -m), cc = pair(c2, c2), gg = pair(gs, gs);
    stream_map<kRowThreads>(p, out, [&](int, uint4 x) {
        if (none) return make_uint4(0, 0, 0, 0);
        float f[E];
        Elem<T>::unpack(x, f);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            float y0, y1;
            unpair(pair_mul(pair_add(pair(f[e], f[e + 1]), minus_m), cc), y0, y1);
            unpair(pair_mul(pair(exp2_fast(y0), exp2_fast(y1)), gg), f[e], f[e + 1]);
        }
        return Elem<T>::pack(f);
    });
}

// The gradients g p - g q at the part's entries, whose logits are x, after the
// part's threads have written theirs.  By the teacher's warp.
template <typename T, typename P>
__device__ __forceinline__ void correct_entries(const Own& own, int n_own, bool zero, const float (&x)[GC_MAX_TOP / 32], T* out,
                                                float g, P g_prob) {
    constexpr int kPer = GC_MAX_TOP / 32;
    const int lane = threadIdx.x & 31;
    float fix[kPer];
    bool first[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        first[i] = false;
        if (k < n_own && !zero) {
            const float q = merged_q(own, k, n_own);
            first[i] = !(q < 0.0f);
            fix[i] = fmaf(-g, q, g_prob(x[i]));
        }
    }
    teacher_wait();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (first[i]) out[own.id[lane + 32 * i]] = Elem<T>::round_to(fix[i]);
}

template <typename T>
__global__ void __launch_bounds__(kTeacherThreads, kStepCtas) k_distill_loss_grad(DistillArgs a) {
    constexpr int kPer = GC_MAX_TOP / 32;
    __shared__ StatSmem stat_smem;
    __shared__ Teacher teacher;
    __shared__ __align__(16) Own own;
    const unsigned rank = cluster_rank(), parts = cluster_size();
    const bool rows = threadIdx.x < kRowThreads;
    const int lane = threadIdx.x & 31;
    const float c2 = a.row.c2;
    const int64_t n = blockIdx.x / parts;
    cluster_announce(parts);
    const RowPart<T> p(a.row, n, rank);
    Stat mine{neg_inf(), 0.0f, 0.0f};
    float x_all[kPer], x_own[kPer];         // read before the row is overwritten
    int n_own = 0;
    if (rows) {
        const Units<kRowThreads> units(p);
        mine = stream_stats<kRowThreads, false, true>(p, units, c2, [](int, float) {});
    } else {
        load_teacher(teacher, a.top_ids + n * a.K, a.top_logits + n * a.K, a.K, a.row.V, c2, rank == 0 ? a.status : nullptr);
        __syncwarp();
        if (rank == 0) load_student(teacher, p.row, a.K, x_all);
        n_own = collect_own(own, teacher, a.K, p.index(p.v0, 0), p.index(p.v1, 0));
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < n_own) x_own[i] = Elem<T>::load_before(p.row + own.id[lane + 32 * i]);
    }
    const Stat cta = block_stats<kRowThreads>(stat_smem, mine, c2);
    cluster_started(parts);
    if (threadIdx.x < parts) {
        st_remote(remote_smem(&stat_smem.part[rank][0], threadIdx.x), cta.m);
        st_remote(remote_smem(&stat_smem.part[rank][1], threadIdx.x), cta.s);
        st_remote(remote_smem(&stat_smem.part[rank][2], threadIdx.x), 0.0f);
    }
    const float w = __ldg(a.weights + n);
    cluster_join(parts);
    const Stat st = join_parts(stat_smem.part, parts, c2);
    const bool zero = w == 0.0f || !teacher.mass;
    const bool none = zero || st.m == neg_inf();
    const float g = w * a.tau;
    const float gs = none ? 0.0f : g / st.s;
    T* out = static_cast<T*>(a.out) + n * a.ld_out;
    if (rows) {
        map_gradient(p, out, none, gs, st.m, c2);
        rows_arrive();
    } else {
        if (rank == 0) {
            const float loss = row_loss(teacher, x_all, st, logf(st.s), a);
            if (lane == 0) a.loss[n] = loss;
        }
        correct_entries(own, n_own, zero, x_own, out, g,
                        [&](float x) { return none ? 0.0f : gs * exp2_fast(exponent(x, st.m, c2)); });
    }
}

// ---------------------------------------------------------------- gradient alone

constexpr int kGradCtas = 4;                // resident per SM

struct DistillGradArgs {
    RowArgs row;
    const int32_t* top_ids;
    const float* top_logits;
    unsigned tiles;                         // CTAs per row
    int K;
    float tau;
    const float* lse;
    const float* weights;
    void* out;
    int64_t ld_out;
    int* status;
};

// The teacher's side of a part, by its warp; the entries that lie in it are counted in n_own.
template <typename T>
struct PartEntries {
    float x[GC_MAX_TOP / 32];               // the student's logits at the part's entries
    int n_own;

    __device__ __forceinline__ void find(const DistillGradArgs& a, int64_t n, const RowPart<T>& p, Teacher& teacher, Own& own,
                                         int* status) {
        load_teacher(teacher, a.top_ids + n * a.K, a.top_logits + n * a.K, a.K, a.row.V, a.row.c2, status);
        __syncwarp();
        n_own = collect_own(own, teacher, a.K, p.index(p.v0, 0), p.index(p.v1, 0));
    }

    __device__ __forceinline__ void gather(const RowPart<T>& p, const Own& own) {
#pragma unroll
        for (int i = 0; i < GC_MAX_TOP / 32; ++i) {
            const int k = (threadIdx.x & 31) + 32 * i;
            if (k < n_own) x[i] = Elem<T>::load_before(p.row + own.id[k]);
        }
    }
};

// The gradient of a row whose lse does not hold its sum, by one CTA: the row is
// read once more before, and nothing is written until then, so it may be in
// place.  2048 x 131072 bf16 of -1e9 with 64 entries take 245 us, where usual
// rows take 163; 300 x 50001 fp32 36 and 20.
template <typename T>
__device__ __noinline__ void whole_row_grad(const DistillGradArgs& a, int64_t n, Teacher& teacher, Own& own) {
    __shared__ StatSmem stat_smem;
    const RowPart<T> p(a.row, n, 0, kWholeRow);
    const bool rows = threadIdx.x < kRowThreads;
    const float c2 = a.row.c2, g = __ldg(a.weights + n) * a.tau;
    T* out = static_cast<T*>(a.out) + n * a.ld_out;
    PartEntries<T> entries;
    if (!rows) {
        entries.find(a, n, p, teacher, own, a.status);
        entries.gather(p, own);
    }
    const Stat st = whole_row_stats<kRowThreads>(p, stat_smem, c2);
    const bool zero = !teacher.mass, none = zero || st.m == neg_inf();
    const float gs = none ? 0.0f : g / st.s;
    if (rows) {
        map_gradient(p, out, none, gs, st.m, c2);
        rows_arrive();
    } else {
        correct_entries(own, entries.n_own, zero, entries.x, out, g,
                        [&](float x) { return none ? 0.0f : gs * exp2_fast(exponent(x, st.m, c2)); });
    }
}

// One CTA per piece of a row, or one for a row whose lse does not hold its sum,
// with a warp of its own for the teacher's entries.
template <typename T>
__global__ void __launch_bounds__(kTeacherThreads, kGradCtas) k_distill_grad(const __grid_constant__ DistillGradArgs a) {
    constexpr int E = Elem<T>::E;
    __shared__ Teacher teacher;
    __shared__ __align__(16) Own own;
    const int64_t n = blockIdx.x / a.tiles;
    const unsigned tile = blockIdx.x % a.tiles;
    const float lse = __ldg(a.lse + n), weight = __ldg(a.weights + n), inv_tau = a.row.inv_tau;
    const RowPart<T> p(a.row, n, tile);
    T* out = static_cast<T*>(a.out) + n * a.ld_out;
    const bool rows = threadIdx.x < kRowThreads, in_place = a.out == a.row.x;
    const float g = weight * a.tau;
    // a row without a weight is zeros, whatever its lse
    const bool holds = lse_holds(lse) || weight == 0.0f;
    if (rows) {
        bool zero = false;
        auto go = [&]() {                               // the teacher's entries are there
            entries_ready();
            if (!holds) return false;
            zero = weight == 0.0f || !teacher.mass;
            return true;
        };
        stream_map<kRowThreads>(p, out, go, [&](int, uint4 w) {
            float f[E];
            if (zero) return make_uint4(0, 0, 0, 0);
            Elem<T>::unpack(floored<T>(w), f);          // masked entries at -2^60: p is 0
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                // log p = y - lse in natural units, so that neither the rounding of
                // lse * log2(e) nor that of 1 / tau scales the row
                const uint64_t lp = log_prob_pair(pair(f[e], f[e + 1]), lse, inv_tau, a.row.inv_tau_low);
                float y0, y1;
                unpair(pair_mul(lp, pair(kLog2e, kLog2e)), y0, y1);
                unpair(pair_mul(pair(exp2_fast(y0), exp2_fast(y1)), pair(g, g)), f[e], f[e + 1]);
            }
            return Elem<T>::pack(f);
        });
        if (holds) rows_arrive();
    } else {
        PartEntries<T> entries;
        entries.find(a, n, p, teacher, own, tile == 0 ? a.status : nullptr);
        if (in_place) entries.gather(p, own);           // before any of them is overwritten
        entries_ready();
        if (holds) {
            if (!in_place) entries.gather(p, own);
            correct_entries(own, entries.n_own, weight == 0.0f || !teacher.mass, entries.x, out, g,
                            [&](float x) { return g * exp2_fast(log_prob_from(x, lse, inv_tau, a.row.inv_tau_low) * kLog2e); });
        }
    }
    if (!holds && tile == 0) whole_row_grad<T>(a, n, teacher, own);
}

// ---------------------------------------------------------------- host

int check_distill(const void* logits, int dtype, int64_t ld, const int32_t* top_ids, const float* top_logits, int K,
                  int64_t N, int64_t V, int64_t max_v, double temperature, int* d_status) {
    if (N < 0 || V < 1 || V > max_v || ld < V || !valid_type(dtype) || !valid_temperature(temperature) || K < 1 || K > GC_MAX_TOP)
        return GC_ERR_INVALID;
    if (N == 0) return GC_OK;
    if (!logits || !top_ids || !top_logits) return GC_ERR_INVALID;
    if (!aligned_to(logits, type_bytes(dtype)) || !aligned_to(top_ids, 4) || !aligned_to(top_logits, 4) ||
        !aligned_to(d_status, 4))
        return GC_ERR_ALIGN;
    return GC_OK;
}

template <typename T>
int launch_loss(DistillArgs a, cudaStream_t s) {
    const int sms = grid_for(1);
    if (sms < 1) return GC_ERR_CUDA;
    const StreamGeometry g = stream_geometry(a.row.N, a.row.V, sizeof(T), 0, sms);
    a.row.part = g.part;
    return g.threads == 128 ? launch_rows(k_distill_loss<T, 128>, g.cluster, a.row.N, 128, 0, 0, a, s)
                            : launch_rows(k_distill_loss<T, 256>, g.cluster, a.row.N, 256, 0, 0, a, s);
}

// The part of a row that a CTA works on at most: 608 parts of 87 KB (a row of
// 256 KB in three) leave L2 room for the lines that come and go, with 8192 such
// rows 785 us; parts of 128 KB begin to be read twice (793 us), parts of 64 KB
// spend more on joins (813 us).
constexpr int64_t kStepPartBytes = 110 * 1024;
constexpr int64_t kMinStepPartBytes = 8 * 1024;

// The smallest cluster whose parts are no larger than kStepPartBytes, and a
// larger one while the rows leave half of the SMs without a CTA and the parts
// stay long.
template <typename T>
int launch_loss_grad(DistillArgs a, cudaStream_t s) {
    const int sms = grid_for(1);
    if (sms < 1) return GC_ERR_CUDA;
    constexpr int E = Elem<T>::E;
    const int64_t bytes = 16 * ((a.row.V + E - 1 + E - 1) / E);    // any alignment of the row
    int cluster = 1;
    while (cluster < kMaxCluster && bytes > cluster * kStepPartBytes) ++cluster;
    while (cluster * 2 <= kMaxCluster && a.row.N <= sms / (cluster * 2) && bytes > cluster * 2 * kMinStepPartBytes) cluster *= 2;
    a.row.part = static_cast<int>((bytes / 16 + cluster - 1) / cluster);
    return launch_rows(k_distill_loss_grad<T>, cluster, a.row.N, kTeacherThreads, 0, 0, a, s);
}

DistillArgs distill_args(const void* logits, int64_t ld, const int32_t* top_ids, const float* top_logits, int K, int64_t N,
                         int64_t V, double temperature, float* loss, int* d_status) {
    DistillArgs a = {};
    a.row.x = logits, a.row.ld = ld, a.row.N = N, a.row.V = static_cast<int>(V);
    a.row.c2 = static_cast<float>(1.4426950408889634 / temperature);
    split_inverse(temperature, &a.row.inv_tau, &a.row.inv_tau_low);
    a.top_ids = top_ids, a.top_logits = top_logits, a.K = K, a.tau = static_cast<float>(temperature);
    a.loss = loss;
    a.status = d_status;
    return a;
}

template <typename T>
int launch_grad(DistillGradArgs a, int64_t slots, cudaStream_t s) {
    constexpr int E = Elem<T>::E;
    a.row.part = map_part(a.row.N, a.row.V, sizeof(T), kRowThreads, slots);
    const int64_t vectors = (a.row.V + 2LL * (E - 1)) / E, tiles = (vectors + a.row.part - 1) / a.row.part;
    if (a.row.N > 0x7fffffffLL / tiles) return GC_ERR_INVALID;
    a.tiles = static_cast<unsigned>(tiles);
    k_distill_grad<T><<<static_cast<unsigned>(a.row.N * tiles), kTeacherThreads, 0, s>>>(a);
    return launch_status();
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

int distill_loss(const void* logits, gc_dtype dtype, int64_t ld, const int32_t* top_ids, const float* top_logits, int K,
                 int64_t N, int64_t V, double temperature, float* loss, float* lse, int* d_status, gc_stream_t stream) {
    const int rc = check_distill(logits, dtype, ld, top_ids, top_logits, K, N, V, GC_MAX_VOCAB, temperature, d_status);
    if (rc != GC_OK || N == 0) return rc;
    if (!loss) return GC_ERR_INVALID;
    if (!aligned_to(loss, 4) || !aligned_to(lse, 4)) return GC_ERR_ALIGN;
    DistillArgs a = distill_args(logits, ld, top_ids, top_logits, K, N, V, temperature, loss, d_status);
    a.lse = lse;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == GC_F32 ? launch_loss<float>(a, s) : launch_loss<__nv_bfloat16>(a, s);
}

int distill_loss_grad(const void* logits, gc_dtype dtype, int64_t ld, const int32_t* top_ids, const float* top_logits, int K,
                      int64_t N, int64_t V, double temperature, const float* weights, float* loss, void* dlogits,
                      int64_t ld_out, int* d_status, gc_stream_t stream) {
    const int rc = check_distill(logits, dtype, ld, top_ids, top_logits, K, N, V, GC_MAX_VOCAB, temperature, d_status);
    if (rc != GC_OK) return rc;
    if (ld_out < V) return GC_ERR_INVALID;
    if (N == 0) return GC_OK;
    if (!loss || !weights || !dlogits) return GC_ERR_INVALID;
    if (!aligned_to(loss, 4) || !aligned_to(weights, 4) || !aligned_to(dlogits, type_bytes(dtype))) return GC_ERR_ALIGN;
    DistillArgs a = distill_args(logits, ld, top_ids, top_logits, K, N, V, temperature, loss, d_status);
    a.weights = weights, a.out = dlogits, a.ld_out = ld_out;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == GC_F32 ? launch_loss_grad<float>(a, s) : launch_loss_grad<__nv_bfloat16>(a, s);
}

int distill_grad(const void* logits, gc_dtype dtype, int64_t ld, const int32_t* top_ids, const float* top_logits, int K,
                 int64_t N, int64_t V, double temperature, const float* lse, const float* weights, void* dlogits,
                 int64_t ld_out, int* d_status, gc_stream_t stream) {
    const int rc =
        check_distill(logits, dtype, ld, top_ids, top_logits, K, N, V, kMaxMapped, temperature, d_status);
    if (rc != GC_OK) return rc;
    if (ld_out < V) return GC_ERR_INVALID;
    if (N == 0) return GC_OK;
    if (!lse || !weights || !dlogits) return GC_ERR_INVALID;
    if (!aligned_to(lse, 4) || !aligned_to(weights, 4) || !aligned_to(dlogits, type_bytes(dtype))) return GC_ERR_ALIGN;
    const int sms = grid_for(1);
    if (sms < 1) return GC_ERR_CUDA;
    DistillGradArgs a = {};
    a.row.x = logits, a.row.ld = ld, a.row.N = N, a.row.V = static_cast<int>(V);
    a.row.c2 = static_cast<float>(1.4426950408889634 / temperature);
    split_inverse(temperature, &a.row.inv_tau, &a.row.inv_tau_low);
    a.top_ids = top_ids, a.top_logits = top_logits, a.K = K;
    a.tau = static_cast<float>(temperature);
    a.lse = lse, a.weights = weights, a.out = dlogits, a.ld_out = ld_out;
    a.status = d_status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == GC_F32 ? launch_grad<float>(a, sms * kGradCtas, s) : launch_grad<__nv_bfloat16>(a, sms * kGradCtas, s);
}

}  // extern "C"
