// logit_rows.cuh -- a row of logits, cut into parts for the CTAs of a cluster,
// and the statistics of its softmax; shared by logprobs.cu and distill.cu.
#pragma once

#include "lm_common.cuh"

namespace gc {

constexpr int kMaxCluster = 8;              // the portable cluster size
constexpr int64_t kMaxMapped = 1LL << 30;   // longest row of the kernels that map it piece by piece: int indices

struct RowArgs {
    const void* x;
    int64_t ld;
    int64_t N;
    int V;
    int part;                               // vectors per CTA
    float c2;                               // log2(e) / temperature
    float inv_tau, inv_tau_low;             // 1 / temperature, and what it is above the first
};

// ---------------------------------------------------------------- cluster

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// Before a CTA writes another's memory, every CTA of the cluster has started:
// announce at the start, wait before the first write.
__device__ __forceinline__ void cluster_announce(unsigned parts) {
    if (parts > 1) cluster_arrive();
}
__device__ __forceinline__ void cluster_started(unsigned parts) {
    if (parts > 1) cluster_wait();
}
// What the cluster's CTAs have written is there for each of them.
__device__ __forceinline__ void cluster_join(unsigned parts) {
    if (parts > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}

// The address of `p` (shared memory of this CTA) in CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t remote_smem(const void* p, unsigned rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

__device__ __forceinline__ void st_remote(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void st_remote(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_remote(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// ---------------------------------------------------------------- the part of a row

constexpr int kWholeRow = 1 << 30;          // vectors: a part that holds any row

// A row starts anywhere, so its 16-byte vectors are counted from the aligned
// address at or below its start: the first and the last may have lanes outside
// the row ("ragged"), which are read by element and hold -inf.  A CTA has the
// vectors [v0, v1) of the row, of which [i0, i1) are whole.
template <typename T>
struct RowPart {
    static constexpr int E = Elem<T>::E;
    const T* row;
    int V, shift, v0, v1, i0, i1;

    __device__ __forceinline__ RowPart(const RowArgs& a, int64_t n, unsigned rank) : RowPart(a, n, rank, a.part) {}

    // The same with other parts than the launch's, of `part` vectors.
    __device__ __forceinline__ RowPart(const RowArgs& a, int64_t n, unsigned rank, int part) {
        row = static_cast<const T*>(a.x) + n * a.ld;
        V = a.V;
        shift = row_shift(row);
        const int last = (shift + V - 1) / E;
        v0 = min(static_cast<int>(rank) * part, last + 1);
        v1 = min(v0 + part, last + 1);
        i0 = v0, i1 = v1;
        if (v0 < v1) {
            if (v0 == 0 && shift != 0) i0 = 1;
            if (v1 == last + 1 && shift + V != (last + 1) * E) i1 = last;
            i1 = max(i0, i1);
        }
    }

    __device__ __forceinline__ bool whole(int v) const { return v >= i0 && v < i1; }

    // Index in the row of vector v's element e; outside [0, V) for lanes beyond the row.
    __device__ __forceinline__ int index(int v, int e) const { return v * E - shift + e; }

    __device__ __forceinline__ const uint4* vectors() const { return reinterpret_cast<const uint4*>(row - shift); }

    // Vector v of [v0, v1), whole or ragged.
    __device__ __forceinline__ uint4 load(int v) const {
        if (whole(v)) return __ldcg(vectors() + v);
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = index(v, e);
            f[e] = i >= 0 && i < V ? Elem<T>::load_plain(row + i) : neg_inf();
        }
        return Elem<T>::pack(f);
    }
};

// ---------------------------------------------------------------- softmax statistics

// With c = c2 = log2(e) / temperature: the largest logit m, and
//   s = sum 2^(c (x - m)),  u = sum 2^(c (x - m)) c (x - m)
// The difference comes before the product, so that the largest entry's exponent
// is exactly 0, an offset common to the row cancels, and rows of the type's
// lowest values do not overflow.  m is NaN once a NaN has been seen, and s is
// NaN for a row with a NaN or +inf.
struct Stat {
    float m, s, u;
};

// The same while a thread adds to it: even and odd elements apart.
struct Sums {
    float m;
    uint64_t s, u;
};

__device__ __forceinline__ float exponent(float x, float m, float c2) { return (x - m) * c2; }

// The factor of the sums, and what their exponents change by, when the
// reference goes from `from` to `to` (above it, or NaN).
__device__ __forceinline__ float rescale(float from, float to, float c2, float* change) {
    *change = max_nan(exponent(from, to, c2), -150.0f);
    return exp2_fast(*change);
}

__device__ __forceinline__ void raise(Stat& st, float m, float c2) {
    float d;
    const float f = rescale(st.m, m, c2, &d);
    st.u = f * fmaf(d, st.s, st.u);
    st.s *= f;
    st.m = m;
}

__device__ __forceinline__ void raise(Sums& st, float m, float c2) {
    float d;
    const float f = rescale(st.m, m, c2, &d);
    st.u = pair_mul(pair(f, f), pair_fma(pair(d, d), st.s, st.u));
    st.s = pair_mul(pair(f, f), st.s);
    st.m = m;
}

// Values below -2^60 do not differ from masked ones while |m| < 2^60: their
// power is zero.  Raising them to -2^60 keeps 0 * (-inf) out of u.
constexpr float kFloor = -1152921504606846976.0f;
constexpr uint32_t kFloorBf16x2 = 0xdd80dd80u;

// Whether a gradient may form log p as x / tau - lse.  lse is rounded to fp32: at
// 1024 that is 2^-15 of p, and at 1e9 nothing of the sum's logarithm is left (a
// row of one value would have p = 1 in every place).  Other rows, NaN and the
// infinities among them, need their own maximum and sum.  Below 1024 the largest
// logit is above -1024 tau, so a power that was raised to -2^60 is zero.
__device__ __forceinline__ bool lse_holds(float lse) { return fabsf(lse) < 1024.0f; }

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The vector with everything below -2^60 raised to it.
template <typename T>
__device__ __forceinline__ uint4 floored(uint4 w) {
    if (sizeof(T) == 2)
        return make_uint4(max_bf16x2(w.x, kFloorBf16x2), max_bf16x2(w.y, kFloorBf16x2), max_bf16x2(w.z, kFloorBf16x2),
                          max_bf16x2(w.w, kFloorBf16x2));
    return make_uint4(__float_as_uint(max_nan(__uint_as_float(w.x), kFloor)),
                      __float_as_uint(max_nan(__uint_as_float(w.y), kFloor)),
                      __float_as_uint(max_nan(__uint_as_float(w.z), kFloor)),
                      __float_as_uint(max_nan(__uint_as_float(w.w), kFloor)));
}

// The largest element of n vectors, NaN if any is.
template <typename T, int N>
__device__ __forceinline__ float batch_max(const uint4 (&w)[N]) {
    if (sizeof(T) == 2) {
        uint32_t m = max_bf16x2(max_bf16x2(w[0].x, w[0].y), max_bf16x2(w[0].z, w[0].w));
#pragma unroll
        for (int k = 1; k < N; ++k)
            m = max_bf16x2(m, max_bf16x2(max_bf16x2(w[k].x, w[k].y), max_bf16x2(w[k].z, w[k].w)));
        return max_nan(bf16lo(m), bf16hi(m));
    }
    float m = neg_inf();
#pragma unroll
    for (int k = 0; k < N; ++k)
        m = max_nan(m, max_nan(max_nan(__uint_as_float(w[k].x), __uint_as_float(w[k].y)),
                               max_nan(__uint_as_float(w[k].z), __uint_as_float(w[k].w))));
    return m;
}

// Adds two logits to the sums.
template <bool ENTROPY>
__device__ __forceinline__ void add_pair(Sums& st, float a, float b, uint64_t minus_m, uint64_t cc) {
    const uint64_t y = pair_mul(pair_add(pair(a, b), minus_m), cc);
    float y0, y1;
    unpair(y, y0, y1);
    const uint64_t p = pair(exp2_fast(y0), exp2_fast(y1));
    st.s = pair_add(st.s, p);
    if (ENTROPY) st.u = pair_fma(p, y, st.u);
}

template <typename T, bool ENTROPY, int N>
__device__ __forceinline__ void accumulate(Sums& st, const uint4 (&w)[N], float vm, float c2) {
    if (!(vm <= st.m) && st.m == st.m) raise(st, vm, c2);
    if (fabsf(st.m) < -kFloor) {
        const uint64_t minus_m = pair(-st.m, -st.m), cc = pair(c2, c2);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float f[Elem<T>::E];
            Elem<T>::unpack(ENTROPY ? floored<T>(w[k]) : w[k], f);
#pragma unroll
            for (int e = 0; e < Elem<T>::E; e += 2) add_pair<ENTROPY>(st, f[e], f[e + 1], minus_m, cc);
        }
    } else if (st.m != neg_inf()) {         // not a real logit: huge, infinite or NaN
        float s = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float f[Elem<T>::E];
            Elem<T>::unpack(w[k], f);
#pragma unroll
            for (int e = 0; e < Elem<T>::E; ++e) {
                const float y = max_nan(exponent(f[e], st.m, c2), -150.0f), p = exp2_fast(y);
                s += p;
                u = fmaf(p, y, u);
            }
        }
        st.s = pair_add(st.s, pair(s, 0.0f));
        st.u = pair_add(st.u, pair(u, 0.0f));
    }
}

__device__ __forceinline__ Stat finish(const Sums& st) {
    float s0, s1, u0, u1;
    unpair(st.s, s0, s1);
    unpair(st.u, u0, u1);
    return Stat{st.m, s0 + s1, u0 + u1};
}

// Shared-memory scratch of the joins.
constexpr int kMaxRowWarps = 8;

struct StatSmem {
    float warp_m[kMaxRowWarps], warp_s[kMaxRowWarps], warp_u[kMaxRowWarps];
    float part[kMaxCluster][4];             // (m, s, u) of each CTA of the cluster
};

// The CTA's statistics from TH threads, the same in every thread.  Warps above
// these take part in the barriers alone.
template <int TH>
__device__ __forceinline__ Stat block_stats(StatSmem& sm, Stat st, float c2) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = warp_max_nan(st.m);
    if (lane == 0 && warp < TH / 32) sm.warp_m[warp] = m;
    __syncthreads();
    m = sm.warp_m[0];
#pragma unroll
    for (int w = 1; w < TH / 32; ++w) m = max_nan(m, sm.warp_m[w]);
    if (m != st.m) raise(st, m, c2);
    const float s = warp_sum(st.s), u = warp_sum(st.u);
    if (lane == 0 && warp < TH / 32) sm.warp_s[warp] = s, sm.warp_u[warp] = u;
    __syncthreads();
    Stat r{m, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < TH / 32; ++w) r.s += sm.warp_s[w], r.u += sm.warp_u[w];
    return r;
}

// The row's statistics from its parts.
__device__ __forceinline__ Stat join_parts(const float (&part)[kMaxCluster][4], unsigned parts, float c2) {
    float m = neg_inf();
    for (unsigned k = 0; k < parts; ++k) m = max_nan(m, part[k][0]);
    Stat r{m, 0.0f, 0.0f};
    for (unsigned k = 0; k < parts; ++k) {
        Stat st{part[k][0], part[k][1], part[k][2]};
        if (st.m != m) raise(st, m, c2);
        r.s += st.s;
        r.u += st.u;
    }
    return r;
}

// The log probability of logit x.
__device__ __forceinline__ float log_prob(const Stat& st, float ln_s, float x, const RowArgs& a) {
    return st.m == neg_inf() ? neg_inf() : fmaf(x - st.m, a.inv_tau, -ln_s);
}

// With 1 / temperature in two terms, as the gradients take it: one alone is off
// by up to 2^-24 of lse, twice lse's own rounding.
__device__ __forceinline__ float row_lse(const Stat& st, float ln_s, const RowArgs& a) {
    return st.m == neg_inf() ? neg_inf() : fmaf(st.m, a.inv_tau, fmaf(st.m, a.inv_tau_low, ln_s));
}

// ---------------------------------------------------------------- launch

// Launches `clusters` clusters of `cluster` CTAs with `smem` bytes of dynamic
// shared memory each, of `most` that the kernel ever takes.
template <typename Args>
int launch_rows(void (*kernel)(Args), int cluster, int64_t clusters, int threads, size_t smem, size_t most, const Args& a,
                cudaStream_t s) {
    if (clusters > 0x7fffffffLL / cluster) return GC_ERR_INVALID;
    if (allow_smem(kernel, smem, most) != GC_OK) return GC_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return GC_ERR_CUDA;
    }
    return GC_OK;
}

}  // namespace gc
