// lm_common.cuh -- what the language-model kernels (embed.cu, logprobs.cu,
// distill.cu) share: argument checks, the limit of dynamic shared memory,
// 16-byte vectors of either element type, token ids, the base-2 exponential and
// log probabilities from a stored lse.
#pragma once

#include "gc_common.cuh"

namespace gc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

inline bool valid_type(int t) { return t == GC_F32 || t == GC_BF16; }
inline bool valid_id_type(int t) { return t == GC_I32 || t == GC_I64; }
inline size_t type_bytes(int t) { return t == GC_F32 ? 4 : 2; }
// Within it, logits up to 2^60 have finite exponents, and those 2^52 apart or
// more the power zero (logit_rows.cuh).
inline bool valid_temperature(double t) { return t >= 1e-6 && t <= 1e6; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------- shared memory

// The dynamic shared memory that a kernel gets without asking: 48 KB less its
// static memory, for which 4 KB are left.
constexpr size_t kUnaskedSmem = 44 * 1024;

// Lets launches of `kernel` have `smem` bytes of dynamic shared memory.  The
// limit belongs to the kernel on the device, not to the call: another host
// thread may be between asking and launching, so every call asks for the same,
// the most that the kernel ever takes.
template <typename Kernel>
int allow_smem(Kernel* kernel, size_t smem, size_t most) {
    if (smem > kUnaskedSmem && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    static_cast<int>(most)) != cudaSuccess) {
        cudaGetLastError();
        return GC_ERR_CUDA;
    }
    return GC_OK;
}

// ---------------------------------------------------------------- elements

// Reads of memory that this kernel also writes, its other threads and CTAs among
// them: volatile, so that the compiler keeps them on their side of a barrier (a
// logit read before its gradient takes its place, a part of a sum read after the
// counter said that it is there).  From L2, where other SMs' writes are.
__device__ __forceinline__ float load_ordered(const float* p) {
    float x;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(x) : "l"(__cvta_generic_to_global(p)) : "memory");
    return x;
}
__device__ __forceinline__ unsigned short load_ordered(const unsigned short* p) {
    unsigned short x;
    asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(x) : "l"(__cvta_generic_to_global(p)) : "memory");
    return x;
}
__device__ __forceinline__ float4 load_ordered(const float4* p) {
    float4 x;
    asm volatile("ld.global.cg.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "l"(__cvta_generic_to_global(p))
                 : "memory");
    return x;
}

// A 16-byte vector holds E elements of T, read and written as floats.  load() is
// of memory that the kernel only reads, load_plain() of elements that this
// thread alone writes, load_before() of what others write after a barrier.
template <typename T>
struct Elem;

template <>
struct Elem<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ float load(const float* p) { return __ldg(p); }
    static __device__ __forceinline__ float load_plain(const float* p) { return __ldcg(p); }
    static __device__ __forceinline__ float load_before(const float* p) { return load_ordered(p); }
    static __device__ __forceinline__ float round_to(float x) { return x; }
    static __device__ __forceinline__ void unpack(uint4 w, float (&f)[4]) {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

template <>
struct Elem<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
        return bf16lo(__ldg(reinterpret_cast<const unsigned short*>(p)));
    }
    static __device__ __forceinline__ float load_plain(const __nv_bfloat16* p) {
        return bf16lo(__ldcg(reinterpret_cast<const unsigned short*>(p)));
    }
    static __device__ __forceinline__ float load_before(const __nv_bfloat16* p) {
        return bf16lo(load_ordered(reinterpret_cast<const unsigned short*>(p)));
    }
    static __device__ __forceinline__ __nv_bfloat16 round_to(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ void unpack(uint4 w, float (&f)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = bf16lo(u[k]);
            f[2 * k + 1] = bf16hi(u[k]);
        }
    }
    static __device__ __forceinline__ uint32_t pack2bf(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack2bf(f[0], f[1]), pack2bf(f[2], f[3]), pack2bf(f[4], f[5]), pack2bf(f[6], f[7]));
    }
};

// Two floats in one register pair: one instruction works on both, each rounded
// as alone.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ---------------------------------------------------------------- token ids

// ids[i] of either type; -1 for an absent token, and for one >= V, which is
// recorded in *status.
template <typename I>
__device__ __forceinline__ int64_t load_id(const I* ids, int64_t i, int64_t V, int* status) {
    const int64_t id = static_cast<int64_t>(__ldg(ids + i));
    if (id >= V) {
        if (status) atomicExch(status, GC_ERR_INVALID);
        return -1;
    }
    return id < 0 ? -1 : id;
}

__device__ __forceinline__ int64_t load_id(const void* ids, bool i64, int64_t i, int64_t V, int* status) {
    return i64 ? load_id(static_cast<const long long*>(ids), i, V, status)
               : load_id(static_cast<const int*>(ids), i, V, status);
}

// ---------------------------------------------------------------- arithmetic

// 2^x; results below 2^-126 are zero.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger of the two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// x / tau - lse, with 1 / tau in two terms: the first fma cancels exactly
// where the two are close, and what the rounding of 1 / tau left out is added.
__device__ __forceinline__ float log_prob_from(float x, float lse, float inv_tau, float inv_tau_low) {
    const float d = fmaf(x, inv_tau, -lse);
    return d == neg_inf() ? d : fmaf(x, inv_tau_low, d);
}

// The same of two.
__device__ __forceinline__ uint64_t log_prob_pair(uint64_t x, float lse, float inv_tau, float inv_tau_low) {
    return pair_fma(x, pair(inv_tau_low, inv_tau_low), pair_fma(x, pair(inv_tau, inv_tau), pair(-lse, -lse)));
}

inline void split_inverse(double tau, float* high, float* low) {
    *high = static_cast<float>(1.0 / tau);
    *low = static_cast<float>(1.0 / tau - static_cast<double>(*high));
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- geometry of a row

// A row of V elements of T that starts anywhere: 16-byte vectors are counted
// from the aligned address at or below the row's start, so vector v holds the
// elements v * E - shift .. v * E - shift + E - 1, of which the first and last
// vectors' may lie outside the row.
template <typename T>
__device__ __forceinline__ int row_shift(const T* row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

}  // namespace gc
