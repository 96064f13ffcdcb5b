// Device helpers of the sequence operators.
#pragma once

#include "dev_common.h"

namespace miconv {

// The rows of sequence s: a row of the batch, or a clamped piece of the packed
// row.  row0 is the batch row of the tensors, start the first position in it.
struct SeqSpan { int64_t row0, start, len; };
__device__ __forceinline__ SeqSpan seq_span(const int32_t *offsets, int64_t s, int64_t L)
{
    if (!offsets) return {s, 0, L};
    int64_t a = offsets[s], b = offsets[s + 1];
    a = a < 0 ? 0 : (a > L ? L : a);
    b = b < a ? a : (b > L ? L : b);
    return {0, a, b - a};
}

// exp2, log2 and reciprocal of the hardware (1 ulp).  The compiler's exp2f
// would add a rescaling for subnormal results, which here are factors that
// vanish against the rest of a sum.
__device__ __forceinline__ float hw_exp2(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float hw_log2(float v) { return __builtin_amdgcn_logf(v); }
__device__ __forceinline__ float hw_rcp(float v) { return __builtin_amdgcn_rcpf(v); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 1 / (1 + exp(-v)): exp2 overflows to infinity for v below -88, where the
// reciprocal gives the limit 0.
__device__ __forceinline__ float sigmoid(float v) { return hw_rcp(1.f + hw_exp2(-kLog2e * v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d/dv of v sigmoid(v), from q = sigmoid(v).
__device__ __forceinline__ float silu_slope(float v, float q) { return q * (1.f + v * (1.f - q)); }

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) <= 1.  1 + e drops low
// bits of a small e; what it drops, e - ((1 + e) - 1), is exact and is added
// back (the logarithm's slope is 1 there), so the result keeps full relative
// precision down to the smallest e.
__device__ __forceinline__ float softplus(float v)
{
    const float e = hw_exp2(-kLog2e * __builtin_fabsf(v));
    const float u = 1.f + e;
    const float lost = e - (u - 1.f);
    return fmaxf(v, 0.f) + __builtin_fmaf(kLn2, hw_log2(u), lost);
}

// V consecutive elements from any element-aligned address (one wide load: the
// hardware takes unaligned global accesses).
template <typename T, int V> struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[V]; };
template <typename T, int V> struct Raw { T v[V]; };
template <typename T, int V> __device__ __forceinline__ Raw<T, V> load_raw(const T *p)
{
    Raw<T, V> r;
    __builtin_memcpy(&r, reinterpret_cast<const Pack<T, V> *>(p), sizeof(r));
    return r;
}
template <typename T, int V> __device__ __forceinline__ void load_f32(const T *p, float (&o)[V])
{
    const Raw<T, V> r = load_raw<T, V>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = to_f32(r.v[i]);
}
template <typename T, int V> __device__ __forceinline__ void store_f32(T *p, const float (&v)[V])
{
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = from_f32<T>(v[i]);
    __builtin_memcpy(reinterpret_cast<Pack<T, V> *>(p), &r, sizeof(r));
}

// Element strides of a [rows, channels, positions] tensor.
struct S3 { int64_t n, c, l; };

}  // namespace miconv
