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

// Quotient and remainder; 64-bit division is a long sequence without a unit of
// its own, and nearly all indexes fit 32.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t &rest)
{
    if (((a | b) >> 32) == 0) {
        const uint32_t q = (uint32_t)a / (uint32_t)b;
        rest = (uint32_t)a - q * (uint32_t)b;
        return q;
    }
    const int64_t q = a / b;
    rest = a - q * b;
    return q;
}

// The sequence whose chunks, numbered start / chunk + sequence on, reach
// `slot` -- the last one with start < (slot - seq + 1) chunk -- and its rows; the
// first one where none does.  first: the number of its first chunk.  For a whole
// wave and one slot.  64 sequences are tested at a time and the found one's rows
// taken from the lane that tested it, so up to 64 sequences cost the one load
// that its rows alone would.  All numbers are below 2^31 here, and a wave that
// starts waits for each of these operations.
__device__ __forceinline__ SeqSpan seq_of_slot(const int32_t *offsets, int seqs, int L, uint32_t chunk, int slot, int &seq,
                                               int &first)
{
    const int lane = threadIdx.x & 63;
    const auto row = [&](int v) { return v < 0 ? 0 : (v > L ? L : v); };
    seq = 0;
    for (int n = seqs;;) {
        const int by = (n + 63) >> 6, k = lane * by, s = seq + k;
        int a = 0, b = 0;
        bool in = k < n;
        if (in) a = offsets[s], b = offsets[s + 1];
        in = in && s <= slot && (uint64_t)(uint32_t)(slot - s + 1) * chunk > (uint32_t)row(a);
        const uint64_t all = __ballot(in);
        const int last = all ? __builtin_popcountll(all) - 1 : 0;
        seq += last * by, n -= last * by;
        if (by <= 1 || !all) {
            const int start = row(__builtin_amdgcn_readlane(a, last)), end = row(__builtin_amdgcn_readlane(b, last));
            first = (int)((uint32_t)start / chunk) + seq;
            return {0, start, end > start ? end - start : 0};
        }
        if (n > by) n = by;
    }
}
// Chunks of a sequence of this length; one, to take the state on, of an empty one.
__device__ __forceinline__ int64_t chunks_of(int64_t len, int64_t chunk)
{
    int64_t rest;
    return len > 0 ? divide(len - 1, chunk, rest) + 1 : 1;
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

// V elements as they are in memory, held as 32-bit words (held as elements, a
// 16-bit one would take a register of its own).
template <typename T, int V> struct Raw {
    static constexpr int n = (V * (int)sizeof(T) + 3) / 4;
    uint32_t w[n];
    __device__ __forceinline__ float f(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return i & 1 ? hi_f32(w[i / 2], T()) : lo_f32(w[i / 2], T());
    }
    __device__ __forceinline__ void set(int i, T v)   // on words that are zero there
    {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v);
        else w[i / 2] |= (uint32_t)v.u << (i & 1 ? 16 : 0);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < n; ++i) w[i] = 0;
    }
};
// V consecutive elements from any element-aligned address (one wide load: the
// hardware takes unaligned global accesses).
template <typename T, int V> struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[V]; };
template <typename T, int V> __device__ __forceinline__ Raw<T, V> load_raw(const T *p)
{
    Raw<T, V> r;
    if constexpr (V * sizeof(T) < 4) r.w[0] = p->u;
    else __builtin_memcpy(r.w, reinterpret_cast<const Pack<T, V> *>(p), sizeof(r));
    return r;
}
template <typename T, int V> __device__ __forceinline__ void load_f32(const T *p, float (&o)[V])
{
    const Raw<T, V> r = load_raw<T, V>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = r.f(i);
}
// ONCE: 16 bytes that the kernel does not read again, past the L2's lines in use.
template <typename T, int V, bool ONCE = false> __device__ __forceinline__ void store_f32(T *p, const float (&v)[V])
{
    if constexpr (V == 1) *p = from_f32<T>(v[0]);
    else {
        Raw<T, V> r;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) r.w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
        }
        if constexpr (ONCE && sizeof(r) == 16) {
            typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
            __builtin_nontemporal_store(any4{r.w[0], r.w[1], r.w[2], r.w[3]}, reinterpret_cast<any4 *>(p));
        } else __builtin_memcpy(reinterpret_cast<Pack<T, V> *>(p), r.w, sizeof(r));
    }
}

// A workgroup barrier that waits for this wave's LDS accesses only.
// __syncthreads() would also drain the loads of the next tile, which are meant
// to stay in flight across it.
__device__ __forceinline__ void lds_sync() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Element strides of a [rows, channels, positions] tensor.
struct S3 { int64_t n, c, l; };

}  // namespace miconv
