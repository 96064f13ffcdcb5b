// The RMS norm with the residual's addition, an output in the input's type or
// in 8 bits with scales, and its gradients:
//   v = x + residual,  rstd = 1 / sqrt(mean v^2 + value),  y = v rstd w
//   dx = gstate + rstd (w gy - u mean(w gy u)),  dw = sum_rows gy u,  u = v rstd.
//
// Bound by memory: a few operations per element.  Every row is read once and
// stays in registers between its sums and its results: 64, 256 or 1024 threads
// share a row (norm_threads), each with up to 8 pieces of 8 channels, 16 bytes
// of a 16-bit type.  y comes from the unrounded sum v, one rounding from the
// result.  The gradients start from x and residual, whose sum they form again, or
// from v as it was stored, which is one tensor less to read and rounds each term
// of dw once more (16384 x 4096 bf16: dw is off by 0.0024 of its norm for 0.0017,
// which its own rounding makes, and the call takes 107 us for 134).
//
// Measured (bf16, medians of traced kernels): 8192 x 5120 with residual, scales of
// 128 channels and 8-bit output 64 us, 4.6 TB/s of the 5.1 that a copy reaches;
// 16384 x 4096 with residual in 16 bits 86 us (6.2 TB/s), its gradients 143 us from
// x and residual, 115 from the stored sum (4.7 TB/s), and 5.7 for dw's sum; 32 rows
// of 4096 5.2 us, the time of a launch, two waits for memory and two joins.
// Gradients of more than 8192 channels lack registers: 256 threads of 8 pieces hold
// 410, one wave a SIMD (4096 x 12288 181 us, 1.7 TB/s), 1024 threads of 4 and 8
// pieces spill 88 and 319 (2048 x 32768 271 us, 1.5 TB/s).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {
namespace {

constexpr int kPiece = 8;
constexpr float kF8Max = 448.f;
constexpr float kF8Least = 0x1p-112f;   // of a group's largest value: 448 divided by it stays finite

struct NormP {
    const void *x, *w, *res, *gy, *gs;
    void *y, *sum, *dx;
    float *scales, *rstd, *part;
    S3 xs, ress, ys, sums, scs, gys, gss, dxs;
    int64_t w_c, rstd_n, rstd_l;
    int64_t rows, C, L;
    int pieces;    // of 8 channels, the last one may be cut
    int group;     // lanes that share a scale; 0: the whole row
    float eps, inv_c;
};

// A thread's piece of a row.  DENSE (channels contiguous, 8 or more): the last
// piece is moved back inside C and repeats `dup` of its neighbour's channels,
// which sums leave out and stores write twice, alike; loads never stand behind
// a branch, where they would be waited for one by one.
template <bool DENSE> struct Piece {
    int64_t c;
    int n, dup;   // channels of its own; repeated ones in front of them
    __device__ __forceinline__ Piece(const NormP &p, int at)
    {
        c = (int64_t)at * kPiece;
        n = c + kPiece <= p.C ? kPiece : (int)(c < p.C ? p.C - c : 0);
        dup = 0;
        if (DENSE) {
            dup = kPiece - n;
            if (c > p.C - kPiece) c = p.C - kPiece;
        }
    }
    __device__ __forceinline__ bool mine(int j) const { return DENSE ? j >= dup : j < n; }
    template <typename T> __device__ __forceinline__ void get(const T *row, int64_t cs, float (&o)[kPiece]) const
    {
        if constexpr (DENSE) load_f32<T, kPiece>(row + c, o);
        else {
#pragma unroll
            for (int j = 0; j < kPiece; ++j) o[j] = j < n ? to_f32(row[(c + j) * cs]) : 0.f;
        }
    }
    template <typename T> __device__ __forceinline__ void put(T *row, int64_t cs, const float (&v)[kPiece]) const
    {
        if (n == 0) return;
        if constexpr (DENSE) store_f32<T, kPiece>(row + c, v);
        else {
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                if (j < n) row[(c + j) * cs] = from_f32<T>(v[j]);
        }
    }
};
// Eight values in e4m3, rounded to nearest even.
__device__ __forceinline__ uint2 to_f8(const float (&v)[kPiece])
{
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    return uint2{(uint32_t)lo, (uint32_t)hi};
}
// What a group is scaled by: a NaN stays one.
__device__ __forceinline__ float span_of(float top) { return top == 0.f ? kF8Max : top < kF8Least ? kF8Least : top; }
// The larger one, or a NaN.
__device__ __forceinline__ float top_of(float a, float b) { return a > b || a != a ? a : b; }

template <int W, typename F> __device__ __forceinline__ float over_lanes(float v, F f)
{
#pragma unroll
    for (int d = 1; d < W; d *= 2) v = f(v, __shfl_xor(v, d));
    return v;
}
// Over the TPR threads of a row; sh: a place of its own for each call in flight.
template <int TPR, typename F> __device__ __forceinline__ float over_row(float v, float *sh, F f)
{
    v = over_lanes<64>(v, f);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) sh[wave] = v;
        lds_sync();
        v = sh[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) v = f(v, sh[w]);
    }
    return v;
}

// P: pieces of a thread.  A row's loads are all on their way before the first is
// used, and nothing else is kept of it; more threads a row for few rows, fewer for
// many, where the joins cost (norm_threads).
template <typename T, bool F8, int TPR, int P, bool DENSE>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void norm_fwd(const NormP p)
{
    __shared__ float sh[2][16];
    constexpr int PER = TPR == 64 ? 4 : 1;   // rows of a workgroup
    const int tid = threadIdx.x & (TPR - 1);
    const int64_t row = (int64_t)blockIdx.x * PER + (PER > 1 ? threadIdx.x >> 6 : 0);
    if (row >= p.rows) return;
    int64_t l;
    const int64_t n = divide(row, p.L, l);
    const auto at = [&](const void *t, const S3 &s) { return static_cast<const T *>(t) + n * s.n + l * s.l; };
    const bool has = p.res != nullptr;
    const T *x = at(p.x, p.xs), *res = has ? at(p.res, p.ress) : x;
    const int64_t res_c = has ? p.ress.c : p.xs.c;
    float v[P][kPiece], ss = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const Piece<DENSE> q(p, i * TPR + tid);
        float r[kPiece];
        q.get(x, p.xs.c, v[i]), q.get(res, res_c, r);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[i][j] += has ? r[j] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const Piece<DENSE> q(p, i * TPR + tid);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
            const float t = q.mine(j) ? v[i][j] : 0.f;
            ss = __builtin_fmaf(t, t, ss);
        }
    }
    ss = over_row<TPR>(ss, sh[0], [](float a, float b) { return a + b; });
    const float rstd = 1.f / __builtin_sqrtf(__builtin_fmaf(ss, p.inv_c, p.eps));
    if (p.rstd && tid == 0) p.rstd[n * p.rstd_n + l * p.rstd_l] = rstd;

    T *sum = const_cast<T *>(at(p.sum, p.sums)), *y = const_cast<T *>(at(p.y, p.ys));
    uint8_t *y8 = static_cast<uint8_t *>(p.y) + n * p.ys.n + l * p.ys.l;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const Piece<DENSE> q(p, i * TPR + tid);
        if (has) q.put(sum, p.sums.c, v[i]);
        float w[kPiece];
        q.get(static_cast<const T *>(p.w), p.w_c, w);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[i][j] = v[i][j] * rstd * w[j];
        if constexpr (!F8) q.put(y, p.ys.c, v[i]);
        else {
#pragma unroll
            for (int j = 0; j < kPiece; ++j) top = top_of(top, q.mine(j) ? __builtin_fabsf(v[i][j]) : 0.f);
        }
    }
    if constexpr (F8) {
        float *scales = p.scales + n * p.scs.n + l * p.scs.l;
        if (p.group == 0) {
            top = over_row<TPR>(top, sh[1], top_of);
            top = span_of(top);
            if (tid == 0) *scales = top / kF8Max;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const Piece<DENSE> q(p, i * TPR + tid);
            float t = top;
            if (p.group) {   // whole pieces, and lanes past the end are a group's all or none
                t = 0.f;
#pragma unroll
                for (int j = 0; j < kPiece; ++j) t = top_of(t, __builtin_fabsf(v[i][j]));
                for (int d = 1; d < p.group; d *= 2) t = top_of(t, __shfl_xor(t, d));
                t = span_of(t);
                if (q.n && (tid & (p.group - 1)) == 0) scales[(i * TPR + tid) / p.group * p.scs.c] = t / kF8Max;
            }
            const float f = kF8Max / t;
            float o[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j) o[j] = v[i][j] * f;
            const uint2 b = to_f8(o);
            if (q.n == 0) continue;
            if constexpr (DENSE) {
                struct __attribute__((packed, aligned(1))) Eight { uint32_t lo, hi; };
                Eight e{b.x, b.y};
                *reinterpret_cast<Eight *>(y8 + q.c) = e;
            } else {
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    if (j < q.n) y8[(q.c + j) * p.ys.c] = (uint8_t)((j < 4 ? b.x : b.y) >> (j % 4 * 8));
            }
        }
    }
}

// A workgroup goes through rows and keeps its threads' part of dw in registers:
// 1024 workgroups at most, whose parts of dw are 17 MB for 4096 channels, 3% of what
// 16384 rows move.
template <typename T, int TPR, int P, bool DENSE, bool RES> __global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void norm_bwd(const NormP p)
{
    __shared__ float sh[2][16];
    __shared__ float join[TPR == 64 ? 3 * 64 * P * kPiece : 1];
    constexpr int PER = TPR == 64 ? 4 : 1;
    const int tid = threadIdx.x & (TPR - 1), sub = PER > 1 ? threadIdx.x >> 6 : 0;
    float w[P][kPiece], dw[P][kPiece];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        Piece<DENSE>(p, i * TPR + tid).get(static_cast<const T *>(p.w), p.w_c, w[i]);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) dw[i][j] = 0.f;
    }
    int buf = 0;
    for (int64_t row = (int64_t)blockIdx.x * PER + sub; row < p.rows; row += (int64_t)gridDim.x * PER, buf ^= 1) {
        int64_t l;
        const int64_t n = divide(row, p.L, l);
        const auto at = [&](const void *t, const S3 &s) { return static_cast<const T *>(t) + n * s.n + l * s.l; };
        const T *x = at(p.x, p.xs), *gy = at(p.gy, p.gys);
        const float rstd = p.rstd[n * p.rstd_n + l * p.rstd_l];
        float u[P][kPiece], g[P][kPiece], dot = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const Piece<DENSE> q(p, i * TPR + tid);
            q.get(x, p.xs.c, u[i]), q.get(gy, p.gys.c, g[i]);
            if constexpr (RES) {
                float r[kPiece];
                q.get(at(p.res, p.ress), p.ress.c, r);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) u[i][j] += r[j];
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const Piece<DENSE> q(p, i * TPR + tid);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                u[i][j] *= rstd;
                dw[i][j] = __builtin_fmaf(g[i][j], u[i][j], dw[i][j]);
                g[i][j] *= w[i][j];
                dot = __builtin_fmaf(q.mine(j) ? g[i][j] : 0.f, u[i][j], dot);
            }
        }
        if (!p.dx) continue;
        dot = over_row<TPR>(dot, sh[buf], [](float a, float b) { return a + b; }) * p.inv_c;
        const bool has = p.gs != nullptr;
        const T *gs = has ? at(p.gs, p.gss) : gy;
        const int64_t gs_c = has ? p.gss.c : p.gys.c;
        T *dx = const_cast<T *>(at(p.dx, p.dxs));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const Piece<DENSE> q(p, i * TPR + tid);
            float o[kPiece];
            q.get(gs, gs_c, o);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) o[j] = __builtin_fmaf(rstd, __builtin_fmaf(-u[i][j], dot, g[i][j]), has ? o[j] : 0.f);
            q.put(dx, p.dxs.c, o);
        }
    }
    if (!p.part) return;
    if constexpr (PER > 1) {   // the four waves' sums
        if (sub) {
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) join[((sub - 1) * P * kPiece + i * kPiece + j) * 64 + tid] = dw[i][j];
        }
        __syncthreads();
        if (sub) return;
        for (int s = 0; s < PER - 1; ++s)
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) dw[i][j] += join[(s * P * kPiece + i * kPiece + j) * 64 + tid];
    }
    float *part = p.part + (int64_t)blockIdx.x * p.C;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        Piece<DENSE>(p, i * TPR + tid).put(part, 1, dw[i]);
    }
}

// dw from the workgroups' parts, in a fixed order.
template <typename T> __global__ __launch_bounds__(1024) void norm_dw(const float *part, int64_t parts, int64_t C, T *dw, int64_t dw_c)
{
    __shared__ float sums[16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.f;
    if (c < C)
#pragma unroll 16
        for (int64_t i = wave; i < parts; i += 16) v += part[i * C + c];
    sums[wave][lane] = v;
    __syncthreads();
    if (wave || c >= C) return;
    for (int w = 1; w < 16; ++w) v += sums[w][lane];
    dw[c * dw_c] = from_f32<T>(v);
}

S3 s3(const conv_tensor &t) { return {t.strides[0], t.strides[1], t.rank > 2 ? t.strides[2] : 0}; }

NormP base(const lm_plan_t &p, lm_ptrs q)
{
    NormP a = {};
    a.x = q[LM_X], a.w = q[LM_W], a.res = q[LM_STATE_IN], a.gy = q[LM_GY], a.gs = q[LM_GSTATE];
    a.y = q[LM_Y], a.sum = q[LM_STATE_OUT], a.dx = q[LM_DX];
    a.scales = static_cast<float *>(q[LM_SCALES]), a.rstd = static_cast<float *>(q[LM_SAVED]);
    a.xs = s3(p.t[LM_X]), a.ress = s3(p.t[LM_STATE_IN]), a.ys = s3(p.t[LM_Y]), a.sums = s3(p.t[LM_STATE_OUT]);
    a.scs = s3(p.t[LM_SCALES]), a.gys = s3(p.t[LM_GY]), a.gss = s3(p.t[LM_GSTATE]), a.dxs = s3(p.t[LM_DX]);
    a.w_c = p.t[LM_W].strides[0];
    a.rstd_n = p.t[LM_SAVED].strides[0], a.rstd_l = p.t[LM_SAVED].rank > 1 ? p.t[LM_SAVED].strides[1] : 0;
    a.rows = p.seqs * p.L, a.C = p.C, a.L = p.L;
    a.pieces = (int)lm_cdiv(p.C, kPiece);
    a.group = p.G > 1 ? (int)(p.C / p.G / kPiece) : 0;
    a.eps = p.args.value, a.inv_c = 1.f / (float)p.C;
    return a;
}

// f(threads of a row, pieces of a thread, whether channels are contiguous): the
// pieces that norm_threads leaves, in powers of two, or the most of them for
// channels apart, whose gradients then spill 320 to 1100 registers at 256 and 1024
// threads (4 x 2048 x 4096 in the order [N, C, L]: 1.2 to 1.4 ms).
template <typename F> void with_shape(const lm_plan_t &p, const NormP &a, F f)
{
    bool dense = a.w_c == 1 && p.C >= kPiece;
    for (int s : {LM_X, LM_STATE_IN, LM_STATE_OUT, LM_Y, LM_GY, LM_GSTATE, LM_DX})
        if (p.t[s].rank && p.t[s].strides[1] != 1) dense = false;
    const int threads = norm_threads(a.rows, p.C), each = (int)lm_cdiv(a.pieces, threads);
    const auto go = [&](auto t, auto n) { f(t, n, std::true_type()); };
    const std::integral_constant<int, 64> wave;
    const std::integral_constant<int, 256> four;
    const std::integral_constant<int, 1024> all;
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> quad;
    const std::integral_constant<int, 8> eight;
    if (!dense) {
        if (threads == 64) f(wave, quad, std::false_type());
        else if (threads == 256) f(four, eight, std::false_type());
        else f(all, eight, std::false_type());
    } else if (threads == 64) {
        if (each <= 1) go(wave, one);
        else if (each <= 2) go(wave, two);
        else go(wave, quad);
    } else if (threads == 256) {
        if (each <= 2) go(four, two);
        else if (each <= 4) go(four, quad);
        else go(four, eight);
    } else {
        if (each <= 1) go(all, one);
        else if (each <= 2) go(all, two);
        else if (each <= 4) go(all, quad);
        else go(all, eight);
    }
}

}  // namespace

int launch_lm_norm(const lm_plan_t &p, lm_ptrs q, hipStream_t s)
{
    const NormP a = base(p, q);
    if (!a.rows) return CONV_OK;
    const bool f8 = p.t[LM_Y].dtype == LM_F8;
    const auto go = [&](auto t) {
        typedef decltype(t) T;
        with_shape(p, a, [&](auto threads, auto pieces, auto dense) {
            constexpr int TPR = decltype(threads)::value, P = decltype(pieces)::value;
            constexpr bool D = decltype(dense)::value;
            const unsigned groups = (unsigned)lm_cdiv(a.rows, TPR == 64 ? 4 : 1), size = TPR == 64 ? 256 : TPR;
            if (f8) norm_fwd<T, true, TPR, P, D><<<groups, size, 0, s>>>(a);
            else norm_fwd<T, false, TPR, P, D><<<groups, size, 0, s>>>(a);
        });
    };
    if (p.dtype == CONV_F32) go(float());
    else if (p.dtype == CONV_F16) go(f16_t());
    else go(bf16_t());
    return lm_launch_status();
}

int launch_lm_norm_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    NormP a = base(p, q);
    a.part = q[LM_DW] ? static_cast<float *>(ws) : nullptr;
    const int64_t groups = norm_bwd_groups(p);
    const auto go = [&](auto t) {
        typedef decltype(t) T;
        with_shape(p, a, [&](auto threads, auto pieces, auto dense) {
            constexpr int TPR = decltype(threads)::value, P = decltype(pieces)::value;
            constexpr bool D = decltype(dense)::value;
            const unsigned size = TPR == 64 ? 256 : TPR;
            if (a.res) norm_bwd<T, TPR, P, D, true><<<(unsigned)groups, size, 0, s>>>(a);
            else norm_bwd<T, TPR, P, D, false><<<(unsigned)groups, size, 0, s>>>(a);
        });
        if (q[LM_DW])
            norm_dw<T><<<(unsigned)lm_cdiv(p.C, 64), 1024, 0, s>>>(a.part, groups, p.C, static_cast<T *>(q[LM_DW]), p.t[LM_DW].strides[0]);
    };
    if (p.dtype == CONV_F32) go(float());
    else if (p.dtype == CONV_F16) go(f16_t());
    else go(bf16_t());
    return lm_launch_status();
}

}  // namespace miconv
