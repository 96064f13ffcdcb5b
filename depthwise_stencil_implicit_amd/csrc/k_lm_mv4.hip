// Products of a few rows with 4-bit weights and group scales:
//   y[m,n] = bias[n] + sum_k x[m,k] s[n,k/group] (q[n,k] - z[n,k/group]).
//
// Bound by the weights' bytes.  The rows of x are one operand of a 16x16x32
// matrix instruction and 16 outputs' weights the other, so up to 16 rows cost
// what one does, and the vector unit only widens the weights: two nibbles at
// once become the low bits of a 16-bit float whose exponent gives them weight
// 1 (bf16 0x4300 | q = 128 + q, f16 0x6400 | q = 1024 + q), one shift and one
// and-or.  With bf16 rows the excess is taken out in f32 where a group ends,
//   sum (q - z) x = sum (128 + q) x - (128 + z) sum x,
// sum x from a matrix instruction whose weights are ones; products of 16-bit
// rows with such integers are exact in f32.  f16 rows subtract 1032 from each
// pair of weights, exactly.  f32 rows are split into three bf16 terms, which
// hold all 24 bits, against exact weights.
//
// A workgroup owns 16 outputs; its waves take blocks of 128 columns in turn
// (each lane 16 bytes = 32 weights of one output), and join through LDS.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {
namespace {

constexpr int kMvWaves = 8;

struct MvP {
    const void *x, *scales, *zeros, *bias;
    const uint8_t *w;
    void *y;
    int64_t M, N, K, group, groups;
    int64_t xs_m, xs_k, w_n, sc_n, sc_g, z_n, z_g, bs, ys_m, ys_n;
};

template <typename T> struct MvOp { typedef T in; };          // the matrix instruction's type
template <> struct MvOp<float> { typedef bf16_t in; };

// The eight weights of a word, pairs (0,4) (1,5) (2,6) (3,7), for rows of type
// T: plus 128 (bf16 rows: their own rounding is 2^15 times the f32 sum's, so
// the excess costs nothing that shows) or minus 8.
__device__ __forceinline__ uint4 widen(uint32_t w, bf16_t)
{
    constexpr uint32_t m = 0x000f000fu, e = 0x43004300u;
    return uint4{(w & m) | e, ((w >> 4) & m) | e, ((w >> 8) & m) | e, ((w >> 12) & m) | e};
}
__device__ __forceinline__ uint4 widen(uint32_t w, f16_t)
{
    constexpr uint32_t m = 0x000f000fu, e = 0x64006400u;
    const auto f = [](uint32_t v) {
        const f16x2 r = __builtin_bit_cast(f16x2, v) - f16x2{(_Float16)1032.f, (_Float16)1032.f};
        return __builtin_bit_cast(uint32_t, r);
    };
    return uint4{f((w & m) | e), f(((w >> 4) & m) | e), f(((w >> 8) & m) | e), f(((w >> 12) & m) | e)};
}
// As bf16 too, but subtracted: a pair is widened to two f32 by its place in
// the register, and what is left of 128 + q - 136 fits the upper halves.
__device__ __forceinline__ uint4 widen(uint32_t w, float)
{
    const uint4 v = widen(w, bf16_t());
    const auto f = [](uint32_t u) {
        const float lo = __uint_as_float(u << 16) - 136.f, hi = __uint_as_float(u & 0xffff0000u) - 136.f;
        return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    };
    return uint4{f(v.x), f(v.y), f(v.z), f(v.w)};
}
// What a widened weight is over the nibble.
template <typename T> constexpr float excess() { return std::is_same<T, bf16_t>::value ? 128.f : -8.f; }
template <typename I> __device__ __forceinline__ uint4 ones()
{
    const uint32_t v = std::is_same<I, bf16_t>::value ? 0x3f803f80u : 0x3c003c00u;
    return uint4{v, v, v, v};
}

// Eight values of a row in the order of a widened word: (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ uint4 pair_up(const uint4 &u)
{
    return uint4{__builtin_amdgcn_perm(u.z, u.x, 0x05040100u), __builtin_amdgcn_perm(u.z, u.x, 0x07060302u),
                 __builtin_amdgcn_perm(u.w, u.y, 0x05040100u), __builtin_amdgcn_perm(u.w, u.y, 0x07060302u)};
}

// acc += x w, sx += x 1 for one block of 32 columns.
template <typename T>
__device__ __forceinline__ void mv_mma(const Raw<T, 8> &x, const uint4 &w, f32x4 &acc, f32x4 &sx, bool want_sx)
{
    typedef typename MvOp<T>::in I;
    if constexpr (std::is_same<T, float>::value) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x.f(i);
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            uint4 a;
            a.x = pack2<bf16_t>(v[0], v[4]), a.y = pack2<bf16_t>(v[1], v[5]);
            a.z = pack2<bf16_t>(v[2], v[6]), a.w = pack2<bf16_t>(v[3], v[7]);
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] -= lo_f32(u[i], bf16_t()), v[i + 4] -= hi_f32(u[i], bf16_t());
            mma_16x16x32(a, w, acc, bf16_t());
            if (want_sx) mma_16x16x32(a, ones<bf16_t>(), sx, bf16_t());
        }
    } else {
        const uint4 a = pair_up(__builtin_bit_cast(uint4, x));
        mma_16x16x32(a, w, acc, I());
        if (want_sx) mma_16x16x32(a, ones<I>(), sx, I());
    }
}

// The words of a block as loaded (lane group g holds the 32 columns 32 g ..
// of its output) -> word j of lane group g holds columns 32 j + 8 g ..: a 4x4
// transposition over the lane groups.
__device__ __forceinline__ void transpose_words(uint32_t (&w)[4])
{
    const auto s16 = [](uint32_t &a, uint32_t &b) {
        const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
        a = r[0], b = r[1];
    };
    const auto s32 = [](uint32_t &a, uint32_t &b) {
        const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        a = r[0], b = r[1];
    };
    s16(w[0], w[1]), s16(w[2], w[3]);
    s32(w[0], w[2]), s32(w[1], w[3]);
}

// WIDE: every block of 128 columns lies in one group.  DENSE: x's columns are
// contiguous.
template <typename T, bool WIDE, bool DENSE> __global__ __launch_bounds__(64 * kMvWaves) void mv4(const MvP p)
{
    constexpr int kAhead = sizeof(T) == 4 ? 2 : 4;   // blocks of a wave in flight
    __shared__ float s_acc[kMvWaves][16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kb = lane >> 4, col = lane & 15;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16;
    const int64_t n = n0 + col < p.N ? n0 + col : p.N - 1;
    const uint8_t *w = p.w + n * p.w_n;
    const T *x = static_cast<const T *>(p.x) + (m0 + col < p.M ? m0 + col : p.M - 1) * p.xs_m;
    const T *sc = static_cast<const T *>(p.scales) + n * p.sc_n;
    const bool has_z = p.zeros;
    const T *ze = has_z ? static_cast<const T *>(p.zeros) + n * p.z_n : sc;
    const int64_t ze_g = has_z ? p.z_g : p.sc_g;
    const bool want_sx = std::is_same<T, bf16_t>::value || has_z;

    struct Block {
        uint4 w;
        Raw<T, 8> x[4];
        T s[WIDE ? 1 : 4], z[WIDE ? 1 : 4];
    };
    // Lanes past the last row, output or column repeat one that exists: rows
    // and outputs past the end are not stored, columns are cleared in x below.
    const int K = (int)p.K, group = (int)p.group;
    const auto fetch = [&](int b, Block &o) {
        const int k0 = b * 128;
        o.w = *reinterpret_cast<const uint4 *>(w + (WIDE || k0 + 32 * kb < K ? k0 + 32 * kb : 0) / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int k = k0 + (WIDE ? 32 * kb + 8 * j : 32 * j + 8 * kb);
            if (!WIDE && k >= K) k = 0;
            if constexpr (DENSE) o.x[j] = load_raw<T, 8>(x + k);
            else {
                o.x[j].zero();
#pragma unroll
                for (int i = 0; i < 8; ++i) o.x[j].set(i, x[(k + i) * p.xs_k]);
            }
        }
#pragma unroll
        for (int j = 0; j < (WIDE ? 1 : 4); ++j) {
            const int k = k0 + 32 * j;
            const int64_t g = (WIDE || k < K ? k : k0) / group;
            o.s[j] = sc[g * p.sc_g];
            o.z[j] = ze[g * ze_g];
        }
    };
    f32x4 y = {0, 0, 0, 0};
    const auto flush = [&](const f32x4 &acc, const f32x4 &sx, T s, T z) {
        const float sf = to_f32(s);
        if (want_sx) {
            const float off = excess<T>() + (has_z ? to_f32(z) : 8.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(sf, __builtin_fmaf(-off, sx[i], acc[i]), y[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(sf, acc[i], y[i]);
        }
    };
    const int blocks = (int)((p.K + 127) / 128);
    Block ring[kAhead];
#pragma unroll
    for (int r = 0; r < kAhead; ++r)
        if (wave + r * kMvWaves < blocks) fetch(wave + r * kMvWaves, ring[r]);
    for (int b0 = wave; b0 < blocks; b0 += kMvWaves * kAhead) {
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            const int b = b0 + r * kMvWaves;
            if (b >= blocks) break;
            Block cur = ring[r];
            if (b + kMvWaves * kAhead < blocks) fetch(b + kMvWaves * kAhead, ring[r]);
            if (!WIDE && b == blocks - 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (b * 128 + 32 * j + 8 * kb >= K) cur.x[j].zero();
            }
            uint32_t word[4] = {cur.w.x, cur.w.y, cur.w.z, cur.w.w};
            f32x4 acc = {0, 0, 0, 0}, sx = {0, 0, 0, 0};
            if (!WIDE) transpose_words(word);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mv_mma<T>(cur.x[j], widen(word[j], T()), acc, sx, want_sx);
                if (!WIDE) {
                    flush(acc, sx, cur.s[j], cur.z[j]);
                    acc = f32x4{0, 0, 0, 0}, sx = f32x4{0, 0, 0, 0};
                }
            }
            if (WIDE) flush(acc, sx, cur.s[0], cur.z[0]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_acc[wave][kb * 4 + i][col] = y[i];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
        if (m0 + m < p.M && n0 + c < p.N) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kMvWaves; ++i) v += s_acc[i][m][c];
            if (p.bias) v += to_f32(static_cast<const T *>(p.bias)[(n0 + c) * p.bs]);
            static_cast<T *>(p.y)[(m0 + m) * p.ys_m + (n0 + c) * p.ys_n] = from_f32<T>(v);
        }
    }
}

}  // namespace

int launch_lm_mv4(const lm_plan_t &p, lm_ptrs q, hipStream_t s)
{
    MvP a = {};
    a.x = q[LM_X], a.scales = q[LM_SCALES], a.zeros = q[LM_ZEROS], a.bias = q[LM_BIAS];
    a.w = static_cast<const uint8_t *>(q[LM_W]);
    a.y = q[LM_Y];
    a.M = p.seqs, a.N = p.C, a.K = p.K, a.groups = p.G, a.group = p.K / p.G;
    a.xs_m = p.t[LM_X].strides[0], a.xs_k = p.t[LM_X].strides[1], a.w_n = p.t[LM_W].strides[0];
    a.sc_n = p.t[LM_SCALES].strides[0], a.sc_g = p.t[LM_SCALES].strides[1];
    a.z_n = p.t[LM_ZEROS].strides[0], a.z_g = p.t[LM_ZEROS].strides[1];
    a.bs = p.t[LM_BIAS].strides[0], a.ys_m = p.t[LM_Y].strides[0], a.ys_n = p.t[LM_Y].strides[1];
    const dim3 grid((unsigned)lm_cdiv(a.N, 16), (unsigned)lm_cdiv(a.M, 16));
    const bool wide = a.group % 128 == 0;
    const auto go = [&](auto t) {
        typedef decltype(t) T;
        if (a.xs_k == 1 || a.K == 1) {
            if (wide) mv4<T, true, true><<<grid, 64 * kMvWaves, 0, s>>>(a);
            else mv4<T, false, true><<<grid, 64 * kMvWaves, 0, s>>>(a);
        } else {
            if (wide) mv4<T, true, false><<<grid, 64 * kMvWaves, 0, s>>>(a);
            else mv4<T, false, false><<<grid, 64 * kMvWaves, 0, s>>>(a);
        }
    };
    if (p.dtype == CONV_F32) go(float());
    else if (p.dtype == CONV_F16) go(f16_t());
    else go(bf16_t());
    return lm_launch_status();
}

}  // namespace miconv
