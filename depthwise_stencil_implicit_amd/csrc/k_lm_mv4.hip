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
// What that costs in bits: the bf16 sums are about 30 times what is wanted of
// them, so where they are taken apart 5 of f32's 24 bits are gone, 11 more than
// the result's own rounding keeps.  It shows only where the terms of a row
// cancel to 2^-11 of their size.  An infinity in a row of x makes its products
// NaN (infinity less infinity), where a sum of products could be infinite.
//
// A workgroup works on tiles of 16 outputs; its waves take blocks of 128
// columns in turn (each lane 16 bytes = 32 weights of one output) and join
// through LDS.  mv4_tiles keeps the rows of x in registers over many tiles, so
// its loop only streams weights; mv4_stream, for other groups, rows under 128
// columns and over 130944, loads x with each block.
//
// Measured: 4 rows, 8192 x 65536 bf16 in 68 us (4.1 TB/s; mv4_stream 177), one
// row, 4096 x 8192 in 8.2 us, of which a launch is 1.8 and the weights' bytes
// 3.4; 11 rows, 5120 x 2501 f16 with zeros in 12 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {
namespace {

constexpr int kMvWaves = 8;      // of mv4_stream
constexpr int kTileWaves = 16;   // of mv4_tiles, at most

struct MvP {
    const void *x, *scales, *zeros, *bias;
    const uint8_t *w;
    void *y;
    int64_t M, N, K, group;
    uint32_t block_group;   // 2^20 group 128ths of a block, rounded up: block -> group
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

// Eight values of a row as matrix operands: themselves, or three bf16 terms of
// f32 ones.
template <typename T> struct XOp {
    static constexpr int n = sizeof(T) == 4 ? 3 : 1;
    uint4 v[n];
    __device__ __forceinline__ void set(const Raw<T, 8> &x)
    {
        if constexpr (n == 3) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = x.f(i);
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                const uint32_t u[4] = {pack2<bf16_t>(f[0], f[4]), pack2<bf16_t>(f[1], f[5]), pack2<bf16_t>(f[2], f[6]),
                                       pack2<bf16_t>(f[3], f[7])};
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] -= lo_f32(u[i], bf16_t()), f[i + 4] -= hi_f32(u[i], bf16_t());
                v[part] = uint4{u[0], u[1], u[2], u[3]};
            }
        } else v[0] = pair_up(__builtin_bit_cast(uint4, x));
    }
    // acc += x w
    __device__ __forceinline__ void times(const uint4 &w, f32x4 &acc) const
    {
#pragma unroll
        for (int part = 0; part < n; ++part) mma_16x16x32(v[part], w, acc, typename MvOp<T>::in());
    }
};

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

// Any group that is a multiple of 32 columns and any row length.  WIDE: every
// block of 128 columns lies in one group.
template <typename T, bool WIDE> __global__ __launch_bounds__(64 * kMvWaves) void mv4_stream(const MvP p)
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
            o.x[j] = load_raw<T, 8>(x + k);
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
                XOp<T> x8;
                x8.set(cur.x[j]);
                x8.times(widen(word[j], T()), acc);
                if (want_sx) x8.times(ones<typename MvOp<T>::in>(), sx);
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

// V elements (2 or 4) moved down by `by` < V places.
template <int V, typename R> __device__ __forceinline__ void move_down(R &r, int by)
{
    if constexpr (R::n == V) {   // words
#pragma unroll
        for (int s = 1; s < V; s *= 2)
#pragma unroll
            for (int i = 0; i + s < V; ++i) r.w[i] ^= (r.w[i] ^ r.w[i + s]) & (by & s ? ~0u : 0u);
    } else if constexpr (V == 2) r.w[0] >>= 16 * by;
    else {
        const uint64_t v = ((uint64_t)r.w[1] << 32 | r.w[0]) >> (16 * by);
        r.w[0] = (uint32_t)v, r.w[1] = (uint32_t)(v >> 32);
    }
}

// GR columns per group (128: one group holds a block or more), NB blocks of
// every wave with their x in registers.  With GR < 128 the last block may be
// cut short at a multiple of 32 columns: its missing weights and scales are
// read from columns that exist, against zeros in x.  Not with NB = 4, whose
// registers are full: mv4_parts gives a cut row's parts at most 32 blocks.
// (4 rows, 8160 x 32768 in groups of 32: 50 us for bf16, 116 with mv4_stream;
// 4160 x 16384 f32 25 and 50; one row, 8160 x 4000 f32 24 and 23.)
// Each block's weights of the next tile are requested as soon as the present
// ones are used, so NB KiB per wave stay in flight across the barrier of a tile.
template <typename T, int GR, int NB, bool Z>
__global__ __launch_bounds__(64 * kTileWaves) void mv4_tiles(const MvP p, int tiles, float *partial)
{
    constexpr int NG = 128 / GR;
    constexpr bool cut = GR < 128 && NB < 4;
    extern __shared__ __attribute__((aligned(16))) float sh[];   // sums of x [block][group][16], then [2][wave][16][17]
    const int waves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kb = lane >> 4,
              col = lane & 15;
    // Blocks of this part of the columns: first .. first + blocks - 1.
    const int K = (int)p.K, all = (K + 127) / 128, groups = K / GR,
              first = (int)(blockIdx.z * (int64_t)all / gridDim.z),
              blocks = (int)((blockIdx.z + 1) * (int64_t)all / gridDim.z) - first;
    const int m0 = blockIdx.y * 16, rows = p.M - m0 < 16 ? (int)p.M - m0 : 16;
    constexpr bool want_sx = std::is_same<T, bf16_t>::value || Z;
    const T *x = static_cast<const T *>(p.x) + (m0 + (col < rows ? col : rows - 1)) * p.xs_m;
    const T *sc = static_cast<const T *>(p.scales), *ze = static_cast<const T *>(p.zeros);
    float *s_sx = sh + wave * NB * NG * 16;
    float *s_acc = sh + waves * NB * NG * 16;

    struct Block {
        uint4 w;
        Raw<T, NG> s;
        Raw<T, Z ? NG : 1> z;
    } ring[NB];
    // Offsets from uniform bases fit 32 bits (mv4_parts sees to it).
    const auto fetch = [&](int tile, int r) {
        const int b = first + (wave + r * waves < blocks ? wave + r * waves : 0);
        const uint32_t n = tile * 16 + col < (int)p.N ? tile * 16 + col : (int)p.N - 1;
        const uint32_t in_block = !cut || b * 128 + 32 * kb < K ? kb * 16 : 0;
        ring[r].w = *reinterpret_cast<const uint4 *>(p.w + b * 64 + (n * (uint32_t)p.w_n + in_block));
        const int g = GR == 128 ? (int)((uint32_t)b * p.block_group >> 20) : !cut || b * NG < groups - NG ? b * NG : groups - NG;
        ring[r].s = load_raw<T, NG>(sc + g + n * (uint32_t)p.sc_n);
        if constexpr (Z) ring[r].z = load_raw<T, NG>(ze + g + n * (uint32_t)p.z_n);
    };
#pragma unroll
    for (int r = 0; r < NB; ++r) fetch(blockIdx.x, r);

    // All loads of x before the first use of one.
    Raw<T, 8> raw[NB][4];
    const auto x_at = [&](int r, int j) {
        const int b = wave + r * waves;
        const int k = (first + (b < blocks ? b : 0)) * 128;
        return GR == 128 ? k + 32 * kb + 8 * j : (!cut || k + 32 * j < K ? k + 32 * j : 0) + 8 * kb;
    };
#pragma unroll
    for (int r = 0; r < NB; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[r][j].zero();
    if (col < rows) {   // lanes of rows past the end load nothing
#pragma unroll
        for (int r = 0; r < NB; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[r][j] = load_raw<T, 8>(x + x_at(r, j));
    }
    XOp<T> xa[NB][4];
#pragma unroll
    for (int r = 0; r < NB; ++r) {
        f32x4 sx = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (wave + r * waves >= blocks || (cut && (first + wave + r * waves) * 128 + 32 * j >= K)) raw[r][j].zero();
            xa[r][j].set(raw[r][j]);
            xa[r][j].times(ones<typename MvOp<T>::in>(), sx);
            if ((j + 1) * 32 % GR == 0) {   // the same in every column: the first lane of each four rows keeps it
                if (col == 0) *reinterpret_cast<f32x4 *>(s_sx + (r * NG + (j + 1) * 32 / GR - 1) * 16 + kb * 4) = sx;
                sx = f32x4{0, 0, 0, 0};
            }
        }
    }
    int buf = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
        f32x4 y = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < NB; ++r) {
            uint32_t word[4] = {ring[r].w.x, ring[r].w.y, ring[r].w.z, ring[r].w.w};
            Raw<T, NG> s = ring[r].s;
            auto z = ring[r].z;
            if constexpr (cut) {   // the cut block's scales were read with those before them
                const int over = (first + wave + r * waves + 1) * NG - groups, by = over > 0 && over < NG ? over : 0;
                move_down<NG>(s, by);
                if constexpr (Z) move_down<NG>(z, by);
            }
            fetch(tile + (int)gridDim.x < tiles ? tile + (int)gridDim.x : tile, r);
            if (GR < 128) transpose_words(word);
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                xa[r][j].times(widen(word[j], T()), acc);
                if ((j + 1) * 32 % GR) continue;
                const int g = (j + 1) * 32 / GR - 1;
                if constexpr (want_sx) {
                    const f32x4 sx = *reinterpret_cast<const f32x4 *>(s_sx + (r * NG + g) * 16 + kb * 4);
                    const float off = excess<T>() + (Z ? z.f(g) : 8.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(-off, sx[i], acc[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(s.f(g), acc[i], y[i]), acc[i] = 0.f;
            }
            // Blocks mixed by the scheduler would not fit the registers.
            __builtin_amdgcn_sched_barrier(0);
        }
        float *mine = s_acc + (buf * waves + wave) * (16 * 17);
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(kb * 4 + i) * 17 + col] = y[i];   // all rows: a condition would move the sums behind it
        lds_sync();
        const int m = threadIdx.x >> 4;
        const int64_t n = (int64_t)tile * 16 + col;
        if (m < rows && n < p.N) {
            const float *all = s_acc + buf * waves * (16 * 17) + m * 17 + col;
            float v[kTileWaves];
#pragma unroll
            for (int i = 0; i < kTileWaves; ++i) v[i] = i < waves ? all[i * 16 * 17] : 0.f;
#pragma unroll
            for (int w = 1; w < kTileWaves; w *= 2)
#pragma unroll
                for (int i = 0; i < kTileWaves; i += 2 * w) v[i] += v[i + w];
            if (partial) partial[(blockIdx.z * p.M + m0 + m) * p.N + n] = v[0];
            else {
                if (p.bias) v[0] += to_f32(static_cast<const T *>(p.bias)[n * p.bs]);
                static_cast<T *>(p.y)[(m0 + m) * p.ys_m + n * p.ys_n] = from_f32<T>(v[0]);
            }
        }
    }
}

// Sums of the parts of the columns.
template <typename T> __global__ __launch_bounds__(256) void mv4_sums(const MvP p, const float *partial, int parts)
{
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N) return;
    const float bias = p.bias ? to_f32(static_cast<const T *>(p.bias)[n * p.bs]) : 0.f;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        float v = 0.f;
        for (int i = 0; i < parts; ++i) v += partial[(i * p.M + m) * p.N + n];
        static_cast<T *>(p.y)[m * p.ys_m + n * p.ys_n] = from_f32<T>(v + bias);
    }
}

// x with its columns apart -> contiguous rows in the workspace.
template <typename T> __global__ __launch_bounds__(256) void mv4_rows(const MvP p, T *out)
{
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= p.K) return;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) out[m * p.K + k] = static_cast<const T *>(p.x)[m * p.xs_m + k * p.xs_k];
}

template <typename T, int GR> void run_tiles(const MvP &a, int parts, float *partial, hipStream_t s)
{
    // The fewest blocks per wave: a short call's time is its longest wave's.
    const int blocks = (int)lm_cdiv(lm_cdiv(a.K, 128), parts), nb = blocks <= 16 ? 1 : blocks <= 32 ? 2 : 4;
    const int waves = (int)lm_cdiv(blocks, nb), tiles = (int)lm_cdiv(a.N, 16);
    // At least four waves finish a tile of 16 rows.
    const int threads = 64 * (waves < 4 ? 4 : waves);
    // As many workgroups as are resident at once on 256 compute units.
    const int resident = 256 * (1024 / threads);
    const dim3 grid((unsigned)(tiles < resident ? tiles : resident), (unsigned)lm_cdiv(a.M, 16), (unsigned)parts);
    const size_t lds = (size_t)(threads / 64) * (nb * (128 / GR) * 16 + 2 * 16 * 17) * sizeof(float);
    const auto go = [&](auto n) {
        constexpr int NB = decltype(n)::value;
        if (a.zeros) mv4_tiles<T, GR, NB, true><<<grid, threads, lds, s>>>(a, tiles, partial);
        else mv4_tiles<T, GR, NB, false><<<grid, threads, lds, s>>>(a, tiles, partial);
    };
    if (nb == 1) go(std::integral_constant<int, 1>());
    else if constexpr (sizeof(T) == 2) {
        if (nb == 2) go(std::integral_constant<int, 2>());
        else go(std::integral_constant<int, 4>());
    }
    if (partial)
        mv4_sums<T><<<dim3((unsigned)lm_cdiv(a.N, 256), (unsigned)(a.M < 65535 ? a.M : 65535)), 256, 0, s>>>(a, partial,
                                                                                                          parts);
}

}  // namespace

int launch_lm_mv4(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    MvP a = {};
    a.x = q[LM_X], a.scales = q[LM_SCALES], a.zeros = q[LM_ZEROS], a.bias = q[LM_BIAS];
    a.w = static_cast<const uint8_t *>(q[LM_W]);
    a.y = q[LM_Y];
    a.M = p.seqs, a.N = p.C, a.K = p.K, a.group = p.K / p.G;
    a.xs_m = p.t[LM_X].strides[0], a.xs_k = p.t[LM_X].strides[1], a.w_n = p.t[LM_W].strides[0];
    a.sc_n = p.t[LM_SCALES].strides[0], a.sc_g = p.t[LM_SCALES].strides[1];
    a.z_n = p.t[LM_ZEROS].strides[0], a.z_g = p.t[LM_ZEROS].strides[1];
    a.bs = p.t[LM_BIAS].strides[0], a.ys_m = p.t[LM_Y].strides[0], a.ys_n = p.t[LM_Y].strides[1];
    // Exact for the blocks of mv4_parts (fewer than 1024).
    a.block_group = a.group % 128 ? 0 : (uint32_t)((1 << 20) / (a.group / 128) + 1);
    const dim3 grid((unsigned)lm_cdiv(a.N, 16), (unsigned)lm_cdiv(a.M, 16));
    const bool wide = a.group % 128 == 0;
    const auto go = [&](auto t) {
        typedef decltype(t) T;
        if (a.xs_k != 1 && a.K > 1) {
            mv4_rows<T><<<dim3((unsigned)lm_cdiv(a.K, 256), (unsigned)(a.M < 65535 ? a.M : 65535)), 256, 0, s>>>(
                a, static_cast<T *>(ws));
            a.x = ws, a.xs_m = a.K, a.xs_k = 1;
        }
        if (const int parts = mv4_parts(p)) {
            float *partial = parts > 1 ? reinterpret_cast<float *>(static_cast<char *>(ws) + mv4_rows_bytes(p)) : nullptr;
            if (wide) run_tiles<T, 128>(a, parts, partial, s);
            else if (a.group == 64) run_tiles<T, 64>(a, parts, partial, s);
            else run_tiles<T, 32>(a, parts, partial, s);
        } else if (wide) mv4_stream<T, true><<<grid, 64 * kMvWaves, 0, s>>>(a);
        else mv4_stream<T, false><<<grid, 64 * kMvWaves, 0, s>>>(a);
    };
    if (p.dtype == CONV_F32) go(float());
    else if (p.dtype == CONV_F16) go(f16_t());
    else go(bf16_t());
    return lm_launch_status();
}

}  // namespace miconv
