// Low-rank adapters of many requests beside a shared projection:
//   y[m] = base[m] + scaling[e] scales[m] B[e] (A[e] x[m]),  e = index[m].
//
// Bound by memory: x, base and y once, and the adapters that the rows name.
// Two kernels, both on the matrix cores.  adapters_in leaves A[e] x[m] in f32:
// workgroups take a tile of rows and a part of the columns, their waves share
// the part's columns and join in LDS.  adapters_out adds the parts up and
// multiplies by B[e], a tile of rows and 256 outputs per workgroup.
//
// A tile of 16 or 64 rows may name several adapters: each is taken for the
// whole tile in turn -- or by workgroups of its own, `slots` at a time, so that
// the tokens of many requests do not wait for each other -- and only its rows
// are kept.  Lanes of other rows load the row of a neighbour that has it: the
// rows of a matrix product do not touch each other.
//
// The inner sums stay f32 into the second product: they are cut into three
// bf16 terms, which hold all 24 bits, against exact weights (f16 weights are
// two bf16 terms, f32 ones go through the f32 instruction).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {
namespace {

constexpr int kWaves = 4;
constexpr int kUnit = 64;            // columns that a wave takes at a time: whole lines of 16-bit rows
constexpr int kRanks = 64;           // of an inner product's workgroup, and of a staged piece
constexpr int kOut = LM_ADAPTER_N;   // outputs of a workgroup
constexpr int kStride = kRanks + 8;  // of a staged row: 16-byte reads of 8 rows on different banks

struct AdapterP {
    const void *x, *a, *b, *base;
    const float *scales, *scaling;
    const int32_t *index;
    void *y;
    float *t;   // [parts][rows][width]
    S3 xs, as, bs, bases, ys, scs;   // as, bs: (adapter, row, column)
    int64_t scaling_e, L;
    int rows, K, N, R, E, parts, slots, width, tiles, blocks, groups;
    bool in_place;
};

struct f8_t { uint8_t u; };

// Eight values along a product's inner axis, as the matrix instruction takes
// them; Oct<X, T>: eight of memory type X for a product in type T.
template <typename T> struct Frag { uint4 v; };
template <> struct Frag<float> { float v[8]; };
template <typename X> using Oct = Raw<X, 8>;
template <typename T> __device__ __forceinline__ Frag<T> frag_of(const Raw<T, 8> &o)
{
    Frag<T> f;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f.v[i] = o.f(i);
    } else f.v = uint4{o.w[0], o.w[1], o.w[2], o.w[3]};
    return f;
}
// e4m3 fits bf16 and f16.
struct Oct8 { uint32_t w[2]; };
template <typename T> __device__ __forceinline__ Frag<T> frag_of(const Oct8 &o)
{
    Frag<T> f;
    f32x2 v[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[2 * i] = __builtin_bit_cast(f32x2, __builtin_amdgcn_cvt_pk_f32_fp8(o.w[i], false));
        v[2 * i + 1] = __builtin_bit_cast(f32x2, __builtin_amdgcn_cvt_pk_f32_fp8(o.w[i], true));
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.v[2 * i] = v[i][0], f.v[2 * i + 1] = v[i][1];
    } else f.v = uint4{pack2<T>(v[0][0], v[0][1]), pack2<T>(v[1][0], v[1][1]), pack2<T>(v[2][0], v[2][1]), pack2<T>(v[3][0], v[3][1])};
    return f;
}
template <typename T> __device__ __forceinline__ Raw<T, 8> load_oct(const T *p) { return load_raw<T, 8>(p); }
__device__ __forceinline__ Oct8 load_oct(const f8_t *p)
{
    struct __attribute__((packed, aligned(1))) Bytes { uint32_t w[2]; };
    const Bytes b = *reinterpret_cast<const Bytes *>(p);
    return {b.w[0], b.w[1]};
}
// The first n of eight values, any distance apart; the rest zero.
template <typename T> __device__ __forceinline__ Raw<T, 8> load_some(const T *p, int64_t step, int n)
{
    Raw<T, 8> r;
    r.zero();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) r.set(i, p[i * step]);
    return r;
}
__device__ __forceinline__ Oct8 load_some(const f8_t *p, int64_t step, int n)
{
    Oct8 r = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) r.w[i / 4] |= (uint32_t)p[i * step].u << (i % 4 * 8);
    return r;
}
template <typename T> __device__ __forceinline__ void mma(const Frag<T> &a, const Frag<T> &b, f32x4 &c)
{
    if constexpr (sizeof(T) == 4) mma_16x16x32_f32(a.v, b.v, c);
    else mma_16x16x32(a.v, b.v, c, T());
}

// The adapters of a tile's rows, lane r holding row r's.  take() gives those of
// one slot in turn: the adapter and the set of its rows.
struct Named {
    uint64_t left;
    int mine, turn;
    __device__ __forceinline__ Named(const AdapterP &p, int row0, int rows)
    {
        const int lane = threadIdx.x & 63;
        mine = lane < rows && row0 + lane < p.rows ? p.index[row0 + lane] : -1;
        if (mine < 0 || mine >= p.E) mine = -1;
        left = __ballot(mine >= 0), turn = 0;
    }
    __device__ __forceinline__ bool take(int slot, int slots, int &e, uint64_t &set)
    {
        while (left) {
            e = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
            set = __ballot(mine == e);
            left &= ~set;
            if (turn++ % slots == slot) return true;
        }
        return false;
    }
};
// Element offset of row m of a [N, columns, L] tensor.
__device__ __forceinline__ int64_t row_at(const AdapterP &p, const S3 &s, int m)
{
    int64_t l;
    const int64_t n = divide(m, p.L, l);
    return n * s.n + l * s.l;
}

// --------------------------------------------------------- x times A[e]^T --

// MF, RF: sixteens of rows and ranks.
template <typename T, typename X, int MF, int RF, bool DENSE> __global__ __launch_bounds__(64 * kWaves) void adapters_in(const AdapterP p)
{
    __shared__ f32x4 join[kWaves][MF * RF][64];
    typedef decltype(load_oct(static_cast<const X *>(nullptr))) XOct;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int at = blockIdx.x;
    const int part = at % p.parts;
    at /= p.parts;
    const int rank0 = at % p.groups * (16 * RF), row0 = at / p.groups * (16 * MF);
    const int units = (p.K + kUnit - 1) / kUnit;
    const int u1 = (int)((int64_t)units * (part + 1) / p.parts), whole = DENSE ? p.K / kUnit : 0;
    const int u0 = (int)((int64_t)units * part / p.parts) + wave;
    Named named(p, row0, 16 * MF);
    int e;
    uint64_t set;
    while (named.take(blockIdx.y, p.slots, e, set)) {
        const X *x[MF];
        const T *a[RF];
        const int k = (lane >> 4) * 8;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int r = m * 16 + (lane & 15);
            x[m] = static_cast<const X *>(p.x) + row_at(p, p.xs, row0 + (set >> r & 1 ? r : __builtin_ctzll(set))) + k * p.xs.c;
        }
#pragma unroll
        for (int j = 0; j < RF; ++j) {
            const int r = rank0 + j * 16 + (lane & 15);
            a[j] = static_cast<const T *>(p.a) + e * p.as.n + (r < p.R ? r : p.R - 1) * p.as.c + k * p.as.l;
        }
        f32x4 acc[MF][RF] = {};
        const auto product = [&](const XOct (&xo)[MF], const Raw<T, 8> (&ao)[RF]) {
            Frag<T> xf[MF];
#pragma unroll
            for (int m = 0; m < MF; ++m) xf[m] = frag_of<T>(xo[m]);
#pragma unroll
            for (int j = 0; j < RF; ++j) {
                const Frag<T> af = frag_of<T>(ao[j]);
#pragma unroll
                for (int m = 0; m < MF; ++m) mma<T>(af, xf[m], acc[m][j]);
            }
        };
        const int end = u1 < whole ? u1 : whole;
        if (u0 < end) {
            XOct xo[2][MF];
            Raw<T, 8> ao[2][RF];
            const auto fetch = [&](int u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int m = 0; m < MF; ++m) xo[h][m] = load_oct(x[m] + (int64_t)u * kUnit + h * 32);
#pragma unroll
                    for (int j = 0; j < RF; ++j) ao[h][j] = load_oct(a[j] + (int64_t)u * kUnit + h * 32);
                }
            };
            fetch(u0);
            for (int u = u0; u < end; u += kWaves) {
                XOct xn[2][MF];
                Raw<T, 8> an[2][RF];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int m = 0; m < MF; ++m) xn[h][m] = xo[h][m];
#pragma unroll
                    for (int j = 0; j < RF; ++j) an[h][j] = ao[h][j];
                }
                fetch(u + kWaves < end ? u + kWaves : u);
                product(xn[0], an[0]), product(xn[1], an[1]);
            }
        }
        // Units cut short, or all of them where columns lie apart.
        for (int u = u0; u < u1; u += kWaves) {
            if (u < whole) continue;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int c = u * kUnit + h * 32, n = p.K - c - k;
                XOct xo[MF];
                Raw<T, 8> ao[RF];
#pragma unroll
                for (int m = 0; m < MF; ++m) xo[m] = load_some(x[m] + c * p.xs.c, p.xs.c, n);
#pragma unroll
                for (int j = 0; j < RF; ++j) ao[j] = load_some(a[j] + c * p.as.l, p.as.l, n);
                product(xo, ao);
            }
        }
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int j = 0; j < RF; ++j) join[wave][m * RF + j][lane] = acc[m][j];
        __syncthreads();
        for (int f = wave; f < MF * RF; f += kWaves) {
            f32x4 sum = join[0][f][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) sum += join[w][f][lane];
            const int r = f / RF * 16 + (lane & 15), rank = rank0 + f % RF * 16 + (lane >> 4) * 4;
            if (rank < p.width && (set >> r & 1))
                *reinterpret_cast<f32x4 *>(p.t + ((int64_t)part * p.rows + row0 + r) * p.width + rank) = sum;
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------- times B[e]^T --

template <typename T> struct TermOf { typedef bf16_t type; static constexpr int n = 3; };
template <> struct TermOf<float> { typedef float type; static constexpr int n = 1; };

// v as the sum of three bf16 values, each the leading bits of what is left.
__device__ __forceinline__ void split(float v, uint16_t (&o)[3])
{
    const uint32_t u = __float_as_uint(v) & 0xffff0000u;
    const bool finite = __builtin_fabsf(v) < __builtin_inff();
    const float rest = finite ? v - __uint_as_float(u) : 0.f;
    const uint32_t w = __float_as_uint(rest) & 0xffff0000u;
    o[0] = finite ? (uint16_t)(u >> 16) : from_f32<bf16_t>(v).u;
    o[1] = (uint16_t)(w >> 16);
    o[2] = (uint16_t)(__float_as_uint(rest - __uint_as_float(w)) >> 16);
}

template <typename T, int MF, bool DENSE> __global__ __launch_bounds__(64 * kWaves) void adapters_out(const AdapterP p)
{
    typedef typename TermOf<T>::type U;
    constexpr int NT = TermOf<T>::n, MR = 16 * MF;
    __shared__ __attribute__((aligned(16))) U terms[NT][MR * kStride];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int row0 = blockIdx.x / p.blocks * MR, n0 = blockIdx.x % p.blocks * kOut + wave * 64;
    const int quad = lane >> 4, col = lane & 15;
    Named named(p, row0, MR);

    f32x4 acc[MF][4];
    // acc onto the rows of `set`: a lane's outputs are eight neighbours of a row, twice.
    const auto leave = [&](uint64_t set) {
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int r = m * 16 + col;
            if (!(set >> r & 1)) continue;
            T *y = static_cast<T *>(p.y) + row_at(p, p.ys, row0 + r);
            const T *base = p.base ? static_cast<const T *>(p.base) + row_at(p, p.bases, row0 + r) : nullptr;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = n0 + h * 32 + quad * 8;
                if (n >= p.N) continue;
                float v[8];
                if (DENSE && n + 8 <= p.N) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.f;
                    if (base) load_f32<T, 8>(base + n, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += acc[m][2 * h + i / 4][i % 4];
                    store_f32<T, 8>(y + n, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (n + i < p.N)
                            y[(n + i) * p.ys.c] = from_f32<T>((base ? to_f32(base[(n + i) * p.bases.c]) : 0.f) + acc[m][2 * h + i / 4][i % 4]);
                }
            }
        }
    };
    const auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[m][q] = f32x4{};
    };
    if (blockIdx.y == 0 && !p.in_place) {   // rows without an adapter
        const uint64_t none = __ballot(lane < MR && row0 + lane < p.rows && named.mine < 0);
        if (none) clear(), leave(none);
    }
    int e;
    uint64_t set;
    while (named.take(blockIdx.y, p.slots, e, set)) {
        clear();
        const float gain = p.scaling ? p.scaling[e * p.scaling_e] : 1.f;
        for (int rank0 = 0; rank0 < p.R; rank0 += kRanks) {
            const int ranks = p.width - rank0 < kRanks ? p.width - rank0 : kRanks;   // 32 or 64
            // The parts' sums of the adapter's rows, four ranks a thread.
            for (int i = threadIdx.x; i < MR * (kRanks / 4); i += 64 * kWaves) {
                const int r = i / (kRanks / 4), c = i % (kRanks / 4) * 4;
                f32x4 v = {};
                if (set >> r & 1 && c < ranks) {
                    const float *t = p.t + ((int64_t)row0 + r) * p.width + rank0 + c;
                    for (int s = 0; s < p.parts; ++s) v += *reinterpret_cast<const f32x4 *>(t + (int64_t)s * p.rows * p.width);
                    const float f = p.scales ? gain * p.scales[row_at(p, p.scs, row0 + r)] : gain;
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = rank0 + c + j < p.R ? v[j] * f : 0.f;
                }
                if constexpr (NT == 1) *reinterpret_cast<f32x4 *>(&terms[0][r * kStride + c]) = v;
                else {
                    uint16_t o[4][3];
#pragma unroll
                    for (int j = 0; j < 4; ++j) split(v[j], o[j]);
#pragma unroll
                    for (int s = 0; s < 3; ++s)
                        *reinterpret_cast<uint2 *>(&terms[s][r * kStride + c]) =
                            uint2{o[0][s] | (uint32_t)o[1][s] << 16, o[2][s] | (uint32_t)o[3][s] << 16};
                }
            }
            __syncthreads();
            if (n0 < p.N)
                for (int k0 = 0; k0 < ranks; k0 += 32) {
                    const int k = k0 + quad * 8, rank = rank0 + k;
                    Raw<T, 8> bo[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {   // which output is row `col` of the product's tile q
                        int n = n0 + (q >> 1) * 32 + (col >> 2) * 8 + (q & 1) * 4 + (col & 3);
                        n = n < p.N ? n : p.N - 1;
                        const T *b = static_cast<const T *>(p.b) + e * p.bs.n + n * p.bs.c;
                        if constexpr (DENSE) {   // R is a multiple of 8
                            bo[q] = load_oct(b + (rank < p.R ? rank : 0));
                            if (rank >= p.R) bo[q].zero();
                        } else bo[q] = load_some(b + rank * p.bs.l, p.bs.l, p.R - rank);
                    }
#pragma unroll
                    for (int m = 0; m < MF; ++m) {
                        Frag<U> tf[NT];
#pragma unroll
                        for (int s = 0; s < NT; ++s) {
                            const U *t = &terms[s][(m * 16 + col) * kStride + k];
                            __builtin_memcpy(&tf[s], __builtin_assume_aligned(t, 16), sizeof(tf[s]));
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if constexpr (std::is_same<T, f16_t>::value) {
                                Frag<bf16_t> hi, lo;   // 8 and 3 bits
                                uint32_t h[4], l[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float v0 = bo[q].f(2 * i), v1 = bo[q].f(2 * i + 1);
                                    const uint32_t u0 = __float_as_uint(v0) & 0xffff0000u, u1 = __float_as_uint(v1) & 0xffff0000u;
                                    const float r0 = __builtin_isinf(v0) ? 0.f : v0 - __uint_as_float(u0);
                                    const float r1 = __builtin_isinf(v1) ? 0.f : v1 - __uint_as_float(u1);
                                    h[i] = u0 >> 16 | u1, l[i] = __float_as_uint(r0) >> 16 | (__float_as_uint(r1) & 0xffff0000u);
                                }
                                hi.v = uint4{h[0], h[1], h[2], h[3]}, lo.v = uint4{l[0], l[1], l[2], l[3]};
                                mma<bf16_t>(lo, tf[1], acc[m][q]), mma<bf16_t>(hi, tf[2], acc[m][q]);
                                mma<bf16_t>(lo, tf[0], acc[m][q]), mma<bf16_t>(hi, tf[1], acc[m][q]);
                                mma<bf16_t>(hi, tf[0], acc[m][q]);
                            } else {
                                const Frag<T> bf = frag_of<T>(bo[q]);
#pragma unroll
                                for (int s = NT - 1; s >= 0; --s) mma<T>(bf, tf[s], acc[m][q]);
                            }
                        }
                    }
                }
            __syncthreads();
        }
        leave(set);
    }
}

S3 s3(const conv_tensor &t) { return {t.strides[0], t.strides[1], t.rank > 2 ? t.strides[2] : 0}; }

}  // namespace

int launch_lm_adapters(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    const AdapterShape shape = adapter_shape(p);
    if (q[LM_Z] && q[LM_Z] == q[LM_Y])   // in place, not over itself in another order
        for (int i = 0; i < p.t[LM_Y].rank; ++i)
            if (p.t[LM_Y].sizes[i] > 1 && p.t[LM_Z].strides[i] != p.t[LM_Y].strides[i]) return CONV_EINVAL;
    AdapterP a = {};
    a.x = q[LM_X], a.a = q[LM_A], a.b = q[LM_B], a.base = q[LM_Z], a.y = q[LM_Y];
    a.scales = static_cast<const float *>(q[LM_SCALES]), a.scaling = static_cast<const float *>(q[LM_D]);
    a.index = static_cast<const int32_t *>(q[LM_ROWS]);
    a.t = static_cast<float *>(ws);
    a.xs = s3(p.t[LM_X]), a.as = s3(p.t[LM_A]), a.bs = s3(p.t[LM_B]), a.bases = s3(p.t[LM_Z]), a.ys = s3(p.t[LM_Y]), a.scs = s3(p.t[LM_SCALES]);
    a.scaling_e = p.t[LM_D].strides[0], a.L = p.L;
    a.rows = (int)p.seqs, a.K = (int)p.K, a.N = (int)p.C, a.R = (int)p.S, a.E = (int)p.G;
    a.parts = shape.parts, a.slots = shape.slots, a.width = shape.width;
    a.tiles = (int)lm_cdiv(p.seqs, shape.rows), a.blocks = (int)lm_cdiv(p.C, kOut), a.groups = (int)lm_cdiv(p.S, kRanks);
    a.in_place = a.base == a.y;
    const bool f8 = p.t[LM_X].dtype == LM_F8;
    const bool dense_in = (a.xs.c == 1 && a.as.l == 1) || p.K == 1;
    const bool dense_out = a.bs.l == 1 && a.R % 8 == 0 && a.ys.c == 1 && (!a.base || a.bases.c == 1);
    const dim3 in((unsigned)(a.tiles * a.groups * a.parts), (unsigned)a.slots), out((unsigned)(a.tiles * a.blocks), (unsigned)a.slots);
    const auto run = [&](auto t, auto x) {
        typedef decltype(t) T;
        typedef decltype(x) X;
        const auto ranks = [&](auto mf, auto dense) {
            constexpr int MF = decltype(mf)::value;
            constexpr bool D = decltype(dense)::value;
            if (a.R <= 16) adapters_in<T, X, MF, 1, D><<<in, 64 * kWaves, 0, s>>>(a);
            else if (a.R <= 32) adapters_in<T, X, MF, 2, D><<<in, 64 * kWaves, 0, s>>>(a);
            else adapters_in<T, X, MF, 4, D><<<in, 64 * kWaves, 0, s>>>(a);
        };
        const auto rows = [&](auto mf) {
            constexpr int MF = decltype(mf)::value;
            if (a.E > 0) {
                if (dense_in) ranks(mf, std::true_type());
                else ranks(mf, std::false_type());
            }
            if (dense_out) adapters_out<T, MF, true><<<out, 64 * kWaves, 0, s>>>(a);
            else adapters_out<T, MF, false><<<out, 64 * kWaves, 0, s>>>(a);
        };
        if (shape.rows == 64) rows(std::integral_constant<int, 4>());
        else rows(std::integral_constant<int, 1>());
    };
    const auto types = [&](auto t) {
        if (f8) run(t, f8_t());
        else run(t, t);
    };
    if (p.dtype == CONV_F32) types(float());
    else if (p.dtype == CONV_F16) types(f16_t());
    else types(bf16_t());
    return lm_launch_status();
}

}  // namespace miconv
