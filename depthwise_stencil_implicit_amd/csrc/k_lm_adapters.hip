// Low-rank adapters of many requests beside a shared projection:
//   y[m] = base[m] + scaling[e] scales[m] B[e] (A[e] x[m]),  e = index[m].
//
// Bound by memory: x, base and y once, and the adapters that the rows name.
// Two kernels, both on the matrix cores.  adapters_in leaves A[e] x[m] in f32:
// workgroups take some rows and a part of the columns, their waves share the
// part's columns and join in LDS.  adapters_out adds the parts up, keeps them
// in LDS and multiplies by B[e], 64 outputs per wave at a time.
//
// The rows of a workgroup share an adapter.  Three ways to find them, by the
// number of rows and adapters (adapter_shape): the workgroup of every 16th row that
// names an adapter gathers those rows by a look at all of index; tiles of 64 rows
// in the adapters' order, which each workgroup of adapters_in finds by counting
// all of index, and lists for the kernel behind; or such tiles that adapters_sort,
// one workgroup, has listed before.  (Tiles of neighbours, which may name several
// adapters, took each of them in turn: four changes in 8192 rows made the call 1.3
// times as long, tokens among prompts many times.)
//
// The inner sums stay f32 into the second product: they are cut into three
// bf16 terms, which hold all 24 bits, against exact weights (f16 weights are
// two bf16 terms, f32 ones go through the f32 instruction).  y is rounded once.
//
// Measured (medians of traced kernels): bf16 8192 rows, 4096 columns, 8192 outputs,
// rank 32, 6 adapters: in 24 us, 5 of them to find the rows, out 69 (3.9 TB/s of
// the 5.1 that a copy reaches).  8-bit rows, 4100 x 5120 to 5120, rank 64: 21 and
// 33.  32 tokens of 24 adapters, 4096 x 4096, rank 16: 5.5 and 7.4, a launch and
// three waits for memory each.  What adapters_in asks for (x, and A once for each
// 64 rows) comes at about 4 TB/s, so high ranks cost it (8192 x 4096: rank 16 28
// us, 64 47, 128 70, which goes through x twice).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = LM_ADAPTER_TILE;   // rows of a sorted tile
constexpr int kUnit = 64;            // columns that a wave takes at a time: whole lines of 16-bit rows
constexpr int kRanks = 64;           // of an adapters_in workgroup; staged at most beside weights in registers
constexpr int kOutRows = 2;          // sixteens of rows of adapters_out's tile: with four it was 1.2 to 1.7 times as long
constexpr int kOut = LM_ADAPTER_N;   // outputs of a workgroup at a time

struct AdapterP {
    const void *x, *a, *b, *base;
    const float *scales, *scaling;
    const int32_t *index;
    void *y;
    float *t;   // [parts][rows][width]
    int *order, *tile_count;
    int4 *tiles;
    S3 xs, as, bs, bases, ys, scs;   // as, bs: (adapter, row, column)
    int64_t scaling_e, L;
    int rows, K, N, R, E, parts, width, groups, spans, reps;   // outputs of a workgroup: reps of kOut, spans of them
    bool in_place;
};

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
struct f8_t { uint8_t u; };
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
// Sixteen neighbours, the first and the second eight.
template <typename T> __device__ __forceinline__ void load_both(const T *p, Raw<T, 8> &a, Raw<T, 8> &b)
{
    a = load_oct(p), b = load_oct(p + 8);
}
__device__ __forceinline__ void load_both(const f8_t *p, Oct8 &a, Oct8 &b)
{
    struct __attribute__((packed, aligned(1))) Bytes { uint32_t w[4]; };
    const Bytes v = *reinterpret_cast<const Bytes *>(p);
    a = {{v.w[0], v.w[1]}}, b = {{v.w[2], v.w[3]}};
}
// The first n of V values, any distance apart; the rest, all of them for an n
// below one, zero.  There is an (n - 1)th value at p in any case, which loads
// past the end repeat: behind branches they would be waited for one by one.
template <int V, typename T> __device__ __forceinline__ Raw<T, V> load_some(const T *p, int64_t step, int n)
{
    T v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[(i < n ? i : n - 1) * step];
    Raw<T, V> r;
    r.zero();
#pragma unroll
    for (int i = 0; i < V; ++i) r.set(i, i < n ? v[i] : T{});
    return r;
}
template <int V> __device__ __forceinline__ Oct8 load_some(const f8_t *p, int64_t step, int n)
{
    uint8_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[(i < n ? i : n - 1) * step].u;
    Oct8 r = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i / 4] |= (uint32_t)(i < n ? v[i] : 0) << (i % 4 * 8);
    return r;
}
// Four values past the L2's lines in use: the kernel does not read them again.
template <typename T> __device__ __forceinline__ void store_piece(T *p, const float (&v)[4])
{
    if constexpr (sizeof(T) == 4) store_f32<T, 4, true>(p, v);
    else {
        typedef uint32_t any2 __attribute__((ext_vector_type(2), aligned(2)));
        __builtin_nontemporal_store(any2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])}, reinterpret_cast<any2 *>(p));
    }
}
template <typename T> __device__ __forceinline__ void mma(const Frag<T> &a, const Frag<T> &b, f32x4 &c)
{
    if constexpr (sizeof(T) == 4) mma_16x16x32_f32(a.v, b.v, c);
    else mma_16x16x32(a.v, b.v, c, T());
}

// A workgroup's rows, at most MR of them (`set`, `list`), and their adapter e, one
// outside 0 .. E - 1 for rows without any.  Made by all waves; ends in a barrier.
template <bool GATHER, int MR> struct Group;
template <int MR> struct Group<false, MR> {
    uint64_t set;
    int e;
    const int *list;
    __device__ __forceinline__ Group(const AdapterP &p, int at, int *rows) : list(rows)
    {
        constexpr int PER = kTile / MR;   // of a listed tile
        const int lane = threadIdx.x & 63;
        set = 0;
        if (at / PER >= *p.tile_count) return;
        const int4 tile = p.tiles[at / PER];   // adapter, first place in the order, rows
        const int first = at % PER * MR, n = tile.z - first < MR ? tile.z - first : MR;
        if (n <= 0) return;
        e = tile.x;
        set = n >= 64 ? ~0ull : (1ull << n) - 1;
        if (threadIdx.x < MR && lane < n) rows[lane] = p.order[tile.y + first + lane];
        lds_sync();
    }
    __device__ __forceinline__ int row(int r) const { return list[r]; }
};
template <int MR> struct Group<true, MR> {
    uint64_t set;
    int e;
    const int *list;
    __device__ __forceinline__ Group(const AdapterP &p, int m, int *rows) : list(rows)
    {
        constexpr int LOOKS = LM_ADAPTER_FEW / 64;
        const int lane = threadIdx.x & 63;
        int v[LOOKS];
#pragma unroll
        for (int j = 0; j < LOOKS; ++j) v[j] = p.index[j * 64 + lane < p.rows ? j * 64 + lane : p.rows - 1];
        e = __builtin_amdgcn_readfirstlane(p.index[m]);
        int count = 0, first = 0;   // rows of the adapter so far, those in front of m
#pragma unroll
        for (int j = 0; j < LOOKS; ++j) {
            const uint64_t same = __ballot(j * 64 + lane < p.rows && v[j] == e);
            if (m >> 6 == j) first = count + __builtin_popcountll(same & ((1ull << (m & 63)) - 1));
            const int place = count + __builtin_popcountll(same & ((1ull << lane) - 1)) - first;
            if (m >> 6 <= j && threadIdx.x < 64 && same >> lane & 1 && place >= 0 && place < 16) rows[place] = j * 64 + lane;
            count += __builtin_popcountll(same);
        }
        const int n = count - first;
        set = first % 16 ? 0 : n >= 16 ? 0xffff : (1ull << n) - 1;
        lds_sync();
    }
    __device__ __forceinline__ int row(int r) const { return list[r]; }
};
// The group of a tile that nothing has listed yet: of few adapters' rows, each
// workgroup counts all of index and takes those whose turn it is.  at: the
// places of one workgroup of each tile, which lists it for the kernel behind.
struct FoundGroup {
    uint64_t set;
    int e;
    const int *list;
    __device__ __forceinline__ FoundGroup(const AdapterP &p, int at, bool lists, int *rows) : list(rows)
    {
        constexpr int STEPS = LM_ADAPTER_FIND / (64 * kWaves);
        __shared__ int counts[kWaves][64];
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int per = (p.rows + 64 * kWaves - 1) / (64 * kWaves), from = wave * per * 64;   // steps of a wave; its rows
        const auto row_of = [&](int s) { return from + s * 64 + lane; };
        int v[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) v[s] = p.index[row_of(s) < p.rows ? row_of(s) : p.rows - 1];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) v[s] = s >= per || row_of(s) >= p.rows ? -1 : v[s] < 0 || v[s] >= p.E ? p.E : v[s];
        int count = 0;   // rows of adapter `lane` here; p.E: of none
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            for (uint64_t left = __ballot(v[s] >= 0); left;) {
                const int now = __builtin_amdgcn_readlane(v[s], __builtin_ctzll(left));
                const uint64_t same = __ballot(v[s] == now);
                count += lane == now ? __builtin_popcountll(same) : 0;
                left &= ~same;
            }
        counts[wave][lane] = count;
        lds_sync();
        int n = 0, front = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) front += w < wave ? counts[w][lane] : 0, n += counts[w][lane];
        const int t = (n + kTile - 1) / kTile;
        int upto = t;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int a = __shfl_up(upto, d);
            if (lane >= d) upto += a;
        }
        const uint64_t mine = __ballot(lane <= p.E && at < upto && at >= upto - t);
        set = 0;
        const int all = __builtin_amdgcn_readlane(upto, p.E);
        if (lists && at == 0 && threadIdx.x == 0) *p.tile_count = all;
        if (!mine) return;
        e = __builtin_ctzll(mine);
        const int first = (at - __builtin_amdgcn_readlane(upto - t, e)) * kTile, left = __builtin_amdgcn_readlane(n, e) - first;
        const int rows_here = left < kTile ? left : kTile;
        int place = __builtin_amdgcn_readlane(front, e) - first;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const uint64_t same = __ballot(v[s] == e);
            const int i = place + __builtin_popcountll(same & ((1ull << lane) - 1));
            if (v[s] == e && i >= 0 && i < kTile) rows[i] = row_of(s);
            place += __builtin_popcountll(same);
        }
        set = rows_here >= 64 ? ~0ull : (1ull << rows_here) - 1;
        lds_sync();
        if (lists && wave == 0) {
            if (lane == 0) p.tiles[at] = int4{e < p.E ? e : -1, at * kTile, rows_here, 0};
            if (lane < rows_here) p.order[at * kTile + lane] = rows[lane];
        }
    }
    __device__ __forceinline__ int row(int r) const { return list[r]; }
};
// Element offset of row m of a [N, columns, L] tensor.
__device__ __forceinline__ int64_t row_at(const AdapterP &p, const S3 &s, int m)
{
    int64_t l;
    const int64_t n = divide(m, p.L, l);
    return n * s.n + l * s.l;
}

// --------------------------------------------------------- rows by adapter --

// The rows in the order of their adapters (in their own order within one, so
// results repeat; 9 us for 8192 rows in runs, latency of its passes), and tiles of them; rows without an adapter are in tiles of
// their own.  Each wave counts and then places a stretch of rows; kSorted
// adapters at a time, and those without in the first turn's last bucket.
constexpr int kSorted = 896;
__global__ __launch_bounds__(1024) void adapters_sort(const AdapterP p)
{
    __shared__ int counts[16][kSorted + 1];
    __shared__ int2 sums[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t each = ((int64_t)p.rows + 1023) / 1024 * 64, from = wave * each, to = from + each < p.rows ? from + each : p.rows;
    int rows = 0, tiles = 0;   // placed so far
    for (int64_t e0 = 0; e0 == 0 || e0 < p.E; e0 += kSorted) {
        // Eight steps' loads at a time.
        int idx[8];
        const auto load = [&](int64_t i) {
#pragma unroll
            for (int s = 0; s < 8; ++s) idx[s] = p.index[i + s * 64 + lane < to ? i + s * 64 + lane : to - 1];
        };
        const auto bucket = [&](int64_t i, int e) {
            if (i >= to) return -1;
            if (e < 0 || e >= p.E) return e0 == 0 ? kSorted : -1;
            return e >= e0 && e < e0 + kSorted ? (int)(e - e0) : -1;
        };
        for (int i = tid; i < 16 * (kSorted + 1); i += 1024) (&counts[0][0])[i] = 0;
        __syncthreads();
        for (int64_t i = from; i < to; i += 512) {
            load(i);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int b = bucket(i + s * 64 + lane, idx[s]);
                uint64_t left = __ballot(b >= 0);
                while (left) {
                    const int now = __builtin_amdgcn_readlane(b, __builtin_ctzll(left));
                    const uint64_t same = __ballot(b == now);
                    if (lane == 0) counts[wave][now] += __builtin_popcountll(same);
                    left &= ~same;
                }
            }
        }
        __syncthreads();
        // Bucket tid: its rows, its tiles, and the sums of both in front of it.
        int n = 0;
        if (tid <= kSorted) {
#pragma unroll
            for (int w = 0; w < 16; ++w) n += counts[w][tid];
        }
        const int t = (n + kTile - 1) / kTile;
        int2 upto{n, t};
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int a = __shfl_up(upto.x, d), b = __shfl_up(upto.y, d);
            if (lane >= d) upto.x += a, upto.y += b;
        }
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        int2 all{0, 0}, front{0, 0};
        for (int w = 0; w < 16; ++w) {
            if (w == wave) front = all;
            all.x += sums[w].x, all.y += sums[w].y;
        }
        int at = rows + front.x + upto.x - n;
        const int tile = tiles + front.y + upto.y - t;
        for (uint64_t with = __ballot(t > 0); with; with &= with - 1) {   // a bucket's tiles by the whole wave
            const int who = __builtin_ctzll(with), bucket_n = __builtin_amdgcn_readlane(n, who);
            const int bucket_at = __builtin_amdgcn_readlane(at, who), bucket_tile = __builtin_amdgcn_readlane(tile, who);
            const int e = wave * 64 + who < kSorted ? (int)e0 + wave * 64 + who : -1;
            for (int i = lane; i * kTile < bucket_n; i += 64)
                p.tiles[bucket_tile + i] = int4{e, bucket_at + i * kTile, bucket_n - i * kTile < kTile ? bucket_n - i * kTile : kTile, 0};
        }
        if (tid <= kSorted) {
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                const int c = counts[w][tid];
                counts[w][tid] = at, at += c;
            }
        }
        __syncthreads();
        for (int64_t i = from; i < to; i += 512) {
            if (to - from > 512) load(i);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int64_t at = i + s * 64 + lane;
                const int b = bucket(at, idx[s]);
                uint64_t left = __ballot(b >= 0);
                while (left) {
                    const int now = __builtin_amdgcn_readlane(b, __builtin_ctzll(left));
                    const uint64_t same = __ballot(b == now);
                    const int first = counts[wave][now];
                    if (b == now) p.order[first + __builtin_popcountll(same & ((1ull << lane) - 1))] = (int)at;
                    if (lane == 0) counts[wave][now] = first + __builtin_popcountll(same);
                    left &= ~same;
                }
            }
        }
        __syncthreads();
        rows += all.x, tiles += all.y;
    }
    if (tid == 0) *p.tile_count = tiles;
}

// --------------------------------------------------------- x times A[e]^T --

// MF, RF: sixteens of rows (gathered: one) and ranks.
template <typename T, typename X, int MF, int RF, bool DENSE, bool FIND> __global__ __launch_bounds__(64 * kWaves) void adapters_in(const AdapterP p)
{
    constexpr bool GATHER = MF == 1;
    __shared__ f32x4 join[kWaves][MF * RF][64];
    __shared__ int list[16 * MF];
    typedef typename std::conditional<sizeof(X) == 1, Oct8, Raw<T, 8>>::type XOct;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int at = blockIdx.x;
    const int part = at % p.parts;
    at /= p.parts;
    const int rank0 = at % p.groups * (16 * RF), tile = GATHER ? blockIdx.y : at / p.groups;
    const int units = (p.K + kUnit - 1) / kUnit;
    const int whole = DENSE ? p.K / kUnit : 0;
    const int piece = part * kWaves + wave;
    const int u0 = (int)((int64_t)units * piece / (p.parts * kWaves)), u1 = (int)((int64_t)units * (piece + 1) / (p.parts * kWaves));
    const auto group = [&] {
        if constexpr (FIND) return FoundGroup(p, tile, part == 0 && rank0 == 0, list);
        else return Group<GATHER, 16 * MF>(p, tile, list);
    }();
    const uint64_t set = group.set;
    const int64_t e = group.e;
    if (!set || e < 0 || e >= p.E) return;
    {
        const X *x[MF];
        const T *a[RF];
        // A lane's part of a unit: sixteen neighbours, eight for each of two
        // products (which columns meet there is the same for both sides).
        const int k = (lane >> 4) * 16;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int r = m * 16 + (lane & 15);
            x[m] = static_cast<const X *>(p.x) + row_at(p, p.xs, group.row(set >> r & 1 ? r : 0)) + k * p.xs.c;
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
            // Two units' registers in turn: handed on from one to the other
            // they would be waited for at once.
            XOct xo[2][2][MF];
            Raw<T, 8> ao[2][2][RF];
            const int count = end - u0, turn = GATHER ? 0 : tile % count;   // from another one on for each tile, as in adapters_out
            const auto fetch = [&](int i, XOct (&xs)[2][MF], Raw<T, 8> (&as)[2][RF]) {
                i = (i < count ? i : 0) + turn;
                const int64_t c = (int64_t)(u0 + (i < count ? i : i - count)) * kUnit;
#pragma unroll
                for (int m = 0; m < MF; ++m) load_both(x[m] + c, xs[0][m], xs[1][m]);
#pragma unroll
                for (int j = 0; j < RF; ++j) load_both(a[j] + c, as[0][j], as[1][j]);
            };
            fetch(0, xo[0], ao[0]);
            for (int i = 0; i < count; i += 2) {
                fetch(i + 1, xo[1], ao[1]);
                __builtin_amdgcn_sched_barrier(0);
                product(xo[0][0], ao[0][0]), product(xo[0][1], ao[0][1]);
                if (i + 1 >= count) break;
                fetch(i + 2, xo[0], ao[0]);
                __builtin_amdgcn_sched_barrier(0);
                product(xo[1][0], ao[1][0]), product(xo[1][1], ao[1][1]);
            }
        }
        // Units cut short, or all of them where columns lie apart.
        for (int u = u0 > whole ? u0 : whole; u < u1; ++u) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int c = u * kUnit + h * 8, n = p.K - c - k;
                XOct xo[MF];
                Raw<T, 8> ao[RF];
#pragma unroll
                for (int m = 0; m < MF; ++m) xo[m] = load_some<8>(x[m] + c * p.xs.c, p.xs.c, n);
#pragma unroll
                for (int j = 0; j < RF; ++j) ao[j] = load_some<8>(a[j] + c * p.as.l, p.as.l, n);
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
                *reinterpret_cast<f32x4 *>(p.t + ((int64_t)part * p.rows + group.row(r)) * p.width + rank) = sum;
        }
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

// Eight weights against the terms of a row.
template <typename T> struct Weights { Frag<T> f; };
template <> struct Weights<f16_t> { Frag<bf16_t> hi, lo; };   // 8 and 3 bits
template <typename T> __device__ __forceinline__ Weights<T> weights_of(const Raw<T, 8> &o)
{
    Weights<T> w;
    if constexpr (std::is_same<T, f16_t>::value) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v0 = o.f(2 * i), v1 = o.f(2 * i + 1);
            const uint32_t u0 = __float_as_uint(v0) & 0xffff0000u, u1 = __float_as_uint(v1) & 0xffff0000u;
            const float r0 = __builtin_isinf(v0) ? 0.f : v0 - __uint_as_float(u0);
            const float r1 = __builtin_isinf(v1) ? 0.f : v1 - __uint_as_float(u1);
            h[i] = u0 >> 16 | u1, l[i] = __float_as_uint(r0) >> 16 | (__float_as_uint(r1) & 0xffff0000u);
        }
        w.hi.v = uint4{h[0], h[1], h[2], h[3]}, w.lo.v = uint4{l[0], l[1], l[2], l[3]};
    } else w.f = frag_of<T>(o);
    return w;
}
template <typename T, typename U> __device__ __forceinline__ void mma_terms(const Weights<T> &w, const Frag<U> (&t)[TermOf<T>::n], f32x4 &c)
{
    if constexpr (std::is_same<T, f16_t>::value) {
        mma<bf16_t>(t[1], w.lo, c), mma<bf16_t>(t[2], w.hi, c);
        mma<bf16_t>(t[0], w.lo, c), mma<bf16_t>(t[1], w.hi, c), mma<bf16_t>(t[0], w.hi, c);
    } else {
#pragma unroll
        for (int s = TermOf<T>::n - 1; s >= 0; --s) mma<T>(t[s], w.f, c);
    }
}

// A wave takes 64 outputs at a time: a lane's four neighbours of four rows per
// sixteen, so that sixteen lanes read and write a line of a 16-bit row.
// KS: 32s of ranks; 0: any number of them, their weights loaded in turn.  DENSE:
// outputs are contiguous, and each one's weights.  OCTS: ranks are a multiple of
// eight; if not, eight weights from one on may belong to the outputs behind, are
// loaded all the same, and masked when they are used (one by one they made rank
// 4 of 4096 x 4096 take 64 us for 20 at rank 8).
template <typename T, int MF, int KS, bool DENSE, bool OCTS> __global__ __launch_bounds__(64 * kWaves) void adapters_out(const AdapterP p)
{
    typedef typename TermOf<T>::type U;
    constexpr bool GATHER = MF == 1;
    constexpr int NT = TermOf<T>::n, MR = 16 * MF, NQ = 4;
    constexpr int RANKS = KS ? kRanks : LM_MAX_RANK, STRIDE = RANKS + 8;   // 16-byte reads of 8 rows on different banks
    __shared__ __attribute__((aligned(16))) U terms[NT][MR * STRIDE];
    __shared__ int list[MR];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int quad = lane >> 4, col = lane & 15;
    const int tile = GATHER ? blockIdx.y : blockIdx.x / p.spans, span = GATHER ? blockIdx.x : blockIdx.x % p.spans;
    // The workgroup's 256s of outputs, from another one on for each tile: rows
    // are powers of two apart often enough that tiles at one column would keep
    // to a few of the memory's channels.
    const int block0 = span * p.reps, left = (p.N + kOut - 1) / kOut - block0, blocks = left < p.reps ? left : p.reps;
    const int turn = GATHER ? 0 : tile % blocks;
    const auto place = [&](int i) {
        i = i < blocks ? i : 0;
        i += turn;
        return (block0 + (i < blocks ? i : i - blocks)) * kOut + wave * 64;
    };
    const Group<GATHER, MR> group(p, tile, list);
    const uint64_t set = group.set;
    const int e = group.e;
    if (!set) return;

    // Offsets of a lane's rows, m * 16 + quad * 4 + i of the tile.
    int64_t yo[MF][4], bo[MF][4];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = m * 16 + quad * 4 + i, row = group.row(set >> r & 1 ? r : 0);
            yo[m][i] = row_at(p, p.ys, row);
            bo[m][i] = p.base ? row_at(p, p.bases, row) : 0;
        }
    const T *base = static_cast<const T *>(p.base ? p.base : p.b);
    T *y = static_cast<T *>(p.y);
    // Past the last output, or without a base, loads repeat what is there.
    const auto get_base = [&](int n0, Raw<T, 4> (&o)[MF][4]) {
        const int n = n0 + col * 4;
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DENSE) o[m][i] = load_raw<T, 4>(base + bo[m][i] + (!p.base ? 0 : n <= p.N - 4 ? n : p.N - 4));
                else if (p.base) o[m][i] = load_some<4>(base + bo[m][i] + n * p.bases.c, p.bases.c, p.N - n);
            }
    };
    const auto leave = [&](int n0, const Raw<T, 4> (&o)[MF][4], const f32x4 (&acc)[MF][NQ]) {
        const int n = n0 + col * 4;
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!(set >> (m * 16 + quad * 4 + i) & 1)) continue;
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = (p.base ? o[m][i].f(j) : 0.f) + acc[m][j][i];
                if (DENSE && n + 4 <= p.N) store_piece(y + yo[m][i] + n, v);
                else {
                    if (DENSE && p.base && n < p.N) {   // the last piece of a row was loaded from its end
                        const int by = n - (p.N - 4);
#pragma unroll
                        for (int j = 0; j < 3; ++j) {
                            const float f = by == 1 ? o[m][i].f(j + 1) : by == 2 ? o[m][i].f(j + 2 < 4 ? j + 2 : 3) : o[m][i].f(3);
                            v[j] = f + acc[m][j][i];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < p.N) y[yo[m][i] + (n + j) * p.ys.c] = from_f32<T>(v[j]);
                }
            }
    };
    if (e < 0 || e >= p.E) {   // rows without an adapter
        if (p.in_place) return;
        const f32x4 zero[MF][NQ] = {};
        Raw<T, 4> o[2][MF][4];
        get_base(place(0), o[0]);
        for (int i = 0; i < blocks; i += 2) {
            get_base(place(i + 1), o[1]);
            __builtin_amdgcn_sched_barrier(0);
            leave(place(i), o[0], zero);
            if (i + 1 >= blocks) break;
            get_base(place(i + 2), o[0]);
            __builtin_amdgcn_sched_barrier(0);
            leave(place(i + 1), o[1], zero);
        }
        return;
    }
    const T *b = static_cast<const T *>(p.b) + e * p.bs.n;
    // Where the last eight weights of all adapters start, from this one's first.
    const int64_t last = (p.E - 1 - e) * p.bs.n + (p.N - 1) * p.bs.c + p.R - 8;
    const float gain = p.scaling ? p.scaling[e * p.scaling_e] : 1.f;
    // Weights for the outputs n0 .. n0 + 63 from `rank` on; tile q
    // of a product has every fourth output from n0 + q on.
    const auto get_weights = [&](int n0, int rank, Raw<T, 8> (&o)[NQ]) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            int n = n0 + col * 4 + q;
            n = n < p.N ? n : p.N - 1;
            if constexpr (OCTS) o[q] = load_oct(b + n * p.bs.c + (rank < p.R ? rank : 0));
            else if constexpr (DENSE) {
                const int64_t at = n * p.bs.c + (rank < p.R ? rank : 0);
                o[q] = load_oct(b + (at < last ? at : last));
            } else o[q] = load_some<8>(b + n * p.bs.c + rank * p.bs.l, p.bs.l, p.R - rank);
        }
    };
    // The parts' sums of the rows, scaled and cut into terms.
    const auto stage = [&]() {
        const int quads = p.width / 4;
        for (int i = threadIdx.x; i < MR * quads; i += 64 * kWaves) {
            const int r = i / quads, c = i % quads * 4;
            f32x4 v = {};
            if (set >> r & 1 && c < p.R) {
                const int row = group.row(r);
                const float *t = p.t + (int64_t)row * p.width + c;
                const float f = p.scales ? gain * p.scales[row_at(p, p.scs, row)] : gain;
                constexpr int AT_ONCE = GATHER ? 16 : 4;   // all of a short call's, which waits for them
                for (int s0 = 0; s0 < p.parts; s0 += AT_ONCE) {
                    f32x4 u[AT_ONCE];
#pragma unroll
                    for (int s = 0; s < AT_ONCE; ++s)
                        u[s] = *reinterpret_cast<const f32x4 *>(t + (int64_t)(s0 + s < p.parts ? s0 + s : 0) * p.rows * p.width);
#pragma unroll
                    for (int s = 0; s < AT_ONCE; ++s) v += s0 + s < p.parts ? u[s] : f32x4{};
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = c + j < p.R ? v[j] * f : 0.f;
            }
            if constexpr (NT == 1) *reinterpret_cast<f32x4 *>(&terms[0][r * STRIDE + c]) = v;
            else {
                uint16_t o[4][3];
#pragma unroll
                for (int j = 0; j < 4; ++j) split(v[j], o[j]);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    *reinterpret_cast<uint2 *>(&terms[s][r * STRIDE + c]) =
                        uint2{o[0][s] | (uint32_t)o[1][s] << 16, o[2][s] | (uint32_t)o[3][s] << 16};
            }
        }
    };
    // acc += the staged terms from k on times the weights o.  Ranks past the
    // last are zeros in the terms; weights there are an earlier rank's.
    const auto multiply = [&](const Raw<T, 8> (&o)[NQ], int n0, int k, f32x4 (&acc)[MF][NQ]) {
        Frag<U> t[MF][NT];
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int s = 0; s < NT; ++s)
                __builtin_memcpy(&t[m][s], __builtin_assume_aligned(&terms[s][(m * 16 + col) * STRIDE + k + quad * 8], 16), sizeof(t[m][s]));
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            Raw<T, 8> w = o[q];
            const int rank = k + quad * 8;
            if constexpr (!OCTS && DENSE) {
                int n = n0 + col * 4 + q;
                n = n < p.N ? n : p.N - 1;
                const int64_t over = n * p.bs.c + (rank < p.R ? rank : 0) - last;   // of the last adapter's last outputs
                if (__ballot(over > 0)) shift_row<T, 8>(w, over > 0 ? (int)over : 0);
#pragma unroll
                for (int i = 0; i < w.n; ++i) {
                    constexpr int per = 4 / sizeof(T);
                    const int has = p.R - rank - i * per;   // of the word's elements
                    w.w[i] = has >= per ? w.w[i] : has > 0 ? w.w[i] & 0xffffu : 0u;
                }
            } else if (rank >= p.R) w.zero();
            const Weights<T> wf = weights_of<T>(w);
#pragma unroll
            for (int m = 0; m < MF; ++m) mma_terms<T, U>(wf, t[m], acc[m][q]);
        }
    };
    if constexpr (KS > 0) {   // staged once; the next outputs' base in flight
        Raw<T, 8> w[KS][NQ];
        Raw<T, 4> o[2][MF][4];
        const auto get_all = [&](int n0) {
#pragma unroll
            for (int k = 0; k < KS; ++k) get_weights(n0, k * 32 + quad * 8, w[k]);
        };
        const auto finish = [&](int i, const Raw<T, 4> (&os)[MF][4]) {
            f32x4 acc[MF][NQ] = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) multiply(w[k], place(i), k * 32, acc);
            __builtin_amdgcn_sched_barrier(0);
            get_all(place(i + 1));
            leave(place(i), os, acc);
        };
        get_all(place(0)), get_base(place(0), o[0]);
        stage();
        __syncthreads();
        for (int i = 0; i < blocks; i += 2) {
            get_base(place(i + 1), o[1]);
            __builtin_amdgcn_sched_barrier(0);
            finish(i, o[0]);
            if (i + 1 >= blocks) break;
            get_base(place(i + 2), o[0]);
            __builtin_amdgcn_sched_barrier(0);
            finish(i + 1, o[1]);
        }
    } else {
        stage();
        __syncthreads();
        for (int i = 0; i < blocks; ++i) {
            const int n0 = place(i);
            Raw<T, 4> o[MF][4];
            if constexpr (DENSE) get_base(n0, o);
            f32x4 acc[MF][NQ] = {};
            Raw<T, 8> w[2][NQ];
            get_weights(n0, quad * 8, w[0]);
            for (int k = 0; k < p.R; k += 64) {
                if (k + 32 < p.R) get_weights(n0, k + 32 + quad * 8, w[1]);
                multiply(w[0], n0, k, acc);
                if (k + 32 >= p.R) break;
                if (k + 64 < p.R) get_weights(n0, k + 64 + quad * 8, w[0]);
                multiply(w[1], n0, k + 32, acc);
            }
            if constexpr (!DENSE) get_base(n0, o);
            leave(n0, o, acc);
        }
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
    a.parts = shape.parts, a.width = shape.width, a.reps = shape.reps;
    const bool few = shape.rows == 1;   // a workgroup for each row, which gathers its like
    a.spans = (int)lm_cdiv(p.C, (int64_t)kOut * shape.reps), a.groups = (int)lm_cdiv(p.S, kRanks);
    const unsigned tiles = (unsigned)shape.tiles, tiles_out = tiles * (few ? 1 : kTile / (16 * kOutRows));
    if (!few) {
        a.tiles = reinterpret_cast<int4 *>(static_cast<char *>(ws) + adapter_sums_bytes(p));
        a.order = reinterpret_cast<int *>(a.tiles + shape.tiles);
        a.tile_count = a.order + (shape.find ? shape.tiles * kTile : p.seqs);
        if (!shape.find) adapters_sort<<<1, 1024, 0, s>>>(a);
    }
    a.in_place = a.base == a.y;
    const bool f8 = p.t[LM_X].dtype == LM_F8;
    const bool dense_in = adapter_dense_in(p);
    const bool octs = a.R % 8 == 0;
    // With strides of their own, ranks that are not eights would need a far last place.
    const bool runs = a.bs.l == 1 && (octs || (a.bs.c >= a.R && a.bs.n >= (a.N - 1) * a.bs.c + a.R && (a.N - 1) * a.bs.c + a.R >= 8));
    // Without a base the loads in its place are of B, which has to have something.
    const bool dense_out = runs && a.N >= 4 && a.ys.c == 1 && (a.base ? a.bases.c == 1 : a.E > 0);
    const dim3 in((few ? 1 : tiles) * a.groups * a.parts, few ? tiles : 1), out((few ? 1 : tiles_out) * a.spans, few ? tiles_out : 1);
    const auto run = [&](auto t, auto x) {
        typedef decltype(t) T;
        typedef decltype(x) X;
        const auto ranks = [&](auto mf, auto dense, auto find) {
            constexpr int MF = decltype(mf)::value;
            constexpr bool D = decltype(dense)::value, FIND = decltype(find)::value;
            if (a.R <= 16) adapters_in<T, X, MF, 1, D, FIND><<<in, 64 * kWaves, 0, s>>>(a);
            else if (a.R <= 32) adapters_in<T, X, MF, 2, D, FIND><<<in, 64 * kWaves, 0, s>>>(a);
            else adapters_in<T, X, MF, 4, D, FIND><<<in, 64 * kWaves, 0, s>>>(a);
        };
        const auto rows = [&](auto mf) {
            constexpr int MF = decltype(mf)::value;
            if (a.E > 0) {
                if constexpr (MF > 1) {
                    if (shape.find) ranks(mf, std::true_type(), std::true_type());
                    else if (dense_in) ranks(mf, std::true_type(), std::false_type());
                    else ranks(mf, std::false_type(), std::false_type());
                } else if (dense_in) ranks(mf, std::true_type(), std::false_type());
                else ranks(mf, std::false_type(), std::false_type());
            }
            constexpr int MO = MF == 1 ? 1 : kOutRows, size = 64 * kWaves;
            if (!dense_out) adapters_out<T, MO, 0, false, false><<<out, size, 0, s>>>(a);
            else if (octs && a.R <= 32) adapters_out<T, MO, 1, true, true><<<out, size, 0, s>>>(a);
            else if (octs && a.R <= 64) adapters_out<T, MO, 2, true, true><<<out, size, 0, s>>>(a);
            else if (octs) adapters_out<T, MO, 0, true, true><<<out, size, 0, s>>>(a);
            else if (a.R <= 32) adapters_out<T, MO, 1, true, false><<<out, size, 0, s>>>(a);
            else adapters_out<T, MO, 0, true, false><<<out, size, 0, s>>>(a);
        };
        if (few) rows(std::integral_constant<int, 1>());
        else rows(std::integral_constant<int, 4>());
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
