// What the scan's kernels share: parameters, the staged tile and cross-lane sums.
//
// A workgroup owns 64 channels of one group and walks along the sequence in
// tiles.  Its core waves run the recurrence: a row of 16 lanes holds NS states
// of 16 channels, a wave four such rows, and QW waves share the channels (S <=
// 4 QW NS = W; states past S have A = B = C = 0).  Up to 16 states one wave does;
// two waves with half the states each issue a tenth more instructions and took
// a tenth longer (97 for 87 us).
//
// B and C are the same for all channels, so a row loads 16 different values of
// its states with one LDS read and takes each by a row broadcast in the
// instruction that uses it; reading them to every lane kept LDS busy half the
// time.
//
// Four staging waves work a tile ahead of the core and one behind: they load a
// tile, put d = softplus(dt + dt_bias) and d x -- one transcendental chain per
// (step, channel), not one per lane -- and B and C in f32 into LDS, and take the
// core's sums out again through D, the gate and the stores.  x, dt and z cross
// from HBM once and stay in the staging waves' registers between the two.  With
// one kind of wave that did both in turn, a SIMD stood idle at every barrier
// and behind every store (twice the time).
#pragma once

#include <type_traits>
#include <utility>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {

struct S4 { int64_t n, g, s, l; };

struct ScanP {
    const void *x, *dt, *Bm, *Cm, *z, *gy;
    const float *A, *D, *bias, *s0, *gs;
    void *y, *dx, *ddt, *dz;
    float *s1, *saved, *ds;
    float *carry_h, *carry_d;        // per chunk: state or gradient leaving it, sum of d
    float *part_bc, *part_c;         // backward sums of a workgroup
    const int32_t *off, *rows;
    S3 xs, dts, zs, ys, gys, dxs, ddts, dzs;
    S4 Bs, Cs;
    S3 s0s, s1s, gss, dss;           // (sequence, channel, state)
    int64_t A_c, A_s, D_s, bias_s;
    int64_t seqs, C, L, S, chunk, chunks, Cg, blocks_g, blocks, rows_total, parts, state_rows;
    int softplus, dense, slots;
};

constexpr int kCH = LM_SCAN_CH;
constexpr int kStage = 256;          // staging threads, behind the core's
constexpr int kRow = kCH + 16;       // padded f32 row: four rows x 16 channels on 64 banks

// Loads of a staging thread never stand behind a branch: a register that two
// paths may have written is settled, and so waited for, where they meet, and
// the loads of a tile would go out one by one (they did: 2 us each).  Rows and
// channels past the end are clamped to the last ones instead, and masked when
// the values are used.
//
// V channels of one row from c0 on.  DENSE: channels are contiguous and the
// tensor has at least V of them; a group that would pass the end starts at
// C - V, and shift_row moves its channels into place.
template <typename T, int V, bool DENSE>
__device__ __forceinline__ Raw<T, V> get_row(const T *row, int64_t cs, int64_t c0, int64_t C)
{
    if constexpr (DENSE) return load_raw<T, V>(row + (c0 < C - V ? c0 : C - V));
    else {
        Raw<T, V> r;
        r.zero();
#pragma unroll
        for (int i = 0; i < V; ++i) r.set(i, row[(c0 + i < C ? c0 + i : C - 1) * cs]);
        return r;
    }
}
template <typename T, int V> __device__ __forceinline__ void shift_row(Raw<T, V> &r, int by)
{
    constexpr int n = Raw<T, V>::n, per = 4 / sizeof(T);   // words, elements of a word
    if (per == 2 && (by & 1)) {
#pragma unroll
        for (int i = 0; i < n; ++i) r.w[i] = r.w[i] >> 16 | (i + 1 < n ? r.w[i + 1] << 16 : 0);
    }
#pragma unroll
    for (int s = 1; s < n; s *= 2)
        if (by & s * per) {
#pragma unroll
            for (int i = 0; i < n; ++i) r.w[i] = i + s < n ? r.w[i + s] : 0;
        }
}
template <typename T, int V> __device__ __forceinline__ void put_row(T *p, int64_t cs, int n, const float (&v)[V])
{
    if (cs == 1 && n >= V) store_f32<T, V>(p, v);
    else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i * cs] = from_f32<T>(v[i]);
    }
}
// A log2(e), the decay's exponent per unit of d.  An infinite A stands at the
// largest number: exp2(d A2) keeps its limit 0 for any d that counts, and steps
// with d = 0 (those past the end among them) leave the state as it is, where 0
// times infinity would be NaN.
__device__ __forceinline__ float rate(float A)
{
    const float v = kLog2e * A;
    return __builtin_isinf(v) ? __builtin_copysignf(__FLT_MAX__, v) : v;
}
// V values per channel of an f32 parameter, zero without it or past the end.
template <int V> __device__ __forceinline__ void get_param(const float *p, int64_t st, int64_t c0, int n, float (&o)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = p && i < n ? p[(c0 + i) * st] : 0.f;
}

// Where a workgroup stands.
struct ScanAt {
    int64_t seq, ch, c0;     // sequence, chunk, first channel
    int64_t first, part;     // numbers of the sequence's first chunk and of this one among all
    int g, nc;               // group, channels of this workgroup
    SeqSpan sp;
    int64_t t0, t1;          // its steps of the sequence
};
// chunks: a sequence's workgroups of this launch per channel block; numbered: how
// many of its chunks have a number.  A place between packed sequences gets a
// chunk past its sequence's end.
__device__ __forceinline__ ScanAt scan_at(const ScanP &p, int64_t chunks, int64_t numbered)
{
    ScanAt a;
    // All of these are below 2^31.
    const uint32_t b = blockIdx.x, r = b / (uint32_t)p.blocks, cb = b - r * (uint32_t)p.blocks;
    a.part = r;
    // Out of the straight path (prompt of 8 x 1024 x 2048 x 16: 76.7 us in it, 75.7 out of it).
    if (__builtin_expect(p.slots, 0)) {
        int seq, first;
        a.sp = seq_of_slot(p.off, (int)p.seqs, (int)p.L, (uint32_t)p.chunk, (int)r, seq, first);
        a.seq = seq, a.first = first, a.ch = (int)r - first;
        if (a.ch < 0) a.sp.len = 0, a.ch = 1;   // in front of the first sequence
    } else {
        const uint32_t seq = r / (uint32_t)chunks;
        a.seq = seq, a.ch = r - seq * (uint32_t)chunks, a.first = seq * numbered;
        a.sp = seq_span(p.off, a.seq, p.L);
    }
    a.g = (int)(cb / (uint32_t)p.blocks_g);
    const int64_t in_g = (int64_t)(cb - a.g * (uint32_t)p.blocks_g) * kCH;
    a.c0 = a.g * p.Cg + in_g;
    a.nc = (int)(p.Cg - in_g < kCH ? p.Cg - in_g : kCH);
    a.t0 = a.ch * p.chunk;
    a.t1 = p.chunks == 1 || a.t0 + p.chunk > a.sp.len ? a.sp.len : a.t0 + p.chunk;
    return a;
}

// First saved state of a sequence.  ceil(len / CK) states follow it; packed
// sequences cannot meet since floor(start / CK) + s grows by at least that.
template <int CK> __device__ __forceinline__ int64_t saved_at(const ScanP &p, const ScanAt &a)
{
    return p.off ? a.sp.start / CK + a.seq : a.seq * ((p.L + CK - 1) / CK);
}

// Words of a step's B and C in LDS: the steps that a row broadcast gathers lie
// on different banks (8 x 1024 x 2048 channels of 16 states: 83 us of kernel,
// 84 with rows end to end).
constexpr int bc_row(int W) { return W <= 8 ? 2 * W : W == 16 ? 48 : W == 32 ? 80 : 160; }

// B and C of a tile on their way to LDS: threads 0 .. 127 hold n neighbouring
// states of one row of B, threads 128 .. 255 of C.  DENSE: states are
// contiguous and S a multiple of n.
template <typename T, int W, int TB, bool DENSE> struct BcRegs {
    static constexpr int n = TB * W / 128;
    Raw<T, n> v;
    const T *base;
    int64_t sl;
    int row, s0, to;
    __device__ __forceinline__ BcRegs(const ScanP &p, const ScanAt &a, int tid)
    {
        const int e = tid % 128 * n;
        const S4 &st = tid < 128 ? p.Bs : p.Cs;
        row = e / W, s0 = e % W;
        to = row * bc_row(W) + (tid < 128 ? 0 : W) + s0;
        base = static_cast<const T *>(tid < 128 ? p.Bm : p.Cm) + a.sp.row0 * st.n + a.g * st.g + a.sp.start * st.l;
        if (DENSE) base += s0 < p.S ? s0 : 0;
        sl = st.l;
    }
    __device__ __forceinline__ void fetch(const ScanP &p, int64_t t, int64_t t1)
    {
        const T *q = base + (t + row < t1 ? t + row : t1 - 1) * sl;
        if constexpr (DENSE) v = load_raw<T, n>(q);
        else {
            v.zero();
            const int64_t ss = threadIdx.x % kStage < 128 ? p.Bs.s : p.Cs.s;
#pragma unroll
            for (int i = 0; i < n; ++i) v.set(i, q[(s0 + i < p.S ? s0 + i : p.S - 1) * ss]);
        }
    }
    __device__ __forceinline__ void put(const ScanP &p, float *sh, int64_t t, int64_t t1) const   // [TB][2][W]
    {
#pragma unroll
        for (int i = 0; i < n; ++i) sh[to + i] = t + row < t1 && s0 + i < p.S ? v.f(i) : 0.f;
    }
};

// f(0) .. f(N-1) with constant arguments.
template <typename F, int... I> __device__ __forceinline__ void each(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F f) { each(f, std::make_integer_sequence<int, N>()); }

// Lane N of every row of 16 lanes, to all of them.
template <int N> __device__ __forceinline__ float row_bcast(float v)
{
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), 0x150 + N, 0xf, 0xf, true));
}

// A row's states of B or C for four steps: value j NS + i (step j, state i) in
// register / 16, lane % 16.
template <int NS, int W> struct States4 {
    static constexpr int n = NS < 4 ? 1 : NS / 4;
    float v[n];
    __device__ __forceinline__ void load(const float *bc, int lane)   // bc: the row's states of the first step
    {
#pragma unroll
        for (int m = 0; m < n; ++m) {
            const int f = (m * 16 + (lane & 15)) % (4 * NS);
            v[m] = bc[f / NS * bc_row(W) + f % NS];
        }
    }
    template <int J, int I> __device__ __forceinline__ float at() const
    {
        return row_bcast<(J * NS + I) % 16>(v[(J * NS + I) / 16]);
    }
};

// y[j] = sum_i C[j][i] h[j][i] of four steps and two states.  The compiler
// folds a row broadcast into a multiplication but not into a multiply-add.
// The s_nop gives c the two wait states that a cross-lane read needs, should
// it have been moved by the vector unit just before.
__device__ __forceinline__ void dot4(float c, const float (&h)[4][2], float (&y)[4])
{
    asm("s_nop 1\n\t"
        "v_mul_f32_dpp %0, %4, %5 row_newbcast:0 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %1, %4, %7 row_newbcast:2 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %2, %4, %9 row_newbcast:4 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %3, %4, %11 row_newbcast:6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %4, %6 row_newbcast:1 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %8 row_newbcast:3 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %10 row_newbcast:5 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %4, %12 row_newbcast:7 row_mask:0xf bank_mask:0xf"
        : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
        : "v"(c), "v"(h[0][0]), "v"(h[0][1]), "v"(h[1][0]), "v"(h[1][1]), "v"(h[2][0]), "v"(h[2][1]), "v"(h[3][0]),
          "v"(h[3][1]));
}

// The same for four states.
__device__ __forceinline__ void dot4(float c, const float (&h)[4][4], float (&y)[4])
{
    asm("s_nop 1\n\t"
        "v_mul_f32_dpp %0, %4, %5 row_newbcast:0 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %1, %4, %9 row_newbcast:4 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %2, %4, %13 row_newbcast:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %3, %4, %17 row_newbcast:12 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %4, %6 row_newbcast:1 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %10 row_newbcast:5 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %14 row_newbcast:9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %4, %18 row_newbcast:13 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %4, %7 row_newbcast:2 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %11 row_newbcast:6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %15 row_newbcast:10 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %4, %19 row_newbcast:14 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %4, %8 row_newbcast:3 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %12 row_newbcast:7 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %16 row_newbcast:11 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %4, %20 row_newbcast:15 row_mask:0xf bank_mask:0xf"
        : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
        : "v"(c), "v"(h[0][0]), "v"(h[0][1]), "v"(h[0][2]), "v"(h[0][3]), 
          "v"(h[1][0]), "v"(h[1][1]), "v"(h[1][2]), "v"(h[1][3]), "v"(h[2][0]), "v"(h[2][1]), "v"(h[2][2]), "v"(h[2][3]), 
          "v"(h[3][0]), "v"(h[3][1]), "v"(h[3][2]), "v"(h[3][3]));
}

// One step of the backward recurrence for two states: r[i] += C[J][i] s,
// ch = sum_i C[J][i] h[i], rb = sum_i B[J][i] r[i] (the new r).
template <int J>
__device__ __forceinline__ void back(float c, float b, float s, const float (&h)[2], float (&r)[2], float &ch, float &rb)
{
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %4, %6 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %6 row_newbcast:%10 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %2, %4, %7 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %3, %5, %0 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %8 row_newbcast:%10 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %5, %1 row_newbcast:%10 row_mask:0xf bank_mask:0xf"
        : "+&v"(r[0]), "+&v"(r[1]), "=&v"(ch), "=&v"(rb)
        : "v"(c), "v"(b), "v"(s), "v"(h[0]), "v"(h[1]), "n"(2 * J), "n"(2 * J + 1));
}

// The same for four states.
template <int J>
__device__ __forceinline__ void back(float c, float b, float s, const float (&h)[4], float (&r)[4], float &ch, float &rb)
{
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %6, %8 row_newbcast:%13 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %6, %8 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %6, %8 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %6, %8 row_newbcast:%16 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %4, %6, %9 row_newbcast:%13 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32_dpp %5, %7, %0 row_newbcast:%13 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %4, %6, %10 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %5, %7, %1 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %4, %6, %11 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %5, %7, %2 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %4, %6, %12 row_newbcast:%16 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %5, %7, %3 row_newbcast:%16 row_mask:0xf bank_mask:0xf"
        : "+&v"(r[0]), "+&v"(r[1]), "+&v"(r[2]), "+&v"(r[3]), "=&v"(ch), "=&v"(rb)
        : "v"(c), "v"(b), "v"(s), "v"(h[0]), "v"(h[1]), "v"(h[2]), "v"(h[3]), "n"(4 * J), "n"(4 * J + 1),
          "n"(4 * J + 2), "n"(4 * J + 3));
}

// What a lane reads from LDS for four steps: d and d x of its channel, B and
// (WITH_C) C of its row.
template <int NS, int W, bool WITH_C> struct Steps4 {
    float2 v[4];
    States4<NS, W> b, c;
    __device__ __forceinline__ void load(const float2 (*in)[kCH], const float *bc, int k, int ch, int q, int lane)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = in[k + j][ch];
        b.load(bc + k * bc_row(W) + q * NS, lane);
        if constexpr (WITH_C) c.load(bc + k * bc_row(W) + W + q * NS, lane);
    }
};

// A lane's NS states of channel c in [row, channel, state] memory at any
// strides; states past S are zero.
template <int NS>
__device__ __forceinline__ void get_states(const float *p, const S3 &st, int64_t row, int64_t c, int s0, int64_t S,
                                           float (&h)[NS])
{
    const float *q = p + row * st.n + c * st.c + s0 * st.l;
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = s0 + i < S ? q[i * st.l] : 0.f;
}
template <int NS>
__device__ __forceinline__ void put_states(float *p, const S3 &st, int64_t row, int64_t c, int s0, int64_t S,
                                           const float (&h)[NS])
{
    float *q = p + row * st.n + c * st.c + s0 * st.l;
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (s0 + i < S) q[i * st.l] = h[i];
}

// What enters a chunk: v <- exp(A d[k]) v + left[k] over `count` chunks from
// `first` on, `by` chunks apart, d and left as the pass before stored them.
// Eight chunks' loads are in flight together.
template <int NS, int W>
__device__ __forceinline__ void fold_chunks(const ScanP &p, int64_t first, int64_t by, int64_t count, int64_t c, int s0,
                                            const float (&A2)[NS], float (&v)[NS])
{
    for (int64_t j0 = 0; j0 < count; j0 += 8) {
        float d[8], left[8][NS];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t k = (first + (j0 + j < count ? j0 + j : count - 1) * by) * p.C + c;
            d[j] = p.carry_d[k];
            load_f32<float, NS>(p.carry_h + k * W + s0, left[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j0 + j >= count) break;
#pragma unroll
            for (int i = 0; i < NS; ++i) v[i] = __builtin_fmaf(hw_exp2(d[j] * A2[i]), v[i], left[j][i]);
        }
    }
}

// Sums of lane pairs 16 (32) apart: lanes of even rows (of the lower half)
// receive that of a, the others that of b.
__device__ __forceinline__ float halve16(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float halve32(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sums over a wave's four rows of four values; row r receives that of v[r].
__device__ __forceinline__ float rows4(const float (&v)[4])
{
    return halve32(halve16(v[0], v[1]), halve16(v[2], v[3]));
}

inline S3 lm_s3(const conv_tensor &t) { return {t.strides[0], t.strides[1], t.rank > 2 ? t.strides[2] : 0}; }
inline S4 lm_s4(const conv_tensor &t) { return {t.strides[0], t.strides[1], t.strides[2], t.rank > 3 ? t.strides[3] : 0}; }

inline ScanP scan_params(const lm_plan_t &p, lm_ptrs q)
{
    const auto f = [&](int s) { return static_cast<float *>(q[s]); };
    ScanP a = {};
    a.x = q[LM_X], a.dt = q[LM_DT], a.Bm = q[LM_B], a.Cm = q[LM_C], a.z = q[LM_Z], a.gy = q[LM_GY];
    a.A = f(LM_A), a.D = f(LM_D), a.bias = f(LM_DT_BIAS), a.s0 = f(LM_STATE_IN), a.gs = f(LM_GSTATE);
    a.y = q[LM_Y], a.dx = q[LM_DX], a.ddt = q[LM_DDT], a.dz = q[LM_DZ];
    a.s1 = f(LM_STATE_OUT), a.saved = f(LM_SAVED), a.ds = f(LM_DSTATE);
    a.off = static_cast<const int32_t *>(q[LM_OFFSETS]), a.rows = static_cast<const int32_t *>(q[LM_ROWS]);
    a.xs = lm_s3(p.t[LM_X]), a.dts = lm_s3(p.t[LM_DT]), a.zs = lm_s3(p.t[LM_Z]), a.ys = lm_s3(p.t[LM_Y]);
    a.gys = lm_s3(p.t[LM_GY]), a.dxs = lm_s3(p.t[LM_DX]), a.ddts = lm_s3(p.t[LM_DDT]), a.dzs = lm_s3(p.t[LM_DZ]);
    a.Bs = lm_s4(p.t[LM_B]), a.Cs = lm_s4(p.t[LM_C]);
    a.s0s = lm_s3(p.t[LM_STATE_IN]), a.s1s = lm_s3(p.t[LM_STATE_OUT]);
    a.gss = lm_s3(p.t[LM_GSTATE]), a.dss = lm_s3(p.t[LM_DSTATE]);
    a.A_c = p.t[LM_A].strides[0], a.A_s = p.t[LM_A].strides[1];
    a.D_s = p.t[LM_D].strides[0], a.bias_s = p.t[LM_DT_BIAS].strides[0];
    a.seqs = p.seqs, a.C = p.C, a.L = p.L, a.S = p.S, a.chunk = p.chunk, a.chunks = p.chunks;
    a.Cg = p.C / p.G;
    a.blocks_g = lm_cdiv(a.Cg, LM_SCAN_CH);
    a.blocks = a.blocks_g * p.G;
    a.rows_total = p.t[LM_X].sizes[0] * p.L;
    a.state_rows = p.t[LM_STATE_OUT].sizes[0];
    a.parts = lm_parts(p), a.slots = lm_slots(p);
    a.softplus = (p.args.flags & LM_SOFTPLUS) != 0;
    return a;
}

// Whether the staging waves may load V channels and n states at once.
inline bool scan_dense(const lm_plan_t &p, const ScanP &a, int V, int n)
{
    for (int s : {LM_X, LM_DT, LM_Z, LM_GY})
        if (p.t[s].rank && p.t[s].strides[1] != 1 && p.C > 1) return false;
    return p.C >= V && p.S % n == 0 && (a.Bs.s == 1 || p.S == 1) && (a.Cs.s == 1 || p.S == 1);
}

// f(T) for the element type, f(NS) for the states per lane.
template <typename F> void with_type(int32_t dtype, F f)
{
    if (dtype == CONV_F32) f(float());
    else if (dtype == CONV_F16) f(f16_t());
    else f(bf16_t());
}
template <typename F> void with_ns(int64_t S, F f)
{
    const ScanShape s = scan_shape(S);
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    if (s.qw == 2 && s.ns == 8) f(std::integral_constant<int, 8>(), two);
    else if (s.qw == 2) f(four, two);
    else if (s.ns == 4) f(four, one);
    else if (s.ns == 2) f(two, one);
    else f(one, one);
}

}  // namespace miconv
