// The selective state space scan, forward, and its step for single tokens:
//   d = softplus(dt + bias),  h[s] <- exp(d A[s]) h[s] + d x B[s],
//   y = (sum_s C[s] h[s] + D x) silu(z).
//
// The decay differs for every (step, channel, state), so there is no matrix
// product to hand to the matrix cores: the work is one exponential, two
// multiplications and two multiply-adds per (step, channel, state) on the
// vector unit, against 8 bytes (16-bit types) per (step, channel).  At the
// unit's issue rates (exponential 3.4 ns per wave and SIMD, row broadcasts 1.8,
// plain operations 1.1) that is 38 us for 8 x 1024 x 2048 channels of 16 states
// and 11 us for the parts per (step, channel); the memory's share is 26 us.
//
// Measured, bf16, 16 states: 8 x 1024 x 2048 in 76 us (one core wave per SIMD
// issues every 3 ns), 1 x 32768 x 1536 in 342 us, two fifths of them in the
// first pass over the chunks.  8 x 1024 x 2048 in f32 takes 87 us (bf16 with as
// many calls 83), with positions contiguous 111 to 114, of 32 states 127, of 64
// 250.
#include <hip/hip_runtime.h>

#include "lm_scan.h"

namespace miconv {
namespace {

constexpr int kTB = 32;              // steps of a tile: 8 channels of one row per staging thread

template <int NS, int QW, bool PRE> struct FwdLds {
    float2 in[2][kTB][kCH];                                          // d, d x
    __attribute__((aligned(16))) float bc[2][kTB * bc_row(4 * QW * NS)];
    __attribute__((aligned(16))) float y[PRE ? 1 : 2][PRE ? 1 : QW][kTB][kRow];
};

// The staging waves of one workgroup.
template <typename T, int NS, int QW, bool PRE, bool DENSE>
__device__ __forceinline__ void fwd_stage(const ScanP &p, const ScanAt &at, FwdLds<NS, QW, PRE> &sh, int tid)
{
    const int tr = tid >> 3, tc = (tid & 7) * 8;
    const int tn = at.nc - tc;
    const int64_t sc = at.c0 + tc;
    const int shift = DENSE && sc > p.C - 8 ? (int)(sc - (p.C - 8)) : 0;
    const bool any_shift = at.c0 + kCH > p.C;
    const auto row_of = [&](const void *base, const S3 &st) {
        return static_cast<const T *>(base) + at.sp.row0 * st.n + at.sp.start * st.l;
    };
    const T *px = row_of(p.x, p.xs), *pdt = row_of(p.dt, p.dts);
    const bool has_z = !PRE && p.z;
    const T *pz = has_z ? row_of(p.z, p.zs) : px;
    const S3 zs = has_z ? p.zs : p.xs;
    T *py = p.y ? const_cast<T *>(row_of(p.y, p.ys)) + sc * p.ys.c : nullptr;
    float bias[8], D[8];
    get_param<8>(p.bias, p.bias_s, sc, tn, bias);
    get_param<8>(p.D, p.D_s, sc, tn, D);
    Raw<T, 8> nx, ndt, nz, cx, cz, ox, oz;   // tile being loaded; in the core; leaving
    BcRegs<T, 4 * QW * NS, kTB, DENSE> bc(p, at, tid);
    const auto fetch = [&](int64_t t) {
        const int64_t l = t + tr < at.t1 ? t + tr : at.t1 - 1;
        nx = get_row<T, 8, DENSE>(px + l * p.xs.l, p.xs.c, sc, p.C);
        ndt = get_row<T, 8, DENSE>(pdt + l * p.dts.l, p.dts.c, sc, p.C);
        if (!PRE) nz = get_row<T, 8, DENSE>(pz + l * zs.l, zs.c, sc, p.C);
        bc.fetch(p, t, at.t1);
    };
    const auto stage = [&](int64_t t, int buf) {
        if (any_shift) {
            shift_row(nx, shift), shift_row(ndt, shift);
            if (!PRE) shift_row(nz, shift);
        }
        const bool row_in = t + tr < at.t1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float d = ndt.f(i) + bias[i];
            if (p.softplus) d = softplus(d);
            const bool in = row_in && i < tn;
            sh.in[buf][tr][tc + i] = make_float2(in ? d : 0.f, in ? d * nx.f(i) : 0.f);
        }
        bc.put(p, sh.bc[buf], t, at.t1);
    };
    const auto leave = [&](int64_t t, int buf) {
        if constexpr (!PRE) {
            if (!py || t + tr >= at.t1) return;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float y = sh.y[buf][0][tr][tc + i];
                if constexpr (QW == 2) y += sh.y[buf][1][tr][tc + i];
                o[i] = __builtin_fmaf(D[i], ox.f(i), y);
                if (has_z) o[i] *= silu(oz.f(i));
            }
            put_row<T, 8>(py + (t + tr) * p.ys.l, p.ys.c, tn, o);
        }
    };
    if (at.t0 < at.t1) {
        fetch(at.t0);
        stage(at.t0, 0);
        cx = nx, cz = nz;
        fetch(at.t0 + kTB);
    }
    lds_sync();
    int buf = 0;
    for (int64_t t = at.t0; t < at.t1; t += kTB, buf ^= 1) {
        // The core is at tile t in buf.
        stage(t + kTB, buf ^ 1);
        const Raw<T, 8> sx = nx, sz = nz;
        fetch(t + 2 * kTB);
        if (t > at.t0) leave(t - kTB, buf ^ 1);
        ox = cx, oz = cz, cx = sx, cz = sz;
        lds_sync();
    }
    if (at.t0 < at.t1) leave(at.t0 + (at.t1 - 1 - at.t0) / kTB * kTB, buf ^ 1);
}

// PRE: only the state that leaves a chunk entered with zero, and the chunk's
// sum of d (its decay is exp(A sum d)); the main pass folds them into the
// state its chunk starts from.
// Up to 16 states two workgroups fit a compute unit.
template <typename T, int NS, int QW, bool PRE, bool DENSE>
__global__ __launch_bounds__(256 * QW + kStage, DENSE && QW == 1 ? 4 : QW + 1) void scan_fwd(const ScanP p)
{
    constexpr int W = 4 * QW * NS, CK = ScanShape{NS, QW}.save_steps();
    __shared__ FwdLds<NS, QW, PRE> sh;
    const ScanAt at = scan_at(p, PRE ? p.chunks - 1 : p.chunks, p.chunks - 1);
    if (PRE ? at.t0 + p.chunk >= at.sp.len : (at.t0 >= at.sp.len && at.ch > 0)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= 4 * QW) {
        fwd_stage<T, NS, QW, PRE, DENSE>(p, at, sh, (int)threadIdx.x - 256 * QW);
        return;
    }

    // NS states of one channel: those of row q of its 4 QW.
    const int lane = threadIdx.x & 63, row = lane >> 4, half = wave >> 2, q = half * 4 + row,
              c = (wave & 3) * 16 + (lane & 15);
    const bool real = c < at.nc;
    const int64_t cc = at.c0 + c;
    float A2[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] = real && q * NS + i < p.S ? rate(p.A[cc * p.A_c + (q * NS + i) * p.A_s]) : 0.f, h[i] = 0.f;
    if (!PRE && real) {
        if (p.s0) get_states<NS>(p.s0, p.s0s, at.seq, cc, q * NS, p.S, h);
        fold_chunks<NS, W>(p, at.first, 1, at.ch, cc, q * NS, A2, h);
    }
    float *saved = !PRE && p.saved && real
                       ? p.saved + ((saved_at<CK>(p, at) + at.t0 / CK) * p.C + cc) * W + q * NS : nullptr;
    float sum_d = 0.f;
    lds_sync();
    int buf = 0;
    for (int64_t t = at.t0; t < at.t1; t += kTB, buf ^= 1) {
        const int steps = at.t1 - t < kTB ? (int)(at.t1 - t) : kTB;
        // Four steps at a time, their LDS reads one group ahead; steps past
        // the end have d = 0 and leave the state as it is.
        Steps4<NS, W, !PRE> g[2];
        g[0].load(sh.in[buf], sh.bc[buf], 0, c, q, lane);
        for (int k0 = 0; k0 < steps; k0 += 16) {
            each<4>([&](auto group) {
                constexpr int G = decltype(group)::value;
                const int k = k0 + 4 * G;
                const Steps4<NS, W, !PRE> &cur = g[G & 1];
                g[(G & 1) ^ 1].load(sh.in[buf], sh.bc[buf], (k + 4) % kTB, c, q, lane);
                // Without the barrier the reads sink to their uses.
                __builtin_amdgcn_sched_barrier(0);
                if (!PRE && 4 * G % CK == 0 && saved && k < steps) {
                    store_f32<float, NS>(saved, h);
                    saved += p.C * W;
                }
                float a[4][NS], hs[4][NS], y4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < NS; ++i) a[j][i] = hw_exp2(cur.v[j].x * A2[i]);
                each<4>([&](auto step) {
                    constexpr int j = decltype(step)::value;
                    y4[j] = 0.f;
                    each<NS>([&](auto state) {
                        constexpr int i = decltype(state)::value;
                        h[i] = __builtin_fmaf(a[j][i], h[i], cur.v[j].y * cur.b.template at<j, i>());
                        hs[j][i] = h[i];
                        if constexpr (!PRE && NS != 2 && NS != 4) y4[j] = __builtin_fmaf(cur.c.template at<j, i>(), h[i], y4[j]);
                    });
                    if (PRE) sum_d += cur.v[j].x;
                });
                if constexpr (!PRE && (NS == 2 || NS == 4)) dot4(cur.c.v[0], hs, y4);
                if constexpr (!PRE) sh.y[buf][half][k + row][c] = rows4(y4);
            });
        }
        lds_sync();
    }
    if (!real) return;
    if (PRE) {
        const int64_t k = (at.first + at.ch) * p.C + cc;
#pragma unroll
        for (int i = 0; i < NS; ++i) p.carry_h[k * W + q * NS + i] = h[i];
        if (q == 0) p.carry_d[k] = sum_d;
    } else if (p.s1 && at.t1 == at.sp.len) {
        put_states<NS>(p.s1, p.s1s, at.seq, cc, q * NS, p.S, h);
    }
}

template <int CTRL> __device__ __forceinline__ float quad(float v)
{
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// Sum over four neighbouring lanes.
__device__ __forceinline__ float quad_sum(float v)
{
    v += quad<0xB1>(v);        // lanes 1 0 3 2
    return v + quad<0x4E>(v);  // lanes 2 3 0 1
}

// One token for each batch row; four lanes per (row, channel), the state is
// read and written once.
template <typename T, int NS> __global__ __launch_bounds__(256) void scan_step(const ScanP p)
{
    const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 2;
    const int q = threadIdx.x & 3;
    if (item >= p.seqs * p.C) return;   // the four lanes of an item leave together
    int64_t c, in_g;
    const int64_t n = divide(item, p.C, c);
    T *y = static_cast<T *>(p.y) + n * p.ys.n + c * p.ys.c;
    int64_t row = n;
    if (p.rows) {
        row = p.rows[n];
        if (row < 0 || row >= p.state_rows) {
            if (q == 0) *y = from_f32<T>(0.f);
            return;
        }
    }
    float h[NS], A[NS], b[NS], cv[NS];
    const int64_t g = divide(c, p.Cg, in_g);
    const T *pb = static_cast<const T *>(p.Bm) + n * p.Bs.n + g * p.Bs.g + q * NS * p.Bs.s;
    const T *pc = static_cast<const T *>(p.Cm) + n * p.Cs.n + g * p.Cs.g + q * NS * p.Cs.s;
    float *ph = p.s1 + row * p.s1s.n + c * p.s1s.c + q * NS * p.s1s.l;
    const float *pA = p.A + c * p.A_c + q * NS * p.A_s;
    if (p.dense) {   // whole quarters of contiguous states: one access each
        load_f32<float, NS>(ph, h);
        load_f32<float, NS>(pA, A);
        load_f32<T, NS>(pb, b);
        load_f32<T, NS>(pc, cv);
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const bool in = q * NS + i < p.S;
            h[i] = in ? ph[i * p.s1s.l] : 0.f;
            A[i] = in ? pA[i * p.A_s] : 0.f;
            b[i] = in ? to_f32(pb[i * p.Bs.s]) : 0.f;
            cv[i] = in ? to_f32(pc[i * p.Cs.s]) : 0.f;
        }
    }
    const float x = to_f32(static_cast<const T *>(p.x)[n * p.xs.n + c * p.xs.c]);
    float d = to_f32(static_cast<const T *>(p.dt)[n * p.dts.n + c * p.dts.c]);
    if (p.bias) d += p.bias[c * p.bias_s];
    if (p.softplus) d = softplus(d);
    const float dx = d * x, d2 = d * kLog2e;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        // d = 0 leaves the state also where A is infinite (as rate() does).
        h[i] = __builtin_fmaf(hw_exp2(d2 != 0.f ? d2 * A[i] : 0.f), h[i], dx * b[i]);
        o = __builtin_fmaf(cv[i], h[i], o);
    }
    if (p.dense) store_f32<float, NS>(ph, h);
    else put_states<NS>(p.s1, p.s1s, row, c, q * NS, p.S, h);
    o = quad_sum(o);
    if (q) return;
    if (p.D) o = __builtin_fmaf(p.D[c * p.D_s], x, o);
    if (p.z) o *= silu(to_f32(static_cast<const T *>(p.z)[n * p.zs.n + c * p.zs.c]));
    *y = from_f32<T>(o);
}

}  // namespace

int launch_lm_scan(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    ScanP a = scan_params(p, q);
    if (a.seqs == 0) return CONV_OK;
    const bool dense = scan_dense(p, a, 8, scan_shape(p.S).width() / 4);
    a.carry_d = static_cast<float *>(ws);
    a.carry_h = a.carry_d + lm_cdiv(scan_carries(p) * a.C, 4) * 4;
    const int pre = (int)(scan_carries(p) * a.blocks), grid = (int)(lm_parts(p) * a.blocks);
    with_type(p.dtype, [&](auto t) {
        with_ns(p.S, [&](auto n, auto w) {
            typedef decltype(t) T;
            constexpr int NS = decltype(n)::value, QW = decltype(w)::value, threads = 256 * QW + kStage;
            if (dense) {
                if (pre) scan_fwd<T, NS, QW, true, true><<<pre, threads, 0, s>>>(a);
                scan_fwd<T, NS, QW, false, true><<<grid, threads, 0, s>>>(a);
            } else {
                if (pre) scan_fwd<T, NS, QW, true, false><<<pre, threads, 0, s>>>(a);
                scan_fwd<T, NS, QW, false, false><<<grid, threads, 0, s>>>(a);
            }
        });
    });
    return lm_launch_status();
}

int launch_lm_scan_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s)
{
    ScanP a = scan_params(p, q);
    if (a.seqs == 0) return CONV_OK;
    int ns = 1;
    while (4 * ns < p.S) ns *= 2;
    a.dense = p.S == 4 * ns && a.s1s.l == 1 && a.A_s == 1 && a.Bs.s == 1 && a.Cs.s == 1;
    with_type(p.dtype, [&](auto t) {
        typedef decltype(t) T;
        const int grid = (int)lm_cdiv(a.seqs * a.C * 4, 256);
        if (ns == 1) scan_step<T, 1><<<grid, 256, 0, s>>>(a);
        else if (ns == 2) scan_step<T, 2><<<grid, 256, 0, s>>>(a);
        else if (ns == 4) scan_step<T, 4><<<grid, 256, 0, s>>>(a);
        else if (ns == 8) scan_step<T, 8><<<grid, 256, 0, s>>>(a);
        else scan_step<T, 16><<<grid, 256, 0, s>>>(a);
    });
    return lm_launch_status();
}

}  // namespace miconv
