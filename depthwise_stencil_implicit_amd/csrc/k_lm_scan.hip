// The selective state space scan, forward, and its step for single tokens:
//   d = softplus(dt + bias),  h[s] <- exp(d A[s]) h[s] + d x B[s],
//   y = (sum_s C[s] h[s] + D x) silu(z).
//
// The decay differs for every (step, channel, state), so there is no matrix
// product to hand to the matrix cores: the work is one exponential, two
// multiplications and two multiply-adds per (step, channel, state) on the
// vector unit, against 8 bytes (16-bit types) per (step, channel).
#include <hip/hip_runtime.h>

#include "lm_scan.h"

namespace miconv {
namespace {

// PRE: only the state that leaves a chunk entered with zero, and the chunk's
// sum of d (its decay is exp(A sum d)); the main pass folds them into the
// state its chunk starts from.
template <typename T, int NS, bool PRE> __global__ __launch_bounds__(256) void scan_fwd(const ScanP p)
{
    constexpr int CK = NS <= 4 ? 16 : 64 / NS;
    __shared__ float2 s_in[kTB][kCH];
    __shared__ __attribute__((aligned(16))) float s_bc[kTB * 8 * NS];
    __shared__ __attribute__((aligned(16))) float s_y[PRE ? 1 : kTB][kRow];

    const ScanAt at = scan_at(p, PRE ? p.chunks - 1 : p.chunks);
    if (PRE ? at.t0 + p.chunk >= at.sp.len : (at.t0 >= at.sp.len && at.ch > 0)) return;

    // Staging place: one row, eight channels.
    const int tr = threadIdx.x >> 3, tc = (threadIdx.x & 7) * 8;
    const int tn = at.nc - tc;
    const int64_t sc = at.c0 + tc;
    const auto row_of = [&](const void *base, const S3 &st) {
        return static_cast<const T *>(base) + at.sp.row0 * st.n + sc * st.c + (at.sp.start + tr) * st.l;
    };
    const T *px = row_of(p.x, p.xs), *pdt = row_of(p.dt, p.dts);
    const T *pz = p.z ? row_of(p.z, p.zs) : nullptr;
    T *py = p.y ? const_cast<T *>(row_of(p.y, p.ys)) : nullptr;
    float bias[8], D[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bias[i] = p.bias && i < tn ? p.bias[(sc + i) * p.bias_s] : 0.f;
        D[i] = p.D && i < tn ? p.D[(sc + i) * p.D_s] : 0.f;
    }

    // Core place: a quarter of one channel's states.
    const int lane = threadIdx.x & 63, q = lane & 3, c = (threadIdx.x >> 6) * 16 + (lane >> 2);
    const bool real = c < at.nc;
    const int64_t cc = at.c0 + c;
    float A2[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] = real && q * NS + i < p.S ? kLog2e * p.A[cc * p.A_c + (q * NS + i) * p.A_s] : 0.f, h[i] = 0.f;
    if (!PRE && real) {
        if (p.s0) get_states<NS>(p.s0, p.s0s, at.seq, cc, q * NS, p.S, h);
        for (int64_t j = 0; j < at.ch; ++j) {
            const int64_t k = (at.seq * (p.chunks - 1) + j) * p.C + cc;
            const float d = p.carry_d[k];
#pragma unroll
            for (int i = 0; i < NS; ++i)
                h[i] = __builtin_fmaf(hw_exp2(d * A2[i]), h[i], p.carry_h[(k * 4 + q) * NS + i]);
        }
    }
    float *saved = !PRE && p.saved && real ? p.saved + (saved_at<CK>(p, at) * p.C + cc) * 4 * NS + q * NS : nullptr;
    float sum_d = 0.f;

    Raw<T, 8> nx, ndt, nz;
    BcRegs<T, NS> bc;
    const auto fetch = [&](int64_t t) {
        if (t + tr < at.t1) {
            nx = get8(px + t * p.xs.l, p.xs.c, tn);
            ndt = get8(pdt + t * p.dts.l, p.dts.c, tn);
            if (!PRE && pz) nz = get8(pz + t * p.zs.l, p.zs.c, tn);
        } else {
            __builtin_memset(&nx, 0, sizeof(nx));
        }
        bc.fetch(p, at, t, at.t1);
    };
    fetch(at.t0);
    for (int64_t t = at.t0; t < at.t1; t += kTB) {
        const Raw<T, 8> x = nx, dt = ndt, z = nz;
        const bool row_in = t + tr < at.t1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float d = 0.f;
            if (row_in && i < tn) {
                d = to_f32(dt.v[i]) + bias[i];
                if (p.softplus) d = softplus(d);
            }
            s_in[tr][tc + i] = make_float2(d, d * to_f32(x.v[i]));
        }
        bc.put(s_bc);
        if (t + kTB < at.t1) fetch(t + kTB);
        __syncthreads();
        const int steps = at.t1 - t < kTB ? (int)(at.t1 - t) : kTB;
        for (int k = 0; k < steps; k += 4) {
            if (!PRE && saved && k % CK == 0) {
                float *o = saved + ((t + k) / CK) * p.C * 4 * NS;
#pragma unroll
                for (int i = 0; i < NS; ++i) o[i] = h[i];
            }
            float y4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = s_in[k + j][c];
                const float *row = s_bc + (k + j) * 8 * NS + q * NS;
                float b[NS], cv[NS];
                lds_states<NS>(row, b);
                if (!PRE) lds_states<NS>(row + 4 * NS, cv);
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const float a = hw_exp2(v.x * A2[i]);
                    h[i] = __builtin_fmaf(a, h[i], v.y * b[i]);
                    if (!PRE) y = __builtin_fmaf(cv[i], h[i], y);
                }
                y4[j] = y;
                if (PRE) sum_d += v.x;
            }
            if (!PRE) s_y[k + q][c] = quad_sum4(y4, q);
        }
        __syncthreads();
        if (!PRE && py && row_in) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = __builtin_fmaf(D[i], to_f32(x.v[i]), s_y[tr][tc + i]);
                if (pz) o[i] *= silu(to_f32(z.v[i]));
            }
            put8(py + t * p.ys.l, p.ys.c, tn, o);
        }
    }
    if (!real) return;
    if (PRE) {
        const int64_t k = (at.seq * (p.chunks - 1) + at.ch) * p.C + cc;
#pragma unroll
        for (int i = 0; i < NS; ++i) p.carry_h[(k * 4 + q) * NS + i] = h[i];
        if (q == 0) p.carry_d[k] = sum_d;
    } else if (p.s1 && at.t1 == at.sp.len) {
        put_states<NS>(p.s1, p.s1s, at.seq, cc, q * NS, p.S, h);
    }
}

// One token for each batch row; four lanes per (row, channel), the state is
// read and written once.
template <typename T, int NS> __global__ __launch_bounds__(256) void scan_step(const ScanP p)
{
    const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 2;
    const int q = threadIdx.x & 3;
    if (item >= p.seqs * p.C) return;   // the four lanes of an item leave together
    const int64_t n = item / p.C, c = item - n * p.C;
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
    get_states<NS>(p.s1, p.s1s, row, c, q * NS, p.S, h);
    const int64_t g = c / p.Cg;
    const T *pb = static_cast<const T *>(p.Bm) + n * p.Bs.n + g * p.Bs.g + q * NS * p.Bs.s;
    const T *pc = static_cast<const T *>(p.Cm) + n * p.Cs.n + g * p.Cs.g + q * NS * p.Cs.s;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const bool in = q * NS + i < p.S;
        A[i] = in ? p.A[c * p.A_c + (q * NS + i) * p.A_s] : 0.f;
        b[i] = in ? to_f32(pb[i * p.Bs.s]) : 0.f;
        cv[i] = in ? to_f32(pc[i * p.Cs.s]) : 0.f;
    }
    const float x = to_f32(static_cast<const T *>(p.x)[n * p.xs.n + c * p.xs.c]);
    float d = to_f32(static_cast<const T *>(p.dt)[n * p.dts.n + c * p.dts.c]);
    if (p.bias) d += p.bias[c * p.bias_s];
    if (p.softplus) d = softplus(d);
    const float dx = d * x, d2 = d * kLog2e;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        h[i] = __builtin_fmaf(hw_exp2(d2 * A[i]), h[i], dx * b[i]);
        o = __builtin_fmaf(cv[i], h[i], o);
    }
    put_states<NS>(p.s1, p.s1s, row, c, q * NS, p.S, h);
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
    a.carry_d = static_cast<float *>(ws);
    a.carry_h = a.carry_d + lm_cdiv(a.seqs * (a.chunks - 1) * a.C, 4) * 4;
    with_type(p.dtype, [&](auto t) {
        with_ns(p.S, [&](auto n) {
            typedef decltype(t) T;
            constexpr int NS = decltype(n)::value;
            if (a.chunks > 1) scan_fwd<T, NS, true><<<(int)(a.seqs * (a.chunks - 1) * a.blocks), 256, 0, s>>>(a);
            scan_fwd<T, NS, false><<<(int)(a.seqs * a.chunks * a.blocks), 256, 0, s>>>(a);
        });
    });
    return lm_launch_status();
}

int launch_lm_scan_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s)
{
    const ScanP a = scan_params(p, q);
    if (a.seqs == 0) return CONV_OK;
    with_type(p.dtype, [&](auto t) {
        with_ns(p.S, [&](auto n) {
            scan_step<decltype(t), decltype(n)::value><<<(int)lm_cdiv(a.seqs * a.C * 4, 256), 256, 0, s>>>(a);
        });
    });
    return lm_launch_status();
}

}  // namespace miconv
