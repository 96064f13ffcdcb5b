// Gradients of the selective scan.  With s = gy silu(z) and r[t] the gradient
// that reaches state h[t],
//   r[t] = C[t] s[t] + a[t+1] r[t+1],            a = exp(d A),
//   dC[t] = sum_c s h[t],   dB[t] = sum_c r d x,   dx = d sum_s r B + D s,
//   dd = sum_s r A (a h[t-1]) + x sum_s r B,      dA = sum_t r d (a h[t-1]),
// and dz = gy (sum_s C h + D x) silu'(z), ddt = dd softplus'.
//
// States come from the saved ones: CK steps are run forward again from a saved
// state, a and a h[t-1] stay in registers (2 CK NS = 128 values per lane), then
// the same steps are run in reverse.  Running the recurrence backwards instead
// (h[t-1] = (h[t] - d x B) / a) would divide by factors near zero.
//
// Sums over states cross four lanes; sums over channels (dB, dC) cross the
// sixteen channels of a wave by halving exchanges, then the four waves through
// LDS, and leave the workgroup as f32 parts that scan_bwd_bc adds in a fixed
// order, as scan_bwd_c does for dA, dD and the bias over the sequences.
#include <hip/hip_runtime.h>

#include "lm_scan.h"

namespace miconv {
namespace {

// Sum of two values over lane pairs 8 (4) apart inside a row of 16: lanes with
// bit 3 (2) clear receive the sum of a, the others that of b.  One asm block
// for two pairs, with the two wait states that a cross-lane read of a register
// needs after its last write by the vector unit.
__device__ __forceinline__ void halve8(float a0, float b0, float a1, float b1, float &r0, float &r1)
{
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %0, %2, %2 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %0, %3, %3 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %1, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xc"
        : "=&v"(r0), "=&v"(r1)
        : "v"(a0), "v"(b0), "v"(a1), "v"(b1));
}
__device__ __forceinline__ void halve4(float a0, float b0, float a1, float b1, float &r0, float &r1)
{
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %0, %2, %2 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
        "v_add_f32_dpp %0, %3, %3 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
        "v_add_f32_dpp %1, %4, %4 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
        "v_add_f32_dpp %1, %5, %5 row_shr:4 row_mask:0xf bank_mask:0xa"
        : "=&v"(r0), "=&v"(r1)
        : "v"(a0), "v"(b0), "v"(a1), "v"(b1));
}
// The same across rows: lanes of even (lower) rows receive the sum of a.
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
// Sums over the sixteen channels of a wave of eight values per lane: the lane
// receives that of v[4 bit4 + 2 bit2 + bit3] -- still to be added over bit 5.
__device__ __forceinline__ float halve_channels(const float (&v)[8])
{
    float r0, r1, r2, r3, z0, z1;
    halve8(v[0], v[1], v[2], v[3], r0, r1);
    halve8(v[4], v[5], v[6], v[7], r2, r3);
    halve4(r0, r1, r2, r3, z0, z1);
    return halve16(z0, z1);
}

// PRE: only the gradient that leaves a chunk at its front when none enters at
// its end, and the chunk's sum of d.
template <typename T, int NS, bool PRE> __global__ __launch_bounds__(256) void scan_bwd(const ScanP p)
{
    constexpr int CK = NS <= 4 ? 16 : 64 / NS;
    constexpr int NB = NS < 4 ? 4 : NS;      // states per lane in the exchanges
    __shared__ float2 s_in[kTB][kCH];        // d, d x
    __shared__ float s_s[kTB][kCH];          // s = gy silu(z)
    __shared__ __attribute__((aligned(16))) float s_bc[kTB * 8 * NS];
    __shared__ __attribute__((aligned(16))) float s_o[PRE ? 1 : 3][PRE ? 1 : kTB][kRow];   // sums over s of r B, r A a h, C h
    __shared__ float s_red[PRE ? 1 : 4][PRE ? 1 : kTB][8 * NS];

    const ScanAt at = scan_at(p, p.chunks);
    if (at.t0 >= at.sp.len && at.ch > 0) return;
    if (PRE && at.ch == 0) return;

    const int tr = threadIdx.x >> 3, tc = (threadIdx.x & 7) * 8;
    const int tn = at.nc - tc;
    const int64_t sc = at.c0 + tc;
    const auto row_of = [&](const void *base, const S3 &st) {
        return base ? static_cast<const T *>(base) + at.sp.row0 * st.n + sc * st.c + (at.sp.start + tr) * st.l : nullptr;
    };
    const T *px = row_of(p.x, p.xs), *pdt = row_of(p.dt, p.dts), *pz = row_of(p.z, p.zs), *pgy = row_of(p.gy, p.gys);
    float bias[8], D[8], sum_D[8] = {}, sum_b[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bias[i] = p.bias && i < tn ? p.bias[(sc + i) * p.bias_s] : 0.f;
        D[i] = p.D && i < tn ? p.D[(sc + i) * p.D_s] : 0.f;
    }

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane & 3, c = wave * 16 + (lane >> 2);
    const bool real = c < at.nc;
    const int64_t cc = at.c0 + c;
    float A[NS], dA[NS] = {}, r[NS] = {};    // r: the gradient that enters from the step behind
#pragma unroll
    for (int i = 0; i < NS; ++i) A[i] = real && q * NS + i < p.S ? p.A[cc * p.A_c + (q * NS + i) * p.A_s] : 0.f;
    if (!PRE && real) {
        if (p.gs) get_states<NS>(p.gs, p.gss, at.seq, cc, q * NS, p.S, r);
        int64_t last = (at.sp.len - 1) / p.chunk;
        if (last > p.chunks - 1) last = p.chunks - 1;
        for (int64_t j = last; j > at.ch; --j) {
            const int64_t k = (at.seq * p.chunks + j) * p.C + cc;
            const float d = p.carry_d[k] * kLog2e;
#pragma unroll
            for (int i = 0; i < NS; ++i)
                r[i] = __builtin_fmaf(hw_exp2(d * A[i]), r[i], p.carry_h[(k * 4 + q) * NS + i]);
        }
    }
    const float *saved = p.saved + (saved_at<CK>(p, at) * p.C + cc) * 4 * NS + q * NS;
    float sum_d = 0.f;

    Raw<T, 8> nx, ndt, nz, ng;
    BcRegs<T, NS> bc;
    float nh[kTB / CK][NS];
    const auto fetch = [&](int64_t t) {
        __builtin_memset(&nx, 0, sizeof(nx));
        __builtin_memset(&ndt, 0, sizeof(ndt));
        __builtin_memset(&nz, 0, sizeof(nz));
        __builtin_memset(&ng, 0, sizeof(ng));
        if (t + tr < at.t1) {
            nx = get8(px + t * p.xs.l, p.xs.c, tn);
            ndt = get8(pdt + t * p.dts.l, p.dts.c, tn);
            ng = get8(pgy + t * p.gys.l, p.gys.c, tn);
            if (pz) nz = get8(pz + t * p.zs.l, p.zs.c, tn);
        }
        bc.fetch(p, at, t, at.t1);
        if (!PRE) {
#pragma unroll
            for (int k = 0; k < kTB / CK; ++k)
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    nh[k][i] = real && t + k * CK < at.t1 ? saved[(t / CK + k) * p.C * 4 * NS + i] : 0.f;
        }
    };
    const int64_t tiles = (at.t1 - at.t0 + kTB - 1) / kTB;
    if (tiles > 0) fetch(at.t0 + (tiles - 1) * kTB);
    for (int64_t tile = tiles - 1; tile >= 0; --tile) {
        const int64_t t = at.t0 + tile * kTB;
        const Raw<T, 8> x = nx, dt = ndt, z = nz, gy = ng;
        float h0[kTB / CK][NS];
#pragma unroll
        for (int k = 0; k < kTB / CK; ++k)
#pragma unroll
            for (int i = 0; i < NS; ++i) h0[k][i] = nh[k][i];
        const bool row_in = t + tr < at.t1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float d = 0.f;
            if (row_in && i < tn) {
                d = to_f32(dt.v[i]) + bias[i];
                if (p.softplus) d = softplus(d);
            }
            s_in[tr][tc + i] = make_float2(d, d * to_f32(x.v[i]));
            float s = to_f32(gy.v[i]);
            if (pz) s *= silu(to_f32(z.v[i]));
            s_s[tr][tc + i] = s;
        }
        bc.put(s_bc);
        if (tile > 0) fetch(t - kTB);
        __syncthreads();
        if (PRE) {
            for (int k = kTB - 1; k >= 0; --k) {
                const float2 v = s_in[k][c];
                const float s = s_s[k][c], d2 = v.x * kLog2e;
                float cv[NS];
                lds_states<NS>(s_bc + k * 8 * NS + 4 * NS + q * NS, cv);
#pragma unroll
                for (int i = 0; i < NS; ++i) r[i] = hw_exp2(d2 * A[i]) * __builtin_fmaf(cv[i], s, r[i]);
                sum_d += v.x;
            }
        } else {
#pragma unroll
            for (int part = kTB / CK - 1; part >= 0; --part) {
                if (t + part * CK >= at.t1) continue;
                float a[CK][NS], u[CK][NS], h[NS];
#pragma unroll
                for (int i = 0; i < NS; ++i) h[i] = h0[part][i];
#pragma unroll
                for (int k = 0; k < CK; ++k) {
                    const float2 v = s_in[part * CK + k][c];
                    const float d2 = v.x * kLog2e;
                    float b[NS];
                    lds_states<NS>(s_bc + (part * CK + k) * 8 * NS + q * NS, b);
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        a[k][i] = hw_exp2(d2 * A[i]);
                        u[k][i] = a[k][i] * h[i];
                        h[i] = __builtin_fmaf(v.y, b[i], u[k][i]);
                    }
                }
                float o4[3][4], pair[NB / 4];
#pragma unroll
                for (int k = CK - 1; k >= 0; --k) {
                    const int row = part * CK + k;
                    const float2 v = s_in[row][c];
                    const float s = s_s[row][c];
                    float b[NS], cv[NS], vb[NB], vc[NB];
                    lds_states<NS>(s_bc + row * 8 * NS + q * NS, b);
                    lds_states<NS>(s_bc + row * 8 * NS + 4 * NS + q * NS, cv);
                    float rb = 0.f, ra = 0.f, ch = 0.f;
#pragma unroll
                    for (int i = 0; i < NB; ++i) vb[i] = vc[i] = 0.f;
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const float rr = __builtin_fmaf(cv[i], s, r[i]);
                        const float hh = __builtin_fmaf(v.y, b[i], u[k][i]);
                        vb[i] = rr * v.y;
                        vc[i] = s * hh;
                        rb = __builtin_fmaf(rr, b[i], rb);
                        ch = __builtin_fmaf(cv[i], hh, ch);
                        const float w = rr * u[k][i];
                        ra = __builtin_fmaf(w, A[i], ra);
                        dA[i] = __builtin_fmaf(w, v.x, dA[i]);
                        r[i] = a[k][i] * rr;
                    }
                    o4[0][k & 3] = rb, o4[1][k & 3] = ra, o4[2][k & 3] = ch;
                    if ((k & 3) == 0) {
#pragma unroll
                        for (int j = 0; j < 3; ++j) s_o[j][row + q][c] = quad_sum4(o4[j], q);
                    }
                    // dB and dC of two steps meet in the last exchange.
#pragma unroll
                    for (int m = 0; m < NB / 4; ++m) {
                        const float v8[8] = {vb[4 * m], vb[4 * m + 1], vb[4 * m + 2], vb[4 * m + 3],
                                             vc[4 * m], vc[4 * m + 1], vc[4 * m + 2], vc[4 * m + 3]};
                        const float got = halve_channels(v8);
                        if (k & 1) pair[m] = got;
                        else {
                            const float both = halve32(got, pair[m]);
                            const int i = 4 * m + ((lane >> 2) & 1) * 2 + ((lane >> 3) & 1);
                            if (i < NS)
                                s_red[wave][row + (lane >> 5)][((lane >> 4) & 1) * 4 * NS + q * NS + i] = both;
                        }
                    }
                }
            }
        }
        __syncthreads();
        if (PRE) continue;
        // The workgroup's parts of dB and dC.
        const int rows = at.t1 - t < kTB ? (int)(at.t1 - t) : kTB;
        float *part = p.part_bc + (((at.c0 - at.g * p.Cg) / kCH + at.g * p.blocks_g) * p.rows_total +
                                   at.sp.row0 * p.L + at.sp.start + t) * 8 * NS;
        for (int e = threadIdx.x; e < rows * 8 * NS; e += 256) {
            const int k = e / (8 * NS), j = e % (8 * NS);
            part[e] = (s_red[0][k][j] + s_red[1][k][j]) + (s_red[2][k][j] + s_red[3][k][j]);
        }
        if (row_in) {
            float ox[8], od[8], oz[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = s_in[tr][tc + i].x, s = s_s[tr][tc + i], xv = to_f32(x.v[i]);
                const float rb = s_o[0][tr][tc + i];
                ox[i] = __builtin_fmaf(D[i], s, d * rb);
                float dd = __builtin_fmaf(xv, rb, s_o[1][tr][tc + i]);
                if (p.softplus) dd *= sigmoid(to_f32(dt.v[i]) + bias[i]);
                od[i] = dd;
                sum_b[i] += dd;
                sum_D[i] = __builtin_fmaf(s, xv, sum_D[i]);
                const float zv = to_f32(z.v[i]);
                oz[i] = to_f32(gy.v[i]) * __builtin_fmaf(D[i], xv, s_o[2][tr][tc + i]) * silu_slope(zv, sigmoid(zv));
            }
            const auto put = [&](void *base, const S3 &st, const float (&v)[8]) {
                put8(static_cast<T *>(base) + at.sp.row0 * st.n + sc * st.c + (at.sp.start + t + tr) * st.l, st.c, tn, v);
            };
            put(p.dx, p.dxs, ox);
            put(p.ddt, p.ddts, od);
            if (pz) put(p.dz, p.dzs, oz);
        }
        // The next tile's staging overwrites s_in, s_s and s_bc only.
        __syncthreads();
    }
    if (PRE) {
        if (!real) return;
        const int64_t k = (at.seq * p.chunks + at.ch) * p.C + cc;
#pragma unroll
        for (int i = 0; i < NS; ++i) p.carry_h[(k * 4 + q) * NS + i] = r[i];
        if (q == 0) p.carry_d[k] = sum_d;
        return;
    }
    if (real && p.ds && at.ch == 0) put_states<NS>(p.ds, p.dss, at.seq, cc, q * NS, p.S, r);
    // Parts of dA (4 NS per channel), dD and the bias, laid out [part][channel][4 NS + 2].
    float *pc = p.part_c + ((at.seq * p.chunks + at.ch) * p.C + at.c0) * (4 * NS + 2);
    if (real) {
#pragma unroll
        for (int i = 0; i < NS; ++i) pc[c * (4 * NS + 2) + q * NS + i] = dA[i];
    }
    float (&sum)[kTB][kRow] = reinterpret_cast<float (&)[kTB][kRow]>(s_o[0]);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[tr][tc + i] = which ? sum_b[i] : sum_D[i];
        __syncthreads();
        if ((int)threadIdx.x < at.nc) {
            float v = 0.f;
            for (int k = 0; k < kTB; ++k) v += sum[k][threadIdx.x];
            pc[threadIdx.x * (4 * NS + 2) + 4 * NS + which] = v;
        }
    }
}

// dB and dC: the parts of a group's workgroups.  One thread per (row, kind, state).
template <typename T>
__global__ __launch_bounds__(256) void scan_bwd_bc(const float *part, int64_t rows, int64_t L, int64_t blocks_g, int G,
                                                   int S, int W, T *dB, S4 bs, T *dC, S4 cs)
{
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= rows * 2 * W * G) return;
    const int64_t per = rows * 2 * W, g = e / per, in = e - g * per, row = in / (2 * W);
    const int j = (int)(in - row * 2 * W), s = j % W;
    if (s >= S) return;
    const float *q = part + g * blocks_g * per + in;
    float a[4] = {};
    int64_t i = 0;
    for (; i + 4 <= blocks_g; i += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] += q[(i + k) * per];
    for (; i < blocks_g; ++i) a[0] += q[i * per];
    const T v = from_f32<T>((a[0] + a[1]) + (a[2] + a[3]));
    const int64_t n = row / L, l = row - n * L;
    if (j < W) dB[n * bs.n + g * bs.g + s * bs.s + l * bs.l] = v;
    else dC[n * cs.n + g * cs.g + s * cs.s + l * cs.l] = v;
}

// dA, dD and the bias's gradient: the parts of all sequences and chunks.  A
// part of an empty chunk was never written and is left out.
__global__ __launch_bounds__(256) void scan_bwd_c(const ScanP p, int W, float *dA, int64_t a_c, int64_t a_s, float *dD,
                                                  int64_t d_s, float *db, int64_t b_s)
{
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, n = p.C * (W + 2);
    if (e >= n) return;
    float v = 0.f;
    for (int64_t seq = 0; seq < p.seqs; ++seq) {
        const SeqSpan sp = seq_span(p.off, seq, p.L);
        for (int64_t ch = 0; ch < p.chunks && (ch == 0 || ch * p.chunk < sp.len); ++ch)
            v += p.part_c[(seq * p.chunks + ch) * n + e];
    }
    const int64_t c = e / (W + 2);
    const int j = (int)(e - c * (W + 2));
    if (j < p.S) dA[c * a_c + j * a_s] = v;
    else if (j == W && dD) dD[c * d_s] = v;
    else if (j == W + 1 && db) db[c * b_s] = v;
}

}  // namespace

int launch_lm_scan_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    ScanP a = scan_params(p, q);
    const int W = 4 * scan_ns(p.S);
    float *f = static_cast<float *>(ws);
    a.part_bc = f, f += a.blocks * a.rows_total * 2 * W;
    a.part_c = f, f += lm_cdiv(a.seqs * a.chunks * a.C * (W + 2), 4) * 4;
    a.carry_d = f, f += lm_cdiv(a.seqs * a.chunks * a.C, 4) * 4;
    a.carry_h = f;
    const int grid = (int)(a.seqs * a.chunks * a.blocks);
    with_type(p.dtype, [&](auto t) {
        typedef decltype(t) T;
        with_ns(p.S, [&](auto n) {
            constexpr int NS = decltype(n)::value;
            if (grid == 0) return;
            if (a.chunks > 1) scan_bwd<T, NS, true><<<grid, 256, 0, s>>>(a);
            scan_bwd<T, NS, false><<<grid, 256, 0, s>>>(a);
        });
        if (a.rows_total > 0) scan_bwd_bc<T><<<(int)lm_cdiv(a.rows_total * 2 * W * p.G, 256), 256, 0, s>>>(
            a.part_bc, a.rows_total, p.L, a.blocks_g, (int)p.G, (int)p.S, W, static_cast<T *>(q[LM_DB]),
            lm_s4(p.t[LM_DB]), static_cast<T *>(q[LM_DC]), lm_s4(p.t[LM_DC]));
    });
    scan_bwd_c<<<(int)lm_cdiv(p.C * (W + 2), 256), 256, 0, s>>>(
        a, W, static_cast<float *>(q[LM_DA]), p.t[LM_DA].strides[0], p.t[LM_DA].strides[1], static_cast<float *>(q[LM_DD]),
        p.t[LM_DD].strides[0], static_cast<float *>(q[LM_DDT_BIAS]), p.t[LM_DDT_BIAS].strides[0]);
    return lm_launch_status();
}

}  // namespace miconv
