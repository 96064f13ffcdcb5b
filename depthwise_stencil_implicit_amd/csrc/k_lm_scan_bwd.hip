// Gradients of the selective scan.  With s = gy silu(z) and r[t] the gradient
// that reaches state h[t],
//   r[t] = C[t] s[t] + a[t+1] r[t+1],            a = exp(d A),
//   dC[t] = sum_c s h[t],   dB[t] = sum_c r d x,   dx = d sum_s r B + D s,
//   dd = sum_s r A (a h[t-1]) + x sum_s r B,      dA = sum_t r d (a h[t-1]),
// and dz = gy (sum_s C h + D x) silu'(z), ddt = dd softplus'.
//
// States come from the saved ones: CK steps are run forward again from a saved
// state, a and h[t-1] stay in registers (2 CK NS = 128 values per lane, 64 above
// 16 states), then the same steps are run in reverse.  Running the recurrence
// backwards instead (h[t-1] = (h[t] - d x B) / a) would divide by factors near
// zero.  Above 32 states 52 of a lane's registers do not fit and spill, in the
// kernels for other layouts 6 to 58 (f32 and up to 16 states most).
//
// Sums over states cross the four rows of a wave; sums over channels (dB, dC)
// cross a row's sixteen channels by halving exchanges, then the four waves
// through LDS, and leave the workgroup as f32 parts that scan_bwd_bc adds in a
// fixed order, as scan_bwd_c does for dA, dD and the bias over the sequences.
//
// Bound by vector issue, 73 instructions per step and wave (20 for the forward
// steps, 36 for the reverse ones, 17 for the exchanges), and some 85 scalar
// registers kept in vector lanes.  Measured, bf16, 8 x 2048 x 2048 channels of 16
// states: 447 us, and 13 for scan_bwd_bc.  8 x 1024 x 2048 with its forward call:
// 16 states 314 us (f32 329, positions contiguous 418 and 605), 32 states 489, 64
// states 1890.
#include <hip/hip_runtime.h>

#include "lm_scan.h"

namespace miconv {
namespace {

// Sums of eight values over the four channels of a row of 16 lanes, halving
// the values with the lanes: over lanes 8 apart, where lanes with bit 3 clear
// keep the even values' sums, then 4 apart likewise by bit 2.  The lane
// receives z0 = sum of v[2 bit2 + bit3], z1 = sum of v[4 + 2 bit2 + bit3].
// One asm block: a cross-lane read of a register needs two wait states after
// its last write by the vector unit; the s_nop gives them to the inputs, two
// instructions in between give them to each intermediate.
__device__ __forceinline__ void halve_row(const float (&v)[8], float &z0, float &z1)
{
    float r0, r1, r2, r3;
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %3, %8, %8 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %4, %10, %10 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %5, %12, %12 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %2, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %3, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %4, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %5, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %0, %2, %2 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
        "v_add_f32_dpp %0, %3, %3 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
        "v_add_f32_dpp %1, %4, %4 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
        "v_add_f32_dpp %1, %5, %5 row_shr:4 row_mask:0xf bank_mask:0xa"
        : "=&v"(z0), "=&v"(z1), "=&v"(r0), "=&v"(r1), "=&v"(r2), "=&v"(r3)
        : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]));
}
// The same over lanes 2 and 1 apart, by selection.
__device__ __forceinline__ float halve_quad(float a, float b, bool second, bool pairs)
{
    const auto across = [&](float v) {
        const uint32_t u = __float_as_uint(v);
        return __uint_as_float(pairs ? __builtin_amdgcn_mov_dpp(u, 0x4E, 0xf, 0xf, true)     // lanes 2 3 0 1
                                     : __builtin_amdgcn_mov_dpp(u, 0xB1, 0xf, 0xf, true));   // lanes 1 0 3 2
    };
    const float sa = a + across(a), sb = b + across(b);
    return second ? sb : sa;
}

// Steps of a tile: LDS holds two of them, and its 128 threads of B take whole
// states.
constexpr int bwd_tile(int W) { return W <= 16 ? 32 : W <= 32 ? 16 : 8; }

template <int NS, int QW, bool PRE> struct BwdLds {
    static constexpr int W = 4 * QW * NS, TB = bwd_tile(W);
    float2 in[2][TB][kCH];                                         // d, d x
    float s[2][TB][kCH];                                           // gy silu(z)
    __attribute__((aligned(16))) float bc[2][TB * bc_row(W)];
    // Sums over s of r B, r A a h, C h.
    __attribute__((aligned(16))) float o[PRE ? 1 : 2][3][PRE ? 1 : QW][PRE ? 1 : TB][kRow];
    float red[PRE ? 1 : 2][4][PRE ? 1 : TB][2 * W];                // dB, dC of 16 channels
};

// The staging waves: tiles in descending order.
template <typename T, int NS, int QW, bool PRE, bool DENSE>
__device__ __forceinline__ void bwd_stage(const ScanP &p, const ScanAt &at, BwdLds<NS, QW, PRE> &sh, int tid)
{
    constexpr int W = 4 * QW * NS, TB = bwd_tile(W), V = TB / 4;
    const int tr = tid / (256 / TB), tc = tid % (256 / TB) * V;
    const int tn = at.nc - tc;
    const int64_t sc = at.c0 + tc;
    const int shift = DENSE && sc > p.C - V ? (int)(sc - (p.C - V)) : 0;
    const bool any_shift = at.c0 + kCH > p.C, has_z = p.z != nullptr;
    const auto row_of = [&](const void *base, const S3 &st) {
        return static_cast<const T *>(base) + at.sp.row0 * st.n + at.sp.start * st.l;
    };
    const T *px = row_of(p.x, p.xs), *pdt = row_of(p.dt, p.dts), *pgy = row_of(p.gy, p.gys);
    const T *pz = has_z ? row_of(p.z, p.zs) : px;
    const S3 zs = has_z ? p.zs : p.xs;
    float bias[V], D[V], sum_D[V] = {}, sum_b[V] = {};
    get_param<V>(p.bias, p.bias_s, sc, tn, bias);
    get_param<V>(p.D, p.D_s, sc, tn, D);
    struct Tile { Raw<T, V> x, dt, z, gy; } nt, ct, ot;   // being loaded; in the core; leaving
    BcRegs<T, W, TB, DENSE> bc(p, at, tid);
    const auto fetch = [&](int64_t t) {
        int64_t l = t + tr < at.t1 ? t + tr : at.t1 - 1;
        if (l < at.t0) l = at.t0;   // before the chunk: loaded for nothing
        nt.x = get_row<T, V, DENSE>(px + l * p.xs.l, p.xs.c, sc, p.C);
        nt.dt = get_row<T, V, DENSE>(pdt + l * p.dts.l, p.dts.c, sc, p.C);
        nt.gy = get_row<T, V, DENSE>(pgy + l * p.gys.l, p.gys.c, sc, p.C);
        nt.z = get_row<T, V, DENSE>(pz + l * zs.l, zs.c, sc, p.C);
        bc.fetch(p, t < at.t0 ? at.t0 : t, at.t1);
    };
    const auto stage = [&](int64_t t, int buf) {
        if (any_shift) shift_row(nt.x, shift), shift_row(nt.dt, shift), shift_row(nt.gy, shift), shift_row(nt.z, shift);
        const bool row_in = t + tr < at.t1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float d = nt.dt.f(i) + bias[i];
            if (p.softplus) d = softplus(d);
            const bool in = row_in && i < tn;
            sh.in[buf][tr][tc + i] = make_float2(in ? d : 0.f, in ? d * nt.x.f(i) : 0.f);
            float s = nt.gy.f(i);
            if (has_z) s *= silu(nt.z.f(i));
            sh.s[buf][tr][tc + i] = in ? s : 0.f;
        }
        bc.put(p, sh.bc[buf], t, at.t1);
    };
    const auto leave = [&](int64_t t, int buf) {
        if constexpr (!PRE) {
            const int rows = at.t1 - t < TB ? (int)(at.t1 - t) : TB;
            float *part = p.part_bc + (((at.c0 - at.g * p.Cg) / kCH + at.g * p.blocks_g) * p.rows_total +
                                       at.sp.row0 * p.L + at.sp.start + t) * 2 * W;
            const float *red = &sh.red[buf][0][0][0];
            constexpr int n = TB * 2 * W;
            for (int e = tid; e < rows * 2 * W; e += kStage)
                part[e] = (red[e] + red[n + e]) + (red[2 * n + e] + red[3 * n + e]);
            if (t + tr >= at.t1) return;
            const auto sum = [&](int which, int i) {
                float v = sh.o[buf][which][0][tr][tc + i];
                if constexpr (QW == 2) v += sh.o[buf][which][1][tr][tc + i];
                return v;
            };
            float ox[V], od[V], oz[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xv = ot.x.f(i), g = ot.gy.f(i), raw = ot.dt.f(i) + bias[i];
                const float d = p.softplus ? softplus(raw) : raw;
                float s = g;
                if (has_z) {
                    const float zv = ot.z.f(i), qz = sigmoid(zv);
                    s *= zv * qz;
                    oz[i] = g * __builtin_fmaf(D[i], xv, sum(2, i)) * silu_slope(zv, qz);
                }
                const float rb = sum(0, i);
                ox[i] = __builtin_fmaf(D[i], s, d * rb);
                float dd = __builtin_fmaf(kLn2, sum(1, i), xv * rb);   // summed with A log2(e)
                if (p.softplus) dd *= sigmoid(raw);
                od[i] = dd;
                sum_b[i] += i < tn ? dd : 0.f;
                sum_D[i] += i < tn ? s * xv : 0.f;
            }
            const auto put = [&](void *base, const S3 &st, const float (&v)[V]) {
                put_row<T, V>(static_cast<T *>(base) + at.sp.row0 * st.n + sc * st.c + (at.sp.start + t + tr) * st.l, st.c, tn,
                              v);
            };
            put(p.dx, p.dxs, ox);
            put(p.ddt, p.ddts, od);
            if (has_z) put(p.dz, p.dzs, oz);
        }
    };
    const int tiles = (int)((at.t1 - at.t0 + TB - 1) / TB);
    const auto at_tile = [&](int k) { return at.t0 + (int64_t)k * TB; };
    if (tiles > 0) {
        fetch(at_tile(tiles - 1));
        stage(at_tile(tiles - 1), 0);
        ct = nt;
        fetch(at_tile(tiles - 2));
    }
    lds_sync();
    int buf = 0;
    for (int k = tiles - 1; k >= 0; --k, buf ^= 1) {
        // The core is at tile k in buf.
        if (k > 0) stage(at_tile(k - 1), buf ^ 1);
        const Tile st = nt;
        fetch(at_tile(k - 2));
        if (k < tiles - 1) leave(at_tile(k + 1), buf ^ 1);
        ot = ct, ct = st;
        lds_sync();
    }
    if (tiles > 0) leave(at_tile(0), buf ^ 1);
    if constexpr (!PRE) {
        // Sums of D's and the bias's gradients over the rows of the staging waves.
        float(*sum)[kRow] = sh.o[0][0][0];
        float *pc = p.part_c + (at.part * p.C + at.c0) * (W + 2);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            lds_sync();
#pragma unroll
            for (int i = 0; i < V; ++i) sum[tr][tc + i] = which ? sum_b[i] : sum_D[i];
            lds_sync();
            if (tid < at.nc) {
                float v = 0.f;
                for (int k = 0; k < TB; ++k) v += sum[k][tid];
                pc[tid * (W + 2) + W + which] = v;
            }
        }
    }
}

// PRE: only the gradient that leaves a chunk at its front when none enters at
// its end, and the chunk's sum of d.
template <typename T, int NS, int QW, bool PRE, bool DENSE>
__global__ __launch_bounds__(256 * QW + kStage) void scan_bwd(const ScanP p)
{
    constexpr int W = 4 * QW * NS, CK = ScanShape{NS, QW}.save_steps(), TB = bwd_tile(W), PARTS = TB / CK;
    __shared__ BwdLds<NS, QW, PRE> sh;
    const ScanAt at = scan_at(p, p.chunks, p.chunks);
    if (at.t0 >= at.sp.len && at.ch > 0) {
        if (!PRE)   // a place without a chunk adds nothing to the sums
            for (int e = threadIdx.x; e < at.nc * (W + 2); e += blockDim.x) p.part_c[(at.part * p.C + at.c0) * (W + 2) + e] = 0.f;
        return;
    }
    if (PRE && at.ch == 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= 4 * QW) {
        bwd_stage<T, NS, QW, PRE, DENSE>(p, at, sh, (int)threadIdx.x - 256 * QW);
        return;
    }

    const int lane = threadIdx.x & 63, lrow = lane >> 4, half = wave >> 2, q = half * 4 + lrow,
              c = (wave & 3) * 16 + (lane & 15);
    const bool real = c < at.nc;
    const int64_t cc = at.c0 + c;
    float A2[NS], dA[NS] = {}, r[NS] = {};   // A log2(e); r: the gradient that enters from the step behind
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] = real && q * NS + i < p.S ? rate(p.A[cc * p.A_c + (q * NS + i) * p.A_s]) : 0.f;
    if (!PRE && real) {
        if (p.gs) get_states<NS>(p.gs, p.gss, at.seq, cc, q * NS, p.S, r);
        const int64_t last = p.chunks == 1 ? 0 : chunks_of(at.sp.len, p.chunk) - 1;
        if (last > at.ch) fold_chunks<NS, W>(p, at.first + last, -1, last - at.ch, cc, q * NS, A2, r);
    }
    const float *saved = p.saved + ((saved_at<CK>(p, at) + at.t0 / CK) * p.C + cc) * W + q * NS;
    float sum_d = 0.f;
    const int tiles = (int)((at.t1 - at.t0 + TB - 1) / TB);
    float nh[PARTS][NS] = {};                // states saved in a tile, loaded a tile ahead
    const auto fetch = [&](int k) {
        if (PRE || k < 0) return;
#pragma unroll
        for (int j = 0; j < PARTS; ++j) {
            if (real && at.t0 + (int64_t)k * TB + j * CK < at.t1)
                load_f32<float, NS>(saved + ((int64_t)k * PARTS + j) * p.C * W, nh[j]);
        }
    };
    fetch(tiles - 1);
    lds_sync();
    int buf = 0;
    for (int tile = tiles - 1; tile >= 0; --tile, buf ^= 1) {
        const int64_t t = at.t0 + (int64_t)tile * TB;
        const float2(*in)[kCH] = sh.in[buf];
        const float(*ss)[kCH] = sh.s[buf];
        const float *bc = sh.bc[buf];
        if constexpr (PRE) {
            for (int k0 = TB - 4; k0 >= 0; k0 -= 4) {
                States4<NS, W> cs;
                cs.load(bc + k0 * bc_row(W) + W + q * NS, lane);
                each<4>([&](auto step) {
                    constexpr int j = 3 - decltype(step)::value;
                    const float d = in[k0 + j][c].x, s = ss[k0 + j][c];
                    each<NS>([&](auto state) {
                        constexpr int i = decltype(state)::value;
                        r[i] = hw_exp2(d * A2[i]) * __builtin_fmaf(cs.template at<j, i>(), s, r[i]);
                    });
                    sum_d += d;
                });
            }
        } else {
            float h0[PARTS][NS];
#pragma unroll
            for (int j = 0; j < PARTS; ++j)
#pragma unroll
                for (int i = 0; i < NS; ++i) h0[j][i] = nh[j][i];
            fetch(tile - 1);
#pragma unroll 1
            for (int part = PARTS - 1; part >= 0; --part) {
                if (t + part * CK >= at.t1) continue;
                const int row0 = part * CK;
                float a[CK][NS], h[CK + 1][NS];   // h[k]: the state before step k
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    h[0][i] = h0[0][i];
#pragma unroll
                    for (int j = 1; j < PARTS; ++j) h[0][i] = part == j ? h0[j][i] : h[0][i];
                }
                each<CK / 4>([&](auto group) {
                    constexpr int k0 = 4 * decltype(group)::value;
                    Steps4<NS, W, false> g;
                    g.load(in, bc, row0 + k0, c, q, lane);
                    each<4>([&](auto step) {
                        constexpr int j = decltype(step)::value, k = k0 + j;
                        each<NS>([&](auto state) {
                            constexpr int i = decltype(state)::value;
                            a[k][i] = hw_exp2(g.v[j].x * A2[i]);
                            h[k + 1][i] = __builtin_fmaf(a[k][i], h[k][i], g.v[j].y * g.b.template at<j, i>());
                        });
                    });
                });
                each<CK / 4>([&](auto group) {
                    constexpr int k0 = CK - 4 - 4 * decltype(group)::value;
                    const int row = row0 + k0;
                    Steps4<NS, W, true> g;
                    g.load(in, bc, row, c, q, lane);
                    float s[4], o4[3][4], vb[4][NS], vc[4][NS];
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] = ss[row + j][c];
                    each<4>([&](auto step) {
                        constexpr int j = 3 - decltype(step)::value, k = k0 + j;
                        float ra = 0.f, rb = 0.f, ch = 0.f;
                        if constexpr (NS == 2 || NS == 4) back<j>(g.c.v[0], g.b.v[0], s[j], h[k + 1], r, ch, rb);
                        else
                            each<NS>([&](auto state) {
                                constexpr int i = decltype(state)::value;
                                const float cv = g.c.template at<j, i>();
                                r[i] = __builtin_fmaf(cv, s[j], r[i]);
                                ch = __builtin_fmaf(cv, h[k + 1][i], ch);
                                rb = __builtin_fmaf(g.b.template at<j, i>(), r[i], rb);
                            });
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            vb[j][i] = r[i] * g.v[j].y;
                            vc[j][i] = s[j] * h[k + 1][i];
                            r[i] *= a[k][i];
                            const float w = r[i] * h[k][i];
                            ra = __builtin_fmaf(w, A2[i], ra);
                            dA[i] = __builtin_fmaf(w, g.v[j].x, dA[i]);
                        }
                        o4[0][j] = rb, o4[1][j] = ra, o4[2][j] = ch;
                    });
#pragma unroll
                    for (int j = 0; j < 3; ++j) sh.o[buf][j][half][row + lrow][c] = rows4(o4[j]);
                    // Four steps' dB and dC of two states (or of one): eight
                    // values at a time meet in halve_row -- two steps', kind by
                    // bit 2, state by bit 3 -- then the steps by bits 1 and 0.
                    const int bit0 = lane & 1, bit1 = lane >> 1 & 1, bit2 = lane >> 2 & 1, bit3 = lane >> 3 & 1;
#pragma unroll
                    for (int m = 0; m < NS; m += 2) {
                        const auto at2 = [&](const float (&v)[4][NS], int j, int i) { return m + i < NS ? v[j][m + i] : 0.f; };
                        float z[4];
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const float v8[8] = {at2(vb, j, 0), at2(vb, j, 1), at2(vc, j, 0), at2(vc, j, 1),
                                                 at2(vb, j + 1, 0), at2(vb, j + 1, 1), at2(vc, j + 1, 0), at2(vc, j + 1, 1)};
                            halve_row(v8, z[j], z[j + 1]);
                        }
                        // Steps 0, 1 and 2, 3 by bit 0, the two pairs by bit 1.
                        const float e = halve_quad(z[0], z[1], bit0, false), l = halve_quad(z[2], z[3], bit0, false);
                        const float all = halve_quad(e, l, bit1, true);
                        if (NS > 1 || bit3 == 0)
                            sh.red[buf][wave & 3][row + 2 * bit1 + bit0][bit2 * W + q * NS + m + (NS > 1 ? bit3 : 0)] = all;
                    }
                });
            }
        }
        lds_sync();
    }
    if constexpr (PRE) {
        if (!real) return;
        const int64_t k = (at.first + at.ch) * p.C + cc;
#pragma unroll
        for (int i = 0; i < NS; ++i) p.carry_h[k * W + q * NS + i] = r[i];
        if (q == 0) p.carry_d[k] = sum_d;
    } else {
        // The staging waves' four barriers of the last sums.
        for (int k = 0; k < 4; ++k) lds_sync();
        if (!real) return;
        if (p.ds && at.ch == 0) put_states<NS>(p.ds, p.dss, at.seq, cc, q * NS, p.S, r);
        // Parts of dA (4 NS per channel), dD and the bias, laid out [part][channel][4 NS + 2].
        float *pc = p.part_c + (at.part * p.C + at.c0) * (W + 2);
#pragma unroll
        for (int i = 0; i < NS; ++i) pc[c * (W + 2) + q * NS + i] = dA[i];
    }
}

// dB and dC: the parts of a group's workgroups.  One thread per (row, kind, state).
template <typename T>
__global__ __launch_bounds__(256) void scan_bwd_bc(const float *part, int64_t rows, int64_t L, int64_t blocks_g, int G,
                                                   int S, int W, T *dB, S4 bs, T *dC, S4 cs)
{
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= rows * 2 * W * G) return;
    const int64_t per = rows * 2 * W;
    int64_t in, j, l;
    const int64_t g = divide(e, per, in), row = divide(in, 2 * W, j), s = j < W ? j : j - W;
    if (s >= S) return;
    const float *q = part + g * blocks_g * per + in;
    float a[4] = {};
    int64_t i = 0;
    for (; i + 4 <= blocks_g; i += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] += q[(i + k) * per];
    for (; i < blocks_g; ++i) a[0] += q[i * per];
    const T v = from_f32<T>((a[0] + a[1]) + (a[2] + a[3]));
    const int64_t n = divide(row, L, l);
    if (j < W) dB[n * bs.n + g * bs.g + s * bs.s + l * bs.l] = v;
    else dC[n * cs.n + g * cs.g + s * cs.s + l * cs.l] = v;
}

// dA, dD and the bias's gradient: the parts of all sequences and chunks.
__global__ __launch_bounds__(256) void scan_bwd_c(const ScanP p, int W, float *dA, int64_t a_c, int64_t a_s, float *dD,
                                                  int64_t d_s, float *db, int64_t b_s)
{
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, n = p.C * (W + 2);
    if (e >= n) return;
    float v = 0.f;
    for (int64_t k = 0; k < p.parts; ++k) v += p.part_c[k * n + e];
    int64_t j;
    const int64_t c = divide(e, W + 2, j);
    if (j < p.S) dA[c * a_c + j * a_s] = v;
    else if (j == W && dD) dD[c * d_s] = v;
    else if (j == W + 1 && db) db[c * b_s] = v;
}

}  // namespace

int launch_lm_scan_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    ScanP a = scan_params(p, q);
    const int W = scan_shape(p.S).width(), TB = bwd_tile(W);
    float *f = static_cast<float *>(ws);
    a.part_bc = f, f += a.blocks * a.rows_total * 2 * W;
    a.part_c = f, f += lm_cdiv(lm_parts(p) * a.C * (W + 2), 4) * 4;
    a.carry_d = f, f += lm_cdiv(lm_parts(p) * a.C, 4) * 4;
    a.carry_h = f;
    const bool dense = scan_dense(p, a, TB / 4, TB * W / 128);
    const int grid = (int)(lm_parts(p) * a.blocks);
    with_type(p.dtype, [&](auto t) {
        typedef decltype(t) T;
        with_ns(p.S, [&](auto n, auto w) {
            constexpr int NS = decltype(n)::value, QW = decltype(w)::value, threads = 256 * QW + kStage;
            if (grid == 0) return;
            if (dense) {
                if (a.chunks > 1) scan_bwd<T, NS, QW, true, true><<<grid, threads, 0, s>>>(a);
                scan_bwd<T, NS, QW, false, true><<<grid, threads, 0, s>>>(a);
            } else {
                if (a.chunks > 1) scan_bwd<T, NS, QW, true, false><<<grid, threads, 0, s>>>(a);
                scan_bwd<T, NS, QW, false, false><<<grid, threads, 0, s>>>(a);
            }
        });
        if (a.rows_total > 0) scan_bwd_bc<T><<<(int)lm_cdiv(a.rows_total * 2 * W * p.G, 256), 256, 0, s>>>(
            a.part_bc, a.rows_total, p.L, a.blocks_g, (int)p.G, (int)p.S, W, static_cast<T *>(q[LM_DB]),
            lm_s4(p.t[LM_DB]), static_cast<T *>(q[LM_DC]), lm_s4(p.t[LM_DC]));
    });
    if (p.C > 0) scan_bwd_c<<<(int)lm_cdiv(p.C * (W + 2), 256), 256, 0, s>>>(
        a, W, static_cast<float *>(q[LM_DA]), p.t[LM_DA].strides[0], p.t[LM_DA].strides[1], static_cast<float *>(q[LM_DD]),
        p.t[LM_DD].strides[0], static_cast<float *>(q[LM_DDT_BIAS]), p.t[LM_DDT_BIAS].strides[0]);
    return lm_launch_status();
}

}  // namespace miconv
