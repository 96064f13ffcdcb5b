// lm_plan: checks of the sequence operators' descriptors and arguments, and
// how their long axis is split.  lm_run: checks of the pointers, dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "lm_check.h"

namespace {

using namespace miconv;

// Which tensors an operator may have.
uint64_t allowed(int op)
{
    const auto m = [](std::initializer_list<int> l) {
        uint64_t v = 0;
        for (int s : l) v |= 1ull << s;
        return v;
    };
    switch (op) {
    case LM_CONV: return m({LM_X, LM_W, LM_BIAS, LM_Y, LM_STATE_IN, LM_STATE_OUT, LM_OFFSETS});
    case LM_CONV_BWD:
        return m({LM_X, LM_W, LM_BIAS, LM_STATE_IN, LM_OFFSETS, LM_GY, LM_GSTATE, LM_DX, LM_DW, LM_DBIAS, LM_DSTATE});
    case LM_CONV_STEP: return m({LM_X, LM_W, LM_BIAS, LM_Y, LM_STATE_OUT, LM_ROWS});
    case LM_SCAN:
        return m({LM_X, LM_DT, LM_A, LM_B, LM_C, LM_D, LM_Z, LM_DT_BIAS, LM_Y, LM_STATE_IN, LM_STATE_OUT, LM_OFFSETS, LM_SAVED});
    case LM_SCAN_BWD:
        return m({LM_X, LM_DT, LM_A, LM_B, LM_C, LM_D, LM_Z, LM_DT_BIAS, LM_OFFSETS, LM_SAVED, LM_GY, LM_GSTATE, LM_DX, LM_DDT,
                  LM_DA, LM_DB, LM_DC, LM_DD, LM_DZ, LM_DDT_BIAS, LM_DSTATE});
    case LM_SCAN_STEP: return m({LM_X, LM_DT, LM_A, LM_B, LM_C, LM_D, LM_Z, LM_DT_BIAS, LM_Y, LM_STATE_OUT, LM_ROWS});
    case LM_MV4: return m({LM_X, LM_W, LM_BIAS, LM_Y, LM_SCALES, LM_ZEROS});
    case LM_GATED: return m({LM_X, LM_A, LM_B, LM_D, LM_Y, LM_STATE_IN, LM_STATE_OUT, LM_OFFSETS, LM_SAVED});
    case LM_GATED_BWD:
        return m({LM_X, LM_A, LM_B, LM_D, LM_OFFSETS, LM_SAVED, LM_GY, LM_GSTATE, LM_DX, LM_DA, LM_DB, LM_DD, LM_DSTATE});
    case LM_GATED_STEP: return m({LM_X, LM_A, LM_B, LM_D, LM_Y, LM_STATE_OUT, LM_ROWS});
    case LM_NORM: return m({LM_X, LM_W, LM_Y, LM_STATE_IN, LM_STATE_OUT, LM_SCALES, LM_SAVED});
    case LM_NORM_BWD: return m({LM_X, LM_W, LM_STATE_IN, LM_GY, LM_GSTATE, LM_SAVED, LM_DX, LM_DW});
    case LM_ADAPTERS: return m({LM_X, LM_A, LM_B, LM_ROWS, LM_Z, LM_D, LM_SCALES, LM_Y});
    default: return 0;
    }
}

// A grid has fewer than 2^32 threads in each dimension.  The largest launch of
// the call is looked at (in double: sizes may be any).
bool one_launch(const lm_plan_t &p)
{
    const double C = (double)p.C, parts = (double)lm_parts(p);
    double threads = 0;
    const auto add = [&](double groups, double size) { threads = std::max(threads, std::ceil(groups) * size); };
    switch (p.op) {
    case LM_CONV: case LM_CONV_BWD: case LM_CONV_STEP:
        add(std::ceil(C / conv_width(p)) * parts / 256, 256);
        if (p.op == LM_CONV_BWD) add(C * (double)(p.K + 1) / 64, 1024);
        break;
    case LM_SCAN: case LM_SCAN_BWD: {
        const ScanShape shape = scan_shape(p.S);
        add(parts * (double)p.G * std::ceil(C / (double)p.G / LM_SCAN_CH), 256 * (shape.qw + 1));
        if (p.op == LM_SCAN_BWD) {
            add((double)p.t[LM_X].sizes[0] * (double)p.L * 2 * shape.width() * (double)p.G / 256, 256);
            add(C * (shape.width() + 2) / 256, 256);
        }
        break;
    }
    case LM_SCAN_STEP: add((double)p.seqs * C * 4 / 256, 256); break;
    case LM_MV4:
        if (mv4_parts(p) == 0) add(C / 16, 512);
        add(C / 256, 256), add((double)p.K / 256, 256);
        if (lm_cdiv(p.seqs, 16) > 65535) return false;   // rows of x lie along the second dimension
        break;
    }
    return threads < 4294967296.0 && parts < 2147483648.0;
}

// Rows per chunk and chunks per sequence of a convolution: the kernel's
// threads own a few channels each, and 2^18 of them are four waves for every
// SIMD, which hide the memory's latency (the forward kernel's registers let two
// or three of them run at a time, the backward one's four).  A chunk reads K-1
// rows of its neighbour again, so it is never shorter than min_rows.
void conv_chunks(lm_plan_t &p, int64_t max_len, int64_t per_thread, int64_t min_rows)
{
    int64_t rows = forced_rows(p, max_len);
    if (rows <= 0) {
        const int64_t total = p.t[LM_OFFSETS].rank ? p.L : p.seqs * p.L;
        rows = total * lm_cdiv(p.C, per_thread) / (1 << 18);
        rows = std::min<int64_t>(std::max(rows, min_rows), 128);
    }
    p.chunk = rows;
    p.chunks = std::max<int64_t>(1, lm_cdiv(max_len, rows));
}

// The scan along one sequence is serial; a workgroup per 64 channels fills the
// SIMDs of one compute unit by itself, two together (up to 16 states, forward)
// take about 1.5 times as long.  Splitting the long axis fills more units, at
// the price of a first pass over the chunks for the states between them (0.7
// of the main pass).  Of the chunk counts up to 64 the one with the least
// estimated time is taken; a workgroup's start costs about 48 steps.
void scan_chunks(lm_plan_t &p, int64_t max_len)
{
    constexpr int64_t tile = 32;
    const int64_t blocks = p.G * lm_cdiv(p.C / p.G, LM_SCAN_CH);
    const bool packed = p.t[LM_OFFSETS].rank > 0;
    const double pair = p.op == LM_SCAN && p.S <= 16 ? 1.5 : 2.0;
    int64_t rows = forced_rows(p, max_len);
    if (rows <= 0) {
        const int64_t len = std::max<int64_t>(max_len, 1);
        double best = 0;
        for (int64_t n = 1; n <= 64; ++n) {
            const int64_t chunk = lm_cdiv(lm_cdiv(len, n), tile) * tile;
            if (n > 1 && chunk < 2 * tile) break;
            // Packed sequences are of unlike lengths: whole chunks of all rows and half a one each.
            const double groups = (packed ? (double)p.L / chunk + 0.5 * p.seqs : (double)p.seqs * lm_cdiv(len, chunk)) * blocks;
            const double per_cu = std::max(1.0, packed ? groups / 256 : (double)lm_cdiv((int64_t)groups, 256));
            const double time = per_cu < 2 ? per_cu : pair * std::floor(per_cu / 2) + std::fmod(per_cu, 2.0);
            const double cost = time * (chunk + 48) * (n > 1 ? 1.7 : 1.0) + (n > 1 ? 48 : 0);
            if (n == 1 || cost < best) best = cost, rows = chunk;
        }
    }
    p.chunk = lm_cdiv(rows, tile) * tile;
    p.chunks = std::max<int64_t>(1, lm_cdiv(max_len, p.chunk));
}

}  // namespace

extern "C" int lm_plan(int32_t op, const conv_tensor *t, const lm_args *args, lm_plan_t *out, char *err, size_t err_len)
{
    Checker k{t, err, err_len};
    if (err && err_len) err[0] = 0;
    if (!t || !args || !out) return CONV_EINVAL;
    if (!allowed(op)) {
        k.fail(CONV_EINVAL, "unknown operator %d", op);
        return k.status;
    }
    for (int s = 0; s < LM_NSLOT; ++s)
        if (t[s].rank < 0 || t[s].rank > CONV_MAX_RANK || (t[s].rank > 0 && !(allowed(op) >> s & 1))) {
            k.fail(CONV_EINVAL, "%s is not a tensor of this operator", kNames[s]);
            return k.status;
        }
    for (int s = 0; s < LM_NSLOT; ++s)
        for (int i = 0; i < t[s].rank; ++i)
            if (t[s].sizes[i] < 0) {
                k.fail(CONV_EINVAL, "%s has a negative size", kNames[s]);
                return k.status;
            }
    if (op >= LM_GATED) {
        lm_plan_t p;
        memset(&p, 0, sizeof(p));
        p.op = op, p.args = *args;
        memcpy(p.t, t, sizeof(p.t));
        if (lm_plan_layer(op, k, *args, p) == CONV_OK) *out = p;
        return k.status;
    }
    const bool step = op == LM_CONV_STEP || op == LM_SCAN_STEP, conv = op <= LM_CONV_STEP, mv = op == LM_MV4;
    const bool bwd = op == LM_CONV_BWD || op == LM_SCAN_BWD;
    const conv_tensor &x = t[LM_X];
    if (x.rank != (step || mv ? 2 : 3)) {
        k.fail(CONV_EINVAL, "x has %d dims, %d expected", x.rank, step || mv ? 2 : 3);
        return k.status;
    }
    if (x.dtype != CONV_F32 && x.dtype != CONV_F16 && x.dtype != CONV_BF16) {
        k.fail(CONV_EINVAL, "x has to be float32, float16 or bfloat16");
        return k.status;
    }
    lm_plan_t p;
    memset(&p, 0, sizeof(p));
    p.op = op, p.dtype = x.dtype, p.args = *args;
    memcpy(p.t, t, sizeof(p.t));
    const int32_t dt = x.dtype;
    const int64_t e = elem(dt);
    if (args->max_len < 0 || args->chunk < 0 || (args->flags & ~(conv ? LM_SILU : mv ? 0 : LM_SOFTPLUS))) {
        k.fail(CONV_EINVAL, "unknown flags or negative lengths");
        return k.status;
    }

    if (mv) {
        p.seqs = x.sizes[0], p.K = x.sizes[1], p.C = t[LM_W].sizes[0], p.L = 1;
        p.G = t[LM_SCALES].rank == 2 ? t[LM_SCALES].sizes[1] : 0;
        k.want(LM_X, dt, {p.seqs, p.K});
        if (k.status == CONV_OK && (p.K < 1 || p.K % 2)) k.fail(CONV_EINVAL, "x needs an even number of columns");
        k.want(LM_W, LM_U8, {p.C, p.K / 2});
        k.want(LM_SCALES, dt, {p.C, p.G});
        k.want(LM_ZEROS, dt, {p.C, p.G}, true);
        k.want(LM_BIAS, dt, {p.C}, true);
        k.want(LM_Y, dt, {p.seqs, p.C});
        k.output(LM_Y);
        if (k.status != CONV_OK) return k.status;
        if (p.G < 1 || p.K % p.G) {
            k.fail(CONV_EINVAL, "%lld columns do not make %lld groups", (long long)p.K, (long long)p.G);
            return k.status;
        }
        if ((p.K / p.G) % 32) {
            k.fail(CONV_EUNSUPPORTED, "groups of %lld columns: multiples of 32 are supported", (long long)(p.K / p.G));
            return k.status;
        }
        if (t[LM_W].strides[1] != 1 || (p.C > 1 && t[LM_W].strides[0] % 16)) {
            k.fail(CONV_EUNSUPPORTED, "w needs contiguous rows a multiple of 16 bytes apart");
            return k.status;
        }
        if (p.K > 0x7fffff00 || !one_launch(p)) {
            k.fail(CONV_EUNSUPPORTED, "too many rows for one launch");
            return k.status;
        }
        p.workspace_bytes = mv4_rows_bytes(p) + (mv4_parts(p) > 1 ? mv4_parts(p) * p.seqs * p.C * 4 : 0);
        p.flops = 2 * p.seqs * p.K * p.C;
        p.bytes = p.C * p.K / 2 + p.C * p.G * e * (k.has(LM_ZEROS) ? 2 : 1) + (p.seqs * (p.K + p.C) + (k.has(LM_BIAS) ? p.C : 0)) * e;
        *out = p;
        return CONV_OK;
    }

    const bool packed = k.has(LM_OFFSETS);
    const int64_t N = x.sizes[0];
    p.C = x.sizes[1], p.L = step ? 1 : x.sizes[2];
    p.seqs = packed ? t[LM_OFFSETS].sizes[0] - 1 : N;
    if (packed) {
        if (p.seqs < 0) k.fail(CONV_EINVAL, "offsets needs at least one element");
        k.want(LM_OFFSETS, LM_I32, {p.seqs + 1});
        if (k.status == CONV_OK && N != 1) k.fail(CONV_EINVAL, "a packed x has one row, not %lld", (long long)N);
        if (k.status == CONV_OK && t[LM_OFFSETS].strides[0] != 1 && p.seqs > 0) k.fail(CONV_EINVAL, "offsets has to be contiguous");
        if (k.status == CONV_OK && p.L > 0x7fffffff) k.fail(CONV_EINVAL, "offsets are 32-bit: at most 2^31 - 1 rows");
    }
    const int64_t max_len = !packed ? p.L : (args->max_len > 0 ? std::min(args->max_len, p.L) : p.L);
    const auto like_x = [&](int s, bool optional = false) {
        if (step) k.want(s, dt, {N, p.C}, optional);
        else k.want(s, dt, {N, p.C, p.L}, optional);
    };
    like_x(LM_X);
    if (bwd) like_x(LM_GY), like_x(LM_DX, conv), k.output(LM_DX);
    else like_x(LM_Y, op == LM_SCAN), k.output(LM_Y);
    // A state of a step lives in a table of at least as many rows as the batch
    // (of any number when the rows are named).
    const int64_t st_rows = step ? t[LM_STATE_OUT].sizes[0] : p.seqs;
    if (k.status == CONV_OK && step) {
        k.want(LM_ROWS, LM_I32, {N}, true);
        if (k.status == CONV_OK && k.has(LM_ROWS) && t[LM_ROWS].strides[0] != 1 && N > 1) k.fail(CONV_EINVAL, "rows has to be contiguous");
        if (k.status == CONV_OK && !k.has(LM_ROWS) && st_rows != N) k.fail(CONV_EINVAL, "the state has %lld rows, x %lld", (long long)st_rows, (long long)N);
    }
    if (conv) {
        if (k.status == CONV_OK && t[LM_W].rank != 2) k.fail(CONV_EINVAL, "w has %d dims, 2 expected", t[LM_W].rank);
        p.K = t[LM_W].sizes[1];
        k.want(LM_W, dt, {p.C, p.K});
        k.want(LM_BIAS, dt, {p.C}, true);
        if (k.status == CONV_OK && p.K < 1) k.fail(CONV_EINVAL, "w has no taps");
        if (k.status == CONV_OK && p.K > LM_MAX_TAPS) k.fail(CONV_EUNSUPPORTED, "%lld taps: 1 to %d are supported", (long long)p.K, LM_MAX_TAPS);
        for (int s : {LM_STATE_IN, LM_STATE_OUT, LM_GSTATE, LM_DSTATE})
            k.want(s, dt, {s == LM_STATE_OUT ? st_rows : p.seqs, p.C, p.K - 1}, !(step && s == LM_STATE_OUT));
        if (bwd) {
            k.want(LM_DW, dt, {p.C, p.K}, true);
            k.want(LM_DBIAS, dt, {p.C}, true);
        }
    } else {
        p.S = t[LM_A].rank == 2 ? t[LM_A].sizes[1] : 0;
        p.G = t[LM_B].rank >= 2 ? t[LM_B].sizes[1] : 0;
        k.want(LM_A, CONV_F32, {p.C, p.S});
        if (k.status == CONV_OK && (p.S < 1 || p.S > LM_MAX_STATES)) k.fail(CONV_EUNSUPPORTED, "%lld states: 1 to %d are supported", (long long)p.S, LM_MAX_STATES);
        for (int s : {LM_B, LM_C}) {
            if (step) k.want(s, dt, {N, p.G, p.S});
            else k.want(s, dt, {N, p.G, p.S, p.L});
        }
        if (k.status == CONV_OK && (p.G < 1 || p.C % p.G)) k.fail(CONV_EINVAL, "%lld channels do not make %lld groups", (long long)p.C, (long long)p.G);
        like_x(LM_DT);
        like_x(LM_Z, true);
        for (int s : {LM_D, LM_DT_BIAS}) k.want(s, CONV_F32, {p.C}, true);
        for (int s : {LM_STATE_IN, LM_STATE_OUT, LM_GSTATE, LM_DSTATE})
            k.want(s, CONV_F32, {s == LM_STATE_OUT ? st_rows : p.seqs, p.C, p.S}, !(step && s == LM_STATE_OUT));
        if (bwd) {
            like_x(LM_DDT);
            k.want(LM_DA, CONV_F32, {p.C, p.S});
            k.want(LM_DB, dt, {N, p.G, p.S, p.L}), k.want(LM_DC, dt, {N, p.G, p.S, p.L});
            if (k.has(LM_Z)) like_x(LM_DZ);
            if (k.has(LM_D)) k.want(LM_DD, CONV_F32, {p.C});
            if (k.has(LM_DT_BIAS)) k.want(LM_DDT_BIAS, CONV_F32, {p.C});
            for (const auto &pr : {std::make_pair(LM_Z, LM_DZ), std::make_pair(LM_D, LM_DD), std::make_pair(LM_DT_BIAS, LM_DDT_BIAS)})
                if (k.status == CONV_OK && k.has(pr.second) && !k.has(pr.first)) k.fail(CONV_EINVAL, "%s without %s", kNames[pr.second], kNames[pr.first]);
        }
    }
    for (int s : {LM_STATE_OUT, LM_DSTATE, LM_DW, LM_DBIAS, LM_DDT, LM_DA, LM_DB, LM_DC, LM_DD, LM_DZ, LM_DDT_BIAS}) k.output(s);
    if (k.status != CONV_OK) return k.status;

    const int64_t rows = packed ? p.L : N * p.L, cells = rows * p.C;
    if (conv) {
        if (!step) conv_chunks(p, max_len, bwd ? 2 : 16 / e, bwd ? 32 : 8);
        else p.chunk = p.chunks = 1;
        if (bwd && (k.has(LM_DW) || k.has(LM_DBIAS))) p.workspace_bytes = lm_parts(p) * p.C * (p.K + 1) * 4;
        const int64_t st = p.seqs * p.C * (p.K - 1) * e * ((k.has(LM_STATE_IN) || step) + k.has(LM_STATE_OUT) + k.has(LM_GSTATE) + k.has(LM_DSTATE));
        const int64_t act = args->flags & LM_SILU ? 4 : 0;
        p.bytes = cells * e * (bwd ? 2 + k.has(LM_DX) : 2) + st + (bwd ? 2 : 1) * p.C * (p.K + k.has(LM_BIAS)) * e;
        p.flops = cells * (bwd ? 6 * p.K + 2 * act : 2 * p.K + act);
    } else {
        const int W = scan_shape(p.S).width(), ck = scan_shape(p.S).save_steps();
        if (!step) scan_chunks(p, max_len);
        else p.chunk = p.chunks = 1;
        p.saved_floats = step ? 0 : (packed ? p.L / ck + p.seqs + 1 : N * lm_cdiv(p.L, ck)) * p.C * W;
        if (k.has(LM_SAVED) || op == LM_SCAN_BWD) k.want(LM_SAVED, CONV_F32, {p.saved_floats});
        if (k.status == CONV_OK && k.has(LM_SAVED) && t[LM_SAVED].strides[0] != 1 && p.saved_floats > 1) k.fail(CONV_EINVAL, "saved has to be contiguous");
        if (k.status != CONV_OK) return k.status;
        const int64_t blocks = p.G * lm_cdiv(p.C / p.G, LM_SCAN_CH);
        const int64_t parts = lm_parts(p), carries = scan_carries(p);
        if (op == LM_SCAN) p.workspace_bytes = 4 * (lm_cdiv(carries * p.C, 4) * 4 + carries * p.C * W);
        if (op == LM_SCAN_BWD)
            p.workspace_bytes = 4 * (blocks * N * p.L * 2 * W + lm_cdiv(parts * p.C * (W + 2), 4) * 4 + lm_cdiv(parts * p.C, 4) * 4 +
                                     parts * p.C * W);
        const int64_t io = 3 + k.has(LM_Z), bc = 2 * p.G * p.S * rows * e;
        p.bytes = cells * e * (bwd ? 2 * io : io) + (bwd ? 2 : 1) * (bc + p.C * (p.S + k.has(LM_D) + k.has(LM_DT_BIAS)) * 4) +
                  p.seqs * p.C * p.S * 4 * (k.has(LM_STATE_IN) + (step ? 2 : k.has(LM_STATE_OUT)) + k.has(LM_GSTATE) + k.has(LM_DSTATE));
        p.flops = cells * (bwd ? 20 * p.S + 40 : 7 * p.S + 16);
    }
    if (!one_launch(p)) {
        k.fail(CONV_EUNSUPPORTED, "too many rows for one launch");
        return k.status;
    }
    *out = p;
    return CONV_OK;
}

extern "C" int lm_run(const lm_plan_t *p, void *const *q, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!p || !q) return CONV_EINVAL;
    for (int s = 0; s < LM_NSLOT; ++s) {
        const conv_tensor &t = p->t[s];
        int64_t n = t.rank > 0;
        for (int i = 0; i < t.rank; ++i) n *= t.sizes[i];
        if (!q[s] && n > 0) return CONV_EINVAL;
        if (q[s] && t.rank == 0) return CONV_EINVAL;
        if (reinterpret_cast<uintptr_t>(q[s]) % (uintptr_t)std::max<int64_t>(1, elem(t.dtype))) return CONV_EALIGN;
    }
    if (p->op == LM_MV4 && reinterpret_cast<uintptr_t>(q[LM_W]) % 16) return CONV_EALIGN;
    if (p->op < LM_MV4 && reinterpret_cast<uintptr_t>(q[LM_SAVED]) % 16) return CONV_EALIGN;   // read as whole vectors
    if (p->workspace_bytes > 0) {
        if (!workspace || workspace_bytes < (size_t)p->workspace_bytes) return CONV_EINVAL;
        if (reinterpret_cast<uintptr_t>(workspace) % 256) return CONV_EALIGN;
    }
    // Sums are written without their terms too, as zeros: those over sequences
    // (dw, dA ...) without sequences, those over channels (dB, dC) without channels.
    if ((p->C == 0 && p->op != LM_SCAN_BWD) || ((p->op == LM_MV4 || p->op == LM_ADAPTERS) && p->seqs == 0)) return CONV_OK;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (p->op) {
    case LM_CONV: return launch_lm_conv(*p, q, s);
    case LM_CONV_BWD: return launch_lm_conv_bwd(*p, q, workspace, s);
    case LM_CONV_STEP: return launch_lm_conv_step(*p, q, s);
    case LM_SCAN: return launch_lm_scan(*p, q, workspace, s);
    case LM_SCAN_BWD: return launch_lm_scan_bwd(*p, q, workspace, s);
    case LM_SCAN_STEP: return launch_lm_scan_step(*p, q, s);
    case LM_MV4: return launch_lm_mv4(*p, q, workspace, s);
    case LM_GATED: return launch_lm_gated(*p, q, workspace, s);
    case LM_GATED_BWD: return launch_lm_gated_bwd(*p, q, workspace, s);
    case LM_GATED_STEP: return launch_lm_gated_step(*p, q, s);
    case LM_NORM: return launch_lm_norm(*p, q, s);
    case LM_NORM_BWD: return launch_lm_norm_bwd(*p, q, workspace, s);
    case LM_ADAPTERS: return launch_lm_adapters(*p, q, workspace, s);
    default: return CONV_EINVAL;
    }
}
