// Plans of the gated recurrence, the RMS norm and the adapters: checks of their
// tensors, how their work is split.
#include <cmath>

#include "lm_check.h"

namespace miconv {
namespace {

// The grids' threads, in double: sizes may be any.
bool fits(double groups, double size) { return std::ceil(groups) * size < 4294967296.0; }

// Rows per chunk and chunks per sequence of the recurrence.
//
// Forward: a workgroup that walks down whole sequences takes 6 us a tile, or its
// share of the memory where more than 210 of them run (0.0285 us for each).
// Every tile a workgroup of its own takes 0.036 us for each tile and 12 to begin
// with: 8 x 2048 x 2048 in 85 us for 101, 12 x 2048 x 2048 in 187 for 109.
// Backward: chunks by the least estimated time; what enters them takes a pass
// over two of seven tensors, and a workgroup's start about a tile (8 x 2048 x
// 2048: whole 186 us, chunks of 1024 and 512 rows 136; 1 x 1024 x 4096: whole
// 330, 256 rows 41, 128 rows 29).
void gated_chunks(lm_plan_t &p, int64_t max_len)
{
    const int64_t blocks = lm_cdiv(p.C, 64 * gated_width(p)), tile = LM_GATED_TILE, len = std::max<int64_t>(max_len, 1);
    const bool packed = p.t[LM_OFFSETS].rank > 0;
    int64_t rows = forced_rows(p, max_len);
    if (rows > 0) {
        if (p.op == LM_GATED && rows < len) rows = tile;
    } else if (p.op == LM_GATED) {
        const double groups = (double)p.seqs * blocks;
        const double tiles = (packed ? (double)p.L / tile + 0.5 * p.seqs : (double)p.seqs * lm_cdiv(len, tile)) * blocks;
        // Packed sequences are of unlike lengths: the longest one counts, and all of them together.
        const double walk = std::max(lm_cdiv(len, tile) * std::max(6.0, packed ? 0 : 0.0285 * groups), 0.0285 * tiles);
        rows = len > tile && walk > 0.036 * tiles + 12 ? tile : len;
    } else {
        double best = 0;
        for (int64_t n = 1; n <= 256; ++n) {
            const int64_t chunk = lm_cdiv(lm_cdiv(len, n), tile) * tile;
            const double groups = (packed && n > 1 ? (double)p.L / chunk + 0.5 * p.seqs : (double)p.seqs * lm_cdiv(len, chunk)) * blocks;
            const double per_cu = packed ? std::max(1.0, groups / 256) : std::ceil(groups / 256);
            const double cost = per_cu * (chunk + tile) * (n > 1 ? 1.3 : 1.0) + (n > 1 ? tile : 0);
            if (n == 1 || cost < best) best = cost, rows = chunk;
            if (chunk == tile) break;
        }
    }
    p.chunk = lm_cdiv(rows, tile) * tile;
    p.chunks = std::max<int64_t>(1, lm_cdiv(max_len, p.chunk));
}

int plan_gated(int op, Checker &k, const lm_args &args, lm_plan_t &p)
{
    const bool step = op == LM_GATED_STEP, bwd = op == LM_GATED_BWD;
    const conv_tensor &x = k.t[LM_X];
    if (x.rank != (step ? 2 : 3)) return k.fail(CONV_EINVAL, "x has %d dims, %d expected", x.rank, step ? 2 : 3), k.status;
    const bool packed = k.has(LM_OFFSETS);
    const int32_t dt = x.dtype;
    const int64_t N = x.sizes[0], e = elem(dt);
    p.C = x.sizes[1], p.L = step ? 1 : x.sizes[2];
    p.seqs = packed ? k.t[LM_OFFSETS].sizes[0] - 1 : N;
    if (!(args.value >= 0) || std::isinf(args.value)) k.fail(CONV_EINVAL, "the factor of the decay has to be finite and not negative");
    if (packed) {
        if (p.seqs < 0) k.fail(CONV_EINVAL, "offsets needs at least one element");
        k.want(LM_OFFSETS, LM_I32, {p.seqs + 1});
        if (k.status == CONV_OK && N != 1) k.fail(CONV_EINVAL, "a packed x has one row, not %lld", (long long)N);
        if (k.status == CONV_OK && k.t[LM_OFFSETS].strides[0] != 1 && p.seqs > 0) k.fail(CONV_EINVAL, "offsets has to be contiguous");
        if (k.status == CONV_OK && p.L > 0x7fffffff) k.fail(CONV_EINVAL, "offsets are 32-bit: at most 2^31 - 1 rows");
    }
    const int64_t max_len = !packed ? p.L : (args.max_len > 0 ? std::min(args.max_len, p.L) : p.L);
    const auto like_x = [&](int s, bool optional = false) {
        if (step) k.want(s, dt, {N, p.C}, optional);
        else k.want(s, dt, {N, p.C, p.L}, optional);
    };
    like_x(LM_X), like_x(LM_A), like_x(LM_B);
    k.want(LM_D, CONV_F32, {p.C});
    if (bwd) like_x(LM_GY), like_x(LM_DX), like_x(LM_DA), like_x(LM_DB), k.want(LM_DD, CONV_F32, {p.C});
    else like_x(LM_Y, op == LM_GATED);
    const int64_t st_rows = step ? k.t[LM_STATE_OUT].sizes[0] : p.seqs;
    if (step) {
        k.want(LM_ROWS, LM_I32, {N}, true);
        if (k.status == CONV_OK && k.has(LM_ROWS) && k.t[LM_ROWS].strides[0] != 1 && N > 1) k.fail(CONV_EINVAL, "rows has to be contiguous");
        if (k.status == CONV_OK && !k.has(LM_ROWS) && st_rows != N) k.fail(CONV_EINVAL, "the state has %lld rows, x %lld", (long long)st_rows, (long long)N);
    }
    for (int s : {LM_STATE_IN, LM_STATE_OUT, LM_GSTATE, LM_DSTATE})
        k.want(s, CONV_F32, {s == LM_STATE_OUT ? st_rows : p.seqs, p.C}, !(step && s == LM_STATE_OUT));
    for (int s : {LM_Y, LM_STATE_OUT, LM_DX, LM_DA, LM_DB, LM_DD, LM_DSTATE}) k.output(s);
    if (k.status != CONV_OK) return k.status;

    const int64_t cells = (packed ? p.L : N * p.L) * p.C;
    p.chunk = p.chunks = 1;
    if (!step) {
        gated_chunks(p, max_len);
        p.saved_floats = (packed ? p.L / LM_GATED_SAVE + p.seqs + 1 : N * lm_cdiv(p.L, LM_GATED_SAVE)) * p.C;
        if (k.has(LM_SAVED) || bwd) k.want(LM_SAVED, CONV_F32, {p.saved_floats});
        if (k.status == CONV_OK && k.has(LM_SAVED) && k.t[LM_SAVED].strides[0] != 1 && p.saved_floats > 1) k.fail(CONV_EINVAL, "saved has to be contiguous");
        if (k.status != CONV_OK) return k.status;
        const int64_t parts = lm_parts(p);
        p.workspace_bytes = gated_look(p) ? 16 * parts * p.C + 128 * lm_cdiv(p.C, 64 * gated_width(p)) : 4 * p.C * ((p.chunks > 1 ? 2 * parts : 0) + (bwd ? parts : 0));
    }
    const double groups = (double)lm_parts(p) * std::ceil((double)p.C / (64 * gated_width(p)));
    if (!(step ? fits((double)N * p.C / gated_step_width(p) / 256, 256) : fits(groups, 1024) && (!gated_look(p) || fits(2 * (double)(lm_parts(p) + 16) * p.C, 1))) || !fits((double)p.C / 64, 1024) ||
        lm_parts(p) >= 0x7fffffff)
        return k.fail(CONV_EUNSUPPORTED, "too many rows for one launch"), k.status;
    const int64_t states = (step ? 2 : k.has(LM_STATE_IN) + k.has(LM_STATE_OUT)) + k.has(LM_GSTATE) + k.has(LM_DSTATE);
    p.bytes = cells * e * (bwd ? 7 : 3 + k.has(LM_Y)) + p.seqs * p.C * 4 * states + p.C * 4 * (1 + bwd);
    p.flops = cells * (bwd ? 40 : 20);
    return k.status;
}

int plan_norm(int op, Checker &k, const lm_args &args, lm_plan_t &p)
{
    const bool bwd = op == LM_NORM_BWD;
    const conv_tensor &x = k.t[LM_X];
    if (x.rank != 2 && x.rank != 3) return k.fail(CONV_EINVAL, "x has %d dims, 2 or 3 expected", x.rank), k.status;
    const int32_t dt = x.dtype;
    const int64_t N = x.sizes[0], e = elem(dt);
    p.seqs = N, p.C = x.sizes[1], p.L = x.rank == 3 ? x.sizes[2] : 1;
    if (!(args.value >= 0) || std::isinf(args.value)) k.fail(CONV_EINVAL, "what is added to the mean has to be finite and not negative");
    const auto shaped = [&](int s, int32_t type, int64_t columns, bool optional) {
        if (x.rank == 3) k.want(s, type, {N, columns, p.L}, optional);
        else k.want(s, type, {N, columns}, optional);
    };
    shaped(LM_X, dt, p.C, false);
    k.want(LM_W, dt, {p.C});
    if (x.rank == 3) k.want(LM_SAVED, CONV_F32, {N, p.L}, !bwd);
    else k.want(LM_SAVED, CONV_F32, {N}, !bwd);
    if (bwd) {
        shaped(LM_STATE_IN, dt, p.C, true), shaped(LM_GY, dt, p.C, false), shaped(LM_GSTATE, dt, p.C, true), shaped(LM_DX, dt, p.C, true);
        k.want(LM_DW, dt, {p.C}, true);
        if (k.status == CONV_OK && !k.has(LM_DX) && !k.has(LM_DW)) k.fail(CONV_EINVAL, "no gradient wanted");
        if (k.status == CONV_OK && k.has(LM_GSTATE) && !k.has(LM_DX)) k.fail(CONV_EINVAL, "gstate without dx");
    } else {
        const bool f8 = k.t[LM_Y].dtype == LM_F8 && k.has(LM_Y);
        shaped(LM_Y, f8 ? LM_F8 : dt, p.C, false);
        shaped(LM_STATE_IN, dt, p.C, true), shaped(LM_STATE_OUT, dt, p.C, true);
        if (k.status == CONV_OK && k.has(LM_STATE_IN) != k.has(LM_STATE_OUT)) k.fail(CONV_EINVAL, "state_out comes with state_in, and only with it");
        if (k.status == CONV_OK && k.has(LM_SCALES) != f8) k.fail(CONV_EINVAL, "scales come with an 8-bit y, and only with it");
        if (k.status == CONV_OK && f8) {
            p.G = k.t[LM_SCALES].rank >= 2 ? k.t[LM_SCALES].sizes[1] : 0;
            shaped(LM_SCALES, CONV_F32, p.G, false);
            if (k.status == CONV_OK && (p.G < 1 || p.C % p.G)) k.fail(CONV_EINVAL, "%lld channels do not make %lld groups", (long long)p.C, (long long)p.G);
            const int64_t group = p.G > 0 ? p.C / p.G : 0;
            if (k.status == CONV_OK && p.G > 1 && group != 32 && group != 64 && group != 128)
                k.fail(CONV_EUNSUPPORTED, "groups of %lld channels: 32, 64, 128 or all are supported", (long long)group);
        }
    }
    for (int s : {LM_Y, LM_STATE_OUT, LM_SCALES, LM_DX, LM_DW}) k.output(s);
    if (!bwd) k.output(LM_SAVED);
    if (k.status != CONV_OK) return k.status;
    if (p.C < 1) return k.fail(CONV_EINVAL, "x has no channels"), k.status;
    if (p.C > LM_NORM_MAX) return k.fail(CONV_EUNSUPPORTED, "%lld channels: 1 to %d are supported", (long long)p.C, LM_NORM_MAX), k.status;
    p.chunk = p.chunks = 1;
    const double all = (double)N * (double)p.L;
    const int64_t rows = all < 4294967296.0 ? N * p.L : 0;
    if (!fits(all, 64) || !fits(all, (double)norm_threads(rows, p.C))) return k.fail(CONV_EUNSUPPORTED, "too many rows for one launch"), k.status;
    if (bwd && k.has(LM_DW)) p.workspace_bytes = norm_bwd_groups(p) * p.C * 4;
    const int64_t cells = rows * p.C;
    p.bytes = bwd ? cells * e * (2 + k.has(LM_STATE_IN) + k.has(LM_GSTATE) + k.has(LM_DX)) + rows * 4 + p.C * e * (1 + k.has(LM_DW))
                  : cells * e * (k.has(LM_STATE_IN) ? 3 : 1) + cells * elem(k.t[LM_Y].dtype) + p.C * e + rows * 4 * (p.G + k.has(LM_SAVED));
    p.flops = cells * (bwd ? 10 : 6);
    return k.status;
}

int plan_adapters(Checker &k, lm_plan_t &p)
{
    const conv_tensor &x = k.t[LM_X], &a = k.t[LM_A];
    if (x.rank != 2 && x.rank != 3) return k.fail(CONV_EINVAL, "x has %d dims, 2 or 3 expected", x.rank), k.status;
    if (a.rank != 3) return k.fail(CONV_EINVAL, "A has %d dims, 3 expected", a.rank), k.status;
    const int32_t dt = a.dtype;
    if (dt != CONV_F32 && dt != CONV_F16 && dt != CONV_BF16) return k.fail(CONV_EINVAL, "A has to be float32, float16 or bfloat16"), k.status;
    const bool f8 = x.dtype == LM_F8;
    const int64_t N = x.sizes[0], L = x.rank == 3 ? x.sizes[2] : 1, E = a.sizes[0], e = elem(dt);
    p.dtype = dt;
    p.K = x.sizes[1], p.C = k.t[LM_B].rank == 3 ? k.t[LM_B].sizes[1] : 0, p.L = L, p.S = a.sizes[1], p.G = E;
    const auto shaped = [&](int s, int32_t type, int64_t columns, bool optional) {
        if (x.rank == 3) k.want(s, type, {N, columns, L}, optional);
        else k.want(s, type, {N, columns}, optional);
    };
    shaped(LM_X, f8 ? LM_F8 : dt, p.K, false);
    k.want(LM_A, dt, {E, p.S, p.K});
    k.want(LM_B, dt, {E, p.C, p.S});
    if (x.rank == 3) k.want(LM_ROWS, LM_I32, {N, L});
    else k.want(LM_ROWS, LM_I32, {N});
    if (k.status == CONV_OK) {
        const conv_tensor &i = k.t[LM_ROWS];
        const bool one = i.sizes[0] <= 1, last = i.rank == 2 ? i.sizes[1] <= 1 : true;
        if (i.rank == 1 ? !one && i.strides[0] != 1 : (!last && i.strides[1] != 1) || (!one && i.strides[0] != L))
            k.fail(CONV_EINVAL, "rows has to be contiguous");
    }
    k.want(LM_D, CONV_F32, {E}, true);
    shaped(LM_Z, dt, p.C, true);
    shaped(LM_Y, dt, p.C, false);
    k.output(LM_Y);
    if (k.status == CONV_OK && k.has(LM_SCALES) != f8) k.fail(CONV_EINVAL, "scales come with an 8-bit x, and only with it");
    shaped(LM_SCALES, CONV_F32, 1, true);
    if (k.status != CONV_OK) return k.status;
    if (p.S < 1 || p.S > LM_MAX_RANK) return k.fail(CONV_EUNSUPPORTED, "rank %lld: 1 to %d are supported", (long long)p.S, LM_MAX_RANK), k.status;
    // Rows, columns and outputs are counted in 32 bits (their places in memory in 64).
    const double rows = (double)N * (double)L;
    if (rows >= 0x7fffff00 || p.K > 0x7fffff00 || p.C > 0x7fffff00 || E > 0x7fffffff) return k.fail(CONV_EUNSUPPORTED, "too many rows for one launch"), k.status;
    p.seqs = N * L;
    const AdapterShape s = adapter_shape(p);
    p.chunk = s.rows, p.chunks = s.parts;
    const double tiles = s.rows == 1 ? 1 : (double)s.tiles;   // gathered rows lie along the grid's second dimension
    if (!fits(tiles * s.parts * lm_cdiv(p.S, 64), 256) || !fits(2 * tiles * lm_cdiv(p.C, (int64_t)LM_ADAPTER_N * s.reps), 256))
        return k.fail(CONV_EUNSUPPORTED, "too many rows for one launch"), k.status;
    p.workspace_bytes = adapter_sums_bytes(p) + (s.rows == 1 ? 0 : lm_cdiv(16 * s.tiles + 4 * ((s.find ? s.tiles * s.rows : p.seqs) + 1), 256) * 256);
    p.flops = 2 * p.seqs * p.S * (p.K + p.C);
    p.bytes = p.seqs * (p.K * elem(x.dtype) + p.C * e * (1 + k.has(LM_Z)) + 4 + (f8 ? 4 : 0)) + std::min(E, p.seqs) * p.S * (p.K + p.C) * e;
    return k.status;
}

}  // namespace

int lm_plan_layer(int op, Checker &k, const lm_args &args, lm_plan_t &p)
{
    const conv_tensor &x = k.t[LM_X];
    if (args.max_len < 0 || args.chunk < 0 || args.flags) return k.fail(CONV_EINVAL, "unknown flags or negative lengths"), k.status;
    if (op == LM_ADAPTERS || op == LM_NORM || op == LM_NORM_BWD) {
        if (args.max_len || args.chunk) return k.fail(CONV_EINVAL, "no lengths or chunks in this operator"), k.status;
    }
    if (op == LM_ADAPTERS) return plan_adapters(k, p);
    if (x.rank > 0 && x.dtype != CONV_F32 && x.dtype != CONV_F16 && x.dtype != CONV_BF16)
        return k.fail(CONV_EINVAL, "x has to be float32, float16 or bfloat16"), k.status;
    p.dtype = x.dtype;
    return op == LM_NORM || op == LM_NORM_BWD ? plan_norm(op, k, args, p) : plan_gated(op, k, args, p);
}

}  // namespace miconv
