// Host-side internals of the sequence operators: the plan's limits and the
// launchers, one per operator.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "../../include/miconv_lm.h"

namespace miconv {

constexpr int LM_MAX_TAPS = 8;
constexpr int LM_MAX_STATES = 64;

// Scan: channels of one workgroup; how S states lie over lanes.  Four rows of
// 16 lanes share a channel, eight above 16 states; each holds ns of them.
constexpr int LM_SCAN_CH = 64;
struct ScanShape {
    int ns, qw;                                       // states per lane, core waves per 16 channels
    constexpr int width() const { return 4 * qw * ns; }                       // states with padding
    constexpr int save_steps() const { return qw == 1 ? 16 : 32 / ns; }       // steps between saved states
};
inline ScanShape scan_shape(int64_t S)
{
    const int qw = S <= 16 ? 1 : 2;
    int ns = 1;
    while (4 * qw * ns < S) ns *= 2;
    return {ns, qw};
}
inline int64_t lm_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Chunks of all sequences of a call.  Packed sequences that may have several
// number theirs start / chunk + sequence on: ceil(length / chunk), or one, fit
// before the next one's first, so L / chunk + sequences places hold them all
// however unlike the lengths are (sequences times the longest one's chunks grow
// with the product: the gradients of 300 f16 sequences in 9000 x 1024 without a
// max_len took 1250 us, and 36 so).  A place that no chunk has adds zeros to
// sums.  A sequence longer than max_len has its rest in the last chunk only
// where one chunk is planned for each.
inline bool lm_slots(const lm_plan_t &p) { return p.t[LM_OFFSETS].rank > 0 && p.chunks > 1; }
inline int64_t lm_parts(const lm_plan_t &p)
{
    return lm_slots(p) ? (p.seqs > 0 ? p.L / p.chunk + p.seqs : 0) : p.seqs * p.chunks;
}
// Channels of a convolution's thread: 16 bytes of contiguous ones, or one.  The
// backward walk's registers hold two.  A step takes two, enough threads for
// small batches, but one of an odd number: the state moves in place, so no two
// threads may share a channel.
inline int conv_width(const lm_plan_t &p)
{
    if (p.op == LM_CONV_STEP) return p.C % 2 ? 1 : 2;
    const int V = p.op == LM_CONV_BWD ? 2 : p.dtype == CONV_F32 ? 4 : 8;
    for (int s : {LM_X, LM_Y, LM_GY, LM_DX})
        if (p.t[s].rank && p.t[s].strides[1] != 1) return 1;
    return p.C >= V ? V : 1;
}
// States (gradients) between the scan's chunks: the forward pass needs none of
// a sequence's last one.
inline int64_t scan_carries(const lm_plan_t &p)
{
    return p.op == LM_SCAN && !lm_slots(p) ? p.seqs * (p.chunks - 1) : lm_parts(p);
}

// 4-bit products: bytes of x made contiguous (0: x's rows are), and the parts
// of the columns whose x fits the registers of 16 waves -- four blocks of 128
// columns each for 16-bit types, one for f32 (three terms).  0 parts: weights or scales that
// the register kernel does not take.
inline int64_t mv4_rows_bytes(const lm_plan_t &p)
{
    const int64_t bytes = p.seqs * p.K * (p.dtype == CONV_F32 ? 4 : 2);
    return p.t[LM_X].strides[1] != 1 && p.K > 1 ? lm_cdiv(bytes, 256) * 256 : 0;
}
inline int mv4_parts(const lm_plan_t &p)
{
    const int64_t group = p.K / p.G, blocks = lm_cdiv(p.K, 128);
    for (int s : {LM_SCALES, LM_ZEROS})
        if (p.t[s].rank && p.G > 1 && p.t[s].strides[1] != 1) return 0;
    for (int s : {LM_W, LM_SCALES, LM_ZEROS})   // offsets of 32 bits
        if (p.t[s].rank && p.t[s].strides[0] > 0x7fffffff / (p.C + 1)) return 0;
    if (p.C > 0x7fffff00 || p.K < 128 || blocks >= 1024 || (group % 128 && group != 64 && group != 32)) return 0;
    return (int)lm_cdiv(blocks, p.dtype == CONV_F32 ? 16 : p.K % 128 ? 32 : 64);
}

// The recurrence: rows of a workgroup's tile, steps between saved states,
// channels of a thread (two of 16 bits make a word; other memory orders take
// one, as do single channels).
constexpr int LM_GATED_TILE = 128, LM_GATED_SAVE = 64;
inline bool gated_look(const lm_plan_t &p) { return p.op == LM_GATED && p.chunks > 1; }   // tile by tile over the axis
inline int gated_width(const lm_plan_t &p)
{
    if (p.dtype == CONV_F32 || p.C < 2) return 1;
    for (int s : {LM_X, LM_A, LM_B, LM_Y, LM_GY, LM_DX, LM_DA, LM_DB})
        if (p.t[s].rank && p.t[s].strides[1] != 1) return 1;
    return 2;
}
// Of a step's thread: two of any type, but one of an odd number (the state moves
// in place, so no two threads may share a channel).
inline int gated_step_width(const lm_plan_t &p) { return p.C % 2 ? 1 : 2; }

// The norm: channels that a workgroup's registers hold, workgroups of the
// gradients, each of which leaves one row of dw's sums.
constexpr int LM_NORM_MAX = 65536;
inline int norm_threads(int64_t rows, int64_t C)   // threads of a row
{
    if (rows >= 2048) return C <= 2048 ? 64 : C <= 16384 ? 256 : 1024;
    return C <= 512 ? 64 : C <= 4096 ? 256 : 1024;
}
inline int64_t norm_bwd_groups(const lm_plan_t &p)
{
    const int64_t rows = p.seqs * p.L, t = norm_threads(rows, p.C), per = t == 64 ? 4 : 1;
    return std::max<int64_t>(1, std::min<int64_t>(lm_cdiv(rows, per), t == 1024 ? 256 : 1024));
}

// Adapters: rows of a workgroup (1: those of its row's adapter, gathered),
// tiles of that many (rows of one adapter, so each may leave one short), parts of
// the columns of x, 256s of outputs of a workgroup, width of a row of inner sums.
// About one workgroup of adapters_in for each compute unit (with two it took 26
// us for 21 of 4096 rows and rank 64) and three of adapters_out (8192 rows and
// outputs, rank 32: 70 us; with one 79, two 73, four 70).
//
// Up to LM_ADAPTER_FEW rows are gathered, up to LM_ADAPTER_FIND of few adapters (a
// lane counts each, and the rows without) found by each workgroup of adapters_in,
// others sorted in a launch before it: 8192 rows, 4096 columns and outputs, 32
// adapters, sorted 54 us in runs and 87 in any order, found 49 and 76.  FIND is what
// a workgroup's registers hold of index, 32 a lane, and COUNTED what its lanes do,
// not where the sort would win: 63 adapters in any order, found, against 64, sorted,
// took 129 us against 152 there, but 192 against 149 with 2048 columns and outputs
// and rank 64, where counting is more of the work.  Tiles of 64
// beat the gathered 16 where adapters have 16 rows or more and the rows are long
// (200 rows of 8 adapters, 4096 columns and outputs: 18 us for 21; 1024: 16 for 12;
// of 40 adapters 4096: 30 for 18).
constexpr int LM_MAX_RANK = 256, LM_ADAPTER_N = 256, LM_ADAPTER_FEW = 512, LM_ADAPTER_TILE = 64;
constexpr int LM_ADAPTER_FIND = 8192, LM_ADAPTER_COUNTED = 63;
struct AdapterShape { int rows, parts, reps, width; int64_t tiles; bool find; };
inline bool adapter_dense_in(const lm_plan_t &p) { return (p.t[LM_X].strides[1] == 1 && p.t[LM_A].strides[2] == 1) || p.K == 1; }
inline AdapterShape adapter_shape(const lm_plan_t &p)
{
    AdapterShape s;
    const bool counted = p.G > 0 && p.G <= LM_ADAPTER_COUNTED && p.seqs <= LM_ADAPTER_FIND && adapter_dense_in(p);
    const bool few = p.seqs <= LM_ADAPTER_FEW && !(counted && p.seqs >= 16 * p.G && p.seqs * (p.K + p.C) > 1 << 20);
    s.rows = few ? 1 : LM_ADAPTER_TILE;
    s.tiles = few ? p.seqs : p.seqs / s.rows + std::min(p.seqs, p.G + 1);
    s.find = counted && !few;
    // Workgroups with work: gathered, one for each adapter and each 16 rows; of
    // tiles, one for each 64 rows, or for an eighth of the adapters where those are
    // more (4096 columns and outputs, rank 16, 1000 adapters: 513 rows 83 us for 185,
    // 1024 rows 115 for 284).  How many of them the rows name is not known here
    // (with 6 of the 1000 named 513 rows take 34 us for 31, 1024 rows 35 for 47).
    const int64_t groups =
        std::max<int64_t>(1, few ? std::min(p.seqs, p.G + p.seqs / 16) : std::max(lm_cdiv(p.seqs, s.rows), std::min(p.seqs, p.G / 8)));
    s.parts = (int)std::max<int64_t>(1, std::min<int64_t>({lm_cdiv(256, groups), lm_cdiv(p.K, 256), 16}));
    const int64_t most = p.S <= 32 ? 768 : 384;   // the more ranks, the longer what each of them does first
    const int64_t blocks = std::max<int64_t>(1, lm_cdiv(p.C, LM_ADAPTER_N)), with_work = few ? groups : 2 * groups;
    // Gathered, rows whose adapter an earlier one takes start workgroups that end
    // at once, 3 ns each (500 rows of 8 adapters, 4096 outputs: 27 us for 33).
    const int64_t launched = few ? lm_cdiv(4096, std::max<int64_t>(p.seqs, 1)) : blocks;
    const int64_t spans = std::max<int64_t>(1, std::min<int64_t>({blocks, launched, (most + with_work / 2) / with_work}));
    s.reps = (int)lm_cdiv(blocks, spans);
    s.width = (int)lm_cdiv(p.S, 32) * 32;
    return s;
}
inline int64_t adapter_sums_bytes(const lm_plan_t &p)
{
    const AdapterShape s = adapter_shape(p);
    return lm_cdiv(4 * p.seqs * s.parts * s.width, 256) * 256;
}

typedef void *const *lm_ptrs;
int launch_lm_conv(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_conv_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_conv_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_scan(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_scan_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_scan_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_gated(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_gated_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_gated_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_norm(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_norm_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_adapters(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_mv4(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);

inline int lm_launch_status() { return hipGetLastError() == hipSuccess ? CONV_OK : CONV_EDEVICE; }

}  // namespace miconv
