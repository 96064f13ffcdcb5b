// Host-side internals of the sequence operators: the plan's limits and the
// launchers, one per operator.
#pragma once

#include <hip/hip_runtime_api.h>

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

typedef void *const *lm_ptrs;
int launch_lm_conv(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_conv_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_conv_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_scan(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_scan_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);
int launch_lm_scan_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s);
int launch_lm_mv4(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s);

inline int lm_launch_status() { return hipGetLastError() == hipSuccess ? CONV_OK : CONV_EDEVICE; }

}  // namespace miconv
