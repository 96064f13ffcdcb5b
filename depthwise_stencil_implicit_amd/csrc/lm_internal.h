// Host-side internals of the sequence operators: the plan's limits and the
// launchers, one per operator.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "../../include/miconv_lm.h"

namespace miconv {

constexpr int LM_MAX_TAPS = 8;
constexpr int LM_MAX_STATES = 64;

// Scan: channels of one workgroup, steps of one staged tile.
constexpr int LM_SCAN_CH = 64;
constexpr int LM_SCAN_TB = 32;

// States per lane: four lanes share a channel.
inline int scan_ns(int64_t S)
{
    int ns = 1;
    while (4 * ns < S) ns *= 2;
    return ns;
}
// Steps between saved states, the length the backward kernel keeps in
// registers: 64 values of exp(d A) per lane.
inline int scan_save_steps(int64_t S) { return scan_ns(S) <= 4 ? 16 : 64 / scan_ns(S); }
inline int64_t lm_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
