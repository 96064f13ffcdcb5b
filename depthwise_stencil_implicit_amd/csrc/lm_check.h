// Checks of the sequence operators' descriptors, shared by the planners.
#pragma once

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "lm_internal.h"

namespace miconv {

inline const char *const kNames[LM_NSLOT] = {
    "x",   "w", "bias", "y", "state_in", "state_out", "offsets", "gy",  "gstate",  "dx",     "dw",   "dbias",  "dstate", "dt",
    "A",   "B", "C",    "D", "z",        "dt_bias",   "ddt",     "dA",  "dB",      "dC",     "dD",   "dz",     "ddt_bias",
    "saved", "rows", "scales", "zeros"};

inline int64_t elem(int32_t dtype)
{
    switch (dtype) {
    case CONV_F32: case LM_I32: return 4;
    case CONV_F16: case CONV_BF16: return 2;
    case LM_U8: case LM_F8: return 1;
    default: return 0;
    }
}

struct Checker {
    const conv_tensor *t;
    char *err;
    size_t len;
    int status = CONV_OK;

    bool fail(int st, const char *fmt, ...) __attribute__((format(printf, 3, 4)))
    {
        if (status == CONV_OK) {
            status = st;
            if (err && len) {
                va_list ap;
                va_start(ap, fmt);
                vsnprintf(err, len, fmt, ap);
                va_end(ap);
            }
        }
        return false;
    }
    bool has(int s) const { return t[s].rank > 0; }
    // Tensor s with these sizes and type; present unless optional.
    bool want(int s, int32_t dtype, std::initializer_list<int64_t> sizes, bool optional = false)
    {
        if (status != CONV_OK) return false;
        const conv_tensor &d = t[s];
        if (!has(s)) return optional ? true : fail(CONV_EINVAL, "%s is missing", kNames[s]);
        if (d.rank != (int)sizes.size()) return fail(CONV_EINVAL, "%s has %d dims, %d expected", kNames[s], d.rank, (int)sizes.size());
        if (d.dtype != dtype) return fail(CONV_EINVAL, "%s has another element type than the call needs", kNames[s]);
        int i = 0;
        for (int64_t v : sizes) {
            if (d.sizes[i] != v)
                return fail(CONV_EINVAL, "%s has size %lld in dim %d, %lld expected", kNames[s], (long long)d.sizes[i], i, (long long)v);
            if (d.strides[i] < 0) return fail(CONV_EINVAL, "%s has a negative stride", kNames[s]);
            ++i;
        }
        return true;
    }
    // An output has no two elements in one place.
    bool output(int s)
    {
        if (status != CONV_OK || !has(s)) return status == CONV_OK;
        const conv_tensor &d = t[s];
        int order[CONV_MAX_RANK], n = 0;
        for (int i = 0; i < d.rank; ++i) {
            if (d.sizes[i] == 0) return true;
            if (d.sizes[i] > 1) order[n++] = i;
        }
        std::sort(order, order + n, [&](int a, int b) { return d.strides[a] < d.strides[b]; });
        int64_t span = 1;
        for (int i = 0; i < n; ++i) {
            if (d.strides[order[i]] < span) return fail(CONV_EINVAL, "output %s overlaps itself", kNames[s]);
            span = (d.sizes[order[i]] - 1) * d.strides[order[i]] + span;
        }
        return true;
    }
};

// Rows per chunk that the caller asks for (0: none), no more than there are.
inline int64_t forced_rows(const lm_plan_t &p, int64_t max_len)
{
    return std::min(p.args.chunk, std::max<int64_t>(max_len, 1));
}

// Plans of the recurrence, the norm and the adapters; `k` has looked at every
// descriptor's rank and sizes.
int lm_plan_layer(int op, Checker &k, const lm_args &args, lm_plan_t &p);

}  // namespace miconv
