// The short causal convolution of a sequence, its gradients and its step for
// single tokens:
//   p[c,t] = b[c] + sum_{k<K} w[c,k] xx[c, t-K+1+k],   y = act(p),
// xx the rows of x behind the K-1 values of the incoming state.
//
// Bound by memory: 2 K + 4 operations for 2 elements moved.  A thread owns V
// neighbouring channels and walks down a chunk of rows with the last K-1 rows,
// the weights and the bias in registers, so x is read once but for the K-1
// rows in front of each chunk.  Lanes lie along the channels: with channels
// contiguous a wave reads and writes whole lines (V elements per lane, at any
// element alignment); other strides take V = 1.
//
// Measured, bf16, K = 4: 4 x 2048 x 4096 in 28 us (4.9 TB/s; a large copy
// reaches 5.1); output and gradients of 8 x 2048 x 2048 in 88 us, of which the
// backward walk takes 55 (2 channels per thread and 64-row chunks; 4 channels
// and 32 rows read a seventh more and took 64).  In f32 the prompt takes 58 us
// (4.6 TB/s), with positions contiguous 240 and in bf16 234: lanes L elements
// apart use a word of each line they fetch.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {
namespace {

// Rows of a block: their loads are in flight while the block before is used.
constexpr int kRows = 8, kRowsBwd = 4;

struct ConvP {
    const void *x, *w, *b, *s0, *gy, *gs;
    void *y, *s1, *dx, *ds;
    float *part;
    const int32_t *off, *rows;
    S3 xs, ys, s0s, s1s, gys, gss, dxs, dss;
    int64_t ws_c, ws_k, bs;
    int64_t seqs, C, L, chunk, chunks, parts, cvs, state_rows;
    int silu, w_dense, slots;
};

// Where a thread works: chunk ch of sequence seq, which is chunk `part` of all,
// and the first channel.  Neighbouring threads take neighbouring channels; the
// last group of V is moved back inside C and repeats its neighbour's results.
// ch is -1 at a place between packed sequences that no chunk has.
struct ConvAt {
    int64_t seq, ch, c, part;
    SeqSpan sp;
};
template <int V> __device__ __forceinline__ bool conv_item(const ConvP &p, ConvAt &a)
{
    const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    a.part = divide(item, p.cvs, a.c);
    if (!p.slots && a.part >= p.parts) return false;
    // Out of the straight path, whose start would be half a us longer (prompt of
    // 4 x 2048 x 4096: 28.3 for 27.8).
    if (__builtin_expect(p.slots, 0)) {
        // The first lane's sequence by the whole wave, then on to the lane's own.
        const int part = (int)a.part;
        int seq, first;
        a.sp = seq_of_slot(p.off, (int)p.seqs, (int)p.L, (uint32_t)p.chunk, __builtin_amdgcn_readfirstlane(part), seq, first);
        while (seq + 1 < p.seqs && a.sp.start + a.sp.len < (part - seq) * p.chunk) {
            a.sp = seq_span(p.off, ++seq, p.L);
            first = (int)((uint32_t)a.sp.start / (uint32_t)p.chunk) + seq;
        }
        a.seq = seq, a.ch = part - first;
        if (a.ch * p.chunk >= a.sp.len && a.ch > 0) a.ch = -1;
    } else {
        a.seq = divide(a.part, p.chunks, a.ch);
        a.sp = seq_span(p.off, a.seq, p.L);
    }
    a.c *= V;
    if (a.c > p.C - V) a.c = p.C - V;
    return a.part < p.parts;
}
__device__ __forceinline__ int64_t chunk_end(const ConvP &p, const ConvAt &a)
{
    const int64_t end = (a.ch + 1) * p.chunk;
    return end < a.sp.len ? end : a.sp.len;
}

template <typename T, int V> __device__ __forceinline__ void get(const T *p, int64_t cs, float (&o)[V])
{
    if constexpr (V == 1) o[0] = to_f32(*p);
    else load_f32<T, V>(p, o);
}
template <typename T, int V> __device__ __forceinline__ void put(T *p, int64_t cs, const float (&v)[V])
{
    if constexpr (V == 1) *p = from_f32<T>(v[0]);
    else store_f32<T, V, true>(p, v);
}
// V channels of one row at any channel stride (state rows, parameters).
template <typename T, int V> __device__ __forceinline__ void get_strided(const T *p, int64_t cs, float (&o)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = to_f32(p[i * cs]);
}
template <typename T, int V> __device__ __forceinline__ void put_strided(T *p, int64_t cs, const float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) p[i * cs] = from_f32<T>(v[i]);
}

template <typename T, int K, int V>
__device__ __forceinline__ void get_weights(const ConvP &p, int64_t c, float (&w)[K][V], float (&b)[V])
{
    const T *wp = static_cast<const T *>(p.w) + c * p.ws_c;
    if (p.w_dense) {   // [C, K] without gaps: V K neighbouring elements
        float f[K * V];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            float v[V];
            get<T, V>(wp + i * V, 1, v);
#pragma unroll
            for (int j = 0; j < V; ++j) f[i * V + j] = v[j];
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) w[k][i] = f[i * K + k];
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) get_strided<T, V>(wp + k * p.ws_k, p.ws_c, w[k]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.f;
    if (p.b) get_strided<T, V>(static_cast<const T *>(p.b) + c * p.bs, p.bs, b);
}

// R rows of V channels from row t of a walk on, p at row t.  Rows past the last
// repeat it: behind a branch their registers would be waited for where the
// paths meet.
template <typename T, int V, int R>
__device__ __forceinline__ void get_rows(const T *p, int64_t stride, int64_t t, int64_t last, Raw<T, V> (&o)[R])
{
    const int left = last - t < R ? (int)(last - t) : R;
#pragma unroll
    for (int r = 0; r < R; ++r) o[r] = load_raw<T, V>(p + (r < left ? r : left) * stride);
}

// Row t of the extended input (t >= -(K-1)): x, the incoming state, or zero.
template <typename T, int K, int V>
__device__ __forceinline__ void get_front(const ConvP &p, int64_t seq, const T *x, int64_t c, int64_t t, float (&o)[V])
{
    if (t >= 0) get<T, V>(x + t * p.xs.l, p.xs.c, o);
    else {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.f;
        if (p.s0)
            get_strided<T, V>(static_cast<const T *>(p.s0) + seq * p.s0s.n + c * p.s0s.c + (K - 1 + t) * p.s0s.l, p.s0s.c,
                              o);
    }
}

template <typename T, int K, int V> __global__ __launch_bounds__(256) void conv_fwd(const ConvP p)
{
    ConvAt at;
    if (!conv_item<V>(p, at) || at.ch < 0) return;
    const SeqSpan sp = at.sp;
    const int64_t seq = at.seq, c = at.c, t0 = at.ch * p.chunk, t1 = chunk_end(p, at);
    const T *x0 = static_cast<const T *>(p.x) + sp.row0 * p.xs.n + c * p.xs.c + sp.start * p.xs.l;
    const T *x = x0 + t0 * p.xs.l;
    T *y = static_cast<T *>(p.y) + sp.row0 * p.ys.n + c * p.ys.c + (sp.start + t0) * p.ys.l;

    Raw<T, V> next[kRows];
    if (t0 < t1) get_rows(x, p.xs.l, t0, t1 - 1, next);
    float w[K][V], b[V];
    get_weights<T, K, V>(p, c, w, b);
    float h[K - 1 + kRows][V];   // the K-1 rows in front of the block, then the block
#pragma unroll
    for (int k = 0; k < K - 1; ++k) get_front<T, K, V>(p, seq, x0, c, t0 - (K - 1) + k, h[k]);
    for (int64_t t = t0; t < t1; t += kRows) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) h[K - 1 + r][i] = next[r].f(i);
        x += kRows * p.xs.l;
        get_rows(x, p.xs.l, t + kRows, t1 - 1, next);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (t + r >= t1) break;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float a = b[i];
#pragma unroll
                for (int k = 0; k < K; ++k) a = __builtin_fmaf(w[k][i], h[r + k][i], a);
                o[i] = p.silu ? silu(a) : a;
            }
            put<T, V>(y + r * p.ys.l, p.ys.c, o);
        }
        y += kRows * p.ys.l;
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) h[k][i] = h[kRows + k][i];
    }
    if (K > 1 && p.s1 && t1 == sp.len) {
        T *s1 = static_cast<T *>(p.s1) + seq * p.s1s.n + c * p.s1s.c;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            float v[V];
            get_front<T, K, V>(p, seq, x0, c, t1 - (K - 1) + k, v);
            put_strided<T, V>(s1 + k * p.s1s.l, p.s1s.c, v);
        }
    }
}

// One token for each batch row; the state row moves up by one in place.
template <typename T, int K, int V> __global__ __launch_bounds__(256) void conv_step(const ConvP p)
{
    ConvAt at;
    if (!conv_item<V>(p, at)) return;
    const int64_t n = at.seq, c = at.c;
    T *y = static_cast<T *>(p.y) + n * p.ys.n + c * p.ys.c;
    int64_t row = n;
    if (p.rows) {
        row = p.rows[n];
        if (row < 0 || row >= p.state_rows) {
            const float zero[V] = {};
            put_strided<T, V>(y, p.ys.c, zero);
            return;
        }
    }
    const T *x = static_cast<const T *>(p.x) + n * p.xs.n + c * p.xs.c;
    T *st = static_cast<T *>(p.s1) + row * p.s1s.n + c * p.s1s.c;
    float h[K][V], w[K][V], b[V], o[V];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        if (p.s1s.c == 1) get<T, V>(st + k * p.s1s.l, 1, h[k]);
        else get_strided<T, V>(st + k * p.s1s.l, p.s1s.c, h[k]);
    }
    if (p.xs.c == 1) get<T, V>(x, 1, h[K - 1]);
    else get_strided<T, V>(x, p.xs.c, h[K - 1]);
    get_weights<T, K, V>(p, c, w, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float a = b[i];
#pragma unroll
        for (int k = 0; k < K; ++k) a = __builtin_fmaf(w[k][i], h[k][i], a);
        o[i] = p.silu ? silu(a) : a;
    }
    if (p.ys.c == 1) put<T, V>(y, 1, o);
    else put_strided<T, V>(y, p.ys.c, o);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        if (p.s1s.c == 1) put<T, V>(st + k * p.s1s.l, 1, h[k + 1]);
        else put_strided<T, V>(st + k * p.s1s.l, p.s1s.c, h[k + 1]);
    }
}

// Gradients in one walk, a block of rows at a time: the pre-activations are
// recomputed from x, g = gy act'(p) joins the K-1 rows of g before the block,
// dx leaves K-1 rows behind it, and dw, db gather over the chunk's own rows.
// The walk runs K-1 rows past the chunk for dx (their dw belongs to the next
// chunk).  The sums of a chunk go to part [number of the chunk][C][K+1];
// conv_bwd_sums adds them in a fixed order.
template <typename T, int K, int V> __global__ __launch_bounds__(256) void conv_bwd(const ConvP p)
{
    constexpr int R = kRowsBwd;
    ConvAt at;
    if (!conv_item<V>(p, at)) return;
    float *part = p.part ? p.part + (at.part * p.C + at.c) * (K + 1) : nullptr;
    if (at.ch < 0) {
        if (part) {
#pragma unroll
            for (int i = 0; i < V * (K + 1); ++i) part[i] = 0.f;
        }
        return;
    }
    const SeqSpan sp = at.sp;
    const int64_t seq = at.seq, ch = at.ch, c = at.c, t0 = ch * p.chunk, t1 = chunk_end(p, at);
    float dw[K][V] = {}, db[V] = {};
    const T *x0 = static_cast<const T *>(p.x) + sp.row0 * p.xs.n + c * p.xs.c + sp.start * p.xs.l;
    const T *x = x0 + t0 * p.xs.l;
    const T *gy = static_cast<const T *>(p.gy) + sp.row0 * p.gys.n + c * p.gys.c + (sp.start + t0) * p.gys.l;
    // Where the row of the gradient that the block's first row completes goes.
    T *dx = p.dx ? static_cast<T *>(p.dx) + sp.row0 * p.dxs.n + c * p.dxs.c + (sp.start + t0 - (K - 1)) * p.dxs.l : nullptr;
    const int64_t end = t1 + (K - 1);                       // rows walked
    const int64_t has = end < sp.len ? end : sp.len;        // rows that exist
    Raw<T, V> nx[R], ng[R];
    if (has > 0) get_rows(x, p.xs.l, t0, has - 1, nx), get_rows(gy, p.gys.l, t0, has - 1, ng);
    float w[K][V], b[V];
    get_weights<T, K, V>(p, c, w, b);
    float h[K - 1 + R][V], g[K - 1 + R][V];   // the K-1 rows in front of the block, then the block
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        get_front<T, K, V>(p, seq, x0, c, t0 - (K - 1) + k, h[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) g[k][i] = 0.f;
    }
    for (int64_t t = t0; t < end; t += R) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) h[K - 1 + r][i] = nx[r].f(i), g[K - 1 + r][i] = ng[r].f(i);
        if (has > 0) {
            x += R * p.xs.l, gy += R * p.gys.l;
            get_rows(x, p.xs.l, t + R, has - 1, nx), get_rows(gy, p.gys.l, t + R, has - 1, ng);
        }
        // MASK: rows past the chunk's end, at most in its last blocks.
        const auto gather = [&](auto masked) {
            constexpr bool MASK = decltype(masked)::value;
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float v = g[K - 1 + r][i];
                    if (p.silu) {
                        float a = b[i];
#pragma unroll
                        for (int k = 0; k < K; ++k) a = __builtin_fmaf(w[k][i], h[r + k][i], a);
                        v *= silu_slope(a, sigmoid(a));
                    }
                    if (MASK && t + r >= has) v = 0.f;
                    g[K - 1 + r][i] = v;
                    if (MASK && t + r >= t1) continue;
                    db[i] += v;
#pragma unroll
                    for (int k = 0; k < K; ++k) dw[k][i] = __builtin_fmaf(v, h[r + k][i], dw[k][i]);
                }
            }
        };
        if (t + R <= t1) gather(std::false_type());
        else gather(std::true_type());
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t to = t + r - (K - 1);   // the row whose gradient is complete
            if (to >= t1) break;
            if (to < t0 && !(ch == 0 && to < 0)) continue;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                o[i] = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) o[i] = __builtin_fmaf(w[k][i], g[K - 1 + r - k][i], o[i]);
            }
            if (p.gs && to >= sp.len - (K - 1)) {
                float v[V];
                get_strided<T, V>(static_cast<const T *>(p.gs) + seq * p.gss.n + c * p.gss.c +
                                      (to - (sp.len - (K - 1))) * p.gss.l,
                                  p.gss.c, v);
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] += v[i];
            }
            if (to >= 0) {
                if (dx) put<T, V>(dx + r * p.dxs.l, p.dxs.c, o);
            } else if (p.ds) {
                put_strided<T, V>(static_cast<T *>(p.ds) + seq * p.dss.n + c * p.dss.c + (K - 1 + to) * p.dss.l,
                                  p.dss.c, o);
            }
        }
        if (dx) dx += R * p.dxs.l;
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) h[k][i] = h[R + k][i], g[k][i] = g[R + k][i];
    }
    if (part) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int k = 0; k < K; ++k) part[i * (K + 1) + k] = dw[k][i];
            part[i * (K + 1) + K] = db[i];
        }
    }
}

// Sums of the chunks' parts: 64 outputs (of C (K+1)) per workgroup, a
// sixteenth of the parts per wave, joined in a fixed order.
template <typename T>
__global__ __launch_bounds__(1024) void conv_bwd_sums(const float *part, int64_t parts, int64_t C, int K, T *dw,
                                                      int64_t dws_c, int64_t dws_k, T *db, int64_t dbs)
{
    __shared__ float sh[16][64];
    const int64_t out = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63), n = C * (K + 1);
    const int q = threadIdx.x >> 6;
    float a[4] = {};
    if (out < n) {
        const int64_t lo = parts * q / 16, hi = parts * (q + 1) / 16;
        int64_t i = lo;
        for (; i + 4 <= hi; i += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] += part[(i + j) * n + out];
        for (; i < hi; ++i) a[0] += part[i * n + out];
    }
    sh[q][threadIdx.x & 63] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (q == 0 && out < n) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += sh[i][threadIdx.x];
        int64_t k;
        const int64_t c = divide(out, K + 1, k);
        if (k < K) {
            if (dw) dw[c * dws_c + k * dws_k] = from_f32<T>(v);
        } else if (db) db[c * dbs] = from_f32<T>(v);
    }
}

S3 s3(const conv_tensor &t) { return {t.strides[0], t.strides[1], t.rank > 2 ? t.strides[2] : 0}; }

ConvP base(const lm_plan_t &p, lm_ptrs q)
{
    ConvP a = {};
    a.x = q[LM_X], a.w = q[LM_W], a.b = q[LM_BIAS], a.s0 = q[LM_STATE_IN], a.gy = q[LM_GY], a.gs = q[LM_GSTATE];
    a.y = q[LM_Y], a.s1 = q[LM_STATE_OUT], a.dx = q[LM_DX], a.ds = q[LM_DSTATE];
    a.off = static_cast<const int32_t *>(q[LM_OFFSETS]);
    a.rows = static_cast<const int32_t *>(q[LM_ROWS]);
    a.xs = s3(p.t[LM_X]), a.ys = s3(p.t[LM_Y]), a.s0s = s3(p.t[LM_STATE_IN]), a.s1s = s3(p.t[LM_STATE_OUT]);
    a.gys = s3(p.t[LM_GY]), a.gss = s3(p.t[LM_GSTATE]), a.dxs = s3(p.t[LM_DX]), a.dss = s3(p.t[LM_DSTATE]);
    a.ws_c = p.t[LM_W].strides[0], a.ws_k = p.t[LM_W].strides[1], a.bs = p.t[LM_BIAS].strides[0];
    a.seqs = p.seqs, a.C = p.C, a.L = p.L, a.chunk = p.chunk, a.chunks = p.chunks, a.parts = lm_parts(p);
    a.slots = lm_slots(p);
    if (p.chunks == 1) a.chunk = int64_t(1) << 62;   // whole sequences, also longer ones than expected
    a.state_rows = p.t[LM_STATE_OUT].sizes[0];
    a.silu = (p.args.flags & LM_SILU) != 0;
    a.w_dense = a.ws_c == p.K && (a.ws_k == 1 || p.K == 1);
    return a;
}

int blocks_of(ConvP &a, int V)
{
    a.cvs = lm_cdiv(a.C, V);
    return (int)lm_cdiv(a.cvs * a.parts, 256);
}

// f(k) for the tap count as a constant.
template <typename F> void with_taps(int64_t K, F f)
{
    switch (K) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 5: f(std::integral_constant<int, 5>()); break;
    case 6: f(std::integral_constant<int, 6>()); break;
    case 7: f(std::integral_constant<int, 7>()); break;
    case 8: f(std::integral_constant<int, 8>()); break;
    }
}

template <typename T> void fwd(const lm_plan_t &p, ConvP a, hipStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    const bool vec = conv_width(p) == V;
    with_taps(p.K, [&](auto k) {
        constexpr int K = decltype(k)::value;
        if (vec) {
            const int g = blocks_of(a, V);
            if (g) conv_fwd<T, K, V><<<g, 256, 0, s>>>(a);
        } else {
            const int g = blocks_of(a, 1);
            if (g) conv_fwd<T, K, 1><<<g, 256, 0, s>>>(a);
        }
    });
}

template <typename T> void step(const lm_plan_t &p, ConvP a, hipStream_t s)
{
    with_taps(p.K, [&](auto k) {
        constexpr int K = decltype(k)::value;
        if (conv_width(p) == 2) {
            const int g = blocks_of(a, 2);
            if (g) conv_step<T, K, 2><<<g, 256, 0, s>>>(a);
        } else {
            const int g = blocks_of(a, 1);
            if (g) conv_step<T, K, 1><<<g, 256, 0, s>>>(a);
        }
    });
}

template <typename T> void bwd(const lm_plan_t &p, ConvP a, lm_ptrs q, hipStream_t s)
{
    constexpr int V = 2;
    const bool vec = conv_width(p) == V;
    with_taps(p.K, [&](auto k) {
        constexpr int K = decltype(k)::value;
        if (vec) {
            const int g = blocks_of(a, V);
            if (g) conv_bwd<T, K, V><<<g, 256, 0, s>>>(a);
        } else {
            const int g = blocks_of(a, 1);
            if (g) conv_bwd<T, K, 1><<<g, 256, 0, s>>>(a);
        }
    });
    if (q[LM_DW] || q[LM_DBIAS]) {
        const conv_tensor &w = p.t[LM_DW], &b = p.t[LM_DBIAS];
        conv_bwd_sums<T><<<(int)lm_cdiv(p.C * (p.K + 1), 64), 1024, 0, s>>>(
            a.part, a.parts, p.C, (int)p.K, static_cast<T *>(q[LM_DW]), w.strides[0], w.strides[1],
            static_cast<T *>(q[LM_DBIAS]), b.strides[0]);
    }
}

}  // namespace

int launch_lm_conv(const lm_plan_t &p, lm_ptrs q, hipStream_t s)
{
    const ConvP a = base(p, q);
    if (p.dtype == CONV_F32) fwd<float>(p, a, s);
    else if (p.dtype == CONV_F16) fwd<f16_t>(p, a, s);
    else fwd<bf16_t>(p, a, s);
    return lm_launch_status();
}

int launch_lm_conv_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s)
{
    const ConvP a = base(p, q);
    if (p.dtype == CONV_F32) step<float>(p, a, s);
    else if (p.dtype == CONV_F16) step<f16_t>(p, a, s);
    else step<bf16_t>(p, a, s);
    return lm_launch_status();
}

int launch_lm_conv_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    ConvP a = base(p, q);
    a.part = q[LM_DW] || q[LM_DBIAS] ? static_cast<float *>(ws) : nullptr;
    if (p.dtype == CONV_F32) bwd<float>(p, a, q, s);
    else if (p.dtype == CONV_F16) bwd<f16_t>(p, a, q, s);
    else bwd<bf16_t>(p, a, q, s);
    return lm_launch_status();
}

}  // namespace miconv
