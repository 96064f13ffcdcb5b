// The gated linear recurrence, its gradients and its step for single tokens:
//   k = value softplus(decay),  a = exp(-k sigmoid(r)),
//   h <- a h + sqrt(1 - a^2) sigmoid(i) x,   y = h.
//
// Bound by memory and the vector unit alike: 8 bytes (16-bit types) and about
// 46 issue slots per element, of which 24 are its six transcendentals; the
// gradients 14 bytes and about 100.  So everything is read once, and what the
// long axis needs is done on the chip: a workgroup owns 64 V neighbouring
// channels and walks down tiles of rows, each of its 16 waves taking a piece
// of the tile.  A piece is a map h -> P h + s; the waves leave (P, s) in LDS,
// and behind one barrier each folds those in front of it into its start and
// goes through its rows again, whose factors are still in registers.  Loads of
// the next tile are in flight meanwhile.  Lanes lie along the channels, so a
// wave reads whole lines of rows of channels.
//
// Few sequences leave units idle.  Forward, each tile is then a workgroup of its
// own (gated_tile): it holds its rows' factors in registers, puts its (P, s)
// where the tiles behind it look, finds what enters it from the sixteen tiles in
// front -- the nearest one whose end is known, and the maps of those since --
// and goes through its rows.  So the tensors are still read once (a first pass
// for the maps took 1 x 65536 x 2560 498 us).  Backward, a first pass over two of
// the seven tensors leaves the (P, s) of chunks, and a workgroup folds those
// behind its own.
//
// Measured (bf16, rows of channels; medians of traced kernels): 8 x 2048 x 4096
// whole sequences 118 us, 4.6 TB/s of the 5.1 that a copy reaches; 1 x 65536 x
// 2560 in tiles 370 us, 3.6 TB/s (and 7 to clear their words); gradients, 8 x 2048
// x 4096, 206 to 228 us, 4.1 to 4.6 TB/s.  What the tiles of 16-bit types lose,
// beside the wait for their loads and for the tiles in front: at 64 registers six
// are spilled, 16 bytes of a lane written and read again (330 MB on 1311), and
// each tile pays for the masks of the last one, 51 vector instructions an element
// for 32 of gated_fwd.  f32 spills none and takes 565 us, 1.08 of its bytes' time.
//
// Everything between load and store is f32; y and the gradients are rounded once.
// A state that has overflowed (an infinity in x) may come out as NaN further on
// where the map's P has run down to zero, h infinite: 0 times infinity.
//
// 1 - a^2 comes from a where a is clear of 1, and from four terms of the
// exponential's series where 2 k sigmoid(r) < 1/16: there a has lost what the
// difference needs.  Both are within 2^-19 at the seam.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_dev.h"
#include "lm_internal.h"

namespace miconv {
namespace {

constexpr int kWaves = 16;
constexpr int kFwd = LM_GATED_TILE / kWaves;   // rows of a wave
constexpr int kBwd = LM_GATED_SAVE / kWaves;

struct GatedP {
    const void *x, *r, *i, *gy;
    const float *decay, *s0, *gs;
    void *y, *dx, *dr, *di;
    float *s1, *ds, *saved, *dd;
    float *sums, *part;   // (P, s) of each chunk and channel; terms of ddecay
    uint64_t *ahead;      // tickets, then the (P, s) and the end of each tile
    const int32_t *off, *rows;
    S3 xs, rs, is, ys, gys, dxs, drs, dis;
    int64_t s0_n, s0_c, s1_n, s1_c, gs_n, gs_c, ds_n, ds_c, decay_c, dd_c;
    int64_t seqs, C, L, chunk, chunks, parts, state_rows;
    uint32_t blocks;
    int slots;
    float value;
};

// What a workgroup works on: chunk ch of sequence seq (ch = -1: a place between
// packed sequences that no chunk has), its rows t0 .. t1 of the sequence.
struct GatedAt {
    int64_t part, seq, ch, nch, first;   // first: the sequence's place among saved states
    SeqSpan sp;
    int64_t t0, t1;
};
__device__ __forceinline__ GatedAt gated_at(const GatedP &p, uint32_t group)
{
    GatedAt a;
    a.part = group / p.blocks;
    a.nch = p.chunks;
    if (p.slots) {
        int seq, first;
        a.sp = seq_of_slot(p.off, (int)p.seqs, (int)p.L, (uint32_t)p.chunk, (int)a.part, seq, first);
        a.seq = seq, a.ch = a.part - first, a.nch = chunks_of(a.sp.len, p.chunk);
        if (a.ch < 0 || a.ch >= a.nch) a.ch = -1;
    } else {
        a.seq = divide(a.part, p.chunks, a.ch);
        a.sp = seq_span(p.off, a.seq, p.L);
    }
    a.t0 = a.ch * p.chunk;
    // One chunk is the whole sequence, also one longer than max_len.
    a.t1 = p.chunks == 1 || a.t0 + p.chunk > a.sp.len ? a.sp.len : a.t0 + p.chunk;
    a.first = p.off ? a.sp.start / LM_GATED_SAVE + a.seq : a.seq * ((p.L + LM_GATED_SAVE - 1) / LM_GATED_SAVE);
    return a;
}

// The channels of a lane.  The last lanes' are moved back inside C and repeat
// their neighbours' results (`own`: they need not be stored).
template <int V> struct LaneAt {
    int64_t c;
    bool own;
    __device__ __forceinline__ LaneAt(const GatedP &p, uint32_t block)
    {
        c = (int64_t)block * 64 * V + (threadIdx.x & 63) * V;
        own = c < p.C;
        if (c > p.C - V) c = p.C - V;
    }
};

// A tensor's rows at a lane's channels: DENSE channels lie at 32-bit offsets
// from a place all lanes share.
template <typename T, int V, bool DENSE> struct RowsAt {
    T *base;
    int64_t step;
    typename std::conditional<DENSE, uint32_t, int64_t>::type at;
    template <typename P> __device__ __forceinline__ RowsAt(P *t, const S3 &st, const SeqSpan &sp, int64_t c, uint32_t block)
    {
        const int64_t c0 = DENSE ? (int64_t)block * 64 * V : 0;
        base = static_cast<T *>(const_cast<typename std::remove_const<P>::type *>(t)) + sp.row0 * st.n + sp.start * st.l;
        if (DENSE) {
            // The first lane's channels may be moved back too.
            base += c0 - V;
            at = (uint32_t)(c - c0 + V) * (uint32_t)sizeof(T);
        } else at = c * st.c * (int64_t)sizeof(T);
        step = st.l;
    }
    __device__ __forceinline__ T *row(int64_t t) const
    {
        return reinterpret_cast<T *>(reinterpret_cast<char *>(base + t * step) + at);
    }
};
template <typename T, int V> __device__ __forceinline__ void put(T *p, const float (&v)[V]) { store_f32<T, V>(p, v); }

// Rows t .. t + R - 1, those past the last one repeated: a load behind a branch
// would be waited for where the paths meet.  One address after the other: a
// product for each row kept the scalar unit busy for half of a tile's time.
template <typename T, int V, bool DENSE, int R>
__device__ __forceinline__ void get_rows(const RowsAt<T, V, DENSE> &p, int64_t t, int64_t last, Raw<T, V> (&o)[R])
{
    const int left = last - t < R ? (int)(last - t) : R;
    const T *row = p.base + (left < 0 ? last : t) * p.step;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        o[r] = load_raw<T, V>(reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) + p.at));
        row += r < left ? p.step : 0;
    }
}

// -k log2(e) of a lane's channels.
template <int V> __device__ __forceinline__ void get_rate(const GatedP &p, int64_t c, float (&k2)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) k2[v] = -kLog2e * p.value * softplus(p.decay[(c + v) * p.decay_c]);
}
// sqrt(1 - a^2) for t2 = log2(a) <= 0: with u = -2 ln2 t2, u - u^2/2 + u^3/6 -
// u^4/24 where u < 1/16.
__device__ __forceinline__ float complement(float t2, float a)
{
    constexpr float c = 2.f * kLn2;
    const float series = t2 * __builtin_fmaf(t2, __builtin_fmaf(t2, __builtin_fmaf(t2, -c * c * c * c / 24, -c * c * c / 6), -c * c / 2), -c);
    return __builtin_amdgcn_sqrtf(t2 > -0.0625f / c ? series : __builtin_fmaf(-a, a, 1.f));
}

// v through the maps (P, s) of `count` chunks from `first` on, eight loads at a
// time: one after the other they were 0.6 us each.
template <int V> __device__ __forceinline__ void fold(const GatedP &p, int64_t first, int step, int64_t count, int64_t c, float (&o)[V])
{
    const float2 *s = reinterpret_cast<const float2 *>(p.sums) + c;
    for (int64_t j = 0; j < count; j += 8) {
        float2 m[8][V];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) m[i][v] = s[(first + (j + i < count ? j + i : count - 1) * step) * p.C + v];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = j + i < count ? __builtin_fmaf(m[i][v].x, o[v], m[i][v].y) : o[v];
    }
}

// a and sqrt(1 - a^2) sigmoid(i) x of rows from t on, and their map: P and s go
// on from what they are.  Rows past the end leave everything as it is; a walk
// meets them in its last tile only.
template <int R, bool WALK, typename T, int V>
__device__ __forceinline__ void factors(const Raw<T, V> (&x)[R], const Raw<T, V> (&r)[R], const Raw<T, V> (&i)[R], const float (&k2)[V],
                                        int64_t t, int64_t end, float (&a)[R][V], float (&b)[R][V], float (&P)[V], float (&s)[V])
{
    const auto work = [&](auto cut) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool in = !decltype(cut)::value || t + j < end;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float t2 = k2[v] * sigmoid(r[j].f(v)), f = hw_exp2(t2);
                const float g = complement(t2, f) * sigmoid(i[j].f(v)) * x[j].f(v);
                a[j][v] = in ? f : 1.f, b[j][v] = in ? g : 0.f;
                P[v] *= a[j][v], s[v] = __builtin_fmaf(a[j][v], s[v], b[j][v]);
            }
        }
    };
    if (WALK && t + R <= end) work(std::false_type());
    else work(std::true_type());
}

// ---------------------------------------------------------------- forward --

// Whole sequences: bound by memory where 256 workgroups or more run.
template <typename T, int V, bool DENSE> __global__ __launch_bounds__(64 * kWaves) void gated_fwd(const GatedP p)
{
    __shared__ __attribute__((aligned(16))) float2 sums[2][kWaves][64 * V];
    __shared__ float carry[2][64 * V];
    constexpr int R = kFwd;
    const int waves = blockDim.x >> 6;   // 16 where there is more than a tile
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lv = (threadIdx.x & 63) * V;
    const GatedAt at = gated_at(p, blockIdx.x);
    const uint32_t block = blockIdx.x - (uint32_t)at.part * p.blocks;
    const LaneAt<V> lane(p, block);
    const int64_t c = lane.c;
    const RowsAt<T, V, DENSE> px(p.x, p.xs, at.sp, c, block), pr(p.r, p.rs, at.sp, c, block), pi(p.i, p.is, at.sp, c, block);

    Raw<T, V> nx[R], nr[R], ni[R];
    const int64_t w0 = at.t0 + wave * R;
    if (at.t0 < at.t1) get_rows(px, w0, at.t1 - 1, nx), get_rows(pr, w0, at.t1 - 1, nr), get_rows(pi, w0, at.t1 - 1, ni);
    float k2[V], h[V];
    get_rate<V>(p, c, k2);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if (wave == waves - 1) {   // this wave carries the state from tile to tile
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (p.s0) h[v] = p.s0[at.seq * p.s0_n + (c + v) * p.s0_c];
            carry[0][lv + v] = h[v];
        }
    }
    int buf = 0;
    for (int64_t t = at.t0; t < at.t1; t += LM_GATED_TILE, buf ^= 1) {
        const int64_t tw = t + wave * R;
        float a[R][V], b[R][V], P[V], s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) P[v] = 1.f, s[v] = 0.f;
        factors<R, true>(nx, nr, ni, k2, tw, at.t1, a, b, P, s);
        if (t + LM_GATED_TILE < at.t1) {
            const int64_t n = tw + LM_GATED_TILE;
            get_rows(px, n, at.t1 - 1, nx), get_rows(pr, n, at.t1 - 1, nr), get_rows(pi, n, at.t1 - 1, ni);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sums[buf][wave][lv + v] = make_float2(P[v], s[v]);
        lds_sync();
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = carry[buf][lv + v];
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 q = sums[buf][w][lv + v];
                h[v] = __builtin_fmaf(q.x, h[v], q.y);
            }
        if (p.saved && lane.own && (wave * R) % LM_GATED_SAVE == 0 && tw < at.t1) {
#pragma unroll
            for (int v = 0; v < V; ++v) p.saved[(at.first + tw / LM_GATED_SAVE) * p.C + c + v] = h[v];
        }
        const RowsAt<T, V, DENSE> py(p.y, p.ys, at.sp, c, block);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(a[r][v], h[v], b[r][v]);
            if (p.y && tw + r < at.t1 && lane.own) put<T, V>(py.row(tw + r), h);
        }
        if (wave == waves - 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) carry[buf ^ 1][lv + v] = h[v];
        }
    }
    if (wave != waves - 1 || !lane.own || !p.s1) return;
#pragma unroll
    for (int v = 0; v < V; ++v) p.s1[at.seq * p.s1_n + (c + v) * p.s1_c] = h[v];
}

// Words that tiles leave for those behind them: never all ones, which says that
// nothing has been left yet.  They carry their own validity, so atomics without
// an order do.
constexpr uint64_t kNothing = ~0ull;
constexpr int kTicket = 16;   // words between tickets: lines of their own
__device__ __forceinline__ uint64_t word_of(float a, float b)
{
    const uint32_t u = a != a ? 0x7fc00000u : __float_as_uint(a);
    return u | (uint64_t)__float_as_uint(b) << 32;
}
__device__ __forceinline__ void leave_word(uint64_t *p, uint64_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint64_t look(const uint64_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
// A wait that cannot end (offsets that do not ascend) is given up after this many
// looks, with NaN for a state: each is a load's wait, several hundred ns, so tens
// of ms in all where a tile takes tens of us.
constexpr int kPatience = 1 << 17;

__global__ __launch_bounds__(256) void gated_clear(const GatedP p, int64_t words)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, tickets = (int64_t)p.blocks * kTicket;
    if (i < tickets + words) p.ahead[i] = i < tickets ? 0 : kNothing;
}

// One tile of a sequence.  Two workgroups of 64 registers share a unit, so one's
// loads cover the other's wait.  Tiles of the same channels are taken by a ticket, so
// those that a tile waits for have been started before it, and each leaves its
// (P, s) before it waits itself: all waits end.
template <typename T, int V, bool DENSE> __global__ __launch_bounds__(64 * kWaves, 8) void gated_tile(const GatedP p)
{
    __shared__ __attribute__((aligned(16))) float2 sums[kWaves][64 * V];
    __shared__ __attribute__((aligned(16))) float2 front[kWaves][64 * V];
    __shared__ int reach, missing;
    __shared__ uint32_t ticket;
    constexpr int R = kFwd;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lv = (threadIdx.x & 63) * V;
    const uint32_t block = blockIdx.x % p.blocks;
    if (threadIdx.x == 0) ticket = atomicAdd(reinterpret_cast<uint32_t *>(p.ahead + (int64_t)block * kTicket), 1u);
    __syncthreads();
    const GatedAt at = gated_at(p, (uint32_t)__builtin_amdgcn_readfirstlane(ticket) * p.blocks);
    const LaneAt<V> lane(p, block);
    const int64_t c = lane.c, tw = at.t0 + wave * R;
    if (at.ch < 0) return;
    uint64_t *map_of = p.ahead + (int64_t)p.blocks * kTicket + at.part * p.C + c, *end_of = map_of + p.parts * p.C;
    float a[R][V], b[R][V], P[V], s[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, s[v] = 0.f;
    if (at.t0 < at.t1) {
        const RowsAt<T, V, DENSE> px(p.x, p.xs, at.sp, c, block), pr(p.r, p.rs, at.sp, c, block), pi(p.i, p.is, at.sp, c, block);
        Raw<T, V> nx[R], nr[R], ni[R];
        get_rows(pr, tw, at.t1 - 1, nr), get_rows(pi, tw, at.t1 - 1, ni), get_rows(px, tw, at.t1 - 1, nx);
        float k2[V];
        get_rate<V>(p, c, k2);
        factors<R, false>(nx, nr, ni, k2, tw, at.t1, a, b, P, s);
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v) a[r][v] = 1.f, b[r][v] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sums[wave][lv + v] = make_float2(P[v], s[v]);
    lds_sync();
    if (wave == kWaves - 1 && at.ch + 1 < at.nch) {   // the tile's map, for those behind it
#pragma unroll
        for (int v = 0; v < V; ++v) P[v] = 1.f, s[v] = 0.f;
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 q = sums[w][lv + v];
                s[v] = __builtin_fmaf(q.x, s[v], q.y), P[v] *= q.x;
            }
#pragma unroll
        for (int v = 0; v < V; ++v) leave_word(map_of + v, word_of(P[v], s[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = at.ch == 0 && p.s0 ? p.s0[at.seq * p.s0_n + (c + v) * p.s0_c] : 0.f;
    if (at.ch > 0) {
        const int near = at.ch < kWaves ? (int)at.ch : kWaves;
        for (int looks = 0;;) {   // the first wave's count
            // One channel's words tell how far to reach: to the nearest tile
            // whose end is there, over tiles whose maps are.
            if (wave == 0) {
                const int w = threadIdx.x & 15, back = w < near ? w : near - 1;
                const uint64_t *of = threadIdx.x & 16 ? map_of : end_of;
                int to = -1;
                while (looks++ < kPatience) {
                    const uint64_t there = __ballot(look(of - (back + 1) * p.C) != kNothing);
                    const int ends = (int)there & 0xffff & ((1 << near) - 1), maps = (int)(there >> 16) & 0xffff;
                    to = ends ? __builtin_ctz(ends) : -1;
                    if (to >= 0 && (maps & ((1 << to) - 1)) == (1 << to) - 1) break;
                    to = -1;
                }
                reach = to, missing = 0;
            }
            lds_sync();
            const int to = __builtin_amdgcn_readfirstlane(reach);
            if (to < 0) break;
            if (wave <= to) {
                const uint64_t *of = (wave < to ? map_of : end_of) - (wave + 1) * p.C;
                bool here = true;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint64_t m = look(of + v);
                    here = here && m != kNothing;
                    front[wave][lv + v] = make_float2(__uint_as_float((uint32_t)m), __uint_as_float((uint32_t)(m >> 32)));
                }
                if (__ballot(!here) != 0) missing = 1;
            }
            lds_sync();
            const bool again = __builtin_amdgcn_readfirstlane(missing) != 0;
            if (!again) {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = front[to][lv + v].x;
                for (int w = to - 1; w >= 0; --w)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float2 q = front[w][lv + v];
                        h[v] = __builtin_fmaf(q.x, h[v], q.y);
                    }
                break;
            }
            lds_sync();
        }
        if (__builtin_amdgcn_readfirstlane(reach) < 0)
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = __builtin_nanf("");
    }
    // The end by the map, not by the rows: what a tile behind finds then does
    // not depend on how far it has had to reach.
    if (wave == kWaves - 1 && at.ch + 1 < at.nch) {
#pragma unroll
        for (int v = 0; v < V; ++v) leave_word(end_of + v, word_of(__builtin_fmaf(P[v], h[v], s[v]), 0.f));
    }
    for (int w = 0; w < wave; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 q = sums[w][lv + v];
            h[v] = __builtin_fmaf(q.x, h[v], q.y);
        }
    if (p.saved && lane.own && (wave * R) % LM_GATED_SAVE == 0 && tw < at.t1) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.saved[(at.first + tw / LM_GATED_SAVE) * p.C + c + v] = h[v];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = b[r][v] = __builtin_fmaf(a[r][v], h[v], b[r][v]);
    if (wave == kWaves - 1 && at.ch == at.nch - 1 && p.s1 && lane.own) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.s1[at.seq * p.s1_n + (c + v) * p.s1_c] = h[v];
    }
    if (!p.y || !lane.own) return;
    const RowsAt<T, V, DENSE> py(p.y, p.ys, at.sp, c, block);
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (tw + r < at.t1) put<T, V>(py.row(tw + r), b[r]);
}

// --------------------------------------------------------------- backward --

// With q_t = a_t (gy_t + q_{t+1}) the rows of a chunk are a map of q too: (P, s)
// of every chunk that another is in front of.
template <typename T, int V, bool DENSE> __global__ __launch_bounds__(64 * kWaves) void gated_bwd_sums(const GatedP p)
{
    __shared__ __attribute__((aligned(16))) float2 sums[2][kWaves][64 * V];
    constexpr int R = kFwd;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lv = (threadIdx.x & 63) * V;
    const GatedAt at = gated_at(p, blockIdx.x);
    const uint32_t block = blockIdx.x - (uint32_t)at.part * p.blocks;
    if (at.ch <= 0) return;
    const LaneAt<V> lane(p, block);
    const int64_t c = lane.c, rows = at.t1 - at.t0;
    const RowsAt<T, V, DENSE> pr(p.r, p.rs, at.sp, c, block), pg(p.gy, p.gys, at.sp, c, block);
    float k2[V], q[V], all[V];
    Raw<T, V> nr[R], ng[R];
    int64_t t = at.t0 + (rows - 1) / LM_GATED_TILE * LM_GATED_TILE;   // chunks behind the first have rows
    get_rows(pr, t + wave * R, at.t1 - 1, nr), get_rows(pg, t + wave * R, at.t1 - 1, ng);
    get_rate<V>(p, c, k2);
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = 0.f, all[v] = 1.f;
    for (int buf = 0; t >= at.t0; t -= LM_GATED_TILE, buf ^= 1) {
        const int64_t tw = t + wave * R;
        float P[V], s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) P[v] = 1.f, s[v] = 0.f;
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
            const bool in = tw + r < at.t1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float f = hw_exp2(k2[v] * sigmoid(nr[r].f(v)));
                const float a = in ? f : 1.f;
                P[v] *= a, s[v] = a * (s[v] + (in ? ng[r].f(v) : 0.f));
            }
        }
        if (t > at.t0) {
            const int64_t n = tw - LM_GATED_TILE;
            get_rows(pr, n, at.t1 - 1, nr), get_rows(pg, n, at.t1 - 1, ng);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sums[buf][wave][lv + v] = make_float2(P[v], s[v]);
        lds_sync();
        if (wave == 0) {
            for (int w = kWaves - 1; w >= 0; --w)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float2 m = sums[buf][w][lv + v];
                    q[v] = __builtin_fmaf(m.x, q[v], m.y), all[v] *= m.x;
                }
        }
    }
    if (wave == 0 && lane.own) {
#pragma unroll
        for (int v = 0; v < V; ++v) reinterpret_cast<float2 *>(p.sums)[at.part * p.C + c + v] = make_float2(all[v], q[v]);
    }
}

// Bound by memory (seven tensors) and by one workgroup a unit: 116 registers of a
// lane, which a limit of 64 spilled.  Tiles from the last one up.  Each starts from the saved state in front of it;
// the waves' maps of h go down through LDS, those of q up.
template <typename T, int V, bool DENSE> __global__ __launch_bounds__(64 * kWaves) void gated_bwd(const GatedP p)
{
    __shared__ __attribute__((aligned(16))) float2 hs[2][kWaves][64 * V];
    __shared__ float qs[2][kWaves][64 * V];
    __shared__ float carry[2][64 * V];
    constexpr int R = kBwd;
    const int waves = blockDim.x >> 6;   // 16 where there is more than a tile
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lv = (threadIdx.x & 63) * V;
    const GatedAt at = gated_at(p, blockIdx.x);
    const uint32_t block = blockIdx.x - (uint32_t)at.part * p.blocks;
    const LaneAt<V> lane(p, block);
    const int64_t c = lane.c;
    if (at.ch < 0) {
        if (wave == 0 && lane.own) {
#pragma unroll
            for (int v = 0; v < V; ++v) p.part[at.part * p.C + c + v] = 0.f;
        }
        return;
    }
    const RowsAt<T, V, DENSE> px(p.x, p.xs, at.sp, c, block), pr(p.r, p.rs, at.sp, c, block), pi(p.i, p.is, at.sp, c, block),
        pg(p.gy, p.gys, at.sp, c, block), dx(p.dx, p.dxs, at.sp, c, block), dr(p.dr, p.drs, at.sp, c, block),
        di(p.di, p.dis, at.sp, c, block);
    Raw<T, V> nx[R], nr[R], ni[R], ng[R];
    float ns[V], k2[V], k[V], dk[V], q[V];
    const auto fetch = [&](int64_t t) {
        const int64_t tw = t + wave * R, last = at.t1 - 1;
        get_rows(px, tw, last, nx), get_rows(pr, tw, last, nr), get_rows(pi, tw, last, ni), get_rows(pg, tw, last, ng);
#pragma unroll
        for (int v = 0; v < V; ++v) ns[v] = p.saved[(at.first + t / LM_GATED_SAVE) * p.C + c + v];
    };
    int64_t t = at.t0 + (at.t1 - at.t0 - 1) / LM_GATED_SAVE * LM_GATED_SAVE;
    if (at.t0 < at.t1) fetch(t);
    else t = at.t0 - 1;
    get_rate<V>(p, c, k2);
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = -kLn2 * k2[v], dk[v] = 0.f, q[v] = 0.f;
    if (wave == 0) {   // this wave carries q from tile to tile
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (p.gs) q[v] = p.gs[at.seq * p.gs_n + (c + v) * p.gs_c];
        fold<V>(p, at.part - at.ch + at.nch - 1, -1, at.nch - 1 - at.ch, c, q);
#pragma unroll
        for (int v = 0; v < V; ++v) carry[0][lv + v] = q[v];
    }
    for (int buf = 0; t >= at.t0; t -= LM_GATED_SAVE, buf ^= 1) {
        const int64_t tw = t + wave * R;
        float a[R][V], m[R][V], rho[R][V], iota[R][V], x[R][V], g[R][V], h[V], P[V], s[V], z[V];
#pragma unroll
        for (int v = 0; v < V; ++v) P[v] = 1.f, s[v] = 0.f, z[v] = 0.f, h[v] = ns[v];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = tw + r < at.t1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                rho[r][v] = sigmoid(nr[r].f(v)), iota[r][v] = sigmoid(ni[r].f(v));
                const float t2 = k2[v] * rho[r][v], f = hw_exp2(t2), cm = complement(t2, f);
                a[r][v] = in ? f : 1.f, m[r][v] = in ? cm : 0.f;
                x[r][v] = in ? nx[r].f(v) : 0.f, g[r][v] = in ? ng[r].f(v) : 0.f;
                if (!in) rho[r][v] = iota[r][v] = 0.f;
                P[v] *= a[r][v], s[v] = __builtin_fmaf(a[r][v], s[v], m[r][v] * iota[r][v] * x[r][v]);
            }
        }
#pragma unroll
        for (int r = R - 1; r >= 0; --r)
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = a[r][v] * (g[r][v] + z[v]);
        if (t > at.t0) fetch(t - LM_GATED_SAVE);
#pragma unroll
        for (int v = 0; v < V; ++v) hs[buf][wave][lv + v] = make_float2(P[v], s[v]), qs[buf][wave][lv + v] = z[v];
        lds_sync();
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 f = hs[buf][w][lv + v];
                h[v] = __builtin_fmaf(f.x, h[v], f.y);
            }
#pragma unroll
        for (int v = 0; v < V; ++v) q[v] = carry[buf][lv + v];
        for (int w = waves - 1; w > wave; --w)
#pragma unroll
            for (int v = 0; v < V; ++v) q[v] = __builtin_fmaf(hs[buf][w][lv + v].x, q[v], qs[buf][w][lv + v]);
        float before[R][V];   // h in front of each row
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                before[r][v] = h[v];
                h[v] = __builtin_fmaf(a[r][v], h[v], m[r][v] * iota[r][v] * x[r][v]);
            }
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
            float ox[V], orr[V], oi[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float gh = g[r][v] + q[v], ag = a[r][v] * gh;
                q[v] = ag;
                const float gi = gh * iota[r][v];
                ox[v] = gi * m[r][v];
                oi[v] = ox[v] * x[r][v] * (1.f - iota[r][v]);
                const float am = m[r][v] > 0.f ? a[r][v] * a[r][v] * hw_rcp(m[r][v]) : m[r][v];
                const float dl = __builtin_fmaf(ag, before[r][v], -(gi * x[r][v] * am)) * rho[r][v];
                dk[v] += dl;
                orr[v] = -k[v] * dl * (1.f - rho[r][v]);
            }
            if (tw + r < at.t1 && lane.own) {
                put<T, V>(dx.row(tw + r), ox), put<T, V>(dr.row(tw + r), orr), put<T, V>(di.row(tw + r), oi);
            }
        }
        if (wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) carry[buf ^ 1][lv + v] = q[v];
        }
    }
    if (wave == 0 && p.ds && at.ch == 0 && lane.own) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.ds[at.seq * p.ds_n + (c + v) * p.ds_c] = q[v];
    }
    lds_sync();   // the last tile's maps have been read
#pragma unroll
    for (int v = 0; v < V; ++v) qs[0][wave][lv + v] = dk[v];
    lds_sync();
    if (wave == 0 && lane.own) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float sum = 0.f;
            for (int w = 0; w < waves; ++w) sum += qs[0][w][lv + v];
            p.part[at.part * p.C + c + v] = sum;
        }
    }
}

// ddecay from the chunks' terms, in a fixed order.
__global__ __launch_bounds__(1024) void gated_ddecay(const GatedP p)
{
    __shared__ float sums[16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.f;
    if (c < p.C)
#pragma unroll 8
        for (int64_t i = wave; i < p.parts; i += 16) v += p.part[i * p.C + c];
    sums[wave][lane] = v;
    __syncthreads();
    if (wave || c >= p.C) return;
    for (int w = 1; w < 16; ++w) v += sums[w][lane];
    p.dd[c * p.dd_c] = -p.value * sigmoid(p.decay[c * p.decay_c]) * v;
}

// ------------------------------------------------------------------- step --

// One token for each batch row, its state moved in place.  Latency: 64 rows of
// 4096 channels 4.0 us, of which an empty launch is 1.7.
template <typename T, int V> __global__ __launch_bounds__(256) void gated_step(const GatedP p, uint32_t per)
{
    int64_t cv;
    const int64_t n = divide((int64_t)blockIdx.x * 256 + threadIdx.x, per, cv), c = cv * V;
    if (n >= p.seqs) return;
    T *y = static_cast<T *>(p.y) + n * p.ys.n + c * p.ys.c;
    const auto store = [&](const float (&v)[V]) {
        if (V == 1 || p.ys.c == 1) put<T, V>(y, v);
        else {
#pragma unroll
            for (int j = 0; j < V; ++j) y[j * p.ys.c] = from_f32<T>(v[j]);
        }
    };
    int64_t row = n;
    if (p.rows) {
        row = p.rows[n];
        if (row < 0 || row >= p.state_rows) {
            const float zero[V] = {};
            store(zero);
            return;
        }
    }
    const auto load = [&](const void *t, const S3 &st, float (&o)[V]) {
        const T *v = static_cast<const T *>(t) + n * st.n + c * st.c;
        if (V == 1 || st.c == 1) load_f32<T, V>(v, o);
        else {
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = to_f32(v[j * st.c]);
        }
    };
    float x[V], r[V], i[V], h[V], k2[V];
    load(p.x, p.xs, x), load(p.r, p.rs, r), load(p.i, p.is, i);
    float *st = p.s1 + row * p.s1_n + c * p.s1_c;
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = st[j * p.s1_c];
    get_rate<V>(p, c, k2);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float t2 = k2[j] * sigmoid(r[j]), a = hw_exp2(t2);
        h[j] = __builtin_fmaf(a, h[j], complement(t2, a) * sigmoid(i[j]) * x[j]);
        st[j * p.s1_c] = h[j];
    }
    store(h);
}

S3 s3(const conv_tensor &t) { return {t.strides[0], t.strides[1], t.rank > 2 ? t.strides[2] : 0}; }

GatedP base(const lm_plan_t &p, lm_ptrs q, void *ws)
{
    GatedP a = {};
    const auto f = [&](int s) { return static_cast<float *>(q[s]); };
    a.x = q[LM_X], a.r = q[LM_A], a.i = q[LM_B], a.gy = q[LM_GY];
    a.y = q[LM_Y], a.dx = q[LM_DX], a.dr = q[LM_DA], a.di = q[LM_DB];
    a.decay = f(LM_D), a.s0 = f(LM_STATE_IN), a.gs = f(LM_GSTATE), a.s1 = f(LM_STATE_OUT), a.ds = f(LM_DSTATE);
    a.saved = f(LM_SAVED), a.dd = f(LM_DD);
    a.off = static_cast<const int32_t *>(q[LM_OFFSETS]), a.rows = static_cast<const int32_t *>(q[LM_ROWS]);
    a.xs = s3(p.t[LM_X]), a.rs = s3(p.t[LM_A]), a.is = s3(p.t[LM_B]), a.ys = s3(p.t[LM_Y]), a.gys = s3(p.t[LM_GY]);
    a.dxs = s3(p.t[LM_DX]), a.drs = s3(p.t[LM_DA]), a.dis = s3(p.t[LM_DB]);
    const auto pair = [&](int s, int64_t &n, int64_t &c) { n = p.t[s].strides[0], c = p.t[s].strides[1]; };
    pair(LM_STATE_IN, a.s0_n, a.s0_c), pair(LM_STATE_OUT, a.s1_n, a.s1_c), pair(LM_GSTATE, a.gs_n, a.gs_c), pair(LM_DSTATE, a.ds_n, a.ds_c);
    a.decay_c = p.t[LM_D].strides[0], a.dd_c = p.t[LM_DD].strides[0];
    a.seqs = p.seqs, a.C = p.C, a.L = p.L, a.chunk = p.chunk, a.chunks = p.chunks, a.parts = lm_parts(p), a.slots = lm_slots(p);
    a.blocks = (uint32_t)lm_cdiv(p.C, 64 * gated_width(p));
    a.state_rows = p.t[LM_STATE_OUT].sizes[0];
    a.value = p.args.value;
    a.ahead = static_cast<uint64_t *>(ws), a.sums = static_cast<float *>(ws);
    a.part = a.sums + (p.chunks > 1 ? 2 * a.parts * p.C : 0);
    return a;
}

// Threads of a workgroup whose waves take `rows` each: no waves without rows where
// no sequence has a tile's (24 x 4 x 3800 f32, output and gradients: 29 us for 65).
unsigned group_size(const GatedP &a, int rows)
{
    return 64 * (unsigned)(a.chunks > 1 ? kWaves : std::max<int64_t>(1, std::min<int64_t>(kWaves, lm_cdiv(a.L, rows))));
}

// f(type, channels of a thread, whether channels are contiguous).
template <typename F> void with_type(const lm_plan_t &p, F f)
{
    const auto widths = [&](auto t) {
        typedef decltype(t) T;
        if constexpr (sizeof(T) == 2) {
            if (gated_width(p) == 2) return f(t, std::integral_constant<int, 2>(), std::true_type());
            f(t, std::integral_constant<int, 1>(), std::false_type());
        } else {
            for (int s : {LM_X, LM_A, LM_B, LM_Y, LM_GY, LM_DX, LM_DA, LM_DB})
                if (p.t[s].rank && p.t[s].strides[1] != 1) return f(t, std::integral_constant<int, 1>(), std::false_type());
            f(t, std::integral_constant<int, 1>(), std::true_type());
        }
    };
    if (p.dtype == CONV_F32) widths(float());
    else if (p.dtype == CONV_F16) widths(f16_t());
    else widths(bf16_t());
}

}  // namespace

int launch_lm_gated(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    const GatedP a = base(p, q, ws);
    const unsigned groups = (unsigned)(a.parts * a.blocks);
    if (!groups) return CONV_OK;
    with_type(p, [&](auto t, auto v, auto dense) {
        typedef decltype(t) T;
        constexpr int V = decltype(v)::value;
        constexpr bool D = decltype(dense)::value;
        if (a.chunks > 1) {
            const int64_t words = 2 * a.parts * a.C;
            gated_clear<<<(unsigned)lm_cdiv(words + (int64_t)a.blocks * kTicket, 256), 256, 0, s>>>(a, words);
            gated_tile<T, V, D><<<groups, 64 * kWaves, 0, s>>>(a);
        } else gated_fwd<T, V, D><<<groups, group_size(a, kFwd), 0, s>>>(a);
    });
    return lm_launch_status();
}

int launch_lm_gated_bwd(const lm_plan_t &p, lm_ptrs q, void *ws, hipStream_t s)
{
    const GatedP a = base(p, q, ws);
    const unsigned groups = (unsigned)(a.parts * a.blocks);
    if (groups)
        with_type(p, [&](auto t, auto v, auto dense) {
            typedef decltype(t) T;
            constexpr int V = decltype(v)::value;
            constexpr bool D = decltype(dense)::value;
            if (a.chunks > 1) gated_bwd_sums<T, V, D><<<groups, 64 * kWaves, 0, s>>>(a);
            gated_bwd<T, V, D><<<groups, group_size(a, kBwd), 0, s>>>(a);
        });
    gated_ddecay<<<(unsigned)lm_cdiv(p.C, 64), 1024, 0, s>>>(a);
    return lm_launch_status();
}

int launch_lm_gated_step(const lm_plan_t &p, lm_ptrs q, hipStream_t s)
{
    const GatedP a = base(p, q, nullptr);
    const bool two = gated_step_width(p) == 2;
    const uint32_t per = (uint32_t)(two ? p.C / 2 : p.C);
    const unsigned groups = (unsigned)lm_cdiv(p.seqs * per, 256);
    if (!groups) return CONV_OK;
    const auto go = [&](auto t) {
        typedef decltype(t) T;
        if (two) gated_step<T, 2><<<groups, 256, 0, s>>>(a, per);
        else gated_step<T, 1><<<groups, 256, 0, s>>>(a, per);
    };
    if (p.dtype == CONV_F32) go(float());
    else if (p.dtype == CONV_F16) go(f16_t());
    else go(bf16_t());
    return lm_launch_status();
}

}  // namespace miconv
