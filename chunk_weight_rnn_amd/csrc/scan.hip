// Gated linear recurrence of every channel over packed sequences, and its
// gradients:
//
//   h_t = a_t h_{t-1} + x_t,
//   g_t = dout_t + a_{t+1} g_{t+1},  dx_t = g_t,  da_t = g_t h_{t-1}.
//
// HBM bound: two operations per value read.  A stretch of tokens acts on the
// state that enters it as h -> P h + H, with P the product of its gates and H
// its result from zero, so that stretches can be read side by side: a workgroup
// takes a slab of channels (V per lane) of one sequence and walks over tiles of
// E2TTT_SCAN_TILE tokens, every wave with R of them in registers and the next
// tile's on their way.  The waves exchange their (P, H) through the LDS, each
// folds those before it onto the tile's state, and runs its tokens a second
// time from registers, now from the right state: the outputs are those of the
// recurrence itself, not of products and sums over the stretch.
//
// The gradient walks the same way from the last tile to the first.  It needs
// the states again, which out holds rounded: they are computed once more from
// the saved states at the tiles' starts, which costs no more reading than out
// would (x in its place).
//
// Where sequences and slabs are too few for the chip (PARTS), each sequence is
// cut into parts of `part` tokens; a first launch reads the gates and inputs of
// all but the last for their (P, H), and the second folds those before its part.
#include "attn_common.h"

namespace e2ttt {
namespace {

using attn::clamped;

constexpr int R = 16;                     // tokens of a wave per tile
constexpr int NW = E2TTT_SCAN_TILE / R;   // waves of a workgroup
constexpr int TILE = E2TTT_SCAN_TILE;

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

// One sequence, or one part of it: tokens [lo, hi) of the n from tok0 on.
struct Stretch {
    int seq, tok0, n, lo, hi;
};

__device__ __forceinline__ Stretch whole_sequence(const ScanArgs& a, int s) {
    Stretch r{s, clamped(a.cu[s], (int)a.N), 0, 0, 0};
    const int n = clamped(a.cu[s + 1], (int)a.N) - r.tok0;
    r.n = r.hi = n > 0 ? n : 0;
    return r;
}

__device__ __forceinline__ bool find_part(const ScanArgs& a, int t, Stretch& r) {
    attn::Item it;
    const int part = a.part;
    if (!attn::find_item(a.cu, a.S, (int)a.N, t, attn::kInOrder,
                         [&](int n) { return n > part ? (n - 1) / part + 1 : 1; }, it))
        return false;
    r = {it.seq, it.tok0, it.n, it.tile * part, it.n};
    if (r.n - r.lo > part) r.hi = r.lo + part;
    return true;
}

// Rows of the workspace and of starts: parts, or tiles, of the sequences before,
// and never past the end whatever the offsets hold.
__device__ __forceinline__ int64_t row_of(const Stretch& r, int len) { return r.tok0 / len + r.seq; }

// `rows` tokens' values of this lane's channels from p on; the others are `fill`.
template <typename T, int V>
__device__ __forceinline__ void load(Pack<T, V> (&x)[R], const T* p, int64_t stride, int rows, bool in, float fill) {
    Pack<T, V> f;
#pragma unroll
    for (int e = 0; e < V; ++e) f.v[e] = (T)fill;
    if (rows >= R) {
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = in ? *(const Pack<T, V>*)(p + r * stride) : f;
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = in && r < rows ? *(const Pack<T, V>*)(p + r * stride) : f;
    }
}

template <int V>
__device__ __forceinline__ void load_state(float (&h)[V], const float* p, bool in) {
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = in && p ? p[e] : 0.f;
}
template <int V>
__device__ __forceinline__ void store_state(float* p, const float (&h)[V], bool in) {
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (in) p[e] = h[e];
}

// Outputs of the tokens of no sequence: block b of a.clear.
template <typename T>
__device__ __forceinline__ void clear_rows(const ScanArgs& a, T* p, int b) {
    const int64_t lo = clamped(a.cu[0], (int)a.N), end = clamped(a.cu[a.S], (int)a.N), hi = end > lo ? end : lo;
    const int64_t first = lo * a.C, count = (lo + a.N - hi) * a.C, skip = (hi - lo) * a.C;
    for (int64_t i = (int64_t)b * blockDim.x + threadIdx.x; i < count; i += (int64_t)a.clear * blockDim.x)
        p[i < first ? i : i + skip] = (T)0.f;
}

// The state before this part, from the (P, H) of the parts on the way to it:
// parts [0, count) in steps of `dir` from row `first` on.  Every wave folds its
// share, then all of them together.
template <int V>
__device__ __forceinline__ void fold_parts(const ScanArgs& a, float (&h)[V], float (*sh)[2][64 * V], int64_t first, int dir,
                                           int count, int c, bool in) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (count + NW - 1) / NW, i0 = wave * per, i1 = i0 + per < count ? i0 + per : count;
    float P[V], H[V];
#pragma unroll
    for (int e = 0; e < V; ++e) P[e] = 1.f, H[e] = 0.f;
    for (int i = i0; i < i1; ++i) {
        const float* s = a.sums + (first + (int64_t)dir * i) * 2 * a.C + c;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float p = in ? s[e] : 1.f, q = in ? s[a.C + e] : 0.f;
            H[e] = __builtin_fmaf(p, H[e], q);
            P[e] *= p;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sh[wave][0][lane * V + e] = P[e], sh[wave][1][lane * V + e] = H[e];
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = __builtin_fmaf(sh[w][0][lane * V + e], h[e], sh[w][1][lane * V + e]);
    __syncthreads();
}

template <typename TX, typename TA, int V, bool PARTS>
__global__ __launch_bounds__(64 * NW) void scan_fwd_kernel(ScanArgs a) {
    __shared__ float sh[2][NW][2][64 * V];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x >= a.groups) {
        clear_rows(a, (TX*)a.out, blockIdx.x - a.groups);
        return;
    }
    const int c = ((int)(blockIdx.x % a.slabs) * 64 + lane) * V;
    const bool in = c < a.C;
    Stretch s;
    if (PARTS) {
        if (!find_part(a, blockIdx.x / a.slabs, s)) return;
    } else {
        s = whole_sequence(a, blockIdx.x / a.slabs);
    }
    float h[V];
    load_state<V>(h, (PARTS ? a.first : a.h0) ? (PARTS ? a.first : a.h0) + (int64_t)s.seq * a.C + c : nullptr, in);
    if (PARTS && s.lo > 0) fold_parts<V>(a, h, sh[0], row_of(s, a.part), 1, s.lo / a.part, c, in);
    const TX* xp = (const TX*)a.x + (s.tok0 + (int64_t)wave * R) * a.x_tok + c;
    const TA* ap = (const TA*)a.a + (s.tok0 + (int64_t)wave * R) * a.a_tok + c;
    TX* op = (TX*)a.out + (s.tok0 + (int64_t)wave * R) * a.C + c;
    float* st = a.starts ? a.starts + row_of(s, TILE) * a.C + c : nullptr;
    Pack<TX, V> x[R];
    Pack<TA, V> g[R];
    load(x, xp + s.lo * a.x_tok, a.x_tok, s.hi - s.lo - wave * R, in, 0.f);
    load(g, ap + s.lo * a.a_tok, a.a_tok, s.hi - s.lo - wave * R, in, 1.f);
    int buf = 0;
    for (int t = s.lo; t < s.hi; t += TILE, buf ^= 1) {
        Pack<TX, V> xn[R];
        Pack<TA, V> gn[R];
        const int64_t tn = t + TILE;
        load(xn, xp + tn * a.x_tok, a.x_tok, s.hi - t - TILE - wave * R, in, 0.f);
        load(gn, ap + tn * a.a_tok, a.a_tok, s.hi - t - TILE - wave * R, in, 1.f);
        float P[V], H[V];
#pragma unroll
        for (int e = 0; e < V; ++e) P[e] = 1.f, H[e] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                H[e] = __builtin_fmaf((float)g[r].v[e], H[e], (float)x[r].v[e]);
                P[e] *= (float)g[r].v[e];
            }
#pragma unroll
        for (int e = 0; e < V; ++e) sh[buf][wave][0][lane * V + e] = P[e], sh[buf][wave][1][lane * V + e] = H[e];
        __syncthreads();  // one barrier a tile: the other buffer was read before it
        if (st && wave == 0) store_state<V>(st + (int64_t)(t / TILE) * a.C, h, in);
        float mine[V];
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (w == wave) mine[e] = h[e];
                h[e] = __builtin_fmaf(sh[buf][w][0][lane * V + e], h[e], sh[buf][w][1][lane * V + e]);
            }
        const int rows = s.hi - t - wave * R;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Pack<TX, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                mine[e] = __builtin_fmaf((float)g[r].v[e], mine[e], (float)x[r].v[e]);
                o.v[e] = (TX)mine[e];
            }
            if (in && r < rows) *(Pack<TX, V>*)(op + (int64_t)(t + r) * a.C) = o;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = xn[r], g[r] = gn[r];
    }
    if (!a.state || s.hi != s.n) return;
    __syncthreads();  // state may be h0, which every wave has used by now
    if (wave == 0) store_state<V>(a.state + (int64_t)s.seq * a.C + c, h, in);
}

// Sequences of a few tokens: a wave each and slab, no exchange.
template <typename TX, typename TA, int V>
__global__ __launch_bounds__(256) void scan_short_kernel(ScanArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int past = (int)blockIdx.x - (a.groups + 3) / 4;
    if (past >= 0) {
        clear_rows(a, (TX*)a.out, past);
        return;
    }
    const int unit = (int)blockIdx.x * 4 + wave;
    if (unit >= a.groups) return;
    const int c = (unit % a.slabs * 64 + lane) * V;
    const bool in = c < a.C;
    const Stretch s = whole_sequence(a, unit / a.slabs);
    float h[V];
    load_state<V>(h, a.h0 ? a.h0 + (int64_t)s.seq * a.C + c : nullptr, in);
    const TX* xp = (const TX*)a.x + s.tok0 * a.x_tok + c;
    const TA* ap = (const TA*)a.a + s.tok0 * a.a_tok + c;
    TX* op = (TX*)a.out + (int64_t)s.tok0 * a.C + c;
    float* st = a.starts ? a.starts + row_of(s, TILE) * a.C + c : nullptr;
    for (int t = 0; t < s.n; t += R) {
        Pack<TX, V> x[R];
        Pack<TA, V> g[R];
        load(x, xp + t * a.x_tok, a.x_tok, s.n - t, in, 0.f);
        load(g, ap + t * a.a_tok, a.a_tok, s.n - t, in, 1.f);
        if (st && t % TILE == 0) store_state<V>(st + (int64_t)(t / TILE) * a.C, h, in);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Pack<TX, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[e] = __builtin_fmaf((float)g[r].v[e], h[e], (float)x[r].v[e]);
                o.v[e] = (TX)h[e];
            }
            if (in && r < s.n - t) *(Pack<TX, V>*)(op + (int64_t)(t + r) * a.C) = o;
        }
    }
    if (a.state) store_state<V>(a.state + (int64_t)s.seq * a.C + c, h, in);
}

// (P, H) of the parts that others follow (forward), or (P, K) of those that others
// precede (BWD: c -> P c + K, the gradient a part hands to the one before it).
// Every wave takes a stretch of its part, then all of them together.  The state
// that a sequence begins with is copied, so that the second launch may write the
// new one in its place.
template <typename TX, typename TA, int V, bool BWD>
__global__ __launch_bounds__(64 * NW) void scan_parts_kernel(ScanArgs a) {
    __shared__ float sh[NW][2][64 * V];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = ((int)(blockIdx.x % a.slabs) * 64 + lane) * V;
    const bool in = c < a.C;
    Stretch s;
    if (!find_part(a, blockIdx.x / a.slabs, s)) return;
    if (!BWD && s.lo == 0 && a.first && wave == 0) {
        float h[V];
        load_state<V>(h, a.h0 + (int64_t)s.seq * a.C + c, in);
        store_state<V>(a.first + (int64_t)s.seq * a.C + c, h, in);
    }
    if (BWD ? s.lo == 0 : s.hi == s.n) return;
    const int per = ((s.hi - s.lo + NW - 1) / NW + R - 1) / R * R;
    const int t0 = s.lo + wave * per, t1 = t0 + per < s.hi ? t0 + per : s.hi;
    const TX* xp = (const TX*)a.x + s.tok0 * a.x_tok + c;
    const TA* ap = (const TA*)a.a + s.tok0 * a.a_tok + c;
    float P[V], H[V];
#pragma unroll
    for (int e = 0; e < V; ++e) P[e] = 1.f, H[e] = 0.f;
    const int steps = t1 > t0 ? (t1 - t0 + R - 1) / R : 0;
    auto at = [&](int i) { return t0 + (BWD ? steps - 1 - i : i) * R; };
    Pack<TX, V> x[R];
    Pack<TA, V> g[R];
    if (steps > 0) {
        load(x, xp + at(0) * a.x_tok, a.x_tok, t1 - at(0), in, 0.f);
        load(g, ap + at(0) * a.a_tok, a.a_tok, t1 - at(0), in, 1.f);
    }
    for (int i = 0; i < steps; ++i) {
        Pack<TX, V> xn[R];
        Pack<TA, V> gn[R];
        const bool more = i + 1 < steps;
        load(xn, xp + at(more ? i + 1 : i) * a.x_tok, a.x_tok, more ? t1 - at(i + 1) : 0, in, 0.f);
        load(gn, ap + at(more ? i + 1 : i) * a.a_tok, a.a_tok, more ? t1 - at(i + 1) : 0, in, 1.f);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int r = BWD ? R - 1 - k : k;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float av = (float)g[r].v[e], xv = (float)x[r].v[e];
                H[e] = BWD ? av * (xv + H[e]) : __builtin_fmaf(av, H[e], xv);
                P[e] *= av;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = xn[r], g[r] = gn[r];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sh[wave][0][lane * V + e] = P[e], sh[wave][1][lane * V + e] = H[e];
    __syncthreads();
    if (wave != 0) return;
    float Q[V], K[V];
#pragma unroll
    for (int e = 0; e < V; ++e) Q[e] = 1.f, K[e] = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        const int w = BWD ? NW - 1 - k : k;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            K[e] = __builtin_fmaf(sh[w][0][lane * V + e], K[e], sh[w][1][lane * V + e]);
            Q[e] *= sh[w][0][lane * V + e];
        }
    }
    float* o = a.sums + (row_of(s, a.part) + s.lo / a.part) * 2 * a.C + c;
    store_state<V>(o, Q, in);
    store_state<V>(o + a.C, K, in);
}

template <typename TX, typename TA, int V, bool PARTS>
__global__ __launch_bounds__(64 * NW) void scan_bwd_kernel(ScanArgs a) {
    __shared__ float sh[2][NW][3][64 * V];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x >= a.groups) {
        clear_rows(a, (TX*)a.out, blockIdx.x - a.groups);
        clear_rows(a, (TA*)a.da, blockIdx.x - a.groups);
        return;
    }
    const int c = ((int)(blockIdx.x % a.slabs) * 64 + lane) * V;
    const bool in = c < a.C;
    Stretch s;
    if (PARTS) {
        if (!find_part(a, blockIdx.x / a.slabs, s)) return;
    } else {
        s = whole_sequence(a, blockIdx.x / a.slabs);
    }
    float gc[V];  // what reaches the state after the tile: a_{t+1} g_{t+1}
    load_state<V>(gc, a.h0 ? a.h0 + (int64_t)s.seq * a.C + c : nullptr, in);
    if (PARTS && s.hi < s.n) {
        const int last = (s.n - 1) / a.part, mine = s.lo / a.part;
        fold_parts<V>(a, gc, (float (*)[2][64 * V])&sh[0][0][0][0], row_of(s, a.part) + last, -1, last - mine, c, in);
    }
    const TX* xp = (const TX*)a.x + (s.tok0 + (int64_t)wave * R) * a.x_tok + c;
    const TA* ap = (const TA*)a.a + (s.tok0 + (int64_t)wave * R) * a.a_tok + c;
    const int64_t o0 = (s.tok0 + (int64_t)wave * R) * a.C + c;
    const TX* dp = (const TX*)a.dout + o0;
    const float* st = a.starts + row_of(s, TILE) * a.C + c;
    Pack<TX, V> x[R], d[R];
    Pack<TA, V> g[R];
    float h0[V];
    auto fetch = [&](int t, Pack<TX, V> (&x)[R], Pack<TX, V> (&d)[R], Pack<TA, V> (&g)[R], float (&h0)[V]) {
        const int rows = t >= s.lo ? s.hi - t - wave * R : 0;
        load(x, xp + t * a.x_tok, a.x_tok, rows, in, 0.f);
        load(g, ap + t * a.a_tok, a.a_tok, rows, in, 1.f);
        load(d, dp + (int64_t)t * a.C, a.C, rows, in, 0.f);
        load_state<V>(h0, st + (int64_t)(t / TILE) * a.C, in && t >= s.lo);
    };
    int t = s.hi > s.lo ? s.lo + (s.hi - s.lo - 1) / TILE * TILE : s.lo - TILE;
    fetch(t, x, d, g, h0);
    int buf = 0;
    for (; t >= s.lo; t -= TILE, buf ^= 1) {
        Pack<TX, V> xn[R], dn[R];
        Pack<TA, V> gn[R];
        float hn[V];
        fetch(t - TILE, xn, dn, gn, hn);
        float P[V], H[V], K[V];
#pragma unroll
        for (int e = 0; e < V; ++e) P[e] = 1.f, H[e] = 0.f, K[e] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                H[e] = __builtin_fmaf((float)g[r].v[e], H[e], (float)x[r].v[e]);
                P[e] *= (float)g[r].v[e];
                K[e] = (float)g[R - 1 - r].v[e] * ((float)d[R - 1 - r].v[e] + K[e]);
            }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            sh[buf][wave][0][lane * V + e] = P[e];
            sh[buf][wave][1][lane * V + e] = H[e];
            sh[buf][wave][2][lane * V + e] = K[e];
        }
        __syncthreads();
        float mine[V];
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (w == wave) mine[e] = h0[e];
                h0[e] = __builtin_fmaf(sh[buf][w][0][lane * V + e], h0[e], sh[buf][w][1][lane * V + e]);
            }
        float cin[V];
#pragma unroll
        for (int w = NW - 1; w >= 0; --w)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (w == wave) cin[e] = gc[e];
                gc[e] = __builtin_fmaf(sh[buf][w][0][lane * V + e], gc[e], sh[buf][w][2][lane * V + e]);
            }
        float before[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                before[r][e] = mine[e];
                mine[e] = __builtin_fmaf((float)g[r].v[e], mine[e], (float)x[r].v[e]);
            }
        const int rows = s.hi - t - wave * R;
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
            Pack<TX, V> ox;
            Pack<TA, V> oa;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float gt = (float)d[r].v[e] + cin[e];
                ox.v[e] = (TX)gt;
                oa.v[e] = (TA)(gt * before[r][e]);
                cin[e] = (float)g[r].v[e] * gt;
            }
            if (in && r < rows) {
                *(Pack<TX, V>*)((TX*)a.out + o0 + (int64_t)(t + r) * a.C) = ox;
                *(Pack<TA, V>*)((TA*)a.da + o0 + (int64_t)(t + r) * a.C) = oa;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = xn[r], d[r] = dn[r], g[r] = gn[r];
#pragma unroll
        for (int e = 0; e < V; ++e) h0[e] = hn[e];
    }
    if (a.state && wave == 0 && s.lo == 0) store_state<V>(a.state + (int64_t)s.seq * a.C + c, gc, in);
}

template <typename TX, typename TA, int V>
hipError_t forward(const ScanArgs& a, hipStream_t s) {
    const dim3 bl(64 * NW), gr((unsigned)(a.groups + a.clear));
    if (a.shorts) {
        scan_short_kernel<TX, TA, V><<<dim3((unsigned)((a.groups + 3) / 4 + a.clear)), dim3(256), 0, s>>>(a);
    } else if (a.part) {
        scan_parts_kernel<TX, TA, V, false><<<dim3((unsigned)a.groups), bl, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        scan_fwd_kernel<TX, TA, V, true><<<gr, bl, 0, s>>>(a);
    } else {
        scan_fwd_kernel<TX, TA, V, false><<<gr, bl, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <typename TX, typename TA, int V>
hipError_t backward(const ScanArgs& a, hipStream_t s) {
    const dim3 bl(64 * NW), gr((unsigned)(a.groups + a.clear));
    if (a.part) {
        ScanArgs b = a;  // the gradient of the parts goes through gates and dout
        b.x = a.dout;
        b.x_tok = a.C;
        scan_parts_kernel<TX, TA, V, true><<<dim3((unsigned)a.groups), bl, 0, s>>>(b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        scan_bwd_kernel<TX, TA, V, true><<<gr, bl, 0, s>>>(a);
    } else {
        scan_bwd_kernel<TX, TA, V, false><<<gr, bl, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_forward(const ScanArgs& a, hipStream_t s) {
    if (a.x_f32) return forward<float, float, 1>(a, s);
    if (a.gate_f32) return a.pairs ? forward<__bf16, float, 2>(a, s) : forward<__bf16, float, 1>(a, s);
    return a.pairs ? forward<__bf16, __bf16, 2>(a, s) : forward<__bf16, __bf16, 1>(a, s);
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
    if (a.x_f32) return backward<float, float, 1>(a, s);
    if (a.gate_f32) return a.pairs ? backward<__bf16, float, 2>(a, s) : backward<__bf16, float, 1>(a, s);
    return a.pairs ? backward<__bf16, __bf16, 2>(a, s) : backward<__bf16, __bf16, 1>(a, s);
}

}  // namespace e2ttt
