// One token for each row of logits, by temperature, top-k, top-p and min-p,
// from a given random number of the row (the definition is in
// include/e2ttt_tokens.h).
//
// A workgroup per row.  Nothing is sorted: a filter keeps a stretch of the order by
// falling logit, so what it needs is the logit at which the running count or
// weight reaches a target.  Equal logits at that border are kept by index.
//
// The row is read once for the maximum of every tile (512 values of a wave) and of
// every thread and, as the settings ask for them, the tiles' weights and the counts
// of the logits in bins of 1/64 of a power of two, 31 powers deep, that move along
// with the largest logit so far.  Then
//  * without a filter the tile that holds the token follows from the tiles' weights,
//    and it alone is read again;
//  * the top_k largest lie at or above the top_k-th largest of the threads' maxima,
//    and little more does (k of 1024: -1024 ln(1 - k/1024) logits);
//  * for top_p the bins' counts say within which bins the border lies, up to the
//    2^(1/64) that the weights in a bin differ by.
// A second pass, over the tiles whose maximum is that large, gathers the logits from
// there on in a list, some hundred at most times; or, where they are many, those of
// the border's bins alone, and sums the weights above tile by tile.  The border is
// found in the list, the list's weights go to their tiles, and one tile is read again.
// A list of up to 128 is one wave's, which compares all with all.
// Rows whose border lies deeper than the bins reach, or where more than kList logits
// share its bins (equal ones, say), go the slow way: histograms of the whole row.
//
// Weights are whole multiples of 2^-44 of the largest, so that sums of up to 2^18
// of them are exact in 64 bits: any order of summation gives the same, and the
// border cases of the definition (a target met exactly) come out as written.  The
// tiles' weights of the first pass, taken before the maximum is known, are 64-bit
// floats added in one order: exact for equal logits, and else to 2^-45 of the largest
// per logit, as the rounding is that they leave out.
//
// What bounds it: of long rows the exponentials, some 20 instructions in 64 bits for
// every logit where its weight is needed, and the histogram (64 additions in the LDS
// take some 25 cycles, and 6 each where they are to one address: so threads that agree
// add once); of a few rows the chain of barriers.  One row of 32000 in bf16 with all
// filters 17 us, 64 of them with top_p 50, 256 rows of 128257 in fp32 101 (1.3 TB/s); of
// equal logits, the slow way, 86 and 280.
#include "tokens_internal.h"

namespace e2ttt {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2 * kThreads;
constexpr int kOne = 44;         // a weight of one is 2^44
constexpr int E = 8;             // values of a thread in a step of the row
constexpr int kTile = 64 * E;
constexpr int kStep = kTile * kWaves;
constexpr int kTiles = (E2TTT_SAMPLE_VOCAB + 8 + kStep - 1) / kStep * kWaves;
constexpr int kList = 8192;      // logits that are gathered, at most
constexpr int kTable = 1024;     // exponents are in 1024ths of a power of two
constexpr int kBinShift = 4;     // and bins in 16 of those
constexpr int kWhole = 31 * 64;  // bins from the newest on that lack nothing
constexpr int kMostBin = 256 * 64;  // past it bins count anew, so that no weight overflows
constexpr int kOneWave = 128;    // logits of a list that one wave deals with
constexpr int kByMaxima = 1000;  // top_k up to which the threads' maxima tell
static_assert(kTiles <= kThreads && kTable == kThreads, "a thread per tile, and per entry");

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// --------------------------------------------------------- over a wave's lanes
// x of the lane that `CTRL` names, `none` where there is none.
template <int CTRL, int ROWS, typename X>
__device__ __forceinline__ X from_lane(X x, X none) {
    if constexpr (sizeof(X) == 4) {
        const int r = __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, false);
        return __builtin_bit_cast(X, r);
    } else {
        const u64 n = __builtin_bit_cast(u64, none), v = __builtin_bit_cast(u64, x);
        const unsigned lo = __builtin_amdgcn_update_dpp((int)n, (int)v, CTRL, ROWS, 0xf, false);
        const unsigned hi = __builtin_amdgcn_update_dpp((int)(n >> 32), (int)(v >> 32), CTRL, ROWS, 0xf, false);
        return __builtin_bit_cast(X, (u64)hi << 32 | lo);
    }
}
// op over the lanes up to this one.
template <typename X, class F>
__device__ __forceinline__ X wave_scan(X x, X none, F&& op) {
    x = op(x, from_lane<0x111, 0xf>(x, none));  // row_shr:1, 2, 4, 8 within 16 lanes
    x = op(x, from_lane<0x112, 0xf>(x, none));
    x = op(x, from_lane<0x114, 0xf>(x, none));
    x = op(x, from_lane<0x118, 0xf>(x, none));
    x = op(x, from_lane<0x142, 0xa>(x, none));  // row_bcast:15, row_bcast:31
    x = op(x, from_lane<0x143, 0xc>(x, none));
    return x;
}
template <typename X>
__device__ __forceinline__ X wave_inclusive(X x) {
    return wave_scan(x, X{}, [](X a, X b) { return a + b; });
}
template <typename X>
__device__ __forceinline__ X lane_of(X x, int lane) {
    if constexpr (sizeof(X) == 4) {
        return __builtin_bit_cast(X, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
    } else {
        const u64 v = __builtin_bit_cast(u64, x);
        const unsigned lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
        return __builtin_bit_cast(X, (u64)hi << 32 | lo);
    }
}
template <typename X>
__device__ __forceinline__ X last_lane(X x) { return lane_of(x, 63); }
__device__ __forceinline__ float wave_max(float x) {
    return last_lane(wave_scan(x, neg_inf(), [](float a, float b) { return fmaxf(a, b); }));
}
__device__ __forceinline__ int lanes_below(u64 m) {
    return __builtin_amdgcn_mbcnt_hi((unsigned)(m >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)m, 0));
}

// Sum of x over the threads before this one, and over all of them, in one order.
template <typename X>
__device__ __forceinline__ X block_exclusive(X x, X* wave_sums, X* total) {
    const int wave = threadIdx.x >> 6;
    const X incl = wave_inclusive(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) wave_sums[wave] = incl;
    __syncthreads();
    // every 16 lanes add up the waves' sums
    X v = wave_sums[threadIdx.x & (kWaves - 1)];
    const X own = v;
    v += from_lane<0x111, 0xf>(v, X{});
    v += from_lane<0x112, 0xf>(v, X{});
    v += from_lane<0x114, 0xf>(v, X{});
    v += from_lane<0x118, 0xf>(v, X{});
    *total = lane_of(v, kWaves - 1);
    return lane_of(v - own, __builtin_amdgcn_readfirstlane(wave)) + (incl - x);
}

// -------------------------------------------------------------------- logits
// Order of the values as whole numbers (never of a NaN); zeros of either sign are equal.
__device__ __forceinline__ unsigned key_of(float x) {
    const float y = x + 0.f;
    const unsigned u = __builtin_bit_cast(unsigned, y);
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// A row, from the last address on at or before its first value that 16 divides:
// step j of thread t holds E values from place (j kThreads + t) E on.  Places before
// and past the row hold -infinity.  A NaN stays one, and no comparison takes it.
template <typename T>
struct Row {
    static constexpr int U = E * sizeof(T) / 16;
    struct Raw {
        u32x4 u[U];
    };
    const T* p;  // aligned
    int off, V;  // places before the row, values in it
    int steps;
    const float* tops;  // largest value of every tile
    __device__ __forceinline__ Row(const T* row, int V_, const float* tops_) : V(V_), tops(tops_) {
        off = (int)((uintptr_t)row % 16 / sizeof(T));
        p = row - off;
        steps = (V + off + kStep - 1) / kStep;
    }
    // Index of value e of this thread's step j.
    __device__ __forceinline__ int index(int j, int e) const { return (j * kThreads + (int)threadIdx.x) * E + e - off; }
    __device__ __forceinline__ Raw load(int j) const {
        const int first = index(j, 0);
        Raw r;
        if (first >= 0 && first + E <= V) {
#pragma unroll
            for (int k = 0; k < U; ++k) r.u[k] = *(const u32x4*)(p + off + first + k * (E / U));
        } else {
            T t[E];
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = first + e >= 0 && first + e < V ? p[off + first + e] : (T)neg_inf();
            __builtin_memcpy(&r, t, sizeof r);
        }
        return r;
    }
    static __device__ __forceinline__ void values(const Raw& r, float (&x)[E]) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const unsigned u = r.u[k][w];
                if constexpr (sizeof(T) == 2) {
                    x[2 * w] = __builtin_bit_cast(float, u << 16);
                    x[2 * w + 1] = __builtin_bit_cast(float, u & 0xffff0000u);
                } else {
                    x[4 * k + w] = __builtin_bit_cast(float, u);
                }
            }
    }
    // f(j, values) for the steps of this wave whose tile's largest value is wanted, the
    // next one's loads in flight.
    template <class P, class F>
    __device__ __forceinline__ void each(P&& wanted, F&& f) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        auto next = [&](int j) {
            while (j < steps && !wanted(tops[j * kWaves + wave])) ++j;
            return __builtin_amdgcn_readfirstlane(j);
        };
        int j = next(0);
        if (j >= steps) return;
        Raw raw = load(j);
#pragma unroll 1
        while (j < steps) {
            const int jn = next(j + 1);
            Raw more = raw;
            if (jn < steps) more = load(jn);
            float x[E];
            values(raw, x);
            f(j, x);
            j = jn;
            raw = more;
        }
    }
};

// A few logits and their indices in the LDS.
struct List {
    const unsigned* keys;
    const int* at;
    int n;
    template <class P, class F>
    __device__ __forceinline__ void each(P&&, F&& f) const {
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kThreads) {
            const int i = i0 + (int)threadIdx.x;
            const float x[1] = {i < n ? value_of(keys[i]) : __builtin_nanf("")};
            f(i, x);
        }
    }
};

// Weights of finite logits and -infinity: scaled(x) = 2^44 exp((x - top) / T) in 64
// bits, to 2^-47 of its value, and fixed(x) rounded to a whole number.  The exponent
// in 1024ths of a power of two: its whole part picks a power from the table, and the
// rest goes through a polynomial of degree 3.  Exactly 2^44 for x = top.
struct Weight {
    double c, top;        // c = 1024 log2(e) / T
    const double* table;  // 2^(i / 1024)
    __device__ __forceinline__ Weight(float T, float top_, const double* table_)
        : c(kTable * 1.4426950408889634074 / (double)T), top((double)top_), table(table_) {}
    __device__ __forceinline__ double exponent(float x) const {
        return fmax(((double)x - top) * c, -1000.0 * kTable);  // also of NaN: nothing
    }
    static constexpr double magic = 6755399441055744.0;  // 1.5 2^52: what is added to it is rounded to a whole number
    static __device__ __forceinline__ int whole(double t) { return (int)(unsigned)__builtin_bit_cast(u64, t + magic); }
    __device__ __forceinline__ double scaled(float x) const { return power(exponent(x)); }
    __device__ __forceinline__ double power(double t) const {
        constexpr double a1 = 0.69314718055994530942 / kTable, a2 = a1 * a1 / 2, a3 = a1 * a1 * a1 / 6;
        const int k = whole(t);
        const double r = t - ((t + magic) - magic);
        const double q = fma(fma(fma(a3, r, a2), r, a1), r, 1.0);
        const u64 w = __builtin_bit_cast(u64, table[k & (kTable - 1)] * q);
        return __builtin_bit_cast(double, w + ((u64)(unsigned)(((k >> 10) + kOne) << 20) << 32));
    }
    static __device__ __forceinline__ u64 round(double w) {  // to nearest even, below 2^52
        return __builtin_bit_cast(u64, w + 4503599627370496.0) & (((u64)1 << 52) - 1);
    }
    __device__ __forceinline__ u64 fixed(float x) const { return round(scaled(x)); }
};

// x = m 2^-s in [0, 1), times n: floor, and whether that is all of it.
__device__ __forceinline__ u64 part_of(float x, u64 n, bool* whole) {
    const unsigned u = __builtin_bit_cast(unsigned, x), e = u >> 23;
    const u64 m = e ? (u & 0x7fffffu) | 0x800000u : u;
    const int s = 150 - (int)(e ? e : 1);  // 24 and more
    const u64 lo = m * n, hi = __umul64hi(m, n);
    if (s < 64) {
        *whole = (lo & (((u64)1 << s) - 1)) == 0;
        return (hi << (64 - s)) | (lo >> s);
    }
    if (s < 128) {
        *whole = lo == 0 && (s == 64 || (hi & (((u64)1 << (s - 64)) - 1)) == 0);
        return hi >> (s - 64);
    }
    *whole = m == 0 || n == 0;
    return 0;
}
__device__ __forceinline__ u64 part_up(float x, u64 n) {  // rounded up, at least 1
    bool whole;
    const u64 r = part_of(x, n, &whole);
    return r + (!whole || r == 0);
}

struct Shared {
    u64 hist[kBins];
    double table[kTable];
    unsigned keys[kList];
    int at[kList];
    float tops[kTiles];   // largest value of each tile
    float refs[kTiles];   // what its weight of the first pass is relative to
    u64 sum[kTiles];      // its weight (a double), then that of what is kept of it
    int ties[kTiles];     // slow way: its logits at the border
    float wtop[2][kWaves];
    float wave_f[kWaves];
    double wave_d[kWaves];
    u64 wave[kWaves];
    u64 picked[2];        // measure before the picked bin, and in it
    unsigned bin, lo, hi;
    int index, last;
};

struct Settings {
    float T, top_p, min_p, u;
    int top_k;
    bool by_k, by_p;
};

// What top-k and top-p leave: logits above `key`, and the first `keep` of those at it.
struct Kept {
    unsigned key = 0;
    u64 keep = ~(u64)0;
};

// The weight of a value that min-p keeps, else 0.
struct Weigh {
    const Weight& w;
    double least;
    __device__ __forceinline__ Weigh(const Weight& w_, float min_p) : w(w_), least((double)min_p * (double)((u64)1 << kOne)) {}
    __device__ __forceinline__ u64 operator()(float x) const {
        const double d = w.scaled(x);
        return d >= least ? Weight::round(d) : 0;
    }
};

// ---------------------------------------------------------------- histograms
// hist[bin] += n for the active lanes.  A wave whose lanes all mean one bin adds
// once: rows of few different logits would else wait for one address.
__device__ __forceinline__ void add(u64* hist, int bin, u64 n, bool active) {
    const u64 m = __ballot(active);
    if (!m) return;
    const int first = __builtin_amdgcn_readlane(bin, __builtin_ctzll(m));
    if (__popcll(m) > 8 && __ballot(active && bin == first) == m) {
        const u64 x = last_lane(wave_inclusive(active ? n : 0));
        if ((threadIdx.x & 63) == 0) atomicAdd(&hist[first], x);
        return;
    }
    if (active) atomicAdd(&hist[bin], n);
}

__device__ __forceinline__ void clear_bins(Shared& s) {
    s.hist[threadIdx.x] = 0;
    s.hist[threadIdx.x + kThreads] = 0;
    __syncthreads();
}

// The bin at which the running sum of the histogram reaches the target (>= 1).
// False where the whole falls short of it.
__device__ __forceinline__ bool pick(Shared& s, u64 target, int* bin, u64* before, u64* in) {
    __syncthreads();
    const u64 h0 = s.hist[2 * threadIdx.x], h1 = s.hist[2 * threadIdx.x + 1];
    u64 all;
    const u64 ex = block_exclusive(h0 + h1, s.wave, &all);
    if (all < target) return false;
    if (ex < target && target <= ex + h0 + h1) {
        const bool second = target > ex + h0;
        s.bin = 2 * threadIdx.x + second;
        s.picked[0] = second ? ex + h0 : ex;
        s.picked[1] = second ? h1 : h0;
    }
    __syncthreads();
    *bin = (int)s.bin;
    *before = s.picked[0];
    *in = s.picked[1];
    return true;
}

// A border in the order by falling logit.
struct Border {
    unsigned key;  // logits above it are kept, below it not
    u64 before;    // measure of those above
    u64 in;        // and of those at it
};

// Where the running measure (weights, or the count of logits) of the logits >= low
// reaches the target; false if that is not among those with weight.
template <bool MASS, class Logits>
__device__ __forceinline__ bool find_border(Shared& s, const Logits& logits, const Weight& w, float top, float T, float low, u64 target,
                                            Border& out) {
    auto measure = [&](float x, bool active) { return MASS ? (__ballot(active) ? w.fixed(x) : 0) : (u64)1; };
    // bins of 1/64 of the temperature; the last takes all that has no weight
    const float per_bin = fminf(64.f / T, 1e30f);
    auto bin_of = [&](float x) { return (int)fminf((top - x) * per_bin, (float)(kBins - 1)); };
    auto wanted = [&](float tile_top) { return tile_top >= low; };
    clear_bins(s);
    if (threadIdx.x == 0) s.lo = 0xffffffffu, s.hi = 0;
    logits.each(wanted, [&](int, auto& x) {
#pragma unroll
        for (float v : x) {
            const bool active = v >= low;
            add(s.hist, bin_of(v), measure(v, active), active);
        }
    });
    int bin;
    u64 before, in;
    if (!pick(s, target, &bin, &before, &in) || bin == kBins - 1) return false;
    out.before = before;
    target -= before;
    {
        unsigned lo = 0xffffffffu, hi = 0;
        logits.each(wanted, [&](int, auto& x) {
#pragma unroll
            for (float v : x) {
                const unsigned k = key_of(v);
                if (v >= low && bin_of(v) == bin) {
                    lo = lo < k ? lo : k;
                    hi = hi > k ? hi : k;
                }
            }
        });
        if (hi != 0) {
            atomicMin(&s.lo, lo);
            atomicMax(&s.hi, hi);
        }
    }
    __syncthreads();
    unsigned lo = s.lo, hi = s.hi;
#pragma unroll 1
    while (lo != hi) {
        int shift = 0;
        while ((hi - lo) >> shift >= (unsigned)kBins) ++shift;
        clear_bins(s);
        const float least = value_of(lo), most = value_of(hi);
        logits.each([&](float tile_top) { return tile_top >= least; }, [&](int, auto& x) {
#pragma unroll
            for (float v : x) {
                const bool active = v >= least && v <= most;
                if (__ballot(active)) add(s.hist, active ? (int)((hi - key_of(v)) >> shift) : 0, measure(v, active), active);
            }
        });
        if (!pick(s, target, &bin, &before, &in)) return false;  // not reached: the range's measure is at least the target
        out.before += before;
        target -= before;
        const unsigned above = hi - ((unsigned)bin << shift);
        const unsigned room = ((1u << shift) - 1) < above - lo ? (1u << shift) - 1 : above - lo;
        lo = above - room;
        hi = above;
    }
    out.key = lo;
    out.in = in;
    return true;
}

__device__ __forceinline__ void answer(const SampleArgs& a, int64_t r, int token, double weight, double total) {
    a.token[r] = token;
    if (a.logprob) a.logprob[r] = (float)log(weight / total);
}

// ------------------------------------------------------- rows without a filter
// The token from the tiles' weights, `mine` of this thread's.
template <typename T>
__device__ __forceinline__ void draw_from_tiles(Shared& s, const Row<T>& row, const Weight& w, double mine, const Settings& c,
                                                const SampleArgs& a, int64_t r) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (threadIdx.x == 0) s.index = 0;
    double total;
    const double before = block_exclusive(mine, s.wave_d, &total), at = (double)c.u * total;
    // the last tile that begins at or before the place: one with weight, since sums only grow there
    if (const u64 m = __ballot(mine > 0 && before <= at); m && lane == 63 - __builtin_clzll(m)) atomicMax(&s.index, (int)threadIdx.x);
    __syncthreads();
    const int tile = s.index, j = tile / kWaves;
    if ((int)threadIdx.x == tile) s.wave_d[0] = at - before;
    __syncthreads();
    if (wave != tile % kWaves) return;
    const double left = s.wave_d[0];
    float x[E];
    row.values(row.load(j), x);
    u64 v[E], sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) sum += v[e] = w.fixed(x[e]);
    u64 run = wave_inclusive(sum) - sum;
    // the first value whose running weight exceeds it; where the tile's sum is less by
    // what rounding the weights left out, the last value with weight
    int found = -1, last = -1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (v[e]) last = e;
        if ((double)run <= left && left < (double)(run + v[e])) found = e;
        run += v[e];
    }
    const u64 some = __ballot(found >= 0), any = __ballot(last >= 0);
    const int at_lane = some ? __builtin_ctzll(some) : 63 - __builtin_clzll(any);
    if (lane != at_lane) return;
    if (!some) found = last;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e == found) answer(a, r, row.index(j, e), (double)v[e], total);
}

// Rows whose largest logit is infinite: the tokens that have it, equal ones.
template <typename T>
__device__ __forceinline__ void draw_infinite(Shared& s, const Row<T>& row, float top, const Settings& c, const SampleArgs& a, int64_t r) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (threadIdx.x < kTiles) s.sum[threadIdx.x] = 0;
    __syncthreads();
    auto count = [&](const float (&x)[E]) {
        int n = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) n += x[e] == top;
        return n;
    };
    row.each([&](float tile_top) { return tile_top == top; }, [&](int j, const float (&x)[E]) {
        const int n = last_lane(wave_inclusive(count(x)));
        if (lane == 0) s.sum[j * kWaves + wave] = (u64)n;
    });
    __syncthreads();
    const u64 mine = threadIdx.x < kTiles ? s.sum[threadIdx.x] : 0;
    u64 n;
    const u64 before = block_exclusive(mine, s.wave, &n);
    if (c.by_k && (u64)c.top_k < n) n = (u64)c.top_k;
    if (c.by_p) n = part_up(c.top_p, n);
    bool whole;
    const u64 at = part_of(c.u, n, &whole);
    if (before <= at && at < before + mine) {
        s.bin = threadIdx.x;
        s.picked[0] = at - before;
    }
    __syncthreads();
    const int tile = (int)s.bin, j = tile / kWaves;
    if (wave != tile % kWaves) return;
    float x[E];
    row.values(row.load(j), x);
    const int here = count(x);
    int run = wave_inclusive(here) - here;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (x[e] == top && run++ == (int)s.picked[0]) answer(a, r, row.index(j, e), 1.0, (double)n);
}

// ------------------------------------------------------------------ the list
// The least value for which `is` holds, as it does for `top` and all values from
// the one asked for up to it: 64 keys at a time.
template <class P>
__device__ __forceinline__ float least_value(float top, P&& is) {
    unsigned no = key_of(neg_inf()), yes = key_of(top);  // not a logit with weight, and one for which it holds
    while (yes - no > 1) {
        const unsigned step = (yes - no - 1) / 64 + 1, left = (yes - no - 1) / step;  // so many keys lie between
        const unsigned lane = threadIdx.x & 63, key = no + (lane + 1) * step;
        const u64 m = __ballot(lane < left && is(value_of(key)));
        const int first = m ? __builtin_ctzll(m) : (int)left;
        if (m) yes = no + (first + 1) * step;
        no += first * step;
    }
    return value_of(yes);
}

// Logits from `lo` on and below `hi` go into the list, and the weights of those from
// `hi` on become their tiles' sums; false if there are too many.
template <typename T>
__device__ __forceinline__ bool gather(Shared& s, const Row<T>& row, const Weight& w, float lo, float hi, List& list) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (threadIdx.x == 0) s.index = 0;
    if (threadIdx.x < kTiles) s.sum[threadIdx.x] = 0;
    __syncthreads();
    row.each([&](float x) { return x >= lo; }, [&](int j, const float (&x)[E]) {
        bool any = false;
#pragma unroll
        for (int e = 0; e < E; ++e) any |= x[e] >= hi;
        if (__ballot(any)) {
            u64 sum = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const u64 v = w.fixed(x[e]);
                sum += x[e] >= hi ? v : 0;
            }
            sum = wave_inclusive(sum);
            if (lane == 63) s.sum[j * kWaves + wave] = sum;
        }
        int mine = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) mine += x[e] >= lo && x[e] < hi;
        const int incl = wave_inclusive(mine), all = last_lane(incl);
        if (all == 0) return;
        int base = 0;
        if (lane == 0) base = atomicAdd(&s.index, all);
        int to = __builtin_amdgcn_readfirstlane(base) + incl - mine;
        if (to + mine > kList) return;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (x[e] >= lo && x[e] < hi) {
                s.keys[to] = key_of(x[e]);
                s.at[to++] = row.index(j, e);
            }
    });
    __syncthreads();
    list = {s.keys, s.at, s.index};
    return list.n <= kList;
}

// Where the running measure of a list in order of index reaches the target (which
// it does).
template <class F>
__device__ __forceinline__ int find_index(Shared& s, const List& list, int V, u64 target, F&& measure) {
    int lo = 0, shift = 0;
    while ((V - 1) >> shift >= kBins) ++shift;
#pragma unroll 1
    for (;;) {
        clear_bins(s);
#pragma unroll 1
        for (int i = threadIdx.x; i < list.n; i += kThreads) {
            const int d = list.at[i] - lo;
            if (d >= 0 && d >> shift < kBins)
                if (const u64 m = measure(i)) atomicAdd(&s.hist[d >> shift], m);
        }
        int bin;
        u64 before, in;
        pick(s, target, &bin, &before, &in);
        target -= before;
        lo += bin << shift;
        if (shift == 0) return lo;
        shift = 0;  // the histogram takes that bin and what follows it, which the target does not reach
    }
}

// top-k and top-p on a list, above which `n_above` logits are.  goal: the weight to
// reach from the top of the row on, 0 where the list tells.  A list that ends where
// min-p does may fall short of the targets, and is then kept as a whole.
__device__ __forceinline__ bool filter_list(Shared& s, const List& list, const Weight& w, float top, const Settings& c, u64 n_above,
                                            u64 goal, bool short_list, Kept& kept, bool* all_ties) {
    *all_ties = true;
    u64 spare = 0;  // weight at the border that top-k has dropped
    if (c.by_k) {
        Border b;
        if (find_border<false>(s, list, w, top, c.T, neg_inf(), (u64)c.top_k - n_above, b)) {
            kept.key = b.key;
            kept.keep = c.top_k - n_above - b.before;
            *all_ties = kept.keep == b.in;
            spare = (b.in - kept.keep) * w.fixed(value_of(b.key));
        } else if (n_above) {
            return false;
        }  // else the list is shorter, or what lies at the border has no weight
    }
    if (!c.by_p) return true;
    const float low = kept.key == 0 ? neg_inf() : value_of(kept.key);
    u64 sum = 0, all;
    if (goal == 0) {  // the list holds all that top-k keeps, or the whole row
        list.each(0, [&](int, auto& x) {
#pragma unroll
            for (float v : x) sum += v >= low ? w.fixed(v) : 0;
        });
        block_exclusive(sum, s.wave, &all);
        goal = part_up(c.top_p, all - spare);
    } else {
        sum = threadIdx.x < kTiles ? s.sum[threadIdx.x] : 0;
        block_exclusive(sum, s.wave, &all);
        if (goal <= all) return false;
        goal -= all;
    }
    Border b;
    if (!find_border<true>(s, list, w, top, c.T, low, goal, b)) return short_list;
    const u64 each = w.fixed(value_of(b.key));
    kept.key = b.key;
    kept.keep = (goal - b.before + each - 1) / each;
    *all_ties = kept.keep * each == b.in;
    return true;
}

// The token among the tiles' sums and what is kept of the list.
template <typename T>
__device__ __forceinline__ void draw_from_list(Shared& s, const Row<T>& row, const List& list, const Weight& w, const Settings& c,
                                               const Kept& kept, bool all_ties, const SampleArgs& a, int64_t r) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Weigh weigh(w, c.min_p);
    int last = 0x7fffffff;  // the index of the last tie that is kept
    if (!all_ties) last = find_index(s, list, a.V, kept.keep, [&](int i) { return (u64)(list.keys[i] == kept.key); });
    auto measure = [&](unsigned k, int index, float x) { return k > kept.key || (k == kept.key && index <= last) ? weigh(x) : 0; };
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < list.n; i += kThreads) {
        const u64 m = measure(list.keys[i], list.at[i], value_of(list.keys[i]));
        if (m) atomicAdd(&s.sum[(list.at[i] + row.off) / kTile], m);
    }
    __syncthreads();
    const u64 mine = threadIdx.x < kTiles ? s.sum[threadIdx.x] : 0;
    u64 total;
    const u64 before = block_exclusive(mine, s.wave, &total);
    bool whole;
    const u64 at = part_of(c.u, total, &whole);
    if (before <= at && at < before + mine) {
        s.bin = threadIdx.x;
        s.picked[0] = at - before;
    }
    __syncthreads();
    const int tile = (int)s.bin, j = tile / kWaves;
    if (wave != tile % kWaves) return;
    const u64 left = s.picked[0];
    float x[E];
    row.values(row.load(j), x);
    u64 v[E], sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) sum += v[e] = x[e] == x[e] ? measure(key_of(x[e]), row.index(j, e), x[e]) : 0;
    u64 run = wave_inclusive(sum) - sum;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (run <= left && left < run + v[e]) answer(a, r, row.index(j, e), (double)v[e], (double)total);
        run += v[e];
    }
}

// The same for a list of up to 64 H that all that is kept is in, by one wave, H
// logits per lane: each finds what stands before it, in the order of logits and then,
// among what is kept, in the order of indices.  False as filter_list's.
template <int H>
__device__ __forceinline__ bool draw_from_few(const List& list, const Weight& w, const Settings& c, u64 goal, bool short_list,
                                              const SampleArgs& a, int64_t r) {
    const int lane = threadIdx.x & 63;
    const Weigh weigh(w, c.min_p);
    unsigned key[H];
    int at[H], rank[H] = {};
    u64 v[H], before[H] = {}, all = 0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int i = 64 * h + lane;
        key[h] = i < list.n ? list.keys[i] : 0;
        at[h] = i < list.n ? list.at[i] : 0x7fffffff;
        v[h] = i < list.n ? w.fixed(value_of(key[h])) : 0;
    }
    auto others = [&](auto&& f) {  // f(key, index, weight) of each
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int n = list.n - 64 * h < 64 ? list.n - 64 * h : 64;
            for (int i = 0; i < n; ++i) f(lane_of(key[h], i), lane_of(at[h], i), lane_of(v[h], i));
        }
    };
    others([&](unsigned k, int p, u64 m) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const bool first = k > key[h] || (k == key[h] && p < at[h]);
            rank[h] += first;
            before[h] += first ? m : 0;
        }
    });
#pragma unroll
    for (int h = 0; h < H; ++h) all += !c.by_k || rank[h] < c.top_k ? v[h] : 0;
    all = last_lane(wave_inclusive(all));
    if (goal == 0) goal = part_up(c.top_p, all);  // the list holds all that top-k keeps, or the whole row
    if (c.by_p && all < goal && !short_list) return false;
    u64 total = 0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const bool kept = (!c.by_k || rank[h] < c.top_k) && (!c.by_p || before[h] < goal);
        v[h] = 64 * h + lane < list.n && kept ? weigh(value_of(key[h])) : 0;
        total += v[h];
        before[h] = 0;
    }
    total = last_lane(wave_inclusive(total));
    bool whole;
    const u64 to = part_of(c.u, total, &whole);
    others([&](unsigned, int p, u64 m) {
#pragma unroll
        for (int h = 0; h < H; ++h) before[h] += p < at[h] ? m : 0;
    });
#pragma unroll
    for (int h = 0; h < H; ++h)
        if (before[h] <= to && to < before[h] + v[h]) answer(a, r, at[h], (double)v[h], (double)total);
    return true;
}

// -------------------------------------------------------------- the slow way
// The same with passes over the whole row.
template <typename T>
__device__ __forceinline__ void draw_from_row(Shared& s, const Row<T>& row, const Weight& w, float top, const Settings& c, double weight,
                                              const SampleArgs& a, int64_t r) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float border = neg_inf();  // logits above it are kept, of those at it the first `keep`
    u64 keep = ~(u64)0;
    bool every = true;
    Border b;
    u64 spare = 0;
    if (c.by_k && find_border<false>(s, row, w, top, c.T, neg_inf(), (u64)c.top_k, b)) {
        border = value_of(b.key);
        keep = c.top_k - b.before;
        every = false;
        spare = (b.in - keep) * w.fixed(border);
    }
    if (c.by_p) {
        u64 goal;
        if (weight > 0) {
            goal = (u64)ceil((double)c.top_p * weight * (1 - 0x1p-48));
            goal += goal == 0;
        } else {
            u64 sum = 0, all;
            row.each([&](float tile_top) { return tile_top >= border; }, [&](int, const float (&x)[E]) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (__ballot(x[e] >= border)) {
                        const u64 v = w.fixed(x[e]);
                        sum += x[e] >= border ? v : 0;
                    }
            });
            block_exclusive(sum, s.wave, &all);
            goal = part_up(c.top_p, all - spare);
        }
        if (find_border<true>(s, row, w, top, c.T, border, goal, b)) {
            border = value_of(b.key);
            const u64 each = w.fixed(border);
            keep = (goal - b.before + each - 1) / each;
            every = false;
        }
    }
    const Weigh weigh(w, c.min_p);
    const u64 at_border = every ? 0 : weigh(border);
    if (threadIdx.x < kTiles) s.sum[threadIdx.x] = 0, s.ties[threadIdx.x] = 0;
    __syncthreads();
    auto is_tie = [&](float x) { return x == border && !every; };
    row.each([&](float tile_top) { return tile_top >= border; }, [&](int j, const float (&x)[E]) {
        u64 sum = 0;
        int ties = 0;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (__ballot(x[e] >= border)) {
                ties += is_tie(x[e]);
                const u64 v = weigh(x[e]);
                sum += x[e] >= border && !is_tie(x[e]) ? v : 0;
            }
        sum = wave_inclusive(sum);
        ties = wave_inclusive(ties);
        if (lane == 63) {
            s.sum[j * kWaves + wave] = sum;
            s.ties[j * kWaves + wave] = ties;
        }
    });
    __syncthreads();
    // a thread per tile, in order of index: its ties that are kept, its weight
    const int t = threadIdx.x, n = t < kTiles ? s.ties[t] : 0;
    u64 all_ties, total;
    const u64 ties_before = block_exclusive((u64)n, s.wave, &all_ties);
    const u64 room = keep > ties_before ? keep - ties_before : 0;
    const u64 mine = (t < kTiles ? s.sum[t] : 0) + at_border * (room < (u64)n ? room : (u64)n);
    const u64 before = block_exclusive(mine, s.wave, &total);
    bool whole;
    const u64 at = part_of(c.u, total, &whole);
    if (before <= at && at < before + mine) {
        s.bin = t;
        s.picked[0] = at - before;
        s.picked[1] = ties_before;
    }
    __syncthreads();
    const int tile = (int)s.bin, j = tile / kWaves;
    if (wave != tile % kWaves) return;
    const u64 left = s.picked[0];
    float x[E];
    row.values(row.load(j), x);
    int ties = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) ties += is_tie(x[e]);
    u64 used = s.picked[1] + wave_inclusive(ties) - ties;
    u64 v[E], sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool tie = is_tie(x[e]);
        v[e] = x[e] >= border && (!tie || used < keep) ? weigh(x[e]) : 0;
        used += tie;
        sum += v[e];
    }
    u64 run = wave_inclusive(sum) - sum;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (run <= left && left < run + v[e]) answer(a, r, row.index(j, e), (double)v[e], (double)total);
        run += v[e];
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), t = threadIdx.x;
    const Row<T> row((const T*)a.logits + r * a.stride, a.V, s.tops);
    typename Row<T>::Raw raw = row.load(0);

    Settings c;
    c.T = a.temperature ? a.temperature[r] : a.T;
    c.top_k = a.top_k ? a.top_k[r] : a.k;
    c.top_p = a.top_p ? a.top_p[r] : a.p;
    c.min_p = a.min_p ? a.min_p[r] : a.mp;
    c.u = a.u[r];
    if (!(c.top_p >= 0.f)) c.top_p = c.top_p != c.top_p ? 1.f : 0.f;
    if (!(c.min_p <= 1.f)) c.min_p = c.min_p != c.min_p ? 0.f : 1.f;
    c.u = c.u >= 0.f ? fminf(c.u, 0x1.fffffep-1f) : 0.f;
    c.by_k = c.top_k > 0 && c.top_k < a.V;
    c.by_p = c.top_p < 1.f;
    const bool greedy = !(c.T > 0.f), small = a.V <= kList;  // a small row is a list
    const bool maxima = !greedy && !small && c.by_k && c.top_k <= kByMaxima;
    const bool counts = !greedy && !small && !maxima && (c.by_k || c.by_p);
    const bool weights = !greedy && !c.by_k && (c.by_p ? !small : !(c.min_p > 0.f));

    if (!greedy) s.table[t] = exp2((double)t / kTable);
    if (t < kTiles) s.tops[t] = neg_inf();
    unsigned* const count = (unsigned*)s.hist;
    clear_bins(s);
    float best = neg_inf();            // of this thread
    float top = neg_inf(), ref = 0.f;  // bins count from ref, a value that was the largest
    int newest = 0;                    // the bin of the largest so far
    bool lost = false;                 // bins fell out that may matter
#pragma unroll 1
    for (int j = 0; j < row.steps; ++j) {
        typename Row<T>::Raw more = raw;
        if (j + 1 < row.steps) more = row.load(j + 1);
        float x[E];
        row.values(raw, x);
        raw = more;
        float m = x[0];
#pragma unroll
        for (int e = 1; e < E; ++e) m = fmaxf(m, x[e]);
        best = fmaxf(best, m);
        m = wave_max(m);
        const int tile = j * kWaves + wave;
        if (lane == 0) s.tops[tile] = m;
        float by = m;  // what the tile's weight is relative to
        if (counts) {
            const float old = top;
            if (lane == 0) s.wtop[j & 1][wave] = m;
            __syncthreads();
            top = fmaxf(top, wave_max(s.wtop[j & 1][lane % kWaves]));
            if (top > old) {
                const double exponent = Weight(c.T, ref, s.table).exponent(top);
                int now = 0, n = kBins;
                if (old != neg_inf() && exponent < (newest + kBins) * (double)(1 << kBinShift) && newest < kMostBin) {
                    now = Weight::whole(exponent) >> kBinShift;
                    n = now - newest;
                } else {  // all bins fall out
                    lost = lost || newest >= kMostBin;
                    ref = top;
                }
                // bins come in at the top, in the place of those that fall out at the bottom
                for (int i = t; i < n; i += kThreads) count[(now - i) & (kBins - 1)] = 0;
                newest = now;
                __syncthreads();
            }
            by = ref;
        }
        if (m == neg_inf() || !(counts || weights)) {
            if (lane == 0) s.sum[tile] = 0, s.refs[tile] = m;
            continue;
        }
        const Weight w(c.T, by, s.table);
        double exponent[E];
#pragma unroll
        for (int e = 0; e < E; ++e) exponent[e] = w.exponent(x[e]);
        if (weights) {
            double sum = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) sum += w.power(exponent[e]);
            sum = wave_inclusive(sum);
            if (lane == 63) s.sum[tile] = __builtin_bit_cast(u64, sum), s.refs[tile] = by;
        }
        if (counts) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int b = Weight::whole(exponent[e]) >> kBinShift;
                if (x[e] > neg_inf() && newest - b < kBins - 1) atomicAdd(&count[b & (kBins - 1)], 1u);
            }
        }
    }
    __syncthreads();
    top = neg_inf();
    for (int i = lane; i < kTiles; i += 64) top = fmaxf(top, s.tops[i]);
    top = wave_max(top);
    if (greedy || top == neg_inf()) {
        if (t == 0) s.index = 0x7fffffff;
        __syncthreads();
        int at = 0x7fffffff;
        row.each([&](float tile_top) { return tile_top == top; }, [&](int j, const float (&x)[E]) {
#pragma unroll
            for (int e = E - 1; e >= 0; --e)
                if (x[e] == top) {
                    const int i = row.index(j, e);
                    at = i < at ? i : at;
                }
        });
        if (at != 0x7fffffff) atomicMin(&s.index, at);
        __syncthreads();
        if (t == 0) {
            const bool none = top == neg_inf();
            a.token[r] = none ? -1 : s.index;
            if (a.logprob) a.logprob[r] = none ? __builtin_nanf("") : 0.f;
        }
        return;
    }
    if (top == -neg_inf()) {
        draw_infinite(s, row, top, c, a, r);
        return;
    }

    const Weight w(c.T, top, s.table);
    double weight = 0;  // of the row, in 2^-44
    if (weights) {      // a tile's, relative to the row's maximum; 0 where no value of it has any
        const float m = t < kTiles ? s.tops[t] : neg_inf();
        const double mine = w.fixed(m) ? __builtin_bit_cast(double, s.sum[t]) * (w.scaled(s.refs[t]) * 0x1p-44) : 0.0;
        if (!c.by_p) {
            draw_from_tiles(s, row, w, mine, c, a, r);
            return;
        }
        block_exclusive(mine, s.wave_d, &weight);
    }

    // the list need not reach below min-p, unless top-p takes a weight from it
    const bool part = c.min_p > 0.f && !(c.by_p && (c.by_k || small));
    const float floor_x = part ? top + c.T * (0.69314718f * __builtin_amdgcn_logf(c.min_p) - 0.001f) : neg_inf();
    float lo = floor_x, hi = -neg_inf();
    u64 n_above = 0, goal = 0;
    bool fits = true, short_list = part;  // the list ends at min-p
    if (maxima) {
        // bins of 1/64 of the temperature; the last takes all that has no weight
        const float per_bin = fminf(64.f / c.T, 1e30f);
        auto bin_of = [&](float x) { return (int)fminf((top - x) * per_bin, (float)(kBins - 1)); };
        add(s.hist, bin_of(best), 1, true);
        int bin;
        u64 before, in;
        pick(s, (u64)c.top_k, &bin, &before, &in);
        bin = bin < kBins - 1 ? bin : kBins - 2;
        lo = fmaxf(lo, least_value(top, [&](float x) { return bin_of(x) <= bin; }));
    }
    if (counts) {
        const Weight by(c.T, ref, s.table);
        const int floor_bin = Weight::whole(by.exponent(floor_x)) >> kBinShift;
        // the two bins of this thread, from the newest down, and what their counts weigh at least
        const int i = 2 * t, end = (part && newest - floor_bin < kWhole ? newest - floor_bin + 1 : kWhole) / 2;
        const unsigned n0 = i < kWhole ? count[(newest - i) & (kBins - 1)] : 0, n1 = i + 1 < kWhole ? count[(newest - i - 1) & (kBins - 1)] : 0;
        u64 all;
        const u64 before = block_exclusive((u64)(n0 + n1), s.wave, &all), upto = before + n0 + n1;
        bool may = false, must = false;  // the border may lie in these bins, or above or in them
        if (c.by_k) {
            may = must = upto >= (u64)c.top_k;
        } else {
            // exponents are rounded: the least of a bin's is half a step below its first
            const float deep = (float)((double)((newest - i) * 16) - 0.5 - by.exponent(top)) * (1.f / kTable);
            const float w0 = __builtin_amdgcn_exp2f(deep), mine = (float)n0 * w0 + (float)n1 * (w0 * 0.98922819f);  // 2^(-1/64)
            float sum;
            const float least = block_exclusive(mine, s.wave_f, &sum) + mine;
            goal = (u64)ceil((double)c.top_p * weight * (1 - 0x1p-48));  // what rounding added to the weight takes no logit in
            goal += goal == 0;
            const float want = (float)goal * 0x1p-44f;
            must = least >= want * 1.0005f;
            may = least * 1.0115f >= want;  // 2^(1/64), and as much for rounding on either side
        }
        // the border's pairs of bins: from the first that may hold it to the first that it cannot lie below
        if (t == 0) s.index = s.last = kThreads;
        __syncthreads();
        if (const u64 m = __ballot(may); m && lane == __builtin_ctzll(m)) atomicMin(&s.index, t);
        if (const u64 m = __ballot(must); m && lane == __builtin_ctzll(m)) atomicMin(&s.last, t);
        __syncthreads();
        const int first = s.index < end ? s.index : end, last = s.last < end ? s.last : end;
        fits = !lost && (s.last < kWhole / 2 || (part && end < kWhole / 2));
        short_list = part && last == end;
        if (t == last) s.picked[0] = upto;
        if (t == first) s.picked[1] = before;
        __syncthreads();
        auto from_bin = [&](int b) {
            return least_value(top, [&](float x) { return Weight::whole(by.exponent(x)) >= b * (1 << kBinShift); });
        };
        lo = fmaxf(lo, from_bin(newest - 2 * last - 1));
        const u64 most = s.picked[0], skipped = s.picked[1];
        if (most > (u64)kList) {  // only the bins themselves
            const int first_bin = newest - 2 * first;
            if (first > 0) hi = from_bin(first_bin + 1);
            n_above = skipped;
            fits = fits && most - skipped <= (u64)kList && !(c.by_k && c.by_p) && !(part && first_bin <= floor_bin);
        }
        __syncthreads();
    }
    lo = fmaxf(lo, -3.402823466e38f);  // not -infinity
    List list;
    if (fits && gather(s, row, w, lo, hi, list)) {
        if (list.n <= kOneWave && hi == -neg_inf()) {
            if (wave == 0) {
                const bool ok = list.n <= 64 ? draw_from_few<1>(list, w, c, goal, short_list, a, r)
                                             : draw_from_few<2>(list, w, c, goal, short_list, a, r);
                if (t == 0) s.bin = ok;
            }
            __syncthreads();
            if (s.bin) return;
        } else {
            Kept kept;
            bool all_ties;
            if (filter_list(s, list, w, top, c, n_above, goal, short_list, kept, &all_ties)) {
                draw_from_list(s, row, list, w, c, kept, all_ties, a, r);
                return;
            }
        }
    }
    __syncthreads();
    draw_from_row(s, row, w, top, c, weight, a, r);
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
    const dim3 gr((unsigned)a.rows), bl(kThreads);
    if (a.f32) sample_kernel<float><<<gr, bl, 0, s>>>(a);
    else sample_kernel<__bf16><<<gr, bl, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace e2ttt
