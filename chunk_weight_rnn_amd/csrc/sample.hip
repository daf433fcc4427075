// One token for each row of logits, by temperature, top-k, top-p and min-p,
// from a given random number of the row (the definition is in
// include/e2ttt_tokens.h).
//
// A workgroup holds a row in the LDS (rows of more than 128 KiB are read again for
// each pass, from the cache).  Nothing is sorted: a filter keeps a
// stretch of the order by falling logit, so what it needs is the logit at which
// the running count or weight reaches a target, found with a histogram in the
// LDS over ever smaller ranges: first 2048 bins evenly over the logits that have
// weight, then 2048 over the bit patterns of the bin's logits, until one value
// is left.  Equal logits at the border are kept by index.
//
// Weights are whole multiples of 2^-44 of the largest, so that sums of up to 2^18
// of them are exact in 64 bits: any order of summation gives the same, and the
// border cases of the definition (a target met exactly) come out as written.
// The exponential is computed in 64 bits, to 2^-47 of its value: a table of 64
// powers of two and a polynomial of degree 5.
#include "tokens_internal.h"

namespace e2ttt {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2 * kThreads;
constexpr int kOne = 44;        // a weight of one is 2^44
constexpr int kTiles = 1024;    // pieces of a row that a wave holds side by side, at most

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// A logit as it is used: NaN is never chosen, and zeros are equal.
__device__ __forceinline__ unsigned clean(unsigned u, __bf16) {  // two of them
    unsigned r = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        unsigned x = (u >> (16 * h)) & 0xffffu;
        if ((x & 0x7fffu) > 0x7f80u) x = 0xff80u;
        if (x == 0x8000u) x = 0;
        r |= x << (16 * h);
    }
    return r;
}
__device__ __forceinline__ unsigned clean(unsigned u, float) {
    if ((u & 0x7fffffffu) > 0x7f800000u) u = 0xff800000u;
    return u == 0x80000000u ? 0u : u;
}
// Order of the values as whole numbers.
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}

template <typename T>
__device__ __forceinline__ void values(u32x4 u, float (&x)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            x[2 * w] = __builtin_bit_cast(float, u[w] << 16);
            x[2 * w + 1] = __builtin_bit_cast(float, u[w] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const unsigned one = u[w];
            x[w] = __builtin_bit_cast(float, one);
        }
    }
}

// A row in units of 16 bytes, E values, from the last address on at or before its
// first value that 16 divides: unit j kThreads + thread is this thread's j-th.
// NU > 0: up to NU of them in the LDS, where each thread reads what it wrote
// itself; 0: in memory.  Places before and past the row hold -infinity.
template <typename T, int NU>
struct Row {
    static constexpr int E = 16 / sizeof(T);
    const T* p;  // aligned
    int off, V;  // places before the row, values in it
    int steps;
    u32x4* lds;
    __device__ __forceinline__ Row(const T* row, int V_, u32x4* lds_) : V(V_), lds(lds_) {
        off = (int)((uintptr_t)row % 16 / sizeof(T));
        p = row - off;
        steps = (V + off + E * kThreads - 1) / (E * kThreads);
    }
    // Index of value e of this thread's unit of step j.
    __device__ __forceinline__ int index(int j, int e) const { return (j * kThreads + (int)threadIdx.x) * E + e - off; }
    __device__ __forceinline__ u32x4 load(int j) const {
        const int first = index(j, 0);
        u32x4 u;
        if (first >= 0 && first + E <= V) {
            u = *(const u32x4*)(p + off + first);
        } else {
            T t[E];
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = first + e >= 0 && first + e < V ? p[off + first + e] : (T)neg_inf();
            __builtin_memcpy(&u, t, 16);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) u[w] = clean(u[w], T{});
        return u;
    }
    // f(j, values) for every step j, all threads together; `fresh`: from memory,
    // into the LDS.
    template <bool FRESH = false, class F>
    __device__ __forceinline__ void each(F&& f) const {
        float x[E];
        if constexpr (NU > 0 && !FRESH) {
#pragma unroll 1
            for (int j = 0; j < steps; ++j) {
                values<T>(lds[j * kThreads + threadIdx.x], x);
                f(j, x);
            }
        } else {
            u32x4 next = load(0);
#pragma unroll 1
            for (int j = 0; j < steps; ++j) {
                const u32x4 u = next;
                if (j + 1 < steps) next = load(j + 1);
                if constexpr (NU > 0) lds[j * kThreads + threadIdx.x] = u;
                values<T>(u, x);
                f(j, x);
            }
        }
    }
};

// Weights: scaled(x) = 2^44 exp((x - max) / T) in 64 bits, fixed(x) rounded to a
// whole number.
struct Weight {
    double c, max;  // c = 64 log2(e) / T
    float top;
    const double* table;  // 2^(i / 64)
    __device__ __forceinline__ double scaled(float x) const {
        double t = ((double)x - max) * c;
        t = fmax(t, -64.0 * 47);  // -infinity, and NaN of infinities, to a weight that rounds to 0
        const double k = rint(t), r = (t - k) * (0.69314718055994530942 / 64);
        double q = 1.0 / 120;
        q = fma(q, r, 1.0 / 24);
        q = fma(q, r, 1.0 / 6);
        q = fma(q, r, 0.5);
        q = fma(q, r, 1.0);
        q = fma(q, r, 1.0);
        const int i = (int)k;
        const double w = ldexp(table[i & 63] * q, (i >> 6) + kOne);
        return x == top ? (double)((u64)1 << kOne) : w;
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

struct Shared {
    u64 hist[kBins];
    double table[64];
    u64 sum[kTiles];     // weight of what is kept without question, of each tile
    int ties[kTiles];    // logits at the border
    u64 wave[kWaves];
    u64 picked[2];       // measure before the picked bin, and in it
    unsigned bin, lo, hi;
    int index;
};

template <typename X>
__device__ __forceinline__ X wave_inclusive(X x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const X y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// Sum of x over the threads before this one, and over all of them.
__device__ __forceinline__ u64 block_exclusive(u64 x, u64* wave_sums, u64* total) {
    const int wave = threadIdx.x >> 6;
    const u64 incl = wave_inclusive(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) wave_sums[wave] = incl;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += wave_sums[w];
        all += wave_sums[w];
    }
    *total = all;
    return before + incl - x;
}

// hist[bin] += n for the active lanes.  A wave whose lanes all mean one bin adds
// once: rows of few different logits would else wait for one address.
__device__ __forceinline__ void add(u64* hist, int bin, u64 n, bool active) {
    const u64 m = __ballot(active);
    if (!m) return;
    const int first = __builtin_amdgcn_readlane(bin, __builtin_ctzll(m));
    if (__popcll(m) > 8 && __ballot(active && bin == first) == m) {
        u64 x = active ? n : 0;
#pragma unroll
        for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
        if ((threadIdx.x & 63) == 0) atomicAdd(&hist[first], x);
        return;
    }
    if (active) atomicAdd(&hist[bin], n);
}

// The bin at which the running sum of the histogram reaches the target (>= 1).
// False where the whole falls short of it.
__device__ __forceinline__ bool pick(Shared& s, u64 target, int* bin, u64* before, u64* in) {
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
    __syncthreads();
    return true;
}

__device__ __forceinline__ void clear_bins(Shared& s) {
    s.hist[threadIdx.x] = 0;
    s.hist[threadIdx.x + kThreads] = 0;
    __syncthreads();
}

// A border in the order by falling logit.
struct Border {
    unsigned key;  // logits above it are kept, below it not
    u64 before;    // measure of those above
    u64 in;        // and of those at it
};

// Where the running measure (weights, or the count of logits) of the logits with
// keys >= low reaches the target; false if that is not among those with weight.
template <bool MASS, typename T, int NU>
__device__ __forceinline__ bool find_border(Shared& s, const Row<T, NU>& row, const Weight& w, float per_bin, unsigned low, u64 target,
                                            Border& out) {
    constexpr int E = Row<T, NU>::E;
    auto measure = [&](float x, bool active) { return MASS ? (__ballot(active) ? w.fixed(x) : 0) : (u64)1; };
    // bins of 1/64 of the temperature; the last takes all that has no weight
    auto bin_of = [&](float x) {
        const float d = w.top - x;  // NaN: both are infinite
        return d > 0.f ? (int)fminf(d * per_bin, (float)(kBins - 1)) : 0;
    };
    clear_bins(s);
    row.each([&](int, const float (&x)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const bool active = key_of(x[e]) >= low;
            add(s.hist, bin_of(x[e]), measure(x[e], active), active);
        }
    });
    __syncthreads();
    int bin;
    u64 before, in;
    if (!pick(s, target, &bin, &before, &in) || bin == kBins - 1) return false;
    out.before = before;
    target -= before;
    if (threadIdx.x == 0) s.lo = 0xffffffffu, s.hi = 0;
    __syncthreads();
    {
        unsigned lo = 0xffffffffu, hi = 0;
        row.each([&](int, const float (&x)[E]) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const unsigned k = key_of(x[e]);
                if (k >= low && bin_of(x[e]) == bin) {
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
    while (lo != hi) {
        int shift = 0;
        while ((hi - lo) >> shift >= (unsigned)kBins) ++shift;
        clear_bins(s);
        row.each([&](int, const float (&x)[E]) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const unsigned k = key_of(x[e]);
                const bool active = k >= lo && k <= hi;
                if (__ballot(active)) add(s.hist, active ? (int)((hi - k) >> shift) : 0, measure(x[e], active), active);
            }
        });
        __syncthreads();
        if (!pick(s, target, &bin, &before, &in)) return false;  // not reached: the range's measure is at least the target
        out.before += before;
        target -= before;
        const unsigned top = hi - ((unsigned)bin << shift);
        const unsigned room = ((1u << shift) - 1) < top - lo ? (1u << shift) - 1 : top - lo;
        lo = top - room;
        hi = top;
    }
    out.key = lo;
    out.in = in;
    return true;
}

template <typename T, int NU>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
    constexpr int E = 16 / sizeof(T);
    __shared__ Shared s;
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    __shared__ u32x4 held[NU ? NU * kThreads : 1];
    const Row<T, NU> row((const T*)a.logits + r * a.stride, a.V, held);
    if (threadIdx.x < 64) s.table[threadIdx.x] = exp2((double)threadIdx.x / 64);

    float T0 = a.temperature ? a.temperature[r] : a.T;
    int top_k = a.top_k ? a.top_k[r] : a.k;
    float top_p = a.top_p ? a.top_p[r] : a.p, min_p = a.min_p ? a.min_p[r] : a.mp, u = a.u[r];
    if (!(top_p >= 0.f)) top_p = top_p != top_p ? 1.f : 0.f;
    if (!(min_p <= 1.f)) min_p = min_p != min_p ? 0.f : 1.f;
    u = u >= 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;

    // the largest, and where it first stands
    float top = neg_inf();
    row.template each<true>([&](int, const float (&x)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) top = fmaxf(top, x[e]);
    });
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) s.wave[wave] = key_of(top);
    if (threadIdx.x == 0) s.index = 0x7fffffff;
    __syncthreads();
    unsigned best = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) best = best > (unsigned)s.wave[w] ? best : (unsigned)s.wave[w];
    top = __builtin_bit_cast(float, best & 0x80000000u ? best ^ 0x80000000u : ~best);
    __syncthreads();
    if (!(T0 > 0.f) || top == neg_inf()) {
        int at = 0x7fffffff;
        row.each([&](int j, const float (&x)[E]) {
#pragma unroll
            for (int e = E - 1; e >= 0; --e)
                if (x[e] == top) {
                    const int i = row.index(j, e);
                    at = i < at ? i : at;
                }
        });
        if (at != 0x7fffffff) atomicMin(&s.index, at);
        __syncthreads();
        if (threadIdx.x == 0) {
            const bool none = top == neg_inf();
            a.token[r] = none ? -1 : s.index;
            if (a.logprob) a.logprob[r] = none ? __builtin_nanf("") : 0.f;
        }
        return;
    }
    const Weight w{64 * 1.4426950408889634074 / (double)T0, (double)top, top, s.table};
    const float per_bin = fminf(64.f / T0, 1e30f);

    // the border: logits above `key` are kept, of those at it the first `keep`
    unsigned key = 0;
    u64 keep = ~(u64)0, spare = 0;  // spare: weight at the border that top-k has dropped
    if (top_k > 0 && top_k < a.V) {
        Border b;
        if (find_border<false>(s, row, w, per_bin, 0u, (u64)top_k, b)) {
            key = b.key;
            keep = top_k - b.before;
            const unsigned bits = key & 0x80000000u ? key ^ 0x80000000u : ~key;
            spare = (b.in - keep) * w.fixed(__builtin_bit_cast(float, bits));
        }
    }
    if (top_p < 1.f) {
        u64 sum = 0, total;
        row.each([&](int, const float (&x)[E]) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool in = key_of(x[e]) >= key;
                if (__ballot(in)) sum += in ? w.fixed(x[e]) : 0;
            }
        });
        block_exclusive(sum, s.wave, &total);
        bool whole;
        u64 target = part_of(top_p, total - spare, &whole);
        if (!whole || target == 0) ++target;
        Border b;
        if (find_border<true>(s, row, w, per_bin, key, target, b)) {
            key = b.key;
            const unsigned bits = key & 0x80000000u ? key ^ 0x80000000u : ~key;
            const u64 each = w.fixed(__builtin_bit_cast(float, bits));
            keep = (target - b.before + each - 1) / each;
        }
    }

    // weights of what is kept, by tiles: step j of a wave
    const double least = (double)min_p * (double)((u64)1 << kOne);
    const unsigned bits = key & 0x80000000u ? key ^ 0x80000000u : ~key;
    const float at_border = __builtin_bit_cast(float, bits);
    auto weigh = [&](float x) {
        const double d = w.scaled(x);
        return d >= least ? Weight::round(d) : 0;
    };
    const u64 border = keep == ~(u64)0 ? 0 : weigh(at_border);
    row.each([&](int j, const float (&x)[E]) {
        u64 sum = 0;
        int ties = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const unsigned k = key_of(x[e]);
            if (__ballot(k >= key)) {
                const bool tie = k == key && keep != ~(u64)0;
                ties += tie;
                const u64 v = weigh(x[e]);
                sum += k >= key && !tie ? v : 0;
            }
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
    const int tiles = row.steps * kWaves, t = threadIdx.x;
    const int n = t < tiles ? s.ties[t] : 0;
    u64 all_ties;
    const u64 ties_before = block_exclusive((u64)n, s.wave, &all_ties);
    const u64 room = keep > ties_before ? keep - ties_before : 0;
    const u64 mine = (t < tiles ? s.sum[t] : 0) + border * (room < (u64)n ? room : (u64)n);
    u64 total;
    const u64 before = block_exclusive(mine, s.wave, &total);
    bool whole;
    const u64 at = part_of(u, total, &whole);
    if (before <= at && at < before + mine) {
        s.bin = t;
        s.picked[0] = at - before;
        s.picked[1] = ties_before;
    }
    __syncthreads();
    const int tile = (int)s.bin;
    if (wave != tile % kWaves) return;
    // in that tile: the first value whose running weight exceeds `left`
    const u64 left = s.picked[0];
    u64 used = s.picked[1];
    row.each([&](int j, const float (&x)[E]) {
        if (j != tile / kWaves) return;
        int ties = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) ties += key_of(x[e]) == key && keep != ~(u64)0;
        used += wave_inclusive(ties) - ties;
        u64 v[E], sum = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const unsigned k = key_of(x[e]);
            const bool tie = k == key && keep != ~(u64)0;
            v[e] = k > key || (k == key && (!tie || used < keep)) ? weigh(x[e]) : 0;
            used += tie;
            sum += v[e];
        }
        u64 run = wave_inclusive(sum) - sum;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (run <= left && left < run + v[e]) {
                a.token[r] = row.index(j, e);
                if (a.logprob) a.logprob[r] = (float)log((double)v[e] / (double)total);
            }
            run += v[e];
        }
    });
}

template <typename T>
hipError_t launch(const SampleArgs& a, hipStream_t s) {
    const dim3 gr((unsigned)a.rows), bl(kThreads);
    const int unit = 16 / (int)sizeof(T), units = (a.V + unit - 1 + kThreads * unit - 1) / (kThreads * unit);
    if (units <= 1) sample_kernel<T, 1><<<gr, bl, 0, s>>>(a);
    else if (units <= 4) sample_kernel<T, 4><<<gr, bl, 0, s>>>(a);
    else if (units <= 8) sample_kernel<T, 8><<<gr, bl, 0, s>>>(a);
    else sample_kernel<T, 0><<<gr, bl, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
    return a.f32 ? launch<float>(a, s) : launch<__bf16>(a, s);
}

}  // namespace e2ttt
