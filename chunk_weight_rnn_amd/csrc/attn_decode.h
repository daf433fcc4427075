// Work of the decoding kernels (attn_decode.hip, attn8_decode.hip): the line of
// units, what a workgroup takes of it, and the end of an item.
#pragma once

#include "attn_common.h"

namespace e2ttt {
namespace attn {
namespace {

static __device__ const int no_page = -1;

constexpr int BM = 32;     // rows of an item
constexpr int BW = 32;     // keys of a unit per wave
constexpr int UNIT = 128;  // keys of a unit
constexpr float kLazy = 8.f;  // as in attn_fwd.hip

struct Work {
    int seq, tok0, n, kept;  // sequence
    int kvh, rt, tiles;      // key head, row tile, row tiles of the sequence
    int lo, nb;              // first key and units of the sequence
    int block;               // unit asked for
    int before;              // units of the line before this item
};

// Per sequence: new tokens, tokens kept, first visible key, row tiles, units.
struct Seq {
    int tok0, n, kept, lo, tiles, nb;
};
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int s) {
    Seq q{};
    if (s < a.S) {
        q.tok0 = clamped(a.cu[s], (int)a.N);
        const int n = clamped(a.cu[s + 1], (int)a.N) - q.tok0;
        q.n = n > 0 ? n : 0;
        q.kept = kept_tokens(a.pg, s, q.n);
        q.lo = a.window > 0 && q.kept - a.window + 1 > 0 ? (q.kept - a.window + 1) & ~(BW - 1) : 0;
        q.tiles = (q.n * a.G + BM - 1) / BM;
        q.nb = (q.kept + q.n - q.lo + UNIT - 1) / UNIT;
    }
    return q;
}

// All units of the call; q0: the first 64 sequences, a lane each.
__device__ __forceinline__ int total_units(const AttnArgs& a, const Seq& q0, int lane) {
    int t = 0;
    for (int s0 = 0; s0 < a.S; s0 += 64) {
        const Seq q = s0 == 0 ? q0 : seq_of(a, s0 + lane);
        t += q.tiles * q.nb * a.K;
    }
    return last_lane(wave_scan<false>(t));
}

// The item that holds unit t of the line (UNITS), or the t-th item.
template <bool UNITS>
__device__ __forceinline__ bool find_work(const AttnArgs& a, const Seq& q0, int t, int lane, Work& w) {
    int base = 0, units = 0;  // of the sequences before this step
    for (int s0 = 0; s0 < a.S; s0 += 64) {
        const Seq q = s0 == 0 ? q0 : seq_of(a, s0 + lane);
        const int mu = q.tiles * q.nb * a.K, m = UNITS ? mu : q.tiles * a.K;
        const int iu = wave_scan<false>(mu), incl = UNITS ? iu : wave_scan<false>(m);
        const unsigned long long past = __ballot(base + incl > t);
        if (past) {
            const int l = __builtin_ctzll(past);
            auto get = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
            w.seq = s0 + l;
            w.tok0 = get(q.tok0);
            w.n = get(q.n);
            w.kept = get(q.kept);
            w.lo = get(q.lo);
            w.nb = get(q.nb);
            w.tiles = get(q.tiles);
            const int first = base + get(incl - m);  // of this sequence
            const int local = t - first;
            const int item = UNITS ? local / w.nb : local;
            w.block = UNITS ? local - item * w.nb : 0;
            w.before = units + get(iu - mu) + item * w.nb;
            w.kvh = item / w.tiles;
            w.rt = item - w.kvh * w.tiles;
            return true;
        }
        base += last_lane(incl);
        units += last_lane(iu);
    }
    return false;
}

// Units per workgroup: equal shares.
__device__ __forceinline__ int share(int total, int groups) { return total > 0 ? (total + groups - 1) / groups : 1; }

// Row stride of the area in which the four waves' outputs meet, and its size.
template <int DP>
constexpr int kMergeRow = DP + 4;
template <int DP>
constexpr int kMergeFloats = 4 * BM * kMergeRow<DP>;

// The four waves' sums of an item (or of a workgroup's stretch of it) together,
// into the output or, where others have a part, the partial results' slot.
template <int DP, bool SPLIT>
__device__ __forceinline__ void finish_item(const AttnArgs& a, const Work& w, const f32x16 (&acc)[DP / 32], float m, float l,
                                            bool live, bool whole, int slot, float* area, float (&stat)[4][2][BM]) {
    constexpr int DT = DP / 32, OLD = kMergeRow<DP>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31, G = a.G;
    const int rows = w.n * G, r0 = w.rt * BM;
    if (g == 0) {
        stat[wave][0][col] = m;
        stat[wave][1][col] = l;
    }
    __syncthreads();  // also: every stage has been read
    float mm = neg_inf();
#pragma unroll
    for (int v = 0; v < 4; ++v) mm = fmaxf(mm, stat[v][0][col]);
    const float mu = mm == neg_inf() ? 0.f : mm;
    const float f = __builtin_amdgcn_exp2f(m - mu);
    if (live) {
        float* o = area + (wave * BM + col) * OLD + 4 * g;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = acc[dt][4 * j + e] * f;
                *(f32x4*)(o + 32 * dt + 8 * j) = x;
            }
    }
    __syncthreads();
    const int count = rows - r0 < BM ? rows - r0 : BM;
    for (int x = threadIdx.x; x < count * (DP / 4); x += 256) {
        const int r = x / (DP / 4), d = x % (DP / 4) * 4;
        if (d >= a.D) continue;
        float mt = neg_inf(), lt = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) mt = fmaxf(mt, stat[v][0][r]);
        const float mr = mt == neg_inf() ? 0.f : mt;
        f32x4 s = {};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            lt += stat[v][1][r] * __builtin_amdgcn_exp2f(stat[v][0][r] - mr);
            s += *(const f32x4*)(area + (v * BM + r) * OLD + d);
        }
        const float inv = lt > 0.f ? 1.f / lt : lt;  // a row that sees nothing gives 0; NaN stays
        s *= inv;
        const int rr = r0 + r, tk = div_group(rr, G, a.gmagic), hd = w.kvh * G + rr - tk * G;
        if (!SPLIT || whole) {
            bf16x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = (__bf16)s[e];
            *(bf16x4*)((__bf16*)a.out + ((int64_t)(w.tok0 + tk) * a.H + hd) * a.D + d) = o;
        } else {
            *(f32x4*)(a.po + ((int64_t)slot * BM + r) * a.D + d) = s;
            if (d == 0) a.pl[(int64_t)slot * BM + r] = lt > 0.f ? mt + __builtin_amdgcn_logf(lt) : (lt == 0.f ? neg_inf() : lt);
        }
    }
}

}  // namespace
}  // namespace attn
}  // namespace e2ttt
