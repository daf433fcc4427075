// Causal grouped-head attention in fp32 on the fp32 MFMA: forward over packed
// sequences and over a paged cache, and the gradients.  The same one-pass
// softmax, row packing and operand orientation as the bf16 kernels
// (attn_common.h, attn_fwd.hip, attn_bwd.hip), on 16x16x4 tiles: a 16x16
// accumulator holds rows 4 (lane / 16) + i, i = 0..3, of column lane % 16, and
// element i is the operand of k-step i of the next product as it stands, with
// the k index of lane group u at step i meaning row 4 u + i.
//
// The fp32 MFMA issues at a sixteenth of the bf16 rate, so the products bound
// these kernels and tiles are simply staged through registers.  What is scarce
// in fp32's small layers is workgroups: four heads over two rows of 2K leave
// half the chip idle in tiles of 64 rows or keys.  So the four waves of a
// workgroup share few rows or keys (16) and split the other axis, and add their
// parts in the LDS at the end.
#include "attn_common.h"

namespace e2ttt {
namespace attn {
namespace {

constexpr int BM = 16;   // rows of a workgroup (forward, dq): 4 waves, 16 keys of a tile each
constexpr int BN = 64;   // keys of a staged tile
constexpr int BK = 16;   // keys of a workgroup (dkdv): 8 waves, 16 rows of a tile each
constexpr int BR = 128;  // rows of a staged tile (dkdv)

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Sum or maximum over the four lane groups that hold one column.
__device__ __forceinline__ float groups_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}
__device__ __forceinline__ float groups_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}

// A staged tile: rows of DP values, padded by four so that the 16 rows of a
// fragment start on different banks.
template <int DP, int ROWS, int THREADS>
struct Tile {
    static constexpr int LD = DP + 4;
    static constexpr int U = ROWS * DP / 4 / THREADS;  // 16-byte units per thread
    float v[ROWS * LD];
};

// Buffers of a tile: with two, one barrier per tile is enough.  At a head
// dimension of 128 two would leave room for only one workgroup per compute unit.
template <int DP>
constexpr int kBuffers = DP == 64 ? 2 : 1;

// The fragments of rows 4 u + 0..3 (from `tile` on) by columns, all of them at
// once: operand of k-step i and column tile dt.
template <int DP>
struct ColFrags {
    float v[4][DP / 16];
    __device__ __forceinline__ void load(const float* tile, int u, int col) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int dt = 0; dt < DP / 16; ++dt) v[i][dt] = tile[(4 * u + i) * (DP + 4) + 16 * dt + col];
    }
};

// Row fragment of k-steps 4 s .. 4 s + 3: columns 16 s + 4 u + 0..3.
template <int DP>
__device__ __forceinline__ f32x4 row4(const float* tile, int row, int s, int u) {
    return *(const f32x4*)(tile + row * (DP + 4) + 16 * s + 4 * u);
}

// A row's fragments straight from memory (zeros outside the head dimension).
template <int DP>
__device__ __forceinline__ void load_row(f32x4 (&f)[DP / 16], const float* p, bool live, int u, int D) {
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int d = 16 * s + 4 * u;
        f32x4 z = {};
        f[s] = live && d < D ? *(const f32x4*)(p + d) : z;
    }
}

// <row, f> for this lane's column, and acc += w row where w is not zero: the
// terms of sums that are not finite (attn_common.h).
template <int S4>
__device__ __forceinline__ float dot_row4(const float* row, const f32x4 (&f)[S4], int u, int D) {
    float t = 0.f;
#pragma unroll
    for (int s = 0; s < S4; ++s) {
        const int d = 16 * s + 4 * u;
        if (d >= D) continue;
        const f32x4 x = *(const f32x4*)(row + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) t = __builtin_fmaf(x[e], f[s][e], t);
        __builtin_amdgcn_sched_barrier(0);  // a rare path: few registers rather than overlap
    }
    return groups_sum(t);
}
template <int S4>
__device__ __forceinline__ void add_row4(f32x4 (&acc)[S4], const float* row, float w, int u, int D) {
#pragma unroll
    for (int dt = 0; dt < S4; ++dt) {
        const int d = 16 * dt + 4 * u;
        if (w == 0.f || d >= D) continue;
        const f32x4 x = *(const f32x4*)(row + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[dt][e] = __builtin_fmaf(w, x[e], acc[dt][e]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int DP, int DT>
__device__ __forceinline__ void store_cols(float* o, const f32x4 (&acc)[DT], float f, int u, int D) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
        const int d = 16 * dt + 4 * u;
        if (d < D) *(f32x4*)(o + d) = acc[dt] * f;
    }
}

template <int DP, bool PAGED>
__global__ __launch_bounds__(256, 2) void attn_f32_fwd_kernel(AttnArgs a) {
    using TL = Tile<DP, BN, 256>;
    constexpr int S4 = DP / 16;
    constexpr int NB = kBuffers<DP>;
    __shared__ TL kts[NB], vts[NB];
    __shared__ float stat[2][4][BM];
    int b = blockIdx.x;
    if constexpr (PAGED) {
        const int tiles = a.ntiles * a.nsplit * a.K;
        if (b >= tiles) {
            append_block<float>(a, b - tiles);
            return;
        }
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = lane >> 4, col = lane & 15, G = a.G;
    const int kvh = b % a.K;
    b /= a.K;
    const int split = b % a.nsplit, t = b / a.nsplit;
    Item it;
    if (!find_item(a.cu, a.S, (int)a.N, t, row_cap(a.window, G, BM), [&](int n) { return (n * G + BM - 1) / BM; }, it)) return;
    const int r0 = it.tile * BM;
    const int rows = it.n * G;
    int kept = 0;
    if constexpr (PAGED) kept = kept_tokens(a.pg, it.seq, it.n);
    const int first = kept + div_group(r0, G, a.gmagic);
    const int last = kept + div_group(r0 + BM < rows ? r0 + BM - 1 : rows - 1, G, a.gmagic);
    const int begin = a.window > 0 && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
    const int lo = begin & ~(BN - 1);
    const int nb = (last - lo) / BN + 1;
    const int per = (nb + a.nsplit - 1) / a.nsplit;
    const int j0 = split * per, j1 = j0 + per < nb ? j0 + per : nb;

    const int row = r0 + col;
    const bool live = row < rows;
    const int tok = live ? div_group(row, G, a.gmagic) : 0, hg = live ? row - tok * G : 0;
    const int qpos = live ? kept + tok : -1;
    const int qlow = a.window > 0 ? qpos - a.window : -1;
    const int64_t qtok = it.tok0 + tok;
    const int head = kvh * G + hg;

    f32x4 qf[S4];
    load_row<DP>(qf, (const float*)a.q + qtok * a.q_tok + (int64_t)head * a.q_head, live, u, a.D);

    const float* ksrc = (const float*)a.k + it.tok0 * a.k_tok + kvh * a.k_head;
    const float* vsrc = (const float*)a.v + it.tok0 * a.v_tok + kvh * a.v_head;
    const int fresh = PAGED ? (a.pg.append ? kept : 0x7fffffff) : 0;
    // key and value of a position; null where it is read as zeros
    auto rows_of = [&](int pos, const float*& kp, const float*& vp) {
        kp = vp = nullptr;
        if (pos < begin || pos > last) return;
        if (!PAGED || pos >= fresh) {
            kp = ksrc + (int64_t)(pos - fresh) * a.k_tok;
            vp = vsrc + (int64_t)(pos - fresh) * a.v_tok;
            return;
        }
        const int pi = pos >> a.pg.shift;
        const int page = pi < a.pg.wide ? a.pg.table[(int64_t)it.seq * a.pg.wide + pi] : -1;
        if ((unsigned)page >= (unsigned)a.pg.pages) return;
        const int64_t slot = pos & ((1 << a.pg.shift) - 1);
        kp = (const float*)a.pg.kc + page * a.pg.k_page + kvh * a.pg.k_head + slot * a.pg.k_slot;
        vp = (const float*)a.pg.vc + page * a.pg.v_page + kvh * a.pg.v_head + slot * a.pg.v_slot;
    };
    f32x4 kr[TL::U], vr[TL::U];
    auto load_tile = [&](int j) {
#pragma unroll
        for (int i = 0; i < TL::U; ++i) {
            const int x = i * 256 + threadIdx.x;
            const int c = x % (DP / 4) * 4;
            const float *kp, *vp;
            rows_of(lo + j * BN + x / (DP / 4), kp, vp);
            f32x4 z = {};
            kr[i] = kp && c < a.D ? *(const f32x4*)(kp + c) : z;
            vr[i] = vp && c < a.D ? *(const f32x4*)(vp + c) : z;
        }
    };

    f32x4 acc[S4] = {};
    float m = neg_inf(), l = 0.f;
    if (j0 < j1) load_tile(j0);
    for (int j = j0; j < j1; ++j) {
        TL &kt = kts[NB == 2 ? j & 1 : 0], &vt = vts[NB == 2 ? j & 1 : 0];
        if (NB == 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < TL::U; ++i) {
            const int x = i * 256 + threadIdx.x;
            const int o = x / (DP / 4) * TL::LD + x % (DP / 4) * 4;
            *(f32x4*)(kt.v + o) = kr[i];
            *(f32x4*)(vt.v + o) = vr[i];
        }
        __syncthreads();
        if (j + 1 < j1) load_tile(j + 1);
        const int w0 = 16 * wave, p0 = lo + j * BN + w0;
        ColFrags<DP> vf;
        vf.load(vt.v + w0 * TL::LD, u, col);
        f32x4 sc = {}, so = {};  // two chains, so that no product waits for the one before it
#pragma unroll
        for (int s = 0; s < S4; ++s) {
            const f32x4 kf = row4<DP>(kt.v, w0 + col, s, u);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                sc = mfma4(kf[e], qf[s][e], sc);
                so = mfma4(kf[e + 1], qf[s][e + 1], so);
            }
        }
        sc += so;
        float mx = neg_inf();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * u + i;
            if (p > qpos || p <= qlow) sc[i] = neg_inf();
            mx = fmaxf(mx, sc[i]);
        }
        mx = groups_max(mx) * a.sl2;
        const float mn = fmaxf(m, mx);
        const float mu = mn == neg_inf() ? 0.f : mn;
        const float f = __builtin_amdgcn_exp2f(m - mu);
        m = mn;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < S4; ++dt) acc[dt] *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sc[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], a.sl2, -mu));
            l += sc[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) acc[dt] = mfma4(vf.v[i][dt], sc[i], acc[dt]);
    }
    l = groups_sum(l);
    // keys of this wave, position by position, where its sums are not finite
    auto wave_keys = [&](int first_tile, int tiles, auto&& f) {
#pragma unroll 1
        for (int i = first_tile * 16; i < tiles * 16; ++i) f(lo + i / 16 * BN + 16 * wave + i % 16);
    };
    if (j0 < j1 && first != last) {
        const float bad = not_finite(acc);
        if (__any(bad != bad && l == l)) {
            const float mu = m == neg_inf() ? 0.f : m;
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) acc[dt] = f32x4{};
            wave_keys(j0, j1, [&](int p) {
                const float *kp, *vp;
                rows_of(p, kp, vp);
                if (!kp) return;
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_row4(kp, qf, u, a.D), a.sl2, -mu));
                add_row4(acc, vp, p > qpos || p <= qlow ? 0.f : x, u, a.D);
            });
        }
    }
    // the four waves together
    __syncthreads();
    float* area = kts[0].v + (16 * wave + col) * TL::LD + 4 * u;
    if (u == 0) {
        stat[0][wave][col] = m;
        stat[1][wave][col] = l;
    }
#pragma unroll
    for (int dt = 0; dt < S4; ++dt) *(f32x4*)(area + 16 * dt) = acc[dt];
    __syncthreads();
    if (wave > 0 || !live) return;
    {
        float mw[4], mn = neg_inf();
#pragma unroll
        for (int w = 0; w < 4; ++w) mn = fmaxf(mn, mw[w] = stat[0][w][col]);
        const float mu = mn == neg_inf() ? 0.f : mn;
        l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = __builtin_amdgcn_exp2f(mw[w] - mu);
            l += stat[1][w][col] * f;
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) {
                const f32x4 x = *(const f32x4*)(area + 16 * w * TL::LD + 16 * dt) * f;
                acc[dt] = w == 0 ? x : acc[dt] + x;
            }
        }
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : l;  // a row that sees nothing gives 0; NaN stays
    const float lse2 = l > 0.f ? m + __builtin_amdgcn_logf(l) : (l == 0.f ? neg_inf() : l);
    if (a.nsplit > 1) {
        const int64_t at = ((int64_t)split * a.N + qtok) * a.H + head;
        if (u == 0) a.pl[at] = lse2;
        if (j0 < j1) store_cols<DP, S4>(a.po + at * a.D, acc, inv, u, a.D);
        return;
    }
    if (a.lse && u == 0) a.lse[qtok * a.H + head] = lse2 * kLn2;
    store_cols<DP, S4>((float*)a.out + (qtok * a.H + head) * a.D, acc, inv, u, a.D);
}

template <int DP>
__global__ __launch_bounds__(256, 2) void attn_f32_dq_kernel(AttnBwdArgs a) {
    using TL = Tile<DP, BN, 256>;
    constexpr int S4 = DP / 16;
    constexpr int NB = kBuffers<DP>;
    __shared__ TL kts[NB], vts[NB];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = lane >> 4, col = lane & 15, G = a.G;
    const int kvh = blockIdx.x % a.K, t = blockIdx.x / a.K;
    Item it;
    if (!find_item(a.cu, a.S, (int)a.N, t, row_cap(a.window, G, BM), [&](int n) { return (n * G + BM - 1) / BM; }, it)) return;
    const int r0 = it.tile * BM;
    const int rows = it.n * G;
    const int first = div_group(r0, G, a.gmagic);
    const int last = div_group(r0 + BM < rows ? r0 + BM - 1 : rows - 1, G, a.gmagic);
    const int begin = a.window > 0 && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
    const int lo = begin & ~(BN - 1);
    const int nb = (last - lo) / BN + 1;
    const int row = r0 + col;
    const bool live = row < rows;
    const int tok = live ? div_group(row, G, a.gmagic) : 0, hg = live ? row - tok * G : 0;
    const int qpos = live ? tok : -1;
    const int qlow = a.window > 0 ? qpos - a.window : -1;
    const int64_t qtok = it.tok0 + tok;
    const int head = kvh * G + hg;
    const int64_t at = qtok * a.H + head;

    f32x4 qf[S4], df[S4], of[S4];
    load_row<DP>(qf, (const float*)a.q + qtok * a.q_tok + (int64_t)head * a.q_head, live, u, a.D);
    load_row<DP>(df, (const float*)a.dout + at * a.D, live, u, a.D);
    load_row<DP>(of, (const float*)a.out + at * a.D, live, u, a.D);
    float delta = 0.f;
#pragma unroll
    for (int s = 0; s < S4; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) delta = __builtin_fmaf(df[s][e], of[s][e], delta);
    delta = groups_sum(delta);
    if (live && u == 0 && wave == 0) a.stats[at] = delta;
    const float lse2 = live ? a.lse[at] * kLog2e : 0.f;

    const float* ksrc = (const float*)a.k + it.tok0 * a.k_tok + kvh * a.k_head;
    const float* vsrc = (const float*)a.v + it.tok0 * a.v_tok + kvh * a.v_head;
    f32x4 kr[TL::U], vr[TL::U];
    auto load_tile = [&](int j) {
#pragma unroll
        for (int i = 0; i < TL::U; ++i) {
            const int x = i * 256 + threadIdx.x;
            const int pos = lo + j * BN + x / (DP / 4), c = x % (DP / 4) * 4;
            f32x4 z = {};
            const bool in = pos >= begin && pos <= last && c < a.D;
            kr[i] = in ? *(const f32x4*)(ksrc + pos * a.k_tok + c) : z;
            vr[i] = in ? *(const f32x4*)(vsrc + pos * a.v_tok + c) : z;
        }
    };
    f32x4 acc[S4] = {};
    load_tile(0);
    for (int j = 0; j < nb; ++j) {
        TL &kt = kts[NB == 2 ? j & 1 : 0], &vt = vts[NB == 2 ? j & 1 : 0];
        if (NB == 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < TL::U; ++i) {
            const int x = i * 256 + threadIdx.x;
            const int o = x / (DP / 4) * TL::LD + x % (DP / 4) * 4;
            *(f32x4*)(kt.v + o) = kr[i];
            *(f32x4*)(vt.v + o) = vr[i];
        }
        __syncthreads();
        if (j + 1 < nb) load_tile(j + 1);
        const int w0 = 16 * wave, p0 = lo + j * BN + w0;
        ColFrags<DP> kc;
        kc.load(kt.v + w0 * TL::LD, u, col);
        f32x4 sc = {}, dp = {};
#pragma unroll
        for (int s = 0; s < S4; ++s) {
            const f32x4 kf = row4<DP>(kt.v, w0 + col, s, u), vf = row4<DP>(vt.v, w0 + col, s, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc = mfma4(kf[e], qf[s][e], sc);
                dp = mfma4(vf[e], df[s][e], dp);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * u + i;
            const float ds = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], a.sl2, -lse2)) * (dp[i] - delta);
            sc[i] = p > qpos || p <= qlow ? 0.f : ds;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) acc[dt] = mfma4(kc.v[i][dt], sc[i], acc[dt]);
    }
    if (first != last) {  // sums that are not finite, as in the forward
        const float bad = not_finite(acc);
        if (__any(bad != bad && lse2 == lse2 && delta == delta)) {
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) acc[dt] = f32x4{};
#pragma unroll 1
            for (int i = 0; i < nb * 16; ++i) {
                const int p = lo + i / 16 * BN + 16 * wave + i % 16;
                if (p < begin || p > last) continue;
                const float* kp = ksrc + p * a.k_tok;
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_row4(kp, qf, u, a.D), a.sl2, -lse2));
                const float y = x * (dot_row4(vsrc + p * a.v_tok, df, u, a.D) - delta);
                add_row4(acc, kp, p > qpos || p <= qlow ? 0.f : y, u, a.D);
            }
        }
    }
    __syncthreads();
    float* area = kts[0].v + (16 * wave + col) * TL::LD + 4 * u;
#pragma unroll
    for (int dt = 0; dt < S4; ++dt) *(f32x4*)(area + 16 * dt) = acc[dt];
    __syncthreads();
    if (wave > 0 || !live) return;
#pragma unroll
    for (int w = 1; w < 4; ++w)
#pragma unroll
        for (int dt = 0; dt < S4; ++dt) acc[dt] += *(const f32x4*)(area + 16 * w * TL::LD + 16 * dt);
    store_cols<DP, S4>((float*)a.dq + at * a.D, acc, a.scale, u, a.D);
}

template <int DP>
__global__ __launch_bounds__(512, 2) void attn_f32_dkdv_kernel(AttnBwdArgs a) {
    using TL = Tile<DP, BR, 512>;
    constexpr int S4 = DP / 16;
    constexpr int NB = kBuffers<DP>;
    __shared__ TL qts[NB], dts[NB];
    __shared__ __attribute__((aligned(16))) float stats[NB][2][BR];  // lse (base 2), delta
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = lane >> 4, col = lane & 15, G = a.G;
    const int kvh = blockIdx.x % a.K, t = blockIdx.x / a.K;
    Item it;
    if (!find_item(a.cu, a.S, (int)a.N, t, row_cap(a.window, 1, BK), [&](int n) { return (n + BK - 1) / BK; }, it)) return;
    const int k0 = (it.tiles - 1 - it.tile) * BK;  // the first keys of a sequence have the most rows
    const int rows = it.n * G;
    const int klast = k0 + BK < it.n ? k0 + BK - 1 : it.n - 1;
    const int rbeg = k0 * G & ~(BR - 1);
    const int64_t re = a.window > 0 ? ((int64_t)klast + a.window) * G : rows;
    const int rend = re < rows ? (int)re : rows;
    const int nb = (rend - rbeg + BR - 1) / BR;
    const int key = k0 + col;
    const bool live = key < it.n;
    const int64_t ktok = it.tok0 + (live ? key : 0);
    const int rlo = live ? key * G : 0x7fffffff;
    const int64_t rh = a.window > 0 ? ((int64_t)key + a.window) * G : rows;
    const int rhi = rh < rows ? (int)rh : rows;

    f32x4 kf[S4], vf[S4];
    load_row<DP>(kf, (const float*)a.k + ktok * a.k_tok + (int64_t)kvh * a.k_head, live, u, a.D);
    load_row<DP>(vf, (const float*)a.v + ktok * a.v_tok + (int64_t)kvh * a.v_head, live, u, a.D);

    const float* qsrc = (const float*)a.q + it.tok0 * a.q_tok + (int64_t)kvh * G * a.q_head;
    const int64_t first_row = (int64_t)it.tok0 * a.H + kvh * G;
    const float* dsrc = (const float*)a.dout + first_row * a.D;
    f32x4 qr[TL::U], dr[TL::U];
    float st = 0.f;
    auto load_tile = [&](int j) {
#pragma unroll
        for (int i = 0; i < TL::U; ++i) {
            const int x = i * 512 + threadIdx.x;
            const int r = rbeg + (nb - 1 - j) * BR + x / (DP / 4), c = x % (DP / 4) * 4;
            f32x4 z = {};
            qr[i] = dr[i] = z;
            if (r < rend && c < a.D) {
                const int tk = div_group(r, G, a.gmagic), hg = r - tk * G;
                qr[i] = *(const f32x4*)(qsrc + tk * a.q_tok + hg * a.q_head + c);
                dr[i] = *(const f32x4*)(dsrc + ((int64_t)tk * a.H + hg) * a.D + c);
            }
        }
        if (threadIdx.x < 2 * BR) {
            const int r = rbeg + (nb - 1 - j) * BR + (threadIdx.x & (BR - 1));
            st = 0.f;
            if (r < rend) {
                const int tk = div_group(r, G, a.gmagic), hg = r - tk * G;
                const int64_t at = first_row + (int64_t)tk * a.H + hg;
                st = threadIdx.x < BR ? a.lse[at] * kLog2e : a.stats[at];
            }
        }
    };
    f32x4 dk[S4] = {}, dv[S4] = {};
    if (nb > 0) load_tile(0);  // from the last rows back, as in attn_bwd.hip
    for (int j = 0; j < nb; ++j) {
        TL &qt = qts[NB == 2 ? j & 1 : 0], &dt_ = dts[NB == 2 ? j & 1 : 0];
        float(&stat)[2][BR] = stats[NB == 2 ? j & 1 : 0];
        if (NB == 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < TL::U; ++i) {
            const int x = i * 512 + threadIdx.x;
            const int o = x / (DP / 4) * TL::LD + x % (DP / 4) * 4;
            *(f32x4*)(qt.v + o) = qr[i];
            *(f32x4*)(dt_.v + o) = dr[i];
        }
        if (threadIdx.x < 2 * BR) (&stat[0][0])[threadIdx.x] = st;
        __syncthreads();
        if (j + 1 < nb) load_tile(j + 1);
        const int w0 = 16 * wave, p0 = rbeg + (nb - 1 - j) * BR + w0;
        ColFrags<DP> qc, dc;
        qc.load(qt.v + w0 * TL::LD, u, col);
        dc.load(dt_.v + w0 * TL::LD, u, col);
        f32x4 sc = {}, dp = {};
#pragma unroll
        for (int s = 0; s < S4; ++s) {
            const f32x4 qf = row4<DP>(qt.v, w0 + col, s, u), df = row4<DP>(dt_.v, w0 + col, s, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc = mfma4(qf[e], kf[s][e], sc);
                dp = mfma4(df[e], vf[s][e], dp);
            }
        }
        const f32x4 ls = *(const f32x4*)&stat[0][w0 + 4 * u], de = *(const f32x4*)&stat[1][w0 + 4 * u];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = p0 + 4 * u + i;
            const bool out = r < rlo || r >= rhi;
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], a.sl2, -ls[i]));
            sc[i] = out ? 0.f : p;
            dp[i] = out ? 0.f : p * (dp[i] - de[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) {
                dv[dt] = mfma4(dc.v[i][dt], sc[i], dv[dt]);
                dk[dt] = mfma4(qc.v[i][dt], dp[i], dk[dt]);
            }
    }
    const float bad = not_finite(dk) + not_finite(dv);
    if (__any(bad != bad)) {  // as in the forward
#pragma unroll
        for (int dt = 0; dt < S4; ++dt) dk[dt] = dv[dt] = f32x4{};
#pragma unroll 1
        for (int i = 0; i < nb * 16; ++i) {
            const int r = rbeg + i / 16 * BR + 16 * wave + i % 16;
            if (r >= rend) continue;
            const int tk = div_group(r, G, a.gmagic), hg = r - tk * G;
            const int64_t at = first_row + (int64_t)tk * a.H + hg;
            const float *qp = qsrc + tk * a.q_tok + hg * a.q_head, *op = (const float*)a.dout + at * a.D;
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_row4(qp, kf, u, a.D), a.sl2, -a.lse[at] * kLog2e));
            const float y = x * (dot_row4(op, vf, u, a.D) - a.stats[at]);
            const bool out = r < rlo || r >= rhi;
            add_row4(dv, op, out ? 0.f : x, u, a.D);
            add_row4(dk, qp, out ? 0.f : y, u, a.D);
        }
    }
    // the eight parts of the rows together, in order
    __syncthreads();
    const int o = (16 * wave + col) * TL::LD + 4 * u;
#pragma unroll
    for (int dt = 0; dt < S4; ++dt) {
        *(f32x4*)(qts[0].v + o + 16 * dt) = dk[dt];
        *(f32x4*)(dts[0].v + o + 16 * dt) = dv[dt];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * BK * (DP / 4); x += 512) {
        const int which = x / (BK * (DP / 4)), kk = x / (DP / 4) % BK, d = x % (DP / 4) * 4;
        if (k0 + kk >= it.n || d >= a.D) continue;
        const float* src = (which ? dts[0].v : qts[0].v) + kk * TL::LD + d;
        f32x4 y = *(const f32x4*)src;
#pragma unroll
        for (int w = 1; w < 8; ++w) y += *(const f32x4*)(src + 16 * w * TL::LD);
        float* dst = (which ? (float*)a.dv : (float*)a.dk) + (((int64_t)it.tok0 + k0 + kk) * a.K + kvh) * a.D + d;
        *(f32x4*)dst = which ? y : y * a.scale;
    }
}

template <int DP>
hipError_t launch_fwd(const AttnArgs& a, hipStream_t s) {
    const bool paged = a.pg.kc != nullptr;
    const int64_t grid = (int64_t)a.ntiles * a.K * a.nsplit + (paged ? append_blocks(a, 4) : 0);
    if (grid == 0) return hipSuccess;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if (paged)
        attn_f32_fwd_kernel<DP, true><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a);
    else
        attn_f32_fwd_kernel<DP, false><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <int DP>
hipError_t launch_bwd(const AttnBwdArgs& a, hipStream_t s) {
    const int64_t dq_grid = (a.N * a.G / BM + a.S) * a.K, dkv_grid = (a.N / BK + a.S) * a.K;
    if (dq_grid > 0x7fffffff || dkv_grid > 0x7fffffff) return hipErrorInvalidValue;
    attn_f32_dq_kernel<DP><<<dim3((unsigned)dq_grid), dim3(256), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attn_f32_dkdv_kernel<DP><<<dim3((unsigned)dkv_grid), dim3(512), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_fwd_f32(const AttnArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch_fwd<64>(a, s) : attn::launch_fwd<128>(a, s);
}

hipError_t launch_attn_bwd_f32(const AttnBwdArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch_bwd<64>(a, s) : attn::launch_bwd<128>(a, s);
}

}  // namespace e2ttt
