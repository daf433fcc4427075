// Causal grouped-head attention in fp32 on the fp32 MFMA: forward over packed
// sequences and over a paged cache, and the gradients.  The same one-pass
// softmax, row packing and operand orientation as the bf16 kernels
// (attn_common.h, attn_fwd.hip, attn_bwd.hip), on 16x16x4 tiles: a 16x16
// accumulator holds rows 4 u + i, u = lane / 16, i = 0..3, of column lane % 16,
// and element i is the operand of k-step i of the next product as it stands,
// with the k index of lane group u at step i meaning row 4 u + i.
//
// The fp32 MFMA issues at a sixteenth of the bf16 rate, so a tile's operands
// have a thousand cycles to arrive, and they come straight from memory into
// registers: nothing is staged in the LDS, and no wave waits for another until
// the sums are added at the end.  A staged row serves twice, by rows (k-steps
// along the head dimension) and by columns (k-steps along the rows); by columns
// a lane takes four neighbouring columns, so that its loads are 16 bytes wide
// too: accumulator 4 h + c of an output then holds column 64 h + 4 m + c in its
// row m.  Each operand has one set of registers, refilled as soon as its
// products are done, while the others' run.
//
// What is scarce in fp32's small layers is workgroups: four heads over two rows
// of 2K leave half the chip idle in tiles of 64 rows or keys.  So the four waves
// of a workgroup share few rows or keys (16), take the tiles of the other axis
// in turn, and add their parts in the LDS; and in the backward the other axis of
// an item is shared out over several workgroups where the items are few.
//
// Four heads of 64 over two key heads, rows of 2048 and 840 tokens: forward 41 us
// (61 Tflop/s), dq 53 (71), dk and dv 71 (71), the join 5, of the 154 that a large
// library product reaches.  The products take half the time on their SIMDs; the
// rest is each wave's way in and out (a wave has about ten tiles) and vector
// instructions, which do not run beside the fp32 MFMA.  (Tiles staged in the LDS,
// with a barrier each: 58, 62 and 99 us.)
#include "attn_common.h"

namespace e2ttt {
namespace attn {
namespace {

constexpr int BN = 64;  // keys of a step of a workgroup (forward, dq): 16 per wave
constexpr int kWaves = 4;
constexpr float kLazy = 8.f;  // as in attn_fwd.hip

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Sum or maximum over the four lane groups that hold one column: a swap of x with
// itself gives each lane its own and the other group's value, in the same order
// in both.
struct Pair {
    float a, b;
};
template <class V>
__device__ __forceinline__ Pair pair_of(const V& r) {
    const unsigned a = r[0], b = r[1];
    return Pair{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ Pair swap16(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    return pair_of(__builtin_amdgcn_permlane16_swap(u, u, false, false));
}
__device__ __forceinline__ Pair swap32(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    return pair_of(__builtin_amdgcn_permlane32_swap(u, u, false, false));
}
__device__ __forceinline__ float groups_sum(float x) {
    const Pair p = swap16(x), q = swap32(p.a + p.b);
    return q.a + q.b;
}
__device__ __forceinline__ float groups_max(float x) {
    const Pair p = swap16(x), q = swap32(fmaxf(p.a, p.b));
    return fmaxf(q.a, q.b);
}

// Loads at a lane's byte offset from a base that the wave shares, so that a tile
// costs no address arithmetic on the vector unit (which the products wait for);
// zeros at kOutside.
typedef __amdgpu_buffer_rsrc_t Base;
__device__ __forceinline__ Base base_of(const float* p) {
    const uint64_t x = (uint64_t)p;
    const uint64_t lo = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)x);
    const uint64_t hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(x >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void*)(hi << 32 | lo), 0, (int)kOutside, RSRC_W3);
}
__device__ __forceinline__ f32x4 load4(Base b, unsigned off) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
}
__device__ __forceinline__ float load1(Base b, unsigned off) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, (int)off, 0, 0));
}

// Offsets of a tile of 16 rows: by rows, of row col, and by columns, of rows
// 4 u + 0..3 (see load_row and ColFrags).  at(r): elements from the base to row r.
template <int DP>
struct RowOffsets {
    unsigned v[DP / 16];
    template <class F>
    __device__ __forceinline__ void init(F&& at, int u, int col, int D) {
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            const int d = 16 * s + 4 * u;
            v[s] = d < D ? (unsigned)(4 * (at(col) + d)) : kOutside;
        }
    }
    __device__ __forceinline__ void load(f32x4 (&f)[DP / 16], Base b, bool in) const {
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) f[s] = load4(b, in ? v[s] : kOutside);
    }
};
template <int DP>
struct ColOffsets {
    unsigned v[4][DP / 64];
    template <class F>
    __device__ __forceinline__ void init(F&& at, int u, int col, int D) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < DP / 64; ++h) {
                const int d = 64 * h + 4 * col;
                v[i][h] = (unsigned)(4 * (at(4 * u + i) + (d < D ? d : 0)));
            }
    }
    template <class F>
    __device__ __forceinline__ void load(f32x4 (&f)[4][DP / 64], Base b, F&& in) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < DP / 64; ++h) f[i][h] = load4(b, in(i) ? v[i][h] : kOutside);
    }
};

// A row by rows: f[s] are its columns 16 s + 4 u + 0..3, the operands of k-steps
// 4 s .. 4 s + 3.  Zeros for a row that is not `in` and past the head dimension.
template <int S4>
__device__ __forceinline__ void load_row(f32x4 (&f)[S4], const float* p, bool in, int u, int D) {
#pragma unroll
    for (int s = 0; s < S4; ++s) {
        const int d = 16 * s + 4 * u;
        f[s] = *(const f32x4*)(in && d < D ? p + d : (const float*)zeros);
    }
}

// Rows 4 u + 0..3 by columns: v[i][h] are columns 64 h + 4 col + 0..3 of row i,
// the operands of k-step i.  (Lanes past the head dimension read the row's start:
// their results are not used.)
template <int DP>
struct ColFrags {
    f32x4 v[4][DP / 64];
    __device__ __forceinline__ void load(int i, const float* p, bool in, int col, int D) {
        const float* q = in ? p : (const float*)zeros;
#pragma unroll
        for (int h = 0; h < DP / 64; ++h) {
            const int d = 64 * h + 4 * col;
            v[i][h] = *(const f32x4*)(q + (d < D ? d : 0));
        }
    }
    __device__ __forceinline__ float get(int i, int dt) const { return v[i][dt / 4][dt % 4]; }
};

// Four neighbouring values e of an output row: columns 64 h + 16 u + 4 e + 0..3.
template <int S4>
__device__ __forceinline__ f32x4 four(const f32x4 (&acc)[S4], int h, int e) {
    return f32x4{acc[4 * h][e], acc[4 * h + 1][e], acc[4 * h + 2][e], acc[4 * h + 3][e]};
}
template <int S4>
__device__ __forceinline__ void store_cols(float* o, const f32x4 (&acc)[S4], float f, int u, int D) {
#pragma unroll
    for (int h = 0; h < S4 / 4; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = 64 * h + 16 * u + 4 * e;
            if (d < D) *(f32x4*)(o + d) = four(acc, h, e) * f;
        }
}
// A wave's sums into its rows of the area where the waves meet, and acc += f
// times those of another.
template <int S4>
__device__ __forceinline__ void put(float* area, const f32x4 (&acc)[S4], int u) {
#pragma unroll
    for (int h = 0; h < S4 / 4; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) *(f32x4*)(area + 64 * h + 16 * u + 4 * e) = four(acc, h, e);
}
template <int S4>
__device__ __forceinline__ void add(f32x4 (&acc)[S4], const float* area, float f, int u) {
#pragma unroll
    for (int h = 0; h < S4 / 4; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f32x4 x = *(const f32x4*)(area + 64 * h + 16 * u + 4 * e);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[4 * h + c][e] = __builtin_fmaf(x[c], f, acc[4 * h + c][e]);
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
    for (int h = 0; h < S4 / 4; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = 64 * h + 16 * u + 4 * e;
            if (w == 0.f || d >= D) continue;
            const f32x4 x = *(const f32x4*)(row + d);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[4 * h + c][e] = __builtin_fmaf(w, x[c], acc[4 * h + c][e]);
            __builtin_amdgcn_sched_barrier(0);
        }
}

// Row r of a key head's rows.
struct Place {
    int tok, head;
    int64_t at;  // in [N][H] order
    bool live;
};
template <class A>
__device__ __forceinline__ Place place(const A& a, int tok0, int kvh, int r, int rows) {
    const bool live = r >= 0 && r < rows;
    const int rr = live ? r : 0, tok = div_group(rr, a.G, a.gmagic), head = kvh * a.G + rr - tok * a.G;
    return Place{tok, head, ((int64_t)tok0 + tok) * a.H + head, live};
}

template <int DP, bool PAGED>
__global__ __launch_bounds__(256, DP == 64 ? 4 : 2) void attn_f32_fwd_kernel(AttnArgs a) {
    constexpr int S4 = DP / 16, LD = DP + 4, BM = kF32Rows;
    __shared__ __attribute__((aligned(16))) float area[kWaves][BM * LD];
    __shared__ float stat[2][kWaves][BM];
    int b = blockIdx.x;
    if (const int past = b - a.ntiles * a.nsplit * a.K; past >= 0) {  // as in attn_fwd.hip
        if (past < a.clear) clear_block<float>(a, past);
        else if constexpr (PAGED) append_block<float>(a, past - a.clear);
        return;
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
    const int w0 = lo + 16 * wave;                                    // this wave's keys of step j: w0 + BN j + 0..15
    const int jw = j1 < nb || w0 + BN * (j1 - 1) <= last ? j1 : j1 - 1;  // and its last step + 1

    const Place x = place(a, it.tok0, kvh, r0 + col, rows);
    const int qpos = x.live ? kept + x.tok : -1;
    const int qlow = a.window > 0 ? qpos - a.window : -1;
    f32x4 qf[S4];
    load_row(qf, (const float*)a.q + (it.tok0 + x.tok) * a.q_tok + (int64_t)x.head * a.q_head, x.live, u, a.D);

    const int fresh = PAGED ? (a.pg.append ? kept : 0x7fffffff) : 0;
    const float* ksrc = (const float*)a.k + it.tok0 * a.k_tok + kvh * a.k_head - (int64_t)fresh * a.k_tok;
    const float* vsrc = (const float*)a.v + it.tok0 * a.v_tok + kvh * a.v_head - (int64_t)fresh * a.v_tok;
    const float* kcache = PAGED ? (const float*)a.pg.kc + kvh * a.pg.k_head : nullptr;
    const float* vcache = PAGED ? (const float*)a.pg.vc + kvh * a.pg.v_head : nullptr;
    // the page of a position (-1: none that is read), and its key and value, read
    // as zeros unless `in`
    auto page_of = [&](int pos) {
        const int pi = pos >> a.pg.shift;
        const bool held = PAGED && pos >= begin && pos <= last && pos < fresh && pi < a.pg.wide;
        return held ? a.pg.table[(int64_t)it.seq * a.pg.wide + pi] : -1;
    };
    auto seen = [&](int pos, int page) {
        return pos >= begin && pos <= last && (!PAGED || pos >= fresh || (unsigned)page < (unsigned)a.pg.pages);
    };
    auto key_of = [&](int pos, int page) {
        if (!PAGED || pos >= fresh) return ksrc + pos * a.k_tok;
        return kcache + (page * a.pg.k_page + (pos & ((1 << a.pg.shift) - 1)) * a.pg.k_slot);
    };
    auto value_of = [&](int pos, int page) {
        if (!PAGED || pos >= fresh) return vsrc + pos * a.v_tok;
        return vcache + (page * a.pg.v_page + (pos & ((1 << a.pg.shift) - 1)) * a.pg.v_slot);
    };
    f32x4 kf[S4];
    ColFrags<DP> vf;
    RowOffsets<DP> ko;  // packed sequences
    ColOffsets<DP> vo;
    if constexpr (!PAGED) {
        ko.init([&](int r) { return r * a.k_tok; }, u, col, a.D);
        vo.init([&](int r) { return r * a.v_tok; }, u, col, a.D);
    }
    int page = -1;  // of position w0 + BN j + col of the next step
    auto load_pages = [&](int j) { return PAGED ? page_of(w0 + BN * j + col) : -1; };
    auto load_keys = [&](int j) {
        const int p0 = w0 + BN * j, pos = p0 + col;
        if constexpr (PAGED) {
            load_row(kf, key_of(pos, page), seen(pos, page), u, a.D);
        } else {
            const Base kb = base_of(ksrc + p0 * a.k_tok);
            ko.load(kf, kb, seen(pos, -1));
        }
    };
    auto load_values = [&](int j) {
        const int p0 = w0 + BN * j;
        if constexpr (PAGED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pos = p0 + 4 * u + i, p = __shfl(page, 4 * u + i);
                vf.load(i, value_of(pos, p), seen(pos, p), col, a.D);
            }
        } else {
            const Base vb = base_of(vsrc + p0 * a.v_tok);
            vo.load(vf.v, vb, [&](int i) { return seen(p0 + 4 * u + i, -1); });
        }
    };

    f32x4 acc[S4] = {};
    float m = neg_inf(), l = 0.f;
    if (j0 < jw) {
        page = load_pages(j0);
        load_keys(j0);
        load_values(j0);
        page = load_pages(j0 + 1);
    }
    for (int j = j0; j < jw; ++j) {
        const int p0 = w0 + BN * j, ahead = load_pages(j + 2), next = j + 1 < jw ? j + 1 : j;
        f32x4 sc = {}, so = {};  // two chains, so that no product waits for the one before it
#pragma unroll
        for (int s = 0; s < S4; ++s)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                sc = mfma4(kf[s][e], qf[s][e], sc);
                so = mfma4(kf[s][e + 1], qf[s][e + 1], so);
            }
        load_keys(next);
        __builtin_amdgcn_sched_barrier(0);
        sc += so;
        if (p0 + 15 > first || (a.window > 0 && p0 <= last - a.window)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = p0 + 4 * u + i;
                if (p > qpos || p <= qlow) sc[i] = neg_inf();
            }
        }
        const float mx = groups_max(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]))) * a.sl2;
        if (__any(mx > m + kLazy)) {
            const float mn = fmaxf(m, mx);
            const float f = __builtin_amdgcn_exp2f(m - (mn == neg_inf() ? 0.f : mn));
            m = mn;
            l *= f;
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) acc[dt] *= f;
        }
        const float mu = m == neg_inf() ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sc[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], a.sl2, -mu));
            l += sc[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) acc[dt] = mfma4(vf.get(i, dt), sc[i], acc[dt]);
        load_values(next);
        __builtin_amdgcn_sched_barrier(0);
        page = ahead;
    }
    l = groups_sum(l);
    if (j0 < jw && first != last) {  // sums that are not finite, position by position
        const float bad = not_finite(acc);
        if (__any(bad != bad && l == l)) {
            const float mu = m == neg_inf() ? 0.f : m;
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) acc[dt] = f32x4{};
#pragma unroll 1
            for (int i = j0 * 16; i < jw * 16; ++i) {
                const int p = w0 + i / 16 * BN + i % 16, pg = page_of(p);
                if (!seen(p, pg)) continue;
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_row4(key_of(p, pg), qf, u, a.D), a.sl2, -mu));
                add_row4(acc, value_of(p, pg), p > qpos || p <= qlow ? 0.f : e, u, a.D);
            }
        }
    }
    // the four waves together
    if (u == 0) {
        stat[0][wave][col] = m;
        stat[1][wave][col] = l;
    }
    put(area[wave] + col * LD, acc, u);
    __syncthreads();
    if (wave > 0 || !x.live) return;
    float mw[kWaves], mn = neg_inf(), sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mn = fmaxf(mn, mw[w] = stat[0][w][col]);
    const float mu = mn == neg_inf() ? 0.f : mn;
    f32x4 o[S4] = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(mw[w] - mu);
        sum += stat[1][w][col] * f;
        add(o, area[w] + col * LD, f, u);
    }
    const float inv = sum > 0.f ? 1.f / sum : sum;  // a row that sees nothing gives 0; NaN stays
    const float lse2 = sum > 0.f ? mn + __builtin_amdgcn_logf(sum) : (sum == 0.f ? neg_inf() : sum);
    if (a.nsplit > 1) {
        const int64_t at = (int64_t)split * a.N * a.H + x.at;
        if (u == 0) a.pl[at] = lse2;
        if (j0 < j1) store_cols(a.po + at * a.D, o, inv, u, a.D);
        return;
    }
    if (a.lse && u == 0) a.lse[x.at] = lse2 * kLn2;
    store_cols((float*)a.out + x.at * a.D, o, inv, u, a.D);
}

template <int DP, int RT>
__global__ __launch_bounds__(256, 2) void attn_f32_dq_kernel(AttnBwdArgs a) {
    constexpr int S4 = DP / 16, LD = DP + 4, BM = 16 * RT;
    __shared__ __attribute__((aligned(16))) float area[kWaves][BM * LD];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = lane >> 4, col = lane & 15, G = a.G;
    if (const int past = (int)(blockIdx.x + a.clear) - (int)gridDim.x; past >= 0) {  // as in attn_bwd.hip
        fill_outside(a.cu, a.S, a.N, a.dq, (int64_t)a.H * a.D * 4, 0, past, a.clear);
        return;
    }
    const int kvh = blockIdx.x % a.K, part = blockIdx.x / a.K % a.dq_parts, t = blockIdx.x / a.K / a.dq_parts;
    Item it;
    if (!find_item(a.cu, a.S, (int)a.N, t, row_cap(a.window, G, BM), [&](int n) { return (n * G + BM - 1) / BM; }, it)) return;
    const int r0 = it.tile * BM;
    const int rows = it.n * G;
    const int first = div_group(r0, G, a.gmagic);
    const int last = div_group(r0 + BM < rows ? r0 + BM - 1 : rows - 1, G, a.gmagic);
    const int begin = a.window > 0 && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
    // this wave's tiles of 16 keys: from w0 on, every W keys
    const int W = 16 * kWaves * a.dq_parts;
    const int w0 = (begin & ~15) + 16 * (kWaves * part + wave);
    const int nb = w0 <= last ? (last - w0) / W + 1 : 0;

    int qpos[RT], qlow[RT];
    float delta[RT], lse2[RT];
    f32x4 qf[RT][S4], df[RT][S4];
#pragma unroll
    for (int c = 0; c < RT; ++c) {
        const Place x = place(a, it.tok0, kvh, r0 + 16 * c + col, rows);
        qpos[c] = x.live ? x.tok : -1;
        qlow[c] = a.window > 0 ? qpos[c] - a.window : -1;
        load_row(qf[c], (const float*)a.q + (it.tok0 + x.tok) * a.q_tok + (int64_t)x.head * a.q_head, x.live, u, a.D);
        load_row(df[c], (const float*)a.dout + x.at * a.D, x.live, u, a.D);
        f32x4 of[S4];
        load_row(of, (const float*)a.out + x.at * a.D, x.live, u, a.D);
        float d = 0.f;
#pragma unroll
        for (int s = 0; s < S4; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) d = __builtin_fmaf(df[c][s][e], of[s][e], d);
        delta[c] = groups_sum(d);
        if (x.live && u == 0 && wave == 0 && part == 0) a.stats[x.at] = delta[c];
        lse2[c] = x.live ? a.lse[x.at] * kLog2e : 0.f;
    }

    const float* ksrc = (const float*)a.k + it.tok0 * a.k_tok + kvh * a.k_head;
    const float* vsrc = (const float*)a.v + it.tok0 * a.v_tok + kvh * a.v_head;
    f32x4 kf[S4], vf[S4];
    ColFrags<DP> kc;
    auto seen = [&](int pos) { return pos >= begin && pos <= last; };
    RowOffsets<DP> kro, vro;
    ColOffsets<DP> kco;
    kro.init([&](int r) { return r * a.k_tok; }, u, col, a.D);
    vro.init([&](int r) { return r * a.v_tok; }, u, col, a.D);
    kco.init([&](int r) { return r * a.k_tok; }, u, col, a.D);
    auto load_rows = [&](int p0) {
        const Base kb = base_of(ksrc + p0 * a.k_tok), vb = base_of(vsrc + p0 * a.v_tok);
        const bool in = seen(p0 + col);
        kro.load(kf, kb, in);
        vro.load(vf, vb, in);
    };
    auto load_cols = [&](int p0) {
        const Base kb = base_of(ksrc + p0 * a.k_tok);
        kco.load(kc.v, kb, [&](int i) { return seen(p0 + 4 * u + i); });
    };
    f32x4 acc[RT][S4] = {};
    if (nb > 0) {
        load_rows(w0);
        load_cols(w0);
    }
    for (int j = 0; j < nb; ++j) {
        const int p0 = w0 + W * j, next = j + 1 < nb ? p0 + W : p0;
        f32x4 sc[RT] = {}, dp[RT] = {};
#pragma unroll
        for (int s = 0; s < S4; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < RT; ++c) {
                    sc[c] = mfma4(kf[s][e], qf[c][s][e], sc[c]);
                    dp[c] = mfma4(vf[s][e], df[c][s][e], dp[c]);
                }
        load_rows(next);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < RT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[c][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[c][i], a.sl2, -lse2[c])) * (dp[c][i] - delta[c]);
            }
        if (p0 + 15 > first || (a.window > 0 && p0 <= last - a.window)) {
#pragma unroll
            for (int c = 0; c < RT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = p0 + 4 * u + i;
                    if (p > qpos[c] || p <= qlow[c]) sc[c][i] = 0.f;
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int dt = 0; dt < S4; ++dt)
#pragma unroll
                for (int c = 0; c < RT; ++c) acc[c][dt] = mfma4(kc.get(i, dt), sc[c][i], acc[c][dt]);
        load_cols(next);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int c = 0; c < RT; ++c) {
        if (first != last) {  // sums that are not finite, as in the forward
            const float bad = not_finite(acc[c]);
            if (__any(bad != bad && lse2[c] == lse2[c] && delta[c] == delta[c])) {
#pragma unroll
                for (int dt = 0; dt < S4; ++dt) acc[c][dt] = f32x4{};
#pragma unroll 1
                for (int i = 0; i < nb * 16; ++i) {
                    const int p = w0 + i / 16 * W + i % 16;
                    if (!seen(p)) continue;
                    const float* kp = ksrc + p * a.k_tok;
                    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_row4(kp, qf[c], u, a.D), a.sl2, -lse2[c]));
                    const float y = x * (dot_row4(vsrc + p * a.v_tok, df[c], u, a.D) - delta[c]);
                    add_row4(acc[c], kp, p > qpos[c] || p <= qlow[c] ? 0.f : y, u, a.D);
                }
            }
        }
        put(area[wave] + (16 * c + col) * LD, acc[c], u);
    }
    __syncthreads();
    if (wave >= RT) return;
    const int rr = 16 * wave + col;
    const Place x = place(a, it.tok0, kvh, r0 + rr, rows);
    if (!x.live) return;
    f32x4 o[S4] = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) add(o, area[w] + rr * LD, 1.f, u);
    if (a.dq_parts > 1)
        store_cols(a.part + ((int64_t)part * a.N * a.H + x.at) * a.D, o, 1.f, u, a.D);
    else
        store_cols((float*)a.dq + x.at * a.D, o, a.scale, u, a.D);
}

// STEADY: the group's size divides 16, so that a tile starts on a token and a
// lane's offsets are the same in every tile, and the strides keep them in 31 bits.
template <int DP, int RT, bool STEADY>
__global__ __launch_bounds__(256, DP == 64 ? 2 : 1) void attn_f32_dkdv_kernel(AttnBwdArgs a) {
    constexpr int S4 = DP / 16, LD = DP + 4, BK = 16 * RT;
    __shared__ __attribute__((aligned(16))) float area[2][kWaves][BK * LD];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = lane >> 4, col = lane & 15, G = a.G;
    if (const int past = (int)(blockIdx.x + a.clear) - (int)gridDim.x; past >= 0) {
        fill_outside(a.cu, a.S, a.N, a.dk, (int64_t)a.K * a.D * 4, 0, past, a.clear);
        fill_outside(a.cu, a.S, a.N, a.dv, (int64_t)a.K * a.D * 4, 0, past, a.clear);
        return;
    }
    const int kvh = blockIdx.x % a.K, part = blockIdx.x / a.K % a.dkv_parts, t = blockIdx.x / a.K / a.dkv_parts;
    Item it;
    if (!find_item(a.cu, a.S, (int)a.N, t, row_cap(a.window, 1, BK), [&](int n) { return (n + BK - 1) / BK; }, it)) return;
    const int k0 = (it.tiles - 1 - it.tile) * BK;  // the first keys of a sequence have the most rows
    const int rows = it.n * G;
    const int klast = k0 + BK < it.n ? k0 + BK - 1 : it.n - 1;
    const bool ragged = k0 + BK > it.n;
    const int rbeg = k0 * G & ~15;
    const int64_t re = a.window > 0 ? ((int64_t)klast + a.window) * G : rows;
    const int rend = re < rows ? (int)re : rows;
    // tiles of 16 rows from the last one back (as in attn_bwd.hip): this wave's
    // from `top` on, every W rows
    const int W = 16 * kWaves * a.dkv_parts, w = kWaves * part + wave;
    const int tiles = (rend - rbeg + 15) / 16;
    const int top = rbeg + 16 * (tiles - 1 - w);
    const int nb = w < tiles ? 16 * (tiles - 1 - w) / W + 1 : 0;

    // rows that see the key of lane column col of tile c: [rlo, rhi)
    int rlo[RT], rhi[RT];
    f32x4 kf[RT][S4], vf[RT][S4];
#pragma unroll
    for (int c = 0; c < RT; ++c) {
        const int key = k0 + 16 * c + col;
        const bool live = key < it.n;
        const int64_t ktok = it.tok0 + (live ? key : 0);
        rlo[c] = live ? key * G : 0x7fffffff;
        const int64_t rh = a.window > 0 ? ((int64_t)key + a.window) * G : rows;
        rhi[c] = rh < rows ? (int)rh : rows;
        load_row(kf[c], (const float*)a.k + ktok * a.k_tok + (int64_t)kvh * a.k_head, live, u, a.D);
        load_row(vf[c], (const float*)a.v + ktok * a.v_tok + (int64_t)kvh * a.v_head, live, u, a.D);
    }

    const float *qsrc = (const float*)a.q + it.tok0 * a.q_tok, *dout = (const float*)a.dout;
    f32x4 qf[S4], of[S4], ls, de;
    ColFrags<DP> qc, oc;
    auto row_of = [&](const Place& x) { return qsrc + x.tok * a.q_tok + x.head * a.q_head; };
    RowOffsets<DP> qro, oro;
    ColOffsets<DP> qco, oco;
    unsigned so[4];
    const int64_t first_row = (int64_t)it.tok0 * a.H + kvh * G;  // row 0 in [N][H] order
    if constexpr (STEADY) {
        auto q_at = [&](int r) {
            const int tk = div_group(r, G, a.gmagic);
            return tk * a.q_tok + (r - tk * G) * a.q_head;
        };
        auto at = [&](int r) {
            const int tk = div_group(r, G, a.gmagic);
            return (int64_t)tk * a.H + r - tk * G;
        };
        qro.init(q_at, u, col, a.D);
        qco.init(q_at, u, col, a.D);
        oro.init([&](int r) { return at(r) * a.D; }, u, col, a.D);
        oco.init([&](int r) { return at(r) * a.D; }, u, col, a.D);
#pragma unroll
        for (int i = 0; i < 4; ++i) so[i] = (unsigned)(4 * at(4 * u + i));
    }
    auto load_rows = [&](int p0) {
        if constexpr (STEADY) {
            const int64_t tk = div_group(p0, G, a.gmagic), x = first_row + tk * a.H;
            const Base qb = base_of(qsrc + (int64_t)kvh * G * a.q_head + tk * a.q_tok), ob = base_of(dout + x * a.D);
            const bool in = p0 + col < rend;
            qro.load(qf, qb, in);
            oro.load(of, ob, in);
        } else {
            const Place x = place(a, it.tok0, kvh, p0 + col, rend);
            load_row(qf, row_of(x), x.live, u, a.D);
            load_row(of, dout + x.at * a.D, x.live, u, a.D);
        }
    };
    auto load_cols = [&](int p0) {
        if constexpr (STEADY) {
            const int64_t tk = div_group(p0, G, a.gmagic), x = first_row + tk * a.H;
            const Base qb = base_of(qsrc + (int64_t)kvh * G * a.q_head + tk * a.q_tok), ob = base_of(dout + x * a.D);
            const Base lb = base_of(a.lse + x), sb = base_of(a.stats + x);
            auto in = [&](int i) { return p0 + 4 * u + i < rend; };
            qco.load(qc.v, qb, in);
            oco.load(oc.v, ob, in);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ls[i] = load1(lb, in(i) ? so[i] : kOutside);
                de[i] = load1(sb, in(i) ? so[i] : kOutside);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Place x = place(a, it.tok0, kvh, p0 + 4 * u + i, rend);
                qc.load(i, row_of(x), x.live, col, a.D);
                oc.load(i, dout + x.at * a.D, x.live, col, a.D);
                ls[i] = a.lse[x.at];
                de[i] = a.stats[x.at];
            }
        }
    };
    f32x4 dk[RT][S4] = {}, dv[RT][S4] = {};
    if (nb > 0) {
        load_rows(top);
        load_cols(top);
    }
    for (int j = 0; j < nb; ++j) {
        const int p0 = top - W * j, next = j + 1 < nb ? p0 - W : p0;
        f32x4 sc[RT] = {}, dp[RT] = {};
#pragma unroll
        for (int s = 0; s < S4; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < RT; ++c) {
                    sc[c] = mfma4(qf[s][e], kf[c][s][e], sc[c]);
                    dp[c] = mfma4(of[s][e], vf[c][s][e], dp[c]);
                }
        load_rows(next);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < RT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[c][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[c][i], a.sl2, -ls[i] * kLog2e));
                dp[c][i] = sc[c][i] * (dp[c][i] - de[i]);
            }
        if (ragged || p0 < klast * G || p0 + 16 > rend || (a.window > 0 && p0 + 16 > ((int64_t)k0 + a.window) * G)) {
#pragma unroll
            for (int c = 0; c < RT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = p0 + 4 * u + i;
                    const bool out = r < rlo[c] || r >= rhi[c];
                    sc[c][i] = out ? 0.f : sc[c][i];
                    dp[c][i] = out ? 0.f : dp[c][i];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int dt = 0; dt < S4; ++dt)
#pragma unroll
                for (int c = 0; c < RT; ++c) {
                    dv[c][dt] = mfma4(oc.get(i, dt), sc[c][i], dv[c][dt]);
                    dk[c][dt] = mfma4(qc.get(i, dt), dp[c][i], dk[c][dt]);
                }
        load_cols(next);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int c = 0; c < RT; ++c) {
        const float bad = not_finite(dk[c]) + not_finite(dv[c]);
        if (__any(bad != bad)) {  // as in the forward
#pragma unroll
            for (int dt = 0; dt < S4; ++dt) dk[c][dt] = dv[c][dt] = f32x4{};
#pragma unroll 1
            for (int i = 0; i < nb * 16; ++i) {
                const int r = top - W * (i / 16) + i % 16;
                const Place x = place(a, it.tok0, kvh, r, rend);
                if (!x.live) continue;
                const float *qp = row_of(x), *op = dout + x.at * a.D;
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_row4(qp, kf[c], u, a.D), a.sl2, -a.lse[x.at] * kLog2e));
                const float ds = p * (dot_row4(op, vf[c], u, a.D) - a.stats[x.at]);
                const bool out = r < rlo[c] || r >= rhi[c];
                add_row4(dv[c], op, out ? 0.f : p, u, a.D);
                add_row4(dk[c], qp, out ? 0.f : ds, u, a.D);
            }
        }
        put(area[0][wave] + (16 * c + col) * LD, dk[c], u);
        put(area[1][wave] + (16 * c + col) * LD, dv[c], u);
    }
    // the four waves' rows together, in order
    __syncthreads();
    float* parts = a.part + (a.dq_parts > 1 ? a.dq_parts * a.N * a.H * a.D : 0);
    for (int x = threadIdx.x; x < 2 * BK * (DP / 4); x += 256) {
        const int which = x / (BK * (DP / 4)), kk = x / (DP / 4) % BK, d = x % (DP / 4) * 4;
        if (k0 + kk >= it.n || d >= a.D) continue;
        const float* src = area[which][0] + kk * LD + d;
        f32x4 y = *(const f32x4*)src;
#pragma unroll
        for (int v = 1; v < kWaves; ++v) y += *(const f32x4*)(src + v * (BK * LD));
        const int64_t o = (((int64_t)it.tok0 + k0 + kk) * a.K + kvh) * a.D + d;
        if (a.dkv_parts > 1)
            *(f32x4*)(parts + ((int64_t)part * 2 + which) * a.N * a.K * a.D + o) = y;
        else
            *(f32x4*)((which ? (float*)a.dv : (float*)a.dk) + o) = which ? y : y * a.scale;
    }
}

// The gradients from the parts' sums, in order: dq, then dk, then dv.  (Tokens
// outside every sequence have none, and their zeros already.)
__global__ __launch_bounds__(256) void attn_f32_parts_kernel(AttnBwdArgs a) {
    const int64_t nq = a.dq_parts > 1 ? a.N * a.H * a.D : 0, nk = a.dkv_parts > 1 ? a.N * a.K * a.D : 0;
    int64_t o = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    const float* src = a.part + o;
    float* dst = (float*)a.dq;
    int64_t stride = nq, heads = a.H;
    int parts = a.dq_parts;
    float f = a.scale;
    if (o >= nq) {
        o -= nq;
        if (o >= 2 * nk) return;
        src = a.part + a.dq_parts * nq + o;
        stride = 2 * nk;
        heads = a.K;
        parts = a.dkv_parts;
        dst = (float*)a.dk;
        if (o >= nk) {
            o -= nk;
            dst = (float*)a.dv;
            f = 1.f;
        }
    }
    const int64_t tok = o / (heads * a.D);
    if (tok < clamped(a.cu[0], (int)a.N) || tok >= clamped(a.cu[a.S], (int)a.N)) return;
    f32x4 y = {};
    for (int p = 0; p < parts; ++p) y += *(const f32x4*)(src + p * stride);
    *(f32x4*)(dst + o) = y * f;
}

// Tiles of 16 rows (dq) or keys (dkdv) of a wave in the backward, which share its
// loads: two where their operands and sums fit in 256 registers.  (Two rows of up
// to 2K, four heads of 64: dq 53 us with two, 64 with one; dkdv 71 and 68, the
// forward 52 and 44, its loads being fewer: one.)
constexpr int bwd_tiles(int64_t D) { return D <= 64 ? 2 : 1; }

template <int DP>
hipError_t launch_fwd(const AttnArgs& a, hipStream_t s) {
    const bool paged = a.pg.kc != nullptr;
    const int64_t grid = (int64_t)a.ntiles * a.K * a.nsplit + a.clear + (paged ? append_blocks(a, 4) : 0);
    if (grid == 0) return hipSuccess;
    if (grid > kMaxGroups) return hipErrorInvalidConfiguration;
    if (paged)
        attn_f32_fwd_kernel<DP, true><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a);
    else
        attn_f32_fwd_kernel<DP, false><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <int DP>
hipError_t launch_bwd(const AttnBwdArgs& a, hipStream_t s) {
    constexpr int RT = bwd_tiles(DP), B = 16 * RT;
    const int64_t dq_grid = (a.N * a.G / B + a.S) * a.K * a.dq_parts + a.clear;
    const int64_t dkv_grid = (a.N / B + a.S) * a.K * a.dkv_parts + a.clear;
    const int64_t sums = a.N * a.D * ((a.dq_parts > 1 ? a.H : 0) + (a.dkv_parts > 1 ? 2 * a.K : 0));
    const int64_t sum_grid = (sums / 4 + 255) / 256;
    if (dq_grid > kMaxGroups || dkv_grid > kMaxGroups || sum_grid > kMaxGroups) return hipErrorInvalidConfiguration;
    attn_f32_dq_kernel<DP, RT><<<dim3((unsigned)dq_grid), dim3(256), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (16 % a.G == 0 && a.q_head < (1 << 25) / a.G) attn_f32_dkdv_kernel<DP, RT, true><<<dim3((unsigned)dkv_grid), dim3(256), 0, s>>>(a);
    else attn_f32_dkdv_kernel<DP, RT, false><<<dim3((unsigned)dkv_grid), dim3(256), 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess || sums == 0) return e;
    attn_f32_parts_kernel<<<dim3((unsigned)sum_grid), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

// Workgroups that share an item's keys (dq) or rows (dkdv), so that the longest
// items of a small call do not keep the others waiting: as many as give each
// compute unit two workgroups (the same layer's forward and backward, 170 us:
// with one per compute unit 44 us more, with four 4 us more).
static int parts_of(int64_t items) {
    const int64_t n = items > 0 ? (512 + items - 1) / items : 1;
    return (int)(n > 8 ? 8 : n);
}
void attn_f32_parts(int64_t N, int64_t G, int64_t K, int64_t D, int* dq, int* dkv) {
    const int64_t B = 16 * attn::bwd_tiles(D);
    *dq = parts_of((N * G + B - 1) / B * K);
    *dkv = parts_of((N + B - 1) / B * K);
}

hipError_t launch_attn_fwd_f32(const AttnArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch_fwd<64>(a, s) : attn::launch_fwd<128>(a, s);
}

hipError_t launch_attn_bwd_f32(const AttnBwdArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch_bwd<64>(a, s) : attn::launch_bwd<128>(a, s);
}

}  // namespace e2ttt
