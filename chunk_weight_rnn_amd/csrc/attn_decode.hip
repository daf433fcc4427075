// Attention of few new tokens per sequence over a paged cache, bf16 (plain
// decoding: one token each).
//
// HBM bound: every visible key and value once.  An item is a sequence, a key
// head and a tile of 32 rows (the group's heads of up to 32 / G tokens), and
// its keys are cut into units of 128.  Contexts differ, so items are not the
// grid: the units of all items stand in one line, every workgroup takes an
// equal stretch of it, and where a stretch begins or ends inside an item the
// partial result goes to the workspace and a second launch joins it.  A
// workgroup is one per compute unit, 4 waves that each stream their own 32
// keys of a unit through two LDS stages of their own (no barrier until the
// item ends).  A stage is refilled as soon as it has been used, so that a wave
// waits with both in flight, 128 KiB per compute unit; page indices go through
// the LDS too, two units ahead, because a wait for one in a register would be a
// wait for every copy before it.
//
// The products are the same as in attn_fwd.hip, S^T = K Q^T and O^T += V^T P^T
// on 32x32 tiles; a group of 4 heads fills 4 of the 32 columns, which costs
// nothing here, since the MFMAs need a fifth of the time of the copies.
//
// 64 tokens at contexts of 2K to 16K, 16 heads of 128 over 4: 189 us, 5.5 TB/s of
// keys and values (a large copy moves 5.1, a read alone at most 6.3).  One token at
// a context of 513 in one launch: 14.0 us, of which the keys take 9, at the 28 bytes
// per ns that a compute unit can take in; the rest is the launch and the way to the
// first key.
#include "attn_decode.h"

namespace e2ttt {
namespace attn {
namespace {

template <int DP, bool SPLIT>
__global__ __launch_bounds__(256, 1) void attn_decode_kernel(AttnArgs a, int groups) {
    constexpr int TILE = BW * DP * 2;            // a wave's keys (or values) of a unit
    constexpr int RPI = 512 / DP;                // rows per copy instruction
    constexpr int NI = BW / RPI, CH = DP / 8;
    constexpr int KS = DP / 16, DT = DP / 32;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[4][2][2][TILE];  // [wave][stage][K, V]
    __shared__ float stat[4][2][BM];                                             // [wave][m, l]
    __shared__ __attribute__((aligned(256))) int pages[4][4][64];                // [wave][unit % 4][key]
    static_assert(kMergeFloats<DP> * 4 <= (int)sizeof(lds), "the merge area fits in the stages");

    if ((int)blockIdx.x >= groups) {
        const int past = blockIdx.x - groups;
        if (past < a.clear) clear_block<__bf16>(a, past);
        else append_block<__bf16>(a, past - a.clear);
        return;
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31, G = a.G;
    const Seq q0 = seq_of(a, lane);
    int u, uend;
    if (SPLIT) {
        const int total = total_units(a, q0, lane), per = share(total, groups);
        u = blockIdx.x * per < total ? blockIdx.x * per : total;
        uend = u + per < total ? u + per : total;
    } else {
        u = blockIdx.x;
        uend = u + 1;
    }
    const unsigned rb0 = row_base<DP>(col, g), tb0 = tr_base<DP>(lane);
    const int crow = lane / CH;
    const unsigned base = lds_addr(&lds[wave][0][0][0]);

    bool first_seg = true;
    while (u < uend) {
        Work w;
        if (!find_work<SPLIT>(a, q0, u, lane, w)) return;
        const int b0 = w.block, b1 = SPLIT ? (w.nb < b0 + uend - u ? w.nb : b0 + uend - u) : w.nb;
        const bool whole = b0 == 0 && b1 == w.nb;

        const int rows = w.n * G, r0 = w.rt * BM;
        const int row = r0 + col;
        const bool live = row < rows;
        const int tok = live ? div_group(row, G, a.gmagic) : 0, hg = live ? row - tok * G : 0;
        const int qpos = live ? w.kept + tok : -1;
        const int qlow = a.window > 0 ? qpos - a.window : -1;
        const int first = w.kept + div_group(r0, G, a.gmagic);
        const int last = w.kept + div_group(r0 + BM < rows ? r0 + BM - 1 : rows - 1, G, a.gmagic);
        const int64_t qtok = w.tok0 + tok;
        const int head = w.kvh * G + hg;

        bf16x8 qf[KS];
        const __bf16* qp = (const __bf16*)a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 8 * chunk_of(s, g);
            bf16x8 z = {};
            qf[s] = live && d < a.D ? *(const bf16x8*)(qp + d) : z;
        }
        PageCopy<DP, NI, BW> pc;
        pc.init(a, w.kvh, w.tok0, w.kept, 0);
        pc.begin = a.window > 0 ? first - a.window + 1 : 0;
        pc.end = last + 1;
        const int* table = a.pg.table + (int64_t)w.seq * a.pg.wide;

        // This wave's part of unit b, in two steps: the pages of its keys, and
        // two units later the keys and values themselves.  Each is always the
        // same number of copies, which the waits below count.
        auto copy_pages = [&](int b) {
            const int pos = w.lo + b * UNIT + BW * wave + col, pi = pos >> a.pg.shift;
            const bool in = b < b1 && pos >= pc.begin && pos < pc.end && pos < pc.fresh && pi < a.pg.wide;
            copy4_at(in ? table + pi : &no_page, lds_addr(&pages[wave][b & 3][0]));
        };
        auto copy_part = [&](int b) {
            const unsigned dst = base + (b & 1) * (2 * TILE);
            const int* pg = &pages[wave][b & 3][crow];
            pc.copy(a, w.lo + b * UNIT + BW * wave, dst, dst + TILE, [&](int i) { return pg[RPI * i]; });
        };

        f32x16 acc[DT] = {};
        float m = neg_inf(), l = 0.f;
        copy_pages(b0);
        copy_pages(b0 + 1);
        wait_vm<0>();
        copy_part(b0);
        copy_pages(b0 + 2);
        if (b0 + 1 < b1) copy_part(b0 + 1);
        copy_pages(b0 + 3);
        for (int b = b0; b < b1; ++b) {
            const int stage = b & 1;
            // all but the next unit's copies and the page copy after them
            if (b + 1 < b1) wait_vm<2 * NI + 1>();
            else wait_vm<0>();
            const int p0 = w.lo + b * UNIT + BW * wave;
            if (p0 <= last) {
                const unsigned char *kt = lds[0][0][0], *vt = lds[0][0][1];
                const unsigned rb = rb0 + (2 * wave + stage) * (2 * TILE), tb = tb0 + (2 * wave + stage) * (2 * TILE);
                f32x16 sc = {};
#pragma unroll
                for (int s = 0; s < KS; ++s) sc = mfma32(row_frag(kt, rb, s), qf[s], sc);
                if (p0 + BW - 1 > first || a.window > 0 || r0 + BM > rows) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int p = p0 + acc_row(i, g);
                        if (p > qpos || p <= qlow) sc[i] = neg_inf();
                    }
                }
                float mx = sc[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i]);
                mx = fmaxf(mx, other_half(mx, lane)) * a.sl2;
                if (__any(mx > m + kLazy)) {
                    const float mn = fmaxf(m, mx);
                    const float f = mn == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(m - mn);
                    m = mn;
                    l *= f;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[dt][i] *= f;
                }
                const float mu = m == neg_inf() ? 0.f : m;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sc[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], a.sl2, -mu));
                    l += sc[i];
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const bf16x8 pf = pack_half(sc, s);
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt)
                        acc[dt] = mfma32(tr_frag<DP>(vt + s * (32 * DP), tb, dt), pf, acc[dt]);
                }
            }
            if (b + 2 < b1) {
                wait_lds();  // the stage has been read
                copy_part(b + 2);
                copy_pages(b + 4);
            }
        }
        l += other_half(l, lane);
        // rows of more than one position whose sums are not finite (attn_common.h)
        if (first != last) {
            const float bad = not_finite(acc);
            if (__any(bad != bad && l == l)) {
                const float mu = m == neg_inf() ? 0.f : m;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) acc[dt] = f32x16{};
#pragma unroll 1
                for (int i = b0 * BW; i < b1 * BW; ++i) {
                    const int p = w.lo + i / BW * UNIT + BW * wave + i % BW;
                    const char *kp = pc.template row<false>(a, table, p), *vp = pc.template row<true>(a, table, p);
                    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_rows<DP>(kp, (const char*)qp, a.D, lane), a.sl2, -mu));
                    add_row<DP>(acc, vp, p > qpos || p <= qlow ? 0.f : to_bf16(x), a.D, lane);
                }
            }
        }

        finish_item<DP, SPLIT>(a, w, acc, m, l, live, whole, 2 * blockIdx.x + (first_seg ? 0 : 1), (float*)&lds[0][0][0][0], stat);
        __syncthreads();  // the area is the next item's stages
        u += b1 - b0;
        first_seg = false;
        if (!SPLIT) break;
    }
}

// Joins the items that span several workgroups' stretches; one workgroup per
// item, a wave per row.
template <int DP>
__global__ __launch_bounds__(256) void attn_decode_join_kernel(AttnArgs a, int groups) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, G = a.G;
    const Seq q0 = seq_of(a, lane);
    const int total = total_units(a, q0, lane), per = share(total, groups);
    Work w;
    if (!find_work<false>(a, q0, blockIdx.x, lane, w)) return;
    const int before = w.before;
    const int w0 = before / per, w1 = (before + w.nb - 1) / per;
    if (w0 == w1) return;
    const int rows = w.n * G, r0 = w.rt * BM;
    const int count = rows - r0 < BM ? rows - r0 : BM;
    const int d = 2 * lane;
    for (int r = wave; r < count; r += 4) {
        auto slot_row = [&](int v) { return (int64_t)(2 * v + (v == w0 && before > v * per ? 1 : 0)) * BM + r; };
        // a lane per stretch, 64 at a time
        float m = neg_inf();
        for (int v0 = w0; v0 <= w1; v0 += 64)
            m = max_or_nan(m, wave_max_or_nan(v0 + lane <= w1 ? a.pl[slot_row(v0 + lane)] : neg_inf()));
        float o0 = 0.f, o1 = 0.f, sum = 0.f;
        for (int v0 = w0; v0 <= w1; v0 += 64) {
            const float x = v0 + lane <= w1 ? a.pl[slot_row(v0 + lane)] : neg_inf();
            const float f = x == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(x - m);
            sum += f;
            const int n = w1 + 1 - v0 < 64 ? w1 + 1 - v0 : 64;
            join_rows(n, f, d < a.D, [&](int i) { return a.po + slot_row(v0 + i) * a.D + d; }, o0, o1);
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.f ? 1.f / sum : sum;
        const int rr = r0 + r, tk = div_group(rr, G, a.gmagic), hd = w.kvh * G + rr - tk * G;
        if (d < a.D) {
            __bf16* o = (__bf16*)a.out + ((int64_t)(w.tok0 + tk) * a.H + hd) * a.D + d;
            o[0] = (__bf16)(o0 * inv);
            o[1] = (__bf16)(o1 * inv);
        }
    }
}

template <int DP>
hipError_t join(const AttnArgs& a, int64_t items, hipStream_t s) {
    attn_decode_join_kernel<DP><<<dim3((unsigned)items), dim3(256), 0, s>>>(a, a.shares);
    return hipGetLastError();
}

template <int DP>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    const int64_t items = (int64_t)a.ntiles * a.K;
    const int64_t groups = a.nsplit > 1 ? a.shares : items;
    const int64_t grid = groups + a.clear + append_blocks(a, 8);
    if (grid > kMaxGroups || items > kMaxGroups) return hipErrorInvalidConfiguration;
    if (a.nsplit > 1)
        attn_decode_kernel<DP, true><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a, (int)groups);
    else
        attn_decode_kernel<DP, false><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a, (int)groups);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.nsplit == 1) return e;
    return join<DP>(a, items, s);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_decode_join(const AttnArgs& a, hipStream_t s) {
    const int64_t items = (int64_t)a.ntiles * a.K;
    return a.D <= 64 ? attn::join<64>(a, items, s) : attn::join<128>(a, items, s);
}

hipError_t launch_attn_decode_bf16(const AttnArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch<64>(a, s) : attn::launch<128>(a, s);
}

}  // namespace e2ttt
