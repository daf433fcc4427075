// Attention of few new tokens per sequence over a paged cache in 8 bits (plain
// decoding: one token each).
//
// The work is shared out as in attn_decode.hip: units of 128 keys of all items in
// one line, an equal stretch of it per workgroup, four waves that each stream their
// own 32 keys through LDS stages of their own.  A stage is half as large, so that where
// the keys are shared out two workgroups fit a compute unit: bound by HBM and by what a
// wave does with a unit, one after the other, which a second wave on the same SIMD fills
// (64 sequences at up to 16383 keys, 16 heads of 128 over 4, 520 MB: 149 us with one
// workgroup of four stages, 107 with two of two, and 5 each to write the new tokens and
// to join).  Without sharing a workgroup has four stages.  A wave needs the page of
// each of its keys for the copies, and the scale of each key and value, which come
// with them, a byte per lane (keys' in lanes 0..31, values' in lanes 32..63).
//
// The tiles stay in 8 bits in the LDS and are widened as operands.  A key row is one
// lane's, and the conversion takes its scale; a value operand holds eight keys per
// lane (transposing reads of 8-bit tiles), so the values' scales go into the
// probabilities instead, where a power of two changes no rounding.
#include "attn8.h"
#include "attn_decode.h"

namespace e2ttt {
namespace attn {
namespace {

// A tile holds 32 rows of DP bytes, 16-byte chunk c of row t at chunk c ^ swz8(t).
// Two reads have to be free of bank conflicts (64 four-byte banks):
//  * row fragments, 16 bytes: lanes 8a .. 8a+7 of both halves together, eight
//    consecutive rows at a chunk and, in the other half, at that chunk with its
//    highest bit flipped; the swizzle spreads rows of the same place in the 256
//    bytes over the other bits;
//  * transpose fragments, 8 bytes: lanes 0..31 together, rows {0..3, 8..11} (or 4
//    on) at two neighbouring chunks; the swizzle's higher bits spread them.
template <int DP>
__device__ __forceinline__ int swz8(int t) {
    if constexpr (DP == 128) return ((t >> 2) & 1) | (t & 2) | (((t >> 3) & 1) << 2);
    else return ((t >> 2) & 1) | (((t >> 3) & 1) << 1);
}

// 1 byte per lane to 4 bytes of the LDS.
__device__ __forceinline__ void copy1_at(const void* p, unsigned lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p)
                 : "memory", "m0");
}

template <int DP, bool SPLIT>
__global__ __launch_bounds__(256, SPLIT ? 2 : 1) void attn_decode8_kernel(AttnArgs a, int groups) {
    constexpr int NS = SPLIT ? 2 : 4;         // LDS stages of a wave
    constexpr int TILE = BW * DP;             // a wave's keys (or values) of a unit
    constexpr int CH = DP / 16, RPI = 64 / CH;  // chunks of a row, rows per copy instruction
    constexpr int NI = BW / RPI;
    constexpr int KP = DP / 32, DT = DP / 32;  // pairs of 16-wide steps over the head dimension
    constexpr int COPIES = 2 * NI + 2;         // of a unit: keys, values, scales, and pages later
    constexpr int STAGES = 8 * NS * TILE, AREA = kMergeFloats<DP> * 4 > STAGES ? kMergeFloats<DP> * 4 : STAGES;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[AREA];  // [wave][stage][K, V][TILE], then the merge area
    __shared__ float stat[4][2][BM];
    __shared__ __attribute__((aligned(256))) int pages[4][2 * NS][64];            // [wave][unit % 2 NS][key, twice]
    __shared__ __attribute__((aligned(256))) unsigned scales[4][NS][64];          // [wave][stage][keys', values']

    if ((int)blockIdx.x >= groups) {
        clear_block<__bf16>(a, blockIdx.x - groups);
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
    // this lane's places in a tile: its key's chunks; rows and chunk of a transposing read
    const unsigned rb = (unsigned)(col * DP), rs = (unsigned)(16 * ((CH / 2 * g) ^ swz8<DP>(col)));
    const int tp = lane & 15, tr = tp >> 1, trow = (tr < 4 ? tr : tr + 4) + 4 * g;
    const unsigned tb = (unsigned)(trow * DP + 16 * (((lane >> 4) & 1) ^ swz8<DP>(trow)) + 8 * (tp & 1));
    const int crow = lane / CH;
    const unsigned base = lds_addr(lds + wave * (2 * NS * TILE));
    const int mask = (1 << a.pg.shift) - 1;

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
        const int begin = a.window > 0 ? first - a.window + 1 : 0, end = last + 1;  // positions that a row sees
        const int64_t qtok = w.tok0 + tok;
        const int head = w.kvh * G + hg;

        bf16x8 qf[2 * KP];
        const __bf16* qp = (const __bf16*)a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
#pragma unroll
        for (int s = 0; s < 2 * KP; ++s) {
            const int d = 16 * ((s >> 1) + CH / 2 * g) + 8 * (s & 1);
            bf16x8 z = {};
            qf[s] = live && d < a.D ? *(const bf16x8*)(qp + d) : z;
        }
        const int* table = a.pg.table + (int64_t)w.seq * a.pg.wide;
        const unsigned char* kc = (const unsigned char*)a.pg.kc + w.kvh * a.pg.k_head;
        const unsigned char* vc = (const unsigned char*)a.pg.vc + w.kvh * a.pg.v_head;
        // Units begin at multiples of 32 keys: within a page a key's slot is its place
        // in the unit plus, where a page holds whole units, the unit's place in the page.
        int64_t ko[NI], vo[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = RPI * i + crow, c = (lane % CH) ^ swz8<DP>(r);
            const bool in = 16 * c < a.D;
            ko[i] = in ? (r & mask) * a.pg.k_slot + 16 * c : -1;
            vo[i] = (r & mask) * a.pg.v_slot + 16 * c;
        }

        // This wave's part of unit b, in two steps: the pages of its keys, and NS
        // units later the keys, values and scales.  Each is always the same number
        // of copies, which the waits below count.
        auto copy_pages = [&](int b) {
            const int pos = w.lo + b * UNIT + BW * wave + col, pi = pos >> a.pg.shift;
            const bool in = b < b1 && pos >= begin && pos < end && pi < a.pg.wide;
            copy4_at(in ? table + pi : &no_page, lds_addr(&pages[wave][b & (2 * NS - 1)][0]));
        };
        auto copy_part = [&](int b) {
            const int p0 = w.lo + b * UNIT + BW * wave, in_page = p0 & mask, stage = b & (NS - 1);
            const unsigned dst = base + stage * (2 * TILE);
            const int* pg = &pages[wave][b & (2 * NS - 1)][0];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int p = pg[RPI * i + crow];
                const bool ok = (unsigned)p < (unsigned)a.pg.pages && ko[i] >= 0;
                copy16_at(ok ? kc + (p * a.pg.k_page + in_page * a.pg.k_slot + ko[i]) : zeros, dst + 1024 * i);
                copy16_at(ok ? vc + (p * a.pg.v_page + in_page * a.pg.v_slot + vo[i]) : zeros, dst + TILE + 1024 * i);
            }
            const int p = pg[col];
            const int64_t at = (((int64_t)p * a.K + w.kvh) << a.pg.shift) + ((p0 + col) & mask);
            copy1_at((unsigned)p < (unsigned)a.pg.pages ? (g ? a.pg.vs : a.pg.ks) + at : zeros, lds_addr(&scales[wave][stage][0]));
        };

        f32x16 acc[DT] = {};
        float m = neg_inf(), l = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) copy_pages(b0 + i);
        wait_vm<0>();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (b0 + i < b1) copy_part(b0 + i);
            copy_pages(b0 + NS + i);
        }
        for (int b = b0; b < b1; ++b) {
            // unit b has come, and the pages of unit b + NS: what may be outstanding are
            // the units after it, with a copy of pages each
            static_assert(NS == 2 || NS == 4, "a wait for each number of units on their way");
            const int after = b1 - 1 - b;
            if (NS == 4 && after >= 3) wait_vm<3 * COPIES>();
            else if (NS == 4 && after == 2) wait_vm<2 * COPIES>();
            else if (after >= 1) wait_vm<COPIES>();
            else wait_vm<0>();
            const int stage = b & (NS - 1), p0 = w.lo + b * UNIT + BW * wave;
            if (p0 <= last) {
                const unsigned char *kt = lds + (wave * NS + stage) * (2 * TILE), *vt = kt + TILE;
                const unsigned* sl = scales[wave][stage];
                const float kscale = scale_bits(sl[col]);
                f32x16 sc = {};
#pragma unroll
                for (int s = 0; s < KP; ++s) {
                    const u32x4 x = *(const u32x4*)(kt + (rb + (rs ^ (16 * s))));
                    sc = mfma32(widen(x[0], x[1], kscale), qf[2 * s], sc);
                    sc = mfma32(widen(x[2], x[3], kscale), qf[2 * s + 1], sc);
                }
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
                for (int j = 0; j < 4; ++j) {
                    const u32x4 e = *(const u32x4*)(sl + 32 + 8 * j + 4 * g);  // of rows acc_row(4 j .. 4 j + 3, g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[4 * j + i], a.sl2, -mu));
                        l += x;
                        const unsigned b = e[i];
                        sc[4 * j + i] = b == 255 && x != 0.f ? __builtin_nanf("") : __builtin_ldexpf(x, (int)b - 127);
                    }
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const bf16x8 pf = pack_half(sc, s);
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_t*)(vt + ((tb ^ (32 * dt)) + s * (16 * DP))));
                        acc[dt] = mfma32(widen((unsigned)x[0], (unsigned)x[1], 1.f), pf, acc[dt]);
                    }
                }
            }
            if (b + NS < b1) {
                wait_lds();  // the stage has been read
                copy_part(b + NS);
                copy_pages(b + 2 * NS);
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
                    const Pos8 kp = position8<false>(a, table, w.kvh, p, begin, end);
                    const Pos8 vp = position8<true>(a, table, w.kvh, p, begin, end);
                    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot8(kp, qp, a.D, lane), a.sl2, -mu));
                    add8<DP>(acc, vp, p > qpos || p <= qlow ? 0.f : to_bf16(x), a.D, lane);
                }
            }
        }
        wait_lds();
        finish_item<DP, SPLIT>(a, w, acc, m, l, live, whole, 2 * blockIdx.x + (first_seg ? 0 : 1), (float*)lds, stat);
        __syncthreads();  // the area is the next item's stages
        u += b1 - b0;
        first_seg = false;
        if (!SPLIT) break;
    }
}

template <int DP>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    const int64_t items = (int64_t)a.ntiles * a.K;
    const int64_t groups = a.nsplit > 1 ? a.shares : items;
    const int64_t grid = groups + a.clear;
    if (grid > kMaxGroups || items > kMaxGroups) return hipErrorInvalidConfiguration;
    if (a.nsplit > 1)
        attn_decode8_kernel<DP, true><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a, (int)groups);
    else
        attn_decode8_kernel<DP, false><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a, (int)groups);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || a.nsplit == 1 ? e : launch_attn_decode_join(a, s);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_decode8(const AttnArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch<64>(a, s) : attn::launch<128>(a, s);
}

}  // namespace e2ttt
