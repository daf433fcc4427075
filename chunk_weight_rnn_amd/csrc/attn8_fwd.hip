// Attention of chunks of new tokens over a paged cache in 8 bits.
//
// The tiles, the softmax and the products are those of attn_fwd.hip.  A tile of 64
// keys and values is read into registers, 16 bytes of a row at a time, a tile ahead
// of its use, widened to bf16 with its row's scale and written to the LDS once for
// the four waves, while the tile before it is multiplied: 32 conversions per wave
// and tile, where widening the operands of each wave would take 128.  Bound as
// attn_fwd.hip is, by the softmax beside the products (8 chunks of 256 over a window of
// 2048, 16 heads of 128 over 4: 48 us, 430 Tflop/s; with a bf16 cache 43).
#include "attn8.h"

namespace e2ttt {
namespace attn {
namespace {

constexpr int BM = kFwdRows;  // 4 waves x 32
constexpr int BN = 64;        // keys of a tile
constexpr float kLazy = 8.f;  // as in attn_fwd.hip

template <int DP, bool SPLIT>
__global__ __launch_bounds__(256, 2) void attn_fwd8_kernel(AttnArgs a) {
    constexpr int TILE = BN * DP * 2;
    constexpr int KS = DP / 16, DT = DP / 32;
    constexpr int CH = DP / 16, NI = BN * CH / 256, RPI = 256 / CH;  // a thread's rows of a tile: RPI i + crow
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2][2][TILE];  // [stage][K, V]

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31;
    int b = blockIdx.x;
    if (const int past = b - a.ntiles * a.nsplit * a.K; past >= 0) {
        clear_block<__bf16>(a, past);
        return;
    }
    const int kvh = b % a.K;
    b /= a.K;
    const int split = SPLIT ? b % a.nsplit : 0;
    const int t = SPLIT ? b / a.nsplit : b;
    Item it;
    const int G = a.G;
    if (!find_item(a.cu, a.S, (int)a.N, t, kInOrder, [&](int n) { return (n * G + BM - 1) / BM; }, it)) return;
    const int r0 = it.tile * BM;
    const int rows = it.n * G;
    const int kept = kept_tokens(a.pg, it.seq, it.n);
    const int first = kept + div_group(r0, G, a.gmagic);                                      // position of the tile's first row
    const int last = kept + div_group(r0 + BM < rows ? r0 + BM - 1 : rows - 1, G, a.gmagic);  // and of its last
    const int lo = a.window > 0 && first - a.window + 1 > 0 ? (first - a.window + 1) & ~(BN - 1) : 0;
    const int begin = a.window > 0 ? first - a.window + 1 : 0, end = last + 1;  // positions that a row sees
    const int nb = (last - lo) / BN + 1;
    int j0 = 0, j1 = nb;
    if (SPLIT) {
        const int per = (nb + a.nsplit - 1) / a.nsplit;
        j0 = split * per;
        j1 = j0 + per < nb ? j0 + per : nb;
    }

    // this lane's row
    const int row = r0 + 32 * wave + col;
    const bool live = row < rows;
    const int tok = live ? div_group(row, G, a.gmagic) : 0, hg = live ? row - tok * G : 0;
    const int qpos = live ? kept + tok : -1;
    const int qlow = a.window > 0 ? qpos - a.window : -1;  // keys at or below it are out of the window
    const int64_t qtok = it.tok0 + tok;
    const int head = kvh * G + hg;

    bf16x8 qf[KS];
    const __bf16* qp = (const __bf16*)a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int d = 8 * chunk_of(s, g);
        bf16x8 z = {};
        qf[s] = live && d < a.D ? *(const bf16x8*)(qp + d) : z;
    }

    // this thread's part of a tile, and where its 16 values go
    const int* table = a.pg.table + (int64_t)it.seq * a.pg.wide;
    const int crow = threadIdx.x / CH, cc = threadIdx.x % CH, mask = (1 << a.pg.shift) - 1;
    const bool in = 16 * cc < a.D;
    const unsigned char* kc = (const unsigned char*)a.pg.kc + kvh * a.pg.k_head + 16 * cc;
    const unsigned char* vc = (const unsigned char*)a.pg.vc + kvh * a.pg.v_head + 16 * cc;
    int page[NI];  // of the tile that is read next
    auto load_pages = [&](int j) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int pos = lo + j * BN + RPI * i + crow, pi = pos >> a.pg.shift;
            page[i] = j < j1 && pos >= begin && pos < end && pi < a.pg.wide ? table[pi] : -1;
        }
    };
    u32x4 kx[NI], vx[NI];
    unsigned ke[NI], ve[NI];
    auto read_tile = [&](int j) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int pos = lo + j * BN + RPI * i + crow, p = page[i];
            const int64_t slot = pos & mask;
            u32x4 z = {};
            kx[i] = vx[i] = z;
            ke[i] = ve[i] = 0;
            if ((unsigned)p < (unsigned)a.pg.pages && in) {
                kx[i] = *(const u32x4*)(kc + (p * a.pg.k_page + slot * a.pg.k_slot));
                vx[i] = *(const u32x4*)(vc + (p * a.pg.v_page + slot * a.pg.v_slot));
                const int64_t at = (((int64_t)p * a.K + kvh) << a.pg.shift) + slot;
                ke[i] = a.pg.ks[at];
                ve[i] = a.pg.vs[at];
            }
        }
    };
    auto write_tile = [&](int stage) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = RPI * i + crow, c0 = (2 * cc) ^ swz<DP>(r), c1 = (2 * cc + 1) ^ swz<DP>(r);
            unsigned char *kt = lds[stage][0] + r * (2 * DP), *vt = lds[stage][1] + r * (2 * DP);
            const float ks = scale_bits(ke[i]), vs = scale_bits(ve[i]);
            *(bf16x8*)(kt + 16 * c0) = widen(kx[i][0], kx[i][1], ks);
            *(bf16x8*)(kt + 16 * c1) = widen(kx[i][2], kx[i][3], ks);
            *(bf16x8*)(vt + 16 * c0) = widen(vx[i][0], vx[i][1], vs);
            *(bf16x8*)(vt + 16 * c1) = widen(vx[i][2], vx[i][3], vs);
        }
    };

    const unsigned rb0 = row_base<DP>(col, g), tb0 = tr_base<DP>(lane);

    f32x16 acc[DT] = {};
    float m = neg_inf(), l = 0.f;
    // rows of this wave: the positions that bound its masks
    const int wr0 = r0 + 32 * wave;
    const int wfirst = kept + div_group(wr0, G, a.gmagic);
    const int wlast = kept + div_group(wr0 + 31 < rows ? wr0 + 31 : rows - 1, G, a.gmagic);
    const bool wlive = wr0 < rows;

    if (j0 < j1) {
        load_pages(j0);
        read_tile(j0);
        load_pages(j0 + 1);
        write_tile(0);
        read_tile(j0 + 1);
        load_pages(j0 + 2);
    }
    for (int j = j0; j < j1; ++j) {
        const int stage = (j - j0) & 1;
        barrier_lds();  // the tile is written, and the other stage has been read
        if (j + 1 < j1) {
            write_tile(stage ^ 1);
            read_tile(j + 2);
            load_pages(j + 3);
        }
        const int p0 = lo + j * BN;
        if (!wlive || p0 > wlast || (a.window > 0 && p0 + BN - 1 <= wfirst - a.window)) continue;
        const unsigned char *kt = lds[0][0], *vt = lds[0][1];
        const unsigned rb = rb0 + stage * (2 * TILE), tb = tb0 + stage * (2 * TILE);
        f32x16 sc[2] = {};
        read_ahead<2 * KS, 4>([&](auto n) { return row_frag(kt + n % 2 * (64 * DP), rb, n / 2); },
                              [&](auto n, bf16x8 f) { sc[n % 2] = mfma32(f, qf[n / 2], sc[n % 2]); });
        if (p0 + BN - 1 > wfirst || (a.window > 0 && p0 <= wlast - a.window) || wr0 + 32 > rows) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int p = p0 + 32 * h + acc_row(i, g);
                    if (p > qpos || p <= qlow) sc[h][i] = neg_inf();
                }
        }
        float mx = max_of(sc[0], sc[1]);
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
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sc[h][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[h][i], a.sl2, -mu));
                sum += sc[h][i];
            }
        l += sum;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bf16x8 pf = pack_half(sc[s >> 1], s & 1);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
                acc[dt] = mfma32(tr_frag<DP>(vt + s * (32 * DP), tb, dt), pf, acc[dt]);
        }
    }

    l += other_half(l, lane);
    // a wave on the edge of the mask whose scores are fine and whose sums are not
    if (wlive && j0 < j1 && (lo + j1 * BN > wfirst + 1 || (a.window > 0 && lo + j0 * BN <= wlast - a.window))) {
        const float bad = not_finite(acc);
        if (__any(bad != bad && l == l)) {
            const int stop = lo + j1 * BN < wlast + 1 ? lo + j1 * BN : wlast + 1;
            const float mu = m == neg_inf() ? 0.f : m;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[dt] = f32x16{};
#pragma unroll 1
            for (int p = lo + j0 * BN; p < stop; ++p) {
                const Pos8 kp = position8<false>(a, table, kvh, p, begin, end), vp = position8<true>(a, table, kvh, p, begin, end);
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot8(kp, qp, a.D, lane), a.sl2, -mu));
                add8<DP>(acc, vp, p > qpos || p <= qlow ? 0.f : to_bf16(x), a.D, lane);
            }
        }
    }
    if (!live) return;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a row that sees nothing gives 0; NaN stays
    if (SPLIT) {
        const int64_t at = ((int64_t)split * a.N + qtok) * a.H + head;
        if (g == 0) a.pl[at] = l > 0.f ? m + __builtin_amdgcn_logf(l) : (l == 0.f ? neg_inf() : l);
        float* o = a.po + at * a.D;
        if (j0 < j1) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = 32 * dt + 8 * j + 4 * g;
                    if (d < a.D) {
                        f32x4 w;
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = acc[dt][4 * j + e] * inv;
                        *(f32x4*)(o + d) = w;
                    }
                }
        }
        return;
    }
    __bf16* o = (__bf16*)a.out + (qtok * a.H + head) * a.D;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * dt + 8 * j + 4 * g;
            if (d < a.D) {
                bf16x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = (__bf16)(acc[dt][4 * j + e] * inv);
                *(bf16x4*)(o + d) = w;
            }
        }
}

template <int DP>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    const int64_t grid = (int64_t)a.ntiles * a.K * a.nsplit + a.clear;
    if (grid == 0) return hipSuccess;
    if (grid > kMaxGroups) return hipErrorInvalidConfiguration;
    const dim3 gr((unsigned)grid), bl(256);
    if (a.nsplit > 1)
        attn_fwd8_kernel<DP, true><<<gr, bl, 0, s>>>(a);
    else
        attn_fwd8_kernel<DP, false><<<gr, bl, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_fwd8(const AttnArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch<64>(a, s) : attn::launch<128>(a, s);
}

}  // namespace e2ttt
