// Gradients of the causal grouped-head attention, bf16 MFMA:
//
//   p_ij = exp(s_ij - lse_i),        delta_i = <dout_i, out_i>,
//   ds_ij = p_ij (<dout_i, v_j> - delta_i),
//   dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,
//   dq_i = scale sum_j ds_ij k_j.
//
// Two kernels, each with its sums in registers: attn_dq_kernel owns query rows
// and walks over keys (and computes delta for the other), attn_dkdv_kernel
// owns keys and walks over the rows of their whole group.  That is seven
// products instead of the five of a single kernel, but no sum passes through
// memory and none depends on the order of workgroups: a single kernel would
// add dq to HBM in fp32 from every key block.
//
// Scores are recomputed in the orientation in which p and ds leave the MFMA as
// the next product's operand (attn_common.h): S^T with a query per lane for
// dq, S with a key per lane for dk and dv.
//
// 12 packed sequences of up to 2K, 16 heads of 128 over 4: dq 103 us (three
// products, 744 Tflop/s), dk and dv 177 us (four, 577).  Bound by each wave's own
// chain: two waves per SIMD, the registers' limit, hide the exponentials, the
// packing and the LDS reads of the next operands only in part.
#include "attn_common.h"

namespace e2ttt {
namespace attn {
namespace {

constexpr int BM = 128;  // rows of a workgroup (dq): 4 waves x 32
constexpr int BN = 64;   // keys of a staged tile (dq)
constexpr int BK = 64;   // keys of a workgroup (dkdv)
constexpr int BR = 64;   // rows of a staged tile (dkdv)

template <int DP>
struct CopyPlan {
    static constexpr int RPI = 512 / DP;       // rows per copy instruction
    static constexpr int NI = (BN / 4) / RPI;  // instructions per wave and tensor
    static constexpr int CH = DP / 8;          // chunks per row
};

// Two accumulator columns' worth of output, d-major per lane: 4 consecutive
// values of the head dimension per store.
template <int DT>
__device__ __forceinline__ void store_row(__bf16* o, const f32x16 (&acc)[DT], float f, int g, int D) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * dt + 8 * j + 4 * g;
            if (d < D) {
                bf16x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = (__bf16)(acc[dt][4 * j + e] * f);
                *(bf16x4*)(o + d) = w;
            }
        }
}

// 128 rows per workgroup over tiles of 64 keys, as the forward.  delta is computed
// from dout and out where the row's operands are loaded.
template <int DP>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(AttnBwdArgs a) {
    constexpr int TILE = BN * DP * 2;
    constexpr int KS = DP / 16, DT = DP / 32;
    using P = CopyPlan<DP>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2][2][TILE];  // [stage][K, V]

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31, G = a.G;
    if (const int past = (int)(blockIdx.x + a.clear) - (int)gridDim.x; past >= 0) {  // no rows: outside every sequence
        fill_outside(a.cu, a.S, a.N, a.dq, (int64_t)a.H * a.D * 2, 0, past, a.clear);
        return;
    }
    const int kvh = blockIdx.x % a.K, t = blockIdx.x / a.K;
    Item it;
    if (!find_item(a.cu, a.S, (int)a.N, t, row_cap(a.window, G, BM), [&](int n) { return (n * G + BM - 1) / BM; }, it)) return;
    const int r0 = it.tile * BM;
    const int rows = it.n * G;
    const int first = div_group(r0, G, a.gmagic);
    const int last = div_group(r0 + BM < rows ? r0 + BM - 1 : rows - 1, G, a.gmagic);
    const int lo = a.window > 0 && first - a.window + 1 > 0 ? (first - a.window + 1) & ~(BN - 1) : 0;
    const int nb = (last - lo) / BN + 1;

    const int row = r0 + 32 * wave + col;
    const bool live = row < rows;
    const int tok = live ? div_group(row, G, a.gmagic) : 0, hg = live ? row - tok * G : 0;
    const int qpos = live ? tok : -1;
    const int qlow = a.window > 0 ? qpos - a.window : -1;
    const int64_t qtok = it.tok0 + tok;
    const int head = kvh * G + hg;
    const int64_t at = qtok * a.H + head;

    bf16x8 qf[KS], df[KS];
    float delta = 0.f;
    {
        const __bf16* qp = (const __bf16*)a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
        const __bf16* dp = (const __bf16*)a.dout + at * a.D;
        const __bf16* op = (const __bf16*)a.out + at * a.D;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 8 * chunk_of(s, g);
            const bool in = live && d < a.D;
            bf16x8 z = {};
            qf[s] = in ? *(const bf16x8*)(qp + d) : z;
            df[s] = in ? *(const bf16x8*)(dp + d) : z;
            const bf16x8 of = in ? *(const bf16x8*)(op + d) : z;
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)df[s][e], (float)of[e], delta);
        }
    }
    delta += other_half(delta, lane);
    const float lse2 = live ? a.lse[at] * kLog2e : 0.f;

    const char* ksrc = (const char*)a.k + 2 * (it.tok0 * a.k_tok + kvh * a.k_head);
    const char* vsrc = (const char*)a.v + 2 * (it.tok0 * a.v_tok + kvh * a.v_head);
    const int crow = lane / P::CH, cpc = lane % P::CH;
    unsigned koff[P::NI], voff[P::NI];
#pragma unroll
    for (int i = 0; i < P::NI; ++i) {
        const int r = 16 * wave + P::RPI * i + crow;
        const int c = cpc ^ swz<DP>(r);
        const bool in = 8 * c < a.D;
        koff[i] = in ? (unsigned)(r * a.k_tok * 2 + 16 * c) : kOutside;
        voff[i] = in ? (unsigned)(r * a.v_tok * 2 + 16 * c) : kOutside;
    }
    const unsigned base = lds_addr(&lds[0][0][0]) + wave * (TILE / 4);
    auto copy_tile = [&](int j, int stage) {
        const unsigned dst = base + stage * (2 * TILE);
        const int p0 = lo + j * BN;
        const int left = last + 1 - p0 < BN ? last + 1 - p0 : BN;
        const u32x4 kr = buffer_rsrc(ksrc + (int64_t)p0 * a.k_tok * 2, (int)((left - 1) * a.k_tok * 2) + 2 * a.D);
        const u32x4 vr = buffer_rsrc(vsrc + (int64_t)p0 * a.v_tok * 2, (int)((left - 1) * a.v_tok * 2) + 2 * a.D);
#pragma unroll
        for (int i = 0; i < P::NI; ++i) {
            copy16(kr, dst + 1024 * i, koff[i]);
            copy16(vr, dst + TILE + 1024 * i, voff[i]);
        }
    };
    const unsigned rb0 = row_base<DP>(col, g), tb0 = tr_base<DP>(lane);

    f32x16 acc[DT] = {};
    const int wr0 = r0 + 32 * wave;
    const int wfirst = div_group(wr0, G, a.gmagic);
    const int wlast = div_group(wr0 + 31 < rows ? wr0 + 31 : rows - 1, G, a.gmagic);
    const bool wlive = wr0 < rows;

    // whether this wave's rows see anything of tile j
    auto sees = [&](int j) {
        const int p0 = lo + j * BN;
        return wlive && p0 <= wlast && !(a.window > 0 && p0 + BN - 1 <= wfirst - a.window);
    };
    // sc = p (dp - minus) of half h of tile j, zero where masked
    f32x16 sc;
    auto gradients = [&](int j, int h, float minus) {
        const int p0 = lo + j * BN;
        const unsigned rb = rb0 + (j & 1) * (2 * TILE);
        f32x16 dp = {};
        sc = f32x16{};
        read_ahead<2 * KS, 4>([&](auto n) { return row_frag(lds[0][n % 2] + h * (64 * DP), rb, n / 2); },
                              [&](auto n, bf16x8 f) {
                                  if constexpr (n % 2 == 0) sc = mfma32(f, qf[n / 2], sc);
                                  else dp = mfma32(f, df[n / 2], dp);
                              });
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sc[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], a.sl2, -lse2)) * (dp[i] - minus);
        if (p0 + BN - 1 > wfirst || (a.window > 0 && p0 <= wlast - a.window) || wr0 + 32 > rows) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int p = p0 + 32 * h + acc_row(i, g);
                if (p > qpos || p <= qlow) sc[i] = 0.f;
            }
        }
    };

    copy_tile(0, 0);
    if (nb <= 2) {
        // Rows that see few keys: delta = sum_j p_ij dp_ij, from the same fp32
        // products.  <dout, out> takes out as it was rounded to bf16, an error
        // that matters where few keys leave out about as large as a value; over
        // more keys out shrinks, and the error with it.
        if (nb == 2) copy_tile(1, 1);
        wait_vm<0>();
        barrier_lds();
        delta = 0.f;
#pragma unroll 1
        for (int jh = 0; jh < 2 * nb; ++jh) {
            if (!sees(jh >> 1)) continue;
            gradients(jh >> 1, jh & 1, 0.f);
#pragma unroll
            for (int i = 0; i < 16; ++i) delta += sc[i];
        }
        delta += other_half(delta, lane);
    }
    for (int j = 0; j < nb; ++j) {
        wait_vm<0>();
        barrier_lds();
        if (j + 1 < nb) copy_tile(j + 1, (j + 1) & 1);
        if (!sees(j)) continue;
        const unsigned char* kt = lds[0][0];
        const unsigned tb = tb0 + (j & 1) * (2 * TILE);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            gradients(j, h, delta);
            const bf16x8 sf[2] = {pack_half(sc, 0), pack_half(sc, 1)};
            read_ahead<2 * DT, 4>([&](auto n) { return tr_frag<DP>(kt + (2 * h + n / DT) * (32 * DP), tb, n % DT); },
                                  [&](auto n, bf16x8 f) { acc[n % DT] = mfma32(f, sf[n / DT], acc[n % DT]); });
        }
    }
    // a wave on the edge of the mask whose sums are not finite (attn_common.h)
    if (wlive && (lo + nb * BN > wfirst + 1 || (a.window > 0 && lo <= wlast - a.window))) {
        const float bad = not_finite(acc);
        if (__any(bad != bad && lse2 == lse2 && delta == delta)) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[dt] = f32x16{};
            int ln = lane;  // opaque, so that nothing is shared with the loop above
            asm volatile("" : "+v"(ln));
            const char* qp = (const char*)a.q + 2 * (qtok * a.q_tok + (int64_t)head * a.q_head);
            const char* op = (const char*)a.dout + 2 * at * a.D;
#pragma unroll 1
            for (int p = lo; p <= wlast; ++p) {
                const char* kp = ksrc + (int64_t)p * a.k_tok * 2;
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_rows<DP>(kp, qp, a.D, ln), a.sl2, -lse2));
                const float y = x * (dot_rows<DP>(vsrc + (int64_t)p * a.v_tok * 2, op, a.D, ln) - delta);
                add_row<DP>(acc, kp, p > qpos || p <= qlow ? 0.f : to_bf16(y), a.D, ln);
            }
        }
    }
    if (!live) return;
    if (g == 0) {  // what the other kernel's accumulators start from
        a.stats[at] = -lse2 / a.sl2;
        a.stats[a.N * a.H + at] = -delta;
    }
    store_row<DT>((__bf16*)a.dq + at * a.D, acc, a.scale, g, a.D);
}

// 64 keys per workgroup, over tiles of 64 rows: wave (kw, rw) takes 32 keys and
// 32 rows of each tile, and the two partial sums of a key are added at the end, in
// order.  The sums and the key and value operands take 192 of a wave's 256
// registers, so fragments are read four products ahead (read_ahead): left to the
// compiler every product waits for its own read, 1.8 times the time.
template <int DP>
__global__ __launch_bounds__(256, 2) void attn_dkdv_kernel(AttnBwdArgs a) {
    constexpr int TILE = BR * DP * 2;
    constexpr int KS = DP / 16, DT = DP / 32;
    constexpr int RPI = 512 / DP, NI = 16 / RPI, CH = DP / 8;  // copy instructions per wave and tensor, 16 rows
    constexpr int OLD = DP + 4;                                // row stride of the final sums, floats
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2][2][TILE];  // [stage][Q, dout]
    __shared__ __attribute__((aligned(256))) float stat[2][2][BR];            // [stage][-lse / scale, -delta]
    __shared__ __attribute__((aligned(16))) unsigned offs[2][256][NI];   // [Q, dout]: copy offsets of a thread
    static_assert(BK * OLD * 4 <= 4 * TILE, "the final sums fit in the stages");

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kw = wave & 1, rw = wave >> 1;
    const int g = lane >> 5, col = lane & 31, G = a.G;
    if (const int past = (int)(blockIdx.x + a.clear) - (int)gridDim.x; past >= 0) {
        fill_outside(a.cu, a.S, a.N, a.dk, (int64_t)a.K * a.D * 2, 0, past, a.clear);
        fill_outside(a.cu, a.S, a.N, a.dv, (int64_t)a.K * a.D * 2, 0, past, a.clear);
        return;
    }
    const int kvh = blockIdx.x % a.K, t = blockIdx.x / a.K;
    Item it;
    if (!find_item(a.cu, a.S, (int)a.N, t, row_cap(a.window, 1, BK), [&](int n) { return (n + BK - 1) / BK; }, it)) return;
    const int k0 = (it.tiles - 1 - it.tile) * BK;  // the first keys of a sequence have the most rows
    const int rows = it.n * G;
    const int klast = k0 + BK < it.n ? k0 + BK - 1 : it.n - 1;
    const int rbeg = k0 * G / BR * BR;
    const int64_t re = a.window > 0 ? ((int64_t)klast + a.window) * G : rows;
    const int rend = re < rows ? (int)re : rows;  // rows that see some key of the block: [k0 G, rend)
    const int nb = (rend - rbeg + BR - 1) / BR;

    const int key = k0 + 32 * kw + col;
    const bool live = key < it.n;
    const int64_t ktok = it.tok0 + (live ? key : 0);
    // rows that see this lane's key: [rlo, rhi)
    const int rlo = live ? key * G : 0x7fffffff;
    const int64_t rh = a.window > 0 ? ((int64_t)key + a.window) * G : rows;
    const int rhi = rh < rows ? (int)rh : rows;

    bf16x8 kf[KS], vf[KS];
    {
        const __bf16* kp = (const __bf16*)a.k + ktok * a.k_tok + (int64_t)kvh * a.k_head;
        const __bf16* vp = (const __bf16*)a.v + ktok * a.v_tok + (int64_t)kvh * a.v_head;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 8 * chunk_of(s, g);
            const bool in = live && d < a.D;
            bf16x8 z = {};
            kf[s] = in ? *(const bf16x8*)(kp + d) : z;
            vf[s] = in ? *(const bf16x8*)(vp + d) : z;
        }
    }

    const int crow = 16 * wave + lane / CH, cpc = lane % CH;
    const unsigned base = lds_addr(&lds[0][0][0]) + wave * (16 * DP * 2);
    const unsigned sbase = lds_addr(&stat[0][0][0]);
    const char* qsrc = (const char*)a.q + 2 * (it.tok0 * a.q_tok + (int64_t)kvh * G * a.q_head);
    const int64_t first_row = (int64_t)it.tok0 * a.H + kvh * G;  // row 0 in [N][H] order
    const char* dsrc = (const char*)a.dout + 2 * first_row * a.D;
    // A group whose size divides the tile starts every tile on a token: a
    // lane's offsets are the same in all of them, and only the base moves.
    // Otherwise they come anew from the row number, and at 128 columns through
    // spilled registers, each of whose loads waits for the copies before it: 12
    // heads over 4 take 224 us for three quarters of the work of 16, which take 177.
    const bool steady = BR % G == 0 && a.q_head < (1 << 22) / G && a.q_tok < (1 << 30) / BR;
    // (They wait in the LDS: the accumulators leave no registers for them.)
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int rr = crow + RPI * i, tk = div_group(rr, G, a.gmagic), hg = rr - tk * G;
        const int c = cpc ^ swz<DP>(rr);
        const bool in = 8 * c < a.D && steady;
        offs[0][threadIdx.x][i] = in ? (unsigned)(2 * (tk * a.q_tok + hg * a.q_head) + 16 * c) : kOutside;
        offs[1][threadIdx.x][i] = in ? (unsigned)(2 * (tk * a.H + hg) * a.D + 16 * c) : kOutside;
    }
    auto copy_tile = [&](int j, int stage) {
        const unsigned dst = base + stage * (2 * TILE);
        const int t0 = rbeg + (nb - 1 - j) * BR;
        if (steady) {
            const int64_t tk = div_group(t0, G, a.gmagic);
            const u32x4 qr = buffer_rsrc(qsrc + 2 * tk * a.q_tok, (int)kOutside);
            const u32x4 dr = buffer_rsrc(dsrc + 2 * tk * a.H * a.D, (int)kOutside);
            if (t0 + BR <= rows) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    copy16(qr, dst + 1024 * i, offs[0][threadIdx.x][i]);
                    copy16(dr, dst + TILE + 1024 * i, offs[1][threadIdx.x][i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const bool in = t0 + crow + RPI * i < rows;
                    copy16(qr, dst + 1024 * i, in ? offs[0][threadIdx.x][i] : kOutside);
                    copy16(dr, dst + TILE + 1024 * i, in ? offs[1][threadIdx.x][i] : kOutside);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int rr = crow + RPI * i;
                const int r = t0 + rr, c = cpc ^ swz<DP>(rr);
                const char *qp = (const char*)zeros, *dp = (const char*)zeros;
                if (8 * c < a.D && r < rows) {
                    const int tk = div_group(r, G, a.gmagic), hg = r - tk * G;
                    qp = qsrc + 2 * (tk * a.q_tok + hg * a.q_head) + 16 * c;
                    dp = dsrc + 2 * ((int64_t)tk * a.H + hg) * a.D + 16 * c;
                }
                copy16_at(qp, dst + 1024 * i);
                copy16_at(dp, dst + TILE + 1024 * i);
            }
        }
        // the statistics of the tile's rows: 64 of them per wave, BR of each kind
        if (64 * wave < 2 * BR) {
            const int x = 64 * wave + lane, r = t0 + (x & (BR - 1));
            const int tk = div_group(r < rows ? r : 0, G, a.gmagic), hg = r < rows ? r - tk * G : 0;
            copy4_at(a.stats + (x < BR ? 0 : a.N * a.H) + first_row + (int64_t)tk * a.H + hg,
                     sbase + stage * (2 * BR * 4) + wave * 256);
        }
    };
    const unsigned rb0 = row_base<DP>(col, g) + rw * (64 * DP), tb0 = tr_base<DP>(lane) + rw * (64 * DP);

    f32x16 dk[DT] = {}, dv[DT] = {};
    const int wk0 = k0 + 32 * kw;  // this wave's keys
    const int wklast = wk0 + 31;
    const bool wlive = wk0 < it.n;

    // from the last rows back: the key blocks of a sequence that run at the same
    // time begin on the same tiles and find them in the L2 cache
    if (nb > 0) copy_tile(0, 0);
    for (int j = 0; j < nb; ++j) {
        const int stage = j & 1;
        wait_vm<0>();
        barrier_lds();
        if (j + 1 < nb) copy_tile(j + 1, stage ^ 1);
        const int p0 = rbeg + (nb - 1 - j) * BR + 32 * rw;
        if (!wlive || p0 + 31 < wk0 * G || p0 >= rows) continue;
        const unsigned char *qt = lds[0][0], *ot = lds[0][1];
        const unsigned rb = rb0 + stage * (2 * TILE), tb = tb0 + stage * (2 * TILE);
        const bool edge = p0 < wklast * G || p0 + 32 > rows || wklast >= it.n ||
                          (a.window > 0 && p0 + 32 > ((int64_t)wk0 + a.window) * G);
        const float* st = &stat[stage][0][32 * rw + 4 * g];
        // <q, k> - lse / scale and <dout, v> - delta: the accumulators start
        // from the rows' statistics
        f32x16 sc, dp;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const f32x4 ls = *(const f32x4*)(st + 8 * b), de = *(const f32x4*)(st + BR + 8 * b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc[4 * b + e] = ls[e];
                dp[4 * b + e] = de[e];
            }
        }
        read_ahead<2 * KS, 4>([&](auto n) { return row_frag(n % 2 ? ot : qt, rb, n / 2); },
                              [&](auto n, bf16x8 f) {
                                  if constexpr (n % 2 == 0) sc = mfma32(f, kf[n / 2], sc);
                                  else dp = mfma32(f, vf[n / 2], dp);
                              });
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sc[i] = __builtin_amdgcn_exp2f(sc[i] * a.sl2);
            dp[i] *= sc[i];
        }
        if (edge) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = p0 + acc_row(i, g);
                const bool out = r < rlo || r >= rhi;
                sc[i] = out ? 0.f : sc[i];
                dp[i] = out ? 0.f : dp[i];
            }
        }
        const bf16x8 pf[2] = {pack_half(sc, 0), pack_half(sc, 1)}, sf[2] = {pack_half(dp, 0), pack_half(dp, 1)};
        __builtin_amdgcn_sched_barrier(0);
        read_ahead<4 * DT, 4>([&](auto n) { return tr_frag<DP>((n % 2 ? qt : ot) + n / (2 * DT) * (32 * DP), tb, n / 2 % DT); },
                              [&](auto n, bf16x8 f) {
                                  constexpr int s = n / (2 * DT), dt = n / 2 % DT;
                                  if constexpr (n % 2 == 0) dv[dt] = mfma32(f, pf[s], dv[dt]);
                                  else dk[dt] = mfma32(f, sf[s], dk[dt]);
                              });
    }
    // Sums that are not finite (attn_common.h): every block has its keys' own
    // rows on the edge of the mask.  (Everything is computed and loaded anew
    // from an opaque lane number: what this path shared with the loop above
    // would cost that registers, and a spilled fragment there waits for every
    // copy in flight, as the copies of groups that do not divide a tile do.)
    if (wlive) {
        const float bad = not_finite(dk) + not_finite(dv);
        if (__any(bad != bad)) {
            int ln = threadIdx.x & 63;
            asm volatile("" : "+v"(ln));
            const int ky = k0 + 32 * kw + (ln & 31);
            const bool lv = ky < it.n;
            const int lo = lv ? ky * G : 0x7fffffff;
            const int64_t h64 = a.window > 0 ? ((int64_t)ky + a.window) * G : rows;
            const int hi = h64 < rows ? (int)h64 : rows;
            const char* kp = (const char*)a.k + 2 * ((it.tok0 + (lv ? ky : 0)) * a.k_tok + (int64_t)kvh * a.k_head);
            const char* vp = (const char*)a.v + 2 * ((it.tok0 + (lv ? ky : 0)) * a.v_tok + (int64_t)kvh * a.v_head);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) dk[dt] = dv[dt] = f32x16{};
#pragma unroll 1
            for (int r = rbeg; r < rend; ++r) {
                if (((r - rbeg) / 32) % 2 != rw) continue;
                const int tk = div_group(r, G, a.gmagic), hg = r - tk * G;
                const int64_t at = first_row + (int64_t)tk * a.H + hg;
                const char* qp = qsrc + 2 * (tk * a.q_tok + hg * a.q_head);
                const char* op = (const char*)a.dout + 2 * at * a.D;
                const float x = __builtin_amdgcn_exp2f((dot_rows<DP>(qp, kp, a.D, ln) + a.stats[at]) * a.sl2);
                const float y = x * (dot_rows<DP>(op, vp, a.D, ln) + a.stats[a.N * a.H + at]);
                const bool out = r < lo || r >= hi;
                add_row<DP>(dv, op, out ? 0.f : to_bf16(x), a.D, ln);
                add_row<DP>(dk, qp, out ? 0.f : to_bf16(y), a.D, ln);
            }
        }
    }
    float* area = (float*)&lds[0][0][0] + (32 * kw + col) * OLD + 4 * g;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        f32x16(&x)[DT] = which == 0 ? dv : dk;
        barrier_lds();  // the stages, or the sums before, have been read
        if (rw > 0) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(f32x4*)(area + 32 * dt + 8 * j) = f32x4{x[dt][4 * j], x[dt][4 * j + 1], x[dt][4 * j + 2], x[dt][4 * j + 3]};
        }
        barrier_lds();
        if (rw > 0) continue;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 y = *(const f32x4*)(area + 32 * dt + 8 * j);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[dt][4 * j + e] += y[e];
            }
        if (live) store_row<DT>((__bf16*)(which == 0 ? a.dv : a.dk) + (ktok * a.K + kvh) * a.D, x, which == 0 ? 1.f : a.scale, g, a.D);
    }
}

template <int DP>
hipError_t launch(const AttnBwdArgs& a, hipStream_t s) {
    const int64_t dq_grid = (a.N * a.G / BM + a.S) * a.K + a.clear, dkv_grid = (a.N / BK + a.S) * a.K + a.clear;
    if (dq_grid > kMaxGroups || dkv_grid > kMaxGroups) return hipErrorInvalidConfiguration;
    attn_dq_kernel<DP><<<dim3((unsigned)dq_grid), dim3(256), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attn_dkdv_kernel<DP><<<dim3((unsigned)dkv_grid), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_bwd_bf16(const AttnBwdArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch<64>(a, s) : attn::launch<128>(a, s);
}

}  // namespace e2ttt
