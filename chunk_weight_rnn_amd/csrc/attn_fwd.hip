// Causal grouped-head attention, bf16 MFMA forward: packed sequences, and new
// tokens over a paged cache.
//
//   s_ij = scale <q_i, k_j>,   out_i = sum_j exp(s_ij - lse_i) v_j
//
// One pass over the keys with the running maximum m and sum l of the softmax:
// a key tile's scores S^T = K Q^T leave the MFMA with a query per lane, so the
// maximum, the exponentials and the rescaling need no exchange beyond the two
// lane halves, and P^T, packed to bf16, is the second operand of
// O^T += V^T P^T as it stands (attn_common.h).  V^T comes from the row-major
// tile by the transpose read.
//
// A workgroup is 4 waves of 32 rows each over shared tiles of 64 keys, two
// stages deep; two workgroups share a compute unit, so that one's softmax
// (VALU) runs beside the other's products.
//
// 16 heads of 128, a sequence of 16K under a window of 2K: 294 us a call, 877
// Tflop/s of the 1340 that a large library product reaches; 16 packed prompts of up
// to 2K over 4 key heads, 103 us, 673.  (Another card ran both a tenth slower.)  The
// matrix pipe is busy 43 % of the time: what bounds
// the kernel is the softmax's vector instructions (an exponential, a fused
// multiply-add and half a pack per score), which run beside the products only in
// part.  Tried and slower: products of one tile beside the softmax of the one
// before it in one wave (4 to 8 %: the third stage of keys costs registers that
// the reads ahead need), and tiles of 32 keys with three waves per SIMD (5 %).
#include "attn_common.h"

namespace e2ttt {
namespace attn {
namespace {

constexpr int BM = kFwdRows;  // 4 waves x 32
constexpr int BN = 64;   // keys of a tile

// The running maximum is only raised when a row exceeds it by this many
// powers of two: sums up to 2^8 times larger lose nothing in fp32, and most
// tiles skip the rescaling of the outputs.
constexpr float kLazy = 8.f;

// A wave's part of a tile copy: BN / 4 rows, 1 KiB (1024 / (2 DP) rows) per
// instruction.
template <int DP>
struct CopyPlan {
    static constexpr int RPI = 512 / DP;       // rows per instruction
    static constexpr int NI = (BN / 4) / RPI;  // instructions per wave and tensor
    static constexpr int CH = DP / 8;          // chunks per row
};

template <int DP, bool PAGED, bool SPLIT>
__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(AttnArgs a) {
    constexpr int TILE = BN * DP * 2;
    constexpr int KS = DP / 16, DT = DP / 32;
    using P = CopyPlan<DP>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2][2][TILE];  // [stage][K, V]

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 5, col = lane & 31;
    int b = blockIdx.x;
    // blocks past the tiles write the rows outside every sequence, and the new
    // tokens into their slots
    if (const int past = b - a.ntiles * a.nsplit * a.K; past >= 0) {
        if (past < a.clear) clear_block<__bf16>(a, past);
        else if constexpr (PAGED) append_block<__bf16>(a, past - a.clear);
        return;
    }
    const int kvh = b % a.K;
    b /= a.K;
    const int split = SPLIT ? b % a.nsplit : 0;
    const int t = SPLIT ? b / a.nsplit : b;
    Item it;
    const int G = a.G;
    // new tokens all see their whole cache, and split tiles are short: in order
    // (8 chunks of 256 tokens over a window of 2048: 61 us, by work 75 us);
    // whole tiles by work (16 packed prompts up to 2048: 122 us in order, 103 us)
    const int cap = PAGED || SPLIT ? kInOrder : row_cap(a.window, G, BM);
    if (!find_item(a.cu, a.S, (int)a.N, t, cap, [&](int n) { return (n * G + BM - 1) / BM; }, it)) return;
    const int r0 = it.tile * BM;
    const int rows = it.n * G;
    int kept = 0;
    if constexpr (PAGED) {
        kept = kept_tokens(a.pg, it.seq, it.n);
    }
    const int first = kept + div_group(r0, G, a.gmagic);                                            // position of the tile's first row
    const int last = kept + div_group(r0 + BM < rows ? r0 + BM - 1 : rows - 1, G, a.gmagic);  // and of its last
    const int lo = a.window > 0 && first - a.window + 1 > 0 ? (first - a.window + 1) & ~(BN - 1) : 0;
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
    {
        const __bf16* qp = (const __bf16*)a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 8 * chunk_of(s, g);
            bf16x8 z = {};
            qf[s] = live && d < a.D ? *(const bf16x8*)(qp + d) : z;
        }
    }

    const char* ksrc = (const char*)a.k + 2 * (it.tok0 * a.k_tok + kvh * a.k_head);
    const char* vsrc = (const char*)a.v + 2 * (it.tok0 * a.v_tok + kvh * a.v_head);
    // copy offsets: row (within this wave's quarter) and chunk of this lane
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

    PageCopy<DP, P::NI, BN> pc;
    const int* table = nullptr;
    if constexpr (PAGED) {
        pc.init(a, kvh, it.tok0, kept, 16 * wave);
        pc.begin = a.window > 0 ? first - a.window + 1 : 0;
        pc.end = last + 1;
        table = a.pg.table + (int64_t)it.seq * a.pg.wide;
    }
    int page[P::NI];  // paged: the next tile's page indices, loaded a tile ahead
    auto load_pages = [&](int j) {
        if constexpr (PAGED) pc.load_pages(a, table, lo + j * BN, page);
    };
    auto copy_tile = [&](int j, int stage) {
        const unsigned dst = base + stage * (2 * TILE);
        const int p0 = lo + j * BN;
        if constexpr (PAGED) {
            pc.copy(a, p0, dst, dst + TILE, [&](int i) { return page[i]; });
        } else {
            const int left = last + 1 - p0 < BN ? last + 1 - p0 : BN;  // rows of the tile that exist
            const u32x4 kr = buffer_rsrc(ksrc + (int64_t)p0 * a.k_tok * 2, (int)((left - 1) * a.k_tok * 2) + 2 * a.D);
            const u32x4 vr = buffer_rsrc(vsrc + (int64_t)p0 * a.v_tok * 2, (int)((left - 1) * a.v_tok * 2) + 2 * a.D);
#pragma unroll
            for (int i = 0; i < P::NI; ++i) {
                copy16(kr, dst + 1024 * i, koff[i]);
                copy16(vr, dst + TILE + 1024 * i, voff[i]);
            }
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
        copy_tile(j0, 0);
        load_pages(j0 + 1);
    }
    for (int j = j0; j < j1; ++j) {
        const int stage = (j - j0) & 1;
        wait_vm<0>();
        barrier_lds();
        if (j + 1 < j1) {
            copy_tile(j + 1, stage ^ 1);
            load_pages(j + 2);
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
            const int end = lo + j1 * BN < wlast + 1 ? lo + j1 * BN : wlast + 1;
            const float mu = m == neg_inf() ? 0.f : m;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[dt] = f32x16{};
            const char* qp = (const char*)a.q + 2 * (qtok * a.q_tok + (int64_t)head * a.q_head);
#pragma unroll 1
            for (int p = lo + j0 * BN; p < end; ++p) {
                const char *kp, *vp;
                if constexpr (PAGED) {
                    kp = pc.template row<false>(a, table, p);
                    vp = pc.template row<true>(a, table, p);
                } else {
                    kp = ksrc + (int64_t)p * a.k_tok * 2;
                    vp = vsrc + (int64_t)p * a.v_tok * 2;
                }
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(dot_rows<DP>(kp, qp, a.D, lane), a.sl2, -mu));
                add_row<DP>(acc, vp, p > qpos || p <= qlow ? 0.f : to_bf16(x), a.D, lane);
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
    if (a.lse && g == 0) a.lse[qtok * a.H + head] = l > 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : (l == 0.f ? neg_inf() : l);
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

// Joins the partial results of a split call,
//   out = sum_i 2^(pl_i - m) po_i / sum_i 2^(pl_i - m),
// half a wave per (token, head) with four values per lane; lane i of the half
// holds the weight of key range i (at most 32).
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    typedef T out4 __attribute__((ext_vector_type(4)));
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t NH = a.N * a.H;
    const int lane = threadIdx.x & 63, g = lane >> 5, i = lane & 31, d = 4 * i;
    // a token outside every sequence has no partial results (and its output already)
    const int tok = (int)(r / a.H);
    const bool live = r < NH && tok >= clamped(a.cu[0], (int)a.N) && tok < clamped(a.cu[a.S], (int)a.N);
    const bool in = live && d < a.D;
    const float x = live && i < a.nsplit ? a.pl[i * NH + r] : neg_inf();
    // the partial rows come beside the weights; those of weight 0 are not used
    f32x4 v[8], o = {};
    auto load = [&](int s0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f32x4 z = {};
            v[e] = in && s0 + e < a.nsplit ? *(const f32x4*)(a.po + ((s0 + e) * NH + r) * a.D + d) : z;
        }
    };
    load(0);
    float m = x;
#pragma unroll
    for (int k = 16; k; k >>= 1) m = max_or_nan(m, __shfl_xor(m, k));
    const float f = x == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(x - m);
    float w = f;
#pragma unroll
    for (int k = 16; k; k >>= 1) w += __shfl_xor(w, k);
    for (int s0 = 0; s0 < a.nsplit; s0 += 8) {
        if (s0 > 0) load(s0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float fe = __shfl(f, 32 * g + ((s0 + e) & 31));
            if (s0 + e < a.nsplit && fe != 0.f) o += v[e] * fe;
        }
    }
    const float inv = w > 0.f ? 1.f / w : w;
    if (in) {
        out4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (T)(o[e] * inv);
        *(out4*)((T*)a.out + r * a.D + d) = y;
    }
    if (live && a.lse && i == 0) a.lse[r] = w == 0.f ? neg_inf() : (m + __builtin_amdgcn_logf(w)) * kLn2;
}

template <int DP>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    const bool paged = a.pg.kc != nullptr;
    const int64_t grid = (int64_t)a.ntiles * a.K * a.nsplit + a.clear + (paged ? append_blocks(a, 8) : 0);
    if (grid == 0) return hipSuccess;
    if (grid > kMaxGroups) return hipErrorInvalidConfiguration;
    const dim3 gr((unsigned)grid), bl(256);
    if (paged && a.nsplit > 1)
        attn_fwd_kernel<DP, true, true><<<gr, bl, 0, s>>>(a);
    else if (paged)
        attn_fwd_kernel<DP, true, false><<<gr, bl, 0, s>>>(a);
    else if (a.nsplit > 1)
        attn_fwd_kernel<DP, false, true><<<gr, bl, 0, s>>>(a);
    else
        attn_fwd_kernel<DP, false, false><<<gr, bl, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_fwd_bf16(const AttnArgs& a, hipStream_t s) {
    return a.D <= 64 ? attn::launch<64>(a, s) : attn::launch<128>(a, s);
}

hipError_t launch_attn_join(const AttnArgs& a, bool f32, hipStream_t s) {
    const int64_t grid = (a.N * a.H + 7) / 8;
    if (grid == 0) return hipSuccess;
    if (grid > kMaxGroups) return hipErrorInvalidConfiguration;
    if (f32)
        attn::attn_join_kernel<float><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a);
    else
        attn::attn_join_kernel<__bf16><<<dim3((unsigned)grid), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace e2ttt
