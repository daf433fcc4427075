// Shared by the attention kernels (attn_fwd.hip, attn_decode.hip,
// attn_bwd.hip, attn_f32.hip): the work items of packed sequences, and the LDS tile
// layout of the bf16 MFMA kernels.
//
// A row is one (token, query head) pair.  The G = heads / kv_heads query
// heads that share a key head are packed into the rows of one tile, token
// major: row r of a sequence's key head is token r / G, head r % G of its
// group.  So a key/value tile that was staged once serves the whole group, in
// the backward the sums over a group are ordinary sums over rows, and a single
// new token still fills as many rows as its group has heads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "layer_internal.h"

namespace e2ttt {
namespace attn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4_t;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Value of the lane that holds the same column in the other half (lane ^ 32).
__device__ __forceinline__ float other_half(float x, int lane) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, lane < 32 ? r[1] : r[0]);
}

// Row r's token, r / G (the host bounds r G below 2^32).
__device__ __forceinline__ int div_group(int r, int G, unsigned magic) {
    return G == 1 ? r : (int)__umulhi((unsigned)r, magic);
}

template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        static_for<N, I + 1>(f);
    }
}

// ------------------------------------------------------------- work items
// A sequence of n tokens has a number of tiles, of rows or of keys, whose work
// grows with their index (causal: a later row sees more keys) up to a cap (the
// window).  The t-th workgroup takes the t-th tile in order of falling work
// over all sequences, in kClasses steps: a workgroup with much work that starts
// last would leave the rest of the chip idle.  Every wave searches for itself,
// from the offsets in memory (clamped, so that whatever they hold no address
// leaves the tensors); with more than 64 sequences there are many tiles of
// each kind, and they are taken sequence by sequence; so they are with cap = 0,
// where work is level and neighbours had better share their keys in the cache.
// False past the last tile.
struct Item {
    int seq, tok0, n;  // sequence, its first token, its length
    int tile, tiles;   // tile within the sequence, tiles of the sequence
};
constexpr int kClasses = 16;

__device__ __forceinline__ int clamped(int x, int hi) { return x < 0 ? 0 : (x > hi ? hi : x); }

// Inclusive sum (or maximum, x >= 0) over the lanes up to this one.
template <bool MAX>
__device__ __forceinline__ int wave_scan(int x) {
#define E2TTT_STEP(ctrl, rows)                                                     \
    {                                                                              \
        const int y = __builtin_amdgcn_update_dpp(0, x, ctrl, rows, 0xf, false);   \
        x = MAX ? (x > y ? x : y) : x + y;                                         \
    }
    E2TTT_STEP(0x111, 0xf)  // row_shr:1, 2, 4, 8 within 16 lanes
    E2TTT_STEP(0x112, 0xf)
    E2TTT_STEP(0x114, 0xf)
    E2TTT_STEP(0x118, 0xf)
    E2TTT_STEP(0x142, 0xa)  // row_bcast:15, row_bcast:31
    E2TTT_STEP(0x143, 0xc)
#undef E2TTT_STEP
    return x;
}
__device__ __forceinline__ int last_lane(int x) { return __builtin_amdgcn_readlane(x, 63); }

// Tiles of BM rows from which on the window keeps the work the same.
__device__ __forceinline__ int row_cap(int window, int G, int BM) {
    const int64_t c = (int64_t)window * G / BM + 1;
    return window == 0 || c > 0x7fffffff ? 0x7fffffff : (int)c;
}

constexpr int kInOrder = 0;

template <class F>
__device__ __forceinline__ bool find_item(const int* __restrict__ cu, int S, int N, int t, int cap, F&& tiles_of,
                                          Item& it) {
    const int lane = threadIdx.x & 63;
    auto load = [&](int s, int& a, int& n, int& m) {
        a = n = m = 0;
        if (s < S) {
            a = clamped(cu[s], N);
            n = clamped(cu[s + 1], N) - a;
            n = n > 0 ? n : 0;
            m = tiles_of(n);
        }
    };
    auto take = [&](int s0, int l, int a, int n, int m) {
        it.seq = s0 + l;
        it.tok0 = __builtin_amdgcn_readlane(a, l);
        it.n = __builtin_amdgcn_readlane(n, l);
        it.tiles = __builtin_amdgcn_readlane(m, l);
    };
    int a, n, m;
    if (S <= 64 && cap > 0) {
        load(lane, a, n, m);
        const int most = last_lane(wave_scan<true>(m));
        const int step = ((most < cap ? most : cap) + kClasses - 1) / kClasses;
        for (int c = kClasses - 1; c >= 0; --c) {
            const int lo = c * step;
            int k = m > lo ? m - lo : 0;
            if (c < kClasses - 1 && k > step) k = step;
            const int incl = wave_scan<false>(k);
            const unsigned long long past = __ballot(incl > t);
            if (past) {
                const int l = __builtin_ctzll(past);
                take(0, l, a, n, m);
                it.tile = lo + __builtin_amdgcn_readlane(incl, l) - 1 - t;
                return true;
            }
            t -= last_lane(incl);
        }
        return false;
    }
    for (int s0 = 0; s0 < S; s0 += 64) {
        load(s0 + lane, a, n, m);
        const int incl = wave_scan<false>(m);
        const unsigned long long past = __ballot(incl > t);
        if (past) {
            const int l = __builtin_ctzll(past);
            take(s0, l, a, n, m);
            it.tile = __builtin_amdgcn_readlane(incl, l) - 1 - t;
            return true;
        }
        t -= last_lane(incl);
    }
    return false;
}

// Block b of `blocks`: the rows of tokens outside every sequence, which see
// nothing, in a tensor of `bytes` per token; `what` in every four of them.
__device__ __forceinline__ void fill_outside(const int* __restrict__ cu, int S, int64_t N, void* p, int64_t bytes,
                                             unsigned what, int b, int blocks) {
    const int64_t lo = clamped(cu[0], (int)N), end = clamped(cu[S], (int)N), hi = end > lo ? end : lo;
    const int64_t words = bytes / 4, count = (lo + N - hi) * words, skip = (hi - lo) * words;
    unsigned* w = (unsigned*)p;
    if (words % 4 == 0 && (uintptr_t)p % 16 == 0) {
        for (int64_t i = ((int64_t)b * 256 + threadIdx.x) * 4; i < count; i += (int64_t)blocks * 1024)
            *(u32x4*)(w + (i < lo * words ? i : i + skip)) = u32x4{what, what, what, what};
        return;
    }
    for (int64_t i = (int64_t)b * 256 + threadIdx.x; i < count; i += (int64_t)blocks * 256)
        w[i < lo * words ? i : i + skip] = what;
}

// Outputs of the forward there: out 0, lse the log of an empty sum.
template <typename T>
__device__ __forceinline__ void clear_block(const AttnArgs& a, int b) {
    fill_outside(a.cu, a.S, a.N, a.out, (int64_t)a.H * a.D * sizeof(T), 0, b, a.clear);
    if (a.lse) fill_outside(a.cu, a.S, a.N, a.lse, (int64_t)a.H * 4, 0xff800000u, b, a.clear);
}

// Tokens a sequence has in the cache, clamped to what its page table holds.
__device__ __forceinline__ int kept_tokens(const PagedKV& pg, int seq, int n) {
    const int64_t room = ((int64_t)pg.wide << pg.shift) - n;
    return clamped(pg.cached[seq], room > 0 ? (int)room : 0);
}

// Writes new tokens' keys and values into their slots: block b of
// append_blocks, one 16-byte chunk of k and of v per thread.  Nothing else in
// the call reads these slots: positions >= cached come from k and v.
template <typename T>
__device__ __forceinline__ void append_block(const AttnArgs& a, int b) {
    constexpr int E = 16 / sizeof(T);
    const int64_t u = (int64_t)b * 256 + threadIdx.x;
    const int ch = a.D / E;
    const int64_t nk = u / ch;
    const int64_t n = nk / a.K;
    if (n >= a.N) return;
    const int c = (int)(u - nk * ch) * E, kvh = (int)(nk - n * a.K);
    int lo = 0, hi = a.S;  // the last sequence that starts at or before token n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= n) lo = mid;
        else hi = mid;
    }
    const int t0 = clamped(a.cu[lo], (int)a.N), count = clamped(a.cu[lo + 1], (int)a.N) - t0;
    const int i = (int)n - t0;
    if (i < 0 || i >= count) return;
    const int64_t pos = (int64_t)kept_tokens(a.pg, lo, count) + i;
    if ((pos >> a.pg.shift) >= a.pg.wide) return;
    const int page = a.pg.table[(int64_t)lo * a.pg.wide + (pos >> a.pg.shift)];
    if ((unsigned)page >= (unsigned)a.pg.pages) return;
    const int64_t slot = pos & (((int64_t)1 << a.pg.shift) - 1);
    const u32x4 kx = *(const u32x4*)((const T*)a.k + n * a.k_tok + kvh * a.k_head + c);
    const u32x4 vx = *(const u32x4*)((const T*)a.v + n * a.v_tok + kvh * a.v_head + c);
    *(u32x4*)((T*)a.pg.kc + page * a.pg.k_page + kvh * a.pg.k_head + slot * a.pg.k_slot + c) = kx;
    *(u32x4*)((T*)a.pg.vc + page * a.pg.v_page + kvh * a.pg.v_head + slot * a.pg.v_slot + c) = vx;
}

// -------------------------------------------------------------- LDS tiles
// A bf16 tile holds rows of DP values (DP = 64 or 128, head dims below it
// filled with zeros), 2 DP bytes each, with 16-byte chunk c of row t at
// physical chunk c ^ swz(t).  Two reads have to be free of bank conflicts (64
// four-byte banks, i.e. 16 chunks side by side):
//  * row fragments, ds_read_b128: lanes 8a .. 8a+7 and 32+8a .. 32+8a+7 are
//    served together, eight consecutive rows at a chunk and at the same chunk
//    with bit 1 flipped (chunk_of), which the swizzle puts on 16 different
//    chunk columns;
//  * transpose fragments, ds_read_b64_tr_b16: lanes 0..31 together, four
//    consecutive rows at four aligned chunks; rows r .. r+3 land on different
//    groups of four chunk columns.
template <int DP>
__device__ __forceinline__ int swz(int t) {
    if constexpr (DP == 128) return ((t & 3) << 2) | ((t >> 2) & 3);
    else return (((t >> 1) & 1) << 2) | ((t >> 2) & 3);
}

// Chunk of the head dimension that lane half g holds at k-step s of a
// 32x32x16 product over it.  Any order does, if both operands follow it.
__device__ __forceinline__ constexpr int chunk_of(int s, int g) { return ((s >> 1) << 2) | (g << 1) | (s & 1); }

// Fragments are addressed by one register each, the offset of the stage's tile
// included, from which every chunk is an exclusive or away: kept per chunk, the
// addresses would take a dozen registers that the accumulators need.
//
// Row fragment, k-step s: operand row t.
template <int DP>
__device__ __forceinline__ unsigned row_base(int t, int g) {
    return (unsigned)(t * (2 * DP) + 16 * (chunk_of(0, g) ^ swz<DP>(t)));
}
__device__ __forceinline__ bf16x8 row_frag(const unsigned char* lds, unsigned rb, int s) {
    return *(const bf16x8*)(lds + (rb ^ (16 * chunk_of(s, 0))));
}

// Transpose fragment dt, 16 tile rows from `lds` on: operand row = head-dim
// column 32 dt + lane % 32, operand k 0..3 = tile rows 4 (lane / 32) + {0..3},
// k 4..7 the same + 8.  This is the row order in which a 32x32 accumulator
// holds its rows, so an accumulator packed to bf16 is the other operand
// without any exchange.  (Eight rows on flip bit 1 of the swizzle; sixteen rows
// on keep it.)
template <int DP>
__device__ __forceinline__ unsigned tr_base(int lane) {
    const int p = lane & 15, G = lane >> 4;
    const int r = 4 * (G >> 1) + (p >> 2);
    const int chunk = 2 * (G & 1) + ((p & 3) >> 1);
    return (unsigned)(r * (2 * DP) + 16 * (chunk ^ swz<DP>(r)) + 8 * (p & 1));
}
template <int DP>
__device__ __forceinline__ bf16x8 tr_frag(const unsigned char* lds, unsigned tb, int dt) {
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t*)(lds + (tb ^ (64 * dt))));
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t*)(lds + (tb ^ (64 * dt + 32)) + 16 * DP));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// N products with the fragments of each read AHEAD products before it, in this
// order.  (Left to itself the compiler, short of registers, reads every fragment
// into the same ones and waits for it.)
template <int N, int AHEAD, class R, class M>
__device__ __forceinline__ void read_ahead(R&& read, M&& product) {
    bf16x8 f[AHEAD];
    static_for<(AHEAD < N ? AHEAD : N)>([&](auto n) { f[n] = read(n); });
    static_for<N>([&](auto n) {
        product(n, f[n % AHEAD]);
        if constexpr (n + AHEAD < N) f[n % AHEAD] = read(std::integral_constant<int, n + AHEAD>{});
        __builtin_amdgcn_sched_barrier(0);
    });
}

// Largest value of one or two accumulators in this lane (NaN only if all are).
// The three-operand maximum is written out because fmaxf would first quiet
// each operand in an instruction of its own.  Every asm depends on an ordinary
// maximum of both accumulators, so that the compiler has placed the wait for
// the products before it.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float max_of(const f32x16& x, const f32x16& y) {
    const float m = fmaxf(x[0], y[0]);
    float a = max3(m, x[1], x[2]), b = max3(m, y[1], y[2]);
#pragma unroll
    for (int i = 3; i < 15; i += 2) {
        a = max3(a, x[i], x[i + 1]);
        b = max3(b, y[i], y[i + 1]);
    }
    return fmaxf(max3(a, x[15], y[15]), b);
}

// Row of a 32x32 accumulator element i in lane half g.
__device__ __forceinline__ constexpr int acc_row(int i, int g) { return 8 * (i >> 2) + 4 * g + (i & 3); }

// Half hs (elements 8 hs .. 8 hs + 7, 16 rows) of an accumulator as a bf16
// operand, rounded to nearest even.
__device__ __forceinline__ bf16x8 pack_half(const f32x16& x, int hs) {
    bf16x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (__bf16)x[8 * hs + e];
    return r;
}

static __device__ __align__(256) unsigned char zeros[512];  // read in place of rows outside a sequence

// ------------------------------------------- NaN and Inf in masked places
// A masked key has weight 0, but the matrix unit computes 0 * NaN: a NaN or Inf
// in a key or value would reach rows that do not see it, wherever both lie in
// one tile.  Rows outside a sequence and positions that no row of a tile sees
// are zeros in the LDS; what is left are the tiles on the edge of a mask.  So a
// wave that walked over such a tile looks at its sums, and if one of them is not
// finite, and only then, it computes its sums again, term by term from memory
// and without the masked terms.

// NaN if a value is not finite, else zero.
template <int DT, class V>
__device__ __forceinline__ float not_finite(const V (&acc)[DT]) {
    float t = 0.f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < (int)(sizeof(V) / 4); ++i) t = __builtin_fmaf(acc[dt][i], 0.f, t);
    return t;
}

// <row, mine>: mine is this lane's column's own row; each lane half takes half
// of the chunks.
template <int DP>
__device__ __forceinline__ float dot_rows(const char* row, const char* mine, int D, int lane) {
    float t = 0.f;
#pragma unroll 1
    for (int c = lane >> 5; c < D / 8; c += 2) {
        const bf16x8 x = *(const bf16x8*)(row + 16 * c), y = *(const bf16x8*)(mine + 16 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) t = __builtin_fmaf((float)x[e], (float)y[e], t);
    }
    return t + other_half(t, lane);
}

// acc += w row, where w is not zero.
template <int DP>
__device__ __forceinline__ void add_row(f32x16 (&acc)[DP / 32], const char* row, float w, int D, int lane) {
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * dt + 8 * j + 4 * (lane >> 5);
            if (w == 0.f || d >= D) continue;
            const bf16x4 x = *(const bf16x4*)(row + 2 * d);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[dt][4 * j + e] = __builtin_fmaf(w, (float)x[e], acc[dt][4 * j + e]);
            __builtin_amdgcn_sched_barrier(0);
        }
}

__device__ __forceinline__ float to_bf16(float x) { return (float)(__bf16)x; }

// ------------------------------------------------------- copies to the LDS
// dword 3 of a raw buffer resource (gfx9 family: 32-bit data format, no swizzle)
constexpr int RSRC_W3 = 0x00020000;
constexpr unsigned kOutside = 0x7fffff00u;  // a buffer offset past every resource here: reads zeros

__device__ __forceinline__ u32x4 buffer_rsrc(const void* base, int num_bytes) {
    const unsigned long long p = (unsigned long long)base;
    u32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((unsigned)p);
    r[1] = __builtin_amdgcn_readfirstlane((unsigned)(p >> 32) & 0xFFFFu);
    r[2] = __builtin_amdgcn_readfirstlane((unsigned)num_bytes);
    r[3] = RSRC_W3;
    return r;
}

// 16 bytes per lane from base + voff (zeros at or past the resource's end) to
// LDS byte lds + 16 lane.  No register is written; wait with wait_vm.
__device__ __forceinline__ void copy16(u32x4 rsrc, unsigned lds, unsigned voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

// The same from a 64-bit address per lane.
__device__ __forceinline__ void copy16_at(const void* p, unsigned lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p)
                 : "memory", "m0");
}

// 4 bytes per lane.
__device__ __forceinline__ void copy4_at(const void* p, unsigned lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p)
                 : "memory", "m0");
}

__device__ __forceinline__ unsigned lds_addr(const void* p) {
    return __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
    asm volatile("" ::: "memory");
}

// Waits for this wave's LDS accesses, not for its copies in flight.  A stage may
// be refilled only after it: the compiler does not know where a copy writes, so
// by itself it keeps a fragment's read before its product, not before the copy.
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
}

// Workgroup barrier after that wait.
__device__ __forceinline__ void barrier_lds() {
    wait_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Copies T consecutive positions of one (sequence, key head) to the LDS, from
// the cache's pages and, from position `fresh` on, from the new tokens; this
// wave its rows row0 + RPI i + crow (one instruction moves RPI rows).
//
// Positions start at multiples of T, so within a page the slot of a row is a
// constant of the lane (pages shorter than T) or a constant plus the tile's
// place in its page: a tile that lies in the cache as a whole costs no address
// arithmetic where it lies in one page, and else one 64-bit multiply-add per
// address.  The other tiles (a sequence's last, and the first under a window)
// take the general way, row by row.
template <int DP, int NI, int T>
struct PageCopy {
    static constexpr int RPI = 512 / DP, CH = DP / 8;
    const char *kc, *vc, *kn, *vn;  // this key head in page 0 and in the sequence's new tokens
    int fresh, begin, end;          // positions outside [begin, end) are read as zeros
    int row0;
    unsigned ko[NI], vo[NI];

    __device__ __forceinline__ void init(const AttnArgs& a, int kvh, int tok0, int kept, int row0_) {
        const int lane = threadIdx.x & 63, mask = (1 << a.pg.shift) - 1;
        row0 = row0_;
        kn = (const char*)a.k + 2 * (tok0 * a.k_tok + kvh * a.k_head);
        vn = (const char*)a.v + 2 * (tok0 * a.v_tok + kvh * a.v_head);
        kc = (const char*)a.pg.kc + 2 * kvh * a.pg.k_head;
        vc = (const char*)a.pg.vc + 2 * kvh * a.pg.v_head;
        fresh = a.pg.append ? kept : 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = row0 + RPI * i + lane / CH, c = (lane % CH) ^ swz<DP>(r);
            const bool in = 8 * c < a.D;
            ko[i] = in ? (unsigned)((r & mask) * a.pg.k_slot * 2 + 16 * c) : kOutside;
            vo[i] = in ? (unsigned)((r & mask) * a.pg.v_slot * 2 + 16 * c) : kOutside;
        }
    }
    // The page of position pos (-1: none that is read).
    __device__ __forceinline__ int page_of(const AttnArgs& a, const int* table, int pos) const {
        const int pi = pos >> a.pg.shift;
        return pos >= begin && pos < end && pos < fresh && pi < a.pg.wide ? table[pi] : -1;
    }
    // Pages of this lane's rows of the tile at p0; where it lies in one page, one
    // scalar load in page[0].
    __device__ __forceinline__ void load_pages(const AttnArgs& a, const int* table, int p0, int (&page)[NI]) const {
        if ((1 << a.pg.shift) >= T) {
            const int pi = __builtin_amdgcn_readfirstlane(p0 >> a.pg.shift);
            const int p = p0 < end && p0 < fresh && pi < a.pg.wide ? table[pi] : -1;
#pragma unroll
            for (int i = 0; i < NI; ++i) page[i] = p;
            return;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) page[i] = page_of(a, table, p0 + row0 + RPI * i + (int)(threadIdx.x & 63) / CH);
    }
    // The key or value of one position.
    template <bool V>
    __device__ __forceinline__ const char* row(const AttnArgs& a, const int* table, int pos) const {
        if (pos < begin || pos >= end) return (const char*)zeros;
        if (pos >= fresh) return (V ? vn : kn) + 2 * (pos - fresh) * (V ? a.v_tok : a.k_tok);
        const int p = page_of(a, table, pos);
        if ((unsigned)p >= (unsigned)a.pg.pages) return (const char*)zeros;
        const int64_t slot = pos & ((1 << a.pg.shift) - 1);
        return (V ? vc : kc) + 2 * (p * (V ? a.pg.v_page : a.pg.k_page) + slot * (V ? a.pg.v_slot : a.pg.k_slot));
    }
    // Keys and values from position p0 on; page(i): the page of this lane's row
    // of instruction i.
    template <class F>
    __device__ __forceinline__ void copy(const AttnArgs& a, int p0, unsigned kdst, unsigned vdst, F&& page) const {
        const int mask = (1 << a.pg.shift) - 1;
        if (p0 >= begin && p0 + T <= end && p0 + T <= fresh) {
            const char* kb = kc + (int64_t)(p0 & mask) * a.pg.k_slot * 2;
            const char* vb = vc + (int64_t)(p0 & mask) * a.pg.v_slot * 2;
            const unsigned kp = (unsigned)a.pg.k_page * 2, vp = (unsigned)a.pg.v_page * 2;
            if (mask + 1 >= T) {
                const unsigned p = (unsigned)__builtin_amdgcn_readfirstlane(page(0));
                const int size = p < (unsigned)a.pg.pages ? (int)kOutside : 0;
                const u32x4 kr = buffer_rsrc(kb + (uint64_t)p * kp, size), vr = buffer_rsrc(vb + (uint64_t)p * vp, size);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    copy16(kr, kdst + 1024 * i, ko[i]);
                    copy16(vr, vdst + 1024 * i, vo[i]);
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const unsigned p = (unsigned)page(i);
                const bool ok = p < (unsigned)a.pg.pages && ko[i] != kOutside;
                copy16_at(ok ? kb + ((uint64_t)p * kp + ko[i]) : (const char*)zeros, kdst + 1024 * i);
                copy16_at(ok ? vb + ((uint64_t)p * vp + vo[i]) : (const char*)zeros, vdst + 1024 * i);
            }
            return;
        }
        const int lane = threadIdx.x & 63;
#pragma unroll 1
        for (int i = 0; i < NI; ++i) {
            const int r = row0 + RPI * i + lane / CH, pos = p0 + r;
            const int64_t c = 16 * ((lane % CH) ^ swz<DP>(r));
            const int p = page(i);
            const char *kp = (const char*)zeros, *vp = (const char*)zeros;
            if (c < 2 * a.D && pos >= begin && pos < end) {
                if (pos >= fresh) {
                    kp = kn + 2 * (pos - fresh) * a.k_tok + c;
                    vp = vn + 2 * (pos - fresh) * a.v_tok + c;
                } else if ((unsigned)p < (unsigned)a.pg.pages) {
                    const int64_t slot = pos & mask;
                    kp = kc + 2 * (p * a.pg.k_page + slot * a.pg.k_slot) + c;
                    vp = vc + 2 * (p * a.pg.v_page + slot * a.pg.v_slot) + c;
                }
            }
            copy16_at(kp, kdst + 1024 * i);
            copy16_at(vp, vdst + 1024 * i);
        }
    }
};

// ------------------------------------------------------- partial results
__device__ __forceinline__ float max_or_nan(float x, float y) { return x != x ? x : (y != y ? y : fmaxf(x, y)); }
__device__ __forceinline__ float wave_max_or_nan(float x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x = max_or_nan(x, __shfl_xor(x, d));
    return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// Adds n partial rows, two values per lane, with lane i's weight f for row i;
// eight loads in flight, beside the loads that the weights come from.  Rows of
// weight 0 saw nothing, and what is read of them is not used.
template <class F>
__device__ __forceinline__ void join_rows(int n, float f, bool in, F&& row, float& o0, float& o1) {
    for (int i0 = 0; i0 < n; i0 += 8) {
        float2 v[8];
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = float2{0.f, 0.f};
            if (i0 + e < n && in) v[e] = *(const float2*)row(i0 + e);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = i0 + e < n ? __shfl(f, i0 + e) : 0.f;
            o0 = w[e] != 0.f ? __builtin_fmaf(w[e], v[e].x, o0) : o0;
            o1 = w[e] != 0.f ? __builtin_fmaf(w[e], v[e].y, o1) : o1;
        }
    }
}

// Blocks that append_block needs (none when nothing is appended).
inline int64_t append_blocks(const AttnArgs& a, int elems) {
    return a.pg.append ? (a.N * a.K * (a.D / elems) + 255) / 256 : 0;
}

}  // namespace attn
}  // namespace e2ttt
