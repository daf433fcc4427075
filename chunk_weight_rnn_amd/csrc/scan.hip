// Gated linear recurrence of every channel over packed sequences, and its
// gradients:
//
//   h_t = a_t h_{t-1} + x_t,
//   g_t = dout_t + a_{t+1} g_{t+1},  dx_t = g_t,  da_t = g_t h_{t-1}.
//
// HBM bound: two operations per value read (one sequence of 16384 tokens, 2048 channels
// in bf16: 63 us, 3.2 TB/s; 8 of up to 2048 tokens with gates in fp32: 38 us, the
// gradients 46).  A stretch of tokens acts on the state that enters it as h -> P h + H,
// with P the product of its gates and H its result from zero, so that stretches can be
// read side by side.  A workgroup
// takes one tile, E2TTT_SCAN_TILE tokens of a slab of channels (one per lane), every
// wave R of them in registers, and reads it once:
//  * the waves exchange their (P, H) through the LDS, and the tile's is published;
//  * the state that enters the tile follows from those of the tiles before it: the
//    waves wait for the kLook nearest, the farthest of which has to have its end state
//    published, and all of them are folded in order;
//  * the tile's end state is published for the tiles after it, and each wave runs
//    its tokens a second time from registers, now from the right state: the outputs
//    are those of the recurrence itself, not of products and sums over the stretch.
// An end state is the fold of the one before it and the tile's (P, H) wherever it is
// computed, so that results do not depend on who was first.
//
// Workgroups take their tiles by a ticket, in the order of the sequences, so a tile
// waits only for tiles that were taken before it, by workgroups that run already and
// finish theirs in the order they took them, and words only grow, whatever the offsets
// hold: every wait ends.  (One that does not, because another call was given the same
// workspace meanwhile, is given up after seconds of looking, scan_wait.h, and its results
// are NaN.)  What is published is a word of 64 bits, stored
// and loaded as a whole past the caches of the compute dies, so nothing has to be flushed.
//
// The gradient goes the same way from the last tile to the first.  It needs
// the states again, which out holds rounded: they are computed once more from
// the saved states at the tiles' starts, which costs no more reading than out
// would (x in its place).
#include <type_traits>

#include "attn_common.h"
#include "scan_wait.h"

namespace e2ttt {
namespace {

using attn::clamped;
typedef unsigned long long u64;

constexpr int R = 16;                     // tokens of a wave
constexpr int NW = E2TTT_SCAN_TILE / R;   // waves of a workgroup
constexpr int TILE = E2TTT_SCAN_TILE;

// A tile of a sequence: tokens [lo, lo + n) of the sequence at tok0, tile `tile` of `tiles`.
struct Tile {
    int seq, tok0, lo, n, tile, tiles;
    // Tiles of the sequence that come before this one, on the way that is taken.
    int before;
    // Row of the published words and of starts: the tiles of the sequences before, and
    // never past the end whatever the offsets hold.
    __device__ __forceinline__ int64_t row() const { return tok0 / TILE + seq + tile; }
};

// The t-th tile: a sequence's tiles from its end (BWD), as the search goes, or its start.
template <bool BWD>
__device__ __forceinline__ bool find_tile(const ScanArgs& a, int t, Tile& r) {
    attn::Item it;
    if (!attn::find_item(a.cu, a.S, (int)a.N, t, attn::kInOrder, [](int n) { return n > TILE ? (n - 1) / TILE + 1 : 1; }, it)) return false;
    const auto same = [](int v) { return __builtin_amdgcn_readfirstlane(v); };  // of all lanes: rows in scalars
    it = {same(it.seq), same(it.tok0), same(it.n), same(it.tile), same(it.tiles)};
    const int from_end = it.tiles - 1 - it.tile, tile = BWD ? it.tile : from_end;
    r = {it.seq, it.tok0, tile * TILE, it.n - tile * TILE, tile, it.tiles, BWD ? from_end : tile};
    if (r.n > TILE) r.n = TILE;
    return true;
}

// Channel c of `rows` tokens from p on, which is the same for all lanes (so rows are
// addressed by scalars); the others are `fill`.
template <typename T, int K>
__device__ __forceinline__ void load(T (&x)[K], const T* p, int64_t stride, int rows, unsigned c, bool in, float fill) {
#pragma unroll
    for (int r = 0; r < K; ++r) x[r] = (T)fill;
    if (!in) return;
    if (rows >= K) {
#pragma unroll
        for (int r = 0; r < K; ++r, p += stride) x[r] = p[c];
    } else {
#pragma unroll
        for (int r = 0; r < K; ++r, p += stride)
            if (r < rows) x[r] = p[c];
    }
}

// Outputs of the tokens of no sequence: block b of a.clear.
template <typename T>
__device__ __forceinline__ void clear_rows(const ScanArgs& a, T* p, int b) {
    const int64_t lo = clamped(a.cu[0], (int)a.N), end = clamped(a.cu[a.S], (int)a.N), hi = end > lo ? end : lo;
    const int64_t first = lo * a.C, count = (lo + a.N - hi) * a.C, skip = (hi - lo) * a.C;
    for (int64_t i = (int64_t)b * blockDim.x + threadIdx.x; i < count; i += (int64_t)a.clear * blockDim.x)
        p[i < first ? i : i + skip] = (T)0.f;
}

// ------------------------------------------------------------ published words
// One per tile and channel, 0 before the launch: {H, P + 1 as bits}, then
// {the state after the tile, kState}, which is more than any of P.
constexpr unsigned kState = 0xffffffffu;
__device__ __forceinline__ u64 word_of(float h, unsigned key) { return (u64)key << 32 | __builtin_bit_cast(unsigned, h); }
__device__ __forceinline__ unsigned key_of(float P) { return P != P ? 0x7fc00001u : __builtin_bit_cast(unsigned, P) + 1; }
__device__ __forceinline__ float applied(u64 w, float h) {
    const unsigned key = (unsigned)(w >> 32);
    const float H = __builtin_bit_cast(float, (unsigned)w);
    return key == kState ? H : __builtin_fmaf(__builtin_bit_cast(float, key - 1), h, H);
}
__device__ __forceinline__ void publish(u64* p, u64 w) { __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
// Never in place of a state: sequences that overlap, by offsets that fall, share words.
__device__ __forceinline__ void publish_first(u64* p, u64 w) {
    __hip_atomic_fetch_max(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 published(const u64* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

__global__ __launch_bounds__(256) void scan_clear_kernel(u64* words, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) words[i] = 0;
}

// Words before the tiles': whether a wait was given up, and a ticket counter for each
// slab (tiles wait for tiles of their slab alone, and additions to one address take
// their turn: 2000 of them some 50 us), 64 bytes apart.
__host__ __device__ __forceinline__ int64_t header_words(int64_t C) { return 8 * ((C + 63) / 64 + 1); }

// The next tile of a slab that nobody has taken.
__device__ __forceinline__ int take_ticket(const ScanArgs& a, int slab) {
    return (int)__hip_atomic_fetch_add((unsigned*)(a.words + 8 * (slab + 1)), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state h that enters the tile from the `before` tiles in direction -dir, the
// words of the nearest at `row`: each wave waits for its share of the kLook nearest,
// the farthest of which has to be a state, and all are folded in order.  Words that are
// there cost one way to memory, some 2 us, and a chain of states takes some 5 us every
// kLook tiles (16384 tokens of 2048 channels: 78 us with 16 and two words per tile and
// channel, 66 so).
constexpr int kLook = 32;
__device__ __forceinline__ void enter(const ScanArgs& a, float& h, u64 (*sh)[64], int64_t row, int dir, int before, int c, bool in) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = before < kLook ? before : kLook;
    const u64* const base = a.words + header_words(a.C) + row * a.C + c;
    u64 w[kLook / NW];
#pragma unroll
    for (int j = 0; j < kLook / NW; ++j) {
        const int i = wave + j * NW;
        w[j] = word_of(0.f, kState);
        if (i < n && in) w[j] = published(base - (int64_t)dir * i * a.C);
    }
#pragma unroll
    for (int j = 0; j < kLook / NW; ++j) {
        const int i = wave + j * NW;
        if (i >= n) break;
        const unsigned want = i == kLook - 1 ? kState : 1;
        u64 since = 0;
        for (unsigned tries = 1; __ballot((unsigned)(w[j] >> 32) < want); ++tries) {
            if (tries % 64 == 0) {
                const u64 now = wall_clock64();
                if (since == 0) since = now;
                if (gives_up(tries, now - since) || published(a.words) != 0) {
                    publish(a.words, 1);
                    w[j] = word_of(__builtin_nanf(""), kState);
                    break;
                }
            }
            __builtin_amdgcn_s_sleep(1);
            if (in) w[j] = published(base - (int64_t)dir * i * a.C);
        }
        sh[i][lane] = w[j];
    }
    __syncthreads();
#pragma unroll 4
    for (int i = n - 1; i >= 0; --i) h = applied(sh[i][lane], h);
}

// Workgroups stay, kStay on a compute unit, and take tile after tile: the next one's
// tokens are on their way while this one's state is awaited and its outputs go out
// (16384 tokens of 2048 channels: 100 us with a workgroup per tile, three on a compute
// unit).  One channel per lane: with two, 67 us against 63, and half the workgroups for
// few channels.
constexpr int kStay = 2;
template <typename TX, typename TA, bool CHAIN>
__global__ __launch_bounds__(64 * NW, 2 * kStay) void scan_fwd_kernel(ScanArgs a) {
    __shared__ float2 all[2][NW + 1][64];  // (P, H) of the waves and of the tile
    __shared__ u64 words_of[CHAIN ? kLook : 1][64];
    __shared__ int tickets[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x >= a.groups) {
        clear_rows(a, (TX*)a.out, blockIdx.x - a.groups);
        return;
    }
    const int slab = blockIdx.x % a.slabs, c = slab * 64 + lane;
    const bool in = c < a.C;
    Tile next;
    TX nx[R];
    TA ng[R];
    float nh;  // the next tile's tokens, and the state that enters it if no tile is before it
    bool more;
    auto fetch = [&](int turn) {
        more = find_tile<false>(a, turn, next);
        if (!more) return;
        const int rows = next.n - wave * R;
        const int64_t tok = next.tok0 + next.lo + wave * R;
        nh = next.before == 0 && a.h0 && in ? a.h0[(int64_t)next.seq * a.C + c] : 0.f;
        load(nx, (const TX*)a.x + tok * a.x_tok, a.x_tok, rows, c, in, 0.f);
        load(ng, (const TA*)a.a + tok * a.a_tok, a.a_tok, rows, c, in, 1.f);
    };
    if (CHAIN && threadIdx.x == 0) tickets[0] = take_ticket(a, slab), tickets[1] = take_ticket(a, slab);
    if (CHAIN) __syncthreads();
    fetch(CHAIN ? tickets[0] : (int)blockIdx.x / a.slabs);
    for (int k = 1; more; ++k) {
        float2 (*const sh)[64] = all[k & 1];
        const Tile s = next;
        float h = nh;
        TX x[R];
        TA g[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = nx[r], g[r] = ng[r];
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            H = __builtin_fmaf((float)g[r], H, (float)x[r]);
            P *= (float)g[r];
        }
        sh[wave][lane] = make_float2(P, H);
        asm volatile("" : "+v"(h));  // is here before the barrier: state may be h0
        __syncthreads();
        const int turn = tickets[k & 1];
        u64* const word = CHAIN ? a.words + header_words(a.C) + s.row() * a.C + c : nullptr;
        const bool last = s.tile == s.tiles - 1;
        if (wave == NW - 1) {
            float p = 1.f, q = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float2 f = sh[w][lane];
                q = __builtin_fmaf(f.x, q, f.y);
                p *= f.x;
            }
            sh[NW][lane] = make_float2(p, q);
            if (CHAIN && s.before > 0 && !last && in) publish_first(word, word_of(q, key_of(p)));
        }
        if (CHAIN) {
            fetch(turn);
            if (threadIdx.x == 0) tickets[~k & 1] = take_ticket(a, slab);
            if (s.before > 0) enter(a, h, words_of, s.row() - 1, 1, s.before, c, in);
        } else {
            more = false;
        }
        float end = 0.f;
        if (wave == NW - 1) {
            end = __builtin_fmaf(sh[NW][lane].x, h, sh[NW][lane].y);
            if (CHAIN && !last && in) publish(word, word_of(end, kState));
        }
        if (a.starts && s.n > 0 && wave == 0 && in) a.starts[s.row() * a.C + c] = h;
        for (int w = 0; w < wave; ++w) h = __builtin_fmaf(sh[w][lane].x, h, sh[w][lane].y);
        const int rows = s.n - wave * R;
        TX* op = (TX*)a.out + (s.tok0 + s.lo + wave * R) * a.C;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            h = __builtin_fmaf((float)g[r], h, (float)x[r]);
            if (in && r < rows) op[c] = (TX)h;
            op += a.C;
        }
        if (a.state && last && wave == NW - 1 && in) a.state[(int64_t)s.seq * a.C + c] = end;
    }
}

// Sequences of a few tokens: a wave each and slab, no exchange; sixteen tokens' loads
// together, and fewer where fewer are left (one token each of 64 sequences, 2048 channels:
// always sixteen 6.3 us, so 2.5).  The host knows the lengths' sum alone, so that any of
// them may be long: above kAlone tokens, where a wave's ways to memory one after the other
// add up, a sequence is left to workgroups of their own, a.helpers per slab, that each look
// through their share of the sequences and walk through a long one tile by tile, the state
// in registers (256 sequences of one token and one of 3800: 70 us; as a wave's 580, alone in
// tiles side by side 21; without a long one the helpers cost 0.2 us at most).
constexpr int kAlone = 4 * R;
template <typename TX, typename TA>
__device__ __forceinline__ void walk(const ScanArgs& a, float2 (*all)[NW][64], int& turn, int seq, int tok0, int n, int c, bool in) {
    constexpr int K = R * 2 / sizeof(TX);  // tokens of a wave at a time: few enough registers for eight waves side by side
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float h = a.h0 && in ? a.h0[(int64_t)seq * a.C + c] : 0.f;
    float* st = a.starts ? a.starts + (int64_t)(tok0 / TILE + seq) * a.C + c : nullptr;
#pragma unroll 1
    for (int lo = 0; lo < n; lo += K * NW) {
        const int t = lo + wave * K;
        const int64_t tok = (int64_t)tok0 + t;
        TX x[K];
        TA g[K];
        int64_t xs = a.x_tok, as = a.a_tok, os = a.C;  // as below
        asm volatile("" : "+s"(xs), "+s"(as), "+s"(os));
        load(x, (const TX*)a.x + tok * a.x_tok, xs, n - t, c, in, 0.f);
        load(g, (const TA*)a.a + tok * a.a_tok, as, n - t, c, in, 1.f);
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int r = 0; r < K; ++r) {
            H = __builtin_fmaf((float)g[r], H, (float)x[r]);
            P *= (float)g[r];
        }
        float2 (*const sh)[64] = all[turn];  // the other half is still being read
        turn ^= 1;
        sh[wave][lane] = make_float2(P, H);
        asm volatile("" : "+v"(h));  // is here before the barrier: state may be h0
        __syncthreads();
        if (st && wave == 0 && in && lo % TILE == 0) st[(int64_t)(lo / TILE) * a.C] = h;
        float end = h;
#pragma unroll 2
        for (int w = 0; w < NW; ++w) {
            const float2 f = sh[w][lane];
            if (w == wave) h = end;
            end = __builtin_fmaf(f.x, end, f.y);
        }
        TX* op = (TX*)a.out + tok * a.C;
#pragma unroll
        for (int r = 0; r < K; ++r) {
            h = __builtin_fmaf((float)g[r], h, (float)x[r]);
            if (in && r < n - t) op[c] = (TX)h;
            op += os;
        }
        h = end;
    }
    if (a.state && wave == NW - 1 && in) a.state[(int64_t)seq * a.C + c] = h;
}

template <typename TX, typename TA>
__global__ __launch_bounds__(64 * NW, 8) void scan_short_kernel(ScanArgs a) {
    __shared__ float2 all[2][NW][64];  // (P, H) of the waves
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int b = (int)blockIdx.x;
    if (b < a.helpers * a.slabs) {
        const int c = b % a.slabs * 64 + lane, mine = b / a.slabs;
        int turn = 0;
        for (int64_t s0 = mine; s0 < a.S; s0 += 64 * a.helpers) {  // the same for all waves
            const int64_t seq = s0 + lane * a.helpers;
            const int tok0 = seq < a.S ? clamped(a.cu[seq], (int)a.N) : 0;
            const int n = seq < a.S ? clamped(a.cu[seq + 1], (int)a.N) - tok0 : 0;
            for (u64 longs = __ballot(n > kAlone); longs; longs &= longs - 1) {
                const int i = __builtin_ctzll(longs);
                walk<TX, TA>(a, all, turn, (int)s0 + i * a.helpers, __builtin_amdgcn_readlane(tok0, i), __builtin_amdgcn_readlane(n, i), c, c < a.C);
            }
        }
        return;
    }
    b -= a.helpers * a.slabs;
    const int past = b - (a.groups + NW - 1) / NW;
    if (past >= 0) {
        clear_rows(a, (TX*)a.out, past);
        return;
    }
    const int unit = b * NW + wave;
    if (unit >= a.groups) return;
    const int c = unit % a.slabs * 64 + lane;
    const bool in = c < a.C;
    const int seq = unit / a.slabs, tok0 = clamped(a.cu[seq], (int)a.N), n = clamped(a.cu[seq + 1], (int)a.N) - tok0;
    if (n > kAlone) return;
    float h = a.h0 && in ? a.h0[(int64_t)seq * a.C + c] : 0.f;
    const TX* xp = (const TX*)a.x + tok0 * a.x_tok;
    const TA* ap = (const TA*)a.a + tok0 * a.a_tok;
    TX* op = (TX*)a.out + (int64_t)tok0 * a.C;
    if (a.starts && n > 0 && in) a.starts[(int64_t)(tok0 / TILE + seq) * a.C + c] = h;
    auto step = [&](int t, auto count) {
        constexpr int K = decltype(count)::value;
        TX x[K];
        TA g[K];
        // else the compiler keeps a multiple of the strides for every row over the loop, in more
        // scalars than there are (256 sequences of 16 tokens: 15.9 us, so 13.0)
        int64_t xs = a.x_tok, as = a.a_tok, os = a.C;
        asm volatile("" : "+s"(xs), "+s"(as), "+s"(os));
        load(x, xp + t * a.x_tok, xs, n - t, c, in, 0.f);
        load(g, ap + t * a.a_tok, as, n - t, c, in, 1.f);
        TX* o = op + t * a.C;
#pragma unroll
        for (int r = 0; r < K; ++r, o += os) {
            h = __builtin_fmaf((float)g[r], h, (float)x[r]);
            if (in && r < n - t) o[c] = (TX)h;
        }
    };
    int t = 0;
    for (; n - t > 4; t += R) step(t, std::integral_constant<int, R>{});
    if (n - t > 1) step(t, std::integral_constant<int, 4>{});
    else if (n - t == 1) step(t, std::integral_constant<int, 1>{});
    if (a.state && in) a.state[(int64_t)seq * a.C + c] = h;
}

template <typename TX, typename TA, bool CHAIN>
__global__ __launch_bounds__(64 * NW, 4) void scan_bwd_kernel(ScanArgs a) {
    __shared__ float sh[NW + 1][3][64];  // (P, H, K) of the waves, (P, K) of the tile
    __shared__ u64 words_of[CHAIN ? kLook : 1][64];
    __shared__ int ticket;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x >= a.groups) {
        clear_rows(a, (TX*)a.out, blockIdx.x - a.groups);
        clear_rows(a, (TA*)a.da, blockIdx.x - a.groups);
        return;
    }
    const int slab = blockIdx.x % a.slabs, c = slab * 64 + lane;
    const bool in = c < a.C;
    if (CHAIN && threadIdx.x == 0) ticket = take_ticket(a, slab);
    if (CHAIN) __syncthreads();
    Tile s;
    if (!find_tile<true>(a, CHAIN ? ticket : (int)blockIdx.x / a.slabs, s)) return;
    const int rows = s.n - wave * R;
    const int64_t tok = s.tok0 + s.lo + wave * R;
    TX x[R], d[R];
    TA g[R];
    load(g, (const TA*)a.a + tok * a.a_tok, a.a_tok, rows, c, in, 1.f);
    load(d, (const TX*)a.dout + tok * a.C, a.C, rows, c, in, 0.f);
    load(x, (const TX*)a.x + tok * a.x_tok, a.x_tok, rows, c, in, 0.f);
    // the gradient that comes from after the tile, a_{t+1} g_{t+1}, and the state before it
    float gc = s.before == 0 && a.h0 && in ? a.h0[(int64_t)s.seq * a.C + c] : 0.f;
    float h = s.n > 0 && in ? a.starts[s.row() * a.C + c] : 0.f;
    float P = 1.f, H = 0.f, K = 0.f;  // h -> P h + H over the wave's tokens, and the gradient's c -> P c + K
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        P *= (float)g[r];
        K = (float)g[r] * ((float)d[r] + K);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) H = __builtin_fmaf((float)g[r], H, (float)x[r]);
    sh[wave][0][lane] = P, sh[wave][1][lane] = H, sh[wave][2][lane] = K;
    __syncthreads();
    u64* const word = CHAIN ? a.words + header_words(a.C) + s.row() * a.C + c : nullptr;
    if (wave == 0) {
        float p = 1.f, q = 0.f;
#pragma unroll
        for (int w = NW - 1; w >= 0; --w) {
            q = __builtin_fmaf(sh[w][0][lane], q, sh[w][2][lane]);
            p *= sh[w][0][lane];
        }
        sh[NW][0][lane] = p, sh[NW][2][lane] = q;
        if (CHAIN && s.before > 0 && s.tile > 0 && in) publish_first(word, word_of(q, key_of(p)));
    }
    if (CHAIN && s.before > 0) enter(a, gc, words_of, s.row() + 1, -1, s.before, c, in);
    if (wave == 0 && in) {
        const float end = __builtin_fmaf(sh[NW][0][lane], gc, sh[NW][2][lane]);
        if (CHAIN && s.tile > 0) publish(word, word_of(end, kState));
        if (a.state && s.tile == 0) a.state[(int64_t)s.seq * a.C + c] = end;
    }
    for (int w = NW - 1; w > wave; --w) gc = __builtin_fmaf(sh[w][0][lane], gc, sh[w][2][lane]);
    for (int w = 0; w < wave; ++w) h = __builtin_fmaf(sh[w][0][lane], h, sh[w][1][lane]);
    float before[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        before[r] = h;
        h = __builtin_fmaf((float)g[r], h, (float)x[r]);
    }
    const int64_t o0 = (tok + R - 1) * a.C;
    TX* xp = (TX*)a.out + o0;
    TA* ap = (TA*)a.da + o0;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        const float gt = (float)d[r] + gc;
        gc = (float)g[r] * gt;
        if (in && r < rows) xp[c] = (TX)gt, ap[c] = (TA)(gt * before[r]);
        xp -= a.C;
        ap -= a.C;
    }
}

// Clears the published words of a call whose tiles wait for each other.
hipError_t clear_words(const ScanArgs& a, hipStream_t s) {
    const int64_t n = scan_words(a.N, a.S, a.C), groups = (n + 1023) / 1024;
    scan_clear_kernel<<<dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, s>>>(a.words, n);
    return hipGetLastError();
}

template <typename TX, typename TA>
hipError_t forward(ScanArgs a, hipStream_t s) {
    const dim3 bl(64 * NW);
    if (a.shorts) {
        // as many as there may be long sequences, and up to 512 workgroups
        const int64_t most = a.N / (kAlone + 1), fit = a.slabs < 512 ? 512 / a.slabs : 1;
        a.helpers = (int)(most < fit ? most : fit);
        scan_short_kernel<TX, TA><<<dim3((unsigned)(a.helpers * a.slabs + (a.groups + NW - 1) / NW + a.clear)), bl, 0, s>>>(a);
    } else if (a.words) {
        int cus = 0;
        hipError_t e = device_cu_count(&cus);
        if (e == hipSuccess) e = clear_words(a, s);
        if (e != hipSuccess) return e;
        const int stay = (kStay * cus + a.slabs - 1) / a.slabs * a.slabs;
        if (a.groups > stay) a.groups = stay;
        scan_fwd_kernel<TX, TA, true><<<dim3((unsigned)(a.groups + a.clear)), bl, 0, s>>>(a);
    } else {
        scan_fwd_kernel<TX, TA, false><<<dim3((unsigned)(a.groups + a.clear)), bl, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <typename TX, typename TA>
hipError_t backward(const ScanArgs& a, hipStream_t s) {
    const dim3 bl(64 * NW), gr((unsigned)(a.groups + a.clear));
    if (a.words) {
        const hipError_t e = clear_words(a, s);
        if (e != hipSuccess) return e;
        scan_bwd_kernel<TX, TA, true><<<gr, bl, 0, s>>>(a);
    } else {
        scan_bwd_kernel<TX, TA, false><<<gr, bl, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

int64_t scan_words(int64_t N, int64_t S, int64_t C) { return header_words(C) + (N / TILE + S) * C; }

hipError_t launch_scan_forward(const ScanArgs& a, hipStream_t s) {
    if (a.x_f32) return forward<float, float>(a, s);
    return a.gate_f32 ? forward<__bf16, float>(a, s) : forward<__bf16, __bf16>(a, s);
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
    if (a.x_f32) return backward<float, float>(a, s);
    return a.gate_f32 ? backward<__bf16, float>(a, s) : backward<__bf16, __bf16>(a, s);
}

}  // namespace e2ttt
