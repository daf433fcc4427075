// Token lookup with a scale, and its gradient:
//
//   out[n] = scale table[t_n],   dtable[v] = scale sum_{n: t_n = v} dout[n].
//
// HBM bound: the lookup reads and writes a row per token, the gradient reads a
// row per token and writes every row of the table, most of which are zeros.
//
// The gradient sums rows of equal tokens in the order they come in, in 32 bits,
// without floating-point atomics, in three launches:
//
// 1. The places of the tokens are sorted by token, places of equal ones in
//    order.  A workgroup owns a range of tokens and reads all of them twice: once
//    to count those below its range and, wave by wave, each of its own; then to
//    put every place where it belongs.  No workgroup waits for another, and the
//    reads (the tokens alone, from the L2 cache) are little beside the rows, though they
//    grow with tokens times workgroups (rows of 64, in all: 30 us from 16384 tokens, 138 from
//    131072; of 2048, 97 and 391).
// 2. A wave per row of the table and 1024 columns sums its places' rows from registers
//    and writes the row.  Rows with more than kEmbedPiece places (a text's commonest
//    words) are left to waves that own a piece of the sorted places each: a wave's
//    places come in few ways to memory, so none is still at work when the others are
//    done (16384 tokens of a text, a table of 32000 rows of 2048 in fp32, 262 MB of them:
//    137 us with pieces of 32 and two rows on their way, 72 with 16 and eight; a fill of
//    the table alone is 33).
// 3. The pieces of such rows are summed in order.
//
// The whole gradient of that table takes 17 us for the order, 72 and 10; the lookup
// before it 29 (200 MB at most), and a lookup of eight tokens is one launch, 7 us.
#include "tokens_internal.h"

namespace e2ttt {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// V values from p, aligned to 16 bytes (or all of them) where V is more than one.
template <typename T, int V>
constexpr int kAtOnce = V * sizeof(T) < 16 ? V : 16 / sizeof(T);
template <typename T, int V>
__device__ __forceinline__ void read(float (&x)[V], const T* p) {
    constexpr int E = kAtOnce<T, V>;
    typedef T Vec __attribute__((ext_vector_type(E)));
#pragma unroll
    for (int i = 0; i < V / E; ++i) {
        const Vec u = *(const Vec*)(p + i * E);
#pragma unroll
        for (int e = 0; e < E; ++e) x[i * E + e] = (float)u[e];
    }
}
template <typename T, int V>
__device__ __forceinline__ void write(T* p, const float (&x)[V], float scale) {
    constexpr int E = kAtOnce<T, V>;
    typedef T Vec __attribute__((ext_vector_type(E)));
#pragma unroll
    for (int i = 0; i < V / E; ++i) {
        Vec u;
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = (T)(x[i * E + e] * scale);
        *(Vec*)(p + i * E) = u;
    }
}

// A token, or -1 for one outside the table.
__device__ __forceinline__ int token_of(const EmbedArgs& a, int64_t n) {
    const int64_t t = a.wide ? ((const int64_t*)a.tokens)[n] : ((const int*)a.tokens)[n];
    return t >= 0 && t < a.V ? (int)t : -1;
}

// Tokens n, n + 64, ..., -1 from `end` on; all on their way at once.
template <int U>
__device__ __forceinline__ void tokens_of(const EmbedArgs& a, int (&t)[U], int64_t n, int64_t end) {
    int64_t x[U];
    if (a.wide) {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = n + u * 64 < end ? ((const int64_t*)a.tokens)[n + u * 64] : -1;
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = n + u * 64 < end ? ((const int*)a.tokens)[n + u * 64] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] = x[u] >= 0 && x[u] < a.V ? (int)x[u] : -1;
}

// HIP counts the threads along a grid dimension in 32 bits.
constexpr int64_t kGridX = 1 << 21;
dim3 grid_of(int64_t groups, unsigned z = 1) {
    return groups <= kGridX ? dim3((unsigned)groups, 1, z) : dim3((unsigned)kGridX, (unsigned)((groups + kGridX - 1) / kGridX), z);
}
__device__ __forceinline__ int64_t group_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// 2^shift threads per row.
template <typename TI, typename TO, int V>
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedArgs a, int shift) {
    const int64_t n = (group_index() << (8 - shift)) + (threadIdx.x >> shift);
    if (n >= a.N) return;
    const int t = token_of(a, n);
    const TI* in = (const TI*)a.in + t * a.W;
    TO* out = (TO*)a.out + n * a.W;
    for (int64_t c = (int64_t)(threadIdx.x & ((1 << shift) - 1)) * V; c < a.W; c += (int64_t)V << shift) {
        float x[V] = {};
        if (t >= 0) read<TI, V>(x, in + c);
        write<TO, V>(out + c, x, a.scale);
    }
}

// ------------------------------------------------------------ 1: the order
constexpr int kOrderWaves = 16;
constexpr int kRange = 512;  // tokens of a workgroup's range, at most

__device__ __forceinline__ int lanes_below(unsigned long long m) {
    return __builtin_amdgcn_mbcnt_hi((unsigned)(m >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)m, 0));
}
__device__ __forceinline__ int wave_inclusive(int x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// Tokens [v0, v0 + 2^bits) of this workgroup.
__global__ __launch_bounds__(64 * kOrderWaves) void embed_order_kernel(EmbedArgs a, int bits) {
    __shared__ int cnt[kOrderWaves][kRange];  // places of each token in a wave's stretch; then where the next one goes
    __shared__ int sums[kOrderWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, R = 1 << bits;
    const int v0 = (int)blockIdx.x << bits;
    for (int i = threadIdx.x; i < kOrderWaves * R; i += 64 * kOrderWaves) cnt[i >> bits][i & (R - 1)] = 0;
    __syncthreads();
    const int64_t per = ((a.N + kOrderWaves - 1) / kOrderWaves + 63) / 64 * 64;
    const int64_t n0 = wave * per, n1 = n0 + per < a.N ? n0 + per : a.N;
    int below = 0;
    constexpr int U = 8;  // tokens on their way to a lane
    for (int64_t i = n0; i < n1; i += 64 * U) {
        int t[U];
        tokens_of<U>(a, t, i + lane, n1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            below += t[u] >= 0 && t[u] < v0;
            const int r = t[u] - v0;
            if (t[u] >= 0 && r >= 0 && r < R) atomicAdd(&cnt[wave][r], 1);
        }
    }
    below = wave_inclusive(below);
    if (lane == 63) sums[wave] = below;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) base += sums[w];
    __syncthreads();
    // a thread per token of the range (R <= 512 <= threads)
    int mine = 0;
    if ((int)threadIdx.x < R)
        for (int w = 0; w < kOrderWaves; ++w) mine += cnt[w][threadIdx.x];
    const int incl = wave_inclusive(mine);
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) base += sums[w];
    int at = base + incl - mine;
    if ((int)threadIdx.x < R) {
        if (v0 + (int)threadIdx.x < a.V) a.start[v0 + threadIdx.x] = at;
        for (int w = 0; w < kOrderWaves; ++w) {
            const int c = cnt[w][threadIdx.x];
            cnt[w][threadIdx.x] = at;
            at += c;
        }
        if (v0 + (int)threadIdx.x == a.V - 1) a.start[a.V] = at;
    }
    __syncthreads();
    for (int64_t i = n0; i < n1; i += 64 * U) {
        int t[U];
        tokens_of<U>(a, t, i + lane, n1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = t[u] - v0;
            const bool in = t[u] >= 0 && r >= 0 && r < R;
            unsigned long long same = __ballot(in);
            if (!same) continue;
            for (int b = 0; b < bits; ++b) {  // lanes with the same token
                const unsigned long long set = __ballot((r >> b) & 1);
                same &= (r >> b) & 1 ? set : ~set;
            }
            if (in) {
                const int rank = lanes_below(same), to = cnt[wave][r];
                a.order[to + rank] = (int)(i + u * 64 + lane);
                if (rank == 0) cnt[wave][r] = to + __popcll(same);
            }
        }
    }
}

// ------------------------------------------------------------- 2: the sums
// acc += the rows of `count` places, kEmbedPiece at most, from order[s] on; columns c0 on.
template <typename TI, int V, int NU>
__device__ __forceinline__ void sum_places(const EmbedArgs& a, float (&acc)[NU][V], int s, int count, int64_t c0) {
    constexpr int E = kAtOnce<TI, V>, kFit = 32 / (NU * V) * (int)(4 / sizeof(TI)), U = kFit < 2 ? 2 : kFit;
    typedef TI Vec __attribute__((ext_vector_type(E)));
    const int lane = threadIdx.x & 63;
    const int mine = lane < count ? a.order[s + lane] : 0;
    for (int k = 0; k < count; k += U) {
        Vec x[U][NU][V / E];  // U places' rows on their way together
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t n = __builtin_amdgcn_readlane(mine, (k + j) & 63);
            const TI* row = (const TI*)a.in + n * a.W;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                const int64_t c = c0 + ((int64_t)i * 64 + lane) * V;
#pragma unroll
                for (int p = 0; p < V / E; ++p)
                    if (k + j < count && c < a.W) x[j][i][p] = *(const Vec*)(row + c + p * E);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (k + j < count) {
#pragma unroll
                for (int i = 0; i < NU; ++i)
#pragma unroll
                    for (int q = 0; q < V; ++q) acc[i][q] += (float)x[j][i][q / E][q % E];
            }
    }
}

template <typename TO, int V, int NU>
__device__ __forceinline__ void write_row(const EmbedArgs& a, TO* row, const float (&acc)[NU][V], float scale, int64_t c0) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int64_t c = c0 + ((int64_t)i * 64 + lane) * V;
        if (c < a.W) write<TO, V>(row + c, acc[i], scale);
    }
}

// A wave per piece, then one per row of the table; 64 V NU columns each.
template <typename TI, typename TO, int V, int NU>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedArgs a, int64_t pieces) {
    const int64_t w = group_index() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)blockIdx.z * (64 * V * NU);
    if (w < pieces) {
        const int total = a.start[a.V], b0 = (int)w * kEmbedPiece;
        const int b1 = b0 + kEmbedPiece < total ? b0 + kEmbedPiece : total;
        if (b0 >= b1) return;
        // the row that the piece begins in, and the one it ends in
        for (int k = 0; k < 2; ++k) {
            const int v = token_of(a, a.order[k == 0 ? b0 : b1 - 1]);
            const int s = a.start[v], e = a.start[v + 1];
            const bool starts = s >= b0;
            if (e - s > kEmbedPiece && starts == (k == 1)) {
                float acc[NU][V] = {};
                const int lo = s > b0 ? s : b0, hi = e < b1 ? e : b1;
                sum_places<TI, V, NU>(a, acc, lo, hi - lo, c0);
                write_row<float, V, NU>(a, a.part + (2 * w + k) * a.W, acc, 1.f, c0);
            }
        }
        return;
    }
    const int64_t v = w - pieces;
    if (v >= a.V) return;
    const int s = a.start[v], e = a.start[v + 1];
    if (e - s > kEmbedPiece) return;
    float acc[NU][V] = {};
    sum_places<TI, V, NU>(a, acc, s, e - s, c0);
    write_row<TO, V, NU>(a, (TO*)a.out + v * a.W, acc, a.scale, c0);
}

// ------------------------------------------------------------- 3: the join
// A workgroup per piece, which has work where a row with many places begins in
// it: that row's pieces, a stretch of them per wave and then the waves in order.
constexpr int kJoinWaves = 8;
template <typename TO, int V>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(EmbedArgs a) {
    __shared__ float sh[kJoinWaves][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t w = group_index();
    const int total = a.start[a.V];
    if (w * kEmbedPiece >= total) return;
    const int b0 = (int)w * kEmbedPiece, b1 = b0 + kEmbedPiece < total ? b0 + kEmbedPiece : total;
    const int v = token_of(a, a.order[b1 - 1]);
    const int s = a.start[v], e = a.start[v + 1];
    if (e - s <= kEmbedPiece || s < b0) return;
    const int last = (e - 1) / kEmbedPiece, count = last - (int)w + 1;
    const int per = (count + kJoinWaves - 1) / kJoinWaves;
    const int i0 = wave * per, i1 = i0 + per < count ? i0 + per : count;
    const int64_t c = ((int64_t)blockIdx.z * 64 + lane) * V;
    float acc[V] = {};
    if (c < a.W) {
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {  // the first piece of the row is one it begins in
            const float* p = a.part + (2 * (w + i) + (i == 0)) * a.W + c;
            float x[V];
            read<float, V>(x, p);
#pragma unroll
            for (int q = 0; q < V; ++q) acc[q] += x[q];
        }
    }
#pragma unroll
    for (int q = 0; q < V; ++q) sh[wave][lane * V + q] = acc[q];
    __syncthreads();
    if (wave != 0 || c >= a.W) return;
#pragma unroll
    for (int k = 1; k < kJoinWaves; ++k)
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] += sh[k][lane * V + q];
    write<TO, V>((TO*)a.out + (int64_t)v * a.W + c, acc, a.scale);
}

template <typename TI, typename TO, int V>
hipError_t forward(const EmbedArgs& a, hipStream_t s) {
    int shift = 3;  // threads per row
    while (shift < 8 && ((int64_t)V << shift) < a.W) ++shift;
    embed_fwd_kernel<TI, TO, V><<<grid_of((a.N + (256 >> shift) - 1) >> (8 - shift)), dim3(256), 0, s>>>(a, shift);
    return hipGetLastError();
}

template <typename TI, typename TO, int V, int NU>
hipError_t sums(const EmbedArgs& a, int64_t pieces, hipStream_t s) {
    const unsigned z = (unsigned)((a.W + 64 * V * NU - 1) / (64 * V * NU));
    embed_sum_kernel<TI, TO, V, NU><<<grid_of((pieces + a.V + 3) / 4, z), dim3(256), 0, s>>>(a, pieces);
    return hipGetLastError();
}

template <typename TI, typename TO, int V>
hipError_t backward(const EmbedArgs& a, hipStream_t s) {
    int bits = 0;  // a workgroup per compute unit, each with as few tokens as that leaves
    while (bits < 9 && ((int64_t)a.V >> bits) > 256) ++bits;
    static_assert(1 << 9 == kRange, "a workgroup's range fits its counters");
    const int64_t groups = ((int64_t)a.V + (1 << bits) - 1) >> bits;
    embed_order_kernel<<<dim3((unsigned)groups), dim3(64 * kOrderWaves), 0, s>>>(a, bits);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t pieces = a.N > kEmbedPiece ? (a.N + kEmbedPiece - 1) / kEmbedPiece : 0;
    // 64 V columns to a wave while all of them fit the chip at once (256 rows of 512: 7 us,
    // 26 with 16 times 64), else more, so that fewer look for their places
    const int64_t narrow = (a.W + 64 * V - 1) / (64 * V);
    e = (pieces + a.V) * narrow <= 8192 ? sums<TI, TO, V, 1>(a, pieces, s) : sums<TI, TO, V, 16 / V>(a, pieces, s);
    if (e != hipSuccess || pieces == 0) return e;
    embed_join_kernel<TO, V><<<grid_of(pieces, (unsigned)((a.W + 64 * V - 1) / (64 * V))), dim3(64 * kJoinWaves), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding_forward(const EmbedArgs& a, hipStream_t s) {
    if (a.in_f32 && a.out_f32) return a.vec ? forward<float, float, 4>(a, s) : forward<float, float, 1>(a, s);
    if (a.in_f32) return a.vec ? forward<float, __bf16, 8>(a, s) : forward<float, __bf16, 1>(a, s);
    if (a.out_f32) return a.vec ? forward<__bf16, float, 8>(a, s) : forward<__bf16, float, 1>(a, s);
    return a.vec ? forward<__bf16, __bf16, 8>(a, s) : forward<__bf16, __bf16, 1>(a, s);
}

hipError_t launch_embedding_backward(const EmbedArgs& a, hipStream_t s) {
    if (a.in_f32 && a.out_f32) return a.vec ? backward<float, float, 4>(a, s) : backward<float, float, 1>(a, s);
    if (a.in_f32) return a.vec ? backward<float, __bf16, 4>(a, s) : backward<float, __bf16, 1>(a, s);
    if (a.out_f32) return a.vec ? backward<__bf16, float, 4>(a, s) : backward<__bf16, float, 1>(a, s);
    return a.vec ? backward<__bf16, __bf16, 8>(a, s) : backward<__bf16, __bf16, 1>(a, s);
}

}  // namespace e2ttt
