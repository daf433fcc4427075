// New tokens' keys and values into the pages of a cache in 8 bits: 16 lanes a row,
// its largest magnitude, the scale's exponent from that number's bits, and the
// values times the exact inverse, rounded to nearest even.  One chain of reads per row:
// the offsets, the page, the row (one token 2.7 us, 64 of 4 key heads 5.3).
#include "attn8.h"

namespace e2ttt {
namespace attn {
namespace {

__global__ __launch_bounds__(256) void append8_kernel(AttnArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kAppend8Rows + (threadIdx.x >> 4);
    const int lane = threadIdx.x & 15, c = 8 * lane;
    const bool is_v = u & 1;
    const int64_t nk = u >> 1, n = nk / a.K;
    if (n >= a.N) return;
    const int kvh = (int)(nk - n * a.K);
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
    const __bf16* src = (const __bf16*)(is_v ? a.v : a.k) + n * (is_v ? a.v_tok : a.k_tok) + kvh * (is_v ? a.v_head : a.k_head);
    bf16x8 x = {};
    if (c < a.D) x = *(const bf16x8*)(src + c);
    unsigned top = 0;  // the largest magnitude's bits: NaN above infinity above all others
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = (float)x[e];
        const unsigned m = __builtin_bit_cast(unsigned, f) & 0x7fffffffu;
        top = top > m ? top : m;
    }
#pragma unroll
    for (int d = 8; d; d >>= 1) {
        const unsigned m = __shfl_xor(top, d);
        top = top > m ? top : m;
    }
    const bool bad = top >= 0x7f800000u;
    // top = 1.m 2^(e - 127) <= 1.75 2^8 scale
    int b = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    b = top == 0 ? 127 : (bad ? 255 : (b > 0 ? b : 0));
    const float inv = __builtin_bit_cast(float, (unsigned)(254 - b) << 23);
    u32x2 y = {0x7f7f7f7fu, 0x7f7f7f7fu};
    if (!bad) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unsigned w = __builtin_amdgcn_cvt_pk_fp8_f32((float)x[4 * h] * inv, (float)x[4 * h + 1] * inv, 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32((float)x[4 * h + 2] * inv, (float)x[4 * h + 3] * inv, w, true);
            y[h] = w;
        }
    }
    unsigned char* to = (unsigned char*)(is_v ? a.pg.vc : a.pg.kc) + page * (is_v ? a.pg.v_page : a.pg.k_page) +
                        kvh * (is_v ? a.pg.v_head : a.pg.k_head) + slot * (is_v ? a.pg.v_slot : a.pg.k_slot);
    if (c < a.D) *(u32x2*)(to + c) = y;
    if (lane == 0) (is_v ? a.pg.vs : a.pg.ks)[(((int64_t)page * a.K + kvh) << a.pg.shift) + slot] = (unsigned char)b;
}

}  // namespace
}  // namespace attn

hipError_t launch_append8(const AttnArgs& a, hipStream_t s) {
    const int64_t grid = (2 * a.N * a.K + kAppend8Rows - 1) / kAppend8Rows;
    if (grid > kMaxGroups) return hipErrorInvalidConfiguration;
    attn::append8_kernel<<<dim3((unsigned)grid), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace e2ttt
