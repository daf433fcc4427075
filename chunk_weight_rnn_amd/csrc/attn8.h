// Shared by the kernels over a paged cache in 8 bits (attn8_append.hip,
// attn8_decode.hip, attn8_fwd.hip):
//
//   k_j = 2^(b_j - 127) k8_j,  v_j likewise,  e4m3 values and a scale per slot and
//   key head, the smallest power of two that brings the largest magnitude to 448.
//
// A power of two loses nothing against other scales, since the values are floats,
// and makes everything after it exact: an 8-bit value times its scale is a bf16
// number, so the products are those of attn_decode.hip and attn_fwd.hip on bf16
// operands, and the only rounding that is new is the one into the cache.  The
// conversion instruction takes the scale along.  As there, probabilities are rounded to
// bf16 for the second product, which the matrix instructions take at sixteen times the rate
// of fp32: outputs are 1.25 to 1.4 times as far from 64 bits as a plain form in
// fp32 is, whose one rounding is the output's (0.0021 to 0.0023 of the norm, 0.0017).
//
// The new tokens are written by a launch before (attn8_append.hip): what attends reads the
// cache alone, so that tokens fed one by one and in chunks see the same keys.
#pragma once

#include "attn_common.h"

namespace e2ttt {
namespace attn {
namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2_t;

// Eight e4m3 values times a scale, whose exponent field alone counts (0: 2^-127,
// 255: NaN), as bf16.
__device__ __forceinline__ bf16x8 widen(unsigned lo, unsigned hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ float scale_bits(unsigned b) { return __builtin_bit_cast(float, b << 23); }

// --------------------------------------------- one position, term by term
struct Pos8 {  // a position's key or value, and its scale; zeros where none is read
    const unsigned char* row;
    unsigned char scale;
};
template <bool V>
__device__ __forceinline__ Pos8 position8(const AttnArgs& a, const int* table, int kvh, int pos, int begin, int end) {
    if (pos < begin || pos >= end || (pos >> a.pg.shift) >= a.pg.wide) return {zeros, 0};
    const int p = table[pos >> a.pg.shift];
    if ((unsigned)p >= (unsigned)a.pg.pages) return {zeros, 0};
    const int64_t slot = pos & ((1 << a.pg.shift) - 1);
    const unsigned char* s = V ? a.pg.vs : a.pg.ks;
    return {(const unsigned char*)(V ? a.pg.vc : a.pg.kc) + p * (V ? a.pg.v_page : a.pg.k_page) +
                kvh * (V ? a.pg.v_head : a.pg.k_head) + slot * (V ? a.pg.v_slot : a.pg.k_slot),
            s[(((int64_t)p * a.K + kvh) << a.pg.shift) + slot]};
}
__device__ __forceinline__ float dot8(const Pos8& k, const __bf16* q, int D, int lane) {
    float t = 0.f;
#pragma unroll 1
    for (int c = lane >> 5; c < D / 8; c += 2) {
        const u32x2 u = *(const u32x2*)(k.row + 8 * c);
        const bf16x8 x = widen(u[0], u[1], scale_bits(k.scale)), y = *(const bf16x8*)(q + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) t = __builtin_fmaf((float)x[e], (float)y[e], t);
    }
    return t + other_half(t, lane);
}
template <int DP>
__device__ __forceinline__ void add8(f32x16 (&acc)[DP / 32], const Pos8& v, float w, int D, int lane) {
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * dt + 8 * j + 4 * (lane >> 5);
            if (w == 0.f || d >= D) continue;
            const unsigned u = *(const unsigned*)(v.row + d);
            const bf16x8 x = widen(u, u, scale_bits(v.scale));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[dt][4 * j + e] = __builtin_fmaf(w, (float)x[e], acc[dt][4 * j + e]);
            __builtin_amdgcn_sched_barrier(0);
        }
}

}  // namespace
}  // namespace attn
}  // namespace e2ttt
