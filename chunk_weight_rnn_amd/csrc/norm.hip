// Root-mean-square norm with the residual's addition, and its gradients:
//
//   h = x + residual (rounded to the stream's type),
//   rstd = 1 / sqrt(mean(h^2) + eps),  xhat = h rstd,  y = xhat weight,
//   dx = dh + rstd (g - xhat mean(g xhat)), g = dy weight,
//   dweight = sum over rows of dy xhat,
//
// y in the stream's type or as 8-bit floats (e4m3) with a scale per row.
//
// HBM bound.  A row is held in registers, so every tensor passes once: WPR
// waves per row (one up to 64 threads' worth, four up to 256), NV units of V
// consecutive values per thread (V = 16 bytes' worth where every row starts on
// 16 bytes, else 1).  The weight's gradient is summed in registers over the rows
// a workgroup walks, written once per workgroup and summed by a second launch in a
// fixed order.
//
// 16384 rows of 2048 in bf16: forward with residual and 8-bit output 43 us where
// calls repeat one input, which the last-level cache holds in part, and 53 us a
// call on changing ones, 4.5 TB/s; backward with the stream's gradient 53 us, 5.1
// TB/s, and 5 for the sum of the 512 partial weight gradients (a large copy: 5.1).
#include <type_traits>

#include "layer_internal.h"

namespace e2ttt {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T, int V>
struct alignas(sizeof(T) * V) Unit {
    T v[V];
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}
__device__ __forceinline__ unsigned max_bits(unsigned x, unsigned y) { return x > y ? x : y; }
__device__ __forceinline__ unsigned wave_max(unsigned x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x = max_bits(x, __shfl_xor(x, d));
    return x;
}

// Over the WPR waves of a row (one workgroup per row for WPR > 1); the same
// order in every wave.
template <int WPR>
__device__ __forceinline__ float row_sum(float x, float* sh) {
    x = wave_sum(x);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sh[wave] = x;
        __syncthreads();
        x = sh[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) x += sh[w];
    }
    return x;
}
template <int WPR>
__device__ __forceinline__ unsigned row_max(unsigned x, float* sh) {
    x = wave_max(x);
    if constexpr (WPR > 1) {
        unsigned* const us = (unsigned*)sh;
        const int wave = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) us[wave] = x;
        __syncthreads();
        x = us[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) x = max_bits(x, us[w]);
    }
    return x;
}

// A magnitude as a whole number: ordered as the values are, and NaN above all of
// them, so that a maximum keeps it.
__device__ __forceinline__ unsigned magnitude(float x) { return __builtin_bit_cast(unsigned, x) & 0x7fffffffu; }

// One fp32 pair to e4m3, low two bytes.
__device__ __forceinline__ unsigned pk8(float a, float b) {
    return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

// HIP takes fewer than 2^32 threads along a dimension of a grid, which 2^31 rows
// of a workgroup each exceed: the workgroups stand in two dimensions.
constexpr int64_t kGridX = 1 << 21;
dim3 grid_of(int64_t groups) {
    return groups <= kGridX ? dim3((unsigned)groups) : dim3((unsigned)kGridX, (unsigned)((groups + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t group_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

constexpr float kF8Max = 448.f;

// A row's scale, from its largest magnitude: NaN if that is, 1 for zeros.  Not less
// than the smallest value there is: a scale of 0 would make NaN of the row's zeros.
__device__ __forceinline__ float scale_of(unsigned top) {
    const float s = __builtin_bit_cast(float, top) / kF8Max;
    return top == 0 ? 1.f : (s == 0.f ? __builtin_bit_cast(float, 1u) : s);
}

// y / scale inside the format's range: a subnormal scale can round the
// quotient of the row's largest value past it, which the conversion would turn
// into NaN.  NaN stays NaN.
__device__ __forceinline__ float quotient(float y, float scale) {
    const float q = y / scale;
    return q > kF8Max ? kF8Max : (q < -kF8Max ? -kF8Max : q);
}

template <typename T, int V, int WPR, int NV>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a) {
    constexpr int TPR = 64 * WPR;  // threads per row
    __shared__ float sh[16];
    const int64_t row = WPR == 1 ? group_index() * 4 + (threadIdx.x >> 6) : group_index();
    if (row >= a.rows) return;
    const int t = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int W = (int)a.width;
    using U = Unit<T, V>;
    const T* x = (const T*)a.x + row * W;
    const T* res = a.residual ? (const T*)a.residual + row * W : nullptr;
    U u[NV], ur[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c < W) {
            u[i] = *(const U*)(x + c);
            if (res) ur[i] = *(const U*)(res + c);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c < W) {
            if (res) {
#pragma unroll
                for (int e = 0; e < V; ++e) u[i].v[e] = (T)((float)u[i].v[e] + (float)ur[i].v[e]);
                *(U*)((T*)a.h + row * W + c) = u[i];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) ss = __builtin_fmaf((float)u[i].v[e], (float)u[i].v[e], ss);
        }
    }
    ss = row_sum<WPR>(ss, sh);
    const float rstd = rsqrtf(ss / (float)W + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    if (!a.bits8) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c < W) {
                const Unit<float, V> w = *(const Unit<float, V>*)(a.weight + c);
#pragma unroll
                for (int e = 0; e < V; ++e) u[i].v[e] = (T)((float)u[i].v[e] * rstd * w.v[e]);
                *(U*)((T*)a.y + row * W + c) = u[i];
            }
        }
        return;
    }
    float y[NV][V];
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c < W) {
            const Unit<float, V> w = *(const Unit<float, V>*)(a.weight + c);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[i][e] = (float)u[i].v[e] * rstd * w.v[e];
                top = max_bits(top, magnitude(y[i][e]));
            }
        }
    }
    const float scale = scale_of(row_max<WPR>(top, sh));
    if (t == 0) a.scale[row] = scale;
    unsigned char* y8 = (unsigned char*)a.y + row * W;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c < W) {
            Unit<unsigned char, V> o;
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const unsigned p = pk8(quotient(y[i][e], scale), V > 1 ? quotient(y[i][e + (V > 1)], scale) : 0.f);
                o.v[e] = (unsigned char)p;
                if (V > 1) o.v[e + (V > 1)] = (unsigned char)(p >> 8);
            }
            *(Unit<unsigned char, V>*)(y8 + c) = o;
        }
    }
}

// Rows too wide for registers: one workgroup per row, reading it again for
// each pass.  A thread only reads back what it wrote itself (h may be x or
// residual).
template <typename T>
__global__ __launch_bounds__(1024) void norm_fwd_wide_kernel(NormArgs a) {
    __shared__ float sh[16];
    const int64_t row = group_index();
    if (row >= a.rows) return;
    const int W = (int)a.width;
    const T* x = (const T*)a.x + row * W;
    const T* res = a.residual ? (const T*)a.residual + row * W : nullptr;
    T* h = (T*)a.h + row * W;
    float ss = 0.f;
    for (int c = threadIdx.x; c < W; c += 1024) {
        T u = x[c];
        if (res) {
            u = (T)((float)u + (float)res[c]);
            h[c] = u;
        }
        ss = __builtin_fmaf((float)u, (float)u, ss);
    }
    const T* u = res ? h : x;
    ss = row_sum<16>(ss, sh);
    const float rstd = rsqrtf(ss / (float)W + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (!a.bits8) {
        for (int c = threadIdx.x; c < W; c += 1024) ((T*)a.y)[row * W + c] = (T)((float)u[c] * rstd * a.weight[c]);
        return;
    }
    unsigned top = 0;
    for (int c = threadIdx.x; c < W; c += 1024) top = max_bits(top, magnitude((float)u[c] * rstd * a.weight[c]));
    const float scale = scale_of(row_max<16>(top, sh));
    if (threadIdx.x == 0) a.scale[row] = scale;
    for (int c = threadIdx.x; c < W; c += 1024)
        ((unsigned char*)a.y)[row * W + c] = (unsigned char)pk8(quotient(((float)u[c] * rstd) * a.weight[c], scale), 0.f);
}

// Gradients with the row in registers.  A wave (WPR = 1) or workgroup walks
// rows; dweight sums stay in registers.
template <typename T, int V, int WPR, int NV>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormBwdArgs a) {
    constexpr int TPR = 64 * WPR;
    __shared__ float sh[16];
    __shared__ float comb[WPR == 1 ? 4 * 64 * NV * V : 1];
    const int wave = threadIdx.x >> 6, t = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int W = (int)a.width;
    using U = Unit<T, V>;
    float dw[NV][V] = {};
    float w[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) w[i][e] = c + e < W ? a.weight[c + e] : 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * (WPR == 1 ? 4 : 1);
    for (int64_t row = WPR == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x; row < a.rows; row += step) {
        const T* dyp = (const T*)a.dy + row * W;
        const T* hp = (const T*)a.h + row * W;
        const T* dhp = a.dh ? (const T*)a.dh + row * W : nullptr;
        U dy[NV], h[NV], dh[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c < W) {
                dy[i] = *(const U*)(dyp + c);
                h[i] = *(const U*)(hp + c);
                if (dhp) dh[i] = *(const U*)(dhp + c);
            }
        }
        const float rstd = a.rstd[row];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c < W) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (float)h[i].v[e] * rstd, d = (float)dy[i].v[e];
                    s = __builtin_fmaf(d * w[i][e], xh, s);
                    dw[i][e] = __builtin_fmaf(d, xh, dw[i][e]);
                }
            }
        }
        s = row_sum<WPR>(s, sh) / (float)W;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c < W) {
                U o;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (float)h[i].v[e] * rstd;
                    float d = rstd * ((float)dy[i].v[e] * w[i][e] - xh * s);
                    if (dhp) d += (float)dh[i].v[e];
                    o.v[e] = (T)d;
                }
                *(U*)((T*)a.dx + row * W + c) = o;
            }
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * W;
    if constexpr (WPR == 1) {  // the workgroup's four waves together, in order
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) comb[(wave * NV * V + i * V + e) * 64 + t] = dw[i][e];
        __syncthreads();
        for (int k = wave; k < NV * V; k += 4) {
            const int c = ((k / V) * 64 + t) * V + k % V;
            if (c < W) {
                float x = 0.f;
#pragma unroll
                for (int v = 0; v < 4; ++v) x += comb[(v * NV * V + k) * 64 + t];
                part[c] = x;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c + e < W) part[c + e] = dw[i][e];
        }
    }
}

// Rows too wide for registers: dx by one workgroup per row, reading it twice,
// and the weight's partial sums by a thread per column over a slice of rows.
template <typename T>
__global__ __launch_bounds__(1024) void norm_bwd_wide_dx_kernel(NormBwdArgs a) {
    __shared__ float sh[16];
    const int64_t row = group_index();
    if (row >= a.rows) return;
    const int W = (int)a.width;
    const T *dy = (const T*)a.dy + row * W, *h = (const T*)a.h + row * W;
    const float rstd = a.rstd[row];
    float s = 0.f;
    for (int c = threadIdx.x; c < W; c += 1024)
        s = __builtin_fmaf((float)dy[c] * a.weight[c], (float)h[c] * rstd, s);
    s = row_sum<16>(s, sh) / (float)W;
    for (int c = threadIdx.x; c < W; c += 1024) {
        float d = rstd * ((float)dy[c] * a.weight[c] - (float)h[c] * rstd * s);
        if (a.dh) d += (float)((const T*)a.dh)[row * W + c];
        ((T*)a.dx)[row * W + c] = (T)d;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_wide_dw_kernel(NormBwdArgs a) {
    const int W = (int)a.width;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= W) return;
    float s = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
        s = __builtin_fmaf((float)((const T*)a.dy)[row * W + c], (float)((const T*)a.h)[row * W + c] * a.rstd[row], s);
    a.part[(int64_t)blockIdx.y * W + c] = s;
}

// dweight[c] = sum over groups of part[group][c]: 16 columns per workgroup, 16
// threads each over the groups.
__global__ __launch_bounds__(256) void norm_dw_sum_kernel(const float* part, float* dweight, int groups, int W) {
    __shared__ float sh[16][17];
    const int cc = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + cc;
    float s = 0.f;
    if (c < W)
#pragma unroll 8
        for (int gi = k; gi < groups; gi += 16) s += part[(int64_t)gi * W + c];
    sh[k][cc] = s;
    __syncthreads();
    if (k == 0 && c < W) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) x += sh[i][cc];
        dweight[c] = x;
    }
}

template <typename T>
constexpr int kVec = 16 / sizeof(T);

template <typename T>
hipError_t norm_forward(const NormArgs& a, hipStream_t s) {
    constexpr int V = kVec<T>;
    const int64_t W = a.width;
    const dim3 per_row = grid_of(a.rows), four = grid_of((a.rows + 3) / 4);
    if (a.vec) {
        if (W <= 64 * V * 4) norm_fwd_kernel<T, V, 1, 4><<<four, dim3(256), 0, s>>>(a);
        else if (W <= 256 * V * 4) norm_fwd_kernel<T, V, 4, 4><<<per_row, dim3(256), 0, s>>>(a);
        else norm_fwd_wide_kernel<T><<<per_row, dim3(1024), 0, s>>>(a);
    } else {
        if (W <= 64 * 16) norm_fwd_kernel<T, 1, 1, 16><<<four, dim3(256), 0, s>>>(a);
        else if (W <= 256 * 16) norm_fwd_kernel<T, 1, 4, 16><<<per_row, dim3(256), 0, s>>>(a);
        else norm_fwd_wide_kernel<T><<<per_row, dim3(1024), 0, s>>>(a);
    }
    return hipGetLastError();
}

// Rows that the register form of the backward holds: 0 none, 1 a wave's, 4 a workgroup's.
template <typename T>
int bwd_waves(int64_t W, bool vec) {
    const int64_t one = vec ? 64 * kVec<T> * 4 : 64 * 16;
    return W <= one ? 1 : (W <= 4 * one ? 4 : 0);
}

template <typename T>
hipError_t norm_backward(const NormBwdArgs& a, hipStream_t s) {
    constexpr int V = kVec<T>;
    const int64_t W = a.width;
    const int groups = norm_bwd_groups(a.rows);
    const int waves = bwd_waves<T>(W, a.vec);
    const dim3 gr(groups), bl(256);
    if (a.rows == 0) {  // an empty sum
        norm_dw_sum_kernel<<<dim3((unsigned)((W + 15) / 16)), bl, 0, s>>>(nullptr, a.dweight, 0, (int)W);
        return hipGetLastError();
    }
    if (waves == 0) {
        norm_bwd_wide_dw_kernel<T><<<dim3((unsigned)((W + 255) / 256), groups), bl, 0, s>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        norm_bwd_wide_dx_kernel<T><<<grid_of(a.rows), dim3(1024), 0, s>>>(a);
    } else if (a.vec) {
        if (waves == 1) norm_bwd_kernel<T, V, 1, 4><<<gr, bl, 0, s>>>(a);
        else norm_bwd_kernel<T, V, 4, 4><<<gr, bl, 0, s>>>(a);
    } else {
        if (waves == 1) norm_bwd_kernel<T, 1, 1, 16><<<gr, bl, 0, s>>>(a);
        else norm_bwd_kernel<T, 1, 4, 16><<<gr, bl, 0, s>>>(a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm_dw_sum_kernel<<<dim3((unsigned)((W + 15) / 16)), bl, 0, s>>>(a.part, a.dweight, groups, (int)W);
    return hipGetLastError();
}

}  // namespace

// Workgroups of the backward, each with its own partial weight gradient: as
// many as keep the chip busy, but few rows' worth of partial sums (forward and
// backward of 16384 rows of 2048: 126 us with 256, 106 with 512, 116 with 1024).
int norm_bwd_groups(int64_t rows) {
    const int64_t g = (rows + 7) / 8;
    return (int)(g < 1 ? 1 : (g > 512 ? 512 : g));
}

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s) {
    return a.f32 ? norm_forward<float>(a, s) : norm_forward<__bf16>(a, s);
}

hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t s) {
    return a.f32 ? norm_backward<float>(a, s) : norm_backward<__bf16>(a, s);
}

}  // namespace e2ttt
