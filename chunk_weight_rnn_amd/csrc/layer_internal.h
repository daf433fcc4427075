// Internal declarations of the hybrid layer's operators (include/e2ttt_layer.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/e2ttt_layer.h"

namespace e2ttt {

hipError_t device_cu_count(int* ncu);

// Workgroups of 256 threads in a grid, at most: HIP counts the threads along a
// dimension in 32 bits, and a larger grid wraps around without an error.
// Launchers return hipErrorInvalidConfiguration for it, before they launch.
constexpr int64_t kMaxGroups = (1 << 24) - 1;

// Key/value pages of a paged call; kc == nullptr: packed sequences, no cache.
struct PagedKV {
    void *kc, *vc;                   // pool, written where new tokens are appended
    int64_t k_page, k_head, k_slot;  // strides in elements
    int64_t v_page, v_head, v_slot;
    const int* table;   // [S][wide] page indices
    const int* cached;  // [S] tokens in the cache before the call
    int wide, pages, shift;
    int append;  // keys at positions >= cached come from k / v, and go into the cache
    unsigned char *ks, *vs;  // 8-bit cache: biased exponents of the scales, [pages][K][page size]
};

struct AttnArgs {
    const void *q, *k, *v;
    void* out;
    float* lse;     // [N][H], may be null
    const int* cu;  // [S + 1]
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;  // strides in elements
    int64_t N;
    int S, H, K, G, D;
    unsigned gmagic;  // floor(2^32 / G) + 1: r / G = umulhi(r, gmagic) while r G < 2^32
    int window;       // 0: none
    float sl2;    // scale * log2(e)
    int ntiles;   // row tiles at most, over all sequences
    int nsplit;   // key ranges per row tile; > 1: partial results, joined after
    int decode;   // paged: the kernel for few rows per sequence
    int shares;   // decode, nsplit > 1: workgroups that the keys are shared out over
    int clear;    // workgroups that write the rows of tokens outside every sequence
    float* po;    // [nsplit][N][H][D] partial outputs
    float* pl;    // [nsplit][N][H] their base-2 log sums
    PagedKV pg;
};

constexpr int kFwdRows = 128;  // rows of a tile of the forward, bf16
constexpr int kF32Rows = 16;   // and fp32
hipError_t launch_attn_fwd_bf16(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_fwd_f32(const AttnArgs& a, hipStream_t s);
// Few new tokens per sequence over a paged cache; nsplit > 1: the keys of all
// items shared out evenly over `shares` workgroups, po / pl [2 shares][32][D] /
// [2 shares][32].  One workgroup per compute
// unit: its LDS stages fill one (16 sequences at 2000 keys: 22.0 us, with twice as
// many half as long 27.5; 64 at 12000 the same).
constexpr int kDecodeGroups = 256;
hipError_t launch_attn_decode_bf16(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_decode_join(const AttnArgs& a, hipStream_t s);  // of D up to 128
hipError_t launch_attn_join(const AttnArgs& a, bool f32, hipStream_t s);
// The same over a cache in 8 bits; the new tokens go into it in a launch before.  Two
// workgroups per compute unit, whose stages are half as large.
constexpr int kDecode8Groups = 512;
constexpr int kAppend8Rows = 16;  // rows of keys and values per workgroup
hipError_t launch_append8(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_decode8(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_fwd8(const AttnArgs& a, hipStream_t s);

struct AttnBwdArgs {
    const void *q, *k, *v, *out, *dout;
    const float* lse;
    const int* cu;
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
    int64_t N;
    int S, H, K, G, D;
    unsigned gmagic;
    int window;
    float sl2, scale;
    float* stats;  // [2][N][H] workspace: bf16 -lse / scale and -delta of each row; fp32 delta alone
    void *dq, *dk, *dv;
    // fp32: workgroups that share a tile of rows (dq) or a block of keys (dk, dv);
    // > 1: their sums [dq_parts][N][H][D] and [dkv_parts][2][N][K][D], joined after
    int dq_parts, dkv_parts;
    float* part;
    int clear;  // as in AttnArgs
};
void attn_f32_parts(int64_t N, int64_t G, int64_t K, int64_t D, int* dq, int* dkv);
hipError_t launch_attn_bwd_bf16(const AttnBwdArgs& a, hipStream_t s);
hipError_t launch_attn_bwd_f32(const AttnBwdArgs& a, hipStream_t s);

struct NormArgs {
    const void *x, *residual;  // residual may be null
    const float* weight;
    void* y;  // the stream's type, or 8 bits with a scale per row
    float* scale;
    void* h;  // x + residual in the stream's type (null without residual)
    float* rstd;
    int64_t rows, width;
    float eps;
    int f32, bits8;
    int vec;  // every row of every tensor starts on 16 bytes
};
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s);

struct NormBwdArgs {
    const void *dy, *h, *dh;  // dh may be null
    const float *weight, *rstd;
    void* dx;
    float *dweight, *part;  // part: [norm_bwd_groups][width]
    int64_t rows, width;
    int f32;
    int vec;  // as in NormArgs
};
int norm_bwd_groups(int64_t rows);
hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t s);

struct ScanArgs {
    const void *x, *a;
    const float* h0;  // [S][C] state before a sequence (forward) or gradient after it (backward), may be null
    const int* cu;    // [S + 1]
    void* out;        // [N][C]; backward: dx
    float* state;     // [S][C] state after a sequence, or the gradient before it; may be null
    float* starts;    // states before every E2TTT_SCAN_TILE tokens; forward: may be null
    const void* dout;  // backward
    void* da;
    int64_t x_tok, a_tok;  // strides in elements
    int64_t N, C;
    int S;
    int x_f32, gate_f32;
    int slabs;    // of 64 lanes, over the channels
    int groups;   // (tile or sequence, slab) pairs
    int shorts;   // forward: sequences of a few tokens
    int helpers;  // shorts: workgroups per slab for those that are long all the same
    int clear;    // workgroups that write the rows of tokens outside every sequence
    unsigned long long* words;  // what tiles tell each other, scan_words of them; null where no sequence has two
};
int64_t scan_words(int64_t N, int64_t S, int64_t C);
constexpr int64_t kMaxScanGroups = 1 << 22;  // of 512 threads
hipError_t launch_scan_forward(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s);

}  // namespace e2ttt
