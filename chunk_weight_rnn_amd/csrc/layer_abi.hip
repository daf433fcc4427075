// Host side of the C ABI in include/e2ttt_layer.h: validation (before any
// device call), workspace layout, and dispatch on the caller's stream.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "abi_util.h"
#include "layer_internal.h"

namespace e2ttt {
namespace {

constexpr int64_t kCUs = 256;  // compute units of the MI355X

// Elements from the first to past the last of [n][h][D] with these strides.
int64_t reach(int64_t n, int64_t h, int64_t D, int64_t tok, int64_t head) {
    return n > 0 && h > 0 ? (n - 1) * tok + (h - 1) * head + D : 0;
}

bool stride_ok(int64_t s, int64_t es) { return s >= 0 && s % (16 / es) == 0; }

// Sizes, types and strides.  Limits keep every 32-bit index of the kernels in
// range: row numbers, r G in the division by the group, and a tile's byte
// offsets in the buffer copies, which hold token strides.  Head strides are only
// kept where their products fit in 64 bits.
int attention_desc_status(const e2ttt_attention_desc* d, bool packed_kv) {
    if (!d || d->reserved != 0) return E2TTT_ERR_INVALID_ARG;
    if (d->io_dtype != E2TTT_F32 && d->io_dtype != E2TTT_BF16) return E2TTT_ERR_INVALID_ARG;
    if (d->window < 0 || d->tokens < 0 || d->seqs < 0) return E2TTT_ERR_INVALID_ARG;
    if (d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads || d->D < 1) return E2TTT_ERR_INVALID_ARG;
    if (!(d->scale > 0.f) || !isfinite(d->scale)) return E2TTT_ERR_INVALID_ARG;
    if (d->D % 8 || d->D > 128) return E2TTT_ERR_UNSUPPORTED;
    const int64_t es = elem(d->io_dtype), lim[2] = {(int64_t)1 << 23, (int64_t)1 << 40};  // token, head
    if (d->heads > 65536 || d->seqs >= (1 << 28) || d->tokens > 0x7fffffff) return E2TTT_ERR_UNSUPPORTED;
    const int64_t st[6] = {d->q_tok, d->q_head, d->k_tok, d->k_head, d->v_tok, d->v_head};
    const int64_t sizes[6] = {d->tokens, d->heads, d->tokens, d->kv_heads, d->tokens, d->kv_heads};
    for (int i = 0; i < (packed_kv ? 6 : 2); ++i)  // the stride of a dimension of one is never used
        if (sizes[i] > 1 && !stride_ok(st[i], es)) return E2TTT_ERR_INVALID_ARG;
    if (d->tokens > 1 && (d->q_tok < d->D || (packed_kv && (d->k_tok < d->D || d->v_tok < d->D))))
        return E2TTT_ERR_INVALID_ARG;
    for (int i = 0; i < (packed_kv ? 6 : 2); ++i)
        if (sizes[i] > 1 && st[i] > lim[i % 2]) return E2TTT_ERR_UNSUPPORTED;
    const int64_t G = d->heads / d->kv_heads;
    if ((d->tokens + 256) * d->heads > 0x7fffffff) return E2TTT_ERR_UNSUPPORTED;
    if ((d->tokens + 256) * G >= ((int64_t)1 << 32) / G) return E2TTT_ERR_UNSUPPORTED;
    return E2TTT_OK;
}

// `es`: bytes of the cache's elements.
int paged_desc_status(const e2ttt_paged_desc* d, bool append, int64_t es) {
    if (!d) return E2TTT_ERR_INVALID_ARG;
    const int st = attention_desc_status(&d->a, append);
    if (st != E2TTT_OK) return st;
    if (d->pages < 0 || d->table_width < 0 || d->page_size < 1 || (d->page_size & (d->page_size - 1)))
        return E2TTT_ERR_INVALID_ARG;
    const int64_t D = d->a.D;
    const int64_t s[6] = {d->kc_page, d->kc_head, d->kc_slot, d->vc_page, d->vc_head, d->vc_slot};
    const int64_t n[3] = {d->pages, d->a.kv_heads, d->page_size}, lim[3] = {1 << 30, (int64_t)1 << 40, 1 << 23};
    for (int i = 0; i < 6; ++i)  // slots that the call writes must not overlap
        if (n[i % 3] > 1 && (!stride_ok(s[i], es) || s[i] < D)) return E2TTT_ERR_INVALID_ARG;
    for (int i = 0; i < 6; ++i)
        if (n[i % 3] > 1 && s[i] > lim[i % 3]) return E2TTT_ERR_UNSUPPORTED;  // 32-bit factors of the kernels
    if (d->pages > 0x7fffffff || d->page_size > (1 << 24)) return E2TTT_ERR_UNSUPPORTED;
    if (d->table_width > 0x7fffffff || d->table_width * d->page_size + d->a.tokens + 256 > 0x7fffffff)
        return E2TTT_ERR_UNSUPPORTED;
    return E2TTT_OK;
}

int paged_desc_status(const e2ttt_paged_desc* d, bool append) {
    return paged_desc_status(d, append, d ? elem(d->a.io_dtype) : 1);
}

int paged8_desc_status(const e2ttt_paged_desc* d, bool append) {
    const int st = paged_desc_status(d, append, 1);
    if (st != E2TTT_OK) return st;
    return d->a.io_dtype != E2TTT_BF16 || d->a.D % 16 ? E2TTT_ERR_UNSUPPORTED : E2TTT_OK;
}

AttnArgs make_args(const e2ttt_attention_desc& d) {
    AttnArgs a{};
    a.N = d.tokens;
    a.S = (int)d.seqs;
    a.H = (int)d.heads;
    a.K = (int)d.kv_heads;
    a.G = a.H / a.K;
    a.D = (int)d.D;
    a.gmagic = (unsigned)(((uint64_t)1 << 32) / a.G + 1);
    a.window = d.window;
    a.sl2 = d.scale * 1.4426950408889634f;
    // Such tokens are rare, and their number is only known on the device: enough
    // workgroups to write rows at some TB/s, and too few to notice where there are none.
    const int64_t units = (d.tokens * d.heads * d.D * elem(d.io_dtype) / 16 + 255) / 256;
    a.clear = (int)(units < 64 ? units : 64);
    a.q_tok = d.q_tok;
    a.q_head = d.q_head;
    a.k_tok = d.k_tok;
    a.k_head = d.k_head;
    a.v_tok = d.v_tok;
    a.v_head = d.v_head;
    if (a.N == 1) a.q_tok = a.k_tok = a.v_tok = a.D;  // strides of a dimension of one are not checked
    return a;
}

// Row tiles and key ranges.  Where the row tiles alone would leave compute
// units idle, the keys of each are split into ranges of at least 256 that run
// side by side; about two workgroups per compute unit are wanted.
void plan(AttnArgs& a, bool f32, int64_t longest) {
    const int bm = f32 ? kF32Rows : kFwdRows;
    a.ntiles = (int)(a.N * a.G / bm + a.S);
    a.nsplit = 1;
    const int64_t items = (a.N * a.G + bm - 1) / bm * a.K;  // at least so many do work
    const int64_t seen = (int64_t)a.window + bm / a.G + 64;  // positions that a tile's rows see, at most
    if (a.window > 0 && longest > seen) longest = seen;
    if (items > 0 && items < kCUs) {
        // 8 chunks of up to 256 tokens over a window of 2048, 208 tiles: 76 us
        // whole, 56 in 2 ranges, 46 in 3, 52 in 4 (and 9 for the join); one
        // chunk at 16K, 32 tiles: 67 us in 8, 51 in 16, 65 in 20
        int64_t n = (2 * kCUs + items - 1) / items;
        const int64_t most = (longest + 255) / 256;
        if (n > most) n = most;
        a.nsplit = (int)(n < 1 ? 1 : (n > 32 ? 32 : n));
    }
}

// A paged call of few rows per sequence on average goes to the decoding kernel
// (bf16), which needs one launch where no context can be longer than
// kOneLaunch keys, and two where the keys are shared out.  Where the two cross
// depends on how many sequences there are (one token each, 16 heads of 128 over 4,
// us in one launch and in two): one sequence at 512 keys 12.7 and 12.8, at 640 14.7
// and 12.9, at 1000 19.6 and 12.3; 16 sequences at 640 14.7 and 18.5, at 700 16.5
// and 15.1, at 1000 19.7 and 16.4; 64 at 640 19.0 and 23.0, at 1000 25.2 and 29.1.
constexpr int64_t kOneLaunch = 640;
// Over a cache in 8 bits (with the launch that writes the new token), one sequence and
// 16: at 250 keys 11.8 and 13.5, 12.5 and 14.3, at 380 13.9 and 13.4, 14.9 and 14.4, at 500
// 16.1 and 13.4, 16.9 and 14.5; 64, whose items are a workgroup for every compute unit: at
// 500 18.4 and 20.3, at 760 24.1 and 25.3, at 1000 28.6 and 27.7.
constexpr int64_t kOneLaunch8 = 384, kOneLaunch8Full = 768;
void plan_paged(AttnArgs& a, bool f32, bool bits8, int64_t longest) {
    const int64_t units = (longest + a.N + 127) / 128, tiles = a.N * a.G / 32 + a.S;
    if (!f32 && a.N * a.G <= 32 * (int64_t)a.S && tiles * a.K <= 0x7fffffff / (units + 1)) {
        a.decode = 1;
        a.ntiles = (int)tiles;
        if (a.window > 0 && longest > (int64_t)a.window + 64) longest = (int64_t)a.window + 64;
        const int64_t one = !bits8 ? kOneLaunch : tiles * a.K < kDecodeGroups ? kOneLaunch8 : kOneLaunch8Full;
        a.nsplit = longest <= one ? 1 : 2;
        a.shares = bits8 ? kDecode8Groups : kDecodeGroups;
        return;
    }
    plan(a, f32, longest);
}

size_t partial_rows(const AttnArgs& a) {
    return a.decode ? (size_t)2 * a.shares * 32 : (size_t)a.nsplit * a.N * a.H;
}

size_t split_bytes(const AttnArgs& a) {
    if (a.nsplit == 1) return 0;
    const size_t rows = partial_rows(a);
    return (rows * a.D * 4 + kWsAlign - 1) / kWsAlign * kWsAlign + rows * 4;
}

void set_split(AttnArgs& a, void* ws) {
    if (a.nsplit == 1) return;
    const size_t rows = partial_rows(a);
    a.po = (float*)ws;
    a.pl = (float*)((char*)ws + (rows * a.D * 4 + kWsAlign - 1) / kWsAlign * kWsAlign);
}

int launch_status(hipError_t e) {
    if (e == hipErrorInvalidConfiguration) return E2TTT_ERR_UNSUPPORTED;  // kMaxGroups
    return e == hipSuccess ? E2TTT_OK : E2TTT_ERR_HIP;
}

int run_forward(AttnArgs& a, bool f32, hipStream_t s) {
    if (a.decode) return launch_status(launch_attn_decode_bf16(a, s));
    hipError_t e = f32 ? launch_attn_fwd_f32(a, s) : launch_attn_fwd_bf16(a, s);
    if (e == hipSuccess && a.nsplit > 1) e = launch_attn_join(a, f32, s);  // split calls have few rows
    return launch_status(e);
}

// All launches of a call, before the first of them: the cache is not extended by a
// call that is refused.
bool grids8_ok(const AttnArgs& a) {
    const int64_t items = (int64_t)a.ntiles * a.K, append = (2 * a.N * a.K + kAppend8Rows - 1) / kAppend8Rows;
    const int64_t attend = (a.decode ? (a.nsplit > 1 ? a.shares : items) : items * a.nsplit) + a.clear;
    return items <= kMaxGroups && attend <= kMaxGroups && append <= kMaxGroups && (a.N * a.H + 7) / 8 <= kMaxGroups;
}

int run_forward8(AttnArgs& a, hipStream_t s) {
    if (!grids8_ok(a)) return E2TTT_ERR_UNSUPPORTED;
    if (a.pg.append) {
        const hipError_t e = launch_append8(a, s);
        if (e != hipSuccess) return launch_status(e);
        a.pg.append = 0;
    }
    if (a.decode) return launch_status(launch_attn_decode8(a, s));
    hipError_t e = launch_attn_fwd8(a, s);
    if (e == hipSuccess && a.nsplit > 1) e = launch_attn_join(a, false, s);
    return launch_status(e);
}

bool norm_desc_ok(const e2ttt_norm_desc* d) {
    return d && d->reserved == 0 && (d->io_dtype == E2TTT_F32 || d->io_dtype == E2TTT_BF16) &&
           (d->bits8 == 0 || d->bits8 == 1) && d->rows >= 0 && d->width >= 1 && d->eps >= 0.f && isfinite(d->eps);
}

// Whether every row starts on 16 bytes in all of these (null ones do not count).
int norm_rows_aligned(const e2ttt_norm_desc* d, std::initializer_list<const void*> ps) {
    bool ok = d->width * elem(d->io_dtype) % 16 == 0;
    for (const void* p : ps) ok = ok && (uintptr_t)p % 16 == 0;
    return ok;
}

bool norm_supported(const e2ttt_norm_desc* d) { return d->width <= 65536 && d->rows <= 0x7fffffff; }

int scan_desc_status(const e2ttt_scan_desc* d) {
    if (!d) return E2TTT_ERR_INVALID_ARG;
    if (d->io_dtype != E2TTT_F32 && d->io_dtype != E2TTT_BF16) return E2TTT_ERR_INVALID_ARG;
    if (d->gate_dtype != E2TTT_F32 && d->gate_dtype != d->io_dtype) return E2TTT_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->seqs < 0 || d->width < 1) return E2TTT_ERR_INVALID_ARG;
    if (d->tokens > 1 && (d->x_tok < d->width || d->a_tok < d->width)) return E2TTT_ERR_INVALID_ARG;
    // offsets within a sequence are 32-bit, and so is a tile past its end
    if (d->tokens > 0x7fffffff - 4096 || d->seqs >= (1 << 28) || d->width > (1 << 24)) return E2TTT_ERR_UNSUPPORTED;
    const int64_t lim = (int64_t)1 << 31;
    if (d->tokens > 1 && (d->x_tok > lim || d->a_tok > lim)) return E2TTT_ERR_UNSUPPORTED;
    return E2TTT_OK;
}

// Slabs and workgroups.
ScanArgs scan_plan(const e2ttt_scan_desc& d, bool backward) {
    ScanArgs a{};
    a.N = d.tokens;
    a.C = d.width;
    a.S = (int)d.seqs;
    a.x_f32 = d.io_dtype == E2TTT_F32;
    a.gate_f32 = d.gate_dtype == E2TTT_F32;
    a.x_tok = d.tokens > 1 ? d.x_tok : d.width;
    a.a_tok = d.tokens > 1 ? d.a_tok : d.width;
    const int64_t slabs = (d.width + 63) / 64;
    a.slabs = (int)slabs;
    // A wave per sequence while they have 16 tokens at most on average, or 4 where no
    // sequence can have two tiles, so that there are no words to clear (2048 channels, us so and with a
    // workgroup per tile: 64 sequences of one token 2.5 and 12.9, of 16 5.9 and 20, 256 of 16
    // 13 and 64; 8 of 4 2.6 and 4.2, of 16 4.9 and 4.2).  Longer ones gain as well where
    // all are alike (64 of 48: 14 and 22).  Single long ones among them are taken by whole
    // workgroups of the same launch.
    a.shorts = !backward && d.tokens <= (d.tokens > E2TTT_SCAN_TILE ? 16 : 4) * d.seqs;
    const int64_t groups = (a.shorts ? d.seqs : d.tokens / E2TTT_SCAN_TILE + d.seqs) * slabs;
    a.groups = (int)(groups < kMaxScanGroups ? groups : kMaxScanGroups + 1);
    const int64_t units = (d.tokens * d.width + 2047) / 2048;
    a.clear = (int)(units < 64 ? units : 64);
    return a;
}

size_t scan_bytes(const e2ttt_scan_desc& d, bool backward) {
    if (d.tokens <= E2TTT_SCAN_TILE || scan_plan(d, backward).shorts) return 0;
    return (size_t)scan_words(d.tokens, d.seqs, d.width) * 8;
}

}  // namespace
}  // namespace e2ttt

using namespace e2ttt;

extern "C" {

size_t e2ttt_attention_workspace_size(const e2ttt_attention_desc* d) {
    if (attention_desc_status(d, true) != E2TTT_OK) return kBad;
    AttnArgs a = make_args(*d);
    plan(a, d->io_dtype == E2TTT_F32, d->tokens);
    return split_bytes(a);
}

int e2ttt_attention_forward(const e2ttt_attention_desc* d, const void* q, const void* k, const void* v,
                            const int32_t* cu, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const int st = attention_desc_status(d, true);
    if (st != E2TTT_OK) return st;
    if (d->tokens == 0 || d->seqs == 0) return E2TTT_OK;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu, 4) ||
        (lse && !aligned(lse, 4)))
        return E2TTT_ERR_INVALID_ARG;
    const bool f32 = d->io_dtype == E2TTT_F32;
    const int64_t es = elem(d->io_dtype), N = d->tokens, H = d->heads, K = d->kv_heads, D = d->D;
    AttnArgs a = make_args(*d);
    plan(a, f32, N);
    const size_t need = split_bytes(a);
    const int wst = workspace_status(ws, ws_bytes, need);
    if (wst != E2TTT_OK) return wst;
    const Span in[4] = {span(q, es * reach(N, H, D, d->q_tok, d->q_head)), span(k, es * reach(N, K, D, d->k_tok, d->k_head)),
                        span(v, es * reach(N, K, D, d->v_tok, d->v_head)), span(cu, 4 * (d->seqs + 1))};
    const Span outs[3] = {span(out, es * N * H * D), span(lse, 4 * N * H), span(ws, (int64_t)need)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.lse = lse;
    a.cu = cu;
    set_split(a, ws);
    return run_forward(a, f32, (hipStream_t)stream);
}

static size_t stats_bytes(const e2ttt_attention_desc& d) {
    return ((size_t)(d.tokens * d.heads) * 8 + kWsAlign - 1) / kWsAlign * kWsAlign;
}

size_t e2ttt_attention_backward_workspace_size(const e2ttt_attention_desc* d) {
    if (attention_desc_status(d, true) != E2TTT_OK) return kBad;
    const size_t stats = stats_bytes(*d);
    if (d->io_dtype != E2TTT_F32) return stats;
    int dq, dkv;
    attn_f32_parts(d->tokens, d->heads / d->kv_heads, d->kv_heads, d->D, &dq, &dkv);
    return stats + 4 * (size_t)(d->tokens * d->D) * ((dq > 1 ? dq * d->heads : 0) + (dkv > 1 ? 2 * dkv * d->kv_heads : 0));
}

int e2ttt_attention_backward(const e2ttt_attention_desc* d, const void* q, const void* k, const void* v,
                             const void* out, const float* lse, const void* dout, const int32_t* cu, void* dq,
                             void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
    const int st = attention_desc_status(d, true);
    if (st != E2TTT_OK) return st;
    if (d->tokens == 0 || d->seqs == 0) return E2TTT_OK;
    const void* const ps[8] = {q, k, v, out, dout, dq, dk, dv};
    for (const void* p : ps)
        if (!aligned(p, 16)) return E2TTT_ERR_INVALID_ARG;
    if (!aligned(cu, 4) || !aligned(lse, 4)) return E2TTT_ERR_INVALID_ARG;
    const size_t need = e2ttt_attention_backward_workspace_size(d);
    const int wst = workspace_status(ws, ws_bytes, need);
    if (wst != E2TTT_OK) return wst;
    const int64_t es = elem(d->io_dtype), N = d->tokens, H = d->heads, K = d->kv_heads, D = d->D;
    const Span in[7] = {span(q, es * reach(N, H, D, d->q_tok, d->q_head)), span(k, es * reach(N, K, D, d->k_tok, d->k_head)),
                        span(v, es * reach(N, K, D, d->v_tok, d->v_head)), span(out, es * N * H * D),
                        span(lse, 4 * N * H), span(dout, es * N * H * D), span(cu, 4 * (d->seqs + 1))};
    const Span outs[4] = {span(dq, es * N * H * D), span(dk, es * N * K * D), span(dv, es * N * K * D),
                          span(ws, (int64_t)need)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    const AttnArgs f = make_args(*d);
    AttnBwdArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.dout = dout;
    a.lse = lse;
    a.cu = cu;
    a.q_tok = f.q_tok;
    a.q_head = f.q_head;
    a.k_tok = f.k_tok;
    a.k_head = f.k_head;
    a.v_tok = f.v_tok;
    a.v_head = f.v_head;
    a.N = N;
    a.S = f.S;
    a.H = f.H;
    a.K = f.K;
    a.G = f.G;
    a.D = f.D;
    a.gmagic = f.gmagic;
    a.window = f.window;
    a.sl2 = f.sl2;
    a.scale = d->scale;
    a.clear = f.clear;
    a.stats = (float*)ws;
    attn_f32_parts(N, f.G, K, D, &a.dq_parts, &a.dkv_parts);
    a.part = (float*)((char*)ws + stats_bytes(*d));
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    const hipError_t e = d->io_dtype == E2TTT_F32 ? launch_attn_bwd_f32(a, (hipStream_t)stream)
                                                  : launch_attn_bwd_bf16(a, (hipStream_t)stream);
    return launch_status(e);
}

static size_t paged_bytes(const e2ttt_paged_desc* d, bool bits8) {
    AttnArgs a = make_args(d->a);
    plan_paged(a, d->a.io_dtype == E2TTT_F32, bits8, d->table_width * d->page_size);
    return split_bytes(a);
}

size_t e2ttt_paged_workspace_size(const e2ttt_paged_desc* d) {
    return paged_desc_status(d, false) == E2TTT_OK ? paged_bytes(d, false) : kBad;
}

// bits8: a cache of one-byte elements, with a scale per slot and head.
static int paged_attention(const e2ttt_paged_desc* d, bool bits8, const void* q, const void* k, const void* v, void* k_cache,
                           void* v_cache, void* k_scale, void* v_scale, const int32_t* table, const int32_t* cu,
                           const int32_t* cached, void* out, void* ws, size_t ws_bytes, void* stream) {
    const bool append = k || v;
    const int st = bits8 ? paged8_desc_status(d, append) : paged_desc_status(d, append);
    if (st != E2TTT_OK) return st;
    const int64_t N = d->a.tokens, S = d->a.seqs, H = d->a.heads, K = d->a.kv_heads, D = d->a.D;
    if (N == 0 || S == 0) return E2TTT_OK;
    if (append && (!aligned(k, 16) || !aligned(v, 16))) return E2TTT_ERR_INVALID_ARG;  // both or neither
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cu, 4) || !aligned(cached, 4)) return E2TTT_ERR_INVALID_ARG;
    if (d->pages > 0 && (!aligned(k_cache, 16) || !aligned(v_cache, 16))) return E2TTT_ERR_INVALID_ARG;
    if (d->table_width > 0 && !aligned(table, 4)) return E2TTT_ERR_INVALID_ARG;
    const bool f32 = d->a.io_dtype == E2TTT_F32;
    AttnArgs a = make_args(d->a);
    plan_paged(a, f32, bits8, d->table_width * d->page_size);
    if (bits8 && d->pages > 0 && (!k_scale || !v_scale)) return E2TTT_ERR_INVALID_ARG;
    const size_t need = split_bytes(a);
    const int wst = workspace_status(ws, ws_bytes, need);
    if (wst != E2TTT_OK) return wst;
    const int64_t es = elem(d->a.io_dtype), cs = bits8 ? 1 : es, P = d->pages, ps = d->page_size;
    const Span kc = span(k_cache, P > 0 ? cs * ((P - 1) * d->kc_page + (K - 1) * d->kc_head + (ps - 1) * d->kc_slot + D) : 0);
    const Span vc = span(v_cache, P > 0 ? cs * ((P - 1) * d->vc_page + (K - 1) * d->vc_head + (ps - 1) * d->vc_slot + D) : 0);
    const Span in[6] = {span(q, es * reach(N, H, D, d->a.q_tok, d->a.q_head)),
                        append ? span(k, es * reach(N, K, D, d->a.k_tok, d->a.k_head)) : Span{},
                        append ? span(v, es * reach(N, K, D, d->a.v_tok, d->a.v_head)) : Span{},
                        span(table, 4 * S * d->table_width), span(cu, 4 * (S + 1)), span(cached, 4 * S)};
    const Span outs[2] = {span(out, es * N * H * D), span(ws, (int64_t)need)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    const Span scales[2] = {span(k_scale, bits8 ? P * K * ps : 0), span(v_scale, bits8 ? P * K * ps : 0)};
    const Span caches[4] = {kc, vc, scales[0], scales[1]};  // one tensor may hold both, interleaved
    for (const Span& c : caches) {
        for (const Span& o : outs)
            if (c.meets(o)) return E2TTT_ERR_ALIAS;
        for (const Span& i : in)
            if (c.meets(i)) return E2TTT_ERR_ALIAS;
    }
    if (scales[0].meets(scales[1])) return E2TTT_ERR_ALIAS;
    for (const Span& s : scales)
        if (s.meets(kc) || s.meets(vc)) return E2TTT_ERR_ALIAS;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.cu = cu;
    // an empty pool: a non-null address selects the paged kernel, no page index is inside the pool
    a.pg.kc = k_cache ? k_cache : out;
    a.pg.vc = v_cache ? v_cache : out;
    a.pg.k_page = d->kc_page;
    a.pg.k_head = d->kc_head;
    a.pg.k_slot = d->kc_slot;
    a.pg.v_page = d->vc_page;
    a.pg.v_head = d->vc_head;
    a.pg.v_slot = d->vc_slot;
    if (P == 1) a.pg.k_page = a.pg.v_page = 0;  // strides of a dimension of one are not checked
    if (ps == 1) a.pg.k_slot = a.pg.v_slot = 0;
    a.pg.table = table;
    a.pg.cached = cached;
    a.pg.wide = (int)d->table_width;
    a.pg.pages = (int)P;
    a.pg.append = append;
    while ((int64_t)1 << a.pg.shift < ps) ++a.pg.shift;
    a.pg.ks = (unsigned char*)(P > 0 ? k_scale : nullptr);
    a.pg.vs = (unsigned char*)(P > 0 ? v_scale : nullptr);
    set_split(a, ws);
    return bits8 ? run_forward8(a, (hipStream_t)stream) : run_forward(a, f32, (hipStream_t)stream);
}

int e2ttt_paged_attention(const e2ttt_paged_desc* d, const void* q, const void* k, const void* v, void* k_cache,
                          void* v_cache, const int32_t* table, const int32_t* cu, const int32_t* cached, void* out,
                          void* ws, size_t ws_bytes, void* stream) {
    return paged_attention(d, false, q, k, v, k_cache, v_cache, nullptr, nullptr, table, cu, cached, out, ws, ws_bytes, stream);
}

size_t e2ttt_paged8_workspace_size(const e2ttt_paged_desc* d) {
    return paged8_desc_status(d, false) == E2TTT_OK ? paged_bytes(d, true) : kBad;
}

int e2ttt_paged8_attention(const e2ttt_paged_desc* d, const void* q, const void* k, const void* v, void* k_cache,
                           void* v_cache, void* k_scale, void* v_scale, const int32_t* table, const int32_t* cu,
                           const int32_t* cached, void* out, void* ws, size_t ws_bytes, void* stream) {
    return paged_attention(d, true, q, k, v, k_cache, v_cache, k_scale, v_scale, table, cu, cached, out, ws, ws_bytes, stream);
}

int e2ttt_norm_forward(const e2ttt_norm_desc* d, const void* x, const void* residual, const float* weight, void* y,
                       float* scale, void* h, float* rstd, void* stream) {
    if (!norm_desc_ok(d)) return E2TTT_ERR_INVALID_ARG;
    if (!norm_supported(d)) return E2TTT_ERR_UNSUPPORTED;
    if (d->rows == 0) return E2TTT_OK;
    if ((residual == nullptr) != (h == nullptr)) return E2TTT_ERR_INVALID_ARG;
    const size_t es = elem(d->io_dtype);
    if (!aligned(x, es) || !aligned(weight, 4) || !aligned(y, d->bits8 ? 1 : es)) return E2TTT_ERR_INVALID_ARG;
    if (residual && (!aligned(residual, es) || !aligned(h, es))) return E2TTT_ERR_INVALID_ARG;
    if (d->bits8 ? !aligned(scale, 4) : scale != nullptr) return E2TTT_ERR_INVALID_ARG;
    if (rstd && !aligned(rstd, 4)) return E2TTT_ERR_INVALID_ARG;
    const int64_t n = d->rows * d->width, b = n * es;
    const Span xs = span(x, b), rs = span(residual, b), hs = span(h, b);
    const Span in[3] = {h == x ? Span{} : xs, h == residual ? Span{} : rs, span(weight, 4 * d->width)};
    const Span outs[4] = {hs, span(y, d->bits8 ? n : b), span(scale, 4 * d->rows), span(rstd, 4 * d->rows)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    NormArgs a{x, residual, weight, y, scale, h, rstd, d->rows, d->width, d->eps, d->io_dtype == E2TTT_F32, d->bits8,
               norm_rows_aligned(d, {x, residual, weight, y, h})};
    return launch_norm_forward(a, (hipStream_t)stream) == hipSuccess ? E2TTT_OK : E2TTT_ERR_HIP;
}

size_t e2ttt_norm_backward_workspace_size(const e2ttt_norm_desc* d) {
    if (!norm_desc_ok(d) || !norm_supported(d)) return kBad;
    return d->rows == 0 ? 0 : (size_t)norm_bwd_groups(d->rows) * d->width * 4;
}

int e2ttt_norm_backward(const e2ttt_norm_desc* d, const void* dy, const void* h, const float* weight,
                        const float* rstd, const void* dh, void* dx, float* dweight, void* ws, size_t ws_bytes,
                        void* stream) {
    if (!norm_desc_ok(d) || d->bits8) return E2TTT_ERR_INVALID_ARG;
    if (!norm_supported(d)) return E2TTT_ERR_UNSUPPORTED;
    if (!aligned(dweight, 4)) return E2TTT_ERR_INVALID_ARG;
    const size_t es = elem(d->io_dtype);
    const int64_t b = d->rows * d->width * es;
    if (d->rows > 0) {
        if (!aligned(dy, es) || !aligned(h, es) || !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(dx, es) ||
            (dh && !aligned(dh, es)))
            return E2TTT_ERR_INVALID_ARG;
        const size_t need = e2ttt_norm_backward_workspace_size(d);
        const int wst = workspace_status(ws, ws_bytes, need);
        if (wst != E2TTT_OK) return wst;
        const Span in[5] = {span(dy, b), span(h, b), span(weight, 4 * d->width), span(rstd, 4 * d->rows),
                            dx == dh ? Span{} : span(dh, b)};
        const Span outs[3] = {span(dx, b), span(dweight, 4 * d->width), span(ws, (int64_t)need)};
        const int ast = alias_status(in, outs);
        if (ast != E2TTT_OK) return ast;
    }
    NormBwdArgs a{dy, h, dh, weight, rstd, dx, dweight, (float*)ws, d->rows, d->width, d->io_dtype == E2TTT_F32,
                  norm_rows_aligned(d, {dy, h, dh, weight, dx})};
    return launch_norm_backward(a, (hipStream_t)stream) == hipSuccess ? E2TTT_OK : E2TTT_ERR_HIP;
}

size_t e2ttt_scan_workspace_size(const e2ttt_scan_desc* d) {
    return scan_desc_status(d) == E2TTT_OK ? scan_bytes(*d, false) : kBad;
}

int e2ttt_scan_forward(const e2ttt_scan_desc* d, const void* x, const void* a, const float* h0, const int32_t* cu,
                       void* out, float* state, float* starts, void* ws, size_t ws_bytes, void* stream) {
    const int st = scan_desc_status(d);
    if (st != E2TTT_OK) return st;
    if (d->seqs == 0) return E2TTT_OK;
    const size_t es = elem(d->io_dtype), gs = elem(d->gate_dtype);
    const int64_t N = d->tokens, S = d->seqs, C = d->width;
    if (!aligned(cu, 4) || (h0 && !aligned(h0, 4)) || (state && !aligned(state, 4)) || (starts && !aligned(starts, 4)))
        return E2TTT_ERR_INVALID_ARG;
    if (N > 0 && (!aligned(x, es) || !aligned(a, gs) || !aligned(out, es))) return E2TTT_ERR_INVALID_ARG;
    ScanArgs r = scan_plan(*d, false);
    if (r.groups > kMaxScanGroups) return E2TTT_ERR_UNSUPPORTED;
    const size_t need = scan_bytes(*d, false);
    const int wst = workspace_status(ws, ws_bytes, need);
    if (wst != E2TTT_OK) return wst;
    const Span in[4] = {span(x, es * reach(N, 1, C, r.x_tok, 0)), span(a, gs * reach(N, 1, C, r.a_tok, 0)),
                        h0 == state ? Span{} : span(h0, 4 * S * C), span(cu, 4 * (S + 1))};
    const Span outs[4] = {span(out, es * N * C), span(state, 4 * S * C),
                          span(starts, 4 * (N / E2TTT_SCAN_TILE + S) * C), span(ws, (int64_t)need)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    r.x = x;
    r.a = a;
    r.h0 = h0;
    r.cu = cu;
    r.out = out;
    r.state = state;
    r.starts = starts;
    r.words = need ? (unsigned long long*)ws : nullptr;
    return launch_status(launch_scan_forward(r, (hipStream_t)stream));
}

size_t e2ttt_scan_backward_workspace_size(const e2ttt_scan_desc* d) {
    return scan_desc_status(d) == E2TTT_OK ? scan_bytes(*d, true) : kBad;
}

int e2ttt_scan_backward(const e2ttt_scan_desc* d, const void* dout, const void* x, const void* a, const float* starts,
                        const float* dstate, const int32_t* cu, void* dx, void* da, float* dh0, void* ws,
                        size_t ws_bytes, void* stream) {
    const int st = scan_desc_status(d);
    if (st != E2TTT_OK) return st;
    if (d->seqs == 0) return E2TTT_OK;
    const size_t es = elem(d->io_dtype), gs = elem(d->gate_dtype);
    const int64_t N = d->tokens, S = d->seqs, C = d->width;
    if (!aligned(cu, 4) || !aligned(starts, 4) || (dstate && !aligned(dstate, 4)) || (dh0 && !aligned(dh0, 4)))
        return E2TTT_ERR_INVALID_ARG;
    if (N > 0 && (!aligned(x, es) || !aligned(a, gs) || !aligned(dout, es) || !aligned(dx, es) || !aligned(da, gs)))
        return E2TTT_ERR_INVALID_ARG;
    ScanArgs r = scan_plan(*d, true);
    if (r.groups > kMaxScanGroups) return E2TTT_ERR_UNSUPPORTED;
    const size_t need = scan_bytes(*d, true);
    const int wst = workspace_status(ws, ws_bytes, need);
    if (wst != E2TTT_OK) return wst;
    const Span in[6] = {span(x, es * reach(N, 1, C, r.x_tok, 0)), span(a, gs * reach(N, 1, C, r.a_tok, 0)),
                        span(dout, es * N * C), span(starts, 4 * (N / E2TTT_SCAN_TILE + S) * C),
                        span(dstate, 4 * S * C), span(cu, 4 * (S + 1))};
    const Span outs[4] = {span(dx, es * N * C), span(da, gs * N * C), span(dh0, 4 * S * C), span(ws, (int64_t)need)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    r.x = x;
    r.a = a;
    r.h0 = dstate;
    r.cu = cu;
    r.out = dx;
    r.da = da;
    r.dout = dout;
    r.state = dh0;
    r.starts = const_cast<float*>(starts);
    r.words = need ? (unsigned long long*)ws : nullptr;
    return launch_status(launch_scan_backward(r, (hipStream_t)stream));
}

}  // extern "C"
