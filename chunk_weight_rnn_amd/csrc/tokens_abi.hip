// Host side of the C ABI in include/e2ttt_tokens.h: validation (before any
// device call), workspace layout, and dispatch on the caller's stream.
#include <math.h>

#include <initializer_list>

#include "abi_util.h"
#include "tokens_internal.h"

namespace e2ttt {
namespace {

int embedding_desc_status(const e2ttt_embedding_desc* d) {
    if (!d) return E2TTT_ERR_INVALID_ARG;
    for (int t : {d->table_dtype, d->io_dtype})
        if (t != E2TTT_F32 && t != E2TTT_BF16) return E2TTT_ERR_INVALID_ARG;
    if (d->token_bytes != 4 && d->token_bytes != 8) return E2TTT_ERR_INVALID_ARG;
    if (!isfinite(d->scale) || d->tokens < 0 || d->vocab < 1 || d->width < 1) return E2TTT_ERR_INVALID_ARG;
    if (d->vocab > (1 << 24) || d->width > (1 << 20) || d->tokens > 0x7fffffff - 4096) return E2TTT_ERR_UNSUPPORTED;
    return E2TTT_OK;
}

// From `in` of one type to `out` of the other.
EmbedArgs embed_args(const e2ttt_embedding_desc& d, const void* tokens, const void* in, int in_type, void* out, int out_type) {
    EmbedArgs a{};
    a.tokens = tokens;
    a.in = in;
    a.out = out;
    a.N = d.tokens;
    a.W = d.width;
    a.V = (int)d.vocab;
    a.wide = d.token_bytes == 8;
    a.in_f32 = in_type == E2TTT_F32;
    a.out_f32 = out_type == E2TTT_F32;
    const int64_t unit = a.in_f32 && a.out_f32 ? 4 : 8;  // 16 bytes of the smaller type
    a.vec = d.width % unit == 0 && (uintptr_t)in % 16 == 0 && (uintptr_t)out % 16 == 0;
    a.scale = d.scale;
    return a;
}

struct EmbedLayout {  // of the backward's workspace
    size_t order, part, total;
};
EmbedLayout embed_layout(const e2ttt_embedding_desc& d) {
    auto up = [](size_t n) { return (n + kWsAlign - 1) / kWsAlign * kWsAlign; };
    EmbedLayout l;
    l.order = up((size_t)(d.vocab + 1) * 4);
    l.part = l.order + up((size_t)d.tokens * 4);
    // a row of up to kEmbedPiece places is not cut
    const size_t pieces = d.tokens > kEmbedPiece ? (size_t)(d.tokens + kEmbedPiece - 1) / kEmbedPiece : 0;
    l.total = l.part + 2 * pieces * (size_t)d.width * 4;
    return l;
}

int sample_desc_status(const e2ttt_sample_desc* d) {
    if (!d || d->reserved != 0) return E2TTT_ERR_INVALID_ARG;
    if (d->io_dtype != E2TTT_F32 && d->io_dtype != E2TTT_BF16) return E2TTT_ERR_INVALID_ARG;
    if (!(d->temperature >= 0.f) || !isfinite(d->temperature) || !(d->top_p >= 0.f) || !(d->min_p >= 0.f) || d->min_p > 1.f)
        return E2TTT_ERR_INVALID_ARG;
    if (d->rows < 0 || d->vocab < 1 || (d->rows > 1 && d->row_stride < d->vocab)) return E2TTT_ERR_INVALID_ARG;
    if (d->vocab > E2TTT_SAMPLE_VOCAB || d->rows >= (1 << 22) || (d->rows > 1 && d->row_stride > ((int64_t)1 << 40)))
        return E2TTT_ERR_UNSUPPORTED;
    return E2TTT_OK;
}

}  // namespace
}  // namespace e2ttt

using namespace e2ttt;

extern "C" {

int e2ttt_embedding_forward(const e2ttt_embedding_desc* d, const void* tokens, const void* table, void* out, void* stream) {
    const int st = embedding_desc_status(d);
    if (st != E2TTT_OK) return st;
    if (d->tokens == 0) return E2TTT_OK;
    const size_t es = elem(d->io_dtype), ts = elem(d->table_dtype);
    if (!aligned(tokens, d->token_bytes) || !aligned(table, ts) || !aligned(out, es)) return E2TTT_ERR_INVALID_ARG;
    const int64_t N = d->tokens, W = d->width;
    const Span in[2] = {span(tokens, N * d->token_bytes), span(table, ts * d->vocab * W)}, outs[1] = {span(out, es * N * W)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    const EmbedArgs a = embed_args(*d, tokens, table, d->table_dtype, out, d->io_dtype);
    return launch_embedding_forward(a, (hipStream_t)stream) == hipSuccess ? E2TTT_OK : E2TTT_ERR_HIP;
}

size_t e2ttt_embedding_backward_workspace_size(const e2ttt_embedding_desc* d) {
    return embedding_desc_status(d) == E2TTT_OK ? embed_layout(*d).total : kBad;
}

int e2ttt_embedding_backward(const e2ttt_embedding_desc* d, const void* dout, const void* tokens, void* dtable, void* ws,
                             size_t ws_bytes, void* stream) {
    const int st = embedding_desc_status(d);
    if (st != E2TTT_OK) return st;
    const size_t es = elem(d->io_dtype), ts = elem(d->table_dtype);
    if (!aligned(dtable, ts)) return E2TTT_ERR_INVALID_ARG;
    if (d->tokens > 0 && (!aligned(tokens, d->token_bytes) || !aligned(dout, es))) return E2TTT_ERR_INVALID_ARG;
    const EmbedLayout l = embed_layout(*d);
    const int wst = workspace_status(ws, ws_bytes, l.total);
    if (wst != E2TTT_OK) return wst;
    const int64_t N = d->tokens, W = d->width;
    const Span in[2] = {span(tokens, N * d->token_bytes), span(dout, es * N * W)};
    const Span outs[2] = {span(dtable, ts * d->vocab * W), span(ws, (int64_t)l.total)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    EmbedArgs a = embed_args(*d, tokens, dout, d->io_dtype, dtable, d->table_dtype);
    a.start = (int*)ws;
    a.order = (int*)((char*)ws + l.order);
    a.part = (float*)((char*)ws + l.part);
    return launch_embedding_backward(a, (hipStream_t)stream) == hipSuccess ? E2TTT_OK : E2TTT_ERR_HIP;
}

size_t e2ttt_sample_workspace_size(const e2ttt_sample_desc* d) { return sample_desc_status(d) == E2TTT_OK ? 0 : kBad; }

int e2ttt_sample(const e2ttt_sample_desc* d, const void* logits, const float* u, const float* temperature,
                 const int32_t* top_k, const float* top_p, const float* min_p, int64_t* token, float* logprob, void* ws,
                 size_t ws_bytes, void* stream) {
    const int st = sample_desc_status(d);
    if (st != E2TTT_OK) return st;
    if (d->rows == 0) return E2TTT_OK;
    const size_t es = elem(d->io_dtype);
    if (!aligned(logits, es) || !aligned(u, 4) || !aligned(token, 8)) return E2TTT_ERR_INVALID_ARG;
    for (const void* p : {(const void*)temperature, (const void*)top_k, (const void*)top_p, (const void*)min_p, (const void*)logprob})
        if (p && !aligned(p, 4)) return E2TTT_ERR_INVALID_ARG;
    const size_t need = e2ttt_sample_workspace_size(d);
    const int wst = workspace_status(ws, ws_bytes, need);
    if (wst != E2TTT_OK) return wst;
    const int64_t n = d->rows, stride = n > 1 ? d->row_stride : d->vocab;
    const Span in[6] = {span(logits, es * ((n - 1) * stride + d->vocab)), span(u, 4 * n), span(temperature, 4 * n),
                        span(top_k, 4 * n), span(top_p, 4 * n), span(min_p, 4 * n)};
    const Span outs[3] = {span(token, 8 * n), span(logprob, 4 * n), span(ws, (int64_t)need)};
    const int ast = alias_status(in, outs);
    if (ast != E2TTT_OK) return ast;
    const SampleArgs a{logits, u, temperature, top_p, min_p, top_k, token, logprob, n, stride, (int)d->vocab,
                       d->io_dtype == E2TTT_F32, d->temperature, d->top_p, d->min_p, d->top_k};
    return launch_sample(a, (hipStream_t)stream) == hipSuccess ? E2TTT_OK : E2TTT_ERR_HIP;
}

}  // extern "C"
