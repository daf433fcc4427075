// Host-side checks that the C ABI's translation units share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/e2ttt.h"

namespace e2ttt {
namespace {

constexpr size_t kWsAlign = 256;
constexpr size_t kBad = (size_t)-1;

struct Span {  // the bytes a tensor reaches; empty for a null or empty one
    uintptr_t lo = 0, hi = 0;
    bool meets(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};

Span span(const void* p, int64_t bytes) {
    Span s;
    if (p && bytes > 0) s = {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
    return s;
}

bool aligned(const void* p, size_t n) { return p && (uintptr_t)p % n == 0; }

int64_t elem(int dtype) { return dtype == E2TTT_BF16 ? 2 : 4; }

int workspace_status(const void* ws, size_t have, size_t need) {
    if (need == 0) return E2TTT_OK;
    return !ws || have < need || (uintptr_t)ws % kWsAlign ? E2TTT_ERR_WORKSPACE : E2TTT_OK;
}

template <int NI, int NO>
int alias_status(const Span (&in)[NI], const Span (&out)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (out[o].meets(in[i])) return E2TTT_ERR_ALIAS;
        for (int p = 0; p < o; ++p)
            if (out[o].meets(out[p])) return E2TTT_ERR_ALIAS;
    }
    return E2TTT_OK;
}

}  // namespace
}  // namespace e2ttt
