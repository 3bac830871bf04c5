// Host-side argument checks that the operators' C ABI files share.
#pragma once

#include "kda.h"

#include <stdint.h>

#include <initializer_list>

namespace kda {

inline size_t esize(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }
inline bool dtype_ok(kda_dtype dt) { return dt == KDA_F32 || dt == KDA_BF16; }
inline bool act_ok(kda_activation a) { return a == KDA_ACT_NONE || a == KDA_ACT_SILU || a == KDA_ACT_SIGMOID; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// byte ranges [a, a + na) and [b, b + nb) share a byte
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || !na || !nb) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y ? y - x < na : x - y < nb;
}
// The bytes a tensor's token rows take: `rows` rows of `width` bytes, `stride`
// bytes apart.
struct Span {
    const void* p;
    long long rows, stride, width;
};
// Two tensors share a byte.  Rows of one spacing that keep to columns of their
// own (views of one wider buffer) do not.
inline bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const long long na = (a.rows - 1) * a.stride + a.width, nb = (b.rows - 1) * b.stride + b.width;
    if (!overlap(a.p, (size_t)na, b.p, (size_t)nb)) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
        const long long s = a.stride;
        const long long d = (long long)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
        const long long m = ((d % s) + s) % s;      // where b's row starts in a's
        return m < a.width || m + b.width > s;
    }
    return true;
}
inline Span flat_span(const void* p, size_t bytes) { return Span{p, 1, (long long)bytes, (long long)bytes}; }
// an output shares a byte with an input or with another output
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& in : ins)
            if (overlap(*o, in)) return true;
        for (const Span* other = outs.begin(); other != o; ++other)
            if (overlap(*o, *other)) return true;
    }
    return false;
}
// tokens of a call; row indices are int in the kernels
inline bool token_count(const int* cu, int N, int T, long long* M) {
    *M = cu ? (long long)T : (long long)N * T;
    return *M <= 2147483647LL - 4096;
}

}  // namespace kda

#define KDA_LAUNCH(name, call)                                                          \
    do {                                                                                \
        if (profiled(name, stream, [&] { return call; }) != hipSuccess) return KDA_ERR_HIP; \
    } while (0)
