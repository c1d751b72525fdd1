// checks.h -- host-side argument checks shared by the extern "C" boundaries
// (library-internal).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "internal.h"

namespace ms {

inline bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Span {
    const void* p;
    size_t bytes;
};

// Whether any of `outs` overlaps another of them or any of `ins`.
inline bool overlaps(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    const auto hit = [](const Span& a, const Span& b) {
        if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
        const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
        return x < y + b.bytes && y < x + a.bytes;
    };
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto q = o + 1; q != outs.end(); ++q)
            if (hit(*o, *q)) return true;
        for (const Span& i : ins)
            if (hit(*o, i)) return true;
    }
    return false;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? MOE_SHUFFLE_OK : hip_fail(e); }

}  // namespace ms
