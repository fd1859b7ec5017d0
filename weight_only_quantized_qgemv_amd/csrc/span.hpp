// span.hpp — a row's share of a packed list, from offsets that the caller
// filled on the device and the host cannot check. Plain C++ (constexpr serves
// host and device alike), so that its ends are tested on the CPU.
#pragma once

#include <stdint.h>

namespace qp {

// Entries first .. first + count - 1 of a list.
struct Span {
    uint32_t first, count;
};

// Entries lo .. hi - 1 of a list of len (below 2^31) as far as they are inside
// it, whatever lo and hi are: first + count <= len. An index into the span is
// counted from its first entry, unsigned: below 2^31, so a stride on from it
// does not wrap.
constexpr Span held_span(int32_t lo, int32_t hi, int64_t len)
{
    const int64_t a = lo < 0 ? 0 : lo < len ? lo : len;
    const int64_t b = hi < a ? a : hi < len ? hi : len;
    return Span{(uint32_t)a, (uint32_t)(b - a)};
}

} // namespace qp
