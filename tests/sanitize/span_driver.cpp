// span_driver.cpp — held_span (csrc/span.hpp) at the ends of its arguments: a
// span is inside its list whatever the offsets are, and is the part of lo .. hi
// that the list has. Built for the host alone under
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_span_host.py.
#include <cstdint>
#include <cstdio>

#include "../../weight_only_quantized_qgemv_amd/csrc/span.hpp"

int main()
{
    const int64_t lens[] = {0, 1, 2, 511, 512, 20000, INT32_MAX - 2048, INT32_MAX - 1, INT32_MAX};
    const int32_t ends[] = {INT32_MIN, INT32_MIN + 1, -50, -1, 0, 1, 2, 511, 512, 15000, 20000, 20001,
                            INT32_MAX - 2048, INT32_MAX - 511, INT32_MAX - 1, INT32_MAX};
    int failures = 0;
    for (int64_t len : lens)
        for (int32_t lo : ends)
            for (int32_t hi : ends) {
                const qp::Span s = qp::held_span(lo, hi, len);
                // Entry i is in the span where max(lo, 0) <= i < min(hi, len).
                const int64_t from = lo > 0 ? lo : 0, to = hi < len ? hi : len;
                const int64_t want = to > from ? to - from : 0;
                bool good = (int64_t)s.first + s.count <= len && s.count == want && (want == 0 || s.first == from);
                // The last index a thread forms: one stride of 2048 past the
                // count, which must neither wrap nor pass the test again.
                const uint32_t past = s.count + 2048u;
                good = good && past > s.count;
                if (!good) {
                    std::fprintf(stderr, "FAIL lo=%d hi=%d len=%lld: first=%u count=%u\n", lo, hi, (long long)len,
                                 s.first, s.count);
                    ++failures;
                }
            }
    if (failures == 0)
        std::puts("all spans inside");
    return failures != 0;
}
