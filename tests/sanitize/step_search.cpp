// Which sequence a row falls to, and which a work-group takes next, at counts of
// sequences next to 2^31, for a build under AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_step_search.py). The kernels walk
// sequences with the same functions.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "step_plan.hpp"

using namespace sgemm_impl;

namespace {

int failures = 0;

void expect(bool ok, const char *what, long long a = 0, long long b = 0, long long c = 0)
{
    if (!ok) {
        std::fprintf(stderr, "FAILED: %s (%lld, %lld, %lld)\n", what, a, b, c);
        ++failures;
    }
}

// n sums, i + 1 at place i, of which none is held; a place that is not one of theirs is a failure.
struct Sums {
    int n;
    std::int64_t operator[](int i) const
    {
        expect(i >= 0 && i < n, "a sum that is not there was read", i, n);
        return std::int64_t(i) + 1;
    }
};

}  // namespace

int main()
{
    const int counts[] = {0, 1, 2, 63, 64, 65, 1 << 30, (1 << 30) + 1, (1 << 30) + 12345, INT_MAX - 1, INT_MAX};
    for (int n : counts)
        for (std::int64_t x : {std::int64_t(0), std::int64_t(1), std::int64_t(n) / 2, std::int64_t(n) - 2, std::int64_t(n) - 1, std::int64_t(n)}) {
            if (x < 0) continue;
            expect(above(Sums{n}, n, x) == (x < n ? int(x) : n), "above", n, x, above(Sums{n}, n, x));
        }
    for (int seqs : counts)
        for (int step : {1, 2, 96, 4096, 1 << 22, INT_MAX})
            for (std::int64_t seq : {std::int64_t(0), std::int64_t(seqs) - step, std::int64_t(seqs) - step - 1, std::int64_t(seqs) - 1}) {
                if (seq < 0 || seq >= seqs) continue;
                const std::int64_t next = seq + step;
                expect(next_sequence(int(seq), step, seqs) == (next < seqs ? next : seqs), "next_sequence", seqs, step, seq);
            }
    if (failures) return 1;
    std::printf("step search ok\n");
    return 0;
}
