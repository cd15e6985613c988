// The host-only layout entry points of the products held in few bits, driven
// over edge-case sizes for a build under AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_lowbit_shapes.py).
#include <climits>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "sgemm.h"

namespace {

int failures = 0;

void expect(bool ok, const char *what, long long a, long long b, long long c)
{
    if (!ok) {
        std::fprintf(stderr, "FAILED: %s (%lld, %lld, %lld)\n", what, a, b, c);
        ++failures;
    }
}

}  // namespace

int main()
{
    const int sizes[] = {INT_MIN, -1, 0, 1, 7, 8, 9, 16, 17, 33, 255, 256, 4093, 1 << 20, 1 << 30, INT_MAX};
    for (int dtype : {-1, 0, 1, 2, 3})
        for (int M : sizes)
            for (int N : sizes)
                for (int K : sizes)
                    for (int cus : {INT_MIN, 0, 1, 256, INT_MAX}) {
                        int s[5] = {};
                        if (sgemm_w4_shape(dtype, M, N, K, cus, s) != SGEMM_OK) continue;
                        expect(s[0] >= 16 && s[1] >= 16 && s[2] >= 1 && s[3] >= 1 && s[2] * s[3] <= 16 && s[4] >= 0, "sgemm_w4_shape", M, N, K);
                        expect(s[0] > 16 || M <= 16, "rows", M, N, K);
                    }
    alignas(16) static char codes[16];
    static float scales[1];
    static int arrays[2];
    for (int n : sizes)
        for (int heads : {1, 8, 65536})
            for (int dim : {16, 128, 256})
                for (int ld : sizes)
                    for (int window : sizes) {
                        const sgemm_kv8_cache c{codes, codes, scales, scales, 1, heads, 1024, dim};
                        const sgemm_kv8_batch b{arrays, arrays, arrays, n, ld, n, n};
                        int s[4] = {};
                        if (sgemm_kv8_attend_shape(&c, &b, heads * 7, window, 0, s) != SGEMM_OK) continue;
                        expect((s[0] == 16 || s[0] == 32) && (s[1] == 1 || s[1] == 4) && s[2] >= 1 && s[3] >= 1 && s[3] <= 64,
                               "sgemm_kv8_attend_shape", n, ld, window);
                        expect((s[3] > 1) == (sgemm_kv8_attend_workspace_size(&c, &b, heads * 7, window, 0) > 0) || n == 0,
                               "splits have a workspace", n, ld, window);
                    }
    if (failures) return 1;
    std::printf("lowbit shapes ok\n");
    return 0;
}
