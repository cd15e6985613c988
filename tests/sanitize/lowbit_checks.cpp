// Host-only entry points of the products held in few bits, driven over
// edge-case arguments for a build under AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_lowbit_host.py). No pointer passed
// here is dereferenced but those of the two structures.
#include <climits>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "sgemm.h"

namespace {

int failures = 0;

void expect(bool ok, const char *what, long long a = 0, long long b = 0, long long c = 0)
{
    if (!ok) {
        std::fprintf(stderr, "FAILED: %s (%lld, %lld, %lld)\n", what, a, b, c);
        ++failures;
    }
}

bool is_status(int s) { return s <= 0 && s >= SGEMM_ERR_MASK; }

template <class T> T *fake(std::uintptr_t addr) { return reinterpret_cast<T *>(addr); }

}  // namespace

int main()
{
    const int sizes[] = {INT_MIN, -1, 0, 1, 7, 16, 31, 32, 64, 128, 256, 4093, 1 << 20, 1 << 30, INT_MAX};
    const std::uintptr_t top = UINTPTR_MAX - 4095;
    for (int M : sizes)
        for (int N : sizes)
            for (int K : sizes)
                for (int ld : sizes) {
                    const int g = ld / 2 * 2;
                    int s = sgemm_w4_check_args(0, 1, M, N, K, g, 1.0f, fake<void>(1 << 20), ld, fake<unsigned char>(top), ld,
                                                fake<void>(1 << 24), ld, fake<unsigned char>(top), ld, 0.0f, fake<float>(top), ld);
                    expect(is_status(s), "sgemm_w4_check_args", M, N, K);
                    s = sgemm_w4_pack_check_args(2, 0, N, K, 32, fake<void>(top), ld, fake<unsigned char>(1 << 20), ld,
                                                 fake<void>(1 << 24), ld, nullptr, 0);
                    expect(is_status(s), "sgemm_w4_pack_check_args", N, K, ld);
                }
    const int blocks[] = {INT_MIN, -16, 0, 15, 16, 48, 64, 1024, 2048, INT_MAX};
    const int dims[] = {INT_MIN, 0, 8, 16, 80, 256, 272, INT_MAX};
    for (int pages : sizes)
        for (int n : sizes)
            for (int block : blocks)
                for (int dim : dims)
                    for (int ld : sizes) {
                        const sgemm_kv8_cache c{fake<void>(top & ~std::uintptr_t(15)), fake<void>(1 << 20), fake<float>(1 << 21),
                                                fake<float>(top), pages, n, block, dim};
                        const sgemm_kv8_batch b{fake<int>(top), fake<int>(64), fake<int>(128), n, ld, n, ld};
                        expect(is_status(sgemm_kv8_check_args(&c, &b, 0, fake<void>(top), ld, n, fake<void>(4096), n, ld)),
                               "sgemm_kv8_check_args", pages, n, ld);
                        expect(is_status(sgemm_kv8_attend_check_args(&c, &b, 1, n, fake<void>(top), ld, n, 1.0f, 1, ld, fake<float>(top),
                                                                     n, ld, fake<void>(top), SIZE_MAX)),
                               "sgemm_kv8_attend_check_args", pages, n, ld);
                        for (int cus : {INT_MIN, 0, 1, 256, INT_MAX})
                            expect(sgemm_kv8_attend_workspace_size(&c, &b, n, ld, cus) <= (std::size_t(1) << 40),
                                   "workspace size bounded", pages, n, ld);
                    }
    if (failures) return 1;
    std::printf("lowbit checks ok\n");
    return 0;
}
