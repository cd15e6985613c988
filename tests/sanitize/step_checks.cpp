// Host-only entry points of a serving step, driven over edge-case arguments
// for a build under AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_step_host.py). No pointer passed here is dereferenced but those
// of the structures.
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
    const int sizes[] = {INT_MIN, -1, 0, 1, 7, 16, 31, 64, 128, 256, 1024, 1 << 20, 1 << 30, INT_MAX};
    const std::uintptr_t top = UINTPTR_MAX - 4095;
    const int blocks[] = {INT_MIN, -16, 0, 15, 16, 48, 64, 1024, 2048, INT_MAX};
    const int dims[] = {INT_MIN, 0, 8, 16, 80, 256, 272, INT_MAX};
    for (int pages : sizes)
        for (int n : sizes)
            for (int block : blocks)
                for (int dim : dims)
                    for (int ld : sizes) {
                        const sgemm_kv4_cache c{fake<void>(top & ~std::uintptr_t(15)), fake<void>(1 << 20), fake<void>(1 << 21),
                                                fake<void>(top & ~std::uintptr_t(15)), pages, n, block, dim};
                        const sgemm_kv8_batch b{fake<int>(top), fake<int>(64), fake<int>(128), n, ld, n, ld};
                        expect(is_status(sgemm_kv4_check_args(&c, &b, 0, fake<void>(top), ld, n, fake<void>(4096), n, ld)),
                               "sgemm_kv4_check_args", pages, n, ld);
                        expect(is_status(sgemm_kv4_attend_check_args(&c, &b, 1, n, fake<void>(top), ld, n, 1.0f, 1, ld, fake<float>(top),
                                                                     n, ld, fake<void>(top), SIZE_MAX)),
                               "sgemm_kv4_attend_check_args", pages, n, ld);
                        for (int cus : {INT_MIN, 0, 1, 256, INT_MAX})
                            expect(sgemm_kv4_attend_workspace_size(&c, &b, n, ld, cus) <= (std::size_t(1) << 40),
                                   "workspace size bounded", pages, n, ld);
                        int s[4] = {};
                        if (sgemm_kv4_attend_shape(&c, &b, n, ld, 0, s) != SGEMM_OK) continue;
                        expect((s[0] == 4 || s[0] == 8 || s[0] == 16 || s[0] == 32) && (s[1] == 1 || s[1] == 4) && s[2] >= 1 && s[3] >= 0,
                               "sgemm_kv4_attend_shape", n, ld, dim);
                        expect((s[3] > 0) == (sgemm_kv4_attend_workspace_size(&c, &b, n, ld, 0) > 0) || n == 0 || ld == 0,
                               "shared tokens have a workspace", n, ld, dim);
                    }
    for (int rows : sizes)
        for (int dim : sizes)
            for (int rot : sizes)
                for (int ld : sizes)
                    for (int hs : sizes) {
                        const sgemm_rope_rows q{fake<void>(top), fake<void>(1 << 20), hs, ld, hs, hs, ld};
                        const sgemm_rope_rows k{fake<void>(1 << 20), fake<void>(top), rows, hs, ld, ld, hs};
                        for (const sgemm_rope_rows *second : {static_cast<const sgemm_rope_rows *>(nullptr), &k})
                            expect(is_status(sgemm_rope_check_args(0, 1, rows, dim, rot, 0, 1, 1.0f, fake<int>(top), fake<double>(64), &q, second)),
                                   "sgemm_rope_check_args", rows, dim, ld);
                    }
    for (int seqs : sizes)
        for (int columns : sizes)
            for (int block : blocks)
                for (int pool : sizes)
                    for (int rows : sizes) {
                        const sgemm_kv_step t{fake<int>(top), fake<int>(1 << 20), fake<int>(1 << 24), fake<int>(64), fake<int>(top),
                                              fake<int>(1 << 28), fake<int>(top), fake<long long>(top), fake<int>(64), seqs, columns, block, pool, rows};
                        expect(is_status(sgemm_kv_tables_check_args(&t)), "sgemm_kv_tables_check_args", seqs, columns, rows);
                    }
    if (failures) return 1;
    std::printf("step checks ok\n");
    return 0;
}
