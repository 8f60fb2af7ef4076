// Host-side drive of the argument checks of the operators around the layer
// under ASan/UBSan (built by tests/test_rows_sanitize.py).  Every call fails
// validation or has no rows, so nothing is launched.
#include <cstdint>
#include <cstdio>
#include <limits>
#include <random>

#include "moe.h"

static int failures = 0;
#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            std::fprintf(stderr, "CHECK failed at line %d: %s\n", __LINE__, #c); \
            ++failures;                                                       \
        }                                                                     \
    } while (0)

static void* at(uintptr_t i) { return reinterpret_cast<void*>(uintptr_t(0x7f0000000000ull) + (i << 36)); }

int main() {
    const int32_t big = std::numeric_limits<int32_t>::max(), low = std::numeric_limits<int32_t>::min();
    const int32_t sizes[] = {low, -1, 0, 1, 7, 8, 64, 128, 129, 256, 32768, 1 << 20, (1 << 20) + 128, 1 << 30,
                             (1 << 30) + 1, big - 127, big};
    std::mt19937 rng(7);
    auto any = [&] { return sizes[rng() % (sizeof(sizes) / sizeof(*sizes))]; };
    auto u8 = [](void* p) { return static_cast<uint8_t*>(p); };
    auto f32 = [](void* p) { return static_cast<float*>(p); };
    for (int i = 0; i < 200000; ++i) {
        const int32_t r = any(), c = any(), n = any(), e = any(), q = int32_t(rng() % 5) - 1;
        // outputs over their inputs, so that sizes which pass are refused by the overlap check
        // (its byte counts are what overflows first)
        CHECK(moe_rmsnorm(at(0), at(1), at(2), 1e-6f, r, c, q, at(2), at(3), u8(at(4)), at(4), nullptr) <= 0);
        CHECK(moe_silu_mul(at(0), r, c, 0.0f, q, at(0), u8(at(1)), at(2), nullptr) <= 0);
        CHECK(moe_gemm_fp8(u8(at(0)), f32(at(1)), u8(at(2)), f32(at(3)), r, n, c, at(0), nullptr) <= 0);
        CHECK(moe_grouped_gemm(at(0), q == 1 ? f32(at(1)) : nullptr, at(2), q == 1 ? f32(at(3)) : nullptr,
                               static_cast<int32_t*>(at(4)), r, e, n, c, q, at(0), nullptr) <= 0);
        // null pointers
        if (r != 0) {
            CHECK(moe_rmsnorm(nullptr, nullptr, nullptr, 0.0f, r, c, q, nullptr, nullptr, nullptr, nullptr, nullptr) < 0);
            CHECK(moe_silu_mul(nullptr, r, c, 1.0f, q, nullptr, nullptr, nullptr, nullptr) < 0);
            CHECK(moe_gemm_fp8(nullptr, nullptr, nullptr, nullptr, r, n, c, nullptr, nullptr) < 0);
            CHECK(moe_grouped_gemm(nullptr, nullptr, nullptr, nullptr, nullptr, r, e, n, c, q, nullptr, nullptr) < 0);
        }
    }
    CHECK(moe_rmsnorm(nullptr, nullptr, nullptr, 0.0f, 0, 128, 0, nullptr, nullptr, nullptr, nullptr, nullptr) == 0);
    CHECK(moe_grouped_gemm(nullptr, nullptr, nullptr, nullptr, nullptr, 0, 1, 1, 64, 0, nullptr, nullptr) == 0);
    std::printf(failures ? "rows sanitize harness: %d failures\n" : "rows sanitize harness: ok\n", failures);
    return failures != 0;
}
