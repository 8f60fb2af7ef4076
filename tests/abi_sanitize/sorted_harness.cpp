// Host-side drive of the argument checks of the operators that sort a batch by
// expert, bring it back and run it in 8-bit integers, under ASan/UBSan (built by
// tests/test_sorted_sanitize.py).  Every call fails validation or has nothing to
// do, so nothing is launched.
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

template <typename T = void>
static T* at(uintptr_t i) { return reinterpret_cast<T*>(uintptr_t(0x7f0000000000ull) + (i << 36)); }

int main() {
    const int32_t big = std::numeric_limits<int32_t>::max(), low = std::numeric_limits<int32_t>::min();
    const int32_t sizes[] = {low, -1, 0, 1, 2, 7, 8, 16, 64, 65, 128, 256, 1024, 1025, 32768, 32784, 1 << 20,
                             (1 << 20) + 128, 1 << 24, 1 << 30, (1 << 30) + 1, big - 127, big};
    std::mt19937 rng(11);
    auto any = [&] { return sizes[rng() % (sizeof(sizes) / sizeof(*sizes))]; };
    using f32 = float;
    using i32 = int32_t;
    using i8 = int8_t;
    for (int i = 0; i < 200000; ++i) {
        const int32_t t = any(), k = any(), e = any(), c = any(), n = any();
        const int32_t xt = int32_t(rng() % 7) - 1, rt = int32_t(rng() % 7) - 1;
        const int64_t room = int64_t(any());
        const int64_t need = moe_sort_scratch_bytes(t, k, e);
        CHECK(need < 0 || need <= int64_t(256) * 1024 * 4);
        // outputs over their inputs, so that sizes which pass are refused by the overlap check
        // (its byte counts are what overflows first)
        if (t != 0) {
            CHECK(moe_sort_rows(at(0), xt ? at<f32>(1) : nullptr, at<i32>(2), t, k, e, c, xt, rt, at(0),
                                rt ? at<f32>(3) : nullptr, at<i32>(4), at<i32>(5), at(6), room, nullptr) < 0);
            CHECK(moe_combine_rows(at(0), at<i32>(1), at<f32>(2), t, k, c, n, at(2), nullptr) < 0);
            CHECK(moe_combine_rows_bwd(at(0), at(1), at<i32>(2), at<f32>(3), t, k, c, n, at(4), at<f32>(2), nullptr) < 0);
            CHECK(moe_sort_rows(nullptr, nullptr, nullptr, t, k, e, c, xt, rt, nullptr, nullptr, nullptr, nullptr,
                                nullptr, room, nullptr) < 0);
            CHECK(moe_combine_rows(nullptr, nullptr, nullptr, t, k, c, n, nullptr, nullptr) < 0);
            CHECK(moe_combine_rows_bwd(nullptr, nullptr, nullptr, nullptr, t, k, c, n, nullptr, nullptr, nullptr) < 0);
            CHECK(moe_quant_act_int8(at(0), t, c, at<i8>(0), at<f32>(1), nullptr) < 0);
            CHECK(moe_silu_mul_int8(at(0), t, c, 0.0f, at<i8>(0), at<f32>(1), nullptr) < 0);
            CHECK(moe_gemm_int8(at<i8>(0), at<f32>(1), at<i8>(2), at<f32>(3), t, n, c, at(0), nullptr) < 0);
            CHECK(moe_grouped_gemm(at(0), at<f32>(1), at(2), at<f32>(3), at<i32>(4), t, e, n, c, MOE_WDTYPE_INT8, at(0),
                                   nullptr) < 0);
        }
        moe_gemm_plan_info info;
        CHECK(moe_gemm_plan(t, e, n, c, MOE_WDTYPE_INT8, &info) <= 0);
    }
    CHECK(moe_combine_rows(nullptr, nullptr, nullptr, 0, 1, 8, 0, nullptr, nullptr) == 0);
    CHECK(moe_combine_rows_bwd(nullptr, nullptr, nullptr, nullptr, 0, 1, 8, 0, nullptr, nullptr, nullptr) == 0);
    CHECK(moe_gemm_int8(nullptr, nullptr, nullptr, nullptr, 0, 1, 16, nullptr, nullptr) == 0);
    std::printf(failures ? "sorted sanitize harness: %d failures\n" : "sorted sanitize harness: ok\n", failures);
    return failures != 0;
}
