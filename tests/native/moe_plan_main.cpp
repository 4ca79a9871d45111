// What the expert layer's products make of a plan of any contents (no GPU). Run by tests/test_moe_plan.py; prints the failed
// checks and exits with their number.
#include <climits>
#include <cstdio>
#include <random>
#include <type_traits>

#include "moe_plan.h"

namespace {

int failures = 0;
#define CHECK(c)                                                        \
    do {                                                                \
        if (!(c)) {                                                     \
            std::printf("check failed at line %d: %s\n", __LINE__, #c); \
            if (++failures > 20) return;                                \
        }                                                               \
    } while (0)

// no addresses: a plan's numbers are all that the products take from it
static_assert(sizeof(wq::MoeWork) == 4 * sizeof(int) && std::is_same<decltype(wq::MoeWork::expert), int>::value, "numbers only");

void in_range(wq::MoeWork w, int E, int N) {
    const wq::MoeWork b = wq::bounded(w, E, N);
    CHECK(b.expert >= 0 && b.expert < E);
    CHECK(b.rows >= 0 && b.first >= 0 && (long)b.first + b.rows <= N);
    const int s = wq::bounded_slot(w.first, N);
    CHECK(s >= 0 && s < N);
}

void any_contents() {
    const int ends[] = {INT_MIN, INT_MIN + 1, -65536, -1, 0, 1, 2, 15, 16, 17, 255, 256, 1023, 1024, 16383, 16384, 16385, 65536, INT_MAX - 1, INT_MAX};
    std::mt19937 rng(1);
    const int sizes[][2] = {{1, 1}, {1, 16384}, {16, 256}, {1024, 257}, {1024, 16384}, {7, 3}};
    for (const auto &n : sizes) {
        for (int e : ends)
            for (int r : ends)
                for (int f : ends) in_range({e, r, f, 0}, n[0], n[1]);
        for (int i = 0; i < 200000; ++i) in_range({(int)rng(), (int)rng(), (int)rng(), 0}, n[0], n[1]);
        for (int i = 0; i < 200000; ++i) in_range({(int)(rng() % 2048) - 512, (int)(rng() % 32768) - 8192, (int)(rng() % 32768) - 8192, 0}, n[0], n[1]);
    }
}

void good_plans_stay() {
    std::mt19937 rng(2);
    for (int i = 0; i < 200000; ++i) {
        const int E = 1 + (int)(rng() % 1024), N = 1 + (int)(rng() % 16384), first = (int)(rng() % N), rows = 1 + (int)(rng() % (N - first)),
                  e = (int)(rng() % E);
        const wq::MoeWork b = wq::bounded({e, rows, first, 0}, E, N);
        CHECK(b.expert == e && b.rows == rows && b.first == first);
        CHECK(wq::bounded_slot(first, N) == first);
        CHECK(wq::bounded({e, 0, first, 0}, E, N).rows == 0);
    }
}

} // namespace

int main() {
    any_contents();
    good_plans_stay();
    if (failures == 0) std::printf("all checks passed\n");
    return failures;
}
