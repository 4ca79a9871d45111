// What the expert layer's products make of a plan of any contents (no GPU). Run by tests/test_moe_plan.py; prints the failed
// checks and exits with their number.
#include <climits>
#include <cstdio>
#include <initializer_list>
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

void phases_fit_their_buffer() {
    for (int m : {1, 2, 3, 4, 8})
        for (int wk : {1, 2, 4})
            for (int pos : {128, 256, 512}) {
                const int rows = wq::moe_rows(m, wk, pos);
                CHECK(rows >= 1 && rows <= 4 * m && rows <= 64);
                for (int n = 1; n <= rows; ++n)
                    for (int steps : {1, 2, 3, 4, 5, 15, 16, 17, 48, 1000, 1 << 21}) {
                        const int all = wq::moe_steps(steps, wk), per = wq::moe_phase(m, wk, pos, n, all);
                        CHECK(all % 2 == 0 && all * wk >= steps && (all - 2) * wk < steps);
                        CHECK(per >= 2 && per % 2 == 0 && per <= all);
                        // parts in rows of 16 bytes more than their positions, and a unit a step
                        CHECK((long)n * 4 * (per * wk * pos + 16) + (long)n * per * wk * 4 <= wq::moe_lds(m));
                        const long pieces = (long)n * per * wk * pos / wq::kMoePiece; // counted by 32-bit reciprocals
                        CHECK(pieces < 65536);
                    }
            }
}

void forms() {
    for (int gated = 0; gated < 2; ++gated)
        for (int O : {1, 16, 17, 127, 1610, 3300, 65536, 1 << 22})
            for (int steps : {1, 3, 4, 15, 16, 1000})
                for (int ops : {1, 2, 4, 8})
                    for (int active : {1, 3, 64, 1024})
                        for (int turned = 0; turned < 2; ++turned) {
                            const wq::MoeForm f = wq::moe_form(gated, O, steps, turned, ops, active, 256);
                            const int out = wq::moe_outputs(gated, f.wk), tiles = (O + out - 1) / out;
                            CHECK(f.m == (turned && ops >= 4 ? 3 : ops) && (f.wk == 1 || f.wk == 2 || f.wk == 4));
                            CHECK(f.tiles >= 1 && f.tiles <= tiles && (f.tiles == 1 || !wq::moe_big(f.m)));
                        }
    // one token, 8 of 16 experts of 2048 x 6144 in int4; 64 tokens on 256 such experts
    const wq::MoeForm one = wq::moe_form(true, 2048, 24, false, 1, 8, 256), many = wq::moe_form(true, 2048, 24, false, 1, 222, 256);
    CHECK(one.m == 1 && one.wk == 2 && one.tiles == 1 && many.wk == 1 && many.tiles == 9);
}

} // namespace

int main() {
    any_contents();
    good_plans_stay();
    phases_fit_their_buffer();
    forms();
    if (failures == 0) std::printf("all checks passed\n");
    return failures;
}
