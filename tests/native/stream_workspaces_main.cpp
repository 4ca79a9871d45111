// Rules of the streams' workspaces, against a memory that records every block (no GPU). Run by
// tests/test_stream_workspaces.py; prints the failed checks and exits with their number.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "stream_workspaces.h"

namespace {

int failures = 0;
#define CHECK(c)                                                        \
    do {                                                                \
        if (!(c)) {                                                     \
            std::printf("check failed at line %d: %s\n", __LINE__, #c); \
            ++failures;                                                 \
        }                                                               \
    } while (0)

struct Memory {
    std::set<void *> there;
    size_t bytes = 0, limit = ~size_t(0);
    int idles = 0, allocs = 0;
    int alloc(void **p, size_t n) {
        if (bytes + n > limit) return -5;
        *p = reinterpret_cast<void *>(0x1000 + 0x100 * size_t(++allocs)); // an address is never given twice
        there.insert(*p);
        bytes += n;
        return 0;
    }
    void release(void *p, size_t n) {
        CHECK(there.erase(p) == 1);
        bytes -= n;
    }
    int idle() { return ++idles, 0; }
};

constexpr size_t MB = size_t(1) << 20;
const void *stream(int i) { return reinterpret_cast<const void *>(size_t(i)); }

struct Fixture {
    Memory m;
    wq::StreamWorkspaces ws;
    int rc = 0;
    void *take(size_t n, int st, bool capturing = false) {
        void *p = nullptr;
        rc = ws.take(m, n, stream(st), capturing, -8, &p);
        return rc == 0 ? p : nullptr;
    }
};

void growth_without_graphs() {
    Fixture f;
    void *a = f.take(MB, 1);
    CHECK(a && f.take(2 * MB, 1) == a && f.m.allocs == 1); // whole units of 2 MB
    void *b = f.take(3 * MB, 1);
    CHECK(b && b != a && f.m.there.size() == 1 && f.m.bytes == 4 * MB && f.m.idles > 0); // the old one is freed, the device idle
    CHECK(f.take(MB, 2) != b);
}

void captured_block_outlives_growth() {
    Fixture f;
    void *a = f.take(MB, 1);
    CHECK(f.take(MB, 1, true) == a);
    CHECK(f.take(MB, 1) == a); // eager calls of the stream go on with it
    void *b = f.take(9 * MB, 1);
    CHECK(b && b != a && f.m.there.count(a) && f.m.there.count(b));
    CHECK(f.take(5 * MB, 1, true) == b);
    void *c = f.take(20 * MB, 1);
    CHECK(c && c != b && f.m.there.count(a) && f.m.there.count(b));
    void *d = f.take(30 * MB, 1); // c was in no graph
    CHECK(d && !f.m.there.count(c) && f.m.there.size() == 3);
}

void captured_block_of_another_stream_outlives_growth() {
    Fixture f;
    void *a = f.take(8 * MB, 1);
    CHECK(f.take(4 * MB, 7, true) == a); // stream 7 has none: the largest
    f.take(16 * MB, 1);
    CHECK(f.m.there.count(a));
}

void captured_block_does_not_pass_to_another_stream() {
    Fixture f;
    void *a = f.take(8 * MB, 1);
    CHECK(f.take(MB, 1, true) == a);
    for (int s = 2; s <= 40; ++s) { // more streams than slots
        void *p = f.take(MB, s);
        CHECK(p && p != a);
    }
    CHECK(f.m.there.count(a));
    void *b = f.take(MB, 1); // the stream itself comes back, to a block of its own
    CHECK(b && b != a && f.m.there.size() == size_t(wq::StreamWorkspaces::kSlots) + 1);
}

void capture_never_allocates_or_waits() {
    Fixture f;
    CHECK(f.take(MB, 1, true) == nullptr && f.rc == -8);
    f.take(MB, 1);
    const int allocs = f.m.allocs, idles = f.m.idles;
    CHECK(f.take(3 * MB, 1, true) == nullptr && f.rc == -8);
    CHECK(f.take(2 * MB, 1, true) != nullptr && f.m.allocs == allocs && f.m.idles == idles);
}

void failed_growth() {
    Fixture f;
    f.m.limit = 10 * MB;
    void *a = f.take(4 * MB, 1);
    CHECK(f.take(4 * MB, 1, true) == a);
    CHECK(f.take(8 * MB, 1) == nullptr && f.rc == -5 && f.m.there.count(a)); // the graph's block counts and stays
    CHECK(f.take(4 * MB, 1) == a);
    Fixture g;
    g.m.limit = 10 * MB;
    g.take(4 * MB, 1);
    CHECK(g.take(12 * MB, 1) == nullptr && g.rc == -5);
    CHECK(g.take(2 * MB, 1) != nullptr && g.m.there.size() == 1);
}

} // namespace

int main() {
    growth_without_graphs();
    captured_block_outlives_growth();
    captured_block_of_another_stream_outlives_growth();
    captured_block_does_not_pass_to_another_stream();
    capture_never_allocates_or_waits();
    failed_growth();
    if (failures == 0) std::printf("all checks passed\n");
    return failures;
}
