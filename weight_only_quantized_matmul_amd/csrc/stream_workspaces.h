// The workspaces of a device's streams: which block a call gets, when a block
// grows, and how long it lives. Host code without HIP, so that the rules can be
// tested on a machine without a GPU.
#pragma once

#include <cstddef>

namespace wq {

// One block a stream. Only calls on that stream use it and they run in stream
// order, so it is reused without any wait; a block is freed, or passes to
// another stream, only once the device is idle.
//
// A call being captured into a graph never waits or allocates: it takes its
// stream's block if that is large enough, else the largest one that is, else it
// is refused. The graph holds the block's address for as long as it is replayed,
// which nobody here sees end, so such a block is never freed and never passes to
// another stream: its stream goes on with it until a call needs more, and then
// leaves it to the graph and gets a new one.
class StreamWorkspaces {
public:
    static constexpr int kSlots = 8;

    // M: int alloc(void **, size_t) (0 or an error), void release(void *, size_t), int idle() (0 or an error).
    // A result other than 0 is what M returned, or `refused`; *out is set with 0 only.
    template <typename M>
    int take(M &&memory, size_t bytes, const void *stream, bool capturing, int refused, void **out) {
        Slot *e = nullptr;
        for (Slot &s : slots_)
            if (s.live && s.stream == stream) e = &s;
        if (capturing) {
            if (e == nullptr || e->cap < bytes) {
                e = nullptr;
                for (Slot &s : slots_)
                    if (s.live && s.cap >= bytes && (e == nullptr || s.cap > e->cap)) e = &s;
            }
            if (e == nullptr) return refused;
            e->in_graph = true;
            *out = e->p;
            return 0;
        }
        const bool adopt = e == nullptr;
        if (adopt) {
            for (Slot &s : slots_)
                if (!s.live && e == nullptr) e = &s;
            if (e == nullptr) {
                e = &slots_[0];
                for (Slot &s : slots_)
                    if (s.last < e->last) e = &s;
            }
        }
        const bool grow = bytes > e->cap, other = adopt && e->live;
        if (e->in_graph && (grow || other)) { // left to the graph
            Slot fresh;
            const int rc = make(memory, bytes, &fresh);
            if (rc != 0) return rc;
            fresh.last = e->last;
            *e = fresh;
        } else {
            if (grow || other) {
                const int rc = memory.idle();
                if (rc != 0) return rc;
            }
            if (grow) {
                if (e->p != nullptr) memory.release(e->p, e->cap);
                const unsigned long long last = e->last;
                *e = Slot();
                const int rc = make(memory, bytes, e);
                if (rc != 0) return rc;
                e->last = last;
            }
        }
        e->stream = stream;
        e->live = true;
        e->last = ++clock_;
        *out = e->p;
        return 0;
    }

private:
    struct Slot {
        const void *stream = nullptr;
        bool live = false;
        bool in_graph = false; // a captured call holds p
        void *p = nullptr;
        size_t cap = 0; // bytes
        unsigned long long last = 0;
    };

    template <typename M>
    static int make(M &&memory, size_t bytes, Slot *s) {
        constexpr size_t kUnit = size_t(2) << 20;
        const size_t cap = (bytes + kUnit - 1) / kUnit * kUnit;
        const int rc = memory.alloc(&s->p, cap);
        if (rc != 0) {
            s->p = nullptr;
            return rc;
        }
        s->cap = cap;
        return 0;
    }

    Slot slots_[kSlots];
    unsigned long long clock_ = 0;
};

} // namespace wq
