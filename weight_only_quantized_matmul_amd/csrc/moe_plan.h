// The plan of an expert layer's products: the chosen experts, their rows, and the order of all slots by expert. Code without
// HIP, so that the rules can be tested on a machine without a GPU.
//
// A plan lies in a stream's workspace, which a captured call keeps and its
// stream goes on using: where the two run at once, which nobody may ask for,
// one of them reads what the other wrote, numbers of any kind. A plan therefore
// holds no addresses, and what is read of it is brought into range before use:
// such calls give wrong numbers and touch nothing that is not theirs.
#pragma once

namespace wq {

// An expert, how many rows it has, and where their slots t * k + j stand in the order.
struct MoeWork {
    int expert, rows, first;
    int pad;
};

// The work read from a plan over E experts and N slots: `expert` in [0, E), first .. first + rows within [0, N).
constexpr MoeWork bounded(MoeWork w, int E, int N) {
    const bool there = w.expert >= 0 && w.expert < E && w.first >= 0 && w.first < N && w.rows > 0;
    MoeWork b{0, 0, 0, 0};
    if (there) {
        b.expert = w.expert;
        b.first = w.first;
        b.rows = w.rows < N - w.first ? w.rows : N - w.first;
    }
    return b;
}

// A slot read from the order of N.
constexpr int bounded_slot(int slot, int N) { return slot >= 0 && slot < N ? slot : 0; }

} // namespace wq
