// What decides how an expert layer's products run, and the plan that they take from memory: the chosen experts, their rows,
// and the order of all slots by expert. Code without HIP, so that the rules can be tested on a machine without a GPU.
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

// ---------------------------------------------------------------------------
// A block's four waves share its work: WR groups of output rows, WK waves along the rows' bytes. A wave has kMoeTiles tiles of
// 16 rows of weights (gate and up of the same 16 outputs, or 32 outputs of down).
constexpr int kMoeWaves = 4;
constexpr int kMoeTiles = 2;
constexpr int kMoePiece = 16; // positions that a thread makes parts of, or brings, at a time

// Outputs of a block's tile.
constexpr int moe_outputs(bool gated, int wk) { return (gated ? 16 : 16 * kMoeTiles) * kMoeWaves / wk; }

// Three operands and more: two blocks a CU with more registers, else three.
constexpr bool moe_big(int m) { return m >= 3; }

// Bytes of a phase's parts and units: with the waves' sums and the slots, a third (half) of a CU's 160 KB. (Three blocks with
// 44 KB: 5 tokens on 8 experts of 2048 x 6144 in int2 33.7 us instead of 32.9.)
constexpr int moe_lds(int m) { return moe_big(m) ? 74 * 1024 : 99 * 512; }

// Rows that a block takes at a time: four an operand, as many as have room for two steps of every wave. pos: positions a step.
constexpr int moe_rows(int m, int wk, int pos) {
    const int unit = 4 * (2 * wk * pos + 16) + 4 * 2 * wk;
    return moe_lds(m) / unit < 4 * m ? moe_lds(m) / unit : 4 * m;
}

// Pieces of a thread that are loaded ahead of the weights.
constexpr int moe_ahead(int m) { return m == 8 ? 0 : 2; }

// A wave's steps of a tile: wk, wk + WK, ...; all waves take an even number of them, past the row on activations of 0.
constexpr int moe_steps(int steps, int wk) { return ((steps + wk - 1) / wk + 1) & ~1; }

// A phase: as many of a wave's `all` steps as the buffer holds activations of n rows of (where parts stand prepared, and are
// brought ahead, no more than what the threads hold); an even number.
constexpr int moe_phase(int m, int wk, int pos, int n, int all) {
    const int fit = ((moe_lds(m) / n - 64) / (wk * (4 * pos + 4))) & ~1;
    int held = fit;
    if (moe_big(m) && moe_ahead(m) > 0) {
        held = (moe_ahead(m) * 64 * kMoeWaves * kMoePiece / (n * wk * pos)) & ~1;
        held = held < 2 ? 2 : held;
    }
    const int per = fit < held ? fit : held;
    return all < per ? all : per;
}

// How one product runs.
struct MoeForm {
    int m;     // operands of 16 stacked rows, four activations each
    int wk;    // waves along the rows' bytes
    int tiles; // tiles of outputs that a block takes one after another
};

// The form for matrices of O rows of `steps` steps. operands: what the rows an expert has ask for; turned: groups of scales that
// do not cover whole halves of a step; active: experts that some token chose.
constexpr MoeForm moe_form(bool gated, int O, int steps, bool turned, int operands, int active, int cus) {
    MoeForm f{0, 0, 0};
    f.m = operands >= 4 && turned ? 3 : operands; // (of turned operands, more than three would spill; in int2 three do)
    // Waves along the rows' bytes only as far as the outputs alone leave CUs with less than two blocks, and rows of some length:
    // one token, 8 experts of 2048 x 6144 in int4 34.4 us with two for both products, 36.7 with one, 38.9 with four; 17 tokens on
    // 64 experts of 768 x 2048 42.2 us with one, 49.0 with two; 5 tokens on 8 experts in int2 34.8 with two, 40.2 with one, 42.9
    // with four.
    const int out = moe_outputs(gated, 1);
    const long most = (long)active * ((O + out - 1) / out); // blocks with none of them
    f.wk = most >= 2 * cus || steps < 4 ? 1 : most >= cus || steps < 16 ? 2 : 4;
    // As many tiles a block as leave three blocks a CU; with prepared parts, which would be brought anew, one.
    const int o = moe_outputs(gated, f.wk);
    const long tiles = (O + o - 1) / o, per = moe_big(f.m) ? 1 : tiles * active / (3 * cus);
    f.tiles = (int)(per < 1 ? 1 : per > tiles ? tiles : per);
    return f;
}

} // namespace wq
