// pa_tree_ring.h - where the tree attention's tiles of K and V lie in shared memory, and
// what a copy into such a place waits for.  Plain C++: the kernel runs these rules, and a
// test on the host runs them under every order of its threads.
//
// Barriers: per slot, its tile has arrived; per tile i, by i % 4, its scores and its output
// are done.  A wait sees a phase's parity alone, so it has to come before the phase after
// next can end: scores (or output) t is waited for by a load that scores (output) t + 4
// cannot be done without.
#pragma once

namespace pa {

// K of tile i is read by its scores, V by its output.
enum class TreeRead { none, scores, output };

template <int D, bool KV8>
struct TreeRing {
    // Slots of a bf16 pool, D = 128: one ring in the order of their use, K of a tile two
    // outputs ahead, K0 K1 V0 K2 V1 K3 V2 ..  (A ring of two for K and one of three for V left
    // K's loads in the chain: 16 wide trees 137 us, 131 with this one.)  D = 64: the even slots
    // are K's and the odd ones V's, four tiles each.  (In one ring of eight V3 takes K0's place:
    // a late wait for scores 0 could miss its phase, since nothing holds back scores 4, and of
    // four tiles K0's arrival was waited for in a slot that V3 had filled.)
    static constexpr int kRing = D == 64 ? 8 : 5;
    // Of an FP8 pool: K's codes, and V converted.
    static constexpr int kKSlots = 3, kVSlots = 2;
    static constexpr int kSlots = KV8 ? kKSlots + kVSlots : kRing;

    struct Place {
        int slot, use;  // how often the slot was filled before
    };
    struct After {
        TreeRead what;
        int tile;
    };

    static constexpr Place in_ring(int n) { return {n % kRing, n / kRing}; }
    static constexpr Place k(int i) {
        return KV8       ? Place{i % kKSlots, i / kKSlots}
               : D == 64 ? Place{2 * (i % 4), i / 4}
                         : in_ring(i ? 2 * i - 1 : 0);
    }
    static constexpr Place v(int i) {
        return KV8       ? Place{kKSlots + i % kVSlots, i / kVSlots}
               : D == 64 ? Place{2 * (i % 4) + 1, i / 4}
                         : in_ring(2 * i + 2);
    }

    // What read the slot of tile i's K (V) before.
    static constexpr After k_after(int i) {
        if (KV8) return i >= kKSlots ? After{TreeRead::scores, i - kKSlots} : After{};
        if (D == 128)  // V of tile i - 4 (K 0 before K 3)
            return i >= 4   ? After{TreeRead::output, i - 4}
                   : i == 3 ? After{TreeRead::scores, 0}
                            : After{};
        return i >= 4 ? After{TreeRead::scores, i - 4} : After{};
    }
    static constexpr After v_after(int i) {
        if (KV8) return i >= kVSlots ? After{TreeRead::output, i - kVSlots} : After{};
        if (D == 128)  // K of tile i - 1
            return i >= 2 ? After{TreeRead::scores, i - 1} : After{};
        return i >= 4 ? After{TreeRead::output, i - 4} : After{};
    }

    // At its end a warp waits until its last copies (as many as it can have in flight) have
    // landed: by the slot's barrier, or, where V of a later tile may have K's slot, by the
    // scores that read it.
    static constexpr int kInFlight = KV8 ? 3 : 4;
    static constexpr bool kKLandsByScores = !KV8 && D == 128;
};

}  // namespace pa
