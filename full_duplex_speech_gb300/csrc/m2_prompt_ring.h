// How the warps of a CTA of m2_attn_prompt_tile.cu use its ring of shared memory,
// written over a ring type, so that a host model runs the same code
// (tests/prompt_ring/model.cpp).
//
// A pair's pieces of the ring: the keys and values of its chunks in turn, then
// room for the output of each tile that has rows. A stage's barriers are waited
// on by the parity of a piece's turn. Such a wait is right while the turn before
// is over, and the turn behind cannot be: two turns off, it passes at once or
// never. What makes it so:
//   - whoever waits for a piece has before waited for one that lies at most
//     kRingStages ahead of it, or for what comes behind such a one;
//   - a stage is refilled only when everyone who waits for its piece has.
#pragma once

#ifdef __CUDACC__
#define M2_RING_FN __device__ __forceinline__
#else
#define M2_RING_FN inline
#endif

namespace m2 {

constexpr int kRingStages = 5;

// Pieces of a pair of `chunks` chunks whose outputs need `outputs` pieces (0 to 2).
// A pair without chunks (its session is refused) has none: nothing that its tiles
// wait for would tell them that the pieces of the pairs before have had their turns.
M2_RING_FN int ring_pieces(int chunks, int outputs) { return chunks > 0 ? 2 * chunks + outputs : 0; }

// The pieces p .. end - 1 of a pair whose first is `first`: put(p) when its stage
// is free. False (and no further piece) when a wait ran out.
template <typename Ring, typename Put>
M2_RING_FN bool ring_fill(Ring& ring, int first, int p, int end, Put put) {
    for (; p < end; ++p) {
        if (first + p >= kRingStages && !ring.wait_empty(first + p - kRingStages)) return false;
        put(p);
    }
    return true;
}

// What has landed, in turn: look(p), then it is ready.
template <typename Ring, typename Look>
M2_RING_FN void ring_look(Ring& ring, int first, int pieces, Look look) {
    for (int p = 0; p < pieces; ++p) {
        if (!ring.wait_full(first + p)) break;
        look(p);
        ring.arrive_ready(first + p);
    }
}

// A tile's wait for the room of its output, behind its products. (For what looks at
// the pieces to have come by: the tile empties the room by itself, and a look that
// came after the stage's next piece had landed would wait for its own answer to that.)
template <typename Ring> M2_RING_FN bool ring_room(Ring& ring, int piece) { return ring.wait_ready(piece); }

}  // namespace m2
