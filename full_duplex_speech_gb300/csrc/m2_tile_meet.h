// How the warps of a tile hand its chunks over (m2_attn_paged_tile.cu), written
// over a barrier type `Bar`, so that a host model runs the same code
// (tests/tile_meet/model.cpp).
//
// A tile i with n chunks has meetings 0 .. n: at meeting j its weights of chunk
// j - 1 (at 0: its rows of q) are whole, and so are the operands of the products
// that follow. Six warps make each of them: the tile's four softmax warps, the
// warp that issues the products and the warp that has seen the operands from
// memory, the last two in turn for both tiles.
//
// Everyone waits in every meeting. A barrier counts arrivals, not who makes
// them: a warp that only arrived, and went on because a bounded wait of its own
// had run out, would be counted for one meeting twice, and the warps that it
// then leaves behind would never be let go. Between two meetings a warp waits
// for nothing without a limit, so every meeting takes place, also when some
// have given up.
#pragma once

#ifdef __CUDACC__
#define M2_MEET_FN __device__ __forceinline__
#else
#define M2_MEET_FN inline
#endif

namespace m2 {

// A softmax warp of tile i: work(j) makes the weights of chunk j.
template <typename Bar, typename Work>
M2_MEET_FN void tile_rows_meet(Bar bar, int i, int chunks, Work work) {
    if (chunks > 0) bar.sync(i);
    for (int j = 0; j < chunks; ++j) {
        work(j);
        bar.sync(i);
    }
}

// A warp that serves both tiles, of chunks0 and chunks1 <= chunks chunks:
// before(j) ahead of the meetings j, then after(i, j) behind that of tile i.
template <typename Bar, typename Before, typename After>
M2_MEET_FN void tile_turns_meet(Bar bar, int chunks, int chunks0, int chunks1, Before before, After after) {
    for (int j = 0; j <= chunks; ++j) {
        before(j);
#ifdef __CUDACC__
#pragma unroll
#endif
        for (int i = 0; i < 2; ++i) {
            const int n = i ? chunks1 : chunks0;
            if (n == 0 || j > n) continue;
            bar.sync(i);
            after(i, j);
        }
    }
}

}  // namespace m2
