// The way of an epilogue warp of the block-scaled product (gemm_fp8.cu) through its tiles.
//
// Where the output is staged, the four warps of a warpgroup meet at barriers that wait without a
// limit, once or more a tile.  So a warp whose own bounded wait gave up must not leave by itself:
// its siblings may have seen the same phase complete just after it gave up.  It goes on to the
// tile's vote (a wait that gave up has raised the CTA's abort flag, so later ones return at once),
// and all four leave by what the vote says of that flag.  Plain C++, so that the order is tested on
// the host with waits that fail at every place.
#pragma once

#ifdef __CUDACC__
#define MTFM_FLOW __device__ __forceinline__
#else
#define MTFM_FLOW inline
#endif

namespace mtfm {

// scale():   fetches the scale of the next block.
// begin(t):  start of a tile.
// blocks(t): adds up the tile's blocks (and, kAhead, fetches the next tile's first scale).
// vote():    the warpgroup's decision: whether no wait has given up.
// finish(t): the tile's output; a wait in it that gives up is found by the next tile's vote.
// next():    end of a tile.
// kAhead: a tile's first scale is fetched before the loop and in the last block of the tile before.
template <bool kAhead, class Scale, class Begin, class Blocks, class Vote, class Finish,
          class Next>
MTFM_FLOW void epilogue_tiles(int first, int n_tiles, int step, Scale scale, Begin begin, Blocks blocks, Vote vote,
                              Finish finish, Next next) {
  if (kAhead && first < n_tiles) scale();
  for (int t = first; t < n_tiles; t += step) {
    begin(t);
    if (!kAhead) scale();
    blocks(t);
    if (!vote()) break;
    finish(t);
    next();
  }
}

}  // namespace mtfm
