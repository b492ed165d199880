// Barriers of the decode attention's tiles (attention_tc.cu). Plain C++ for the host too.
#pragma once

#ifdef __CUDACC__
#define DMTP_TILES __host__ __device__ __forceinline__
#else
#define DMTP_TILES inline
#endif

// A CTA's tiles are numbered through. Two of them are under way: a tile's scores are issued before
// the weights of the tile before it are waited for, so the softmax may be done with both when the
// issuing thread looks. A parity tells only the phase in progress from the one before it: a single
// barrier, two phases on, shows the parity of one that is not there yet, and the wait for it never
// ends. So what is told of a tile (its scores, its weights) goes to one of two barriers in turn, of
// which the next phase needs what the waiting side has not issued.
constexpr int kTileBars = 2;
DMTP_TILES int tile_bar(int tile) { return tile % kTileBars; }
DMTP_TILES unsigned tile_parity(int tile) { return (unsigned)(tile / kTileBars) & 1u; }
