// fp4_turns.h -- how the accumulators of the 4-bit product's CTA pairs go from tile to tile
// (kernels_fp4_pair.cu): which one a cluster's n-th tile has, and which phases of the barriers it
// waits for.  Plain functions, so that every order of the arrivals can be walked on a host.
//
// Even tiles of a cluster have one accumulator, odd ones the other; the two share some columns.  The
// MMAs of tile n write the common columns, which the epilogue must have read of tile n - 1, and
// columns of their own, which it must have read of tile n - 2.  A warp of the epilogue reads its
// common columns of a tile, arrives, then reads its own ones: its arrival for tile n - 1 comes behind
// everything it reads of tile n - 2, so that one wait covers both.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define DGB_TURNS __host__ __device__ __forceinline__
#else
#define DGB_TURNS inline
#endif

namespace dgb {

// the accumulator of a cluster's n-th tile, and the parity of the phase of acc_full that says its sums
// are complete
DGB_TURNS uint32_t fp4_turn(uint32_t n) { return n & 1u; }

// The parity of the phase of acc_empty that tile n's MMAs wait for, its n-th: every warp arrives once
// a tile, and for no tile whose sums are not made, so the barrier cannot be a phase further.
DGB_TURNS uint32_t fp4_empty_parity(uint32_t n) { return (n & 1u) ^ 1u; }

}  // namespace dgb
