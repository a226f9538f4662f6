// Host-side launches of the gated delta rule's kernels.
#pragma once

#include <type_traits>

#include "gdelta.h"

namespace gdelta {

// How the forward pass over the chunks has its 16-column tiles: up to kPairTiles of them (kPairTilesSave with what a backward
// pass reads, 16-bit inputs) each has two waves of its own; more share their chunks' fragments in LDS, or, f32 inputs, have
// one wave each.  2048 tokens of 128 x 128: bf16 forwards 155 us against 186 at 64 heads (512 tiles), 249 against 217 at
// 80; bf16 training passes 318 against 330 at 32 heads (256 tiles), 408 and 403 at 40, 574 and 558 at 64; f32 forwards 305
// against 395 at 64 heads, 541 and 514 at 96, training passes 972 and 1076, 1447 and 1429.
constexpr unsigned kPairTiles = 512, kPairTilesSave = 256;

// Tiles of a workgroup that shares its fragments in LDS (it fills a CU): 3 where that takes no more rounds over the 256 CUs
// than 4, and one (ONE) while there is a CU for each.  The forward pass of 80 heads of 8 tiles takes 566 us with 3 and 665
// with 4, the reverse pass 570 and 689; a training pass of 2048 tokens 1089 with 3 and 896 with 4 at 128 heads, 316 with
// one tile and 326 with 3 at 32, 487 and 409 at 40.  With 2 it was within 2 % of 3, with 8 slower than 4 at every count of
// heads.  launch(integral_constant, grid).
template <bool ONE, class Launch>
void ring_tiles(unsigned heads, unsigned tiles, Launch launch) {
  const unsigned g3 = heads * ((tiles + 2) / 3), g4 = heads * ((tiles + 3) / 4);
  if constexpr (ONE) {
    if (heads * tiles <= 256) return launch(std::integral_constant<int, 1>{}, heads * tiles);
  }
  if ((g3 + 255) / 256 <= (g4 + 255) / 256) launch(std::integral_constant<int, 3>{}, g3);
  else launch(std::integral_constant<int, 4>{}, g4);
}

// Chunked forward; `save`: also what the backward pass reads.
hipError_t launch_fwd(Act act, const FwdArgs& a, bool save, hipStream_t st);
// Token-by-token forward (a.h0 may be a.h_last).
hipError_t launch_step(Act act, const FwdArgs& a, hipStream_t st);
// Backward of the chunked forward that saved.
hipError_t launch_bwd(Act act, const BwdArgs& a, hipStream_t st);

}  // namespace gdelta
