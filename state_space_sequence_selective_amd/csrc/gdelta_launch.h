// Host-side launches of the gated delta rule's kernels.
#pragma once

#include "gdelta.h"

namespace gdelta {

// Up to this many 16-column tiles the passes over the chunks give two waves to each: 1024 SIMDs hold one wave of theirs
// each (over 256 registers), so more tiles than 512 would wait for others to end.
constexpr unsigned kPairTiles = 512;

// Chunked forward; `save`: also what the backward pass reads.
hipError_t launch_fwd(Act act, const FwdArgs& a, bool save, hipStream_t st);
// Token-by-token forward (a.h0 may be a.h_last).
hipError_t launch_step(Act act, const FwdArgs& a, hipStream_t st);
// Backward of the chunked forward that saved.
hipError_t launch_bwd(Act act, const BwdArgs& a, hipStream_t st);

}  // namespace gdelta
