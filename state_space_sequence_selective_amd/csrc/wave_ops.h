// Sums, maxima and scans over the lanes of a wave by DPP (no LDS traffic): gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace waveops {

// lane exchanges inside rows of 16 lanes (DPP): lane ^ 1, lane ^ 2, 7 - lane of each half, 15 - lane
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum8(float v) {   // over aligned groups of eight lanes
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  return v + dpp<0x141>(v);
}
__device__ __forceinline__ float sum16(float v) {   // over the 16 lanes of one l / 16 group
  v = sum8(v);
  return v + dpp<0x140>(v);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp(static_cast<int>(u), CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp(static_cast<int>(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double sum16(double v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  return v + dpp<0x140>(v);
}

// lane 15 of rows 0 and 2 to rows 1 and 3, then lane 31 to rows 2 and 3; zero elsewhere
__device__ __forceinline__ float bcast15(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xa, 0xf, false));
}
__device__ __forceinline__ float bcast31(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xc, 0xf, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ float wave_max(float v) {   // of values >= 0
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  v = fmaxf(v, bcast15(v));
  return last_lane(fmaxf(v, bcast31(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  v += bcast15(v);
  return last_lane(v + bcast31(v));
}
// inclusive sums over the wave's lanes
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, true);
  return v + __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double wave_scan(double v) {
  v = scan_step<0x111, 0xf>(v);   // from the lane 1, 2, 4, 8 below in the row
  v = scan_step<0x112, 0xf>(v);
  v = scan_step<0x114, 0xf>(v);
  v = scan_step<0x118, 0xf>(v);
  v = scan_step<0x142, 0xa>(v);
  return scan_step<0x143, 0xc>(v);
}

}  // namespace waveops
