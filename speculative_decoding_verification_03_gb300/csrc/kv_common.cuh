// Shared by the kernels around the paged key-value cache: finding a packed
// token's sequence, a token tree's ancestors, and the e4m3 conversions.
#pragma once

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

// The sequence of packed token t: the largest b in [0, B) with start[b] <= t
// (-1 if there is none, or start[B] <= t: a token of padding).  All lanes of a
// warp search together, 32 probes a round, so 1024 sequences take two
// dependent loads and not ten.
__device__ __forceinline__ int find_sequence(const int32_t *start, int B, int t, int lane) {
  int lo = 0, n = B;  // the answer lies in [lo, lo + n), or start[lo] > t
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool le = at < n && __ldg(start + lo + at) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return (__ldg(start + lo) <= t && t < __ldg(start + B)) ? lo : -1;
}

// Parent of node i > 0 of a chunk's tree; bad entries are taken as 0 and
// reported, so every walk towards the root ends.
__device__ __forceinline__ int tree_parent(const int32_t *parents, int tree_nodes, int i, bool &bad) {
  if (i >= tree_nodes) {
    bad = true;
    return 0;
  }
  const int p = __ldg(parents + i);
  if (p < 0 || p >= i) {
    bad = true;
    return 0;
  }
  return p;
}

// Two fp32 values to two e4m3 or e5m2 codes (nearest even, saturating), `lo` in the
// low byte, and e4m3 pairs widened to half pairs (exact).
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_from_f32(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ float2 f32x2_from_f16x2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ uint32_t bf16x2_from_f32(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^(byte - 127) for a scale byte in [1, 254]
__device__ __forceinline__ float scale_of_byte(uint32_t byte) { return __uint_as_float(byte << 23); }

}  // namespace sv
