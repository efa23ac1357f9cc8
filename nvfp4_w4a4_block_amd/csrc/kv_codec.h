// The FP8 KV-cache codec's conversion, shared by the codec (kv_fp8.hip) and the
// paged cache's append (kv_pages.hip), whose bytes are the same.
#pragma once

#include "device_common.h"

namespace nvfp4 {

// Four values -> four E4M3 bytes (value i in byte i) with the hardware
// conversion after clamping to +-448.  On gfx950 this is, for every finite
// input, round to nearest even with saturation and the input's sign bit (checked
// on 50M inputs: every E4M3 midpoint and its float32 neighbours, subnormals,
// signed zeros and saturating values): the clamp supplies the saturation that
// the conversion alone would turn into NaN.  The clamp's minimum and maximum are
// those that keep NaN (v_maximum3_f32, v_minimum3_f32; v_med3_f32 would make it
// -448), which the conversion turns into a NaN code.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const auto clamp = [](float y) {
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(y, -kE4M3Max), kE4M3Max);
  };
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp(a), clamp(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp(c), clamp(d), w, true);
}

}  // namespace nvfp4
