// rope.cuh -- rotary angles shared by idx_rope and idx_latent_append.
//
// A pair turns by position * f radians.  f / (2 pi) is held as a 64-bit binary
// fraction of a turn (the step); position * step modulo 2^64 then is the
// fraction of a turn with the whole turns already taken off, exact for any
// 64-bit position, in one integer multiply.  Its top 32 bits, signed, are the
// angle in units of pi times 2^31; rounding them to fp32 costs at most
// pi * 2^-25 = 1e-7 radians, below the rounding of the fp32 products.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dsaidx {

// (cos, sin) of the angle, times the amplitude.
__device__ __forceinline__ float2 rope_cs(int64_t position, uint64_t step, float amplitude) {
    const uint64_t phase = static_cast<uint64_t>(position) * step;
    const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

// The pair (a, b) turned: (a c - b s, a s + b c).
__device__ __forceinline__ float2 rope_turn(float a, float b, float2 cs) {
    return make_float2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

}  // namespace dsaidx
