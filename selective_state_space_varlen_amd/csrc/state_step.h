// Shared by the single-token steps on pools of states.
#pragma once

#include "delta_common.h"

namespace ssmp {

// A workgroup takes 32 columns of one head's state, eight lanes of 16 bytes to
// a row (one 128-byte line): 4 workgroups a head at Dv = 128, so that a single
// sequence of 32 heads already has 128 of them.
constexpr int kStepCols = 32;
constexpr int kStepThreads = 256;
constexpr int kStepRowGroups = kStepThreads / (kStepCols / 4);  // 32
constexpr int kStepMaxDk = 128;

// The state passes once each way and would push everything else out of the
// caches: without temporal hint 246 us for 256 sequences of 32 heads of
// 128 x 128, with it 211 (5.1 TB/s); the same 4.7 us for one sequence.
__device__ __forceinline__ float4 state_load(const float* p) {
    const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void state_store(float* p, float4 v) {
    __builtin_nontemporal_store(f32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<f32x4*>(p));
}

}  // namespace ssmp
