// Outputs of the tile kernels on their way from the matrix unit's order to rows of y.
#pragma once

#include "w4_device.h"

namespace w4 {

// Outputs by way of LDS: sixteen rows of 64 outputs that a wavefront holds in the
// matrix unit's order are written to a stage of its own, kStagePitch words a row, and
// stored from there 16 bytes per lane, so that one store covers whole lines of y (4096 x 9216
// fp32 outputs of K = 1152: 94 us, and 115 us with each lane's outputs stored from its
// registers; bf16 64 us either way).  Stores go by 16 bytes whatever the
// alignment of a row of y, which the hardware allows (N = 9217: bf16 78 us, 140 us one
// output at a time; fp32 99 and 211 us).
// (The pitch of 68 words spreads sixteen rows over the banks.)
constexpr int kStagePitch = 68, kStageBytes = 16 * kStagePitch * 4;

typedef uint32_t piece_at_any __attribute__((ext_vector_type(4), aligned(1)));

// Stores rows m0 .. m0 + 15 below m1, outputs n0 .. n0 + 63 below N: value(word, s, e) of the
// staged words is the output of row m0 + stage_row(s) and column n0 + stage_col() + e.
template <bool kF32>
constexpr int kStageOut = kF32 ? 4 : 8;  // consecutive outputs per lane
template <bool kF32>
__device__ __forceinline__ int stage_col() {
  return kStageOut<kF32> * ((threadIdx.x & 63) % (64 / kStageOut<kF32>));
}
template <bool kF32>
__device__ __forceinline__ int stage_row(int s) {
  return kStageOut<kF32> * s + (threadIdx.x & 63) / (64 / kStageOut<kF32>);
}
// kPast: whole pieces are stored past the caches.
template <bool kF32, bool kPast = false, class Value>
__device__ __forceinline__ void store_stage(const uint32_t* stage, void* y, int N, int m0, int m1, int n0, Value value) {
  constexpr int E = kStageOut<kF32>;
  // the stage is this wavefront's own, and its LDS operations run in order
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  const int n = n0 + stage_col<kF32>(), count = min(E, N - n);
#pragma unroll
  for (int s = 0; s < 16 / E; ++s) {
    const int m = m0 + stage_row<kF32>(s);
    if (m >= m1 || count <= 0) continue;
    const uint4* from = reinterpret_cast<const uint4*>(stage + stage_row<kF32>(s) * kStagePitch + stage_col<kF32>());
    float v[E];
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const uint4 w = from[e / 4];
      v[e] = value(w.x, s, e);
      v[e + 1] = value(w.y, s, e + 1);
      v[e + 2] = value(w.z, s, e + 2);
      v[e + 3] = value(w.w, s, e + 3);
    }
    const int64_t at = (int64_t)m * N + n;
    if constexpr (kF32) {
      float* to = static_cast<float*>(y) + at;
      if (count == E) {
        if constexpr (kPast)
          __builtin_nontemporal_store(
              piece_at_any{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])},
              reinterpret_cast<piece_at_any*>(to));
        else __builtin_memcpy(to, v, 16);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e < count) to[e] = v[e];
      }
    } else {
      uint16_t* to = static_cast<uint16_t*>(y) + at;
      uint32_t u[E / 2];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) u[e] = f32x2_to_bf16x2(v[2 * e], v[2 * e + 1]);
      if (count == E) {
        if constexpr (kPast) __builtin_nontemporal_store(piece_at_any{u[0], u[1], u[2], u[3]}, reinterpret_cast<piece_at_any*>(to));
        else __builtin_memcpy(to, u, 16);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e < count) to[e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
      }
    }
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace w4
