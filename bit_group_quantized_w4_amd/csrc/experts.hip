// The way to the experts and back: the slots of a router's choice (tokens x top, the
// expert of each) sorted by expert, rows of x copied into that order, and the experts'
// rows weighted and added up token by token, with the gradients of both.
//
//   place[t][j]   row of slot (t, j): slots of expert 0 first, those of one expert in
//                 their own order (a stable counting sort); -1 for a slot of no expert
//   xs[place[t][j]] = x[t],               dx[t] = sum_j dxs[place[t][j]]
//   out[t] = sum_j w[t][j] y[place[t][j]],
//   dy[place[t][j]] = w[t][j] dout[t],    dw[t][j] = sum_k dout[t][k] y[place[t][j]][k]
//
// Sums run in fp32 in a fixed order; nothing is added with atomics but counts.
#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {
namespace {

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
// The expert of slot i; `experts` for one that is not in [0, experts).
template <typename Id>
__device__ __forceinline__ int key_of(const Id* __restrict__ ids, int i, int experts) {
  const Id v = ids[i];
  return v >= 0 && v < (Id)experts ? (int)v : experts;
}

// Exclusive prefix sums of count[0 .. n) in LDS, by a block of 256 threads; count[n] = all.
__device__ __forceinline__ void scan_counts(int* count, int n, int* wave_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int before = 0;
  for (int at = 0; at < n; at += 256) {
    const int i = at + threadIdx.x;
    const int v = i < n ? count[i] : 0;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    if (lane == 63) wave_sum[wave] = s;
    __syncthreads();
    int base = before;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    before += wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];
    if (i < n) count[i] = base + s - v;
    __syncthreads();
  }
  if (threadIdx.x == 0) count[n] = before;
  __syncthreads();
}

// Counts of each block's `chunk` slots by expert: hist[block][experts + 1].
template <typename Id>
__global__ __launch_bounds__(256) void expert_count_kernel(const Id* __restrict__ ids, int slots, int chunk, int experts,
                                                           int* __restrict__ hist) {
  extern __shared__ int lds[];
  for (int e = threadIdx.x; e <= experts; e += 256) lds[e] = 0;
  __syncthreads();
  const int from = blockIdx.x * chunk, to = min(slots, from + chunk);
  for (int i = from + threadIdx.x; i < to; i += 256) atomicAdd(&lds[key_of(ids, i, experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= experts; e += 256) hist[(int64_t)blockIdx.x * (experts + 1) + e] = lds[e];
}

// Places of each block's slots.  The block's first row of expert e is the rows of the
// experts before it and of the blocks before this one; within the block, 256 slots at a
// time, a slot's rank among its expert's is found by comparing keys: the lanes of its
// wavefront before it by a match of all key bits, the wavefronts before by their counts.
template <typename Id>
__global__ __launch_bounds__(256) void expert_place_kernel(const Id* __restrict__ ids, int slots, int chunk, int experts,
                                                           const int* __restrict__ hist, int* __restrict__ offsets,
                                                           int* __restrict__ place, int* __restrict__ order) {
  extern __shared__ int lds[];  // next row of each expert [experts + 2], then the counts of four wavefronts
  __shared__ int wave_sum[4];
  __shared__ int keys[256];
  int* next = lds;
  const int bins = experts + 1, blocks = gridDim.x;
  for (int e = threadIdx.x; e < bins; e += 256) {
    int all = 0;
    for (int b = 0; b < blocks; ++b) all += hist[(int64_t)b * bins + e];
    next[e] = all;
  }
  __syncthreads();
  scan_counts(next, bins, wave_sum);
  const int valid = next[experts];  // rows of the experts, the dropped slots come after
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= experts; e += 256) offsets[e] = next[e];
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += 256) {
    int before = 0;
    for (int b = 0; b < (int)blockIdx.x; ++b) before += hist[(int64_t)b * bins + e];
    next[e] += before;
  }
  __syncthreads();
  const int from = blockIdx.x * chunk, to = min(slots, from + chunk);
  for (int i0 = from; i0 < to; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const int key = i < to ? key_of(ids, i, experts) : -1;
    keys[threadIdx.x] = key;
    __syncthreads();
    int rank = 0, same = 0;  // of the 256, slots of this expert before this one, and in all
    if (key >= 0) {
      for (int j = 0; j < 256; ++j) {
        const bool eq = keys[j] == key;
        same += eq;
        rank += eq && j < (int)threadIdx.x;
      }
      const int row = next[key] + rank;
      place[i] = key < experts ? row : -1;
      order[row] = key < experts ? i : -1;
    }
    __syncthreads();
    if (key >= 0 && rank == same - 1) next[key] += same;
    __syncthreads();
  }
  (void)valid;
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(1)));

// A row of `bytes` bytes is moved in pieces of 16 at any alignment (which the hardware
// allows); the last piece ends with the row, over bytes of the one before.  A row
// shorter than 16 bytes is moved byte by byte.
__device__ __forceinline__ int64_t piece_at(int64_t p, int64_t bytes) { return min<int64_t>(p * 16, bytes - 16); }

// A block per token: its row is read once and written to the rows of its slots.  Rows that
// no slot has (behind the last expert's) are filled with zeros, `top` of them per block.
__global__ __launch_bounds__(256) void expert_take_kernel(const uint8_t* __restrict__ x, int64_t bytes, int top,
                                                          int slots, const int* __restrict__ valid_at,
                                                          const int* __restrict__ place, uint8_t* __restrict__ xs) {
  const int t = blockIdx.x;
  const int valid = min(max(*valid_at, 0), slots);
  const uint8_t* from = x + (int64_t)t * bytes;
  const int64_t pieces = bytes < 16 ? 0 : (bytes + 15) / 16;
  for (int64_t p = threadIdx.x; p < pieces; p += 256) {
    const int64_t at = piece_at(p, bytes);
    const u32x4a v = *reinterpret_cast<const u32x4a*>(from + at);
    for (int j = 0; j < top; ++j) {
      const int row = place[t * top + j];
      if ((unsigned)row < (unsigned)slots) *reinterpret_cast<u32x4a*>(xs + row * bytes + at) = v;
    }
    for (int j = max(0, valid - t * top); j < top; ++j)
      *reinterpret_cast<u32x4a*>(xs + (int64_t)(t * top + j) * bytes + at) = u32x4a{0, 0, 0, 0};
  }
  if (bytes < 16 && threadIdx.x < bytes) {
    const uint8_t v = from[threadIdx.x];
    for (int j = 0; j < top; ++j) {
      const int row = place[t * top + j];
      if ((unsigned)row < (unsigned)slots) xs[row * bytes + threadIdx.x] = v;
    }
    for (int j = max(0, valid - t * top); j < top; ++j) xs[(int64_t)(t * top + j) * bytes + threadIdx.x] = 0;
  }
}

__device__ __forceinline__ float value_at(const void* p, bool f32, int64_t i) {
  if (f32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ void put_value(void* p, bool f32, int64_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v);
}

// out[t] = sum_j w[t][j] y[place[t][j]], a block per token (w nullptr: ones).
__global__ __launch_bounds__(256) void expert_combine_kernel(const CombineArgs a) {
  const int t = blockIdx.x;
  for (int64_t k = threadIdx.x; k < a.K; k += 256) {
    float s = 0.0f;
    for (int j = 0; j < a.top; ++j) {
      const int row = a.place[t * a.top + j];
      if ((unsigned)row >= (unsigned)a.slots) continue;
      const float w = a.w ? value_at(a.w, a.w_f32, t * a.top + j) : 1.0f;
      s = fmaf(w, value_at(a.y, a.y_f32, row * a.K + k), s);
    }
    put_value(a.out, a.out_f32, t * a.K + k, s);
  }
}

// A block per token; dy or dw may be nullptr.
__global__ __launch_bounds__(256) void expert_combine_backward_kernel(const CombineBackwardArgs a) {
  __shared__ float part[4];
  const int t = blockIdx.x;
  for (int j = 0; j < a.top; ++j) {
    const int slot = t * a.top + j, row = a.place[slot];
    const bool there = (unsigned)row < (unsigned)a.slots;
    const float w = a.w ? value_at(a.w, a.w_f32, slot) : 1.0f;
    float s = 0.0f;
    if (there)
      for (int64_t k = threadIdx.x; k < a.K; k += 256) {
        const float g = value_at(a.dout, a.out_f32, t * a.K + k);
        if (a.dy) put_value(a.dy, a.y_f32, row * a.K + k, w * g);
        if (a.dw) s = fmaf(g, value_at(a.y, a.y_f32, row * a.K + k), s);
      }
    if (a.dw) {
#pragma unroll
      for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
      __syncthreads();
      if (threadIdx.x == 0) put_value(a.dw, a.w_f32, slot, part[0] + part[1] + part[2] + part[3]);
      __syncthreads();
    }
  }
  if (a.dy) {
    const int valid = min(max(*a.valid_at, 0), a.slots);
    for (int j = max(0, valid - t * a.top); j < a.top; ++j)
      for (int64_t k = threadIdx.x; k < a.K; k += 256) put_value(a.dy, a.y_f32, (int64_t)(t * a.top + j) * a.K + k, 0.0f);
  }
}

// Slots per block of the sort: at least 1024, at most 64 blocks.
int sort_chunk(int64_t slots) {
  const int64_t per = (slots + 63) / 64;
  return (int)((per < 1024 ? 1024 : per) + 255) / 256 * 256;
}
int sort_blocks(int64_t slots) {
  const int chunk = sort_chunk(slots);
  const int64_t n = (slots + chunk - 1) / chunk;
  return n < 1 ? 1 : (int)n;
}

template <typename Id>
hipError_t launch_sort(const Id* ids, int64_t slots, int64_t experts, int32_t* offsets, int32_t* place, int32_t* order,
                       int* hist, hipStream_t st) {
  const int chunk = sort_chunk(slots), blocks = sort_blocks(slots);
  const size_t lds = (size_t)(experts + 2) * sizeof(int);
  expert_count_kernel<Id><<<blocks, 256, lds, st>>>(ids, (int)slots, chunk, (int)experts, hist);
  if (const hipError_t e = hipGetLastError()) return e;
  expert_place_kernel<Id><<<blocks, 256, lds, st>>>(ids, (int)slots, chunk, (int)experts, hist, offsets, place, order);
  return hipGetLastError();
}

}  // namespace

size_t expert_sort_workspace(int64_t slots, int64_t experts) {
  return (size_t)sort_blocks(slots) * (size_t)(experts + 1) * sizeof(int);
}

hipError_t launch_expert_sort(const void* ids, bool wide, int64_t slots, int64_t experts, int32_t* offsets, int32_t* place,
                              int32_t* order, void* workspace, hipStream_t st) {
  int* hist = static_cast<int*>(workspace);
  return wide ? launch_sort(static_cast<const int64_t*>(ids), slots, experts, offsets, place, order, hist, st)
              : launch_sort(static_cast<const int32_t*>(ids), slots, experts, offsets, place, order, hist, st);
}

hipError_t launch_expert_take(const void* x, int64_t tokens, int64_t bytes, int64_t top, const int32_t* offsets,
                              int64_t experts, const int32_t* place, void* xs, hipStream_t st) {
  expert_take_kernel<<<(unsigned)tokens, 256, 0, st>>>(static_cast<const uint8_t*>(x), bytes, (int)top,
                                                       (int)(tokens * top), offsets + experts, place,
                                                       static_cast<uint8_t*>(xs));
  return hipGetLastError();
}

hipError_t launch_expert_combine(const CombineArgs& a, hipStream_t st) {
  expert_combine_kernel<<<(unsigned)(a.slots / a.top), 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const CombineBackwardArgs& a, hipStream_t st) {
  expert_combine_backward_kernel<<<(unsigned)(a.slots / a.top), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace w4
