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
// Sums run in fp32 in a fixed order; nothing is added with atomics but counts.  Every kernel
// moves bytes: what they cannot do without is each row read once and written once.
#include "w4_device.h"
#include "w4_launch.h"
#include "w4_rows.h"

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

// Exclusive prefix sums of count[0 .. n) in LDS, by a block of 256 threads.
__device__ __forceinline__ void scan_counts(int* count, int n, int* wave_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int before = 0;
  for (int at = 0; at < n; at += 256) {
    const int i = at + threadIdx.x;
    const int v = i < n ? count[i] : 0;
    const int s = lanes_upto(v);
    if (lane == 63) wave_sum[wave] = s;
    __syncthreads();
    int base = before;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    before += wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];
    if (i < n) count[i] = base + s - v;
    __syncthreads();
  }
}

// Counts of each block's `chunk` slots by expert: hist[block][experts + 1].
template <typename Id>
__global__ __launch_bounds__(256) void expert_count_kernel(const Id* __restrict__ ids, int slots, int chunk, int experts,
                                                           int* __restrict__ hist) {
  extern __shared__ int count[];
  for (int e = threadIdx.x; e <= experts; e += 256) count[e] = 0;
  __syncthreads();
  const int from = blockIdx.x * chunk, to = min(slots, from + chunk);
  for (int i = from + threadIdx.x; i < to; i += 256) atomicAdd(&count[key_of(ids, i, experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= experts; e += 256) hist[(int64_t)blockIdx.x * (experts + 1) + e] = count[e];
}

// Places of each block's slots.  The block's first row of expert e follows the rows of the
// experts before it and those of the blocks before this one.  Within the block, 256 slots at
// a time: the lanes of a wavefront with a slot's key are found by one ballot per bit of
// the keys, and the wavefronts take their turns at the expert's next row.
//
// Bound by latency: 32760 slots of 128 experts take 9 us, 3 of them the counts; 120000 of 500 21 us.
template <typename Id>
__global__ __launch_bounds__(256) void expert_place_kernel(const Id* __restrict__ ids, int slots, int chunk, int experts,
                                                           const int* __restrict__ hist, int* __restrict__ offsets,
                                                           int* __restrict__ place, int* __restrict__ order) {
  extern __shared__ int lds[];
  __shared__ int wave_sum[4];
  const int bins = experts + 1, blocks = gridDim.x;
  int *next = lds, *before = lds + bins;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < 2 * bins; e += 256) lds[e] = 0;
  __syncthreads();
  // each wavefront adds up a quarter of the blocks
  const int b0 = blocks * wave / 4, b1 = blocks * (wave + 1) / 4;
  for (int e = lane; e < bins; e += 64) {
    int all = 0, mine = 0;
    for (int b = b0; b < b1; b += 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {  // on their way together
        const int v = b + i < b1 ? hist[(int64_t)(b + i) * bins + e] : 0;
        all += v;
        mine += b + i < (int)blockIdx.x ? v : 0;
      }
    }
    atomicAdd(&next[e], all);
    atomicAdd(&before[e], mine);
  }
  __syncthreads();
  scan_counts(next, bins, wave_sum);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < bins; e += 256) offsets[e] = next[e];
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += 256) next[e] += before[e];
  __syncthreads();

  const int bits = 32 - __builtin_clz(bins);
  const int from = blockIdx.x * chunk, to = min(slots, from + chunk);
  for (int i0 = from; i0 < to; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const int key = i < to ? key_of(ids, i, experts) : -1;
    uint64_t same = __ballot(key >= 0);
    for (int k = 0; k < bits; ++k) {
      const uint64_t set = __ballot(key >> k & 1);
      same &= key >> k & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1)), n = __popcll(same);
    int row = 0;
    for (int w = 0; w < 4; ++w) {
      if (w == wave) {
        if (key >= 0) row = next[key] + rank;
        // one lane of each key writes what the others have read: the fence and the barrier hold the
        // compiler to that order, the LDS runs a wavefront's operations in it
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (key >= 0 && rank == n - 1) next[key] = row + 1;
      }
      __syncthreads();
    }
    if (key >= 0) {
      place[i] = key < experts ? row : -1;
      order[row] = key < experts ? i : -1;
    }
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
// A row is moved in pieces of 16 bytes at any alignment (which the hardware allows); the
// last piece ends with the row, over bytes of the one before.  Rows shorter than that go
// value by value.
typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(1)));

// Loads and stores past the caches, which pays where whole lines are written (us through the
// caches and past them: 4095 x 5120 bf16 to eight rows each 76 and 66; 20000 x 700 to
// six, whose rows end inside a line, 33 and 52).
template <bool kPast>
__device__ __forceinline__ void put_piece(void* to, const u32x4a& v) {
  if constexpr (kPast) __builtin_nontemporal_store(v, static_cast<u32x4a*>(to));
  else *static_cast<u32x4a*>(to) = v;
}
template <bool kPast>
__device__ __forceinline__ u32x4a get_piece(const void* from) {
  if constexpr (kPast) return __builtin_nontemporal_load(static_cast<const u32x4a*>(from));
  else return *static_cast<const u32x4a*>(from);
}
inline bool whole_lines(const void* p, int64_t row_bytes) {
  return row_bytes % 128 == 0 && reinterpret_cast<uintptr_t>(p) % 128 == 0;
}

__host__ __device__ constexpr int64_t pieces_of(int64_t bytes) { return bytes < 16 ? 1 : (bytes + 15) / 16; }

// Piece p of a row is read from `from` and written to the rows of xs that its token's slots have
// (row(j), j < top), and zeros to the rows that no slot has among the token's share of them.
template <bool kPast, class Row>
__device__ __forceinline__ void take_piece(const uint8_t* from, int64_t bytes, int64_t p, int top, int slots, int first,
                                           int valid, uint8_t* xs, Row row) {
  if (bytes >= 16) {
    const int64_t at = min<int64_t>(p * 16, bytes - 16);
    const u32x4a v = *reinterpret_cast<const u32x4a*>(from + at);
    for (int j = 0; j < top; ++j) {
      const int r = row(j);
      if ((unsigned)r < (unsigned)slots) put_piece<kPast>(xs + r * bytes + at, v);
    }
    for (int j = max(0, valid - first); j < top; ++j) put_piece<kPast>(xs + (int64_t)(first + j) * bytes + at, u32x4a{0, 0, 0, 0});
  } else {
    for (int64_t b = 0; b < bytes; ++b) {
      const uint8_t v = from[b];
      for (int j = 0; j < top; ++j) {
        const int r = row(j);
        if ((unsigned)r < (unsigned)slots) xs[r * bytes + b] = v;
      }
      for (int j = max(0, valid - first); j < top; ++j) xs[(int64_t)(first + j) * bytes + b] = 0;
    }
  }
}

// A row is read once and written to the rows of its token's slots: `lanes` lanes of a
// wavefront (a power of two, 64 for long rows) take that many pieces of one token each.
//
// Bound by memory: 4095 rows of 5120 bf16 to eight rows each (377 MB) take 66 us (5.7 TB/s).
template <bool kUniform, bool kPast>
__global__ __launch_bounds__(256) void expert_take_kernel(const uint8_t* __restrict__ x, int64_t bytes, int slots, int top,
                                                          const int* __restrict__ valid_at, const int* __restrict__ place,
                                                          uint8_t* __restrict__ xs, int lanes, int chunks, int t0, int t1) {
  const int64_t pieces = pieces_of(bytes);
  int64_t task;
  int64_t p;
  if constexpr (kUniform) {
    task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p = threadIdx.x & 63;
  } else {
    task = ((int64_t)blockIdx.x * 256 + threadIdx.x) / lanes;
    p = threadIdx.x & (lanes - 1);
  }
  int t = (int)(task / chunks);
  p += (task - (int64_t)t * chunks) * lanes;
  t += t0;
  if (t >= t1 || p >= pieces) return;
  const int valid = min(max(*valid_at, 0), slots);
  take_piece<kPast>(x + t * bytes, bytes, p, top, slots, t * top, valid, xs, [&](int j) { return place[t * top + j]; });
}

// Few slots: the sort and the rows of a call in one launch.  A block has one token and every
// slot's key in LDS; a slot's row is the number of slots that come before it, by expert and
// then by index, which 256 threads count with ballots.  The offsets (the number of keys below
// each) are shared out over the blocks.  `bytes` 0: no rows.
constexpr int kFewSlots = 2048, kMostTop = 64, kFewCounts = 8192;

template <typename Id>
__global__ __launch_bounds__(256) void expert_dispatch_kernel(const uint8_t* __restrict__ x, int64_t bytes,
                                                              const Id* __restrict__ ids, int tokens, int top, int experts,
                                                              int* __restrict__ offsets, int* __restrict__ place,
                                                              int* __restrict__ order, uint8_t* __restrict__ xs) {
  __shared__ int keys[kFewSlots];
  __shared__ int counts[4][kMostTop + 1];
  const int slots = tokens * top, t = blockIdx.x, first = t * top;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int i = threadIdx.x; i < slots; i += 256) keys[i] = key_of(ids, i, experts);
  __syncthreads();
  if (t < tokens) {
    // counts[wave][j]: of the wavefront's keys, those before slot `first + j`; j == top: those of an expert
    for (int j = 0; j <= top; ++j) {
      const int key = j < top ? keys[first + j] : experts, at = j < top ? first + j : 0;
      int n = 0;
      for (int i0 = 64 * wave; i0 < slots; i0 += 256) {
        const int i = i0 + lane, k = i < slots ? keys[i] : experts + 1;
        n += __popcll(__ballot(k < key || (k == key && i < at)));
      }
      if (lane == 0) counts[wave][j] = n;
    }
  }
  __syncthreads();
  if (t < tokens) {
    auto row = [&](int j) { return counts[0][j] + counts[1][j] + counts[2][j] + counts[3][j]; };
    const int valid = row(top);
    for (int j = threadIdx.x; j < top; j += 256) {
      const bool there = keys[first + j] < experts;
      place[first + j] = there ? row(j) : -1;
      if (there) order[row(j)] = first + j;
      if (first + j >= valid) order[first + j] = -1;
    }
    if (bytes)
      for (int64_t p = threadIdx.x; p < pieces_of(bytes); p += 256)
        take_piece<false>(x + t * bytes, bytes, p, top, slots, first, valid, xs,
                   [&](int j) { return keys[first + j] < experts ? row(j) : -1; });
  }
  if (slots <= 64) {
    for (int e = t * 256 + threadIdx.x; e <= experts; e += gridDim.x * 256) {
      int n = 0;
      for (int i = 0; i < slots; ++i) n += keys[i] < e;
      offsets[e] = n;
    }
  } else {
    for (int e = t * 4 + wave; e <= experts; e += gridDim.x * 4) {
      int n = 0;
      for (int i0 = 0; i0 < slots; i0 += 64) {
        const int i = i0 + lane;
        n += __popcll(__ballot(i < slots && keys[i] < e));
      }
      if (lane == 0) offsets[e] = n;
    }
  }
}

// Values of a piece, and pieces of values: 16 bytes of y hold 8 bf16 or 4 fp32.
template <bool kF32>
constexpr int kPer = kF32 ? 4 : 8;

template <bool kF32>
__device__ __forceinline__ void widen(const u32x4a& v, float (&to)[kPer<kF32>]) {
#pragma unroll
  for (int e = 0; e < kPer<kF32>; ++e)
    to[e] = kF32 ? __uint_as_float(v[e]) : __uint_as_float(e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
}

// N consecutive values (4 or 8) of either type, at any alignment.
template <int N>
__device__ __forceinline__ void load_values(const void* from, bool f32, int64_t at, float (&to)[N]) {
  if (f32) {
    __builtin_memcpy(to, static_cast<const float*>(from) + at, 4 * N);
  } else {
    uint32_t u[N / 2];
    __builtin_memcpy(u, static_cast<const uint16_t*>(from) + at, 2 * N);
#pragma unroll
    for (int e = 0; e < N; ++e) to[e] = __uint_as_float(e & 1 ? u[e >> 1] & 0xFFFF0000u : u[e >> 1] << 16);
  }
}
typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(1)));
template <bool kPast, int N>
__device__ __forceinline__ void store_values(void* to, bool f32, int64_t at, const float (&v)[N]) {
  if (f32) {
    float* out = static_cast<float*>(to) + at;
#pragma unroll
    for (int e = 0; e < N; e += 4)
      put_piece<kPast>(out + e, u32x4a{__float_as_uint(v[e]), __float_as_uint(v[e + 1]), __float_as_uint(v[e + 2]),
                                       __float_as_uint(v[e + 3])});
  } else {
    uint16_t* out = static_cast<uint16_t*>(to) + at;
    if constexpr (N == 8) {
      put_piece<kPast>(out, u32x4a{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                                   f32x2_to_bf16x2(v[6], v[7])});
    } else {
      const u32x2a u = {f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3])};
      if constexpr (kPast) __builtin_nontemporal_store(u, reinterpret_cast<u32x2a*>(out));
      else *reinterpret_cast<u32x2a*>(out) = u;
    }
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

constexpr int kRowsAtOnce = 8;  // rows of y whose pieces are in flight together

// The rows of slots j0 .. j0 + 7 of token t, -1 for those that have none, and their weights, 0 for those.
template <class Args>
__device__ __forceinline__ void slots_of(const Args& a, int t, int j0, int (&row)[kRowsAtOnce], float (&w)[kRowsAtOnce]) {
#pragma unroll
  for (int j = 0; j < kRowsAtOnce; ++j) {
    const int slot = t * a.top + min(j0 + j, a.top - 1);
    const int r = a.place[slot];
    const bool there = j0 + j < a.top && (unsigned)r < (unsigned)a.slots;
    row[j] = there ? r : -1;
    w[j] = a.w ? value_at(a.w, a.w_f32, slot) : 1.0f;
    if (!there) w[j] = 0.0f;
  }
}

// The pieces at value `at` of those rows; zeros for the rows that are not there.
template <bool kPast, bool kF32>
__device__ __forceinline__ void load_rows(const void* y, int64_t K, const int (&row)[kRowsAtOnce], int64_t at,
                                          u32x4a (&v)[kRowsAtOnce]) {
#pragma unroll
  for (int j = 0; j < kRowsAtOnce; ++j) {
    v[j] = u32x4a{0, 0, 0, 0};
    if (row[j] >= 0)
      v[j] = get_piece<kPast>(static_cast<const uint8_t*>(y) + (row[j] * K + at) * (kF32 ? 4 : 2));
  }
}

// out[t] = sum_j w[t][j] y[place[t][j]] (w nullptr: ones): `lanes` lanes of a wavefront take
// that many pieces of one token, eight slots at a time.
//
// Bound by memory: 4095 x 8 rows of 5120 bf16, 1/16 of them dropped (356 MB), take 60 us (5.9 TB/s); 8 tokens
// of two rows of 2560 3 us, the latency of a place and of its row.
template <bool kUniform, bool kF32>
__global__ __launch_bounds__(256) void expert_combine_kernel(const CombineArgs a, int lanes, int chunks, int t0,
                                                             int t1) {
  constexpr int V = kPer<kF32>;
  int64_t task;
  int p;
  if constexpr (kUniform) {
    task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p = threadIdx.x & 63;
  } else {
    task = ((int64_t)blockIdx.x * 256 + threadIdx.x) / lanes;
    p = threadIdx.x & (lanes - 1);
  }
  int t = (int)(task / chunks);
  p += (int)(task - (int64_t)t * chunks) * lanes;
  t += t0;
  if (t >= t1 || (int64_t)p * V >= a.K) return;
  int row[kRowsAtOnce];
  float w[kRowsAtOnce];
  if (a.K < V) {
    for (int64_t k = 0; k < a.K; ++k) {
      float s = 0.0f;
      for (int j0 = 0; j0 < a.top; j0 += kRowsAtOnce) {
        slots_of(a, t, j0, row, w);
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j)
          if (row[j] >= 0) s = fmaf(w[j], value_at(a.y, kF32, row[j] * a.K + k), s);
      }
      put_value(a.out, a.out_f32, t * a.K + k, s);
    }
    return;
  }
  const int64_t at = min<int64_t>((int64_t)p * V, a.K - V);
  float s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = 0.0f;
  for (int j0 = 0; j0 < a.top; j0 += kRowsAtOnce) {
    slots_of(a, t, j0, row, w);
    u32x4a v[kRowsAtOnce];
    load_rows<false, kF32>(a.y, a.K, row, at, v);
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j) {
      float f[V];
      widen<kF32>(v[j], f);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = fmaf(w[j], f[e], s[e]);
    }
  }
  // Past the caches at every length: rows of out follow each other, so that those which end inside a
  // line gain too (us through the caches and past them: 4095 x 8 rows of 5120 bf16 74.6 and 69.8, of 5121
  // 75.1 and 71.5, fp32 146.6 and 139.7; 20000 x 6 of 700 41.6 and 38.8; 16384 x 2 of 1027 28.9 and 27.7; 32767 x
  // 2 of 257 19.8 and 17.9).  Calls of 5 us or less with such rows take 0.2 us longer (8 x 2 of 2561 3.6 and
  // 3.8; of 512 x 2 of 2560, whole lines, 4.7 and 4.6).
  store_values<true>(a.out, a.out_f32, t * a.K + at, s);
}

// The gradients: W wavefronts of a block, or (W = 0) `lanes` lanes of a wavefront, have a
// token.  They go through its row of dout piece by piece, write w dout to the rows of
// its slots and add up dout y for each of them, eight slots at a time.  dy or dw may be nullptr.
//
// Bound by memory: the same 4095 x 8 rows (692 MB) take 119 to 140 us (4.9 to 5.8 TB/s).
template <int W, bool kPast, bool kF32>
__global__ __launch_bounds__(256) void expert_combine_backward_kernel(const CombineBackwardArgs a, int lanes) {
  constexpr int V = kPer<kF32>;
  const int tokens = a.slots / a.top;
  const int span = W ? 64 * W : lanes;  // threads of a token
  const int t = W ? (int)blockIdx.x * (4 / (W ? W : 1)) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / (W ? W : 1)
                  : (int)(((int64_t)blockIdx.x * 256 + threadIdx.x) / lanes);
  const int mine = threadIdx.x & (span - 1);
  __shared__ float part[4][kRowsAtOnce];
  if (W < 4 && t >= tokens) return;  // (W = 4: a block for each token)
  const int valid = a.dy ? min(max(*a.valid_at, 0), a.slots) : 0;
  const int first = t * a.top;
  const bool whole = a.K >= V;  // else one value at a time
  const int64_t pieces = whole ? (a.K + V - 1) / V : a.K;
  for (int j0 = 0; j0 < a.top; j0 += kRowsAtOnce) {
    int row[kRowsAtOnce];
    float w[kRowsAtOnce], sum[kRowsAtOnce];
    slots_of(a, t, j0, row, w);
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j) sum[j] = 0.0f;
    for (int64_t p = mine; p < pieces; p += span) {
      if (whole) {
        const int64_t at = min<int64_t>(p * V, a.K - V);
        const int fresh = (int)(p * V - at);  // values of the piece that the one before has too
        float g[V];
        load_values<V>(a.dout, a.out_f32, t * a.K + at, g);
        u32x4a v[kRowsAtOnce];
        if (a.dw) load_rows<kPast, kF32>(a.y, a.K, row, at, v);
        if (a.dy) {
#pragma unroll
          for (int j = 0; j < kRowsAtOnce; ++j) {
            float d[V];
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = w[j] * g[e];
            if (row[j] >= 0) store_values<kPast>(a.dy, kF32, row[j] * a.K + at, d);
          }
          const float none[V] = {};
          for (int j = max(j0, valid - first); j < min(a.top, j0 + kRowsAtOnce); ++j)
            store_values<kPast>(a.dy, kF32, (int64_t)(first + j) * a.K + at, none);
        }
        if (a.dw) {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (e < fresh) g[e] = 0.0f;
#pragma unroll
          for (int j = 0; j < kRowsAtOnce; ++j) {
            float f[V];
            widen<kF32>(v[j], f);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[j] = fmaf(g[e], e < fresh ? 0.0f : f[e], sum[j]);
          }
        }
      } else {
        const float g = value_at(a.dout, a.out_f32, t * a.K + p);
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j) {
          if (row[j] < 0) continue;
          if (a.dy) put_value(a.dy, kF32, row[j] * a.K + p, w[j] * g);
          if (a.dw) sum[j] = fmaf(g, value_at(a.y, kF32, row[j] * a.K + p), sum[j]);
        }
        if (a.dy)
          for (int j = max(j0, valid - first); j < min(a.top, j0 + kRowsAtOnce); ++j)
            put_value(a.dy, kF32, (int64_t)(first + j) * a.K + p, 0.0f);
      }
    }
    if (!a.dw) continue;
    // (an infinity or NaN of dout times the zeros of a dropped slot is NaN: its sum is zero all the same)
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j)
      if (row[j] < 0) sum[j] = 0.0f;
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j)
      for (int d = min(span, 64) / 2; d; d >>= 1) sum[j] += __shfl_xor(sum[j], d);
    if constexpr (W == 4) {
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j) part[wave][j] = sum[j];
      }
      __syncthreads();
      if (threadIdx.x < kRowsAtOnce && j0 + (int)threadIdx.x < a.top) {
        const int j = threadIdx.x;
        put_value(a.dw, a.w_f32, first + j0 + j, part[0][j] + part[1][j] + part[2][j] + part[3][j]);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int j = 0; j < kRowsAtOnce; ++j)
        if (mine == 0 && j0 + j < a.top) put_value(a.dw, a.w_f32, first + j0 + j, sum[j]);
    }
  }
}

// Slots per block of the sort: 64 blocks, and 128 from 2048 slots in each on, as every block
// reads the counts of all (us: 8192 slots of 128 experts 7.7 by 256, 8.6 by 512 and 10.6 by 1024; 32760
// 10.3, 9.1 and 10.8; 120000 of 500 21.0 by 2048, 22.3 by 1024; 262136 of 128 24.7 by 4096, 18.0 by 2048).
int sort_chunk(int64_t slots) {
  const int64_t per = (slots + 63) / 64;
  return (int)((per < 1 ? 1 : per <= 2048 ? per : (per + 1) / 2) + 255) / 256 * 256;
}
int sort_blocks(int64_t slots) {
  const int chunk = sort_chunk(slots);
  const int64_t n = (slots + chunk - 1) / chunk;
  return n < 1 ? 1 : (int)n;
}

// Whether a call is one launch: its blocks count every slot once per slot of their own (us, the
// sort alone and with rows of 2560 bf16, in one launch and in several: 16 x 8 slots 3.9 and 5.7, 6.5
// and 8.5; 128 x 8 7.6 and 8.1, 10.5 and 11.3; 2048 x 1 8.1 and 7.5, 11.2 and 11.7; but 256 x 8 12.0
// and 8.5, 15.8 and 11.9).
bool few_slots(int64_t tokens, int64_t top) {
  return tokens * top <= kFewSlots && top <= kMostTop && tokens * top * top <= kFewCounts;
}

// Lanes of a wavefront that share a row of `pieces` pieces, and how many times they need to.
// (us, take, combine and its gradients of 32768 tokens to four rows each, and with a wavefront for
// every row: rows of 32 bf16 4.1, 3.7 and 8.2, and 9.5, 16.6 and 59.8; of 128 8.3, 7.2 and 25.5, and 9.0, 16.9
// and 69.2; of 256 14.5, 14.7 and 45.2, and 12.6, 17.5 and 75.5.)
struct Lanes {
  int lanes, chunks;
};
Lanes lanes_of(int64_t pieces) {
  int lanes = 64;
  while (lanes > 1 && lanes / 2 >= pieces) lanes /= 2;
  return {lanes, (int)((pieces + lanes - 1) / lanes)};
}

// Runs launch(blocks, t0, t1) over tokens t0 .. t1 - 1 in launches of less than 2^31 threads.
template <class Launch>
hipError_t by_tokens(int64_t tokens, Lanes l, Launch launch) {
  const int64_t per = (int64_t)l.lanes * l.chunks, most = (kMaxThreads / 2 - 256) / per;
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t n = tokens - t < most ? tokens - t : most;
    launch((unsigned)((n * per + 255) / 256), (int)t, (int)(t + n));
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

template <typename Id>
hipError_t launch_sort(const Id* ids, int64_t tokens, int64_t top, int64_t experts, int32_t* offsets, int32_t* place,
                       int32_t* order, int* hist, const void* x, int64_t bytes, void* xs, hipStream_t st) {
  const int64_t slots = tokens * top;
  if (few_slots(tokens, top)) {
    expert_dispatch_kernel<Id><<<(unsigned)(tokens ? tokens : 1), 256, 0, st>>>(
        static_cast<const uint8_t*>(x), bytes, ids, (int)tokens, (int)top, (int)experts, offsets, place, order,
        static_cast<uint8_t*>(xs));
    return hipGetLastError();
  }
  const int chunk = sort_chunk(slots), blocks = sort_blocks(slots);
  const size_t lds = (size_t)(experts + 1) * sizeof(int);
  expert_count_kernel<Id><<<blocks, 256, lds, st>>>(ids, (int)slots, chunk, (int)experts, hist);
  if (const hipError_t e = hipGetLastError()) return e;
  expert_place_kernel<Id><<<blocks, 256, 2 * lds, st>>>(ids, (int)slots, chunk, (int)experts, hist, offsets, place, order);
  if (const hipError_t e = hipGetLastError()) return e;
  return bytes ? launch_expert_take(x, tokens, bytes, top, offsets, experts, place, xs, st) : hipSuccess;
}

}  // namespace

size_t expert_sort_workspace(int64_t tokens, int64_t top, int64_t experts) {
  return few_slots(tokens, top) ? 0 : (size_t)sort_blocks(tokens * top) * (size_t)(experts + 1) * sizeof(int);
}

hipError_t launch_expert_dispatch(const void* x, int64_t bytes, const void* ids, bool wide, int64_t tokens, int64_t top,
                                  int64_t experts, int32_t* offsets, int32_t* place, int32_t* order, void* xs,
                                  void* workspace, hipStream_t st) {
  int* hist = static_cast<int*>(workspace);
  return wide ? launch_sort(static_cast<const int64_t*>(ids), tokens, top, experts, offsets, place, order, hist, x, bytes, xs, st)
              : launch_sort(static_cast<const int32_t*>(ids), tokens, top, experts, offsets, place, order, hist, x, bytes, xs, st);
}

hipError_t launch_expert_take(const void* x, int64_t tokens, int64_t bytes, int64_t top, const int32_t* offsets,
                              int64_t experts, const int32_t* place, void* xs, hipStream_t st) {
  const Lanes l = lanes_of(pieces_of(bytes));
  return by_tokens(tokens, l, [&](unsigned blocks, int t0, int t1) {
    auto* from = static_cast<const uint8_t*>(x);
    auto* to = static_cast<uint8_t*>(xs);
    const int slots = (int)(tokens * top);
    auto go = [&](auto kernel) {
      kernel<<<blocks, 256, 0, st>>>(from, bytes, slots, (int)top, offsets + experts, place, to, l.lanes, l.chunks, t0, t1);
    };
    if (l.lanes < 64) go(expert_take_kernel<false, false>);
    else if (whole_lines(xs, bytes)) go(expert_take_kernel<true, true>);
    else go(expert_take_kernel<true, false>);
  });
}

hipError_t launch_expert_combine(const CombineArgs& a, hipStream_t st) {
  const int64_t per = a.y_f32 ? 4 : 8;
  const Lanes l = lanes_of(a.K < per ? 1 : (a.K + per - 1) / per);
  return by_tokens(a.slots / a.top, l, [&](unsigned blocks, int t0, int t1) {
    if (l.lanes == 64) {
      if (a.y_f32) expert_combine_kernel<true, true><<<blocks, 256, 0, st>>>(a, 64, l.chunks, t0, t1);
      else expert_combine_kernel<true, false><<<blocks, 256, 0, st>>>(a, 64, l.chunks, t0, t1);
    } else {
      if (a.y_f32) expert_combine_kernel<false, true><<<blocks, 256, 0, st>>>(a, l.lanes, l.chunks, t0, t1);
      else expert_combine_kernel<false, false><<<blocks, 256, 0, st>>>(a, l.lanes, l.chunks, t0, t1);
    }
  });
}

hipError_t launch_expert_combine_backward(const CombineBackwardArgs& a, hipStream_t st) {
  const int64_t per = a.y_f32 ? 4 : 8, tokens = a.slots / a.top;
  const Lanes l = lanes_of(a.K < per ? a.K : (a.K + per - 1) / per);
  // A block per token while there are few (us by block and by wavefront, 512, 1023, 1500 and 2048 tokens:
  // x 2 rows of 2560 9.3 and 14.2, 12.1 and 15.1, 19.7 and 17.8, 23.0 and 18.9; x 8 rows of 2560 16.6 and 26.1, 24.8 and
  // 30.2, 41.0 and 40.7, 47.7 and 44.7; x 8 rows of 700 9.0 and 12.1, 11.2 and 13.2, 18.1 and 15.5, 20.6 and 16.8; x 1
  // row of 1024 6.3 and 6.9, 8.0 and 8.0, 12.4 and 8.9, 14.7 and 9.2; rows of 5120 gain up to 2048: x 8 40.1 and 54.8,
  // 66.2 and 77.5, 79.3 and 83.4 from 1023 on; 4095 x 8 152 and 140).
  const bool past = a.dy && a.dw ? whole_lines(a.dy, a.K * (a.y_f32 ? 4 : 2)) && whole_lines(a.y, a.K * (a.y_f32 ? 4 : 2))
                                 : whole_lines(a.dy, a.K * (a.y_f32 ? 4 : 2));
  auto go = [&](auto w4, auto w1, auto w0) {
    if (l.lanes < 64) w0<<<(unsigned)((tokens * l.lanes + 255) / 256), 256, 0, st>>>(a, l.lanes);
    else if (l.chunks > 1 && tokens < 1024) w4<<<(unsigned)tokens, 256, 0, st>>>(a, 64);
    else w1<<<(unsigned)((tokens + 3) / 4), 256, 0, st>>>(a, 64);
  };
  if (a.y_f32 && past)
    go(expert_combine_backward_kernel<4, true, true>, expert_combine_backward_kernel<1, true, true>,
       expert_combine_backward_kernel<0, false, true>);
  else if (a.y_f32)
    go(expert_combine_backward_kernel<4, false, true>, expert_combine_backward_kernel<1, false, true>,
       expert_combine_backward_kernel<0, false, true>);
  else if (past)
    go(expert_combine_backward_kernel<4, true, false>, expert_combine_backward_kernel<1, true, false>,
       expert_combine_backward_kernel<0, false, false>);
  else
    go(expert_combine_backward_kernel<4, false, false>, expert_combine_backward_kernel<1, false, false>,
       expert_combine_backward_kernel<0, false, false>);
  return hipGetLastError();
}

}  // namespace w4
