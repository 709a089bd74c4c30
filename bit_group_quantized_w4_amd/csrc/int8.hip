// 8-bit integers with one scale per output channel (weights) and one per token
// (activations): the two quantizers, the layout conversion, and the product
//
//   y[m][n] = sx[m] * d[n] * sum_k xq[m][k] q[n][k],
//
// dense or with the rows sorted by expert.  The sum runs in int32 and is exact
// (K <= 130944 keeps |sum| <= 2^14 K below 2^31), so neither its order nor the
// way K is divided changes a bit of the result; the rounding is that of the sum
// to fp32 and of the two products with the scales.
//
// Native layout of the weights: tiles of 16 rows x 64 inputs, 1 KiB each, row
// blocks outermost, then the tiles along K.  Lane L of a tile holds the 16 codes
// of row L % 16, inputs 16 (L / 16) .. + 15: the B operand of one
// v_mfma_i32_16x16x64_i8, read by a wavefront with one coalesced load.
#include "w4_device.h"
#include "w4_launch.h"
#include "w4_rows.h"

#include <float.h>

namespace w4 {
namespace {

constexpr int kStep = 64;           // inputs per tile
constexpr float kMaxCode8 = 127.0f;  // largest magnitude maps to code +-127
constexpr uint32_t kOob = 0x80000000u;  // buffer offsets from here on read zeros

typedef int i32x4 __attribute__((__vector_size__(4 * sizeof(int))));

__device__ __forceinline__ i32x4 mfma16x16x64(const i32x4& a, const i32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// Code of v against the scale d: round half away of the IEEE quotient.
__device__ __forceinline__ int code_of(float v, float d) {
  const float t = v / d;
  float r = truncf(t);
  r = fabsf(t - r) >= 0.5f ? r + copysignf(1.0f, t) : r;
  return (int)fminf(fmaxf(r, -kMaxCode8), kMaxCode8);
}

// Byte offset of input k of row n in the native layout.
__device__ __forceinline__ int64_t native_at(int64_t n, int64_t k, int64_t K) {
  return ((n >> 4) * (K / kStep) + k / kStep) * 1024 + ((k >> 4) & 3) * 256 + (n & 15) * 16 + (k & 15);
}

// One block per row: the row's largest magnitude, then its codes.
// kNative: rows are a weight's, written as tiles (rows N .. of the last row
// block as zeros); otherwise tokens, written row-major.
template <typename T, bool kNative>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t K,
                                                            int8_t* __restrict__ q, float* __restrict__ scale) {
  const int64_t row = blockIdx.x;
  __shared__ float smax[4];
  __shared__ int sbad[4];
  float amax = 0.0f;
  int bad = 0;
  if (row < rows) {
    for (int64_t k = threadIdx.x; k < K; k += 256) {
      const float a = fabsf(load_f32(x + row * K + k));
      bad |= !(a <= FLT_MAX);
      amax = fmaxf(amax, a);
    }
  }
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    amax = fmaxf(amax, __shfl_xor(amax, s));
    bad |= __shfl_xor(bad, s);
  }
  if ((threadIdx.x & 63) == 0) {
    smax[threadIdx.x >> 6] = amax;
    sbad[threadIdx.x >> 6] = bad;
  }
  __syncthreads();
  amax = fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3]));
  bad = sbad[0] | sbad[1] | sbad[2] | sbad[3];
  const float d = bad ? __uint_as_float(kNanBits) : amax / kMaxCode8;
  const bool usable = !bad && d != 0.0f && row < rows;
  for (int64_t k = threadIdx.x; k < K; k += 256) {
    const int c = usable ? code_of(load_f32(x + row * K + k), d) : 0;
    q[kNative ? native_at(row, k, K) : row * K + k] = (int8_t)c;
  }
  if (threadIdx.x == 0 && row < rows) scale[row] = d;
}

// Canonical [N][K] <-> native tiles, 16 codes per thread.
template <bool kPack>
__global__ __launch_bounds__(256) void repack_kernel(const int8_t* __restrict__ src, int64_t N, int64_t K,
                                                     int64_t chunks, int8_t* __restrict__ dst) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 16-byte chunk of the native layout
  if (i >= chunks) return;
  const int64_t tile = i >> 6, tiles = K / kStep, r = tile / tiles;
  const int lane = (int)(i & 63);
  const int64_t n = r * kTileRows + (lane & 15), k = (tile - r * tiles) * kStep + 16 * (lane >> 4);
  const uint4* canon = reinterpret_cast<const uint4*>((kPack ? src : dst) + n * K + k);
  if constexpr (kPack)
    reinterpret_cast<uint4*>(dst)[i] = n < N ? *canon : make_uint4(0, 0, 0, 0);
  else if (n < N)
    *const_cast<uint4*>(canon) = reinterpret_cast<const uint4*>(src)[i];
}

struct I8Args {
  const int8_t* xq;
  const float* sx;
  const int* offsets;  // nullptr: dense
  const int8_t* q;
  const float* d;
  void* y;
  int M, K, N, experts;
  int wide;  // every row of y starts at a multiple of 16 bytes
};

template <bool kF32>
__device__ __forceinline__ void store_scaled(const I8Args& a, int m, int n, int sum, float sx, float d) {
  const float v = (float)sum * sx * d;
  const int64_t i = (int64_t)m * a.N + n;
  if constexpr (kF32)
    static_cast<float*>(a.y)[i] = v;
  else
    static_cast<uint16_t*>(a.y)[i] = f32_to_bf16_rne(v);
}

// Streaming form: a block owns R row blocks of 16 outputs and one tile of 16 MT
// rows of x; its NW wavefronts divide K.  Lane l of a wavefront holds
// A[l % 16][16 (l / 16) .. + 15] of x, the tile's B operand and
// D[4 (l / 16) + j][l % 16], j = 0..3.
template <int MT, int R, int NW, bool kF32>
__global__ __launch_bounds__(NW * 64) void w8a8_stream_kernel(const I8Args a) {
  const int nb = (a.N + kTileRows - 1) / kTileRows, panels = (nb + R - 1) / R;
  const int t = blockIdx.x / panels, rb0 = (blockIdx.x - t * panels) * R;
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, 16 * MT, t, rt)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, kb = lane >> 4;
  const int steps = a.K / kStep;
  const int s0 = (int)((int64_t)steps * wave / NW), s1 = (int)((int64_t)steps * (wave + 1) / NW);

  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.q + (int64_t)rt.expert * nb * kTileRows * a.K, (uint32_t)nb * kTileRows * (uint32_t)a.K);
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.xq + (int64_t)rt.r0 * a.K, (uint32_t)(rt.r1 - rt.r0) * (uint32_t)a.K);
  uint32_t wo[R], xo[MT];
#pragma unroll
  for (int r = 0; r < R; ++r) wo[r] = rb0 + r < nb ? ((uint32_t)(rb0 + r) * steps * 64u + lane) * 16u : kOob;
#pragma unroll
  for (int i = 0; i < MT; ++i)
    xo[i] = 16 * i + nl < rt.r1 - rt.r0 ? (uint32_t)(16 * i + nl) * (uint32_t)a.K + 16u * kb : kOob;

  i32x4 acc[MT][R];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[i][r] = i32x4{0, 0, 0, 0};
  for (int s = s0; s < s1; ++s) {
    i32x4 w[R], x[MT];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = bitcast<i32x4>(bload<0>(rw, wo[r] + (uint32_t)s * 1024u));
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = bitcast<i32x4>(bload<0>(rx, xo[i] + (uint32_t)s * kStep));
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[i][r] = mfma16x16x64(x[i], w[r], acc[i][r]);
  }

  __shared__ i32x4 red[NW][MT * R][64];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) red[wave][i * R + r][lane] = acc[i][r];
  __syncthreads();
  for (int c = wave; c < MT * R; c += NW) {
    const int i = c / R, r = c - i * R;
    const int n = (rb0 + r) * kTileRows + nl;
    if (n >= a.N) continue;
    i32x4 v = red[0][c][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[w][c][lane];
    const float d = a.d[(int64_t)rt.expert * a.N + n];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = rt.r0 + 16 * i + 4 * kb + j;
      if (m < rt.r1) store_scaled<kF32>(a, m, n, v[j], a.sx[m], d);
    }
  }
}

// Tile form, for many rows: a block of WM x WN wavefronts owns BM = 16 WM TM rows
// of x and BN = 16 WN TN outputs; each wavefront holds TM x TN tiles of 16 x 16
// sums in registers.  A step is 128 inputs: the block's slices of x and of the
// weights go to LDS straight from memory (no registers in between), one step
// ahead of the products, in two halves of LDS.
//
// x is row-major, 128 bytes of a row per step: lane l of a load takes row
// l / 8 of eight, and its 16-byte chunk (l % 8) ^ (l / 8), so that chunk c of row
// r sits at position c ^ (r % 8) of the row's 128 bytes and the sixteen rows of
// an operand are read without bank conflicts.
//
// The weights are the first operand, so a lane holds four consecutive rows of
// the first operand, D[4 (l / 16) + e][l % 16], for one row of x.  Row 4 q + e of
// tile j of a wavefront's four is output 16 q + 4 j + e: a lane ends with sixteen
// consecutive outputs of its row, a wavefront with 64.  A row block's 2 KiB of a
// step are 64 bytes apart from the next one's in LDS, which spreads the four
// row blocks that one operand then touches over the banks.
//
// Rows past the tile's last and row blocks past the matrix's last re-read the
// last one; nothing of them is stored.
constexpr int kRowBlockLds = 2 * 1024 + 64;

template <int WM, int WN, int TM, bool kF32>
__global__ __launch_bounds__(WM* WN * 64, 1) void w8a8_tile_kernel(const I8Args a, int panels) {
  constexpr int TN = 4;  // sixteen consecutive outputs per lane
  constexpr int NW = WM * WN, BM = 16 * WM * TM, BN = 16 * WN * TN;
  constexpr int kHalf = BM * 128 + BN / 16 * kRowBlockLds;  // bytes of one step
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;         // 1 KiB loads per wavefront and step
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN, "loads shared out evenly");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kHalf];

  const int tiles = count_row_tiles(a.offsets, a.experts, a.M, BM);
  if ((int)blockIdx.x >= tiles * panels) return;
  int t, p;
  tile_of_block(blockIdx.x, tiles, panels, t, p);
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, BM, t, rt)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, kb = lane >> 4;
  const int wm = wave / WN, wn = wave - wm * WN;
  const int K = a.K, nb = (a.N + kTileRows - 1) / kTileRows, rb0 = p * (BN / 16);
  const int rows = rt.r1 - rt.r0;

  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.q + (int64_t)rt.expert * nb * kTileRows * K, (uint32_t)nb * kTileRows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.xq + (int64_t)rt.r0 * K, (uint32_t)rows * (uint32_t)K);
  uint32_t xo[LA], wo[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i)
    xo[i] = (uint32_t)min(8 * (wave * LA + i) + (lane >> 3), rows - 1) * (uint32_t)K +
            16u * ((lane & 7) ^ (lane >> 3));
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int c = wave * LB + i;  // half c % 2 of row block c / 2
    wo[i] = (uint32_t)min(rb0 + (c >> 1), nb - 1) * 16u * (uint32_t)K + (c & 1) * 1024u + 16u * lane;
  }
  typedef __attribute__((address_space(3))) void* lds_ptr;
  auto load_step = [&](int s, int half) {
    uint8_t* to = lds + half * kHalf;
#pragma unroll
    for (int i = 0; i < LA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr)(to + (wave * LA + i) * 1024), 16, (int)xo[i], s * 128, 0,
                                               0);
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int c = wave * LB + i;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (lds_ptr)(to + BM * 128 + (c >> 1) * kRowBlockLds + (c & 1) * 1024), 16, (int)wo[i], s * 2048, 0, 0);
    }
  };

  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  const uint32_t xa = (uint32_t)(wm * TM * 16 + nl) * 128u + 16u * (kb ^ (nl & 7));  // chunk kb of the lane's row
  const uint32_t wa = (uint32_t)BM * 128u + (uint32_t)(wn * TN + (nl >> 2)) * kRowBlockLds + 256u * kb + 16u * (nl & 3);
  i32x4 x[2][TM], w[2][TN];
  auto read_step = [&](int half) {
    const uint8_t* at = lds + half * kHalf;
    // this step's slices are in LDS (every wavefront has waited for its own
    // loads), and the other half has been read by all
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < TN; ++j) w[h][j] = *reinterpret_cast<const i32x4*>(at + wa + j * 64 + h * 1024);
#pragma unroll
      for (int i = 0; i < TM; ++i) x[h][i] = *reinterpret_cast<const i32x4*>(at + (xa ^ (64u * h)) + i * 2048);
    }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma16x16x64(w[h][j], x[h][i], acc[i][j]);
  };
  const int steps = K / 128;
  load_step(0, 0);
  for (int s = 0; s + 1 < steps; ++s) {
    read_step(s & 1);
    __builtin_amdgcn_sched_barrier(0);
    load_step(s + 1, (s + 1) & 1);  // after the reads: they would be held up behind it
    __builtin_amdgcn_sched_barrier(0);
    multiply();
  }
  read_step((steps - 1) & 1);
  multiply();

  const int n0 = 16 * rb0 + 64 * wn + 16 * kb;  // this lane's first output
  if (n0 >= a.N) return;
  const int count = min(16, a.N - n0);
  float d[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) d[e] = a.d[(int64_t)rt.expert * a.N + n0 + min(e, count - 1)];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = rt.r0 + 16 * (wm * TM + i) + nl;
    if (m >= rt.r1) continue;
    const float sx = a.sx[m];
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = (float)acc[i][e >> 2][e & 3] * sx * d[e];
    const int64_t at = (int64_t)m * a.N + n0;
    if constexpr (kF32) {
      float* y = static_cast<float*>(a.y) + at;
      if (a.wide && count == 16) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(y + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < count) y[e] = v[e];
      }
    } else {
      uint16_t* y = static_cast<uint16_t*>(a.y) + at;
      if (a.wide && count == 16) {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          u[e] = (uint32_t)f32_to_bf16_rne(v[2 * e]) | (uint32_t)f32_to_bf16_rne(v[2 * e + 1]) << 16;
        *reinterpret_cast<uint4*>(y) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(y + 8) = make_uint4(u[4], u[5], u[6], u[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < count) y[e] = f32_to_bf16_rne(v[e]);
      }
    }
  }
}

}  // namespace

hipError_t launch_quantize_w8(const float* W, int64_t N, int64_t K, int8_t* q, float* d, hipStream_t stream) {
  const unsigned blocks = (unsigned)((N + kTileRows - 1) / kTileRows * kTileRows);
  quantize_rows_kernel<float, true><<<blocks, 256, 0, stream>>>(W, N, K, q, d);
  return hipGetLastError();
}

hipError_t launch_quantize_tokens(const void* x, bool f32, int64_t M, int64_t K, int8_t* xq, float* sx,
                                  hipStream_t stream) {
  if (f32)
    quantize_rows_kernel<float, false><<<(unsigned)M, 256, 0, stream>>>(static_cast<const float*>(x), M, K, xq, sx);
  else
    quantize_rows_kernel<uint16_t, false><<<(unsigned)M, 256, 0, stream>>>(static_cast<const uint16_t*>(x), M, K, xq,
                                                                           sx);
  return hipGetLastError();
}

hipError_t launch_pack_w8(const int8_t* src, int64_t N, int64_t K, int8_t* dst, bool pack, hipStream_t stream) {
  const int64_t chunks = (N + kTileRows - 1) / kTileRows * K;  // 16 rows x K codes / 16
  const unsigned blocks = (unsigned)((chunks + 255) / 256);
  if (pack)
    repack_kernel<true><<<blocks, 256, 0, stream>>>(src, N, K, chunks, dst);
  else
    repack_kernel<false><<<blocks, 256, 0, stream>>>(src, N, K, chunks, dst);
  return hipGetLastError();
}

hipError_t launch_linear_w8a8(const int8_t* xq, const float* sx, int64_t M, int64_t K, const int32_t* offsets,
                              int64_t experts, const int8_t* q, const float* d, int64_t N, void* y, bool f32,
                              hipStream_t stream) {
  const I8Args a{xq, sx, offsets, q, d, y, (int)M, (int)K, (int)N, (int)experts,
                 (reinterpret_cast<uintptr_t>(y) | (uintptr_t)(N * (f32 ? 4 : 2))) % 16 == 0};
  const int64_t nb = (N + kTileRows - 1) / kTileRows;
  if (M > 64 * experts) {
    const int64_t tiles = max_row_tiles(M, experts, offsets != nullptr, 256), panels = (nb + 15) / 16;
    if (tiles * panels > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    if (f32)
      w8a8_tile_kernel<2, 4, 8, true><<<(unsigned)(tiles * panels), 512, 0, stream>>>(a, (int)panels);
    else
      w8a8_tile_kernel<2, 4, 8, false><<<(unsigned)(tiles * panels), 512, 0, stream>>>(a, (int)panels);
    return hipGetLastError();
  }
  const int64_t blocks = max_row_tiles(M, experts, offsets != nullptr, 16) * nb;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  if (f32)
    w8a8_stream_kernel<1, 1, 4, true><<<(unsigned)blocks, 256, 0, stream>>>(a);
  else
    w8a8_stream_kernel<1, 1, 4, false><<<(unsigned)blocks, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace w4
