// Microscaled 4-bit floating point (OCP Microscaling Formats, MXFP4): E2M1
// elements, one E8M0 scale (a power of two) per block of 32 inputs, for weights
// and for activations.  The two quantizers and their inverses, the layout
// conversion, and the product
//
//   y[m][n] = sum_k x^[m][k] w^[n][k]
//
// dense or with the rows sorted by expert, in v_mfma_scale_f32_16x16x128_f8f6f4:
// a lane holds one block (32 codes, 16 bytes) of a row of each operand and the
// block's scale, and the unit adds 128 scaled products to an fp32 sum.
//
// Native layout of the weights: for every 256 inputs of a row block of 16 rows two
// tiles of 1 KiB.  Lane L of both holds row L % 16, inputs 64 (L / 16) .. + 63, the
// first block in tile 0 and the second in tile 1.  So a tile is an operand of one
// product (both operands take their inputs in this order), read by a wavefront
// with one coalesced load, and the two scales that a lane needs are consecutive bytes
// of a row of scales, in memory order for the activations too.  The scales of the
// weights are a word for each lane and 512 inputs.
#include "w4_device.h"
#include "w4_launch.h"
#include "w4_rows.h"

namespace w4 {
namespace {

constexpr int kBlock = 32;    // inputs per scale
constexpr int kPair = 256;    // inputs per pair of tiles
constexpr int kWord = 512;    // inputs per word of scales
// The offset of an operand of a step past the last one, added to that of its row (see
// int8.hip): one matrix's codes, and one tile's rows of x, take less than 2 GiB, so the
// sum lies outside the buffer.
constexpr uint32_t kOob = 0x80000000u;
constexpr uint32_t kNanScale = 255;

typedef int i32x8 __attribute__((__vector_size__(8 * sizeof(int))));
typedef float f32x2 __attribute__((__vector_size__(2 * sizeof(float))));

// c + sum over 128 inputs of a b, byte SA (SB) of a lane's word being the scale of its block.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_mx4(const uint4& a, const uint4& b, const f32x4& c, uint32_t sa, uint32_t sb) {
  const i32x8 va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  constexpr int kE2M1 = 4;
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, kE2M1, kE2M1, SA, (int)sa, SB, (int)sb);
}

// ---------------------------------------------------------------------------
// quantizers
// ---------------------------------------------------------------------------
// Eight consecutive values of a lane: 16 bytes of bf16, or 32 of fp32.
template <bool kF32>
struct Eight {
  uint4 c[kF32 ? 2 : 1];
};

template <bool kF32, int AUX>
__device__ __forceinline__ Eight<kF32> load_eight(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  Eight<kF32> v;
  v.c[0] = bload<AUX>(rs, off);
  if constexpr (kF32) v.c[1] = bload<AUX>(rs, off + 16);
  return v;
}

// Exponent field of the largest magnitude of the four lanes' 32 values (255: a NaN or an
// infinity is among them).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <bool kF32>
__device__ __forceinline__ uint32_t block_exponent(const Eight<kF32>& v) {
  uint32_t m;
  if constexpr (kF32) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      m = max(max(max(m, v.c[i].x & 0x7FFFFFFFu), max(v.c[i].y & 0x7FFFFFFFu, v.c[i].z & 0x7FFFFFFFu)), v.c[i].w & 0x7FFFFFFFu);
    m >>= 23;
  } else {
    auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu); };
    const u16x2 p = __builtin_elementwise_max(__builtin_elementwise_max(mag(v.c[0].x), mag(v.c[0].y)),
                                              __builtin_elementwise_max(mag(v.c[0].z), mag(v.c[0].w)));
    m = (uint32_t)max(p[0], p[1]) >> 7;
  }
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // lanes 1, 0, 3, 2 of four
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lanes 2, 3, 0, 1
  return m;
}

// E8M0 byte of a block whose largest magnitude has exponent field `m`: that power of two over
// 4, the largest of E2M1, and at least 2^-127.
__device__ __forceinline__ uint32_t scale_of(uint32_t m) { return m == 255 ? kNanScale : m > 2 ? m - 2 : 0; }

// Codes of eight values against a scale byte.  The conversion divides by the power of two,
// rounds to the nearest code, ties to the even one, and saturates; subnormal values and
// scales included (compared with the definition for every exponent of the scale).
template <bool kF32>
__device__ __forceinline__ uint32_t encode_eight(const Eight<kF32>& v, uint32_t s) {
  const float d = __uint_as_float(s << 23);
  uint32_t o = 0;
  if constexpr (kF32) {
    auto f = [](uint32_t u) { return __uint_as_float(u); };
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f(v.c[0].x), f(v.c[0].y), d, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f(v.c[0].z), f(v.c[0].w), d, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f(v.c[1].x), f(v.c[1].y), d, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f(v.c[1].z), f(v.c[1].w), d, 3);
  } else {
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.c[0].x), d, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.c[0].y), d, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.c[0].z), d, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.c[0].w), d, 3);
  }
  return s == kNanScale ? 0 : o;
}

// Values of eight codes under a scale byte (255 gives NaN, whatever the code).
template <bool kF32>
__device__ __forceinline__ Eight<kF32> decode_eight(uint32_t o, uint32_t s) {
  const float d = __uint_as_float(s << 23);
  Eight<kF32> v;
  if constexpr (kF32) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(o, d, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(o, d, 1);
    const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(o, d, 2), g = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(o, d, 3);
    v.c[0] = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(b[0]), __float_as_uint(b[1]));
    v.c[1] = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(g[0]), __float_as_uint(g[1]));
  } else {
    v.c[0] = make_uint4(bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 0)),
                        bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 1)),
                        bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 2)),
                        bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 3)));
  }
  return v;
}

// Activations: rows, codes and scales are all in memory order, so the matrix is one
// run of blocks whatever its shape.  A wavefront takes 2048 values, four times eight
// per lane, four lanes to a block.
template <bool kF32>
__global__ __launch_bounds__(256) void quantize_tokens_kernel(const uint8_t* __restrict__ x, int64_t values,
                                                              uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  constexpr int kIn = kF32 ? 4 : 2, kSpan = 2048;
  const int lane = threadIdx.x & 63;
  const int64_t at = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kSpan;
  if (at >= values) return;
  const int left = (int)min<int64_t>(values - at, kSpan);  // a multiple of 128
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(x + at * kIn, (uint32_t)left * kIn);
  Eight<kF32> v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) v[u] = load_eight<kF32, kNonTemporal>(rs, (uint32_t)(u * 512 + lane * 8) * kIn);
  uint32_t mine = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t s = scale_of(block_exponent<kF32>(v[u]));
    if ((lane & 3) == u) mine = s;
    if (u * 512 + lane * 8 < left)
      *reinterpret_cast<uint32_t*>(q + (at + u * 512 + lane * 8) / 2) = encode_eight<kF32>(v[u], s);
  }
  // lane 4 b + u has the scale of block b of part u
  const int b = (lane & 3) * 16 + (lane >> 2);
  if (b * kBlock < left) scales[at / kBlock + b] = (uint8_t)mine;
}

template <bool kF32>
__global__ __launch_bounds__(256) void dequantize_tokens_kernel(const uint8_t* __restrict__ q,
                                                                const uint8_t* __restrict__ scales, int64_t values,
                                                                uint8_t* __restrict__ x) {
  constexpr int kOut = kF32 ? 4 : 2, kSpan = 2048;
  const int lane = threadIdx.x & 63;
  const int64_t at = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kSpan;
  if (at >= values) return;
  const int left = (int)min<int64_t>(values - at, kSpan);
  uint32_t o[4], s[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = u * 512 + lane * 8;
    o[u] = i < left ? *reinterpret_cast<const uint32_t*>(q + (at + i) / 2) : 0;
    s[u] = i < left ? scales[(at + i) / kBlock] : 0;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = u * 512 + lane * 8;
    if (i >= left) continue;
    const Eight<kF32> v = decode_eight<kF32>(o[u], s[u]);
    uint4* to = reinterpret_cast<uint4*>(x + (at + i) * kOut);
    to[0] = v.c[0];
    if constexpr (kF32) to[1] = v.c[1];
  }
}

// Where a wavefront that goes through 16 rows x 512 inputs finds what lane l holds in
// load (i, u): row 4 i + l / 16, inputs 128 u + 8 (l % 16) .. + 7, the dword l % 4 of
// the 16 bytes of block 4 u + (l % 16) / 4.
struct NativeAt {
  uint32_t code;   // byte offset in the 4 KiB of codes
  uint32_t scale;  // byte offset in the 256 bytes of scales
};
__device__ __forceinline__ NativeAt native_at(int lane, int i, int u) {
  const int row = 4 * i + (lane >> 4), b = 4 * u + ((lane & 15) >> 2);
  const int half = b >> 3, quarter = (b & 7) >> 1, t = b & 1;
  return {(uint32_t)((2 * half + t) * 1024 + (quarter * 16 + row) * 16 + (lane & 3) * 4),
          (uint32_t)((quarter * 16 + row) * 4 + 2 * half + t)};
}

// Weights: a wavefront takes 16 rows x 512 inputs, reads whole lines of a row and
// writes 64-byte runs of its tiles.  Padding (rows N .., inputs K ..) reads zeros, which
// give codes and scales of zero.
template <bool kF32>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const uint8_t* __restrict__ W, int64_t N, int K, int words,
                                                               int64_t items, uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ scales) {
  constexpr int kIn = kF32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= items) return;
  const int64_t r = item / words;
  const int c = (int)(item - r * words);
  const int rows = (int)min<int64_t>(N - r * kTileRows, kTileRows);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(W + r * kTileRows * K * kIn, (uint32_t)rows * (uint32_t)K * kIn);
  const int pairs = (K + kPair - 1) / kPair;
  uint8_t* qt = q + (r * pairs + 2 * c) * 2048;
  uint8_t* st = scales + (r * words + c) * 256;
  const int left = K - c * kWord;              // inputs of this word's 512 that there are
  const int padded = (pairs - 2 * c) * kPair;  // and with the padding of their codes
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t row = (uint32_t)(4 * i + (lane >> 4));
    Eight<kF32> v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = 128 * u + 8 * (lane & 15);
      v[u] = load_eight<kF32, 0>(rs, k < left ? (row * (uint32_t)K + (uint32_t)(c * kWord + k)) * kIn : kOob);
    }
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t s = scale_of(block_exponent<kF32>(v[u]));
      if ((lane & 3) == u) mine = s;
      if (128 * u + 8 * (lane & 15) < padded)
        *reinterpret_cast<uint32_t*>(qt + native_at(lane, i, u).code) = encode_eight<kF32>(v[u], s);
    }
    st[native_at(lane, i, lane & 3).scale] = (uint8_t)mine;
  }
}

template <bool kF32>
__global__ __launch_bounds__(256) void dequantize_weights_kernel(const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ scales, int64_t N, int K,
                                                                 int words, int64_t items, uint8_t* __restrict__ W) {
  constexpr int kOut = kF32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= items) return;
  const int64_t r = item / words;
  const int c = (int)(item - r * words);
  const int pairs = (K + kPair - 1) / kPair;
  const uint8_t* qt = q + (r * pairs + 2 * c) * 2048;
  const uint8_t* st = scales + (r * words + c) * 256;
  const int left = K - c * kWord;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = r * kTileRows + 4 * i + (lane >> 4);
    uint32_t o[4], s[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const NativeAt at = native_at(lane, i, u);
      const bool there = n < N && 128 * u + 8 * (lane & 15) < left;
      o[u] = there ? *reinterpret_cast<const uint32_t*>(qt + at.code) : 0;
      s[u] = there ? st[at.scale] : 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = 128 * u + 8 * (lane & 15);
      if (n >= N || k >= left) continue;
      const Eight<kF32> v = decode_eight<kF32>(o[u], s[u]);
      uint4* to = reinterpret_cast<uint4*>(W + (n * K + c * kWord + k) * kOut);
      to[0] = v.c[0];
      if constexpr (kF32) to[1] = v.c[1];
    }
  }
}

// Codes [N][K / 2] and scales [N][K / 32] row-major <-> native: a thread has one lane of
// a row block's 512 inputs, up to four blocks and their word of scales.
template <bool kPack>
__global__ __launch_bounds__(256) void repack_mx4_kernel(uint8_t* __restrict__ canon, uint8_t* __restrict__ canon_scales,
                                                         int64_t N, int K, int words, int64_t items,
                                                         uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= items) return;
  const int64_t r = item / words;
  const int c = (int)(item - r * words);
  const int pairs = (K + kPair - 1) / kPair;
  const int64_t n = r * kTileRows + (lane & 15);
  uint32_t word = 0;
  uint32_t* ws = reinterpret_cast<uint32_t*>(scales + (r * words + c) * 256) + lane;
  if constexpr (!kPack) word = *ws;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int k = c * kWord + (b >> 1) * kPair + 64 * (lane >> 4) + (b & 1) * kBlock;
    const bool there = n < N && k < K;
    uint4* qt = reinterpret_cast<uint4*>(q + ((r * pairs + 2 * c + (b >> 1)) * 2 + (b & 1)) * 1024) + lane;
    if constexpr (kPack) {
      if (2 * c + (b >> 1) < pairs)
        *qt = there ? *reinterpret_cast<const uint4*>(canon + (n * K + k) / 2) : make_uint4(0, 0, 0, 0);
      if (there) word |= (uint32_t)canon_scales[(n * K + k) / kBlock] << (8 * b);
    } else if (there) {
      *reinterpret_cast<uint4*>(canon + (n * K + k) / 2) = *qt;
      canon_scales[(n * K + k) / kBlock] = (uint8_t)(word >> (8 * b));
    }
  }
  if constexpr (kPack) *ws = word;
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
struct MxArgs {
  const uint8_t* xq;
  const uint8_t* xs;
  const int* offsets;  // nullptr: dense
  const uint8_t* q;
  const uint8_t* s;
  void* y;
  int M, K, N, experts;
};

template <bool kF32>
__device__ __forceinline__ void store_value(void* y, int64_t i, float v) {
  if constexpr (kF32)
    static_cast<float*>(y)[i] = v;
  else
    static_cast<uint16_t*>(y)[i] = f32_to_bf16_rne(v);
}

// Streaming form: a block owns R row blocks of 16 outputs and one tile of 16 rows of x;
// its NW wavefronts divide K.  Lane l of a wavefront holds row l % 16 of x and of the
// row block, inputs 64 (l / 16) .. + 63 of 256, and D[4 (l / 16) + j][l % 16], j = 0..3,
// all straight from memory.
template <int R, int NW, bool kF32>
__global__ __launch_bounds__(NW * 64) void mx4_stream_kernel(const MxArgs a) {
  const int nb = (a.N + kTileRows - 1) / kTileRows, panels = (nb + R - 1) / R;
  const int t = blockIdx.x / panels, rb0 = (blockIdx.x - t * panels) * R;
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, 16, t, rt)) return;
  __shared__ f32x4 red[NW][R][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, h = lane >> 4;
  const int pairs = (a.K + kPair - 1) / kPair, words = (a.K + kWord - 1) / kWord;
  const int w0 = (int)((int64_t)words * wave / NW), w1 = (int)((int64_t)words * (wave + 1) / NW);
  const uint32_t codes = (uint32_t)nb * (uint32_t)pairs * 2048u, scales = (uint32_t)nb * (uint32_t)words * 256u;
  const int rows = rt.r1 - rt.r0;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.q + (int64_t)rt.expert * codes, codes);
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(a.s + (int64_t)rt.expert * scales, scales);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.xq + (int64_t)rt.r0 * (a.K / 2), (uint32_t)rows * (uint32_t)(a.K / 2));
  const __amdgpu_buffer_rsrc_t rsx =
      make_rsrc(a.xs + (int64_t)rt.r0 * (a.K / kBlock), (uint32_t)rows * (uint32_t)(a.K / kBlock));

  f32x4 acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = f32x4{0, 0, 0, 0};
  for (int c = w0; c < w1; ++c) {
    uint32_t sw[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      sw[r] = __builtin_amdgcn_raw_buffer_load_b32(rsw, (int)(((uint32_t)(rb0 + r) * words + c) * 256u + 4u * lane), 0, 0);
    uint4 x[4], w[R][4];
    uint32_t sx[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int k = c * kWord + p * kPair + 64 * h;  // this lane's first input
      const bool there = k < a.K;
      sx[p] = __builtin_amdgcn_raw_buffer_load_b16(
          rsx, (int)(there ? (uint32_t)(nl * (a.K / kBlock) + k / kBlock) : kOob), 0, 0);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        x[2 * p + b] = bload<0>(rx, there ? (uint32_t)nl * (uint32_t)(a.K / 2) + (uint32_t)(k / 2 + 16 * b) : kOob);
#pragma unroll
        for (int r = 0; r < R; ++r)
          w[r][2 * p + b] = bload<0>(rw, 2 * c + p < pairs ? (((uint32_t)(rb0 + r) * pairs + 2 * c + p) * 128u + 64u * b + lane) * 16u : kOob);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      acc[r] = mfma_mx4<0, 0>(x[0], w[r][0], acc[r], sx[0], sw[r]);
      acc[r] = mfma_mx4<1, 1>(x[1], w[r][1], acc[r], sx[0], sw[r]);
      acc[r] = mfma_mx4<0, 2>(x[2], w[r][2], acc[r], sx[1], sw[r]);
      acc[r] = mfma_mx4<1, 3>(x[3], w[r][3], acc[r], sx[1], sw[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) red[wave][r][lane] = acc[r];
  __syncthreads();
  for (int r = wave; r < R; r += NW) {
    const int n = (rb0 + r) * kTileRows + nl;
    if (n >= a.N) continue;
    f32x4 v = red[0][r][lane];
#pragma unroll
    for (int w_ = 1; w_ < NW; ++w_) v += red[w_][r][lane];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = rt.r0 + 4 * h + j;
      if (m < rt.r1) store_value<kF32>(a.y, (int64_t)m * a.N + n, v[j]);
    }
  }
}

struct MxGrid {
  int BM, BN, threads;
  int64_t panels, blocks;
};

MxGrid mx4_grid(int64_t M, int64_t N, int64_t experts, bool grouped) {
  MxGrid g{16, 32, 128, 0, 0};
  g.panels = (N + g.BN - 1) / g.BN;
  g.blocks = max_row_tiles(M, experts, grouped, g.BM) * g.panels;
  return g;
}

// Wavefronts of one launch of the kernels that give each a piece of work: less than 2^31
// threads.
constexpr int64_t kMostWaves = (kMaxThreads / 2) / 64 - 4;

// Runs launch(first, count) over `items` pieces of work, in pieces of at most `most`.
template <class Launch>
hipError_t in_launches(int64_t items, int64_t most, Launch launch) {
  for (int64_t at = 0; at < items; at += most) {
    launch(at, items - at < most ? items - at : most);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize_mx4(const void* W, bool f32, int64_t N, int64_t K, uint8_t* q, uint8_t* s, hipStream_t st) {
  const int64_t words = (K + kWord - 1) / kWord, pairs = (K + kPair - 1) / kPair, es = f32 ? 4 : 2;
  return in_launches((N + kTileRows - 1) / kTileRows, kMostWaves / words, [&](int64_t r, int64_t n) {
    const uint8_t* from = static_cast<const uint8_t*>(W) + r * kTileRows * K * es;
    const int64_t items = n * words, rows = N - r * kTileRows;
    uint8_t *qt = q + r * pairs * 2048, *sc = s + r * words * 256;
    const unsigned blocks = (unsigned)((items + 3) / 4);
    if (f32) quantize_weights_kernel<true><<<blocks, 256, 0, st>>>(from, rows, (int)K, (int)words, items, qt, sc);
    else quantize_weights_kernel<false><<<blocks, 256, 0, st>>>(from, rows, (int)K, (int)words, items, qt, sc);
  });
}

hipError_t launch_dequantize_mx4(const uint8_t* q, const uint8_t* s, int64_t N, int64_t K, void* W, bool f32,
                                 hipStream_t st) {
  const int64_t words = (K + kWord - 1) / kWord, pairs = (K + kPair - 1) / kPair, es = f32 ? 4 : 2;
  return in_launches((N + kTileRows - 1) / kTileRows, kMostWaves / words, [&](int64_t r, int64_t n) {
    uint8_t* to = static_cast<uint8_t*>(W) + r * kTileRows * K * es;
    const int64_t items = n * words, rows = N - r * kTileRows;
    const uint8_t *qt = q + r * pairs * 2048, *sc = s + r * words * 256;
    const unsigned blocks = (unsigned)((items + 3) / 4);
    if (f32) dequantize_weights_kernel<true><<<blocks, 256, 0, st>>>(qt, sc, rows, (int)K, (int)words, items, to);
    else dequantize_weights_kernel<false><<<blocks, 256, 0, st>>>(qt, sc, rows, (int)K, (int)words, items, to);
  });
}

hipError_t launch_pack_mx4(uint8_t* canon, uint8_t* canon_scales, int64_t N, int64_t K, uint8_t* q, uint8_t* s, bool pack,
                           hipStream_t st) {
  const int64_t words = (K + kWord - 1) / kWord, pairs = (K + kPair - 1) / kPair;
  return in_launches((N + kTileRows - 1) / kTileRows, kMostWaves / words, [&](int64_t r, int64_t n) {
    const int64_t items = n * words, rows = N - r * kTileRows;
    uint8_t *cq = canon + r * kTileRows * K / 2, *cs = canon_scales + r * kTileRows * K / kBlock;
    uint8_t *qt = q + r * pairs * 2048, *sc = s + r * words * 256;
    const unsigned blocks = (unsigned)((items + 3) / 4);
    if (pack) repack_mx4_kernel<true><<<blocks, 256, 0, st>>>(cq, cs, rows, (int)K, (int)words, items, qt, sc);
    else repack_mx4_kernel<false><<<blocks, 256, 0, st>>>(cq, cs, rows, (int)K, (int)words, items, qt, sc);
  });
}

hipError_t launch_quantize_tokens_mx4(const void* x, bool f32, int64_t M, int64_t K, uint8_t* xq, uint8_t* xs,
                                      hipStream_t st) {
  return in_launches((M * K + 2047) / 2048, kMostWaves, [&](int64_t at, int64_t n) {
    const uint8_t* from = static_cast<const uint8_t*>(x) + at * 2048 * (f32 ? 4 : 2);
    const int64_t values = M * K - at * 2048 < n * 2048 ? M * K - at * 2048 : n * 2048;
    uint8_t *q = xq + at * 1024, *s = xs + at * (2048 / kBlock);
    const unsigned blocks = (unsigned)((n + 3) / 4);
    if (f32) quantize_tokens_kernel<true><<<blocks, 256, 0, st>>>(from, values, q, s);
    else quantize_tokens_kernel<false><<<blocks, 256, 0, st>>>(from, values, q, s);
  });
}

hipError_t launch_dequantize_tokens_mx4(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, void* x, bool f32,
                                        hipStream_t st) {
  return in_launches((M * K + 2047) / 2048, kMostWaves, [&](int64_t at, int64_t n) {
    uint8_t* to = static_cast<uint8_t*>(x) + at * 2048 * (f32 ? 4 : 2);
    const int64_t values = M * K - at * 2048 < n * 2048 ? M * K - at * 2048 : n * 2048;
    const uint8_t *q = xq + at * 1024, *s = xs + at * (2048 / kBlock);
    const unsigned blocks = (unsigned)((n + 3) / 4);
    if (f32) dequantize_tokens_kernel<true><<<blocks, 256, 0, st>>>(q, s, values, to);
    else dequantize_tokens_kernel<false><<<blocks, 256, 0, st>>>(q, s, values, to);
  });
}

bool fits_linear_mx4(int64_t M, int64_t N, int64_t experts, bool grouped) {
  const MxGrid g = mx4_grid(M, N, experts, grouped);
  return g.blocks * g.threads < kMaxThreads;
}

hipError_t launch_linear_mx4(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, const int32_t* offsets,
                             int64_t experts, const uint8_t* q, const uint8_t* s, int64_t N, void* y, bool f32,
                             hipStream_t st) {
  const MxArgs a{xq, xs, offsets, q, s, y, (int)M, (int)K, (int)N, (int)experts};
  const MxGrid g = mx4_grid(M, N, experts, offsets != nullptr);
  const unsigned blocks = (unsigned)g.blocks;
  if (f32) mx4_stream_kernel<2, 2, true><<<blocks, 128, 0, st>>>(a);
  else mx4_stream_kernel<2, 2, false><<<blocks, 128, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace w4
