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
#include "w4_stage.h"

#include <type_traits>

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
// A lane has 16 bytes of consecutive values: eight bf16, so that four lanes share a block,
// or four fp32 and eight lanes.
template <bool kF32>
constexpr int kValues = kF32 ? 4 : 8;
template <bool kF32>
constexpr int kSharers = kBlock / kValues<kF32>;

// Exponent field of the largest magnitude of the block (255: a NaN or an infinity is among
// its values), from the values of its lanes.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <bool kF32>
__device__ __forceinline__ uint32_t block_exponent(const uint4& v) {
  uint32_t m;
  if constexpr (kF32) {
    m = max(max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu), max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu)) >> 23;
  } else {
    auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu); };
    const u16x2 p = __builtin_elementwise_max(__builtin_elementwise_max(mag(v.x), mag(v.y)),
                                              __builtin_elementwise_max(mag(v.z), mag(v.w)));
    m = (uint32_t)max(p[0], p[1]) >> 7;
  }
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // lanes 1, 0, 3, 2 of four
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lanes 2, 3, 0, 1
  if constexpr (kF32) m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));  // eight, mirrored
  return m;
}

// E8M0 byte of a block whose largest magnitude has exponent field `m`: that power of two over
// 4, the largest of E2M1, and at least 2^-127.
__device__ __forceinline__ uint32_t scale_of(uint32_t m) { return m == 255 ? kNanScale : m > 2 ? m - 2 : 0; }

// Codes of a lane's values against a scale byte (fp32: 16 bits).  The conversion divides by
// the power of two, rounds to the nearest code, ties to the even one, and saturates;
// subnormal values and scales included (compared with the definition for every exponent of
// the scale).
template <bool kF32>
__device__ __forceinline__ uint32_t encode(const uint4& v, uint32_t s) {
  const float d = __uint_as_float(s << 23);
  uint32_t o = 0;
  if constexpr (kF32) {
    auto f = [](uint32_t u) { return __uint_as_float(u); };
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f(v.x), f(v.y), d, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f(v.z), f(v.w), d, 1);
  } else {
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.x), d, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.y), d, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.z), d, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, bitcast<bf16x2>(v.w), d, 3);
  }
  return s == kNanScale ? 0 : o;
}

// Values of a lane's codes under a scale byte (255 gives NaN, whatever the code).
template <bool kF32>
__device__ __forceinline__ v4u decode(uint32_t o, uint32_t s) {
  const float d = __uint_as_float(s << 23);
  if constexpr (kF32) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(o, d, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(o, d, 1);
    return v4u{__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(b[0]), __float_as_uint(b[1])};
  } else {
    return v4u{bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 0)),
               bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 1)),
               bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 2)),
               bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, d, 3))};
  }
}

// Activations: rows, codes and scales are all in memory order, so the matrix is one
// run of blocks whatever its shape.  A wavefront takes 2048 values, 1 KiB per load.
//
// Bound by memory: 4099 x 28672 bf16 (298 MB) take 46 us (6.5 TB/s; a copy reaches 5.1), fp32
// 86 us (6.2); back to bf16 43 us.
template <bool kF32>
__global__ __launch_bounds__(256) void quantize_tokens_kernel(const uint8_t* __restrict__ x, int64_t values,
                                                              uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  constexpr int kIn = kF32 ? 4 : 2, V = kValues<kF32>, kSpan = 2048, kLoads = kSpan / 64 / V;
  const int lane = threadIdx.x & 63;
  const int64_t at = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kSpan;
  if (at >= values) return;
  const int left = (int)min<int64_t>(values - at, kSpan);  // a multiple of 128
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(x + at * kIn, (uint32_t)left * kIn);
  uint4 v[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) v[u] = bload<kNonTemporal>(rs, (uint32_t)(u * 64 + lane) * 16u);
  uint32_t mine = 0, o[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const uint32_t s = scale_of(block_exponent<kF32>(v[u]));
    if (lane % kSharers<kF32> == u) mine = s;
    o[u] = encode<kF32>(v[u], s);
  }
  uint32_t* to = reinterpret_cast<uint32_t*>(q + at / 2);
  if constexpr (kF32) {
    // of two loads, an even lane stores its pair's codes of the first, an odd one those of the second
#pragma unroll
    for (int u = 0; u < kLoads; u += 2) {
      const bool odd = lane & 1;
      const uint32_t give = odd ? o[u] : o[u + 1], keep = odd ? o[u + 1] : o[u];
      const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0xB1, 0xF, 0xF, true);  // lanes 1, 0, 3, 2
      const int i = (u + odd) * 32 + lane / 2;
      if (i * 8 < left) to[i] = odd ? got | keep << 16 : keep | got << 16;
    }
  } else {
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if ((u * 64 + lane) * V < left) to[u * 64 + lane] = o[u];
  }
  // lane kSharers b + u has the scale of block b of load u
  const int b = lane % kSharers<kF32> * (64 / kSharers<kF32>) + lane / kSharers<kF32>;
  if (b * kBlock < left) scales[at / kBlock + b] = (uint8_t)mine;
}

template <bool kF32>
__global__ __launch_bounds__(256) void dequantize_tokens_kernel(const uint8_t* __restrict__ q,
                                                                const uint8_t* __restrict__ scales, int64_t values,
                                                                uint8_t* __restrict__ x) {
  constexpr int kOut = kF32 ? 4 : 2, V = kValues<kF32>, kSpan = 2048, kLoads = kSpan / 64 / V;
  const int lane = threadIdx.x & 63;
  const int64_t at = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kSpan;
  if (at >= values) return;
  const int left = (int)min<int64_t>(values - at, kSpan);
  uint32_t o[kLoads], s[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = (u * 64 + lane) * V;
    if constexpr (kF32) o[u] = i < left ? *reinterpret_cast<const uint16_t*>(q + (at + i) / 2) : 0;
    else o[u] = i < left ? *reinterpret_cast<const uint32_t*>(q + (at + i) / 2) : 0;
    s[u] = i < left ? scales[(at + i) / kBlock] : 0;
  }
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = (u * 64 + lane) * V;
    if (i < left) __builtin_nontemporal_store(decode<kF32>(o[u], s[u]), reinterpret_cast<v4u*>(x + (at + i) * kOut));
  }
}

// Weights: a block of four wavefronts takes 16 rows x 512 inputs, each wavefront whole lines
// of four rows; the codes change between the two orders in LDS, 16 runs of 256 bytes (one
// quarter of the lanes in one of the four tiles) 272 bytes apart, which spreads a row's blocks
// over the banks.
struct NativeBlock {
  uint32_t code, scale;  // byte offsets in LDS of block b (0 .. 15) of row `row`
};
constexpr int kRunLds = 256 + 16;
__device__ __forceinline__ NativeBlock native_block(int row, int b) {
  const int half = b >> 3, quarter = (b & 7) >> 1, t = b & 1;
  return {(uint32_t)(((2 * half + t) * 4 + quarter) * kRunLds + row * 16), (uint32_t)((quarter * 16 + row) * 4 + 2 * half + t)};
}

// Padding (rows N .., inputs K ..) reads zeros, which give codes and scales of zero.
//
// Bound by memory: 28672 x 8192 fp32 (1.06 GB) take 172 us (6.2 TB/s), bf16 89 (6.7); back to
// bf16 83 us.  (Codes stored from the lanes that made them, 64 bytes of a tile at a time, and
// loads through the caches: 217 and 132 us; values stored through the caches 140.)
template <bool kF32>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const uint8_t* __restrict__ W, int64_t N, int K, int words,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  constexpr int kIn = kF32 ? 4 : 2, V = kValues<kF32>, kParts = kWord / 64 / V;
  __shared__ __attribute__((aligned(16))) uint8_t codes[16 * kRunLds], scale[256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t item = blockIdx.x, r = item / words;
  const int c = (int)(item - r * words);
  const int rows = (int)min<int64_t>(N - r * kTileRows, kTileRows);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(W + r * kTileRows * K * kIn, (uint32_t)rows * (uint32_t)K * kIn);
  const int left = K - c * kWord;  // inputs of this word's 512 that there are
  uint4 v[4][kParts];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const int k = (p * 64 + lane) * V;
      v[i][p] = bload<kNonTemporal>(rs, k < left ? ((uint32_t)(4 * wave + i) * (uint32_t)K + (uint32_t)(c * kWord + k)) * kIn : kOob);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const NativeBlock at = native_block(4 * wave + i, (p * 64 + lane) / kSharers<kF32>);
      const uint32_t s = scale_of(block_exponent<kF32>(v[i][p])), o = encode<kF32>(v[i][p], s);
      const int part = lane % kSharers<kF32>;
      if constexpr (kF32) *reinterpret_cast<uint16_t*>(codes + at.code + 2 * part) = (uint16_t)o;
      else *reinterpret_cast<uint32_t*>(codes + at.code + 4 * part) = o;
      if (part == 0) scale[at.scale] = (uint8_t)s;
    }
  __syncthreads();
  const int pairs = (K + kPair - 1) / kPair;
  if ((int)(threadIdx.x >> 7) < pairs - 2 * c)  // (two tiles for each 256 inputs)
    reinterpret_cast<uint4*>(q + (r * pairs + 2 * c) * 2048)[threadIdx.x] =
        *reinterpret_cast<const uint4*>(codes + (threadIdx.x >> 4) * kRunLds + (threadIdx.x & 15) * 16);
  if (threadIdx.x < 16)
    reinterpret_cast<uint4*>(scales + (r * words + c) * 256)[threadIdx.x] = reinterpret_cast<const uint4*>(scale)[threadIdx.x];
}

template <bool kF32>
__global__ __launch_bounds__(256) void dequantize_weights_kernel(const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ scales, int64_t N, int K,
                                                                 int words, uint8_t* __restrict__ W) {
  constexpr int kOut = kF32 ? 4 : 2, V = kValues<kF32>, kParts = kWord / 64 / V;
  __shared__ __attribute__((aligned(16))) uint8_t codes[16 * kRunLds], scale[256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t item = blockIdx.x, r = item / words;
  const int c = (int)(item - r * words);
  const int pairs = (K + kPair - 1) / kPair;
  if ((int)(threadIdx.x >> 7) < pairs - 2 * c)
    *reinterpret_cast<uint4*>(codes + (threadIdx.x >> 4) * kRunLds + (threadIdx.x & 15) * 16) =
        reinterpret_cast<const uint4*>(q + (r * pairs + 2 * c) * 2048)[threadIdx.x];
  if (threadIdx.x < 16)
    reinterpret_cast<uint4*>(scale)[threadIdx.x] = reinterpret_cast<const uint4*>(scales + (r * words + c) * 256)[threadIdx.x];
  __syncthreads();
  const int left = K - c * kWord;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = r * kTileRows + 4 * wave + i;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const int k = (p * 64 + lane) * V, part = lane % kSharers<kF32>;
      if (n >= N || k >= left) continue;
      const NativeBlock at = native_block(4 * wave + i, (p * 64 + lane) / kSharers<kF32>);
      uint32_t o;
      if constexpr (kF32) o = *reinterpret_cast<const uint16_t*>(codes + at.code + 2 * part);
      else o = *reinterpret_cast<const uint32_t*>(codes + at.code + 4 * part);
      __builtin_nontemporal_store(decode<kF32>(o, scale[at.scale]), reinterpret_cast<v4u*>(W + (n * K + c * kWord + k) * kOut));
    }
  }
}

// Codes [N][K / 2] and scales [N][K / 32] row-major <-> native: a thread has one lane of
// a row block's 512 inputs, up to four blocks and their word of scales.
//
// Bound by its requests, 16 bytes of 16 rows per load and a byte of scales per lane: 28672 x 8192 (250 MB)
// takes 59 us packed and 65 unpacked (4.2 and 3.8 TB/s), 9216 x 2560 8.1 and 7.8.
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
  bool lines;  // rows of y are whole lines of memory
};

template <bool kF32>
__device__ __forceinline__ void store_value(void* y, int64_t i, float v) {
  if constexpr (kF32)
    static_cast<float*>(y)[i] = v;
  else
    static_cast<uint16_t*>(y)[i] = f32_to_bf16_rne(v);
}

// What a block needs to find its operands: buffers of the expert's weights and scales, of
// the tile's rows of x and their scales, and the sizes they are addressed with.
struct Operands {
  __amdgpu_buffer_rsrc_t w, ws, x, xs;
  int pairs, words, blocks;  // per row: of 256 inputs, of 512, of 32
};

__device__ __forceinline__ Operands operands_of(const MxArgs& a, const RowTile& rt) {
  Operands o;
  o.pairs = (a.K + kPair - 1) / kPair;
  o.words = (a.K + kWord - 1) / kWord;
  o.blocks = a.K / kBlock;
  const uint32_t nb = (uint32_t)(a.N + kTileRows - 1) / kTileRows, rows = (uint32_t)(rt.r1 - rt.r0);
  const uint32_t codes = nb * (uint32_t)o.pairs * 2048u, scales = nb * (uint32_t)o.words * 256u;
  o.w = make_rsrc(a.q + (int64_t)rt.expert * codes, codes);
  o.ws = make_rsrc(a.s + (int64_t)rt.expert * scales, scales);
  o.x = make_rsrc(a.xq + (int64_t)rt.r0 * (a.K / 2), rows * (uint32_t)(a.K / 2));
  o.xs = make_rsrc(a.xs + (int64_t)rt.r0 * o.blocks, rows * (uint32_t)o.blocks);
  return o;
}

// Streaming form, for few rows: a block owns R row blocks of 16 outputs and one tile of 16
// rows of x; its NW wavefronts divide K.  Lane l of a wavefront holds row l % 16 of x and of
// a row block, inputs 64 (l / 16) .. + 63 of 256, and D[4 (l / 16) + j][l % 16], j = 0..3,
// all straight from memory, D pairs of tiles ahead of the products.
//
// Bound by the weight stream: 13 rows of 28672 x 8192 (125 MB) take 22.3 us (5.6 TB/s); one row of
// 9216 x 2560 4.8 us, the latency of its loads and of the join over K.  (Three or four pairs ahead
// leave fewer wavefronts room: 23.2 and 23.5 us.)
template <int R, int NW, int kCache, bool kF32>
__device__ __forceinline__ void stream_row_tile(const MxArgs& a, const RowTile& rt, int rb0, f32x4 (&red)[NW][R][64]) {
  constexpr int D = 2;
  const Operands o = operands_of(a, rt);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, h = lane >> 4;
  const int s0 = (int)((int64_t)o.pairs * wave / NW), s1 = (int)((int64_t)o.pairs * (wave + 1) / NW);
  uint32_t wo[R], wso[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    wo[r] = (uint32_t)(rb0 + r) * (uint32_t)o.pairs * 2048u + 16u * lane;
    wso[r] = (uint32_t)(rb0 + r) * (uint32_t)o.words * 256u + 4u * lane;
  }
  const uint32_t xo = (uint32_t)nl * (uint32_t)(a.K / 2) + 32u * h, xso = (uint32_t)nl * (uint32_t)o.blocks + 2u * h;

  f32x4 acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = f32x4{0, 0, 0, 0};
  // a ring of D pairs' operands; a pair past the wavefront's last, and inputs past K, read zeros
  // (see kOob), so that every load is unconditional
  uint4 w[D][R][2], x[D][2];
  uint32_t sw[D][R], sx[D];
  auto issue = [&](int c, int s) {
    const uint32_t ow = s < s1 ? (uint32_t)s * 2048u : kOob, ows = s < s1 ? (uint32_t)(s >> 1) * 256u + 2u * (s & 1) : kOob;
    const bool there = s < s1 && 8 * s + 2 * h < o.blocks;
    const uint32_t ox = there ? (uint32_t)s * 128u : kOob, oxs = there ? (uint32_t)s * 8u : kOob;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[c][r][0] = bload<kCache>(o.w, wo[r] + ow);
      w[c][r][1] = bload<kCache>(o.w, wo[r] + ow + 1024u);
      sw[c][r] = __builtin_amdgcn_raw_buffer_load_b16(o.ws, (int)(wso[r] + ows), 0, 0);
    }
    x[c][0] = bload<0>(o.x, xo + ox);
    x[c][1] = bload<0>(o.x, xo + ox + 16u);
    sx[c] = __builtin_amdgcn_raw_buffer_load_b16(o.xs, (int)(xso + oxs), 0, 0);
  };
#pragma unroll
  for (int c = 0; c < D; ++c) {
    issue(c, s0 + c);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int s = s0; s < s1; s += D) {
#pragma unroll
    for (int c = 0; c < D; ++c) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[r] = mfma_mx4<0, 0>(x[c][0], w[c][r][0], acc[r], sx[c], sw[c][r]);
        acc[r] = mfma_mx4<1, 1>(x[c][1], w[c][r][1], acc[r], sx[c], sw[c][r]);
      }
      issue(c, s + c + D);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  auto store = [&](int r, const f32x4& v) {
    const int n = (rb0 + r) * kTileRows + nl;
    if (n >= a.N) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = rt.r0 + 4 * h + j;
      if (m < rt.r1) store_value<kF32>(a.y, (int64_t)m * a.N + n, v[j]);
    }
  };
  if constexpr (NW == 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) store(r, acc[r]);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) red[wave][r][lane] = acc[r];
    __syncthreads();
    for (int r = wave; r < R; r += NW) {
      f32x4 v = red[0][r][lane];
#pragma unroll
      for (int i = 1; i < NW; ++i) v += red[i][r][lane];
      store(r, v);
    }
  }
}

// kPast: an expert's weights are read past the caches, unless another row tile of the
// expert reads them too (13 rows of 28672 x 8192 22.3 us past them, 23.7 through them).
template <int R, int NW, bool kPast, bool kF32>
__global__ __launch_bounds__(NW * 64) void mx4_stream_kernel(const MxArgs a) {
  const int nb = (a.N + kTileRows - 1) / kTileRows, panels = (nb + R - 1) / R;
  const int t = blockIdx.x / panels, rb0 = (blockIdx.x - t * panels) * R;
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, 16, t, rt)) return;
  __shared__ f32x4 red[NW][R][64];
  if (kPast && rt.alone) stream_row_tile<R, NW, kNonTemporal, kF32>(a, rt, rb0, red);
  else stream_row_tile<R, NW, 0, kF32>(a, rt, rb0, red);
}

// Sums of TM row tiles of a wavefront, lane l's outputs n0 + 16 (l / 16) .. + 15 of rows
// m0 + l % 16 + 16 i, stored by way of `stage` (kStageBytes of the wavefront's own).  Past the
// caches where that writes whole lines, which leaves the L2 to x and the weights (us through
// the caches and past them: 8190 rows of 9216 x 2560 123 and 110, 4096 of 17408 x 5120 194 and 187; but 4096 of
// 9217 x 2560, whose rows end inside a line, 70 and 86).
template <int TM, bool kF32>
__device__ __forceinline__ void store_tile(const MxArgs& a, const RowTile& rt, int m0, int n0, const f32x4 (&acc)[TM][4],
                                           uint8_t* stage) {
  uint32_t* words = reinterpret_cast<uint32_t*>(stage);
  const int lane = threadIdx.x & 63;
  auto value = [](uint32_t w, int, int) { return __uint_as_float(w); };
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4*>(words + (lane & 15) * kStagePitch + 16 * (lane >> 4) + 4 * j) = acc[i][j];
    if (a.lines) store_stage<kF32, true>(words, a.y, a.N, m0 + 16 * i, rt.r1, n0, value);
    else store_stage<kF32>(words, a.y, a.N, m0 + 16 * i, rt.r1, n0, value);
  }
}

// Tile forms, for more rows: a block of WM x WN wavefronts owns BM = 16 WM TM rows of x and
// BN = 64 WN outputs; each wavefront holds TM x 4 tiles of 16 x 16 sums in registers.
// A step is 256 inputs: the block's slices of x and of the weights, and every other step the
// scales of two, go to LDS straight from memory (no registers in between).
//
// x is row-major, 128 bytes of a row per step: eight chunks of 16 bytes, one block each.
// Block 2 q + t is what lane quarter q multiplies in product t of the step.  It sits at
// position (q + 4 t) ^ (r % 8) of row r, so that the sixteen rows of an operand are
// read without bank conflicts.
//
// The weights are the first operand, so a lane holds four consecutive rows of it,
// D[4 (l / 16) + e][l % 16], for one row of x.  Row 4 q + e of tile j of a wavefront's four is
// output 16 q + 4 j + e: a lane ends with sixteen consecutive outputs of its row.  A row
// block's 2 KiB of a step are 64 bytes apart from the next one's in LDS, which spreads
// the four row blocks that one operand touches over the banks.
//
// Scales: 16 bytes of a row of x are its blocks' in two steps; the 1 KiB of four row
// blocks is put in the order in which the operands of tile j read it.  A lane of a row of x
// takes its bytes from two words of the four; where a pair of steps reaches past K, the
// bytes of blocks that are not there (the next row's: they could be NaN) become zeros.
//
// Rows past the tile's last, row blocks past the matrix's last and inputs past K lie
// outside their buffers: such loads give zeros (see kOob).  Buffers check each word of a
// load by itself.
constexpr int kRowBlockLds = 2 * 1024 + 64;

template <int WM, int WN, int TM>
struct TileShape {
  static constexpr int TN = 4, NW = WM * WN, BM = 16 * WM * TM, BN = 16 * WN * TN;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;    // 1 KiB loads per wavefront and step: x, weights
  static constexpr int SA = (BM + 63) / 64, SB = BN / 64;      // 1 KiB loads of scales per two steps
  static constexpr int kSl = (SA + SB + NW - 1) / NW;          // of them per wavefront (some come twice)
  static constexpr int kX = BM * 128, kBuffer = kX + BN / 16 * kRowBlockLds, kScales = (SA + SB) * 1024;
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN && LB % 2 == 0, "loads shared out evenly");
};

// Loads and operand reads of a wavefront of a tile (see above).
template <int WM, int WN, int TM>
struct TileWave : TileShape<WM, WN, TM> {
  using S = TileShape<WM, WN, TM>;
  Operands o;
  int lane, wave, wm, wn, xblock;
  uint32_t xo, wo, k_half;              // offsets of the loads
  uint32_t xa, wa, xsa, wsa;            // and of the reads in LDS
  uint32_t xsel, xsel_tail;             // bytes of a row's two words that are the lane's scales
  typedef __attribute__((address_space(3))) void* lds_ptr;

  __device__ __forceinline__ TileWave(const MxArgs& a, const RowTile& rt, int rb0) : o(operands_of(a, rt)) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave - wm * WN;
    k_half = (uint32_t)(a.K / 2);
    rb = rb0;
    const int nl = lane & 15, kb = lane >> 4, pos = (lane & 7) ^ (lane >> 3);
    xblock = 2 * (pos & 3) + (pos >> 2);
    xo = (uint32_t)(8 * wave * S::LA + (lane >> 3)) * k_half + 16u * xblock;
    wo = (uint32_t)(rb0 + wave * S::LB / 2) * (uint32_t)o.pairs * 2048u + 16u * lane;
    xa = (uint32_t)(wm * TM * 16 + nl) * 128u + 16u * (kb ^ (nl & 7));
    wa = (uint32_t)S::kX + (uint32_t)(wn * S::TN + (nl >> 2)) * kRowBlockLds + 256u * kb + 16u * (nl & 3);
    xsa = (uint32_t)(wm * TM * 16 + nl) * 16u + 4u * (kb >> 1);
    wsa = (uint32_t)(S::SA + wn) * 1024u + 16u * (4 * (nl >> 2) + kb) + 4u * (nl & 3);
    const int rest = o.blocks & 15;
    xsel = kb & 1 ? 0x07060302u : 0x05040100u;
    xsel_tail = (2 * kb < rest ? xsel & 0xFFFFu : 0x0C0Cu) | (8 + 2 * kb < rest ? xsel & 0xFFFF0000u : 0x0C0C0000u);
  }
  // Load i of LA + LB of this wavefront's for step s (zeros past the last step).
  __device__ __forceinline__ void load(int i, int s, uint8_t* to) const {
    if (i < S::LA) {
      const uint32_t k = 8 * s + xblock < o.blocks ? (uint32_t)s * 128u : kOob;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(o.x, (lds_ptr)(to + (wave * S::LA + i) * 1024), 16,
                                               (int)(xo + (uint32_t)(8 * i) * k_half + k), 0, 0, 0);
    } else {
      const uint32_t k = s < o.pairs ? (uint32_t)s * 2048u : kOob;
      const int r = (i - S::LA) >> 1, t = (i - S::LA) & 1;  // row block, tile
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          o.w, (lds_ptr)(to + S::kX + (wave * S::LB / 2 + r) * kRowBlockLds + t * 1024), 16,
          (int)(wo + (uint32_t)(r * o.pairs) * 2048u + 1024u * t + k), 0, 0, 0);
    }
  }
  // The scales of steps s and s + 1 (s even).
  __device__ __forceinline__ void load_scales(int s, uint8_t* to) const {
#pragma unroll
    for (int i = 0; i < S::kSl; ++i) {
      const int u = (wave * S::kSl + i) % (S::SA + S::SB);
      const bool of_x = u < S::SA;
      const __amdgpu_buffer_rsrc_t rs = of_x ? o.xs : o.ws;
      const uint32_t so = of_x ? (uint32_t)(64 * u + lane) * (uint32_t)o.blocks
                               : (uint32_t)(rb + 4 * (u - S::SA) + ((lane >> 2) & 3)) * (uint32_t)o.words * 256u +
                                     16u * (4 * (lane & 3) + (lane >> 4));
      const uint32_t k = s < o.pairs ? (uint32_t)s << (of_x ? 3 : 7) : kOob;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(to + u * 1024), 16, (int)(so + k), 0, 0, 0);
    }
  }
  __device__ __forceinline__ uint4 read_w(int t, int j, const uint8_t* from) const {
    return *reinterpret_cast<const uint4*>(from + wa + j * 64 + t * 1024);
  }
  __device__ __forceinline__ uint4 read_x(int t, int i, const uint8_t* from) const {
    return *reinterpret_cast<const uint4*>(from + (xa ^ (64u * t)) + i * 2048);
  }
  __device__ __forceinline__ uint32_t read_ws(int j, const uint8_t* from) const {
    return *reinterpret_cast<const uint32_t*>(from + wsa + j * 256);
  }
  __device__ __forceinline__ void read_xs(int i, const uint8_t* from, uint32_t (&to)[2]) const {
    const uint32_t* at = reinterpret_cast<const uint32_t*>(from + xsa + i * 256);
    to[0] = at[0];
    to[1] = at[2];
  }
  // The lane's four scales of a row of x for steps s and s + 1, of what read_xs read.
  __device__ __forceinline__ uint32_t take_xs(int s, const uint32_t (&v)[2]) const {
    return __builtin_amdgcn_perm(v[1], v[0], 8 * s + 16 > o.blocks ? xsel_tail : xsel);
  }
  int rb;
};

typedef std::integral_constant<int, 0> Zero;
typedef std::integral_constant<int, 1> One;

__device__ __forceinline__ void operands_ready() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
}

// Every read of LDS that this wavefront has issued is done, and so are its loads into LDS but
// for the last `left`; and so are the other wavefronts'.
template <int kLeft>
__device__ __forceinline__ void all_done() {
  static_assert(kLeft < 64, "vmcnt");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (kLeft & 15) | (kLeft >> 4) << 14);  // vmcnt(kLeft) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Many rows: two buffers, loads one step ahead.  4096 rows of 17408 x 5120 take 172 to 188 us, 3.9 to
// 4.2 PFLOP/s (a large library product of this format reaches 3.0 on the same card; the matrix
// units alone, on random codes, 7.0).  The products of a step run in four parts
// (half of the rows times one of the two products).  Operands are read from LDS one
// part ahead, beside the products of the part before.  The next step's loads are issued one by one in
// the first two parts, as one load holds up the wavefront while the address unit of
// the CU takes it (all beside the first part 237 us, beside two 224), each behind a product,
// which runs meanwhile (8190 rows of 9216 x 2560 110.3 us ahead of the products, 108.7 behind).  kAhead: a
// share of the lines that the step after next needs is touched
// early, so that its loads find them in the L2 of the XCD: share `share_x` of eight of
// the rows and `share_w` of four of the row blocks (-1: all of them), as the blocks that run at
// one time on an XCD hold four row tiles or more times up to eight panels (band_tile): 224 and
// 205 us.  What is left above the matrix units' own time: the loads (without them 171 us where it took
// 237), reads of scales (8 us) and the last, partial round.  (Four wavefronts of 128 x 128
// with their sums in the accumulation registers read a third less from LDS, but one wavefront
// per SIMD hides nothing: 306 us.)
template <int WM, int WN, int TM, bool kAhead, bool kF32, int L0, int L1, int LS>
__device__ __forceinline__ void run_tile(const MxArgs& a, const RowTile& rt, int rb0, int share_x, int share_w,
                                         uint8_t (&lds0)[L0], uint8_t (&lds1)[L1], uint8_t (&scales)[LS],
                                         uint8_t* touched) {
  using S = TileShape<WM, WN, TM>;
  constexpr int TN = S::TN, TH = TM / 2, NW = S::NW;
  static_assert(TH * 2 == TM && (S::LA + S::LB) % 2 == 0 && S::kSl == 1, "parts");
  static_assert(S::kBuffer <= L0 && S::kBuffer <= L1 && S::kScales <= LS, "buffers");
  const TileWave<WM, WN, TM> tw(a, rt, rb0);
  const int steps = tw.o.pairs;
  const bool touch_x = tw.wave < NW / 2;
  const __amdgpu_buffer_rsrc_t touch_rs = touch_x ? tw.o.x : tw.o.w;
  const uint32_t touch_at =
      touch_x ? (tw.lane < S::BM / 4 / NW ? (uint32_t)(S::BM / 8 * share_x + S::BM / 4 / NW * tw.wave + tw.lane) * tw.k_half : kOob)
      : share_w < 0 ? (uint32_t)(rb0 + S::BN / 64 * (tw.wave - NW / 2) + (tw.lane >> 4)) * (uint32_t)steps * 2048u +
                          128u * (tw.lane & 15)
                    : (tw.lane < 16 ? (uint32_t)(rb0 + S::BN / 64 * share_w + tw.wave - NW / 2) * (uint32_t)steps * 2048u +
                                          128u * tw.lane
                                    : kOob);
  auto touch = [&](int s) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(touch_rs, (typename TileWave<WM, WN, TM>::lds_ptr)(touched + tw.wave * 256), 4,
                                             (int)(touch_at + ((uint32_t)min(s, steps - 1) << (touch_x ? 7 : 11))), 0, 0, 0);
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  uint4 x[2][TH], w[2][TN];  // x by row half, w by product
  uint32_t sx[2][TH], sx_read[TH][2], sw[TN], sw_read[TN];
  // the products t of row half c of a step of parity P; beside(i) comes before row tile i's, after(i)
  // behind the first of them
  auto multiply = [&](auto parity, auto product, int c, auto beside, auto after) {
    constexpr int t = decltype(product)::value, kByte = 2 * decltype(parity)::value + t;
#pragma unroll
    for (int i = 0; i < TH; ++i) {
      beside(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        acc[c * TH + i][j] = mfma_mx4<kByte, kByte>(w[t][j], x[c][i], acc[c * TH + i][j], sw[j], sx[c][i]);
        if (j == 0) {
          __builtin_amdgcn_sched_barrier(0);
          after(i);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // A step of parity P whose slices are in `cur`, with the last part of the step before; its
  // own last part is left to the next.
  auto step = [&](auto parity, auto other, int s, uint8_t* cur, uint8_t* nxt) {
    constexpr bool even = decltype(parity)::value == 0;
    constexpr int kReads = TN + TH, kHalf = (S::LA + S::LB) / 2;
    auto read = [&](int t, int i) {  // share i of TH of product t's operands
#pragma unroll
      for (int r = (i * kReads + TH - 1) / TH; r < ((i + 1) * kReads + TH - 1) / TH; ++r) {
        if (r < TN) w[t][r] = tw.read_w(t, r, cur);
        else x[0][r - TN] = tw.read_x(t, r - TN, cur);
      }
    };
    auto load = [&](int half, int i) {
#pragma unroll
      for (int l = half * kHalf + i * kHalf / TH; l < half * kHalf + (i + 1) * kHalf / TH; ++l) tw.load(l, s + 1, nxt);
    };
    all_done<kAhead ? 1 : 0>();  // `cur` is filled, and nothing reads `nxt` any more
    multiply(other, One(), 1, [&](int i) {
      read(0, i);
      if constexpr (even) {
        tw.read_xs(i, scales, sx_read[i]);
#pragma unroll
        for (int j = i * TN / TH; j < (i + 1) * TN / TH; ++j) sw_read[j] = tw.read_ws(j, scales);
      }
    }, [&](int i) {
      load(0, i);
      if (!even && i == 0) tw.load_scales(s + 1, scales);
    });
    operands_ready();
    if constexpr (even) {
#pragma unroll
      for (int i = 0; i < TH; ++i) sx[0][i] = tw.take_xs(s, sx_read[i]);
#pragma unroll
      for (int j = 0; j < TN; ++j) sw[j] = sw_read[j];
    }
    multiply(parity, Zero(), 0, [&](int i) {
      x[1][i] = tw.read_x(0, TH + i, cur);
      if constexpr (even) tw.read_xs(TH + i, scales, sx_read[i]);
    }, [&](int i) { load(1, i); });
    operands_ready();
    if constexpr (even) {
#pragma unroll
      for (int i = 0; i < TH; ++i) sx[1][i] = tw.take_xs(s, sx_read[i]);
    }
    multiply(parity, Zero(), 1, [&](int i) {
      read(1, i);
    }, [&](int i) {
      if (kAhead && i == 0) touch(s + 2);  // the last of the step: what all_done leaves in flight
    });
    operands_ready();
    multiply(parity, One(), 0, [&](int i) { x[1][i] = tw.read_x(1, TH + i, cur); }, [](int) {});
  };

#pragma unroll
  for (int i = 0; i < S::LA + S::LB; ++i) tw.load(i, 0, lds0);
  tw.load_scales(0, scales);
  if constexpr (kAhead) touch(1);
#pragma unroll
  for (int j = 0; j < TN; ++j) {  // no step before the first
    w[1][j] = make_uint4(0, 0, 0, 0);
    sw[j] = 0;
  }
#pragma unroll
  for (int i = 0; i < TH; ++i) {
    x[1][i] = make_uint4(0, 0, 0, 0);
    sx[1][i] = 0;
  }
  for (int s = 0; s < steps; s += 2) {  // an odd last step is followed by one of zeros
    step(Zero(), One(), s, lds0, lds1);
    step(One(), Zero(), s + 1, lds1, lds0);
  }
  multiply(One(), One(), 1, [](int) {}, [](int) {});
  all_done<0>();  // no load into LDS is left, and nothing reads what the stages overwrite
  static_assert(NW * kStageBytes <= L0, "stages fit a buffer");
  store_tile<TM, kF32>(a, rt, rt.r0 + 16 * tw.wm * TM, 16 * rb0 + 64 * tw.wn, acc, lds0 + tw.wave * kStageBytes);
}

// 256 x 256 per block of eight wavefronts, one block per CU.  What is left of the tiles
// after whole rounds of kCus, if at most a quarter of a round, is cut into four tiles of 128 x
// 128 each, which fill another round in less than half the time of whole tiles (us whole and
// cut: 2048 rows of 9216 x 2560 44 and 34, 4096 of 17408 x 5120 206 and 195); a tile of at most 128 rows (an
// expert's last) is half as high.  (Blocks that go from tile to tile, the next one's first loads
// issued before the outputs are stored, took 1 to 4% longer.)
constexpr int kCus = 256, kMostCut = kCus / 4;

template <bool kF32>
__global__ __launch_bounds__(512, 1) void mx4_tile_kernel(const MxArgs a, int panels) {
  using Whole = TileShape<2, 4, 8>;
  // variables of their own, each named outright where it is used: the compiler then knows
  // that loads into one are no reason to wait before reading another
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[Whole::kBuffer], lds1[Whole::kBuffer], scales[Whole::kScales];
  __shared__ uint8_t touched[Whole::NW * 256];
  const int tiles = count_row_tiles(a.offsets, a.experts, a.M, 256);
  // (offsets whose ranges overlap could make more tiles than the launch covers)
  const int total = min(tiles, ((int)gridDim.x - 3 * kMostCut) / panels) * panels;
  const int cut = total % kCus <= kMostCut ? total % kCus : 0;
  int b = blockIdx.x, quarter = -1;
  if (b >= total - cut) {
    const int i = b - (total - cut);
    quarter = i & 3;
    b = total - cut + (i >> 2);
    if (b >= total) return;
  }
  BandTile bt;
  if (!band_tile(a.offsets, a.experts, a.M, 256, panels, slot_of_block(b, total), bt)) return;
  RowTile rt = bt.rt;
  const int p = bt.p, share_w = bt.height < 4 ? -1 : bt.in & 3;
  if (quarter >= 0) {
    const int rb0 = 16 * p + 8 * (quarter & 1);
    rt.r0 += 128 * (quarter >> 1);
    rt.r1 = min(rt.r1, rt.r0 + 128);
    if (rt.r0 < rt.r1 && rb0 * kTileRows < a.N) run_tile<4, 2, 2, false, kF32>(a, rt, rb0, 0, 0, lds0, lds1, scales, touched);
  } else if (rt.r1 - rt.r0 <= 128) {
    run_tile<2, 4, 4, true, kF32>(a, rt, 16 * p, p & 7, share_w, lds0, lds1, scales, touched);
  } else {
    run_tile<2, 4, 8, true, kF32>(a, rt, 16 * p, p & 7, share_w, lds0, lds1, scales, touched);
  }
}

// Fewer rows: smaller tiles, four buffers, loads three steps ahead, two parts (one product each)
// per step; a load is issued behind a product, which runs meanwhile (64 rows of 2561 x 9216 9.4 us ahead
// of the products, 8.9 behind).  333 rows of 2561 x 9216 take 12.0 us as 64 x 64 (36.7 streamed, 14.8 as 64 x
// 128, 19.8 as 128 x 128 of this form, 32 as 256 x 256).  (Eight matrices in turn; forty, whose codes come from
// memory: 12.6 us for the 64 rows, 13.8 for the 333.)
//
// Bound by the rate at which a CU loads into LDS, 18 KB of a step in 0.2 us: on the card where 333 rows take
// 11.2 us, the loads alone, without products and reads of LDS, take 11.0; the rest alone 8.1, an empty loop
// 4.0; 41 blocks (64 rows) take no less than 246.  Six or eight buffers change nothing (11.5 and 12.8, with the steps past the
// last); two 20 us.  (Two wavefronts for each tile twice as high, one product of a step each, read
// 24 KB of LDS instead of 40, and take 11.9 with the join; groups of wavefronts that divide the steps 13;
// operands straight to registers, K divided among the wavefronts, 20.)
template <int WM, int WN, int TM, bool kF32>
__global__ __launch_bounds__(WM* WN * 64) void mx4_deep_kernel(const MxArgs a, int panels) {
  using S = TileShape<WM, WN, TM>;
  constexpr int TN = S::TN;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[S::kBuffer], lds1[S::kBuffer], lds2[S::kBuffer], lds3[S::kBuffer],
      scales0[S::kScales], scales2[S::kScales];
  // (offsets whose ranges overlap could make more tiles than the launch covers)
  const int total = min(count_row_tiles(a.offsets, a.experts, a.M, S::BM), (int)gridDim.x / panels) * panels;
  if ((int)blockIdx.x >= total) return;
  BandTile bt;
  if (!band_tile(a.offsets, a.experts, a.M, S::BM, panels, slot_of_block(blockIdx.x, total), bt)) return;
  const RowTile& rt = bt.rt;
  const int p = bt.p;
  const int rb0 = p * (S::BN / 16);
  const TileWave<WM, WN, TM> tw(a, rt, rb0);
  const int steps = tw.o.pairs;

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  uint4 x[2][TM], w[2][TN];  // by product
  uint32_t sx[TM], sx_read[TM][2], sw[TN], sw_read[TN];
  // the products q of a step of parity P; before(i) comes ahead of row tile i's, after(m) behind product m
  auto multiply = [&](auto parity, auto product, auto before, auto after) {
    constexpr int q = decltype(product)::value, kByte = 2 * decltype(parity)::value + q;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      before(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        acc[i][j] = mfma_mx4<kByte, kByte>(w[q][j], x[q][i], acc[i][j], sw[j], sx[i]);
        __builtin_amdgcn_sched_barrier(0);
        after(i * TN + j);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // A step of parity P: `far` is loaded for step s + 3 (with scales, where that is even).
  auto step = [&](auto parity, auto other, int s, uint8_t* cur, uint8_t* far, uint8_t* cur_scales, uint8_t* far_scales) {
    constexpr bool even = decltype(parity)::value == 0;
    constexpr int kLoads = S::LA + S::LB, kReads = TN + TM;
    auto read = [&](int q, int i) {  // share i of TM of product q's operands
#pragma unroll
      for (int r = (i * kReads + TM - 1) / TM; r < ((i + 1) * kReads + TM - 1) / TM; ++r) {
        if (r < TN) w[q][r] = tw.read_w(q, r, cur);
        else x[q][r - TN] = tw.read_x(q, r - TN, cur);
      }
    };
    all_done<2 * kLoads + S::kSl>();  // all but the loads of the next two steps
    multiply(
        other, One(),
        [&](int i) {
          read(0, i);
          if constexpr (even) {
            tw.read_xs(i, cur_scales, sx_read[i]);
#pragma unroll
            for (int j = i * TN / TM; j < (i + 1) * TN / TM; ++j) sw_read[j] = tw.read_ws(j, cur_scales);
          }
        },
        [&](int m) {
#pragma unroll
          for (int l = m * kLoads / (TM * TN); l < (m + 1) * kLoads / (TM * TN); ++l) tw.load(l, s + 3, far);
        });
    operands_ready();
    if constexpr (even) {
#pragma unroll
      for (int i = 0; i < TM; ++i) sx[i] = tw.take_xs(s, sx_read[i]);
#pragma unroll
      for (int j = 0; j < TN; ++j) sw[j] = sw_read[j];
    }
    multiply(parity, Zero(), [&](int i) { read(1, i); },
             [&](int m) {
               if (!even && m == TM * TN - 1) tw.load_scales(s + 3, far_scales);
             });
  };
#pragma unroll
  for (int j = 0; j < TN; ++j) {  // no step before the first
    w[1][j] = make_uint4(0, 0, 0, 0);
    sw[j] = 0;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    x[1][i] = make_uint4(0, 0, 0, 0);
    sx[i] = 0;
  }
  auto load_step = [&](int s, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < S::LA + S::LB; ++i) tw.load(i, s, to);
  };
  load_step(0, lds0);
  tw.load_scales(0, scales0);
  load_step(1, lds1);
  load_step(2, lds2);
  tw.load_scales(2, scales2);
  for (int s = 0; s < steps; s += 4) {  // steps past the last are of zeros
    step(Zero(), One(), s, lds0, lds3, scales0, nullptr);
    step(One(), Zero(), s + 1, lds1, lds0, nullptr, scales0);
    step(Zero(), One(), s + 2, lds2, lds1, scales2, nullptr);
    step(One(), Zero(), s + 3, lds3, lds2, nullptr, scales2);
  }
  operands_ready();
  multiply(One(), One(), [](int) {}, [](int) {});
  all_done<0>();  // no load into LDS is left, and nothing reads what the stages overwrite
  static_assert((S::NW + 1) / 2 * kStageBytes <= S::kBuffer, "stages fit two buffers");
  store_tile<TM, kF32>(a, rt, rt.r0 + 16 * tw.wm * TM, 16 * rb0 + 64 * tw.wn, acc,
                       (tw.wave & 1 ? lds1 : lds0) + (tw.wave >> 1) * kStageBytes);
}

// ---------------------------------------------------------------------------
// launch configuration
// ---------------------------------------------------------------------------
enum class Mx4 { kTile256, kDeep128, kDeep64x128, kDeep64, kDeep32x64, kStream1x4, kStream2x4, kStream2x2, kStream2x1 };

struct Mx4Shape {
  Mx4 kind;
  int BM, BN, threads;
  // the estimate of a call's time, us: start + (steps of 256 inputs) * max(one, all * blocks / slots),
  // and no less than bare + steps * step, what few blocks take
  int slots;
  double start, one, all, bare, step;
};
// Constants that lose least by the choice over the times of all these kernels (other weights than
// the last call's) on 14 matrices, N from 300 to 28672 and K from 128 to 9216, at 17 to 3000 rows and on 5
// sets of 8 to 128 experts at 13 to 400 rows each, popularity as 1 / rank and its root: 2.6% on
// average against the best of them each time, 32% at most.  (Constants fitted to one half of the
// sizes lose 2.6 to 3.5% on the other, and so do rounds of blocks counted as whole.)
// Two of them fit with `one` at zero, which says nothing of few outputs and many inputs: for these
// bare and step, from the times of launches of few blocks.  On 15 more matrices, N from 33 to 8192 and
// K from 9216 to 130944, and 3 sets of experts, the choice loses 3.6% on average and 53% at most (32%
// and 168% without bare and step: 64 rows of 2048 x 28672 took 60.4 us as 64 x 128, and take 22.5
// streamed); on 240 sizes drawn from N of 16 to 28672, K of 128 to 28672 and up to 128 experts 4.4%
// and 75% (4060 rows of 54 experts of 25 x 15360, streamed 24.4 us, as 32 x 64 13.9).
constexpr Mx4Shape kMx4Shapes[] = {
    {Mx4::kTile256, 256, 256, 512, 256, 3.4, 0, 1.77, 0, 0},
    {Mx4::kDeep128, 128, 128, 256, 256, 6.2, 0.473, 0.669, 0, 0},
    {Mx4::kDeep64x128, 64, 128, 256, 256, 9.7, 0, 0.395, 4.1, 0.295},
    {Mx4::kDeep64, 64, 64, 256, 512, 3.7, 0.227, 0.669, 0, 0},
    {Mx4::kDeep32x64, 32, 64, 128, 512, 3.6, 0.2, 0.547, 0, 0},
    {Mx4::kStream2x2, 16, 32, 128, 2048, 3.8, 0, 1.33, 3.4, 0.125},
    {Mx4::kStream2x1, 16, 32, 64, 4096, 2.7, 0.343, 1.53, 0, 0},
    {Mx4::kStream2x4, 16, 32, 256, 0, 0, 0, 0, 0, 0},
    {Mx4::kStream1x4, 16, 16, 256, 0, 0, 0, 0, 0, 0},
};

// The kernel for M rows shared out over `experts` matrices of N x K (their true sizes are on
// the GPU).  Up to 16 rows each the
// streaming form with as many wavefronts as there are few outputs (us, one row: 2560 x 9216 as
// one row block and four wavefronts 4.9, as two and four 5.4, two and two 6.3, two and
// one 10; 5120 x 5120 6.4, 5.5, 6.0, 8.6; 9216 x 2560 5.7, 5.9, 5.2, 5.5; 13 rows of 28672 x 8192
// 31, 28.5, 25.8, 23.7.  Experts drawn at random: 2 rows of 64 of 2048 x 2560 (nb 256) 3.9, 4.1, 4.0, 4.7; 4
// rows 4.9, 4.7, 4.4, 4.9; 16 rows 13.3, 11.5, 11.0, 9.1; 8 rows of 128 of 1408 x 2560 (nb 704) 5.9, 6.0, 5.5,
// 5.4; of 256 of 2048 x 896 (nb 1024) 5.9, 5.0, 4.3, 4.4; no such call of 8 sets of experts gained more than 4%
// by another of the four).  An expert that has all rows is streamed 16 at a time all the same: 512 rows of
// one of 64 of 2048 x 2560 13.6 us, as 64 x 64 7.4.  Beyond that the smallest estimate.  512 rows: 2560 x 9216
// take 14.6 us as 64 x 128 (160 blocks), 18.3 as 64 x 64, 19.2 as 128 x 128 and 31 as 256 x 256 (20 blocks);
// 17408 x 5120 (codes from memory) 59, 58, 50, which the estimate takes, and 41.
Mx4 choose_mx4(int64_t M, int64_t N, int64_t K, int64_t experts) {
  const int64_t busy = experts < M ? experts : M, rows = (M + busy - 1) / busy;
  const int64_t nb = (N + kTileRows - 1) / kTileRows * busy, steps = (K + kPair - 1) / kPair;
  if (rows <= 16) return nb < 256 ? Mx4::kStream1x4 : nb < 384 ? Mx4::kStream2x4 : nb < 1024 ? Mx4::kStream2x2 : Mx4::kStream2x1;
  Mx4 best = Mx4::kTile256;
  double least = 0;
  for (const Mx4Shape& s : kMx4Shapes) {
    if (s.slots == 0) continue;
    // experts are not evenly busy: half a row tile more for each
    const int64_t spread = M / s.BM + busy / 2;
    const int64_t tiles = busy == 1 ? (M + s.BM - 1) / s.BM : spread > busy ? spread : busy;
    const int64_t blocks = tiles * ((N + s.BN - 1) / s.BN);
    double load = (double)blocks / s.slots;
    if (s.kind == Mx4::kTile256) {  // whole rounds, the last one cut
      const int64_t left = blocks % kCus;
      load = (double)(blocks / kCus) + (left == 0 ? 0 : left <= kMostCut ? 0.45 : 1);
    }
    const double full = s.start + (double)steps * (load * s.all > s.one ? load * s.all : s.one);
    const double few = s.bare + (double)steps * s.step, cost = full > few ? full : few;
    if (least == 0 || cost < least) {
      least = cost;
      best = s.kind;
    }
  }
  return best;
}

// The kernel of a call, and its grid.
struct MxGrid {
  Mx4 kind;
  int threads;
  int64_t panels, blocks;
};

MxGrid mx4_grid(int64_t M, int64_t N, int64_t K, int64_t experts, bool grouped) {
  const Mx4 kind = choose_mx4(M, N, K, experts);
  MxGrid g{kind, 0, 0, 0};
  for (const Mx4Shape& s : kMx4Shapes)
    if (s.kind == kind) {
      g.threads = s.threads;
      g.panels = (N + s.BN - 1) / s.BN;
      g.blocks = max_row_tiles(M, experts, grouped, s.BM) * g.panels + (kind == Mx4::kTile256 ? 3 * kMostCut : 0);
    }
  return g;
}

template <bool kF32>
hipError_t launch_product(const MxArgs& a, hipStream_t st) {
  const MxGrid g = mx4_grid(a.M, a.N, a.K, a.experts, a.offsets != nullptr);
  const unsigned blocks = (unsigned)g.blocks;
  const int panels = (int)g.panels;
  switch (g.kind) {
    case Mx4::kTile256: mx4_tile_kernel<kF32><<<blocks, 512, 0, st>>>(a, panels); break;
    case Mx4::kDeep128: mx4_deep_kernel<2, 2, 4, kF32><<<blocks, 256, 0, st>>>(a, panels); break;
    case Mx4::kDeep64x128: mx4_deep_kernel<2, 2, 2, kF32><<<blocks, 256, 0, st>>>(a, panels); break;
    case Mx4::kDeep64: mx4_deep_kernel<4, 1, 1, kF32><<<blocks, 256, 0, st>>>(a, panels); break;
    case Mx4::kDeep32x64: mx4_deep_kernel<2, 1, 1, kF32><<<blocks, 128, 0, st>>>(a, panels); break;
    case Mx4::kStream1x4: mx4_stream_kernel<1, 4, false, kF32><<<blocks, 256, 0, st>>>(a); break;
    case Mx4::kStream2x4: mx4_stream_kernel<2, 4, false, kF32><<<blocks, 256, 0, st>>>(a); break;
    case Mx4::kStream2x2: mx4_stream_kernel<2, 2, false, kF32><<<blocks, 128, 0, st>>>(a); break;
    case Mx4::kStream2x1: {
      // Past the caches from 12 MiB of one matrix and from 32 MiB of experts that the call can read (what
      // the L2s of the eight XCDs hold together).  Us through the caches and past them, one row: 16384 x
      // 1408 (11 MiB) 4.53 and 4.75, 65536 x 384 (12 MiB) 6.06 and 5.68, 28672 x 1408 (19 MiB) 6.72 and
      // 6.19, 28672 x 5120 (70 MiB) 15.8 and 14.2; 16 rows 4.90 and 5.15, 6.74 and 6.56, 7.14 and 6.70, 17.2
      // and 16.1.  Experts drawn at random: 4 rows of 32 of 2560 x 4096 (20 MiB) 6.60 and 7.67, 32 of 256 of
      // 2048 x 896 (28 MiB) 8.24 and 8.38, 24 of 64 of 1408 x 2048 (33 MiB) 8.73 and 8.04, 16 of 64 of 2048 x
      // 2560 (40 MiB) 9.75 and 9.05, 16 of 32 of 2560 x 4096 (80 MiB) 17.9 and 16.2.  Between 16 and 32 MiB
      // either may win, by 7% at most below 32 (16 of 64 of 2048 x 1408, 22 MiB: 7.05 and 6.64); where one
      // expert has all the rows, past them takes up to 13% longer (14 rows of one of 32: 6.1 and 6.9).
      const int64_t busy = a.experts < a.M ? a.experts : a.M, bytes = busy * a.N * a.K / 2;
      if (bytes >= (busy == 1 ? 12 : 32) * (int64_t(1) << 20))
        mx4_stream_kernel<2, 1, true, kF32><<<blocks, 64, 0, st>>>(a);
      else mx4_stream_kernel<2, 1, false, kF32><<<blocks, 64, 0, st>>>(a);
      break;
    }
  }
  return hipGetLastError();
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
  return in_launches((N + kTileRows - 1) / kTileRows, kMostWaves / 4 / words, [&](int64_t r, int64_t n) {
    const uint8_t* from = static_cast<const uint8_t*>(W) + r * kTileRows * K * es;
    const int64_t rows = N - r * kTileRows;
    uint8_t *qt = q + r * pairs * 2048, *sc = s + r * words * 256;
    const unsigned blocks = (unsigned)(n * words);
    if (f32) quantize_weights_kernel<true><<<blocks, 256, 0, st>>>(from, rows, (int)K, (int)words, qt, sc);
    else quantize_weights_kernel<false><<<blocks, 256, 0, st>>>(from, rows, (int)K, (int)words, qt, sc);
  });
}

hipError_t launch_dequantize_mx4(const uint8_t* q, const uint8_t* s, int64_t N, int64_t K, void* W, bool f32,
                                 hipStream_t st) {
  const int64_t words = (K + kWord - 1) / kWord, pairs = (K + kPair - 1) / kPair, es = f32 ? 4 : 2;
  return in_launches((N + kTileRows - 1) / kTileRows, kMostWaves / 4 / words, [&](int64_t r, int64_t n) {
    uint8_t* to = static_cast<uint8_t*>(W) + r * kTileRows * K * es;
    const int64_t rows = N - r * kTileRows;
    const uint8_t *qt = q + r * pairs * 2048, *sc = s + r * words * 256;
    const unsigned blocks = (unsigned)(n * words);
    if (f32) dequantize_weights_kernel<true><<<blocks, 256, 0, st>>>(qt, sc, rows, (int)K, (int)words, to);
    else dequantize_weights_kernel<false><<<blocks, 256, 0, st>>>(qt, sc, rows, (int)K, (int)words, to);
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

bool fits_linear_mx4(int64_t M, int64_t N, int64_t K, int64_t experts, bool grouped) {
  const MxGrid g = mx4_grid(M, N, K, experts, grouped);
  return g.blocks * g.threads < kMaxThreads;
}

hipError_t launch_linear_mx4(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, const int32_t* offsets,
                             int64_t experts, const uint8_t* q, const uint8_t* s, int64_t N, void* y, bool f32,
                             hipStream_t st) {
  const bool lines = N * (f32 ? 4 : 2) % 128 == 0 && reinterpret_cast<uintptr_t>(y) % 128 == 0;
  const MxArgs a{xq, xs, offsets, q, s, y, (int)M, (int)K, (int)N, (int)experts, lines};
  return f32 ? launch_product<true>(a, st) : launch_product<false>(a, st);
}

}  // namespace w4
