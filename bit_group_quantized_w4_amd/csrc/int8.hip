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

namespace w4 {
namespace {

constexpr int kStep = 64;           // inputs per tile
constexpr float kMaxCode8 = 127.0f;  // largest magnitude maps to code +-127
// Added to the offset of an operand of a step past the last one: one matrix's codes, and
// one tile's rows of x, take less than 2 GiB, so an offset inside its buffer ends outside
// it and reads zeros without touching memory, and so does that of a row of x that the tile
// does not have (at most 2^25).  Only a row block past the matrix's last one, of codes
// within 32 MiB of 2 GiB, can end inside the buffer again (the sum wraps): it reads codes
// of this matrix, they meet zeros of x, and the outputs are past N, which no kernel stores.
constexpr uint32_t kOob = 0x80000000u;

typedef int i32x4 __attribute__((__vector_size__(4 * sizeof(int))));

__device__ __forceinline__ i32x4 mfma16x16x64(const i32x4& a, const i32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Byte offset of input k of row n in the native layout.
__device__ __forceinline__ int64_t native_at(int64_t n, int64_t k, int64_t K) {
  return ((n >> 4) * (K / kStep) + k / kStep) * 1024 + ((k >> 4) & 3) * 256 + (n & 15) * 16 + (k & 15);
}

// Code of v against the scale d: round half away of the IEEE quotient.
__device__ __forceinline__ uint32_t code_of(float v, float d) {
  const float t = v / d;
  float r = truncf(t);
  r = fabsf(t - r) >= 0.5f ? r + copysignf(1.0f, t) : r;
  return (uint32_t)(int)fminf(fmaxf(r, -kMaxCode8), kMaxCode8) & 0xFFu;
}

// Value j of a 16-byte chunk: four fp32, or eight bf16.
template <bool kF32>
__device__ __forceinline__ float value_of(const uint4& c, int j) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  if constexpr (kF32) return __uint_as_float(w[j]);
  return __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
}

// The largest magnitude bits of a chunk joined with `m`: as integers, a NaN is above
// infinity and infinity above every finite value.  bf16: two maxima, one per half.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <bool kF32>
__device__ __forceinline__ uint32_t max_bits(const uint4& c, uint32_t m) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kF32)
      m = max(m, w[i] & 0x7FFFFFFFu);
    else
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                 __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu)));
  }
  return m;
}

// Quantizes one row with `TPR` threads: the row's largest magnitude, then its codes.
// The first C chunks of 16 bytes per thread stay in registers between the two, so
// that a row is read once; what is left of a longer one is read again (from a cache).
// kNative: rows of a weight, written as tiles; blocks go to the eight XCDs in turn,
// and each XCD is given whole row blocks, row after row, so that the 16 bytes that
// a row adds to each 256 meet in one L2.  Otherwise tokens, written row-major.
//
// Codes: with y = 1 / d rounded, v * y + 1.5 * 2^23 has the nearest integer of v * y in
// its low bits, in one fma.  v * y is within 127.5 * 2^-24 of v / d, and the IEEE quotient
// that the code is defined by within 2^-18 of it: together less than 2^-16, so the
// code is the same unless v * y lies that near to a half-integer.  Where a thread
// of the wavefront finds one of its chunk's values within 2^-15 of a half (a share of 2^-14
// of the values: 1.6% of the wavefront's fp32 chunks of 256 values, 3% of its bf16 ones of
// 512), or the scale lies outside [2^-100, 2^100], the chunk's codes are
// formed from the IEEE quotients.
//
// Bound by memory: 28672 x 8192 weights (1.17 GB) take 232 us (5.1 TB/s; a copy
// reaches 4.9), 4099 x 28672 bf16 tokens (353 MB) 58.6 us (6.0 TB/s).
template <bool kF32, bool kNative, int TPR, int C>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void quantize_rows_kernel(const void* __restrict__ x, int rows,
                                                                              int padded, int K,
                                                                              int8_t* __restrict__ q,
                                                                              float* __restrict__ scale) {
  constexpr int E = kF32 ? 4 : 8;                 // values per chunk
  constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;  // rows per block
  const int at = threadIdx.x % TPR;
  int row = blockIdx.x * RPB + (RPB > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0);
  if constexpr (kNative) {
    constexpr int kBlocks = kTileRows / RPB;  // blocks per row block
    const int i = blockIdx.x / kXcds;
    row = ((i / kBlocks) * kXcds + blockIdx.x % kXcds) * kTileRows + (i % kBlocks) * RPB +
          (RPB > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0);
  }
  const bool real = row < rows;
  // (a row of padding reads zeros, and so does a chunk past the row's end)
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(static_cast<const uint8_t*>(x) + (int64_t)(real ? row : 0) * K * (kF32 ? 4 : 2),
                                              real ? (uint32_t)K * (kF32 ? 4u : 2u) : 0u);
  const int chunks = K / E;
  uint4 c[C];
#pragma unroll
  for (int i = 0; i < C; ++i) c[i] = bload<kNonTemporal>(rs, (uint32_t)(at + i * TPR) * 16u);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) m = max_bits<kF32>(c[i], m);
  for (int i = at + C * TPR; i < chunks; i += TPR) m = max_bits<kF32>(bload<0>(rs, (uint32_t)i * 16u), m);
  if constexpr (!kF32) m = max(m & 0xFFFFu, m >> 16) << 16;
#pragma unroll
  for (int s = 32; s; s >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s));
  if constexpr (TPR > 64) {
    __shared__ uint32_t part[TPR / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) m = max(m, part[w]);
  }
  const bool bad = m >= 0x7F800000u;
  const float d = bad ? __uint_as_float(kNanBits) : __uint_as_float(m) / kMaxCode8;
  const bool usable = !bad && d != 0.0f;
  const float y = 1.0f / (usable ? d : 1.0f);
  const bool far = !(d >= 0x1p-100f && d <= 0x1p+100f);
  auto codes = [&](const uint4& v, uint32_t (&out)[E / 4]) {
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
    uint32_t b[E];
    float worst = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float f = value_of<kF32>(v, j), r = fmaf(f, y, kMagic);
      b[j] = __float_as_uint(r);
      worst = fmaxf(worst, fabsf(fmaf(f, y, kMagic - r)));
    }
    if (__ballot(worst > 0.5f - 0x1p-15f || far)) {
#pragma unroll
      for (int j = 0; j < E; ++j) b[j] = usable ? code_of(value_of<kF32>(v, j), d) : 0;
    }
#pragma unroll
    for (int w = 0; w < E / 4; ++w) {  // the low bytes of four words
      const uint32_t lo = __builtin_amdgcn_perm(b[4 * w + 1], b[4 * w], 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(b[4 * w + 3], b[4 * w + 2], 0x04000C0Cu);
      out[w] = lo | hi;
    }
  };
  auto store = [&](int i, const uint32_t (&o)[E / 4]) {
    int8_t* to = q + (kNative ? native_at(row, (int64_t)i * E, K) : (int64_t)row * K + (int64_t)i * E);
    if constexpr (E == 8)
      *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
    else
      *reinterpret_cast<uint32_t*>(to) = o[0];
  };
  if (row >= padded) return;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (at + i * TPR < chunks) {
      uint32_t o[E / 4];
      codes(c[i], o);
      store(at + i * TPR, o);
    }
  }
  for (int i = at + C * TPR; i < chunks; i += TPR) {
    uint32_t o[E / 4];
    codes(bload<0>(rs, (uint32_t)i * 16u), o);
    store(i, o);
  }
  if (at == 0 && real) scale[row] = d;
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

// Outputs by way of LDS: sixteen rows of 64 outputs that a wavefront holds in the
// matrix unit's order are written to a stage of its own, kStagePitch words a row, and
// stored from there 16 bytes per lane, so that one store covers whole lines of y (4096 x 9216
// fp32 outputs of K = 1152: 94 us, and 115 us with each lane's outputs stored from its
// registers; bf16 64 us either way).  Stores go by 16 bytes whatever the
// alignment of a row of y, which the hardware allows (N = 9217: bf16 78 us, 140 us one
// output at a time; fp32 99 and 211 us).
// (The pitch of 68 words spreads sixteen rows over the banks.)
constexpr int kStagePitch = 68, kStageBytes = 16 * kStagePitch * 4;

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
template <bool kF32, class Value>
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
        __builtin_memcpy(to, v, 16);
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
        __builtin_memcpy(to, u, 16);
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

// Sums of TM row tiles of a wavefront, lane l's outputs n0 + 16 (l / 16) .. + 15 of rows
// m0 + l % 16 + 16 i, scaled and stored by way of `stage` (kStageBytes of the
// wavefront's own).
template <int TM, bool kF32>
__device__ __forceinline__ void store_tile(const I8Args& a, const RowTile& rt, int m0, int n0, const i32x4 (&acc)[TM][4],
                                           uint8_t* stage) {
  constexpr int E = kStageOut<kF32>;
  uint32_t* words = reinterpret_cast<uint32_t*>(stage);
  const int lane = threadIdx.x & 63;
  float d[E], sx[TM][16 / E];
#pragma unroll
  for (int e = 0; e < E; ++e) d[e] = a.d[(int64_t)rt.expert * a.N + min(n0 + stage_col<kF32>() + e, a.N - 1)];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int s = 0; s < 16 / E; ++s) sx[i][s] = a.sx[min(m0 + 16 * i + stage_row<kF32>(s), rt.r1 - 1)];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<i32x4*>(words + (lane & 15) * kStagePitch + 16 * (lane >> 4) + 4 * j) = acc[i][j];
    store_stage<kF32>(words, a.y, a.N, m0 + 16 * i, rt.r1, n0,
                      [&](uint32_t w, int s, int e) { return (float)(int)w * sx[i][s] * d[e]; });
  }
}

// Streaming form, for few rows: a block owns R row blocks of 16 outputs and one
// tile of 16 MT rows of x; its NW wavefronts divide K.  Lane l of a wavefront holds
// A[l % 16][16 (l / 16) .. + 15] of x, the tile's B operand and
// D[4 (l / 16) + j][l % 16], j = 0..3, all straight from memory.
//
// Bound by the weight stream: 13 rows of 28672 x 8192 take 40 us (5.9 TB/s).
template <int MT, int R, int NW, int kCache, bool kF32>
__device__ __forceinline__ void stream_row_tile(const I8Args& a, const RowTile& rt, int rb0,
                                                i32x4 (&red)[NW][MT * R][64]) {
  constexpr int kWide = MT > R ? MT : R;
  constexpr int D = kWide >= 4 ? 2 : 8 / kWide;  // steps in flight: about 8 KiB per wavefront
  const int nb = (a.N + kTileRows - 1) / kTileRows;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, kb = lane >> 4;
  const int steps = a.K / kStep;
  const int s0 = (int)((int64_t)steps * wave / NW), s1 = (int)((int64_t)steps * (wave + 1) / NW);

  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.q + (int64_t)rt.expert * nb * kTileRows * a.K, (uint32_t)nb * kTileRows * (uint32_t)a.K);
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.xq + (int64_t)rt.r0 * a.K, (uint32_t)(rt.r1 - rt.r0) * (uint32_t)a.K);
  // (row blocks past the matrix's last and rows past the tile's last lie outside the buffers)
  uint32_t wo[R], xo[MT];
#pragma unroll
  for (int r = 0; r < R; ++r) wo[r] = ((uint32_t)(rb0 + r) * steps * 64u + lane) * 16u;
#pragma unroll
  for (int i = 0; i < MT; ++i) xo[i] = (uint32_t)(16 * i + nl) * (uint32_t)a.K + 16u * kb;

  i32x4 acc[MT][R];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[i][r] = i32x4{0, 0, 0, 0};
  // a ring of D steps' operands; a step past the wavefront's last reads zeros (see
  // kOob), so that every load is unconditional
  uint4 w[D][R], x[D][MT];
  auto issue = [&](int c, int s) {
    const uint32_t ow = s < s1 ? (uint32_t)s * 1024u : kOob, ox = s < s1 ? (uint32_t)s * kStep : kOob;
#pragma unroll
    for (int r = 0; r < R; ++r) w[c][r] = bload<kCache>(rw, wo[r] + ow);
#pragma unroll
    for (int i = 0; i < MT; ++i) x[c][i] = bload<0>(rx, xo[i] + ox);
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
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[i][r] = mfma16x16x64(bitcast<i32x4>(x[c][i]), bitcast<i32x4>(w[c][r]), acc[i][r]);
      issue(c, s + c + D);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

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
    for (int w_ = 1; w_ < NW; ++w_) v += red[w_][c][lane];
    const float d = a.d[(int64_t)rt.expert * a.N + n];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = rt.r0 + 16 * i + 4 * kb + j;
      if (m < rt.r1) store_scaled<kF32>(a, m, n, v[j], a.sx[m], d);
    }
  }
}

// kPast: an expert's weights are read past the caches, unless another row tile of the
// expert reads them too.  (us as graph nodes, other weights than the last call's, through
// the caches and past them: 13 rows of 28672 x 8192 44.8 and 39.5, 32 rows of 16 experts of
// 5120 x 2560 37.0 and 32.4.  Where experts have several row tiles, past for all and for
// the lone tiles only: 96 rows of 8 experts of 14336 x 4096, popularity falling as 1 / rank,
// 92.6 and 86.1, all on one expert 51.3 and 39.6; 192 rows of 16 of 5120 x 2560, 44.6 and
// 42.3, on one 24.1 and 18.7; evenly shared out equal.)
template <int MT, int R, int NW, bool kPast, bool kF32>
__global__ __launch_bounds__(NW * 64) void w8a8_stream_kernel(const I8Args a) {
  const int nb = (a.N + kTileRows - 1) / kTileRows, panels = (nb + R - 1) / R;
  const int t = blockIdx.x / panels, rb0 = (blockIdx.x - t * panels) * R;
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, 16 * MT, t, rt)) return;
  __shared__ i32x4 red[NW][MT * R][64];
  if (kPast && rt.alone) stream_row_tile<MT, R, NW, kNonTemporal, kF32>(a, rt, rb0, red);
  else stream_row_tile<MT, R, NW, 0, kF32>(a, rt, rb0, red);
}

// Tile form, for many rows: a block of WM x WN wavefronts owns BM = 16 WM TM rows
// of x and BN = 64 WN outputs; each wavefront holds TM x 4 tiles of 16 x 16 sums
// in registers.  A step is 128 inputs: the block's slices of x and of the weights
// go to LDS straight from memory (no registers in between), one step ahead of the
// products, in two LDS buffers.
//
// x is row-major, 128 bytes of a row per step: lane l of a load takes row
// l / 8 of eight, and its 16-byte chunk (l % 8) ^ (l / 8), so that chunk c of row
// r sits at position c ^ (r % 8) of the row's 128 bytes and the sixteen rows of
// an operand are read without bank conflicts.  (Steps of 64 inputs in four
// buffers, three steps ahead, took half lines of x: 7% slower at 256 x 256.)
//
// The weights are the first operand, so a lane holds four consecutive rows of
// the first operand, D[4 (l / 16) + e][l % 16], for one row of x.  Row 4 q + e of
// tile j of a wavefront's four is output 16 q + 4 j + e: a lane ends with sixteen
// consecutive outputs of its row, a wavefront with 64.  A row block's 2 KiB of a
// step are 64 bytes apart from the next one's in LDS, which spreads the four
// row blocks that one operand then touches over the banks.
//
// The products of a step run in four parts (half of the rows times half of the
// inputs).  Operands are read from LDS one part ahead, beside the products of the
// part before, and the next step's loads are issued beside the first part: one
// load holds up the wavefront for the 16 cycles that the address unit of the CU
// takes for it, which eight wavefronts would otherwise spend in turn before any
// product (4096 rows of 17408 x 5120: 361 us with all reads and loads first, 338
// with both spread).  Now 310 to 329 us, 2.2 to 2.4 POP/s: the clock falls from 2.4 to
// 2.04 GHz at that rate, a CU has a tile 81% of the time (1088 tiles are five rounds of 256,
// the last a quarter full), and the matrix units are busy in 65% of those cycles.
//
// Rows past the tile's last, row blocks past the matrix's last and steps past the
// last one lie outside their buffers: such loads give zeros (see kOob).
constexpr int kRowBlockLds = 2 * 1024 + 64;

template <int WM, int WN, int TM, int OCC, bool kF32>
__global__ __launch_bounds__(WM* WN * 64, OCC) void w8a8_tile_kernel(const I8Args a, int panels) {
  constexpr int TN = 4;       // sixteen consecutive outputs per lane
  constexpr int TH = TM / 2;  // row tiles per part
  constexpr int NW = WM * WN, BM = 16 * WM * TM, BN = 16 * WN * TN;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KiB loads per wavefront and step
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN && LB % 2 == 0 && TH * 2 == TM, "loads shared out evenly");
  constexpr int kX = BM * 128, kBuffer = kX + BN / 16 * kRowBlockLds;
  // two variables, each named outright where it is used: the compiler then knows
  // that loads into one are no reason to wait before reading the other
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kBuffer], lds1[kBuffer];

  // (offsets whose ranges overlap could make more tiles than the launch covers)
  const int tiles = min(count_row_tiles(a.offsets, a.experts, a.M, BM), (int)gridDim.x / panels);
  if ((int)blockIdx.x >= tiles * panels) return;
  int t, p;
  tile_of_block(blockIdx.x, tiles, panels, t, p);
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, BM, t, rt)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, kb = lane >> 4;
  const int wm = wave / WN, wn = wave - wm * WN;
  const int K = a.K, nb = (a.N + kTileRows - 1) / kTileRows, rb0 = p * (BN / 16);
  const int rows = rt.r1 - rt.r0, steps = K / 128;

  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.q + (int64_t)rt.expert * nb * kTileRows * K, (uint32_t)nb * kTileRows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.xq + (int64_t)rt.r0 * K, (uint32_t)rows * (uint32_t)K);
  const uint32_t xo = (uint32_t)(8 * wave * LA + (lane >> 3)) * (uint32_t)K + 16u * ((lane & 7) ^ (lane >> 3));
  const uint32_t wo = (uint32_t)(rb0 + wave * LB / 2) * 16u * (uint32_t)K + 16u * lane;
  typedef __attribute__((address_space(3))) void* lds_ptr;
  // load i of this wavefront's for step s (zeros past the last step)
  auto load = [&](int i, int s, uint8_t* to) {
    if (i < LA) {
      const uint32_t k = s < steps ? (uint32_t)s * 128u : kOob;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr)(to + (wave * LA + i) * 1024), 16,
                                               (int)(xo + (uint32_t)(8 * i * K) + k), 0, 0, 0);
    } else {
      const uint32_t k = s < steps ? (uint32_t)s * 2048u : kOob;
      const int r = (i - LA) >> 1, h = (i - LA) & 1;  // row block, half of the step
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr)(to + kX + (wave * LB / 2 + r) * kRowBlockLds + h * 1024), 16,
                                               (int)(wo + (uint32_t)(16 * r * K + 1024 * h) + k), 0, 0, 0);
    }
  };
  auto load_step = [&](int s, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) load(i, s, to);
  };
  // Every load into LDS and every read of it that this wavefront has issued is
  // done, and so are the other wavefronts'.
  auto all_done = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  const uint32_t xa = (uint32_t)(wm * TM * 16 + nl) * 128u + 16u * (kb ^ (nl & 7));
  const uint32_t wa = (uint32_t)kX + (uint32_t)(wn * TN + (nl >> 2)) * kRowBlockLds + 256u * kb + 16u * (nl & 3);
  i32x4 x[2][TH], w[2][TN];  // x by row half, w by input half
  auto read_w = [&](int h, int j, const uint8_t* from) {
    w[h][j] = *reinterpret_cast<const i32x4*>(from + wa + j * 64 + h * 1024);
  };
  auto read_x = [&](int h, int c, int i, const uint8_t* from) {
    x[c][i] = *reinterpret_cast<const i32x4*>(from + (xa ^ (64u * h)) + (c * TH + i) * 2048);
  };
  // the products of row half c and input half h; beside(i) comes before row tile i's
  auto multiply = [&](int c, int h, auto beside) {
#pragma unroll
    for (int i = 0; i < TH; ++i) {
      beside(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[c * TH + i][j] = mfma16x16x64(w[h][j], x[c][i], acc[c * TH + i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto operands_ready = [] {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
  };
  // A step whose slices are in `cur`, with the last part of the step before; its
  // own last part is left to the next.
  auto step = [&](int s, uint8_t* cur, uint8_t* nxt) {
    constexpr int kLoads = LA + LB, kReads = TN + TH;
    auto read = [&](int h, int i) {  // share i of TH of input half h's operands
#pragma unroll
      for (int r = (i * kReads + TH - 1) / TH; r < ((i + 1) * kReads + TH - 1) / TH; ++r) {
        if (r < TN) read_w(h, r, cur);
        else read_x(h, 0, r - TN, cur);
      }
    };
    all_done();  // `cur` is filled, and nothing reads `nxt` any more
    __builtin_amdgcn_sched_barrier(0);
    multiply(1, 1, [&](int i) {
#pragma unroll
      for (int l = i * kLoads / TH; l < (i + 1) * kLoads / TH; ++l) load(l, s + 1, nxt);
      read(0, i);
    });
    operands_ready();
    multiply(0, 0, [&](int i) { read_x(0, 1, i, cur); });
    operands_ready();
    multiply(1, 0, [&](int i) { read(1, i); });
    operands_ready();
    multiply(0, 1, [&](int i) { read_x(1, 1, i, cur); });
  };

  load_step(0, lds0);
#pragma unroll
  for (int j = 0; j < TN; ++j) w[1][j] = i32x4{0, 0, 0, 0};  // no step before the first
#pragma unroll
  for (int i = 0; i < TH; ++i) x[1][i] = i32x4{0, 0, 0, 0};
  for (int s = 0; s < steps; s += 2) {  // an odd last step is followed by one of zeros
    step(s, lds0, lds1);
    step(s + 1, lds1, lds0);
  }
  multiply(1, 1, [](int) {});
  all_done();  // no load into LDS is left, and nothing reads what the stages overwrite
  static_assert(NW * kStageBytes <= kBuffer, "stages fit a buffer");
  store_tile<TM, kF32>(a, rt, rt.r0 + 16 * wm * TM, 16 * rb0 + 64 * wn, acc, lds0 + wave * kStageBytes);
}

// The same for fewer rows, where a launch has too few tiles to fill the GPU and
// each block's time is the latency of its loads: smaller tiles, steps of 64 inputs
// in four LDS buffers, loaded three steps ahead, and G groups of WM x WN
// wavefronts that divide K and add their sums at the end.
//
// 64 bytes of a row per step: lane l of a load takes row l / 4 of sixteen and its
// chunk (l % 4) ^ t, t = 0, 2, 3, 1 for rows 0-3, 4-7, 8-11, 12-15, which keeps the
// operand reads free of bank conflicts (LDS serves lanes 0-3, 12-15 and 20-27 of
// a 16-byte read together).  333 rows of 2561 x 9216: 21 us with 64 x 64 tiles and
// two groups, 43 us as 128 x 128 tiles of the kernel above.  Bound by what L2 delivers: a
// block alone takes 0.12 us per 128 inputs, 246 of them at once 0.24 us; together they load
// 290 MB (14 TB/s, 77% of the requests hits), and the matrix units are busy in 24% of
// the cycles; four groups, twice the loads in flight, take 1 us longer.
__device__ __forceinline__ uint32_t quad_swizzle(int t) { return (0x78u >> (2 * t)) & 3u; }

template <int WM, int WN, int TM, int G, bool kF32>
__global__ __launch_bounds__(WM* WN* G * 64) void w8a8_deep_kernel(const I8Args a, int panels) {
  constexpr int TN = 4, TH = TM / 2;
  constexpr int NW = WM * WN, BM = 16 * WM * TM, BN = 16 * WN * TN;
  constexpr int LA = BM / 16 / NW, LB = BN / 16 / NW;  // 1 KiB loads per wavefront and step
  static_assert(LA * NW * 16 == BM && LB * NW * 16 == BN && TH * 2 == TM, "loads shared out evenly");
  constexpr int kRowBlock = 1024 + 64;
  constexpr int kX = BM * 64, kBuffer = kX + BN / 16 * kRowBlock;
  static_assert(TM * TN * NW * 1024 <= 4 * kBuffer, "a group's sums fit its buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[G * kBuffer], lds1[G * kBuffer], lds2[G * kBuffer],
      lds3[G * kBuffer];

  // (offsets whose ranges overlap could make more tiles than the launch covers)
  const int tiles = min(count_row_tiles(a.offsets, a.experts, a.M, BM), (int)gridDim.x / panels);
  if ((int)blockIdx.x >= tiles * panels) return;
  int t, p;
  tile_of_block(blockIdx.x, tiles, panels, t, p);
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, BM, t, rt)) return;
  const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, kb = lane >> 4;
  const int g = wave_all / NW, wave = wave_all - g * NW;
  const int wm = wave / WN, wn = wave - wm * WN;
  const int K = a.K, nb = (a.N + kTileRows - 1) / kTileRows, rb0 = p * (BN / 16);
  const int rows = rt.r1 - rt.r0, steps = K / kStep;
  const int per = (steps + G - 1) / G, first = g * per, last = min(first + per, steps);  // the group's steps

  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.q + (int64_t)rt.expert * nb * kTileRows * K, (uint32_t)nb * kTileRows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.xq + (int64_t)rt.r0 * K, (uint32_t)rows * (uint32_t)K);
  const uint32_t xo = (uint32_t)(16 * wave * LA + (lane >> 2)) * (uint32_t)K + 16u * ((lane & 3) ^ quad_swizzle(lane >> 4));
  const uint32_t wo = (uint32_t)(rb0 + wave * LB) * 16u * (uint32_t)K + 16u * lane;
  typedef __attribute__((address_space(3))) void* lds_ptr;
  auto load = [&](int i, int s, uint8_t* to) {
    to += g * kBuffer;
    if (i < LA) {
      const uint32_t k = s < last ? (uint32_t)s * 64u : kOob;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr)(to + (wave * LA + i) * 1024), 16,
                                               (int)(xo + (uint32_t)(16 * i * K) + k), 0, 0, 0);
    } else {
      const uint32_t k = s < last ? (uint32_t)s * 1024u : kOob;
      const int r = i - LA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr)(to + kX + (wave * LB + r) * kRowBlock), 16,
                                               (int)(wo + (uint32_t)(16 * r * K) + k), 0, 0, 0);
    }
  };
  auto load_step = [&](int s, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) load(i, s, to);
  };

  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const uint32_t xa = (uint32_t)(g * kBuffer) + (uint32_t)(wm * TM * 16 + nl) * 64u + 16u * (kb ^ quad_swizzle(nl >> 2));
  const uint32_t wa = (uint32_t)(g * kBuffer + kX) + (uint32_t)(wn * TN + (nl >> 2)) * kRowBlock + 256u * kb + 16u * (nl & 3);
  i32x4 x[2][TH], w[2][TN];  // x by row half, w by step parity
  auto multiply = [&](int c, int v, auto beside) {
#pragma unroll
    for (int i = 0; i < TH; ++i) {
      beside(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[c * TH + i][j] = mfma16x16x64(w[v][j], x[c][i], acc[c * TH + i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto step = [&](int s, int v, uint8_t* cur, uint8_t* prev) {
    constexpr int kLoads = LA + LB, kReads = TN + TH;
    asm volatile("" ::: "memory");
    constexpr int kLeft = 2 * kLoads;  // vmcnt: the last two steps' loads; lgkmcnt(0)
    __builtin_amdgcn_s_waitcnt(0x0070 | (kLeft & 15) | (kLeft >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    multiply(1, v ^ 1, [&](int i) {  // the last part of the step before
#pragma unroll
      for (int l = i * kLoads / TH; l < (i + 1) * kLoads / TH; ++l) load(l, s + 3, prev);
#pragma unroll
      for (int r = (i * kReads + TH - 1) / TH; r < ((i + 1) * kReads + TH - 1) / TH; ++r) {
        if (r < TN) w[v][r] = *reinterpret_cast<const i32x4*>(cur + wa + r * 64);
        else x[0][r - TN] = *reinterpret_cast<const i32x4*>(cur + xa + (r - TN) * 1024);
      }
    });
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
    multiply(0, v, [&](int i) { x[1][i] = *reinterpret_cast<const i32x4*>(cur + xa + (TH + i) * 1024); });
  };
#pragma unroll
  for (int j = 0; j < TN; ++j) w[1][j] = i32x4{0, 0, 0, 0};  // no step before the first
#pragma unroll
  for (int i = 0; i < TH; ++i) x[1][i] = i32x4{0, 0, 0, 0};
  load_step(first, lds0);
  load_step(first + 1, lds1);
  load_step(first + 2, lds2);
  for (int s = 0; s < per; s += 4) {  // every group takes the same number of steps, zeros at the end
    step(first + s, 0, lds0, lds3);
    step(first + s + 1, 1, lds1, lds0);
    step(first + s + 2, 0, lds2, lds1);
    step(first + s + 3, 1, lds3, lds2);
  }
  multiply(1, 1, [](int) {});
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0): no load into LDS is left,
  __builtin_amdgcn_s_barrier();        // and nothing reads what is overwritten now
  asm volatile("" ::: "memory");
  if constexpr (G > 1) {
    // chunk c of a group's sums, 1 KiB per wavefront, in buffer c % 4
    auto chunk = [&](int gg, int c) {
      uint8_t* b = c % 4 == 0 ? lds0 : c % 4 == 1 ? lds1 : c % 4 == 2 ? lds2 : lds3;
      return reinterpret_cast<i32x4*>(b + gg * kBuffer + ((c / 4) * NW + wave) * 1024 + 16 * lane);
    };
    if (g > 0) {
#pragma unroll
      for (int c = 0; c < TM * TN; ++c) *chunk(g, c) = acc[c / TN][c % TN];
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int gg = 1; gg < G; ++gg)
#pragma unroll
      for (int c = 0; c < TM * TN; ++c) acc[c / TN][c % TN] += *chunk(gg, c);
  }
  // (the first group's part of the buffers holds no sums)
  static_assert(NW <= 4 && kStageBytes <= kBuffer, "a stage per buffer");
  uint8_t* stage = wave == 0 ? lds0 : wave == 1 ? lds1 : wave == 2 ? lds2 : lds3;
  store_tile<TM, kF32>(a, rt, rt.r0 + 16 * wm * TM, 16 * rb0 + 64 * wn, acc, stage);
}

// ---------------------------------------------------------------------------
// launch configuration
// ---------------------------------------------------------------------------
enum class W8a8 { kTile256, kTile128, kDeep128, kDeep64x128, kDeep64, kStream32x64, kStream16x64, kRows16 };

// The kernel for M rows shared out over `experts` matrices of N x K (their true
// sizes are on the GPU: all are taken to be as busy as the average one).  Up to 16
// rows each the weight stream is all there is to do.  Of grouped calls with 13 to 16 rows per
// expert on average many have experts with more than 16; two row tiles per block read the
// weights of those once.  There neither form is best everywhere (us, 16 and 32 rows per
// block, popularity as 1 / sqrt(rank): 1024 rows of 64 experts of 1408 x 2560 53.8 and 50.7, of
// 2048 x 2048 51.6 and 49.0, 128 of 8 of 14336 x 4096 92.1 and 85.7; but 128 of 8 of 2560 x 2560
// 15.7 and 16.6, 512 of 32 of 2560 x 1408 27.2 and 29.1, and 16 rows for each expert 76.2 and
// 87.2 at 14336 x 4096), up to 12 the first nearly is (640 rows of the 64 experts of 2048 x
// 2048 45.5 and 48.1, 96 of 8 of 14336 x 4096 79.4 and 86.3).  Beyond that the smallest
// estimate wins, in us per 128 inputs, from times measured on the 2560 x 9216,
// 9216 x 2560, 28672 x 8192 and 17408 x 5120 matrices at 32 to 4096 rows: `one` while
// every block has a CU for itself, `all` for each further full set of `slots` blocks.
// Small tiles win until the larger ones fill the GPU: 512 rows of 2560 x 9216 take
// 27 us as 64 x 128 (160 blocks), 35 us as 64 x 64 and 48 us as 128 x 128 (80 blocks);
// at 2048 rows 69, 82 and 60 us.
W8a8 choose_w8a8(int64_t M, int64_t N, int64_t experts, bool grouped) {
  const int64_t busy = experts < M ? experts : M, rows = (M + busy - 1) / busy;
  if (rows <= 16) return rows <= 12 || M <= 16 ? W8a8::kRows16 : W8a8::kStream32x64;
  struct Shape {
    W8a8 kind;
    int BM, BN, slots;
    double one, all;
  };
  static const Shape shapes[] = {
      {W8a8::kTile256, 256, 256, 256, 1.68, 1.68},     {W8a8::kTile128, 128, 128, 512, 0.66, 1.07},
      {W8a8::kDeep128, 128, 128, 512, 0.52, 1.24},     {W8a8::kDeep64x128, 64, 128, 768, 0.40, 1.40},
      {W8a8::kDeep64, 64, 64, 512, 0.34, 0.70},        {W8a8::kStream32x64, 32, 64, 256, 0.22, 0.33},
      {W8a8::kStream16x64, 16, 64, 256, 0.17, 0.21},
  };
  W8a8 best = W8a8::kTile256;
  double least = 0;
  for (const Shape& s : shapes) {
    const int64_t blocks = busy * ((rows + s.BM - 1) / s.BM) * ((N + s.BN - 1) / s.BN);
    double cost = s.one;
    if (blocks > 256) {
      // The largest tiles run in whole rounds; smaller ones fill the gaps, and so do the
      // experts' partial tiles, which take less power (4096 rows of 16 experts of 5120 x 4096:
      // 127 us as 256 x 256, 148 as 128 x 128; 2048 rows 114 and 96).
      const double rounds = s.BM == 256 && !grouped ? (double)((blocks + 255) / 256) : (double)blocks / s.slots;
      cost = rounds * s.all > s.one ? rounds * s.all : s.one;
    }
    if (least == 0 || cost < least) {
      least = cost;
      best = s.kind;
    }
  }
  return best;
}

// The kernel of a call, and its grid.
struct W8a8Grid {
  W8a8 kind;
  int BM, BN, threads;
  int64_t panels, blocks;
};

W8a8Grid w8a8_grid(int64_t M, int64_t N, int64_t experts, bool grouped) {
  W8a8Grid g{choose_w8a8(M, N, experts, grouped), 0, 0, 256, 0, 0};
  auto tile = [&](int BM, int BN, int threads) {
    g.BM = BM;
    g.BN = BN;
    g.threads = threads;
  };
  switch (g.kind) {
    case W8a8::kTile256: tile(256, 256, 512); break;
    case W8a8::kTile128:
    case W8a8::kDeep128: tile(128, 128, 256); break;
    case W8a8::kDeep64x128: tile(64, 128, 256); break;
    case W8a8::kDeep64: tile(64, 64, 256); break;
    case W8a8::kStream32x64: tile(32, 64, 256); break;
    case W8a8::kStream16x64: tile(16, 64, 256); break;
    case W8a8::kRows16: {
      // Two row blocks per wavefront once that leaves enough blocks, and K divided
      // between two wavefronts where the row blocks alone fill the GPU, else four
      // (one row: 2560 x 9216 6.6 us as one row block and four wavefronts, 9.0 as two
      // and two; 9216 x 2560 6.6 and 6.4; 5120 x 17408 16.5 as two and four, 19.9 as
      // one and four).
      const int64_t nb = (N + kTileRows - 1) / kTileRows * (experts < M ? experts : M);
      if (nb < 256) tile(16, 16, 256);
      else tile(16, 32, nb < 512 ? 256 : 128);
      break;
    }
  }
  g.panels = (N + g.BN - 1) / g.BN;
  g.blocks = max_row_tiles(M, experts, grouped, g.BM) * g.panels;
  return g;
}

template <bool kF32>
hipError_t launch_w8a8(const I8Args& a, hipStream_t st) {
  const W8a8Grid g = w8a8_grid(a.M, a.N, a.experts, a.offsets != nullptr);
  const unsigned blocks = (unsigned)g.blocks;
  const int panels = (int)g.panels;
  switch (g.kind) {
    case W8a8::kTile256:
      w8a8_tile_kernel<2, 4, 8, 1, kF32><<<blocks, 512, 0, st>>>(a, panels);
      break;
    case W8a8::kTile128:
      w8a8_tile_kernel<2, 2, 4, 2, kF32><<<blocks, 256, 0, st>>>(a, panels);
      break;
    case W8a8::kDeep128:
      w8a8_deep_kernel<2, 2, 4, 1, kF32><<<blocks, 256, 0, st>>>(a, panels);
      break;
    case W8a8::kDeep64x128:
      w8a8_deep_kernel<2, 2, 2, 1, kF32><<<blocks, 256, 0, st>>>(a, panels);
      break;
    case W8a8::kDeep64:
      w8a8_deep_kernel<2, 1, 2, 2, kF32><<<blocks, 256, 0, st>>>(a, panels);
      break;
    case W8a8::kStream32x64:
      w8a8_stream_kernel<2, 4, 4, false, kF32><<<blocks, 256, 0, st>>>(a);
      break;
    case W8a8::kStream16x64:
      w8a8_stream_kernel<1, 4, 4, false, kF32><<<blocks, 256, 0, st>>>(a);
      break;
    case W8a8::kRows16: {
      // Weights of 64 MiB or more are read past the caches, which is faster while each call has
      // other weights than the last one (one row, us through the caches and past them: 17408 x 5120
      // 20.4 and 18.2, 8192 x 8192 15.7 and 14.1).  Called again and again, a matrix that the
      // 256 MB last-level cache holds is often faster through it (28672 x 8192 35.1 and 37.7; 17408
      // x 5120 15.9 and 15.0, its 13 rows 17.8 and 18.3).  Below, the threshold leaves up to
      // a tenth to the caches: 8192 x 5120 10.5 and 9.5, again and again 8.0 and 7.7.
      const bool past = (int64_t)a.experts * a.N * a.K >= (int64_t)64 << 20;
      if (g.BN == 16) w8a8_stream_kernel<1, 1, 4, false, kF32><<<blocks, 256, 0, st>>>(a);
      else if (g.threads == 256 && past) w8a8_stream_kernel<1, 2, 4, true, kF32><<<blocks, 256, 0, st>>>(a);
      else if (g.threads == 256) w8a8_stream_kernel<1, 2, 4, false, kF32><<<blocks, 256, 0, st>>>(a);
      else if (past) w8a8_stream_kernel<1, 2, 2, true, kF32><<<blocks, 128, 0, st>>>(a);
      else w8a8_stream_kernel<1, 2, 2, false, kF32><<<blocks, 128, 0, st>>>(a);
      break;
    }
  }
  return hipGetLastError();
}

// A wavefront per row while four chunks per lane hold it, else 256 threads with up to
// 16 chunks each, else 1024.
template <bool kF32, bool kNative>
hipError_t launch_rows(const void* x, int64_t rows, int64_t K, int8_t* q, float* scale, hipStream_t st) {
  const int64_t padded = kNative ? (rows + kTileRows - 1) / kTileRows * kTileRows : rows;
  const int64_t chunks = K / (kF32 ? 4 : 8);
  // native: whole row blocks for each XCD in turn
  const int64_t all = kNative ? (padded / kTileRows + kXcds - 1) / kXcds * kXcds * kTileRows : rows;
  const unsigned n = (unsigned)all;
  const int r = (int)rows, p = (int)padded, k = (int)K;
  if (chunks <= 4 * 64)
    quantize_rows_kernel<kF32, kNative, 64, 4><<<(n + 3) / 4, 256, 0, st>>>(x, r, p, k, q, scale);
  else if (chunks <= 4 * 256)
    quantize_rows_kernel<kF32, kNative, 256, 4><<<n, 256, 0, st>>>(x, r, p, k, q, scale);
  else if (chunks <= 8 * 256)
    quantize_rows_kernel<kF32, kNative, 256, 8><<<n, 256, 0, st>>>(x, r, p, k, q, scale);
  else if (chunks <= 16 * 256)
    quantize_rows_kernel<kF32, kNative, 256, 16><<<n, 256, 0, st>>>(x, r, p, k, q, scale);
  else
    quantize_rows_kernel<kF32, kNative, 1024, 16><<<n, 1024, 0, st>>>(x, r, p, k, q, scale);
  return hipGetLastError();
}

// Launches of at most 2^31 threads, whole sets of row blocks each: 64 to 1024 threads a row.
template <bool kF32, bool kNative>
hipError_t launch_quantize_rows(const void* x, int64_t rows, int64_t K, int8_t* q, float* scale, hipStream_t st) {
  const int64_t chunks = K / (kF32 ? 4 : 8);
  const int64_t most = (kMaxThreads / 2) / (chunks <= 4 * 64 ? 64 : chunks <= 16 * 256 ? 256 : 1024);
  for (int64_t at = 0; at < rows; at += most) {
    const int64_t n = rows - at < most ? rows - at : most;
    const hipError_t e = launch_rows<kF32, kNative>(static_cast<const uint8_t*>(x) + at * K * (kF32 ? 4 : 2), n, K,
                                                    q + at * K, scale + at, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize_w8(const float* W, int64_t N, int64_t K, int8_t* q, float* d, hipStream_t stream) {
  return launch_quantize_rows<true, true>(W, N, K, q, d, stream);
}

hipError_t launch_quantize_tokens(const void* x, bool f32, int64_t M, int64_t K, int8_t* xq, float* sx,
                                  hipStream_t stream) {
  return f32 ? launch_quantize_rows<true, false>(x, M, K, xq, sx, stream)
             : launch_quantize_rows<false, false>(x, M, K, xq, sx, stream);
}

hipError_t launch_pack_w8(const int8_t* src, int64_t N, int64_t K, int8_t* dst, bool pack, hipStream_t stream) {
  // launches of at most 2^30 threads, whole row blocks each (16 rows x K codes / 16 a thread)
  const int64_t most = (kMaxThreads / 4) / K * kTileRows;
  for (int64_t at = 0; at < N; at += most) {
    const int64_t n = N - at < most ? N - at : most;
    const int64_t chunks = (n + kTileRows - 1) / kTileRows * K;
    const unsigned blocks = (unsigned)((chunks + 255) / 256);
    if (pack)
      repack_kernel<true><<<blocks, 256, 0, stream>>>(src + at * K, n, K, chunks, dst + at * K);
    else
      repack_kernel<false><<<blocks, 256, 0, stream>>>(src + at * K, n, K, chunks, dst + at * K);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

bool fits_linear_w8a8(int64_t M, int64_t N, int64_t experts, bool grouped) {
  const W8a8Grid g = w8a8_grid(M, N, experts, grouped);
  return g.blocks * g.threads < kMaxThreads;
}

hipError_t launch_linear_w8a8(const int8_t* xq, const float* sx, int64_t M, int64_t K, const int32_t* offsets,
                              int64_t experts, const int8_t* q, const float* d, int64_t N, void* y, bool f32,
                              hipStream_t stream) {
  const I8Args a{xq, sx, offsets, q, d, y, (int)M, (int)K, (int)N, (int)experts};
  return f32 ? launch_w8a8<true>(a, stream) : launch_w8a8<false>(a, stream);
}

}  // namespace w4
