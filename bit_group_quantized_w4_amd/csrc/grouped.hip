// Rows sorted by expert times each expert's 4-bit group-quantized weight:
//
//   y[m][n] = sum_g d_e[n][g] sum_{k in g} q_e[n][k] x[m][k],
//
// e the expert whose range of `offsets` holds row m.  Codes and scales of every
// expert are in the native layout of the dense linear; partial sums of a group
// are formed from the exact codes in bf16 MFMA with fp32 accumulation and scaled
// by the group's d in fp32, as there.
//
// A nibble u = q + 8 is widened to bf16 1 + u/16 = 1.5 + q/16 (unpack_word); a
// group's partial starts from -1.5 * (sum of its x), so that it ends as
// sum(q x) / 16; the factor 16 is applied with the output.
#include "w4_device.h"
#include "w4_launch.h"
#include "w4_rows.h"

namespace w4 {
namespace {

// Added to the offset of an operand of a group past the last one: one expert's codes, its
// scales, and one tile's rows of x take less than 2 GiB each, so an offset inside its
// buffer ends outside it and reads zeros without touching memory, and so does that of a row
// of x that the tile does not have (below 2^28).  Only a row block past the expert's last
// one, of codes within 128 MiB of 2 GiB, can end inside the buffer again (the sum wraps): it
// reads codes of this expert, they meet zeros of x, and the outputs are past N, which no
// kernel stores.
constexpr uint32_t kOob = 0x80000000u;
constexpr uint32_t kNeg15x2 = 0xBFC0BFC0u;  // bf16 -1.5 in both halves

struct GroupedArgs {
  const uint16_t* x;
  const int* offsets;
  const uint8_t* q;
  const void* d;
  void* y;
  int M, K, N, experts;
};

template <bool kF32>
__device__ __forceinline__ void store_out(const GroupedArgs& a, int m, int n, float v) {
  const int64_t i = (int64_t)m * a.N + n;
  if constexpr (kF32)
    static_cast<float*>(a.y)[i] = v;
  else
    static_cast<uint16_t*>(a.y)[i] = f32_to_bf16_rne(v);
}

__device__ __forceinline__ f32x4 mfma16x16x32(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Streaming form, for experts with few rows: a block owns R row blocks of 16
// outputs and a tile of 16 rows of x; its NW wavefronts divide the groups.  Each
// wavefront keeps D groups of codes, scales and x in flight, straight from memory;
// a group past its last reads zeros (see kOob), so that every load is unconditional.
// Codes are read through the caches, since an expert with more than 16 rows is read by
// several blocks.  Bound by the latency of a few dependent loads (offsets, then codes):
// 16 rows of 64 experts of 2048 x 2560, 9.7 us for 44.7 MB (4.6 TB/s) in a run of calls,
// 10.9 us as graph nodes; three or four groups in flight, and past the caches, took 12.7
// and 14.0 us there.
template <int R, int NW, bool S16, bool kF32>
__global__ __launch_bounds__(NW * 64) void grouped_stream_kernel(const GroupedArgs a) {
  constexpr int D = 2;
  const int nb = (a.N + kTileRows - 1) / kTileRows, panels = (nb + R - 1) / R;
  const int t = blockIdx.x / panels, rb0 = (blockIdx.x - t * panels) * R;
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, 16, t, rt)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, kb = lane >> 4;
  const int G = a.K / kGroup, Q = (G + 3) >> 2, GP = 4 * Q;
  const int g0 = (int)((int64_t)G * wave / NW), g1 = (int)((int64_t)G * (wave + 1) / NW);
  constexpr uint32_t kScale = S16 ? 2u : 4u;
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.x + (int64_t)rt.r0 * a.K, (uint32_t)(rt.r1 - rt.r0) * (uint32_t)a.K * 2u);
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.q + (int64_t)rt.expert * nb * GP * 1024, (uint32_t)nb * GP * 1024u);
  const __amdgpu_buffer_rsrc_t rd = make_rsrc(static_cast<const uint8_t*>(a.d) + (int64_t)rt.expert * nb * GP * 16 * kScale,
                                              (uint32_t)nb * GP * 16u * kScale);
  // (row blocks past the last one lie outside the buffers, as rows of x past the tile's last do)
  const uint32_t xo = ((uint32_t)nl * a.K + 8u * kb) * 2u, qo = (uint32_t)rb0 * GP * 1024u + 16u * lane,
                 so = ((uint32_t)rb0 * Q * 16u + nl) * 4u * kScale;
  uint4 x[D][4], w[D][R];
  uint32_t d[D][R];
  auto issue = [&](int c, int g) {
    const bool in = g < g1;
    const uint32_t kx = in ? (uint32_t)g * 256u : kOob, kq = in ? (uint32_t)g * 1024u : kOob;
    const uint32_t kd = in ? ((uint32_t)(g >> 2) * 64u + (uint32_t)(g & 3)) * kScale : kOob;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[c][r] = bload<0>(rq, qo + (uint32_t)(r * GP) * 1024u + kq);
      const int o = (int)(so + (uint32_t)(r * Q) * 64u * kScale + kd);
      if constexpr (S16)
        d[c][r] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rd, o, 0, 0);
      else
        d[c][r] = __builtin_amdgcn_raw_buffer_load_b32(rd, o, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[c][i] = bload<0>(rx, xo + 64u * i + kx);
  };
  const UnpackConsts uc = unpack_consts();
  const bf16x8 kneg = bitcast<bf16x8>(u32x4{kNeg15x2, kNeg15x2, kNeg15x2, kNeg15x2});

  f32x4 acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < D; ++c) {
    issue(c, g0 + c);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int g = g0; g < g1; g += D) {
#pragma unroll
    for (int c = 0; c < D; ++c) {
      f32x4 off = f32x4{0.f, 0.f, 0.f, 0.f}, v[R];
      float dr[R];
#pragma unroll
      for (int i = 0; i < 4; ++i) off = mfma16x16x32(bitcast<bf16x8>(x[c][i]), kneg, off);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v[r] = off;
        dr[r] = __uint_as_float(S16 ? d[c][r] << 16 : d[c][r]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t word = i == 0 ? w[c][r].x : i == 1 ? w[c][r].y : i == 2 ? w[c][r].z : w[c][r].w;
          uint32_t b[4];
          unpack_word(word, b, uc);
          v[r] = mfma16x16x32(bitcast<bf16x8>(x[c][i]), bitcast<bf16x8>(u32x4{b[0], b[1], b[2], b[3]}), v[r]);
        }
      issue(c, g + c + D);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = fmaf(dr[r], v[r][e], acc[r][e]);
    }
  }

  __shared__ f32x4 red[NW][R][64];
#pragma unroll
  for (int r = 0; r < R; ++r) red[wave][r][lane] = acc[r];
  __syncthreads();
  for (int r = wave; r < R; r += NW) {
    const int n = (rb0 + r) * kTileRows + nl;
    if (n >= a.N) continue;
    f32x4 v = red[0][r][lane];
#pragma unroll
    for (int u = 1; u < NW; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += red[u][r][lane][e];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = rt.r0 + 4 * kb + e;
      if (m < rt.r1) store_out<kF32>(a, m, n, 16.0f * v[e]);
    }
  }
}

// Tile form, for experts with many rows: a block of WM x WN wavefronts owns
// BM = 16 WM TM rows of x and BN = 64 WN outputs, each wavefront TM x 4 tiles of
// 16 x 16 outputs.  A step is one group of 128 inputs.
//
// x goes to LDS straight from memory, two steps ahead, in three buffers.  Lane l of
// a load takes row l / 16 of four and its 16-byte chunk (l % 16) ^ (row % 16), so
// that the sixteen rows of an operand are read without bank conflicts.  Codes go
// straight to registers (each is used by one of the block's wavefronts) and are widened
// there.
//
// The partial sums of a group start from -1.5 * (sum of its x), which depends on the
// row alone: each wavefront forms it for one row tile of the block with four MFMAs
// against a constant operand, a step ahead, and shares it through LDS; the first
// MFMA of every chain takes it as its third operand.  Per step and wavefront that is
// 4 MFMAs beside 16 TM.
//
// The four output tiles j of a step follow each other; beside the products of one
// run the scaled accumulation of the one before, the widening of the next one's
// codes and the loads.  The barrier of a step stands before the last tile's products
// of the group before: beside these the operands of the new group are read.
//
// 8190 rows of eight experts, 9216 x 2560: 381 to 390 us (1000 TFLOP/s at 1.94 GHz; up to
// 425 us where the power limit lowers the clock further).  Bound by the issue of vector
// instructions: beside each MFMA there are 3.3 (1.65 widen codes, 0.94 accumulate, the rest
// are addresses and loads), four cycles each, and the matrix units, sixteen cycles an
// MFMA, are busy in 62% of the cycles that a CU has work.  64 rows per block (two blocks of four wavefronts per CU, whose
// barriers do not wait for each other) beat 128 rows in one block of eight (437 us).
//
// Steps past the last group (there are up to two, for the three buffers) read zeros (see
// kOob).
template <int WM, int WN, int TM, bool S16, bool kF32>
__global__ __launch_bounds__(WM* WN * 64, 2) void grouped_tile_kernel(const GroupedArgs a, int panels) {
  constexpr int TN = 4, NW = WM * WN, BM = 16 * WM * TM, BN = 16 * WN * TN;
  constexpr int LA = BM / 4 / NW;  // 1 KiB loads of x per wavefront and step
  static_assert(LA * NW * 4 == BM && LA <= 4 && 4 % LA == 0, "loads of x shared out evenly, within 16 rows");
  __shared__ __attribute__((aligned(1024))) uint8_t x0[BM * 256], x1[BM * 256], x2[BM * 256];
  __shared__ __attribute__((aligned(1024))) float off0[BM], off1[BM], off2[BM];

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
  const int K = a.K, G = K / kGroup, Q = (G + 3) >> 2, GP = 4 * Q;
  const int nb = (a.N + kTileRows - 1) / kTileRows, rb0 = p * (BN / 16) + wn * TN;
  const int rows = rt.r1 - rt.r0;

  constexpr uint32_t kScale = S16 ? 2u : 4u;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (int64_t)rt.r0 * K, (uint32_t)rows * (uint32_t)K * 2u);
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.q + (int64_t)rt.expert * nb * GP * 1024, (uint32_t)nb * GP * 1024u);
  const __amdgpu_buffer_rsrc_t rd = make_rsrc(static_cast<const uint8_t*>(a.d) + (int64_t)rt.expert * nb * GP * 16 * kScale,
                                              (uint32_t)nb * GP * 16u * kScale);
  uint32_t xo = (uint32_t)(4 * wave * LA + kb) * (uint32_t)K * 2u + 16u * (nl ^ ((4 * wave * LA + kb) & 15));
  const uint32_t qo = (uint32_t)rb0 * GP * 1024u + 16u * lane;
  const uint32_t so = ((uint32_t)rb0 * Q * 16u + nl) * 4u * kScale;
  typedef __attribute__((address_space(3))) void* lds_ptr;
  auto load_x = [&](int i, int g, uint8_t* to) {
    // rows 4 (wave LA + i) ..: 4 i of them further than xo, chunks exchanged by the same 4 i
    const uint32_t k = g < G ? (uint32_t)g * 256u : kOob;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr)(to + (wave * LA + i) * 1024), 16,
                                             (int)((xo ^ (64u * i)) + (uint32_t)(8 * i * K) + k), 0, 0, 0);
  };
  uint4 w[TN];
  uint32_t word3 = 0;  // the last word of tile 3, widened after its registers are loaded anew
  float d[TN];      // scales of the group in work
  uint32_t dn[TN];  // of the next, as loaded
  auto load_w = [&](int j, int g) {
    const uint32_t k = g < G ? (uint32_t)g * 1024u : kOob;
    w[j] = bload<0>(rq, qo + (uint32_t)(j * GP) * 1024u + k);
  };
  auto load_d = [&](int j, int g) {
    const uint32_t k = g < G ? ((uint32_t)(g >> 2) * 64u + (uint32_t)(g & 3)) * kScale : kOob;
    const int o = (int)(so + (uint32_t)(j * Q) * 64u * kScale + k);
    if constexpr (S16)
      dn[j] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rd, o, 0, 0);
    else
      dn[j] = __builtin_amdgcn_raw_buffer_load_b32(rd, o, 0, 0);
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  bf16x8 x[TM][4], b[4];
  f32x4 off[TM], c[2][TM];
  uint32_t xa = (uint32_t)(wm * TM * 16 + nl) * 256u + 16u * (kb ^ nl);
  const UnpackConsts uc = unpack_consts();
  const bf16x8 kneg = bitcast<bf16x8>(u32x4{kNeg15x2, kNeg15x2, kNeg15x2, kNeg15x2});

  auto read_x = [&](int i, const uint8_t* from) {  // the four inputs-octets of 32-input step i
#pragma unroll
    for (int m = 0; m < TM; ++m) x[m][i] = *reinterpret_cast<const bf16x8*>(from + (xa ^ (64u * i)) + m * 4096);
  };
  // Word i of a tile's codes as its four pairs of bf16, pair q at a time.
  auto widen = [&](int i, uint32_t word, int q) {
    u32x4 v = bitcast<u32x4>(b[i]);
    v[q] = ((q == 0 ? word : rotr32(word, 4 * q)) & uc.mask) | uc.magic;
    b[i] = bitcast<bf16x8>(v);
  };
  auto word_of = [&](int i, int j) { return i == 0 ? w[j].x : i == 1 ? w[j].y : i == 2 ? w[j].z : w[j].w; };
  // 32-input step i of an output tile's products into buffer s.  An MFMA occupies
  // the matrix unit for as long as four vector instructions take: after each come
  // its share of row tile i's accumulation acc += da c for the tile before (ja, in the
  // other buffer) and of the widening of one word into b[(i + 3) & 3], whose last
  // use the step before was.
  auto multiply = [&](int s, int i, int ja, float da, uint32_t word) {
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      c[s][m] = mfma16x16x32(x[m][i], b[i], i == 0 ? off[m] : c[s][m]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = m * 4 / TM; e < (m + 1) * 4 / TM; ++e) {
        if (i < TM) acc[i][ja][e] = fmaf(da, c[s ^ 1][i][e], acc[i][ja][e]);
        widen((i + 3) & 3, word, e);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // -1.5 * sum of x over the group in `from`, for one row tile of the block
  const uint32_t tile = (uint32_t)(wm * TM + wn % TM);
  bf16x8 xt[4];
  auto read_tile = [&](const uint8_t* from) {
#pragma unroll
    for (int i = 0; i < 4; ++i) xt[i] = *reinterpret_cast<const bf16x8*>(from + ((xa ^ (64u * i)) + (uint32_t)(wn % TM) * 4096u));
  };
  auto write_off = [&](float* to) {
    f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) v = mfma16x16x32(xt[i], kneg, v);
    // every column holds the same sums: lanes of one quarter write the same bytes
    *reinterpret_cast<f32x4*>(to + tile * 16u + 4u * kb) = v;
  };
  auto read_off = [&](const float* from) {
#pragma unroll
    for (int m = 0; m < TM; ++m) off[m] = *reinterpret_cast<const f32x4*>(from + (wm * TM + m) * 16 + 4 * kb);
  };
#define W4_FENCE __builtin_amdgcn_sched_barrier(0)
  // Group g: x in `cur`, its start values in `ocur`; the next group's x in `nxt`,
  // its start values go to `onxt`; the one after that is loaded into `far`.
  auto step = [&](int g, const uint8_t* cur, const uint8_t* nxt, uint8_t* far, const float* ocur, float* onxt) {
    asm volatile("" ::: "memory");
    // the x of the next group has landed: only the 2 TN loads of codes and scales
    // issued after it may be outstanding
    __builtin_amdgcn_s_waitcnt(0x0070 | (2 * TN));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // the addresses derived from these are cheaper formed anew than kept (256 VGPRs)
    asm volatile("" : "+v"(xa), "+v"(xo));
    W4_FENCE;
    // last output tile of the group before
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      multiply(1, i, 2, d[2], i == 0 ? word3 : word_of(i - 1, 0));
      read_x(i, cur);
#pragma unroll
      for (int l = i * LA / 4; l < (i + 1) * LA / 4; ++l) load_x(l, g + 2, far);
      W4_FENCE;
    }
    read_off(ocur);
    const float d3 = d[3];
#pragma unroll
    for (int j = 0; j < TN; ++j) d[j] = __uint_as_float(S16 ? dn[j] << 16 : dn[j]);
    W4_FENCE;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        multiply(j & 1, i, (j + 3) & 3, j == 0 ? d3 : d[j - 1], i == 0 ? word_of(3, j) : word_of(i - 1, j + 1));
        if (j == 0) load_d(i, g + 1);
        if (i == 1) load_w(j, g + 1);  // its last word was widened beside step 0
        if (i == 0 && j == 1) read_tile(nxt);
        if (i == 1 && j == 2) write_off(onxt);
        W4_FENCE;
      }
    }
    word3 = w[3].w;
    load_w(3, g + 1);
    W4_FENCE;
  };

  // before the first group: products of zeros stand in for the group before it
#pragma unroll
  for (int i = 0; i < LA; ++i) load_x(i, 0, x0);
#pragma unroll
  for (int i = 0; i < LA; ++i) load_x(i, 1, x1);
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    load_w(j, 0);
    load_d(j, 0);
    d[j] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[i] = bitcast<bf16x8>(u32x4{0, 0, 0, 0});
#pragma unroll
    for (int m = 0; m < TM; ++m) x[m][i] = bitcast<bf16x8>(u32x4{0, 0, 0, 0});
  }
#pragma unroll
  for (int m = 0; m < TM; ++m) off[m] = c[0][m] = c[1][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  read_tile(x0);
  write_off(off0);
  for (int g = 0; g < G; g += 3) {
    step(g, x0, x1, x2, off0, off1);
    step(g + 1, x1, x2, x0, off1, off2);
    step(g + 2, x2, x0, x1, off2, off0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) multiply(1, i, 2, d[2], word3);  // (only step 3's word is still to be widened)
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[m][3][e] = fmaf(d[3], c[1][m][e], acc[m][3][e]);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load into LDS outlives the block
#undef W4_FENCE

  // Stores past the tile's last row or the matrix's last output lie outside the
  // buffer and are dropped.  (Codes below 2 GiB keep N below 2^23, and the 64 rows of
  // y below 2 GiB.)
  static_assert(BM <= 64, "offsets into the rows of y below kOob");
  constexpr uint32_t kOut = kF32 ? 4u : 2u;
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(static_cast<uint8_t*>(a.y) + (int64_t)rt.r0 * a.N * kOut,
                                              (uint32_t)rows * (uint32_t)a.N * kOut);
  const uint32_t pitch = (uint32_t)a.N * kOut;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = (rb0 + j) * kTileRows + nl;
    const uint32_t at = n < a.N ? (uint32_t)(16 * wm * TM + 4 * kb) * pitch + (uint32_t)n * kOut : kOob;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint32_t o = at + (uint32_t)(16 * m + e) * pitch;
        const float v0 = 16.0f * acc[m][j][e], v1 = 16.0f * acc[m][j][e + 1];
        if constexpr (kF32) {
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v0), ry, (int)o, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v1), ry, (int)(o + pitch), 0, 0);
        } else {
          const uint32_t v = f32x2_to_bf16x2(v0, v1);
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)v, ry, (int)o, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v >> 16), ry, (int)(o + pitch), 0, 0);
        }
      }
  }
}

// The kernel goes by the average rows of an expert that has any (the true sizes are on
// the GPU).  Up to 8 the weight stream is all there is to do: four row blocks per
// wavefront once they leave 640 blocks or more, else two (32 rows of 64 experts of
// 1408 x 2560: 15.6 us either way; 64 rows of eight of 9216 x 2560: 26.5 against 28.9;
// 16 rows of eight of 2560 x 9216: two, 26.6 against 36).  Up to 64, tiles of 32 rows
// (256 rows of 16 experts of 5120 x 2560: 34.8 us, 38.0 streamed, 43.3 as 64 rows; 4096
// rows of 64 of 1408 x 2560: 71.4 and 81.3); beyond, 64 rows (1024 rows of eight of
// 9216 x 2560: 75.6 us, 86.0 as 32 rows).
struct GroupedGrid {
  int BM, threads;
  bool four;
  int64_t panels, blocks;
};

GroupedGrid grouped_grid(int64_t M, int64_t N, int64_t experts) {
  const int64_t busy = experts < M ? experts : M, rows = (M + busy - 1) / busy;
  const int64_t nb = (N + kTileRows - 1) / kTileRows;
  GroupedGrid g;
  g.four = busy * nb >= 2560;
  g.BM = rows <= 8 ? 16 : rows <= 64 ? 32 : 64;
  g.threads = rows > 8 ? 256 : 128;
  const int BN = rows > 8 ? 256 : g.four ? 64 : 32;
  g.panels = (N + BN - 1) / BN;
  g.blocks = max_row_tiles(M, experts, true, g.BM) * g.panels;
  return g;
}

template <bool S16, bool kF32>
hipError_t launch_grouped(const GroupedArgs& a, hipStream_t st) {
  const GroupedGrid g = grouped_grid(a.M, a.N, a.experts);
  const unsigned n = (unsigned)g.blocks;
  if (g.BM == 64) grouped_tile_kernel<1, 4, 4, S16, kF32><<<n, 256, 0, st>>>(a, (int)g.panels);
  else if (g.BM == 32) grouped_tile_kernel<1, 4, 2, S16, kF32><<<n, 256, 0, st>>>(a, (int)g.panels);
  else if (g.four) grouped_stream_kernel<4, 2, S16, kF32><<<n, 128, 0, st>>>(a);
  else grouped_stream_kernel<2, 2, S16, kF32><<<n, 128, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

bool fits_linear_grouped(int64_t M, int64_t N, int64_t experts) {
  const GroupedGrid g = grouped_grid(M, N, experts);
  return g.blocks * g.threads < kMaxThreads;
}

hipError_t launch_linear_grouped(const uint16_t* x, int64_t M, int64_t K, const int32_t* offsets, int64_t experts,
                                 const uint8_t* q, const void* d, bool s16, int64_t N, void* y, bool f32,
                                 hipStream_t stream) {
  const GroupedArgs a{x, offsets, q, d, y, (int)M, (int)K, (int)N, (int)experts};
  const int kind = (s16 ? 2 : 0) | (f32 ? 1 : 0);
  return kind == 0   ? launch_grouped<false, false>(a, stream)
         : kind == 1 ? launch_grouped<false, true>(a, stream)
         : kind == 2 ? launch_grouped<true, false>(a, stream)
                     : launch_grouped<true, true>(a, stream);
}

}  // namespace w4
