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

constexpr uint32_t kOob = 0x80000000u;  // buffer offsets from here on read zeros
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

template <bool S16>
__device__ __forceinline__ float load_scale(const void* d, int64_t i) {
  if constexpr (S16)
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(d)[i] << 16);
  else
    return static_cast<const float*>(d)[i];
}

// A block owns one 16-output row block and a tile of 16 rows of x; its NW
// wavefronts divide the groups.
template <int NW, bool S16, bool kF32>
__global__ __launch_bounds__(NW * 64) void grouped_stream_kernel(const GroupedArgs a) {
  const int nb = (a.N + kTileRows - 1) / kTileRows;
  const int t = blockIdx.x / nb, rb = blockIdx.x - t * nb;
  RowTile rt;
  if (!find_row_tile(a.offsets, a.experts, a.M, 16, t, rt)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, kb = lane >> 4;
  const int G = a.K / kGroup, Q = (G + 3) >> 2, GP = 4 * Q;
  const int g0 = (int)((int64_t)G * wave / NW), g1 = (int)((int64_t)G * (wave + 1) / NW);
  const uint4* q = reinterpret_cast<const uint4*>(a.q) + ((int64_t)rt.expert * nb + rb) * GP * kTileLanes + lane;
  const int64_t s0 = (((int64_t)rt.expert * nb + rb) * Q * kTileRows + nl) * 4;
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.x + (int64_t)rt.r0 * a.K, (uint32_t)(rt.r1 - rt.r0) * (uint32_t)a.K * 2u);
  const uint32_t xo = nl < rt.r1 - rt.r0 ? ((uint32_t)nl * a.K + 8u * kb) * 2u : kOob;
  const UnpackConsts uc = unpack_consts();
  const bf16x8 kneg = bitcast<bf16x8>(u32x4{kNeg15x2, kNeg15x2, kNeg15x2, kNeg15x2});

  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g = g0; g < g1; ++g) {
    const uint4 w = q[(int64_t)g * kTileLanes];
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    f32x4 c = f32x4{0.f, 0.f, 0.f, 0.f};
    bf16x8 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = bitcast<bf16x8>(bload<0>(rx, xo + (uint32_t)g * 256u + 64u * i));
      c = mfma16x16x32(x[i], kneg, c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b[4];
      unpack_word(words[i], b, uc);
      c = mfma16x16x32(x[i], bitcast<bf16x8>(u32x4{b[0], b[1], b[2], b[3]}), c);
    }
    const float d = load_scale<S16>(a.d, s0 + (int64_t)(g >> 2) * kTileRows * 4 + (g & 3));
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = fmaf(d, c[j], acc[j]);
  }

  __shared__ f32x4 red[NW][64];
  red[wave][lane] = acc;
  __syncthreads();
  const int n = rb * kTileRows + nl;
  if (wave != 0 || n >= a.N) return;
#pragma unroll
  for (int w = 1; w < NW; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += red[w][lane][j];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = rt.r0 + 4 * kb + j;
    if (m < rt.r1) store_out<kF32>(a, m, n, 16.0f * acc[j]);
  }
}

}  // namespace

hipError_t launch_linear_grouped(const uint16_t* x, int64_t M, int64_t K, const int32_t* offsets, int64_t experts,
                                 const uint8_t* q, const void* d, bool s16, int64_t N, void* y, bool f32,
                                 hipStream_t stream) {
  const GroupedArgs a{x, offsets, q, d, y, (int)M, (int)K, (int)N, (int)experts};
  const int64_t blocks = max_row_tiles(M, experts, true, 16) * ((N + kTileRows - 1) / kTileRows);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const unsigned nblk = (unsigned)blocks;
  if (s16 && f32) grouped_stream_kernel<4, true, true><<<nblk, 256, 0, stream>>>(a);
  else if (s16) grouped_stream_kernel<4, true, false><<<nblk, 256, 0, stream>>>(a);
  else if (f32) grouped_stream_kernel<4, false, true><<<nblk, 256, 0, stream>>>(a);
  else grouped_stream_kernel<4, false, false><<<nblk, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace w4
