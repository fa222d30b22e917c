// A product of 8-bit operands with a scale for each block of 128.
//
//   out[r, n] = sum_kb a_scale[kb, r] w_scale[n / 128, kb] sum_{k in block kb} a[r, k] w[n, k]
//
// a [rows, K] and w [N, K] e4m3, blocks of 128 k.  One V_MFMA_F32_16X16X128_F8F6F4 covers
// a block, so its 16 x 16 sums start from zero and are added to the running fp32 sums
// with one multiply-add per value by the block's scale: the scales cost no extra pass and
// no extra accumulator.  w is the matrix instruction's A operand and a its B operand, so a
// lane holds one row of a: the row's scale is one register, and its four values of a tile
// are neighbouring columns of the output.
//
// Tiled kernel: operands go from memory straight into LDS (one 128-k block per step, a
// ring of stages; mfma_big.h's loads and waits), 16-byte chunk c of a row's eight at slot
// c ^ ((row >> 1) & 7): the 16 rows that a fragment read touches then fall on distinct
// banks.  Rows and k past the end of an operand read as zeros.
#include "dfs_device.h"
#include "dfs_internal.h"
#include "mfma_big.h"

namespace dfs {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 128;  // k per scale and per step

struct LinearArgs {
  const uint8_t* a;
  const float* a_scale;  // [G, rows]
  const uint8_t* w;
  const float* w_scale;  // [ceil(N / 128), G]
  void* out;
  int64_t rows, N;
  int K, G;
};

// The 16 x 16 sums of one block of 128 k, from zero.
__device__ __forceinline__ f32x4 block_mfma(const i32x8& w, const i32x8& a) {
  // both operands e4m3 (format 0), unit scales (exponent 127)
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                          0x7f7f7f7f);
}

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  return f != f ? 0x7fc0u : (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// Four neighbouring columns n .. n + 3 of a row; `whole`: N is a multiple of 4.
template <bool kBf16>
__device__ __forceinline__ void store4(void* out, int64_t row, int64_t N, int64_t n, f32x4 v, bool whole) {
  if (whole) {
    if (n < N) {
      if constexpr (kBf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + row * N + n) =
            make_uint2(bf16_bits(v.x) | (bf16_bits(v.y) << 16), bf16_bits(v.z) | (bf16_bits(v.w) << 16));
      else
        *reinterpret_cast<f32x4*>(static_cast<float*>(out) + row * N + n) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) {
        if constexpr (kBf16)
          static_cast<uint16_t*>(out)[row * N + n + i] = (uint16_t)bf16_bits(v[i]);
        else
          static_cast<float*>(out)[row * N + n + i] = v[i];
      }
  }
}

// WN x WR waves, each TN x TR tiles of 16 columns (of w) x 16 rows (of a).
template <int WN_, int WR_, int TN_, int TR_, int S_>
struct Tile {
  static constexpr int WN = WN_, WR = WR_, TN = TN_, TR = TR_, S = S_;
  static constexpr int kWaves = WN * WR, kThreads = 64 * kWaves;
  static constexpr int BN = 16 * TN * WN, BR = 16 * TR * WR;
  static_assert(kBlock % (16 * TN) == 0, "a wave's columns share a scale");
  static constexpr int kScaleLoads = BR / 64;  // 64 rows' scales a load
  static_assert(BR % 64 == 0 && kWaves % kScaleLoads == 0, "scale loads");
  static constexpr int kLoads = (BN + BR) / 8 / kWaves;  // 8 rows x 128 bytes a load
  static_assert((BN + BR) % (8 * kWaves) == 0, "loads");
  static constexpr int kPerStep = kLoads + 1;  // loads of a wave per step, the scales' among them
  static constexpr int kStage = (BN + BR) * kBlock + 4 * BR;
  static constexpr int kLds = S * kStage;
};

__device__ __forceinline__ void dma4(big::rsrc_t rsrc, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(lds_base)
               : "memory", "m0");
}

constexpr uint32_t kPastEnd = 0x80000000u;  // an offset past every operand's range: reads zeros

// Step ks of the tile into `stage`: w's rows, a's rows, a's scales.
template <class C>
__device__ __forceinline__ void load_step(char* stage, big::rsrc_t w, big::rsrc_t a, const float* scales, int64_t rows,
                                          int64_t nr, int K, int ks, int wave, int lane) {
  const int rr = lane >> 3, slot = lane & 7;
#pragma unroll
  for (int i = 0; i < C::kLoads; ++i) {
    const int j = wave + C::kWaves * i;
    const bool isW = j < C::BN / 8;
    const int row = 8 * (isW ? j : j - C::BN / 8) + rr;
    const int k = ks * kBlock + 16 * (slot ^ ((row >> 1) & 7));
    const uint32_t voff = k < K ? (uint32_t)row * (uint32_t)K + (uint32_t)k : kPastEnd;
    const uint32_t dst = (uint32_t)reinterpret_cast<uintptr_t>((big::lds_ptr_t)(stage + j * 1024));
    big::dma16(isW ? w : a, voff, __builtin_amdgcn_readfirstlane(dst));
  }
  // every wave issues one scale load, so that all count the same loads; some repeat another's
  const int p = wave % C::kScaleLoads;
  const uint32_t dst =
      (uint32_t)reinterpret_cast<uintptr_t>((big::lds_ptr_t)(stage + (C::BN + C::BR) * kBlock + 256 * p));
  dma4(big::span_rsrc(scales + ks * rows, nr * 4), (uint32_t)(64 * p + lane) * 4, __builtin_amdgcn_readfirstlane(dst));
}

__device__ __forceinline__ i32x8 read_frag(const char* rows16, int r, int g) {
  const int sw = (r >> 1) & 7;  // rows 16 apart keep the same swizzle
  const char* p = rows16 + r * kBlock;
  const int4 lo = *reinterpret_cast<const int4*>(p + 16 * ((2 * g) ^ sw));
  const int4 hi = *reinterpret_cast<const int4*>(p + 16 * ((2 * g + 1) ^ sw));
  return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

template <class C, bool kBf16>
__global__ __launch_bounds__(C::kThreads) void linear_q8_tile_kernel(LinearArgs p) {
  __shared__ __align__(1024) char lds[C::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int wn = wave / C::WR, wr = wave % C::WR;
  const int rtiles = (int)((p.rows + C::BR - 1) / C::BR);
  const int64_t n0 = (int64_t)(blockIdx.x / rtiles) * C::BN, r0 = (int64_t)(blockIdx.x % rtiles) * C::BR;
  const int64_t nn = min((int64_t)C::BN, p.N - n0), nr = min((int64_t)C::BR, p.rows - r0);
  const big::rsrc_t w = big::span_rsrc(p.w + n0 * p.K, nn * p.K);
  const big::rsrc_t a = big::span_rsrc(p.a + r0 * p.K, nr * p.K);
  f32x4 acc[C::TN][C::TR];
#pragma unroll
  for (int i = 0; i < C::TN; ++i)
#pragma unroll
    for (int j = 0; j < C::TR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // this wave's scales of w, 64 blocks at a time, a lane each
  const int64_t wcol = n0 + 16 * C::TN * wn;
  const float* wsrow = p.w_scale + (min(wcol, p.N - 1) / kBlock) * p.G;
  float wsl = 0.f;
  const int n = p.G;
#pragma unroll
  for (int j = 0; j < C::S - 1; ++j)
    load_step<C>(lds + j * C::kStage, w, a, p.a_scale + r0, p.rows, nr, p.K, j < n ? j : n - 1, wave, lane);
  for (int ks = 0; ks < n; ++ks) {
    if ((ks & 63) == 0) wsl = wsrow[min(ks + lane, n - 1)];
    big::wait_vmcnt<(C::S - 2) * C::kPerStep>();
    big::bar();
    const int nxt = ks + C::S - 1;
    load_step<C>(lds + (nxt % C::S) * C::kStage, w, a, p.a_scale + r0, p.rows, nr, p.K, nxt < n ? nxt : n - 1, wave, lane);
    const char* st = lds + (ks % C::S) * C::kStage;
    const float ws = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wsl), ks & 63));
    i32x8 fa[C::TR];
    float sc[C::TR];
#pragma unroll
    for (int j = 0; j < C::TR; ++j) {
      const int row = 16 * (C::TR * wr + j);
      fa[j] = read_frag(st + (C::BN + row) * kBlock, r, g);
      sc[j] = *reinterpret_cast<const float*>(st + (C::BN + C::BR) * kBlock + 4 * (row + r)) * ws;
    }
#pragma unroll
    for (int i = 0; i < C::TN; ++i) {
      const i32x8 fw = read_frag(st + 16 * (C::TN * wn + i) * kBlock, r, g);
#pragma unroll
      for (int j = 0; j < C::TR; ++j) {
        const f32x4 t = block_mfma(fw, fa[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(t[e], sc[j], acc[i][j][e]);
      }
    }
  }
  big::wait_vmcnt<0>();
  const bool whole = (p.N & 3) == 0;
#pragma unroll
  for (int j = 0; j < C::TR; ++j) {
    const int64_t row = r0 + 16 * (C::TR * wr + j) + r;
    if (row >= p.rows) continue;
#pragma unroll
    for (int i = 0; i < C::TN; ++i) store4<kBf16>(p.out, row, p.N, wcol + 16 * i + 4 * g, acc[i][j], whole);
  }
}

template <class C, bool kBf16>
hipError_t launch_tile(const LinearArgs& p, hipStream_t stream) {
  const dim3 grid((uint32_t)(cdiv(p.rows, C::BR) * cdiv(p.N, C::BN)));
  linear_q8_tile_kernel<C, kBf16><<<grid, dim3(C::kThreads), 0, stream>>>(p);
  return hipGetLastError();
}

using Mid = Tile<2, 2, 4, 4, 2>;  // 128 x 128

}  // namespace

size_t linear_q8_workspace_bytes(int64_t rows, int64_t N, int64_t K) { return 0; }

hipError_t launch_linear_q8(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale,
                            int64_t rows, int64_t N, int64_t K, bool bf16_out, void* out, void* ws,
                            hipStream_t stream) {
  const LinearArgs p{a, a_scale, w, w_scale, out, rows, N, (int)K, (int)cdiv(K, kBlock)};
  return bf16_out ? launch_tile<Mid, true>(p, stream) : launch_tile<Mid, false>(p, stream);
}

}  // namespace dfs
