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
//
// What bounds it (MI355X): 4096 x 151936 x 5120, 2920 to 3020 us, 2110 to 2180 TFLOP/s: 64 KB a step into each
// CU's LDS, which alone take 2240 us (18 bytes a clock, also where all of it hits the L2);
// products and LDS reads without them take 1990.  Through registers instead they alone take
// 1500, but the step as a whole is no faster for it (3050).  One row of 5120 x 4096, 6.8 to 7.1 us, and 16
// of 151936 x 5120, 138 to 148: reading w.
#include "dfs_device.h"
#include "dfs_internal.h"
#include "mfma_big.h"

#include <type_traits>

namespace dfs {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

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

// The 16 x 16 sums of one block of 128 k, from zero.  A lane holds 32 k of a row of w and of a.
//
// kExact false: V_MFMA_F32_16X16X128_F8F6F4 on the e4m3 values.  It aligns every eight products
// of neighbouring k to the largest of them and cuts each off at 2^-13 of it (measured, one value
// at a time), then adds as in fp32: at most 7 x 2^-13 of each eight's largest is lost, 2e-5 (2-norm,
// relative) of normally distributed data, which a bf16 output (2^-8) does not show and an fp32 one
// does.  Where large products cancel it is more than what is left, in either output.
// kExact true: the values widened to bf16 (exact) through V_MFMA_F32_16X16X32_BF16, whose
// sums are fp32 sums, at half the rate.
template <bool kExact>
struct Operand;
template <>
struct Operand<false> {
  i32x8 v;
  Operand() = default;
  __device__ __forceinline__ explicit Operand(const i32x8& x) : v(x) {}
};
template <>
struct Operand<true> {
  bf16x8 v[4];
  Operand() = default;
  __device__ __forceinline__ explicit Operand(const i32x8& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * i + j], 1.0f, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * i + j], 1.0f, true);
        v[i][4 * j] = lo.x, v[i][4 * j + 1] = lo.y, v[i][4 * j + 2] = hi.x, v[i][4 * j + 3] = hi.y;
      }
  }
};
__device__ __forceinline__ f32x4 block_mfma(const Operand<false>& w, const Operand<false>& a) {
  // both operands e4m3 (format 0), unit scales (exponent 127)
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                          0x7f7f7f7f);
}
__device__ __forceinline__ f32x4 block_mfma(const Operand<true>& w, const Operand<true>& a) {
  f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], a.v[i], t, 0, 0, 0);
  return t;
}
// acc += t sc
__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& t, float sc) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = fmaf(t[e], sc, acc[e]);
}

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  return f != f ? 0x7fc0u : (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// Rows of an output start at any multiple of a value, so vectors go out unaligned (2394 x 139762 x 416,
// bf16: 358 us, and 529 with single values wherever N was no multiple of 8).
typedef uint2 __attribute__((aligned(2))) uint2_any;
typedef uint4 __attribute__((aligned(2))) uint4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

// Four neighbouring columns n .. n + 3 of a row.
template <bool kBf16>
__device__ __forceinline__ void store4(void* out, int64_t row, int64_t N, int64_t n, f32x4 v) {
  if (n + 4 <= N) {
    if constexpr (kBf16)
      *reinterpret_cast<uint2_any*>(static_cast<uint16_t*>(out) + row * N + n) =
          make_uint2(bf16_bits(v.x) | (bf16_bits(v.y) << 16), bf16_bits(v.z) | (bf16_bits(v.w) << 16));
    else
      *reinterpret_cast<f32x4_any*>(static_cast<float*>(out) + row * N + n) = v;
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

// WN x WR waves, each TN x TR tiles of 16 columns (of w) x 16 rows (of a); KG such groups, each
// with a ring of S stages of its own, take the blocks of k in turn.
template <int WN_, int WR_, int TN_, int TR_, int S_, int KG_ = 1>
struct Tile {
  static constexpr int WN = WN_, WR = WR_, TN = TN_, TR = TR_, S = S_, KG = KG_;
  static constexpr int kWaves = WN * WR, kThreads = 64 * kWaves * KG;  // waves of a group
  static constexpr int BN = 16 * TN * WN, BR = 16 * TR * WR;
  static_assert(kBlock % (16 * TN) == 0, "a wave's columns share a scale");
  static constexpr int kScaleLoads = BR / 64;  // 64 rows' scales a load
  static_assert(BR % 64 == 0 && kWaves > kScaleLoads, "a wave for w's scales");
  static constexpr int kLoads = (BN + BR) / 8 / kWaves;  // 8 rows x 128 bytes a load
  static_assert((BN + BR) % (8 * kWaves) == 0, "loads");
  static constexpr int kPerStep = kLoads + 1;  // loads of a wave per step, the scales' among them
  static constexpr int kScales = (BN + BR) * kBlock;        // a's scales in a stage, w's after them
  static constexpr int kStage = kScales + 4 * BR + 256;
  static constexpr int kLds = KG * S * kStage;
  static_assert((KG - 1) * BN * BR * 4 <= kLds, "the groups' sums meet in the ring's LDS");
  static constexpr int kMinWaves = kWaves * KG / 4;  // per SIMD
};

__device__ __forceinline__ void dma4(big::rsrc_t rsrc, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(lds_base)
               : "memory", "m0");
}

constexpr uint32_t kPastEnd = 0x80000000u;  // an offset past every operand's range: reads zeros

// The loads of a tile's steps: w's rows, a's rows, both sides' scales.
template <class C>
struct Loader {
  const uint8_t *w, *a;   // the tile's first rows
  int nn, nr;             // rows that there are
  const float* scales;    // this wave's part of them at step 0, values to the next step, bytes
  int64_t scale_step;
  int scale_bytes;
  uint32_t scale_off, scale_dst;  // of this lane's, from there; in a stage
  int K, wave, lane;
  uint32_t off;           // of this lane's 16 bytes in eight rows of step 0
  int chunk;              // and its first k there

  __device__ __forceinline__ void init() {
    // eight rows from a multiple of eight on: the swizzle of row 8 j + x depends on j's parity,
    // which is the wave's
    static_assert(C::kWaves % 2 == 0, "a wave's loads share their swizzle");
    chunk = 16 * ((lane & 7) ^ (((8 * wave + (lane >> 3)) >> 1) & 7));
    off = (uint32_t)(lane >> 3) * (uint32_t)K + (uint32_t)chunk;
  }
  // Load i of step ks into `stage`; the last step's k past K, and rows past the end, read as zeros.
  __device__ __forceinline__ void one(uint32_t stage, int ks, int i) const {
    static_assert(C::BN / 8 % C::kWaves == 0, "a load is w's for all waves or a's");
    const int j = wave + C::kWaves * i;
    const bool isw = i < C::BN / 8 / C::kWaves;
    const int row = 8 * (isw ? j : j - C::BN / 8);
    const int left = max((isw ? nn : nr) - row, 0);
    int pitch = K;
    // formed anew every time where a wave has many: kept across steps, the resources of all
    // loads spill (with four the asm costs 3 to 6%)
    if constexpr (C::kLoads > 4) asm volatile("" : "+s"(pitch));
    const big::rsrc_t r = big::span_rsrc((isw ? w : a) + row * pitch, left * pitch);
    uint32_t voff = off + (uint32_t)ks * kBlock;
    if ((ks + 1) * kBlock > K && ks * kBlock + chunk >= K) voff = kPastEnd;
    big::dma16(r, voff, __builtin_amdgcn_readfirstlane(stage + j * 1024));
  }
  // Every wave issues one load of scales, so that all count the same: a's by 64 rows, w's
  // (lane b: of the tile's b-th 128 columns) by the others.  They go through LDS with the
  // operands: a load into a register under a condition, now and then, made every step wait
  // for all loads in flight.  No branch here, which would part the step's instructions.
  __device__ __forceinline__ void scale(uint32_t stage, int ks) const {
    dma4(big::span_rsrc(scales + (int64_t)ks * scale_step, scale_bytes), scale_off,
         __builtin_amdgcn_readfirstlane(stage + scale_dst));
  }
};

// This lane's 32 k of a block: chunks g and g + 4 of row r (any 32, if w and a take the same; these two
// keep the 16 lanes that LDS serves at a time, which come from two neighbouring g, on distinct banks).
__device__ __forceinline__ i32x8 read_frag(const char* rows16, int r, int g) {
  const int sw = (r >> 1) & 7;  // rows 16 apart keep the same swizzle
  const char* p = rows16 + r * kBlock;
  const int4 lo = *reinterpret_cast<const int4*>(p + 16 * (g ^ sw));
  const int4 hi = *reinterpret_cast<const int4*>(p + 16 * ((g + 4) ^ sw));
  return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

// Tile (row, column) of workgroup `id`.  Workgroups go round the eight XCDs in turn, each
// with an L2 of its own: an XCD takes a contiguous run of the tiles, in the order column
// groups of four, rows, columns of the group, so that the 32 that it runs at a time are
// about 8 rows x 4 columns of tiles and share what they read.
__device__ __forceinline__ int2 tile_of(uint32_t id, uint32_t count, int rtiles, int ntiles) {
  const uint32_t xcd = id & 7, each = count / 8, extra = count % 8;
  const uint32_t i = xcd * each + min(xcd, extra) + id / 8;
  const uint32_t group = i / (4 * rtiles), in = i % (4 * rtiles);
  const uint32_t width = min(4u, (uint32_t)ntiles - 4 * group);
  return make_int2(in / width, 4 * group + in % width);
}

template <class C, bool kBf16>
__global__ __launch_bounds__(C::kThreads, C::kMinWaves) void linear_q8_tile_kernel(LinearArgs p) {
  __shared__ __align__(1024) char lds[C::kLds];
  const int lane = threadIdx.x & 63;
  const int kg = uniform(threadIdx.x >> 6) / C::kWaves, wave = uniform(threadIdx.x >> 6) % C::kWaves;
  const int r = lane & 15, g = lane >> 4;
  const int wn = wave / C::WR, wr = wave % C::WR;
  const int2 at = tile_of(blockIdx.x, gridDim.x, (int)((p.rows + C::BR - 1) / C::BR), (int)((p.N + C::BN - 1) / C::BN));
  // 32-bit and uniform, so that addresses are formed by scalar instructions
  const int n0 = uniform(at.y) * C::BN, r0 = uniform(at.x) * C::BR;
  const int nn = min(C::BN, (int)p.N - n0), nr = min(C::BR, (int)p.rows - r0);
  Loader<C> in;
  in.w = p.w + (int64_t)n0 * p.K;
  in.a = p.a + (int64_t)r0 * p.K;
  in.nn = nn, in.nr = nr;
  if (wave < C::kScaleLoads) {
    in.scales = p.a_scale + r0;
    in.scale_step = p.rows;
    in.scale_bytes = nr * 4;
    in.scale_off = (64 * wave + lane) * 4;
    in.scale_dst = C::kScales + 256 * wave;
  } else {
    in.scales = p.w_scale + (int64_t)(n0 / kBlock) * p.G;
    in.scale_step = 1;
    in.scale_bytes = ((nn + kBlock - 1) / kBlock - 1) * p.G * 4 + 4;
    in.scale_off = lane * p.G * 4;
    in.scale_dst = C::kScales + 4 * C::BR;
  }
  in.K = p.K, in.wave = wave, in.lane = lane;
  in.init();
  f32x4 acc[C::TN][C::TR];
#pragma unroll
  for (int i = 0; i < C::TN; ++i)
#pragma unroll
    for (int j = 0; j < C::TR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int n = p.G, steps = (n + C::KG - 1) / C::KG;  // this group's: blocks kg, kg + KG, ...
  const char* ring = lds + kg * C::S * C::kStage;
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((big::lds_ptr_t)lds) + kg * C::S * C::kStage;
#pragma unroll
  for (int j = 0; j < C::S - 1; ++j) {
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) in.one(lds0 + j * C::kStage, min(j * C::KG + kg, n - 1), i);
    in.scale(lds0 + j * C::kStage, min(j * C::KG + kg, n - 1));
  }
  constexpr bool kExact = !kBf16;
  typedef Operand<kExact> Op;
  // Loads issued per column tile.  With two stages they are due at the step's end: twice as many, and
  // so all of them in its first half (4096 x 151936 x 5120: 3005 -> 2944 us; with more stages the
  // even spread is better, 192 x 5120 x 5120: 13.5 against 14.7).
  constexpr bool kSoon = C::S == 2;
  constexpr int kSpread = (kSoon ? 2 : 1) * ((C::kLoads + C::TN - 1) / C::TN);
  for (int ks = 0; ks < steps; ++ks) {
    big::wait_vmcnt<(C::S - 2) * C::kPerStep>();
    big::bar();
    if (C::KG > 1 && ks * C::KG + kg >= n) break;  // in the last step, which nothing follows
    const int nxt = min((ks + C::S - 1) * C::KG + kg, n - 1);  // past the end: the last block again
    const uint32_t fill = lds0 + (ks + C::S - 1) % C::S * C::kStage;
    const char* st = ring + (ks % C::S) * C::kStage;
    Op fa[C::TR];
    float sc[C::TR];
    // A column tile's products while the one before is added up, the next one's fragment is
    // read and a load or two of a later step go out, in exactly this order: the matrix
    // instructions then follow each other without waiting for any of it.
    Op fw[3];
    f32x4 t[2][C::TR];
    const char* wt = st + 16 * C::TN * wn * kBlock;
    fw[0] = Op(read_frag(wt, r, g));
    fw[1] = Op(read_frag(wt + 16 * kBlock, r, g));
#pragma unroll
    for (int j = 0; j < C::TR; ++j) {
      const int row = 16 * (C::TR * wr + j);
      fa[j] = Op(read_frag(st + (C::BN + row) * kBlock, r, g));
    }
#pragma unroll
    for (int j = 0; j < C::TR; ++j)
      sc[j] = *reinterpret_cast<const float*>(st + C::kScales + 4 * (16 * (C::TR * wr + j) + r));
    const float ws = *reinterpret_cast<const float*>(st + C::kScales + 4 * C::BR + 4 * (16 * C::TN * wn / kBlock));
#pragma unroll
    for (int i = 0; i < C::TN; ++i) {
#pragma unroll
      for (int j = 0; j < C::TR; ++j) {
        t[i & 1][j] = block_mfma(fw[i % 3], fa[j]);
        __builtin_amdgcn_sched_barrier(0);
        if (j == 0) {
          if (i + 2 < C::TN) fw[(i + 2) % 3] = Op(read_frag(wt + 16 * (i + 2) * kBlock, r, g));
#pragma unroll
          for (int x = i * kSpread; x < min((i + 1) * kSpread, C::kLoads); ++x) in.one(fill, nxt, x);
          if (i == (kSoon ? 0 : C::TN - 1)) in.scale(fill, nxt);
        }
        if (i == 0) sc[j] *= ws;
        if (i > 0) add_scaled(acc[i - 1][j], t[(i - 1) & 1][j], sc[j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int j = 0; j < C::TR; ++j) add_scaled(acc[C::TN - 1][j], t[(C::TN - 1) & 1][j], sc[j]);
  }
  big::wait_vmcnt<0>();
  big::bar();  // everyone is done with the ring
  if constexpr (C::KG > 1) {  // the groups' sums, in their order
    f32x4* sums = reinterpret_cast<f32x4*>(lds) + wave * C::TN * C::TR * 64 + lane;
    constexpr int kOne = C::kWaves * C::TN * C::TR * 64;
    if (kg > 0)
#pragma unroll
      for (int i = 0; i < C::TN; ++i)
#pragma unroll
        for (int j = 0; j < C::TR; ++j) sums[(kg - 1) * kOne + (i * C::TR + j) * 64] = acc[i][j];
    __syncthreads();
    if (kg == 0)
#pragma unroll
      for (int k = 1; k < C::KG; ++k)
#pragma unroll
        for (int i = 0; i < C::TN; ++i)
#pragma unroll
          for (int j = 0; j < C::TR; ++j) acc[i][j] += sums[(k - 1) * kOne + (i * C::TR + j) * 64];
    __syncthreads();
    if (kg > 0) return;
  }
  // A wave's tile goes out by way of LDS, 16 rows at a time, so that a row's columns leave as
  // one run (a lane holds 4 columns of a row: written from there they went out in 32-byte
  // pieces, which took 10% of the kernel at 4096 x 151936 x 5120).
  typedef typename std::conditional<kBf16, uint16_t, float>::type Out;
  constexpr int kCols = 16 * C::TN, kPitch = kCols + 16 / (int)sizeof(Out);
  static_assert(C::kWaves * 16 * kPitch * (int)sizeof(Out) <= C::kLds, "the tiles' LDS");
  Out* mine = reinterpret_cast<Out*>(lds) + wave * 16 * kPitch;
  const int col0 = n0 + kCols * wn, cols = min(kCols, (int)p.N - col0);
#pragma unroll
  for (int j = 0; j < C::TR; ++j) {
#pragma unroll
    for (int i = 0; i < C::TN; ++i) {
      Out* to = mine + r * kPitch + 16 * i + 4 * g;
      const f32x4 v = acc[i][j];
      if constexpr (kBf16)
        *reinterpret_cast<uint2*>(to) =
            make_uint2(bf16_bits(v.x) | (bf16_bits(v.y) << 16), bf16_bits(v.z) | (bf16_bits(v.w) << 16));
      else
        *reinterpret_cast<f32x4*>(to) = v;
    }
    const int row0 = r0 + 16 * (C::TR * wr + j), rows = min(16, (int)p.rows - row0);
    Out* out = static_cast<Out*>(p.out) + (int64_t)row0 * p.N + col0;
    constexpr int kVec = 16 / sizeof(Out), kPer = kCols / kVec;
#pragma unroll
    for (int u = lane; u < 16 * kPer; u += 64) {
      const int y = u / kPer, x = u % kPer * kVec;
      if (y < rows && x + kVec <= cols)
        *reinterpret_cast<uint4_any*>(out + y * p.N + x) = *reinterpret_cast<const uint4*>(mine + y * kPitch + x);
    }
    if (cols % kVec != 0 && cols < kCols) {  // the last columns, behind the last whole vector
      const int y = lane >> 2;
      for (int x = max(cols, 0) / kVec * kVec + (lane & 3); x < cols; x += 4)
        if (y < rows) out[y * p.N + x] = mine[y * kPitch + x];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before it is written again
  }
}

template <class C, bool kBf16>
hipError_t launch_tile(const LinearArgs& p, hipStream_t stream) {
  const dim3 grid((uint32_t)(cdiv(p.rows, C::BR) * cdiv(p.N, C::BN)));
  linear_q8_tile_kernel<C, kBf16><<<grid, dim3(C::kThreads), 0, stream>>>(p);
  return hipGetLastError();
}

using Big = Tile<2, 4, 8, 4, 2>;      // 256 x 256, one workgroup a CU
using Mid = Tile<2, 2, 4, 4, 2>;      // 128 x 128, two
using Tall = Tile<4, 2, 2, 2, 3>;     // 128 columns x 64 rows, two
using Small = Tile<2, 2, 2, 2, 3>;    // 64 x 64, three
using Pair = Tile<2, 2, 2, 2, 4, 2>;  // 64 x 64 by two groups of waves, one
using Wide = Tile<4, 1, 2, 4, 3>;     // 128 columns x 64 rows, two

// Few rows: the time is that of reading w once.  No LDS ring: a workgroup's eight waves
// take the blocks of k in turn, each reads NB blocks' fragments of w (16 rows x 128 bytes:
// whole cache lines) and of a (from the L2) straight into registers, all in flight at once,
// and the waves' sums are added through LDS in wave order at the end.  Straight-line code:
// a load under a condition makes the compiler wait for it where the paths join.
// 32 k of `row` from k on as two 16-byte loads; k past K - 16 reads the last 16 bytes.
__device__ __forceinline__ i32x8 load_frag(const uint8_t* row, int k, int K) {
  const int4 lo = *reinterpret_cast<const int4*>(row + min(k, K - 16));
  const int4 hi = *reinterpret_cast<const int4*>(row + min(k + 16, K - 16));
  return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

template <int RT, int MT, int NB, bool kBf16>
__global__ __launch_bounds__(512) void linear_q8_few_kernel(LinearArgs p) {
  constexpr int W = 8;
  __shared__ __attribute__((aligned(16))) f32x4 part[W][MT * RT][64];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * MT);
  const uint8_t* wrow[MT];
  const uint8_t* arow[RT];
  int64_t row[RT];
#pragma unroll
  for (int i = 0; i < MT; ++i) wrow[i] = p.w + min(n0 + 16 * i + r, p.N - 1) * p.K;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    row[j] = min((int64_t)(16 * j + r), p.rows - 1);
    arow[j] = p.a + row[j] * p.K;
  }
  const float* ws = p.w_scale + n0 / kBlock * p.G;
  f32x4 acc[MT][RT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kb0 = wave; kb0 < p.G; kb0 += W * NB) {
    i32x8 fw[NB][MT], fa[NB][RT];
    float sc[NB][RT], wsc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // k past K reads a row's own last 16 bytes; a's are then cleared, so that they count for
      // nothing (what is not finite in a row of w makes its column so anyway).  A block past the last
      // is all such k, and takes a scale of zero: the last block's may be infinite.
      const int kb = min(kb0 + W * b, p.G - 1), k = (kb0 + W * b) * kBlock + 32 * g;
#pragma unroll
      for (int i = 0; i < MT; ++i) fw[b][i] = load_frag(wrow[i], k, p.K);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        fa[b][j] = load_frag(arow[j], k, p.K);
        sc[b][j] = p.a_scale[(int64_t)kb * p.rows + row[j]];
      }
      wsc[b] = ws[kb];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int k = (kb0 + W * b) * kBlock + 32 * g;
      Operand<true> oa[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k + 16 * (e / 4) >= p.K) fa[b][j][e] = 0;
        oa[j] = Operand<true>(fa[b][j]);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const Operand<true> ow(fw[b][i]);
#pragma unroll
        for (int j = 0; j < RT; ++j)
          add_scaled(acc[i][j], block_mfma(ow, oa[j]), b == 0 || kb0 + W * b < p.G ? sc[b][j] * wsc[b] : 0.f);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) part[wave][i * RT + j][lane] = acc[i][j];
  __syncthreads();
  for (int t = wave; t < MT * RT; t += W) {
    f32x4 v = part[0][t][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][t][lane];
    const int i = t / RT, j = t % RT;
    if (16 * j + r < p.rows) store4<kBf16>(p.out, 16 * j + r, p.N, n0 + 16 * i + 4 * g, v);
  }
}

template <int RT, int MT, int NB, bool kBf16>
hipError_t launch_few(const LinearArgs& p, hipStream_t stream) {
  linear_q8_few_kernel<RT, MT, NB, kBf16><<<dim3((uint32_t)cdiv(p.N, 16 * MT)), dim3(512), 0, stream>>>(p);
  return hipGetLastError();
}

// Few rows and many columns: as above, but a workgroup stays for a run of column tiles (16
// columns each), a wave keeps its blocks' fragments of a in registers throughout, and the
// next tile's w is read while this one is multiplied.  (Reading a for every workgroup cost
// a third of the whole: 183 us against 140 at 16 x 151936 x 5120.)  The waves' sums of four
// tiles meet in LDS at a time, and leave as 256-byte runs.
template <int RT, int NB, bool kBf16>
__global__ __launch_bounds__(512, 2) void linear_q8_stream_kernel(LinearArgs p) {
  constexpr int W = 8, GT = 4;
  __shared__ __attribute__((aligned(16))) f32x4 part[2][GT][W][RT][64];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  // Workgroup b's tiles, in turn: 4 (b + i grid) .. + 3 for every whole round i of four tiles
  // each, then rest + b, rest + b + grid, ... of what is left (together the workgroups read
  // through w in address order: with a run of its own for each they took 153 us against 140).
  const int ntiles = (int)((p.N + 15) / 16), grid = gridDim.x, me = blockIdx.x;
  const int rounds = ntiles / (GT * grid), rest = rounds * GT * grid;
  const int left = ntiles - rest > me ? (ntiles - rest - me + grid - 1) / grid : 0;
  auto tile_at = [&](int i) {
    const int t = i < GT * rounds ? GT * (me + i / GT * grid) + i % GT : rest + me + (i - GT * rounds) * grid;
    return min(t, ntiles - 1);
  };
  i32x8 fa[NB][RT];
  float sa[NB][RT];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int kb = wave + W * b, k = kb * kBlock + 32 * g;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int64_t row = min((int64_t)(16 * j + r), p.rows - 1);
      fa[b][j] = load_frag(p.a + row * p.K, k, p.K);
      sa[b][j] = p.a_scale[(int64_t)min(kb, p.G - 1) * p.rows + row];
      if (kb >= p.G) sa[b][j] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + 16 * (e / 4) >= p.K) fa[b][j][e] = 0;  // k past K counts for nothing (see above)
    }
  }
  struct Columns {
    i32x8 w[NB];
    float scale;  // lane b: of block wave + W b
  };
  Columns c[2];
  auto load = [&](Columns& c, int i) {
    const int t = tile_at(i);
    const uint8_t* row = p.w + min((int64_t)t * 16 + r, p.N - 1) * p.K;
#pragma unroll
    for (int b = 0; b < NB; ++b) c.w[b] = load_frag(row, (wave + W * b) * kBlock + 32 * g, p.K);
    c.scale = p.w_scale[(int64_t)t * 16 / kBlock * p.G + min(wave + W * (lane & 7), p.G - 1)];
    __builtin_amdgcn_sched_barrier(0);
  };
  auto compute = [&](const Columns& c, f32x4 (&to)[W][RT][64]) {
    f32x4 acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float ws = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(c.scale), b));
      if (b == NB - 1 && wave + W * b >= p.G) ws = 0.f;  // only the last one may lie past the last block
      const Operand<true> fw(c.w[b]);
#pragma unroll
      for (int j = 0; j < RT; ++j) add_scaled(acc[j], block_mfma(fw, Operand<true>(fa[b][j])), sa[b][j] * ws);
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) to[wave][j][lane] = acc[j];
    __builtin_amdgcn_sched_barrier(0);
  };
  // The sums of four tiles (or the n last ones): a wave takes four rows, 16 lanes a row's 64 columns.
  auto reduce = [&](f32x4 (&from)[GT][W][RT][64], int i, int n) {
    big::bar();
    const int j = wave >> 2, row = 4 * (wave & 3) + (lane >> 4), u = (lane & 15) >> 2;
    if (j < RT && u < n) {
      const int src = 16 * (lane & 3) + row;
      f32x4 v = from[u][0][j][src];
#pragma unroll
      for (int w = 1; w < W; ++w) v += from[u][w][j][src];
      if (16 * j + row < p.rows)
        store4<kBf16>(p.out, 16 * j + row, p.N, (int64_t)tile_at(i + u) * 16 + 4 * (lane & 3), v);
    }
  };
  load(c[0], 0);
  int buf = 0;
  for (int i = 0; i < GT * rounds; i += GT, buf ^= 1) {
#pragma unroll
    for (int u = 0; u < GT; ++u) {
      load(c[(u + 1) & 1], i + u + 1);
      compute(c[u & 1], part[buf][u]);
    }
    reduce(part[buf], i, GT);
  }
  if (left == 0) return;
  const int i = GT * rounds;
  load(c[1], i + 1);
  compute(c[0], part[buf][0]);
  if (left > 1) {
    load(c[0], i + 2);
    compute(c[1], part[buf][1]);
    if (left > 2) {
      load(c[1], i + 3);
      compute(c[0], part[buf][2]);
      compute(c[1], part[buf][3]);
    }
  }
  reduce(part[buf], i, left);
}

template <int RT, bool kBf16>
hipError_t launch_stream(const LinearArgs& p, hipStream_t stream) {
  const dim3 grid(256), block(512);
  const int nb = (p.G + 7) / 8;  // blocks of k of a wave
  if (nb == 1) {
    linear_q8_stream_kernel<RT, 1, kBf16><<<grid, block, 0, stream>>>(p);
  } else if (nb == 2) {
    linear_q8_stream_kernel<RT, 2, kBf16><<<grid, block, 0, stream>>>(p);
  } else if (nb == 3) {
    linear_q8_stream_kernel<RT, 3, kBf16><<<grid, block, 0, stream>>>(p);
  } else if constexpr (RT == 1) {
    if (nb == 4)
      linear_q8_stream_kernel<RT, 4, kBf16><<<grid, block, 0, stream>>>(p);
    else
      linear_q8_stream_kernel<RT, 5, kBf16><<<grid, block, 0, stream>>>(p);
  }
  return hipGetLastError();
}

// Which kernel (times in us, bf16 output unless said, by rows x N x K):
//   up to 16 rows  the streaming kernel from 16384 columns on, up to K = 5120 (16 x 151936 x 5120,
//                  fp32: 138 against 175), else the one for few rows (1 x 5120 x 4096: 6.8 to 7.1)
//   up to 32 rows  the same, the streaming one up to 24 blocks of k (its fragments of a spill
//                  beyond; 32 x 5120 x 4096: 9.9 against 11.3 in tiles)
//   up to 64 rows  128 x 64 tiles from 16384 columns on (64 x 151936 x 5120: 153 against 177 in
//                  64 x 64), else as for more
//   more           256 x 256 tiles, one to a CU, or 128 x 128 from 300 on, two to a CU (1024 x 10240 x
//                  5120: 82 against 108 in 64 x 64, and 66 in 256 x 256), by their rounds: a round of the large ones
//                  takes 1600 / 1024 of a round of the others, whose last, if short, takes half of
//                  one and half of its share (4096 x 151936 x 5120: 2950 against 3590; 4096 x 4096 x
//                  4096: 69 against 85; 1024 x 65536 x 2048: 156 against 199; 2048 x 5120 x 5120, 640
//                  small ones: 77 against 78; 2560 x 8192 x 4096, 320 large ones: 121 against 109).
//                  Fewer: 64 x 64.  One for each CU or less, and two groups of waves take the blocks
//                  of k in turn (192 x 5120 x 5120: 13.3 against 16.6).  Two for each or less, and
//                  more than three, and one workgroup of eight waves takes two of them (333 x 5003 x
//                  2064: 11.7 against 12.8; 640 x 6000 x 4096, 940 tiles: 27.9 against 32.3; but 512 x 5120
//                  x 4096, 640 tiles: 26.4 against 23.3).  With an fp32 output (twice the matrix
//                  instructions) that is so beyond three only (333 x 5003 x 2064: 17.3 against 16.4),
//                  and the 256 x 256 tile spills: 128 x 128 takes its place.
template <bool kBf16>
hipError_t launch_linear(const LinearArgs& p, hipStream_t stream) {
  const bool columns = p.N >= 16384;
  if (p.rows <= 32) {
    if (columns && p.rows <= 16 && p.G <= 40) return launch_stream<1, kBf16>(p, stream);
    if (columns && p.rows > 16 && p.G <= 24) return launch_stream<2, kBf16>(p, stream);
    if (p.rows <= 16) return launch_few<1, 2, 2, kBf16>(p, stream);
    if (!columns) return launch_few<2, 2, 1, kBf16>(p, stream);
  }
  if (p.rows <= 64 && columns) return launch_tile<Wide, kBf16>(p, stream);
  const int64_t big = cdiv(p.rows, Big::BR) * cdiv(p.N, Big::BN), mid = cdiv(p.rows, Mid::BR) * cdiv(p.N, Mid::BN);
  if constexpr (kBf16)
    if (1600 * cdiv(big, 256) < 1024 * (mid / 512) + (mid % 512 ? 512 + mid % 512 : 0))
      return launch_tile<Big, kBf16>(p, stream);
  if (mid >= 300) return launch_tile<Mid, kBf16>(p, stream);
  const int64_t tiles = cdiv(p.rows, Small::BR) * cdiv(p.N, Small::BN);
  if (tiles <= 256) return launch_tile<Pair, kBf16>(p, stream);
  if ((kBf16 && tiles <= 512) || tiles > 768) return launch_tile<Tall, kBf16>(p, stream);
  return launch_tile<Small, kBf16>(p, stream);
}

}  // namespace

hipError_t launch_linear_q8(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale,
                            int64_t rows, int64_t N, int64_t K, bool bf16_out, void* out, hipStream_t stream) {
  const LinearArgs p{a, a_scale, w, w_scale, out, rows, N, (int)K, (int)cdiv(K, kBlock)};
  return bf16_out ? launch_linear<true>(p, stream) : launch_linear<false>(p, stream);
}

}  // namespace dfs
