// Root-mean-square norm with the residual's addition and an 8-bit output.
//
//   s = x + residual,  y_c = s_c w_c / sqrt(sum_c s_c^2 / d + eps),
//   for each group of 128 columns  scale = max(max|y| / 448, 2^-100),  q_c = e4m3(y_c / scale).
//
// One pass over the data: a row is read once into registers (8 values per lane per step),
// the sum of squares is reduced over its waves, and a group's 128 values are 16
// neighbouring lanes, so its largest value is four DPP steps.  Bound by memory: 16320 x 5120 bf16
// with a residual, 112 us, 5.3 TB/s; 16 rows, 4.7 us on the device.  s stays in fp32 from the
// addition to the quantisation: the rounded sum that later layers read (out_total) is not
// what is normalised.
//
// The quotient.  1 / sqrt(...) is common to a group, so y / scale = 448 s w / max|s w|: taken in
// 64 bits, where s w is exact, and rounded to fp32 and from there to e4m3, as a quotient of 64
// bits is converted.  In fp32 its four or five roundings moved a few of a million values, those
// that lie next to the border of two e4m3 steps, to the other step.
#include "dfs_device.h"
#include "dfs_internal.h"

namespace dfs {
namespace {

constexpr int kVec = 8;                // values per lane per step
constexpr int kStep = kVec * kWave;    // columns a wave covers per step
constexpr float kE4m3Max = 448.0f;     // largest finite e4m3 value

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  uint8_t* q;
  float* scale;
  void* total;
  void* normed;
  int64_t rows;
  int d;
  float eps;
};

template <bool kBf16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[kVec]) {
  if constexpr (kBf16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool kBf16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[kVec]) {
  if constexpr (kBf16) {
    f32x8 f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) f[j] = v[j];
    *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(p) + i) = __builtin_convertvector(f, bf16x8);  // to nearest, ties to even
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The largest of 16 neighbouring lanes, in each of them (DPP row rotations).
__device__ __forceinline__ uint32_t row16_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xF, 0xF, false));  // row_ror:8
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x124, 0xF, 0xF, false));  // row_ror:4
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x122, 0xF, 0xF, false));  // row_ror:2
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x121, 0xF, 0xF, false));  // row_ror:1
  return x;
}

// The same of doubles that are not negative: they compare as whole numbers.
template <int kCtrl>
__device__ __forceinline__ double max_ror(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, kCtrl, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), kCtrl, 0xF, 0xF, false);
  return fmax(x, __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double row16_max(double x) {
  return max_ror<0x121>(max_ror<0x122>(max_ror<0x124>(max_ror<0x128>(x))));
}

__device__ __forceinline__ float wave_sum(float v, int lane) {
#pragma unroll
  for (int j = 32; j > 0; j >>= 1) v += __uint_as_float(xor_lanes(__float_as_uint(v), j, lane));
  return v;
}

// A row by kWaves waves, NV steps each; kWaves == 1: four rows per workgroup, one per wave.
template <bool kBf16, bool kRes, int NV, int kWaves>
__global__ __launch_bounds__(kWaves == 1 ? 4 * kWave : kWaves* kWave) void norm_q8_kernel(NormArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = kWaves == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  if (kWaves == 1 && row >= a.rows) return;
  const int part = kWaves == 1 ? 0 : wave;
  const int64_t base = row * a.d;
  float s[NV][kVec];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * kWaves + part) * kStep + lane * kVec;
#pragma unroll
    for (int j = 0; j < kVec; ++j) s[i][j] = 0.f;
    if (c < a.d) {
      load8<kBf16>(a.x, base + c, s[i]);
      if constexpr (kRes) {
        float r[kVec];
        load8<kBf16>(a.residual, base + c, r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[i][j] += r[j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum = fmaf(s[i][j], s[i][j], sum);
  sum = wave_sum(sum, lane);
  if constexpr (kWaves > 1) {
    __shared__ float parts[kWaves];
    if (lane == 0) parts[wave] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += parts[w];
  }
  const float ms = sum / (float)a.d + a.eps;
  // a sum that is not finite has no norm: the whole row is NaN
  const float inv = sum < INFINITY ? 1.0f / sqrtf(ms) : NAN;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * kWaves + part) * kStep + lane * kVec;
    const bool in = c < a.d;
    float y[kVec];
    double p[kVec];  // s w
    uint32_t most = 0;
    double pmost = 0.0;
    if (in) {
      if (kRes && a.total) store8<kBf16>(a.total, base + c, s[i]);
      float w[kVec];
      load8<kBf16>(a.weight, c, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        y[j] = s[i][j] * inv * w[j];
        p[j] = (double)s[i][j] * (double)w[j];
        pmost = fmax(pmost, fabs(p[j]));
      }
      if (a.normed) store8<kBf16>(a.normed, base + c, y);
      // magnitudes as integers: order-preserving, and a NaN is the largest of all
#pragma unroll
      for (int j = 0; j < kVec; ++j) most = max(most, __float_as_uint(y[j]) & 0x7fffffffu);
    }
    const float top = __uint_as_float(row16_max(most));
    const float scale = top != top ? top : fmaxf(top / kE4m3Max, 0x1p-100f);
    pmost = row16_max(pmost);
    if (in) {
      // 448 / pmost to about 2^-50: far more than what is left of it
      double k = __builtin_amdgcn_rcp(pmost);
      k = fma(fma(-pmost, k, 1.0), k, k);
      k = scale > 0x1p-100f ? fma(fma(-pmost, k, 1.0), k, k) * (double)kE4m3Max : (double)inv * 0x1p100;
      if (top < INFINITY) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[j] = (float)(p[j] * k);
      } else {  // over an infinite scale: 0 or, where y is not finite itself, NaN
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[j] *= top != top ? NAN : 0.f;
      }
      int w0 = 0, w1 = 0;
      w0 = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], w0, false);
      w0 = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w0, true);
      w1 = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], w1, false);
      w1 = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], w1, true);
      *reinterpret_cast<int2*>(a.q + base + c) = make_int2(w0, w1);
      if ((lane & 15) == 0) a.scale[(int64_t)(c >> 7) * a.rows + row] = scale;
    }
  }
}

template <bool kBf16, bool kRes>
hipError_t launch(const NormArgs& a, hipStream_t stream) {
  const int steps = (a.d + kStep - 1) / kStep;
#define DFS_NORM(NV, W)                                                                                         \
  norm_q8_kernel<kBf16, kRes, NV, W>                                                                            \
      <<<dim3((uint32_t)(W == 1 ? cdiv(a.rows, 4) : a.rows)), dim3(W == 1 ? 256 : 64 * W), 0, stream>>>(a)
  if (steps <= 1) {
    DFS_NORM(1, 1);
  } else if (steps <= 2) {
    DFS_NORM(1, 2);
  } else if (steps <= 4) {
    DFS_NORM(1, 4);
  } else if (steps <= 8) {
    DFS_NORM(2, 4);
  } else if (steps <= 12) {
    DFS_NORM(3, 4);
  } else if (steps <= 16) {
    DFS_NORM(4, 4);
  } else if (steps <= 32) {
    DFS_NORM(4, 8);
  } else if (steps <= 64) {
    DFS_NORM(4, 16);
  } else {
    DFS_NORM(8, 16);
  }
#undef DFS_NORM
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_q8(const void* x, const void* residual, const void* weight, bool bf16, int64_t rows, int64_t d,
                          float eps, uint8_t* q, float* scale, void* total, void* normed, hipStream_t stream) {
  const NormArgs a{x, residual, weight, q, scale, total, normed, rows, (int)d, eps};
  if (bf16) return residual ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
  return residual ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace dfs
