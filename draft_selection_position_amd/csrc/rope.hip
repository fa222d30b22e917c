// Rotary positions: queries and keys turned on their way from a projection's rows to dense heads
// or into a paged cache, and the positions of a drafted tree's nodes.
//
// Pair i of a head is turned by the angle a = position freqs[i]:
//   (x1, x2) -> A (x1 cos a - x2 sin a, x2 cos a + x1 sin a).
// Pure data movement but for the angles, which all heads of a token share: a wave takes heads of
// one token, computes the token's angles once, a lane each, into LDS, and every lane keeps the
// sines and cosines of the pairs that it has in all of its heads.
//
// Angles.  a / (pi / 2) = n + r, |r| <= 1/2, in 64 bits with what the products' roundings lose carried along: position times
// frequency has up to 56 bits, and its last ones are worth 2^-21 of a turn's quarter at position 2^32 and frequency 1.  So r is
// off by 2^-53 wherever n is exact, n < 2^53; beyond that an angle has no digits left.  Sine and cosine of r pi / 2 are their series in fp32
// (the terms left out are below 2^-29 and 2^-33); n picks the quadrant.
//
// Bound by memory: 16320 tokens of 32 + 8 heads of 128, k and v out of their joint rows too, bf16, 401 MB read and written: 78.5 us, 5.1
// TB/s; 65536 tokens of 16 prompts into pages of 64 with their queries, 1.6 GB: 305 us, 5.3 TB/s; 4003 x 25 heads of 80,
// 20 of them turned, fp32: 12.8 us.  One token: 3.2 us on the device, the launch and two latencies; a block of 17 into
// the cache: 3.9 (starts, length and page in turn).  4096 trees' positions: 3.2 us.  Carrying the roundings of the angles costs little or
// nothing (against angles without, in turn: 80.1 and 79.5 us at 16320 tokens, 307.0 and 306.4 at 65536, 3.8 and 3.7 at one).
#include <algorithm>
#include <type_traits>

#include "dfs_device.h"
#include "dfs_internal.h"

namespace dfs {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kMaxPairs = 512;  // of a head

struct Args {
  RopeJob j;
  const int32_t* positions;  // dense outputs
  // pages
  CacheView c;
  const int32_t* starts;
  const int32_t* prefix_len;
  int32_t* out_lens;
  int batch;
  int heads;      // of all kinds
  int units;      // of a head: 2 W values each
  int per;        // heads of a wave's pass (units <= 64)
  int passes;     // of a token
  int splits;     // waves of a token
};

// cos and sin of pos f, times the amplitude.
__device__ __forceinline__ float2 turn_of(int64_t pos, float f, float amplitude) {
  constexpr double kHigh = 0.63661977236758134308, kLow = -3.9357353350364971764e-17;  // 2 / pi
  const double p = (double)pos, angle = p * (double)f;
  const double n = rint(angle * kHigh);
  double r = fma(angle, kHigh, -n) + fma(angle, kLow, fma(p, (double)f, -angle) * kHigh);
  const double m = rint(r);  // a border's other side; all that is left of an angle past 2^53
  r -= m;
  const float x = (float)r * 1.57079632679489661923f;
  const int k = (int)(((int64_t)n & 3) + ((int64_t)m & 3)) & 3;
  const float z = x * x;
  float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, 1/7!, 1/5!, 1/3!
  s = fmaf(s, z, 8.33333333e-3f);
  s = fmaf(s, z, -1.66666667e-1f);
  s = fmaf(s * z, x, x);
  float c = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);  // 1/10!, 1/8!, 1/6!, 1/4!, 1/2!
  c = fmaf(c, z, -1.38888889e-3f);
  c = fmaf(c, z, 4.16666667e-2f);
  c = fmaf(c, z, -0.5f);
  c = fmaf(c, z, 1.0f);
  const float cs = k & 1 ? s : c, sn = k & 1 ? c : s;
  return make_float2(amplitude * (k == 1 || k == 2 ? -cs : cs), amplitude * (k >= 2 ? -sn : sn));
}

// `bytes` neighbouring bytes as they are.
template <int bytes>
struct RawOf;
template <>
struct RawOf<2> {
  typedef uint16_t type;
};
template <>
struct RawOf<4> {
  typedef uint32_t type;
};
template <>
struct RawOf<8> {
  typedef uint2 type;
};
template <>
struct RawOf<16> {
  typedef uint4 type;
};

// 2 W values of a head, first and second half, as they lie in memory and as numbers.
template <bool kBf16, int W>
struct Unit {
  typedef typename RawOf<W * (kBf16 ? 2 : 4)>::type Raw;
  Raw one, two;
  __device__ __forceinline__ static void widen(const Raw& r, float (&f)[W]) {
    if constexpr (!kBf16) {
      __builtin_memcpy(f, &r, sizeof(r));
    } else {
      uint16_t b[W];
      __builtin_memcpy(b, &r, sizeof(r));
#pragma unroll
      for (int e = 0; e < W; ++e) f[e] = bf16_to_f32(b[e]);
    }
  }
  __device__ __forceinline__ static Raw narrow(const float (&f)[W]) {
    Raw r;
    if constexpr (!kBf16) {
      __builtin_memcpy(&r, f, sizeof(r));
    } else {
      __bf16 b[W];
#pragma unroll
      for (int e = 0; e < W; ++e) b[e] = (__bf16)f[e];  // to nearest, ties to even
      __builtin_memcpy(&r, b, sizeof(r));
    }
    return r;
  }
  // Pair e is (one[e], two[e]), or with kInter the e-th two neighbours of all 2 W.
  template <bool kInter>
  __device__ __forceinline__ void turn(const float (&c)[W], const float (&s)[W]) {
    float f[2][W];
    widen(one, f[0]);
    widen(two, f[1]);
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int i1 = kInter ? 2 * e : e, i2 = kInter ? 2 * e + 1 : W + e;
      float& x1 = f[i1 / W][i1 % W];
      float& x2 = f[i2 / W][i2 % W];
      const float y1 = fmaf(x1, c[e], -(x2 * s[e])), y2 = fmaf(x2, c[e], x1 * s[e]);
      x1 = y1;
      x2 = y2;
    }
    one = narrow(f[0]);
    two = narrow(f[1]);
  }
};

// The sequence that row `row` belongs to: that of the first end above it.  64 ends at a time.
__device__ __forceinline__ int sequence_of(const int32_t* ends, int batch, int row, int lane) {
  int lo = 0, n = batch;  // among ends[lo .. lo + n - 1]
  while (n > 64) {
    const int each = (n + 63) / 64, at = min((lane + 1) * each, n) - 1;
    const int below = __popcll(__ballot(ends[lo + at] <= row));  // pieces that end at or before the row
    if (below == 64) return batch;
    lo += below * each;
    n = min(each, n - below * each);
    if (n <= 0) return batch;  // not in order
  }
  return lo + __popcll(__ballot(lane < n && ends[lo + min(lane, n - 1)] <= row));
}

template <bool kBf16, int W, bool kInter, bool kPaged>
__global__ __launch_bounds__(kThreads) void rope_kernel(Args a) {
  constexpr int kBatch = 2;  // passes whose loads go out together
  __shared__ float2 turns[kWaves][kMaxPairs];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  if constexpr (kPaged) {
    for (int b = blockIdx.x * kThreads + threadIdx.x; a.out_lens && b < a.batch; b += gridDim.x * kThreads) {
      const int rows = (int)a.j.rows;
      const int n = min(max(a.starts[b + 1], 0), rows) - min(max(a.starts[b], 0), rows);
      a.out_lens[b] = (int32_t)min((int64_t)max(a.c.lens[b], 0) + max(n, 0), (int64_t)INT32_MAX);
    }
  }
  const uint32_t w = blockIdx.x * kWaves + wave;
  const int token = (int)(w / a.splits), split = (int)(w % a.splits);
  if (token >= a.j.rows) return;
  int64_t pos;
  int64_t slot = -1;  // of the token in the pools: page * heads of a page * rows of a page + row
  if constexpr (kPaged) {
    const int b = uniform(sequence_of(a.starts + 1, a.batch, token, lane));
    if (b >= a.batch) return;
    const int i = token - max(a.starts[b], 0);
    if (i < 0) return;
    const int64_t at = (int64_t)max(a.c.lens[b], 0) + i;
    pos = at + (a.prefix_len ? max(*a.prefix_len, 0) : 0);
    if ((at >> a.c.page_shift) < a.c.table_width) {
      const int page = a.c.block_table[(int64_t)b * a.c.table_width + (at >> a.c.page_shift)];
      if (page >= 0 && page < a.c.n_pages)
        slot = (((int64_t)page * a.c.kv_heads) << a.c.page_shift) + (at & ((1 << a.c.page_shift) - 1));
    }
  } else {
    pos = a.positions[token];
  }
  const int pairs = a.j.rot_dim / 2, D = a.j.head_dim;
  for (int i = lane; i < pairs; i += 64) turns[wave][i] = turn_of(pos, a.j.freqs[i], a.j.amplitude);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // a wave's own

  const int in_pass = a.units <= 64 ? lane / a.units : 0;
  const int hq = a.j.of[0].heads, hk = a.j.of[1].heads;
  for (int u = a.units <= 64 ? lane % a.units : lane; u < a.units; u += 64) {
    const bool turned = u * 2 * W < a.j.rot_dim;
    const int one = turned && !kInter ? u * W : 2 * W * u, two = turned && !kInter ? one + pairs : one + W;
    float c[W], s[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const float2 t = turned ? turns[wave][u * W + e] : make_float2(1.f, 0.f);
      c[e] = t.x;
      s[e] = t.y;
    }
    for (int p = split; p < a.passes; p += kBatch * a.splits) {
      Unit<kBf16, W> x[kBatch];
      char* to[kBatch];
      bool turn[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int head = (p + k * a.splits) * a.per + in_pass;
        const bool is_q = head < hq, is_k = !is_q && head < hq + hk;
        const int h = is_q ? head : is_k ? head - hq : head - hq - hk;
        const RopeHeads& of = a.j.of[0];
        const char* in = static_cast<const char*>(is_q ? of.in : is_k ? a.j.of[1].in : a.j.of[2].in);
        char* out = static_cast<char*>(is_q ? of.out : is_k ? a.j.of[1].out : a.j.of[2].out);
        const int64_t stride = is_q ? of.stride : is_k ? a.j.of[1].stride : a.j.of[2].stride;
        const int heads = is_q ? hq : is_k ? hk : a.j.of[2].heads;
        constexpr int kSize = kBf16 ? 2 : 4;
        in += ((int64_t)token * stride + h * D) * kSize;
        int64_t row = (int64_t)token * heads + h;
        bool there = in_pass < a.per && head < a.heads;
        if constexpr (kPaged) {
          if (!is_q) {
            out = static_cast<char*>(is_k ? a.c.k_pages : a.c.v_pages);
            row = slot + ((int64_t)h << a.c.page_shift);
            there = there && slot >= 0;
          }
        }
        to[k] = there ? out + row * D * kSize : nullptr;
        turn[k] = turned && (is_q || is_k);
        if (there) {
          x[k].one = *reinterpret_cast<const typename Unit<kBf16, W>::Raw*>(in + one * kSize);
          x[k].two = *reinterpret_cast<const typename Unit<kBf16, W>::Raw*>(in + two * kSize);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        constexpr int kSize = kBf16 ? 2 : 4;
        if (!to[k]) continue;
        if (turn[k]) x[k].template turn<kInter>(c, s);
        *reinterpret_cast<typename Unit<kBf16, W>::Raw*>(to[k] + one * kSize) = x[k].one;
        *reinterpret_cast<typename Unit<kBf16, W>::Raw*>(to[k] + two * kSize) = x[k].two;
      }
    }
  }
}

// Pairs that a lane has at once: 16 bytes of each half (pairs apart), or of all (neighbours), where the head
// and what is turned of it divide so; else fewer.
template <class F>
hipError_t with_width(const RopeJob& j, F f) {
  int w = (j.bf16 ? 8 : 4) / (j.interleaved ? 2 : 1);
  while (w > 1 && (j.rot_dim % (2 * w) || j.head_dim % (2 * w))) w /= 2;
  auto bf = [&](auto bf16) {
    switch (w) {
      case 8: return f(bf16, std::integral_constant<int, decltype(bf16)::value ? 8 : 4>{});  // bf16 alone
      case 4: return f(bf16, std::integral_constant<int, 4>{});
      case 2: return f(bf16, std::integral_constant<int, 2>{});
      default: return f(bf16, std::integral_constant<int, 1>{});
    }
  };
  return j.bf16 ? bf(std::true_type{}) : bf(std::false_type{});
}

template <bool kPaged>
hipError_t run(Args a, hipStream_t stream) {
  return with_width(a.j, [&](auto bf16, auto width) {
    constexpr bool kBf16 = decltype(bf16)::value;
    constexpr int W = decltype(width)::value;
    a.heads = a.j.of[0].heads + a.j.of[1].heads + a.j.of[2].heads;
    a.units = a.j.head_dim / (2 * W);
    a.per = a.units <= 64 ? 64 / a.units : 1;
    a.passes = (int)cdiv(a.heads, a.per);
    // few tokens: a wave for every pass
    a.splits = (int)std::min<int64_t>(a.passes, std::max<int64_t>(1, 8192 / a.j.rows));
    const dim3 grid((uint32_t)cdiv(a.j.rows * a.splits, kWaves));
    if (a.j.interleaved)
      rope_kernel<kBf16, W, true, kPaged><<<grid, dim3(kThreads), 0, stream>>>(a);
    else
      rope_kernel<kBf16, W, false, kPaged><<<grid, dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
  });
}

// A wave per tree: a lane's node has as many ancestors as bits beside its own.
__global__ __launch_bounds__(kThreads) void tree_positions_kernel(const int32_t* parents, const int32_t* lens,
                                                                  const int32_t* prefix_len, int batch, int T,
                                                                  int32_t* out) {
  const int lane = threadIdx.x & 63, b = blockIdx.x * kWaves + uniform(threadIdx.x >> 6);
  if (b >= batch) return;
  const int most = 1 << 30;
  const int64_t before = (int64_t)min(max(lens[b], 0), most) + (prefix_len ? min(max(*prefix_len, 0), most) : 0);
  const uint64_t bits = tree_bits(lane < T ? parents[(int64_t)b * T + lane] : -2, T, lane);
  if (lane < T)
    out[(int64_t)b * T + lane] = (int32_t)min(before + (bits ? (int)__popcll(bits) - 1 : 0), (int64_t)INT32_MAX);
}

}  // namespace

hipError_t launch_tree_positions(const int32_t* parents, const int32_t* lens, const int32_t* prefix_len, int64_t batch,
                                 int64_t T, int32_t* out, hipStream_t stream) {
  tree_positions_kernel<<<dim3((uint32_t)cdiv(batch, kWaves)), dim3(kThreads), 0, stream>>>(parents, lens, prefix_len,
                                                                                         (int)batch, (int)T, out);
  return hipGetLastError();
}

hipError_t launch_rope(const RopeJob& job, const int32_t* positions, hipStream_t stream) {
  Args a{};
  a.j = job;
  a.positions = positions;
  return run<false>(a, stream);
}

hipError_t launch_cache_append(const RopeJob& job, const CacheView& c, const int32_t* starts, const int32_t* prefix_len,
                               int64_t batch, int32_t* out_lens, hipStream_t stream) {
  Args a{};
  a.j = job;
  a.c = c;
  a.starts = starts;
  a.prefix_len = prefix_len;
  a.out_lens = out_lens;
  a.batch = (int)batch;
  return run<true>(a, stream);
}

}  // namespace dfs
