// Attention of a whole batch's query rows over a prefix that its sequences share.
//
// All rows of a kv head (sequences x nodes x heads of the group) against the prefix's keys: one large pair of matrix
// products with a softmax between, in pieces that are joined with the sequences' own keys later.  The layout is tree
// attention's (S^T = K Q^T, O^T = V^T P^T, a lane holds one query row), but a wave has 64 rows, as two halves of 32
// in turns: while the matrix cores work for one half (its next scores and its last weights' product with V),
// the vector unit takes the other's exponentials.  Every fragment that a wave reads from LDS serves both halves:
// at 32 rows a wave, LDS reads take as long as the products.
//
// The loop is straight: a branch in it (a load under a condition, a last step of another shape) ends a stretch that the
// compiler mixes matrix, vector and scalar instructions in, and a wave that is alone on its SIMD fills the gaps of
// one only with another of its own.  So pages are looked up by scalar loads, addresses are scalar sums, loads past
// the end fetch the last stage again, and the one branch (a maximum that lags, or the prefix's end) is out of the way.
//
// Weights are rounded to bf16 for the second product, 2^-8 of each at most, as in tree attention, and the sums take them as they
// were: the roundings of a sum's many weights cancel (2-norm errors 0.00228 with either kind of sum; 0.0016 with weights
// in fp32, which is the output's own rounding).
//
// What bounds it (MI355X; cycles of a SIMD for a half's 32 x 32 scores, 512 of matrix cores at head 128): 890 in the loop, of which 710
// are matrix and vector instructions as a wave alone issues them, 80 loads into LDS, 65 the barrier, 65 LDS reads; 1010 with
// the starts and ends of the ranges.  64 x 17 rows x 4 heads of 128 for each of 8 kv heads, 16384 keys: 281 to 308 us (up to 331 from a cold
// start), 950 to 1040 TFLOP/s at 1.9 to 2.0 GHz (32 rows a wave, two waves a SIMD: 480).
// Head 64: 540 in all, 256 of matrix cores.  What the two waves issue nearly fills it: 426 of vector instructions (89, of which 16
// exponentials at 8 cycles), 107 of scalar ones, 24 of LDS reads; a wave waits for its turn to issue for a third of its time, for memory
// or the barrier for a tenth.  12 x 63 x 6 rows for 4 kv heads, 60001 keys: 320 to 350 us, 830 TFLOP/s (480 to 500).
#include <algorithm>
#include <type_traits>

#include "attn_tile.h"
#include "dfs_internal.h"
#include "prefix.h"

namespace dfs {
namespace {

struct PrefixArgs {
  CacheView c;  // of one sequence
  const uint16_t* q;
  float* part_o;   // [Hkv, slots, kRows, D]
  float* part_ml;  // [Hkv, slots, kRows, 2]
  PrefixCut cut;
  int rows, group, q_heads;
  float c2;
};

template <int D_>
struct PCfg {
  static constexpr int D = D_;
  static constexpr int kWaves = 4, kThreads = 64 * kWaves;
  static constexpr int kRows = kPrefixRows;  // of a workgroup
  static constexpr int NB = D == 64 ? 1 : 2;  // blocks of 32 keys of a step
  static constexpr int kKeys = 32 * NB;      // of a stage, and of a step
  static constexpr int kRowBytes = 2 * D, kChunks = kRowBytes / 16, kRowsPerLoad = 64 / kChunks;
  static constexpr int kHalf = kKeys * kRowBytes;       // K (or V) of a stage
  static constexpr int S = NB == 1 ? 8 : 4;             // stages of either
  static constexpr int kLoads = kHalf / 1024 / kWaves;  // of a wave, of a stage's K (or V)
  static constexpr int kRing = 2 * S * kHalf;
  static constexpr int kPages = 256;                    // bytes of a wave's pages of a stage
  static constexpr int kSlots = S + 2;                  // of them
  static constexpr int kLds = kRing + kWaves * kSlots * kPages;
  static constexpr int kMinWaves = D == 64 ? 2 : 1;  // per SIMD
};

// Half of a wave's rows.
template <class C>
struct Half {
  f32x16 o[C::D / 32];
  f32x16 s[C::NB];        // scores of a step's keys
  bf16x8 p[C::NB][2];     // weights of the step before
  bf16x8 q[C::D / 16];
  float m, l;    // maximum and sum,
  float off;     // what is taken from a score's exponent: the maximum, if there is one,
  float lim;     // and how far a score may go beyond it
  float top;     // the largest of the step's scores
};

template <class C>
__device__ __forceinline__ void read_k(lds_t kt, const Frag<C>& at, bf16x8 (&kf)[C::NB][C::D / 16]) {
  typedef __attribute__((address_space(3))) const bf16x8* k_ptr;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int x = 0; x < C::D / 16; ++x) kf[nb][x] = *(k_ptr)(kt + nb * 32 * C::kRowBytes + (at.k ^ (32 * x)));
}

template <class C>
__device__ __forceinline__ void read_v(lds_t vt, const Frag<C>& at, bf16x8 (&vf)[C::NB][2][C::D / 32]) {
  typedef __attribute__((address_space(3))) s16x4* tr_ptr;
  uint32_t from[C::D / 32];
#pragma unroll
  for (int dt = 0; dt < C::D / 32; ++dt) {
    from[dt] = (uint32_t)(uintptr_t)(vt + at.v[dt]);
    asm("" : "+v"(from[dt]));  // one address each; the rest are the reads' own offsets
  }
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int kc = 0; kc < 2; ++kc)
#pragma unroll
      for (int dt = 0; dt < C::D / 32; ++dt) {
        union {
          s16x4 half[2];
          bf16x8 all;
        } f;
#pragma unroll
        for (int z = 0; z < 2; ++z)
          f.half[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (tr_ptr)((lds_t)(uintptr_t)from[dt] + (32 * nb + 16 * kc + 8 * z) * C::kRowBytes));
        vf[nb][kc][dt] = f.all;
      }
}

// The scores of a step's keys for half x.
template <class C>
__device__ __forceinline__ void scores(Half<C>& x, const bf16x8 (&kf)[C::NB][C::D / 16]) {
  f32x16 s[C::NB];
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
    s[nb] = f32x16{};
#pragma unroll
    for (int i = 0; i < C::D / 16; ++i) s[nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[nb][i], x.q[i], s[nb], 0, 0, 0);
  }
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) x.s[nb] = s[nb];
}

template <class C>
__device__ __forceinline__ void weigh(Half<C>& x, const bf16x8 (&vf)[C::NB][2][C::D / 32]) {
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int kc = 0; kc < 2; ++kc)
#pragma unroll
      for (int dt = 0; dt < C::D / 32; ++dt)
        x.o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[nb][kc][dt], x.p[nb][kc], x.o[dt], 0, 0, 0);
}

// Scores become weights: first all of the exponents, so that none waits for the one before it.
template <class C>
__device__ __forceinline__ void soften(Half<C>& x, float c2) {
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x.s[nb][i] = fmaf(x.s[nb][i], c2, -x.off);
    asm volatile("" : "+v"(x.s[nb]));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x.s[nb][i] = __builtin_amdgcn_exp2f(x.s[nb][i]);
      sum[i & 1] += x.s[nb][i];
    }
#pragma unroll
    for (int kc = 0; kc < 2; ++kc) {
      union {
        bf16x2 two[4];
        bf16x8 all;
      } pf;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf.two[i] = __builtin_convertvector(f32x2{x.s[nb][8 * kc + 2 * i], x.s[nb][8 * kc + 2 * i + 1]}, bf16x2);
      x.p[nb][kc] = pf.all;
      asm volatile("" : "+v"(x.p[nb][kc]));  // here and no later
    }
  }
  x.l += sum[0] + sum[1];
}

template <class C>
__device__ __forceinline__ float largest(const Half<C>& x, int lane) {
  float top = x.s[0][0];
#pragma unroll
  for (int i = 1; i < 16 * C::NB; ++i) top = fmaxf(top, x.s[i / 16][i % 16]);
  return fmaxf(top, xor32(top, lane));
}

// Before a step's scores become weights: those past the prefix's end count as -inf, and the row's maximum follows
// when it lags (see tree attention).  last: infinite for the step that the prefix may end in, else zero; left: the keys
// from the step's first on.
template <class C>
__device__ __forceinline__ void settle(Half<C>& x, float c2, float last, int left, int lane) {
  if (__builtin_expect(__ballot(!(fmaf(x.top, c2, last) <= x.lim)) != 0, 0)) {
    if (left < C::kKeys) {
      int mine = left - 4 * (lane >> 5);
      asm volatile("" : "+v"(mine));  // nothing of this ahead of the branch
#pragma unroll
      for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * nb + 8 * (i / 4) + i % 4 >= mine) x.s[nb][i] = -INFINITY;
      x.top = largest<C>(x, lane);
    }
    const float m = fmaxf(x.m, x.top * c2);
    const float f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(x.m - m);
    x.l *= f;
#pragma unroll
    for (int dt = 0; dt < C::D / 32; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) x.o[dt][i] *= f;
    x.m = m;
    x.off = m == -INFINITY ? 0.f : m;
    x.lim = m + kLag;
  }
}

template <int D, bool kWide>
__global__ __launch_bounds__(PCfg<D>::kThreads, PCfg<D>::kMinWaves) void prefix_attention_kernel(PrefixArgs a) {
  typedef PCfg<D> C;
  __shared__ __attribute__((aligned(1024))) char lds[C::kLds];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
  const int Hkv = a.c.kv_heads;
  const int second = blockIdx.x / (Hkv * a.cut.C);  // of a pair of workgroups (the first ones start first)
  const int head = blockIdx.x % Hkv, w = blockIdx.x / Hkv - second * a.cut.C;
  const int len = a.c.len(0);
  PrefixCut cut = a.cut;
  cut.cut((len + kPrefixKeys - 1) / kPrefixKeys);
  if (len == 0) return;
  const Frag<C> at(lane);
  const uint32_t ring0 = lds_addr(lds), pages0 = ring0 + C::kRing + wave * C::kSlots * C::kPages;
  const char* my_pages = lds + C::kRing + wave * C::kSlots * C::kPages;
  const int64_t page_bytes = ((int64_t)Hkv << a.c.page_shift) * C::kRowBytes;
  const int in_page = (1 << a.c.page_shift) - 1;
  const int32_t* table = a.c.block_table;
  const int rr = lane / C::kChunks, slot = lane % C::kChunks;
  // of the rows that this wave loads (16 or 32 apart) the slots are the same
  const int row0 = wave * C::kRowsPerLoad + rr;
  const uint32_t k_off = rr * C::kRowBytes + 16 * k_slot<C>(slot, row0), v_off = rr * C::kRowBytes + 16 * v_slot<C>(slot, row0);

  int turn = 0;
  int64_t x = 0, x_end = 0;  // of what is shared: key tiles x .. x_end - 1, all row tiles' in a row
  while (true) {
    int rt, first, last, k = 0;  // row tile, its key tiles, and the number of its piece that they are
    if (turn < cut.whole) {
      rt = turn * cut.C + w, first = 0, last = cut.tiles;
    } else if (w < cut.f * cut.n) {
      if (turn > cut.whole) break;
      k = w / cut.n;
      rt = cut.whole * cut.C + w % cut.n;
      first = k * cut.each, last = cut.rest ? first + cut.each : min(first + cut.each, cut.tiles);
      if (first >= last) break;
    } else {
      if (cut.n == 0 || cut.rest == 0) break;
      const int v = w - cut.f * cut.n;
      if (turn == cut.whole) {
        x = v * cut.share;
        x_end = min(x + cut.share, (int64_t)cut.n * cut.rest);
      }
      if (x >= x_end) break;
      const int r = (int)(x / cut.rest), from = (int)(x - (int64_t)r * cut.rest);
      const int to = (int)min((int64_t)cut.rest, from + x_end - x);
      k = cut.f + v - (int)((int64_t)r * cut.rest / cut.share);
      rt = cut.whole * cut.C + r;
      first = cut.f * cut.each + from, last = cut.f * cut.each + to;
      x += to - from;
    }
    const int64_t piece = cut.slot(rt) + cut.pair * k + second;
    ++turn;
    if (cut.pair > 1) {
      const int half = first + (int)(((int64_t)(last - first) * PrefixCut::kFirst + 32) / 64);
      first = second ? half : first, last = second ? last : half;
    }
    const int base = first * kPrefixKeys, end_key = min(last * kPrefixKeys, len);
    const int n = (end_key - base + C::kKeys - 1) / C::kKeys;  // stages

    // Where the rows of stage i lie that this wave loads; past the range's last stage that one again, past the
    // prefix's end the last key's.  kWide: the rows of one load lie in one page, which is looked up by scalar loads.
    struct Off {
      int64_t of[C::kLoads];
    };
    auto row_off = [&](int page, int key) {
      return (int64_t)min(max(page, 0), a.c.n_pages - 1) * page_bytes + (int64_t)((head << a.c.page_shift) + (key & in_page)) * C::kRowBytes;
    };
    auto wide_off = [&](int i) {
      typedef const __attribute__((address_space(4))) int32_t* const_ptr;
      Off o;
#pragma unroll
      for (int u = 0; u < C::kLoads; ++u) {
        const int key = base + min(i, n - 1) * C::kKeys + (wave + C::kWaves * u) * C::kRowsPerLoad;
        o.of[u] = row_off(*(const_ptr)(table + (min(key, len - 1) >> a.c.page_shift)), key);
      }
      return o;
    };
    // Smaller pages: the pages of a stage's keys, through LDS.
    auto look_up = [&](int i) {
      const int key = min(base + i * C::kKeys + (lane & (C::kKeys - 1)), len - 1);
      dma4(table + (key >> a.c.page_shift), __builtin_amdgcn_readfirstlane(pages0 + i % C::kSlots * C::kPages));
    };
    auto load = [&](int i, auto kv, const Off& o) {
      constexpr int kV = decltype(kv)::value;
      const char* pool = static_cast<const char*>(kV ? a.c.v_pages : a.c.k_pages);
      const uint32_t to = ring0 + (kV * C::S + i % C::S) * C::kHalf + wave * 1024;
#pragma unroll
      for (int u = 0; u < C::kLoads; ++u) {
        const uint32_t lds_at = __builtin_amdgcn_readfirstlane(to + u * C::kWaves * 1024);
        if constexpr (kWide) {
          dma16s(pool + o.of[u], kV ? v_off : k_off, lds_at);
        } else {
          const int* pages = reinterpret_cast<const int*>(my_pages + min(i, n - 1) % C::kSlots * C::kPages);
          const int row = (wave + C::kWaves * u) * C::kRowsPerLoad + rr, key = min(base + min(i, n - 1) * C::kKeys + row, len - 1);
          dma16<false>(pool + row_off(pages[row], key) + 16 * (kV ? v_slot<C>(slot, row) : k_slot<C>(slot, row)), lds_at);
        }
      }
    };
    constexpr std::integral_constant<int, 0> kK{};
    constexpr std::integral_constant<int, 1> kV{};

    Half<C> A, B;
    const int row_a = rt * C::kRows + 64 * wave + (lane & 31);
    auto begin = [&](Half<C>& x, int row) {
      const int qrow = min(row, a.rows - 1), t = qrow / a.group, gh = qrow % a.group;
      const uint16_t* q = a.q + ((int64_t)t * a.q_heads + head * a.group + gh) * D + 8 * h;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) x.q[i] = *reinterpret_cast<const bf16x8*>(q + 16 * i);
      if constexpr (D == 128) {
        // 256 registers that vector instructions reach do not hold all: the queries live in the other 256
#pragma unroll
        for (int i = 0; i < D / 16; ++i) asm volatile("" : "+a"(x.q[i]));
      }
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) x.o[dt] = f32x16{};
      x.m = x.lim = -INFINITY;
      x.l = x.off = 0.f;
    };
    if (n > 0) {
      if (!kWide) {
#pragma unroll 1
        for (int i = 0; i < C::S + 2; ++i) look_up(i);
        big::wait_vmcnt<0>();
        asm volatile("" ::: "memory");
      }
#pragma unroll 1
      for (int i = 0; i < C::S; ++i) {
        const Off o = kWide ? wide_off(i) : Off{};
        load(i, kK, o);
        if (i < C::S - 1) load(i, kV, o);
      }
    }
    begin(A, row_a);
    begin(B, row_a + 32);
    if (n > 0) {
      if (!kWide) {
#pragma unroll 1
        for (int i = C::S + 2; i < 2 * C::S; ++i) look_up(i);
      }
      big::wait_vmcnt<0>();
      big::bar();
      auto k_at = [&](int i) { return (lds_t)(lds + i % C::S * C::kHalf); };
      auto v_at = [&](int i) { return (lds_t)(lds + (C::S + i % C::S) * C::kHalf); };
      auto left = [&](int i) { return len - (base + i * C::kKeys); };
      bf16x8 kf[C::NB][D / 16], vf[C::NB][2][D / 32];
      read_k<C>(k_at(0), at, kf);
      scores<C>(A, kf);
      scores<C>(B, kf);
      A.top = largest<C>(A, lane);
      B.top = largest<C>(B, lane);
      settle<C>(A, a.c2, INFINITY, left(0), lane);
      settle<C>(B, a.c2, INFINITY, left(0), lane);
      soften<C>(A, a.c2);
      read_k<C>(k_at(1), at, kf);  // behind the last one: that one again, not used
      big::bar();
      Off v0 = kWide ? wide_off(C::S - 1) : Off{}, v1 = kWide ? wide_off(C::S) : Off{}, k1 = kWide ? wide_off(C::S + 1) : Off{};
      load(C::S, kK, v1);
#pragma unroll 1
      for (int i = 0; i < n - 1; ++i) {
        // stage i's V and stage i + 2's K are here, and everyone is done with V before and K up to stage i + 1
        big::wait_vmcnt<(C::S - 2) * 2 * C::kLoads>();
        big::bar();
        const float last = i == n - 2 ? INFINITY : 0.f;
        // A's next scores and last product, B's weights
        if (!kWide) look_up(i + 2 * C::S);
        load(i + C::S - 1, kV, v0);
        read_v<C>(v_at(i), at, vf);
        scores<C>(A, kf);
        soften<C>(B, a.c2);
        weigh<C>(A, vf);
        A.top = largest<C>(A, lane);
        settle<C>(A, a.c2, last, left(i + 1), lane);
        // B's next scores and last product, A's weights
        load(i + C::S + 1, kK, k1);
        v0 = v1, v1 = k1;
        if (kWide) k1 = wide_off(i + C::S + 2);
        scores<C>(B, kf);
        read_k<C>(k_at(i + 2), at, kf);
        soften<C>(A, a.c2);
        weigh<C>(B, vf);
        B.top = largest<C>(B, lane);
        settle<C>(B, a.c2, last, left(i + 1), lane);
      }
      big::wait_vmcnt<0>();
      big::bar();
      if (left(n - 1) < C::kKeys) {
        // V rows past the end: a weight of zero must not meet what is not finite in them
        char* vt = lds + (C::S + (n - 1) % C::S) * C::kHalf;
        for (int u = left(n - 1) * C::kChunks + (int)threadIdx.x; u < C::kKeys * C::kChunks; u += C::kThreads)
          *reinterpret_cast<uint4*>(vt + 16 * u) = make_uint4(0, 0, 0, 0);
        big::bar();
      }
      read_v<C>(v_at(n - 1), at, vf);
      soften<C>(B, a.c2);
      weigh<C>(A, vf);
      weigh<C>(B, vf);
    }

    auto end = [&](Half<C>& x, int row) {
      const float l = x.l + xor32(x.l, lane);
      if (row >= a.rows) return;
      const int64_t slot = (head * cut.slots() + piece) * C::kRows + row % C::kRows;
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<f32x4*>(a.part_o + slot * D + 32 * dt + 8 * u + 4 * h) =
              f32x4{x.o[dt][4 * u], x.o[dt][4 * u + 1], x.o[dt][4 * u + 2], x.o[dt][4 * u + 3]};
      if (h == 0) *reinterpret_cast<f32x2*>(a.part_ml + 2 * slot) = f32x2{x.m, l};
    };
    end(A, row_a);
    end(B, row_a + 32);
    __syncthreads();  // everyone is done with the ring
  }
}

}  // namespace

hipError_t launch_prefix_attention(const CacheView& prefix, const PrefixCut& cut, const void* q, int64_t rows,
                                   int64_t group, int64_t D, float c2, float* part_o, float* part_ml,
                                   hipStream_t stream) {
  PrefixArgs a{};
  a.c = prefix;
  a.q = static_cast<const uint16_t*>(q);
  a.part_o = part_o;
  a.part_ml = part_ml;
  a.cut = cut;
  a.rows = (int)rows;
  a.group = (int)group;
  a.q_heads = (int)(group * prefix.kv_heads);
  a.c2 = c2;
  const dim3 grid((uint32_t)(prefix.kv_heads * cut.C * cut.pair));
  const bool wide = ((int64_t)1 << prefix.page_shift) >= 1024 / (2 * D);  // a load's 1 KB of rows in one page
  if (D == 64)
    wide ? prefix_attention_kernel<64, true><<<grid, dim3(256), 0, stream>>>(a)
         : prefix_attention_kernel<64, false><<<grid, dim3(256), 0, stream>>>(a);
  else
    wide ? prefix_attention_kernel<128, true><<<grid, dim3(256), 0, stream>>>(a)
         : prefix_attention_kernel<128, false><<<grid, dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace dfs
