// Attention of a tree of drafted tokens over a paged cache.
//
// Query row (t, h) of a sequence sees every key of the sequence's cache and the tree's
// nodes that are t or its ancestors:
//   out = sum_j softmax_j(scale q . k_j) v_j
// with the running maximum and sum of one pass over the keys.
//
// The query rows that share a kv head (nodes x heads of the group) are the columns of the
// matrix products: S^T = K Q^T and O^T = V^T P^T on V_MFMA_F32_32X32X16_BF16, so that a
// lane holds scores of one row only: its maximum and sum need one exchange with the lane
// 32 away, a rescale is one factor per lane, and P^T's registers are already the second
// product's operand (its 16 keys per instruction are taken in the order in which S^T's
// sums lie; V^T comes out of LDS in the same order by the transposing read).  P is rounded
// to bf16 for the matrix cores (at most 2^-8 per weight, as the output's own rounding; the sums of
// weights take them as they were): 2-norm errors of 0.0018 to 0.0023 against 0.0016 of the output's
// rounding alone.  Scores, maxima, sums and O stay in fp32.
//
// K and V tiles go from memory straight into LDS, through a ring of stages.  Up to 32 query
// rows: four waves take tiles of 32 keys of their own and never wait for each other until they
// are joined at the end.  More rows: the waves of a workgroup share a tile of 64, 32 rows each.
// Pages are looked up two ring lengths ahead, through LDS as well: a load into a register
// in the loop would make the compiler wait for everything in flight.  Work is split along
// the keys: the tiles of all sequences in a row are cut evenly over the workgroups of a
// head, whatever the lengths are; sequences that were cut are joined by a second kernel
// from fp32 partial results.  A sequence's nodes are keys like the cache's, right behind them.
//
// What bounds it (MI355X): 64 sequences of 17 nodes, 4 heads to a kv head of 128, 0 to 8192 cached
// keys: 205 to 209 us, memory at 5.3 TB/s.  2 x 64 nodes x 6 heads to a kv head of 64, 131001 keys: 144 to
// 149 us, 700 TFLOP/s; a head of 64 costs as many exponentials as products' cycles, and the
// card holds 2.0 GHz under it.  One token, 4001 keys: 12.0 us, two launches and a chain of four
// memory latencies (lengths, pages, keys, pieces); its 16 MB would take 2.5.
#include "dfs_device.h"
#include "dfs_internal.h"
#include "mfma_big.h"

namespace dfs {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kUnused = -1.0f;  // for a sum of weights
constexpr float kLag = 8.0f;  // a maximum may lag this far (in powers of two) before sums are rescaled

struct AttnArgs {
  CacheView c;
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* parents;
  uint16_t* out;
  float* part_o;   // [Hkv, row tiles, 2 G, rows of a tile, D]
  float* part_ml;  // [Hkv, row tiles, 2 G, rows of a tile, 2]: maximum and sum; of an unused node's row the last piece has kUnused
  int2* pieces;    // [batch]: the first and the last part with a tile of the sequence (NULL: nothing to join)
  int batch, T, group, G, row_tiles;
  bool whole;  // parts are sequences
  int spread;  // 16-lane groups that join a row's pieces: 1, 4 or 16
  float c2;  // scale * log2(e)
};

// KW key groups x RW row groups of waves, a ring of S stages of 32 SUB keys; kOnce: one workgroup
// has all rows of a head.
template <int D_, int KW_, int RW_, int S_, int SUB_ = 1, bool kOnce_ = true>
struct Cfg {
  static constexpr int D = D_, KW = KW_, RW = RW_, S = S_;
  static_assert(KW == 1 || RW == 1, "waves share a tile, or have their own");
  static constexpr int kWaves = KW * RW, kThreads = 64 * kWaves;
  static constexpr bool kOnce = kOnce_;
  static constexpr int kRows = 32 * RW;            // query rows of a workgroup
  static constexpr int SUB = SUB_, kKeys = 32 * SUB;  // keys of a group's step
  static constexpr int kTile = KW * kKeys;         // of a workgroup's
  static constexpr int kRowBytes = 2 * D;          // of a key in LDS
  static constexpr int kChunks = kRowBytes / 16;   // 16-byte chunks
  static constexpr int kRowsPerLoad = 64 / kChunks;
  static constexpr int kHalf = kKeys * kRowBytes;  // K (or V) of a group's step
  static constexpr int kLoadsAll = kKeys / kRowsPerLoad;    // loads of them
  static constexpr int kLoads = (kLoadsAll + RW - 1) / RW;  // of a wave (some repeated when uneven)
  static constexpr int kInFlight = (S - 2) * 2 * kLoads;    // loads of the steps after the one that is waited for
  static constexpr int kStage = 2 * kHalf;         // of a key group
  static constexpr int kAhead = 2 * (S - 1);       // steps that pages are looked up ahead
  static constexpr int kPages = 256;               // bytes of a wave's pages of one step
  static constexpr int kRing = KW * S * kStage;
  static constexpr int kJoin = KW > 1 ? KW * (D / 2 + 2) * 256 : 0;  // key groups meet in the ring's LDS
  static_assert(kJoin <= kRing, "LDS of the join");
  static constexpr int kLds = kRing + kWaves * (kAhead + 1) * kPages;
  static constexpr int kMost = D == 64 ? 3 : 2;  // waves that a SIMD's registers hold
  static constexpr int kByLds = 163840 / (kLds + 2304), kByWaves = 4 * kMost / kWaves;
  static constexpr int kGroups = kByLds < kByWaves ? kByLds : kByWaves;  // workgroups of a CU
  // Three waves of a SIMD: the oldest is served first and the last ends far behind (95, 106 and
  // 128 us), alone on its SIMD.  A wave gives way as it gets on: 147.3 -> 142.8 us at 2 x 64
  // nodes x 131001 keys; with two waves it gains nothing.
  static constexpr bool kEven = kGroups * kWaves > 8;
  static constexpr int kMinWaves = kGroups * kWaves > 8 ? 3 : kGroups * kWaves > 4 ? 2 : 1;  // per SIMD
};

// 16 bytes per lane from memory straight into LDS at lds_base + 16 lane; kOnce: nobody else
// reads them (64 sequences x 17 nodes, 8192 keys: 203 us against 221 without the hint).
template <bool kOnce>
__device__ __forceinline__ void dma16(const void* p, uint32_t lds_base) {
  if constexpr (kOnce)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt"
                 :
                 : "v"(p), "s"(lds_base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(p), "s"(lds_base)
                 : "memory", "m0");
}

// 4 bytes per lane, at lds_base + 4 lane.
__device__ __forceinline__ void dma4(const void* p, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(p), "s"(lds_base) : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((big::lds_ptr_t)p);
}

// Where chunk c of key `row` lies: K so that 16 rows' equal chunks, V so that four rows'
// equal 64-byte blocks fall on distinct banks.
template <class C>
__device__ __forceinline__ int k_slot(int c, int row) {
  return C::kChunks == 16 ? c ^ (row & 15) : c ^ ((row >> 1) & 7);
}
template <class C>
__device__ __forceinline__ int v_slot(int c, int row) {
  return C::kChunks == 16 ? c ^ ((row & 3) << 2) : c ^ (((row >> 1) & 1) << 2);
}

__device__ __forceinline__ float xor32(float x, int lane) {
  return __uint_as_float(xor_lanes(__float_as_uint(x), 32, lane));
}

__device__ __forceinline__ uint64_t shfl64(uint64_t x, int src) {
  return ((uint64_t)(uint32_t)__shfl((uint32_t)(x >> 32), src) << 32) | (uint32_t)__shfl((uint32_t)x, src);
}

// Tiles of a sequence: its keys are the cache's and right behind them the tree's.
template <class C>
__device__ __forceinline__ int seq_tiles(const AttnArgs& a, int b) {
  return (a.c.len(b) + a.T + C::kTile - 1) / C::kTile;
}

// Parts that `total` tiles are cut into: from 32 a sequence on of four tiles or more, as the join reads every
// row once for each (68 rows of 128, 4001 keys: 20.4 us against 23.0).
__device__ __forceinline__ int parts_of(const AttnArgs& a, int total) {
  return min(min(a.G, total), max(32 * a.batch, (total + 3) / 4));
}

// a b / c rounded down, for a b < 2^53 and c < 2^32: the quotient is at least 1 / c away from
// the next whole number above it, far more than its rounding in 64 bits.
__device__ __forceinline__ int mul_div(int a, int b, int c) { return (int)((double)a * (double)b / (double)c); }

// Total tiles, and the sequence that holds tile `want(total)` with the tiles before it.
struct Where {
  int total, before, seq;
};
// Up to 64 sequences: a lane each, every wave by itself.
template <class C, class F>
__device__ __forceinline__ Where locate_wave(const AttnArgs& a, int lane, F want) {
  const int mine = lane < a.batch ? seq_tiles<C>(a, lane) : 0;
  int upto = mine;  // tiles of the sequences up to this lane's
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl(upto, max(lane - d, 0));
    if (lane >= d) upto += v;
  }
  Where w;
  w.total = __builtin_amdgcn_readlane(upto, 63);
  const int x = want(w.total);
  w.seq = __popcll(__ballot(lane < a.batch && upto <= x));
  w.before = __builtin_amdgcn_readlane(upto - mine, w.seq);
  return w;
}
// More: a run of sequences per thread; scratch: kThreads + 2 values of LDS.
template <class C, class F>
__device__ __forceinline__ Where locate(const AttnArgs& a, int* scratch, F want) {
  if (a.batch == 1) return Where{seq_tiles<C>(a, 0), 0, 0};
  if (a.batch <= 64) return locate_wave<C>(a, threadIdx.x & 63, want);
  constexpr int kThreads = C::kThreads;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int lo = threadIdx.x * per, hi = min(lo + per, a.batch);
  int mine = 0;
#pragma unroll 1
  for (int b = lo; b < hi; ++b) mine += seq_tiles<C>(a, b);
  scratch[threadIdx.x] = mine;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll 8
  for (int i = 0; i < kThreads; ++i) {
    const int v = scratch[i];
    if (i < (int)threadIdx.x) before += v;
    total += v;
  }
  const int x = want(total);
  if (x >= before && x < before + mine) {
    int b = lo, at = before;
#pragma unroll 1
    for (int n; x >= at + (n = seq_tiles<C>(a, b)); ++b) at += n;
    scratch[kThreads] = at;
    scratch[kThreads + 1] = b;
  }
  __syncthreads();
  return Where{total, scratch[kThreads], scratch[kThreads + 1]};
}

// The nodes that node `lane` (parent p; none: -2) sees, as bits (none for an unused node):
// itself and, by doubling along the parents, its ancestors.
__device__ __forceinline__ uint64_t tree_bits(int p, int T, int lane) {
  const bool used = p >= -1 && p < lane;
  uint64_t bits = used ? 1ull << lane : 0;
  if (!used) p = -1;
#pragma unroll 1
  for (int reach = 1; reach < T; reach *= 2) {
    const int src = p < 0 ? lane : p;
    const uint32_t lo = __shfl((uint32_t)bits, src), hi = __shfl((uint32_t)(bits >> 32), src);
    const int pp = __shfl(p, src);
    if (p >= 0) {
      bits |= ((uint64_t)hi << 32) | lo;
      p = pp;
    }
  }
  return bits;
}

template <class C>
struct State {
  f32x16 o[C::D / 32];  // o[dt][i]: d = 32 dt + 8 (i / 4) + 4 half + i % 4 of this lane's row
  float m, l;           // maximum (in powers of two; -inf: nothing seen) and sum
};

// Clears the V rows of keys that are not `there`: a weight of zero must not meet what is
// not finite in them.  In the rows of `nodes` also what is not finite; says whether this lane
// found any.
template <class C>
__device__ __forceinline__ bool clear_rows(char* vt, int rw, int lane, uint64_t there, uint64_t nodes) {
  bool odd = false;
#pragma unroll 1
  for (int u = rw * 64 + lane; u < C::kKeys * C::kChunks; u += 64 * C::RW) {
    const int row = u / C::kChunks;
    uint4* at = reinterpret_cast<uint4*>(vt + row * C::kRowBytes + 16 * (u % C::kChunks));
    if (!((there >> row) & 1)) {
      *at = make_uint4(0, 0, 0, 0);
    } else if ((nodes >> row) & 1) {
      uint4 v = *at;
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      bool here = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u, here = true;
        if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu, here = true;
      }
      if (here) *at = make_uint4(w[0], w[1], w[2], w[3]), odd = true;
    }
  }
  return odd;
}

typedef __attribute__((address_space(3))) char* lds_t;

// Where a lane's fragments of a tile lie, from the start of its K (or V) rows.  K: key
// `lane % 32`, chunk 2 x + half at k ^ 32 x.  V: keys 4 half + lane / 4 % 4 (+ 8, 16, ...),
// the 16 d of the lane's group of 16 in 64-byte block dt at v[dt].
template <class C>
struct Frag {
  uint32_t k, v[C::D / 32];
  __device__ __forceinline__ explicit Frag(int lane) {
    const int r = lane & 31, h = lane >> 5, q = (lane >> 2) & 3;
    k = r * C::kRowBytes + 16 * k_slot<C>(h, r);
#pragma unroll
    for (int dt = 0; dt < C::D / 32; ++dt)
      v[dt] = (4 * h + q) * C::kRowBytes + 16 * v_slot<C>(4 * dt + 2 * ((lane >> 4) & 1), q) + 8 * (lane & 3);
  }
};

// A step's keys: scores, weights, sums.  `masked`: only the keys whose bit is set in this
// lane's `sees` count.  Its tiles of 32 keys go side by side, so that one's matrix products
// run under the other's exponentials.
template <class C>
__device__ __forceinline__ void step(lds_t kt, lds_t vt, const Frag<C>& at, const bf16x8 (&qf)[C::D / 16], float c2,
                                     int lane, bool masked, uint64_t sees, State<C>& st) {
  typedef __attribute__((address_space(3))) const bf16x8* k_ptr;
  typedef __attribute__((address_space(3))) s16x4* tr_ptr;
  constexpr int kSub = 32 * C::kRowBytes;  // bytes of 32 keys
  f32x16 s[C::SUB];
#pragma unroll
  for (int sub = 0; sub < C::SUB; ++sub) {
    s[sub] = f32x16{};
#pragma unroll
    for (int x = 0; x < C::D / 16; ++x) {
      const bf16x8 kf = *(k_ptr)(kt + sub * kSub + (at.k ^ (32 * x)));
      s[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[x], s[sub], 0, 0, 0);
    }
  }
  if (masked) {
#pragma unroll
    for (int sub = 0; sub < C::SUB; ++sub) {
      const uint32_t bits = (uint32_t)(sees >> (32 * sub)) >> (4 * (lane >> 5));
#pragma unroll
      for (int i = 0; i < 16; ++i) s[sub][i] = (bits >> (8 * (i / 4) + i % 4)) & 1 ? s[sub][i] : -INFINITY;
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int i = 1; i < 16 * C::SUB; ++i) top = fmaxf(top, s[i / 16][i % 16]);
  top = fmaxf(top, xor32(top, lane)) * c2;
  // A row's maximum follows only when it lags by more than 2^8: weights are then at most
  // 2^8 and nothing is lost, and most steps leave the sums alone.
  if (__ballot(top > st.m + kLag)) {
    const float m = fmaxf(st.m, top);
    const float f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.l *= f;
#pragma unroll
    for (int dt = 0; dt < C::D / 32; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[dt][i] *= f;
    st.m = m;
  }
  const float m0 = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
  for (int sub = 0; sub < C::SUB; ++sub) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[sub][i] = __builtin_amdgcn_exp2f(fmaf(s[sub][i], c2, -m0));
      sum += s[sub][i];
    }
    st.l += sum;
#pragma unroll
    for (int kc = 0; kc < 2; ++kc) {
      union {
        bf16x2 two[4];
        bf16x8 all;
      } pf;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pf.two[i] = __builtin_convertvector(f32x2{s[sub][8 * kc + 2 * i], s[sub][8 * kc + 2 * i + 1]}, bf16x2);
      }
#pragma unroll
      for (int dt = 0; dt < C::D / 32; ++dt) {
        union {
          s16x4 half[2];
          bf16x8 all;
        } vf;
#pragma unroll
        for (int z = 0; z < 2; ++z)
          vf.half[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (tr_ptr)(vt + sub * kSub + at.v[dt] + (16 * kc + 8 * z) * C::kRowBytes));
        st.o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf.all, pf.all, st.o[dt], 0, 0, 0);
      }
    }
  }
}

// What the waves of a key group wrote to LDS is there for all of them.
template <class C>
__device__ __forceinline__ void group_sync() {
  if constexpr (C::RW > 1)
    big::bar();
  else
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

template <class C>
__global__ __launch_bounds__(C::kThreads, C::kMinWaves) void tree_attention_kernel(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::kLds];
  __shared__ int scratch[C::kThreads + 2];
  __shared__ int s_odd[C::KW];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int kw = wave / C::RW, rw = wave % C::RW;
  const int Hkv = a.c.kv_heads;
  // Workgroups go round the eight XCDs in turn: the row tiles of a part are eight apart, so
  // that they run side by side on one XCD and read the part's keys into its L2 once.
  const int turn = blockIdx.x / (8 * a.row_tiles), rt = blockIdx.x / 8 % a.row_tiles;
  const int unit = turn * 8 + blockIdx.x % 8;  // (head, part)
  if (unit >= Hkv * a.G) return;
  const int head = unit / a.G, g = unit % a.G;
  // part g: the tiles x .. x_end - 1, at least one
  int x = 0, x_end, seq = g, before = 0, total = 0, parts = 0;
  if (a.whole) {
    x_end = seq_tiles<C>(a, g);
  } else {
    const Where w = locate<C>(a, scratch, [&](int total) {
      return min(mul_div(g, total, parts_of(a, total)), total - 1);
    });
    total = uniform(w.total), parts = parts_of(a, total);
    if (g >= parts) return;
    x = uniform(mul_div(g, total, parts));
    x_end = uniform(mul_div(g + 1, total, parts));
    seq = uniform(w.seq), before = uniform(w.before);
  }
  const int steps = x_end - x;
  if constexpr (C::kEven) __builtin_amdgcn_s_setprio(3);
  const int rows = a.T * a.group;
  const int row = rt * C::kRows + 32 * rw + (lane & 31);
  const int qrow = min(row, rows - 1), t = qrow / a.group, gh = qrow % a.group;
  const int h = lane >> 5;
  const int64_t slot0 = ((int64_t)head * a.row_tiles + rt) * 2 * a.G;
  const Frag<C> at(lane);
  const uint32_t ring0 = lds_addr(lds) + kw * C::S * C::kStage;
  const uint32_t pages0 = lds_addr(lds) + C::kRing + wave * (C::kAhead + 1) * C::kPages;
  const char* ring = lds + kw * C::S * C::kStage;
  const char* my_pages = lds + C::kRing + wave * (C::kAhead + 1) * C::kPages;
  const int64_t page_bytes = ((int64_t)Hkv << a.c.page_shift) * C::kRowBytes;

  while (x < x_end) {
    const int len = a.c.len(seq);
    const int tiles = (len + a.T + C::kTile - 1) / C::kTile;
    const int first = x - before, last = min(tiles, x_end - before);
    // for the join: tile y is in part floor(((y + 1) parts - 1) / total)
    if (a.pieces && first == 0 && head == 0 && rt == 0 && threadIdx.x == 0)
      a.pieces[seq] = make_int2(g, (int)(((double)(before + tiles) * (double)parts - 1.0) / (double)total));
    const int n = last - first;  // steps
    // nothing cached: no entry of the table counts, and look-ups read the length (unused) in its place
    const int32_t* table = len > 0 ? a.c.block_table + (int64_t)seq * a.c.table_width : a.c.lens + seq;
    // Pages of a step's keys or more: they lie in one, read by a scalar load a step ahead.
    const bool wide = (1 << a.c.page_shift) >= C::kKeys;
    auto wide_page = [&](int i) {
      typedef const __attribute__((address_space(4))) int32_t* const_ptr;
      const int key = min((first + i) * C::kTile + kw * C::kKeys, len - 1);
      return *(const_ptr)(table + (max(key, 0) >> a.c.page_shift));
    };
    // Smaller ones: the pages of step i's keys, into its slot of this wave's ring.
    auto look_up = [&](int i) {
      const int key = min((first + i) * C::kTile + kw * C::kKeys + (lane & (C::kKeys - 1)), len - 1);
      dma4(table + (max(key, 0) >> a.c.page_shift),
           __builtin_amdgcn_readfirstlane(pages0 + i % (C::kAhead + 1) * C::kPages));
    };
    // This wave's share of step i's K and V rows.
    auto load = [&](int i, int wide_id) {
      const int base = (first + i) * C::kTile + kw * C::kKeys;
      const int rr = lane / C::kChunks, slot = lane % C::kChunks;
      const uint32_t to = ring0 + i % C::S * C::kStage;
      const int* pages = reinterpret_cast<const int*>(my_pages + i % (C::kAhead + 1) * C::kPages);
      const char* kp = static_cast<const char*>(a.c.k_pages);
      const char* vp = static_cast<const char*>(a.c.v_pages);
      const int in_page = (1 << a.c.page_shift) - 1;
      if (base + C::kKeys > len) {  // nodes among them, or nothing
#pragma unroll
        for (int u = 0; u < C::kLoads; ++u) {
          int j = rw + C::RW * u;
          if (C::kLoadsAll % C::RW != 0) j = min(j, C::kLoadsAll - 1);  // the last rows again
          const int row = j * C::kRowsPerLoad + rr, key = base + row;
          const int page = min(max(wide ? wide_id : pages[row], 0), a.c.n_pages - 1);
          const int64_t cached = (int64_t)page * page_bytes +
                                 (int64_t)((head << a.c.page_shift) + (key & in_page)) * C::kRowBytes;
          const int64_t node = (((int64_t)seq * a.T + min(key - len, a.T - 1)) * Hkv + head) * C::kRowBytes;
          const bool tree = key >= len;
          dma16<C::kOnce>((tree ? reinterpret_cast<const char*>(a.k_new) + node : kp + cached) + 16 * k_slot<C>(slot, row),
                          __builtin_amdgcn_readfirstlane(to + j * 1024));
          dma16<C::kOnce>((tree ? reinterpret_cast<const char*>(a.v_new) + node : vp + cached) + 16 * v_slot<C>(slot, row),
                          __builtin_amdgcn_readfirstlane(to + C::kHalf + j * 1024));
        }
        return;
      }
      if (wide) {
        const int page = min(max(wide_id, 0), a.c.n_pages - 1);
        const int64_t off = (int64_t)page * page_bytes +
                            (int64_t)((head << a.c.page_shift) + (base & in_page)) * C::kRowBytes;
#pragma unroll
        for (int u = 0; u < C::kLoads; ++u) {
          int j = rw + C::RW * u;
          if (C::kLoadsAll % C::RW != 0) j = min(j, C::kLoadsAll - 1);
          const int row = j * C::kRowsPerLoad + rr;
          dma16<C::kOnce>(kp + off + row * C::kRowBytes + 16 * k_slot<C>(slot, row), __builtin_amdgcn_readfirstlane(to + j * 1024));
          dma16<C::kOnce>(vp + off + row * C::kRowBytes + 16 * v_slot<C>(slot, row),
                          __builtin_amdgcn_readfirstlane(to + C::kHalf + j * 1024));
        }
        return;
      }
#pragma unroll
      for (int u = 0; u < C::kLoads; ++u) {
        int j = rw + C::RW * u;
        if (C::kLoadsAll % C::RW != 0) j = min(j, C::kLoadsAll - 1);
        const int row = j * C::kRowsPerLoad + rr;
        const int page = min(max(pages[row], 0), a.c.n_pages - 1);
        const int64_t off = (int64_t)page * page_bytes +
                            (int64_t)((head << a.c.page_shift) + ((base + row) & in_page)) * C::kRowBytes;
        dma16<C::kOnce>(kp + off + 16 * k_slot<C>(slot, row), __builtin_amdgcn_readfirstlane(to + j * 1024));
        dma16<C::kOnce>(vp + off + 16 * v_slot<C>(slot, row), __builtin_amdgcn_readfirstlane(to + C::kHalf + j * 1024));
      }
    };
    if (!wide) {
#pragma unroll 1
      for (int i = 0; i < C::S - 1; ++i) look_up(i);
    }
    const int64_t qoff = (((int64_t)seq * a.T + t) * Hkv * a.group + head * a.group + gh) * C::D;
    bf16x8 qf[C::D / 16];
#pragma unroll
    for (int i = 0; i < C::D / 16; ++i) qf[i] = *reinterpret_cast<const bf16x8*>(a.q + qoff + 16 * i + 8 * h);
    uint64_t sees = 0, used = 0;  // of this lane's row; all used nodes
    if (last == tiles || last * C::kTile > len) {
      const uint64_t bits = tree_bits(lane < a.T ? a.parents[(int64_t)seq * a.T + lane] : -2, a.T, lane);
      sees = shfl64(bits, t);
      used = __ballot(bits != 0);
    }
    State<C> st;
#pragma unroll
    for (int dt = 0; dt < C::D / 32; ++dt) st.o[dt] = f32x16{};
    st.m = -INFINITY;
    st.l = 0.f;
    big::wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    int next_page = wide ? wide_page(0) : 0;
#pragma unroll 1
    for (int i = 1 - C::S; i < n; ++i) {
      if (i >= 0) {
        // step i's rows are here, and the pages of step i + S - 1; everyone is done with the stage before
        if (i + C::S - 1 <= n)
          big::wait_vmcnt<C::kInFlight>();
        else
          big::wait_vmcnt<0>();
        group_sync<C>();
      }
      if (i + C::S - 1 < n) {
        if (!wide) look_up(i + C::kAhead);
        load(i + C::S - 1, next_page);
        if (wide) next_page = wide_page(i + C::S);
      }
      if (i < 0) continue;
      if constexpr (C::kEven) {
        const int rest = x_end - (before + first + i);
        if (rest == steps / 2) __builtin_amdgcn_s_setprio(2);
        if (rest == steps / 4) __builtin_amdgcn_s_setprio(1);
        if (rest == steps / 8) __builtin_amdgcn_s_setprio(0);
      }
      char* kt = const_cast<char*>(ring) + i % C::S * C::kStage;
      char* vt = kt + C::kHalf;
      const int base = (first + i) * C::kTile + kw * C::kKeys;  // first key
      const int cached = len - base, left = cached + a.T;         // of the cache's, of all, from there on
      const bool masked = cached < C::kKeys;
      uint64_t see = ~0ull;
      if (masked) {
        const uint64_t old = cached > 0 ? (1ull << cached) - 1 : 0;  // cached < 64
        auto placed = [&](uint64_t nodes) {
          return cached >= 0 ? nodes << cached : left > 0 ? nodes >> -cached : 0;
        };
        const uint64_t nodes = placed(used);
        see = old | placed(sees);
        const bool odd = clear_rows<C>(vt, rw, lane, old | nodes, nodes);
        if (rw == 0 && lane == 0) s_odd[kw] = 0;
        group_sync<C>();
        if (__ballot(odd) && lane == 0) s_odd[kw] = 1;
        group_sync<C>();
      }
      if (left > 0) step<C>((lds_t)kt, (lds_t)vt, at, qf, a.c2, lane, masked, see, st);
      if (masked && left > 0 && s_odd[kw]) {
        // what is not finite in a node's V (cleared above) reaches the rows that see the node, and no others
#pragma unroll 1
        for (int k = max(cached, 0); k < min(C::kKeys, left); ++k) {
          const uint16_t* v = a.v_new + (((int64_t)seq * a.T + k - cached) * Hkv + head) * C::D;
          const bool on = (see >> k) & 1;
#pragma unroll
          for (int dt = 0; dt < C::D / 32; ++dt) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint16_t u = v[32 * dt + 8 * (e / 4) + 4 * h + e % 4];
              if ((u & 0x7f80) == 0x7f80 && on) st.o[dt][e] += bf16_to_f32(u);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }
    __syncthreads();

    // A lane's values in fours, d = 4 h + 8 u of its row.  Key groups: joined through LDS, a
    // share of the fours to each wave (one wave for all of them: 1.8 us against 1.1 for a
    // single token).
    const bool whole = first == 0 && last == tiles;
    constexpr int kFours = C::D / 8, kMine = kFours / C::KW;
    float m = st.m, l = st.l + xor32(st.l, lane);
    f32x4 o[kMine];
    if constexpr (C::KW == 1) {
#pragma unroll
      for (int u = 0; u < kMine; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[u][e] = st.o[u / 4][4 * (u % 4) + e];
    } else {
      static_assert(C::RW == 1, "a wave has all rows");
      f32x4* sh = reinterpret_cast<f32x4*>(lds) + lane;
      f32x2* ml = reinterpret_cast<f32x2*>(lds + C::KW * kFours * 1024) + lane;
      if (row < rows) {
#pragma unroll
        for (int u = 0; u < kFours; ++u)
          sh[64 * (kFours * wave + u)] =
              f32x4{st.o[u / 4][4 * (u % 4)], st.o[u / 4][4 * (u % 4) + 1], st.o[u / 4][4 * (u % 4) + 2], st.o[u / 4][4 * (u % 4) + 3]};
        ml[64 * wave] = f32x2{m, l};
      }
      __syncthreads();
      if (row < rows) {
        f32x2 of[C::KW];
        m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < C::KW; ++k) {
          of[k] = ml[64 * k];
          m = fmaxf(m, of[k].x);
        }
#pragma unroll
        for (int u = 0; u < kMine; ++u) o[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < C::KW; ++k) {
          const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(of[k].x - m);
          l = fmaf(of[k].y, f, l);
#pragma unroll
          for (int u = 0; u < kMine; ++u) {
            const f32x4 v = sh[64 * (kFours * k + kMine * wave + u)];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[u][e] = fmaf(v[e], f, o[u][e]);
          }
        }
      }
    }
    if (row < rows) {
      const int d0 = 8 * kMine * kw + 4 * h;
      if (whole) {
        const float inv = sees && l != 0.f ? 1.0f / l : 0.f;
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = inv != 0.f ? o[u][e] * inv : 0.f;
          union {
            bf16x2 b[2];
            uint2 u;
          } pk;
          pk.b[0] = __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2);
          pk.b[1] = __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2);
          *reinterpret_cast<uint2*>(a.out + qoff + d0 + 8 * u) = pk.u;
        }
      } else {
        const int64_t slot = (slot0 + 2 * g + (first == 0 ? 1 : 0)) * C::kRows + 32 * rw + (lane & 31);
#pragma unroll
        for (int u = 0; u < kMine; ++u) *reinterpret_cast<f32x4*>(a.part_o + slot * C::D + d0 + 8 * u) = o[u];
        if (h == 0 && kw == 0)
          *reinterpret_cast<f32x2*>(a.part_ml + 2 * slot) = f32x2{m, last == tiles && !sees ? kUnused : l};
      }
    }
    __syncthreads();
    x = before + last;
    before += tiles;
    ++seq;
  }
}

// Sequences cut over several workgroups: their pieces joined.  16 lanes hold a row's D
// values and take every `spread`-th of its pieces, two at a time, statistics and values in
// one go: ceil(pieces / (2 spread)) rounds of memory latency for a row.  16 rows a workgroup for few
// pieces (spread 1), 4 for more (a wave a row), or one; by the parts for each sequence on average, so
// a long sequence among many short ones takes more rounds than it would have to.
template <class C>
__global__ __launch_bounds__(256) void tree_attention_join_kernel(AttnArgs a) {
  constexpr int kPer = C::D / 16;  // values of a lane
  constexpr int kAtOnce = 2;       // pieces in flight, per group of lanes
  __shared__ float tops[4], sums[4][kPer + 1][16];
  const int spread = a.spread;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int Hkv = a.c.kv_heads, rows = a.T * a.group;
  const int each = 16 / spread, chunks = (rows + each - 1) / each;
  const int seq = blockIdx.x / (Hkv * chunks), head = blockIdx.x / chunks % Hkv;
  const int row0 = blockIdx.x % chunks * each;
  const int2 at = a.pieces[seq];
  const int g0 = uniform(at.x), g1 = uniform(at.y);
  if (g0 == g1) return;  // one piece: written already
  const int sub = 4 * wave + (lane >> 4);  // of the workgroup's 16 groups of lanes
  const int row = row0 + sub / spread;
  const int qrow = min(row, rows - 1), t = qrow / a.group;
  const int64_t slot0 = ((int64_t)head * a.row_tiles + qrow / C::kRows) * 2 * a.G;
  const float end = a.part_ml[2 * ((slot0 + 2 * g1) * C::kRows + qrow % C::kRows) + 1];
  float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) o[e] = 0.f;
  for (int g = g0 + sub % spread; g <= g1; g += kAtOnce * spread) {
    f32x2 ml[kAtOnce];
    f32x4 v[kAtOnce][kPer / 4];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int gk = min(g + k * spread, g1);
      const int64_t slot = (slot0 + 2 * gk + (gk == g0 ? 1 : 0)) * C::kRows + qrow % C::kRows;
      ml[k] = *reinterpret_cast<const f32x2*>(a.part_ml + 2 * slot);
#pragma unroll
      for (int e = 0; e < kPer / 4; ++e)
        v[k][e] = *reinterpret_cast<const f32x4*>(a.part_o + slot * C::D + (lane & 15) * kPer + 4 * e);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);  // a piece counted again changes no maximum
    const float m0 = top == -INFINITY ? 0.f : top;
    const float was = __builtin_amdgcn_exp2f(m - m0);
    l *= was;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] *= was;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (g + k * spread <= g1) {
        const float f = __builtin_amdgcn_exp2f(ml[k].x - m0);
        l = fmaf(ml[k].y, f, l);
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = fmaf(v[k][e / 4][e % 4], f, o[e]);
      }
    }
    m = top;
  }
  if (spread > 1) {
    float top = m;
#pragma unroll
    for (int j = 16; j <= 32; j += 16) top = fmaxf(top, __uint_as_float(xor_lanes(__float_as_uint(top), j, lane)));
    if (spread > 4) {
      if (lane == 0) tops[wave] = top;
      __syncthreads();
      top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    }
    const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
    l *= f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] *= f;
#pragma unroll
    for (int j = 16; j <= 32; j += 16) {
      l += __uint_as_float(xor_lanes(__float_as_uint(l), j, lane));
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] += __uint_as_float(xor_lanes(__float_as_uint(o[e]), j, lane));
    }
    if (spread > 4) {
      if (lane < 16) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) sums[wave][e][lane] = o[e];
        sums[wave][kPer][lane] = l;
      }
      __syncthreads();
      l = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        l += sums[w][kPer][lane & 15];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] += sums[w][e][lane & 15];
      }
    }
  }
  if (row >= rows || sub % spread > 0) return;
  const bool some = end != kUnused && l != 0.f;
  const float inv = some ? 1.0f / l : 0.f;
  union {
    bf16x2 b[kPer / 2];
    uint2 u[kPer / 4];
  } pk;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    pk.b[e / 2] = __builtin_convertvector(some ? f32x2{o[e] * inv, o[e + 1] * inv} : f32x2{0.f, 0.f}, bf16x2);
  uint16_t* out = a.out + (((int64_t)seq * a.T + t) * Hkv * a.group + head * a.group + row % a.group) * C::D +
                  (lane & 15) * kPer;
#pragma unroll
  for (int e = 0; e < kPer / 4; ++e) reinterpret_cast<uint2*>(out)[e] = pk.u[e];
}

template <class C>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  tree_attention_kernel<C><<<dim3((uint32_t)(cdiv((int64_t)a.G * a.c.kv_heads, 8) * 8 * a.row_tiles)), dim3(C::kThreads), 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.pieces) return e;
  tree_attention_join_kernel<C><<<
      dim3((uint32_t)(a.batch * a.c.kv_heads * cdiv(a.T * a.group, 16 / a.spread))), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

// Query rows of a head, and the configurations that take them: up to 32 the waves have keys
// of their own; more rows share them, 128 to a workgroup.  64 keys a step and two stages
// against 32 keys and four (a barrier for every 16 KB): 203 us against 217 at 64 sequences x 17
// nodes x 8192 keys, head 128; 147 against 162 at 2 x 64 nodes x 131001 keys, head 64.  65 to 96 rows of
// 128: three waves (211 us against 214 by four at 64 x 17 nodes x 8192 keys); of 64: four, an idle one
// among them (120 against 144: by three, twelve waves on a CU, the registers do not suffice; of 18 more
// sizes all gain, 2 x 28 nodes x 3 heads x 23520 keys 16.6 against 17.5, 64 x 17 nodes x 5 heads x 1000 keys
// 28.3 against 36.8).
template <int D, class F>
auto with_cfg(int64_t rows, F f) {
  if (rows <= 32) return f(Cfg<D, 4, 1, D == 64 ? 3 : 2, 1>{});
  if (rows <= 64) return f(Cfg<D, 1, 2, 2, 2>{});
  if constexpr (D == 128)
    if (rows <= 96) return f(Cfg<D, 1, 3, 2, 2>{});
  if (rows <= 128) return f(Cfg<D, 1, 4, 2, 2>{});
  return f(Cfg<D, 1, 4, 2, 2, false>{});
}

}  // namespace

AttnPlan plan_tree_attention(const CacheView& c, int64_t batch, int64_t T, int64_t group, int64_t D) {
  const int64_t rows = T * group;
  auto plan = [&](auto cfg) {
    typedef decltype(cfg) C;
    AttnPlan p{};
    p.row_tiles = cdiv(rows, C::kRows);
    // tiles when all lengths are full: no more parts than that
    const int64_t each = cdiv(((int64_t)c.table_width << c.page_shift) + T, (int64_t)C::kTile), most = batch * each;
    p.G = 256 * C::kGroups / (p.row_tiles * c.kv_heads);
    p.G = p.G < 1 ? 1 : p.G > most ? most : p.G;
    // Few tiles a sequence at most, by the table's width (the lengths are on the device: a table for more
    // keys cuts sequences however short they are): a part for each and no join (4 x 9 nodes, page 256: 8.0 us
    // against 10.2; 39 x 33 nodes, up to 61 keys: 17.8 against 24.4; 13 x 56 nodes, 7 heads, 243 keys: 16.2
    // against 27.9; at worst 2 x 18 nodes, 3 heads, 115 keys: 14.0 against 12.8).
    p.whole = each <= 4 || (each <= 8 && batch * c.kv_heads * p.row_tiles >= 48);
    if (p.whole) p.G = batch;
    const int64_t slots = (int64_t)c.kv_heads * p.row_tiles * 2 * p.G * C::kRows;
    const bool join = p.G > 1 && !p.whole;
    p.part_bytes = join ? align_up((size_t)(slots * D) * 4, 256) : 0;
    p.ml_bytes = join ? align_up((size_t)slots * 8, 256) : 0;
    p.ws_bytes = join ? p.part_bytes + p.ml_bytes + align_up((size_t)batch * 8, 256) : 0;
    return p;
  };
  return D == 64 ? with_cfg<64>(rows, plan) : with_cfg<128>(rows, plan);
}

hipError_t launch_tree_attention(const AttnPlan& p, const CacheView& c, const void* q, const void* k_new,
                                 const void* v_new, const int32_t* parents, int64_t batch, int64_t T, int64_t group,
                                 int64_t D, double scale, void* out, void* ws, hipStream_t stream) {
  AttnArgs a{};
  a.c = c;
  a.q = static_cast<const uint16_t*>(q);
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.parents = parents;
  a.out = static_cast<uint16_t*>(out);
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part_bytes);
  a.pieces = p.ws_bytes == 0 ? nullptr : reinterpret_cast<int2*>(static_cast<char*>(ws) + p.part_bytes + p.ml_bytes);
  a.whole = p.whole;
  a.batch = (int)batch;
  a.T = (int)T;
  a.group = (int)group;
  a.G = (int)p.G;
  a.row_tiles = (int)p.row_tiles;
  a.spread = p.G >= 32 * batch ? 16 : p.G >= 8 * batch ? 4 : 1;  // by its pieces
  a.c2 = attention_c2(scale);
  auto run = [&](auto cfg) { return launch<decltype(cfg)>(a, stream); };
  return D == 64 ? with_cfg<64>(T * group, run) : with_cfg<128>(T * group, run);
}

}  // namespace dfs
