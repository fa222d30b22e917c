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
// to bf16 for the matrix cores (relative 2^-9 per weight, as the output's own rounding);
// scores, maxima, sums and O stay in fp32.
//
// K and V tiles go from memory straight into LDS, two stages: one lands while the other is
// computed.  Waves of a workgroup: RW row groups of 32 rows share a key tile, KW key groups
// take tiles of their own (few rows) and are joined at the end.  Work is split along the
// keys: the tiles of all sequences in a row are cut evenly over the workgroups of a head,
// whatever the lengths are; sequences that were cut are joined by a second kernel from
// fp32 partial results.
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

constexpr int kMaxNodes = 64;
constexpr float kLag = 8.0f;  // a maximum may lag this far (in powers of two) before sums are rescaled

struct AttnArgs {
  CacheView c;
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* parents;
  uint16_t* out;
  float* part_o;   // [Hkv, row tiles, 2 G, rows of a tile, D]
  float* part_ml;  // [Hkv, row tiles, 2 G, rows of a tile, 2]
  int batch, T, group, G, row_tiles;
  float c2;  // scale * log2(e)
};

template <int D_, int KW_, int RW_, int TK_>
struct Cfg {
  static constexpr int D = D_, KW = KW_, RW = RW_, TK = TK_;
  static constexpr int kWaves = KW * RW, kThreads = 64 * kWaves;
  static constexpr int kRows = 32 * RW;            // query rows of a workgroup
  static constexpr int kTile = KW * TK;            // keys per step
  static constexpr int kRowBytes = 2 * D;          // of a key in LDS
  static constexpr int kChunks = kRowBytes / 16;   // 16-byte chunks
  static constexpr int kRowsPerLoad = 64 / kChunks;
  static constexpr int kHalf = TK * kRowBytes;     // K (or V) of a key group's step
  static constexpr int kLoadsAll = 2 * TK / kRowsPerLoad;              // of a key group per step
  static constexpr int kLoads = (kLoadsAll + RW - 1) / RW;             // of a wave (some repeated when uneven)
  static constexpr int kStage = KW * 2 * kHalf;
  static constexpr int kLds = 2 * kStage;
  static constexpr int kMinWaves = kLds > 81920 ? 1 : 2;  // per SIMD: one workgroup of a CU, or two
};

// 16 bytes per lane from memory straight into LDS at lds_base + 16 lane.
__device__ __forceinline__ void dma16(const void* p, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p), "s"(lds_base) : "memory", "m0");
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

// Tiles of a sequence: its cache's, and the tree's.
__device__ __forceinline__ int seq_tiles(int len, int tile) { return (len + tile - 1) / tile + 1; }

// Total tiles, and the sequence that holds tile `want(total)` with the tiles before it.
struct Where {
  int64_t total, before;
  int seq;
};
template <int kThreads, class F>
__device__ __forceinline__ Where locate(const AttnArgs& a, int tile, int64_t* scratch, F want) {
  // each thread a run of sequences; scratch: kThreads + 2 values of LDS
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int lo = threadIdx.x * per, hi = min(lo + per, a.batch);
  int64_t mine = 0;
  for (int b = lo; b < hi; ++b) mine += seq_tiles(a.c.len(b), tile);
  scratch[threadIdx.x] = mine;
  __syncthreads();
  int64_t before = 0, total = 0;
  const int active = min(kThreads, (a.batch + per - 1) / per);
  for (int i = 0; i < active; ++i) {
    const int64_t v = scratch[i];
    if (i < (int)threadIdx.x) before += v;
    total += v;
  }
  const int64_t x = want(total);
  if (x >= before && x < before + mine) {
    int b = lo;
    int64_t at = before;
    for (int n; x >= at + (n = seq_tiles(a.c.len(b), tile)); ++b) at += n;
    scratch[kThreads] = at;
    scratch[kThreads + 1] = b;
  }
  __syncthreads();
  Where w{total, scratch[kThreads], (int)scratch[kThreads + 1]};
  __syncthreads();
  return w;
}

// The nodes that node `lane` sees, as bits (none for an unused node): itself and, by
// doubling along the parents, its ancestors.
__device__ __forceinline__ uint64_t tree_bits(const int32_t* parents, int T, int lane) {
  int p = lane < T ? parents[lane] : -2;
  const bool used = p >= -1 && p < lane;
  uint64_t bits = used ? 1ull << lane : 0;
  if (!used) p = -1;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
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

__device__ __forceinline__ uint64_t shfl64(uint64_t x, int src) {
  return ((uint64_t)(uint32_t)__shfl((uint32_t)(x >> 32), src) << 32) | (uint32_t)__shfl((uint32_t)x, src);
}

template <class C>
struct State {
  f32x16 o[C::D / 32];  // o[dt][i]: d = 32 dt + 8 (i / 4) + 4 half + i % 4 of this lane's row
  float m, l;           // maximum (in powers of two; -inf: nothing seen) and sum
};

// Loads of one step into `stage`: this wave's share of its key group's K and V rows.
// row_of(key of the tile) gives the row's K address; V lies `v_off` bytes after it.
template <class C, class F>
__device__ __forceinline__ void load_tile(char* group, int rw, int lane, F row_of) {
  const int rr = lane / C::kChunks, slot = lane % C::kChunks;
#pragma unroll
  for (int i = 0; i < C::kLoads; ++i) {
    int j = rw + C::RW * i;
    if (C::kLoadsAll % C::RW != 0) j = min(j, C::kLoadsAll - 1);
    const bool isv = j >= C::kLoadsAll / 2;
    const int row = (isv ? j - C::kLoadsAll / 2 : j) * C::kRowsPerLoad + rr;
    const int chunk = isv ? v_slot<C>(slot, row) : k_slot<C>(slot, row);
    const char* p = row_of(row, isv) + 16 * chunk;
    dma16(p, __builtin_amdgcn_readfirstlane(lds_addr(group + j * 1024)));
  }
}

// Clears the V rows of keys that are not `there`: a weight of zero must not meet what is
// not finite in them.  With `others` also what is not finite in the rows that are; says
// whether this lane found any.
template <class C>
__device__ __forceinline__ bool clear_rows(char* vt, int rw, int lane, uint64_t there, bool others) {
  bool odd = false;
#pragma unroll 1
  for (int u = rw * 64 + lane; u < C::TK * C::kChunks; u += 64 * C::RW) {
    const int row = u / C::kChunks;
    uint4* at = reinterpret_cast<uint4*>(vt + row * C::kRowBytes + 16 * (u % C::kChunks));
    if (!((there >> row) & 1)) {
      *at = make_uint4(0, 0, 0, 0);
    } else if (others) {
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

// A step's TK keys: scores, weights, sums.  `masked`: only the keys whose bit is set in
// this lane's `sees` count.
template <class C>
__device__ __forceinline__ void step(lds_t kt, lds_t vt, const Frag<C>& at, const bf16x8 (&qf)[C::D / 16], float c2,
                                     int lane, bool masked, uint64_t sees, State<C>& st) {
  typedef __attribute__((address_space(3))) const bf16x8* k_ptr;
  typedef __attribute__((address_space(3))) s16x4* tr_ptr;
  const int h = lane >> 5;
#pragma unroll
  for (int sub = 0; sub < C::TK / 32; ++sub) {
    f32x16 s = {};
#pragma unroll
    for (int x = 0; x < C::D / 16; ++x) {
      const bf16x8 kf = *(k_ptr)(kt + (at.k ^ (32 * x)) + sub * 32 * C::kRowBytes);
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[x], s, 0, 0, 0);
    }
    if (masked) {
      const uint32_t bits = (uint32_t)(sees >> (32 * sub)) >> (4 * h);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = (bits >> (8 * (i / 4) + i % 4)) & 1 ? s[i] : -INFINITY;
    }
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
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
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c2, -m0));
      sum += s[i];
    }
    st.l += sum;
#pragma unroll
    for (int kc = 0; kc < 2; ++kc) {
      union {
        bf16x2 two[4];
        bf16x8 all;
      } pf;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf.two[i] = __builtin_convertvector(f32x2{s[8 * kc + 2 * i], s[8 * kc + 2 * i + 1]}, bf16x2);
#pragma unroll
      for (int dt = 0; dt < C::D / 32; ++dt) {
        union {
          s16x4 half[2];
          bf16x8 all;
        } vf;
#pragma unroll
        for (int z = 0; z < 2; ++z)
          vf.half[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (tr_ptr)(vt + at.v[dt] + (32 * sub + 16 * kc + 8 * z) * C::kRowBytes));
        st.o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf.all, pf.all, st.o[dt], 0, 0, 0);
      }
    }
  }
}

template <class C>
__global__ __launch_bounds__(C::kThreads, C::kMinWaves) void tree_attention_kernel(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::kLds];
  __shared__ int64_t scratch[C::kThreads + 2];
  __shared__ int s_odd;
  if (threadIdx.x == 0) s_odd = 0;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int kw = wave / C::RW, rw = wave % C::RW;
  const int per_head = a.G * a.row_tiles;
  const int head = blockIdx.x / per_head, rt = blockIdx.x % per_head % a.row_tiles,
            g = blockIdx.x % per_head / a.row_tiles;
  // part g of min(G, total): the tiles x .. x_end - 1, at least one
  const Where w = locate<C::kThreads>(a, C::kTile, scratch, [&](int64_t total) {
    return min(g * total / min((int64_t)a.G, total), total - 1);
  });
  const int64_t parts = min((int64_t)a.G, w.total);
  if (g >= parts) return;
  int64_t x = g * w.total / parts;
  const int64_t x_end = (g + 1) * w.total / parts;
  const int Hkv = a.c.kv_heads, rows = a.T * a.group;
  const int row = rt * C::kRows + 32 * rw + (lane & 31);
  const int qrow = min(row, rows - 1), t = qrow / a.group, gh = qrow % a.group;
  const int h = lane >> 5;
  int seq = w.seq;
  int64_t before = w.before;
  const int64_t slot0 = ((int64_t)head * a.row_tiles + rt) * 2 * a.G;
  const Frag<C> at(lane);

  while (x < x_end) {
    const int len = a.c.len(seq);
    const int tiles = seq_tiles(len, C::kTile);
    const int first = (int)(x - before), last = (int)min((int64_t)tiles, x_end - before);
    const int32_t* table = a.c.block_table + (int64_t)seq * a.c.table_width;
    const int64_t qoff = (((int64_t)seq * a.T + t) * Hkv * a.group + head * a.group + gh) * C::D;
    bf16x8 qf[C::D / 16];
#pragma unroll
    for (int i = 0; i < C::D / 16; ++i) qf[i] = *reinterpret_cast<const bf16x8*>(a.q + qoff + 16 * i + 8 * h);
    State<C> st;
#pragma unroll
    for (int dt = 0; dt < C::D / 32; ++dt) st.o[dt] = f32x16{};
    st.m = -INFINITY;
    st.l = 0.f;
    const uint64_t bits = tree_bits(a.parents + (int64_t)seq * a.T, a.T, lane);
    const uint64_t sees = shfl64(bits, t);  // this lane's row
    const uint64_t used = __ballot(bits != 0);

    // the page of this lane's key of a tile; looked up one step before its loads
    auto page_of = [&](int tile) {
      const int key = min(tile * C::kTile + kw * C::TK + (lane & (C::TK - 1)), len - 1);
      return key >= 0 ? table[key >> a.c.page_shift] : 0;
    };
    auto load = [&](int tile, int pages, char* stage) {
      char* grp = stage + kw * 2 * C::kHalf;
      if (tile < tiles - 1) {
        load_tile<C>(grp, rw, lane, [&](int k, bool isv) {
          const int key = min(tile * C::kTile + kw * C::TK + k, len - 1);
          const int page = min(max(__shfl(pages, k), 0), a.c.n_pages - 1);
          const int64_t at = (((int64_t)page * Hkv + head) << a.c.page_shift) + (key & ((1 << a.c.page_shift) - 1));
          return static_cast<const char*>(isv ? a.c.v_pages : a.c.k_pages) + at * C::kRowBytes;
        });
      } else {
        load_tile<C>(grp, rw, lane, [&](int k, bool isv) {
          const int node = min(kw * C::TK + k, a.T - 1);
          const int64_t at = ((int64_t)seq * a.T + node) * Hkv + head;
          return reinterpret_cast<const char*>(isv ? a.v_new : a.k_new) + at * C::kRowBytes;
        });
      }
    };
    load(first, page_of(first), lds);
    int pages = page_of(min(first + 1, tiles - 1));
    for (int i = first; i < last; ++i) {
      char* stage = lds + ((i - first) & 1) * C::kStage;
      // the tile and the pages of the next one are here; everyone is done with the other stage
      big::wait_vmcnt<0>();
      big::bar();
      if (i + 1 < last) load(i + 1, pages, lds + ((i + 1 - first) & 1) * C::kStage);
      pages = page_of(min(i + 2, tiles - 1));
      char* kt = stage + kw * 2 * C::kHalf;
      char* vt = kt + C::kHalf;
      const int left = i < tiles - 1 ? len - i * C::kTile - kw * C::TK : a.T - kw * C::TK;  // keys that there are
      const bool tree = i == tiles - 1;
      bool masked = false;
      uint64_t see = ~0ull;
      if (tree || len - i * C::kTile < C::kTile) {
        // the tree's tile, or the cache's last one
        masked = true;
        uint64_t there = left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1 : 0;
        see = there;
        if (tree) {
          const bool any = left > 0;
          there = any ? used >> (kw * C::TK) : 0;
          see = any ? sees >> (kw * C::TK) : 0;
        }
        const bool odd = clear_rows<C>(vt, rw, lane, there, tree);
        if (__ballot(odd) && lane == 0) s_odd = 1;
        big::bar();
      }
      if (left > 0) step<C>((lds_t)kt, (lds_t)vt, at, qf, a.c2, lane, masked, see, st);
      if (tree && s_odd && left > 0) {
        // what is not finite in a node's V (cleared above) reaches the rows that see the node, and no others
#pragma unroll 1
        for (int k = 0; k < min(C::TK, left); ++k) {
          const uint16_t* v = a.v_new + (((int64_t)seq * a.T + kw * C::TK + k) * Hkv + head) * C::D;
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

    // join the key groups
    const bool whole = first == 0 && last == tiles;
    st.l += xor32(st.l, lane);
    if constexpr (C::KW > 1) {
      float* sh = reinterpret_cast<float*>(lds);
      constexpr int kSlot = (C::D / 2 + 2) * 64;  // a wave's values
      if (kw > 0) {
        float* mine = sh + (wave - C::RW) * kSlot + lane;
#pragma unroll
        for (int dt = 0; dt < C::D / 32; ++dt)
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[64 * (16 * dt + i)] = st.o[dt][i];
        mine[64 * (C::D / 2)] = st.m;
        mine[64 * (C::D / 2 + 1)] = st.l;
      }
      __syncthreads();
      if (kw == 0) {
#pragma unroll 1
        for (int k = 1; k < C::KW; ++k) {
          const float* other = sh + ((k - 1) * C::RW + rw) * kSlot + lane;
          const float om = other[64 * (C::D / 2)], ol = other[64 * (C::D / 2 + 1)];
          const float m = fmaxf(st.m, om);
          const float f0 = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.m - m);
          const float f1 = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(om - m);
          st.l = st.l * f0 + ol * f1;
#pragma unroll
          for (int dt = 0; dt < C::D / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) st.o[dt][i] = st.o[dt][i] * f0 + other[64 * (16 * dt + i)] * f1;
          st.m = m;
        }
      }
    }
    if (kw == 0 && row < rows) {
      if (whole) {
        const float inv = sees && st.l != 0.f ? 1.0f / st.l : 0.f;
        uint16_t* o = a.out + qoff;
#pragma unroll
        for (int dt = 0; dt < C::D / 32; ++dt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = inv != 0.f ? st.o[dt][4 * e + i] * inv : 0.f;
            const bf16x2 lo = __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2);
            const bf16x2 hi = __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2);
            union {
              bf16x2 b[2];
              uint2 u;
            } pk;
            pk.b[0] = lo;
            pk.b[1] = hi;
            *reinterpret_cast<uint2*>(o + 32 * dt + 8 * e + 4 * h) = pk.u;
          }
      } else {
        const int64_t slot = (slot0 + 2 * g + (first == 0 ? 1 : 0)) * C::kRows + 32 * rw + (lane & 31);
        float* o = a.part_o + slot * C::D;
#pragma unroll
        for (int dt = 0; dt < C::D / 32; ++dt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f32x4*>(o + 32 * dt + 8 * e + 4 * h) =
                f32x4{st.o[dt][4 * e], st.o[dt][4 * e + 1], st.o[dt][4 * e + 2], st.o[dt][4 * e + 3]};
        if (h == 0) *reinterpret_cast<f32x2*>(a.part_ml + 2 * slot) = f32x2{st.m, st.l};
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) s_odd = 0;
    x = before + last;
    before += tiles;
    ++seq;
  }
}

// Sequences cut over several workgroups: their pieces joined.  Workgroup (sequence, kv head).
template <class C>
__global__ __launch_bounds__(256) void tree_attention_join_kernel(AttnArgs a) {
  __shared__ int64_t scratch[256 + 2];
  __shared__ int s_used[kMaxNodes];
  const int Hkv = a.c.kv_heads;
  const int seq = blockIdx.x / Hkv, head = blockIdx.x % Hkv;
  // tiles before this sequence
  const int per = (a.batch + 255) / 256;
  int64_t mine = 0, upto = 0;
  for (int b = threadIdx.x * per; b < min((int)(threadIdx.x + 1) * per, a.batch); ++b) {
    const int n = seq_tiles(a.c.len(b), C::kTile);
    mine += n;
    if (b < seq) upto += n;
  }
  // two sums over the threads
  auto sum = [&](int64_t v) {
    scratch[threadIdx.x] = v;
    __syncthreads();
    for (int s = 128; s > 0; s >>= 1) {
      if ((int)threadIdx.x < s) scratch[threadIdx.x] += scratch[threadIdx.x + s];
      __syncthreads();
    }
    const int64_t r = scratch[0];
    __syncthreads();
    return r;
  };
  const int64_t total = sum(mine), before = sum(upto);
  const int tiles = seq_tiles(a.c.len(seq), C::kTile);
  const int64_t parts = min((int64_t)a.G, total);  // and the first and last of them with a tile of this sequence
  const int g0 = (int)(((before + 1) * parts - 1) / total), g1 = (int)(((before + tiles) * parts - 1) / total);
  if (g0 == g1) return;  // one piece: written already
  if (threadIdx.x < 64) s_used[threadIdx.x] = tree_bits(a.parents + (int64_t)seq * a.T, a.T, threadIdx.x) != 0;
  __syncthreads();
  const int rows = a.T * a.group;
  for (int u = threadIdx.x; u < rows * (C::D / 4); u += 256) {
    const int row = u / (C::D / 4), d = u % (C::D / 4) * 4;
    const int rt = row / C::kRows, rr = row % C::kRows;
    const int64_t slot0 = ((int64_t)head * a.row_tiles + rt) * 2 * a.G;
    auto slot = [&](int g) { return (slot0 + 2 * g + (g == g0 ? 1 : 0)) * C::kRows + rr; };
    float m = -INFINITY;
    for (int g = g0; g <= g1; ++g) m = fmaxf(m, a.part_ml[2 * slot(g)]);
    float l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    const float m0 = m == -INFINITY ? 0.f : m;
    for (int g = g0; g <= g1; ++g) {
      const f32x2 ml = *reinterpret_cast<const f32x2*>(a.part_ml + 2 * slot(g));
      const float f = __builtin_amdgcn_exp2f(ml.x - m0);
      l += ml.y * f;
      const f32x4 p = *reinterpret_cast<const f32x4*>(a.part_o + slot(g) * C::D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += p[i] * f;
    }
    const int t = row / a.group;
    const bool some = s_used[t] && l != 0.f;
    const float inv = some ? 1.0f / l : 0.f;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = some ? o[i] * inv : 0.f;
    const bf16x2 lo = __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2);
    const bf16x2 hi = __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2);
    union {
      bf16x2 b[2];
      uint2 u;
    } pk;
    pk.b[0] = lo;
    pk.b[1] = hi;
    *reinterpret_cast<uint2*>(a.out + (((int64_t)seq * a.T + t) * Hkv * a.group + head * a.group + row % a.group) * C::D +
                              d) = pk.u;
  }
}

template <class C>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  tree_attention_kernel<C><<<dim3((uint32_t)(a.G * a.row_tiles * a.c.kv_heads)), dim3(C::kThreads), 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.G == 1) return e;
  tree_attention_join_kernel<C><<<dim3((uint32_t)(a.batch * a.c.kv_heads)), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

// Few rows: waves take keys of their own; more rows: they share the keys.
template <int D>
hipError_t launch_d(int kind, const AttnArgs& a, hipStream_t stream) {
  switch (kind) {
    case 0: return launch<Cfg<D, 4, 1, 32>>(a, stream);
    case 1: return launch<Cfg<D, 2, 2, 32>>(a, stream);
    case 2: return launch<Cfg<D, 1, 3, 64>>(a, stream);
    default: return launch<Cfg<D, 1, 4, 64>>(a, stream);
  }
}

}  // namespace

AttnPlan plan_tree_attention(const CacheView& c, int64_t batch, int64_t T, int64_t group, int64_t D) {
  AttnPlan p{};
  const int64_t rows = T * group;
  p.kind = rows <= 32 ? 0 : rows <= 64 ? 1 : rows <= 96 ? 2 : 3;
  p.tile_rows = p.kind == 0 ? 32 : p.kind == 1 ? 64 : p.kind == 2 ? 96 : 128;
  p.row_tiles = cdiv(rows, p.tile_rows);
  const int64_t tile = p.kind == 0 ? 128 : 64;
  const int64_t most = batch * (cdiv((int64_t)c.table_width << c.page_shift, tile) + 1);  // tiles, all lengths full
  p.G = kAttnBlocks / (p.row_tiles * c.kv_heads);
  p.G = p.G < 1 ? 1 : p.G > most ? most : p.G;
  const int64_t slots = (int64_t)c.kv_heads * p.row_tiles * 2 * p.G * p.tile_rows;
  p.part_bytes = p.G > 1 ? align_up((size_t)(slots * D) * 4, 256) : 0;
  p.ws_bytes = p.G > 1 ? p.part_bytes + align_up((size_t)slots * 8, 256) : 0;
  return p;
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
  a.batch = (int)batch;
  a.T = (int)T;
  a.group = (int)group;
  a.G = (int)p.G;
  a.row_tiles = (int)p.row_tiles;
  a.c2 = (float)(scale * 1.4426950408889634);
  return D == 64 ? launch_d<64>(p.kind, a, stream) : launch_d<128>(p.kind, a, stream);
}

}  // namespace dfs
