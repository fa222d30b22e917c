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
//
// A batch with a shared prefix takes the same steps over two sets of keys: the prefix's, with the rows of the whole
// batch as those of one sequence (by the kernel here, or for many by one of its own: prefix.hip), and every
// sequence's own.  Both leave pieces, and the join takes a row's of either kind; only where there are few keys in all does
// every sequence take the prefix's as if they were its own, in one launch without pieces.  4 tokens, 8 kv heads x 4 of 128, 4001 + up to
// 77 keys: 14.3 us, two launches as above; 256 tokens, 16384 + up to 1024 keys: 187 to 207 us, of which 78 the prefix,
// 102 the own keys (5.2 TB/s) and 10 the join; each by itself (no prefix known) would read 17.2 GB.
#include <algorithm>
#include <type_traits>

#include "../../include/dfs.h"
#include "attn_tile.h"
#include "dfs_internal.h"

namespace dfs {
namespace {

constexpr float kUnused = -1.0f;  // for a sum of weights

// What a workgroup's keys are.  kTree: a sequence's cache and tree, the whole answer.  Of a batch with a shared prefix:
// kOwn the same, but a piece of the answer, to be joined with the prefix's; kPrefix the prefix, for the rows of the whole
// batch as the one sequence that it is (no node is a key then, and every row sees all); kBoth, of short ones, the prefix's and
// right behind them the sequence's, the whole answer.
enum Role { kTree, kOwn, kPrefix, kBoth };

struct AttnArgs {
  CacheView c;
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* parents;
  uint16_t* out;
  float* part_o;   // [Hkv, row tiles, 2 G, rows of a tile, D]; kOwn: cut_slots (2 G, or none of parts that are
                   // sequences) and one for each sequence that is in one piece, of slot_rows
  float* part_ml;  // [Hkv, row tiles, 2 G, rows of a tile, 2]: maximum and sum; of an unused node's row the last piece has kUnused
  int2* pieces;    // [batch]: the first and the last part with a tile of the sequence (NULL: nothing to join)
  int batch, T, group, G, row_tiles;
  bool whole;  // parts are sequences
  int spread;  // 16-lane groups that join a row's pieces: 1, 4 or 16
  float c2;  // scale * log2(e)
  // Of a batch with a shared prefix.
  int cut_slots;
  int slot_rows;  // kOwn: of a slot, as many as there are where one tile has them all
  // the prefix's pieces: [Hkv, slots, rows of a tile, D] as the prefix's own kernel leaves them, or by tree
  // attention's [Hkv, parts, rows of the batch, D] with their count, and their maxima and sums
  float* prefix_o;
  float* prefix_ml;
  bool large;
  PrefixCut cut;
  const int32_t* prefix_table;
  const int32_t* prefix_len;
  int prefix_most;  // the longest that its table has
  int* prefix_count;
  int prefix_G;
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

__device__ __forceinline__ uint64_t shfl64(uint64_t x, int src) {
  return ((uint64_t)(uint32_t)__shfl((uint32_t)(x >> 32), src) << 32) | (uint32_t)__shfl((uint32_t)x, src);
}

// The prefix's length, where its keys are in front of a sequence's own.
template <Role kRole>
__device__ __forceinline__ int in_front(const AttnArgs& a) {
  return kRole == kBoth ? min(max(*a.prefix_len, 0), a.prefix_most) : 0;
}
// Tiles of a sequence: its keys are the cache's and right behind them the tree's.
template <class C, Role kRole>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int len) {
  return (len + (kRole == kPrefix ? 0 : a.T) + C::kTile - 1) / C::kTile;
}
template <class C, Role kRole>
__device__ __forceinline__ int seq_tiles(const AttnArgs& a, int b) {
  return tiles_of<C, kRole>(a, in_front<kRole>(a) + a.c.len(b));
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
template <class C, Role kRole, class F>
__device__ __forceinline__ Where locate_wave(const AttnArgs& a, int lane, F want) {
  const int mine = lane < a.batch ? seq_tiles<C, kRole>(a, lane) : 0;
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
template <class C, Role kRole, class F>
__device__ __forceinline__ Where locate(const AttnArgs& a, int* scratch, F want) {
  if (a.batch == 1) return Where{seq_tiles<C, kRole>(a, 0), 0, 0};
  if (a.batch <= 64) return locate_wave<C, kRole>(a, threadIdx.x & 63, want);
  constexpr int kThreads = C::kThreads;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int lo = threadIdx.x * per, hi = min(lo + per, a.batch);
  int mine = 0;
#pragma unroll 1
  for (int b = lo; b < hi; ++b) mine += seq_tiles<C, kRole>(a, b);
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
    for (int n; x >= at + (n = seq_tiles<C, kRole>(a, b)); ++b) at += n;
    scratch[kThreads] = at;
    scratch[kThreads + 1] = b;
  }
  __syncthreads();
  return Where{total, scratch[kThreads], scratch[kThreads + 1]};
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

// Of a row of a batch with a shared prefix, numbered through the batch: the prefix's pieces, how many there are, the first
// one's slot, and the slots from one to the next.
struct PrefixPieces {
  int n;
  int64_t first, apart;
};
__device__ __forceinline__ PrefixPieces prefix_pieces(const AttnArgs& a, int head, int row) {
  if (!a.large) {
    const int64_t rows = (int64_t)a.batch * a.T * a.group;
    return PrefixPieces{*a.prefix_count, head * a.prefix_G * rows + row, rows};
  }
  PrefixCut cut = a.cut;
  cut.cut((min(max(*a.prefix_len, 0), a.prefix_most) + kPrefixKeys - 1) / kPrefixKeys);
  const int rt = row / kPrefixRows;
  return PrefixPieces{cut.count(rt), (head * cut.slots() + cut.slot(rt)) * kPrefixRows + row % kPrefixRows, kPrefixRows};
}

template <class C>
struct Shared {
  char lds[C::kLds];
  int scratch[C::kThreads + 2];
  int s_odd[C::KW];
};

template <class C, Role kRole>
__device__ __forceinline__ void attend(const AttnArgs& a, int block, Shared<C>& shared) {
  char* const lds = shared.lds;
  int* const scratch = shared.scratch;
  int* const s_odd = shared.s_odd;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int kw = wave / C::RW, rw = wave % C::RW;
  const int Hkv = a.c.kv_heads;
  // Workgroups go round the eight XCDs in turn: the row tiles of a part are eight apart, so
  // that they run side by side on one XCD and read the part's keys into its L2 once.
  const int turn = block / (8 * a.row_tiles), rt = block / 8 % a.row_tiles;
  const int unit = turn * 8 + block % 8;  // (head, part)
  if (unit >= Hkv * a.G) return;
  const int head = unit / a.G, g = unit % a.G;
  // part g: the tiles x .. x_end - 1, at least one
  int x = 0, x_end, seq = g, before = 0, total = 0, parts = 0;
  if (a.whole) {
    x_end = seq_tiles<C, kRole>(a, g);
  } else {
    const Where w = locate<C, kRole>(a, scratch, [&](int total) {
      return min(mul_div(g, total, parts_of(a, total)), total - 1);
    });
    total = uniform(w.total), parts = parts_of(a, total);
    if (kRole == kPrefix && unit == 0 && rt == 0 && threadIdx.x == 0) *a.prefix_count = parts;
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
  const int64_t slot0 = ((int64_t)head * a.row_tiles + rt) * (kRole == kOwn ? a.cut_slots + a.batch : 2 * a.G);
  const Frag<C> at(lane);
  const uint32_t ring0 = lds_addr(lds) + kw * C::S * C::kStage;
  const uint32_t pages0 = lds_addr(lds) + C::kRing + wave * (C::kAhead + 1) * C::kPages;
  const char* ring = lds + kw * C::S * C::kStage;
  const char* my_pages = lds + C::kRing + wave * (C::kAhead + 1) * C::kPages;
  const int64_t page_bytes = ((int64_t)Hkv << a.c.page_shift) * C::kRowBytes;

  while (x < x_end) {
    const int front = in_front<kRole>(a), own = a.c.len(seq), len = front + own;
    const int tiles = tiles_of<C, kRole>(a, len);
    const int first = x - before, last = min(tiles, x_end - before);
    // for the join: tile y is in part floor(((y + 1) parts - 1) / total)
    if (a.pieces && first == 0 && head == 0 && rt == 0 && threadIdx.x == 0)
      a.pieces[seq] = make_int2(
          g, kRole == kOwn && a.whole ? g : (int)(((double)(before + tiles) * (double)parts - 1.0) / (double)total));
    const int n = last - first;  // steps
    // nothing cached: no entry of the table counts, and look-ups read the length (unused) in its place
    const int32_t* table = own > 0 ? a.c.block_table + (int64_t)seq * a.c.table_width : a.c.lens + seq;
    // Pages of a step's keys or more: they lie in one, read by a scalar load a step ahead.
    const bool wide = kRole != kBoth && (1 << a.c.page_shift) >= C::kKeys;
    auto wide_page = [&](int i) {
      typedef const __attribute__((address_space(4))) int32_t* const_ptr;
      const int key = min((first + i) * C::kTile + kw * C::kKeys, len - 1);
      return *(const_ptr)(table + (max(key, 0) >> a.c.page_shift));
    };
    // Smaller ones: the pages of step i's keys, into its slot of this wave's ring.
    auto look_up = [&](int i) {
      const int key = min((first + i) * C::kTile + kw * C::kKeys + (lane & (C::kKeys - 1)), len - 1);
      dma4(kRole == kBoth ? page_entry(a.prefix_table, table, front, key, a.c.page_shift) : table + (max(key, 0) >> a.c.page_shift),
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
      auto place = [&](int key) { return key < front ? key : key - front; };
      if (base + C::kKeys > len) {  // nodes among them, or nothing
#pragma unroll
        for (int u = 0; u < C::kLoads; ++u) {
          int j = rw + C::RW * u;
          if (C::kLoadsAll % C::RW != 0) j = min(j, C::kLoadsAll - 1);  // the last rows again
          const int row = j * C::kRowsPerLoad + rr, key = kRole == kPrefix ? min(base + row, len - 1) : base + row;
          const int page = min(max(wide ? wide_id : pages[row], 0), a.c.n_pages - 1);
          const int64_t cached = (int64_t)page * page_bytes +
                                 (int64_t)((head << a.c.page_shift) + (place(key) & in_page)) * C::kRowBytes;
          const int64_t node = (((int64_t)seq * a.T + min(key - len, a.T - 1)) * Hkv + head) * C::kRowBytes;
          const bool tree = kRole != kPrefix && key >= len;
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
                            (int64_t)((head << a.c.page_shift) + (place(base + row) & in_page)) * C::kRowBytes;
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
    if (kRole != kPrefix && (last == tiles || last * C::kTile > len)) {
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
      const int cached = len - base, left = cached + (kRole == kPrefix ? 0 : a.T);  // of the cache's, of all, from there on
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
      if (kRole != kPrefix && masked && left > 0 && s_odd[kw]) {
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
    const bool whole = (kRole == kTree || kRole == kBoth) && first == 0 && last == tiles;
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
        const int64_t slot =
            kRole == kPrefix ? ((int64_t)head * a.prefix_G + g) * rows + row
            : kRole == kOwn  ? (slot0 + (first == 0 && last == tiles ? a.cut_slots + seq : 2 * g + (first == 0 ? 1 : 0))) * a.slot_rows +
                                  32 * rw + (lane & 31)
                             : (slot0 + 2 * g + (first == 0 ? 1 : 0)) * C::kRows + 32 * rw + (lane & 31);
        float* part_o = kRole == kPrefix ? a.prefix_o : a.part_o;
        float* part_ml = kRole == kPrefix ? a.prefix_ml : a.part_ml;
#pragma unroll
        for (int u = 0; u < kMine; ++u) *reinterpret_cast<f32x4*>(part_o + slot * C::D + d0 + 8 * u) = o[u];
        if (h == 0 && kw == 0)
          *reinterpret_cast<f32x2*>(part_ml + 2 * slot) = f32x2{m, kRole != kPrefix && last == tiles && !sees ? kUnused : l};
      }
    }
    __syncthreads();
    x = before + last;
    before += tiles;
    ++seq;
  }
}

template <class C, Role kRole>
__global__ __launch_bounds__(C::kThreads, C::kMinWaves) void tree_attention_kernel(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) Shared<C> shared;
  attend<C, kRole>(a, blockIdx.x, shared);
}

// The prefix for few rows, by the first n workgroups, and the sequences' own keys beside it.
template <class C>
__global__ __launch_bounds__(C::kThreads, C::kMinWaves) void beside_prefix_kernel(AttnArgs prefix, AttnArgs own, int n) {
  __shared__ __attribute__((aligned(1024))) Shared<C> shared;
  if ((int)blockIdx.x < n)
    attend<C, kPrefix>(prefix, blockIdx.x, shared);
  else
    attend<C, kOwn>(own, blockIdx.x - n, shared);
}

// Sequences cut over several workgroups: their pieces joined.  16 lanes hold a row's D
// values and take every `spread`-th of its pieces, two at a time, statistics and values in
// one go: ceil(pieces / (2 spread)) rounds of memory latency for a row.  16 rows a workgroup for few
// pieces (spread 1), 4 for more (a wave a row), or one; by the parts for each sequence on average, so
// a long sequence among many short ones takes more rounds than it would have to.
// kShared: a shared prefix's pieces come first.
template <class C, bool kShared>
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
  if (!kShared && g0 == g1) return;  // one piece: written already
  const int sub = 4 * wave + (lane >> 4);  // of the workgroup's 16 groups of lanes
  const int row = row0 + sub / spread;
  const int qrow = min(row, rows - 1), t = qrow / a.group;
  const PrefixPieces of = kShared ? prefix_pieces(a, head, seq * rows + qrow) : PrefixPieces{};
  const int before = of.n;
  const int last = before + g1 - g0;
  const int64_t slot0 = ((int64_t)head * a.row_tiles + qrow / C::kRows) * (kShared ? a.cut_slots + a.batch : 2 * a.G);
  const bool whole = kShared && g0 == g1;  // a sequence in one piece
  const int slot_rows = kShared ? a.slot_rows : C::kRows;
  const float end = a.part_ml[2 * ((slot0 + (whole ? a.cut_slots + seq : 2 * g1)) * slot_rows + qrow % C::kRows) + 1];
  float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) o[e] = 0.f;
  for (int g = sub % spread; g <= last; g += kAtOnce * spread) {
    f32x2 ml[kAtOnce];
    f32x4 v[kAtOnce][kPer / 4];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int gk = min(g + k * spread, last) - before;
      const bool shared = kShared && gk < 0;
      const int64_t slot = shared ? of.first + (gk + before) * of.apart
                                  : (slot0 + (whole ? a.cut_slots + seq : 2 * (g0 + gk) + (gk == 0 ? 1 : 0))) * slot_rows +
                                        qrow % C::kRows;
      const float* part_o = shared ? a.prefix_o : a.part_o;
      const float* part_ml = shared ? a.prefix_ml : a.part_ml;
      ml[k] = *reinterpret_cast<const f32x2*>(part_ml + 2 * slot);
#pragma unroll
      for (int e = 0; e < kPer / 4; ++e)
        v[k][e] = *reinterpret_cast<const f32x4*>(part_o + slot * C::D + (lane & 15) * kPer + 4 * e);
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
      if (g + k * spread <= last) {
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
uint32_t blocks_of(const AttnArgs& a) {
  return (uint32_t)(cdiv((int64_t)a.G * a.c.kv_heads, 8) * 8 * a.row_tiles);
}

template <class C, bool kShared>
hipError_t launch_join(const AttnArgs& a, hipStream_t stream) {
  tree_attention_join_kernel<C, kShared><<<
      dim3((uint32_t)(a.batch * a.c.kv_heads * cdiv(a.T * a.group, 16 / a.spread))), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

template <class C, Role kRole>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  tree_attention_kernel<C, kRole><<<dim3(blocks_of<C>(a)), dim3(C::kThreads), 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.pieces || kRole == kPrefix) return e;
  return launch_join<C, kRole == kOwn>(a, stream);
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

// How a batch goes over its shared prefix.  Few rows or few products: tree attention's kernel, in one launch with the
// sequences' own keys, so that the call is two launches.  From 3 x 2^32 products of a kind on (rows x heads x the
// prefix's longest x D), and more than 384 rows: the prefix's own kernel, which is half as fast again but fills
// slowly and takes tiles of 256 rows (us, own kernel against the other: heads of 128, 512 rows x 8 heads x 32768 keys 99 and 106, 4352 x 8 x
// 8000 167 and 230, 4536 x 4 x 8000 105 and 124; below, 2176 x 4 x 8000 70 and 65, 4352 x 8 x 2000 80 and 77, 768 x 8 x 16384 94 and 98, 1020 x
// 4 x 16384 83 and 66, 544 x 8 x 1000 44 and 28, 384 x 8 x 65536 179 and 171.  Heads of 64, 4352 x 8 x 8000 112 and 158, 4352 x 4 x 16000 114
// and 141, 17227 x 4 x 4000 136 and 201; below, 4352 x 8 x 2000 61 and 55, 4352 x 4 x 8000 81 and 78, 4536 x 4 x 8000 81 and 65).
// Products are not all that decides, for row tiles fill the card's workgroups well or badly: below the bound the own kernel gains at 4352 x 4 of 128
// x 4000 (78 and 126) and x 2000 (60 and 74), 6426 x 4 of 128 x 2000 (76 and 79), 17227 x 4 of 128 x 900 (103 and 113), of 64 x 2000 (103 and 115),
// 4352 x 8 of 64 x 4000 (84 and 89), and above it loses at 6426 x 4 of 64 x 8000 (107 and 89), 4536 x 4 of 64 x 16000 (118 and 112).
bool prefix_is_large(int64_t rows, int64_t kv_heads, int64_t D, int64_t longest) {
  return rows > 384 && (double)rows * (double)kv_heads * (double)D * (double)longest >= 3.0 * 4294967296.0;
}
// In one launch the own keys go by the rows of the whole batch, in tiles that one sequence's rows do not fill: up to so many
// keys of a sequence, and of all sequences and heads, the saved launch pays (us, lengths in mixed order; 4 heads to a kv head of 128: 16
// tokens x 8 kv heads, up to 4000 own keys 46 and 49, 8000 67 and 65, 16000 121 and 107; 64 x 8, 1500 60 and 71, 3000 104 and 100,
// 8000 224 and 193; 128 x 8, 8000 418 and 362; 20 x 17 nodes x 8, 3000 57 and 70; of 64: 100 x 5 x 4, 3000 66 and 70, 256 x 1
// x 4 of 8, 5000 167 and 147, 30 x 9 x 4, 5000 38 and 52).
bool beside_prefix(int64_t pairs, int64_t longest) { return longest <= 8192 && pairs * longest <= 5 << 18; }
// Up to 32 rows of a sequence and head, 1024 of these or more and no long one: a wave for each, four or more of them on a
// CU, where a workgroup that goes through several in turn waits for each one's start.  Behind long ones the last wave ends
// late.  (us a call, lengths in mixed order, against a launch of their own or the prefix's; 4 heads to a kv head: 256 tokens x 8 kv
// heads of 128, up to 100 own keys 108 and 139, 1024 191 and 204; 128 x 8, 1000 94 and 99, 2000 145 and 143, 4000 237 and 206;
// 200 x 8 nodes x 8, 1500 239 and 245; of 64: 512 x 8, 1000 161 and 192, 2000 243 and 234, 4000 440 and 384; 200 x 5 nodes x 6,
// 1500 93 and 107.)
bool own_by_waves(int64_t rows, int64_t pairs, int64_t longest) { return rows <= 32 && pairs >= 1024 && longest <= 1536; }

// Few keys in all, by the tables' widths: a workgroup takes the prefix's and a sequence's own, in one launch and without
// pieces, although every sequence reads the prefix again (us, against the other ways; heads of 128, 4 to each of 8 kv heads: 64 x 17
// nodes, prefix 100, up to 50 own keys 20 and 35, 550 and 50 35 and 44, 900 and 50 49 and 50; 32 tokens, 300 and 100 14 and 18, 4
// tokens 13.0 and 12.5 but a launch less for the host, 8 tokens, 900 and 50 20 and 13; 183 x 26 nodes, 7 x 2, 2 and 65 40 and 62; 107 x 23, 4
// x 7 of 64, 600 43 and 56).  Up to 32 rows a CU holds one workgroup, so that a 257th begins when another ends: 32 tokens x 8 heads of 128, 300
// and 100 13.7 and 18.1, 33 22.4 and 18.3, 48 24.3 and 19.2, 64 25.6 and 24.8, 96 (not taken) 37 and 27; with 6 nodes 36 26.4 and 23.8, 48 27.3
// and 28.1, 64 28.6 and 29.4; of 64, 33 15.6 and 14.3, 64 16.7 and 17.4, with 6 nodes 33 16.6 and 21.6, 64 18.5 and 24.4: between 256
// and 512 pairs few rows lose and more rows gain.  Beyond 32 rows any number of pairs gains: 8 x 17 nodes x 8 heads, 128 and 40 13.5 and 16.2, 256 x
// 17 x 8 64 and 98, 1024 x 17 x 4 123 and 247, 550 and 60 251 and 348; at worst 600 x 40 nodes x 4 heads, 550 and 60 148 and 144.
bool few_keys(int64_t rows, int64_t pairs, int64_t longest) {
  if (rows <= 32) return longest <= 512 && pairs <= 512;
  return longest <= 256 || (longest <= 768 && pairs * cdiv(rows, 128) >= 48);
}

template <int D, class F>
auto with_own_cfg(int64_t rows, bool single, F f) {
  if (single) return f(Cfg<D, 1, 1, 2, 1>{});
  return with_cfg<D>(rows, f);
}

template <class F>
AttnPlan plan_attention(const CacheView& c, int64_t batch, int64_t T, int64_t group, int64_t D, bool whole, F with) {
  const int64_t rows = T * group;
  return with([&](auto cfg) {
    typedef decltype(cfg) C;
    AttnPlan p{};
    p.row_tiles = cdiv(rows, C::kRows);
    // tiles when all lengths are full: no more parts than that
    const int64_t each = cdiv(((int64_t)c.table_width << c.page_shift) + T, (int64_t)C::kTile), most = batch * each;
    p.slots = 256 * C::kGroups;
    p.G = p.slots / (p.row_tiles * c.kv_heads);
    p.G = p.G < 1 ? 1 : p.G > most ? most : p.G;
    // Few tiles a sequence at most, by the table's width (the lengths are on the device: a table for more
    // keys cuts sequences however short they are): a part for each and no join (4 x 9 nodes, page 256: 8.0 us
    // against 10.2; 39 x 33 nodes, up to 61 keys: 17.8 against 24.4; 13 x 56 nodes, 7 heads, 243 keys: 16.2
    // against 27.9; at worst 2 x 18 nodes, 3 heads, 115 keys: 14.0 against 12.8).
    p.whole = whole || each <= 4 || (each <= 8 && batch * c.kv_heads * p.row_tiles >= 48);
    if (p.whole) p.G = batch;
    p.tile_rows = C::kRows;
    const int64_t rows = (int64_t)c.kv_heads * p.row_tiles * 2 * p.G * C::kRows;
    const bool join = p.G > 1 && !p.whole;
    p.part_bytes = join ? align_up((size_t)(rows * D) * 4, 256) : 0;
    p.ml_bytes = join ? align_up((size_t)rows * 8, 256) : 0;
    p.ws_bytes = join ? p.part_bytes + p.ml_bytes + align_up((size_t)batch * 8, 256) : 0;
    return p;
  });
}

}  // namespace

AttnPlan plan_tree_attention(const CacheView& c, int64_t batch, int64_t T, int64_t group, int64_t D) {
  return plan_attention(c, batch, T, group, D, false, [&](auto plan) {
    return D == 64 ? with_cfg<64>(T * group, plan) : with_cfg<128>(T * group, plan);
  });
}

namespace {

AttnArgs attention_args(const AttnPlan& p, const CacheView& c, const void* q, const void* k_new, const void* v_new,
                        const int32_t* parents, int64_t batch, int64_t T, int64_t group, double scale, void* out) {
  AttnArgs a{};
  a.c = c;
  a.q = static_cast<const uint16_t*>(q);
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.parents = parents;
  a.out = static_cast<uint16_t*>(out);
  a.whole = p.whole;
  a.batch = (int)batch;
  a.T = (int)T;
  a.group = (int)group;
  a.G = (int)p.G;
  a.row_tiles = (int)p.row_tiles;
  a.c2 = attention_c2(scale);
  return a;
}

}  // namespace

hipError_t launch_tree_attention(const AttnPlan& p, const CacheView& c, const void* q, const void* k_new,
                                 const void* v_new, const int32_t* parents, int64_t batch, int64_t T, int64_t group,
                                 int64_t D, double scale, void* out, void* ws, hipStream_t stream) {
  AttnArgs a = attention_args(p, c, q, k_new, v_new, parents, batch, T, group, scale, out);
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part_bytes);
  a.pieces = p.ws_bytes == 0 ? nullptr : reinterpret_cast<int2*>(static_cast<char*>(ws) + p.part_bytes + p.ml_bytes);
  a.spread = p.G >= 32 * batch ? 16 : p.G >= 8 * batch ? 4 : 1;  // by its pieces
  auto run = [&](auto cfg) { return launch<decltype(cfg), kTree>(a, stream); };
  return D == 64 ? with_cfg<64>(T * group, run) : with_cfg<128>(T * group, run);
}

SharedPlan plan_shared_attention(const CacheView& c, const CacheView& prefix, int64_t batch, int64_t T, int64_t group,
                                 int64_t D) {
  SharedPlan p{};
  const int64_t all_rows = batch * T * group;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  int64_t rows;
  const int64_t longest = (int64_t)c.table_width << c.page_shift, prefix_longest = (int64_t)prefix.table_width << prefix.page_shift;
  p.both = few_keys(T * group, batch * c.kv_heads, prefix_longest + longest + T);
  if (p.both) {
    p.own = plan_attention(c, batch, T, group, D, true, [&](auto plan) {
      return D == 64 ? with_cfg<64>(T * group, plan) : with_cfg<128>(T * group, plan);
    });
    p.ws_bytes = 256;
    return p;
  }
  p.large = prefix_is_large(all_rows, c.kv_heads, D, prefix_longest);
  p.single = own_by_waves(T * group, batch * c.kv_heads, longest);
  p.beside = !p.large && !p.single && beside_prefix(batch * c.kv_heads, longest);
  p.cfg_rows = p.beside ? all_rows : T * group;
  p.own = plan_attention(c, batch, T, group, D, p.single, [&](auto plan) {
    return D == 64 ? with_own_cfg<64>(p.cfg_rows, p.single, plan) : with_own_cfg<128>(p.cfg_rows, p.single, plan);
  });
  if (p.large) {
    p.cut = PrefixCut::plan(cdiv(all_rows, kPrefixRows), std::max<int64_t>(1, 256 / c.kv_heads), prefix_pair(D));
    rows = c.kv_heads * p.cut.slots() * kPrefixRows;
    p.prefix_parts = p.cut.pair * (p.cut.whole ? 1 : p.cut.parts);
  } else {
    const AttnPlan all = plan_tree_attention(prefix, 1, batch * T, group, D);
    p.prefix_tiles = all.row_tiles;
    const int64_t most = cdiv(prefix_longest, 32);  // tiles have 32 keys or more
    // both in one launch, where they fit
    const int64_t slots = !p.beside ? all.slots : std::max<int64_t>(all.slots / 2, all.slots - p.own.G * p.own.row_tiles * c.kv_heads);
    p.prefix_parts = std::min(most, std::max<int64_t>(1, slots / (all.row_tiles * c.kv_heads)));
    rows = c.kv_heads * p.prefix_parts * all_rows;
    p.count = take(4);
  }
  p.cut_slots = p.own.whole ? 0 : 2 * p.own.G;
  p.slot_rows = p.own.row_tiles == 1 ? T * group : p.own.tile_rows;
  const int64_t own_rows = c.kv_heads * p.own.row_tiles * (p.cut_slots + batch) * p.slot_rows;
  p.own_o = take((size_t)(own_rows * D) * 4);
  p.own_ml = take((size_t)own_rows * 8);
  p.pieces = take((size_t)batch * 8);
  p.prefix_o = take((size_t)(rows * D) * 4);
  p.prefix_ml = take((size_t)rows * 8);
  p.ws_bytes = off;
  return p;
}

hipError_t launch_shared_attention(const SharedPlan& p, const CacheView& c, const CacheView& prefix, const void* q,
                                   const void* k_new, const void* v_new, const int32_t* parents, int64_t batch,
                                   int64_t T, int64_t group, int64_t D, double scale, void* out, void* ws,
                                   hipStream_t stream) {
  AttnArgs a = attention_args(p.own, c, q, k_new, v_new, parents, batch, T, group, scale, out);
  char* w = static_cast<char*>(ws);
  a.part_o = reinterpret_cast<float*>(w + p.own_o);
  a.part_ml = reinterpret_cast<float*>(w + p.own_ml);
  a.pieces = reinterpret_cast<int2*>(w + p.pieces);
  a.prefix_o = reinterpret_cast<float*>(w + p.prefix_o);
  a.prefix_ml = reinterpret_cast<float*>(w + p.prefix_ml);
  a.large = p.large;
  a.cut = p.cut;
  a.prefix_len = prefix.lens;
  a.prefix_most = prefix.table_width << prefix.page_shift;
  a.prefix_G = (int)p.prefix_parts;
  a.cut_slots = (int)p.cut_slots;
  a.slot_rows = (int)p.slot_rows;
  if (p.both) {
    a.prefix_table = prefix.block_table;
    a.pieces = nullptr;
    auto run = [&](auto cfg) { return launch<decltype(cfg), kBoth>(a, stream); };
    return D == 64 ? with_cfg<64>(T * group, run) : with_cfg<128>(T * group, run);
  }
  const int64_t pieces = p.prefix_parts + cdiv(p.own.G, batch);
  // by a row's pieces, but no more workgroups than help (16 rows x 8 heads, 28 pieces: 14.2 us a call by 16 against 16.5 by 4;
  // 128 x 8 x 4 rows, 17 pieces: 96 by 4 against 107)
  a.spread = pieces < 8 ? 1 : batch * T * group * c.kv_heads <= 2048 ? 16 : 4;
  if (p.large) {
    const hipError_t e = launch_prefix_attention(prefix, p.cut, q, batch * T * group, group, D, a.c2, a.prefix_o, a.prefix_ml, stream);
    if (e != hipSuccess) return e;
    auto own = [&](auto cfg) { return launch<decltype(cfg), kOwn>(a, stream); };
    return D == 64 ? with_own_cfg<64>(T * group, p.single, own) : with_own_cfg<128>(T * group, p.single, own);
  }
  a.prefix_count = reinterpret_cast<int*>(w + p.count);
  AttnArgs b = a;
  b.c = prefix;
  b.batch = 1;
  b.T = (int)(batch * T);
  b.G = b.prefix_G;
  b.row_tiles = (int)p.prefix_tiles;
  b.whole = false;
  b.pieces = nullptr;
  auto run = [&](auto cfg) {
    typedef decltype(cfg) C;
    if (!p.beside) {
      const hipError_t e = launch<C, kPrefix>(b, stream);
      if (e != hipSuccess) return e;
      auto own = [&](auto cfg) { return launch<decltype(cfg), kOwn>(a, stream); };
      return with_own_cfg<C::D>(T * group, p.single, own);
    }
    const uint32_t n = blocks_of<C>(b);
    beside_prefix_kernel<C><<<dim3(n + blocks_of<C>(a)), dim3(C::kThreads), 0, stream>>>(b, a, (int)n);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_join<C, true>(a, stream);
  };
  return D == 64 ? with_cfg<64>(batch * T * group, run) : with_cfg<128>(batch * T * group, run);
}

}  // namespace dfs
