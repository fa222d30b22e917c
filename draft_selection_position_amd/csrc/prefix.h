// How the work on a shared prefix is cut (attention over it: prefix.hip; the join of its pieces: attention.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dfs {

// The entry of a table that holds the page of key `key`, where the prefix's `front` keys lie in front of a sequence's own:
// the prefix's or the sequence's.  Key -1: there are none at all, and what stands in for the sequence's table is read.
__host__ __device__ __forceinline__ const int32_t* page_entry(const int32_t* prefix_table, const int32_t* table,
                                                              int front, int key, int page_shift) {
  const bool of_front = key >= 0 && key < front;
  const int at = of_front ? key : key - front;
  return (of_front ? prefix_table : table) + ((at > 0 ? at : 0) >> page_shift);
}

// Row tiles x key tiles of a kv head over its C workgroups, as evenly as it goes with few pieces.  First whole row
// tiles, a workgroup each and C at a time; the n < C that are left, with f = C / n workgroups each and e = C % n over:
// workgroup (tile, c) takes `each` key tiles from c * each on, and the e others share what lies behind f * each of
// every tile, row tile by row tile.  A range costs as much as kStart key tiles more than it has:
// each + kStart = what the others get, n / e ranges of (tiles - f each) + kStart.  Workgroups of a head then go along
// the same keys side by side, in one or two places, and read them out of the L2.
// Where a CU holds two workgroups (`pair` 2), two share a range.  The one that started first is served first, and gets on
// that much faster: it takes kFirst / 64 of the range's key tiles.
struct PrefixCut {
  static constexpr int kFirst = 40, kStart = 4, kLeast = 2;  // key tiles; a range or a part has no fewer than kLeast
  int pair, C, whole, n, f, e, parts;  // on the host: from row tiles and C; parts: ranges of one of the n at most
  int tiles, each, rest;         // on the device: from the prefix's length; `rest` of a row tile is shared,
  int64_t share;                 // so much of it by one of the e

  __host__ static PrefixCut plan(int64_t row_tiles, int64_t C, int pair) {
    PrefixCut p{};
    p.pair = pair;
    p.C = (int)C;
    p.whole = (int)(row_tiles / C);
    p.n = (int)(row_tiles % C);
    if (p.n) p.f = p.C / p.n, p.e = p.C % p.n, p.parts = p.f + (p.e ? 2 : 0);
    return p;
  }
  // Slots of partial results for a head's row tiles: one for each workgroup of a range.
  __host__ __device__ int64_t slots() const { return pair * ((int64_t)whole * C + (int64_t)n * parts); }

  __device__ __forceinline__ void cut(int t) {
    tiles = t;
    if (n == 0) return;
    each = max((t + f - 1) / f, min(kLeast, t));
    rest = 0;
    if (e) {
      const int s = (int)(((int64_t)n * (t + kStart) + C - 1) / C);
      if (s >= kLeast && t - (int64_t)f * s >= kLeast) {
        each = s;
        rest = t - f * s;
        share = ((int64_t)n * rest + e - 1) / e;  // more than `rest`: a row tile's meets two of the e at most
      }
    }
  }
  // Pieces of row tile rt, and the first one's slot.
  __device__ __forceinline__ int count(int rt) const {
    if (tiles == 0) return 0;
    const int r = rt - whole * C;
    if (r < 0) return pair;
    if (rest == 0) return pair * ((tiles + each - 1) / each);
    return pair * (f + (int)(((int64_t)(r + 1) * rest - 1) / share - (int64_t)r * rest / share) + 1);
  }
  __device__ __forceinline__ int64_t slot(int rt) const {
    const int r = rt - whole * C;
    return pair * (r < 0 ? rt : (int64_t)whole * C + (int64_t)r * parts);
  }
};

}  // namespace dfs
