// For every key that a workgroup looks up of a sequence with a prefix in front (the tiles' keys, those past the last
// key as the last): which table is read, and where.  Lines: front own page_shift, then for each key "P i", "T i" or
// "L" (what stands in for the table of a sequence with nothing cached).
#include <cstdio>

#include "../../draft_selection_position_amd/csrc/prefix.h"

int main() {
  static int32_t prefix[4096], own_table[4096], lens[1];
  int front, own, shift;
  while (std::scanf("%d %d %d", &front, &own, &shift) == 3) {
    const int len = front + own;
    const int32_t* table = own > 0 ? own_table : lens;
    for (int k = 0; k < len + 64; ++k) {
      const int32_t* at = dfs::page_entry(prefix, table, front, k < len - 1 ? k : len - 1, shift);
      if (at >= prefix && at < prefix + 4096)
        std::printf("P%d ", (int)(at - prefix));
      else if (at >= own_table && at < own_table + 4096)
        std::printf("T%d ", (int)(at - own_table));
      else
        std::printf(at == lens ? "L " : "? ");
    }
    std::printf("\n");
  }
  return 0;
}
