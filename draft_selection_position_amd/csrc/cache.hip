// Accepted tokens into a paged cache.
//
// For sequence b and i < counts[b]: the K and V rows of node nodes[b, i] go to position
// lens[b] + i of the sequence, page block_table[b, position / page], row position % page.
// Pure data movement, bound by memory (or by the launch, for few tokens): one workgroup
// per accepted token moves its K and V rows of all heads, 16 bytes per lane; a row of one
// head is contiguous on both sides.  One sequence's tokens: 2.4 us on the device, the launch;
// 256 sequences', up to 33 each, 8 heads of 128: 6.4 us for 18 MB read and written, one round
// of workgroups that each wait for counts, lengths, page and rows in turn.
#include "dfs_device.h"
#include "dfs_internal.h"

namespace dfs {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void cache_commit_kernel(CacheView c, const uint4* k_new, const uint4* v_new,
                                                                const int32_t* nodes, const int32_t* counts, int T,
                                                                int P, int32_t* out_lens) {
  const int b = blockIdx.x / P, i = blockIdx.x % P;
  const int n = min(max(counts[b], 0), P);
  const int64_t len = max(c.lens[b], 0);
  if (i == 0 && threadIdx.x == 0 && out_lens) out_lens[b] = (int32_t)(len + n);
  if (i >= n) return;
  const int64_t at = len + i;
  if ((at >> c.page_shift) >= c.table_width) return;
  const int page = c.block_table[(int64_t)b * c.table_width + (at >> c.page_shift)];
  const int node = nodes ? nodes[(int64_t)b * P + i] : i;
  if (page < 0 || page >= c.n_pages || node < 0 || node >= T) return;
  const int64_t row = at & ((1 << c.page_shift) - 1);
  const int vecs = c.row_bytes / 16, all = c.kv_heads * vecs;  // 16-byte pieces of a head's row, of a token
  for (int t = threadIdx.x; t < 2 * all; t += kThreads) {
    const bool isv = t >= all;
    const int u = isv ? t - all : t;
    const int h = u / vecs, p = u % vecs;
    const int64_t src = ((int64_t)b * T + node) * all + u;
    const int64_t dst = ((((int64_t)page * c.kv_heads + h) << c.page_shift) + row) * vecs + p;
    uint4* pages = static_cast<uint4*>(isv ? c.v_pages : c.k_pages);
    pages[dst] = (isv ? v_new : k_new)[src];
  }
}

}  // namespace

hipError_t launch_cache_commit(const CacheView& c, const void* k_new, const void* v_new, const int32_t* nodes,
                               const int32_t* counts, int64_t batch, int64_t T, int64_t P, int32_t* out_lens,
                               hipStream_t stream) {
  cache_commit_kernel<<<dim3((uint32_t)(batch * P)), dim3(kThreads), 0, stream>>>(
      c, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), nodes, counts, (int)T, (int)P, out_lens);
  return hipGetLastError();
}

}  // namespace dfs
