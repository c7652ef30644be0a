// Attention of a tree of drafted tokens over the paged cache
// (pa_decode_tree): one warp per (sequence, node, head).
#include "attn_rows.cuh"
#include "serve_ops.h"

namespace pa {

namespace {

template <typename T, typename KvT, int D>
__global__ void __launch_bounds__(128) tree_rows_kernel(const TreeParams p) {
  __shared__ float sq[4][D];
  const int warp = threadIdx.x >> 5;
  const long long rows = (long long)p.num_seqs * p.q_len * p.n_q;
  for (long long i = blockIdx.x * 4ll + warp; i < rows; i += gridDim.x * 4ll) {
    const int h = (int)(i % p.n_q);
    const long long sn = i / p.n_q;
    const int node = (int)(sn % p.q_len), s = (int)(sn / p.q_len);
    const int raw_c = p.context_lens[s], raw_n = p.tree_lens ? p.tree_lens[s] : p.q_len;
    const int ctx = min(max(raw_c, 0), p.max_blocks * 16), n = min(max(raw_n, 0), p.q_len);
    if (raw_c > ctx) flag_error(p.dev_err, PA_DEVERR_BLOCK_ID);
    if (raw_n != n) flag_error(p.dev_err, PA_DEVERR_QUERY_LOC);
    const int32_t* bt = p.block_tables + (size_t)s * p.max_blocks;
    const uint64_t mask = node < n ? p.masks[sn] : 0;
    const int P = ctx - n;
    attend_row<D>(
        static_cast<T*>(p.out) + i * D, static_cast<const T*>(p.q) + i * D,
        static_cast<const KvT*>(p.k_pool), static_cast<const KvT*>(p.v_pool), 0ll,
        node < n ? ctx : 0, p.scale_log2, p.out_mul, sq[warp],
        [&](int key) -> long long {
          const int b = bt[key >> 4];
          if (b < 0 || b >= p.num_blocks) {
            flag_error(p.dev_err, PA_DEVERR_BLOCK_ID);
            return -1;
          }
          return (((long long)b * p.n_kv + h / p.group) * 16 + (key & 15)) * D;
        },
        [&](int key) { return key < P || (mask >> (key - P)) & 1; });
  }
}

template <typename T, typename KvT>
cudaError_t launch_t(const TreeParams& p, int D, cudaStream_t st) {
  const long long rows = (long long)p.num_seqs * p.q_len * p.n_q;
  const unsigned grid = (unsigned)((rows + 3) / 4 < 148 * 64 ? (rows + 3) / 4 : 148 * 64);
  D == 128 ? tree_rows_kernel<T, KvT, 128><<<grid, 128, 0, st>>>(p)
           : tree_rows_kernel<T, KvT, 64><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const TreeParams& p, int D, bool bf16, bool fp8, cudaStream_t st) {
  if (p.num_seqs == 0) return cudaSuccess;
  if (bf16)
    return fp8 ? launch_t<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st)
               : launch_t<__nv_bfloat16, __nv_bfloat16>(p, D, st);
  return fp8 ? launch_t<__half, __nv_fp8_e4m3>(p, D, st) : launch_t<__half, __half>(p, D, st);
}

}  // namespace pa
