// Whole-prompt attention (pa_prefill_packed): one warp per (token, head).
#include "attn_rows.cuh"
#include "serve_ops.h"

namespace pa {

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const PromptParams p) {
  __shared__ float sq[4][D];
  const int warp = threadIdx.x >> 5;
  const long long rows = (long long)p.total * p.n_q;
  for (long long i = blockIdx.x * 4ll + warp; i < rows; i += gridDim.x * 4ll) {
    const int h = (int)(i % p.n_q), t = (int)(i / p.n_q);
    // the sequence that owns row t (the last one whose start is at or before it)
    for (int s = 0; s < p.num_seqs; ++s) {
      const int a = p.query_start_loc[s], b = min(p.query_start_loc[s + 1], p.total);
      if (a < 0 || b < a) {
        if (i == 0) flag_error(p.dev_err, PA_DEVERR_QUERY_LOC);
        continue;
      }
      if (t < a || t >= b) continue;
      const int hk = h / p.group;
      const T* k = static_cast<const T*>(p.k) + a * p.k_stride + hk * D;
      const T* v = static_cast<const T*>(p.v) + a * p.v_stride + hk * D;
      attend_row<D>(static_cast<T*>(p.out) + i * D,
                    static_cast<const T*>(p.q) + t * p.q_stride + h * D, k, v,
                    p.v_stride - p.k_stride, t - a + 1, p.scale_log2, 1.f, sq[warp],
                    [&](int key) { return key * p.k_stride; }, [](int) { return true; });
    }
  }
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, int D, bool bf16, cudaStream_t st) {
  if (p.total == 0 || p.num_seqs == 0) return cudaSuccess;
  const long long rows = (long long)p.total * p.n_q;
  const unsigned grid = (unsigned)((rows + 3) / 4 < 148 * 64 ? (rows + 3) / 4 : 148 * 64);
  if (bf16)
    D == 128 ? prompt_rows_kernel<__nv_bfloat16, 128><<<grid, 128, 0, st>>>(p)
             : prompt_rows_kernel<__nv_bfloat16, 64><<<grid, 128, 0, st>>>(p);
  else
    D == 128 ? prompt_rows_kernel<__half, 128><<<grid, 128, 0, st>>>(p)
             : prompt_rows_kernel<__half, 64><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
