// One attention row per warp: the 32 lanes take 32 keys at a time (each lane
// one whole dot product), the running maximum and sum of the softmax are kept
// in fp32, and the weights are handed round by shuffles for O += P V.
#pragma once

#include "pa_device.cuh"

namespace pa {

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_fp8_e4m3 x) { return (float)x; }

// keys 0 .. n - 1; row(key) gives the key's element offset in k and v (or a
// negative value: zeros), seen(key) whether the row attends to it
template <int D, typename T, typename KvT, typename RowFn, typename SeenFn>
__device__ void attend_row(T* out, const T* q, const KvT* k, const KvT* v, long long vdiff, int n,
                           float scale_log2, float out_mul, float* sq, RowFn row, SeenFn seen) {
  const int lane = threadIdx.x & 31;
  for (int d = lane; d < D; d += 32) sq[d] = to_float(q[d]) * scale_log2;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32] = {};
  for (int base = 0; base < n; base += 32) {
    const int key = base + lane;
    const bool ok = key < n && seen(key);
    const long long r = key < n ? row(key) : -1;
    float x = -INFINITY;
    if (ok) {
      x = 0.f;
      if (r >= 0)
        for (int d = 0; d < D; ++d) x = fmaf(sq[d], to_float(k[r + d]), x);
    }
    float t = x;
    for (int s = 16; s; s >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
    const float mn = fmaxf(m, t);
    const float sub = mn == -INFINITY ? 0.f : mn;
    const float a = exp2f(m - sub), w = ok ? exp2f(x - sub) : 0.f;
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] *= a;
    const uint32_t live = __ballot_sync(0xffffffffu, ok && r >= 0);
    for (uint32_t b = live; b; b &= b - 1) {
      const int j = __ffs(b) - 1;
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const long long rj = __shfl_sync(0xffffffffu, r, j);
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        o[e] = fmaf(wj, to_float(v[rj + vdiff * (key - lane + j) + 32 * e + lane]), o[e]);
    }
  }
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  const float inv = l == 0.f ? 0.f : out_mul / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) out[32 * e + lane] = T(o[e] * inv);
  __syncwarp();
}

}  // namespace pa
