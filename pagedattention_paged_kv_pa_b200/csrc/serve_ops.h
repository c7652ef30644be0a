// Launchers of the steps around decode -- whole-prompt attention, attention of
// a tree of drafted tokens, moving the accepted tokens' K/V -- that the C ABI
// shim calls.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace pa {

// SMs of the current device.
int device_sms();

// Allows `bytes` of dynamic shared memory to a kernel on the current device;
// `done` (one per kernel, zero at first) remembers the devices it was set on.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done);

// How long the waits of these kernels last, and (skip_tile >= 0) a tile that the
// load warps of every CTA leave out, as if it had never arrived (the
// pa_test_*_timeout hooks).
struct WaitParams {
  uint32_t wait_ns = (uint32_t)kWaitLimitNs;
  int skip_tile = -1;
};

// Whole-prompt attention: sequence s owns rows query_start_loc[s] ..
// query_start_loc[s + 1] - 1 of q, k, v and out.
struct PromptParams {
  void* out;  // [total][n_q][D]
  const int32_t* query_start_loc;
  int32_t* dev_err;
  float scale_log2;  // scale x log2(e)
  int n_q, n_kv, group, num_seqs, total;
  int log2_hb;       // heads of a tile: the power of two in the group size, <= 16
  WaitParams waits;  // skip_tile counts a CTA's K and V tiles
};
// tmq: 3-D map over q viewed as [total][n_q][D], box {64, 2^log2_hb, 128 /
// 2^log2_hb}; tmk / tmv: over k and v viewed as [total][n_kv][D], box {64, 1,
// 128}; all with the 128-byte swizzle.
cudaError_t launch_prompt(const PromptParams& p, int D, bool bf16, const CUtensorMap* tmq,
                          const CUtensorMap* tmk, const CUtensorMap* tmv, cudaStream_t st);

// Attention of a tree of drafted tokens over the paged cache.
struct TreeParams {
  void* out;  // [num_seqs][q_len][n_q][D]
  const void *q, *k_pool, *v_pool;
  const int32_t *block_tables, *context_lens, *tree_lens;
  const uint64_t* masks;  // [num_seqs][q_len]
  int32_t* dev_err;
  float scale_log2;  // scale x log2(e) (x k_scale for fp8 caches)
  float out_mul;     // v_scale for fp8 caches, else 1
  int n_q, n_kv, group, num_seqs, q_len, max_blocks, num_blocks;
  int q_box_nodes;  // nodes of the query map's box
  WaitParams waits;  // skip_tile counts a CTA's K tiles
  // set by launch_tree
  float* ws_o;     // [CTA][2 slots][rows][D] unnormalised segment outputs
  float2* ws_ml;   // [CTA][2 slots][rows] (log2-domain maximum, sum)
  int row_groups;  // CTAs side by side over the same keys
  int step_keys, log2_step;  // keys of a step of the work split
  int seg_cost;    // fixed costs of a unit, in steps
};
constexpr int kTreeCtas = 148;  // most CTAs of a launch: the workspace is laid out for them
size_t tree_ws_bytes(int q_len, int group, int D);
// tmq (16-bit caches): 3-D map over q viewed as [num_seqs x q_len][n_q][D], box
// {64, group, q_box_nodes}, q_box_nodes = min(q_len, 128 / group); tmk / tmv:
// 2-D maps over the pools viewed as [num_blocks x n_kv x 16][D], box {64, 16}
// with the 128-byte swizzle, for E4M3 {D, 16} with the D-byte swizzle.
cudaError_t launch_tree(TreeParams& p, int D, bool bf16, bool fp8, void* workspace,
                        const CUtensorMap* tmq, const CUtensorMap* tmk, const CUtensorMap* tmv,
                        cudaStream_t st);

// Moving the accepted tokens' rows, all layers of a launch at once.
constexpr int kCompactLayers = 64;  // layers per launch (pointers travel as arguments)
struct CompactParams {
  void* pools[2 * kCompactLayers];  // k_pool, v_pool of each layer
  const int32_t *block_tables, *context_lens, *tree_lens, *accepted, *accepted_lens;
  int32_t* dev_err;
  int n_layers, num_seqs, q_len, max_accepted, max_blocks, num_blocks, n_kv;
  int chunks;  // 16-byte pieces of a row of one kv head
};
cudaError_t launch_compact(const CompactParams& p, cudaStream_t st);

}  // namespace pa
