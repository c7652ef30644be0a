// Moving the accepted tokens' K/V rows into place (pa_compact_tokens).
//
// Sequence s's tree occupies positions P .. P + n - 1 of its cache (P its
// prefix); the rows of the accepted nodes a_0 < a_1 < ... go to positions P,
// P + 1, ....  Because the list increases strictly, a_j >= j > i for every
// later j: the row written as number i is the source of no later move, so one
// thread may take the moves in order, a few at a time, and only ever needs
// the loads of a batch to precede the batch's stores.  A thread owns the same
// 16 bytes of every row it moves, so no two threads touch the same address.
//
// What bounds it is HBM, and before that the CTAs' chain of dependent reads
// (lengths, list, block table) ahead of the first row: with 32 layers, 128
// sequences and paths of up to 8 nodes (8 kv heads of 128, bf16) 14.1 us with
// the SMs filled once, 17.8 us with a CTA for every 256 pieces; 5.3 TB/s.  One
// layer and 4 sequences: 1.7 us.
#include "pa_device.cuh"
#include "serve_ops.h"

namespace pa {

namespace {

constexpr int kMaxNodes = 64;
constexpr int kBatch = 8;  // rows in flight per thread

// grid (sequence, piece of the launch's 16-byte columns)
__global__ void __launch_bounds__(256) compact_kernel(const CompactParams p) {
  __shared__ long long src[kMaxNodes], dst[kMaxNodes];  // 16-byte units within a pool
  __shared__ int n_moves;
  const int s = blockIdx.x, lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const bool report = blockIdx.y == 0;
    const int ctx = p.context_lens[s], m = p.accepted_lens[s];
    const int n = p.tree_lens ? p.tree_lens[s] : p.q_len;
    int err = 0, count = 0;
    if (n < 0 || n > p.q_len || ctx < n) err = PA_DEVERR_QUERY_LOC;
    else if (m < 0 || m > p.max_accepted) err = PA_DEVERR_SLOT;
    const int32_t* acc = p.accepted + (size_t)s * p.max_accepted;
    const int32_t* bt = p.block_tables + (size_t)s * p.max_blocks;
    if (!err) {
      // every entry checked before any row moves
      bool bad = false;
      for (int i = lane; i < m; i += 32) {
        const int a = acc[i];
        bad |= a < 0 || a >= n || (i > 0 && acc[i - 1] >= a);
      }
      if (__any_sync(0xffffffffu, bad)) err = PA_DEVERR_SLOT;
    }
    if (!err) {
      for (int i0 = 0; i0 < m; i0 += 32) {
        const int i = i0 + lane;
        long long a = -1, b = -1;
        if (i < m && acc[i] != i) {
          const int pa = ctx - n + acc[i], pb = ctx - n + i;
          const int ba = pa / 16 < p.max_blocks ? bt[pa / 16] : -1;
          const int bb = pb / 16 < p.max_blocks ? bt[pb / 16] : -1;
          if (ba < 0 || ba >= p.num_blocks || bb < 0 || bb >= p.num_blocks) {
            if (report) flag_error(p.dev_err, PA_DEVERR_BLOCK_ID);
          } else {
            a = ((long long)ba * p.n_kv * 16 + pa % 16) * p.chunks;
            b = ((long long)bb * p.n_kv * 16 + pb % 16) * p.chunks;
          }
        }
        const uint32_t live = __ballot_sync(0xffffffffu, a >= 0);
        if (a >= 0) {
          const int at = count + __popc(live & ((1u << lane) - 1));
          src[at] = a;
          dst[at] = b;
        }
        count += __popc(live);
      }
    } else if (report && lane == 0) {
      flag_error(p.dev_err, err);
    }
    if (lane == 0) n_moves = count;
  }
  __syncthreads();
  const int m = n_moves;
  if (m == 0) return;
  const int per_pool = p.n_kv * p.chunks;
  const int units = 2 * p.n_layers * per_pool;
  for (int u = blockIdx.y * 256 + threadIdx.x; u < units; u += gridDim.y * 256) {
    const int r = u % per_pool;
    // kv head r / chunks: 16 rows further on; piece r % chunks of its row
    uint4* pool = static_cast<uint4*>(p.pools[u / per_pool]) +
                  (long long)(r / p.chunks) * 16 * p.chunks + r % p.chunks;
    for (int i0 = 0; i0 < m; i0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < m) x[i] = pool[src[i0 + i]];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < m) pool[dst[i0 + i]] = x[i];
    }
  }
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t st) {
  const long long units = 2ll * p.n_layers * p.n_kv * p.chunks;
  // as many CTAs a sequence as it has work for, but no more than fill the SMs
  // once (8 to an SM): each begins by reading and checking its sequence's list
  const long long most = (units + 255) / 256, fill = 8ll * device_sms() / p.num_seqs;
  const unsigned y = (unsigned)(most < fill ? most : (fill > 1 ? fill : 1));
  compact_kernel<<<dim3((unsigned)p.num_seqs, y), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
