// Attention of a tree of drafted tokens over the paged cache (pa_decode_tree)
// on tcgen05 tensor cores.
//
// Node i of a sequence attends to the prefix and to the nodes of its mask:
// out = sum of 2^(s_u - m) v_u / l over those keys u, s = scale log2(e) q . k,
// in one pass with the running (m, l) of attn_tile.cuh.  Only the last tiles
// of a context hold tree nodes; there a row's 64-bit mask, shifted to the
// tile, says which keys it sees.
//
// Rows.  For one (sequence, kv head) the (node, query head) pairs are rows of
// 128-row tiles, QT = floor(128 / G) nodes of G heads to a tile, so that a K/V
// tile of 128 keys is read once for all heads of its kv head.  A CTA holds two
// tiles, A and B, in TMEM (S 128 fp32 columns, P over S as 16-bit pairs, O):
// the tensor cores work on one while the softmax of the other runs.
//  - Trees of one tile (SPLIT): A and B are the same rows over alternate key
//    tiles, merged at the end of a run of keys.  K/V bytes bound these.
//  - Larger trees: A and B are two row tiles over the same keys; trees of more
//    than two tiles take two CTAs side by side over the same keys (the second
//    reader of a K/V tile finds it in L2).
//
// Work split.  Persistent CTAs.  The (sequence, kv head) units lie end to end,
// measured in key steps (256 keys when split, else 128) plus seg_cost steps'
// worth of time for a unit's fixed costs; share c of C is [c T / C, (c + 1) T /
// C) of the total T.  A run of a unit's steps inside one share is a segment.  A
// segment that is the whole unit writes the output; others write their
// unnormalised O and (m, l) to one of their CTA's two workspace slots (0: the
// unit began in an earlier share, 1: it ends in a later one), which
// tree_merge_kernel, a programmatic dependent, combines in share order.
//
// Roles: warps 0-3 softmax of A, 4-7 of B (one thread per row), warps 8 and 9
// issue the MMAs of A and B, warps 10 and 11 load K (and Q), 12 and 13 V (16-token
// blocks by TMA through the block table; rows of the block a context ends in
// are copied, rows past it and blocks with a bad id zeroed by the warp itself),
// warp 14 walks the share.  E4M3 caches: K and V arrive as raw tiles, and warps
// 16-19 widen K, 20-23 V to the f16 operands (code x 2^-8, exact, undone by the
// score and output scales); the K converters also write the query rows, scaled
// by a power of two into f16's range when they are bf16, and P is f16.  Every
// wait is bounded; a role that gives up flags PA_DEVERR_TIMEOUT and leaves, and
// the CTA drains its loads and MMAs and frees TMEM.
//
// Measured back to back in a CUDA graph: 64 contexts of up to 8,000 with 16 nodes,
// 64/8 heads of 128, bf16, 145 us = 5.5 TB/s of K/V (HBM bounds it; over seconds
// the power limit, 1,485 MHz and 170 us); 16 of up to 8,191 with 64 nodes 130 us =
// 735 TFLOP/s (the chain P -> O += P V -> S -> softmax); 96 of up to 4,000 with 24 nodes, 32/8 x 128, E4M3, 135 us = 2.4 TB/s
// (the chain through the converters; issue 50 %, ALU 41 %); one context of 777 with
// 8 nodes 14.9 us with the merge, of 8 alone 11.7 us (start-up of two kernels).
#include <type_traits>

#include "attn_tile.cuh"
#include "serve_ops.h"

namespace pa {

namespace {

using attn::kTileM;
using attn::kTileN;

// two load warps each for K (10, 11) and V (12, 13)
constexpr int kMmaWarp = 8, kLoadWarp = 10, kSchedWarp = 14, kConvWarp = 16;  // 15 idle
constexpr int kSegs = 4;  // segments scheduled ahead
constexpr uint32_t kTmemCols = 512;
// rows and warps of a merge CTA: one wave of CTAs, each of which finds its unit
constexpr int kMergeRows = 32, kMergeWarps = 16;

template <int D, bool FP8, bool SPLIT>
struct Lay {
  static constexpr int kOp = kTileN * D * 2;  // one 16-bit Q, K or V tile
  static constexpr int kRaw = kTileN * D;     // one E4M3 K or V tile
  static constexpr int kQ = SPLIT ? 1 : 2;    // Q tiles
  static constexpr int kScale = 128 / D;
  // K and V stages.  Split: even numbers, so that a stage always belongs to the
  // same tile X (a segment takes an even number of stages, the last one empty
  // if need be) and X's MMA warp sees every phase of its stages' barriers
  static constexpr int kKS = (FP8 ? 2 : (SPLIT ? 4 : 3)) * kScale;
  static constexpr int kVS = (FP8 && !SPLIT && D == 128 ? 1 : 2) * kScale;
  static_assert(!SPLIT || (kKS % 2 == 0 && kVS % 2 == 0), "a stage per tile");
  static constexpr int kRS = FP8 ? 2 * kScale : 0;  // raw K stages, and raw V stages
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kQ * kOp;
  static constexpr int kVOff = kKOff + kKS * kOp;
  static constexpr int kRawOff = kVOff + kVS * kOp;
  static constexpr int kRedOff = kRawOff + 2 * kRS * kRaw;  // [2][128] float2
  static constexpr int kBarOff = kRedOff + (SPLIT ? 2048 : 0);
  static constexpr int kExpOff = kBarOff + 768;  // E4M3: the query rows' exponents, int8
  static constexpr int kSmem = kExpOff + 256 * kQ;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  // TMEM columns: S_A 0, S_B 128; a 64-wide head leaves room for P beside S, so
  // that S of the next tile is made while the softmax works on this one
  static constexpr bool kSepP = D == 64;
  static constexpr int tP(int x) { return kSepP ? 256 + 64 * x : 128 * x; }
  static constexpr int tO(int x) { return kSepP ? 384 + 64 * x : 256 + 128 * x; }
  static constexpr int kThreads = FP8 ? 768 : 512;
  // The softmax reads S once into 128 registers, or (kLean) twice 64 at a time
  // with one copy of the code for both halves, which the instruction cache
  // prefers: E4M3 trees 165 -> 132 us, 16 x 64-node bf16 trees 133 -> 131 us;
  // 64-wide 16-bit heads, whose next S is made early, 38 -> 39 us.
  static constexpr bool kLean = FP8 || D == 128;
  // registers: 768 x 80 = 61,440 = 256 x 128 + 512 x 56, or 512 x 128 = 65,536 =
  // 256 x 144 + 256 x 112 = 256 x 184 + 256 x 72
  static constexpr int kSoftRegs = FP8 ? 128 : (kLean ? 144 : 184);
  static constexpr int kOtherRegs = FP8 ? 56 : (kLean ? 112 : 72);
  // readers of a segment: 8 softmax warps, 2 MMA, 4 loads, 8 converters
  static constexpr uint32_t kReaders = FP8 ? 22 : 14;
};

struct Seg {
  int s, h;    // s < 0: no more
  int ctx, n;  // context length, nodes
  int t0, t1;  // key tiles
  int slot;    // workspace slot, or -1: the whole unit
};

struct Bars {
  uint64_t k_full[8], k_empty[8], v_full[4], v_empty[4], raw_full[2][4], raw_empty[2][4];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], o_free[2], red[2];
  uint64_t s_empty[2], pv_done[2];  // P beside S only
  uint64_t done[2], turn[2];
  Seg segs[kSegs];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 768, "barriers");

using attn::wait_all;
using attn::wait_ok;

// The segment stream as one role reads it.
struct Reader {
  int k = 0;
  __device__ __forceinline__ bool next(Bars* B, const TreeParams& p, Seg& g) {
    const int slot = k % kSegs;
    if (!wait_ok(&B->seg_full[slot], (k / kSegs) & 1, B, p)) return false;
    g = B->segs[slot];
    ++k;
    return g.s >= 0;
  }
  __device__ __forceinline__ void done(Bars* B) { mbar_arrive(&B->seg_empty[(k - 1) % kSegs]); }
};

// ------------------------------------------------------------- work split
__device__ __forceinline__ int seq_ctx(const TreeParams& p, int s) {
  return min(max(__ldg(&p.context_lens[s]), 0), p.max_blocks * 16);
}
__device__ __forceinline__ int seq_nodes(const TreeParams& p, int s) {
  return p.tree_lens ? min(max(__ldg(&p.tree_lens[s]), 0), p.q_len) : p.q_len;
}
__device__ __forceinline__ int seq_steps(const TreeParams& p, int s) {
  const int n = seq_nodes(p, s), c = seq_ctx(p, s);
  return n > 0 ? (c + p.step_keys - 1) >> p.log2_step : 0;
}
__device__ __forceinline__ int weight(const TreeParams& p, int steps) {
  return steps > 0 ? steps + p.seg_cost : 0;
}

// T, by one warp; `first` gets the weight of sequence `lane`; flags lengths out
// of range when `report`
__device__ long long total_weight(const TreeParams& p, int lane, bool report, int& first) {
  long long part = first = lane < p.num_seqs ? weight(p, seq_steps(p, lane)) : 0;
#pragma unroll 1
  for (int s = 32 + lane; s < p.num_seqs; s += 32) part += weight(p, seq_steps(p, s));
  if (report) {
    int err = 0;
#pragma unroll 1
    for (int s = lane; s < p.num_seqs; s += 32) {
      const int n = p.tree_lens ? __ldg(&p.tree_lens[s]) : p.q_len;
      if (n < 0 || n > p.q_len) err |= PA_DEVERR_QUERY_LOC;
      if (__ldg(&p.context_lens[s]) > p.max_blocks * 16) err |= PA_DEVERR_BLOCK_ID;
    }
    if (err) flag_error(p.dev_err, err);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) part += __shfl_xor_sync(0xffffffffu, part, m);
  return part * p.n_kv;
}
__device__ __forceinline__ int quotient(long long a, int b) {
  return a < 0x7fffffff ? (int)a / b : (int)(a / b);
}
// The shares: share c starts at floor(c T / C) = c floor(T / C) + floor(c (T mod
// C) / C).  With fewer positions than CTAs, C is T, so that none is empty.
struct Shares {
  long long each;
  int C, rest;
  __device__ Shares(long long T, int ctas) {
    C = T < ctas ? max((int)T, 1) : ctas;
    each = T < 0x7fffffff ? (int)T / C : T / C;
    rest = (int)(T - each * C);
  }
  __device__ __forceinline__ long long start(int c) const { return each * c + c * rest / C; }
};
// The sequence whose span [gs, gs + n_kv w) of positions holds X, by one warp.
__device__ bool locate(const TreeParams& p, long long X, int lane, int first, int& s_out,
                       long long& gs_out, int& w_out) {
  long long acc = 0;
#pragma unroll 1
  for (int base = 0; base < p.num_seqs; base += 32) {
    const int s = base + lane;
    const int n = base == 0 ? first : (s < p.num_seqs ? weight(p, seq_steps(p, s)) : 0);
    int incl = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += v;
    }
    const long long gs = acc + (long long)(incl - n) * p.n_kv;
    const long long ge = acc + (long long)incl * p.n_kv;
    const uint32_t hit = __ballot_sync(0xffffffffu, gs <= X && X < ge);
    if (hit) {
      const int src = __ffs(hit) - 1;
      s_out = __shfl_sync(0xffffffffu, s, src);
      gs_out = __shfl_sync(0xffffffffu, gs, src);
      w_out = __shfl_sync(0xffffffffu, n, src);
      return true;
    }
    acc += (long long)__shfl_sync(0xffffffffu, incl, 31) * p.n_kv;
  }
  return false;
}

// ------------------------------------------------------------------- tiles
// 16-bit operand tile with the 128-byte swizzle: 128 rows of 64 elements in
// D / 64 halves 16 KiB apart; chunk = 8 consecutive elements
__device__ __forceinline__ uint32_t op_off(int row, int chunk) {
  return (chunk >> 3) * 16384 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
// E4M3 tile: 128 rows of D bytes, 128- or 64-byte swizzle; chunk = 16 codes
template <int D>
__device__ __forceinline__ uint32_t raw_off(int row, int chunk) {
  return D == 128 ? swz128(row * 128 + chunk * 16) : swz64(row * 64 + chunk * 16);
}

// The block id of lane m < 4's block 4 half + m of tile t (-1 past the context).
__device__ __forceinline__ int block_id(const TreeParams& p, const Seg& g, int t, int half,
                                        int lane) {
  const int blk = t * 8 + half * 4 + lane;
  return lane < 4 && blk * 16 < g.ctx ? __ldg(&p.block_tables[(size_t)g.s * p.max_blocks + blk])
                                      : -1;
}

// Loads half of tile t of a (sequence, kv head) into `dst`, by one warp: whole
// blocks of the context by TMA, the other rows written here.
template <int D, bool FP8>
__device__ __forceinline__ void load_tile(const TreeParams& p, const Seg& g, int t, int half, uint8_t* dst,
                                          const CUtensorMap* map, const uint8_t* pool,
                                          uint64_t* full, int lane, int phys, bool report,
                                          uint64_t policy) {
  constexpr int kRow = FP8 ? D : 2 * D;  // bytes of a row
  const int b = half * 4 + lane, blk = t * 8 + b;
  const bool in_ctx = lane < 4 && blk * 16 < g.ctx;
  const bool in_range = phys >= 0 && phys < p.num_blocks;
  if (report && in_ctx && !in_range) flag_error(p.dev_err, PA_DEVERR_BLOCK_ID);
  const bool whole = in_ctx && in_range && blk * 16 + 16 <= g.ctx;
  const uint32_t whole_m = __ballot_sync(0xffffffffu, whole);
  for (uint32_t pm = __ballot_sync(0xffffffffu, lane < 4 && !whole); pm; pm &= pm - 1) {
    const int ph = __shfl_sync(0xffffffffu, phys, __ffs(pm) - 1);
    const int m = half * 4 + __ffs(pm) - 1;  // block of the tile
    const bool ok_id = ph >= 0 && ph < p.num_blocks;
    const int nvalid = ok_id ? max(0, min(16, g.ctx - (t * 8 + m) * 16)) : 0;
    const uint8_t* src = pool + (long long)(ok_id ? ph * p.n_kv + g.h : 0) * 16 * kRow;
#pragma unroll
    for (int u = 0; u < kRow / 32; ++u) {  // 16 rows of kRow / 16 chunks
      const int idx = lane + 32 * u, r = idx / (kRow / 16), cc = idx % (kRow / 16);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < nvalid) v = __ldg(reinterpret_cast<const uint4*>(src + r * kRow + cc * 16));
      *reinterpret_cast<uint4*>(dst + (FP8 ? raw_off<D>(16 * m + r, cc)
                                           : op_off(16 * m + r, cc))) = v;
    }
  }
  tc::fence_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive_expect_tx(full, __popc(whole_m) * 16u * kRow);
  __syncwarp();
  if (whole) {
    const int y = (phys * p.n_kv + g.h) * 16;  // row of the [rows][D] view
    if constexpr (FP8) {
      tma_load_2d_hint(dst + b * 16 * kRow, map, full, 0, y, policy);
    } else {
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        tma_load_2d_hint(dst + h * 16384 + b * 2048, map, full, 64 * h, y, policy);
    }
  }
}

// A query row as the f16 operand row `r` of an E4M3 cache's products: a bf16 row
// is multiplied by 2^e first, e left in *exponent for its scores; no row (null):
// zeros.
template <bool BF16, int D>
__device__ __forceinline__ void write_query_row(uint8_t* tile, int r, const void* row,
                                                int8_t* exponent) {
  const uint4* src = static_cast<const uint4*>(row);
  int e = 0;
  if constexpr (BF16) {
    uint32_t mag = 0;
#pragma unroll 4
    for (int ch = 0; ch < D / 8; ++ch) {
      const uint4 v = row ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
      mag = max(max(mag, max(bf16x2_max_mag(v.x), bf16x2_max_mag(v.y))),
                max(bf16x2_max_mag(v.z), bf16x2_max_mag(v.w)));
    }
    e = f16_row_shift(mag);
  }
  *exponent = (int8_t)e;
  const float up = exp2i(e);
#pragma unroll 4
  for (int ch = 0; ch < D / 8; ++ch) {
    uint4 v = row ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
    if constexpr (BF16)
      v = make_uint4(bf16x2_to_f16x2_scaled(v.x, up), bf16x2_to_f16x2_scaled(v.y, up),
                     bf16x2_to_f16x2_scaled(v.z, up), bf16x2_to_f16x2_scaled(v.w, up));
    *reinterpret_cast<uint4*>(tile + op_off(r, ch)) = v;
  }
}

// bits of keys first .. first + 31 that a row with tree mask `mask` and the
// prefix 0 .. P - 1 sees
__device__ __forceinline__ uint32_t seen_bits(int first, int P, uint64_t mask) {
  const int sh = first - P;  // the node at the first key
  if (sh <= -32) return 0xffffffffu;
  if (sh < 0) return (uint32_t)(mask << -sh) | ((1u << -sh) - 1u);
  return sh < 64 ? (uint32_t)(mask >> sh) : 0u;
}

template <bool BF16, int D, bool FP8, bool SPLIT>
__global__ void __launch_bounds__(FP8 ? 768 : 512, 1)
    tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmq,
                const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using L = Lay<D, FP8, SPLIT>;
  constexpr bool kOpBf16 = BF16 && !FP8;  // the operands' type
  constexpr int KS = L::kKS, VS = L::kVS, RS = FP8 ? L::kRS : 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* B = reinterpret_cast<Bars*>(smem + L::kBarOff);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrg = p.row_groups, rg = blockIdx.x % nrg;  // CTAs side by side
  const int G = p.group, QT = kTileM / G;
  // nodes of this CTA's tile X that sequence g has
  auto tile_nodes = [&](const Seg& g, int x) -> int {
    return max(0, min(QT, g.n - (SPLIT ? 0 : 2 * rg + x) * QT));
  };

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&B->k_full[s], FP8 ? 128 : 2);
      mbar_init(&B->k_empty[s], SPLIT ? 1 : 2);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&B->v_full[s], FP8 ? 128 : 2);
      mbar_init(&B->v_empty[s], SPLIT ? 1 : 2);
    }
    for (int s = 0; s < RS; ++s) {
      for (int v = 0; v < 2; ++v) {
        mbar_init(&B->raw_full[v][s], 2);
        mbar_init(&B->raw_empty[v][s], 128);
      }
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&B->seg_full[s], 1);
      mbar_init(&B->seg_empty[s], L::kReaders);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&B->q_full[x], FP8 ? 128 : 1);
      mbar_init(&B->done[x], 1);
      mbar_init(&B->turn[x], 1);
      mbar_init(&B->q_empty[x], SPLIT ? 2 : 1);
      mbar_init(&B->s_full[x], 1);
      mbar_init(&B->p_half[x], 128);
      mbar_init(&B->p_full[x], 128);
      mbar_init(&B->s_empty[x], 128);
      mbar_init(&B->pv_done[x], 1);
      mbar_init(&B->o_full[x], 1);
      mbar_init(&B->o_free[x], SPLIT ? 256 : 128);
      mbar_init(&B->red[x], 128);
    }
    B->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::alloc(&B->tmem_base, kTmemCols);
  if (warp == kLoadWarp && lane == 0) {
    if (!FP8) prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = B->tmem_base;

  if (warp >= kMmaWarp) {
    tc::regs_dec<L::kOtherRegs>();
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // --------------------------------------------------------- MMA issuers
      // one warp per tile X: per step j, O_X += P_X V of step j - 1 and S_X =
      // Q_X K^T of step j (in this order where P lies over S: the tensor core
      // keeps it; else S first).  The whole warp walks the steps and waits, one
      // lane issues.  The waits of one warp run while the other's MMAs do.  Where
      // A and B share the key tiles and the products bound them they take turns,
      // so that one's batch is not spread over the other's and their softmax
      // passes fall into opposite phases.
      constexpr bool kTurns = !SPLIT && !L::kSepP;
      constexpr uint32_t idesc_s = tc::idesc_f16(kOpBf16, false, kTileM, kTileN);
      constexpr uint32_t idesc_pv = tc::idesc_f16(kOpBf16, true, kTileM, D);
      constexpr uint64_t kOpStep = L::kOp >> 4;  // descriptors count 16 bytes
      const int x = warp - kMmaWarp, qx = SPLIT ? 0 : x;
      const uint64_t dQ = tc::smem_desc(sbase + L::kQOff + qx * L::kOp),
                     dK = tc::smem_desc(sbase + L::kKOff),
                     dV = tc::smem_desc(sbase + L::kVOff, 16384);
      const uint32_t tS = tmem + x * 128, tP = tmem + L::tP(x), tO = tmem + L::tO(x);
      Reader rd;
      Seg g;
      bool ok = true, issued = false;
      uint32_t c = 0;  // key tiles before this segment
      uint32_t segs = 0, items = 0, tiles = 0, turns = 0;
      auto scores = [&](uint64_t k, bool last) {
        tc::fence_after();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (kk >> 2) * 1024 + (kk & 3) * 2;
            tc::mma(tS, dQ + off, k + off, idesc_s, kk > 0);
          }
          tc::commit(&B->s_full[x]);
          if (last) tc::commit(&B->q_empty[qx]);
        }
        __syncwarp();
      };
      while (ok && __all_sync(0xffffffffu, rd.next(B, p, g))) {
        if (lane == 0) rd.done(B);
        __syncwarp();
        const int nt = g.t1 - g.t0, n = SPLIT ? (nt + 1) / 2 : nt;  // A always has a tile
        const int mine = x == 0 ? n : (SPLIT ? nt / 2 : (tile_nodes(g, 1) > 0 ? nt : 0));
        if (SPLIT || mine > 0)
          ok = wait_all(&B->q_full[qx], (SPLIT ? segs : items) & 1, B, p);
        // (split: a tile without a step is done with Q)
        if (SPLIT && mine == 0 && lane == 0) mbar_arrive(&B->q_empty[0]);
        const uint32_t before = SPLIT ? segs : items;  // O_X read out so often
        for (int j = 0; j <= n && ok; ++j, ++turns) {
          const bool do_pv = j > 0 && j <= mine, do_s = j < mine;
          // split: every second key tile (and stage); else all of them, with
          // rows or without
          const uint32_t ck = c + (SPLIT ? 2 * j + x : j), cv = ck - (SPLIT ? 2 : 1);
          const bool use_k = j < n, use_v = j > 0;
          const int sk = ck % KS, sv = cv % VS;
          const uint64_t v = dV + sv * kOpStep, k = dK + sk * kOpStep;
          const uint32_t par = (tiles - 1) & 1;
          if (use_v) ok = wait_all(&B->v_full[sv], (cv / VS) & 1, B, p);
          if (use_k) ok = ok && wait_all(&B->k_full[sk], (ck / KS) & 1, B, p);
          if (L::kSepP && do_s) {  // S beside P: as soon as the softmax has read the last S
            if (tiles > 0) ok = ok && wait_all(&B->s_empty[x], (tiles - 1) & 1, B, p);
            if (!ok) break;
            scores(k, j == mine - 1);
          }
          if (do_pv) {
            ok = ok && wait_all(&B->p_half[x], par, B, p);
            if (j == 1 && before > 0)
              ok = ok && wait_all(&B->o_free[x], (before - 1) & 1, B, p);
          }
          if (kTurns && (x > 0 || turns > 0))
            ok = ok && wait_all(&B->turn[x], (turns - 1 + x) & 1, B, p);
          if (!ok) break;
          if (do_pv) {
            tc::fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 16 keys a step = two 8-row groups of V
                tc::mma_ts(tO, tP + kk * 8, v + kk * 128, idesc_pv,
                           (j == 1 && kk == 0) ? 0u : 1u);
            }
            __syncwarp();
            ok = wait_all(&B->p_full[x], par, B, p);
            if (!ok) break;
            tc::fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 4; kk < 8; ++kk)
                tc::mma_ts(tO, tP + kk * 8, v + kk * 128, idesc_pv, 1u);
              if (L::kSepP) tc::commit(&B->pv_done[x]);
              if (j == mine) tc::commit(&B->o_full[x]);
            }
            __syncwarp();
          }
          if (!L::kSepP && do_s) scores(k, j == mine - 1);
          if (tc::elect_one()) {
            if (kTurns) mbar_arrive(&B->turn[x ^ 1]);
            // a stage is free once the MMAs on it are done (both warps', unless
            // split)
            if (use_v) tc::commit(&B->v_empty[sv]);
            if (use_k) tc::commit(&B->k_empty[sk]);
          }
          __syncwarp();
          issued = true;
          tiles += do_s;
        }
        c += SPLIT ? 2 * n : nt;
        ++segs;
        items += mine > 0;
      }
      // everything issued above has completed before TMEM is released
      if (issued) {
        if (tc::elect_one()) tc::commit(&B->done[x]);
        __syncwarp();
        mbar_wait(&B->done[x], 0, p.waits.wait_ns);
      }
    } else if (warp >= kLoadWarp && warp < kLoadWarp + 4) {
      // ---------------------------------------------------------------- loads
      // two warps for K, two for V: each loads half the blocks of every tile
      // (a copy takes a lane of a warp about 100 clocks to issue)
      const bool vop = warp >= kLoadWarp + 2;
      const int half = (warp - kLoadWarp) & 1;
      const int NS = FP8 ? RS : (vop ? VS : KS);
      uint64_t* full = FP8 ? B->raw_full[vop] : (vop ? B->v_full : B->k_full);
      uint64_t* empty = FP8 ? B->raw_empty[vop] : (vop ? B->v_empty : B->k_empty);
      constexpr int kStage = FP8 ? L::kRaw : L::kOp;
      uint8_t* ring = smem + (FP8 ? L::kRawOff + (vop ? RS * kStage : 0)
                                  : (vop ? L::kVOff : L::kKOff));
      const uint8_t* pool = static_cast<const uint8_t*>(vop ? p.v_pool : p.k_pool);
      const CUtensorMap* map = vop ? &tmv : &tmk;
      // K/V are read once (or twice at about the same time)
      const uint64_t policy = l2_policy_evict_first();
      const bool q_too = !FP8 && warp == kLoadWarp;  // the first one loads Q
      Reader rd;
      Seg g;
      bool ok = true;
      uint32_t c = 0;
      int nq[2] = {0, 0};
      while (ok && __all_sync(0xffffffffu, rd.next(B, p, g))) {
        __syncwarp();
        if (lane == 0) rd.done(B);
        int id = block_id(p, g, g.t0, half, lane);
        for (int t = g.t0; t < g.t1 && ok; ++t, ++c) {
          // the next tile's block ids arrive while this tile waits for a stage
          const int id_next = t + 1 < g.t1 ? block_id(p, g, t + 1, half, lane) : -1;
          const int st = c % NS;
          if (c >= (uint32_t)NS) ok = wait_all(&empty[st], (c / NS - 1) & 1, B, p);
          if (!ok) break;
          if (vop || c != (uint32_t)p.waits.skip_tile)
            load_tile<D, FP8>(p, g, t, half, ring + st * kStage, map, pool, &full[st], lane, id,
                              !vop, policy);
          id = id_next;
          if (SPLIT && !FP8 && t + 1 == g.t1 && ((g.t1 - g.t0) & 1)) {  // B's empty stage
            ++c;
            const int se = c % NS;
            if (c >= (uint32_t)NS) ok = wait_all(&empty[se], (c / NS - 1) & 1, B, p);
            if (!ok) break;
            if (lane == 0) mbar_arrive(&full[se]);
          }
          if (q_too && t == g.t0) {
#pragma unroll
            for (int x = 0; x < L::kQ; ++x) {
              if (!ok || tile_nodes(g, x) == 0) continue;
              if (nq[x] > 0) ok = wait_all(&B->q_empty[x], (nq[x] - 1) & 1, B, p);
              if (!ok) continue;
              ++nq[x];
              if (lane == 0) {
                uint8_t* d = smem + L::kQOff + x * L::kOp;
                const int node = (SPLIT ? 0 : 2 * rg + x) * QT;
                mbar_arrive_expect_tx(&B->q_full[x], p.q_box_nodes * G * D * 2);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                  tc::tma_load_3d(d + h * 16384, &tmq, &B->q_full[x], 64 * h, g.h * G,
                                  g.s * p.q_len + node);
              }
              __syncwarp();
            }
          }
        }
      }
      // loads in flight land before the CTA exits
      for (uint32_t u = c > (uint32_t)NS ? c - NS : 0; u < c; ++u)
        mbar_wait(&full[u % NS], (u / NS) & 1, p.waits.wait_ns);
      if (q_too)
#pragma unroll
        for (int x = 0; x < L::kQ; ++x)
          if (nq[x] > 0) mbar_wait(&B->q_full[x], (nq[x] - 1) & 1, p.waits.wait_ns);
    } else if (warp == kSchedWarp) {
      // ------------------------------------------------------------ scheduler
      int first;
      const Shares sh(total_weight(p, lane, blockIdx.x == 0, first), gridDim.x / nrg);
      const int sc = blockIdx.x / nrg;
      const long long gbeg = sh.start(sc), gend = sh.start(sc + 1);
      int s = 0, w = 0, h = 0, step = 0;
      long long gs = 0;
      bool more = sc < sh.C && gbeg < gend && locate(p, gbeg, lane, first, s, gs, w);
      if (more) {
        h = quotient(gbeg - gs, w);
        step = max(0, (int)(gbeg - gs - (long long)h * w) - p.seg_cost);
      }
      for (int k = 0;;) {
        Seg g;
        g.s = -1;
        bool emit = !more;
        if (more) {
          const int steps = w - p.seg_cost;
          const long long u = gs + (long long)h * w + p.seg_cost;  // of the unit's first step
          if (u + step >= gend) {
            more = false;
            continue;
          }
          const int end = (int)min((long long)steps, gend - u);
          g.s = s;
          g.h = h;
          g.ctx = seq_ctx(p, s);
          g.n = seq_nodes(p, s);
          const int tps = p.step_keys / kTileN, nt = (g.ctx + kTileN - 1) / kTileN;
          g.t0 = step * tps;
          g.t1 = min(nt, end * tps);
          g.slot = step > 0 ? 0 : (end < steps ? 1 : -1);
          emit = tile_nodes(g, 0) > 0;  // the second CTA of a small tree has no rows
          step = 0;
          if (end < steps) {
            more = false;
          } else if (++h == p.n_kv) {
            h = 0;
            gs += (long long)p.n_kv * w;
            do {
              ++s;
              w = s < p.num_seqs ? weight(p, seq_steps(p, s)) : 0;
            } while (s < p.num_seqs && w == 0);
            more = s < p.num_seqs;
          }
        }
        if (!emit) continue;
        const int slot = k % kSegs;
        const bool ok = k < kSegs || wait_ok(&B->seg_empty[slot], (k / kSegs - 1) & 1, B, p);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) {
          B->segs[slot] = g;
          mbar_arrive(&B->seg_full[slot]);
        }
        __syncwarp();
        ++k;
        if (g.s < 0) break;
      }
    } else if (FP8 && warp >= kConvWarp) {
      // ------------------------------------- converters: 4 warps for K, 4 for V
      const bool vop = warp >= kConvWarp + 4;
      const int ct = (threadIdx.x - 32 * kConvWarp) & 127;
      const int NS = vop ? VS : KS;
      uint64_t* full = vop ? B->v_full : B->k_full;
      uint64_t* empty = vop ? B->v_empty : B->k_empty;
      constexpr int kCh = D / 16;  // 16-code chunks of a row
      Reader rd;
      Seg g;
      bool ok = true;
      uint32_t c = 0, cr = 0;  // operand tiles, raw tiles
      int nq[2] = {0, 0};
      while (ok && __all_sync(0xffffffffu, rd.next(B, p, g))) {
        __syncwarp();
        if (lane == 0) rd.done(B);
        // the K converters write the segment's query rows first
#pragma unroll
        for (int x = 0; x < L::kQ; ++x) {
          const int nodes = tile_nodes(g, x);
          if (vop || !ok || nodes == 0) continue;
          // S of the segment before is done: its rows are done with, and the
          // exponents of the one before that have been read (its P was written)
          if (nq[x] > 0) ok = wait_all(&B->q_empty[x], (nq[x] - 1) & 1, B, p);
          if (!ok) continue;
          const int ri = ct / G, node = (SPLIT ? 0 : 2 * rg + x) * QT + ri;
          write_query_row<BF16, D>(
              smem + L::kQOff + x * L::kOp, ct,
              ri < nodes ? static_cast<const T16*>(p.q) +
                               (((size_t)g.s * p.q_len + node) * p.n_q + g.h * G + ct - ri * G) * D
                         : nullptr,
              reinterpret_cast<int8_t*>(smem + L::kExpOff) + ((nq[x] & 1) * L::kQ + x) * 128 + ct);
          tc::fence_async_smem();
          mbar_arrive(&B->q_full[x]);
          ++nq[x];
        }
        for (int t = g.t0; t < g.t1 && ok; ++t, ++c, ++cr) {
          const int st = c % NS, rs = cr % RS;
          bool w = wait_ok(&B->raw_full[vop][rs], (cr / RS) & 1, B, p);
          w = w && (c < (uint32_t)NS || wait_ok(&empty[st], (c / NS - 1) & 1, B, p));
          ok = __all_sync(0xffffffffu, w);
          if (!ok) break;
          const uint8_t* src = smem + L::kRawOff + ((vop ? RS : 0) + rs) * L::kRaw;
          uint8_t* dst = smem + (vop ? L::kVOff : L::kKOff) + st * L::kOp;
#pragma unroll 2
          for (int m = 0; m < kCh; ++m) {
            // 8 lanes take 8 rows of one chunk, then the next chunk: their
            // 16-byte stores fall into different banks (the swizzle turns with
            // the row)
            const int key = (ct & 7) + 8 * (ct / (8 * kCh)) + (128 / kCh) * m, cc = (ct >> 3) % kCh;
            const uint4 x = *reinterpret_cast<const uint4*>(src + raw_off<D>(key, cc));
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[2 * e] = e4m3x2_to_f16x2_div256(xw[e], 0x4140u);
              y[2 * e + 1] = e4m3x2_to_f16x2_div256(xw[e], 0x4342u);
            }
            *reinterpret_cast<uint4*>(dst + op_off(key, 2 * cc)) =
                make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(dst + op_off(key, 2 * cc + 1)) =
                make_uint4(y[4], y[5], y[6], y[7]);
          }
          mbar_arrive(&B->raw_empty[vop][rs]);
          tc::fence_async_smem();
          mbar_arrive(&full[st]);
        }
        if (SPLIT && ok && ((g.t1 - g.t0) & 1)) {  // B's empty stage
          const int st = c % NS;
          if (c >= (uint32_t)NS) ok = wait_all(&empty[st], (c / NS - 1) & 1, B, p);
          if (ok) mbar_arrive(&full[st]);
          ++c;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    tc::regs_inc<L::kSoftRegs>();
    const int x = warp >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row = TMEM lane
    const int ri = r / G, rh = r - ri * G;  // its node within the tile, its head
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lanes, tP = tmem + L::tP(x) + lanes,
                   tO = tmem + L::tO(x) + lanes;
    // rows without a node, and sequences without context: zeros
    if (rg == 0)
      for (int s = blockIdx.x / nrg; s < p.num_seqs; s += gridDim.x / nrg) {
        const int from = seq_ctx(p, s) > 0 ? seq_nodes(p, s) : 0;
        uint4* o = reinterpret_cast<uint4*>(static_cast<T16*>(p.out) +
                                            (size_t)s * p.q_len * p.n_q * D);
#pragma unroll 1
        for (int i = from * p.n_q * D / 8 + threadIdx.x; i < p.q_len * p.n_q * D / 8; i += 256)
          o[i] = make_uint4(0, 0, 0, 0);
      }
    Reader rd;
    Seg g;
    int t = 0, n_mine = 0, n_segs = 0;
    bool ok = true;
    while (ok && __all_sync(0xffffffffu, rd.next(B, p, g))) {
      __syncwarp();
      if (lane == 0) rd.done(B);
      const int nodes = tile_nodes(g, x);
      if (nodes == 0) continue;  // (never when split)
      const int seg = n_segs++;
      const int node = (SPLIT ? 0 : 2 * rg + x) * QT + ri;
      const bool valid = ri < nodes;  // (ri < QT: rows past QT G are not)
      const bool live = q4 * 32 < nodes * G;
      const size_t row = ((size_t)g.s * p.q_len + (valid ? node : 0)) * p.n_q + g.h * G + rh;
      uint64_t mask = valid ? __ldg(&p.masks[(size_t)g.s * p.q_len + node]) : 0ull;
      if (g.n < 64) mask &= (1ull << g.n) - 1ull;
      float sl = p.scale_log2;
      const int P = g.ctx - g.n;  // keys before the tree; may be negative
      float m = -INFINITY, l = 0.f;
      const int nt = g.t1 - g.t0;
      bool any = false;
      for (int ti = SPLIT ? x : 0; ti < nt; ti += SPLIT ? 2 : 1, ++t) {
        ok = wait_all(&B->s_full[x], t & 1, B, p);
        if (!ok) break;
        if (FP8 && !any)  // the row went in times 2^e
          sl *= exp2i(-reinterpret_cast<int8_t*>(
              smem + L::kExpOff)[((seg & 1) * L::kQ + (SPLIT ? 0 : x)) * 128 + r]);
        if (live) {  // rows without a node: nothing reads their P or O
          tc::fence_after();
          const int key = (g.t0 + ti) * kTileN;
          const bool full = key + kTileN <= P && p.scale_log2 > 0.f;
          uint32_t vis[4] = {};
          if (!full) {
#pragma unroll
            for (int w = 0; w < 4; ++w) vis[w] = seen_bits(key + 32 * w, P, mask);
          }
          float s[L::kLean ? 64 : kTileN];
          float mx, sle = L::kLean && !full ? 1.f : sl;
          if constexpr (L::kLean) {
            mx = attn::tile_max_halves(tS, full, vis, sl);
          } else {
            attn::load_scores(tS, s);
            if (L::kSepP) {
              tc::fence_before();
              mbar_arrive(&B->s_empty[x]);
            }
            mx = attn::tile_max(s, full, vis, sle);
          }
          const float mn = fmaxf(m, mx);
          const bool grow = mn > m + attn::kRescaleLog2;
          float alpha = 1.f;
          if (grow) {
            alpha = exp2f(m - mn);  // 0 on the row's first keys
            l *= alpha;
            m = mn;
          }
          // O += P V of the tile before is done where P lies over S: S of this
          // tile came after it
          if (any && __any_sync(0xffffffffu, grow)) {
            if (L::kSepP)
              ok = wait_all(&B->pv_done[x], (t - 1) & 1, B, p);
            if (!ok) break;
            tc::fence_after();
            attn::rescale_o(tO, D, alpha);
          }
          // a row that has seen no key yet: its weights are 0
          const float neg_m = m == -INFINITY ? 0.f : -m;
          uint32_t pk[32];
#pragma unroll(L::kLean ? 1 : 2)
          for (int h = 0; h < 2; ++h) {
            if constexpr (L::kLean) {
              attn::load_half(tS + 64 * h, full, h ? vis[2] : vis[0], h ? vis[3] : vis[1], sl, s);
              if (L::kSepP && h == 1) {
                tc::fence_before();
                mbar_arrive(&B->s_empty[x]);
              }
            }
            l += attn::tile_weights<kOpBf16, 64>(s + (L::kLean ? 0 : 64 * h), sle, neg_m, pk);
            if (L::kSepP && h == 0 && t > 0) {  // P of the tile before has been read
              ok = wait_all(&B->pv_done[x], (t - 1) & 1, B, p);
              if (!ok) break;
              tc::fence_after();
            }
            tc::st32x32b_x32(tP + 32 * h, pk);
            tc::wait_st();
            tc::fence_before();
            mbar_arrive(h ? &B->p_full[x] : &B->p_half[x]);
          }
          if (!ok) break;
        } else {
          if (L::kSepP) {
            mbar_arrive(&B->s_empty[x]);
            // not ahead of the other warps' P of the tile before
            if (t > 0)
              ok = wait_all(&B->pv_done[x], (t - 1) & 1, B, p);
            if (!ok) break;
          }
          mbar_arrive(&B->p_half[x]);
          mbar_arrive(&B->p_full[x]);
        }
        any = true;
      }
      if (!ok) break;
      // ------------------------------------------------ segment epilogue
      if (any) {
        ok = wait_all(&B->o_full[x], n_mine & 1, B, p);
        if (!ok) break;
        ++n_mine;
      }
      // the row's columns from c0 on (split: 64 of 128 for each tile's warps, the
      // only 64 for A's): w0 O_A + w1 O_B when split (the
      // other tile's (m, l) come through shared memory), else w0 O_X
      const int c0 = SPLIT && D == 128 ? x * 64 : 0;
      float w0 = 1.f, w1 = 0.f;
      if constexpr (SPLIT) {
        float2* red = reinterpret_cast<float2*>(smem + L::kRedOff) + r;
        // (the segment before was read out by both)
        if (seg > 0)
          ok = wait_all(&B->o_free[0], (seg - 1) & 1, B, p);
        if (!ok) break;
        red[x * 128] = make_float2(m, l);
        tc::fence_before();
        mbar_arrive(&B->red[x]);
        ok = wait_all(&B->red[x ^ 1], seg & 1, B, p);
        if (!ok) break;
        const float2 a = red[0], b = red[128];
        m = fmaxf(a.x, b.x);
        // (a sum that is not finite stays so)
        w0 = m == -INFINITY ? 0.f : exp2f(a.x - m);
        w1 = m == -INFINITY ? 0.f : exp2f(b.x - m);
        l = m == -INFINITY ? a.y + b.y : w0 * a.y + w1 * b.y;
      } else if (m == -INFINITY) {
        w0 = 0.f;
      }
      tc::fence_after();
      const size_t slot = g.slot < 0 ? 0
                                     : ((size_t)blockIdx.x * 2 + g.slot) * (SPLIT ? 128 : 256) +
                                           (SPLIT ? 0 : x * 128) + r;
      if (g.slot < 0) {
        const float inv = l == 0.f ? 0.f : p.out_mul / l;
        w0 *= inv;
        w1 *= inv;
      } else if (valid && (!SPLIT || x == 0)) {
        p.ws_ml[slot] = make_float2(m, l);
      }
      if (live && !(SPLIT && D == 64 && x == 1)) {
        // (B without a key tile: its O may hold anything, its weight is zero)
        const uint32_t ta = tmem + L::tO(SPLIT ? 0 : x) + lanes + c0,
                       tb = tmem + L::tO(nt > 1 ? 1 : 0) + lanes + c0;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 64) {
          if (SPLIT && D == 128 && cc > 0) break;  // 64 of 128 columns each
          if (g.slot < 0)
            attn::store_rows<T16, SPLIT, D>(ta + cc, tb + cc, static_cast<T16*>(p.out) + c0 + cc,
                                            valid ? (int)row : -1, w0, w1);
          else
            attn::store_rows<float, SPLIT, D>(ta + cc, tb + cc, p.ws_o + c0 + cc,
                                              valid ? (int)slot : -1, w0, w1);
        }
      }
      tc::fence_before();
      if constexpr (SPLIT) {
        mbar_arrive(&B->o_free[0]);
        mbar_arrive(&B->o_free[1]);
      } else {
        mbar_arrive(&B->o_free[x]);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc::dealloc(tmem, kTmemCols);
  }
}

// Combines the segments of the units split between shares.  CTA (c, y) looks
// at the boundary between shares c and c + 1: if it cuts a unit whose first
// step lies in share c, this CTA merges kMergeRows of the unit's rows, a warp a
// row, from the shares' slots in order.  Every other row was written whole.
template <typename OutT, int D, bool SPLIT>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeParams p, int ctas) {
  __shared__ int sh_s, sh_h, sh_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  // finding the unit reads only the lengths, so it overlaps the attention
  // kernel (this grid is its programmatic dependent); pdl_wait comes before
  // the workspace is read
  if (warp == 0) {
    int s = -1, h = 0, last = c;
    int first;
    const Shares sh(total_weight(p, lane, false, first), ctas);
    if (c + 1 < sh.C) {
      const long long X = sh.start(c + 1);
      int s0, w;
      long long gs;
      if (locate(p, X, lane, first, s0, gs, w)) {
        h = quotient(X - gs, w);
        const long long u = gs + (long long)h * w + p.seg_cost, end = u + w - p.seg_cost;
        if (u < X && u >= sh.start(c)) {
          s = s0;
          // the last share with steps of the unit
#pragma unroll 1
          for (int k = c + 1 + lane;; k += 32) {
            const uint32_t in = __ballot_sync(0xffffffffu, k < sh.C && sh.start(k) < end);
            last += __popc(in);
            if (in != 0xffffffffu) break;
          }
        }
      }
    }
    if (lane == 0) {
      sh_s = s;
      sh_h = h;
      sh_last = last;
    }
  }
  __syncthreads();
  pdl_wait();  // the attention kernel's results
  if (sh_s < 0) return;
  const int G = p.group, QT = kTileM / G, n = seq_nodes(p, sh_s), last = sh_last;
  constexpr int RW = SPLIT ? 128 : 256, V = D / 32;  // rows of a slot, floats a lane
  constexpr bool kBf = std::is_same<OutT, __nv_bfloat16>::value;
#pragma unroll 1
  for (int k = warp; k < kMergeRows; k += kMergeWarps) {
    const int row = blockIdx.y * kMergeRows + k;  // of the CTAs side by side: RW each
    const int rg = row / RW, in = row % RW, r = in % kTileM;
    const int node = (row / kTileM) * QT + r / G;
    if (r / G >= QT || node >= n) continue;
    auto slot = [&](int cc) -> size_t {
      return ((size_t)(cc * p.row_groups + rg) * 2 + (cc == c ? 1 : 0)) * RW + in;
    };
    auto load_piece = [&](int cc, float (&y)[V]) {
      const float* o = p.ws_o + slot(cc) * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = o[e];
    };
    constexpr int kPre = 4;
    float M = -INFINITY, Ls = 0.f, acc[V] = {};
#pragma unroll 1
    for (int c0 = c; c0 <= last; c0 += 32) {  // 32 pieces at a time, a lane each
      const int nc = min(32, last - c0 + 1);
      // the first pieces' rows come with the weights, not after them
      float pre[kPre][V];
#pragma unroll
      for (int i = 0; i < kPre; ++i)
        if (i < nc) load_piece(c0 + i, pre[i]);
      const float2 v = lane < nc ? p.ws_ml[slot(c0 + lane)] : make_float2(-INFINITY, 0.f);
      const float mn = fmaxf(M, warp_max_xor(v.x, 1));
      if (mn == -INFINITY) {  // nothing seen, unless a sum is not a number
        if (__any_sync(0xffffffffu, v.y != 0.f)) Ls = NAN;
        continue;
      }
      const float old = exp2f(M - mn), w = exp2f(v.x - mn);
      M = mn;
      Ls *= old;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= old;
      auto add = [&](int i, const float (&y)[V]) {
        const float wi = __shfl_sync(0xffffffffu, w, i), li = __shfl_sync(0xffffffffu, v.y, i);
        Ls += wi * li;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += wi == 0.f ? 0.f : wi * y[e];
      };
#pragma unroll
      for (int i = 0; i < kPre; ++i)
        if (i < nc) add(i, pre[i]);
#pragma unroll 1
      for (int i = kPre; i < nc; ++i) {
        float y[V];
        load_piece(c0 + i, y);
        add(i, y);
      }
    }
    const float inv = Ls == 0.f ? 0.f : p.out_mul / Ls;
    uint32_t* out = reinterpret_cast<uint32_t*>(
        static_cast<OutT*>(p.out) +
        (((size_t)sh_s * p.q_len + node) * p.n_q + sh_h * G + r % G) * D + lane * V);
#pragma unroll
    for (int e = 0; e < V; e += 2) out[e / 2] = pack2<kBf>(acc[e] * inv, acc[e + 1] * inv);
  }
}

template <bool BF16, int D, bool FP8, bool SPLIT>
cudaError_t launch_t(const TreeParams& p, const CUtensorMap* tmq, const CUtensorMap* tmk,
                     const CUtensorMap* tmv, cudaStream_t st) {
  using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using L = Lay<D, FP8, SPLIT>;
  static std::atomic<unsigned long long> set{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(tree_kernel<BF16, D, FP8, SPLIT>),
                             L::kSmem, set);
  if (e != cudaSuccess) return e;
  int shares = device_sms() < kTreeCtas ? device_sms() : kTreeCtas;
  shares /= p.row_groups;
  tree_kernel<BF16, D, FP8, SPLIT>
      <<<shares * p.row_groups, L::kThreads, L::kSmem, st>>>(p, *tmq, *tmk, *tmv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)shares, (SPLIT ? 128 : 256) / kMergeRows * p.row_groups);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<T16, D, SPLIT>, p, shares);
}

template <bool BF16, int D>
cudaError_t launch_d(const TreeParams& p, bool fp8, const CUtensorMap* tmq, const CUtensorMap* tmk,
                     const CUtensorMap* tmv, cudaStream_t st) {
  const bool split = p.step_keys == 2 * kTileN;
  if (fp8)
    return split ? launch_t<BF16, D, true, true>(p, tmq, tmk, tmv, st)
                 : launch_t<BF16, D, true, false>(p, tmq, tmk, tmv, st);
  return split ? launch_t<BF16, D, false, true>(p, tmq, tmk, tmv, st)
               : launch_t<BF16, D, false, false>(p, tmq, tmk, tmv, st);
}

}  // namespace

size_t tree_ws_bytes(int q_len, int group, int D) {
  const int tiles = (q_len + kTileM / group - 1) / (kTileM / group);
  const size_t rows = (size_t)kTreeCtas * 2 * (tiles == 1 ? 128 : 256);
  return rows * D * sizeof(float) + rows * sizeof(float2);
}

cudaError_t launch_tree(TreeParams& p, int D, bool bf16, bool fp8, void* workspace,
                        const CUtensorMap* tmq, const CUtensorMap* tmk, const CUtensorMap* tmv,
                        cudaStream_t st) {
  if (p.num_seqs == 0) return cudaSuccess;
  // The most nodes of the batch choose the kernel: one tile, or two for all (and a
  // second CTA beside, since TMEM holds two), so that small trees beside a large one
  // leave B idle.  64 contexts of up to 8,000, 64/8 heads of 128, bf16, trees of 4 to
  // 16 nodes: 145 us with q_len 16, 174 with 17, 323 with 40; three of them with 40
  // nodes 368.
  const int qt = kTileM / p.group, tiles = (p.q_len + qt - 1) / qt;
  p.row_groups = tiles > 2 ? 2 : 1;
  p.step_keys = tiles == 1 ? 2 * kTileN : kTileN;
  p.log2_step = tiles == 1 ? 8 : 7;
  // measured, against the time of a step: 1.6 (16-bit, 128 wide), 1.0 (64
  // wide), 1.5 (E4M3), 1.5 (a step of one tile)
  p.seg_cost = tiles == 1 && !fp8 && D == 64 ? 1 : 2;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = reinterpret_cast<float2*>(p.ws_o + (size_t)kTreeCtas * 2 * (tiles == 1 ? 128 : 256) * D);
  if (D == 128)
    return bf16 ? launch_d<true, 128>(p, fp8, tmq, tmk, tmv, st)
                : launch_d<false, 128>(p, fp8, tmq, tmk, tmv, st);
  return bf16 ? launch_d<true, 64>(p, fp8, tmq, tmk, tmv, st)
              : launch_d<false, 64>(p, fp8, tmq, tmk, tmv, st);
}

}  // namespace pa
