// Whole-prompt attention (pa_prefill_packed) on tcgen05 tensor cores.
//
// out[r][h] = sum over keys u <= r of r's sequence of 2^(s_u - m) v_u / l, with
// s = scale log2(e) q . k, m the row's maximum and l the sum of the weights:
// one pass over the keys with the running (m, l) of attn_tile.cuh.
//
// Tiles.  A 128-row tile is HB query heads of one kv head (HB: the power of
// two in the group size, at most 16) times QT = 128 / HB consecutive queries,
// row r = query r / HB, head r % HB; so each K/V tile of 128 keys serves HB
// heads and every group size fills its tiles.  An item of work is two such
// tiles, A and B, one behind the other in the sequence, over the same keys: the
// tensor cores work on one while the softmax of the other runs.  TMEM holds S
// of A and B (128 fp32 columns each; P goes over S as 16-bit pairs) and O of
// A and B.
//
// Persistent CTAs, one per SM.  The items are ordered by their position in
// their sequence, the last ones (which see the most keys) first, over all
// sequences together, so the CTAs, which take them in turn there and back,
// end at about the same time: a scheduler warp walks that order from the
// sequence starts alone (no list in memory, no order of arrival), ahead of the
// other warps.
//
// Roles: warps 0-3 softmax of tile A, warps 4-7 of tile B (one thread per
// row, its 128 scores in registers), warps 8 and 9 issue the MMAs of A and B,
// warp 10 loads Q, K and V by TMA (K and V share a ring of stages), warp 11
// schedules, warp 12 zeroes the rows of an item's last V tile that lie behind
// its sequence (another sequence's values or padding: 0 x NaN must not reach
// O).  Every wait is bounded; a role that gives up flags PA_DEVERR_TIMEOUT and
// leaves, and the CTA drains its loads and MMAs and frees TMEM.
//
// Measured back to back in a CUDA graph (and sustained over seconds, where 128-
// wide heads run into the power limit): 16,384 tokens of 32/8 heads of 128, bf16,
// 1.73 ms = 1,273 TFLOP/s of causal products (2.04 ms); 16 prompts of up to 2,100
// tokens, 64/8 x 128, 311 us = 947 TFLOP/s (370 us); 8 of up to 1,500, 32/8 x 64,
// 51.4 us; one of 37 tokens 8.0 us, of 1 token 6.5 us.  A tile takes 1,820 clocks
// on the first (time x SM clock over a CTA's 1,785 tiles) and 2,030 active ones on
// the second, whose CTAs come to the end of an item 24 times, against 1,024 of
// either its products or its exponentials (tensor pipe and XU at 47 %).  128-wide
// heads: the chain P -> O += P V -> next S -> softmax, since P lies over S for want
// of TMEM.  64-wide heads (P beside S) and short prompts: the ends of items, where
// the softmax warps write O before they begin the next one (2,600 clocks a tile on
// the third, 4.7 items a CTA).
#include <type_traits>

#include "attn_tile.cuh"
#include "serve_ops.h"

namespace pa {

namespace {

using attn::kTileM;
using attn::kTileN;

constexpr int kThreads = 512;
constexpr int kMmaWarp = 8, kLoadWarp = 10, kSchedWarp = 11, kFixWarp = 12;  // 13-15 idle
constexpr int kItems = 4;              // items scheduled ahead
constexpr uint32_t kItemReaders = 12;  // 8 softmax warps, 2 MMA, loads, fixer
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 10;

template <int D>
struct Lay {
  static constexpr int kOp = kTileN * D * 2;       // one Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQOff = 0, kKVOff = 2 * kOp;
  static constexpr int kBarOff = kKVOff + kStages * kOp;
  static constexpr int kSmem = kBarOff + 1024 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  // TMEM columns: S_A 0, S_B 128; a 64-wide head leaves room for P beside S, so
  // that S of the next tile is made while the softmax works on this one
  static constexpr bool kSepP = D == 64;
  static constexpr int tP(int x) { return kSepP ? 256 + 64 * x : 128 * x; }
  static constexpr int tO(int x) { return kSepP ? 384 + 64 * x : 256 + 128 * x; }
  static_assert(kStages <= kMaxStages, "stage barriers");
};

struct Item {
  int start;   // first row of the sequence; < 0: no more items
  int len;     // its tokens
  int i0;      // first query of tile A; B follows QT later
  int h0;      // first q head
  int nkt[2];  // key tiles of A and B (B: 0 when the sequence ends before it)
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t raw[kMaxStages];  // a V tile whose tail warp 12 has yet to zero
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], o_free[2];
  uint64_t s_empty[2], pv_done[2];  // P beside S only
  uint64_t done[2], turn[2];
  Item items[kItems];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 1024, "barriers");

using attn::wait_all;
using attn::wait_ok;

// The item stream as one role reads it.
struct Reader {
  int k = 0;
  __device__ __forceinline__ bool next(Bars* B, const PromptParams& p, Item& it) {
    const int slot = k % kItems;
    if (!wait_ok(&B->item_full[slot], (k / kItems) & 1, B, p)) return false;
    it = B->items[slot];
    ++k;
    return it.start >= 0;
  }
  // the item is copied: its slot may be filled again (one arrival per reader)
  __device__ __forceinline__ void done(Bars* B) { mbar_arrive(&B->item_empty[(k - 1) % kItems]); }
};

// The length of sequence s (0 behind the last one) and its first row, where the
// starts are in order and within the tensors.
__device__ __forceinline__ int span_of(const PromptParams& p, int s, int& start) {
  if (s >= p.num_seqs) return 0;
  start = __ldg(&p.query_start_loc[s]);
  return (int)((uint32_t)__ldg(&p.query_start_loc[s + 1]) - (uint32_t)start);
}
// The same of other starts, for the 32 sequences of a warp (s = that of this
// lane): each start counts as the largest of 0 and the ones up to it, at most
// `total`, so that no row belongs to two sequences and the items are no more than
// starts in order have.  `before`: the largest up to these sequences, 0 at first.
__device__ __forceinline__ int span_in_order(const PromptParams& p, int s, int lane, int& before,
                                             int& start) {
  int a = 0, b = 0;
  if (s < p.num_seqs) {
    a = min(max(__ldg(&p.query_start_loc[s]), 0), p.total);
    b = min(max(__ldg(&p.query_start_loc[s + 1]), 0), p.total);
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, a, m);
    if (lane >= m) a = max(a, v);
  }
  start = max(a, before);
  b = max(b, start);  // the next sequence's start
  before = __shfl_sync(0xffffffffu, b, 31);
  return b - start;
}

// Of the last key tile of item tile X: how many of its four 32-key parts some
// row sees.
__device__ __forceinline__ int last_parts(const Item& it, int x, int QT) {
  const int keys = min(it.len, it.i0 + (x + 1) * QT);
  return (((keys - 1) & (kTileN - 1)) >> 5) + 1;
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const PromptParams p, const __grid_constant__ CUtensorMap tmq,
                  const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using L = Lay<D>;
  constexpr int NS = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* B = reinterpret_cast<Bars*>(smem + L::kBarOff);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lhb = p.log2_hb, QT = kTileM >> lhb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&B->full[s], 1);
      mbar_init(&B->empty[s], 2);
      mbar_init(&B->raw[s], 1);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(&B->item_full[s], 1);
      mbar_init(&B->item_empty[s], kItemReaders);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&B->done[x], 1);
      mbar_init(&B->turn[x], 1);
      mbar_init(&B->q_full[x], 1);
      mbar_init(&B->q_empty[x], 1);
      mbar_init(&B->s_full[x], 1);
      mbar_init(&B->p_half[x], 128);
      mbar_init(&B->p_full[x], 128);
      mbar_init(&B->s_empty[x], 128);
      mbar_init(&B->pv_done[x], 1);
      mbar_init(&B->o_full[x], 1);
      mbar_init(&B->o_free[x], 128);
    }
    B->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::alloc(&B->tmem_base, kTmemCols);
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = B->tmem_base;

  // 512 threads at 128 registers: 65,536 = 256 x 192 + 256 x 64
  if (warp >= kMmaWarp) {
  tc::regs_dec<64>();
  if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ------------------------------------------------------------ MMA issuers
    // one warp per tile X: per key tile j, O_X += P_X V of tile j - 1 and S_X =
    // Q_X K^T of tile j (in this order where P lies over S: the tensor core
    // keeps it; else S first).  The whole warp walks the tiles and waits, one
    // lane issues.  The waits of one warp run while the other's MMAs do; they
    // take turns, so that one's batch is not spread over the other's and the
    // softmax passes of A and B fall into opposite phases.
    constexpr uint32_t idesc_s = tc::idesc_f16(BF16, false, kTileM, 0);  // N by tile
    constexpr uint32_t idesc_pv = tc::idesc_f16(BF16, true, kTileM, D);
    constexpr uint64_t kOpStep = L::kOp >> 4;  // descriptors count 16 bytes
    constexpr bool kTurns = !L::kSepP;
    const int x = warp - kMmaWarp;
    const uint64_t dQ = tc::smem_desc(sbase + L::kQOff + x * L::kOp),
                   dK = tc::smem_desc(sbase + L::kKVOff),
                   dV = tc::smem_desc(sbase + L::kKVOff, 16384);
    const uint32_t tS = tmem + x * 128, tP = tmem + L::tP(x), tO = tmem + L::tO(x);
    Reader rd;
    Item it;
    bool ok = true, issued = false;
    uint32_t c = 0;  // stages used before this tile: K of tile j in c, V in c + 1
    uint32_t items = 0, tiles = 0, turns = 0;
    auto scores = [&](uint64_t k, bool last, int parts) {
      tc::fence_after();
      if (tc::elect_one()) {
        const uint32_t idesc = idesc_s | (uint32_t)(parts * 4) << 17;  // N = 32 parts
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (kk >> 2) * 1024 + (kk & 3) * 2;
          tc::mma(tS, dQ + off, k + off, idesc, kk > 0);
        }
        tc::commit(&B->s_full[x]);
        if (last) tc::commit(&B->q_empty[x]);
      }
      __syncwarp();
    };
    while (ok && __all_sync(0xffffffffu, rd.next(B, p, it))) {
      if (lane == 0) rd.done(B);
      __syncwarp();
      const int n = max(it.nkt[0], it.nkt[1]), mine = x ? it.nkt[1] : it.nkt[0];
      const int ends = last_parts(it, x, QT);  // of the last key tile
      if (mine > 0) ok = wait_all(&B->q_full[x], items & 1, B, p);
      for (int j = 0; j <= n && ok; ++j, c += 2) {
        const uint32_t cv = c - 1;
        const int sk = c % NS, sv = cv % NS;
        const bool do_pv = j > 0 && j <= mine, do_s = j < mine;
        const uint64_t v = dV + sv * kOpStep, k = dK + sk * kOpStep;
        const uint32_t par = (tiles - 1) & 1;
        if (j > 0) ok = wait_all(&B->full[sv], (cv / NS) & 1, B, p);
        if (j < n) ok = ok && wait_all(&B->full[sk], (c / NS) & 1, B, p);
        if (L::kSepP && do_s) {  // S beside P: as soon as the softmax has read the last S
          if (tiles > 0) ok = ok && wait_all(&B->s_empty[x], (tiles - 1) & 1, B, p);
          if (!ok) break;
          scores(k, j == mine - 1, j == mine - 1 ? ends : 4);
        }
        if (do_pv) {
          if (j == 1 && items > 0)
            ok = ok && wait_all(&B->o_free[x], (items - 1) & 1, B, p);
          ok = ok && wait_all(&B->p_half[x], par, B, p);
        }
        // (an item's first S goes ahead out of turn)
        if (kTurns && j > 0) {
          if (x > 0 || turns > 0)
            ok = ok && wait_all(&B->turn[x], (turns - 1 + x) & 1, B, p);
          ++turns;
        }
        if (!ok) break;
        if (do_pv) {
          const int nk = j == mine ? 2 * ends : 8;  // 16 keys a step = two 8-row groups of V
          tc::fence_after();
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < nk)
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
              if (kk < nk) tc::mma_ts(tO, tP + kk * 8, v + kk * 128, idesc_pv, 1u);
            if (L::kSepP) tc::commit(&B->pv_done[x]);
            if (j == mine) tc::commit(&B->o_full[x]);
          }
          __syncwarp();
        }
        if (!L::kSepP && do_s) scores(k, j == mine - 1, j == mine - 1 ? ends : 4);
        if (tc::elect_one()) {
          if (kTurns && j > 0) mbar_arrive(&B->turn[x ^ 1]);
          // a stage is free once both warps' MMAs on it are done
          if (j > 0) tc::commit(&B->empty[sv]);
          if (j < n) tc::commit(&B->empty[sk]);
        }
        __syncwarp();
        issued = true;
        tiles += do_s;
      }
      c -= 2;  // the last step had no K
      items += mine > 0;
    }
    // everything issued above has completed before TMEM is released
    if (issued) {
      if (tc::elect_one()) tc::commit(&B->done[x]);
      __syncwarp();
      mbar_wait(&B->done[x], 0, p.waits.wait_ns);
    }
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      Reader rd;
      Item it{};
      bool ok = true;
      uint32_t c = 0;
      int nq0 = 0, nq1 = 0;  // Q tiles of A and B
      auto tile = [&](const CUtensorMap* map, int kvh, int row, bool tail) {
        const int st = c % NS;
        if (c >= (uint32_t)NS && !wait_ok(&B->empty[st], ((c / NS) - 1) & 1, B, p))
          return false;
        if (c == (uint32_t)p.waits.skip_tile) {
          ++c;
          return true;
        }
        uint8_t* d = smem + L::kKVOff + st * L::kOp;
        // the arrival of a V tile with a tail to zero is warp 12's
        uint64_t* bar = tail ? &B->raw[st] : &B->full[st];
        mbar_arrive_expect_tx(bar, L::kOp);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tc::tma_load_3d(d + h * 16384, map, bar, 64 * h, kvh, row);
        ++c;
        return true;
      };
      auto query = [&](int x) {
        if (!ok || (x ? it.nkt[1] : it.nkt[0]) == 0) return;
        int& used = x ? nq1 : nq0;
        if (used > 0) ok = wait_ok(&B->q_empty[x], (used - 1) & 1, B, p);
        if (!ok) return;
        ++used;
        uint8_t* d = smem + L::kQOff + x * L::kOp;
        mbar_arrive_expect_tx(&B->q_full[x], L::kOp);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tc::tma_load_3d(d + h * 16384, &tmq, &B->q_full[x], 64 * h, it.h0,
                          it.start + it.i0 + x * QT);
      };
      while (ok && rd.next(B, p, it)) {
        rd.done(B);
        const int n = max(it.nkt[0], it.nkt[1]), kvh = it.h0 / p.group;
        for (int j = 0; j < n && ok; ++j) {
          // Q of A is free to load long before a stage is, Q of B a little after
          if (j == 0) query(0);
          ok = ok && tile(&tmk, kvh, it.start + j * kTileN, false);
          if (j == 0) query(1);
          ok = ok && tile(&tmv, kvh, it.start + j * kTileN, (j + 1) * kTileN > it.len);
        }
      }
      // loads in flight land before the CTA exits
      for (uint32_t u = c > (uint32_t)NS ? c - NS : 0; u < c; ++u)
        mbar_wait(&B->full[u % NS], (u / NS) & 1, p.waits.wait_ns);
      if (nq0 > 0) mbar_wait(&B->q_full[0], (nq0 - 1) & 1, p.waits.wait_ns);
      if (nq1 > 0) mbar_wait(&B->q_full[1], (nq1 - 1) & 1, p.waits.wait_ns);
    }
  } else if (warp == kSchedWarp) {
    // ------------------------------------------------------------ scheduler
    // level = position of an item in its sequence, in items; the levels are
    // walked downwards, within a level the sequences that reach it in order,
    // and the head groups of each.  Only the first 32 sequences are kept, the others
    // are looked through again for every item: 32/8 heads of 128, prompts of 16 to
    // 64 tokens, 0.23 us a prompt for 256 of them, 0.30 for 1,024, 1.0 for 4,096
    const unsigned hgroups = p.n_q >> lhb;
    const int lspan = 8 - lhb, span = 1 << lspan;  // queries of an item
    auto items_of = [&](int len) { return (len + span - 1) >> lspan; };
    // the first 32 sequences, kept
    int start0 = 0, len0 = span_of(p, lane, start0), before0 = 0;
    int top = 0;
    bool ordered = true;
    auto look = [&](int a, int n) {
      // (a negative end gives n < 0 or, wrapped, a + n >= 2^31)
      if (a < 0 || n < 0 || n > p.total - a)
        ordered = false;
      else
        top = max(top, items_of(n));
    };
    look(start0, len0);
#pragma unroll 1
    for (int s = 32 + lane; s < p.num_seqs; s += 32) {
      int a;
      const int n = span_of(p, s, a);
      look(a, n);
    }
    ordered = __all_sync(0xffffffffu, ordered);
    if (!ordered) {
      if (blockIdx.x == 0 && lane == 0) flag_error(p.dev_err, PA_DEVERR_QUERY_LOC);
      top = 0;
      int start, before = 0;
#pragma unroll 1
      for (int s0 = 0; s0 < p.num_seqs; s0 += 32)
        top = max(top, items_of(span_in_order(p, s0 + lane, lane, before, start)));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (!ordered) len0 = span_in_order(p, lane, lane, before0, start0);
    int level = top, cnt = 0;
    unsigned base = 0;  // (sequence, level) pairs before this level
    bool more = true;
    for (int k = 0; more; ++k) {
      // there and back: the CTA that got the longest item of one round gets
      // the shortest of the next
      const unsigned idx =
          (unsigned)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      const unsigned want = idx / hgroups;
      while (more && want >= base + cnt) {
        base += cnt;
        --level;
        cnt = 0;
        if (level < 0) {
          more = false;
        } else {
          int n = items_of(len0) > level, start, before = before0;
#pragma unroll 1
          for (int s0 = 32; s0 < p.num_seqs; s0 += 32)
            n += items_of(ordered ? span_of(p, s0 + lane, start)
                                  : span_in_order(p, s0 + lane, lane, before, start)) > level;
          cnt = __reduce_add_sync(0xffffffffu, n);
        }
      }
      Item it;
      it.start = -1;
      it.len = 0;
      if (more) {
        int r = (int)(want - base), start = start0, len = len0, before = before0;
#pragma unroll 1
        for (int s0 = 0;;) {
          const bool has = items_of(len) > level;
          const uint32_t m = __ballot_sync(0xffffffffu, has);
          const uint32_t hit = __ballot_sync(
              0xffffffffu, has && __popc(m & ((1u << lane) - 1u)) == r);
          if (hit) {
            it.start = __shfl_sync(0xffffffffu, start, __ffs(hit) - 1);
            it.len = __shfl_sync(0xffffffffu, len, __ffs(hit) - 1);
            break;
          }
          r -= __popc(m);
          s0 += 32;
          if (s0 >= p.num_seqs) break;  // (the level's items were counted: not reached)
          len = ordered ? span_of(p, s0 + lane, start)
                        : span_in_order(p, s0 + lane, lane, before, start);
        }
        more = it.start >= 0;
        // of an odd number of tiles the first, which sees the fewest keys, is
        // alone in its item
        const bool odd = ((it.len + QT - 1) >> (lspan - 1)) & 1;
        it.i0 = max(0, level * span - (odd ? QT : 0));
        it.h0 = (int)(idx - want * hgroups) << lhb;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = it.i0 + x * QT;
          it.nkt[x] = i < it.len && !(x == 1 && odd && level == 0)
                          ? (min(it.len, i + QT) + kTileN - 1) / kTileN
                          : 0;
        }
      }
      const int slot = k % kItems;
      bool ok = k < kItems || wait_ok(&B->item_empty[slot], (k / kItems - 1) & 1, B, p);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        B->items[slot] = it;
        mbar_arrive(&B->item_full[slot]);
      }
      __syncwarp();
    }
  } else if (warp == kFixWarp) {
    // ------------------------------------------------- rows behind a sequence
    Reader rd;
    Item it;
    uint32_t c = 0, phase = 0;  // stages used; per stage, the parity of its next tail
    while (__all_sync(0xffffffffu, rd.next(B, p, it))) {
      __syncwarp();
      if (lane == 0) rd.done(B);
      const int n = max(it.nkt[0], it.nkt[1]);
      c += 2 * n;
      const int valid = it.len - (n - 1) * kTileN;  // rows of the last tile
      if (valid >= kTileN) continue;
      const int st = (c - 1) % NS;
      if (!wait_all(&B->raw[st], (phase >> st) & 1, B, p)) break;
      phase ^= 1u << st;
      uint8_t* d = smem + L::kKVOff + st * L::kOp;
      // 128-byte rows; the swizzle stays within a row
      for (int u = valid * 8 + lane; u < kTileN * 8; u += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          *reinterpret_cast<uint4*>(d + h * 16384 + u * 16) = make_uint4(0, 0, 0, 0);
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->full[st]);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax
    tc::regs_inc<192>();
    const int x = warp >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row = TMEM lane
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lanes, tP = tmem + L::tP(x) + lanes,
                   tO = tmem + L::tO(x) + lanes;
    const float sl = p.scale_log2;
    Reader rd;
    Item it;
    int t = 0, n_mine = 0;
    bool ok = true;
    while (ok && __all_sync(0xffffffffu, rd.next(B, p, it))) {
      __syncwarp();
      if (lane == 0) rd.done(B);
      const int nkt = x ? it.nkt[1] : it.nkt[0];
      if (nkt == 0) continue;
      const int qw = it.i0 + x * QT + ((q4 * 32) >> lhb);  // the warp's first query
      const int qi = it.i0 + x * QT + (r >> lhb);          // this row's
      const bool live = qw < it.len;
      attn::RowState st{-INFINITY, 0.f};
      for (int j = 0; j < nkt; ++j, ++t) {
        ok = wait_all(&B->s_full[x], t & 1, B, p);
        if (!ok) break;
        if (live) {  // rows behind the sequence: nothing reads their P or O
          tc::fence_after();
          const bool full = j * kTileN + kTileN - 1 <= qw && sl > 0.f;
          uint32_t vis[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) vis[w] = attn::bits_upto(j * kTileN + 32 * w, qi);
          float s[kTileN];
          attn::load_scores(tS, s);
          if (L::kSepP) {
            tc::fence_before();
            mbar_arrive(&B->s_empty[x]);
          }
          float sle = sl;
          const float mx = attn::tile_max(s, full, vis, sle);
          const float mn = fmaxf(st.m, mx);
          const bool grow = mn > st.m + attn::kRescaleLog2;
          float alpha = 1.f;
          if (grow) {
            alpha = exp2f(st.m - mn);  // 0 on the first tile
            st.l *= alpha;
            st.m = mn;
          }
          // O += P V of the tile before is done where P lies over S: S of this
          // tile came after it
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            if (L::kSepP)
              ok = wait_all(&B->pv_done[x], (t - 1) & 1, B, p);
            if (!ok) break;
            tc::fence_after();
            attn::rescale_o(tO, D, alpha);
          }
          const float neg_m = st.m == -INFINITY ? 0.f : -st.m;
          uint32_t pk[16];
          const int parts = j == nkt - 1 ? last_parts(it, x, QT) : 4;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c < parts) {  // no row of the tile sees the rest
              st.l += attn::tile_weights<BF16, 32>(s + 32 * c, sle, neg_m, pk);
              if (L::kSepP && c == 0 && t > 0) {  // P of the tile before has been read
                ok = wait_all(&B->pv_done[x], (t - 1) & 1, B, p);
                if (!ok) break;
                tc::fence_after();
              }
              tc::st32x32b_x16(tP + 16 * c, pk);
            }
            if (c & 1) {
              tc::wait_st();
              tc::fence_before();
              mbar_arrive(c == 1 ? &B->p_half[x] : &B->p_full[x]);
            }
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
      }
      if (!ok) break;
      ok = wait_all(&B->o_full[x], n_mine & 1, B, p);
      if (!ok) break;
      ++n_mine;
      const bool valid = qi < it.len;
      const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
      const int row = valid ? (it.start + qi) * p.n_q + it.h0 + (r & ((1 << lhb) - 1)) : -1;
      tc::fence_after();
      if (live) {
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 64)
          attn::store_rows<T16, false, D>(tO + cc, 0, static_cast<T16*>(p.out) + cc, row, inv, 0.f);
        tc::fence_before();
      }
      mbar_arrive(&B->o_free[x]);
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

template <bool BF16, int D>
cudaError_t launch_t(const PromptParams& p, const CUtensorMap* tmq, const CUtensorMap* tmk,
                     const CUtensorMap* tmv, cudaStream_t st) {
  static std::atomic<unsigned long long> set{0};
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(prompt_kernel<BF16, D>), Lay<D>::kSmem, set);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be items
  const int span = 2 * (kTileM >> p.log2_hb);
  const long long most = ((long long)p.total / span + p.num_seqs) * (p.n_q >> p.log2_hb);
  const int sms = device_sms();
  prompt_kernel<BF16, D><<<(unsigned)(most < sms ? most : sms), kThreads, Lay<D>::kSmem, st>>>(
      p, *tmq, *tmk, *tmv);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, int D, bool bf16, const CUtensorMap* tmq,
                          const CUtensorMap* tmk, const CUtensorMap* tmv, cudaStream_t st) {
  if (p.total == 0 || p.num_seqs == 0) return cudaSuccess;
  if (D == 128)
    return bf16 ? launch_t<true, 128>(p, tmq, tmk, tmv, st)
                : launch_t<false, 128>(p, tmq, tmk, tmv, st);
  return bf16 ? launch_t<true, 64>(p, tmq, tmk, tmv, st)
              : launch_t<false, 64>(p, tmq, tmk, tmv, st);
}

}  // namespace pa
