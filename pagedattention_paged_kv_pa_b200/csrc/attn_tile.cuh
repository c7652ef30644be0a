// The softmax of one row of a 128-row attention tile by one thread: scores
// come from TMEM (S = Q K^T, fp32), the weights go back over them as 16-bit
// pairs, the A operand of O += P V.
//
// With the scores in log2 units (s = scale log2(e) q . k) the thread keeps the
// maximum m it has exponentiated against and the sum l of 2^(s - m); O in TMEM
// holds the sum of 2^(s - m) v.  When the row's maximum grows by more than
// kRescaleLog2, l and O are multiplied by 2^(m - m') and m becomes m'; up to
// there the weights may exceed 1 by that factor, which fp32 sums and 16-bit
// weights (f16 up to 65504) hold.
//
// What bounds it is the exponential: 16 a clock and SM on the special-function
// unit, i.e. 1024 clocks for a 128 x 128 tile, as long as the two products of
// a 128-wide head take on the tensor cores.  (A quarter or a half of them as
// polynomials on the FMA pipe measured the same or slower: a warp's issue and
// latencies, not the unit, then set the pace.  Two threads a row, 16 softmax
// warps, measured 2.61 ms against 1.96 ms on a 16,384-token prompt.)
#pragma once

#include <type_traits>

#include "tile_ops.cuh"

namespace pa {
namespace attn {

constexpr int kTileM = 128;           // rows of a tile: one per TMEM lane
constexpr int kTileN = 128;           // keys per tile
constexpr float kRescaleLog2 = 8.f;   // lazy rescale threshold (factor 256)

// ------------------------------------------------------------------- waits
// A bounded wait in few instructions (the kernels have dozens of them, and
// their code would otherwise outgrow the instruction caches): it gives up after
// p.waits.wait_ns (at most a second, below 2^31: the timer's low word wraps), or
// when another role of the CTA has given up.  Giving up flags PA_DEVERR_TIMEOUT.
__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}

template <typename Bars, typename Params>
__device__ __forceinline__ bool wait_ok(uint64_t* bar, uint32_t parity, Bars* B,
                                        const Params& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = timer_lo();
#pragma unroll 1
  do {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&B->abort_flag)) return false;
  } while (timer_lo() - t0 < p.waits.wait_ns);
  flag_error(p.dev_err, PA_DEVERR_TIMEOUT);
  *reinterpret_cast<volatile int*>(&B->abort_flag) = 1;
  return false;
}
// the same for a whole warp, which goes on or gives up together
template <typename Bars, typename Params>
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, Bars* B,
                                         const Params& p) {
  return __all_sync(0xffffffffu, wait_ok(bar, parity, B, p));
}

// ------------------------------------------------- two fp32 values at a time
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void un2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

struct RowState {
  float m, l;  // maximum exponentiated against (log2 units), sum of the weights
};

// bits of keys first .. first + 31 that are at or below the last visible key
__device__ __forceinline__ uint32_t bits_upto(int first, int last) {
  const int n = last - first + 1;
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// The row's scores of a tile: 128 columns of S at `ts` (this warp's lanes).
__device__ __forceinline__ void load_scores(uint32_t ts, float (&x)[kTileN]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
#pragma unroll
  for (int c = 0; c < kTileN; c += 32) tc::ld32x32b_x32(ts + c, r + c);
  tc::wait_ld();
}

// Largest score of the row in log2 units; with a mask (full false) x becomes
// the scores in log2 units, -inf where vis has no bit, and sl 1.
__device__ __forceinline__ float tile_max(float (&x)[kTileN], bool full, const uint32_t (&vis)[4],
                                          float& sl) {
  if (!full) {
#pragma unroll
    for (int e = 0; e < kTileN; ++e) x[e] = (vis[e >> 5] >> (e & 31)) & 1u ? x[e] * sl : -INFINITY;
    sl = 1.f;
  }
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < kTileN; e += 8)
#pragma unroll
    for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], fmaxf(x[e + 2 * c], x[e + 2 * c + 1]));
  return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl;
}

// The same 64 keys at a time, for kernels whose threads cannot hold 128 scores:
// the maximum is taken on one reading of S, the weights on another.  The 64
// scores at `ts`, masked by the two words of vis unless full (then in log2
// units).
__device__ __forceinline__ void load_half(uint32_t ts, bool full, uint32_t vis0, uint32_t vis1,
                                          float sl, float (&x)[64]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  tc::ld32x32b_x32(ts, r);
  tc::ld32x32b_x32(ts + 32, r + 32);
  tc::wait_ld();
  if (!full) {
#pragma unroll
    for (int e = 0; e < 64; ++e)
      x[e] = ((e < 32 ? vis0 : vis1) >> (e & 31)) & 1u ? x[e] * sl : -INFINITY;
  }
}
__device__ __forceinline__ float tile_max_halves(uint32_t ts, bool full, const uint32_t (&vis)[4],
                                                 float sl) {
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float x[64];
    load_half(ts + 64 * h, full, h ? vis[2] : vis[0], h ? vis[3] : vis[1], sl, x);
#pragma unroll
    for (int e = 0; e < 64; e += 8)
#pragma unroll
      for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], fmaxf(x[e + 2 * c], x[e + 2 * c + 1]));
  }
  const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
  return full ? mx * sl : mx;
}

// Multiplies `cols` columns of the row's O by alpha.
__device__ __forceinline__ void rescale_o(uint32_t to, int cols, float alpha) {
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    uint32_t o[32];
    tc::ld32x32b_x32(to + c, o);
    tc::wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
    tc::st32x32b_x32(to + c, o);
  }
  tc::wait_st();
}

// Weights 2^(x sl - m) of NK keys into pk as 16-bit pairs; returns their fp32 sum.
// Masked scores are -inf, with sl = 1 (tile_max has scaled the others), so that
// tiles with and without a mask run the same code.
// The pairs are the A operand of O += P V, which has V's 16-bit type (f16 where V is
// E4M3): each weight is off by at most half a step of it, 2^-8 or 2^-11 of the
// weight, as much as the output's own rounding.  The sum is of the weights before
// that, whose errors do not average out in a sum of a few keys.
template <bool BF16, int NK>
__device__ __forceinline__ float tile_weights(const float* x, float sl, float neg_m,
                                              uint32_t* pk) {
  uint64_t s[2] = {0ull, 0ull};
  const uint64_t nm = f2(neg_m, neg_m), s2 = f2(sl, sl);
#pragma unroll
  for (int c = 0; c < NK / 2; ++c) {
    float a, b;
    un2(fma2(f2(x[2 * c], x[2 * c + 1]), s2, nm), a, b);
    a = tc::ex2(a);
    b = tc::ex2(b);
    s[c & 1] = add2(s[c & 1], f2(a, b));
    pk[c] = pack2<BF16>(a, b);
  }
  float a, b;
  un2(add2(s[0], s[1]), a, b);
  return a + b;
}

// ------------------------------------------------------------------ output
// A warp's 32 rows of O leave through the 16x256b shape: four threads hold 8
// adjacent columns of a row, so that one store of the warp covers 8 rows by 32
// bytes, whole sectors (for 16-bit output after an exchange between
// neighbours).  A thread storing its own row instead touches 32 lines with
// every store: 403 against 344 us on 16 ragged prompts.

// Writes 64 columns of the warp's 32 rows: w0 x the ones at TMEM address ta, plus
// w1 x the ones at tb when TWO.  row (this thread's row of an array
// of rows of LD elements at `base`; negative: none), w0 and w1 are those of the
// row that this thread has by number; OutT is the output type (16-bit), or
// float.
template <typename OutT, bool TWO, int LD>
__device__ __forceinline__ void store_rows(uint32_t ta, uint32_t tb, OutT* base, int row,
                                           float w0, float w1) {
  constexpr bool kBf = std::is_same<OutT, __nv_bfloat16>::value;
  const int lane = threadIdx.x & 31, q = lane & 3;
  const bool odd = q & 1;
  const uint32_t rows = __ballot_sync(0xffffffffu, row >= 0);
#pragma unroll 1
  for (int hf = 0; hf < 2; ++hf) {  // rows 0 .. 15, then 16 .. 31
    if ((rows >> (16 * hf) & 0xffffu) == 0) continue;
    uint32_t a[32], b[TWO ? 32 : 1];
    tc::ld16x256b_x8(ta + ((uint32_t)(16 * hf) << 16), a);
    if constexpr (TWO) tc::ld16x256b_x8(tb + ((uint32_t)(16 * hf) << 16), b);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // rows lane / 4 and lane / 4 + 8 of them
      const int src = 16 * hf + 8 * i + (lane >> 2);
      const int r = __shfl_sync(0xffffffffu, row, src);
      const float v0 = __shfl_sync(0xffffffffu, w0, src);
      OutT* out = base + (long long)r * LD;
      uint64_t y[8];  // columns 8 k + 2 q, + 1
#pragma unroll
      for (int k = 0; k < 8; ++k)
        y[k] = mul2(f2(__uint_as_float(a[4 * k + 2 * i]), __uint_as_float(a[4 * k + 2 * i + 1])),
                    f2(v0, v0));
      if constexpr (TWO) {
        const float v1 = __shfl_sync(0xffffffffu, w1, src);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          y[k] = fma2(f2(__uint_as_float(b[4 * k + 2 * i]), __uint_as_float(b[4 * k + 2 * i + 1])),
                      f2(v1, v1), y[k]);
      }
      if constexpr (std::is_same<OutT, float>::value) {
        if (r >= 0)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint64_t*>(out + 8 * k + 2 * q) = y[k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {  // even threads take group k, odd ones k + 1
          float x0, x1, z0, z1;
          un2(y[k], x0, x1);
          un2(y[k + 1], z0, z1);
          const uint32_t x = pack2<kBf>(x0, x1), z = pack2<kBf>(z0, z1);
          const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? x : z, 1);
          if (r >= 0)
            *reinterpret_cast<uint2*>(out + 8 * (k + odd) + 4 * (q >> 1)) =
                odd ? make_uint2(got, z) : make_uint2(x, got);
        }
      }
      __syncwarp();
    }
  }
}

}  // namespace attn
}  // namespace pa
