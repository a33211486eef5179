// ssm_attn_prefill.h -- what the prompt-attention kernels (ssm_attn_prefill.hip, ssm_attn_split.hip) share.
//
// Rows.  The query heads that share a key head are packed into the rows of a tile: row r of a sequence
// is token r / G, query head kv_head * G + r % G (G = query heads per key head).  A key tile is then
// read once for all G heads, and a short sequence fills a tile G times better.
#pragma once
#include "ssm_attn.h"

namespace ssm {
namespace attn {

// Limits of a call, so that the kernels' ints hold: they step up to 256 keys past a sequence's end, and add the counts of
// tiles (of 32 rows or more) of 64 sequences, each of which may claim every row where the offsets are not in order.
constexpr int64_t MAX_KEYS = (int64_t)INT32_MAX - (1 << 20), MAX_ROWS = (int64_t(1) << 30) - 32;

typedef short s16x4 __attribute__((ext_vector_type(4)));
#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

struct PrefillArgs {
  View q, k, v, out;
  float* lse;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, Hq, Hkv, G, D;
  int causal;
  float scale_log2;  // scale * log2(e)
  unsigned g_times, g_shift;  // division by G
};

// x / G for 0 <= x < 2^31: with s = ceil(log2 G) and m = ceil(2^(31 + s) / G), which is in [2^31, 2^32), x m / 2^(31 + s) is
// above x / G by less than x / 2^31 / G, too little to reach the next whole number.
inline void set_group(PrefillArgs& a, int G) {
  a.G = G;
  a.g_shift = 0;
  while ((int64_t(1) << a.g_shift) < G) ++a.g_shift;
  a.g_times = (unsigned)(((uint64_t(1) << (31 + a.g_shift)) + G - 1) / G);
}
__device__ __forceinline__ int by_group(const PrefillArgs& a, int x) {
  return (int)(__umulhi(2u * (unsigned)x, a.g_times) >> a.g_shift);
}

// Keys that a token (below lq) of a sequence sees: the first ones.  In an order whose sums stay within 32 bits.
__device__ __forceinline__ int seen_of(const PrefillArgs& a, int lq, int lk, int token) {
  return a.causal ? max(lk - (lq - 1 - token), 0) : lk;
}

// Inclusive prefix sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // the 16 lanes of a row: 1, 2, 4, 8 to the right
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row 0's sum into row 1, row 2's into 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // the lower half's into the upper half
  return x;
}

struct Work {
  int tile, tiles;     // of the sequence's rows
  int q0, lq, k0, lk;  // its queries and keys
};

// The same value, of which the compiler knows nothing: what is computed from it stays where it stands, instead of
// being kept in registers through the loop over keys, which needs them all.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// (q0, lq, k0, lk) of sequence b; empty past the last.
__device__ __forceinline__ int4 bounds(const PrefillArgs& a, int b) {
  int4 s = {0, 0, 0, 0};
  if (b < a.B) {
    s.x = min(max(a.cu_q[b], 0), a.Tq);
    s.y = max(min(a.cu_q[b + 1], a.Tq) - s.x, 0);
    s.z = min(max(a.cu_k[b], 0), a.Tk);
    s.w = max(min(a.cu_k[b + 1], a.Tk) - s.z, 0);
  }
  return s;
}

__device__ __forceinline__ int tiles_of(const PrefillArgs& a, int QT, int lq) {
  return (int)(((unsigned)(lq * a.G) + QT - 1) / QT);
}

// The sequence and tile that hold tile `idx` of the packed batch (false past the end).  Each wave finds
// it by itself: 64 sequences at a time, a prefix sum of their tile counts over the lanes.
__device__ __forceinline__ bool find_tile(const PrefillArgs& a, int QT, int64_t idx, Work& w) {
  const int lane = threadIdx.x & 63;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int4 q = bounds(a, b0 + lane);
    const int n = tiles_of(a, QT, q.y), incl = wave_scan(n);
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (idx < base + total) {
      const int want = (int)(idx - base);
      const int at = __ffsll((unsigned long long)__ballot(incl > want)) - 1;
      w.tiles = __builtin_amdgcn_readlane(n, at);
      w.tile = want - (__builtin_amdgcn_readlane(incl, at) - w.tiles);
      w.q0 = __builtin_amdgcn_readlane(q.x, at);
      w.lq = __builtin_amdgcn_readlane(q.y, at);
      w.k0 = __builtin_amdgcn_readlane(q.z, at);
      w.lk = __builtin_amdgcn_readlane(q.w, at);
      return true;
    }
    base += total;
  }
  return false;
}

// The two halves' values of one row joined: max / sum over lane and lane ^ 32.
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Key heads and tiles (at most: the sum of ceil(rows / QT) over the sequences) of no more than `places` workgroups,
// heads first: the eight XCDs take workgroups in turn, so that with eight heads each XCD's L2 holds the keys of one.
inline int64_t tiles_at_most(const PrefillArgs& a, int QT) { return (int64_t)a.Tq * a.G / QT + a.B; }
inline dim3 tiles_grid(const PrefillArgs& a, int QT, int places) {
  const int64_t tiles = tiles_at_most(a, QT);
  int64_t most = places / a.Hkv;
  most = most < 1 ? 1 : most > 65535 ? 65535 : most;
  return dim3(a.Hkv, (unsigned)(tiles < most ? tiles : most));
}

// The key axis split over a workgroup's waves (ssm_attn_split.hip); the launch's error is left for hipGetLastError.
void launch_split(const PrefillArgs& a, bool bf16, hipStream_t s);

}  // namespace attn
}  // namespace ssm
