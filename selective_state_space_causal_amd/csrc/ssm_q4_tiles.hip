// ssm_q4_tiles.hip -- ssm_q4_linear of include/ssm_block.h for any number of tokens, in tiles of BM rows of the weight by BT
// tokens, 128 columns at a step, 32 x 32 products.
//
// The codes are widened to bf16 by the waves that use them (one conversion for two weights), and e4m3 tokens likewise.  Many
// tiles are bound by the matrix cores, few by a step's own latency and by how many CUs have one; so the form goes by how many
// tiles there are (launch_form).
//   q4_ring   everything goes straight from memory to a ring of steps in LDS; groups of waves share a tile's columns
//   q4_pair   bf16 and fp32 tokens, more tiles than that: tokens through two LDS buffers, the weight straight into the operands
#include "ssm_q4_linear.h"

namespace ssm {
namespace block {
namespace {

// Tile `id` of tiles_t x tiles_m: ids that follow one another at a distance of 8 run on one XCD, which takes a contiguous part
// of the tiles, 8 token tiles wide, so that its L2 holds the rows and tokens that they share.
struct Tile {
  unsigned t, m;
};
__device__ __forceinline__ Tile tile_of(unsigned id, unsigned tiles_t, unsigned tiles_m) {
  constexpr unsigned XCDS = 8, WIDE = 8;
  const unsigned n = tiles_t * tiles_m, per = n / XCDS, more = n % XCDS, xcd = id % XCDS;
  const unsigned i = xcd * per + (xcd < more ? xcd : more) + id / XCDS;
  const unsigned group = i / (WIDE * tiles_m), first = group * WIDE;
  const unsigned wide = tiles_t - first < WIDE ? tiles_t - first : WIDE, in = i - group * WIDE * tiles_m;
  return Tile{first + in % wide, in / wide};
}

// N outputs p[m ..] of a token, 16 bytes: in one piece where the output's rows allow it (wide) and M has them all.
template <int N>
__device__ __forceinline__ void store_piece(char* p, int64_t m, const LinearArgs& a, const u32x4& v) {
  constexpr int ES = 16 / N;
  if (m >= a.M) return;
  p += m * ES;
  if (a.wide && m + N <= a.M) {
    *reinterpret_cast<u32x4*>(p) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (m + i < a.M) {
      if constexpr (ES == 2)
        reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
      else
        reinterpret_cast<unsigned*>(p)[i] = v[i];
    }
}

// A wave's tiles: a lane holds one token of each 32 (the first: `token`), and rows 8 g + 4 h + {0..3} of each 32 (from m_first).
template <int X, int NT, int NM>
__device__ __forceinline__ void store_tile(const LinearArgs& a, const f32x16 (&acc)[NT][NM], int64_t token, int64_t m_first, int h) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t row = token + t * 32;
    const bool live = row < a.T;
    float scale = 1.0f;
    if constexpr (x_scaled<X>()) scale = live ? a.x_scale[row] : 0.0f;
    char* const p = a.out.p + row * a.out.stride;
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
      for (int g = 0; g < 4; g += 2) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x_scaled<X>() ? acc[t][j][4 * g + i] * scale : acc[t][j][4 * g + i];
        const int64_t m = m_first + j * 32 + 8 * g;
        if (a.out_bf16) {
          // the halves of 8 rows are in the two halves of the wave: the upper one's first for the lower one's second
          const auto lo = __builtin_amdgcn_permlane32_swap(pack_bf16(y[0], y[1]), pack_bf16(y[4], y[5]), false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(pack_bf16(y[2], y[3]), pack_bf16(y[6], y[7]), false, false);
          if (live) store_piece<8>(p, m + 8 * h, a, u32x4{lo[0], hi[0], lo[1], hi[1]});
        } else if (live) {
          const u32x4 u = {__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])};
          const u32x4 v = {__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7])};
          store_piece<4>(p, m + 4 * h, a, u);
          store_piece<4>(p, m + 8 + 4 * h, a, v);
        }
      }
  }
}

// ---------------------------------------------------------------- many tiles

// NW waves along the rows, so that each weight is loaded and converted once.  Tokens lie in LDS as bf16, fp32 ones as three planes of
// parts; bf16 tokens go there straight from memory.
template <int X, int BM, int BT, int NW>
__global__ __launch_bounds__(64 * NW, X == X_F32 ? 1 : 2) void q4_pair(const LinearArgs a) {
  constexpr int ES = x_size<X>(), PL = planes<X>(), RB = 256, PLANE = BT * RB, TILE = PLANE * PL;
  constexpr int THREADS = 64 * NW;
  constexpr int NT = BT / 32, NM = BM / NW / 32;  // a wave's 32 x 32 tiles
  constexpr int PIECES = BT * 128 * ES / 16 / THREADS;  // 16-byte loads of a thread for a step's tokens
  static_assert((X == X_BF16 || X == X_F32) && PIECES * THREADS * 16 == BT * 128 * ES && 2 * TILE <= 160 * 1024, "");
  __shared__ __attribute__((aligned(16))) char lds[2 * TILE];

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l32 = lane % 32, h = lane / 32;
  const Tile tile = tile_of(blockIdx.x, (unsigned)((a.T + BT - 1) / BT), (unsigned)((a.M + BM - 1) / BM));
  const int64_t t0 = (int64_t)__builtin_amdgcn_readfirstlane(tile.t) * BT, m0 = (int64_t)__builtin_amdgcn_readfirstlane(tile.m) * BM;
  const int wm = wave * (NM * 32), steps = (int)a.kt;

  // a lane's rows of the weight, from the workgroup's first: at most 2^27 (16 tiles of 16 rows, 2^13 of 128 columns, 1 KB each)
  const int64_t first = m0 / 16;
  const char* const cbase = a.codes + first * a.kt * 1024;
  const char* const sbase = a.scales + first * a.k4 * 256;
  unsigned co[NM], so[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    int mt = (wm + i * 32) / 16 + l32 / 16;
    if (first + mt >= a.mt) mt = (int)(a.mt - 1 - first);  // past the last row: any, not stored
    co[i] = (unsigned)mt * (unsigned)a.kt * 1024u + (h * 16 + l32 % 16) * 16;
    so[i] = (unsigned)mt * (unsigned)a.k4 * 256u + (h * 16 + l32 % 16) * 4;
  }

  // bf16: whole steps of 128 columns; load i of a wave fills 1 KB.  Rows past the last token repeat it.
  const char* const xp = a.x.p + t0 * a.x.stride;
  const int last = (int)(a.T - 1 - t0 < BT ? a.T - 1 - t0 : BT), whole = (int)(a.K / 128);
  const auto direct = [&](int kb, char* buf) {
    const __amdgpu_buffer_rsrc_t r = resource(xp + (int64_t)kb * RB);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int p = (i * NW + wave) * 1024 + lane * 16, t = p / RB;
      const int off = min(t, last) * (int)a.x.stride + ((p % RB / 16) ^ swap_of<X>(t)) * 16;  // below 2^31: 127 rows of 2^23 bytes
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(void, buf + (i * NW + wave) * 1024), 16, off, 0, 0, 0);
    }
  };
  // Through registers: any step, zeros past the last column.
  const auto load_piece = [&](int kb, int i) {
    const int p = i * THREADS + threadIdx.x, t = p / (8 * ES), at = p % (8 * ES);  // 8 * ES pieces to a token's 128 columns
    const int64_t k = (int64_t)kb * 128 + at * (16 / ES);
    u32x4 v = {0, 0, 0, 0};
    if (t0 + t < a.T && k < a.K) v = *reinterpret_cast<const u32x4*>(xp + t * a.x.stride + k * ES);
    return v;
  };
  const auto keep_piece = [&](char* buf, int i, const u32x4& v) {
    const int p = i * THREADS + threadIdx.x, t = p / (8 * ES), at = p % (8 * ES);
    char* const row = buf + t * RB;
    if constexpr (X == X_BF16) {
      *reinterpret_cast<u32x4*>(row + (at ^ swap_of<X>(t)) * 16) = v;
    } else {  // 4 values: half a piece of each plane
      float r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = __uint_as_float(v[e]);
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        const u32x2 w = {pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3])};
        *reinterpret_cast<u32x2*>(row + k * PLANE + ((at / 2) ^ swap_of<X>(t)) * 16 + at % 2 * 8) = w;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          r[2 * e] -= __uint_as_float(w[e] << 16);
          r[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
        }
      }
    }
  };
  u32x4 xr[X == X_F32 ? PIECES : 1];
  const auto begin_x = [&](int kb, char* buf) {
    if (kb >= steps) return;
    if constexpr (X == X_BF16) {
      if (kb < whole) direct(kb, buf);
    } else {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) xr[i] = load_piece(kb, i);
    }
  };
  const auto end_x = [&](int kb, char* buf) {
    if constexpr (X == X_BF16) {
      if (kb < steps && kb >= whole) {  // the last step of an odd width: one piece after the other, no registers held for it
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) keep_piece(buf, i, load_piece(kb, i));
      }
    } else if (kb < steps) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) keep_piece(buf, i, xr[i]);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): what goes straight to LDS is there
    __syncthreads();
  };
  // Groups 2 v + h of a step's 128 columns.
  const auto load_w = [&](int kb, u32x4 (&cc)[NM][2], unsigned (&ss)[NM][2]) {
    if (kb >= steps) return;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const char* const c = cbase + (int64_t)kb * 1024 + v * 512;
      const char* const s = sbase + (int64_t)(kb >> 2) * 256 + v * 128 + (kb & 3);
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        cc[i][v] = *reinterpret_cast<const u32x4*>(c + co[i]);
        ss[i][v] = *reinterpret_cast<const uint8_t*>(s + so[i]);
      }
    }
  };

  // The tokens of the next product are read under this one; the barriers keep the compiler from reading all of a step's at
  // once, for which there are no registers.
  f32x16 acc[NT][NM] = {};
  const auto multiply = [&](const char* buf, const u32x4 (&cc)[NM][2], const unsigned (&ss)[NM][2]) {
    const char* rows = buf + l32 * RB;  // of the first tile of tokens; 32 is a multiple of what swap_of repeats at
    const int swap = swap_of<X>(l32);
    bf16x8 x[2][NT][PL];
    const auto read = [&](int n) {  // product n: columns 64 (n / 4) + 32 h + 8 (n % 4)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < PL; ++k)
          x[n % 2][t][k] = *reinterpret_cast<const bf16x8*>(rows + k * PLANE + t * 32 * RB + (((n / 4 * 8 + h * 4 + n % 4) ^ swap) * 16));
    };
    read(0);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if (n < 7) read(n + 1);
      bf16x8 w[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) w[i] = weights8(cc[i][n / 4][n % 4], pow2(ss[i][n / 4]));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = PL - 1; k >= 0; --k)
#pragma unroll
          for (int i = 0; i < NM; ++i) acc[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[i], x[n % 2][t][k], acc[t][i], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  u32x4 c[2][NM][2];
  unsigned s[2][NM][2];
  begin_x(0, lds);
  load_w(0, c[0], s[0]);
  end_x(0, lds);
  const auto step = [&](int kb, char* from, char* to, int i) {
    begin_x(kb + 1, to);
    load_w(kb + 1, c[1 - i], s[1 - i]);
    multiply(from, c[i], s[i]);
    end_x(kb + 1, to);
  };
  for (int kb = 0; kb < steps; kb += 2) {
    step(kb, lds, lds + TILE, 0);
    if (kb + 1 < steps) step(kb + 1, lds + TILE, lds, 1);
  }
  store_tile<X>(a, acc, t0 + l32, m0 + wm, h);
}

// ---------------------------------------------------------------- fewer tiles, and e4m3

// BM rows by BT tokens, with a ring of ST steps in LDS, into which tokens, codes and scales all go straight from memory.  A step's
// loads are ST - 1 steps ahead of its products, and each wave waits for its own of the step at hand only, then for the others
// at one barrier.  A step is KG blocks of 128 columns, each for a group of WM x WT waves: with one wave to a SIMD its reads,
// conversions and products follow one another (a step of 64 x 64 took 1000 cycles, 256 of them products); groups fill each
// other's gaps.  Their sums are joined in LDS, in order.
template <int X, int BM, int BT, int WM, int WT, int KG, int ST>
__global__ __launch_bounds__(64 * WM * WT * KG, 1) void q4_ring(const LinearArgs a) {
  constexpr int RB = 128 * x_size<X>(), NW = WM * WT * KG, RT = BM / 16;  // row tiles
  constexpr int NT = BT / WT / 32, NM = BM / WM / 32;
  constexpr int XS = BT * RB, CS = RT * 1024, SS = RT * 256, STAGE = KG * (XS + CS + SS);
  constexpr int XI = XS / 1024, XL = KG * XI / NW, CL = KG * RT / NW, LOADS = XL + 2 * CL;  // a wave's loads of a step
  static_assert(XL * NW == KG * XI && CL >= 1 && CL * NW == KG * RT && ST * STAGE <= 160 * 1024 && (ST - 2) * LOADS < 64, "");
  static_assert((KG - 1) * BM * BT * 4 <= ST * STAGE, "");
  __shared__ __attribute__((aligned(16))) char lds[ST * STAGE];

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l32 = lane % 32, h = lane / 32;
  const Tile tile = tile_of(blockIdx.x, (unsigned)((a.T + BT - 1) / BT), (unsigned)((a.M + BM - 1) / BM));
  const int64_t t0 = (int64_t)__builtin_amdgcn_readfirstlane(tile.t) * BT, m0 = (int64_t)__builtin_amdgcn_readfirstlane(tile.m) * BM;
  const int wt = wave % WT * (NT * 32), wm = wave / WT % WM * (NM * 32), group = wave / (WM * WT);
  const int blocks = (int)a.kt, steps = (blocks + KG - 1) / KG;
  const int whole = (int)(a.K / 128), last = (int)(a.T - 1 - t0 < BT ? a.T - 1 - t0 : BT);
  const char* const xp = a.x.p + t0 * a.x.stride;
  const int64_t first = m0 / 16;
  const int rows_left = (int)(a.mt - 1 - first < RT ? a.mt - 1 - first : RT);  // row tiles past the last repeat it, not stored

  const auto load = [&](int step, char* buf) {
    const int k0 = step * KG;
#pragma unroll
    for (int i = 0; i < CL; ++i) {  // block r / RT of the step (past the last one: that again, not used), row tile r % RT
      const int r = i * NW + wave, kb = min(k0 + r / RT, blocks - 1), row = min(r % RT, rows_left);
      const __amdgpu_buffer_rsrc_t rc = resource(a.codes + ((first + row) * a.kt + kb) * 1024);
      const __amdgpu_buffer_rsrc_t rs = resource(a.scales + ((first + row) * a.k4 + (kb >> 2)) * 256);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, LDS_PTR(void, buf + KG * XS + r * 1024), 16, lane * 16, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, LDS_PTR(void, buf + KG * (XS + CS) + r * 256), 4, lane * 4, 0, 0, 0);
    }
    if (k0 + KG <= whole) {
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const int r = i * NW + wave, at = r % XI * 1024 + lane * 16, t = at / RB;
        const int off = min(t, last) * (int)a.x.stride + ((at % RB / 16) ^ swap_of<X>(t)) * 16;  // below 2^31: 127 rows of 2^24 bytes
        __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(xp + (int64_t)(k0 + r / XI) * RB), LDS_PTR(void, buf + r * 1024), 16, off, 0, 0, 0);
      }
    } else {  // the last step of an odd width: zeros past the last column
#pragma unroll 1
      for (int i = 0; i < XL; ++i) {
        const int r = i * NW + wave, at = r % XI * 1024 + lane * 16, t = at / RB, piece = (at % RB / 16) ^ swap_of<X>(t);
        const int64_t k = (int64_t)(k0 + r / XI) * RB + piece * 16;
        u32x4 v = {0, 0, 0, 0};
        if (k < a.K * x_size<X>()) v = *reinterpret_cast<const u32x4*>(xp + min(t, last) * a.x.stride + k);
        *reinterpret_cast<u32x4*>(buf + r * 1024 + lane * 16) = v;
      }
    }
  };

  f32x16 acc[NT][NM] = {};
  const auto multiply = [&](int kb, const char* buf) {
    const char* rows = buf + group * XS + (wt + l32) * RB;
    const int swap = swap_of<X>(l32);
    const char* codes = buf + KG * XS + group * CS + (wm / 16 + l32 / 16) * 1024 + (h * 16 + l32 % 16) * 16;
    const char* scales = buf + KG * (XS + CS) + group * SS + (wm / 16 + l32 / 16) * 256 + (h * 16 + l32 % 16) * 4 + (kb & 3);
    u32x4 cc[NM][2];  // groups 2 v + h of the block's columns
    unsigned ss[NM][2];
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        cc[i][v] = *reinterpret_cast<const u32x4*>(codes + i * 2048 + v * 512);
        ss[i][v] = *reinterpret_cast<const uint8_t*>(scales + i * 512 + v * 128);
      }
    // Product n: columns 64 (n / 4) + 32 h + 8 (n % 4); fp32 tokens are read one product ahead, the others all at once.
    constexpr int AHEAD = X == X_F32 ? 2 : 8;
    Eight<X> x[AHEAD][NT];
    const auto read = [&](int n) {
#pragma unroll
      for (int t = 0; t < NT; ++t) x[n % AHEAD][t].read(rows + t * 32 * RB, n / 4 * 8 + h * 4 + n % 4, swap);
    };
#pragma unroll
    for (int n = 0; n < AHEAD - 1; ++n) read(n);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if (n + AHEAD - 1 < 8) read(n + AHEAD - 1);
      bf16x8 w[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) w[i] = weights8(cc[i][n / 4][n % 4], pow2(ss[i][n / 4]));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        bf16x8 p[planes<X>()];
        x[n % AHEAD][t].parts(p);
#pragma unroll
        for (int k = planes<X>() - 1; k >= 0; --k)
#pragma unroll
          for (int i = 0; i < NM; ++i) acc[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[i], p[k], acc[t][i], 0, 0, 0);
      }
      if constexpr (X == X_F32) __builtin_amdgcn_sched_barrier(0);
    }
  };

#pragma unroll
  for (int p = 0; p < ST - 1; ++p)
    if (p < steps) load(p, lds + p * STAGE);
  int at = 0;  // of the step at hand in the ring
  const auto everyone = [] {  // the compiler keeps what is read and written on either side there
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int st = 0; st < steps; ++st) {
    // This wave's loads of the step are done once no more than the later steps' are on their way; with fewer steps left, or
    // one that came through registers, all are waited for.  The barrier covers the other waves' loads, and their reads of
    // the step before, whose place is filled next.
    __builtin_amdgcn_sched_barrier(0);
    if (st + ST - 2 < steps && (st + ST - 1) * KG <= whole)
      __builtin_amdgcn_s_waitcnt(0x0070 | ((ST - 2) * LOADS & 15) | ((ST - 2) * LOADS >> 4 << 14));
    else
      __builtin_amdgcn_s_waitcnt(0x0070);
    everyone();
    const int to = at == 0 ? ST - 1 : at - 1;
    if (st + ST - 1 < steps) load(st + ST - 1, lds + to * STAGE);
    __builtin_amdgcn_sched_barrier(0);
    const int kb = st * KG + group;
    if (kb < blocks) multiply(kb, lds + at * STAGE);
    at = at == ST - 1 ? 0 : at + 1;
  }
  if constexpr (KG > 1) {
    __syncthreads();  // the ring is read
    f32x4* const mine = reinterpret_cast<f32x4*>(lds) + wave % (WM * WT) * (NT * NM * 256) + lane;
#pragma unroll
    for (int g = 1; g < KG; ++g)
#pragma unroll
      for (int i = 0; i < NT * NM * 4; ++i) {
        const f32x16& v = acc[i / 4 / NM][i / 4 % NM];
        const int e = i % 4 * 4;
        if (group == g) mine[(g - 1) * (BM * BT / 4) + i * 64] = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
      }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < KG; ++g)
#pragma unroll
      for (int i = 0; i < NT * NM * 4; ++i) {
        const f32x4 v = mine[(g - 1) * (BM * BT / 4) + i * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i / 4 / NM][i / 4 % NM][i % 4 * 4 + e] += v[e];
      }
  }
  store_tile<X>(a, acc, t0 + wt + l32, m0 + wm, h);
}

// ---------------------------------------------------------------- the form of a call

int64_t tiles_of(const LinearArgs& a, int bm, int bt) { return (a.T + bt - 1) / bt * ((a.M + bm - 1) / bm); }

template <int X, int BM, int BT, int NW>
hipError_t pair(const LinearArgs& a, hipStream_t s) {
  q4_pair<X, BM, BT, NW><<<dim3((unsigned)tiles_of(a, BM, BT)), dim3(64 * NW), 0, s>>>(a);
  return hipGetLastError();
}

template <int X, int BM, int BT, int WM, int WT, int KG, int ST>
hipError_t ring(const LinearArgs& a, hipStream_t s) {
  q4_ring<X, BM, BT, WM, WT, KG, ST><<<dim3((unsigned)tiles_of(a, BM, BT)), dim3(64 * WM * WT * KG), 0, s>>>(a);
  return hipGetLastError();
}

// q4_pair in the tile whose fullest CU has the fewest products, each tile's weighed by what it takes for the same ones where there
// are many tiles.  us in the tiles in this order, rows by tokens:
//   bf16   (256, 128), (256, 96), (256, 64), (128, 96), (128, 64)
//     4096 by 16384 x 4096   399 (1378 TFLOP/s), 422, 426, 442, 448; with four waves of 64 x 64 in (128, 128) 460
//     1000 by 4096 x 4096   51, 42, 32.9, 39, 32.7     1200   51, 42.4, 47, 42.0, 42.9     1600   52, 66, 51, 57, 54
//     2048 by 4096 x 4096   57, 69, 58, 63, 60         2200   84, 70, 76, 64.6, 71         3000   89, 81, 84, 87, 87
//     5000 by 2560 x 5120   116, 139, 129, 125, 124: it takes the last, where the first is faster   8192   184, 189, 181, 191, 192
//   fp32   (256, 32), (128, 32)
//     4096 by 4096 x 4096   352, 405; in (128, 64) 498   1000   91, 110   600   75, 73   300 by 5120 x 2560   29, 33
//     300 by 2560 x 2560   28, 23                        64 by 65536 x 2560   62, 75
template <int X>
hipError_t pair_form(const LinearArgs& a, hipStream_t s) {
  const auto cost = [&](int bm, int bt, int us) { return (tiles_of(a, bm, bt) + 255) / 256 * (bm * bt / 64) * us; };
  if constexpr (X == X_F32) return cost(256, 32, 352) <= cost(128, 32, 405) ? pair<X, 256, 32, 8>(a, s) : pair<X, 128, 32, 4>(a, s);
  const int64_t c[5] = {cost(256, 128, 399), cost(256, 96, 422), cost(256, 64, 426), cost(128, 96, 442), cost(128, 64, 448)};
  int best = 0;
  for (int i = 1; i < 5; ++i)
    if (c[i] < c[best]) best = i;
  if constexpr (X == X_BF16)
    return best == 0   ? pair<X, 256, 128, 4>(a, s)
           : best == 1 ? pair<X, 256, 96, 4>(a, s)
           : best == 2 ? pair<X, 256, 64, 4>(a, s)
           : best == 3 ? pair<X, 128, 96, 4>(a, s)
                       : pair<X, 128, 64, 4>(a, s);
  return hipErrorInvalidValue;
}

// The smallest tile of which there is at most one to a CU: each CU's share of the columns' way is then shortest, and no CU has
// a second one while others have none.  us by tile, (32, 32), (64, 32), (64, 64), (128, 64), (128, 128) rows by tokens:
//   bf16   128 tokens by 4096 x 4096   -, 9.9, 13.6, 17.6, 30     300 by 5120 x 2560   35, 23, 18, 12.7, 20
//          64 by 16384 x 4096   29, 18, 13.9, 17.5, 30
//   e4m3   64 by 4096 x 8192   9.6, 14.8, 19, 36, 59   128 by 4096 x 4096   11.4, 9.0, 11.7, 20, -
//          300 by 5120 x 2560   -, 23, 17, 14.3, 21.5
// 96 tokens by 128 rows is the largest of those (600 by 4096 x 4096, [the next form]: bf16 24.5 [29.9], e4m3 24.3 [29]).  Past that:
//   bf16   q4_pair in the tile whose fullest CU has the least to multiply (pair_form)
//   e4m3   up to 512 tiles of 128 x 64 with two steps in the ring, two or three of them to a CU (1000 by 4096 x 4096 33.5, 35 in
//          128 x 128); then 128 x 192 where that is one to a CU (1500 by 4096 x 4096 46.6, 53 in 128 x 128); 256 x 128 where that
//          is (2048 by 4096 x 4096 58.6, 61) and from more than 768 tiles of 128 x 128 on (4096 by 16384 x 4096 404, 450; 3000 by
//          4096 x 4096, 768 tiles, 89, 88); else 128 x 128
// Up to 32 and up to 64 tokens a tile has no more of them, however many rows there are: reading the weight bounds the call.
// Without and with that, us: 32 bf16 tokens by 65536 x 2560 37, 18.5 (5.1 TB/s), by 32768 x 4096 19.7, 14.8; e4m3 29, 18.3 and
// 21, 15.5.  64 by 65536 x 2560 bf16 41, 31, e4m3 41, 27.
// fp32 tokens by 64 rows where that is one to a CU: 32 by 16384 x 4096 28 us, 40 by 128 rows.
template <int X>
hipError_t launch_form(const LinearArgs& a, hipStream_t s) {
  const auto once = [&](int bm, int bt) { return tiles_of(a, bm, bt) <= 256; };
  if constexpr (X == X_F32) {
    if (once(32, 32)) return ring<X, 32, 32, 1, 1, 4, 2>(a, s);
    if (once(64, 32)) return ring<X, 64, 32, 2, 1, 2, 2>(a, s);
    return pair_form<X>(a, s);
  } else {
    constexpr bool E = x_size<X>() == 1;  // half of the LDS: more steps
    if (once(32, 32)) return ring<X, 32, 32, 1, 1, E ? 8 : 4, 3>(a, s);
    if (once(64, 32)) return ring<X, 64, 32, 2, 1, 4, E ? 3 : 2>(a, s);
    if (a.T <= 32) return once(128, 32) ? ring<X, 128, 32, 4, 1, 2, 3>(a, s) : ring<X, 128, 32, 4, 1, 2, 2>(a, s);
    if (once(64, 64)) return ring<X, 64, 64, 2, 2, E ? 4 : 2, 3>(a, s);
    if (once(128, 64)) return ring<X, 128, 64, 4, 1, 2, E ? 4 : 2>(a, s);
    if (once(128, 96)) return ring<X, 128, 96, 4, 1, 2, 2>(a, s);
    if constexpr (E)
      if (tiles_of(a, 128, 64) <= 512) return ring<X, 128, 64, 4, 1, 2, 2>(a, s);
    if (a.T <= 64) return ring<X, 128, 64, 4, 1, E ? 2 : 1, E ? 2 : 3>(a, s);
    if constexpr (X == X_BF16) return pair_form<X>(a, s);
    if constexpr (E) {
      if (once(128, 192)) return ring<X, 128, 192, 4, 2, 1, 2>(a, s);
      if (tiles_of(a, 128, 128) > 768 || once(256, 128)) return ring<X, 256, 128, 4, 2, 1, 2>(a, s);
      return ring<X, 128, 128, 4, 2, 1, 2>(a, s);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_q4_tiles(const LinearArgs& a, int x, hipStream_t s) {
  return x == X_F32 ? launch_form<X_F32>(a, s) : x == X_BF16 ? launch_form<X_BF16>(a, s) : launch_form<X_E4M3>(a, s);
}

}  // namespace block
}  // namespace ssm

extern "C" int ssm_q4_linear(int64_t tokens, int32_t x_dtype, int32_t out_dtype, const ssm_rows* x, const float* x_scale,
                             const ssm_q4_weight* q, const ssm_rows* out, void* stream) {
  using namespace ssm::block;
  if (tokens < 0 || tokens >= MAX_TOKENS) return SSM_ERR_SHAPE;
  if (x_dtype != SSM_F32 && x_dtype != SSM_BF16 && x_dtype != SSM_E4M3) return SSM_ERR_DTYPE;
  if (out_dtype != SSM_F32 && out_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  if (const int st = check_q4(q)) return st;
  if (tokens * q->out_features > MAX_OUTPUTS) return SSM_ERR_SHAPE;
  if (tokens == 0) return SSM_OK;  // its tensors have no addresses
  if ((x_dtype == SSM_E4M3) != (x_scale != nullptr)) return SSM_ERR_NULL;
  const int64_t T = tokens, M = q->out_features, K = q->in_features, es = size_of(x_dtype), os = size_of(out_dtype);
  if (const int st = check_rows(x, es, 16)) return st;
  if (const int st = check_rows(out, os, os)) return st;
  if (!aligned(x_scale, 4)) return SSM_ERR_ALIGN;
  const Span so = rows_span(out, T, M, os);
  if (overlaps(so, codes_span(q)) || overlaps(so, scales_span(q)) || overlaps(so, span(x_scale, x_scale ? T * 4 : 0)))
    return SSM_ERR_ALIAS;
  if (!writable(out, T, M) || rows_overlap(out, M, os, x, K, es, T)) return SSM_ERR_ALIAS;
  LinearArgs a = {};
  a.x = rows_of(x, es);
  a.out = rows_of(out, os);
  a.codes = static_cast<const char*>(q->codes);
  a.scales = static_cast<const char*>(q->scales);
  a.x_scale = x_scale;
  a.T = T;
  a.M = M;
  a.K = K;
  a.kt = (K + 127) / 128;
  a.k4 = (K + 511) / 512;
  a.mt = (M + 15) / 16;
  a.out_bf16 = out_dtype == SSM_BF16;
  a.wide = aligned(out->data, 16) && out->stride * os % 16 == 0;
  const hipStream_t s = ready(stream);
  const hipError_t e = rows_takes(a, x_dtype)  ? launch_q4_rows(a, x_dtype, s)
                       : few_takes(a, x_dtype) ? launch_q4_few(a, x_dtype, s)
                                               : launch_q4_tiles(a, x_dtype, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}
