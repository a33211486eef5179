// ssm_q4_tiles.hip -- ssm_q4_linear of include/ssm_block.h for any number of tokens.
//
// A workgroup makes BM rows of the weight by BT tokens, 128 columns at a step.  The tokens' tile goes straight from memory to
// one of two LDS buffers while the other is multiplied (fp32 tokens, and e4m3 ones for an fp32 output, through registers, where
// they become bf16); the weight goes from memory straight into the operands: a lane loads the groups of its own row, 16 bytes
// each, and widens them to bf16 (bf16 and fp32 tokens) or hands them to the instruction that takes codes and scales (e4m3
// tokens).  32 x 32 products.  LDS pieces of 16 bytes are exchanged within a token's row so that the lanes of a read fall on
// different banks.  Where there are too few tiles for the CUs, several workgroups share a tile's columns, write fp32 sums to
// the workspace, and a second launch adds them in order.
#include "ssm_q4_linear.h"

#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

namespace ssm {
namespace block {
namespace {

// fp32 tokens lie in LDS as three planes of bf16 parts.
template <int X>
constexpr int planes() {
  return X == X_F32 ? 3 : 1;
}
template <int X>
constexpr int row_bytes() {
  return X == X_E4M3 ? 128 : 256;
}

// What is exchanged in token row t of a plane: piece c (16 bytes) lies at place c ^ swap(t), so that 16 neighbouring rows'
// pieces c cover all 64 banks.
template <int X>
__device__ __forceinline__ int swap_of(int t) {
  return X == X_E4M3 ? (t >> 1) & 7 : t & 15;
}
template <int X>
__device__ __forceinline__ int place(int t, int c) {
  return t * row_bytes<X>() + ((c ^ swap_of<X>(t)) * 16);
}

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

__device__ __forceinline__ unsigned f2u(float v) { return __float_as_uint(v); }

// N outputs p[m ..] of a token, 16 bytes: in one piece where the output's rows allow it (wide) and M has them all.
template <int N, typename OUT>
__device__ __forceinline__ void store_rows(OUT* p, int64_t m, int64_t M, bool live, bool wide, const u32x4& v) {
  if (!live || m >= M) return;
  if (wide && m + N <= M) {
    *reinterpret_cast<u32x4*>(p + m) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (m + i < M) {
      if constexpr (sizeof(OUT) == 2)
        p[m + i] = bf16_t{(uint16_t)(v[i / 2] >> (16 * (i % 2)))};
      else
        p[m + i] = __uint_as_float(v[i]);
    }
}

// WM x WT waves: along rows and along tokens.
template <int X, int BM, int BT, int WM, int WT, typename OUT>
__global__ __launch_bounds__(64 * WM * WT, X == X_F32 && BT == 64 ? 1 : 2) void q4_tiles(const LinearArgs a, int splits) {
  constexpr int ES = x_size<X>(), PL = planes<X>(), RB = row_bytes<X>(), PLANE = BT * RB, TILE = PLANE * PL;
  constexpr int NW = WM * WT, THREADS = 64 * NW;
  constexpr int NT = BT / WT / 32, NM = BM / WM / 32;  // a wave's 32 x 32 tiles
  constexpr bool BIG = BM == 256;
  constexpr bool DIRECT = X == X_BF16 || X == X_E4M3;
  constexpr int PIECES = BT * 128 * ES / 16 / THREADS;  // 16-byte loads of a thread for a step's tokens
  static_assert(PIECES >= 1 && PIECES * THREADS * 16 == BT * 128 * ES && 2 * TILE <= 160 * 1024, "");
  __shared__ __attribute__((aligned(16))) char lds[2 * TILE];

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l32 = lane % 32, h = lane / 32;
  const Tile tile = tile_of(blockIdx.x, (unsigned)((a.T + BT - 1) / BT), (unsigned)((a.M + BM - 1) / BM));
  const int64_t t0 = (int64_t)__builtin_amdgcn_readfirstlane(tile.t) * BT, m0 = (int64_t)__builtin_amdgcn_readfirstlane(tile.m) * BM;
  const int wt = wave % WT * (NT * 32), wm = wave / WT * (NM * 32);
  // this workgroup's share of the steps
  const int k_lo = (int)(a.kt * blockIdx.y / splits), k_hi = (int)(a.kt * (blockIdx.y + 1) / splits);

  // a lane's rows of the weight, from the workgroup's first: below 2^32 (17 tiles of 16 rows, 2^13 of 128 columns, 1 KB each)
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

  // Tokens straight into LDS, whole steps of 128 columns: load i of a wave fills 1 KB.  Rows past the last token repeat it.
  const char* const xp = a.x.p + t0 * a.x.stride;
  const int last = (int)(a.T - 1 - t0 < BT ? a.T - 1 - t0 : BT);
  const auto direct = [&](int kb, char* buf) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(xp + (int64_t)kb * RB), (short)0, 0x7FFFFFFF, 0x00020000);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int p = (i * NW + wave) * 1024 + lane * 16, t = p / RB;
      const int off = min(t, last) * (int)a.x.stride + ((p % RB / 16) ^ swap_of<X>(t)) * 16;  // below 2^31: 255 rows of 2^23 bytes
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
  const auto store_piece = [&](char* buf, int i, const u32x4& v) {
    const int p = i * THREADS + threadIdx.x, t = p / (8 * ES), at = p % (8 * ES);
    if constexpr (X == X_WIDE) {
      *reinterpret_cast<bf16x8*>(buf + place<X>(t, 2 * at)) = widen8(v[0], v[1]);
      *reinterpret_cast<bf16x8*>(buf + place<X>(t, 2 * at + 1)) = widen8(v[2], v[3]);
    } else if constexpr (X != X_F32) {
      *reinterpret_cast<u32x4*>(buf + place<X>(t, at)) = v;
    } else {  // 4 values: half a piece of each plane
      float r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = __uint_as_float(v[e]);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const u32x2 w = {pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3])};
        *reinterpret_cast<u32x2*>(buf + k * PLANE + place<X>(t, at / 2) + at % 2 * 8) = w;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          r[2 * e] -= __uint_as_float(w[e] << 16);
          r[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
        }
      }
    }
  };
  u32x4 xr[DIRECT ? 1 : PIECES];
  const int whole = (int)(a.K / 128);  // steps without a column past the last
  const auto begin_x = [&](int kb, char* buf) {
    if (kb >= k_hi) return;
    if constexpr (DIRECT) {
      if (kb < whole) direct(kb, buf);
    } else {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) xr[i] = load_piece(kb, i);
    }
  };
  const auto end_x = [&](int kb, char* buf) {
    if constexpr (DIRECT) {
      if (kb < k_hi && kb >= whole) {  // the last step of an odd width: one piece after the other, no registers held for it
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) store_piece(buf, i, load_piece(kb, i));
      }
    } else if (kb < k_hi) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) store_piece(buf, i, xr[i]);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): what goes straight to LDS is there
    __syncthreads();
  };
  // Groups 2 v + h of a step's 128 columns.
  const auto load_w = [&](int kb, int v, u32x4 (&cc)[NM][2], unsigned (&ss)[NM][2]) {
    if (kb >= k_hi) return;
    const char* const c = cbase + (int64_t)kb * 1024 + v * 512;
    const char* const s = sbase + (int64_t)(kb >> 2) * 256 + v * 128 + (kb & 3);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      cc[i][v] = *reinterpret_cast<const u32x4*>(c + co[i]);
      ss[i][v] = *reinterpret_cast<const uint8_t*>(s + so[i]);
    }
  };

  // The tokens of the next product are read under this one; the barriers keep the compiler from reading all of a step's at
  // once, for which there are no registers.
  f32x16 acc[NT][NM] = {};
  const auto multiply = [&](const char* buf, const u32x4 (&cc)[NM][2], const unsigned (&ss)[NM][2], const auto& half_done) {
    const char* rows = buf + (wt + l32) * RB;  // of the first tile of tokens; wt and 32 are multiples of what swap_of repeats at
    const int swap = swap_of<X>(l32);
    if constexpr (X == X_E4M3) {
      u32x4 x[2][NT][2];
      const auto read = [&](int v) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            x[v][t][p] = *reinterpret_cast<const u32x4*>(rows + t * 32 * RB + (((4 * v + 2 * p + h) ^ swap) * 16));
      };
      read(0);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        if (v == 0) read(1);
        i32x8 w[NM];
#pragma unroll
        for (int i = 0; i < NM; ++i) w[i] = i32x8{(int)cc[i][v][0], (int)cc[i][v][1], (int)cc[i][v][2], (int)cc[i][v][3], 0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const i32x8 xv = __builtin_bit_cast(i32x8, __builtin_shufflevector(x[v][t][0], x[v][t][1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
          for (int i = 0; i < NM; ++i)
            acc[t][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[i], xv, acc[t][i], 4, 0, 0, (int)ss[i][v], 0, 0x7F7F7F7F);
        }
        if (v == 0) half_done();
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      bf16x8 x[2][NT][PL];
      const auto read = [&](int n) {  // product n = 4 v + j: columns 64 v + 32 h + 8 j
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
        if (n == 3) half_done();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  begin_x(k_lo, lds);
  if constexpr (BIG) {
    // No registers for two steps' weights: the first half of the next one's comes in once this one's is used, the second
    // half of a step's at its beginning.
    u32x4 c[NM][2];
    unsigned s[NM][2];
    load_w(k_lo, 0, c, s);
    end_x(k_lo, lds);
    const auto step = [&](int kb, char* from, char* to) {
      begin_x(kb + 1, to);
      load_w(kb, 1, c, s);
      __builtin_amdgcn_sched_barrier(0);
      multiply(from, c, s, [&] { load_w(kb + 1, 0, c, s); });
      end_x(kb + 1, to);
    };
    for (int kb = k_lo; kb < k_hi; kb += 2) {
      step(kb, lds, lds + TILE);
      if (kb + 1 < k_hi) step(kb + 1, lds + TILE, lds);
    }
  } else {
    u32x4 c[2][NM][2];
    unsigned s[2][NM][2];
    load_w(k_lo, 0, c[0], s[0]);
    load_w(k_lo, 1, c[0], s[0]);
    end_x(k_lo, lds);
    const auto step = [&](int kb, char* from, char* to, int i) {
      begin_x(kb + 1, to);
      load_w(kb + 1, 0, c[1 - i], s[1 - i]);
      load_w(kb + 1, 1, c[1 - i], s[1 - i]);
      multiply(from, c[i], s[i], [] {});
      end_x(kb + 1, to);
    };
    for (int kb = k_lo; kb < k_hi; kb += 2) {
      step(kb, lds, lds + TILE, 0);
      if (kb + 1 < k_hi) step(kb + 1, lds + TILE, lds, 1);
    }
  }

  // A lane holds one token, and rows 8 g + 4 h + {0..3} of each 32.
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t row = t0 + wt + t * 32 + l32;
    const bool live = row < a.T;
    if (splits > 1) {
      float* p = a.partial + (blockIdx.y * a.T + row) * a.Mp;
#pragma unroll
      for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int64_t m = m0 + wm + j * 32 + 8 * g + 4 * h;
          if (live && m < a.M)
            *reinterpret_cast<f32x4*>(p + m) = f32x4{acc[t][j][4 * g], acc[t][j][4 * g + 1], acc[t][j][4 * g + 2], acc[t][j][4 * g + 3]};
        }
      continue;
    }
    float scale = 1.0f;
    if constexpr (x_scaled<X>()) scale = live ? a.x_scale[row] : 0.0f;
    OUT* p = reinterpret_cast<OUT*>(a.out.p + row * a.out.stride);
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
      for (int g = 0; g < 4; g += 2) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x_scaled<X>() ? acc[t][j][4 * g + i] * scale : acc[t][j][4 * g + i];
        const int64_t m = m0 + wm + j * 32 + 8 * g;
        if constexpr (sizeof(OUT) == 2) {
          // the halves of 8 rows are in the two halves of the wave: the upper one's first for the lower one's second
          const auto lo = __builtin_amdgcn_permlane32_swap(pack_bf16(y[0], y[1]), pack_bf16(y[4], y[5]), false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(pack_bf16(y[2], y[3]), pack_bf16(y[6], y[7]), false, false);
          store_rows<8>(p, m + 8 * h, a.M, live, a.wide, u32x4{lo[0], hi[0], lo[1], hi[1]});
        } else {
          store_rows<4>(p, m + 4 * h, a.M, live, a.wide, u32x4{f2u(y[0]), f2u(y[1]), f2u(y[2]), f2u(y[3])});
          store_rows<4>(p, m + 8 + 4 * h, a.M, live, a.wide, u32x4{f2u(y[4]), f2u(y[5]), f2u(y[6]), f2u(y[7])});
        }
      }
  }
}

// Sums of the parts, in order, four rows of the weight to a thread.
template <bool SCALED, typename OUT>
__global__ __launch_bounds__(256) void q4_join(const LinearArgs a, int splits) {
  const int64_t per = a.Mp / 4, n = a.T * per, step = (int64_t)gridDim.x * 256;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < n; o += step) {
    const int64_t t = o / per, m = o % per * 4;
    f32x4 y = {0, 0, 0, 0};
    for (int i = 0; i < splits; ++i) y += *reinterpret_cast<const f32x4*>(a.partial + (i * n + o) * 4);
    if constexpr (SCALED) y *= a.x_scale[t];
    OUT* p = reinterpret_cast<OUT*>(a.out.p + t * a.out.stride);
    if constexpr (sizeof(OUT) == 4) {
      store_rows<4>(p, m, a.M, true, a.wide, u32x4{f2u(y[0]), f2u(y[1]), f2u(y[2]), f2u(y[3])});
    } else {
      const u32x2 v = {pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
      if (a.wide && m + 4 <= a.M) {
        *reinterpret_cast<u32x2*>(p + m) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (m + i < a.M) p[m + i] = bf16_t{(uint16_t)(v[i / 2] >> (16 * (i % 2)))};
      }
    }
  }
}

template <int X, int BM, int BT, int WM, int WT, typename OUT>
hipError_t launch(const LinearArgs& a, int splits, hipStream_t s) {
  const int64_t tiles = (a.T + BT - 1) / BT * ((a.M + BM - 1) / BM);
  q4_tiles<X, BM, BT, WM, WT, OUT><<<dim3((unsigned)tiles, (unsigned)splits), dim3(64 * WM * WT), 0, s>>>(a, splits);
  if (const hipError_t e = hipGetLastError()) return e;
  if (splits > 1) {
    const int64_t want = (a.T * a.Mp / 4 + 255) / 256;
    q4_join<x_scaled<X>(), OUT><<<dim3((unsigned)(want < 4096 ? want : 4096)), dim3(256), 0, s>>>(a, splits);
  }
  return hipGetLastError();
}

// The form of a call: tokens and rows of a tile, and how many workgroups share its columns.
struct Form {
  int bm, bt, splits;
};

Form form_of(int64_t T, int x_dtype, int64_t M, int64_t K) {
  const auto tiles = [&](int bm, int bt) { return (T + bt - 1) / bt * ((M + bm - 1) / bm); };
  Form f = {128, T <= 32 ? 32 : T <= 64 || x_dtype == X_F32 ? 64 : 128, 1};
  if (f.bt == 128 && tiles(256, 256) >= 192) return Form{256, 256, 1};
  // two workgroups to a CU are wanted, and four steps of 128 columns at least for each
  const int64_t steps = (K + 127) / 128;
  int64_t n = 512 / tiles(f.bm, f.bt);
  if (n > steps / 4) n = steps / 4;
  f.splits = n < 1 ? 1 : n > 16 ? 16 : (int)n;
  return f;
}

template <int X, typename OUT>
hipError_t launch_form(const LinearArgs& a, const Form& f, hipStream_t s) {
  if (f.bt == 32) return launch<X, 128, 32, 4, 1, OUT>(a, f.splits, s);
  if (f.bt == 64) return launch<X, 128, 64, X == X_F32 ? 2 : 4, X == X_F32 ? 2 : 1, OUT>(a, f.splits, s);
  if constexpr (X != X_F32) {
    if (f.bt == 128) return launch<X, 128, 128, 2, 2, OUT>(a, f.splits, s);
    return launch<X, 256, 256, 4, 2, OUT>(a, f.splits, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_q4_tiles(const LinearArgs& a, int x_dtype, int out_dtype, hipStream_t s) {
  const Form f = form_of(a.T, x_dtype, a.M, a.K);
  const bool bf16 = out_dtype == SSM_BF16;
  if (x_dtype == X_F32) return bf16 ? launch_form<X_F32, bf16_t>(a, f, s) : launch_form<X_F32, float>(a, f, s);
  if (x_dtype == X_BF16) return bf16 ? launch_form<X_BF16, bf16_t>(a, f, s) : launch_form<X_BF16, float>(a, f, s);
  return bf16 ? launch_form<X_E4M3, bf16_t>(a, f, s) : launch_form<X_WIDE, float>(a, f, s);
}

int q4_tiles_splits(int64_t T, int x_dtype, int64_t M, int64_t K) { return form_of(T, x_dtype, M, K).splits; }

}  // namespace block
}  // namespace ssm

extern "C" {

size_t ssm_q4_linear_workspace_bytes(int64_t tokens, int32_t x_dtype, int64_t out_features, int64_t in_features) {
  using namespace ssm::block;
  if (tokens < 1 || tokens >= MAX_TOKENS || !q4_sizes(out_features, in_features)) return 0;
  if (x_dtype != SSM_F32 && x_dtype != SSM_BF16 && x_dtype != SSM_E4M3) return 0;
  if (tokens <= ROWS_MAX_TOKENS || tokens * out_features > MAX_OUTPUTS) return 0;
  const int splits = q4_tiles_splits(tokens, x_dtype, out_features, in_features);
  return splits > 1 ? (size_t)splits * tokens * ((out_features + 3) / 4 * 4) * 4 : 0;
}

int ssm_q4_linear(int64_t tokens, int32_t x_dtype, int32_t out_dtype, const ssm_rows* x, const float* x_scale,
                  const ssm_q4_weight* q, const ssm_rows* out, void* workspace, size_t workspace_bytes, void* stream) {
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
  const size_t need = ssm_q4_linear_workspace_bytes(T, x_dtype, M, K);
  if (need && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return SSM_ERR_ALIGN;
  const Span so = rows_span(out, T, M, os), sw = span(workspace, (int64_t)need);
  const Span ins[3] = {codes_span(q), scales_span(q), span(x_scale, x_scale ? T * 4 : 0)};
  for (const Span& i : ins)
    if (overlaps(so, i) || overlaps(sw, i)) return SSM_ERR_ALIAS;
  if (!writable(out, T, M) || overlaps(so, sw) || overlaps(sw, rows_span(x, T, K, es)) || rows_overlap(out, M, os, x, K, es, T))
    return SSM_ERR_ALIAS;
  LinearArgs a = {};
  a.x = rows_of(x, es);
  a.out = rows_of(out, os);
  a.codes = static_cast<const char*>(q->codes);
  a.scales = static_cast<const char*>(q->scales);
  a.x_scale = x_scale;
  a.partial = static_cast<float*>(workspace);
  a.T = T;
  a.M = M;
  a.K = K;
  a.kt = (K + 127) / 128;
  a.k4 = (K + 511) / 512;
  a.mt = (M + 15) / 16;
  a.Mp = (M + 3) / 4 * 4;
  a.wide = aligned(out->data, 16) && out->stride * os % 16 == 0;
  const hipStream_t s = ready(stream);
  const hipError_t e = T <= ROWS_MAX_TOKENS ? launch_q4_rows(a, x_dtype, out_dtype, s)
                                            : launch_q4_tiles(a, x_dtype, out_dtype, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

}  // extern "C"
