// ssm_attn_split.hip -- prompt attention (ssm_attn_prefill of include/ssm_attn.h) with the keys split over a
// workgroup's waves: all of fp32, and bf16 calls of few rows.
//
// A workgroup has 32 rows; its waves take 32 keys in turn and join their results at the end, so that few rows still
// fill the chip and a row's way along the keys is a fraction of their number.  A wave reads its operands straight from
// memory, no LDS.  Scores are computed transposed, S^T = K Q^T, with 32x32 matrix instructions: a lane holds 16 scores of
// ONE row (column lane & 31), the other 16 being in lane ^ 32, in the order that the right operand of
// O^T = V^T P^T wants.  K's channels may come in any order if Q's do too: 16-byte reads of both.  Lane m of V's
// operand holds VE neighbouring channels of its keys, for VE output tiles (bf16: turned in registers into each
// channel's keys).  A step's V is loaded while its scores are computed, the next step's K while its output is.
// Past a sequence's end keys are read as zeros (the buffer's bounds) and masked.
//
// fp32 operands are split into three bf16 each, x = h + m + l to 2^-27 of x (each the remainder of the last,
// rounded), and multiplied as hh + hm + mh + mm + hl + lh: what is left out, ml + lm + ll, is below 2^-25 of a product,
// half of what one fp32 rounding may be.  Six bf16 products take 3/8 of the time of the fp32 matrix instruction on the
// same numbers (a sixteenth of bf16's rate).
#include "ssm_attn_prefill.h"

namespace ssm {
namespace attn {
namespace {

typedef unsigned u32;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_view(const char* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, bytes, 0x00020000);
}

// 16-byte pieces 2 i + half of a lane's row (at `row`).  Past the row's end a piece of it that lies within: it meets zeros
// of Q.  Both pieces of an i lie within or neither does, but for the last one of bf16 rows of 16 n + 8 values.
template <int NQ, int ES>
__device__ __forceinline__ void load_k(u32x4* k, const char* p, int bytes, int row, int half, int row_bytes) {
  const __amdgpu_buffer_rsrc_t r = rows_view(p, bytes);
  const int at = row + (ES == 4 || row_bytes > 16 ? half * 16 : 0);
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const bool edge = ES == 2 && i * 32 < row_bytes && i * 32 + 16 == row_bytes;  // the upper half's is past the end
    const int v = edge ? row + (half ? 0 : i * 32) : at, s = !edge && i * 32 < row_bytes ? i * 32 : 0;
    k[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, v, s, 0));
  }
}

// VW words of 16 keys (the ones of score i in a lane's order) of each of NB blocks.
template <int NB, int VW>
__device__ __forceinline__ void load_v(u32 (*v)[NB][VW], const char* p, int bytes, const int* at, int ts) {
  const __amdgpu_buffer_rsrc_t r = rows_view(p, bytes);
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int row = (8 * (i / 4) + i % 4) * ts;
      if constexpr (VW == 4) {
        const u32x4 t = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at[n], row, 0));
        v[i][n][0] = t[0], v[i][n][1] = t[1], v[i][n][2] = t[2], v[i][n][3] = t[3];
      } else if constexpr (VW == 2) {
        const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at[n], row, 0));
        v[i][n][0] = t[0], v[i][n][1] = t[1];
      } else {
        v[i][n][0] = __builtin_amdgcn_raw_buffer_load_b32(r, at[n], row, 0);
      }
    }
}

struct Three {
  bf16x8 h, m, l;
};
__device__ __forceinline__ Three split(const float (&x)[8]) {
  u32x4 t[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const u32 w = pack_bf16(a, b);
      t[j][i] = w;
      a -= __uint_as_float(w << 16), b -= __uint_as_float(w & 0xFFFF0000u);  // exact
    }
  }
  return Three{__builtin_bit_cast(bf16x8, t[0]), __builtin_bit_cast(bf16x8, t[1]), __builtin_bit_cast(bf16x8, t[2])};
}
__device__ __forceinline__ Three split(u32x4 a, u32x4 b) {
  const float x[8] = {__uint_as_float(a[0]), __uint_as_float(a[1]), __uint_as_float(a[2]), __uint_as_float(a[3]),
                      __uint_as_float(b[0]), __uint_as_float(b[1]), __uint_as_float(b[2]), __uint_as_float(b[3])};
  return split(x);
}
// The small terms first.
__device__ __forceinline__ f32x16 product(const Three& a, const Three& b, f32x16 c) {
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.l, b.h, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.h, b.l, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.m, b.m, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.m, b.h, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.h, b.m, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.h, b.h, c, 0, 0, 0);
}

template <typename IO, int DP, int NW>
__global__ __launch_bounds__(NW * 64, NW / 4) void attn_split(PrefillArgs a) {
  constexpr bool BF = sizeof(IO) == 2;
  constexpr int ES = sizeof(IO), QT = 32, NQ = DP * ES / 32;
  // Channels of a lane, blocks of 32 VE, words of a lane's channels of one key
  constexpr int VE = DP % 128 == 0 ? 4 : DP % 64 == 0 ? 2 : 1, NB = DP / (32 * VE), VW = VE * ES / 4;
  static_assert(VW >= 1, "bf16 takes two channels at a time");
  constexpr bool QREG = BF || DP <= 64;  // Q in registers beside a step's K, V and output, else in LDS (fp32's is three parts)
  __shared__ float wml[NW][32][2];
  __shared__ __attribute__((aligned(16))) float wo[NW][32][32 * VE + 4];
  __shared__ __attribute__((aligned(16))) u32x4 ql[QREG ? 1 : BF ? NQ : NQ / 2 * 3][64];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kts = (int)a.k.ts, vts = (int)a.v.ts, row_bytes = a.D * ES;
  int vo[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) vo[n] = 4 * half * vts + ((n * 32 + col) * VE < a.D ? (n * 32 + col) * VE * ES : 0);

  const int h = blockIdx.x;
  Work w;
  for (int64_t idx = blockIdx.y; find_tile(a, QT, idx, w); idx += gridDim.y) {
    const int tile = w.tiles - 1 - w.tile;  // causal: the tiles with the most keys first
    const int q0 = w.q0, lq = w.lq, k0 = w.k0, lk = w.lk;
    const int rows = lq * a.G, r0 = tile * QT;
    const int r = r0 + col, rc = min(r, rows - 1);
    const int tok = by_group(a, rc), g = rc - tok * a.G;
    const auto seen_by = [&](int token) { return seen_of(a, lq, lk, token); };
    const int seen = seen_by(tok);
    const int first = __builtin_amdgcn_readfirstlane(seen_by(by_group(a, r0)));
    const int last = __builtin_amdgcn_readfirstlane(seen_by(by_group(a, min(r0 + 31, rows - 1))));

    const char* kp = a.k.p + (int64_t)k0 * a.k.ts + (int64_t)h * a.k.hs;
    const char* vp = a.v.p + (int64_t)k0 * a.v.ts + (int64_t)h * a.v.hs;
    const auto span = [&](int j0, int ts) { return (min(lk - j0, 32) - 1) * ts + row_bytes; };  // bytes of a step's rows
    u32x4 kx[NQ];
    int j0 = wave * 32;
    if (j0 < last) load_k<NQ, ES>(kx, kp + (int64_t)j0 * a.k.ts, span(j0, kts), col * kts, half, row_bytes);
    const char* qp = a.q.p + (int64_t)(q0 + tok) * a.q.ts + (int64_t)(h * a.G + g) * a.q.hs;
    const auto read_q = [&](int i) {
      const int e = (2 * i + half) * 16;
      return e < row_bytes ? *reinterpret_cast<const u32x4*>(qp + e) : u32x4{0, 0, 0, 0};
    };
    // Q: pieces as K's; of fp32, two pieces at a time in three parts
    constexpr int NP = BF ? NQ : NQ / 2, PARTS = BF ? 1 : 3;
    bf16x8 qf[QREG ? NP : 1][PARTS];
    if constexpr (!QREG) __syncthreads();
#pragma unroll
    for (int i = QREG ? 0 : wave; i < NP; i += QREG ? 1 : NW) {
      bf16x8 x[PARTS];
      if constexpr (BF) {
        x[0] = __builtin_bit_cast(bf16x8, read_q(i));
      } else {
        const Three t = split(read_q(2 * i), read_q(2 * i + 1));
        x[0] = t.h, x[1] = t.m, x[2] = t.l;
      }
#pragma unroll
      for (int j = 0; j < PARTS; ++j) {
        if constexpr (QREG) qf[i][j] = x[j];
        else ql[i * PARTS + j][lane] = __builtin_bit_cast(u32x4, x[j]);
      }
    }
    if constexpr (!QREG) __syncthreads();
    const auto part = [&](int i, int j) {
      return QREG ? qf[QREG ? i : 0][j] : __builtin_bit_cast(bf16x8, ql[QREG ? 0 : i * PARTS + j][lane]);
    };
    f32x16 o[NB * VE] = {};
    float m = -INFINITY, l = 0.0f;

    for (; j0 < last; j0 += NW * 32) {
      u32 vx[16][NB][VW];
      load_v<NB, VW>(vx, vp + (int64_t)j0 * a.v.ts, span(j0, vts), vo, vts);
      __builtin_amdgcn_sched_barrier(0);
      f32x16 s = {};
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if constexpr (BF)
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kx[i]), part(i, 0), s, 0, 0, 0);
        else
          s = product(split(kx[2 * i], kx[2 * i + 1]), Three{part(i, 0), part(i, 1), part(i, 2)}, s);
      }
      __builtin_amdgcn_sched_barrier(0);
      const int jn = j0 + NW * 32;
      if (jn < last) load_k<NQ, ES>(kx, kp + (int64_t)jn * a.k.ts, span(jn, kts), col * kts, half, row_bytes);
      __builtin_amdgcn_sched_barrier(0);
      if (j0 + 32 > first) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = j0 + 8 * (i / 4) + 4 * half + i % 4 < seen ? s[i] : -INFINITY;
      }
      float mx = m;
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[i] * a.scale_log2);
      mx = half_max(mx);
      const float mc = mx == -INFINITY ? 0.0f : mx, alpha = hw_exp2(m - mc);
      m = mx;
      l *= alpha;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = hw_exp2(fmaf(s[i], a.scale_log2, -mc));
        l += s[i];
      }
#pragma unroll
      for (int c = 0; c < NB * VE; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[c][i] *= alpha;
#pragma unroll
      for (int t = 0; t < 2; ++t) {  // 16 keys: this half holds keys 4 half + {0..3, 8..11} of them
        if constexpr (BF) {
          u32x4 pf;  // weights rounded to bf16 once, as in attn_prefill: a call's form does not change its precision
#pragma unroll
          for (int i = 0; i < 4; ++i) pf[i] = pack_bf16(s[8 * t + 2 * i], s[8 * t + 2 * i + 1]);
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < VE; ++c) {
              u32x4 vf;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const u32 x = vx[8 * t + 2 * i][n][c / 2], y = vx[8 * t + 2 * i + 1][n][c / 2];
                vf[i] = c % 2 == 0 ? pair_lo(x, y) : pair_hi(x, y);
              }
              f32x16& oc = o[n * VE + c];
              oc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf), __builtin_bit_cast(bf16x8, pf), oc,
                                                           0, 0, 0);
            }
        } else {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = s[8 * t + i];
          const Three p = split(x);
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < VE; ++c) {
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(vx[8 * t + i][n][c]);
              o[n * VE + c] = product(split(x), p, o[n * VE + c]);
            }
        }
      }
    }

    // Join the waves: their outputs on one maximum, then sums in wave order.
    l = half_sum(l);
    __syncthreads();
    if (half == 0) wml[wave][col][0] = m;
    __syncthreads();
    float top = wml[0][col][0];
#pragma unroll
    for (int x = 1; x < NW; ++x) top = fmaxf(top, wml[x][col][0]);
    const float f = hw_exp2(m - (top == -INFINITY ? 0.0f : top));
    if (half == 0) wml[wave][col][1] = l * f;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      constexpr int BC = 32 * VE;
      if (n > 0) __syncthreads();
      // rows of the product: channel lane m of V = 8 (i / 4) + 4 half + i % 4
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int c = 0; c < VE; ++c) wo[wave][col][(8 * (i / 4) + 4 * half + i % 4) * VE + c] = o[n * VE + c][i] * f;
      __syncthreads();
      for (int i = threadIdx.x; i < 32 * (BC / 4); i += NW * 64) {
        const int row = i / (BC / 4), e = (i - row * (BC / 4)) * 4, rr = r0 + row;
        if (n * BC + e >= a.D || rr >= rows) continue;
        f32x4 y = {};
        float sum = 0.0f, hm = -INFINITY;
#pragma unroll
        for (int x = 0; x < NW; ++x) {
          y += *reinterpret_cast<const f32x4*>(&wo[x][row][e]);
          sum += wml[x][row][1];
          hm = fmaxf(hm, wml[x][row][0]);
        }
        y *= sum > 0.0f ? 1.0f / sum : 0.0f;
        const int t = by_group(a, rr), head = h * a.G + rr - t * a.G;
        char* op = a.out.p + (int64_t)(q0 + t) * a.out.ts + (int64_t)head * a.out.hs + (n * BC + e) * ES;
        if constexpr (BF) *reinterpret_cast<u32x2*>(op) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        else *reinterpret_cast<f32x4*>(op) = y;
        if (a.lse && n == 0 && e == 0)
          a.lse[(int64_t)(q0 + t) * a.Hq + head] = sum > 0.0f ? (hm + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
      }
    }
  }
}

// Waves of a workgroup: eight, two a SIMD, where registers allow (fp32 rows of 96 and 128 channels with Q in LDS: four waves
// to eight, 1000 tokens of 8 and 2 heads 39.6 to 36.7 us, four prompts of up to 1000 of 32 and 8 195 to 178).  fp32 rows of 64 channels fit twice on a CU with four: eight gain
// 10% while the tiles leave CUs half empty, and lose 25 to 60% after.
template <typename IO, int DP>
void launch_dp(const PrefillArgs& a, hipStream_t s) {
  constexpr bool BF = sizeof(IO) == 2;
  if constexpr (DP <= 128) {
    if (BF || DP > 64 || tiles_at_most(a, 32) * a.Hkv <= 512) {
      attn_split<IO, DP, 8><<<tiles_grid(a, 32, INT32_MAX), dim3(512), 0, s>>>(a);
      return;
    }
  }
  if constexpr (DP > 128 || (!BF && DP <= 64)) attn_split<IO, DP, 4><<<tiles_grid(a, 32, INT32_MAX), dim3(256), 0, s>>>(a);
}

}  // namespace

void launch_split(const PrefillArgs& a, bool bf16, hipStream_t s) {
  if (a.D <= 64) bf16 ? launch_dp<bf16_t, 64>(a, s) : launch_dp<float, 64>(a, s);
  else if (a.D <= 96 && !bf16) launch_dp<float, 96>(a, s);
  else if (a.D <= 128) bf16 ? launch_dp<bf16_t, 128>(a, s) : launch_dp<float, 128>(a, s);
  else if (a.D <= 192) bf16 ? launch_dp<bf16_t, 192>(a, s) : launch_dp<float, 192>(a, s);
  else bf16 ? launch_dp<bf16_t, 256>(a, s) : launch_dp<float, 256>(a, s);
}

}  // namespace attn
}  // namespace ssm
