// ssm_attn_decode.hip -- ssm_attn_decode_step of include/ssm_attn.h: one query token per sequence
// against the paged key/value cache.
//
// The cache is read once, and that bounds it.  The query heads of a key head (up to 16 at a time) are
// the columns of 16x16 matrix products, so a key is read once for all of them: S^T = K Q^T, then
// O^T = V^T P^T with the softmax's running maximum and sum.
//
// A wave works on 32 keys at a time, straight from memory to registers:
//   K  row m of score tile t is key 8 (m / 4) + 4 t + m % 4 of the 32, which leaves lane quarter w with
//      the weights of keys 8 w .. 8 w + 7 in order, as the second product's right operand wants them.  The
//      channels of a product may come in any order if Q's do too, so a lane reads whole 16-byte pieces.
//   V  the second product's left operand needs one channel's keys along a lane's registers.  Quarter w
//      reads its 8 keys, lane m of it VE neighbouring channels of each, and the 8 x VE block is turned in
//      registers while it is widened; tile c of the output then is channels m VE + c, and a
//      lane ends with 4 VE neighbouring channels of one head.
// All of a step's loads are issued before its first product, and are hidden by the other waves of a SIMD: three of
// them up to head_dim 128, with registers for one set of keys each, measured better than two that load 32 keys ahead
// (64 sequences of up to 8192 int8 tokens, 8 key heads of 128: 122 us, 4.6 TB/s, against 132); two above (32 sequences,
// 4 key heads of 256: 45 us against 76 with one); fewer in fp32, whose keys or parts of q take the registers.
// The page numbers are read a step ahead, by the scalar unit.
//
// 8-bit codes are exact in bf16, so fp32 calls multiply them as bf16 too: q and the weights are split into three bf16,
// x = h + m + l to 2^-27 of x (each the remainder of the last, rounded; |x| up to 2^127), and the three products take a fifth of the
// time of the fp32 matrix instruction.  A cache of fp32 is multiplied in fp32.
//
// The long axis is split into chunks, one workgroup each; its waves take 32 keys in turn and join their
// results in LDS.  With more than one chunk the partial results (maximum, sum, unnormalised output, fp32)
// are joined by a second kernel.  Both joins add in a fixed order.
#include "ssm_attn.h"

namespace ssm {
namespace attn {
namespace {

constexpr int STEP = 32;  // keys of a wave's step
constexpr int COLS = 16;  // query heads of a workgroup
constexpr int NW = 4;     // waves of a workgroup

struct DecodeArgs {
  View q, out;
  float* lse;
  Cache c;
  const int32_t* table;
  const int32_t* lens;
  int64_t W;  // table width
  int B, Hq, G, groups;  // groups: 16-head groups of a key head
  int chunks;            // most chunks of a sequence
  float scale_log2;
  float* po;  // [B, Hq, chunks, D]
  float* ml;  // [B, Hq, chunks, 2]: maximum (of scores * log2 e), sum
};

constexpr int MIN_SHARE = 8;   // steps of a chunk, at least: two for each wave

// Tables that no kernel writes, as constant memory: entries that a whole wave shares are read by the scalar unit, whose
// loads do not wait for the vector loads of keys and values.
typedef const __attribute__((address_space(4))) int32_t* ConstInts;
__device__ __forceinline__ ConstInts constant(const int32_t* p) { return (ConstInts)(uintptr_t)p; }

__device__ __forceinline__ int sequence_length(const DecodeArgs& a, int b) {
  const int64_t cap = a.W << a.c.page_shift;
  const int64_t n = constant(a.lens)[b];
  return (int)(n < 0 ? 0 : n > cap ? cap : n);
}

// Steps of each of a sequence's chunks: equal shares, but no smaller ones than MIN_SHARE.
__device__ __forceinline__ int share_of(const DecodeArgs& a, int steps) {
  return max((steps + a.chunks - 1) / a.chunks, MIN_SHARE);
}

// Code j of a word as fp32.
template <int KV>
__device__ __forceinline__ float widen_one(unsigned w, int j) {
  if constexpr (KV == SSM_KV_I8) return (float)(int8_t)(w >> (8 * j));
  const auto x = j < 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false) : __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return x[j & 1];
}

// Codes 2 p and 2 p + 1 of a word as bf16 (exact: an int8 or e4m3 value has at most 8 significant bits).
template <int KV>
__device__ __forceinline__ unsigned widen_pair(unsigned w, int p) {
  if constexpr (KV == SSM_KV_I8) return pack_bf16(widen_one<KV>(w, 2 * p), widen_one<KV>(w, 2 * p + 1));
  return p == 0 ? __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false))
                : __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
}

// Two values rounded to bf16, and what that leaves of them (exact).
__device__ __forceinline__ unsigned take_bf16(float& x0, float& x1) {
  const unsigned w = pack_bf16(x0, x1);
  x0 -= __uint_as_float(w << 16);
  x1 -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}

// Element c of one channel piece as fp32: V words w of VE elements of CS bytes.
template <int KV, int CS>
__device__ __forceinline__ float element_f32(const unsigned* w, int c) {
  if constexpr (CS == 4) return __uint_as_float(w[c]);
  else return widen_one<KV>(w[c / 4], c % 4);
}

__device__ __forceinline__ float quarters_max(float x) {  // over the lanes with the same lane & 15
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float quarters_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <int BYTES>
__device__ __forceinline__ void load_words(unsigned* w, const char* p) {
  if constexpr (BYTES == 16) {
    const u32x4 x = *reinterpret_cast<const u32x4_a4*>(p);
    w[0] = x[0], w[1] = x[1], w[2] = x[2], w[3] = x[3];
  } else if constexpr (BYTES == 8) {
    const u32x2 x = *reinterpret_cast<const u32x2_a4*>(p);
    w[0] = x[0], w[1] = x[1];
  } else {
    w[0] = *reinterpret_cast<const unsigned*>(p);
  }
}

// Waves of a SIMD.  Measured on both sides: bf16 (three and two, above), and codes in fp32 past 192 channels.  The others follow
// from the registers of a step and have no figures of one wave more or less; 129 to 192 channels of codes in fp32 spill 14
// registers with two waves, past 192 channels an unquantised cache spills 12 (bf16) and 28 (fp32).
constexpr int waves_of(bool bf16, bool codes, int DP) {
  if (bf16) return DP > 128 ? 2 : 3;
  if (codes) return DP > 192 ? 1 : DP > 64 ? 2 : 3;  // 59 sequences of 818 keys of 256: 37 us, 46 with two
  return DP > 128 ? 1 : 2;
}

// A workgroup is one (chunk, 16 heads of a key head, sequence).
template <typename IO, int KV, int DP>
__global__ __launch_bounds__(NW * 64, waves_of(sizeof(IO) == 2, KV != SSM_KV_IO, DP)) void attn_decode(DecodeArgs a) {
  constexpr bool BF = sizeof(IO) == 2, CODES = KV != SSM_KV_IO;
  constexpr int CS = CODES ? 1 : sizeof(IO);
  constexpr int QPARTS = BF ? 1 : 3, WPARTS = BF ? 2 : 3;  // bf16 that make one value of q and one weight
  // K: pieces of KB bytes; 16, but 8 of 8-bit codes where a row may be that short
  constexpr int KB = CS == 1 && DP == 64 ? 8 : 16, KE = KB / CS, NK = DP / (4 * KE), KW = KB / 4;
  // V: VE channels of a lane, NB blocks of 16 VE channels
  constexpr int VE = CS == 4 || DP % 128 ? 4 : 8, NB = DP / (16 * VE), VW = VE * CS / 4;
  __shared__ float wml[NW][COLS][2];
  extern __shared__ __attribute__((aligned(16))) float wo[];  // [NW][heads][16 VE]
  const int lane = threadIdx.x & 63, col = lane & 15, w4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = a.c.D, row_bytes = D * CS, page_mask = (1 << a.c.page_shift) - 1;
  const int pages = (int)(a.c.slots >> a.c.page_shift);

  const int chunk = blockIdx.x, kh = blockIdx.y / a.groups;
  const int g0 = (blockIdx.y - kh * a.groups) * COLS, ng = min(a.G - g0, COLS);

  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    const int len = sequence_length(a, b), steps = (len + STEP - 1) / STEP, share = share_of(a, steps);
    const int s_end = min(chunk * (int64_t)share + share, (int64_t)steps);
    if (chunk > 0 && chunk * (int64_t)share >= steps) continue;

    const int head = kh * a.G + g0 + min(col, ng - 1);
    const char* qp = a.q.p + (int64_t)b * a.q.ts + (int64_t)head * a.q.hs;
    // Q in the order of K's pieces.  Where a row ends, a lane reads an earlier piece of it against zeros.
    int koff[NK];
    unsigned qf[NK][BF || CODES ? KE / 2 * QPARTS : KE];  // bf16 by eights of channels, the parts of an eight one after another
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int e = (4 * i + w4) * KE;
      koff[i] = (e + KE <= D ? e : e < D ? D - KE : 0) * CS;
      constexpr int QE = BF ? 8 : 4;  // elements of a 16-byte read of q
#pragma unroll
      for (int h = 0; h < KE / QE; ++h) {
        const int at = koff[i] / CS + h * QE;
        u32x4 x = {0, 0, 0, 0};
        if (at >= e && at < D) x = *reinterpret_cast<const u32x4*>(qp + at * (int)sizeof(IO));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BF || !CODES) qf[i][4 * h + j] = x[j];
        }
        if constexpr (!BF && CODES) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float f0 = __uint_as_float(x[2 * j]), f1 = __uint_as_float(x[2 * j + 1]);
#pragma unroll
            for (int part = 0; part < QPARTS; ++part)
              qf[i][(h / 2 * QPARTS + part) * 4 + h % 2 * 2 + j] = take_bf16(f0, f1);
          }
        }
      }
    }
    int voff[NB];  // channels past the row's end are made of its first ones and not stored
#pragma unroll
    for (int n = 0; n < NB; ++n) voff[n] = ((n * 16 + col) * VE < D ? (n * 16 + col) * VE : 0) * CS;

    f32x4 o[NB * VE] = {};
    float m = -INFINITY, l = 0.0f;
    const ConstInts table = constant(a.table) + (int64_t)b * a.W;

    struct Keys {
      unsigned k[2][NK][KW];
      unsigned v[NB][8][VW];
      f32x4 sk[2], sv[2];
    };
    // Pages of the two 16-key groups of a step (pages hold 16 tokens or more); -1 where there are no keys.
    const auto page_of = [&](int step, int group) -> int {
      const int key = step * STEP + 16 * group;
      return step < s_end && key < len ? table[key >> a.c.page_shift] : -1;
    };
    const auto load = [&](Keys& x, int step, int p0, int p1) {
      const auto row_of = [&](int page, int group) -> int64_t {  // an unseen group reads row 0
        const int key = step * STEP + 16 * group;
        return page >= 0 && page < pages ? (((int64_t)page * a.c.heads + kh) << a.c.page_shift) + (key & page_mask) : 0;
      };
      const int64_t r0 = row_of(p0, 0), r1 = row_of(p1, 1);
      // K: key 8 (m / 4) + 4 t + m % 4 lies in group m / 8
      const char* kp = a.c.k + ((col & 8 ? r1 : r0) + 8 * ((col >> 2) & 1) + (col & 3)) * row_bytes;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < NK; ++i) load_words<KB>(x.k[t][i], kp + 4 * t * row_bytes + koff[i]);
      const int64_t rv = (w4 & 2 ? r1 : r0) + 8 * (w4 & 1);
      if constexpr (KV != SSM_KV_IO) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          x.sk[t] = *reinterpret_cast<const f32x4*>(a.c.ks + rv + 4 * t);
          x.sv[t] = *reinterpret_cast<const f32x4*>(a.c.vs + rv + 4 * t);
        }
      }
      const char* vp = a.c.v + rv * row_bytes;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) load_words<VE * CS>(x.v[n][j], vp + j * row_bytes + voff[n]);
    };
    const auto work = [&](Keys& x, int step, int p0, int p1) {
      f32x4 s[2] = {};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          if constexpr (BF || CODES) {
#pragma unroll
            for (int h = 0; h < KE / 8; ++h) {
              u32x4 kf;
              if constexpr (CS == 1)
                kf = u32x4{widen_pair<KV>(x.k[t][i][2 * h], 0), widen_pair<KV>(x.k[t][i][2 * h], 1),
                           widen_pair<KV>(x.k[t][i][2 * h + 1], 0), widen_pair<KV>(x.k[t][i][2 * h + 1], 1)};
              else
                kf = u32x4{x.k[t][i][0], x.k[t][i][1], x.k[t][i][2], x.k[t][i][3]};
#pragma unroll
              for (int part = QPARTS - 1; part >= 0; --part) {  // the small ones first
                const unsigned* qh = qf[i] + (h * QPARTS + part) * 4;
                const u32x4 q = {qh[0], qh[1], qh[2], qh[3]};
                s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf),
                                                               __builtin_bit_cast(bf16x8, q), s[t], 0, 0, 0);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < KE; ++j)
              s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(element_f32<KV, CS>(x.k[t][i], j), __uint_as_float(qf[i][j]),
                                                          s[t], 0, 0, 0);
          }
        }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if constexpr (KV != SSM_KV_IO) s[t] *= x.sk[t];
        s[t] *= a.scale_log2;
      }
      const bool whole = step * STEP + STEP <= len && p0 >= 0 && p0 < pages && p1 >= 0 && p1 < pages;
      if (!whole) {  // what lies in unseen places counts for nothing, whatever it holds
        const int p = w4 & 2 ? p1 : p0, seen = p >= 0 && p < pages ? len - step * STEP - 8 * w4 : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = j < seen;
          s[j / 4][j % 4] = in ? s[j / 4][j % 4] : -INFINITY;
          if constexpr (KV != SSM_KV_IO) x.sv[j / 4][j % 4] = in ? x.sv[j / 4][j % 4] : 0.0f;
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int w = 0; w < VW; ++w) x.v[n][j][w] = in ? x.v[n][j][w] : 0u;
        }
      }
      float mx = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                       fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      mx = quarters_max(mx);
      // The subtracted maximum follows the true one only when it has grown by 2^SLACK: weights stay below
      // 2^SLACK, and the outputs are rescaled a few times in a sequence instead of at every step.
      constexpr float SLACK = 8.0f;
      if (__any(mx > m + SLACK)) {
        const float to = mx > m ? mx : m;
        const float alpha = hw_exp2(m - (to == -INFINITY ? 0.0f : to));
        m = to;
        l *= alpha;
#pragma unroll
        for (int c = 0; c < NB * VE; ++c) o[c] *= alpha;
      }
      const float mc = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = hw_exp2(s[t][i] - mc);
          l += p;  // this quarter's keys only; joined at the end
          s[t][i] = KV != SSM_KV_IO ? p * x.sv[t][i] : p;
        }
      if constexpr (BF || CODES) {
        // bf16: a weight as the sum of two (2^-17), as one alone would be as inexact as the output's own rounding.
        u32x4 pw[WPARTS];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x0 = s[j / 2][j % 2 * 2], x1 = s[j / 2][j % 2 * 2 + 1];
#pragma unroll
          for (int part = 0; part < WPARTS; ++part) pw[part][j] = take_bf16(x0, x1);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int c = 0; c < VE; c += 2) {
            u32x4 v0, v1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const unsigned* ra = x.v[n][2 * j];
              const unsigned* rb = x.v[n][2 * j + 1];
              if constexpr (KV == SSM_KV_I8) {
                v0[j] = pack_bf16(widen_one<KV>(ra[c / 4], c % 4), widen_one<KV>(rb[c / 4], c % 4));
                v1[j] = pack_bf16(widen_one<KV>(ra[c / 4], c % 4 + 1), widen_one<KV>(rb[c / 4], c % 4 + 1));
              } else {
                const unsigned wa = CS == 1 ? widen_pair<KV>(ra[c / 4], c % 4 / 2) : ra[c / 2];
                const unsigned wb = CS == 1 ? widen_pair<KV>(rb[c / 4], c % 4 / 2) : rb[c / 2];
                v0[j] = pair_lo(wa, wb);
                v1[j] = pair_hi(wa, wb);
              }
            }
            f32x4& o0 = o[n * VE + c];
            f32x4& o1 = o[n * VE + c + 1];
#pragma unroll
            for (const u32x4& p : pw) {
              const bf16x8 w = __builtin_bit_cast(bf16x8, p);
              o0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v0), w, o0, 0, 0, 0);
              o1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v1), w, o1, 0, 0, 0);
            }
          }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < VE; ++c)
              o[n * VE + c] = __builtin_amdgcn_mfma_f32_16x16x4f32(element_f32<KV, CS>(x.v[n][j], c), s[j / 4][j % 4],
                                                                   o[n * VE + c], 0, 0, 0);
      }
    };

    int step = chunk * share + wave;
    if (step < s_end) {
      int p0 = page_of(step, 0), p1 = page_of(step, 1);
      for (; step < s_end; step += NW) {
        Keys x;
        const int n0 = page_of(step + NW, 0), n1 = page_of(step + NW, 1);
        load(x, step, p0, p1);
        __builtin_amdgcn_sched_barrier(0);  // every load of the step before its first product
        work(x, step, p0, p1);
        p0 = n0, p1 = n1;
      }
    }

    // Join the waves: their outputs on one maximum, then sums in wave order.
    l = quarters_sum(l);
    __syncthreads();
    if (w4 == 0) wml[wave][col][0] = m;
    __syncthreads();
    float top = wml[0][col][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = fmaxf(top, wml[w][col][0]);
    const float f = hw_exp2(m - (top == -INFINITY ? 0.0f : top));
    if (w4 == 0) wml[wave][col][1] = l * f;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      constexpr int BC = 16 * VE;  // channels of a block
      if (n > 0) __syncthreads();
      if (col < ng) {
        float* at = wo + ((size_t)wave * ng + col) * BC + 4 * w4 * VE;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < VE; c += 4)
            *reinterpret_cast<f32x4*>(at + i * VE + c) =
                f32x4{o[n * VE + c][i], o[n * VE + c + 1][i], o[n * VE + c + 2][i], o[n * VE + c + 3][i]} * f;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < ng * (BC / 4); i += NW * 64) {
        const int g = i / (BC / 4), e = n * BC + (i - g * (BC / 4)) * 4;
        if (e >= D) continue;
        f32x4 y = {};
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          y += *reinterpret_cast<const f32x4*>(wo + ((size_t)w * ng + g) * BC + (e - n * BC));
          sum += wml[w][g][1];
        }
        const int hd = kh * a.G + g0 + g;
        if (a.chunks == 1) {
          y *= sum > 0.0f ? 1.0f / sum : 0.0f;
          char* op = a.out.p + (int64_t)b * a.out.ts + (int64_t)hd * a.out.hs;
          if constexpr (BF) *reinterpret_cast<u32x2*>(op + e * 2) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
          else *reinterpret_cast<f32x4*>(op + e * 4) = y;
        } else {
          *reinterpret_cast<f32x4*>(a.po + (((int64_t)b * a.Hq + hd) * a.chunks + chunk) * D + e) = y;
        }
        if (e == 0) {
          float hm = wml[0][g][0];
#pragma unroll
          for (int w = 1; w < NW; ++w) hm = fmaxf(hm, wml[w][g][0]);
          const int64_t at = (int64_t)b * a.Hq + hd;
          if (a.chunks > 1) {
            a.ml[2 * (at * a.chunks + chunk)] = hm;
            a.ml[2 * (at * a.chunks + chunk) + 1] = sum;
          } else if (a.lse) {
            a.lse[at] = sum > 0.0f ? (hm + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
          }
        }
      }
    }
  }
}

constexpr int MAX_CHUNKS = 1024;
constexpr int JOIN = 256;  // threads of a join

// Joins the chunks of one (sequence, head), LP * 4 of its channels: JOIN / LP slices of the chunks, each
// with a running maximum and sum of its own, then the slices in order.
template <typename IO, int LP>
__global__ __launch_bounds__(JOIN) void attn_decode_join(DecodeArgs a) {
  constexpr int S = JOIN / LP, AT_ONCE = 4;
  __shared__ float part[S][2];
  __shared__ f32x4 acc[JOIN];
  const int tid = threadIdx.x, lp = tid % LP, slice = tid / LP, D = a.c.D;
  const int e = (blockIdx.y * LP + lp) * 4;
  for (int64_t row = blockIdx.x; row < (int64_t)a.B * a.Hq; row += gridDim.x) {
    const int b = (int)(row / a.Hq), head = (int)(row - (int64_t)b * a.Hq);
    const int steps = (sequence_length(a, b) + STEP - 1) / STEP, share = share_of(a, steps);
    const int n = (steps + share - 1) / share;
    const float* ml = a.ml + row * a.chunks * 2;
    const float* po = a.po + row * a.chunks * D + (e < D ? e : 0);
    float m = -INFINITY, l = 0.0f;
    f32x4 y = {};
    for (int c0 = slice; c0 < n; c0 += AT_ONCE * S) {
      float cm[AT_ONCE], cl[AT_ONCE];
      f32x4 cy[AT_ONCE];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int c = c0 + i * S, at = c < n ? c : c0;
        cm[i] = c < n ? ml[2 * at] : -INFINITY;
        cl[i] = c < n ? ml[2 * at + 1] : 0.0f;
        cy[i] = *reinterpret_cast<const f32x4*>(po + (int64_t)at * D);
      }
      float to = m;
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) to = fmaxf(to, cm[i]);
      const float by = to == -INFINITY ? 0.0f : to, f = hw_exp2(m - by);
      y *= f;
      l *= f;
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const float w = hw_exp2(cm[i] - by);
        y += cy[i] * w;
        l += cl[i] * w;
      }
      m = to;
    }
    __syncthreads();  // the last row's use of the shared arrays is over
    if (lp == 0) part[slice][0] = m, part[slice][1] = l;
    acc[tid] = y;
    __syncthreads();
    if (slice == 0) {
#pragma unroll
      for (int i = 1; i < S; ++i) m = fmaxf(m, part[i][0]);
      const float by = m == -INFINITY ? 0.0f : m;
      y = f32x4{};
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const float w = hw_exp2(part[i][0] - by);
        y += acc[i * LP + lp] * w;
        l += part[i][1] * w;
      }
      y *= l > 0.0f ? 1.0f / l : 0.0f;
      char* op = a.out.p + (int64_t)b * a.out.ts + (int64_t)head * a.out.hs;
      if (e < D) {
        if constexpr (sizeof(IO) == 2)
          *reinterpret_cast<u32x2*>(op + e * 2) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        else
          *reinterpret_cast<f32x4*>(op + e * 4) = y;
      }
      if (a.lse && e == 0) a.lse[row] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
    }
  }
}

// Workgroups: several for each place on the chip, so that uneven lengths even out; more cost more starts than they
// even out (the same 64 sequences: 124 us with 2048, 123 with 4096, 131 with 8192, 174 with 16384).
constexpr int64_t TARGET = 4096;
constexpr int64_t MAX_GRID = int64_t(1) << 22;  // keeps a launch within 2^31 work-items

// Most chunks of a sequence, from what the host knows: the table's width, not the lengths.
int chunks_of(int64_t batch, int q_heads, const ssm_kv_cache* c, int64_t table_width) {
  const int64_t groups = (q_heads / c->kv_heads + COLS - 1) / COLS;
  const int64_t units = batch * c->kv_heads * groups, longest = table_width * c->page_size;
  int64_t n = (TARGET + units - 1) / units;
  // Up to twice the least share one chunk does, and no second launch: 5 sequences of up to 300 tokens
  // of 64 channels, unquantised, 5.8 us a call against 8.4 with two launches.
  const int64_t least = MIN_SHARE * STEP, most = longest <= 2 * least ? 1 : (longest + least - 1) / least;
  if (n > most) n = most;
  if (n > MAX_CHUNKS) n = MAX_CHUNKS;
  return (int)(n < 1 ? 1 : n);
}

template <typename IO, int KV, int DP>
hipError_t launch_dp(const DecodeArgs& a, hipStream_t s) {
  constexpr int CS = KV == SSM_KV_IO ? sizeof(IO) : 1, VE = CS == 4 || DP % 128 ? 4 : 8;
  const int ng = a.G < COLS ? a.G : COLS;
  const int heads = a.c.heads * a.groups;
  const int64_t room = MAX_GRID / ((int64_t)a.chunks * heads);  // sequences of a launch's grid
  const dim3 grid(a.chunks, heads, (unsigned)(a.B < room ? a.B : room < 1 ? 1 : room)), tb(NW * 64);
  attn_decode<IO, KV, DP><<<grid, tb, NW * ng * 16 * VE * sizeof(float), s>>>(a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.chunks > 1) {
    // Many chunks: more slices of them, and fewer channels of a workgroup.
    const int lp = a.chunks >= 64 ? 8 : 32;
    const int64_t rows = (int64_t)a.B * a.Hq, jroom = MAX_GRID / 8;
    const dim3 jgrid((unsigned)(rows < jroom ? rows : jroom), (a.c.D + 4 * lp - 1) / (4 * lp));
    if (lp == 8) attn_decode_join<IO, 8><<<jgrid, dim3(JOIN), 0, s>>>(a);
    else attn_decode_join<IO, 32><<<jgrid, dim3(JOIN), 0, s>>>(a);
    e = hipGetLastError();
  }
  return e;
}

template <typename IO, int KV>
hipError_t launch_kv(const DecodeArgs& a, hipStream_t s) {
  if (a.c.D <= 64) return launch_dp<IO, KV, 64>(a, s);
  if (a.c.D <= 128) return launch_dp<IO, KV, 128>(a, s);
  if (a.c.D <= 192) return launch_dp<IO, KV, 192>(a, s);
  return launch_dp<IO, KV, 256>(a, s);
}

template <typename IO>
hipError_t launch_decode_attn(const DecodeArgs& a, int kv, hipStream_t s) {
  if (kv == SSM_KV_IO) return launch_kv<IO, SSM_KV_IO>(a, s);
  if (kv == SSM_KV_I8) return launch_kv<IO, SSM_KV_I8>(a, s);
  return launch_kv<IO, SSM_KV_E4M3>(a, s);
}

// Sizes of a decode call.
int check_decode_sizes(int64_t batch, int32_t q_heads, const ssm_kv_cache* c, int64_t table_width) {
  if (const int st = check_heads(q_heads, c->head_dim)) return st;
  if (const int st = check_heads(c->kv_heads, c->head_dim)) return st;
  if (q_heads % c->kv_heads) return SSM_ERR_SHAPE;
  if (batch < 1 || batch > SSM_ATTN_MAX_BATCH) return SSM_ERR_SHAPE;
  if (c->page_size < SSM_KV_MIN_PAGE || c->page_size > SSM_KV_MAX_PAGE || (c->page_size & (c->page_size - 1)))
    return SSM_ERR_SHAPE;
  // a sequence's keys, rounded up to steps and shares, stay below 2^31
  if (table_width < 1 || table_width > ((int64_t)INT32_MAX - (1 << 20)) / c->page_size) return SSM_ERR_SHAPE;
  return SSM_OK;
}

}  // namespace
}  // namespace attn
}  // namespace ssm

extern "C" {

size_t ssm_attn_decode_workspace_bytes(int64_t batch, int32_t q_heads, const ssm_kv_cache* cache,
                                       int64_t table_width) {
  using namespace ssm::attn;
  if (!cache || check_decode_sizes(batch, q_heads, cache, table_width) != SSM_OK) return 0;
  const int n = chunks_of(batch, q_heads, cache, table_width);
  return n == 1 ? 0 : (size_t)batch * q_heads * n * (cache->head_dim + 2) * sizeof(float);
}

int ssm_attn_decode_step(int64_t batch, int32_t q_heads, int32_t io_dtype, float scale, const ssm_kv_cache* cache,
                         const ssm_view* q, const int32_t* table, int64_t table_width, const int32_t* lens,
                         const ssm_view* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ssm::attn;
  int64_t es, cs;
  if (const int st = check_io(io_dtype, &es)) return st;
  if (const int st = check_cache(cache, es, &cs)) return st;
  if (const int st = check_decode_sizes(batch, q_heads, cache, table_width)) return st;
  if (!isfinite(scale) || !(scale > 0.0f)) return SSM_ERR_SHAPE;
  if (!table || !lens) return SSM_ERR_NULL;
  if (const int st = check_view(q, es)) return st;
  if (const int st = check_view(out, es)) return st;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4)) return SSM_ERR_ALIGN;
  const size_t need = ssm_attn_decode_workspace_bytes(batch, q_heads, cache, table_width);
  if (need && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return SSM_ERR_ALIGN;
  const int64_t B = batch, D = cache->head_dim, H = q_heads;
  if (!writable(out, B, H, D) || views_overlap(out, B, H, q, B, H, D, es)) return SSM_ERR_ALIAS;
  const Span so = view_span(out, B, H, D, es), sl = span(lse, lse ? B * H * 4 : 0), sw = span(workspace, (int64_t)need);
  const Span ins[3] = {view_span(q, B, H, D, es), span(table, B * table_width * 4), span(lens, B * 4)};
  const CacheSpans spans = cache_spans(cache, cs);
  if (overlaps(so, sl) || overlaps(so, sw) || overlaps(sl, sw)) return SSM_ERR_ALIAS;
  if (overlaps(so, ins[1]) || overlaps(so, ins[2])) return SSM_ERR_ALIAS;
  for (const Span& s : ins)
    if (overlaps(sl, s) || overlaps(sw, s)) return SSM_ERR_ALIAS;
  if (cache_overlaps(spans, so) || cache_overlaps(spans, sl) || cache_overlaps(spans, sw)) return SSM_ERR_ALIAS;
  DecodeArgs a = {};
  a.q = bytes_view(q, es);
  a.out = bytes_view(out, es);
  a.lse = lse;
  a.c = cache_of(cache);
  a.table = table;
  a.lens = lens;
  a.W = table_width;
  a.B = (int)batch;
  a.Hq = q_heads;
  a.G = q_heads / cache->kv_heads;
  a.groups = (a.G + COLS - 1) / COLS;
  a.chunks = chunks_of(batch, q_heads, cache, table_width);
  a.scale_log2 = scale * 1.4426950408889634f;
  if (!isfinite(a.scale_log2) || !(a.scale_log2 > 0.0f)) return SSM_ERR_SHAPE;
  a.po = static_cast<float*>(workspace);
  a.ml = a.po + (int64_t)batch * q_heads * a.chunks * cache->head_dim;
  const hipStream_t s = ready(stream);
  const hipError_t e = io_dtype == SSM_BF16 ? launch_decode_attn<ssm::bf16_t>(a, cache->kv_dtype, s)
                                            : launch_decode_attn<float>(a, cache->kv_dtype, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

}  // extern "C"
