// ssm_attn_prefill.hip -- ssm_attn_prefill of include/ssm_attn.h: softmax attention over packed
// prompts, one pass over the keys with the running maximum and sum of each row's softmax.
//
// Rows.  The query heads that share a key head are packed into the rows of a tile: row r of a sequence
// is token r / G, query head kv_head * G + r % G (G = query heads per key head).  A key tile is then
// read once for all G heads, and a short sequence fills a tile G times better.
//
// Products.  Scores are computed transposed, S^T = K Q^T, with 32x32 matrix instructions: a lane then
// holds scores of ONE row (column lane & 31), 16 keys of every 32, the other 16 being in lane ^ 32.
// Row maxima and sums are therefore taken inside a lane, with a single exchange of the two halves, and
// the weights are already in the layout of the second product's right operand, O^T = V^T P^T: the
// order of the keys inside a product is free as long as V is read in the same order.  V's operand needs
// keys along a lane's registers, and V is stored with channels along a row: bf16 uses the LDS read that
// transposes 16-bit elements.
#include "ssm_attn.h"

namespace ssm {
namespace attn {
namespace {

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
};

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

// The sequence and tile that hold tile `idx` of the packed batch (false past the end).  Each wave finds
// it by itself: 64 sequences at a time, a prefix sum of their tile counts over the lanes.
__device__ __forceinline__ bool find_tile(const PrefillArgs& a, int QT, int64_t idx, Work& w) {
  const int lane = threadIdx.x & 63;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int bb = b0 + lane;
    int q0 = 0, lq = 0, k0 = 0, lk = 0;
    if (bb < a.B) {
      q0 = min(max(a.cu_q[bb], 0), a.Tq);
      lq = max(min(a.cu_q[bb + 1], a.Tq) - q0, 0);
      k0 = min(max(a.cu_k[bb], 0), a.Tk);
      lk = max(min(a.cu_k[bb + 1], a.Tk) - k0, 0);
    }
    const int n = (int)(((int64_t)lq * a.G + QT - 1) / QT), incl = wave_scan(n);
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (idx < base + total) {
      const int want = (int)(idx - base);
      const int at = __ffsll((unsigned long long)__ballot(incl > want)) - 1;
      w.tiles = __builtin_amdgcn_readlane(n, at);
      w.tile = want - (__builtin_amdgcn_readlane(incl, at) - w.tiles);
      w.q0 = __builtin_amdgcn_readlane(q0, at);
      w.lq = __builtin_amdgcn_readlane(lq, at);
      w.k0 = __builtin_amdgcn_readlane(k0, at);
      w.lk = __builtin_amdgcn_readlane(lk, at);
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

// A key tile in LDS: rows of CH 16-byte chunks, whose places in the row are exchanged by the row
// number so that lanes reading one chunk of neighbouring rows use different banks.
template <int DP>
struct Tile {
  static constexpr int PITCH = DP == 96 ? 128 : DP;  // elements of a row: the exchange works on 8 or 16 chunks
  static constexpr int CH = PITCH / 8;
  // Sixteen chunks fill the banks once.  Rows of 16 n chunks: any 16 rows' chunks in 16 places.  Rows of 16 n + 8
  // start in the two halves of the banks in turn: 8 places for each half.
  __device__ static int k_swap(int row) { return CH % 16 == 0 ? row & 15 : (row >> 1) & 7; }
  // 32 lanes read 4 chunks of 4 rows each.
  __device__ static int v_swap(int row) { return CH % 16 == 0 ? (row & 3) << 2 : (row & 2) << 1; }
  __device__ static int k_at(int row, int ch) { return (row * CH + (ch ^ k_swap(row))) * 16; }
  __device__ static int v_at(int row, int ch) { return (row * CH + (ch ^ v_swap(row))) * 16; }
};

// A thread's NL pieces of a tile, at byte off[] of its rows, straight into LDS: a wave's 64 pieces in a row, NW
// waves in turn.  Rows past the last one repeat it (CH pieces to a row, ts bytes between rows).  32-bit
// offsets: a tile's rows are within 2 GiB.
template <int NL, int NW, int CH, int KT>
__device__ __forceinline__ void load_tile(const char* p, int ts, const int* off, int last, int wave, char* lds) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, 0x7FFFFFFF, 0x00020000);
  if (last >= KT - 1) {
#pragma unroll
    for (int i = 0; i < NL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(void, lds + (i * NW + wave) * 1024), 16, off[i], 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = ((i * NW + wave) * 64 + (int)(threadIdx.x & 63)) / CH;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(void, lds + (i * NW + wave) * 1024), 16,
                                               off[i] - max(row - last, 0) * ts, 0, 0, 0);
    }
  }
}

// bf16: a workgroup of NW waves has 32 rows a wave; key tiles of KT keys go straight into one of two LDS buffers
// while the other is worked on.
template <int DP, int NW, int KT>
__global__ __launch_bounds__(NW * 64, DP <= 128 ? 2 : 1) void attn_prefill(PrefillArgs a) {
  typedef Tile<DP> L;
  constexpr int QT = NW * 32, NS = KT / 32, ND = DP / 32, NQ = DP / 16, CH = L::CH;
  constexpr int BYTES = KT * CH * 16, NL = KT * CH / (NW * 64);  // a tile's bytes and 16-byte loads of a thread
  static_assert(NW == 4 && KT >= 32, "a buffer for each wave's 32 rows of output");
  // Four arrays, not two of two: the compiler then knows that the loads in flight do not write what is read.
  __shared__ __attribute__((aligned(16))) char kt0[BYTES], kt1[BYTES], vt0[BYTES], vt1[BYTES];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // This thread's pieces of a tile: the chunk of memory that belongs at each place (the first one past a row's end:
  // K's meets zeros of Q, V's gives channels that are not stored).
  const int kts = (int)a.k.ts, vts = (int)a.v.ts;
  int koff[NL], voff[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int c = (i * NW + wave) * 64 + lane, row = c / CH, pos = c - row * CH;
    const int kc = pos ^ L::k_swap(row), vc = pos ^ L::v_swap(row);
    koff[i] = row * kts + (kc * 8 < a.D ? kc : 0) * 16;
    voff[i] = row * vts + (vc * 8 < a.D ? vc : 0) * 16;
  }

  const int h = blockIdx.x;
  Work w;
  for (int64_t idx = blockIdx.y; find_tile(a, QT, idx, w); idx += gridDim.y) {
    const int tile = w.tiles - 1 - w.tile;  // causal: the tiles with the most keys first
    const int q0 = w.q0, lq = w.lq, k0 = w.k0, lk = w.lk;
    const int rows = lq * a.G, r0 = tile * QT + wave * 32;
    const int r = r0 + col, rc = min(r, rows - 1);
    const int tok = rc / a.G, g = rc - tok * a.G;
    // Keys that a row sees: [0, seen).
    const auto seen_by = [&](int token) { return a.causal ? min(max(token + 1 + lk - lq, 0), lk) : lk; };
    const int seen = seen_by(tok);
    const int wave_first = __builtin_amdgcn_readfirstlane(seen_by(min(r0, rows - 1) / a.G));
    const int wave_last = r0 >= rows ? 0 : __builtin_amdgcn_readfirstlane(seen_by(min(r0 + 31, rows - 1) / a.G));
    const int block_last = seen_by(min(tile * QT + QT - 1, rows - 1) / a.G);

    const char* kp = a.k.p + (int64_t)k0 * a.k.ts + (int64_t)h * a.k.hs;
    const char* vp = a.v.p + (int64_t)k0 * a.v.ts + (int64_t)h * a.v.hs;
    // Keys j0 .. j0 + KT - 1 into a buffer; past the end the last key again (finite, masked below).
    const auto load = [&](int j0, char* kt, char* vt) {
      const int last = min(lk - 1 - j0, KT - 1);
      load_tile<NL, NW, CH, KT>(kp + (int64_t)j0 * a.k.ts, kts, koff, last, wave, kt);
      load_tile<NL, NW, CH, KT>(vp + (int64_t)j0 * a.v.ts, vts, voff, last, wave, vt);
    };
    __syncthreads();  // the last tile's reads of the buffers are over
    if (block_last > 0) load(0, kt0, vt0);

    // Q as the right operand: a lane's row, in the order that the K reads below use.
    u32x4 qf[NQ];
    const char* qp = a.q.p + (int64_t)(q0 + tok) * a.q.ts + (int64_t)(h * a.G + g) * a.q.hs;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int ch = 2 * i + half;
      qf[i] = ch * 8 < a.D ? *reinterpret_cast<const u32x4*>(qp + ch * 16) : u32x4{0, 0, 0, 0};
    }
    f32x16 o[ND] = {};
    float m = -INFINITY, l = 0.0f;

    const auto work = [&](int j0, const char* kt, const char* vt) {
      f32x16 s[NS];
      __builtin_amdgcn_s_setprio(1);  // the matrix instructions first: the other wave of a SIMD has the vector unit
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        s[n] = f32x16{};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const u32x4 kf = *reinterpret_cast<const u32x4*>(kt + L::k_at(n * 32 + col, 2 * i + half));
          s[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf), __builtin_bit_cast(bf16x8, qf[i]),
                                                         s[n], 0, 0, 0);
        }
      }
      if (j0 + KT > wave_first) {  // some row of the wave does not see some key of the tile
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = j0 + n * 32 + 8 * (i / 4) + 4 * half + i % 4;
            s[n][i] = key < seen ? s[n][i] : -INFINITY;
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[n][i]);
      mx = half_max(mx) * a.scale_log2;
      // The subtracted maximum follows the true one only when it has grown by 2^SLACK: weights stay below 2^SLACK,
      // and the output is rescaled a few times in a sequence instead of at every tile.
      constexpr float SLACK = 8.0f;
      __builtin_amdgcn_s_setprio(0);
      if (__any(mx > m + SLACK)) {
        const float to = mx > m ? mx : m;
        const float alpha = hw_exp2(m - (to == -INFINITY ? 0.0f : to));
        m = to;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
      }
      const float mc = m == -INFINITY ? 0.0f : m;  // a row that has seen nothing yet: all weights 0
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[n][i] = hw_exp2(fmaf(s[n][i], a.scale_log2, -mc));
          l += s[n][i];  // this half's keys only; joined at the end
        }
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t) {  // 16 keys: this half holds keys 4 half + {0..3, 8..11} of them
          u32x4 pf;
#pragma unroll
          for (int i = 0; i < 4; ++i) pf[i] = pack_bf16(s[n][8 * t + 2 * i], s[n][8 * t + 2 * i + 1]);
          // The transposing read: 16 lanes give 4 rows of 16 channels and get 4 rows of one channel each.
          const int row = n * 32 + 16 * t + 4 * half + (lane & 15) / 4;
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const int e = d * 32 + (col & 16) + (lane & 3) * 4;
            union {
              s16x4 x[2];
              bf16x8 v;
            } vf;
            vf.x[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, vt + L::v_at(row, e / 8) + (e & 4) * 2));
            vf.x[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, vt + L::v_at(row + 8, e / 8) + (e & 4) * 2));
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf.v, __builtin_bit_cast(bf16x8, pf), o[d], 0, 0, 0);
          }
        }
    };

    if (block_last > 0) {
      __syncthreads();
      for (int j0 = 0; j0 < block_last; j0 += 2 * KT) {
        if (j0 + KT < block_last) load(j0 + KT, kt1, vt1);
        if (j0 < wave_last) work(j0, kt0, vt0);
        __syncthreads();
        if (j0 + KT >= block_last) break;
        if (j0 + 2 * KT < block_last) load(j0 + 2 * KT, kt0, vt0);
        if (j0 + KT < wave_last) work(j0 + KT, kt1, vt1);
        __syncthreads();
      }
    }

    // The output through LDS (one of the buffers for each wave; their reads ended at the last barrier), so that
    // memory gets whole rows and not 8 bytes of each.
    l = half_sum(l);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    char* stage = wave == 0 ? kt0 : wave == 1 ? kt1 : wave == 2 ? vt0 : vt1;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x2*>(stage + L::k_at(col, d * 4 + i) + half * 8) =
            u32x2{pack_bf16(o[d][4 * i] * inv, o[d][4 * i + 1] * inv), pack_bf16(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
    const int64_t row_at = (int64_t)(q0 + tok) * a.out.ts + (int64_t)(h * a.G + g) * a.out.hs;
    constexpr int PIECES = DP / 8;
#pragma unroll
    for (int i = 0; i < 32 * PIECES / 64; ++i) {
      const int c = i * 64 + lane, row = c / PIECES, ch = c - row * PIECES;
      const int64_t at = __shfl(row_at, row);
      if (r0 + row < rows && ch * 8 < a.D)
        *reinterpret_cast<u32x4*>(a.out.p + at + ch * 16) = *reinterpret_cast<const u32x4*>(stage + L::k_at(row, ch));
    }
    if (a.lse && half == 0 && r < rows)
      a.lse[(int64_t)(q0 + tok) * a.Hq + h * a.G + g] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
  }
}

constexpr int F32_NW = 4;

// fp32, on the fp32 matrix instructions (a sixteenth of bf16's rate, which bounds it): a wave reads its
// operands straight from memory, no LDS.  A workgroup has 32 rows; its waves take 32 keys in turn, so
// that few rows still fill the chip, and join their results at the end.  K's channels may come in any
// order if Q's do too: 16-byte reads of both.  Lane m of V's operand holds VE neighbouring channels of
// one key, for VE output tiles.  A step's V is loaded while its scores are computed, the next step's K while
// its output is.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_view(const char* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, bytes, 0x00020000);
}

// Pieces 32 i + 16 half of a lane's row (at: its first byte); the first one again past D.
template <int NQ>
__device__ __forceinline__ void load_k32(f32x4* k, const char* p, int bytes, int at, int D) {
  const __amdgpu_buffer_rsrc_t r = rows_view(p, bytes);
#pragma unroll
  for (int i = 0; i < NQ; ++i)
    k[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, i * 8 < D ? i * 32 : 0, 0));
}

template <int NB, int VE>
__device__ __forceinline__ void load_v32(float (*v)[NB * VE], const char* p, int bytes, const int* at, int ts) {
  const __amdgpu_buffer_rsrc_t r = rows_view(p, bytes);
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int row = (8 * (i / 4) + i % 4) * ts;
      float* x = v[i] + n * VE;
      if constexpr (VE == 4) {
        const f32x4 t = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at[n], row, 0));
        x[0] = t[0], x[1] = t[1], x[2] = t[2], x[3] = t[3];
      } else if constexpr (VE == 2) {
        const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at[n], row, 0));
        x[0] = __uint_as_float(t[0]), x[1] = __uint_as_float(t[1]);
      } else {
        x[0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at[n], row, 0));
      }
    }
}

template <int DP>
__global__ __launch_bounds__(F32_NW * 64, 1) void attn_prefill_f32(PrefillArgs a) {
  constexpr int NW = F32_NW, QT = 32, NQ = DP / 8;
  constexpr int VE = DP % 128 == 0 ? 4 : DP % 64 == 0 ? 2 : 1, NB = DP / (32 * VE);  // channels of a lane, blocks of 32 VE
  constexpr bool QREG = DP <= 128;  // Q in registers beside a step's K, V and output, else in LDS
  __shared__ float wml[NW][32][2];
  __shared__ __attribute__((aligned(16))) float wo[NW][32][32 * VE + 4];
  __shared__ __attribute__((aligned(16))) f32x4 ql[QREG ? 1 : NQ][64];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kts = (int)a.k.ts, vts = (int)a.v.ts;
  int vo[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) vo[n] = 4 * half * vts + ((n * 32 + col) * VE < a.D ? (n * 32 + col) * VE * 4 : 0);

  const int h = blockIdx.x;
  Work w;
  for (int64_t idx = blockIdx.y; find_tile(a, QT, idx, w); idx += gridDim.y) {
    const int tile = w.tiles - 1 - w.tile;
    const int q0 = w.q0, lq = w.lq, k0 = w.k0, lk = w.lk;
    const int rows = lq * a.G, r0 = tile * QT;
    const int r = r0 + col, rc = min(r, rows - 1);
    const int tok = rc / a.G, g = rc - tok * a.G;
    const auto seen_by = [&](int token) { return a.causal ? min(max(token + 1 + lk - lq, 0), lk) : lk; };
    const int seen = seen_by(tok);
    const int first = __builtin_amdgcn_readfirstlane(seen_by(r0 / a.G));
    const int last = __builtin_amdgcn_readfirstlane(seen_by(min(r0 + 31, rows - 1) / a.G));

    const char* kp = a.k.p + (int64_t)k0 * a.k.ts + (int64_t)h * a.k.hs;
    const char* vp = a.v.p + (int64_t)k0 * a.v.ts + (int64_t)h * a.v.hs;
    // Bytes of a step's rows: past them, keys read as zeros (masked below).
    const auto span = [&](int j0, int ts) { return (min(lk - j0, 32) - 1) * ts + a.D * 4; };
    f32x4 kx[NQ];
    int j0 = wave * 32;
    if (j0 < last) load_k32<NQ>(kx, kp + (int64_t)j0 * a.k.ts, span(j0, kts), col * kts + half * 16, a.D);
    f32x4 qf[QREG ? NQ : 1];
    const char* qp = a.q.p + (int64_t)(q0 + tok) * a.q.ts + (int64_t)(h * a.G + g) * a.q.hs;
    if constexpr (!QREG) __syncthreads();
#pragma unroll
    for (int i = QREG ? 0 : wave; i < NQ; i += QREG ? 1 : NW) {
      const int e = (2 * i + half) * 4;
      const f32x4 x = e < a.D ? *reinterpret_cast<const f32x4*>(qp + e * 4) : f32x4{};
      if constexpr (QREG) qf[i] = x;
      else ql[i][lane] = x;
    }
    if constexpr (!QREG) __syncthreads();
    f32x16 o[NB * VE] = {};
    float m = -INFINITY, l = 0.0f;

    for (; j0 < last; j0 += NW * 32) {
      float vx[16][NB * VE];
      load_v32<NB, VE>(vx, vp + (int64_t)j0 * a.v.ts, span(j0, vts), vo, vts);
      __builtin_amdgcn_sched_barrier(0);
      f32x16 s = {};
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const f32x4 qx = QREG ? qf[QREG ? i : 0] : ql[QREG ? 0 : i][lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) s = __builtin_amdgcn_mfma_f32_32x32x2f32(kx[i][j], qx[j], s, 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      const int jn = j0 + NW * 32;
      if (jn < last) load_k32<NQ>(kx, kp + (int64_t)jn * a.k.ts, span(jn, kts), col * kts + half * 16, a.D);
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
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int c = 0; c < NB * VE; ++c) o[c] = __builtin_amdgcn_mfma_f32_32x32x2f32(vx[i][c], s[i], o[c], 0, 0, 0);
    }

    // Join the waves, as the decode kernel does: one maximum, then sums in wave order.
    l = half_sum(l);
    __syncthreads();
    if (half == 0) wml[wave][col][0] = m;
    __syncthreads();
    float top = wml[0][col][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = fmaxf(top, wml[w][col][0]);
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
        for (int w = 0; w < NW; ++w) {
          y += *reinterpret_cast<const f32x4*>(&wo[w][row][e]);
          sum += wml[w][row][1];
          hm = fmaxf(hm, wml[w][row][0]);
        }
        const int t = rr / a.G, head = h * a.G + rr - t * a.G;
        *reinterpret_cast<f32x4*>(a.out.p + (int64_t)(q0 + t) * a.out.ts + (int64_t)head * a.out.hs + (n * BC + e) * 4) =
            y * (sum > 0.0f ? 1.0f / sum : 0.0f);
        if (a.lse && n == 0 && e == 0)
          a.lse[(int64_t)(q0 + t) * a.Hq + head] = sum > 0.0f ? (hm + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
      }
    }
  }
}

// Key heads and tiles (at most: the sum of ceil(rows / QT) over the sequences), heads first: the eight XCDs take
// workgroups in turn, so that with eight heads each XCD's L2 holds the keys of one.
dim3 tiles_grid(const PrefillArgs& a, int QT) {
  const int64_t tiles = (int64_t)a.Tq * a.G / QT + a.B, most = 65535;
  return dim3(a.Hkv, (unsigned)(tiles < most ? tiles : most));  // 65535 * 1024 heads * 256 threads: below 2^35
}

template <int DP>
void launch_bf16(PrefillArgs& a, hipStream_t s) {
  constexpr int NW = 4, KT = DP > 128 ? 32 : 64;  // two buffers of K and V: 64 KB, two workgroups on a CU up to 128
  attn_prefill<DP, NW, KT><<<tiles_grid(a, NW * 32), dim3(NW * 64), 0, s>>>(a);
}

template <int DP>
void launch_f32(PrefillArgs& a, hipStream_t s) {
  attn_prefill_f32<DP><<<tiles_grid(a, 32), dim3(F32_NW * 64), 0, s>>>(a);
}

hipError_t launch(PrefillArgs& a, bool bf16, hipStream_t s) {
  if (a.D <= 64) bf16 ? launch_bf16<64>(a, s) : launch_f32<64>(a, s);
  else if (a.D <= 96) bf16 ? launch_bf16<96>(a, s) : launch_f32<96>(a, s);
  else if (a.D <= 128) bf16 ? launch_bf16<128>(a, s) : launch_f32<128>(a, s);
  else if (a.D <= 192) bf16 ? launch_bf16<192>(a, s) : launch_f32<192>(a, s);
  else bf16 ? launch_bf16<256>(a, s) : launch_f32<256>(a, s);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn
}  // namespace ssm

extern "C" int ssm_attn_prefill(const ssm_attn_dims* d, const ssm_view* q, const ssm_view* k, const ssm_view* v,
                                const int32_t* cu_q, const int32_t* cu_k, const ssm_view* out, float* lse,
                                void* stream) {
  using namespace ssm::attn;
  if (!d) return SSM_ERR_NULL;
  int64_t es;
  if (const int st = check_io(d->io_dtype, &es)) return st;
  if (const int st = check_heads(d->q_heads, d->head_dim)) return st;
  if (const int st = check_heads(d->kv_heads, d->head_dim)) return st;
  if (d->q_heads % d->kv_heads) return SSM_ERR_SHAPE;
  if (d->batch < 1 || d->batch > SSM_ATTN_MAX_BATCH) return SSM_ERR_SHAPE;
  if (d->q_tokens < 0 || d->k_tokens < 0 || d->k_tokens > MAX_TOKENS) return SSM_ERR_SHAPE;
  if (d->q_tokens > MAX_TOKENS / (d->q_heads / d->kv_heads)) return SSM_ERR_SHAPE;
  if (!isfinite(d->scale) || !(d->scale > 0.0f) || (d->causal != 0 && d->causal != 1)) return SSM_ERR_SHAPE;
  if (d->q_tokens == 0) return SSM_OK;
  if (!cu_q || !cu_k) return SSM_ERR_NULL;
  if (const int st = check_view(q, es)) return st;
  if (const int st = check_view(out, es)) return st;
  const int64_t Tq = d->q_tokens, Tk = d->k_tokens, D = d->head_dim, Hq = d->q_heads, Hkv = d->kv_heads;
  if (Tk) {
    if (const int st = check_view(k, es)) return st;
    if (const int st = check_view(v, es)) return st;
  }
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4)) return SSM_ERR_ALIGN;
  if (!writable(out, Tq, Hq, D) || views_overlap(out, Tq, Hq, q, Tq, Hq, D, es)) return SSM_ERR_ALIAS;
  const Span so = view_span(out, Tq, Hq, D, es), sl = span(lse, lse ? Tq * Hq * 4 : 0);
  const Span s_cu[2] = {span(cu_q, (d->batch + 1) * 4), span(cu_k, (d->batch + 1) * 4)};
  for (const Span& c : s_cu)
    if (overlaps(so, c) || overlaps(sl, c)) return SSM_ERR_ALIAS;
  if (overlaps(so, sl) || overlaps(sl, view_span(q, Tq, Hq, D, es))) return SSM_ERR_ALIAS;
  if (Tk) {
    if (views_overlap(out, Tq, Hq, k, Tk, Hkv, D, es) || views_overlap(out, Tq, Hq, v, Tk, Hkv, D, es))
      return SSM_ERR_ALIAS;
    if (overlaps(sl, view_span(k, Tk, Hkv, D, es)) || overlaps(sl, view_span(v, Tk, Hkv, D, es))) return SSM_ERR_ALIAS;
  }
  PrefillArgs a = {};
  a.q = bytes_view(q, es);
  a.out = bytes_view(out, es);
  if (Tk) {
    a.k = bytes_view(k, es);
    a.v = bytes_view(v, es);
  }
  a.lse = lse;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.B = (int)d->batch;
  a.Tq = (int)Tq;
  a.Tk = (int)Tk;
  a.Hq = d->q_heads;
  a.Hkv = d->kv_heads;
  a.G = d->q_heads / d->kv_heads;
  a.D = d->head_dim;
  a.causal = d->causal;
  a.scale_log2 = d->scale * 1.4426950408889634f;
  if (!isfinite(a.scale_log2) || !(a.scale_log2 > 0.0f)) return SSM_ERR_SHAPE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = launch(a, d->io_dtype == SSM_BF16, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}
