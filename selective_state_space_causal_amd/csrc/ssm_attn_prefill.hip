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

// Tile `idx` in the order of falling work (key tiles of KT): up to 64 sequences, one a lane (q: its bounds).  The
// tiles with at least c key tiles are counted for a c found by bisection.  top: a c that no tile from here on exceeds,
// made smaller for the calls that follow (with larger idx).
__device__ __forceinline__ bool find_sorted(const PrefillArgs& a, int QT, int KT, int4 q, int64_t idx, int& top, Work& w) {
  const int tiles = tiles_of(a, QT, q.y);
  // Tiles of this lane's sequence whose last row sees more than (c - 1) KT keys.
  const auto at_least = [&](int c) {
    const int64_t x = (int64_t)(c - 1) * KT;
    if (c <= 0) return tiles;
    if (!a.causal) return q.w > x ? tiles : 0;
    const int64_t token = x - (q.w - q.y);  // the first token that sees so many
    if (token >= q.y) return 0;
    return tiles - (token <= 0 ? 0 : (int)(((unsigned)((int)token * a.G) + QT) / QT) - 1);
  };
  const auto total = [&](int n) { return __builtin_amdgcn_readlane(wave_scan(n), 63); };
  if (idx >= total(tiles)) return false;
  const int want = (int)idx;
  int lo = 0, hi = top;  // more than `want` tiles have lo key tiles or more, no more than `want` have hi + 1
  for (int step = 1; lo < hi; step *= 2) {  // the last call's c is near: in growing steps down, then halves
    const int mid = max(hi - step + 1, (lo + hi + 1) >> 1);
    if (total(at_least(mid)) > want) lo = mid;
    else hi = mid - 1;
  }
  top = lo;
  const int more = at_least(lo + 1), n = at_least(lo) - more, incl = wave_scan(n);
  const int rank = want - total(more);
  const int at = __ffsll((unsigned long long)__ballot(incl > rank)) - 1;
  w.tiles = __builtin_amdgcn_readlane(tiles, at);
  w.tile = w.tiles - __builtin_amdgcn_readlane(more + incl, at) + rank;  // the class's tiles end where `more` begin
  w.q0 = __builtin_amdgcn_readlane(q.x, at);
  w.lq = __builtin_amdgcn_readlane(q.y, at);
  w.k0 = __builtin_amdgcn_readlane(q.z, at);
  w.lk = __builtin_amdgcn_readlane(q.w, at);
  return true;
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
// while the other is worked on.  A workgroup takes tiles of rows in turn until there are none, and the key
// tiles of one follow those of the last without a break: the next one's first keys are loaded under the
// last key tile of this one, its queries under that tile's softmax, and the output is stored under what comes then.
// Each head's tiles are dealt out in the order of falling work, forwards and backwards in turn.
template <int DP, int NW, int KT>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(DP <= 192 ? 2 : 1, DP <= 192 ? 2 : 1)))
void attn_prefill(PrefillArgs a) {
  typedef Tile<DP> L;
  constexpr int QT = NW * 32, NS = KT / 32, ND = DP / 32, NQ = DP / 16, CH = L::CH, AHEAD = 4;
  constexpr int BYTES = KT * CH * 16, NL = KT * CH / (NW * 64);  // a tile's bytes and 16-byte loads of a thread
  // Four arrays, not two of two: the compiler then knows that the loads in flight do not write what is read.
  __shared__ __attribute__((aligned(16))) char kt0[BYTES], kt1[BYTES], vt0[BYTES], vt1[BYTES];
  __shared__ int4 seqs[64];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (threadIdx.x < 64) seqs[threadIdx.x] = bounds(a, threadIdx.x);

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
  __syncthreads();

  const int h = blockIdx.x, places = gridDim.y, place = blockIdx.y;
  int64_t dealt = 0;  // tiles dealt to all places before this round
  bool forwards = true;
  int top = (int)(((unsigned)a.Tk + KT - 1) / KT);
  // The next tile of rows; false when there are no more.
  const auto next = [&](Work& w) {
    const int64_t idx = dealt + (forwards ? place : places - 1 - place);
    dealt += places;
    forwards = !forwards;
    if (a.B <= 64) return find_sorted(a, QT, KT, seqs[here(lane)], idx, top, w);
    const bool found = find_tile(a, QT, idx, w);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0) of its loads here, not under the products
    if (!found) return false;
    w.tile = w.tiles - 1 - w.tile;  // causal: a sequence's tiles with the most keys first
    return true;
  };
  // Keys that a token of a sequence sees: [0, seen_by).
  const auto seen_by = [&](const Work& w, int token) {
    return a.causal ? min(max(token + 1 + w.lk - w.lq, 0), w.lk) : w.lk;
  };
  const auto keys_of = [&](const Work& w) {  // of a tile's last row
    return seen_by(w, min(w.tile * QT + QT - 1, w.lq * a.G - 1) / a.G);
  };
  // Keys j0 .. j0 + KT - 1 into a buffer; past the end the last key again (finite, masked below).
  const auto load = [&](const Work& w, int j0, char* kt, char* vt) {
    const int last = min(w.lk - 1 - j0, KT - 1);
    load_tile<NL, NW, CH, KT>(a.k.p + (int64_t)(w.k0 + j0) * a.k.ts + (int64_t)h * a.k.hs, kts, koff, last, wave, kt);
    load_tile<NL, NW, CH, KT>(a.v.p + (int64_t)(w.k0 + j0) * a.v.ts + (int64_t)h * a.v.hs, vts, voff, last, wave, vt);
  };
  // Q as the right operand: a lane's row, in the order that the K reads below use.
  u32x4 qf[NQ];
  const auto load_q = [&](const Work& w) {
    const int c = here(lane), half = c >> 5;
    const int r = min(w.tile * QT + wave * 32 + (c & 31), w.lq * a.G - 1), tok = r / a.G;
    const char* qp = a.q.p + (int64_t)(w.q0 + tok) * a.q.ts + (int64_t)(h * a.G + r - tok * a.G) * a.q.hs;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int ch = 2 * i + half;
      qf[i] = ch * 8 < a.D ? *reinterpret_cast<const u32x4*>(qp + ch * 16) : u32x4{0, 0, 0, 0};
    }
  };

  Work w, nx = {};
  if (!next(w)) return;
  bool more = false, fresh = true;  // more: nx is the next tile; fresh: not yet looked for
  int r0, seen, wave_first, wave_last, block_last, j0;
  f32x16 o[ND];
  float m, l;
  const auto begin = [&] {
    const int rows = w.lq * a.G;
    r0 = w.tile * QT + wave * 32;
    seen = seen_by(w, min(r0 + col, rows - 1) / a.G);
    wave_first = seen_by(w, min(r0, rows - 1) / a.G);
    wave_last = r0 >= rows ? 0 : seen_by(w, min(r0 + 31, rows - 1) / a.G);
    block_last = keys_of(w);
    j0 = 0;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16{};
  };

  const auto work = [&](const char* kt, const char* vt, bool last) {
      // Operands are read some products ahead; the barriers hold each read in its place.
      const auto read_k = [&](int i) {
        return *reinterpret_cast<const bf16x8*>(kt + L::k_at(i / NQ * 32 + col, 2 * (i % NQ) + half));
      };
      f32x16 s[NS];
      bf16x8 kf[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) kf[i] = read_k(i);
      __builtin_amdgcn_s_setprio(1);  // the matrix instructions first: the other wave of a SIMD has the vector unit
#pragma unroll
      for (int i = 0; i < NS * NQ; ++i) {
        f32x16& sn = s[i / NQ];
        if (i % NQ == 0) sn = f32x16{};
        __builtin_amdgcn_sched_barrier(0);
        sn = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i % AHEAD], __builtin_bit_cast(bf16x8, qf[i % NQ]), sn, 0, 0, 0);
        if (i + AHEAD < NS * NQ) kf[i % AHEAD] = read_k(i + AHEAD);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (last) load_q(nx);
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
      // 16 keys at a time: this half holds keys 4 half + {0..3, 8..11} of them.  Under each product of 16 keys go the
      // reads of V for the same product of the next 16, and a share of their weights.
      const auto weight = [&](int i) {
        const float x = hw_exp2(fmaf(s[i / 16][i % 16], a.scale_log2, -mc));
        s[i / 16][i % 16] = x;
        l += x;  // this half's keys only; joined at the end
      };
      const auto packed = [&](int g) {
        u32x4 p;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = pack_bf16(s[g / 2][8 * (g & 1) + 2 * i], s[g / 2][8 * (g & 1) + 2 * i + 1]);
        return __builtin_bit_cast(bf16x8, p);
      };
      const auto read_v = [&](int g, int d) {
        // The transposing read: 16 lanes give 4 rows of 16 channels and get 4 rows of one channel each.
        const int row = g * 16 + 4 * half + (lane & 15) / 4, e = d * 32 + (col & 16) + (lane & 3) * 4;
        union {
          s16x4 x[2];
          bf16x8 v;
        } vf;
        vf.x[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, vt + L::v_at(row, e / 8) + (e & 4) * 2));
        vf.x[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, vt + L::v_at(row + 8, e / 8) + (e & 4) * 2));
        return vf.v;
      };
      constexpr int GROUPS = 2 * NS;
      bf16x8 vf[ND];
#pragma unroll
      for (int d = 0; d < ND; ++d) vf[d] = read_v(0, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) weight(i);
      bf16x8 pf = packed(0);
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          __builtin_amdgcn_sched_barrier(0);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[d], pf, o[d], 0, 0, 0);
          if (g + 1 < GROUPS) {
            vf[d] = read_v(g + 1, d);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i * ND / 8 == d) weight((g + 1) * 8 + i);
          }
        }
        if (g + 1 < GROUPS) pf = packed(g + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    };

  // The halves of a row hold 4 channels of 8 in turn: exchanged, each has whole 16-byte pieces.
  const auto store = [&] {
    l = half_sum(l);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int lane = here(threadIdx.x & 63), half = lane >> 5;
    const int rows = w.lq * a.G, r = r0 + (lane & 31), rc = min(r, rows - 1), tok = rc / a.G, head = h * a.G + rc - tok * a.G;
    char* op = a.out.p + (int64_t)(w.q0 + tok) * a.out.ts + (int64_t)head * a.out.hs + half * 16;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        u32x2 x[2];  // channels 32 d + 8 (i + 0, 1) + 4 half + {0..3}
#pragma unroll
        for (int j = 0; j < 2; ++j)
          x[j] = u32x2{pack_bf16(o[d][4 * (i + j)] * inv, o[d][4 * (i + j) + 1] * inv),
                       pack_bf16(o[d][4 * (i + j) + 2] * inv, o[d][4 * (i + j) + 3] * inv)};
        // the upper half's piece i for the lower half's piece i + 1
        const auto lo = __builtin_amdgcn_permlane32_swap(x[0][0], x[1][0], false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(x[0][1], x[1][1], false, false);
        if (r < rows && d * 32 + (i + half) * 8 < a.D)
          *reinterpret_cast<u32x4*>(op + (d * 4 + i) * 16) = u32x4{lo[0], hi[0], lo[1], hi[1]};
      }
    if (a.lse && half == 0 && r < rows)
      a.lse[(int64_t)(w.q0 + tok) * a.Hq + head] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
  };

  // One key tile, from (kc, vc), while the next one comes into (kn, vn); false when all is done.
  const auto advance = [&](char* kc, char* vc, char* kn, char* vn) {
    const bool ends = j0 + KT >= block_last;
    if (!ends) load(w, j0 + KT, kn, vn);
    if (fresh) more = next(nx), fresh = false;
    if (ends && more && keys_of(nx) > 0) load(nx, 0, kn, vn);
    const bool sees = j0 < wave_last;
    if (sees) work(kc, vc, ends && more);
    if (!sees && ends && more) load_q(nx);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0), said here: the compiler then waits for no load under the products
    __syncthreads();  // the reads of (kc, vc) are over, (kn, vn) and a next tile's Q are there
    if (!ends) {
      j0 += KT;
      return true;
    }
    store();
    if (!more) return false;
    w = nx;
    begin();
    fresh = true;
    return true;
  };

  begin();
  if (block_last > 0) load(w, 0, kt0, vt0);
  load_q(w);
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __syncthreads();
  while (advance(kt0, vt0, kt1, vt1) && advance(kt1, vt1, kt0, vt0)) {
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
dim3 tiles_grid(const PrefillArgs& a, int QT, int places) {
  const int64_t tiles = (int64_t)a.Tq * a.G / QT + a.B;
  int64_t most = places / a.Hkv;
  most = most < 1 ? 1 : most > 65535 ? 65535 : most;
  return dim3(a.Hkv, (unsigned)(tiles < most ? tiles : most));
}

template <int DP>
void launch_bf16(PrefillArgs& a, hipStream_t s) {
  constexpr int NW = 4, KT = DP > 128 ? 32 : 64, PER_CU = DP > 192 ? 1 : 2;  // two buffers of K and V: 64 KB, two workgroups on a CU up to 128
  attn_prefill<DP, NW, KT><<<tiles_grid(a, NW * 32, 256 * PER_CU), dim3(NW * 64), 0, s>>>(a);
}

template <int DP>
void launch_f32(PrefillArgs& a, hipStream_t s) {
  attn_prefill_f32<DP><<<tiles_grid(a, 32, INT32_MAX), dim3(F32_NW * 64), 0, s>>>(a);
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
