// ssm_attn_prefill.hip -- ssm_attn_prefill of include/ssm_attn.h: softmax attention over packed
// prompts, one pass over the keys with the running maximum and sum of each row's softmax.
//
// Products.  Scores are computed transposed, S^T = K Q^T, with 32x32 matrix instructions: a lane then
// holds scores of ONE row (column lane & 31), 16 keys of every 32, the other 16 being in lane ^ 32.
// Row maxima and sums are therefore taken inside a lane, with a single exchange of the two halves, and
// the weights are already in the layout of the second product's right operand, O^T = V^T P^T: the
// order of the keys inside a product is free as long as V is read in the same order.  V's operand needs
// keys along a lane's registers, and V is stored with channels along a row: bf16 uses the LDS read that
// transposes 16-bit elements.
#include "ssm_attn_prefill.h"

namespace ssm {
namespace attn {
namespace {

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

// A lane's 16 bytes at byte `off` of a tile's rows straight into LDS, a wave's 64 pieces in a row.  32-bit offsets: a tile's
// rows are within 2 GiB.
__device__ __forceinline__ void load_piece(const char* p, int off, char* lds) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, 0x7FFFFFFF, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(void, lds), 16, off, 0, 0, 0);
}

// bf16: a workgroup of NW waves has 32 rows for every KS waves, which share the keys: key tiles of KS times KT keys go
// straight into one of two LDS buffers while the other is worked on, KT keys of them for each of the KS.  A workgroup takes tiles of rows in turn until there are none, and the key
// tiles of one follow those of the last without a break: the next one's first keys are loaded under the
// last key tile of this one, its queries under that tile's softmax, and the output is stored under what comes then.
// Each head's tiles are dealt out in the order of falling work, forwards and backwards in turn.
template <int DP, int NW, int KT, int KS>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(DP <= 192 ? 2 : 1, DP <= 192 ? 2 : 1)))
void attn_prefill(PrefillArgs a) {
  typedef Tile<DP> L;
  constexpr int RW = NW / KS, QT = RW * 32, KB = KT * KS, NS = KT / 32, ND = DP / 32, NQ = DP / 16, CH = L::CH, AHEAD = 4;
  constexpr int BYTES = KB * CH * 16, NL = KB * CH / (NW * 64);  // a tile's bytes and 16-byte loads of a thread
  // Four arrays, not two of two: the compiler then knows that the loads in flight do not write what is read.
  __shared__ __attribute__((aligned(16))) char kt0[BYTES], kt1[BYTES], vt0[BYTES], vt1[BYTES];
  __shared__ int4 seqs[64], found_q[2][NW];
  __shared__ int2 found_k[2][NW];
  __shared__ float2 stats[KS > 1 ? NW / 2 : 1][64];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rw = wave % RW, kw = wave / RW;
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
  int top = (int)(((unsigned)a.Tk + KB - 1) / KB);
  // The tile that this place takes in a round; tile -1 past the last.
  const auto find = [&](int round) {
    const int64_t idx = (int64_t)round * places + (round & 1 ? places - 1 - place : place);
    Work w = {};
    bool found;
    if (a.B <= 64) {
      found = find_sorted(a, QT, KB, seqs[here(lane)], idx, top, w);
    } else {
      found = find_tile(a, QT, idx, w);
      w.tile = w.tiles - 1 - w.tile;  // causal: a sequence's tiles with the most keys first
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0) of its loads here, not under the products
    }
    if (!found) w.tile = -1;
    return w;
  };
  // Finding a tile takes a wave some 2000 cycles: from the second on each wave finds another one of the next NW, for all (2 to
  // 5% of calls with several tiles to a place).
  const auto find_batch = [&](int batch) {
    const Work w = find(1 + batch * NW + wave);
    if (here(lane) == 0) {
      found_q[batch & 1][wave] = make_int4(w.tile, w.q0, w.lq, 0);
      found_k[batch & 1][wave] = make_int2(w.k0, w.lk);
    }
  };
  // The next one; false when there are no more.  A barrier lies between two calls: a batch is found two calls after the last one
  // of its place was taken, and three or more before its first is.
  int taken = 0;
  const auto next = [&](Work& w) {
    const int batch = taken / NW, i = taken % NW;
    if (i == 1) find_batch(batch + 1);
    const int4 q = found_q[batch & 1][i];
    const int2 k = found_k[batch & 1][i];
    ++taken;
    w.tile = __builtin_amdgcn_readfirstlane(q.x);
    w.q0 = __builtin_amdgcn_readfirstlane(q.y);
    w.lq = __builtin_amdgcn_readfirstlane(q.z);
    w.k0 = __builtin_amdgcn_readfirstlane(k.x);
    w.lk = __builtin_amdgcn_readfirstlane(k.y);
    return w.tile >= 0;
  };
  // Keys that a token of a sequence sees: [0, seen_by).
  const auto seen_by = [&](const Work& w, int token) { return seen_of(a, w.lq, w.lk, token); };
  const auto keys_of = [&](const Work& w) {  // of a tile's last row
    return seen_by(w, by_group(a, min(w.tile * QT + QT - 1, w.lq * a.G - 1)));
  };
  // A tile of keys on its way.
  struct Coming {
    const char *kp, *vp;
    int keys;  // of them; 0: none comes
  };
  // Whole tiles are asked for piece by piece under the first products where a SIMD has one wave (256 channels: 8000 tokens
  // 413 to 360 us): a wave waits some 800 cycles to issue them.  With two waves a SIMD the other one works meanwhile, and
  // the pieces between the products cost 1 to 4%.
  constexpr bool UNDER = DP > 192;
  const auto coming = [&](const Work& w, int j0) {
    return Coming{a.k.p + (int64_t)(w.k0 + j0) * a.k.ts + (int64_t)h * a.k.hs,
                  a.v.p + (int64_t)(w.k0 + j0) * a.v.ts + (int64_t)h * a.v.hs, min(w.lk - j0, KB)};
  };
  // Piece i of NL of K, then of NL of V, of a whole tile into (kt, vt).
  const auto load_whole = [&](const Coming& t, int i, char* kt, char* vt) {
    if (i < NL) load_piece(t.kp, koff[i], kt + (i * NW + wave) * 1024);
    else load_piece(t.vp, voff[i - NL], vt + ((i - NL) * NW + wave) * 1024);
  };
  // All of a tile; past the last key that one again (finite, masked below).
  const auto load = [&](const Coming& t, char* kt, char* vt) {
    if (!UNDER && t.keys == KB) {
#pragma unroll
      for (int i = 0; i < 2 * NL; ++i) load_whole(t, i, kt, vt);
      return;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int past = max(((i * NW + wave) * 64 + here(lane)) / CH - (t.keys - 1), 0), at = (i * NW + wave) * 1024;
      load_piece(t.kp, koff[i] - past * kts, kt + at);
      load_piece(t.vp, voff[i] - past * vts, vt + at);
    }
  };
  // Q as the right operand: a lane's row, in the order that the K reads below use.
  u32x4 qf[NQ];
  const auto load_q = [&](const Work& w) {
    const int c = here(lane), half = c >> 5;
    const int r = min(w.tile * QT + rw * 32 + (c & 31), w.lq * a.G - 1), tok = by_group(a, r);
    const char* qp = a.q.p + (int64_t)(w.q0 + tok) * a.q.ts + (int64_t)(h * a.G + r - tok * a.G) * a.q.hs;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int ch = 2 * i + half;
      qf[i] = ch * 8 < a.D ? *reinterpret_cast<const u32x4*>(qp + ch * 16) : u32x4{0, 0, 0, 0};
    }
  };

  Work w = find(0), nx = {};
  if (w.tile < 0) return;
  bool more = false, fresh = true;  // more: nx is the next tile; fresh: not yet looked for
  int r0, seen, wave_first, wave_last, block_last, j0;
  f32x16 o[ND];
  float m, l;
  const auto begin = [&] {
    const int rows = w.lq * a.G;
    r0 = w.tile * QT + rw * 32;
    seen = seen_by(w, by_group(a, min(r0 + col, rows - 1)));
    wave_first = seen_by(w, by_group(a, min(r0, rows - 1)));
    wave_last = r0 >= rows ? 0 : seen_by(w, by_group(a, min(r0 + 31, rows - 1)));
    block_last = keys_of(w);
    j0 = 0;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16{};
  };

  const auto work = [&](const char* kt, const char* vt, bool last, const Coming& t, char* kn, char* vn) {
      const bool under = UNDER && t.keys == KB;
      const int j1 = j0 + kw * KT;  // this wave's keys of the tile
      kt += kw * (KT * CH * 16);
      vt += kw * (KT * CH * 16);
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
#pragma unroll
        for (int p = 0; p < 2 * NL; ++p)
          if (p * NS * NQ / (2 * NL) == i && under) load_whole(t, p, kn, vn);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (last) load_q(nx);
      if (j1 + KT > wave_first) {  // some row of the wave does not see some key of the tile
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = j1 + n * 32 + 8 * (i / 4) + 4 * half + i % 4;
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
      // A weight is rounded to bf16 once, 2^-8 of it at most, as much as the output's own rounding (with fp32 weights a ragged batch is
      // off by 1.6e-3 instead of 2.0e-3); a second bf16 of each, as decode has, would be half as many products again, which bound this.
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

  // KS waves' shares of the keys joined, in halves: the upper half of the shares goes to the lower through LDS (kc and vc,
  // which it fills, in turns where it is larger), until the first has all.
  const auto join = [&](char* kc, char* vc) {
    constexpr int PIECES = BYTES / (NW / 2 * 1024);  // 16-byte pieces of a lane that a buffer holds, of NW / 2 waves
#pragma unroll
    for (int g = KS / 2; g >= 1; g /= 2) {
      const bool gives = kw >= g && kw < 2 * g, takes = kw < g;
      const int i = gives ? (kw - g) * RW + rw : wave;
      if (gives) stats[i][lane] = make_float2(m, l);
      float mine = 0.0f, theirs = 0.0f;
#pragma unroll
      for (int p0 = 0; p0 < ND * 4; p0 += 2 * PIECES) {
        const auto piece = [&](int p) {
          return reinterpret_cast<f32x4*>((p < PIECES ? kc + p * (NW / 2 * 1024) : vc + (p - PIECES) * (NW / 2 * 1024)) +
                                          i * 1024 + lane * 16);
        };
        if (gives) {
#pragma unroll
          for (int p = p0; p < ND * 4 && p < p0 + 2 * PIECES; ++p) {
            f32x4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = o[p / 4][p % 4 * 4 + j];
            *piece(p - p0) = x;
          }
        }
        __syncthreads();
        if (takes) {
          if (p0 == 0) {
            const float2 other = stats[i][lane];
            const float to = fmaxf(m, other.x), base = to == -INFINITY ? 0.0f : to;
            mine = hw_exp2(m - base);
            theirs = hw_exp2(other.x - base);
            m = to;
            l = l * mine + other.y * theirs;
          }
#pragma unroll
          for (int p = p0; p < ND * 4 && p < p0 + 2 * PIECES; ++p) {
            const f32x4 x = *piece(p - p0);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[p / 4][p % 4 * 4 + j] = o[p / 4][p % 4 * 4 + j] * mine + x[j] * theirs;
          }
        }
        __syncthreads();
      }
    }
  };

  // The halves of a row hold 4 channels of 8 in turn: exchanged, each has whole 16-byte pieces.
  const auto store = [&] {
    l = half_sum(l);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int lane = here(threadIdx.x & 63), half = lane >> 5;
    const int rows = w.lq * a.G, r = r0 + (lane & 31), rc = min(r, rows - 1), tok = by_group(a, rc), head = h * a.G + rc - tok * a.G;
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
    const bool ends = j0 + KB >= block_last;
    const bool sees = j0 + kw * KT < wave_last;
    if (!UNDER && !ends) load(coming(w, j0 + KB), kn, vn);
    if (fresh) more = next(nx), fresh = false;
    Coming t = ends ? coming(nx, 0) : coming(w, j0 + KB);
    if (ends && (!more || keys_of(nx) <= 0)) t.keys = 0;
    if (UNDER ? t.keys > 0 && !(sees && t.keys == KB) : ends && t.keys > 0) load(t, kn, vn);
    if (sees) work(kc, vc, ends && more, t, kn, vn);
    if (!sees && ends && more) load_q(nx);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0), said here: the compiler then waits for no load under the products
    __syncthreads();  // the reads of (kc, vc) are over, (kn, vn) and a next tile's Q are there
    if (!ends) {
      j0 += KB;
      return true;
    }
    if constexpr (KS > 1) join(kc, vc);
    if (kw == 0) store();
    if (!more) return false;
    w = nx;
    begin();
    fresh = true;
    return true;
  };

  begin();
  if (block_last > 0) load(coming(w, 0), kt0, vt0);
  load_q(w);
  find_batch(0);
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __syncthreads();
  while (advance(kt0, vt0, kt1, vt1) && advance(kt1, vt1, kt0, vt0)) {
  }
}

// How many waves share a tile of rows.  With few tiles a row's way along the keys, or CUs without a second wave a SIMD, set
// the time, and waves that share the keys of 128 or 64 rows are faster; with many, each key tile in LDS should serve as many
// rows as possible.  n: tiles of 128 rows, over all key heads; k: keys of a sequence; both on the average, since the
// lengths are on the device.  head_dim 128, us with (rows, shares) of
//                                       32, 8   64, 4   128, 2   128, 1   256, 1
//   n   64, k  1000 (8 and 2 heads)       18.2    17.3     21.1     23.9
//   n  126, k  2000                       35.3    27.2     34.5     42.4
//   n  258, k  4096                        111    56.7     66.6     78.1      103
//   n  288, k   546 (4 to 8 heads)        48.1    31.9     24.5     27.2     32.1
//   n  514, k  8192                        387     182      147      178      205
//   n  592, k   562 (32 and 8 heads)      93.5    51.1     38.4     31.5     34.8
//   n 1016, k  2000                        419     192      154      134      136
//   n 2056, k  8192                       1534     697      542      514      491
//   n  168, k   143                       20.6    15.4     11.6     11.0     14.7
// 32 rows from memory are taken up to n = 64 (with the mask and 1000 keys or more up to 96 or 128): past 64 of them their workgroups,
// one to a CU, are more than one round.  The table does not settle that border: at its two ends, n = 64 and 126, four shares of
// 64 rows are 5 and 23% faster, and nothing between has been measured, nor other channels.
// Without the mask all tiles of rows are as long, and there is nothing to even out where the tiles are more than the CUs
// (2500 tokens of 4 heads over one key head, n 79: Eight32 64 us, Four64 32; 2000, n 63: 28 and 27, and of 64 channels 15 and 20).
enum Shares { Eight32, Four64, Two128, One128, One256 };
Shares shares_of(const PrefillArgs& a) {
  const int64_t n = tiles_at_most(a, 128) * a.Hkv, k = a.Tk / a.B;
  // 32 rows straight from memory (ssm_attn_split.hip): rows of 64 channels, and those too wide for four shares, gain longer.
  if (n <= 64 || (a.causal && ((n <= 96 && a.D > 192) || (n <= (a.D > 64 && a.D <= 128 ? 96 : 128) && k >= 1024)))) return Eight32;
  if (k < 256) return One128;
  if (n <= (a.causal ? 260 : 130) && (a.D <= 128 || a.D > 192)) return Four64;
  if (n <= (!a.causal ? 260 : k >= 1024 ? 576 : 320) && a.D <= 192) return Two128;
  return k >= 6000 && a.D <= 128 ? One256 : One128;
}

// Two buffers of K and V are 64 KB up to 128 channels for 64 keys, 128 KB for the 128 of two or four shares.  Two waves a
// SIMD, one past 192 channels, whose four waves are two shares of 64 rows.
template <int DP>
void launch_bf16(PrefillArgs& a, Shares how, hipStream_t s) {
  constexpr int KT = DP > 128 ? 32 : 64, PER_CU = DP > 192 ? 1 : 2;
  if constexpr (DP <= 128) {
    if (how == Four64) {
      attn_prefill<DP, 8, 32, 4><<<tiles_grid(a, 64, 256), dim3(512), 0, s>>>(a);
      return;
    }
    if (how == One256) {
      attn_prefill<DP, 8, KT, 1><<<tiles_grid(a, 256, 256), dim3(512), 0, s>>>(a);
      return;
    }
  }
  if constexpr (DP <= 192) {
    if (how == Two128) {
      attn_prefill<DP, 8, KT, 2><<<tiles_grid(a, 128, 256), dim3(512), 0, s>>>(a);
      return;
    }
  } else if (how == Four64) {
    attn_prefill<DP, 4, KT, 2><<<tiles_grid(a, 64, 256), dim3(256), 0, s>>>(a);
    return;
  }
  attn_prefill<DP, 4, KT, 1><<<tiles_grid(a, 128, 256 * PER_CU), dim3(256), 0, s>>>(a);
}

hipError_t launch(PrefillArgs& a, bool bf16, hipStream_t s) {
  const Shares how = bf16 ? shares_of(a) : Eight32;
  if (how == Eight32) launch_split(a, bf16, s);
  else if (a.D <= 64) launch_bf16<64>(a, how, s);
  else if (a.D <= 96) launch_bf16<96>(a, how, s);
  else if (a.D <= 128) launch_bf16<128>(a, how, s);
  else if (a.D <= 192) launch_bf16<192>(a, how, s);
  else launch_bf16<256>(a, how, s);
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
  if (d->q_tokens < 0 || d->k_tokens < 0 || d->k_tokens > MAX_KEYS) return SSM_ERR_SHAPE;
  if (d->q_tokens > MAX_ROWS / (d->q_heads / d->kv_heads)) return SSM_ERR_SHAPE;
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
  set_group(a, d->q_heads / d->kv_heads);
  a.D = d->head_dim;
  a.causal = d->causal;
  a.scale_log2 = d->scale * 1.4426950408889634f;
  if (!isfinite(a.scale_log2) || !(a.scale_log2 > 0.0f)) return SSM_ERR_SHAPE;
  const hipStream_t s = ready(stream);
  const hipError_t e = launch(a, d->io_dtype == SSM_BF16, s);
  return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}
