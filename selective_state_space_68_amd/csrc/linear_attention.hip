// Linear attention with a constant decay per head, prompt form, on the matrix cores.
//
// Per (batch row, head) with lam = exp(log_decay) and the K x V state S:
//     S_t = lam S_{t-1} + k_t v_t^T,    o_t = scale q_t S_t.
// Over a chunk of Q = 64 tokens (n of them present) with E = lam S_in, the state before
// the chunk as its first token sees it, this unrolls into four matrix products:
//     P     = (q k^T) o M,  M[j][i] = lam^(j-i) for i <= j, else 0
//     o     = scale (P v + diag(lam^j) q E)
//     E_out = lam^n E + k^T diag(lam^(n-i)) v
// Only E crosses chunks, in float32 registers.  The gradient is the same form three times
// (LaRole): forwards for dq, backwards in time for dk and dv.  Backwards, row r of the
// sequence is token n_tokens - 1 - r, and E before the first row is the gradient of the
// final state.
//
// One workgroup walks the chunks of one (batch row, head, segment).  A wave owns 16 or 32 columns v of E
// and of the output, so E is used as a matrix operand straight from the registers that accumulate
// it: a product leaves lane (g, c) of a 16 x 16 tile four consecutive rows of column c, and since the
// order of a product's summation index is free, the rows of each tile are assigned so that the two
// tiles of a pair leave a lane 8 consecutive indices: what one operand needs.  q, k and v go from
// memory straight into LDS row by row (16 bytes a lane, no registers); operands that sum over
// tokens (k^T, v^T) come out of the same rows by transposing LDS reads.  P goes through LDS.  The next
// chunk's rows are asked for as early as the tiles allow: k, in two buffers, at the chunk's start; q
// and v once P and the product with E are done, before P v and the state's product.
//
// Roundings (bfloat16 activations; float32 activations use float32 products throughout): the decayed v
// is split into three bfloat16 terms, which carry all 24 bits; E and P as operands of the output (and in
// segments the decayed v of the pass that only feeds it, WT below) into two terms, 16 bits, so that the
// output's own rounding is the one that counts.  One term of P is not enough where a
// gradient's terms cancel.
//
// When the (batch row, head) pairs are too few to fill the chip the sequence is cut into segments: a
// pre-pass forms each segment's own state sum, a small kernel chains them, and the main pass runs
// every segment from its entering E.
//
// What bounds it (measured, one MI355X, bfloat16):
//   8 x 2048, 32 heads of 128, gradient: 350 to 360 us for 1.6 GB of rows read and written by the three roles
//     (4.6 TB/s; 1.3 GB reach memory, the rest is shared in L2).  Matrix instructions take about 6, LDS 5 and
//     vector instructions 5 of the 14 thousand cycles that the two workgroups of a CU take for a chunk
//     each: no unit is full, the 8 waves wait for each other at two barriers a chunk.
//   131072 tokens, 20 heads of 128: 880 to 905 us, 4.6 TB/s (under a trace pre-pass 327, chain 27, main pass 680): memory.
//   4 x 2048, 80 heads of 64: 119 us.  320 workgroups on 256 CUs: the time of a CU with two, 6800 cycles
//     a chunk (5400 alone); 2 or 3 segments cost more than they level (140 and 132 us).
//   float32: the float32 matrix rate (64 x 64: 7200 cycles of products a chunk and workgroup, 2 of them a CU).
//   1 x 77, 24 heads of 64: a kernel of 10.8 us, of which 3 before the first chunk's products, 7 for its two chunks.
// Tried and dropped: a second buffer for q and v (no gain); products and LDS reads interleaved by scheduling
// groups (no gain); streaming loads (5 % faster forwards at 64 x 64, 5 % slower gradients); the output stored
// before the state's product (127 us at 4 x 2048 against 122, 984 against 954 at 131072); neighbouring heads on one
// XCD (no gain; padded rows 118 us against 86); roles with and without a resulting state in two launches
// (gradient at 8 x 2048: 380 against 357).
#include <type_traits>

#include "device_common.hpp"
#include "la_tiles.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kRoom = 8;             // bits of decay between two scalings of the state
constexpr float kMinLog2 = -1.0e4f;  // 2^kMinLog2 == 0 and kMinLog2 * 0 == 0: a decay of exactly 0 works like any other

// log2(lam) of a head, kept finite at the bottom (NaN passes through).
__device__ __forceinline__ float decay_log2(const float* log_decay, int h) {
  const float g = log_decay[h] * kLog2e;
  return g < kMinLog2 ? kMinLog2 : g;
}

// lam^n.  A state passes through thousands of these factors, so they are formed in float64
// and applied as a float32 pair hi + lo: the rounding of lam^n alone would grow to
// n_chunks * 2^-24 over the head's memory.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ double decay_power(const float* log_decay, int h, int n) {
  return n == 0 ? 1.0 : exp(static_cast<double>(log_decay[h]) * n);
}
// (hi is strictly below d and lo above 0, so that an infinite x stays what it is: hi x + lo x would be a NaN with
// lo 0 or of the other sign.  The sum is exact to float32 in either case.)
__device__ __forceinline__ Pair pair_of(double d) {
  float hi = static_cast<float>(d);
  if (d > 0.0 && static_cast<double>(hi) >= d) hi = __builtin_bit_cast(float, __builtin_bit_cast(int, hi) - 1);
  return Pair{hi, static_cast<float>(d - static_cast<double>(hi))};
}
__device__ __forceinline__ float times(const Pair& d, float x) { return __builtin_fmaf(d.hi, x, d.lo * x); }
// lam^n to float32 accuracy at any n: the exponent is reduced in float64.  (exp(), of which the
// factors above take a few a workgroup, costs about a microsecond.)
__device__ __forceinline__ float decay_float(const float* log_decay, int h, int n) {
  double x = static_cast<double>(log_decay[h]) * 1.4426950408889634 * n;
  if (n == 0) x = 0.0;                              // (a decay of exactly 0)
  x = x < -1.0e4 ? -1.0e4 : x > 1.0e4 ? 1.0e4 : x;  // (NaN passes through)
  const double whole = __builtin_floor(x);
  return __builtin_ldexpf(exp2_hw(static_cast<float>(x - whole)), static_cast<int>(whole));
}

__device__ __forceinline__ double uniform_double(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = static_cast<uint32_t>(uniform_int(static_cast<int>(u))),
                 hi = static_cast<uint32_t>(uniform_int(static_cast<int>(u >> 32)));
  return __builtin_bit_cast(double, lo | (hi << 32));
}

__device__ __forceinline__ int row_length(const LaArgs& p, int64_t b) {
  const int L = static_cast<int>(p.L);
  if (!p.lengths) return L;
  const int n = uniform_int(p.lengths[b]);
  return n < 0 ? 0 : (n > L ? L : n);
}

// One tensor's rows into its LDS tile.  Whole chunks take the short way: a uniform address that moves
// on by a chunk, and for each of the wave's instructions (1024 bytes, 64 lanes of 16) the lane's offset,
// formed once.  Scalar work inside the loop costs a chunk dearly (4 x 2048, 80 heads of 64: 138 us with the
// addresses of loads and stores formed there, 122 without).
template <typename ELEM, int RB, int NW, bool PERM>
struct TileLoad {
  static constexpr bool kF32 = sizeof(ELEM) == 4;
  static constexpr int kSlots = RB / 16, kRows = 64 / kSlots;       // slots of a row, rows of an instruction
  static constexpr int kInstr = kQ / kRows / NW;                    // instructions of a wave
  const char* next;                   // lowest address of the chunk to load next
  int64_t move;                       // bytes from a chunk to the next
  uint32_t off[kInstr];

  static __device__ __forceinline__ int slot_of(int row, int lane) {   // (the swizzle is linear in the row's bits)
    return (lane % kSlots) ^ swizzle<RB, kF32, PERM>(row);
  }
  // step: elements from a row to the next (negative: backwards)
  __device__ __forceinline__ void start(const ELEM* base, int64_t step, int chunk, int w, int lane) {
    const int64_t bytes = step * static_cast<int64_t>(sizeof(ELEM));
    move = kQ * bytes;
    next = reinterpret_cast<const char*>(base) + chunk * move + (bytes < 0 ? (kQ - 1) * bytes : 0);
#pragma unroll
    for (int i = 0; i < kInstr; ++i) {
      const int row = (w * kInstr + i) * kRows + lane / kSlots;
      off[i] = static_cast<uint32_t>(bytes < 0 ? kQ - 1 - row : row) * static_cast<uint32_t>(bytes < 0 ? -bytes : bytes) +
               static_cast<uint32_t>(slot_of(row, lane) * 16);
    }
  }
  // ALL: every column is there; else those past `cols` are left as they are (zeros, from the start).
  template <bool ALL>
  __device__ __forceinline__ void whole(uint32_t tile, int cols, int w, int lane) {
#pragma unroll
    for (int i = 0; i < kInstr; ++i)
      if (ALL || slot_of((w * kInstr + i) * kRows + lane / kSlots, lane) * 16 < cols * static_cast<int>(sizeof(ELEM)))
        load_to_lds(tile + (w * kInstr + i) * 1024, next, off[i]);
    next += move;
  }
  // The last chunk: rows past `last` repeat it (they are cleared afterwards).
  static __device__ __forceinline__ void part(uint32_t tile, const ELEM* base, int64_t step, int last, int cols, int w,
                                              int lane) {
#pragma unroll 1
    for (int i = 0; i < kInstr; ++i) {
      const int row = (w * kInstr + i) * kRows + lane / kSlots, slot = slot_of(row, lane), r = row < last ? row : last;
      if (slot * 16 < cols * static_cast<int>(sizeof(ELEM)))
        load_to_lds(tile + (w * kInstr + i) * 1024, reinterpret_cast<const char*>(base + r * step) + slot * 16);
    }
  }
};

// The same in 4-byte words, for rows that start at any word: four times the instructions, 256 bytes
// each, at addresses formed where they are used (4 x 2048, 32 heads of 100: 183 us, 527 element by
// element).  A wave fills the same part of the tile.
template <typename ELEM, int RB, int NW, bool PERM>
__device__ __forceinline__ void load_tile_words(uint32_t tile, const ELEM* base, int64_t step, int last, int cols, int w,
                                                int lane) {
  constexpr int kWords = RB / 4, kInstr = kQ * RB / 256 / NW;
  const int64_t bytes = step * static_cast<int64_t>(sizeof(ELEM));
#pragma unroll 4
  for (int i = 0; i < kInstr; ++i) {
    const int word = (w * kInstr + i) * 64 + lane, row = word / kWords, r = row < last ? row : last;
    const int byte = (word % kWords * 4) ^ (swizzle<RB, sizeof(ELEM) == 4, PERM>(row) << 4);
    if (byte < cols * static_cast<int>(sizeof(ELEM)))
      load_word_to_lds(tile + (w * kInstr + i) * 256, reinterpret_cast<const char*>(base) + r * bytes + byte);
  }
}

// The same element by element, for bfloat16 rows that do not even start at a word (rows past `last` as zeros).
template <typename ELEM, int RB, int NW, bool PERM>
__device__ __forceinline__ void load_tile_scalar(char* tile, const ELEM* base, int64_t step, int last, int cols, int tid) {
  constexpr int kCols = RB / sizeof(ELEM);
  for (int i = tid; i < kQ * kCols; i += 64 * NW) {
    const int row = i / kCols, col = i % kCols;
    ELEM x = ELEM(0);
    if (row <= last && col < cols) x = base[row * step + col];
    const int byte = col * static_cast<int>(sizeof(ELEM));
    *reinterpret_cast<ELEM*>(tile + row * RB + (byte ^ (swizzle<RB, sizeof(ELEM) == 4, PERM>(row) << 4))) = x;
  }
}

// STATE_ONLY: the pre-pass, which leaves each segment's own sum (its state after its last
// token, from zero) in role.seg.  Otherwise the whole of the segment's output.
//
// A wave owns 16 VT columns.  VT = 2 at bfloat16, V > 64: each LDS read and address serves two columns'
// tiles, at 256 registers and 2 waves a SIMD; 8 waves of 16 columns took as long with twice the
// instructions (131072 tokens 1065 us, 1061 with two tiles, when both were tried), and only pairs of tiles
// make 64-byte output pieces (1006).
template <typename ACT, int VD>
constexpr int kColumnTiles = sizeof(typename Op<ACT>::elem) == 2 && VD == 128 ? 2 : 1;

// MOVE: the bytes that a lane of a load moves (16, 4; 0: element by element).  ALL: K = KD and V = VD.
// WT: operand terms of the decayed v: 3, or 2 in the main pass of a sequence in segments, where the state that
// is returned comes from the pre-pass and this one only serves outputs, whose products take E in two terms
// (131072 tokens: 916 us with 3, 877 with 2).  It goes by the number of segments alone, so that neither the
// rows' alignment nor whether a state is asked for changes a bit of the outputs.  (With 2 wherever no state is
// returned the gradient at 8 x 2048, 32 heads of 128, took 323 us without dinitial_state, 349 so.)
template <typename ACT, int KD, int VD, int MOVE, bool ALL, bool STATE_ONLY, int WT>
__global__ __launch_bounds__((4 * VD / kColumnTiles<ACT, VD>), VD == 128 || sizeof(typename Op<ACT>::elem) == 4 ? 2 : 3)
void la_kernel(LaArgs p) {
  constexpr int VT = kColumnTiles<ACT, VD>;
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr bool kF32 = sizeof(elem) == 4;
  constexpr int NW = VD / 16 / VT;
  constexpr int RK = KD * static_cast<int>(sizeof(elem)), RV = VD * static_cast<int>(sizeof(elem));   // row bytes
  constexpr int RP = kQ * static_cast<int>(sizeof(elem));
  constexpr int KT = KD / 32;                       // pairs of state tiles along K
  constexpr int ET = kF32 ? 1 : 2;                  // operand terms of E and of P
  __shared__ __attribute__((aligned(512))) char sQ[STATE_ONLY ? 16 : kQ * RK];
  __shared__ __attribute__((aligned(512))) char sKK[2][kQ * RK];                // k of this chunk and of the next
  __shared__ __attribute__((aligned(512))) char sV[kQ * RV];
  __shared__ __attribute__((aligned(512))) char sP[ET][STATE_ONLY ? 16 : kQ * RP];   // P [j][i]

  const int tid = threadIdx.x, lane0 = tid & 63, w = uniform_int(tid >> 6);
  // Workgroup ids go round the 8 XCDs: the roles of one (batch row, head, segment), which
  // read the same rows, are 8 ids apart, on one XCD and its L2 at about the same time.
  // (32-bit numbers: each 64-bit division is 500 cycles of a short call)
  const uint32_t nseg = static_cast<uint32_t>(p.nseg), heads = static_cast<uint32_t>(p.H);
  const uint32_t per_role = static_cast<uint32_t>(p.batch) * heads * nseg, span = 8u * static_cast<uint32_t>(p.nroles);
  const uint32_t group = blockIdx.x / span, in_group = blockIdx.x - group * span, item = group * 8 + in_group % 8;
  if (item >= per_role) return;
  const LaRole& r = p.role[in_group / 8];
  const uint32_t pair = nseg == 1 ? item : item / nseg, seg = item - pair * nseg, row_b = pair / heads;
  if (STATE_ONLY && seg + 1 == nseg && !r.fin) return;   // (its sum would be read by nobody)
  const int64_t bh = pair, b = row_b;
  const int h = static_cast<int>(pair - row_b * heads);
  const int L = static_cast<int>(p.L);
  const int len = row_length(p, b);
  const int K = r.K, V = r.V, reverse = r.reverse;
  const int nchunks = (L + kQ - 1) / kQ;
  const int live = (len + kQ - 1) / kQ;             // chunks that hold a token
  const int c_begin = static_cast<int>(seg) * static_cast<int>(p.seg_chunks);
  const int c_stop = c_begin + static_cast<int>(p.seg_chunks);
  const int c_end = c_stop < nchunks ? c_stop : nchunks;
  const int c_live = c_end < live ? c_end : live;
  const float g2 = decay_log2(p.log_decay, h);

  // row r of the sequence is token r forwards, len - 1 - r backwards
  const int64_t t_first = reverse ? len - 1 : 0;
  const int t_step = reverse ? -1 : 1;
  const elem* qg = static_cast<const elem*>(r.q) + b * r.qs[0] + (r.qdiv == 1 ? h : h / r.qdiv) * r.qs[2] + t_first * r.qs[1];
  const elem* kg = static_cast<const elem*>(r.k) + b * r.ks[0] + (r.kdiv == 1 ? h : h / r.kdiv) * r.ks[2] + t_first * r.ks[1];
  const elem* vg = static_cast<const elem*>(r.v) + b * r.vs[0] + (r.vdiv == 1 ? h : h / r.vdiv) * r.vs[2] + t_first * r.vs[1];
  const int64_t qstep = r.qs[1] * t_step, kstep = r.ks[1] * t_step, vstep = r.vs[1] * t_step;

  // Ask for the rows of k, or of q and v, of chunk c (in order, from c_begin).
  TileLoad<elem, RK, NW, true> k_load;
  TileLoad<elem, RK, NW, false> q_load;
  TileLoad<elem, RV, NW, false> v_load;
  auto load_k = [&](auto plain, int c, int lane) __attribute__((always_inline)) {
    constexpr bool PLAIN = decltype(plain)::value;
    const int last = len - 1 - c * kQ;
    const int64_t r0 = static_cast<int64_t>(c) * kQ;
    const uint32_t tile = lds_address(sKK[0]) + (c & 1) * (kQ * RK);
    if constexpr (MOVE == 16) {
      if (PLAIN || last >= kQ - 1) k_load.template whole<ALL>(tile, K, w, lane);
      else k_load.part(tile, kg + r0 * kstep, kstep, last, K, w, lane);
    } else if constexpr (MOVE == 4) {
      load_tile_words<elem, RK, NW, true>(tile, kg + r0 * kstep, kstep, last, K, w, lane);
    } else {
      load_tile_scalar<elem, RK, NW, true>(sKK[c & 1], kg + r0 * kstep, kstep, last, K, tid);
    }
  };
  auto load_qv = [&](auto plain, int c, int lane) __attribute__((always_inline)) {
    constexpr bool PLAIN = decltype(plain)::value;
    const int last = len - 1 - c * kQ;
    const int64_t r0 = static_cast<int64_t>(c) * kQ;
    if constexpr (MOVE == 16) {
      if (PLAIN || last >= kQ - 1) {
        if constexpr (!STATE_ONLY) q_load.template whole<ALL>(lds_address(sQ), K, w, lane);
        v_load.template whole<ALL>(lds_address(sV), V, w, lane);
      } else {
        if constexpr (!STATE_ONLY) q_load.part(lds_address(sQ), qg + r0 * qstep, qstep, last, K, w, lane);
        v_load.part(lds_address(sV), vg + r0 * vstep, vstep, last, V, w, lane);
      }
    } else if constexpr (MOVE == 4) {
      if constexpr (!STATE_ONLY)
        load_tile_words<elem, RK, NW, false>(lds_address(sQ), qg + r0 * qstep, qstep, last, K, w, lane);
      load_tile_words<elem, RV, NW, false>(lds_address(sV), vg + r0 * vstep, vstep, last, V, w, lane);
    } else {
      if constexpr (!STATE_ONLY) load_tile_scalar<elem, RK, NW, false>(sQ, qg + r0 * qstep, qstep, last, K, tid);
      load_tile_scalar<elem, RV, NW, false>(sV, vg + r0 * vstep, vstep, last, V, tid);
    }
  };
  // Waits for this wave's part of chunk c's rows (and for its stores of the chunk before).
  auto arrived = [&](int c, int n, int lane) __attribute__((always_inline)) {
    if constexpr (MOVE > 0) {
      __builtin_amdgcn_s_waitcnt(0x0f70);           // vmcnt(0); expcnt and lgkmcnt as they are
      if (n < kQ) {
        clear_tile<RK, NW>(sKK[c & 1], n, w, lane);
        if constexpr (!STATE_ONLY) clear_tile<RK, NW>(sQ, n, w, lane);
        clear_tile<RV, NW>(sV, n, w, lane);
      }
    }
  };
  auto present = [&](int c) { return len - c * kQ < kQ ? len - c * kQ : kQ; };
  // The walk begins: the first chunk's rows are asked for.
  auto ask = [&]() __attribute__((always_inline)) {
    if constexpr (MOVE == 16) {
      k_load.start(kg, kstep, c_begin, w, lane0);
      if constexpr (!STATE_ONLY) q_load.start(qg, qstep, c_begin, w, lane0);
      v_load.start(vg, vstep, c_begin, w, lane0);
    }
    if constexpr (MOVE > 0) {
      if (!ALL) {                                   // columns that the loads leave alone
        clear_tile<RK, NW>(sKK[0], 0, w, lane0);
        clear_tile<RK, NW>(sKK[1], 0, w, lane0);
        if constexpr (!STATE_ONLY) clear_tile<RK, NW>(sQ, 0, w, lane0);
        clear_tile<RV, NW>(sV, 0, w, lane0);
        __builtin_amdgcn_s_waitcnt(0xc07f);         // lgkmcnt(0): before the loads into the same slots
      }
    }
    if (c_begin < c_live) {
      load_k(std::false_type{}, c_begin, lane0);
      load_qv(std::false_type{}, c_begin, lane0);
    }
  };
  ask();

  const int g = lane0 >> 4, c16 = lane0 & 15;
  // E[vt][t][u][e] is the entry k = 32 t + 8 g + 4 u + e, v = 16 (VT w + vt) + c16
  f32x4_t E[VT][KT][2];
  const float* src = nullptr;
  if (!STATE_ONLY) {
    if (nseg > 1) src = r.seg + (bh * nseg + seg) * static_cast<int64_t>(K) * V;
    else if (r.carry) src = r.carry + bh * static_cast<int64_t>(K) * V;
  }
  // this lane's place in a state in memory, and of its entries from there
  auto entry = [&](int vt, int t, int u, int e) { return (32 * t + 4 * u + e) * r.sk + 16 * vt * r.sv; };
  auto there = [&](int vt, int t, int u, int e) {
    return ALL || (32 * t + 8 * g + 4 * u + e < K && 16 * (VT * w + vt) + c16 < V);
  };
  const int place = 8 * g * r.sk + (16 * VT * w + c16) * r.sv;
  // forwards the carried state decays once before the first token; the segments' states have
  const float first = nseg > 1 || reverse || len == 0 ? 1.0f : exp2_hw(g2);
  const bool scaled = c_begin < c_live;             // (below)
  const float entering = scaled ? first * (1.0f / (1 << kRoom)) : first;
  auto enter = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) E[vt][t][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (src) {                                      // (one branch, so that all loads are under way together)
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              E[vt][t][u][e] = src[static_cast<uint32_t>(there(vt, t, u, e) ? place + entry(vt, t, u, e) : 0)];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) E[vt][t][u][e] = there(vt, t, u, e) ? E[vt][t][u][e] * entering : 0.0f;
    }
  };
  enter();

  // The registers hold the state divided by rho = 2^kRoom lam^(64 a), a the chunks since the last
  // time they were scaled back: a chunk then adds lam^(64 - i) v / rho' instead of decaying every entry.
  // Past 2^kRoom of decay the registers are scaled back to a = 0, by a float32 pair from float64, so that no
  // rounding of lam^64 builds up over the thousands of chunks of a head's memory.  rho stays at 1 and more:
  // what the registers hold is never larger than the state itself, so it overflows only where that does (and
  // states below 2^(kRoom - 126) lose bits).
  const double lam_q = uniform_double(decay_power(p.log_decay, h, kQ));
  const double unlam_q = uniform_double(1.0 / lam_q);
  const float g_q = g2 * kQ;
  constexpr double kUp = 1 << kRoom, kDown = 1.0 / kUp;
  int a = 0;
  double rho = scaled ? kUp : 1.0, unrho = kDown;                 // and its inverse
  auto scale_state = [&](double by) __attribute__((always_inline)) {
    const Pair d = pair_of(by);
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) E[vt][t][u][e] = times(d, E[vt][t][u][e]);
  };
  // The last chunk of the sequence (of the segment, in the pre-pass) forwards leaves S, not lam S,
  // and may hold fewer tokens.
  const int n_end = uniform_int(c_begin < c_live ? present(c_live - 1) : 0);
  const int shift = uniform_int((STATE_ONLY || !reverse) && (STATE_ONLY || c_live == live) ? 1 : 0);
  const double lam_end = uniform_double(decay_power(p.log_decay, h, n_end - shift > 0 ? n_end - shift : 0));

  // Tiles of P (16 tokens j by 16 of 32 tokens i; those right of the diagonal are neither formed nor read).
  // 4 waves: three each, (j rows w, the first 32 i) and one tile u of (j rows 2 or 3, the second
  // 32 i).  8 waves: two each, (j rows w % 4, half w / 4 of the i).  Their weights lam^(j-i):
  constexpr bool kThree = NW == 4;
  const int i_half = kThree ? 0 : w >> 2, j_tile = w & 3, j_third = 2 + (w & 1), u_third = uniform_int(w < 2 ? 1 : 0);
  const float io_scale = r.in_scale * r.out_scale;
  const int off0 = 16 * j_tile + c16 - 32 * i_half - 8 * g, off3 = 16 * j_third + c16 - 32 - 8 * g - 4 * u_third;
  auto decay_of = [&](int n) { return exp2_hw(g2 * static_cast<float>(n > 0 ? n : 0)); };
  float pm[8], pm3[4];
  if constexpr (!STATE_ONLY) {
#pragma unroll
    for (int e = 0; e < 8; ++e) pm[e] = decay_of(off0 - e) * io_scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) pm3[e] = decay_of(off3 - e) * io_scale;
  }
  float pw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) pw[e] = uniform_float(exp2_hw(g2 * static_cast<float>(7 - e)));
  float pj[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) pj[jt] = uniform_float(exp2_hw(g2 * static_cast<float>(16 * jt)));
  const float out_decay = exp2_hw(g2 * static_cast<float>(c16)) * r.out_scale;
  const float in_decay = exp2_hw(g2 * static_cast<float>(kQ - 32 - 8 * g - 7)) * r.in_scale;

  // where the output rows of a whole chunk go: backwards, row r of the chunk is 63 - r rows up
  const bool o_f32 = kF32 || r.o_f32;
  char *o_first = nullptr, *o_next = nullptr;
  int64_t o_move = 0;
  uint32_t o_off = 0, o_rows = 0;
  if constexpr (!STATE_ONLY && MOVE == 16) {
    const int esz = o_f32 ? 4 : 2;
    const int64_t bytes = static_cast<int64_t>(p.H) * V * esz, r0 = static_cast<int64_t>(c_begin) * kQ;
    o_first = static_cast<char*>(r.o) + (b * L + (reverse ? len - kQ - r0 : r0)) * bytes + static_cast<int64_t>(h) * V * esz;
    o_next = o_first;
    o_move = (reverse ? -kQ : kQ) * bytes;
    const int col = VT == 2 && esz == 2 ? 16 * VT * w + (g & 1) * 16 + (g >> 1) * 8 : 16 * VT * w + 4 * g;
    o_rows = static_cast<uint32_t>(reverse ? -16 * bytes : 16 * bytes);
    o_off = static_cast<uint32_t>((reverse ? kQ - 1 - c16 : c16) * bytes + col * esz);
  }

  if (c_begin < c_live) arrived(c_begin, present(c_begin), lane0);
  // One chunk.  PLAIN: it and the next are whole, so that nothing is decided inside: with one or two
  // waves a SIMD each branch taken costs its fetch (the gradient at 8 x 2048, 32 heads of 128: 398 us with one
  // loop for every chunk, 358 with one of their own for these).
  auto chunk = [&](auto plain, auto careful, int c) __attribute__((always_inline)) {
    constexpr bool PLAIN = decltype(plain)::value, CAREFUL = decltype(careful)::value;
    const int n = PLAIN ? kQ : present(c);
    const bool more = PLAIN || c + 1 < c_live;
    // (opaque, so that the chunk's many LDS and memory addresses are formed here from the lane's
    // number: kept in registers over the loop they crowd out the state)
    int lane = lane_id();
    asm volatile("" : "+v"(lane));
    const int g = lane >> 4, c16 = lane & 15;
    barrier_lds();                                  // the tiles of chunk c are complete
    const uint32_t k_tile = lds_address(sKK[0]) + (c & 1) * (kQ * RK);
    constexpr int PB = O::kPiece;
    const uint32_t q_rows = O::template row_part<RK, false>(lds_address(sQ), c16, g);
    const uint32_t p_rows = O::template row_part<RP, false>(lds_address(sP[0]), c16, g);
    if (more) load_k(plain, c + 1, lane);

    // ---- P: tiles of k q^T, rows i = 32 t + 8 g + 4 u + e, column j = c16
    if constexpr (!STATE_ONLY) {
      const uint32_t k_rows = O::template row_part<RK, true>(k_tile, 8 * (c16 >> 2) + (c16 & 3), g);
      if (kThree || i_half == 0 || j_tile >= 2) {
        f32x4_t s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) s[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < KT; ++x) {
          const piece qf = O::row(q_rows + j_tile * (16 * RK), 4 * PB * x, 0);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            s[u] = O::mma(O::row(k_rows + i_half * (32 * RK), (4 * PB * x) ^ (swizzle<RK, kF32, true>(4 * u) << 4),
                                 4 * u * RK), qf, s[u]);
        }
        float pv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pv[e] = off0 >= e ? s[e / 4][e % 4] * pm[e] : 0.0f;
        piece ps[ET];
        O::template split<ET>(pv, ps);
#pragma unroll
        for (int m = 0; m < ET; ++m) O::put((p_rows ^ (4 * PB * i_half)) + j_tile * (16 * RP), 0, m * (kQ * RP), ps[m]);
      }
      if constexpr (kThree) {
        f32x4_t s = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        const int flip = u_third ? swizzle<RK, kF32, true>(4) << 4 : 0, offset = 32 * RK + u_third * (4 * RK);
#pragma unroll
        for (int x = 0; x < KT; ++x)
          s = O::mma(O::row(k_rows, (4 * PB * x) ^ flip, offset), O::row(q_rows + j_third * (16 * RK), 4 * PB * x, 0), s);
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pv[e] = off3 >= e ? s[e] * pm3[e] : 0.0f;
        typename O::half ps[ET];
        O::template split4<ET>(pv, ps);
        const uint32_t at = (p_rows ^ (4 * PB) ^ (u_third ? O::half_flip(1) : 0)) + (u_third ? O::half_offset(1) : 0) +
                            j_third * (16 * RP);
#pragma unroll
        for (int m = 0; m < ET; ++m) O::put_half(at + m * (kQ * RP), ps[m]);
      }
    }

    // ---- the wave's own columns of v
    piece vf[VT][2];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      const uint32_t v_cols = O::template column_part<RV, false>(lds_address(sV), 16 * (VT * w + vt), 4, lane);
#pragma unroll
      for (int t = 0; t < 2; ++t) vf[vt][t] = O::template column<RV, false>(v_cols, 0, 32 * t * RV);
    }

    // ---- output from the carried state, transposed: acc[vt][jt] = rows v, column j = 16 jt + c16
    f32x4_t acc[VT][4];
    if constexpr (!STATE_ONLY) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) acc[vt][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        piece q[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) q[jt] = O::row(q_rows, 4 * PB * t, 16 * jt * RK);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          piece ef[ET];
          const float x[8] = {E[vt][t][0][0], E[vt][t][0][1], E[vt][t][0][2], E[vt][t][0][3],
                              E[vt][t][1][0], E[vt][t][1][1], E[vt][t][1][2], E[vt][t][1][3]};
          O::template split<ET>(x, ef);
#pragma unroll
          for (int m = 0; m < ET; ++m)
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) acc[vt][jt] = O::mma(ef[m], q[jt], acc[vt][jt]);
        }
      }
    }
    barrier_lds();                                  // P complete; the tiles of q and v are free
    if (more) load_qv(plain, c + 1, lane);

    // ---- P v, transposed, on top
    if constexpr (!STATE_ONLY) {
      const float f0 = out_decay * static_cast<float>(rho);
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const float f = f0 * pj[jt];
#pragma unroll
        for (int vt = 0; vt < VT; ++vt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[vt][jt][e] *= f;
      }
      if constexpr (!CAREFUL) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          piece pf[4][ET];
#pragma unroll
          for (int jt = 0; jt < 4; ++jt)
#pragma unroll
            for (int m = 0; m < ET; ++m)
              if (t == 0 || jt >= 2) pf[jt][m] = O::row(p_rows, 4 * PB * t, 16 * jt * RP + m * (kQ * RP));
#pragma unroll
          for (int m = 0; m < ET; ++m)
#pragma unroll
            for (int vt = 0; vt < VT; ++vt)
#pragma unroll
              for (int jt = 0; jt < 4; ++jt)
                if (t == 0 || jt >= 2) acc[vt][jt] = O::mma(vf[vt][t], pf[jt][m], acc[vt][jt]);
        }
      } else {
        // without the values that are not finite: a zero of P times one is NaN.  The rows from its token on are.
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          int gone = kQ;                            // first such token of column c16
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float x[8];
            O::unpack(vf[vt][t], x);
#pragma unroll
            for (int e = 7; e >= 0; --e)
              if (!(fabsf(x[e]) < __builtin_huge_valf())) {
                x[e] = 0.0f;
                gone = least(gone, 32 * t + 8 * g + e);
              }
            const piece clean = O::pack(x);
#pragma unroll
            for (int m = 0; m < ET; ++m) {
              __builtin_amdgcn_sched_barrier(0);    // (few registers before speed here)
#pragma unroll
              for (int jt = 2 * t; jt < 4; ++jt)
                acc[vt][jt] = O::mma(clean, O::row(p_rows, 4 * PB * t, 16 * jt * RP + m * (kQ * RP)), acc[vt][jt]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          gone = least(gone, __shfl_xor(gone, 16));
          gone = least(gone, __shfl_xor(gone, 32));
#pragma unroll
          for (int e = 0; e < 4; ++e) {             // (the output's columns are the lanes' columns of v)
            const int from = __shfl(gone, 4 * g + e);
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
              if (16 * jt + c16 >= from) acc[vt][jt][e] = __builtin_nanf("");
          }
        }
      }
      if (!PLAIN && n < kQ) {
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
          if (16 * jt + c16 >= n) {
#pragma unroll
            for (int vt = 0; vt < VT; ++vt) acc[vt][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          }
      }
    }

    // ---- the state: lam^n E + k^T (lam^(n-i) v)
    const bool whole = more || n - shift == kQ;
    if (__builtin_expect(whole && fabsf(g_q * static_cast<float>(a + 1)) < static_cast<float>(kRoom), 1)) {
      ++a;
      rho *= lam_q;
      unrho *= unlam_q;
    } else {
      scale_state((whole ? lam_q : lam_end) * (rho * kDown));      // (with the decay of the chunk just done)
      a = 0;
      rho = kUp;
      unrho = kDown;
    }
    const float wc = in_decay * static_cast<float>(unrho);
    const uint32_t k_cols = O::template column_part<RK, true>(k_tile, 0, 8, lane);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float wgt[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) wgt[e] = (t == 0 ? wc * pj[2] : wc) * pw[e];
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int left = n - shift - (32 * t + 8 * g + e);
          wgt[e] = exp2_hw(g2 * static_cast<float>(left > 0 ? left : 0)) * (r.in_scale * static_cast<float>(kDown));
          asm volatile("" : "+v"(wgt[e]));
        }
      }
      piece wv[VT][WT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        float x[8];
        O::unpack(vf[vt][t], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= wgt[e];
        O::template split<WT>(x, wv[vt]);
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        piece kf[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          kf[u] = O::template column<RK, true>(k_cols, (4 * PB * kt) ^ O::half_flip(u), 32 * t * RK + O::half_offset(u));
#pragma unroll
        for (int m = 0; m < WT; ++m)
#pragma unroll
          for (int vt = 0; vt < VT; ++vt)
#pragma unroll
            for (int u = 0; u < 2; ++u) E[vt][kt][u] = O::mma(kf[u], wv[vt][m], E[vt][kt][u]);
      }
    }
    // (without a next chunk there is nothing to clear)
    arrived(c + 1, !PLAIN && more ? present(c + 1) : kQ, lane);

    // ---- the output rows to memory: lane (g, c) has 4 columns of row 16 jt + c.  They are issued after
    // the wait for the next chunk's rows, so that a wait covers only the stores of the chunk before.
    if constexpr (!STATE_ONLY) {
      auto put = [&](auto* out) __attribute__((always_inline)) {
        using OUT = std::remove_pointer_t<decltype(out)>;
        auto four = [](const f32x4_t& a) __attribute__((always_inline)) {
          if constexpr (sizeof(OUT) == 4) return make_float4(a[0], a[1], a[2], a[3]);
          else return make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
        };
        if (PLAIN || (MOVE == 16 && n == kQ)) {
          // a uniform address that moves on by a chunk, the lane's offset in 16 rows, 16 rows' bytes
          constexpr bool kEight = VT == 2 && sizeof(OUT) == 2;   // columns of a lane, otherwise 4
#pragma unroll
          for (int jt = 0; jt < 4; ++jt) {
            char* rows = o_next + (o_off + static_cast<uint32_t>(jt) * o_rows);
            if constexpr (kEight) {
              // lane groups 2x and 2x + 1 exchange halves: 8 columns a lane, 64 bytes of a row an instruction
              const uint2 a0 = four(acc[0][jt]), a1 = four(acc[1][jt]);
              const auto lo = __builtin_amdgcn_permlane16_swap(a0.x, a1.x, false, false);
              const auto hi = __builtin_amdgcn_permlane16_swap(a0.y, a1.y, false, false);
              if (ALL || 32 * w + (g & 1) * 16 + (g >> 1) * 8 < V)
                *reinterpret_cast<uint4*>(rows) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
            } else {
#pragma unroll
              for (int vt = 0; vt < VT; ++vt)
                if (ALL || 16 * (VT * w + vt) + 4 * g < V)
                  *reinterpret_cast<decltype(four(acc[0][0]))*>(rows + 16 * vt * sizeof(OUT)) = four(acc[vt][jt]);
            }
          }
          o_next += o_move;
          return;
        }
        const int64_t row_stride = static_cast<int64_t>(p.H) * V;
        const int r0 = c * kQ;
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
          const int row = r0 + 16 * jt + c16;
          if (row >= L) continue;
          const int64_t token = reverse && row < len ? len - 1 - row : row;
          OUT* o = out + (b * L + token) * row_stride + static_cast<int64_t>(h) * V;
#pragma unroll
          for (int vt = 0; vt < VT; ++vt) {
            const int v0 = 16 * (VT * w + vt) + 4 * g;
            if (MOVE == 16 || r.o_vec) {
              if (v0 < V) *reinterpret_cast<decltype(four(acc[0][0]))*>(o + v0) = four(acc[vt][jt]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (v0 + e >= V) continue;
                if constexpr (sizeof(OUT) == 4) o[v0 + e] = acc[vt][jt][e];
                else o[v0 + e] = to_bf16(acc[vt][jt][e]);
              }
            }
          }
        }
      };
      if (o_f32) put(static_cast<float*>(r.o));
      else put(static_cast<uint16_t*>(r.o));
    }
  };
  int c = c_begin;
  if constexpr (MOVE == 16) {
    const int last = (c_live < len / kQ ? c_live : len / kQ) - 1;
    for (; c < last; ++c) chunk(std::true_type{}, std::false_type{}, c);
  }
  for (; c < c_live; ++c) chunk(std::false_type{}, std::false_type{}, c);

  // A value of v that is not finite must not reach the outputs before it, but in its own chunk P's zeros times it
  // did.  It stays in every entry of its column of E, so one entry a column tells, here at the end and
  // without a word in the loop; the walk is then made once more with care.  (q's tile is free: it holds
  // the waves' findings.)
  if constexpr (!STATE_ONLY) {
    if (scaled) {
      float z = E[0][0][0][0] * 0.0f;
      if constexpr (VT == 2) z += E[1][0][0][0] * 0.0f;
      const bool found = __builtin_amdgcn_ballot_w64(z != z) != 0;
      const uint32_t at = lds_address(sQ);
      if (lane0 == 0) lds_write<int>(at + 4 * w, found);
      barrier_lds();
      int any = 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) any |= lds_read<int>(at + 4 * i);
      if (__builtin_expect(uniform_int(any), 0)) {
        barrier_lds();                              // (everyone has read them)
        if (lane0 == 0) lds_write<int>(at + 4 * w, 0);
        barrier_lds();
        ask();
        enter();
        a = 0;
        rho = kUp;
        unrho = kDown;
        o_next = o_first;
        arrived(c_begin, present(c_begin), lane0);
#pragma unroll 1
        for (c = c_begin; c < c_live; ++c) chunk(std::false_type{}, std::true_type{}, c);
      }
    }
  }

  // chunks with no token: zeros
  if constexpr (!STATE_ONLY) {
    for (int64_t z = c_live > c_begin ? c_live : c_begin; z < c_end; ++z) {
      for (int i = tid; i < kQ * V; i += 64 * NW) {
        const int64_t token = z * kQ + i / V;
        if (token >= L) break;
        const int64_t o = ((b * L + token) * p.H + h) * V + i % V;
        if (r.o_f32 || kF32) static_cast<float*>(r.o)[o] = 0.0f;
        else static_cast<uint16_t*>(r.o)[o] = 0;
      }
    }
  }

  float* dst = nullptr;
  if (STATE_ONLY) dst = r.seg + (bh * nseg + seg) * static_cast<int64_t>(K) * V;
  else if (nseg == 1 && r.fin) dst = r.fin + bh * static_cast<int64_t>(K) * V;
  if (dst) {
    scale_state(rho);
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (there(vt, t, u, e)) dst[static_cast<uint32_t>(place + entry(vt, t, u, e))] = E[vt][t][u][e];
  }
}

// Chains the segments' own sums T_s into the E entering each segment (written over T_s) and
// the state after the last token.  A thread takes kChain entries 256 apart and reads kAhead segments'
// sums at a time: only the arithmetic is a chain.
constexpr int kChain = 4, kAhead = 8;
__global__ __launch_bounds__(256) void la_chain_kernel(LaArgs p) {
  const LaRole& r = p.role[blockIdx.z];
  const uint32_t row_b = blockIdx.y / static_cast<uint32_t>(p.H);
  const int64_t bh = blockIdx.y;
  const int KV = r.K * r.V;
  const int i0 = blockIdx.x * (256 * kChain) + threadIdx.x;
  const int h = static_cast<int>(blockIdx.y - row_b * static_cast<uint32_t>(p.H));
  const int len = row_length(p, row_b);
  const int seg_tokens = static_cast<int>(p.seg_chunks) * kQ;
  float* slot = r.seg + bh * p.nseg * static_cast<int64_t>(KV);
  const float* carry = r.carry ? r.carry + bh * static_cast<int64_t>(KV) : nullptr;
  float* fin = r.fin ? r.fin + bh * static_cast<int64_t>(KV) : nullptr;
  auto tokens = [&](int k) {
    const int left = len - k * seg_tokens;
    return left < 0 ? 0 : (left < seg_tokens ? left : seg_tokens);
  };
  float s[kChain], T[kAhead][kChain];
#pragma unroll
  for (int x = 0; x < kChain; ++x) s[x] = carry && i0 + 256 * x < KV ? carry[i0 + 256 * x] : 0.0f;
  float l1 = 0.0f;
  Pair lS{0.0f, 0.0f};                              // (the factor that a state meets once a segment; the others, once)
  for (int k0 = 0; k0 < p.nseg; k0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u;
      const bool read = k < p.nseg && tokens(k) > 0 && (k + 1 < p.nseg || fin);   // (the others were not written)
#pragma unroll
      for (int x = 0; x < kChain; ++x)
        T[u][x] = read && i0 + 256 * x < KV ? slot[static_cast<int64_t>(k) * KV + i0 + 256 * x] : 0.0f;
    }
    if (k0 == 0) {                                  // (while the first sums are on their way)
      l1 = decay_float(p.log_decay, h, 1);
      lS = pair_of(decay_power(p.log_decay, h, seg_tokens));
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u;
      if (k >= p.nseg) break;
      const int n = tokens(k);
      const Pair d = n == seg_tokens ? lS : pair_of(static_cast<double>(decay_float(p.log_decay, h, n)));
#pragma unroll
      for (int x = 0; x < kChain; ++x) {
        if (i0 + 256 * x < KV) slot[static_cast<int64_t>(k) * KV + i0 + 256 * x] = r.reverse ? s[x] : l1 * s[x];
        if (n > 0) s[x] = times(d, s[x]) + (r.reverse ? l1 * T[u][x] : T[u][x]);
      }
    }
  }
  if (fin) {
#pragma unroll
    for (int x = 0; x < kChain; ++x)
      if (i0 + 256 * x < KV) fin[i0 + 256 * x] = s[x];
  }
}

// Sums over the state heads that share a head, of one or two tensors.  W values a thread, a row of d
// values by d / W threads, rows a grid apart (so that nothing is divided but the thread's number).
template <typename ACT, int W>
__global__ __launch_bounds__(256) void la_sum_heads_kernel(LaSum a, LaSum b) {
  const LaSum& x = blockIdx.y ? b : a;
  const int per_row = x.d / W, rows = 256 / per_row, t = threadIdx.x / per_row, c = threadIdx.x % per_row * W;
  if (t >= rows) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows + t; row < x.rows; row += step) {
    const float* src = x.part + row * x.share * x.d + c;
    float s[W];
#pragma unroll
    for (int e = 0; e < W; ++e) s[e] = 0.0f;
    for (int i = 0; i < x.share; ++i, src += x.d) {
      if constexpr (W == 4) {
        const float4 y = *reinterpret_cast<const float4*>(src);
        s[0] += y.x; s[1] += y.y; s[2] += y.z; s[3] += y.w;
      } else {
        s[0] += *src;
      }
    }
    if constexpr (W == 4 && ACT::kBytes == 4)
      *reinterpret_cast<float4*>(static_cast<float*>(x.out) + row * x.d + c) = make_float4(s[0], s[1], s[2], s[3]);
    else if constexpr (W == 4)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(x.out) + row * x.d + c) =
          make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    else
      store_act<ACT>(x.out, row * x.d + c, s[0]);
  }
}

__global__ __launch_bounds__(256) void la_copy_state_kernel(float* dst, const float* src, int64_t n) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) dst[i] = src ? src[i] : 0.0f;
}

template <typename ACT, int KD, int VD>
void launch_la_t(const LaArgs& a, bool state_only, hipStream_t s) {
  const int64_t items = (a.batch * a.H * a.nseg + 7) / 8 * 8;
  const dim3 grid(static_cast<unsigned>(items * a.nroles)), block(4 * VD / kColumnTiles<ACT, VD>);
  constexpr int kTerms = ACT::kBytes == 4 ? 1 : 3;
  auto go = [&](auto move, auto all) {
    constexpr int MOVE = decltype(move)::value;
    constexpr bool ALL = decltype(all)::value;
    if (state_only) hipLaunchKernelGGL((la_kernel<ACT, KD, VD, MOVE, ALL, true, kTerms>), grid, block, 0, s, a);
    else if (kTerms == 1 || a.nseg == 1)
      hipLaunchKernelGGL((la_kernel<ACT, KD, VD, MOVE, ALL, false, kTerms>), grid, block, 0, s, a);
    else if constexpr (kTerms == 3)
      hipLaunchKernelGGL((la_kernel<ACT, KD, VD, MOVE, ALL, false, 2>), grid, block, 0, s, a);
  };
  const LaRole& r = a.role[0];
  if (r.move == 16 && r.K == KD && r.V == VD) go(std::integral_constant<int, 16>{}, std::true_type{});
  else if (r.move == 16) go(std::integral_constant<int, 16>{}, std::false_type{});
  else if (ACT::kBytes == 4 || r.move == 4) go(std::integral_constant<int, 4>{}, std::false_type{});
  else if constexpr (ACT::kBytes == 2) go(std::integral_constant<int, 0>{}, std::false_type{});
}

// One launch for all of `a`'s roles, which are alike (below).
void launch_la_roles(const LaArgs& a, Dt dt, bool state_only, hipStream_t s) {
  const bool k2 = a.role[0].K > 64, v2 = a.role[0].V > 64;
  auto go = [&](auto act) {
    using ACT = decltype(act);
    if (k2 && v2) launch_la_t<ACT, 128, 128>(a, state_only, s);
    else if (k2) launch_la_t<ACT, 128, 64>(a, state_only, s);
    else if (v2) launch_la_t<ACT, 64, 128>(a, state_only, s);
    else launch_la_t<ACT, 64, 64>(a, state_only, s);
  };
  if (dt == Dt::BF16) go(ActBF16{});
  else go(ActF32{});
}

}  // namespace

// Segments per sequence.  Where every CU gets a workgroup, one: the pre-pass and the chaining that
// segments need cost more than they gain (the gradient at 8 x 2048, 32 heads of 128, 768 workgroups: 363 us
// with one, 549 with two; 4 x 2048, 80 heads of 64: 122 with one, 140 with two, 132 with three).  With fewer, 2
// workgroups a CU (131072 tokens, 20 heads of 128: 1332 us with 13, 944 with 25, 992 with 51), each at least 4
// chunks long (float32, 5 x 1000, 16 heads of 64 x 128: 107 us with two, 86 with three, 88 with four, 97 with six).
// The count is then derived back from the segment length, so that no segment is without a chunk.
int la_segments(int64_t batch, int64_t L, int64_t H, int roles) {
  const int64_t workgroups = batch * H * roles, nch = (L + kQ - 1) / kQ;
  if (workgroups >= 256) return 1;
  int64_t s = 512 / (workgroups > 0 ? workgroups : 1);
  if (s > nch / 4) s = nch / 4;
  if (s <= 1) return 1;
  const int64_t per = (nch + s - 1) / s;
  return static_cast<int>((nch + per - 1) / per);
}

// The roles of one call: the forward's one, or dq, dk and dv.  Roles of one tile shape go in one
// launch.  With segments, a pre-pass leaves the states' sums of the forward walk (dq's
// role) and of the backward walk (dv's; dk's is the same state with its axes exchanged, in the same
// memory), and the chain kernel turns them into the states that enter the segments.
hipError_t launch_la(const LaArgs& a, Dt dt, hipStream_t s) {
  const int64_t nchunks = (a.L + kQ - 1) / kQ;
  LaArgs all = a;
  all.seg_chunks = (nchunks + a.nseg - 1) / a.nseg;
  // launches `n` of all's roles, those of one tile shape and form together
  auto fits = [](const LaRole& r) { return r.K % 64 == 0 && r.V % 64 == 0; };   // no column of its tiles is empty
  auto run = [&](const int* which, int n, bool state_only) {
    bool done[3] = {};
    for (int i = 0; i < n; ++i) {
      if (done[i]) continue;
      const LaRole& r = all.role[which[i]];
      LaArgs x = all;
      x.nroles = 0;
      for (int j = i; j < n; ++j) {
        const LaRole& o = all.role[which[j]];
        if ((o.K > 64) != (r.K > 64) || (o.V > 64) != (r.V > 64) || o.move != r.move || fits(o) != fits(r)) continue;
        x.role[x.nroles++] = o;
        done[j] = true;
      }
      launch_la_roles(x, dt, state_only, s);
    }
  };
  static constexpr int kAll[3] = {0, 1, 2}, kStates[2] = {0, 2};
  if (a.nseg > 1) {
    const int n = a.nroles > 1 ? 2 : 1;
    run(kStates, n, true);
    LaArgs x = all;
    x.role[1] = all.role[2];
    const dim3 grid(static_cast<unsigned>((a.role[0].K * a.role[0].V + 256 * kChain - 1) / (256 * kChain)),
                    static_cast<unsigned>(a.batch * a.H),
                    static_cast<unsigned>(n));
    hipLaunchKernelGGL(la_chain_kernel, grid, dim3(256), 0, s, x);
  }
  run(kAll, a.nroles, false);
  return hipGetLastError();
}

hipError_t launch_la_sum_heads(const LaSum* sums, int n, Dt dt, hipStream_t s) {
  for (int i = 0; i < n;) {                         // two of one width go in one launch
    const LaSum &a = sums[i], &b = i + 1 < n && sums[i + 1].d == a.d ? sums[i + 1] : a;
    const int both = &a == &b ? 1 : 2;
    const int64_t most = a.rows > b.rows ? a.rows : b.rows;
    auto vector = [](const LaSum& x) { return x.d % 4 == 0 && reinterpret_cast<uintptr_t>(x.out) % 16 == 0; };
    auto go = [&](auto act, auto width) {
      constexpr int W = decltype(width)::value;
      const int64_t rows = 256 / (a.d / W), blocks = (most + rows - 1) / rows;
      const dim3 grid(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), both);
      hipLaunchKernelGGL((la_sum_heads_kernel<decltype(act), W>), grid, dim3(256), 0, s, a, b);
    };
    const bool vec = vector(a) && vector(b);
    if (dt == Dt::BF16) {
      if (vec) go(ActBF16{}, std::integral_constant<int, 4>{});
      else go(ActBF16{}, std::integral_constant<int, 1>{});
    } else {
      if (vec) go(ActF32{}, std::integral_constant<int, 4>{});
      else go(ActF32{}, std::integral_constant<int, 1>{});
    }
    i += both;
  }
  return hipGetLastError();
}

hipError_t launch_la_copy_state(float* dst, const float* src, int64_t n, hipStream_t s) {
  if (n <= 0 || dst == src) return hipSuccess;
  const int64_t blocks = (n + 255) / 256;
  const dim3 grid(static_cast<unsigned>(blocks < 8192 ? blocks : 8192));
  hipLaunchKernelGGL(la_copy_state_kernel, grid, dim3(256), 0, s, dst, src, n);
  return hipGetLastError();
}

}  // namespace ssm
