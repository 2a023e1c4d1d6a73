// The gated delta rule, prompt form, on the matrix cores.
//
// Per (batch row, head) with a_t = exp(g_t) and the K x V state S:
//     u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   S_t = a_t S_{t-1} + k_t u_t^T,   o_t = scale S_t^T q_t.
// Over a chunk of Q = 64 tokens with the entering state E, G the running sum of g and M_ij = exp(G_i - G_j) this
// unrolls into matrix products:
//     A = strictly lower (M_ij k_i.k_j beta_j)      T = (I + A)^-1
//     X = V - exp(G) K E                            W = T X,   U = beta W
//     O = scale (exp(G) Q E + lower(M_ij q_i.k_j) U)
//     E' = exp(G_Q) E + K^T (exp(G_Q - G) U)
// T depends on no state, so a kernel of its own (gd_prepare_kernel, a workgroup a chunk) forms it for all chunks
// at once.  The walk (gd_walk_kernel) takes a (batch row, head)'s chunks one after the other; only E crosses
// chunks, in float32 registers.
//
// The walk's layout is linear attention's: a wave owns 16 or 32 columns of E, and the columns of a state are
// independent, so X, U and E go from product to product in registers.  A product leaves lane (g, c) of a 16 x 16
// tile four consecutive rows of column c; the rows of each pair of tiles are assigned so that the pair leaves a
// lane 8 consecutive indices, which is what an operand needs.  q, k and v go from memory into LDS row by row;
// T comes in operand order straight into registers.
//
// Roundings (bfloat16 activations; float32 activations use float32 products throughout): every value that the
// state depends on enters a product as three bfloat16 terms, which carry 24 bits (E, T, X and the decayed U; a
// product of two such values takes the six partial products that count): the state and what follows from it keep
// float32's accuracy over any number of tokens.  What only the outputs see (E and U in front of them, and the
// scores) has two terms, 16 bits, so that the output's own rounding is the one that counts.
#include <type_traits>

#include "device_common.hpp"
#include "gd_common.hpp"
#include "la_tiles.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

// ---- T of every chunk

// The 16 x 16 block at (r0, c0) of a float32 matrix in LDS with rows of kRow floats, as a left operand whose
// summation index is 4 g + s in step s: a lane's four values are a row's neighbours.
constexpr int kRow = 68;
__device__ __forceinline__ f32x4_t block_mma(const float* a, int ar, int ac, const f32x4_t& b, f32x4_t c, int g, int c16) {
  const float4 x = *reinterpret_cast<const float4*>(a + (ar + c16) * kRow + ac + 4 * g);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.x, b[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.y, b[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.z, b[2], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(x.w, b[3], c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t block_rows(const float* b, int br, int bc, int g, int c16) {
  f32x4_t v;
#pragma unroll
  for (int s = 0; s < 4; ++s) v[s] = b[(br + 4 * g + s) * kRow + bc + c16];
  return v;
}

// BACK: the rows are the chunk's tokens from its last place to its first, as the backward walk takes them; its matrix is
// the same with the lower triangle of M_ji k_i.k_j for M_ij k_i.k_j.
template <typename ACT, int KD, int MOVE, bool BACK>
__global__ __launch_bounds__(256) void gd_prepare_kernel(GdArgs p) {
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr bool kF32 = ACT::kBytes == 4;
  constexpr int RK = KD * static_cast<int>(sizeof(elem)), PB = O::kPiece, KT = KD / 32;
  __shared__ __attribute__((aligned(512))) char sK[kQ * RK];
  __shared__ __attribute__((aligned(16))) float sA[kQ * kRow], sT[kQ * kRow];
  __shared__ float sHi[kQ], sLo[kQ], sB[kQ];

  const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6), g = lane >> 4, c16 = lane & 15;
  const uint32_t nch = static_cast<uint32_t>((p.L + kQ - 1) / kQ), all = static_cast<uint32_t>(p.batch) * p.H * nch;
  for (uint32_t item = blockIdx.x; item < all; item += gridDim.x) {
    const uint32_t pair = item / nch, c = item - pair * nch;
    const uint32_t row_b = pair / static_cast<uint32_t>(p.H);
    const int h = static_cast<int>(pair - row_b * static_cast<uint32_t>(p.H));
    const int64_t b = row_b, t0 = static_cast<int64_t>(c) * kQ;
    const int left = gd_length(p.lengths, static_cast<int>(p.L), b) - static_cast<int>(t0), n = left < kQ ? left : kQ;
    if (n <= 0) continue;                             // (nobody reads the record of a chunk without tokens)
    char* rec = (BACK ? p.rec_back : p.rec) + (static_cast<int64_t>(pair) * nch + c) * kRecord<ACT>;

    const elem* kg = static_cast<const elem*>(p.k) + b * p.ks[0] + (h / p.kdiv) * p.ks[2] + t0 * p.ks[1];
    auto token = [](int row) { return BACK ? kQ - 1 - row : row; };
    if constexpr (MOVE == 16) {
      constexpr int kSlots = RK / 16;
  #pragma unroll
      for (int i = tid; i < kQ * kSlots; i += 256) {
        const int row = i / kSlots, slot = i % kSlots;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (token(row) < n && slot * 16 < p.K * static_cast<int>(sizeof(elem)))
          x = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(kg + token(row) * p.ks[1]) + slot * 16);
        *reinterpret_cast<uint4*>(sK + row * RK + ((slot ^ swizzle<RK, kF32, false>(row)) << 4)) = x;
      }
    } else {
      for (int i = tid; i < kQ * KD; i += 256) {
        const int row = i / KD, col = i % KD;
        elem x = elem(0);
        if (token(row) < n && col < p.K) x = kg[token(row) * p.ks[1] + col];
        const int byte = col * static_cast<int>(sizeof(elem));
        *reinterpret_cast<elem*>(sK + row * RK + (byte ^ (swizzle<RK, kF32, false>(row) << 4))) = x;
      }
    }
    if (w == 0) {
      // the running sum of g, in units of log 2, from float64 as a pair of float32
      const int64_t at = (b * p.L + t0 + lane) * p.H + h;
      double G = 0.0;
      float beta = 0.0f;
      if (lane < n) {
        G = static_cast<double>(p.g[at]) * 1.4426950408889634;
        G = G < kMinGate ? kMinGate : G;              // (NaN passes through)
        beta = p.beta[at];
      }
  #pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const double before = __shfl_up(G, d);
        if (lane >= d) G += before;
      }
      const double left_over = __shfl(G, 63) - G;
      const float hi = static_cast<float>(G), lo = static_cast<float>(G - hi);
      const float ehi = static_cast<float>(left_over), elo = static_cast<float>(left_over - ehi);
      float* vec = reinterpret_cast<float*>(rec + kTBytes<ACT>);
      const float into = exp2_pair(hi, lo);
      const int row = token(lane);                  // (its own inverse)
      vec[kInto * 64 + row] = into;
      vec[kLast * 64 + row] = exp2_pair(ehi, elo);
      vec[kBeta * 64 + row] = beta;
      vec[kSumHi * 64 + row] = hi;
      vec[kSumLo * 64 + row] = lo;
      vec[kWhole * 64 + row] = __shfl(into, 63);
      sHi[row] = hi; sLo[row] = lo; sB[row] = beta;
    }
    __syncthreads();

    // A, the 10 blocks on and below the diagonal.  An entry that is not finite belongs to a token whose state and
    // whose successors' are not either (the walk sees to those); as a zero it leaves the rows before alone.
    const uint32_t rows = O::template row_part<RK, false>(lds_address(sK), c16, g);
    for (int t = w; t < 10; t += 4) {
      const int ib = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, jb = t - ib * (ib + 1) / 2;
      f32x4_t s = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  #pragma unroll
      for (int x = 0; x < KT; ++x)
        s = O::mma(O::row(rows + ib * (16 * RK), 4 * PB * x, 0), O::row(rows + jb * (16 * RK), 4 * PB * x, 0), s);
      const int j = 16 * jb + c16;
      const float jhi = sHi[j], jlo = sLo[j], jbeta = sB[j];
  #pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * ib + 4 * g + e;
        float x = jbeta * (exp2_pair(BACK ? jhi - sHi[i] : sHi[i] - jhi, BACK ? jlo - sLo[i] : sLo[i] - jlo) * s[e]);
        if (i <= j || !(fabsf(x) < __builtin_huge_valf())) x = 0.0f;
        sA[i * kRow + j] = x;
      }
    }
    __syncthreads();

    // the inverses of the diagonal blocks of I + A, one a wave: lane c16 solves for column c16
    {
      const float* a = sA + 16 * w * kRow + 16 * w;
      float x[16];
  #pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == c16 ? 1.0f : 0.0f;
  #pragma unroll
        for (int j4 = 0; j4 < i; j4 += 4) {
          const float4 y = *reinterpret_cast<const float4*>(a + i * kRow + j4);
          s = __builtin_fmaf(-y.x, x[j4], s);
          if (j4 + 1 < i) s = __builtin_fmaf(-y.y, x[j4 + 1 < 16 ? j4 + 1 : 0], s);
          if (j4 + 2 < i) s = __builtin_fmaf(-y.z, x[j4 + 2 < 16 ? j4 + 2 : 0], s);
          if (j4 + 3 < i) s = __builtin_fmaf(-y.w, x[j4 + 3 < 16 ? j4 + 3 : 0], s);
        }
        x[i] = s;
      }
      if (g == 0) {
  #pragma unroll
        for (int i = 0; i < 16; ++i) sT[(16 * w + i) * kRow + 16 * w + c16] = x[i];
      } else if (g == 1 && (w & 1) == 0) {            // the zero blocks right of it
  #pragma unroll
        for (int i = 0; i < 16; ++i) sT[(16 * w + i) * kRow + 16 * w + 16 + c16] = 0.0f;
      }
    }
    __syncthreads();
    // the blocks below, diagonal by diagonal: T_ij = -T_ii sum over m = j .. i-1 of A_im T_mj
    for (int d = 1; d < 4; ++d) {
      if (w < 4 - d) {
        const int i = w + d, j = w;
        f32x4_t s = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        for (int m = j; m < i; ++m) s = block_mma(sA, 16 * i, 16 * m, block_rows(sT, 16 * m, 16 * j, g, c16), s, g, c16);
        const f32x4_t t = block_mma(sT, 16 * i, 16 * i, s, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, g, c16);
  #pragma unroll
        for (int e = 0; e < 4; ++e) sT[(16 * i + 4 * g + e) * kRow + 16 * j + c16] = -t[e];
      }
      __syncthreads();
    }

    // T in operand order: operands 0, 1 are rows 32 t + 8 (c / 4) + 4 u + c % 4 with t = 0, of tokens 0..31; 2, 3
    // those with t = 1 of tokens 0..31; 4, 5 of tokens 32..63
    for (int x = w; x < kT; x += 4) {
      const int row = (x < 2 ? 0 : 32) + 8 * (c16 >> 2) + 4 * (x & 1) + (c16 & 3), col = (x < 4 ? 0 : 32) + 8 * g;
      float v[8];
  #pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = sT[row * kRow + col + e];
      piece t[kTerms<ACT>];
      O::template split<kTerms<ACT>>(v, t);
  #pragma unroll
      for (int m = 0; m < kTerms<ACT>; ++m)
        store_piece(rec + (x * kTerms<ACT> + m) * kPieceBytes<ACT> + lane * (kPieceBytes<ACT> / 64), t[m]);
    }
    __syncthreads();                                  // (the next chunk's K comes where this one's T was read)
  }
}

// ---- rows of a chunk into their LDS tile

// Row r of a tile is token r of its chunk (BACK: token 63 - r).  MOVE: the bytes that a lane moves (16, 4; 0: element by element).
template <typename ELEM, int RB, int NW, bool PERM, int MOVE, bool BACK>
struct ChunkRows {
  static constexpr bool kF32 = sizeof(ELEM) == 4;
  static constexpr int kSlots = RB / 16, kRows = 64 / kSlots;       // slots of a row, rows of an instruction
  static constexpr int kInstr = kQ / kRows / NW;                    // instructions of a wave
  const char* base;                   // token 0
  int64_t bytes;                      // from a token to the next
  int cols;                           // bytes of a row
  uint32_t off[MOVE == 16 ? kInstr : 1];

  static __device__ __forceinline__ int slot_of(int row, int lane) {   // (the swizzle is linear in the row's bits)
    return (lane % kSlots) ^ swizzle<RB, kF32, PERM>(row);
  }
  static __device__ __forceinline__ constexpr int token(int row) { return BACK ? kQ - 1 - row : row; }
  static __device__ __forceinline__ int clamped(int row, int n) { return least(token(row), n - 1); }
  __device__ __forceinline__ void start(const ELEM* at, int64_t stride, int width, int w, int lane) {
    base = reinterpret_cast<const char*>(at);
    bytes = stride * static_cast<int64_t>(sizeof(ELEM));
    cols = width * static_cast<int>(sizeof(ELEM));
    if constexpr (MOVE == 16) {
#pragma unroll
      for (int i = 0; i < kInstr; ++i) {
        const int row = (w * kInstr + i) * kRows + lane / kSlots;
        off[i] = static_cast<uint32_t>(token(row)) * static_cast<uint32_t>(bytes) + static_cast<uint32_t>(slot_of(row, lane) * 16);
      }
    }
  }
  // Chunk c, of which n tokens are there; rows past them repeat the last (they are cleared afterwards).  ALL: every
  // column is there; else those past `cols` are left as they are (zeros, from the start).
  template <bool ALL>
  __device__ __forceinline__ void load(char* tile_ptr, int c, int n, int w, int lane, int tid) {
    const char* from = base + static_cast<int64_t>(c) * kQ * bytes;
    const uint32_t tile = lds_address(tile_ptr);
    if constexpr (MOVE == 16) {
      if (n == kQ) {
#pragma unroll
        for (int i = 0; i < kInstr; ++i)
          if (ALL || slot_of((w * kInstr + i) * kRows + lane / kSlots, lane) * 16 < cols)
            load_to_lds(tile + (w * kInstr + i) * 1024, from, off[i]);
      } else {
#pragma unroll 1
        for (int i = 0; i < kInstr; ++i) {
          const int row = (w * kInstr + i) * kRows + lane / kSlots, slot = slot_of(row, lane);
          if (slot * 16 < cols) load_to_lds(tile + (w * kInstr + i) * 1024, from + clamped(row, n) * bytes + slot * 16);
        }
      }
    } else if constexpr (MOVE == 4) {
      constexpr int kWords = RB / 4, kAll = kQ * RB / 256 / NW;
#pragma unroll 4
      for (int i = 0; i < kAll; ++i) {
        const int word = (w * kAll + i) * 64 + lane, row = word / kWords;
        const int byte = (word % kWords * 4) ^ (swizzle<RB, kF32, PERM>(row) << 4);
        if (byte < cols) load_word_to_lds(tile + (w * kAll + i) * 256, from + clamped(row, n) * bytes + byte);
      }
    } else {
      constexpr int kCols = RB / static_cast<int>(sizeof(ELEM));
      for (int i = tid; i < kQ * kCols; i += 64 * NW) {
        const int row = i / kCols, byte = i % kCols * static_cast<int>(sizeof(ELEM));
        ELEM x = ELEM(0);
        if (token(row) < n && byte < cols) x = *reinterpret_cast<const ELEM*>(from + token(row) * bytes + byte);
        *reinterpret_cast<ELEM*>(tile_ptr + row * RB + (byte ^ (swizzle<RB, kF32, PERM>(row) << 4))) = x;
      }
    }
  }
  // Clears the rows of tokens n.. of the slots that this wave's loads filled.
  static __device__ __forceinline__ void clear(char* tile, int n, int w, int lane) {
    if constexpr (MOVE > 0) {
      constexpr int kAll = kQ * RB / 1024 / NW;
#pragma unroll 1
      for (int i = 0; i < kAll; ++i) {
        const int s = (w * kAll + i) * 64 + lane;
        if (token(s / kSlots) >= n) *reinterpret_cast<uint4*>(tile + s * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
};

// ---- the walk over a sequence's chunks

// kOut: the forward pass.  kSave: the forward walk of the gradient, which keeps W and, every p.every chunks, E.  kBack: the
// backward walk: E is the gradient of the state after the chunk, and with D the outputs' gradient and P the scores
//     X = scale P^T D + exp(G_Q - G) K E      Y = T^T X      dV = beta Y
//     E' = exp(G_Q) E + scale (exp(G) Q)^T D - K^T (beta exp(G) Y)
// with rows from the chunk's last token to its first, so that T^T and P^T are lower triangular here too.
enum { kOut, kSave, kBack };

template <typename ACT, int KD, int VD, int MOVE, bool ALL, int MODE>
__global__ __launch_bounds__((4 * VD / kGdColumnTiles<ACT, VD>), 1)
void gd_walk_kernel(GdArgs p) {
  constexpr bool BACK = MODE == kBack;
  constexpr int VT = kGdColumnTiles<ACT, VD>;
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr bool kF32 = sizeof(elem) == 4;
  constexpr int NW = VD / 16 / VT, NT = kTerms<ACT>, OT = kOutTerms<ACT>;
  constexpr int PT = MODE == kSave ? 0 : BACK ? NT : OT;                        // terms of the scores
  constexpr int RK = KD * static_cast<int>(sizeof(elem)), RV = VD * static_cast<int>(sizeof(elem));   // row bytes
  constexpr int KT = KD / 32;                       // pairs of state tiles along K
  constexpr int PB = O::kPiece, kOne = kPieceBytes<ACT>;
  __shared__ __attribute__((aligned(512))) char sQ[MODE == kSave ? 16 : kQ * RK];
  __shared__ __attribute__((aligned(512))) char sKK[2][kQ * RK];                // k of this chunk and of the next
  __shared__ __attribute__((aligned(512))) char sV[kQ * RV];                    // v, backwards the outputs' gradient
  __shared__ __attribute__((aligned(512))) char sP[PT ? kT * PT * kOne : 16];   // the scores in operand order
  __shared__ __attribute__((aligned(512))) float sVec[2][kVecs * 64];

  const int tid = threadIdx.x, lane0 = tid & 63, w = uniform_int(tid >> 6);
  const uint32_t pair = blockIdx.x, row_b = pair / static_cast<uint32_t>(p.H);
  const int64_t bh = pair, b = row_b;
  const int h = static_cast<int>(pair - row_b * static_cast<uint32_t>(p.H));
  const int L = static_cast<int>(p.L), len = gd_length(p.lengths, static_cast<int>(p.L), b), K = p.K, V = p.V;
  const int nchunks = (L + kQ - 1) / kQ, c_live = (len + kQ - 1) / kQ;   // chunks; those that hold a token

  ChunkRows<elem, RK, NW, BACK, MOVE, BACK> q_rows_in;
  ChunkRows<elem, RK, NW, true, MOVE, BACK> k_rows_in;
  ChunkRows<elem, RV, NW, false, MOVE, BACK> v_rows_in;
  if constexpr (MODE != kSave) q_rows_in.start(static_cast<const elem*>(p.q) + b * p.qs[0] + (h / p.qdiv) * p.qs[2], p.qs[1], K, w, lane0);
  k_rows_in.start(static_cast<const elem*>(p.k) + b * p.ks[0] + (h / p.kdiv) * p.ks[2], p.ks[1], K, w, lane0);
  v_rows_in.start(static_cast<const elem*>(p.v) + b * p.vs[0] + (h / p.vdiv) * p.vs[2], p.vs[1], V, w, lane0);
  const char* recs = (BACK ? p.rec_back : p.rec) + bh * nchunks * kRecord<ACT>;
  auto present = [&](int c) { return len - c * kQ < kQ ? len - c * kQ : kQ; };
  auto ask_k = [&](int c, int lane) __attribute__((always_inline)) {
    k_rows_in.template load<ALL>(sKK[c & 1], c, present(c), w, lane, tid);
    if (w < 2)                                      // the record's vectors: 2 KB
      load_to_lds(lds_address(reinterpret_cast<char*>(sVec[c & 1])) + w * 1024,
                  recs + static_cast<int64_t>(c) * kRecord<ACT> + kTBytes<ACT> + w * 1024 + lane * 16);
  };
  auto ask_qv = [&](int c, int lane) __attribute__((always_inline)) {
    if constexpr (MODE != kSave) q_rows_in.template load<ALL>(sQ, c, present(c), w, lane, tid);
    v_rows_in.template load<ALL>(sV, c, present(c), w, lane, tid);
  };
  // Waits for this wave's part of chunk c's rows (and for everything else it asked for).
  auto arrived = [&](int c, int n, int lane) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0f70);             // vmcnt(0); expcnt and lgkmcnt as they are
    if (n < kQ) {
      k_rows_in.clear(sKK[c & 1], n, w, lane);
      if constexpr (MODE != kSave) q_rows_in.clear(sQ, n, w, lane);
      v_rows_in.clear(sV, n, w, lane);
    }
  };
  if constexpr (MOVE > 0) {
    if (!ALL) {                                     // columns that the loads leave alone
      k_rows_in.clear(sKK[0], 0, w, lane0);
      k_rows_in.clear(sKK[1], 0, w, lane0);
      if constexpr (MODE != kSave) q_rows_in.clear(sQ, 0, w, lane0);
      v_rows_in.clear(sV, 0, w, lane0);
      __builtin_amdgcn_s_waitcnt(0xc07f);           // lgkmcnt(0): before the loads into the same slots
    }
  }
  const int c_first = BACK ? c_live - 1 : 0, c_step = BACK ? -1 : 1;
  if (c_live > 0) {
    ask_k(c_first, lane0);
    ask_qv(c_first, lane0);
  }

  // E[vt][t][u][e] is the entry k = 32 t + 8 g + 4 u + e, v = 16 (VT w + vt) + c16
  const int g0 = lane0 >> 4, c0 = lane0 & 15;
  f32x4_t E[VT][KT][2];
  auto there = [&](int vt, int t, int u, int e) {
    return ALL || (32 * t + 8 * g0 + 4 * u + e < K && 16 * (VT * w + vt) + c0 < V);
  };
  auto place = [&](int vt, int t, int u, int e) {
    return static_cast<uint32_t>((32 * t + 8 * g0 + 4 * u + e) * V + 16 * (VT * w + vt) + c0);
  };
  const float* src = p.carry ? p.carry + bh * static_cast<int64_t>(K) * V : nullptr;
#pragma unroll
  for (int vt = 0; vt < VT; ++vt)
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) E[vt][t][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  if (src) {
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (there(vt, t, u, e)) E[vt][t][u][e] = src[place(vt, t, u, e)];
  }
  if (c_live > 0) arrived(c_first, present(c_first), lane0);
  auto put_state = [&](float* dst) __attribute__((always_inline)) {
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (there(vt, t, u, e)) dst[place(vt, t, u, e)] = E[vt][t][u][e];
  };

#pragma unroll 1
  for (int done = 0, c = c_first; done < c_live; ++done, c += c_step) {
    const int n = present(c);
    const bool more = done + 1 < c_live;
    if constexpr (MODE != kOut) {                   // the state that enters a stretch of p.every chunks
      if (BACK ? done == 0 || (c + 1) % p.every == 0 : c % p.every == 0)
        put_state(p.kept + (bh * ((nchunks + p.every - 1) / p.every) + c / p.every) * static_cast<int64_t>(K) * V);
    }
    // (opaque, so that the chunk's many LDS and memory addresses are formed here from the lane's number)
    int lane = lane_id();
    asm volatile("" : "+v"(lane));
    const int g = lane >> 4, c16 = lane & 15;
    barrier_lds();                                  // the tiles of chunk c are complete
    piece T[kT][NT];
    {
      const char* from = recs + static_cast<int64_t>(c) * kRecord<ACT> + lane * (kOne / 64);
#pragma unroll
      for (int x = 0; x < kT; ++x)
#pragma unroll
        for (int m = 0; m < NT; ++m) load_piece(from + (x * NT + m) * kOne, T[x][m]);
    }
    if (more) ask_k(c + c_step, lane);
    const float* vec = sVec[c & 1];
    const uint32_t k_tile = lds_address(sKK[0]) + (c & 1) * (kQ * RK);
    const uint32_t q_rows = O::template row_part<RK, BACK>(lds_address(sQ), BACK ? 8 * (c16 >> 2) + (c16 & 3) : c16, g);
    const uint32_t k_rows = O::template row_part<RK, true>(k_tile, 8 * (c16 >> 2) + (c16 & 3), g);
    auto eight = [&](int which, int t, float (&x)[8]) __attribute__((always_inline)) {   // a vector's tokens 32 t + 8 g ..
      const float4 a = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g);
      const float4 d = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g + 4);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = d.x; x[5] = d.y; x[6] = d.z; x[7] = d.w;
    };

    // ---- the scores, 16 rows by 32 tokens an operand.  Forwards operand x holds column j = 16 jt + c16 and tokens
    // i = 32 t + 8 g + e, q_j.k_i; x = 0..3 are jt = x, t = 0, the others jt = x - 2, t = 1.  Backwards it is a left
    // operand like T's: rows 32 t' + 8 (c / 4) + 4 u + c % 4, q_i.k_row; x = 0, 1 are t' = t = 0, 2, 3 t' = 1, t = 0,
    // 4, 5 t' = t = 1, u = x % 2.
    if constexpr (MODE != kSave) {
#pragma unroll 1
      for (int x = w; x < kT; x += NW) {
        const int jt = x < 4 ? x : x - 2, t = x < 4 ? 0 : 1, two = x < 2 ? 0 : 1, one = x & 1;
        const int j = BACK ? 32 * two + 8 * (c16 >> 2) + 4 * one + (c16 & 3) : 16 * jt + c16;
        const uint32_t rows = BACK ? q_rows : k_rows;
        f32x4_t s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) s[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int y = 0; y < KT; ++y) {
          piece right;
          if constexpr (BACK)
            right = O::row(k_rows + two * (32 * RK), (4 * PB * y) ^ (one ? swizzle<RK, kF32, true>(4) << 4 : 0), one * (4 * RK));
          else
            right = O::row(q_rows + jt * (16 * RK), 4 * PB * y, 0);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            s[u] = O::mma(O::row(rows + t * (32 * RK), (4 * PB * y) ^ (swizzle<RK, kF32, true>(4 * u) << 4), 4 * u * RK),
                          right, s[u]);
        }
        float hi[8], lo[8], pv[8];
        eight(kSumHi, t, hi);
        eight(kSumLo, t, lo);
        const float jhi = vec[kSumHi * 64 + j], jlo = vec[kSumLo * 64 + j];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float m = BACK ? exp2_pair(hi[e] - jhi, lo[e] - jlo) : exp2_pair(jhi - hi[e], jlo - lo[e]);
          pv[e] = j >= 32 * t + 8 * g + e ? s[e / 4][e % 4] * (p.scale * m) : 0.0f;
        }
        piece ps[PT];
        O::template split<PT>(pv, ps);
#pragma unroll
        for (int m = 0; m < PT; ++m) store_piece(sP + (x * PT + m) * kOne + lane * (kOne / 64), ps[m]);
      }
    }

    // ---- K E (rows token 32 t + 8 g + 4 u + e, column v) and Q E, transposed (rows v, column j = 16 jt + c16)
    f32x4_t R[VT][2][2], acc[VT][4];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) R[vt][t][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) acc[vt][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int y = 0; y < KT; ++y) {
      piece ef[VT][NT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        const float x[8] = {E[vt][y][0][0], E[vt][y][0][1], E[vt][y][0][2], E[vt][y][0][3],
                            E[vt][y][1][0], E[vt][y][1][1], E[vt][y][1][2], E[vt][y][1][3]};
        O::template split<NT>(x, ef[vt]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const piece kf = O::row(k_rows + t * (32 * RK), (4 * PB * y) ^ (swizzle<RK, kF32, true>(4 * u) << 4), 4 * u * RK);
#pragma unroll
          for (int m = NT - 1; m >= 0; --m)
#pragma unroll
            for (int vt = 0; vt < VT; ++vt) R[vt][t][u] = O::mma(kf, ef[vt][m], R[vt][t][u]);
        }
      if constexpr (MODE == kOut) {
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
          const piece qf = O::row(q_rows, 4 * PB * y, 16 * jt * RK);
#pragma unroll
          for (int m = OT - 1; m >= 0; --m)
#pragma unroll
            for (int vt = 0; vt < VT; ++vt) acc[vt][jt] = O::mma(ef[vt][m], qf, acc[vt][jt]);
        }
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
    // (all of T is here before the next loads into LDS are asked for: a partial count of outstanding loads is not
    // relied on where some go to LDS)
    __builtin_amdgcn_s_waitcnt(0x0f70);
#pragma unroll
    for (int x = 0; x < kT; ++x)
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        if constexpr (kF32) asm volatile("" : "+v"(T[x][m].a.x), "+v"(T[x][m].a.y), "+v"(T[x][m].a.z), "+v"(T[x][m].a.w),
                                              "+v"(T[x][m].b.x), "+v"(T[x][m].b.y), "+v"(T[x][m].b.z), "+v"(T[x][m].b.w));
        else asm volatile("" : "+v"(T[x][m].x), "+v"(T[x][m].y), "+v"(T[x][m].z), "+v"(T[x][m].w));
      }
    barrier_lds();                                  // the scores are complete; the tiles of q and v are free
    if constexpr (!BACK) {
      if (more) ask_qv(c + c_step, lane);
    }

    // ---- X = V - exp(G) K E (backwards scale P^T D + exp(G_Q - G) K E), W = T X
    // Forwards, a value that is not finite must not reach earlier tokens' outputs through T's zeros: its column is cut there,
    // its outputs from that token on and its state are NaN.
    float x[VT][2][8];
    float odd = 0.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float with[8];
      eight(BACK ? kLast : kInto, t, with);
      if constexpr (BACK) {
        f32x4_t Z[VT][2];
#pragma unroll
        for (int vt = 0; vt < VT; ++vt)
#pragma unroll
          for (int u = 0; u < 2; ++u) Z[vt][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int from = 0; from <= t; ++from) {
            piece pf[NT];
#pragma unroll
            for (int m = 0; m < NT; ++m)
              load_piece(sP + ((2 * t + 2 * from + u) * NT + m) * kOne + lane * (kOne / 64), pf[m]);
#pragma unroll
            for (int m = NT - 1; m >= 0; --m)
#pragma unroll
              for (int vt = 0; vt < VT; ++vt) Z[vt][u] = O::mma(pf[m], vf[vt][from], Z[vt][u]);
          }
#pragma unroll
        for (int vt = 0; vt < VT; ++vt)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[vt][t][e] = __builtin_fmaf(with[e], R[vt][t][e / 4][e % 4], Z[vt][e / 4][e % 4]);
      } else {
        float beta[8];
        if constexpr (MODE == kOut) {
          eight(kBeta, t, beta);
#pragma unroll
          for (int e = 0; e < 8; ++e) odd = __builtin_fmaf(beta[e], 0.0f, odd);
        }
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          O::unpack(vf[vt][t], x[vt][t]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[vt][t][e] = __builtin_fmaf(-with[e], R[vt][t][e / 4][e % 4], x[vt][t][e]);
            if constexpr (MODE == kOut) odd = __builtin_fmaf(x[vt][t][e], 0.0f, odd);
          }
        }
      }
    }
    const bool bad = MODE == kOut && __builtin_amdgcn_ballot_w64(odd != odd) != 0;
    int gone[VT];                                   // first token of the column that is not finite
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) gone[vt] = kQ;
    if (__builtin_expect(bad, 0)) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float beta[8];
          eight(kBeta, t, beta);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!(fabsf(x[vt][t][e]) < __builtin_huge_valf()) || !(fabsf(beta[e]) < __builtin_huge_valf()))
              gone[vt] = least(gone[vt], 32 * t + 8 * g + e);
        }
        gone[vt] = least(gone[vt], __shfl_xor(gone[vt], 16));
        gone[vt] = least(gone[vt], __shfl_xor(gone[vt], 32));
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (32 * t + 8 * g + e >= gone[vt]) x[vt][t][e] = 0.0f;
      }
    }
    f32x4_t U[VT][2][2];                            // (W, then U)
    {
      piece xf[VT][2][NT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int t = 0; t < 2; ++t) O::template split<NT>(x[vt][t], xf[vt][t]);
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4_t zero = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          U[vt][0][u] = mma_terms<O, NT, NT>(T[u], xf[vt][0], zero);
          U[vt][1][u] = mma_terms<O, NT, NT>(T[4 + u], xf[vt][1], mma_terms<O, NT, NT>(T[2 + u], xf[vt][0], zero));
        }
    }
    if constexpr (MODE != kOut) {                   // kept for the gradients of q and k (every column of the tiles)
      float* w_out = p.w_out + ((bh * nchunks + c) * kQ) * VD + 16 * VT * w + c16;
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = 32 * t + 8 * g + e;
            w_out[(BACK ? kQ - 1 - row : row) * VD + 16 * vt] = U[vt][t][e / 4][e % 4];
          }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float beta[8];
      eight(kBeta, t, beta);
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          U[vt][t][e / 4][e % 4] *= beta[e];
          if (__builtin_expect(bad, 0)) {
            if (32 * t + 8 * g + e >= gone[vt]) U[vt][t][e / 4][e % 4] = 0.0f;
          }
        }
    }
    if constexpr (BACK) {                           // dV, token by token
      const int64_t row_stride = static_cast<int64_t>(p.H) * V;
      const int64_t first = (b * L + static_cast<int64_t>(c) * kQ) * row_stride + static_cast<int64_t>(h) * V;
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        const int col = 16 * (VT * w + vt) + c16;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = kQ - 1 - (32 * t + 8 * g + e);
            if (at >= n || col >= V) continue;
            const float y = U[vt][t][e / 4][e % 4];
            if (p.o_f32) static_cast<float*>(p.o)[first + at * row_stride + col] = y;
            else store_act<ACT>(p.o, first + at * row_stride + col, y);
          }
      }
    }

    // ---- outputs: exp(G) Q E and the scores' product with U on top
    if constexpr (MODE == kOut) {
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const float f = p.scale * vec[kInto * 64 + 16 * jt + c16];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[vt][jt][e] *= f;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      piece uf[VT][OT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        const float y[8] = {U[vt][t][0][0], U[vt][t][0][1], U[vt][t][0][2], U[vt][t][0][3],
                            U[vt][t][1][0], U[vt][t][1][1], U[vt][t][1][2], U[vt][t][1][3]};
        O::template split<OT>(y, uf[vt]);
      }
#pragma unroll
      for (int jt = 2 * t; jt < 4; ++jt) {
        piece pf[OT];
#pragma unroll
        for (int m = 0; m < OT; ++m) load_piece(sP + ((jt + 2 * t) * OT + m) * kOne + lane * (kOne / 64), pf[m]);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) acc[vt][jt] = mma_terms<O, OT, OT>(uf[vt], pf, acc[vt][jt]);
      }
    }
    if (__builtin_expect(bad, 0)) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {               // (the outputs' rows are the lanes' columns of x)
          const int from = __shfl(gone[vt], 4 * g + e);
#pragma unroll
          for (int jt = 0; jt < 4; ++jt)
            if (16 * jt + c16 >= from) acc[vt][jt][e] = __builtin_nanf("");
        }
    }
    }

    // ---- the state: exp(G_Q) E + K^T (exp(G_Q - G) U)
    const float whole = vec[kWhole * 64];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) E[vt][y][u][e] *= whole;
    const uint32_t k_cols = O::template column_part<RK, true>(k_tile, 0, 8, lane);
    const uint32_t q_cols = O::template column_part<RK, true>(lds_address(sQ), 0, 8, lane);   // (backwards)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float with[8];
      eight(BACK ? kInto : kLast, t, with);
      piece wf[VT][NT], df[VT][NT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (BACK ? -with[e] : with[e]) * U[vt][t][e / 4][e % 4];
        O::template split<NT>(y, wf[vt]);
        if constexpr (BACK) {
          O::unpack(vf[vt][t], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= p.scale * with[e];
          O::template split<NT>(y, df[vt]);
        }
      }
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const piece kf =
              O::template column<RK, true>(k_cols, (4 * PB * y) ^ O::half_flip(u), 32 * t * RK + O::half_offset(u));
#pragma unroll
          for (int m = NT - 1; m >= 0; --m)
#pragma unroll
            for (int vt = 0; vt < VT; ++vt) E[vt][y][u] = O::mma(kf, wf[vt][m], E[vt][y][u]);
          if constexpr (BACK) {
            const piece qf =
                O::template column<RK, true>(q_cols, (4 * PB * y) ^ O::half_flip(u), 32 * t * RK + O::half_offset(u));
#pragma unroll
            for (int m = NT - 1; m >= 0; --m)
#pragma unroll
              for (int vt = 0; vt < VT; ++vt) E[vt][y][u] = O::mma(qf, df[vt][m], E[vt][y][u]);
          }
        }
    }
    if constexpr (BACK) {
      barrier_lds();                                // the tiles of q and of the outputs' gradient are free
      if (more) ask_qv(c + c_step, lane);
    }
    if (__builtin_expect(bad, 0)) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
        if (gone[vt] < kQ) {
#pragma unroll
          for (int y = 0; y < KT; ++y)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) E[vt][y][u][e] = __builtin_nanf("");
        }
    }
    arrived(c + c_step, more ? present(c + c_step) : kQ, lane);

    if constexpr (MODE == kOut) {
      // ---- the output rows to memory: lane (g, c) has 4 columns of token 16 jt + c
      auto four = [](const f32x4_t& a) __attribute__((always_inline)) {
        if constexpr (kF32) return make_float4(a[0], a[1], a[2], a[3]);
        else return make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
      };
      const int64_t row_stride = static_cast<int64_t>(p.H) * V;
      elem* out = static_cast<elem*>(p.o) + (b * L + static_cast<int64_t>(c) * kQ) * row_stride + static_cast<int64_t>(h) * V;
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const int row = 16 * jt + c16;
        if (c * kQ + row >= L) continue;
        elem* o = out + row * row_stride;
        if (row >= n) {
#pragma unroll
          for (int vt = 0; vt < VT; ++vt) acc[vt][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          const int v0 = 16 * (VT * w + vt) + 4 * g;
          if (p.o_vec) {
            if (ALL || v0 < V) *reinterpret_cast<decltype(four(acc[0][0]))*>(o + v0) = four(acc[vt][jt]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (v0 + e >= V) continue;
              if constexpr (kF32) o[v0 + e] = acc[vt][jt][e];
              else o[v0 + e] = to_bf16(acc[vt][jt][e]);
            }
          }
        }
      }
    }
  }

  // tokens that are not there: zeros (forwards those of the last chunk have theirs)
  if constexpr (MODE != kSave) {
    for (int z = BACK ? len / kQ : c_live; z < nchunks; ++z) {
      for (int i = tid; i < kQ * V; i += 64 * NW) {
        const int64_t token = static_cast<int64_t>(z) * kQ + i / V;
        if (token >= L) break;
        if (token < len) continue;
        const int64_t at = ((b * L + token) * p.H + h) * V + i % V;
        if (BACK && p.o_f32) static_cast<float*>(p.o)[at] = 0.0f;
        else static_cast<elem*>(p.o)[at] = elem(0);
      }
    }
  }
  if (p.fin) put_state(p.fin + bh * static_cast<int64_t>(K) * V);
}

template <typename ACT, int KD, int VD, int MOVE, bool ALL, int MODE>
void launch_gd_t(const GdArgs& a, hipStream_t s) {
  const int64_t nch = (a.L + kQ - 1) / kQ;
  const int64_t all = a.batch * a.H * nch, most = 1 << 22;       // (a launch's threads are fewer than 2^32)
  const dim3 chunks(static_cast<unsigned>(all < most ? all : most)), pairs(static_cast<unsigned>(a.batch * a.H));
  hipLaunchKernelGGL((gd_prepare_kernel<ACT, KD, MOVE, MODE == kBack>), chunks, dim3(256), 0, s, a);
  hipLaunchKernelGGL((gd_walk_kernel<ACT, KD, VD, MOVE, ALL, MODE>), pairs, dim3(4 * VD / kGdColumnTiles<ACT, VD>), 0, s, a);
}

template <int MODE>
void launch_gd_mode(const GdArgs& a, Dt dt, hipStream_t s) {
  auto go = [&](auto act, auto kd, auto vd) {
    using ACT = decltype(act);
    constexpr int KD = decltype(kd)::value, VD = decltype(vd)::value;
    if (a.move == 16 && a.K == KD && a.V == VD) launch_gd_t<ACT, KD, VD, 16, true, MODE>(a, s);
    else if (a.move == 16) launch_gd_t<ACT, KD, VD, 16, false, MODE>(a, s);
    else if (ACT::kBytes == 4 || a.move == 4) launch_gd_t<ACT, KD, VD, 4, false, MODE>(a, s);
    else if constexpr (ACT::kBytes == 2) launch_gd_t<ACT, KD, VD, 0, false, MODE>(a, s);
  };
  auto shape = [&](auto act) {
    constexpr std::integral_constant<int, 64> n64;
    constexpr std::integral_constant<int, 128> n128;
    if (a.K > 64 && a.V > 64) go(act, n128, n128);
    else if (a.K > 64) go(act, n128, n64);
    else if (a.V > 64) go(act, n64, n128);
    else go(act, n64, n64);
  };
  if (dt == Dt::BF16) shape(ActBF16{});
  else shape(ActF32{});
}

}  // namespace

int64_t gd_record_bytes(Dt dt) { return dt == Dt::BF16 ? kRecord<ActBF16> : kRecord<ActF32>; }

hipError_t launch_gd(const GdArgs& a, Dt dt, hipStream_t s) {
  launch_gd_mode<kOut>(a, dt, s);
  return hipGetLastError();
}

hipError_t launch_gd_walks(const GdArgs& forwards, const GdArgs& backwards, Dt dt, hipStream_t s) {
  launch_gd_mode<kSave>(forwards, dt, s);
  launch_gd_mode<kBack>(backwards, dt, s);
  return hipGetLastError();
}

}  // namespace ssm
