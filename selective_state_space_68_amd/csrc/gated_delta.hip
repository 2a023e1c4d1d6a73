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
// T and the scores depend on no state, so a kernel of its own (gd_prepare_kernel, a wave a chunk) forms them for all chunks
// at once.  The walk (gd_walk_kernel) takes a (batch row, head)'s chunks one after the other; only E crosses
// chunks, in float32 registers.
//
// The walk's layout is linear attention's: a wave owns 16 columns of E, and the columns of a state are
// independent, so X, U and E go from product to product in registers.  A product leaves lane (g, c) of a 16 x 16
// tile four consecutive rows of column c; the rows of each pair of tiles are assigned so that the pair leaves a
// lane 8 consecutive indices, which is what an operand needs.  q, k and v go from memory into LDS row by row;
// T and the scores come in operand order, T straight into registers.
//
// Roundings (bfloat16 activations; float32 activations use float32 products throughout): every value that the
// state depends on enters a product as three bfloat16 terms, which carry 24 bits (E, T, X and the decayed U; a
// product of two such values takes the six partial products that count): the state and what follows from it keep
// float32's accuracy over any number of tokens.  What only the outputs see (E and U in front of them, and the
// scores) has two terms, 16 bits, so that the output's own rounding is the one that counts.
//
// What bounds it (bfloat16, heads of 128): the walk by the chain of a chunk, K E, T X, U and K^T U one after the other with two
// barriers and a wait for the next chunk's tiles: 4 x 2048 tokens, 40 heads: 201 us, 6.3 a chunk (24 MFLOP with the terms) on each of
// the 160 CUs that have a (batch row, head), the matrix units busy for 0.44 of it; a workgroup of half the columns, and so half the
// products, still takes 0.78 of the time.  The prepared records by memory: 67 us there for 254 MB, 3.8 TB/s (131072 tokens, 20
// heads: 522 us, 5.9 TB/s).  A sequence of few heads by both in turn: segments.  The shortest prompts by latency, 10 us a kernel.
#include <type_traits>

#include "device_common.hpp"
#include "gd_common.hpp"
#include "la_tiles.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

// ---- T, the scores and the vectors of every chunk

// A chunk's matrix is worked on by one wave, in LDS by blocks of 16 x 16 on and below the diagonal, rows kRow floats apart.
constexpr int kRow = 20, kBlock = 16 * kRow;
__device__ __forceinline__ constexpr int block_at(int i, int j) { return (i * (i + 1) / 2 + j) * kBlock; }

// c + a b of two blocks, the summation index 4 g + s in step s, so that a lane's four values of a are a row's neighbours and
// those of b are what a product left it.
__device__ __forceinline__ f32x4_t block_mma(const float* a, const f32x4_t& b, f32x4_t c, int g, int c16) {
  const float4 x = *reinterpret_cast<const float4*>(a + c16 * kRow + 4 * g);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.x, b[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.y, b[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.z, b[2], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(x.w, b[3], c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t block_rows(const float* b, int g, int c16) {
  f32x4_t v;
#pragma unroll
  for (int s = 0; s < 4; ++s) v[s] = b[(4 * g + s) * kRow + c16];
  return v;
}

// LDS that a wave wrote is read by its other lanes (a wave's LDS accesses are carried out in order).
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// One wave a chunk: 8 waves a CU (12 for heads of 64) that never wait for each other (4 waves on a chunk met at 7 barriers: 4 x 2048, 40 heads of 128,
// 69 us without the scores, 67 with them now).  Rows come straight from memory in operand order.
// BACK: the rows are the chunk's tokens from its last place to its first, as the backward walk takes them; its matrix is
// the same with M_ji k_i.k_j for M_ij k_i.k_j.  PT: the scores' terms (0: not wanted).
template <typename ACT, int KD, int MOVE, bool BACK, int PT>
__global__ __launch_bounds__(256, 2) void gd_prepare_kernel(GdArgs p) {
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr int KT = KD / 32, NT = kTerms<ACT>, kOne = kPieceBytes<ACT>;
  __shared__ __attribute__((aligned(16))) float blocks[4][10 * kBlock];
  __shared__ __attribute__((aligned(16))) float vectors[4][3][kQ];              // G in two parts, beta

  const int w = uniform_int(threadIdx.x >> 6);
  float *A = blocks[w], *sHi = vectors[w][0], *sLo = vectors[w][1], *sB = vectors[w][2];
  const uint32_t nch = static_cast<uint32_t>((p.L + kQ - 1) / kQ), all = static_cast<uint32_t>(p.batch) * p.H * nch;
  auto token = [](int row) { return BACK ? kQ - 1 - row : row; };               // (its own inverse)
  for (uint32_t item = blockIdx.x * 4 + w; item < all; item += gridDim.x * 4) {
    int lane = lane_id();                           // (opaque: what follows from it is formed here, not kept in spilled registers)
    asm volatile("" : "+v"(lane));
    const int g = lane >> 4, c16 = lane & 15;
    const uint32_t pair = item / nch, c = item - pair * nch;
    const uint32_t row_b = pair / static_cast<uint32_t>(p.H);
    const int h = static_cast<int>(pair - row_b * static_cast<uint32_t>(p.H));
    const int64_t b = row_b, t0 = static_cast<int64_t>(c) * kQ;
    const int left = gd_length(p.lengths, static_cast<int>(p.L), b) - static_cast<int>(t0), n = left < kQ ? left : kQ;
    if (n <= 0) continue;                           // (nobody reads the record of a chunk without tokens)
    char* rec = (BACK ? p.rec_back : p.rec) + static_cast<int64_t>(item) * kRecord<ACT, PT>;
    const int64_t gate = (b * p.L + t0 + lane) * p.H + h;
    const bool on = lane < n;
    const float g_in = on ? p.g[gate] : 0.0f, beta = on ? p.beta[gate] : 0.0f;

    // rows 32 t + 8 (c / 4) + 4 u + c % 4 as operands: columns 32 y + 8 g ..; rows and columns that are not there are zeros
    const elem* kg = static_cast<const elem*>(p.k) + b * p.ks[0] + (h / p.kdiv) * p.ks[2] + t0 * p.ks[1];
    const elem* qg = static_cast<const elem*>(p.q) + b * p.qs[0] + (h / p.qdiv) * p.qs[2] + t0 * p.qs[1];
    const int perm_row = 8 * (c16 >> 2) + (c16 & 3);
    auto load_rows = [&](const elem* base, int64_t stride, int t, piece (&out)[2][KT]) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = token(32 * t + 4 * u + perm_row);
        const elem* from = base + least(at, n - 1) * stride;
#pragma unroll
        for (int y = 0; y < KT; ++y) {
          const int col = 32 * y + 8 * g;
          if constexpr (MOVE == 16) {
            load_piece(reinterpret_cast<const char*>(from + least(col, p.K - 8)), out[u][y]);
            if (at >= n || col >= p.K) out[u][y] = O::zero();
          } else if constexpr (MOVE == 4) {         // (the last columns come at the end of 8 that are there)
            const int start = least(col, p.K - 8);
            load_words(reinterpret_cast<const char*>(from + start), out[u][y]);
            if (32 * y + 32 > p.K) drop_first(out[u][y], least(col - start, 7));
            if (at >= n || col >= p.K) out[u][y] = O::zero();
          } else {
            elem v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const elem x = from[least(col + e, p.K - 1)];
              v[e] = at < n && col + e < p.K ? x : elem(0);
            }
            out[u][y] = __builtin_bit_cast(piece, v);
          }
        }
      }
    };
    piece kp[2][2][KT], qp[2][KT];                  // of q a half at a time
    load_rows(kg, p.ks[1], 0, kp[0]);
    if constexpr (PT > 0) load_rows(qg, p.qs[1], 0, qp);
    load_rows(kg, p.ks[1], 1, kp[1]);

    // the running sum of g, in units of log 2, from float64 as a pair of float32
    {
      double G = static_cast<double>(g_in) * 1.4426950408889634;
      G = G < kMinGate ? kMinGate : G;              // (NaN passes through)
      const bool fast = __builtin_amdgcn_ballot_w64(G < kFastGate) != 0, strong = __builtin_amdgcn_ballot_w64(G < kStrongGate) != 0;
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
      const int row = token(lane);
      vec[kInto * 64 + row] = into;
      vec[kLast * 64 + row] = exp2_pair(ehi, elo);
      vec[kBeta * 64 + row] = beta;
      vec[kSumHi * 64 + row] = hi;
      vec[kSumLo * 64 + row] = lo;
      const float whole = __shfl(into, 63);
      vec[kWhole * 64 + row] = whole;
      if constexpr (!BACK && PT == 0) {
        const bool last = left <= kQ;               // (the gradient of the state behind it is the caller's, of any size)
        vec[kPace * 64 + row] = !fast ? kSlow : whole < nothing(strong) ? kFast : strong || last ? kFastThrough : kSlow;
      }
      sHi[row] = hi; sLo[row] = lo; sB[row] = beta;
    }
    wave_lds();

    // A's and the scores' tiles: rows i = 32 t + 8 g + 4 u + e, column j = 32 two + 8 (c / 4) + 4 one + c % 4, for i <= j.  The
    // scores are q_j.k_i, backwards q_i.k_j.  An entry of A that is not finite (finite keys may have such a product) belongs to a
    // token that is not finite, nor are its successors: for outputs it is a zero, which leaves the rows before alone, and the
    // record says from where on the walk has to make up for it; in the gradient's records it stays.  Behind a decay of 0 or
    // a beta of 0 there is nothing that a key could meet.
    constexpr bool CUT = !BACK && PT > 0;
    int odd = kQ;
    auto tile = [&](int t, int j, const f32x4_t (&s1)[2], const f32x4_t (&s2)[2], int x) __attribute__((always_inline)) {
      const float jhi = sHi[j], jlo = sLo[j];
      float v[8], a[8], poison = 0.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i0 = 32 * t + 8 * g + 4 * u;
        const float4 hi = *reinterpret_cast<const float4*>(sHi + i0), lo = *reinterpret_cast<const float4*>(sLo + i0);
        const float4 be = *reinterpret_cast<const float4*>(sB + i0);
        const float ihi[4] = {hi.x, hi.y, hi.z, hi.w}, ilo[4] = {lo.x, lo.y, lo.z, lo.w}, ib[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float m = BACK ? exp2_pair(ihi[e] - jhi, ilo[e] - jlo) : exp2_pair(jhi - ihi[e], jlo - ilo[e]);
          a[4 * u + e] = i0 + e < j ? ib[e] * (m * s1[u][e]) : 0.0f;
          poison = __builtin_fmaf(a[4 * u + e], 0.0f, poison);
          if constexpr (PT > 0) v[4 * u + e] = i0 + e <= j ? s2[u][e] * (p.scale * m) : 0.0f;
        }
      }
      if (__builtin_expect(__builtin_amdgcn_ballot_w64(poison != poison) != 0, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = 32 * t + 8 * g + i;
          const float m = BACK ? exp2_pair(sHi[at] - jhi, sLo[at] - jlo) : exp2_pair(jhi - sHi[at], jlo - sLo[at]);
          if (fabsf(a[i]) < __builtin_huge_valf()) continue;
          if (m == 0.0f || sB[at] == 0.0f) a[i] = 0.0f;
          else if (CUT) {
            a[i] = 0.0f;
            odd = least(odd, j);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i0 = 32 * t + 8 * g + 4 * u;
        if (i0 / 16 <= j / 16)
          *reinterpret_cast<float4*>(A + block_at(j / 16, i0 / 16) + j % 16 * kRow + i0 % 16) =
              make_float4(a[4 * u], a[4 * u + 1], a[4 * u + 2], a[4 * u + 3]);
      }
      if constexpr (PT > 0) {
        piece ps[PT];
        O::template split<PT>(v, ps);
#pragma unroll
        for (int m = 0; m < PT; ++m)
          store_piece(rec + kTBytes<ACT> + kVecs * 256 + (x * PT + m) * kOne + lane * (kOne / 64), ps[m]);
      }
    };
#pragma unroll
    for (int half = 0; half < 2; ++half) {          // (q's: columns, backwards rows)
      if constexpr (PT > 0) {
        if (half) load_rows(qg, p.qs[1], 1, qp);
      }
#pragma unroll
      for (int other = BACK ? half : 0; other < (BACK ? 2 : half + 1); ++other)
#pragma unroll
        for (int one = 0; one < 2; ++one) {
          const int two = BACK ? other : half, t = BACK ? half : other;
          f32x4_t s1[2], s2[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) s1[u] = s2[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int y = 0; y < KT; ++y)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              s1[u] = O::mma(kp[t][u][y], kp[two][one][y], s1[u]);
              if constexpr (PT > 0)
                s2[u] = BACK ? O::mma(qp[u][y], kp[two][one][y], s2[u]) : O::mma(kp[t][u][y], qp[one][y], s2[u]);
            }
          tile(t, 32 * two + 4 * one + perm_row, s1, s2, 2 * two + 2 * t + one);
        }
    }
    if constexpr (CUT) {
      float* vec = reinterpret_cast<float*>(rec + kTBytes<ACT>);
      if (__builtin_expect(__builtin_amdgcn_ballot_w64(odd < kQ) != 0, 0)) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) odd = least(odd, __shfl_xor(odd, d));
        vec[kWhole * 64 + lane] = __builtin_nanf("");
      }
      vec[kFirstOdd * 64 + lane] = static_cast<float>(odd);
    }
    wave_lds();

    // the inverses of the diagonal blocks of I + A, in place: 16 lanes a block, lane c16 solves for its column
    {
      float* a = A + (g * (g + 1) / 2 + g) * kBlock;
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
      wave_lds();
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i * kRow + c16] = x[i];
    }
    wave_lds();
    // the blocks below, row by row in place: T_ij = -T_ii sum over m = j .. i-1 of A_im T_mj
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      f32x4_t s[3];
#pragma unroll
      for (int j = 0; j < i; ++j) {
        s[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = j; m < i; ++m) s[j] = block_mma(A + block_at(i, m), block_rows(A + block_at(m, j), g, c16), s[j], g, c16);
      }
      wave_lds();
#pragma unroll
      for (int j = 0; j < i; ++j) {
        const f32x4_t t = block_mma(A + block_at(i, i), s[j], f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, g, c16);
#pragma unroll
        for (int e = 0; e < 4; ++e) A[block_at(i, j) + (4 * g + e) * kRow + c16] = -t[e];
      }
      wave_lds();
    }

    // T in operand order: operands 0, 1 are rows 32 t + 8 (c / 4) + 4 u + c % 4 with t = 0, of tokens 0..31; 2, 3
    // those with t = 1 of tokens 0..31; 4, 5 of tokens 32..63
#pragma unroll
    for (int x = 0; x < kT; ++x) {
      const int row = (x < 2 ? 0 : 32) + 4 * (x & 1) + perm_row, ib = row / 16, jb = (x < 4 ? 0 : 2) + (g >> 1);
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (jb <= ib) {
        const float* from = A + (ib * (ib + 1) / 2 + jb) * kBlock + row % 16 * kRow + 8 * (g & 1);
        const float4 y = reinterpret_cast<const float4*>(from)[0], z = reinterpret_cast<const float4*>(from)[1];
        v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w; v[4] = z.x; v[5] = z.y; v[6] = z.z; v[7] = z.w;
      }
      piece t[NT];
      O::template split<NT>(v, t);
#pragma unroll
      for (int m = 0; m < NT; ++m) store_piece(rec + (x * NT + m) * kOne + lane * (kOne / 64), t[m]);
    }
    wave_lds();                                     // (the next chunk's A comes where T was read)
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
      if constexpr (kWords >= 64) {                 // an instruction is of one row: what follows from the row is scalar
        constexpr int kPer = kWords / 64;
#pragma unroll 4
        for (int i = 0; i < kAll; ++i) {
          const int at = w * kAll + i, row = at / kPer;
          const uint32_t byte = static_cast<uint32_t>((256 * (at % kPer) + 4 * lane) ^ (swizzle<RB, kF32, PERM>(row) << 4));
          if (static_cast<int>(byte) < cols) load_word_to_lds(tile + at * 256, from + clamped(row, n) * bytes, byte);
        }
        return;
      }
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
// kState and kBackState: the pre-pass of a walk in segments, which leaves the state that a segment makes of none (N);
// kState's further column blocks carry the identity with no values, which makes M, and E' = M E + N.
enum { kOut, kSave, kBack, kState, kBackState };

// A workgroup takes COLUMNS (64 or 128) columns of one (batch row, head, segment), a wave 16 of them.  A chunk's record comes
// into LDS whole, once a workgroup: T read by every wave for itself kept the loads' unit busy for a quarter of the time.

// Terms of a walk's scores in its chunks' records.
template <typename ACT, int MODE>
constexpr int score_terms() {
  return MODE == kOut ? kOutTerms<ACT> : MODE == kBack || MODE == kBackState ? kTerms<ACT> : 0;
}

// PR: terms of the scores in the records.
template <typename ACT, int KD, int COLUMNS, int MOVE, bool ALL, int MODE, int PR>
__global__ __launch_bounds__(4 * COLUMNS, 2)
void gd_walk_kernel(GdArgs p) {
  constexpr int kColumns = COLUMNS;
  constexpr bool BACK = MODE == kBack || MODE == kBackState, STATE = MODE == kState || MODE == kBackState;
  constexpr bool SCORES = MODE == kOut || BACK;     // q and the scores are needed
  constexpr int PT = score_terms<ACT, MODE>();
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr bool kF32 = sizeof(elem) == 4;
  constexpr int NW = COLUMNS / 16, NT = kTerms<ACT>, OT = kOutTerms<ACT>;
  constexpr int RK = KD * static_cast<int>(sizeof(elem)), RV = kColumns * static_cast<int>(sizeof(elem));   // row bytes
  constexpr int KT = KD / 32;                       // pairs of state tiles along K
  constexpr int PB = O::kPiece, kOne = kPieceBytes<ACT>;
  __shared__ __attribute__((aligned(512))) char sQ[SCORES ? kQ * RK : 16];
  __shared__ __attribute__((aligned(512))) char sKK[2][kQ * RK];                // k of this chunk and of the next
  __shared__ __attribute__((aligned(512))) char sV[kQ * RV];                    // v, backwards the outputs' gradient
  // the record (T, vectors, scores), of this chunk and, where there is room, of the next
  constexpr int kRec = kTBytes<ACT> + kVecs * 256 + (SCORES ? kT * PT * kOne : 0);
  constexpr bool AHEAD = (SCORES ? 3 : 2) * kQ * RK + kQ * RV + 2 * kRec <= 160 * 1024;
  __shared__ __attribute__((aligned(512))) char sRec[AHEAD ? 2 : 1][kRec];

  const int tid = threadIdx.x, lane0 = tid & 63, w = uniform_int(tid >> 6);
  const int K = p.K, V = p.V;
  // Workgroup ids go round the 8 XCDs: the column blocks of one (batch row, head, segment), which read the same rows of q
  // and k, are 8 ids apart, on one XCD and its L2 at about the same time.
  const uint32_t v_blocks = static_cast<uint32_t>((V + kColumns - 1) / kColumns);
  const uint32_t blocks = v_blocks + (MODE == kState ? (K + kColumns - 1) / kColumns : 0), span = 8 * blocks;
  const uint32_t group = blockIdx.x / span, in_group = blockIdx.x - group * span, item = group * 8 + in_group % 8;
  const uint32_t nseg = static_cast<uint32_t>(p.nseg);
  if (item >= static_cast<uint32_t>(p.batch) * p.H * nseg) return;
  const uint32_t block = in_group / 8, pair = nseg == 1 ? item : item / nseg, seg = item - pair * nseg;
  const bool ident = MODE == kState && block >= v_blocks;       // columns of the identity
  const int col0 = kColumns * static_cast<int>(ident ? block - v_blocks : block), width = (ident ? K : V) - col0;
  const uint32_t row_b = pair / static_cast<uint32_t>(p.H);
  const int64_t bh = pair, b = row_b;
  const int h = static_cast<int>(pair - row_b * static_cast<uint32_t>(p.H));
  const int L = static_cast<int>(p.L), len = gd_length(p.lengths, L, b);
  const int nchunks = (L + kQ - 1) / kQ, live = (len + kQ - 1) / kQ;   // chunks; those that hold a token
  const int c_begin = static_cast<int>(seg) * p.seg_chunks, c_stop = least(c_begin + p.seg_chunks, nchunks);
  const int c_end = least(c_stop, live), count = c_end > c_begin ? c_end - c_begin : 0;
  if (STATE) {                                      // sums that nobody reads: of no chunks, and the last of each walk's
    if (count == 0 || (BACK ? seg == 0 : c_end == live && !(ident && p.seg_mt))) return;
  }

  ChunkRows<elem, RK, NW, true, MOVE, BACK> q_rows_in;
  ChunkRows<elem, RK, NW, true, MOVE, BACK> k_rows_in;
  ChunkRows<elem, RV, NW, false, MOVE, BACK> v_rows_in;
  if constexpr (SCORES)
    q_rows_in.start(static_cast<const elem*>(p.q) + b * p.qs[0] + (h / p.qdiv) * p.qs[2], p.qs[1], K, w, lane0);
  k_rows_in.start(static_cast<const elem*>(p.k) + b * p.ks[0] + (h / p.kdiv) * p.ks[2], p.ks[1], K, w, lane0);
  v_rows_in.start(static_cast<const elem*>(p.v) + b * p.vs[0] + (h / p.vdiv) * p.vs[2] + col0, p.vs[1],
                  least(width, kColumns), w, lane0);
  const char* recs = (BACK ? p.rec_back : p.rec) + bh * nchunks * kRecord<ACT, PR>;
  auto present = [&](int c) { return least(len - c * kQ, kQ); };
  auto ask_k = [&](int c, int lane) __attribute__((always_inline)) {
    k_rows_in.template load<ALL>(sKK[c & 1], c, present(c), w, lane, tid);
  };
  auto ask_record = [&](int c, int lane) __attribute__((always_inline)) {
    const uint32_t to = lds_address(sRec[AHEAD ? c & 1 : 0]);
    const char* from = recs + static_cast<int64_t>(c) * kRecord<ACT, PR>;
#pragma unroll
    for (int i = 0; i < (kRec / 1024 + NW - 1) / NW; ++i)
      if (kRec / 1024 % NW == 0 || w + i * NW < kRec / 1024) load_to_lds(to + (w + i * NW) * 1024, from, (w + i * NW) * 1024 + lane * 16);
  };
  auto ask_qv = [&](int c, int lane) __attribute__((always_inline)) {
    if constexpr (SCORES) q_rows_in.template load<ALL>(sQ, c, present(c), w, lane, tid);
    if (!ident) v_rows_in.template load<ALL>(sV, c, present(c), w, lane, tid);
  };
  // Waits for this wave's part of chunk c's rows (and for everything else it asked for).
  auto arrived = [&](int c, int n, int lane) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0f70);             // vmcnt(0); expcnt and lgkmcnt as they are
    if (n < kQ) {
      k_rows_in.clear(sKK[c & 1], n, w, lane);
      if constexpr (SCORES) q_rows_in.clear(sQ, n, w, lane);
      v_rows_in.clear(sV, n, w, lane);
    }
  };
  if constexpr (MOVE > 0) {
    if (!ALL) {                                     // columns that the loads leave alone
      k_rows_in.clear(sKK[0], 0, w, lane0);
      k_rows_in.clear(sKK[1], 0, w, lane0);
      if constexpr (SCORES) q_rows_in.clear(sQ, 0, w, lane0);
      v_rows_in.clear(sV, 0, w, lane0);
      __builtin_amdgcn_s_waitcnt(0xc07f);           // lgkmcnt(0): before the loads into the same slots
    }
  }
  const int c_first = BACK ? c_end - 1 : c_begin, c_step = BACK ? -1 : 1;
  if (count > 0) {
    ask_k(c_first, lane0);
    if (AHEAD) ask_record(c_first, lane0);
    ask_qv(c_first, lane0);
  }

  // E[t][u][e] is the entry k = 32 t + 8 g + 4 u + e, column 16 w + c16 of the block
  const int g0 = lane0 >> 4, col = 16 * w + (lane0 & 15);
  f32x4_t E[KT][2];
  auto there = [&](int t, int u, int e) { return ALL || (32 * t + 8 * g0 + 4 * u + e < K && col < width); };
  auto entry = [&](int t, int u, int e) {           // in a state in memory
    return static_cast<uint32_t>((32 * t + 8 * g0 + 4 * u + e) * V + col0 + col);
  };
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) f(t, u, e);
  };
  const float* src = nullptr;
  if constexpr (!STATE) {
    if (nseg > 1) src = p.seg + (bh * nseg + seg) * static_cast<int64_t>(K) * V;
    else if (p.carry) src = p.carry + bh * static_cast<int64_t>(K) * V;
  }
  each([&](int t, int u, int e) { E[t][u][e] = ident && 32 * t + 8 * g0 + 4 * u + e == col0 + col ? 1.0f : 0.0f; });
  if (src)
    each([&](int t, int u, int e) {
      if (there(t, u, e)) E[t][u][e] = src[entry(t, u, e)];
    });
  auto put_state = [&](float* dst) __attribute__((always_inline)) {
    each([&](int t, int u, int e) {
      if (there(t, u, e)) dst[entry(t, u, e)] = E[t][u][e];
    });
  };
  if (count > 0) arrived(c_first, present(c_first), lane0);

#pragma unroll 1
  for (int done = 0, c = c_first; done < count; ++done, c += c_step) {
    const int n = present(c);
    const bool more = done + 1 < count;
    if constexpr (MODE == kSave || MODE == kBack) { // the state that enters a stretch of p.every chunks
      if (BACK ? c + 1 == live || (c + 1) % p.every == 0 : c % p.every == 0)
        put_state(p.kept + (bh * ((nchunks + p.every - 1) / p.every) + c / p.every) * static_cast<int64_t>(K) * V);
    }
    // (opaque, so that the chunk's many LDS and memory addresses are formed here from the lane's number)
    int lane = lane_id();
    asm volatile("" : "+v"(lane));
    const int g = lane >> 4, c16 = lane & 15;
    barrier_lds();                                  // the tiles of chunk c are complete
    if (!AHEAD) ask_record(c, lane);
    if (more) {
      ask_k(c + c_step, lane);
      if (AHEAD) ask_record(c + c_step, lane);
    }
    const char* rec = sRec[AHEAD ? c & 1 : 0];
    const float* vec = reinterpret_cast<const float*>(rec + kTBytes<ACT>);
    const char *t_in = rec + lane * (kOne / 64), *p_in = t_in + kTBytes<ACT> + kVecs * 256;   // operands of T, of the scores
    const uint32_t k_tile = lds_address(sKK[0]) + (c & 1) * (kQ * RK);
    const int perm_row = 8 * (c16 >> 2) + (c16 & 3);
    const uint32_t q_rows = O::template row_part<RK, true>(lds_address(sQ), perm_row, g);
    const uint32_t k_rows = O::template row_part<RK, true>(k_tile, perm_row, g);
    auto eight = [&](int which, int t, float (&x)[8]) __attribute__((always_inline)) {   // a vector's tokens 32 t + 8 g ..
      const float4 a = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g);
      const float4 d = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g + 4);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = d.x; x[5] = d.y; x[6] = d.z; x[7] = d.w;
    };
    // rows of the permuted tile (t, u), columns 32 y + 8 g ..
    auto permuted = [&](uint32_t rows, int t, int u, int y) __attribute__((always_inline)) {
      return O::row(rows + t * (32 * RK), (4 * PB * y) ^ (u ? swizzle<RK, kF32, true>(4) << 4 : 0), 4 * u * RK);
    };

    // ---- K E (rows token 32 t + 8 g + 4 u + e, column v) and Q E, transposed (rows v, column j = place(jt)).  Products
    // on different sums follow each other, here and below: one on the last's sum waits for it.
    auto place = [&](int jt) { return 32 * (jt / 2) + 4 * (jt % 2) + perm_row; };     // token of column c16 of tile jt
    f32x4_t R[2][2], acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = R[i / 2][i % 2] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int y = 0; y < KT; ++y) {
      piece ef[NT], kf[4], qf[4];
      const float x[8] = {E[y][0][0], E[y][0][1], E[y][0][2], E[y][0][3], E[y][1][0], E[y][1][1], E[y][1][2], E[y][1][3]};
      O::template split<NT>(x, ef);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kf[i] = permuted(k_rows, i / 2, i % 2, y);
        if constexpr (MODE == kOut) qf[i] = permuted(q_rows, i / 2, i % 2, y);
      }
#pragma unroll
      for (int m = NT - 1; m >= 0; --m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i / 2][i % 2] = O::mma(kf[i], ef[m], R[i / 2][i % 2]);
        if constexpr (MODE == kOut) {
          if (m < OT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = O::mma(ef[m], qf[i], acc[i]);
          }
        }
      }
    }
    // ---- the wave's own columns of v
    piece vf[2];
    {
      const uint32_t v_cols = O::template column_part<RV, false>(lds_address(sV), 16 * w, 4, lane);
#pragma unroll
      for (int t = 0; t < 2; ++t) vf[t] = ident ? O::zero() : O::template column<RV, false>(v_cols, 0, 32 * t * RV);
    }
    if (!AHEAD) __builtin_amdgcn_s_waitcnt(0x0f70); // the record is here
    barrier_lds();                                  // ... of every wave; the tiles of q and v are free
    if constexpr (!BACK) {
      if (more) ask_qv(c + c_step, lane);
    }

    // ---- X = V - exp(G) K E (backwards scale P^T D + exp(G_Q - G) K E)
    // Forwards, a value that is not finite must not reach earlier tokens' outputs through T's zeros: its column is cut there,
    // its outputs from that token on and its state are NaN.  So are all columns from a token on whose row of A is not
    // finite (the pre-pass of segments has its NaN from exp(G_Q)).
    float x[2][8];
    float odd = MODE == kOut ? 0.0f * vec[kWhole * 64] : 0.0f;
    f32x4_t Z[2][2];
    if constexpr (BACK) {
#pragma unroll
      for (int i = 0; i < 4; ++i) Z[i / 2][i % 2] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = NT - 1; m >= 0; --m) {
        piece pf[kT];
#pragma unroll
        for (int i = 0; i < kT; ++i) load_piece(p_in + (i * NT + m) * kOne, pf[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) Z[i / 2][i % 2] = O::mma(pf[i], vf[0], Z[i / 2][i % 2]);
#pragma unroll
        for (int u = 0; u < 2; ++u) Z[1][u] = O::mma(pf[4 + u], vf[1], Z[1][u]);
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float with[8];
      eight(BACK ? kLast : kInto, t, with);
      if constexpr (BACK) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[t][e] = __builtin_fmaf(with[e], R[t][e / 4][e % 4], Z[t][e / 4][e % 4]);
      } else {
        O::unpack(vf[t], x[t]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[t][e] = __builtin_fmaf(-with[e], R[t][e / 4][e % 4], x[t][e]);
        if constexpr (MODE == kOut) {
          float beta[8];
          eight(kBeta, t, beta);
#pragma unroll
          for (int e = 0; e < 8; ++e) odd = __builtin_fmaf(x[t][e], 0.0f, __builtin_fmaf(beta[e], 0.0f, odd));
        }
      }
    }
    const bool bad = MODE == kOut && __builtin_amdgcn_ballot_w64(odd != odd) != 0;
    int gone = kQ;                                  // first token of the column that is not finite
    if (__builtin_expect(bad, 0)) {
      gone = static_cast<int>(vec[kFirstOdd * 64]);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float beta[8];
        eight(kBeta, t, beta);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(fabsf(x[t][e]) < __builtin_huge_valf()) || !(fabsf(beta[e]) < __builtin_huge_valf()))
            gone = least(gone, 32 * t + 8 * g + e);
      }
      gone = least(gone, __shfl_xor(gone, 16));
      gone = least(gone, __shfl_xor(gone, 32));
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (32 * t + 8 * g + e >= gone) x[t][e] = 0.0f;
    }

    // ---- W = T X, then U = beta W
    f32x4_t U[2][2];
    {
      piece xf[2][NT];
#pragma unroll
      for (int t = 0; t < 2; ++t) O::template split<NT>(x[t], xf[t]);
      f32x4_t s[kT];
#pragma unroll
      for (int i = 0; i < kT; ++i) s[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = NT - 1; m >= 0; --m) {           // (the products of terms that count at NT terms, largest last)
        piece T[kT];
#pragma unroll
        for (int i = 0; i < kT; ++i) load_piece(t_in + (i * NT + m) * kOne, T[i]);
#pragma unroll
        for (int other = NT - 1 - m; other >= 0; --other)
#pragma unroll
          for (int i = 0; i < kT; ++i) s[i] = O::mma(T[i], xf[i / 4][other], s[i]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        U[0][u] = s[u];
        U[1][u] = s[2 + u] + s[4 + u];
      }
    }
    if constexpr (MODE == kSave || MODE == kBack) { // kept for the gradients of q and k (every column of the tiles)
      float* w_out = p.w_out + ((bh * nchunks + c) * kQ) * p.w_stride + col0 + 16 * w + c16;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int row = 32 * t + 8 * g + e;
          w_out[(BACK ? kQ - 1 - row : row) * p.w_stride] = U[t][e / 4][e % 4];
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float beta[8];
      eight(kBeta, t, beta);
#pragma unroll
      for (int e = 0; e < 8; ++e) U[t][e / 4][e % 4] *= beta[e];
    }
    if (__builtin_expect(bad, 0)) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (32 * t + 8 * g + e >= gone) U[t][e / 4][e % 4] = 0.0f;
    }
    if constexpr (MODE == kBack) {                  // dV, token by token
      const int64_t row_stride = static_cast<int64_t>(p.H) * V;
      const int64_t first = (b * L + static_cast<int64_t>(c) * kQ) * row_stride + static_cast<int64_t>(h) * V + col0;
      if (ALL || 16 * w + c16 < width) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = kQ - 1 - (32 * t + 8 * g + e);
            const float y = U[t][e / 4][e % 4];
            if (at >= n) continue;
            if (p.o_f32) static_cast<float*>(p.o)[first + at * row_stride + 16 * w + c16] = y;
            else store_act<ACT>(p.o, first + at * row_stride + 16 * w + c16, y);
          }
      }
    }

    // ---- outputs: exp(G) Q E and the scores' product with U on top
    if constexpr (MODE == kOut) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const float f = p.scale * vec[kInto * 64 + place(jt)];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[jt][e] *= f;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        piece uf[OT], pf[4][OT];
        const float y[8] = {U[t][0][0], U[t][0][1], U[t][0][2], U[t][0][3], U[t][1][0], U[t][1][1], U[t][1][2], U[t][1][3]};
        O::template split<OT>(y, uf);
#pragma unroll
        for (int jt = 2 * t; jt < 4; ++jt)
#pragma unroll
          for (int m = 0; m < OT; ++m) load_piece(p_in + ((jt + 2 * t) * OT + m) * kOne, pf[jt][m]);
#pragma unroll
        for (int sum = OT - 1; sum >= 0; --sum)
#pragma unroll
          for (int m = 0; m <= sum; ++m)
#pragma unroll
            for (int jt = 2 * t; jt < 4; ++jt) acc[jt] = O::mma(uf[m], pf[jt][sum - m], acc[jt]);
      }
      if (__builtin_expect(bad, 0)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {               // (the outputs' rows are the lanes' columns of x)
          const int from = __shfl(gone, 4 * g + e);
#pragma unroll
          for (int jt = 0; jt < 4; ++jt)
            if (place(jt) >= from) acc[jt][e] = __builtin_nanf("");
        }
      }
    }

    // ---- the state: exp(G_Q) E + K^T (exp(G_Q - G) U), backwards exp(G_Q) E - K^T (exp(G) U) + Q^T (scale exp(G) D)
    const float whole = vec[kWhole * 64];
    each([&](int t, int u, int e) { E[t][u][e] *= whole; });
    const uint32_t k_cols = O::template column_part<RK, true>(k_tile, 0, 8, lane);
    const uint32_t q_cols = O::template column_part<RK, true>(lds_address(sQ), 0, 8, lane);   // (backwards)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float with[8], y[8];
      eight(BACK ? kInto : kLast, t, with);
      piece wf[NT], df[NT];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (BACK ? -with[e] : with[e]) * U[t][e / 4][e % 4];
      O::template split<NT>(y, wf);
      if constexpr (BACK) {
        O::unpack(vf[t], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= p.scale * with[e];
        O::template split<NT>(y, df);
      }
#pragma unroll
      for (int z = 0; z < KT; z += 2) {             // four tiles at a time
        piece kf[4], qf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = (4 * PB * (z + i / 2)) ^ O::half_flip(i % 2), offset = 32 * t * RK + O::half_offset(i % 2);
          kf[i] = O::template column<RK, true>(k_cols, at, offset);
          if constexpr (BACK) qf[i] = O::template column<RK, true>(q_cols, at, offset);
        }
#pragma unroll
        for (int m = NT - 1; m >= 0; --m) {
#pragma unroll
          for (int i = 0; i < 4; ++i) E[z + i / 2][i % 2] = O::mma(kf[i], wf[m], E[z + i / 2][i % 2]);
          if constexpr (BACK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) E[z + i / 2][i % 2] = O::mma(qf[i], df[m], E[z + i / 2][i % 2]);
          }
        }
      }
    }
    if constexpr (BACK) {
      barrier_lds();                                // the tiles of q and of the outputs' gradient are free
      if (more) ask_qv(c + c_step, lane);
    }
    if (__builtin_expect(bad, 0)) {
      if (gone < kQ) each([&](int t, int u, int e) { E[t][u][e] = __builtin_nanf(""); });
    }
    arrived(c + c_step, more ? present(c + c_step) : kQ, lane);

    // ---- the output rows to memory: lane (g, c) has 4 columns of token place(jt)
    if constexpr (MODE == kOut) {
      auto four = [](const f32x4_t& a) __attribute__((always_inline)) {
        if constexpr (kF32) return make_float4(a[0], a[1], a[2], a[3]);
        else return make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
      };
      const int64_t row_stride = static_cast<int64_t>(p.H) * V;
      const int v0 = 16 * w + 4 * g;
      if (n == kQ && p.o_vec) {                     // a uniform address, the lane's offset, 16 rows' bytes
        char* rows = static_cast<char*>(p.o) + ((b * L + static_cast<int64_t>(c) * kQ) * row_stride + static_cast<int64_t>(h) * V + col0) *
                                                   static_cast<int64_t>(sizeof(elem));
        const uint32_t step = static_cast<uint32_t>(row_stride) * sizeof(elem), off = v0 * sizeof(elem);
        if (ALL || v0 < width) {
#pragma unroll
          for (int jt = 0; jt < 4; ++jt) *reinterpret_cast<decltype(four(acc[0]))*>(rows + (off + place(jt) * step)) = four(acc[jt]);
        }
        continue;
      }
      elem* out = static_cast<elem*>(p.o) + (b * L + static_cast<int64_t>(c) * kQ) * row_stride + static_cast<int64_t>(h) * V +
                  col0 + v0;
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const int row = place(jt);
        if (c * kQ + row >= L) continue;
        elem* o = out + row * row_stride;
        if (row >= n) acc[jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (p.o_vec) {
          if (ALL || v0 < width) *reinterpret_cast<decltype(four(acc[0]))*>(o) = four(acc[jt]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (v0 + e >= width) continue;
            if constexpr (kF32) o[e] = acc[jt][e];
            else o[e] = to_bf16(acc[jt][e]);
          }
        }
      }
    }
  }

  // tokens that are not there: zeros (forwards those of the last chunk have theirs)
  if constexpr (MODE == kOut || MODE == kBack) {
    const int from = BACK ? len / kQ : live;
    for (int z = from > c_begin ? from : c_begin; z < c_stop; ++z) {
      for (int i = tid; i < kQ * kColumns; i += 64 * NW) {
        const int64_t token = static_cast<int64_t>(z) * kQ + i / kColumns;
        if (token >= L) break;
        if (token < len || i % kColumns >= width) continue;
        const int64_t at = ((b * L + token) * p.H + h) * V + col0 + i % kColumns;
        if (BACK && p.o_f32) static_cast<float*>(p.o)[at] = 0.0f;
        else static_cast<elem*>(p.o)[at] = elem(0);
      }
    }
  }
  if constexpr (STATE) {
    if (!ident) {
      put_state(p.seg + (bh * nseg + seg) * static_cast<int64_t>(K) * V);
    } else {                                        // whole tiles of M, and its transpose for the backward walk
      float* m = p.seg_m + (bh * nseg + seg) * static_cast<int64_t>(KD * KD);
      float* mt = p.seg_mt ? p.seg_mt + (bh * nseg + seg) * static_cast<int64_t>(KD * KD) : nullptr;
      each([&](int t, int u, int e) {
        const int k = 32 * t + 8 * g0 + 4 * u + e;
        if (COLUMNS > KD && col >= KD) return;
        m[k * KD + col0 + col] = E[t][u][e];
        if (mt) mt[(col0 + col) * KD + k] = E[t][u][e];
      });
    }
  } else if (p.fin) {
    // forwards the segment of the last token that is there has the state after it, backwards the first segment
    if (BACK ? seg == 0 : live == 0 ? seg == 0 : count > 0 && c_end == live) put_state(p.fin + bh * static_cast<int64_t>(K) * V);
  }
}

// The states that enter the segments, over what each made of none: forwards S = M S + N from the first on, backwards
// F = M^T F + N from the last.  A workgroup takes 16 columns through all segments, wave w rows 32 w .. of them; the state
// goes round in operand order through LDS.  Float32 products.
template <int KD, bool BACK>
__global__ __launch_bounds__(2 * KD) void gd_chain_kernel(GdArgs p) {
  using O = Op<ActF32>;
  constexpr int KT = KD / 32;
  __shared__ __attribute__((aligned(16))) F8 sS[2][KT][64];
  const int lane = threadIdx.x & 63, w = uniform_int(threadIdx.x >> 6), g = lane >> 4, c16 = lane & 15;
  const int K = p.K, V = p.V, nseg = p.nseg;
  const int64_t bh = blockIdx.x;
  const int col = 16 * blockIdx.y + c16;
  const int len = gd_length(p.lengths, static_cast<int>(p.L), blockIdx.x / static_cast<uint32_t>(p.H));
  const int live = (len + kQ - 1) / kQ, count = (live + p.seg_chunks - 1) / p.seg_chunks;   // segments with tokens
  float S[8];                                       // rows 32 w + 8 g + e, column c16
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = 32 * w + 8 * g + e;
      f(e, k < K && col < V, k * V + col);
    }
  };
  const float* carry = p.carry ? p.carry + bh * static_cast<int64_t>(K) * V : nullptr;
  each([&](int e, bool in, int at) { S[e] = carry && in ? carry[at] : 0.0f; });
  const float* ms = (BACK ? p.seg_mt : p.seg_m) + bh * nseg * static_cast<int64_t>(KD * KD);
  float* segs = p.seg + bh * nseg * static_cast<int64_t>(K) * V;
  for (int i = 0; i < (count > 0 ? count : 1); ++i) {
    const int s = BACK && count > 0 ? count - 1 - i : i;
    float* at_s = segs + s * static_cast<int64_t>(K) * V;
    const bool on = i + 1 < count;                  // (the last one's result is the walk's to find)
    f32x4_t next[2];
    F8 m[2][KT];
    if (on) {
      each([&](int e, bool in, int at) { next[e / 4][e % 4] = in ? at_s[at] : 0.0f; });
      const float* from = ms + s * static_cast<int64_t>(KD * KD) + (32 * w + 8 * (c16 >> 2) + (c16 & 3)) * KD + 8 * g;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int y = 0; y < KT; ++y) load_piece(reinterpret_cast<const char*>(from + 4 * u * KD + 32 * y), m[u][y]);
    }
    each([&](int e, bool in, int at) {
      if (in) at_s[at] = S[e];
    });
    if (!on) break;
    sS[i & 1][w][lane] = O::pack(S);
    __syncthreads();                                // (the other buffer was read before)
#pragma unroll
    for (int y = 0; y < KT; ++y) {
      const F8 right = sS[i & 1][y][lane];
#pragma unroll
      for (int u = 0; u < 2; ++u) next[u] = O::mma(m[u][y], right, next[u]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) S[e] = next[e / 4][e % 4];
  }
}

template <typename ACT, int KD, int COLUMNS, int MOVE, bool ALL, int MODE, int PR>
void launch_walk(const GdArgs& a, hipStream_t s) {
  const int64_t items = (a.batch * a.H * a.nseg + 7) / 8 * 8;
  const int64_t blocks = (a.V + COLUMNS - 1) / COLUMNS + (MODE == kState ? (a.K + COLUMNS - 1) / COLUMNS : 0);
  hipLaunchKernelGGL((gd_walk_kernel<ACT, KD, COLUMNS, MOVE, ALL, MODE, PR>), dim3(static_cast<unsigned>(items * blocks)),
                     dim3(4 * COLUMNS), 0, s, a);
}

template <typename ACT, int KD, int COLUMNS, int MOVE, bool ALL, int MODE>
void launch_gd_t(const GdArgs& a, hipStream_t s) {
  constexpr bool BACK = MODE == kBack;
  constexpr int PR = score_terms<ACT, MODE>();
  if (a.nseg > 1) {
    launch_walk<ACT, KD, COLUMNS, MOVE, ALL, BACK ? kBackState : kState, PR>(a, s);
    const dim3 grid(static_cast<unsigned>(a.batch * a.H), static_cast<unsigned>((a.V + 15) / 16));
    hipLaunchKernelGGL((gd_chain_kernel<KD, BACK>), grid, dim3(2 * KD), 0, s, a);
  }
  launch_walk<ACT, KD, COLUMNS, MOVE, ALL, MODE, PR>(a, s);
}

// Columns of a workgroup.  128 where more than half of the CUs have work then: the rows of q and k and the record are read once for
// them, and two waves a SIMD hide each other's waits.  64 where that leaves each workgroup a CU of its own, and for rows that
// do not move as whole vectors.  2048 tokens, heads of 128, us with 128 and with 64 columns: bfloat16, 80 pairs of batch row and head 213 and
// 167, 120 pairs 237 and 198, 160 pairs 260 and 341 (two rounds: two workgroups of about 120 KB of LDS do not fit a CU); float32, 80 pairs
// 679 and 486, 160 pairs 767 and 917; 256 pairs, gradient, 1431 and 1568.
bool wide(const GdArgs& a, int KD) {
  return a.move == 16 && a.K == KD && a.V == 128 && a.batch * a.H * a.nseg > 128;
}

template <int MODE>
void launch_gd_mode(const GdArgs& args, Dt dt, hipStream_t s) {
  GdArgs a = args;
  const int64_t nch = (a.L + kQ - 1) / kQ;
  a.seg_chunks = static_cast<int>((nch + a.nseg - 1) / a.nseg);
  auto go = [&](auto act, auto kd) {
    using ACT = decltype(act);
    constexpr int KD = decltype(kd)::value;
    auto prepare = [&](auto move) {
      const int64_t all = (a.batch * a.H * nch + 3) / 4, most = 1 << 22;   // (a launch's threads are fewer than 2^32)
      hipLaunchKernelGGL((gd_prepare_kernel<ACT, KD, decltype(move)::value, MODE == kBack, score_terms<ACT, MODE>()>),
                         dim3(static_cast<unsigned>(all < most ? all : most)), dim3(256), 0, s, a);
    };
    if (a.move == 16) prepare(std::integral_constant<int, 16>{});
    else if (a.move == 4 && a.K >= 8) prepare(std::integral_constant<int, 4>{});
    else prepare(std::integral_constant<int, 0>{});
    if (wide(a, KD)) launch_gd_t<ACT, KD, 128, 16, true, MODE>(a, s);
    else if (a.move == 16 && a.K == KD && a.V % 64 == 0) launch_gd_t<ACT, KD, 64, 16, true, MODE>(a, s);
    else if (a.move == 16) launch_gd_t<ACT, KD, 64, 16, false, MODE>(a, s);
    else if (ACT::kBytes == 4 || a.move == 4) launch_gd_t<ACT, KD, 64, 4, false, MODE>(a, s);
    else if constexpr (ACT::kBytes == 2) launch_gd_t<ACT, KD, 64, 0, false, MODE>(a, s);
  };
  auto shape = [&](auto act) {
    if (a.K > 64) go(act, std::integral_constant<int, 128>{});
    else go(act, std::integral_constant<int, 64>{});
  };
  if (dt == Dt::BF16) shape(ActBF16{});
  else shape(ActF32{});
}

}  // namespace

GdRecords gd_records(Dt dt) {
  auto of = [](auto act) {
    using ACT = decltype(act);
    return GdRecords{kRecord<ACT, score_terms<ACT, kOut>()>, kRecord<ACT, score_terms<ACT, kSave>()>,
                     kRecord<ACT, score_terms<ACT, kBack>()>};
  };
  return dt == Dt::BF16 ? of(ActBF16{}) : of(ActF32{});
}

constexpr int kSegTarget = 256;

// Segments per sequence.  The pre-pass walks V + K columns where the main pass walks V, so segments are worth it only
// where few workgroups walk long sequences: up to kSegTarget workgroups of 128 columns, at least 4 segments, each 4 chunks or
// longer.  The count is then derived back from the segment length, so that no segment is without a chunk.
// us with targets of 128, 256 and 512 and without segments, bfloat16, heads of 128: 131072 tokens, 20 heads: 3351, 3200, 3130, 8967;
// 8192 tokens, 32 heads: 351, 336, 392, 582; 4096, 40: 287, 232, 286, 289; 2048, 20: 95, 110, 111, 145; 8192, 64: 638, 618, 655, 639;
// float32 gradient, 2 x 2047, 24 heads of 64: 675, 509, 535, 677.  Two segments (16384 tokens, 100 heads) 2111 for 1409 without.
int gd_segments(int64_t batch, int64_t L, int64_t H) {
  const int64_t workgroups = batch * H, nch = (L + kQ - 1) / kQ;
  int64_t s = kSegTarget / (workgroups > 0 ? workgroups : 1);
  if (s > nch / 4) s = nch / 4;
  if (s < 4) return 1;
  const int64_t per = (nch + s - 1) / s;
  return static_cast<int>((nch + per - 1) / per);
}

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
