// The gated delta rule: the gradients of q, k, g and beta.
//
// Two walks (gated_delta.hip) leave, for every token, w_t = v_t - a_t S_{t-1}^T k_t and y_t = F_t^T k_t (F_t the gradient
// of S_t, its own output's part included), and the states E and their gradients F before every `every` chunks.
// Stretches of so many chunks are independent from there.  With u = beta w, D the outputs' gradient and all of
// token j in a chunk against its tokens i:
//     dq_j = scale S_j d_j               = scale exp(G_j) E d_j + sum_{i<=j} N1_ji k_i,  N1_ji = scale M_ji d_j.u_i
//     dk_j = F_j u_j - beta_j a_j S_{j-1} y_j, of which the second (forwards, with dq)
//          = -beta_j exp(G_j) E y_j + sum_{i<j} N2_ji k_i,                               N2_ji = -beta_j M_ji y_j.u_i
//     and the first (backwards) = exp(G_Q - G_i) F u_i + sum_{j>=i} N1_ji q_j + sum_{j>i} N2_ji k_j
//     dbeta_j = y_j.w_j
// g: a_t scales everything that passes from before t to t and after, so with r_j = exp(G_j) the state's scale, S / r,
// r q and v / r carry all of it: d loss / d G_j = q_j.dq_j - v_j.dv_j, and dg_t is its sum over j >= t.  Summed over a
// stretch only, onto <F, E> at its end: the sum over a long sequence would lose what a fast decay leaves of it.
// v_j.dv_j = beta_j v_j.y_j = y_j.u_j - k_j.(the second part of dk_j), all of which is at hand.
//
// A workgroup walks one stretch; a wave owns 16 or 32 columns of E^T (of K), so that nothing is summed over waves but
// the tokens' scalars.  Rows of D, W and Y lie in LDS (W and Y as terms, split once a workgroup).  q and k are
// needed as a wave's own columns alone and come straight from memory.
//
// Roundings (bfloat16 activations): forwards 24-bit operands, as g's and beta's gradients are float32; backwards, of
// which only dk's bfloat16 sees anything, 16 bits.
#include <type_traits>

#include "device_common.hpp"
#include "gd_common.hpp"
#include "la_tiles.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kMostEvery = 16;

// 64 rows of RB bytes into an LDS tile by 16 bytes a thread; rows past n and columns past `cols` are zeros.
template <typename ELEM, int RB, bool PERM, int THREADS>
__device__ __forceinline__ void stage_rows(char* tile, const ELEM* base, int64_t stride, int n, int cols, bool vec, int tid) {
  constexpr int kSlots = RB / 16, kPer = 16 / sizeof(ELEM);
  constexpr bool kF32 = sizeof(ELEM) == 4;
  static_assert(kQ * kSlots % THREADS == 0, "");
#pragma unroll
  for (int j = 0; j < kQ * kSlots / THREADS; ++j) {
    const int i = tid + j * THREADS, row = i / kSlots, slot = i % kSlots;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (row < n) {
      const ELEM* at = base + row * stride + slot * kPer;
      if (vec) {
        if (slot * kPer < cols) x = *reinterpret_cast<const uint4*>(at);
      } else {
        ELEM v[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = slot * kPer + e < cols ? at[e] : ELEM(0);
        x = __builtin_bit_cast(uint4, v);
      }
    }
    *reinterpret_cast<uint4*>(tile + row * RB + ((slot ^ swizzle<RB, kF32, PERM>(row)) << 4)) = x;
  }
}

// A float32 [64][WD] matrix into NT tiles of its terms.
template <typename ACT, int WD, int NT, bool PERM, int THREADS>
__device__ __forceinline__ void stage_terms(char* tiles, const float* src, int tid) {
  using O = Op<ACT>;
  constexpr int RB = WD * ACT::kBytes;
  if constexpr (ACT::kBytes == 4) {
    stage_rows<float, RB, PERM, THREADS>(tiles, src, WD, kQ, WD, true, tid);
  } else {
    constexpr int kSlots = WD / 8;
    static_assert(kQ * kSlots % THREADS == 0, "");
#pragma unroll
    for (int j = 0; j < kQ * kSlots / THREADS; ++j) {
      const int i = tid + j * THREADS, row = i / kSlots, slot = i % kSlots;
      const float4 a = *reinterpret_cast<const float4*>(src + row * WD + slot * 8);
      const float4 b = *reinterpret_cast<const float4*>(src + row * WD + slot * 8 + 4);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      typename O::piece p[NT];
      O::template split<NT>(v, p);
#pragma unroll
      for (int m = 0; m < NT; ++m)
        *reinterpret_cast<uint4*>(tiles + m * (kQ * RB) + row * RB + ((slot ^ swizzle<RB, false, PERM>(row)) << 4)) = p[m];
    }
  }
}

// BACK: the second kernel, which adds the backward part of dk.
template <typename ACT, int KD, int VD, bool BACK>
__global__ __launch_bounds__(4 * KD, 1)
void gd_qk_kernel(GdGradArgs p) {
  constexpr int VT = 1;
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr bool kF32 = sizeof(elem) == 4;
  constexpr int NW = KD / 16 / VT, THREADS = 64 * NW, NT = BACK ? kOutTerms<ACT> : kTerms<ACT>;
  constexpr int RV = VD * static_cast<int>(sizeof(elem)), KT = VD / 32, PB = O::kPiece, kOne = kPieceBytes<ACT>;
  constexpr bool PW = !BACK, PY = BACK;             // whose rows are read as permuted ones
  __shared__ __attribute__((aligned(512))) char sD[kQ * RV];
  __shared__ __attribute__((aligned(512))) char sW[NT][kQ * RV];
  __shared__ __attribute__((aligned(512))) char sY[NT][kQ * RV];
  __shared__ __attribute__((aligned(512))) char sN[2][kT * NT * kOne];
  __shared__ __attribute__((aligned(16))) float vec[kVecs * 64];
  __shared__ float sSum[NW][kQ], sDiag[kQ], sAll[BACK ? 1 : kMostEvery * kQ];

  const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6), g = lane >> 4, c16 = lane & 15;
  const int L = static_cast<int>(p.L), K = p.K, V = p.V;
  const int nchunks = (L + kQ - 1) / kQ, stretches = (nchunks + p.every - 1) / p.every;
  const uint32_t pair = blockIdx.x / static_cast<uint32_t>(stretches), s = blockIdx.x - pair * stretches;
  const uint32_t row_b = pair / static_cast<uint32_t>(p.H);
  const int64_t bh = pair, b = row_b;
  const int h = static_cast<int>(pair - row_b * static_cast<uint32_t>(p.H));
  const int len = gd_length(p.lengths, L, b), c_live = (len + kQ - 1) / kQ;
  const int c_begin = static_cast<int>(s) * p.every, c_end = least(c_begin + p.every, c_live);
  const elem* qg = static_cast<const elem*>(p.q) + b * p.qs[0] + (h / p.qdiv) * p.qs[2];
  const elem* kg = static_cast<const elem*>(p.k) + b * p.ks[0] + (h / p.kdiv) * p.ks[2];
  const elem* dg = static_cast<const elem*>(p.d) + b * p.ds[0] + h * p.ds[2];
  const int64_t out_row = static_cast<int64_t>(p.H) * K;
  const int64_t out_base = b * L * out_row + static_cast<int64_t>(h) * K;

  // tokens of this stretch that are not there: zeros
  {
    const int stop = least(L, (c_begin + p.every) * kQ), from = len > c_begin * kQ ? len : c_begin * kQ;
    for (int64_t i = tid; i < static_cast<int64_t>(stop - from) * K; i += THREADS) {
      const int64_t at = out_base + (from + i / K) * out_row + i % K;
      if constexpr (BACK) {
        if (!p.dk_f32) store_act<ACT>(p.dk, at, 0.0f);
      } else {
        if (p.dq_f32) static_cast<float*>(p.dq)[at] = 0.0f;
        else store_act<ACT>(p.dq, at, 0.0f);
        p.dk_part[at] = 0.0f;
      }
    }
    if constexpr (!BACK) {
      for (int i = tid; i < stop - from; i += THREADS) {
        const int64_t at = (b * L + from + i) * p.H + h;
        p.dg[at] = 0.0f;
        p.dbeta[at] = 0.0f;
      }
    }
  }
  if (c_begin >= c_end) return;

  // E[vt][y][u][e] is the entry v = 32 y + 8 g + 4 u + e, k = 16 (VT w + vt) + c16 (backwards of the gradient F)
  f32x4_t E[VT][KT][2];
  auto there = [&](int vt, int y, int u, int e) {
    return 16 * (VT * w + vt) + c16 < K && 32 * y + 8 * g + 4 * u + e < V;
  };
  auto place = [&](int vt, int y, int u, int e) {
    return static_cast<uint32_t>((16 * (VT * w + vt) + c16) * V + 32 * y + 8 * g + 4 * u + e);
  };
  {
    const float* src = (BACK ? p.kept_f : p.kept_e) + (bh * stretches + s) * static_cast<int64_t>(K) * V;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) E[vt][y][u][e] = there(vt, y, u, e) ? src[place(vt, y, u, e)] : 0.0f;
  }
  const uint32_t tile_d = lds_address(sD), tile_w = lds_address(sW[0]), tile_y = lds_address(sY[0]);
  const int perm_row = 8 * (c16 >> 2) + (c16 & 3);
  const uint32_t d_rows = O::template row_part<RV, BACK>(tile_d, BACK ? perm_row : c16, g);
  const uint32_t w_rows = O::template row_part<RV, PW>(tile_w, BACK ? c16 : perm_row, g);
  const uint32_t y_rows = O::template row_part<RV, PY>(tile_y, BACK ? perm_row : c16, g);
  // rows 16 jt + c16, or of the permuted tile (t, u)
  auto natural = [&](uint32_t rows, int jt, int y, int m) { return O::row(rows + jt * (16 * RV), 4 * PB * y, m * (kQ * RV)); };
  auto permuted = [&](uint32_t rows, int t, int u, int y, int m) {
    return O::row(rows + t * (32 * RV), (4 * PB * y) ^ (swizzle<RV, kF32, true>(4 * u) << 4), 4 * u * RV + m * (kQ * RV));
  };
  auto eight = [&](int which, int t, float (&x)[8]) __attribute__((always_inline)) {
    const float4 a = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g);
    const float4 d = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = d.x; x[5] = d.y; x[6] = d.z; x[7] = d.w;
  };

#pragma unroll 1
  for (int done = 0; done < c_end - c_begin; ++done) {
    const int c = BACK ? c_end - 1 - done : c_begin + done;
    const int n = least(len - c * kQ, kQ);
    const int64_t t0 = static_cast<int64_t>(c) * kQ;
    stage_rows<elem, RV, BACK, THREADS>(sD, dg + t0 * p.ds[1], p.ds[1], n, V, p.d_vec, tid);
    stage_terms<ACT, VD, NT, PW, THREADS>(sW[0], p.w + ((bh * nchunks + c) * kQ) * VD, tid);
    stage_terms<ACT, VD, NT, PY, THREADS>(sY[0], p.y + ((bh * nchunks + c) * kQ) * VD, tid);
    {
      const float* from = reinterpret_cast<const float*>(p.rec + (bh * nchunks + c) * kRecord<ACT, 0> + kTBytes<ACT>);
      for (int i = tid; i < kVecs * 64; i += THREADS) vec[i] = from[i];
    }
    // the wave's own columns of k (and of q): tokens 32 t + 8 g + e of column c16
    piece kf[VT][2], qf[VT][2];
    auto columns = [&](const elem* base, int64_t stride, piece (&out)[VT][2]) __attribute__((always_inline)) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        const int col = 16 * (VT * w + vt) + c16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          elem v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = 32 * t + 8 * g + e;
            v[e] = row < n && col < K ? base[(t0 + row) * stride + col] : elem(0);
          }
          out[vt][t] = __builtin_bit_cast(piece, v);
        }
      }
    };
    columns(kg, p.ks[1], kf);
    if constexpr (BACK) columns(qg, p.qs[1], qf);
    __syncthreads();

    // ---- N1 and N2 in operand order.  Forwards as the scores: column j = 16 jt + c16, tokens i = 32 t + 8 g + e.
    // Backwards column i, tokens j; i in the first half takes both halves of j, i in the second the second.
#pragma unroll 1
    for (int z = w; z < 2 * kT; z += NW) {
      const int second = z >= kT, x = second ? z - kT : z;
      const int jt = x < 4 ? x : BACK ? x - 4 : x - 2, t = BACK ? (x < 4 ? 1 : 0) : (x < 4 ? 0 : 1);
      f32x4_t a[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) a[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int y = 0; y < KT; ++y) {
        piece right[NT];
        if (BACK || second) {                       // W, or Y
#pragma unroll
          for (int m = 0; m < NT; ++m) right[m] = natural(BACK ? w_rows : y_rows, jt, y, m);
        } else {
          right[0] = natural(d_rows, jt, y, 0);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (BACK) {
            if (second) {
              piece left[NT];
#pragma unroll
              for (int m = 0; m < NT; ++m) left[m] = permuted(y_rows, t, u, y, m);
              a[u] = mma_terms<O, NT, NT>(left, right, a[u]);
            } else {
              const piece left = permuted(d_rows, t, u, y, 0);
#pragma unroll
              for (int m = NT - 1; m >= 0; --m) a[u] = O::mma(left, right[m], a[u]);
            }
          } else {
            piece left[NT];
#pragma unroll
            for (int m = 0; m < NT; ++m) left[m] = permuted(w_rows, t, u, y, m);
            if (second) {
              a[u] = mma_terms<O, NT, NT>(left, right, a[u]);
            } else {
#pragma unroll
              for (int m = NT - 1; m >= 0; --m) a[u] = O::mma(left[m], right[0], a[u]);
            }
          }
        }
      }
      const int col = 16 * jt + c16;                // forwards j, backwards i
      float hi[8], lo[8], beta[8], v[8];
      eight(kSumHi, t, hi);
      eight(kSumLo, t, lo);
      eight(kBeta, t, beta);
      const float chi = vec[kSumHi * 64 + col], clo = vec[kSumLo * 64 + col], cbeta = vec[kBeta * 64 + col];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 32 * t + 8 * g + e;
        const float m = BACK ? exp2_pair(hi[e] - chi, lo[e] - clo) : exp2_pair(chi - hi[e], clo - lo[e]);
        const float raw = a[e / 4][e % 4];
        const bool in = BACK ? (second ? row > col : row >= col) : (second ? row < col : row <= col);
        if (!BACK && second && row == col) sDiag[col] = raw;
        const float f = second ? -(beta[e] * cbeta) * m : p.scale * (BACK ? cbeta : beta[e]) * m;
        v[e] = in ? raw * f : 0.0f;
      }
      piece out[NT];
      O::template split<NT>(v, out);
#pragma unroll
      for (int m = 0; m < NT; ++m) store_piece(sN[second] + (x * NT + m) * kOne + lane * (kOne / 64), out[m]);
    }

    // ---- the state's part, rows k, column j = 16 jt + c16: acc of D (and of Y), backwards of W
    f32x4_t acc[VT][4], acy[VT][4];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) acc[vt][jt] = acy[vt][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
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
      for (int jt = 0; jt < 4; ++jt) {
        piece r[NT];
#pragma unroll
        for (int m = 0; m < NT; ++m) r[m] = natural(BACK ? w_rows : y_rows, jt, y, m);
        if constexpr (BACK) {
#pragma unroll
          for (int vt = 0; vt < VT; ++vt) acc[vt][jt] = mma_terms<O, NT, NT>(ef[vt], r, acc[vt][jt]);
        } else {
          const piece d = natural(d_rows, jt, y, 0);
#pragma unroll
          for (int vt = 0; vt < VT; ++vt) {
            acy[vt][jt] = mma_terms<O, NT, NT>(ef[vt], r, acy[vt][jt]);
#pragma unroll
            for (int m = NT - 1; m >= 0; --m) acc[vt][jt] = O::mma(ef[vt][m], d, acc[vt][jt]);
          }
        }
      }
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const float beta = vec[kBeta * 64 + 16 * jt + c16];
      const float f = BACK ? vec[kLast * 64 + 16 * jt + c16] * beta : p.scale * vec[kInto * 64 + 16 * jt + c16];
      const float fy = -(beta * vec[kInto * 64 + 16 * jt + c16]);
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[vt][jt][e] *= f;
          if constexpr (!BACK) acy[vt][jt][e] *= fy;
        }
    }
    __syncthreads();                                // N1 and N2 are complete

    // ---- the chunk's own part
#pragma unroll
    for (int x = 0; x < kT; ++x) {
      const int jt = x < 4 ? x : BACK ? x - 4 : x - 2, t = BACK ? (x < 4 ? 1 : 0) : (x < 4 ? 0 : 1);
#pragma unroll
      for (int m = NT - 1; m >= 0; --m) {
        piece n1, n2;
        load_piece(sN[0] + (x * NT + m) * kOne + lane * (kOne / 64), n1);
        load_piece(sN[1] + (x * NT + m) * kOne + lane * (kOne / 64), n2);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          if constexpr (BACK) {
            acc[vt][jt] = O::mma(qf[vt][t], n1, acc[vt][jt]);
            acc[vt][jt] = O::mma(kf[vt][t], n2, acc[vt][jt]);
          } else {
            acc[vt][jt] = O::mma(kf[vt][t], n1, acc[vt][jt]);
            acy[vt][jt] = O::mma(kf[vt][t], n2, acy[vt][jt]);
          }
        }
      }
    }

    // ---- out: lane (g, c) has columns 4 g .. of token 16 jt + c
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const int row = 16 * jt + c16;
      float sum = 0.0f;
      if (row < n) {
        const int64_t token = t0 + row;
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          const int col = 16 * (VT * w + vt) + 4 * g;
          const int64_t at = out_base + token * out_row + col;
          if constexpr (BACK) {
            if (p.part_vec) {
              if (col < K) {
                float4 y = *reinterpret_cast<const float4*>(p.dk_part + at);
                y.x += acc[vt][jt][0]; y.y += acc[vt][jt][1]; y.z += acc[vt][jt][2]; y.w += acc[vt][jt][3];
                if (p.dk_f32) *reinterpret_cast<float4*>(p.dk_part + at) = y;
                else if constexpr (kF32) *reinterpret_cast<float4*>(static_cast<float*>(p.dk) + at) = y;
                else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dk) + at) =
                    make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (col + e >= K) continue;
                const float y = p.dk_part[at + e] + acc[vt][jt][e];
                if (p.dk_f32) p.dk_part[at + e] = y;
                else store_act<ACT>(p.dk, at + e, y);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (col + e >= K) continue;
              sum = __builtin_fmaf(load_act<ACT>(qg, token * p.qs[1] + col + e), acc[vt][jt][e], sum);
              sum = __builtin_fmaf(load_act<ACT>(kg, token * p.ks[1] + col + e), acy[vt][jt][e], sum);
            }
            if (p.part_vec) {
              if (col < K) {
                const f32x4_t& x = acc[vt][jt];
                if (p.dq_f32 || kF32) *reinterpret_cast<float4*>(static_cast<float*>(p.dq) + at) = make_float4(x[0], x[1], x[2], x[3]);
                else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dq) + at) =
                    make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                const f32x4_t& z = acy[vt][jt];
                *reinterpret_cast<float4*>(p.dk_part + at) = make_float4(z[0], z[1], z[2], z[3]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (col + e >= K) continue;
                if (p.dq_f32) static_cast<float*>(p.dq)[at + e] = acc[vt][jt][e];
                else store_act<ACT>(p.dq, at + e, acc[vt][jt][e]);
                p.dk_part[at + e] = acy[vt][jt][e];
              }
            }
          }
        }
      }
      if constexpr (!BACK) {
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (g == 0) sSum[w][row] = sum;
      }
    }

    // ---- the state
    const float whole = vec[kWhole * 64];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) E[vt][y][u][e] *= whole;
    const uint32_t w_cols = O::template column_part<RV, PW>(tile_w, 0, 8, lane);
    const uint32_t y_cols = O::template column_part<RV, PY>(tile_y, 0, 8, lane);
    const uint32_t d_cols = O::template column_part<RV, BACK>(tile_d, 0, 8, lane);
    if (done + 1 < c_end - c_begin || !BACK) {      // (backwards the last is of no use)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float with[8], beta[8], x[8];
        eight(BACK ? kInto : kLast, t, with);
        eight(kBeta, t, beta);
        piece k_in[VT][NT], q_in[VT][NT];
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          O::unpack(kf[vt][t], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= BACK ? -(with[e] * beta[e]) : with[e] * beta[e];
          O::template split<NT>(x, k_in[vt]);
          if constexpr (BACK) {
            O::unpack(qf[vt][t], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= with[e] * p.scale;
            O::template split<NT>(x, q_in[vt]);
          }
        }
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            auto column = [&](uint32_t cols, auto perm, int m) __attribute__((always_inline)) {
              return O::template column<RV, decltype(perm)::value>(cols, (4 * PB * y) ^ O::half_flip(u),
                                                                   32 * t * RV + O::half_offset(u) + m * (kQ * RV));
            };
            piece left[NT];
#pragma unroll
            for (int m = 0; m < NT; ++m)
              left[m] = BACK ? column(y_cols, std::integral_constant<bool, PY>{}, m)
                             : column(w_cols, std::integral_constant<bool, PW>{}, m);
#pragma unroll
            for (int vt = 0; vt < VT; ++vt) E[vt][y][u] = mma_terms<O, NT, NT>(left, k_in[vt], E[vt][y][u]);
            if constexpr (BACK) {
              const piece d = column(d_cols, std::integral_constant<bool, BACK>{}, 0);
#pragma unroll
              for (int vt = 0; vt < VT; ++vt)
#pragma unroll
                for (int m = NT - 1; m >= 0; --m) E[vt][y][u] = O::mma(d, q_in[vt][m], E[vt][y][u]);
            }
          }
      }
    }
    __syncthreads();                                // the tiles are free, the tokens' sums complete
    if constexpr (!BACK) {
      if (tid < n) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) sum += sSum[i][tid];
        sAll[done * kQ + tid] = __builtin_fmaf(-vec[kBeta * 64 + tid], sDiag[tid], sum);
        p.dbeta[(b * L + t0 + tid) * p.H + h] = sDiag[tid];
      }
      __syncthreads();
    }
  }

  if constexpr (!BACK) {
    // <F, E> at the end of the stretch, then the sums back over its tokens
    const float* f = p.kept_f + (bh * stretches + s) * static_cast<int64_t>(K) * V;
    float dot = 0.0f;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (there(vt, y, u, e)) dot = __builtin_fmaf(f[place(vt, y, u, e)], E[vt][y][u][e], dot);
    dot = wave_sum(dot);
    if (lane == 0) sSum[w][0] = dot;
    __syncthreads();
    if (w == 0) {
      double carry = 0.0;
#pragma unroll
      for (int i = 0; i < NW; ++i) carry += sSum[i][0];
      const int first = c_begin * kQ, stop = least(len, c_end * kQ);
      for (int c = c_end - 1; c >= c_begin; --c) {
        const int t = c * kQ + lane;
        double x = t < stop ? static_cast<double>(sAll[t - first]) : 0.0;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const double after = __shfl_down(x, d);
          if (lane + d < 64) x += after;
        }
        x += carry;
        carry = __shfl(x, 0);
        // (the first token of a sequence without a state has nothing to scale)
        if (t < stop) p.dg[(b * L + t) * p.H + h] = t == 0 && !p.carried ? 0.0f : static_cast<float>(x);
      }
    }
  }
}

template <typename ACT, int KD, int VD>
void launch_qk_t(const GdGradArgs& a, hipStream_t s) {
  const int64_t nch = (a.L + kQ - 1) / kQ, stretches = (nch + a.every - 1) / a.every;
  const dim3 grid(static_cast<unsigned>(a.batch * a.H * stretches)), block(4 * KD);
  hipLaunchKernelGGL((gd_qk_kernel<ACT, KD, VD, false>), grid, block, 0, s, a);
  hipLaunchKernelGGL((gd_qk_kernel<ACT, KD, VD, true>), grid, block, 0, s, a);
}

}  // namespace

// Chunks between two kept states: enough stretches for the chip several times over, few states to write and read.
int gd_every(int64_t batch, int64_t L, int64_t H) {
  const int64_t e = batch * H * ((L + kQ - 1) / kQ) / 1024;
  return e < 1 ? 1 : e > kMostEvery ? kMostEvery : static_cast<int>(e);
}

hipError_t launch_gd_qk(const GdGradArgs& a, Dt dt, hipStream_t s) {
  auto shape = [&](auto act) {
    using ACT = decltype(act);
    if (a.K > 64 && a.V > 64) launch_qk_t<ACT, 128, 128>(a, s);
    else if (a.K > 64) launch_qk_t<ACT, 128, 64>(a, s);
    else if (a.V > 64) launch_qk_t<ACT, 64, 128>(a, s);
    else launch_qk_t<ACT, 64, 64>(a, s);
  };
  if (dt == Dt::BF16) shape(ActBF16{});
  else shape(ActF32{});
  return hipGetLastError();
}

}  // namespace ssm
