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
//
// A workgroup walks one stretch; a wave owns 16 columns of E^T (of K), so that only the tokens' scalars are summed over
// waves.  Rows of D, W and Y lie in LDS, W and Y as terms, split once a workgroup; their dot products y.w and y.v are
// taken on the way in.  A chunk's rows are asked for while the one before is worked on.
//
// Roundings (bfloat16 activations): what g's float32 gradient sees (dq, with the states that it is formed from) comes from
// 24-bit operands; what only dk's bfloat16 sees from 16 bits.
#include <type_traits>

#include "device_common.hpp"
#include "gd_common.hpp"
#include "la_tiles.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kMostEvery = 16;

// Eight values of a row, of which `left` are there.
template <typename ACT>
__device__ __forceinline__ typename Op<ACT>::piece load8(const void* base, int64_t at, int left, bool vec) {
  using elem = typename Op<ACT>::elem;
  typename Op<ACT>::piece p = Op<ACT>::zero();
  const elem* from = static_cast<const elem*>(base) + at;
  if (vec) {
    if (left > 0) load_piece(reinterpret_cast<const char*>(from), p);
  } else {
    elem v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? from[e] : elem(0);
    p = __builtin_bit_cast(typename Op<ACT>::piece, v);
  }
  return p;
}
// ... to columns 8 slot .. of an LDS tile's row.
template <int RB, bool PERM>
__device__ __forceinline__ void put8(char* tile, int row, int slot, const uint4& p) {
  *reinterpret_cast<uint4*>(tile + row * RB + ((slot ^ swizzle<RB, false, PERM>(row)) << 4)) = p;
}
template <int RB, bool PERM>
__device__ __forceinline__ void put8(char* tile, int row, int slot, const F8& p) {
  const int flip = swizzle<RB, true, PERM>(row);
  *reinterpret_cast<float4*>(tile + row * RB + (((2 * slot) ^ flip) << 4)) = p.a;
  *reinterpret_cast<float4*>(tile + row * RB + (((2 * slot + 1) ^ flip) << 4)) = p.b;
}

// BACK: the second kernel, which adds the backward part of dk.
template <typename ACT, int KD, int VD, bool BACK>
__global__ __launch_bounds__(4 * KD, 2)
void gd_qk_kernel(GdGradArgs p) {
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr bool kF32 = sizeof(elem) == 4;
  constexpr int NW = KD / 16, THREADS = 64 * NW;
  constexpr int OT = kOutTerms<ACT>, NT = BACK ? OT : kTerms<ACT>;      // terms of Y and N2; of W, E and N1
  constexpr int RV = VD * static_cast<int>(sizeof(elem)), RK = KD * static_cast<int>(sizeof(elem));
  constexpr int KT = VD / 32, PB = O::kPiece, kOne = kPieceBytes<ACT>;
  constexpr bool PW = !BACK, PY = BACK;             // whose rows are read as permuted ones
  constexpr bool TILES = !kF32;                     // q and k by LDS (float32: no room; the waves read their own columns)
  __shared__ __attribute__((aligned(512))) char sD[kQ * RV];
  __shared__ __attribute__((aligned(512))) char sW[NT][kQ * RV];
  __shared__ __attribute__((aligned(512))) char sY[OT][kQ * RV];
  __shared__ __attribute__((aligned(512))) char sK[TILES ? kQ * RK : 16];
  __shared__ __attribute__((aligned(512))) char sQ[TILES && BACK ? kQ * RK : 16];
  __shared__ __attribute__((aligned(512))) char sN1[kT * NT * kOne];
  __shared__ __attribute__((aligned(512))) char sN2[kT * OT * kOne];
  __shared__ __attribute__((aligned(16))) float vec[kVecs * 64];
  __shared__ float sSum[NW][kQ], sDot[2][kQ], sAll[BACK ? 1 : kMostEvery * kQ];

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
  const elem* vg = static_cast<const elem*>(p.v) + b * p.vs[0] + (h / p.vdiv) * p.vs[2];
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

  // ---- a chunk's rows, 8 columns at a time by the threads in turn, in registers on their way to LDS
  constexpr int kV8 = VD / 8, kN = kQ * kV8 / THREADS, kK8 = KD / 8, kNK = kQ * kK8 / THREADS;
  struct Rows {
    F8 w[kN], y[kN];
    piece d[kN], v[BACK ? 1 : kN], k[TILES ? kNK : 1], q[TILES && BACK ? kNK : 1];
    float vec[(kVecs * 64 + THREADS - 1) / THREADS];
  } in;
  auto ask = [&](int c) __attribute__((always_inline)) {
    const int n = least(len - c * kQ, kQ);
    const int64_t t0 = static_cast<int64_t>(c) * kQ, rows = (bh * nchunks + c) * kQ;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = tid + i * THREADS, row = at / kV8, slot = at % kV8, left = row < n ? V - 8 * slot : 0;
      load_piece(reinterpret_cast<const char*>(p.w + (rows + row) * VD + 8 * slot), in.w[i]);
      load_piece(reinterpret_cast<const char*>(p.y + (rows + row) * VD + 8 * slot), in.y[i]);
      in.d[i] = load8<ACT>(dg, (t0 + row) * p.ds[1] + 8 * slot, left, p.d_vec);
      if constexpr (!BACK) in.v[i] = load8<ACT>(vg, (t0 + row) * p.vs[1] + 8 * slot, left, p.v_vec);
    }
    if constexpr (TILES) {
#pragma unroll
      for (int i = 0; i < kNK; ++i) {
        const int at = tid + i * THREADS, row = at / kK8, slot = at % kK8, left = row < n ? K - 8 * slot : 0;
        in.k[i] = load8<ACT>(kg, (t0 + row) * p.ks[1] + 8 * slot, left, p.k_vec);
        if constexpr (BACK) in.q[i] = load8<ACT>(qg, (t0 + row) * p.qs[1] + 8 * slot, left, p.q_vec);
      }
    }
    const float* from = reinterpret_cast<const float*>(p.rec + (bh * nchunks + c) * kRecord<ACT, 0> + kTBytes<ACT>);
#pragma unroll
    for (int i = 0; i < (kVecs * 64 + THREADS - 1) / THREADS; ++i) in.vec[i] = from[least(tid + i * THREADS, kVecs * 64 - 1)];
  };
  auto store = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = tid + i * THREADS, row = at / kV8, slot = at % kV8;
      float x[8], y[8];
      Op<ActF32>::unpack(in.w[i], x);
      Op<ActF32>::unpack(in.y[i], y);
      piece t[NT], o[OT];
      O::template split<NT>(x, t);
      O::template split<OT>(y, o);
#pragma unroll
      for (int m = 0; m < NT; ++m) put8<RV, PW>(sW[m], row, slot, t[m]);
#pragma unroll
      for (int m = 0; m < OT; ++m) put8<RV, PY>(sY[m], row, slot, o[m]);
      put8<RV, BACK>(sD, row, slot, in.d[i]);
      if constexpr (!BACK) {                        // y.w and y.v
        float v[8], yw = 0.0f, yv = 0.0f;
        O::unpack(in.v[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          yw = __builtin_fmaf(y[e], x[e], yw);
          yv = __builtin_fmaf(y[e], v[e], yv);
        }
#pragma unroll
        for (int d = 1; d < kV8; d *= 2) {
          yw += __shfl_xor(yw, d);
          yv += __shfl_xor(yv, d);
        }
        if (slot == 0) {
          sDot[0][row] = yw;
          sDot[1][row] = yv;
        }
      }
    }
    if constexpr (TILES) {
#pragma unroll
      for (int i = 0; i < kNK; ++i) {
        const int at = tid + i * THREADS, row = at / kK8, slot = at % kK8;
        put8<RK, false>(sK, row, slot, in.k[i]);
        if constexpr (BACK) put8<RK, false>(sQ, row, slot, in.q[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < (kVecs * 64 + THREADS - 1) / THREADS; ++i)
      if (tid + i * THREADS < kVecs * 64) vec[tid + i * THREADS] = in.vec[i];
  };
  auto chunk_of = [&](int done) { return BACK ? c_end - 1 - done : c_begin + done; };
  ask(chunk_of(0));

  // E[y][u][e] is the entry v = 32 y + 8 g + 4 u + e, k = 16 w + c16 (backwards of the gradient F)
  const int col = 16 * w + c16;
  f32x4_t E[KT][2];
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int y = 0; y < KT; ++y)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = 32 * y + 8 * g + 4 * u + e;
          f(y, u, e, col < K && v < V, static_cast<uint32_t>(col * V + v));
        }
  };
  {
    const float* src = (BACK ? p.kept_f : p.kept_e) + (bh * stretches + s) * static_cast<int64_t>(K) * V;
    each([&](int y, int u, int e, bool there, uint32_t at) { E[y][u][e] = there ? src[at] : 0.0f; });
  }
  const uint32_t tile_d = lds_address(sD), tile_w = lds_address(sW[0]), tile_y = lds_address(sY[0]);
  const int perm_row = 8 * (c16 >> 2) + (c16 & 3);
  const uint32_t d_rows = O::template row_part<RV, BACK>(tile_d, BACK ? perm_row : c16, g);
  const uint32_t w_rows = O::template row_part<RV, PW>(tile_w, BACK ? c16 : perm_row, g);
  const uint32_t y_rows = O::template row_part<RV, PY>(tile_y, BACK ? perm_row : c16, g);
  // rows 16 jt + c16, or of the permuted tile (t, u), of term m
  auto natural = [&](uint32_t rows, int jt, int y, int m) __attribute__((always_inline)) {
    return O::row(rows + jt * (16 * RV), 4 * PB * y, m * (kQ * RV));
  };
  auto permuted = [&](uint32_t rows, int t, int u, int y, int m) __attribute__((always_inline)) {
    return O::row(rows + t * (32 * RV), (4 * PB * y) ^ (u ? swizzle<RV, kF32, true>(4) << 4 : 0), 4 * u * RV + m * (kQ * RV));
  };
  auto eight = [&](int which, int t, float (&x)[8]) __attribute__((always_inline)) {
    const float4 a = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g);
    const float4 d = *reinterpret_cast<const float4*>(vec + which * 64 + 32 * t + 8 * g + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = d.x; x[5] = d.y; x[6] = d.z; x[7] = d.w;
  };
  const f32x4_t zero = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll 1
  for (int done = 0; done < c_end - c_begin; ++done) {
    const int c = chunk_of(done);
    const int n = least(len - c * kQ, kQ);
    const int64_t t0 = static_cast<int64_t>(c) * kQ;
    store();
    __syncthreads();
    if (done + 1 < c_end - c_begin) ask(chunk_of(done + 1));
    // the wave's own columns of k (and of q): tokens 32 t + 8 g + e of column c16
    piece kf[2], qf[2];
    if constexpr (TILES) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        kf[t] = O::template column<RK, false>(O::template column_part<RK, false>(lds_address(sK), 16 * w, 4, lane), 0, 32 * t * RK);
        if constexpr (BACK)
          qf[t] = O::template column<RK, false>(O::template column_part<RK, false>(lds_address(sQ), 16 * w, 4, lane), 0, 32 * t * RK);
      }
    } else {
      auto columns = [&](const elem* base, int64_t stride, piece (&out)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          elem x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = 32 * t + 8 * g + e;
            const elem y = base[(t0 + least(row, n - 1)) * stride + least(col, K - 1)];
            x[e] = row < n && col < K ? y : elem(0);
          }
          out[t] = __builtin_bit_cast(piece, x);
        }
      };
      columns(kg, p.ks[1], kf);
      if constexpr (BACK) columns(qg, p.qs[1], qf);
    }

    // ---- N1 and N2 in operand order, 16 rows by 32 tokens an operand.  Forwards as the scores: column j = 16 jt + c16, tokens
    // i = 32 t + 8 g + e.  Backwards column i, tokens j; i in the first half takes both halves of j, i in the second the
    // second.
#pragma unroll 1
    for (int x = w; x < kT; x += NW) {
      const int jt = x < 4 ? x : BACK ? x - 4 : x - 2, t = BACK ? (x < 4 ? 1 : 0) : (x < 4 ? 0 : 1);
      f32x4_t a1[2] = {zero, zero}, a2[2] = {zero, zero};
#pragma unroll
      for (int y = 0; y < KT; ++y) {
        piece wr[2][NT], yr[2][OT], dr[2];          // (of the permuted rows two tiles, of the others one)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (BACK) {
            dr[u] = permuted(d_rows, t, u, y, 0);
#pragma unroll
            for (int m = 0; m < OT; ++m) yr[u][m] = permuted(y_rows, t, u, y, m);
          } else {
#pragma unroll
            for (int m = 0; m < NT; ++m) wr[u][m] = permuted(w_rows, t, u, y, m);
          }
        }
        if (BACK) {
#pragma unroll
          for (int m = 0; m < NT; ++m) wr[0][m] = natural(w_rows, jt, y, m);
        } else {
          dr[0] = natural(d_rows, jt, y, 0);
#pragma unroll
          for (int m = 0; m < OT; ++m) yr[0][m] = natural(y_rows, jt, y, m);
        }
#pragma unroll
        for (int m = NT - 1; m >= 0; --m) {
#pragma unroll
          for (int u = 0; u < 2; ++u) a1[u] = BACK ? O::mma(dr[u], wr[0][m], a1[u]) : O::mma(wr[u][m], dr[0], a1[u]);
#pragma unroll
          for (int o = OT - 1 - m; o >= 0; --o)
#pragma unroll
            for (int u = 0; u < 2; ++u) a2[u] = BACK ? O::mma(yr[u][o], wr[0][m], a2[u]) : O::mma(wr[u][m], yr[0][o], a2[u]);
        }
      }
      const int cc = 16 * jt + c16;                 // forwards j, backwards i
      float hi[8], lo[8], beta[8], v1[8], v2[8];
      eight(kSumHi, t, hi);
      eight(kSumLo, t, lo);
      eight(kBeta, t, beta);
      const float chi = vec[kSumHi * 64 + cc], clo = vec[kSumLo * 64 + cc], cbeta = vec[kBeta * 64 + cc];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 32 * t + 8 * g + e;
        const float m = BACK ? exp2_pair(hi[e] - chi, lo[e] - clo) : exp2_pair(chi - hi[e], clo - lo[e]);
        const float mi = m * (BACK ? cbeta : beta[e]), mj = BACK ? beta[e] : cbeta;     // beta of u_i, of y_j
        v1[e] = (BACK ? row >= cc : row <= cc) ? a1[e / 4][e % 4] * (p.scale * mi) : 0.0f;
        v2[e] = (BACK ? row > cc : row < cc) ? a2[e / 4][e % 4] * -(mj * mi) : 0.0f;
      }
      piece o1[NT], o2[OT];
      O::template split<NT>(v1, o1);
      O::template split<OT>(v2, o2);
#pragma unroll
      for (int m = 0; m < NT; ++m) store_piece(sN1 + (x * NT + m) * kOne + lane * (kOne / 64), o1[m]);
#pragma unroll
      for (int m = 0; m < OT; ++m) store_piece(sN2 + (x * OT + m) * kOne + lane * (kOne / 64), o2[m]);
    }

    // ---- the state's part, rows k, column j = 16 jt + c16: acc of D and acy of Y, backwards acc of W
    f32x4_t acc[4], acy[4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) acc[jt] = acy[jt] = zero;
#pragma unroll
    for (int y = 0; y < KT; ++y) {
      piece ef[NT];
      const float x[8] = {E[y][0][0], E[y][0][1], E[y][0][2], E[y][0][3], E[y][1][0], E[y][1][1], E[y][1][2], E[y][1][3]};
      O::template split<NT>(x, ef);
      if constexpr (BACK) {
#pragma unroll
        for (int m = NT - 1; m >= 0; --m) {
          piece r[4];
#pragma unroll
          for (int jt = 0; jt < 4; ++jt) r[jt] = natural(w_rows, jt, y, m);
#pragma unroll
          for (int o = NT - 1 - m; o >= 0; --o)
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) acc[jt] = O::mma(ef[o], r[jt], acc[jt]);
        }
      } else {
        piece d[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) d[jt] = natural(d_rows, jt, y, 0);
#pragma unroll
        for (int m = NT - 1; m >= 0; --m)
#pragma unroll
          for (int jt = 0; jt < 4; ++jt) acc[jt] = O::mma(ef[m], d[jt], acc[jt]);
#pragma unroll
        for (int m = OT - 1; m >= 0; --m) {
          piece r[4];
#pragma unroll
          for (int jt = 0; jt < 4; ++jt) r[jt] = natural(y_rows, jt, y, m);
#pragma unroll
          for (int o = OT - 1 - m; o >= 0; --o)
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) acy[jt] = O::mma(ef[o], r[jt], acy[jt]);
        }
      }
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const float beta = vec[kBeta * 64 + 16 * jt + c16], into = vec[kInto * 64 + 16 * jt + c16];
      const float f = BACK ? vec[kLast * 64 + 16 * jt + c16] * beta : p.scale * into;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[jt][e] *= f;
        if constexpr (!BACK) acy[jt][e] *= -(beta * into);
      }
    }
    // (q's values that meet dq, on their way)
    float q_in[4][4];
    if constexpr (!BACK) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const int64_t at = (t0 + least(16 * jt + c16, n - 1)) * p.qs[1];
        const int first = 16 * w + 4 * g;
        if (p.q_four) {
          if constexpr (kF32) {
            const float4 y = *reinterpret_cast<const float4*>(qg + at + least(first, K - 4));
            q_in[jt][0] = y.x; q_in[jt][1] = y.y; q_in[jt][2] = y.z; q_in[jt][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(qg + at + least(first, K - 4));
            q_in[jt][0] = bf16_lo(y.x); q_in[jt][1] = bf16_hi(y.x); q_in[jt][2] = bf16_lo(y.y); q_in[jt][3] = bf16_hi(y.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) q_in[jt][e] = load_act<ACT>(qg, at + least(first + e, K - 1));
        }
      }
    }
    __syncthreads();                                // N1 and N2 are complete

    // ---- the chunk's own part
#pragma unroll
    for (int m = NT - 1; m >= 0; --m)
#pragma unroll
      for (int x = 0; x < kT; ++x) {
        const int jt = x < 4 ? x : BACK ? x - 4 : x - 2, t = BACK ? (x < 4 ? 1 : 0) : (x < 4 ? 0 : 1);
        piece n1;
        load_piece(sN1 + (x * NT + m) * kOne + lane * (kOne / 64), n1);
        acc[jt] = O::mma(BACK ? qf[t] : kf[t], n1, acc[jt]);
        if (m < OT) {
          piece n2;
          load_piece(sN2 + (x * OT + m) * kOne + lane * (kOne / 64), n2);
          if constexpr (BACK) acc[jt] = O::mma(kf[t], n2, acc[jt]);
          else acy[jt] = O::mma(kf[t], n2, acy[jt]);
        }
      }

    // ---- out: lane (g, c) has columns 16 w + 4 g .. of token 16 jt + c
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const int row = 16 * jt + c16, first = 16 * w + 4 * g;
      const int64_t at = out_base + (t0 + row) * out_row + first;
      if (row < n) {
        if (p.part_vec) {
          if (first < K) {
            const f32x4_t& x = acc[jt];
            float4 y = make_float4(x[0], x[1], x[2], x[3]);
            if constexpr (BACK) {
              const float4 z = *reinterpret_cast<const float4*>(p.dk_part + at);
              y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
              if (p.dk_f32) *reinterpret_cast<float4*>(p.dk_part + at) = y;
              else if constexpr (kF32) *reinterpret_cast<float4*>(static_cast<float*>(p.dk) + at) = y;
              else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dk) + at) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
            } else {
              if (p.dq_f32 || kF32) *reinterpret_cast<float4*>(static_cast<float*>(p.dq) + at) = y;
              else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dq) + at) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
              const f32x4_t& z = acy[jt];
              *reinterpret_cast<float4*>(p.dk_part + at) = make_float4(z[0], z[1], z[2], z[3]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (first + e >= K) continue;
            if constexpr (BACK) {
              const float y = p.dk_part[at + e] + acc[jt][e];
              if (p.dk_f32) p.dk_part[at + e] = y;
              else store_act<ACT>(p.dk, at + e, y);
            } else {
              if (p.dq_f32) static_cast<float*>(p.dq)[at + e] = acc[jt][e];
              else store_act<ACT>(p.dq, at + e, acc[jt][e]);
              p.dk_part[at + e] = acy[jt][e];
            }
          }
        }
      }
      if constexpr (!BACK) {                        // q.dq (its columns past K are zeros of k's)
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = first + e < K ? __builtin_fmaf(q_in[jt][e], acc[jt][e], sum) : sum;
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (g == 0) sSum[w][row] = sum;
      }
    }

    // ---- the state
    if (done + 1 < c_end - c_begin || !BACK) {      // (backwards the last is of no use)
      const float whole = vec[kWhole * 64];
      each([&](int y, int u, int e, bool, uint32_t) { E[y][u][e] *= whole; });
      const uint32_t w_cols = O::template column_part<RV, PW>(tile_w, 0, 8, lane);
      const uint32_t y_cols = O::template column_part<RV, PY>(tile_y, 0, 8, lane);
      const uint32_t d_cols = O::template column_part<RV, BACK>(tile_d, 0, 8, lane);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float with[8], beta[8], x[8];
        eight(BACK ? kInto : kLast, t, with);
        eight(kBeta, t, beta);
        piece k_in[NT], d_in[NT];
        O::unpack(kf[t], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= BACK ? -(with[e] * beta[e]) : with[e] * beta[e];
        O::template split<NT>(x, k_in);
        if constexpr (BACK) {
          O::unpack(qf[t], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= with[e] * p.scale;
          O::template split<NT>(x, d_in);
        }
#pragma unroll
        for (int z = 0; z < KT; z += 2) {           // four tiles at a time
          auto columns = [&](uint32_t cols, auto perm, int m, piece (&out)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              out[i] = O::template column<RV, decltype(perm)::value>(cols, (4 * PB * (z + i / 2)) ^ O::half_flip(i % 2),
                                                                     32 * t * RV + O::half_offset(i % 2) + m * (kQ * RV));
          };
#pragma unroll
          for (int m = NT - 1; m >= 0; --m) {
            piece left[4];
            if constexpr (BACK) columns(y_cols, std::integral_constant<bool, PY>{}, m, left);
            else columns(w_cols, std::integral_constant<bool, PW>{}, m, left);
#pragma unroll
            for (int o = NT - 1 - m; o >= 0; --o)
#pragma unroll
              for (int i = 0; i < 4; ++i) E[z + i / 2][i % 2] = O::mma(left[i], k_in[o], E[z + i / 2][i % 2]);
          }
          if constexpr (BACK) {
            piece left[4];
            columns(d_cols, std::integral_constant<bool, BACK>{}, 0, left);
#pragma unroll
            for (int o = NT - 1; o >= 0; --o)
#pragma unroll
              for (int i = 0; i < 4; ++i) E[z + i / 2][i % 2] = O::mma(left[i], d_in[o], E[z + i / 2][i % 2]);
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
        sAll[done * kQ + tid] = __builtin_fmaf(-vec[kBeta * 64 + tid], sDot[1][tid], sum);
        p.dbeta[(b * L + t0 + tid) * p.H + h] = sDot[0][tid];
      }
      __syncthreads();                              // (before the next chunk's vectors and sums)
    }
  }

  if constexpr (!BACK) {
    // <F, E> at the end of the stretch, then the sums back over its tokens
    const float* f = p.kept_f + (bh * stretches + s) * static_cast<int64_t>(K) * V;
    float dot = 0.0f;
    each([&](int y, int u, int e, bool there, uint32_t at) {
      if (there) dot = __builtin_fmaf(f[at], E[y][u][e], dot);
    });
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
