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
// What bounds it: 8 x 2048 tokens, 32 heads of 128, bfloat16: 456 us and 328, 3.5 and 4.2 TB/s (1.6 and 1.4 GB: W and Y as float32 rows are
// half of it) with the matrix units busy for a third of the time: its one workgroup a CU (142 KB of LDS) reads, multiplies and meets at
// three barriers a chunk.
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

// Eight values of a row from memory, MOVE bytes being the unit in which rows move (16, 4, or 0: element by element).  Nothing is decided
// where they move as vectors or words: rows and columns that are not there repeat the last ones (they are cleared on the way into LDS).
template <int MOVE>
using Offset = std::conditional_t<MOVE == 16, uint32_t, int64_t>;    // within a chunk's rows (vectors': of fewer than 2^32 bytes)
template <typename ACT, int MOVE>
__device__ __forceinline__ typename Op<ACT>::piece load8(const void* base, Offset<MOVE> stride, int row, int n, int col, int width) {
  using elem = typename Op<ACT>::elem;
  const elem* at = static_cast<const elem*>(base);
  const Offset<MOVE> first = static_cast<Offset<MOVE>>(least(row, n - 1)) * stride;
  typename Op<ACT>::piece p;
  if constexpr (MOVE == 16) {
    load_piece(reinterpret_cast<const char*>(at + (first + least(col, width - 8))), p);
  } else if constexpr (MOVE == 4) {
    load_words(reinterpret_cast<const char*>(at + (first + least(col, width - 8))), p);
  } else {
    elem v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = at[first + least(col + e, width - 1)];
    p = __builtin_bit_cast(typename Op<ACT>::piece, v);
  }
  return p;
}
// The values of columns and rows that are there.
template <typename ACT, int MOVE>
__device__ __forceinline__ typename Op<ACT>::piece present(typename Op<ACT>::piece p, int row, int n, int col, int width) {
  using elem = typename Op<ACT>::elem;
  if constexpr (MOVE == 4)
    if (width % 8) drop_first(p, least(col - least(col, width - 8), 7));
  if constexpr (MOVE != 0) {
    return row < n && col < width ? p : Op<ACT>::zero();
  } else {
    struct Eight { elem v[8]; } x = __builtin_bit_cast(Eight, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x.v[e] = row < n && col + e < width ? x.v[e] : elem(0);
    return __builtin_bit_cast(typename Op<ACT>::piece, x);
  }
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

// BACK: the second kernel, which adds the backward part of dk.  MOVE: the unit in which rows of q, k, v and d move; with 16, those of dq
// and dk move as 4 elements.
template <typename ACT, int KD, int VD, int MOVE, bool BACK>
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
  constexpr bool VEC = MOVE == 16;
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
  // the tokens' scalars, of this chunk and of the one before: parts of q.dq, y.w and y.v, beta
  __shared__ float sSum[2][NW][kQ], sDot[2][3][kQ];

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
      if (BACK ? p.dk_f32 : p.dq_f32) static_cast<float*>(BACK ? p.dk : p.dq)[at] = 0.0f;
      else store_act<ACT>(BACK ? p.dk : p.dq, at, 0.0f);
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
  constexpr int kVecRegs = (kVecs * 64 + THREADS - 1) / THREADS;
  struct Rows {
    F8 w[kN], y[kN];
    piece d[kN], v[BACK ? 1 : kN], k[TILES ? kNK : 1], q[TILES && BACK ? kNK : 1];
    float vec[kVecRegs];
  } in;
  // in four parts, 0 to 3, spread over the chunk before: asked for at once, they keep the loads' unit busy for thousands of
  // cycles while the waves wait for their turn
  auto ask = [&](int c, int part, bool wanted) __attribute__((always_inline)) {
    int id = wanted ? tid : 0;
    asm volatile("" : "+v"(id));                    // (so that no address is kept over the loop)
    const int n = least(len - c * kQ, kQ);
    const int64_t t0 = static_cast<int64_t>(c) * kQ, rows = (bh * nchunks + c) * kQ;
    const char *wc = reinterpret_cast<const char*>(p.w + rows * VD), *yc = reinterpret_cast<const char*>(p.y + rows * VD);
    const elem *dc = dg + t0 * p.ds[1], *vc = vg + t0 * p.vs[1], *kc = kg + t0 * p.ks[1], *qc = qg + t0 * p.qs[1];
    const Offset<MOVE> dstep = static_cast<Offset<MOVE>>(p.ds[1]), vstep = static_cast<Offset<MOVE>>(p.vs[1]),
                      kstep = static_cast<Offset<MOVE>>(p.ks[1]), qstep = static_cast<Offset<MOVE>>(p.qs[1]);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = id + i * THREADS, row = at / kV8, col = 8 * (at % kV8);
      if (part == 0) load_piece(wc + static_cast<uint32_t>(32 * at), in.w[i]);
      if (part == 1) load_piece(yc + static_cast<uint32_t>(32 * at), in.y[i]);
      if (part == 2) {
        in.d[i] = load8<ACT, MOVE>(dc, dstep, row, n, col, V);
        if constexpr (!BACK) in.v[i] = load8<ACT, MOVE>(vc, vstep, row, n, col, V);
      }
    }
    if (part < 3) return;
    if constexpr (TILES) {
#pragma unroll
      for (int i = 0; i < kNK; ++i) {
        const int at = id + i * THREADS, row = at / kK8, col = 8 * (at % kK8);
        in.k[i] = load8<ACT, MOVE>(kc, kstep, row, n, col, K);
        if constexpr (BACK) in.q[i] = load8<ACT, MOVE>(qc, qstep, row, n, col, K);
      }
    }
    const float* from = reinterpret_cast<const float*>(p.rec + (bh * nchunks + c) * kRecord<ACT, 0> + kTBytes<ACT>);
#pragma unroll
    for (int i = 0; i < kVecRegs; ++i) in.vec[i] = from[static_cast<uint32_t>(least(id + i * THREADS, kVecs * 64 - 1))];
  };
  auto store = [&](int n, int which) __attribute__((always_inline)) {
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
      put8<RV, BACK>(sD, row, slot, present<ACT, MOVE>(in.d[i], row, n, 8 * slot, V));
      if constexpr (!BACK) {                        // y.w and y.v
        float v[8], yw = 0.0f, yv = 0.0f;
        O::unpack(present<ACT, MOVE>(in.v[i], row, n, 8 * slot, V), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          yw = __builtin_fmaf(y[e], x[e], yw);
          yv = __builtin_fmaf(y[e], v[e], yv);
        }
        yw = row_sum<kV8>(yw);
        yv = row_sum<kV8>(yv);
        if (slot == 0) {
          sDot[which][0][row] = yw;
          sDot[which][1][row] = yv;
        }
      }
    }
    if constexpr (TILES) {
#pragma unroll
      for (int i = 0; i < kNK; ++i) {
        const int at = tid + i * THREADS, row = at / kK8, slot = at % kK8;
        put8<RK, false>(sK, row, slot, present<ACT, MOVE>(in.k[i], row, n, 8 * slot, K));
        if constexpr (BACK) put8<RK, false>(sQ, row, slot, present<ACT, MOVE>(in.q[i], row, n, 8 * slot, K));
      }
    }
#pragma unroll
    for (int i = 0; i < kVecRegs; ++i)
      if (tid + i * THREADS < kVecs * 64) {
        vec[tid + i * THREADS] = in.vec[i];
        if (!BACK && (tid + i * THREADS) / 64 == kBeta) sDot[which][2][tid % 64] = in.vec[i];
      }
  };
  // A chunk's tokens (one wave, when they are complete): dbeta, and in dg's place what the sums at the end are of.
  auto scalars = [&](int done) __attribute__((always_inline)) {
    const int which = done & 1, t = (c_begin + done) * kQ + lane;
    if (t >= len) return;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) sum += sSum[which][i][lane];
    const int64_t at = (b * L + t) * p.H + h;
    p.dg[at] = __builtin_fmaf(-sDot[which][2][lane], sDot[which][1][lane], sum);
    p.dbeta[at] = sDot[which][0][lane];
  };
  auto chunk_of = [&](int done) { return BACK ? c_end - 1 - done : c_begin + done; };
#pragma unroll
  for (int part = 0; part < 4; ++part) ask(chunk_of(0), part, true);

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
    store(n, done & 1);
    __syncthreads();
    if (!BACK && done > 0 && w == NW - 1) scalars(done - 1);      // (the last waves have no part in N1 and N2)
    // what meets dq and dk at the end (asked for before the next chunk's rows, which its arrival need not wait for)
    const int first = 16 * w + 4 * g;               // this lane's columns of token 16 jt + c16 there
    const uint32_t out_step = static_cast<uint32_t>(out_row);
    const int64_t out_at = out_base + t0 * out_row;
    float* part = p.dk_part + ((bh * nchunks + c) * NW + w) * 1024 + lane * 4;
    float meet[4][4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const uint32_t row = static_cast<uint32_t>(least(16 * jt + c16, n - 1));
      if constexpr (BACK) {                         // (dk's forward part, as this lane of the first kernel left it)
        const float4 x = *reinterpret_cast<const float4*>(part + jt * 256);
        meet[jt][0] = x.x; meet[jt][1] = x.y; meet[jt][2] = x.z; meet[jt][3] = x.w;
      } else {                                      // (q)
        const elem* from = qg + t0 * p.qs[1];
        const Offset<MOVE> at = row * static_cast<Offset<MOVE>>(p.qs[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) meet[jt][e] = 0.0f;
        if constexpr (VEC && kF32) {
          const float4 x = *reinterpret_cast<const float4*>(from + (at + least(first, K - 4)));
          meet[jt][0] = x.x; meet[jt][1] = x.y; meet[jt][2] = x.z; meet[jt][3] = x.w;
        } else if constexpr (VEC) {                 // (unpacked where it is used)
          const float2 x = *reinterpret_cast<const float2*>(from + (at + least(first, K - 4)));
          meet[jt][0] = x.x; meet[jt][1] = x.y;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) meet[jt][e] = load_act<ACT>(from, at + least(first + e, K - 1));
        }
      }
    }
    const bool more = done + 1 < c_end - c_begin;
    // (the last chunk asks for one place: after a load on one side of a branch every wait is for all loads)
    const int next = chunk_of(more ? done + 1 : done);
    ask(next, 0, more);
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

    ask(next, 1, more);
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
    ask(next, 2, more);
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
    if constexpr (!BACK) {                          // q.dq
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if constexpr (VEC && !kF32) {
          const uint32_t a = __builtin_bit_cast(uint32_t, meet[jt][0]), d = __builtin_bit_cast(uint32_t, meet[jt][1]);
          meet[jt][0] = bf16_lo(a); meet[jt][1] = bf16_hi(a); meet[jt][2] = bf16_lo(d); meet[jt][3] = bf16_hi(d);
        }
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = first + e < K ? __builtin_fmaf(meet[jt][e], acc[jt][e], sum) : sum;
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (g == 0) sSum[done & 1][w][16 * jt + c16] = sum;
      }
    }
    auto put = [&](auto* out, int jt, const float (&x)[4]) __attribute__((always_inline)) {
      using OUT = std::remove_pointer_t<decltype(out)>;
      const uint32_t at = static_cast<uint32_t>(16 * jt + c16) * out_step + first;
      if constexpr (VEC) {
        if constexpr (sizeof(OUT) == 4) *reinterpret_cast<float4*>(out + at) = make_float4(x[0], x[1], x[2], x[3]);
        else *reinterpret_cast<uint2*>(out + at) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (first + e >= K) continue;
          if constexpr (sizeof(OUT) == 4) out[at + e] = x[e];
          else out[at + e] = to_bf16(x[e]);
        }
      }
    };
    auto put_act = [&](void* out, bool f32, int jt, const float (&x)[4]) __attribute__((always_inline)) {
      if (f32 || kF32) put(static_cast<float*>(out) + out_at, jt, x);
      else put(static_cast<uint16_t*>(out) + out_at, jt, x);
    };
    if (first < K) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (16 * jt + c16 >= n) continue;
        float x[4] = {acc[jt][0], acc[jt][1], acc[jt][2], acc[jt][3]};
        if constexpr (BACK) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] += meet[jt][e];
          put_act(p.dk, p.dk_f32, jt, x);
        } else {
          put_act(p.dq, p.dq_f32, jt, x);
        }
      }
    }
    if constexpr (!BACK) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt)
        *reinterpret_cast<float4*>(part + jt * 256) = make_float4(acy[jt][0], acy[jt][1], acy[jt][2], acy[jt][3]);
    }

    ask(next, 3, more);
    // ---- the state
    if (more || !BACK) {      // (backwards the last is of no use)
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
  }

  if constexpr (!BACK) {
    if (w == NW - 1) scalars(c_end - c_begin - 1);
    // <F, E> at the end of the stretch, then the sums back over its tokens
    const float* f = p.kept_f + (bh * stretches + s) * static_cast<int64_t>(K) * V;
    float dot = 0.0f;
    each([&](int y, int u, int e, bool there, uint32_t at) {
      if (there) dot = __builtin_fmaf(f[at], E[y][u][e], dot);
    });
    dot = wave_sum(dot);
    __syncthreads();                                // (the sums have been read, the tokens' parts are in memory)
    if (lane == 0) sSum[0][w][0] = dot;
    __syncthreads();
    if (w == 0) {
      double carry = 0.0;
#pragma unroll
      for (int i = 0; i < NW; ++i) carry += sSum[0][i][0];
      const int stop = least(len, c_end * kQ);
      for (int c = c_end - 1; c >= c_begin; --c) {
        const int t = c * kQ + lane;
        float* at = p.dg + (b * L + least(t, stop - 1)) * p.H + h;
        double x = t < stop ? static_cast<double>(*at) : 0.0;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const double after = __shfl_down(x, d);
          if (lane + d < 64) x += after;
        }
        x += carry;
        carry = __shfl(x, 0);
        // (the first token of a sequence without a state has nothing to scale)
        if (t < stop) *at = t == 0 && !p.carried ? 0.0f : static_cast<float>(x);
      }
    }
  }
}

template <typename ACT, int KD, int VD>
void launch_qk_t(const GdGradArgs& a, hipStream_t s) {
  const int64_t nch = (a.L + kQ - 1) / kQ, stretches = (nch + a.every - 1) / a.every;
  const dim3 grid(static_cast<unsigned>(a.batch * a.H * stretches)), block(4 * KD);
  auto go = [&](auto move) {
    constexpr int MOVE = decltype(move)::value;
    hipLaunchKernelGGL((gd_qk_kernel<ACT, KD, VD, MOVE, false>), grid, block, 0, s, a);
    hipLaunchKernelGGL((gd_qk_kernel<ACT, KD, VD, MOVE, true>), grid, block, 0, s, a);
  };
  if (a.move == 16) go(std::integral_constant<int, 16>{});
  else if (a.move == 4 && a.K >= 8 && a.V >= 8) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 0>{});
}

}  // namespace

// Chunks between two kept states.  A workgroup of gd_qk_kernel has a CU to itself (the smallest two share one), and a stretch costs its chunks and about as
// much as kStart more for its start (its states, its first rows): the least of that over the chip's rounds.  us, against a fixed 1024
// stretches and against one chunk a stretch: bfloat16, heads of 128: 8 x 2048, 32 heads 1380, 1436, 2369; 2 x 2048, 32 heads 571, 692, 837; 3 x 1777, 17
// heads 476, 650; float32, 4 x 2048, 24 heads of 128 1850, 2040, 2162; of 64 860, 1011, 1011.
int gd_every(int64_t batch, int64_t L, int64_t H, int64_t K, int64_t V, Dt dt) {
  const int64_t places = dt == Dt::F32 && K <= 64 && V <= 64 ? 512 : 256;
  constexpr double kStart = 1.5;
  const int64_t pairs = batch * H, nch = (L + kQ - 1) / kQ;
  int best = 1;
  double least_cost = 0.0;
  for (int e = 1; e <= kMostEvery; ++e) {
    const int64_t rounds = (pairs * ((nch + e - 1) / e) + places - 1) / places;
    const double cost = static_cast<double>(rounds) * (e + kStart);
    if (e > 1 && cost >= least_cost) continue;
    best = e;
    least_cost = cost;
  }
  return best;
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
