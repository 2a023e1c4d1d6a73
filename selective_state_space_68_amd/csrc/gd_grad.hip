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
// g: dg_t is what passes token t, from tokens and states before it to tokens and states from it on; each part carries a_t.
// In a chunk of slow decays it is a sum over later tokens: a_t scales everything that passes, so with r_j = exp(G_j) the
// state's scale, S / r, r q and v / r carry all of it: d loss / d G_j = q_j.dq_j - v_j.dv_j, and dg_t is its sum over j >= t in
// the stretch, in float64, onto <F, E> at its end.  Both dots hold what token j has of itself, which a fast decay leaves
// dg_t far below: at g = -5 the float32 terms' roundings were 1e-3 of dg, at -12 all of it.  So in a chunk with a decay below
// 2^kFastGate = 0.42 the parts are summed, none of which a token has of itself:
//     dg_t = exp(G_Q) <F, E> + sum_{j>=t} from_j + sum_{i<t<=j} (N1_ji q_j.k_i + N2_ji k_j.k_i) + sum_{i<t} to_i,
//     from_j = q_j.(scale exp(G_j) E d_j) + k_j.(-beta_j exp(G_j) E y_j),   to_i = k_i.(exp(G_Q - G_i) F u_i),
// with E before the chunk and F behind it; from_j and the sum over pairs come with dq, to_i with the rest of dk.  <F, E> takes both
// states at once: the first kernel leaves E in memory for the second, where exp(G_Q) is not too small to be seen and
// either a decay is below 1/8 or F is the caller's; else the chunk counts as slow.  Errors of dg against its own size at g = -1 to
// -20 and at single decays of exp(-3) to exp(-30) in slow heads: below 1e-5; a decay of 0 has 0.  The two kernels of the case
// below, whose heads range from slow to fast, took 793 us with sums over later tokens alone and take 839 (float32, 2 x 2047, 24
// heads of 64: 190 and 223).
//
// A workgroup walks one stretch; a wave owns 16 columns of E^T (of K), so that only the tokens' scalars are summed over
// waves.  Rows of D, W and Y lie in LDS, W and Y as terms, split once a workgroup; their dot products y.w and y.v are
// taken on the way in.  A chunk's rows are asked for while the one before is worked on.
//
// What bounds it: 8 x 2048 tokens, 32 heads of 128, bfloat16: 492 us and 347, 3.2 and 4.1 TB/s (1.6 and 1.4 GB: W and Y as float32 rows are
// half of it) with the matrix units busy for a third of the time: its one workgroup a CU (155 and 145 KB of LDS) reads, multiplies and
// meets at three barriers a chunk.
//
// Roundings (bfloat16 activations): what g's float32 gradient sees of dq, with the states that it is formed from, comes from
// 24-bit operands; what dk's bfloat16 sees, and g through k in chunks of fast decays, from 16 bits (y and F u: 2^-17 an operand).
#include <type_traits>

#include "device_common.hpp"
#include "gd_common.hpp"
#include "la_tiles.hpp"
#include "lm_kernels.hpp"
#include "row_sum.hpp"
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
  // of chunks with fast decays: what passes tokens from one of the chunk to another, by operand, and from the first half into
  // tokens of the second; products of the two states
  __shared__ __attribute__((aligned(16))) float sPass[BACK ? 1 : 2][kT][32];
  __shared__ float sOver[BACK ? 1 : 2][32], sThrough[2][NW];

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
  auto chunk_of = [&](int done) { return BACK ? c_end - 1 - done : c_begin + done; };
  auto suffix = [&](auto x) __attribute__((always_inline)) {          // the sum over this lane and those after it
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const auto after = __shfl_down(x, d);
      if (lane + d < 64) x += after;
    }
    return x;
  };
  // A chunk's tokens (one wave, when they are complete).  The first kernel: dbeta, and in dg's place its part of what passes
  // a token, or the terms that the sum over later tokens is of.
  auto scalars = [&](int done, int pace) __attribute__((always_inline)) {
    const int which = done & 1, c = chunk_of(done), t = c * kQ + lane;
    const bool on = t < len;
    const int64_t at = (b * L + (on ? t : len - 1)) * p.H + h;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) sum += sSum[which][i][lane];
    if (pace == kSlow) {
      sum = __builtin_fmaf(-sDot[which][2][lane], sDot[which][1][lane], sum);
    } else {
      const float (&pass)[kT][32] = sPass[BACK ? 0 : which];
      sum = suffix(on ? sum : 0.0f);
      if (lane == 0) reinterpret_cast<float*>(p.rec + (bh * nchunks + c) * kRecord<ACT, 0> + kTBytes<ACT>)[kPace * 64 + 1] = sum;
      const float over = suffix(lane >= 32 && on ? sOver[BACK ? 0 : which][lane & 31] : 0.0f);
      sum += lane < 32 ? (pass[0][lane] + pass[1][lane]) + (pass[2][lane] + pass[3][lane])
                       : (pass[4][lane & 31] + pass[5][lane & 31]) + over;
    }
    if (on) {
      p.dg[at] = sum;
      p.dbeta[at] = sDot[which][0][lane];
    }
  };
  // The second kernel: dg.  carry: what passes from the tokens before this chunk's end to those behind it.
  double carry = 0.0;
  float gate_whole = 0.0f, gate_into = 0.0f, gate_part = 0.0f;        // exp(G_Q), the sum of from_j, the first kernel's part of dg
  auto gate_at = [&](int done, int lane) { return p.dg + (b * L + least(chunk_of(done) * kQ + lane, len - 1)) * p.H + h; };
  auto gates = [&](int done, int pace) __attribute__((always_inline)) {
    const int which = done & 1, t = chunk_of(done) * kQ + lane;
    const bool on = t < len;
    float x = gate_part;
    if (pace == kSlow) {
      const double sum = suffix(on ? static_cast<double>(x) : 0.0) + carry;
      carry = __shfl(sum, 0);
      x = static_cast<float>(sum);
    } else {
      float out = 0.0f, through = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        out += sSum[which][i][lane];
        if (pace == kFastThrough) through += sThrough[which][i];
      }
      if (!on) out = 0.0f;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const float before = __shfl_up(out, d);
        if (lane >= d) out += before;
      }
      const float before = __shfl_up(out, 1);       // of the tokens before this one
      if (lane > 0) x += before;
      through *= gate_whole;
      x += through;
      carry = static_cast<double>(through) + gate_into;
    }
    // (the first token of a sequence without a state has nothing to scale)
    if (on) *gate_at(done, lane) = t == 0 && !p.carried ? 0.0f : x;
  };
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

  int pace = kSlow;
#pragma unroll 1
  for (int done = 0; done < c_end - c_begin; ++done) {
    const int c = chunk_of(done);
    const int n = least(len - c * kQ, kQ);
    const int64_t t0 = static_cast<int64_t>(c) * kQ;
    store(n, done & 1);
    __syncthreads();
    if (done > 0 && w == NW - 1) {                  // (the last waves have no part in N1 and N2)
      if constexpr (BACK) gates(done - 1, pace);
      else scalars(done - 1, pace);
    }
    pace = uniform_int(static_cast<int>(vec[kPace * 64]));
    if constexpr (BACK) {
      gate_whole = vec[kWhole * 64];
      gate_into = vec[kPace * 64 + 1];
      gate_part = *gate_at(done, w == NW - 1 ? lane : 0);
      if (done == 0) carry = vec[kPace * 64 + 2];
    }
    // the state before a chunk, as the first kernel's threads have it
    float4* before = reinterpret_cast<float4*>(p.through + (bh * nchunks + c) * (KD * VD)) + tid;
    if constexpr (BACK) {
      if (pace == kFastThrough) {
        float dot = 0.0f;
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float4 x = before[(2 * y + u) * THREADS];
            const f32x4_t& f = E[y][u];
            dot = __builtin_fmaf(x.x, f[0], __builtin_fmaf(x.y, f[1], __builtin_fmaf(x.z, f[2], __builtin_fmaf(x.w, f[3], dot))));
          }
        dot = wave_sum(dot);
        if (lane == 0) sThrough[done & 1][w] = dot;
      }
    }
    // (rows 16 jt + c16 of q for what passes through the chunk's tokens)
    constexpr int kOps = (kT + NW - 1) / NW;
    piece qn[TILES && !BACK ? kOps : 1][KD / 32];
    if constexpr (TILES && !BACK) {
#pragma unroll
      for (int o = 0; o < kOps; ++o) {
        const int x = w + o * NW, row = 16 * (x < 4 ? x : x - 2) + c16;
        const bool wanted = pace != kSlow && x < kT;
#pragma unroll
        for (int y = 0; y < KD / 32; ++y)
          qn[o][y] = load8<ACT, MOVE>(qg + t0 * p.qs[1], static_cast<Offset<MOVE>>(p.qs[1]), wanted ? row : 0, n, wanted ? 32 * y + 8 * g : 0, K);
      }
    }
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
    if (TILES || BACK) ask(next, 0, more);
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
      if constexpr (!BACK) {
        if (pace != kSlow) {
          // what token j has of token i through the chunk: N1_ji q_j.k_i + N2_ji k_j.k_i, for i < j
          f32x4_t b1[2] = {zero, zero}, b2[2] = {zero, zero};
          if constexpr (TILES) {
            const uint32_t tile_k = lds_address(sK);
            const uint32_t kn = O::template row_part<RK, false>(tile_k, cc, g);
            const uint32_t kp = O::template row_part<RK, false>(tile_k, 32 * t + perm_row, g);
#pragma unroll
            for (int y = 0; y < KD / 32; ++y) {
              const piece qj = present<ACT, MOVE>(kOps > 1 && x >= NW ? qn[kOps - 1][y] : qn[0][y], cc, n, 32 * y + 8 * g, K);
              const piece kj = O::row(kn, 4 * PB * y, 0);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const piece ki = O::row(kp, (4 * PB * y) ^ (u ? swizzle<RK, kF32, false>(4) << 4 : 0), 4 * u * RK);
                b1[u] = O::mma(ki, qj, b1[u]);
                b2[u] = O::mma(ki, kj, b2[u]);
              }
            }
          } else {
            const elem *qc = qg + t0 * p.qs[1], *kc = kg + t0 * p.ks[1];
#pragma unroll 1
            for (int y = 0; y < KD / 32; ++y) {
              auto eight_of = [&](const elem* base, int64_t stride, int row) __attribute__((always_inline)) {
                const int at = 32 * y + 8 * g;
                return present<ACT, MOVE>(load8<ACT, MOVE>(base, static_cast<Offset<MOVE>>(stride), row, n, at, K), row, n, at, K);
              };
              const piece qj = eight_of(qc, p.qs[1], cc), kj = eight_of(kc, p.ks[1], cc);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const piece ki = eight_of(kc, p.ks[1], 32 * t + 4 * u + perm_row);
                b1[u] = O::mma(ki, qj, b1[u]);
                b2[u] = O::mma(ki, kj, b2[u]);
              }
            }
          }
          // summed over i before a token and j from it on: over the lane's tokens i, those of the lanes before, the columns
          float before[8], sum = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            before[e] = sum;
            const float x = __builtin_fmaf(v1[e], b1[e / 4][e % 4], v2[e] * b2[e / 4][e % 4]);
            sum += 32 * t + 8 * g + e < cc ? x : 0.0f;
          }
#pragma unroll
          for (int d = 16; d < 64; d *= 2) {
            const float x = __shfl_up(sum, d);
            if (lane >= d) sum += x;
          }
          const float lanes = __shfl_up(sum, 16);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = 32 * t + 8 * g + e <= cc ? before[e] + (g > 0 ? lanes : 0.0f) : 0.0f;
            before[e] = row_sum<16>(x);
          }
          float* to = sPass[done & 1][x] + 8 * g;
          if (c16 == 0) {
            *reinterpret_cast<float4*>(to) = make_float4(before[0], before[1], before[2], before[3]);
            *reinterpret_cast<float4*>(to + 4) = make_float4(before[4], before[5], before[6], before[7]);
          }
          if (g == 3 && (x == 2 || x == 3)) sOver[done & 1][cc - 32] = sum;
        }
      }
      piece o1[NT], o2[OT];
      O::template split<NT>(v1, o1);
      O::template split<OT>(v2, o2);
#pragma unroll
      for (int m = 0; m < NT; ++m) store_piece(sN1 + (x * NT + m) * kOne + lane * (kOne / 64), o1[m]);
#pragma unroll
      for (int m = 0; m < OT; ++m) store_piece(sN2 + (x * OT + m) * kOne + lane * (kOne / 64), o2[m]);
    }

    if (!TILES && !BACK) ask(next, 0, more);        // (N's loads would wait for these)
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
    if (pace != kSlow) {
      // what passes into a token from before the chunk, q.dq and k.dk of the state's parts; backwards out of the chunk from it
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const int row = 16 * jt + c16;
        float kx[4], sum = 0.0f;
        if constexpr (TILES) {
          const uint2 x = *reinterpret_cast<const uint2*>(sK + row * RK + ((2 * first) ^ (swizzle<RK, false, false>(row) << 4)));
          kx[0] = bf16_lo(x.x); kx[1] = bf16_hi(x.x); kx[2] = bf16_lo(x.y); kx[3] = bf16_hi(x.y);
        } else {
          const elem* from = kg + (t0 + least(row, n - 1)) * p.ks[1];
          if constexpr (VEC) {
            const float4 x = *reinterpret_cast<const float4*>(from + least(first, K - 4));
            kx[0] = x.x; kx[1] = x.y; kx[2] = x.z; kx[3] = x.w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) kx[e] = load_act<ACT>(from, least(first + e, K - 1));
          }
        }
        if constexpr (BACK) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = first + e < K ? __builtin_fmaf(kx[e], acc[jt][e], sum) : sum;
        } else {
          float qx[4] = {meet[jt][0], meet[jt][1], meet[jt][2], meet[jt][3]};
          if constexpr (VEC && !kF32) {
            const uint32_t a = __builtin_bit_cast(uint32_t, qx[0]), d = __builtin_bit_cast(uint32_t, qx[1]);
            qx[0] = bf16_lo(a); qx[1] = bf16_hi(a); qx[2] = bf16_lo(d); qx[3] = bf16_hi(d);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sum = first + e < K ? __builtin_fmaf(qx[e], acc[jt][e], __builtin_fmaf(kx[e], acy[jt][e], sum)) : sum;
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (g == 0) sSum[done & 1][w][row] = sum;
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
    if (!BACK && pace == kSlow) {                   // q.dq
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
      if constexpr (!BACK) {
        if (pace == kFastThrough) {
#pragma unroll
          for (int y = 0; y < KT; ++y)
#pragma unroll
            for (int u = 0; u < 2; ++u) before[(2 * y + u) * THREADS] = make_float4(E[y][u][0], E[y][u][1], E[y][u][2], E[y][u][3]);
        }
      }
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

  if constexpr (BACK) {
    if (w == NW - 1) gates(c_end - c_begin - 1, pace);
  } else {
    if (w == NW - 1) scalars(c_end - c_begin - 1, pace);
    // <F, E> at the end of the stretch
    const float* f = p.kept_f + (bh * stretches + s) * static_cast<int64_t>(K) * V;
    float dot = 0.0f;
    each([&](int y, int u, int e, bool there, uint32_t at) {
      if (there) dot = __builtin_fmaf(f[at], E[y][u][e], dot);
    });
    dot = wave_sum(dot);
    if (lane == 0) sThrough[0][w] = dot;
    __syncthreads();
    if (tid == 0) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) sum += sThrough[0][i];
      reinterpret_cast<float*>(p.rec + (bh * nchunks + c_end - 1) * kRecord<ACT, 0> + kTBytes<ACT>)[kPace * 64 + 2] = sum;
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
// stretches and against one chunk a stretch: bfloat16, heads of 128: 8 x 2048, 32 heads 1436, 1477, 2423; 2 x 2048, 32 heads 571, 688, 831; 3 x 1777, 17
// heads 478, 547, 661; float32, 4 x 2048, 24 heads of 128 1950, 2151, 2238; of 64 945, 988, 964.
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
