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
// One workgroup of 4 waves walks the chunks of one (batch row, head, segment).  Wave w owns
// columns v in [16 VT w, 16 VT (w + 1)) of E and of the output, so E is used as a matrix
// operand straight from the registers that accumulate it: a product leaves lane (g, c) of a
// 16 x 16 tile four consecutive rows of column c, and since the order of a product's
// summation index is free, the rows of each tile are assigned (kperm below) so that the
// two tiles of a pair leave a lane 8 consecutive indices: what one operand needs.  q, k and
// v go through LDS row by row; operands that sum over tokens (k^T, v^T) come out of the same
// rows by transposing LDS reads.  P goes through LDS (each wave forms 16 rows of it).  The
// next chunk's rows are loaded into registers while the current chunk computes.
//
// Roundings (bfloat16 activations; float32 activations use float32 products throughout):
// the decayed v of the state update is split into three bfloat16 terms, which carry all 24
// bits, since the state is a float32 result; E and P as operands of the output are split
// into two terms (16 bits), so that the output's own rounding is the one that counts.
//
// When the (batch row, head) pairs are too few to fill the chip the sequence is cut into
// segments: a pre-pass forms each segment's own state sum, a small kernel chains them, and
// the main pass runs every segment from its entering E.
#include "device_common.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kQ = 64;               // tokens per chunk
constexpr float kMinLog2 = -1.0e4f;  // 2^kMinLog2 == 0 and kMinLog2 * 0 == 0: a decay of exactly 0 works like any other

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// ---- eight values of one lane: a matrix operand (one v_mfma_f32_16x16x32_bf16, lane
// (g, c) holding row/column c and summation indices 8g..8g+7; or eight
// v_mfma_f32_16x16x4_f32, lane group g holding index g of each)
template <typename ACT>
struct Op;

template <>
struct Op<ActBF16> {
  using elem = uint16_t;
  using piece = uint4;
  static constexpr int kPad = 8;     // elements of row padding in LDS (16 bytes)
  static __device__ __forceinline__ f32x4_t mma(const piece& a, const piece& b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
  }
  static __device__ __forceinline__ piece zero() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ piece pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ void unpack(const piece& p, float (&v)[8]) {
    v[0] = bf16_lo(p.x); v[1] = bf16_hi(p.x); v[2] = bf16_lo(p.y); v[3] = bf16_hi(p.y);
    v[4] = bf16_lo(p.z); v[5] = bf16_hi(p.z); v[6] = bf16_lo(p.w); v[7] = bf16_hi(p.w);
  }
  // v = sum of TERMS operands, each the rounding of what the ones before it left
  template <int TERMS>
  static __device__ __forceinline__ void split(const float (&v)[8], piece (&p)[TERMS]) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      p[t] = pack(r);
      if (t + 1 < TERMS) {
        float q[8];
        unpack(p[t], q);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] -= q[e];
      }
    }
  }
  // Values [row0 + 8g + e][col(c)], e = 0..7, of a row-major LDS tile, col(c) = col0 + step (c / 4) + c % 4:
  // two transposing reads of 4 rows each.  Lane i of a 16-lane group gives the address
  // of 4 columns (piece i % 4) of row i / 4 and receives column i of the 4 rows.
  static __device__ __forceinline__ piece column(const elem* tile, int stride, int row0, int col0, int step, int lane) {
    const int g = lane >> 4, i = lane & 15;
    const elem* a = tile + (row0 + 8 * g + (i >> 2)) * stride + col0 + step * (i & 3);
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(a));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(a + 4 * stride));
    const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
    return make_uint4(l.x, l.y, h.x, h.y);
  }
};

struct F8 {
  float4 a, b;
};

template <>
struct Op<ActF32> {
  using elem = float;
  using piece = F8;
  static constexpr int kPad = 4;
  static __device__ __forceinline__ f32x4_t mma(const piece& a, const piece& b, f32x4_t c) {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.x, b.a.x, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.y, b.a.y, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.z, b.a.z, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.w, b.a.w, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.x, b.b.x, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.y, b.b.y, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.z, b.b.z, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.w, b.b.w, c, 0, 0, 0);
  }
  static __device__ __forceinline__ piece zero() {
    return F8{make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  }
  static __device__ __forceinline__ piece pack(const float (&v)[8]) {
    return F8{make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
  }
  static __device__ __forceinline__ void unpack(const piece& p, float (&v)[8]) {
    v[0] = p.a.x; v[1] = p.a.y; v[2] = p.a.z; v[3] = p.a.w;
    v[4] = p.b.x; v[5] = p.b.y; v[6] = p.b.z; v[7] = p.b.w;
  }
  template <int TERMS>
  static __device__ __forceinline__ void split(const float (&v)[8], piece (&p)[TERMS]) {
    static_assert(TERMS == 1, "float32 operands are exact");
    p[0] = pack(v);
  }
  static __device__ __forceinline__ piece column(const elem* tile, int stride, int row0, int col0, int step, int lane) {
    const int g = lane >> 4, c = lane & 15;
    const elem* a = tile + (row0 + 8 * g) * stride + col0 + step * (c >> 2) + (c & 3);
    return F8{make_float4(a[0], a[stride], a[2 * stride], a[3 * stride]),
              make_float4(a[4 * stride], a[5 * stride], a[6 * stride], a[7 * stride])};
  }
};

// log2(lam) of a head, kept finite at the bottom (NaN passes through).
__device__ __forceinline__ float decay_log2(const float* log_decay, int h) {
  const float g = log_decay[h] * kLog2e;
  return g < kMinLog2 ? kMinLog2 : g;
}

// lam^n as a float32 pair hi + lo.  A state passes through thousands of these products, so
// the rounding of lam^n alone would grow to n_chunks * 2^-24 over the head's memory.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair decay_pair(const float* log_decay, int h, int n) {
  double x = static_cast<double>(log_decay[h]) * n;
  if (n == 0) x = 0.0;
  const double d = exp(x);
  const float hi = static_cast<float>(d);
  const float lo = static_cast<float>(d - static_cast<double>(hi));
  return Pair{hi, lo == lo ? lo : 0.0f};              // (inf - inf where lam^n overflows)
}

__device__ __forceinline__ int row_length(const LaArgs& p, int64_t b) {
  const int L = static_cast<int>(p.L);
  if (!p.lengths) return L;
  const int n = p.lengths[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

// A tile row's 8 elements starting at column col of a row of `cols` elements (zeros past it).
template <typename ACT>
__device__ __forceinline__ typename Op<ACT>::piece load_piece(const typename Op<ACT>::elem* row, int col, int cols,
                                                              int vec) {
  using P = typename Op<ACT>::piece;
  if (vec) {
    const int c = col < cols ? col : cols - 8;        // (a whole vector: cols is a multiple of 8)
    P r = *reinterpret_cast<const P*>(row + c);
    return col < cols ? r : Op<ACT>::zero();
  }
  typename Op<ACT>::elem e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? row[col + i] : typename Op<ACT>::elem(0);
  return *reinterpret_cast<const P*>(e);
}

// STATE_ONLY: the pre-pass, which leaves each segment's own sum (its state after its last
// token, from zero) in role.seg.  Otherwise the whole of the segment's output.
template <typename ACT, int KD, int VT, bool STATE_ONLY>
__global__ __launch_bounds__(256) void la_kernel(LaArgs p) {
  using O = Op<ACT>;
  using elem = typename O::elem;
  using piece = typename O::piece;
  constexpr bool kF32 = sizeof(elem) == 4;
  constexpr int VD = 64 * VT;
  constexpr int RK = KD + O::kPad, RV = VD + O::kPad, RS = kQ + O::kPad;
  constexpr int KT = KD / 32;                       // pairs of state tiles along K
  constexpr int NK = KD / 32, NV = VD / 32;         // 8-element pieces per thread of a k (q) and v tile
  constexpr int WT = kF32 ? 1 : 3;                  // operand terms of the decayed v
  constexpr int ET = kF32 ? 1 : 2;                  // operand terms of E and of P
  __shared__ __attribute__((aligned(16))) elem sQ[STATE_ONLY ? 16 : kQ * RK];
  __shared__ __attribute__((aligned(16))) elem sK[kQ * RK];
  __shared__ __attribute__((aligned(16))) elem sV[kQ * RV];
  __shared__ __attribute__((aligned(16))) elem sP[ET][STATE_ONLY ? 16 : kQ * RS];   // P [j][i]

  const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6);
  const int g = lane >> 4, c16 = lane & 15;
  const LaRole& r = p.role[blockIdx.y];
  const int nseg = p.nseg;
  const int64_t bh = blockIdx.x / nseg;
  const int seg = static_cast<int>(blockIdx.x % nseg);
  const int64_t b = bh / p.H;
  const int h = static_cast<int>(bh % p.H);
  const int L = static_cast<int>(p.L);
  const int len = row_length(p, b);
  const int K = r.K, V = r.V, vec = r.vec, reverse = r.reverse;
  const int nchunks = (L + kQ - 1) / kQ;
  const int live = (len + kQ - 1) / kQ;             // chunks that hold a token
  const int c_begin = seg * static_cast<int>(p.seg_chunks);
  const int c_stop = c_begin + static_cast<int>(p.seg_chunks);
  const int c_end = c_stop < nchunks ? c_stop : nchunks;
  const int c_live = c_end < live ? c_end : live;
  const float g2 = decay_log2(p.log_decay, h);
  const Pair dQ = decay_pair(p.log_decay, h, kQ);

  // row r of the sequence is token r forwards, len - 1 - r backwards
  const int64_t t_first = reverse ? len - 1 : 0;
  const int t_step = reverse ? -1 : 1;
  const elem* qg = static_cast<const elem*>(r.q) + b * r.qs[0] + (h / r.qdiv) * r.qs[2] + t_first * r.qs[1];
  const elem* kg = static_cast<const elem*>(r.k) + b * r.ks[0] + (h / r.kdiv) * r.ks[2] + t_first * r.ks[1];
  const elem* vg = static_cast<const elem*>(r.v) + b * r.vs[0] + (h / r.vdiv) * r.vs[2] + t_first * r.vs[1];
  const int64_t qstep = r.qs[1] * t_step, kstep = r.ks[1] * t_step, vstep = r.vs[1] * t_step;

  // E[vt][t][u][e] is the entry k = 32 t + 8 g + 4 u + e, v = 16 (VT w + vt) + c16
  f32x4_t E[VT][KT][2];
  const float* src = nullptr;
  if (!STATE_ONLY) {
    if (nseg > 1) src = r.seg + (bh * nseg + seg) * static_cast<int64_t>(K) * V;
    else if (r.carry) src = r.carry + bh * static_cast<int64_t>(K) * V;
  }
  // forwards the carried state decays once before the first token; the segments' states have
  const float lam1 = exp2_hw(g2);
  const bool decayed = nseg > 1 || reverse || len == 0;
#pragma unroll
  for (int vt = 0; vt < VT; ++vt)
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kk = 32 * t + 8 * g + 4 * u + e, vv = 16 * (VT * w + vt) + c16;
          float x = 0.0f;
          if (src && kk < K && vv < V) {
            x = src[static_cast<int64_t>(kk) * r.sk + static_cast<int64_t>(vv) * r.sv];
            if (!decayed) x *= lam1;
          }
          E[vt][t][u][e] = x;
        }

  piece rq[STATE_ONLY ? 1 : NK], rk[NK], rv[NV];
  // The rows of chunk c into registers; rows past its n tokens reload its last one (zeroed on the way to LDS).
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int r0 = c * kQ;
    const int lim = len - 1 - r0 < kQ - 1 ? len - 1 - r0 : kQ - 1;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int v = tid + 256 * i, row = v / (KD / 8), col = v % (KD / 8) * 8;
      const int64_t t = r0 + (row < lim ? row : lim);
      rk[i] = load_piece<ACT>(kg + t * kstep, col, K, vec);
      if constexpr (!STATE_ONLY) rq[i] = load_piece<ACT>(qg + t * qstep, col, K, vec);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + 256 * i, row = v / (VD / 8), col = v % (VD / 8) * 8;
      const int64_t t = r0 + (row < lim ? row : lim);
      rv[i] = load_piece<ACT>(vg + t * vstep, col, V, vec);
    }
  };
  auto stage = [&](int n) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int v = tid + 256 * i, row = v / (KD / 8), col = v % (KD / 8) * 8;
      *reinterpret_cast<piece*>(&sK[row * RK + col]) = row < n ? rk[i] : O::zero();
      if constexpr (!STATE_ONLY) *reinterpret_cast<piece*>(&sQ[row * RK + col]) = row < n ? rq[i] : O::zero();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + 256 * i, row = v / (VD / 8), col = v % (VD / 8) * 8;
      *reinterpret_cast<piece*>(&sV[row * RV + col]) = row < n ? rv[i] : O::zero();
    }
  };

  if (c_begin < c_live) fetch(c_begin);
  for (int c = c_begin; c < c_live; ++c) {
    const int n = len - c * kQ < kQ ? len - c * kQ : kQ;
    // the last chunk of the sequence (of the segment, in the pre-pass) forwards leaves S, not lam S
    const int shift = (STATE_ONLY || !reverse) && c + 1 == c_live && (STATE_ONLY || c_live == live) ? 1 : 0;
    stage(n);
    if (c + 1 < c_live) fetch(c + 1);
    barrier_lds();

    // ---- P rows j = 16 w + c16: tiles of k q^T, rows i = 32 t + 8 g + 4 u + e
    if constexpr (!STATE_ONLY) {
      const int j = 16 * w + c16;
      piece qf[KT];
#pragma unroll
      for (int x = 0; x < KT; ++x) qf[x] = *reinterpret_cast<const piece*>(&sQ[j * RK + 32 * x + 8 * g]);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float pv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pv[e] = 0.0f;
        if (t == 0 || w >= 2) {                     // the block right of the diagonal is zero
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
            const int krow = 32 * t + 8 * (c16 >> 2) + 4 * u + (c16 & 3);
#pragma unroll
            for (int x = 0; x < KT; ++x)
              s = O::mma(*reinterpret_cast<const piece*>(&sK[krow * RK + 32 * x + 8 * g]), qf[x], s);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int off = j - (32 * t + 8 * g + 4 * u + e);
              const float d = exp2_hw(g2 * static_cast<float>(off > 0 ? off : 0)) * (r.in_scale * r.out_scale);
              pv[4 * u + e] = off >= 0 ? s[e] * d : 0.0f;
            }
          }
        }
        piece ps[ET];
        O::template split<ET>(pv, ps);
#pragma unroll
        for (int m = 0; m < ET; ++m) *reinterpret_cast<piece*>(&sP[m][j * RS + 32 * t + 8 * g]) = ps[m];
      }
    }

    // ---- the wave's own columns of v: as they are (for P v) and decayed (for the state)
    piece vf[VT][2];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < 2; ++t) vf[vt][t] = O::column(sV, RV, 32 * t, 16 * (VT * w + vt), 4, lane);

    // ---- output from the carried state, transposed: acc[vt][jt] = rows v, column j = 16 jt + c16
    f32x4_t acc[VT][4];
    if constexpr (!STATE_ONLY) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) acc[vt][jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        piece ef[VT][ET];
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          const float x[8] = {E[vt][t][0][0], E[vt][t][0][1], E[vt][t][0][2], E[vt][t][0][3],
                              E[vt][t][1][0], E[vt][t][1][1], E[vt][t][1][2], E[vt][t][1][3]};
          O::template split<ET>(x, ef[vt]);
        }
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
          const piece q = *reinterpret_cast<const piece*>(&sQ[(16 * jt + c16) * RK + 32 * t + 8 * g]);
#pragma unroll
          for (int vt = 0; vt < VT; ++vt)
#pragma unroll
            for (int m = 0; m < ET; ++m) acc[vt][jt] = O::mma(ef[vt][m], q, acc[vt][jt]);
        }
      }
    }

    // ---- the state: E = lam^n E + k^T (lam^(n-i) v)
    Pair dn = dQ;
    if (n - shift != kQ) dn = decay_pair(p.log_decay, h, n - shift);
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) E[vt][t][u][e] = __builtin_fmaf(dn.hi, E[vt][t][u][e], dn.lo * E[vt][t][u][e]);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float wgt[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int left = n - shift - (32 * t + 8 * g + e);
        wgt[e] = exp2_hw(g2 * static_cast<float>(left > 0 ? left : 0)) * r.in_scale;
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
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const piece kf = O::column(sK, RK, 32 * t, 32 * kt + 4 * u, 8, lane);
#pragma unroll
          for (int vt = 0; vt < VT; ++vt)
#pragma unroll
            for (int m = 0; m < WT; ++m) E[vt][kt][u] = O::mma(kf, wv[vt][m], E[vt][kt][u]);
        }
    }
    barrier_lds();                                  // P complete; the tiles are free

    // ---- P v, transposed, on top; the output rows to memory
    if constexpr (!STATE_ONLY) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const int j = 16 * jt + c16;
        const float f = exp2_hw(g2 * static_cast<float>(j)) * r.out_scale;
        piece pf[2][ET];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int m = 0; m < ET; ++m)
            if (t == 0 || jt >= 2) pf[t][m] = *reinterpret_cast<const piece*>(&sP[m][j * RS + 32 * t + 8 * g]);
        const int64_t row = static_cast<int64_t>(c) * kQ + j;
        const int64_t token = reverse ? (row < len ? len - 1 - row : row) : row;
        const int64_t o0 = ((b * L + token) * p.H + h) * V;
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          f32x4_t a = acc[vt][jt];
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] *= f;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int m = 0; m < ET; ++m)
              if (t == 0 || jt >= 2) a = O::mma(vf[vt][t], pf[t][m], a);
          if (j >= n) a = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          const int v0 = 16 * (VT * w + vt) + 4 * g;
          if (row < L) {
            if (r.o_f32 || kF32) {
              float* o = static_cast<float*>(r.o) + o0 + v0;
              if (vec) {
                if (v0 < V) *reinterpret_cast<float4*>(o) = make_float4(a[0], a[1], a[2], a[3]);
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (v0 + e < V) o[e] = a[e];
              }
            } else {
              uint16_t* o = static_cast<uint16_t*>(r.o) + o0 + v0;
              if (vec) {
                if (v0 < V) *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (v0 + e < V) o[e] = to_bf16(a[e]);
              }
            }
          }
        }
      }
    }
  }

  // chunks with no token: zeros
  if constexpr (!STATE_ONLY) {
    for (int64_t c = c_live > c_begin ? c_live : c_begin; c < c_end; ++c) {
      for (int i = tid; i < kQ * V; i += 256) {
        const int64_t token = c * kQ + i / V;
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
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kk = 32 * t + 8 * g + 4 * u + e, vv = 16 * (VT * w + vt) + c16;
            if (kk < K && vv < V) dst[static_cast<int64_t>(kk) * r.sk + static_cast<int64_t>(vv) * r.sv] = E[vt][t][u][e];
          }
  }
}

// Chains the segments' own sums T_s into the E entering each segment (written over T_s) and
// the state after the last token.  One thread per state entry.
__global__ __launch_bounds__(256) void la_chain_kernel(LaArgs p) {
  const LaRole& r = p.role[0];
  const int64_t bh = blockIdx.y;
  const int KV = r.K * r.V;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= KV) return;
  const int h = static_cast<int>(bh % p.H);
  const int len = row_length(p, bh / p.H);
  const int seg_tokens = static_cast<int>(p.seg_chunks) * kQ;
  const Pair l1 = decay_pair(p.log_decay, h, 1), lS = decay_pair(p.log_decay, h, seg_tokens);
  float* slot = r.seg + bh * p.nseg * static_cast<int64_t>(KV) + i;
  float s = r.carry ? r.carry[bh * static_cast<int64_t>(KV) + i] : 0.0f;
  auto times = [](const Pair& d, float x) { return __builtin_fmaf(d.hi, x, d.lo * x); };
  for (int k = 0; k < p.nseg; ++k, slot += KV) {
    const int left = len - k * seg_tokens, n = left < 0 ? 0 : (left < seg_tokens ? left : seg_tokens);
    const float T = *slot;
    *slot = r.reverse ? s : times(l1, s);
    if (n == 0) continue;
    const Pair d = n == seg_tokens ? lS : decay_pair(p.log_decay, h, n);
    s = times(d, s) + (r.reverse ? times(l1, T) : T);
  }
  if (r.fin) r.fin[bh * static_cast<int64_t>(KV) + i] = s;
}

template <typename ACT>
__global__ __launch_bounds__(256) void la_sum_heads_kernel(const float* part, void* out, int64_t total, int64_t share,
                                                           int64_t d) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step) {   // [token][head][d]
    const float* src = part + i / d * share * d + i % d;
    float s = 0.0f;
    for (int64_t x = 0; x < share; ++x) s += src[x * d];
    store_act<ACT>(out, i, s);
  }
}

__global__ __launch_bounds__(256) void la_copy_state_kernel(float* dst, const float* src, int64_t n) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) dst[i] = src ? src[i] : 0.0f;
}

template <typename ACT, int KD, int VT>
void launch_la_t(const LaArgs& a, bool state_only, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.batch * a.H * a.nseg), static_cast<unsigned>(a.nroles));
  if (state_only) hipLaunchKernelGGL((la_kernel<ACT, KD, VT, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((la_kernel<ACT, KD, VT, false>), grid, dim3(256), 0, s, a);
}

template <typename ACT>
void launch_la_act(const LaArgs& a, bool state_only, hipStream_t s) {
  const bool k2 = a.role[0].K > 64, v2 = a.role[0].V > 64;
  if (k2 && v2) launch_la_t<ACT, 128, 2>(a, state_only, s);
  else if (k2) launch_la_t<ACT, 128, 1>(a, state_only, s);
  else if (v2) launch_la_t<ACT, 64, 2>(a, state_only, s);
  else launch_la_t<ACT, 64, 1>(a, state_only, s);
}

}  // namespace

int la_segments(int64_t batch, int64_t L, int64_t H, int64_t K, int64_t V) {
  (void)batch; (void)L; (void)H; (void)K; (void)V;
  return 1;
}

// The roles of one call, each launched by itself (their tile shapes differ where K != V).
hipError_t launch_la(const LaArgs& a, Dt dt, hipStream_t s) {
  const int64_t nchunks = (a.L + kQ - 1) / kQ;
  for (int pass = a.nseg > 1 ? 0 : 1; pass < 2; ++pass) {
    for (int i = 0; i < a.nroles; ++i) {
      LaArgs one = a;
      one.role[0] = a.role[i];
      one.nroles = 1;
      one.seg_chunks = (nchunks + a.nseg - 1) / a.nseg;
      // (the roles of dk and dv share one set of segment states: role 2's)
      if (pass == 0 && i == 1) continue;
      if (dt == Dt::BF16) launch_la_act<ActBF16>(one, pass == 0, s);
      else launch_la_act<ActF32>(one, pass == 0, s);
      if (pass == 0) {
        const dim3 grid(static_cast<unsigned>((one.role[0].K * one.role[0].V + 255) / 256),
                        static_cast<unsigned>(a.batch * a.H), 1);
        hipLaunchKernelGGL(la_chain_kernel, grid, dim3(256), 0, s, one);
      }
    }
  }
  return hipGetLastError();
}

hipError_t launch_la_sum_heads(const float* part, void* out, int64_t tokens, int64_t heads, int64_t share, int64_t d,
                               Dt dt, hipStream_t s) {
  const int64_t total = tokens * heads * d, blocks = (total + 255) / 256;
  const dim3 grid(static_cast<unsigned>(blocks < 8192 ? blocks : 8192));
  if (dt == Dt::BF16) hipLaunchKernelGGL(la_sum_heads_kernel<ActBF16>, grid, dim3(256), 0, s, part, out, total, share, d);
  else hipLaunchKernelGGL(la_sum_heads_kernel<ActF32>, grid, dim3(256), 0, s, part, out, total, share, d);
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
