// The norms around a block fused with its gate, residual and residual scale, and their
// gradient.  Row by row over D columns (each piece may be absent):
//     n = post_weight * x * r1,  r1 = rsqrt(mean over the column's group of x^2 + eps)
//     t = n * silu(gate),   h = residual + res_scale * t,
//     y = pre_weight * h * r2,   r2 = rsqrt(mean over the row of h^2 + eps)
// and backwards, with dy and the gradient dh that reaches h from elsewhere,
//     dH = dh + r2 (a - h r2^2 mean(a h)),  a = dy pre_weight;   dresidual = dH
//     dt = dH res_scale,  dn = dt silu(gate),  dgate = dt n silu'(gate)
//     dx = r1 (c - x r1^2 mean over the group of (c x)),  c = dn post_weight
//     dpre_weight = sum over rows of dy h r2,  dpost_weight = sum of dn x r1,
//     dres_scale = sum of dH t.
// (In rows of one column x^2 r1^2 = 1 - eps r1^2, so dx = r1 c eps r1^2: the difference above
// would leave only its rounding.  The same holds for dH.)
//
// A few flops per value: bound by HBM, so every value is read and written once.  A team of
// threads (whole waves, the fewest that cover a row at NV vectors of 8 columns a thread)
// holds a row in registers between the sums and the results, and walks rows a grid apart:
// its columns stay the same, so the weights stay in registers and, backwards, so do the column sums of
// the weights' gradients, which leave once per workgroup; a second kernel adds the workgroups'
// in a fixed order.  The next row is asked for before the current one is computed, past the caches
// (streaming loads and stores: 6.1 TB/s where three tensors are read and one is written, 4.9 without).
//
// Measured: 8192 x 5120 bfloat16 with 80 groups and gate 49 us (5.1 TB/s); the gradient of 16384 x 4096 bfloat16 with
// gate, scale and float32 residual, 32 groups, 314 us (4.7 TB/s; 5.4 is what a copy reaches); 256 x 2560, 6 us: a
// launch, the rows and two sums over them.
#include "device_common.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kTeams = 4;            // rows per workgroup where a row is one wave's

// Column of element e of vector v of thread t.  Blocked: 8 consecutive columns a vector.
// Strided (one group, rows that do not move as vectors): consecutive threads, consecutive columns.
template <bool STRIDED>
__device__ __forceinline__ int col_of(int t, int T, int v, int e) {
  return STRIDED ? (v * 8 + e) * T + t : (v * T + t) * 8 + e;
}

// A row's values of one thread as they lie in memory: packed pairs (bfloat16) or floats.
template <typename ACT, int NV>
struct Row {
  static constexpr int kWords = ACT::kBytes == 2 ? 4 : 8;
  uint32_t w[NV][kWords];
};

template <typename ACT, int NV, bool STRIDED>
__device__ __forceinline__ void load_row(Row<ACT, NV>& r, const void* base, int64_t row0, int D, int t, int T, int vec) {
  using E = typename ACT::storage;
  const E* p = static_cast<const E*>(base) + row0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c0 = (v * T + t) * 8;
    if (!STRIDED && vec) {
      if (c0 < D) {
        const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p + c0);
#pragma unroll
        for (int i = 0; i < Row<ACT, NV>::kWords / 4; ++i) {
          const u32x4_t x = __builtin_nontemporal_load(q + i);
          r.w[v][4 * i] = x[0]; r.w[v][4 * i + 1] = x[1]; r.w[v][4 * i + 2] = x[2]; r.w[v][4 * i + 3] = x[3];
        }
      } else {
#pragma unroll
        for (int i = 0; i < Row<ACT, NV>::kWords; ++i) r.w[v][i] = 0u;
      }
    } else {
      E e8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col_of<STRIDED>(t, T, v, e);
        e8[e] = c < D ? p[c] : E(0);
      }
#pragma unroll
      for (int i = 0; i < Row<ACT, NV>::kWords; ++i) {
        if constexpr (ACT::kBytes == 2)
          r.w[v][i] = static_cast<uint32_t>(e8[2 * i]) | (static_cast<uint32_t>(e8[2 * i + 1]) << 16);
        else
          r.w[v][i] = __float_as_uint(e8[i]);
      }
    }
  }
}

template <typename ACT, int NV>
__device__ __forceinline__ void unpack_row(const Row<ACT, NV>& r, float (&x)[NV][8]) {
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (ACT::kBytes == 2) x[v][e] = e % 2 ? bf16_hi(r.w[v][e / 2]) : bf16_lo(r.w[v][e / 2]);
      else x[v][e] = __uint_as_float(r.w[v][e]);
    }
}

template <typename ACT, int NV, bool STRIDED>
__device__ __forceinline__ void store_row(void* base, int64_t row0, int D, int t, int T, int vec,
                                          const float (&x)[NV][8]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c0 = (v * T + t) * 8;
    if (!STRIDED && vec) {
      if (c0 >= D) continue;
      if constexpr (ACT::kBytes == 2) {
        st_stream(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + row0 + c0),
                  make_uint4(pack_bf16x2(x[v][0], x[v][1]), pack_bf16x2(x[v][2], x[v][3]),
                             pack_bf16x2(x[v][4], x[v][5]), pack_bf16x2(x[v][6], x[v][7])));
      } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(base) + row0 + c0);
        st_stream(q, make_float4(x[v][0], x[v][1], x[v][2], x[v][3]));
        st_stream(q + 1, make_float4(x[v][4], x[v][5], x[v][6], x[v][7]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col_of<STRIDED>(t, T, v, e);
        if (c < D) store_act<ACT>(base, row0 + c, x[v][e]);
      }
    }
  }
}

// A weight's values of this thread's columns (fill where there is no weight or no column).
template <int NV, bool STRIDED>
__device__ __forceinline__ void load_weight(float (&x)[NV][8], const float* w, int D, int t, int T, int vec, float fill) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[v][e] = fill;
    if (!w) continue;
    if (!STRIDED && vec) {
      const int c0 = (v * T + t) * 8;
      if (c0 < D) {
        const float4 a = *reinterpret_cast<const float4*>(w + c0), b = *reinterpret_cast<const float4*>(w + c0 + 4);
        x[v][0] = a.x; x[v][1] = a.y; x[v][2] = a.z; x[v][3] = a.w;
        x[v][4] = b.x; x[v][5] = b.y; x[v][6] = b.z; x[v][7] = b.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col_of<STRIDED>(t, T, v, e);
        if (c < D) x[v][e] = w[c];
      }
    }
  }
}

// A weight's address that is not known before: its loads stay in the loop that they stand in.
__device__ __forceinline__ const float* here(const float* w) {
  asm volatile("" : "+s"(w));
  return w;
}

template <int VECTORS>                              // of a row, at most
struct TeamLds {
  float red[2][kMaxWaves][4];                       // two sets in turn: one barrier a sum
  float buf[2][VECTORS];
};

// Sums of N values over the team's threads, the same in all of them.  A team of one wave needs
// no LDS; `turn` flips with every call.
template <int N, bool ONE_WAVE, typename LDS>
__device__ __forceinline__ void team_sum(float (&s)[N], LDS& lds, int& turn, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = wave_sum(s[i]);
  if constexpr (!ONE_WAVE) {
    float(&red)[kMaxWaves][4] = lds.red[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[threadIdx.x >> 6][i] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.0f;
    for (int w = 0; w < waves; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += red[w][i];
    }
  }
}

// part[v] (the sum over vector v's 8 columns) -> its group's sum, for more than one group.  Groups of
// 8 * 2^k columns up to 512 are summed across lanes; others through LDS, in column order, where every thread adds
// its group's group / 8 sums: wide groups are bound by that (8192 x 5120 bfloat16 with gate: 80 groups 49 us, 8
// groups 64, 2 groups 129; gradient 125, 181, 309).
template <int NV, bool ONE_WAVE, typename LDS>
__device__ __forceinline__ void group_sum(float (&part)[NV], int group, int D, LDS& lds, int& turn, int t, int T) {
  const int span = group / 8;                       // vectors per group
  if ((span & (span - 1)) == 0 && span <= 64) {
    for (int d = 1; d < span; d <<= 1)
#pragma unroll
      for (int v = 0; v < NV; ++v) part[v] += __shfl_xor(part[v], d);
    return;
  }
  float* at = lds.buf[turn];
  turn ^= 1;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if ((v * T + t) * 8 < D) at[v * T + t] = part[v];
  if (ONE_WAVE) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  else __syncthreads();
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * T + t;
    if (i * 8 < D) {
      const int first = i / span * span;
      float s = 0.0f;
      for (int j = 0; j < span; ++j) s += at[first + j];
      part[v] = s;
    }
  }
}

// (the reciprocal is good to a unit in the last place; a division's ten instructions, for every value, are
// what a gated row would be bound by)
__device__ __forceinline__ float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.0f + exp2_hw(-z * kLog2e)); }

// The team of a thread: rows row0, row0 + step, ... of the matrix.
template <bool ONE_WAVE>
struct Team {
  int t, T, waves, index;
  int64_t row, step;
  __device__ Team() {
    T = ONE_WAVE ? 64 : static_cast<int>(blockDim.x);
    index = ONE_WAVE ? uniform_int(threadIdx.x >> 6) : 0;
    t = ONE_WAVE ? threadIdx.x & 63 : threadIdx.x;
    waves = T / 64;
    row = static_cast<int64_t>(blockIdx.x) * (ONE_WAVE ? kTeams : 1) + index;
    step = static_cast<int64_t>(gridDim.x) * (ONE_WAVE ? kTeams : 1);
  }
};

template <typename ACT, typename RES, int NV, int MAXT, bool LEAN, bool STRIDED>
__global__ __launch_bounds__(MAXT == 64 ? 64 * kTeams : MAXT) void norm_fwd_kernel(NormArgs p) {
  constexpr bool ONE_WAVE = MAXT == 64;
  __shared__ TeamLds<MAXT * NV> lds_all[ONE_WAVE ? kTeams : 1];
  const Team<ONE_WAVE> team;
  auto& lds = lds_all[team.index];
  const int D = static_cast<int>(p.D), vec = p.vec, t = team.t, T = team.T, group = static_cast<int>(p.group);
  int turn = 0;
  float w1[NV][8], rs[NV][8], w2[NV][8];
  const float inv_d = 1.0f / static_cast<float>(D), inv_g = 1.0f / static_cast<float>(group);
  Row<ACT, NV> nx, nz;
  Row<RES, NV> nr;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    load_row<ACT, NV, STRIDED>(nx, p.x, row * p.x_row, D, t, T, vec);
    if (p.gate) load_row<ACT, NV, STRIDED>(nz, p.gate, row * p.gate_row, D, t, T, vec);
    if (p.residual) load_row<RES, NV, STRIDED>(nr, p.residual, row * p.D, D, t, T, vec);
  };
  if constexpr (!LEAN) {
    load_weight<NV, STRIDED>(w1, p.w1, D, t, T, vec, 1.0f);
    load_weight<NV, STRIDED>(rs, p.rs, D, t, T, vec, 1.0f);
    load_weight<NV, STRIDED>(w2, p.w2, D, t, T, vec, 1.0f);
  }
  int64_t row = team.row;
  if (!LEAN && row < p.rows) fetch(row);
  for (; row < p.rows; row += team.step) {
    float x[NV][8], z[NV][8], r[NV][8];
    if constexpr (LEAN) fetch(row);
    unpack_row<ACT, NV>(nx, x);
    if (p.gate) unpack_row<ACT, NV>(nz, z);
    if (p.residual) unpack_row<RES, NV>(nr, r);
    if (!LEAN && row + team.step < p.rows) fetch(row + team.step);
    if (p.w1) {
      float part[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        part[v] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) part[v] = __builtin_fmaf(x[v][e], x[v][e], part[v]);
      }
      if (group == D) {
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) s[0] += part[v];
        team_sum<1, ONE_WAVE>(s, lds, turn, team.waves);
#pragma unroll
        for (int v = 0; v < NV; ++v) part[v] = s[0];
      } else {
        group_sum<NV, ONE_WAVE>(part, group, D, lds, turn, t, T);
      }
      if constexpr (LEAN) load_weight<NV, STRIDED>(w1, here(p.w1), D, t, T, vec, 1.0f);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const float r1 = 1.0f / sqrtf(__builtin_fmaf(part[v], inv_g, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] *= r1 * w1[v][e];
      }
    }
    if constexpr (LEAN) load_weight<NV, STRIDED>(rs, here(p.rs), D, t, T, vec, 1.0f);
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float a = x[v][e];
        if (p.gate) a *= z[v][e] * sigmoid_f(z[v][e]);
        a *= rs[v][e];
        if (p.residual) a += r[v][e];
        x[v][e] = a;
        s[0] = __builtin_fmaf(a, a, s[0]);          // (zeros past D)
      }
    if (p.h) store_row<RES, NV, STRIDED>(p.h, row * p.D, D, t, T, vec, x);
    if (p.y) {
      team_sum<1, ONE_WAVE>(s, lds, turn, team.waves);
      if constexpr (LEAN) load_weight<NV, STRIDED>(w2, here(p.w2), D, t, T, vec, 1.0f);
      const float r2 = 1.0f / sqrtf(__builtin_fmaf(s[0], inv_d, p.eps));
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] *= r2 * w2[v][e];
      store_row<ACT, NV, STRIDED>(p.y, row * p.D, D, t, T, vec, x);
    }
  }
}

template <typename ACT, typename RES, int NV, int MAXT, bool LEAN, bool STRIDED>
__global__ __launch_bounds__(MAXT == 64 ? 64 * kTeams : MAXT) void norm_bwd_kernel(NormArgs p) {
  constexpr bool ONE_WAVE = MAXT == 64;
  __shared__ TeamLds<MAXT * NV> lds_all[ONE_WAVE ? kTeams : 1];
  const Team<ONE_WAVE> team;
  auto& lds = lds_all[team.index];
  const int D = static_cast<int>(p.D), vec = p.vec, t = team.t, T = team.T, group = static_cast<int>(p.group);
  int turn = 0;
  float w1[NV][8], rs[NV][8], w2[NV][8];
  // Column sums of this team's rows: in registers, or (the first kLds of as, a2, a1) in LDS, every
  // thread's own, where 1024 threads leave too few registers.
  constexpr int kLds = MAXT == 1024 ? (NV == 1 ? 3 : 2) : 0;
  __shared__ __attribute__((aligned(16))) float sums[kLds ? kLds * NV * 8 * MAXT : 4];
  float a1[NV][8], as[NV][8], a2[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) a1[v][e] = as[v][e] = a2[v][e] = 0.0f;
  auto sum_at = [&](int which, int v, int half) {
    return reinterpret_cast<float4*>(sums) + ((which * NV + v) * 2 + half) * MAXT + t;
  };
  auto take = [&](float (&a)[NV][8], int which) __attribute__((always_inline)) {
    if (which >= kLds) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 x = *sum_at(which, v, i);
        a[v][4 * i] = x.x; a[v][4 * i + 1] = x.y; a[v][4 * i + 2] = x.z; a[v][4 * i + 3] = x.w;
      }
  };
  auto give = [&](const float (&a)[NV][8], int which) __attribute__((always_inline)) {
    if (which >= kLds) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *sum_at(which, v, i) = make_float4(a[v][4 * i], a[v][4 * i + 1], a[v][4 * i + 2], a[v][4 * i + 3]);
  };
  give(as, 0);
  give(a2, 1);
  give(a1, 2);
  const float inv_d = 1.0f / static_cast<float>(D), inv_g = 1.0f / static_cast<float>(group);
  const bool one_group = group == D;
  Row<ACT, NV> nx, nz, ny;
  Row<RES, NV> nh, ng;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    if (p.w2) {
      load_row<RES, NV, STRIDED>(nh, p.hin, row * p.D, D, t, T, vec);
      load_row<ACT, NV, STRIDED>(ny, p.dy, row * p.D, D, t, T, vec);
    }
    load_row<ACT, NV, STRIDED>(nx, p.x, row * p.x_row, D, t, T, vec);
  };
  auto fetch_dh = [&](int64_t row) __attribute__((always_inline)) {
    if (p.dh) load_row<RES, NV, STRIDED>(ng, p.dh, row * p.D, D, t, T, vec);
  };
  auto fetch_gate = [&](int64_t row) __attribute__((always_inline)) {
    if (p.gate) load_row<ACT, NV, STRIDED>(nz, p.gate, row * p.gate_row, D, t, T, vec);
  };
  auto fetch_all = [&](int64_t row) __attribute__((always_inline)) {
    fetch(row);
    fetch_dh(row);
    fetch_gate(row);
  };
  int64_t row = team.row;
  if (!LEAN && row < p.rows) fetch_all(row);
  if constexpr (!LEAN) {
    load_weight<NV, STRIDED>(w1, p.w1, D, t, T, vec, 1.0f);
    load_weight<NV, STRIDED>(rs, p.rs, D, t, T, vec, 1.0f);
    load_weight<NV, STRIDED>(w2, p.w2, D, t, T, vec, 1.0f);
  }
  for (; row < p.rows; row += team.step) {
    float x[NV][8], z[NV][8], dH[NV][8], h[NV][8], dy[NV][8];
    if constexpr (LEAN) fetch(row);
    unpack_row<ACT, NV>(nx, x);
    if (!LEAN && p.gate) unpack_row<ACT, NV>(nz, z);
    if (p.w2) {
      unpack_row<RES, NV>(nh, h);
      unpack_row<ACT, NV>(ny, dy);
    }
    auto take_dh = [&]() __attribute__((always_inline)) {
      if (p.dh) {
        unpack_row<RES, NV>(ng, dH);
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) dH[v][e] = 0.0f;
      }
    };
    if constexpr (!LEAN) take_dh();
    if (!LEAN && row + team.step < p.rows) fetch_all(row + team.step);
    if constexpr (LEAN) load_weight<NV, STRIDED>(w2, here(p.w2), D, t, T, vec, 1.0f);
    // the sums over the row that need nothing but the inputs, together
    float r1[NV], s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      r1[v] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) r1[v] = __builtin_fmaf(x[v][e], x[v][e], r1[v]);
      s[2] += r1[v];
      if (p.w2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] = __builtin_fmaf(h[v][e], h[v][e], s[0]);
          s[1] = __builtin_fmaf(dy[v][e] * w2[v][e], h[v][e], s[1]);
        }
      }
    }
    if (p.w2 || one_group) team_sum<3, ONE_WAVE>(s, lds, turn, team.waves);
    if constexpr (LEAN) {
      fetch_dh(row);
      take_dh();
    }
    if (p.w2) {
      const float r2 = 1.0f / sqrtf(__builtin_fmaf(s[0], inv_d, p.eps));
      const float ra = D > 1 ? r2 : r2 * p.eps * r2 * r2, rh = D > 1 ? r2 * (s[1] * inv_d * r2 * r2) : 0.0f;
      take(a2, 1);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a2[v][e] = __builtin_fmaf(dy[v][e], h[v][e] * r2, a2[v][e]);
          dH[v][e] = __builtin_fmaf(-h[v][e], rh, __builtin_fmaf(dy[v][e] * w2[v][e], ra, dH[v][e]));
        }
    }
    if (p.w2) give(a2, 1);
    if (p.dres) store_row<RES, NV, STRIDED>(p.dres, row * p.D, D, t, T, vec, dH);
    if constexpr (LEAN) {
      fetch_gate(row);
      if (p.gate) unpack_row<ACT, NV>(nz, z);
    }
    // x becomes x r1; n = x r1 post_weight
    if (p.w1) {
      if (one_group) {
#pragma unroll
        for (int v = 0; v < NV; ++v) r1[v] = s[2];
      } else {
        group_sum<NV, ONE_WAVE>(r1, group, D, lds, turn, t, T);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        r1[v] = 1.0f / sqrtf(__builtin_fmaf(r1[v], inv_g, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] *= r1[v];
      }
    }
    if constexpr (LEAN) load_weight<NV, STRIDED>(w1, here(p.w1), D, t, T, vec, 1.0f);
    if constexpr (LEAN) load_weight<NV, STRIDED>(rs, here(p.rs), D, t, T, vec, 1.0f);
    float m[NV];
    take(as, 0);
    take(a1, 2);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      m[v] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = x[v][e] * w1[v][e];
        float act = 1.0f, slope = 0.0f;
        if (p.gate) {
          const float sg = sigmoid_f(z[v][e]);
          act = z[v][e] * sg;
          slope = sg * (1.0f + z[v][e] * (1.0f - sg));
        }
        as[v][e] = __builtin_fmaf(dH[v][e], n * act, as[v][e]);
        const float dt = dH[v][e] * rs[v][e];
        z[v][e] = dt * n * slope;
        const float dn = dt * act;
        a1[v][e] = __builtin_fmaf(dn, x[v][e], a1[v][e]);
        dH[v][e] = dn * w1[v][e];
        m[v] = __builtin_fmaf(dH[v][e], x[v][e], m[v]);
      }
    }
    give(as, 0);
    give(a1, 2);
    if (p.gate) store_row<ACT, NV, STRIDED>(p.dgate, row * p.D, D, t, T, vec, z);
    if (p.w1) {
      if (one_group) {
        float u[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) u[0] += m[v];
        team_sum<1, ONE_WAVE>(u, lds, turn, team.waves);
#pragma unroll
        for (int v = 0; v < NV; ++v) m[v] = u[0];
      } else {
        group_sum<NV, ONE_WAVE>(m, group, D, lds, turn, t, T);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const float rc = D > 1 ? r1[v] : r1[v] * p.eps * r1[v] * r1[v], rx = D > 1 ? r1[v] * (m[v] * inv_g) : 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) dH[v][e] = __builtin_fmaf(-x[v][e], rx, dH[v][e] * rc);
      }
    }
    store_row<ACT, NV, STRIDED>(p.dx, row * p.D, D, t, T, vec, dH);
  }
  // the workgroup's column sums; the teams of a workgroup are added in order
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * 3 * D;
  auto leave = [&](const float (&a)[NV][8], const float* wanted, float* to) __attribute__((always_inline)) {
    if (!wanted) return;
    if constexpr (ONE_WAVE) {
      __shared__ float sum[kTeams][NV * 512];
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = col_of<STRIDED>(t, T, v, e);
          if (c < D) sum[team.index][c] = a[v][e];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += 64 * kTeams) {
        float s = sum[0][c];
#pragma unroll
        for (int i = 1; i < kTeams; ++i) s += sum[i][c];
        to[c] = s;
      }
    } else {
      store_row<ActF32, NV, STRIDED>(to, 0, D, t, T, vec, a);
    }
  };
  take(as, 0);
  take(a2, 1);
  take(a1, 2);
  leave(a1, p.dw1, out);
  leave(as, p.drs, out + D);
  leave(a2, p.dw2, out + 2 * static_cast<int64_t>(D));
}

// Column sums over the workgroups' partial sums: 64 columns by 16 strands of parts a
// workgroup, 16 parts of a strand in flight; strands are added in order.
constexpr int kStrands = 16, kFlight = 16;
__global__ __launch_bounds__(64 * kStrands) void norm_bwd_sum_kernel(NormArgs p) {
  __shared__ float red[kStrands][64];
  const int which = blockIdx.y;
  float* out = which == 0 ? p.dw1 : which == 1 ? p.drs : p.dw2;
  if (!out) return;
  const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const float* src = p.part + which * p.D + (c < p.D ? c : p.D - 1);
  const int64_t step = 3 * p.D;
  float s = 0.0f;
  for (int i = strand; i < p.parts; i += kFlight * kStrands) {
    float v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int k = i + u * kStrands;
      v[u] = src[(k < p.parts ? k : i) * step];
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) s += i + u * kStrands < p.parts ? v[u] : 0.0f;
  }
  red[strand][lane] = s;
  __syncthreads();
  if (strand == 0 && c < p.D) {
#pragma unroll
    for (int i = 1; i < kStrands; ++i) s += red[i][lane];
    out[c] = s;
  }
}

// How a row is laid out over threads: one wave up to 512 columns, else whole waves at one
// vector of 8 columns a thread up to 8192, two past that.  Workgroups of more than 512 threads have
// 128 registers a thread, which hold neither the gradient's sums (they go to LDS) nor the next row and the
// weights: those kernels are LEAN, asking for rows and weights as they need them.  Measured, gradients of
// bfloat16 rows with gate, scale and float32 residual: 8192 x 5120 345 us with the sums in registers (spilled),
// 282 in LDS, 330 with two vectors a thread and 512 threads; 4096 x 8192 257, 205, 215.
struct Shape {
  int threads, rows;                  // threads and rows of a workgroup
};
Shape shape_of(int64_t D) {
  if (D <= 512) return Shape{64 * kTeams, kTeams};
  const int64_t per_wave = D <= 8192 ? 512 : 1024;
  return Shape{static_cast<int>((D + per_wave - 1) / per_wave) * 64, 1};
}

template <typename ACT, typename RES, bool STRIDED>
void launch_norm_s(const NormArgs& a, bool bwd, int blocks, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(static_cast<unsigned>(shape_of(a.D).threads));
  auto go = [&](auto fwd_kernel, auto bwd_kernel) {
    if (bwd) hipLaunchKernelGGL(bwd_kernel, grid, block, 0, s, a);
    else hipLaunchKernelGGL(fwd_kernel, grid, block, 0, s, a);
  };
  if (a.D <= 512)
    go(norm_fwd_kernel<ACT, RES, 1, 64, false, STRIDED>, norm_bwd_kernel<ACT, RES, 1, 64, false, STRIDED>);
  else if (a.D <= 4096)
    go(norm_fwd_kernel<ACT, RES, 1, 512, false, STRIDED>, norm_bwd_kernel<ACT, RES, 1, 512, false, STRIDED>);
  else if (a.D <= 8192)
    go(norm_fwd_kernel<ACT, RES, 1, 1024, false, STRIDED>, norm_bwd_kernel<ACT, RES, 1, 1024, true, STRIDED>);
  else
    go(norm_fwd_kernel<ACT, RES, 2, 1024, true, STRIDED>, norm_bwd_kernel<ACT, RES, 2, 1024, true, STRIDED>);
}

hipError_t launch_norm(const NormArgs& a, Dt dt, Dt rdt, bool bwd, int blocks, hipStream_t s) {
  const bool strided = !a.vec && a.group == a.D;
  if (dt == Dt::F32) {
    if (strided) launch_norm_s<ActF32, ActF32, true>(a, bwd, blocks, s);
    else launch_norm_s<ActF32, ActF32, false>(a, bwd, blocks, s);
  } else if (rdt == Dt::F32) {
    if (strided) launch_norm_s<ActBF16, ActF32, true>(a, bwd, blocks, s);
    else launch_norm_s<ActBF16, ActF32, false>(a, bwd, blocks, s);
  } else {
    if (strided) launch_norm_s<ActBF16, ActBF16, true>(a, bwd, blocks, s);
    else launch_norm_s<ActBF16, ActBF16, false>(a, bwd, blocks, s);
  }
  return hipGetLastError();
}

// Workgroups: at most `most` threads' worth on each of the 256 CUs.  Rows in flight against registers of
// column sums to add up: 1024 forwards (16384 x 2560 109 us, 185 with 512, 134 with 2048; 4096 x 1024 11.6, 14, 15.3;
// where a row takes over 512 threads, 8192 x 5120, 80 groups with gate: 49 us, 51 with 2048; 8192 x 6144 73, 74), 512
// backwards (4096 x 1024 34 us, 44 with 1024, 41 with 256; 16384 x 512 43, 50, 54; 1534 x 769 23, 29, 23).
int blocks_of(int64_t rows, int64_t D, int most) {
  const Shape sh = shape_of(D);
  const int64_t need = (rows + sh.rows - 1) / sh.rows;
  int64_t full = 256 * static_cast<int64_t>(most / sh.threads > 1 ? most / sh.threads : 1);
  return static_cast<int>(need < full ? need : full);
}

}  // namespace

int norm_bwd_parts(int64_t rows, int64_t D) { return blocks_of(rows, D, 512); }

hipError_t launch_norm_fwd(const NormArgs& a, Dt dt, Dt rdt, hipStream_t s) {
  return launch_norm(a, dt, rdt, false, blocks_of(a.rows, a.D, 1024), s);
}

hipError_t launch_norm_bwd(const NormArgs& a, Dt dt, Dt rdt, hipStream_t s) {
  const hipError_t e = launch_norm(a, dt, rdt, true, a.parts, s);
  if (e != hipSuccess) return e;
  if (a.dw1 || a.drs || a.dw2)
    hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3(static_cast<unsigned>((a.D + 63) / 64), 3), dim3(64 * kStrands), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssm
