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
// A few flops per value: bound by HBM, so every value is read and written once.  A team of
// T threads holds a whole row in registers (NV vectors of 8 columns a thread) between the
// sums and the results.  The backward pass runs row blocks: the team's columns stay
// the same over its rows, so the column sums of the weights' gradients accumulate in
// registers and leave once per block; a second kernel adds the blocks in a fixed order.
#include "device_common.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kTeams = 4;            // rows per workgroup where a row is one wave's

// Column of element e of vector v of thread t.  Blocked: 8 consecutive columns a vector.
// Strided (one group, rows that do not move as vectors): consecutive threads, consecutive columns.
template <int T, bool STRIDED>
__device__ __forceinline__ int col_of(int t, int v, int e) {
  return STRIDED ? (v * 8 + e) * T + t : (v * T + t) * 8 + e;
}

template <typename ACT, int T, int NV, bool STRIDED>
__device__ __forceinline__ void load_row(const void* base, int64_t row0, int D, int t, int vec, float (&x)[NV][8]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c0 = (v * T + t) * 8;
    if (!STRIDED && vec) {
      if (c0 < D) {
        load_act8<ACT>(base, row0 + c0, x[v]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] = 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col_of<T, STRIDED>(t, v, e);
        x[v][e] = c < D ? load_act<ACT>(base, row0 + c) : 0.0f;
      }
    }
  }
}

template <typename ACT, int T, int NV, bool STRIDED>
__device__ __forceinline__ void store_row(void* base, int64_t row0, int D, int t, int vec, const float (&x)[NV][8]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c0 = (v * T + t) * 8;
    if (!STRIDED && vec) {
      if (c0 < D) store_act8<ACT>(base, row0 + c0, x[v]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col_of<T, STRIDED>(t, v, e);
        if (c < D) store_act<ACT>(base, row0 + c, x[v][e]);
      }
    }
  }
}

// Sum over the team's threads, the same in all of them.  red: one float per wave of the team.
template <int T>
__device__ __forceinline__ float team_sum(float v, float* red, int t) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    __syncthreads();                                // (the previous sum's readers are done)
    if ((t & 63) == 0) red[t >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += red[i];
  }
  return v;
}

// part[v] (the sum over vector v's 8 columns) -> its group's sum.  Groups of 8 * 2^k columns up
// to 512 are summed across lanes; others through LDS (buf: D / 8 floats), in column order.
template <int T, int NV>
__device__ __forceinline__ void group_sum(float (&part)[NV], int group, int D, float* red, float* buf, int t) {
  if (group == D) {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) s += part[v];
    s = team_sum<T>(s, red, t);
#pragma unroll
    for (int v = 0; v < NV; ++v) part[v] = s;
    return;
  }
  const int span = group / 8;                       // vectors per group
  if ((span & (span - 1)) == 0 && span <= 64) {
    for (int d = 1; d < span; d <<= 1)
#pragma unroll
      for (int v = 0; v < NV; ++v) part[v] += __shfl_xor(part[v], d);
    return;
  }
  if (T > 64) __syncthreads();
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if ((v * T + t) * 8 < D) buf[v * T + t] = part[v];
  if (T > 64) __syncthreads();
  else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * T + t;
    if (i * 8 < D) {
      const int first = i / span * span;
      float s = 0.0f;
      for (int j = 0; j < span; ++j) s += buf[first + j];
      part[v] = s;
    }
  }
  if (T == 64) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.0f / (1.0f + exp2_hw(-z * kLog2e)); }

template <int T, int NV>
struct TeamLds {
  static constexpr int kRows = T == 64 ? kTeams : 1;
  float red[kRows][T / 64];
  float buf[kRows][T * NV];
};

template <typename ACT, typename RES, int T, int NV, bool STRIDED>
__global__ __launch_bounds__(T == 64 ? 64 * kTeams : T) void norm_fwd_kernel(NormArgs p) {
  __shared__ TeamLds<T, NV> lds;
  constexpr int kRows = TeamLds<T, NV>::kRows;
  const int team = kRows > 1 ? uniform_int(threadIdx.x >> 6) : 0, t = kRows > 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + team;
  if (row >= p.rows) return;                        // (whole waves; one row per workgroup where T > 64)
  const int D = static_cast<int>(p.D), vec = p.vec;
  float* red = lds.red[team];
  float x[NV][8];
  load_row<ACT, T, NV, STRIDED>(p.x, row * p.x_row, D, t, vec, x);
  float z[NV][8], r[NV][8];
  if (p.gate) load_row<ACT, T, NV, STRIDED>(p.gate, row * p.gate_row, D, t, vec, z);
  if (p.residual) load_row<RES, T, NV, STRIDED>(p.residual, row * p.D, D, t, vec, r);
  if (p.w1) {
    float part[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      part[v] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) part[v] = __builtin_fmaf(x[v][e], x[v][e], part[v]);
    }
    group_sum<T, NV>(part, static_cast<int>(p.group), D, red, lds.buf[team], t);
    float w[NV][8];
    load_row<ActF32, T, NV, STRIDED>(p.w1, 0, D, t, vec, w);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float r1 = 1.0f / sqrtf(part[v] / static_cast<float>(p.group) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] *= r1 * w[v][e];
    }
  }
  if (p.gate) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] *= z[v][e] * sigmoid_f(z[v][e]);
  }
  if (p.rs) {
    float w[NV][8];
    load_row<ActF32, T, NV, STRIDED>(p.rs, 0, D, t, vec, w);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] *= w[v][e];
  }
  if (p.residual) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] += r[v][e];
  }
  if (p.h) store_row<RES, T, NV, STRIDED>(p.h, row * p.D, D, t, vec, x);
  if (p.y) {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[v][e], x[v][e], s);   // (zeros past D)
    s = team_sum<T>(s, red, t);
    const float r2 = 1.0f / sqrtf(s / static_cast<float>(D) + p.eps);
    float w[NV][8];
    load_row<ActF32, T, NV, STRIDED>(p.w2, 0, D, t, vec, w);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] *= r2 * w[v][e];
    store_row<ACT, T, NV, STRIDED>(p.y, row * p.D, D, t, vec, x);
  }
}

template <typename ACT, typename RES, int T, int NV, bool STRIDED>
__global__ __launch_bounds__(T == 64 ? 64 * kTeams : T) void norm_bwd_kernel(NormArgs p) {
  __shared__ TeamLds<T, NV> lds;
  constexpr int kRows = TeamLds<T, NV>::kRows;
  const int team = kRows > 1 ? uniform_int(threadIdx.x >> 6) : 0, t = kRows > 1 ? threadIdx.x & 63 : threadIdx.x;
  const int part_id = static_cast<int>(blockIdx.x) * kRows + team;
  const int D = static_cast<int>(p.D), vec = p.vec;
  float* red = lds.red[team];
  float a1[NV][8], as[NV][8], a2[NV][8];            // column sums of this block's rows
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) a1[v][e] = as[v][e] = a2[v][e] = 0.0f;
  if (part_id >= p.parts) return;
  const float inv_d = 1.0f / static_cast<float>(D), inv_g = 1.0f / static_cast<float>(p.group);
  for (int64_t row = part_id; row < p.rows; row += p.parts) {
    float dH[NV][8];
    if (p.dh) {
      load_row<RES, T, NV, STRIDED>(p.dh, row * p.D, D, t, vec, dH);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) dH[v][e] = 0.0f;
    }
    float x[NV][8], z[NV][8];
    load_row<ACT, T, NV, STRIDED>(p.x, row * p.x_row, D, t, vec, x);
    if (p.gate) load_row<ACT, T, NV, STRIDED>(p.gate, row * p.gate_row, D, t, vec, z);
    if (p.w2) {
      float h[NV][8], dy[NV][8], w[NV][8];
      load_row<RES, T, NV, STRIDED>(p.hin, row * p.D, D, t, vec, h);
      load_row<ACT, T, NV, STRIDED>(p.dy, row * p.D, D, t, vec, dy);
      load_row<ActF32, T, NV, STRIDED>(p.w2, 0, D, t, vec, w);
      float s = 0.0f, d = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s = __builtin_fmaf(h[v][e], h[v][e], s);
          d = __builtin_fmaf(dy[v][e] * w[v][e], h[v][e], d);
        }
      s = team_sum<T>(s, red, t);
      d = team_sum<T>(d, red, t);
      const float r2 = 1.0f / sqrtf(s * inv_d + p.eps);
      const float m = d * inv_d * r2 * r2;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a2[v][e] = __builtin_fmaf(dy[v][e], h[v][e] * r2, a2[v][e]);
          const float a = dy[v][e] * w[v][e];
          dH[v][e] = __builtin_fmaf(r2, D > 1 ? __builtin_fmaf(-h[v][e], m, a) : a * p.eps * r2 * r2, dH[v][e]);
        }
    }
    if (p.dres) store_row<RES, T, NV, STRIDED>(p.dres, row * p.D, D, t, vec, dH);
    // x becomes x r1; n = x r1 post_weight
    float w1[NV][8], r1[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) r1[v] = 1.0f;
    if (p.w1) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        r1[v] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) r1[v] = __builtin_fmaf(x[v][e], x[v][e], r1[v]);
      }
      group_sum<T, NV>(r1, static_cast<int>(p.group), D, red, lds.buf[team], t);
      load_row<ActF32, T, NV, STRIDED>(p.w1, 0, D, t, vec, w1);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        r1[v] = 1.0f / sqrtf(r1[v] * inv_g + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] *= r1[v];
      }
    }
    float rs[NV][8];
    if (p.rs) load_row<ActF32, T, NV, STRIDED>(p.rs, 0, D, t, vec, rs);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = p.w1 ? x[v][e] * w1[v][e] : x[v][e];
        float act = 1.0f, slope = 0.0f;
        if (p.gate) {
          const float sg = sigmoid_f(z[v][e]);
          act = z[v][e] * sg;
          slope = sg * (1.0f + z[v][e] * (1.0f - sg));
        }
        as[v][e] = __builtin_fmaf(dH[v][e], n * act, as[v][e]);
        float dt = dH[v][e];
        if (p.rs) dt *= rs[v][e];
        z[v][e] = dt * n * slope;
        dH[v][e] = dt * act;                        // dn
      }
    if (p.gate) store_row<ACT, T, NV, STRIDED>(p.dgate, row * p.D, D, t, vec, z);
    if (p.w1) {
      float m[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        m[v] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a1[v][e] = __builtin_fmaf(dH[v][e], x[v][e], a1[v][e]);
          dH[v][e] *= w1[v][e];
          m[v] = __builtin_fmaf(dH[v][e], x[v][e], m[v]);
        }
      }
      group_sum<T, NV>(m, static_cast<int>(p.group), D, red, lds.buf[team], t);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dH[v][e] = r1[v] * (D > 1 ? __builtin_fmaf(-x[v][e], m[v] * inv_g, dH[v][e]) : dH[v][e] * p.eps * r1[v] * r1[v]);
    }
    store_row<ACT, T, NV, STRIDED>(p.dx, row * p.D, D, t, vec, dH);
  }
  float* out = p.part + static_cast<int64_t>(part_id) * 3 * D;
  if (p.dw1) store_row<ActF32, T, NV, STRIDED>(out, 0, D, t, vec, a1);
  if (p.drs) store_row<ActF32, T, NV, STRIDED>(out, D, D, t, vec, as);
  if (p.dw2) store_row<ActF32, T, NV, STRIDED>(out, 2 * static_cast<int64_t>(D), D, t, vec, a2);
}

// Column sums over the blocks, in block order: 64 columns by 4 strands of blocks a workgroup.
__global__ __launch_bounds__(256) void norm_bwd_sum_kernel(NormArgs p) {
  __shared__ float red[4][64];
  const int which = blockIdx.y;
  float* out = which == 0 ? p.dw1 : which == 1 ? p.drs : p.dw2;
  if (!out) return;
  const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float s = 0.0f;
  if (c < p.D)
    for (int i = strand; i < p.parts; i += 4) s += p.part[(static_cast<int64_t>(i) * 3 + which) * p.D + c];
  red[strand][lane] = s;
  __syncthreads();
  if (strand == 0 && c < p.D) out[c] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
}

template <typename ACT, typename RES, int T, int NV, bool STRIDED>
void launch_norm_t(const NormArgs& a, bool bwd, hipStream_t s) {
  constexpr int kRows = TeamLds<T, NV>::kRows;
  const dim3 block(T == 64 ? 64 * kTeams : T);
  const int64_t n = bwd ? a.parts : a.rows;
  const dim3 grid(static_cast<unsigned>((n + kRows - 1) / kRows));
  if (bwd) hipLaunchKernelGGL((norm_bwd_kernel<ACT, RES, T, NV, STRIDED>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_fwd_kernel<ACT, RES, T, NV, STRIDED>), grid, block, 0, s, a);
}

template <typename ACT, typename RES, bool STRIDED>
void launch_norm_s(const NormArgs& a, bool bwd, hipStream_t s) {
  if (a.D <= 512) launch_norm_t<ACT, RES, 64, 1, STRIDED>(a, bwd, s);
  else if (a.D <= 1024) launch_norm_t<ACT, RES, 64, 2, STRIDED>(a, bwd, s);
  else if (a.D <= 2048) launch_norm_t<ACT, RES, 256, 1, STRIDED>(a, bwd, s);
  else if (a.D <= 4096) launch_norm_t<ACT, RES, 256, 2, STRIDED>(a, bwd, s);
  else if (a.D <= 8192) launch_norm_t<ACT, RES, 512, 2, STRIDED>(a, bwd, s);
  else launch_norm_t<ACT, RES, 1024, 2, STRIDED>(a, bwd, s);
}

hipError_t launch_norm(const NormArgs& a, Dt dt, Dt rdt, bool bwd, hipStream_t s) {
  const bool strided = !a.vec && a.group == a.D;
  if (dt == Dt::F32) {
    if (strided) launch_norm_s<ActF32, ActF32, true>(a, bwd, s);
    else launch_norm_s<ActF32, ActF32, false>(a, bwd, s);
  } else if (rdt == Dt::F32) {
    if (strided) launch_norm_s<ActBF16, ActF32, true>(a, bwd, s);
    else launch_norm_s<ActBF16, ActF32, false>(a, bwd, s);
  } else {
    if (strided) launch_norm_s<ActBF16, ActBF16, true>(a, bwd, s);
    else launch_norm_s<ActBF16, ActBF16, false>(a, bwd, s);
  }
  return hipGetLastError();
}

}  // namespace

int norm_bwd_parts(int64_t rows, int64_t D) {
  const int64_t most = D <= 1024 ? 1024 : 512;
  return static_cast<int>(rows < most ? rows : most);
}

hipError_t launch_norm_fwd(const NormArgs& a, Dt dt, Dt rdt, hipStream_t s) {
  return launch_norm(a, dt, rdt, false, s);
}

hipError_t launch_norm_bwd(const NormArgs& a, Dt dt, Dt rdt, hipStream_t s) {
  const hipError_t e = launch_norm(a, dt, rdt, true, s);
  if (e != hipSuccess) return e;
  if (a.dw1 || a.drs || a.dw2)
    hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3(static_cast<unsigned>((a.D + 63) / 64), 3), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssm
