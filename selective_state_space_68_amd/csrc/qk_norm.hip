// Norms of queries and keys for each head, with the position rotation in the same pass, and their gradient.
//
// For a row x of K columns (one token's one head):
//     n = w x r,   r = 1 / sqrt(mean x^2 + eps)  or  1 / sqrt(sum x^2 + eps)     (w left out where it is not given)
//     y = n with its first `rotary` columns turned in pairs by the angles position * inv_freq[pair]
// and backwards, with dn = dy turned back:  dw = sum over rows of dn x r,   dx = r (w dn - x r m),  m = the mean, or the
// sum, of w dn x r over the row.
//
// Every value is read and written once: the kernels are bound by memory (bfloat16 heads of 128: 8192 x 40 without rotation 27 us, 6.1 TB/s;
// gradient of 16384 x 40, rotated, 107 us, 4.7 TB/s, half the vector unit's time).  A row is held by 8 to 64 lanes of a wave, 8 values
// each; a lane has both members of its pairs, so nothing but the row's sum crosses lanes.  A group of lanes takes
// several heads of its token, so that its angles, whose sines and cosines cost more than a row's norm, are formed
// once for all of them: in float64 up to the turn's fraction (position 10^6 leaves 4 bits of a float32 angle), in float32
// from there.  Sums are float32.  The weights' gradients are summed over a group's rows in registers, over a workgroup's
// groups in LDS, and over workgroups by a second kernel, in one order.
#include "device_common.hpp"
#include "lm_kernels.hpp"
#include "row_sum.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kParts = 1024;         // most workgroups of a gradient with weights

// Four consecutive values.
template <typename ACT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&v)[4]) {
  if constexpr (ACT::kBytes == 4) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
  }
}
template <typename ACT>
__device__ __forceinline__ void store4(void* p, int64_t i, const float (&v)[4]) {
  if constexpr (ACT::kBytes == 4)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// 1 / sqrt(x).  The hardware's root takes numbers below 2^-126 for 0: small ones are scaled.
__device__ __forceinline__ float inverse_root(float x) {
  const bool small = x < 0x1p-100f;
  return __builtin_amdgcn_rsqf(small ? x * 0x1p100f : x) * (small ? 0x1p50f : 1.0f);
}

// sin and cos of position * frequency.  (The hardware's sine of turns for bfloat16 rows saved 1 of 128 us: 16384 x 40 heads of
// 128, gradient.)
__device__ __forceinline__ void turn_of(double position, float frequency, float* s, float* c) {
  double turns = position * static_cast<double>(frequency) * 0.15915494309189535;      // over 2 pi
  turns -= __builtin_rint(turns);
  sincospif(static_cast<float>(2.0 * turns), s, c);
}

// The columns of one lane, 8 (VEC: two pieces of 4) or NI pairs or single columns a wave apart, and their turns.
// VEC: K, rotary and all rows allow pieces of 4 elements; each of G lanes has unit `lane` of 8 columns.
// Otherwise G is 64, and item lane + 64 i is pair number that of the rotated columns, or a single column behind them.
template <typename ACT, int G, int NI, bool VEC>
struct Row {
  static constexpr int N = VEC ? 4 : NI;            // pairs of a lane
  int col[N][2];                                    // columns of a pair's members; < 0: none
  float c[N], s[N];
  bool any;                                         // this lane has columns
  bool apart;                                       // (VEC) members of a pair are in the two pieces

  __device__ __forceinline__ void columns(const QkArgs& p, int lane) {
    const int r = p.rotary, half = r / 2;
    if constexpr (VEC) {
      any = 8 * lane < p.K;
      apart = 8 * lane < r && !p.interleaved;
      const int first = apart ? 4 * lane : 8 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        col[i][0] = apart ? first + i : first + 2 * i;
        col[i][1] = apart ? first + half + i : first + 2 * i + 1;
      }
    } else {
      any = true;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int x = lane + 64 * i;
        if (x < half) {
          col[i][0] = p.interleaved ? 2 * x : x;
          col[i][1] = p.interleaved ? 2 * x + 1 : x + half;
        } else {
          col[i][0] = r + x - half < p.K ? r + x - half : -1;
          col[i][1] = -1;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
  }
  __device__ __forceinline__ int pair_of(const QkArgs& p, int lane, int i) const {   // < 0: not rotated
    if constexpr (VEC) {
      if (!any || 8 * lane >= p.rotary) return -1;
      return 4 * lane + i;
    } else {
      const int x = lane + 64 * i;
      return x < p.rotary / 2 ? x : -1;
    }
  }
  __device__ __forceinline__ void turns(const QkArgs& p, int lane, int64_t token, int64_t t) {
    if (!p.rotary) return;
    const double position = static_cast<double>(p.positions ? p.positions[token] : static_cast<int32_t>(t));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pair = pair_of(p, lane, i);
      if (pair >= 0) turn_of(position, p.inv_freq[pair], &s[i], &c[i]);
    }
  }
  // x[i][m]: member m of pair i; 0 where there is none
  __device__ __forceinline__ void load(const void* base, int64_t at, float (&x)[N][2]) const {
    if constexpr (VEC) {
      float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
      if (any) {
        load4<ACT>(base, at + col[0][0], a);
        load4<ACT>(base, at + (apart ? col[0][1] : col[0][0] + 4), b);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i][0] = apart ? a[i] : (i < 2 ? a[2 * i] : b[2 * i - 4]);
        x[i][1] = apart ? b[i] : (i < 2 ? a[2 * i + 1] : b[2 * i - 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m) x[i][m] = col[i][m] >= 0 ? load_act<ACT>(base, at + col[i][m]) : 0.0f;
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t at, const float (&x)[N][2]) const {
    if constexpr (VEC) {
      if (!any) return;
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = apart ? x[i][0] : x[i / 2][i % 2];
        b[i] = apart ? x[i][1] : x[2 + i / 2][i % 2];
      }
      store4<ACT>(base, at + col[0][0], a);
      store4<ACT>(base, at + (apart ? col[0][1] : col[0][0] + 4), b);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          if (col[i][m] >= 0) store_act<ACT>(base, at + col[i][m], x[i][m]);
    }
  }
  __device__ __forceinline__ void weights(const float* w, float (&x)[N][2]) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m) x[i][m] = w && any && col[i][m] >= 0 ? w[col[i][m]] : 1.0f;
  }
  static __device__ __forceinline__ float sum(float v) {
    if constexpr (G == 64) return wave_sum(v);
    v = row_sum<G == 8 ? 8 : 16>(v);
    if constexpr (G == 32) v += __shfl_xor(v, 16);
    return v;
  }
};

// The token and the first head of a group of lanes; a token's heads are dealt to `p.split` groups.
template <int G>
struct Place {
  int lane, group;
  int64_t item, items, step;
  __device__ __forceinline__ Place(const QkArgs& p) {
    lane = threadIdx.x % G;
    group = threadIdx.x / G;
    constexpr int kGroups = kThreads / G;
    item = static_cast<int64_t>(blockIdx.x) * kGroups + group;
    items = p.batch * p.L * p.split;
    step = static_cast<int64_t>(gridDim.x) * kGroups;
  }
  // a / b, for a below `items` and b no larger (32-bit where they are: a 64-bit division is 500 cycles)
  __device__ __forceinline__ int64_t over(int64_t a, int64_t b) const {
    return items < (int64_t(1) << 32) ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
  }
};

template <typename ACT, int G, int NI, bool VEC>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(QkArgs p) {
  using R = Row<ACT, G, NI, VEC>;
  const Place<G> at(p);
  R row;
  row.columns(p, at.lane);
  float wq[R::N][2], wk[R::N][2];
  row.weights(p.qw, wq);
  row.weights(p.kw, wk);
  for (int64_t item = at.item; item < at.items; item += at.step) {
    const int64_t token = p.split == 1 ? item : at.over(item, p.split);
    const int first = static_cast<int>(item - token * p.split);
    const int64_t b = p.batch == 1 ? 0 : at.over(token, p.L), t = token - b * p.L;
    row.turns(p, at.lane, token, t);
    auto heads = [&](int h, int count, const void* in, const int64_t (&st)[3], const float (&wt)[R::N][2], void* out)
                     __attribute__((always_inline)) {
      const int64_t base = b * st[0] + t * st[1], to = token * count;
      for (; h < count; h += p.split) {
        float x[R::N][2];
        row.load(in, base + h * st[2], x);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < R::N; ++i) ss = __builtin_fmaf(x[i][0], x[i][0], __builtin_fmaf(x[i][1], x[i][1], ss));
        ss = R::sum(ss);
        const float r = inverse_root(__builtin_fmaf(ss, p.inv_count, p.eps));
#pragma unroll
        for (int i = 0; i < R::N; ++i) {
          const float a = x[i][0] * r * wt[i][0], d = x[i][1] * r * wt[i][1];
          x[i][0] = __builtin_fmaf(a, row.c[i], -d * row.s[i]);
          x[i][1] = __builtin_fmaf(d, row.c[i], a * row.s[i]);
        }
        row.store(out, (to + h) * p.K, x);
      }
      return h - count;                             // (the first of the next tensor's heads)
    };
    heads(heads(first, p.Hq, p.q, p.qs, wq, p.qo), p.Hk, p.k, p.ks, wk, p.ko);
  }
}

template <typename ACT, int G, int NI, bool VEC>
__global__ __launch_bounds__(kThreads) void qk_norm_bwd_kernel(QkArgs p) {
  using R = Row<ACT, G, NI, VEC>;
  __shared__ float part[kThreads * 2 * R::N];       // a row of K (at most G times a lane's columns) a group
  const Place<G> at(p);
  R row;
  row.columns(p, at.lane);
  float wq[R::N][2], wk[R::N][2], dwq[R::N][2], dwk[R::N][2];
  row.weights(p.qw, wq);
  row.weights(p.kw, wk);
#pragma unroll
  for (int i = 0; i < R::N; ++i) dwq[i][0] = dwq[i][1] = dwk[i][0] = dwk[i][1] = 0.0f;
  for (int64_t item = at.item; item < at.items; item += at.step) {
    const int64_t token = p.split == 1 ? item : at.over(item, p.split);
    const int first = static_cast<int>(item - token * p.split);
    const int64_t b = p.batch == 1 ? 0 : at.over(token, p.L), t = token - b * p.L;
    row.turns(p, at.lane, token, t);
    auto heads = [&](int h, int count, const void* in, const int64_t (&st)[3], const void* grad, const int64_t (&ds)[3],
                     const float (&wt)[R::N][2], float (&dw)[R::N][2], void* out) __attribute__((always_inline)) {
      const int64_t base = b * st[0] + t * st[1], dbase = b * ds[0] + t * ds[1], to = token * count;
      for (; h < count; h += p.split) {
        float x[R::N][2], y[R::N][2];
        row.load(in, base + h * st[2], x);
        row.load(grad, dbase + h * ds[2], y);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < R::N; ++i) ss = __builtin_fmaf(x[i][0], x[i][0], __builtin_fmaf(x[i][1], x[i][1], ss));
        ss = R::sum(ss);
        const float r = inverse_root(__builtin_fmaf(ss, p.inv_count, p.eps));
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < R::N; ++i) {
          const float a = __builtin_fmaf(y[i][0], row.c[i], y[i][1] * row.s[i]);       // dn: turned back
          const float d = __builtin_fmaf(y[i][1], row.c[i], -y[i][0] * row.s[i]);
          x[i][0] *= r;
          x[i][1] *= r;
          dw[i][0] = __builtin_fmaf(a, x[i][0], dw[i][0]);
          dw[i][1] = __builtin_fmaf(d, x[i][1], dw[i][1]);
          y[i][0] = a * wt[i][0];
          y[i][1] = d * wt[i][1];
          dot = __builtin_fmaf(y[i][0], x[i][0], __builtin_fmaf(y[i][1], x[i][1], dot));
        }
        dot = R::sum(dot) * p.inv_count;
#pragma unroll
        for (int i = 0; i < R::N; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m) y[i][m] = r * __builtin_fmaf(-x[i][m], dot, y[i][m]);
        row.store(out, (to + h) * p.K, y);
      }
      return h - count;
    };
    heads(heads(first, p.Hq, p.q, p.qs, p.dqo, p.dqs, wq, dwq, p.qo), p.Hk, p.k, p.ks, p.dko, p.dks, wk, dwk, p.ko);
  }
  constexpr int kGroups = kThreads / G;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!(which ? p.dkw : p.dqw)) continue;
    __syncthreads();
    if (row.any) {
#pragma unroll
      for (int i = 0; i < R::N; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          if (row.col[i][m] >= 0) part[at.group * p.K + row.col[i][m]] = which ? dwk[i][m] : dwq[i][m];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.K; c += kThreads) {
      float s = 0.0f;
      for (int g = 0; g < kGroups; ++g) s += part[g * p.K + c];
      p.part[(static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * p.K + c] = s;
    }
  }
}

// The weights' gradients: the workgroups' sums, 16 columns a workgroup, a column by 64 threads whose parts LDS adds in order.  (A
// wave a column, which reads a line for every value: 7.5 us for 1024 parts of 2 x 128 columns.)
constexpr int kSumColumns = 16, kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void qk_norm_sum_kernel(QkArgs p, int parts) {
  constexpr int kRows = kSumThreads / kSumColumns;
  __shared__ float sums[kRows][kSumColumns];
  const int which = blockIdx.y, row = threadIdx.x / kSumColumns, c16 = threadIdx.x % kSumColumns;
  const int c = blockIdx.x * kSumColumns + c16;
  float* out = which ? p.dkw : p.dqw;
  if (!out) return;
  const float* from = p.part + static_cast<int64_t>(which) * parts * p.K + (c < p.K ? c : p.K - 1);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kParts / kRows; ++i) {
    const int at = row + i * kRows;
    const float x = from[static_cast<int64_t>(at < parts ? at : parts - 1) * p.K];
    s += at < parts ? x : 0.0f;
  }
  sums[row][c16] = s;
  __syncthreads();
  if (row || c >= p.K) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) s += sums[i][c16];
  out[c] = s;
}

int groups_of(const QkArgs& a) {
  if (!a.vec) return kThreads / 64;
  const int lanes = a.K <= 64 ? 8 : a.K <= 128 ? 16 : 32;
  return kThreads / lanes;
}

template <typename ACT, bool BWD>
void launch_t(const QkArgs& a, dim3 grid, hipStream_t s) {
  auto go = [&](auto g, auto ni, auto vec) {
    constexpr int G = decltype(g)::value, NI = decltype(ni)::value;
    constexpr bool VEC = decltype(vec)::value;
    if constexpr (BWD) hipLaunchKernelGGL((qk_norm_bwd_kernel<ACT, G, NI, VEC>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((qk_norm_kernel<ACT, G, NI, VEC>), grid, dim3(kThreads), 0, s, a);
  };
  constexpr std::integral_constant<int, 64> wave;
  constexpr std::integral_constant<int, 1> one;
  if (a.vec) {
    if (a.K <= 64) go(std::integral_constant<int, 8>{}, one, std::true_type{});
    else if (a.K <= 128) go(std::integral_constant<int, 16>{}, one, std::true_type{});
    else go(std::integral_constant<int, 32>{}, one, std::true_type{});
    return;
  }
  const int items = a.K - a.rotary / 2;
  if (items <= 64) go(wave, one, std::false_type{});
  else if (items <= 128) go(wave, std::integral_constant<int, 2>{}, std::false_type{});
  else go(wave, std::integral_constant<int, 4>{}, std::false_type{});
}

// Groups of lanes for a token's heads, and workgroups.  A group's angles cost more than a row, so it takes as many heads as leave
// enough groups: 16384 x 40 heads of 128, rotated, gradient: 120 us with 2 groups a token, 124 with one, 127 with 5, 135 with
// 10.  (Twice the workgroups: 6 % more; half: 25 %.)
dim3 plan(QkArgs* a, int64_t most) {
  const int64_t tokens = a->batch * a->L;
  const int heads = a->Hq + a->Hk, groups = groups_of(*a);
  const int64_t wanted = (32768 + tokens - 1) / tokens;
  const int split = static_cast<int>(wanted < heads ? wanted : heads);
  a->split = split;
  const int64_t blocks = (tokens * split + groups - 1) / groups;
  return dim3(static_cast<unsigned>(blocks < most ? blocks : most));
}

}  // namespace

int qk_norm_parts() { return kParts; }

hipError_t launch_qk_norm(const QkArgs& args, Dt dt, hipStream_t s) {
  QkArgs a = args;
  const dim3 grid = plan(&a, 8192);
  if (dt == Dt::BF16) launch_t<ActBF16, false>(a, grid, s);
  else launch_t<ActF32, false>(a, grid, s);
  return hipGetLastError();
}

hipError_t launch_qk_norm_bwd(const QkArgs& args, Dt dt, hipStream_t s) {
  QkArgs a = args;
  const dim3 grid = plan(&a, a.dqw || a.dkw ? kParts : 8192);
  if (dt == Dt::BF16) launch_t<ActBF16, true>(a, grid, s);
  else launch_t<ActF32, true>(a, grid, s);
  if (a.dqw || a.dkw)
    hipLaunchKernelGGL(qk_norm_sum_kernel, dim3((a.K + kSumColumns - 1) / kSumColumns, 2), dim3(kSumThreads), 0, s, a,
                       static_cast<int>(grid.x));
  return hipGetLastError();
}

}  // namespace ssm
