// What the gated delta rule's kernels share: a chunk's record (T in operand order and the chunk's vectors), sums of
// logarithms as pairs, and products of values in several terms.
#pragma once

#include "device_common.hpp"
#include "la_tiles.hpp"

namespace ssm {
namespace {

constexpr int kT = 6;                     // operands of T (and of the scores): 16 rows by 32 tokens, where it is not zero
constexpr int kVecs = 8;                  // vectors of 64 floats in a chunk's record
// exp(G), exp(G_Q - G), beta, G in two parts, exp(G_Q); in every entry the first token whose row of A is not finite, or 64 (outputs'
// records; exp(G_Q) is NaN there); in the gradient's records what gd_grad.hip needs for g: the chunk's pace in the first entry, in
// the second the sum of what its tokens have from before it, in the third, of a stretch's last chunk, <F, E> behind it
enum { kInto = 0, kLast, kBeta, kSumHi, kSumLo, kWhole, kFirstOdd, kPace };
// A chunk's pace: every decay at least 2^kFastGate; or one is less, and exp(G_Q) below `nothing` (what passes through the whole chunk
// is too little to be seen in a gradient) or above.
enum { kSlow = 0, kFast, kFastThrough };
constexpr double kFastGate = -1.25, kStrongGate = -3.0;
__device__ __forceinline__ float nothing(bool strong) { return strong ? 0x1p-48f : 0x1p-32f; }   // a decay is below 2^kStrongGate
// The least logarithm of a decay (of base 2): 2^kMinGate is 0 in float32.  No lower, as the sum over a chunk with many decays
// of 0 has to stay small for exp2_pair.
constexpr double kMinGate = -160.0;

template <typename ACT>
constexpr int kTerms = ACT::kBytes == 2 ? 3 : 1;       // operand terms of what the state depends on
template <typename ACT>
constexpr int kOutTerms = ACT::kBytes == 2 ? 2 : 1;    // ... and of what outputs alone do
template <typename ACT>
constexpr int kPieceBytes = ACT::kBytes == 2 ? 1024 : 2048;   // an operand of 64 lanes
template <typename ACT>
constexpr int kTBytes = kT * kTerms<ACT> * kPieceBytes<ACT>;
template <typename ACT, int PT>
constexpr int kRecord = kTBytes<ACT> + kVecs * 256 + kT * PT * kPieceBytes<ACT>;   // a chunk's T, vectors and scores in PT terms

// 2^(hi + lo), of first order in lo: the sum of logarithms is kept as a float32 pair, so that a factor exp(G_i - G_j) is as
// good as float32 where the sums themselves are in the thousands.  With a decay of 0 at every other token of a chunk they reach
// 32 x 160 < 2^13, where a difference's lo is up to 2^-11 and what is left out (lo log 2)^2 / 2 = 2^-24.
__device__ __forceinline__ float exp2_pair(float hi, float lo) {
  const float e = exp2_hw(hi);
  return __builtin_fmaf(e, lo * kLn2, e);
}

__device__ __forceinline__ int gd_length(const int32_t* lengths, int L, int64_t b) {
  if (!lengths) return L;
  const int n = uniform_int(lengths[b]);
  return n < 0 ? 0 : (n > L ? L : n);
}

__device__ __forceinline__ void store_piece(char* at, const uint4& p) { *reinterpret_cast<uint4*>(at) = p; }
__device__ __forceinline__ void store_piece(char* at, const F8& p) {
  reinterpret_cast<float4*>(at)[0] = p.a;
  reinterpret_cast<float4*>(at)[1] = p.b;
}
__device__ __forceinline__ void load_piece(const char* at, uint4& p) { p = *reinterpret_cast<const uint4*>(at); }
__device__ __forceinline__ void load_piece(const char* at, F8& p) {
  p.a = reinterpret_cast<const float4*>(at)[0];
  p.b = reinterpret_cast<const float4*>(at)[1];
}

// ... from 4-byte words (the hardware's loads of 16 bytes need no more)
typedef uint32_t words_t __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void load_words(const char* at, uint4& p) {
  const words_t x = *reinterpret_cast<const words_t*>(at);
  p = make_uint4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void load_words(const char* at, F8& p) {
  p.a = __builtin_bit_cast(float4, reinterpret_cast<const words_t*>(at)[0]);
  p.b = __builtin_bit_cast(float4, reinterpret_cast<const words_t*>(at)[1]);
}
// Elements by .. of a piece, zeros behind them (by: 0 .. 7).
__device__ __forceinline__ void drop_first(uint4& p, int by) {
  uint32_t x[5] = {p.x, p.y, p.z, p.w, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = by & 4 ? (i < 2 ? x[i + 2] : 0u) : x[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = by & 2 ? x[i + 1] : x[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = by & 1 ? x[i] >> 16 | x[i + 1] << 16 : x[i];
  p = make_uint4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void drop_first(F8& p, int by) {
  float x[8] = {p.a.x, p.a.y, p.a.z, p.a.w, p.b.x, p.b.y, p.b.z, p.b.w};
#pragma unroll
  for (int d = 4; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = by & d ? (i + d < 8 ? x[i + d < 8 ? i + d : 0] : 0.0f) : x[i];
  p.a = make_float4(x[0], x[1], x[2], x[3]);
  p.b = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace
}  // namespace ssm
