// Tiles of tokens and matrix operands, shared by the kernels that walk a sequence in chunks (linear attention
// and the gated delta rule): operands of the matrix instructions for both activation types, the swizzled LDS
// tiles that they come from, and loads from memory straight into those.
#pragma once

#include "device_common.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kQ = 64;               // tokens per chunk

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// Place of byte `byte` of a row in an LDS tile of RB-byte rows: row RB + (byte ^ 16 swizzle(row)).
// Rows are packed (the loads into LDS leave no room for padding); the 16-byte slots of a
// row are exchanged by the bits of its number so that the rows one read touches at a time lie
// in different banks: 16 consecutive rows and (PERM) the rows {0..3, 8..11, 16..19, 24..27} of the permuted
// tiles at 16 bytes a lane (in whose phases lanes 4..11 of a 16-lane group go with the
// others of the next group, one slot on), and two neighbouring slots of rows {0..3, 8..11}
// (the transposing reads).  It is linear in the row's bits, so an address is one lane
// part, exclusive-or'ed with constants, plus a constant offset.
template <int RB, bool F32, bool PERM>
__device__ __forceinline__ constexpr int swizzle(int row) {
  const int b0 = row & 1, b1 = (row >> 1) & 1, b2 = (row >> 2) & 1, b3 = (row >> 3) & 1,
            b4 = PERM ? (row >> 4) & 1 : 0;
  if (F32) return b1 | (b0 << 1) | ((b2 ^ b4) << 2) | (b3 << 3);
  if (RB == 128) return (b2 ^ b4) | (b1 << 1) | ((b2 ^ b3 ^ b4) << 2);
  return (b2 ^ b4) | (b0 << 1) | (b1 << 2) | ((b2 ^ b3 ^ b4) << 3);
}
typedef __attribute__((address_space(3))) char lds_char_t;
__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char_t*)(p)));
}
template <typename V>
__device__ __forceinline__ V lds_read(uint32_t at) {
  return *(const __attribute__((address_space(3))) V*)(static_cast<uintptr_t>(at));
}
template <typename V>
__device__ __forceinline__ void lds_write(uint32_t at, const V& v) {
  *(__attribute__((address_space(3))) V*)(static_cast<uintptr_t>(at)) = v;
}

// ---- eight values of one lane: a matrix operand (one v_mfma_f32_16x16x32_bf16, lane
// (g, c) holding row/column c and summation indices 8g..8g+7; or eight
// v_mfma_f32_16x16x4_f32, lane group g holding index g of each)
template <typename ACT>
struct Op;

template <>
struct Op<ActBF16> {
  using elem = uint16_t;
  using piece = uint4;
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
      if (t + 1 < TERMS) {                          // r - p, exact: one dot product of p's pair with (-1, 0) or (0, -1)
        const uint32_t pw[4] = {p[t].x, p[t].y, p[t].z, p[t].w};
        uint32_t low = 0x0000bf80u, high = 0xbf800000u;
        asm("" : "+s"(low), "+s"(high));            // (scalar registers: the immediate -1.0 is the high half alone)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          r[e] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, pw[e / 2]),
                                                 __builtin_bit_cast(bf16x2_t, e % 2 ? high : low), r[e], false);
      }
    }
  }
  // the same for 4 values, into one half of each operand
  template <int TERMS>
  static __device__ __forceinline__ void split4(const float (&v)[4], uint2 (&p)[TERMS]) {
    const float x[8] = {v[0], v[1], v[2], v[3], 0.0f, 0.0f, 0.0f, 0.0f};
    piece full[TERMS];
    split<TERMS>(x, full);
#pragma unroll
    for (int t = 0; t < TERMS; ++t) p[t] = make_uint2(full[t].x, full[t].y);
  }
  using half = uint2;
  static __device__ __forceinline__ void put_half(uint32_t at, const half& p) {
    lds_write<u32x2_t>(at, __builtin_bit_cast(u32x2_t, p));
  }
  static constexpr int kPiece = 16;                 // bytes of 8 elements
  // A lane's part of the address of columns 8g.. of row `row`, and the 8 columns at it.
  template <int RB, bool PERM>
  static __device__ __forceinline__ uint32_t row_part(uint32_t tile, int row, int g) {
    return tile + row * RB + ((16 * g) ^ (swizzle<RB, false, PERM>(row) << 4));
  }
  static __device__ __forceinline__ piece row(uint32_t at, int flip, int offset) {
    return __builtin_bit_cast(piece, lds_read<u32x4_t>((at ^ flip) + offset));
  }
  static __device__ __forceinline__ void put(uint32_t at, int flip, int offset, const piece& p) {
    lds_write<u32x4_t>((at ^ flip) + offset, __builtin_bit_cast(u32x4_t, p));
  }
  // Values [8g + e][col(c)], e = 0..7, col(c) = col0 + step (c / 4) + c % 4: two
  // transposing reads of 4 rows each.  Lane i of a 16-lane group gives the address of 4
  // columns (piece i % 4) of row i / 4 and receives column i of the 4 rows.
  template <int RB, bool PERM>
  static __device__ __forceinline__ uint32_t column_part(uint32_t tile, int col0, int step, int lane) {
    const int row = 8 * (lane >> 4) + ((lane & 15) >> 2);
    return tile + row * RB + ((2 * (col0 + step * (lane & 3))) ^ (swizzle<RB, false, PERM>(row) << 4));
  }
  template <int RB, bool PERM>
  static __device__ __forceinline__ piece column(uint32_t at, int flip, int offset) {
    const uint32_t a = (at ^ flip) + offset, b = (at ^ flip ^ (swizzle<RB, false, PERM>(4) << 4)) + offset + 4 * RB;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(static_cast<uintptr_t>(a)));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(static_cast<uintptr_t>(b)));
    const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
    return make_uint4(l.x, l.y, h.x, h.y);
  }
  // The next 4 columns of a piece (u = 1): one half of a slot on.
  static __device__ __forceinline__ constexpr int half_flip(int) { return 0; }
  static __device__ __forceinline__ constexpr int half_offset(int u) { return 8 * u; }
};

struct F8 {
  float4 a, b;
};

template <>
struct Op<ActF32> {
  using elem = float;
  using piece = F8;
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
  template <int TERMS>
  static __device__ __forceinline__ void split4(const float (&v)[4], float4 (&p)[TERMS]) {
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
  }
  using half = float4;
  static __device__ __forceinline__ void put_half(uint32_t at, const half& p) {
    lds_write<f32x4_t>(at, __builtin_bit_cast(f32x4_t, p));
  }
  static constexpr int kPiece = 32;
  template <int RB, bool PERM>
  static __device__ __forceinline__ uint32_t row_part(uint32_t tile, int row, int g) {
    return tile + row * RB + ((32 * g) ^ (swizzle<RB, true, PERM>(row) << 4));
  }
  static __device__ __forceinline__ piece row(uint32_t at, int flip, int offset) {
    return F8{__builtin_bit_cast(float4, lds_read<f32x4_t>((at ^ flip) + offset)),
              __builtin_bit_cast(float4, lds_read<f32x4_t>((at ^ flip ^ 16) + offset))};
  }
  static __device__ __forceinline__ void put(uint32_t at, int flip, int offset, const piece& p) {
    lds_write<f32x4_t>((at ^ flip) + offset, __builtin_bit_cast(f32x4_t, p.a));
    lds_write<f32x4_t>((at ^ flip ^ 16) + offset, __builtin_bit_cast(f32x4_t, p.b));
  }
  template <int RB, bool PERM>
  static __device__ __forceinline__ uint32_t column_part(uint32_t tile, int col0, int step, int lane) {
    const int row = 8 * (lane >> 4);
    return tile + row * RB + ((4 * (col0 + step * ((lane & 15) >> 2) + (lane & 3))) ^ (swizzle<RB, true, PERM>(row) << 4));
  }
  template <int RB, bool PERM>
  static __device__ __forceinline__ piece column(uint32_t at, int flip, int offset) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = lds_read<float>((at ^ flip ^ (swizzle<RB, true, PERM>(e) << 4)) + offset + e * RB);
    return pack(v);
  }
  static __device__ __forceinline__ constexpr int half_flip(int u) { return 16 * u; }
  static __device__ __forceinline__ constexpr int half_offset(int) { return 0; }
};

__device__ __forceinline__ int least(int a, int b) { return a < b ? a : b; }
__device__ __forceinline__ int lane_id() { return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)); }

// A value that is the same in every lane, kept in a scalar register.
__device__ __forceinline__ float uniform_float(float v) {
  return __builtin_bit_cast(float, uniform_int(__builtin_bit_cast(int, v)));
}

// The load is written out (it has no result register; M0 holds the wave's LDS address, lane
// l's 16 bytes go to M0 + 16 l): the compiler would wait for a load into one buffer of k
// before reading the other.  Whoever reads the tile waits first (vmcnt(0), then a barrier).
// (5 wait states lie between a vector write of an address's scalar register and its use.  The
// compiler has M0 reserved, and nothing else in these kernels uses it.)
__device__ __forceinline__ void load_to_lds(uint32_t tile, const char* base, uint32_t off) {
  const int m0 = uniform_int(static_cast<int>(tile));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(m0), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void load_to_lds(uint32_t tile, const char* src) {
  const int m0 = uniform_int(static_cast<int>(tile));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(m0), "v"(src) : "memory");
}
// (4 bytes a lane, to M0 + 4 l)
__device__ __forceinline__ void load_word_to_lds(uint32_t tile, const char* src) {
  const int m0 = uniform_int(static_cast<int>(tile));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off"
               :: "s"(m0), "v"(src) : "memory");
}
// ... from a uniform address and the lane's offset
__device__ __forceinline__ void load_word_to_lds(uint32_t tile, const char* src, uint32_t off) {
  const int m0 = uniform_int(static_cast<int>(tile));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2"
               :: "s"(m0), "v"(off), "s"(src) : "memory");
}

// Clears rows n.. of the slots that this wave's loads filled.
template <int RB, int NW>
__device__ __forceinline__ void clear_tile(char* tile, int n, int w, int lane) {
  constexpr int kSlots = RB / 16, kInstr = kQ * RB / 1024 / NW;
#pragma unroll 1
  for (int i = 0; i < kInstr; ++i) {
    const int s = (w * kInstr + i) * 64 + lane;
    if (s / kSlots >= n) *reinterpret_cast<uint4*>(tile + s * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace
}  // namespace ssm
