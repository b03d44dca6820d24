// Rows of width D inside strided [B][H][S][D] tensors: how kernels find a row,
// read and write its channels as floats, and quantise blocks of 32 channels.
// Shared by the row norms and the 8-bit activation checkpoints.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dsv {

constexpr int kPackBlock = 32;     // channels that share one exponent byte
constexpr int kSMs = 152;          // grids are sized for GB300's SMs
constexpr int kMaxWidth = 16384;   // D: 32 warps, two chunks of 8 channels a lane

// n / d for 0 <= n < 2^31 by a multiplication with a precomputed reciprocal
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994, figure 4.1).
struct FastDiv {
  uint32_t d, m, s;
  __host__ void set(uint32_t div) {
    d = div;
    s = 0;
    while ((uint64_t(1) << s) < div) ++s;
    m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - div)) / div + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

// One group's rows: up to three nested dimensions, outermost first, each with
// a stride for every tensor of the call (elements; the last one counts rows of
// the contiguous [B][H][S] arrays).
constexpr int kMapTensors = 4;
struct RowMap {
  int32_t nd;                        // dimensions in use, 1..3
  uint32_t n;                        // rows of a group
  FastDiv size[3];
  int64_t stride[3][kMapTensors];
  // groups (rows that share their parameters): g = gb * gh_n + gh
  FastDiv gh_n;
  int64_t gb[kMapTensors], gh[kMapTensors];
};

// Offsets of row i of a group, relative to the group's base.
__device__ __forceinline__ void row_offsets(const RowMap& m, uint32_t i, int64_t off[kMapTensors]) {
  if (m.nd == 1) {
#pragma unroll
    for (int t = 0; t < kMapTensors; ++t) off[t] = (int64_t)i * m.stride[0][t];
    return;
  }
  const uint32_t q = m.size[m.nd - 1].div(i);
  const uint32_t r = i - q * m.size[m.nd - 1].d;
  if (m.nd == 2) {
#pragma unroll
    for (int t = 0; t < kMapTensors; ++t) off[t] = (int64_t)q * m.stride[0][t] + (int64_t)r * m.stride[1][t];
    return;
  }
  const uint32_t q2 = m.size[1].div(q);
  const uint32_t r2 = q - q2 * m.size[1].d;
#pragma unroll
  for (int t = 0; t < kMapTensors; ++t)
    off[t] = (int64_t)q2 * m.stride[0][t] + (int64_t)r2 * m.stride[1][t] + (int64_t)r * m.stride[2][t];
}

__device__ __forceinline__ void group_offsets(const RowMap& m, uint32_t g, int64_t off[kMapTensors]) {
  const uint32_t gb = m.gh_n.div(g), gh = g - gb * m.gh_n.d;
#pragma unroll
  for (int t = 0; t < kMapTensors; ++t) off[t] = (int64_t)gb * m.gb[t] + (int64_t)gh * m.gh[t];
}

// ------------------------------------------------------ channels as floats
struct Packed {};   // tag: 8-bit blocks with shared exponents

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Eight channels of a row as they lie in memory (one or two 16-byte loads).
template <class T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void to(float f[8]) const;
};
template <>
__device__ __forceinline__ void Raw8<float>::to(float f[8]) const {
  memcpy(f, v, 32);
}
template <>
__device__ __forceinline__ void Raw8<__nv_bfloat16>::to(float f[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Raw8<__half>::to(float f[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 h;
    memcpy(&h, &w[i], 4);
    const float2 p = __half22float2(h);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ void store8(float* p, const float f[8]) {
  float4* o = reinterpret_cast<float4*>(p);
  o[0] = make_float4(f[0], f[1], f[2], f[3]);
  o[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float f[8]) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  uint4 w;
  memcpy(&w, h, 16);
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void store8(__half* p, const float f[8]) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  uint4 w;
  memcpy(&w, h, 16);
  *reinterpret_cast<uint4*>(p) = w;
}

// A parameter of any of the three types (read once per group of rows).
__device__ __forceinline__ float load_param(const void* p, int type, int64_t i) {
  if (type == DSV_FP32) return static_cast<const float*>(p)[i];
  if (type == DSV_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}

// ---------------------------------------------------------- 8-bit blocks
// A block's exponent byte e is the biased exponent field of its largest
// magnitude, so that magnitude lies in [64, 128) steps of 2^(e-133); below
// e = 7 the step stays at the smallest normal float, 2^-126. Infinities and
// NaN have the field 255, which marks the whole block as NaN. Both x / step
// and q * step are exact in fp32, so the rounding to q is the only one.
__device__ __forceinline__ uint32_t block_exp(uint32_t abs_bits) { return max(abs_bits >> 23, 7u); }
__device__ __forceinline__ float block_step(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7FC00000u : (e - 6u) << 23);
}
// 1 / step; 0 for a block of NaN, whose bytes mean nothing
__device__ __forceinline__ float block_inv(uint32_t e) { return __uint_as_float(e == 255u ? 0u : (260u - e) << 23); }

// x / step to the nearest integer, ties to even, in the low byte: adding
// 1.5 * 2^23 rounds at the integers. Magnitudes in (127.5, 128) steps go to 127.
__device__ __forceinline__ uint32_t quant(float x, float inv) {
  const float r = fmaf(x, inv, 12582912.0f);
  return __float_as_uint(fminf(fmaxf(r, 12582912.0f - 127.0f), 12582912.0f + 127.0f));
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four signed bytes as floats: the byte plus 128 in the low bits of 2^23.
__device__ __forceinline__ void bytes4(uint32_t w, float f[4]) {
  w ^= 0x80808080u;
  const uint32_t k = 0x4B000000u;
  f[0] = __uint_as_float(__byte_perm(w, k, 0x7440)) - 8388736.0f;
  f[1] = __uint_as_float(__byte_perm(w, k, 0x7441)) - 8388736.0f;
  f[2] = __uint_as_float(__byte_perm(w, k, 0x7442)) - 8388736.0f;
  f[3] = __uint_as_float(__byte_perm(w, k, 0x7443)) - 8388736.0f;
}

// Eight channels of one row for one lane. VEC: eight in a row, by 16-byte
// loads (8 bytes and an exponent where packed). Otherwise channel e * 32 + lane
// of the warp's 256, so that every load of the warp is one run of memory, at
// any alignment, and each e is one 32-channel block.
template <class T, bool VEC>
struct Chunk {
  Raw8<T> raw;
  __device__ __forceinline__ void load(const T* row, const uint8_t*, int col, int D) {
    if (col < D) raw.load(row + col); else raw.zero();
  }
  __device__ __forceinline__ void to(float f[8]) const { raw.to(f); }
};
template <class T>
struct Chunk<T, false> {
  T v[8];
  __device__ __forceinline__ void load(const T* row, const uint8_t*, int col, int D) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + e * 32 < D ? __ldg(row + col + e * 32) : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void to(float f[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = to_f32(v[e]);
  }
};
template <>
struct Chunk<Packed, true> {
  uint2 w;
  uint32_t ex;
  __device__ __forceinline__ void load(const int8_t* row, const uint8_t* exps, int col, int D) {
    w = make_uint2(0, 0);
    ex = 7;
    if (col < D) {
      w = __ldg(reinterpret_cast<const uint2*>(row + col));
      ex = __ldg(exps + (col >> 5));
    }
  }
  __device__ __forceinline__ void to(float f[8]) const {
    const float step = block_step(ex);
    bytes4(w.x, f);
    bytes4(w.y, f + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= step;
  }
};
template <>
struct Chunk<Packed, false> {
  float v[8];
  __device__ __forceinline__ void load(const int8_t* row, const uint8_t* exps, int col, int D) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = col + e * 32 < D ? (float)__ldg(row + col + e * 32) * block_step(__ldg(exps + ((col + e * 32) >> 5))) : 0.f;
  }
  __device__ __forceinline__ void to(float f[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[e];
  }
};

// Type of a tensor's elements in memory.
template <class T>
struct Elem {
  using type = T;
};
template <>
struct Elem<Packed> {
  using type = int8_t;
};

template <class T, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int col, int D, const float f[8]) {
  if (VEC) {
    if (col < D) store8(row + col, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e * 32 < D) row[col + e * 32] = from_f32<T>(f[e]);
  }
}

// The chunk's channels as 8-bit blocks (channels past D are zeros).
template <bool VEC>
__device__ __forceinline__ void pack_chunk(int8_t* q, uint8_t* exps, int col, int D, const float f[8]) {
  if (VEC) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t ex = block_exp(top);
    const float inv = block_inv(ex);
    if (col < D) {
      uint2 w;
      w.x = pack4(quant(f[0], inv), quant(f[1], inv), quant(f[2], inv), quant(f[3], inv));
      w.y = pack4(quant(f[4], inv), quant(f[5], inv), quant(f[6], inv), quant(f[7], inv));
      *reinterpret_cast<uint2*>(q + col) = w;
      if ((col & 31) == 0) exps[col >> 5] = (uint8_t)ex;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t ex = block_exp(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(f[e]) & 0x7FFFFFFFu));
      const int at = col + e * 32;
      if (at < D) {
        q[at] = (int8_t)(quant(f[e], block_inv(ex)) & 0xFFu);
        if ((at & 31) == 0) exps[at >> 5] = (uint8_t)ex;
      }
    }
  }
}

// Sum over the L neighbouring lanes that share a row; every lane gets it.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ------------------------------------------------------------ host helpers
inline int elem_size(int type) { return type == DSV_FP32 ? 4 : type == DSV_PACKED ? 1 : 2; }
inline bool is_plain(int type) { return type == DSV_BF16 || type == DSV_FP16 || type == DSV_FP32; }

// Extent of a call: dimensions, width, and the counts the kernels index with 32 bits.
dsv_status validate_extent(const dsv_extent& n);
// Pointers, type, strides and alignment of one tensor; an output's rows must not overlap.
dsv_status validate_rows(const dsv_rows& t, const dsv_extent& n, bool output);
// Whether rows of this tensor take 16-byte loads of eight channels (8-byte ones where packed).
bool rows_take_vectors(const dsv_rows& t, const dsv_extent& n);
// The map of a call's rows: groups over the per-parameter dimensions, the others folded where every tensor allows it.
RowMap make_row_map(const dsv_extent& n, bool per_batch, bool per_head, const dsv_rows* const* tensors, int count);

}  // namespace dsv
