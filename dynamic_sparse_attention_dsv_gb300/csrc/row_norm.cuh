// What the row norms' forward and backward share: their arguments, how rows
// are laid over threads, and how the rows are split over the GPU.
#pragma once
#include <algorithm>

#include "rows.cuh"

namespace dsv {

struct NormParams {
  const void *weight, *bias;
  int32_t type;
  int64_t wb, wh, bb, bh;      // element strides, 0 where shared
  float base;
};

// How a launch lays rows over threads: a lane holds K chunks of eight channels;
// L lanes hold a row (L <= 32), or `warps` warps of 32 do.
struct NormShape {
  int L, K, warps;
  bool vec;
};

inline NormShape norm_shape(int64_t D, bool vec) {
  NormShape s;
  s.vec = vec;
  s.K = vec || D > 256 ? 2 : 1;
  s.L = !vec || D > 256 ? 32 : D > 128 ? 16 : D > 64 ? 8 : 4;
  s.warps = D > 512 ? (int)((D + 511) / 512) : 1;
  return s;
}

constexpr int kMostThreads = 512;

inline int norm_threads(const NormShape& s) {
  return s.warps == 1 ? kMostThreads / 2 : kMostThreads / 32 / s.warps * s.warps * 32;
}
inline int norm_rows(const NormShape& s) {
  return s.warps == 1 ? norm_threads(s) / s.L : norm_threads(s) / 32 / s.warps;
}
inline NormParams norm_params(const dsv_norm_params& p) {
  NormParams q;
  q.weight = p.weight;
  q.bias = p.bias;
  q.type = p.type;
  q.wb = p.per_batch ? p.weight_b : 0;
  q.wh = p.per_head ? p.weight_h : 0;
  q.bb = p.per_batch ? p.bias_b : 0;
  q.bh = p.per_head ? p.bias_h : 0;
  q.base = p.base;
  return q;
}

dsv_status validate_norm_params(const dsv_norm_params& p);

// Type of dx: x's, or dy's where x is an 8-bit checkpoint.
template <class XT, class YT>
struct DxType {
  using type = XT;
};
template <class YT>
struct DxType<Packed, YT> {
  using type = YT;
};

// A thread's place: which of its block's rows it works on, and which channels.
template <int L, int K, bool VEC, bool BLOCK>
struct Place {
  int lane, row, wr, warps, first;       // wr: warp within the row
  __device__ __forceinline__ Place(int warps_) : warps(warps_) {
    lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    row = BLOCK ? warp / warps : threadIdx.x / L;
    wr = BLOCK ? warp - row * warps : 0;
    first = (VEC ? (lane & (L - 1)) * 8 : lane) + (BLOCK ? wr * 256 : 0);
  }
  // channel 0 of chunk k
  __device__ __forceinline__ int col(int k) const { return first + k * (BLOCK ? warps * 256 : VEC ? L * 8 : 256); }
  __device__ __forceinline__ bool leads() const { return BLOCK ? wr == 0 && lane == 0 : (lane & (L - 1)) == 0; }
};

// Parameters of a lane's channels of one chunk (channels past D: 0).
template <bool VEC>
__device__ __forceinline__ void load_params(const void* p, int type, int64_t at, float base, int col, int D,
                                            float2 f[4]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = VEC ? col + e : col + e * 32;
    const float v = c < D ? base + load_param(p, type, at + c) : 0.f;
    if (e & 1) f[e / 2].y = v; else f[e / 2].x = v;
  }
}

// Sum over a row's threads. With BLOCK the row spans several warps: each warp's
// sums pass through shared memory, in two buffers used in turn, so one barrier
// of the row's warps a sum is enough (a buffer is written again only after the
// next sum's barrier, before which its readers are done). The buffers start as
// zeros, so sums are read four at a time whatever the number of warps.
template <int N>
struct alignas(16) RowBuf {
  float v[2][N][16];
};
template <int L, bool BLOCK, int N, class P>
__device__ __forceinline__ void row_sums(float (&v)[N], RowBuf<N>* bufs, int& turn, const P& at) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_sum<L>(v[i]);
  if (BLOCK) {
    float(*buf)[16] = bufs[at.row].v[turn];
    turn ^= 1;
    if (at.lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[i][at.wr] = v[i];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(at.row + 1), "r"(at.warps * 32) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = 0.f;
      for (int j = 0; j < at.warps; j += 4) {
        const float4 p = *reinterpret_cast<const float4*>(&buf[i][j]);
        t += (p.x + p.y) + (p.z + p.w);
      }
      v[i] = t;
    }
  }
}
template <int N>
__device__ __forceinline__ void clear_bufs(RowBuf<N>* bufs, int count) {
  float* p = &bufs[0].v[0][0][0];
  for (int i = threadIdx.x; i < count * (int)(sizeof(RowBuf<N>) / 4); i += blockDim.x) p[i] = 0.f;
  __syncthreads();
}

// 1 / sqrt(v) for v > 0: the approximation and one Newton step
// r + r (1 - v r^2) / 2, to about one unit in the last place.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return v < 3.0e38f ? fmaf(r * 0.5f, fmaf(-v * r, r, 1.f), r) : r;
}

}  // namespace dsv
