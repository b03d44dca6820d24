// What the row norms' forward and backward share: their arguments, how rows
// are laid over threads, and the choice of the kernel.
#pragma once
#include "rows.cuh"

namespace dsv {

struct NormParams {
  const void *weight, *bias;
  int32_t type;
  int64_t wb, wh, bb, bh;      // element strides, 0 where shared
  float base;
};

// How a launch lays rows over threads. L lanes hold one row (8, 16: up to 64,
// 128 channels, eight a lane; 32: a warp or, with `block`, every warp of the
// block), K chunks of 256 channels per warp.
struct NormShape {
  int L, K;
  bool vec, block;
  int threads;
};

constexpr int kNormThreads = 256;

inline NormShape norm_shape(int64_t D, bool vec) {
  NormShape s;
  s.vec = vec;
  s.block = false;
  s.threads = kNormThreads;
  s.K = 1;
  s.L = 32;
  if (vec && D <= 64) {
    s.L = 8;
  } else if (vec && D <= 128) {
    s.L = 16;
  } else if (D > 512) {
    s.block = true;
    s.K = 2;
    s.threads = 32 * (int)((D + 511) / 512);
  } else if (D > 256) {
    s.K = 2;
  }
  return s;
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

// First of a lane's eight channels in chunk k, and the distance between them.
template <int L, bool VEC, bool BLOCK>
__device__ __forceinline__ int norm_col(int k, int lane, int warp, int nwarps) {
  const int chunk = BLOCK ? k * nwarps + warp : k;
  return chunk * 256 + (VEC ? (lane & (L - 1)) * 8 : lane);
}

// Parameters of a lane's channels of one chunk (channels past D: 0).
template <bool VEC>
__device__ __forceinline__ void load_params(const void* p, int type, int64_t at, float base, int col, int D,
                                            float f[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = VEC ? col + e : col + e * 32;
    f[e] = c < D ? base + load_param(p, type, at + c) : 0.f;
  }
}

// Sum over a row's threads. With BLOCK the row spans the block: each warp's
// sums pass through shared memory, in two buffers used in turn, so one barrier
// a sum is enough (a buffer is written again only after the next sum's barrier,
// before which its readers are done).
template <int L, bool BLOCK, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*bufs)[32][N], int& turn, int lane, int warp,
                                         int nwarps) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_sum<L>(v[i]);
  if (BLOCK) {
    float(*buf)[N] = bufs[turn];
    turn ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[warp][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<32>(lane < nwarps ? buf[lane][i] : 0.f);
  }
}

}  // namespace dsv
