// What the row norms' forward and backward share: their arguments, how rows
// are laid over threads, and how the rows are split over the GPU.
#pragma once
#include <algorithm>
#include <atomic>

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

inline NormShape norm_shape(int64_t D, bool vec, int k_vec) {
  NormShape s;
  s.vec = vec;
  s.K = D > 256 ? 2 : vec ? k_vec : 1;
  s.L = !vec || D > 256 ? 32 : D > 128 ? 32 / s.K : D > 64 ? 16 / s.K : 8 / s.K;
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
  static constexpr int kLanes = L;
  int lane, in_row, row, wr, warps, first;       // in_row: lane among the L of its row; wr: warp within the row
  __device__ __forceinline__ Place(int warps_) : warps(warps_) {
    lane = threadIdx.x & 31;
    in_row = lane & (L - 1);
    const int warp = threadIdx.x >> 5;
    row = BLOCK ? warp / warps : threadIdx.x / L;
    wr = BLOCK ? warp - row * warps : 0;
    first = (VEC ? in_row * 8 : lane) + (BLOCK ? wr * 256 : 0);
  }
  // channel 0 of chunk k
  __device__ __forceinline__ int col(int k) const { return first + k * (BLOCK ? warps * 256 : VEC ? L * 8 : 256); }
  __device__ __forceinline__ bool leads() const { return BLOCK ? wr == 0 && lane == 0 : in_row == 0; }
};

// A tensor's rows on their way to the lanes that hold them. Rows that take
// vector loads pass through a ring of NS rows a lane in shared memory, filled by
// asynchronous copies NS - 1 rows ahead: far more bytes in flight than
// registers hold. A lane copies its own channels and reads only
// those, so a wait of its own is all the synchronisation there is. Other rows
// are loaded one row ahead into registers.

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {   // zeros where not in
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <class T, int K, bool VEC, int NS>
struct Feed {   // vector rows of a plain type
  static constexpr int kAhead = NS - 1;
  static constexpr int kPieces = sizeof(T) / 2;                 // 16-byte copies a chunk
  static __host__ __device__ constexpr uint32_t bytes(uint32_t threads) { return NS * K * kPieces * 16 * threads; }
  char* mine;
  uint32_t pitch;
  __device__ __forceinline__ Feed(char* smem) : mine(smem + threadIdx.x * 16), pitch(blockDim.x * 16) {}
  // One sweep of 16 bytes a lane for 16-bit types, two for fp32: each sweep is
  // one run both in memory and in the ring (a sweep of every other 16 bytes, or
  // one scattered in the ring, reads each 32-byte sector twice), so an fp32
  // lane's 32 bytes are copied by two of its neighbours.
  template <class P>
  __device__ __forceinline__ void issue(int slot, const T* row, const T* base, const uint8_t*, const P& at, int D) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int col = kPieces == 1 ? at.col(k) : at.col(k) + (p * P::kLanes - at.in_row) * 4;
        const bool in = col < D;
        copy16(smem_u32(mine + ((slot * K + k) * kPieces + p) * pitch), in ? row + col : base, in);
      }
  }
  template <class P>
  __device__ __forceinline__ void take(int slot, float2 (&f)[K][4], const P& at) {
    if (kPieces > 1) __syncwarp();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Raw8<T> raw;
      const char* from = mine + (slot * K + k) * kPieces * pitch;
      if (kPieces > 1)   // pieces 2 in_row and the next, of the two sweeps
        from += 2 * at.in_row >= P::kLanes ? pitch + (at.in_row - P::kLanes) * 16 : at.in_row * 16;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) raw.v[p] = *reinterpret_cast<const uint4*>(from + p * 16);
      raw.to(f[k]);
    }
  }
  template <class P>
  __device__ __forceinline__ void peek(const uint8_t*, const P&, int) {}
};
template <int K, int NS>
struct Feed<Packed, K, true, NS> {
  static constexpr int kAhead = NS - 1;
  static __host__ __device__ constexpr uint32_t bytes(uint32_t threads) { return NS * K * 8 * threads; }
  char* mine;
  uint32_t pitch, ex[K];
  __device__ __forceinline__ Feed(char* smem) : mine(smem + threadIdx.x * 8), pitch(blockDim.x * 8) {}
  template <class P>
  __device__ __forceinline__ void issue(int slot, const int8_t* row, const int8_t* base, const uint8_t*, const P& at, int D) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = at.col(k) < D;
      copy8(smem_u32(mine + (slot * K + k) * pitch), in ? row + at.col(k) : base, in);
    }
  }
  // the exponents, one row ahead in registers
  template <class P>
  __device__ __forceinline__ void peek(const uint8_t* exps, const P& at, int D) {
#pragma unroll
    for (int k = 0; k < K; ++k) ex[k] = at.col(k) < D ? __ldg(exps + (at.col(k) >> 5)) : 7u;
  }
  template <class P>
  __device__ __forceinline__ void take(int slot, float2 (&f)[K][4], const P&) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Chunk<Packed, true> ch;
      ch.w = *reinterpret_cast<const uint2*>(mine + (slot * K + k) * pitch);
      ch.ex = ex[k];
      ch.to(f[k]);
    }
  }
};
template <class T, int K, bool VEC>
struct Feed<T, K, VEC, 1> {
  static constexpr int kAhead = 1;
  static __host__ __device__ constexpr uint32_t bytes(uint32_t) { return 0; }
  Chunk<T, VEC> ch[K];
  __device__ __forceinline__ Feed(char*) {}
  template <class P, class E>
  __device__ __forceinline__ void issue(int, const E* row, const E*, const uint8_t* exps, const P& at, int D) {
#pragma unroll
    for (int k = 0; k < K; ++k) ch[k].load(row, exps, at.col(k), D);
  }
  template <class P>
  __device__ __forceinline__ void peek(const uint8_t*, const P&, int) {}
  template <class P>
  __device__ __forceinline__ void take(int, float2 (&f)[K][4], const P&) {
#pragma unroll
    for (int k = 0; k < K; ++k) ch[k].to(f[k]);
  }
};
template <int K>
struct Feed<Packed, K, true, 1> {
  static constexpr int kAhead = 1;
  static __host__ __device__ constexpr uint32_t bytes(uint32_t) { return 0; }
  Chunk<Packed, true> ch[K];
  __device__ __forceinline__ Feed(char*) {}
  template <class P, class E>
  __device__ __forceinline__ void issue(int, const E* row, const E*, const uint8_t* exps, const P& at, int D) {
#pragma unroll
    for (int k = 0; k < K; ++k) ch[k].load(row, exps, at.col(k), D);
  }
  template <class P>
  __device__ __forceinline__ void peek(const uint8_t*, const P&, int) {}
  template <class P>
  __device__ __forceinline__ void take(int, float2 (&f)[K][4], const P&) {
#pragma unroll
    for (int k = 0; k < K; ++k) ch[k].to(f[k]);
  }
};

// Opts a kernel into `bytes` of dynamic shared memory, once per device.
template <class F>
inline cudaError_t allow_smem(F* kernel, uint32_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t s = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (s == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return s;
}

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
