// Gradients of the row norm: dx row by row, and the parameters' gradients
// summed over the rows that share them.
#include <algorithm>

#include "row_norm.cuh"

namespace dsv {

struct NormBwdArgs {
  const void *dy, *x;
  const uint8_t* xe;
  void* dx;
  const float *mean, *rstd;
  float *dw, *db;              // gradients, or the partial sums [blocks][2][D]
  NormParams p;
  float inv_d;
  int32_t D, nb;
  int32_t per_group;           // thread blocks a group
  int32_t partial;             // several blocks a group: they leave partial sums
};

// Each thread owns fixed channels, so its share of dweight and dbias stays in
// registers over all its rows; a block's shares are added in a fixed order and
// left in the workspace (or, with one block a group, written as the result).
template <class XT, class YT, int L, int K, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : kNormThreads)
    k_row_norm_bwd(const __grid_constant__ NormBwdArgs a, const __grid_constant__ RowMap m) {
  using XE = typename Elem<XT>::type;
  using DX = typename DxType<XT, YT>::type;
  constexpr int kWarps = kNormThreads / 32;
  constexpr int kCols = (L == 32 ? 256 : L * 8) * K;
  __shared__ float buf[2][32][2];
  __shared__ float sums[BLOCK ? 1 : kWarps][BLOCK ? 1 : kCols + 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const uint32_t g = blockIdx.x / a.per_group, c = blockIdx.x % a.per_group;
  const uint32_t gb = m.gh_n.div(g), gh = g - gb * m.gh_n.d;
  int64_t g0[kMapTensors];
  group_offsets(m, g, g0);

  float w[K][8], aw[K][8], ab[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[k][e] = 1.f;
      aw[k][e] = ab[k][e] = 0.f;
    }
    if (a.p.weight)
      load_params<VEC>(a.p.weight, a.p.type, gb * a.p.wb + gh * a.p.wh, a.p.base,
                       norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps), a.D, w[k]);
  }

  constexpr int kRows = BLOCK ? 1 : kNormThreads / L;
  const uint32_t slot = BLOCK ? 0 : threadIdx.x / L;
  int turn = 0;
  for (uint32_t t = c; (uint64_t)t * kRows < m.n; t += a.per_group) {
    const uint32_t i = t * kRows + slot;
    const bool live = i < m.n;
    int64_t off[kMapTensors];
    row_offsets(m, live ? i : m.n - 1, off);
    const int64_t row = g0[3] + off[3];
    const int D = live ? a.D : 0;        // a row past the last reads and adds zeros
    Chunk<YT, VEC> cy[K];
    Chunk<XT, VEC> cx[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int col = norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps);
      cy[k].load(static_cast<const YT*>(a.dy) + g0[0] + off[0], nullptr, col, D);
      cx[k].load(static_cast<const XE*>(a.x) + g0[1] + off[1], a.xe + row * a.nb, col, D);
    }
    const float mean = a.mean ? __ldg(a.mean + row) : 0.f, rstd = __ldg(a.rstd + row);
    float gy[K][8], xh[K][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int col = norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps);
      cy[k].to(gy[k]);
      cx[k].to(xh[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool in = VEC ? col < D : col + e * 32 < D;
        xh[k][e] = in ? (xh[k][e] - mean) * rstd : 0.f;
        aw[k][e] = fmaf(gy[k][e], xh[k][e], aw[k][e]);
        ab[k][e] += gy[k][e];
        gy[k][e] *= w[k][e];
        s[0] += gy[k][e];
        s[1] = fmaf(gy[k][e], xh[k][e], s[1]);
      }
    }
    row_sums<L, BLOCK, 2>(s, buf, turn, lane, warp, nwarps);
    const float c1 = a.mean ? s[0] * a.inv_d : 0.f, c2 = s[1] * a.inv_d;
    DX* dx = static_cast<DX*>(a.dx) + g0[2] + off[2];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) gy[k][e] = rstd * (gy[k][e] - fmaf(xh[k][e], c2, c1));
      store_chunk<DX, VEC>(dx, norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps), D, gy[k]);
    }
  }

  // the block's sums: lanes that hold the same channels, then the warps in order
  float* out[2];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* base = which ? a.db : a.dw;
    out[which] = !base ? nullptr : a.partial ? base + (int64_t)blockIdx.x * 2 * a.D : base + (int64_t)g * a.D;
    if (!out[which]) continue;
    float(*acc)[8] = which ? ab : aw;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = acc[k][e];
#pragma unroll
        for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        const int col = norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps) + (VEC ? e : e * 32);
        if (BLOCK) {
          if (col < a.D) out[which][col] = v;
        } else if (lane < L) {
          sums[warp][col] = v;
        }
      }
    if (!BLOCK) {
      __syncthreads();
      for (int col = threadIdx.x; col < kCols && col < a.D; col += kNormThreads) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) v += sums[j][col];
        out[which][col] = v;
      }
      __syncthreads();
    }
  }
}

// Adds a group's partial sums, 32 channels a block: thread row j takes the
// partials j, j + 8, ..., then the eight rows are added in order.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(32 * kJoinRows) k_row_norm_join(const float* __restrict__ part, int per_group, int D,
                                                                  float* dw, float* db) {
  __shared__ float sums[2][kJoinRows][32];
  const int blocks_d = (D + 31) / 32;
  const uint32_t g = blockIdx.x / blocks_d;
  const int col = (blockIdx.x % blocks_d) * 32 + threadIdx.x;
  float v[2] = {0.f, 0.f};
  if (col < D)
    for (int j = threadIdx.y; j < per_group; j += kJoinRows) {
      const float* p = part + ((int64_t)g * per_group + j) * 2 * D + col;
      v[0] += p[0];
      v[1] += p[D];
    }
  sums[0][threadIdx.y][threadIdx.x] = v[0];
  sums[1][threadIdx.y][threadIdx.x] = v[1];
  __syncthreads();
  if (threadIdx.y < 2 && col < D) {
    float* out = threadIdx.y ? db : dw;
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < kJoinRows; ++j) t += sums[threadIdx.y][j][threadIdx.x];
    if (out) out[(int64_t)g * D + col] = t;
  }
}

// Blocks of a group: enough to fill the GPU once, at most one per tile of rows.
static int64_t bwd_per_group(int64_t D, int64_t rows, int64_t groups, bool vec) {
  const NormShape s = norm_shape(D, vec);
  const int rows_block = s.block ? 1 : kNormThreads / s.L;
  const int64_t tiles = (rows + rows_block - 1) / rows_block;
  const int64_t want = (int64_t)kSMs * 2 * std::max(1, 512 / s.threads);
  return std::max<int64_t>(1, std::min<int64_t>(tiles, want / std::max<int64_t>(groups, 1)));
}

template <class XT, class YT>
static void dispatch(const NormShape& s, const NormBwdArgs& a, const RowMap& m, uint32_t grid, cudaStream_t st) {
  if (s.vec && s.L == 8) k_row_norm_bwd<XT, YT, 8, 1, true, false><<<grid, s.threads, 0, st>>>(a, m);
  else if (s.vec && s.L == 16) k_row_norm_bwd<XT, YT, 16, 1, true, false><<<grid, s.threads, 0, st>>>(a, m);
  else if (s.block && s.vec) k_row_norm_bwd<XT, YT, 32, 2, true, true><<<grid, s.threads, 0, st>>>(a, m);
  else if (s.block) k_row_norm_bwd<XT, YT, 32, 2, false, true><<<grid, s.threads, 0, st>>>(a, m);
  else if (s.K == 2 && s.vec) k_row_norm_bwd<XT, YT, 32, 2, true, false><<<grid, s.threads, 0, st>>>(a, m);
  else if (s.K == 2) k_row_norm_bwd<XT, YT, 32, 2, false, false><<<grid, s.threads, 0, st>>>(a, m);
  else if (s.vec) k_row_norm_bwd<XT, YT, 32, 1, true, false><<<grid, s.threads, 0, st>>>(a, m);
  else k_row_norm_bwd<XT, YT, 32, 1, false, false><<<grid, s.threads, 0, st>>>(a, m);
}

}  // namespace dsv

using namespace dsv;

static int64_t norm_groups(const dsv_extent& n, bool per_batch, bool per_head) {
  return (per_batch ? n.B : 1) * (per_head ? n.H : 1);
}

extern "C" size_t dsv_layer_norm_bwd_workspace_size(dsv_extent n, int32_t per_batch, int32_t per_head) {
  if (validate_extent(n) != DSV_OK) return 0;
  const int64_t rows = n.B * n.H * n.S, groups = norm_groups(n, per_batch != 0, per_head != 0);
  if (rows == 0) return 0;
  // whether the rows take vector loads is only known to the call: the larger of the two plans
  const int64_t per = std::max(bwd_per_group(n.D, rows / groups, groups, true),
                               bwd_per_group(n.D, rows / groups, groups, false));
  return per == 1 ? 0 : (size_t)groups * per * 2 * n.D * sizeof(float);
}

extern "C" dsv_status dsv_layer_norm_bwd(dsv_rows dy, dsv_rows x, dsv_extent n, dsv_norm_params params,
                                         const float* mean, const float* rstd, dsv_rows dx, float* dweight,
                                         float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  dsv_status v = validate_extent(n);
  if (v != DSV_OK) return v;
  if ((v = validate_rows(dy, n, false)) != DSV_OK || (v = validate_rows(x, n, false)) != DSV_OK ||
      (v = validate_rows(dx, n, true)) != DSV_OK || (v = validate_norm_params(params)) != DSV_OK)
    return v;
  if (!is_plain(dy.type) || !is_plain(dx.type)) return DSV_ERR_INVALID_ARG;
  if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4)) return DSV_ERR_INVALID_ARG;
  if (dx.type != (x.type == DSV_PACKED ? dy.type : x.type)) return DSV_ERR_INVALID_ARG;
  if (x.type != dy.type && x.type != DSV_FP32 && x.type != DSV_PACKED) return DSV_ERR_UNSUPPORTED;
  const int64_t rows = n.B * n.H * n.S, groups = norm_groups(n, params.per_batch != 0, params.per_head != 0);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    for (float* p : {dweight, dbias})
      if (p && groups > 0 && cudaMemsetAsync(p, 0, (size_t)groups * n.D * sizeof(float), st) != cudaSuccess)
        return DSV_ERR_CUDA;
    return DSV_OK;
  }
  if (!rstd) return DSV_ERR_INVALID_ARG;

  const bool vec = rows_take_vectors(dy, n) && rows_take_vectors(x, n) && rows_take_vectors(dx, n);
  const int64_t per = bwd_per_group(n.D, rows / groups, groups, vec);
  const bool join = per > 1 && (dweight || dbias);
  if (join && (!workspace || !aligned(workspace, 256) || workspace_bytes < (size_t)groups * per * 2 * n.D * sizeof(float)))
    return DSV_ERR_WORKSPACE;
  const int64_t join_blocks = groups * ((n.D + 31) / 32);
  if (join && join_blocks >= (int64_t(1) << 31)) return DSV_ERR_UNSUPPORTED;

  NormBwdArgs a;
  a.dy = dy.data;
  a.x = x.data;
  a.xe = static_cast<const uint8_t*>(x.exp);
  a.dx = dx.data;
  a.mean = mean;
  a.rstd = rstd;
  float* part = static_cast<float*>(workspace);
  a.dw = !dweight ? nullptr : join ? part : dweight;
  a.db = !dbias ? nullptr : join ? part + n.D : dbias;
  a.p = norm_params(params);
  a.inv_d = 1.f / (float)n.D;
  a.D = (int32_t)n.D;
  a.nb = (int32_t)((n.D + kPackBlock - 1) / kPackBlock);
  a.per_group = (int32_t)per;
  a.partial = join;
  const dsv_rows* tensors[] = {&dy, &x, &dx};
  const RowMap m = make_row_map(n, params.per_batch != 0, params.per_head != 0, tensors, 3);
  const NormShape s = norm_shape(n.D, vec);
  const uint32_t grid = (uint32_t)(groups * per);
  using bf16 = __nv_bfloat16;
  if (x.type == DSV_BF16) dispatch<bf16, bf16>(s, a, m, grid, st);
  else if (x.type == DSV_FP16) dispatch<__half, __half>(s, a, m, grid, st);
  else if (x.type == DSV_FP32 && dy.type == DSV_FP32) dispatch<float, float>(s, a, m, grid, st);
  else if (x.type == DSV_FP32 && dy.type == DSV_BF16) dispatch<float, bf16>(s, a, m, grid, st);
  else if (x.type == DSV_FP32) dispatch<float, __half>(s, a, m, grid, st);
  else if (dy.type == DSV_FP32) dispatch<Packed, float>(s, a, m, grid, st);
  else if (dy.type == DSV_BF16) dispatch<Packed, bf16>(s, a, m, grid, st);
  else dispatch<Packed, __half>(s, a, m, grid, st);
  if (cudaGetLastError() != cudaSuccess) return DSV_ERR_CUDA;
  if (join) {
    k_row_norm_join<<<(uint32_t)join_blocks, dim3(32, kJoinRows), 0, st>>>(part, (int)per, (int)n.D, dweight, dbias);
    if (cudaGetLastError() != cudaSuccess) return DSV_ERR_CUDA;
  }
  return DSV_OK;
}
