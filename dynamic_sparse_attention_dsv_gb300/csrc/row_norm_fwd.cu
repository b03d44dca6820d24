// Norm of each row over its channels, with the row's 8-bit checkpoint on request.
#include <algorithm>

#include "row_norm.cuh"

namespace dsv {

struct NormFwdArgs {
  const void* x;
  const uint8_t* xe;
  void* y;
  float *mean, *rstd;
  int8_t* pq;
  uint8_t* pe;
  NormParams p;
  float eps, inv_d;
  int32_t center, D, nb;       // nb: blocks of 32 channels a row
  int32_t per_group;           // thread blocks a group
};

// One row per L lanes (or per block): the row stays in registers between the
// sum, the squares around the mean, and the output, so x is read once.
template <class XT, class YT, int L, int K, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : kNormThreads)
    k_row_norm_fwd(const __grid_constant__ NormFwdArgs a, const __grid_constant__ RowMap m) {
  using XE = typename Elem<XT>::type;
  __shared__ float buf[2][32][1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const uint32_t g = blockIdx.x / a.per_group, c = blockIdx.x % a.per_group;
  const uint32_t gb = m.gh_n.div(g), gh = g - gb * m.gh_n.d;
  int64_t g0[kMapTensors];
  group_offsets(m, g, g0);

  float w[K][8], b[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int col = norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[k][e] = 1.f;
      b[k][e] = 0.f;
    }
    if (a.p.weight) load_params<VEC>(a.p.weight, a.p.type, gb * a.p.wb + gh * a.p.wh, a.p.base, col, a.D, w[k]);
    if (a.p.bias) load_params<VEC>(a.p.bias, a.p.type, gb * a.p.bb + gh * a.p.bh, 0.f, col, a.D, b[k]);
  }

  constexpr int kRows = BLOCK ? 1 : kNormThreads / L;     // rows of a block at a time
  int turn = 0;
  const uint32_t slot = BLOCK ? 0 : threadIdx.x / L;
  for (uint32_t t = c; (uint64_t)t * kRows < m.n; t += a.per_group) {
    const uint32_t i = t * kRows + slot;
    const bool live = i < m.n;
    int64_t off[kMapTensors];
    row_offsets(m, live ? i : m.n - 1, off);
    const int64_t row = g0[3] + off[3];
    const XE* x = static_cast<const XE*>(a.x) + g0[0] + off[0];
    Chunk<XT, VEC> ch[K];
    float f[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
      ch[k].load(x, a.xe + row * a.nb, norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps), a.D);
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      ch[k].to(f[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += f[k][e];
    }
    float mean = 0.f;
    if (a.center) {
      row_sums<L, BLOCK, 1>(s, buf, turn, lane, warp, nwarps);
      mean = s[0] * a.inv_d;
    }
    if (a.pq) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        pack_chunk<VEC>(a.pq + row * a.D, a.pe + row * a.nb, norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps),
                        live ? a.D : 0, f[k]);
    }
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int col = norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[k][e] -= mean;
        const bool in = VEC ? col < a.D : col + e * 32 < a.D;
        s[0] += in ? f[k][e] * f[k][e] : 0.f;
      }
    }
    row_sums<L, BLOCK, 1>(s, buf, turn, lane, warp, nwarps);
    const float rstd = 1.f / sqrtf(s[0] * a.inv_d + a.eps);
    if (live) {
      YT* y = static_cast<YT*>(a.y) + g0[1] + off[1];
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[k][e] = fmaf(f[k][e] * rstd, w[k][e], b[k][e]);
        store_chunk<YT, VEC>(y, norm_col<L, VEC, BLOCK>(k, lane, warp, nwarps), a.D, f[k]);
      }
      if ((BLOCK ? threadIdx.x : (threadIdx.x & (L - 1))) == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
  }
}

dsv_status validate_norm_params(const dsv_norm_params& p) {
  if (!p.weight && !p.bias) return DSV_OK;
  if (!is_plain(p.type)) return DSV_ERR_INVALID_ARG;
  const int es = elem_size(p.type);
  if (!aligned(p.weight, es) || !aligned(p.bias, es)) return DSV_ERR_INVALID_ARG;
  constexpr int64_t kMost = int64_t(1) << 40;
  for (int64_t s : {p.weight_b, p.bias_b})
    if (p.per_batch && (s < 0 || s > kMost)) return DSV_ERR_INVALID_ARG;
  for (int64_t s : {p.weight_h, p.bias_h})
    if (p.per_head && (s < 0 || s > kMost)) return DSV_ERR_INVALID_ARG;
  return p.base == p.base && p.base - p.base == 0.f ? DSV_OK : DSV_ERR_INVALID_ARG;
}

template <class XT, class YT, int L, int K, bool VEC, bool BLOCK>
static void launch(const NormFwdArgs& a0, const RowMap& m, int64_t groups, int threads, cudaStream_t st) {
  NormFwdArgs a = a0;
  const int64_t tiles = (m.n + (BLOCK ? 1 : kNormThreads / L) - 1) / (BLOCK ? 1 : kNormThreads / L);
  const int64_t want = (int64_t)kSMs * 8 * 8 * 32 / threads;
  a.per_group = (int32_t)std::min<int64_t>(tiles, std::max<int64_t>(1, want / groups));
  k_row_norm_fwd<XT, YT, L, K, VEC, BLOCK>
      <<<(uint32_t)(groups * a.per_group), threads, 0, st>>>(a, m);
}

template <class XT, class YT>
static void dispatch(const NormShape& s, const NormFwdArgs& a, const RowMap& m, int64_t groups, cudaStream_t st) {
  if (s.vec && s.L == 8) return launch<XT, YT, 8, 1, true, false>(a, m, groups, s.threads, st);
  if (s.vec && s.L == 16) return launch<XT, YT, 16, 1, true, false>(a, m, groups, s.threads, st);
  if (s.block)
    return s.vec ? launch<XT, YT, 32, 2, true, true>(a, m, groups, s.threads, st)
                 : launch<XT, YT, 32, 2, false, true>(a, m, groups, s.threads, st);
  if (s.K == 2)
    return s.vec ? launch<XT, YT, 32, 2, true, false>(a, m, groups, s.threads, st)
                 : launch<XT, YT, 32, 2, false, false>(a, m, groups, s.threads, st);
  return s.vec ? launch<XT, YT, 32, 1, true, false>(a, m, groups, s.threads, st)
               : launch<XT, YT, 32, 1, false, false>(a, m, groups, s.threads, st);
}

}  // namespace dsv

using namespace dsv;

extern "C" dsv_status dsv_layer_norm_fwd(dsv_rows x, dsv_extent n, dsv_norm_params params, float eps, int32_t center,
                                         dsv_rows y, float* mean, float* rstd, dsv_rows pack, void* stream) {
  dsv_status v = validate_extent(n);
  if (v != DSV_OK) return v;
  if ((v = validate_rows(x, n, false)) != DSV_OK || (v = validate_rows(y, n, true)) != DSV_OK ||
      (v = validate_norm_params(params)) != DSV_OK)
    return v;
  if (!(eps > 0.f) || !(eps - eps == 0.f)) return DSV_ERR_INVALID_ARG;
  if (!is_plain(y.type) || !aligned(mean, 4) || !aligned(rstd, 4)) return DSV_ERR_INVALID_ARG;
  if (x.type != y.type && x.type != DSV_FP32 && x.type != DSV_PACKED) return DSV_ERR_UNSUPPORTED;
  if (pack.data) {
    if (pack.type != DSV_PACKED || x.type == DSV_PACKED) return DSV_ERR_INVALID_ARG;
    if ((v = validate_rows(pack, n, true)) != DSV_OK) return v;
  }
  if (n.B * n.H * n.S == 0) return DSV_OK;

  NormFwdArgs a;
  a.x = x.data;
  a.xe = static_cast<const uint8_t*>(x.exp);
  a.y = y.data;
  a.mean = mean;
  a.rstd = rstd;
  a.pq = static_cast<int8_t*>(pack.data);
  a.pe = static_cast<uint8_t*>(pack.exp);
  a.p = norm_params(params);
  a.eps = eps;
  a.inv_d = 1.f / (float)n.D;
  a.center = center != 0;
  a.D = (int32_t)n.D;
  a.nb = (int32_t)((n.D + kPackBlock - 1) / kPackBlock);
  a.per_group = 1;
  const dsv_rows* tensors[] = {&x, &y};
  const RowMap m = make_row_map(n, params.per_batch != 0, params.per_head != 0, tensors, 2);
  const int64_t groups = (params.per_batch ? n.B : 1) * (params.per_head ? n.H : 1);
  const NormShape s = norm_shape(n.D, rows_take_vectors(x, n) && rows_take_vectors(y, n));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using bf16 = __nv_bfloat16;
  const int y_type = y.type;
  if (x.type == DSV_BF16) dispatch<bf16, bf16>(s, a, m, groups, st);
  else if (x.type == DSV_FP16) dispatch<__half, __half>(s, a, m, groups, st);
  else if (x.type == DSV_FP32 && y_type == DSV_FP32) dispatch<float, float>(s, a, m, groups, st);
  else if (x.type == DSV_FP32 && y_type == DSV_BF16) dispatch<float, bf16>(s, a, m, groups, st);
  else if (x.type == DSV_FP32) dispatch<float, __half>(s, a, m, groups, st);
  else if (y_type == DSV_FP32) dispatch<Packed, float>(s, a, m, groups, st);
  else if (y_type == DSV_BF16) dispatch<Packed, bf16>(s, a, m, groups, st);
  else dispatch<Packed, __half>(s, a, m, groups, st);
  return cudaGetLastError() == cudaSuccess ? DSV_OK : DSV_ERR_CUDA;
}
