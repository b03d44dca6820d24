// Host side of the row calls: argument checks and the map from a group's rows
// to their offsets in every tensor.
#include <algorithm>

#include "rows.cuh"

namespace dsv {

dsv_status validate_extent(const dsv_extent& n) {
  if (n.B < 0 || n.H < 0 || n.S < 0 || n.D < 1) return DSV_ERR_INVALID_ARG;
  if (n.D > kMaxWidth) return DSV_ERR_UNSUPPORTED;
  constexpr int64_t kMost = (int64_t(1) << 31) - 1;
  if (n.B > kMost || n.H > kMost || n.S > kMost) return DSV_ERR_UNSUPPORTED;
  // each factor is below 2^31, so no product below overflows 64 bits before it is checked
  if (n.B * n.H > kMost || (n.B * n.H) * n.S > kMost) return DSV_ERR_UNSUPPORTED;
  if (n.B * n.H * n.S * ((n.D + kPackBlock - 1) / kPackBlock) > kMost) return DSV_ERR_UNSUPPORTED;
  return DSV_OK;
}

dsv_status validate_rows(const dsv_rows& t, const dsv_extent& n, bool output) {
  if (t.type != DSV_PACKED && !is_plain(t.type)) return DSV_ERR_INVALID_ARG;
  const bool empty = n.B * n.H * n.S == 0;
  if (t.type == DSV_PACKED) {
    if (!empty && (!t.data || !t.exp)) return DSV_ERR_INVALID_ARG;
    return aligned(t.data, 8) ? DSV_OK : DSV_ERR_INVALID_ARG;
  }
  if (t.exp) return DSV_ERR_INVALID_ARG;
  if (empty) return DSV_OK;
  if (!t.data || !aligned(t.data, elem_size(t.type))) return DSV_ERR_INVALID_ARG;
  struct Dim {
    int64_t size, stride;
  } d[3] = {{n.B, t.b}, {n.H, t.h}, {n.S, t.s}};
  for (const Dim& x : d)
    if (x.size > 1 && (x.stride < 0 || x.stride > (int64_t(1) << 56) / x.size)) return DSV_ERR_INVALID_ARG;
  if (output) {   // in order of stride, each dimension steps over the extent of the ones below it
    std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    int64_t extent = n.D;
    for (const Dim& x : d) {
      if (x.size == 1) continue;
      if (x.stride < extent) return DSV_ERR_INVALID_ARG;
      extent += x.stride * (x.size - 1);
    }
  }
  return DSV_OK;
}

bool rows_take_vectors(const dsv_rows& t, const dsv_extent& n) {
  if (n.D % 8) return false;
  if (t.type == DSV_PACKED) return true;   // contiguous, 8-byte aligned by validate_rows
  const int64_t es = elem_size(t.type);
  return aligned(t.data, 16) && (n.B <= 1 || t.b * es % 16 == 0) && (n.H <= 1 || t.h * es % 16 == 0) &&
         (n.S <= 1 || t.s * es % 16 == 0);
}

RowMap make_row_map(const dsv_extent& n, bool per_batch, bool per_head, const dsv_rows* const* tensors, int count) {
  RowMap m;
  memset(&m, 0, sizeof(m));
  int64_t size[3] = {n.B, n.H, n.S}, st[3][kMapTensors] = {};
  for (int t = 0; t < kMapTensors; ++t) {
    const dsv_rows* r = t < count ? tensors[t] : nullptr;
    const bool packed = r && r->type == DSV_PACKED;
    const int64_t w = packed ? n.D : 1;   // the last slot counts rows; a packed tensor is contiguous
    const bool linear = t == kMapTensors - 1 || packed;
    st[0][t] = linear ? n.H * n.S * w : r ? r->b : 0;
    st[1][t] = linear ? n.S * w : r ? r->h : 0;
    st[2][t] = linear ? w : r ? r->s : 0;
  }
  m.gh_n.set((uint32_t)(per_head ? std::max<int64_t>(n.H, 1) : 1));
  for (int t = 0; t < kMapTensors; ++t) {
    if (per_batch) m.gb[t] = st[0][t];
    if (per_head) m.gh[t] = st[1][t];
  }
  int64_t total = 1;
  int nd = 0;
  int64_t dims[3];
  for (int d = 0; d < 3; ++d) {
    if ((d == 0 && per_batch) || (d == 1 && per_head)) continue;
    total *= size[d];
    if (size[d] == 1) continue;
    bool fold = nd > 0;
    for (int t = 0; t < kMapTensors && fold; ++t) fold = m.stride[nd - 1][t] == st[d][t] * size[d];
    if (fold) {
      dims[nd - 1] *= size[d];
      for (int t = 0; t < kMapTensors; ++t) m.stride[nd - 1][t] = st[d][t];
    } else {
      dims[nd] = size[d];
      for (int t = 0; t < kMapTensors; ++t) m.stride[nd][t] = st[d][t];
      ++nd;
    }
  }
  if (nd == 0) {
    dims[0] = 1;
    nd = 1;
  }
  m.nd = nd;
  m.n = (uint32_t)total;
  for (int d = 0; d < nd; ++d) m.size[d].set((uint32_t)std::max<int64_t>(dims[d], 1));
  return m;
}

}  // namespace dsv
