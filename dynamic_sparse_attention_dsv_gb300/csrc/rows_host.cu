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
  return rows_aligned(t, n, 16);
}

bool rows_aligned(const dsv_rows& t, const dsv_extent& n, int bytes) {
  const int64_t es = elem_size(t.type);
  return aligned(t.data, bytes) && (n.B <= 1 || t.b * es % bytes == 0) && (n.H <= 1 || t.h * es % bytes == 0) &&
         (n.S <= 1 || t.s * es % bytes == 0);
}

RowMap make_row_map(const dsv_extent& n, bool per_batch, bool per_head, const dsv_rows* const* tensors, int count) {
  RowMap m;
  memset(&m, 0, sizeof(m));
  struct Dim {
    int64_t size, st[kMapTensors];
  } dim[3] = {{n.B, {}}, {n.H, {}}, {n.S, {}}};
  for (int t = 0; t < kMapTensors; ++t) {
    const dsv_rows* r = t < count ? tensors[t] : nullptr;
    const bool packed = r && r->type == DSV_PACKED;
    if (t == kRowIndex || packed) {   // contiguous
      dim[2].st[t] = packed ? n.D : 1;
      dim[1].st[t] = n.S * dim[2].st[t];
      dim[0].st[t] = n.H * dim[1].st[t];
    } else if (r) {
      dim[0].st[t] = r->b;
      dim[1].st[t] = r->h;
      dim[2].st[t] = r->s;
    }
  }
  m.gh_n.set((uint32_t)(per_head ? n.H : 1));
  for (int t = 0; t < kMapTensors; ++t) {
    if (per_batch) m.gb[t] = dim[0].st[t];
    if (per_head) m.gh[t] = dim[1].st[t];
  }
  Dim rest[3];
  int nd = 0;
  for (int d = 0; d < 3; ++d) {
    if ((d == 0 && per_batch) || (d == 1 && per_head) || dim[d].size == 1) continue;
    bool fold = nd > 0;
    for (int t = 0; t < kMapTensors && fold; ++t) fold = rest[nd - 1].st[t] == dim[d].st[t] * dim[d].size;
    if (fold) {
      const int64_t outer = rest[--nd].size;
      rest[nd] = dim[d];
      rest[nd++].size *= outer;
    } else {
      rest[nd++] = dim[d];
    }
  }
  int in = nd - 1;                       // the largest dimension, the last of equals
  for (int d = nd - 1; d >= 0; --d)
    if (rest[d].size > rest[in].size) in = d;
  m.n = nd ? (uint32_t)rest[in].size : 1;
  m.per_group = 1;
  int o = 0;
  for (int d = 0; d < nd; ++d) {
    if (d == in) {
      for (int t = 0; t < kMapTensors; ++t) m.step[t] = rest[d].st[t];
    } else {
      m.o_n[o].set((uint32_t)rest[d].size);
      m.per_group *= (uint32_t)rest[d].size;
      for (int t = 0; t < kMapTensors; ++t) m.o[o][t] = rest[d].st[t];
      ++o;
    }
  }
  for (; o < 2; ++o) m.o_n[o].set(1);
  return m;
}

void set_tile_steps(RowMap& m, const dsv_rows* const* tensors, int count, uint32_t rows) {
  for (int t = 0; t < count; ++t) m.tile[t] = m.step[t] * rows * elem_size(tensors[t]->type);
  m.tile[kRowIndex] = m.step[kRowIndex] * rows;
}

Split make_split(int64_t segments, int64_t units, int64_t tile, int64_t most_blocks) {
  Split p;
  p.per_segment = (uint32_t)((units + tile - 1) / tile);
  p.tiles = segments * p.per_segment;
  p.blocks = (uint32_t)std::min(p.tiles, most_blocks);
  return p;
}

}  // namespace dsv
