// 8-bit activation checkpoints: written and restored. A block of 32 channels keeps
// the exponent field of its largest magnitude, which makes its step a power of
// two: x / step and q * step are exact, so there is one rounding, to q.
//
// Bound by HBM, sizeof(x) + 33/32 bytes a channel. Measured on the device, with
// the share of the measured copy bandwidth: 16 heads x 256K tokens x 128
// channels restored to bf16 266 us (90%); 24 heads x 64K x 128 written and
// restored 205 us (88%).
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace dsv {

struct PackArgs {
  void* x;
  int8_t* q;
  uint8_t* e;
  int32_t D, nb;           // nb: blocks of 32 channels a row
  FastDiv per_row;         // blocks of a row, or its pieces where it takes no vector loads
  uint32_t n;              // of a segment
  Split split;
};

// Rows that take vector loads: four lanes a block, eight channels each, kUnits
// blocks a lane whose loads are all issued before the first is used. Bound by
// HBM; what counts is the number of warps that write: at 64K tokens x 24 heads
// x 128 channels pack and unpack together take 229 us with 4 blocks of threads
// an SM (and 4 units), 213 with 6 and 204 with 8 (2 units); the floor is 180.
constexpr int kUnits = 2, kQuads = 64, kActBlocks = 8;
template <class T, bool RESTORE>
__global__ void __launch_bounds__(4 * kQuads, kActBlocks)
    k_act_vec(const __grid_constant__ PackArgs a, const __grid_constant__ RowMap m) {
  using Src = typename std::conditional<RESTORE, Packed, T>::type;
  const uint32_t quad = threadIdx.x >> 2, sub = threadIdx.x & 3;
  int64_t tile = a.split.first(blockIdx.x);
  const int64_t end = a.split.first(blockIdx.x + 1);
  while (tile < end) {
    const uint32_t seg = (uint32_t)(tile / a.split.per_segment);
    uint32_t t = (uint32_t)(tile - (int64_t)seg * a.split.per_segment);
    const uint32_t last = t + (uint32_t)min(end - tile, (int64_t)(a.split.per_segment - t));
    tile += last - t;
    const SegmentAt sa(m, seg);
    T* x = static_cast<T*>(a.x) + sa.in(m, 0);
    const int64_t row0 = sa.in(m, kRowIndex);
    for (; t < last; ++t) {
      Chunk<Src, true, 32> ch[kUnits];
      T* plain[kUnits];
      int8_t* q[kUnits];
      uint8_t* e[kUnits];
      int col[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const uint32_t blk = (t * kUnits + u) * kQuads + quad;
        const uint32_t i = a.per_row.div(min(blk, a.n - 1));
        // a lane past the last block, or past the row's channels, reads and writes nothing
        col[u] = blk < a.n ? (int)((blk - i * a.per_row.d) * 32 + sub * 8) : a.D;
        plain[u] = x + (int64_t)i * m.step[0];
        const int64_t row = row0 + (int64_t)i * m.step[kRowIndex];
        q[u] = a.q + row * a.D;
        e[u] = a.e + row * a.nb;
        if constexpr (RESTORE) ch[u].load(q[u], e[u], col[u], a.D);
        else ch[u].load(plain[u], nullptr, col[u], a.D);
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        float2 f[4];
        ch[u].to(f);
        if constexpr (RESTORE) store_chunk<T, true, 32>(plain[u], col[u], a.D, f);
        else pack_chunk<true, 32>(q[u], e[u], col[u], a.D, f);
      }
    }
  }
}

// Any other rows: L lanes hold a piece of 8 L channels of a row, L = 8 for rows of
// up to 64 channels (a warp a row took 1950 us for 3.5M rows of 12 fp32 channels,
// written and restored; this 420), and kPieces pieces at a time (77K rows of 890
// fp32 channels restored: 137 us with two pieces and four blocks an SM, 103 with
// two and six, 110 with one and eight).
constexpr int kPieces = 2, kScalarBlocks = 6;
template <class T, bool RESTORE, int L>
__global__ void __launch_bounds__(256, kScalarBlocks)
    k_act_scalar(const __grid_constant__ PackArgs a, const __grid_constant__ RowMap m) {
  using Src = typename std::conditional<RESTORE, Packed, T>::type;
  const uint32_t first = threadIdx.x / L, lane = threadIdx.x % L;
  int64_t tile = a.split.first(blockIdx.x);
  const int64_t end = a.split.first(blockIdx.x + 1);
  for (; tile < end; ++tile) {
    const uint32_t seg = (uint32_t)(tile / a.split.per_segment);
    const uint32_t u0 = (uint32_t)(tile - (int64_t)seg * a.split.per_segment) * (256 / L * kPieces) + first;
    const SegmentAt sa(m, seg);
    T* const x = static_cast<T*>(a.x) + sa.in(m, 0);
    const int64_t row0 = sa.in(m, kRowIndex);
    Chunk<Src, false, L> ch[kPieces];
    T* plain[kPieces];
    int8_t* q[kPieces];
    uint8_t* e[kPieces];
    int col[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const uint32_t u = u0 + p * (256 / L), i = a.per_row.div(min(u, a.n - 1));
      // a piece past the last reads and writes nothing
      col[p] = u < a.n ? (int)((u - i * a.per_row.d) * (8 * L) + lane) : a.D;
      plain[p] = x + (int64_t)i * m.step[0];
      const int64_t row = row0 + (int64_t)i * m.step[kRowIndex];
      q[p] = a.q + row * a.D;
      e[p] = a.e + row * a.nb;
      if constexpr (RESTORE) ch[p].load(q[p], e[p], col[p], a.D);
      else ch[p].load(plain[p], nullptr, col[p], a.D);
    }
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      float2 f[4];
      ch[p].to(f);
      if constexpr (RESTORE) store_chunk<T, false, L>(plain[p], col[p], a.D, f);
      else pack_chunk<false, L>(q[p], e[p], col[p], a.D, f);
    }
  }
}

// Up to four contiguous checkpoints of the same size with whole blocks, restored
// to bf16 by one launch: block row y takes tensor y, four lanes a block of 32.
struct RestoreArgs {
  const int8_t* q[4];
  const uint8_t* e[4];
  __nv_bfloat16* out[4];
  int64_t blocks;
};
__global__ void __launch_bounds__(4 * kQuads, kActBlocks) k_act_restore(const __grid_constant__ RestoreArgs a) {
  const int8_t* q = a.q[blockIdx.y];
  const uint8_t* e = a.e[blockIdx.y];
  __nv_bfloat16* out = a.out[blockIdx.y];
  const int quad = threadIdx.x >> 2, sub = (threadIdx.x & 3) * 8;
  for (int64_t b0 = (int64_t)blockIdx.x * (kQuads * kUnits); b0 < a.blocks; b0 += (int64_t)gridDim.x * (kQuads * kUnits)) {
    Chunk<Packed, true, 32> ch[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t b = b0 + u * kQuads + quad;
      ch[u].load(q + b * kPackBlock, e + b, sub, b < a.blocks ? kPackBlock : 0);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t b = b0 + u * kQuads + quad;
      float2 f[4];
      ch[u].to(f);
      store_chunk<__nv_bfloat16, true, 32>(out + b * kPackBlock, sub, b < a.blocks ? kPackBlock : 0, f);
    }
  }
}

template <class T, bool RESTORE>
static void launch(PackArgs a, const RowMap& m, bool vec, cudaStream_t st) {
  if (vec) {
    a.n = m.n * a.nb;
    a.split = make_split(m.per_group, a.n, kQuads * kUnits, kSMs * kActBlocks);
    k_act_vec<T, RESTORE><<<a.split.blocks, 4 * kQuads, 0, st>>>(a, m);
    return;
  }
  const int L = a.D > 64 ? 32 : 8, per_row = (a.D + 8 * L - 1) / (8 * L);
  a.per_row.set((uint32_t)per_row);
  a.n = m.n * per_row;
  a.split = make_split(m.per_group, a.n, 256 / L * kPieces, kSMs * kScalarBlocks);
  if (L == 32) k_act_scalar<T, RESTORE, 32><<<a.split.blocks, 256, 0, st>>>(a, m);
  else k_act_scalar<T, RESTORE, 8><<<a.split.blocks, 256, 0, st>>>(a, m);
}

template <bool RESTORE>
static dsv_status run(const dsv_rows& plain, const dsv_rows& packed, const dsv_extent& n, void* stream) {
  dsv_status v = validate_extent(n);
  if (v != DSV_OK) return v;
  if (!is_plain(plain.type) || packed.type != DSV_PACKED) return DSV_ERR_INVALID_ARG;
  if ((v = validate_rows(plain, n, RESTORE)) != DSV_OK || (v = validate_rows(packed, n, !RESTORE)) != DSV_OK) return v;
  const int64_t rows = n.B * n.H * n.S;
  if (rows == 0) return DSV_OK;
  PackArgs a;
  a.x = plain.data;
  a.q = static_cast<int8_t*>(packed.data);
  a.e = static_cast<uint8_t*>(packed.exp);
  a.D = (int32_t)n.D;
  a.nb = (int32_t)((n.D + kPackBlock - 1) / kPackBlock);
  a.per_row.set((uint32_t)a.nb);
  const dsv_rows* tensors[] = {&plain};
  const RowMap m = make_row_map(n, false, false, tensors, 1);
  const bool vec = rows_take_vectors(plain, n);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (plain.type == DSV_BF16) launch<__nv_bfloat16, RESTORE>(a, m, vec, st);
  else if (plain.type == DSV_FP16) launch<__half, RESTORE>(a, m, vec, st);
  else launch<float, RESTORE>(a, m, vec, st);
  return cudaGetLastError() == cudaSuccess ? DSV_OK : DSV_ERR_CUDA;
}

}  // namespace dsv

using namespace dsv;

extern "C" dsv_status dsv_act_pack(dsv_rows x, dsv_extent n, dsv_rows packed, void* stream) {
  return run<false>(x, packed, n, stream);
}

extern "C" dsv_status dsv_act_unpack(dsv_rows packed, dsv_extent n, dsv_rows y, void* stream) {
  return run<true>(y, packed, n, stream);
}

static size_t restored_bytes(const dsv_shape& s) {
  return round_up((size_t)(s.B * s.H * s.T * s.Y * s.X * s.d) * sizeof(__nv_bfloat16), 256);
}

extern "C" size_t dsv_sparse_attn_bwd_packed_workspace_size(dsv_shape shape, dsv_group group, const int32_t* k_per_head,
                                                            const int64_t* idx_offset, int32_t n_packed) {
  const size_t bwd = dsv_sparse_attn_bwd_workspace_size(shape, group, k_per_head, idx_offset);
  return bwd && n_packed >= 0 && n_packed <= 4 ? bwd + n_packed * restored_bytes(shape) : 0;
}

extern "C" size_t dsv_sparse_attn_bwd_packed_min_workspace_size(dsv_shape shape, dsv_group group,
                                                                const int32_t* k_per_head, const int64_t* idx_offset,
                                                                int32_t n_packed) {
  const size_t bwd = dsv_sparse_attn_bwd_min_workspace_size(shape, group, k_per_head, idx_offset);
  return bwd && n_packed >= 0 && n_packed <= 4 ? bwd + n_packed * restored_bytes(shape) : 0;
}

extern "C" dsv_status dsv_sparse_attn_bwd_packed(dsv_rows Q, dsv_rows K, dsv_rows V, dsv_rows O, const float* LSE,
                                                 const void* dO, const int32_t* idx, const int32_t* k_per_head,
                                                 const int64_t* idx_offset, dsv_shape shape, dsv_group group,
                                                 float scale, void* dQ, void* dK, void* dV, void* workspace,
                                                 size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const dsv_rows* in[4] = {&Q, &K, &V, &O};
  const void* plain[4];
  for (int i = 0; i < 4; ++i) {
    if (in[i]->type != DSV_PACKED && (in[i]->type != DSV_BF16 || in[i]->exp)) return DSV_ERR_INVALID_ARG;
    // a restored tensor lies in the workspace, whose alignment is checked below
    plain[i] = in[i]->type == DSV_PACKED ? workspace : in[i]->data;
  }
  // everything the backward refuses is refused before the restoring launch
  if (!workspace || !aligned(workspace, 256)) return DSV_ERR_WORKSPACE;
  dsv_status v = validate_bwd(plain[0], plain[1], plain[2], plain[3], LSE, dO, idx, k_per_head, idx_offset, shape, group,
                              scale, dQ, dK, dV);
  if (v != DSV_OK) return v;
  const dsv_extent n = {shape.B, shape.H, shape.T * shape.Y * shape.X, shape.d};
  if ((v = validate_extent(n)) != DSV_OK) return v;
  int packed = 0;
  for (const dsv_rows* t : in) {
    if (t->type != DSV_PACKED) continue;
    if ((v = validate_rows(*t, n, false)) != DSV_OK) return v;
    ++packed;
  }
  const size_t front = packed * restored_bytes(shape);
  const size_t least = dsv_sparse_attn_bwd_min_workspace_size(shape, group, idx ? k_per_head : nullptr,
                                                              idx ? idx_offset : nullptr);
  if (workspace_bytes < front + least) return DSV_ERR_WORKSPACE;
  char* at = static_cast<char*>(workspace);
  RestoreArgs r = {};
  r.blocks = n.B * n.H * n.S * n.D / kPackBlock;
  int count = 0;
  for (int i = 0; i < 4; ++i) {
    if (in[i]->type != DSV_PACKED) continue;
    r.q[count] = static_cast<const int8_t*>(in[i]->data);
    r.e[count] = static_cast<const uint8_t*>(in[i]->exp);
    r.out[count++] = reinterpret_cast<__nv_bfloat16*>(at);
    plain[i] = at;
    at += restored_bytes(shape);
  }
  if (count) {
    const int64_t tiles = (r.blocks + kQuads * kUnits - 1) / (kQuads * kUnits);
    const dim3 grid((uint32_t)std::min<int64_t>(tiles, kSMs * kActBlocks), count);
    k_act_restore<<<grid, 4 * kQuads, 0, static_cast<cudaStream_t>(stream)>>>(r);
    if (cudaGetLastError() != cudaSuccess) return DSV_ERR_CUDA;
  }
  return dsv_sparse_attn_bwd(plain[0], plain[1], plain[2], plain[3], LSE, dO, idx, k_per_head, idx_offset, shape, group,
                             scale, dQ, dK, dV, at, workspace_bytes - front, dev_status, stream);
}
