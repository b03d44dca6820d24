// 8-bit activation checkpoints: written and restored.
#include <algorithm>

#include "rows.cuh"

namespace dsv {

struct PackArgs {
  const void* x;
  void* y;
  int8_t* q;
  uint8_t* e;
  int32_t D, nb;
  uint32_t tiles;          // 256-channel pieces of all rows
  FastDiv per_row;         // pieces a row
};

// One warp per 256 channels of a row, eight a lane.
template <class T, bool VEC, bool RESTORE>
__global__ void __launch_bounds__(256) k_act_rows(const __grid_constant__ PackArgs a, const __grid_constant__ RowMap m) {
  const int lane = threadIdx.x & 31;
  for (uint32_t t = blockIdx.x * 8 + (threadIdx.x >> 5); t < a.tiles; t += gridDim.x * 8) {
    const uint32_t i = a.per_row.div(t);
    const int col = (int)(t - i * a.per_row.d) * 256 + (VEC ? lane * 8 : lane);
    int64_t off[kMapTensors];
    row_offsets(m, i, off);
    float f[8];
    if (RESTORE) {
      Chunk<Packed, VEC> ch;
      ch.load(a.q + off[3] * a.D, a.e + off[3] * a.nb, col, a.D);
      ch.to(f);
      store_chunk<T, VEC>(static_cast<T*>(a.y) + off[0], col, a.D, f);
    } else {
      Chunk<T, VEC> ch;
      ch.load(static_cast<const T*>(a.x) + off[0], nullptr, col, a.D);
      ch.to(f);
      pack_chunk<VEC>(a.q + off[3] * a.D, a.e + off[3] * a.nb, col, a.D, f);
    }
  }
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
  a.y = plain.data;
  a.q = static_cast<int8_t*>(packed.data);
  a.e = static_cast<uint8_t*>(packed.exp);
  a.D = (int32_t)n.D;
  a.nb = (int32_t)((n.D + kPackBlock - 1) / kPackBlock);
  const int64_t per_row = (n.D + 255) / 256;
  a.tiles = (uint32_t)(rows * per_row);
  a.per_row.set((uint32_t)per_row);
  const dsv_rows* tensors[] = {&plain};
  const RowMap m = make_row_map(n, false, false, tensors, 1);
  const bool vec = rows_take_vectors(plain, n);
  const uint32_t grid = std::min<uint32_t>((a.tiles + 7) / 8, kSMs * 32);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using bf16 = __nv_bfloat16;
  if (plain.type == DSV_BF16) vec ? k_act_rows<bf16, true, RESTORE><<<grid, 256, 0, st>>>(a, m) : k_act_rows<bf16, false, RESTORE><<<grid, 256, 0, st>>>(a, m);
  else if (plain.type == DSV_FP16) vec ? k_act_rows<__half, true, RESTORE><<<grid, 256, 0, st>>>(a, m) : k_act_rows<__half, false, RESTORE><<<grid, 256, 0, st>>>(a, m);
  else vec ? k_act_rows<float, true, RESTORE><<<grid, 256, 0, st>>>(a, m) : k_act_rows<float, false, RESTORE><<<grid, 256, 0, st>>>(a, m);
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
