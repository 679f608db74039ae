// What the adapters' tensor-core kernels share: operand tiles in shared memory
// and the arguments of the two kernels.
#pragma once

#include "common.cuh"
#include "lora.cuh"
#include "ptx.cuh"

namespace moe {

// Descriptor of an operand tile whose rows run along K (MN-major): `span`
// bytes of M or N to a row (its swizzle's width: 128, 64 or 32), 8 rows to a
// swizzle atom, the next 8 rows of K behind it, the next span of M or N `lead`
// bytes on.
template <int SPAN = 128>
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t lead) {
  constexpr uint64_t layout = SPAN == 128 ? 2 : SPAN == 64 ? 4 : 6;
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(SPAN * 8 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= layout << 61;
  return d;
}
constexpr uint32_t kAMn = 1u << 15;  // instruction descriptor: A is MN-major
constexpr uint32_t kBMn = 1u << 16;  // B is

// 3-D tiled bulk copy (coordinates innermost first)
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// 32 bytes by one store, 32-byte aligned
__device__ __forceinline__ void store32(float* p, const float (&f)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
               "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

// byte offset of 16-byte piece `c` (0..7) of row `r` in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// 128 rows of RP ranks as an MN-major operand: rows of 32, 64 or 128 bytes with
// the swizzle of that width (rank 128: two such tiles).
template <int RP>
struct RankTile {
  static constexpr int ROW = RP >= 64 ? 128 : RP * 2;
  static constexpr int BYTES = 128 * RP * 2;
  static constexpr int LEAD = 128 * ROW;
  // byte offset of ranks 8 c .. 8 c + 7 of row r
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    if constexpr (RP == 16) return r * 32 + ((c ^ (r >> 2 & 1)) << 4);
    else if constexpr (RP == 32) return r * 64 + ((c ^ (r >> 1 & 3)) << 4);
    else return c / 8 * LEAD + swz(r, c % 8);
  }
  __device__ static __forceinline__ uint64_t desc(uint32_t addr, uint32_t lead) { return mn_desc<ROW>(addr, lead); }
};

// The driver's tensor-map encoder and the K-major map of [rows, K] (grouped_gemm.cu)
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_fn();
bool make_map(CUtensorMap* m, const void* base, int ebytes, uint64_t rows, uint64_t K, uint32_t box_rows);
// A map of the adapters' [n, rows, cols] bf16 weights, boxes of one adapter, swizzled by the box's width (64, 32
// or 16 columns); what a box holds outside the adapter is 0
bool make_adapter_map(CUtensorMap* m, const void* base, uint64_t n, uint64_t rows, uint64_t cols, uint32_t box_rows,
                      uint32_t box_cols);

// ---------------------------------------------------------------- the two kernels
// X [rows, W] once: projection P = X M^T and gradient G = X^T V (lora_stream.cu)
struct StreamArgs {
  const __nv_bfloat16* X;
  const __nv_bfloat16* M;   // A [n, R, W] (projection alone) or B [n, W, R]
  const float* V;           // h [rows, R] by row (with the projection) or dh [rows, R] by position
  const float* scale;       // with M = B: goes into P and V
  const int32_t* offsets;
  const int32_t* order;
  int n, rows, W, R;
  int chunk, cols;          // rows and columns of a CTA, multiples of 128; the projection alone: chunk = 128
  int cluster;              // the projection alone: its slices, a power of two up to 8 that covers W
  float* proj;              // [slices][rows][R] by position (alone: [rows][R], the sum); nullptr: not wanted
  float* h_out;             // the projection alone: the same by row, or nullptr
  float* part;              // G's partial sums, by chunk slot; with grad
  void* grad;               // G: [n, W, R] (dB) or [n, R, W] (dA); nullptr: not wanted
  int grad_f32;
  int* status;
};
enum StreamKind { kStreamProject, kStreamBoth, kStreamGrad };
int launch_lora_stream(const StreamArgs& p, StreamKind kind, cudaStream_t s);
int lora_stream_max_cols(int R);  // columns of a CTA that forms G, at most

// out[r] = base[r] + s h[r] W_a (lora_expand.cu)
struct ExpandArgs {
  const float* h;           // [rows][R] by position
  const __nv_bfloat16* M;   // B [n, N, R], or A [n, R, N] (kn)
  const float* scale;       // [n] or nullptr: factor of h
  const int32_t* offsets;
  const int32_t* order;
  int n, rows, N, R;
  int cols;                 // set by the launch
  const void* base;
  void* out;
  float* h_out;             // [rows, R] by row or nullptr: 0 for the rows without an adapter
  int* status;
};
int launch_lora_expand(ExpandArgs p, bool kn, int out_dtype, cudaStream_t s);

}  // namespace moe
