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
// four rows of 128 bytes by tile::gather4 that are not read again: they leave L2 to what is
__device__ __forceinline__ void gather4_once(void* dst, const CUtensorMap* m, uint64_t* bar, int x, const int (&r)[4],
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
      "l"(policy)
      : "memory");
}
// 32 bytes by one store, 32-byte aligned
__device__ __forceinline__ void store32(float* p, const float (&f)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
               "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

// barrier `id` (not 0) of `threads` threads, whole warps
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// byte offset of 16-byte piece `c` (0..7) of row `r` in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// 128 rows of RP ranks, rows of 32, 64 or 128 bytes with the swizzle of that
// width (rank 128: two such tiles).  With the rows along K it is an MN-major
// operand, with the ranks along K a K-major one.
//
// h and dh go from kernel to kernel as such tiles in global memory, one to 128
// rows of an adapter (by tile slot, rows / 128 + n of them) and to each of the
// three bf16 terms an fp32 value splits into: a kernel that multiplies with
// them brings a tile's terms by one bulk copy.
template <int RP>
struct RankTile {
  static constexpr int ROW = RP >= 64 ? 128 : RP * 2;
  static constexpr int BYTES = 128 * RP * 2;
  static constexpr int LEAD = 128 * ROW;
  static constexpr int IMAGE = 3 * BYTES;   // a tile slot's terms
  // byte offset of ranks 8 c .. 8 c + 7 of row r
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    if constexpr (RP == 16) return r * 32 + ((c ^ (r >> 2 & 1)) << 4);
    else if constexpr (RP == 32) return r * 64 + ((c ^ (r >> 1 & 3)) << 4);
    else return c / 8 * LEAD + swz(r, c % 8);
  }
  __device__ static __forceinline__ uint64_t desc(uint32_t addr, uint32_t lead) { return mn_desc<ROW>(addr, lead); }
  // 16 ranks from 16 k on, K-major
  __device__ static __forceinline__ uint64_t kdesc(uint32_t addr, int k) {
    constexpr int PER = ROW / 32;   // k steps to a row
    return mn_desc<ROW>(addr + k / PER * LEAD + k % PER * 32, 16);
  }
};
__host__ __device__ constexpr int padded_rank(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }
inline size_t image_bytes(int rows, int n, int R) {
  return (static_cast<size_t>(rows) / 128 + n) * 3 * 256 * padded_rank(R);
}

// 8 values to the three terms' pieces of a tile's image
template <int RP>
__device__ __forceinline__ void store_terms(uint8_t* image, int r, int c, const float (&v)[8]) {
  uint32_t w[3][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) split3(v[2 * u], v[2 * u + 1], w[0][u], w[1][u], w[2][u]);
#pragma unroll
  for (int q = 0; q < 3; ++q)
    *reinterpret_cast<uint4*>(image + q * RankTile<RP>::BYTES + RankTile<RP>::at(r, c)) =
        make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
}

// untiled bulk copy global -> shared (both 16-byte aligned, whole 16 bytes), counted on `bar`
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

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
  const uint8_t* V;         // images of V's terms, by tile slot
  const float* scale;       // [n] or nullptr: goes into P (the projection alone: into its image)
  const int32_t* offsets;
  const int32_t* order;
  int n, rows, W, R;
  int chunk, cols;          // rows and columns of a CTA, multiples of 128; the projection alone: chunk = 128
  int cluster;              // the projection alone: its slices, a power of two up to 8 that covers W
  float* proj;              // with the gradient: [slices][rows][R] by position, or nullptr: not wanted
  uint8_t* image;           // the projection alone: its images, by tile slot
  float* h_out;             // the projection alone: [rows][R] by row, not scaled, or nullptr
  float* part;              // G's partial sums, for the adapters of more than one chunk, by part_slot
  void* grad;               // G: [n, W, R] (dB) or [n, R, W] (dA), 0 for an adapter without rows; nullptr: not wanted
  int grad_f32;
  bool early;               // the launch before this one in the stream is one of this file's callers' and wrote V alone:
                            // X, M and the plan are loaded before it ends
  bool first;               // of the call's launches that have a status: it starts as MOE_OK
  int* status;
};
// Adapters of more than one chunk lie part_slot(offset) apart: with m > chunk
// rows, floor(2 m / chunk) >= ceil(m / chunk), so they do not overlap and all
// end before part_slot(rows).
__host__ __device__ constexpr size_t part_slot(int offset, int chunk) { return 2 * static_cast<size_t>(offset) / chunk; }
enum StreamKind { kStreamProject, kStreamBoth, kStreamGrad };
int launch_lora_stream(const StreamArgs& p, StreamKind kind, cudaStream_t s);
int lora_stream_max_cols(int R, bool proj);  // columns of a CTA that forms G, at most

// The gradients where an adapter has few rows, in one launch on tiles of kRowsFew rows (lora_few.cu); partial
// sums of adapters of more, by part_slot(offset, kRowsFew)
constexpr int kRowsFew = 16;
int launch_lora_few(const LoraBackwardArgs& q, float* part_A, float* part_B, cudaStream_t s);

// out[r] = base[r] + h[r] W_a (lora_expand.cu)
struct ExpandArgs {
  const uint8_t* h;         // images of h's terms, scaled, by tile slot
  const __nv_bfloat16* M;   // B [n, N, R], or A [n, R, N] (kn)
  const int32_t* offsets;
  const int32_t* order;
  int n, rows, N, R;
  int cols;                 // set by the launch
  const void* base;
  void* out;
  float* h_out;             // [rows, R] by row or nullptr: 0 for the rows without an adapter
  bool apart;               // h is older than the launch before this one, and nothing here and there depends on the
                            // other: this one runs beside it and waits for it at the end
  int* status;
};
int launch_lora_expand(ExpandArgs p, bool kn, int out_dtype, cudaStream_t s);

}  // namespace moe
