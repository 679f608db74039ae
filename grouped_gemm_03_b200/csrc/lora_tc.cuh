// What the adapters' tensor-core kernels share: operand tiles in shared memory
// and the arguments of the two kernels.
#pragma once

#include "common.cuh"
#include "lora.cuh"
#include "ptx.cuh"

namespace moe {

// A K-major operand tile (rows of 64 values, 128-byte swizzle), and one whose
// rows run along K instead (MN-major): 64 values of M or N to a row, 8 rows to
// a swizzle atom, the next 8 rows of K 1024 bytes on, the next 64 of M or N
// `lead` bytes on.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kAMn = 1u << 15;  // instruction descriptor: A is MN-major
constexpr uint32_t kBMn = 1u << 16;  // B is

__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// byte offset of 16-byte piece `c` (0..7) of row `r` in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

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
