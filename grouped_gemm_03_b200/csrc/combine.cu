// Combine: gather each token's k expert outputs back to token order, weight
// them by their gate values and sum, adding the shared expert's row
// ("Dense GEMM -> GroupedGEMM -> TP MoE" §2.2 step 6; "MegaMoE ..." §2.1).
//   out[t] = Y[R + t] + sum_{j<k} w[t, j] * Y[token_to_row[t, j]]
// fp32 accumulation in that fixed order, 16-byte loads.  R is T*k, or the
// first shared row the permute recorded (offsets[E]) when experts have a
// capacity; a slot whose pair overflowed (token_to_row < 0) adds nothing.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kCombThreads = 128;

__device__ __forceinline__ void unpack8(const uint4& r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Grid = tokens x (d / 2048): each thread owns 16 columns (two 16-byte
// pieces) of one token and issues the loads of all k + 1 rows for them before
// it accumulates.
constexpr int kCombCols = kCombThreads * 16;

template <typename OT>
__device__ __forceinline__ void store8(OT* o, const float (&acc)[8]) {
  if constexpr (sizeof(OT) == 4) {
    reinterpret_cast<float4*>(o)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4*>(o)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<uint4*>(h);
  }
}

template <typename OT>
__global__ void __launch_bounds__(kCombThreads) combine_kernel(const __nv_bfloat16* __restrict__ Y,
                                                              const int32_t* __restrict__ t2r,
                                                              const float* __restrict__ w, int has_shared,
                                                              int T, int d, int k, OT* __restrict__ out,
                                                              const int32_t* __restrict__ shared_base) {
  pdl_wait();  // the preceding kernel on the stream is complete and visible
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const int c0 = blockIdx.y * kCombCols + threadIdx.x * 8;               // first piece
  const int c1 = c0 + kCombThreads * 8;                                   // second piece
  const bool p0 = c0 < d, p1 = c1 < d;
  if (!p0) return;
  const size_t R = shared_base ? static_cast<size_t>(__ldg(shared_base)) : static_cast<size_t>(T) * k;
  float a0[8], a1[8];
  if (has_shared) {
    const __nv_bfloat16* ys = Y + (R + t) * d;
    unpack8(__ldg(reinterpret_cast<const uint4*>(ys + c0)), a0);
    if (p1) unpack8(__ldg(reinterpret_cast<const uint4*>(ys + c1)), a1);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) a0[i] = a1[i] = 0.f;
  }
  const int32_t* rows = t2r + static_cast<size_t>(t) * k;
  const float* ws = w + static_cast<size_t>(t) * k;
  int j = 0;
  for (; j + 4 <= k; j += 4) {  // four rows x two pieces in flight
    uint4 r0[4], r1[4];
    float wj[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = __ldg(rows + j + u);
      // an overflowed slot (row < 0) contributes +0 * 0: the sum is unchanged
      const __nv_bfloat16* yr = Y + static_cast<size_t>(row < 0 ? 0 : row) * d;
      wj[u] = row < 0 ? 0.f : __ldg(ws + j + u);
      r0[u] = r1[u] = make_uint4(0, 0, 0, 0);
      if (row >= 0) {
        r0[u] = __ldg(reinterpret_cast<const uint4*>(yr + c0));
        if (p1) r1[u] = __ldg(reinterpret_cast<const uint4*>(yr + c1));
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[8];
      unpack8(r0[u], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) a0[i] = fmaf(wj[u], f[i], a0[i]);
      if (p1) {
        unpack8(r1[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) a1[i] = fmaf(wj[u], f[i], a1[i]);
      }
    }
  }
  for (; j < k; ++j) {
    const int row = __ldg(rows + j);
    if (row < 0) continue;  // overflowed its expert's capacity
    const __nv_bfloat16* yr = Y + static_cast<size_t>(row) * d;
    const float wj = __ldg(ws + j);
    float f[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(yr + c0)), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) a0[i] = fmaf(wj, f[i], a0[i]);
    if (p1) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(yr + c1)), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) a1[i] = fmaf(wj, f[i], a1[i]);
    }
  }
  OT* o = out + static_cast<size_t>(t) * d;
  store8(o + c0, a0);
  if (p1) store8(o + c1, a1);
}

// ---------------------------------------------------------------- gradient
//   dY[token_to_row[t, j]] = w[t, j] * dout[t],   dY[R + t] = dout[t] (shared),
//   dw[t, j] = <Y[token_to_row[t, j]], dout[t]>.
// Bound by memory: dout once, k rows of Y, k (+ 1) rows of dY.  One CTA a
// token, so that dout's row is read once and stays in registers while the k
// rows pass by it; each thread walks 16-byte pieces with eight rows in flight.
constexpr int kCombGradSlots = 8;

__device__ __forceinline__ void load_grad(const __nv_bfloat16* p, float (&g)[8]) {
  unpack8(__ldg(reinterpret_cast<const uint4*>(p)), g);
}
__device__ __forceinline__ void load_grad(const float* p, float (&g)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
}

// rows that this kernel reads once, and writes for another kernel to read
__device__ __forceinline__ uint4 load_once(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void store_once(__nv_bfloat16* p, const float (&f)[8]) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<uint4*>(h));
}

// S: slots of one sweep over the columns (1, 2, 4 or 8); more slots take more sweeps
template <typename GT, int S>
__global__ void __launch_bounds__(256) combine_backward_kernel(
    const GT* __restrict__ dout, const __nv_bfloat16* __restrict__ Y, const int32_t* __restrict__ t2r,
    const float* __restrict__ w, int has_shared, int T, int d, int k, const int32_t* __restrict__ shared_base,
    __nv_bfloat16* __restrict__ dY, float* __restrict__ dw) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float s_dot[8][S];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long rows = static_cast<long long>(T) * (k + (has_shared ? 1 : 0));
  const GT* g_row = dout + static_cast<size_t>(t) * d;
  __nv_bfloat16* shared_row = nullptr;
  if (has_shared && dY) {
    const long long r = (shared_base ? static_cast<long long>(__ldg(shared_base)) : static_cast<long long>(T) * k) + t;
    if (r >= 0 && r < rows) shared_row = dY + r * d;
  }
  for (int j0 = 0; j0 < k; j0 += S) {
    const int n = min(S, k - j0);
    long long row[S];
    float wj[S], dot[S];
#pragma unroll
    for (int u = 0; u < S; ++u) {
      row[u] = u < n ? __ldg(t2r + static_cast<size_t>(t) * k + j0 + u) : -1;
      if (row[u] >= rows) row[u] = -1;
      wj[u] = u < n ? __ldg(w + static_cast<size_t>(t) * k + j0 + u) : 0.f;
      dot[u] = 0.f;
    }
    for (int c = tid * 8; c < d; c += blockDim.x * 8) {
      float g[8];
      load_grad(g_row + c, g);
      uint4 y[S];
      if (dw) {
#pragma unroll
        for (int u = 0; u < S; ++u)
          y[u] = row[u] >= 0 ? load_once(Y + row[u] * d + c) : make_uint4(0, 0, 0, 0);
      }
      if (dY) {  // needs dout alone: these go out while the rows of Y come in
#pragma unroll
        for (int u = 0; u < S; ++u) {
          if (row[u] < 0) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = wj[u] * g[i];
          store_once(dY + row[u] * d + c, v);
        }
        if (shared_row && j0 == 0) store_once(shared_row + c, g);
      }
      if (dw) {
#pragma unroll
        for (int u = 0; u < S; ++u) {
          float f[8];
          unpack8(y[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[u] = fmaf(f[i], g[i], dot[u]);
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int u = 0; u < S; ++u)
      for (int o = 16; o; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
    if (lane == 0) {
#pragma unroll
      for (int u = 0; u < S; ++u) s_dot[warp][u] = dot[u];
    }
    __syncthreads();
    if (tid < n) {
      float all = 0.f;
      for (int v = 0; v < static_cast<int>(blockDim.x) / 32; ++v) all += s_dot[v][tid];
      // a slot without a row reached nothing, whatever dout holds
      const int r = __ldg(t2r + static_cast<size_t>(t) * k + j0 + tid);
      dw[static_cast<size_t>(t) * k + j0 + tid] = r >= 0 && r < rows ? all : 0.f;
    }
    __syncthreads();
  }
}

template <typename GT>
int launch_combine_grad(const GT* dout, const __nv_bfloat16* y, const int32_t* t2r, const float* w, int has_shared,
                        int T, int d, int k, const int32_t* shared_base, __nv_bfloat16* dy, float* dw,
                        cudaStream_t s) {
  // threads that share a row's 16-byte pieces evenly: 7168 columns are 4 rounds
  // of 224 threads, where 256 threads would sit half idle in the fourth
  const int pieces = d / 8, rounds = (pieces + 255) / 256, per = (pieces + rounds - 1) / rounds;
  const dim3 grid(T), block((per + 31) / 32 * 32);
  const char* where = "combine_backward_kernel";
  if (k == 1)
    return launch_pdl(where, combine_backward_kernel<GT, 1>, grid, block, 0, s, dout, y, t2r, w, has_shared, T, d, k,
                      shared_base, dy, dw);
  if (k == 2)
    return launch_pdl(where, combine_backward_kernel<GT, 2>, grid, block, 0, s, dout, y, t2r, w, has_shared, T, d, k,
                      shared_base, dy, dw);
  if (k <= 4)
    return launch_pdl(where, combine_backward_kernel<GT, 4>, grid, block, 0, s, dout, y, t2r, w, has_shared, T, d, k,
                      shared_base, dy, dw);
  return launch_pdl(where, combine_backward_kernel<GT, kCombGradSlots>, grid, block, 0, s, dout, y, t2r, w, has_shared,
                    T, d, k, shared_base, dy, dw);
}

}  // namespace

int launch_combine_backward(const void* dout, int dout_dtype, const void* Y, const int32_t* t2r, const float* w,
                            int has_shared, int T, int d, int k, const int32_t* shared_base, void* dY, float* dw,
                            cudaStream_t s) {
  if (T == 0) return MOE_OK;
  const __nv_bfloat16* y = static_cast<const __nv_bfloat16*>(Y);
  __nv_bfloat16* dy = static_cast<__nv_bfloat16*>(dY);
  if (dout_dtype == MOE_F32)
    return launch_combine_grad(static_cast<const float*>(dout), y, t2r, w, has_shared, T, d, k, shared_base, dy, dw,
                               s);
  return launch_combine_grad(static_cast<const __nv_bfloat16*>(dout), y, t2r, w, has_shared, T, d, k, shared_base, dy,
                             dw, s);
}

int launch_combine(const void* Y, const int32_t* t2r, const float* w, int has_shared, int T, int d, int k,
                   void* out, int out_dtype, cudaStream_t s, const int32_t* shared_base) {
  if (T == 0) return MOE_OK;
  const __nv_bfloat16* y = static_cast<const __nv_bfloat16*>(Y);
  const dim3 grid(T, (d + kCombCols - 1) / kCombCols);
  if (out_dtype == MOE_F32)
    return launch_pdl(__func__, combine_kernel<float>, grid, dim3(kCombThreads), 0, s, y, t2r, w, has_shared, T, d, k,
                      static_cast<float*>(out), shared_base);
  return launch_pdl(__func__, combine_kernel<__nv_bfloat16>, grid, dim3(kCombThreads), 0, s, y, t2r, w, has_shared, T,
                    d, k, static_cast<__nv_bfloat16*>(out), shared_base);
}

}  // namespace moe
