// Gradients of the low-rank adapters, out = base + s_a (x A_a^T) B_a^T, given
// dC = d out and the forward's h = x A^T:
//   dh[r] = s_a dC[r] B_a          dB_a = s_a sum_r dC[r]^T h[r]
//   dx[r] = dx_base[r] + dh[r] A_a  dA_a = sum_r dh[r]^T x[r]
// over the rows r of adapter a.  One streaming pass over dC gives dh and dB, one
// over x gives dA, and the forward's second product, with A in the place of B,
// gives dx.  Each wide operand is read once; what several CTAs add to is
// written as partial sums and added here in a fixed order, so results do not
// vary from run to run.
#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

// dh = the slices' sum, for the rows that have an adapter
__global__ void __launch_bounds__(256) dh_reduce_kernel(const float* __restrict__ part, const int32_t* __restrict__ off,
                                                        int n, int rows, int R, int slices, float* __restrict__ dh) {
  pdl_wait();
  pdl_launch_dependents();
  const size_t all = static_cast<size_t>(rows) * R, used = static_cast<size_t>(held_offset(off, n, rows, n)) * R;
  for (size_t i = (static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 4; i < used;
       i += static_cast<size_t>(gridDim.x) * blockDim.x * 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < slices; ++s) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(part + s * all + i));
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    *reinterpret_cast<float4*>(dh + i) = v;
  }
}

struct GradReduceArgs {
  const float* part[2];   // of dA, dB: partial sums by chunk slot
  void* grad[2];          // nullptr: not wanted
  size_t size[2];         // values of one adapter
  int chunk[2];
  const int32_t* offsets;
  int n, rows;
};

// Adapter blockIdx.y's gradient blockIdx.z (0 dA, 1 dB): the sum over its
// chunks, 0 where it has no rows.  That of a single chunk is there already.
template <typename GT>
__global__ void __launch_bounds__(256) grad_reduce_kernel(const GradReduceArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int a = blockIdx.y, z = blockIdx.z, chunk = p.chunk[z];
  const int b = held_offset(p.offsets, p.n, p.rows, a), e = held_offset(p.offsets, p.n, p.rows, a + 1);
  const int chunks = e > b ? (e - b + chunk - 1) / chunk : 0;
  if (chunks == 1 || !p.grad[z]) return;
  const size_t size = p.size[z];
  const float* part = p.part[z] + static_cast<size_t>(b / chunk + a) * size;
  GT* grad = static_cast<GT*>(p.grad[z]) + a * size;
  for (size_t i = (static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 4; i < size;
       i += static_cast<size_t>(gridDim.x) * blockDim.x * 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < chunks; ++s) {
      const float4 u = __ldcs(reinterpret_cast<const float4*>(part + s * size + i));
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    if constexpr (sizeof(GT) == 4)
      *reinterpret_cast<float4*>(grad + i) = v;
    else
      *reinterpret_cast<uint2*>(grad + i) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
  }
}

// Rows and columns of a CTA of a pass over [rows, W].  An estimate of its time
// from the traffic: the tiles of the busiest SM, each CTA's start and end, and
// the partial sums, which several chunks of an adapter (dA, dB) and several
// slices of a row (dh) write and read again.  How the rows are spread over the
// adapters is on the device; an even spread is taken.
struct Split {
  int chunk, cols;
};
Split split_for(int rows, int n, int W, int R, bool proj) {
  const int max_cols = lora_stream_max_cols(R), per_sm = R <= 32 ? 2 : 1;
  const double ns_per_byte = 148.0 / 6400.0, per_adapter = static_cast<double>(rows) / n;
  Split best{128, 128};
  double best_ns = 1e30;
  for (int cols = 128; cols <= max_cols; cols *= 2)
    for (int chunk = 128; chunk <= 4096; chunk *= 2) {
      const double each = per_adapter < chunk ? 1.0 : per_adapter / chunk + 0.5;
      const double ctas = n * each * ((W + cols - 1) / cols);
      const double waves = ctas / (num_sms() * per_sm) < 1.0 ? 1.0 : ctas / (num_sms() * per_sm) + 0.5;
      const double tile = 128.0 * 128 * 2 * ns_per_byte * per_sm;
      const double used = per_adapter < chunk ? per_adapter : chunk;
      const double cta = (used + 127) / 128 * (cols / 128) * tile + 4000;
      double partial = each > 1.0 ? 8.0 * n * each * W * R : 0.0;
      if (proj) partial += 8.0 * rows * R * ((W + cols - 1) / cols);
      const double ns = waves * cta + partial * ns_per_byte / num_sms() * 0.7;
      if (ns < best_ns) best_ns = ns, best = {chunk, cols};
    }
  return best;
}

struct BackwardLayout {
  Split dc, x;
  size_t dh_part, dh, pA, pB, total;
};
BackwardLayout backward_layout(int rows, int n, int d, int N, int R) {
  BackwardLayout L{};
  size_t off = 256;   // the status word
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  L.dc = split_for(rows, n, N, R, true);
  L.x = split_for(rows, n, d, R, false);
  const size_t slices = (N + L.dc.cols - 1) / L.dc.cols;
  L.dh_part = take(slices * rows * R * 4);
  L.dh = take(static_cast<size_t>(rows) * R * 4);
  L.pA = take((static_cast<size_t>(rows) / L.x.chunk + n) * R * d * 4);
  L.pB = take((static_cast<size_t>(rows) / L.dc.chunk + n) * R * N * 4);
  L.total = off;
  return L;
}

}  // namespace

size_t lora_backward_workspace_bytes(int rows, int n, int d, int N, int R) {
  return backward_layout(rows, n, d, N, R).total;
}

int launch_lora_backward(const LoraBackwardArgs& q, cudaStream_t s) {
  const BackwardLayout L = backward_layout(q.rows, q.n, q.d, q.N, q.R);
  char* ws = static_cast<char*>(q.ws);
  float* dh_part = reinterpret_cast<float*>(ws + L.dh_part);
  float* dh = reinterpret_cast<float*>(ws + L.dh);
  const bool need_dh = q.dx || q.dA;
  if (q.rows == 0) {
    MOE_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(int), s));   // MOE_OK
  } else {
    StreamArgs p{};
    p.X = static_cast<const __nv_bfloat16*>(q.dC), p.M = static_cast<const __nv_bfloat16*>(q.B), p.V = q.h;
    p.scale = q.scale, p.offsets = q.offsets, p.order = q.order, p.n = q.n, p.rows = q.rows, p.W = q.N, p.R = q.R;
    p.chunk = L.dc.chunk, p.cols = L.dc.cols;
    p.proj = need_dh ? dh_part : nullptr;
    p.part = reinterpret_cast<float*>(ws + L.pB), p.grad = q.dB, p.grad_f32 = q.grad_dtype == MOE_F32;
    p.status = reinterpret_cast<int*>(ws);
    int st = launch_lora_stream(p, kStreamBoth, s);
    if (st != MOE_OK) return st;
    const int slices = (q.N + L.dc.cols - 1) / L.dc.cols;
    if (need_dh && slices > 1) {
      const size_t quads = static_cast<size_t>(q.rows) * q.R / 4;
      const unsigned grid = static_cast<unsigned>(quads / 256 + 1 < 1184 ? quads / 256 + 1 : 1184);
      st = launch_pdl("dh_reduce_kernel", dh_reduce_kernel, dim3(grid), dim3(256), 0, s,
                      static_cast<const float*>(dh_part), q.offsets, q.n, q.rows, q.R, slices, dh);
      if (st != MOE_OK) return st;
    } else {
      dh = dh_part;
    }
    if (q.dA) {
      p.X = static_cast<const __nv_bfloat16*>(q.x), p.M = nullptr, p.V = dh, p.scale = nullptr, p.W = q.d;
      p.chunk = L.x.chunk, p.cols = L.x.cols, p.proj = nullptr;
      p.part = reinterpret_cast<float*>(ws + L.pA), p.grad = q.dA;
      st = launch_lora_stream(p, kStreamGrad, s);
      if (st != MOE_OK) return st;
    }
    if (q.dx) {
      ExpandArgs e{};
      e.h = dh, e.M = static_cast<const __nv_bfloat16*>(q.A), e.offsets = q.offsets, e.order = q.order;
      e.n = q.n, e.rows = q.rows, e.N = q.d, e.R = q.R, e.base = q.dx_base, e.out = q.dx;
      e.status = reinterpret_cast<int*>(ws);
      st = launch_lora_expand(e, true, q.dx_dtype, s);
      if (st != MOE_OK) return st;
    }
  }
  if (!q.dA && !q.dB) return MOE_OK;
  GradReduceArgs r{};
  r.part[0] = reinterpret_cast<float*>(ws + L.pA), r.part[1] = reinterpret_cast<float*>(ws + L.pB);
  r.grad[0] = q.dA, r.grad[1] = q.dB;
  r.size[0] = static_cast<size_t>(q.R) * q.d, r.size[1] = static_cast<size_t>(q.R) * q.N;
  r.chunk[0] = L.x.chunk, r.chunk[1] = L.dc.chunk;
  r.offsets = q.offsets, r.n = q.n, r.rows = q.rows;
  // eight blocks to an SM over all the adapters, no more than one pass needs
  const size_t need = (r.size[0] > r.size[1] ? r.size[0] : r.size[1]) / 1024 + 1, share = 8ul * num_sms() / q.n + 1;
  const dim3 grid(static_cast<unsigned>(need < share ? need : share), q.n, 2);
  return launch_pdl("grad_reduce_kernel", q.grad_dtype == MOE_F32 ? grad_reduce_kernel<float> : grad_reduce_kernel<__nv_bfloat16>,
                    grid, dim3(256), 0, s, r);
}

}  // namespace moe
