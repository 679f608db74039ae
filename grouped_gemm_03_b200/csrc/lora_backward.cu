// Gradients of the low-rank adapters, out = base + s_a (x A_a^T) B_a^T, given
// dC = d out and the forward's h = x A^T:
//   dh[r] = s_a dC[r] B_a          dB_a = s_a sum_r dC[r]^T h[r]
//   dx[r] = dx_base[r] + dh[r] A_a  dA_a = sum_r dh[r]^T x[r]
// over the rows r of adapter a.  Two passes, each over one wide operand once:
// dC gives dh and dB, then x gives dA while dh gives dx.  A pass splits the
// rows of an adapter into chunks and the columns into slices; what several
// blocks sum to is written as partial sums and added in a fixed order, so
// results do not vary from run to run.
//
// h and dh enter the products as two bf16 terms (hi + lo): the sums they go
// into are fp32, and one term's rounding would be the largest error in them.
#include "common.cuh"
#include "lora.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 512;        // rows of one partial sum
constexpr int kStep = 128;         // rows of one tile
constexpr int kCols = 128;         // columns of one tile
constexpr int kTileStride = kCols + 8;

template <int RP>
struct GradTile {
  static constexpr int NB = RP == 16 ? 4 : RP == 32 ? 2 : 1;  // tiles of columns a block walks
  static constexpr int VS = RP + 8;
  static constexpr int TILE = kStep * kTileStride * 2;
  static constexpr int TERMS = 2 * kStep * VS * 2;
  // B rows [NB * 128][RP + 8], or A rows [RP][NB * 128 + 8]
  static constexpr int WIDE0 = NB * kCols * VS * 2, WIDE1 = RP * (NB * kCols + 8) * 2;
  static constexpr int SMEM = 2 * TILE + TERMS + (WIDE0 > WIDE1 ? WIDE0 : WIDE1);
};

struct GradArgs {
  const __nv_bfloat16* X;   // dC [rows, W] or x
  const float* V;           // h [rows, R] by row, or dh [rows, R] by position
  const __nv_bfloat16* M;   // B [n, W, R] or A [n, R, W]
  const float* scale;
  const int32_t* offsets;
  const int32_t* order;
  int n, rows, W, R;
  float* dh_part;           // pass over dC: [slices][rows][R] by position
  float* part;              // [slots][W][R] (dB) or [slots][R][W] (dA); nullptr: not wanted
  const void* dx_base;
  void* dx;                 // nullptr: not wanted
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p)))
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p)))
               : "memory");
}
// 16 bytes global -> shared, or 16 zero bytes when !in
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void load2(const __nv_bfloat16* p, float& a, float& b) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  a = __uint_as_float(v << 16), b = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ void load2(const float* p, float& a, float& b) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  a = v.x, b = v.y;
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = pack2(a, b);
}
__device__ __forceinline__ void store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }

// DC: the pass over dC (dh partials, dB); else the pass over x (dx, dA).
template <int RP, bool DC, typename OT>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(const GradArgs p) {
  using L = GradTile<RP>;
  constexpr int NB = L::NB, VS = L::VS;
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint8_t s_raw[];
  __nv_bfloat16* s_tile = reinterpret_cast<__nv_bfloat16*>(s_raw);                       // [2][128][136]
  __nv_bfloat16* s_hi = reinterpret_cast<__nv_bfloat16*>(s_raw + 2 * L::TILE);           // [128][VS]
  __nv_bfloat16* s_lo = s_hi + kStep * VS;
  __nv_bfloat16* s_m = reinterpret_cast<__nv_bfloat16*>(s_raw + 2 * L::TILE + L::TERMS);
  __shared__ int s_row[2][kStep];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  int a, start, end;
  if (!find_tile<kChunk>(p.offsets, p.n, p.rows, blockIdx.x, a, start, end)) return;
  const int col0 = blockIdx.y * NB * kCols;
  const int blocks = min(NB, (p.W - col0 + kCols - 1) / kCols);
  const int W = p.W, R = p.R;
  OT* dx = static_cast<OT*>(p.dx);
  const OT* dx_base = static_cast<const OT*>(p.dx_base);

  if (a == p.n) {  // rows without an adapter: their gradient passes by
    if (DC || !dx || dx == dx_base) return;
    const int w8 = min(NB * kCols, W - col0) / 8;
    for (int i = tid; i < (end - start) * w8; i += kThreads) {
      const int r = p.order[start + i / w8];
      if (r < 0 || r >= p.rows) continue;
      const size_t o = static_cast<size_t>(r) * W + col0 + i % w8 * 8;
      float v[8] = {};
      if (dx_base) load8(dx_base + o, v);
      store8(dx + o, v);
    }
    return;
  }

  // the adapter's slice of B (rows: columns of dC) or A (rows: ranks)
  if (DC) {
    for (int i = tid; i < NB * kCols * (RP / 8); i += kThreads) {
      const int r = i / (RP / 8), j = i % (RP / 8) * 8;
      cp_async16(s_m + r * VS + j, p.M + (static_cast<size_t>(a) * W + min(col0 + r, W - 1)) * R + min(j, R - 8),
                 col0 + r < W && j < R);
    }
  } else {
    for (int i = tid; i < RP * NB * (kCols / 8); i += kThreads) {
      const int j = i / (NB * kCols / 8), k = i % (NB * kCols / 8) * 8;
      cp_async16(s_m + j * (NB * kCols + 8) + k,
                 p.M + (static_cast<size_t>(a) * R + min(j, R - 1)) * W + min(col0 + k, W - 8), j < R && col0 + k < W);
    }
  }

  const float sc = p.scale ? __ldg(p.scale + a) : 1.f;
  const int steps = (end - start + kStep - 1) / kStep;
  auto rows_of = [&](int step) {
    if (tid < kStep) {
      const int at = start + step * kStep + tid;
      const int r = at < end ? p.order[at] : -1;
      s_row[step & 1][tid] = r >= 0 && r < p.rows ? r : -1;
    }
  };
  auto load_tile = [&](int it) {  // tile it % blocks of row step it / blocks
    const int step = it / blocks, col = col0 + it % blocks * kCols;
    __nv_bfloat16* t = s_tile + (it & 1) * (kStep * kTileStride);
#pragma unroll
    for (int i = tid; i < kStep * (kCols / 8); i += kThreads) {
      const int m = i / (kCols / 8), k = i % (kCols / 8) * 8;
      const int r = s_row[step & 1][m];
      const bool in = r >= 0 && col + k < W;
      cp_async16(t + m * kTileStride + k, p.X + (in ? static_cast<size_t>(r) * W + col + k : 0), in);
    }
  };

  float G[NB][RP / 8][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < RP / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) G[b][j][i] = 0.f;

  rows_of(0);
  __syncthreads();
  load_tile(0);
  cp_async_commit();
  for (int step = 0; step < steps; ++step) {
    // the step's h or dh rows in two terms
    for (int i = tid; i < kStep * (RP / 4); i += kThreads) {
      const int m = i / (RP / 4), j = i % (RP / 4) * 4;
      const int at = start + step * kStep + m;
      const int r = DC ? s_row[step & 1][m] : (at < end ? at : -1);
      const float4 v = r >= 0 && j < R ? __ldg(reinterpret_cast<const float4*>(p.V + static_cast<size_t>(r) * R + j))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
      split_store(s_hi + m * VS + j, s_lo + m * VS + j, v, DC ? sc : 1.f);
    }
    if (step + 1 < steps) rows_of(step + 1);
    float dh[RP / 8][4];
#pragma unroll
    for (int j = 0; j < RP / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) dh[j][i] = 0.f;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b >= blocks) break;
      const int it = step * blocks + b;
      if (it + 1 < steps * blocks) {
        load_tile(it + 1);
        cp_async_commit();
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      __syncthreads();
      const __nv_bfloat16* t = s_tile + (it & 1) * (kStep * kTileStride);
      if (DC) {
#pragma unroll
        for (int kk = 0; kk < kCols / 16; ++kk) {
          uint32_t x[4];
          ldsm4(x, t + (warp * 16 + (lane & 15)) * kTileStride + kk * 16 + (lane >> 4) * 8);
#pragma unroll
          for (int j = 0; j < RP / 16; ++j) {
            uint32_t m[4];
            ldsm4t(m, s_m + (b * kCols + kk * 16 + (lane & 15)) * VS + j * 16 + (lane >> 4) * 8);
            mma16816(dh[2 * j], x[0], x[1], x[2], x[3], m[0], m[1]);
            mma16816(dh[2 * j + 1], x[0], x[1], x[2], x[3], m[2], m[3]);
          }
        }
      } else if (dx) {
        uint32_t vh[RP / 16][4], vl[RP / 16][4];
#pragma unroll
        for (int j = 0; j < RP / 16; ++j) {
          ldsm4(vh[j], s_hi + (warp * 16 + (lane & 15)) * VS + j * 16 + (lane >> 4) * 8);
          ldsm4(vl[j], s_lo + (warp * 16 + (lane & 15)) * VS + j * 16 + (lane >> 4) * 8);
        }
        const int r0 = s_row[step & 1][warp * 16 + g], r1 = s_row[step & 1][warp * 16 + g + 8];
        const int col = col0 + b * kCols;
#pragma unroll
        for (int nb = 0; nb < kCols / 16; ++nb) {
          float acc[2][4] = {};
#pragma unroll
          for (int j = 0; j < RP / 16; ++j) {
            uint32_t m[4];
            ldsm4t(m, s_m + (j * 16 + (lane & 15)) * (NB * kCols + 8) + b * kCols + nb * 16 + (lane >> 4) * 8);
            mma16816(acc[0], vl[j][0], vl[j][1], vl[j][2], vl[j][3], m[0], m[1]);
            mma16816(acc[1], vl[j][0], vl[j][1], vl[j][2], vl[j][3], m[2], m[3]);
            mma16816(acc[0], vh[j][0], vh[j][1], vh[j][2], vh[j][3], m[0], m[1]);
            mma16816(acc[1], vh[j][0], vh[j][1], vh[j][2], vh[j][3], m[2], m[3]);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int k = col + nb * 16 + q * 8 + 2 * c;
            if (k >= W) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = h ? r1 : r0;
              if (r < 0) continue;
              const size_t o = static_cast<size_t>(r) * W + k;
              float u = 0.f, v = 0.f;
              if (dx_base) load2(dx_base + o, u, v);
              store2(dx + o, u + acc[q][2 * h], v + acc[q][2 * h + 1]);
            }
          }
        }
      }
      if (p.part) {
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk) {
          uint32_t x[4];  // the tile's transpose: columns as rows
          ldsm4t(x, t + (kk * 16 + (lane & 7) + (lane >> 4) * 8) * kTileStride + warp * 16 + ((lane >> 3) & 1) * 8);
#pragma unroll
          for (int j = 0; j < RP / 16; ++j) {
            uint32_t v[4];
            ldsm4t(v, s_lo + (kk * 16 + (lane & 15)) * VS + j * 16 + (lane >> 4) * 8);
            mma16816(G[b][2 * j], x[0], x[1], x[2], x[3], v[0], v[1]);
            mma16816(G[b][2 * j + 1], x[0], x[1], x[2], x[3], v[2], v[3]);
            ldsm4t(v, s_hi + (kk * 16 + (lane & 15)) * VS + j * 16 + (lane >> 4) * 8);
            mma16816(G[b][2 * j], x[0], x[1], x[2], x[3], v[0], v[1]);
            mma16816(G[b][2 * j + 1], x[0], x[1], x[2], x[3], v[2], v[3]);
          }
        }
      }
      __syncthreads();
    }
    if (DC && p.dh_part) {
      const int m0 = start + step * kStep + warp * 16 + g;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = m0 + 8 * h;
        if (at >= end) continue;
        float* o = p.dh_part + (static_cast<size_t>(blockIdx.y) * p.rows + at) * R;
#pragma unroll
        for (int j = 0; j < RP / 8; ++j)
          if (j * 8 < R) store2(o + j * 8 + 2 * c, sc * dh[j][2 * h], sc * dh[j][2 * h + 1]);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = col0 + b * kCols + warp * 16 + g + 8 * h;
      if (k >= W) continue;
#pragma unroll
      for (int j = 0; j < RP / 8; ++j) {
        if (j * 8 >= R) continue;
        const int j0 = j * 8 + 2 * c;
        if (DC) {
          store2(p.part + (static_cast<size_t>(blockIdx.x) * W + k) * R + j0, G[b][j][2 * h], G[b][j][2 * h + 1]);
        } else {
          float* o = p.part + (static_cast<size_t>(blockIdx.x) * R + j0) * W + k;
          o[0] = G[b][j][2 * h];
          o[W] = G[b][j][2 * h + 1];
        }
      }
    }
  }
}

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

// Adapter blockIdx.y's gradients: the sum over its chunks, 0 where it has no rows.
template <typename GT>
__global__ void __launch_bounds__(256) grad_reduce_kernel(const float* __restrict__ pA, const float* __restrict__ pB,
                                                          const int32_t* __restrict__ off, int n, int rows,
                                                          size_t sizeA, size_t sizeB, GT* __restrict__ dA,
                                                          GT* __restrict__ dB) {
  pdl_wait();
  pdl_launch_dependents();
  const int a = blockIdx.y;
  const int b = held_offset(off, n, rows, a), e = held_offset(off, n, rows, a + 1);
  const size_t first = b / kChunk + a;
  const int chunks = e > b ? (e - b + kChunk - 1) / kChunk : 0;
  const size_t na = dA ? sizeA : 0, total = na + (dB ? sizeB : 0);
  for (size_t i = (static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x * 8) {
    const bool isA = i < na;
    const size_t k = isA ? i : i - na, size = isA ? sizeA : sizeB;
    const float* p = (isA ? pA : pB) + first * size + k;
    float v[8] = {};
    for (int s = 0; s < chunks; ++s) {
      float u[8];
      load8(p + s * size, u);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += u[q];
    }
    store8((isA ? dA : dB) + static_cast<size_t>(a) * size + k, v);
  }
}

template <int RP, bool DC, typename OT>
int launch_grad(const GradArgs& p, cudaStream_t s) {
  using L = GradTile<RP>;
  static std::atomic<uint64_t> done{0};
  auto kernel = grad_kernel<RP, DC, OT>;
  const int st = allow_smem(done, kernel, L::SMEM);
  if (st != MOE_OK) return st;
  const int cols = L::NB * kCols;
  return launch_pdl("grad_kernel", kernel, dim3(static_cast<unsigned>(tile_slots<kChunk>(p.rows, p.n)), (p.W + cols - 1) / cols),
                    dim3(kThreads), L::SMEM, s, p);
}

int slice_cols(int R) {
  return kCols * (R <= 16 ? GradTile<16>::NB : R <= 32 ? GradTile<32>::NB : R <= 64 ? GradTile<64>::NB : GradTile<128>::NB);
}

template <bool DC, typename OT>
int launch_grad_rank(const GradArgs& p, cudaStream_t s) {
  if (p.R <= 16) return launch_grad<16, DC, OT>(p, s);
  if (p.R <= 32) return launch_grad<32, DC, OT>(p, s);
  if (p.R <= 64) return launch_grad<64, DC, OT>(p, s);
  return launch_grad<128, DC, OT>(p, s);
}

struct BackwardLayout {
  size_t dh_part, dh, pA, pB, total;
};
BackwardLayout backward_layout(int rows, int n, int d, int N, int R) {
  BackwardLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t slices = (N + slice_cols(R) - 1) / slice_cols(R);
  const size_t slots = tile_slots<kChunk>(rows, n);
  L.dh_part = take(slices * rows * R * 4);
  L.dh = take(static_cast<size_t>(rows) * R * 4);
  L.pA = take(slots * R * d * 4);
  L.pB = take(slots * R * N * 4);
  L.total = off + 256;
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
  float* pA = reinterpret_cast<float*>(ws + L.pA);
  float* pB = reinterpret_cast<float*>(ws + L.pB);
  if (q.rows > 0) {
    GradArgs p{};
    p.scale = q.scale, p.offsets = q.offsets, p.order = q.order, p.n = q.n, p.rows = q.rows, p.R = q.R;
    p.X = static_cast<const __nv_bfloat16*>(q.dC), p.V = q.h, p.M = static_cast<const __nv_bfloat16*>(q.B), p.W = q.N;
    const bool need_dh = q.dx || q.dA;
    p.dh_part = need_dh ? dh_part : nullptr;
    p.part = q.dB ? pB : nullptr;
    int st = launch_grad_rank<true, float>(p, s);
    if (st != MOE_OK) return st;
    if (need_dh) {
      const int slices = (q.N + slice_cols(q.R) - 1) / slice_cols(q.R);
      const size_t quads = static_cast<size_t>(q.rows) * q.R / 4;
      const unsigned grid = static_cast<unsigned>(quads / 256 + 1 < 1184 ? quads / 256 + 1 : 1184);
      st = launch_pdl("dh_reduce_kernel", dh_reduce_kernel, dim3(grid), dim3(256), 0, s,
                      static_cast<const float*>(dh_part), q.offsets, q.n, q.rows, q.R, slices, dh);
      if (st != MOE_OK) return st;
      p.X = static_cast<const __nv_bfloat16*>(q.x), p.V = dh, p.M = static_cast<const __nv_bfloat16*>(q.A), p.W = q.d;
      p.dh_part = nullptr;
      p.part = q.dA ? pA : nullptr;
      p.dx_base = q.dx_base, p.dx = q.dx;
      st = q.dx_dtype == MOE_F32 ? launch_grad_rank<false, float>(p, s) : launch_grad_rank<false, __nv_bfloat16>(p, s);
      if (st != MOE_OK) return st;
    }
  }
  if (!q.dA && !q.dB) return MOE_OK;
  const size_t sizeA = static_cast<size_t>(q.R) * q.d, sizeB = static_cast<size_t>(q.R) * q.N;
  const size_t blocks = (sizeA + sizeB) / (256 * 8) + 1;
  const dim3 grid(static_cast<unsigned>(blocks < 1024 ? blocks : 1024), q.n);
  if (q.grad_dtype == MOE_F32)
    return launch_pdl("grad_reduce_kernel", grad_reduce_kernel<float>, grid, dim3(256), 0, s,
                      static_cast<const float*>(pA), static_cast<const float*>(pB), q.offsets, q.n, q.rows, sizeA,
                      sizeB, static_cast<float*>(q.dA), static_cast<float*>(q.dB));
  return launch_pdl("grad_reduce_kernel", grad_reduce_kernel<__nv_bfloat16>, grid, dim3(256), 0, s,
                    static_cast<const float*>(pA), static_cast<const float*>(pB), q.offsets, q.n, q.rows, sizeA, sizeB,
                    static_cast<__nv_bfloat16*>(q.dA), static_cast<__nv_bfloat16*>(q.dB));
}

}  // namespace moe
