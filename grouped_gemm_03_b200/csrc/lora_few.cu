// The adapters' gradients where an adapter has few rows (a token or so to a
// request), in one launch:
//   dh[r] = s_a dC[r] B_a           dB_a = s_a sum_r dC[r]^T h[r]
//   dx[r] = dx_base[r] + dh[r] A_a   dA_a = sum_r dh[r]^T x[r]
// A cluster of up to eight CTAs shares a tile of up to 16 rows of one adapter.
// CTA q takes the q-th slice of dC's columns: a warp holds the rows' h in
// registers, walks the columns, reads a column's ranks of B, adds to its share
// of dh and writes the column's ranks of dB.  The shares meet through
// distributed shared memory in rank order; then CTA q takes the q-th slice of
// x's columns, a lane two of them: rank by rank it reads A, adds to dx and writes
// dA.  All in fp32 multiply-adds, for 4 rows or 16, so nothing is split into
// terms; B's and A's next ranks are in flight while these are worked on.
//
// The least it has to do is to write dA and dB, 4 R (d + N) bytes an adapter;
// beside that it is bound by latency (100 rows of 100 adapters, rank 64, 2048
// and 2048 columns: 61 us, 105 MB of gradients; 11 warps to an SM keep its issue
// slots 41 % busy and the shared memory's path 20 %).  The tensor-core passes
// start a CTA and move 128 rows, most of them zeros, for each 256 columns of an
// adapter: 133 us there.  few_rows() in lora_backward.cu has more of both.
#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;

__device__ __forceinline__ void widen(uint32_t v, float& a, float& b) {
  a = __uint_as_float(v << 16), b = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  float2 f;
  widen(*reinterpret_cast<const uint32_t*>(p), f.x, f.y);
  return f;
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) { *reinterpret_cast<uint32_t*>(p) = pack2(a, b); }
__device__ __forceinline__ void store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
// a gradient's pair of values, of its partial sums or of the type it is wanted in
__device__ __forceinline__ void store_grad(float* part, void* grad, bool f32, size_t o, float a, float b) {
  if (part) store2(part + o, a, b);
  else if (f32) store2(static_cast<float*>(grad) + o, a, b);
  else store2(static_cast<__nv_bfloat16*>(grad) + o, a, b);
}

template <int RP>
struct FewTile {
  static constexpr int RL = RP <= 64 ? 2 : 4;       // ranks of a lane
  static constexpr int LN = RP / RL;                // lanes of a column's ranks
  static constexpr int NS = 32 / LN;                // columns of dC a warp takes at once
  static constexpr int CS = kRowsFew + 4;           // row stride of the staged columns: spreads the banks
  static constexpr int STAGE = 64 * CS * 4;         // a warp's 64 columns of dC
  static constexpr int DH = RP * kRowsFew * 4;      // [ranks][rows]
  static constexpr int SMEM = (kFewWarps * (STAGE > DH ? STAGE : DH)) + 2 * DH;
};

// rank-major [ranks][16]: MR rows of a rank
template <int MR>
__device__ __forceinline__ void load_rows(const float* p, float (&f)[MR]) {
#pragma unroll
  for (int i = 0; i < MR; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
  }
}

// dC's slice: dB's columns out, the warp's share of dh to `share` [ranks][16]
template <int RP, int MR>
__device__ __forceinline__ void few_columns(const LoraBackwardArgs& p, int a, const int* s_row, float sc, float* stage,
                                            float* share, int n0, int n1, float* part) {
  using F = FewTile<RP>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, N = p.N, R = p.R;
  const int rank = lane % F::LN * F::RL, sub = lane / F::LN;
  const bool want_dh = p.dx || p.dA, in = rank < R;
  const __nv_bfloat16* dC = static_cast<const __nv_bfloat16*>(p.dC);
  const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(p.B) + static_cast<size_t>(a) * N * R;
  float h[F::RL][MR], dh[F::RL][MR];
#pragma unroll
  for (int r = 0; r < MR; ++r)
#pragma unroll
    for (int u = 0; u < F::RL; u += 2) {
      const float2 v = p.dB && in && s_row[r] >= 0 ? load2(p.h + static_cast<size_t>(s_row[r]) * R + rank + u) : make_float2(0.f, 0.f);
      h[u][r] = v.x * sc, h[u + 1][r] = v.y * sc;
      dh[u][r] = dh[u + 1][r] = 0.f;
    }
  for (int c0 = n0 + warp * 64; c0 < n1; c0 += kFewWarps * 64) {
    const int col = c0 + lane * 2;
    float2 v[MR];
#pragma unroll
    for (int r = 0; r < MR; ++r)
      v[r] = col < n1 && s_row[r] >= 0 ? load2(dC + static_cast<size_t>(s_row[r]) * N + col) : make_float2(0.f, 0.f);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < MR; r += 4) {
      *reinterpret_cast<float4*>(stage + (lane * 2) * F::CS + r) = make_float4(v[r].x, v[r + 1].x, v[r + 2].x, v[r + 3].x);
      *reinterpret_cast<float4*>(stage + (lane * 2 + 1) * F::CS + r) = make_float4(v[r].y, v[r + 1].y, v[r + 2].y, v[r + 3].y);
    }
    __syncwarp();
    const int cols = min(64, n1 - c0);
    // B's ranks of the next BT columns are in flight together
    constexpr int BT = MR == 4 ? 16 : 8;
    for (int i0 = sub; i0 < cols; i0 += F::NS * BT) {
      uint32_t wb[BT][F::RL / 2];
#pragma unroll
      for (int t = 0; t < BT; ++t)
#pragma unroll
        for (int u = 0; u < F::RL / 2; ++u) {
          const int i = i0 + t * F::NS;
          wb[t][u] = want_dh && in && i < cols
                         ? __ldg(reinterpret_cast<const uint32_t*>(B + static_cast<size_t>(c0 + i) * R + rank + 2 * u)) : 0u;
        }
#pragma unroll
      for (int t = 0; t < BT; ++t) {
        const int i = i0 + t * F::NS;
        if (i >= cols) break;
        float c[MR], b[F::RL], g[F::RL];
        load_rows<MR>(stage + i * F::CS, c);
#pragma unroll
        for (int u = 0; u < F::RL; u += 2) widen(wb[t][u / 2], b[u], b[u + 1]);
#pragma unroll
        for (int u = 0; u < F::RL; ++u) {
          g[u] = 0.f;
#pragma unroll
          for (int r = 0; r < MR; ++r) {
            g[u] = fmaf(c[r], h[u][r], g[u]);
            dh[u][r] = fmaf(c[r], b[u], dh[u][r]);
          }
        }
        if (p.dB && in) {
          const size_t o = (part ? 0 : static_cast<size_t>(a) * N * R) + static_cast<size_t>(c0 + i) * R + rank;
#pragma unroll
          for (int u = 0; u < F::RL; u += 2) store_grad(part, p.dB, p.grad_dtype == MOE_F32, o + u, g[u], g[u + 1]);
        }
      }
    }
  }
  // the columns a warp took at once, then this lane's ranks (the stage is done with)
#pragma unroll
  for (int u = 0; u < F::RL; ++u)
#pragma unroll
    for (int r = 0; r < MR; ++r)
      for (int o = F::LN; o < 32; o *= 2) dh[u][r] += __shfl_xor_sync(0xffffffffu, dh[u][r], o);
  __syncwarp();
  if (sub == 0) {
#pragma unroll
    for (int u = 0; u < F::RL; ++u)
#pragma unroll
      for (int r = 0; r < kRowsFew; ++r) share[(rank + u) * kRowsFew + r] = r < MR ? dh[u][r < MR ? r : 0] : 0.f;
  }
}

// x's slice: dx and dA out
template <int RP, int MR, typename OT>
__device__ __forceinline__ void few_ranks(const LoraBackwardArgs& p, int a, const int* s_row, const float* s_dh, int k0, int k1,
                                          float* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = p.d, R = p.R;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(p.A) + static_cast<size_t>(a) * R * d;
  const OT* base = static_cast<const OT*>(p.dx_base);
  OT* dx = static_cast<OT*>(p.dx);
  for (int c0 = k0 + warp * 64; c0 < k1; c0 += kFewWarps * 64) {
    const int col = c0 + lane * 2;
    if (col >= k1) continue;
    float2 v[MR], y[MR];
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      const bool live = s_row[r] >= 0;
      const size_t o = static_cast<size_t>(live ? s_row[r] : 0) * d + col;
      v[r] = p.dA && live ? load2(x + o) : make_float2(0.f, 0.f);
      y[r] = dx && base && live ? load2(base + o) : make_float2(0.f, 0.f);
    }
    auto fetch = [&](int j0, uint32_t (&f)[8]) {   // A's next eight ranks; there are eight or none
#pragma unroll
      for (int t = 0; t < 8; ++t)
        f[t] = dx && j0 < R ? __ldg(reinterpret_cast<const uint32_t*>(A + static_cast<size_t>(j0 + t) * d + col)) : 0u;
    };
    uint32_t next[8];
    fetch(0, next);
    for (int j0 = 0; j0 < R; j0 += 8) {
      uint32_t now[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) now[t] = next[t];
      fetch(j0 + 8, next);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int j = j0 + t;
        float h[MR], b0, b1, g0 = 0.f, g1 = 0.f;
        load_rows<MR>(s_dh + j * kRowsFew, h);
        widen(now[t], b0, b1);
#pragma unroll
        for (int r = 0; r < MR; ++r) {
          g0 = fmaf(h[r], v[r].x, g0), g1 = fmaf(h[r], v[r].y, g1);
          y[r].x = fmaf(h[r], b0, y[r].x), y[r].y = fmaf(h[r], b1, y[r].y);
        }
        if (p.dA)
          store_grad(part, p.dA, p.grad_dtype == MOE_F32,
                     (part ? 0 : static_cast<size_t>(a) * R * d) + static_cast<size_t>(j) * d + col, g0, g1);
      }
    }
    if (dx) {
#pragma unroll
      for (int r = 0; r < MR; ++r)
        if (s_row[r] >= 0) store2(dx + static_cast<size_t>(s_row[r]) * d + col, y[r].x, y[r].y);
    }
  }
}

// partial sums of dA and dB, by part_slot with chunks of 16 rows
struct FewParts {
  float* A;
  float* B;
  int kslice, nslice;   // columns of x and dC a CTA of the cluster takes, multiples of 64
};

template <int RP, typename OT>
__global__ void __launch_bounds__(kFewThreads, RP <= 64 ? 2 : 1) lora_few_kernel(const LoraBackwardArgs p, const FewParts w) {
  using F = FewTile<RP>;
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint8_t s_raw[];
  float* s_part = reinterpret_cast<float*>(s_raw);             // [RP][16] this CTA's share of dh
  float* s_dh = s_part + F::DH / 4;                            // [RP][16] dh
  float* s_warp = s_dh + F::DH / 4;                            // by warp: 64 columns of dC, then its share
  __shared__ int s_row[kRowsFew];
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t CS = cluster_size(), rank = cluster_rank();
  const int d = p.d, N = p.N, R = p.R;
  const int n0 = min(N, static_cast<int>(rank) * w.nslice), n1 = min(N, n0 + w.nslice);
  const int k0 = min(d, static_cast<int>(rank) * w.kslice), k1 = min(d, k0 + w.kslice);
  if (blockIdx.x == 0 && tid == 0) *static_cast<int*>(p.ws) = MOE_OK;
  int a, start, end;
  if (!find_tile<kRowsFew>(p.offsets, p.n, p.rows, blockIdx.x / CS, a, start, end)) {   // the whole cluster leaves
    // the slot of an adapter without rows: its gradients are 0
    if (a < p.n && held_offset(p.offsets, p.n, p.rows, a) >= held_offset(p.offsets, p.n, p.rows, a + 1)) {
      const bool f32 = p.grad_dtype == MOE_F32;
      if (p.dB)
        for (int i = tid * 2; i < (n1 - n0) * R; i += kFewThreads * 2)
          store_grad(nullptr, p.dB, f32, (static_cast<size_t>(a) * N + n0) * R + i, 0.f, 0.f);
      if (p.dA)
        for (int j = 0; j < R; ++j)
          for (int k = k0 + tid * 2; k < k1; k += kFewThreads * 2)
            store_grad(nullptr, p.dA, f32, (static_cast<size_t>(a) * R + j) * d + k, 0.f, 0.f);
    }
    return;
  }
  if (tid < kRowsFew) {
    const int r = start + tid < end ? p.order[start + tid] : -1;
    s_row[tid] = r >= 0 && r < p.rows ? r : -1;
  }
  __syncthreads();
  if (a == p.n) {  // rows without an adapter: their gradient passes by
    OT* dx = static_cast<OT*>(p.dx);
    const OT* base = static_cast<const OT*>(p.dx_base);
    if (!dx || dx == base) return;
    const int w8 = (k1 - k0) / 8;
    for (int i = tid; i < kRowsFew * w8; i += kFewThreads) {
      const int r = s_row[i / w8];
      if (r < 0) continue;
      const size_t o = static_cast<size_t>(r) * d + k0 + i % w8 * 8;
      float v[8] = {};
      if (base) load8(base + o, v);
      store8(dx + o, v);
    }
    return;
  }
  const float sc = p.scale ? __ldg(p.scale + a) : 1.f;
  const int first = held_offset(p.offsets, p.n, p.rows, a), last = held_offset(p.offsets, p.n, p.rows, a + 1);
  const bool whole = last - first <= kRowsFew;   // no other tile adds to it
  const size_t slot = part_slot(first, kRowsFew) + (start - first) / kRowsFew;
  float* pB = whole ? nullptr : w.B + slot * N * R;
  float* pA = whole ? nullptr : w.A + slot * R * d;
  const bool few = end - start <= 4;
  float* mine = s_warp + warp * ((F::STAGE > F::DH ? F::STAGE : F::DH) / 4);
  if (few)
    few_columns<RP, 4>(p, a, s_row, sc, mine, mine, n0, n1, pB);
  else
    few_columns<RP, kRowsFew>(p, a, s_row, sc, mine, mine, n0, n1, pB);
  if (!p.dx && !p.dA) return;   // the whole cluster
  __syncthreads();
  for (int i = tid; i < RP * kRowsFew; i += kFewThreads) {
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < kFewWarps; ++u) v += s_warp[u * ((F::STAGE > F::DH ? F::STAGE : F::DH) / 4) + i];
    s_part[i] = v;
  }
  cluster_arrive();
  cluster_wait();
  for (int i = tid; i < RP * kRowsFew / 4; i += kFewThreads) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t q = 0; q < CS; ++q) {
      const float4 u = ld_cluster(reinterpret_cast<const float4*>(s_part) + i, q);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    reinterpret_cast<float4*>(s_dh)[i] = make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
  }
  cluster_arrive();   // done with the others' shared memory; waited for before this CTA ends
  __syncthreads();
  if (few)
    few_ranks<RP, 4, OT>(p, a, s_row, s_dh, k0, k1, pA);
  else
    few_ranks<RP, kRowsFew, OT>(p, a, s_row, s_dh, k0, k1, pA);
  __syncwarp();
  cluster_wait();
}

template <int RP, typename OT>
int launch_few(const LoraBackwardArgs& q, FewParts w, cudaStream_t s) {
  using F = FewTile<RP>;
  auto kernel = lora_few_kernel<RP, OT>;
  static std::atomic<uint64_t> done{0};
  const int st = allow_smem(done, kernel, F::SMEM);
  if (st != MOE_OK) return st;
  const long long half_full = q.rows / kRowsFew + q.n / 2, one_each = q.n < q.rows ? q.n : q.rows;
  static KnownClusters known;
  const int cs = cluster_for(known, kernel, kFewThreads, F::SMEM, half_full > one_each ? half_full : one_each,
                             q.d > q.N ? q.d : q.N);
  w.kslice = ((q.d + cs - 1) / cs + 63) / 64 * 64;
  w.nslice = ((q.N + cs - 1) / cs + 63) / 64 * 64;
  return launch_cluster("lora_few_kernel", kernel, dim3(static_cast<unsigned>(tile_slots<kRowsFew>(q.rows, q.n) * cs)),
                        dim3(kFewThreads), F::SMEM, cs, s, q, w);
}
template <typename OT>
int launch_few_rank(const LoraBackwardArgs& q, const FewParts& w, cudaStream_t s) {
  if (q.R <= 16) return launch_few<16, OT>(q, w, s);
  if (q.R <= 32) return launch_few<32, OT>(q, w, s);
  if (q.R <= 64) return launch_few<64, OT>(q, w, s);
  return launch_few<128, OT>(q, w, s);
}

}  // namespace

int launch_lora_few(const LoraBackwardArgs& q, float* part_A, float* part_B, cudaStream_t s) {
  const FewParts w{part_A, part_B, 0, 0};
  return q.dx && q.dx_dtype == MOE_F32 ? launch_few_rank<float>(q, w, s) : launch_few_rank<__nv_bfloat16>(q, w, s);
}

}  // namespace moe
