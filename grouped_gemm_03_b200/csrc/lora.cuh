// Device helpers the adapters' forward and backward share: tiles of rows by
// adapter, mma fragments read straight from memory, cluster exchange.
#pragma once

#include <atomic>
#include <cstdint>

#include "common.cuh"

namespace moe {

constexpr int kMaxAdapters = 1024;
constexpr int kMaxRank = 128;
constexpr int kMaxAdapterCols = 1 << 20;

// Tiles of `rows` rows in adapter order, each of one adapter.  Tile u belongs
// to the adapter a with the largest base(a) = offsets[a] / MT + a <= u and is
// its (u - base(a))-th: an adapter of m rows has ceil(m / MT) tiles, which
// never pass base(a + 1).  a == n is the rows without an adapter, behind
// offsets[n].  Offsets are held to [0, rows], so a tile is in bounds whatever
// they hold.  Called by whole warps.
template <int MT>
__host__ __device__ constexpr long long tile_slots(int rows, int n) {
  return static_cast<long long>(rows) / MT + n + 1;
}

__device__ __forceinline__ int held_offset(const int32_t* off, int n, int rows, int a) {
  return a > n ? rows : min(max(__ldg(off + a), 0), rows);
}

__device__ __forceinline__ bool find_tile(const int32_t* off, int n, int rows, int mt, int u, int& a, int& start,
                                          int& end) {
  const int lane = threadIdx.x & 31;
  int lo = 0, size = n + 1;   // the adapter is in [lo, lo + size); base(0) = 0 <= u
  while (size > 1) {
    const int step = (size + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < size && held_offset(off, n, rows, i) / mt + i <= u;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int top = m ? 31 - __clz(m) : 0;
    size = min(step, size - top * step);
    lo += top * step;
  }
  a = lo;
  const int b = held_offset(off, n, rows, a), e = held_offset(off, n, rows, a + 1);
  const long long s = b + static_cast<long long>(u - b / mt - a) * mt;
  if (s < b || s >= e) return false;
  start = static_cast<int>(s);
  end = min(e, start + mt);
  return true;
}
template <int MT>
__device__ __forceinline__ bool find_tile(const int32_t* off, int n, int rows, int u, int& a, int& start, int& end) {
  return find_tile(off, n, rows, MT, u, a, start, end);
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the float4 at this shared-memory address in CTA `rank` of the cluster
__device__ __forceinline__ float4 ld_cluster(const float4* p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// Allow `kernel` this much dynamic shared memory; `done` (one per kernel) holds the devices that do.
template <typename K>
int allow_smem(std::atomic<uint64_t>& done, K kernel, int bytes) {
  int dev = 0;
  MOE_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 64 && (done.load() >> dev & 1)) return MOE_OK;
  MOE_CUDA_CHECK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  if (dev < 64) done.fetch_or(1ull << dev);
  return MOE_OK;
}

// What resident_clusters has been told, by device and cluster size: 0 not asked yet, else the answer + 1.
struct KnownClusters {
  std::atomic<int> at[64][9] = {};
};

// How many clusters of `cs` CTAs of `kernel` are resident together on device `dev` (0: none, or the runtime does not
// say); `known` (one per kernel) holds the answers.  A cluster lies within one group of SMs: with two CTAs to an SM
// 148 pairs fit, but only 71 fours and 33 eights.
template <typename K>
int resident_clusters(KnownClusters& known, int dev, K kernel, int threads, size_t smem, int cs) {
  std::atomic<int>* at = dev >= 0 && dev < 64 ? &known.at[dev][cs] : nullptr;
  if (const int told = at ? at->load() : 0) return told - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();   // an estimate only: the launch itself reports what is wrong
    n = 0;
  }
  if (at) at->store(n + 1);
  return n;
}

// The largest cluster, up to eight CTAs, with which `tiles` clusters are resident together and each CTA has at
// least 128 of `widest` columns.  `tiles` is an average over how the rows may lie; a margin of a sixteenth saved a
// second wave where they lay worse (1021 rows of 12 adapters, rank 64: 28 -> 22 us) and cost as much where they did
// not (18 -> 21).
template <typename K>
int cluster_for(KnownClusters& known, K kernel, int threads, size_t smem, long long tiles, int widest) {
  int cs = 1, dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  while (cs < 8 && widest >= (cs + 1) * 128 && tiles <= resident_clusters(known, dev, kernel, threads, smem, cs + 1)) ++cs;
  return cs;
}

// Launch `kernel` in clusters of `cs` CTAs, allowed to start while the kernel before it finishes.
template <typename... Params, typename... Args>
int launch_cluster(const char* where, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cs,
                   cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  return e == cudaSuccess ? MOE_OK : record_cuda_error(e, where);
}

// ---------------------------------------------------------------- fragments
// D += A B, m16n8k16, bf16 operands, fp32 sums: for tiles of 16 rows, an eighth
// of what a tcgen05 MMA takes.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
// 16 bytes that no one reads again: they leave L1 to the operands that are
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 8 consecutive values; plain loads, since the output may be the same buffer
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// s * v as two bf16 terms: hi the rounded value, lo what that left, rounded.
// An infinite or NaN value stays in hi alone (inf - inf would add a NaN).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2(a, b);
  const float ha = __uint_as_float(hi << 16), hb = __uint_as_float(hi & 0xffff0000u);
  lo = pack2(isfinite(ha) ? a - ha : 0.f, isfinite(hb) ? b - hb : 0.f);
}
// As three terms: hi + mid + lo are all 24 bits of a finite value.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack2(a, b);
  const float ha = __uint_as_float(hi << 16), hb = __uint_as_float(hi & 0xffff0000u);
  split2(isfinite(ha) ? a - ha : 0.f, isfinite(hb) ? b - hb : 0.f, mid, lo);
}
// The A fragments of rows r0 and r1 (g and g + 8 of an m16 tile), K = RP: lane
// c of the quad holds elements 4c .. 4c+3 of each 16 (RP = 16), or 8c .. 8c+7
// of each 32 as its share of two k16 steps; load_b_row deals B alike.
template <int RP>
__device__ __forceinline__ void load_terms(const __nv_bfloat16* r0, const __nv_bfloat16* r1, int c,
                                           uint32_t (&f)[RP / 16][4]) {
  if constexpr (RP == 16) {
    const uint2 u = *reinterpret_cast<const uint2*>(r0 + 4 * c), v = *reinterpret_cast<const uint2*>(r1 + 4 * c);
    f[0][0] = u.x, f[0][1] = v.x, f[0][2] = u.y, f[0][3] = v.y;
  } else {
#pragma unroll
    for (int k = 0; k < RP / 32; ++k) {
      const uint4 u = *reinterpret_cast<const uint4*>(r0 + 32 * k + 8 * c);
      const uint4 v = *reinterpret_cast<const uint4*>(r1 + 32 * k + 8 * c);
      f[2 * k][0] = u.x, f[2 * k][1] = v.x, f[2 * k][2] = u.y, f[2 * k][3] = v.y;
      f[2 * k + 1][0] = u.z, f[2 * k + 1][1] = v.z, f[2 * k + 1][2] = u.w, f[2 * k + 1][3] = v.w;
    }
  }
}
template <int RP>
__device__ __forceinline__ void load_b_row(const __nv_bfloat16* row, bool in, int R, int c,
                                           uint32_t (&b)[RP / 16][2]) {
  if constexpr (RP == 16) {
    const uint2 u = in && 4 * c < R ? __ldg(reinterpret_cast<const uint2*>(row + 4 * c)) : make_uint2(0, 0);
    b[0][0] = u.x, b[0][1] = u.y;
  } else {
#pragma unroll
    for (int k = 0; k < RP / 32; ++k) {
      const uint4 u = in && 32 * k + 8 * c < R ? ldg16(row + 32 * k + 8 * c) : make_uint4(0, 0, 0, 0);
      b[2 * k][0] = u.x, b[2 * k][1] = u.y, b[2 * k + 1][0] = u.z, b[2 * k + 1][1] = u.w;
    }
  }
}

}  // namespace moe
