// Low-rank adapters of many requests beside one projection: the plan that
// orders a batch's rows by adapter, and
//   out[r] = base[r] + s_a (x[r] A_a^T) B_a^T,   a = the row's adapter.
// A_a is [R, d], B_a [N, R] (both K-major like the library's weights).
//
// Forward.  While an adapter's weights are not read too often that way (decode, a
// token or so to a request; mixed steps) one launch does it: a tile is up to 16 rows of one adapter, a cluster of up to
// eight CTAs shares it.  CTA q multiplies the q-th slice of x's columns with
// A_a, the cluster's partial x A^T meet through distributed shared memory in
// rank order, and CTA q then adds its slice of the N output columns.  x, base
// and out cross HBM once and h = x A^T never leaves the chip (unless the caller
// wants it kept).  It is bound by memory and latency, so operands go from global
// memory straight into mma fragments, 16 bytes a lane: a product does not depend
// on the order of its inner index, so lane c of a quad takes 8 consecutive inner
// elements as its share of two k16 steps, and the columns of an output block are
// dealt to the mma's n index so that a lane holds 8 consecutive ones.  No
// shared-memory staging, full sectors both ways.
//
// Else the two products are launches of their own on tiles of 128 rows
// (lora_stream.cu, lora_expand.cu).
//
// h enters the second product as two bf16 terms (hi + lo, 16 bits of mantissa
// together) for a bf16 result and as three (all 24) for an fp32 one: one bf16
// term alone would put its own rounding, 2^-9 a value, beside that of a bf16
// result, and two left 1e-6 of an fp32 one.  base joins the product's sum at its
// end, in fp32: as the accumulator it would be cut off at its own size in every
// one of up to 24 steps (beside a base of 2^12 an fp32 result left the bound of
// its one rounding at every rank; the time is the same either way).
#include <cstdint>

#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- plan
// Stable counting sort of the rows by adapter; rows without one (-1) last.
// Two launches: each block counts its rows' adapters; then each block sums the
// counts before its own (at most kPlanBlocks blocks) and ranks its rows.
constexpr int kPlanThreads = 1024;
constexpr int kPlanBlocks = 128;

int plan_rows_per_block(int rows) {
  const int per = (rows + kPlanBlocks - 1) / kPlanBlocks;
  return (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

__global__ void __launch_bounds__(kPlanThreads) plan_hist_kernel(const int32_t* __restrict__ adapter, int rows, int n,
                                                                 int per, int32_t* __restrict__ cnt,
                                                                 int32_t* __restrict__ err) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int s_cnt[kMaxAdapters + 1];
  for (int e = threadIdx.x; e <= n; e += kPlanThreads) s_cnt[e] = 0;
  __syncthreads();
  const long long r0 = static_cast<long long>(blockIdx.x) * per;
  bool bad = false;
  for (long long r = r0 + threadIdx.x; r < min(r0 + per, static_cast<long long>(rows)); r += kPlanThreads) {
    const int a = adapter[r];
    bad |= a < -1 || a >= n;
    atomicAdd(&s_cnt[a >= 0 && a < n ? a : n], 1);
  }
  bad = __syncthreads_or(bad);
  for (int e = threadIdx.x; e <= n; e += kPlanThreads) cnt[static_cast<size_t>(blockIdx.x) * (n + 1) + e] = s_cnt[e];
  if (threadIdx.x == 0) err[blockIdx.x] = bad;
}

__global__ void __launch_bounds__(kPlanThreads) plan_order_kernel(const int32_t* __restrict__ adapter, int rows, int n,
                                                                  int per, int blocks,
                                                                  const int32_t* __restrict__ cnt,
                                                                  const int32_t* __restrict__ err,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ order, int* status) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int s_at[kMaxAdapters + 1];   // next position of each adapter's rows in this block
  __shared__ int s_warp[32];
  __shared__ int s_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_base = 0;
  __syncthreads();
  for (int e0 = 0; e0 <= n; e0 += kPlanThreads) {  // exclusive scan over the adapters, 1024 at a time
    const int e = e0 + tid;
    int before = 0, all = 0;
    if (e <= n) {
#pragma unroll 8
      for (int b = 0; b < blocks; ++b) {
        const int c = cnt[static_cast<size_t>(b) * (n + 1) + e];
        before += b < static_cast<int>(blockIdx.x) ? c : 0;
        all += c;
      }
    }
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int pre = s_base;
    for (int w = 0; w < warp; ++w) pre += s_warp[w];
    const int start = pre + incl - all;
    if (e <= n) {
      s_at[e] = start + before;
      if (blockIdx.x == 0) offsets[e] = start;   // offsets[n]: the rows that have an adapter
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) s_base = start + all;
    __syncthreads();
  }
  const long long r0 = static_cast<long long>(blockIdx.x) * per;
  for (long long c0 = r0; c0 < min(r0 + per, static_cast<long long>(rows)); c0 += kPlanThreads) {
    const long long r = c0 + tid;
    const bool live = r < rows;
    int a = live ? adapter[r] : -2;
    if (live && (a < 0 || a >= n)) a = n;
    const unsigned same = __match_any_sync(0xffffffffu, a);
    const int rank = __popc(same & ((1u << lane) - 1));
    int at = 0;
    for (int w = 0; w < 32; ++w) {  // warps in row order
      if (warp == w && live) at = s_at[a];
      __syncthreads();
      if (warp == w && live && rank == 0) s_at[a] = at + __popc(same);
      __syncthreads();
    }
    if (live) order[at + rank] = static_cast<int32_t>(r);
  }
  if (blockIdx.x == 0) {
    bool bad = false;
    for (int b = tid; b < blocks; b += kPlanThreads) bad |= err[b] != 0;
    bad = __syncthreads_or(bad);
    if (tid == 0) *status = bad ? MOE_ERR_INVALID : MOE_OK;
  }
}

__global__ void plan_empty_kernel(int n, int32_t* offsets, int* status) {
  pdl_wait();
  pdl_launch_dependents();
  for (int e = threadIdx.x; e <= n; e += blockDim.x) offsets[e] = 0;
  if (threadIdx.x == 0) *status = MOE_OK;
}

// ---------------------------------------------------------------- forward
constexpr int kLoraThreads = 256;

struct LoraArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* A;
  const __nv_bfloat16* B;
  const float* scale;
  const int32_t* offsets;
  const int32_t* order;
  int n, rows, d, N, R;
  const void* base;
  void* out;
  float* h_out;
  int* status;          // nullptr: the caller has no workspace
  int kslice, nslice;   // columns of x / of out a CTA of the cluster takes, multiples of 32
};

constexpr int MT = 16;   // rows of a tile
constexpr int WK = 8;    // warps along the columns

template <int RP, int TERMS>
struct LoraTile {
  static constexpr int HS = RP + 8;                         // row stride of h's bf16 terms: spreads the banks
  static constexpr int RED = WK * MT * RP * 4;              // the warps' partial sums; then h's terms
  static constexpr int HB = TERMS * MT * HS * 2;
  static constexpr int SMEM = (RED > HB ? RED : HB) + MT * RP * 4;
  static constexpr int UK = RP <= 16 ? 4 : RP <= 64 ? 2 : 1;  // k32 steps loaded ahead
};

template <int RP, typename OT>
__global__ void __launch_bounds__(kLoraThreads, RP <= 64 ? 2 : 1) lora_kernel(const LoraArgs p) {
  constexpr int TERMS = sizeof(OT) == 4 ? 3 : 2;
  using L = LoraTile<RP, TERMS>;
  constexpr int HS = L::HS;
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint8_t s_raw[];
  float* s_red = reinterpret_cast<float*>(s_raw);                        // [WK][MT][RP]
  __nv_bfloat16* s_h = reinterpret_cast<__nv_bfloat16*>(s_raw);          // [TERMS][MT][HS], after the sums are read
  float* s_part = reinterpret_cast<float*>(s_raw + L::SMEM - MT * RP * 4);  // [MT][RP]: this CTA's slice of h
  __shared__ int s_row[MT];

  const uint32_t CS = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  int a, start, end;
  if (p.status && blockIdx.x == 0 && tid == 0) *p.status = MOE_OK;   // no wait here can run out
  if (!find_tile<MT>(p.offsets, p.n, p.rows, blockIdx.x / CS, a, start, end)) return;  // the whole cluster leaves
  if (tid < MT) {
    int r = start + tid < end ? p.order[start + tid] : -1;
    s_row[tid] = r >= 0 && r < p.rows ? r : -1;
  }
  __syncthreads();

  const int n0 = rank * p.nslice, n1 = min(p.N, n0 + p.nslice);
  OT* out = static_cast<OT*>(p.out);
  const OT* base = static_cast<const OT*>(p.base);
  if (a == p.n) {  // rows without an adapter
    if (p.h_out)
      for (int i = tid; i < MT * p.R; i += kLoraThreads)
        if (i / p.R % CS == rank && s_row[i / p.R] >= 0) p.h_out[static_cast<size_t>(s_row[i / p.R]) * p.R + i % p.R] = 0.f;
    if (base == out) return;
    const int w8 = (n1 - n0) / 8;
    for (int i = tid; i < MT * w8; i += kLoraThreads) {
      const int r = s_row[i / w8];
      if (r < 0) continue;
      const size_t o = static_cast<size_t>(r) * p.N + n0 + i % w8 * 8;
      float v[8] = {};
      if (base) load8(base + o, v);
      store8(out + o, v);
    }
    return;
  }

  // What the second product takes from memory for a warp's 32 columns, of the first ones on its way while h is
  // formed (up to rank 32: above, the registers go to h).
  constexpr bool kAhead = RP <= 32;
  const int nb0 = n0 + warp * 32;
  size_t ro[2];
  bool rl[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = s_row[g + 8 * h];
    rl[h] = r >= 0;
    ro[h] = static_cast<size_t>(r >= 0 ? r : 0) * p.N + c * 8;
  }
  // the mma's n index g of block t is column (g / 2) * 8 + 2 t + g % 2 of 32
  const __nv_bfloat16* Bc = p.B + (static_cast<size_t>(a) * p.N + (g >> 1) * 8 + (g & 1)) * p.R;
  float v[2][8];
  uint32_t bw[4][RP / 16][2];
  auto fetch = [&](int nb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h][i] = 0.f;
      if (base && nb + c * 8 < n1 && rl[h]) load8(base + ro[h] + nb, v[h]);
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        load_b_row<RP>(Bc + static_cast<size_t>(nb + 2 * t) * p.R, nb + (g >> 1) * 8 < n1, p.R, c, bw[t]);
    }
  };

  // ---- h over this CTA's columns of x
  {
    float acc[RP / 8][4];
#pragma unroll
    for (int j = 0; j < RP / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    const __nv_bfloat16* xr[2];
    bool xl[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = s_row[g + 8 * h];
      xl[h] = r >= 0;
      xr[h] = p.x + static_cast<size_t>(r >= 0 ? r : 0) * p.d + c * 8;
    }
    const __nv_bfloat16* Ar = p.A + (static_cast<size_t>(a) * p.R + g) * p.d + c * 8;
    const int k0 = rank * p.kslice, k1 = min(p.d, k0 + p.kslice);
    for (int kb = k0 + warp * 32; kb < k1; kb += WK * 32 * L::UK) {
      uint4 xv[L::UK][2], av[L::UK][RP / 8];
#pragma unroll
      for (int u = 0; u < L::UK; ++u) {
        const int k = kb + u * WK * 32;
        const bool in = k + c * 8 < k1;
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[u][h] = in && xl[h] ? ldg_stream(xr[h] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < RP / 8; ++j)
          av[u][j] = in && j * 8 + g < p.R ? ldg16(Ar + static_cast<size_t>(j * 8) * p.d + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < L::UK; ++u)
#pragma unroll
        for (int j = 0; j < RP / 8; ++j) {
          mma16816(acc[j], xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y, av[u][j].x, av[u][j].y);
          mma16816(acc[j], xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w, av[u][j].z, av[u][j].w);
        }
    }
    fetch(nb0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* o = s_red + (static_cast<size_t>(warp) * MT + g + 8 * h) * RP + 2 * c;
#pragma unroll
      for (int j = 0; j < RP / 8; ++j) *reinterpret_cast<float2*>(o + 8 * j) = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
    }
  }
  __syncthreads();
  for (int i = tid; i < MT * RP / 4; i += kLoraThreads) {
    float4 v = reinterpret_cast<const float4*>(s_red)[i];
#pragma unroll
    for (int w = 1; w < WK; ++w) {
      const float4 u = reinterpret_cast<const float4*>(s_red + w * MT * RP)[i];
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    reinterpret_cast<float4*>(s_part)[i] = v;
  }
  cluster_arrive();
  cluster_wait();   // every CTA's slice is there (CS = 1: the block's own barrier)
  const float sc = p.scale ? __ldg(p.scale + a) : 1.f;
  for (int i = tid; i < MT * RP / 4; i += kLoraThreads) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t q = 0; q < CS; ++q) {
      const float4 u = ld_cluster(reinterpret_cast<const float4*>(s_part) + i, q);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    const int m = i / (RP / 4), j = i % (RP / 4) * 4;
    if (p.h_out && m % CS == rank && s_row[m] >= 0 && j < p.R)
      *reinterpret_cast<float4*>(p.h_out + static_cast<size_t>(s_row[m]) * p.R + j) = v;
    uint32_t w[3][2];
    split3(v.x * sc, v.y * sc, w[0][0], w[1][0], w[2][0]);
    split3(v.z * sc, v.w * sc, w[0][1], w[1][1], w[2][1]);
#pragma unroll
    for (int q = 0; q < TERMS; ++q)
      *reinterpret_cast<uint2*>(s_h + (q * MT + m) * HS + j) = make_uint2(w[q][0], w[q][1]);
  }
  cluster_arrive();  // done with the others' shared memory; waited for before this CTA ends
  __syncthreads();

  // ---- out over this CTA's columns
  uint32_t hf[TERMS][RP / 16][4];
#pragma unroll
  for (int q = 0; q < TERMS; ++q) load_terms<RP>(s_h + (q * MT + g) * HS, s_h + (q * MT + g + 8) * HS, c, hf[q]);
  for (int nb = nb0; nb < n1; nb += WK * 32) {
    if (nb != nb0) fetch(nb);
    const bool in = nb + c * 8 < n1;
    float acc[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
      uint32_t bt[RP / 16][2];
      if constexpr (kAhead) {
#pragma unroll
        for (int k = 0; k < RP / 16; ++k) bt[k][0] = bw[t][k][0], bt[k][1] = bw[t][k][1];
      } else {
        load_b_row<RP>(Bc + static_cast<size_t>(nb + 2 * t) * p.R, nb + (g >> 1) * 8 < n1, p.R, c, bt);
      }
#pragma unroll
      for (int q = TERMS - 1; q >= 0; --q)   // the small terms first: only the largest's steps cut a whole sum off
#pragma unroll
        for (int k = 0; k < RP / 16; ++k)
          mma16816(acc[t], hf[q][k][0], hf[q][k][1], hf[q][k][2], hf[q][k][3], bt[k][0], bt[k][1]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!in || !rl[h]) continue;
      float o[8];
#pragma unroll
      for (int t = 0; t < 4; ++t) o[2 * t] = v[h][2 * t] + acc[t][2 * h], o[2 * t + 1] = v[h][2 * t + 1] + acc[t][2 * h + 1];
      store8(out + ro[h] + nb, o);
    }
  }
  cluster_wait();
}

template <int RP, typename OT>
int launch_lora_tiles(LoraArgs& p, cudaStream_t s) {
  using L = LoraTile<RP, sizeof(OT) == 4 ? 3 : 2>;
  auto kernel = lora_kernel<RP, OT>;
  static std::atomic<uint64_t> done{0};
  const int st = allow_smem(done, kernel, L::SMEM);
  if (st != MOE_OK) return st;
  // as many CTAs as are resident together: a second wave took 11.3 us where one takes 6.8 (61 rows of 48 adapters,
  // clusters of 8 against 4)
  const long long half_full = p.rows / MT + p.n / 2, one_each = p.n < p.rows ? p.n : p.rows;
  static KnownClusters known;
  const int cs = cluster_for(known, kernel, kLoraThreads, L::SMEM, half_full > one_each ? half_full : one_each,
                             p.d > p.N ? p.d : p.N);
  p.kslice = ((p.d + cs - 1) / cs + 31) / 32 * 32;
  p.nslice = ((p.N + cs - 1) / cs + 31) / 32 * 32;
  return launch_cluster("lora_kernel", kernel, dim3(static_cast<unsigned>(tile_slots<MT>(p.rows, p.n) * cs)),
                        dim3(kLoraThreads), L::SMEM, cs, s, p);
}

template <typename OT>
int launch_lora_rank(LoraArgs& p, cudaStream_t s) {
  if (p.R <= 16) return launch_lora_tiles<16, OT>(p, s);
  if (p.R <= 32) return launch_lora_tiles<32, OT>(p, s);
  if (p.R <= 64) return launch_lora_tiles<64, OT>(p, s);
  return launch_lora_tiles<128, OT>(p, s);
}

}  // namespace

size_t adapter_plan_workspace_bytes(int rows, int n) {
  const int per = plan_rows_per_block(rows);
  const size_t blocks = rows > 0 ? (rows + static_cast<size_t>(per) - 1) / per : 0;
  return 256 + align_up(blocks * (n + 1) * 4, 256) + align_up(blocks * 4, 256);
}

int launch_adapter_plan(const int32_t* adapter, int rows, int n, int32_t* offsets, int32_t* order, void* ws,
                        cudaStream_t s) {
  int* status = static_cast<int*>(ws);
  if (rows == 0) return launch_pdl(__func__, plan_empty_kernel, dim3(1), dim3(256), 0, s, n, offsets, status);
  const int per = plan_rows_per_block(rows);
  const int blocks = static_cast<int>((static_cast<long long>(rows) + per - 1) / per);
  int32_t* cnt = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + 256);
  int32_t* err = cnt + align_up(static_cast<size_t>(blocks) * (n + 1) * 4, 256) / 4;
  const int st = launch_pdl(__func__, plan_hist_kernel, dim3(blocks), dim3(kPlanThreads), 0, s, adapter, rows, n, per,
                            cnt, err);
  if (st != MOE_OK) return st;
  return launch_pdl(__func__, plan_order_kernel, dim3(blocks), dim3(kPlanThreads), 0, s, adapter, rows, n, per, blocks,
                    static_cast<const int32_t*>(cnt), static_cast<const int32_t*>(err), offsets, order, status);
}

// Whether the forward's products are launches of their own, by an estimate of
// both ways' times from what they move.  One launch reads an adapter's weights
// for every 16 of its rows, out of L2 (at 8 TB/s; at 4 above rank 64, where one
// CTA fills an SM), two launches read them for every 128, but start twice and
// leave the last 128 rows of each adapter in part empty.  Measured, one launch
// against two, columns 4096 and 4096 where not given:
//   rank 16:  1024 rows of 8 adapters 10.0 / 18.3 us, 4096 of 1 30.8 / 30.2, 8192 of 1 57.5 / 48.2,
//             8192 of 128 61.5 / 72.7
//   rank 32:  4096 of 16 35.2 / 44.2, 8192 of 8 (7168 columns in) 79.9 / 59.8
//   rank 64:  256 of 8 12.8 / 15.4, 2048 of 4 27.6 / 29.0, 4096 of 4 47.3 / 34.7, 8192 of 32 92.8 / 61.5
//   rank 128: 256 of 4 16.3 / 15.8, 1024 of 16 52.6 / 36.2
// n is taken for the adapters in use, which the host does not know.  Where most
// of those held are not, one launch serves as well (4096 rows, columns 2048 and
// 2048, rank 64): of 1 in use and held 24.2 / 23.1, of 1 in 1024 held 24.8 / 48.7.
bool lora_two_launches(int rows, int n, int d, int N, int R) {
  const double ns_per_hbm_byte = 1 / 6400.0, row = 2.0 * d + 4.0 * N, weights = 2.0 * R * (d + N);
  const double active = n < rows ? n : rows, tiles = rows / 16.0 + 0.5 * active;
  const double one = 4500 + (rows * row + active * weights) * ns_per_hbm_byte + tiles * weights / (R <= 64 ? 8000 : 4000);
  const double two = 9500 + 40.0 * R + ((rows + 32.0 * active) * row + active * weights) / 5000;
  return two < one;
}

size_t lora_workspace_bytes(int rows, int n, int d, int N, int R) {
  return lora_two_launches(rows, n, d, N, R) ? 256 + image_bytes(rows, n, R) : 0;
}

int launch_lora(const LoraForwardArgs& q, cudaStream_t s) {
  int* status = static_cast<int*>(q.ws);
  if (q.rows == 0) {
    if (status) MOE_CUDA_CHECK(cudaMemsetAsync(status, 0, sizeof(int), s));   // MOE_OK
    return MOE_OK;
  }
  if (lora_two_launches(q.rows, q.n, q.d, q.N, q.R)) {
    uint8_t* h = static_cast<uint8_t*>(q.ws) + 256;
    StreamArgs p{};
    p.X = static_cast<const __nv_bfloat16*>(q.x), p.M = static_cast<const __nv_bfloat16*>(q.A);
    p.offsets = q.offsets, p.order = q.order, p.n = q.n, p.rows = q.rows, p.W = q.d, p.R = q.R;
    p.scale = q.scale, p.image = h, p.h_out = q.h_out, p.status = status, p.first = true;
    // slices of a row: as many as leave two CTAs to an SM, up to the portable cluster
    const long long tiles = (static_cast<long long>(q.rows) + 64ll * q.n) / 128 + 1;  // an adapter's last is half full
    p.chunk = 128, p.cluster = 1;
    while (p.cluster < 8 && tiles * p.cluster <= num_sms() && q.d > p.cluster * 128) p.cluster *= 2;
    p.cols = ((q.d + p.cluster - 1) / p.cluster + 127) / 128 * 128;
    const int st = launch_lora_stream(p, kStreamProject, s);
    if (st != MOE_OK) return st;
    ExpandArgs e{};
    e.h = h, e.M = static_cast<const __nv_bfloat16*>(q.B), e.offsets = q.offsets, e.order = q.order;
    e.n = q.n, e.rows = q.rows, e.N = q.N, e.R = q.R, e.base = q.base, e.out = q.out, e.h_out = q.h_out;
    e.status = status;
    return launch_lora_expand(e, false, q.out_dtype, s);
  }
  LoraArgs p{};
  p.x = static_cast<const __nv_bfloat16*>(q.x), p.A = static_cast<const __nv_bfloat16*>(q.A);
  p.B = static_cast<const __nv_bfloat16*>(q.B), p.scale = q.scale, p.offsets = q.offsets, p.order = q.order;
  p.n = q.n, p.rows = q.rows, p.d = q.d, p.N = q.N, p.R = q.R, p.base = q.base, p.out = q.out, p.h_out = q.h_out;
  p.status = status;
  return q.out_dtype == MOE_F32 ? launch_lora_rank<float>(p, s) : launch_lora_rank<__nv_bfloat16>(p, s);
}

}  // namespace moe
