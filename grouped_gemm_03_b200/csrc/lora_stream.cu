// One pass over a wide operand X [rows, W] of the adapters' forward and
// gradients, its products on the tensor cores (tcgen05, fp32 sums in TMEM):
//   projection  P[r] = X[r] M_a^T            h = x A^T,   dh = s dC B
//   gradient    G_a  = sum_r X[r]^T V[r]     dB = dC^T (s h),   dA^T = x^T dh
// over the rows r of adapter a.  X crosses HBM once: the pass over dC does both
// products on the same tile, the one in X's own orientation, the other in
// its transpose, which the MMA reads from the same shared memory (a K-major
// and an MN-major descriptor of one 128-byte-swizzled tile).
//
// A CTA takes a chunk of one adapter's rows and a slice of X's columns and
// walks it in tiles of 128 rows x 128 columns.  The projection alone has
// chunks of 128 rows; the slices of a row meet in a cluster, through
// distributed shared memory and in rank order, so h leaves it complete.  Its
// tiles take turns in up to eight accumulators, added up at the end: the tensor
// cores cut off what an fp32 sum cannot hold, and 112 additions into one left
// 1.8e-6 of h, twice what a matrix product in fp32 leaves.  With
// the gradient, G stays in TMEM until the chunk ends (one accumulator to 128
// columns) and P is complete for the slice after each 128 rows; what several
// CTAs add to (P over slices, G over chunks) is written as fp32 partial sums
// and added in a fixed order by the kernels that follow, except G of an adapter
// with a single chunk, which is written in place.  With ranks up to 32 two CTAs
// share an SM, so that the one's start, end and change of rows hide behind the
// other's loads.
//
// V enters as three bf16 terms (all 24 bits of an fp32 value): G is an fp32
// sum, and fewer terms would leave their rounding as the largest error in it
// (2.7e-6 of the gradient with two, 3.6e-7 of a sum in fp32).  They come split
// and laid out (lora_tc.cuh): split by every slice's CTA again they took 2700
// cycles of each 128 rows, more than the MMAs.  Side by side in the MMA's N
// they take one MMA up to rank 64 (one of 192 columns takes 97 cycles, three of
// 64 take 153), above one after the other into the same accumulator.  Both V
// and B lie with a row's ranks side by side, as in memory: the MMA takes them
// with the ranks along N and the rows along K (MN-major), so nothing is
// transposed on the way.
//
// The first warps load X (tile::gather4, four rows of the plan's order at a
// time, zeros for a row that is not there; the next 128 rows' ids are fetched a
// step ahead), eight more empty TMEM, one thread of the last warp issues the
// MMAs.  gather4 takes a warp about 85 cycles, so eight warps an SM issue them:
// four where two CTAs share it.  Measured on 117 MB in 224 CTAs: 1.7 TB/s from
// one warp an SM, 4.4 from four, 5.2 from eight, 5.7 from two CTAs of four;
// cp.async of 16 bytes by the same warps reaches the same rates alone, but its
// address arithmetic and proxy fences held the whole kernel to 3.5.  An MMA of
// up to 64 columns takes 51 cycles whatever its N (its A operand comes from
// shared memory).
//
// Measured: projection of 8192 rows of 7168 columns at rank 32, 27 us (4.4 TB/s;
// an SM takes in 50 GB/s, the busiest one 1.1 MB); both products of 8191 x 7168
// at rank 64, 67 us, bound by what the SMs take in: 48 KB of V beside 64 KB of
// dC to 128 rows, and the partial sums going out.
//
// Every wait has a time limit; one that runs out raises the block's abort flag,
// every role leaves its loop, copies and MMAs in flight are waited for, TMEM is
// freed and MOE_ERR_TIMEOUT is left in *status.
#include <cstdint>

#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

constexpr int kDrainers = 256;
constexpr int kTile = 128;                 // rows and columns of a tile
constexpr int kSub = kTile * 128;          // bytes of 128 rows x 64 columns
constexpr int kTerms = 3;

template <int RP, bool PROJ, bool GRAD>
struct StreamCfg {
  static constexpr bool STACK = RP <= 64;
  static constexpr int GCOLS = GRAD ? (STACK ? kTerms * RP : RP) : 0;       // TMEM columns of 128 of X's
  static constexpr int BLOCKS = !GRAD ? 1 : RP <= 16 ? 4 : 2;  // 128-column blocks, at most
  static constexpr int PBUF = GRAD ? 2 : RP <= 32 ? 8 : 4;                  // projection accumulators
  static constexpr int PS = RP + 4;                                         // row stride of P in shared memory: spreads the banks
  static constexpr int PCOL = GRAD ? BLOCKS * GCOLS : 0;                    // their first TMEM column
  static constexpr int USED = PCOL + (PROJ ? PBUF * RP : 0);
  static constexpr int TMEM = USED <= 32 ? 32 : USED <= 64 ? 64 : USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
  static constexpr int MSUB = RP * 128;                                     // bytes of A's rows for 64 columns
  static constexpr int RANKS = RankTile<RP>::BYTES;                         // 128 rows of RP ranks: V's term, B's block
  static constexpr int M_ALL = PROJ && GRAD ? BLOCKS * RANKS : 0;           // resident
  static constexpr int STAGE = 2 * kSub + (PROJ && !GRAD ? 2 * MSUB : 0);
  static constexpr int PER_SM = RP <= 32 || (!GRAD && RP <= 64) ? 2 : 1;
  static constexpr int LW = PER_SM == 2 && GRAD ? 4 : 8;                    // warps that load
  static constexpr int MMA_WARP = LW + kDrainers / 32;
  static constexpr int THREADS = (MMA_WARP + 1) * 32;
  static constexpr int GS = RP / 2 + 4;                                     // row stride of a warp's share of G on its way out
  static constexpr int BUDGET = PER_SM == 2 ? 110 * 1024 : 226 * 1024;
  static constexpr int V_ONE = GRAD ? RankTile<RP>::IMAGE : 0;
  static constexpr int VBUF = !GRAD ? 0 : (BUDGET - M_ALL - 2 * V_ONE) / STAGE >= 2 ? 2 : 1;  // two where two stages fit beside
  static constexpr int STAGES_RAW = (BUDGET - M_ALL - VBUF * V_ONE) / STAGE;
  static constexpr int STAGES = STAGES_RAW > 4 ? 4 : STAGES_RAW;
  static constexpr int SMEM = STAGES * STAGE + M_ALL + VBUF * V_ONE + 1024;  // + alignment slack
  static_assert(USED <= 512 && STAGES >= 2 && (GRAD || kTile * PS * 4 <= STAGES * STAGE) &&
                    (kDrainers * GS * 4 <= STAGES * STAGE + M_ALL), "TMEM and shared memory");
};

// N accumulator columns (8, 16 or 32), in flight until the wait
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[8]) { ptx::tmem_ld_32x32b_x8(at, r); }
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[16]) { ptx::tmem_ld_32x32b_x16(at, r); }
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[32]) { ptx::tmem_ld_32x32b_x32(at, r); }

// N columns of G, the terms added up, smallest first
template <bool STACK, int RP, int N>
__device__ __forceinline__ void load_grad(uint32_t at, float (&v)[N]) {
  uint32_t r[N];
  tmem_ld(at, r);
  if constexpr (STACK) {
    uint32_t s[N], t[N];
    tmem_ld(at + RP, s);
    tmem_ld(at + 2 * RP, t);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]) + (__uint_as_float(s[i]) + __uint_as_float(t[i]));
  } else {
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
  }
}

template <int RP, bool PROJ, bool GRAD>
__global__ void __launch_bounds__(StreamCfg<RP, PROJ, GRAD>::THREADS, StreamCfg<RP, PROJ, GRAD>::PER_SM)
    lora_stream_kernel(const StreamArgs p, const __grid_constant__ CUtensorMap map_x,
                       const __grid_constant__ CUtensorMap map_m) {
  using C = StreamCfg<RP, PROJ, GRAD>;
  using RT = RankTile<RP>;
  constexpr int S = C::STAGES, kLoaders = C::LW * 32, kMmaWarp = C::MMA_WARP;
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_m = smem + S * C::STAGE;
  uint8_t* s_v = s_m + C::M_ALL;
  __shared__ __align__(8) uint64_t full[S], empty[S], step_done[2], p_free[2], drained;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    ptx::mbar_init(&step_done[0], 1);
    ptx::mbar_init(&step_done[1], 1);
    ptx::mbar_init(&drained, 1);
    ptx::mbar_init(&p_free[0], kDrainers);
    ptx::mbar_init(&p_free[1], kDrainers);
    s_abort = 0;
    ptx::fence_mbar_init();
  }
  if (!p.early) pdl_wait();
  const uint32_t CS = GRAD ? 1 : cluster_size();
  const int slot = GRAD ? blockIdx.x : blockIdx.x / CS, slice = GRAD ? blockIdx.y : cluster_rank();
  int a, start, end;
  const bool found = find_tile(p.offsets, p.n, p.rows, p.chunk, slot, a, start, end);
  const int W = p.W, R = p.R;
  const int col0 = slice * p.cols;
  const size_t size = static_cast<size_t>(W) * R;   // G's values of one adapter
  if (!found || a == p.n) {   // the whole cluster leaves
    pdl_wait();
    pdl_launch_dependents();
    if (p.first && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.status = MOE_OK;
    if constexpr (GRAD) {     // the slot of an adapter without rows: its gradient is 0
      if (a < p.n && p.grad && held_offset(p.offsets, p.n, p.rows, a) >= held_offset(p.offsets, p.n, p.rows, a + 1)) {
        const size_t first = a * size;
        const int c1 = min(W, col0 + p.cols), lines = PROJ ? 1 : R;       // [W][R]: one run; [R][W]: one to a rank
        const int each = PROJ ? (c1 - col0) * R : c1 - col0, bytes = p.grad_f32 ? 4 : 2;
        for (int i = tid; i < lines * (each / 8); i += C::THREADS) {
          const size_t o = first + (PROJ ? static_cast<size_t>(col0) * R : static_cast<size_t>(i / (each / 8)) * W + col0) +
                           i % (each / 8) * 8;
          for (int u = 0; u < 8 * bytes; u += 16)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.grad) + o * bytes + u) = make_uint4(0, 0, 0, 0);
        }
      }
    }
    return;
  }
  const int blocks = max(0, min(p.cols, W - col0) + kTile - 1) / kTile;  // none behind the last column
  const int steps = (end - start + kTile - 1) / kTile;
  const bool want_p = PROJ && (!GRAD || p.proj), want_g = GRAD && p.grad;

  __syncthreads();
  // The loaders go on with what the launch before this one did not write (early); the others wait for its end,
  // TMEM with them: a block that held some while it waits could keep the ones it waits for from starting.
  uint32_t tmem = 0;
  if (warp >= kLoaders / 32) {
    pdl_wait();
    if (warp == kMmaWarp) {
      if (p.first && blockIdx.x == 0 && blockIdx.y == 0 && lane == 0) *p.status = MOE_OK;
      ptx::tmem_alloc(&s_tmem, C::TMEM);
      ptx::tmem_relinquish();
      pdl_launch_dependents();   // what runs beside this launch finds its TMEM taken
    }
    ptx::tc_fence_before();
    named_barrier(1, C::THREADS - kLoaders);
    ptx::tc_fence_after();
    tmem = s_tmem;
  }
  auto give_up = [&]() {
    s_abort = 1;
    if (p.status) set_status(p.status, MOE_ERR_TIMEOUT);
  };

  if (warp < kLoaders / 32) {
    // ---- X: tile t goes to stage t % S.  Lane l of a warp gathers its (l % Q)-th four rows, columns
    // 64 (l / Q) .. + 63 of the tile's 128; a row that is not there is taken from behind X, as zeros.
    constexpr int Q = 32 / C::LW;
    const int quad = warp * Q + lane % Q, sub = lane / Q;
    // the projection alone needs no rows behind the last: what P holds there is not read
    const int quads = GRAD ? 32 : (end - start + 3) / 4;
    const bool mine = sub < 2 && quad < quads;
    const uint64_t policy = ptx::policy_evict_first();
    int next[4], row[4];
    auto fetch_ids = [&](int step) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = start + step * kTile + quad * 4 + u;
        next[u] = mine && at < end ? __ldg(p.order + at) : -1;
      }
    };
    fetch_ids(0);
    // the first tile slot of this chunk's rows
    const int first = held_offset(p.offsets, p.n, p.rows, a);
    const uint8_t* image = p.V + static_cast<size_t>(first / kTile + a + (start - first) / kTile) * RT::IMAGE;
    bool ok = true;
    int t = 0;
    // A warp with rows to bring is part of every stage's turn, so that none passes it unseen; one without stays out
    // of the loop, where a barrier could turn twice between two of its looks.
    const int my_steps = warp * Q < quads ? steps : 0;
    for (int step = 0; step < my_steps && ok; ++step) {
#pragma unroll
      for (int u = 0; u < 4; ++u) row[u] = next[u] >= 0 && next[u] < p.rows ? next[u] : p.rows;
      if (step + 1 < steps) fetch_ids(step + 1);
      for (int b = 0; b < blocks; ++b, ++t) {
        if (t >= S && !ptx::mbar_wait_warp(&empty[t % S], (t / S - 1) & 1, abort_flag, kWaitLimitNs)) {
          give_up();
          ok = false;
          break;
        }
        uint8_t* dst = smem + t % S * C::STAGE;
        const int col = col0 + b * kTile;
        if (tid == 0) {
          ptx::mbar_arrive_expect_tx(&full[t % S], C::STAGE - (32 - quads) * 1024 + (PROJ && GRAD && step == 0 ? C::RANKS : 0) +
                                                         (want_g && b == 0 ? C::V_ONE : 0));
          if constexpr (PROJ && !GRAD) {   // A's columns of this tile
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_3d(dst + 2 * kSub + h * C::MSUB, &map_m, &full[t % S], col + h * 64, 0, a);
          }
          if constexpr (PROJ && GRAD) {    // B's rows of this block, once
            if (step == 0) {
#pragma unroll
              for (int h = 0; h < RP; h += 64)
                tma_load_3d(s_m + b * C::RANKS + h / 64 * RT::LEAD, &map_m, &full[t % S], h, col, a);
            }
          }
        }
        __syncwarp();
        if (mine)
          gather4_once(dst + sub * kSub + quad * 512, &map_x, &full[t % S], col + sub * 64, row, policy);
        if constexpr (GRAD) {
          if (want_g && b == 0 && warp == 0) {   // V's terms of these rows, where a step's MMAs have left theirs
            constexpr int VB = C::VBUF;
            if (step >= VB && !ptx::mbar_wait_warp(&step_done[(step - VB) & 1], ((step - VB) >> 1) & 1, abort_flag, kWaitLimitNs)) {
              give_up();
              ok = false;
              ++t;
              break;
            }
            if (step == 0) pdl_wait();
            if (lane == 0)
              bulk_load(s_v + step % VB * C::V_ONE, image + static_cast<size_t>(step) * RT::IMAGE, C::V_ONE, &full[t % S]);
          }
        }
      }
    }
    // what is in flight lands before the block ends, whoever gave up
    int never = 0;
    for (int u = t > S ? t - S : 0; u < t; ++u) ptx::mbar_wait_warp(&full[u % S], (u / S) & 1, &never, kWaitLimitNs);
  } else if (warp < kMmaWarp) {
    // ---- P out, and at the end G.  Two warps to a quarter of TMEM's lanes, half the columns each.
    const int et = tid - kLoaders, ew = warp - kLoaders / 32, quarter = ew & 3, half = ew >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const float sc = PROJ && GRAD && p.scale ? __ldg(p.scale + a) : 1.f;
    constexpr int HC = RP / 2 > 32 ? 32 : RP / 2;   // TMEM columns read at once
    bool ok = true;
    for (int step = 0; step < (GRAD && want_p ? steps : 0); ++step) {
      // the step's MMAs are done: P is complete
      if (!ptx::mbar_wait_warp(&step_done[step & 1], (step >> 1) & 1, abort_flag, kWaitLimitNs)) {
        give_up();
        ok = false;
        break;
      }
      if constexpr (PROJ) {
        ptx::tc_fence_after();
        const int at = start + step * kTile + quarter * 32 + lane;
        float* o = p.proj + (static_cast<size_t>(slice) * p.rows + at) * R;
        const uint32_t from = tmem + lane_base + C::PCOL + step % C::PBUF * RP;
#pragma unroll
        for (int u = 0; u < RP / 2; u += HC) {
          uint32_t r[HC];
          __syncwarp();
          tmem_ld(from + half * (RP / 2) + u, r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < HC; e += 8) {
            const int j = half * (RP / 2) + u + e;
            if (at >= end || j >= R) continue;
            float x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = __uint_as_float(r[e + q]) * sc;
            store32(o + j, x);
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&p_free[step % C::PBUF]);
      }
    }
    if constexpr (!GRAD) {   // the slice's P to shared memory, over the stages: their MMAs are done
      float* s_p = reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * C::PS + half * (RP / 2);
      if (blocks == 0) {
        for (int j = 0; j < RP / 2; j += 4) *reinterpret_cast<float4*>(s_p + j) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else if (ptx::mbar_wait_warp(&drained, 0, abort_flag, kWaitLimitNs)) {
        ptx::tc_fence_after();
        const int used = min(blocks, C::PBUF);
#pragma unroll
        for (int j = 0; j < RP / 2; j += 8) {
          float v[8] = {};
          __syncwarp();
#pragma unroll
          for (int q0 = 0; q0 < C::PBUF; q0 += 4) {
            if (q0 >= used) break;
            uint32_t r[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q)   // what was not accumulated into is not added
              tmem_ld(tmem + lane_base + (q0 + q) * RP + half * (RP / 2) + j, r[q]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int u = 0; u < 8; ++u) v[u] += q0 + q < used ? __uint_as_float(r[q][u]) : 0.f;
          }
#pragma unroll
          for (int u = 0; u < 8; u += 4)
            *reinterpret_cast<float4*>(s_p + j + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
        }
      } else {
        give_up();
      }
    }
    if constexpr (GRAD) {
      if (want_g && ok && !ptx::mbar_wait_warp(&drained, 0, abort_flag, kWaitLimitNs)) {
        give_up();
        ok = false;
      }
      if (want_g && ok) {
        ptx::tc_fence_after();
        const int first = held_offset(p.offsets, p.n, p.rows, a), last = held_offset(p.offsets, p.n, p.rows, a + 1);
        const bool whole = last - first <= p.chunk;  // no other chunk adds to it
        float* part = p.part + (part_slot(first, p.chunk) + (start - first) / p.chunk) * size;
        float* g32 = static_cast<float*>(p.grad) + a * size;
        __nv_bfloat16* g16 = static_cast<__nv_bfloat16*>(p.grad) + a * size;
        // [W][R]: through shared memory (over the stages and B: the MMAs are done), where a thread holds a
        // column's ranks, out in whole rows; [R][W]: neighbouring lanes hold neighbouring columns already
        float* s_g = reinterpret_cast<float*>(smem) + ew * 32 * C::GS;
        for (int b = 0; b < blocks; ++b) {
          const int k0 = col0 + b * kTile + quarter * 32, k = k0 + lane;
#pragma unroll
          for (int u = 0; u < RP / 2; u += HC) {
            float x[HC];
            __syncwarp();
            load_grad<C::STACK, RP>(tmem + lane_base + b * C::GCOLS + half * (RP / 2) + u, x);
            if constexpr (PROJ) {
#pragma unroll
              for (int q = 0; q < HC; q += 4)
                *reinterpret_cast<float4*>(s_g + lane * C::GS + u + q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
            } else {
#pragma unroll
              for (int q = 0; q < HC; ++q) {
                const int j = half * (RP / 2) + u + q;
                const size_t o = static_cast<size_t>(j) * W + k;
                if (k >= W || j >= R) continue;
                if (!whole) part[o] = x[q];
                else if (p.grad_f32) g32[o] = x[q];
                else g16[o] = __float2bfloat16_rn(x[q]);
              }
            }
          }
          if constexpr (PROJ) {
            constexpr int PC = RP / 8;     // pieces of 4 ranks in half a row
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PC; ++i) {
              const int m = i * (32 / PC) + lane / PC, j = lane % PC * 4, rank = half * (RP / 2) + j;
              const float4 x = *reinterpret_cast<const float4*>(s_g + m * C::GS + j);
              if (k0 + m >= W || rank >= R) continue;
              const size_t o = static_cast<size_t>(k0 + m) * R + rank;
              if (!whole) *reinterpret_cast<float4*>(part + o) = x;
              else if (p.grad_f32) *reinterpret_cast<float4*>(g32 + o) = x;
              else *reinterpret_cast<uint2*>(g16 + o) = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
            }
          }
        }
      }
    }
    ptx::tc_fence_before();
  } else if (lane == 0) {
    // ---- MMAs
    constexpr uint32_t IP = ptx::make_idesc(128, RP, 1) | (GRAD ? kBMn : 0u);
    constexpr uint32_t IG = ptx::make_idesc(128, C::STACK ? kTerms * RP : RP, 1) | kAMn | kBMn;
    bool ok = true;
    int t = 0;
    for (int step = 0; step < steps && blocks > 0 && ok; ++step) {
      if (GRAD && want_p && step >= C::PBUF)
        ok = ptx::mbar_wait(&p_free[step % C::PBUF], (step / C::PBUF - 1) & 1, abort_flag, kWaitLimitNs);
      for (int b = 0; b < blocks && ok; ++b, ++t) {
        ok = ptx::mbar_wait(&full[t % S], (t / S) & 1, abort_flag, kWaitLimitNs);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t x = ptx::smem_u32(smem + t % S * C::STAGE);
        if (want_p) {
          const uint32_t d = tmem + C::PCOL + (GRAD ? step : b) % C::PBUF * RP;
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // 16 columns at a time
            const uint64_t md =
                GRAD ? RT::desc(ptx::smem_u32(s_m) + b * C::RANKS + k * 16 * RT::ROW, RT::LEAD)
                     : ptx::sw128_kmajor_desc(x + 2 * kSub + k / 4 * C::MSUB) + k % 4 * 2;
            ptx::umma_f16(d, ptx::sw128_kmajor_desc(x + k / 4 * kSub) + k % 4 * 2, md, IP, (GRAD ? b > 0 : b >= C::PBUF) || k > 0);
          }
        }
        if (want_g) {
          const uint32_t v = ptx::smem_u32(s_v) + (C::VBUF == 2 ? (step & 1) * C::V_ONE : 0);
          const uint32_t d = tmem + b * C::GCOLS;
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // 16 rows at a time
            const uint64_t xd = mn_desc(x + k * 2048, kSub);
            if constexpr (C::STACK) {    // the terms side by side: each a unit of the layout
              ptx::umma_f16(d, xd, RT::desc(v + k * 16 * RT::ROW, C::RANKS), IG, step > 0 || k > 0);
            } else {
#pragma unroll
              for (int q = 0; q < kTerms; ++q)
                ptx::umma_f16(d, xd, RT::desc(v + q * C::RANKS + k * 16 * RT::ROW, RT::LEAD), IG,
                              step > 0 || k > 0 || q > 0);
            }
          }
        }
        ptx::umma_commit(&empty[t % S]);
      }
      if (ok) ptx::umma_commit(&step_done[step & 1]);
    }
    ptx::umma_commit(&drained);
    if (!ok) give_up();
    int never = 0;   // what was issued, arrivals too, is waited for before TMEM and the block go
    ptx::mbar_wait(&drained, 0, &never, kWaitLimitNs);
  }
  __syncwarp();
  __syncthreads();
  if constexpr (!GRAD) cluster_arrive();   // this CTA's slice of P is there
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM);
  }
  if constexpr (!GRAD) {
    // CTA `slice` adds up its share of the rows, over the cluster in rank order
    __syncwarp();
    const float sc = p.scale ? __ldg(p.scale + a) : 1.f;
    uint8_t* image = p.image + static_cast<size_t>(slot) * RT::IMAGE;
    auto row_of = [&](int i) { return i / (RP / 4) * static_cast<int>(CS) + slice; };
    auto id_of = [&](int i) {
      return p.h_out && i < kTile / static_cast<int>(CS) * (RP / 4) && start + row_of(i) < end
                 ? __ldg(p.order + start + row_of(i)) : -1;
    };
    int id = id_of(tid);   // in flight across the barrier
    cluster_wait();
    for (int i = tid; i < kTile / static_cast<int>(CS) * (RP / 4); i += C::THREADS) {
      const int m = row_of(i), j = i % (RP / 4) * 4;
      if (start + m >= end) break;   // what the image holds there reaches that row of the product alone
      const float4* from = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + m * C::PS + j);
      float4 x[8], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q)   // all in flight
        if (q < CS) x[q] = ld_cluster(from, q);
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q)
        if (q < CS) v.x += x[q].x, v.y += x[q].y, v.z += x[q].z, v.w += x[q].w;
      if (j >= R) v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < R && id >= 0 && id < p.rows) *reinterpret_cast<float4*>(p.h_out + static_cast<size_t>(id) * R + j) = v;
      id = id_of(i + C::THREADS);
      uint32_t w[kTerms][2];
      split3(v.x * sc, v.y * sc, w[0][0], w[1][0], w[2][0]);
      split3(v.z * sc, v.w * sc, w[0][1], w[1][1], w[2][1]);
#pragma unroll
      for (int q = 0; q < kTerms; ++q)
        *reinterpret_cast<uint2*>(image + q * RT::BYTES + RT::at(m, j / 8) + j % 8 * 2) = make_uint2(w[q][0], w[q][1]);
    }
    __syncwarp();
    cluster_arrive();   // no CTA leaves while another one reads its shared memory
    cluster_wait();
  }
}

template <int RP, bool PROJ, bool GRAD>
int launch_stream(const StreamArgs& p, cudaStream_t s) {
  using C = StreamCfg<RP, PROJ, GRAD>;
  static std::atomic<uint64_t> done{0};
  auto kernel = lora_stream_kernel<RP, PROJ, GRAD>;
  const int st = allow_smem(done, kernel, C::SMEM);
  if (st != MOE_OK) return st;
  CUtensorMap mx, mm;
  if (!make_map(&mx, p.X, 2, p.rows, p.W, 1)) return MOE_ERR_CUDA;
  mm = mx;
  if (PROJ && !GRAD && !make_adapter_map(&mm, p.M, p.n, p.R, p.W, RP, 64)) return MOE_ERR_CUDA;
  if (PROJ && GRAD && !make_adapter_map(&mm, p.M, p.n, p.W, p.R, kTile, RP < 64 ? RP : 64)) return MOE_ERR_CUDA;
  const unsigned slots = static_cast<unsigned>(p.rows / p.chunk + p.n), slices = (p.W + p.cols - 1) / p.cols;
  if constexpr (!GRAD)
    return launch_cluster("lora_stream_kernel", kernel, dim3(slots * p.cluster), dim3(C::THREADS), C::SMEM, p.cluster, s,
                          p, mx, mm);
  else
    return launch_pdl("lora_stream_kernel", kernel, dim3(slots, slices), dim3(C::THREADS), C::SMEM, s, p, mx, mm);
}
template <bool PROJ, bool GRAD>
int launch_stream_rank(const StreamArgs& p, cudaStream_t s) {
  if (p.R <= 16) return launch_stream<16, PROJ, GRAD>(p, s);
  if (p.R <= 32) return launch_stream<32, PROJ, GRAD>(p, s);
  if (p.R <= 64) return launch_stream<64, PROJ, GRAD>(p, s);
  return launch_stream<128, PROJ, GRAD>(p, s);
}

}  // namespace

bool make_adapter_map(CUtensorMap* m, const void* base, uint64_t n, uint64_t rows, uint64_t cols, uint32_t box_rows,
                      uint32_t box_cols) {
  const EncodeTiledFn enc = get_encode_fn();
  if (!enc) {
    record_cuda_error(cudaErrorNotSupported, "cuTensorMapEncodeTiled unavailable from the driver");
    return false;
  }
  const cuuint64_t dims[3] = {cols, rows, n};
  const cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapSwizzle swizzle = box_cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_32B;
  if (enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
    record_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled rejected the adapters' layout");
    return false;
  }
  return true;
}

int lora_stream_max_cols(int R, bool proj) {
  auto blocks = [=](auto with, auto without) { return kTile * (proj ? decltype(with)::BLOCKS : decltype(without)::BLOCKS); };
  return R <= 16   ? blocks(StreamCfg<16, true, true>(), StreamCfg<16, false, true>())
         : R <= 32 ? blocks(StreamCfg<32, true, true>(), StreamCfg<32, false, true>())
         : R <= 64 ? blocks(StreamCfg<64, true, true>(), StreamCfg<64, false, true>())
                   : blocks(StreamCfg<128, true, true>(), StreamCfg<128, false, true>());
}

int launch_lora_stream(const StreamArgs& p, StreamKind kind, cudaStream_t s) {
  if (kind == kStreamProject) return launch_stream_rank<true, false>(p, s);
  if (kind == kStreamBoth) return launch_stream_rank<true, true>(p, s);
  return launch_stream_rank<false, true>(p, s);
}

}  // namespace moe
