// One pass over a wide operand X [rows, W] of the adapters' forward and
// gradients, its products on the tensor cores (tcgen05, fp32 sums in TMEM):
//   projection  P[r] = X[r] M_a^T            h = x A^T,   dh = s dC B
//   gradient    G_a  = sum_r X[r]^T V[r]     dB = dC^T (s h),   dA^T = x^T dh
// over the rows r of adapter a.  X crosses HBM once: the pass over dC does
// both products on the same tile, the one in X's own orientation, the other in
// its transpose, which the MMA reads from the same shared memory (a K-major
// and an MN-major descriptor of one 128-byte-swizzled tile).
//
// A CTA takes a chunk of one adapter's rows and a slice of X's columns and
// walks it in tiles of 128 rows x 128 columns.  The projection alone has
// chunks of 128 rows; the slices of a row meet in a cluster, through
// distributed shared memory and in rank order, so h leaves it complete.  With
// the gradient, G stays in TMEM until the chunk ends (one accumulator to 128
// columns) and P is complete for the slice after each 128 rows; what several
// CTAs add to (P over slices, G over chunks) is written as fp32 partial sums
// and added in a fixed order by the kernels that follow, except G of an adapter
// with a single chunk, which is written in place.  With ranks up to 32 two CTAs
// share an SM, so that the one's start, end and change of rows hide behind the
// other's loads.
//
// V enters as three bf16 terms (all 24 bits of an fp32 value): G is an fp32
// sum, and fewer terms would leave their rounding as the largest error in it.
// Up to rank 32 the terms lie side by side in the MMA's N, which costs nothing
// (an MMA of N <= 64 is bound by reading its A operand); above, one after the
// other into the same accumulator.
//
// Warps 0-3 load X (rows are gathered through the plan's order, 16 bytes a
// cp.async, swizzled by hand), 4-7 prepare V and empty TMEM, one thread of
// warp 8 issues the MMAs.  Every wait has a time limit; one that runs out
// raises the block's abort flag, every role leaves its loop, copies and MMAs in
// flight are waited for, TMEM is freed and MOE_ERR_TIMEOUT is left in *status.
#include <cstdint>

#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

constexpr int kStreamThreads = 288;
constexpr int kTile = 128;                 // rows and columns of a tile
constexpr int kSub = kTile * 128;          // bytes of 128 rows x 64 columns
constexpr int kTerms = 3;

template <int RP, bool PROJ, bool GRAD>
struct StreamCfg {
  static constexpr bool STACK = RP <= 32;
  static constexpr int GCOLS = GRAD ? (STACK ? kTerms * RP : RP) : 0;       // TMEM columns of 128 of X's
  static constexpr int BLOCKS = !GRAD ? 1 : RP <= 16 ? 4 : RP <= 32 ? 2 : RP <= 64 ? 4 : 2;  // 128-column blocks, at most
  static constexpr int PBUF = GRAD ? 2 : 1;                                 // projection accumulators
  static constexpr int PS = RP + 4;                                         // row stride of P in shared memory: spreads the banks
  static constexpr int PCOL = GRAD ? BLOCKS * GCOLS : 0;                    // their first TMEM column
  static constexpr int USED = PCOL + (PROJ ? PBUF * RP : 0);
  static constexpr int TMEM = USED <= 32 ? 32 : USED <= 64 ? 64 : USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
  static constexpr int MSUB = RP * 128;                                     // bytes of M for 64 columns
  static constexpr int M_ALL = PROJ && GRAD ? BLOCKS * 2 * MSUB : 0;        // resident
  static constexpr int V_SUB = GRAD ? kTerms * RP * 128 : 0;                // bytes of V's terms for 64 rows
  static constexpr int STAGE = 2 * kSub + (PROJ && !GRAD ? 2 * MSUB : 0);
  static constexpr int PER_SM = RP <= 32 || (!GRAD && RP <= 64) ? 2 : 1;
  static constexpr int BUDGET = PER_SM == 2 ? 110 * 1024 : 226 * 1024;
  static constexpr int STAGES_RAW = (BUDGET - M_ALL - 2 * V_SUB) / STAGE;
  static constexpr int STAGES = STAGES_RAW > 4 ? 4 : STAGES_RAW;
  static constexpr int SMEM = STAGES * STAGE + M_ALL + 2 * V_SUB + 1024;    // + alignment slack
  static_assert(USED <= 512 && STAGES >= 2 && (GRAD || kTile * PS * 4 <= STAGES * STAGE), "TMEM and shared memory");
};

// 16 accumulator columns from `col` on, the terms added up, smallest first
template <bool STACK, int RP>
__device__ __forceinline__ void load_grad16(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  ptx::tmem_ld_32x32b_x16(at, r);
  if constexpr (STACK) {
    uint32_t s[16], t[16];
    ptx::tmem_ld_32x32b_x16(at + RP, s);
    ptx::tmem_ld_32x32b_x16(at + 2 * RP, t);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[i] = __uint_as_float(r[i]) + (__uint_as_float(s[i]) + __uint_as_float(t[i]));
  } else {
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  }
}

template <int RP, bool PROJ, bool GRAD>
__global__ void __launch_bounds__(kStreamThreads, StreamCfg<RP, PROJ, GRAD>::PER_SM)
    lora_stream_kernel(const StreamArgs p) {
  using C = StreamCfg<RP, PROJ, GRAD>;
  constexpr int S = C::STAGES;
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_m = smem + S * C::STAGE;
  uint8_t* s_v = s_m + C::M_ALL;
  __shared__ __align__(8) uint64_t full[S], empty[S], v_full, step_done[2], p_free[2], drained;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.status && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.status = MOE_OK;
  const uint32_t CS = GRAD ? 1 : cluster_size();
  const int slot = GRAD ? blockIdx.x : blockIdx.x / CS, slice = GRAD ? blockIdx.y : cluster_rank();
  int a, start, end;
  if (!find_tile(p.offsets, p.n, p.rows, p.chunk, slot, a, start, end) || a == p.n) return;  // the whole cluster leaves
  const int W = p.W, R = p.R;
  const int col0 = slice * p.cols;
  const int blocks = max(0, min(p.cols, W - col0) + kTile - 1) / kTile;  // none behind the last column
  const int steps = (end - start + kTile - 1) / kTile;
  const int tiles = steps * blocks;
  const bool want_p = PROJ && p.proj, want_g = GRAD && p.grad;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&full[i], 128);
      ptx::mbar_init(&empty[i], 1);
    }
    ptx::mbar_init(&v_full, 128);
    ptx::mbar_init(&step_done[0], 1);
    ptx::mbar_init(&step_done[1], 1);
    ptx::mbar_init(&drained, 1);
    ptx::mbar_init(&p_free[0], 128);
    ptx::mbar_init(&p_free[1], 128);
    s_abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 8) {
    ptx::tmem_alloc(&s_tmem, C::TMEM);
    ptx::tmem_relinquish();
  } else if (PROJ && GRAD) {
    // M = B's slice, transposed on the way: rank j's row of 64 columns, for each 64
    const __nv_bfloat16* src = p.M + static_cast<size_t>(a) * W * R;
    for (int i = tid; i < blocks * kTile * (RP / 8); i += 256) {
      const int n = i % (blocks * kTile), j = i / (blocks * kTile) * 8;
      const bool in = col0 + n < W && j < R;
      const uint4 v = in ? ldg16(src + static_cast<size_t>(col0 + n) * R + j) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint8_t* t = s_m + n / 64 * C::MSUB;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<uint16_t*>(t + swz(j + u, n % 64 / 8) + n % 8 * 2) =
            static_cast<uint16_t>(w[u / 2] >> (u % 2 * 16));
    }
    ptx::fence_proxy_async_smem();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto give_up = [&]() {
    s_abort = 1;
    if (p.status) set_status(p.status, MOE_ERR_TIMEOUT);
  };

  if (warp < 4) {
    // ---- X: tile t goes to stage t % S; what is landed is handed over S - 1 tiles later
    constexpr int LAG = S - 1;
    int row[16];
    auto hand_over = [&](int t) {
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&full[t % S]);
    };
    bool ok = true;
    int t = 0;
    for (int step = 0; step < steps && ok; ++step) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int at = start + step * kTile + i * 8 + tid / 16;
        const int r = at < end ? __ldg(p.order + at) : -1;
        row[i] = r >= 0 && r < p.rows ? r : -1;
      }
      for (int b = 0; b < blocks; ++b, ++t) {
        if (t >= S && !ptx::mbar_wait(&empty[t % S], (t / S - 1) & 1, abort_flag, kWaitLimitNs)) {
          give_up();
          ok = false;
          break;
        }
        const uint32_t dst = ptx::smem_u32(smem + t % S * C::STAGE);
        const int c16 = tid % 16, col = col0 + b * kTile + c16 * 8;
        const __nv_bfloat16* src = p.X + col;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool in = row[i] >= 0 && col < W;
          cp_async16z(dst + c16 / 8 * kSub + swz(i * 8 + tid / 16, c16 % 8),
                      in ? src + static_cast<size_t>(row[i]) * W : p.X, in);
        }
        if constexpr (PROJ && !GRAD) {  // M = A's columns of this tile
#pragma unroll
          for (int i = 0; i < RP / 8; ++i) {
            const int j = i * 8 + tid / 16;
            const bool in = j < R && col < W;
            cp_async16z(dst + 2 * kSub + c16 / 8 * C::MSUB + swz(j, c16 % 8),
                        in ? p.M + (static_cast<size_t>(a) * R + j) * W + col : p.M, in);
          }
        }
        cp_commit();
        if (t >= LAG) {
          cp_wait<LAG>();
          hand_over(t - LAG);
        }
      }
    }
    cp_wait<0>();
    if (ok)
      for (int u = tiles > LAG ? tiles - LAG : 0; u < tiles; ++u) hand_over(u);
  } else if (warp < 8) {
    // ---- V in, P out, and at the end G
    const int et = tid - 128, ew = warp - 4;
    const uint32_t lane_base = static_cast<uint32_t>(ew * 32) << 16;
    const float sc = PROJ && GRAD && p.scale ? __ldg(p.scale + a) : 1.f;
    auto prepare = [&](int step) {  // rows of V as three terms, rank j's row of 64 of the tile's rows
      if constexpr (GRAD) {
        for (int i = et; i < RP * 16; i += 128) {
          const int j = i % RP, r0 = i / RP * 8;
          float v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int at = start + step * kTile + r0 + u;
            int r = at < end ? (PROJ ? __ldg(p.order + at) : at) : -1;
            if (PROJ && r >= p.rows) r = -1;
            v[u] = r >= 0 && j < R ? __ldg(p.V + static_cast<size_t>(r) * R + j) * sc : 0.f;
          }
          uint32_t w[kTerms][4];
#pragma unroll
          for (int u = 0; u < 4; ++u) split3(v[2 * u], v[2 * u + 1], w[0][u], w[1][u], w[2][u]);
#pragma unroll
          for (int q = 0; q < kTerms; ++q)
            *reinterpret_cast<uint4*>(s_v + r0 / 64 * C::V_SUB + swz(q * RP + j, r0 % 64 / 8)) =
                make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&v_full);
      }
    };
    if (want_g) prepare(0);
    bool ok = true;
    for (int step = 0; step < (GRAD ? steps : 0); ++step) {
      // the step's MMAs are done: V may be replaced, P is complete
      if (!ptx::mbar_wait_warp(&step_done[step & 1], (step >> 1) & 1, abort_flag, kWaitLimitNs)) {
        give_up();
        ok = false;
        break;
      }
      if (want_g && step + 1 < steps) prepare(step + 1);
      if constexpr (PROJ) {
        if (want_p) {
          ptx::tc_fence_after();
          const int at = start + step * kTile + ew * 32 + lane;
          float* o = p.proj + (static_cast<size_t>(slice) * p.rows + at) * R;
          const uint32_t from = tmem + lane_base + C::PCOL + step % C::PBUF * RP;
#pragma unroll
          for (int j = 0; j < RP; j += 16) {
            uint32_t r[16];
            __syncwarp();
            ptx::tmem_ld_32x32b_x16(from + j, r);
            ptx::tmem_ld_wait();
            if (at < end) {
#pragma unroll
              for (int u = 0; u < 16; u += 4)
                if (j + u < R)
                  *reinterpret_cast<float4*>(o + j + u) =
                      make_float4(__uint_as_float(r[u]) * sc, __uint_as_float(r[u + 1]) * sc,
                                  __uint_as_float(r[u + 2]) * sc, __uint_as_float(r[u + 3]) * sc);
            }
          }
          ptx::tc_fence_before();
          ptx::mbar_arrive(&p_free[step % C::PBUF]);
        }
      }
    }
    if constexpr (!GRAD) {   // the slice's P to shared memory, over the stages: their MMAs are done
      float* s_p = reinterpret_cast<float*>(smem) + et * C::PS;
      if (blocks == 0) {
        for (int j = 0; j < RP; j += 4) *reinterpret_cast<float4*>(s_p + j) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else if (ptx::mbar_wait_warp(&step_done[0], 0, abort_flag, kWaitLimitNs)) {
        ptx::tc_fence_after();
#pragma unroll
        for (int j = 0; j < RP; j += 16) {
          uint32_t r[16];
          __syncwarp();
          ptx::tmem_ld_32x32b_x16(tmem + lane_base + j, r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            *reinterpret_cast<uint4*>(s_p + j + u) = make_uint4(r[u], r[u + 1], r[u + 2], r[u + 3]);
        }
      } else {
        give_up();
      }
    }
    if constexpr (GRAD) {
      if (want_g && ok) {
        ptx::tc_fence_after();
        const int first = held_offset(p.offsets, p.n, p.rows, a), last = held_offset(p.offsets, p.n, p.rows, a + 1);
        const bool whole = last - first <= p.chunk;  // no other chunk adds to it
        const size_t size = static_cast<size_t>(W) * R;
        float* part = p.part + static_cast<size_t>(slot) * size;
        float* g32 = static_cast<float*>(p.grad) + a * size;
        __nv_bfloat16* g16 = static_cast<__nv_bfloat16*>(p.grad) + a * size;
        for (int b = 0; b < blocks; ++b) {
          const int k = col0 + b * kTile + ew * 32 + lane;
#pragma unroll
          for (int j = 0; j < RP; j += 16) {
            float v[16];
            __syncwarp();
            load_grad16<C::STACK, RP>(tmem + lane_base + b * C::GCOLS + j, v);
            if (k >= W) {
            } else if constexpr (PROJ) {  // [W][R]: a column's ranks side by side
              const size_t o = static_cast<size_t>(k) * R + j;
#pragma unroll
              for (int u = 0; u < 16; u += 8) {
                if (j + u >= R) continue;
                float x[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) x[q] = v[u + q];
                if (!whole) store8(part + o + u, x);
                else if (p.grad_f32) store8(g32 + o + u, x);
                else store8(g16 + o + u, x);
              }
            } else {                      // [R][W]
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                if (j + u >= R) continue;
                const size_t o = static_cast<size_t>(j + u) * W + k;
                if (!whole) part[o] = v[u];
                else if (p.grad_f32) g32[o] = v[u];
                else g16[o] = __float2bfloat16_rn(v[u]);
              }
            }
          }
        }
      }
    }
    ptx::tc_fence_before();
  } else if (lane == 0) {
    // ---- MMAs
    constexpr uint32_t IP = ptx::make_idesc(128, RP, 1);
    constexpr uint32_t IG = ptx::make_idesc(128, C::STACK ? kTerms * RP : RP, 1) | kAMn;
    bool ok = true;
    int t = 0;
    for (int step = 0; step < steps && blocks > 0 && ok; ++step) {
      if (want_g) ok = ptx::mbar_wait(&v_full, step & 1, abort_flag, kWaitLimitNs);
      if (want_p && step >= C::PBUF)
        ok = ok && ptx::mbar_wait(&p_free[step % C::PBUF], (step / C::PBUF - 1) & 1, abort_flag, kWaitLimitNs);
      for (int b = 0; b < blocks && ok; ++b, ++t) {
        ok = ptx::mbar_wait(&full[t % S], (t / S) & 1, abort_flag, kWaitLimitNs);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t x = ptx::smem_u32(smem + t % S * C::STAGE);
        if (want_p) {
          const uint32_t m = PROJ && !GRAD ? x + 2 * kSub : ptx::smem_u32(s_m) + b * 2 * C::MSUB;
          const uint32_t d = tmem + C::PCOL + step % C::PBUF * RP;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            ptx::umma_f16(d, ptx::sw128_kmajor_desc(x + k / 4 * kSub) + k % 4 * 2,
                          ptx::sw128_kmajor_desc(m + k / 4 * C::MSUB) + k % 4 * 2, IP, b > 0 || k > 0);
        }
        if (want_g) {
          const uint32_t v = ptx::smem_u32(s_v);
          const uint32_t d = tmem + b * C::GCOLS;
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // 16 rows at a time
            const uint64_t xd = mn_desc(x + k * 2048, kSub);
            const uint64_t vd = ptx::sw128_kmajor_desc(v + k / 4 * C::V_SUB) + k % 4 * 2;
            if constexpr (C::STACK) {
              ptx::umma_f16(d, xd, vd, IG, step > 0 || k > 0);
            } else {
#pragma unroll
              for (int q = 0; q < kTerms; ++q)
                ptx::umma_f16(d, xd, vd + (q * RP * 128 >> 4), IG, step > 0 || k > 0 || q > 0);
            }
          }
        }
        ptx::umma_commit(&empty[t % S]);
      }
      if (ok) ptx::umma_commit(&step_done[step & 1]);
    }
    if (!ok) {
      give_up();
      int never = 0;   // what was issued is waited for before TMEM goes
      ptx::umma_commit(&drained);
      ptx::mbar_wait(&drained, 0, &never, kWaitLimitNs);
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM);
  }
  if constexpr (!GRAD) {
    // CTA `slice` adds up its share of the rows, over the cluster in rank order
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int i = tid; i < kTile / static_cast<int>(CS) * (RP / 4); i += kStreamThreads) {
      const int m = i / (RP / 4) * static_cast<int>(CS) + slice, j = i % (RP / 4) * 4;
      if (start + m >= end || j >= R) continue;
      const float4* from = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + m * C::PS + j);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t q = 0; q < CS; ++q) {
        const float4 u = ld_cluster(from, q);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      *reinterpret_cast<float4*>(p.proj + static_cast<size_t>(start + m) * R + j) = v;
      const int r = p.h_out ? __ldg(p.order + start + m) : -1;
      if (r >= 0 && r < p.rows) *reinterpret_cast<float4*>(p.h_out + static_cast<size_t>(r) * R + j) = v;
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
  const unsigned slots = static_cast<unsigned>(p.rows / p.chunk + p.n), slices = (p.W + p.cols - 1) / p.cols;
  if constexpr (!GRAD)
    return launch_cluster("lora_stream_kernel", kernel, dim3(slots * p.cluster), dim3(kStreamThreads), C::SMEM, p.cluster, s, p);
  else
    return launch_pdl("lora_stream_kernel", kernel, dim3(slots, slices), dim3(kStreamThreads), C::SMEM, s, p);
}
template <bool PROJ, bool GRAD>
int launch_stream_rank(const StreamArgs& p, cudaStream_t s) {
  if (p.R <= 16) return launch_stream<16, PROJ, GRAD>(p, s);
  if (p.R <= 32) return launch_stream<32, PROJ, GRAD>(p, s);
  if (p.R <= 64) return launch_stream<64, PROJ, GRAD>(p, s);
  return launch_stream<128, PROJ, GRAD>(p, s);
}

}  // namespace

int lora_stream_max_cols(int R) {
  return kTile * (R <= 16   ? StreamCfg<16, true, true>::BLOCKS
                  : R <= 32 ? StreamCfg<32, true, true>::BLOCKS
                  : R <= 64 ? StreamCfg<64, true, true>::BLOCKS
                            : StreamCfg<128, true, true>::BLOCKS);
}

int launch_lora_stream(const StreamArgs& p, StreamKind kind, cudaStream_t s) {
  if (kind == kStreamProject) return launch_stream_rank<true, false>(p, s);
  if (kind == kStreamBoth) return launch_stream_rank<true, true>(p, s);
  return launch_stream_rank<false, true>(p, s);
}

}  // namespace moe
