// The adapters' second product, out[r] = base[r] + h[r] W_a over the R ranks:
//   forward   h = s x A^T,  W = B^T, B [n, N, R]
//   backward  dx[r] = dx_base[r] + dh[r] A,  W = A,   A [n, R, d]
// on the tensor cores (tcgen05, fp32 sums in TMEM).  Bound by memory: base and
// out cross HBM once, so the kernel is a copy with a small product in its
// middle.  A CTA takes up to 128 rows of one adapter and a slice of the
// columns, 64 at a time: warps 0-3 bring the base tile and the adapter's
// columns (cp.async into a ring of stages), one thread of warp 8 issues the
// 128 x 64 MMAs into one of two accumulators, warps 4-7 add the accumulator to
// the base tile in shared memory, where a thread holds a row, and write it out
// from there, where 8 neighbouring lanes hold one: full 128-byte lines both
// ways although the rows lie scattered.
//
// h enters as two bf16 terms (hi + lo, 2^-17 of it left out) for a bf16 result
// and as three (all of an fp32 value) for an fp32 one: one term's rounding
// would stand beside the result's own.
//
// Waits are limited and abort as in the streaming pass.
#include <cstdint>

#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

constexpr int kExpandThreads = 288;
constexpr int kRows = 128;
constexpr int kBC = 64;  // columns of a block

template <int RP, bool KN, typename OT>
struct ExpandCfg {
  static constexpr int TERMS = sizeof(OT) == 4 ? 3 : 2;
  static constexpr int HSUBS = (TERMS * RP + 63) / 64;
  static constexpr int H = HSUBS * kRows * 128;                    // h's terms, [128][64] tiles
  static constexpr int BASE = kRows * kBC * sizeof(OT);
  static constexpr int WBYTES = KN ? RP * 128 : (RP + 63) / 64 * kBC * 128;
  static constexpr int STAGE = BASE + WBYTES;
  static constexpr int PER_SM = (110 * 1024 - H) / STAGE >= 2 ? 2 : 1;
  static constexpr int STAGES_RAW = ((PER_SM == 2 ? 110 : 224) * 1024 - H) / STAGE;
  static constexpr int STAGES = STAGES_RAW > 4 ? 4 : STAGES_RAW;
  static constexpr int SMEM = STAGES * STAGE + H + 1024;
  static_assert(STAGES >= 2, "shared memory");
};

template <int RP, bool KN, typename OT>
__global__ void __launch_bounds__(kExpandThreads, ExpandCfg<RP, KN, OT>::PER_SM)
    lora_expand_kernel(const ExpandArgs p) {
  using C = ExpandCfg<RP, KN, OT>;
  constexpr int S = C::STAGES;
  constexpr int VEC = 16 / sizeof(OT);          // values of a 16-byte piece
  constexpr int PIECES = kBC / VEC;             // of a row's block: 8 or 16
  constexpr int PER = kRows * PIECES / 128;     // a thread's
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_h = smem + S * C::STAGE;
  __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[2], acc_free[2], h_full, drained;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_row[kRows];
  volatile int* abort_flag = &s_abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int a, start, end;
  if (!find_tile(p.offsets, p.n, p.rows, kRows, blockIdx.x, a, start, end)) return;
  const int N = p.N, R = p.R;
  const int col0 = blockIdx.y * p.cols, col1 = min(N, col0 + p.cols);
  OT* out = static_cast<OT*>(p.out);
  const OT* base = static_cast<const OT*>(p.base);
  if (tid < kRows) {
    const int r = start + tid < end ? __ldg(p.order + start + tid) : -1;
    s_row[tid] = r >= 0 && r < p.rows ? r : -1;
  }
  if (a == p.n) {  // rows without an adapter
    __syncthreads();
    if (p.h_out && blockIdx.y == 0)
      for (int i = tid; i < kRows * R; i += kExpandThreads)
        if (s_row[i / R] >= 0) p.h_out[static_cast<size_t>(s_row[i / R]) * R + i % R] = 0.f;
    if (base == out) return;
    const int w8 = (col1 - col0) / 8;
    for (int i = tid; i < kRows * w8; i += kExpandThreads) {
      const int r = s_row[i / w8];
      if (r < 0) continue;
      const size_t o = static_cast<size_t>(r) * N + col0 + i % w8 * 8;
      float v[8] = {};
      if (base) load8(base + o, v);
      store8(out + o, v);
    }
    return;
  }
  const int blocks = (col1 - col0 + kBC - 1) / kBC;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&full[i], 128);
      ptx::mbar_init(&empty[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&acc_full[i], 1);
      ptx::mbar_init(&acc_free[i], 128);
    }
    ptx::mbar_init(&h_full, 128);
    ptx::mbar_init(&drained, 1);
    s_abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 8) {
    ptx::tmem_alloc(&s_tmem, 2 * kBC);
    ptx::tmem_relinquish();
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
    // ---- base tiles and the adapter's columns
    constexpr int LAG = S - 1;
    auto hand_over = [&](int t) {
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&full[t % S]);
    };
    const __nv_bfloat16* M = p.M + static_cast<size_t>(a) * N * R;
    bool ok = true;
    for (int t = 0; t < blocks; ++t) {
      if (t >= S && !ptx::mbar_wait(&empty[t % S], (t / S - 1) & 1, abort_flag, kWaitLimitNs)) {
        give_up();
        ok = false;
        break;
      }
      const uint32_t dst = ptx::smem_u32(smem + t % S * C::STAGE);
      const int col = col0 + t * kBC;
      if (base) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int m = i * (128 / PIECES) + tid / PIECES, c = tid % PIECES;
          const int r = s_row[m];
          const bool in = r >= 0 && col + c * VEC < col1;
          cp_async16z(dst + c / 8 * (kRows * 128) + swz(m, c % 8),
                      in ? base + static_cast<size_t>(r) * N + col + c * VEC : base, in);
        }
      }
      const uint32_t w = dst + C::BASE;
      if constexpr (KN) {  // rank j's row of 64 columns
        for (int i = tid; i < RP * 8; i += 128) {
          const int j = i / 8, c = i % 8;
          const bool in = j < R && col + c * 8 < col1;
          cp_async16z(w + swz(j, c), in ? M + static_cast<size_t>(j) * N + col + c * 8 : M, in);
        }
      } else {             // column n's row of ranks
#pragma unroll
        for (int i = tid; i < kBC * (RP / 8); i += 128) {
          const int n = i / (RP / 8), c = i % (RP / 8);
          const bool in = col + n < col1 && c * 8 < R;
          cp_async16z(w + c / 8 * (kBC * 128) + swz(n, c % 8),
                      in ? M + static_cast<size_t>(col + n) * R + c * 8 : M, in);
        }
      }
      cp_commit();
      if (t >= LAG) {
        cp_wait<LAG>();
        hand_over(t - LAG);
      }
    }
    cp_wait<0>();
    if (ok)
      for (int u = blocks > LAG ? blocks - LAG : 0; u < blocks; ++u) hand_over(u);
  } else if (warp < 8) {
    // ---- h's terms in, then block by block: accumulator + base, out
    const int et = tid - 128, ew = warp - 4;
    const uint32_t lane_base = static_cast<uint32_t>(ew * 32) << 16;
    const float sc = p.scale ? __ldg(p.scale + a) : 1.f;
    for (int i = et; i < kRows * (RP / 8); i += 128) {
      const int m = i / (RP / 8), j = i % (RP / 8) * 8;
      float v[8] = {};
      if (start + m < end && j < R) load8(p.h + static_cast<size_t>(start + m) * R + j, v);
      uint32_t w[3][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if constexpr (C::TERMS == 3)
          split3(v[2 * u] * sc, v[2 * u + 1] * sc, w[0][u], w[1][u], w[2][u]);
        else
          split2(v[2 * u] * sc, v[2 * u + 1] * sc, w[0][u], w[1][u]);
      }
#pragma unroll
      for (int q = 0; q < C::TERMS; ++q) {
        const int k = q * RP + j;
        *reinterpret_cast<uint4*>(s_h + k / 64 * (kRows * 128) + swz(m, k % 64 / 8)) =
            make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
      }
    }
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(&h_full);
    for (int t = 0; t < blocks; ++t) {
      const bool ok = ptx::mbar_wait_warp(&full[t % S], (t / S) & 1, abort_flag, kWaitLimitNs) &&
                      ptx::mbar_wait_warp(&acc_full[t & 1], (t >> 1) & 1, abort_flag, kWaitLimitNs);
      if (!ok) {
        give_up();
        break;
      }
      ptx::tc_fence_after();
      uint8_t* tile = smem + t % S * C::STAGE;
      const int m = ew * 32 + lane;
      const uint32_t from = tmem + lane_base + (t & 1) * kBC;
#pragma unroll
      for (int k = 0; k < kBC; k += 32) {
        uint32_t r[32];
        __syncwarp();
        ptx::tmem_ld_32x32b_x32(from + k, r);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < 32; u += VEC) {
          const int c = (k + u) / VEC;
          uint4* at = reinterpret_cast<uint4*>(tile + c / 8 * (kRows * 128) + swz(m, c % 8));
          uint4 v = make_uint4(0, 0, 0, 0);
          if (base) v = *at;
          if constexpr (sizeof(OT) == 4) {
            v.x = __float_as_uint(__uint_as_float(v.x) + __uint_as_float(r[u]));
            v.y = __float_as_uint(__uint_as_float(v.y) + __uint_as_float(r[u + 1]));
            v.z = __float_as_uint(__uint_as_float(v.z) + __uint_as_float(r[u + 2]));
            v.w = __float_as_uint(__uint_as_float(v.w) + __uint_as_float(r[u + 3]));
          } else {
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = pack2(__uint_as_float(w[q] << 16) + __uint_as_float(r[u + 2 * q]),
                           __uint_as_float(w[q] & 0xffff0000u) + __uint_as_float(r[u + 2 * q + 1]));
            v = make_uint4(w[0], w[1], w[2], w[3]);
          }
          *at = v;
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&acc_free[t & 1]);
      __syncwarp();
      const int col = col0 + t * kBC;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {  // the warp's 32 rows, PIECES lanes to a row
        const int q = ew * 32 + i * (32 / PIECES) + lane / PIECES, c = lane % PIECES;
        const int r = s_row[q];
        const uint4 v = *reinterpret_cast<const uint4*>(tile + c / 8 * (kRows * 128) + swz(q, c % 8));
        if (r >= 0 && col + c * VEC < col1)
          *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * N + col + c * VEC) = v;
      }
      ptx::mbar_arrive(&empty[t % S]);
    }
  } else if (lane == 0) {
    // ---- MMAs
    constexpr uint32_t ID = ptx::make_idesc(128, kBC, 1) | (KN ? kBMn : 0u);
    bool ok = ptx::mbar_wait(&h_full, 0, abort_flag, kWaitLimitNs);
    const uint32_t h = ptx::smem_u32(s_h);
    for (int t = 0; t < blocks && ok; ++t) {
      ok = ptx::mbar_wait(&full[t % S], (t / S) & 1, abort_flag, kWaitLimitNs);
      if (ok && t >= 2) ok = ptx::mbar_wait(&acc_free[t & 1], ((t >> 1) - 1) & 1, abort_flag, kWaitLimitNs);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t w = ptx::smem_u32(smem + t % S * C::STAGE) + C::BASE;
      const uint32_t d = tmem + (t & 1) * kBC;
#pragma unroll
      for (int q = C::TERMS - 1; q >= 0; --q)  // the small terms first
#pragma unroll
        for (int k = 0; k < RP / 16; ++k) {
          const int kk = q * (RP / 16) + k;
          const uint64_t hd = ptx::sw128_kmajor_desc(h + kk / 4 * (kRows * 128)) + kk % 4 * 2;
          const uint64_t wd = KN ? mn_desc(w + k * 2048, RP * 128)
                                 : ptx::sw128_kmajor_desc(w + k / 4 * (kBC * 128)) + k % 4 * 2;
          ptx::umma_f16(d, hd, wd, ID, q < C::TERMS - 1 || k > 0);
        }
      ptx::umma_commit(&acc_full[t & 1]);
    }
    if (!ok) {
      give_up();
      int never = 0;
      ptx::umma_commit(&drained);
      ptx::mbar_wait(&drained, 0, &never, kWaitLimitNs);
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 2 * kBC);
  }
}

template <int RP, bool KN, typename OT>
int launch_expand_tile(const ExpandArgs& p, cudaStream_t s) {
  using C = ExpandCfg<RP, KN, OT>;
  static std::atomic<uint64_t> done{0};
  auto kernel = lora_expand_kernel<RP, KN, OT>;
  const int st = allow_smem(done, kernel, C::SMEM);
  if (st != MOE_OK) return st;
  return launch_pdl("lora_expand_kernel", kernel, dim3(p.rows / kRows + p.n + 1, (p.N + p.cols - 1) / p.cols),
                    dim3(kExpandThreads), C::SMEM, s, p);
}
template <bool KN, typename OT>
int launch_expand_rank(const ExpandArgs& p, cudaStream_t s) {
  if (p.R <= 16) return launch_expand_tile<16, KN, OT>(p, s);
  if (p.R <= 32) return launch_expand_tile<32, KN, OT>(p, s);
  if (p.R <= 64) return launch_expand_tile<64, KN, OT>(p, s);
  return launch_expand_tile<128, KN, OT>(p, s);
}

}  // namespace

int launch_lora_expand(ExpandArgs p, bool kn, int out_dtype, cudaStream_t s) {
  // columns of a CTA: the widest slice (up to 1024) that still gives every SM two CTAs
  const long long tiles = static_cast<long long>(p.rows) / kRows + p.n;
  p.cols = 1024;
  while (p.cols > 128 && tiles * ((p.N + p.cols - 1) / p.cols) < 2ll * num_sms()) p.cols /= 2;
  if (out_dtype == MOE_F32) return kn ? launch_expand_rank<true, float>(p, s) : launch_expand_rank<false, float>(p, s);
  return kn ? launch_expand_rank<true, __nv_bfloat16>(p, s) : launch_expand_rank<false, __nv_bfloat16>(p, s);
}

}  // namespace moe
