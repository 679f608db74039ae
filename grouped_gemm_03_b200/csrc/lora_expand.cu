// The adapters' second product, out[r] = base[r] + h[r] W_a over the R ranks:
//   forward   h = s x A^T,  W = B^T, B [n, N, R]
//   backward  dx[r] = dx_base[r] + dh[r] A,  W = A,   A [n, R, d]
// on the tensor cores (tcgen05, fp32 sums in TMEM).  Bound by memory: base and
// out cross HBM once, so the kernel is a copy with a small product in its
// middle.  A CTA takes up to 128 rows of one adapter and a slice of the
// columns, 64 at a time: warps 0-3 bring the base tile and the adapter's
// columns (TMA, the rows by gather4, into a ring of stages), one thread of warp
// 12 issues the 128 x 64 MMAs into one of two accumulators, warps 4-11 (two to a
// quarter of the rows, half of the columns each) add the accumulator to the base
// tile in shared memory, where a thread holds a row, and write it out from there,
// where neighbouring lanes hold one: full sectors both ways although the rows lie
// scattered.  Measured: 8192 rows of 4096 columns at rank 32, 29 us (4.6 TB/s
// with its start; 5.8 while it streams).
//
// h comes split and laid out (lora_tc.cuh), scale and all, by one bulk copy: as
// two bf16 terms (2^-17 of it left out) for a bf16 result and as three (all of
// an fp32 value) for an fp32 one.  One term's rounding would stand beside the
// result's own.
//
// Waits are limited and abort as in the streaming pass.
#include <cstdint>

#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

constexpr int kLoaders = 128, kDrainers = 256;
constexpr int kExpandThreads = kLoaders + kDrainers + 32;
constexpr int kMmaWarp = kExpandThreads / 32 - 1;
constexpr int kRows = 128;
constexpr int kBC = 64;  // columns of a block

template <int RP, bool KN, typename OT>
struct ExpandCfg {
  static constexpr int TERMS = sizeof(OT) == 4 ? 3 : 2;
  static constexpr int H = TERMS * RankTile<RP>::BYTES;            // h's terms
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
    lora_expand_kernel(const ExpandArgs p, const __grid_constant__ CUtensorMap map_base,
                       const __grid_constant__ CUtensorMap map_m) {
  using C = ExpandCfg<RP, KN, OT>;
  constexpr int S = C::STAGES;
  constexpr int VEC = 16 / sizeof(OT);          // values of a 16-byte piece
  constexpr int PIECES = kBC / VEC;             // of a row's block: 8 or 16
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_h = smem + S * C::STAGE;
  __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[2], acc_free[2], h_full, drained;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_row[kRows];
  volatile int* abort_flag = &s_abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], kDrainers);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&acc_full[i], 1);
      ptx::mbar_init(&acc_free[i], kDrainers);
    }
    ptx::mbar_init(&h_full, 1);
    ptx::mbar_init(&drained, 1);
    s_abort = 0;
    ptx::fence_mbar_init();
  }
  // Base, the plan and the weights are older than the launch before this one, which writes h: their loads
  // start while it runs.
  int a, start, end;
  const bool found = find_tile(p.offsets, p.n, p.rows, kRows, blockIdx.x, a, start, end);
  if (!found || (a == p.n && !p.apart)) {
    pdl_wait();
    pdl_launch_dependents();
    if (!found) return;
  }
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
    const int w8 = base == out ? 0 : (col1 - col0) / 8;
    for (int i = tid; i < kRows * w8; i += kExpandThreads) {
      const int r = s_row[i / w8];
      if (r < 0) continue;
      const size_t o = static_cast<size_t>(r) * N + col0 + i % w8 * 8;
      float v[8] = {};
      if (base) load8(base + o, v);
      store8(out + o, v);
    }
    if (p.apart) {
      pdl_wait();
      pdl_launch_dependents();
    }
    return;
  }
  const int blocks = (col1 - col0 + kBC - 1) / kBC;

  __syncthreads();
  uint32_t tmem = 0;
  if (warp >= kLoaders / 32) {   // TMEM only then: as in the streaming pass, which has its own before this one starts
    if (!p.apart) pdl_wait();
    if (warp == kMmaWarp) {
      if (!p.apart) pdl_launch_dependents();
      ptx::tmem_alloc(&s_tmem, 2 * kBC);
      ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    named_barrier(1, kExpandThreads - kLoaders);
    ptx::tc_fence_after();
    tmem = s_tmem;
  }
  auto give_up = [&]() {
    s_abort = 1;
    if (p.status) set_status(p.status, MOE_ERR_TIMEOUT);
  };

  if (warp < kLoaders / 32) {
    // ---- base tiles and the adapter's columns.  Lane l of a warp gathers its (l % 8)-th four rows, the
    // (l / 8)-th 128 bytes of the block; a row that is not there is taken from behind base, as zeros.
    constexpr int SUBS = kBC * sizeof(OT) / 128;
    const int quad = warp * 8 + lane % 8, sub = lane / 8, quads = (end - start + 3) / 4;  // none behind the last row
    const uint64_t policy = ptx::policy_evict_first();
    int row[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) row[u] = s_row[quad * 4 + u] >= 0 ? s_row[quad * 4 + u] : p.rows;
    bool ok = true;
    int t = 0;
    auto load_h = [&]() {
      if (warp) return;
      if (!p.apart) pdl_wait();
      if (lane) return;
      ptx::mbar_arrive_expect_tx(&h_full, C::H);
      bulk_load(s_h, p.h + static_cast<size_t>(blockIdx.x) * RankTile<RP>::IMAGE, C::H, &h_full);
    };
    // A warp without rows of base to bring stays out of the loop: the stages would turn without it, and a barrier
    // could turn twice between two of its looks.  Warp 0 brings the weights.
    const int mine = warp == 0 || (base && warp * 8 < quads) ? blocks : 0;
    for (; t < mine; ++t) {
      if (t == S) load_h();   // the ring is full
      if (t >= S && !ptx::mbar_wait_warp(&empty[t % S], (t / S - 1) & 1, abort_flag, kWaitLimitNs)) {
        give_up();
        ok = false;
        break;
      }
      uint8_t* dst = smem + t % S * C::STAGE;
      const int col = col0 + t * kBC;
      if (tid == 0) {
        ptx::mbar_arrive_expect_tx(&full[t % S], C::WBYTES + (base ? quads * 512 * SUBS : 0));
        if constexpr (KN) {  // rank j's row of 64 columns
          tma_load_3d(dst + C::BASE, &map_m, &full[t % S], col, 0, a);
        } else {             // column n's row of ranks
#pragma unroll
          for (int h = 0; h < RP; h += 64)
            tma_load_3d(dst + C::BASE + h / 64 * (kBC * 128), &map_m, &full[t % S], h, col, a);
        }
      }
      __syncwarp();
      if (base && sub < SUBS && quad < quads)
        gather4_once(dst + sub * (kRows * 128) + quad * 512, &map_base, &full[t % S], col + sub * (128 / sizeof(OT)), row,
                     policy);
    }
    if (ok && blocks <= S) load_h();
    // what is in flight lands before the block ends, whoever gave up
    int never = 0;
    for (int u = t > S ? t - S : 0; u < t; ++u) ptx::mbar_wait_warp(&full[u % S], (u / S) & 1, &never, kWaitLimitNs);
    if (warp == 0) ptx::mbar_wait_warp(&h_full, 0, &never, kWaitLimitNs);
  } else if (warp < kMmaWarp) {
    // ---- block by block: accumulator + base, out
    const int ew = warp - kLoaders / 32, quarter = ew & 3, half = ew >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    for (int t = 0; t < blocks; ++t) {
      const bool ok = ptx::mbar_wait_warp(&full[t % S], (t / S) & 1, abort_flag, kWaitLimitNs) &&
                      ptx::mbar_wait_warp(&acc_full[t & 1], (t >> 1) & 1, abort_flag, kWaitLimitNs);
      if (!ok) {
        give_up();
        break;
      }
      ptx::tc_fence_after();
      uint8_t* tile = smem + t % S * C::STAGE;
      const int m = quarter * 32 + lane;
      uint32_t r[32];
      __syncwarp();
      ptx::tmem_ld_32x32b_x32(tmem + lane_base + (t & 1) * kBC + half * 32, r);
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&acc_free[t & 1]);
      constexpr int HP = PIECES / 2;                // pieces of half a row
#pragma unroll
      for (int u = 0; u < 32; u += VEC) {
        const int c = half * HP + u / VEC;
        uint4* at = reinterpret_cast<uint4*>(tile + c / 8 * (kRows * 128) + swz(m, c % 8));
        uint4 x = make_uint4(0, 0, 0, 0);
        if (base) x = *at;
        if constexpr (sizeof(OT) == 4) {
          x.x = __float_as_uint(__uint_as_float(x.x) + __uint_as_float(r[u]));
          x.y = __float_as_uint(__uint_as_float(x.y) + __uint_as_float(r[u + 1]));
          x.z = __float_as_uint(__uint_as_float(x.z) + __uint_as_float(r[u + 2]));
          x.w = __float_as_uint(__uint_as_float(x.w) + __uint_as_float(r[u + 3]));
        } else {
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = pack2(__uint_as_float(w[q] << 16) + __uint_as_float(r[u + 2 * q]),
                         __uint_as_float(w[q] & 0xffff0000u) + __uint_as_float(r[u + 2 * q + 1]));
          x = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *at = x;
      }
      __syncwarp();
      const int col = col0 + t * kBC;
#pragma unroll
      for (int i = 0; i < HP; ++i) {                // the warp's 32 rows, HP lanes to a row
        const int q = quarter * 32 + i * (32 / HP) + lane / HP, c = half * HP + lane % HP;
        const int r2 = s_row[q];
        const uint4 x = *reinterpret_cast<const uint4*>(tile + c / 8 * (kRows * 128) + swz(q, c % 8));
        if (r2 >= 0 && col + c * VEC < col1)
          *reinterpret_cast<uint4*>(out + static_cast<size_t>(r2) * N + col + c * VEC) = x;
      }
      ptx::fence_proxy_async_smem();   // the tile was written to; the next one comes by TMA
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
          const uint64_t hd = RankTile<RP>::kdesc(h + q * RankTile<RP>::BYTES, k);
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
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 2 * kBC);
  }
  if (p.apart) {   // what follows this launch follows the one beside it, too
    pdl_wait();
    pdl_launch_dependents();
  }
}

// base [rows, N] in pieces of one row and 128 bytes
template <typename OT>
bool make_row_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t N) {
  if constexpr (sizeof(OT) == 2) return make_map(m, base, 2, rows, N, 1);
  const EncodeTiledFn enc = get_encode_fn();
  const cuuint64_t dims[2] = {N, rows}, strides[1] = {N * 4};
  const cuuint32_t box[2] = {32, 1}, estr[2] = {1, 1};
  if (!enc || enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
    record_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled rejected the base's layout");
    return false;
  }
  return true;
}

template <int RP, bool KN, typename OT>
int launch_expand_tile(const ExpandArgs& p, cudaStream_t s) {
  using C = ExpandCfg<RP, KN, OT>;
  static std::atomic<uint64_t> done{0};
  auto kernel = lora_expand_kernel<RP, KN, OT>;
  const int st = allow_smem(done, kernel, C::SMEM);
  if (st != MOE_OK) return st;
  CUtensorMap mb, mm;
  if (!(KN ? make_adapter_map(&mm, p.M, p.n, p.R, p.N, RP, 64) : make_adapter_map(&mm, p.M, p.n, p.N, p.R, kBC, 64)))
    return MOE_ERR_CUDA;
  mb = mm;
  if (p.base && !make_row_map<OT>(&mb, p.base, p.rows, p.N)) return MOE_ERR_CUDA;
  return launch_pdl("lora_expand_kernel", kernel, dim3(p.rows / kRows + p.n + 1, (p.N + p.cols - 1) / p.cols),
                    dim3(kExpandThreads), C::SMEM, s, p, mb, mm);
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
  // columns of a CTA: the narrowest slice (of 128 to 1024) with which two CTAs to an SM are all of them;
  // an adapter's last tile is half full on average
  const long long tiles = (static_cast<long long>(p.rows) + 64ll * p.n) / kRows + 1;
  p.cols = 1024;
  while (p.cols > 128 && tiles * ((p.N + p.cols / 2 - 1) / (p.cols / 2)) <= 2ll * num_sms()) p.cols /= 2;
  if (out_dtype == MOE_F32) return kn ? launch_expand_rank<true, float>(p, s) : launch_expand_rank<false, float>(p, s);
  return kn ? launch_expand_rank<true, __nv_bfloat16>(p, s) : launch_expand_rank<false, __nv_bfloat16>(p, s);
}

}  // namespace moe
