// Gradients of the low-rank adapters, out = base + s_a (x A_a^T) B_a^T, given
// dC = d out and the forward's h = x A^T:
//   dh[r] = s_a dC[r] B_a          dB_a = s_a sum_r dC[r]^T h[r]
//   dx[r] = dx_base[r] + dh[r] A_a  dA_a = sum_r dh[r]^T x[r]
// over the rows r of adapter a.  One streaming pass over dC gives dh and dB, one
// over x gives dA, and the forward's second product, with A in the place of B,
// gives dx.  Each wide operand is read once; what several CTAs add to is
// written as partial sums and added here in a fixed order, so results do not
// vary from run to run.  Adapters of few rows take one launch instead
// (lora_few.cu).
#include "common.cuh"
#include "lora.cuh"
#include "lora_tc.cuh"

namespace moe {
namespace {

// The images of a tile's 128 rows, blockIdx.y's share of them: of s h, whose rows
// are the plan's (SLICES false), or of dh, the sum of its slices by position.
// Rows behind an adapter's last are 0: a gradient sums over all 128.
struct TermsArgs {
  const float* h;
  int slices;
  const float* scale;
  const int32_t* offsets;
  const int32_t* order;
  int n, rows, R;
  uint8_t* image;
};
// A piece of 8 ranks is a thread's, or, of many slices, kGroups threads' (the
// lanes 8 apart), each with every kGroups-th slice; they meet by shuffles.
constexpr int kTermsThreads = 256, kGroups = 4;

template <int RP, bool SLICES>
__global__ void __launch_bounds__(kTermsThreads) lora_terms_kernel(const TermsArgs p) {
  constexpr int G = SLICES ? kGroups : 1, PIECES = RP / 8, ROWS = kTermsThreads / G / PIECES;   // rows of a block
  pdl_wait();
  pdl_launch_dependents();
  int a, start, end;
  if (!find_tile(p.offsets, p.n, p.rows, 128, blockIdx.x, a, start, end) || a == p.n) return;
  const int g = SLICES ? threadIdx.x / 8 % G : 0, i = SLICES ? threadIdx.x / 32 * 8 + threadIdx.x % 8 : threadIdx.x;
  const int c = i % PIECES, m = blockIdx.y * ROWS + i / PIECES, at = start + m;
  if (m >= 128) return;   // whole warps: 128 rows fill the last block or half of one
  float v[8] = {};
  if (at < end && c * 8 < p.R) {
    if constexpr (SLICES) {
      const size_t all = static_cast<size_t>(p.rows) * p.R;
      const float* from = p.h + static_cast<size_t>(at) * p.R + c * 8;
#pragma unroll 8
      for (int s = g; s < p.slices; s += G) {
        float u[8];
        load8(from + s * all, u);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += u[q];
      }
    } else {
      const int r = __ldg(p.order + at);
      const float sc = p.scale ? __ldg(p.scale + a) : 1.f;
      if (r >= 0 && r < p.rows) load8(p.h + static_cast<size_t>(r) * p.R + c * 8, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= sc;
    }
  }
  if constexpr (SLICES) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] += __shfl_xor_sync(0xffffffffu, v[q], 8);
      v[q] += __shfl_xor_sync(0xffffffffu, v[q], 16);
    }
    if (g) return;
  }
  store_terms<RP>(p.image + static_cast<size_t>(blockIdx.x) * RankTile<RP>::IMAGE, m, c, v);
}

template <int RP, bool SLICES>
int launch_terms_rank(const TermsArgs& p, cudaStream_t s) {
  constexpr int rows = kTermsThreads / (SLICES ? kGroups : 1) / (RP / 8);
  return launch_pdl("lora_terms_kernel", lora_terms_kernel<RP, SLICES>, dim3(p.rows / 128 + p.n, (128 + rows - 1) / rows),
                    dim3(kTermsThreads), 0, s, p);
}
template <bool SLICES>
int launch_terms(const TermsArgs& p, cudaStream_t s) {
  if (p.R <= 16) return launch_terms_rank<16, SLICES>(p, s);
  if (p.R <= 32) return launch_terms_rank<32, SLICES>(p, s);
  if (p.R <= 64) return launch_terms_rank<64, SLICES>(p, s);
  return launch_terms_rank<128, SLICES>(p, s);
}

struct GradReduceArgs {
  const float* part[2];   // of dA, dB: partial sums by part_slot
  void* grad[2];          // nullptr: not wanted
  size_t size[2];         // values of one adapter
  int chunk[2];
  const int32_t* offsets;
  int n, rows;
};

// Gradient blockIdx.y (0 dA, 1 dB) of the adapters of more than one chunk: the
// sum over the chunks.  That of a single one, or of none, is there already.
// How many adapters have several and which is on the device, so every block
// lists them and the blocks share their values out evenly: with a fixed share of
// the blocks to an adapter, the sums of 4096 rows of one of 1024 adapters were
// a single block's work (a call of rank 64 and 2048 and 2048 columns 7450 us,
// 382 now, most of it the others' zeros; 8191 rows of 16 adapters 138 -> 129).
constexpr int kReduceThreads = 256, kReducePiece = kReduceThreads * 4;

template <typename GT>
__global__ void __launch_bounds__(kReduceThreads) grad_reduce_kernel(const GradReduceArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int s_adapter[kMaxAdapters];
  __shared__ int s_found[kReduceThreads / 32];
  const int z = blockIdx.y, chunk = p.chunk[z], tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!p.grad[z]) return;
  auto chunks_of = [&](int a, int& first) {
    first = held_offset(p.offsets, p.n, p.rows, a);
    const int last = held_offset(p.offsets, p.n, p.rows, a + 1);
    return last > first ? (last - first + chunk - 1) / chunk : 0;
  };
  int found = 0, first;
  for (int a0 = 0; a0 < p.n; a0 += kReduceThreads) {   // in ascending order, the same in every block
    const bool several = a0 + tid < p.n && chunks_of(a0 + tid, first) > 1;
    const unsigned in = __ballot_sync(0xffffffffu, several);
    if (lane == 0) s_found[warp] = __popc(in);
    __syncthreads();
    int at = found;
#pragma unroll
    for (int w = 0; w < kReduceThreads / 32; ++w) {
      at += w < warp ? s_found[w] : 0;
      found += s_found[w];
    }
    if (several) s_adapter[at + __popc(in & ((1u << lane) - 1))] = a0 + tid;
    __syncthreads();
  }
  const size_t size = p.size[z];
  const int pieces = static_cast<int>((size + kReducePiece - 1) / kReducePiece);
  const long long all = static_cast<long long>(found) * pieces;
  for (long long it = blockIdx.x; it < all; it += gridDim.x) {
    const int a = s_adapter[it / pieces];
    const size_t i = static_cast<size_t>(it % pieces) * kReducePiece + tid * 4;
    if (i >= size) continue;
    const int chunks = chunks_of(a, first);
    const float* part = p.part[z] + part_slot(first, chunk) * size + i;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < chunks; ++s) {
      const float4 u = __ldcs(reinterpret_cast<const float4*>(part + s * size));
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    GT* grad = static_cast<GT*>(p.grad[z]) + a * size + i;
    if constexpr (sizeof(GT) == 4)
      *reinterpret_cast<float4*>(grad) = v;
    else
      *reinterpret_cast<uint2*>(grad) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
  }
}

// Rows and columns of a CTA of a pass over [rows, W], from an estimate of its
// time: a CTA's tiles at its share of the memory's rate, its start (3 us to the
// first product) and its gradient's way out, over as many as an SM holds; the
// partial sums, which several chunks of an adapter (dA, dB) and several slices
// of a row (dh) write and read again; the launch that adds them.  How the rows
// are spread over the adapters is on the device: some are taken to have twice
// their even share, the longest CTA to run on for half its time.
// A chunk's sum runs in the tensor cores' accumulator, which cuts off what it
// cannot hold: past 1024 rows that would stand out beside a matrix product's in
// fp32 (1.9e-6 of dB with chunks of 2048 rows, 1.0e-6 with 1024; 0.5e-6 there).
// Above rank 64 the three terms take turns in one accumulator, three times the
// steps: 3.4e-6 of dB and 3.6e-6 of dA with 1024 rows.  512 halve that, but write
// twice the partial sums (rank 128, 8191 rows of 16 adapters 190 -> 237 us, of
// one 4096 x 7168 92 -> 103), 256 leave 1.0e-6 (301, 128 us): 1024 stay.
constexpr int kMaxChunk = 1024;
struct Split {
  int chunk, cols;
};
Split split_for(int rows, int n, int W, int R, bool proj) {
  const int max_cols = lora_stream_max_cols(R, proj), per_sm = R <= 32 ? 2 : 1, sms = num_sms();
  const double rate = 6400.0, mean = static_cast<double>(rows) / (n < rows ? n : rows > 0 ? rows : 1);
  Split best{128, 128};
  double best_ns = 1e30;
  for (int cols = 128; cols <= max_cols; cols *= 2)
    for (int chunk = 128; chunk <= kMaxChunk; chunk *= 2) {
      const int slices = (W + cols - 1) / cols;
      const bool whole = chunk >= (n > 1 ? 2 : 1) * mean;
      const double chunks = whole ? rows / mean : rows / mean * 0.5 + static_cast<double>(rows) / chunk;
      const double ctas = chunks * slices, load = ctas / (sms * per_sm);
      const double tile = 128.0 * 128 * 2 * sms / rate * (ctas > sms ? per_sm : 1);
      const double longest = mean * (n > 1 ? 2 : 1) < chunk ? mean * (n > 1 ? 2 : 1) : chunk;
      const double fixed = 3000 + cols * R * 4 * sms / rate;
      const double ns = load * fixed + (load < 1 ? 1 - load : 0.5) * (fixed + (longest + 127) / 128 * (cols / 128) * tile) +
                        static_cast<double>(rows) / 128 * slices * (cols / 128) * tile / (sms * per_sm) +
                        ((whole ? 0.0 : 8.0 * chunks * W * R) + (proj ? 8.0 * rows * R * slices : 0.0)) / rate +
                        (rows > chunk ? 3000 : 0);
      if (ns < best_ns) best_ns = ns, best = {chunk, cols};
    }
  return best;
}

// Whether one launch on tiles of few rows does it all (lora_few.cu), by the mean
// of rows to an adapter.  A tile of more than four rows costs that launch four
// times the multiply-adds of one with up to four, so what a mean may be depends
// on how much of the time those take (the rank) and on whether such a tile finds
// others beside it (the adapters).  Measured, that launch against the streaming
// passes, us; "spread": the rows lie at random over the adapters, else evenly;
// columns 2048 and 2048, at ranks 16 and 32 with up to 32 adapters 4096 and 4096:
//   rank 16, mean 1 / 2 / 4: of 2 adapters 9/16 9/16 10/16 (spread 15/16), of 8 9/26 9/22 17/22 (19/22), of 32 16/39
//            16/39 17/40 (25/40), of 100 40/91 41/92 44/92 (84/91)
//   rank 32, mean 2 / 4: of 4 14/20 14/18 (23/18), of 8 14/24 18/24 (27/24), of 32 24/51 25/52 (39/52),
//            of 100 38/70 39/70 (70/70)
//   rank 64, spread, mean 1 / 2 / 3 / 4: of 4 20/17 20/17 30/18 30/18, of 8 20/23 20/23 32/24 35/22, of 16 24/30 33/28
//            37/29 42/29, of 24 27/38 29/44 42/45 44/45, of 32 28/48 38/51 44/52 47/53, of 100 85/106 92/123 102/130
//            113/132, of 200 159/193 176/230 207/244 214/248
//   rank 128, spread, mean 1 / 2: of 4 28/21 28/22, of 8 29/27 29/28, of 16 34/38 53/38, of 32 42/67 60/72, of 48 70/82
//            110/98, of 64 74/107 112/129, of 100 205/150 206/173 (evenly 131/189 132/189), of 200 215/276 332/327
bool few_rows(int rows, int n, int R) {
  if (R <= 32) return rows <= 4ll * n;
  if (R <= 64) return n >= 8 && rows <= (n >= 24 ? 4ll : 2ll) * n;
  return n >= 8 && rows <= n;
}

struct BackwardLayout {
  bool few;
  Split dc, x;
  size_t dh_part, image, pA, pB, total;
};
BackwardLayout backward_layout(int rows, int n, int d, int N, int R) {
  BackwardLayout L{};
  size_t off = 256;   // the status word
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  L.few = few_rows(rows, n, R);
  if (L.few) {
    L.dc = L.x = Split{kRowsFew, 0};
    L.pA = take(part_slot(rows, kRowsFew) * R * d * 4);
    L.pB = take(part_slot(rows, kRowsFew) * R * N * 4);
    L.total = off;
    return L;
  }
  L.dc = split_for(rows, n, N, R, true);
  L.x = split_for(rows, n, d, R, false);
  const size_t slices = (N + L.dc.cols - 1) / L.dc.cols;
  L.dh_part = take(slices * rows * R * 4);
  L.image = take(image_bytes(rows, n, R));   // of h, then of dh
  L.pA = take(part_slot(rows, L.x.chunk) * R * d * 4);
  L.pB = take(part_slot(rows, L.dc.chunk) * R * N * 4);
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
  uint8_t* image = reinterpret_cast<uint8_t*>(ws + L.image);
  const size_t sizeA = static_cast<size_t>(q.R) * q.d, sizeB = static_cast<size_t>(q.R) * q.N;
  if (q.rows == 0) {
    MOE_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(int), s));   // MOE_OK
    const size_t bytes = q.grad_dtype == MOE_F32 ? 4 : 2;
    if (q.dA) MOE_CUDA_CHECK(cudaMemsetAsync(q.dA, 0, q.n * sizeA * bytes, s));
    if (q.dB) MOE_CUDA_CHECK(cudaMemsetAsync(q.dB, 0, q.n * sizeB * bytes, s));
    return MOE_OK;
  }
  int st = MOE_OK;
  if (L.few) {
    st = launch_lora_few(q, reinterpret_cast<float*>(ws + L.pA), reinterpret_cast<float*>(ws + L.pB), s);
    if (st != MOE_OK) return st;
  } else {
    const bool need_dh = q.dx || q.dA;
    TermsArgs t{};
    t.scale = q.scale, t.offsets = q.offsets, t.order = q.order, t.n = q.n, t.rows = q.rows, t.R = q.R, t.image = image;
    if (q.dB) {
      t.h = q.h;
      st = launch_terms<false>(t, s);
      if (st != MOE_OK) return st;
    }
    StreamArgs p{};
    p.X = static_cast<const __nv_bfloat16*>(q.dC), p.M = static_cast<const __nv_bfloat16*>(q.B), p.V = image;
    p.scale = q.scale, p.offsets = q.offsets, p.order = q.order, p.n = q.n, p.rows = q.rows, p.W = q.N, p.R = q.R;
    p.chunk = L.dc.chunk, p.cols = L.dc.cols, p.early = q.dB != nullptr;
    p.proj = need_dh ? dh_part : nullptr;
    p.part = reinterpret_cast<float*>(ws + L.pB), p.grad = q.dB, p.grad_f32 = q.grad_dtype == MOE_F32;
    p.status = reinterpret_cast<int*>(ws), p.first = true;
    st = launch_lora_stream(p, kStreamBoth, s);
    if (st != MOE_OK) return st;
    if (need_dh) {
      t.h = dh_part, t.slices = (q.N + L.dc.cols - 1) / L.dc.cols;
      st = launch_terms<true>(t, s);
      if (st != MOE_OK) return st;
    }
    if (q.dA) {
      p.X = static_cast<const __nv_bfloat16*>(q.x), p.M = nullptr, p.W = q.d;
      p.chunk = L.x.chunk, p.cols = L.x.cols, p.early = true, p.first = false, p.proj = nullptr;
      p.part = reinterpret_cast<float*>(ws + L.pA), p.grad = q.dA;
      st = launch_lora_stream(p, kStreamGrad, s);
      if (st != MOE_OK) return st;
    }
    if (q.dx) {
      ExpandArgs e{};
      e.h = image, e.M = static_cast<const __nv_bfloat16*>(q.A), e.offsets = q.offsets, e.order = q.order;
      e.n = q.n, e.rows = q.rows, e.N = q.d, e.R = q.R, e.base = q.dx_base, e.out = q.dx;
      e.status = reinterpret_cast<int*>(ws), e.apart = q.dA != nullptr;
      st = launch_lora_expand(e, true, q.dx_dtype, s);
      if (st != MOE_OK) return st;
    }
  }
  // an adapter of several chunks has to have more rows than one holds
  const bool manyA = q.dA && q.rows > L.x.chunk, manyB = q.dB && q.rows > L.dc.chunk;
  if (!manyA && !manyB) return MOE_OK;
  GradReduceArgs r{};
  r.part[0] = reinterpret_cast<float*>(ws + L.pA), r.part[1] = reinterpret_cast<float*>(ws + L.pB);
  r.grad[0] = manyA ? q.dA : nullptr, r.grad[1] = manyB ? q.dB : nullptr;
  r.size[0] = sizeA, r.size[1] = sizeB;
  r.chunk[0] = L.x.chunk, r.chunk[1] = L.dc.chunk;
  r.offsets = q.offsets, r.n = q.n, r.rows = q.rows;
  // four blocks to an SM, no more than there can be pieces
  size_t most = 1;
  for (int z = 0; z < 2; ++z) {
    const size_t several = static_cast<size_t>(q.rows) / (r.chunk[z] + 1), held = q.n;
    const size_t pieces = (several < held ? several : held) * ((r.size[z] + kReducePiece - 1) / kReducePiece);
    if (r.grad[z] && pieces > most) most = pieces;
  }
  const size_t share = 4ul * num_sms();
  const dim3 grid(static_cast<unsigned>(most < share ? most : share), 2);
  return launch_pdl("grad_reduce_kernel", q.grad_dtype == MOE_F32 ? grad_reduce_kernel<float> : grad_reduce_kernel<__nv_bfloat16>,
                    grid, dim3(kReduceThreads), 0, s, r);
}

}  // namespace moe
