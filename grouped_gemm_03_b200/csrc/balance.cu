// Training the router: the balance loss over sequences with its per-expert
// counts, and the gradient of the router's logits (gates and balance loss in
// one pass over them).
//
// Loss ("MegaMoE ..." §2: alpha * E * sum_i f_i P_i, here per sequence): with
// p = softmax(logits), c[s,e] the (token, slot) pairs of sequence s that chose
// expert e, Q[s,e] the sum of p over its N_s tokens, and S' the sequences that
// have tokens,
//   loss = sum_s coef_s sum_e c[s,e] Q[s,e],   coef_s = alpha E / (k N_s^2 S'),
// which is the mean over sequences of alpha E sum_e f_e P_e with
// f = c / (k N) and P = Q / N.
//
// Gradient: both the raw gates (w_j = p at topk_idx_j) and the loss are linear
// in p, so with G_e = sum_{j: idx_j = e} dw_j + dloss coef_s c[s,e]
//   dlogit_e = p_e (G_e - sum_i G_i p_i).
// Renormalised gates are a softmax over the selected experts alone:
//   w_j = p_j / sum_S p,   dlogit_{idx_j} += w_j (dw_j - sum_S w dw).
//
// One pass over the logits, each row held in registers by L lanes of 16 columns
// (32 past 512 experts), the softmax's maximum and sum by shuffles, the next row
// in flight.  The bytes alone would take 2.8 us (loss, 65536 tokens of 128
// experts, fp16) and 5.5 (gradient, bf16); measured 18.5 and 14.5.  While an SM
// is at work its issue slots are busy 52 % of the time in the loss's first pass
// and 60 % in the gradient: a block has about 150 tokens, five rows to a lane
// group, so what it does once (its sequence's search, the first loads, the
// columns' sums through shared memory and their barriers) weighs as much as its
// rows.  The loss's second launch is a chain of dependent loads and the last
// block's sums.  A batch of 128 tokens takes one launch of 7 us, the gradient of
// 4096 tokens of 256 experts 5.5.
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 256;
constexpr int kBalMinChunk = 32;     // tokens of one block, at least
constexpr int kBalSmall = 512;       // tokens up to which one cluster does both passes
constexpr int kFinCluster = 8;       // CTAs of a small batch's second pass, each a slice of the experts

// A row of E values over L lanes, V values a lane in pieces of C (16 bytes):
// lane l holds columns (q * L + l) * C + c as value q * C + c.
template <typename T>
constexpr int piece() { return 16 / sizeof(T); }
template <typename T>
__device__ __forceinline__ int column(int i, int L, int l) {
  return (i / piece<T>() * L + l) * piece<T>() + i % piece<T>();
}

__device__ __forceinline__ void unpack(const uint4& r, float (&f)[4], float) {
  f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, float (&f)[8], __half) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = v.x, f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void unpack(const uint4& r, float (&f)[8], __nv_bfloat16) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ float from_f32(float v, float) { return v; }
__device__ __forceinline__ __half from_f32(float v, __half) { return __float2half_rn(v); }
__device__ __forceinline__ __nv_bfloat16 from_f32(float v, __nv_bfloat16) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ uint32_t minus_inf_bits(float) { return 0xff800000u; }
__device__ __forceinline__ uint32_t minus_inf_bits(__half) { return 0xfc00fc00u; }
__device__ __forceinline__ uint32_t minus_inf_bits(__nv_bfloat16) { return 0xff80ff80u; }

// A lane's share of a row as it lies in memory, so that the next rows' loads
// can be in flight while this one is worked on.  vec: every row starts on 16
// bytes and E fills whole pieces.
template <typename T, int V>
struct Row {
  static constexpr int C = piece<T>(), Q = V / C;
  uint4 raw[Q];
  // -inf past the row's end; vec = 2: the lanes' pieces are the row
  __device__ __forceinline__ void load(const T* row, int E, int L, int l, int vec) {
    row += l * C;
    const int left = E - l * C, step = L * C;
    if (vec == 2) {
#pragma unroll
      for (int q = 0; q < Q; ++q) raw[q] = *reinterpret_cast<const uint4*>(row + q * step);
      return;
    }
    clear();
    if (vec) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (q * step < left) raw[q] = *reinterpret_cast<const uint4*>(row + q * step);
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        alignas(16) T v[C];
        *reinterpret_cast<uint4*>(v) = raw[q];
#pragma unroll
        for (int u = 0; u < C; ++u)
          if (q * step + u < left) v[u] = row[q * step + u];
        raw[q] = *reinterpret_cast<const uint4*>(v);
      }
    }
  }
  __device__ __forceinline__ void clear() {
    const uint32_t none = minus_inf_bits(T());
#pragma unroll
    for (int q = 0; q < Q; ++q) raw[q] = make_uint4(none, none, none, none);
  }
  // the largest value (a NaN is passed over): of 16-bit types two at a time
  __device__ __forceinline__ float largest() const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
    if constexpr (sizeof(T) == 4) {
      float m = __uint_as_float(w[0]);
#pragma unroll
      for (int i = 1; i < 4 * Q; ++i) m = fmaxf(m, __uint_as_float(w[i]));
      return m;
    } else {
      using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
      T2 m = *reinterpret_cast<const T2*>(&w[0]);
#pragma unroll
      for (int i = 1; i < 4 * Q; ++i) m = __hmax2(m, *reinterpret_cast<const T2*>(&w[i]));
      return fmaxf(to_f32(m.x), to_f32(m.y));
    }
  }
  __device__ __forceinline__ void values(float (&v)[V]) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float f[C];
      unpack(raw[q], f, T());
#pragma unroll
      for (int u = 0; u < C; ++u) v[q * C + u] = f[u];
    }
  }
};

// N consecutive values from a lane's registers to memory
template <typename OT, int N>
__device__ __forceinline__ void store_run(OT* p, const float* v) {
#pragma unroll
  for (int b = 0; b < N; b += 16 / static_cast<int>(sizeof(OT))) {
    constexpr int W = N < 16 / static_cast<int>(sizeof(OT)) ? N : 16 / static_cast<int>(sizeof(OT));
    alignas(16) OT o[W];
#pragma unroll
    for (int u = 0; u < W; ++u) o[u] = from_f32(v[b + u], OT());
    if constexpr (W * sizeof(OT) == 16)
      *reinterpret_cast<uint4*>(p + b) = *reinterpret_cast<const uint4*>(o);
    else
      *reinterpret_cast<uint2*>(p + b) = *reinterpret_cast<const uint2*>(o);
  }
}

__device__ __forceinline__ float group_max(float v, int L) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (o < L) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float group_sum(float v, int L) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (o < L) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 2^x by the hardware, what would be denormal as 0: with the compiler's own
// scaling around it the exponentials were a third of the first pass's work.
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504f;
// e^(v - m), m a row's maximum.  One multiply-add v log2 e - m log2 e serves a
// row whose maximum is within kPlain: the rounding of m log2 e, at most 2^-4
// there (half a step below 2^21), is common to the row and falls out of its
// softmax.  Past it that rounding grows with m (440 at 1e10, more than an
// exponent holds), and v - m comes first: exact next to m, and far from it the
// numerator is 0 either way.
constexpr float kPlain = 1048576.f;
__device__ __forceinline__ float exp_from(float v, float m) {
  return fabsf(m) < kPlain ? exp2_of(fmaf(v, kLog2e, -m * kLog2e)) : exp2_of((v - m) * kLog2e);
}

// The numerators e^(v - m) of a row's softmax, with the row's maximum m and
// 1 / (their sum).  A logit of -inf has probability 0; a row of nothing else (a
// row that is not live is one) has probability 0 throughout: inv = 0.  The
// maximum passes over a NaN, the sum does not, so a NaN logit makes its row NaN.
template <typename T, int V>
__device__ __forceinline__ void softmax_row(const Row<T, V>& row, float (&v)[V], int L, float& m, float& inv) {
  m = group_max(row.largest(), L);
  row.values(v);
  if (m == -INFINITY) m = 0.f;
  if (__all_sync(0xffffffffu, fabsf(m) < kPlain)) {
    const float m2 = -m * kLog2e;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = exp2_of(fmaf(v[i], kLog2e, m2));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = exp_from(v[i], m);
  }
  float z[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < V; ++i) z[i & 1] += v[i];
  const float all = group_sum(z[0] + z[1], L);
  inv = all == 0.f ? 0.f : __fdividef(1.f, all);
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// First token at or after `t` belongs to the sequence this returns: the number
// of sequences that end at or before t (all threads of the block take part).
__device__ int sequence_at(const int32_t* off, int S, int t) {
  int n = 0;
  for (int s0 = 0; s0 < S; s0 += blockDim.x) {
    const int s = s0 + threadIdx.x;
    n += __syncthreads_count(s < S && off[s + 1] <= t);
  }
  return n;
}

struct BalanceArgs {
  const void* logits;
  const int32_t* idx;
  int T, E, k;
  const int32_t* off;   // [S + 1] or nullptr: one sequence of all T tokens
  int S;
  const uint8_t* mask;  // [T] or nullptr
  float alpha;
  int chunk, chunks, L, vec;
  // partial sums by slot = chunk index + sequence index: along the tokens at
  // least one of the two grows from a segment to the next, so slots differ
  float* part_q;        // [chunks + S][E]
  int32_t* part_c;      // [chunks + S][E]
  int32_t* part_n;      // [chunks + S]
  int32_t* part_err;    // [chunks]
  float* share;         // of the loss, [S][groups of kFinCols experts]
  int32_t* tokens;      // [S]
  int* done;            // blocks of the second pass that have finished
  float* loss;
  int32_t* counts;
  float* prob;
  float* coef;
  int* status;
};

// First pass: block b sums the probabilities and counts of its chunk of
// tokens, for each sequence in it.
template <typename T, int V>
__device__ void balance_partial(const BalanceArgs& a, float* s_mem) {
  const int E = a.E, L = a.L;
  const int width = L * V;                                    // padded columns
  float* s_q = s_mem;                                          // [groups][width]
  int* s_c = reinterpret_cast<int*>(s_mem + kBalThreads * V);   // [E]
  __shared__ int s_err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && tid == 0) *a.done = 0;
  const int l = lane % L, group = tid / L, groups = kBalThreads / L;
  const T* logits = static_cast<const T*>(a.logits);
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  // The first rows and, of short chunks with few slots, every token's ids and mask are on their way while the
  // block finds its sequence.
  int off0 = 0, off1 = 0;
  if (a.off && tid < a.S) off0 = a.off[tid], off1 = a.off[tid + 1];
  Row<T, V> row[2];
  bool row_kept[2];
  auto fetch = [&](int u, int r, int end) {   // a row past the end, or masked, is loaded and not used
    const int at = r < end ? r : t0;
    row[u].load(logits + static_cast<size_t>(at) * E, E, L, l, a.vec);
    row_kept[u] = r < end && (!a.mask || a.mask[at]);
  };
  fetch(0, t0 + group, t1);
  constexpr int kAhead = 8;
  const bool ahead = a.k <= kAhead && a.chunk <= kBalThreads;
  int ids[kAhead];
  bool kept = ahead && t0 + tid < t1;
  if (kept) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ids[j] = j < a.k ? a.idx[static_cast<size_t>(t0 + tid) * a.k + j] : -1;
    if (a.mask) kept = a.mask[t0 + tid];
  }
  if (tid == 0) s_err = 0;
  for (int e = tid; e < E; e += kBalThreads) s_c[e] = 0;
  int s = 0;   // the sequence of token t0: as many as end at or before it
  if (a.off) {
    bool bad = tid == 0 && off0 != 0;
    for (int i0 = 0; i0 < a.S; i0 += kBalThreads) {
      const int i = i0 + tid;
      if (i0) off0 = i < a.S ? a.off[i] : 0, off1 = i < a.S ? a.off[i + 1] : 0;
      bad |= i < a.S && (off0 > off1 || off1 > a.T);
      s += __syncthreads_count(i < a.S && off1 <= t0);
    }
    if (bad) atomicOr(&s_err, 2);
  }
  __syncthreads();
  auto count = [&](int e) {
    if (e >= 0 && e < E)
      atomicAdd(&s_c[e], 1);   // whole numbers: the order does not show
    else if (e != -1)
      atomicOr(&s_err, 1);
  };
  int t = t0;
  while (t < t1 && s < a.S) {
    const int end = a.off ? min(t1, a.off[s + 1]) : t1;
    if (end <= t) {
      ++s;
      continue;
    }
    const size_t slot = blockIdx.x + static_cast<size_t>(s);
    int n = 0;
    if (ahead) {
      if (kept && t0 + tid >= t && t0 + tid < end) {
        n = 1;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (j < a.k) count(ids[j]);
      }
    } else {
      for (int r = t + tid; r < end; r += kBalThreads) {
        if (a.mask && !a.mask[r]) continue;
        ++n;
        for (int j = 0; j < a.k; ++j) count(a.idx[static_cast<size_t>(r) * a.k + j]);
      }
    }
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    // a warp's lanes run the same number of rounds: rows past the end do not count
    if (t > t0) fetch(0, t + group, end);
    auto add = [&](int u, int r) {
      if (!(row_kept[u] && r < end)) row[u].clear();   // whatever a token that does not count holds
      float v[V], m, inv;
      softmax_row(row[u], v, L, m, inv);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
    };
    for (int b = t; b < end; b += 2 * groups) {   // one of the two rows in flight while the other is worked on
      if (b + groups < end) fetch(1, b + groups + group, end);
      add(0, b + group);
      if (b + groups >= end) break;
      if (b + 2 * groups < end) fetch(0, b + 2 * groups + group, end);
      add(1, b + groups + group);
    }
    // the lanes' sums meet in a fixed order: `parts` threads to a column, each some of the groups, then those
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(s_q + group * width + column<T>(i, L, l)) =
          make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    __shared__ int s_n[kBalThreads / 32];
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    const int parts = kBalThreads / width, mine = parts > 1 ? groups / parts : groups;
    if (parts > 1) {
      const int e = tid % width, first = tid / width * mine;
      float q = 0.f;
#pragma unroll 8
      for (int g = first; g < first + mine; ++g) q += s_q[g * width + e];
      __syncthreads();
      s_q[tid] = q;   // part tid / width of column e
      __syncthreads();
    }
    for (int e = tid; e < E; e += kBalThreads) {
      float q = 0.f;
#pragma unroll 8
      for (int w = 0; w < (parts > 1 ? parts : groups); ++w) q += s_q[w * width + e];
      a.part_q[slot * E + e] = q;
      a.part_c[slot * E + e] = s_c[e];
      s_c[e] = 0;
    }
    if (tid == 0) {
      int all = 0;
      for (int w = 0; w < kBalThreads / 32; ++w) all += s_n[w];
      a.part_n[slot] = all;
    }
    __syncthreads();
    t = end;
  }
  if (tid == 0) a.part_err[blockIdx.x] = s_err;
}

// Second pass of a small batch, within the cluster: CTA r reduces its slice of
// the experts over the slots of every sequence, `w` threads to a column and `g`
// sequences at once; the CTAs' shares of the loss meet in rank order.
__device__ void balance_finish(const BalanceArgs& a, int cols, int w) {
  constexpr int NT = kBalThreads;
  __shared__ float s_warp[NT / 32];
  __shared__ float s_loss[kFinCluster];
  const int tid = threadIdx.x;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int E = a.E;
  auto slots = [&](int s, int& first, int& last) {  // [first, last) of sequence s
    const int b = a.off ? max(0, min(a.T, a.off[s])) : 0, e = a.off ? max(0, min(a.T, a.off[s + 1])) : a.T;
    first = e > b ? b / a.chunk + s : 0;
    last = e > b ? (e - 1) / a.chunk + s + 1 : 0;
  };
  // the w lanes of a (sequence, column) are neighbours: their sums meet by shuffles
  const int g = NT / (cols * w);                            // sequences at once
  const int j = tid % w, col = tid / w % cols, sg = tid / (cols * w);
  const int e = rank * cols + col;
  float share = 0.f;
  int live = 0;                                             // sequences that have tokens
  for (int s0 = 0; s0 < a.S; s0 += g) {
    const int s = s0 + sg;
    float q = 0.f;
    int c = 0, n = 0;
    if (s < a.S && sg < g) {
      int f, l;
      slots(s, f, l);
#pragma unroll 8
      for (int i = f + j; i < l; i += w) {
        if (e < E) {
          q += a.part_q[static_cast<size_t>(i) * E + e];
          c += a.part_c[static_cast<size_t>(i) * E + e];
        }
        n += a.part_n[i];
      }
    }
    for (int o = w >> 1; o; o >>= 1) {
      q += __shfl_xor_sync(0xffffffffu, q, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    live += __syncthreads_count(j == 0 && col == 0 && n > 0);
    if (j == 0 && s < a.S && sg < g && e < E) {
      const float nf = static_cast<float>(n);
      a.counts[static_cast<size_t>(s) * E + e] = c;
      if (a.prob) a.prob[static_cast<size_t>(s) * E + e] = n > 0 ? __fdiv_rn(q, nf) : 0.f;
      if (n > 0) share += static_cast<float>(c) * q * __fdiv_rn(a.alpha * E, a.k * nf * nf);
    }
  }
  if (rank == 0) {
    for (int s = tid; s < a.S; s += NT) {
      int f, l, n = 0;
      slots(s, f, l);
      for (; f < l; ++f) n += a.part_n[f];
      const float nf = static_cast<float>(n);
      a.coef[s] = n > 0 ? __fdiv_rn(a.alpha * E, a.k * nf * nf * static_cast<float>(live)) : 0.f;
    }
  }
  // the block's share of the loss, in a fixed order
#pragma unroll
  for (int o = 16; o; o >>= 1) share += __shfl_xor_sync(0xffffffffu, share, o);
  if ((tid & 31) == 0) s_warp[tid >> 5] = share;
  __syncthreads();
  if (tid == 0) {
    float all = 0.f;
    for (int i = 0; i < NT / 32; ++i) all += s_warp[i];
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&s_loss[rank])), there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(at));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(all) : "memory");
  }
  cluster_barrier();
  if (rank == 0) {
    int err = 0;
    for (int i = tid; i < a.chunks; i += NT) err |= a.part_err[i];
    if (a.T == 0 && a.off)   // no first pass to look at the offsets: all of them are 0
      for (int i = tid; i <= a.S; i += NT) err |= a.off[i] != 0 ? 2 : 0;
    const int bad = __syncthreads_or(err & 2), odd = __syncthreads_or(err & 1);
    if (tid == 0) {
      float all = 0.f;
      for (int r = 0; r < kFinCluster; ++r) all += s_loss[r];
      *a.loss = live > 0 ? __fdiv_rn(all, static_cast<float>(live)) : 0.f;
      *a.status = bad ? MOE_ERR_BAD_OFFSETS : odd ? MOE_ERR_INVALID : MOE_OK;
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kBalThreads, V <= 16 ? 3 : 2) balance_partial_kernel(const BalanceArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ float s_mem[];
  balance_partial<T, V>(a, s_mem);
}

// Second pass of a large one: a task is a sequence's 8 columns, a block's (BLOCK)
// or a warp's; lane l adds column l % 8 over every fourth slot of its warp's.
// The block that finishes last counts the sequences that have tokens and adds
// the tasks' shares of the loss, in a fixed order whichever block it is.
constexpr int kFinCols = 8;

template <bool BLOCK>
__global__ void __launch_bounds__(kBalThreads) balance_finish_kernel(const BalanceArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int WARPS = kBalThreads / 32;
  __shared__ float s_q[WARPS][kFinCols];
  __shared__ int s_c[WARPS][kFinCols], s_n[WARPS];
  __shared__ float s_sum[WARPS];
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.E;
  const int slabs = (E + kFinCols - 1) / kFinCols;
  const long long tasks = static_cast<long long>(a.S) * slabs, step = BLOCK ? gridDim.x : gridDim.x * WARPS;
  for (long long i = BLOCK ? blockIdx.x : blockIdx.x * WARPS + warp; i < tasks; i += step) {
    const int s = static_cast<int>(i / slabs), slab = static_cast<int>(i % slabs), e = slab * kFinCols + lane % 8;
    const int t0 = a.off ? max(0, min(a.T, a.off[s])) : 0, t1 = a.off ? max(0, min(a.T, a.off[s + 1])) : a.T;
    const int first = t1 > t0 ? t0 / a.chunk + s : 0, last = t1 > t0 ? (t1 - 1) / a.chunk + s + 1 : 0;
    float q = 0.f;
    int c = 0, n = 0;
#pragma unroll 4
    for (int u = first + lane / 8 + (BLOCK ? warp * 4 : 0); u < last; u += BLOCK ? WARPS * 4 : 4) {
      if (e < E) {
        q += a.part_q[static_cast<size_t>(u) * E + e];
        c += a.part_c[static_cast<size_t>(u) * E + e];
      }
      n += a.part_n[u];
    }
#pragma unroll
    for (int o = 8; o < 32; o *= 2) {
      q += __shfl_xor_sync(0xffffffffu, q, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (BLOCK) {
      if (lane < kFinCols) s_q[warp][lane] = q, s_c[warp][lane] = c;
      if (lane == 0) s_n[warp] = n;
      __syncthreads();
      q = 0.f, c = 0, n = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) q += s_q[w][lane % 8], c += s_c[w][lane % 8], n += s_n[w];
      __syncthreads();
      if (warp) continue;
    }
    const float nf = static_cast<float>(n);
    float share = 0.f;
    if (e < E) {
      if (lane < kFinCols) {
        a.counts[static_cast<size_t>(s) * E + e] = c;
        if (a.prob) a.prob[static_cast<size_t>(s) * E + e] = n > 0 ? __fdiv_rn(q, nf) : 0.f;
      }
      share = n > 0 ? static_cast<float>(c) * q : 0.f;
    }
#pragma unroll
    for (int o = 1; o < kFinCols; o *= 2) share += __shfl_xor_sync(0xffffffffu, share, o);
    if (lane == 0) {
      a.share[i] = n > 0 ? share * __fdiv_rn(a.alpha * E, a.k * nf * nf) : 0.f;
      if (slab == 0) a.tokens[s] = n;
    }
  }
  __syncthreads();
  if (tid == 0) {   // the block's results, which the barrier has brought here, before its arrival; the others' after it
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(a.done) : "memory");
    s_last = before == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!s_last) return;
  float sum = 0.f;
  int live = 0, err = 0;
#pragma unroll 4
  for (long long i = tid; i < tasks; i += kBalThreads) sum += __ldcg(a.share + i);
  for (int i = tid; i < a.chunks; i += kBalThreads) err |= a.part_err[i];
  const int first = tid < a.S ? __ldcg(a.tokens + tid) : 0;
  live = first > 0;
  for (int s = tid + kBalThreads; s < a.S; s += kBalThreads) live += __ldcg(a.tokens + s) > 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  live = __reduce_add_sync(0xffffffffu, live);
  err = __reduce_or_sync(0xffffffffu, err);
  if (lane == 0) s_sum[warp] = sum, s_n[warp] = live, s_c[warp][0] = err;
  __syncthreads();
  sum = 0.f, live = 0, err = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) sum += s_sum[w], live += s_n[w], err |= s_c[w][0];
  for (int s = tid; s < a.S; s += kBalThreads) {
    const float nf = static_cast<float>(s == tid ? first : __ldcg(a.tokens + s));
    a.coef[s] = nf > 0.f ? __fdiv_rn(a.alpha * E, a.k * nf * nf * static_cast<float>(live)) : 0.f;
  }
  if (tid == 0) {
    *a.loss = live > 0 ? __fdiv_rn(sum, static_cast<float>(live)) : 0.f;
    *a.status = err & 2 ? MOE_ERR_BAD_OFFSETS : err & 1 ? MOE_ERR_INVALID : MOE_OK;
  }
}

// Both passes of a small batch in one launch, the cluster's CTAs a chunk each.
template <typename T, int V>
__global__ void __launch_bounds__(kBalThreads) __cluster_dims__(kFinCluster, 1, 1)
    balance_small_kernel(const BalanceArgs a, int cols, int w) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ float s_mem[];
  if (static_cast<int>(blockIdx.x) < a.chunks) balance_partial<T, V>(a, s_mem);
  cluster_barrier();   // the partial sums are there, in global memory
  balance_finish(a, cols, w);
}

struct RouterGradArgs {
  const void* logits;
  const int32_t* idx;
  const float* d_w;      // [T, k] or nullptr
  int T, E, k, renorm;
  const int32_t* off;
  int S;
  const uint8_t* mask;
  const int32_t* counts;  // [S, E] or nullptr: no balance loss
  const float* coef;      // [S]
  const float* d_loss;    // device scalar or nullptr (1)
  void* out;
  int chunk, L, vec;
};

// Selected mass below which a renormalised row is worked out again: a probability that underflowed is then less
// than 1e-18 of it.
constexpr float kLowMass = 1e-20f;

// The dense part of a row, p (bal - dot), is written in whole pieces; the
// selected experts' entries are then written over it by the lanes that hold
// the slots (lane l slots l and l + L), which read their own logit again: a
// search of the row's registers for k columns would cost more than the softmax.
template <typename T, typename OT, int V, bool kRenorm, bool kTwo>
__global__ void __launch_bounds__(kBalThreads, V <= 16 ? 3 : 2) router_backward_kernel(const RouterGradArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int E = a.E, L = a.L, k = a.k;
  const int tid = threadIdx.x, lane = tid & 31;
  const int l = lane % L, group = tid / L, groups = kBalThreads / L;
  const T* logits = static_cast<const T*>(a.logits);
  OT* out = static_cast<OT*>(a.out);
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  // one renormalised gate is 1 whatever its logit
  const bool gates = a.d_w && !(kRenorm && k == 1);
  int s = a.counts && a.off ? sequence_at(a.off, a.S, t0) : 0;
  int held = -1;        // the sequence whose counts are in bal
  float c_s = 0.f;
  float bal[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bal[i] = 0.f;
  const float d_loss = a.counts && a.d_loss ? __ldg(a.d_loss) : 1.f;

  constexpr int U = kTwo ? 2 : 1;   // slots to a lane
  Row<T, V> next;
  int next_e[U];
  float next_g[U];
#pragma unroll
  for (int u = 0; u < U; ++u) next_e[u] = -1, next_g[u] = 0.f;
  bool next_kept = false;
  int seq_end = !a.counts || s >= a.S ? 0 : a.off ? a.off[s + 1] : a.T;
  const unsigned group_lanes = (L == 32 ? 0xffffffffu : (1u << L) - 1) << (lane & ~(L - 1));
  auto prefetch = [&](int t) {
    const bool live = t < t1;
    const size_t tr = live ? t : t0;
    next.load(logits + tr * E, E, L, l, a.vec);   // past the end an earlier row again, not written
    next_kept = !a.mask || a.mask[tr];
    if (gates) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = live && l + u * L < k;
        next_e[u] = in ? __ldg(a.idx + tr * k + l + u * L) : -1;
        next_g[u] = in ? __ldg(a.d_w + tr * k + l + u * L) : 0.f;
      }
    }
  };
  prefetch(t0 + group);
  for (int b = t0; b < t1; b += groups) {
    const int t = b + group;
    const bool live = t < t1;
    const int tr = live ? t : t0;
    const T* row = logits + static_cast<size_t>(tr) * E;
    Row<T, V> now = next;
    bool in = false;
    if (a.counts) {
      if (live)
        while (s < a.S && seq_end <= tr) {
          ++s;
          seq_end = s < a.S ? a.off[s + 1] : 0;   // without offsets there is one sequence, which no token passes
        }
      in = live && s < a.S && next_kept;
      if (in && held != s) {
        held = s;
        c_s = __ldg(a.coef + s) * d_loss;
        const int32_t* cnt = a.counts + static_cast<size_t>(s) * E;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = column<T>(i, L, l);
          bal[i] = c < E ? c_s * static_cast<float>(__ldg(cnt + c)) : 0.f;
        }
      }
    }
    int e[U];
    float g[U], x[U], be[U];
    bool some = false;   // a slot without an expert whose gradient is not 0 counts, too
#pragma unroll
    for (int u = 0; u < U; ++u) {
      e[u] = next_e[u] >= 0 && next_e[u] < E ? next_e[u] : -1;
      g[u] = e[u] >= 0 ? next_g[u] : 0.f;
      some |= next_g[u] != 0.f;
      x[u] = e[u] >= 0 ? to_f32(row[e[u]]) : -INFINITY;
      be[u] = e[u] >= 0 && in ? c_s * static_cast<float>(__ldg(a.counts + static_cast<size_t>(s) * E + e[u])) : 0.f;
    }
    if (b + groups < t1) prefetch(t + groups);
    // something to differentiate: else the row's gradient is 0 whatever its logits hold
    const bool any = (__ballot_sync(0xffffffffu, some) & group_lanes) != 0 || in;
    if (!any) now.clear();
    float p[V], m, inv;
    softmax_row(now, p, L, m, inv);
    float dots[2] = {0.f, 0.f};   // sum of p times what it is multiplied with: the loss's part, and the raw gates'
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= inv;
    if (in) {
#pragma unroll
      for (int i = 0; i < V; ++i) dots[i & 1] = fmaf(p[i], bal[i], dots[i & 1]);
    }
    float dot = dots[0] + dots[1];
    float ps[U], z = 0.f, wg = 0.f;
    if (gates) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ps[u] = e[u] >= 0 && any ? exp_from(x[u], m) * inv : 0.f;
        const float pg = e[u] >= 0 ? ps[u] * g[u] : 0.f;
        if (kRenorm)
          z += ps[u], wg += pg;
        else
          dot += pg;
      }
    }
    dot = group_sum(dot, L);
    // the gradients of every slot that chose the same expert (one, as the router gives them)
    float gs[U], ns[U];
#pragma unroll
    for (int u = 0; u < U; ++u) gs[u] = ns[u] = 0.f;
    if (gates) {
      for (int j = 0; j < k; ++j) {
        const int from = (lane & ~(L - 1)) | (j & (L - 1));
        const int ej = __shfl_sync(0xffffffffu, j < L ? e[0] : e[U - 1], from);
        const float gj = __shfl_sync(0xffffffffu, j < L ? g[0] : g[U - 1], from);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          gs[u] += ej == e[u] ? gj : 0.f;
          if (kRenorm) ns[u] += ej == e[u] ? 1.f : 0.f;
        }
      }
    }
    float inv_z = 0.f, pw[U];   // the renormalised gates' numerators: the selected probabilities
#pragma unroll
    for (int u = 0; u < U; ++u) pw[u] = gates ? ps[u] : 0.f;
    if (kRenorm && gates) {   // over the selected experts alone: w = p / z, their gradient w (g - sum w g)
      z = group_sum(z, L);
      wg = group_sum(wg, L);
      // Selected experts far below the row's maximum (chosen by something else than these logits): their masses
      // underflow, so their softmax is taken from their own maximum.
      const bool low = any && z < kLowMass;
      if (__any_sync(0xffffffffu, low)) {
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, x[u]);   // -inf where there is none
        top = group_max(top, L);
        float zl = 0.f, wl = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float pu = low && x[u] > -INFINITY ? exp_from(x[u], top) : 0.f;
          if (low) pw[u] = pu;
          zl += pu, wl += e[u] >= 0 ? pu * g[u] : 0.f;
        }
        zl = group_sum(zl, L);
        wl = group_sum(wl, L);
        if (low) z = zl, wg = wl;
      }
      inv_z = z == 0.f ? 0.f : __fdiv_rn(1.f, z);
      wg *= inv_z;
    }
    if (in) {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= bal[i] - dot;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= -dot;
    }
    OT* o = out + static_cast<size_t>(tr) * E;
#pragma unroll
    for (int q = 0; q < V / piece<T>(); ++q) {
      constexpr int C = piece<T>();
      const int c = (q * L + l) * C;
      if (a.vec) {
        if (live && c < E) store_run<OT, C>(o + c, p + q * C);
      } else {
#pragma unroll
        for (int u = 0; u < C; ++u)
          if (live && c + u < E) o[c + u] = from_f32(p[q * C + u], OT());
      }
    }
    if (gates) {
      __syncwarp();   // the selected entries come after the row's
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!live || !any || e[u] < 0) continue;
        float v;
        if (kRenorm)
          v = fmaf(pw[u] * inv_z, gs[u] - ns[u] * wg, ps[u] * (be[u] - dot));
        else
          v = ps[u] * (be[u] + gs[u] - dot);
        o[e[u]] = from_f32(v, OT());
      }
    }
  }
}

int lanes_for(int E, int V) {  // lanes of a row: a power of two, V columns each
  int L = 1;
  while (L < 32 && L * V < E) L *= 2;
  return L;
}
int values_for(int E) { return E <= 512 ? 16 : 32; }

// Blocks that run at once: three to an SM, two where a lane holds 32 columns (with one, 8192 tokens of 1024
// experts in bf16 took the gradient 29.4 us in three waves, 18.8 in one of two to an SM).
int blocks_at_once(int E) { return num_sms() * (values_for(E) == 16 ? 3 : 2); }

int balance_chunk(int T, int E) {
  if (T <= kBalSmall) return T > 0 ? (T + kFinCluster - 1) / kFinCluster : 1;
  const int c = (T + blocks_at_once(E) - 1) / blocks_at_once(E);
  return c < kBalMinChunk ? kBalMinChunk : c;
}

template <typename T>
int launch_partial(const BalanceArgs& a, int V, int cols, int w, cudaStream_t s) {
  const size_t smem = (static_cast<size_t>(kBalThreads) * V + a.E) * 4;
  const dim3 grid(a.chunks), block(kBalThreads);
  if (a.T <= kBalSmall) {
    const dim3 one(kFinCluster);
    if (V == 16) return launch_pdl(__func__, balance_small_kernel<T, 16>, one, block, smem, s, a, cols, w);
    return launch_pdl(__func__, balance_small_kernel<T, 32>, one, block, smem, s, a, cols, w);
  }
  if (V == 16) return launch_pdl(__func__, balance_partial_kernel<T, 16>, grid, block, smem, s, a);
  return launch_pdl(__func__, balance_partial_kernel<T, 32>, grid, block, smem, s, a);
}

template <typename T, typename OT, int V, bool kTwo>
int launch_grad_rows(const RouterGradArgs& a, int grid, cudaStream_t s) {
  const dim3 g(grid), b(kBalThreads);
  return a.renorm ? launch_pdl("router_backward_kernel", router_backward_kernel<T, OT, V, true, kTwo>, g, b, 0, s, a)
                  : launch_pdl("router_backward_kernel", router_backward_kernel<T, OT, V, false, kTwo>, g, b, 0, s, a);
}
template <typename T, typename OT>
int launch_grad(const RouterGradArgs& a, int V, int grid, cudaStream_t s) {
  if (V == 32) return launch_grad_rows<T, OT, 32, false>(a, grid, s);   // a whole warp to a row
  return a.k > a.L ? launch_grad_rows<T, OT, 16, true>(a, grid, s) : launch_grad_rows<T, OT, 16, false>(a, grid, s);
}

template <typename T>
int launch_grad_to(const RouterGradArgs& a, int out_dtype, int V, int grid, cudaStream_t s) {
  if (out_dtype == MOE_F32) return launch_grad<T, float>(a, V, grid, s);
  if (out_dtype == MOE_F16) return launch_grad<T, __half>(a, V, grid, s);
  return launch_grad<T, __nv_bfloat16>(a, V, grid, s);
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) {
  const size_t chunks = T > 0 ? (T + balance_chunk(T, E) - 1) / balance_chunk(T, E) : 0;
  const size_t slots = chunks + S;
  const size_t tasks = T > kBalSmall ? static_cast<size_t>(S) * ((E + kFinCols - 1) / kFinCols) + S : 0;
  return 256 + align_up(slots * E * 4, 256) * 2 + align_up(slots * 4, 256) + align_up(chunks * 4 + 4, 256) +
         align_up(tasks * 4, 256);
}

int launch_balance_loss(const void* logits, int dtype, const int32_t* idx, int T, int E, int k, const int32_t* off,
                        int S, const uint8_t* mask, float alpha, float* loss, int32_t* counts, float* prob,
                        float* coef, void* ws, cudaStream_t s) {
  BalanceArgs a{};
  const int V = values_for(E);
  a.logits = logits, a.idx = idx, a.T = T, a.E = E, a.k = k, a.off = off, a.S = S, a.mask = mask, a.alpha = alpha;
  a.chunk = balance_chunk(T, E);
  a.chunks = T > 0 ? (T + a.chunk - 1) / a.chunk : 0;
  a.L = lanes_for(E, V);
  a.vec = E % (dtype == MOE_F32 ? 4 : 8) != 0 ? 0 : E == a.L * V ? 2 : 1;
  const size_t slots = static_cast<size_t>(a.chunks) + S, m = align_up(slots * E * 4, 256);
  char* p = static_cast<char*>(ws);
  a.status = reinterpret_cast<int*>(p);
  a.part_q = reinterpret_cast<float*>(p + 256);
  a.part_c = reinterpret_cast<int32_t*>(p + 256 + m);
  a.part_n = reinterpret_cast<int32_t*>(p + 256 + 2 * m);
  a.part_err = reinterpret_cast<int32_t*>(p + 256 + 2 * m + align_up(slots * 4, 256));
  a.done = a.status + 1;
  a.share = reinterpret_cast<float*>(reinterpret_cast<char*>(a.part_err) + align_up(static_cast<size_t>(a.chunks) * 4 + 4, 256));
  a.tokens = reinterpret_cast<int32_t*>(a.share) + static_cast<size_t>(S) * ((E + kFinCols - 1) / kFinCols);
  a.loss = loss, a.counts = counts, a.prob = prob, a.coef = coef;
  // a small batch: columns of a CTA and threads of a column, powers of two
  int cols = 8;
  while (cols * kFinCluster < E) cols *= 2;
  int w = 1;
  while (w < 32 && w * cols < kBalThreads && w * 8 < a.chunks / S + 1) w *= 2;
  const int st = dtype == MOE_F32   ? launch_partial<float>(a, V, cols, w, s)
                 : dtype == MOE_F16 ? launch_partial<__half>(a, V, cols, w, s)
                                    : launch_partial<__nv_bfloat16>(a, V, cols, w, s);
  if (st != MOE_OK || T <= kBalSmall) return st;
  // a sequence of more than 16 slots is worth a block's 32 lanes to a column
  const bool block = a.chunks / S > 16;
  const long long tasks = static_cast<long long>(S) * ((E + kFinCols - 1) / kFinCols), blocks = block ? tasks : (tasks + 7) / 8;
  const dim3 grid(static_cast<unsigned>(blocks < 8 * num_sms() ? blocks : 8 * num_sms()));
  return block ? launch_pdl(__func__, balance_finish_kernel<true>, grid, dim3(kBalThreads), 0, s, a)
               : launch_pdl(__func__, balance_finish_kernel<false>, grid, dim3(kBalThreads), 0, s, a);
}

int launch_router_backward(const void* logits, int dtype, const int32_t* idx, const float* d_w, int T, int E, int k,
                           int renorm, const int32_t* off, int S, const uint8_t* mask, const int32_t* counts,
                           const float* coef, const float* d_loss, void* out, int out_dtype, cudaStream_t s) {
  if (T == 0) return MOE_OK;
  RouterGradArgs a{};
  const int V = values_for(E);
  a.logits = logits, a.idx = idx, a.d_w = d_w, a.T = T, a.E = E, a.k = k, a.renorm = renorm, a.off = off, a.S = S;
  a.mask = counts ? mask : nullptr;   // a token's gates have their gradient whether it counts or not
  a.counts = counts, a.coef = coef, a.d_loss = d_loss, a.out = out;
  a.L = lanes_for(E, V);
  while (a.L * 2 < k) a.L *= 2;   // two slots to a lane
  a.vec = E % (dtype == MOE_F32 ? 4 : 8) != 0 ? 0 : E == a.L * V ? 2 : 1;   // not 0: rows of every output type are stored whole too
  const int groups = kBalThreads / a.L;
  const int blocks = blocks_at_once(E);
  a.chunk = (T + blocks - 1) / blocks;
  a.chunk = (a.chunk + groups - 1) / groups * groups;
  const int grid = (T + a.chunk - 1) / a.chunk;
  if (dtype == MOE_F32) return launch_grad_to<float>(a, out_dtype, V, grid, s);
  if (dtype == MOE_F16) return launch_grad_to<__half>(a, out_dtype, V, grid, s);
  return launch_grad_to<__nv_bfloat16>(a, out_dtype, V, grid, s);
}

}  // namespace moe
