// route.hip -- expert routing: counts, offsets and the row order of the assignments, the balance
// loss and its gradient (htroute.h).
#include <algorithm>

#include "../../include/htroute.h"
#include "kernels.h"

namespace htk {
namespace {

constexpr int kRouteWaves = 16, kRouteChunk = 2048, kRouteBlocks = 256;
constexpr int kLossWaves = 8, kLossBlocks = 256;

// ---- order ---------------------------------------------------------------------------------
struct RParams {
  const int32_t* ids;
  const uint8_t* mask;
  int64_t ld_ids, rows;
  int n, topk, experts, align;   // n: assignments
  int chunk;                     // assignments per workgroup
  int32_t* counts;
  int32_t* offsets;
  int32_t* order;
  int32_t* slot;
  int32_t* hist;                 // gridDim.x x experts
};

// The expert of assignment i, or -1 when it is dropped.
__device__ __forceinline__ int expert_of(const RParams& p, int i) {
  const int t = i / p.topk;
  if (p.mask && !p.mask[t]) return -1;
  const int e = p.ids[(int64_t)t * p.ld_ids + (i - t * p.topk)];
  return e >= 0 && e < p.experts ? e : -1;
}

// Lanes of the wave that hold the same expert (dropped lanes match nothing of interest).
__device__ __forceinline__ unsigned long long same_expert(int e) {
  unsigned long long m = ~0ull;
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const unsigned long long s = __ballot((e >> b) & 1);
    m &= (e >> b) & 1 ? s : ~s;
  }
  return m & __ballot(e >= 0);
}

// Exclusive sum over the 1024 threads of a workgroup; `sums` holds one int per wave.
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  if (lane == 63) sums[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRouteWaves; ++w) {
    before += w < wave ? sums[w] : 0;
    all += sums[w];
  }
  *total = all;
  return before + s - v;
}

// How often each expert occurs in each workgroup's chunk.
__global__ __launch_bounds__(1024) void route_hist(const RParams p) {
  extern __shared__ int sh[];
  for (int e = threadIdx.x; e < p.experts; e += 1024) sh[e] = 0;
  __syncthreads();
  const int end = min((int64_t)p.n, ((int64_t)blockIdx.x + 1) * p.chunk);
  for (int i = blockIdx.x * p.chunk + threadIdx.x; i < end; i += 1024) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(&sh[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += 1024) p.hist[(int64_t)blockIdx.x * p.experts + e] = sh[e];
}

// A stable counting sort.  Each workgroup places its chunk of the assignments, each wave a run of
// it in order: an assignment's row is the expert's first row, plus the expert's assignments in
// earlier chunks (from route_hist), in earlier waves (counted here first), and in earlier steps
// and lanes of its wave.  One chunk needs no route_hist.
__global__ __launch_bounds__(1024) void route_place(const RParams p) {
  extern __shared__ int sh[];       // [waves][experts] then, for the scan, one int per wave
  __shared__ int sums[kRouteWaves];
  const int E = p.experts, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x, nb = gridDim.x;
  for (int i = tid; i < kRouteWaves * E; i += 1024) sh[i] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)b * p.chunk, end = min((int64_t)p.n, begin + p.chunk);
  const int run = (p.chunk + kRouteWaves - 1) / kRouteWaves;
  const int64_t w0 = min(begin + (int64_t)wave * run, end), w1 = min(w0 + run, end);
  int* mine = sh + wave * E;
  for (int64_t i = w0 + lane; i < w1; i += 64) {
    const int e = expert_of(p, (int)i);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  // thread e: its expert's total and the part in earlier chunks
  int before = 0, count = 0;
  if (tid < E) {
    if (nb == 1) {
      for (int w = 0; w < kRouteWaves; ++w) count += sh[w * E + tid];
    } else {
#pragma unroll 8
      for (int c = 0; c < nb; ++c) {
        const int v = p.hist[(int64_t)c * E + tid];
        before += c < b ? v : 0;
        count += v;
      }
    }
  }
  const int room = (count + p.align - 1) / p.align * p.align;
  int total;
  const int first = block_scan(tid < E ? room : 0, sums, &total);
  if (tid < E) {
    int at = first + before;
    for (int w = 0; w < kRouteWaves; ++w) {
      const int v = sh[w * E + tid];
      sh[w * E + tid] = at;
      at += v;
    }
    if (b == 0) {
      p.counts[tid] = count;
      p.offsets[tid] = first;
      if (tid == 0) p.offsets[E] = total;
    }
    // rows that hold no assignment: the fill of each expert, dealt over the workgroups
    if (p.order && tid % nb == b)
      for (int r = first + count; r < first + room; ++r) p.order[r] = -1;
  }
  if (p.order)
    for (int64_t r = total + (int64_t)b * 1024 + tid; r < p.rows; r += (int64_t)nb * 1024) p.order[r] = -1;
  __syncthreads();
  volatile int* next = mine;        // this wave's own; its LDS accesses keep their order
  for (int64_t s = w0; s < w1; s += 64) {
    const int i = (int)s + lane;
    const int e = i < w1 ? expert_of(p, i) : -1;
    const unsigned long long same = same_expert(e);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int at = -1;
    if (e >= 0) at = next[e] + rank;
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && rank == 0) next[e] = at + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < w1) {
      if (p.slot) p.slot[i] = at;
      if (p.order && at >= 0) p.order[at] = i;
    }
  }
}

// ---- balance loss ---------------------------------------------------------------------------
struct BParams {
  const void* logits;
  const uint8_t* mask;
  const int32_t* counts;
  int64_t tokens, ld, ld_d;
  int experts, topk;
  float coef;
  float* partial;      // blocks x experts
  int32_t* partial_n;  // blocks
  float* loss;
  float* prob;
  int32_t* live;
  const float* d_loss;
  void* d_logits;
  int64_t per;         // tokens per workgroup
};

template <int T> struct Elem;
template <> struct Elem<DT_F32> {
  typedef float S;
  __device__ static float up(float v) { return v; }
  __device__ static float down(float v) { return v; }
};
template <> struct Elem<DT_F16> {
  typedef u16 S;
  __device__ static float up(u16 v) { return f16_to_f32(v); }
  __device__ static u16 down(float v) { return f32_to_f16(v); }
};
template <> struct Elem<DT_BF16> {
  typedef u16 S;
  __device__ static float up(u16 v) { return bf16_to_f32(v); }
  __device__ static u16 down(float v) { return f32_to_bf16(v); }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Softmax of one row, lane l holding experts l, l + 64, ...; zero in all for a row of -infinity.
// The maximum keeps a NaN out, the sum carries it to every probability.
template <int T, int NE>
__device__ __forceinline__ void softmax_row(const BParams& p, int64_t t, int lane, float (&v)[NE]) {
  const typename Elem<T>::S* x = (const typename Elem<T>::S*)p.logits + t * p.ld;
  float top = -__builtin_inff();
  static_for<NE>([&](auto i) {
    const int e = lane + 64 * i;
    v[i] = e < p.experts ? Elem<T>::up(x[e]) : -__builtin_inff();
    top = fmaxf(top, v[i]);
  });
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  const float base = top == -__builtin_inff() ? 0.f : top;
  float sum = 0.f;
  static_for<NE>([&](auto i) {
    v[i] = expf(v[i] - base);
    sum += v[i];
  });
  sum = wave_sum(sum);
  const float r = sum == 0.f ? 0.f : 1.f / sum;
  static_for<NE>([&](auto i) { v[i] *= r; });
}

// prob and loss from the workgroups' sums, added in order, in double.
__device__ __forceinline__ void finish_loss(const BParams& p, int blocks) {
  __shared__ double part[1024];
  __shared__ int n_live;
  const int tid = threadIdx.x, nt = blockDim.x;
  if (tid == 0) n_live = 0;
  __syncthreads();
  int n = 0;
  for (int b = tid; b < blocks; b += nt) n += p.partial_n[b];
  if (n) atomicAdd(&n_live, n);     // integers: any order gives the same sum
  __syncthreads();
  n = n_live;
  // G threads for each expert, each over every G-th block; their sums are then added in order
  int G = 1;
  while (2 * G * p.experts <= nt && 2 * G <= blocks) G *= 2;
  double dot = 0.0;
  for (int e0 = 0; e0 < p.experts; e0 += nt / G) {
    const int wide = min(p.experts - e0, nt / G), e = e0 + tid % wide, q = tid / wide;
    double s = 0.0;
    if (q < G) {
#pragma unroll 4
      for (int b = q; b < blocks; b += G) s += p.partial[(int64_t)b * p.experts + e];
      part[q * wide + tid % wide] = s;
    }
    __syncthreads();
    if (tid < wide) {
      s = 0.0;
      for (int g = 0; g < G; ++g) s += part[g * wide + tid];
      const double mean = n > 0 ? s / n : 0.0;
      p.prob[e0 + tid] = (float)mean;
      dot += mean * p.counts[e0 + tid];
    }
    __syncthreads();
  }
  part[tid] = dot;
  __syncthreads();
  for (int d = 512; d > 0; d >>= 1) {
    if (tid < d && tid + d < nt) part[tid] += part[tid + d];
    __syncthreads();
  }
  if (tid == 0) {
    *p.loss = n > 0 ? (float)(p.coef * part[0] * p.experts / ((double)p.topk * n)) : 0.f;
    *p.live = n;
  }
}

// Sums of the probabilities over each workgroup's tokens: a wave takes every 8th of them.
template <int T, int NE>
__global__ __launch_bounds__(kLossWaves * 64) void balance_sums(const BParams p) {
  extern __shared__ float sums[];   // [waves][experts]
  __shared__ int live[kLossWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = blockIdx.x * p.per, t1 = min(t0 + p.per, p.tokens);
  float acc[NE];
  static_for<NE>([&](auto i) { acc[i] = 0.f; });
  int n = 0;
  for (int64_t t = t0 + wave; t < t1; t += kLossWaves) {
    if (p.mask && !p.mask[t]) continue;
    float v[NE];
    softmax_row<T, NE>(p, t, lane, v);
    static_for<NE>([&](auto i) { acc[i] += v[i]; });
    ++n;
  }
  static_for<NE>([&](auto i) {
    if (lane + 64 * i < p.experts) sums[wave * p.experts + lane + 64 * i] = acc[i];
  });
  if (lane == 0) live[wave] = n;
  __syncthreads();
  for (int e = tid; e < p.experts; e += kLossWaves * 64) {
    float s = 0.f;
    for (int w = 0; w < kLossWaves; ++w) s += sums[w * p.experts + e];
    p.partial[(int64_t)blockIdx.x * p.experts + e] = s;
  }
  if (tid == 0) {
    n = 0;
    for (int w = 0; w < kLossWaves; ++w) n += live[w];
    p.partial_n[blockIdx.x] = n;
  }
  if (gridDim.x == 1) {             // one workgroup has all the sums: finish here
    __threadfence_block();
    __syncthreads();
    finish_loss(p, 1);
  }
}

__global__ __launch_bounds__(1024) void balance_finish(const BParams p, int blocks) { finish_loss(p, blocks); }

// g is taken relative to an even load, (experts * counts - topk * n) as an integer: the constant
// drops out of g - sum p g, and what is left has no cancellation to lose bits to.
template <int T, int NE>
__global__ __launch_bounds__(256) void balance_slopes(const BParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * 4, w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int n = *p.live;
  const double kn = (double)p.topk * n;
  const float scale = n > 0 ? (float)((double)*p.d_loss * p.coef / (kn * n)) : 0.f;
  float g[NE];
  static_for<NE>([&](auto i) {
    const int e = lane + 64 * i;
    g[i] = e < p.experts ? scale * (float)((int64_t)p.counts[e] * p.experts - (int64_t)p.topk * n) : 0.f;
  });
  for (int64_t t = w; t < p.tokens; t += waves) {
    float v[NE];
    if (n == 0 || (p.mask && !p.mask[t])) {
      static_for<NE>([&](auto i) { v[i] = 0.f; });
    } else {
      softmax_row<T, NE>(p, t, lane, v);
      float s = 0.f;
      static_for<NE>([&](auto i) { s += v[i] * g[i]; });
      s = wave_sum(s);
      static_for<NE>([&](auto i) { v[i] *= g[i] - s; });
    }
    typename Elem<T>::S* d = (typename Elem<T>::S*)p.d_logits + t * p.ld_d;
    static_for<NE>([&](auto i) {
      if (lane + 64 * i < p.experts) d[lane + 64 * i] = Elem<T>::down(v[i]);
    });
  }
}

int64_t loss_blocks(int64_t tokens) {
  return std::max<int64_t>(1, std::min<int64_t>(kLossBlocks, tokens / (4 * kLossWaves)));
}
int64_t route_blocks(int64_t n) {
  return std::max<int64_t>(1, std::min<int64_t>(kRouteBlocks, (n + kRouteChunk - 1) / kRouteChunk));
}

template <class F> bool with_type(int type, F f) {
  switch (type) {
    case GEMM_F32: f(std::integral_constant<int, DT_F32>{}); return true;
    case GEMM_F16: f(std::integral_constant<int, DT_F16>{}); return true;
    case GEMM_BF16: f(std::integral_constant<int, DT_BF16>{}); return true;
    default: return false;
  }
}
// NE: the experts of a lane, rounded up to a power of two
template <class F> void with_lanes(int experts, F f) {
  if (experts <= 64) f(std::integral_constant<int, 1>{});
  else if (experts <= 128) f(std::integral_constant<int, 2>{});
  else if (experts <= 256) f(std::integral_constant<int, 4>{});
  else if (experts <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_sizes(int64_t tokens, int32_t topk, int32_t experts) {
  if (tokens < 0 || topk < 1 || topk > ROUTE_MAX_TOPK || experts < 1 || experts > ROUTE_MAX_EXPERTS)
    return GEMM_ERR_INVALID_ARG;
  return tokens > INT32_MAX / 2 / topk ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}
int check_logits(int64_t tokens, int32_t topk, int32_t experts, int32_t type, int64_t ld, const void* x) {
  const int rc = check_sizes(tokens, topk, experts);
  if (rc) return rc;
  if (type != GEMM_F32 && type != GEMM_F16 && type != GEMM_BF16) return GEMM_ERR_DTYPE_COMBO;
  if (ld < experts) return GEMM_ERR_LAYOUT;
  if (tokens > 0 && !x) return GEMM_ERR_INVALID_ARG;
  return on(x, type == GEMM_F32 ? 4 : 2) ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

}  // namespace
}  // namespace htk

using namespace htk;

extern "C" {

int route_workspace_size(int64_t tokens, int32_t topk, int32_t experts, size_t* bytes) {
  const int rc = check_sizes(tokens, topk, experts);
  if (rc) return rc;
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  const size_t hist = (size_t)route_blocks(tokens * topk) * experts * 4;
  const size_t loss = (size_t)loss_blocks(tokens) * (experts + 1) * 4;
  *bytes = (std::max(hist, loss) + 255) / 256 * 256;
  return GEMM_OK;
}

int route_experts(const route_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  int rc = check_sizes(a->tokens, a->topk, a->experts);
  if (rc) return rc;
  if (a->align < 1 || a->align > 1024) return GEMM_ERR_INVALID_ARG;
  if (a->ld_ids < a->topk) return GEMM_ERR_LAYOUT;
  if ((a->tokens > 0 && !a->ids) || !a->counts || !a->offsets || !a->workspace) return GEMM_ERR_INVALID_ARG;
  const int64_t n = a->tokens * a->topk;
  if (a->order && a->rows < n + (int64_t)a->experts * (a->align - 1)) return GEMM_ERR_INVALID_ARG;
  if (!on(a->ids, 4) || !on(a->counts, 4) || !on(a->offsets, 4) || !on(a->order, 4) || !on(a->slot, 4) ||
      !on(a->workspace, 16))
    return GEMM_ERR_MISALIGNED;
  rc = arch_status();
  if (rc) return rc;
  RParams p;
  p.ids = a->ids;
  p.mask = a->mask;
  p.ld_ids = a->ld_ids;
  p.rows = a->rows;
  p.n = (int)n;
  p.topk = a->topk;
  p.experts = a->experts;
  p.align = a->align;
  const int64_t blocks = route_blocks(n);
  p.chunk = (int)std::max<int64_t>((n + blocks - 1) / blocks, 1);
  p.counts = a->counts;
  p.offsets = a->offsets;
  p.order = a->order;
  p.slot = a->slot;
  p.hist = static_cast<int32_t*>(a->workspace);
  hipStream_t s = (hipStream_t)stream;
  if (blocks > 1) {
    hipLaunchKernelGGL(route_hist, dim3((unsigned)blocks), dim3(1024), a->experts * 4, s, p);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_LAUNCH;
  }
  hipLaunchKernelGGL(route_place, dim3((unsigned)blocks), dim3(1024), kRouteWaves * a->experts * 4, s, p);
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int balance_loss(const balance_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  int rc = check_logits(a->tokens, a->topk, a->experts, a->type, a->ld, a->logits);
  if (rc) return rc;
  if (!a->counts || !a->loss || !a->prob || !a->live || !a->workspace) return GEMM_ERR_INVALID_ARG;
  if (!on(a->counts, 4) || !on(a->loss, 4) || !on(a->prob, 4) || !on(a->live, 4) || !on(a->workspace, 16))
    return GEMM_ERR_MISALIGNED;
  rc = arch_status();
  if (rc) return rc;
  const int64_t blocks = loss_blocks(a->tokens);
  BParams p = {};
  p.logits = a->logits;
  p.mask = a->mask;
  p.counts = a->counts;
  p.tokens = a->tokens;
  p.ld = a->ld;
  p.experts = a->experts;
  p.topk = a->topk;
  p.coef = a->coef;
  p.partial = static_cast<float*>(a->workspace);
  p.partial_n = reinterpret_cast<int32_t*>(p.partial + blocks * a->experts);
  p.loss = a->loss;
  p.prob = a->prob;
  p.live = a->live;
  p.per = (a->tokens + blocks - 1) / blocks;
  hipStream_t s = (hipStream_t)stream;
  with_type(a->type, [&](auto T) {
    with_lanes(a->experts, [&](auto NE) {
      hipLaunchKernelGGL((balance_sums<decltype(T)::value, decltype(NE)::value>), dim3((unsigned)blocks),
                         dim3(kLossWaves * 64), kLossWaves * a->experts * 4, s, p);
    });
  });
  if (hipGetLastError() != hipSuccess) return GEMM_ERR_LAUNCH;
  if (blocks > 1) {
    hipLaunchKernelGGL(balance_finish, dim3(1), dim3(1024), 0, s, p, (int)blocks);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

int balance_grad(const balance_grad_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  int rc = check_logits(a->tokens, a->topk, a->experts, a->type, a->ld, a->logits);
  if (rc) return rc;
  if (a->ld_d < a->experts) return GEMM_ERR_LAYOUT;
  if (!a->counts || !a->live || !a->d_loss || (a->tokens > 0 && !a->d_logits)) return GEMM_ERR_INVALID_ARG;
  if (!on(a->counts, 4) || !on(a->live, 4) || !on(a->d_loss, 4) || !on(a->d_logits, a->type == GEMM_F32 ? 4 : 2))
    return GEMM_ERR_MISALIGNED;
  rc = arch_status();
  if (rc) return rc;
  if (a->tokens == 0) return GEMM_OK;
  BParams p = {};
  p.logits = a->logits;
  p.mask = a->mask;
  p.counts = a->counts;
  p.tokens = a->tokens;
  p.ld = a->ld;
  p.ld_d = a->ld_d;
  p.experts = a->experts;
  p.topk = a->topk;
  p.coef = a->coef;
  p.live = const_cast<int32_t*>(a->live);
  p.d_loss = a->d_loss;
  p.d_logits = a->d_logits;
  const unsigned blocks = (unsigned)std::min<int64_t>((a->tokens + 3) / 4, 2048);
  hipStream_t s = (hipStream_t)stream;
  with_type(a->type, [&](auto T) {
    with_lanes(a->experts, [&](auto NE) {
      hipLaunchKernelGGL((balance_slopes<decltype(T)::value, decltype(NE)::value>), dim3(blocks), dim3(256), 0, s, p);
    });
  });
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
