// route.hip -- expert routing: counts, offsets and the row order of the assignments, the balance
// loss and its gradient (htroute.h).
#include <algorithm>

#include "../../include/htroute.h"
#include "arch.h"
#include "kernels.h"

namespace htk {
namespace {

constexpr int kRouteWaves = 16, kRouteChunk = 2048, kRouteBlocks = 256;
constexpr int kLossWaves = 16, kLossBlocks = 256;
constexpr int kFinishExperts = 16;
constexpr int kLossHead = 64 * 8 + 16;   // bytes of dots and ticket before the workgroups' sums

// ---- order ---------------------------------------------------------------------------------
struct RParams {
  const int32_t* ids;
  const uint8_t* mask;
  int64_t ld_ids, rows;
  int n, topk, experts, align;   // n: assignments
  int chunk;                     // assignments per workgroup
  int bits;                      // of an expert's number
  int topk_shift;                // s of expert_of
  uint64_t topk_inverse;         // ceil(2^s / topk)
  int32_t* counts;
  int32_t* offsets;
  int32_t* order;
  int32_t* slot;
  int32_t* hist;                 // gridDim.x x experts
};

// The expert of assignment i, or -1 when it is dropped.  The division is one multiplication:
// floor(i / k) = floor(i * ceil(2^s / k) / 2^s) for i < 2^30 and 2^(s - 30) >= k, since the excess of
// the rounded factor, below i / 2^s < 1 / k, is less than the 1 / k to the next whole number.
__device__ __forceinline__ int expert_of(const RParams& p, int i) {
  const int t = (int)((uint64_t)i * p.topk_inverse >> p.topk_shift);
  if (p.mask && !p.mask[t]) return -1;
  const int e = p.ids[(int64_t)t * p.ld_ids + (i - t * p.topk)];
  return e >= 0 && e < p.experts ? e : -1;
}

// Lanes of the wave that hold the same expert (dropped lanes match nothing of interest).
__device__ __forceinline__ unsigned long long same_expert(int e, int bits) {
  unsigned long long m = ~0ull;
  for (int b = 0; b < bits; ++b) {
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
// and lanes of its wave.  One chunk needs no route_hist.  131072 assignments to 256 experts: 3.5 +
// 11 us, the dependent steps of a wave (histogram loads, two passes over LDS, scattered writes); 2048
// assignments a workgroup and 1024 are alike, 4096 costs 3 us more.
__global__ __launch_bounds__(1024) void route_place(const RParams p) {
  extern __shared__ int sh[];       // [waves][experts] then, for the scan, one int per wave
  __shared__ int sums[kRouteWaves];
  const int E = p.experts, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x, nb = gridDim.x;
  const int64_t begin = (int64_t)b * p.chunk, end = min((int64_t)p.n, begin + p.chunk);
  const int run = (p.chunk + kRouteWaves - 1) / kRouteWaves;
  const int64_t w0 = min(begin + (int64_t)wave * run, end), w1 = min(w0 + run, end);
  // the experts of the wave's first steps stay in registers from the count to the placing
  constexpr int KEPT = kRouteChunk / kRouteWaves / 64;
  int kept[KEPT];
  static_for<KEPT>([&](auto k) {
    const int64_t i = w0 + k * 64 + lane;
    kept[k] = i < w1 ? expert_of(p, (int)i) : -1;
  });
  // thread e: its expert's total and the part in earlier chunks (loads that wait for nothing here)
  int before = 0, count = 0;
  if (tid < E && nb > 1) {
#pragma unroll 16
    for (int c = 0; c < nb; ++c) {
      const int v = p.hist[(int64_t)c * E + tid];
      before += c < b ? v : 0;
      count += v;
    }
  }
  for (int i = tid; i < kRouteWaves * E; i += 1024) sh[i] = 0;
  __syncthreads();
  int* mine = sh + wave * E;
  static_for<KEPT>([&](auto k) {
    if (kept[k] >= 0) atomicAdd(&mine[kept[k]], 1);
  });
  for (int64_t i = w0 + KEPT * 64 + lane; i < w1; i += 64) {
    const int e = expert_of(p, (int)i);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  if (tid < E && nb == 1)
    for (int w = 0; w < kRouteWaves; ++w) count += sh[w * E + tid];
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
  auto place = [&](int64_t i, int e) {
    const unsigned long long same = same_expert(e, p.bits);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int at = -1;
    if (e >= 0) at = next[e] + rank;
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && rank == 0) next[e] = at + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < w1) {
      if (p.slot) p.slot[i] = at;
      if (p.order && at >= 0) p.order[at] = (int)i;
    }
  };
  static_for<KEPT>([&](auto k) { if (w0 + k * 64 < w1) place(w0 + k * 64 + lane, kept[k]); });
  for (int64_t s = w0 + KEPT * 64; s < w1; s += 64) {
    const int64_t i = s + lane;
    place(i, i < w1 ? expert_of(p, (int)i) : -1);
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
  double* dots;        // parts of the loss, one for each kFinishExperts experts
  int32_t* ticket;
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

// Sum / maximum over the lanes of a wave, the same in all: DPP steps within rows of 16 and across
// them leave it in the last lane.
template <bool MAX> __device__ __forceinline__ float wave_all(float v) {
  constexpr int idle = MAX ? (int)0xff800000 : 0;   // -infinity or 0 from lanes that do not exist
  auto step = [&](auto ctrl, auto rows) {
    const float o = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        idle, __builtin_bit_cast(int, v), decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
    v = MAX ? fmaxf(v, o) : v + o;
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});  // row_shr:1
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast:15
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // row_bcast:31
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Rows a wave of balance_sums has in hand at once, so that their loads and reductions overlap.
template <int NE> constexpr int rows_at_once() { return NE >= 16 ? 2 : 4; }

// Softmax of R rows t, t + step, ... below `end`, lane l holding experts l, l + 64, ...; zero in all
// for a row of -infinity and for rows that are masked or past the end.  The
// maximum keeps a NaN out, the sum carries it to every probability.  Returns the rows that count,
// a bit each.
template <int T, int NE, int R>
__device__ __forceinline__ int softmax_rows(const BParams& p, int64_t t, int64_t step, int64_t end, int lane,
                                            float (&v)[R][NE]) {
  bool live[R];
  static_for<R>([&](auto q) {
    const int64_t r = t + q * step;
    live[q] = r < end && (!p.mask || p.mask[r]);
  });
  static_for<R>([&](auto q) {
    const typename Elem<T>::S* x = (const typename Elem<T>::S*)p.logits + (t + q * step) * p.ld;
    static_for<NE>([&](auto i) {
      const int e = lane + 64 * i;
      v[q][i] = t + q * step < end && e < p.experts ? Elem<T>::up(x[e]) : -__builtin_inff();
    });
  });
  // (a masked row's values are loaded beside its mask, not behind it, and dropped)
  static_for<R>([&](auto q) { static_for<NE>([&](auto i) { v[q][i] = live[q] ? v[q][i] : -__builtin_inff(); }); });
  int bits = 0;
  static_for<R>([&](auto q) {
    float top = -__builtin_inff();
    static_for<NE>([&](auto i) { top = fmaxf(top, v[q][i]); });
    top = wave_all<true>(top);
    const float base = top == -__builtin_inff() ? 0.f : top;
    float sum = 0.f;
    static_for<NE>([&](auto i) {
      v[q][i] = expf(v[q][i] - base);
      sum += v[q][i];
    });
    sum = wave_all<false>(sum);
    const float r = sum == 0.f ? 0.f : 1.f / sum;
    static_for<NE>([&](auto i) { v[q][i] *= r; });
    bits |= live[q] ? 1 << q : 0;
  });
  return bits;
}

// loss and live from dot = sum over the experts of mean probability x count and the n rows that count
__device__ __forceinline__ void put_loss(const BParams& p, double dot, int n) {
  *p.loss = n > 0 ? (float)(p.coef * dot * p.experts / ((double)p.topk * n)) : 0.f;
  *p.live = n;
}

// 16384 x 256 fp32: sums 9 us, finish 5 us, slopes 12 us.
//
// Sums of the probabilities over each workgroup's tokens: a wave takes every 16th of them.  Only the
// rows that it has in hand are added in fp32; the rest is double, since a wave's rows have no limit
// (in fp32 4 M equal rows were off by 2^-16) and the rounding of equal rows does not average out.
template <int T, int NE>
__global__ __launch_bounds__(kLossWaves * 64) void balance_sums(const BParams p) {
  extern __shared__ float sums[];   // [waves][experts]
  __shared__ int live[kLossWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = blockIdx.x * p.per, t1 = min(t0 + p.per, p.tokens);
  double acc[NE];
  static_for<NE>([&](auto i) { acc[i] = 0.0; });
  int n = 0;
  constexpr int R = rows_at_once<NE>();
  for (int64_t t = t0 + wave; t < t1; t += R * kLossWaves) {
    float v[R][NE];
    n += __popc(softmax_rows<T, NE, R>(p, t, kLossWaves, t1, lane, v));
    static_for<NE>([&](auto i) {
      float s = v[0][i];
      static_for<R - 1>([&](auto q) { s += v[q + 1][i]; });
      acc[i] += s;
    });
  }
  static_for<NE>([&](auto i) {
    if (lane + 64 * i < p.experts) sums[wave * p.experts + lane + 64 * i] = (float)acc[i];
  });
  if (lane == 0) live[wave] = n;
  __syncthreads();
  static_assert(ROUTE_MAX_EXPERTS <= kLossWaves * 64, "a thread for each expert");
  double s = 0.0;
  if (tid < p.experts) {
    for (int w = 0; w < kLossWaves; ++w) s += sums[w * p.experts + tid];
    if (gridDim.x > 1) p.partial[(int64_t)blockIdx.x * p.experts + tid] = (float)s;
  }
  n = 0;
  for (int w = 0; w < kLossWaves; ++w) n += live[w];
  if (gridDim.x > 1) {
    if (tid == 0) p.partial_n[blockIdx.x] = n;
    if (tid == 0 && blockIdx.x == 0) *p.ticket = 0;
    return;
  }
  // one workgroup has all the sums: finish here
  __shared__ double dots[kLossWaves];
  double dot = 0.0;
  if (tid < p.experts) {
    const double mean = n > 0 ? s / n : 0.0;
    p.prob[tid] = (float)mean;
    dot = mean * p.counts[tid];
  }
  for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
  if (lane == 0) dots[wave] = dot;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kLossWaves; ++w) dot += dots[w];
    put_loss(p, dot, n);
  }
}

// prob and loss from the workgroups' sums, added in a fixed order, in double.  A workgroup takes 16
// experts, so that the sums are read by several (by one: 10 us for 256 KB); thread (g, quad) adds
// four experts of every 64th sum.  The last workgroup to end, by a ticket that balance_sums has set
// to zero, adds the workgroups' parts of the loss, in their order.
__global__ __launch_bounds__(256) void balance_finish(const BParams p, int blocks) {
  __shared__ double part[4][kFinishExperts];
  __shared__ int live[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.experts;
  const int quad = tid & 3, first = blockIdx.x * kFinishExperts, e0 = first + quad * 4;
  int n = tid < blocks ? p.partial_n[tid] : 0;
  const int count = tid < kFinishExperts && first + tid < E ? p.counts[first + tid] : 0;
  f32x4 v[kLossBlocks / 64];
  static_for<kLossBlocks / 64>([&](auto k) {
    const int b = (tid >> 2) + k * 64;
    const float* src = p.partial + (int64_t)b * E + e0;
    v[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (b < blocks) {
      if (E % 4 == 0) {
        if (e0 < E) v[k] = *reinterpret_cast<const f32x4*>(src);
      } else {
        static_for<4>([&](auto i) { if (e0 + i < E) v[k][(int)i] = src[(int)i]; });
      }
    }
  });
  static_for<4>([&](auto i) {
    double s = 0.0;
    static_for<kLossBlocks / 64>([&](auto k) { s += v[k][(int)i]; });
    for (int d = 4; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
    if (lane < 4) part[wave][quad * 4 + i] = s;
  });
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d, 64);
  if (lane == 0) live[wave] = n;
  __syncthreads();
  if (wave != 0) return;
  n = live[0] + live[1] + live[2] + live[3];
  double dot = 0.0;
  if (lane < kFinishExperts && first + lane < E) {
    const double s = part[0][lane] + part[1][lane] + part[2][lane] + part[3][lane];
    const double mean = n > 0 ? s / n : 0.0;
    p.prob[first + lane] = (float)mean;
    dot = mean * count;
  }
  for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
  int last = 0;
  if (lane == 0) {
    __hip_atomic_store(p.dots + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(p.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  }
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  static_assert(ROUTE_MAX_EXPERTS <= 64 * kFinishExperts && kLossBlocks == 256, "a lane for each part");
  dot = lane < (int)gridDim.x ? __hip_atomic_load(p.dots + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
  for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
  if (lane == 0) put_loss(p, dot, n);
}

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
  constexpr int R = 2;   // with 2048 workgroups; half of them and 4 rows a wave: 1 us more
  for (int64_t t = w; t < p.tokens; t += R * waves) {
    float v[R][NE];
    const int live = softmax_rows<T, NE, R>(p, t, waves, p.tokens, lane, v);
    static_for<R>([&](auto q) {
      float s = 0.f;
      static_for<NE>([&](auto i) { s += v[q][i] * g[i]; });
      s = wave_all<false>(s);
      const int64_t r = t + q * waves;
      if (r < p.tokens) {
        typename Elem<T>::S* d = (typename Elem<T>::S*)p.d_logits + r * p.ld_d;
        static_for<NE>([&](auto i) {
          if (lane + 64 * i < p.experts) d[lane + 64 * i] = Elem<T>::down(live >> q & 1 ? v[q][i] * (g[i] - s) : 0.f);
        });
      }
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
  const size_t loss = kLossHead + (size_t)loss_blocks(tokens) * (experts + 1) * 4;
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
  p.bits = 0;
  while ((1 << p.bits) < a->experts) ++p.bits;
  p.topk_shift = 30;
  while ((1 << (p.topk_shift - 30)) < a->topk) ++p.topk_shift;
  p.topk_inverse = ((uint64_t(1) << p.topk_shift) + a->topk - 1) / a->topk;
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
  p.dots = static_cast<double*>(a->workspace);
  p.ticket = reinterpret_cast<int32_t*>(p.dots + 64);
  p.partial = reinterpret_cast<float*>(p.dots + kLossHead / 8);
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
    const unsigned parts = (unsigned)((a->experts + kFinishExperts - 1) / kFinishExperts);
    hipLaunchKernelGGL(balance_finish, dim3(parts), dim3(256), 0, s, p, (int)blocks);
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
