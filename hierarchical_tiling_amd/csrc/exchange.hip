// exchange.hip -- tokens to their experts' rows and back (route_gather, route_combine and
// route_combine_grad of htroute.h).
//
//   gather   y(p) = x(order[p] / k)                            combine  out(t) = add(t) + sum_j w(t, j) y(slot(t, j))
//   d_y(p) = w[order[p]] d_out(order[p] / k)                   d_w(t, j) = <d_out(t), y(slot(t, j))>
//
// All are bound by memory: rows of 16-byte pieces, at any alignment.  What goes from tokens to rows
// is done token by token, so that a token is read once for its k rows; order decides who owns a row:
// row p belongs to the token pass if slot[order[p]] == p, and otherwise (rows of no assignment, or
// a slot that is not order's inverse) to the row pass, workgroups of the same launch.  Every row is
// written once whatever order and slot hold.
#include <algorithm>

#include "../../include/htroute.h"
#include "arch.h"
#include "kernels.h"

namespace htk {
namespace {

struct XParams {
  const void* x;            // tokens x cols: gather's x, the gradient's d_out
  void* y;                  // rows x cols: gather's y, the gradient's d_y
  const void* rows_in;      // rows x cols: combine's and the gradient's y
  const void* add;
  void* out;
  void* d_w;
  const void* w;
  const int32_t* order;
  const int32_t* slot;
  int64_t tokens, rows, ldx, ldy, ld_in, ld_add, ld_out;
  int64_t token_blocks;     // workgroups of the token pass
  int cols, topk, assignments, row_group;
  int w_type;
};

// 16-bit and 32-bit elements: VE to a 16-byte piece.
template <int XT> struct El {
  typedef u16 T;
  static constexpr int VE = 8;
  __device__ static float up(T v) { return XT == DT_BF16 ? bf16_to_f32(v) : f16_to_f32(v); }
  __device__ static T down(float v) { return XT == DT_BF16 ? f32_to_bf16(v) : f32_to_f16(v); }
};
template <> struct El<DT_F32> {
  typedef float T;
  static constexpr int VE = 4;
  __device__ static float up(T v) { return v; }
  __device__ static T down(float v) { return v; }
};

__device__ __forceinline__ float weight(const XParams& p, int a) {
  return p.w_type == DT_F32 ? ((const float*)p.w)[a] : p.w_type == DT_BF16 ? bf16_to_f32(((const u16*)p.w)[a])
                                                                         : f16_to_f32(((const u16*)p.w)[a]);
}
__device__ __forceinline__ void store_weight(const XParams& p, int a, float v) {
  if (p.w_type == DT_F32) ((float*)p.d_w)[a] = v;
  else ((u16*)p.d_w)[a] = p.w_type == DT_BF16 ? f32_to_bf16(v) : f32_to_f16(v);
}

// A thread's piece of a row of `cols` elements: VE elements from `at` on, of which those from `first`
// on are its own.  The piece that the row's end cuts is the row's last VE elements, so that it too is
// one load; the elements before `first` are the piece's before, and are not stored.  Rows of
// less than VE elements are pieces of `n` elements.
template <int VE> struct Piece {
  int at, first, n;
  __device__ __forceinline__ Piece(int c, int cols) {
    at = c + VE <= cols ? c : max(cols - VE, 0);
    first = c - at;
    n = min(VE, cols);
  }
};
// Rows are not kept in the caches: what is stored, and the rows that combine and its gradient read.
// Stores that stay in an L2 are written back when the kernel ends, rows scattered over 1.1 GB at half the
// rate: gather 217 us with streamed stores, 381 without (16384 tokens of 4096 to 8 of 256), and 16
// tokens there and back 12.2 and 19.1 us; no size from 1 MB to 1 GB was better without.  So with rows on 16
// bytes.  Of other rows a line is stored in two parts, which meet in an L2 only if they stay there: gather
// does not stream them (8192 tokens of 4099 bf16 to 8: 137 us, streamed 162; of 2050 62 and 83; 16384 of
// 4098 to 2, alone in losing, 83 and 71).  The gradient loses by it as often as it gains, and streams.
typedef u32x4 piece_t __attribute__((aligned(2)));
template <class T, int VE, bool STREAM = false>
__device__ __forceinline__ void load_piece(const T* row, const Piece<VE>& q, T (&e)[VE]) {
  if (q.n == VE) {
    u32x4 w;
    if constexpr (STREAM) w = __builtin_nontemporal_load(reinterpret_cast<const piece_t*>(row + q.at));
    else w = *reinterpret_cast<const piece_t*>(row + q.at);
    __builtin_memcpy(e, &w, 16);
  } else {
    static_for<VE>([&](auto i) { e[i] = i < q.n ? row[(int)i] : T(0); });
  }
}
// OVERLAP: the piece that the row's end cuts is stored whole, its first elements a second time with the
// same values; not where they may have been read before (out that is add).
template <class T, int VE, bool OVERLAP = false, bool STREAM = true>
__device__ __forceinline__ void store_piece(T* row, const Piece<VE>& q, const T (&e)[VE]) {
  if ((OVERLAP || q.first == 0) && q.n == VE) {
    u32x4 w;
    __builtin_memcpy(&w, e, 16);
    if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<piece_t*>(row + q.at));
    else *reinterpret_cast<piece_t*>(row + q.at) = w;
  } else {
    static_for<VE>([&](auto i) {
      if (i >= q.first && i < q.n) __builtin_nontemporal_store(e[i], row + q.at + i);
    });
  }
}

// The token of a thread, tpt threads (whole waves) for each.
__device__ __forceinline__ int64_t token_of(int tpt) {
  return (int64_t)blockIdx.x * (blockDim.x / tpt) + __builtin_amdgcn_readfirstlane((int)threadIdx.x / tpt);
}

// Assignment j of token t: lane j holds its slot, -1 where there is none.
__device__ __forceinline__ int lane_slot(const XParams& p, int64_t t) {
  const int j = threadIdx.x & 63;
  const int s = j < p.topk ? p.slot[t * p.topk + j] : -1;
  return s < p.rows ? s : -1;     // (negative ones stay)
}

// The row pass: row_group rows a wave.  write(p, a) for the rows that no token owns and that order
// gives an assignment a; the others become zeros.
template <class T, class F> __device__ __forceinline__ void rows_left(const XParams& p, F write) {
  const int lane = threadIdx.x & 63;
  const int64_t r0 = (((int64_t)blockIdx.x - p.token_blocks) * (blockDim.x >> 6) + (threadIdx.x >> 6)) * p.row_group;
  const int64_t r = r0 + lane;
  bool mine = lane < p.row_group && r < p.rows;
  int a = -1;
  if (mine) {
    a = p.order[r];
    if (a < 0 || a >= p.assignments) a = -1;
    else if (p.slot && p.slot[a] == r) mine = false;
  }
  constexpr int VE = 16 / (int)sizeof(T);
  for (unsigned long long todo = __ballot(mine && a < 0); todo; todo &= todo - 1) {
    T* y = (T*)p.y + (r0 + __ffsll(todo) - 1) * p.ldy;
    T zero[VE] = {};
    for (int c = lane * VE; c < p.cols; c += 64 * VE) store_piece<T, VE, true>(y, Piece<VE>(c, p.cols), zero);
  }
  for (unsigned long long todo = __ballot(mine && a >= 0); todo; todo &= todo - 1) {
    const int l = __ffsll(todo) - 1;
    write(r0 + l, __builtin_amdgcn_readlane(a, l));
  }
}

template <class T> __device__ __forceinline__ const T* row_at(const void* base, int64_t r, int64_t ld) {
  return (const T*)base + r * ld;
}

// ---- gather --------------------------------------------------------------------------------
// Elements are moved, not looked at: XT is DT_F32 or a 16-bit type.  STREAM: y's rows lie on 16 bytes.
template <int XT, bool STREAM>
__global__ __launch_bounds__(1024) void gather_rows(const XParams p, int tpt) {
  typedef typename El<XT>::T T;
  constexpr int VE = El<XT>::VE, U = 2;
  const int lane = threadIdx.x & 63;
  if ((int64_t)blockIdx.x >= p.token_blocks) {
    rows_left<T>(p, [&](int64_t r, int a) {
      T* y = (T*)p.y + r * p.ldy;
      const T* x = row_at<T>(p.x, a / p.topk, p.ldx);
      for (int c = lane * VE; c < p.cols; c += 64 * VE) {
        const Piece<VE> q(c, p.cols);
        alignas(16) T e[VE];
        load_piece<T, VE>(x, q, e);
        store_piece<T, VE, true, STREAM>(y, q, e);
      }
    });
    return;
  }
  const int64_t t = token_of(tpt);
  if (t >= p.tokens) return;
  const T* x = row_at<T>(p.x, t, p.ldx);
  const int tid = threadIdx.x % tpt;
  alignas(16) T e[U][VE];
  auto load = [&](int c0) {
    static_for<U>([&](auto u) {
      const int c = c0 + (u * tpt + tid) * VE;
      if (c < p.cols) load_piece<T, VE>(x, Piece<VE>(c, p.cols), e[u]);
    });
  };
  load(0);                      // on its way while the slots and the order are looked at
  int s = lane_slot(p, t);
  if (s >= 0 && p.order[s] != t * p.topk + lane) s = -1;     // another's row
  const unsigned long long live = __ballot(s >= 0);
  if (!live) return;
  for (int c0 = 0; c0 < p.cols; c0 += tpt * VE * U) {
    if (c0 > 0) load(c0);
    for (unsigned long long todo = live; todo; todo &= todo - 1) {
      T* y = (T*)p.y + (int64_t)__builtin_amdgcn_readlane(s, __ffsll(todo) - 1) * p.ldy;
      static_for<U>([&](auto u) {
        const int c = c0 + (u * tpt + tid) * VE;
        if (c < p.cols) store_piece<T, VE, true, STREAM>(y, Piece<VE>(c, p.cols), e[u]);
      });
    }
  }
}

// ---- combine -------------------------------------------------------------------------------
// B terms of a piece, whose loads are all issued before one is used.
template <int XT, int B, bool W>
__device__ __forceinline__ void add_terms(const XParams& p, int s, float w, unsigned long long& todo,
                                          const Piece<El<XT>::VE>& q, float (&sum)[El<XT>::VE]) {
  typedef typename El<XT>::T T;
  constexpr int VE = El<XT>::VE;
  alignas(16) T e[B][VE];
  float f[B];
  static_for<B>([&](auto b) {
    const int j = __ffsll(todo) - 1;
    todo &= todo - 1;
    load_piece<T, VE, true>(row_at<T>(p.rows_in, __builtin_amdgcn_readlane(s, j), p.ld_in), q, e[b]);
    if constexpr (W) f[b] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), j));
  });
  static_for<B>([&](auto b) {
    static_for<VE>([&](auto i) {
      const float v = El<XT>::up(e[b][i]);
      sum[i] = W ? __builtin_fmaf(f[b], v, sum[i]) : sum[i] + v;
    });
  });
}

template <int XT, bool W>
__global__ __launch_bounds__(1024) void combine_rows(const XParams p, int tpt) {
  typedef typename El<XT>::T T;
  constexpr int VE = El<XT>::VE;
  const int64_t t = token_of(tpt);
  if (t >= p.tokens) return;
  const int lane = threadIdx.x & 63, s = lane_slot(p, t);
  const float w = W && s >= 0 ? weight(p, (int)t * p.topk + lane) : 0.f;
  const unsigned long long live = __ballot(s >= 0);
  for (int c = (int)(threadIdx.x % tpt) * VE; c < p.cols; c += tpt * VE) {
    const Piece<VE> q(c, p.cols);
    float sum[VE];
    static_for<VE>([&](auto i) { sum[i] = 0.f; });
    alignas(16) T e[VE];
    if (p.add) load_piece<T, VE>(row_at<T>(p.add, t, p.ld_add), q, e);
    if (p.add) static_for<VE>([&](auto i) { sum[i] = El<XT>::up(e[i]); });
    unsigned long long todo = live;
    int n = __popcll(live);
    for (; n >= 8; n -= 8) add_terms<XT, 8, W>(p, s, w, todo, q, sum);
    if (n >= 4) { add_terms<XT, 4, W>(p, s, w, todo, q, sum); n -= 4; }
    if (n >= 2) { add_terms<XT, 2, W>(p, s, w, todo, q, sum); n -= 2; }
    if (n >= 1) add_terms<XT, 1, W>(p, s, w, todo, q, sum);
    static_for<VE>([&](auto i) { e[i] = El<XT>::down(sum[i]); });
    store_piece<T, VE>((T*)p.out + t * p.ld_out, q, e);
  }
}

// ---- gradients of combine ------------------------------------------------------------------
// Sum over the wave, in lane 63.
__device__ __forceinline__ float wave_sum(float v) {
  auto step = [&](auto ctrl, auto rows) {
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value,
                                                               decltype(rows)::value, 0xf, false));
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});  // row_shr:1, 2, 4, 8
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast:15, 31
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
  return v;
}

// B assignments of a token: their rows of d_y, and their dots with d_out.  own: the lanes (assignments)
// whose row of d_y this token writes; those without a slot are not in `todo`.
template <int XT, int B, bool DY, bool DW>
__device__ __forceinline__ void grad_terms(const XParams& p, const typename El<XT>::T* d_out, int s, float w,
                                           unsigned long long own, unsigned long long& todo, int tid, int tpt,
                                           float* sums) {
  typedef typename El<XT>::T T;
  constexpr int VE = El<XT>::VE;
  int j[B], at[B];
  float f[B], dot[B];
  static_for<B>([&](auto b) {
    j[b] = __ffsll(todo) - 1;
    todo &= todo - 1;
    at[b] = __builtin_amdgcn_readlane(s, j[b]);
    f[b] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), j[b]));
    dot[b] = 0.f;
  });
  for (int c = tid * VE; c < p.cols; c += tpt * VE) {
    const Piece<VE> q(c, p.cols);
    alignas(16) T d[VE], e[DW ? B : 1][VE];
    load_piece<T, VE>(d_out, q, d);
    if constexpr (DW) static_for<B>([&](auto b) { load_piece<T, VE, true>(row_at<T>(p.rows_in, at[b], p.ld_in), q, e[b]); });
    float v[VE];
    static_for<VE>([&](auto i) { v[i] = El<XT>::up(d[i]); });
    if constexpr (DY) {
      static_for<B>([&](auto b) {
        if (own >> j[b] & 1) {
          alignas(16) T o[VE];
          static_for<VE>([&](auto i) { o[i] = El<XT>::down(f[b] * v[i]); });
          store_piece<T, VE, true>((T*)p.y + (int64_t)at[b] * p.ldy, q, o);
        }
      });
    }
    if constexpr (DW) {
      static_for<VE>([&](auto i) {
        if (i < q.first || i >= q.n) v[i] = 0.f;          // another piece's, or past the row
      });
      static_for<B>([&](auto b) {
        static_for<VE>([&](auto i) {
          const float y = i >= q.first && i < q.n ? El<XT>::up(e[b][i]) : 0.f;
          dot[b] = __builtin_fmaf(v[i], y, dot[b]);
        });
      });
    }
  }
  if constexpr (DW) {
    static_for<B>([&](auto b) {
      const float v = wave_sum(dot[b]);
      if ((tid & 63) == 63) sums[j[b]] = v;
    });
  }
}

template <int XT, bool DY, bool DW>
__global__ __launch_bounds__(1024) void combine_rows_grad(const XParams p, int tpt) {
  typedef typename El<XT>::T T;
  constexpr int VE = El<XT>::VE;
  __shared__ float sums[16][64];         // of each wave, by assignment
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int64_t)blockIdx.x >= p.token_blocks) {
    rows_left<T>(p, [&](int64_t r, int a) {
      T* y = (T*)p.y + r * p.ldy;
      const T* d = row_at<T>(p.x, a / p.topk, p.ldx);
      const float f = weight(p, a);
      for (int c = lane * VE; c < p.cols; c += 64 * VE) {
        const Piece<VE> q(c, p.cols);
        alignas(16) T e[VE];
        load_piece<T, VE>(d, q, e);
        static_for<VE>([&](auto i) { e[i] = El<XT>::down(f * El<XT>::up(e[i])); });
        store_piece<T, VE, true>(y, q, e);
      }
    });
    return;
  }
  const int64_t t = token_of(tpt);
  const bool in = t < p.tokens;
  const int tid = threadIdx.x % tpt, s = in ? lane_slot(p, t) : -1, a = (int)t * p.topk + lane;
  if (in) {
    const float w = DY && s >= 0 ? weight(p, a) : 0.f;
    const unsigned long long own = DY ? __ballot(s >= 0 && p.order[max(s, 0)] == a) : 0;
    unsigned long long todo = DW ? __ballot(s >= 0) : own;
    int n = __popcll(todo);
    const T* d_out = row_at<T>(p.x, t, p.ldx);
    for (; n >= 8; n -= 8) grad_terms<XT, 8, DY, DW>(p, d_out, s, w, own, todo, tid, tpt, sums[wave]);
    if (n >= 4) { grad_terms<XT, 4, DY, DW>(p, d_out, s, w, own, todo, tid, tpt, sums[wave]); n -= 4; }
    if (n >= 2) { grad_terms<XT, 2, DY, DW>(p, d_out, s, w, own, todo, tid, tpt, sums[wave]); n -= 2; }
    if (n >= 1) grad_terms<XT, 1, DY, DW>(p, d_out, s, w, own, todo, tid, tpt, sums[wave]);
  }
  if constexpr (DW) {
    __syncthreads();
    if (in && tid < p.topk) {           // (tid < 64: lane == tid) the token's waves, in order
      float v = 0.f;
      if (s >= 0)
        for (int k = 0; k < tpt / 64; ++k) v += sums[wave + k][tid];
      store_weight(p, a, v);
    }
  }
}

// ---- launch --------------------------------------------------------------------------------
// Sizes that all three share.  Assignments and rows are 32-bit numbers, and a launch has fewer than
// 2^32 threads: up to 2^31 for the tokens, and a wave for each 4 rows (2^30).
constexpr int64_t kMostTokens = int64_t(1) << 23, kMostRows = int64_t(1) << 26, kMostCols = int64_t(1) << 24;
constexpr int64_t kMostThreads = int64_t(1) << 31;

struct Shape {
  int tpt, threads;         // threads for each token, and of a workgroup
  int64_t token_blocks, row_blocks;
  int row_group;
};
// Threads for each token: one for each piece, a wave at least and `most` threads at most.  Combine takes
// up to 1024 (16384 x 4096 bf16 196 us, with two pieces a thread 204; 500 x 7000 f32 14 and 23), gather
// 1024 for up to 256 tokens, when its chain of loads and stores counts (37 x 2051 f16 3.8 us, with 256
// threads 7.6), and 256 for more (300 x 4096 5.0 us, with 1024 5.6; 500 x 7000 f32 15.3 and 17.5).  The
// gradient, which joins its threads' sums, takes 1024 for up to 1024 tokens and 256 for more: 500 x 7000
// f32 31 us and 38, 16384 x 2048 f32 219 and 210.  The row pass looks at 4 rows a wave, at 1 while that
// makes few workgroups.
Shape shape_of(int64_t tokens, int64_t rows, int64_t cols, int ve, int most) {
  const int64_t pieces = (cols + ve - 1) / ve;
  Shape s;
  s.tpt = 64;
  while (s.tpt < pieces && s.tpt < most && tokens * s.tpt < kMostThreads / 2) s.tpt *= 2;
  s.threads = std::max(s.tpt, 256);
  s.token_blocks = (tokens * s.tpt + s.threads - 1) / s.threads;
  s.row_group = rows <= 4096 ? 1 : 4;
  const int64_t per = s.threads / 64 * s.row_group;
  s.row_blocks = (rows + per - 1) / per;
  return s;
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool known(int type) { return type == GEMM_F32 || type == GEMM_F16 || type == GEMM_BF16; }
int size_of(int type) { return type == GEMM_F32 ? 4 : 2; }

int check(int64_t tokens, int64_t rows, int64_t cols, int topk, int type) {
  if (tokens < 0 || rows < 0 || cols < 0 || tokens > kMostTokens || rows > kMostRows || cols > kMostCols)
    return GEMM_ERR_INVALID_ARG;
  if (topk < 1 || topk > ROUTE_MAX_TOPK) return GEMM_ERR_INVALID_ARG;
  if (!known(type)) return GEMM_ERR_DTYPE_COMBO;
  return GEMM_OK;
}

}  // namespace
}  // namespace htk

using namespace htk;

extern "C" {

int route_gather(const gather_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  int rc = check(a->tokens, a->rows, a->cols, a->topk, a->type);
  if (rc) return rc;
  if (a->ldx < a->cols || a->ldy < a->cols) return GEMM_ERR_LAYOUT;
  const int size = size_of(a->type);
  if (!on(a->x, size) || !on(a->y, size) || !on(a->order, 4) || !on(a->slot, 4)) return GEMM_ERR_MISALIGNED;
  const bool any = a->rows > 0 && a->cols > 0;
  if (any && (!a->y || !a->order || (a->tokens > 0 && !a->x))) return GEMM_ERR_INVALID_ARG;
  rc = arch_status();
  if (rc) return rc;
  if (!any) return GEMM_OK;
  XParams p = {};
  p.x = a->x;
  p.y = a->y;
  p.order = a->order;
  p.slot = a->slot;
  p.tokens = a->tokens;
  p.rows = a->rows;
  p.ldx = a->ldx;
  p.ldy = a->ldy;
  p.cols = (int)a->cols;
  p.topk = a->topk;
  p.assignments = (int)(a->tokens * a->topk);
  const Shape h = shape_of(a->tokens, a->rows, a->cols, 16 / size, a->tokens <= 256 ? 1024 : 256);
  p.token_blocks = a->slot ? h.token_blocks : 0;
  p.row_group = h.row_group;
  const dim3 grid((unsigned)(p.token_blocks + h.row_blocks)), block(h.threads);
  hipStream_t s = (hipStream_t)stream;
  auto go = [&](auto xt) {
    constexpr int XT = decltype(xt)::value;
    if (on(a->y, 16) && a->ldy * size % 16 == 0) hipLaunchKernelGGL((gather_rows<XT, true>), grid, block, 0, s, p, h.tpt);
    else hipLaunchKernelGGL((gather_rows<XT, false>), grid, block, 0, s, p, h.tpt);
  };
  if (a->type == GEMM_F32) go(std::integral_constant<int, DT_F32>{});
  else go(std::integral_constant<int, DT_BF16>{});
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int route_combine(const combine_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  int rc = check(a->tokens, a->rows, a->cols, a->topk, a->type);
  if (rc) return rc;
  if (a->weights && !known(a->weight_type)) return GEMM_ERR_DTYPE_COMBO;
  if (a->ldy < a->cols || a->ld_out < a->cols || (a->add && a->ld_add < a->cols)) return GEMM_ERR_LAYOUT;
  const int size = size_of(a->type);
  if (!on(a->y, size) || !on(a->out, size) || !on(a->add, size) || !on(a->slot, 4) ||
      (a->weights && !on(a->weights, size_of(a->weight_type))))
    return GEMM_ERR_MISALIGNED;
  const bool any = a->tokens > 0 && a->cols > 0;
  if (any && (!a->out || !a->slot || (a->rows > 0 && !a->y))) return GEMM_ERR_INVALID_ARG;
  rc = arch_status();
  if (rc) return rc;
  if (!any) return GEMM_OK;
  XParams p = {};
  p.rows_in = a->y;
  p.add = a->add;
  p.out = a->out;
  p.w = a->weights;
  p.w_type = a->weight_type;
  p.slot = a->slot;
  p.tokens = a->tokens;
  p.rows = a->rows;
  p.ld_in = a->ldy;
  p.ld_add = a->ld_add;
  p.ld_out = a->ld_out;
  p.cols = (int)a->cols;
  p.topk = a->topk;
  const Shape h = shape_of(a->tokens, 0, a->cols, 16 / size, 1024);
  const dim3 grid((unsigned)h.token_blocks), block(h.threads);
  hipStream_t s = (hipStream_t)stream;
  auto go = [&](auto xt) {
    if (a->weights) hipLaunchKernelGGL((combine_rows<decltype(xt)::value, true>), grid, block, 0, s, p, h.tpt);
    else hipLaunchKernelGGL((combine_rows<decltype(xt)::value, false>), grid, block, 0, s, p, h.tpt);
  };
  if (a->type == GEMM_F32) go(std::integral_constant<int, DT_F32>{});
  else if (a->type == GEMM_F16) go(std::integral_constant<int, DT_F16>{});
  else go(std::integral_constant<int, DT_BF16>{});
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int route_combine_grad(const combine_grad_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  int rc = check(a->tokens, a->rows, a->cols, a->topk, a->type);
  if (rc) return rc;
  if (!known(a->weight_type)) return GEMM_ERR_DTYPE_COMBO;
  if (a->ld_out < a->cols || (a->d_weights && a->ldy < a->cols) || (a->d_y && a->ld_dy < a->cols)) return GEMM_ERR_LAYOUT;
  const int size = size_of(a->type), ws = size_of(a->weight_type);
  if (!on(a->d_out, size) || !on(a->y, size) || !on(a->d_y, size) || !on(a->order, 4) || !on(a->slot, 4) ||
      !on(a->weights, ws) || !on(a->d_weights, ws))
    return GEMM_ERR_MISALIGNED;
  const bool dy = a->d_y && a->rows > 0 && a->cols > 0, dw = a->d_weights && a->tokens > 0;
  if (dy && (!a->order || (a->tokens > 0 && (!a->slot || !a->weights || !a->d_out)))) return GEMM_ERR_INVALID_ARG;
  if (dw && (!a->slot || (a->cols > 0 && (!a->d_out || (a->rows > 0 && !a->y))))) return GEMM_ERR_INVALID_ARG;
  if (!a->d_y && !a->d_weights && a->tokens > 0 && a->rows > 0 && a->cols > 0) return GEMM_ERR_INVALID_ARG;
  rc = arch_status();
  if (rc) return rc;
  if (!dy && !dw) return GEMM_OK;
  XParams p = {};
  p.x = a->d_out;
  p.y = a->d_y;
  p.rows_in = a->y;
  p.w = a->weights;
  p.w_type = a->weight_type;
  p.d_w = a->d_weights;
  p.order = a->order;
  p.slot = a->slot;
  p.tokens = a->tokens;
  p.rows = a->rows;
  p.ldx = a->ld_out;
  p.ldy = a->ld_dy;
  p.ld_in = a->ldy;
  p.cols = (int)a->cols;
  p.topk = a->topk;
  p.assignments = (int)(a->tokens * a->topk);
  const Shape h = shape_of(a->tokens, a->rows, a->cols, 16 / size, a->tokens <= 1024 ? 1024 : 256);
  p.token_blocks = h.token_blocks;
  p.row_group = h.row_group;
  const dim3 grid((unsigned)(h.token_blocks + (dy ? h.row_blocks : 0))), block(h.threads);
  hipStream_t s = (hipStream_t)stream;
  auto go = [&](auto xt) {
    constexpr int XT = decltype(xt)::value;
    if (dy && dw) hipLaunchKernelGGL((combine_rows_grad<XT, true, true>), grid, block, 0, s, p, h.tpt);
    else if (dy) hipLaunchKernelGGL((combine_rows_grad<XT, true, false>), grid, block, 0, s, p, h.tpt);
    else hipLaunchKernelGGL((combine_rows_grad<XT, false, true>), grid, block, 0, s, p, h.tpt);
  };
  if (a->type == GEMM_F32) go(std::integral_constant<int, DT_F32>{});
  else if (a->type == GEMM_F16) go(std::integral_constant<int, DT_F16>{});
  else go(std::integral_constant<int, DT_BF16>{});
  return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
