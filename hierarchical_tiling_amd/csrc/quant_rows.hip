// quant_rows.hip -- quantisation of rows to 8-bit integers (quant_rows of htint8.h).
//
//   t = max(largest |x|, 127 * 2^-126),  scale = t / 127,  q = clamp(rint(x * (127 / t)), -127, 127)
//
// A row is read once and kept in registers between the maximum and the conversion.  Bound by
// memory: 16384 x 8192 bf16 66 us, 6.1 TB/s (a copy reaches 5.0, a kernel that only reads 6.3).  Codes
// are stored past the caches (16384 x 8192 75 -> 70 us, 20000 x 2048 26 -> 20; small ones are alike).
#include <algorithm>

#include "../../include/htint8.h"
#include "arch.h"
#include "kernels.h"

namespace htk {
namespace {

struct QRParams {
  const void* x;
  const void* gate;
  const int32_t* index;
  u8* q;
  float* scale;
  int64_t rows, ldx, ldg, x_rows, ldq;
  int cols, q_cols;         // q_cols: written columns, zeros past the data
  int index_div, act;
};

template <int XT> struct RowType;
template <> struct RowType<DT_F32> {
  typedef float T;
  __device__ static float up(float v) { return v; }
};
template <> struct RowType<DT_BF16> {
  typedef u16 T;
  __device__ static float up(u16 v) { return bf16_to_f32(v); }
};
template <> struct RowType<DT_F16> {
  typedef u16 T;
  __device__ static float up(u16 v) { return f16_to_f32(v); }
};

// Columns c .. c + 7 of a row as fp32, zero past its end.  The loads of a chunk that a row ends in have
// clamped addresses; 16-byte loads go at any alignment.
typedef u32x4 piece_t __attribute__((aligned(2)));
typedef uint64_t codes_t __attribute__((aligned(1)));
template <int XT, bool STREAM> __device__ __forceinline__ void row8(const void* row, int c, int cols, float (&v)[8]) {
  typedef typename RowType<XT>::T T;
  const T* src = (const T*)row;
  if (c + 8 <= cols) {
    alignas(16) T e[8];
    const piece_t* from = reinterpret_cast<const piece_t*>(src + c);
    static_for<(int)sizeof(e) / 16>([&](auto h) {
      const u32x4 w = STREAM ? (u32x4)__builtin_nontemporal_load(from + h) : (u32x4)from[(int)h];
      __builtin_memcpy(reinterpret_cast<char*>(e) + 16 * h, &w, 16);
    });
    static_for<8>([&](auto i) { v[i] = RowType<XT>::up(e[i]); });
  } else if (c < cols) {
    T e[8];
    static_for<8>([&](auto i) { e[i] = src[min(c + i, cols - 1)]; });
    static_for<8>([&](auto i) { v[i] = c + i < cols ? RowType<XT>::up(e[i]) : 0.f; });
  } else {
    static_for<8>([&](auto i) { v[i] = 0.f; });
  }
}

template <int XT, bool GATE, bool STREAM>
__device__ __forceinline__ void values8(const QRParams& p, const void* x, const void* gate, int c, float (&v)[8]) {
  row8<XT, STREAM>(x, c, p.cols, v);
  if constexpr (GATE) {
    float g[8];
    row8<XT, STREAM>(gate, c, p.cols, g);
    static_for<8>([&](auto i) { v[i] = c + i < p.cols ? activate(p.act, g[i]) * v[i] : 0.f; });
  }
}

// |x| as an integer: ordered as the magnitudes are, with infinity and then NaN above all.
__device__ __forceinline__ u32 magnitude(const float (&v)[8], u32 m) {
  static_for<8>([&](auto i) { m = max(m, __builtin_bit_cast(u32, v[i]) & 0x7fffffffu); });
  return m;
}

// Maximum over the wave, in every lane.
__device__ __forceinline__ u32 wave_max(u32 v) {
  auto step = [&](auto ctrl, auto rows) {
    v = max(v, (u32)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});  // row_shr:1, 2, 4, 8
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast:15, 31
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
  return (u32)__builtin_amdgcn_readlane((int)v, 63);
}

// Four codes.  The product is rounded to fp32 before it is rounded to a whole number: adding 1.5 * 2^23
// does that to the nearest with ties to even and leaves the number in the low byte.
__device__ __forceinline__ u32 codes4(float a, float b, float c, float d, float inverse) {
#pragma clang fp contract(off)
  auto one = [&](float v) {
#pragma clang fp contract(off)
    const float t = __builtin_amdgcn_fmed3f(v * inverse, -127.f, 127.f);
    return __builtin_bit_cast(u32, t + 12582912.f) & 0xffu;
  };
  return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
}

__device__ __forceinline__ void store8(const QRParams& p, u8* q, int c, const float (&v)[8], float inverse, bool bad) {
  if (c >= p.q_cols) return;
  uint64_t w = (uint64_t)codes4(v[4], v[5], v[6], v[7], inverse) << 32 | codes4(v[0], v[1], v[2], v[3], inverse);
  if (bad) w = 0;
  if (c + 8 <= p.q_cols) {
    __builtin_nontemporal_store(w, reinterpret_cast<codes_t*>(q + c));
  } else {
    const int n = p.q_cols - c;
#pragma unroll 1
    for (int i = 0; i < n; ++i, w >>= 8) q[c + i] = (u8)w;
  }
}

// TPR threads take a row, NC pieces of 8 columns each (TPR * 8 columns apart); rows of more than
// TPR * NC * 8 columns (LONG) are read a second time for the conversion.
template <int XT, bool GATE, bool STREAM, int TPR, int NC, bool LONG>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rows_to_int8(const QRParams p) {
  constexpr int PER = TPR < 256 ? 256 / TPR : 1, NW = TPR / 64;
  __shared__ u32 tops[NW > 1 ? NW : 1];
  const int tid = threadIdx.x % TPR;
  const int64_t r = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * PER +
                    (PER > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR) : 0);
  if (r >= p.rows) return;
  int64_t from = r;
  if (p.index) {
    const int at = p.index[r];
    from = at < 0 ? -1 : p.index_div == 1 ? at : (int)((u32)at / (u32)p.index_div);
    if (from >= p.x_rows) from = -1;
  }
  typedef typename RowType<XT>::T T;
  const T* x = (const T*)p.x + max(from, (int64_t)0) * p.ldx;
  const T* gate = (const T*)p.gate + max(from, (int64_t)0) * p.ldg;
  float v[NC][8];
  u32 top = 0;
  static_for<NC>([&](auto k) { static_for<8>([&](auto i) { v[k][i] = 0.f; }); });
  if (from >= 0) {
    static_for<NC>([&](auto k) { values8<XT, GATE, STREAM>(p, x, gate, (k * TPR + tid) * 8, v[k]); });
    static_for<NC>([&](auto k) { top = magnitude(v[k], top); });
    if constexpr (LONG) {
      for (int c = (NC * TPR + tid) * 8; c < p.cols; c += TPR * 8) {
        float w[8];
        values8<XT, GATE, STREAM>(p, x, gate, c, w);
        top = magnitude(w, top);
      }
    }
  }
  top = wave_max(top);
  if constexpr (NW > 1) {
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
    u32 m = tops[tid % NW];     // every wave takes the maximum of the NW entries
    static_for<NW == 4 ? 2 : 4>([&](auto d) { m = max(m, (u32)__shfl_xor((int)m, 1 << d, 64)); });
    top = m;
  }
  const bool bad = top >= 0x7f800000u;
  const float t = fmaxf(__builtin_bit_cast(float, bad ? 0u : top), 127.f * 0x1p-126f);
  const float inverse = 127.f / t;
  if (tid == 0) p.scale[r] = bad ? __builtin_nanf("") : t / 127.f;
  u8* q = p.q + r * p.ldq;
  static_for<NC>([&](auto k) { store8(p, q, (k * TPR + tid) * 8, v[k], inverse, bad); });
  if constexpr (LONG) {
    for (int c = (NC * TPR + tid) * 8; c < p.q_cols; c += TPR * 8) {
      float w[8];
      static_for<8>([&](auto i) { w[i] = 0.f; });
      if (from >= 0) values8<XT, GATE, STREAM>(p, x, gate, c, w);
      store8(p, q, c, w, inverse, bad);
    }
  }
}

// A dimension of a launch has fewer than 2^32 threads: the workgroups are dealt over two dimensions.
constexpr int64_t kMostX = int64_t(1) << 21;
dim3 grid_of(int64_t blocks) {
  const int64_t x = std::min(blocks, kMostX);
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

// Threads for each row: a wave for short rows, a workgroup for longer ones, and more of them while there
// are too few rows to fill the card (480 x 2048 with 256 threads a row 2.8 us, a wave 3.4, gated 3.6 and
// 6.7; 4096 x 2048 6.5 and 6.0; 1 x 8192 with 1024 threads 2.6, 256 3.1; 2000 x 8192 10.8 and 9.4).
// Few rows, and rows that are read twice, are not streamed (below).
constexpr int kHeld = 1024 * 4 * 8;      // columns that a workgroup holds; rows of more are read twice
template <int XT, bool GATE, bool STREAM> hipError_t launch(const QRParams& p, hipStream_t s) {
  auto go = [&](auto kernel, int tpr) {
    const int per = tpr < 256 ? 256 / tpr : 1;
    hipLaunchKernelGGL(kernel, grid_of((p.rows + per - 1) / per), dim3(tpr < 256 ? 256 : tpr), 0, s, p);
  };
  const int n = p.q_cols;
  if (n <= 512) go(rows_to_int8<XT, GATE, STREAM, 64, 1, false>, 64);
  else if (n <= 2048 && p.rows <= 1024) go(rows_to_int8<XT, GATE, false, 256, 1, false>, 256);
  else if (n <= 1024) go(rows_to_int8<XT, GATE, STREAM, 64, 2, false>, 64);
  else if (n <= 2048) go(rows_to_int8<XT, GATE, STREAM, 64, 4, false>, 64);
  else if (n <= 4096) go(rows_to_int8<XT, GATE, STREAM, 256, 2, false>, 256);
  else if (n <= 8192 && p.rows <= 256) go(rows_to_int8<XT, GATE, false, 1024, 1, false>, 1024);
  else if (n <= 8192) go(rows_to_int8<XT, GATE, STREAM, 256, 4, false>, 256);
  else if (n <= kHeld) go(rows_to_int8<XT, GATE, STREAM, 1024, 4, false>, 1024);
  else go(rows_to_int8<XT, GATE, false, 1024, 4, true>, 1024);
  return hipGetLastError();
}
// An input that no cache holds and whose rows are read once is read past the caches: 16384 x 8192 bf16 (256
// MiB) 72 -> 69 us, 16384 x 4096 (128) 36.8 -> 34.9, 16384 x 2048 with a gate (128) 36.7 -> 34.0, 16384 x
// 8192 f32 (512) 120 -> 114, 65536 x 2048 bf16 in another order (256) 80 -> 75; but 20000 x 2048 bf16 (78)
// 22.9 -> 24.3, 8192 x 2048 with a gate (64) 17.0 -> 20.1, 4096 x 4096 f32 (64) 15.1 -> 17.5.  Rows that go to
// several places come from the caches after the first time: 65536 rows from 16384 x 4096 bf16 (128) 119 with
// them, 131 past them, 32768 from 16384 x 4096 f32 (256) 101 and 119, with a gate (bf16, 256) 109 and 118.  So do
// rows that are read twice: 4000 x 40000 bf16 89 and 92, f32 148 and 173, 2000 x 65536 f32 138 and 168.
constexpr int64_t kStreamBytes = int64_t(1) << 27;
template <int XT> hipError_t launch_type(const QRParams& p, hipStream_t s) {
  const int64_t each = (XT == DT_F32 ? 4 : 2) * (p.gate ? 2 : 1);
  const bool big = p.rows <= p.x_rows && p.q_cols <= kHeld && p.rows * p.cols >= kStreamBytes / each;
  if (p.gate) return big ? launch<XT, true, true>(p, s) : launch<XT, true, false>(p, s);
  return big ? launch<XT, false, true>(p, s) : launch<XT, false, false>(p, s);
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace htk

using namespace htk;

extern "C" int quant_rows(const quant_rows_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  constexpr int64_t kMost = INT32_MAX / 2, kMostCols = int64_t(1) << 24;
  if (a->rows < 0 || a->cols < 0 || a->rows > kMost || a->cols > kMostCols) return GEMM_ERR_INVALID_ARG;
  if ((a->pad != 0 && a->pad != 1) || a->index_div < 1) return GEMM_ERR_INVALID_ARG;
  if (a->act < GEMM_ACT_NONE || a->act > GEMM_ACT_SILU || (!a->gate && a->act != GEMM_ACT_NONE)) return GEMM_ERR_INVALID_ARG;
  if (a->row_index && (a->x_rows < 0 || a->x_rows > kMost)) return GEMM_ERR_INVALID_ARG;
  if (a->x_type != GEMM_F32 && a->x_type != GEMM_F16 && a->x_type != GEMM_BF16) return GEMM_ERR_DTYPE_COMBO;
  if (a->ldx < a->cols || a->ldq < a->cols || (a->gate && a->ldg < a->cols)) return GEMM_ERR_LAYOUT;
  const int xs = a->x_type == GEMM_F32 ? 4 : 2;
  if (!on(a->x, xs) || !on(a->gate, xs) || !on(a->scale, 4) || !on(a->row_index, 4)) return GEMM_ERR_MISALIGNED;
  if (a->rows > 0) {
    if (!a->scale || (a->cols > 0 && !a->q)) return GEMM_ERR_INVALID_ARG;
    if (a->cols > 0 && !a->x && !(a->row_index && a->x_rows == 0)) return GEMM_ERR_INVALID_ARG;
  }
  const int rc = arch_status();
  if (rc) return rc;
  if (a->rows == 0) return GEMM_OK;
  QRParams p;
  p.x = a->x;
  p.gate = a->gate;
  p.index = a->row_index;
  p.q = static_cast<u8*>(a->q);
  p.scale = a->scale;
  p.rows = a->rows;
  p.ldx = a->ldx;
  p.ldg = a->ldg;
  p.x_rows = a->row_index ? a->x_rows : a->rows;
  p.ldq = a->ldq;
  p.cols = (int)a->cols;
  p.q_cols = (int)(a->pad ? std::min(a->ldq, (a->cols + 15) / 16 * 16) : a->cols);
  p.index_div = a->index_div;
  p.act = a->act;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t err = a->x_type == GEMM_F32   ? launch_type<DT_F32>(p, s)
                         : a->x_type == GEMM_F16 ? launch_type<DT_F16>(p, s)
                                                 : launch_type<DT_BF16>(p, s);
  return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
