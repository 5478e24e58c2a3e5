// quant.hip -- block quantisation to e4m3 (quant_blocks of htscaled.h).
//
// For a block with largest magnitude top:  t = max(top, 448 * 2^-126), scale = t / 448,
// q = e4m3(clamp(x * (448 / t))).  Both kernels read x once, keep the block in registers between
// the maximum and the conversion, and are bound by memory.
#include <algorithm>

#include "../../include/htscaled.h"
#include "arch.h"
#include "kernels.h"

namespace htk {
namespace {

struct QParams {
  const void* x;
  const int32_t* index;
  u8* q;
  u8* qt;
  float* scale;
  float* scale_t;
  int64_t rows, cols, ldx, x_rows;
  int64_t ldq, ldqt, q_cols, qt_cols;   // q_cols, qt_cols: written columns, zeros past the data
  int64_t scale_r, scale_c, scale_t_c, scale_t_r;
  int index_div, pow2, block;           // block: one scale for 128 x 128
  int x_vec, q_vec, qt_vec;             // rows start on 16 (x, qt) and 8 (q) bytes
};

template <int XT> struct XType;
template <> struct XType<DT_F32> {
  typedef float T;
  __device__ static float up(float v) { return v; }
};
template <> struct XType<DT_BF16> {
  typedef u16 T;
  __device__ static float up(u16 v) { return bf16_to_f32(v); }
};
template <> struct XType<DT_F16> {
  typedef u16 T;
  __device__ static float up(u16 v) { return f16_to_f32(v); }
};

// The source rows of result rows r .. r + N - 1, -1 for a row of zeros.  All indices are loaded
// before one is used.
template <int N> __device__ __forceinline__ void source_rows(const QParams& p, int64_t r, int64_t (&s)[N]) {
  if (!p.index) {
    static_for<N>([&](auto i) { s[i] = r + i < p.rows ? r + i : -1; });
    return;
  }
  int at[N];
  static_for<N>([&](auto i) { at[i] = p.index[min(r + i, p.rows - 1)]; });
  static_for<N>([&](auto i) {
    const bool ok = r + i < p.rows && at[i] >= 0;
    const int64_t q = p.index_div == 1 ? at[i] : (int)((u32)at[i] / (u32)p.index_div);
    s[i] = ok && q < p.x_rows ? q : -1;
  });
}

// Loads have clamped addresses in place of conditions, and what they fetch in vain is dropped
// afterwards: loads under conditions of their own wait for each other (64 single ones of a patch of
// 8 x 8 at odd columns took 12 us).
//
// Columns c .. c + 7 of source row s as fp32; zero past the row and for s < 0.
template <int XT>
__device__ __forceinline__ void load8(const QParams& p, int64_t s, int64_t c, float (&v)[8]) {
  typedef typename XType<XT>::T T;
  static_for<8>([&](auto i) { v[i] = 0.f; });
  if (p.x_rows == 0) return;        // there is nothing to clamp to
  const T* src = (const T*)p.x + max(s, (int64_t)0) * p.ldx;
  if (p.x_vec && c + 8 <= p.cols) {
    constexpr int PER = 16 / (int)sizeof(T);
    static_for<8 / PER>([&](auto h) {
      const u32x4 w = reinterpret_cast<const u32x4*>(src + c)[(int)h];
      const T* e = reinterpret_cast<const T*>(&w);
      static_for<PER>([&](auto i) { v[h * PER + i] = XType<XT>::up(e[(int)i]); });
    });
  } else {
    T e[8];
    static_for<8>([&](auto i) { e[i] = src[min(c + i, p.cols - 1)]; });
    static_for<8>([&](auto i) { v[i] = c + i < p.cols ? XType<XT>::up(e[i]) : 0.f; });
  }
  static_for<8>([&](auto i) { v[i] = s < 0 ? 0.f : v[i]; });
}

// |x| as an integer: ordered as the magnitudes are, with infinity and then NaN above all.
__device__ __forceinline__ u32 mag(float x) { return __builtin_bit_cast(u32, x) & 0x7fffffffu; }

// Maximum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ u32 row_max(u32 v) {
  v = max(v, (u32)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));  // row_ror:8
  v = max(v, (u32)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
  v = max(v, (u32)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
  return max(v, (u32)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
}

struct Scale {
  float scale, inverse;   // both NaN for a block with an infinity or a NaN
};
__device__ __forceinline__ Scale scale_of(u32 top, int pow2) {
  Scale s;
  const bool bad = top >= 0x7f800000u;
  if (pow2) {
    // top = 1.f * 2^e: the least power of two s with top / s <= 448 = 1.75 * 2^8 is 2^(e - 8), one
    // more when the fraction is above 1.75
    const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    const int c = max(e, -126);
    s.scale = __builtin_bit_cast(float, (u32)(c + 127) << 23);
    s.inverse = __builtin_bit_cast(float, (u32)(127 - c) << 23);
  } else {
    const float t = fmaxf(__builtin_bit_cast(float, bad ? 0u : top), 448.f * 0x1p-126f);
    s.scale = t / 448.f;
    s.inverse = 448.f / t;
  }
  if (bad) s.scale = s.inverse = __builtin_nanf("");
  return s;
}

// Four e4m3 codes; the products are rounded to fp32, then to nearest even in the conversion.
__device__ __forceinline__ u32 codes4(float a, float b, float c, float d, float inverse) {
  auto clip = [&](float v) { return __builtin_amdgcn_fmed3f(v * inverse, -448.f, 448.f); };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clip(a), clip(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(clip(c), clip(d), w, true);
  return inverse == inverse ? (u32)w : 0x7f7f7f7fu;
}

// 8 codes at row r, columns c .. c + 7: those below `cols` data, zeros up to q_cols.
__device__ __forceinline__ void store8(const QParams& p, int64_t r, int64_t c, u32 lo, u32 hi) {
  u8* d = p.q + r * p.ldq + c;
  const uint64_t w = (uint64_t)hi << 32 | lo;
  if (p.q_vec && c + 8 <= p.q_cols) {
    *reinterpret_cast<uint64_t*>(d) = w;
  } else {
    const int n = (int)min((int64_t)8, p.q_cols - c);
    uint64_t left = w;
#pragma unroll 1
    for (int i = 0; i < n; ++i, left >>= 8) d[i] = (u8)left;
  }
}
// Codes past the data are zero even in a block whose scale is NaN.
__device__ __forceinline__ u32 keep(u32 w, int left) {
  return left >= 4 ? w : left <= 0 ? 0u : w & (0xffffffffu >> (8 * (4 - left)));
}

// A dimension of a launch has fewer than 2^32 threads, and one with more runs as what is left modulo
// 2^32, without an error: the workgroups are dealt over two dimensions.
constexpr int64_t kMostX = int64_t(1) << 22;
dim3 grid_of(int64_t blocks) {
  const int64_t x = std::min(blocks, kMostX);
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ u32 block_id() { return blockIdx.y * gridDim.x + blockIdx.x; }

// Scales for each row and 128 columns, row-major: a wave takes 512 columns of a row, a lane 8
// neighbouring ones, the 16 lanes of a DPP row one block.  One row of 8192: 2.7 us, a launch.
template <int XT>
__global__ __launch_bounds__(256) void quant_rows(const QParams p, int64_t units, int segs) {
  const int lane = threadIdx.x & 63;
  const int64_t u = (int64_t)block_id() * 4 + (threadIdx.x >> 6);
  if (u >= units) return;
  const int64_t r = u / segs, c = (u - r * segs) * 512 + lane * 8;
  float v[8];
  int64_t s1[1];
  source_rows<1>(p, r, s1);
  load8<XT>(p, s1[0], c, v);
  u32 m = 0;
  static_for<8>([&](auto i) { m = max(m, mag(v[i])); });
  const Scale s = scale_of(row_max(m), p.pow2);
  const int left = (int)(p.cols - c);
  store8(p, r, c, keep(codes4(v[0], v[1], v[2], v[3], s.inverse), left),
         keep(codes4(v[4], v[5], v[6], v[7], s.inverse), left - 4));
  if ((lane & 15) == 0 && c < p.cols) p.scale[r * p.scale_r + c / 128 * p.scale_c] = s.scale;
}

// 8 x 8 values of a lane.  16-bit types stay packed, two to a register, and their magnitudes are
// compared as 16-bit integers (they are ordered alike, infinity and NaN on top).
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
template <int XT> struct Patch {
  u32x4 w[8];
  __device__ __forceinline__ void load(const QParams& p, const int64_t (&s)[8], int64_t c) {
    static_for<8>([&](auto i) { w[i] = u32x4{0, 0, 0, 0}; });
    if (p.x_rows == 0) return;
    const u16* x = (const u16*)p.x;
    if (p.x_vec && c + 8 <= p.cols) {
      static_for<8>([&](auto i) { w[i] = *reinterpret_cast<const u32x4*>(x + max(s[i], (int64_t)0) * p.ldx + c); });
    } else {
      static_for<8>([&](auto i) {
        const u16* src = x + max(s[i], (int64_t)0) * p.ldx;
        u32 e[8];
        static_for<8>([&](auto j) { e[j] = src[min(c + j, p.cols - 1)]; });
        static_for<4>([&](auto d) {
          w[i][(int)d] = (c + 2 * d < p.cols ? e[2 * d] : 0u) | (c + 2 * d + 1 < p.cols ? e[2 * d + 1] << 16 : 0u);
        });
      });
    }
    static_for<8>([&](auto i) { w[i] = s[i] < 0 ? u32x4{0, 0, 0, 0} : w[i]; });
  }
  template <int I, int J> __device__ __forceinline__ float at() const {
    if constexpr (XT == DT_BF16) return __builtin_bit_cast(float, J % 2 ? w[I][J / 2] & 0xffff0000u : w[I][J / 2] << 16);
    else return f16_to_f32((u16)(w[I][J / 2] >> (16 * (J % 2))));
  }
  __device__ __forceinline__ static u32 max2(u32 a, u32 b) {
    return __builtin_bit_cast(u32, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  }
  __device__ __forceinline__ static u32 wide(u32 m) {  // the fp32 bits of a 16-bit magnitude
    return XT == DT_BF16 ? m << 16 : __builtin_bit_cast(u32, f16_to_f32((u16)m));
  }
  // largest magnitude of row i / of each column over the 8 rows, as fp32 bits
  __device__ __forceinline__ u32 row_top(int i) const {
    u32 m = 0;
    static_for<4>([&](auto d) { m = max2(m, w[i][(int)d] & 0x7fff7fffu); });
    return wide(max(m & 0xffffu, m >> 16));
  }
  __device__ __forceinline__ void col_top(u32 (&top)[8]) const {
    static_for<4>([&](auto d) {
      u32 m = 0;
      static_for<8>([&](auto i) { m = max2(m, w[i][(int)d] & 0x7fff7fffu); });
      top[2 * d] = wide(m & 0xffffu);
      top[2 * d + 1] = wide(m >> 16);
    });
  }
};
template <> struct Patch<DT_F32> {
  float v[8][8];
  __device__ __forceinline__ void load(const QParams& p, const int64_t (&s)[8], int64_t c) {
    static_for<8>([&](auto i) { load8<DT_F32>(p, s[i], c, v[i]); });
  }
  template <int I, int J> __device__ __forceinline__ float at() const { return v[I][J]; }
  __device__ __forceinline__ u32 row_top(int i) const {
    u32 m = 0;
    static_for<8>([&](auto j) { m = max(m, mag(v[i][j])); });
    return m;
  }
  __device__ __forceinline__ void col_top(u32 (&top)[8]) const {
    static_for<8>([&](auto j) {
      top[j] = 0;
      static_for<8>([&](auto i) { top[j] = max(top[j], mag(v[i][j])); });
    });
  }
};

// A 128 x 128 tile: row-major and transposed codes from one read, with scales by row and by
// column, or one scale for the tile.  Thread (ty, lx) holds rows 8 ty .. + 7 of columns 8 lx .. + 7;
// thread i makes the scale of column i or row i - 128 from the maxima in LDS, once, which keeps the
// code short: a small matrix pays for fetching it.  The transposed codes go through LDS (chunk ^
// column / 8, so that the 16 lanes of a write fall on different banks) and leave as 16-byte chunks.
// 8192 x 8192 bf16 both ways: 60 us, 4.6 TB/s (a copy reaches 4.7); with each thread making the
// scales of all its rows and columns 73 us, a matrix of 21 x 3323 19 us in place of 12.
template <int XT>
__global__ __launch_bounds__(256) void quant_tiles(const QParams p, int tiles_c, u32 tiles) {
  __shared__ u32 tops[256];       // of the columns, then the rows; [0] of the tile
  __shared__ alignas(16) float inverse[256];
  __shared__ uint64_t turned[128 * 16];
  const int tid = threadIdx.x, lx = tid & 15, ty = tid >> 4;
  const u32 tile = block_id();
  if (tile >= tiles) return;
  const int64_t rb = tile / (u32)tiles_c, cb = tile % (u32)tiles_c;
  const int64_t r0 = rb * 128 + ty * 8, c0 = cb * 128 + lx * 8;
  tops[tid] = 0;
  Patch<XT> v;
  int64_t from[8];
  source_rows<8>(p, r0, from);
  v.load(p, from, c0);
  __syncthreads();
  // maxima: the same whatever the order
  if (p.block) {
    u32 m = 0;
    static_for<8>([&](auto i) { m = max(m, v.row_top(i)); });
    m = row_max(m);
    if (lx == 0) atomicMax(&tops[0], m);
  } else {
    if (p.qt) {
      u32 top[8];
      v.col_top(top);
      static_for<8>([&](auto j) {
        u32 m = top[j];
        m = max(m, (u32)__shfl_xor((int)m, 16, 64));
        m = max(m, (u32)__shfl_xor((int)m, 32, 64));
        if ((tid & 48) == 0) atomicMax(&tops[lx * 8 + j], m);
      });
    }
    if (p.q) {
      static_for<8>([&](auto i) {
        const u32 m = row_max(v.row_top(i));
        if (lx == 0) tops[128 + ty * 8 + i] = m;
      });
    }
  }
  __syncthreads();
  const Scale s = scale_of(tops[p.block ? 0 : tid], p.pow2);
  inverse[tid] = s.inverse;
  if (p.block) {
    if (tid == 0) p.scale[rb * p.scale_r + cb * p.scale_c] = s.scale;
  } else if (tid < 128) {
    const int64_t c = cb * 128 + tid;
    if (p.qt && c < p.cols) p.scale_t[c * p.scale_t_c + rb * p.scale_t_r] = s.scale;
  } else {
    const int64_t r = rb * 128 + tid - 128;
    if (p.q && r < p.rows) p.scale[r * p.scale_r + cb * p.scale_c] = s.scale;
  }
  __syncthreads();
  const int rows = (int)(p.rows - r0), cols = (int)(p.cols - c0);   // of the patch that are data
  if (p.qt) {
    static_for<8>([&](auto j) {
      const int col = lx * 8 + j;
      const float f = inverse[col];
      const u32 lo = keep(codes4(v.template at<0, j>(), v.template at<1, j>(), v.template at<2, j>(), v.template at<3, j>(), f), rows);
      const u32 hi = keep(codes4(v.template at<4, j>(), v.template at<5, j>(), v.template at<6, j>(), v.template at<7, j>(), f), rows - 4);
      turned[col * 16 + (((ty >> 1) ^ (lx & 7)) << 1 | (ty & 1))] = (uint64_t)hi << 32 | lo;
    });
  }
  if (p.q) {
    static_for<8>([&](auto i) {
      const float f = inverse[128 + ty * 8 + i];
      if (i < rows)
        store8(p, r0 + i, c0, keep(codes4(v.template at<i, 0>(), v.template at<i, 1>(), v.template at<i, 2>(), v.template at<i, 3>(), f), cols),
               keep(codes4(v.template at<i, 4>(), v.template at<i, 5>(), v.template at<i, 6>(), v.template at<i, 7>(), f), cols - 4));
    });
  }
  if (!p.qt) return;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int q = tid + it * 256, col = q >> 3, ch = q & 7;
    const int64_t c = cb * 128 + col, r = rb * 128 + ch * 16;
    if (c >= p.cols || r >= p.qt_cols) continue;
    const u32x4 w = *reinterpret_cast<const u32x4*>(&turned[col * 16 + ((ch ^ ((col >> 3) & 7)) << 1)]);
    u8* d = p.qt + c * p.ldqt + r;
    if (p.qt_vec && r + 16 <= p.qt_cols) {
      *reinterpret_cast<u32x4*>(d) = w;
    } else {
      const u8* e = reinterpret_cast<const u8*>(&w);
#pragma unroll
      for (int b = 0; b < 16; ++b)
        if (r + b < p.qt_cols) d[b] = e[b];
    }
  }
}

template <int XT> hipError_t launch(const QParams& p, hipStream_t s, bool* too_large) {
  if (!p.block && !p.qt) {
    const int64_t segs = (p.q_cols + 511) / 512, units = p.rows * segs, blocks = (units + 3) / 4;
    if (blocks > INT32_MAX) { *too_large = true; return hipSuccess; }
    hipLaunchKernelGGL(quant_rows<XT>, grid_of(blocks), dim3(256), 0, s, p, units, (int)segs);
  } else {
    const int64_t tc = (p.cols + 127) / 128, blocks = (p.rows + 127) / 128 * tc;
    if (blocks > INT32_MAX) { *too_large = true; return hipSuccess; }
    hipLaunchKernelGGL(quant_tiles<XT>, grid_of(blocks), dim3(256), 0, s, p, (int)tc, (u32)blocks);
  }
  return hipGetLastError();
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether every i * si + j * sj with i < n and j < m is a place of its own (strides not below 0): the
// lines of one stride have to end before the other's next one begins.
bool own_places(int64_t n, int64_t si, int64_t m, int64_t sj) {
  if (n <= 1) return m <= 1 || sj > 0;
  if (m <= 1) return si > 0;
  return si < sj ? si > 0 && (sj - 1) / si >= n - 1 : sj > 0 && (si - 1) / sj >= m - 1;
}

}  // namespace
}  // namespace htk

using namespace htk;

extern "C" int quant_blocks(const quant_args* a, void* stream) {
  if (!a) return GEMM_ERR_INVALID_ARG;
  constexpr int64_t kMost = INT32_MAX / 2;
  if (a->rows < 0 || a->cols < 0 || a->rows > kMost || a->cols > kMost) return GEMM_ERR_INVALID_ARG;
  if (a->block_rows != 1 && a->block_rows != 128) return GEMM_ERR_INVALID_ARG;
  if ((a->pow2 != 0 && a->pow2 != 1) || (a->pad != 0 && a->pad != 1) || a->index_div < 1) return GEMM_ERR_INVALID_ARG;
  if (a->row_index && (a->x_rows < 0 || a->x_rows > kMost)) return GEMM_ERR_INVALID_ARG;
  if (a->x_type != GEMM_F32 && a->x_type != GEMM_F16 && a->x_type != GEMM_BF16) return GEMM_ERR_DTYPE_COMBO;
  const bool block = a->block_rows == 128;
  if (a->ldx < a->cols || (a->q && a->ldq < a->cols) || (a->qt && a->ldqt < a->rows)) return GEMM_ERR_LAYOUT;
  if (a->scale && (a->scale_r < 0 || a->scale_c < 0)) return GEMM_ERR_LAYOUT;
  if (a->scale_t && (a->scale_t_c < 0 || a->scale_t_r < 0)) return GEMM_ERR_LAYOUT;
  if (a->rows > 0 && a->cols > 0) {   // buffers of an empty matrix may be NULL
    if (!a->q && !a->qt) return GEMM_ERR_INVALID_ARG;
    if (block ? (!a->scale || a->scale_t) : ((a->q != nullptr) != (a->scale != nullptr) ||
                                             (a->qt != nullptr) != (a->scale_t != nullptr)))
      return GEMM_ERR_INVALID_ARG;
    if (!a->x && !(a->row_index && a->x_rows == 0)) return GEMM_ERR_INVALID_ARG;
    // scales of several blocks at one place would be written by all of them
    const int64_t rb = (a->rows + 127) / 128, cb = (a->cols + 127) / 128;
    if (a->scale && !own_places(block ? rb : a->rows, a->scale_r, cb, a->scale_c)) return GEMM_ERR_LAYOUT;
    if (a->scale_t && !own_places(a->cols, a->scale_t_c, rb, a->scale_t_r)) return GEMM_ERR_LAYOUT;
  }
  const int xs = a->x_type == GEMM_F32 ? 4 : 2;
  if (!on(a->x, xs) || !on(a->scale, 4) || !on(a->scale_t, 4) || !on(a->row_index, 4)) return GEMM_ERR_MISALIGNED;
  const int rc = arch_status();
  if (rc) return rc;
  if (a->rows == 0 || a->cols == 0) return GEMM_OK;
  QParams p;
  p.x = a->x;
  p.index = a->row_index;
  p.q = static_cast<u8*>(a->q);
  p.qt = static_cast<u8*>(a->qt);
  p.scale = a->scale;
  p.scale_t = a->scale_t;
  p.rows = a->rows;
  p.cols = a->cols;
  p.ldx = a->ldx;
  p.x_rows = a->row_index ? a->x_rows : a->rows;
  p.ldq = a->ldq;
  p.ldqt = a->ldqt;
  p.q_cols = !a->q ? 0 : a->pad ? std::min(a->ldq, (a->cols + 15) / 16 * 16) : a->cols;
  p.qt_cols = !a->qt ? 0 : a->pad ? std::min(a->ldqt, (a->rows + 15) / 16 * 16) : a->rows;
  p.scale_r = a->scale_r;
  p.scale_c = a->scale_c;
  p.scale_t_c = a->scale_t_c;
  p.scale_t_r = a->scale_t_r;
  p.index_div = a->index_div;
  p.pow2 = a->pow2;
  p.block = block;
  p.x_vec = on(a->x, 16) && a->ldx * xs % 16 == 0;
  p.q_vec = on(a->q, 8) && a->ldq % 8 == 0;
  p.qt_vec = on(a->qt, 16) && a->ldqt % 16 == 0;
  bool too_large = false;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t err = a->x_type == GEMM_F32   ? launch<DT_F32>(p, s, &too_large)
                         : a->x_type == GEMM_F16 ? launch<DT_F16>(p, s, &too_large)
                                                 : launch<DT_BF16>(p, s, &too_large);
  if (too_large) return GEMM_ERR_INVALID_ARG;
  return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
