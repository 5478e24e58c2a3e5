// scaled.h -- gfx950 kernels of the block-scaled e4m3 products (htscaled.h).
//
//   D(m, n) = act(alpha * rs[m] * sum_b sA(m, b) sB(n, b) * [sum_{k in block b} A(m, k) B(n, k)]
//                 + beta C(m, n) + bias[n])
//
// A block of k is 128 long: exactly one v_mfma_f32_16x16x128_f8f6f4.  Its sum over the block
// starts from zero and is then added to the fp32 accumulator with one fused multiply-add by
// sA * sB, so fp32 scales of any value cost 4 VALU operations for each matrix instruction (16 of
// its 32 issue cycles on a SIMD; they run beside the other wave's, or the next, MFMA).
//
// Operands are swapped in the instruction: B's rows (n) are its A operand and A's rows (m) its B
// operand.  A lane's four accumulators are then four neighbouring n of one m: one A scale
// serves them all, a 128-wide B scale is the same for the whole wave, and the outputs of a lane
// are contiguous in D.
#pragma once

#include "kernels.h"

namespace htk {

constexpr int kSB = 128;  // values of k per scale

struct SParams {
  const u8* A;
  const u8* B;
  const float* a_scale;
  const float* b_scale;
  const void* C;             // nullptr: not read
  void* D;
  const void* bias;          // nullptr: none
  const float* row_scale;    // nullptr: none
  const int32_t* offsets;    // groups
  float* workspace;          // fp32 planes, split_k > 1
  int64_t M, N, K;
  int64_t lda, ldb, ldc, ldd;
  int64_t a_sm, a_sk, b_sn, b_sk;
  int64_t a_l, b_l, c_l, d_l, as_l, bs_l;  // elements from one product to the next
  float alpha, beta;
  int act, form, groups;
  int tiles_m, tiles_n;
  int split_k, blocks_per_split;           // slices of k, in blocks of 128
};

enum : int { FORM_SINGLE = 0, FORM_BATCH = 1, FORM_ROWS = 2, FORM_K = 3 };

// One workgroup's share: its product's operands, its tile and its blocks of k.
struct STile {
  const u8* A;               // row 0 of the product (group), k = 0
  const u8* B;
  const float* a_scale;
  const float* b_scale;
  const void* C;
  void* D;
  const float* row_scale;
  int64_t M;                 // rows of this product or group
  int64_t m0, n0;
  int64_t k0, k1;            // k0 a multiple of 128
};

// Inclusive maximum / sum over the lanes of a wave (values >= 0), by DPP: shifts within rows of 16
// lanes, then the last lane of a row broadcast to the rows after it.
template <bool MAX> __device__ __forceinline__ int wave_scan(int v) {
  auto step = [&](auto ctrl, auto rows) {
    const int o = __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
    v = MAX ? max(v, o) : v + o;
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});  // row_shr:1
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast:15
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // row_bcast:31
  return v;
}

// 64 groups of rows, a lane each: the rows [lo, hi) of group c + lane, with the offsets clamped
// and made non-decreasing, and the running number of tiles.  `top` is the largest offset before.
struct GroupLane {
  int lo, hi, tiles, upto;
};
template <int BM>
__device__ __forceinline__ GroupLane group_lane(const SParams& p, int c, int lane, int top) {
  const int M = (int)p.M, i = c + lane;
  GroupLane r;
  r.lo = max(wave_scan<true>(i <= p.groups ? min(max(p.offsets[i], 0), M) : 0), top);
  r.hi = i < p.groups ? max(r.lo, min(max(p.offsets[i + 1], 0), M)) : r.lo;
  r.tiles = (r.hi - r.lo + BM - 1) / BM * p.tiles_n;
  r.upto = wave_scan<false>(r.tiles);
  return r;
}

// Workgroup id -> place in the tile order: ids are dealt to the 8 XCDs in turn, and each XCD gets
// a contiguous range, so that neighbours in the order share an L2.
__device__ __forceinline__ int xcd_order(int pid, int n) {
  const int per = n >> 3, extra = n & 7, x = pid & 7;
  return x * per + min(x, extra) + (pid >> 3);
}
// Tile t of a product with tm x tn tiles: 4 tile rows at a time, column by column.
__device__ __forceinline__ void walk_tiles(int t, int tm, int tn, int& m, int& n) {
  const int width = 4 * tn, group = t / width, first = group * 4;
  const int rows = min(tm - first, 4), within = t - group * width;
  m = first + within % rows;
  n = within / rows;
}

// The tile of this workgroup; false for one that has none (it exits before its first barrier).
// Groups of rows: every wave scans the offsets, 64 groups at a time, for the number of tiles and
// then for the group that holds its own; no launch before the product is needed for it.
template <int BM, int BN, class OT>
__device__ __forceinline__ bool tile_share(const SParams& p, STile& s) {
  s.A = p.A;
  s.B = p.B;
  s.a_scale = p.a_scale;
  s.b_scale = p.b_scale;
  s.C = p.C;
  s.D = p.D;
  s.row_scale = p.row_scale;
  s.M = p.M;
  s.k0 = 0;
  s.k1 = p.K;
  int tm = p.tiles_m, t;
  const int lane = threadIdx.x & 63;
  if (p.form == FORM_ROWS) {
    const int G = p.groups;
    int total = 0, top = 0;
    GroupLane q;
    for (int c = 0; c < G; c += 64) {
      q = group_lane<BM>(p, c, lane, top);
      total += __builtin_amdgcn_readlane(q.upto, 63);
      top = __builtin_amdgcn_readlane(q.hi, 63);
    }
    if ((int)blockIdx.x >= total) return false;
    t = xcd_order(blockIdx.x, total);
    int e = 0, group0 = 0;
    top = 0;
    for (int c = 0; c < G; c += 64) {
      group0 = c;
      if (G > 64) q = group_lane<BM>(p, c, lane, top);
      const unsigned long long past = __ballot(q.upto > t);
      if (past != 0) {
        e = __ffsll(past) - 1;
        break;
      }
      t -= __builtin_amdgcn_readlane(q.upto, 63);
      top = __builtin_amdgcn_readlane(q.hi, 63);
    }
    t -= __builtin_amdgcn_readlane(q.upto - q.tiles, e);
    const int lo_e = __builtin_amdgcn_readlane(q.lo, e), hi_e = __builtin_amdgcn_readlane(q.hi, e);
    e += group0;
    s.A += (int64_t)lo_e * p.lda;
    s.a_scale += (int64_t)lo_e * p.a_sm;
    s.B += e * p.b_l;
    s.b_scale += e * p.bs_l;
    if (s.C) s.C = (const OT*)s.C + (int64_t)lo_e * p.ldc;
    s.D = (OT*)s.D + (int64_t)lo_e * p.ldd;
    if (s.row_scale) s.row_scale += lo_e;
    s.M = hi_e - lo_e;
    tm = (int)((s.M + BM - 1) / BM);
  } else {
    const int64_t z = blockIdx.z;
    if (p.form == FORM_BATCH) {
      s.A += z * p.a_l;
      s.B += z * p.b_l;
      s.a_scale += z * p.as_l;
      s.b_scale += z * p.bs_l;
    }
    if (p.form != FORM_SINGLE) {
      if (s.C) s.C = (const OT*)s.C + z * p.c_l;
      s.D = (OT*)s.D + z * p.d_l;
    }
    if (p.form == FORM_K) {
      int lo = 0, hi = 0;
      const int K = (int)p.K;
      for (int i = lane; i <= (int)z + 1; i += 64) {
        const int v = min(max(p.offsets[i], 0), K);
        hi = max(hi, v);
        if (i <= (int)z) lo = max(lo, v);
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) {
        lo = max(lo, __shfl_xor(lo, d, 64));
        hi = max(hi, __shfl_xor(hi, d, 64));
      }
      lo = __builtin_amdgcn_readfirstlane(lo);
      hi = __builtin_amdgcn_readfirstlane(hi);
      // an end at K itself may lie inside a block; a group that starts there is empty
      s.k0 = lo == K ? (K + kSB - 1) / kSB * (int64_t)kSB : lo / kSB * kSB;
      s.k1 = hi == K ? K : hi / kSB * kSB;
      if (s.k1 < s.k0) s.k1 = s.k0;
    }
    if (p.split_k > 1) {
      s.k0 = min((int64_t)blockIdx.y * p.blocks_per_split * kSB, p.K);
      s.k1 = min(s.k0 + (int64_t)p.blocks_per_split * kSB, p.K);
    }
    t = xcd_order(blockIdx.x, gridDim.x);
  }
  int m, n;
  walk_tiles(t, tm, p.tiles_n, m, n);
  s.m0 = (int64_t)m * BM;
  s.n0 = (int64_t)n * BN;
  return true;
}

// C, bias and D of either output type.
template <class OT> struct SOut;
template <> struct SOut<u16> {
  __device__ static float load(const void* p, int64_t i) { return bf16_to_f32(((const u16*)p)[i]); }
  __device__ static u16 bits(float v) { return f32_to_bf16(v); }
};
template <> struct SOut<float> {
  __device__ static float load(const void* p, int64_t i) { return ((const float*)p)[i]; }
  __device__ static float bits(float v) { return v; }
};

// One output from its fp32 sum; rounded once, to D's type.
template <class OT>
__device__ __forceinline__ void finish_one(const SParams& p, const STile& s, int64_t row, int64_t col, float sum) {
  float v = p.alpha * sum;
  if (s.row_scale) v *= s.row_scale[row];
  if (s.C) v += p.beta * SOut<OT>::load(s.C, row * p.ldc + col);
  if (p.bias) v += SOut<OT>::load(p.bias, col);
  ((OT*)s.D)[row * p.ldd + col] = SOut<OT>::bits(activate(p.act, v));
}

// One block of k of a 16 x 16 piece: the fragments of a lane (32 codes of one row) and their
// product.  The 8-bit matrix instructions take 8 neighbouring k at a time and drop of each product
// what lies below 2^(E - 13), 2^E being the largest product of the codes' powers of two, towards zero
// (probed product by product; all four fp8 forms were alike on random codes: 1.3e-5 to 5.6e-5 of the
// sum of the sizes).  The 7 others of a group then lose less than 7 * 2^-13 of its largest product,
// 2^-10 of the sizes at most.  For a result that is not small beside what it sums that is below half
// a step of bf16, so bf16 outputs take the 8-bit instruction; where large products cancel it is more,
// which the header says.  fp32 outputs take the codes as bf16, which holds them exactly, through the
// bf16 instruction at half the rate, whose sums keep fp32 (1e-8 to 8e-8 in the same measurement).
template <class OT> struct Frag;
template <> struct Frag<u16> {
  u32x4 w[2];
  __device__ __forceinline__ void set(int u, const u32x4& v) { w[u] = v; }
};
__device__ __forceinline__ f32x4 mfma_block(const Frag<u16>& n, const Frag<u16>& m) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
  Atom<DT_F8, 16>::mma(c, n.w, m.w, 0);
  return c;
}
template <> struct Frag<float> {
  bf16x8 w[4];
  __device__ __forceinline__ void set(int u, const u32x4& v) {
    static_for<2>([&](auto h) {
      static_for<2>([&](auto d) {
        static_for<2>([&](auto s) {
          const auto two = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * h + d], 1.0f, s != 0);
          w[2 * u + h][4 * d + 2 * s] = two[0];
          w[2 * u + h][4 * d + 2 * s + 1] = two[1];
        });
      });
    });
  }
};
__device__ __forceinline__ f32x4 mfma_block(const Frag<float>& n, const Frag<float>& m) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
  static_for<4>([&](auto q) { c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n.w[q], m.w[q], c, 0, 0, 0); });
  return c;
}

// ------------------------------------------------------------------------------------------
// Any alignment: 64 x 64 tiles, single-byte predicated loads through registers into LDS.  The
// kernel for operands that the 16-byte loads cannot read, and the plainest form of the
// operation: one block of k at a time, two barriers each.
// ------------------------------------------------------------------------------------------
template <class OT>
__global__ __launch_bounds__(256) void scaled_narrow(const SParams p, int b_block) {
  __shared__ u32x4 lds[128 * 8];              // 64 rows of A, then 64 rows of B
  STile s;
  if (!tile_share<64, 64, OT>(p, s)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int x = lane & 15, g = lane >> 4;
  f32x4 acc[2][2];
  static_for<2>([&](auto i) { static_for<2>([&](auto j) { acc[i][j] = f32x4{}; }); });
  for (int64_t k = s.k0; k < s.k1; k += kSB) {
#pragma unroll 1
    for (int q = tid; q < 128 * 8; q += 256) {
      const int row = q >> 3, c = q & 7;
      const int64_t r = row < 64 ? s.m0 + row : s.n0 + row - 64;
      const bool live = r < (row < 64 ? s.M : p.N);
      const u8* src = (row < 64 ? s.A + r * p.lda : s.B + r * p.ldb) + k + c * 16;
      u32x4 v;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        u32 w = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (live && k + c * 16 + d * 4 + b < s.k1) w |= (u32)src[d * 4 + b] << (8 * b);
        v[d] = w;
      }
      lds[swizzled_slot<8>(row, c)] = v;
    }
    __syncthreads();
    const int64_t kb = k / kSB;
    float sa[2];
    f32x4 sb[2];
    static_for<2>([&](auto i) {
      const int64_t m = s.m0 + wm + i * 16 + x;
      sa[i] = m < s.M ? s.a_scale[m * p.a_sm + kb * p.a_sk] : 0.f;
      static_for<4>([&](auto r) {
        const int64_t n = s.n0 + wn + i * 16 + g * 4 + r;
        sb[i][(int)r] = n < p.N ? s.b_scale[(b_block == 1 ? n : n / kSB) * p.b_sn + kb * p.b_sk] : 0.f;
      });
    });
    Frag<OT> fa[2], fb[2];
    static_for<2>([&](auto i) {
      static_for<2>([&](auto u) {
        fa[i].set(u, lds[swizzled_slot<8>(wm + i * 16 + x, g + 4 * u)]);
        fb[i].set(u, lds[swizzled_slot<8>(64 + wn + i * 16 + x, g + 4 * u)]);
      });
    });
    static_for<2>([&](auto i) {
      static_for<2>([&](auto j) {
        const f32x4 t = mfma_block(fb[j], fa[i]);
        static_for<4>([&](auto r) {
          acc[i][j][(int)r] = __builtin_fmaf(t[(int)r], sa[i] * sb[j][(int)r], acc[i][j][(int)r]);
        });
      });
    });
    __syncthreads();
  }
  static_for<2>([&](auto i) {
    static_for<2>([&](auto j) {
      static_for<4>([&](auto r) {
        const int64_t m = s.m0 + wm + i * 16 + x, n = s.n0 + wn + j * 16 + g * 4 + r;
        if (m < s.M && n < p.N) finish_one<OT>(p, s, m, n, acc[i][j][(int)r]);
      });
    });
  });
}

// ------------------------------------------------------------------------------------------
// The outputs of a lane: RM rows m, and in each of them RN pieces of 4 neighbouring columns.  The
// columns of a wave are dealt so that JP pieces of a lane make 16 bytes of D and the four lane
// groups c4 make 64 neighbouring bytes: piece j of group c4 starts at column
//   (j / JP) * 16 JP + c4 * 4 JP + (j % JP) * 4,
// i.e. LDS row j * 16 + y of the wave's B tile holds that column plus y % 4, c4 = y / 4.
// ------------------------------------------------------------------------------------------
template <class OT> struct Cols {
  static constexpr int VO = 16 / (int)sizeof(OT), JP = VO / 4;
  __device__ static constexpr int of(int j, int c4) { return (j / JP) * 16 * JP + c4 * 4 * JP + (j % JP) * 4; }
};

// Whole 16-byte loads of C and stores of D: one straight copy of the code for each activation and
// for C or none, because the epilogue runs once a tile and its instructions are fetched anew each
// time.  All of a lane's C is loaded first (D may be C, so no load could pass a store).
template <class OT, int RM, int RN, int ACT, bool HAS_C, class RowOf>
__device__ __forceinline__ void store_whole(const SParams& p, const STile& s, f32x4 (&acc)[RM][RN], RowOf row_of,
                                            int64_t col0, int x, int c4) {
  typedef Cols<OT> CM;
  constexpr int VO = CM::VO, NQ = RN / CM::JP;
  const int64_t col = col0 + CM::of(0, c4);
  u32x4 bias[NQ], c[HAS_C ? RM : 1][NQ];
  if constexpr (HAS_C) {
    static_for<RM>([&](auto i) {
      const int64_t row = row_of(i, x);
      static_for<NQ>([&](auto q) {
        c[i][q] = u32x4{0, 0, 0, 0};
        if (row < s.M) c[i][q] = *reinterpret_cast<const u32x4*>((const OT*)s.C + row * p.ldc + col + CM::of(q * CM::JP, 0));
      });
    });
  }
  static_for<NQ>([&](auto q) {
    bias[q] = u32x4{0, 0, 0, 0};
    if (p.bias) bias[q] = *reinterpret_cast<const u32x4*>((const OT*)p.bias + col + CM::of(q * CM::JP, 0));
  });
  static_for<RM>([&](auto i) {
    const int64_t row = row_of(i, x);
    if (row < s.M) {
      const float rs = s.row_scale ? s.row_scale[row] : 1.f;
      OT* d = (OT*)s.D + row * p.ldd + col;
      static_for<NQ>([&](auto q) {
        alignas(16) OT o[VO];
        static_for<VO>([&](auto e) {
          float v = acc[i][q * CM::JP + e / 4][e % 4] * p.alpha * rs;
          if constexpr (HAS_C) v += p.beta * SOut<OT>::load(&c[i][q], e);
          v += SOut<OT>::load(&bias[q], e);
          o[e] = SOut<OT>::bits(ACT == 1 ? relu(v) : ACT == 2 ? gelu(v) : ACT == 3 ? silu(v) : v);
        });
        *reinterpret_cast<u32x4*>(d + CM::of(q * CM::JP, 0)) = *reinterpret_cast<const u32x4*>(o);
      });
    }
  });
}

// The outputs of a workgroup with BN columns: col0 is the wave's first column, row_of(i, x) the row
// of row block i in lane x = lane % 16.  `lds` is the kernel's LDS, at least 16 x 68 floats a wave.
template <class OT, int BN, int RM, int RN, class RowOf>
__device__ __forceinline__ void store_outputs(const SParams& p, const STile& s, f32x4 (&acc)[RM][RN],
                                              RowOf row_of, int64_t col0, u32x4* lds, int wave) {
  typedef Cols<OT> CM;
  const int lane = threadIdx.x & 63, x = lane & 15, c4 = lane >> 4;
  __syncthreads();              // the operands in LDS have been read
  if (col0 >= p.N) return;
  const bool c_ok = !s.C || (p.ldc % CM::VO == 0 && (reinterpret_cast<uintptr_t>(s.C) & 15) == 0);
  if (col0 + 16 * RN <= p.N && c_ok && p.split_k <= 1 && p.ldd % CM::VO == 0 &&
      ((reinterpret_cast<uintptr_t>(s.D) | reinterpret_cast<uintptr_t>(p.bias)) & 15) == 0) {
    auto whole = [&](auto act) {
      if (s.C) store_whole<OT, RM, RN, decltype(act)::value, true>(p, s, acc, row_of, col0, x, c4);
      else store_whole<OT, RM, RN, decltype(act)::value, false>(p, s, acc, row_of, col0, x, c4);
    };
    if (p.act == 0) whole(std::integral_constant<int, 0>{});
    else if (p.act == 3) whole(std::integral_constant<int, 3>{});
    else if (p.act == 2) whole(std::integral_constant<int, 2>{});
    else whole(std::integral_constant<int, 1>{});
    return;
  }
  // everything else element by element, a row block of the wave at a time through LDS, so that a
  // row's neighbours are stored together; a lane has one column, and U rows in hand at once (D may
  // be C: their C is loaded before any is stored)
  constexpr int W = 16 * RN, PITCH = W + 4, U = 8;
  static_assert(W == 64, "a lane for each column");
  float* mine = reinterpret_cast<float*>(lds) + wave * 16 * PITCH;
  const int64_t col = col0 + lane;
  const bool in = col < p.N;
  const float bias = p.bias && in ? SOut<OT>::load(p.bias, col) : 0.f;
  float* plane = p.split_k > 1 ? p.workspace + (int64_t)blockIdx.y * p.M * p.N : nullptr;
  static_for<RM>([&](auto i) {
    static_for<RN>([&](auto j) { *reinterpret_cast<f32x4*>(&mine[x * PITCH + CM::of(j, c4)]) = acc[i][j]; });
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
    for (int r0 = 0; r0 < 16; r0 += U) {
      float v[U], c[U];
      static_for<U>([&](auto u) {
        const int64_t row = row_of(i, r0 + u);
        const bool ok = in && row < s.M;
        v[u] = mine[(r0 + u) * PITCH + lane];
        c[u] = 0.f;
        if (plane) {
          if (ok) plane[row * p.N + col] = v[u];
        } else {
          v[u] *= p.alpha;
          if (s.row_scale && ok) v[u] *= s.row_scale[row];
          if (s.C && ok) c[u] = SOut<OT>::load(s.C, row * p.ldc + col);
        }
      });
      if (!plane) {
        static_for<U>([&](auto u) {
          const int64_t row = row_of(i, r0 + u);
          const float y = activate(p.act, (s.C ? v[u] + p.beta * c[u] : v[u]) + bias);
          if (in && row < s.M) ((OT*)s.D)[row * p.ldd + col] = SOut<OT>::bits(y);
        });
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  });
}

typedef __attribute__((address_space(1))) const void gbl_void_t;

// ------------------------------------------------------------------------------------------
// Tiled kernel: BM x BN outputs by WM x WN waves, blocks of k in a ring of ST LDS stages filled
// by DMA, one barrier per block.  A stage holds the BM + BN rows of 128 bytes (XOR-swizzled
// chunks) and their BM + BN scales, fetched by 4-byte DMA so that scales may have any strides.
//
// Rows are placed in LDS so that a lane's rows are neighbours: LDS row i * 16 + x of a wave's A
// tile is its row x * RM + i, and LDS row j * 16 + y of its B tile the column that Cols gives.  The
// lane's A scales are then contiguous in LDS, and its outputs in D.  The placement costs nothing:
// every DMA lane has its own source address.
//
// Measured, two workgroups a CU: bf16 out 0.55 us for a block of a 128 x 128 tile and 0.36 us for one
// of 64 x 128 (8192^3: 560 to 590 and 730 to 740 us; with row-major scales of A or scales of single
// columns 632 and 644), where LDS traffic and the barrier bound it; with one
// workgroup a CU 0.72 and 0.43.  fp32 out 1.0 us (4096 x 8192 x 5120 with scales of single columns:
// 330 us, 1,040 TFLOP/s) is bound by issue: a wave's block of 64 x 64 has 64 matrix instructions of
// 8 issue cycles, 128 conversions and 128 scale operations of 4.  Two workgroups of 4 waves hide each
// other's phases; one workgroup with four stages took 737 us.  Reading fragments a block ahead, six
// stages, and 2 or 8 waves that share one block of the same tile changed nothing or lost.
//
// KH = 2, for fewer tiles than two a CU: two halves of the waves take the even and the odd blocks of
// k, each through a ring of its own, and join in LDS at the end.  They overlap as two workgroups
// would, without a split's planes in memory: 333 x 4096 x 8192 33 -> 29 us (fp32 48 -> 43), 1000 x
// 4096 x 4096 with 128 x 128 tiles 29 -> 26.  With more tiles two workgroups a CU overlap their
// prologues and epilogues too (128 rows over 64 experts 80 us, with halves 95).
// ------------------------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int ST, int BB, class OT, int OCC, int KH>
__global__ __launch_bounds__(KH * WM * WN * 64, OCC) void scaled_tile(const SParams p) {
  constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, RM = TM / 16, RN = TN / 16;
  constexpr int OPS_T = (BM + BN) / 8 / NW;          // tile DMA instructions per wave and block
  constexpr int SCI = (BM + BN) / 64;                // scale DMA instructions per block
  constexpr int OPS_S = (SCI + NW - 1) / NW;
  constexpr int OPS = OPS_T + OPS_S;
  constexpr int STAGE = (BM + BN) * 8 + (BM + BN) / 4;  // 16-byte chunks
  static_assert((BM + BN) % (8 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0, "DMA blocks over the waves");
  static_assert(TN <= kSB && kSB % TN == 0, "one 128-wide B scale per wave");
  __shared__ u32x4 lds[KH * ST * STAGE];
  STile s;
  if (!tile_share<BM, BN, OT>(p, s)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int half = KH == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid / (NW * 64));
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) - half * NW;
  u32x4* ring = lds + half * ST * STAGE;
  const int wm = wave / WN, wn = wave % WN;
  const int x = lane & 15, g = lane >> 4;

  const char* a_tile = uniform_ptr((const char*)s.A + s.m0 * p.lda + s.k0);
  const char* b_tile = uniform_ptr((const char*)s.B + s.n0 * p.ldb + s.k0);
  const int64_t K = uniform_i64(s.k1 - s.k0);
  const int64_t a_span = uniform_i64((s.M - s.m0 - 1) * p.lda + K);
  const int64_t b_span = uniform_i64((p.N - s.n0 - 1) * p.ldb + K);
  const int nk = (int)((K + kSB - 1) / kSB);

  // DMA instruction i of this wave fills LDS rows 8 blk .. 8 blk + 7 (A's, then B's), blk =
  // wave + NW i: lane l row 8 blk + l / 8, slot l % 8, which holds chunk (l % 8) ^ key(row).
  uint32_t off[OPS_T];
  const int chunk = (lane & 7) ^ row_key<8>((wave & 1) * 8 + (lane >> 3));
  static_for<OPS_T>([&](auto i) {
    const int R = (wave + NW * i) * 8 + (lane >> 3);
    if (R < BM) {
      const int w = R / TM, q = R % TM;
      off[i] = (uint32_t)((w * TM + (q & 15) * RM + (q >> 4)) * p.lda) + chunk * 16;
    } else {
      const int w = (R - BM) / TN, q = (R - BM) % TN, y = q & 15;
      off[i] = (uint32_t)((w * TN + Cols<OT>::of(q >> 4, y >> 2) + (y & 3)) * p.ldb) + chunk * 16;
    }
  });
  static_assert(NW % 2 == 0, "the row key of a wave's DMA blocks is the same in all of them");
  // scale addresses: lane l of instruction i fetches scale 64 i + l (A's rows, then B's)
  const float* sc_ptr[OPS_S];
  int64_t sc_step[OPS_S];
  const int64_t kb0 = s.k0 / kSB;
  static_for<OPS_S>([&](auto i) {
    const int q = ((wave + NW * i) % SCI) * 64 + lane;
    if (q < BM) {
      const int64_t m = min(s.m0 + q, s.M - 1);
      sc_ptr[i] = s.a_scale + m * p.a_sm + kb0 * p.a_sk;
      sc_step[i] = p.a_sk;
    } else {
      const int64_t n = min(s.n0 + q - BM, p.N - 1);
      sc_ptr[i] = s.b_scale + (BB == 1 ? n : n / kSB) * p.b_sn + kb0 * p.b_sk;
      sc_step[i] = p.b_sk;
    }
  });
  // Step t of a half is block t KH + half.  Blocks past the last are issued as zeros, so that the wait counts are the same throughout.
  auto dma = [&](int t, int stage) {
    u32x4* st = ring + stage * STAGE;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a_tile, a_span), rb = make_rsrc(b_tile, b_span);
    const int b = t * KH + half;
    const int64_t k = (int64_t)b * kSB;
    const bool in_k = k + chunk * 16 < K;
    static_for<OPS_T>([&](auto i) {
      const int blk = wave + NW * i;
      const uint32_t o = in_k ? off[i] : kOobOffset;
      if ((NW * i + NW) * 8 <= BM || blk * 8 < BM)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(st + blk * 64), 16, o, (int)k, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t*)(st + blk * 64), 16, o, (int)k, 0, 0);
    });
    static_for<OPS_S>([&](auto i) {
      const int ins = (wave + NW * i) % SCI;
      const float* src = sc_ptr[i] + (int64_t)min(b, nk - 1) * sc_step[i];
      __builtin_amdgcn_global_load_lds((gbl_void_t*)src, (lds_void_t*)(st + (BM + BN) * 8 + ins * 16), 4, 0, 0);
    });
  };

  f32x4 acc[RM][RN];
  static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { acc[i][j] = f32x4{}; }); });
  int slot[2];
  static_for<2>([&](auto u) { slot[u] = swizzled_slot<8>(x, g + 4 * u); });

  auto compute = [&](int stage) {
    const u32x4* st = ring + stage * STAGE;
    const u32x4* la = st + wm * TM * 8;
    const u32x4* lb = st + (BM + wn * TN) * 8;
    const float* ls = reinterpret_cast<const float*>(st + (BM + BN) * 8);
    Frag<OT> fb[RN];
    static_for<RN>([&](auto j) { static_for<2>([&](auto u) { fb[j].set(u, lb[j * 128 + slot[u]]); }); });
    float sa[RM];
    static_for<RM>([&](auto i) { sa[i] = ls[wm * TM + x * RM + i]; });
    f32x4 sb[BB == 1 ? RN : 1];
    if constexpr (BB == 1) {
      static_for<RN>([&](auto j) { sb[j] = *reinterpret_cast<const f32x4*>(&ls[BM + wn * TN + Cols<OT>::of(j, g)]); });
    } else {
      const float one = ls[BM + wn * TN];
      static_for<RM>([&](auto i) { sa[i] *= one; });
    }
    static_for<RM>([&](auto i) {
      Frag<OT> fa;
      static_for<2>([&](auto u) { fa.set(u, la[i * 128 + slot[u]]); });
      f32x4 t[RN];
      static_for<RN>([&](auto j) { t[j] = mfma_block(fb[j], fa); });
      static_for<RN>([&](auto j) {
        static_for<4>([&](auto r) {
          const float w = BB == 1 ? sa[i] * sb[BB == 1 ? (int)j : 0][(int)r] : sa[i];
          acc[i][j][(int)r] = __builtin_fmaf(t[j][(int)r], w, acc[i][j][(int)r]);
        });
      });
    });
  };

  if (nk > 0) {
    static_for<ST - 1>([&](auto q) { dma(q, q); });
    int stage = 0;
    for (int t = 0; t * KH < nk; ++t) {
      // block t has landed for this wave and, behind the barrier, for all; the stage refilled
      // next was last read before it
      wait_counts<(ST - 2) * OPS, true>();
      barrier_nofence();
      int next = stage + ST - 1;
      if (next >= ST) next -= ST;
      dma(t + ST - 1, next);
      if (KH == 1 || t * KH + half < nk) compute(stage);
      if (++stage == ST) stage = 0;
    }
    wait_counts<0, true>();  // zero blocks issued past the end
  }
  if constexpr (KH == 2) {      // the second half's sums are added to the first's, which stores
    static_assert(NW * RM * RN * 64 <= KH * ST * STAGE, "its sums fit the ring");
    f32x4* sums = reinterpret_cast<f32x4*>(lds) + wave * RM * RN * 64 + lane;
    __syncthreads();
    if (half == 1) static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { sums[(i * RN + j) * 64] = acc[i][j]; }); });
    __syncthreads();
    if (half == 0) static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { acc[i][j] += sums[(i * RN + j) * 64]; }); });
  }
  store_outputs<OT, BN, RM, RN>(p, s, acc, [&](int i, int r) { return s.m0 + wm * TM + r * RM + i; },
                                half == 0 ? s.n0 + wn * TN : p.N, lds, wave);
}

// ------------------------------------------------------------------------------------------
// Streaming kernel for few rows (decode): the cost is reading B once.  A workgroup owns 16 NBW
// columns and 16 RM rows; its WK waves take slices of k, each streaming its blocks of B (and the
// L2-resident rows of A) through a private LDS ring of R blocks by DMA, with no barrier in the
// loop.  The partial sums meet in LDS, in the order of the waves.  Bound by memory: 16 x 16384 x 8192
// takes 26.5 us (5.1 TB/s; whole 128-byte rows of B by DMA, two blocks in flight a wave), 1 x 4096 x
// 4096 5.6 us, most of it launch and the first loads.  With a short k (16 blocks) the waves' ramp
// costs more than the tiled kernel's barriers: 128 rows over 64 experts, K 2048, 105 us against 80.
// ------------------------------------------------------------------------------------------
template <int RM, int NBW, int WK, int R, int BB, class OT, int OCC>
__global__ __launch_bounds__(WK * 64, OCC) void scaled_stream(const SParams p) {
  constexpr int BM = 16 * RM, BN = 16 * NBW, ROWS = BM + BN;
  constexpr int OPS_S = (ROWS + 63) / 64, OPS = ROWS / 8 + OPS_S;
  constexpr int BLK = ROWS * 8 + OPS_S * 16;         // 16-byte chunks of a ring block
  constexpr int NT = WK * 64;
  static_assert(R >= 2 && (R - 2) * OPS < 64, "vmcnt range");
  static_assert(BN <= kSB && kSB % BN == 0, "one 128-wide B scale per workgroup");
  __shared__ u32x4 ring[WK][R][BLK];
  STile s;
  if (!tile_share<BM, BN, OT>(p, s)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int x = lane & 15, g = lane >> 4;
  const int64_t K = uniform_i64(s.k1 - s.k0);
  const int nb = (int)((K + kSB - 1) / kSB), per = (nb + WK - 1) / WK;
  const int b0 = wave * per, nloc = max(0, min(b0 + per, nb) - b0);

  const char* a_tile = uniform_ptr((const char*)s.A + s.m0 * p.lda + s.k0);
  const char* b_tile = uniform_ptr((const char*)s.B + s.n0 * p.ldb + s.k0);
  const int64_t a_span = uniform_i64((s.M - s.m0 - 1) * p.lda + K);
  const int64_t b_span = uniform_i64((p.N - s.n0 - 1) * p.ldb + K);
  const float* sc_ptr[OPS_S];
  int64_t sc_step[OPS_S];
  const int64_t kb0 = s.k0 / kSB + b0;
  static_for<OPS_S>([&](auto i) {
    const int q = i * 64 + lane;
    if (q < BN) {                                     // B's rows first, as in the ring block
      const int64_t n = min(s.n0 + q, p.N - 1);
      sc_ptr[i] = s.b_scale + (BB == 1 ? n : n / kSB) * p.b_sn + kb0 * p.b_sk;
      sc_step[i] = p.b_sk;
    } else {
      const int64_t m = min(s.m0 + q - BN, s.M - 1);
      sc_ptr[i] = s.a_scale + m * p.a_sm + kb0 * p.a_sk;
      sc_step[i] = p.a_sk;
    }
  });
  auto issue = [&](int j, auto slot) {
    const bool live = j < nloc;
    const int64_t kb = (int64_t)(b0 + j) * kSB;
    const int sk = live ? (int)kb : 0;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a_tile, a_span), rb = make_rsrc(b_tile, b_span);
    static_for<ROWS / 8>([&](auto c) {
      constexpr bool IS_A = c * 8 >= BN;
      const int row = 8 * c + (lane >> 3), src = IS_A ? row - BN : row;
      const int ch = (lane & 7) ^ row_key<8>(row);
      const uint32_t o = live && kb + ch * 16 < K ? (uint32_t)(src * (IS_A ? p.lda : p.ldb)) + ch * 16 : kOobOffset;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(IS_A ? ra : rb, (lds_void_t*)(&ring[wave][slot][c * 64]), 16, o, sk, 0, 0);
    });
    const int js = max(0, min(j, nloc - 1));
    if (nloc > 0)
      static_for<OPS_S>([&](auto i) {
        __builtin_amdgcn_global_load_lds((gbl_void_t*)(sc_ptr[i] + js * sc_step[i]),
                                         (lds_void_t*)(&ring[wave][slot][ROWS * 8 + i * 16]), 4, 0, 0);
      });
  };
  f32x4 acc[RM][NBW];
  static_for<RM>([&](auto i) { static_for<NBW>([&](auto j) { acc[i][j] = f32x4{}; }); });
  auto compute = [&](auto slot) {
    const u32x4* blk = &ring[wave][slot][0];
    const float* ls = reinterpret_cast<const float*>(blk + ROWS * 8);
    Frag<OT> fb[NBW];
    static_for<NBW>([&](auto j) {
      static_for<2>([&](auto u) { fb[j].set(u, blk[swizzled_slot<8>(j * 16 + x, g + 4 * u)]); });
    });
    static_for<RM>([&](auto i) {
      Frag<OT> fa;
      static_for<2>([&](auto u) { fa.set(u, blk[swizzled_slot<8>(BN + i * 16 + x, g + 4 * u)]); });
      const float sa = ls[BN + i * 16 + x];
      static_for<NBW>([&](auto j) {
        const f32x4 t = mfma_block(fb[j], fa);
        static_for<4>([&](auto r) {
          const float w = sa * ls[BB == 1 ? j * 16 + g * 4 + (int)r : 0];
          acc[i][j][(int)r] = __builtin_fmaf(t[(int)r], w, acc[i][j][(int)r]);
        });
      });
    });
  };
  static_for<R - 1>([&](auto q) { issue(q, q); });
  for (int j = 0; j < nloc; j += R) {
    static_for<R>([&](auto q) {
      wait_counts<(R - 2) * OPS, true>();
      issue(j + q + R - 1, std::integral_constant<int, (q + R - 1) % R>{});
      if (j + q < nloc) compute(q);
    });
  }
  wait_counts<0, true>();
  __syncthreads();
  // [WK][BM][BN + 4]: rows padded by 16 bytes, so that the 16 rows a store instruction writes
  // spread over the banks
  constexpr int PITCH = BN + 4;
  static_assert(sizeof(ring) >= sizeof(float) * WK * BM * PITCH, "partial sums fit the ring");
  float* part = reinterpret_cast<float*>(&ring[0][0][0]);
  static_for<RM>([&](auto i) {
    static_for<NBW>([&](auto j) {
      *reinterpret_cast<f32x4*>(&part[(wave * BM + i * 16 + x) * PITCH + j * 16 + g * 4]) = acc[i][j];
    });
  });
  __syncthreads();
  for (int q = tid; q < BM * BN; q += NT) {
    const int row = q / BN, c = q % BN;
    const int64_t m = s.m0 + row, n = s.n0 + c;
    if (m >= s.M || n >= p.N) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) sum += part[(w * BM + row) * PITCH + c];
    if (p.split_k > 1) p.workspace[((int64_t)blockIdx.y * p.M + m) * p.N + n] = sum;
    else finish_one<OT>(p, s, m, n, sum);
  }
}

// ------------------------------------------------------------------------------------------
// Ping-pong kernel, 256 x 256 outputs, 128-wide B scales, bf16 out: two groups of four waves, one
// wave of each on every SIMD, take turns between a read phase (fragments from LDS, DMA, scales)
// and a compute phase (matrix instructions and the multiply-adds of their sums), a barrier
// between phases; group 1 runs one phase behind group 0.  Group g computes rows [128 g, 128 g +
// 128), wave q of it columns [64 q, 64 q + 64).
//
// The accumulators (128 registers), the scales and the instruction's own sums leave no room for
// all fragments of a block, so a wave holds its B fragments and the first A fragments from the
// read phase and reads the other A fragments while it computes.  LDS (160 KiB): each A half in
// two slots, B in three.
//   * Half g of A(v) is read by group g in its read and compute phases of v (2v + g, 2v + g + 1).
//     Group g issues half g of A(v + 1) in its read phase of v -- the slot's last reader was its
//     compute phase of v - 1 -- and waits for it at the end of its compute phase of v.
//   * B(v) is read in phases 2v and 2v + 1.  Each group issues its half of B(v + 2) in its read
//     phase of v (the slot held B(v - 1)) and waits for it at the end of its read phase of v + 1.
// A read phase issues 3 scale loads, 4 DMAs of A and 4 of B, in that order, so "A(v + 1) is
// there" is at most 4 in flight at the end of the compute phase, and "B(v + 1) is there" at most
// 11 at the end of the read phase.  Blocks past the end are issued as zeros to keep the counts.
//
// 8192^3 takes 428 to 440 us (2,500 to 2,570 TFLOP/s): matrix units busy 72 % of the cycles at 1.75
// GHz, the board's power limit; the same tile with one barrier a block took 540.  Preferring the
// computing wave gave 3.5 %; an epilogue that stores 16-byte pieces 32 bytes apart cost 20 us.
// ------------------------------------------------------------------------------------------
template <class OT>
__global__ __launch_bounds__(512, 1) void scaled_pp(const SParams p) {
  constexpr int BM = 256, BN = 256, RM = 8, RN = 4, HALF = 128 * 8, B0 = 4 * HALF;
  __shared__ u32x4 lds[10 * HALF];
  STile s;
  if (!tile_share<BM, BN, OT>(p, s)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = wave >> 2, wq = wave & 3;
  const int x = lane & 15, c4 = lane >> 4;
  const char* a_tile = uniform_ptr((const char*)s.A + s.m0 * p.lda + s.k0);
  const char* b_tile = uniform_ptr((const char*)s.B + s.n0 * p.ldb + s.k0);
  const int64_t K = uniform_i64(s.k1 - s.k0);
  const int64_t a_span = uniform_i64((s.M - s.m0 - 1) * p.lda + K);
  const int64_t b_span = uniform_i64((p.N - s.n0 - 1) * p.ldb + K);
  const int nk = (int)((K + kSB - 1) / kSB);
  const int64_t kb0 = s.k0 / kSB;
  // scales of this lane's rows m0 + 128 g + 8 x .. + 7, and of this wave's columns
  const char* sa_base = uniform_ptr((const char*)(s.a_scale + s.m0 + kb0 * p.a_sk));
  const char* sb_base = uniform_ptr((const char*)(s.b_scale + min(s.n0 + wq * 64, p.N - 1) / kSB * p.b_sn + kb0 * p.b_sk));
  const int64_t sa_span = uniform_i64((s.M - s.m0) * 4);
  const uint32_t sa_off = (uint32_t)(g * 128 + x * 8) * 4;

  // LDS row i * 16 + x of an A half is its row x * 8 + i; row q * 64 + j * 16 + y of B the column of
  // Cols.  A wave issues blocks q, q + 4, q + 8, q + 12 (8 rows each) of a half: in A 2 rows apart in
  // the source, in B 32, 64 and 96 columns.
  const int prow = wq * 8 + (lane >> 3);
  const int chunk = (lane & 7) ^ row_key<8>(prow);
  const uint32_t a_off = (uint32_t)((g * 128 + (prow & 15) * 8 + (prow >> 4)) * p.lda) + chunk * 16;
  const uint32_t b_off = (uint32_t)((g * 128 + Cols<OT>::of(prow >> 4, (prow & 15) >> 2) + (prow & 3)) * p.ldb) + chunk * 16;

  f32x4 acc[RM][RN];
  static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { acc[i][j] = f32x4{}; }); });
  int slot[2];
  static_for<2>([&](auto u) { slot[u] = swizzled_slot<8>(x, c4 + 4 * u); });

  auto dma_a = [&](int t) {
    const int64_t k = (int64_t)t * kSB;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a_tile, a_span);
    u32x4* dst = lds + (g * 2 + (t & 1)) * HALF;
    uint32_t o = a_off;
    asm volatile("" : "+v"(o));   // formed here, not kept in more registers
    const bool in_k = k + chunk * 16 < K;
    static_for<4>([&](auto i) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(dst + (wq + 4 * i) * 64), 16,
                                               in_k ? o + (uint32_t)(2 * i * p.lda) : kOobOffset, (int)k, 0, 0);
    });
  };
  auto dma_b = [&](int t) {
    const int64_t k = (int64_t)t * kSB;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(b_tile, b_span);
    u32x4* dst = lds + B0 + (t % 3) * 2 * HALF + g * HALF;
    uint32_t o = b_off;
    asm volatile("" : "+v"(o));
    const bool in_k = k + chunk * 16 < K;
    static_for<4>([&](auto i) {
      constexpr int cols = Cols<OT>::of(2 * (i & 1), 0) + (i >> 1) * 64;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(dst + (wq + 4 * i) * 64), 16,
                                               in_k ? o + (uint32_t)(cols * p.ldb) : kOobOffset, (int)k, 0, 0);
    });
  };
  constexpr int HELD = 2;           // A fragments read in the read phase
  constexpr int LAG = 2;            // instructions between a sum and its addition
  Frag<u16> fa[RM], fb[RN];
  f32x4 sa0, sa1;
  float sb;
  auto read_a = [&](int t, auto i) {
    int at = (g * 2 + (t & 1)) * HALF;
    static_for<2>([&](auto u) { fa[i].w[u] = lds[at + slot[u] + i * 128]; });
  };
  auto phase_end = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    barrier_nofence();
    __builtin_amdgcn_sched_barrier(0);
  };
  if (nk > 0) {
    dma_a(0);
    dma_b(0);
    dma_b(1);
    wait_counts<0, true>();
    barrier_nofence();
    if (g == 1) phase_end();
    for (int v = 0; v < nk; ++v) {
      {
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(sa_base + (int64_t)v * p.a_sk * 4, sa_span);
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(sb_base + (int64_t)v * p.b_sk * 4, 4);
        sa0 = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, sa_off, 0, 0));
        sa1 = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, sa_off + 16, 0, 0));
        sb = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rb, 0, 0, 0));
      }
      __builtin_amdgcn_sched_barrier(0);
      static_for<RN>([&](auto j) {
        static_for<2>([&](auto u) { fb[j].w[u] = lds[B0 + (v % 3) * 2 * HALF + wq * 64 * 8 + slot[u] + j * 128]; });
      });
      static_for<HELD>([&](auto i) { read_a(v, i); });
      dma_a(v + 1);
      dma_b(v + 2);
      wait_counts<11, true>();
      phase_end();
      // compute phase: the sums of an instruction are added LAG instructions later, when they are
      // there; the wave is preferred to the one that reads
      __builtin_amdgcn_s_setprio(1);
      f32x4 t[LAG + 1];
      float w[RM];
      static_for<4>([&](auto i) {
        w[i] = sa0[(int)i] * sb;
        w[4 + i] = sa1[(int)i] * sb;
      });
      static_for<RM * RN + LAG>([&](auto n) {
        if constexpr (n % RN == 0 && n / RN + HELD < RM) read_a(v, std::integral_constant<int, n / RN + HELD>{});
        if constexpr (n < RM * RN) t[n % (LAG + 1)] = mfma_block(fb[n % RN], fa[n / RN]);
        if constexpr (n >= LAG) {
          constexpr int o = n - LAG, i = o / RN, j = o % RN;
          static_for<4>([&](auto r) {
            acc[i][j][(int)r] = __builtin_fmaf(t[o % (LAG + 1)][(int)r], w[i], acc[i][j][(int)r]);
          });
        }
      });
      static_for<RM * RN + LAG>([&](auto n) {
        if constexpr (n % RN == 0 && n / RN + HELD < RM) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        if constexpr (n < RM * RN) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if constexpr (n >= LAG) __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
      });
      __builtin_amdgcn_s_setprio(0);
      wait_counts<4, true>();
      phase_end();
    }
    if (g == 0) phase_end();
    wait_counts<0, true>();
  }
  store_outputs<OT, BN, RM, RN>(p, s, acc, [&](int i, int r) { return s.m0 + g * 128 + r * 8 + i; },
                                s.n0 + wq * 64, lds, wave);
}

// The planes of a split k, added in order, and the epilogue.
template <class OT>
__global__ __launch_bounds__(256) void scaled_join(const SParams p) {
  STile s;
  s.C = p.C;
  s.D = p.D;
  s.row_scale = p.row_scale;
  const int64_t MN = p.M * p.N;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < MN; e += (int64_t)gridDim.x * 256) {
    const int64_t row = e / p.N, col = e - row * p.N;
    float sum = 0.f;
    for (int q = 0; q < p.split_k; ++q) sum += p.workspace[q * MN + e];
    finish_one<OT>(p, s, row, col, sum);
  }
}

}  // namespace htk
