// int8.h -- gfx950 kernels of the products in 8-bit integers (htint8.h).
//
//   D(m, n) = act(((sum_k A(m, k) B(n, k)) * (alpha sA(m))) * sB(n) + beta C(m, n) + bias[n])
//
// The sum is one 32-bit integer accumulator, fed by v_mfma_i32_16x16x64_i8 (16 cycles of a SIMD's
// matrix unit, the rate of the 8-bit floats), and exact: slices and orders of k give the same bits (and
// so does every kernel, as all take the steps behind the sum alike, scaled_sum), and nothing but matrix
// instructions and fragment reads stands in the loop over k.
//
// Operands are swapped in the instruction, as in scaled.h: B's rows (n) are its A operand and A's
// rows (m) its B operand, so that a lane's four accumulators are four neighbouring n of one m.
// A and B are taken in blocks of 128 along k (an LDS row of 8 chunks of 16 bytes, XOR-swizzled);
// two instructions take a block: lane group g = lane / 16 supplies chunk g to the first and chunk
// 4 + g to the second.
//
// K need not be a multiple of 16: a chunk that K ends in is loaded whole, and A's bytes past K are
// cleared in the fragments of the last block.  Zeros in one operand are enough for integers.
#pragma once

#include "scaled.h"

namespace htk {

typedef int i32x4 __attribute__((ext_vector_type(4)));

template <> struct SOut<_Float16> {
  __device__ static float load(const void* p, int64_t i) { return (float)((const _Float16*)p)[i]; }
  __device__ static _Float16 bits(float v) { return (_Float16)v; }
};

__device__ __forceinline__ void mma_i8(i32x4& c, const u32x4& n, const u32x4& m) {
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, n), __builtin_bit_cast(i32x4, m), c, 0, 0, 0);
}

// The bytes of a chunk that lie below `left`; the others cleared.
__device__ __forceinline__ u32x4 keep_bytes(u32x4 w, int left) {
  static_for<4>([&](auto d) {
    const int l = left - 4 * d;
    w[(int)d] = l >= 4 ? w[(int)d] : l <= 0 ? 0u : w[(int)d] & (0xffffffffu >> (8 * (4 - l)));
  });
  return w;
}

// 16 bytes at any address of global memory, as one access.
__device__ __forceinline__ u32x4 load16(const void* p) {
  u32x4 w;
  __builtin_memcpy(&w, p, 16);
  return w;
}

// One output before its activation; sa is alpha times A's scale.  Every kernel takes these steps with
// these roundings, so that an output's bits do not depend on which it is: left to the compiler, some
// rounded the product with sb before the bias was added to it, and others did not.
template <bool HAS_C>
__device__ __forceinline__ float scaled_sum(int sum, float sa, float sb, float beta, float c, float bias) {
#pragma clang fp contract(off)
  const float t = (float)sum * sa;
  return HAS_C ? __builtin_fmaf(beta, c, t * sb) + bias : __builtin_fmaf(t, sb, bias);
}

// ------------------------------------------------------------------------------------------
// Outputs.  A lane has RM rows and in each RN pieces of 4 columns, dealt as Cols says, so that VO
// outputs are 16 bytes of D, loaded (C) and stored as one piece at any alignment (the memory system
// splits those that cross a line).  Waves whose columns all lie below N have a straight copy of the
// code for each activation (with C, for none and for any), with D's rows on whole lines and without;
// in the others (EDGE) a piece that N cuts goes element by element.  Nothing but C is loaded between
// the stores: a wave waits for its stores before it sees a later load (an edge path that took row
// blocks through LDS cost the 6 workgroups of the last columns 6 us: 333 x 4064 x 8192 31.9 us in place
// of 25.7).  With k in slices the integer sums go to the slice's plane.
// ------------------------------------------------------------------------------------------
// What a lane's outputs need besides their sums and C: scales of its rows and columns, and the bias of
// its pieces.  Kernels with registers to spare load it before their loop, so that a short product
// does not wait for memory once more at its end.
template <class OT, int RM, int RN> struct Finish {
  typedef Cols<OT> CM;
  static constexpr int VO = CM::VO, NQ = RN / CM::JP;
  float sa[RM];
  f32x4 sb[RN];
  u32x4 bias[NQ];

  // Columns of piece q (of the lane whose first column is col) below N.
  __device__ static __forceinline__ int left(const SParams& p, int64_t col, int q) {
    return (int)min(p.N - col - CM::of(q * CM::JP, 0), (int64_t)VO);
  }
  // 16 bytes of piece q of a row, zeros past N.
  template <bool EDGE>
  __device__ static __forceinline__ u32x4 piece(const SParams& p, const void* base, int64_t row, int64_t ld, int64_t col,
                                                int q) {
    const OT* src = (const OT*)base + row * ld + col + CM::of(q * CM::JP, 0);
    if (!EDGE || left(p, col, q) == VO) return load16(src);
    alignas(16) OT e[VO];
    static_for<VO>([&](auto i) { e[i] = i < left(p, col, q) ? src[(int)i] : OT(0); });
    u32x4 w;
    __builtin_memcpy(&w, e, 16);
    return w;
  }
  // Split products and those without k read no scales, waves past N nothing.
  template <class RowOf> __device__ __forceinline__ void load(const SParams& p, const STile& s, RowOf row_of, int64_t col0) {
    const int lane = threadIdx.x & 63, x = lane & 15, c4 = lane >> 4;
    static_for<RM>([&](auto i) { sa[i] = 0.f; });
    static_for<RN>([&](auto j) { sb[j] = f32x4{}; });
    static_for<NQ>([&](auto q) { bias[q] = u32x4{0, 0, 0, 0}; });
    if (col0 >= p.N || p.split_k > 1) return;
    const bool whole = col0 + 16 * RN <= p.N;
    if (p.K > 0) {
      static_for<RN>([&](auto j) {
        const int64_t n = col0 + CM::of(j, c4);
        if (whole) __builtin_memcpy(&sb[j], s.b_scale + n, 16);
        else static_for<4>([&](auto r) { sb[j][(int)r] = s.b_scale[min(n + r, p.N - 1)]; });
      });
      static_for<RM>([&](auto i) { sa[i] = s.a_scale[min(row_of(i, x), s.M - 1)]; });
    }
    if (p.bias) {
      const int64_t col = col0 + CM::of(0, c4);
      static_for<NQ>([&](auto q) {
        bias[q] = whole ? piece<false>(p, p.bias, 0, 0, col, q) : piece<true>(p, p.bias, 0, 0, col, q);
      });
    }
  }
};

// Stores of whole lines of 128 bytes go past the caches: 4096 x 4096 x 128 13.0 -> 11.6 us, 2048^3 16.3 ->
// 15.3, experts prefill 104 -> 101, 8192^3 403 -> 396 (a graph's runs, in turn).  Rows that lines do not fit
// go through them: 4001^3 66 us, streamed 70.  (Without the exchange of pieces below, a store has 64 bytes
// of 16 rows and none is streamed: 13.6, 16.1, 104 and 402.)
typedef u32x4 unaligned16 __attribute__((aligned(2)));
template <bool LINES> __device__ __forceinline__ void store_line(void* to, const u32x4& w, bool live) {
  if (!live) return;
  if constexpr (LINES) __builtin_nontemporal_store(w, reinterpret_cast<unaligned16*>(to));
  else *reinterpret_cast<unaligned16*>(to) = w;
}

template <class OT, int RM, int RN, int ACT, bool HAS_C, bool EDGE, bool LINES, class RowOf>
__device__ __forceinline__ void store_pieces(const SParams& p, const STile& s, const i32x4 (&acc)[RM][RN],
                                             const Finish<OT, RM, RN>& f, RowOf row_of, int64_t col, int x) {
  typedef Finish<OT, RM, RN> F;
  typedef Cols<OT> CM;
  constexpr int VO = F::VO, NQ = F::NQ, RG = RM % 2 == 0 ? 2 : 1;
  // once for all rows, and not where they are loaded: that would be a wait before the loop
  float sa[RM], bias[NQ][VO];
  static_for<RM>([&](auto i) { sa[i] = f.sa[i] * p.alpha; });
  static_for<NQ>([&](auto q) { static_for<VO>([&](auto e) { bias[q][e] = SOut<OT>::load(&f.bias[q], e); }); });
  // RG row blocks at a time, whose C is loaded before they are stored: D may be C, and more in hand at
  // once would not fit the registers
  static_for<RM / RG>([&](auto i0) {
    u32x4 c[RG][NQ];
    static_for<RG>([&](auto h) {
      const int64_t row = row_of(i0 * RG + h, x);
      static_for<NQ>([&](auto q) {
        c[h][q] = u32x4{0, 0, 0, 0};
        if constexpr (HAS_C)
          if (row < s.M) c[h][q] = F::template piece<EDGE>(p, s.C, row, p.ldc, col, q);
      });
    });
    static_for<RG>([&](auto h) {
      constexpr int i = i0 * RG + h;
      auto form = [&](auto q, OT (&o)[VO]) {
        static_for<VO>([&](auto e) {
          constexpr int j = q * CM::JP + e / 4, r = e % 4;
          const float y = scaled_sum<HAS_C>(acc[i][j][r], sa[i], f.sb[j][r], p.beta,
                                            HAS_C ? SOut<OT>::load(&c[h][q], e) : 0.f, bias[q][e]);
          o[e] = SOut<OT>::bits(ACT < 0    ? activate(p.act, y)
                                : ACT == 1 ? relu(y)
                                : ACT == 2 ? gelu(y)
                                : ACT == 3 ? silu(y)
                                           : y);
        });
      };
      if constexpr (!EDGE && NQ % 2 == 0) {
        // lanes x and x ^ 1 swap pieces, so that a store has 8 lanes on the even one's row and its 128
        // bytes, and the next store the odd one's
        const bool odd = x & 1;
        const int64_t even_row = row_of(i, x & ~1), odd_row = row_of(i, x | 1);
        static_for<NQ / 2>([&](auto half) {
          constexpr int q = 2 * half;
          alignas(16) OT o[2][VO];
          form(std::integral_constant<int, q>{}, o[0]);
          form(std::integral_constant<int, q + 1>{}, o[1]);
          u32x4 w[2], theirs;
          __builtin_memcpy(w, o, 32);
          static_for<4>([&](auto d) {
            const u32 give = odd ? w[0][(int)d] : w[1][(int)d];
            theirs[(int)d] = (u32)__builtin_amdgcn_update_dpp(0, (int)give, 0xb1, 0xf, 0xf, true);  // quad_perm:[1,0,3,2]
          });
          OT* to = (OT*)s.D + col + (odd ? CM::of((q + 1) * CM::JP, 0) : CM::of(q * CM::JP, 0));
          store_line<LINES>(to + even_row * p.ldd, odd ? theirs : w[0], even_row < s.M);
          store_line<LINES>(to + odd_row * p.ldd, odd ? w[1] : theirs, odd_row < s.M);
        });
      } else {
        const int64_t row = row_of(i, x);
        if (row < s.M) {
          OT* d = (OT*)s.D + row * p.ldd + col;
          static_for<NQ>([&](auto q) {
            alignas(16) OT o[VO];
            form(q, o);
            OT* to = d + CM::of(q * CM::JP, 0);
            const int left = EDGE ? F::left(p, col, q) : VO;
            if (!EDGE || left == VO) {
              __builtin_memcpy(to, o, 16);
            } else {
              static_for<VO>([&](auto e) {
                if (e < left) to[(int)e] = o[e];
              });
            }
          });
        }
      }
    });
  });
}

// col0: the wave's first column (at or past N for a wave that stores nothing); row_of(i, x): the row
// of row block i in lane x = lane % 16.
template <class OT, int RM, int RN, class RowOf>
__device__ __forceinline__ void store_sums(const SParams& p, const STile& s, const i32x4 (&acc)[RM][RN],
                                           const Finish<OT, RM, RN>& f, RowOf row_of, int64_t col0) {
  typedef Cols<OT> CM;
  const int lane = threadIdx.x & 63, x = lane & 15, c4 = lane >> 4;
  if (col0 >= p.N) return;
  if (p.split_k > 1) {
    int* plane = reinterpret_cast<int*>(p.workspace) + (int64_t)blockIdx.y * p.M * p.N + col0;
    static_for<RM>([&](auto i) {
      const int64_t row = row_of(i, x);
      if (row < s.M) {
        static_for<RN>([&](auto j) {
          int* to = plane + row * p.N + CM::of(j, c4);
          const int64_t left = p.N - col0 - CM::of(j, c4);
          if (left >= 4) __builtin_memcpy(to, &acc[i][j], 16);
          else static_for<4>([&](auto r) {
            if (r < left) to[(int)r] = acc[i][j][(int)r];
          });
        });
      }
    });
    return;
  }
  const int64_t col = col0 + CM::of(0, c4);
  auto go = [&](auto act, auto with_c, auto edge, auto lines) {
    store_pieces<OT, RM, RN, decltype(act)::value, decltype(with_c)::value, decltype(edge)::value, decltype(lines)::value>(
        p, s, acc, f, row_of, col, x);
  };
  constexpr std::integral_constant<int, -1> any_act{};
  constexpr std::integral_constant<int, 0> no_act{};
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  if (col0 + 16 * RN > p.N) {
    if (s.C) go(any_act, yes, yes, no);
    else go(any_act, no, yes, no);
    return;
  }
  auto whole = [&](auto lines) {
    if (s.C) {
      if (p.act == 0) go(no_act, yes, no, lines);
      else go(any_act, yes, no, lines);
    } else if (p.act == 0) go(no_act, no, no, lines);
    else if (p.act == 3) go(std::integral_constant<int, 3>{}, no, no, lines);
    else if (p.act == 2) go(std::integral_constant<int, 2>{}, no, no, lines);
    else go(std::integral_constant<int, 1>{}, no, no, lines);
  };
  if (((reinterpret_cast<uintptr_t>(s.D) | (uintptr_t)(p.ldd * (int64_t)sizeof(OT))) & 127) == 0) whole(yes);
  else whole(no);
}

// One output from its sum, its scales and its bias.
template <class OT>
__device__ __forceinline__ void finish_int(const SParams& p, const STile& s, int64_t row, int64_t col, int sum, float sa,
                                           float sb, float bias) {
  const float sa_alpha = sa * p.alpha;
  const float v = s.C ? scaled_sum<true>(sum, sa_alpha, sb, p.beta, SOut<OT>::load(s.C, row * p.ldc + col), bias)
                      : scaled_sum<false>(sum, sa_alpha, sb, 0.f, 0.f, bias);
  ((OT*)s.D)[row * p.ldd + col] = SOut<OT>::bits(activate(p.act, v));
}

// Spans of a tile's rows for the range checks: up to the end of the chunk that K ends in.
__device__ __forceinline__ int64_t row_span(int64_t rows, int64_t ld, int64_t K) {
  return uniform_i64((rows - 1) * ld + (K + 15) / 16 * 16);
}

// ------------------------------------------------------------------------------------------
// Any alignment: BM x BN tiles by 2 x 2 waves, chunks through registers (16-byte loads at any byte)
// into two LDS buffers, the loads of a block issued a block ahead, one barrier a block.  The rows
// are placed in LDS as in the tiled kernel below.  Loads of rows past M or N have clamped addresses;
// their outputs are not stored.  4096 x 4096 x 4095 without padding 123 us (rows on 16 bytes: 56), 333 x
// 4096 x 8191 45 (27), 16 x 4096 x 4095 in 8 slices 15 (7): a load's latency is hidden by one block
// only, and the chunks cross registers.
// ------------------------------------------------------------------------------------------
template <int BM, int BN, class OT, int OCC>
__global__ __launch_bounds__(256, OCC) void i8_any(const SParams p) {
  constexpr int TM = BM / 2, TN = BN / 2, RM = TM / 16, RN = TN / 16, ROWS = BM + BN, NCH = ROWS * 8 / 256;
  static_assert(BM % 32 == 0 && BN % 32 == 0, "a thread's chunk is A's or B's for all threads");
  __shared__ u32x4 lds[2 * ROWS * 8];
  STile s;
  if (!tile_share<BM, BN, OT>(p, s)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, x = lane & 15, g = lane >> 4;
  const int c = tid & 7;
  const u8* src[NCH];           // chunk c of this thread's rows, at k = k0
  static_for<NCH>([&](auto i) {
    const int R = (tid >> 3) + i * 32;
    if constexpr (i * 32 < BM) {
      const int w = R / TM, q = R % TM;
      src[i] = s.A + min(s.m0 + w * TM + (q & 15) * RM + (q >> 4), s.M - 1) * p.lda;
    } else {
      const int w = (R - BM) / TN, q = (R - BM) % TN, y = q & 15;
      src[i] = s.B + min(s.n0 + w * TN + Cols<OT>::of(q >> 4, y >> 2) + (y & 3), p.N - 1) * p.ldb;
    }
    src[i] += s.k0 + c * 16;
  });
  const int64_t K = s.k1 - s.k0;
  const int nk = (int)((K + kSB - 1) / kSB);
  u32x4 w[NCH];
  auto load = [&](int t) {
    const int64_t k = (int64_t)t * kSB;
    if (k + kSB <= K) {
      static_for<NCH>([&](auto i) { w[i] = load16(src[i] + k); });
      return;
    }
    const int left = (int)(K - k) - c * 16;     // bytes of this chunk below K
    static_for<NCH>([&](auto i) { w[i] = u32x4{0, 0, 0, 0}; });
    if (left >= 16) {
      static_for<NCH>([&](auto i) { w[i] = load16(src[i] + k); });
    } else if (left > 0 && s.k1 >= 16) {
      // the 16 bytes that end at K, moved down to the chunk's first bytes
      static_for<NCH>([&](auto i) {
        const u32x4 v = load16(src[i] + k + left - 16);
        uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
        const int bits = (16 - left) * 8;
        if (bits < 64) {
          lo = lo >> bits | hi << (64 - bits);
          hi >>= bits;
        } else {
          lo = hi >> (bits - 64);
          hi = 0;
        }
        w[i] = u32x4{(u32)lo, (u32)(lo >> 32), (u32)hi, (u32)(hi >> 32)};
      });
    } else if (left > 0) {                      // rows of less than 16 bytes
      static_for<NCH>([&](auto i) {
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int b = 0; b < left; ++b) {
          const uint64_t v = src[i][k + b];
          if (b < 8) lo |= v << (8 * b);
          else hi |= v << (8 * b - 64);
        }
        w[i] = u32x4{(u32)lo, (u32)(lo >> 32), (u32)hi, (u32)(hi >> 32)};
      });
    }
  };
  i32x4 acc[RM][RN];
  static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { acc[i][j] = i32x4{}; }); });
  if (nk > 0) load(0);
  auto row_of = [&](int i, int r) { return s.m0 + wm * TM + r * RM + i; };
  Finish<OT, RM, RN> finish;
  finish.load(p, s, row_of, s.n0 + wn * TN);
  for (int t = 0; t < nk; ++t) {
    u32x4* st = lds + (t & 1) * ROWS * 8;
    static_for<NCH>([&](auto i) { st[swizzled_slot<8>((tid >> 3) + i * 32, c)] = w[i]; });
    __syncthreads();            // behind it the other buffer has been read by all
    if (t + 1 < nk) load(t + 1);
    static_for<2>([&](auto u) {
      u32x4 fa[RM], fb[RN];
      static_for<RN>([&](auto j) { fb[j] = st[swizzled_slot<8>(BM + wn * TN + j * 16 + x, g + 4 * u)]; });
      static_for<RM>([&](auto i) { fa[i] = st[swizzled_slot<8>(wm * TM + i * 16 + x, g + 4 * u)]; });
      static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { mma_i8(acc[i][j], fb[j], fa[i]); }); });
    });
  }
  store_sums<OT, RM, RN>(p, s, acc, finish, row_of, s.n0 + wn * TN);
}

// ------------------------------------------------------------------------------------------
// Tiled kernel: BM x BN outputs by WM x WN waves, blocks of k in a ring of ST LDS stages filled by
// DMA, one barrier per block.  Rows are placed in LDS so that a lane's rows are neighbours and its
// outputs contiguous (scaled_tile in scaled.h).  KH = 2, for few tiles: two halves of the waves take
// the even and the odd blocks of k through rings of their own and join in LDS at the end.
//
// 333 x 4096 x 8192 26.5 us: 0.31 us for a block of 64 x 128, 744 cycles of which LDS moves 72 KiB in
// 576; only 192 of 256 CUs have a tile.  64 experts of 8 rows, N 2048, K 2048: 53 us, 5.1 TB/s of
// weights.  Tried in place of it: B's rows straight into registers, without LDS (42 us for the 333 rows: 16
// lanes that load from 16 rows take 16 cycles for each load); waves of 128 x 64 with blocks of 64 along
// k and two workgroups a CU (4096^3 70 us, the ping-pong kernel 56); 64 x 128 by two waves of 64 x 64 (68
// us for the experts), 64 x 256 and 32 x 256 tiles (within 4 % either way).
// ------------------------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int ST, class OT, int OCC, int KH>
__global__ __launch_bounds__(KH * WM * WN * 64, OCC) void i8_tile(const SParams p) {
  constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, RM = TM / 16, RN = TN / 16;
  constexpr int OPS = (BM + BN) / 8 / NW;            // DMA instructions per wave and block
  constexpr int STAGE = (BM + BN) * 8;               // 16-byte chunks
  static_assert((BM + BN) % (8 * NW) == 0 && NW % 2 == 0, "DMA blocks over the waves, one row key for a wave's");
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
  const int64_t a_span = row_span(s.M - s.m0, p.lda, K), b_span = row_span(p.N - s.n0, p.ldb, K);
  const int nk = (int)((K + kSB - 1) / kSB);
  const int cut = (int)(K & 15) ? (int)(K - (int64_t)(nk - 1) * kSB) : 0;   // bytes of a last block that ends in a chunk

  // DMA instruction i of this wave fills LDS rows 8 blk .. 8 blk + 7 (A's, then B's), blk =
  // wave + NW i: lane l row 8 blk + l / 8, slot l % 8, which holds chunk (l % 8) ^ key(row).
  uint32_t off[OPS];
  const int chunk = (lane & 7) ^ row_key<8>((wave & 1) * 8 + (lane >> 3));
  static_for<OPS>([&](auto i) {
    const int R = (wave + NW * i) * 8 + (lane >> 3);
    if (R < BM) {
      const int w = R / TM, q = R % TM;
      off[i] = (uint32_t)((w * TM + (q & 15) * RM + (q >> 4)) * p.lda) + chunk * 16;
    } else {
      const int w = (R - BM) / TN, q = (R - BM) % TN, y = q & 15;
      off[i] = (uint32_t)((w * TN + Cols<OT>::of(q >> 4, y >> 2) + (y & 3)) * p.ldb) + chunk * 16;
    }
  });
  // Step t of a half is block t KH + half.  Blocks past the last are issued as zeros, so that the
  // wait counts are the same throughout.
  auto dma = [&](int t, int stage) {
    u32x4* st = ring + stage * STAGE;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a_tile, a_span), rb = make_rsrc(b_tile, b_span);
    const int64_t k = (int64_t)(t * KH + half) * kSB;
    const bool in_k = k + chunk * 16 < K;
    const int sk = t * KH + half < nk ? (int)k : 0;
    static_for<OPS>([&](auto i) {
      const int blk = wave + NW * i;
      const uint32_t o = in_k ? off[i] : kOobOffset;
      if ((NW * i + NW) * 8 <= BM || blk * 8 < BM)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(st + blk * 64), 16, o, sk, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t*)(st + blk * 64), 16, o, sk, 0, 0);
    });
  };

  i32x4 acc[RM][RN];
  static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { acc[i][j] = i32x4{}; }); });
  int slot[2];
  static_for<2>([&](auto u) { slot[u] = swizzled_slot<8>(x, g + 4 * u); });

  auto compute = [&](int stage, bool last) {
    const u32x4* la = ring + stage * STAGE + wm * TM * 8;
    const u32x4* lb = ring + stage * STAGE + (BM + wn * TN) * 8;
    u32x4 fa[2][RM], fb[2][RN];
    static_for<2>([&](auto u) {
      static_for<RN>([&](auto j) { fb[u][j] = lb[j * 128 + slot[u]]; });
      static_for<RM>([&](auto i) { fa[u][i] = la[i * 128 + slot[u]]; });
    });
    if (last && cut)
      static_for<2>([&](auto u) { static_for<RM>([&](auto i) { fa[u][i] = keep_bytes(fa[u][i], cut - (g + 4 * u) * 16); }); });
    static_for<2>([&](auto u) {
      static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { mma_i8(acc[i][j], fb[u][j], fa[u][i]); }); });
    });
  };

  auto row_of = [&](int i, int r) { return s.m0 + wm * TM + r * RM + i; };
  const int64_t col0 = half == 0 ? s.n0 + wn * TN : p.N;
  Finish<OT, RM, RN> finish;
  finish.load(p, s, row_of, col0);
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
      if (KH == 1 || t * KH + half < nk) compute(stage, t * KH + half == nk - 1);
      if (++stage == ST) stage = 0;
    }
    wait_counts<0, true>();  // zero blocks issued past the end
  }
  if constexpr (KH == 2) {      // the second half's sums are added to the first's, which stores
    static_assert(NW * RM * RN * 64 <= KH * ST * STAGE, "its sums fit the ring");
    i32x4* sums = reinterpret_cast<i32x4*>(lds) + wave * RM * RN * 64 + lane;
    __syncthreads();
    if (half == 1) static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { sums[(i * RN + j) * 64] = acc[i][j]; }); });
    __syncthreads();
    if (half == 0) static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { acc[i][j] += sums[(i * RN + j) * 64]; }); });
  }
  store_sums<OT, RM, RN>(p, s, acc, finish, row_of, col0);
}

// ------------------------------------------------------------------------------------------
// Streaming kernel for few rows (decode): the cost is reading B once.  A workgroup owns 16 NBW
// columns and 16 RM rows; its WK waves take slices of k, each streaming its blocks of B (and the
// L2-resident rows of A) through a private LDS ring of R blocks by DMA, with no barrier in the
// loop.  The waves' sums meet in LDS.  16 x 16384 x 8192 takes 26.4 us, 5.1 TB/s of the 6.3 that a
// kernel reaches that only reads; 1 x 4096 x 4096 5.9 us, most of it the launch and one chain of loads.
// ------------------------------------------------------------------------------------------
template <int RM, int NBW, int WK, int R, class OT, int OCC>
__global__ __launch_bounds__(WK * 64, OCC) void i8_stream(const SParams p) {
  constexpr int BM = 16 * RM, BN = 16 * NBW, ROWS = BM + BN, OPS = ROWS / 8, BLK = ROWS * 8, NT = WK * 64;
  static_assert(R >= 2 && (R - 2) * OPS < 64, "vmcnt range");
  __shared__ u32x4 ring[WK][R][BLK];
  STile s;
  if (!tile_share<BM, BN, OT>(p, s)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int x = lane & 15, g = lane >> 4;
  const int64_t K = uniform_i64(s.k1 - s.k0);
  const int nb = (int)((K + kSB - 1) / kSB), per = (nb + WK - 1) / WK;
  const int b0 = wave * per, nloc = max(0, min(b0 + per, nb) - b0);
  const int cut = (int)(K & 15) ? (int)(K - (int64_t)(nb - 1) * kSB) : 0;

  const char* a_tile = uniform_ptr((const char*)s.A + s.m0 * p.lda + s.k0);
  const char* b_tile = uniform_ptr((const char*)s.B + s.n0 * p.ldb + s.k0);
  const int64_t a_span = row_span(s.M - s.m0, p.lda, K), b_span = row_span(p.N - s.n0, p.ldb, K);
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
  };
  // scales and bias of the outputs that this thread joins: before the loop, as they would otherwise be
  // one more wait for memory in a kernel of a few microseconds
  constexpr int NO = (BM * BN + NT - 1) / NT;
  float sa[NO], sb[NO], bias[NO];
  static_for<NO>([&](auto o) {
    const int q = min(tid + o * NT, BM * BN - 1);
    const int64_t m = min(s.m0 + q / BN, s.M - 1), n = min(s.n0 + q % BN, p.N - 1);
    const bool scaled = p.K > 0 && p.split_k <= 1;
    sa[o] = scaled ? s.a_scale[m] : 0.f;
    sb[o] = scaled ? s.b_scale[n] : 0.f;
    bias[o] = p.bias ? SOut<OT>::load(p.bias, n) : 0.f;
  });
  i32x4 acc[RM][NBW];
  static_for<RM>([&](auto i) { static_for<NBW>([&](auto j) { acc[i][j] = i32x4{}; }); });
  auto compute = [&](auto slot, bool last) {
    const u32x4* blk = &ring[wave][slot][0];
    u32x4 fa[2][RM], fb[2][NBW];
    static_for<2>([&](auto u) {
      static_for<NBW>([&](auto j) { fb[u][j] = blk[swizzled_slot<8>(j * 16 + x, g + 4 * u)]; });
      static_for<RM>([&](auto i) { fa[u][i] = blk[swizzled_slot<8>(BN + i * 16 + x, g + 4 * u)]; });
    });
    if (last && cut)
      static_for<2>([&](auto u) { static_for<RM>([&](auto i) { fa[u][i] = keep_bytes(fa[u][i], cut - (g + 4 * u) * 16); }); });
    static_for<2>([&](auto u) {
      static_for<RM>([&](auto i) { static_for<NBW>([&](auto j) { mma_i8(acc[i][j], fb[u][j], fa[u][i]); }); });
    });
  };
  static_for<R - 1>([&](auto q) { issue(q, q); });
  for (int j = 0; j < nloc; j += R) {
    static_for<R>([&](auto q) {
      wait_counts<(R - 2) * OPS, true>();
      issue(j + q + R - 1, std::integral_constant<int, (q + R - 1) % R>{});
      if (j + q < nloc) compute(q, b0 + j + q == nb - 1);
    });
  }
  wait_counts<0, true>();
  __syncthreads();
  // [WK][BM][BN + 4]: rows padded by 16 bytes, so that the 16 rows a store instruction writes
  // spread over the banks
  constexpr int PITCH = BN + 4;
  static_assert(sizeof(ring) >= sizeof(int) * WK * BM * PITCH, "partial sums fit the ring");
  int* part = reinterpret_cast<int*>(&ring[0][0][0]);
  static_for<RM>([&](auto i) {
    static_for<NBW>([&](auto j) {
      *reinterpret_cast<i32x4*>(&part[(wave * BM + i * 16 + x) * PITCH + j * 16 + g * 4]) = acc[i][j];
    });
  });
  __syncthreads();
  static_for<NO>([&](auto o) {
    const int q = tid + o * NT, row = q / BN, c = q % BN;
    const int64_t m = s.m0 + row, n = s.n0 + c;
    if (q < BM * BN && m < s.M && n < p.N) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < WK; ++w) sum += part[(w * BM + row) * PITCH + c];
      if (p.split_k > 1) reinterpret_cast<int*>(p.workspace)[((int64_t)blockIdx.y * p.M + m) * p.N + n] = sum;
      else finish_int<OT>(p, s, m, n, sum, sa[o], sb[o], bias[o]);
    }
  });
}

// ------------------------------------------------------------------------------------------
// Ping-pong kernel, 256 x 256 outputs: two groups of four waves, one wave of each on every SIMD,
// take turns between a read phase (the fragments of a block from LDS, DMA of later blocks) and a
// compute phase (64 matrix instructions), a barrier between phases; group 1 runs one phase behind.
// Group g computes rows [128 g, 128 g + 128), wave q of it columns [64 q, 64 q + 64).  LDS (160
// KiB): each A half in two slots, B in three; the units and their waits are those of gemm_pp
// (pingpong.h): group g issues A half 1 - g of block v + 1 + g and its half of B(v + 2) in its read
// phase of block v, 8 instructions, and lets at most those 8 be in flight at the end of it.
//
// 8192^3 takes 383 to 404 us on several cards (2,720 to 2,870 TOP/s; the library's int8 product reached
// 2,380): matrix units busy 78 % of the cycles at 1.8 GHz, the board's power limit.  Short products pay
// for the first blocks and the stores, which nothing overlaps (4096 x 4096 x 128, one block, 11.6 us, 7 of
// them the outputs): experts prefill, 8190 rows over 32, 97 to 105 us at 44 % busy.  Preferring the
// computing wave lost 0.5 to 4 %.  A form whose workgroups take several tiles, the next one's first blocks
// coming during the stores, spilled 248 registers (39 with both groups working in every tile, none without
// the epilogue, or with one tile) and was not run.
// ------------------------------------------------------------------------------------------
template <class OT>
__global__ __launch_bounds__(512, 1) void i8_pp(const SParams p) {
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
  const int64_t a_span = row_span(s.M - s.m0, p.lda, K), b_span = row_span(p.N - s.n0, p.ldb, K);
  const int nk = (int)((K + kSB - 1) / kSB);
  const int cut = (int)(K & 15) ? (int)(K - (int64_t)(nk - 1) * kSB) : 0;

  // LDS row i * 16 + x of an A half is its row x * 8 + i; row q * 64 + j * 16 + y of B the column of
  // Cols.  A wave issues blocks q, q + 4, q + 8, q + 12 (8 rows each) of a half: in A 2 rows apart in
  // the source, in B 32, 64 and 96 columns.
  const int prow = wq * 8 + (lane >> 3);
  const int chunk = (lane & 7) ^ row_key<8>(prow);
  const uint32_t a_off = (uint32_t)(((prow & 15) * 8 + (prow >> 4)) * p.lda) + chunk * 16;
  const uint32_t a_half = (uint32_t)(128 * p.lda);
  const uint32_t b_off = (uint32_t)((g * 128 + Cols<OT>::of(prow >> 4, (prow & 15) >> 2) + (prow & 3)) * p.ldb) + chunk * 16;

  i32x4 acc[RM][RN];
  static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { acc[i][j] = i32x4{}; }); });
  int slot[2];
  static_for<2>([&](auto u) { slot[u] = swizzled_slot<8>(x, c4 + 4 * u); });

  auto dma_a = [&](int half, int t) {   // half of A(t) into its slot t % 2
    const int64_t k = (int64_t)t * kSB;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a_tile, a_span);
    u32x4* dst = lds + (half * 2 + (t & 1)) * HALF;
    uint32_t o = a_off + (half ? a_half : 0u);
    asm volatile("" : "+v"(o));   // formed here, not kept in more registers
    const bool in_k = k + chunk * 16 < K;
    static_for<4>([&](auto i) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(dst + (wq + 4 * i) * 64), 16,
                                               in_k ? o + (uint32_t)(2 * i * p.lda) : kOobOffset, t < nk ? (int)k : 0, 0, 0);
    });
  };
  auto dma_b = [&](int t) {             // this group's half of B(t) into slot t % 3
    const int64_t k = (int64_t)t * kSB;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(b_tile, b_span);
    u32x4* dst = lds + B0 + (t % 3) * 2 * HALF + g * HALF;
    uint32_t o = b_off;
    asm volatile("" : "+v"(o));
    const bool in_k = k + chunk * 16 < K;
    static_for<4>([&](auto i) {
      constexpr int cols = Cols<OT>::of(2 * (i & 1), 0) + (i >> 1) * 64;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(dst + (wq + 4 * i) * 64), 16,
                                               in_k ? o + (uint32_t)(cols * p.ldb) : kOobOffset, t < nk ? (int)k : 0, 0, 0);
    });
  };
  // a group whose rows all lie past M (half of a group's last tiles) leaves the SIMDs to the other
  const bool works = s.m0 + g * 128 < s.M;
  u32x4 fa[2][RM], fb[2][RN];
  auto read_frags = [&](int t) {
    static_for<2>([&](auto u) {
      int ia = (g * 2 + (t & 1)) * HALF + slot[u], ib = B0 + (t % 3) * 2 * HALF + wq * 64 * 8 + slot[u];
      asm volatile("" : "+v"(ia), "+v"(ib));
      static_for<RM>([&](auto i) { fa[u][i] = lds[ia + i * 128]; });
      static_for<RN>([&](auto j) { fb[u][j] = lds[ib + j * 128]; });
    });
  };
  auto phase_end = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    barrier_nofence();
    __builtin_amdgcn_sched_barrier(0);
  };
  if (nk > 0) {
    if (g == 0) {
      dma_a(0, 0);
      dma_a(1, 0);
    } else {
      dma_a(0, 1);
    }
    dma_b(0);
    dma_b(1);
    wait_counts<0, true>();
    barrier_nofence();
    if (g == 1) phase_end();
    for (int v = 0; v < nk; ++v) {
      if (works) read_frags(v);
      dma_a(1 - g, v + 1 + g);
      dma_b(v + 2);
      if (v == nk - 1 && cut)
        static_for<2>([&](auto u) { static_for<RM>([&](auto i) { fa[u][i] = keep_bytes(fa[u][i], cut - (c4 + 4 * u) * 16); }); });
      wait_counts<8, true>();
      phase_end();
      if (works)
        static_for<2>([&](auto u) {
          static_for<RM>([&](auto i) { static_for<RN>([&](auto j) { mma_i8(acc[i][j], fb[u][j], fa[u][i]); }); });
        });
      phase_end();
    }
    if (g == 0) phase_end();
    wait_counts<0, true>();     // zero blocks issued past the end
  }
  auto row_of = [&](int i, int r) { return s.m0 + g * 128 + r * 8 + i; };
  Finish<OT, RM, RN> finish;
  finish.load(p, s, row_of, s.n0 + wq * 64);
  store_sums<OT, RM, RN>(p, s, acc, finish, row_of, s.n0 + wq * 64);
}

// The planes of a split k, added, and the epilogue.
template <class OT>
__global__ __launch_bounds__(256) void i8_join(const SParams p) {
  STile s;
  s.a_scale = p.a_scale;
  s.b_scale = p.b_scale;
  s.C = p.C;
  s.D = p.D;
  const int64_t MN = p.M * p.N;
  const int* planes = reinterpret_cast<const int*>(p.workspace);
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < MN; e += (int64_t)gridDim.x * 256) {
    const int64_t row = e / p.N, col = e - row * p.N;
    int sum = 0;
    for (int q = 0; q < p.split_k; ++q) sum += planes[q * MN + e];
    finish_int<OT>(p, s, row, col, sum, s.a_scale[row], s.b_scale[col], p.bias ? SOut<OT>::load(p.bias, col) : 0.f);
  }
}

typedef hipError_t (*int8_launch)(const SParams&, dim3, hipStream_t);

// The kernels in the order of int8.hip's table; each output type is instantiated in a file of its
// own (int8_bf16.hip, int8_f16.hip, int8_f32.hip), so that they build in parallel.
enum { I8_ANY64, I8_ANY128, I8_S16, I8_S16N, I8_S32, I8_S64, I8_T64, I8_T64K, I8_T128, I8_T128K, I8_PP, I8_JOIN, I8_COUNT };
struct Int8Launches {
  int8_launch go[I8_COUNT];
};
const Int8Launches& int8_bf16();
const Int8Launches& int8_f16();
const Int8Launches& int8_f32();

template <int BM, int BN, class OT, int OCC> hipError_t go_any(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((i8_any<BM, BN, OT, OCC>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}
template <int BM, int BN, int WM, int WN, int ST, int OCC, int KH, class OT>
hipError_t go_tile(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((i8_tile<BM, BN, WM, WN, ST, OT, OCC, KH>), grid, dim3(KH * WM * WN * 64), 0, s, p);
  return hipGetLastError();
}
template <int RM, int NBW, int WK, int R, int OCC, class OT>
hipError_t go_stream(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((i8_stream<RM, NBW, WK, R, OT, OCC>), grid, dim3(WK * 64), 0, s, p);
  return hipGetLastError();
}
template <class OT> hipError_t go_pp(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL(i8_pp<OT>, grid, dim3(512), 0, s, p);
  return hipGetLastError();
}
template <class OT> hipError_t go_join(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL(i8_join<OT>, grid, dim3(256), 0, s, p);
  return hipGetLastError();
}
template <class OT> const Int8Launches& int8_launches() {
  static const Int8Launches table = {
      {&go_any<64, 128, OT, 2>, &go_any<128, 128, OT, 2>, &go_stream<1, 2, 4, 3, 2, OT>, &go_stream<1, 1, 8, 4, 1, OT>,
       &go_stream<2, 2, 4, 3, 1, OT>, &go_stream<4, 2, 4, 3, 1, OT>, &go_tile<64, 128, 2, 2, 3, 2, 1, OT>,
       &go_tile<64, 128, 2, 2, 3, 1, 2, OT>, &go_tile<128, 128, 2, 2, 2, 2, 1, OT>,
       &go_tile<128, 128, 2, 2, 2, 1, 2, OT>, &go_pp<OT>, &go_join<OT>}};
  return table;
}

}  // namespace htk
