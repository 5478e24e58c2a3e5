// scaled.hip -- block-scaled e4m3 products: host side of htscaled.h's gemm_scaled_* and the
// instantiations of the kernels in scaled.h.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/htscaled.h"
#include "arch.h"
#include "scaled.h"

using namespace htk;

namespace {

constexpr uint32_t kLive = 0x53434c44u, kDead = 0xdeadbeefu;
constexpr int64_t kCUs = 256;

typedef hipError_t (*scaled_launch)(const SParams&, dim3, hipStream_t);

// One kernel: its tile, its launch for b_block 128 / 1 and bf16 / f32 outputs, and what choose()
// goes by: workgroups a CU holds at once (occ), waves (or halves of them) that share k (kw),
// microseconds for a block of k while a CU has one workgroup (c1) and while it has occ of them (c2),
// for bf16 and f32 outputs, and for each round of workgroups beside them (round).  Measured on
// MI355X.
struct Cost {
  int occ, kw;
  float c1[2], c2[2], round;
};
struct Variant {
  const char* name;
  int bm, bn, waves, lds;
  Cost cost;
  scaled_launch launch[2][2];
};

template <int BM, int BN, int WM, int WN, int ST, int OCC, int KH, int BB, class OT>
hipError_t go_tile(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((scaled_tile<BM, BN, WM, WN, ST, BB, OT, OCC, KH>), grid, dim3(KH * WM * WN * 64), 0, s, p);
  return hipGetLastError();
}
template <int RM, int NBW, int WK, int R, int OCC, int BB, class OT>
hipError_t go_stream(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((scaled_stream<RM, NBW, WK, R, BB, OT, OCC>), grid, dim3(WK * 64), 0, s, p);
  return hipGetLastError();
}
template <int BB, class OT> hipError_t go_narrow(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((scaled_narrow<OT>), grid, dim3(256), 0, s, p, BB);
  return hipGetLastError();
}

hipError_t go_pp(const SParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL(scaled_pp<u16>, grid, dim3(512), 0, s, p);
  return hipGetLastError();
}

#define HT_TILE(NAME, BM, BN, WM, WN, ST, OCC, KH, ...)                                                   \
  {NAME, BM, BN, KH * WM * WN, KH * ST * (BM + BN) * 132, __VA_ARGS__,                                    \
   {{&go_tile<BM, BN, WM, WN, ST, OCC, KH, 128, u16>, &go_tile<BM, BN, WM, WN, ST, OCC, KH, 128, float>}, \
    {&go_tile<BM, BN, WM, WN, ST, OCC, KH, 1, u16>, &go_tile<BM, BN, WM, WN, ST, OCC, KH, 1, float>}}}
#define HT_STREAM(NAME, RM, NBW, WK, R, OCC, ...)                                                 \
  {NAME, 16 * RM, 16 * NBW, WK,                                                                   \
   WK * R * (16 * (RM + NBW) * 128 + (16 * (RM + NBW) + 63) / 64 * 256), __VA_ARGS__,             \
   {{&go_stream<RM, NBW, WK, R, OCC, 128, u16>, &go_stream<RM, NBW, WK, R, OCC, 128, float>},     \
    {&go_stream<RM, NBW, WK, R, OCC, 1, u16>, &go_stream<RM, NBW, WK, R, OCC, 1, float>}}}

enum { V_NARROW, V_S16, V_S16N, V_S32, V_S64, V_T64, V_T64K, V_T128, V_T128K, V_PP, V_COUNT };
#define HT_COST(...) {__VA_ARGS__}
const Variant kVariants[V_COUNT] = {
    {"narrow_64x64", 64, 64, 4, 16384, {2, 1, {3.f, 3.f}, {6.f, 6.f}, 2.f},
     {{&go_narrow<128, u16>, &go_narrow<128, float>}, {&go_narrow<1, u16>, &go_narrow<1, float>}}},
    HT_STREAM("stream_16x32_w4", 1, 2, 4, 3, 2, HT_COST(2, 4, {.38f, .42f}, {.80f, .90f}, 1.5f)),
    HT_STREAM("stream_16x16_w8", 1, 1, 8, 4, 1, HT_COST(1, 8, {.38f, .40f}, {.38f, .40f}, 2.f)),
    HT_STREAM("stream_32x32_w4", 2, 2, 4, 3, 1, HT_COST(1, 4, {.55f, .65f}, {.55f, .65f}, 3.f)),
    HT_STREAM("stream_64x32_w4", 4, 2, 4, 3, 1, HT_COST(1, 4, {1.0f, 1.2f}, {1.0f, 1.2f}, 3.f)),
    HT_TILE("tile_64x128_w2x2", 64, 128, 2, 2, 3, 2, 1, HT_COST(2, 1, {.43f, .80f}, {.72f, 1.30f}, 1.5f)),
    HT_TILE("tile_64x128_w2x2x2", 64, 128, 2, 2, 3, 1, 2, HT_COST(1, 2, {.72f, 1.30f}, {.72f, 1.30f}, 2.5f)),
    HT_TILE("tile_128x128_w2x2", 128, 128, 2, 2, 2, 2, 1, HT_COST(2, 1, {.72f, 1.25f}, {1.09f, 2.00f}, 1.5f)),
    HT_TILE("tile_128x128_w2x2x2", 128, 128, 2, 2, 2, 1, 2, HT_COST(1, 2, {1.09f, 2.00f}, {1.09f, 2.00f}, 3.f)),
    {"pingpong_256x256", 256, 256, 8, 160 * 1024, {1, 1, {1.40f, 0.f}, {1.40f, 0.f}, 6.f},
     {{&go_pp, nullptr}, {nullptr, nullptr}}},
};

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

struct gemm_scaled_s {
  uint32_t magic;
  gemm_scaled_desc d;
  int64_t batch;
  int variant;       // for operands the 16-byte loads can read
  int split;         // slices of k of that variant
  int64_t per;       // blocks of k per slice
  bool vec;          // leading dimensions, strides and K allow 16-byte loads
};

namespace {

// Row tiles of a launch: for groups of rows the most that any offsets can need.
int64_t row_tiles(const gemm_scaled_s& h, int bm) {
  const int64_t t = up(h.d.M, bm);
  return h.d.form == GEMM_SCALED_ROWS ? std::min(h.d.M, h.d.M / bm + h.batch) : t;
}

// Workgroups of a launch along x, and whether a launch can have them: a dimension of one has fewer
// than 2^32 threads, and the runtime runs one with more as what is left modulo 2^32, without an error.
int64_t grid_x(const gemm_scaled_s& h, const Variant& v) { return row_tiles(h, v.bm) * up(h.d.N, v.bn); }
bool fits(const gemm_scaled_s& h, const Variant& v) { return grid_x(h, v) * v.waves * 64 <= int64_t(UINT32_MAX); }

// Expected row tiles of a launch, for groups of rows from a routing that spreads M rows over the
// groups: the groups that get any, and what a group's last tile leaves empty.
double expected_row_tiles(const gemm_scaled_s& h, int bm) {
  const double M = double(h.d.M);
  if (h.d.form != GEMM_SCALED_ROWS) return std::ceil(M / bm);
  const double hit = std::max(1.0, h.batch * (1.0 - std::exp(-M / h.batch)));
  return hit * std::max(1.0, M / hit / bm + 0.4);
}

// Predicted microseconds of a variant with k in `split` slices: rounds of workgroups at the
// measured cost of a block, against the time that the operands' bytes take at 5.2 TB/s (the less of
// the two counts a quarter: they overlap, not fully), plus the second kernel of a split.  Over 80
// products and groups (1 to 14000 rows, 272 to 16384 columns, both output types, each kernel forced in
// turn: profiles/scaled_choice_check.txt) the choice was on average 4 % above the fastest kernel, 71 of
// them within 12 %; the worst, 1.4 to 1.5 times, are about 100 rows with a short k, which the streaming
// kernels do better than predicted, a group of 440 rows whose last tile of 256 is mostly empty, and
// fewer rows than groups.  A rule on rows alone (streaming kernels up to 64 rows, k split until 512
// workgroups) cost up to 2.3 times the fastest (1000 rows over 32 experts: 141 against 61 us).
double predict(const gemm_scaled_s& h, const Variant& v, int split) {
  const gemm_scaled_desc& d = h.d;
  const Cost& c = v.cost;
  const int f32 = d.d_type == GEMM_F32;
  const double many = d.form == GEMM_SCALED_BATCH || d.form == GEMM_SCALED_K ? double(h.batch) : 1.0;
  const double wgs = expected_row_tiles(h, v.bm) * up(d.N, v.bn) * many * split;
  const double k = d.form == GEMM_SCALED_K ? double(d.K) / h.batch : double(d.K);
  const double steps = std::ceil(std::ceil(k / kSB) / split / c.kw);
  const double whole = std::floor(wgs / (kCUs * c.occ)), load = wgs / kCUs - whole * c.occ;  // last round's
  double last = 0.0;
  if (load > 0.0) last = steps * (c.c1[f32] + (c.c2[f32] - c.c1[f32]) * std::max(0.0, load - 1.0)) + c.round;
  const double work = 2.0 + whole * (steps * c.c2[f32] + c.round) + last;
  const double hit = d.form == GEMM_SCALED_ROWS ? h.batch * (1.0 - std::exp(-double(d.M) / h.batch)) : many;
  const double a_many = d.form == GEMM_SCALED_BATCH ? many : 1.0, b_many = d.form == GEMM_SCALED_K ? 1.0 : hit;
  const double d_many = d.form == GEMM_SCALED_ROWS ? 1.0 : many;
  const double bytes = a_many * d.M * d.K + b_many * d.N * d.K + d_many * d.M * d.N * (f32 ? 4.0 : 2.0);
  const double mem = bytes / 5.2e6;
  double us = std::max(work, mem) + 0.25 * std::min(work, mem);
  if (split > 1) us += 6.0 + split * double(d.M) * d.N * 8.0 / 4.0e6;
  return us;
}

void set_split(gemm_scaled_s* h, int64_t want) {
  const int64_t blocks = std::max<int64_t>(up(h->d.K, kSB), 1);
  want = std::max<int64_t>(1, std::min(want, blocks));
  h->per = up(blocks, want);
  h->split = (int)up(blocks, h->per);
}

// The variant (and, for one product, the split of k) with the least predicted time.
void choose(gemm_scaled_s* h) {
  const gemm_scaled_desc& d = h->d;
  h->variant = V_NARROW;
  set_split(h, 1);
  if (!h->vec) return;
  const int bb = d.b_block == 1, f32 = d.d_type == GEMM_F32;
  double best = 0.0;
  for (int i = V_NARROW + 1; i < V_COUNT; ++i) {
    const Variant& v = kVariants[i];
    if (!v.launch[bb][f32] || (i == V_PP && d.a_scale_m != 1) || !fits(*h, v)) continue;
    for (int s = 1; s <= 16; s *= 2) {
      const bool forced = d.split_k > 0 || d.form != GEMM_SCALED_SINGLE;
      if (forced && s > 1) break;
      if (s > 1 && (s * 4 > up(d.K, kSB))) break;
      const double us = predict(*h, v, forced && d.split_k > 1 ? d.split_k : s);
      if (h->variant == V_NARROW || us < best) {
        best = us;
        h->variant = i;
        set_split(h, forced ? std::max(d.split_k, 1) : s);
      }
    }
  }
}

}  // namespace

extern "C" {

int gemm_scaled_create(const gemm_scaled_desc* desc, gemm_scaled_t* out) {
  if (!desc || !out) return GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  const gemm_scaled_desc& d = *desc;
  constexpr int64_t kMost = INT32_MAX / 2;
  if (d.M < 0 || d.N < 0 || d.K < 0 || d.M > kMost || d.N > kMost || d.K > kMost) return GEMM_ERR_INVALID_ARG;
  if (d.act < GEMM_ACT_NONE || d.act > GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
  if (d.form < GEMM_SCALED_SINGLE || d.form > GEMM_SCALED_K) return GEMM_ERR_INVALID_ARG;
  if (d.b_block != 1 && d.b_block != GEMM_SCALED_BLOCK) return GEMM_ERR_INVALID_ARG;
  for (int32_t f : {d.has_c, d.has_bias, d.has_row_scale})
    if (f != 0 && f != 1) return GEMM_ERR_INVALID_ARG;
  if (d.split_k < 0 || d.split_k > 64 || (d.split_k > 1 && d.form != GEMM_SCALED_SINGLE)) return GEMM_ERR_INVALID_ARG;
  if (d.form == GEMM_SCALED_SINGLE ? (d.batch != 0 && d.batch != 1) : (d.batch < 1 || d.batch > 65535))
    return GEMM_ERR_INVALID_ARG;
  if (d.d_type != GEMM_BF16 && d.d_type != GEMM_F32) return GEMM_ERR_DTYPE_COMBO;
  if (d.lda < d.K || d.ldb < d.K || d.ldd < d.N || (d.has_c && d.ldc < d.N)) return GEMM_ERR_LAYOUT;
  for (int64_t s : {d.a_scale_m, d.a_scale_k, d.b_scale_n, d.b_scale_k})
    if (s < 0) return GEMM_ERR_LAYOUT;
  const bool batch = d.form == GEMM_SCALED_BATCH, rows = d.form == GEMM_SCALED_ROWS, ks = d.form == GEMM_SCALED_K;
  if (batch && (d.a_stride_l < 0 || d.a_scale_l < 0)) return GEMM_ERR_LAYOUT;
  if ((batch || rows) && (d.b_stride_l < 0 || d.b_scale_l < 0)) return GEMM_ERR_LAYOUT;
  if ((batch || ks) && (d.d_stride_l < 0 || (d.has_c && d.c_stride_l < 0))) return GEMM_ERR_LAYOUT;
  if ((batch || ks) && d.batch > 1 && d.d_stride_l == 0 && d.M > 0 && d.N > 0) return GEMM_ERR_INVALID_ARG;
  const int rc = arch_status();
  if (rc) return rc;
  gemm_scaled_s h;
  std::memset(&h, 0, sizeof(h));
  h.d = d;
  h.batch = d.form == GEMM_SCALED_SINGLE ? 1 : d.batch;
  // 16-byte loads: whole chunks along k, rows and products on 16 bytes, and a tile's rows within
  // the 31 bits of a buffer offset
  h.vec = d.K % 16 == 0 && d.lda % 16 == 0 && d.ldb % 16 == 0 && (!batch || d.a_stride_l % 16 == 0) &&
          (!(batch || rows) || d.b_stride_l % 16 == 0) && 256 * d.lda + d.K < (int64_t(1) << 31) &&
          256 * d.ldb + d.K < (int64_t(1) << 31);
  choose(&h);
  if (!fits(h, kVariants[h.variant])) return GEMM_ERR_INVALID_ARG;
  gemm_scaled_s* p = new (std::nothrow) gemm_scaled_s(h);
  if (!p) return GEMM_ERR_INVALID_ARG;
  p->magic = kLive;
  *out = p;
  return GEMM_OK;
}

int gemm_scaled_workspace_size(gemm_scaled_t h, size_t* bytes) {
  if (!h || h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  *bytes = h->split > 1 ? (size_t)h->split * (size_t)h->d.M * (size_t)h->d.N * 4 : 0;
  return GEMM_OK;
}

int gemm_scaled_get_info(gemm_scaled_t h, gemm_scaled_info* info) {
  if (!h || h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  if (!info) return GEMM_ERR_INVALID_ARG;
  const Variant& v = kVariants[h->variant];
  std::memset(info, 0, sizeof(*info));
  info->bm = v.bm;
  info->bn = v.bn;
  info->waves = v.waves;
  info->lds_bytes = v.lds;
  info->split_k = h->split;
  info->grid = grid_x(*h, v) * h->split * (h->d.form == GEMM_SCALED_ROWS ? 1 : h->batch);
  std::strncpy(info->name, v.name, sizeof(info->name) - 1);
  return GEMM_OK;
}

int gemm_scaled_run(gemm_scaled_t h, const gemm_scaled_args* a, void* stream) {
  if (!h || h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  if (!a) return GEMM_ERR_INVALID_ARG;
  const gemm_scaled_desc& d = h->d;
  const bool groups = d.form == GEMM_SCALED_ROWS || d.form == GEMM_SCALED_K;
  if (groups != (a->offsets != nullptr)) return GEMM_ERR_INVALID_ARG;
  if ((d.has_bias != 0) != (a->bias != nullptr) || (d.has_row_scale != 0) != (a->row_scale != nullptr))
    return GEMM_ERR_INVALID_ARG;
  if (!d.has_c && a->beta != 0.0f) return GEMM_ERR_INVALID_ARG;
  const bool read_c = d.has_c && a->beta != 0.0f;
  const size_t osz = d.d_type == GEMM_F32 ? 4 : 2;
  if (!on(a->offsets, 4) || !on(a->bias, osz) || !on(a->row_scale, 4)) return GEMM_ERR_MISALIGNED;
  if (d.M == 0 || d.N == 0) return GEMM_OK;
  if (!a->D || (read_c && !a->C)) return GEMM_ERR_INVALID_ARG;
  if (d.K > 0 && (!a->A || !a->B || !a->a_scale || !a->b_scale)) return GEMM_ERR_INVALID_ARG;
  if (!on(a->D, osz) || (read_c && !on(a->C, osz)) || !on(a->a_scale, 4) || !on(a->b_scale, 4))
    return GEMM_ERR_MISALIGNED;
  const bool vec = h->vec && on(a->A, 16) && on(a->B, 16);
  const Variant& v = kVariants[vec ? h->variant : V_NARROW];
  const int split = vec ? h->split : 1;
  if (split > 1 && (!a->workspace || !on(a->workspace, 16))) return GEMM_ERR_INVALID_ARG;
  SParams p;
  std::memset(&p, 0, sizeof(p));
  p.A = static_cast<const u8*>(a->A);
  p.B = static_cast<const u8*>(a->B);
  p.a_scale = a->a_scale;
  p.b_scale = a->b_scale;
  p.C = read_c ? a->C : nullptr;
  p.D = a->D;
  p.bias = a->bias;
  p.row_scale = a->row_scale;
  p.offsets = a->offsets;
  p.workspace = static_cast<float*>(a->workspace);
  p.M = d.M;
  p.N = d.N;
  p.K = d.K;
  p.lda = d.lda;
  p.ldb = d.ldb;
  p.ldc = d.ldc;
  p.ldd = d.ldd;
  p.a_sm = d.a_scale_m;
  p.a_sk = d.a_scale_k;
  p.b_sn = d.b_scale_n;
  p.b_sk = d.b_scale_k;
  p.a_l = d.a_stride_l;
  p.b_l = d.b_stride_l;
  p.c_l = d.c_stride_l;
  p.d_l = d.d_stride_l;
  p.as_l = d.a_scale_l;
  p.bs_l = d.b_scale_l;
  p.alpha = a->alpha;
  p.beta = a->beta;
  p.act = d.act;
  p.form = d.form;
  p.groups = (int)h->batch;
  p.tiles_m = (int)up(d.M, v.bm);
  p.tiles_n = (int)up(d.N, v.bn);
  p.split_k = split;
  p.blocks_per_split = (int)h->per;
  if (!fits(*h, v)) return GEMM_ERR_INVALID_ARG;     // of a handle made for another alignment
  const int64_t grid = grid_x(*h, v);
  const unsigned gz = d.form == GEMM_SCALED_ROWS ? 1 : (unsigned)h->batch;
  hipStream_t s = (hipStream_t)stream;
  const int bb = d.b_block == 1, f32 = d.d_type == GEMM_F32;
  if (v.launch[bb][f32](p, dim3((unsigned)grid, (unsigned)split, gz), s) != hipSuccess) return GEMM_ERR_LAUNCH;
  if (split > 1) {
    const unsigned blocks = (unsigned)std::min<int64_t>(up(d.M * d.N, 256), 4096);
    if (f32) hipLaunchKernelGGL(scaled_join<float>, dim3(blocks), dim3(256), 0, s, p);
    else hipLaunchKernelGGL(scaled_join<u16>, dim3(blocks), dim3(256), 0, s, p);
    if (hipGetLastError() != hipSuccess) return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

int gemm_scaled_destroy(gemm_scaled_t h) {
  if (!h) return GEMM_OK;
  if (h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  h->magic = kDead;
  delete h;
  return GEMM_OK;
}

}  // extern "C"
