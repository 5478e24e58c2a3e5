// scaled.hip -- block-scaled e4m3 products: host side of htscaled.h's gemm_scaled_* and the
// instantiations of the kernels in scaled.h.
#include <cstring>
#include <new>

#include "../../include/htscaled.h"
#include "scaled.h"

using namespace htk;

namespace {

constexpr uint32_t kLive = 0x53434c44u, kDead = 0xdeadbeefu;
constexpr int64_t kCUs = 256;

typedef hipError_t (*scaled_launch)(const SParams&, dim3, hipStream_t);

// One kernel: its tile, and its launch for b_block 128 / 1 and bf16 / f32 outputs.
struct Variant {
  const char* name;
  int bm, bn, waves, lds, stream;
  scaled_launch launch[2][2];
};

template <int BM, int BN, int WM, int WN, int ST, int OCC, int BB, class OT>
hipError_t go_tile(const SParams& p, dim3 grid, hipStream_t s) {
  constexpr bool pipe = sizeof(OT) == 2;
  hipLaunchKernelGGL((scaled_tile<BM, BN, WM, WN, ST, BB, OT, OCC, pipe>), grid, dim3(WM * WN * 64), 0, s, p);
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

#define HT_TILE(NAME, BM, BN, WM, WN, ST, OCC)                                                    \
  {NAME, BM, BN, WM * WN, ST * (BM + BN) * 132, 0,                                                \
   {{&go_tile<BM, BN, WM, WN, ST, OCC, 128, u16>, &go_tile<BM, BN, WM, WN, ST, OCC, 128, float>}, \
    {&go_tile<BM, BN, WM, WN, ST, OCC, 1, u16>, &go_tile<BM, BN, WM, WN, ST, OCC, 1, float>}}}
#define HT_STREAM(NAME, RM, NBW, WK, R, OCC)                                                      \
  {NAME, 16 * RM, 16 * NBW, WK, WK * R * (16 * (RM + NBW) * 128 + (16 * (RM + NBW) + 63) / 64 * 256), 1, \
   {{&go_stream<RM, NBW, WK, R, OCC, 128, u16>, &go_stream<RM, NBW, WK, R, OCC, 128, float>},     \
    {&go_stream<RM, NBW, WK, R, OCC, 1, u16>, &go_stream<RM, NBW, WK, R, OCC, 1, float>}}}

enum { V_NARROW, V_S16, V_S16N, V_S32, V_S64, V_T64, V_T128, V_PP, V_COUNT };
const Variant kVariants[V_COUNT] = {
    {"narrow_64x64", 64, 64, 4, 16384, 0,
     {{&go_narrow<128, u16>, &go_narrow<128, float>}, {&go_narrow<1, u16>, &go_narrow<1, float>}}},
    HT_STREAM("stream_16x32_w4", 1, 2, 4, 3, 2),
    HT_STREAM("stream_16x16_w8", 1, 1, 8, 4, 1),
    HT_STREAM("stream_32x32_w4", 2, 2, 4, 3, 1),
    HT_STREAM("stream_64x32_w4", 4, 2, 4, 3, 1),
    HT_TILE("tile_64x128_w2x2", 64, 128, 2, 2, 3, 2),
    HT_TILE("tile_128x128_w2x2", 128, 128, 2, 2, 2, 2),
    {"pingpong_256x256", 256, 256, 8, 160 * 1024, 0, {{&go_pp, nullptr}, {nullptr, nullptr}}},
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

// Which kernel, by the rows an average product or group has.  (Rule re-measured with the kernels;
// see the figures at choose().)
void choose(gemm_scaled_s* h) {
  const gemm_scaled_desc& d = h->d;
  h->split = 1;
  h->per = up(d.K, kSB);
  if (!h->vec) {
    h->variant = V_NARROW;
    return;
  }
  const int64_t many = d.form == GEMM_SCALED_BATCH || d.form == GEMM_SCALED_K ? h->batch : 1;
  const double rows = d.form == GEMM_SCALED_ROWS ? double(d.M) / h->batch : double(d.M);
  if (rows <= 16) h->variant = up(d.N, 32) * row_tiles(*h, 16) * many >= kCUs ? V_S16 : V_S16N;
  else if (rows <= 32) h->variant = V_S32;
  else if (rows <= 64) h->variant = V_S64;
  else if (up(d.N, 256) * row_tiles(*h, 256) * many >= kCUs && rows > 128 && d.d_type == GEMM_BF16 &&
           d.b_block == kSB && d.a_scale_m == 1)
    h->variant = V_PP;
  else if (up(d.N, 128) * row_tiles(*h, 128) * many >= kCUs) h->variant = V_T128;
  else h->variant = V_T64;
  const Variant& v = kVariants[h->variant];
  if (d.form == GEMM_SCALED_SINGLE) {
    int64_t want = d.split_k;
    const int64_t blocks = up(d.K, kSB), tiles = up(d.M, v.bm) * up(d.N, v.bn);
    if (want == 0 && tiles > 0 && !v.stream) want = std::min<int64_t>(2 * kCUs / std::max<int64_t>(tiles, 1), blocks / 4);
    want = std::max<int64_t>(1, std::min(want, blocks));
    if (want > 1) {
      h->per = up(blocks, want);
      h->split = (int)up(blocks, h->per);
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
  info->grid = row_tiles(*h, v.bm) * up(h->d.N, v.bn) * h->split * (h->d.form == GEMM_SCALED_ROWS ? 1 : h->batch);
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
  const int64_t grid = row_tiles(*h, v.bm) * p.tiles_n;
  if (grid > INT32_MAX) return GEMM_ERR_INVALID_ARG;
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
