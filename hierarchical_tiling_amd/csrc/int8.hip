// int8.hip -- products in 8-bit integers: host side of htint8.h's gemm_int8_*.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/htint8.h"
#include "arch.h"
#include "int8.h"

using namespace htk;

namespace {

constexpr uint32_t kLive = 0x494e5438u, kDead = 0xdeadbeefu;
constexpr int64_t kCUs = 256;

// One kernel (of Int8Launches): its tile, whether it loads rows at any byte, and what choose() goes by:
// workgroups a CU holds at once (occ), waves (or halves of them) that share k (kw), microseconds for a
// block of 128 of k while a CU has one workgroup (c1) and while it has occ of them (c2), and for each
// round of workgroups beside them (round).  Measured on MI355X.
struct Cost {
  int occ, kw;
  float c1, c2, round;
};
struct Variant {
  const char* name;
  int bm, bn, waves, lds, any;
  Cost cost;
};

const Variant kVariants[] = {
    {"any_64x128", 64, 128, 4, 2 * 192 * 128, 1, {2, 1, 1.2f, 1.28f, 3.f}},
    {"any_128x128", 128, 128, 4, 2 * 256 * 128, 1, {2, 1, 1.6f, 1.75f, 4.f}},
    {"stream_16x32_w4", 16, 32, 4, 4 * 3 * 48 * 128, 0, {2, 4, .316f, .667f, 2.6f}},
    {"stream_16x16_w8", 16, 16, 8, 8 * 4 * 32 * 128, 0, {1, 8, .282f, .282f, 2.6f}},
    {"stream_32x32_w4", 32, 32, 4, 4 * 3 * 64 * 128, 0, {1, 4, .394f, .394f, 3.1f}},
    {"stream_64x32_w4", 64, 32, 4, 4 * 3 * 96 * 128, 0, {1, 4, .588f, .588f, 4.4f}},
    {"tile_64x128_w2x2", 64, 128, 4, 3 * 192 * 128, 0, {2, 1, .359f, .664f, 2.7f}},
    {"tile_64x128_w2x2x2", 64, 128, 8, 2 * 3 * 192 * 128, 0, {1, 2, .600f, .600f, 4.1f}},
    {"tile_128x128_w2x2", 128, 128, 4, 2 * 256 * 128, 0, {2, 1, .613f, .975f, 3.2f}},
    {"tile_128x128_w2x2x2", 128, 128, 8, 2 * 2 * 256 * 128, 0, {1, 2, .937f, .937f, 4.9f}},
    {"pingpong_256x256", 256, 256, 8, 160 * 1024, 0, {1, 1, 1.13f, 1.13f, 6.9f}},
};
constexpr int kCount = sizeof(kVariants) / sizeof(kVariants[0]);
static_assert(kCount == I8_JOIN, "the kernels of Int8Launches");

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t out_size(int d_type) { return d_type == GEMM_F32 ? 4 : 2; }

struct Pick {
  int variant;       // -1: none
  int split;         // slices of k
  int64_t per;       // blocks of k per slice
};

}  // namespace

struct gemm_int8_s {
  uint32_t magic;
  gemm_int8_desc d;
  int64_t batch;
  bool vec;          // leading dimensions and strides allow 16-byte DMA
  Pick pick, any;    // for bases on 16 bytes, and for others
};

namespace {

// Row tiles of a launch: for groups of rows the most that any offsets can need.
int64_t row_tiles(const gemm_int8_s& h, int bm) {
  const int64_t t = up(h.d.M, bm);
  return h.d.form == GEMM_INT8_ROWS ? std::min(h.d.M, h.d.M / bm + h.batch) : t;
}

// Workgroups of a launch along x, and whether a launch can have them: a dimension of one has fewer
// than 2^32 threads, and the runtime runs one with more as what is left modulo 2^32, without an error.
int64_t grid_x(const gemm_int8_s& h, const Variant& v) { return row_tiles(h, v.bm) * up(h.d.N, v.bn); }
bool fits(const gemm_int8_s& h, const Variant& v) { return grid_x(h, v) * v.waves * 64 <= int64_t(UINT32_MAX); }

// Expected row tiles of a launch, for groups of rows from a routing that spreads M rows over the
// groups: the groups that get any, and what a group's last tile leaves empty.
double expected_row_tiles(const gemm_int8_s& h, int bm) {
  const double M = double(h.d.M);
  if (h.d.form != GEMM_INT8_ROWS) return std::ceil(M / bm);
  const double hit = std::max(1.0, h.batch * (1.0 - std::exp(-M / h.batch)));
  return hit * std::max(1.0, M / hit / bm + 0.4);
}

// Predicted microseconds of a variant with k in `split` slices: rounds of workgroups at the cost of a
// block, against the time that the operands' bytes take at 6 TB/s (of the less of the two 0.41 counts:
// they overlap in part), plus the second kernel of a split.  The costs are fitted to 132 products and
// groups of rows (1 to 16384 rows, 512 to 14336 columns, k of 512 to 8192, 8 to 128 experts, each kernel
// and slices of k forced in turn), before stores went out in whole lines and a group of waves without rows
// did no work: then the choice was on average 0.4 % above the fastest and 7 % at most, with the kernels as
// they are 0.6 % and 17 % (16384 rows over 128 experts, 224 us for 191; the next 9 %, 3000 x 1024 x 8192).
double predict(const gemm_int8_s& h, const Variant& v, int split) {
  const gemm_int8_desc& d = h.d;
  const Cost& c = v.cost;
  const double many = d.form == GEMM_INT8_BATCH ? double(h.batch) : 1.0;
  const double wgs = expected_row_tiles(h, v.bm) * up(d.N, v.bn) * many * split;
  const double steps = std::ceil(std::ceil(double(d.K) / kSB) / split / c.kw);
  const double whole = std::floor(wgs / (kCUs * c.occ)), load = wgs / kCUs - whole * c.occ;  // last round's
  double last = 0.0;
  if (load > 0.0) last = steps * (c.c1 + (c.c2 - c.c1) * std::max(0.0, load - 1.0)) + c.round;
  const double work = 1.6 + whole * (steps * c.c2 + c.round) + last;
  const double hit = d.form == GEMM_INT8_ROWS ? h.batch * (1.0 - std::exp(-double(d.M) / h.batch)) : many;
  const double bytes = many * d.M * d.K + hit * d.N * d.K + many * d.M * d.N * double(out_size(d.d_type));
  const double mem = bytes / 6.0e6;
  double us = std::max(work, mem) + 0.41 * std::min(work, mem);
  if (split > 1) us += 2.6 + split * double(d.M) * d.N * 8.0 / 4.8e6;
  return us;
}

Pick with_split(const gemm_int8_s& h, int variant, int64_t want) {
  const int64_t blocks = std::max<int64_t>(up(h.d.K, kSB), 1);
  Pick p;
  p.variant = variant;
  p.per = up(blocks, std::max<int64_t>(1, std::min(want, blocks)));
  p.split = (int)up(blocks, p.per);
  return p;
}

// The variant (and, for one product, the split of k, up to `most`) with the least predicted time among
// those that load rows at any byte, or that need 16-byte rows.
Pick choose(const gemm_int8_s& h, bool any, int most) {
  const gemm_int8_desc& d = h.d;
  Pick best = with_split(h, -1, 1);
  double least = 0.0;
  for (int i = 0; i < kCount; ++i) {
    const Variant& v = kVariants[i];
    if ((v.any != 0) != any || !fits(h, v)) continue;
    for (int s = 1; s <= 16; s *= 2) {
      const bool forced = d.split_k > 0 || d.form != GEMM_INT8_SINGLE;
      if ((forced && s > 1) || s > most) break;
      if (s > 1 && s * 4 > up(d.K, kSB)) break;
      const int split = forced ? std::max(d.split_k, 1) : s;
      const double us = predict(h, v, split);
      if (best.variant < 0 || us < least) {
        least = us;
        best = with_split(h, i, split);
      }
    }
  }
  return best;
}

size_t plane_bytes(const gemm_int8_s& h, const Pick& p) {
  return p.split > 1 ? (size_t)p.split * (size_t)h.d.M * (size_t)h.d.N * 4 : 0;
}

}  // namespace

extern "C" {

int gemm_int8_create(const gemm_int8_desc* desc, gemm_int8_t* out) {
  if (!desc || !out) return GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  const gemm_int8_desc& d = *desc;
  constexpr int64_t kMost = INT32_MAX / 2;
  if (d.M < 0 || d.N < 0 || d.K < 0 || d.M > kMost || d.N > kMost || d.K > GEMM_INT8_MAX_K) return GEMM_ERR_INVALID_ARG;
  if (d.act < GEMM_ACT_NONE || d.act > GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
  if (d.form < GEMM_INT8_SINGLE || d.form > GEMM_INT8_ROWS) return GEMM_ERR_INVALID_ARG;
  for (int32_t f : {d.has_c, d.has_bias})
    if (f != 0 && f != 1) return GEMM_ERR_INVALID_ARG;
  if (d.split_k < 0 || d.split_k > 64 || (d.split_k > 1 && d.form != GEMM_INT8_SINGLE)) return GEMM_ERR_INVALID_ARG;
  if (d.form == GEMM_INT8_SINGLE ? (d.batch != 0 && d.batch != 1) : (d.batch < 1 || d.batch > 65535))
    return GEMM_ERR_INVALID_ARG;
  if (d.d_type != GEMM_BF16 && d.d_type != GEMM_F16 && d.d_type != GEMM_F32) return GEMM_ERR_DTYPE_COMBO;
  if (d.lda < d.K || d.ldb < d.K || d.ldd < d.N || (d.has_c && d.ldc < d.N)) return GEMM_ERR_LAYOUT;
  const bool batch = d.form == GEMM_INT8_BATCH, rows = d.form == GEMM_INT8_ROWS;
  if (batch && (d.a_stride_l < 0 || d.a_scale_l < 0 || d.d_stride_l < 0 || (d.has_c && d.c_stride_l < 0)))
    return GEMM_ERR_LAYOUT;
  if ((batch || rows) && (d.b_stride_l < 0 || d.b_scale_l < 0)) return GEMM_ERR_LAYOUT;
  if (batch && d.batch > 1 && d.d_stride_l == 0 && d.M > 0 && d.N > 0) return GEMM_ERR_INVALID_ARG;
  const int rc = arch_status();
  if (rc) return rc;
  gemm_int8_s h;
  std::memset(&h, 0, sizeof(h));
  h.d = d;
  h.batch = d.form == GEMM_INT8_SINGLE ? 1 : d.batch;
  // 16-byte loads: rows and products on 16 bytes, and a tile's rows within the 31 bits of a buffer
  // offset
  h.vec = d.lda % 16 == 0 && d.ldb % 16 == 0 && (!batch || d.a_stride_l % 16 == 0) &&
          (!(batch || rows) || d.b_stride_l % 16 == 0) && 257 * d.lda < (int64_t(1) << 31) &&
          257 * d.ldb < (int64_t(1) << 31);
  if (h.vec) h.pick = choose(h, false, 16);
  // for bases off 16 bytes in a handle for 16-byte rows: no more slices than its workspace holds
  const bool usual = h.vec && h.pick.variant >= 0;
  h.any = choose(h, true, usual ? h.pick.split : 16);
  if (!usual) h.pick = h.any;
  if (h.pick.variant < 0) return GEMM_ERR_INVALID_ARG;
  gemm_int8_s* p = new (std::nothrow) gemm_int8_s(h);
  if (!p) return GEMM_ERR_INVALID_ARG;
  p->magic = kLive;
  *out = p;
  return GEMM_OK;
}

int gemm_int8_workspace_size(gemm_int8_t h, size_t* bytes) {
  if (!h || h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  *bytes = plane_bytes(*h, h->pick);     // (of which h->any needs no more)
  return GEMM_OK;
}

int gemm_int8_get_info(gemm_int8_t h, gemm_int8_info* info) {
  if (!h || h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  if (!info) return GEMM_ERR_INVALID_ARG;
  const Variant& v = kVariants[h->pick.variant];
  std::memset(info, 0, sizeof(*info));
  info->bm = v.bm;
  info->bn = v.bn;
  info->waves = v.waves;
  info->lds_bytes = v.lds;
  info->split_k = h->pick.split;
  info->grid = grid_x(*h, v) * h->pick.split * (h->d.form == GEMM_INT8_BATCH ? h->batch : 1);
  std::strncpy(info->name, v.name, sizeof(info->name) - 1);
  return GEMM_OK;
}

int gemm_int8_run(gemm_int8_t h, const gemm_int8_args* a, void* stream) {
  if (!h || h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  if (!a) return GEMM_ERR_INVALID_ARG;
  const gemm_int8_desc& d = h->d;
  if ((d.form == GEMM_INT8_ROWS) != (a->offsets != nullptr)) return GEMM_ERR_INVALID_ARG;
  if (d.has_bias ? !a->bias && d.N > 0 : a->bias != nullptr) return GEMM_ERR_INVALID_ARG;
  if (!d.has_c && a->beta != 0.0f) return GEMM_ERR_INVALID_ARG;
  const bool read_c = d.has_c && a->beta != 0.0f;
  const size_t osz = out_size(d.d_type);
  if (!on(a->offsets, 4) || !on(a->bias, osz)) return GEMM_ERR_MISALIGNED;
  if (d.M == 0 || d.N == 0) return GEMM_OK;
  if (!a->D || (read_c && !a->C)) return GEMM_ERR_INVALID_ARG;
  if (d.K > 0 && (!a->A || !a->B || !a->a_scale || !a->b_scale)) return GEMM_ERR_INVALID_ARG;
  if (!on(a->D, osz) || (read_c && !on(a->C, osz)) || !on(a->a_scale, 4) || !on(a->b_scale, 4))
    return GEMM_ERR_MISALIGNED;
  const Pick& pick = h->vec && on(a->A, 16) && on(a->B, 16) ? h->pick : h->any;
  if (pick.variant < 0) return GEMM_ERR_INVALID_ARG;     // 2^32 threads with this alignment's tiles
  const Variant& v = kVariants[pick.variant];
  if (pick.split > 1 && (!a->workspace || !on(a->workspace, 16))) return GEMM_ERR_INVALID_ARG;
  SParams p;
  std::memset(&p, 0, sizeof(p));
  p.A = static_cast<const u8*>(a->A);
  p.B = static_cast<const u8*>(a->B);
  p.a_scale = a->a_scale;
  p.b_scale = a->b_scale;
  p.C = read_c ? a->C : nullptr;
  p.D = a->D;
  p.bias = a->bias;
  p.offsets = a->offsets;
  p.workspace = static_cast<float*>(a->workspace);
  p.M = d.M;
  p.N = d.N;
  p.K = d.K;
  p.lda = d.lda;
  p.ldb = d.ldb;
  p.ldc = d.ldc;
  p.ldd = d.ldd;
  p.a_sm = 1;
  p.a_l = d.a_stride_l;
  p.b_l = d.b_stride_l;
  p.c_l = d.c_stride_l;
  p.d_l = d.d_stride_l;
  p.as_l = d.a_scale_l;
  p.bs_l = d.b_scale_l;
  p.alpha = d.K > 0 ? a->alpha : 0.f;     // without k no alpha, were it infinite, reaches D
  p.beta = a->beta;
  p.act = d.act;
  p.form = d.form == GEMM_INT8_ROWS ? FORM_ROWS : d.form == GEMM_INT8_BATCH ? FORM_BATCH : FORM_SINGLE;
  p.groups = (int)h->batch;
  p.tiles_m = (int)up(d.M, v.bm);
  p.tiles_n = (int)up(d.N, v.bn);
  p.split_k = pick.split;
  p.blocks_per_split = (int)pick.per;
  const unsigned gz = d.form == GEMM_INT8_BATCH ? (unsigned)h->batch : 1;
  hipStream_t s = (hipStream_t)stream;
  const Int8Launches& l = d.d_type == GEMM_BF16 ? int8_bf16() : d.d_type == GEMM_F16 ? int8_f16() : int8_f32();
  if (l.go[pick.variant](p, dim3((unsigned)grid_x(*h, v), (unsigned)pick.split, gz), s) != hipSuccess) return GEMM_ERR_LAUNCH;
  if (pick.split > 1) {
    const dim3 blocks((unsigned)std::min<int64_t>(up(d.M * d.N, 256), 4096));
    if (l.go[I8_JOIN](p, blocks, s) != hipSuccess) return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

int gemm_int8_destroy(gemm_int8_t h) {
  if (!h) return GEMM_OK;
  if (h->magic != kLive) return GEMM_ERR_BAD_HANDLE;
  h->magic = kDead;
  delete h;
  return GEMM_OK;
}

}  // extern "C"
