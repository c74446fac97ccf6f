// Host half of the C ABI of rotary positions, the 8-bit cache and attention
// over it (tern_rope*, tern_kv_* in tern.h): argument checks, workspace
// sizing, choice of kernel and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "internal.h"
#include "kv.h"

namespace {

tern_status fail(tern_status s, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return tern::record_failure(s, msg);
}

// A launch that would need too large a grid is not made, and says so.
#define KV_HIP(call)                                                                                                \
  do {                                                                                                              \
    hipError_t e_ = (call);                                                                                         \
    if (e_ == hipErrorInvalidConfiguration) return fail(TERN_E_UNSUPPORTED, "the call needs too many workgroups"); \
    if (e_ != hipSuccess) return fail(TERN_E_HIP, "%s: %s", #call, hipGetErrorString(e_));                          \
  } while (0)

#define KV_TRY(expr)              \
  do {                            \
    tern_status s_ = (expr);      \
    if (s_ != TERN_OK) return s_; \
  } while (0)

tern_status check_ptr(const void* p, const char* name, size_t align) {
  if (!p) return fail(TERN_E_INVAL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1)) return fail(TERN_E_ALIGN, "%s is not %zu-byte aligned", name, align);
  return TERN_OK;
}

// Rows of heads, `stride` elements apart.
tern_status check_rows(const void* p, int64_t stride, const char* name) {
  KV_TRY(check_ptr(p, name, 16));
  if (stride < 0) return fail(TERN_E_INVAL, "%s has the row stride %lld", name, (long long)stride);
  if (stride % 8) return fail(TERN_E_ALIGN, "%s has the row stride %lld, not a multiple of 8", name, (long long)stride);
  return TERN_OK;
}

tern_status check_rotary(const tern_rotary* r, int dim, const char* name) {
  if (r->rot < 0 || r->rot > dim || r->rot % 2)
    return fail(TERN_E_INVAL, "%s turns %d of %d elements", name, r->rot, dim);
  if (r->rot) KV_TRY(check_ptr(r->freq, "freq", 8));
  if (r->norm) KV_TRY(check_ptr(r->norm, "norm", 16));
  return TERN_OK;
}

tern::Rotary rotary_of(const tern_rotary* r) {
  tern::Rotary o = {};
  if (!r) return o;
  o.freq = r->freq;
  o.norm = r->norm;
  o.amp = r->amp;
  o.eps = r->eps;
  o.rot = r->rot;
  o.inter = r->interleaved != 0;
  o.on = 1;
  return o;
}

tern_status check_shape(const tern_kv* c) {
  if (!c) return fail(TERN_E_INVAL, "cache descriptor is NULL");
  if (c->heads < 1 || c->pages < 0) return fail(TERN_E_INVAL, "cache of %d heads, %d pages", c->heads, c->pages);
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(TERN_E_UNSUPPORTED, "head size %d is not 64, 128 or 256", c->dim);
  if (c->heads > 65535) return fail(TERN_E_UNSUPPORTED, "%d heads: 65535 at most", c->heads);
  return TERN_OK;
}

tern_status check_cache(const tern_kv* c) {
  KV_TRY(check_shape(c));
  if (!c->pages) return TERN_OK;
  KV_TRY(check_ptr(c->k, "k", 16));
  KV_TRY(check_ptr(c->v, "v", 16));
  KV_TRY(check_ptr(c->k_scale, "k_scale", 4));
  return check_ptr(c->v_scale, "v_scale", 4);
}

tern_status check_sizes(const tern_kv_batch* b) {
  if (!b) return fail(TERN_E_INVAL, "batch descriptor is NULL");
  if (b->count < 0 || b->rows < 0 || b->max_rows < 0 || b->max_len < 0 || b->max_pages < 0)
    return fail(TERN_E_INVAL, "batch of count=%d rows=%d max_rows=%d max_len=%d max_pages=%d", b->count, b->rows,
                b->max_rows, b->max_len, b->max_pages);
  if (b->rows > tern::kMaxRows || b->max_rows > tern::kMaxRows)
    return fail(TERN_E_UNSUPPORTED, "%d rows, %d of a sequence: %d at most", b->rows, b->max_rows, tern::kMaxRows);
  return TERN_OK;
}

tern_status check_batch(const tern_kv_batch* b) {
  KV_TRY(check_sizes(b));
  if (!b->start && (long long)b->count * b->max_rows != b->rows)
    return fail(TERN_E_INVAL, "%d sequences of %d rows are not %d rows", b->count, b->max_rows, b->rows);
  return TERN_OK;
}

// Whether a call has nothing to do.
bool nothing(const tern_kv_batch* b) { return !b->count || !b->rows || !b->max_rows; }

// The arrays of a batch with rows.
tern_status check_arrays(const tern_kv* c, const tern_kv_batch* b) {
  if (!c->pages) return fail(TERN_E_INVAL, "the cache has no pages");
  KV_TRY(check_cache(c));
  KV_TRY(check_ptr(b->len, "len", 4));
  if (b->start) KV_TRY(check_ptr(b->start, "start", 4));
  if (b->max_pages) KV_TRY(check_ptr(b->pages, "pages", 4));
  return TERN_OK;
}

tern::Cache cache_of(const tern_kv* c) { return {c->k, c->v, c->k_scale, c->v_scale, c->heads, c->pages}; }
int most_rows(const tern_kv_batch* b) { return std::min(b->max_rows, b->rows); }
tern::Batch batch_of(const tern_kv_batch* b) {
  return {b->start, b->len, b->pages, b->count, b->rows, most_rows(b), b->max_pages};
}

// Pages that a sequence's rows may lie in.
int items_of(const tern_kv_batch* b) { return (most_rows(b) + 2 * (tern::kPage - 1)) / tern::kPage; }

// Workgroups of 256 threads, one a (page, head) of the keys or the values; -1: more
// than a grid has.  The heads are divided by: all four sizes together pass 64 bits.
long long page_blocks(const tern_kv* c, const tern_kv_batch* b) {
  const long long pages = 2ll * b->count * items_of(b);
  return pages <= ((1 << 24) - 1) / c->heads ? pages * c->heads : -1;
}

// How attention runs.
struct AttnPlan {
  int blocks;  // of 16 rows in the kernel for few rows, 1 or 2; 0: tiles
  int pieces, whole, shares, parts, per, tiles, tile;
  bool join;
  size_t rows, info;  // of partial sums, and units whose pieces are noted
};
constexpr int kPieces = 2048;     // of the kernel for few rows: two wavefronts on each SIMD
// A unit is cut into at most so many pieces: more make the joining longer than
// the pieces shorter (us, pages a piece at least 1 / 2 / 3 / 4: one token of 8
// cache heads after 1000 tokens 8.9 / 10.2 / 12.4 / 13.1, 4000 10.9 / 11.3 / 12.6 /
// 14.7, 16000 18.8 / 16.1 / 15.1 / 16.0).
constexpr int kUnitPieces = 96;
// Units of so few pages are not cut: a page more costs a wavefront 1.5 us,
// joining 4.5 us.
constexpr int kWholePages = 3;
// Nor are units that are many for their pages: joining then costs more than
// the wait for the longest ones.  32 query heads over 8, ragged lengths,
// cut -> whole: 512 units of up to 8 pages 16.9 -> 15.9 us, of 16 20.4 -> 27.1;
// 1024 of 8 27.7 -> 19.0; 2048 of 16 71.9 -> 61.7, of 64 210 -> 231; 4096 of 32
// 220 -> 204, of 128 710 -> 764.  Four rows each, 1024 of 8: 40.5 -> 20.3.
constexpr int kWholeUnits = 64;  // for every page
// One block of rows: a workgroup of two, four or eight wavefronts, as many as the
// card holds for all units, has a whole unit where each wavefront then has at most
// a page more than a piece of the line, and few enough that uneven lengths do not
// count (us, line -> shared; 32 heads over 8 of 128 dimensions unless said): one sequence
// of 500, 1000 and 1500 tokens 8.6 -> 7.2, 8.8 -> 9.2, 9.2 -> 12.4; 32 of 500 and 1500
// 15.1 -> 9.7, 24.3 -> 19.9; 64 ragged ones of up to 500, 2000 and 8192 15.5 -> 12.4, 34.5 ->
// 33.4, 112 -> 122; 64 of up to 500, 16 heads over 4 of 256 dimensions, 17.4 -> 12.5.
constexpr int kSharePages = 12;
constexpr int kTileSlots = 1024;  // parts of tiles at most, where tiles are cut

// Pages that `rows` neighbouring rows see at most.
int pages_of(const tern_kv_batch* b, int window, int rows) {
  long long tokens = b->max_len;
  if (window > 0) tokens = std::min<long long>(tokens, (long long)window + rows + tern::kPage);
  return (int)((tokens + tern::kPage - 1) / tern::kPage);
}

// Parts for `groups` tiles of `rows` rows that see `pages` pages at most, `mean` on
// average, and their time, in us, by a model whose figures are fitted to
// measurements of 48 shapes (profiles/kv_attention_parts.txt: on average its choices
// are 0.3 % slower than the best ones, at most 4 %; on 32 shapes that the fit
// did not have 2.6 %, at most 22 %).  A page takes a workgroup `step`, or `share`
// times that where a CU has `holds` workgroups.  Tiles of different lengths fill CUs
// unevenly: more than 160 of them count as sharing CUs (with 256 in its place the
// 48 shapes' choices are 1.6 % slower than the best, at most 22 %, the 32 others'
// 2.2 %, at most 16 %).  Joining takes 1.5 and what the parts' sums take to be
// written and read.  Uncut and cut, us: 128-row tiles, 64 of 125 pages, 4 / 8 / 12
// parts 176 -> 56.1 / 47.0 / 52.7; 16 of 63 pages, 8 / 16 / 32 parts 96.0 -> 22.6 / 20.5 /
// 23.6; a prompt of 2048, 128 tiles, 4 / 6 / 8 parts 52.7 -> 35.1 / 31.9 / 41.6.  Tiles of
// 64 and of 128 rows, us, each at its best number of
// parts: prompts of 256, 512, 1024 and 4096 tokens 10.1 and 13.1, 15.1 and 19.5, 25.5
// and 30.9, 80 and 65; 64 sequences of 40 rows 35.7 and 44.0; 512 rows after 7500
// tokens 114 and 88.8; 8192 rows 789 and 592.
struct Cost {
  double step, share;
  int holds;
};
constexpr Cost kMidCost[3] = {{0.8, 1.9, 4}, {1.25, 1.33, 2}, {1.95, 1.15, 1}};  // of 64, 128, 256 dimensions
constexpr Cost kTileCost[3] = {{1.05, 1.4, 2}, {1.5, 1.37, 2}, {2.75, 1.0, 1}};
int parts_for(long long groups, int pages, double mean, int dim, int rows, double& least) {
  const Cost c = (rows == tern::kAttnMid ? kMidCost : kTileCost)[dim / 128];
  const int slots = 256 * c.holds, alone = mean < pages - 1 ? 160 : 256;
  int best = 1;
  least = 1e30;
  for (int n = 1; n == 1 || (n <= pages && groups * n <= kTileSlots); n += 1 + n / 8) {
    const int per = (pages + n - 1) / n;
    const double all = groups * std::min<double>(n, mean / per);  // workgroups that have pages
    double us = std::max(1.0, all <= alone ? 1.0 : std::ceil(all / slots) * c.share) * per * c.step;
    if (n == 1) us = std::max(std::min(us, groups * mean * c.step * c.share / slots), pages * c.step);  // long tiles first
    if (n > 1) us += 1.5 + 1.3e-6 * groups * n * dim * rows;
    if (us < least) {
      least = us;
      best = n;
    }
  }
  return best;
}

// Rows up to which a unit goes to the kernel for few rows; above one block of 16
// only where there are more pages than kFewPages, which it reads faster.  us, few
// rows / tiles: 4 sequences of 8 cache heads of 256 dimensions, 20 rows each, after
// 3000 tokens (1500 pages) 36 / 25, 8 after 8000 (8000 pages) 78 / 87; of 128 dimensions,
// 32 rows each, 1 after 4000 (504) 16.7 / 11.6, 4 after 8000 (4000) 27.9 / 26.4, 256 after
// 500 (16384) 62 / 78; 20 rows each, 4 ragged ones of up to 120000 (60000) 153 / 206; 64
// rows each, 8 after 8000, four blocks, not kept, 75 / 48.
constexpr int kFewRows = 32, kFewPages = 4096;

thread_local int g_tile_rows = 0;  // of this thread's tiles, 0: by the rule

// One kernel serves a call, that of its longest sequence: the host does not know
// the others' rows.  Single tokens beside a prompt's chunk then walk their pages on
// tiles, a workgroup each (us, together and in two calls: 63 tokens after up to 8192
// beside 2048 rows after 1000 476 and 190, 31 after up to 2000 beside 512 rows 64 and 34).
AttnPlan plan_of(const tern_kv* c, const tern_kv_batch* b, int group, int window, bool causal) {
  AttnPlan p = {};
  const long long rows = (long long)most_rows(b) * group, units = (long long)b->count * c->heads;
  const int pages = pages_of(b, window, most_rows(b));
  if (rows <= tern::kAttnFew || (rows <= kFewRows && units * pages > kFewPages)) {
    p.blocks = rows <= 16 ? 1 : 2;
    const int waves = p.blocks * c->dim > 128 ? kPieces / 2 : kPieces, line = (int)((units * pages + waves - 1) / waves);
    p.shares = 1;
    if (p.blocks == 1)
      for (int w = 2; w <= (c->dim > 128 ? 4 : 8); w *= 2)
        if (units * w <= (c->dim == 64 ? 2 * waves : waves)) p.shares = w;  // four wavefronts a SIMD at 64 dimensions
    const int each = (pages + p.shares - 1) / p.shares;
    if (each > line + 1 || each > kSharePages) p.shares = 1;
    p.whole = p.shares > 1 || pages <= kWholePages || units >= (long long)kWholeUnits * pages;
    p.pieces = (int)(p.whole ? units : std::min<long long>(waves, units * pages));
    p.per = (pages + kUnitPieces - 1) / kUnitPieces;
    p.join = !p.whole;
    p.rows = p.join ? (size_t)p.pieces * 2 * rows : 0;
    p.info = p.join ? units : 0;
    return p;
  }
  double least = 1e30;
  const int only = g_tile_rows;
  for (const int tile : {tern::kAttnMid, tern::kAttnTile}) {
    if (only && tile != only) continue;
    const int tiles = (int)((rows + tile - 1) / tile), tokens = std::min(most_rows(b), (tile - 1) / group + 2);
    const int pages = std::max(1, pages_of(b, window, tokens));
    const double fewer = causal && !window ? 0.5 * (most_rows(b) - tokens) / tern::kPage : 0.0;
    double us = 0.0;
    const int n = parts_for(tiles * units, pages, std::max(1.0, pages - fewer), c->dim, tile, us);
    if (us >= least) continue;
    least = us;
    p.tile = tile;
    p.tiles = tiles;
    p.per = (pages + n - 1) / n;
    p.parts = (pages + p.per - 1) / p.per;
  }
  p.join = p.parts > 1;
  p.rows = p.join ? (size_t)p.tiles * units * p.parts * p.tile : 0;
  return p;
}

size_t attn_need(const AttnPlan& p, const tern_kv* c) { return p.rows * (c->dim + 2) * 4 + p.info * 8; }

// The most that any batch with no more sequences and rows and no larger
// max_len needs: few rows leave at most kPieces pairs of slots, tiles kTileSlots
// parts.
size_t attn_need_upto(const tern_kv* c, const tern_kv_batch* b, int group) {
  const double rows = (double)b->rows * group, pages = pages_of(b, 0, 0);
  const double few = 2.0 * std::min<double>(kPieces, (double)b->count * c->heads * pages) * std::min<double>(rows, kFewRows);
  const double groups = (double)b->count * c->heads * std::ceil(rows / tern::kAttnMid);
  const double tiles = rows <= tern::kAttnFew ? 0.0 : std::min<double>(groups * pages, kTileSlots) * tern::kAttnTile;
  return (size_t)(std::max(few, tiles) * (c->dim + 2) * 4) + (size_t)b->count * c->heads * 8;
}

tern_status check_heads(const tern_kv* c, const tern_kv_batch* b, int q_heads) {
  if (q_heads < 1 || q_heads % c->heads)
    return fail(TERN_E_INVAL, "%d query heads over %d cache heads", q_heads, c->heads);
  if (q_heads > 65535 || (long long)b->max_rows * (q_heads / c->heads) > (1 << 30))
    return fail(TERN_E_UNSUPPORTED, "%d query heads, %d rows of a sequence: too many", q_heads, b->max_rows);
  if ((long long)b->count * c->heads > (1 << 24) || (long long)b->count * c->heads * b->max_pages > 0x7fffffff)
    return fail(TERN_E_UNSUPPORTED, "%d cache heads of %d sequences, %d pages: too many", c->heads, b->count, b->max_pages);
  return TERN_OK;
}

}  // namespace

extern "C" {

tern_status tern_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double low, double high,
                                  int32_t trained, double* freq, float* amp) {
  if (rot < 0 || rot % 2) return fail(TERN_E_INVAL, "rot=%d must be even", rot);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(TERN_E_INVAL, "base=%g must be above 1", base);
  if (rot && !freq) return fail(TERN_E_INVAL, "freq is NULL");
  if (!amp) return fail(TERN_E_INVAL, "amp is NULL");
  if (scaling < TERN_ROPE_PLAIN || scaling > TERN_ROPE_WAVES) return fail(TERN_E_UNSUPPORTED, "unknown scaling %d", scaling);
  if (scaling != TERN_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(TERN_E_INVAL, "factor=%g must be 1 or more", factor);
  const bool bands = scaling == TERN_ROPE_RAMP || scaling == TERN_ROPE_WAVES;
  if (bands && (!(low > 0.0) || !(high > low) || !std::isfinite(high) || trained < 1))
    return fail(TERN_E_INVAL, "low=%g, high=%g, trained=%d: 0 < low < high and a length are wanted", low, high, trained);
  const double turn = 2.0 * M_PI;
  if (scaling == TERN_ROPE_BASE && rot > 2) base *= std::pow(factor, (double)rot / (rot - 2));
  // the pair (as a real number) that turns `turns` times in the trained length
  auto pair_of = [&](double turns) { return 0.5 * rot * std::log(trained / (turns * turn)) / std::log(base); };
  const double first = bands ? std::max(0.0, std::floor(pair_of(high))) : 0.0;
  const double last = bands ? std::min(rot - 1.0, std::ceil(pair_of(low))) : 0.0;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    double keep = 1.0;  // of f; the rest is f / factor
    if (scaling == TERN_ROPE_LINEAR) keep = 0.0;
    if (scaling == TERN_ROPE_RAMP) keep = 1.0 - std::min(1.0, std::max(0.0, (i - first) / std::max(last - first, 1e-3)));
    if (scaling == TERN_ROPE_WAVES) keep = std::min(1.0, std::max(0.0, (trained * f / turn - low) / (high - low)));
    freq[i] = f * keep + f / (scaling == TERN_ROPE_BASE ? 1.0 : factor) * (1.0 - keep);
    if (keep == 1.0) freq[i] = f;
  }
  *amp = scaling == TERN_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return TERN_OK;
}

tern_status tern_rope(const uint16_t* x, int64_t x_stride, int32_t m, int32_t heads, int32_t dim, const int32_t* pos,
                      const tern_rotary* r, uint16_t* out, int64_t out_stride, void* stream) {
  if (m < 0 || heads < 0 || dim < 0) return fail(TERN_E_INVAL, "m=%d heads=%d dim=%d", m, heads, dim);
  if (dim % 8 || dim > 512) return fail(TERN_E_UNSUPPORTED, "head size %d is no multiple of 8 up to 512", dim);
  if (!r) return fail(TERN_E_INVAL, "rotary descriptor is NULL");
  if (!m || !heads || !dim) return TERN_OK;
  KV_TRY(check_rows(x, x_stride, "x"));
  KV_TRY(check_rows(out, out_stride, "out"));
  if (m > 1 && out_stride < (int64_t)heads * dim)
    return fail(TERN_E_INVAL, "rows of out overlap: %d heads of %d, %lld apart", heads, dim, (long long)out_stride);
  if (m > 1 && out == x && out_stride != x_stride)
    return fail(TERN_E_INVAL, "out is x with the row stride %lld, not %lld", (long long)out_stride, (long long)x_stride);
  KV_TRY(check_ptr(pos, "pos", 4));
  KV_TRY(check_rotary(r, dim, "rotary"));
  tern::RopeArgs a = {};
  a.x = x;
  a.out = out;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.pos = pos;
  a.r = rotary_of(r);
  a.m = m;
  a.heads = heads;
  a.dim = dim;
  KV_HIP(tern::launch_rope(a, (hipStream_t)stream));
  return TERN_OK;
}

tern_status tern_kv_check(const tern_kv* c) { return check_cache(c); }

tern_status tern_kv_write(const tern_kv* c, const tern_kv_batch* b, const uint16_t* k, int64_t k_stride,
                          const uint16_t* v, int64_t v_stride, const tern_rotary* rope, const uint16_t* q,
                          int64_t q_stride, int32_t q_heads, const tern_rotary* q_rope, uint16_t* q_out, void* stream) {
  KV_TRY(check_shape(c));
  KV_TRY(check_batch(b));
  if (rope) KV_TRY(check_rotary(rope, c->dim, "rope"));
  if (q) {
    if (!q_rope) return fail(TERN_E_INVAL, "q_rope is NULL");
    KV_TRY(check_rotary(q_rope, c->dim, "q_rope"));
    if (q_heads < 0 || q_heads > (1 << 20)) return fail(TERN_E_INVAL, "%d query heads", q_heads);
  }
  if (nothing(b)) return TERN_OK;
  KV_TRY(check_arrays(c, b));
  KV_TRY(check_rows(k, k_stride, "k"));
  KV_TRY(check_rows(v, v_stride, "v"));
  if (q && q_heads) {
    KV_TRY(check_rows(q, q_stride, "q"));
    KV_TRY(check_ptr(q_out, "q_out", 16));
    if (b->rows > 1 && q_out == q && q_stride != (int64_t)q_heads * c->dim)
      return fail(TERN_E_INVAL, "q_out is q, whose rows are %lld apart", (long long)q_stride);
  }
  tern::WriteArgs a = {};
  a.c = cache_of(c);
  a.b = batch_of(b);
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.rk = rotary_of(rope);
  if (q && q_heads) {
    a.q = q;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.q_heads = q_heads;
    a.rq = rotary_of(q_rope);
  }
  a.items = items_of(b);
  const long long blocks = page_blocks(c, b);
  if (blocks < 0) return fail(TERN_E_UNSUPPORTED, "the call needs too many workgroups");
  a.kv_blocks = (int)blocks;
  KV_HIP(tern::launch_kv_write(a, c->dim, (hipStream_t)stream));
  return TERN_OK;
}

tern_status tern_kv_read(const tern_kv* c, const tern_kv_batch* b, void* k, void* v, int32_t dtype, void* stream) {
  KV_TRY(check_shape(c));
  KV_TRY(check_batch(b));
  if (dtype != TERN_F16 && dtype != TERN_F32) return fail(TERN_E_UNSUPPORTED, "unknown output dtype %d", dtype);
  if (nothing(b) || (!k && !v)) return TERN_OK;
  KV_TRY(check_arrays(c, b));
  if (k) KV_TRY(check_ptr(k, "k", 16));
  if (v) KV_TRY(check_ptr(v, "v", 16));
  tern::ReadArgs a = {};
  a.c = cache_of(c);
  a.b = batch_of(b);
  a.k = k;
  a.v = v;
  a.f32 = dtype == TERN_F32;
  a.items = items_of(b);
  if (page_blocks(c, b) < 0) return fail(TERN_E_UNSUPPORTED, "the call needs too many workgroups");
  KV_HIP(tern::launch_kv_read(a, c->dim, (hipStream_t)stream));
  return TERN_OK;
}

size_t tern_kv_attention_workspace_bytes(const tern_kv* c, const tern_kv_batch* b, int32_t q_heads) {
  if (check_shape(c) != TERN_OK || check_sizes(b) != TERN_OK || check_heads(c, b, q_heads) != TERN_OK) return 0;
  return std::max<size_t>(256, attn_need_upto(c, b, q_heads / c->heads));
}

int32_t tern_kv_attention_parts(const tern_kv* c, const tern_kv_batch* b, int32_t q_heads, int32_t window) {
  if (check_shape(c) != TERN_OK || check_sizes(b) != TERN_OK || check_heads(c, b, q_heads) != TERN_OK || window < 0) return -1;
  if (nothing(b)) return 0;
  const AttnPlan p = plan_of(c, b, q_heads / c->heads, window, true);
  return p.blocks ? p.pieces : -1 - p.parts;
}

int32_t tern_kv_tile_rows(int32_t rows) {
  const int before = g_tile_rows;
  if (rows == 0 || rows == tern::kAttnMid || rows == tern::kAttnTile) g_tile_rows = rows;
  return before;
}

tern_status tern_kv_attention(const tern_kv* c, const tern_kv_batch* b, const uint16_t* q, int64_t q_stride,
                              int32_t q_heads, float scale, int32_t window, int32_t causal, uint16_t* y, void* ws,
                              size_t ws_bytes, void* stream) {
  KV_TRY(check_shape(c));
  KV_TRY(check_batch(b));
  KV_TRY(check_heads(c, b, q_heads));
  if (!(scale >= 0.0f) || !std::isfinite(scale)) return fail(TERN_E_INVAL, "scale=%g must be finite and not negative", scale);
  if (window < 0) return fail(TERN_E_INVAL, "window=%d must not be negative", window);
  if (window && !causal) return fail(TERN_E_UNSUPPORTED, "a window needs causal rows");
  if (nothing(b)) return TERN_OK;
  KV_TRY(check_arrays(c, b));
  KV_TRY(check_rows(q, q_stride, "q"));
  if (q_stride > tern::kMaxStride) return fail(TERN_E_UNSUPPORTED, "q has the row stride %lld: %d at most", (long long)q_stride, tern::kMaxStride);
  KV_TRY(check_ptr(y, "y", 16));
  const AttnPlan p = plan_of(c, b, q_heads / c->heads, window, causal != 0);
  const size_t need = attn_need(p, c);
  if (need && (!ws || ws_bytes < need))
    return fail(TERN_E_WORKSPACE, "workspace of %zu bytes, %zu are needed", ws ? ws_bytes : (size_t)0, need);
  if (ws) KV_TRY(check_ptr(ws, "workspace", 16));  // also one that this call does not need
  tern::AttnArgs a = {};
  a.c = cache_of(c);
  a.b = batch_of(b);
  a.q = q;
  a.q_stride = q_stride;
  a.y = y;
  a.part = (float*)ws;
  a.scale = scale * (float)M_LOG2E;
  a.q_heads = q_heads;
  a.group = q_heads / c->heads;
  a.window = window;
  a.causal = causal != 0;
  a.info = (int2*)(a.part + p.rows * (c->dim + 2));
  a.pieces = p.pieces;
  a.whole = p.whole;
  a.parts = p.parts;
  a.per = p.per;
  a.tiles = p.tiles;
  const hipStream_t s = (hipStream_t)stream;
  if (p.blocks)
    KV_HIP(tern::launch_attn_rows(a, c->dim, p.blocks, p.shares, s));
  else
    KV_HIP(p.tile == tern::kAttnMid ? tern::launch_attn_mid(a, c->dim, s) : tern::launch_attn_tile(a, c->dim, s));
  if (p.join) KV_HIP(p.blocks ? tern::launch_attn_join_rows(a, c->dim, s) : tern::launch_attn_join_tile(a, c->dim, p.tile, s));
  return TERN_OK;
}

}  // extern "C"
