// Host half of the 4-bit layers' C ABI (tern_q4_*, tern_route in tern.h):
// argument checks, workspace sizing, choice of kernel and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>

#include "internal.h"
#include "q4.h"

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
#define Q4_HIP(call)                                                                                                   \
  do {                                                                                                                 \
    hipError_t e_ = (call);                                                                                            \
    if (e_ == hipErrorInvalidConfiguration) return fail(TERN_E_UNSUPPORTED, "the product needs too many workgroups"); \
    if (e_ != hipSuccess) return fail(TERN_E_HIP, "%s: %s", #call, hipGetErrorString(e_));                             \
  } while (0)

#define Q4_TRY(expr)                  \
  do {                                \
    tern_status s_ = (expr);          \
    if (s_ != TERN_OK) return s_;     \
  } while (0)

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

tern_status check_ptr(const void* p, bool needed, const char* name, size_t align) {
  if (!p) return needed ? fail(TERN_E_INVAL, "%s is NULL", name) : TERN_OK;
  if (reinterpret_cast<uintptr_t>(p) & (align - 1)) return fail(TERN_E_ALIGN, "%s is not %zu-byte aligned", name, align);
  return TERN_OK;
}

tern_status check_shape(const tern_q4* w) {
  if (!w) return fail(TERN_E_INVAL, "matrix descriptor is NULL");
  if (w->n < 0 || w->k < 0 || w->count < 0)
    return fail(TERN_E_INVAL, "negative shape n=%d k=%d count=%d", w->n, w->k, w->count);
  if (w->group != 32 && w->group != 64 && w->group != 128)
    return fail(TERN_E_UNSUPPORTED, "4-bit group %d is not 32, 64 or 128", w->group);
  if (w->k % w->group) return fail(TERN_E_UNSUPPORTED, "k=%d must be a multiple of group %d", w->k, w->group);
  // buffer descriptors hold 128 activation rows, their offsets 31 bits; n is rounded up to a tile
  if (w->k > (1 << 22) || w->n > 0x7fffff00) return fail(TERN_E_UNSUPPORTED, "n=%d or k=%d is too large", w->n, w->k);
  return TERN_OK;
}

tern_status check_q4(const tern_q4* w) {
  Q4_TRY(check_shape(w));
  const bool body = w->n > 0 && w->k > 0 && w->count > 0;
  Q4_TRY(check_ptr(w->codes, body, "codes", 16));
  Q4_TRY(check_ptr(w->scale, body, "scale", 2));
  return TERN_OK;
}

tern_status check_rows(int m) {
  if (m < 0) return fail(TERN_E_INVAL, "m=%d must not be negative", m);
  if (m > 0x7fffff00) return fail(TERN_E_UNSUPPORTED, "m=%d is too large", m);  // rounded up to a tile
  return TERN_OK;
}

size_t words_of(const tern_q4* w) { return (size_t)w->count * (size_t)w->n * (size_t)(w->k / 8); }

int tile_cols(int tile) { return tile <= tern::kQ4TileSmall ? 128 : 256; }

long long tiles_of(int m, int n, int tile) {
  return (long long)((m + tile - 1) / tile) * ((n + tile_cols(tile) - 1) / tile_cols(tile));
}

// The tile size of a plain product: the one whose busiest CU is done first,
// where a tile costs its 32 x 32 blocks times the tenths below.  Every tile
// decodes its own codes, so few rows make a block dear, dearest where a group
// is short.  us, 64 / 96 / 128 rows: 512 x 12288 x 4096 59.7 / 74 / 59.5 (group
// 32 with zero points 97 / - / 86), 400 x 12288 x 4096 57.8 / 51.0 / 60, 1024 x
// 5120 x 2560 38.5 / 34.4 / -, 4096 x 2560 x 9728 (group 64) 303 / 274 / 327,
// 2048 x 4096 x 4096 88 / - / 71.9, 512 x 4096 x 4096 29.7 / - / -.
// Up to 32 rows a tile of 32 (24 x 131072 x 2560 47 us, 61 with 64 rows).
int pick_tile(int m, int n, int group) {
  if (m <= 32) return tern::kQ4TileTiny;
  const int tile[] = {tern::kQ4TileSmall, tern::kQ4TileMid, tern::kQ4TileLarge};
  const int tenths[] = {group < 128 ? 30 : 28, 23, 21};
  int best = 0;
  long long least = 0;
  for (int i = 0; i < 3; ++i) {
    const long long blocks = (long long)(tile[i] / 32) * (tile_cols(tile[i]) / 32);
    const long long cost = (tiles_of(m, n, tile[i]) + 255) / 256 * blocks * tenths[i];
    if (!best || cost < least) {
      best = tile[i];
      least = cost;
    }
  }
  return best;
}

// The tile kernel holds a matrix's scales in one buffer below 2 GiB.
bool tile_scales_fit(int n, int k) { return (long long)n * (k / 32) * 2 < (1ll << 31); }

// How a plain product runs.  Rows kernel: up to 16 activation rows, up to 160
// unless tiles abound, and up to 320 where tiles would not fill the card (us,
// rows against tiles: m = 24, 131072 x 2560 57, 47; m = 64 94, 66; m = 64,
// 32768 x 2560 22.8, 21.9; m = 128, 12288 x 4096 23.6, 27.6; m = 160, 19456 x
// 2560 29.8, 28.4; m = 128, 4096 x 4096 13.9, 17.7; m = 256, 2560 x 9728 29.8,
// 30.2; m = 256, 12288 x 4096 41.6, 40.4).  K parts where tiles are few: some 512 workgroups, at
// least eight K steps each.
struct Route {
  bool rows;
  int tile, splits, tps;
};

Route route_of(int m, int n, int k, int group) {
  Route r = {};
  const int steps = (k + 127) / 128;
  const long long small = tiles_of(m, n, tern::kQ4TileSmall);
  r.rows = m <= 16 || (m <= 160 && small < 384) || (m <= 320 && small < 256) || !tile_scales_fit(n, k);
  r.tile = pick_tile(m, n, group);
  r.splits = 1;
  if (!r.rows && small < 256) r.splits = std::max(1, (int)std::min<long long>(512 / std::max(small, 1ll), steps / 8));
  r.tps = std::max(1, (steps + r.splits - 1) / r.splits);
  r.splits = std::max(1, (steps + r.tps - 1) / r.tps);
  return r;
}

size_t plain_ws(int m, const tern_q4* w) {
  const Route r = route_of(m, w->n, w->k, w->group);
  return !r.rows && r.splits > 1 ? (size_t)r.splits * m * w->n * 4 : 0;
}

// The most that any call with up to m rows needs.  K parts come with more than
// 320 rows, five of the tiles that route_of counts; the most of a tile's rows
// takes the most.
size_t plain_ws_upto(int m, const tern_q4* w) {
  size_t most = plain_ws(m, w);
  const int tile = tern::kQ4TileSmall;
  for (long long r = 6 * tile; r < m && tiles_of((int)r, w->n, tile) < 256; r += tile)
    most = std::max(most, plain_ws((int)r, w));
  return most;
}

tern::Q4Args args_of(const tern_q4* w) {
  tern::Q4Args a = {};
  a.codes = w->codes;
  a.scale = w->scale;
  a.zero = w->zero;
  a.n = w->n;
  a.k = w->k;
  a.splits = 1;
  a.tps = (w->k + 127) / 128;
  a.experts = w->count;
  return a;
}

// ---- experts
// Few slots: every slot is a tile of its own and a token's down products are
// summed in its own workgroup; nothing has to be sorted, which saves two
// launches, but slots that share an expert read it once each.  Taken up to 32
// slots while what is read again, with slots spread evenly over the experts,
// stays below 32 MB.  us slot by slot / on tiles (MB read again): 64 experts of
// 2560 x 1024, top 8, 1 token 15 / 24 (0), 2 tokens 23 / 31 (4), 4 tokens 35 / 41
// (22); 128 of 2048 x 768, 4 tokens 23 / 35 (7); 16 of 4096 x 1056 at group 32,
// top 2, 4 tokens 26 / 32 (9), 8 tokens 39 / 39 (36), 16 tokens 68 / 47 (116); 8
// of 4096 x 2048, 4 tokens 27 / 29 (32), 8 tokens 45 / 34 (111); 8 of 4096 x
// 14336, 1 token 49 / 59 (0), 2 tokens 84 / 81 (44), 16 tokens 498 / 180 (1600); 4
// of 1024 x 512, top 1, 16 tokens 11 / 15 (10), 32 tokens 16 / 15 (22).
constexpr int kDirectSlots = 32;
constexpr double kDirectAgain = 32e6;

bool slot_by_slot(const tern_q4* up, const tern_q4* down, int m, int topk) {
  const long long slots = (long long)m * topk;
  if (slots > kDirectSlots) return false;
  double missed = 1.0;  // the share of the experts that no token names
  for (int t = 0; t < m; ++t) missed *= 1.0 - std::min(1.0, (double)topk / down->count);
  const double bytes = ((double)up->n * up->k + (double)down->n * down->k) / 2;
  return (slots - down->count * (1.0 - missed)) * bytes <= kDirectAgain || m == 1;
}
// Slots of one round, and bytes of its inner values and partials (but for a
// single token's).  16384 tokens, 8 of 64 experts of 2560 x 1024: 3.62 ms in two
// rounds, 3.61 in one of 1.8 GiB.
constexpr int kRoundSlots = 1 << 19;
constexpr long long kRoundBytes = 1ll << 30;

struct ExpertsPlan {
  bool direct, tile;
  int rows, max_tiles;
  size_t h, part, tiles, ntiles, order, place, bytes;  // offsets in the workspace
};

ExpertsPlan plan_tokens(const tern_q4* up, const tern_q4* down, int m, int topk) {
  ExpertsPlan p = {};
  const int experts = down->count, inner = down->k, n = down->n;
  const size_t slots = (size_t)m * topk;
  p.direct = slot_by_slot(up, down, m, topk);
  // Tiles of 8 or 16 rows on the rows kernel (its tiles are a grid's y) or of
  // 32 or 64 on the tile kernel, by the rows an expert has on average; short
  // groups make the tile kernel's decoding dear.  us of a whole call, 8 / 16 /
  // 32 / 64: 64 experts of 2560 x 1024 at group 128, 2 rows an expert 57 / 62 /
  // 63 / -, 4 rows 72 / 76 / 76 / -, 6 rows 81 / 83 / 79 / 103, 12 rows 114 / 105
  // / 92 / 110, 25 rows - / 150 / 106 / 123, 37 rows - / 197 / 127 / 133, 62 rows
  // - / - / 180 / 177, 125 rows - / - / 303 / 278; 128 of 2048 x 768, 2 rows 64 /
  // 70 / 74 / -, 8 rows 108 / 106 / 95 / 120; 8 of 4096 x 2048 at group 64, 5
  // rows 41 / 40 / 49 / -, 10 rows 55 / 51 / 50 / 63, 20 rows 76 / 66 / 62 / 64,
  // 50 rows - / - / 77 / 92, 100 rows - / - / 122 / 114; 16 of 4096 x 1056 at
  // group 32, 2.6 rows 47 / 48 / 62 / -, 8 rows 63 / 61 / 69 / 90, 12 rows 76 / 69
  // / 84 / 105, 20 rows 102 / 82 / 88 / 111, 32 rows - / 107 / 90 / 123, 50 rows -
  // / - / 124 / 126, 100 rows - / - / 176 / 173.
  const size_t mean = slots / experts;
  p.rows = mean < 5 ? tern::kQ4TileFew
           : mean * up->group < 768 ? tern::kQ4TileRows
           : mean < 60 ? tern::kQ4TileTiny : tern::kQ4TileSmall;
  if (!tile_scales_fit(up->n, up->k) || !tile_scales_fit(n, inner)) p.rows = tern::kQ4TileRows;
  p.tile = p.rows > tern::kQ4TileRows;
  p.max_tiles = (int)std::min<size_t>(slots, slots / p.rows + experts);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  p.h = take(slots * inner * 2 * (p.direct ? tern::kInnerSlot : tern::kInnerTile));
  if (!p.direct) {
    p.part = take(slots * n * 4);
    p.tiles = take(std::min(slots, slots / tern::kQ4TileFew + experts) * 16);  // whatever the rows: it grows with the slots
    p.ntiles = take(4);
    p.order = take(slots * 4);
    p.place = take(slots * 4);
  }
  p.bytes = at;
  return p;
}

// Tokens of one round: their x stays below a buffer's 2 GiB and their tiles
// below a grid's y (what one launch can take at most), and the workspace does
// not grow with m without end.
int launch_tokens(const tern_q4* up, int m, int topk) {
  const long long by_x = up->k ? ((1ll << 31) - 1) / (2ll * up->k) : m;
  return (int)std::max<long long>(1, std::min<long long>({(long long)m, by_x, (long long)kRoundSlots / topk}));
}
int round_tokens(const tern_q4* up, const tern_q4* down, int m, int topk) {
  const long long token = topk * (4ll * down->n + 2ll * tern::kInnerTile * down->k);
  const long long by_bytes = token ? kRoundBytes / token : m;
  return (int)std::max<long long>(1, std::min<long long>(launch_tokens(up, m, topk), by_bytes));
}

// What a call with m tokens needs, and what any with up to m does.
size_t experts_ws(const tern_q4* up, const tern_q4* down, int m, int topk) {
  if (m <= 0) return 0;
  const int most = round_tokens(up, down, m, topk);
  const size_t rest = m % most ? plan_tokens(up, down, m % most, topk).bytes : 0;
  return std::max(plan_tokens(up, down, most, topk).bytes, rest);
}
size_t experts_ws_upto(const tern_q4* up, const tern_q4* down, int m, int topk) {
  size_t most = experts_ws(up, down, m, topk);  // on tiles it grows with the tokens
  for (int t = 1; t < m && (long long)t * topk <= kDirectSlots; ++t)
    most = std::max(most, plan_tokens(up, down, t, topk).bytes);
  return most;
}

// Whether a round's grids can be launched, those of the kernels it runs on.
bool plan_fits(const tern_q4* down, const ExpertsPlan& p, int m) {
  auto fits = [](long long width, int cols, long long rows, int threads) {
    return tern::grid_fits((width + cols - 1) / cols * rows, threads);
  };
  if (p.direct)
    return fits(down->k, 16, 1, 64 * tern::kUpSlotWaves) &&
           fits(down->n, 16, 1, 64 * (m == 1 ? tern::kDownOneTokenWaves : tern::kDownTokenWaves));
  if (p.tile) return fits(down->k, 64, p.max_tiles, 256) && fits(down->n, 128, p.max_tiles, 256);
  return fits(down->k, 16, 1, 64 * tern::kUpWaves) && fits(down->n, 16 * tern::kDownPanels, 1, 64 * tern::kDownWaves);
}

tern_status check_experts(const tern_q4* up, const tern_q4* down, int m, int topk) {
  Q4_TRY(check_shape(up));
  Q4_TRY(check_shape(down));
  if (m < 0) return fail(TERN_E_INVAL, "m=%d must not be negative", m);
  if (up->count < 1 || up->count != down->count)
    return fail(TERN_E_INVAL, "%d gate/up and %d down matrices", up->count, down->count);
  if (up->count > 1024) return fail(TERN_E_UNSUPPORTED, "%d experts: 1024 at most", up->count);
  if (up->n % 2 || up->n / 2 != down->k)
    return fail(TERN_E_INVAL, "gate/up has %d rows, down k=%d: twice as many are wanted", up->n, down->k);
  if (topk < 1) return fail(TERN_E_INVAL, "topk=%d must be positive", topk);
  if (topk > kRoundSlots) return fail(TERN_E_UNSUPPORTED, "topk=%d: %d at most", topk, kRoundSlots);
  if ((long long)m * topk > 0x7fffffffll) return fail(TERN_E_UNSUPPORTED, "m=%d, topk=%d: too many slots", m, topk);
  return TERN_OK;
}

}  // namespace

extern "C" {

tern_status tern_q4_check(const tern_q4* w) { return check_q4(w); }

size_t tern_q4_workspace_bytes(const tern_q4* w, int32_t m) {
  if (check_shape(w) != TERN_OK || check_rows(m) != TERN_OK) return 0;
  return std::max<size_t>(256, plain_ws_upto(m, w));
}

int32_t tern_q4_tile_rows(const tern_q4* w, int32_t m) {
  if (check_shape(w) != TERN_OK || check_rows(m) != TERN_OK) return -1;
  const Route r = route_of(m, w->n, w->k, w->group);
  return r.rows ? 0 : r.tile;
}

int32_t tern_q4_experts_tile_rows(const tern_q4* gate_up, const tern_q4* down, int32_t m, int32_t topk) {
  if (check_experts(gate_up, down, m, topk) != TERN_OK) return -1;
  if (m == 0) return 0;
  const ExpertsPlan p = plan_tokens(gate_up, down, round_tokens(gate_up, down, m, topk), topk);
  return p.direct ? 0 : p.rows;
}

tern_status tern_q4_pack(const uint8_t* q, const tern_q4* dst, void* ws, size_t ws_bytes, void* stream) {
  Q4_TRY(check_shape(dst));
  const size_t words = words_of(dst);
  if (!words) return TERN_OK;
  Q4_TRY(check_ptr(q, true, "q", 8));
  Q4_TRY(check_ptr(dst->codes, true, "codes", 16));
  if (!ws || ws_bytes < 4) return fail(TERN_E_WORKSPACE, "workspace of %zu bytes, 4 are needed", ws_bytes);
  Q4_TRY(check_ptr(ws, true, "workspace", 16));
  const hipStream_t s = (hipStream_t)stream;
  Q4_HIP(tern::launch_q4_pack(q, words, const_cast<uint8_t*>(dst->codes), (uint32_t*)ws, s));
  uint32_t flag = 0;
  Q4_HIP(hipMemcpyAsync(&flag, ws, 4, hipMemcpyDeviceToHost, s));
  Q4_HIP(hipStreamSynchronize(s));
  if (flag) return fail(TERN_E_INVAL, "code above 15");
  return TERN_OK;
}

tern_status tern_q4_unpack(const tern_q4* src, uint8_t* q, void* stream) {
  Q4_TRY(check_shape(src));
  const size_t words = words_of(src);
  if (!words) return TERN_OK;
  Q4_TRY(check_ptr(src->codes, true, "codes", 16));
  Q4_TRY(check_ptr(q, true, "q", 8));
  Q4_HIP(tern::launch_q4_unpack(src->codes, words, q, (hipStream_t)stream));
  return TERN_OK;
}

tern_status tern_q4_gemm(const tern_q4* w, const uint16_t* x, int32_t m, void* y, int32_t y_dtype, void* ws,
                         size_t ws_bytes, void* stream) {
  Q4_TRY(check_q4(w));
  if (w->count != 1) return fail(TERN_E_INVAL, "tern_q4_gemm takes one matrix (count=%d)", w->count);
  Q4_TRY(check_rows(m));
  if (y_dtype != TERN_F16 && y_dtype != TERN_F32) return fail(TERN_E_UNSUPPORTED, "unknown output dtype %d", y_dtype);
  if (m == 0 || w->n == 0) return TERN_OK;
  Q4_TRY(check_ptr(x, w->k > 0, "x", 16));
  Q4_TRY(check_ptr(y, true, "y", y_dtype == TERN_F32 ? 4 : 2));
  const size_t need = plain_ws(m, w);
  if (need && (!ws || ws_bytes < need))
    return fail(TERN_E_WORKSPACE, "workspace of %zu bytes, %zu are needed", ws ? ws_bytes : (size_t)0, need);
  if (need) Q4_TRY(check_ptr(ws, true, "workspace", 16));
  tern::Q4Args a = args_of(w);
  a.x = x;
  a.y = y;
  a.m = m;
  a.y_f32 = y_dtype == TERN_F32;
  const hipStream_t s = (hipStream_t)stream;
  const Route r = route_of(m, w->n, w->k, w->group);
  if (r.rows) {
    Q4_HIP(tern::launch_q4_rows(tern::kQ4Plain, w->group, a, 0, 0, s));
    return TERN_OK;
  }
  a.splits = r.splits;
  a.tps = r.tps;
  a.partial = (float*)ws;
  Q4_HIP(tern::launch_q4_tile(tern::kQ4Plain, w->group, a, 0, r.tile, s));
  if (a.splits > 1) Q4_HIP(tern::launch_q4_reduce(a, s));
  return TERN_OK;
}

size_t tern_q4_experts_workspace_bytes(const tern_q4* gate_up, const tern_q4* down, int32_t m, int32_t topk) {
  if (check_experts(gate_up, down, m, topk) != TERN_OK) return 0;
  return std::max<size_t>(256, experts_ws_upto(gate_up, down, m, topk));
}

tern_status tern_q4_experts(const tern_q4* gate_up, const tern_q4* down, const uint16_t* x, int32_t m,
                            const int32_t* ids, const float* weights, int32_t topk, void* y, int32_t y_dtype, void* ws,
                            size_t ws_bytes, void* stream) {
  Q4_TRY(check_experts(gate_up, down, m, topk));
  Q4_TRY(check_q4(gate_up));
  Q4_TRY(check_q4(down));
  if (y_dtype != TERN_F16 && y_dtype != TERN_F32) return fail(TERN_E_UNSUPPORTED, "unknown output dtype %d", y_dtype);
  if (m == 0 || down->n == 0) return TERN_OK;
  Q4_TRY(check_ptr(x, gate_up->k > 0, "x", 16));
  Q4_TRY(check_ptr(ids, true, "ids", 4));
  Q4_TRY(check_ptr(weights, true, "weights", 4));
  Q4_TRY(check_ptr(y, true, "y", y_dtype == TERN_F32 ? 4 : 2));
  const size_t need = experts_ws(gate_up, down, m, topk);
  if (need && (!ws || ws_bytes < need))
    return fail(TERN_E_WORKSPACE, "workspace of %zu bytes, %zu are needed", ws ? ws_bytes : (size_t)0, need);
  Q4_TRY(check_ptr(ws, false, "workspace", 16));
  uint8_t* base = (uint8_t*)ws;
  const hipStream_t s = (hipStream_t)stream;
  const int most = round_tokens(gate_up, down, m, topk), f32 = y_dtype == TERN_F32;
  // what one launch could not take is refused, however small the rounds are
  for (int mt : {launch_tokens(gate_up, m, topk), most, m % most ? m % most : most})
    if (!plan_fits(down, plan_tokens(gate_up, down, mt, topk), mt))
      return fail(TERN_E_UNSUPPORTED, "m=%d, n=%d: the products need too many workgroups", m, down->n);
  for (int t = 0, mt; t < m; t += mt) {
    mt = std::min(most, m - t);
    const ExpertsPlan p = plan_tokens(gate_up, down, mt, topk);
    uint8_t* yt = (uint8_t*)y + (size_t)t * down->n * (f32 ? 4 : 2);
    tern::Q4Args u = args_of(gate_up), d = args_of(down);
    u.x = x + (size_t)t * gate_up->k;
    u.y = base + p.h;
    d.x = (const uint16_t*)(base + p.h);
    u.m = d.m = mt;
    u.ids = d.ids = ids + (size_t)t * topk;
    u.gates = d.gates = weights + (size_t)t * topk;
    u.topk = d.topk = topk;
    if (p.direct) {
      if (down->k) Q4_HIP(tern::launch_q4_rows(tern::kQ4UpSlot, gate_up->group, u, mt * topk, 0, s));
      d.y = yt;
      d.y_f32 = f32;
      Q4_HIP(tern::launch_q4_rows(tern::kQ4DownToken, down->group, d, mt, 0, s));
      continue;
    }
    u.tiles = d.tiles = (const int4*)(base + p.tiles);
    u.ntiles = d.ntiles = (const int32_t*)(base + p.ntiles);
    u.slots = d.slots = (const int32_t*)(base + p.order);
    d.y = base + p.part;
    Q4_HIP(tern::launch_q4_plan(u.ids, mt * topk, down->count, p.rows, (int4*)(base + p.tiles),
                                (int32_t*)(base + p.ntiles), (int32_t*)(base + p.order), (int32_t*)(base + p.place), s));
    auto product = [&](int mode, int group, const tern::Q4Args& a) {
      return p.tile ? tern::launch_q4_tile(mode, group, a, p.max_tiles, p.rows, s)
                    : tern::launch_q4_rows(mode, group, a, p.max_tiles, p.rows, s);
    };
    if (down->k) Q4_HIP(product(tern::kQ4Up, gate_up->group, u));
    Q4_HIP(product(tern::kQ4Down, down->group, d));
    Q4_HIP(tern::launch_q4_combine((const float*)(base + p.part), (const int32_t*)(base + p.place), u.gates, mt, topk,
                                   down->n, yt, f32, s));
  }
  return TERN_OK;
}

tern_status tern_route(const void* logits, int32_t l_dtype, int32_t m, const tern_router* r, int32_t* ids,
                       float* weights, void* stream) {
  if (!r) return fail(TERN_E_INVAL, "router descriptor is NULL");
  if (m < 0) return fail(TERN_E_INVAL, "m=%d must not be negative", m);
  if (l_dtype != TERN_F16 && l_dtype != TERN_F32) return fail(TERN_E_UNSUPPORTED, "unknown logits dtype %d", l_dtype);
  if (r->score != TERN_SCORE_SOFTMAX && r->score != TERN_SCORE_SIGMOID)
    return fail(TERN_E_UNSUPPORTED, "unknown score %d", r->score);
  if (r->experts < 1 || r->groups < 1 || r->experts % r->groups)
    return fail(TERN_E_INVAL, "%d experts in %d groups", r->experts, r->groups);
  if (r->experts > 1024 || r->groups > 64)
    return fail(TERN_E_UNSUPPORTED, "%d experts in %d groups: 1024 in 64 at most", r->experts, r->groups);
  if (r->keep_groups < 1 || r->keep_groups > r->groups)
    return fail(TERN_E_INVAL, "keep_groups=%d of %d groups", r->keep_groups, r->groups);
  if (r->group_best != 1 && r->group_best != 2)
    return fail(TERN_E_UNSUPPORTED, "group_best=%d is not 1 or 2", r->group_best);
  if (r->topk < 1 || r->topk > r->keep_groups * (r->experts / r->groups))
    return fail(TERN_E_INVAL, "topk=%d of %d experts", r->topk, r->keep_groups * (r->experts / r->groups));
  if (r->topk > 64) return fail(TERN_E_UNSUPPORTED, "topk=%d: 64 at most", r->topk);
  if (m == 0) return TERN_OK;
  Q4_TRY(check_ptr(logits, true, "logits", l_dtype == TERN_F32 ? 4 : 2));
  Q4_TRY(check_ptr(r->bias, false, "bias", 4));
  Q4_TRY(check_ptr(ids, true, "ids", 4));
  Q4_TRY(check_ptr(weights, true, "weights", 4));
  tern::RouteArgs a = {};
  a.bias = r->bias;
  a.experts = r->experts;
  a.topk = r->topk;
  a.groups = r->groups;
  a.best = r->group_best;
  a.keep = r->keep_groups;
  a.renorm = r->renorm != 0;
  a.sigmoid = r->score == TERN_SCORE_SIGMOID;
  a.scale = r->scale;
  constexpr int most = 1 << 24;  // tokens of a launch
  for (int t = 0; t < m; t += std::min(most, m - t)) {
    a.m = std::min(most, m - t);
    a.logits = (const uint8_t*)logits + (size_t)t * r->experts * (l_dtype == TERN_F32 ? 4 : 2);
    a.ids = ids + (size_t)t * r->topk;
    a.weights = weights + (size_t)t * r->topk;
    Q4_HIP(tern::launch_route(a, l_dtype == TERN_F16, (hipStream_t)stream));
  }
  return TERN_OK;
}

}  // extern "C"
