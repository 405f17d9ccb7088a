// Paged NVFP4 K/V cache for gfx950: host side and C ABI of the entry points
// nvfp4_kv_* (include/nvfp4rq.h).  Kernels: plan.hpp (block tables and slots),
// append.hpp (quantizing writes), attention.hpp (attention over the pages);
// layout.hpp has the record's layout.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "nvfp4rq.h"
#include "host.hpp"
#include "layout.hpp"
#include "plan.hpp"
#include "append.hpp"
#include "attention.hpp"

namespace nvfp4rq {
namespace {

int log2_of(int64_t v) {
  int s = 0;
  while ((int64_t{1} << s) < v) ++s;
  return s;
}

// A block table of more entries would have a size that 64 bits do not hold.
bool table_fits(int64_t requests, int64_t width) { return width == 0 || requests <= (int64_t{1} << 60) / width; }

bool page_size_ok(int64_t p) { return p >= 16 && p <= 65536 && (p & (p - 1)) == 0; }
bool head_dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

int64_t page_bytes(int32_t page_size, int32_t head_dim) {
  if (!page_size_ok(page_size) || !head_dim_ok(head_dim)) return -1;
  return static_cast<int64_t>(page_size) * head_dim * 9 / 8;
}

nvfp4_status check_cache_shape(const nvfp4_kv_cache* c) {
  if (!c) return NVFP4_ERR_NULL;
  if (page_bytes(c->page_size, c->head_dim) < 0 || c->pages < 1 || c->pages > INT32_MAX || c->kv_heads < 1 ||
      c->kv_heads > 65535)
    return NVFP4_ERR_SHAPE;
  // pages * kv_heads * bytes below 2^62
  if (c->pages > (int64_t{1} << 62) / (page_bytes(c->page_size, c->head_dim) * c->kv_heads)) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

nvfp4_status check_cache(const nvfp4_kv_cache* c) {
  const nvfp4_status st = check_cache_shape(c);
  if (st != NVFP4_OK) return st;
  if (!c->data || !c->amax) return NVFP4_ERR_NULL;
  if (c->rotate != 0 && c->rotate != 1) return NVFP4_ERR_ARG;
  if (!kv_aligned(c->data, 16) || !kv_aligned(c->amax, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

Span cache_span(const nvfp4_kv_cache* c) {
  return span_of(c->data, c->pages * c->kv_heads * page_bytes(c->page_size, c->head_dim));
}

KvView view_of(const nvfp4_kv_cache* c) {
  return KvView{c->data, c->amax, c->pages, c->kv_heads, log2_of(c->page_size), c->rotate};
}

// Strides of a [tokens, heads, dim] array in elements of `size` bytes, and its
// span in bytes.
nvfp4_status check_rows(int64_t tokens, int32_t heads, int32_t dim, const int64_t strides[2], int size,
                        const void* p, Span* span) {
  if (!strides) return NVFP4_ERR_NULL;
  const int64_t ts = strides[0], hs = strides[1];
  if (ts < 0 || hs < 0) return NVFP4_ERR_SHAPE;
  const int64_t most = int64_t{1} << 60;
  if ((tokens > 1 && ts > most / tokens / size) || (heads > 1 && hs > most / heads / size)) return NVFP4_ERR_SHAPE;
  // a stride that its count does not use may be any: no product of it is formed
  if (ts % (16 / size) != 0 || hs % (16 / size) != 0 || !kv_aligned(p, 16)) return NVFP4_ERR_ALIGN;
  *span = span_of(p, tokens == 0 ? 0 : ((tokens - 1) * ts + (heads - 1) * hs + dim) * size);
  return NVFP4_OK;
}

// ---------------------------------------------------------------- plan

nvfp4_status plan(const int32_t* cached, const int32_t* added, int64_t requests, int32_t page_size, int32_t* table,
                  int64_t width, const int32_t* free_pages, int64_t free_count, const int32_t* head_in,
                  int64_t* slots, int64_t max_tokens, int32_t* cu_q, int32_t* kv_lens, int32_t* head_out,
                  int32_t* missing, hipStream_t st) {
  if (requests < 0 || requests > INT32_MAX || width < 0 || width > INT32_MAX || free_count < 0 ||
      free_count > INT32_MAX || max_tokens < 0 || max_tokens > INT32_MAX || !page_size_ok(page_size) ||
      !table_fits(requests, width))
    return NVFP4_ERR_SHAPE;
  const bool has_table = requests != 0 && width != 0;
  if ((requests != 0 && (!cached || !added || !kv_lens)) || (has_table && !table) || (free_count != 0 && !free_pages) ||
      (max_tokens != 0 && !slots) || !head_in || !cu_q || !head_out || !missing)
    return NVFP4_ERR_NULL;
  for (const void* p : {static_cast<const void*>(cached), static_cast<const void*>(added),
                        static_cast<const void*>(table), static_cast<const void*>(free_pages),
                        static_cast<const void*>(head_in), static_cast<const void*>(cu_q),
                        static_cast<const void*>(kv_lens), static_cast<const void*>(head_out),
                        static_cast<const void*>(missing)})
    if (!kv_aligned(p, 4)) return NVFP4_ERR_ALIGN;
  if (!kv_aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  const Span in[4] = {span_of(cached, 4 * requests), span_of(added, 4 * requests), span_of(free_pages, 4 * free_count),
                      span_of(head_in, 4)};
  const Span out[6] = {span_of(table, 4 * requests * width), span_of(slots, 8 * max_tokens),
                       span_of(cu_q, 4 * (requests + 1)),    span_of(kv_lens, 4 * requests),
                       span_of(head_out, 4),                 span_of(missing, 8)};
  for (int i = 0; i < 6; ++i) {
    if (out[i].lo == out[i].hi) continue;
    for (const Span& s : in)
      if (s.lo != s.hi && spans_meet(out[i], s)) return NVFP4_ERR_ARG;
    for (int j = i + 1; j < 6; ++j)
      if (out[j].lo != out[j].hi && spans_meet(out[i], out[j])) return NVFP4_ERR_ARG;
  }
  PlanArgs a{cached, added, table, free_pages, head_in, slots, max_tokens, cu_q, kv_lens, head_out, missing,
             width, free_count, static_cast<int32_t>(requests), log2_of(page_size)};
  int64_t grid = (max_tokens + kPlanThreads - 1) / kPlanThreads;
  if (grid > 2 * kv_device_cus()) grid = 2 * kv_device_cus();
  if (grid < 1) grid = 1;
  return kv_launch(kv_plan_kernel, dim3(static_cast<unsigned>(grid)), dim3(kPlanThreads), st, a);
}

// ---------------------------------------------------------------- append

template <typename T, int D>
nvfp4_status launch_append(AppendArgs<T> a, int rotate, hipStream_t st) {
  constexpr int kTokens = kThreads / (D / 16);
  a.groups = static_cast<int32_t>((int64_t{a.tokens} + kTokens - 1) / kTokens);
  // 4 workgroups a compute unit or fewer, each taking several groups: they
  // advance through the rows together.  65536 tokens of 8 heads of 128 in f32:
  // 131 us at 2, 129 us at 4, 134 us at 8, 140 us at 16.
  const int64_t per = static_cast<int64_t>(a.cache.kv_heads) * 2;
  int64_t x = (4LL * kv_device_cus() + per - 1) / per;
  if (x > a.groups) x = a.groups;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(a.cache.kv_heads), 2);
  return rotate ? kv_launch(kv_append_kernel<T, D, true>, grid, dim3(kThreads), st, a)
                : kv_launch(kv_append_kernel<T, D, false>, grid, dim3(kThreads), st, a);
}

template <typename T>
nvfp4_status append(const T* k, const T* v, int64_t tokens, const int64_t k_strides[2], const int64_t v_strides[2],
                    const int64_t* slots, const nvfp4_kv_cache* cache, hipStream_t st) {
  nvfp4_status r = check_cache(cache);
  if (r != NVFP4_OK) return r;
  if (tokens < 0 || tokens > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (tokens != 0 && (!k || !v || !slots)) return NVFP4_ERR_NULL;
  Span spans[3];
  r = check_rows(tokens, cache->kv_heads, cache->head_dim, k_strides, sizeof(T), k, &spans[0]);
  if (r != NVFP4_OK) return r;
  r = check_rows(tokens, cache->kv_heads, cache->head_dim, v_strides, sizeof(T), v, &spans[1]);
  if (r != NVFP4_OK) return r;
  if (!kv_aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  if (tokens == 0) return NVFP4_OK;
  spans[2] = span_of(slots, 8 * tokens);
  const Span data = cache_span(cache);
  for (const Span& s : spans)
    if (spans_meet(s, data)) return NVFP4_ERR_ARG;
  if (spans_meet(span_of(cache->amax, 8), data)) return NVFP4_ERR_ARG;
  AppendArgs<T> a{{k, v}, {k_strides[0], v_strides[0]}, {k_strides[1], v_strides[1]}, slots, view_of(cache),
                  static_cast<int32_t>(tokens), 0};
  switch (cache->head_dim) {
    case 64: return launch_append<T, 64>(a, cache->rotate, st);
    case 128: return launch_append<T, 128>(a, cache->rotate, st);
    default: return launch_append<T, 256>(a, cache->rotate, st);
  }
}

// ---------------------------------------------------------------- attention

// One kernel's launch, and its part of the workspace: the partial sums of two
// units a workgroup, head_dim + 2 floats a row, then a RangeUnit a workgroup.
struct AttnLaunch {
  bool on;
  bool ranged;       // the tiles are dealt out; otherwise a workgroup takes a unit
  int64_t wgs;
  int64_t part_rows;
  int64_t bytes(int32_t head_dim) const {
    return ranged ? 4 * part_rows * (head_dim + 2) + wgs * int64_t{sizeof(RangeUnit)} : 0;
  }
};
struct AttnPlan {
  AttnLaunch rows, tiles;  // requests of few rows, and tiles of many
  int32_t few;
  int32_t row_tiles;       // rows kernel: 16-row tiles of a unit
  int32_t tile_count;
  int64_t bytes(int32_t head_dim) const { return rows.bytes(head_dim) + tiles.bytes(head_dim); }
};

constexpr int kIdleTiles = 4;

// Waves of a workgroup of the tiles kernel: two a SIMD, or at head_dim 256,
// where a wave's registers fill it, one.
constexpr int tile_waves(int d) { return d <= 128 ? 8 : 4; }

// How the launches are shaped, from sizes alone: the workspace depends on it.
nvfp4_status plan_attention(int64_t tokens, int32_t q_heads, const nvfp4_kv_cache* c, const nvfp4_kv_batch* b,
                            bool f32, AttnPlan* p) {
  const nvfp4_status st = check_cache_shape(c);
  if (st != NVFP4_OK) return st;
  if (!b) return NVFP4_ERR_NULL;
  if (q_heads < 1 || q_heads % c->kv_heads != 0 || tokens < 0 || tokens > kMostRows / q_heads || b->requests < 0 ||
      b->requests > INT32_MAX - 1 || b->table_width < 0 || b->table_width > INT32_MAX ||
      !table_fits(b->requests, b->table_width) || b->max_q < 0 || b->max_kv < 0)
    return NVFP4_ERR_SHAPE;
  const int64_t group = q_heads / c->kv_heads, cus = kv_device_cus();
  int64_t max_q = b->max_q < tokens ? b->max_q : tokens;
  if (max_q < 1) max_q = 1;
  // Requests of few rows go to the rows kernel, the others to the tiles kernel;
  // a single request of many tokens to the latter alone.  Where the estimate
  // leaves only the former, the rows kernel takes all of them, whatever they
  // turn out to be.  Few rows are 64, two units of the rows kernel: 64 requests
  // of 64 rows over 8k keys of 8 heads take 288 us there and 463 us on tiles of
  // 256 rows, and of 128 rows over 4k keys 288 us and 249 us.  At head_dim 256,
  // where a tile has 128 rows, they are 128: 657 us and 1027 us over 4k keys,
  // and with 256 rows 335 us and 266 us.  Twice as many are few where all units
  // of the call run at once, two a compute unit.  Over 2048 and 8192 keys, in
  // us on the rows kernel and on the tiles kernel: 16 requests of 128 rows on 8
  // heads of 128 (512 units) 40 and 59, 132 and 153, 17 of them 56 and 50, 172
  // and 152, a single one 24 and 35, 43 and 42; fp32 on 5 heads of 64, 25
  // requests of 126 rows (500 units) 38 and 45, 132 and 131, 26 of them 54 and
  // 45, 174 and 124.  At head_dim 256 the limit comes early for short keys: 32
  // requests of 256 rows on one head 44 and 101, 157 and 208, 33 of them 61 and
  // 93, 199 and 191.
  const int64_t forced = kv_env_int("NVFP4RQ_KV_FEW_ROWS");
  int64_t few = forced ? forced : c->head_dim == 256 ? 128 : 64;
  const int64_t unit_rows = 16 * most_row_tiles(c->head_dim);
  if (!forced && max_q * group <= 2 * few &&
      b->requests * c->kv_heads * ((max_q * group - 1) / unit_rows + 1) <= 2 * cus)
    few *= 2;
  const bool only_few = max_q * group <= few;
  const int64_t few_rows = only_few ? max_q * group : few;
  p->row_tiles = few_rows > 16 ? most_row_tiles(c->head_dim) : 1;
  p->few = only_few ? INT32_MAX : (b->requests == 1 || group > few) ? 0 : static_cast<int32_t>(few);
  // The rows kernel: a workgroup a unit, with nothing to join, where the units
  // are short, and the longer they may be the more of the resident workgroups
  // they fill: 64 tiles, 128 from a third on, 256 from two thirds on (of which
  // a single long request among short ones takes 54 us).  Otherwise ranges, one
  // for each resident workgroup, or fewer where the estimate says that each
  // would have too little.  With 8 heads of 128, one token a request, in us
  // whole and in ranges: 1 request over 776 keys 16 and 20, over 2000 17 and
  // 21, over 5000 33 and 20; 32 over 3000 keys 24 and 33; 64 over 3000 keys 40
  // and 54; 256 over up to 4000 146 and 164.  About the limits, with 8 query
  // heads a key head and 768 resident workgroups: 8 and 16 requests (no third)
  // over 2048 keys 17 and 21, 16 and 20, over 4096 27 and 23, 27 and 34; 31 and
  // 32 requests (a third from 32 on) over 4096 29 and 41, 30 and 41, over 8192
  // 56 and 63, 56 and 65; 63, 64 and 65 requests (two thirds from 64 on) over
  // 8192 98 and 114, 102 and 117, 128 and 115.  Where the lengths are between a
  // quarter of that and all of it: 32 requests over 8192 51 and 49, 63, 64 and
  // 65 over 8192 79 and 78, 78 and 79, 95 and 81.  So the limits sit where
  // ragged lengths break even; equal lengths whose units fill the same number
  // of rounds of the compute units would gain some 15% by staying whole past
  // them, and one unit over such a number loses as much.
  const int64_t keys = b->window > 0 && b->max_kv > b->window + max_q ? b->window + max_q : b->max_kv;
  p->rows = AttnLaunch{p->few > 0, true, kv_env_int("NVFP4RQ_KV_ROWS_WGS"), 0};
  if (p->rows.wgs == 0) {
    const int64_t resident = cus * rows_waves(f32, c->head_dim, p->row_tiles);
    const int64_t tiles = keys / kTile + (keys % kTile != 0), row_tiles = (few_rows - 1) / (16 * p->row_tiles) + 1;
    const int64_t units = b->requests * c->kv_heads * row_tiles;
    const int64_t fills = units >= resident ? 3 : 3 * units / resident;  // thirds
    p->rows.wgs = resident;
    if (units > 0 && units <= INT32_MAX / 256 && tiles <= (fills >= 2 ? 256 : fills == 1 ? 128 : 64)) {
      p->rows.ranged = false;
      p->rows.wgs = units;
    } else if (units > 0 && tiles / kMinTiles + 1 < resident / units) {
      p->rows.wgs = (tiles / kMinTiles + 1) * units;
    }
  }
  p->rows.part_rows = p->rows.wgs * 2 * 16 * p->row_tiles;
  // Tiles of rows, as many as their ragged ends can make.  A workgroup takes
  // one of them, the longest first.  Where they are fewer than the compute
  // units, each takes an equal range of their tiles of keys instead, if the
  // longest is kIdleTiles tiles or more above the mean: 8 requests of up to 512
  // tokens over 7.7k keys take 207 us and not 250, 300 tokens over 9000 keys of
  // 4 heads 105 us and not 252.  Below, the partial sums cost more than they
  // save: a prompt of 300 tokens takes 21 us whole and 42 us in ranges, one of
  // 2048 tokens 72 us and 90 us.
  const int64_t tile_rows = 32 * tile_waves(c->head_dim);
  const int64_t count = tokens * group / tile_rows + b->requests, units = count * c->kv_heads;
  if (units > INT32_MAX) return NVFP4_ERR_SHAPE;
  p->tile_count = static_cast<int32_t>(count);
  const int64_t wgs = kv_env_int("NVFP4RQ_KV_TILE_WGS");
  const int64_t longest = keys / (2048 * tile_waves(c->head_dim) / c->head_dim);
  const bool idle = units < cus && longest / cus * (cus - units) + longest % cus * (cus - units) / cus >= kIdleTiles;
  p->tiles = AttnLaunch{!only_few, wgs ? true : idle, wgs ? wgs : cus, 0};
  if (!p->tiles.ranged) p->tiles.wgs = units;
  if (p->tiles.on && p->tiles.wgs > UINT32_MAX / (64 * tile_waves(c->head_dim))) return NVFP4_ERR_SHAPE;
  p->tiles.part_rows = p->tiles.wgs * 2 * tile_rows;
  if (p->rows.wgs > INT32_MAX / 256 || (p->tiles.ranged && p->tiles.wgs > INT32_MAX / 1024)) return NVFP4_ERR_SHAPE;
  if (!p->rows.on) p->rows = AttnLaunch{false, false, 0, 0};
  if (!p->tiles.on) p->tiles = AttnLaunch{false, false, 0, 0};
  return NVFP4_OK;
}

// A kernel on its part of the workspace, which it advances; join: what it
// leaves to be joined.
template <typename T, int D>
nvfp4_status launch_part(void (*kernel)(AttnArgs<T>), int threads, AttnArgs<T> a, const AttnLaunch& part, int rows,
                         float** work, JoinPart* join, hipStream_t st) {
  a.part = *work;
  a.part_ml = part.part_rows * D;
  a.units = part.ranged ? reinterpret_cast<RangeUnit*>(*work + part.part_rows * (D + 2)) : nullptr;
  a.by_grid = FastDiv::make(static_cast<uint32_t>(part.wgs));
  *work += part.bytes(D) / 4;
  if (part.ranged && part.wgs > 1)
    *join = JoinPart{a.part, a.part_ml, a.units, static_cast<int32_t>(part.wgs), rows};
  return kv_launch(kernel, dim3(static_cast<unsigned>(part.wgs)), dim3(threads), st, a);
}

template <typename T, int D, int RT>
nvfp4_status launch_rows(const AttnArgs<T>& a, const AttnPlan& p, float** work, JoinPart* join, hipStream_t st) {
  const bool small_pages = a.cache.shift == 4, split = p.rows.ranged;
  auto kernel = split ? kv_attn_rows_kernel<T, D, RT, false, true> : kv_attn_rows_kernel<T, D, RT, false, false>;
  if (small_pages)
    kernel = split ? kv_attn_rows_kernel<T, D, RT, true, true> : kv_attn_rows_kernel<T, D, RT, true, false>;
  return launch_part<T, D>(kernel, 64 * kAttnWaves, a, p.rows, 16 * RT, work, join, st);
}

template <typename T, int D>
nvfp4_status launch_attention(AttnArgs<T> a, const AttnPlan& p, hipStream_t st) {
  constexpr int kWaves = tile_waves(D);
  float* work = a.part;
  a.few = p.few;
  a.tiles = p.tile_count;
  JoinPart joins[2] = {};
  nvfp4_status r = NVFP4_OK;
  if (p.tiles.on)
    r = launch_part<T, D>(
        p.tiles.ranged ? kv_attn_tiles_kernel<T, D, kWaves, true> : kv_attn_tiles_kernel<T, D, kWaves, false>,
        64 * kWaves, a, p.tiles, 32 * kWaves, &work, &joins[0], st);
  if (r == NVFP4_OK && p.rows.on)
    r = p.row_tiles == 1 ? launch_rows<T, D, 1>(a, p, &work, &joins[1], st)
                         : launch_rows<T, D, most_row_tiles(D)>(a, p, &work, &joins[1], st);
  const int64_t wgs = static_cast<int64_t>(joins[0].wgs) + joins[1].wgs;
  if (r != NVFP4_OK || wgs == 0) return r;
  const dim3 grid(static_cast<unsigned>(wgs), joins[0].wgs ? 2 * kWaves : 4 * p.row_tiles);
  return kv_launch(kv_attn_join_kernel<T, D>, grid, dim3(256), st, a, joins[0], joins[1]);
}

template <typename T>
nvfp4_status attention(const T* q, int64_t tokens, int32_t q_heads, const int64_t q_strides[2],
                       const nvfp4_kv_cache* cache, const nvfp4_kv_batch* batch, T* out,
                       const int64_t out_strides[2], void* workspace, int64_t workspace_bytes, hipStream_t st) {
  AttnPlan p;
  nvfp4_status r = plan_attention(tokens, q_heads, cache, batch, sizeof(T) == 4, &p);
  if (r != NVFP4_OK) return r;
  r = check_cache(cache);
  if (r != NVFP4_OK) return r;
  if (batch->causal != 0 && batch->causal != 1) return NVFP4_ERR_ARG;
  if (batch->window < 0 || (batch->window > 0 && !batch->causal)) return NVFP4_ERR_ARG;
  if (!(batch->scale > 0.0f) || std::isinf(batch->scale)) return NVFP4_ERR_ARG;
  Span sq, so;
  r = check_rows(tokens, q_heads, cache->head_dim, q_strides, sizeof(T), q, &sq);
  if (r != NVFP4_OK) return r;
  r = check_rows(tokens, q_heads, cache->head_dim, out_strides, sizeof(T), out, &so);
  if (r != NVFP4_OK) return r;
  if (tokens == 0 || batch->requests == 0) return NVFP4_OK;
  if (!q || !out || !batch->cu_q || !batch->kv_lens || (batch->table_width != 0 && !batch->table)) return NVFP4_ERR_NULL;
  if (!kv_aligned(batch->cu_q, 4) || !kv_aligned(batch->kv_lens, 4) || !kv_aligned(batch->table, 4))
    return NVFP4_ERR_ALIGN;
  // rows of out must be distinct memory
  const int64_t dim = cache->head_dim;
  const int64_t ot = out_strides[0], oh = out_strides[1];
  const bool token_major = ot >= (q_heads - 1) * oh + dim && (q_heads == 1 || oh >= dim);
  const bool head_major = oh >= (tokens - 1) * ot + dim && (tokens == 1 || ot >= dim);
  if (!(tokens == 1 && (q_heads == 1 || oh >= dim)) && !token_major && !head_major) return NVFP4_ERR_ARG;
  const int64_t need = p.bytes(cache->head_dim);
  if (need > 0) {
    if (!workspace) return NVFP4_ERR_NULL;
    if (!kv_aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    if (workspace_bytes < need) return NVFP4_ERR_ARG;
  }
  const Span work = span_of(workspace, need);
  const Span ins[] = {sq, cache_span(cache), span_of(cache->amax, 8), span_of(batch->cu_q, 4 * (batch->requests + 1)),
                      span_of(batch->kv_lens, 4 * batch->requests),
                      span_of(batch->table, 4 * batch->requests * batch->table_width)};
  for (const Span& s : ins) {
    if (s.lo == s.hi) continue;
    if (spans_meet(s, so) || (need > 0 && spans_meet(s, work))) return NVFP4_ERR_ARG;
  }
  if (need > 0 && spans_meet(so, work)) return NVFP4_ERR_ARG;
  const int group = q_heads / cache->kv_heads;
  const int64_t reach = batch->table_width * cache->page_size;
  AttnArgs<T> a{q, out, q_strides[0], q_strides[1], out_strides[0], out_strides[1], view_of(cache),
                batch->table, batch->cu_q, batch->kv_lens, batch->table_width,
                static_cast<int32_t>(reach < kMostKeys ? reach : kMostKeys),
                static_cast<int32_t>(tokens), static_cast<int32_t>(batch->requests), group,
                batch->causal, batch->window, batch->scale, 0, static_cast<float*>(workspace), 0, 0, nullptr,
                FastDiv::make(static_cast<uint32_t>(cache->kv_heads)), FastDiv::make(static_cast<uint32_t>(group)),
                FastDiv::make(1)};
  switch (cache->head_dim) {
    case 64: return launch_attention<T, 64>(a, p, st);
    case 128: return launch_attention<T, 128>(a, p, st);
    default: return launch_attention<T, 256>(a, p, st);
  }
}

}  // namespace
}  // namespace nvfp4rq

using namespace nvfp4rq;

// ---------------------------------------------------------------- C ABI

extern "C" {

int64_t nvfp4_kv_page_bytes(int32_t page_size, int32_t head_dim) { return page_bytes(page_size, head_dim); }

nvfp4_status nvfp4_kv_plan(const int32_t* cached, const int32_t* added, int64_t requests, int32_t page_size,
                           int32_t* table, int64_t table_width, const int32_t* free_pages, int64_t free_count,
                           const int32_t* head_in, int64_t* slots, int64_t max_tokens, int32_t* cu_q,
                           int32_t* kv_lens, int32_t* head_out, int32_t* missing, hipStream_t stream) {
  return plan(cached, added, requests, page_size, table, table_width, free_pages, free_count, head_in, slots,
              max_tokens, cu_q, kv_lens, head_out, missing, stream);
}

nvfp4_status nvfp4_kv_append(const uint16_t* k, const uint16_t* v, int64_t tokens, const int64_t k_strides[2],
                             const int64_t v_strides[2], const int64_t* slots, const nvfp4_kv_cache* cache,
                             hipStream_t stream) {
  return append(k, v, tokens, k_strides, v_strides, slots, cache, stream);
}

nvfp4_status nvfp4_kv_append_f32(const float* k, const float* v, int64_t tokens, const int64_t k_strides[2],
                                 const int64_t v_strides[2], const int64_t* slots, const nvfp4_kv_cache* cache,
                                 hipStream_t stream) {
  return append(k, v, tokens, k_strides, v_strides, slots, cache, stream);
}

int64_t nvfp4_kv_attention_workspace(int64_t tokens, int32_t q_heads, const nvfp4_kv_cache* cache,
                                     const nvfp4_kv_batch* batch) {
  int64_t most = -1;  // of either type
  for (bool f32 : {false, true}) {
    AttnPlan p;
    if (plan_attention(tokens, q_heads, cache, batch, f32, &p) != NVFP4_OK) return -1;
    if (p.bytes(cache->head_dim) > most) most = p.bytes(cache->head_dim);
  }
  return most;
}

nvfp4_status nvfp4_kv_attention(const uint16_t* q, int64_t tokens, int32_t q_heads, const int64_t q_strides[2],
                                const nvfp4_kv_cache* cache, const nvfp4_kv_batch* batch, uint16_t* out,
                                const int64_t out_strides[2], void* workspace, int64_t workspace_bytes,
                                hipStream_t stream) {
  return attention(q, tokens, q_heads, q_strides, cache, batch, out, out_strides, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_kv_attention_f32(const float* q, int64_t tokens, int32_t q_heads, const int64_t q_strides[2],
                                    const nvfp4_kv_cache* cache, const nvfp4_kv_batch* batch, float* out,
                                    const int64_t out_strides[2], void* workspace, int64_t workspace_bytes,
                                    hipStream_t stream) {
  return attention(q, tokens, q_heads, q_strides, cache, batch, out, out_strides, workspace, workspace_bytes, stream);
}

}  // extern "C"
