// Attention of new tokens over the paged NVFP4 cache (include/nvfp4rq.h,
// nvfp4_kv_attention).
//
//   S_rj = scale q_r.k_j over the keys that row r sees, O_r = sum_j p_rj v_j /
//   sum_j p_rj, p_rj = exp(S_rj - m_r).
//
// Rotation: H16 is orthonormal, so q.k = (q H).(k H) and sum p v = (sum p v H)
// H: the cache stays rotated, and each query and each output row is rotated
// once.
//
// Number formats: a decoded value without its tensor's scale g, E2M1 * E4M3,
// has 6 significant bits between 2^-10 and 2688 and is exact in fp16; g enters
// the logits' factor (K) and the final scaling (V).  Both products run on the
// fp16 matrix instructions with binary32 sums.  A rotated query row is scaled
// by a power of two that brings its largest value into [2^12, 2^13), then
// rounded to fp16; the softmax weights are scaled by 2^12, so that they lose
// nothing to fp16's subnormals above 2^-26.  Where q is binary32 (kSplit) both
// are taken as hi + lo, two fp16 numbers with 22 bits, and each product is
// two matrix instructions.
//
// Everything is computed transposed, S^T = K Q^T and O^T = V^T P^T: a matrix
// instruction's result then has one query row per lane column, so a row's
// maximum, sum and rescaling factor live in its own lanes, and the lane that
// holds S^T values of 8 tokens holds exactly the P^T operand of the second
// product; no value moves between lanes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../common.hpp"
#include "host.hpp"
#include "layout.hpp"

namespace nvfp4rq {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kWeightBits = 12.0f;   // softmax weights are held times 2^12
// A row's maximum is raised, and its sums rescaled, only once a logit passes it
// by 2^3: weights stay below 2^15, inside fp16.
constexpr float kRaise = 3.0f;

// What a workgroup leaves for the joining of its first unit's parts.
struct RangeUnit {
  int64_t chunk;                   // tiles of a workgroup
  int32_t row0, rows, base, head;  // the unit: its request's first query and rows, its first row, its head
  int32_t off, tiles;              // tiles of it before this workgroup's, and in all
};

template <typename T>
struct AttnArgs {
  const T* q;
  T* out;
  int64_t q_token, q_head, o_token, o_head;  // strides
  KvView cache;
  const int32_t *table, *cu_q, *kv_lens;
  int64_t table_width;
  int32_t reach;                    // keys that a row of the table has room for, kMostKeys at most
  int32_t tokens, requests, group;  // group: query heads per key head
  int32_t causal, window;
  float scale;
  int32_t few;       // requests of at most this many rows go to the rows kernel
  // partial sums of a launch: [slot][row][D], then (m, l) pairs from part_ml
  // floats on
  float* part;
  int64_t part_ml;
  int32_t tiles;       // of rows, of the tiles kernel
  RangeUnit* units;    // of each workgroup; null where none is shared
  FastDiv by_heads, by_group, by_grid;
};

// ---------------------------------------------------------------- decoding

// 8 codes (one dword) times their scale, given in both halves.
__device__ __forceinline__ half8_t decode8(uint32_t w, half2_t s) {
  union { half2_t h[4]; half8_t v; } u;
  u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s;
  u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
  u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s;
  u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
  return u.v;
}

// 8 codes times 8 scales.
__device__ __forceinline__ half8_t decode8(uint32_t w, const half2_t s[4]) {
  union { half2_t h[4]; half8_t v; } u;
  u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s[0];
  u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s[1];
  u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s[2];
  u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s[3];
  return u.v;
}

// The two codes of byte `byte` of w; a constant after unrolling.
__device__ __forceinline__ half2_t code_pair(uint32_t w, int byte) {
  switch (byte) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
  }
}

// Two E4M3 bytes (the low or the high two of w).
template <bool HIGH>
__device__ __forceinline__ half2_t scale2(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH);
}

// V's scales of 8 tokens.  Byte 0x7F, which no write leaves, reads as 448, not
// NaN: the weight of a key that a row does not see is 0, and 0 times whatever
// a page holds has to stay 0.
__device__ __forceinline__ void v_scales8(u32x2 w, half2_t s[4]) {
  const half2_t top = {(_Float16)448.0f, (_Float16)448.0f};
  s[0] = __builtin_elementwise_min(scale2<false>(w.x), top);
  s[1] = __builtin_elementwise_min(scale2<true>(w.x), top);
  s[2] = __builtin_elementwise_min(scale2<false>(w.y), top);
  s[3] = __builtin_elementwise_min(scale2<true>(w.y), top);
}

// Transposes 8 x 8 nibbles: nibble j of word i becomes nibble i of word j.
__device__ __forceinline__ void transpose_nibbles(uint32_t w[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // halves between words i and i + 4
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    w[i + 4] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // bytes between words i and i + 2
    const int i = (k & 1) + 4 * (k >> 1);
    const uint32_t a = w[i], b = w[i + 2];
    w[i] = __builtin_amdgcn_perm(b, a, 0x06020400u);
    w[i + 2] = __builtin_amdgcn_perm(b, a, 0x07030501u);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // nibbles between words i and i + 1
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
    w[i + 1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
  }
}

// ---------------------------------------------------------------- lanes

// Maximum and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_over_rows(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_rows(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// 8 consecutive values as binary32.
__device__ __forceinline__ void load_half(const uint16_t* p, float z[8]) {
  widen8(*reinterpret_cast<const uint4*>(p), z);
}
__device__ __forceinline__ void load_half(const float* p, float z[8]) {
  const float4* q = reinterpret_cast<const float4*>(p);
  const float4 a = q[0], b = q[1];
  z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
  z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
}

__device__ __forceinline__ void rotate16_block(float* z) {
  stages_1_2_4(z);
  stages_1_2_4(z + 8);
  stage_8(z, z + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] *= 0.25f;
}

__device__ __forceinline__ void store16(float* p, const float* z) {
  float4* o = reinterpret_cast<float4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  union { bf16x2 h; uint32_t u; } c;
  c.h = bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)};  // to nearest even
  return c.u;
}
__device__ __forceinline__ void store16(uint16_t* p, const float* z) {
  uint4* o = reinterpret_cast<uint4*>(p);
  o[0] = make_uint4(bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3]), bf16_pair(z[4], z[5]), bf16_pair(z[6], z[7]));
  o[1] = make_uint4(bf16_pair(z[8], z[9]), bf16_pair(z[10], z[11]), bf16_pair(z[12], z[13]),
                    bf16_pair(z[14], z[15]));
}

// The power of two that brings a row's largest |value| into [2^12, 2^13), as
// an exponent: 0 for a zero row, and for one with an infinity or a NaN, which
// then reach the products as they are.
__device__ __forceinline__ int row_exponent(float top) {
  const uint32_t u = __float_as_uint(top) & 0x7FFFFFFFu;
  if (u == 0u || u >= 0x7F800000u) return 0;
  return 12 - (__builtin_amdgcn_frexp_expf(top) - 1);
}

// The factor of a row's products in the log2 domain, scale log2(e) g 2^-e.
// Significands and exponents apart: however small g or the scale, what the
// other or the query's 2^e makes up for keeps its bits.  Not 0, so that a
// masked logit stays -inf (|s| < 2^34: nothing is lost), and not infinite, so
// that a logit of 0 stays 0.  NaN where the maximum is none: results then show
// it.
__device__ __forceinline__ float logit_factor(float scale, float amax, int e) {
  const float g = global_scale(amax);
  const float f = __builtin_amdgcn_frexp_mantf(scale) * kLog2e * __builtin_amdgcn_frexp_mantf(g);
  const int x = __builtin_amdgcn_frexp_expf(scale) + __builtin_amdgcn_frexp_expf(g) - e;
  constexpr float kMost = 0x1.fffffep127f;
  return g <= kMost ? __builtin_amdgcn_fmed3f(__builtin_ldexpf(f, x), 0x1p-126f, kMost) : NAN;
}

// What brings a row's sums to its result, g / l: where g is so small that the
// quotient may be subnormal (l < 2^46), times 2^100, with `back` to take that
// off the result after everything else.  0 for a row without keys.
struct OutScale {
  float g, back;
  __device__ __forceinline__ float over(float l) const { return l == 0.0f ? 0.0f : g / l; }
};
__device__ __forceinline__ OutScale out_scale(float amax) {
  const float g = global_scale(amax);
  const bool small = g < 0x1p-60f;
  return OutScale{small ? g * 0x1p100f : g, small ? 0x1p-100f : 1.0f};
}

// Inclusive sum over the wave.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 of a row to the next
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
  return v;
}

// ---------------------------------------------------------------- a request

constexpr int kMostKeys = INT32_MAX - 65535;  // key arithmetic past the last tile stays in 32 bits
constexpr int kMostRows = INT32_MAX - 65535;  // tokens * query heads: a unit's first row past the last one, too
struct Request {
  int row0, n, kv;  // first row of q, queries, keys
};
template <typename T>
__device__ __forceinline__ Request request_of(const AttnArgs<T>& a, int r) {
  int lo = a.cu_q[r], hi = a.cu_q[r + 1];
  lo = lo < 0 ? 0 : (lo > a.tokens ? a.tokens : lo);
  hi = hi < lo ? lo : (hi > a.tokens ? a.tokens : hi);
  const int kv = a.kv_lens[r];
  return Request{lo, hi - lo, kv < 0 ? 0 : (kv > kMostKeys ? kMostKeys : kv)};
}

// Keys [lo, hi) that any of the queries [i0, i1) of a request sees; empty when
// hi <= lo.  Those past the table's row are left out, so that a length too
// large costs no time: a query that sees one is NaN whatever the others hold
// (see_of).
struct Keys {
  int lo, hi;
};
template <typename T>
__device__ __forceinline__ Keys keys_of(const AttnArgs<T>& a, const Request& r, int i0, int i1) {
  Keys k{0, r.kv < a.reach ? r.kv : a.reach};
  if (a.causal) {
    const int64_t last = static_cast<int64_t>(r.kv) - r.n + i1 - 1;
    if (last + 1 < k.hi) k.hi = last < -1 ? 0 : static_cast<int>(last + 1);
  }
  if (a.window) {
    const int64_t first = static_cast<int64_t>(r.kv) - r.n + i0 - a.window + 1;
    if (first > 0) k.lo = first > k.hi ? k.hi : static_cast<int>(first);
  }
  return k;
}

// Keys [lo, hi) of query i among those of keys_of; NaN in *sum, the row's sum
// of weights to begin with, where it sees others past them, else 0.
template <typename T>
__device__ __forceinline__ Keys see_of(const AttnArgs<T>& a, const Request& r, int i, float* sum) {
  const int64_t pos = static_cast<int64_t>(r.kv) - r.n + i;
  Keys k{0, r.kv};
  if (a.causal && pos + 1 < r.kv) k.hi = pos < 0 ? 0 : static_cast<int>(pos + 1);
  if (a.window && pos - a.window + 1 > 0) k.lo = static_cast<int>(pos - a.window + 1);
  *sum = k.hi > a.reach && k.hi > k.lo ? NAN : 0.0f;
  if (k.hi > a.reach) k.hi = a.reach;
  return k;
}

// The attention kernels' work is units, some rows of one key head, each with
// the tiles of keys that any of its rows sees (one at least, whose keys may all
// be masked).  The units' tiles, laid end to end, are dealt out evenly: every
// workgroup takes a range of the same length, so it works through the end of
// one unit, whole units, and the beginning of another, and the ragged lengths
// of the requests do not matter.  Units that several workgroups share are
// joined by a second kernel.
struct Range {
  int32_t id;       // which of the ranges
  int64_t at, end;  // tiles
  int64_t chunk;    // end - at, or more where the tiles end
};
// The workgroup's range of `total` tiles, a multiple of `step` long; false when
// it is empty.
template <typename T>
__device__ __forceinline__ bool take_range(const AttnArgs<T>& a, int64_t total, int step, int least, Range* r) {
  int64_t chunk = total <= INT32_MAX - static_cast<int64_t>(gridDim.x)
                      ? a.by_grid.div(static_cast<uint32_t>(total + gridDim.x - 1))
                      : (total + gridDim.x - 1) / gridDim.x;
  chunk = (chunk + step - 1) / step * step;
  if (chunk < least) chunk = least;
  r->chunk = chunk;
  r->at = r->id * chunk;
  r->end = r->at + chunk < total ? r->at + chunk : total;
  if (r->at < r->end) return true;
  if (a.units && threadIdx.x == 0) a.units[r->id].off = 0;
  return false;
}

// The same from the tiles of `n` groups of units, `times` over: each thread adds
// up a run of groups, a scan over the workgroup gives where the runs begin.
// Also the time and the group that hold the range's first tile, and where that
// group begins.
template <int WAVES, typename T, typename F>
__device__ __forceinline__ bool deal_out(const AttnArgs<T>& a, int n, F tiles, int times, int step, int least, Range* r,
                                         int* time, int* group, int64_t* group_at) {
  __shared__ int64_t run_start[64 * WAVES];
  __shared__ int64_t wave_sums[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int run = static_cast<int>((static_cast<int64_t>(n) + 64 * WAVES - 1) / (64 * WAVES));
  const int64_t g0 = static_cast<int64_t>(tid) * run;
  int64_t mine = 0;
  for (int64_t i = g0; i < g0 + run && i < n; ++i) mine += tiles(static_cast<int>(i));
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 63) wave_sums[wv] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w < wv) sum += wave_sums[w];
    total += wave_sums[w];
  }
  run_start[tid] = sum - mine;
  __syncthreads();
  if (!take_range(a, total * times, step, least, r)) return false;
  *time = static_cast<int>(r->at / total);
  const int64_t first = r->at - *time * total;
  int i = 0;  // the last run that begins at or before the range
#pragma unroll
  for (int d = 64 * WAVES / 2; d > 0; d >>= 1)
    if (run_start[i + d] <= first) i += d;
  int64_t at = run_start[i];
  int g = i * run;
  for (int64_t k = tiles(g); first >= at + k; k = tiles(++g)) at += k;
  *group = __builtin_amdgcn_readfirstlane(g);
  *group_at = r->at - (first - at);
  return true;
}

// Scales a block of an output row, rotates it back and writes it.
template <typename T>
__device__ __forceinline__ void write_block(const AttnArgs<T>& a, int row0, int head, int row, int block,
                                            float z[16], float f, float back) {
  const int oi = static_cast<int>(a.by_group.div(static_cast<uint32_t>(row)));
  const int oh = head * a.group + (row - oi * a.group);
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] *= f;
  if (a.cache.rotate) rotate16_block(z);
  if (back != 1.0f) {  // the same for every row
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] *= back;
  }
  store16(a.out + static_cast<int64_t>(row0 + oi) * a.o_token + oh * a.o_head + block * 16, z);
}

// ---------------------------------------------------------------- few rows

// A unit is 16 RT query rows of one key head of a request (its tokens times
// the heads that share the key head), its tiles 32 keys; units go by requests,
// then rows, then heads.  They are dealt out by tiles (SPLIT) or as whole units.
// The four waves take every fourth tile each and merge at a unit's end.
//
// Reading the pages is what has to be done, and decoding them costs the vector
// units about as long, so a wave keeps the next tile's bytes on their way (in
// registers) while it multiplies the present one, looks up the pages of its
// next 32 tiles at once, two lanes a tile, and leaves the matrix units, which
// have time to spare, twice the work for V: a byte of V holds two elements of
// one token, and converts to two neighbouring k-slots of an operand.  Instead
// of transposing codes until neighbours are two tokens of one element (some 45
// vector instructions a tile), the weights are given once as (p, 0) and once
// as (0, p), which sums the even and the odd elements apart.
//
// One token each of 64 requests over up to 8192 keys of 8 heads of 128: 80 us,
// 4.7 TB/s of K and V; 2 requests over up to 262144 keys: 83 us in the kernel,
// 5.8 TB/s, and 7 us in the join.  Small calls (one token over 777 keys: 10.6
// us) are bound by their chain of loads: lengths, pages, bytes, each a
// microsecond or more.
constexpr int kAttnWaves = 4;
constexpr int kTile = 32;     // keys
// Tiles of a workgroup's range, at least: 7 requests of 33 tokens in a window of
// 1024 take 22 us, with 8 tiles 25, with 32 tiles 26.
constexpr int kMinTiles = 16;

// A tile's bytes as a lane holds them: K rows tok, tok + 4 of its quarter of
// D, V's octet of its slice.
template <int D>
struct RowsRaw {
  uint32_t k[2][D / 32], ks[2];
  uint32_t v[D / 16];
  u32x2 vs;
};

// N words; ONCE: read once, past the caches' retention (400 MB read by a plain
// kernel: 7.0 TB/s so, 6.2 TB/s with ordinary loads).
template <bool ONCE, typename V>
__device__ __forceinline__ V load_vector(const uint8_t* p) {
  if constexpr (ONCE)
    return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
  else
    return *reinterpret_cast<const V*>(p);
}
template <bool ONCE, int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 2) {
    const u32x2 v = load_vector<ONCE, u32x2>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 v = load_vector<ONCE, u32x4>(p + 4 * i);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  }
}

// Waves a SIMD that the rows kernel's registers are cut to: what it takes
// without going to scratch memory.
constexpr int rows_waves(bool split, int d, int rt) {
  if (rt == 1) return d == 64 ? (split ? 3 : 4) : d == 128 ? (split ? 2 : 3) : (split ? 1 : 2);
  return d == 64 ? 2 : d == 128 && !split ? 2 : 1;
}
// 16-row tiles of a unit.  At head_dim 256 one of 32 rows fills a SIMD's
// registers with one wave: 41.9 us against 36.3 with two units of 16 (12
// requests of 32 rows over 16000 keys).
constexpr int most_row_tiles(int d) { return d == 256 ? 1 : 2; }

template <typename T, int D, int RT, bool PAGE16, bool SPLIT>
__global__ __launch_bounds__(64 * kAttnWaves, rows_waves(sizeof(T) == 4, D, RT)) void kv_attn_rows_kernel(
    AttnArgs<T> a) {
  using Rec = KvRecord<D>;
  constexpr bool kSplit = sizeof(T) == 4;
  constexpr int L = Rec::L, KK = D / 32, NB = D / 64;  // k-steps, blocks of a lane's share of a row
  constexpr int NQ = kSplit ? 2 : 1, kRows = 16 * RT;
  constexpr bool kOnce = D < 256;  // there two row groups may read the same pages
  __shared__ float merge_o[kAttnWaves][16][D + 4];
  __shared__ float merge_ml[kAttnWaves][16][2];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int shift = a.cache.shift, heads = a.cache.kv_heads;
  const int64_t record = Rec::bytes(shift);
  auto query_of = [&](int row) { return static_cast<int>(a.by_group.div(static_cast<uint32_t>(row))); };
  auto rows_of = [&](const Request& q) {  // at most kMostRows: tokens * query heads is
    const int rows = q.n * a.group;
    return rows > a.few ? 0 : rows;
  };
  // keys of rows base .. base + kRows - 1, and their tiles: one at least, whose
  // keys may all be masked
  auto keys_at = [&](const Request& q, int rows, int base) {
    return keys_of(a, q, query_of(base), query_of(rows - base > kRows ? base + kRows - 1 : rows - 1) + 1);
  };
  auto tiles_of = [&](Keys k) { return k.hi > k.lo ? (k.hi + kTile - 1) / kTile - k.lo / kTile : 1; };

  // what is dealt out: tiles, or whole units
  constexpr int kStep = SPLIT ? kAttnWaves : 1, kLeast = SPLIT ? kMinTiles : 1;
  auto cost_of = [&](Keys k) { return SPLIT ? tiles_of(k) : 1; };

  auto cost_at = [&](const Request& q) {
    const int rows = rows_of(q);
    int64_t n = 0;
    for (int base = 0; base < rows; base += kRows) n += cost_of(keys_at(q, rows, base));
    return n * heads;
  };
  Range range;
  range.id = blockIdx.x;
  int req;
  Request rq;
  int64_t unit_at;  // where the unit that holds range.at begins
  constexpr int64_t kFewTiles = 1 << 24;
  bool small = a.requests <= 64;
  if (small) {
    // A lane per request, whose running sum each wave forms for itself,
    // without a barrier (1.0 us instead of 2.9 from the kernel's start).
    Request mine{0, 0, 0};
    int64_t cost = 0;
    if (lane < a.requests) {
      mine = request_of(a, lane);
      cost = cost_at(mine);
    }
    small = !__any(cost > kFewTiles);
    if (small) {
      const int n = static_cast<int>(cost), sum = wave_scan(n);
      if (!take_range(a, __builtin_amdgcn_readlane(sum, 63), kStep, kLeast, &range)) return;
      // the last request that begins at or before the range
      req = 63 - __builtin_clzll(__ballot(sum - n <= range.at));
      rq = Request{__builtin_amdgcn_readlane(mine.row0, req), __builtin_amdgcn_readlane(mine.n, req),
                   __builtin_amdgcn_readlane(mine.kv, req)};
      unit_at = __builtin_amdgcn_readlane(sum - n, req);
    }
  }
  if (!small) {
    int once;
    if (!deal_out<kAttnWaves>(a, a.requests, [&](int r) { return cost_at(request_of(a, r)); }, 1, kStep,
                              kLeast, &range, &once, &req, &unit_at))
      return;
    rq = request_of(a, req);
  }
  int64_t at = range.at;
  const int64_t end = range.end;
  int rows = rows_of(rq), base = 0, head = 0;
  Keys keys = keys_at(rq, rows, base);
  int unit_cost = cost_of(keys);
  while (at >= unit_at + static_cast<int64_t>(unit_cost) * heads) {
    unit_at += static_cast<int64_t>(unit_cost) * heads;
    base += kRows;
    keys = keys_at(rq, rows, base);
    unit_cost = cost_of(keys);
  }
  head = at - unit_at <= INT32_MAX ? static_cast<int>(at - unit_at) / unit_cost
                                   : static_cast<int>((at - unit_at) / unit_cost);
  unit_at += static_cast<int64_t>(head) * unit_cost;
  if (SPLIT && tid == 0)
    a.units[blockIdx.x] =
        RangeUnit{range.chunk, rq.row0, rows, base, head, static_cast<int32_t>(at - unit_at), unit_cost};

  // the units of the range, one after the other
  for (bool first_unit = true; at < end; first_unit = false) {
    if (!first_unit) {
      if (++head == heads) {
        head = 0;
        base += kRows;
        while (base >= rows) {  // at < end: there is a request with rows
          if (++req >= a.requests) return;
          rq = request_of(a, req);
          rows = rows_of(rq);
          base = 0;
        }
        keys = keys_at(rq, rows, base);
        unit_cost = cost_of(keys);
      }
      unit_at = at;
    }
    const int i0 = query_of(base);
    const int i1 = query_of(rows - base > kRows ? base + kRows - 1 : rows - 1) + 1;
    const int off = static_cast<int>(at - unit_at);
    const int here = static_cast<int>(end - at < unit_cost - off ? end - at : unit_cost - off);
    const int t0 = keys.lo / kTile + off, t_first = t0 + wv, t_end = t0 + (SPLIT ? here : tiles_of(keys));
    const bool whole = !SPLIT || here == unit_cost;
    const int32_t* row_table = a.table + static_cast<int64_t>(req) * a.table_width;

    // pages of 32 of the wave's tiles from its b-th on: lane 2 i + h has the
    // page of tile b + i's half h, -1 where that is none of the cache's or no
    // row sees any of the half's keys
    auto lookup = [&](int b) -> int {
      const int key = (t_first + kAttnWaves * (b + (lane >> 1))) * kTile + 16 * (lane & 1);
      const int64_t col = key >> shift;
      int p = -1;
      if (key < t_end * kTile && key < keys.hi && key + 16 > keys.lo) p = row_table[col];
      return p >= 0 && p < a.cache.pages ? p : -1;
    };
    int pages = lookup(0), pages_at = 0;
    float z[RT][D / 4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = base + 16 * rt + r16;
      if (row < rows) {
        const int qi = query_of(row), qh = head * a.group + row - qi * a.group;
        const T* p = a.q + static_cast<int64_t>(rq.row0 + qi) * a.q_token + qh * a.q_head + g * (D / 4);
#pragma unroll
        for (int b = 0; b < NB; ++b) load_block(p, b, z[rt] + 16 * b, z[rt] + 16 * b + 8);
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) z[rt][i] = 0.0f;
      }
    }

    // Row r16 of K tile u (of 16) is token 8 (r16 / 4) + r16 % 4 + 4 u, so that
    // the lane's logits are those of its octet's tokens 4 u .. 4 u + 3; tokens
    // of r16 / 8 = 1, and octets of g / 2 = 1, are in the tile's second half.
    const int k_tok = 8 * ((r16 >> 2) & 1) + (r16 & 3), v_oct = g & 1;
    const int k_half = r16 >> 3, v_half = g >> 1;
    const uint32_t k_lane = static_cast<uint32_t>(Rec::k_row(k_tok)) + g * (D / 8);
    const uint32_t ks_lane = static_cast<uint32_t>(Rec::k_scales(shift) + Rec::k_scale(k_tok, g * NB));
    const uint32_t v_lane = static_cast<uint32_t>(Rec::v_codes(shift) + Rec::v_slice(8 * v_oct, r16));
    const uint32_t vs_lane = static_cast<uint32_t>(Rec::v_scales(shift) + Rec::v_scale(8 * v_oct, r16 * L / 16));
    const int in_page = (1 << shift) - 1;
    // The wave's i-th tile; past the last one, and where a page is not there,
    // page 0 is read and not used: the loads are unconditional, so that the
    // wait for one tile's bytes leaves the next one's in flight.  A tile lies
    // on one page, or, with pages of 16 tokens, on two.
    auto load = [&](RowsRaw<D>& raw, int i, bool* bad0, bool* bad1) {
      if (i - pages_at >= 32) {
        pages_at = i;
        pages = lookup(i);
      }
      const int key0 = (t_first + kAttnWaves * i) * kTile;
      const int p0 = __builtin_amdgcn_readlane(pages, 2 * (i - pages_at));
      const int p1 = __builtin_amdgcn_readlane(pages, 2 * (i - pages_at) + 1);
      *bad0 = p0 < 0;
      *bad1 = p1 < 0;
      const uint8_t *kr, *sr, *vr, *wr;
      if constexpr (PAGE16) {
        const int64_t rec0 = (static_cast<int64_t>(p0 < 0 ? 0 : p0) * heads + head) * record;
        const int64_t apart = (static_cast<int64_t>(p1 < 0 ? 0 : p1) * heads + head) * record - rec0;
        const uint8_t* rec = a.cache.data + rec0;
        const uint8_t *kh = rec + (apart & -static_cast<int64_t>(k_half)), *vh = rec + (apart & -static_cast<int64_t>(v_half));
        kr = kh + k_lane;
        sr = kh + ks_lane;
        vr = vh + v_lane;
        wr = vh + vs_lane;
      } else {
        // both halves on the page of one that is there
        const int p = p0 < 0 ? (p1 < 0 ? 0 : p1) : p0;
        const uint8_t* rec = a.cache.data + (static_cast<int64_t>(p) * heads + head) * record;
        const int in = key0 & in_page;
        kr = rec + Rec::k_row(in) + (k_lane + k_half * static_cast<uint32_t>(Rec::k_row(16)));
        sr = rec + Rec::k_scale(in, 0) + (ks_lane + k_half * static_cast<uint32_t>(Rec::k_scale(16, 0)));
        vr = rec + Rec::v_slice(in, 0) + (v_lane + v_half * static_cast<uint32_t>(Rec::v_slice(16, 0)));
        wr = rec + Rec::v_scale(in, 0) + (vs_lane + v_half * static_cast<uint32_t>(Rec::v_scale(16, 0)));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        load_words<kOnce, KK>(kr + u * Rec::k_row(4), raw.k[u]);
        const uint8_t* s = sr + u * Rec::k_scale(4, 0);
        if constexpr (NB == 1) raw.ks[u] = *s;
        else if constexpr (NB == 2) raw.ks[u] = *reinterpret_cast<const uint16_t*>(s);
        else raw.ks[u] = *reinterpret_cast<const uint32_t*>(s);
      }
      load_words<kOnce, L>(vr, raw.v);
      raw.vs = *reinterpret_cast<const u32x2*>(wr);
    };
    RowsRaw<D> even, odd;
    bool e0, e1, o0, o1;
    load(even, 0, &e0, &e1);

    // the lane's quarter of its rows of Q^T, rotated, as fp16 operands
    half8_t qf[RT][NQ][KK];
    float c[RT];                  // logit factors, log2 domain
    int see_lo[RT], see_hi[RT];   // keys that the row sees
    float m[RT], l[RT];           // maximum and sum of its weights
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = base + 16 * rt + r16;
      const int qi = query_of(row < rows ? row : 0);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (a.cache.rotate) rotate16_block(z[rt] + 16 * b);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(z[rt][i]));
      const int e = row_exponent(max_over_rows(top));
#pragma unroll
      for (int k = 0; k < KK; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = __builtin_ldexpf(z[rt][8 * k + j], e);
          const _Float16 h = static_cast<_Float16>(v);
          qf[rt][0][k][j] = h;
          if (kSplit) qf[rt][NQ - 1][k][j] = static_cast<_Float16>(v - static_cast<float>(h));
        }
      c[rt] = logit_factor(a.scale, a.cache.amax[0], e);
      const Keys see = see_of(a, rq, qi, &l[rt]);
      see_lo[rt] = see.lo;
      see_hi[rt] = see.hi;
    }
    // keys that every row sees
    const Keys inner{a.window ? keys_of(a, rq, i1 - 1, i1).lo : 0, keys_of(a, rq, i0, i0 + 1).hi};

    f32x4 o[RT][L];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY;
#pragma unroll
      for (int j = 0; j < L; ++j) o[rt][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    auto use = [&](const RowsRaw<D>& raw, int i, bool bad0, bool bad1) {
      const int key0 = (t_first + kAttnWaves * i) * kTile;
      f32x4 s[RT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const half2_t lo = scale2<false>(raw.ks[u]), hi = scale2<true>(raw.ks[u]);
#pragma unroll
        for (int k = 0; k < KK; ++k) {
          const int b = k / 2;  // block of the lane's share
          const _Float16 f = (b < 2 ? lo : hi)[b & 1];
          const half8_t kf = decode8(raw.k[u][k], half2_t{f, f});
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int x = 0; x < NQ; ++x)
              s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[rt][x][k], s[rt][u], 0, 0, 0);
        }
      }
      // the lane's octet: tokens 8 g .. 8 g + 7
      const int key8 = key0 + 8 * g;
      const bool edge = key0 < inner.lo || key0 + kTile > inner.hi || bad0 || bad1;
      u32x2 vs = raw.vs;
      if (edge) {
        const bool vbad = g >= 2 ? bad1 : bad0;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bool seen = key8 + j >= see_lo[rt] && key8 + j < see_hi[rt];
            if (!seen || vbad) s[rt][j >> 2][j & 3] = seen ? NAN : -INFINITY;
          }
        // keys that no row sees hold anything: their V is taken as 0
        uint64_t keep = ~uint64_t{0};
        const int before = keys.lo - key8, after = key8 + 8 - keys.hi;
        if (vbad || before >= 8 || after >= 8) {
          keep = 0;
        } else {
          if (before > 0) keep &= ~uint64_t{0} << (8 * before);
          if (after > 0) keep &= ~uint64_t{0} >> (8 * after);
        }
        vs.x &= static_cast<uint32_t>(keep);
        vs.y &= static_cast<uint32_t>(keep >> 32);
      }
      // weights of the octet's tokens 4 q .. 4 q + 3 at k-slots 2 i (x = 0) or
      // 2 i + 1 (x = 1) of the token's pair, the other slot 0
      half8_t pf[RT][NQ][2][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = s[rt][0][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = __builtin_fmaxf(top, s[rt][j >> 2][j & 3]);
        top = max_over_rows(top) * c[rt];
        if (__any(top > m[rt] + kRaise)) {
          const float mn = __builtin_fmaxf(m[rt], top);
          const float f = m[rt] == mn ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - mn);
          l[rt] *= f;
#pragma unroll
          for (int j = 0; j < L; ++j) o[rt][j] *= f;
          m[rt] = mn;
        }
        const float shift_m = (m[rt] == -INFINITY ? 0.0f : m[rt]) - kWeightBits;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][j >> 2][j & 3], c[rt], -shift_m));
          l[rt] += p;
          const _Float16 h = static_cast<_Float16>(p), zero = static_cast<_Float16>(0.0f);
          const int q = j >> 2, i = 2 * (j & 3);
          pf[rt][0][q][0][i] = h;
          pf[rt][0][q][0][i + 1] = zero;
          pf[rt][0][q][1][i] = zero;
          pf[rt][0][q][1][i + 1] = h;
          if (kSplit) {
            const _Float16 rest = static_cast<_Float16>(p - static_cast<float>(h));
            pf[rt][NQ - 1][q][0][i] = rest;
            pf[rt][NQ - 1][q][0][i + 1] = zero;
            pf[rt][NQ - 1][q][1][i] = zero;
            pf[rt][NQ - 1][q][1][i + 1] = rest;
          }
        }
      }
      // V: 8 tokens of the L elements n L .. n L + L - 1, n = r16
      half2_t sc[4];
      v_scales8(vs, sc);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < L / 2; ++e) {  // elements 2 e, 2 e + 1 of tokens 4 q .. 4 q + 3
          union { half2_t h[4]; half8_t v; } vf;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int tok = 4 * q + j;
            const _Float16 f = sc[tok >> 1][tok & 1];
            if constexpr (L == 4)  // a token's 4 codes are half a word
              vf.h[j] = code_pair(raw.v[tok >> 1], 2 * (tok & 1) + e) * half2_t{f, f};
            else
              vf.h[j] = code_pair(raw.v[tok * (L / 8) + (e >> 2)], e & 3) * half2_t{f, f};
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int x = 0; x < NQ; ++x)
#pragma unroll
              for (int odd = 0; odd < 2; ++odd)
                o[rt][2 * e + odd] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf.v, pf[rt][x][q][odd], o[rt][2 * e + odd], 0, 0, 0);
        }
    };

    const int count = t_end > t_first ? (t_end - t_first + kAttnWaves - 1) / kAttnWaves : 0;
    for (int i = 0; i < count; i += 2) {
      load(odd, i + 1, &o0, &o1);
      use(even, i, e0, e1);
      load(even, i + 2, &e0, &e1);
      if (i + 1 < count) use(odd, i + 1, o0, o1);
    }

    // merge the four waves: the lane holds elements (4 g + i) L + j of its rows
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (base + 16 * rt >= rows) break;
      const float lt = sum_over_rows(l[rt]);
      if (g == 0) {
        merge_ml[wv][r16][0] = m[rt];
        merge_ml[wv][r16][1] = lt;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < L; ++j) merge_o[wv][r16][(4 * g + i) * L + j] = o[rt][j][i];
      __syncthreads();
      for (int u = threadIdx.x; u < 16 * L; u += 64 * kAttnWaves) {  // a block of a row
        const int rr = u / L, b = u % L;
        const int orow = base + 16 * rt + rr;
        if (orow >= rows) continue;
        float mm = merge_ml[0][rr][0];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) mm = __builtin_fmaxf(mm, merge_ml[w][rr][0]);
        float z[16], ll = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) {
          const float mw = merge_ml[w][rr][0];
          const float f = mw == mm ? 1.0f : __builtin_amdgcn_exp2f(mw - mm);
          ll = __builtin_fmaf(f, merge_ml[w][rr][1], ll);
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = __builtin_fmaf(f, merge_o[w][rr][b * 16 + i], z[i]);
        }
        if (!whole) {
          // slot 0: the unit that the range begins with; 1: one that begins in it
          const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (first_unit ? 0 : 1)) * kRows + orow - base;
          store16(a.part + slot * D + b * 16, z);
          if (b == 0) {
            a.part[a.part_ml + 2 * slot] = mm;
            a.part[a.part_ml + 2 * slot + 1] = ll;
          }
        } else {
          const OutScale gv = out_scale(a.cache.amax[1]);
          write_block(a, rq.row0, head, orow, b, z, gv.over(ll), gv.back);
        }
      }
      __syncthreads();  // the next rows write the merge buffers again
    }
    at += here;
  }
}

// ---------------------------------------------------------------- many rows

// A unit is 32 rows a wave of one key head, its tiles 2048 NW / D keys (NW
// waves); units go by heads, then tiles of rows.  A tile of K and V is decoded
// once for all waves, into LDS, in the order in which the matrix instructions
// read it: a fragment of 64 lanes x 16 bytes for each 32 x 16 operand.  Half
// the waves decode V, half K; the next tile's bytes are on their way while the
// present one is multiplied, and are decoded into the other buffer.
//
// With many units a workgroup takes one of them; with few, their tiles are
// dealt out evenly (RANGED), which costs writing and joining partial sums of up
// to two units a workgroup.
//
// Bound by the SIMDs' issue and by power.  A tile of 128 keys at head_dim 128
// takes a SIMD 8350 cycles, 4096 of them in matrix instructions and about as
// many in the softmax (2 waves' exp2, fma, sum and conversion of 64 logits a
// lane, 3200) and in decoding (900); LDS serves 512 KB of operands in 4096.
// The waves overlap these little, at a clock of 1.9 GHz.  A whole prompt of
// 8192 tokens, 32 query heads on 8, takes 553 us, 994 TFLOP/s, with a large
// fp16 matrix product of the library at 1405.  Slower: 4 waves of 32 rows (603
// us), 4 waves of 64 rows with the next tile's logits beside this one's weights
// (742 us), weights summed by dot products (556 us).
constexpr int kFragBytes = 64 * 16 + 16;  // the odd 16 bytes spread K's writes over the banks: 569 us, 576 without
constexpr int kMinKeys = 256;             // of a workgroup's range
// A unit's own cost, its queries and its output, in tiles (a tile takes 4.3 us,
// the rest of a unit 9 us): a prompt of 2048 tokens in 256 ranges takes 90 us
// so, 98 us at 1 tile, 96 us at 4 and 119 us at none.
constexpr int kUnitTiles = 2;
typedef float f32x16 __attribute__((ext_vector_type(16)));

// The request and the first row of tile `tile`.  Request i's tiles begin at
// floor(cu_i group / BM) + i, which leaves each at least as many as it needs
// without anything having been counted: floor((a + n) / b) + 1 - floor(a / b)
// >= ceil(n / b).
template <int BM, typename T>
__device__ __forceinline__ int tile_start(const AttnArgs<T>& a, int r) {
  int c = a.cu_q[r];
  c = c < 0 ? 0 : (c > a.tokens ? a.tokens : c);
  return static_cast<int>(static_cast<uint32_t>(c) * static_cast<uint32_t>(a.group) / BM) + r;
}
template <int BM, typename T>
__device__ __forceinline__ int tile_request(const AttnArgs<T>& a, int tile) {
  int lo = 0, hi = a.requests;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (tile_start<BM>(a, mid) <= tile) lo = mid; else hi = mid;
  }
  return lo;
}

// What a thread holds of a tile between its loads and its decoding: for V one
// cell of 8 tokens x 8 elements, for K two pieces of 32 elements of a token.
struct TileRaw {
  u32x4 w0, w1;
  uint32_t s0, s1;
};

// A workgroup of NW waves; its tile of keys is 2048 NW / D long, which its
// threads decode in one go.
template <int D, int NW>
struct TileShape {
  static constexpr int BM = 32 * NW;        // rows
  static constexpr int BN = 2048 * NW / D;  // keys
  static constexpr int F = 4 * NW;          // fragments of K, and of V
  static constexpr int KC = D / 32;         // pieces of a K row
  static constexpr int VC = D / 8;          // cells across a V row
  static constexpr int JW = 32 / VC;        // elements of a cell in one 32-row operand
  static constexpr int GA = VC / 8;
};

template <typename T, int D, int NW, bool RANGED>
__global__ __launch_bounds__(64 * NW, NW / 4) void kv_attn_tiles_kernel(AttnArgs<T> a) {
  using Rec = KvRecord<D>;
  using Sh = TileShape<D, NW>;
  constexpr bool kSplit = sizeof(T) == 4;
  constexpr int NQ = kSplit ? 2 : 1, KS = D / 16, NT = Sh::BN / 32, DT = D / 32, L = Rec::L;
  constexpr int kBufBytes = 2 * Sh::F * kFragBytes;
  constexpr int kUnitCost = RANGED ? kUnitTiles : 0;
  __shared__ __attribute__((aligned(16))) uint8_t frags[2 * kBufBytes];  // twice: K's, then V's
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  const int shift = a.cache.shift, heads = a.cache.kv_heads;
  const int64_t record = Rec::bytes(shift);
  auto query_of = [&](int row) { return static_cast<int>(a.by_group.div(static_cast<uint32_t>(row))); };
  // rows of a request that this kernel takes
  auto rows_of = [&](const Request& q) {
    const int rows = q.n * a.group;
    return rows <= a.few ? 0 : rows;
  };
  auto keys_at = [&](const Request& q, int rows, int base) {
    return keys_of(a, q, query_of(base), query_of(rows - base > Sh::BM ? base + Sh::BM - 1 : rows - 1) + 1);
  };
  // tiles of a unit, with kUnitCost to deal out before its first one
  auto tiles_of = [&](Keys k) {
    return kUnitCost + (k.hi > k.lo ? (k.hi + Sh::BN - 1) / Sh::BN - k.lo / Sh::BN : 1);
  };
  // first row of the tile of rows within its request; past its last where there
  // is none
  auto base_of = [&](int row_tile, int r) {
    const int64_t b = static_cast<int64_t>(row_tile - tile_start<Sh::BM>(a, r)) * Sh::BM;
    return b < 0 || b > INT32_MAX ? INT32_MAX : static_cast<int>(b);
  };

  int row_tile, head, req;
  int64_t at = 0, end = 1, unit_at = 0, chunk = 0;
  // Workgroup b runs on XCD b % 8: ranges that lie next to each other, and so
  // read the same head's pages, go to the same one and its L2 (a whole prompt
  // of 8192 tokens in 256 ranges: 1129 us without).
  int range_id = blockIdx.x;
  if (gridDim.x % 8 == 0) range_id = (range_id & 7) * (gridDim.x / 8) + (range_id >> 3);
  if constexpr (RANGED) {
    Range range;
    range.id = range_id;
    auto tiles_at = [&](int t) -> int64_t {
      const int r = tile_request<Sh::BM>(a, t);
      const Request q = request_of(a, r);
      const int rows = rows_of(q), base = base_of(t, r);
      return base < rows ? tiles_of(keys_at(q, rows, base)) : 0;
    };
    constexpr int kLeast = kMinKeys / Sh::BN > 0 ? kMinKeys / Sh::BN : 1;
    if (!deal_out<NW>(a, a.tiles, tiles_at, heads, 1, kLeast, &range, &head, &row_tile, &unit_at)) return;
    at = range.at;
    end = range.end;
    chunk = range.chunk;
  } else {
    const uint32_t back = a.by_heads.div(blockIdx.x);
    head = static_cast<int>(blockIdx.x - back * a.by_heads.d);
    // last tiles first: under a causal mask they have the most keys
    row_tile = a.tiles - 1 - static_cast<int>(back);
  }
  req = __builtin_amdgcn_readfirstlane(tile_request<Sh::BM>(a, row_tile));
  Request rq = request_of(a, req);
  int rows = rows_of(rq), base = base_of(row_tile, req);
  if (base >= rows) return;  // only where a workgroup takes one unit
  Keys keys = keys_at(rq, rows, base);
  int unit_tiles = tiles_of(keys);
  if constexpr (RANGED) {
    if (tid == 0)
      a.units[range_id] = RangeUnit{chunk, rq.row0, rows, base, head, static_cast<int32_t>(at - unit_at), unit_tiles};
  } else {
    end = unit_tiles;
  }

  for (bool first_unit = true; at < end; first_unit = false) {
    if (RANGED && !first_unit) {
      do {  // at < end: there is a tile with rows
        if (++row_tile == a.tiles) {
          row_tile = 0;
          if (++head == heads) return;
        }
        req = __builtin_amdgcn_readfirstlane(tile_request<Sh::BM>(a, row_tile));
        rq = request_of(a, req);
        rows = rows_of(rq);
        base = base_of(row_tile, req);
      } while (base >= rows);
      keys = keys_at(rq, rows, base);
      unit_tiles = tiles_of(keys);
      unit_at = at;
    }
    const int off = static_cast<int>(at - unit_at);
    const int here = static_cast<int>(end - at < unit_tiles - off ? end - at : unit_tiles - off);
    auto tile_at = [&](int n) { return keys.lo / Sh::BN + (n > kUnitCost ? n - kUnitCost : 0); };
    const int t0 = tile_at(off), t1 = tile_at(off + here);
    const bool whole = !RANGED || here == unit_tiles;
    const int32_t* row_table = a.table + static_cast<int64_t>(req) * a.table_width;
    auto last_of = [&](int first, int count) { return rows - first > count ? first + count - 1 : rows - 1; };

    // this wave's rows
    const int wbase = base + 32 * wv;
    const bool wave_live = wbase < rows;
    const int row = wbase + r32;
    const bool live = row < rows;
    const int qi = query_of(live ? row : 0);
    const int qh = head * a.group + (live ? row : 0) - qi * a.group;
    Keys inner{0, 0};  // keys that all of them see
    if (wave_live) {
      const int w0 = query_of(wbase), w1 = query_of(last_of(wbase, 32)) + 1;
      inner = Keys{a.window ? keys_of(a, rq, w1 - 1, w1).lo : 0, keys_of(a, rq, w0, w0 + 1).hi};
    }
    half8_t qf[NQ][KS];
    float c;
    {
      // the lane's half of every block of its row; the butterfly's last stage
      // takes the other half from the lane 32 away
      float top = 0.0f;
      const T* p = a.q + static_cast<int64_t>(rq.row0 + qi) * a.q_token + qh * a.q_head + 8 * half;
      const uint32_t sign = static_cast<uint32_t>(half) << 31;
      float mine[KS][8];
#pragma unroll
      for (int b = 0; b < KS; ++b) {
        if (live) {
          load_half(p + 16 * b, mine[b]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) mine[b][i] = 0.0f;
        }
        if (a.cache.rotate) {
          stages_1_2_4(mine[b]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t z = __float_as_uint(mine[b][i]);
            const auto both = __builtin_amdgcn_permlane32_swap(z, z, false, false);
            mine[b][i] = 0.25f * (__uint_as_float(both[0]) + __uint_as_float(both[1] ^ sign));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(mine[b][i]));
      }
      {
        const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        top = __builtin_fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1]));
      }
      const int e = row_exponent(top);
#pragma unroll
      for (int b = 0; b < KS; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = __builtin_ldexpf(mine[b][i], e);
          const _Float16 h = static_cast<_Float16>(v);
          qf[0][b][i] = h;
          if (kSplit) qf[NQ - 1][b][i] = static_cast<_Float16>(v - static_cast<float>(h));
        }
      c = logit_factor(a.scale, a.cache.amax[0], e);
    }
    float m = -INFINITY, l;
    const Keys see = see_of(a, rq, qi, &l);
    f32x16 o[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] = 0.0f;

    // The part of a tile that this thread decodes: a V cell (8 tokens of 8
    // elements), or two K pieces (32 elements of a token) some tokens apart.
    // Its first token, and its places in a record (codes and scales advance by
    // D / 2 and L bytes a token in both layouts) and in the buffer.
    const bool does_v = (wv & 2) == 0;
    const int part = ((wv >> 2) * 2 + (wv & 1)) * 64 + lane;
    int tok;
    uint32_t code_at, scale_at, put_at;
    if (does_v) {
      const int vc = part % Sh::VC, vo = part / Sh::VC;
      tok = 8 * vo;
      // cell vc is slice vc, or half a slice, or two slices
      code_at = static_cast<uint32_t>(Rec::v_codes(shift)) +
                (L == 16 ? (vc >> 1) * (4 * L) + (vc & 1) * 4 : vc * 32);
      scale_at = static_cast<uint32_t>(Rec::v_scales(shift)) + (vc >> 1) * 8;
      put_at = (Sh::F + (vo >> 1)) * kFragBytes + ((vo & 1) * 32 + vc) * 16;
    } else {
      const int piece = part % Sh::KC;
      tok = part / Sh::KC;
      code_at = piece * 16;
      scale_at = static_cast<uint32_t>(Rec::k_scales(shift)) + piece * 2;
      // token tk of 32 is row 8 (2 (tk / 16) + (tk / 4) % 2) + 4 ((tk / 8) % 2) +
      // tk % 4, so that a lane's results are whole octets
      const int tk = tok & 31;
      put_at = ((tok >> 5) * KS + 2 * piece) * kFragBytes +
               (8 * (2 * (tk >> 4) + ((tk >> 2) & 1)) + 4 * ((tk >> 3) & 1) + (tk & 3)) * 16;
    }
    constexpr int kApart = 32 * NW / Sh::KC;  // a multiple of 16 tokens
    constexpr int kApartBytes = kApart == 16 ? 16 * 16 : (kApart / 32) * KS * kFragBytes;

    // Every load below is unconditional, from a place that is there: a wait for
    // one then leaves the later ones in flight, and nothing is waited for where
    // it is loaded.  Past the table's row, where no key is seen, the last entry
    // is read, for an id outside the cache page 0; neither is used.
    const int32_t* ids_from = a.table_width > 0 ? row_table : a.cu_q;
    const int last_col = a.table_width > 0 ? static_cast<int>(a.table_width) - 1 : 0;
    const int in_page = (1 << shift) - 1;
    int32_t id0, id1;  // pages of the next tile's bytes to load
    auto load_ids = [&](int t) {
      const int c0 = (t * Sh::BN + tok) >> shift, c1 = (t * Sh::BN + tok + kApart) >> shift;
      id0 = ids_from[c0 < last_col ? c0 : last_col];
      id1 = ids_from[c1 < last_col ? c1 : last_col];
    };
    TileRaw raw;
    bool bad0, bad1;  // the page is not there
    const int64_t page_stride = a.cache.kv_heads * record;
    const uint8_t* data = a.cache.data + head * record;
    auto record_of = [&](int32_t id, bool* bad) -> const uint8_t* {
      *bad = static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.cache.pages);
      return data + static_cast<int64_t>(*bad ? 0 : id) * page_stride;
    };
    auto load_raw = [&](int t) {
      const int key = t * Sh::BN + tok;
      const uint8_t* rec = record_of(id0, &bad0);
      const uint32_t at = key & in_page;
      const uint8_t* codes = rec + (code_at + at * (D / 2));
      const uint8_t* scales = rec + (scale_at + at * L);
      if (does_v) {
        const u32x2 sc = *reinterpret_cast<const u32x2*>(scales);
        if constexpr (L == 16) {
          const uint32_t* q = reinterpret_cast<const uint32_t*>(codes);
          raw.w0 = u32x4{q[0], q[2], q[4], q[6]};
          raw.w1 = u32x4{q[8], q[10], q[12], q[14]};
        } else {
          raw.w0 = reinterpret_cast<const u32x4*>(codes)[0];
          raw.w1 = reinterpret_cast<const u32x4*>(codes)[1];
        }
        raw.s0 = sc.x;
        raw.s1 = sc.y;
      } else {
        raw.w0 = *reinterpret_cast<const u32x4*>(codes);
        raw.s0 = *reinterpret_cast<const uint16_t*>(scales);
        const int key1 = key + kApart;
        rec = record_of(id1, &bad1);
        const uint32_t at1 = key1 & in_page;
        raw.w1 = *reinterpret_cast<const u32x4*>(rec + (code_at + at1 * (D / 2)));
        raw.s1 = *reinterpret_cast<const uint16_t*>(rec + (scale_at + at1 * L));
      }
    };
    auto put = [&](int buf, int off, half8_t v) {
      *reinterpret_cast<half8_t*>(frags + buf * kBufBytes + put_at + off) = v;
    };
    auto decode_k = [&](int buf, int off, u32x4 w, uint32_t sc) {
      const half2_t pr = scale2<false>(sc);
      const half2_t c0 = {pr[0], pr[0]}, c1 = {pr[1], pr[1]};
      put(buf, off, decode8(w.x, c0));
      put(buf, off + 512, decode8(w.y, c0));
      put(buf, off + kFragBytes, decode8(w.z, c1));
      put(buf, off + kFragBytes + 512, decode8(w.w, c1));
    };
    auto decode = [&](int t, int buf) {
      if (!does_v) {
        // NaN logits where the page is not there
        decode_k(buf, 0, raw.w0, bad0 ? 0x7F7Fu : raw.s0);
        decode_k(buf, kApartBytes, raw.w1, bad1 ? 0x7F7Fu : raw.s1);
        return;
      }
      const int key8 = t * Sh::BN + tok;
      if (bad0 || key8 < keys.lo || key8 + 8 > keys.hi) {
        // keys that no row of the workgroup sees hold anything: scale 0
        uint64_t keep = ~uint64_t{0};
        const int before = keys.lo - key8, after = key8 + 8 - keys.hi;
        if (bad0 || before >= 8 || after >= 8) {
          keep = 0;
        } else {
          if (before > 0) keep &= ~uint64_t{0} << (8 * before);
          if (after > 0) keep &= ~uint64_t{0} >> (8 * after);
        }
        raw.s0 &= static_cast<uint32_t>(keep);
        raw.s1 &= static_cast<uint32_t>(keep >> 32);
      }
      half2_t sc[4];
      v_scales8(u32x2{raw.s0, raw.s1}, sc);
      const u32x4 p = raw.w0, q = raw.w1;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (L == 4) {  // two slices of 4 elements, 2 bytes a token
          w[2 * i] = __builtin_amdgcn_perm(q[i], p[i], 0x05040100u);
          w[2 * i + 1] = __builtin_amdgcn_perm(q[i], p[i], 0x07060302u);
        } else {
          w[i] = p[i];
          w[4 + i] = q[i];
        }
      }
      transpose_nibbles(w);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        put(buf, (j / Sh::JW) * (Sh::BN / 16) * kFragBytes + Sh::VC * (j % Sh::JW) * 16, decode8(w[j], sc));
    };

    // A tile, 64 keys at a time.
    constexpr int SU = NT < 2 ? 1 : 2;
    auto multiply = [&](int t, int buf) {
#pragma unroll 1
      for (int u0 = 0; u0 < NT; u0 += SU) {
        const int key0 = t * Sh::BN + 32 * u0;
        const uint8_t* kp = frags + buf * kBufBytes + lane * 16 + u0 * KS * kFragBytes;
        const uint8_t* vp = frags + buf * kBufBytes + lane * 16 + (Sh::F + 2 * u0) * kFragBytes;
        f32x16 s[SU];
#pragma unroll
        for (int u = 0; u < SU; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int u = 0; u < SU; ++u) {
            const half8_t kf = *reinterpret_cast<const half8_t*>(kp + (u * KS + k) * kFragBytes);
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[x][k], s[u], 0, 0, 0);
          }
        // four operands on their way from LDS ahead of the one that is multiplied
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int k = 0; k < SU * KS - 4; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x008, NQ, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 4 * NQ, 0);
        if (key0 < inner.lo || key0 + 32 * SU > inner.hi) {
          const int lo = see.lo - key0 - 8 * half, hi = see.hi - key0 - 8 * half;
#pragma unroll
          for (int u = 0; u < SU; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int at = 32 * u + 16 * (i / 8) + i % 8;
              if (at < lo || at >= hi) s[u][i] = -INFINITY;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < SU; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[u][i]);
        {
          auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
          top = __builtin_fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1])) * c;
        }
        if (__any(top > m + kRaise)) {
          const float mn = __builtin_fmaxf(m, top);
          const float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
          l *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] *= f;
          m = mn;
        }
        const float shift_m = (m == -INFINITY ? 0.0f : m) - kWeightBits;
#pragma unroll
        for (int u = 0; u < SU; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            half8_t pf[NQ];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][8 * v + i], c, -shift_m));
              l += p;
              const _Float16 h = static_cast<_Float16>(p);
              pf[0][i] = h;
              if (kSplit) pf[NQ - 1][i] = static_cast<_Float16>(p - static_cast<float>(h));
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const half8_t vf =
                  *reinterpret_cast<const half8_t*>(vp + (d * (Sh::BN / 16) + 2 * u + v) * kFragBytes);
#pragma unroll
              for (int x = 0; x < NQ; ++x) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[x], o[d], 0, 0, 0);
            }
          }
      }
    };

    // A tile's bytes are loaded an iteration before they are decoded.  Of a
    // SIMD's two waves one decodes V, first, and multiplies then; the other
    // multiplies first and decodes K then, so that the vector units' work of
    // one lies beside the matrix units' of the other.
    if (t1 > t0) {
      load_ids(t0);
      load_raw(t0);
      load_ids(t0 + 1);
      decode(t0, 0);
      load_raw(t0 + 1);
      load_ids(t0 + 2);
      __syncthreads();
      for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1;
        // past the last tile: not used
        if (does_v) {
          decode(t + 1, buf ^ 1);
          load_raw(t + 2);
          load_ids(t + 3);
        }
        if (wave_live) multiply(t, buf);
        if (!does_v) {
          decode(t + 1, buf ^ 1);
          load_raw(t + 2);
          load_ids(t + 3);
        }
        __syncthreads();
      }
    }

    if (wave_live) {
      auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
      l = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
    }
    if (live) {
      // slot 0: the unit that the range begins with; 1: one that begins in it
      const int64_t slot = (2 * static_cast<int64_t>(range_id) + (first_unit ? 0 : 1)) * Sh::BM + (row - base);
      if (!whole && half == 0) {
        a.part[a.part_ml + 2 * slot] = m;
        a.part[a.part_ml + 2 * slot + 1] = l;
      }
      const OutScale gv = out_scale(a.cache.amax[1]);
      const float f = gv.over(l);
      // element 8 c + j, c = 8 ga + 4 half + b, is in o[j / JW][4 (ga + GA (j % JW)) + b]
#pragma unroll
      for (int ga = 0; ga < Sh::GA; ++ga)
#pragma unroll
        for (int b = 0; b < 4; b += 2) {
          float z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = i % 8;
            z[i] = o[j / Sh::JW][4 * (ga + Sh::GA * (j % Sh::JW)) + b + i / 8];
          }
          const int block = (8 * ga + 4 * half + b) / 2;
          if (!whole)
            store16(a.part + slot * D + block * 16, z);
          else
            write_block(a, rq.row0, head, row, block, z, f, gv.back);
        }
    }
    at += here;
  }
}

// ---------------------------------------------------------------- joining

// What a launch left to join: the partial sums of units of `rows` rows, and the
// units of its workgroups.
struct JoinPart {
  const float* part;
  int64_t part_ml;
  const RangeUnit* units;
  int32_t wgs, rows;
};

// Row `row` of a unit from its `n` partial sums, by one wave: lane b + L s0
// sums block b of parts s0, s0 + 64 / L, ...; the lanes of a block then add up.
// slot(s): the row's place in part s.
template <typename T, int D, typename SLOT>
__device__ __forceinline__ void join_row(const AttnArgs<T>& a, const JoinPart& p, int row0, int head, int row, int n,
                                         SLOT slot) {
  constexpr int L = D / 16, kLanes = 64 / L, kAtOnce = 32 / kLanes;
  const int lane = threadIdx.x & 63, b = lane % L, s0 = lane / L;
  const float2* ml = reinterpret_cast<const float2*>(p.part + p.part_ml);
  // 32 parts at a time, whose loads do not wait for each other nor, the first,
  // for the maximum
  float4 v[kAtOnce][4];
  float2 e[kAtOnce];
  auto fetch = [&](int s) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int64_t at = slot(s + k * kLanes < n ? s + k * kLanes : 0);
      e[k] = ml[at];
      const float4* x = reinterpret_cast<const float4*>(p.part + at * D + b * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k][i] = x[i];
    }
  };
  float mm = lane < n ? ml[slot(lane)].x : -INFINITY;
  fetch(s0);
  for (int s = lane + 64; s < n; s += 64) mm = __builtin_fmaxf(mm, ml[slot(s)].x);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mm = __builtin_fmaxf(mm, __shfl_xor(mm, d));
  float z[16], ll = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  const OutScale gv = out_scale(a.cache.amax[1]);
  for (int s = s0; s < n; s += 32) {
    if (s != s0) fetch(s);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (s + k * kLanes >= n) continue;
      const float f = e[k].x == mm ? 1.0f : __builtin_amdgcn_exp2f(e[k].x - mm);
      ll = __builtin_fmaf(f, e[k].y, ll);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[4 * i] = __builtin_fmaf(f, v[k][i].x, z[4 * i]);
        z[4 * i + 1] = __builtin_fmaf(f, v[k][i].y, z[4 * i + 1]);
        z[4 * i + 2] = __builtin_fmaf(f, v[k][i].z, z[4 * i + 2]);
        z[4 * i + 3] = __builtin_fmaf(f, v[k][i].w, z[4 * i + 3]);
      }
    }
  }
#pragma unroll
  for (int d = L; d < 64; d <<= 1) {
    ll += __shfl_xor(ll, d);
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] += __shfl_xor(z[i], d);
  }
  if (s0 == 0) write_block(a, row0, head, row, b, z, gv.over(ll), gv.back);
}

// Workgroups (w, .) join the unit that workgroup w's range of tiles begins
// inside, if that is the first range to do so; first those of one launch, then
// those of the other.
template <typename T, int D>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(AttnArgs<T> a, JoinPart first, JoinPart second) {
  const bool other = blockIdx.x >= static_cast<uint32_t>(first.wgs);
  const JoinPart p = other ? second : first;
  const int w = static_cast<int>(blockIdx.x) - (other ? first.wgs : 0);
  const RangeUnit u = p.units[w];
  if (u.off == 0 || u.off > u.chunk) return;
  const int count = u.rows - u.base < p.rows ? u.rows - u.base : p.rows;
  // parts: the range before this one's (its slot 0 if the unit begins with
  // it), this one's and those after it
  const int64_t w0 = static_cast<int64_t>(w) - 1;
  const int n = static_cast<int>((u.chunk - u.off + u.tiles - 1) / u.chunk) + 1;
  const int first_slot = u.off == u.chunk ? 0 : 1;
  auto slot = [&](int s, int r) { return (2 * (w0 + s) + (s == 0 ? first_slot : 0)) * p.rows + r; };
  if (n <= 4) {
    // a lane a block of a row, which sums its parts by itself
    constexpr int L = D / 16;
    const OutScale gv = out_scale(a.cache.amax[1]);
    const float2* ml = reinterpret_cast<const float2*>(p.part + p.part_ml);
    for (int i = 256 * blockIdx.y + threadIdx.x; i < count * L; i += 256 * gridDim.y) {
      const int r = i / L, b = i % L;
      float2 e[4];
      float4 v[4][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int64_t at = slot(s < n ? s : 0, r);
        e[s] = ml[at];
        const float4* x = reinterpret_cast<const float4*>(p.part + at * D + b * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[s][k] = x[k];
      }
      float mm = e[0].x;
#pragma unroll
      for (int s = 1; s < 4; ++s) mm = __builtin_fmaxf(mm, e[s].x);
      float z[16], ll = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) z[k] = 0.0f;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s >= n) continue;
        const float f = e[s].x == mm ? 1.0f : __builtin_amdgcn_exp2f(e[s].x - mm);
        ll = __builtin_fmaf(f, e[s].y, ll);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[4 * k] = __builtin_fmaf(f, v[s][k].x, z[4 * k]);
          z[4 * k + 1] = __builtin_fmaf(f, v[s][k].y, z[4 * k + 1]);
          z[4 * k + 2] = __builtin_fmaf(f, v[s][k].z, z[4 * k + 2]);
          z[4 * k + 3] = __builtin_fmaf(f, v[s][k].w, z[4 * k + 3]);
        }
      }
      write_block(a, u.row0, u.head, u.base + r, b, z, gv.over(ll), gv.back);
    }
    return;
  }
  for (int r = 4 * blockIdx.y + (threadIdx.x >> 6); r < count; r += 4 * gridDim.y)
    join_row<T, D>(a, p, u.row0, u.head, u.base + r, n, [&](int s) { return slot(s, r); });
}

}  // namespace
}  // namespace nvfp4rq
