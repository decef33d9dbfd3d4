// libibp_kv: an 8-bit KV page cache and the attention that reads it, for AMD
// Instinct MI355X (gfx950, CDNA4).  Formats and calls: include/ibp_kv.h.
//
// Times below are of one launch by kernel trace unless something else is said;
// rates count the bytes that the operation cannot do without.  A large copy
// reaches 6.1 TB/s on this card.
//
//   append     one wave per 16-token tile that gets tokens: HBM, 5.3 TB/s
//   attention  workgroups of 4 waves over parts of a head's pages, each wave with
//              running statistics of its own, joined in LDS and, where a head
//              has several workgroups, by a second launch: HBM, 5.7-6.3 TB/s on
//              long contexts; vector arithmetic and the two launches on short ones
//   evict      one workgroup per row: vector arithmetic and the phases of a row
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "ibp_kv.h"

namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 16;       // tokens of a tile
// Tiles that a wave takes at a time: 64 tokens of narrow heads, 32 of wider
// ones, whose tiles and accumulators take more registers (64 tokens of 128
// dims measured the same at 40 registers more).
constexpr int step_tiles(int dj, int mt) { return dj * mt <= 1 ? 4 : 2; }
// Workgroups of the attention kernel that a compute unit holds at once: their
// accumulators, queries and tiles on the way fill the registers.
constexpr int workgroups_per_unit(int dj, int mt) { return dj * mt <= 4 ? 2 : 1; }
// The most groups of 16 query rows that a unit takes.  128 dims, 64 query rows, 4
// x 8 heads x 14,000 tokens: 51 us as two units of 32, 59 us as one of 64 (both
// launches); 64 dims: 40 and 43 us; 256 dims, 24 rows: 39 us as one unit, 48 us
// as two of 16.
constexpr int kQueryTiles = 2;
constexpr int kUnit = 1024;     // bytes of a tile that one wide load of a wave takes
constexpr float kGrowth = 8.f;  // log2 of how far exponentials may exceed the scale of the sums
constexpr int kMaxParts = 512;  // workgroups that the chip holds at once, at most
// Query rows of a unit that one thread adds up for its tile.  8 rows of 131k
// tokens: 5.6 us so, 9.4 us with the rows spread over the waves; 64 rows of 14k:
// 13.2 us so, 8.9 us spread.
constexpr int kFewRows = 16;
constexpr int kLdsMass = 4096;  // shares of tiles that a workgroup that works alone keeps in LDS
constexpr int kExpMin = -126, kExpMax = 119;  // exponents of a page's scale
constexpr float kE4m3Max = 448.f;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------- conversions ----

template <bool F16>
__device__ __forceinline__ float to_float(uint16_t x) {
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, x);
  return __builtin_bit_cast(float, (uint32_t)x << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t to_half(float x) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// Eight e4m3 codes as eight 16-bit numbers, which hold them exactly.
template <bool F16>
__device__ __forceinline__ u32x4 widen8(uint32_t lo, uint32_t hi) {
  u32x4 r;
  if constexpr (F16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true));
  }
  return r;
}

template <bool F16>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 p;
  p[0] = (__bf16)a;
  p[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, p);
}

__device__ __forceinline__ float bf16_low(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float bf16_high(uint32_t p) {
  return __builtin_bit_cast(float, p & 0xFFFF0000u);
}

__device__ __forceinline__ bool finite(float x) {
  return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float power2(int e) {
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

// Smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8), in a scale's range.
// Zero and subnormal numbers end at the lowest.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __builtin_bit_cast(uint32_t, amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kExpMin), kExpMax);
}

// Smallest e with scale <= 2^e: the exponent of a page's scale, which an
// append writes as a power of two.
__device__ __forceinline__ int held_exponent(float scale) {
  const uint32_t b = __builtin_bit_cast(uint32_t, scale);
  const int e = (int)((b >> 23) & 255) - 127 + ((b & 0x7FFFFFu) ? 1 : 0);
  return min(max(e, kExpMin), kExpMax);
}

// The number to convert for x / 2^e: saturated, and NaN for what is not finite.
__device__ __forceinline__ float code_value(float x, float inv) {
  const float y = fminf(fmaxf(x * inv, -kE4m3Max), kE4m3Max);
  return finite(x) ? y : __builtin_bit_cast(float, 0x7FC00000u);
}

// The top bits of the bytes of `c` that are one of the two NaN codes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t c) {
  return ~(((c & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & 0x80808080u;
}

// Rounded to nearest, ties to even; NaN becomes 0x7F whatever its sign (which
// the compiler may choose for a NaN constant).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r & ~nan_codes((uint32_t)r);
}

// Four codes of scale `was` at another scale: ratio = was / now, at most 1.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  return codes4(code_value(a[0], ratio), code_value(a[1], ratio), code_value(b[0], ratio),
                code_value(b[1], ratio));
}

__device__ __forceinline__ uint32_t byte_mask(int n) {  // the first n bytes of four
  return n <= 0 ? 0u : n >= 4 ? ~0u : (1u << (8 * n)) - 1u;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// ---------------------------------------------------------------- waves ----

template <int CTRL>
__device__ __forceinline__ float row_rotate(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}

// The two values that lanes l and l ^ 16 (l ^ 32) hold, the same in both.
__device__ __forceinline__ f32x2 both16(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return f32x2{__builtin_bit_cast(float, (uint32_t)y[0]), __builtin_bit_cast(float, (uint32_t)y[1])};
}
__device__ __forceinline__ f32x2 both32(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return f32x2{__builtin_bit_cast(float, (uint32_t)y[0]), __builtin_bit_cast(float, (uint32_t)y[1])};
}

// Maximum and sum over the wave, in every lane: rotations within 16 lanes, then
// swaps of rows.
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, row_rotate<0x121>(x));
  x = fmaxf(x, row_rotate<0x122>(x));
  x = fmaxf(x, row_rotate<0x124>(x));
  x = fmaxf(x, row_rotate<0x128>(x));
  f32x2 y = both16(x);
  y = both32(fmaxf(y[0], y[1]));
  return fmaxf(y[0], y[1]);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x121, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x122, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x124, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xF, 0xF, false));
  const auto y = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max((uint32_t)y[0], (uint32_t)y[1]);
  const auto z = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max((uint32_t)z[0], (uint32_t)z[1]);
}

__device__ __forceinline__ float wave_sum(float x) {
  x += row_rotate<0x121>(x);
  x += row_rotate<0x122>(x);
  x += row_rotate<0x124>(x);
  x += row_rotate<0x128>(x);
  f32x2 y = both16(x);
  y = both32(y[0] + y[1]);
  return y[0] + y[1];
}

// n plus the bits of `mask` that belong to lower lanes.
__device__ __forceinline__ uint32_t lanes_below(uint64_t mask, uint32_t n) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, n));
}

// Sum over the lanes up to this one: shifts within 16 lanes, then the last lane
// of a row to the rows after it.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false);
  return x;
}

// ---------------------------------------------------------------- rows ----

struct Pool {
  uint8_t* k_codes;
  float* k_scales;
  uint8_t* v_codes;
  float* v_scales;
  uint32_t n_pages;     // ids at or past this are holes
  uint32_t page_bytes;  // of the keys, and of the values
  uint32_t tile_shift;  // log2 of a page's tiles
};

// Division of numbers below 2^31 by one that the host knows: with 2^l >= d the
// multiplier ceil(2^(31 + l) / d) is off by less than 2^l / d, too little to
// show.  (A division by a number in a register takes some 30 instructions.)
struct Divisor {
  uint32_t d, mul, shift;
};

__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor& x) {
  return (uint32_t)(((uint64_t)n * x.mul) >> x.shift);
}

struct Rows {
  const int32_t* pages;
  const int32_t* lengths;
  const int32_t* counts;
  Divisor heads;
  uint32_t max_pages;
  int32_t capacity;  // tokens
  int32_t n_new;
};

struct Strided {
  uint16_t* data;
  int64_t seq, token, head;
  uint32_t wide;  // 16-byte accesses are aligned
};

__device__ __forceinline__ int row_length(const Rows& r, uint32_t row) {
  return min(max(r.lengths[row], 0), r.capacity);
}

__device__ __forceinline__ int new_count(const Rows& r, uint32_t seq) {
  return r.counts ? min(max(r.counts[seq], 0), r.n_new) : r.n_new;
}

// -------------------------------------------------------------- append ----

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x4 load8(const uint16_t* p, bool wide) {
  if (wide) return *(const u32x4*)p;
  u16x8 h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = p[i];
  return __builtin_bit_cast(u32x4, h);
}

// Largest magnitude of the 16-bit numbers so far, in each half: as whole
// numbers, which order magnitudes, infinity and NaN at the top.
__device__ __forceinline__ uint32_t magnitude_max(uint32_t m, uint32_t x) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                __builtin_bit_cast(u16x2, x & 0x7FFF7FFFu)));
}

template <bool F16>
__device__ __forceinline__ bool not_finite(uint32_t half) {
  return (half & 0x7FFFu) >= (F16 ? 0x7C00u : 0x7F80u);
}

// The lane's largest finite magnitude: 0 in place of what is not finite.
template <bool F16>
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t x) {
  if (not_finite<F16>(x)) x &= 0xFFFF0000u;
  if (not_finite<F16>(x >> 16)) x &= 0xFFFFu;
  return magnitude_max(m, x);
}

// Codes of the pairs a and b at the scale 2^e.  `plain`: all are finite and
// within the scale, which the conversion of pairs then does as it is (it
// rounds to nearest, ties to even).
template <bool F16>
__device__ __forceinline__ uint32_t codes_of(uint32_t a, uint32_t b, bool plain, float scale, float inv) {
  if (plain) {
    i16x2 r = {0, 0};
    if constexpr (F16) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2, a), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2, b), scale, true);
    } else {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, a), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, b), scale, true);
    }
    return __builtin_bit_cast(uint32_t, r);
  }
  return codes4(code_value(to_float<F16>((uint16_t)a), inv), code_value(to_float<F16>((uint16_t)(a >> 16)), inv),
                code_value(to_float<F16>((uint16_t)b), inv), code_value(to_float<F16>((uint16_t)(b >> 16)), inv));
}

// One wave per 16-token tile of a page that receives new tokens; the waves of
// a page exchange their largest value through LDS.  A lane's 16 bytes of a
// key unit are 16 dims of one token, so keys go straight from the loads to
// the store.  A lane's 16 bytes of a value unit are 4 tokens x 4 dims: the
// lane that loads 8 dims of 4 tokens writes 8 words of 4 codes to LDS, from
// which units are read back.  Bound by HBM: 4 prompts of 4096 tokens x 32 heads
// x 128 dims (403 MB moved) take 75 us, 5.3 TB/s; with plain stores 78 us, with
// non-temporal loads as well 76 us.
template <int DJ, bool F16>
__global__ __launch_bounds__(kThreads) void append_kernel(Pool pool, Rows rows, Strided k,
                                                          Strided v, Divisor pages_per_row,
                                                          uint32_t n_tasks) {
  constexpr int D = 64 * DJ;
  constexpr int kOctets = D / 8;
  constexpr int kPasses = (kOctets * 4 + kWave - 1) / kWave;
  __shared__ uint32_t s_tile[kWaves][4 * D];
  __shared__ float s_max[2][kWaves];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int tiles = 1 << pool.tile_shift;
  const uint32_t task = blockIdx.x * (kWaves >> pool.tile_shift) + (wave >> pool.tile_shift);
  const int tile = wave & (tiles - 1);
  // heads first: what neighbouring workgroups read lies together in [seq][token][head]
  const uint32_t line = quotient(min(task, n_tasks - 1), rows.heads);
  const uint32_t head = min(task, n_tasks - 1) - line * rows.heads.d;
  const uint32_t seq = quotient(line, pages_per_row), row = seq * rows.heads.d + head;
  const int end = row_length(rows, row), count = new_count(rows, seq);
  const int first = max(end - count, 0);      // position of the first new token that exists
  const int origin = end - count;             // position of token 0
  const int page_shift = 4 + (int)pool.tile_shift;
  const int page = (first >> page_shift) + (int)(line - seq * pages_per_row.d);
  const int page_at = page << page_shift, at = page_at + tile * kTile;
  const bool reached = task < n_tasks && count > 0 && page < (int)rows.max_pages && page_at < end;
  int32_t id = -1;
  if (reached) id = rows.pages[(uint64_t)row * rows.max_pages + page];

  // keys: token at + lane % 16, dims 64 j + 16 (lane / 16) + 0..15
  u32x4 kx[DJ][2], vx[kPasses][4];
  const int kt = at + lane % 16, kg = lane / 16;
#pragma unroll
  for (int j = 0; j < DJ; ++j) kx[j][0] = kx[j][1] = u32x4{0, 0, 0, 0};
  if (reached && kt >= first && kt < end) {
    const uint16_t* p = k.data + seq * k.seq + (int64_t)(kt - origin) * k.token + head * k.head + 16 * kg;
#pragma unroll
    for (int j = 0; j < DJ; ++j) {
      kx[j][0] = load8(p + 64 * j, k.wide);
      kx[j][1] = load8(p + 64 * j + 8, k.wide);
    }
  }
  // values: octet `item % kOctets` of dims, tokens at + 4 (item / kOctets) + 0..3
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int item = p * kWave + lane;
    const int g = item / kOctets, o = item % kOctets;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = at + 4 * g + r;
      vx[p][r] = u32x4{0, 0, 0, 0};
      if (reached && g < 4 && t >= first && t < end)
        vx[p][r] = load8(v.data + seq * v.seq + (int64_t)(t - origin) * v.token + head * v.head + 8 * o, v.wide);
    }
  }
  const bool live = (uint32_t)id < pool.n_pages;
  uint32_t km = 0, vm = 0;
#pragma unroll
  for (int j = 0; j < DJ; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) km = magnitude_max(km, kx[j][i / 4][i % 4]);
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int i = 0; i < 16; ++i) vm = magnitude_max(vm, vx[p][i / 4][i % 4]);
  const bool k_odd = __ballot(not_finite<F16>(km) || not_finite<F16>(km >> 16)) != 0;
  const bool v_odd = __ballot(not_finite<F16>(vm) || not_finite<F16>(vm >> 16)) != 0;
  if (k_odd) {
    km = 0;
#pragma unroll
    for (int j = 0; j < DJ; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) km = finite_max<F16>(km, kx[j][i / 4][i % 4]);
  }
  if (v_odd) {
    vm = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
#pragma unroll
      for (int i = 0; i < 16; ++i) vm = finite_max<F16>(vm, vx[p][i / 4][i % 4]);
  }
  float k_max = wave_max(to_float<F16>((uint16_t)max(km & 0xFFFFu, km >> 16)));
  float v_max = wave_max(to_float<F16>((uint16_t)max(vm & 0xFFFFu, vm >> 16)));
  // a page that held tokens keeps a larger scale
  const bool held = live && page_at < first;
  float k_was = 0.f, v_was = 0.f;
  if (held) {
    k_was = pool.k_scales[id];
    v_was = pool.v_scales[id];
  }
  if (tiles > 1) {  // read by all waves of the page before one of them writes
    if (lane == 0) {
      s_max[0][wave] = k_max;
      s_max[1][wave] = v_max;
    }
    __syncthreads();
    for (int w = wave & ~(tiles - 1), n = 0; n < tiles; ++n) {
      k_max = fmaxf(k_max, s_max[0][w + n]);
      v_max = fmaxf(v_max, s_max[1][w + n]);
    }
  }
  if (!live) return;
  int ke = scale_exponent(k_max), ve = scale_exponent(v_max);
  if (held) {
    ke = max(ke, held_exponent(k_was));
    ve = max(ve, held_exponent(v_was));
  }
  ke = uniform(ke);
  ve = uniform(ve);
  const float k_scale = power2(ke), v_scale = power2(ve);
  const float k_inv = power2(-ke), v_inv = power2(-ve);
  const float k_ratio = k_was * k_inv, v_ratio = v_was * v_inv;
  const bool k_plain = !k_odd && ke > kExpMin && ke < kExpMax, v_plain = !v_odd && ve > kExpMin && ve < kExpMax;
  if (tile == 0 && lane == 0) {
    pool.k_scales[id] = k_scale;
    pool.v_scales[id] = v_scale;
  }
  const uint64_t base = (uint64_t)(uint32_t)id * pool.page_bytes + (uint32_t)(tile * kTile * D);
  uint8_t* kp = pool.k_codes + base + lane * 16;
  uint8_t* vp = pool.v_codes + base + lane * 16;

  const bool k_old = kt < first;
#pragma unroll
  for (int j = 0; j < DJ; ++j) {
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = codes_of<F16>(kx[j][i / 2][i % 2 * 2], kx[j][i / 2][i % 2 * 2 + 1], k_plain, k_scale, k_inv);
    if (k_old) {
      c = *(const u32x4*)(kp + j * kUnit);
      if (k_ratio != 1.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = rescale4(c[i], k_ratio);
      }
    }
    __builtin_nontemporal_store(c, (u32x4*)(kp + j * kUnit));
  }

  uint32_t* tile_words = s_tile[wave];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int item = p * kWave + lane;
    const int g = item / kOctets, o = item % kOctets;
    if (g < 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // dims d and d + 1 of tokens 0, 1 and of tokens 2, 3
        const uint32_t a = codes_of<F16>(vx[p][0][i], vx[p][1][i], v_plain, v_scale, v_inv);
        const uint32_t b = codes_of<F16>(vx[p][2][i], vx[p][3][i], v_plain, v_scale, v_inv);
        const int d = 8 * o + 2 * i;
        uint32_t* word = tile_words + (d / 64) * 256 + g * 64 + (d % 16) * 4 + d % 64 / 16;
        word[0] = __builtin_amdgcn_perm(b, a, 0x06040200u);
        word[4] = __builtin_amdgcn_perm(b, a, 0x07050301u);
      }
    }
  }
  // the wave's own words only: LDS operations of a wave stay in order
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const uint32_t old = byte_mask(first - (at + 4 * kg));
#pragma unroll
  for (int j = 0; j < DJ; ++j) {
    u32x4 c = *(const u32x4*)(tile_words + j * 256 + lane * 4);
    if (old) {
      const u32x4 was = *(const u32x4*)(vp + j * kUnit);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = v_ratio != 1.f ? rescale4(was[i], v_ratio) : was[i];
        c[i] = (c[i] & ~old) | (w & old);
      }
    }
    __builtin_nontemporal_store(c, (u32x4*)(vp + j * kUnit));
  }
}

// ----------------------------------------------------------- attention ----

struct Attention {
  Pool pool;
  Rows rows;
  Strided q, out;
  const float* w_in;
  float* w_out;
  float* ws_o;     // [part][unit_rows][D] sums of p v
  f32x2* ws_ml;    // [part][unit_rows] maximum and sum
  float* ws_mass;  // [unit][unit_rows][cap_tiles] log2 of a tile's share of exp2(s)
  int32_t* ws_of;  // [unit][2] first part and number of parts, of units that have a token
  float scale;     // scale * log2(e)
  Divisor group;
  Divisor m_groups;    // units a head's query rows are cut into
  Divisor unit_rows;   // query rows of a unit
  int32_t m_rows;      // group * n_new: query rows of a key/value head
  int32_t cap_tiles;
  uint32_t wave_rows;    // the joining kernel has a query row for each wave
  uint32_t mass_in_lds;  // the unit's shares fit kLdsMass, and no other workgroup needs them
  uint32_t n_units;
  uint32_t n_rows;
  uint32_t n_parts;  // workgroups that the units are spread over; n_units: one each
  Divisor weight_blocks;  // of a row, in the joining kernel
};

// Which part of which unit a workgroup takes.
struct Part {
  uint32_t row;
  int len;         // tokens of the row
  int group;       // of the head's query rows
  int index, of;   // the unit is cut into `of` parts
  uint32_t first;  // part 0 of the unit; the next ones are m_groups apart
  uint32_t slot;   // this part
  bool idle;
};

// A unit (some query rows of a head) reads the tiles up to what its last query
// sees, in steps.
struct Plan {
  uint32_t row, seq, head;
  int m0;      // first query row
  int origin;  // position of new token 0
  int count;
  int end;     // tokens that some query sees
  int full;    // tokens that every query with any sees
  int tiles, steps;
  int part_steps, parts;
};

constexpr int kRowsPerLane = 6;  // of the rows that share out the workgroups

// Shares the workgroups out: with C = ceil(all steps / (n_parts - n_units)) a
// row of s steps gets ceil(s / C) workgroups for each of its units, n_parts at
// most together.  Long rows get more than short ones, so that no workgroup
// works long after the others.  Every wave works it out from the lengths.
//   lane l: rows 6 l .. 6 l + 5, `share` workgroups a unit each, `before` those
//   of the rows before them.
template <int ST>
__device__ __forceinline__ void share_out(const Attention& a, int lane, int (&len)[kRowsPerLane],
                                          int (&share)[kRowsPerLane], int& before) {
  int total = 0;
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    const uint32_t row = lane * kRowsPerLane + i;
    len[i] = row < a.n_rows ? row_length(a.rows, row) : 0;
    share[i] = (int)(((uint32_t)len[i] + kTile * ST - 1) / (kTile * ST));
    total += share[i];
  }
  const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)wave_scan((uint32_t)total), kWave - 1) *
                       a.m_groups.d;
  const uint32_t room = a.n_parts - a.n_units;
  const uint32_t c = max((all + room - 1) / room, (uint32_t)kWaves);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    share[i] = (int)(((uint32_t)share[i] + c - 1) / c);
    mine += share[i];
  }
  before = (int)wave_scan((uint32_t)mine) - mine;
}

// Workgroups go to the 8 XCDs in turn, each with an L2 of its own: the units of a
// head that read the same tiles are 8 workgroups apart.
constexpr uint32_t kXcds = 8;

template <int ST>
__device__ __forceinline__ Part part_of_workgroup(const Attention& a, uint32_t w, int lane) {
  Part t;
  uint32_t x = w;
  t.group = 0;
  if (a.m_groups.d > 1) {
    const uint32_t n = a.n_parts / a.m_groups.d, even = n / kXcds * kXcds;
    if (w < even * a.m_groups.d) {
      const uint32_t turn = w / kXcds, y = quotient(turn, a.m_groups);
      t.group = (int)(turn - y * a.m_groups.d);
      x = y * kXcds + w % kXcds;
    } else {
      const uint32_t rest = w - even * a.m_groups.d, y = quotient(rest, a.m_groups);
      t.group = (int)(rest - y * a.m_groups.d);
      x = even + y;
    }
  }
  t.slot = x * a.m_groups.d + t.group;
  if (a.n_parts == a.n_units) {
    t.row = x;
    t.len = row_length(a.rows, x);
    t.index = 0;
    t.of = 1;
    t.first = t.slot;
    t.idle = false;
    return t;
  }
  int lens[kRowsPerLane], share[kRowsPerLane], before;
  share_out<ST>(a, lane, lens, share, before);
  int row = 0, len = 0, index = 0, of = 0, first = 0;
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    if ((int)x >= before && (int)x < before + share[i]) {
      row = lane * kRowsPerLane + i;
      len = lens[i];
      index = (int)x - before;
      of = share[i];
      first = before;
    }
    before += share[i];
  }
  const uint64_t who = __ballot(of != 0);
  t.idle = who == 0;
  const int src = t.idle ? 0 : __builtin_ctzll(who);
  t.row = (uint32_t)__builtin_amdgcn_readlane(row, src);
  t.len = __builtin_amdgcn_readlane(len, src);
  t.index = __builtin_amdgcn_readlane(index, src);
  t.of = __builtin_amdgcn_readlane(of, src);
  t.first = (uint32_t)__builtin_amdgcn_readlane(first, src) * a.m_groups.d + t.group;
  return t;
}

// The parts of a unit, as its part 0 left them (a row without a token has none,
// and what is read for it is not used).
__device__ __forceinline__ Part parts_of_unit(const Attention& a, uint32_t row, int group) {
  Part t;
  t.row = row;
  t.group = group;
  t.index = 0;
  t.idle = false;
  const uint32_t unit = row * a.m_groups.d + group;
  t.len = row_length(a.rows, row);
  t.first = unit;
  t.of = 1;
  if (a.n_parts != a.n_units) {
    const int first = a.ws_of[2 * unit], of = a.ws_of[2 * unit + 1];
    t.first = t.len > 0 ? (uint32_t)first : 0u;
    t.of = t.len > 0 ? of : 1;
  }
  return t;
}

template <int MT, int ST>
__device__ __forceinline__ Plan plan_unit(const Attention& a, const Part& t) {
  Plan p;
  p.row = t.row;
  p.seq = quotient(p.row, a.rows.heads);
  p.head = p.row - p.seq * a.rows.heads.d;
  p.m0 = t.group * (MT * 16);
  p.count = new_count(a.rows, p.seq);
  p.origin = t.len - p.count;
  const int t_low = (int)quotient(p.m0, a.group);
  const int t_high = min((int)quotient(min(p.m0 + MT * 16, a.m_rows) - 1, a.group), p.count - 1);
  p.end = t_high >= t_low ? max(p.origin + t_high + 1, 0) : 0;
  p.full = max(p.origin + t_low + 1, 1);
  p.tiles = (p.end + kTile - 1) / kTile;
  p.steps = (p.tiles + ST - 1) / ST;
  p.part_steps = t.of > 1 ? (p.steps + t.of - 1) / t.of : max(p.steps, 1);
  p.parts = p.steps ? (p.steps + p.part_steps - 1) / p.part_steps : 0;
  return p;
}

// Tokens of the row that query row m sees; 0: none, or no such row.
__device__ __forceinline__ int seen_by(const Attention& a, const Plan& p, int m) {
  const int t = (int)quotient(m, a.group);
  return m < a.m_rows && t < p.count ? max(p.origin + t + 1, 0) : 0;
}

__device__ __forceinline__ uint16_t* row_of(const Strided& x, const Attention& a, const Plan& p, int m) {
  const int t = (int)quotient(m, a.group);
  return x.data + p.seq * x.seq + (int64_t)t * x.token +
         ((int64_t)p.head * a.group.d + (m - t * (int)a.group.d)) * x.head;
}

template <int DJ, int MT>
struct State {
  f32x4 o[MT][4 * DJ];  // o[h * 4 + c][r]: dim 64 h + 16 c + 4 (lane / 16) + r of query lane % 16
  float m[MT];          // about the maximum so far (log2) of query lane % 16: what its sums are scaled by
  float l[MT];          // the lane's part of the running sum
};

// Read-only data at an address that is the same for the whole wave: scalar
// loads, which the compiler does not choose by itself next to stores.
template <class T>
__device__ __forceinline__ T scalar(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

// The page ids of a step's tiles; of tiles past the row's end the last one's.
template <int ST>
struct Ids {
  uint32_t id[ST];
};

template <int ST>
__device__ __forceinline__ Ids<ST> ids_of_step(const Attention& a, const Plan& p, int step) {
  const int32_t* pages = a.rows.pages + (uint64_t)p.row * a.rows.max_pages;
  Ids<ST> x;
#pragma unroll
  for (int t = 0; t < ST; ++t)
    x.id[t] = (uint32_t)scalar(pages + (min(step * ST + t, p.tiles - 1) >> a.pool.tile_shift));
  return x;
}

// Where a step's tiles are.  Tiles that are holes or past the row's end have `ok`
// unset and the place of a page that can be read all the same.
template <int ST>
struct Where {
  uint64_t at[ST];  // byte of the tile in the pool
  float ks[ST], vs[ST];
  bool ok[ST];
};

template <int DJ, int ST>
__device__ __forceinline__ Where<ST> find_step(const Attention& a, const Plan& p, int step,
                                               const Ids<ST>& ids) {
  Where<ST> w;
#pragma unroll
  for (int t = 0; t < ST; ++t) {
    const int tile = step * ST + t, there = min(tile, p.tiles - 1);
    const bool in = ids.id[t] < a.pool.n_pages;
    w.ok[t] = in && tile < p.tiles;
    const uint32_t page = in ? ids.id[t] : 0u;
    w.at[t] = (uint64_t)page * a.pool.page_bytes +
              (uint32_t)((there & ((1 << a.pool.tile_shift) - 1)) * (DJ * kUnit));
    w.ks[t] = scalar(a.pool.k_scales + page);
    w.vs[t] = scalar(a.pool.v_scales + page);
  }
  return w;
}

// Scalar loads return in no order, so that a wait for one is a wait for all.
// This makes it here, for what was asked for a step ago, before more is.
template <int ST>
__device__ __forceinline__ void arrive(const Where<ST>& w, const Ids<ST>& ids) {
#pragma unroll
  for (int t = 0; t < ST; ++t) asm volatile("" ::"s"(w.ks[t]), "s"(w.vs[t]), "s"(ids.id[t]));
  __builtin_amdgcn_sched_barrier(0);
}

// Non-temporal where a unit has all of its head's query rows, so that no other
// workgroup of the call comes back for the tiles: 16 x 32 heads x 4096 tokens
// take 85.6 us so (6.3 TB/s), 95.8 us with plain loads.  (By a template: of two
// branches with one kind each the compiler makes plain loads.)
template <int DJ, int ST, bool ONCE>
__device__ __forceinline__ void load_tiles(const uint8_t* codes, const Where<ST>& w, int byte,
                                           u32x4 (&x)[ST][DJ]) {
#pragma unroll
  for (int t = 0; t < ST; ++t)
#pragma unroll
    for (int j = 0; j < DJ; ++j) {
      const u32x4* p = (const u32x4*)(codes + w.at[t] + j * kUnit + byte);
      if constexpr (ONCE)
        x[t][j] = __builtin_nontemporal_load(p);
      else
        x[t][j] = *p;
    }
}

// The largest of the four lanes that hold a query.
__device__ __forceinline__ float query_max(float x) {
  f32x2 y = both16(x);
  y = both32(fmaxf(y[0], y[1]));
  return fmaxf(y[0], y[1]);
}

// Sums over lanes l, l ^ 16 of x (for even lane / 16) and of y (for odd).
__device__ __forceinline__ float pair_sum16(float x, float y) {
  const auto z = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, y), false, false);
  return __builtin_bit_cast(float, (uint32_t)z[0]) + __builtin_bit_cast(float, (uint32_t)z[1]);
}

// Sums over lanes l, l ^ 32 of x (for the lower half) and of y (for the upper).
__device__ __forceinline__ float pair_sum32(float x, float y) {
  const auto z = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, y), false, false);
  return __builtin_bit_cast(float, (uint32_t)z[0]) + __builtin_bit_cast(float, (uint32_t)z[1]);
}

// A step of a wave is 16 ST tokens against its 16 MT query rows.
//   S^T = K Q^T: the lane gets the scores of query lane % 16 with tokens
//   4 (lane / 16) + r of each tile.  These are, without any exchange, the
//   P^T operand of O^T = V^T P^T when the matrix instruction's index k is
//   taken as (tile of the pair, r) within lane / 16, and the layout of a value
//   tile gives V^T in the same order.
//   e4m3 codes are exact in both 16-bit types; the keys' scale comes in with the
//   scores, the values' with the weights.
template <int DJ, bool F16, int MT, int ST>
__device__ __forceinline__ void scores(const u32x4 (&k)[ST][DJ], const u32x4 (&q)[MT][DJ][2],
                                       f32x4 (&s)[MT][ST]) {
#pragma unroll
  for (int t = 0; t < ST; ++t) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) s[mt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DJ; ++j)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const u32x4 kk = widen8<F16>(k[t][j][2 * half], k[t][j][2 * half + 1]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[mt][t] = mfma<F16>(kk, q[mt][j][half], s[mt][t]);
      }
  }
}

// P times the page's scale goes into the second product as two 16-bit terms
// (bf16, so that any scale fits): the products keep 16 bits of P, where one term
// would round P to 8 and be the largest error of an fp16 output.  The second
// product is twice as long for it, which the loads hide.
template <int MT, int ST>
struct Probs {
  u32x4 hi[MT][ST / 2], lo[MT][ST / 2];
};

// Takes out of a step what its queries may not see: scores become minus
// infinity, value bytes that no query sees (they may hold anything) 0.  A NaN
// value that only some of the queries see is 0 to the products, and those that
// see it get NaN here; so do values of a scale that is not finite, which would
// make a NaN of an unseen token's weight of 0.
template <int DJ, int MT, int ST>
__device__ __forceinline__ void mask_step(const Plan& p, int step, int lane, const int (&seen)[MT],
                                          Where<ST>& w, f32x4 (&s)[MT][ST], u32x4 (&v)[ST][DJ],
                                          State<DJ, MT>& st) {
  const int at = step * (kTile * ST) + 4 * (lane / 16);  // the lane's first token
#pragma unroll
  for (int t = 0; t < ST; ++t) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!w.ok[t] || at + 16 * t + r >= seen[mt]) s[mt][t][r] = -INFINITY;
    const uint32_t odd = finite(w.vs[t]) ? 0u : 0x7F7F7F7Fu;  // NaN's code
    if (!w.ok[t] || odd) w.vs[t] = 0.f;
    const uint32_t inside = w.ok[t] ? byte_mask(p.end - (at + 16 * t)) : 0u;
    uint32_t any = 0;
#pragma unroll
    for (int h = 0; h < DJ; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[t][h][c] = (v[t][h][c] | odd) & inside;
        any |= nan_codes(v[t][h][c]);
      }
    if (__ballot(any != 0)) {
#pragma unroll
      for (int h = 0; h < DJ; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t nan = (nan_codes(v[t][h][c]) >> 7) * 255u;
          v[t][h][c] &= ~nan;
          const u32x4 is = widen8<false>(nan & 0x38383838u, 0u);  // 1 where NaN
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int n = seen[mt] - (at + 16 * t);
            const u32x4 sees = {n <= 0 ? 0u : n == 1 ? 0x3F80u : 0x3F803F80u,
                                n <= 2 ? 0u : n == 3 ? 0x3F80u : 0x3F803F80u, 0u, 0u};
            const f32x4 found = mfma<false>(is, sees, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (found[r] > 0.f) st.o[mt][h * 4 + c][r] = NAN;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int DJ, int MT, int ST>
__device__ __forceinline__ void softmax(const Attention& a, const Plan& p, int step, int lane,
                                        const Where<ST>& w, f32x4 (&s)[MT][ST], float* mass_row,
                                        float* mass_lds, State<DJ, MT>& st, Probs<MT, ST>& out) {
  const int g = lane / 16;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, s[mt][t][r]);
    // Exponentials may grow to 2^kGrowth before the sums are brought to a new
    // maximum: with 16 queries to a wave one of them has a new one at most steps.
    if (__ballot(top > st.m[mt] + kGrowth)) {
      const float m = fmaxf(st.m[mt], query_max(top));
      const float keep = exp2_fast(st.m[mt] - (m == -INFINITY ? 0.f : m));
      st.m[mt] = m;
      st.l[mt] *= keep;
#pragma unroll
      for (int i = 0; i < 4 * DJ; ++i) st.o[mt][i] *= keep;
    }
    const float base = st.m[mt] == -INFINITY ? 0.f : st.m[mt];
    float mass[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t) {
      float y[4], z[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[r] = exp2_fast(s[mt][t][r] - base);
        z[r] = y[r] * w.vs[t];
      }
      mass[t] = (y[0] + y[1]) + (y[2] + y[3]);
      const uint32_t h0 = pack_bf16(z[0], z[1]), h1 = pack_bf16(z[2], z[3]);
      out.hi[mt][t / 2][t % 2 * 2] = h0;
      out.hi[mt][t / 2][t % 2 * 2 + 1] = h1;
      out.lo[mt][t / 2][t % 2 * 2] = pack_bf16(z[0] - bf16_low(h0), z[1] - bf16_high(h0));
      out.lo[mt][t / 2][t % 2 * 2 + 1] = pack_bf16(z[2] - bf16_low(h1), z[3] - bf16_high(h1));
    }
    // lane / 16 = t gets the sum of tile t (with two tiles, of tile t % 2)
    float mine = pair_sum16(mass[0], mass[1]);
    if constexpr (ST == 4)
      mine = pair_sum32(mine, pair_sum16(mass[2], mass[3]));
    else
      mine = pair_sum32(mine, mine);
    const bool sole = ST == 4 || g < ST;
    if (sole) st.l[mt] += mine;
    if (a.w_out) {
      const int tile = step * ST + g, m_local = mt * 16 + lane % 16;
      if (sole && tile < p.tiles && m_local < (int)a.unit_rows.d) {
        const float share = base + log2_fast(mine);
        if (a.mass_in_lds)
          mass_lds[m_local * a.cap_tiles + tile] = share;
        else
          mass_row[(uint64_t)m_local * a.cap_tiles + tile] = share;
      }
    }
  }
}

template <int DJ, int MT, int ST>
__device__ __forceinline__ void gather_values(const u32x4 (&v)[ST][DJ], const Probs<MT, ST>& pr,
                                              State<DJ, MT>& st) {
#pragma unroll
  for (int pair = 0; pair < ST / 2; ++pair)
#pragma unroll
    for (int h = 0; h < DJ; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const u32x4 vv = widen8<false>(v[2 * pair][h][c], v[2 * pair + 1][h][c]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          st.o[mt][h * 4 + c] = mfma<false>(vv, pr.hi[mt][pair], st.o[mt][h * 4 + c]);
          st.o[mt][h * 4 + c] = mfma<false>(vv, pr.lo[mt][pair], st.o[mt][h * 4 + c]);
        }
      }
}

// log2 of the sum of exp2 over a row's tokens; +inf where there is none, so
// that every share comes out as 0.
__device__ __forceinline__ float log_total(float m, float l) {
  return l == 0.f ? INFINITY : (m == -INFINITY ? 0.f : m) + log2_fast(l);
}

// The shares that tile `tile` got from eight query rows of a unit (m, m + stride,
// ...), and their sum as weights: lse is the rows' log_total (+inf for rows that
// see nothing, whose shares are not written).
struct Shares {
  float x[8];
};

__device__ __forceinline__ Shares load_shares(const Attention& a, const float* mass, int m, int stride,
                                              int tile) {
  Shares s;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    s.x[i] = m + i * stride < (int)a.unit_rows.d ? mass[(uint64_t)(m + i * stride) * a.cap_tiles + tile] : 0.f;
  return s;
}

__device__ __forceinline__ float sum_shares(const Attention& a, const Shares& s, const float* lse, int m,
                                            int stride) {
  float w = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = m + i * stride;
    if (row < (int)a.unit_rows.d) w += lse[row] == INFINITY ? 0.f : exp2_fast(s.x[i] - lse[row]);
  }
  return w;
}

// Adds up the tiles of a page, which neighbouring lanes hold, and writes it.
__device__ __forceinline__ void write_weight(const Attention& a, uint32_t row, int tile, float w) {
  const int shift = (int)a.pool.tile_shift;
  if (shift >= 1) w += __shfl_xor(w, 1);
  if (shift == 2) w += __shfl_xor(w, 2);
  if (tile >= a.cap_tiles || (tile & ((1 << shift) - 1))) return;
  const uint64_t at = (uint64_t)row * a.rows.max_pages + (uint32_t)(tile >> shift);
  a.w_out[at] = a.w_in[at] + w;
}

// A workgroup takes one part of one unit; its waves take steps in turn, with
// running maximum and sum, and join at the end.  With one part a unit the result
// is written here, else it is left in the workspace for the joining kernel, and so
// is what weights need where a row has several units or parts.  ONCE: the unit has
// all query rows of its head.
//
// Everything of a step stays in the wave's registers: the tiles' layouts give the
// operands of the matrix instructions as they are loaded, and scores become
// weights in place.  What it reads once bounds it: 16 x 32 heads x 4096 tokens of
// 128 dims 85.4 us, 6.3 TB/s; two contexts of 131k and 91k tokens, 8 heads, 8
// queries each, 80.7 us, 5.7 TB/s.  Short rows pay some 6 us for finding their
// pages, the joining and the launch (291 tokens: 7.2 us); 72 ragged rows with 25
// queries of 64 dims, 43 MB, take 16.4 us: vector instructions for half of the
// cycles, a third in the steps (250 a step), a sixth before and after; matrix
// instructions for 13%.
template <int DJ, bool F16, int MT, bool ONCE>
__global__ __launch_bounds__(kThreads, workgroups_per_unit(DJ, MT)) void attention_kernel(Attention a) {
  constexpr int D = 64 * DJ;
  constexpr int ST = step_tiles(DJ, MT);
  constexpr int kPitch = 64 + 4;  // floats of a query row of 64 dims in LDS
  __shared__ __attribute__((aligned(16))) float s_o[kWaves][16][kPitch];
  __shared__ f32x2 s_ml[kWaves][MT * 16];
  __shared__ float s_lse[MT * 16];
  __shared__ float s_mass[kLdsMass];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const bool whole = a.n_parts == a.n_units, alone = whole && a.m_groups.d == 1;
  const Part part = part_of_workgroup<ST>(a, blockIdx.x, lane);
  if (part.idle) return;
  const uint32_t unit = part.row * a.m_groups.d + part.group;
  const Plan p = plan_unit<MT, ST>(a, part);
  const int first = part.index * p.part_steps;
  const int last = min(first + p.part_steps, p.steps);
  if (part.index == 0 && threadIdx.x == 0 && a.n_parts != a.n_units) {
    a.ws_of[2 * unit] = (int32_t)part.first;
    a.ws_of[2 * unit + 1] = part.of;
  }
  if (first >= last && !whole) return;

  u32x4 q[MT][DJ][2];
  int seen[MT];
  State<DJ, MT> st;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m = p.m0 + mt * 16 + lane % 16;
    seen[mt] = seen_by(a, p, m);
    const uint16_t* src = row_of(a.q, a, p, m) + 16 * (lane / 16);
#pragma unroll
    for (int j = 0; j < DJ; ++j)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        u16x8 x = {0, 0, 0, 0, 0, 0, 0, 0};
        if (seen[mt] > 0) {
          if (a.q.wide) {
            x = *(const u16x8*)(src + 64 * j + 8 * half);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = src[64 * j + 8 * half + i];
          }
        }
        q[mt][j][half] = __builtin_bit_cast(u32x4, x);
      }
    st.m[mt] = -INFINITY;
    st.l[mt] = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * DJ; ++i) st.o[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float* mass_row = a.ws_mass + (uint64_t)unit * a.unit_rows.d * a.cap_tiles;

  // While a step is computed the next one's tiles are on their way, and the page
  // ids of the one after: its keys take the registers of this one's as soon as
  // the scores are done, its values once they have been summed.  The loads are
  // made at the last step too, of one 16 bytes by all lanes: with a branch about
  // them the compiler's wait for the values would be one for the next keys too.
  int step = first + wave;
  if (step < last) {
    u32x4 k[ST][DJ], v[ST][DJ];
    Where<ST> here = find_step<DJ, ST>(a, p, step, ids_of_step<ST>(a, p, step));
    Ids<ST> ids = ids_of_step<ST>(a, p, min(step + kWaves, last - 1));
    load_tiles<DJ, ST, ONCE>(a.pool.k_codes, here, lane * 16, k);
    load_tiles<DJ, ST, ONCE>(a.pool.v_codes, here, lane * 16, v);
    while (true) {
      const int next_step = step + kWaves;
      const bool more = next_step < last;
      const int byte = more ? lane * 16 : 0;
      arrive<ST>(here, ids);
      Where<ST> next = find_step<DJ, ST>(a, p, more ? next_step : step, ids);
      ids = ids_of_step<ST>(a, p, min(next_step + kWaves, last - 1));
      f32x4 s[MT][ST];
      scores<DJ, F16, MT, ST>(k, q, s);
      load_tiles<DJ, ST, ONCE>(a.pool.k_codes, next, byte, k);
      bool plain = (step + 1) * (kTile * ST) <= p.full;
#pragma unroll
      for (int t = 0; t < ST; ++t) plain = plain && here.ok[t];
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const float c = here.ks[t] * a.scale;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[mt][t] *= c;
      }
      if (!plain) mask_step<DJ, MT, ST>(p, step, lane, seen, here, s, v, st);
      Probs<MT, ST> pr;
      softmax<DJ, MT, ST>(a, p, step, lane, here, s, mass_row, s_mass, st, pr);
      gather_values<DJ, MT, ST>(v, pr, st);
      load_tiles<DJ, ST, ONCE>(a.pool.v_codes, next, byte, v);
      if (!more) break;
      here = next;
      step = next_step;
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    st.l[mt] = pair_sum16(st.l[mt], st.l[mt]);
    st.l[mt] = pair_sum32(st.l[mt], st.l[mt]);
  }

  if (lane < 16) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) s_ml[wave][mt * 16 + lane] = f32x2{st.m[mt], st.l[mt]};
  }
  __syncthreads();
  const int n = threadIdx.x / 16, d4 = threadIdx.x % 16 * 4;  // query and dims of the joining
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m_local = mt * 16 + n, m = p.m0 + m_local;
    float top = -INFINITY, total = 0.f, f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_ml[w][m_local][0]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = exp2_fast(s_ml[w][m_local][0] - base);
      total += s_ml[w][m_local][1] * f[w];
    }
    const uint64_t slot = (uint64_t)part.slot * a.unit_rows.d + m_local;
    const bool here = m_local < (int)a.unit_rows.d && m < a.m_rows;
    const float share = total == 0.f ? 0.f : 1.f / total;
    const bool any = seen_by(a, p, m) > 0;
    if (d4 == 0) {
      if (alone)
        s_lse[m_local] = any ? log_total(top, total) : INFINITY;
      else if (here && (!whole || a.w_out))
        a.ws_ml[slot] = f32x2{top, total};
    }
#pragma unroll
    for (int h = 0; h < DJ; ++h) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *(f32x4*)&s_o[wave][lane % 16][16 * c + 4 * (lane / 16)] = st.o[mt][h * 4 + c];
      __syncthreads();
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) o += *(const f32x4*)&s_o[w][n][d4] * f[w];
      if (!here) continue;
      const int d = 64 * h + d4;
      if (whole) {
        uint16_t* dst = row_of(a.out, a, p, m) + d;
        u16x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = any ? to_half<F16>(o[r] * share) : 0;
        if (a.out.wide) {
          *(u16x4*)dst = y;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) dst[r] = y[r];
        }
      } else {
        *(f32x4*)(a.ws_o + slot * D + d) = o;
      }
    }
  }
  if (!alone || !a.w_out) return;
  __syncthreads();
  for (int base = 0; base < a.cap_tiles; base += kThreads) {  // whole waves: lanes add to each other
    const int tile = base + (int)threadIdx.x;
    float w = 0.f;
    if (tile < p.tiles)
      for (int m = 0; m < (int)a.unit_rows.d; m += 8)
        w += sum_shares(a, load_shares(a, a.mass_in_lds ? s_mass : mass_row, m, 1, tile), s_lse, m, 1);
    write_weight(a, p.row, tile, w);
  }
}

// The factors, in LDS, that the sums of a unit's parts (up to kMaxParts) take for
// a query row.
__device__ __forceinline__ void join_parts(const Attention& a, const Part& t, int parts, int m_local,
                                           int lane, float* factors) {
  auto part = [&](int n) {
    return a.ws_ml[((uint64_t)t.first + (uint64_t)n * a.m_groups.d) * a.unit_rows.d + m_local];
  };
  const f32x2 mine = lane < parts ? part(lane) : f32x2{-INFINITY, 0.f};
  float top = mine[0];
  for (int n = lane + kWave; n < parts; n += kWave) top = fmaxf(top, part(n)[0]);
  top = wave_max(top);
  const float base = top == -INFINITY ? 0.f : top;
  const float f = exp2_fast(mine[0] - base);
  float total = f * mine[1];
  for (int n = lane + kWave; n < parts; n += kWave) total += exp2_fast(part(n)[0] - base) * part(n)[1];
  total = wave_sum(total);
  const float share = total == 0.f ? 0.f : 1.f / total;
  factors[lane] = f * share;
  for (int n = lane + kWave; n < parts; n += kWave) factors[n] = exp2_fast(part(n)[0] - base) * share;
}

// Joins the parts.  The first workgroups take a query row each, or one for each
// of their waves where the units have few parts on average (264 units x 14 rows
// in 2 parts, with weights: 11.9 us by workgroups, 7.6 us so); the others take 256 or 64 tiles
// of a row each and sum their weights.  4-6 us with one unit to a head, which is the
// latency of its three loads that wait for each other.
template <int DJ, bool F16, int MT>
__global__ __launch_bounds__(kThreads) void combine_kernel(Attention a) {
  constexpr int D = 64 * DJ;
  constexpr int ST = step_tiles(DJ, MT);
  constexpr int kVec = D / 4;                 // threads of a row of the output
  constexpr int kGroups = kThreads / kVec;    // parts summed at a time
  constexpr int kAhead = 4;
  __shared__ __attribute__((aligned(16))) f32x4 s_sum[kGroups][kVec];
  __shared__ float s_f[kWaves][kMaxParts];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const uint32_t out_rows = a.n_parts == a.n_units ? 0u : a.n_units * a.unit_rows.d;
  const uint32_t out_blocks = a.wave_rows ? (out_rows + kWaves - 1) / kWaves : out_rows;
  if (blockIdx.x < out_blocks && a.wave_rows) {
    const uint32_t x = blockIdx.x * kWaves + wave, unit = quotient(x, a.unit_rows);
    if (x >= out_rows) return;
    const int m_local = (int)(x - unit * a.unit_rows.d);
    const uint32_t row = quotient(unit, a.m_groups);
    const Part t = parts_of_unit(a, row, (int)(unit - row * a.m_groups.d));
    const Plan p = plan_unit<MT, ST>(a, t);
    const int m = p.m0 + m_local;
    if (m >= a.m_rows) return;
    const int parts = seen_by(a, p, m) > 0 ? p.parts : 0;
    join_parts(a, t, parts, m_local, lane, s_f[wave]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    float o[DJ];  // dims 64 j + lane
#pragma unroll
    for (int j = 0; j < DJ; ++j) o[j] = 0.f;
#pragma unroll 4
    for (int n = 0; n < parts; ++n) {
      const float* sums = a.ws_o + (((uint64_t)t.first + (uint64_t)n * a.m_groups.d) * a.unit_rows.d + m_local) * D;
      const float f = s_f[wave][n];
#pragma unroll
      for (int j = 0; j < DJ; ++j) o[j] += sums[64 * j + lane] * f;
    }
    uint16_t* dst = row_of(a.out, a, p, m);
#pragma unroll
    for (int j = 0; j < DJ; ++j) dst[64 * j + lane] = to_half<F16>(o[j]);
    return;
  }
  if (blockIdx.x < out_blocks) {
    const uint32_t unit = quotient(blockIdx.x, a.unit_rows);
    const int m_local = (int)(blockIdx.x - unit * a.unit_rows.d);
    const uint32_t row = quotient(unit, a.m_groups);
    const Part t = parts_of_unit(a, row, (int)(unit - row * a.m_groups.d));
    const Plan p = plan_unit<MT, ST>(a, t);
    const int m = p.m0 + m_local;
    if (m >= a.m_rows) return;
    const int parts = seen_by(a, p, m) > 0 ? p.parts : 0;
    const int d4 = threadIdx.x % kVec, group = threadIdx.x / kVec;
    auto sums_of = [&](int n) {
      return *(const f32x4*)(a.ws_o + (((uint64_t)t.first + (uint64_t)n * a.m_groups.d) * a.unit_rows.d + m_local) * D + 4 * d4);
    };
    // the first parts' sums are on their way while the factors are worked out
    f32x4 o = {0.f, 0.f, 0.f, 0.f}, ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int n = group + i * kGroups;
      ahead[i] = group < kGroups && n < parts ? sums_of(n) : o;
    }
    if (wave == 0) join_parts(a, t, parts, m_local, lane, s_f[0]);
    __syncthreads();
    if (group < kGroups) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (group + i * kGroups < parts) o += ahead[i] * s_f[0][group + i * kGroups];
#pragma unroll 4
      for (int n = group + kAhead * kGroups; n < parts; n += kGroups) o += sums_of(n) * s_f[0][n];
      s_sum[group][d4] = o;
    }
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) o += s_sum[i][d4];
    uint16_t* dst = row_of(a.out, a, p, m) + 4 * d4;
    u16x4 y;
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = to_half<F16>(o[r]);
    if (a.out.wide) {
      *(u16x4*)dst = y;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) dst[r] = y[r];
    }
    return;
  }

  // With few query rows 256 tiles, each thread with all rows of its tile; with
  // many 64, wave w with rows w, w + 4, ..
  const uint32_t b = blockIdx.x - out_blocks;
  const uint32_t row = quotient(b, a.weight_blocks);
  const int stride = a.unit_rows.d > kFewRows ? kWaves : 1, start = stride == 1 ? 0 : wave;
  const int tile = (int)((b - row * a.weight_blocks.d) * (kThreads / stride)) +
                   (stride == 1 ? (int)threadIdx.x : lane);
  int spread = 1;  // lanes that hold a query row each; the others share its parts
  while (spread * kWaves < (int)a.unit_rows.d) spread *= 2;
  float w = 0.f;
  for (int g = 0; g < (int)a.m_groups.d; ++g) {
    const Part t = parts_of_unit(a, row, g);
    const Plan p = plan_unit<MT, ST>(a, t);
    const float* mass = a.ws_mass + ((uint64_t)row * a.m_groups.d + g) * a.unit_rows.d * a.cap_tiles;
    Shares first;
    if (tile < p.tiles) first = load_shares(a, mass, start, stride, tile);
    const int m = lane % spread * kWaves + wave;
    float top = -INFINITY, total = 0.f;
    if (m < (int)a.unit_rows.d && seen_by(a, p, p.m0 + m) > 0) {
#pragma unroll 4
      for (int n = lane / spread; n < p.parts; n += kWave / spread) {
        const f32x2 ml = a.ws_ml[((uint64_t)t.first + (uint64_t)n * a.m_groups.d) * a.unit_rows.d + m];
        const float higher = fmaxf(top, ml[0]), base = higher == -INFINITY ? 0.f : higher;
        total = total * exp2_fast(top - base) + ml[1] * exp2_fast(ml[0] - base);
        top = higher;
      }
    }
    for (int x = spread; x < kWave; x *= 2) {
      const float other = __shfl_xor(top, x), rest = __shfl_xor(total, x);
      const float higher = fmaxf(top, other), base = higher == -INFINITY ? 0.f : higher;
      total = total * exp2_fast(top - base) + rest * exp2_fast(other - base);
      top = higher;
    }
    if (lane < spread) s_f[0][m] = log_total(top, total);
    __syncthreads();
    if (tile < p.tiles) {
      w += sum_shares(a, first, s_f[0], start, stride);
      for (int i = start + 8 * stride; i < (int)a.unit_rows.d; i += 8 * stride)
        w += sum_shares(a, load_shares(a, mass, i, stride, tile), s_f[0], i, stride);
    }
    __syncthreads();
  }
  if (stride == 1) return write_weight(a, row, tile, w);
  float* sums = (float*)s_sum;
  sums[threadIdx.x] = w;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int i = 1; i < kWaves; ++i) w += sums[i * kWave + lane];
  write_weight(a, row, tile, w);
}

// ------------------------------------------------------------ eviction ----

struct Evict {
  const int32_t* pages;
  const int32_t* lengths;
  const float* weights;
  int32_t* pages_out;
  float* weights_out;
  int32_t* lengths_out;
  uint32_t max_pages;
  int32_t capacity;
  uint32_t page_shift;  // log2 of a page's tokens
  uint32_t keep, sink, recent;
};

// Whole numbers above 0 in the order of the weights.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __builtin_bit_cast(uint32_t, w + 0.f);  // -0 is 0
  const uint32_t key = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return w == w ? key : 0xFF800001u;  // NaN: one above infinity
}

// What a row's workgroup does: keep the protected pages and, of pages lo .. hi
// - 1, the `want` heaviest.
struct Choice {
  uint64_t at;  // the row's place in the tables
  int len;
  uint32_t held, left, lo, hi, want;
  bool full;
};

// A buffer of `bytes` bytes at an address that is the same for the whole wave.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00027000);
}

__device__ __forceinline__ Choice choice_of(const Evict& e, uint32_t row) {
  Choice c;
  c.at = (uint64_t)row * e.max_pages;
  c.len = min(max(e.lengths[row], 0), e.capacity);
  c.held = ((uint32_t)c.len + (1u << e.page_shift) - 1u) >> e.page_shift;
  c.full = c.held > e.keep;
  c.left = c.full ? e.keep : c.held;
  c.lo = e.sink;
  c.hi = c.full ? c.held - e.recent : c.held;
  c.want = c.full ? e.keep - e.sink - e.recent : 0;
  return c;
}

// One workgroup per row of up to THREADS * R pages, the weights in LDS.
// The weight of the last page to stay is found from counts in LDS: the keys
// between the smallest and the largest are counted in 1024 equal ranges, the
// range that holds the wanted one is cut into 1024 again, and so on.  (Bisecting
// with one count a round takes 25 rounds where this takes 2 or 3: 16,384 pages x
// 768 rows spent 47 us on it.)  With the counts of every 64 pages in LDS each
// page then knows its place.
// 768 rows of 16,384 pages (153 MB for those held, 201 MB with the spare entries)
// take 51 us: 1.5 workgroups to a place on the chip, and the loads, the choice and
// the stores of those that run together come one after the other (a row alone
// takes 17 us).  Without the buffers' bounds, with a branch for each page, 59 us.
template <int THREADS, int R>
__global__ __launch_bounds__(THREADS, 8) void evict_kernel(Evict e) {
  constexpr int kW = THREADS / kWave;
  constexpr int kUnroll = R < 8 ? R : 8;
  constexpr int kChunks = R * kW;  // of 64 pages, chunk i * kW + wave
  constexpr int kRanges = 1024, kMine = kRanges / kWave;  // of a lane that adds them up
  constexpr uint32_t kStays = 0xFFFFFFFFu;  // above every weight's key; 0 is below
  static_assert(kChunks <= 256, "a wave scans them, four to a lane");
  static_assert(THREADS > kWave && R <= 32);
  static_assert(THREADS * R < 65536, "two counts to a word");
  __shared__ __attribute__((aligned(16))) uint32_t s_count[2][kRanges];
  __shared__ uint32_t s_bound[2][kW];
  __shared__ uint32_t s_pick[3];
  __shared__ uint32_t s_chunk[256];      // pages that stay, and ties in the upper half
  __shared__ uint32_t s_key[R][THREADS];  // a thread reads its own only
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const Choice c = choice_of(e, blockIdx.x);
  if (threadIdx.x == 0) e.lengths_out[blockIdx.x] = c.len - (int)((c.held - c.left) << e.page_shift);
  // Buffers that end with the row: what lies past it is read as 0 and not
  // written, without a branch for each.  The whole offset is the lane's: a scalar
  // one would take no part in the check.
  const uint32_t bytes = e.max_pages * 4u;
  const auto weights = row_buffer(e.weights + c.at, bytes), weights_out = row_buffer(e.weights_out + c.at, bytes);
  const auto pages = row_buffer(e.pages + c.at, bytes), pages_out = row_buffer(e.pages_out + c.at, bytes);
  const int mine = (int)threadIdx.x * 4;
  // everything is asked for at once; the ids arrive while the places are worked out
  uint32_t w[R], id[R];
#pragma unroll
  for (int i = 0; i < R; ++i) w[i] = __builtin_amdgcn_raw_buffer_load_b32(weights, mine + i * THREADS * 4, 0, 0);
#pragma unroll
  for (int i = 0; i < R; ++i) id[i] = __builtin_amdgcn_raw_buffer_load_b32(pages, mine + i * THREADS * 4, 0, 0);
  const uint32_t span = c.full ? c.hi - c.lo : 0u;
  uint32_t low = 0xFFFFFFFFu, high = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint32_t p = (uint32_t)i * THREADS + threadIdx.x;
    uint32_t key = p < c.held ? kStays : 0u;
    if (p - c.lo < span) {
      key = weight_key(__builtin_bit_cast(float, w[i]));
      low = min(low, key);
      high = max(high, key);
    }
    s_key[i][threadIdx.x] = key;
  }
  uint32_t last = kStays - 1u, ties = 0;  // stay: keys above `last` and the first `ties` equal to it
  if (c.want) {
    low = ~wave_max(~low);
    high = wave_max(high);
    if (lane == 0) {
      s_bound[0][wave] = low;
      s_bound[1][wave] = high;
    }
    for (int i = threadIdx.x; i < kRanges; i += THREADS) s_count[0][i] = 0;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kW; ++x) {
      low = min(low, s_bound[0][x]);
      high = max(high, s_bound[1][x]);
    }
    low = (uint32_t)uniform((int)low);
    high = (uint32_t)uniform((int)high);
    // the key is in low .. high; `over` < want keys are above high
    uint32_t over = 0;
    uint32_t within = 0;  // which of the thread's keys are, from the second round on
    last = low;
    for (int round = 0; low < high; ++round) {
      const int shift = max(22 - (int)__builtin_clz(high - low), 0);
      uint32_t* count = s_count[round & 1];
      if (round < 2) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint32_t above_low = s_key[i][threadIdx.x] - low;
          if (above_low <= high - low) {
            atomicAdd(&count[above_low >> shift], 1u);
            within |= 1u << i;
          }
        }
        if (round == 0) within = 0;
      } else {  // few are left
        for (uint32_t left = within; left; left &= left - 1) {
          const int i = __builtin_ctz(left);
          const uint32_t above_low = s_key[i][threadIdx.x] - low;
          if (above_low <= high - low)
            atomicAdd(&count[above_low >> shift], 1u);
          else
            within &= ~(1u << i);
        }
      }
      __syncthreads();
      if (wave == 0) {
        // lane l adds up ranges from kMine (63 - l); the lane that holds the
        // wanted one has its ranges looked at one to a lane
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < kMine; i += 4) {
          const u32x4 four = *(const u32x4*)&count[kMine * (kWave - 1 - lane) + i];
          mine += (four[0] + four[1]) + (four[2] + four[3]);
        }
        uint32_t before = over + wave_scan(mine) - mine;
        const int src = __builtin_ctzll(__ballot(before < c.want && before + mine >= c.want));
        before = (uint32_t)__builtin_amdgcn_readlane((int)before, src);
        const int range = kMine * (kWave - src) - 1 - lane;
        const uint32_t n = lane < kMine ? count[range] : 0u;
        before += wave_scan(n) - n;
        if (before < c.want && before + n >= c.want) {
          s_pick[0] = (uint32_t)range;
          s_pick[1] = before;
          s_pick[2] = before + n;
        }
      } else {
        for (int i = (int)threadIdx.x - kWave; i < kRanges; i += THREADS - kWave) s_count[(round & 1) ^ 1][i] = 0;
      }
      __syncthreads();
      low += (uint32_t)uniform((int)s_pick[0]) << shift;
      over = (uint32_t)uniform((int)s_pick[1]);
      if (high - low >= 1u << shift) high = low + ((1u << shift) - 1u);  // no sum past 32 bits
      last = low;
      if ((uint32_t)uniform((int)s_pick[2]) == c.want) {  // the whole range stays
        last = low - 1u;
        over = c.want;
        break;
      }
    }
    ties = c.want - over;
  }

#pragma unroll kUnroll
  for (int i = 0; i < R; ++i) {
    const uint32_t key = s_key[i][threadIdx.x];
    uint32_t n = (uint32_t)__popcll(__ballot(key > last));
    if (ties) n += (uint32_t)__popcll(__ballot(key == last)) << 16;
    if (lane == 0) s_chunk[i * kW + wave] = n;
  }
  __syncthreads();
  if (wave == 0) {  // counts before each chunk
    uint32_t x[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = 4 * lane + i < kChunks ? s_chunk[4 * lane + i] : 0u;
      sum += x[i];
    }
    uint32_t before = wave_scan(sum) - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * lane + i < kChunks) s_chunk[4 * lane + i] = before;
      before += x[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint32_t p = (uint32_t)i * THREADS + threadIdx.x;
    const uint32_t key = s_key[i][threadIdx.x], chunk = s_chunk[i * kW + wave];
    uint32_t before = lanes_below(__ballot(key > last), chunk & 0xFFFFu);  // pages that stay before this one
    bool stays = key > last;
    if (ties) {
      const uint32_t tie = lanes_below(__ballot(key == last), chunk >> 16);
      stays = stays || (key == last && tie < ties);
      before += min(tie, ties);
    }
    // past the row's pages `before` is `left`, so that they keep their places
    const uint32_t to = stays ? before : c.left + p - before;
    __builtin_amdgcn_raw_buffer_store_b32(id[i], pages_out, (int)to * 4, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(key != 0u && !stays ? 0u : w[i], weights_out, (int)to * 4, 0, 0);
  }
}

// Rows of any length: the weight is found digit by digit (8 bits at a time,
// from counts in LDS), the weights read again for each (172 us for the 768 rows
// above).
__global__ __launch_bounds__(kThreads) void evict_long_kernel(Evict e) {
  __shared__ uint32_t s_count[256];
  __shared__ uint32_t s_pick[2];
  __shared__ uint32_t s_sum[2][kWaves];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const Choice ch = choice_of(e, blockIdx.x);
  const uint64_t at = ch.at;
  const float* weights = e.weights + at;
  const uint32_t held = ch.held, left = ch.left, lo = ch.lo, hi = ch.hi;
  const bool full = ch.full;
  if (threadIdx.x == 0) e.lengths_out[blockIdx.x] = ch.len - (int)((held - left) << e.page_shift);

  uint32_t key = 0, want = ch.want;
  if (full && want) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      s_count[threadIdx.x] = 0;
      __syncthreads();
      for (uint32_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        const uint32_t k = weight_key(weights[i]);
        if (shift == 24 || (k ^ key) >> (shift + 8) == 0) atomicAdd(&s_count[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (wave == 0) {  // lane l: digits 255 - 4 l down to 252 - 4 l
        uint32_t c[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += c[i] = s_count[255 - 4 * lane - i];
        uint32_t before = wave_scan(mine) - mine;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before < want && before + c[i] >= want) {
            s_pick[0] = 255u - 4u * lane - i;
            s_pick[1] = want - before;
          }
          before += c[i];
        }
      }
      __syncthreads();
      key |= s_pick[0] << shift;
      want = s_pick[1];
    }
  }

  // kept: above the key, the first `want` equal to it, and the protected ones
  uint32_t above_before = 0, equal_before = 0;
  for (uint32_t base = 0; base < e.max_pages; base += kThreads) {
    const uint32_t i = base + threadIdx.x;
    const bool in = i < e.max_pages;
    const float w = in ? weights[i] : 0.f;
    const int32_t id = in ? e.pages[at + i] : 0;
    const bool middle = full && i >= lo && i < hi;
    const uint32_t k = weight_key(w);
    const bool above = i < held && (!middle || (want && k > key));
    const bool equal = middle && want && k == key;
    const uint64_t ba = __ballot(above), be = __ballot(equal);
    if (lane == 0) {
      s_sum[0][wave] = (uint32_t)__popcll(ba);
      s_sum[1][wave] = (uint32_t)__popcll(be);
    }
    __syncthreads();
    uint32_t a = above_before, q = equal_before;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
      if (x < wave) {
        a += s_sum[0][x];
        q += s_sum[1][x];
      }
      above_before += s_sum[0][x];
      equal_before += s_sum[1][x];
    }
    __syncthreads();
    const uint64_t under = (1ull << lane) - 1ull;
    a += (uint32_t)__popcll(ba & under);
    q += (uint32_t)__popcll(be & under);
    if (in) {
      const bool kept = above || (equal && q < want);
      const uint32_t kept_before = a + min(q, want);
      uint32_t to = i;
      if (i < held) to = kept ? kept_before : left + (i - kept_before);
      e.pages_out[at + to] = id;
      e.weights_out[at + to] = i < held && !kept ? 0.f : w;
    }
  }
}

// ------------------------------------------------------------------ host ----

thread_local int g_last_hip = 0;

int hip_fail(hipError_t e) {
  g_last_hip = (int)e;
  return IBP_ERR_HIP;
}

int pending_hip_error() {
  const hipError_t e = hipPeekAtLastError();
  return e == hipSuccess ? IBP_OK : hip_fail(e);
}

int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? IBP_OK : hip_fail(e);
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// Workgroups of a launch, which has fewer than 2^32 threads.
constexpr uint64_t max_grid(uint64_t threads) { return 0xFFFFFFFFull / threads; }

int check_cache(const ibp_kv_cache* c) {
  if (!c) return IBP_ERR_INVALID_ARGUMENT;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64) return IBP_ERR_UNSUPPORTED;
  if (c->head_dim == 0 || c->head_dim % 64 || c->head_dim > 256) return IBP_ERR_UNSUPPORTED;
  if (c->n_pages == 0) return IBP_OK;  // every id is a hole
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
      !aligned(c->v_scales, 4))
    return IBP_ERR_LAYOUT;
  return IBP_OK;
}

// 0 rows is no error; the caller returns at once.
int check_table(const ibp_kv_table* t, uint64_t page_tokens, uint64_t* n_rows) {
  if (!t) return IBP_ERR_INVALID_ARGUMENT;
  if (t->n_seqs && t->kv_heads > (1ull << 30) / t->n_seqs) return IBP_ERR_INVALID_ARGUMENT;
  *n_rows = t->n_seqs * t->kv_heads;
  if (*n_rows == 0) return IBP_OK;
  if (t->max_pages > 0x7FFFFFFFull / page_tokens) return IBP_ERR_INVALID_ARGUMENT;
  if (!t->lengths || (t->max_pages && !t->pages)) return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(t->lengths, 4) || !aligned(t->pages, 4)) return IBP_ERR_LAYOUT;
  return IBP_OK;
}

int check_tensor(const ibp_kv_tensor* x) {
  if (!x || !x->data) return IBP_ERR_INVALID_ARGUMENT;
  return aligned(x->data, 2) ? IBP_OK : IBP_ERR_LAYOUT;
}

// Whether rows of `d` elements lie on each other along one axis, as those of a
// broadcast tensor do.
bool rows_overlap(uint64_t size, int64_t stride, uint32_t d) {
  return size > 1 && stride < (int64_t)d && stride > -(int64_t)d;
}

Pool make_pool(const ibp_kv_cache* c) {
  Pool p;
  p.k_codes = c->k_codes;
  p.k_scales = c->k_scales;
  p.v_codes = c->v_codes;
  p.v_scales = c->v_scales;
  p.n_pages = (uint32_t)std::min<uint64_t>(c->n_pages, 1ull << 31);
  p.page_bytes = c->page_tokens * c->head_dim;
  p.tile_shift = c->page_tokens == 16 ? 0 : c->page_tokens == 32 ? 1 : 2;
  return p;
}

Divisor make_divisor(uint32_t d) {
  Divisor x = {d, 0, 31};
  while ((1ull << (x.shift - 31)) < d) ++x.shift;
  x.mul = (uint32_t)(((1ull << x.shift) + d - 1) / std::max<uint32_t>(d, 1));
  return x;
}

Rows make_rows(const ibp_kv_table* t, uint32_t page_tokens, uint64_t n_new, const int32_t* counts) {
  Rows r;
  r.pages = t->pages;
  r.lengths = t->lengths;
  r.counts = counts;
  r.heads = make_divisor((uint32_t)t->kv_heads);
  r.max_pages = (uint32_t)t->max_pages;
  r.capacity = (int32_t)(t->max_pages * page_tokens);
  r.n_new = (int32_t)n_new;
  return r;
}

Strided make_strided(const ibp_kv_tensor* x) {
  Strided s;
  s.data = (uint16_t*)x->data;
  s.seq = x->seq_stride;
  s.token = x->token_stride;
  s.head = x->head_stride;
  s.wide = aligned(x->data, 16) && x->seq_stride % 8 == 0 && x->token_stride % 8 == 0 &&
           x->head_stride % 8 == 0;
  return s;
}

template <int DJ, bool F16>
void launch_append(const Pool& pool, const Rows& rows, const Strided& k, const Strided& v,
                   uint32_t pages_per_row, uint32_t tasks, hipStream_t st) {
  const uint32_t per_group = kWaves >> pool.tile_shift;
  hipLaunchKernelGGL((append_kernel<DJ, F16>), dim3((tasks + per_group - 1) / per_group),
                     dim3(kThreads), 0, st, pool, rows, k, v, make_divisor(pages_per_row), tasks);
}

// How the query rows of a head are cut into units, and the units into parts.
struct Shape {
  int mt;
  int32_t m_rows, m_groups, unit_rows, cap_tiles;
  uint32_t n_units, n_parts;
  uint32_t weight_blocks;  // of a row, in the joining kernel
  uint32_t join_blocks;    // workgroups of the joining kernel; 0: it is not launched
  bool wave_rows, mass_in_lds;
  uint64_t of_at, mass_at, ml_at, bytes;  // in the workspace; the sums come first
};

// Compute units of the current device, read once per device; 256 where a HIP
// error is pending, which is not this library's to clear, and where there is no
// device.
int compute_units() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, n = 0;
  if (hipPeekAtLastError() != hipSuccess) return 256;
  if (hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kDevices) {
    n = known[dev].load(std::memory_order_relaxed);
    if (n == 0 && hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess)
      known[dev].store(n, std::memory_order_relaxed);
  }
  if (n <= 0) {
    (void)hipGetLastError();
    n = 256;
  }
  return n;
}

bool make_shape(uint64_t n_rows, uint64_t max_pages, uint32_t page_tokens, uint32_t head_dim,
                uint64_t group, uint64_t n_new, bool weights, int cus, Shape* s) {
  if (n_new && group > (1ull << 24) / n_new) return false;
  const uint64_t m = group * n_new;
  s->m_rows = (int32_t)m;
  s->mt = m <= 16 ? 1 : kQueryTiles;
  const uint64_t per_unit = 16ull * s->mt;
  s->m_groups = (int32_t)((m + per_unit - 1) / per_unit);
  s->unit_rows = (int32_t)std::min<uint64_t>(m, per_unit);
  s->cap_tiles = (int32_t)(max_pages * page_tokens / kTile);
  const uint64_t units = n_rows * s->m_groups;
  if (units > max_grid(kThreads)) return false;
  s->n_units = (uint32_t)units;
  // As many parts as keep all workgroups on the chip at once: what comes after them
  // would start over with an empty pipeline.  Rows of up to four steps a wave are
  // not worth the second launch, which costs about as much as those.  Units that
  // fill three quarters of the chip are cut for the sake of rows much longer than
  // the others: of 264 rows of 128 dims and 14 query rows, one with 4538 tokens
  // and the rest with 454, 17.1 us cut and 30.9 whole (384 rows: 22.1 and 31.7);
  // rows of 454 to 4538 tokens pay the second launch for it, 42.4 us cut and 39.7
  // whole (384 rows: 64.8 and 58.4).  Past that, and past the rows whose lengths
  // share_out holds, every unit is a workgroup, whatever its row's length.
  const int st = step_tiles((int)head_dim / 64, s->mt);
  const uint64_t steps = (uint64_t)(s->cap_tiles + st - 1) / st;
  const uint64_t slots = std::min<uint64_t>((uint64_t)workgroups_per_unit((int)head_dim / 64, s->mt) * cus, kMaxParts);
  s->n_parts = s->n_units;
  if (units && units <= slots / 4 * 3 && n_rows <= (uint64_t)kWave * kRowsPerLane && steps > 4 * kWaves &&
      steps * units < (1ull << 31))  // the sums of share_out
    s->n_parts = (uint32_t)(std::min<uint64_t>(slots, units * ((steps + kWaves - 1) / kWaves + 1)) / s->m_groups *
                            s->m_groups);
  const bool whole = s->n_parts == s->n_units, alone = whole && s->m_groups <= 1;
  const uint64_t parts = (uint64_t)s->n_parts * s->unit_rows;
  s->ml_at = whole ? 0 : parts * head_dim * 4;
  s->of_at = s->ml_at + (alone || (whole && !weights) ? 0 : parts * 8);
  s->mass_at = (s->of_at + (s->n_parts != s->n_units ? units * 8 : 0) + 15) / 16 * 16;
  s->mass_in_lds = alone && (uint64_t)s->unit_rows * s->cap_tiles <= (uint64_t)kLdsMass;
  s->bytes = s->mass_at + (weights && !s->mass_in_lds ? units * s->unit_rows * s->cap_tiles * 4 : 0);
  // The joining kernel: output rows of units that were cut, weights of rows whose
  // workgroups do not finish them.
  const uint64_t out_rows = whole ? 0 : units * s->unit_rows;
  const uint32_t block_tiles = s->unit_rows > kFewRows ? kWave : kThreads;
  s->wave_rows = s->n_parts <= 8ull * s->n_units;
  s->weight_blocks = ((uint32_t)s->cap_tiles + block_tiles - 1) / block_tiles;
  const uint64_t join = (s->wave_rows ? (out_rows + kWaves - 1) / kWaves : out_rows) +
                        (weights && !(whole && s->m_groups == 1) ? n_rows * s->weight_blocks : 0);
  s->join_blocks = (uint32_t)join;
  return join <= max_grid(kThreads);
}

template <int DJ, bool F16, int MT>
void launch_attention(const Attention& a, uint32_t join_blocks, hipStream_t st) {
  if (a.n_units && a.m_groups.d == 1)
    hipLaunchKernelGGL((attention_kernel<DJ, F16, MT, true>), dim3(a.n_parts), dim3(kThreads), 0, st, a);
  if constexpr (MT == kQueryTiles)  // only such units are one of several
    if (a.m_groups.d > 1)
      hipLaunchKernelGGL((attention_kernel<DJ, F16, MT, false>), dim3(a.n_parts), dim3(kThreads), 0, st, a);
  if (join_blocks)
    hipLaunchKernelGGL((combine_kernel<DJ, F16, MT>), dim3(join_blocks), dim3(kThreads), 0, st, a);
}

template <int DJ, bool F16>
void launch_attention_mt(const Attention& a, const Shape& s, hipStream_t st) {
  if (s.mt == 1) return launch_attention<DJ, F16, 1>(a, s.join_blocks, st);
  launch_attention<DJ, F16, kQueryTiles>(a, s.join_blocks, st);
}

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

int ibp_kv_last_hip_error(void) { return g_last_hip; }

const char* ibp_kv_status_string(int status) {
  switch (status) {
    case IBP_OK: return "ok";
    case IBP_ERR_INVALID_ARGUMENT: return "invalid argument";
    case IBP_ERR_UNSUPPORTED: return "unsupported page size, head size or type";
    case IBP_ERR_LAYOUT: return "misaligned pointer";
    case IBP_ERR_HIP: return "HIP error";
    default: return "unknown status";
  }
}

int ibp_kv_append(const ibp_kv_cache* cache, const ibp_kv_table* table, uint32_t dtype,
                  uint64_t n_new, const ibp_kv_tensor* k, const ibp_kv_tensor* v,
                  const int32_t* counts, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (dtype > IBP_KV_FP16) return IBP_ERR_UNSUPPORTED;
  uint64_t n_rows = 0;
  rc = check_table(table, cache->page_tokens, &n_rows);
  if (rc || n_rows == 0 || n_new == 0 || table->max_pages == 0 || cache->n_pages == 0) return rc;
  if (n_new > 0x7FFFFFFFull) return IBP_ERR_INVALID_ARGUMENT;
  if ((rc = check_tensor(k)) || (rc = check_tensor(v))) return rc;
  if (!aligned(counts, 4)) return IBP_ERR_LAYOUT;
  const uint64_t pt = cache->page_tokens;
  const uint64_t per_row = std::min<uint64_t>((n_new + pt - 2) / pt + 1, table->max_pages);
  const uint64_t per_group = (uint64_t)kWaves * kTile / pt;
  if (per_row > max_grid(kThreads) * per_group / n_rows) return IBP_ERR_INVALID_ARGUMENT;
  rc = pending_hip_error();
  if (rc) return rc;
  const Pool pool = make_pool(cache);
  const Rows rows = make_rows(table, cache->page_tokens, n_new, counts);
  const Strided ks = make_strided(k), vs = make_strided(v);
  hipStream_t st = (hipStream_t)stream;
  const uint32_t tasks = (uint32_t)(n_rows * per_row);
  switch (cache->head_dim / 64 * 2 + dtype) {
    case 2: launch_append<1, false>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
    case 3: launch_append<1, true>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
    case 4: launch_append<2, false>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
    case 5: launch_append<2, true>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
    case 6: launch_append<3, false>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
    case 7: launch_append<3, true>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
    case 8: launch_append<4, false>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
    default: launch_append<4, true>(pool, rows, ks, vs, (uint32_t)per_row, tasks, st); break;
  }
  return launched();
}

uint64_t ibp_kv_attention_workspace_bytes(const ibp_kv_cache* cache, const ibp_kv_table* table,
                                          uint64_t q_heads, uint64_t n_new, int with_weights) {
  uint64_t n_rows = 0;
  if (check_cache(cache) || !table || table->kv_heads == 0 || q_heads % table->kv_heads) return 0;
  if (table->n_seqs && table->kv_heads > (1ull << 30) / table->n_seqs) return 0;
  if (table->max_pages > 0x7FFFFFFFull / cache->page_tokens) return 0;
  n_rows = table->n_seqs * table->kv_heads;
  Shape s;
  if (!make_shape(n_rows, table->max_pages, cache->page_tokens, cache->head_dim,
                  q_heads / table->kv_heads, n_new, with_weights != 0, compute_units(), &s))
    return 0;
  return s.bytes;
}

int ibp_kv_attention(const ibp_kv_cache* cache, const ibp_kv_table* table, uint32_t dtype,
                     uint64_t q_heads, uint64_t n_new, const ibp_kv_tensor* q,
                     const ibp_kv_tensor* out, const int32_t* counts, float scale,
                     const float* weights, float* weights_out, void* workspace,
                     uint64_t workspace_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (dtype > IBP_KV_FP16) return IBP_ERR_UNSUPPORTED;
  uint64_t n_rows = 0;
  rc = check_table(table, cache->page_tokens, &n_rows);
  if (rc || n_rows == 0) return rc;
  if (q_heads == 0 || q_heads % table->kv_heads || !weights != !weights_out || !(scale - scale == 0.f))
    return IBP_ERR_INVALID_ARGUMENT;
  if (n_new && ((rc = check_tensor(q)) || (rc = check_tensor(out)))) return rc;
  if (n_new && (rows_overlap(table->n_seqs, out->seq_stride, cache->head_dim) ||
                rows_overlap(n_new, out->token_stride, cache->head_dim) ||
                rows_overlap(q_heads, out->head_stride, cache->head_dim)))
    return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(counts, 4) || !aligned(weights, 4) || !aligned(weights_out, 4)) return IBP_ERR_LAYOUT;
  if (!aligned(workspace, 16)) return IBP_ERR_LAYOUT;
  Shape s;
  if (!make_shape(n_rows, table->max_pages, cache->page_tokens, cache->head_dim,
                  q_heads / table->kv_heads, n_new, weights != nullptr, compute_units(), &s))
    return IBP_ERR_INVALID_ARGUMENT;
  if (s.bytes && (!workspace || workspace_bytes < s.bytes)) return IBP_ERR_INVALID_ARGUMENT;
  rc = pending_hip_error();
  if (rc) return rc;
  Attention a{};
  a.pool = make_pool(cache);
  a.rows = make_rows(table, cache->page_tokens, n_new, counts);
  if (cache->n_pages == 0) a.rows.capacity = 0;  // holes only: nothing to see, and no page to read
  if (n_new) {
    a.q = make_strided(q);
    a.out = make_strided(out);
  }
  a.w_in = weights;
  a.w_out = weights_out;
  a.ws_o = (float*)workspace;
  a.ws_ml = (f32x2*)((char*)workspace + s.ml_at);
  a.ws_mass = (float*)((char*)workspace + s.mass_at);
  a.ws_of = (int32_t*)((char*)workspace + s.of_at);
  a.scale = scale * 1.44269504088896340736f;
  a.group = make_divisor((uint32_t)(q_heads / table->kv_heads));
  a.m_rows = s.m_rows;
  a.m_groups = make_divisor((uint32_t)s.m_groups);
  a.unit_rows = make_divisor((uint32_t)s.unit_rows);
  a.cap_tiles = s.cap_tiles;
  a.mass_in_lds = s.mass_in_lds;
  a.wave_rows = s.wave_rows;
  a.n_units = s.n_units;
  a.n_rows = (uint32_t)n_rows;
  a.n_parts = s.n_parts;
  a.weight_blocks = make_divisor(s.weight_blocks);
  hipStream_t st = (hipStream_t)stream;
  switch (cache->head_dim / 64 * 2 + dtype) {
    case 2: launch_attention_mt<1, false>(a, s, st); break;
    case 3: launch_attention_mt<1, true>(a, s, st); break;
    case 4: launch_attention_mt<2, false>(a, s, st); break;
    case 5: launch_attention_mt<2, true>(a, s, st); break;
    case 6: launch_attention_mt<3, false>(a, s, st); break;
    case 7: launch_attention_mt<3, true>(a, s, st); break;
    case 8: launch_attention_mt<4, false>(a, s, st); break;
    default: launch_attention_mt<4, true>(a, s, st); break;
  }
  return launched();
}

int ibp_kv_evict(const ibp_kv_table* table, uint32_t page_tokens, uint64_t keep_pages,
                 uint64_t sink_pages, uint64_t recent_pages, const float* weights,
                 int32_t* pages_out, float* weights_out, int32_t* lengths_out, void* stream) {
  if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64) return IBP_ERR_UNSUPPORTED;
  uint64_t n_rows = 0;
  int rc = check_table(table, page_tokens, &n_rows);
  if (rc) return rc;
  if (recent_pages == 0 || sink_pages > keep_pages || recent_pages > keep_pages - sink_pages)
    return IBP_ERR_INVALID_ARGUMENT;
  if (n_rows == 0) return IBP_OK;
  const uint64_t n = n_rows * table->max_pages * 4, nl = n_rows * 4;
  if (!lengths_out || (n && (!weights || !pages_out || !weights_out))) return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(weights, 4) || !aligned(pages_out, 4) || !aligned(weights_out, 4) || !aligned(lengths_out, 4))
    return IBP_ERR_LAYOUT;
  const void* in[3] = {table->pages, weights, table->lengths};
  void* outs[3] = {pages_out, weights_out, lengths_out};
  const uint64_t size[3] = {n, n, nl};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3; ++j)
      if (overlap(in[i], size[i], outs[j], size[j]) || (i < j && overlap(outs[i], size[i], outs[j], size[j])))
        return IBP_ERR_INVALID_ARGUMENT;
  const bool wide = table->max_pages > 1024 && table->max_pages <= 16384;  // 1024 threads a row
  if (n_rows > max_grid(wide ? 1024 : kThreads)) return IBP_ERR_INVALID_ARGUMENT;
  rc = pending_hip_error();
  if (rc) return rc;
  Evict e;
  e.pages = table->pages;
  e.lengths = table->lengths;
  e.weights = weights;
  e.pages_out = pages_out;
  e.weights_out = weights_out;
  e.lengths_out = lengths_out;
  e.max_pages = (uint32_t)table->max_pages;
  e.capacity = (int32_t)(table->max_pages * page_tokens);
  e.page_shift = page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : 6;
  e.keep = (uint32_t)std::min<uint64_t>(keep_pages, 0xFFFFFFFFull);
  e.sink = (uint32_t)std::min<uint64_t>(sink_pages, 0xFFFFFFFFull);
  e.recent = (uint32_t)std::min<uint64_t>(recent_pages, 0xFFFFFFFFull);
  const dim3 grid((uint32_t)n_rows);
  hipStream_t st = (hipStream_t)stream;
  // The smallest that holds a row: 512 rows of 1024 pages take 7.7 us with 256
  // threads and 10.8 with 1024, 512 rows of 4096 pages 14.2 us with 4 pages a
  // thread and 21.6 with 16.  Past 16384 pages the keys no longer fit LDS.
  if (table->max_pages <= 1024)
    hipLaunchKernelGGL((evict_kernel<256, 4>), grid, dim3(256), 0, st, e);
  else if (table->max_pages <= 4096)
    hipLaunchKernelGGL((evict_kernel<1024, 4>), grid, dim3(1024), 0, st, e);
  else if (table->max_pages <= 16384)
    hipLaunchKernelGGL((evict_kernel<1024, 16>), grid, dim3(1024), 0, st, e);
  else
    hipLaunchKernelGGL(evict_long_kernel, grid, dim3(kThreads), 0, st, e);
  return launched();
}

}  // extern "C"
