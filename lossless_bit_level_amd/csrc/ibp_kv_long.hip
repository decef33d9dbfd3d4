// libibp_kv_long: appends with rotated positions, outlines and selection of
// pages, and attention over a shared prefix, on the 8-bit KV pages of libibp_kv,
// for AMD Instinct MI355X (gfx950, CDNA4).  Calls: include/ibp_kv_long.h.
//
// Times below are of one launch by kernel trace unless something else is said; rates
// count the bytes that the operation cannot do without.  A large copy reaches 6.1 TB/s
// on this card, a large bf16 product 1.35 PFLOP/s.
//
//   append_rotated   as append, the rotation between its loads and its conversions, the
//                    outline from the codes it has in registers; queries in further
//                    workgroups of the launch: HBM, 5.0 TB/s
//   outline          a wave for a run of a row's pages: HBM and half as much in vector
//                    instructions, 4.8 TB/s
//   select           rows of few pages in one launch, a workgroup each; of more in two,
//                    scores by workgroups of 256 pages: a chain of dependent loads
//   attention_shared the prefix's units and the rows' in one launch, joined by a second:
//                    HBM with few query rows, with many the instructions of the softmax
//                    and the matrix products
#include "ibp_kv_core.h"

#include "ibp_kv_long.h"

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

struct Angles {
  const float* cos;
  const float* sin;
  const int32_t* positions;
  uint32_t n_positions;
  int32_t half;  // pairs
};

// ------------------------------------------------ largest and smallest ----

// NaN wins.
__device__ __forceinline__ f16x2 pair_max(f16x2 a, f16x2 b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ f16x2 pair_min(f16x2 a, f16x2 b) { return __builtin_elementwise_minimum(a, b); }

// Smallest e with a <= 127 * 2^e (127 = 1.984375 * 2^6), for a > 0.
__device__ __forceinline__ int whole_exponent(float a) {
  const uint32_t b = __builtin_bit_cast(uint32_t, a);
  return (int)(b >> 23) - 127 - 6 + ((b & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
}

// What lanes l and l ^ 16 (l ^ 32) hold, the same in both.
struct Pair16 {
  f16x2 a, b;
};
__device__ __forceinline__ Pair16 both16(f16x2 x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return {__builtin_bit_cast(f16x2, (uint32_t)y[0]), __builtin_bit_cast(f16x2, (uint32_t)y[1])};
}
__device__ __forceinline__ Pair16 both32(f16x2 x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return {__builtin_bit_cast(f16x2, (uint32_t)y[0]), __builtin_bit_cast(f16x2, (uint32_t)y[1])};
}

// The largest and the smallest so far of the numbers of four codes (a word) in each
// of several tokens; NaN where one was.
struct Bounds4 {
  f16x2 hi[2], lo[2];
  __device__ __forceinline__ void clear() {
    hi[0] = hi[1] = f16x2{-INFINITY, -INFINITY};
    lo[0] = lo[1] = f16x2{INFINITY, INFINITY};
  }
  // Two words, since an instruction takes the largest of three.
  __device__ __forceinline__ void take(uint32_t a, uint32_t b) {
    const f16x2 a0 = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false));
    const f16x2 a1 = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true));
    const f16x2 b0 = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false));
    const f16x2 b1 = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true));
    hi[0] = pair_max(pair_max(hi[0], a0), b0);
    hi[1] = pair_max(pair_max(hi[1], a1), b1);
    lo[0] = pair_min(pair_min(lo[0], a0), b0);
    lo[1] = pair_min(pair_min(lo[1], a1), b1);
  }
  __device__ __forceinline__ void join(const Bounds4& x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      hi[h] = pair_max(hi[h], x.hi[h]);
      lo[h] = pair_min(lo[h], x.lo[h]);
    }
  }
  __device__ __forceinline__ float largest() const {  // magnitude: hi >= lo
    const f16x2 x = pair_max(pair_max(hi[0], -lo[0]), pair_max(hi[1], -lo[1]));
    return __builtin_elementwise_maximum((float)x[0], (float)x[1]);
  }
};

// Four numbers in units of 1 / per, at most 127 of them, rounded up, or down.  128 more is
// a positive number, which one instruction makes a byte of.
template <bool UP>
__device__ __forceinline__ uint32_t whole4(const f16x2 (&x)[2], float per) {
  uint32_t word = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float y = __builtin_fmaf((float)x[b / 2][b % 2], per, 128.f);  // exact
    word = __builtin_amdgcn_cvt_pk_u8_f32(UP ? __builtin_ceilf(y) : __builtin_floorf(y), b, word);
  }
  return word ^ 0x80808080u;
}

// Bounds of the keys of a tile, four dims to a lane, through the wave's words in LDS:
// kc are the lane's codes of token lane % 16, dims 64 j + 16 (lane / 16) + 0..15, as
// pages have them; the tile has `tokens` of them (none: at most 0).  A lane reads its
// dims of a run of tokens and joins them with the lanes that have the others.
constexpr int kKeyPitch = 64 + 4;  // words of 16 dims, so that lanes of different dims read different banks

template <int DJ>
__device__ __forceinline__ Bounds4 tile_bounds(const u32x4 (&kc)[DJ], uint32_t* words, int lane, int tokens) {
  constexpr int kLanes = 16 * DJ, kParts = kWave / kLanes;  // of a token, of the tokens
  constexpr int kRun = kTile / kParts;
#pragma unroll
  for (int j = 0; j < DJ; ++j) *(u32x4*)(words + (4 * j + lane / 16) * kKeyPitch + 4 * (lane % 16)) = kc[j];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int r = lane % kLanes, from = min(lane / kLanes, kParts - 1) * kRun;
  Bounds4 x;
  x.clear();
  if (tokens > 0) {
    const uint32_t* mine = words + r / 4 * kKeyPitch + r % 4;
    if (tokens >= kTile) {
#pragma unroll
      for (int i = 0; i < kRun; i += 2) x.take(mine[4 * (from + i)], mine[4 * (from + i + 1)]);
    } else {  // past the tile's tokens the last one again
      auto word = [&](int i) { return mine[4 * min(from + i, tokens - 1)]; };
#pragma unroll
      for (int i = 0; i < kRun; i += 2) x.take(word(i), word(i + 1));
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (DJ == 1) {
      const Pair16 y = both16(x.hi[h]), z = both16(x.lo[h]);
      x.hi[h] = pair_max(y.a, y.b);
      x.lo[h] = pair_min(z.a, z.b);
    }
    if constexpr (DJ <= 2) {
      const Pair16 y = both32(x.hi[h]), z = both32(x.lo[h]);
      x.hi[h] = pair_max(y.a, y.b);
      x.lo[h] = pair_min(z.a, z.b);
    }
  }
  __builtin_amdgcn_wave_barrier();  // the wave's reads are before what it writes next
  return x;
}

// Writes the outline of a page from its bounds.
template <int DJ>
__device__ __forceinline__ void write_outline(const ibp_kv_outlines& o, const Bounds4& x, int lane, uint32_t id, float k_scale) {
  constexpr int D = 64 * DJ;
  // magnitudes are in the order of their bits, NaN of either sign above them
  const uint32_t top = (uint32_t)uniform((int)wave_max(__builtin_bit_cast(uint32_t, x.largest())));
  const bool bad = top > 0x7F800000u || !finite(k_scale);
  const int e = max(whole_exponent(__builtin_bit_cast(float, top)), -15);
  const float per = bad ? 0.f : power2(-e);
  if (lane == 0) o.scales[id] = bad ? NAN : k_scale * power2(e);
  if (lane >= 16 * DJ) return;
  uint32_t* to = (uint32_t*)(o.codes + (uint64_t)id * (2 * D)) + lane;
  to[0] = bad ? 0u : whole4<true>(x.hi, per);
  to[D / 4] = bad ? 0u : whole4<false>(x.lo, per);
}

// ------------------------------------------------------------- rotation ----

// Where the other number of a pair is: half a rotation away, which with all dims
// of an even number of 64s rotated is in the same lane's registers, or next to it.
enum class Pairs { kFar, kLane, kNeighbour };

struct Floats8 {
  float x[8];
};

template <bool F16>
__device__ __forceinline__ Floats8 floats_of(u32x4 h) {
  Floats8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.x[i] = to_float<F16>((uint16_t)(h[i / 2] >> (i % 2 * 16)));
  return r;
}

// Each product and each sum rounded: plain 32-bit arithmetic gives the same.
__device__ __forceinline__ float turned_first(float x, float y, float c, float s) {
#pragma clang fp contract(off)
  const float a = x * c, b = y * s;
  return a - b;
}
__device__ __forceinline__ float turned_second(float x, float y, float c, float s) {
#pragma clang fp contract(off)
  const float a = y * c, b = x * s;
  return a + b;
}

template <Pairs PAIRS>
struct Turn {
  static constexpr bool kTurns = true;
  Angles t;
  ibp_kv_outlines o;  // codes null: none

  __device__ __forceinline__ int position(const Rows& rows, uint32_t seq, int token, int place) const {
    return t.positions ? t.positions[(uint64_t)seq * (uint32_t)rows.n_new + (uint32_t)token] : place;
  }

  // cos and sin of N pairs from pair `i` on (a multiple of 4); NaN outside the tables.
  template <int N>
  __device__ __forceinline__ void angles(int pos, int i, float (&c)[N], float (&s)[N]) const {
    const bool in = (uint32_t)pos < t.n_positions;
    const uint64_t at = (uint64_t)(in ? (uint32_t)pos : 0u) * (uint32_t)t.half + (uint32_t)i;
#pragma unroll
    for (int n = 0; n < N; n += 4) {
      f32x4 a = {NAN, NAN, NAN, NAN}, b = a;
      if (in) {
        a = *(const f32x4*)(t.cos + at + n);
        b = *(const f32x4*)(t.sin + at + n);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        c[n + r] = a[r];
        s[n + r] = b[r];
      }
    }
  }

  // Eight numbers, whole pairs of neighbours, in place.
  __device__ __forceinline__ void neighbours(int pos, int d, Floats8& f) const {
    float c[4], s[4];
    angles(pos, d / 2, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f.x[2 * i], y = f.x[2 * i + 1];
      f.x[2 * i] = turned_first(x, y, c[i], s[i]);
      f.x[2 * i + 1] = turned_second(x, y, c[i], s[i]);
    }
  }

  // Eight pairs from pair `i` on, in place.
  __device__ __forceinline__ void pairs(int pos, int i, Floats8& a, Floats8& b) const {
    float c[8], s[8];
    angles(pos, i, c, s);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float x = a.x[n], y = b.x[n];
      a.x[n] = turned_first(x, y, c[n], s[n]);
      b.x[n] = turned_second(x, y, c[n], s[n]);
    }
  }

  // The outline of the page whose tile a wave has just made (codes kc, as tile_bounds
  // takes them); a page's waves meet in LDS.  All waves of the workgroup call this.
  template <int DJ>
  __device__ __forceinline__ void outline(const u32x4 (&kc)[DJ], int wave, int lane, int tile, int tiles, int tokens, bool there,
                                          uint32_t id, float k_scale) const {
    if (!o.codes) return;
    __shared__ __attribute__((aligned(16))) uint32_t s_keys[kWaves][4 * DJ * kKeyPitch];
    Bounds4 x = tile_bounds<DJ>(kc, s_keys[wave], lane, tokens);
    if (tiles > 1) {
      *(u32x4*)(s_keys[wave] + 4 * lane) = __builtin_bit_cast(u32x4, x);
      __syncthreads();
      if (tile == 0)
        for (int n = 1; n < tiles; ++n) x.join(__builtin_bit_cast(Bounds4, *(const u32x4*)(s_keys[wave + n] + 4 * lane)));
    }
    if (there && tile == 0) write_outline<DJ>(o, x, lane, id, k_scale);
  }

  // The lane's numbers of a key, dims 64 j + 16 g + 0..15, turned.  `key`: its dim
  // 0; kx: what the lane has of it.
  template <int DJ, bool F16>
  __device__ __forceinline__ void keys(const uint16_t* key, bool wide, int g, int pos, const u32x4 (&kx)[DJ][2],
                                       float (&ky)[DJ][16]) const {
    if constexpr (PAIRS == Pairs::kLane) {
#pragma unroll
      for (int j = 0; j < DJ / 2; ++j)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          Floats8 a = floats_of<F16>(kx[j][o]), b = floats_of<F16>(kx[j + DJ / 2][o]);
          pairs(pos, 64 * j + 16 * g + 8 * o, a, b);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ky[j][8 * o + i] = a.x[i];
            ky[j + DJ / 2][8 * o + i] = b.x[i];
          }
        }
    } else {
#pragma unroll
      for (int j = 0; j < DJ; ++j)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int d = 64 * j + 16 * g + 8 * o;
          Floats8 a = floats_of<F16>(kx[j][o]);
          if (d < 2 * t.half) {
            if constexpr (PAIRS == Pairs::kNeighbour) {
              neighbours(pos, d, a);
            } else {
              const bool first = d < t.half;
              const int other = first ? d + t.half : d - t.half;
              Floats8 b = floats_of<F16>(load8(key + other, wide));
              float c[8], s[8];
              angles(pos, first ? d : other, c, s);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                a.x[i] = first ? turned_first(a.x[i], b.x[i], c[i], s[i]) : turned_second(b.x[i], a.x[i], c[i], s[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) ky[j][8 * o + i] = a.x[i];
        }
    }
  }
};

constexpr uint32_t kHeadRun = 4;  // heads of a token that a thread turns by the same angles

struct Queries {
  Strided q, out;
  Divisor runs, group, n_new;  // runs of kHeadRun heads
  uint32_t q_heads;
  uint32_t n_items;  // 16 numbers of a run of queries each
};

template <bool F16>
__device__ __forceinline__ void store8(uint16_t* p, bool wide, const Floats8& f, bool there) {
  u16x8 h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = there ? to_half<F16>(f.x[i]) : (uint16_t)0;
  if (wide) {
    *(u16x8*)p = h;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = h[i];
  }
}

// 16 numbers of each query of a run: eight pairs, or what is not rotated.
template <int DJ, bool F16, Pairs PAIRS>
__device__ __forceinline__ void turn_query(const Queries& a, const Rows& rows, const Turn<PAIRS>& turn, uint32_t x) {
  constexpr uint32_t kItems = 4 * DJ;
  if (x >= a.n_items) return;
  const uint32_t y = x / kItems;
  const int item = (int)(x - y * kItems), half = turn.t.half;
  const uint32_t t = quotient(y, a.runs), head = (y - t * a.runs.d) * kHeadRun;
  const uint32_t seq = quotient(t, a.n_new), i = t - seq * a.n_new.d;
  const bool rotated = PAIRS == Pairs::kNeighbour ? 16 * item < 2 * half : 8 * item < half;
  int d0 = 16 * item, d1 = d0 + 8;
  if (PAIRS != Pairs::kNeighbour) {
    d0 = rotated ? 8 * item : 2 * half + 16 * (item - half / 8);
    d1 = rotated ? d0 + half : d0 + 8;
  }
  const int count = new_count(rows, seq);
  u32x4 v[kHeadRun][2];
  int place[kHeadRun];
  bool there[kHeadRun];
#pragma unroll
  for (uint32_t h = 0; h < kHeadRun; ++h) {
    const uint32_t at = min(head + h, a.q_heads - 1);
    place[h] = row_length(rows, seq * rows.heads.d + quotient(at, a.group)) - count + (int)i;
    there[h] = (int)i < count && place[h] >= 0;
    v[h][0] = v[h][1] = u32x4{0, 0, 0, 0};
    if (there[h]) {
      const uint16_t* p = a.q.data + (int64_t)seq * a.q.seq + (int64_t)i * a.q.token + (int64_t)at * a.q.head;
      v[h][0] = load8(p + d0, a.q.wide);
      v[h][1] = load8(p + d1, a.q.wide);
    }
  }
  // heads of a sequence are at the same place but where their rows differ
  float c[8], s[8];
  int known = 0;
  bool any = false;
#pragma unroll
  for (uint32_t h = 0; h < kHeadRun; ++h) {
    if (head + h >= a.q_heads) break;
    Floats8 f = floats_of<F16>(v[h][0]), g = floats_of<F16>(v[h][1]);
    if (there[h] && rotated) {
      const int pos = turn.position(rows, seq, (int)i, place[h]);
      if (!any || pos != known) turn.angles(pos, PAIRS == Pairs::kNeighbour ? d0 / 2 : d0, c, s);
      known = pos;
      any = true;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float& first = PAIRS == Pairs::kNeighbour ? (n < 4 ? f.x[2 * n % 8] : g.x[2 * n % 8]) : f.x[n];
        float& second = PAIRS == Pairs::kNeighbour ? (n < 4 ? f.x[2 * n % 8 + 1] : g.x[2 * n % 8 + 1]) : g.x[n];
        const float p = first, q = second;
        first = turned_first(p, q, c[n], s[n]);
        second = turned_second(p, q, c[n], s[n]);
      }
    }
    uint16_t* to = a.out.data + (int64_t)seq * a.out.seq + (int64_t)i * a.out.token + (int64_t)(head + h) * a.out.head;
    store8<F16>(to + d0, a.out.wide, f, there[h]);
    store8<F16>(to + d1, a.out.wide, g, there[h]);
  }
}

// The first workgroups append, the others rotate the queries.  4 prompts of 4096 tokens x
// 32 heads of 128 dims, with as many query heads and outlines: 682 MB in 136 us, 5.0 TB/s
// (of what is moved, 759 MB with the angles, 5.5); with the outlines in a launch of their
// own 157 us.  One user's token: 5.6 us.
template <int DJ, bool F16, Pairs PAIRS>
__global__ __launch_bounds__(kThreads) void append_rotated_kernel(Pool pool, Rows rows, Strided k, Strided v,
                                                                  Divisor pages_per_row, uint32_t n_tasks,
                                                                  Turn<PAIRS> turn, Queries queries,
                                                                  uint32_t append_blocks) {
  if (blockIdx.x < append_blocks)
    append_tile<DJ, F16>(pool, rows, k, v, pages_per_row, n_tasks, turn);
  else
    turn_query<DJ, F16, PAIRS>(queries, rows, turn, (blockIdx.x - append_blocks) * kThreads + threadIdx.x);
}

// -------------------------------------------------------------- outline ----

// A row's waves share its pages evenly, up to 64 to a wave, which takes them one after
// the other, a tile at a time: it has their ids and scales at once, and the next tiles
// are on their way while one is looked at.  e4m3 codes are exact in 16 bits, two to an instruction.
// Two contexts of 131k and 91k tokens x 8 heads of 128 dims: 257 MB in 54 us, 4.8 TB/s,
// of which reading the codes alone takes 48; a tile is 100 vector instructions, with 150
// it took 60.  (A wave for two pages at most: 62 us; four lanes to 16 dims, so that a load
// takes 64 bytes of a place: 68 us, both of those with 150.)
template <int DJ>
__global__ __launch_bounds__(kThreads) void outline_kernel(Pool pool, Rows rows, ibp_kv_outlines o, Divisor chunks,
                                                           uint32_t n_chunks) {
  constexpr int kAhead = DJ <= 2 ? 4 : 2;  // tiles on their way
  __shared__ __attribute__((aligned(16))) uint32_t s_keys[kWaves][4 * DJ * kKeyPitch];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const uint32_t task = blockIdx.x * kWaves + wave;
  if (task >= n_chunks) return;
  const uint32_t row = quotient(task, chunks), seq = quotient(row, rows.heads);
  const int end = row_length(rows, row), count = new_count(rows, seq);
  const int page_shift = 4 + (int)pool.tile_shift, tiles = 1 << pool.tile_shift;
  const int held = (end + (1 << page_shift) - 1) >> page_shift;
  const int touched = max(end - count, 0) >> page_shift;
  const int wave_pages = (int)quotient((uint32_t)(held - touched) + chunks.d - 1u, chunks);
  const int from = touched + (int)(task - row * chunks.d) * wave_pages;
  const int pages = count > 0 ? min(held - from, wave_pages) : 0;
  if (pages <= 0) return;
  uint32_t ids = ~0u;
  if (lane < pages) ids = (uint32_t)rows.pages[(uint64_t)row * rows.max_pages + (uint32_t)(from + lane)];
  float scales = 0.f;
  if (ids < pool.n_pages) scales = pool.k_scales[ids];
  // tile 0 of the first of the pages, and so on; the last one again past the last
  const int units = uniform(min(pages << pool.tile_shift, ((end + kTile - 1) / kTile) - (from << pool.tile_shift)));
  auto id_of = [&](int unit) { return (uint32_t)__builtin_amdgcn_readlane((int)ids, unit >> pool.tile_shift); };
  u32x4 w[kAhead][DJ];
  auto load = [&](int unit, u32x4 (&to)[DJ]) {
    unit = min(unit, units - 1);
    const uint32_t id = id_of(unit), at = id < pool.n_pages ? id : 0u;
    const uint8_t* p = pool.k_codes + (uint64_t)at * pool.page_bytes + (uint32_t)((unit & (tiles - 1)) * (DJ * kUnit));
#pragma unroll
    for (int j = 0; j < DJ; ++j) to[j] = __builtin_nontemporal_load((const u32x4*)(p + j * kUnit + lane * 16));
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, w[i]);
  Bounds4 x;
  x.clear();
  for (int first = 0; first < units; first += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int unit = first + i;
      if (unit < units) {
        x.join(tile_bounds<DJ>(w[i], s_keys[wave], lane, end - (from << page_shift) - unit * kTile));
        if ((unit & (tiles - 1)) == tiles - 1 || unit == units - 1) {
          const uint32_t id = id_of(unit);
          if (id < pool.n_pages)
            write_outline<DJ>(o, x, lane, id, __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, scales), unit >> pool.tile_shift)));
          x.clear();
        }
      }
      load(unit + kAhead, w[i]);
    }
  }
}

// ------------------------------------------------------------ selection ----

struct Select {
  Rows rows;
  uint32_t n_pages;
  const int8_t* codes;
  const float* outline_scales;
  Strided q;
  Divisor group;
  int32_t m_rows;  // query rows of a key/value head
  float* scores;   // [row][max_pages]
  Divisor chunks;  // of a row, in the scoring kernel
  uint32_t page_shift;
  uint32_t keep, sink, recent;
  int32_t* pages_out;
  int32_t* lengths_out;
  int32_t* places_out;
};

// What a row's workgroup does: keep the protected pages and, of pages lo .. hi
// - 1, the `want` with the largest scores.
struct Selection {
  int len;
  uint32_t held, left, lo, hi, want;
  bool full;
};

__device__ __forceinline__ Selection selection_of(const Select& s, uint32_t row) {
  Selection c;
  c.len = row_length(s.rows, row);
  c.held = ((uint32_t)c.len + (1u << s.page_shift) - 1u) >> s.page_shift;
  c.full = c.held > s.keep;
  c.left = c.full ? s.keep : c.held;
  c.lo = s.sink;
  c.hi = c.full ? c.held - s.recent : c.held;
  c.want = c.full ? s.keep - s.sink - s.recent : 0;
  return c;
}

// Groups of 16 pages that a wave has in registers.
constexpr int score_groups(int dj) { return dj <= 2 ? 4 : 2; }
constexpr int score_pages(int dj, int threads) { return 16 * score_groups(dj) * (threads / kWave); }  // of a workgroup at a time

// Scores of a row's pages.  S of 16 queries and 16 pages is a product of 8-bit
// matrices: a query's whole numbers in two limbs of at most 127, those of positive
// numbers against the largest and those of negative ones against the smallest of each
// dim.  With the sums of the upper limbs shifted by 7 the lower ones add on top; all is
// exact in 32 bits (16256 * 127 * 256 < 2^30).
template <int DJ>
struct ScoreLds {
  __attribute__((aligned(16))) uint32_t limbs[DJ][2][2][kWave][4];  // as the lanes of the matrix instructions take them
  float unit[16];                                                   // 0: no query
};

// Whose pages and queries.
struct ScoreRow {
  __amdgpu_buffer_rsrc_t pages;  // ends with the row
  uint32_t seq, head;
  int count, origin;
};

__device__ __forceinline__ ScoreRow score_row(const Select& s, const Selection& c, uint32_t row) {
  ScoreRow r;
  r.pages = row_buffer(s.rows.pages + (uint64_t)row * s.rows.max_pages, s.rows.max_pages * 4u);
  r.seq = quotient(row, s.rows.heads);
  r.head = row - r.seq * s.rows.heads.d;
  r.count = new_count(s.rows, r.seq);
  r.origin = c.len - r.count;
  return r;
}

// 16 queries to four waves: wave w has 4 w .. 4 w + 3, 16 lanes each; lane x has dims
// 64 j + 4 x + 0..3.
template <int DJ>
struct Queries16 {
  uint16_t q[DJ][4];
  int token;  // -1: no such row
};

template <int DJ>
__device__ __forceinline__ Queries16<DJ> load_queries(const Select& s, const ScoreRow& r, int m0, int wave, int lane) {
  Queries16<DJ> y;
  const int n = wave * 4 + lane / 16, x = lane % 16, m = m0 + n;
  const int t = (int)quotient((uint32_t)m, s.group);
  y.token = n < 16 && m < s.m_rows ? t : -1;
#pragma unroll
  for (int j = 0; j < DJ; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y.q[j][i] = 0;
    if (y.token >= 0) {
      const uint16_t* src = s.q.data + (int64_t)r.seq * s.q.seq + (int64_t)t * s.q.token +
                            ((int64_t)r.head * s.group.d + (m - t * (int)s.group.d)) * s.q.head + 64 * j + 4 * x;
      if (s.q.wide) {
        const u16x4 h = *(const u16x4*)src;
#pragma unroll
        for (int i = 0; i < 4; ++i) y.q[j][i] = h[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y.q[j][i] = src[i];
      }
    }
  }
  return y;
}

// Groups of 16 queries whose limbs are in LDS at a time: 32 KB.
constexpr int query_slots(int dj) { return dj <= 2 ? 4 : 2; }

template <int DJ, bool F16>
__device__ __forceinline__ void write_limbs(const Queries16<DJ>& y, const ScoreRow& r, ScoreLds<DJ>& lds, int wave, int lane) {
  const int n = wave * 4 + lane / 16, x = lane % 16;
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < DJ; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, y.q[j][i] & 0x7FFFu);
  float amax = not_finite<F16>(top) ? INFINITY : to_float<F16>((uint16_t)top);
  amax = fmaxf(amax, row_rotate<0x121>(amax));
  amax = fmaxf(amax, row_rotate<0x122>(amax));
  amax = fmaxf(amax, row_rotate<0x124>(amax));
  amax = fmaxf(amax, row_rotate<0x128>(amax));
  // 127 * 128 * 2^e is 127 * 2^(e + 7)
  const bool counts = y.token >= 0 && y.token < r.count && r.origin + y.token >= 0 && finite(amax);
  const int e = counts ? max(whole_exponent(amax) - 7, -126) : 0;
  const float per = power2(-e);
  if (x == 0) lds.unit[n] = counts ? power2(e) : 0.f;
#pragma unroll
  for (int j = 0; j < DJ; ++j) {
    uint32_t words[2][2] = {{0, 0}, {0, 0}};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int whole = counts ? (int)__builtin_rintf(to_float<F16>(y.q[j][i]) * per) : 0;
      const int upper = (whole + 64) >> 7, lower = whole - 128 * upper;
      const int side = whole < 0 ? 1 : 0;
      const uint32_t u = (uint32_t)(upper & 255) << (8 * i), l = (uint32_t)(lower & 255) << (8 * i);
      words[0][0] |= side ? 0u : u;
      words[0][1] |= side ? 0u : l;
      words[1][0] |= side ? u : 0u;
      words[1][1] |= side ? l : 0u;
    }
#pragma unroll
    for (int end = 0; end < 2; ++end)
#pragma unroll
      for (int limb = 0; limb < 2; ++limb) lds.limbs[j][end][limb][x / 4 * 16 + n][x % 4] = words[end][limb];
  }
}

// The outlines of pages first + 16 p + lane % 16.  Ids are asked for before the row's
// length is known.
template <int DJ>
struct PageSet {
  static constexpr int P = score_groups(DJ);
  u32x4 b[P][DJ][2];
  float scale[P];
  bool live[P];
};

template <int DJ>
struct PageIds {
  uint32_t id[score_groups(DJ)];
};

template <int DJ>
__device__ __forceinline__ PageIds<DJ> load_ids(const ScoreRow& r, uint32_t first, int lane) {
  PageIds<DJ> x;
#pragma unroll
  for (int p = 0; p < score_groups(DJ); ++p)
    x.id[p] = __builtin_amdgcn_raw_buffer_load_b32(r.pages, (int)(first + 16 * p + lane % 16) * 4, 0, 0);
  return x;
}

template <int DJ>
__device__ __forceinline__ PageSet<DJ> load_outlines(const Select& s, const Selection& c, const PageIds<DJ>& ids, uint32_t first,
                                                     int lane) {
  constexpr int D = 64 * DJ;
  PageSet<DJ> x;
#pragma unroll
  for (int p = 0; p < x.P; ++p) {
    const uint32_t page = first + 16 * p + lane % 16;
    x.live[p] = page >= c.lo && page < c.hi && ids.id[p] < s.n_pages;
    const uint32_t at = x.live[p] ? ids.id[p] : 0u;
    x.scale[p] = 0.f;
    if (s.n_pages == 0) continue;
    x.scale[p] = s.outline_scales[at];
    const int8_t* codes = s.codes + (uint64_t)at * (2 * D) + (lane / 16) * 16;
#pragma unroll
    for (int j = 0; j < DJ; ++j)
#pragma unroll
      for (int end = 0; end < 2; ++end) x.b[p][j][end] = *(const u32x4*)(codes + end * D + 64 * j);
  }
  return x;
}

// The largest so far over the queries in LDS: the lane has queries 4 (lane / 16) + r of
// page lane % 16 of each group.
template <int DJ>
__device__ __forceinline__ void take_queries(const PageSet<DJ>& x, const ScoreLds<DJ>& lds, int lane, float (&best)[PageSet<DJ>::P]) {
  constexpr int P = PageSet<DJ>::P;
  i32x4 sum[P];
#pragma unroll
  for (int p = 0; p < P; ++p) sum[p] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int limb = 0; limb < 2; ++limb) {
#pragma unroll
    for (int j = 0; j < DJ; ++j)
#pragma unroll
      for (int end = 0; end < 2; ++end) {
        const i32x4 a = *(const i32x4*)lds.limbs[j][end][limb][lane];
#pragma unroll
        for (int p = 0; p < P; ++p)
          sum[p] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, __builtin_bit_cast(i32x4, x.b[p][j][end]), sum[p], 0, 0, 0);
      }
    if (limb == 0) {
#pragma unroll
      for (int p = 0; p < P; ++p) sum[p] <<= 7;
    }
  }
  float unit[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) unit[r] = lds.unit[4 * (lane / 16) + r];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r) best[p] = unit[r] > 0.f ? fmaxf(best[p], (float)sum[p][r] * unit[r]) : best[p];
}

// The score of page first + lane, for lanes below 16 P.
template <int DJ>
__device__ __forceinline__ float score_of_lane(const PageSet<DJ>& x, float (&best)[PageSet<DJ>::P], int lane) {
  float mine = 0.f;
#pragma unroll
  for (int p = 0; p < x.P; ++p) {
    f32x2 y = both16(best[p]);
    y = both32(fmaxf(y[0], y[1]));
    const float score = x.live[p] ? fmaxf(y[0], y[1]) * x.scale[p] : -INFINITY;
    if (p == 0 || lane / 16 == p) mine = score;
  }
  return mine;
}

// The limbs of queries m0 .. of the row, as many as there are slots; the first four waves
// make them, all wait.
template <int DJ, bool F16>
__device__ __forceinline__ void fill_slots(const Select& s, const ScoreRow& r, ScoreLds<DJ> (&lds)[query_slots(DJ)], int m0,
                                           int wave, int lane, Queries16<DJ> (&q)[query_slots(DJ)]) {
#pragma unroll
  for (int i = 0; i < query_slots(DJ); ++i)
    if (wave < 4 && m0 + 16 * i < s.m_rows) write_limbs<DJ, F16>(q[i], r, lds[i], wave, lane);
  __syncthreads();
}

template <int DJ>
__device__ __forceinline__ void load_slots(const Select& s, const ScoreRow& r, int m0, int wave, int lane,
                                           Queries16<DJ> (&q)[query_slots(DJ)]) {
#pragma unroll
  for (int i = 0; i < query_slots(DJ); ++i)
    if (m0 + 16 * i < s.m_rows) q[i] = load_queries<DJ>(s, r, m0 + 16 * i, wave, lane);
}

template <int DJ>
__device__ __forceinline__ void take_slots(const Select& s, const PageSet<DJ>& x, const ScoreLds<DJ> (&lds)[query_slots(DJ)], int m0,
                                           int lane, float (&best)[PageSet<DJ>::P]) {
  for (int i = 0; i < query_slots(DJ) && m0 + 16 * i < s.m_rows; ++i) take_queries<DJ>(x, lds[i], lane, best);
}

// Scores of a run of a row's pages, into the workspace.  Bound by its chain of loads,
// lengths and ids, then outlines: two contexts of 131k and 91k tokens x 8 heads (28 MB)
// 11.2 us.
template <int DJ, bool F16>
__global__ __launch_bounds__(kThreads) void score_kernel(Select s) {
  constexpr int P = PageSet<DJ>::P, kSlots = query_slots(DJ);
  __shared__ ScoreLds<DJ> lds[kSlots];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const uint32_t row = quotient(blockIdx.x, s.chunks);
  const uint32_t from = (blockIdx.x - row * s.chunks.d) * score_pages(DJ, kThreads), first = from + wave * (16 * P);
  // Queries and ids before the row's length is known; the queries first, since loads
  // return in order and the outlines are on their way while the limbs are made.
  const Selection c = selection_of(s, row);
  const ScoreRow r = score_row(s, c, row);
  Queries16<DJ> q[kSlots];
  load_slots<DJ>(s, r, 0, wave, lane, q);
  const PageIds<DJ> ids = load_ids<DJ>(r, first, lane);
  if (!c.full || !c.want || from >= c.hi || from + score_pages(DJ, kThreads) <= c.lo) return;
  const PageSet<DJ> x = load_outlines<DJ>(s, c, ids, first, lane);
  float best[P];
#pragma unroll
  for (int p = 0; p < P; ++p) best[p] = -INFINITY;
  for (int m0 = 0; m0 < s.m_rows; m0 += 16 * kSlots) {
    if (m0) {
      load_slots<DJ>(s, r, m0, wave, lane, q);
      __syncthreads();
    }
    fill_slots<DJ, F16>(s, r, lds, m0, wave, lane, q);
    take_slots<DJ>(s, x, lds, m0, lane, best);
  }
  const float mine = score_of_lane<DJ>(x, best, lane);
  const uint32_t page = first + lane;
  if (lane < 16 * P && page >= c.lo && page < c.hi) s.scores[(uint64_t)row * s.rows.max_pages + page] = mine;
}

// Writes what stays, in order, and -1 past it.
__device__ __forceinline__ void fill_rest(const Select& s, uint32_t row, uint32_t left, uint32_t threads) {
  for (uint32_t i = left + threadIdx.x; i < s.keep; i += threads) {
    s.pages_out[(uint64_t)row * s.keep + i] = -1;
    s.places_out[(uint64_t)row * s.keep + i] = -1;
  }
}

// The key of page p of a row, for cut_of; `score`: if it is one to be chosen from.
__device__ __forceinline__ uint32_t page_key(const Selection& c, uint32_t p, float score) {
  if (c.want && p - c.lo < c.hi - c.lo) return weight_key(score);
  return p < c.held && (!c.full || p < c.lo || p >= c.hi) ? kStays : 0u;
}

// Chooses and writes: id[i] is that of the thread's page i.  Through buffers that end
// with the row, whatever the scores were.
template <int THREADS, int R>
__device__ __forceinline__ void write_selection(const Select& s, const Selection& c, ChoiceLds<THREADS, R>& lds, uint32_t row,
                                                uint32_t low, uint32_t high, const uint32_t (&id)[R], int wave, int lane, int used) {
  const Cut cut = cut_of<THREADS, R>(lds, low, high, c.want, wave, lane, used);
  count_chunks<THREADS, R>(lds, cut, wave, lane, used);
  const uint64_t at = (uint64_t)row * s.keep;
  const auto pages_out = row_buffer(s.pages_out + at, s.keep * 4u), places_out = row_buffer(s.places_out + at, s.keep * 4u);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < used) {
      const Stay x = stay_of<THREADS, R>(lds, cut, i, lds.key[i][threadIdx.x], wave);
      if (x.stays) {
        __builtin_amdgcn_raw_buffer_store_b32(id[i], pages_out, (int)x.before * 4, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b32((uint32_t)i * THREADS + threadIdx.x, places_out, (int)x.before * 4, 0, 0);
      }
    }
  }
  fill_rest(s, row, c.left, THREADS);
}

// One workgroup per row of up to THREADS * R pages, their scores in the workspace: 16
// rows of 8192 and 5664 pages 7.6 us, the rounds of the choice and the barriers between.
// (With ids asked for once it is known what stays 13 us; where all pages of a row of the
// largest size were looked at, and what does not stay written past the row's end, 9.4.)
template <int THREADS, int R>
__global__ __launch_bounds__(THREADS) void select_kernel(Select s) {
  __shared__ ChoiceLds<THREADS, R> lds;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const uint32_t row = blockIdx.x;
  const uint64_t at = (uint64_t)row * s.rows.max_pages;
  const auto scores = row_buffer(s.scores + at, s.rows.max_pages * 4u), pages = row_buffer(s.rows.pages + at, s.rows.max_pages * 4u);
  uint32_t w[R], id[R];
#pragma unroll
  for (int i = 0; i < R; ++i) w[i] = __builtin_amdgcn_raw_buffer_load_b32(scores, (int)threadIdx.x * 4 + i * THREADS * 4, 0, 0);
#pragma unroll
  for (int i = 0; i < R; ++i) id[i] = __builtin_amdgcn_raw_buffer_load_b32(pages, (int)threadIdx.x * 4 + i * THREADS * 4, 0, 0);
  const Selection c = selection_of(s, row);
  if (threadIdx.x == 0) s.lengths_out[row] = c.len - (int)((c.held - c.left) << s.page_shift);
  uint32_t low = 0xFFFFFFFFu, high = 0;
  const int used = (int)((c.held + THREADS - 1) / THREADS);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < used) {
      const uint32_t p = (uint32_t)i * THREADS + threadIdx.x;
      const uint32_t key = page_key(c, p, __builtin_bit_cast(float, w[i]));
      if (c.want && p - c.lo < c.hi - c.lo) {
        low = min(low, key);
        high = max(high, key);
      }
      lds.key[i][threadIdx.x] = key;
    }
  }
  write_selection<THREADS, R>(s, c, lds, row, low, high, id, wave, lane, used);
}

// Rows of up to THREADS * R pages, scored and chosen from in one launch: 16 x 32 rows of
// 180 to 256 pages (30 MB) 11.5 us, which is the chain lengths and ids, outlines, limbs,
// products, rounds of the choice, stores.
template <int DJ, bool F16, int THREADS, int R>
__global__ __launch_bounds__(THREADS) void select_short_kernel(Select s) {
  constexpr int P = PageSet<DJ>::P;
  constexpr int kAtOnce = score_pages(DJ, THREADS), kTimes = THREADS * R / kAtOnce;
  constexpr int kSlots = query_slots(DJ);
  __shared__ ScoreLds<DJ> score[kSlots];
  __shared__ ChoiceLds<THREADS, R> lds;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const uint32_t row = blockIdx.x;
  const Selection c = selection_of(s, row);
  const ScoreRow r = score_row(s, c, row);
  Queries16<DJ> q[kSlots];
  load_slots<DJ>(s, r, 0, wave, lane, q);
  PageIds<DJ> ids = load_ids<DJ>(r, wave * (16 * P), lane);
  uint32_t id[R];
#pragma unroll
  for (int i = 0; i < R; ++i) id[i] = __builtin_amdgcn_raw_buffer_load_b32(r.pages, (int)threadIdx.x * 4 + i * THREADS * 4, 0, 0);
  if (threadIdx.x == 0) s.lengths_out[row] = c.len - (int)((c.held - c.left) << s.page_shift);
  uint32_t low = 0xFFFFFFFFu, high = 0;
  const int used = (int)((c.held + THREADS - 1) / THREADS);
  if (c.want) {
    const int times = (int)min((c.hi + kAtOnce - 1) / kAtOnce, (uint32_t)kTimes);
    for (int i = 0; i < times; ++i) {
      const uint32_t first = i * kAtOnce + wave * (16 * P);
      const PageSet<DJ> x = load_outlines<DJ>(s, c, ids, first, lane);
      ids = load_ids<DJ>(r, first + kAtOnce, lane);
      float best[P];
#pragma unroll
      for (int p = 0; p < P; ++p) best[p] = -INFINITY;
      for (int m0 = 0; m0 < s.m_rows; m0 += 16 * kSlots) {
        const bool turns = s.m_rows > 16 * kSlots;  // the slots are filled again for each run of pages
        if (turns && (i || m0)) {
          load_slots<DJ>(s, r, m0, wave, lane, q);
          __syncthreads();
        }
        if (turns || i == 0) fill_slots<DJ, F16>(s, r, score, m0, wave, lane, q);
        take_slots<DJ>(s, x, score, m0, lane, best);
      }
      const float mine = score_of_lane<DJ>(x, best, lane);
      const uint32_t p = first + lane;
      if (lane < 16 * P) lds.key[p / THREADS][p % THREADS] = page_key(c, p, mine);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint32_t p = (uint32_t)i * THREADS + threadIdx.x;
      if (i >= used) continue;
      if (p - c.lo < c.hi - c.lo) {
        low = min(low, lds.key[i][threadIdx.x]);
        high = max(high, lds.key[i][threadIdx.x]);
      } else if (p >= (uint32_t)times * kAtOnce) {  // not scored
        lds.key[i][threadIdx.x] = page_key(c, p, 0.f);
      }
    }
  } else {
    for (int i = 0; i < used; ++i) lds.key[i][threadIdx.x] = page_key(c, (uint32_t)i * THREADS + threadIdx.x, 0.f);
  }
  write_selection<THREADS, R>(s, c, lds, row, low, high, id, wave, lane, used);
}

// Rows of any length: the score is found digit by digit (8 bits at a time, from
// counts in LDS), the scores read again for each.
__global__ __launch_bounds__(kThreads) void select_long_kernel(Select s) {
  __shared__ uint32_t s_count[256];
  __shared__ uint32_t s_pick[2];
  __shared__ uint32_t s_sum[2][kWaves];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const uint32_t row = blockIdx.x;
  const Selection c = selection_of(s, row);
  if (threadIdx.x == 0) s.lengths_out[row] = c.len - (int)((c.held - c.left) << s.page_shift);
  const uint64_t at = (uint64_t)row * s.rows.max_pages;
  uint32_t key = 0, want = c.want;
  if (want) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      s_count[threadIdx.x] = 0;
      __syncthreads();
      for (uint32_t i = c.lo + threadIdx.x; i < c.hi; i += kThreads) {
        const uint32_t k = weight_key(s.scores[at + i]);
        if (shift == 24 || (k ^ key) >> (shift + 8) == 0) atomicAdd(&s_count[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (wave == 0) {  // lane l: digits 255 - 4 l down to 252 - 4 l
        uint32_t n[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += n[i] = s_count[255 - 4 * lane - i];
        uint32_t before = wave_scan(mine) - mine;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before < want && before + n[i] >= want) {
            s_pick[0] = 255u - 4u * lane - i;
            s_pick[1] = want - before;
          }
          before += n[i];
        }
      }
      __syncthreads();
      key |= s_pick[0] << shift;
      want = s_pick[1];
    }
  }
  uint32_t above_before = 0, equal_before = 0;
  for (uint32_t base = 0; base < c.held; base += kThreads) {
    const uint32_t i = base + threadIdx.x;
    const bool middle = c.full && i >= c.lo && i < c.hi;
    const uint32_t k = middle && want ? weight_key(s.scores[at + i]) : 0u;
    const bool above = i < c.held && (!middle || (want && k > key));
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
    a += lanes_below(ba, 0);
    q += lanes_below(be, 0);
    if (above || (equal && q < want)) {
      const uint32_t to = a + min(q, want);
      s.pages_out[(uint64_t)row * s.keep + to] = s.rows.pages[at + i];
      s.places_out[(uint64_t)row * s.keep + to] = (int32_t)i;
    }
  }
  fill_rest(s, row, c.left, kThreads);
}

// ---------------------------------------------------- a shared prefix ----

// A prefix under many query rows, where the arithmetic counts.  As attend_part, a
// workgroup takes one part of one unit and its waves take steps of 32 tokens in
// turn; but a unit is four groups of 16 query rows (two of wide heads), whose
// queries are in LDS, where all waves read them, and two waves share a SIMD, so
// that one's matrix instructions run beside the other's exponentials.
//
// An exponential is taken once, of the score plus the logarithm of the values'
// scale,
//     z_j = exp2(s_j + log2(vs_j) - M),
// so that the second product takes z as it is, with the codes; its largest is what
// M follows.  The softmax's sum needs exp2(s_j) alone: with L the logarithm of the
// part's largest scale a tile's sum of z times 2^L / vs is that in units of
// 2^(M - L).
// z goes into the product in fp16: at most 2^kTop, its largest at least 2^kStart
// (M is that far below the largest when it is set), and off by 2^-11 of itself or by
// 2^-25, half of fp16's smallest step.  That is 2^-32 of the largest z, so that
// with scales at most 2^kNear apart a weight is off by 2^-11 of itself or 2^-24 of
// the largest weight, whichever is more.  Outputs of bf16 have 8 bits.
// This is for these outputs, and for scales that are powers of two, as an append
// writes them, and no further apart: a part with others (pages of zeros have the
// smallest of all) and outputs of fp16 take attend_part's softmax and second product,
// 16 bits of any weight.
//
// 96 x 64 queries of 128 dims over 32,768 tokens x 8 heads, and own rows of 70 to 700
// tokens: calls back to back 125 us with 8 of joining, 0.83 PFLOP/s (a traced launch 130
// to 155), with the matrix cores busy for 36% of the time and the vector units for half
// of it.  A step of 64 x 32 scores is 64 matrix instructions (1043 cycles) and some 225
// others (about 1080); the prefix alone takes 115 us at 2.17 GHz, 2440 cycles for each of
// a SIMD's 102 steps: more than both one after the other, so that what its two waves
// overlap goes into waits.  (Own rows' workgroups before the prefix's, so that their
// loads run beside its arithmetic: 3 to 8 us more.)  The softmax's instructions cost a
// quarter of it; the exponentials alone, the loads and the order of the instructions
// nothing that shows.  With attend_part's softmax and product for every part, a step is
// 96 matrix instructions and more of the others: 169 us; 16 x 4 queries over 16,384
// tokens 24.8 and 25.8 us (the latter in fp16, which has no other way).
constexpr float kTop = 15.f, kStart = 7.f;
constexpr int kNear = 8;
constexpr int many_tiles(int dj) { return dj <= 2 ? 4 : 2; }  // groups of 16 query rows

__device__ __forceinline__ float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }

template <int DJ, int MT>
struct ManyLds {
  union {
    u32x4 q[MT][DJ][2][kWave];  // as the lanes of the matrix instructions take them
    float o[kWaves][16][64 + 4];
  };
  f32x2 ml[kWaves][MT * 16];
  struct {
    uint32_t high, low;
  } scales[kWaves];
};

// The steps of a wave, from `step` on.  NEAR: with z, the part's scales near each other.
template <int DJ, bool F16, bool NEAR>
__device__ __forceinline__ void many_steps(const Attention& a, const Plan& p, const ManyLds<DJ, many_tiles(DJ)>& lds, int step, int last,
                                           int lane, int scale_log, State<DJ, many_tiles(DJ)>& st) {
  constexpr int MT = many_tiles(DJ), ST = 2;
  if (step >= last) return;
  const float c_scale = fabsf(a.scale);
  u32x4 k[ST][DJ], v[ST][DJ];
  Where<ST> here = find_step<DJ, ST>(a, p, step, ids_of_step<ST>(a, p, step));
  Ids<ST> ids = ids_of_step<ST>(a, p, min(step + kWaves, last - 1));
  load_tiles<DJ, ST, false>(a.pool.k_codes, here, lane * 16, k);
  load_tiles<DJ, ST, false>(a.pool.v_codes, here, lane * 16, v);
  while (true) {
    const int next_step = step + kWaves;
    const bool more = next_step < last;
    const int byte = more ? lane * 16 : 0;
    arrive<ST>(here, ids);
    Where<ST> next = find_step<DJ, ST>(a, p, more ? next_step : step, ids);
    ids = ids_of_step<ST>(a, p, min(next_step + kWaves, last - 1));
    f32x4 s[MT][ST];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int t = 0; t < ST; ++t) s[mt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DJ; ++j)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        u32x4 kk[ST];
#pragma unroll
        for (int t = 0; t < ST; ++t) kk[t] = widen8<F16>(k[t][j][2 * half], k[t][j][2 * half + 1]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const u32x4 q = lds.q[mt][j][half][lane];
#pragma unroll
          for (int t = 0; t < ST; ++t) s[mt][t] = mfma<F16>(kk[t], q, s[mt][t]);
        }
      }
    load_tiles<DJ, ST, false>(a.pool.k_codes, next, byte, k);
    bool plain = (step + 1) * (kTile * ST) <= p.full;
    float c[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t) {
      plain = plain && here.ok[t];
      c[t] = here.ks[t] * c_scale;
    }
    int seen[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) seen[mt] = p.end;
    if constexpr (NEAR) {
      float lv[ST], back[ST];
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        plain = plain && here.ks[t] >= 0.f;  // keys of a scale below 0 turn the order
        // a hole's place has any scale, and its weights are 0
        const int e = here.ok[t] ? (int)(__builtin_bit_cast(uint32_t, here.vs[t]) >> 23) - 127 : scale_log;
        lv[t] = (float)e;
        back[t] = power2(scale_log - e);
      }
      if (!plain) {
#pragma unroll
        for (int t = 0; t < ST; ++t) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[mt][t] *= c[t];
          c[t] = 1.f;
        }
        mask_step<DJ, MT, ST>(p, step, lane, seen, here, s, v, st);
      }
      float top[MT];
      bool higher = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        top[mt] = -INFINITY;
#pragma unroll
        for (int t = 0; t < ST; ++t) {
          const float x = maximum(maximum(maximum(s[mt][t][0], s[mt][t][1]), s[mt][t][2]), s[mt][t][3]);
          top[mt] = maximum(top[mt], __builtin_fmaf(x, c[t], lv[t]));
        }
        higher = higher || top[mt] > st.m[mt] + kTop;
      }
      if (__ballot(higher)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float m = fmaxf(st.m[mt], query_max(top[mt]) - kStart);
          const float keep = exp2_fast(st.m[mt] - (m == -INFINITY ? 0.f : m));
          st.m[mt] = m;
          st.l[mt] *= keep;
#pragma unroll
          for (int i = 0; i < 4 * DJ; ++i) st.o[mt][i] *= keep;
        }
      }
      u32x4 z16[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float base = st.m[mt] == -INFINITY ? 0.f : st.m[mt];
#pragma unroll
        for (int t = 0; t < ST; ++t) {
          const float b = lv[t] - base;
          float z[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) z[r] = exp2_fast(__builtin_fmaf(s[mt][t][r], c[t], b));
          st.l[mt] = __builtin_fmaf((z[0] + z[1]) + (z[2] + z[3]), back[t], st.l[mt]);
          const f16x2 h0 = {(_Float16)z[0], (_Float16)z[1]}, h1 = {(_Float16)z[2], (_Float16)z[3]};
          z16[mt][2 * t] = __builtin_bit_cast(uint32_t, h0);
          z16[mt][2 * t + 1] = __builtin_bit_cast(uint32_t, h1);
        }
      }
#pragma unroll
      for (int h = 0; h < DJ; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const u32x4 vv = widen8<true>(v[0][h][x], v[1][h][x]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) st.o[mt][h * 4 + x] = mfma<true>(vv, z16[mt], st.o[mt][h * 4 + x]);
        }
    } else {
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[mt][t] *= c[t];
      if (!plain) mask_step<DJ, MT, ST>(p, step, lane, seen, here, s, v, st);
      Probs<MT, ST> pr;
      softmax<DJ, MT, ST, false>(a, p, step, lane, here, s, nullptr, nullptr, st, pr);
      gather_values<DJ, MT, ST>(v, pr, st);
    }
    load_tiles<DJ, ST, false>(a.pool.v_codes, next, byte, v);
    if (!more) return;
    here = next;
    step = next_step;
  }
}

template <int DJ, bool F16>
__device__ __forceinline__ void attend_many(const Attention& a, uint32_t block) {
  constexpr int D = 64 * DJ, MT = many_tiles(DJ), ST = 2;
  __shared__ __attribute__((aligned(16))) ManyLds<DJ, MT> lds;
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const Part part = part_of_shared(a, block);
  const Plan p = plan_shared<MT, ST>(a, part);
  const int first = part.index * p.part_steps, last = min(first + p.part_steps, p.steps);
  if (first >= last) return;

  // the queries, negated where the scale is below 0, so that the largest product gives
  // the largest score
  const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
  for (int i = wave; i < MT * DJ; i += kWaves) {
    const int mt = i / DJ, j = i % DJ, m = p.m0 + mt * 16 + lane % 16;
    u32x4 x[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (m < a.m_rows) {
      const uint16_t* src = row_of_all(a.q, a, p, m) + 64 * j + 16 * (lane / 16);
      x[0] = load8(src, a.q.wide);
      x[1] = load8(src + 8, a.q.wide);
    }
    lds.q[mt][j][0][lane] = x[0] ^ sign;
    lds.q[mt][j][1][lane] = x[1] ^ sign;
  }
  bool near = false;
  int scale_log = 0;  // L
  if constexpr (!F16) {
    // the largest and the smallest scale, as bits; all ones: one of them is no power of two
    const int tiles_of_page = 1 << a.pool.tile_shift;
    const int from = first * ST / tiles_of_page, to = (min(last * ST, p.tiles) + tiles_of_page - 1) / tiles_of_page;
    const int32_t* pages = a.rows.pages + (uint64_t)p.row * a.rows.max_pages;
    uint32_t high = 0, low = ~0u;
    for (int i = from + (int)threadIdx.x; i < to; i += kThreads) {
      const uint32_t id = (uint32_t)pages[i];
      if (id >= a.pool.n_pages) continue;
      const uint32_t x = __builtin_bit_cast(uint32_t, a.pool.v_scales[id]);
      high = max(high, (x & 0x807FFFFFu) || x == 0 || x >= 0x7F800000u ? ~0u : x);
      low = min(low, x);
    }
    high = wave_max(high);
    low = ~wave_max(~low);
    if (lane == 0) lds.scales[wave] = {high, low};
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      high = max(high, lds.scales[w].high);
      low = min(low, lds.scales[w].low);
    }
    near = uniform(high != ~0u && (int)(high >> 23) - (int)(low >> 23) <= kNear);
    scale_log = uniform(near && high ? (int)(high >> 23) - 127 : 0);
  } else {
    __syncthreads();
  }

  State<DJ, MT> st;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    st.m[mt] = -INFINITY;
    st.l[mt] = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * DJ; ++i) st.o[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if constexpr (!F16) {
    if (near) many_steps<DJ, F16, true>(a, p, lds, first + wave, last, lane, scale_log, st);
  }
  if (!near) many_steps<DJ, F16, false>(a, p, lds, first + wave, last, lane, scale_log, st);
  const float lift = near ? kTop : 0.f;  // of the statistics
  // the waves' sums together, a group of 16 query rows and 64 dims at a time; left with
  // the statistics that attend_part leaves, of the scores alone
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    st.l[mt] = pair_sum16(st.l[mt], st.l[mt]);
    st.l[mt] = pair_sum32(st.l[mt], st.l[mt]);
  }
  if (lane < 16) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) lds.ml[wave][mt * 16 + lane] = f32x2{st.m[mt], st.l[mt]};
  }
  __syncthreads();
  const int n = threadIdx.x / 16, d4 = threadIdx.x % 16 * 4;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m_local = mt * 16 + n, m = p.m0 + m_local;
    float top = -INFINITY, total = 0.f, f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds.ml[w][m_local][0]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = exp2_fast(lds.ml[w][m_local][0] - base - lift);
      total += lds.ml[w][m_local][1] * f[w];
    }
    const uint64_t slot = (uint64_t)part.slot * a.unit_rows.d + m_local;
    const bool there = m_local < (int)a.unit_rows.d && m < a.m_rows;
    if (d4 == 0 && there) a.ws_ml[slot] = f32x2{top + lift - (float)scale_log, total};
    const float unit = power2(scale_log);
#pragma unroll
    for (int h = 0; h < DJ; ++h) {
      __syncthreads();
#pragma unroll
      for (int x = 0; x < 4; ++x)
        *(f32x4*)&lds.o[wave][lane % 16][16 * x + 4 * (lane / 16)] = st.o[mt][h * 4 + x];
      __syncthreads();
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) o += *(const f32x4*)&lds.o[w][n][d4] * f[w];
      if (there) *(f32x4*)(a.ws_o + slot * D + 64 * h + d4) = o * unit;
    }
  }
}

// With few query rows bound by HBM: 16 x 32 rows of 256 to 512 tokens behind 4096 (86 MB)
// 17.2 us; as two launches 24.
// The first workgroups take the prefix (KIND 1 and 2: one unit of as many groups of
// 16 query rows to a head; 0: many), the others the rows' own tokens, MT groups of
// query rows to a unit.  One launch: the rows' workgroups take the places of the
// prefix's as these end.
template <int DJ, bool F16, int KIND, int MT, bool ONCE>
__global__ __launch_bounds__(kThreads, workgroups_per_unit(DJ, KIND > MT ? KIND : MT)) void shared_kernel(Attention a, Attention b,
                                                                                       uint32_t prefix_blocks) {
  if (blockIdx.x >= prefix_blocks) return attend_part<DJ, F16, MT, ONCE, Sums::kLeft>(b, blockIdx.x - prefix_blocks);
  if constexpr (KIND == 0)
    attend_many<DJ, F16>(a, blockIdx.x);
  else
    attend_part<DJ, F16, KIND, true, Sums::kShared>(a, blockIdx.x);
}

// Joins the sums over the prefix (a) with those over a row's own tokens (b), a
// query row to each wave.  3.5 to 8 us: its loads wait for each other.
template <int DJ, bool F16, int MT>
__global__ __launch_bounds__(kThreads) void join_shared_kernel(Attention a, Attention b, Divisor rows_of_head,
                                                               uint32_t n_rows, int shared_step_tiles) {
  constexpr int D = 64 * DJ;
  constexpr int ST = step_tiles(DJ, MT);
  __shared__ float s_f[kWaves][2 * kMaxParts];
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const uint32_t x = blockIdx.x * kWaves + wave;
  if (x >= n_rows) return;
  const uint32_t row = quotient(x, rows_of_head);
  const int m = (int)(x - row * rows_of_head.d);
  const uint32_t group = quotient((uint32_t)m, b.unit_rows);
  const int own_local = m - (int)(group * b.unit_rows.d);
  const Part t = parts_of_unit(b, row, (int)group);
  const Plan p = plan_unit<MT, ST>(b, t);
  const bool any = seen_by(b, p, m) > 0;
  // the prefix's units are of the query rows of all sequences
  const uint32_t all = p.seq * rows_of_head.d + (uint32_t)m;
  const uint32_t unit = quotient(all, a.unit_rows);
  const int local = (int)(all - unit * a.unit_rows.d);
  const uint32_t first = (p.head * a.m_groups.d + unit) * a.shared_parts;
  const int tiles = (row_length(a.rows, p.head) + kTile - 1) / kTile;
  const int steps = (tiles + shared_step_tiles - 1) / shared_step_tiles;
  const int part_steps = max((steps + (int)a.shared_parts - 1) / (int)a.shared_parts, 1);
  const int shared = any ? (steps + part_steps - 1) / part_steps : 0, parts = any ? shared + p.parts : 0;
  auto slot = [&](int n) {
    return n < shared ? (uint64_t)(first + n) * a.unit_rows.d + local
                      : ((uint64_t)t.first + (uint64_t)(n - shared) * b.m_groups.d) * b.unit_rows.d + own_local;
  };
  auto part = [&](int n) { return n < shared ? a.ws_ml[slot(n)] : b.ws_ml[slot(n)]; };
  float top = -INFINITY, total = 0.f;
  for (int n = lane; n < parts; n += kWave) top = fmaxf(top, part(n)[0]);
  top = wave_max(top);
  const float base = top == -INFINITY ? 0.f : top;
  for (int n = lane; n < parts; n += kWave) {
    const f32x2 ml = part(n);
    const float f = exp2_fast(ml[0] - base);
    s_f[wave][n] = f;
    total += f * ml[1];
  }
  total = wave_sum(total);
  const float share = total == 0.f ? 0.f : 1.f / total;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  float o[DJ];  // dims 64 j + lane
#pragma unroll
  for (int j = 0; j < DJ; ++j) o[j] = 0.f;
#pragma unroll 4
  for (int n = 0; n < parts; ++n) {
    const float* sums = (n < shared ? a.ws_o : b.ws_o) + slot(n) * D;
    const float f = s_f[wave][n];
#pragma unroll
    for (int j = 0; j < DJ; ++j) o[j] += sums[64 * j + lane] * f;
  }
  uint16_t* dst = row_of(b.out, b, p, m);
#pragma unroll
  for (int j = 0; j < DJ; ++j) dst[64 * j + lane] = to_half<F16>(o[j] * share);
}

// ------------------------------------------------------------------ host ----

int check_outlines(const ibp_kv_outlines* o, const ibp_kv_cache* c) {
  if (!o) return IBP_ERR_INVALID_ARGUMENT;
  if (c->n_pages == 0) return IBP_OK;
  if (!o->codes || !o->scales) return IBP_ERR_INVALID_ARGUMENT;
  return aligned(o->codes, 16) && aligned(o->scales, 4) ? IBP_OK : IBP_ERR_LAYOUT;
}

// Pages of a row that n_new tokens may be in.
uint64_t touched_pages(uint64_t n_new, uint64_t page_tokens, uint64_t max_pages) {
  return std::min<uint64_t>((n_new + page_tokens - 2) / page_tokens + 1, max_pages);
}

template <int DJ, bool F16, Pairs PAIRS>
void launch_append_rotated(const Pool& pool, const Rows& rows, const Strided& k, const Strided& v, uint32_t per_row,
                           uint32_t tasks, const Angles& t, const ibp_kv_outlines& o, const Queries& q, hipStream_t st) {
  const uint32_t per_group = kWaves >> pool.tile_shift;
  const uint32_t append = (tasks + per_group - 1) / per_group;
  const uint32_t turn = (q.n_items + kThreads - 1) / kThreads;
  hipLaunchKernelGGL((append_rotated_kernel<DJ, F16, PAIRS>), dim3(append + turn), dim3(kThreads), 0, st, pool, rows, k, v,
                     make_divisor(per_row), tasks, Turn<PAIRS>{t, o}, q, append);
}

template <int DJ, bool F16>
void launch_append_pairs(const Pool& pool, const Rows& rows, const Strided& k, const Strided& v, uint32_t per_row,
                         uint32_t tasks, const Angles& t, bool interleaved, const ibp_kv_outlines& o, const Queries& q,
                         hipStream_t st) {
  if (interleaved) return launch_append_rotated<DJ, F16, Pairs::kNeighbour>(pool, rows, k, v, per_row, tasks, t, o, q, st);
  if constexpr (DJ % 2 == 0)
    if (t.half == 32 * DJ) return launch_append_rotated<DJ, F16, Pairs::kLane>(pool, rows, k, v, per_row, tasks, t, o, q, st);
  launch_append_rotated<DJ, F16, Pairs::kFar>(pool, rows, k, v, per_row, tasks, t, o, q, st);
}

// Waves to a compute unit that the pages of an outline call are spread over: two
// contexts of 131k and 91k tokens x 8 heads (257 MB) take 54.0 us so, 53.7 with 12, 63.5
// with 8, 57.0 with 24 and 59.9 with 32, since each begins with a chain of three loads.
constexpr int kOutlineWaves = 16;

int launch_outline(const ibp_kv_cache* cache, const ibp_kv_outlines* o, const Rows& rows, uint64_t n_rows,
                   uint64_t n_new, int cus, hipStream_t st) {
  const Pool pool = make_pool(cache);
  const int dj = (int)cache->head_dim / 64;
  const uint64_t per_row = touched_pages(n_new, cache->page_tokens, rows.max_pages);
  const uint64_t waves = (uint64_t)kOutlineWaves * cus;
  const uint64_t wave_pages = std::min<uint64_t>(std::max<uint64_t>((n_rows * per_row + waves - 1) / waves, 1), kWave);
  const uint64_t chunks = (per_row + wave_pages - 1) / wave_pages, tasks = n_rows * chunks;
  const dim3 grid((uint32_t)((tasks + kWaves - 1) / kWaves)), threads(kThreads);
  const Divisor d = make_divisor((uint32_t)chunks);
  const uint32_t n = (uint32_t)tasks;
  switch (dj) {
    case 1: hipLaunchKernelGGL(outline_kernel<1>, grid, threads, 0, st, pool, rows, *o, d, n); break;
    case 2: hipLaunchKernelGGL(outline_kernel<2>, grid, threads, 0, st, pool, rows, *o, d, n); break;
    case 3: hipLaunchKernelGGL(outline_kernel<3>, grid, threads, 0, st, pool, rows, *o, d, n); break;
    default: hipLaunchKernelGGL(outline_kernel<4>, grid, threads, 0, st, pool, rows, *o, d, n); break;
  }
  return launched();
}

// Whether the tasks of a wave for each touched page, or of a workgroup of `per_group`,
// are more than a launch (and a Divisor's numbers) can have.
bool too_many(uint64_t n_rows, uint64_t per_row, uint64_t per_group) {
  return per_row && (per_row > 0x7FFFFFFFull / n_rows || n_rows * per_row / per_group >= max_grid(kThreads));
}

// Rows that are chosen from as they are scored, and the scores of the others.
constexpr uint64_t kShortPages = 1024;
uint64_t select_bytes(uint64_t n_rows, uint64_t max_pages) { return max_pages <= kShortPages ? 0 : n_rows * max_pages * 4; }

template <int DJ, bool F16>
void launch_select(const Select& s, uint64_t n_rows, uint64_t max_pages, hipStream_t st) {
  const dim3 rows((uint32_t)n_rows);
  // Rows of few pages are scored and chosen from in one launch, which needs no workspace:
  // 8 rows of 251 pages 8 us, 11 to 12 as two; 16 x 32 rows of up to 256 pages 12 us, 20 as
  // two; 64 x 8 rows of 1000 pages 31 us, 34 as two.  Few long rows pay for it, since a
  // workgroup scores 256 pages at a time (128 of wide heads): 8 rows of 512 pages of 64, 128
  // and 256 dims take 8.6, 10.4 and 14.4 us, of 1000 pages 12.1, 15.5 and 22; as two launches
  // each of these takes 10.5 to 12.  (With 1024 threads and all pages at once the 16 x 32
  // rows take 19 us, 72 rows of 50 to 500 pages the same 10 us.)
  if (max_pages <= kShortPages) {
    hipLaunchKernelGGL((select_short_kernel<DJ, F16, 256, 4>), rows, dim3(256), 0, st, s);
    return;
  }
  if (s.keep > s.sink + s.recent && max_pages > s.keep)  // else there is nothing to choose
    hipLaunchKernelGGL((score_kernel<DJ, F16>), dim3((uint32_t)n_rows * s.chunks.d), dim3(kThreads), 0, st, s);
  if (max_pages <= 4096)
    hipLaunchKernelGGL((select_kernel<1024, 4>), rows, dim3(1024), 0, st, s);
  else if (max_pages <= 16384)
    hipLaunchKernelGGL((select_kernel<1024, 16>), rows, dim3(1024), 0, st, s);
  else
    hipLaunchKernelGGL(select_long_kernel, rows, dim3(kThreads), 0, st, s);
}

// The prefix of a call, as units of the query rows of all sequences, each cut into
// `parts`; and where the sums are in the workspace.
struct SharedShape {
  Shape own;
  int mt, step;
  bool many;
  int32_t m_rows, m_groups, unit_rows;
  uint32_t n_units, parts, n_rows, join_blocks;
  uint64_t own_o, ml, own_ml, own_of, bytes;
};

bool make_shared_shape(uint64_t n_seqs, uint64_t heads, uint64_t prefix_pages, uint64_t own_pages, uint32_t page_tokens,
                       uint32_t head_dim, uint64_t group, uint64_t n_new, int cus, SharedShape* s) {
  if (!make_shape(n_seqs * heads, own_pages, page_tokens, head_dim, group, n_new, false, cus, &s->own)) return false;
  const uint64_t own_rows = group * n_new;
  if (n_seqs && own_rows > 0x7FFFFFFFull / n_seqs) return false;
  const uint64_t m = own_rows * n_seqs;
  if (m && heads > 0x7FFFFFFFull / m) return false;
  const int dj = (int)head_dim / 64;
  s->m_rows = (int32_t)m;
  // 32 rows a head as one unit of attend_part 25 us, as half of one of attend_many 32 (32,768
  // tokens x 8 heads); 768 rows as units of 32 279 us, of 64 127.
  s->many = m > 32;
  s->mt = m <= 16 ? 1 : m <= 32 ? 2 : many_tiles(dj);
  s->step = s->many ? 2 : step_tiles(dj, s->mt);
  const uint64_t per_unit = 16ull * s->mt;
  s->m_groups = (int32_t)((m + per_unit - 1) / per_unit);
  s->unit_rows = (int32_t)std::min<uint64_t>(m, per_unit);
  const uint64_t units = heads * s->m_groups;
  s->n_units = (uint32_t)units;
  const uint64_t steps = (prefix_pages * page_tokens / kTile + s->step - 1) / s->step;
  const uint64_t slots = (uint64_t)workgroups_per_unit(dj, s->many ? s->own.mt : s->mt) * cus / (s->many ? 1 : 2);
  // Steps of a wave at least: with four a part's sums are worth their place in the join.  40
  // rows x 2 heads over 65,536 tokens 55 us with one, 36 with four, 31 with eight; x 8 heads
  // over 8192 28, 19 and 22; 64 rows x 8 over 2048 15.8, 17.0 and 21.9.
  const uint64_t part = (s->many ? 4 : 1) * kWaves;
  s->parts = 1;
  if (units)
    s->parts = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>({slots / units, (steps + part - 1) / part, (uint64_t)kMaxParts}));
  if (units * s->parts + s->own.n_parts > max_grid(kThreads)) return false;
  const uint64_t shared_slots = units * s->parts * s->unit_rows, own_slots = (uint64_t)s->own.n_parts * s->own.unit_rows;
  s->own_o = shared_slots * head_dim * 4;
  s->ml = s->own_o + own_slots * head_dim * 4;
  s->own_ml = s->ml + shared_slots * 8;
  s->own_of = s->own_ml + own_slots * 8;
  s->bytes = s->own_of + (s->own.n_parts != s->own.n_units ? (uint64_t)s->own.n_units * 8 : 0);
  s->n_rows = (uint32_t)(heads * m);
  s->join_blocks = (s->n_rows + kWaves - 1) / kWaves;
  return s->join_blocks <= max_grid(kThreads);
}

template <int DJ, bool F16>
void launch_shared(const Attention& a, const Attention& b, const SharedShape& s, const Divisor& rows_of_head,
                   hipStream_t st) {
  const uint32_t prefix = s.n_units * s.parts;
  const dim3 grid(prefix + s.own.n_parts), join(s.join_blocks), threads(kThreads);
  const bool several = b.m_groups.d > 1;  // units of own query rows; those of the prefix are many then
  if (s.own.mt == 1) {
    if (s.many)
      hipLaunchKernelGGL((shared_kernel<DJ, F16, 0, 1, true>), grid, threads, 0, st, a, b, prefix);
    else if (s.mt == 1)
      hipLaunchKernelGGL((shared_kernel<DJ, F16, 1, 1, true>), grid, threads, 0, st, a, b, prefix);
    else
      hipLaunchKernelGGL((shared_kernel<DJ, F16, 2, 1, true>), grid, threads, 0, st, a, b, prefix);
    hipLaunchKernelGGL((join_shared_kernel<DJ, F16, 1>), join, threads, 0, st, a, b, rows_of_head, s.n_rows, s.step);
  } else {
    if (several)
      hipLaunchKernelGGL((shared_kernel<DJ, F16, 0, kQueryTiles, false>), grid, threads, 0, st, a, b, prefix);
    else if (s.many)
      hipLaunchKernelGGL((shared_kernel<DJ, F16, 0, kQueryTiles, true>), grid, threads, 0, st, a, b, prefix);
    else
      hipLaunchKernelGGL((shared_kernel<DJ, F16, 2, kQueryTiles, true>), grid, threads, 0, st, a, b, prefix);
    hipLaunchKernelGGL((join_shared_kernel<DJ, F16, kQueryTiles>), join, threads, 0, st, a, b, rows_of_head, s.n_rows, s.step);
  }
}

// The prefix's table, of one sequence and as many heads.
int check_prefix(const ibp_kv_table* prefix, const ibp_kv_table* table, uint64_t page_tokens) {
  uint64_t heads = 0;
  if (!prefix || prefix->n_seqs != 1 || prefix->kv_heads != table->kv_heads) return IBP_ERR_INVALID_ARGUMENT;
  return check_table(prefix, page_tokens, &heads);
}

}  // namespace

extern "C" {

int ibp_kv_long_last_hip_error(void) { return g_last_hip; }

int ibp_kv_append_rotated(const ibp_kv_cache* cache, const ibp_kv_table* table, uint32_t dtype, uint64_t n_new,
                          const ibp_kv_tensor* k, const ibp_kv_tensor* v, const int32_t* counts,
                          const ibp_kv_rotation* rotation, uint64_t q_heads, const ibp_kv_tensor* q,
                          const ibp_kv_tensor* q_out, const ibp_kv_outlines* outlines, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (dtype > IBP_KV_FP16) return IBP_ERR_UNSUPPORTED;
  uint64_t n_rows = 0;
  rc = check_table(table, cache->page_tokens, &n_rows);
  if (rc) return rc;
  if (!rotation || !q != !q_out) return IBP_ERR_INVALID_ARGUMENT;
  if (rotation->rotary_dim == 0 || rotation->rotary_dim % 16 || rotation->rotary_dim > cache->head_dim || rotation->interleaved > 1)
    return IBP_ERR_UNSUPPORTED;
  if (rotation->n_positions && (!rotation->cos || !rotation->sin)) return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(rotation->cos, 16) || !aligned(rotation->sin, 16) || !aligned(rotation->positions, 4)) return IBP_ERR_LAYOUT;
  if (outlines && (rc = check_outlines(outlines, cache))) return rc;
  if (n_rows == 0 || n_new == 0) return IBP_OK;
  if (n_new > 0x7FFFFFFFull) return IBP_ERR_INVALID_ARGUMENT;
  if ((rc = check_tensor(k)) || (rc = check_tensor(v))) return rc;
  if (!aligned(counts, 4)) return IBP_ERR_LAYOUT;
  const bool pages = table->max_pages != 0 && cache->n_pages != 0;
  const uint64_t per_row = pages ? touched_pages(n_new, cache->page_tokens, table->max_pages) : 0;
  if (too_many(n_rows, per_row, (uint64_t)kWaves * kTile / cache->page_tokens)) return IBP_ERR_INVALID_ARGUMENT;
  Queries queries{};
  if (q) {
    if (q_heads == 0 || q_heads % table->kv_heads) return IBP_ERR_INVALID_ARGUMENT;
    if ((rc = check_tensor(q)) || (rc = check_tensor(q_out))) return rc;
    if (rows_overlap(table->n_seqs, q_out->seq_stride, cache->head_dim) ||
        rows_overlap(n_new, q_out->token_stride, cache->head_dim) ||
        rows_overlap(q_heads, q_out->head_stride, cache->head_dim))
      return IBP_ERR_INVALID_ARGUMENT;
    // items, and with the pages' workgroups the grid
    const uint64_t most = 0x7FFFFFFFull / (cache->head_dim / 16) / table->n_seqs;
    if (n_new > most || q_heads > most / n_new) return IBP_ERR_INVALID_ARGUMENT;
    const uint64_t runs = (q_heads + kHeadRun - 1) / kHeadRun;
    queries.n_items = (uint32_t)(table->n_seqs * n_new * runs * (cache->head_dim / 16));
    queries.runs = make_divisor((uint32_t)runs);
    queries.q_heads = (uint32_t)q_heads;
    queries.q = make_strided(q);
    queries.out = make_strided(q_out);
    queries.group = make_divisor((uint32_t)(q_heads / table->kv_heads));
    queries.n_new = make_divisor((uint32_t)n_new);
  }
  const uint64_t tasks = n_rows * per_row;
  if (tasks / (kWaves * kTile / cache->page_tokens) + queries.n_items / kThreads + 2 > max_grid(kThreads))
    return IBP_ERR_INVALID_ARGUMENT;
  if (tasks == 0 && queries.n_items == 0) return IBP_OK;
  rc = pending_hip_error();
  if (rc) return rc;
  const Pool pool = make_pool(cache);
  const Rows rows = make_rows(table, cache->page_tokens, n_new, counts);
  const Strided ks = make_strided(k), vs = make_strided(v);
  Angles t;
  t.cos = rotation->cos;
  t.sin = rotation->sin;
  t.positions = rotation->positions;
  t.n_positions = (uint32_t)std::min<uint64_t>(rotation->n_positions, 1ull << 31);
  t.half = (int32_t)rotation->rotary_dim / 2;
  hipStream_t st = (hipStream_t)stream;
  const uint32_t pr = (uint32_t)std::max<uint64_t>(per_row, 1), n = (uint32_t)tasks;
  const bool il = rotation->interleaved != 0;
  const ibp_kv_outlines o = outlines ? *outlines : ibp_kv_outlines{nullptr, nullptr};
  switch (cache->head_dim / 64 * 2 + dtype) {
    case 2: launch_append_pairs<1, false>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
    case 3: launch_append_pairs<1, true>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
    case 4: launch_append_pairs<2, false>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
    case 5: launch_append_pairs<2, true>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
    case 6: launch_append_pairs<3, false>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
    case 7: launch_append_pairs<3, true>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
    case 8: launch_append_pairs<4, false>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
    default: launch_append_pairs<4, true>(pool, rows, ks, vs, pr, n, t, il, o, queries, st); break;
  }
  return launched();
}

int ibp_kv_outline(const ibp_kv_cache* cache, const ibp_kv_outlines* outlines, const ibp_kv_table* table,
                   uint64_t n_new, const int32_t* counts, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  uint64_t n_rows = 0;
  rc = check_table(table, cache->page_tokens, &n_rows);
  if (rc || (rc = check_outlines(outlines, cache))) return rc;
  if (n_rows == 0 || n_new == 0 || table->max_pages == 0 || cache->n_pages == 0) return IBP_OK;
  if (n_new > 0x7FFFFFFFull) return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(counts, 4)) return IBP_ERR_LAYOUT;
  if (too_many(n_rows, touched_pages(n_new, cache->page_tokens, table->max_pages), kWaves)) return IBP_ERR_INVALID_ARGUMENT;
  rc = pending_hip_error();
  if (rc) return rc;
  return launch_outline(cache, outlines, make_rows(table, cache->page_tokens, n_new, counts), n_rows, n_new, compute_units(),
                        (hipStream_t)stream);
}

uint64_t ibp_kv_select_workspace_bytes(const ibp_kv_cache* cache, const ibp_kv_table* table) {
  uint64_t n_rows = 0;
  if (check_cache(cache) || !table || check_table(table, cache->page_tokens, &n_rows)) return 0;
  return select_bytes(n_rows, table->max_pages);
}

int ibp_kv_select(const ibp_kv_cache* cache, const ibp_kv_outlines* outlines, const ibp_kv_table* table,
                  uint32_t dtype, uint64_t q_heads, uint64_t n_new, const ibp_kv_tensor* q, const int32_t* counts,
                  uint64_t keep_pages, uint64_t sink_pages, uint64_t recent_pages, int32_t* pages_out,
                  int32_t* lengths_out, int32_t* places_out, void* workspace, uint64_t workspace_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (dtype > IBP_KV_FP16) return IBP_ERR_UNSUPPORTED;
  const uint64_t pt = cache->page_tokens;
  uint64_t n_rows = 0;
  rc = check_table(table, pt, &n_rows);
  if (rc || (rc = check_outlines(outlines, cache))) return rc;
  if (recent_pages == 0 || sink_pages > keep_pages || recent_pages > keep_pages - sink_pages || keep_pages > 0x7FFFFFFFull / pt)
    return IBP_ERR_INVALID_ARGUMENT;
  if (n_new > 0x7FFFFFFFull || recent_pages < (n_new ? (n_new + pt - 2) / pt + 1 : 1)) return IBP_ERR_INVALID_ARGUMENT;
  if (n_rows == 0) return IBP_OK;
  if (q_heads == 0 || q_heads % table->kv_heads) return IBP_ERR_INVALID_ARGUMENT;
  if (n_new && (rc = check_tensor(q))) return rc;
  if (!pages_out || !lengths_out || !places_out) return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(counts, 4) || !aligned(pages_out, 4) || !aligned(lengths_out, 4) || !aligned(places_out, 4) || !aligned(workspace, 16))
    return IBP_ERR_LAYOUT;
  const uint64_t group = q_heads / table->kv_heads;
  if (n_new && group > (1ull << 24) / n_new) return IBP_ERR_INVALID_ARGUMENT;
  const uint64_t table_bytes = n_rows * table->max_pages * 4, bytes = select_bytes(n_rows, table->max_pages);
  if (bytes && (!workspace || workspace_bytes < bytes)) return IBP_ERR_INVALID_ARGUMENT;
  if (keep_pages > (1ull << 60) / n_rows) return IBP_ERR_INVALID_ARGUMENT;
  const uint64_t kept = n_rows * keep_pages * 4;
  const void* in[3] = {table->pages, table->lengths, workspace};
  void* outs[3] = {pages_out, places_out, lengths_out};
  const uint64_t in_size[3] = {table_bytes, n_rows * 4, bytes}, out_size[3] = {kept, kept, n_rows * 4};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3; ++j)
      if (overlap(in[i], in_size[i], outs[j], out_size[j]) || (i < j && overlap(outs[i], out_size[i], outs[j], out_size[j])))
        return IBP_ERR_INVALID_ARGUMENT;
  const int dj = (int)cache->head_dim / 64;
  const uint64_t at_once = (uint64_t)score_pages(dj, kThreads), chunks = (table->max_pages + at_once - 1) / at_once;
  if (n_rows > max_grid(1024) || chunks > max_grid(kThreads) / n_rows) return IBP_ERR_INVALID_ARGUMENT;
  rc = pending_hip_error();
  if (rc) return rc;
  Select s{};
  s.rows = make_rows(table, (uint32_t)pt, n_new, counts);
  s.n_pages = (uint32_t)std::min<uint64_t>(cache->n_pages, 1ull << 31);
  s.codes = outlines->codes;
  s.outline_scales = outlines->scales;
  if (n_new) s.q = make_strided(q);
  s.group = make_divisor((uint32_t)group);
  s.m_rows = (int32_t)(group * n_new);
  s.scores = (float*)workspace;
  s.chunks = make_divisor((uint32_t)std::max<uint64_t>(chunks, 1));
  s.page_shift = pt == 16 ? 4 : pt == 32 ? 5 : 6;
  s.keep = (uint32_t)keep_pages;
  s.sink = (uint32_t)sink_pages;
  s.recent = (uint32_t)recent_pages;
  s.pages_out = pages_out;
  s.lengths_out = lengths_out;
  s.places_out = places_out;
  hipStream_t st = (hipStream_t)stream;
  switch (dj * 2 + dtype) {
    case 2: launch_select<1, false>(s, n_rows, table->max_pages, st); break;
    case 3: launch_select<1, true>(s, n_rows, table->max_pages, st); break;
    case 4: launch_select<2, false>(s, n_rows, table->max_pages, st); break;
    case 5: launch_select<2, true>(s, n_rows, table->max_pages, st); break;
    case 6: launch_select<3, false>(s, n_rows, table->max_pages, st); break;
    case 7: launch_select<3, true>(s, n_rows, table->max_pages, st); break;
    case 8: launch_select<4, false>(s, n_rows, table->max_pages, st); break;
    default: launch_select<4, true>(s, n_rows, table->max_pages, st); break;
  }
  return launched();
}

uint64_t ibp_kv_attention_shared_workspace_bytes(const ibp_kv_cache* cache, const ibp_kv_table* prefix,
                                                 const ibp_kv_table* table, uint64_t q_heads, uint64_t n_new) {
  uint64_t n_rows = 0;
  if (check_cache(cache) || check_table(table, cache->page_tokens, &n_rows) || check_prefix(prefix, table, cache->page_tokens)) return 0;
  if (n_rows == 0 || q_heads == 0 || q_heads % table->kv_heads || n_new == 0) return 0;
  SharedShape s;
  if (!make_shared_shape(table->n_seqs, table->kv_heads, prefix->max_pages, table->max_pages, cache->page_tokens,
                         cache->head_dim, q_heads / table->kv_heads, n_new, compute_units(), &s))
    return 0;
  return s.bytes;
}

int ibp_kv_attention_shared(const ibp_kv_cache* cache, const ibp_kv_table* prefix, const ibp_kv_table* table,
                            uint32_t dtype, uint64_t q_heads, uint64_t n_new, const ibp_kv_tensor* q,
                            const ibp_kv_tensor* out, const int32_t* counts, float scale, void* workspace,
                            uint64_t workspace_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (dtype > IBP_KV_FP16) return IBP_ERR_UNSUPPORTED;
  uint64_t n_rows = 0;
  rc = check_table(table, cache->page_tokens, &n_rows);
  if (rc || (rc = check_prefix(prefix, table, cache->page_tokens))) return rc;
  if (n_rows == 0) return IBP_OK;
  if (q_heads == 0 || q_heads % table->kv_heads || !std::isfinite(scale_log2(scale))) return IBP_ERR_INVALID_ARGUMENT;
  if (n_new == 0) return IBP_OK;
  if ((rc = check_tensor(q)) || (rc = check_tensor(out))) return rc;
  if (rows_overlap(table->n_seqs, out->seq_stride, cache->head_dim) ||
      rows_overlap(n_new, out->token_stride, cache->head_dim) ||
      rows_overlap(q_heads, out->head_stride, cache->head_dim))
    return IBP_ERR_INVALID_ARGUMENT;
  if (!aligned(counts, 4) || !aligned(workspace, 16)) return IBP_ERR_LAYOUT;
  const uint64_t group = q_heads / table->kv_heads;
  SharedShape s;
  if (!make_shared_shape(table->n_seqs, table->kv_heads, prefix->max_pages, table->max_pages, cache->page_tokens,
                         cache->head_dim, group, n_new, compute_units(), &s))
    return IBP_ERR_INVALID_ARGUMENT;
  if (s.bytes && (!workspace || workspace_bytes < s.bytes)) return IBP_ERR_INVALID_ARGUMENT;
  rc = pending_hip_error();
  if (rc) return rc;
  Attention a{}, b{};
  a.pool = b.pool = make_pool(cache);
  a.rows = make_rows(prefix, cache->page_tokens, n_new, nullptr);
  b.rows = make_rows(table, cache->page_tokens, n_new, counts);
  if (cache->n_pages == 0) a.rows.capacity = b.rows.capacity = 0;  // holes only: nothing to see, and no page to read
  a.q = b.q = make_strided(q);
  a.out = b.out = make_strided(out);
  a.scale = b.scale = scale_log2(scale);
  a.group = b.group = make_divisor((uint32_t)group);
  a.n_new = b.n_new = make_divisor((uint32_t)n_new);
  char* ws = (char*)workspace;
  a.ws_o = (float*)ws;
  b.ws_o = (float*)(ws + s.own_o);
  a.ws_ml = (f32x2*)(ws + s.ml);
  b.ws_ml = (f32x2*)(ws + s.own_ml);
  b.ws_of = (int32_t*)(ws + s.own_of);
  a.m_rows = s.m_rows;
  a.m_groups = make_divisor((uint32_t)s.m_groups);
  a.unit_rows = make_divisor((uint32_t)s.unit_rows);
  a.n_units = s.n_units;
  a.n_rows = (uint32_t)table->kv_heads;
  a.n_parts = s.n_units * s.parts;
  a.shared_parts = s.parts;
  b.m_rows = s.own.m_rows;
  b.m_groups = make_divisor((uint32_t)s.own.m_groups);
  b.unit_rows = make_divisor((uint32_t)s.own.unit_rows);
  b.cap_tiles = s.own.cap_tiles;
  b.n_units = s.own.n_units;
  b.n_rows = (uint32_t)n_rows;
  b.n_parts = s.own.n_parts;
  const Divisor rows_of_head = make_divisor((uint32_t)(group * n_new));
  hipStream_t st = (hipStream_t)stream;
  switch (cache->head_dim / 64 * 2 + dtype) {
    case 2: launch_shared<1, false>(a, b, s, rows_of_head, st); break;
    case 3: launch_shared<1, true>(a, b, s, rows_of_head, st); break;
    case 4: launch_shared<2, false>(a, b, s, rows_of_head, st); break;
    case 5: launch_shared<2, true>(a, b, s, rows_of_head, st); break;
    case 6: launch_shared<3, false>(a, b, s, rows_of_head, st); break;
    case 7: launch_shared<3, true>(a, b, s, rows_of_head, st); break;
    case 8: launch_shared<4, false>(a, b, s, rows_of_head, st); break;
    default: launch_shared<4, true>(a, b, s, rows_of_head, st); break;
  }
  return launched();
}

}  // extern "C"
