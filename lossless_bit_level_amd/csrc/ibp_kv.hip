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
#include "ibp_kv_core.h"

namespace {

template <int DJ, bool F16>
__global__ __launch_bounds__(kThreads) void append_kernel(Pool pool, Rows rows, Strided k,
                                                          Strided v, Divisor pages_per_row,
                                                          uint32_t n_tasks) {
  append_tile<DJ, F16>(pool, rows, k, v, pages_per_row, n_tasks, NoTurn());
}

template <int DJ, bool F16, int MT, bool ONCE>
__global__ __launch_bounds__(kThreads, workgroups_per_unit(DJ, MT)) void attention_kernel(Attention a) {
  attend_part<DJ, F16, MT, ONCE, Sums::kFinished>(a, blockIdx.x);
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

// What a row's workgroup does: keep the protected pages and, of pages lo .. hi
// - 1, the `want` heaviest.
struct Choice {
  uint64_t at;  // the row's place in the tables
  int len;
  uint32_t held, left, lo, hi, want;
  bool full;
};

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

// One workgroup per row of up to THREADS * R pages, the weights in LDS.  With the
// counts of every 64 pages there each page knows its place.
// 768 rows of 16,384 pages (153 MB for those held, 201 MB with the spare entries)
// take 51 us: 1.5 workgroups to a place on the chip, and the loads, the choice and
// the stores of those that run together come one after the other (a row alone
// takes 17 us).  Without the buffers' bounds, with a branch for each page, 59 us.
template <int THREADS, int R>
__global__ __launch_bounds__(THREADS, 8) void evict_kernel(Evict e) {
  __shared__ ChoiceLds<THREADS, R> s;
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
    s.key[i][threadIdx.x] = key;
  }
  const Cut cut = cut_of<THREADS, R>(s, low, high, c.want, wave, lane);
  count_chunks<THREADS, R>(s, cut, wave, lane);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint32_t p = (uint32_t)i * THREADS + threadIdx.x;
    const uint32_t key = s.key[i][threadIdx.x];
    const Stay x = stay_of<THREADS, R>(s, cut, i, key, wave);
    // past the row's pages `before` is `left`, so that they keep their places
    const uint32_t to = x.stays ? x.before : c.left + p - x.before;
    __builtin_amdgcn_raw_buffer_store_b32(id[i], pages_out, (int)to * 4, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(key != 0u && !x.stays ? 0u : w[i], weights_out, (int)to * 4, 0, 0);
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

template <int DJ, bool F16>
void launch_append(const Pool& pool, const Rows& rows, const Strided& k, const Strided& v,
                   uint32_t pages_per_row, uint32_t tasks, hipStream_t st) {
  const uint32_t per_group = kWaves >> pool.tile_shift;
  hipLaunchKernelGGL((append_kernel<DJ, F16>), dim3((tasks + per_group - 1) / per_group),
                     dim3(kThreads), 0, st, pool, rows, k, v, make_divisor(pages_per_row), tasks);
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
  if (q_heads == 0 || q_heads % table->kv_heads || !weights != !weights_out || !std::isfinite(scale_log2(scale)))
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
  a.scale = scale_log2(scale);
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
