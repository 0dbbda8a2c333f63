// The embedding whose rows are dealt out to the ranks, and the gradient of its
// table by sorted tokens (see hbmc_embedding).
//
// The lookup copies rows: HBM bound, a wave a piece of a row (32768 rows of 4096
// bf16 in 69 us: 7.7 TB/s of rows read and written, the table's frequent rows
// coming from the caches).
//
// The gradient sorts (id, place) pairs, place = rank << 26 | token, with a
// stable radix sort of digits of at most ten bits, so that a row's tokens lie
// together in a fixed order; then a wave adds up `chunk` sorted tokens over 64
// vectors' columns, writing every id's row that lies within the chunk and leaving
// the sums of a first or last id that other chunks share to a joining kernel.
// No float is added atomically, so the sums' order, and with it every bit, is
// fixed.  It reads each gradient row once.  32768 tokens of 4096 bf16 added to
// 65536 fp32 rows take 157 us: the sort 25 us (four launches of one round trip
// or two each), the sums 118 us (their 0.6 GB at 5.4 TB/s: tokens' rows and the
// table's lie scattered), the joining 7 to 10 us.  Few tokens take one launch
// without sorting (embed_few_kernel).
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

constexpr uint32_t kPlaceBits = 26;
constexpr uint32_t kMaxBins = 1024;
constexpr uint32_t kSortWaves = 16;

// Where lane `lane` of piece `piece` (64 vectors) of a row starts; the row's
// last vector ends with the row, its first `dup` elements being its neighbour's.
template <int VE>
struct Column {
  uint32_t at, dup;
  bool on;
  __device__ __forceinline__ Column(uint32_t v, uint32_t width) {
    const uint32_t n = (width + VE - 1) / VE;
    on = v < n;
    const uint32_t c = on ? v : n - 1;
    at = c * VE + VE > width ? width - VE : c * VE;
    dup = v == n - 1 ? n * VE - width : 0;
  }
};

__device__ __forceinline__ int64_t load_id(const unsigned char* p, int id_bytes, uint64_t i) {
  return id_bytes == 8 ? reinterpret_cast<const int64_t*>(p)[i] : reinterpret_cast<const int32_t*>(p)[i];
}

// Vectors a lane copies of a row.  (32768 rows of 4096 bf16, stored past the
// cache: 69 us with two, 71.5 with four, 83 with eight; 99 with one.)
constexpr uint32_t kPiece = 2;

template <int DT, int VE, bool NT>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a) {
  typedef Pack<DT, VE> K;
  const uint32_t rank = blockIdx.y, lane = threadIdx.x & 63;
  const uint32_t pieces = (a.width + VE * 64 * kPiece - 1) / (VE * 64 * kPiece);
  const uint64_t units = uint64_t(a.tokens[rank]) * pieces;
  const unsigned char* ids = a.ids[rank];
  for (uint64_t unit = uint64_t(blockIdx.x) * 4 + uniform(threadIdx.x >> 6); unit < units; unit += uint64_t(gridDim.x) * 4) {
    const uint64_t token = pieces == 1 ? unit : unit / pieces;
    const uint32_t piece = pieces == 1 ? 0 : static_cast<uint32_t>(unit - token * pieces);
    const int64_t id = load_id(ids, a.id_bytes, token);
    const bool inside = id >= 0 && id < static_cast<int64_t>(a.vocab);
    const uint32_t row = uniform(inside ? static_cast<uint32_t>(id) : 0u);
    const uint32_t owner = row / a.seg;
    const unsigned char* from = a.rows[owner] + uint64_t(row - owner * a.seg) * a.width * K::E;
    unsigned char* to = a.out[rank] + token * a.width * K::E;
    typename K::raw v[kPiece] = {};
    if (uniform(inside ? 1u : 0u)) {
#pragma unroll
      for (uint32_t k = 0; k < kPiece; ++k) {
        const Column<VE> c((piece * kPiece + k) * 64 + lane, a.width);
        if (c.on) v[k] = K::load(from + uint64_t(c.at) * K::E);
      }
    }
#pragma unroll
    for (uint32_t k = 0; k < kPiece; ++k) {
      const Column<VE> c((piece * kPiece + k) * 64 + lane, a.width);
      if (!c.on) continue;
      float f[VE];
      K::widen(v[k], f);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = inside ? f[i] * a.scale : 0.0f;
      if constexpr (NT) K::store_nt(to + uint64_t(c.at) * K::E, K::narrow(f));
      else K::store(to + uint64_t(c.at) * K::E, K::narrow(f));
    }
  }
}

// ---------------------------------------------------------------- the sort

struct SortArgs {
  const unsigned char* ids[kMaxRanks];
  uint32_t tokens[kMaxRanks];
  int P, id_bytes;
  uint32_t vocab, total, tiles, bits, passes;
  uint32_t* hist;     // [tiles][kMaxBins], of the pass at work
  uint32_t* key[2];   // sorted so far, and place beside it
  uint32_t* place[2];
  unsigned char* touched;  // 1 for each id that occurs, or nullptr
  // the table's gradient cleared by the workgroups past the tiles (nullptr: not)
  unsigned char* clear[kMaxRanks];
  uint64_t clear_bytes[kMaxRanks];
  uint32_t clear_units, clear_first;  // units of kClearUnit bytes a rank; the first of this launch
};

constexpr uint32_t kClearUnit = 1024 * 16 * 8;

// The unit-th piece of the ranks' gradients set to zero.
__device__ __forceinline__ void clear_piece(const SortArgs& a, uint32_t unit) {
  const uint32_t rank = unit / a.clear_units;
  const uint64_t from = uint64_t(unit - rank * a.clear_units) * kClearUnit, end = a.clear_bytes[rank];
  unsigned char* to = a.clear[rank];
#pragma unroll
  for (uint32_t k = 0; k < 8; ++k) {
    const uint64_t at = from + (k * 1024 + threadIdx.x) * 16;
    if (at + 16 <= end) {
      *reinterpret_cast<u32x4_any*>(to + at) = u32x4{};
    } else {
      for (uint64_t b = at; b < end; b += 2) *reinterpret_cast<uint16_t*>(to + b) = 0;  // whole elements of 2 or 4 bytes
    }
  }
}

// Ranks' first tokens among all ranks' in LDS.
__device__ __forceinline__ void rank_starts(const SortArgs& a, uint32_t* before) {
  if (threadIdx.x < 64) {
    uint32_t x = static_cast<int>(threadIdx.x) < a.P ? a.tokens[threadIdx.x] : 0;
    const uint32_t own = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t y = __shfl_up(x, d);
      if (static_cast<int>(threadIdx.x) >= d) x += y;
    }
    before[threadIdx.x] = x - own;
  }
  __syncthreads();
}

// The i-th token of all ranks: its id (vocab where it is none) and place.
__device__ __forceinline__ uint32_t token_key(const SortArgs& a, const uint32_t* before, uint32_t i, uint32_t* place) {
  uint32_t r = 0;
#pragma unroll
  for (uint32_t step = 32; step > 0; step >>= 1)
    if (r + step < static_cast<uint32_t>(a.P) && before[r + step] <= i) r += step;
  const uint32_t token = i - before[r];
  *place = r << kPlaceBits | token;
  const int64_t id = load_id(a.ids[r], a.id_bytes, token);
  return id >= 0 && id < static_cast<int64_t>(a.vocab) ? static_cast<uint32_t>(id) : a.vocab;
}

// A tile's counts of the pass's digit; before the first pass also clears
// `touched`.  R: pairs a thread.
template <int R>
__global__ __launch_bounds__(1024) void embed_count_kernel(SortArgs a, uint32_t pass) {
  __shared__ uint32_t before[64], bins[kMaxBins];
  if (blockIdx.x >= a.tiles) {
    clear_piece(a, a.clear_first + blockIdx.x - a.tiles);
    return;
  }
  const uint32_t shift = pass * a.bits, mask = (1u << a.bits) - 1;
  bins[threadIdx.x] = 0;
  if (pass == 0) rank_starts(a, before);
  else __syncthreads();
  const uint32_t lo = blockIdx.x * R * 1024;
#pragma unroll
  for (uint32_t r = 0; r < R; ++r) {
    const uint32_t i = lo + r * 1024 + threadIdx.x;
    uint32_t place;
    if (i < a.total) atomicAdd(&bins[(pass == 0 ? token_key(a, before, i, &place) : a.key[(pass + 1) & 1][i]) >> shift & mask], 1u);
  }
  __syncthreads();
  a.hist[blockIdx.x * kMaxBins + threadIdx.x] = bins[threadIdx.x];
  if (a.touched && pass == 0)
    for (uint32_t w = blockIdx.x * 1024 + threadIdx.x; w < (a.vocab + 3) / 4; w += a.tiles * 1024)
      reinterpret_cast<uint32_t*>(a.touched)[w] = 0;
}

// Lanes of the wave whose digit equals this lane's (`on` lanes only).
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, uint32_t bits, bool on) {
  uint64_t same = __ballot(on);
  for (uint32_t b = 0; b < bits; ++b) {
    const bool bit = digit >> b & 1;
    const uint64_t ones = __ballot(bit);
    same &= bit ? ones : ~ones;
  }
  return same;
}

__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Where a tile's pairs go: each wave ranks its own stretch of 64 * R pairs by
// digit, counting in LDS as it goes, and the waves' counts and the tiles'
// (`all` and `prior`: of bin threadIdx.x in all tiles, in those before this
// one) become each wave's first positions.  to[r]: the r-th pair's position.
template <int R, typename Counts>
__device__ __forceinline__ void sort_positions(const uint32_t (&key)[R], const bool (&on)[R], uint32_t shift, uint32_t bits,
                                               uint32_t (*count)[kMaxBins], uint32_t* scan, Counts&& counts, uint32_t (&to)[R]) {
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t mask = (1u << bits) - 1;
  const uint64_t below = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (uint32_t w = 0; w < kSortWaves; ++w) count[w][threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t digit = key[r] >> shift & mask;
    const uint64_t same = same_digit(digit, bits, on[r]);
    to[r] = 0;
    if (on[r]) to[r] = count[wave][digit] + __popcll(same & below);
    wave_order();
    if (on[r] && (same & below) == 0) count[wave][digit] += __popcll(same);
    wave_order();
  }
  __syncthreads();
  uint32_t all, prior;
  counts(&all, &prior);
  uint32_t x = all;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    if (static_cast<int>(lane) >= d) x += y;
  }
  if (lane == 63) scan[wave] = x;
  __syncthreads();
  uint32_t first = x - all + prior;
  for (uint32_t w = 0; w < wave; ++w) first += scan[w];
#pragma unroll
  for (uint32_t w = 0; w < kSortWaves; ++w) {
    const uint32_t c = count[w][threadIdx.x];
    count[w][threadIdx.x] = first;
    first += c;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (on[r]) to[r] += count[wave][key[r] >> shift & mask];
}

// Marks the ids that occur, a byte each: stores of one value need no order
// (bits set by atomics took 85 us for 32768 tokens, a third of them in one word).
template <int R>
__device__ __forceinline__ void mark(const SortArgs& a, const uint32_t (&key)[R], const bool (&on)[R]) {
  if (!a.touched) return;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (on[r] && key[r] < a.vocab) a.touched[key[r]] = 1;
}

template <int R>
__global__ __launch_bounds__(1024) void embed_sort_kernel(SortArgs a, uint32_t pass) {
  __shared__ uint32_t before[64], scan[kSortWaves], count[kSortWaves][kMaxBins];
  if (blockIdx.x >= a.tiles) {
    clear_piece(a, a.clear_first + blockIdx.x - a.tiles);
    return;
  }
  if (pass == 0) rank_starts(a, before);
  const uint32_t lo = blockIdx.x * R * 1024 + uniform(threadIdx.x >> 6) * R * 64 + (threadIdx.x & 63);
  uint32_t key[R], place[R], to[R];
  bool on[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t i = lo + r * 64;
    on[r] = i < a.total;
    key[r] = place[r] = 0;
    if (on[r]) {
      if (pass == 0) {
        key[r] = token_key(a, before, i, &place[r]);
      } else {
        key[r] = a.key[(pass + 1) & 1][i];
        place[r] = a.place[(pass + 1) & 1][i];
      }
    }
  }
  // The tiles' counts, on their way while the pairs are ranked: 16 at once, the
  // last ones too (one after another they took 2 us of the launch's 9 for 12 tiles).
  uint32_t all = 0, prior = 0, t = 0;
  const uint32_t* h = a.hist + threadIdx.x;
  for (; t + 16 <= a.tiles; t += 16) {
#pragma unroll
    for (uint32_t k = 0; k < 16; ++k) {
      const uint32_t c = h[(t + k) * kMaxBins];
      all += c;
      prior += t + k < blockIdx.x ? c : 0;
    }
  }
  if (t < a.tiles) {
    uint32_t c[16];
#pragma unroll
    for (uint32_t k = 0; k < 16; ++k) c[k] = h[min(t + k, a.tiles - 1) * kMaxBins];
#pragma unroll
    for (uint32_t k = 0; k < 16; ++k) {
      all += t + k < a.tiles ? c[k] : 0;
      prior += t + k < blockIdx.x ? c[k] : 0;
    }
  }
  sort_positions<R>(key, on, pass * a.bits, a.bits, count, scan, [&](uint32_t* x, uint32_t* y) { *x = all, *y = prior; }, to);
  if (pass == 0) mark<R>(a, key, on);
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (on[r]) {
      a.key[pass & 1][to[r]] = key[r];
      a.place[pass & 1][to[r]] = place[r];
    }
}

// All passes of a call whose pairs are one tile, between them in LDS.
template <int R>
__global__ __launch_bounds__(1024) void embed_sort_all_kernel(SortArgs a) {
  __shared__ uint32_t before[64], scan[kSortWaves], count[kSortWaves][kMaxBins];
  __shared__ uint2 pairs[R * 1024];
  if (blockIdx.x >= 1) {
    clear_piece(a, a.clear_first + blockIdx.x - 1);
    return;
  }
  rank_starts(a, before);
  if (a.touched) {
    for (uint32_t w = threadIdx.x; w < (a.vocab + 3) / 4; w += 1024) reinterpret_cast<uint32_t*>(a.touched)[w] = 0;
    __threadfence();
    __syncthreads();
  }
  const uint32_t lo = uniform(threadIdx.x >> 6) * R * 64 + (threadIdx.x & 63);
  uint32_t key[R], place[R], to[R];
  bool on[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    on[r] = lo + r * 64 < a.total;
    key[r] = place[r] = 0;
    if (on[r]) key[r] = token_key(a, before, lo + r * 64, &place[r]);
  }
  mark<R>(a, key, on);
  for (uint32_t pass = 0; pass < a.passes; ++pass) {
    sort_positions<R>(key, on, pass * a.bits, a.bits, count, scan, [&](uint32_t* all, uint32_t* prior) {
      *all = *prior = 0;
#pragma unroll
      for (uint32_t w = 0; w < kSortWaves; ++w) *all += count[w][threadIdx.x];
    }, to);
    if (pass + 1 == a.passes) break;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (on[r]) pairs[to[r]] = uint2{key[r], place[r]};
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (on[r]) {
        const uint2 p = pairs[lo + r * 64];
        key[r] = p.x;
        place[r] = p.y;
      }
    // the next pass's first barrier is behind its counts alone: pairs are
    // written again only after its later ones
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (on[r]) {
      a.key[0][to[r]] = key[r];
      a.place[0][to[r]] = place[r];
    }
}

// ---------------------------------------------------------------- the sums

struct SumArgs {
  const unsigned char* rows[kMaxRanks];
  unsigned char* out[kMaxRanks];
  uint32_t seg, vocab, width, total, chunk, chunks;
  float scale;
  const uint32_t* key;
  const uint32_t* place;
  const unsigned char* touched;  // the rows that occur, for those that clear the others
  bool accumulate;
  float* partial;           // [chunks][2][width]: of a chunk's first id, of its last
  uint32_t sum_groups;      // workgroups that add; those after them clear rows
  uint32_t clear_rows;      // rows a wave clears
};

// Where the lane's columns of id `key` lie in the gradient, and what is there.
template <int GT>
__device__ __forceinline__ unsigned char* grad_at(const SumArgs& a, uint32_t key, uint32_t at) {
  const uint32_t owner = key / a.seg;
  return a.out[owner] + (uint64_t(key - owner * a.seg) * a.width + at) * Width<GT>::bytes;
}
template <int GT, int VE>
__device__ __forceinline__ void load_row(const unsigned char* p, float (&f)[VE]) {
  if constexpr (VE * Width<GT>::bytes <= 16) {
    Pack<GT, VE>::widen(Pack<GT, VE>::load(p), f);
  } else {
#pragma unroll
    for (int i = 0; i < VE; i += 4) {
      const f32x4_any v = *reinterpret_cast<const f32x4_any*>(p + i * 4);
      f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
  }
}

// The finished sum of id `key` (scaled, and added to `old` where the call
// accumulates), at the lane's columns.
template <int GT, int VE>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, const Column<VE>& c, float (&acc)[VE],
                                          const float (&old)[VE]) {
  if (!c.on) return;
  unsigned char* to = grad_at<GT>(a, key, c.at);
#pragma unroll
  for (int i = 0; i < VE; ++i) acc[i] = a.accumulate ? old[i] + acc[i] * a.scale : acc[i] * a.scale;
  if constexpr (VE > 1) {
    if (a.accumulate && c.dup != 0) {
      // a row's last two lanes share columns; only one of them may add
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float one[1] = {acc[i]};
        if (i >= static_cast<int>(c.dup)) Pack<GT, 1>::store(to + i * Width<GT>::bytes, Pack<GT, 1>::narrow(one));
      }
      return;
    }
  }
  if constexpr (VE * Width<GT>::bytes <= 16) Pack<GT, VE>::store(to, Pack<GT, VE>::narrow(acc));
  else store_floats<VE>(reinterpret_cast<float*>(to), acc);
}

template <int DT, int GT, int VE>
__global__ __launch_bounds__(256) void embed_sum_kernel(SumArgs a) {
  typedef Pack<DT, VE> K;
  // Tokens whose loads are in flight: 32768 of 4096 into 65536 rows 158 us with
  // eight, 172 with four.
  constexpr uint32_t U = 8;
  const uint32_t lane = threadIdx.x & 63;
  if (blockIdx.x >= a.sum_groups) {
    constexpr int GE = VE == 1 ? 1 : 16 / Width<GT>::bytes;
    typedef Pack<GT, GE> Z;
    const uint32_t first = ((blockIdx.x - a.sum_groups) * 4 + uniform(threadIdx.x >> 6)) * a.clear_rows;
    for (uint32_t r = first; r < first + a.clear_rows && r < a.vocab; ++r) {
      if (a.touched[r]) continue;
      const uint32_t owner = r / a.seg;
      unsigned char* to = a.out[owner] + uint64_t(r - owner * a.seg) * a.width * Z::E;
      for (uint32_t v = lane; v * GE < a.width; v += 64) {
        const Column<GE> c(v, a.width);
        Z::store(to + uint64_t(c.at) * Z::E, typename Z::raw{});
      }
    }
    return;
  }
  const uint32_t pieces = (a.width + VE * 64 - 1) / (VE * 64);
  const uint64_t unit = uint64_t(blockIdx.x) * 4 + uniform(threadIdx.x >> 6);
  const uint32_t chunk = static_cast<uint32_t>(unit / pieces);
  if (chunk >= a.chunks) return;
  const Column<VE> c(static_cast<uint32_t>(unit - uint64_t(chunk) * pieces) * 64 + lane, a.width);
  const uint32_t lo = chunk * a.chunk, hi = min(lo + a.chunk, a.total);
  const uint32_t keys = lo + lane < hi ? a.key[lo + lane] : a.vocab;
  const uint32_t places = lo + lane < hi ? a.place[lo + lane] : 0;
  const uint32_t n = __popcll(__ballot(keys < a.vocab));  // tokens without a row come last
  if (n == 0) return;
  const auto key_of = [&](uint32_t t) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(keys), t)); };
  const uint32_t begun = lo > 0 ? uniform(a.key[lo - 1]) : a.vocab;     // the id that began in an earlier chunk
  const uint32_t after = hi < a.total ? uniform(a.key[hi]) : a.vocab;  // the id that a later chunk begins with
  float* partial = a.partial + uint64_t(chunk) * 2 * a.width + c.at;
  float acc[VE] = {};
  for (uint32_t t = 0; t < n; t += U) {
    typename K::raw v[U];
    float old[U][VE] = {};
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      const uint32_t at = min(t + u, n - 1);
      const uint32_t pl = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(places), at));
      const unsigned char* row = a.rows[pl >> kPlaceBits] + uint64_t(pl & ((1u << kPlaceBits) - 1)) * a.width * K::E;
      v[u] = K::stream(row + c.at * K::E);
    }
    if (a.accumulate) {
      // what the rows finished here hold, on its way with their tokens
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        if (t + u >= n) continue;
        const uint32_t key = key_of(t + u), next = t + u + 1 < n ? key_of(t + u + 1) : after;
        if (key != next && key != begun) load_row<GT, VE>(grad_at<GT>(a, key, c.at), old[u]);
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      if (t + u >= n) continue;
      float f[VE];
      K::widen(v[u], f);
#pragma unroll
      for (int i = 0; i < VE; ++i) acc[i] += f[i];
      const uint32_t key = key_of(t + u), next = t + u + 1 < n ? key_of(t + u + 1) : after;
      if (key != next || t + u + 1 == n) {
        // the id's last token here: finished, or left for joining
        if (key != begun && key != next) write_row<GT, VE>(a, key, c, acc, old[u]);
        else if (c.on) store_floats<VE>(partial + (key == begun ? 0 : a.width), acc);
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[i] = 0.0f;
      }
    }
  }
}

// Joins the sums of an id that spans chunks: a workgroup for each piece of a row
// and the chunk the id begins in (most find nothing to join), its four waves
// taking a quarter of the later chunks each.  One workgroup a chunk, for all of
// a row's pieces, took twice as long: a frequent id is then one compute unit's.
template <int DT, int GT, int VE>
__global__ __launch_bounds__(256) void embed_join_kernel(SumArgs a) {
  __shared__ float parts[4][VE][64];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t pieces = (a.width + VE * 64 - 1) / (VE * 64);
  const uint32_t chunk = blockIdx.x / pieces;
  const uint32_t lo = chunk * a.chunk, hi = lo + a.chunk;
  const uint32_t key = uniform(a.key[hi - 1]), next = uniform(a.key[hi]);
  const uint32_t first = uniform(a.key[lo]), before = lo > 0 ? uniform(a.key[lo - 1]) : a.vocab;
  if (key >= a.vocab || next != key || (first == key && before == key)) return;  // ends here, or began earlier
  const Column<VE> c((blockIdx.x - chunk * pieces) * 64 + lane, a.width);
  const uint64_t step = uint64_t(2) * a.width;
  const float* head = a.partial + (chunk + 1) * step + c.at;
  uint32_t n = 0;  // later chunks that begin with the id
  for (uint32_t from = chunk + 1; from < a.chunks; from += 64) {
    const uint32_t mine = from + lane;
    const bool same = mine < a.chunks && a.key[uint64_t(mine) * a.chunk] == key;
    const uint32_t more = __popcll(__ballot(same));  // sorted: the first of them
    n += more;
    if (more < 64) break;
  }
  const uint32_t each = (n + 3) / 4, end = min(n, (wave + 1) * each);
  float acc[VE] = {};
  uint32_t t = wave * each;
  for (; t + 4 <= end; t += 4) {
    float f[4][VE];
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u) load_row<kF32, VE>(reinterpret_cast<const unsigned char*>(head + (t + u) * step), f[u]);
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < VE; ++i) acc[i] += f[u][i];
  }
  for (; t < end; ++t) {
    float f[VE];
    load_row<kF32, VE>(reinterpret_cast<const unsigned char*>(head + t * step), f);
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[i] += f[i];
  }
#pragma unroll
  for (int i = 0; i < VE; ++i) parts[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave != 0) return;
  float old[VE] = {};
  if (a.accumulate) load_row<GT, VE>(grad_at<GT>(a, key, c.at), old);
  load_row<kF32, VE>(reinterpret_cast<const unsigned char*>(head - step + a.width), acc);  // the id's beginning
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[i] += parts[w][i][lane];
  write_row<GT, VE>(a, key, c, acc, old);
}

// ------------------------------------------------------------- few tokens

// A call of few tokens in one launch, with no sort and no workspace: a workgroup
// for each token and `per` pieces of a row asks every token for its id; the first
// token of an id adds up all of that id's, in the tokens' order, and the others
// leave.  Most ids occur once or a few times: a wave then takes a piece; more than
// kAlone * per tokens are dealt out to the four waves, piece by piece.  The
// workgroups past those clear the rows that have no token.  8 ranks, bf16 into
// fp32, added: 64 tokens of 4096 6.8 us and 512 of 2048 8.2 us, where the sort's
// three launches take 18 and 20; what bounds it is a chain of four round trips
// (ranks' tokens, ids, gradient rows, stores) and, from 1000 workgroups on, that
// each reads all ids.
struct FewArgs {
  SortArgs t;
  SumArgs m;
  uint32_t per;         // pieces a workgroup adds
  uint32_t clear_each;  // rows a workgroup clears
};

constexpr uint32_t kAlone = 8;

// ROUNDS: tokens a lane compares.
template <int DT, int GT, int VE, int ROUNDS>
__global__ __launch_bounds__(256) void embed_few_kernel(FewArgs a) {
  typedef Pack<DT, VE> K;
  constexpr uint32_t kMost = ROUNDS * 256;
  __shared__ uint32_t before[64], list[kMost];
  __shared__ uint64_t masks[ROUNDS * 4];
  __shared__ float parts[4][VE][64];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const SumArgs& m = a.m;
  rank_starts(a.t, before);
  uint32_t key[ROUNDS], place[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const uint32_t i = r * 256 + threadIdx.x;
    key[r] = m.vocab;
    place[r] = 0;
    if (i < m.total) key[r] = token_key(a.t, before, i, &place[r]);
  }
  if (blockIdx.x >= m.sum_groups) {
    // list[x]: row `first + x` of the rank has a token
    const uint32_t each = a.clear_each, units = (m.seg + each - 1) / each;
    const uint32_t unit = blockIdx.x - m.sum_groups, rank = unit / units, first = (unit - rank * units) * each;
    const uint32_t base = rank * m.seg;  // may pass the vocabulary's end on a rank that owns nothing
    const uint32_t rows = base >= m.vocab ? 0 : min(m.seg, m.vocab - base);
    const uint32_t n = first >= rows ? 0 : min(each, rows - first);
    if (threadIdx.x < each) list[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const uint32_t x = key[r] - (base + first);  // wraps for rows before
      if (key[r] < m.vocab && x < n) list[x] = 1;
    }
    __syncthreads();
    constexpr int GE = VE == 1 ? 1 : 16 / Width<GT>::bytes;
    typedef Pack<GT, GE> Z;
    const uint32_t vectors = (m.width + GE - 1) / GE;
    unsigned char* to = m.out[rank] + uint64_t(first) * m.width * Z::E;
    if (vectors >= 64) {
      for (uint32_t x = wave; x < n; x += 4) {
        if (uniform(list[x])) continue;
        for (uint32_t v = lane; v < vectors; v += 64)
          Z::store(to + (uint64_t(x) * m.width + Column<GE>(v, m.width).at) * Z::E, typename Z::raw{});
      }
    } else {
      for (uint32_t v = threadIdx.x; v < n * vectors; v += 256) {
        const uint32_t x = v / vectors;
        if (!list[x]) Z::store(to + (uint64_t(x) * m.width + Column<GE>(v - x * vectors, m.width).at) * Z::E, typename Z::raw{});
      }
    }
    return;
  }
  const uint32_t pieces = (m.width + VE * 64 - 1) / (VE * 64), shares = (pieces + a.per - 1) / a.per;
  const uint32_t token = blockIdx.x / shares, from = (blockIdx.x - token * shares) * a.per;
  uint32_t own_place;
  const uint32_t own = uniform(token_key(a.t, before, token, &own_place));
  if (own >= m.vocab) return;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const uint64_t same = __ballot(key[r] == own);
    if (lane == 0) masks[r * 4 + wave] = same;
  }
  __syncthreads();
  uint32_t n = 0, at[ROUNDS];  // tokens of the id; of those, before this wave's r-th 64
  bool leads = true;
#pragma unroll
  for (uint32_t k = 0; k < ROUNDS * 4; ++k) {
    const uint64_t same = uniform(masks[k]);
    if (k % 4 == wave) at[k / 4] = n;
    if (n == 0 && same != 0) leads = k * 64 + __builtin_ctzll(same) == token;
    n += __popcll(same);
  }
  if (!leads) return;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const uint64_t same = __ballot(key[r] == own);
    if (key[r] == own) list[at[r] + __popcll(same & ((uint64_t(1) << lane) - 1))] = place[r];
  }
  __syncthreads();
  // the lo-th to the hi-th of the id's tokens
  const auto add = [&](const Column<VE>& c, uint32_t lo, uint32_t hi, float (&acc)[VE]) {
    constexpr uint32_t U = kAlone;
    for (uint32_t t = lo; t < hi; t += U) {
      typename K::raw v[U];
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        if (t + u >= hi) continue;
        const uint32_t pl = uniform(list[t + u]);
        v[u] = K::load(m.rows[pl >> kPlaceBits] + (uint64_t(pl & ((1u << kPlaceBits) - 1)) * m.width + c.at) * K::E);
      }
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        if (t + u >= hi) continue;
        float f[VE];
        K::widen(v[u], f);
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[i] += f[i];
      }
    }
  };
  if (n <= kAlone * a.per) {
    if (wave >= a.per || from + wave >= pieces) return;
    const Column<VE> c((from + wave) * 64 + lane, m.width);
    float old[VE] = {}, acc[VE] = {};
    if (m.accumulate) load_row<GT, VE>(grad_at<GT>(m, own, c.at), old);
    add(c, 0, n, acc);
    write_row<GT, VE>(m, own, c, acc, old);
    return;
  }
  const uint32_t each = (n + 3) / 4, lo = wave * each, hi = min(n, lo + each);
  for (uint32_t piece = from; piece < min(from + a.per, pieces); ++piece) {
    const Column<VE> c(piece * 64 + lane, m.width);
    float old[VE] = {}, acc[VE] = {};
    if (wave == 0 && m.accumulate) load_row<GT, VE>(grad_at<GT>(m, own, c.at), old);
    add(c, lo, hi, acc);
    __syncthreads();  // the piece before is joined
#pragma unroll
    for (int i = 0; i < VE; ++i) parts[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave != 0) continue;
#pragma unroll
    for (int w = 1; w < 4; ++w)
#pragma unroll
      for (int i = 0; i < VE; ++i) acc[i] += parts[w][i][lane];
    write_row<GT, VE>(m, own, c, acc, old);
  }
}

}  // namespace dev

namespace {

using namespace dev;

template <int N>
using Int = std::integral_constant<int, N>;

template <typename F>
hipError_t with_type(int dtype, uint32_t width, F&& f) {
  const bool one = width < (dtype == kF32 ? 4u : 8u);
  if (dtype == kF32) return one ? f(Int<kF32>(), Int<1>()) : f(Int<kF32>(), Int<4>());
  if (dtype == kF16) return one ? f(Int<kF16>(), Int<1>()) : f(Int<kF16>(), Int<8>());
  return one ? f(Int<kBF16>(), Int<1>()) : f(Int<kBF16>(), Int<8>());
}

uint32_t vector_elems(int dtype, uint64_t width) {
  const uint32_t full = dtype == kF32 ? 4 : 8;
  return width < full ? 1 : full;
}

hipError_t go(const void* f, uint64_t groups, uint32_t threads, void** argv, hipStream_t stream) {
  return hipLaunchKernel(f, dim3(static_cast<uint32_t>(groups)), dim3(threads), argv, 0, stream);
}

constexpr uint32_t kMaxChunk = 64;  // a lane holds each token's pair
// Tokens that one workgroup sorts by itself, in 8 us (1024) to 26 us (8192); the
// four launches of the other way take 24 us for 16384.
constexpr uint32_t kSingleTile = 8192;
// Tokens that are added without sorting, in us beside the sort's way (8 ranks, bf16
// into fp32, added): 1024 of 256 9.0 and 20; 1024 of 4096 20.7 and 22; the time
// grows with the square of the tokens from there.
constexpr uint32_t kFewTokens = 1024;
// Of those, the pieces of rows up to which a workgroup takes one and not four:
// 512 tokens of 2048 (2048 pieces) 8.2 us with one and 11.6 with four, 1024 of 2048
// (4096) 17.5 and 18.2, 512 of 8192 (8192) 21 and 14.5.
constexpr uint32_t kFewPieces = 4096;

template <typename F>
hipError_t with_rounds(uint32_t rounds, F&& f) {
  switch (rounds) {
    case 1: return f(Int<1>());
    case 2: return f(Int<2>());
    case 4: return f(Int<4>());
    default: return f(Int<8>());
  }
}

}  // namespace

hipError_t launch_embed(int dtype, const EmbedArgs& a, hipStream_t stream) {
  uint64_t most = 0, total = 0;
  for (int r = 0; r < a.P; ++r) {
    most = std::max<uint64_t>(most, a.tokens[r]);
    total += a.tokens[r];
  }
  const bool nt = total * a.width * (dtype == kF32 ? 4 : 2) >= kStreamBytes;
  return with_type(dtype, a.width, [&](auto dt, auto ve) {
    const uint64_t pieces = (a.width + ve * 64 * kPiece - 1) / (ve * 64 * kPiece);
    const uint64_t groups = std::min<uint64_t>((most * pieces + 3) / 4, 1 << 20);
    void* argv[] = {const_cast<EmbedArgs*>(&a)};
    return hipLaunchKernel(nt ? reinterpret_cast<const void*>(&embed_kernel<dt, ve, true>)
                              : reinterpret_cast<const void*>(&embed_kernel<dt, ve, false>),
                           dim3(static_cast<uint32_t>(groups), static_cast<uint32_t>(a.P)), dim3(256), argv, 0, stream);
  });
}

namespace {
uint64_t row_pieces(int dtype, uint64_t width) {
  const uint64_t piece = vector_elems(dtype, width) * 64;
  return (width + piece - 1) / piece;
}
}  // namespace

// The joining launch is the largest: fewer than tokens / 64 * pieces workgroups
// of 256 threads there (kMaxChunk tokens a chunk in calls this large).
bool embed_grad_fits(int dtype, uint64_t total, uint64_t width) {
  return total * row_pieces(dtype, width) <= uint64_t(1) << 30;
}

EmbedGradSplit split_embed_grad(int dtype, uint64_t total, uint64_t vocab, uint64_t width) {
  EmbedGradSplit d;
  d.total = total;
  const uint64_t pieces = row_pieces(dtype, width);
  d.few = total > 0 && total <= kFewTokens && pieces <= 4096;  // at most 2^20 workgroups
  if (d.few) return d;
  uint32_t bits = 0;  // of the largest key, vocab itself
  while (vocab >> bits) ++bits;
  d.passes = (bits + 9) / 10;
  d.bits = (bits + d.passes - 1) / d.passes;
  // pairs a thread sorts: one workgroup up to kSingleTile tokens, else 64 of them while
  // eight pairs a thread are enough
  d.rounds = 1;
  while (d.rounds < 8 && total > uint64_t(1024) * d.rounds * (total <= kSingleTile ? 1 : 64)) d.rounds *= 2;
  d.tiles = static_cast<uint32_t>((total + 1024 * d.rounds - 1) / (1024 * d.rounds));
  // Without accumulation the rows are cleared: all of them beside the sort, which
  // leaves HBM idle, while few of them are written again; else those without a
  // token beside the sums.  All and those, us: 2500 tokens, 50001 rows 32 and 45;
  // 32768 tokens, 131072 rows 259 and 264, 65536 rows 187 and 191; 65536 tokens,
  // 8192 rows 109 and 104.
  d.clear_all = total <= vocab / 4;
  // Tokens a wave adds up: few, so that a wave's loads are one round trip, while
  // the waves are few; more of them leave fewer sums to join.  8 ranks, bf16 into
  // fp32, added: 4096 tokens of 1024 with 8 and 16 29 and 31.5 us; 32768 of 1024 65
  // and 59; 131072 of 512 with 16, 32 and 64 94, 86 and 93.
  d.chunk = total <= kSingleTile ? 8 : 16;
  while (d.chunk < kMaxChunk && (total * pieces / d.chunk > 8192 || total / d.chunk > 4096)) d.chunk *= 2;
  d.chunks = static_cast<uint32_t>((total + d.chunk - 1) / d.chunk);
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t from = at;
    at += (bytes + 255) / 256 * 256;
    return from;
  };
  d.key_a = take(total * 4);
  d.key_b = take(total * 4);
  d.place_a = take(total * 4);
  d.place_b = take(total * 4);
  d.hist = take(uint64_t(d.tiles) * kMaxBins * 4);
  d.touched = take((vocab + 3) / 4 * 4);
  d.partial = take(uint64_t(d.chunks) * 2 * width * 4);
  d.bytes = at;
  return d;
}

namespace {

// A call of few tokens (embed_few_kernel).
hipError_t launch_few(int dtype, int grad_dtype, const SortArgs& s, const SumArgs& m, hipStream_t stream) {
  FewArgs a = {s, m, 1, 0};
  uint64_t clear = 0;
  if (!m.accumulate) {
    // 64 KiB a workgroup, or a row where that is more
    const uint64_t row = uint64_t(m.width) * (grad_dtype == kF32 ? 4 : 2);
    a.clear_each = static_cast<uint32_t>(std::clamp<uint64_t>(65536 / row, 1, 256));
    clear = uint64_t(s.P) * ((m.seg + a.clear_each - 1) / a.clear_each);
  }
  return with_type(dtype, m.width, [&](auto dt, auto ve) {
    const uint32_t pieces = (m.width + ve * 64 - 1) / (ve * 64);
    a.per = m.total * pieces <= kFewPieces ? 1 : 4;
    a.m.sum_groups = m.total * ((pieces + a.per - 1) / a.per);
    const bool wide = grad_dtype == kF32 && dt != kF32;
    void* argv[] = {&a};
    return with_rounds(m.total <= 256 ? 1 : m.total <= 512 ? 2 : 4, [&](auto r) {
      if constexpr (r > 4) return hipErrorInvalidValue;
      else return go(wide ? reinterpret_cast<const void*>(&embed_few_kernel<dt, kF32, ve, r>)
                          : reinterpret_cast<const void*>(&embed_few_kernel<dt, dt, ve, r>),
                     a.m.sum_groups + clear, 256, argv, stream);
    });
  });
}

}  // namespace

hipError_t launch_embed_grad(int dtype, int grad_dtype, const EmbedArgs& a, const EmbedGradSplit& d, bool accumulate,
                             unsigned char* workspace, hipStream_t stream) {
  SortArgs s = {};
  SumArgs m = {};
  for (int r = 0; r < a.P; ++r) {
    s.ids[r] = a.ids[r];
    s.tokens[r] = a.tokens[r];
    m.rows[r] = a.rows[r];
    m.out[r] = a.out[r];
  }
  s.P = a.P;
  s.id_bytes = a.id_bytes;
  s.vocab = m.vocab = a.vocab;
  s.total = m.total = static_cast<uint32_t>(d.total);
  m.seg = a.seg;
  m.width = a.width;
  m.scale = a.scale;
  m.accumulate = accumulate;
  if (d.few) return launch_few(dtype, grad_dtype, s, m, stream);
  s.tiles = d.tiles;
  s.bits = d.bits;
  s.passes = d.passes;
  s.hist = reinterpret_cast<uint32_t*>(workspace + d.hist);
  s.key[0] = reinterpret_cast<uint32_t*>(workspace + d.key_a);
  s.key[1] = reinterpret_cast<uint32_t*>(workspace + d.key_b);
  s.place[0] = reinterpret_cast<uint32_t*>(workspace + d.place_a);
  s.place[1] = reinterpret_cast<uint32_t*>(workspace + d.place_b);
  s.touched = accumulate || d.clear_all ? nullptr : workspace + d.touched;
  uint64_t units = 0;  // pieces to clear, in equal shares by the sort's launches
  if (!accumulate && d.clear_all) {
    const uint64_t row = uint64_t(a.width) * (grad_dtype == kF32 ? 4 : 2);
    for (int r = 0; r < a.P; ++r) {
      s.clear[r] = a.out[r];
      s.clear_bytes[r] = segment_count(a.vocab, a.P, r) * row;
    }
    s.clear_units = static_cast<uint32_t>((s.clear_bytes[0] + kClearUnit - 1) / kClearUnit);
    units = uint64_t(s.clear_units) * a.P;
  }
  const uint32_t launches = d.tiles <= 1 ? 1 : 2 * d.passes;
  uint32_t launch = 0;
  // the grid of the next launch: the tiles and its share of the clearing
  const auto grid = [&]() {
    s.clear_first = static_cast<uint32_t>(units * launch / launches);
    const uint32_t end = static_cast<uint32_t>(units * ++launch / launches);
    return std::max(d.tiles, 1u) + end - s.clear_first;
  };
  hipError_t e = hipSuccess;
  if (d.tiles <= 1) {
    // with no tokens at all it only clears
    if (d.total == 0 && accumulate) return hipSuccess;
    e = with_rounds(d.rounds, [&](auto r) {
      const uint64_t groups = grid();
      void* argv[] = {&s};
      return go(reinterpret_cast<const void*>(&embed_sort_all_kernel<r>), groups, 1024, argv, stream);
    });
  } else {
    e = with_rounds(d.rounds, [&](auto r) {
      hipError_t f = hipSuccess;
      for (uint32_t pass = 0; f == hipSuccess && pass < d.passes; ++pass) {
        void* argv[] = {&s, &pass};
        uint64_t groups = grid();
        f = go(reinterpret_cast<const void*>(&embed_count_kernel<r>), groups, 1024, argv, stream);
        if (f != hipSuccess) break;
        groups = grid();
        f = go(reinterpret_cast<const void*>(&embed_sort_kernel<r>), groups, 1024, argv, stream);
      }
      return f;
    });
  }
  if (e != hipSuccess) return e;
  m.chunk = d.chunk;
  m.chunks = d.chunks;
  const int sorted = d.tiles <= 1 ? 0 : (d.passes - 1) & 1;
  m.key = s.key[sorted];
  m.place = s.place[sorted];
  m.touched = s.touched;
  m.partial = reinterpret_cast<float*>(workspace + d.partial);
  return with_type(dtype, a.width, [&](auto dt, auto ve) {
    const uint64_t pieces = (a.width + ve * 64 - 1) / (ve * 64);
    const uint64_t units = uint64_t(d.chunks) * pieces;
    m.clear_rows = std::max<uint32_t>(8, a.vocab >> 22);  // at most 2^20 workgroups
    const uint64_t clear = accumulate || d.clear_all ? 0 : (uint64_t(a.vocab) + 4 * m.clear_rows - 1) / (4 * m.clear_rows);
    m.sum_groups = static_cast<uint32_t>((units + 3) / 4);
    const bool wide = grad_dtype == kF32 && dt != kF32;
    void* argv[] = {&m};
    const void* sum = wide ? reinterpret_cast<const void*>(&embed_sum_kernel<dt, kF32, ve>)
                           : reinterpret_cast<const void*>(&embed_sum_kernel<dt, dt, ve>);
    const void* join = wide ? reinterpret_cast<const void*>(&embed_join_kernel<dt, kF32, ve>)
                            : reinterpret_cast<const void*>(&embed_join_kernel<dt, dt, ve>);
    hipError_t r = m.sum_groups + clear == 0 ? hipSuccess : go(sum, m.sum_groups + clear, 256, argv, stream);
    if (r == hipSuccess && d.chunks > 1) r = go(join, (d.chunks - 1) * pieces, 256, argv, stream);
    return r;
  });
}

}  // namespace hbmc
