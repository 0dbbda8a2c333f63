// The embedding whose rows are dealt out to the ranks, and the gradient of its
// table by sorted tokens (see hbmc_embedding).
//
// The lookup copies rows: HBM bound, a wave a piece of 256 vectors of a row.
//
// The gradient sorts (id, place) pairs, place = rank << 26 | token, with a
// stable radix sort of two digits (three above 2^20 ids), so that a row's
// tokens lie together in a fixed order; then a wave adds up `chunk` sorted
// tokens of 64 vectors' columns, writing every id's row that lies within the
// chunk and leaving the sums of a first or last id that other chunks share to
// a small joining kernel.  No float is added atomically, so the sums' order,
// and with it every bit, is fixed.  It reads each gradient row once: HBM bound
// but for the sort, whose launches are what a small call costs.
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

constexpr uint32_t kPiece = 4;  // vectors a lane copies of a row

template <int DT, int VE>
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
      K::store(to + uint64_t(c.at) * K::E, K::narrow(f));
    }
  }
}

// ---------------------------------------------------------------- the sort

struct SortArgs {
  const unsigned char* ids[kMaxRanks];
  uint32_t tokens[kMaxRanks];
  int P, id_bytes;
  uint32_t vocab, total, tile, tiles, bits, passes;
  uint32_t* hist;     // [passes][tiles][kMaxBins]
  uint32_t* key[2];   // sorted so far, and place beside it
  uint32_t* place[2];
  uint32_t* touched;  // a bit for each id that occurs, or nullptr
};

// Ranks' first tokens among all ranks' (before[P] = total) in LDS.
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

__device__ __forceinline__ void read_pair(const SortArgs& a, const uint32_t* before, uint32_t pass, uint32_t i,
                                          uint32_t* key, uint32_t* place) {
  if (pass == 0) {
    *key = token_key(a, before, i, place);
  } else {
    *key = a.key[(pass + 1) & 1][i];
    *place = a.place[(pass + 1) & 1][i];
  }
}

// First pass over the ids: the first digit's counts in each tile; clears the
// later digits' counts and the touched bits.
__global__ __launch_bounds__(1024) void embed_count_kernel(SortArgs a) {
  __shared__ uint32_t before[64], bins[kMaxBins];
  const uint32_t n = 1u << a.bits;
  rank_starts(a, before);
  bins[threadIdx.x] = 0;
  __syncthreads();
  const uint32_t lo = blockIdx.x * a.tile, hi = min(lo + a.tile, a.total);
  for (uint32_t i = lo + threadIdx.x; i < hi; i += 1024) {
    uint32_t place;
    atomicAdd(&bins[token_key(a, before, i, &place) & (n - 1)], 1u);
  }
  __syncthreads();
  a.hist[blockIdx.x * kMaxBins + threadIdx.x] = bins[threadIdx.x];
  for (uint32_t p = 1; p < a.passes; ++p) a.hist[(p * a.tiles + blockIdx.x) * kMaxBins + threadIdx.x] = 0;
  if (a.touched)
    for (uint32_t w = blockIdx.x * 1024 + threadIdx.x; w < (a.vocab + 31) / 32; w += gridDim.x * 1024) a.touched[w] = 0;
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

// One stable pass over a tile's pairs.  Every wave counts its own stretch of
// the tile by digit, the counts become each wave's first positions, and the
// wave places its pairs in order.
template <bool SINGLE>
__device__ __forceinline__ void sort_pass(const SortArgs& a, const uint32_t* before, uint32_t pass, uint32_t (*count)[kMaxBins],
                                          uint32_t* scan) {
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t tile = SINGLE ? 0 : blockIdx.x;
  const uint32_t shift = pass * a.bits, mask = (1u << a.bits) - 1;
  const bool last = pass + 1 == a.passes;
  const uint32_t stretch = a.tile / kSortWaves;
  const uint32_t lo = tile * a.tile + wave * stretch;
  const uint64_t below = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (uint32_t w = 0; w < kSortWaves; ++w) count[w][threadIdx.x] = 0;
  __syncthreads();
  for (uint32_t r = 0; r < stretch && lo + r < a.total; r += 64) {
    const uint32_t i = lo + r + lane;
    const bool on = i < a.total;
    uint32_t key = 0, place;
    if (on) read_pair(a, before, pass, i, &key, &place);
    const uint32_t digit = key >> shift & mask;
    const uint64_t same = same_digit(digit, a.bits, on);
    if (on && (same & below) == 0) count[wave][digit] += __popcll(same);
    wave_order();
    // a frequent id's bit is mostly there already (an old value read only costs the atomic)
    if (pass == 0 && a.touched && on && key < a.vocab && !(a.touched[key >> 5] >> (key & 31) & 1))
      atomicOr(&a.touched[key >> 5], 1u << (key & 31));
  }
  __syncthreads();
  {
    // bin threadIdx.x: pairs in all tiles, and in the tiles before this one
    uint32_t all = 0, prior = 0;
    if constexpr (SINGLE) {
#pragma unroll
      for (uint32_t w = 0; w < kSortWaves; ++w) all += count[w][threadIdx.x];
    } else {
      const uint32_t* h = a.hist + uint64_t(pass) * a.tiles * kMaxBins + threadIdx.x;
#pragma unroll 8
      for (uint32_t t = 0; t < a.tiles; ++t) {
        const uint32_t c = h[t * kMaxBins];
        all += c;
        prior += t < tile ? c : 0;
      }
    }
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
  }
  __syncthreads();
  uint32_t* next = last ? nullptr : a.hist + uint64_t(pass + 1) * a.tiles * kMaxBins;
  for (uint32_t r = 0; r < stretch && lo + r < a.total; r += 64) {
    const uint32_t i = lo + r + lane;
    const bool on = i < a.total;
    uint32_t key = 0, place = 0;
    if (on) read_pair(a, before, pass, i, &key, &place);
    const uint32_t digit = key >> shift & mask;
    const uint64_t same = same_digit(digit, a.bits, on);
    const uint32_t to = on ? count[wave][digit] + __popcll(same & below) : 0;
    wave_order();
    if (on && (same & below) == 0) count[wave][digit] += __popcll(same);
    wave_order();
    if (on) {
      a.key[pass & 1][to] = key;
      a.place[pass & 1][to] = place;
      if constexpr (!SINGLE) {
        if (next) atomicAdd(&next[to / a.tile * kMaxBins + (key >> (shift + a.bits) & mask)], 1u);
      }
    }
  }
}

__global__ __launch_bounds__(1024) void embed_sort_kernel(SortArgs a, uint32_t pass) {
  __shared__ uint32_t before[64], scan[kSortWaves], count[kSortWaves][kMaxBins];
  rank_starts(a, before);
  sort_pass<false>(a, before, pass, count, scan);
}

// All passes of a call whose pairs are one tile.
__global__ __launch_bounds__(1024) void embed_sort_all_kernel(SortArgs a) {
  __shared__ uint32_t before[64], scan[kSortWaves], count[kSortWaves][kMaxBins];
  rank_starts(a, before);
  if (a.touched)
    for (uint32_t w = threadIdx.x; w < (a.vocab + 31) / 32; w += 1024) a.touched[w] = 0;
  for (uint32_t pass = 0; pass < a.passes; ++pass) {
    // the pairs of the last pass, and the cleared bits, before this one
    __threadfence();
    __syncthreads();
    sort_pass<true>(a, before, pass, count, scan);
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
  const uint32_t* touched;  // nullptr: add to the rows that occur, leave the others
  float* partial;           // [chunks][2][width]: of a chunk's first id, of its last
  uint32_t sum_groups;      // workgroups that add; those after them clear rows
  uint32_t clear_rows;      // rows a wave clears
};

// The finished sum of id `key`, at the lane's columns.
template <int DT, int GT, int VE>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, const Column<VE>& c, float (&acc)[VE]) {
  constexpr uint32_t G = Width<GT>::bytes;
  const uint32_t owner = key / a.seg;
  unsigned char* to = a.out[owner] + (uint64_t(key - owner * a.seg) * a.width + c.at) * G;
  if (!c.on) return;
#pragma unroll
  for (int i = 0; i < VE; ++i) acc[i] *= a.scale;
  if (a.touched == nullptr) {
    if (c.dup != 0) {
      // a row's last two lanes share columns; only one of them may add
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (i < static_cast<int>(c.dup)) continue;
        float old[1];
        Pack<GT, 1>::widen(Pack<GT, 1>::load(to + i * G), old);
        old[0] += acc[i];
        Pack<GT, 1>::store(to + i * G, Pack<GT, 1>::narrow(old));
      }
      return;
    }
    float old[VE];
    if constexpr (GT == DT) {
      Pack<GT, VE>::widen(Pack<GT, VE>::load(to), old);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) old[i] = reinterpret_cast<const float*>(to)[i];
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[i] += old[i];
  }
  if constexpr (GT == DT) Pack<GT, VE>::store(to, Pack<GT, VE>::narrow(acc));
  else store_floats<VE>(reinterpret_cast<float*>(to), acc);
}

template <int DT, int GT, int VE>
__global__ __launch_bounds__(256) void embed_sum_kernel(SumArgs a) {
  typedef Pack<DT, VE> K;
  const uint32_t lane = threadIdx.x & 63;
  if (blockIdx.x >= a.sum_groups) {
    constexpr int GE = VE == 1 ? 1 : 16 / Width<GT>::bytes;
    typedef Pack<GT, GE> Z;
    const uint32_t first = ((blockIdx.x - a.sum_groups) * 4 + uniform(threadIdx.x >> 6)) * a.clear_rows;
    for (uint32_t r = first; r < first + a.clear_rows && r < a.vocab; ++r) {
      if (a.touched[r >> 5] >> (r & 31) & 1) continue;
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
  uint32_t cur = uniform(a.key[lo]);
  if (cur >= a.vocab) return;  // tokens without a row come last
  bool shared = lo > 0 && uniform(a.key[lo > 0 ? lo - 1 : 0]) == cur;  // the current id began in an earlier chunk
  const uint32_t after = hi < a.total ? uniform(a.key[hi]) : a.vocab;
  float* partial = a.partial + uint64_t(chunk) * 2 * a.width + c.at;
  float acc[VE] = {};
  const auto finish = [&](bool goes_on) {
    if (!shared && !goes_on) write_row<DT, GT, VE>(a, cur, c, acc);
    else if (c.on) store_floats<VE>(partial + (shared ? 0 : a.width), acc);
  };
  for (uint32_t base = lo; base < hi; base += 64) {
    const uint32_t i = base + lane;
    const uint32_t keys = i < hi ? a.key[i] : a.vocab;
    const uint32_t places = i < hi ? a.place[i] : 0;
    const uint32_t n = __popcll(__ballot(keys < a.vocab));  // sorted: the first n lanes
    for (uint32_t t = 0; t < n; t += 8) {
      typename K::raw v[8];
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) {
        const uint32_t pl = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(places), min(t + u, n - 1)));
        const unsigned char* row = a.rows[pl >> kPlaceBits] + uint64_t(pl & ((1u << kPlaceBits) - 1)) * a.width * K::E;
        v[u] = K::stream(row + c.at * K::E);
      }
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) {
        if (t + u < n) {
          const uint32_t key = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(keys), t + u));
          if (key != cur) {
            finish(false);
#pragma unroll
            for (int i2 = 0; i2 < VE; ++i2) acc[i2] = 0.0f;
            cur = key;
            shared = false;
          }
          float f[VE];
          K::widen(v[u], f);
#pragma unroll
          for (int i2 = 0; i2 < VE; ++i2) acc[i2] += f[i2];
        }
      }
    }
    if (n < 64) break;
  }
  finish(after == cur);
}

// Joins the sums of an id that spans chunks: by the chunk it begins in.
template <int DT, int GT, int VE>
__global__ __launch_bounds__(256) void embed_join_kernel(SumArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t pieces = (a.width + VE * 64 - 1) / (VE * 64);
  const uint64_t unit = uint64_t(blockIdx.x) * 4 + uniform(threadIdx.x >> 6);
  const uint32_t chunk = static_cast<uint32_t>(unit / pieces);
  if (chunk + 1 >= a.chunks) return;
  const uint32_t lo = chunk * a.chunk, hi = lo + a.chunk;
  const uint32_t key = uniform(a.key[hi - 1]);
  if (key >= a.vocab || uniform(a.key[hi]) != key) return;                              // ends here
  if (lo > 0 && uniform(a.key[lo]) == key && uniform(a.key[lo - 1]) == key) return;     // began earlier
  const Column<VE> c(static_cast<uint32_t>(unit - uint64_t(chunk) * pieces) * 64 + lane, a.width);
  const float* head = a.partial + c.at;
  const uint64_t step = uint64_t(2) * a.width;
  float acc[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) acc[i] = head[chunk * step + a.width + i];
  for (uint32_t next = chunk + 1; next < a.chunks; next += 64) {
    const uint32_t mine = next + lane;
    const bool same = mine < a.chunks && a.key[uint64_t(mine) * a.chunk] == key;
    const uint32_t n = __popcll(__ballot(same));  // sorted: the first n of them
    uint32_t t = 0;
    for (; t + 4 <= n; t += 4) {
      float f[4][VE];
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < VE; ++i) f[u][i] = head[(next + t + u) * step + i];
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[i] += f[u][i];
    }
    for (; t < n; ++t)
#pragma unroll
      for (int i = 0; i < VE; ++i) acc[i] += head[(next + t) * step + i];
    if (n < 64) break;
  }
  write_row<DT, GT, VE>(a, key, c, acc);
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

constexpr uint32_t kSingleTile = 8192;  // tokens that one workgroup sorts by itself

}  // namespace

hipError_t launch_embed(int dtype, const EmbedArgs& a, hipStream_t stream) {
  uint64_t most = 0;
  for (int r = 0; r < a.P; ++r) most = std::max<uint64_t>(most, a.tokens[r]);
  return with_type(dtype, a.width, [&](auto dt, auto ve) {
    const uint64_t pieces = (a.width + ve * 64 * kPiece - 1) / (ve * 64 * kPiece);
    const uint64_t groups = std::min<uint64_t>((most * pieces + 3) / 4, 1 << 20);
    void* argv[] = {const_cast<EmbedArgs*>(&a)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&embed_kernel<dt, ve>),
                           dim3(static_cast<uint32_t>(groups), static_cast<uint32_t>(a.P)), dim3(256), argv, 0, stream);
  });
}

EmbedGradSplit split_embed_grad(int dtype, uint64_t total, uint64_t vocab, uint64_t width) {
  EmbedGradSplit d;
  d.total = total;
  uint32_t bits = 0;  // of the largest key, vocab itself
  while (vocab >> bits) ++bits;
  d.passes = (bits + 9) / 10;
  d.bits = (bits + d.passes - 1) / d.passes;
  // sorting workgroups: one for few tokens, else up to 64
  const uint64_t each = total <= kSingleTile ? total : (total + 63) / 64;
  d.tile = static_cast<uint32_t>((each + 1023) / 1024 * 1024);
  d.tiles = d.tile == 0 ? 0 : static_cast<uint32_t>((total + d.tile - 1) / d.tile);
  // tokens a wave adds up: enough waves to fill the chip, few sums to join
  const uint64_t pieces = (width + vector_elems(dtype, width) * 64 - 1) / (vector_elems(dtype, width) * 64);
  d.chunk = 16;
  while (d.chunk < 256 && total * pieces / d.chunk > 16384) d.chunk *= 2;
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
  d.hist = take(uint64_t(d.passes) * d.tiles * kMaxBins * 4);
  d.touched = take((vocab + 31) / 32 * 4);
  d.partial = take(uint64_t(d.chunks) * 2 * width * 4);
  d.bytes = at;
  return d;
}

hipError_t launch_embed_grad(int dtype, int grad_dtype, const EmbedArgs& a, const EmbedGradSplit& d, bool accumulate,
                             unsigned char* workspace, hipStream_t stream) {
  SortArgs s = {};
  for (int r = 0; r < a.P; ++r) {
    s.ids[r] = a.ids[r];
    s.tokens[r] = a.tokens[r];
  }
  s.P = a.P;
  s.id_bytes = a.id_bytes;
  s.vocab = a.vocab;
  s.total = static_cast<uint32_t>(d.total);
  s.tile = d.tile;
  s.tiles = d.tiles;
  s.bits = d.bits;
  s.passes = d.passes;
  s.hist = reinterpret_cast<uint32_t*>(workspace + d.hist);
  s.key[0] = reinterpret_cast<uint32_t*>(workspace + d.key_a);
  s.key[1] = reinterpret_cast<uint32_t*>(workspace + d.key_b);
  s.place[0] = reinterpret_cast<uint32_t*>(workspace + d.place_a);
  s.place[1] = reinterpret_cast<uint32_t*>(workspace + d.place_b);
  s.touched = accumulate ? nullptr : reinterpret_cast<uint32_t*>(workspace + d.touched);
  hipError_t e = hipSuccess;
  if (d.tiles <= 1) {
    // with no tokens at all it only clears the touched bits
    if (d.total == 0 && accumulate) return hipSuccess;
    void* argv[] = {&s};
    e = go(reinterpret_cast<const void*>(&embed_sort_all_kernel), 1, 1024, argv, stream);
  } else {
    void* argv[] = {&s};
    e = go(reinterpret_cast<const void*>(&embed_count_kernel), d.tiles, 1024, argv, stream);
    for (uint32_t pass = 0; e == hipSuccess && pass < d.passes; ++pass) {
      void* pargv[] = {&s, &pass};
      e = go(reinterpret_cast<const void*>(&embed_sort_kernel), d.tiles, 1024, pargv, stream);
    }
  }
  if (e != hipSuccess) return e;
  SumArgs m = {};
  for (int r = 0; r < a.P; ++r) {
    m.rows[r] = a.rows[r];
    m.out[r] = a.out[r];
  }
  m.seg = a.seg;
  m.vocab = a.vocab;
  m.width = a.width;
  m.total = s.total;
  m.chunk = d.chunk;
  m.chunks = d.chunks;
  m.scale = a.scale;
  m.key = s.key[(d.passes - 1) & 1];
  m.place = s.place[(d.passes - 1) & 1];
  m.touched = s.touched;
  m.partial = reinterpret_cast<float*>(workspace + d.partial);
  return with_type(dtype, a.width, [&](auto dt, auto ve) {
    const uint64_t pieces = (a.width + ve * 64 - 1) / (ve * 64);
    const uint64_t units = uint64_t(d.chunks) * pieces;
    m.clear_rows = std::max<uint32_t>(8, a.vocab >> 22);  // at most 2^20 workgroups
    const uint64_t clear = accumulate ? 0 : (uint64_t(a.vocab) + 4 * m.clear_rows - 1) / (4 * m.clear_rows);
    m.sum_groups = static_cast<uint32_t>((units + 3) / 4);
    const bool wide = grad_dtype == kF32 && dt != kF32;
    void* argv[] = {&m};
    const void* sum = wide ? reinterpret_cast<const void*>(&embed_sum_kernel<dt, kF32, ve>)
                           : reinterpret_cast<const void*>(&embed_sum_kernel<dt, dt, ve>);
    const void* join = wide ? reinterpret_cast<const void*>(&embed_join_kernel<dt, kF32, ve>)
                            : reinterpret_cast<const void*>(&embed_join_kernel<dt, dt, ve>);
    hipError_t r = m.sum_groups + clear == 0 ? hipSuccess : go(sum, m.sum_groups + clear, 256, argv, stream);
    if (r == hipSuccess && d.chunks > 1) r = go(join, m.sum_groups, 256, argv, stream);
    return r;
  });
}

}  // namespace hbmc
