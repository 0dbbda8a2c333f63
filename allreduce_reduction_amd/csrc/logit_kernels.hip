// Penalties for repeated tokens, biases and grammar masks on logits whose
// columns are dealt out to the ranks (see hbmc_adjust_logits).
//
// A workgroup takes a tile of one rank's columns of a row.  It counts the row's
// tokens that lie in its tile in LDS (one word a column: integer additions, so
// their order changes nothing and a token named often is penalised once), adds up
// the biases of each named column in list order, then passes over its columns
// once.  Columns that the mask forbids are not read; in place, columns that stay
// as they are are neither read nor written, and without a mask only the named
// columns are looked at.
//
// Alone, the pass over the columns runs at the rate of a copy (512 x 131072 bf16 under
// masks, 38 us).  With lists a workgroup's life is a chain of some five waits for
// memory, about 5 us, of which 32 waves a compute unit hide what they can: 256 rows of
// 131072 bf16 with 2048 tokens in place 29 us, without a mask, for its few named columns
// alone, 25; 128 x 200064 fp32 with 16384 tokens to other memory 47 us (217 MB, 4.6 TB/s),
// one row 4.3 us.  Every tile reads its row's tokens: 8 rows of 100000 in place 68 to 70 us,
// 6.4 MB of them read by each of a row's 64 workgroups.  Loading tokens by
// 16 bytes, lengths, biases and mask asked for before the first barrier, and finding a
// bias by its column's word took the 128 rows from 104 us to 48.
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

constexpr uint32_t kLogitThreads = 512;
constexpr uint32_t kTokenVectors = 2;  // 16-byte loads of tokens of a thread, in flight at once

// A column's word: its count in the row's output (19 bits), whether the row's
// prompt holds it, and the place of its bias plus one (12 bits; 0: none).
constexpr uint32_t kCountBits = 19, kPrompt = 1u << kCountBits, kCount = kPrompt - 1, kBiasShift = kCountBits + 1;
static_assert(kCount == kMaxHistory && (1u << (32 - kBiasShift)) - 1 == kMaxBias, "a word's fields");

// Every wave's accesses of LDS done.  No __syncthreads(): that would wait for the
// loads that are on their way to registers meanwhile.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ int64_t integer_at(const unsigned char* p, int bytes, uint64_t i) {
  return bytes == 8 ? reinterpret_cast<const int64_t*>(p)[i] : reinterpret_cast<const int32_t*>(p)[i];
}

struct Penalty {
  float repetition, frequency, presence;
};

__device__ __forceinline__ float adjust(float z, uint32_t word, const Penalty& p, const float* sums) {
  if (word & (kPrompt | kCount)) {
    z = z > 0.0f ? z / p.repetition : z * p.repetition;
    const uint32_t count = word & kCount;
    if (count) z = z - p.frequency * static_cast<float>(count) - p.presence;
  }
  if (word >> kBiasShift) z += sums[(word >> kBiasShift) - 1];
  return z;
}

// The mask's bits of the `N` columns from column c of a row; `one`: in one byte.
template <uint32_t N>
__device__ __forceinline__ uint32_t mask_bits(const unsigned char* row, uint32_t bytes, uint32_t c, bool one) {
  const uint32_t at = c >> 3;
  uint32_t b = row[at];
  if (!one && at + 1 < bytes) b |= static_cast<uint32_t>(row[at + 1]) << 8;
  return (b >> (c & 7)) & ((1u << N) - 1);
}

// A row's tokens, by the whole workgroup, several 16-byte loads a thread at once;
// the last few that fill no load are one thread's each.
template <int BYTES>
struct Tokens {
  static constexpr uint32_t N = 16 / BYTES, ROUND = kLogitThreads * kTokenVectors * N;
  const unsigned char* row;
  uint32_t history;
  u32x4 v[kTokenVectors];
  __device__ __forceinline__ uint32_t place(uint32_t base, uint32_t j) const { return base + (j * kLogitThreads + threadIdx.x) * N; }
  __device__ __forceinline__ void load(uint32_t base) {
    typedef u32x4 ids __attribute__((aligned(4)));
#pragma unroll
    for (uint32_t j = 0; j < kTokenVectors; ++j) {
      v[j] = u32x4{~0u, ~0u, ~0u, ~0u};
      if (place(base, j) + N <= history) v[j] = *reinterpret_cast<const ids*>(row + uint64_t(place(base, j)) * BYTES);
    }
  }
  // f(position, id - col0) for the tokens below `end` that are columns [col0, col0 + n),
  // the first round loaded before.
  template <typename F>
  __device__ __forceinline__ void each(uint32_t end, uint32_t col0, uint32_t n, F&& f) {
    for (uint32_t base = 0; base < end; base += ROUND) {
      if (base > 0) load(base);
#pragma unroll
      for (uint32_t j = 0; j < kTokenVectors; ++j) {
        const uint32_t at = place(base, j);
#pragma unroll
        for (uint32_t e = 0; e < N; ++e) {
          const uint32_t c = v[j][e * BYTES / 4] - col0;
          if (c < n && at + e < end && (BYTES == 4 || v[j][(e * BYTES / 4 + 1) % 4] == 0)) f(at + e, c);
        }
      }
    }
    const uint32_t last = history / N * N + threadIdx.x;
    if (threadIdx.x < N && last < end) {
      const int64_t id = integer_at(row, BYTES, last);
      if (id >= col0 && id < static_cast<int64_t>(col0) + n) f(last, static_cast<uint32_t>(id - col0));
    }
  }
};

// The type's -infinity, as often as a word holds it.
template <int DT>
constexpr uint32_t kMinusInfinity = DT == kF32 ? 0xff800000u : DT == kF16 ? 0xfc00fc00u : 0xff80ff80u;

constexpr uint32_t kLogitTile = 8192;  // columns of a workgroup at most

// How a tile's columns are passed over.
enum { kNamed = 0, kInPlace = 1, kApart = 2, kPast = 3 };  // named ones alone, in place; all, in place, to other memory, past the caches

// Where columns have several biases: the first of them gets its place into the column's
// word and adds up the others in their order.  Those others are marked, 64 of the list to
// a word of `follows`, and the first in `followed`, so that only the marked are compared:
// of 4095 biases with one repeated 18 us where 9 are all apart, not 1960 as when every
// bias is compared with all; with 409 repeated 28, every one twice 204, all of one column 486.
__device__ __forceinline__ void add_repeated(uint32_t* word, const int32_t* names, float* sums, uint32_t n, uint64_t* follows, uint32_t* followed) {
  const auto each = [&](auto&& f) {
    for (uint32_t i = threadIdx.x; i < n; i += kLogitThreads)
      if (names[i] >= 0) f(i, word + names[i]);
  };
  // the last place for every such column (the one bias that finds its own there by chance
  // is in it too), then the least
  for (uint32_t i = threadIdx.x; i * 32 < n; i += kLogitThreads) followed[i] = 0;
  each([&](uint32_t i, uint32_t* w) {
    if (*w >> kBiasShift != i + 1) atomicOr(w, ~0u << kBiasShift);
  });
  meet();
  each([&](uint32_t i, uint32_t* w) { atomicMin(w, (i + 1) << kBiasShift | (*w & (kPrompt | kCount))); });
  meet();
  for (uint32_t i = threadIdx.x; i < n; i += kLogitThreads) {
    const uint32_t first = names[i] >= 0 ? (word[names[i]] >> kBiasShift) - 1 : i;
    const uint64_t wave = __ballot(first != i);
    if (i % 64 == 0) follows[i / 64] = wave;
    if (first != i) atomicOr(followed + first / 32, 1u << first % 32);
  }
  meet();
  for (uint32_t i = threadIdx.x; i < n; i += kLogitThreads) {
    if (!(followed[i / 32] >> i % 32 & 1)) continue;
    float total = sums[i];
    for (uint32_t k0 = i / 64; k0 * 64 < n; ++k0)
      for (uint64_t left = follows[k0]; left; left &= left - 1) {
        const uint32_t k = k0 * 64 + static_cast<uint32_t>(__builtin_ctzll(left));
        if (names[k] == names[i]) total += sums[k];
      }
    sums[i] = total;
  }
}

template <int DT, bool LISTS, int PASS, int BYTES>
__global__ __launch_bounds__(kLogitThreads, 8) void adjust_logits(LogitArgs a) {
  typedef Pack<DT, 16 / Width<DT>::bytes> V;
  typedef Pack<DT, 1> One;
  constexpr uint32_t E = V::E, VE = 16 / E, kAll = (1u << VE) - 1;
  constexpr uint32_t VECTORS = E == 4 ? 4 : 2;  // of columns of a thread, in flight at once: a tile of 8192
  extern __shared__ __attribute__((aligned(16))) uint32_t words[];
  __shared__ uint32_t twice;  // whether a column of the tile has several biases
  __shared__ uint64_t follows[kMaxBias / 64 + 1];  // see add_repeated
  __shared__ uint32_t followed[kMaxBias / 32 + 1];
  const uint64_t row = blockIdx.x;
  const uint32_t rank = blockIdx.y;
  const uint64_t col = uint64_t(rank) * a.seg;
  const uint32_t cols = col < a.vocab ? min(a.seg, a.vocab - static_cast<uint32_t>(col)) : 0;
  const uint32_t first = blockIdx.z * a.tile;
  if (first >= cols) return;
  const uint32_t n = min(a.tile, cols - first), col0 = static_cast<uint32_t>(col) + first;
  const unsigned char* const in = a.logits[rank] + (row * cols + first) * E;
  unsigned char* const out = a.out[rank] + (row * cols + first) * E;
  // single columns before the first 16-byte boundary of the output and after the last
  const uint32_t head = min(n, (16 - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out)) & 15)) % 16 / E);
  const uint32_t vectors = (n - head) / VE, tail = head + vectors * VE;
  const uint32_t pad = (4 - head % 4) % 4;  // a vector's words begin on 16 bytes
  uint32_t* const word = words + pad;
  float* const sums = reinterpret_cast<float*>(words + (a.tile + 4));
  int32_t* const names = reinterpret_cast<int32_t*>(sums + a.biases);
  Penalty p = {1.0f, 0.0f, 0.0f};
  const unsigned char* const mask = PASS != kNamed && a.mask ? a.mask + row * a.mask_bytes : nullptr;
  const bool one_byte = (col0 + head) % VE == 0;  // a vector's bits of the mask
  uint32_t allowed[VECTORS];
  u32x4 z[VECTORS];
  const auto bits_of = [&](uint32_t v0) {
#pragma unroll
    for (uint32_t j = 0; j < VECTORS; ++j)
      allowed[j] = mask ? mask_bits<VE>(mask, a.mask_bytes, col0 + head + min(v0 + j * kLogitThreads, vectors - 1) * VE, one_byte) : kAll;
  };
  const auto load = [&](uint32_t v, uint32_t j) {
    const unsigned char* const from = in + uint64_t(head + v * VE) * E;
    z[j] = PASS == kPast ? V::stream(from) : V::load(from);
  };
  // what is read whatever the lists hold: in place, columns that the mask forbids in part
  const auto load_early = [&](uint32_t v0) {
#pragma unroll
    for (uint32_t j = 0; j < VECTORS; ++j)
      if (v0 + j * kLogitThreads < vectors && allowed[j] != 0 && (PASS != kInPlace || allowed[j] != kAll)) load(v0 + j * kLogitThreads, j);
  };
  if constexpr (LISTS) {
    // All that is known where to find is asked for before the first barrier.
    Tokens<BYTES> tokens{a.tokens + row * a.history * BYTES, a.tokens ? a.history : 0, {}};
    uint32_t end = 0, start = 0;
    if (a.tokens) {
      tokens.load(0);
      int64_t length = a.lengths ? integer_at(a.lengths, a.length_bytes, row) : a.history;
      length = min(max(length, int64_t(0)), static_cast<int64_t>(a.history));
      const int64_t prompt = a.prompt_lengths ? integer_at(a.prompt_lengths, a.length_bytes, row) : 0;
      end = static_cast<uint32_t>(length);
      start = static_cast<uint32_t>(min(max(prompt, int64_t(0)), length));
      if (a.repetition) p.repetition = a.repetition[row];
      if (a.frequency) p.frequency = a.frequency[row];
      if (a.presence) p.presence = a.presence[row];
    }
    int64_t bias_id = -1;
    float bias = 0.0f;
    const auto load_bias = [&](uint32_t i) {
      bias_id = integer_at(a.bias_ids, a.bias_id_bytes, row * a.biases + i);
      bias = a.bias[row * a.biases + i];
    };
    if (threadIdx.x < a.biases) load_bias(threadIdx.x);
    if constexpr (PASS != kNamed) {
      if (vectors > 0) bits_of(threadIdx.x);
    }
    for (uint32_t i = threadIdx.x; i < (pad + n + 3) / 4; i += kLogitThreads) reinterpret_cast<u32x4*>(words)[i] = u32x4{0, 0, 0, 0};
    if (threadIdx.x == 0) twice = 0;
    meet();
    // Biases add their place plus one to a column's word: of several that name one
    // column, at most one then finds its own there.
    for (uint32_t i = threadIdx.x; i < a.biases; i += kLogitThreads) {
      if (i >= kLogitThreads) load_bias(i);
      sums[i] = bias;
      const bool mine = bias_id >= col0 && bias_id < static_cast<int64_t>(col0) + n;
      names[i] = mine ? static_cast<int32_t>(bias_id - col0) : -1;
      if (mine) atomicAdd(word + names[i], (i + 1) << kBiasShift);
    }
    if constexpr (PASS != kNamed) load_early(threadIdx.x);
    const bool prompts = a.repetition != nullptr;
    tokens.each(end, col0, n, [&](uint32_t i, uint32_t c) {
      if (i >= start) atomicAdd(word + c, 1u);
      else if (prompts) atomicOr(word + c, kPrompt);
    });
    meet();
    if (a.biases) {
      for (uint32_t i = threadIdx.x; i < a.biases; i += kLogitThreads)
        if (names[i] >= 0 && word[names[i]] >> kBiasShift != i + 1) twice = 1;
      meet();
      if (twice) {
        add_repeated(word, names, sums, a.biases, follows, followed);
        meet();
      }
    }
    if constexpr (PASS == kNamed) {
      // each named column by the first thread to come for it
      const auto visit = [&](uint32_t c) {
        const uint32_t w = word[c] ? atomicExch(word + c, 0u) : 0;
        if (w == 0) return;
        float f[1];
        One::widen(One::load(in + uint64_t(c) * E), f);
        f[0] = adjust(f[0], w, p, sums);
        One::store(out + uint64_t(c) * E, One::narrow(f));
      };
      for (uint32_t i = threadIdx.x; i < a.biases; i += kLogitThreads)
        if (names[i] >= 0) visit(static_cast<uint32_t>(names[i]));
      if (end > Tokens<BYTES>::ROUND) tokens.load(0);
      tokens.each(end, col0, n, [&](uint32_t, uint32_t c) { visit(c); });
      return;
    }
  }
  for (uint32_t v0 = threadIdx.x; v0 < vectors; v0 += kLogitThreads * VECTORS) {
    if (!LISTS || v0 >= kLogitThreads * VECTORS) {
      bits_of(v0);
      load_early(v0);
    }
    // the words of vector v of the tile, and whether any of them is not zero
    const auto words_of = [&](uint32_t v, uint32_t (&w)[VE]) {
      uint32_t any = 0;
#pragma unroll
      for (uint32_t e = 0; e < VE; e += 4) {
        const u32x4 four = *reinterpret_cast<const u32x4*>(word + head + v * VE + e);
        w[e] = four.x, w[e + 1] = four.y, w[e + 2] = four.z, w[e + 3] = four.w;
        any |= four.x | four.y | four.z | four.w;
      }
      return any != 0;
    };
    bool on[VECTORS], lists[VECTORS];
#pragma unroll
    for (uint32_t j = 0; j < VECTORS; ++j) {
      const uint32_t v = v0 + j * kLogitThreads;
      uint32_t w[VE];
      on[j] = v < vectors;
      lists[j] = LISTS && on[j] && allowed[j] != 0 && words_of(v, w);
      if constexpr (PASS == kInPlace) {
        if (on[j] && allowed[j] == kAll) {
          on[j] = lists[j];
          if (on[j]) load(v, j);
        }
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < VECTORS; ++j) {
      if (!on[j]) continue;
      const uint32_t v = v0 + j * kLogitThreads;
      if (lists[j]) {
        uint32_t w[VE];
        words_of(v, w);
        // each alone: converting its neighbours too would set a signalling NaN's quiet bit
#pragma unroll
        for (uint32_t e = 0; e < VE; ++e) {
          if (w[e] == 0) continue;
          const uint32_t shift = e * E % 4 * 8, bits = E == 4 ? ~0u : 0xffffu << shift, at = e * E / 4;
          float f[1];
          One::widen(E == 4 ? z[j][at] : z[j][at] >> shift & 0xffffu, f);
          f[0] = adjust(f[0], w[e], p, sums);
          z[j][at] = (z[j][at] & ~bits) | One::narrow(f) << shift;
        }
      }
      if (mask) {
        // -infinity over the forbidden columns' bits
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          if constexpr (E == 4) {
            z[j][e] = allowed[j] >> e & 1 ? z[j][e] : kMinusInfinity<DT>;
          } else {
            const uint32_t low = static_cast<uint32_t>(static_cast<int32_t>(allowed[j] << (31 - 2 * e)) >> 31) & 0xffffu;
            const uint32_t high = static_cast<uint32_t>(static_cast<int32_t>(allowed[j] << (30 - 2 * e)) >> 31) & 0xffff0000u;
            const uint32_t keep = low | high;
            z[j][e] = (z[j][e] & keep) | (kMinusInfinity<DT> & ~keep);
          }
        }
      }
      unsigned char* const to = out + uint64_t(head + v * VE) * E;
      if constexpr (PASS == kPast) V::store_nt(to, z[j]);
      else V::store(to, z[j]);
    }
  }
  // the single columns: `head` before the vectors and fewer than a vector after
  uint32_t c = threadIdx.x;
  if (c >= head) c += tail - head;
  if (c < n) {
    const uint32_t w = LISTS ? word[c] : 0;
    const bool allowed = !mask || mask_bits<1>(mask, a.mask_bytes, col0 + c, true);
    if (!(PASS == kInPlace && allowed && w == 0)) {
      typename One::raw r = kMinusInfinity<DT> >> (32 - 8 * E);
      if (allowed) {
        r = One::load(in + uint64_t(c) * E);
        if (w) {
          float f[1];
          One::widen(r, f);
          f[0] = adjust(f[0], w, p, sums);
          r = One::narrow(f);
        }
      }
      One::store(out + uint64_t(c) * E, r);
    }
  }
}

}  // namespace dev

// Tiles of 8192 columns, whose words leave a compute unit four workgroups; smaller
// ones only where they would leave compute units without work, since every tile
// reads all of its row's tokens.  bf16, 8 ranks of 131072 columns in all, 2048
// tokens, tiles of 8192, 4096 and 2048: 256 rows 31, 42 and 71 us, 8 rows 6.4, 5.3 and
// 5.6, one row 5.4, 4.6 and 4.4.
uint32_t logit_tile(uint64_t rows, uint64_t seg, int P) {
  uint64_t tile = dev::kLogitTile;
  while (tile > 2048 && rows * static_cast<uint64_t>(P) * ((seg + tile - 1) / tile) < 512) tile /= 2;
  return static_cast<uint32_t>(std::min<uint64_t>(tile, (seg + 3) / 4 * 4));
}

namespace {

template <int DT>
hipError_t launch(const LogitArgs& a, hipStream_t stream) {
  // rows first: with rows in eights, a row's tiles share an XCD and its tokens the L2
  const dim3 grid(static_cast<uint32_t>(a.rows), static_cast<uint32_t>(a.P), a.tiles);
  const uint32_t lds = a.tokens || a.biases ? (a.tile + 4 + 2 * a.biases) * 4 : 0;
  const bool lists = a.tokens || a.biases, past = a.rows * a.vocab * dev::Width<DT>::bytes >= kStreamBytes;
  const int pass = a.in_place ? (a.mask ? dev::kInPlace : dev::kNamed) : past ? dev::kPast : dev::kApart;
  const auto go = [&](auto kernel) { kernel<<<grid, dev::kLogitThreads, lds, stream>>>(a); };
  const auto listed = [&](auto bytes) {
    constexpr int BYTES = decltype(bytes)::value;
    if (pass == dev::kNamed) go(dev::adjust_logits<DT, true, dev::kNamed, BYTES>);
    else if (pass == dev::kInPlace) go(dev::adjust_logits<DT, true, dev::kInPlace, BYTES>);
    else if (pass == dev::kApart) go(dev::adjust_logits<DT, true, dev::kApart, BYTES>);
    else go(dev::adjust_logits<DT, true, dev::kPast, BYTES>);
  };
  if (lists && a.tokens && a.id_bytes == 8) listed(std::integral_constant<int, 8>{});
  else if (lists) listed(std::integral_constant<int, 4>{});
  else if (pass == dev::kInPlace) go(dev::adjust_logits<DT, false, dev::kInPlace, 4>);
  else if (pass == dev::kApart) go(dev::adjust_logits<DT, false, dev::kApart, 4>);
  else go(dev::adjust_logits<DT, false, dev::kPast, 4>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logits(int dtype, const LogitArgs& a, hipStream_t stream) {
  return dtype == dev::kF32 ? launch<dev::kF32>(a, stream) : dtype == dev::kF16 ? launch<dev::kF16>(a, stream) : launch<dev::kBF16>(a, stream);
}

}  // namespace hbmc
