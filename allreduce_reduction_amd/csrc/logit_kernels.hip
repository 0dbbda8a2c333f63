// Penalties for repeated tokens, biases and grammar masks on logits whose
// columns are dealt out to the ranks (see hbmc_adjust_logits).
//
// A workgroup takes a tile of one rank's columns of a row.  It counts the row's
// tokens that lie in its tile in LDS (one word a column: integer additions, so
// their order changes nothing and a token named often is penalised once), adds up
// the biases of each named column in list order, then passes over its columns
// once.  Columns that the mask forbids are not read; in place, columns that stay
// as they are are neither read nor written.
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

constexpr uint32_t kLogitThreads = 512;
constexpr uint32_t kLogitVectors = 2;  // of a thread, in flight at once

// A column's word: its count in the row's output (19 bits), whether the row holds
// it at all, and the place of its bias plus one (12 bits).
constexpr uint32_t kCountBits = 19, kSeen = 1u << kCountBits, kCount = kSeen - 1, kBiasShift = kCountBits + 1;

__device__ __forceinline__ int64_t integer_at(const unsigned char* p, int bytes, uint64_t i) {
  return bytes == 8 ? reinterpret_cast<const int64_t*>(p)[i] : reinterpret_cast<const int32_t*>(p)[i];
}

struct Penalty {
  float repetition, frequency, presence;
};

__device__ __forceinline__ float adjust(float z, uint32_t word, const Penalty& p, const float* sums) {
  if (word & (kSeen | kCount)) {
    if (word & kSeen) z = z > 0.0f ? z / p.repetition : z * p.repetition;
    const uint32_t count = word & kCount;
    if (count) z = z - p.frequency * static_cast<float>(count) - p.presence;
  }
  if (word >> kBiasShift) z += sums[(word >> kBiasShift) - 1];
  return z;
}

// The mask's bits of the `N` columns from column c of a row.
template <uint32_t N>
__device__ __forceinline__ uint32_t mask_bits(const unsigned char* row, uint32_t bytes, uint32_t c) {
  const uint32_t at = c >> 3;
  uint32_t b = row[at];
  if ((c & 7) + N > 8 && at + 1 < bytes) b |= static_cast<uint32_t>(row[at + 1]) << 8;
  return (b >> (c & 7)) & ((1u << N) - 1);
}

template <int DT>
__global__ __launch_bounds__(kLogitThreads) void adjust_logits(LogitArgs a) {
  typedef Pack<DT, 16 / Width<DT>::bytes> V;
  typedef Pack<DT, 1> One;
  constexpr uint32_t E = V::E, VE = 16 / E, kAll = (1u << VE) - 1;
  extern __shared__ __attribute__((aligned(16))) uint32_t words[];
  const uint32_t per_row = static_cast<uint32_t>(a.P) * a.tiles;
  const uint64_t row = blockIdx.x / per_row;
  const uint32_t at = blockIdx.x % per_row, rank = at / a.tiles;
  const uint64_t col = uint64_t(rank) * a.seg;
  const uint32_t cols = col < a.vocab ? min(a.seg, a.vocab - static_cast<uint32_t>(col)) : 0;
  const uint32_t first = (at % a.tiles) * a.tile;
  if (first >= cols) return;
  const uint32_t n = min(a.tile, cols - first), col0 = static_cast<uint32_t>(col) + first;
  const unsigned char* const in = a.logits[rank] + (row * cols + first) * E;
  unsigned char* const out = a.out[rank] + (row * cols + first) * E;
  // single columns before the first 16-byte boundary of the output and after the last
  const uint32_t head = min(n, (16 - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out)) & 15)) % 16 / E);
  const uint32_t vectors = (n - head) / VE, tail = head + vectors * VE;
  const uint32_t pad = (4 - head % 4) % 4;  // a vector's words begin on 16 bytes
  const bool lists = a.tokens || a.biases;
  uint32_t* const word = words + pad;
  float* const sums = reinterpret_cast<float*>(words + (a.tile + 4));
  int32_t* const names = reinterpret_cast<int32_t*>(sums + a.biases);
  Penalty p = {1.0f, 0.0f, 0.0f};
  if (lists) {
    for (uint32_t i = threadIdx.x; i < n; i += kLogitThreads) word[i] = 0;
    for (uint32_t i = threadIdx.x; i < a.biases; i += kLogitThreads) {
      const int64_t id = integer_at(a.bias_ids, a.bias_id_bytes, row * a.biases + i);
      names[i] = id >= col0 && id < static_cast<int64_t>(col0) + n ? static_cast<int32_t>(id - col0) : -1;
      sums[i] = a.bias[row * a.biases + i];
    }
    __syncthreads();
    if (a.tokens) {
      int64_t length = a.lengths ? integer_at(a.lengths, a.length_bytes, row) : a.history;
      length = min(max(length, int64_t(0)), static_cast<int64_t>(a.history));
      int64_t prompt = a.prompt_lengths ? integer_at(a.prompt_lengths, a.length_bytes, row) : 0;
      prompt = min(max(prompt, int64_t(0)), length);
      const uint32_t end = static_cast<uint32_t>(length), start = static_cast<uint32_t>(prompt);
      const uint64_t base = row * a.history;
      for (uint32_t i = threadIdx.x; i < end; i += kLogitThreads) {
        const int64_t id = integer_at(a.tokens, a.id_bytes, base + i);
        if (id >= col0 && id < static_cast<int64_t>(col0) + n) {
          uint32_t* const w = word + (id - col0);
          if (i >= start) atomicAdd(w, 1u);
          if (a.repetition) atomicOr(w, kSeen);
        }
      }
      if (a.repetition) p.repetition = a.repetition[row];
      if (a.frequency) p.frequency = a.frequency[row];
      if (a.presence) p.presence = a.presence[row];
    }
    // a named column's first entry adds up all of them
    float total[kMaxBias / kLogitThreads + 1];
#pragma unroll
    for (uint32_t h = 0; h < kMaxBias / kLogitThreads + 1; ++h) {
      const uint32_t i = threadIdx.x + h * kLogitThreads;
      total[h] = 0.0f;
      if (i < a.biases && names[i] >= 0) {
        bool leads = true;
        for (uint32_t k = 0; k < i; ++k) leads = leads && names[k] != names[i];
        total[h] = sums[i];
        for (uint32_t k = i + 1; k < a.biases; ++k)
          if (names[k] == names[i]) total[h] += sums[k];
        if (leads) atomicOr(word + names[i], (i + 1) << kBiasShift);
      }
    }
    if (a.biases) {
      __syncthreads();
#pragma unroll
      for (uint32_t h = 0; h < kMaxBias / kLogitThreads + 1; ++h) {
        const uint32_t i = threadIdx.x + h * kLogitThreads;
        if (i < a.biases) sums[i] = total[h];
      }
    }
    __syncthreads();
  }
  const unsigned char* const mask = a.mask ? a.mask + row * a.mask_bytes : nullptr;
  const float masked = -__builtin_inff();
  for (uint32_t v0 = threadIdx.x; v0 < vectors; v0 += kLogitThreads * kLogitVectors) {
    u32x4 z[kLogitVectors];
    uint32_t allowed[kLogitVectors], w[kLogitVectors][VE];
    bool on[kLogitVectors];
#pragma unroll
    for (uint32_t j = 0; j < kLogitVectors; ++j) {
      const uint32_t v = v0 + j * kLogitThreads, c = head + v * VE;
      on[j] = v < vectors;
      allowed[j] = kAll;
      uint32_t any = 0;
#pragma unroll
      for (uint32_t e = 0; e < VE; ++e) w[j][e] = 0;
      if (on[j]) {
        if (mask) allowed[j] = mask_bits<VE>(mask, a.mask_bytes, col0 + c);
        if (lists) {
#pragma unroll
          for (uint32_t e = 0; e < VE; e += 4) {
            const u32x4 four = *reinterpret_cast<const u32x4*>(word + c + e);
            w[j][e] = four.x, w[j][e + 1] = four.y, w[j][e + 2] = four.z, w[j][e + 3] = four.w;
            any |= four.x | four.y | four.z | four.w;
          }
        }
        if (a.in_place && allowed[j] == kAll && any == 0) on[j] = false;
        else if (allowed[j] != 0) z[j] = V::load(in + uint64_t(c) * E);
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < kLogitVectors; ++j) {
      if (!on[j]) continue;
      float f[VE];
      uint32_t any = 0;
#pragma unroll
      for (uint32_t e = 0; e < VE; ++e) any |= w[j][e];
      if (any != 0 || allowed[j] != kAll) {
        V::widen(z[j], f);
#pragma unroll
        for (uint32_t e = 0; e < VE; ++e) {
          if (w[j][e]) f[e] = adjust(f[e], w[j][e], p, sums);
          if (!(allowed[j] >> e & 1)) f[e] = masked;
        }
        z[j] = V::narrow(f);
      }
      V::store(out + uint64_t(head + (v0 + j * kLogitThreads) * VE) * E, z[j]);
    }
  }
  // the single columns: `head` before the vectors and fewer than a vector after
  uint32_t c = threadIdx.x;
  if (c >= head) c += tail - head;
  if (c < n) {
    const uint32_t w = lists ? word[c] : 0;
    const bool allowed = !mask || mask_bits<1>(mask, a.mask_bytes, col0 + c);
    if (!(a.in_place && allowed && w == 0)) {
      float f[1] = {masked};
      typename One::raw r = One::narrow(f);
      if (allowed) {
        r = One::load(in + uint64_t(c) * E);
        if (w) {
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

uint32_t logit_tile(int dtype, uint64_t rows, uint64_t seg, int P) {
  (void)dtype, (void)rows, (void)P;
  return static_cast<uint32_t>(std::min<uint64_t>(8192, (seg + 3) / 4 * 4));
}

hipError_t launch_logits(int dtype, const LogitArgs& a, hipStream_t stream) {
  const uint32_t grid = static_cast<uint32_t>(a.rows * a.tiles * static_cast<uint64_t>(a.P));
  const uint32_t lds = a.tokens || a.biases ? (a.tile + 4 + 2 * a.biases) * 4 : 0;
  if (dtype == dev::kF32) dev::adjust_logits<dev::kF32><<<grid, dev::kLogitThreads, lds, stream>>>(a);
  else if (dtype == dev::kF16) dev::adjust_logits<dev::kF16><<<grid, dev::kLogitThreads, lds, stream>>>(a);
  else dev::adjust_logits<dev::kBF16><<<grid, dev::kLogitThreads, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace hbmc
