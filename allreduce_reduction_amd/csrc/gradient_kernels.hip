// The global norm of many gradient tensors, and their clipping (see
// hbmc_gradients_clip).
//
// No gradient can be scaled before the last has been read, so the data is passed
// over twice: a launch leaves one partial sum a workgroup, and the next joins
// them and scales: every workgroup by itself, in the same order, or with many
// pieces (kGradJoined) by a factor that a launch between them leaves.  Sums are kept
// in 64 bits, so that no square overflows, none is lost, and the norm is that of the
// gradients rounded once to 32 whatever their number.
//
// HBM bounds large calls: 268 million fp32 gradients (1.07 GB) are gathered in 161 us
// (6.6 TB/s) and clipped in 526 (6.1 TB/s over both reads and the writes); 8 copies of
// 48 million bf16 gathered from one and written in 176 us.  Small calls are two
// launches' latency: 1 million on one rank 8.7 us.
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

constexpr uint32_t kGradThreads = 256, kGradVectors = 4;  // of a piece: four vectors a thread
static_assert(kGradThreads * kGradVectors * 16 == kGradPieceBytes, "a piece is one round of its threads");

// What a thread gathers: sums of squares or of sizes, or the largest size, kept
// as its bits (a NaN's are above every number's).
template <int NORM>
struct Gather {
  double sum = 0.0;
  __device__ __forceinline__ void add(float x) {
    const double d = static_cast<double>(x);
    if constexpr (NORM == 2) sum = __builtin_fma(d, d, sum);
    else sum += __builtin_fabs(d);
  }
  __device__ __forceinline__ double value() const { return sum; }
};
template <>
struct Gather<0> {
  uint32_t top = 0;
  __device__ __forceinline__ void add(float x) { top = max(top, f2u(x) & 0x7fffffffu); }
  __device__ __forceinline__ double value() const { return static_cast<double>(u2f(top)); }
};

template <int NORM>
__device__ __forceinline__ double join(double a, double b) {
  if constexpr (NORM != 0) return a + b;
  const uint64_t x = __builtin_bit_cast(uint64_t, a), y = __builtin_bit_cast(uint64_t, b);
  return x > y ? a : b;  // sizes: their bits are in their order, a NaN's above
}

// Addresses of eight of a tensor's other copies.
struct Others {
  unsigned char* copy[8];
  __device__ __forceinline__ void load(const GradPiece& p, unsigned char* const* others, uint32_t from) {
    if (p.copies < 2) return;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) copy[k] = others[p.first + min(from + k, p.copies - 2u)];
  }
};

// A piece in the registers of the 256 threads `t` of it, as it lies in memory.
struct Held {
  u32x4 v[kGradVectors];
  uint32_t single;  // of the few elements that fill no vector
  template <int DT, bool STREAM>
  __device__ __forceinline__ void load(const GradPiece& p, uint32_t t) {
    typedef Pack<DT, 16 / Width<DT>::bytes> V;
    constexpr uint32_t VE = 16 / V::E;
    const uint32_t vectors = p.count / VE, last = vectors * VE + t;
#pragma unroll
    for (uint32_t j = 0; j < kGradVectors; ++j) {
      const uint32_t i = t + j * kGradThreads;
      v[j] = u32x4{0, 0, 0, 0};
      if (i < vectors) v[j] = STREAM ? V::stream(p.data + uint64_t(i) * 16) : V::load(p.data + uint64_t(i) * 16);
    }
    single = 0;
    if (last < p.count) single = Pack<DT, 1>::load(p.data + uint64_t(last) * V::E);
  }
  template <int DT, typename G>
  __device__ __forceinline__ void gather(G& g) const {
    typedef Pack<DT, 16 / Width<DT>::bytes> V;
    constexpr uint32_t VE = 16 / V::E;
    float f[VE], one[1];
#pragma unroll
    for (uint32_t j = 0; j < kGradVectors; ++j) {
      V::widen(v[j], f);
#pragma unroll
      for (uint32_t e = 0; e < VE; ++e) g.add(f[e]);
    }
    Pack<DT, 1>::widen(single, one);
    g.add(one[0]);
  }
  template <int DT>
  __device__ __forceinline__ void scale(float factor) {
    typedef Pack<DT, 16 / Width<DT>::bytes> V;
    constexpr uint32_t VE = 16 / V::E;
    float f[VE], one[1];
#pragma unroll
    for (uint32_t j = 0; j < kGradVectors; ++j) {
      V::widen(v[j], f);
#pragma unroll
      for (uint32_t e = 0; e < VE; ++e) f[e] *= factor;
      v[j] = V::narrow(f);
    }
    Pack<DT, 1>::widen(single, one);
    one[0] *= factor;
    single = Pack<DT, 1>::narrow(one);
  }
  template <int DT, bool STREAM>
  __device__ __forceinline__ void store(unsigned char* to, uint32_t count, uint32_t t) const {
    typedef Pack<DT, 16 / Width<DT>::bytes> V;
    constexpr uint32_t VE = 16 / V::E;
    const uint32_t vectors = count / VE, last = vectors * VE + t;
#pragma unroll
    for (uint32_t j = 0; j < kGradVectors; ++j) {
      const uint32_t i = t + j * kGradThreads;
      if (i >= vectors) continue;
      if constexpr (STREAM) V::store_nt(to + uint64_t(i) * 16, v[j]);
      else V::store(to + uint64_t(i) * 16, v[j]);
    }
    if (last < count) Pack<DT, 1>::store(to + uint64_t(last) * V::E, single);
  }
  // To a copy at another place in a line of 128 bytes than the piece, which lies in
  // `lds`: its vectors are put together there, since stores that cross 16 bytes are slow (8
  // copies of 48 million bf16 gradients, seven of them so: 234 us, and 176 so).
  template <int DT, bool STREAM>
  static __device__ __forceinline__ void store_shifted(unsigned char* to, const uint32_t* lds, uint32_t count, uint32_t t) {
    typedef Pack<DT, 16 / Width<DT>::bytes> V;
    constexpr uint32_t E = V::E, VE = 16 / E;
    const uint32_t head = min(count, (128 - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to)) & 127)) % 128 / E);
    const uint32_t vectors = (count - head) / VE, tail = head + vectors * VE;
#pragma unroll
    for (uint32_t j = 0; j < kGradVectors; ++j) {
      const uint32_t i = t + j * kGradThreads;
      if (i >= vectors) continue;
      const uint32_t at = head * E + i * 16, turn = at % 4 * 8;
      uint32_t w[5];
      u32x4 r;
#pragma unroll
      for (uint32_t k = 0; k < 5; ++k) w[k] = lds[at / 4 + k];
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) r[k] = __builtin_amdgcn_alignbit(w[k + 1], w[k], turn);
      if constexpr (STREAM) V::store_nt(to + at, r);
      else V::store(to + at, r);
    }
    uint32_t c = t;
    if (c >= head) c += tail - head;
    if (c < count) Pack<DT, 1>::store(to + uint64_t(c) * E, Pack<DT, 1>::load(reinterpret_cast<const unsigned char*>(lds) + c * E));
  }
  // To every copy of the piece, eight of their addresses at a time, the first of them
  // in `to`.  With `lds`, by way of it where a copy lies at another place in a line
  // (p.shifted: any does).
  template <int DT, bool STREAM>
  __device__ __forceinline__ void store_all(const GradPiece& p, unsigned char* const* others, uint32_t t, uint32_t* lds, Others to) const {
    constexpr uint32_t E = Width<DT>::bytes, VE = 16 / E;
    if (lds && p.shifted) {
      const uint32_t vectors = p.count / VE, last = vectors * VE + t;
#pragma unroll
      for (uint32_t j = 0; j < kGradVectors; ++j) {
        const uint32_t i = t + j * kGradThreads;
        if (i < vectors) *reinterpret_cast<u32x4*>(lds + i * 4) = v[j];
      }
      if (last < p.count) Pack<DT, 1>::store(reinterpret_cast<unsigned char*>(lds) + last * E, single);
      __syncthreads();
    }
    store<DT, STREAM>(p.data, p.count, t);
    for (uint32_t c = 0; c + 1 < p.copies; c += 8) {
      if (c > 0) to.load(p, others, c);
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        if (c + k + 1 >= p.copies) continue;
        unsigned char* const at = to.copy[k] + p.offset;
        if (lds && ((reinterpret_cast<uintptr_t>(at) ^ reinterpret_cast<uintptr_t>(p.data)) & 127) != 0) store_shifted<DT, STREAM>(at, lds, p.count, t);
        else store<DT, STREAM>(at, p.count, t);
      }
    }
  }
};

// f(type) for the piece's type.
template <typename F>
__device__ __forceinline__ void by_type(uint32_t dtype, F&& f) {
  if (dtype == kF32) f(std::integral_constant<int, kF32>{});
  else if (dtype == kF16) f(std::integral_constant<int, kF16>{});
  else f(std::integral_constant<int, kBF16>{});
}

// The workgroup's values joined, in every thread.
template <int NORM>
__device__ __forceinline__ double join_workgroup(double x, double* shared) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x = join<NORM>(x, __shfl_xor(x, d));
  if (threadIdx.x % 64 == 0) shared[threadIdx.x / 64] = x;
  __syncthreads();
  x = shared[0];
  for (uint32_t w = 1; w < blockDim.x / 64; ++w) x = join<NORM>(x, shared[w]);
  return x;
}

// The factor of every gradient, from the gathered total.
template <int NORM>
__device__ __forceinline__ float factor_of(const GradArgs& a, double total, bool writes) {
  const double norm = __builtin_fabs(a.scale) * (NORM == 2 ? __builtin_sqrt(total) : total);
  if (writes) *a.norm_out = static_cast<float>(norm);
  const double most = norm + a.eps;
  const double clip = a.max_norm >= most ? 1.0 : a.max_norm / most;
  return static_cast<float>(a.scale * clip);
}

// One partial sum a workgroup, over every gridDim.x-th piece, whose record is on
// its way while the piece before is read.
template <int NORM, bool STREAM>
__global__ __launch_bounds__(kGradThreads) void grad_gather(GradArgs a) {
  __shared__ double shared[kGradThreads / 64];
  Gather<NORM> g;
  GradPiece next = a.pieces[blockIdx.x];
  for (uint32_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    const GradPiece p = next;
    if (i + gridDim.x < a.n) next = a.pieces[i + gridDim.x];
    by_type(p.dtype, [&](auto type) {
      Held h;
      h.load<decltype(type)::value, STREAM>(p, threadIdx.x);
      h.gather<decltype(type)::value>(g);
    });
  }
  const double x = join_workgroup<NORM>(g.value(), shared);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = x;
}

// The partial sums joined, in every thread.
template <int NORM>
__device__ __forceinline__ double join_partial(const GradArgs& a, double* shared) {
  double x = 0.0;
  for (uint32_t i = threadIdx.x; i < a.sums; i += kGradThreads) x = join<NORM>(x, a.partial[i]);
  return join_workgroup<NORM>(x, shared);
}

// The norm, and the factor to where the partial sums end.
template <int NORM>
__global__ __launch_bounds__(kGradThreads) void grad_factor(GradArgs a) {
  __shared__ double shared[kGradThreads / 64];
  const float factor = factor_of<NORM>(a, join_partial<NORM>(a, shared), threadIdx.x == 0);
  if (threadIdx.x == 0) *reinterpret_cast<float*>(a.partial + a.sums) = factor;
}

// The pieces scaled, a workgroup each.  FACTOR: by the factor that grad_factor left;
// else (few pieces) every workgroup joins the partial sums itself, while its piece
// is read.  Last pieces first: what was gathered last may still be cached.
template <int NORM, bool FACTOR, bool STREAM>
__global__ __launch_bounds__(kGradThreads) void grad_scale(GradArgs a) {
  __shared__ double shared[kGradThreads / 64];
  __shared__ __attribute__((aligned(16))) uint32_t lds[kGradPieceBytes / 4 + 4];
  const GradPiece p = a.pieces[a.n - 1 - blockIdx.x];
  float factor = 1.0f;
  if constexpr (FACTOR) {
    factor = *reinterpret_cast<const float*>(a.partial + a.sums);
    if (factor == 1.0f) return;
  }
  by_type(p.dtype, [&](auto type) {
    constexpr int DT = decltype(type)::value;
    Held h;
    Others to;
    h.load<DT, STREAM>(p, threadIdx.x);
    to.load(p, a.others, 0);
    if constexpr (!FACTOR) factor = factor_of<NORM>(a, join_partial<NORM>(a, shared), blockIdx.x == 0 && threadIdx.x == 0);
    if (factor == 1.0f) return;
    h.scale<DT>(factor);
    h.store_all<DT, STREAM>(p, a.others, threadIdx.x, lds, to);
  });
}

// Few pieces: one workgroup of four groups of 256 threads holds them, so that they
// are read once, by one launch.
constexpr uint32_t kFewGroups = 4, kFewRounds = 2;

template <int NORM>
__global__ __launch_bounds__(kGradThreads * kFewGroups) void grad_few(GradArgs a) {
  __shared__ double shared[kGradThreads * kFewGroups / 64];
  const uint32_t group = uniform(threadIdx.x / kGradThreads), t = threadIdx.x % kGradThreads;
  Gather<NORM> g;
  Held h[kFewRounds];
#pragma unroll
  for (uint32_t r = 0; r < kFewRounds; ++r)
    if (group + r * kFewGroups < a.n) {
      const GradPiece p = a.pieces[group + r * kFewGroups];
      by_type(p.dtype, [&](auto type) { h[r].template load<decltype(type)::value, false>(p, t); });
    }
#pragma unroll
  for (uint32_t r = 0; r < kFewRounds; ++r)
    if (group + r * kFewGroups < a.n)
      by_type(a.pieces[group + r * kFewGroups].dtype, [&](auto type) { h[r].template gather<decltype(type)::value>(g); });
  const double x = join_workgroup<NORM>(g.value(), shared);
  const float factor = factor_of<NORM>(a, x, threadIdx.x == 0);
  if (!a.clip || factor == 1.0f) return;
#pragma unroll
  for (uint32_t r = 0; r < kFewRounds; ++r)
    if (group + r * kFewGroups < a.n) {
      const GradPiece p = a.pieces[group + r * kFewGroups];
      by_type(p.dtype, [&](auto type) {
        Others to;
        to.load(p, a.others, 0);
        h[r].template scale<decltype(type)::value>(factor);
        h[r].template store_all<decltype(type)::value, false>(p, a.others, t, nullptr, to);
      });
    }
}

}  // namespace dev

namespace {

// Each measured on both its sides, fp32 (us).
// Of the gathering launch at most, eight a compute unit: the norm of 2^26 in 1024 45.1,
// 2048 45.1, 4096 47.9.
constexpr uint32_t kGradGroups = 2048;
// Pieces up to which every scaling workgroup joins the sums, sparing a launch: 1 million
// 8.7 and 9.8, 8 million (2000 pieces) 20.7 and 23.2, 16 million 37.1 and 36.7.
constexpr uint32_t kGradJoined = 2048;
// Written by the one workgroup of grad_few at most: 20000 elements 5.5 and 6.0 in two
// launches, 30000 6.2 and 6.2, 4 copies of 20000 10.4 and 7.8.
constexpr uint64_t kGradFewBytes = 128 << 10;
// The memory-side cache.  A norm alone of more is read past the caches: 2^28 161 and 181;
// clipping reads the gradients again and finds the last of them there: 526, past them 540.
constexpr uint64_t kGradCached = uint64_t(256) << 20;

bool few(uint64_t pieces, uint64_t written) { return pieces <= dev::kFewGroups * dev::kFewRounds && written <= kGradFewBytes; }

}  // namespace

uint32_t grad_sums(uint64_t pieces, uint64_t written) {
  return few(pieces, written) ? 0 : static_cast<uint32_t>(std::min<uint64_t>(pieces, kGradGroups));
}

namespace {

template <int NORM>
hipError_t launch(const GradArgs& a, hipStream_t stream) {
  if (a.sums == 0) {
    dev::grad_few<NORM><<<1, dev::kGradThreads * dev::kFewGroups, 0, stream>>>(a);
    return hipGetLastError();
  }
  if (!a.clip && a.read > kGradCached) dev::grad_gather<NORM, true><<<a.sums, dev::kGradThreads, 0, stream>>>(a);
  else dev::grad_gather<NORM, false><<<a.sums, dev::kGradThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.clip && a.n <= kGradJoined) {
    dev::grad_scale<NORM, false, false><<<a.n, dev::kGradThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  dev::grad_factor<NORM><<<1, dev::kGradThreads, 0, stream>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || !a.clip) return e;
  // 2^25 74 and 84 within them, 2^24 45 and 38
  if (a.written >= kStreamBytes) dev::grad_scale<0, true, true><<<a.n, dev::kGradThreads, 0, stream>>>(a);
  else dev::grad_scale<0, true, false><<<a.n, dev::kGradThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grad(const GradArgs& a, hipStream_t stream) {
  return a.norm == 2 ? launch<2>(a, stream) : a.norm == 1 ? launch<1>(a, stream) : launch<0>(a, stream);
}

}  // namespace hbmc
