// The global norm of many gradient tensors, and their clipping (see
// hbmc_gradients_clip).
//
// No gradient can be scaled before the last has been read, so the data is passed
// over twice: a launch leaves one partial sum a workgroup, and the next joins
// them (every workgroup by itself, in the same order) and scales.  Sums are kept
// in 64 bits, so that no square overflows, none is lost, and the norm is right to
// the last bit of its 32 whatever the number of gradients.
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

constexpr uint32_t kGradThreads = 256, kGradVectors = 4;  // a piece: four vectors a thread
static_assert(kGradThreads * kGradVectors * 16 == kGradPieceBytes, "a piece is one round of its workgroup");

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

template <int NORM, int DT, uint32_t THREADS>
__device__ __forceinline__ void gather(const GradPiece& p, Gather<NORM>& g) {
  typedef Pack<DT, 16 / Width<DT>::bytes> V;
  typedef Pack<DT, 1> One;
  constexpr uint32_t VE = 16 / V::E;
  const uint32_t vectors = p.count / VE;
  u32x4 v[kGradVectors];
#pragma unroll
  for (uint32_t j = 0; j < kGradVectors; ++j) {
    const uint32_t i = threadIdx.x + j * kGradThreads;
    v[j] = i < vectors ? V::load(p.data + uint64_t(i) * 16) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (uint32_t j = 0; j < kGradVectors; ++j) {
    float f[VE];
    V::widen(v[j], f);
#pragma unroll
    for (uint32_t e = 0; e < VE; ++e) g.add(f[e]);
  }
  const uint32_t last = vectors * VE + threadIdx.x;
  if (last < p.count) {
    float f[1];
    One::widen(One::load(p.data + uint64_t(last) * V::E), f);
    g.add(f[0]);
  }
}

template <int NORM>
__device__ __forceinline__ void gather(const GradPiece& p, Gather<NORM>& g) {
  if (p.dtype == kF32) gather<NORM, kF32, kGradThreads>(p, g);
  else if (p.dtype == kF16) gather<NORM, kF16, kGradThreads>(p, g);
  else gather<NORM, kBF16, kGradThreads>(p, g);
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

template <int DT, bool STREAM>
__device__ __forceinline__ void scale(const GradPiece& p, unsigned char* const* others, float factor) {
  typedef Pack<DT, 16 / Width<DT>::bytes> V;
  typedef Pack<DT, 1> One;
  constexpr uint32_t VE = 16 / V::E;
  const uint32_t vectors = p.count / VE;
  u32x4 v[kGradVectors];
#pragma unroll
  for (uint32_t j = 0; j < kGradVectors; ++j) {
    const uint32_t i = threadIdx.x + j * kGradThreads;
    if (i < vectors) v[j] = V::load(p.data + uint64_t(i) * 16);
  }
  const uint32_t last = vectors * VE + threadIdx.x;
  uint32_t single = 0;
  if (last < p.count) single = One::load(p.data + uint64_t(last) * V::E);
#pragma unroll
  for (uint32_t j = 0; j < kGradVectors; ++j) {
    float f[VE];
    V::widen(v[j], f);
#pragma unroll
    for (uint32_t e = 0; e < VE; ++e) f[e] *= factor;
    v[j] = V::narrow(f);
  }
  float f[1];
  One::widen(single, f);
  f[0] *= factor;
  single = One::narrow(f);
  for (uint32_t c = 0; c < p.copies; ++c) {
    unsigned char* to = c == 0 ? p.data : others[p.first + c - 1] + p.offset;
#pragma unroll
    for (uint32_t j = 0; j < kGradVectors; ++j) {
      const uint32_t i = threadIdx.x + j * kGradThreads;
      if (i < vectors) {
        if constexpr (STREAM) V::store_nt(to + uint64_t(i) * 16, v[j]);
        else V::store(to + uint64_t(i) * 16, v[j]);
      }
    }
    if (last < p.count) One::store(to + uint64_t(last) * V::E, single);
  }
}

template <bool STREAM>
__device__ __forceinline__ void scale(const GradPiece& p, unsigned char* const* others, float factor) {
  if (p.dtype == kF32) scale<kF32, STREAM>(p, others, factor);
  else if (p.dtype == kF16) scale<kF16, STREAM>(p, others, factor);
  else scale<kBF16, STREAM>(p, others, factor);
}

// One partial sum a workgroup, over every gridDim.x-th piece.
template <int NORM>
__global__ __launch_bounds__(kGradThreads) void grad_gather(GradArgs a) {
  __shared__ double shared[kGradThreads / 64];
  Gather<NORM> g;
  for (uint32_t i = blockIdx.x; i < a.n; i += gridDim.x) gather(a.pieces[i], g);
  const double x = join_workgroup<NORM>(g.value(), shared);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = x;
}

// The partial sums joined, then (with a.clip) the pieces scaled, last pieces
// first: what the gathering launch read last may still be cached.
template <int NORM, bool STREAM>
__global__ __launch_bounds__(kGradThreads) void grad_scale(GradArgs a) {
  __shared__ double shared[kGradThreads / 64];
  double x = 0.0;
  for (uint32_t i = threadIdx.x; i < a.sums; i += kGradThreads) x = join<NORM>(x, a.partial[i]);
  x = join_workgroup<NORM>(x, shared);
  const float factor = factor_of<NORM>(a, x, blockIdx.x == 0 && threadIdx.x == 0);
  if (!a.clip || factor == 1.0f) return;
  for (uint32_t i = blockIdx.x; i < a.n; i += gridDim.x) scale<STREAM>(a.pieces[a.n - 1 - i], a.others, factor);
}

// Few pieces: one workgroup, one launch, nothing kept.
template <int NORM>
__global__ __launch_bounds__(kGradThreads) void grad_few(GradArgs a) {
  __shared__ double shared[kGradThreads / 64];
  Gather<NORM> g;
  for (uint32_t i = 0; i < a.n; ++i) gather(a.pieces[i], g);
  const double x = join_workgroup<NORM>(g.value(), shared);
  const float factor = factor_of<NORM>(a, x, threadIdx.x == 0);
  if (!a.clip || factor == 1.0f) return;
  for (uint32_t i = 0; i < a.n; ++i) scale<false>(a.pieces[i], a.others, factor);
}

}  // namespace dev

constexpr uint32_t kGradGroups = 2048, kGradFew = 4;

uint32_t grad_sums(uint64_t pieces) {
  return pieces <= kGradFew ? 0 : static_cast<uint32_t>(std::min<uint64_t>(pieces, kGradGroups));
}

namespace {

template <int NORM>
hipError_t launch(const GradArgs& a, hipStream_t stream) {
  if (a.sums == 0) {
    dev::grad_few<NORM><<<1, dev::kGradThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  dev::grad_gather<NORM><<<a.sums, dev::kGradThreads, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const uint32_t groups = a.clip ? std::min(a.n, kGradGroups) : 1;
  if (a.stream) dev::grad_scale<NORM, true><<<groups, dev::kGradThreads, 0, stream>>>(a);
  else dev::grad_scale<NORM, false><<<groups, dev::kGradThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grad(const GradArgs& a, hipStream_t stream) {
  return a.norm == 2 ? launch<2>(a, stream) : a.norm == 1 ? launch<1>(a, stream) : launch<0>(a, stream);
}

}  // namespace hbmc
