// Products in 8-bit integers with a scale for each token and channel, and the
// rounding of tokens to them (see hbmc_quantize_rows, hbmc_product).
//
// The sum over the inner width is a sum of whole numbers: exact in 32 bits
// whatever its order, so where the inner width is dealt out to the ranks the
// ranks' partial sums go into one accumulator and their AllReduce costs nothing.
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// ------------------------------------------------------- rounding to 8 bits

constexpr uint32_t kQuantThreads = 256;

// A workgroup a row: the largest size, as its bits (a NaN's and an infinity's are
// above every number's), then the codes.
template <int DT>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows(QuantizeArgs a) {
  typedef Pack<DT, 1> One;
  constexpr uint32_t E = One::E;
  __shared__ uint32_t shared[kQuantThreads / 64];
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
  uint32_t top = 0;
  for (int r = 0; r < a.P; ++r) {
    const uint64_t lo = uint64_t(r) * a.seg;
    const uint32_t n = lo < a.width ? min(a.seg, a.width - static_cast<uint32_t>(lo)) : 0;
    for (uint32_t i = threadIdx.x; i < n; i += kQuantThreads) {
      float f[1];
      One::widen(One::load(a.x[r] + (row * n + i) * E), f);
      top = max(top, f2u(f[0]) & 0x7fffffffu);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  if (threadIdx.x % 64 == 0) shared[threadIdx.x / 64] = top;
  __syncthreads();
  for (uint32_t w = 0; w < kQuantThreads / 64; ++w) top = max(top, shared[w]);
  const float most = u2f(top), by = 1.0f / most * 127.0f;
  const bool counts = top < 0x7f800000u && by < __builtin_inff();
  if (threadIdx.x == 0) a.scale[row] = counts ? most / 127.0f : top < 0x7f800000u ? 0.0f : __builtin_nanf("");
  for (int r = 0; r < a.P; ++r) {
    const uint64_t lo = uint64_t(r) * a.seg;
    const uint32_t n = lo < a.width ? min(a.seg, a.width - static_cast<uint32_t>(lo)) : 0;
    for (uint32_t i = threadIdx.x; i < n; i += kQuantThreads) {
      float f[1];
      One::widen(One::load(a.x[r] + (row * n + i) * E), f);
      const float c = fminf(fmaxf(__builtin_rintf(f[0] * by), -127.0f), 127.0f);
      a.q[r][row * n + i] = static_cast<unsigned char>(counts ? static_cast<int>(c) : 0);
    }
  }
  __syncthreads();
  }
}

// ----------------------------------------------------------------- products

// 16 codes of a row of `n` from position k, zeros past its end.  gfx950 loads
// global memory at any address.
__device__ __forceinline__ i32x4 codes16(const unsigned char* row, uint32_t n, uint32_t k) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= n) {
    typedef i32x4 any __attribute__((aligned(1)));
    return *reinterpret_cast<const any*>(row + k);
  }
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i)
    if (k + i < n) v[i / 4] |= static_cast<int32_t>(static_cast<uint32_t>(row[k + i]) << (8 * (i % 4)));
  return v;
}

// Four channels of a token: v scaled by the token and each channel.
template <int DT>
__device__ __forceinline__ void store4(unsigned char* out, uint64_t at, uint32_t n, const float (&f)[4]) {
  typedef Pack<DT, 1> One;
  constexpr uint32_t E = One::E;
  unsigned char* const p = out + at * E;
  if (n >= 4) {
    if constexpr (DT == kF32) {
      *reinterpret_cast<f32x4_any*>(p) = f32x4_any{f[0], f[1], f[2], f[3]};
    } else {
      typedef Pack<DT, 8> K;
      *reinterpret_cast<u32x2_any*>(p) = u32x2{K::narrow2(f[0], f[1]), K::narrow2(f[2], f[3])};
    }
    return;
  }
#pragma unroll
  for (uint32_t i = 0; i < 3; ++i) {
    const float one[1] = {f[i]};
    if (i < n) One::store(p + i * E, One::narrow(one));
  }
}

constexpr uint32_t kTile = 64, kStep = 64, kPitch = kStep + 16;  // bytes of a staged row: 16 more, so that rows fall on other banks

// A tile of 64 tokens by 64 channels: four waves of 32 by 32, staged through LDS
// 64 codes of the inner width at a time, at any alignment.
template <int DT>
__global__ __launch_bounds__(256) void product_tiles(ProductArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char sx[kTile * kPitch], sw[kTile * kPitch];
  const bool dealt = a.form == 0;  // channels dealt out
  const uint32_t tiles_n = ((dealt ? a.channel_seg : a.channels) + kTile - 1) / kTile;
  const uint32_t tiles_t = (a.rows + kTile - 1) / kTile;
  uint32_t b = blockIdx.x;
  const uint32_t tt = b % tiles_t;
  b /= tiles_t;
  const uint32_t tn = b % tiles_n, own = b / tiles_n;  // `own`: the rank whose product this is (forms 0 and 1)
  const uint64_t before = uint64_t(own) * a.channel_seg;
  const uint32_t channels = !dealt ? a.channels : before < a.channels ? min(a.channel_seg, a.channels - static_cast<uint32_t>(before)) : 0;
  const uint32_t t0 = tt * kTile, n0 = tn * kTile;
  if (n0 >= channels) return;
  const int r0 = a.form <= 1 ? static_cast<int>(own) : 0, r1 = a.form <= 1 ? r0 + 1 : a.P;
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, wt = wave % 2 * 32, wn = wave / 2 * 32;
  i32x4 acc[2][2] = {};
  for (int r = r0; r < r1; ++r) {
    const uint64_t lo = dealt ? 0 : uint64_t(r) * a.inner_seg;
    const uint32_t inner = dealt ? a.inner : lo < a.inner ? min(a.inner_seg, a.inner - static_cast<uint32_t>(lo)) : 0;
    const uint32_t row = threadIdx.x / 4, part = threadIdx.x % 4 * 16;
    for (uint32_t k = 0; k < inner; k += kStep) {
      i32x4 vx = {0, 0, 0, 0}, vw = {0, 0, 0, 0};
      if (t0 + row < a.rows) vx = codes16(a.x[r] + uint64_t(t0 + row) * inner, inner, k + part);
      if (n0 + row < channels) vw = codes16(a.w[r] + uint64_t(n0 + row) * inner, inner, k + part);
      __syncthreads();
      *reinterpret_cast<i32x4*>(sx + row * kPitch + part) = vx;
      *reinterpret_cast<i32x4*>(sw + row * kPitch + part) = vw;
      __syncthreads();
      i32x4 fx[2], fw[2];
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        fx[i] = *reinterpret_cast<const i32x4*>(sx + (wt + i * 16 + lane % 16) * kPitch + lane / 16 * 16);
        fw[i] = *reinterpret_cast<const i32x4*>(sw + (wn + i * 16 + lane % 16) * kPitch + lane / 16 * 16);
      }
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fx[i], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const uint32_t t = t0 + wt + i * 16 + lane % 16;
    if (t >= a.rows) continue;
    const float xs = a.x_scale[t];
#pragma unroll
    for (uint32_t j = 0; j < 2; ++j) {
      const uint32_t n = n0 + wn + j * 16 + lane / 16 * 4;
      if (n >= channels) continue;
      float f[4];
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e)
        f[e] = static_cast<float>(acc[i][j][e]) * xs * (n + e < channels ? a.w_scale[own][n + e] : 0.0f);
      const uint32_t left = channels - n;
      if (a.form <= 1) store4<DT>(a.out[own], uint64_t(t) * channels + n, left, f);
      else if (a.form == 2) {
        for (int r = 0; r < a.P; ++r) store4<DT>(a.out[r], uint64_t(t) * channels + n, left, f);
      } else {
        store4<DT>(a.out[t / a.row_seg], uint64_t(t % a.row_seg) * channels + n, left, f);
      }
    }
  }
}

}  // namespace dev

hipError_t launch_quantize(int dtype, const QuantizeArgs& a, hipStream_t stream) {
  const uint32_t grid = static_cast<uint32_t>(std::min<uint64_t>(a.rows, 1 << 20));
  if (dtype == dev::kF32) dev::quantize_rows<dev::kF32><<<grid, dev::kQuantThreads, 0, stream>>>(a);
  else if (dtype == dev::kF16) dev::quantize_rows<dev::kF16><<<grid, dev::kQuantThreads, 0, stream>>>(a);
  else dev::quantize_rows<dev::kBF16><<<grid, dev::kQuantThreads, 0, stream>>>(a);
  return hipGetLastError();
}

namespace {

uint64_t tiles_of(const ProductArgs& a, uint64_t tile) {
  const uint64_t tiles_n = ((a.form == 0 ? a.channel_seg : a.channels) + tile - 1) / tile;
  return (a.rows + tile - 1) / tile * tiles_n * (a.form <= 1 ? a.P : 1);
}

}  // namespace

bool product_fits(const ProductArgs& a) { return tiles_of(a, dev::kTile) < uint64_t(1) << 24; }

hipError_t launch_product(int dtype, const ProductArgs& a, hipStream_t stream) {
  const uint64_t grid = tiles_of(a, dev::kTile);
  if (dtype == dev::kF32) dev::product_tiles<dev::kF32><<<static_cast<uint32_t>(grid), 256, 0, stream>>>(a);
  else if (dtype == dev::kF16) dev::product_tiles<dev::kF16><<<static_cast<uint32_t>(grid), 256, 0, stream>>>(a);
  else dev::product_tiles<dev::kBF16><<<static_cast<uint32_t>(grid), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace hbmc
