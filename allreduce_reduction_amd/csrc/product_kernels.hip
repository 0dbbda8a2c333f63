// Products in 8-bit integers with a scale for each token and channel, and the
// rounding of tokens to them (see hbmc_quantize_rows, hbmc_product).
//
// The sum over the inner width is a sum of whole numbers: exact in 32 bits
// whatever its order, so where the inner width is dealt out to the ranks the
// ranks' partial sums go into one accumulator and their AllReduce costs nothing.
//
// Kernels by what bounds them: many tokens, the matrix cores and what feeds them
// (product_wide, aligned rows; product_tiles, any others); few tokens, the weights'
// bytes (the same in narrow tiles); few results, the latency of a long sum
// (product_few).  On one MI355X, 8 ranks, calls one after the other: 4096 tokens of 8192
// codes by 4096 channels, scattered by tokens, 106 to 110 us from box to box (2500 to
// 2580 TOP/s; the vendor library's product of the same sizes 115 where this took 109);
// 64 of 4096 by 131072, the channels dealt out, 102 us (5.3 TB/s); 3 of 8192 by 4096 so
// 8.6 us (3.9 TB/s), their sum to all ranks 9.1.
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// ------------------------------------------------------- rounding to 8 bits

// The larger sizes of two words of elements: as whole numbers, whose order is
// theirs (a NaN's and an infinity's are above every number's).
template <int DT>
__device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) {
  if constexpr (DT == kF32) {
    return max(top, w & 0x7fffffffu);
  } else {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top), __builtin_bit_cast(u16x2, w & 0x7fff7fffu)));
  }
}

// x * by, rounded to a whole number in the low bits: 1.5 * 2^23 has steps of one.
__device__ __forceinline__ uint32_t code(float x, float by) { return f2u(x * by + 12582912.0f); }
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t top_dpp(uint32_t x) {
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(x), static_cast<int>(x), CTRL, ROWS, 0xf, false)));
}
// The largest of a wave, by steps as wave_max's.
__device__ __forceinline__ uint32_t wave_top(uint32_t x) {
  x = top_dpp<0x111, 0xf>(x);
  x = top_dpp<0x112, 0xf>(x);
  x = top_dpp<0x114, 0xf>(x);
  x = top_dpp<0x118, 0xf>(x);
  x = top_dpp<0x142, 0xa>(x);
  x = top_dpp<0x143, 0xc>(x);
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 63));
}

// A workgroup a row: the largest size, then the codes.  A row of up to VECTORS
// pieces a wave (64 vectors of a rank's columns each) stays in registers and is read
// once; a longer one (LONG) is read twice.  A rank's last vector ends with its
// columns and overlaps its neighbour, which changes no maximum and writes the same
// codes twice; VE is 1 where a rank has less than a vector.  No load waits behind a
// branch (behind one for each ragged end, each waited for the one before it).  HBM
// bounds it: 4096 rows of 8192 bf16, 100 MB, 23 us on 8 ranks and 18 on one (4.4 and
// 5.5 TB/s), 8192 rows 38 us (5.2 TB/s).  inverse_of: 2^32 / a rank's pieces, rounded
// up: exact for the 128 pieces that are not LONG.
template <int DT, int VE, uint32_t THREADS, uint32_t VECTORS, bool LONG>
__global__ __launch_bounds__(THREADS) void quantize_rows(QuantizeArgs a, uint32_t inverse_of) {
  typedef Pack<DT, VE> V;
  constexpr uint32_t E = V::E, WAVES = THREADS / 64;
  __shared__ uint32_t shared[WAVES];
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint32_t per_rank = (a.seg + 64 * VE - 1) / (64 * VE);
  const uint32_t ranks = (a.width + a.seg - 1) / a.seg, all = per_rank * ranks;  // of those that own columns
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    typename V::raw x[VECTORS];
    // of the wave's j-th piece (the last one again past the end): rank, and the lane's place in the rank's rows
    uint32_t rank[VECTORS];
    uint64_t place[VECTORS];
    const auto load = [&](uint32_t p0) {
#pragma unroll
      for (uint32_t j = 0; j < VECTORS; ++j) {
        const uint32_t p = min(p0 + j * WAVES, all - 1);
        rank[j] = LONG ? p / per_rank : per_rank == 1 ? p : __umulhi(p, inverse_of);
        const uint32_t n = min(a.seg, a.width - rank[j] * a.seg);
        place[j] = row * n + min(((p - rank[j] * per_rank) * 64 + lane) * VE, n - VE);
      }
#pragma unroll
      for (uint32_t j = 0; j < VECTORS; ++j) x[j] = LONG ? V::load(a.x[rank[j]] + place[j] * E) : V::stream(a.x[rank[j]] + place[j] * E);
    };
    uint32_t top = 0;
    for (uint32_t p0 = wave; p0 < all; p0 += WAVES * VECTORS) {
      load(p0);
#pragma unroll
      for (uint32_t j = 0; j < VECTORS; ++j) {
        if constexpr (VE == 1) {
          top = larger<DT>(top, x[j]);
        } else {
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) top = larger<DT>(top, x[j][e]);
        }
      }
      if (!LONG) break;
    }
    if constexpr (DT == kBF16) top = max(top << 16, top & 0xffff0000u);
    if constexpr (DT == kF16) top = max(f2u(widen_f16(top & 0xffffu)), f2u(widen_f16(top >> 16)));
    top = wave_top(top);
    if constexpr (WAVES > 1) {
      if (lane == 0) shared[wave] = top;
      __syncthreads();
#pragma unroll
      for (uint32_t w = 0; w < WAVES; ++w) top = max(top, shared[w]);
      __syncthreads();
    }
    const float most = u2f(top), inverse = 1.0f / most * 127.0f;
    const bool counts = top < 0x7f800000u && inverse < __builtin_inff();
    if (threadIdx.x == 0) a.scale[row] = counts ? most / 127.0f : top < 0x7f800000u ? 0.0f : __builtin_nanf("");
    for (uint32_t p0 = wave; p0 < all; p0 += WAVES * VECTORS) {
      if (LONG) load(p0);
#pragma unroll
      for (uint32_t j = 0; j < VECTORS; ++j) {
        float f[VE];
        uint32_t c[VE];
        V::widen(x[j], f);
#pragma unroll
        for (uint32_t e = 0; e < VE; ++e) c[e] = counts ? code(f[e], inverse) : 0;
        unsigned char* const to = a.q[rank[j]] + place[j];
        if constexpr (VE == 8) *reinterpret_cast<u32x2_any*>(to) = u32x2{bytes4(c[0], c[1], c[2], c[3]), bytes4(c[4], c[5], c[6], c[7])};
        else if constexpr (VE == 4) *reinterpret_cast<u32_any*>(to) = bytes4(c[0], c[1], c[2], c[3]);
        else *to = static_cast<unsigned char>(c[0]);
      }
      if (!LONG) break;
    }
  }
}

// ----------------------------------------------------------------- products

// Rows of codes at any alignment and of any width.  gfx950 loads global memory at
// any address, but no load leaves its row: a chunk of 16 codes that would pass the
// row's end is the row's last 16 instead, tokens and channels alike, and the
// tokens' lose (keep_from) those that earlier chunks have had, so that a product
// counts once.  Without a branch at each load, behind which the next would wait.
__device__ __forceinline__ i32x4 keep_from(i32x4 v, uint32_t first) {  // zeros before byte `first`; from 16 on, all
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e) {
    const uint32_t lost = min(first > 4 * e ? first - 4 * e : 0, 4u);
    v[e] &= static_cast<int32_t>(static_cast<uint32_t>(0xffffffffull << (8 * lost)));
  }
  return v;
}
// 16 codes of row r from position k, one by one, zeros past the `inner` ones: where a
// rank has rows of fewer than 16.  For a sum over the ranks `inner` is all of them's,
// rank after rank, so that many ranks with few codes take one stage and not one each.
__device__ __forceinline__ i32x4 short_chunk(const ProductArgs& a, const unsigned char* const* ranks, uint64_t r, uint32_t rank, uint32_t inner,
                                             uint32_t k) {
  i32x4 v = {0, 0, 0, 0};
  const uint32_t each = a.form >= 2 ? a.inner_seg : inner;
  uint32_t q = a.form >= 2 ? k / each : rank, off = a.form >= 2 ? k % each : k;
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i) {
    if (k + i >= inner) continue;
    const uint32_t n = a.form >= 2 ? min(each, a.inner - q * each) : inner;
    v[i / 4] |= static_cast<int32_t>(static_cast<uint32_t>(ranks[q][r * n + off]) << (8 * (i % 4)));
    if (a.form >= 2 && ++off == each) off = 0, ++q;
    else if (a.form < 2) ++off;
  }
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

// Token t's sums of channels [n, n + 4), those below `channels`, to where the form puts them.
template <int DT>
__device__ __forceinline__ void store_results(const ProductArgs& a, uint32_t own, uint32_t channels, uint32_t t, uint32_t n, i32x4 sum,
                                              float x_scale) {
  float f[4];
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e) f[e] = static_cast<float>(sum[e]) * x_scale * (n + e < channels ? a.w_scale[own][n + e] : 0.0f);
  const uint32_t left = channels - n;
  if (a.form <= 1) {
    store4<DT>(a.out[own], uint64_t(t) * channels + n, left, f);
  } else if (a.form == 2) {
    for (int r = 0; r < a.P; ++r) store4<DT>(a.out[r], uint64_t(t) * channels + n, left, f);
  } else {
    store4<DT>(a.out[t / a.row_seg], uint64_t(t % a.row_seg) * channels + n, left, f);
  }
}

// A wave's 16 * FT tokens from t0 by 16 * FN channels from n0.  They go through its
// SHARE bytes of LDS, so that rows of its channels are stored whole (128 bytes and
// more of a 256 by 256 tile's; 4096 x 4096 results of 8192 codes 118 us without, 108
// so, to 8 ranks 271 and 147).
template <int DT, uint32_t FT, uint32_t FN, uint32_t SHARE>
__device__ __forceinline__ void store_tile(const ProductArgs& a, uint32_t own, uint32_t channels, uint32_t t0, uint32_t n0,
                                           const i32x4 (&acc)[FT][FN], unsigned char* mine, uint32_t lane) {
  typedef Pack<DT, 16 / Width<DT>::bytes> V;
  typedef Pack<DT, 1> One;
  constexpr uint32_t E = V::E, VE = 16 / E, NW = FN * 16, PITCH = NW * E + 16;
  constexpr uint32_t FITS = SHARE / PITCH / 16, BATCH = FITS >= FT ? FT : FITS >= FT / 2 ? FT / 2 : FITS >= FT / 4 ? FT / 4 : 1;
  static_assert(FITS >= 1 && FT % BATCH == 0, "a batch of 16 rows at least");
#pragma unroll
  for (uint32_t i0 = 0; i0 < FT; i0 += BATCH) {
#pragma unroll
    for (uint32_t i = i0; i < i0 + BATCH; ++i) {
      const uint32_t t = t0 + i * 16 + lane % 16;
      const float xs = a.x_scale[min(t, a.rows - 1)];
#pragma unroll
      for (uint32_t j = 0; j < FN; ++j) {
        const uint32_t n = j * 16 + lane / 16 * 4;
        float f[4];
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) f[e] = static_cast<float>(acc[i][j][e]) * xs * a.w_scale[own][min(n0 + n + e, channels - 1)];
        unsigned char* const to = mine + ((i - i0) * 16 + lane % 16) * PITCH + n * E;
        if constexpr (DT == kF32) *reinterpret_cast<u32x4*>(to) = u32x4{f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3])};
        else *reinterpret_cast<u32x2*>(to) = u32x2{Pack<DT, 8>::narrow2(f[0], f[1]), Pack<DT, 8>::narrow2(f[2], f[3])};
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr uint32_t CHUNKS_ROW = NW * E / 16;
#pragma unroll
    for (uint32_t c0 = 0; c0 < BATCH * 16 * CHUNKS_ROW; c0 += 64) {
      const uint32_t c = c0 + lane, r = c / CHUNKS_ROW, n = n0 + c % CHUNKS_ROW * VE, t = t0 + i0 * 16 + r;
      if (c0 + 64 > BATCH * 16 * CHUNKS_ROW && c >= BATCH * 16 * CHUNKS_ROW) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * PITCH + c % CHUNKS_ROW * 16);
      if (t >= a.rows || n >= channels) continue;
      const uint32_t left_n = channels - n;
      const auto put = [&](unsigned char* out, uint32_t row_of) {
        unsigned char* const to = out + (uint64_t(row_of) * channels + n) * E;
        if (left_n >= VE) {
          V::store(to, v);
        } else {
#pragma unroll
          for (uint32_t e = 0; e + 1 < VE; ++e)
            if (e < left_n) One::store(to + e * E, v[e * E / 4] >> (e * E % 4 * 8));
        }
      };
      if (a.form <= 1) {
        put(a.out[own], t);
      } else if (a.form == 2) {
        for (int r2 = 0; r2 < a.P; ++r2) put(a.out[r2], t);
      } else {
        put(a.out[t / a.row_seg], t % a.row_seg);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- tiles at any alignment

// A tile of TT tokens by TN channels of WT by WN waves, whose rows may begin and
// end anywhere: 128 codes of each at a time through registers into one of two
// halves of LDS, the next of them on their way while one is multiplied.  Loads of 16
// bytes at odd addresses bound it: 4096 tokens of 8200 codes by 4096 channels, 8 ranks
// of 1025 codes, 295 us, where 8192 codes through here take 196 and in tiles of aligned
// rows 106.  981 tokens of 3038 codes by 461 channels 17 us.
constexpr uint32_t kAhead = 4;

template <int DT, uint32_t TT, uint32_t TN, uint32_t WT, uint32_t WN, bool SHORT>
__global__ __launch_bounds__(64 * WT * WN) void product_tiles(ProductArgs a) {
  constexpr uint32_t WAVES = WT * WN, ROWS = TT + TN, EACH = ROWS / 8 / WAVES;  // rows of a thread's loads
  constexpr uint32_t FT = TT / WT / 16, FN = TN / WN / 16;
  static_assert(TT % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0, "a load's rows are of one operand");
  __shared__ __attribute__((aligned(16))) unsigned char halves[2][ROWS * 128];
  const bool dealt = a.form == 0;
  const uint32_t tiles_n = ((dealt ? a.channel_seg : a.channels) + TN - 1) / TN;
  const uint32_t tiles_t = (a.rows + TT - 1) / TT;
  uint32_t b = blockIdx.x;
  const uint32_t tt = b % tiles_t;
  b /= tiles_t;
  const uint32_t tn = b % tiles_n, own = b / tiles_n;
  const uint64_t before = uint64_t(own) * a.channel_seg;
  const uint32_t channels = !dealt ? a.channels : before < a.channels ? min(a.channel_seg, a.channels - static_cast<uint32_t>(before)) : 0;
  const uint32_t t0 = tt * TT, n0 = tn * TN;
  if (n0 >= channels) return;
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint32_t wt = wave % WT * (TT / WT), wn = wave / WT * (TN / WN);
  // the next 128 codes to load: rank, its inner width, position in it
  uint32_t rank = a.form <= 1 ? own : 0, k = 0, inner = 0;
  const uint32_t end = a.form <= 1 ? own + 1 : static_cast<uint32_t>(a.P);
  const auto open = [&]() {
    const uint64_t lo = dealt ? 0 : uint64_t(rank) * a.inner_seg;
    inner = rank >= end || lo >= a.inner ? 0 : dealt ? a.inner : min(a.inner_seg, a.inner - static_cast<uint32_t>(lo));
    if (SHORT && a.form >= 2) inner = rank == 0 ? a.inner : 0;  // all ranks' codes of a row, one rank after the other
    k = 0;
  };
  const uint32_t row = wave * 8 + lane / 8, chunk = lane % 8;
  struct Codes {
    i32x4 v[EACH];
    uint32_t lost;  // of the tokens' 16 at the front (see keep_from)
    bool any = false, last = false;
  };
  const auto load = [&](Codes& c) {
    c.any = inner > 0;
    if (!c.any) return;
    c.last = k + 128 > inner;
    const uint32_t wanted = k + chunk * 16, at = SHORT ? wanted : min(wanted, inner - 16);
    c.lost = wanted - at;
#pragma unroll
    for (uint32_t j = 0; j < EACH; ++j) {
      const bool is_x = j * 8 * WAVES < TT;
      const uint32_t r = j * 8 * WAVES + row - (is_x ? 0 : TT);
      // rows past the last one repeat it: their results are not stored
      const uint32_t of = is_x ? min(r, a.rows - 1 - t0) : min(r, channels - 1 - n0);
      if constexpr (SHORT) {
        c.v[j] = short_chunk(a, is_x ? a.x : a.w, (is_x ? t0 : n0) + of, rank, inner, at);
      } else {
        const unsigned char* const from = is_x ? a.x[rank] + uint64_t(t0) * inner : a.w[rank] + uint64_t(n0) * inner;
        c.v[j] = *reinterpret_cast<const i32x4_any*>(from + (of * inner + at));
      }
    }
    k += 128;
    if (k >= inner) {
      ++rank;
      open();
    }
  };
  // a row's chunk c lies at place c ^ (row % 8), so that 8 rows' equal chunks lie on all banks
  const auto put = [&](unsigned char* to, Codes& c) {
    if (!SHORT && c.last) {
#pragma unroll
      for (uint32_t j = 0; j < TT / 8 / WAVES; ++j) c.v[j] = keep_from(c.v[j], c.lost);
    }
#pragma unroll
    for (uint32_t j = 0; j < EACH; ++j)
      *reinterpret_cast<i32x4*>(to + (j * 8 * WAVES + row) * 128 + (chunk ^ row % 8) * 16) = c.v[j];
  };
  i32x4 acc[FT][FN] = {};
  const auto multiply = [&](const unsigned char* from) {
#pragma unroll
    for (uint32_t s = 0; s < 2; ++s) {
      i32x4 fx[FT], fw[FN];
      const uint32_t place = ((s * 4 + lane / 16) ^ (lane % 8)) * 16;
#pragma unroll
      for (uint32_t j = 0; j < FN; ++j) fw[j] = *reinterpret_cast<const i32x4*>(from + (TT + wn + j * 16 + lane % 16) * 128 + place);
#pragma unroll
      for (uint32_t i = 0; i < FT; ++i) fx[i] = *reinterpret_cast<const i32x4*>(from + (wt + i * 16 + lane % 16) * 128 + place);
#pragma unroll
      for (uint32_t i = 0; i < FT; ++i)
#pragma unroll
        for (uint32_t j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fx[i], acc[i][j], 0, 0, 0);
    }
  };
  // Every wave's codes in LDS, and read.  No __syncthreads(): that would wait for
  // the codes still on their way to registers.
  const auto meet = []() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  open();
  Codes c[kAhead];
#pragma unroll
  for (uint32_t s = 0; s < kAhead; ++s) load(c[s]);
  bool more = c[0].any;  // a rank may hold none of the inner width
  if (more) put(halves[0], c[0]);
  meet();
  while (more) {
#pragma unroll
    for (uint32_t s = 0; s < kAhead; ++s) {  // halves[s % 2] holds the codes to multiply, c[s] is free, the others hold the next
      load(c[s]);
      multiply(halves[s % 2]);
      more = c[(s + 1) % kAhead].any;
      if (!more) break;
      put(halves[(s + 1) % 2], c[(s + 1) % kAhead]);
      meet();
    }
  }
  meet();
  store_tile<DT, FT, FN, sizeof(halves) / WAVES>(a, own, channels, t0 + wt, n0 + wn, acc, halves[0] + wave * (sizeof(halves) / WAVES), lane);
}

// ---- tiles of aligned rows

// A buffer resource of `bytes` from p: loads past its end give zeros.
__device__ __forceinline__ i32x4 resource(const unsigned char* p, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return i32x4{static_cast<int32_t>(at), static_cast<int32_t>(at >> 32 & 0xffff), static_cast<int32_t>(bytes), 0x00020000};
}

typedef __attribute__((address_space(3))) unsigned char lds_byte;

// 16 bytes a lane from `at` of the resource to 1 KiB of LDS.  In assembly, since
// the compiler's own form makes it wait for every such load before a read of LDS;
// there is no register that it fills, and the kernel counts the loads itself.  M0 holds
// the place in LDS, and is named as an output (with the compiler writing it, 64 x 8192 x
// 4096 on 8 ranks takes 16.6 us for 16.3); "memory" keeps accesses of LDS on their side.
__device__ __forceinline__ void load_lds(i32x4 from, uint32_t at, uint32_t to) {
  uint32_t place;
  asm volatile("s_mov_b32 %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               : "=&{m0}"(place) : "v"(at), "s"(from), "s"(to) : "memory");
}

constexpr uint32_t kWide = 128;  // codes of the inner width in a stage: a row of LDS

// A tile of TT tokens by TN channels, WT by WN waves.  STAGES stages of 128 codes of
// its rows lie in LDS, loaded there without a register between; a wave holds 64 codes
// of its rows and multiplies them while it reads the next 64, so that neither the
// loads, the reads nor the products wait for one another but at one barrier a stage.
// 256 by 256 on 8 waves of 128 by 64, 4096 x 8192 x 4096: 106 us; 128 before reads and
// products were taken in turn and 118 before rows were stored whole; with instructions of
// 32 x 32 x 32 135 where 128; with stages of 64 codes, three to six, 127 to 139 where 118;
// without its loads 84, without its reads of LDS 106, with neither 81.
// TURN: each workgroup begins elsewhere in the inner width, so that those that stream
// weights do not all ask for the same columns of their rows at once (64 x 4096 x 131072
// 122 us without, 102 so; large tiles gain nothing).
template <int DT, uint32_t TT, uint32_t TN, uint32_t WT, uint32_t WN, uint32_t STAGES, bool TURN>
__global__ __launch_bounds__(64 * WT * WN) void product_wide(ProductArgs a) {
  constexpr uint32_t WAVES = WT * WN, ROWS = TT + TN, LOADS = ROWS / 8 / WAVES;  // a wave's loads of a stage, 8 rows each
  constexpr uint32_t FT = TT / WT / 16, FN = TN / WN / 16;
  static_assert(TT % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0, "a load's rows are of one operand");
  static_assert(STAGES >= 2 && (STAGES - 1) * LOADS < 64, "counted in the hardware's six bits");
  constexpr uint32_t STAGE = ROWS * kWide;
  __shared__ __attribute__((aligned(1024))) unsigned char stages[STAGES * STAGE];
  const bool dealt = a.form == 0;
  const uint32_t tiles_n = ((dealt ? a.channel_seg : a.channels) + TN - 1) / TN;
  const uint32_t tiles_t = (a.rows + TT - 1) / TT;
  // workgroups go to the eight XCDs in turn: each takes a run of tiles, four
  // tiles of tokens deep, that share rows in its L2
  uint32_t b = blockIdx.x;
  if (gridDim.x % 8 == 0) b = b % 8 * (gridDim.x / 8) + b / 8;
  const uint32_t own = b / (tiles_t * tiles_n);
  b -= own * tiles_t * tiles_n;
  const uint32_t group = b / (4 * tiles_n), deep = min(4u, tiles_t - 4 * group);
  b -= group * 4 * tiles_n;
  const uint32_t tt = 4 * group + b % deep, tn = b / deep;
  const uint64_t before = uint64_t(own) * a.channel_seg;
  const uint32_t channels = !dealt ? a.channels : before < a.channels ? min(a.channel_seg, a.channels - static_cast<uint32_t>(before)) : 0;
  const uint32_t t0 = tt * TT, n0 = tn * TN;
  if (n0 >= channels) return;
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint32_t wt = wave % WT * (TT / WT), wn = wave / WT * (TN / WN);
  const uint32_t rows_t = min(TT, a.rows - t0), rows_n = min(TN, channels - n0);

  // the next stage to load: rank, its inner width, position in it
  uint32_t rank = a.form <= 1 ? own : 0, k = 0, inner = 0, left = 0, todo = 0;
  const uint32_t end = a.form <= 1 ? own + 1 : static_cast<uint32_t>(a.P);
  for (uint32_t r = rank; r < end; ++r) {
    const uint64_t lo = dealt ? 0 : uint64_t(r) * a.inner_seg;
    if (lo < a.inner) left += ((dealt ? a.inner : min(a.inner_seg, a.inner - static_cast<uint32_t>(lo))) + kWide - 1) / kWide;
  }
  // a wave's load: 8 rows of 8 chunks of 16 codes; row r's chunk c lies at place
  // c ^ (r % 8) of its row, so that 8 rows' equal chunks lie on all banks
  const uint32_t row = lane / 8, chunk = (lane % 8 ^ row) * 16;
  const uint32_t turned = TURN ? blockIdx.x : 0;
  i32x4 px = resource(nullptr, 0), pw = px;
  uint32_t place = 0;  // the lane's in the first of its loads
  const auto open = [&]() {
    const uint64_t lo = dealt ? 0 : uint64_t(rank) * a.inner_seg;
    inner = rank >= end || lo >= a.inner ? 0 : dealt ? a.inner : min(a.inner_seg, a.inner - static_cast<uint32_t>(lo));
    todo = (inner + kWide - 1) / kWide;
    k = todo ? (turned % todo) * kWide : 0;
    if (inner == 0) return;  // past the last: loads give zeros
    px = resource(a.x[rank] + uint64_t(t0) * inner, rows_t * inner);
    pw = resource(a.w[rank] + uint64_t(n0) * inner, rows_n * inner);
    place = (wave * 8 + row) * inner + chunk;
  };
  // The j-th of the wave's loads of a stage, and the step to the next stage.
  const auto load = [&](unsigned char* to, uint32_t j) {
    const uint32_t at = place + k + (k + chunk < inner ? 0 : 0x40000000);  // chunks past the inner width: zeros
    const uint32_t first = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)to)) + wave * 1024;
    const bool is_x = j < TT / 8 / WAVES;
    load_lds(is_x ? px : pw, at + (is_x ? j : j - TT / 8 / WAVES) * (WAVES * 8) * inner, first + j * WAVES * 1024);
  };
  const auto advance = [&]() {
    if (inner == 0) return;
    k = k + kWide < inner ? k + kWide : 0;
    if (--todo == 0) {
      ++rank;
      open();
    }
  };
  const auto load_all = [&](unsigned char* to) {
#pragma unroll
    for (uint32_t j = 0; j < LOADS; ++j) load(to, j);
    advance();
  };
  struct Codes {
    i32x4 w[FN], x[FT];
  };
  // The i-th read of 64 codes of a stage: channels, then tokens.
  const auto read = [&](const unsigned char* from, uint32_t half, uint32_t i, Codes& c) {
    const uint32_t place_of = ((half * 4 + lane / 16) ^ (lane % 8)) * 16;
    if (i < FN) c.w[i] = *reinterpret_cast<const i32x4*>(from + (TT + wn + i * 16 + lane % 16) * kWide + place_of);
    else c.x[i - FN] = *reinterpret_cast<const i32x4*>(from + (wt + (i - FN) * 16 + lane % 16) * kWide + place_of);
  };
  i32x4 acc[FT][FN] = {};
  // The products of 64 codes.  Between the rows of them go the reads of the next 64
  // (`half` of `from`) and, with `to`, the loads of a stage, one by one: many at once
  // would fill the memory pipe, and the products behind them would wait.
  const auto multiply = [&](const Codes& c, const unsigned char* from, uint32_t half, Codes& next, unsigned char* to) {
#pragma unroll
    for (uint32_t i = 0; i < FT; ++i) {
#pragma unroll
      for (uint32_t r = i * (FT + FN) / FT; r < (i + 1) * (FT + FN) / FT; ++r) read(from, half, r, next);
      if (to) {
#pragma unroll
        for (uint32_t r = i * LOADS / FT; r < (i + 1) * LOADS / FT; ++r) load(to, r);
      }
#pragma unroll
      for (uint32_t j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(c.w[j], c.x[i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The next stage's loads done (as many as later stages' may be on their way),
  // every wave's too, and the stage before it read by all.
  const auto meet = [&]() {
    constexpr uint32_t pending = (STAGES - 2) * LOADS;
    // lgkmcnt 0: its reads are done; no access of LDS moves over this
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(pending) : "memory");
  };
  Codes first, second;
  // One stage, whose first 64 codes are read: its others are read under their
  // products, the next stage's first under the others', and this stage's place is
  // loaded again once all have read it.
  const auto step = [&](unsigned char* now, unsigned char* next) {
    multiply(first, now, 1, second, nullptr);
    meet();
    multiply(second, next, 0, first, now);
    advance();
    return --left > 0;
  };
  open();
#pragma unroll
  for (uint32_t s = 0; s < STAGES; ++s) load_all(stages + s * STAGE);
  {
    constexpr uint32_t pending = (STAGES - 1) * LOADS;
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(pending) : "memory");
  }
#pragma unroll
  for (uint32_t i = 0; i < FT + FN; ++i) read(stages, 0, i, first);
  for (bool more = left > 0; more;) {  // (a rank may hold none of the inner width)
#pragma unroll
    for (uint32_t s = 0; s < STAGES; ++s)
      if (!(more = step(stages + s * STAGE, stages + (s + 1) % STAGES * STAGE))) break;
  }
  // nothing on its way to LDS, and every stage read by all
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  store_tile<DT, FT, FN, STAGES * STAGE / WAVES>(a, own, channels, t0 + wt, n0 + wn, acc, stages + wave * (STAGES * STAGE / WAVES), lane);
}

// ---- few results

// Few tokens by few channels.  A workgroup takes 16 by 16 of them, so that few still
// fill the card; its waves take pieces of the inner width in turn, 256 codes of every
// row straight from memory in the layout that the matrix instruction reads, the next
// piece in flight while one is multiplied, and their sums are joined through LDS.  Rows
// of 16 codes at least, at any alignment (see keep_from).  Latency bounds it; rows about
// 1024 bytes apart, off alignment, also fall on one another in L1: 16 x 8200 x 256 on 8
// ranks 38 us, 11112 codes 24.5.
constexpr uint32_t kFewWaves = 16, kFewSteps = 4;

template <int DT>
__global__ __launch_bounds__(64 * kFewWaves) void product_few(ProductArgs a) {
  __shared__ i32x4 part[kFewWaves][64];
  constexpr uint32_t kPiece = 64 * kFewSteps;
  const bool dealt = a.form == 0;
  const uint32_t tiles_n = ((dealt ? a.channel_seg : a.channels) + 15) / 16;
  const uint32_t tiles_t = (a.rows + 15) / 16, t0 = blockIdx.x % tiles_t * 16;
  const uint32_t tn = blockIdx.x / tiles_t % tiles_n, own = blockIdx.x / tiles_t / tiles_n;
  const uint64_t before = uint64_t(own) * a.channel_seg;
  const uint32_t channels = !dealt ? a.channels : before < a.channels ? min(a.channel_seg, a.channels - static_cast<uint32_t>(before)) : 0;
  const uint32_t n0 = tn * 16;
  if (n0 >= channels) return;
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint32_t each = dealt ? a.inner : a.inner_seg, per_rank = (each + kPiece - 1) / kPiece;
  const uint32_t r0 = a.form <= 1 ? own : 0;
  const uint32_t pieces = per_rank * (a.form <= 1 ? 1 : static_cast<uint32_t>(a.P));
  // tokens and channels past the last one repeat it: their results are not stored
  const uint32_t row_t = min(lane % 16, a.rows - 1 - t0), row_n = min(lane % 16, channels - 1 - n0);
  const auto inner_of = [&](uint32_t rank) {
    const uint64_t lo = dealt ? 0 : uint64_t(rank) * a.inner_seg;
    return dealt ? a.inner : lo < a.inner ? min(a.inner_seg, a.inner - static_cast<uint32_t>(lo)) : 0;
  };
  struct Codes {
    i32x4 w[kFewSteps], x[kFewSteps];
  };
  const auto load = [&](uint32_t p, Codes& c) {
    const uint32_t rank = r0 + p / per_rank, k0 = p % per_rank * kPiece, inner = inner_of(rank);
    if (k0 >= inner) {  // past a rank with fewer pieces
#pragma unroll
      for (uint32_t s = 0; s < kFewSteps; ++s) c.x[s] = i32x4{0, 0, 0, 0};
      return;
    }
    const unsigned char* const w = a.w[rank] + uint64_t(n0) * inner;
    const unsigned char* const x = a.x[rank] + uint64_t(t0) * inner;
#pragma unroll
    for (uint32_t s = 0; s < kFewSteps; ++s) {
      const uint32_t k = min(k0 + s * 64 + lane / 16 * 16, inner - 16);
      c.w[s] = *reinterpret_cast<const i32x4_any*>(w + (row_n * inner + k));
      c.x[s] = *reinterpret_cast<const i32x4_any*>(x + (row_t * inner + k));
    }
  };
  i32x4 acc = {0, 0, 0, 0};
  const auto multiply = [&](uint32_t p, Codes& c) {
    const uint32_t k0 = p % per_rank * kPiece, inner = inner_of(r0 + p / per_rank);
    if (k0 < inner && k0 + kPiece > inner) {
#pragma unroll
      for (uint32_t s = 0; s < kFewSteps; ++s) {
        const uint32_t k = k0 + s * 64 + lane / 16 * 16;
        c.x[s] = keep_from(c.x[s], k - min(k, inner - 16));
      }
    }
#pragma unroll
    for (uint32_t s = 0; s < kFewSteps; ++s) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(c.w[s], c.x[s], acc, 0, 0, 0);
  };
  Codes first, second;
  uint32_t p = wave;
  if (p < pieces) {
    load(p, first);
    for (;;) {
      if (p + kFewWaves < pieces) load(p + kFewWaves, second);
      multiply(p, first);
      p += kFewWaves;
      if (p >= pieces) break;
      if (p + kFewWaves < pieces) load(p + kFewWaves, first);
      multiply(p, second);
      p += kFewWaves;
      if (p >= pieces) break;
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  i32x4 sum = part[0][lane];
#pragma unroll
  for (uint32_t w = 1; w < kFewWaves; ++w) sum += part[w][lane];
  const uint32_t t = t0 + lane % 16, n = n0 + lane / 16 * 4;
  if (t < a.rows && n < channels) store_results<DT>(a, own, channels, t, n, sum, a.x_scale[t]);
}

}  // namespace dev

namespace {

template <int DT, int VE>
void launch(const QuantizeArgs& a, hipStream_t stream) {
  const uint64_t per_rank = (a.seg + uint64_t(64) * VE - 1) / (64 * VE), pieces = per_rank * ((a.width + a.seg - 1) / a.seg);
  const uint32_t by = static_cast<uint32_t>(std::min<uint64_t>(UINT32_MAX, ((uint64_t(1) << 32) + per_rank - 1) / per_rank));
  const uint32_t grid = static_cast<uint32_t>(std::min<uint64_t>(a.rows, 1 << 20));
  // The fewest waves of these that hold a row (bf16, us, 8 ranks unless said).  One wave or
  // four: 16384 rows of 512 on one rank (1 piece) 12 and 21, of 2048 (4) 18 and 37, of 2560
  // (5) - and 37.  Four or 16: 4096 rows of 8192 (16) 23 and 42, of 11008 (24) - and 44, of
  // 16384 (32) - and 49.  16 of four vectors or of eight: 2048 rows of 28672 (56) 37 and 55,
  // of 32768 (64) 40 and 58.  16 of eight or read twice: of 36864 (72) 60 and 55, of 60000
  // (120) 85 and 92.  A piece past the row's last is the last one again, loaded and stored, so
  // a row that just misses a kind pays for the next one whole: 4096 x 8200 57 where x 8192 23
  // (eight waves of four would take 29, but are not among the kinds).
  if (pieces <= 4) dev::quantize_rows<DT, VE, 64, 4, false><<<grid, 64, 0, stream>>>(a, by);
  else if (pieces <= 16) dev::quantize_rows<DT, VE, 256, 4, false><<<grid, 256, 0, stream>>>(a, by);
  else if (pieces <= 64) dev::quantize_rows<DT, VE, 1024, 4, false><<<grid, 1024, 0, stream>>>(a, by);
  else if (pieces <= 128) dev::quantize_rows<DT, VE, 1024, 8, false><<<grid, 1024, 0, stream>>>(a, by);
  else dev::quantize_rows<DT, VE, 1024, 4, true><<<grid, 1024, 0, stream>>>(a, by);
}

template <int DT>
hipError_t launch(const QuantizeArgs& a, hipStream_t stream) {
  constexpr uint32_t VE = 16 / dev::Width<DT>::bytes;
  const uint32_t shortest = a.width % a.seg ? a.width % a.seg : a.seg;
  if (shortest < VE) launch<DT, 1>(a, stream);
  else launch<DT, VE>(a, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(int dtype, const QuantizeArgs& a, hipStream_t stream) {
  return dtype == dev::kF32 ? launch<dev::kF32>(a, stream) : dtype == dev::kF16 ? launch<dev::kF16>(a, stream) : launch<dev::kBF16>(a, stream);
}

namespace {

// Tiles of `tokens` by `channels` results.
uint64_t tiles_of(const ProductArgs& a, uint64_t tokens, uint64_t channels) {
  const uint64_t tiles_n = ((a.form == 0 ? a.channel_seg : a.channels) + channels - 1) / channels;
  return (a.rows + tokens - 1) / tokens * tiles_n * (a.form <= 1 ? a.P : 1);
}
uint64_t tiles_of(const ProductArgs& a, uint64_t tile) { return tiles_of(a, tile, tile); }

}  // namespace

bool product_fits(const ProductArgs& a) {
  return tiles_of(a, 64) <= kMaxProductTiles;
}

namespace {

// Whether every row of codes begins on 16 bytes and holds whole chunks of 16.
bool whole_chunks(const ProductArgs& a) {
  const bool dealt = a.form == 0;
  if ((dealt ? a.inner : a.inner_seg) % 16 != 0 || a.inner % 16 != 0) return false;
  for (int r = 0; r < a.P; ++r)
    if ((reinterpret_cast<uintptr_t>(a.x[r]) | reinterpret_cast<uintptr_t>(a.w[r])) % 16 != 0) return false;
  return true;
}

template <int DT>
void launch_few(const ProductArgs& a, hipStream_t stream) {
  dev::product_few<DT><<<static_cast<uint32_t>(tiles_of(a, 16)), 64 * dev::kFewWaves, 0, stream>>>(a);
}

template <int DT, uint32_t TT, uint32_t TN, uint32_t WT, uint32_t WN, bool SHORT = false>
void launch_any(const ProductArgs& a, hipStream_t stream) {
  dev::product_tiles<DT, TT, TN, WT, WN, SHORT><<<static_cast<uint32_t>(tiles_of(a, TT, TN)), 64 * WT * WN, 0, stream>>>(a);
}

template <int DT, uint32_t TT, uint32_t TN, uint32_t WT, uint32_t WN, uint32_t STAGES, bool TURN = false>
void launch_wide(const ProductArgs& a, hipStream_t stream) {
  dev::product_wide<DT, TT, TN, WT, WN, STAGES, TURN><<<static_cast<uint32_t>(tiles_of(a, TT, TN)), 64 * WT * WN, 0, stream>>>(a);
}

template <int DT>
hipError_t launch(const ProductArgs& a, hipStream_t stream) {
  const uint32_t shortest = a.form == 0 ? a.inner : a.inner % a.inner_seg ? a.inner % a.inner_seg : a.inner_seg;
  // Times below are us, of 8 ranks.  A single round of small workgroups is left to
  // product_few: 41 x 10496 x 1024 11.2 (in tiles of 64 by 32 20.5), 131 x 3989 x 28 9.3
  // (64 by 64 19.9), 3 x 8192 x 4096 8.6 (32 by 32 11.5); two rounds are not, 16 x 4096 x
  // 8192 11.2 (8.7), 512 x 3989 x 512 31 (21), but of one token at any alignment, whose
  // lanes ask for one row: 1 x 4099 x 8190 16.0 (18.6).
  const bool whole = whole_chunks(a);
  const auto rounds = [](uint64_t tiles) { return static_cast<double>((tiles + 255) / 256); };
  if (shortest < 16) {
    // 4096 x 100 x 4096 in tiles of 128 and 64 105 and 130; 1024 x 100 x 1024, 64 tiles of 128: 18.9 and 17.7.
    // Every rank's codes go one by one, also where the last alone has fewer than 16: 256 x 4548 x 4096
    // over 64 ranks (72 each, 12) 420, x 4608 (72 each) 61; x 465 over 16 (30 each, 15) 55, x 480 18.
    if (tiles_of(a, 128) >= 512) launch_any<DT, 128, 128, 2, 4, true>(a, stream);
    else launch_any<DT, 64, 64, 2, 2, true>(a, stream);
  } else if (tiles_of(a, 16) <= (whole || a.rows > 1 ? 256 : 512)) {
    launch_few<DT>(a, stream);
  } else if (!whole) {
    // so much to begin with and for a round of 256 tiles: 1024 x 8200 x 4096 in tiles of 64 and 128 115 and 73, 512 tokens 62 and 70
    if (10 + 27 * rounds(tiles_of(a, 64)) <= 25 + 62 * rounds(tiles_of(a, 128))) launch_any<DT, 64, 64, 2, 2>(a, stream);
    else launch_any<DT, 128, 128, 2, 4>(a, stream);
  } else if (a.rows <= 32) {
    // 16 x 4096 x 131072 in the first and the second 93 and 102 (tiles of 64 by 64 103), x 12288, 192 tiles, 10.3 and 11.2, x 8192 9.3 and 8.7
    if (tiles_of(a, 32, 64) >= 192) launch_wide<DT, 32, 64, 1, 4, 4, true>(a, stream);
    else launch_wide<DT, 32, 32, 2, 2, 8>(a, stream);
  } else if (a.rows <= 64 && tiles_of(a, 64) <= 128) {
    // more workgroups: 64 x 8192 x 4096 16.4, in tiles of 64 by 64 19.0; 64 x 4096 x 16384, 256 tiles of those, 13.9 in both
    launch_wide<DT, 64, 32, 2, 2, 4>(a, stream);
  } else if (a.rows <= 64 && tiles_of(a, 64, 256) >= 256) {
    // the tokens read by fewer: 64 x 4096 x 65536 52 and x 131072 102, in tiles of 64 by 64 59 and 111; x 32768, 128 tiles, 33.9 and 32.7
    launch_wide<DT, 64, 256, 2, 4, 4, true>(a, stream);
  } else {
    // us for a round of 256 tiles over 8192 codes: x 8192 x 4096 in tiles of 256, 128 and
    // 64, 4096 tokens 106, 149 and 211, 2048 84, 74 and 104, 1024 83, 41 and 57, 512 82, 35
    // and 29, 256 -, 32 and 20.  Other widths do not scale by their codes alone, but keep the
    // order: x 1024 26, 37 and 51; 23, 20 and 27; 22, 11 and 15; -, 9.9 and 8.3; -, 9.7 and
    // 6.9; x 28672 362, 521 and 772; 322, 266 and 411; 329, 144 and 217; -, 128 and 118; -,
    // 130 and 69.  So do results to all ranks (1024 tokens 98, 53 and 78) and the ranks' own
    // parts (46, 61 and 82)
    const double large = 107 * rounds(tiles_of(a, 256)), middle = 38 * rounds(tiles_of(a, 128)), small = 4 + 13 * rounds(tiles_of(a, 64));
    if (small <= middle && small <= large) launch_wide<DT, 64, 64, 2, 2, 4>(a, stream);
    else if (middle <= large) launch_wide<DT, 128, 128, 2, 4, 4>(a, stream);
    else launch_wide<DT, 256, 256, 2, 4, 2>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product(int dtype, const ProductArgs& a, hipStream_t stream) {
  return dtype == dev::kF32 ? launch<dev::kF32>(a, stream) : dtype == dev::kF16 ? launch<dev::kF16>(a, stream) : launch<dev::kBF16>(a, stream);
}

}  // namespace hbmc
