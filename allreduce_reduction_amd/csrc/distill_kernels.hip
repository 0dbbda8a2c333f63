// Distillation from a teacher's top logits over logits whose columns are dealt
// out to the ranks, and the gradient of the logits (see hbmc_distill_loss).
//
// Both directions read the logits once: a wave takes a piece of a row's columns
// on one rank, all its vectors in flight at once.  The loss leaves each piece's
// maximum and its sum of exponentials relative to that maximum, and one wave a
// row joins them (log-sum-exp over the ranks) and adds the teacher's few terms;
// few short rows take one launch, a workgroup a row.  The gradient needs no join:
// a wave recomputes the teacher's distribution, writes temperature * loss_grad * p
// over its piece and then the columns that the teacher names.  HBM bounds both:
// 2048 x 131072 bf16 logits over 8 ranks, 537 MB, are read in 77 us (7.0 TB/s; the
// joining launch takes 7 more), read and written in 167 us (6.4 TB/s).  The
// exponentials come second (a quarter-rate instruction an element).
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

// Vectors of a lane in a piece: all in flight at once, more of them where nothing
// is stored.  8 ranks, bf16, 2048 x 131072: gradient with two, four and eight 187,
// 169 and 183 us; loss of 2048 x 100277 with four, six and eight 73, 85 and 72.
constexpr uint32_t kLossVectors = 8, kGradVectors = 4;

template <int DT, uint32_t VECTORS>
struct Piece {
  static constexpr int VE = 16 / Width<DT>::bytes;
  static constexpr uint32_t kElems = 64 * VECTORS * VE;
};

// exp(x) by the hardware's 2^x: about one unit of the last place, and the
// argument's rounding by the product, |x| * 2^-24.  For what is rounded to 16 bits,
// summed over many columns, or a teacher's q; fp32 gradients take the library's.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

__device__ __forceinline__ int64_t teacher_id(const DistillArgs& a, uint64_t i) {
  return a.id_bytes == 8 ? reinterpret_cast<const int64_t*>(a.ids)[i] : reinterpret_cast<const int32_t*>(a.ids)[i];
}

// The i-th teacher entry: its column (vocab where it does not count) and its
// logit.
__device__ __forceinline__ uint32_t teacher_entry(const DistillArgs& a, uint64_t i, float* t) {
  const int64_t id = teacher_id(a, i);
  float f[1];
  if (a.teacher_dtype == kF32) Pack<kF32, 1>::widen(Pack<kF32, 1>::load(a.teacher + i * 4), f);
  else if (a.teacher_dtype == kF16) Pack<kF16, 1>::widen(Pack<kF16, 1>::load(a.teacher + i * 2), f);
  else Pack<kBF16, 1>::widen(Pack<kBF16, 1>::load(a.teacher + i * 2), f);
  *t = f[0];
  return id >= 0 && id < static_cast<int64_t>(a.vocab) && f[0] != -__builtin_inff() ? static_cast<uint32_t>(id) : a.vocab;
}

// A row's teacher entries: a lane's first kHeld stay in registers, so that they
// are read once; further ones are read where they are used.  (Gradient of 2048
// x 50001 bf16 logits with 256 entries a row, when this was chosen: 110 us with
// four held, 126 with two, 115 with eight, 131 with 16.  Now 95; with 64 entries
// 78, with 1024 373.)
constexpr uint32_t kHeld = 4;
struct Teacher {
  float t[kHeld];
  uint32_t col[kHeld];  // vocab: does not count
  float top, sum;       // maximum and sum of exponentials
  __device__ __forceinline__ void load(const DistillArgs& a, uint64_t row, uint32_t lane) {
#pragma unroll
    for (uint32_t h = 0; h < kHeld; ++h) {
      col[h] = a.vocab;
      t[h] = 0.0f;
      if (h * 64 + lane < a.top) col[h] = teacher_entry(a, row * a.top + h * 64 + lane, &t[h]);
    }
  }
  // f(entry's logit, column) for the lane's entries that count.
  template <typename F>
  __device__ __forceinline__ void each(const DistillArgs& a, uint64_t row, uint32_t lane, F&& f) const {
#pragma unroll
    for (uint32_t h = 0; h < kHeld; ++h)
      if (col[h] < a.vocab) f(t[h], col[h]);
    for (uint32_t k = kHeld * 64 + lane; k < a.top; k += 64) {
      float x;
      const uint32_t c = teacher_entry(a, row * a.top + k, &x);
      if (c < a.vocab) f(x, c);
    }
  }
  // Fills top and sum; false where no entry counts.  The differences to the
  // largest entry are taken before the factor 1 / temperature: above 1 it would
  // take entries at the type's lowest or largest value past fp32's range, and a
  // row of them alone has differences of zero.
  __device__ __forceinline__ bool stats(const DistillArgs& a, uint64_t row, uint32_t lane) {
    float m = -__builtin_inff(), s = 0.0f;
    bool any = false;
    each(a, row, lane, [&](float x, uint32_t) {
      any = true;
      m = fmaxf(m, x);
    });
    if (__ballot(any) == 0) return false;
    top = wave_max(m);
    const float inv = 1.0f / a.temperature;
    each(a, row, lane, [&](float x, uint32_t) { s += exp_fast((x - top) * inv); });
    sum = wave_sum(s);
    return true;
  }
};

template <int DT>
__device__ __forceinline__ float logit_at(const DistillArgs& a, uint64_t row, uint32_t col) {
  const uint32_t owner = col / a.seg;
  const uint32_t cols = min(a.seg, a.vocab - owner * a.seg);
  float f[1];
  typedef Pack<DT, 1> K;
  K::widen(K::load(a.logits[owner] + (row * cols + (col - owner * a.seg)) * K::E), f);
  return f[0];
}

// A wave's piece: columns [first, limit) of the rank's `cols` of a row.  The last
// piece takes up to one vector a lane more, so that few columns past a multiple of
// the others' size are no piece of their own.
struct Place {
  uint64_t row;
  uint32_t rank, first, limit, cols;
};
__device__ __forceinline__ Place place_of(const DistillArgs& a, uint32_t row, uint32_t rank, uint32_t piece, uint32_t elems) {
  const uint64_t lo = uint64_t(rank) * a.seg;
  const uint32_t cols = lo >= a.vocab ? 0 : min(a.seg, a.vocab - static_cast<uint32_t>(lo));
  const uint32_t first = piece * elems;
  const uint32_t limit = piece + 1 == a.pieces || first + elems > cols ? cols : first + elems;
  return Place{row, rank, first, limit, cols};
}
// The unit-th piece of rank blockIdx.y.  Rank after rank the waves at work go
// through one buffer from end to end: with the ranks' pieces of a row side by
// side the gradient of 2048 x 131072 bf16 logits over 8 ranks took 185 us, so 167.
__device__ __forceinline__ Place place_of(const DistillArgs& a, uint32_t unit, uint32_t elems) {
  const uint32_t row = unit / a.pieces;
  return place_of(a, row, blockIdx.y, unit - row * a.pieces, elems);
}

// A lane's columns of a piece: its vectors, and for a piece that ends its
// rank's columns the columns past the last whole vector, one a lane.  Columns
// that are not there read as -infinity.
template <int DT, uint32_t VECTORS, bool WHOLE, bool STREAM>
struct Columns {
  static constexpr int VE = 16 / Width<DT>::bytes;
  typedef Pack<DT, VE> K;
  typedef Pack<DT, 1> K1;
  static constexpr uint32_t kCount = WHOLE ? VECTORS : VECTORS + 1;
  uint32_t at, end, rest;  // first column, end of the whole vectors, the lane's single column
  bool has_rest;
  typename K::raw v[kCount];
  uint32_t one;
  __device__ __forceinline__ Columns(const Place& p, uint32_t lane) {
    at = p.first + lane * VE;
    end = p.limit / VE * VE;
    rest = end + lane;
    has_rest = !WHOLE && rest < p.limit;
  }
  __device__ __forceinline__ bool on(uint32_t k) const { return WHOLE || at + k * 64 * VE < end; }
  __device__ __forceinline__ uint64_t byte(uint32_t k) const { return uint64_t(at + k * 64 * VE) * K::E; }
  __device__ __forceinline__ void load(const unsigned char* row) {
    constexpr uint32_t none = DT == kF32 ? 0xff800000u : (DT == kBF16 ? 0xff80ff80u : 0xfc00fc00u);
#pragma unroll
    for (uint32_t k = 0; k < kCount; ++k) {
      if constexpr (!WHOLE) v[k] = typename K::raw{none, none, none, none};
      if (on(k)) v[k] = STREAM ? K::stream(row + byte(k)) : K::load(row + byte(k));
    }
    one = none;
    if (has_rest) one = K1::load(row + uint64_t(rest) * K::E);
  }
  __device__ __forceinline__ float single() const {
    float f[1];
    K1::widen(one, f);
    return f[0];
  }
};

template <int DT, bool WHOLE, bool STREAM>
__device__ __forceinline__ float2 piece_stats(const Place& p, const unsigned char* row, uint32_t lane, float inv) {
  constexpr int VE = Piece<DT, kLossVectors>::VE;
  typedef Pack<DT, VE> K;
  Columns<DT, kLossVectors, WHOLE, STREAM> c(p, lane);
  c.load(row);
  float m = WHOLE ? -__builtin_inff() : c.single();
#pragma unroll
  for (uint32_t k = 0; k < c.kCount; ++k) {
    float f[VE];
    K::widen(c.v[k], f);
#pragma unroll
    for (int i = 0; i < VE; ++i) m = fmaxf(m, f[i]);
  }
  m = wave_max(m);
  const float base = m == -__builtin_inff() ? 0.0f : m, scale2 = inv * kLog2e;
  float s = WHOLE ? 0.0f : __builtin_amdgcn_exp2f((c.single() - base) * scale2);
#pragma unroll
  for (uint32_t k = 0; k < c.kCount; ++k) {
    float f[VE];
    K::widen(c.v[k], f);
#pragma unroll
    for (int i = 0; i < VE; ++i) s += __builtin_amdgcn_exp2f((f[i] - base) * scale2);
  }
  return float2{m, wave_sum(s)};
}

template <int DT, bool STREAM>
__global__ __launch_bounds__(256) void distill_part_kernel(DistillArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t units = static_cast<uint32_t>(a.rows) * a.pieces;  // below 2^32
  const float inv = 1.0f / a.temperature;
  for (uint32_t block = blockIdx.x; block < units / 4 + 1; block += gridDim.x) {
    const uint32_t unit = block * 4 + uniform(threadIdx.x >> 6);
    if (unit >= units) return;
    const Place p = place_of(a, unit, Piece<DT, kLossVectors>::kElems);
    const unsigned char* row = a.logits[p.rank] + p.row * p.cols * Width<DT>::bytes;
    float2 r = {-__builtin_inff(), 0.0f};
    const bool whole = p.limit - p.first == Piece<DT, kLossVectors>::kElems;
    if (p.first < p.cols) r = whole ? piece_stats<DT, true, STREAM>(p, row, lane, inv) : piece_stats<DT, false, STREAM>(p, row, lane, inv);
    if (lane == 0) a.partial[p.row * a.parts + p.rank * a.pieces + p.first / Piece<DT, kLossVectors>::kElems] = r;
  }
}

// A row's teacher entries and the student's logits at the held ones.
template <int DT>
struct RowEntries {
  Teacher e;
  float z[kHeld];
  __device__ __forceinline__ void load(const DistillArgs& a, uint64_t row, uint32_t lane) {
    e.load(a, row, lane);
#pragma unroll
    for (uint32_t h = 0; h < kHeld; ++h) z[h] = e.col[h] < a.vocab ? logit_at<DT>(a, row, e.col[h]) : 0.0f;
  }
};

// One wave: joins a row's (maximum, sum) pairs, adds the teacher's terms and
// stores the row's loss and log-sum-exp.
template <int DT>
__device__ __forceinline__ void finish_row(const DistillArgs& a, uint64_t row, uint32_t lane, const float2* part, uint32_t parts,
                                           RowEntries<DT>& entries) {
  Teacher& e = entries.e;
  const float (&z)[kHeld] = entries.z;
  const float inv = 1.0f / a.temperature;
  float m = -__builtin_inff(), s = 0.0f;
  for (uint32_t i = lane; i < parts; i += 64) m = fmaxf(m, part[i].x);
  m = wave_max(m);
  const float base = m == -__builtin_inff() ? 0.0f : m;
  // a piece of -inf alone has the sum 0 (or NaN)
  for (uint32_t i = lane; i < parts; i += 64)
    s += part[i].y * expf((part[i].x == -__builtin_inff() ? 0.0f : part[i].x - base) * inv);
  s = wave_sum(s);
  const float log_s = logf(s), lse = base * inv + log_s;
  float loss = 0.0f;
  if (e.stats(a, row, lane)) {
    const float log_sum = logf(e.sum), inv_sum = 1.0f / e.sum;
    const auto add = [&](float t, float logit) {
      const float far = (t - e.top) * inv, q = exp_fast(far) * inv_sum;
      // from the difference to the row's maximum: base * inv and with it lse may
      // lie past fp32's range.  s is zero for a row of -infinity alone.
      const float log_p = s == 0.0f ? -__builtin_inff() : (logit - base) * inv - log_s;
      const float term = q * (far - log_sum - log_p);
      loss += q == 0.0f ? 0.0f : term;
    };
#pragma unroll
    for (uint32_t h = 0; h < kHeld; ++h)
      if (e.col[h] < a.vocab) add(e.t[h], z[h]);
    for (uint32_t k = kHeld * 64 + lane; k < a.top; k += 64) {
      float t;
      const uint32_t col = teacher_entry(a, row * a.top + k, &t);
      if (col < a.vocab) add(t, logit_at<DT>(a, row, col));
    }
    loss = wave_sum(loss) * a.temperature * a.temperature;
  }
  if (lane == 0) {
    a.loss[row] = loss;
    a.lse[row] = lse;
  }
}

// Joins the pieces of distill_part_kernel: one wave a row.
template <int DT>
__global__ __launch_bounds__(256) void distill_join_kernel(DistillArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  for (uint64_t row = uint64_t(blockIdx.x) * 4 + uniform(threadIdx.x >> 6); row < a.rows; row += uint64_t(gridDim.x) * 4) {
    RowEntries<DT> entries;
    entries.load(a, row, lane);
    finish_row<DT>(a, row, lane, a.partial + row * a.parts, a.parts, entries);
  }
}

// The whole loss of few short rows in one launch: a workgroup a row, a wave
// every 16th piece.
constexpr uint32_t kRowWaves = 16;
template <int DT>
__global__ __launch_bounds__(64 * kRowWaves) void distill_row_kernel(DistillArgs a) {
  __shared__ float2 pairs[kRowWaves];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint64_t row = blockIdx.x;
  const float inv = 1.0f / a.temperature;
  RowEntries<DT> entries;
  if (wave == 0) entries.load(a, row, lane);
  float2 all = {-__builtin_inff(), 0.0f};
  for (uint32_t part = wave; part < a.parts; part += kRowWaves) {
    const uint32_t rank = part / a.pieces;
    const Place p = place_of(a, static_cast<uint32_t>(row), rank, part - rank * a.pieces, Piece<DT, kLossVectors>::kElems);
    if (p.first >= p.cols) continue;
    const unsigned char* at = a.logits[p.rank] + row * p.cols * Width<DT>::bytes;
    const bool whole = p.limit - p.first == Piece<DT, kLossVectors>::kElems;
    const float2 r = whole ? piece_stats<DT, true, false>(p, at, lane, inv) : piece_stats<DT, false, false>(p, at, lane, inv);
    // (m, s) pairs joined relative to their larger maximum; -infinity adds nothing but a NaN
    const float m = fmaxf(all.x, r.x), base = m == -__builtin_inff() ? 0.0f : m;
    all.y = all.y * exp_fast(((all.x == -__builtin_inff() ? base : all.x) - base) * inv) +
            r.y * exp_fast(((r.x == -__builtin_inff() ? base : r.x) - base) * inv);
    all.x = m;
  }
  if (lane == 0) pairs[wave] = all;
  __syncthreads();
  if (wave == 0) finish_row<DT>(a, row, lane, pairs, kRowWaves, entries);
}

// A teacher entry of a wave's piece: its column on the rank, its q, and the
// bits to store there.
struct Entry {
  uint32_t col;
  float q;
  uint32_t bits;
};

__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int DT, bool WHOLE, bool STREAM>
__device__ __forceinline__ void piece_grad(const DistillArgs& a, const Place& p, uint32_t lane, Entry* list) {
  constexpr int VE = Piece<DT, kGradVectors>::VE;
  typedef Pack<DT, VE> K;
  typedef Pack<DT, 1> K1;
  const uint64_t off = p.row * p.cols * K::E;
  const unsigned char* row = a.logits[p.rank] + off;
  unsigned char* out = a.grads[p.rank] + off;
  const float given = a.loss_grad[p.row], by = given * a.temperature, lse = a.lse[p.row];
  const float inv = 1.0f / a.temperature;
  Columns<DT, kGradVectors, WHOLE, STREAM> c(p, lane);
  Teacher teach;
  bool some = given != 0.0f;
  if (some) {
    teach.load(a, p.row, lane);
    c.load(row);
    some = teach.stats(a, p.row, lane);
  }
  if (!some) {
#pragma unroll
    for (uint32_t k = 0; k < c.kCount; ++k)
      if (c.on(k)) K::store(out + c.byte(k), typename K::raw{});
    if (c.has_rest) K1::store(out + uint64_t(c.rest) * K::E, 0);
    return;
  }
  // p = exp(z / temperature - lse).  The quotient is rounded by itself, as it was
  // for lse, so that the row's largest logit, however large, cancels: fused, the
  // difference would hold its rounding error.  Zero throughout where lse is an
  // infinity: z * FLT_MIN is finite or -infinity itself, of which that is taken.
  const bool past = __builtin_isinf(lse);
  const float scale = past ? __FLT_MIN__ : inv, shift = past ? -__builtin_inff() : -lse;
  const auto prob = [&](float z) {
    const float x = z * scale + shift;
    if constexpr (DT == kF32) return expf(x);
    else return exp_fast(x);
  };
  const uint32_t lo = p.rank * a.seg;
  const float inv_sum = 1.0f / teach.sum;
  uint32_t n = 0;
  for (uint32_t h = 0; h * 64 < a.top; ++h) {
    float t = 0.0f;
    uint32_t col = a.vocab;
    if (h < kHeld) {
#pragma unroll
      for (uint32_t g = 0; g < kHeld; ++g)
        if (g == h) t = teach.t[g], col = teach.col[g];
    } else {
      if (h * 64 + lane < a.top) col = teacher_entry(a, p.row * a.top + h * 64 + lane, &t);
    }
    const bool in = col < a.vocab && col >= lo + p.first && col - lo < p.limit;
    const uint64_t who = __ballot(in);
    if (in) {
      Entry& e = list[n + __popcll(who & ((uint64_t(1) << lane) - 1))];
      e.col = col - lo;
      e.q = exp_fast((t - teach.top) * inv) * inv_sum;
    }
    n += __popcll(who);
  }
  wave_order();
  // the values at the named columns, from the logits before they are written
  // over (grads may be logits); a column named twice gets one value twice
  for (uint32_t e = lane; e < n; e += 64) {
    const uint32_t col = list[e].col;
    float q = 0.0f, z[1];
    for (uint32_t j = 0; j < n; ++j) q += list[j].col == col ? list[j].q : 0.0f;
    K1::widen(K1::load(row + uint64_t(col) * K::E), z);
    const float value[1] = {by * (prob(z[0]) - q)};
    list[e].bits = K1::narrow(value);
  }
  wave_order();
#pragma unroll
  for (uint32_t k = 0; k < c.kCount; ++k) {
    float f[VE];
    K::widen(c.v[k], f);
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = by * prob(f[i]);
    if (c.on(k)) {
      if constexpr (STREAM) K::store_nt(out + c.byte(k), K::narrow(f));
      else K::store(out + c.byte(k), K::narrow(f));
    }
  }
  if (c.has_rest) {
    const float f[1] = {by * prob(c.single())};
    K1::store(out + uint64_t(c.rest) * K::E, K1::narrow(f));
  }
  wave_order();  // the same wave's stores to the same places follow
  for (uint32_t e = lane; e < n; e += 64) K1::store(out + uint64_t(list[e].col) * K::E, list[e].bits);
  wave_order();  // the list is free again
}

template <int DT, bool STREAM>
__global__ __launch_bounds__(256) void distill_grad_kernel(DistillArgs a) {
  extern __shared__ Entry lists[];  // [4][top]
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t units = static_cast<uint32_t>(a.rows) * a.pieces;
  for (uint32_t block = blockIdx.x; block < units / 4 + 1; block += gridDim.x) {
    const uint32_t unit = block * 4 + wave;
    if (unit >= units) return;
    const Place p = place_of(a, unit, Piece<DT, kGradVectors>::kElems);
    if (p.first >= p.cols) continue;
    const bool whole = p.limit - p.first == Piece<DT, kGradVectors>::kElems;
    if (whole) piece_grad<DT, true, STREAM>(a, p, lane, lists + wave * a.top);
    else piece_grad<DT, false, STREAM>(a, p, lane, lists + wave * a.top);
  }
}

}  // namespace dev

namespace {

using namespace dev;

// Four waves a workgroup for `waves` waves of each of P ranks.
hipError_t go(const void* f, uint64_t waves, int P, uint32_t shared, void** argv, hipStream_t stream) {
  const uint32_t groups = static_cast<uint32_t>(std::min<uint64_t>((waves + 3) / 4, 1 << 22));
  return hipLaunchKernel(f, dim3(groups, static_cast<uint32_t>(P)), dim3(256), argv, shared, stream);
}

constexpr uint64_t kFewRows = 512, kShortRow = uint64_t(256) << 10;

#define HBMC_BY_TYPE(kernel, ...)                                                        \
  (dtype == kF32   ? reinterpret_cast<const void*>(&kernel<kF32 __VA_ARGS__>)            \
   : dtype == kF16 ? reinterpret_cast<const void*>(&kernel<kF16 __VA_ARGS__>)            \
                   : reinterpret_cast<const void*>(&kernel<kBF16 __VA_ARGS__>))
#define HBMC_COMMA ,

// Logits of kStreamBytes and more are read, and their gradients stored, past
// the memory-side cache; of smaller ones the loss leaves them there for the
// gradient.  8 ranks, bf16, 131072 columns, with and without, loss and
// gradient: 2048 rows 87 and 100 us, 186 and 198; 256 rows 19.2 and 18.7, 30.7
// and 25 (nontemporal stores alone 25).
bool streams(int dtype, const DistillArgs& a) {
  return a.rows * a.vocab * (dtype == kF32 ? 4 : 2) >= kStreamBytes;
}

// Whether a loss takes one launch, a workgroup a row, instead of a launch for
// pieces and one that joins them.  8 ranks, 64 entries, one and two launches,
// us: one bf16 row of 32000 columns 6 and 11.5, of 131072 (256 KiB) 10.4 and
// 11.5; 256 rows of 32000 7.5 and 11.6, of 131072 14.8 and 18.5; 512 rows 12.7
// and 14, 30.7 and 30.7; 1024 rows of 32000 22.5 and 19.3; one fp32 row of
// 262144 (1 MiB) 19 and 11.8.
bool by_rows(int dtype, const DistillArgs& a) {
  return a.rows <= kFewRows && uint64_t(a.vocab) * (dtype == kF32 ? 4 : 2) <= kShortRow;
}

}  // namespace

uint64_t distill_workspace(int dtype, const DistillArgs& a) {
  return by_rows(dtype, a) ? 0 : a.rows * a.parts * sizeof(float2);
}

uint32_t distill_pieces(int dtype, bool grad, uint64_t seg) {
  const uint32_t vector = 64 * (dtype == kF32 ? 4 : 8), elems = vector * (grad ? kGradVectors : kLossVectors);
  return seg <= elems + vector ? 1 : static_cast<uint32_t>((seg - vector + elems - 1) / elems);
}

hipError_t launch_distill(int dtype, const DistillArgs& a, hipStream_t stream) {
  void* argv[] = {const_cast<DistillArgs*>(&a)};
  if (by_rows(dtype, a))
    return hipLaunchKernel(HBMC_BY_TYPE(distill_row_kernel), dim3(static_cast<uint32_t>(a.rows)), dim3(64 * kRowWaves), argv, 0, stream);
  const void* part = streams(dtype, a) ? HBMC_BY_TYPE(distill_part_kernel, HBMC_COMMA true)
                                       : HBMC_BY_TYPE(distill_part_kernel, HBMC_COMMA false);
  const hipError_t e = go(part, a.rows * a.pieces, a.P, 0, argv, stream);
  if (e != hipSuccess) return e;
  return go(HBMC_BY_TYPE(distill_join_kernel), a.rows, 1, 0, argv, stream);
}

hipError_t launch_distill_grad(int dtype, const DistillArgs& a, hipStream_t stream) {
  void* argv[] = {const_cast<DistillArgs*>(&a)};
  const void* grad = streams(dtype, a) ? HBMC_BY_TYPE(distill_grad_kernel, HBMC_COMMA true)
                                       : HBMC_BY_TYPE(distill_grad_kernel, HBMC_COMMA false);
  return go(grad, a.rows * a.pieces, a.P, 4 * a.top * sizeof(Entry), argv, stream);
}

#undef HBMC_COMMA
#undef HBMC_BY_TYPE

}  // namespace hbmc
