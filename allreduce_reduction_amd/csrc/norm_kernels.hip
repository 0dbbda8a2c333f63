// The norms before and after a block's end over the ranks' partial sums, with
// gate and residual scale, and their gradient (see hbmc_reduce_norm).
//
//   s = sum of the ranks' rows        r1 = 1 / rms(s)     n = s * r1 * w1
//   h = residual + scale * gate * n   r2 = 1 / rms(h)     out = h * r2 * w2
// and back, with g the sum of the ranks' gradients and a = g * w2,
//   u = h * r2                        dh = r2 * (a - u * mean(a * u)) + dresidual_out
//   b = scale * gate * w1 * dh        v = s * r1    ds = r1 * (b - v * mean(b * v))
// (mean(a * u) is r2 * mean(a * h): no power of r1 or r2, which would leave
// fp32's range long before the rows' squares do.)
//
// Both directions stream: a row is P operand rows in, P copies out and a few
// rows of one rank, each touched once, with every row statistic taken from
// registers.  What bounds them is HBM, at the rate of as many streams written as
// read: 4096 rows of 4096 bf16 over 8 ranks move 638 MB forward in 111 us (5.7
// TB/s) and 671 MB backward in 139 (4.8, 5.2 without the joining of the weights'
// gradients); a copy of one stream reaches 7.  One row alone takes 5.6 us: the
// launch and one round trip.
#include <algorithm>

#include "rowops.hpp"

namespace hbmc {
namespace dev {

// A row is held by WAVES waves, VPT vectors of VE elements a lane; SLOTS rows
// share a workgroup.  Rows of 16 waves (kWide) have 128 registers a lane: they
// read weights, and in the gradient the row's own operands, again where they are
// used (from L2) instead of holding them, and keep the gradient's sums over the
// rows in LDS.
template <int WAVES, int SLOTS>
struct RowTile {
  static constexpr int kThreads = 64 * WAVES;
  static constexpr int kSlots = SLOTS;
  static constexpr int kGroup = kThreads * kSlots;
  static constexpr bool kWide = WAVES == 16;
};

template <int WAVES>
using ForwardTile = RowTile<WAVES, (WAVES >= 4 ? 1 : 4 / WAVES)>;
// The gradient's workgroups stay for many rows and leave one row of partial
// sums each, so short rows share a workgroup of eight waves.  8 ranks, bf16, us
// with 16, eight and four waves: 16384 rows of 512 81, 75 and 95; 8192 of 1024
// 80, 77 and 96; 4096 of 2048 80, 78 and 95.
constexpr int grad_slots(int waves) { return waves >= 8 ? 1 : 8 / waves; }
template <int WAVES>
using GradTile = RowTile<WAVES, grad_slots(WAVES)>;

// Where a lane's k-th vector of a row starts.  The last vector of a row whose
// width is no multiple of VE ends with the row, overlapping its neighbour by
// `dup` elements: both lanes compute and store the same values there, and the
// row sums leave them out once.
template <int VE, int VPT, int WAVES>
struct Lane {
  uint32_t at[VPT];   // first element
  bool on[VPT];       // holds elements of the row
  uint32_t dup[VPT];  // leading elements the neighbour holds too
  __device__ __forceinline__ Lane(uint32_t tid, uint32_t width) {
    const uint32_t n = (width + VE - 1) / VE;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint32_t v = tid + k * 64 * WAVES;
      on[k] = v < n;
      const uint32_t c = on[k] ? v : n - 1;  // idle lanes read what the last one reads
      at[k] = c * VE + VE > width ? width - VE : c * VE;
      dup[k] = v == n - 1 ? n * VE - width : 0;
    }
  }
  // Has the compiler form the addresses that follow here, instead of keeping
  // them in registers between uses.
  __device__ __forceinline__ void forget(int k) { asm volatile("" : "+v"(at[k]), "+v"(dup[k])); }
};

// Sums over a row's waves of N values that every wave holds; `turn` counts the
// workgroup's calls, so that the buffer written is never one still being read.
template <int WAVES, int SLOTS, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float* red, uint32_t slot, uint32_t wave, uint32_t* turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
  if constexpr (WAVES > 1) {
    constexpr int kWidth = SLOTS * WAVES * 4;
    float* mine = red + (*turn & 1) * kWidth + slot * WAVES * 4;
    ++*turn;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) mine[wave * 4 + i] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += mine[w * 4 + i];
    }
  }
}

// Sum over the ranks of their rows' vectors, ranks ascending, with the loads of
// several ranks in flight.
template <int DT, int VE, int VPT, typename L>
__device__ __forceinline__ void sum_ranks(const unsigned char* const* bufs, int P, uint64_t row_off, const L& lane,
                                          float (&s)[VPT][VE]) {
  typedef Pack<DT, VE> K;
  constexpr int U = VPT == 1 ? 8 : 4 / VPT;
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) s[k][i] = 0.0f;
  int p = 0;
  for (; p + U <= P; p += U) {
    typename K::raw t[U][VPT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < VPT; ++k) t[u][k] = K::stream(bufs[p + u] + row_off + uint64_t(lane.at[k]) * K::E);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float f[VE];
        K::widen(t[u][k], f);
#pragma unroll
        for (int i = 0; i < VE; ++i) s[k][i] += f[i];
      }
  }
  if (p < P) {
    // the last P % U ranks: their loads issued together too
    typename K::raw t[U][VPT] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p + u < P) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) t[u][k] = K::stream(bufs[p + u] + row_off + uint64_t(lane.at[k]) * K::E);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p + u < P) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          float f[VE];
          K::widen(t[u][k], f);
#pragma unroll
          for (int i = 0; i < VE; ++i) s[k][i] += f[i];
        }
      }
  }
}

// One vector to every rank, rank after rank: issued eight at a time the same
// stores took 5% longer (8 ranks, 32 MiB each).
template <typename K, bool NT>
__device__ __forceinline__ void store_ranks(unsigned char* const* bufs, int P, uint64_t off, typename K::raw v) {
  for (int p = 0; p < P; ++p) {
    if constexpr (NT) K::store_nt(bufs[p] + off, v);
    else K::store(bufs[p] + off, v);
  }
}

// Sum of the terms f(i) of the lane's k-th vector that count for its row.
template <int VE, typename L, typename F>
__device__ __forceinline__ float vector_sum(const L& lane, int k, F&& f) {
  float part = 0.0f;
#pragma unroll
  for (int i = 0; i < VE; ++i) part += f(i);
  if (lane.dup[k] != 0) {
    part = 0.0f;
#pragma unroll
    for (int i = 0; i < VE; ++i) part += i >= static_cast<int>(lane.dup[k]) ? f(i) : 0.0f;
  }
  return lane.on[k] ? part : 0.0f;
}

template <int DT, int VE, int VPT, int WAVES, bool NT>
__global__ __launch_bounds__(ForwardTile<WAVES>::kGroup) void norm_kernel(NormPtrs a, NormShape s) {
  typedef Pack<DT, VE> K;
  typedef ForwardTile<WAVES> R;
  __shared__ float red[WAVES > 1 ? 2 * R::kSlots * WAVES * 4 : 1];
  const uint32_t wave_id = uniform(threadIdx.x >> 6);
  const uint32_t slot = wave_id / WAVES, wave = wave_id % WAVES;
  const Lane<VE, VPT, WAVES> lane(threadIdx.x - slot * R::kThreads, s.width);
  const unsigned char* w2p = static_cast<const unsigned char*>(s.pre_weight);
  const unsigned char* w1p = static_cast<const unsigned char*>(s.post_weight);
  const unsigned char* gp = static_cast<const unsigned char*>(s.gate);
  const float inv = 1.0f / static_cast<float>(s.width);
  uint32_t turn = 0;
  for (uint32_t base = blockIdx.x * R::kSlots; base < s.rows; base += gridDim.x * R::kSlots) {
    const bool active = base + slot < s.rows;
    const uint32_t row = uniform(active ? base + slot : s.rows - 1);
    const uint32_t owner = row / s.seg;
    const uint64_t off = uint64_t(row) * s.width * K::E, local = uint64_t(row - owner * s.seg) * s.width * K::E;
    const uint64_t gate_off = gp ? uint64_t(row / s.gate_rows) * s.width * K::E : 0;
    typename K::raw res[VPT], w2[VPT] = {}, w1[VPT] = {}, gt[VPT] = {};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint32_t b = lane.at[k] * K::E;
      res[k] = K::stream(a.residual[owner] + local + b);
      if constexpr (!R::kWide) {
        w2[k] = K::load(w2p + b);
        if (w1p) w1[k] = K::load(w1p + b);
        if (gp) gt[k] = K::load(gp + gate_off + b);
      }
    }
    float x[VPT][VE];
    sum_ranks<DT, VE, VPT>(a.parts, s.P, off, lane, x);
    if (a.save && active) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (lane.on[k]) K::store(a.sums[owner] + local + lane.at[k] * K::E, K::narrow(x[k]));
    }
    if (w1p) {
      float q[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < VPT; ++k) q[0] += vector_sum<VE>(lane, k, [&](int i) { return x[k][i] * x[k][i]; });
      row_sums<WAVES, R::kSlots>(q, red, slot, wave, &turn);
      const float r1 = 1.0f / sqrtf(q[0] * inv + s.post_eps);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float w[VE];
        if constexpr (R::kWide) w1[k] = K::load(w1p + lane.at[k] * K::E);
        K::widen(w1[k], w);
#pragma unroll
        for (int i = 0; i < VE; ++i) x[k][i] = x[k][i] * r1 * w[i];
      }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float r[VE];
      if (gp) {
        float g[VE];
        if constexpr (R::kWide) gt[k] = K::load(gp + gate_off + lane.at[k] * K::E);
        K::widen(gt[k], g);
#pragma unroll
        for (int i = 0; i < VE; ++i) x[k][i] *= g[i];
      }
      K::widen(res[k], r);
#pragma unroll
      for (int i = 0; i < VE; ++i) x[k][i] = r[i] + s.scale * x[k][i];
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) q[0] += vector_sum<VE>(lane, k, [&](int i) { return x[k][i] * x[k][i]; });
    row_sums<WAVES, R::kSlots>(q, red, slot, wave, &turn);
    const float r2 = 1.0f / sqrtf(q[0] * inv + s.pre_eps);
    // every operand is in registers by now in every wave of the row, so the
    // outputs may lie where the operands lay
    if (active) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (lane.on[k]) {
          const uint32_t b = lane.at[k] * K::E;
          K::store(a.residual_out[owner] + local + b, K::narrow(x[k]));
          float w[VE];
          if constexpr (R::kWide) w2[k] = K::load(w2p + b);
          K::widen(w2[k], w);
#pragma unroll
          for (int i = 0; i < VE; ++i) x[k][i] = x[k][i] * r2 * w[i];
          const typename K::raw y = K::narrow(x[k]);
          store_ranks<K, NT>(a.out, s.P, off + b, y);
        }
    }
  }
}

template <int DT, int VE, int VPT, int WAVES, bool NT>
__global__ __launch_bounds__(GradTile<WAVES>::kGroup) void norm_grad_kernel(NormGradPtrs a, NormShape s) {
  typedef Pack<DT, VE> K;
  typedef GradTile<WAVES> R;
  __shared__ float red[WAVES > 1 ? 2 * R::kSlots * WAVES * 4 : 1];
  const uint32_t wave_id = uniform(threadIdx.x >> 6);
  const uint32_t slot = wave_id / WAVES, wave = wave_id % WAVES;
  Lane<VE, VPT, WAVES> lane(threadIdx.x - slot * R::kThreads, s.width);
  const unsigned char* w2p = static_cast<const unsigned char*>(s.pre_weight);
  const unsigned char* w1p = static_cast<const unsigned char*>(s.post_weight);
  const unsigned char* gp = static_cast<const unsigned char*>(s.gate);
  const bool has_sum = w1p || gp;
  const float inv = 1.0f / static_cast<float>(s.width);
  const uint32_t chunk = blockIdx.x;
  constexpr int D = R::kWide ? 1 : VPT;
  // Sums over the rows: of g * h * r2 (the weight's gradient) and of
  // A = scale * dh * s * r1, from which both other gradients follow, the gate
  // row being the same for a whole group: post_weight's is the sum over the
  // groups of gate * A, the gate's is post_weight * A.
  float d2[D][VE] = {}, da[D][VE] = {};
  __shared__ __align__(16) float held[R::kWide ? 2 : 1][R::kWide ? VPT * VE * R::kThreads : 4];
  // the k-th vector's i-th element in `held`: a lane's 16 bytes side by side with its neighbours'
  const auto slot_of = [&](int k, int i) { return ((k * VE + i) / 4 * R::kThreads + threadIdx.x) * 4 + i % 4; };
  if constexpr (R::kWide) {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int i = 0; i < VE; ++i) held[0][slot_of(k, i)] = held[1][slot_of(k, i)] = 0.0f;
  }
  float* const mine = a.partial + uint64_t(a.direct ? chunk * R::kSlots + slot : chunk) * a.sets * s.width;
  if (a.direct && w1p) {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (lane.on[k]) {
        const float zero[VE] = {};
        store_floats<VE>(mine + s.width + lane.at[k], zero);
      }
  }
  uint32_t turn = 0;
  for (uint32_t it = 0; it < a.iterations; ++it) {
    uint32_t row, last, group = 0;  // `last`: the end of the rows it may come from
    bool flush = false;
    if (a.direct) {
      // whole gate groups: the slot's j-th one, row after row
      const uint32_t j = it / s.gate_rows, in = it - j * s.gate_rows;
      group = chunk * a.groups_per_chunk + slot + j * R::kSlots;
      row = group * s.gate_rows + in;
      last = s.rows;
      flush = in + 1 == s.gate_rows && group * s.gate_rows < s.rows;
    } else {
      // a gate group's rows dealt to its chunks in turn, so that the rows in
      // work at one time lie side by side in memory
      const uint32_t g = chunk / a.chunks_per_group, first = g * s.gate_rows;
      row = first + (chunk - g * a.chunks_per_group + it * a.chunks_per_group) * R::kSlots + slot;
      last = s.rows - first < s.gate_rows ? s.rows : first + s.gate_rows;
    }
    const bool active = row < last;
    row = uniform(active ? row : s.rows - 1);
    const uint32_t owner = row / s.seg;
    const uint64_t off = uint64_t(row) * s.width * K::E, local = uint64_t(row - owner * s.seg) * s.width * K::E;
    const uint64_t gate_off = gp ? uint64_t(row / s.gate_rows) * s.width * K::E : 0;
    typename K::raw hr[D], sr[D] = {}, w2[D], w1[D] = {}, gt[D] = {}, ir[VPT] = {};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint32_t b = lane.at[k] * K::E;
      if (a.has_in) ir[k] = K::stream(a.residual_in[owner] + local + b);
      if constexpr (!R::kWide) {
        hr[k] = K::stream(a.hidden[owner] + local + b);
        if (has_sum) sr[k] = K::stream(a.sums[owner] + local + b);
        w2[k] = K::load(w2p + b);
        if (w1p) w1[k] = K::load(w1p + b);
        if (gp) gt[k] = K::load(gp + gate_off + b);
      }
    }
    float g[VPT][VE];
    sum_ranks<DT, VE, VPT>(a.out_grads, s.P, off, lane, g);
    float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int j = R::kWide ? 0 : k;
      if constexpr (R::kWide) {
        __builtin_amdgcn_sched_barrier(0);  // one vector's operands at a time in registers
        lane.forget(k);
        const uint32_t b = lane.at[k] * K::E;
        hr[0] = K::load(a.hidden[owner] + local + b);
        if (w1p) sr[0] = K::load(a.sums[owner] + local + b);
        w2[0] = K::load(w2p + b);
      }
      float h[VE], w[VE];
      K::widen(hr[j], h);
      K::widen(w2[j], w);
      q[0] += vector_sum<VE>(lane, k, [&](int i) { return h[i] * h[i]; });
      q[1] += vector_sum<VE>(lane, k, [&](int i) { return g[k][i] * w[i] * h[i]; });
      if (w1p) {
        float x[VE];
        K::widen(sr[j], x);
        q[2] += vector_sum<VE>(lane, k, [&](int i) { return x[i] * x[i]; });
      }
    }
    row_sums<WAVES, R::kSlots>(q, red, slot, wave, &turn);
    const float r2 = 1.0f / sqrtf(q[0] * inv + s.pre_eps);
    const float c2 = r2 * (q[1] * inv);
    const float r1 = w1p ? 1.0f / sqrtf(q[2] * inv + s.post_eps) : 1.0f;
    // g becomes the gradient of the hidden row, then of the norm's output
    float inner[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int j = R::kWide ? 0 : k;
      if constexpr (R::kWide) {
        __builtin_amdgcn_sched_barrier(0);
        lane.forget(k);
      }
      const uint32_t b = lane.at[k] * K::E;
      if constexpr (R::kWide) {
        hr[0] = K::load(a.hidden[owner] + local + b);
        if (has_sum) sr[0] = K::load(a.sums[owner] + local + b);
        w2[0] = K::load(w2p + b);
        if (w1p) w1[0] = K::load(w1p + b);
        if (gp) gt[0] = K::load(gp + gate_off + b);
      }
      float h[VE], w[VE], x[VE], in[VE] = {};
      K::widen(hr[j], h);
      K::widen(w2[j], w);
      K::widen(sr[j], x);
      if (a.has_in) K::widen(ir[k], in);
      if (active) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          if constexpr (R::kWide) held[0][slot_of(k, i)] += g[k][i] * (h[i] * r2);
          else d2[j][i] += g[k][i] * (h[i] * r2);
        }
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) g[k][i] = r2 * (g[k][i] * w[i] - h[i] * r2 * c2) + in[i];
      if (active && lane.on[k]) K::store(a.residual_out[owner] + local + b, K::narrow(g[k]));
#pragma unroll
      for (int i = 0; i < VE; ++i) g[k][i] *= s.scale;
      if (has_sum && active) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          if constexpr (R::kWide) held[1][slot_of(k, i)] += g[k][i] * (x[i] * r1);
          else da[j][i] += g[k][i] * (x[i] * r1);
        }
      }
      if (gp) {
        K::widen(gt[j], w);
#pragma unroll
        for (int i = 0; i < VE; ++i) g[k][i] *= w[i];
      }
      if (w1p) {
        K::widen(w1[j], w);
#pragma unroll
        for (int i = 0; i < VE; ++i) g[k][i] *= w[i];
        inner[0] += vector_sum<VE>(lane, k, [&](int i) { return g[k][i] * x[i]; });
      }
    }
    if (w1p) {
      row_sums<WAVES, R::kSlots>(inner, red, slot, wave, &turn);
      const float c1 = r1 * (inner[0] * inv);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int j = R::kWide ? 0 : k;
        if constexpr (R::kWide) {
          __builtin_amdgcn_sched_barrier(0);
          lane.forget(k);
          sr[0] = K::load(a.sums[owner] + local + lane.at[k] * K::E);
        }
        float x[VE];
        K::widen(sr[j], x);
#pragma unroll
        for (int i = 0; i < VE; ++i) g[k][i] = r1 * (g[k][i] - x[i] * r1 * c1);
      }
    }
    if (active) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (lane.on[k]) {
          const typename K::raw y = K::narrow(g[k]);
          store_ranks<K, NT>(a.part_grads, s.P, off + lane.at[k] * K::E, y);
        }
    }
    if (flush) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int j = R::kWide ? 0 : k;
        const uint32_t b = lane.at[k] * K::E;
        if constexpr (R::kWide) {
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            da[0][i] = held[1][slot_of(k, i)];
            held[1][slot_of(k, i)] = 0.0f;
          }
        }
        if (lane.on[k]) {
          float w[VE], to[VE];
          if (w1p) {
            // added up in memory, element by element: a row's last two lanes
            // share some, and only one of them may add
            float* sum = mine + s.width + lane.at[k];
            K::widen(K::load(gp + gate_off + b), w);
#pragma unroll
            for (int i = 0; i < VE; ++i)
              if (i >= static_cast<int>(lane.dup[k])) sum[i] += da[j][i] * w[i];
            K::widen(K::load(w1p + b), w);
          }
#pragma unroll
          for (int i = 0; i < VE; ++i) to[i] = w1p ? da[j][i] * w[i] : da[j][i];
          store_floats<VE>(a.gate_grad + uint64_t(group) * s.width + lane.at[k], to);
        }
#pragma unroll
        for (int i = 0; i < VE; ++i) da[j][i] = 0.0f;
      }
    }
  }
  if constexpr (R::kSlots > 1) {
    if (!a.direct) {
      // one row of partial sums for all slots, slots ascending
      __shared__ float all[R::kGroup * VPT * VE];
      const auto join = [&](float (&d)[D][VE]) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int i = 0; i < VE; ++i) all[(k * VE + i) * R::kGroup + threadIdx.x] = d[k][i];
        __syncthreads();
        if (slot == 0) {
#pragma unroll
          for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i)
              for (int w = 1; w < R::kSlots; ++w) d[k][i] += all[(k * VE + i) * R::kGroup + w * R::kThreads + threadIdx.x];
        }
      };
      join(d2);
      if (has_sum) join(da);
      if (slot != 0) return;
    }
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    if (lane.on[k]) {
      const int j = R::kWide ? 0 : k;
      if constexpr (R::kWide) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          d2[0][i] = held[0][slot_of(k, i)];
          da[0][i] = held[1][slot_of(k, i)];
        }
      }
      store_floats<VE>(mine + lane.at[k], d2[j]);
      if (has_sum && !a.direct) store_floats<VE>(mine + s.width + lane.at[k], da[j]);
    }
}

// Joins the partial sums into the weights' gradients: 64 columns a workgroup,
// its 16 waves taking every 16th partial row.  blockIdx.y: pre_weight, then
// post_weight, then the gate's groups.
struct NormJoin {
  const float* partial;
  float* pre;
  float* post;                  // nullptr: none
  float* gate;
  const unsigned char* gate_w;  // rows that weigh the second set's sums for post, or nullptr
  const unsigned char* post_w;  // weighs them for the gate, or nullptr
  uint64_t count, per_group;    // partial rows in all, of one gate group
  uint32_t sets, width;
};
template <int DT>
__device__ __forceinline__ float one_float(const unsigned char* p, uint64_t i) {
  typedef Pack<DT, 1> K;
  float f[1];
  K::widen(K::load(p + i * K::E), f);
  return f[0];
}
template <int DT>
__global__ __launch_bounds__(1024) void norm_join_kernel(NormJoin j) {
  __shared__ float red[16][64];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t col = blockIdx.x * 64 + lane;
  uint32_t job = blockIdx.y;
  const bool is_pre = job == 0, is_post = job == 1 && j.post;
  float* out = is_pre ? j.pre : j.post;
  uint64_t lo = 0, hi = j.count;
  float by = 1.0f;
  if (!is_pre && !is_post) {
    job -= j.post ? 2 : 1;
    lo = job * j.per_group;
    hi = lo + j.per_group;
    out = j.gate + uint64_t(job) * j.width;
  }
  const bool weigh = is_post && j.gate_w;  // a gate row for each group's partial rows
  float total = 0.0f;
  if (col < j.width) {
    if (!is_pre && !is_post && j.post_w) by = one_float<DT>(j.post_w, col);
    const float* from = j.partial + (is_pre ? 0 : j.width) + col;
    const uint64_t step = uint64_t(j.sets) * j.width;
    uint64_t r = lo + wave;
    for (; r + 7 * 16 < hi; r += 8 * 16) {
      float t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = from[(r + u * 16) * step];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        total += weigh ? t[u] * one_float<DT>(j.gate_w, (r + u * 16) / j.per_group * j.width + col) : t[u];
    }
    for (; r < hi; r += 16)
      total += weigh ? from[r * step] * one_float<DT>(j.gate_w, r / j.per_group * j.width + col) : from[r * step];
  }
  red[wave][lane] = total;
  __syncthreads();
  if (wave == 0 && col < j.width) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += red[w][lane];
    out[col] = sum * by;
  }
}

}  // namespace dev

namespace {

using namespace dev;

// Vectors a lane and waves a row, by row vectors n of 16 bytes (or single
// elements below one vector).
struct RowForm {
  int ve, vpt, waves;
};
RowForm row_form(int dtype, uint32_t width, bool grad, uint32_t rows) {
  const int full = dtype == kF32 ? 4 : 8;
  if (width < static_cast<uint32_t>(full)) return {1, 1, 1};
  const uint32_t n = (width + full - 1) / full;
  // Forward, two vectors a lane from 512 rows on.  8 ranks, bf16, two vectors
  // and one: 8192 rows of 1024 60 and 66 us, 4096 of 2048 58.5 and 66, 4096 of
  // 4096 111 and 115, 2048 of 8192 115 and 128; 256 rows of 4096 10.2 and 9.4.
  // The gradient holds three times as much a lane and takes one, but for the
  // widths above 512 vectors (2048 rows of 8192: 146 and 149 us).
  const int two = !grad && rows >= 512 ? 2 : 1;
  if (n <= 64) return {full, 1, 1};
  if (n <= 128) return {full, two, 2 / two};
  if (n <= 256) return {full, two, 4 / two};
  if (n <= 512) return {full, two, 8 / two};
  if (n <= 1024) return grad ? RowForm{full, 2, 8} : RowForm{full, two, 16 / two};
  if (n <= 2048) return {full, 2, 16};
  return {full, 4, 16};  // fp32 only: 16 elements a lane at most
}

template <int N>
using Int = std::integral_constant<int, N>;

template <int DT, int VE, bool GRAD, typename F>
hipError_t with_waves(const RowForm& r, F&& f) {
  const Int<DT> dt;
  const Int<VE> ve;
  switch (r.vpt * 100 + r.waves) {
    case 101: return f(dt, ve, Int<1>(), Int<1>());
    case 102: return f(dt, ve, Int<1>(), Int<2>());
    case 104: return f(dt, ve, Int<1>(), Int<4>());
    case 108: return f(dt, ve, Int<1>(), Int<8>());
    case 208: return f(dt, ve, Int<2>(), Int<8>());
    case 216: return f(dt, ve, Int<2>(), Int<16>());
    default: break;
  }
  if constexpr (!GRAD) {
    switch (r.vpt * 100 + r.waves) {
      case 201: return f(dt, ve, Int<2>(), Int<1>());
      case 202: return f(dt, ve, Int<2>(), Int<2>());
      case 204: return f(dt, ve, Int<2>(), Int<4>());
      case 116: return f(dt, ve, Int<1>(), Int<16>());
      default: break;
    }
  }
  if constexpr (DT == kF32) {
    if (r.vpt == 4) return f(dt, ve, Int<4>(), Int<16>());
  }
  return hipErrorInvalidValue;
}

template <bool GRAD, typename F>
hipError_t with_form(int dtype, const RowForm& r, F&& f) {
  if (r.ve == 1) {
    const Int<1> one;
    if (dtype == kF32) return f(Int<kF32>(), one, one, one);
    if (dtype == kF16) return f(Int<kF16>(), one, one, one);
    return f(Int<kBF16>(), one, one, one);
  }
  if (dtype == kF32) return with_waves<kF32, 4, GRAD>(r, f);
  if (dtype == kF16) return with_waves<kF16, 8, GRAD>(r, f);
  return with_waves<kBF16, 8, GRAD>(r, f);
}

constexpr uint32_t kMaxGrid = 1 << 20;  // workgroups of a launch; the kernel strides past it

uint32_t up(uint32_t n, uint32_t by) { return n / by + (n % by != 0); }

// Whether the ranks' copies are stored with the nontemporal hint.  8 ranks,
// bf16, width 4096, with and without: 4096 rows (256 MiB) 111 and 125 us, their
// gradient 139 and 150; 2048 rows 58 and 62, 79 and 86; 1024 rows (64 MiB) 31
// and 27, 47 and 47.
bool stream_out(int dtype, const NormShape& s) {
  return uint64_t(s.rows) * s.width * (dtype == kF32 ? 4 : 2) * s.P >= kStreamBytes;
}

}  // namespace

hipError_t launch_norm(int dtype, const NormPtrs& a, const NormShape& s, hipStream_t stream) {
  const bool nt = stream_out(dtype, s);
  return with_form<false>(dtype, row_form(dtype, s.width, false, s.rows), [&](auto dt, auto ve, auto vpt, auto waves) {
    constexpr uint32_t kSlots = ForwardTile<waves>::kSlots;
    void* argv[] = {const_cast<NormPtrs*>(&a), const_cast<NormShape*>(&s)};
    return hipLaunchKernel(nt ? reinterpret_cast<const void*>(&norm_kernel<dt, ve, vpt, waves, true>)
                              : reinterpret_cast<const void*>(&norm_kernel<dt, ve, vpt, waves, false>),
                           dim3(std::min(up(s.rows, kSlots), kMaxGrid)), dim3(ForwardTile<waves>::kGroup), argv, 0, stream);
  });
}

NormGradSplit split_norm_grad(int dtype, const NormShape& s) {
  NormGradSplit d;
  const uint32_t S = grad_slots(row_form(dtype, s.width, true, s.rows).waves);
  // One workgroup a compute unit: each more leaves a row of partial sums more
  // (4096 rows of 4096, 8 ranks, bf16: 139 us with 256, 149 with 384, 144 with
  // 512, 152 with 1024 workgroups, 190 with 128).  Fewer where gate groups are
  // direct and longer than C / S rows: each slot takes at least a whole one
  // (8192 rows of 512, 8 ranks, bf16: one gate row 38 us; 16 rows a gate, 64
  // workgroups, 78; 32 rows, 32 workgroups, 123; 33 rows, not direct, 51).
  const uint32_t target = 256;
  const uint32_t C = up(std::max(up(s.rows, target), 1u), S) * S;  // rows a chunk
  const uint32_t R = s.gate_rows;
  d.groups = s.rows == 0 ? 0 : (s.rows - 1) / R + 1;
  d.direct = s.gate && d.groups > 1 && R <= C;
  if (d.direct) {
    d.groups_per_chunk = std::max(C / R / S, 1u) * S;
    d.chunks = up(d.groups, d.groups_per_chunk);
    d.iterations = d.groups_per_chunk / S * R;
  } else {
    d.chunks_per_group = up(R, C);
    d.chunks = d.groups * d.chunks_per_group;
    d.iterations = up(R, d.chunks_per_group * S);
  }
  d.sets = s.post_weight || (s.gate && !d.direct) ? 2 : 1;
  d.sums = d.direct ? d.chunks * S : d.chunks;
  d.bytes = uint64_t(d.sums) * d.sets * s.width * sizeof(float);
  return d;
}

hipError_t launch_norm_grad(int dtype, NormGradPtrs& a, const NormShape& s, const NormGradSplit& d, float* pre_grad,
                            float* post_grad, float* gate_grad, hipStream_t stream) {
  a.gate_grad = gate_grad;
  a.chunks_per_group = d.chunks_per_group;
  a.groups_per_chunk = d.groups_per_chunk;
  a.iterations = d.iterations;
  a.sets = d.sets;
  a.direct = d.direct;
  if (d.chunks > 0) {
    const bool nt = stream_out(dtype, s);
    const RowForm form = row_form(dtype, s.width, true, s.rows);
    const hipError_t e = with_form<true>(dtype, form, [&](auto dt, auto ve, auto vpt, auto waves) {
      void* argv[] = {&a, const_cast<NormShape*>(&s)};
      return hipLaunchKernel(nt ? reinterpret_cast<const void*>(&norm_grad_kernel<dt, ve, vpt, waves, true>)
                                : reinterpret_cast<const void*>(&norm_grad_kernel<dt, ve, vpt, waves, false>),
                             dim3(d.chunks), dim3(GradTile<waves>::kGroup), argv, 0, stream);
    });
    if (e != hipSuccess) return e;
  }
  NormJoin j;
  j.partial = a.partial;
  j.pre = pre_grad;
  j.post = s.post_weight ? post_grad : nullptr;
  j.gate = gate_grad;
  j.gate_w = d.direct ? nullptr : static_cast<const unsigned char*>(s.gate);
  j.post_w = static_cast<const unsigned char*>(s.post_weight);
  j.count = d.sums;
  j.per_group = std::max(d.chunks_per_group, 1u);
  j.sets = d.sets;
  j.width = s.width;
  const uint32_t jobs = 1 + (s.post_weight ? 1 : 0) + (s.gate && !d.direct ? d.groups : 0);
  const void* join = dtype == kF32   ? reinterpret_cast<const void*>(&norm_join_kernel<kF32>)
                     : dtype == kF16 ? reinterpret_cast<const void*>(&norm_join_kernel<kF16>)
                                     : reinterpret_cast<const void*>(&norm_join_kernel<kBF16>);
  void* argv[] = {&j};
  return hipLaunchKernel(join, dim3((s.width + 63) / 64, jobs), dim3(1024), argv, 0, stream);
}

}  // namespace hbmc
