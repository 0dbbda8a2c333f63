// Host <-> kernel interface of the operators over the ranks (norms at a block's
// end, embedding, distillation loss, gradient clipping, logits' penalties and
// masks, 8-bit products) and the device helpers they share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "elemops.hpp"
#include "plan.hpp"

namespace hbmc {

// How n rows or columns are dealt out: rank r owns [r * each, min(n, (r + 1) * each)).
inline uint64_t segment_each(uint64_t n, int P) { return (n + P - 1) / P; }
inline uint64_t segment_count(uint64_t n, int P, int r) {
  const uint64_t each = segment_each(n, P), lo = each * static_cast<uint64_t>(r);
  return lo >= n ? 0 : (n - lo < each ? n - lo : each);
}

// Outputs of at least this many bytes are stored with the nontemporal hint, past
// the memory-side cache; smaller ones are left there for whoever reads them
// next.  Embedding rows and then a copy of them, 8 ranks, bf16, width 4096, with
// and without the hint: 32 MiB 28.5 and 25.9 us, 64 MiB 56 and 52, 128 MiB 106
// and 119, 256 MiB 203 and 202 (the embedding alone 69 and 77).
constexpr uint64_t kStreamBytes = uint64_t(96) << 20;

// ------------------------------------------------- norms at a block's end

constexpr uint64_t kNormMaxWidth = 16384;  // 16 elements a thread, 1024 threads

struct NormShape {
  uint32_t rows, seg;  // rows (below 2^31), rows a rank owns
  uint32_t width;
  uint32_t gate_rows;  // rows that share a gate row, at most `rows`
  int P;
  float scale, pre_eps, post_eps;
  const void* pre_weight;
  const void* post_weight;
  const void* gate;
};

struct NormPtrs {
  const unsigned char* parts[kMaxRanks];
  unsigned char* out[kMaxRanks];
  const unsigned char* residual[kMaxRanks];
  unsigned char* residual_out[kMaxRanks];
  unsigned char* sums[kMaxRanks];
  bool save;
};

struct NormGradPtrs {
  const unsigned char* out_grads[kMaxRanks];
  unsigned char* part_grads[kMaxRanks];
  const unsigned char* hidden[kMaxRanks];
  const unsigned char* sums[kMaxRanks];
  const unsigned char* residual_in[kMaxRanks];
  unsigned char* residual_out[kMaxRanks];
  bool has_in;
  float* gate_grad;  // written here only when `direct`
  float* partial;    // [sums][sets][width]
  // A workgroup's chunk of rows (see split_norm_grad).
  uint32_t chunks_per_group, groups_per_chunk, iterations;
  uint32_t sets;
  bool direct;
};

// Rows of the gradient kernel dealt to workgroups: the number of partial sums
// and the workspace they need.
struct NormGradSplit {
  uint32_t chunks = 0, chunks_per_group = 0, groups_per_chunk = 0, iterations = 0, groups = 0;
  uint32_t sums = 0, sets = 1;  // rows of partial sums, kinds of sums in a row
  bool direct = false;
  uint64_t bytes = 0;
};
NormGradSplit split_norm_grad(int dtype, const NormShape& s);
hipError_t launch_norm(int dtype, const NormPtrs& a, const NormShape& s, hipStream_t stream);
hipError_t launch_norm_grad(int dtype, NormGradPtrs& a, const NormShape& s, const NormGradSplit& d, float* pre_grad,
                            float* post_grad, float* gate_grad, hipStream_t stream);

// -------------------------------------------------------------- embedding

constexpr uint64_t kMaxVocab = uint64_t(1) << 30;
constexpr uint64_t kMaxTokens = uint64_t(1) << 26;  // of one rank: a token's place is (rank << 26 | token)

struct EmbedArgs {
  const unsigned char* rows[kMaxRanks];  // tables, or gradients of the outputs
  const unsigned char* ids[kMaxRanks];
  unsigned char* out[kMaxRanks];         // outputs, or gradients of the tables
  uint32_t tokens[kMaxRanks];
  uint32_t seg;                          // vocabulary rows a rank owns
  uint32_t vocab, width;
  int P, id_bytes;
  float scale;
};

// Workspace of the gradient, from the tokens' total.
struct EmbedGradSplit {
  uint64_t total = 0;        // tokens of all ranks
  uint32_t rounds = 0, tiles = 0;  // pairs a thread sorts, sorting workgroups
  uint32_t bits = 0, passes = 0;
  uint32_t chunk = 0, chunks = 0;  // sorted tokens a wave adds up
  bool clear_all = false;          // clear every row, not only those without a token
  bool few = false;                // one launch, without sorting
  uint64_t key_a = 0, key_b = 0, place_a = 0, place_b = 0, hist = 0, touched = 0, partial = 0;  // byte offsets
  uint64_t bytes = 0;
};
EmbedGradSplit split_embed_grad(int dtype, uint64_t total, uint64_t vocab, uint64_t width);
// Whether every launch of the gradient stays below 2^32 threads.
bool embed_grad_fits(int dtype, uint64_t total, uint64_t width);
hipError_t launch_embed(int dtype, const EmbedArgs& a, hipStream_t stream);
hipError_t launch_embed_grad(int dtype, int grad_dtype, const EmbedArgs& a, const EmbedGradSplit& d, bool accumulate,
                             unsigned char* workspace, hipStream_t stream);

// ------------------------------------------------------ distillation loss

constexpr uint64_t kMaxTop = 1024;
constexpr float kLog2e = 1.44269504088896340736f;  // the kernels' exponents: differences * (1 / temperature * kLog2e)

struct DistillArgs {
  const unsigned char* logits[kMaxRanks];
  unsigned char* grads[kMaxRanks];
  uint64_t rows;
  uint32_t vocab, seg, top;
  int P, teacher_dtype, id_bytes;
  float temperature;
  const unsigned char* teacher;
  const unsigned char* ids;
  float* loss;
  float* lse;
  const float* loss_grad;
  float2* partial;  // [rows][parts]: (maximum, sum) of a piece of a rank's columns
  uint32_t parts, pieces;  // pieces of a rank's columns, pieces of all ranks
};
// Pieces of a rank's columns of a row, a wave's work each.
uint32_t distill_pieces(int dtype, bool grad, uint64_t seg);
uint64_t distill_workspace(int dtype, const DistillArgs& a);  // bytes of the loss
hipError_t launch_distill(int dtype, const DistillArgs& a, hipStream_t stream);
hipError_t launch_distill_grad(int dtype, const DistillArgs& a, hipStream_t stream);

// ------------------------------------------- norm and clipping of gradients

// A piece of a gradient tensor, a workgroup's work at a time.
struct GradPiece {
  unsigned char* data;
  uint64_t offset;  // bytes into the tensor: the piece's place in the other copies
  uint32_t count;   // elements
  uint32_t dtype;
  uint32_t first;   // of the other copies' addresses
  uint16_t copies;  // buffers that hold the tensor, `data`'s included
  uint16_t shifted; // whether any lies at another place in a line of 128 bytes
};

struct GradArgs {
  const GradPiece* pieces;
  unsigned char* const* others;  // the tensors' other copies
  uint32_t n;
  uint32_t sums;  // partial sums in `partial`
  int norm;       // 1, 2, or 0 for the largest value
  bool clip;      // whether the gradients are scaled
  uint64_t read, written;  // bytes of the tensors, of all their copies
  double scale, max_norm, eps;
  double* partial;
  float* norm_out;
};

constexpr uint64_t kGradPieceBytes = uint64_t(16) << 10;
constexpr uint64_t kMaxGradPieces = uint64_t(1) << 23;  // a workgroup each: below 2^32 threads
// Partial sums of so many pieces, whose copies hold `written` bytes (0: none are kept).
uint32_t grad_sums(uint64_t pieces, uint64_t written);
hipError_t launch_grad(const GradArgs& a, hipStream_t stream);

// ------------------------------------ penalties, biases and masks on logits

constexpr uint64_t kMaxHistory = (uint64_t(1) << 19) - 1;  // a column's count and its flags share 32 bits
constexpr uint64_t kMaxBias = (uint64_t(1) << 12) - 1;

struct LogitArgs {
  const unsigned char* logits[kMaxRanks];
  unsigned char* out[kMaxRanks];
  uint64_t rows;
  uint32_t vocab, seg;
  uint32_t tile, tiles;  // columns of a workgroup, tiles of a rank's columns
  int P, id_bytes, length_bytes, bias_id_bytes;
  bool in_place;
  const unsigned char* tokens;
  const unsigned char* prompt_lengths;
  const unsigned char* lengths;
  uint32_t history;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const unsigned char* bias_ids;
  const float* bias;
  uint32_t biases;
  const unsigned char* mask;
  uint32_t mask_bytes;  // of a row
};
uint32_t logit_tile(uint64_t rows, uint64_t seg, int P);
constexpr uint64_t kMaxLogitTiles = uint64_t(1) << 22;  // of a call: below 2^32 threads
hipError_t launch_logits(int dtype, const LogitArgs& a, hipStream_t stream);

// ---------------------------------------------- products in 8-bit integers

constexpr uint64_t kMaxInner = (uint64_t(1) << 17) - 1;  // sums of products of 8-bit values stay below 2^31

struct QuantizeArgs {
  const unsigned char* x[kMaxRanks];
  unsigned char* q[kMaxRanks];
  float* scale;
  uint64_t rows;
  uint32_t width, seg;
  int P;
};
hipError_t launch_quantize(int dtype, const QuantizeArgs& a, hipStream_t stream);

struct ProductArgs {
  const unsigned char* x[kMaxRanks];
  const unsigned char* w[kMaxRanks];
  const float* w_scale[kMaxRanks];
  unsigned char* out[kMaxRanks];
  const float* x_scale;
  uint32_t rows, row_seg;           // rows, rows that a rank owns
  uint32_t inner, inner_seg;        // inner width, of one rank
  uint32_t channels, channel_seg;   // channels, of one rank
  int P;
  int form;  // hbmc_product_form_t
};
constexpr uint64_t kMaxProductTiles = uint64_t(1) << 22;  // of 64 x 64 results: every launch stays below 2^32 threads
bool product_fits(const ProductArgs& a);
hipError_t launch_product(int dtype, const ProductArgs& a, hipStream_t stream);

// --------------------------------------------------------- device helpers

namespace dev {

// Vectors at any element alignment: gfx950 loads and stores global memory at
// any address, so rows of odd width need no path of their own.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// VE elements of type DT as they lie in memory, VE one or a 16-byte vector's.
template <int DT, int VE>
struct Pack {
  static constexpr uint32_t E = Width<DT>::bytes;
  static constexpr bool kVector = VE * E == 16;
  static_assert(kVector || VE == 1, "a vector or one element");
  typedef typename std::conditional<kVector, u32x4, uint32_t>::type raw;

  static __device__ __forceinline__ raw load(const unsigned char* p) {
    if constexpr (kVector) return *reinterpret_cast<const u32x4_any*>(p);
    else return load_elem<E>(p);
  }
  // For data read once.
  static __device__ __forceinline__ raw stream(const unsigned char* p) {
    if constexpr (kVector) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
    else return load_elem<E>(p);
  }
  static __device__ __forceinline__ void store(unsigned char* p, raw v) {
    if constexpr (kVector) *reinterpret_cast<u32x4_any*>(p) = v;
    else store_elem<E>(p, v);
  }
  // With the nontemporal hint, for outputs larger than the memory-side cache can hold.
  static __device__ __forceinline__ void store_nt(unsigned char* p, raw v) {
    if constexpr (kVector) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
    else store_elem<E>(p, v);
  }
  static __device__ __forceinline__ void widen(raw v, float (&f)[VE]) {
    if constexpr (!kVector) {
      f[0] = DT == kF32 ? u2f(v) : (DT == kBF16 ? u2f(v << 16) : widen_f16(v));
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == kF32) {
          f[i] = u2f(w[i]);
        } else if constexpr (DT == kBF16) {
          f[2 * i] = u2f(w[i] << 16);
          f[2 * i + 1] = u2f(w[i] & 0xffff0000u);
        } else {
          f[2 * i] = widen_f16(w[i] & 0xffffu);
          f[2 * i + 1] = widen_f16(w[i] >> 16);
        }
      }
    }
  }
  static __device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    if constexpr (DT == kBF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
    else return narrow_f16(lo) | (narrow_f16(hi) << 16);
  }
  static __device__ __forceinline__ raw narrow(const float (&f)[VE]) {
    if constexpr (!kVector) {
      if constexpr (DT == kF32) return f2u(f[0]);
      else return narrow2(f[0], 0.0f) & 0xffffu;
    } else if constexpr (DT == kF32) {
      return u32x4{f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3])};
    } else {
      return u32x4{narrow2(f[0], f[1]), narrow2(f[2], f[3]), narrow2(f[4], f[5]), narrow2(f[6], f[7])};
    }
  }
};

// VE floats at p.
template <int VE>
__device__ __forceinline__ void store_floats(float* p, const float (&f)[VE]) {
  if constexpr (VE == 1) {
    *p = f[0];
  } else {
#pragma unroll
    for (int i = 0; i < VE; i += 4) *reinterpret_cast<f32x4_any*>(p + i) = f32x4_any{f[i], f[i + 1], f[i + 2], f[i + 3]};
  }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float old, float x) {
  return u2f(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(f2u(old)), static_cast<int>(f2u(x)),
                                                              CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ float lane63(float x) {
  return u2f(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(f2u(x)), 63)));
}
// Sum and maximum over a whole wave (every lane active), in one fixed order:
// shifts by 1, 2, 4, 8 within rows of 16 lanes, then the rows joined.
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp_or<0x111, 0xf>(0.0f, x);
  x += dpp_or<0x112, 0xf>(0.0f, x);
  x += dpp_or<0x114, 0xf>(0.0f, x);
  x += dpp_or<0x118, 0xf>(0.0f, x);
  x += dpp_or<0x142, 0xa>(0.0f, x);
  x += dpp_or<0x143, 0xc>(0.0f, x);
  return lane63(x);
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp_or<0x111, 0xf>(x, x));
  x = fmaxf(x, dpp_or<0x112, 0xf>(x, x));
  x = fmaxf(x, dpp_or<0x114, 0xf>(x, x));
  x = fmaxf(x, dpp_or<0x118, 0xf>(x, x));
  x = fmaxf(x, dpp_or<0x142, 0xa>(x, x));
  x = fmaxf(x, dpp_or<0x143, 0xc>(x, x));
  return lane63(x);
}

__device__ __forceinline__ uint32_t uniform(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(x)));
}
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
  return (static_cast<uint64_t>(uniform(static_cast<uint32_t>(x >> 32))) << 32) | uniform(static_cast<uint32_t>(x));
}

}  // namespace dev
}  // namespace hbmc
