// Declarations and small device helpers shared by the training-step operators:
// token embedding (embed.hip), layer norm (norm.hip) and the orthogonalised
// update (orthogonalize.hip). gfx950 only.
#pragma once

#include "common.h"

namespace pg {

// ---------------------------------------------------------------------------
// Vectors of 8 elements at any element alignment. gfx950 runs with unaligned
// global access enabled, so an 8-element move is 16-byte instructions whatever
// the row's address; rows of odd widths need no path of their own.

typedef __bf16 bf16v2_t __attribute__((ext_vector_type(2)));
typedef float f32v2_t __attribute__((ext_vector_type(2)));

// Two floats to packed bf16, nearest even, NaN kept; a in the low half.
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  const f32v2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16v2_t));
}

// Raw 8-element vector of T (float: 32 bytes, uint16_t holding bf16: 16).
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ float get(int i) const { return v[i]; }
};
template <>
struct Raw8<uint16_t> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};

// Between a wave's LDS writes and reads of them by its other lanes: orders the
// accesses for the compiler (a wave's LDS operations take effect in order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Part vectors move single elements, whole ones 16 bytes at a time. STREAM
// marks data that this call touches once and that is larger than the caches
// when speed matters: non-temporal stores and loads.
typedef uint32_t u32v4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool STREAM>
__device__ __forceinline__ void load16(const void* p, uint32_t (&w)[4]) {
  const auto* q = static_cast<const u32v4_any*>(p);
  const u32v4_any v = STREAM ? __builtin_nontemporal_load(q) : *q;
  w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  auto* q = static_cast<u32v4_any*>(p);
  const u32v4_any v = {a, b, c, d};
  if constexpr (STREAM) __builtin_nontemporal_store(v, q);
  else *q = v;
}

// p[0 .. min(8, left)) with zeros behind; left <= 0 reads nothing.
template <bool STREAM = false>
__device__ __forceinline__ Raw8<float> load8(const float* p, int left) {
  Raw8<float> r;
  if (left >= 8) {
    uint32_t a[4], b[4];
    load16<STREAM>(p, a);
    load16<STREAM>(p + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[i] = __uint_as_float(a[i]);
      r.v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < left ? p[i] : 0.f;
  }
  return r;
}
template <bool STREAM = false>
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* p, int left) {
  Raw8<uint16_t> r;
  if (left >= 8) {
    load16<STREAM>(p, r.w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < left ? p[2 * i] : 0u;
      const uint32_t hi = 2 * i + 1 < left ? p[2 * i + 1] : 0u;
      r.w[i] = lo | (hi << 16);
    }
  }
  return r;
}

// p[0 .. min(8, left)) = x, rounded to nearest even for bf16.
template <bool STREAM = false>
__device__ __forceinline__ void store8(float* p, const float (&x)[8], int left) {
  if (left >= 8) {
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      store16<STREAM>(p + i, __float_as_uint(x[i]), __float_as_uint(x[i + 1]),
                      __float_as_uint(x[i + 2]), __float_as_uint(x[i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = x[i];
  }
}
template <bool STREAM = false>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8], int left) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2_bf16(x[2 * i], x[2 * i + 1]);
  if (left >= 8) {
    store16<STREAM>(p, w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

// ---------------------------------------------------------------------------
// Launchers (all return hipError_t); arguments validated by api_train.hip.

hipError_t launch_embed(int32_t table_dtype, const void* table, int64_t V, int d, float scale,
                        const int32_t* tokens, int64_t n, int32_t out_dtype, void* out,
                        int64_t ld, int32_t* status, hipStream_t s);

// Row gradients of the embedding: workspace geometry, then the launcher
// (dtable NULL: sparse urows / ugrad / n_unique; otherwise dense).
struct EmbedPlan {
  int bits, rb, passes;       // key bits, bits per digit, digit passes
  int chunk;                  // sorted positions per reduction chunk
  int64_t nblk;               // blocks of a sort pass
  int64_t nchunk;
  int64_t off_keys[2], off_vals[2], off_counts, off_totals, off_heads, off_part, off_list;
  int64_t bytes;
};
EmbedPlan embed_plan(int64_t n, int64_t V, int d);
hipError_t launch_embed_backward(const EmbedPlan& p, const void* dout, int32_t dtype, int64_t ld,
                                 const int32_t* tokens, int64_t n, int64_t V, int d, float scale,
                                 int64_t* urows, float* ugrad, int64_t* n_unique, float* dtable,
                                 int accumulate, void* workspace, hipStream_t s);

constexpr int kNormMaxD = 16384;
hipError_t launch_layer_norm(const void* x, int32_t dtype, int64_t n, int d, int64_t ldx,
                             const float* gamma, const float* beta, float eps, void* y,
                             int64_t ldy, float* mean, float* rstd, hipStream_t s);
int64_t layer_norm_partials(int64_t n, int d);     // partial rows of the weight gradients
hipError_t launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                      int32_t dtype, int64_t n, int d, const float* gamma,
                                      const float* mean, const float* rstd, const void* add,
                                      int64_t ldadd, void* dx, int64_t lddx, float* dgamma,
                                      float* dbeta, float* part, hipStream_t s);

// Orthogonalised update: workspace geometry for n_mat matrices of r x c.
struct OrthoPlan {
  int m, n;                   // smaller and larger side
  int mp, np;                 // padded to whole tiles
  int small;                  // one block per matrix, in shared memory
  int norm_blocks;            // blocks of the norm reduction per matrix
  int64_t off_norm, off_x, off_xh, off_yh[2], off_o, off_d, off_b, off_bd;
  int64_t bytes;
};
OrthoPlan ortho_plan(int64_t n_mat, int64_t rows, int64_t cols);
struct OrthoArgs {
  int steps, split;           // split: leading steps on operands of two halves
  float a, b, c, eps, scale;
};
hipError_t launch_orthogonalize(const OrthoPlan& p, const void* G, int32_t dtype, int64_t n_mat,
                                int rows, int cols, const OrthoArgs& oa, uint16_t* out,
                                void* workspace, hipStream_t s);

}  // namespace pg
