// Layer norm and its backward pass (gfx950).
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps),
//   y = (x - mu) rstd gamma + beta                        (beta optional)
//   with xh = (x - mu) rstd, g = gamma dy:
//   dx = rstd (g - mean(g) - xh mean(g xh)) (+ add),
//   dgamma = sum over rows of dy xh, dbeta = sum over rows of dy.
//
// Both directions are bound by memory and read each tensor once. A group of
// L lanes (rows up to 512 columns) or W waves (beyond) holds a whole row in
// registers, so mean and variance are two sums over registers (the variance
// of the centred values, no cancellation). A block walks many rows with the
// next row's loads in flight and gamma, beta in LDS. The backward pass keeps
// the columns' dgamma and dbeta sums in registers over all rows a group
// visits; blocks leave one partial row each and a second kernel adds those
// in a fixed order -- no atomics, results repeat.
#include <type_traits>

#include "train.h"

namespace pg {
namespace {

// Sum over the group of L lanes, in every lane.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int s = L / 2; s >= 1; s >>= 1) x += __shfl_xor(x, s, 64);
  return x;
}
// A whole wave: six adds on the vector unit's own lane moves (four shifts in
// rows of 16, two row broadcasts) leave the sum in lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_moved(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, true));
}
template <>
__device__ __forceinline__ float group_sum<64>(float x) {
  x = add_moved<0x111, 0xF>(x);        // row_shr:1
  x = add_moved<0x112, 0xF>(x);
  x = add_moved<0x114, 0xF>(x);
  x = add_moved<0x118, 0xF>(x);
  x = add_moved<0x142, 0xA>(x);        // row_bcast:15 into rows 1 and 3
  x = add_moved<0x143, 0xC>(x);        // row_bcast:31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// Threads of a block: one row's waves, or four waves of rows of their own.
template <int W>
constexpr int kNormThreads = W > 1 ? 64 * W : 256;

// A row's geometry: L lanes, W waves (L == 64 if W > 1), CH vectors of 8
// columns a lane: vector k of lane l of wave w starts at column
// 8 (l + L (w + W k)).
template <int L, int W, int CH>
struct Geo {
  static constexpr int NT = kNormThreads<W>;
  static constexpr int ROWS = NT / (L * W);          // rows a block holds at once
  static constexpr int STEP = 8 * L * W;             // columns between a lane's vectors
  static constexpr int COLS = STEP * CH;
};

// gamma (or beta) in LDS, as two planes of 16-byte halves of each 8-column
// vector: lanes then read consecutive 16-byte words.
template <int COLS, int NT>
__device__ __forceinline__ void stage_weights(float4 (&sh)[2][COLS / 8], const float* w, int d) {
  for (int v = threadIdx.x; v < COLS / 8; v += NT) {
    const Raw8<float> r = w ? load8(w + 8 * v, d - 8 * v) : Raw8<float>{};
    sh[0][v] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    sh[1][v] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
  }
}
template <int N>
__device__ __forceinline__ Raw8<float> staged(const float4 (&sh)[2][N], int v) {
  const float4 a = sh[0][v], b = sh[1][v];
  return Raw8<float>{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// y may be x itself: a row is read whole before any of it is written, and the
// rows prefetched are the group's own.
template <typename T, int L, int W, int CH>
__global__ __launch_bounds__(kNormThreads<W>) void norm_kernel(
    const T* x, int64_t n, int d, int64_t ldx, const float* __restrict__ gamma,
    const float* __restrict__ beta, float eps, T* y, int64_t ldy,
    float* __restrict__ mean, float* __restrict__ rstd) {
  using G = Geo<L, W, CH>;
  __shared__ float red[2][G::NT / 64];
  __shared__ float4 sg[2][G::COLS / 8], sb[2][G::COLS / 8];
  const int ln = threadIdx.x & (L - 1);
  const int wv = W > 1 ? threadIdx.x >> 6 : 0;
  const int c0 = 8 * (ln + L * wv);
  const float fd = (float)d;       // divided by, not multiplied with 1/d: exact where the sum is
  const int64_t stride = (int64_t)gridDim.x * G::ROWS;
  int64_t r = (int64_t)blockIdx.x * G::ROWS + threadIdx.x / (L * W);
  auto fetch = [&](int64_t row, Raw8<T> (&v)[CH]) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + G::STEP * k;
      v[k] = load8(x + (row < n ? row : 0) * ldx + c, row < n ? d - c : 0);
    }
  };
  // sum over the waves of a row; two slots in turn, so one barrier is enough
  auto join = [&](float s, int slot) {
    if constexpr (W == 1) return s;
    if ((threadIdx.x & 63) == 0) red[slot][wv] = s;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += red[slot][w];
    return t;
  };
  Raw8<T> v[CH];
  fetch(r, v);
  stage_weights<G::COLS, G::NT>(sg, gamma, d);
  stage_weights<G::COLS, G::NT>(sb, beta, d);
  __syncthreads();
  // the trip count is the block's: its first row decides
  for (int64_t r0 = (int64_t)blockIdx.x * G::ROWS; r0 < n; r0 += stride, r += stride) {
    Raw8<T> next[CH];
    fetch(r + stride, next);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[k].get(i);  // zeros behind the row
    const float mu = join(group_sum<L>(s), 0) / fd;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int left = d - (c0 + G::STEP * k);
      if (left >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = v[k].get(i) - mu;
          q += t * t;
        }
      } else if (left > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = i < left ? v[k].get(i) - mu : 0.f;
          q += t * t;
        }
      }
    }
    const float var = join(group_sum<L>(q), 1) / fd;
    const float rs = 1.0f / sqrtf(var + eps);
    if (r < n) {
      if (ln == 0 && wv == 0) {
        if (mean) mean[r] = mu;
        if (rstd) rstd[r] = rs;
      }
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = c0 + G::STEP * k;
        if (c >= d) continue;
        const Raw8<float> g = staged(sg, c >> 3), b = staged(sb, c >> 3);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (v[k].get(i) - mu) * rs * g.v[i] + b.v[i];
        store8<true>(y + r * ldy + c, o, d - c);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) v[k] = next[k];
  }
}

// dx may be dy or add, for the same reasons. Partial rows: block b leaves
// dgamma at part[b][0][dp), dbeta at part[b][1][dp), dp = d rounded up to 8.
template <typename T, int L, int W, int CH, bool ADD>
__global__ __launch_bounds__(kNormThreads<W>) void norm_backward_kernel(
    const T* dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, int64_t n, int d,
    const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* add, int64_t ldadd, T* dx, int64_t lddx,
    float* __restrict__ part) {
  using G = Geo<L, W, CH>;
  __shared__ float red[2][2][G::NT / 64];
  __shared__ float4 sg[2][G::COLS / 8];              // gamma
  __shared__ float sums[G::ROWS > 1 ? G::COLS : 1];
  const int ln = threadIdx.x & (L - 1);
  const int wv = W > 1 ? threadIdx.x >> 6 : 0;
  const int grp = threadIdx.x / (L * W);
  const int c0 = 8 * (ln + L * wv);
  const float fd = (float)d;
  const int64_t stride = (int64_t)gridDim.x * G::ROWS;
  int64_t r = (int64_t)blockIdx.x * G::ROWS + grp;
  // four vectors a lane of fp32 leave no registers for a third prefetched
  // tensor (123 spilled): add is then read where it is added. 4,000 rows of
  // 12,288: 165 us (4.8 TB/s), 261 prefetched; bf16 holds it and takes 98
  constexpr bool LATE = ADD && CH == 4 && sizeof(T) == 4;
  struct Row {
    Raw8<T> x[CH], y[CH], a[ADD && !LATE ? CH : 1];
    float mu, rs;
  };
  auto fetch = [&](int64_t row, Row& v) {
    const bool live = row < n;
    const int64_t rc = live ? row : 0;
    v.mu = mean[rc];
    v.rs = rstd[rc];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + G::STEP * k, left = live ? d - c : 0;
      v.x[k] = load8<true>(x + rc * ldx + c, left);
      v.y[k] = load8<true>(dy + rc * lddy + c, left);
      if constexpr (ADD && !LATE) v.a[k] = load8<true>(add + rc * ldadd + c, left);
    }
  };
  Row v;
  fetch(r, v);
  stage_weights<G::COLS, G::NT>(sg, gamma, d);
  __syncthreads();
  float ag[CH][8] = {}, ab[CH][8] = {};
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * G::ROWS; r0 < n; r0 += stride, r += stride) {
    Row next;
    fetch(r + stride, next);
    const bool live = r < n;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + G::STEP * k;
      const Raw8<float> gm = staged(sg, c >> 3);
      auto take = [&](int i, float xh) {
        const float g = v.y[k].get(i) * gm.v[i];
        s1 += g;
        s2 += g * xh;
        ag[k][i] += v.y[k].get(i) * xh;
        ab[k][i] += v.y[k].get(i);
      };
      // dy and gamma are zero behind the row's end, dy for rows past n; xh is
      // finite there only if mu and rs are, so it is selected away
      if (c + 8 <= d && live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) take(i, (v.x[k].get(i) - v.mu) * v.rs);
      } else if (c < d && live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) take(i, c + i < d ? (v.x[k].get(i) - v.mu) * v.rs : 0.f);
      }
    }
    s1 = group_sum<L>(s1);
    s2 = group_sum<L>(s2);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) {
        red[flip][0][wv] = s1;
        red[flip][1][wv] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        s1 += red[flip][0][w];
        s2 += red[flip][1][w];
      }
      flip ^= 1;
    }
    const float m1 = s1 / fd, m2 = s2 / fd;
    if (live) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = c0 + G::STEP * k;
        if (c >= d) continue;
        const Raw8<float> gm = staged(sg, c >> 3);
        Raw8<T> a{};
        if constexpr (LATE) a = load8<true>(add + r * ldadd + c, d - c);
        else if constexpr (ADD) a = v.a[k];
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (v.x[k].get(i) - v.mu) * v.rs;
          o[i] = v.rs * (v.y[k].get(i) * gm.v[i] - m1 - xh * m2);
          if constexpr (ADD) o[i] += a.get(i);
        }
        store8<true>(dx + r * lddx + c, o, d - c);
      }
    }
    v = next;
  }
  // one partial row per block; the groups of a block are joined in order
  const int dp = (d + 7) / 8 * 8;
  float* out = part + (int64_t)blockIdx.x * 2 * dp;
  if constexpr (G::ROWS > 1) {
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      for (int g = 0; g < G::ROWS; ++g) {
        __syncthreads();
        if (grp == g) {
#pragma unroll
          for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int c = c0 + G::STEP * k + i;
              const float a = which ? ab[k][i] : ag[k][i];
              sums[c] = g == 0 ? a : sums[c] + a;
            }
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < dp; c += G::NT) out[which * dp + c] = sums[c];
    }
  } else {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + G::STEP * k;
      if (c >= d) continue;
      store8(out + c, ag[k], 8);
      store8(out + dp + c, ab[k], 8);
    }
  }
}

// dgamma, dbeta = sums of the partial rows in order: a block takes 64
// columns, each of its 16 waves a contiguous run of partial rows.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void norm_join_kernel(
    const float* __restrict__ part, int64_t rows, int d, int dp, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  __shared__ float red[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;              // column of [dgamma | dbeta], 2 dp wide
  const int64_t per = (rows + kJoinWaves - 1) / kJoinWaves;
  const int64_t lo = wave * per, hi = lo + per < rows ? lo + per : rows;
  float s = 0.f;
  if (c < 2 * dp) {
#pragma unroll 16
    for (int64_t r = lo; r < hi; ++r) s += part[r * 2 * dp + c];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave || c >= 2 * dp) return;
  float t = 0.f;
#pragma unroll
  for (int q = 0; q < kJoinWaves; ++q) t += red[q][lane];
  const int col = c < dp ? c : c - dp;
  if (col >= d) return;
  float* out = c < dp ? dgamma : dbeta;
  if (out) out[col] = t;
}

// The row geometry for width d, as f(L, W, CH) with integral constants:
// lanes of one wave up to 512 columns, then as many waves as make one vector
// a lane, then more vectors.
template <int V>
using IC = std::integral_constant<int, V>;
template <typename F>
void with_geometry(int d, F f) {
  if (d <= 64) return f(IC<8>{}, IC<1>{}, IC<1>{});
  if (d <= 128) return f(IC<16>{}, IC<1>{}, IC<1>{});
  if (d <= 256) return f(IC<32>{}, IC<1>{}, IC<1>{});
  switch ((d + 511) / 512) {
    case 1: return f(IC<64>{}, IC<1>{}, IC<1>{});
    case 2: return f(IC<64>{}, IC<2>{}, IC<1>{});
    case 3: return f(IC<64>{}, IC<3>{}, IC<1>{});
    case 4: return f(IC<64>{}, IC<4>{}, IC<1>{});
    case 5: return f(IC<64>{}, IC<5>{}, IC<1>{});
    case 6: return f(IC<64>{}, IC<6>{}, IC<1>{});
    case 7: return f(IC<64>{}, IC<7>{}, IC<1>{});
    case 8: return f(IC<64>{}, IC<8>{}, IC<1>{});
  }
  if (d <= 8192) return f(IC<64>{}, IC<8>{}, IC<2>{});
  return f(IC<64>{}, IC<8>{}, IC<4>{});
}

// Blocks that walk n rows: enough to fill the chip's 256 compute units
// `waves` waves deep, no more than there are rows, and past one block a unit
// `per` rows a group or more. 131,072 rows of 2,560 bf16:
// forward 296, 264 and 316 us at 15, 20 and 30 waves, backward 511, 490, 512
// and 542 us at 10, 15, 20 and 30. Whole blocks only: a backward block of
// eight waves, rows beyond 3,584 columns, has a unit to itself, eight waves
// deep (65,536 bf16 rows, with add: 4,096 columns 421 us, 5.1 TB/s, 3,584
// columns 314 us, 6.0; 32,768 of 8,192, two vectors a lane, 351 us, 6.1).
template <int L, int W>
int64_t norm_blocks(int64_t n, int waves, int per) {
  constexpr int NT = kNormThreads<W>;
  constexpr int64_t ROWS = NT / (L * W);
  const int64_t one = (n + ROWS - 1) / ROWS, few = (one + per - 1) / per;
  const int64_t need = std::min<int64_t>(one, std::max<int64_t>(few, 256));
  return std::min<int64_t>(need, 256 * (int64_t)(waves * 64 / NT));
}
constexpr int kForwardWaves = 20, kBackwardWaves = 15;
// Rows a backward group takes before a block beyond the 256th starts: each
// block's partial row costs as much as two thirds of a bf16 row of all four
// tensors (4,095 rows of 1,001 fp32: 22, 20, 23 and 31 us at 2, 4, 8 and 16).
constexpr int kBackwardRows = 4;

}  // namespace

hipError_t launch_layer_norm(const void* x, int32_t dtype, int64_t n, int d, int64_t ldx,
                             const float* gamma, const float* beta, float eps, void* y,
                             int64_t ldy, float* mean, float* rstd, hipStream_t s) {
  with_geometry(d, [&](auto L, auto W, auto CH) {
    const dim3 grid((unsigned)norm_blocks<L(), W()>(n, kForwardWaves, 1)), block(kNormThreads<W()>);
    if (dtype == PG_F32)
      hipLaunchKernelGGL((norm_kernel<float, L(), W(), CH()>), grid, block, 0, s,
                         static_cast<const float*>(x), n, d, ldx, gamma, beta, eps,
                         static_cast<float*>(y), ldy, mean, rstd);
    else
      hipLaunchKernelGGL((norm_kernel<uint16_t, L(), W(), CH()>), grid, block, 0, s,
                         static_cast<const uint16_t*>(x), n, d, ldx, gamma, beta, eps,
                         static_cast<uint16_t*>(y), ldy, mean, rstd);
  });
  return hipGetLastError();
}

int64_t layer_norm_partials(int64_t n, int d) {
  int64_t blocks = 0;
  with_geometry(d, [&](auto L, auto W, auto) {
    blocks = norm_blocks<L(), W()>(n, kBackwardWaves, kBackwardRows);
  });
  return blocks;
}

hipError_t launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                      int32_t dtype, int64_t n, int d, const float* gamma,
                                      const float* mean, const float* rstd, const void* add,
                                      int64_t ldadd, void* dx, int64_t lddx, float* dgamma,
                                      float* dbeta, float* part, hipStream_t s) {
  const int64_t blocks = layer_norm_partials(n, d);
  if (blocks > 0)
    with_geometry(d, [&](auto L, auto W, auto CH) {
      auto go = [&](auto* yp, auto* xp, auto* ap, auto* op, auto ADD) {
        using T = std::remove_pointer_t<decltype(op)>;
        hipLaunchKernelGGL((norm_backward_kernel<T, L(), W(), CH(), ADD()>), dim3((unsigned)blocks),
                           dim3(kNormThreads<W()>), 0, s, yp, lddy, xp, ldx, n, d, gamma, mean,
                           rstd, ap, ldadd, op, lddx, part);
      };
      auto typed = [&](auto t) {
        using T = decltype(t);
        const T* yp = static_cast<const T*>(dy);
        const T* xp = static_cast<const T*>(x);
        const T* ap = static_cast<const T*>(add);
        if (add) go(yp, xp, ap, static_cast<T*>(dx), std::true_type{});
        else go(yp, xp, ap, static_cast<T*>(dx), std::false_type{});
      };
      if (dtype == PG_F32) typed(float{});
      else typed(uint16_t{});
    });
  const int dp = (d + 7) / 8 * 8;
  hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((2 * dp + 63) / 64)),
                     dim3(64 * kJoinWaves), 0, s, part, blocks, d, dp, dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace pg
