// Layer norm and its backward pass (gfx950).
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps),
//   y = (x - mu) rstd gamma + beta                        (beta optional)
//   with xh = (x - mu) rstd, g = gamma dy:
//   dx = rstd (g - mean(g) - xh mean(g xh)) (+ add),
//   dgamma = sum over rows of dy xh, dbeta = sum over rows of dy.
//
// Both directions read each tensor once: a group of L lanes (a wave or less)
// or W waves holds a whole row in registers, so mean and variance are two
// sums over registers (the variance of the centred values, no cancellation).
// The backward pass keeps the columns' dgamma and dbeta sums in registers
// over all rows a group visits; blocks leave one partial row each and a
// second kernel adds those in a fixed order -- no atomics, results repeat.
#include "train.h"

namespace pg {
namespace {

constexpr int kThreads = 256;

template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int s = L / 2; s >= 1; s >>= 1) x += __shfl_xor(x, s, 64);
  return x;
}

// Sum over the W waves that share a row (every lane gets it). red holds 2 W
// floats per slot; callers alternate the slot, so one barrier is enough.
template <int W>
__device__ __forceinline__ float wave_join(float x, float* red, int wave) {
  if constexpr (W == 1) return x;
  if ((threadIdx.x & 63) == 0) red[wave] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) s += red[w];
  return s;
}

// y may be x itself, dx may be dy or add: a row is read whole before any of
// it is written.
//
// A row's geometry: L lanes, W waves (L == 64 if W > 1), CH chunks of 8
// columns a lane: chunk k of lane l of wave w starts at column
// 8 (l + L (w + W k)).
template <typename T, int L, int W, int CH>
__global__ __launch_bounds__(W == 16 ? 1024 : kThreads) void norm_kernel(
    const T* x, int64_t n, int d, int64_t ldx, const float* __restrict__ gamma,
    const float* __restrict__ beta, float eps, T* y, int64_t ldy,
    float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int NT = W == 16 ? 1024 : kThreads;
  constexpr int ROWS = NT / (L * W);                 // rows a block holds at once
  __shared__ float red[2][NT / 64];
  const int ln = threadIdx.x & (L - 1);
  const int wv = W > 1 ? (threadIdx.x >> 6) % W : 0;
  float* red0 = &red[0][(threadIdx.x >> 6) / W * W];
  float* red1 = &red[1][(threadIdx.x >> 6) / W * W];
  const int c0 = 8 * (ln + L * wv);
  const float fd = (float)d;       // divided by, not multiplied with 1/d: exact where the sum is
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < n; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t r = r0 + threadIdx.x / (L * W);
    const bool live = r < n;
    const T* src = x + (live ? r : 0) * ldx;
    Raw8<T> v[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + 8 * L * W * k;
      v[k] = load8(src + c, live ? d - c : 0);
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[k].get(i);  // zeros behind the row
    const float mu = wave_join<W>(group_sum<L>(s), red0, wv) / fd;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int left = d - (c0 + 8 * L * W * k);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = i < left ? v[k].get(i) - mu : 0.f;
        q += t * t;
      }
    }
    const float var = wave_join<W>(group_sum<L>(q), red1, wv) / fd;
    const float rs = 1.0f / sqrtf(var + eps);
    if (!live) continue;
    if (ln == 0 && wv == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
    T* dst = y + r * ldy;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + 8 * L * W * k, left = d - c;
      if (left <= 0) continue;
      const Raw8<float> g = load8(gamma + c, left);
      Raw8<float> b{};
      if (beta) b = load8(beta + c, left);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = (v[k].get(i) - mu) * rs * g.v[i] + b.v[i];
      store8(dst + c, o, left);
    }
  }
}

// Partial rows: block b leaves dgamma at part[b][0][dp), dbeta at
// part[b][1][dp), dp = d rounded up to 8.
template <typename T, int L, int W, int CH>
__global__ __launch_bounds__(W == 16 ? 1024 : kThreads) void norm_backward_kernel(
    const T* dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, int64_t n, int d,
    const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* add, int64_t ldadd, T* dx, int64_t lddx,
    float* __restrict__ part) {
  constexpr int NT = W == 16 ? 1024 : kThreads;
  constexpr int ROWS = NT / (L * W);
  constexpr int COLS = 8 * L * W * CH;               // columns a row's group covers
  __shared__ float red[4][NT / 64];
  __shared__ __attribute__((aligned(16))) float sh[COLS];   // gamma, then the joined sums
  const int ln = threadIdx.x & (L - 1);
  const int wv = W > 1 ? (threadIdx.x >> 6) % W : 0;
  const int grp = threadIdx.x / (L * W);
  const int c0 = 8 * (ln + L * wv);
  const float fd = (float)d;
  for (int c = threadIdx.x; c < COLS; c += NT) sh[c] = c < d ? gamma[c] : 0.f;
  __syncthreads();
  float ag[CH][8] = {}, ab[CH][8] = {};
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < n; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t r = r0 + grp;
    const bool live = r < n;
    const int64_t rc = live ? r : 0;
    Raw8<T> vx[CH], vy[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + 8 * L * W * k, left = live ? d - c : 0;
      vx[k] = load8(x + rc * ldx + c, left);
      vy[k] = load8(dy + rc * lddy + c, left);
    }
    const float mu = mean[rc], rs = rstd[rc];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + 8 * L * W * k;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // dy and gamma are zero behind the row's end and for rows past n;
        // xh is finite there only if mu and rs are, so it is selected away
        const float xh = c + i < d && live ? (vx[k].get(i) - mu) * rs : 0.f;
        const float g = vy[k].get(i) * sh[c + i];
        s1 += g;
        s2 += g * xh;
        ag[k][i] += vy[k].get(i) * xh;
        ab[k][i] += vy[k].get(i);
      }
    }
    float* rd = &red[2 * flip][0] + (threadIdx.x >> 6) / W * W;
    float* rd2 = &red[2 * flip + 1][0] + (threadIdx.x >> 6) / W * W;
    flip ^= 1;
    s1 = group_sum<L>(s1);
    s2 = group_sum<L>(s2);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) {
        rd[wv] = s1;
        rd2[wv] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        s1 += rd[w];
        s2 += rd2[w];
      }
    }
    const float m1 = s1 / fd, m2 = s2 / fd;
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = c0 + 8 * L * W * k, left = d - c;
      if (left <= 0) continue;
      Raw8<T> va{};
      if (add) va = load8(add + r * ldadd + c, left);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (vx[k].get(i) - mu) * rs;
        o[i] = rs * (vy[k].get(i) * sh[c + i] - m1 - xh * m2);
        if (add) o[i] += va.get(i);
      }
      store8(dx + r * lddx + c, o, left);
    }
  }
  // join the block's groups in order through LDS, one partial row per block
  const int dp = (d + 7) / 8 * 8;
  float* pg_ = part + (int64_t)blockIdx.x * 2 * dp;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    for (int g = 0; g < ROWS; ++g) {
      __syncthreads();
      if (grp == g) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + 8 * L * W * k + i;
            const float a = which ? ab[k][i] : ag[k][i];
            sh[c] = g == 0 ? a : sh[c] + a;
          }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < dp; c += NT) pg_[which * dp + c] = c < d ? sh[c] : 0.f;
    __syncthreads();
  }
}

// dgamma, dbeta = sums of the partial rows in order: a block takes 16
// columns, 16 threads a column, each a contiguous run of partial rows.
__global__ __launch_bounds__(kThreads) void norm_join_kernel(
    const float* __restrict__ part, int64_t rows, int d, int dp, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  __shared__ float red[16][17];
  const int cl = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cl;                // column of [dgamma | dbeta], 2 dp wide
  const int64_t per = (rows + 15) / 16;
  const int64_t lo = seg * per, hi = lo + per < rows ? lo + per : rows;
  float s = 0.f;
  if (c < 2 * dp) {
#pragma unroll 8
    for (int64_t r = lo; r < hi; ++r) s += part[r * 2 * dp + c];
  }
  red[seg][cl] = s;
  __syncthreads();
  if (seg || c >= 2 * dp) return;
  float t = 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) t += red[q][cl];
  const int col = c < dp ? c : c - dp;
  if (col >= d) return;
  float* out = c < dp ? dgamma : dbeta;
  if (out) out[col] = t;
}

// The row geometry for width d, as f(L, W, CH) with integral constants.
template <int V>
using IC = std::integral_constant<int, V>;
template <typename F>
void with_geometry(int d, F f) {
  if (d <= 64) f(IC<8>{}, IC<1>{}, IC<1>{});
  else if (d <= 128) f(IC<16>{}, IC<1>{}, IC<1>{});
  else if (d <= 256) f(IC<32>{}, IC<1>{}, IC<1>{});
  else if (d <= 512) f(IC<64>{}, IC<1>{}, IC<1>{});
  else if (d <= 1024) f(IC<64>{}, IC<1>{}, IC<2>{});
  else if (d <= 1536) f(IC<64>{}, IC<1>{}, IC<3>{});
  else if (d <= 2048) f(IC<64>{}, IC<1>{}, IC<4>{});
  else if (d <= 2560) f(IC<64>{}, IC<1>{}, IC<5>{});
  else if (d <= 4096) f(IC<64>{}, IC<4>{}, IC<2>{});
  else if (d <= 8192) f(IC<64>{}, IC<4>{}, IC<4>{});
  else f(IC<64>{}, IC<16>{}, IC<2>{});
}

}  // namespace

hipError_t launch_layer_norm(const void* x, int32_t dtype, int64_t n, int d, int64_t ldx,
                             const float* gamma, const float* beta, float eps, void* y,
                             int64_t ldy, float* mean, float* rstd, hipStream_t s) {
  with_geometry(d, [&](auto L, auto W, auto CH) {
    constexpr int NT = W() == 16 ? 1024 : kThreads;
    constexpr int64_t ROWS = NT / (L() * W());
    const int64_t blocks = (n + ROWS - 1) / ROWS;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
    if (dtype == PG_F32)
      hipLaunchKernelGGL((norm_kernel<float, L(), W(), CH()>), grid, dim3(NT), 0, s,
                         static_cast<const float*>(x), n, d, ldx, gamma, beta, eps,
                         static_cast<float*>(y), ldy, mean, rstd);
    else
      hipLaunchKernelGGL((norm_kernel<uint16_t, L(), W(), CH()>), grid, dim3(NT), 0, s,
                         static_cast<const uint16_t*>(x), n, d, ldx, gamma, beta, eps,
                         static_cast<uint16_t*>(y), ldy, mean, rstd);
  });
  return hipGetLastError();
}

int64_t layer_norm_partials(int64_t n, int d) {
  int64_t rows = 1;
  with_geometry(d, [&](auto L, auto W, auto) {
    rows = (W() == 16 ? 1024 : kThreads) / (L() * W());
  });
  const int64_t blocks = (n + rows - 1) / rows;
  return blocks < 1024 ? blocks : 1024;
}

hipError_t launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                      int32_t dtype, int64_t n, int d, const float* gamma,
                                      const float* mean, const float* rstd, const void* add,
                                      int64_t ldadd, void* dx, int64_t lddx, float* dgamma,
                                      float* dbeta, float* part, hipStream_t s) {
  const int64_t blocks = layer_norm_partials(n, d);
  if (blocks > 0)
    with_geometry(d, [&](auto L, auto W, auto CH) {
      constexpr int NT = W() == 16 ? 1024 : kThreads;
      const dim3 grid((unsigned)blocks);
      if (dtype == PG_F32)
        hipLaunchKernelGGL((norm_backward_kernel<float, L(), W(), CH()>), grid, dim3(NT), 0, s,
                           static_cast<const float*>(dy), lddy, static_cast<const float*>(x), ldx,
                           n, d, gamma, mean, rstd, static_cast<const float*>(add), ldadd,
                           static_cast<float*>(dx), lddx, part);
      else
        hipLaunchKernelGGL((norm_backward_kernel<uint16_t, L(), W(), CH()>), grid, dim3(NT), 0, s,
                           static_cast<const uint16_t*>(dy), lddy,
                           static_cast<const uint16_t*>(x), ldx, n, d, gamma, mean, rstd,
                           static_cast<const uint16_t*>(add), ldadd, static_cast<uint16_t*>(dx),
                           lddx, part);
    });
  const int dp = (d + 7) / 8 * 8;
  hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((2 * dp + 15) / 16)), dim3(kThreads), 0, s,
                     part, blocks, d, dp, dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace pg
