// Orthogonalised update: Newton-Schulz products (gfx950).
//
// X_0 = G / (||G||_F + eps) with its smaller side first (X is m x n, m <= n;
// a tall G is taken transposed), then `steps` times
//   A = X X^T,  B = b A + c A A,  X <- a X + B X,
// which maps every singular value s of X to a s + b s^3 + c s^5 and leaves
// the singular vectors; out = scale X.
//
// The products run on the matrix cores in fp16 with fp32 accumulation. What
// keeps the rounding to fp16 far below the result's bf16:
//   * X itself stays in fp32 and enters as (a + B_ii) X_ij in the epilogue;
//     only the products read an fp16 copy;
//   * the diagonals of A and B, where most of their weight is, stay in fp32
//     vectors: A = D + O and B = E + F with O, F of zero diagonal,
//       F_ij = (b + c (D_i + D_j)) O_ij + c (O O)_ij           (i != j)
//       E_i  = b D_i + c ((O O)_ii + D_i^2);
//   * fixed powers of two place the fp16 copies: X 2^10, O 2^12, F 2^9, far
//     from overflow for every iterate the entry point admits (singular values
//     at most 3, |b s^2 + c s^4| at most 100) and with subnormals below 2^-33.
// bf16 operands, the usual choice, would be eight times coarser.
#include "train.h"

namespace pg {
namespace {

constexpr int kThreads = 256;
constexpr int kPad = 128;                 // padded sides are multiples of this
constexpr int kNormBlocks = 64;
constexpr float kSX = 1024.f, kSO = 4096.f, kSF = 512.f;   // fp16 placements

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float g_at(const float* G, int64_t i) { return G[i]; }
__device__ __forceinline__ float g_at(const uint16_t* G, int64_t i) { return bf16_to_f32(G[i]); }

// Sum of squares of matrix blockIdx.y in double (no overflow for any fp32
// input), one partial per block.
template <typename T>
__global__ __launch_bounds__(kThreads) void ns_norm_kernel(const T* __restrict__ G, int64_t count,
                                                           double* __restrict__ part) {
  __shared__ double sh[kThreads];
  const T* g = G + (int64_t)blockIdx.y * count;
  double s = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < count;
       i += (int64_t)gridDim.x * kThreads) {
    const double v = (double)g_at(g, i);
    s += v * v;
  }
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int o = kThreads / 2; o >= 1; o >>= 1) {
    if (threadIdx.x < o) sh[threadIdx.x] += sh[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sh[0];
}

// X, its fp16 copy and the copy's transpose from G, 64 x 64 tiles of X with
// zeros in the padding.
template <typename T>
__global__ __launch_bounds__(kThreads) void ns_load_kernel(
    const T* __restrict__ G, int rows, int cols, const double* __restrict__ part, int parts,
    float eps, int mp, int np, float* __restrict__ X, _Float16* __restrict__ Xh,
    _Float16* __restrict__ Yh) {
  __shared__ float t[64][65];
  const int64_t mat = blockIdx.z;
  double s = 0.0;
  for (int q = 0; q < parts; ++q) s += part[mat * parts + q];
  const double inv = s == 0.0 ? 0.0 : 1.0 / (sqrt(s) + (double)eps);
  const T* g = G + mat * rows * cols;
  const bool tall = rows > cols;                 // X = G^T
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;     // tile of X
  const int g0 = tall ? j0 : i0, h0 = tall ? i0 : j0;       // the same tile of G
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll 4
  for (int q = 0; q < 16; ++q) {
    const int r = g0 + ty + 4 * q, c = h0 + tx;
    t[ty + 4 * q][tx] =
        r < rows && c < cols ? (float)((double)g_at(g, (int64_t)r * cols + c) * inv) : 0.f;
  }
  __syncthreads();
  const int64_t base = mat * mp * np;
#pragma unroll 4
  for (int q = 0; q < 16; ++q) {
    const int a = ty + 4 * q;
    const float x = tall ? t[tx][a] : t[a][tx];            // X[i0 + a][j0 + tx]
    const float y = tall ? t[a][tx] : t[tx][a];            // X[i0 + tx][j0 + a]
    X[base + (int64_t)(i0 + a) * np + j0 + tx] = x;
    Xh[base + (int64_t)(i0 + a) * np + j0 + tx] = (_Float16)(x * kSX);
    Yh[base + (int64_t)(j0 + a) * mp + i0 + tx] = (_Float16)(y * kSX);
  }
}

enum { NS_GRAM, NS_POLY, NS_UPDATE };

struct NsArgs {
  const _Float16* P;      // left operand rows, K contiguous
  const _Float16* Q;      // right operand rows, K contiguous
  int K, mp, np;
  float a, b, c, scale;
  float* X;               // fp32 iterate [mp][np]
  _Float16 *Xh, *Yh;      // next copies (update)
  _Float16* O;            // A without its diagonal
  float* D;
  _Float16* F;            // B without its diagonal
  float* E;
  uint16_t* out;          // last update: the result, rows x cols
  int rows, cols;
};

// 64 x 64 tile of P Q^T, four waves of one 32 x 32 block each.
template <int MODE>
__global__ __launch_bounds__(kThreads) void ns_gemm_kernel(NsArgs g) {
  __shared__ __attribute__((aligned(16))) _Float16 sp[64][72], sq[64][72];
  const int64_t mat = blockIdx.z;
  const int64_t mm = mat * g.mp * g.mp, mn = mat * g.mp * g.np;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  const int K = g.K;
  const _Float16* P = g.P + (MODE == NS_GRAM ? mn : mm) + (int64_t)i0 * K;
  const _Float16* Q = g.Q + (MODE == NS_POLY ? mm : mn) + (int64_t)j0 * K;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
  f32x16_t acc = {};
  for (int k0 = 0; k0 < K; k0 += 64) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int e = threadIdx.x + q * kThreads, r = e >> 3, c = (e & 7) * 8;
      *reinterpret_cast<uint4*>(&sp[r][c]) =
          *reinterpret_cast<const uint4*>(P + (int64_t)r * K + k0 + c);
      *reinterpret_cast<uint4*>(&sq[r][c]) =
          *reinterpret_cast<const uint4*>(Q + (int64_t)r * K + k0 + c);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int kc = s * 16 + 8 * (lane >> 5);
      const f16x8_t pf = *reinterpret_cast<const f16x8_t*>(&sp[wi + (lane & 31)][kc]);
      const f16x8_t qf = *reinterpret_cast<const f16x8_t*>(&sq[wj + (lane & 31)][kc]);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(pf, qf, acc, 0, 0, 0);
    }
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int i = i0 + wi + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3);
    const int j = j0 + wj + (lane & 31);
    if constexpr (MODE == NS_GRAM) {
      const float v = acc[q] * (1.f / (kSX * kSX));
      g.O[mm + (int64_t)i * g.mp + j] = (_Float16)(i == j ? 0.f : v * kSO);
      if (i == j) g.D[mat * g.mp + i] = v;
    } else if constexpr (MODE == NS_POLY) {
      const float aa = acc[q] * (1.f / (kSO * kSO));
      const float di = g.D[mat * g.mp + i], dj = g.D[mat * g.mp + j];
      const float o = (float)g.O[mm + (int64_t)i * g.mp + j] * (1.f / kSO);
      const float f = (g.b + g.c * (di + dj)) * o + g.c * aa;
      g.F[mm + (int64_t)i * g.mp + j] = (_Float16)(i == j ? 0.f : f * kSF);
      if (i == j) g.E[mat * g.mp + i] = g.b * di + g.c * (aa + di * di);
    } else {
      const int64_t at = mn + (int64_t)i * g.np + j;
      const float x = (g.a + g.E[mat * g.mp + i]) * g.X[at] + acc[q] * (1.f / (kSF * kSX));
      if (g.out) {
        const bool tall = g.rows > g.cols;
        const int r = tall ? j : i, c = tall ? i : j;
        if (r < g.rows && c < g.cols)
          g.out[(mat * g.rows + r) * g.cols + c] = (uint16_t)pack2_bf16(g.scale * x, 0.f);
      } else {
        g.X[at] = x;
        g.Xh[at] = (_Float16)(x * kSX);
        g.Yh[mn + (int64_t)j * g.mp + i] = (_Float16)(x * kSX);
      }
    }
  }
}

int64_t al(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

OrthoPlan ortho_plan(int64_t n_mat, int64_t rows, int64_t cols) {
  OrthoPlan p{};
  p.m = (int)(rows < cols ? rows : cols);
  p.n = (int)(rows < cols ? cols : rows);
  p.mp = (p.m + kPad - 1) / kPad * kPad;
  p.np = (p.n + kPad - 1) / kPad * kPad;
  p.norm_blocks = kNormBlocks;
  const int64_t mn = n_mat * p.mp * p.np, mm = n_mat * p.mp * p.mp;
  int64_t off = 0;
  p.off_norm = off; off += al(n_mat * p.norm_blocks * 8);
  p.off_x = off; off += al(mn * 4);
  p.off_xh = off; off += al(mn * 2);
  for (int i = 0; i < 2; ++i) { p.off_yh[i] = off; off += al(mn * 2); }
  p.off_o = off; off += al(mm * 2);
  p.off_d = off; off += al(n_mat * p.mp * 4);
  p.off_b = off; off += al(mm * 2);
  p.off_bd = off; off += al(n_mat * p.mp * 4);
  p.bytes = off;
  return p;
}

hipError_t launch_orthogonalize(const OrthoPlan& p, const void* G, int32_t dtype, int64_t n_mat,
                                int rows, int cols, const OrthoArgs& oa, uint16_t* out,
                                void* workspace, hipStream_t s) {
  auto* ws = static_cast<uint8_t*>(workspace);
  auto* norm = reinterpret_cast<double*>(ws + p.off_norm);
  auto* X = reinterpret_cast<float*>(ws + p.off_x);
  auto* Xh = reinterpret_cast<_Float16*>(ws + p.off_xh);
  _Float16* Yh[2] = {reinterpret_cast<_Float16*>(ws + p.off_yh[0]),
                     reinterpret_cast<_Float16*>(ws + p.off_yh[1])};
  auto* O = reinterpret_cast<_Float16*>(ws + p.off_o);
  auto* D = reinterpret_cast<float*>(ws + p.off_d);
  auto* F = reinterpret_cast<_Float16*>(ws + p.off_b);
  auto* E = reinterpret_cast<float*>(ws + p.off_bd);
  const dim3 block(kThreads);
  const unsigned nm = (unsigned)n_mat;
  const dim3 lgrid((unsigned)(p.np / 64), (unsigned)(p.mp / 64), nm);
  auto load = [&](auto* g) {
    hipLaunchKernelGGL(ns_norm_kernel, dim3((unsigned)p.norm_blocks, nm), block, 0, s, g,
                       (int64_t)rows * cols, norm);
    hipLaunchKernelGGL(ns_load_kernel, lgrid, block, 0, s, g, rows, cols, norm, p.norm_blocks,
                       oa.eps, p.mp, p.np, X, Xh, Yh[0]);
  };
  if (dtype == PG_F32) load(static_cast<const float*>(G));
  else load(static_cast<const uint16_t*>(G));
  const dim3 sq((unsigned)(p.mp / 64), (unsigned)(p.mp / 64), nm);
  for (int k = 0; k < oa.steps; ++k) {
    NsArgs g{};
    g.mp = p.mp; g.np = p.np;
    g.a = oa.a; g.b = oa.b; g.c = oa.c; g.scale = oa.scale;
    g.X = X; g.Xh = Xh; g.O = O; g.D = D; g.F = F; g.E = E;
    g.rows = rows; g.cols = cols;
    g.P = Xh; g.Q = Xh; g.K = p.np;
    hipLaunchKernelGGL(ns_gemm_kernel<NS_GRAM>, sq, block, 0, s, g);
    g.P = O; g.Q = O; g.K = p.mp;
    hipLaunchKernelGGL(ns_gemm_kernel<NS_POLY>, sq, block, 0, s, g);
    g.P = F; g.Q = Yh[k & 1]; g.Yh = Yh[(k + 1) & 1];
    g.out = k + 1 == oa.steps ? out : nullptr;
    hipLaunchKernelGGL(ns_gemm_kernel<NS_UPDATE>, lgrid, block, 0, s, g);
  }
  return hipGetLastError();
}

}  // namespace pg
