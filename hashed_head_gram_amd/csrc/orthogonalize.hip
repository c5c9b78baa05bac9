// Orthogonalised update: Newton-Schulz products (gfx950).
//
// X_0 = G / (||G||_F + eps) with its smaller side first (X is m x n, m <= n;
// a tall G is taken transposed), then `steps` times
//   A = X X^T,  B = b A + c A A,  X <- a X + B X,
// which maps every singular value s of X to a s + b s^3 + c s^5 and leaves
// the singular vectors; out = scale X.
//
// The products run on the matrix cores in fp16 with fp32 accumulation. What
// keeps that rounding below the result's own, bf16's, on common spectra:
//   * X itself stays in fp32 and enters as (a + B_ii) X_ij in the epilogue;
//     only the products read an fp16 copy;
//   * the diagonals of A and B, where most of their weight is, stay in fp32
//     vectors: A = D + O and B = E + F with O, F of zero diagonal,
//       F_ij = (b + c (D_i + D_j)) O_ij + c (O O)_ij           (i != j)
//       E_i  = b D_i + c ((O O)_ii + D_i^2);
//   * fixed powers of two place the fp16 copies: X 2^10, O 2^12, F 2^9, far
//     from overflow for every iterate the entry point admits (singular values
//     at most 3, |b s^2 + c s^4| at most 100); values below 2^-24, 2^-26 and
//     2^-23 become subnormals, in steps of 2^-34, 2^-36 and 2^-33.
// bf16 operands, the usual choice, would be eight times coarser.
//
// Rounding that falls on directions G nearly lacks grows with them, up to |a|
// times a step. Where a call's polynomial and steps let it grow past the
// result's own rounding (ortho_split), the leading steps take every operand as
// two fp16 halves, about 22 bits, and three products for one: hi hi, hi lo and
// lo hi, as one K three times as long. Relative 2-norm before the result's
// rounding, half the directions 1e-3 of the others, 256 x 1024: 5 steps 2.9e-3
// in plain fp16; 8 steps 3.3e-2, with leading halves 1e-3. Such a step takes
// about 2.6 times as long (ten of five 2560 x 1280: 2800 to 2820 us, 1320 in
// plain fp16). The halves need no memory of their own: they lie where nothing else
// lives at the time.
//
// A and B are symmetric: only tiles on and below the diagonal are computed,
// the others are their mirror images. The products run as tiles of P Q^T with
// both operands K-contiguous: A = Xh Xh^T, O O^T, and F Yh^T with Yh the
// transpose of Xh, which the update writes beside it.
//
// The tile kernel: K advances 64 at a time through an LDS ring filled by
// direct global-to-LDS loads, rows swizzled so that fragment reads meet no
// bank conflicts; v_mfma_f32_32x32x16_f16, with the Q fragment as its A
// operand, so a lane's accumulators are runs of four consecutive columns of
// one row. The epilogue passes each 32 x 32 block through a patch of LDS that
// is the wave's own, so that rows and, for the mirrored and transposed copies,
// columns leave in whole runs: stores straight from the accumulators, 16 to
// 32 bytes a row, took up to 3.4 of a small product's 9 us.
//
// Matrices of up to 64 x 256 take one launch instead of 3 steps + 2: a block
// holds its matrix in LDS through all steps. There the operands are split
// into two fp16 values each (22 bits; three products for one), for with few
// columns less averages out and the products cost next to nothing.
#include <type_traits>

#include "train.h"

namespace pg {
namespace {

constexpr int kThreads = 256;
constexpr int kPad = 128;                 // padded sides are multiples of this
constexpr int kNormBlocks = 256;           // most partial sums of a matrix's norm
constexpr float kSX = 1024.f, kSO = 4096.f, kSF = 512.f;   // fp16 placements

template <int V>
using IC = std::integral_constant<int, V>;

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float g_at(const float* G, int64_t i) { return G[i]; }
__device__ __forceinline__ float g_at(const uint16_t* G, int64_t i) { return bf16_to_f32(G[i]); }

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
         ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16);
}
__device__ __forceinline__ float low_part(float x) { return x - (float)(_Float16)x; }
__device__ __forceinline__ float half_at(uint2 v, int u) {   // u-th of four packed halves
  const uint32_t bits = ((u & 2) ? v.y : v.x) >> (16 * (u & 1));
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Sum over the block in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double s, double* sh) {
  sh[threadIdx.x] = s;
  __syncthreads();
#pragma unroll
  for (int o = kThreads / 2; o >= 1; o >>= 1) {
    if ((int)threadIdx.x < o) sh[threadIdx.x] += sh[threadIdx.x + o];
    __syncthreads();
  }
  return sh[0];
}

// Sum of squares of matrix blockIdx.y in double (no overflow for any fp32
// input), one partial per block.
template <typename T>
__global__ __launch_bounds__(kThreads) void ns_norm_kernel(const T* __restrict__ G, int64_t count,
                                                           double* __restrict__ part) {
  __shared__ double sh[kThreads];
  const T* g = G + (int64_t)blockIdx.y * count;
  double s = 0.0;
  const int64_t step = (int64_t)gridDim.x * kThreads * 8;
#pragma unroll 4
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8; i < count; i += step) {
    const Raw8<T> x = load8(g + i, (int)(count - i < 8 ? count - i : 8));
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const double v = (double)x.get(u);
      s += v * v;
    }
  }
  s = block_sum(s, sh);
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// X, its fp16 copy and the copy's transpose from G, 64 x 64 tiles of X with
// zeros in the padding.
template <typename T>
__global__ __launch_bounds__(kThreads) void ns_load_kernel(
    const T* __restrict__ G, int rows, int cols, const double* __restrict__ part, int parts,
    float eps, int mp, int np, float* __restrict__ X, _Float16* __restrict__ Xh,
    _Float16* __restrict__ Yh) {
  __shared__ float t[64][65];
  __shared__ double sh[kThreads];
  const int64_t mat = blockIdx.z;
  const T* g = G + mat * rows * cols;
  const bool tall = rows > cols;                 // X = G^T
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;     // tile of X
  const int g0 = tall ? j0 : i0, h0 = tall ? i0 : j0;       // the same tile of G
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  float v[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int r = g0 + ty + 4 * q, c = h0 + tx;
    v[q] = r < rows && c < cols ? g_at(g, (int64_t)r * cols + c) : 0.f;
  }
  const double s = block_sum((int)threadIdx.x < parts ? part[mat * parts + threadIdx.x] : 0.0, sh);
  // 1 / (norm + eps) as f 2^e: it may lie outside fp32's range, the products
  // with G's values do not; fp64 products took 9 us of 54 at 5 x 2560 x 1280
  int e = 0;
  const float f = (float)frexp(s == 0.0 ? 0.0 : 1.0 / (sqrt(s) + (double)eps), &e);
#pragma unroll
  for (int q = 0; q < 16; ++q) t[ty + 4 * q][tx] = ldexpf(v[q], e) * f;
  __syncthreads();
  // 16 threads a row of the tile, four columns each, four rows a thread
  const int64_t base = mat * mp * np;
  const int c = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int a = (threadIdx.x >> 4) + 16 * q;
    float x[4], y[4];                            // X[i0 + a][j0 + c ..], X[i0 + c ..][j0 + a]
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      x[u] = tall ? t[c + u][a] : t[a][c + u];
      y[u] = tall ? t[a][c + u] : t[c + u][a];
    }
    const int64_t at = base + (int64_t)(i0 + a) * np + j0 + c;
    *reinterpret_cast<float4*>(X + at) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint2*>(Xh + at) =
        make_uint2(pack_half(x[0] * kSX, x[1] * kSX), pack_half(x[2] * kSX, x[3] * kSX));
    *reinterpret_cast<uint2*>(Yh + base + (int64_t)(j0 + a) * mp + i0 + c) =
        make_uint2(pack_half(y[0] * kSX, y[1] * kSX), pack_half(y[2] * kSX, y[3] * kSX));
  }
}

// The scaled fp16 copies of X as two halves (lo nullable), TRANSPOSED: of its
// transpose; 64 x 64 tiles. Bound by memory: five 2560 x 1280 20 us (6.4 TB/s).
template <bool TRANSPOSED>
__global__ __launch_bounds__(kThreads) void ns_copy_kernel(const float* __restrict__ X, int mp,
                                                           int np, _Float16* __restrict__ hi,
                                                           _Float16* __restrict__ lo) {
  __shared__ float t[64][65];
  const int64_t base = (int64_t)blockIdx.z * mp * np;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  const int c = (threadIdx.x & 15) * 4, a0 = threadIdx.x >> 4;
  auto put = [&](int64_t at, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(hi + at) = make_uint2(pack_half(f[0], f[1]), pack_half(f[2], f[3]));
    if (lo)
      *reinterpret_cast<uint2*>(lo + at) =
          make_uint2(pack_half(low_part(f[0]), low_part(f[1])),
                     pack_half(low_part(f[2]), low_part(f[3])));
  };
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int a = a0 + 16 * q;
    const int64_t at = base + (int64_t)(i0 + a) * np + j0 + c;
    const float4 x = *reinterpret_cast<const float4*>(X + at);
    const float f[4] = {x.x * kSX, x.y * kSX, x.z * kSX, x.w * kSX};
    if constexpr (TRANSPOSED) {
#pragma unroll
      for (int u = 0; u < 4; ++u) t[a][c + u] = f[u];
    } else {
      put(at, f);
    }
  }
  if constexpr (TRANSPOSED) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int a = a0 + 16 * q;
      const float f[4] = {t[c][a], t[c + 1][a], t[c + 2][a], t[c + 3][a]};
      put(base + (int64_t)(j0 + a) * mp + i0 + c, f);
    }
  }
}

enum { NS_GRAM, NS_POLY, NS_UPDATE };

struct NsArgs {
  const _Float16* P;      // left operand rows, K contiguous
  const _Float16* Q;      // right operand rows, K contiguous
  int K, mp, np;
  int tiles;              // tiles of one matrix
  int cols_t;             // update: tiles along a row
  float a, b, c, scale;
  float* X;               // fp32 iterate [mp][np]
  _Float16 *Xh, *Yh;      // next copies (update)
  _Float16* O;            // A without its diagonal
  float* D;
  _Float16* F;            // B without its diagonal
  float* E;
  uint16_t* out;          // last update: the result, rows x cols
  int rows, cols;
  int64_t plo, qlo;       // split: bytes from the operands to their low halves
  _Float16 *Ol, *Fl;      // split: low halves of O and F
};

typedef __attribute__((address_space(3))) void lds_void_t;

// s_waitcnt with only a vmcnt limit (vmcnt[3:0], expcnt[6:4], lgkmcnt[11:8],
// vmcnt[5:4] in bits [15:14]).
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// Direct global-to-LDS load: each lane moves 16 bytes from base + off; the
// wave writes 1 KiB at LDS address lds + 16 lane. No memory clobber: the ring
// orders it with counted waits and barriers. s_nop: a load that reads M0 needs
// a wait state behind the write of M0, which the compiler, seeing no load in
// the asm, does not add.
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(lds));
}

__device__ __forceinline__ void ring_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// BM x BN tile of P Q^T by KS groups of WM x WN waves; S stages in the ring, a
// stage being 64 of K for each group. Two groups halve the chain of stages of
// a small product, whose time is latency; their sums are joined at the end.
// SPLIT: operands of two halves, K walked three times; the update then writes
// X alone, whose copies ns_copy_kernel makes. Five 2560 x 1280: Gram 107
// us, polynomial 63, update 123; unsplit 38, 26 and 67.
template <int MODE, int BM, int BN, int WM, int WN, int S, int KS, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN * KS) void ns_tile_kernel(NsArgs g) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN;          // a wave's part
  constexpr int FM = TM / 32, FN = TN / 32;
  constexpr int PL = BM / 8 / NW, QL = BN / 8 / NW;  // loads of 8 rows a wave and stage
  constexpr int L = PL + QL;
  constexpr int kStage = (BM + BN) * 128;
  static_assert(PL >= 1 && QL >= 1 && TM % 32 == 0 && TN % 32 == 0 && (S - 1) * L < 64, "tile");
  static_assert(MODE == NS_UPDATE || (BM == BN && TM * TN <= 4096), "mirrored tiles");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[S * KS * kStage];

  // consecutive tiles run on one of the 8 XCDs and share operands in its L2
  const int64_t total = gridDim.x, per = total / 8;
  int64_t id = blockIdx.x;
  if (id < per * 8) id = (id & 7) * per + (id >> 3);
  const int64_t mat = id / g.tiles;
  const int t = (int)(id - mat * g.tiles);
  int bi, bj;
  if constexpr (MODE == NS_UPDATE) {
    bi = t / g.cols_t;
    bj = t - bi * g.cols_t;
  } else {                                           // t = bi (bi + 1) / 2 + bj, bj <= bi
    bi = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while (bi * (bi + 1) / 2 > t) --bi;
    while ((bi + 1) * (bi + 2) / 2 <= t) ++bi;
    bj = t - bi * (bi + 1) / 2;
  }
  const int i0 = bi * BM, j0 = bj * BN;
  const int64_t mm = mat * g.mp * g.mp, mn = mat * g.mp * g.np;
  const int64_t K = g.K;
  const auto* P = reinterpret_cast<const uint8_t*>(g.P + (MODE == NS_GRAM ? mn : mm) + i0 * K);
  const auto* Q = reinterpret_cast<const uint8_t*>(g.Q + (MODE == NS_POLY ? mm : mn) + j0 * K);

  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int ks = all / NW, wave = all % NW;
  const int wm = wave / WN, wn = wave % WN;
  const int fr = lane & 31;

  // A stage's row is 128 bytes, eight 16-byte chunks, chunk c at position
  // c ^ ((row / 2) % 8): the 16 lanes a 16-byte read serves together then
  // touch 16 different slots of a 256-byte line. A load covers 8 rows.
  const int dr = lane >> 3;
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ (dr >> 1)) * 16);
  const uint32_t ring0 = (uint32_t)(uintptr_t)(const lds_void_t*)ring;
  const int K1 = (int)(K / (64 * KS));               // stages of one walk of K
  auto issue = [&](int kt) {
    const uint32_t at = ring0 + ((kt % S) * KS + ks) * kStage;
    const uint8_t *pb = P, *qb = Q;
    int kw = kt;
    if constexpr (SPLIT) {
      if (kt >= 2 * K1) {
        kw -= 2 * K1;
        pb += g.plo;
      } else if (kt >= K1) {
        kw -= K1;
        qb += g.qlo;
      }
    }
    const int64_t k0 = (int64_t)(kw * KS + ks) * 64;
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      const int grp = wave * PL + q;
      load_to_lds(pb + (grp * 8 * K + k0) * 2,
                  (uint32_t)(dr * K * 2) + (chunk ^ (uint32_t)((grp & 1) * 64)), at + grp * 1024);
    }
#pragma unroll
    for (int q = 0; q < QL; ++q) {
      const int grp = wave * QL + q;
      load_to_lds(qb + (grp * 8 * K + k0) * 2,
                  (uint32_t)(dr * K * 2) + (chunk ^ (uint32_t)((grp & 1) * 64)),
                  at + BM * 128 + grp * 1024);
    }
  };
  auto frags = [&](int kt, int st, f16x8_t (&pf)[FM], f16x8_t (&qf)[FN]) {
    const uint8_t* sp = ring + ((kt % S) * KS + ks) * kStage;
    const uint8_t* sq = sp + BM * 128;
    const int c = ((st * 2 + (lane >> 5)) ^ ((fr >> 1) & 7)) * 16;
#pragma unroll
    for (int a = 0; a < FM; ++a)
      pf[a] = *reinterpret_cast<const f16x8_t*>(sp + (wm * TM + a * 32 + fr) * 128 + c);
#pragma unroll
    for (int b = 0; b < FN; ++b)
      qf[b] = *reinterpret_cast<const f16x8_t*>(sq + (wn * TN + b * 32 + fr) * 128 + c);
  };

  // In the epilogue a lane has, of each 32 x 32 block, rows er + 8 p and
  // columns ec .. ec + 3: eight lanes a row. What it reads there is fetched
  // before the first stage, where the registers hold it (PRE), otherwise one
  // block ahead: a load behind stores waits for them.
  const int er = lane >> 3, ec = (lane & 7) * 4;
  constexpr bool PRE = FM * FN <= 4;
  uint2 oin[MODE == NS_POLY ? FM : 1][MODE == NS_POLY ? FN : 1][4];
  uint2 olin[MODE == NS_POLY && SPLIT ? FM : 1][MODE == NS_POLY && SPLIT ? FN : 1][4];
  float4 xin[MODE == NS_UPDATE ? (PRE ? FM * FN : 2) : 1][4];
  float4 djin[FN];
  float din[FM][4];
  auto fetch_x = [&](int t) {
    if constexpr (MODE == NS_UPDATE) {
      const int i = i0 + wm * TM + t / FN * 32 + er, j = j0 + wn * TN + t % FN * 32 + ec;
#pragma unroll
      for (int p = 0; p < 4; ++p)
        xin[PRE ? t : t & 1][p] =
            *reinterpret_cast<const float4*>(g.X + mn + (int64_t)(i + 8 * p) * g.np + j);
    }
  };
  if (ks == 0) {
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i = i0 + wm * TM + a * 32 + er + 8 * p;
        if constexpr (MODE == NS_POLY) din[a][p] = g.D[mat * g.mp + i];
        if constexpr (MODE == NS_UPDATE) din[a][p] = g.a + g.E[mat * g.mp + i];
        if constexpr (MODE == NS_POLY)
#pragma unroll
          for (int b = 0; b < FN; ++b) {
            const int j = j0 + wn * TN + b * 32 + ec;
            oin[a][b][p] = *reinterpret_cast<const uint2*>(g.O + mm + (int64_t)i * g.mp + j);
            if constexpr (SPLIT)
              olin[a][b][p] = *reinterpret_cast<const uint2*>(g.Ol + mm + (int64_t)i * g.mp + j);
            if (a == 0 && p == 0)
              djin[b] = *reinterpret_cast<const float4*>(g.D + mat * g.mp + j);
          }
      }
#pragma unroll
    for (int t = 0; t < (PRE ? FM * FN : 1); ++t) fetch_x(t);
  }

  // one tile a wave: two accumulators in turn, so products need not wait
  constexpr int AC = FM * FN == 1 ? 2 : 1;
  f32x16_t sums[AC][FM][FN] = {};
  auto& acc = sums[0];
  const int KT = SPLIT ? 3 * K1 : K1;
  constexpr int PD = S - 1;                          // stages in flight
#pragma unroll
  for (int st = 0; st < PD; ++st)
    if (st < KT) issue(st);
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt has landed when at most the later issued ones are outstanding;
    // behind the barrier every wave is done with stage kt - 1, whose place
    // stage kt + PD takes
    if (KT - 1 - kt >= PD - 1) wait_loads<(PD - 1) * L>();
    else wait_loads<0>();                            // the last stages: all of them
    ring_barrier();
    if (kt + PD < KT) issue(kt + PD);
    f16x8_t pf[2][FM], qf[2][FN];
    frags(kt, 0, pf[0], qf[0]);
    // the reads of step st + 1 go out between the products of step st
    constexpr int RD = FM + FN, MF = FM * FN, RPM = (RD + MF - 1) / MF;
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      if (st < 3) frags(kt, st + 1, pf[(st + 1) & 1], qf[(st + 1) & 1]);
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
          sums[st % AC][a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
              qf[st & 1][b], pf[st & 1][a], sums[st % AC][a][b], 0, 0, 0);
      if (st == 0) __builtin_amdgcn_sched_group_barrier(0x100, RD, 0);
      if (st < 3) {
        constexpr int FULL = RD / RPM, REM = RD - FULL * RPM;
#pragma unroll
        for (int q = 0; q < FULL; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // one product
          __builtin_amdgcn_sched_group_barrier(0x100, RPM, 0);   // RPM reads
        }
        if constexpr (REM > 0) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, REM, 0);
        }
        constexpr int REST = MF - FULL - (REM > 0 ? 1 : 0);
        if constexpr (REST > 0) __builtin_amdgcn_sched_group_barrier(0x008, REST, 0);
      } else {
        __builtin_amdgcn_sched_group_barrier(0x008, MF, 0);
      }
    }
  }

  if constexpr (AC == 2)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[0][0][q] += sums[1][0][0][q];
  __syncthreads();                                   // the ring is read; now it is scratch
  constexpr int kLd = 36;                            // floats of a patch row: no bank conflicts
  float* patch = reinterpret_cast<float*>(ring) + wave * 32 * kLd;
  if constexpr (KS == 2) {                           // the second group's sums, by way of LDS
    static_assert(FM * FN == 1 && NW * (32 * kLd + 1024) * 4 <= S * KS * kStage, "join");
    float* j = reinterpret_cast<float*>(ring) + NW * 32 * kLd + wave * 1024 + lane;
    if (ks == 1)
#pragma unroll
      for (int q = 0; q < 16; ++q) j[64 * q] = acc[0][0][q];
    __syncthreads();
    if (ks == 1) return;
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[0][0][q] += j[64 * q];
  }

  // Epilogue, one 32 x 32 block after the other.
  const int half = lane >> 5;
  const bool tall = g.rows > g.cols;
  auto halves = [](const float (&f)[4]) {
    return make_uint2(pack_half(f[0], f[1]), pack_half(f[2], f[3]));
  };
  auto lows = [](const float (&f)[4]) {
    return make_uint2(pack_half(low_part(f[0]), low_part(f[1])),
                      pack_half(low_part(f[2]), low_part(f[3])));
  };
  // four of the result's values from column c of row r on, inside its edges
  auto put_out = [&](int r, int c, const float (&f)[4]) {
    if (r >= g.rows) return;
    const uint2 v = make_uint2(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]));
    uint16_t* dst = g.out + mat * g.rows * g.cols + (int64_t)r * g.cols + c;
    if (c + 4 <= g.cols) {
      __builtin_memcpy(dst, &v, 8);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + u < g.cols) dst[u] = (uint16_t)(((u & 2) ? v.y : v.x) >> (16 * (u & 1)));
    }
  };
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      const int t = a * FN + b;
      const int ib = i0 + wm * TM + a * 32, jb = j0 + wn * TN + b * 32;
      if (!PRE && t + 1 < FM * FN) fetch_x(t + 1);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(patch + fr * kLd + 8 * q + 4 * half) =
            make_float4(acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2],
                        acc[a][b][4 * q + 3]);
      wave_sync();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i = ib + er + 8 * p, j = jb + ec;
        float4* slot = reinterpret_cast<float4*>(patch + (er + 8 * p) * kLd + ec);
        const float4 s4 = *slot;
        const float v[4] = {s4.x, s4.y, s4.z, s4.w};
        float f[4];
        if constexpr (MODE == NS_GRAM) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            f[u] = v[u] * (kSO / (kSX * kSX));
            if (ib == jb && i == j + u) {            // the diagonal
              g.D[mat * g.mp + i] = v[u] * (1.f / (kSX * kSX));
              f[u] = 0.f;
            }
          }
          *reinterpret_cast<uint2*>(g.O + mm + (int64_t)i * g.mp + j) = halves(f);
          if constexpr (SPLIT)
            *reinterpret_cast<uint2*>(g.Ol + mm + (int64_t)i * g.mp + j) = lows(f);
        } else if constexpr (MODE == NS_POLY) {
          const float di = din[a][p];
          const float dj[4] = {djin[b].x, djin[b].y, djin[b].z, djin[b].w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float o = half_at(oin[a][b][p], u);
            if constexpr (SPLIT) o += half_at(olin[a][b][p], u);
            o *= 1.f / kSO;
            const float aa = v[u] * (1.f / (kSO * kSO));
            f[u] = ((g.b + g.c * (di + dj[u])) * o + g.c * aa) * kSF;
            if (ib == jb && i == j + u) {
              g.E[mat * g.mp + i] = g.b * di + g.c * (aa + di * di);
              f[u] = 0.f;
            }
          }
          *reinterpret_cast<uint2*>(g.F + mm + (int64_t)i * g.mp + j) = halves(f);
          if constexpr (SPLIT)
            *reinterpret_cast<uint2*>(g.Fl + mm + (int64_t)i * g.mp + j) = lows(f);
        } else {
          const float4 x = xin[PRE ? t : t & 1][p];
          const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) f[u] = din[a][p] * xs[u] + v[u] * (1.f / (kSF * kSX));
          if (g.out) {                               // the result, no more copies
#pragma unroll
            for (int u = 0; u < 4; ++u) f[u] *= g.scale;
            if (!tall) put_out(i, j, f);
          } else {
            *reinterpret_cast<float4*>(g.X + mn + (int64_t)i * g.np + j) =
                make_float4(f[0], f[1], f[2], f[3]);
            if constexpr (!SPLIT) {
#pragma unroll
              for (int u = 0; u < 4; ++u) f[u] *= kSX;
              *reinterpret_cast<uint2*>(g.Xh + mn + (int64_t)i * g.np + j) = halves(f);
            }
          }
        }
        *slot = make_float4(f[0], f[1], f[2], f[3]);
      }
      wave_sync();
      // columns: the mirrored block, the transpose, or a tall matrix's result
      const bool cols = MODE == NS_UPDATE ? (g.out ? tall : !SPLIT) : bi != bj;
      if (cols) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int j = jb + er + 8 * p, i = ib + ec;
          float f[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) f[u] = patch[(ec + u) * kLd + er + 8 * p];
          if constexpr (MODE == NS_UPDATE) {
            if (g.out)
              put_out(j, i, f);
            else
              *reinterpret_cast<uint2*>(g.Yh + mn + (int64_t)j * g.mp + i) = halves(f);
          } else {
            _Float16* m = (MODE == NS_GRAM ? g.O : g.F) + mm;
            *reinterpret_cast<uint2*>(m + (int64_t)j * g.mp + i) = halves(f);
            if constexpr (SPLIT) {
              _Float16* l = (MODE == NS_GRAM ? g.Ol : g.Fl) + mm;
              *reinterpret_cast<uint2*>(l + (int64_t)j * g.mp + i) = lows(f);
            }
          }
        }
      }
      wave_sync();
    }
}

// ---------------------------------------------------------------------------
// Small matrices: one block each

constexpr int kSmallM = 64, kSmallN = 256, kSmallThreads = 512;

struct Split {
  _Float16 hi, lo;
};
__device__ __forceinline__ Split split_half(float x) {
  const _Float16 h = (_Float16)x;
  return {h, (_Float16)(x - (float)h)};
}

typedef float f32x4s_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));

// X is 64 x 32 NT with zeros in the padding. v_mfma_f32_16x16x32_f16: lane l
// holds row l % 16, K elements 8 (l / 16) .. + 7 of each operand, and of the
// result rows 4 (l / 16) + 0..3 (left operand), column l % 16 (right). Wave w
// owns tiles (w / 2, 2 (w % 2) + 0..1) of A and B, whose fp32 A it keeps, and
// tiles (w % 4, w / 4 + 2 t) of X, whose fp32 values it keeps throughout. A
// and B are symmetric, so a lane's four rows of one column are written as
// four columns of one row.
template <typename T, int NT>
__global__ __launch_bounds__(kSmallThreads) void ns_small_kernel(
    const T* __restrict__ G, int rows, int cols, OrthoArgs oa, uint16_t* __restrict__ out) {
  constexpr int NP = 32 * NT;
  constexpr int LX = NP + 8, LM = kSmallM + 8;       // padded rows: no bank conflicts
  __shared__ __attribute__((aligned(16))) _Float16 x_hi[kSmallM * LX], x_lo[kSmallM * LX];
  __shared__ __attribute__((aligned(16))) _Float16 y_hi[NP * LM], y_lo[NP * LM];
  __shared__ __attribute__((aligned(16))) _Float16 s_hi[kSmallM * LM], s_lo[kSmallM * LM];
  __shared__ double red[kSmallThreads / 64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int l16 = lane & 15, l4 = lane >> 4;
  const bool tall = rows > cols;
  const T* g = G + (int64_t)blockIdx.x * rows * cols;
  uint16_t* o = out + (int64_t)blockIdx.x * rows * cols;
  const int m = tall ? cols : rows, n = tall ? rows : cols;
  const int xi = (wave & 3) * 16 + 4 * l4;           // first of the lane's rows of X
  auto xj = [&](int t) { return ((wave >> 2) + 2 * t) * 16 + l16; };
  auto at = [&](int i, int j) { return tall ? (int64_t)j * cols + i : (int64_t)i * cols + j; };

  float x[NT][4];
  double ss = 0.0;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[t][q] = xi + q < m && xj(t) < n ? g_at(g, at(xi + q, xj(t))) : 0.f;
      ss += (double)x[t][q] * (double)x[t][q];
    }
#pragma unroll
  for (int w = 32; w >= 1; w >>= 1) ss += __shfl_xor(ss, w, 64);
  if (lane == 0) red[wave] = ss;
  __syncthreads();
  ss = 0.0;
#pragma unroll
  for (int w = 0; w < kSmallThreads / 64; ++w) ss += red[w];
  int e = 0;                                         // 1 / (norm + eps) = f 2^e
  const float f = (float)frexp(ss == 0.0 ? 0.0 : 1.0 / (sqrt(ss) + (double)oa.eps), &e);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) x[t][q] = ldexpf(x[t][q], e) * f;

  // four values of one column of a tile into row `r` of a symmetric or
  // transposed matrix
  auto put4 = [&](_Float16* hi, _Float16* lo, int r, int c, const float (&v)[4], float f) {
    f16x4_t h, l;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const Split s = split_half(v[q] * f);
      h[q] = s.hi;
      l[q] = s.lo;
    }
    *reinterpret_cast<f16x4_t*>(hi + r * LM + c) = h;
    *reinterpret_cast<f16x4_t*>(lo + r * LM + c) = l;
  };
  auto put_x = [&] {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      put4(y_hi, y_lo, xj(t), xi, x[t], kSX);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const Split s = split_half(x[t][q] * kSX);
        x_hi[(xi + q) * LX + xj(t)] = s.hi;
        x_lo[(xi + q) * LX + xj(t)] = s.lo;
      }
    }
  };
  // rows p of one split matrix times rows q of another, K elements each
  auto product = [&](const _Float16* ph, const _Float16* pl, int pld, int p, const _Float16* qh,
                     const _Float16* ql, int qld, int q, auto K) {
    f32x4s_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k0 = 0; k0 < K(); k0 += 32) {
      const int k = k0 + 8 * l4;
      const f16x8_t ah = *reinterpret_cast<const f16x8_t*>(ph + (p + l16) * pld + k);
      const f16x8_t al = *reinterpret_cast<const f16x8_t*>(pl + (p + l16) * pld + k);
      const f16x8_t bh = *reinterpret_cast<const f16x8_t*>(qh + (q + l16) * qld + k);
      const f16x8_t bl = *reinterpret_cast<const f16x8_t*>(ql + (q + l16) * qld + k);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah, bh, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah, bl, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(al, bh, acc, 0, 0, 0);
    }
    return acc;
  };
  const int ai = (wave >> 1) * 16;
  auto aj = [&](int t) { return (2 * (wave & 1) + t) * 16; };

  put_x();
  __syncthreads();
  for (int step = 0; step < oa.steps; ++step) {
    float A[2][4], B[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {                    // A = X X^T
      const f32x4s_t acc = product(x_hi, x_lo, LX, ai, x_hi, x_lo, LX, aj(t), IC<NP>{});
#pragma unroll
      for (int q = 0; q < 4; ++q) A[t][q] = acc[q] * (1.f / (kSX * kSX));
      put4(s_hi, s_lo, aj(t) + l16, ai + 4 * l4, A[t], kSO);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {                    // B = b A + c A A
      const f32x4s_t acc = product(s_hi, s_lo, LM, ai, s_hi, s_lo, LM, aj(t), IC<kSmallM>{});
#pragma unroll
      for (int q = 0; q < 4; ++q) B[t][q] = oa.b * A[t][q] + oa.c * (acc[q] * (1.f / (kSO * kSO)));
    }
    __syncthreads();                                 // A is read; B takes its place
#pragma unroll
    for (int t = 0; t < 2; ++t) put4(s_hi, s_lo, aj(t) + l16, ai + 4 * l4, B[t], kSF);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {                   // X <- a X + B X
      const f32x4s_t acc = product(s_hi, s_lo, LM, (wave & 3) * 16, y_hi, y_lo, LM,
                                   ((wave >> 2) + 2 * t) * 16, IC<kSmallM>{});
#pragma unroll
      for (int q = 0; q < 4; ++q) x[t][q] = oa.a * x[t][q] + acc[q] * (1.f / (kSF * kSX));
    }
    if (step + 1 == oa.steps) break;
    __syncthreads();                                 // X's copies are read
    put_x();
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (xi + q < m && xj(t) < n)
        o[at(xi + q, xj(t))] = (uint16_t)pack2_bf16(oa.scale * x[t][q], 0.f);
}

int64_t al(int64_t x) { return (x + 255) / 256 * 256; }


}  // namespace

OrthoPlan ortho_plan(int64_t n_mat, int64_t rows, int64_t cols) {
  OrthoPlan p{};
  p.m = (int)(rows < cols ? rows : cols);
  p.n = (int)(rows < cols ? cols : rows);
  p.small = p.m <= kSmallM && p.n <= kSmallN;
  if (p.small) {
    p.bytes = 256;                                   // not used; a size of its own all the same
    return p;
  }
  p.mp = (p.m + kPad - 1) / kPad * kPad;
  p.np = (p.n + kPad - 1) / kPad * kPad;
  const int64_t need = (rows * cols + kThreads * 32 - 1) / (kThreads * 32);
  p.norm_blocks = (int)(need < kNormBlocks ? need : kNormBlocks);
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
  if (p.small) {
    auto small = [&](auto* g, auto NT) {
      hipLaunchKernelGGL((ns_small_kernel<std::remove_const_t<std::remove_pointer_t<decltype(g)>>, NT()>),
                         dim3((unsigned)n_mat), dim3(kSmallThreads), 0, s, g, rows, cols, oa, out);
    };
    auto by_width = [&](auto* g) {
      if (p.n <= 64) small(g, IC<2>{});
      else if (p.n <= 128) small(g, IC<4>{});
      else small(g, IC<8>{});
    };
    if (dtype == PG_F32) by_width(static_cast<const float*>(G));
    else by_width(static_cast<const uint16_t*>(G));
    return hipGetLastError();
  }
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
  // The tile of a product: the largest that leaves a chip of 256 compute units
  // work for most of them. Larger tiles read operands less often, smaller ones
  // start more work at once. Measured, us of a whole call with and without:
  // 256 x 256 updates at 256 blocks (4096 x 4096) 1853 and 1988, at 100 (two
  // 2560 x 1280) 405 and 340; 128 x 128 at 136 blocks (2048 x 2048) 408 and
  // 429, at 128 (32 of 256 x 256) 125 and 111. Up to 256 blocks of 64 x 64 two
  // groups of waves share a tile's K (768 x 1024: 121 and 131); beyond, two
  // blocks share a compute unit instead (32 of 256 x 256: 111 and 138).
  // Products of halves follow the same rule (ten steps of five 2560 x 1280 2824
  // us, 2990 without 256 x 256; of 32 of 256 x 256 399 us, 441 without four
  // stages).
  auto launch = [&](auto MODE, auto SPLIT, const NsArgs& args) {
    constexpr bool UPDATE = MODE() == NS_UPDATE;
    NsArgs g = args;
    auto blocks = [&](int B) {
      const int64_t ti = p.mp / B;
      return n_mat * (UPDATE ? ti * (p.np / B) : ti * (ti + 1) / 2);
    };
    auto go = [&](auto B, auto WM, auto WN, auto S, auto KS) {
      g.cols_t = p.np / B();
      g.tiles = (int)(blocks(B()) / n_mat);
      hipLaunchKernelGGL((ns_tile_kernel<MODE(), B(), B(), WM(), WN(), S(), KS(), SPLIT()>),
                         dim3((unsigned)blocks(B())), dim3(64 * WM() * WN() * KS()), 0, s, g);
    };
    if constexpr (UPDATE)
      if (p.mp % 256 == 0 && p.np % 256 == 0 && blocks(256) >= 200)
        return go(IC<256>{}, IC<2>{}, IC<4>{}, IC<2>{}, IC<1>{});
    if (blocks(128) > 128) return go(IC<128>{}, IC<2>{}, IC<2>{}, IC<2>{}, IC<1>{});
    if (blocks(64) > 256) return go(IC<64>{}, IC<2>{}, IC<2>{}, IC<4>{}, IC<1>{});
    go(IC<64>{}, IC<2>{}, IC<2>{}, IC<3>{}, IC<2>{});
  };
  auto copies = [&](auto TRANSPOSED, _Float16* hi, _Float16* lo) {
    hipLaunchKernelGGL(ns_copy_kernel<TRANSPOSED()>, lgrid, block, 0, s, X, p.mp, p.np, hi, lo);
  };
  const auto bytes = [](const _Float16* to, const _Float16* from) {
    return (int64_t)(reinterpret_cast<const uint8_t*>(to) - reinterpret_cast<const uint8_t*>(from));
  };
  for (int k = 0; k < oa.steps; ++k) {
    NsArgs g{};
    g.mp = p.mp; g.np = p.np;
    g.a = oa.a; g.b = oa.b; g.c = oa.c; g.scale = oa.scale;
    g.X = X; g.Xh = Xh; g.O = O; g.D = D; g.F = F; g.E = E;
    g.rows = rows; g.cols = cols;
    g.out = k + 1 == oa.steps ? out : nullptr;
    if (k < oa.split) {
      // The low halves lie, of X in the first transpose (free until the
      // update), of O in the second (as long), of F in X's copy (read by the
      // Gram product alone), of the transpose in the second again.
      g.Ol = Yh[1]; g.Fl = Xh;
      copies(IC<0>{}, Xh, Yh[0]);
      g.P = Xh; g.Q = Xh; g.K = p.np; g.plo = g.qlo = bytes(Yh[0], Xh);
      launch(IC<NS_GRAM>{}, std::true_type{}, g);
      g.P = O; g.Q = O; g.K = p.mp; g.plo = g.qlo = bytes(g.Ol, O);
      launch(IC<NS_POLY>{}, std::true_type{}, g);
      copies(IC<1>{}, Yh[0], Yh[1]);
      g.P = F; g.Q = Yh[0]; g.plo = bytes(g.Fl, F); g.qlo = bytes(Yh[1], Yh[0]);
      launch(IC<NS_UPDATE>{}, std::true_type{}, g);
      if (k + 1 == oa.split && k + 1 < oa.steps) {   // what the plain steps start from
        copies(IC<0>{}, Xh, nullptr);
        copies(IC<1>{}, Yh[(k + 1) & 1], nullptr);
      }
      continue;
    }
    g.P = Xh; g.Q = Xh; g.K = p.np;
    launch(IC<NS_GRAM>{}, std::false_type{}, g);
    g.P = O; g.Q = O; g.K = p.mp;
    launch(IC<NS_POLY>{}, std::false_type{}, g);
    g.P = F; g.Q = Yh[k & 1]; g.Yh = Yh[(k + 1) & 1];
    launch(IC<NS_UPDATE>{}, std::false_type{}, g);
  }
  return hipGetLastError();
}

}  // namespace pg
