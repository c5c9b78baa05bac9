// The head's logits for few tokens, where reading the table once is what counts.
#pragma once

#include "head_tile.h"

namespace pg {
namespace {

// ---------------------------------------------------------------------------
// Few tokens

// Maxima and sums of few tokens over 128 rows of the table: what counts is
// reading the table once, from where it lies and whatever its width. Blocks of
// up to 64 tokens, those of one tile of the table next to each other. A wave has
// 32 rows to itself and takes the fragments of 16 x 16 x 32 products straight
// from memory, 16 rows by 64 bytes a load, the 512 bytes of a row (fp32 256) one
// behind the other; the next ones are under way while the last are multiplied.
// The tokens' part of a chunk goes through LDS, which the four waves share:
// fetched by every wave for itself it took as many loads as the table. fp32
// operands are split in registers into three bf16 planes (24 bits), six products
// for one, so nothing has to be placed or copied.
//
// 32 tokens, 128,000 rows of 2560, bf16: 118 us, 5.5 TB/s (a bare read of the
// same pattern 107). On the way: fragments of 32 x 32 x 16, 32 bytes a row and
// load, 162 us; tokens fetched by every wave 160; parts of 16 rows in turn
// instead of a row's 138; 256 bytes of a row at a time 125; without the barrier
// it would be 115.
struct FewArgs {
  const void *h, *table;
  int64_t ld, n, V;
  int d, groups;           // of 64 tokens
  float c2;
  float2* part;            // [tiles of 128 rows][n]
};

// dz instead of maxima and sums: rows_pad rows, zeros behind the tokens and
// behind the table.
struct FewDz {
  const float *a, *lse2;
  uint16_t* dz;
  int64_t ldz, plane;      // elements
  int rows_pad;
  int* top;                // fp32: kTops exponents, raised to T's largest element's (nullable)
  // fp16: levels of the columns, and what they need of the sparse positions
  const int32_t* sidx;
  const float* sval;
  int count;
  int64_t v0;              // vocabulary row of column 0
  uint8_t* level;          // [ldz]: all tokens are one group
  int* any;
};
constexpr int kTops = 512;

// Largest finite magnitude of a fragment, and m.
__device__ __forceinline__ float few_top(const Raw8<float>& v, float m) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float a = fabsf(v.v[u]);
    m = a < INFINITY ? fmaxf(m, a) : m;
  }
  return m;
}
// A wave's share of the exponent of T's largest element, whose rows dz reads in
// fp32 in any case (65,536 rows of 2048, 8 tokens: 712 us; a pass of its own took 105
// more).
__device__ __forceinline__ void few_put_top(const FewDz& z, float m) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  // (a maximum: the order of the waves does not matter)
  if (z.top && (threadIdx.x & 63) == 0) atomicMax(z.top + blockIdx.x % kTops, exponent_of(m));
}
// dz of token tok at four columns from their logits in base 2.
__device__ __forceinline__ void few_exp(const FewDz& z, int64_t tok, int64_t n, float (&v)[4]) {
  const float a = tok < n ? z.a[tok] : 0.f, l = tok < n ? z.lse2[tok] : 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = a == 0.f ? 0.f : a * __builtin_amdgcn_exp2f(v[q] - l);
}
// Largest |dz| at the sparse positions of the block's COLS columns from col on, as
// bits. The first ones, all of cross entropy's, are under way from the kernel's start.
struct FewStops {
  int32_t id;
  float val;
  __device__ __forceinline__ void start(const FewDz& z) {
    const int i = threadIdx.x;
    id = i < z.count ? z.sidx[i] : -1;
    val = i < z.count ? z.sval[i] : 0.f;
  }
  template <int COLS>
  __device__ __forceinline__ void join(const FewDz& z, int64_t col, uint32_t* stop) const {
    auto put = [&](int32_t at, float x) {
      const int64_t v = at - z.v0 - col;
      if (v >= 0 && v < COLS) atomicMax(stop + v, __float_as_uint(x) & 0x7FFFFFFFu);
    };
    if (threadIdx.x < COLS) stop[threadIdx.x] = 0;
    __syncthreads();
    put(id, val);
#pragma unroll 4
    for (int i = threadIdx.x + 256; i < z.count; i += 256) put(z.sidx[i], z.sval[i]);
  }
};
// Largest of the 16 lanes' values.
__device__ __forceinline__ uint32_t max_of16(uint32_t x) {
  x = max(x, dpp<0x128>(x));                         // 8 apart
  x = max(x, dpp<0x141>(x));                         // 8 mirrored
  x = max(x, dpp<0x4E>(x));                          // 2 apart
  return max(x, dpp<0xB1>(x));                       // next
}
// Stores it; MODE 1: fp16, two halves (fp32 operands); 2: two bf16 halves.
template <int MODE>
__device__ __forceinline__ void few_dz(const FewDz& z, int64_t tok, int64_t col,
                                       const float (&f)[4]) {
  using H = Half<MODE == 1>;
  const uint2 w = make_uint2(H::pack(f[0], f[1]), H::pack(f[2], f[3]));
  uint16_t* to = z.dz + tok * z.ldz + col;
  *reinterpret_cast<uint2*>(to) = w;
  *reinterpret_cast<uint2*>(to + z.plane) =
      make_uint2(H::pack(f[0] - H::lo(w.x), f[1] - H::hi(w.x)),
                 H::pack(f[2] - H::lo(w.y), f[3] - H::hi(w.y)));
}
// Zeros in dz's rows from `from` on, `cols` (a multiple of 4) from col on; by the block.
__device__ __forceinline__ void few_dz_zero(const FewDz& z, int from, int64_t col, int cols) {
  const int per = cols / 4;
  for (int i = threadIdx.x; i < (z.rows_pad - from) * per; i += 256) {
    uint16_t* to = z.dz + (from + i / per) * z.ldz + col + i % per * 4;
    *reinterpret_cast<uint2*>(to) = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(to + z.plane) = make_uint2(0, 0);
  }
}

// Lifts four columns from col on, their largest |dz| in m as bits of fp32, f(t, q)
// this lane's tokens'.
template <int TB, typename F>
__device__ __forceinline__ void few_lift(const FewDz& z, int64_t col, const uint32_t (&m)[4],
                                         int fr, F f) {
  uint32_t l[4];
  bool lifted = false;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    l[q] = level_of(m[q] >> 16);
    const bool some = l[q] != kFlat && l[q] != kEmpty;
    lifted |= some;
    const float by = __uint_as_float((127u + (some ? l[q] : 0u)) << 23);
#pragma unroll
    for (int t = 0; t < TB; ++t) f(t, q) *= by;
  }
  if (fr == 0) {
    *reinterpret_cast<uint32_t*>(z.level + col) = l[0] | l[1] << 8 | l[2] << 16 | l[3] << 24;
    if (lifted) *z.any = 1;
  }
}

// A fragment of 8 elements as bf16 (fp32: its three planes).
template <typename T>
__device__ __forceinline__ void planes_of(const Raw8<T>& v, uint4 (&f)[sizeof(T) == 4 ? 3 : 1]) {
  if constexpr (sizeof(T) == 4) {
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = v.v[u];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        w[u] = pack2_bf16(x[2 * u], x[2 * u + 1]);
        x[2 * u] -= __uint_as_float(w[u] << 16);
        x[2 * u + 1] -= __uint_as_float(w[u] & 0xFFFF0000u);
      }
      f[p] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    f[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  }
}
// acc += w h of two fragments' planes, small products first.
template <int P>
__device__ __forceinline__ void mma_planes(const uint4 (&w)[P], const uint4 (&h)[P], f32x4_t& acc) {
  auto mma = [&](int a, int b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[a]),
                                                  __builtin_bit_cast(bf16x8_t, h[b]), acc, 0, 0, 0);
  };
  if constexpr (P == 3) {
    mma(2, 0);
    mma(0, 2);
    mma(1, 1);
    mma(1, 0);
    mma(0, 1);
  }
  mma(0, 0);
}

template <typename T, int TB, int DZ>
__global__ __launch_bounds__(256, 2) void head_few_kernel(FewArgs g, FewDz dz) {
  static_assert(DZ == 0 || (DZ == 1) == (sizeof(T) == 4), "dz of fp32 operands is fp16");
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int ST = F32 ? 2 : 8;                    // steps of 32 of K under way
  constexpr int P = F32 ? 3 : 1, KC = 32 * ST;
  constexpr int RB = KC * 2;                         // bytes of a token's row in LDS
  constexpr int CH = 16 * TB * KC / 8;               // its 8-element chunks in all
  constexpr int HL = (CH + 255) / 256;               // of them a thread
  __shared__ __attribute__((aligned(256))) uint8_t hs[2][P][16 * TB * RB];
  __shared__ float2 red[4][16 * TB];
  __shared__ uint32_t stop[DZ == 1 ? 128 : 1];
  FewStops stops;
  if constexpr (DZ == 1) stops.start(dz);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, kq = lane >> 4;
  // a tile's groups run 8 blocks apart: on one XCD, where they share its L2
  const uint32_t id = blockIdx.x;
  const uint32_t grp = g.groups == 1 ? 0 : (id >> 3) % g.groups;
  const uint32_t tile = g.groups == 1 ? id : (id >> 3) / g.groups * 8 + (id & 7);
  if (DZ == 0 && (int64_t)tile * 128 >= g.V) return;
  const int64_t v0 = (int64_t)tile * 128 + wave * 32, x0 = (int64_t)grp * 64;
  const T* wp[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t v = v0 + r * 16 + fr;
    wp[r] = static_cast<const T*>(g.table) + (v < g.V ? v : g.V - 1) * g.d + kq * 8;
  }
  // 16-byte chunk c of token x in LDS: the 16 tokens a read serves together
  // meet every bank once
  auto place = [](int x, int c) {
    static_assert(RB == 512 || RB == 128, "chunks of a row over the banks");
    return RB == 512 ? x * 512 + ((c ^ (x & 15)) * 16) : x * 128 + ((c ^ ((x >> 1) & 7)) * 16);
  };
  const T* hp[HL];
  int hc[HL];
#pragma unroll
  for (int u = 0; u < HL; ++u) {
    const int i = u * 256 + threadIdx.x, x = i / (KC / 8);
    hc[u] = i % (KC / 8) * 8;
    hp[u] = static_cast<const T*>(g.h) + (x0 + x < g.n ? x0 + x : g.n - 1) * g.ld + hc[u];
  }
  f32x4_t acc[TB][2] = {};
  float top = 0.f;
  Raw8<T> hr[HL], wr[2][ST][2];
  auto load = [&](int k, Raw8<T> (&w)[ST][2]) {
    const bool all = k + KC <= g.d;
#pragma unroll
    for (int u = 0; u < HL; ++u)
      if (HL * 256 == CH || u * 256 + (int)threadIdx.x < CH)
        hr[u] = load8(hp[u] + k, all ? 8 : g.d - k - hc[u]);
    // a row's 64-byte parts one behind the other: the other way round it took 12 us more
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int s = 0; s < ST; ++s)
        w[s][r] = load8(wp[r] + k + s * 32, all ? 8 : g.d - k - s * 32 - kq * 8);
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int u = 0; u < HL; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (HL * 256 == CH || i < CH) {
        uint4 f[P];
        planes_of(hr[u], f);
#pragma unroll
        for (int p = 0; p < P; ++p)
          *reinterpret_cast<uint4*>(hs[buf][p] + place(i / (KC / 8), i % (KC / 8))) = f[p];
      }
    }
  };
  auto multiply = [&](int buf, const Raw8<T> (&w)[ST][2]) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      uint4 wf[2][P];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        planes_of(w[s][r], wf[r]);
        if constexpr (F32 && DZ == 1) top = few_top(w[s][r], top);
      }
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        uint4 hf[P];
#pragma unroll
        for (int p = 0; p < P; ++p)
          hf[p] = *reinterpret_cast<const uint4*>(hs[buf][p] + place(t * 16 + fr, s * 4 + kq));
#pragma unroll
        for (int r = 0; r < 2; ++r) mma_planes(wf[r], hf, acc[t][r]);
      }
    }
  };
  // One barrier a chunk: a buffer is written again two chunks on, behind the
  // barrier that every wave reaches with its reads of it done.
  const int chunks = (g.d + KC - 1) / KC;
  int at = (int)(tile % chunks);                     // tiles start apart
  auto chunk = [&](int c, int buf, const Raw8<T> (&w)[ST][2], Raw8<T> (&next)[ST][2]) {
    stage(buf);
    at = at + 1 == chunks ? 0 : at + 1;
    if (c + 1 < chunks) load(at * KC, next);
    wait_lds();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    multiply(buf, w);
  };
  load(at * KC, wr[0]);
  for (int c = 0; c < chunks; c += 2) {
    chunk(c, 0, wr[0], wr[1]);
    if (c + 1 < chunks) chunk(c + 1, 1, wr[1], wr[0]);
  }

  // a lane has rows 16 r + 4 kq + q of the wave's 32, token 16 t + fr
  if constexpr (DZ != 0) {
    float f[TB][2][4];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          f[t][r][q] = v0 + r * 16 + 4 * kq + q < g.V ? acc[t][r][q] * g.c2 : -INFINITY;
        few_exp(dz, t * 16 + fr, g.n, f[t][r]);
      }
    if constexpr (DZ == 1) {
      stops.template join<128>(dz, (int64_t)tile * 128, stop);
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t col = v0 + r * 16 + 4 * kq;
      if constexpr (DZ == 1) {
        uint32_t m[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          m[q] = 0;
#pragma unroll
          for (int t = 0; t < TB; ++t) m[q] = max(m[q], __float_as_uint(fabsf(f[t][r][q])));
          m[q] = max(max_of16(m[q]), stop[wave * 32 + r * 16 + 4 * kq + q]);
        }
        few_lift<TB>(dz, col, m, fr, [&](int t, int q) -> float& { return f[t][r][q]; });
      }
#pragma unroll
      for (int t = 0; t < TB; ++t) few_dz<DZ>(dz, t * 16 + fr, col, f[t][r]);
    }
    few_dz_zero(dz, 16 * TB, (int64_t)tile * 128, 128);
    if constexpr (F32 && DZ == 1) few_put_top(dz, top);
    return;
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    float z[2][4], m = -INFINITY;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        z[r][q] = v0 + r * 16 + 4 * kq + q < g.V ? acc[t][r][q] * g.c2 : -INFINITY;
        m = fmaxf(m, z[r][q]);
      }
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const float ref = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) s += __builtin_amdgcn_exp2f(z[r][q] - ref);
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (kq == 0) red[wave][t * 16 + fr] = make_float2(m, s);
  }
  __syncthreads();
  const int x = threadIdx.x;
  if (x < 16 * TB && x0 + x < g.n) {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, red[w][x].x);
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < 4; ++w) s += red[w][x].y * __builtin_amdgcn_exp2f(red[w][x].x - ref);
    g.part[(int64_t)tile * g.n + x0 + x] = make_float2(m, s);
  }
}

// The same where the table is short too and blocks of 128 rows would leave most
// of the chip idle: a block has 32 rows, its four waves share K and their sums
// meet in LDS, so a chain of loads is a quarter as long. Fragments of the tokens
// come straight from memory here. DZ: leaves dz (rows_pad rows, zeros behind the
// tokens and behind the table) instead of maxima and sums.
template <typename T, int TB, int DZ>
__global__ __launch_bounds__(256, sizeof(T) == 4 && TB == 4 ? 1 : 2) void head_few_split_kernel(
    FewArgs g, FewDz z) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int ST = F32 ? 2 : 4, P = F32 ? 3 : 1, KC = 32 * ST;
  static_assert(DZ == 0 || (DZ == 1) == F32, "dz of fp32 operands is fp16");
  __shared__ f32x4_t join[4][TB * 2][64];
  __shared__ uint32_t stop[DZ == 1 ? 32 : 1];
  FewStops stops;
  if constexpr (DZ == 1) stops.start(z);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, kq = lane >> 4;
  const int64_t v0 = (int64_t)blockIdx.x * 32;
  const T *wp[2], *hp[TB];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t v = v0 + r * 16 + fr;
    wp[r] = static_cast<const T*>(g.table) + (v < g.V ? v : g.V - 1) * g.d + kq * 8;
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int64_t x = t * 16 + fr;
    hp[t] = static_cast<const T*>(g.h) + (x < g.n ? x : g.n - 1) * g.ld + kq * 8;
  }
  f32x4_t acc[TB][2] = {};
  float top = 0.f;
  struct Step {
    Raw8<T> w[2], h[TB];
  };
  auto load = [&](int k, Step (&to)[ST]) {
    const bool all = k + KC <= g.d;
    auto left = [&](int s) { return all ? 8 : g.d - k - s * 32 - kq * 8; };
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int s = 0; s < ST; ++s) to[s].w[r] = load8(wp[r] + k + s * 32, left(s));
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int s = 0; s < ST; ++s) to[s].h[t] = load8(hp[t] + k + s * 32, left(s));
  };
  auto multiply = [&](const Step (&x)[ST]) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      uint4 wf[2][P];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        planes_of(x[s].w[r], wf[r]);
        if constexpr (F32 && DZ == 1) top = few_top(x[s].w[r], top);
      }
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        uint4 hf[P];
        planes_of(x[s].h[t], hf);
#pragma unroll
        for (int r = 0; r < 2; ++r) mma_planes(wf[r], hf, acc[t][r]);
      }
    }
  };
  Step x[2][ST];
  int k = wave * KC;
  if (k < g.d) load(k, x[0]);
  for (; k < g.d; k += 8 * KC) {
    if (k + 4 * KC < g.d) load(k + 4 * KC, x[1]);
    multiply(x[0]);
    if (k + 4 * KC < g.d) {
      if (k + 8 * KC < g.d) load(k + 8 * KC, x[0]);
      multiply(x[1]);
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) join[wave][t * 2 + r][lane] = acc[t][r];
  __syncthreads();
  // wave t has token block t from here on: rows 16 r + 4 kq + q, token 16 t + fr
  const int64_t tok = wave * 16 + fr;
  float v[2][4], m = -INFINITY;
  if (wave < TB) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const f32x4_t sum = (join[0][wave * 2 + r][lane] + join[1][wave * 2 + r][lane]) +
                          (join[2][wave * 2 + r][lane] + join[3][wave * 2 + r][lane]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[r][q] = v0 + r * 16 + 4 * kq + q < g.V ? sum[q] * g.c2 : -INFINITY;
        m = fmaxf(m, v[r][q]);
      }
    }
    if constexpr (DZ == 0) {
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float ref = m == -INFINITY ? 0.f : m;
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) s += __builtin_amdgcn_exp2f(v[r][q] - ref);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (kq == 0 && tok < g.n) g.part[(int64_t)blockIdx.x * g.n + tok] = make_float2(m, s);
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) few_exp(z, tok, g.n, v[r]);
    }
  }
  if constexpr (DZ == 1) {
    // the token blocks' largest meet where the sparse positions' are
    stops.template join<32>(z, v0, stop);
    if (wave < TB)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t m4 = max_of16(__float_as_uint(fabsf(v[r][q])));
          if (fr == 0) atomicMax(stop + r * 16 + 4 * kq + q, m4);
        }
    __syncthreads();
    if (wave < TB)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t m4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) m4[q] = stop[r * 16 + 4 * kq + q];
        few_lift<1>(z, v0 + r * 16 + 4 * kq, m4, fr, [&](int, int q) -> float& { return v[r][q]; });
      }
  }
  if constexpr (DZ != 0) {
    if (wave < TB)
#pragma unroll
      for (int r = 0; r < 2; ++r) few_dz<DZ>(z, tok, v0 + r * 16 + 4 * kq, v[r]);
    few_dz_zero(z, 16 * TB, v0, 32);
  }
  if constexpr (F32 && DZ == 1) few_put_top(z, top);
}

}  // namespace
}  // namespace pg
