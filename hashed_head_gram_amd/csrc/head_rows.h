// Row kernels of the head's losses: joining the tiles along the vocabulary, the
// teacher's shares, what the backward pass needs of each row, operand copies,
// sparse positions and the sums of split products.
#pragma once

#include "head_few.h"

namespace pg {
namespace {

// ---------------------------------------------------------------------------
// Rows

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// Dot product of two rows of d elements by one wave, in every lane.
template <typename T>
__device__ __forceinline__ float row_dot(const T* x, const T* y, int d, int lane) {
  float s = 0.f;
  int c = lane * 8;
#pragma unroll 4
  for (; c + 8 <= d; c += 512) {
    const Raw8<T> a = load8(x + c, 8), b = load8(y + c, 8);
#pragma unroll
    for (int u = 0; u < 8; ++u) s = fmaf(a.get(u), b.get(u), s);
  }
  if (c < d) {
    const Raw8<T> a = load8(x + c, d - c), b = load8(y + c, d - c);
#pragma unroll
    for (int u = 0; u < 8; ++u) s = fmaf(a.get(u), b.get(u), s);
  }
  return wave_sum(s);
}

constexpr int kMaxK = 256;                 // teacher's entries a token
constexpr int kPer = kMaxK / 64;           // of them a lane

// The teacher's shares of a row by one wave: q[u] belongs to entry lane + 64 u,
// 0 where there is none. Returns the sum of q log q; any: an entry has weight.
// Differences before the division by the temperature: what is divided may leave
// fp32's range, and they are exact between close values.
__device__ __forceinline__ float teacher_shares(const int32_t* ids, const float* t, int k,
                                                int64_t V, float inv_tau, int lane, int (&id)[kPer],
                                                float (&q)[kPer], bool& any) {
  float m = -INFINITY, x[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int j = lane + 64 * u;
    id[u] = j < k ? ids[j] : -1;
    if (id[u] < 0 || id[u] >= V) id[u] = -1;
    x[u] = id[u] >= 0 ? t[j] : -INFINITY;
    m = fmaxf(m, x[u]);
  }
  m = wave_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    q[u] = id[u] >= 0 ? expf((x[u] - ref) * inv_tau) : 0.f;
    s += q[u];
  }
  s = wave_sum(s);
  any = !(s == 0.f);
  float e = 0.f;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    if (any) q[u] /= s;
    if (q[u] != 0.f) e += q[u] * logf(q[u]);
  }
  return wave_sum(e);
}

// Joins the tiles' maxima and sums along the vocabulary and forms the losses:
// blocks of R rows by NT threads, NT / R threads a row for the join, whole waves
// a row for the dot products that its targets name. Sixteen rows by 1024 threads,
// or, where there are few, one by 256.
struct JoinArgs {
  const float2* part;
  int64_t parts;
  int64_t n;
  int d;
  const void* h;
  int64_t ld;
  const void* table;
  int64_t V;
  float scale, inv_tau;
  const int32_t* ids;      // [n][k] (cross entropy: k = 1)
  const float* teacher;    // nullable: cross entropy
  int k;
  int picked;              // logits holds z already
  float *loss, *lse, *logits;
};
template <typename T, int kJoinRows, int NT>
__global__ __launch_bounds__(NT) void head_join_kernel(JoinArgs g) {
  constexpr int NW = NT / 64, WR = NW / kJoinRows;   // waves, and of them a row
  __shared__ float2 red[NW][kJoinRows];
  __shared__ float lse_s[kJoinRows];
  __shared__ float zs[kJoinRows][kMaxK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * kJoinRows;
  // dot products
  const int r = wave / WR;
  const int64_t row = r0 + r;
  if (row < g.n && g.picked) {
    for (int j = wave % WR * 64 + lane; j < g.k; j += WR * 64) {
      const int id = g.ids[row * g.k + j];
      zs[r][j] = id >= 0 && id < g.V ? g.logits[row * g.k + j] : 0.f;
    }
  } else if (row < g.n) {
    const T* hr = static_cast<const T*>(g.h) + row * g.ld;
    const T* tab = static_cast<const T*>(g.table);
    for (int j = wave % WR; j < g.k; j += WR) {
      const int id = g.ids[row * g.k + j];
      float z = 0.f;
      if (id >= 0 && id < g.V) z = g.scale * row_dot(hr, tab + (int64_t)id * g.d, g.d, lane);
      if (lane == 0) zs[r][j] = z;
    }
  }
  {
    const int rr = tid % kJoinRows;
    const int64_t jr = r0 + rr < g.n ? r0 + rr : g.n - 1;
    float m = -INFINITY, s = 0.f;
#pragma unroll 4
    for (int64_t p = tid / kJoinRows; p < g.parts; p += NT / kJoinRows) {
      const float2 v = g.part[p * g.n + jr];
      const float hi = fmaxf(m, v.x), ref = hi == -INFINITY ? 0.f : hi;
      s = s * __builtin_amdgcn_exp2f(m - ref) + v.y * __builtin_amdgcn_exp2f(v.x - ref);
      m = hi;
    }
#pragma unroll
    for (int o = kJoinRows; o < 64; o <<= 1) {
      const float om = __shfl_xor(m, o), os = __shfl_xor(s, o);
      const float hi = fmaxf(m, om), ref = hi == -INFINITY ? 0.f : hi;
      s = s * __builtin_amdgcn_exp2f(m - ref) + os * __builtin_amdgcn_exp2f(om - ref);
      m = hi;
    }
    if (lane < kJoinRows) red[wave][lane] = make_float2(m, s);
  }
  __syncthreads();
  if (tid < kJoinRows) {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, red[w][tid].x);
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += red[w][tid].y * __builtin_amdgcn_exp2f(red[w][tid].x - ref);
    // log(s 2^m)
    const float l = (m + log2f(s)) * kLn2;
    lse_s[tid] = l;
    if (r0 + tid < g.n) g.lse[r0 + tid] = l;
  }
  __syncthreads();
  if (wave % WR || row >= g.n) return;
  const float l = lse_s[r];
  if (!g.teacher) {
    // The sum is never below one of its terms; of a certain token the two, summed
    // in different orders, may come out the other way round (NaN stays).
    const int id = g.ids[row];
    const float x = id >= 0 && id < g.V ? l - zs[r][0] : 0.f;
    if (lane == 0) g.loss[row] = x < 0.f ? 0.f : x;
    return;
  }
  int id[kPer];
  float q[kPer];
  bool any;
  const float ent = teacher_shares(g.ids + row * g.k, g.teacher + row * g.k, g.k, g.V, g.inv_tau,
                                   lane, id, q, any);
  float x = 0.f;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int j = lane + 64 * u;
    if (j < g.k) {
      g.logits[row * g.k + j] = zs[r][j];
      if (q[u] != 0.f) x += q[u] * (l - zs[r][j] * g.inv_tau);
    }
  }
  x = wave_sum(x);
  // (the square may leave fp32's range)
  if (lane == 0) g.loss[row] = any ? (ent + x) / g.inv_tau / g.inv_tau : 0.f;
}

// Sorts the entries of each row tile by column tile: a block a row tile, counts,
// a running sum, places. The order inside a tile is free: every entry has a
// place of its own to write to. Fetched as dot products of their own, 8,192
// tokens' 64 entries at width 2,560 took 520 of 4,900 us; sorted, 18, and picked
// from the tiles' accumulators.
constexpr int kMostTiles = 8192;
__global__ __launch_bounds__(1024) void head_bin_kernel(const int32_t* ids, int64_t n, int k,
                                                        int64_t V, int b, int tiles, int64_t cap,
                                                        uint32_t* list, int* starts) {
  __shared__ int count[kMostTiles];
  __shared__ int part[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * b;
  const int total = (int)((n - r0 < b ? n - r0 : b) * k);
  const int shift = b == 256 ? 8 : 7;
  for (int i = tid; i < tiles; i += 1024) count[i] = 0;
  __syncthreads();
  const int32_t* src = ids + r0 * k;
  for (int i = tid; i < total; i += 1024) {
    const int id = src[i];
    if (id >= 0 && id < V) atomicAdd(&count[id >> shift], 1);
  }
  __syncthreads();
  int* out = starts + (int64_t)blockIdx.x * (tiles + 1);
  int base = 0;
  for (int t0 = 0; t0 < tiles; t0 += 1024) {         // exclusive running sum
    const int v = t0 + tid < tiles ? count[t0 + tid] : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    if (lane == 63) part[wave] = x;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += part[w];
      all += part[w];
    }
    if (t0 + tid < tiles) {
      count[t0 + tid] = before + x - v;
      out[t0 + tid] = before + x - v;
    }
    base += all;
    __syncthreads();
  }
  if (tid == 0) out[tiles] = base;
  for (int i = tid; i < total; i += 1024) {
    const int id = src[i];
    if (id >= 0 && id < V) {
      const int row = i / k;
      list[blockIdx.x * cap + atomicAdd(&count[id >> shift], 1)] =
          (uint32_t)row | ((uint32_t)(id & (b - 1)) << 8) | ((uint32_t)(i - row * k) << 16);
    }
  }
}

// ---------------------------------------------------------------------------
// Operand copies

__device__ __forceinline__ int wave_imax(int v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, __shfl_xor(v, o));
  return v;
}
// Largest of n exponents, in every thread of a block of 256.
__device__ __forceinline__ int block_exponent(const int* part, int n, int* sh) {
  int e = kNone;
  for (int i = threadIdx.x; i < n; i += 256) e = max(e, part[i]);
  e = wave_imax(e);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = e;
  __syncthreads();
  e = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
  __syncthreads();
  return e;
}
// 2^this brings a value of exponent e to 2^kTop.
__device__ __forceinline__ int placement(int e) { return e == kNone ? 0 : kTop - e; }

template <typename T>
__device__ __forceinline__ int exponent_of8(const T* p, int left) {
  const Raw8<T> v = load8(p, left);
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float a = fabsf(v.get(u));
    if (a < INFINITY) m = fmaxf(m, a);               // NaN and infinity aside
  }
  return exponent_of(m);
}

// src[c .. c + 8) times 2^e as fp16 halves (zeros behind d, or all zeros).
template <typename T>
__device__ __forceinline__ void put_halves(const T* src, int d, int c, bool keep, int e,
                                           uint16_t* dst, int64_t plane) {
  float x[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) x[u] = 0.f;
  if (keep && c < d) {
    const Raw8<T> v = load8(src + c, d - c);
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = ldexpf(v.get(u), e);
  }
  uint32_t w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = pack2_f16(x[2 * u], x[2 * u + 1]);
  *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      w[u] = pack2_f16(x[2 * u] - lo_f16(w[u]), x[2 * u + 1] - hi_f16(w[u]));
    *reinterpret_cast<uint4*>(dst + plane + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void put_raw(const uint16_t* src, int d, int c, bool keep,
                                        uint16_t* dst) {
  Raw8<uint16_t> v{};
  if (keep && c < d) v = load8(src + c, d - c);
  *reinterpret_cast<uint4*>(dst + c) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

// Tokens up to which the forward pass reads the table by fragments, a group of 64
// after the other: bf16 that tiles can read in place (65 tokens of 128,000 x 2560:
// 161 us by tiles, 213 by two groups), bf16 that they cannot (385 wide: 53 us for
// 128, 60 by tiles), fp32, which tiles need split and placed (320 tokens: 1,228 us,
// 1,600 by tiles; 512: 1,902 and 1,670)
constexpr int kFew = 64, kFewOdd = 128, kFewF32 = 320;
// and rows of the table up to which they are read 32 a block, one block a compute
// unit (2048 wide, 32 tokens: 15 us for 23 at 8,192 rows, 26 for 24 at 16,384)
constexpr int64_t kFewShort = 8192;
// Tokens up to which bf16 tables are used as they are for dh too: dz is then two
// bf16 halves (16 bits), two products for one, and the fp16 copies, three more
// passes over the table, fall away (65,536 rows of 2048, 8 tokens: 295 us; a fifth
// more with them).
constexpr int kWide = 256;
constexpr int kScanBlocks = 512;
static_assert(kTops <= kScanBlocks, "they share part_w");
constexpr int kRowBlocks = 2048;           // most blocks over rows, four waves each

// What all row kernels know of a call's rows (row pieces: of the piece).
struct RowArgs {
  const void* h;
  int64_t ld;
  int64_t n, rows_pad, vec_pad;
  int d, dp;
  const void* table;
  int64_t V;
  float scale, inv_tau;
  const int32_t* ids;
  const float *teacher, *logits;    // distillation
  int k;
  const float *lse, *dloss, *dlse;
  float *a, *lse2, *rowf;
  int* row_exp;                     // dz's rows hold 2^-row_exp times their values; kNone: zeros
  int32_t* sidx;
  float* sval;
  int *part_h, *part_w;             // exponents by block: of 2^row_exp h, of T
  int *all_h, *all_w;               // what dT and dh undo: minus their placements
  int nparts_h, nparts_w;
  int clear_w;                      // start part_w: a later kernel raises it
  uint32_t* stop;                   // largest |sval| by vocabulary row, as bits of fp32 (nullable)
  int* clear;                       // cleared by the first kernel
  int64_t nclear;
  int placed;                       // dz in fp16, placed by powers of two; 0: two bf16 halves
  uint16_t *hp, *hz;                // fp16 h for dT; h for the logits (NULL: read in place)
  float c2;
};

// First kernel of the backward pass. The first `row_blocks` blocks, a wave a
// row: the weight a of the row's softmax (with scale), its lse in base 2, the
// gradient at its sparse positions, and the placement of its dz. The others:
// the exponent of T's largest element (with clear_w there are none).
template <typename T>
__global__ __launch_bounds__(256) void head_stats_kernel(RowArgs g, int row_blocks) {
  __shared__ int sh[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int top = kNone;
  if ((int)blockIdx.x >= row_blocks) {
    const int64_t count = g.V * g.d, step = (int64_t)(gridDim.x - row_blocks) * 2048;
    const T* t = static_cast<const T*>(g.table);
#pragma unroll 4
    for (int64_t i = ((int64_t)blockIdx.x - row_blocks) * 2048 + threadIdx.x * 8; i < count;
         i += step)
      top = max(top, exponent_of8(t + i, (int)(count - i < 8 ? count - i : 8)));
  } else {
    if (g.clear_w && blockIdx.x == 0)
      for (int i = threadIdx.x; i < g.nparts_w; i += 256) g.part_w[i] = kNone;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < g.nclear; i += row_blocks * 256)
      g.clear[i] = 0;
    for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < g.vec_pad; row += row_blocks * 4) {
      const T* hr = static_cast<const T*>(g.h) + row * g.ld;
      float a = 0.f, l2 = 0.f, w = 0.f;
      int e = kNone, re = kNone;
      if (row < g.n) {
        const float l = g.lse[row], dl = g.dloss[row];
        l2 = l * kLog2e;
        int id[kPer];
        float q[kPer];
        bool valid;
        if (!g.teacher) {
          id[0] = g.ids[row];
          valid = id[0] >= 0 && id[0] < g.V;
          w = valid ? g.scale * dl : 0.f;
          a = w + (g.dlse ? g.scale * g.dlse[row] : 0.f);
        } else {
          teacher_shares(g.ids + row * g.k, g.teacher + row * g.k, g.k, g.V, g.inv_tau, lane, id,
                         q, valid);
          a = w = valid ? dl * g.scale / g.inv_tau : 0.f;
        }
        // a NaN weight stays one
        const bool keep = !(a == 0.f && w == 0.f);
        if (keep) {
          const float bound = fabsf(a) + fabsf(w);
          re = g.placed && exponent_of(bound) != kNone ? exponent_of(bound) - kTop : 0;
          if (g.placed) {
            for (int c = lane * 8; c < g.d; c += 512) e = max(e, exponent_of8(hr + c, g.d - c));
            e = wave_imax(e);
            if (e != kNone) top = max(top, e + re);
          }
        }
        const int place = keep ? -re : 0;
        if (!g.teacher) {
          float val = 0.f;
          if (valid && keep) {
            const T* t = static_cast<const T*>(g.table) + (int64_t)id[0] * g.d;
            const float z = g.scale * row_dot(hr, t, g.d, lane);
            val = ldexpf(a, place) * __builtin_amdgcn_exp2f((z - l) * kLog2e);
            val = (a == 0.f ? 0.f : val) - ldexpf(w, place);
          }
          if (lane == 0) {
            g.sidx[row] = valid && keep ? id[0] : -1;
            g.sval[row] = val;
          }
        } else {
          // an id named more than once: its first entry carries the sum
          float sum[kPer];
          bool first[kPer];
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            sum[u] = 0.f;
            first[u] = id[u] >= 0;
          }
          for (int j = 0; j < g.k; ++j) {
            int oid = 0;
            float oq = 0.f;
#pragma unroll
            for (int u = 0; u < kPer; ++u)
              if ((j >> 6) == u) {
                oid = __shfl(id[u], j & 63);
                oq = __shfl(q[u], j & 63);
              }
#pragma unroll
            for (int u = 0; u < kPer; ++u)
              if (oid >= 0 && id[u] == oid) {
                sum[u] += oq;
                if (j < lane + 64 * u) first[u] = false;
              }
          }
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int j = lane + 64 * u;
            if (j < g.k) {
              const bool put = first[u] && keep;
              const float p = __builtin_amdgcn_exp2f(
                  (g.logits[row * g.k + j] * g.inv_tau - l) * kLog2e);
              g.sidx[row * g.k + j] = put ? id[u] : -1;
              g.sval[row * g.k + j] = put ? ldexpf(w, place) * (p - sum[u]) : 0.f;
            }
          }
        }
        a = ldexpf(a, place);
      }
      if (lane == 0) {
        g.a[row] = a;
        g.lse2[row] = l2;
        g.row_exp[row] = re;
      }
      if constexpr (sizeof(T) == 2)
        if (!g.placed && row < g.rows_pad)           // h for dT, zeros in rows without weight
          for (int c = lane * 8; c < g.dp; c += 512)
            put_raw(row < g.n ? hr : static_cast<const T*>(g.h), g.d, c, re != kNone,
                    g.hp + row * g.dp);
    }
  }
  top = wave_imax(top);
  if (lane == 0) sh[wave] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    top = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
    if ((int)blockIdx.x < row_blocks) g.part_h[blockIdx.x] = top;
    else g.part_w[blockIdx.x - row_blocks] = top;
  }
}

// Exponent of the largest element, for the forward pass of fp32 operands.
template <typename T>
__global__ __launch_bounds__(256) void head_scan_kernel(const T* t, int64_t count, int* part) {
  __shared__ int sh[4];
  int top = kNone;
#pragma unroll 4
  for (int64_t i = (int64_t)blockIdx.x * 2048 + threadIdx.x * 8; i < count;
       i += (int64_t)gridDim.x * 2048)
    top = max(top, exponent_of8(t + i, (int)(count - i < 8 ? count - i : 8)));
  top = wave_imax(top);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
}

// Copies of the operands. The first `row_blocks` blocks, a wave a row of h: for
// the logits (hz: fp16 halves placed by the row's own largest element, or bf16
// as it is) and for dT (hp). The others: rows of a piece of T, as fp16 (wp) and,
// where the logits cannot read it in place, as bf16 (wz). Zeros behind d and
// behind the rows.
struct PieceArgs {
  const void* src;
  int64_t rows, rows_pad;
  uint16_t *wp, *wz;
  const uint8_t* level;    // by row, of columns that dz has already (nullable)
  const int* any;          // whether some of them are lifted
};

template <typename T>
__global__ __launch_bounds__(256) void head_copy_kernel(RowArgs g, PieceArgs w, int row_blocks) {
  __shared__ int sh[4];
  constexpr bool F32 = sizeof(T) == 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool scaled = g.nparts_w > 0;
  const int pw = scaled ? placement(block_exponent(g.part_w, g.nparts_w, sh)) : 0;
  if ((int)blockIdx.x >= row_blocks) {
    const int per = g.dp / 8;
    const int64_t total = w.rows_pad * per, step = (int64_t)(gridDim.x - row_blocks) * 256;
    const uint8_t* level = w.level && *w.any ? w.level : nullptr;
    for (int64_t i = ((int64_t)blockIdx.x - row_blocks) * 256 + threadIdx.x; i < total; i += step) {
      const int64_t r = i / per;
      const int c = (int)(i - r * per) * 8;
      const bool in = r < w.rows;
      const T* src = static_cast<const T*>(w.src) + (in ? r : 0) * g.d;
      if (w.wp) {
        const int l = level && level[r] != kEmpty ? level[r] : kFlat;
        put_halves(src, g.d, c, in, pw - l, w.wp + r * g.dp, w.rows_pad * g.dp);
      }
      if constexpr (!F32)
        if (w.wz) put_raw(src, g.d, c, in, w.wz + r * g.dp);
    }
    return;
  }
  if (g.stop) {
    // the columns' largest |dz| at sparse positions, up to where a column is flat:
    // that value is stored, whichever store or maximum comes last
    const int64_t total = g.n * g.k;
    const uint32_t flat = (uint32_t)(127 + kRare) << 23;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += row_blocks * 256) {
      const int id = g.sidx[i];
      if (id < 0) continue;
      const uint32_t x = __float_as_uint(g.sval[i]) & 0x7FFFFFFFu;
      if (x >= flat) g.stop[id] = flat;
      else if (x > 0) atomicMax(g.stop + id, x);
    }
  }
  int ph = 0;
  if (g.hp) ph = placement(block_exponent(g.part_h, g.nparts_h, sh));
  if (blockIdx.x == 0 && threadIdx.x == 0 && g.hp) {
    *g.all_h = -ph;
    *g.all_w = -pw;
  }
  for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < g.vec_pad; row += row_blocks * 4) {
    const bool in = row < g.n;
    const T* src = static_cast<const T*>(g.h) + (in ? row : 0) * g.ld;
    if constexpr (F32) {
      // the logits' copy, and the factor that undoes its placement
      if (g.hz) {
        int e = kNone;
        if (in) {
          for (int c = lane * 8; c < g.d; c += 512) e = max(e, exponent_of8(src + c, g.d - c));
          e = wave_imax(e);
        }
        const int p = placement(e);
        // (where the largest elements of h and T never meet, the power may leave
        // fp32's range; the products it scales are zeros then)
        if (lane == 0) {
          const float f = ldexpf(g.c2, -p - pw);
          g.rowf[row] = fminf(fmaxf(f, -3.4028235e38f), 3.4028235e38f);
        }
        if (row < g.rows_pad)
          for (int c = lane * 8; c < g.dp; c += 512)
            put_halves(src, g.d, c, in, p, g.hz + row * g.dp, g.rows_pad * g.dp);
      }
    } else {
      if (g.hz && row < g.rows_pad)
        for (int c = lane * 8; c < g.dp; c += 512) put_raw(src, g.d, c, in, g.hz + row * g.dp);
    }
    if (g.hp && row < g.rows_pad) {
      const int re = in ? g.row_exp[row] : kNone;
      const bool keep = re != kNone;                 // rows without weight add zeros
      for (int c = lane * 8; c < g.dp; c += 512)
        put_halves(src, g.d, c, keep, keep ? ph + re : 0, g.hp + row * g.dp, g.rows_pad * g.dp);
    }
  }
}

// dz of a piece between its tiles and its products.
struct DzArgs {
  const int32_t* sidx;
  const float* sval;
  int64_t n, rows;         // tokens, rows of dz
  int k;
  int64_t v0, cols;        // first vocabulary row, columns without padding
  uint16_t* dz;
  int64_t ldz, plane;      // columns; elements between halves
  int planes, f16;
  // fp16: levels by group of rows and column
  const uint8_t* level;
  int group, groups;       // rows of a group, how many
  const int* any;
  int* col_exp;            // [ldz] where any: what dT's rows undo, minus the columns' own level
  uint16_t* wp;            // [ldz][dp] T's copy, its halves `wplane` elements apart
  int dp;
  int64_t wplane;
};

// Writes the sparse positions over dz, each at the level of its group, whose
// largest value they were counted in. The first `col_blocks` blocks: the columns'
// own levels, the lowest of their groups.
__global__ __launch_bounds__(256) void head_sparse_kernel(DzArgs g, int col_blocks) {
  if ((int)blockIdx.x < col_blocks) {
    if (*g.any == 0) return;
    for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < g.ldz; v += col_blocks * 256) {
      int l = kEmpty;
#pragma unroll 8
      for (int i = 0; i < g.groups; ++i) l = min(l, (int)g.level[i * g.ldz + v]);
      g.col_exp[v] = l == kEmpty ? 0 : -l;
    }
    return;
  }
  const int64_t total = g.n * g.k, step = (int64_t)(gridDim.x - col_blocks) * 256;
  for (int64_t i = ((int64_t)blockIdx.x - col_blocks) * 256 + threadIdx.x; i < total; i += step) {
    const int64_t v = (int64_t)g.sidx[i] - g.v0;
    if (v < 0 || v >= g.cols) continue;
    const int64_t row = i / g.k;
    float x = g.sval[i];
    if (g.f16) {
      const int l = g.level[row / g.group * g.ldz + v];
      if (l != kEmpty) x = ldexpf(x, l);
    }
    uint16_t* p = g.dz + row * g.ldz + v;
    const uint32_t w = g.f16 ? pack2_f16(x, 0.f) : pack2_bf16(x, 0.f);
    *p = (uint16_t)w;
    const float left = x - (g.f16 ? lo_f16(w) : __uint_as_float(w << 16));
    if (g.planes > 1) p[g.plane] = (uint16_t)(g.f16 ? pack2_f16(left, 0.f) : pack2_bf16(left, 0.f));
  }
}

// Eight fp16 numbers and their low halves (zeros where there are none) times 2^e[i].
__device__ __forceinline__ void scale_halves(uint4& hi, uint4& lo, const int (&e)[8]) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
  uint32_t w[4], r[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float x = ldexpf(lo_f16(h[u]) + lo_f16(l[u]), e[2 * u]);
    const float y = ldexpf(hi_f16(h[u]) + hi_f16(l[u]), e[2 * u + 1]);
    w[u] = pack2_f16(x, y);
    r[u] = pack2_f16(x - lo_f16(w[u]), y - hi_f16(w[u]));
  }
  hi = make_uint4(w[0], w[1], w[2], w[3]);
  lo = make_uint4(r[0], r[1], r[2], r[3]);
}
// N of them, `step` elements apart, those from `count` on left alone.
template <int N>
__device__ __forceinline__ void scale_at(uint16_t* p, int64_t step, int64_t plane, int planes,
                                         int count, const int (&e)[8]) {
  uint4 hi[N], lo[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    hi[i] = lo[i] = make_uint4(0, 0, 0, 0);
    if (i < count) {
      hi[i] = *reinterpret_cast<const uint4*>(p + i * step);
      if (planes > 1) lo[i] = *reinterpret_cast<const uint4*>(p + i * step + plane);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    scale_halves(hi[i], lo[i], e);
    if (i < count) {
      *reinterpret_cast<uint4*>(p + i * step) = hi[i];
      if (planes > 1) *reinterpret_cast<uint4*>(p + i * step + plane) = lo[i];
    }
  }
}

// Where columns are lifted and dz has more than one group: their groups of rows to
// their own level, and T's rows in the copy for dh down by as much. The first `dz_blocks` blocks take dz, 256 columns
// of a group at a time. One load a block where nothing is lifted (5 us); all of
// 16,384 x 25,152 columns read and written in 340 us, 4.8 TB/s.
__global__ __launch_bounds__(256) void head_level_kernel(DzArgs g, int dz_blocks) {
  if (*g.any == 0) return;
  if ((int)blockIdx.x < dz_blocks) {
    const int64_t chunks = (g.ldz + 255) / 256;
    for (int64_t i = blockIdx.x; i < chunks * g.groups; i += dz_blocks) {
      const int64_t grp = i / chunks, col = (i - grp * chunks) * 256 + (threadIdx.x & 31) * 8;
      if (col >= g.ldz) continue;
      int e[8];
      bool some = false;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int l = g.level[grp * g.ldz + col + u];
        e[u] = l == kEmpty ? 0 : -g.col_exp[col + u] - l;
        some |= e[u] != 0;
      }
      if (!some) continue;
      const int64_t end = (grp + 1) * g.group < g.rows ? (grp + 1) * g.group : g.rows;
      for (int64_t r = grp * g.group + (threadIdx.x >> 5); r < end; r += 32)
        scale_at<4>(g.dz + r * g.ldz + col, 8 * g.ldz, g.plane, g.planes, (int)((end - r + 7) / 8),
                    e);
    }
    return;
  }
  const int per = g.dp / 8;
  const int64_t total = g.ldz * per, step = (int64_t)(gridDim.x - dz_blocks) * 256;
  for (int64_t i = ((int64_t)blockIdx.x - dz_blocks) * 256 + threadIdx.x; i < total; i += step) {
    const int64_t v = i / per;
    const int x = g.col_exp[v];
    if (x == 0) continue;
    const int e[8] = {x, x, x, x, x, x, x, x};
    scale_at<1>(g.wp + v * g.dp + (i - v * per) * 8, 0, g.wplane, g.planes, 1, e);
  }
}

// Sums the results of K's splits in order, adds prev, and stores: two products.
struct SumArgs {
  const float* part;
  int splits;
  int64_t stride, ld_part;             // elements
  int64_t M, N;
  const float* prev;
  int64_t ld_prev;
  void* out;
  int64_t ld_out;
  int out_bf16;
};
__global__ __launch_bounds__(256) void head_sum_kernel(SumArgs a, SumArgs b, int na) {
  // 32 groups of four columns a block; eight threads a group take every eighth
  // split (one thread took 66 us for 180 splits of 32 x 59)
  __shared__ float4 sh[8][32];
  const bool first = (int)blockIdx.x < na;
  const SumArgs& g = first ? a : b;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t per = (g.N + 3) / 4, total = g.M * per;
  const int64_t step = (int64_t)(first ? na : (int)gridDim.x - na) * 32;
  for (int64_t i0 = ((int64_t)blockIdx.x - (first ? 0 : na)) * 32; i0 < total; i0 += step) {
    const int64_t i = i0 + x;
    const int64_t row = i / per, col = (i - row * per) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < total) {
      const float* p = g.part + row * g.ld_part + col;   // rows of whole tiles
#pragma unroll 4
      for (int s = y; s < g.splits; s += 8) {
        const float4 t = *reinterpret_cast<const float4*>(p + s * g.stride);
        v.x += t.x;
        v.y += t.y;
        v.z += t.z;
        v.w += t.w;
      }
    }
    sh[y][x] = v;
    __syncthreads();
    if (y == 0 && i < total) {
#pragma unroll
      for (int s = 1; s < 8; ++s) {
        const float4 t = sh[s][x];
        v.x += t.x;
        v.y += t.y;
        v.z += t.z;
        v.w += t.w;
      }
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (col + u < g.N) {
          const float r = g.prev ? f[u] + g.prev[row * g.ld_prev + col + u] : f[u];
          if (g.out_bf16)
            static_cast<uint16_t*>(g.out)[row * g.ld_out + col + u] = (uint16_t)pack2_bf16(r, 0.f);
          else
            static_cast<float*>(g.out)[row * g.ld_out + col + u] = r;
        }
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void head_zero_kernel(uint16_t* out, int64_t count) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += step) out[i] = 0;
}

}  // namespace
}  // namespace pg
